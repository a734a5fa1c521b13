"""References of the bf16 shared-prefix decode that move: a row's later tiles exceed the
first one's scores by more than 2^60 and its O is rescaled on the way.

Scores of thousands make a comparison with 64 bits loose: a float32 sum of 576
products errs by up to 576 * 2^-24 sum |q k| scale, which shifts every weight by e to
that. So a call is also compared with itself cut into ranges of one tile: no
reference ever moves there, the ranges are merged in float32, and the scores are the
same bits. The two differ by the roundings of the weights and of x alone, one half
step of bf16 each on either side. The first test, on the CPU, holds that bound
against the formula with O left unscaled.
"""
import math

import pytest
import torch

C, DR = 512, 64
HALF = torch.finfo(torch.bfloat16).eps / 2
TILE, MOVE = 128, 60.0


def _inputs(case, Lp):
    """q (B, H, C + DR), prefix rows, own rows per sequence, in bf16."""
    g = torch.Generator().manual_seed(61)
    r = lambda *s: torch.randn(s, generator=g)
    if case == "own":
        # eight sequences share a block of rows, four in each CTA of its pair; some grow in
        # their second tile, in one of the CTAs alone or in both
        B, H, lens = 8, 16, [10, 300, 129, 0, 260, 1, 300, 200]
        prefix, own = r(Lp, C + DR), [r(n, C + DR) for n in lens]
        for b, f in ((1, 60.0), (2, 40.0), (6, 70.0), (7, 8.0)):
            own[b][128:] *= f
    else:
        # all rows' scores climb twice and fall between
        B, H, lens = 3, 32, [100, 0, 64]
        prefix, own = r(Lp, C + DR), [r(n, C + DR) for n in lens]
        prefix[200:300] *= 40.0
        prefix[300:400] *= 8.0
        prefix[400:] *= 90.0
    return (r(B, H, C + DR) * 0.8).bfloat16(), prefix.bfloat16(), [o.bfloat16() for o in own]


CASES = [("own", 0), ("own", 70), ("climb", 600)]


def _tiles(q, prefix, own, b):
    """The scores (log2 units, float64) and values of a sequence's tiles."""
    qq = q[b].double()
    for src in (prefix, own[b]):
        for t in range(0, len(src), TILE):
            k = src[t:t + TILE].double()
            yield qq @ k.T * (0.07 * math.log2(math.e)), k[:, :C]


def _formula(q, prefix, own, b, rescale=True):
    """The kernel's rule in 64 bits: x, sum_t p_t |v_t|, and how many rows move their reference."""
    H = q.shape[1]
    m, l = torch.full((H,), -math.inf, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
    o, size = torch.zeros(H, C, dtype=torch.float64), torch.zeros(H, C, dtype=torch.float64)
    moved = torch.zeros(H, dtype=torch.bool)
    for s, v in _tiles(q, prefix, own, b):
        top = s.amax(1)
        move = top > m + MOVE
        moved |= move & (m > -math.inf)
        f = torch.where(move & (m > -math.inf), 2.0 ** (m - top), torch.ones_like(m))
        m = torch.where(move, top, m)
        p = 2.0 ** (s - m[:, None])
        l = l * f + p.sum(1)
        o = (o * f[:, None] if rescale else o) + p @ v
        size = size * f[:, None] + p @ v.abs()
    return o / l[:, None], size / l[:, None], moved


def _bound(x, size):
    # a weight's rounding and x's, on either side; the exponentials' 2^-22 and float32 sums far below
    return 2 * HALF * (size + x.abs()) + 2e-5 * size


@pytest.mark.parametrize("case,Lp", CASES)
def test_the_bound_rejects_an_unscaled_o(case, Lp):
    q, prefix, own = _inputs(case, Lp)
    seen = 0
    for b in range(len(own)):
        if Lp + len(own[b]) == 0:
            continue
        x, size, moved = _formula(q, prefix, own, b)
        bad, _, _ = _formula(q, prefix, own, b, rescale=False)
        off = ((bad - x).abs() > _bound(x, size)).any(1)
        assert not off[~moved].any()
        # not all: scores up to 2^60 above a moved reference outweigh what was left unscaled
        if moved.any():
            assert off[moved].float().mean() >= 0.7
        seen += int(moved.sum())
    assert seen >= 16


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("case,Lp", CASES)
def test_references_that_move(case, Lp, splits):
    from latent_kv_decode_b200 import ops
    q, prefix, own = _inputs(case, Lp)
    B, H = q.shape[:2]
    lens = [len(o) for o in own]
    rows = torch.zeros((B, max(lens), C + DR), dtype=torch.bfloat16)
    for b, o in enumerate(own):
        rows[b, :len(o)] = o
    d, p, rows = q[:, :, None].cuda(), prefix.cuda(), rows.cuda()
    per_block = 128 // H                                             # sequences of a block of rows
    ranges = -(-Lp // TILE) + max(sum(-(-n // TILE) for n in lens[b:b + per_block]) for b in range(0, B, per_block))
    call = lambda n: ops.mla_prefix_decode(d[..., :C].contiguous(), d[..., C:].contiguous(), p[:, :C] if Lp else None,
                                           p[:, C:] if Lp else None, rows[..., :C], rows[..., C:], 0.07, num_splits=n,
                                           seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    (x, lse), (y, lse_y) = call(splits), call(ranges)
    for b in range(B):
        got, same = x[b, :, 0].cpu().double(), y[b, :, 0].cpu().double()
        if Lp + lens[b] == 0:
            assert (got == 0).all() and (lse[b] == -math.inf).all()
            continue
        want, size, _ = _formula(q, prefix, own, b)
        assert ((got - same).abs() <= _bound(same, size)).all(), f"sequence {b}"
        # float32 sums of the same scores
        assert ((lse[b] - lse_y[b]).abs() <= 2.0 ** -20 * lse_y[b].abs() + 1e-5).all()
        # against 64 bits, row by row: the scores' own error moves the weights
        k = torch.cat([prefix, own[b]]).double()
        at = 576 * 2.0 ** -24 * (q[b].double().abs() @ k.abs().T).amax(1) * 0.07
        tol = HALF * (size + want.abs()) + (torch.expm1(2 * at)[:, None] + 2e-5) * size
        assert ((got - want).abs() <= tol).all(), f"sequence {b}"
