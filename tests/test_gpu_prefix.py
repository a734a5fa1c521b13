"""GPU parity of mla_prefix_decode (a batch that shares a prefix) against a plain
fp64 evaluation of its formula, sequence by sequence: the concatenation of the
prefix's and the sequence's own rows, the visibility rules, softmax, latent sum.

Tolerances. float32: the harness's 1e-4. bf16 outputs: a weight is rounded once
to bf16 (half a step, at most 2^-8 relative) and x once more:
|dx| <= 2^-8 (sum_t p_t |v_t| + |x|) plus float32 accumulation far below it;
``_oracle`` evaluates that from the fp64 weights. lse is a float32 sum of float32
exponentials over at most 2^17 tokens (pairwise per thread, so a few 2^-24 of
the sum) of scores whose own float32 accumulation over 576 products errs by
576 * 2^-24 * sum |q k| * scale: bounded by 2e-4 for the draws used here.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

C = 512
HALF = torch.finfo(torch.bfloat16).eps / 2     # 2^-8


def _case(B, H, Q, Dr, Lp, lens, *, dtype=torch.bfloat16, page=0, prefix_paged=None, causal=False, mask=None,
          sinks=False, seed=0, Lk=None, pad=0, fill=None, qscale=0.8):
    """Inputs on the GPU. ``fill`` goes into every cache row no query may see."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(dtype)

    prefix_paged = bool(page) if prefix_paged is None else prefix_paged
    W = C + Dr + pad
    Lk = Lk if Lk is not None else max(lens)
    d = dict(B=B, H=H, Q=Q, Dr=Dr, Lp=Lp, lens=lens, causal=causal, scale=1.0 / math.sqrt(128 + Dr), page=page, Lk=Lk)
    d["q_lat"], d["q_pe"] = normal(B, H, Q, C, scale=qscale), normal(B, H, Q, Dr) if Dr else None
    prefix = normal(Lp, W)
    own = [normal(n, W) for n in lens]
    d["mask"] = None if mask is None else torch.as_tensor(mask, dtype=torch.uint8)
    d["sinks"] = torch.randn(H, generator=g) if sinks else None
    d["rows"] = [torch.cat([prefix, o]).double() for o in own]
    junk = 0.0 if fill is None else fill

    def hide(rows, pos0):
        if d["mask"] is not None and fill is not None:
            rows = rows.clone()
            rows[d["mask"][pos0:pos0 + len(rows)] == 0] = fill
        return rows

    prefix, own = hide(prefix, 0), [hide(o, Lp) for o in own]
    need = lambda n: -(-n // page)
    if page:
        total = (need(Lp) if prefix_paged else 0) + sum(map(need, lens)) + 1
        perm = torch.randperm(total, generator=g).to(torch.int32)
        pool = torch.full((total, page, W), junk, dtype=dtype)
        k = 0

        def put(rows, width):
            nonlocal k
            n = need(len(rows))
            t = torch.full((width,), -1, dtype=torch.int32)
            t[:n] = perm[k:k + n]
            for i in range(n):
                part = rows[i * page:(i + 1) * page]
                pool[perm[k + i], :len(part)] = part
            k += n
            return t

        width = max(1, max(map(need, lens)))
        if prefix_paged:
            d["prefix_table"] = put(prefix, max(1, need(Lp)))[:max(1, need(Lp))].cuda()
        d["table"] = torch.stack([put(o, width) for o in own]).cuda()
        pool = pool.cuda()
        d["kv"], d["pe"] = pool[..., :C], pool[..., C:C + Dr]
        if prefix_paged:
            d["pkv"], d["ppe"] = d["kv"], d["pe"]
        d["Lk"] = Lk = width * page
    else:
        own_t = torch.full((B, max(1, Lk), W), junk, dtype=dtype)
        for b, o in enumerate(own):
            own_t[b, :len(o)] = o
        own_t = own_t.cuda()
        d["kv"], d["pe"] = own_t[..., :C], own_t[..., C:C + Dr]
    if not prefix_paged:
        p = prefix.cuda()
        d["pkv"], d["ppe"] = p[:, :C], p[:, C:C + Dr]
    d["dtype"] = dtype
    return d


def _run(d, **kw):
    from latent_kv_decode_b200 import ops
    c = lambda t: None if t is None else t.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    has_own = d["Lk"] > 0
    args = dict(prefix_len=d["Lp"], prefix_table=d.get("prefix_table"),
                seq_lens=torch.tensor(d["lens"], dtype=torch.int32).cuda() if has_own else None,
                block_table=d.get("table"), page_size=d["page"] or 64, causal=d["causal"], causal_mask=c(d["mask"]),
                sinks=c(d["sinks"]), err_flag=err)
    args.update(kw)
    Dr = d["Dr"]
    x, lse = ops.mla_prefix_decode(c(d["q_lat"]), c(d["q_pe"]), d["pkv"] if d["Lp"] else None,
                                   d["ppe"] if d["Lp"] and Dr else None, d["kv"] if has_own else None,
                                   d["pe"] if has_own and Dr else None, d["scale"], **args)
    torch.cuda.synchronize()
    return x, lse, int(err.item())


def _visible(d, b, q):
    n = d["Lp"] + d["lens"][b]
    v = torch.ones(n, dtype=torch.bool)
    if d["mask"] is not None:
        v &= d["mask"][:n] != 0
    if d["causal"]:
        v &= torch.arange(n) <= n - d["Q"] + q
    return v


def _oracle(d):
    """x, lse and the bound on |x - exact| for bf16 outputs, fp64."""
    B, H, Q = d["B"], d["H"], d["Q"]
    x = torch.zeros(B, H, Q, C, dtype=torch.float64)
    lse = torch.full((B, H, Q), -math.inf, dtype=torch.float64)
    bound = torch.zeros_like(x)
    for b in range(B):
        k = d["rows"][b][:, :C + d["Dr"]]
        for q in range(Q):
            v = _visible(d, b, q)
            qq = d["q_lat"][b, :, q].double()
            if d["Dr"]:
                qq = torch.cat([qq, d["q_pe"][b, :, q].double()], -1)
            kk = k[v]
            s = qq @ kk.T * d["scale"]
            if d["sinks"] is not None:
                s = torch.cat([s, d["sinks"].double()[:, None]], 1)
                kk = torch.cat([kk, torch.zeros(1, kk.shape[1], dtype=torch.float64)])
            if s.shape[1] == 0:
                continue
            lse[b, :, q] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[b, :, q, None])
            x[b, :, q] = p @ kk[:, :C]
            bound[b, :, q] = HALF * (p @ kk[:, :C].abs() + x[b, :, q].abs())
    return x, lse, bound


def _check(d, **kw):
    x, lse, err = _run(d, **kw)
    assert err == 0
    xo, lo, bound = _oracle(d)
    fin = torch.isfinite(lo)
    assert torch.equal(torch.isfinite(lse.cpu()), fin)
    if d["dtype"] == torch.float32:
        assert ((x.cpu().double() - xo).abs() <= 1e-4 + 1e-4 * xo.abs()).all()
        assert ((lse.cpu().double() - lo)[fin].abs() <= 1e-4).all()
    else:
        # 2e-5: float32 accumulation and the exponential's own error, on values of order 1
        over = (x.cpu().double() - xo).abs() - (bound + 2e-5)
        assert (over <= 0).all(), f"worst {over.max().item():.3e} over the bound"
        assert ((lse.cpu().double() - lo)[fin].abs() <= 2e-4).all()
    assert (x.cpu()[~fin] == 0).all() and (lse.cpu()[~fin] == -math.inf).all()


SHAPES = [
    # B, H, Q, Lp, own lengths
    (1, 8, 1, 1, [1]),
    (2, 8, 1, 7, [1, 3]),
    (3, 16, 1, 128, [0, 1, 200]),
    (9, 16, 2, 300, [2, 64, 65, 130, 2, 3, 128, 127, 129]),   # three blocks, sequences cut between blocks
    (5, 24, 1, 65, [4, 5, 6, 7, 300]),                        # 120 rows: a ragged block
    (2, 128, 1, 513, [33, 1]),
    (3, 40, 4, 260, [4, 70, 9]),                              # 160 rows per sequence
    (1, 128, 4, 129, [10]),
    (17, 8, 1, 640, list(range(17))),                         # seventeen sequences, two blocks
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("page", [0, 64, 128, 16])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, page, dtype):
    B, H, Q, Lp, lens = shape
    _check(_case(B, H, Q, 64, Lp, lens, dtype=dtype, page=page, causal=Q > 1, seed=B + H, fill=math.nan))


@pytest.mark.parametrize("Dr", [0, 32, 64])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rope_widths(Dr, dtype):
    _check(_case(4, 16, 1, Dr, 200, [3, 130, 0, 64], dtype=dtype, seed=Dr))


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40, 130, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_splits_with_empty_ranges(splits, dtype):
    _check(_case(6, 32, 1, 64, 700, [0, 5, 64, 129, 1, 300], dtype=dtype, seed=splits, sinks=True), num_splits=splits)


@pytest.mark.parametrize("Lp,lens", [(0, [1, 40, 200]), (257, [0, 0, 0]), (0, [0, 0, 0])])
@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_without_prefix_or_own_tokens(Lp, lens, sinks, dtype):
    _check(_case(3, 16, 1, 64, Lp, lens, dtype=dtype, sinks=sinks, seed=3))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_causal_rows_reaching_back_into_the_prefix(dtype):
    # fewer own tokens than queries: the first queries do not see the prefix's last tokens
    _check(_case(4, 8, 4, 64, 130, [0, 1, 3, 4], dtype=dtype, causal=True, seed=5))
    _check(_case(2, 8, 4, 64, 2, [0, 1], dtype=dtype, causal=True, seed=6))      # rows that see nothing


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("fill", [None, math.nan, math.inf])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_mask_over_positions(page, fill, dtype):
    g = np.random.default_rng(7)
    mask = (g.random(300 + 128) < 0.6).astype(np.uint8)
    mask[128:256] = 0                                # a whole tile hidden
    _check(_case(4, 16, 1, 64, 300, [128, 1, 64, 90], dtype=dtype, page=page, mask=mask, fill=fill, seed=8))
    _check(_case(2, 16, 1, 64, 100, [20, 28], dtype=dtype, page=page, mask=np.zeros(428, np.uint8), fill=fill, seed=9))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_sequences_bad_values_stay_with_it(dtype):
    # a non-finite own row makes its sequence's rows NaN and leaves the others alone
    for bad in (math.nan, math.inf):
        d = _case(4, 16, 1, 64, 200, [30, 140, 1, 64], dtype=dtype, seed=10)
        good = _run(d)
        d["kv"][1, 100, 17] = bad
        x, lse, _ = _run(d)
        # a query whose product with +inf is -inf gives that token the weight e^-inf = 0;
        # every other row of the sequence is NaN
        hit = torch.ones(16, dtype=torch.bool) if math.isnan(bad) else d["q_lat"][1, :, 0, 17] > 0
        assert hit.any() and torch.isnan(x[1][hit]).all() and torch.isnan(lse[1][hit]).all()
        keep = [0, 2, 3]
        assert torch.equal(x[keep], good[0][keep]) and torch.equal(lse[keep], good[1][keep])
        x, lse, _ = _run(d, num_splits=3)
        assert torch.isnan(x[1][hit]).all() and torch.isfinite(x[keep]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_row_that_sees_only_a_bad_value_is_nan(dtype):
    d = _case(2, 8, 1, 64, 0, [1, 1], dtype=dtype, seed=11)
    d["kv"][0, 0, 3] = math.nan
    x, lse, _ = _run(d)
    assert torch.isnan(x[0]).all() and torch.isnan(lse[0]).all()
    assert torch.equal(x[1].float(), d["kv"][1, 0].float().expand(8, 1, C))


@pytest.mark.parametrize("page", [64, 16])
def test_bad_pages_are_flagged_and_skipped(page):
    d = _case(3, 16, 1, 64, 256, [100, 64, 130], page=page, seed=12)
    # the same sequences without the pages' tokens
    mask = torch.ones(256 + 192, dtype=torch.uint8)
    mask[page:2 * page] = 0
    want = _run(dict(d, mask=mask))[:2]
    d["prefix_table"][1] = 10 ** 6
    x, lse, err = _run(d)
    assert err & 1
    # masked and skipped tokens give the same sums in the same order
    assert torch.equal(x, want[0]) and torch.equal(lse, want[1])
    d["table"][0, 0] = -7
    x, lse, err = _run(d)
    assert err & 1 and torch.isfinite(x.float()).all()
    assert torch.equal(x[1:], want[0][1:])


def test_lengths_out_of_range_are_flagged_and_clamped():
    d = _case(3, 16, 1, 64, 200, [50, 40, 30], seed=13, Lk=50)
    x, lse, err = _run(d, seq_lens=torch.tensor([50, -3, 10 ** 6], dtype=torch.int32).cuda())
    assert err & 1
    want = _run(dict(d, lens=[50, 0, 50]))
    assert torch.equal(x, want[0]) and torch.equal(lse, want[1])


def test_scores_that_climb_far_above_the_first_tile():
    # the reference moves in later tiles (scores 2^60 above the first), up and down again
    d = _case(3, 32, 1, 64, 600, [100, 0, 64], seed=14)
    grow = torch.ones(600, dtype=torch.float64)
    grow[200:300], grow[300:400], grow[400:] = 40.0, 8.0, 90.0
    p = d["pkv"]
    p.copy_((p.double() * grow.cuda()[:, None]).to(p.dtype))
    pc = p.cpu().double()
    for b in range(3):
        d["rows"][b][:600, :C] = pc
    x, lse, err = _run(d)
    assert err == 0
    xo, lo, bound = _oracle(d)
    # scores reach several hundred: their float32 accumulation errs by up to
    # 576 * 2^-24 of sum |q k| scale <= 3e-5 * 4e3, which moves every weight by that
    rel = 576 * 2.0 ** -24 * 4e3
    assert ((x.cpu().double() - xo).abs() <= bound + rel * pc.abs().max()).all()
    assert ((lse.cpu().double() - lo).abs() <= rel).all()


@pytest.mark.parametrize("Lp", [0, 70])
@pytest.mark.parametrize("splits", [1, 3])
def test_references_that_start_and_move_in_either_half_of_a_block(Lp, splits):
    # eight sequences share a block of 128 rows, four in each CTA of its pair; their
    # rows see a first token in different tiles, and some grow far above it
    lens = [10, 300, 129, 0, 260, 1, 300, 200]
    d = _case(8, 16, 1, 64, Lp, lens, seed=21)
    for b, f in ((1, 60.0), (2, 40.0), (6, 70.0), (7, 8.0)):
        own = d["kv"][b]
        own[128:lens[b]] = (own[128:lens[b]].double() * f).to(own.dtype)
        d["rows"][b][Lp:, :C] = own[:lens[b]].cpu().double()
    x, lse, err = _run(d, num_splits=splits)
    assert err == 0
    xo, lo, bound = _oracle(d)
    fin = torch.isfinite(lo)
    # as above: 576 * 2^-24 of sum |q k| scale <= 4e3 moves every weight
    rel = 576 * 2.0 ** -24 * 4e3
    big = max(r.abs().max().item() for r in d["rows"] if len(r))
    assert ((x.cpu().double() - xo).abs()[fin] <= (bound + rel * big)[fin]).all()
    assert ((lse.cpu().double() - lo).abs()[fin] <= rel).all()
    assert (x.cpu()[~fin] == 0).all() and (lse.cpu()[~fin] == -math.inf).all()


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("power", [-90, 0, 90])
def test_float32_products_keep_float32s_precision(power, page):
    # one token, one channel of the scores: lse is a single product times the scale. Its
    # operands' parts add up exactly, six products of parts are added (2^-23 each), what
    # is left out is below 3 * 2^-25, and the scale rounds once: 8 * 2^-23 of the value
    d = _case(5, 24, 1, 64, 1, [0] * 5, dtype=torch.float32, page=page, seed=23)
    ch = 37
    q = d["q_lat"]
    q[..., ch] *= 2.0 ** power
    if power > 0:
        q[0, 0, 0, ch], q[1, 2, 0, ch] = 3.4e38, -3.3961e38            # beyond bf16's largest value
    d["q_pe"].zero_()
    row = d["pkv"][d["prefix_table"][0].item()][0] if page else d["pkv"][0]
    k = row[ch].item() * 2.0 ** -power
    rest = torch.zeros_like(row)
    rest[ch] = k
    row.copy_(rest)
    x, lse, err = _run(d)
    assert err == 0
    want = q[..., ch].double() * float(row[ch]) * d["scale"]
    # the call's scale is float32: half a step of it more
    assert ((lse.cpu().double() - want).abs() <= 9 * 2.0 ** -23 * want.abs()).all()
    # the only token's weight is 1
    assert ((x.cpu() - row.cpu()).abs() <= 3 * 2.0 ** -23 * row.abs().cpu()).all()


def test_float32_rows_with_a_non_finite_query():
    d = _case(3, 16, 1, 64, 40, [5, 6, 7], dtype=torch.float32, seed=24)
    good = _run(d)
    d["q_lat"][1, 3, 0, 5] = math.inf
    d["q_lat"][2, 4, 0, 6] = math.nan
    x, lse, err = _run(d)
    hit = torch.zeros(3, 16, dtype=torch.bool)
    hit[1, 3] = hit[2, 4] = True
    assert torch.isnan(x[:, :, 0].cpu()[hit]).all() and torch.isfinite(x[:, :, 0].cpu()[~hit]).all()
    xo, lo, _ = _oracle(d)
    assert ((x[:, :, 0].cpu().double() - xo[:, :, 0])[~hit].abs() <= 1e-4).all()
    assert ((good[0] - x)[:, :, 0].cpu()[~hit].abs() <= 2e-4).all()


def test_strided_rows_and_separate_storage():
    d = _case(4, 16, 1, 64, 300, [3, 70, 128, 1], pad=64, seed=15)            # 640-wide rows
    _check(d)
    _check(_case(4, 16, 1, 64, 300, [3, 70, 128, 1], page=64, prefix_paged=False, seed=16))


def test_equals_mla_decode_on_the_concatenated_cache():
    from latent_kv_decode_b200 import ops
    d = _case(3, 128, 1, 64, 256, [64, 100, 7], page=64, seed=17)
    x, lse, _ = _run(d, num_splits=1)
    table = torch.cat([d["prefix_table"].expand(3, -1), d["table"]], 1).contiguous()
    y, ly = ops.decode(d["q_lat"].cuda(), d["q_pe"].cuda(), d["kv"], d["pe"], d["scale"], block_table=table,
                       seq_lens=torch.tensor([256 + n for n in d["lens"]], dtype=torch.int32).cuda(), num_splits=1)
    # two roundings of the weights, two of x
    tol = 2 * _oracle(d)[2] + 4e-5
    assert ((x.double() - y.double()).abs().cpu() <= tol).all() and ((lse - ly).abs() <= 4e-4).all()


def test_large_pool_offsets_pass_32_bits():
    # rows whose element offsets are beyond 2^31: a pool of 4.3 GB
    from latent_kv_decode_b200 import ops
    page, pages = 64, 2 ** 31 // (64 * 576) + 300
    pool = torch.zeros((pages, page, 576), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    top = torch.tensor([[pages - 1, pages - 2], [pages - 3, pages - 4]], dtype=torch.int32)
    pool[pages - 6:] = torch.randn((6, page, 576), generator=g, device="cuda").bfloat16()
    q_lat = torch.randn((2, 16, 1, C), generator=g, device="cuda").bfloat16()
    q_pe = torch.randn((2, 16, 1, 64), generator=g, device="cuda").bfloat16()
    ptab = torch.tensor([pages - 5, pages - 6], dtype=torch.int32)
    lens = torch.tensor([100, 128], dtype=torch.int32)
    small, shift = pool[pages - 6:].clone(), pages - 6
    run = lambda pl, s: ops.mla_prefix_decode(q_lat, q_pe, pl[..., :C], pl[..., C:], pl[..., :C], pl[..., C:], 0.07,
                                              prefix_len=128, prefix_table=(ptab - s).cuda(), seq_lens=lens.cuda(),
                                              block_table=(top - s).cuda())
    a, b = run(pool, 0), run(small, shift)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
