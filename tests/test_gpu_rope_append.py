"""GPU parity of mla_rope_append against a plain fp64 evaluation: rows copied bit for
bit, pairs turned by position * theta^(-2j/Dr), everything else left as it was.

Tolerance of a turned pair (a, b): the angle's whole turns are dropped in double
and its fraction rounded to float (2^-25 turns at most, 2^-22.3 radians); sine
and cosine add an ulp or two (2^-22 together); the float product and sum round
three times (3 2^-24). That is below 2^-20 (|a| + |b|); the result is rounded once to
its type (half a step: eps / 2).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

C = 512


def _turn(v, pos, theta):
    """v (..., Dr) fp64 pairs turned by pos (broadcast over v's leading dims) theta^(-2j/Dr)."""
    Dr = v.shape[-1]
    j = torch.arange(Dr // 2, dtype=torch.float64)
    ang = pos[..., None].double() * theta ** (-2.0 * j / Dr)
    e, o = v[..., 0::2], v[..., 1::2]
    return torch.stack([e * ang.cos() - o * ang.sin(), e * ang.sin() + o * ang.cos()], -1).flatten(-2)


def _close(got, src, pos, theta, dtype):
    want = _turn(src.double(), pos, theta)
    size = src.double().unflatten(-1, (-1, 2)).abs().sum(-1).repeat_interleave(2, -1)
    tol = 2.0 ** -20 * size + torch.finfo(dtype).eps / 2 * (want.abs() + 2.0 ** -20 * size)
    assert ((got.double() - want).abs() <= tol).all(), ((got.double() - want).abs() - tol).max()


def _case(new, past, H, Dr, dtype, page, seed, slack=3, offset=0):
    g = torch.Generator().manual_seed(seed)
    N, lens = sum(new), [n + p for n, p in zip(new, past)]
    d = dict(new=new, lens=lens, H=H, Dr=Dr, dtype=dtype, page=page, offset=offset)
    # rows of wider projections: the position parts start 16 bytes off a 64-byte line
    d["kv_a"] = torch.randn(N, C + Dr + 8, generator=g).to(dtype)
    d["q"] = torch.randn(N, H, 128 + Dr, generator=g).to(dtype) if H else None
    if page:
        need = [max(1, -(-n // page)) for n in lens]
        total = sum(need) + slack
        perm = torch.randperm(total, generator=g).to(torch.int32)
        d["table"] = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
        k = 0
        for b, n in enumerate(need):
            d["table"][b, :n] = perm[k:k + n]
            k += n
        d["rows"] = torch.randn(total, page, C + Dr, generator=g).to(dtype)
    else:
        d["table"] = None
        d["rows"] = torch.randn(len(lens), max(1, max(lens)) + slack, C + Dr, generator=g).to(dtype)
    return d


def _run(d, ragged, **kw):
    from latent_kv_decode_b200 import ops
    Dr, B = d["Dr"], len(d["lens"])
    rows = d["rows"].cuda()
    kv_a = d["kv_a"].cuda()
    c, k = kv_a[:, :C], kv_a[:, C:C + Dr]
    q = d["q"].cuda()[..., 128:] if d["H"] else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(q_pe=q, block_table=None if d["table"] is None else d["table"].cuda(), page_size=d["page"] or 64,
                pos_offset=d["offset"], err_flag=err)
    if ragged:
        args["cu_tokens"] = torch.tensor([0] + d["new"]).cumsum(0).to(torch.int32).cuda()
    else:
        Q = d["new"][0]
        c, k = c.unflatten(0, (B, Q)), k.unflatten(0, (B, Q))
        args["q_pe"] = None if q is None else q.unflatten(0, (B, Q))
    args.update(kw)
    out = ops.mla_rope_append(c, k, rows[..., :C], rows[..., C:], torch.tensor(d["lens"], dtype=torch.int32).cuda(),
                              **args)
    torch.cuda.synchronize()
    return rows.cpu(), None if out is None else out.cpu(), int(err.item())


def _check(d, ragged, theta=10000.0, **kw):
    rows, out, err = _run(d, ragged, **kw)
    assert err == 0
    Dr, new, lens = d["Dr"], d["new"], d["lens"]
    touched = torch.zeros(rows.shape[:2], dtype=torch.bool)
    n = 0
    for b in range(len(new)):
        for i in range(new[b]):
            t = lens[b] - new[b] + i
            at = (int(d["table"][b, t // d["page"]]), t % d["page"]) if d["page"] else (b, t)
            touched[at] = True
            assert torch.equal(rows[at][:C], d["kv_a"][n, :C])
            pos = torch.tensor(d["offset"] + t)
            _close(rows[at][C:], d["kv_a"][n, C:C + Dr], pos, theta, d["dtype"])
            if out is not None:
                got = out[n] if ragged else out[b, :, i]
                _close(got, d["q"][n, :, 128:], pos, theta, d["dtype"])
            n += 1
    assert torch.equal(rows[~touched], d["rows"][~touched])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Dr", [32, 64])
@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("B,Q,H", [(1, 1, 8), (5, 1, 128), (3, 4, 24), (2, 130, 1)])
def test_uniform(B, Q, H, page, Dr, dtype):
    _check(_case([Q] * B, [(7 * b) % 70 for b in range(B)], H, Dr, dtype, page, seed=B + Q, offset=4096), False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("new", [[1], [0, 3, 0, 0, 65, 1], [200, 0], [0, 0, 0], list(range(9)) * 40])
def test_ragged(new, page, dtype):
    _check(_case(new, [(11 * b) % 67 for b in range(len(new))], 16, 64, dtype, page, seed=len(new)), True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_far_positions_and_other_bases(dtype):
    for offset, theta in ((2 ** 20 - 3, 10000.0), (2 ** 28, 10000.0), (131072, 500000.0), (5, 3.0)):
        d = _case([2, 2], [5, 60], 8, 64, dtype, 64, seed=1, offset=offset)
        _check(d, False, theta=theta, rope_theta=theta)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_without_queries_in_place_and_given_output(dtype):
    from latent_kv_decode_b200 import ops
    d = _case([2, 2, 2], [0, 9, 64], 0, 64, dtype, 64, seed=2)
    _check(d, False)
    d = _case([3, 0, 2], [0, 9, 64], 8, 64, dtype, 64, seed=3)
    want = _run(d, True)[1]
    q = d["q"].cuda()
    got = _run(d, True, q_pe=q[..., 128:], q_out=q[..., 128:])[1]            # rotated where they lie
    assert torch.equal(got, want)
    assert torch.equal(q[..., :128].cpu(), d["q"][..., :128])
    d = _case([2, 2], [0, 9], 8, 64, dtype, 0, seed=4)
    want = _run(d, False)[1]
    wide = torch.zeros((2, 8, 2, 192), dtype=dtype, device="cuda")
    assert torch.equal(_run(d, False, q_out=wide[..., 128:])[1], want)
    assert (wide[..., :128] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_off_16_byte_boundaries(dtype):
    """Sources, queries and caches that only have their elements' alignment."""
    from latent_kv_decode_b200 import ops
    d = _case([3, 1], [5, 20], 8, 64, dtype, 0, seed=5)
    want = _run(d, True)
    odd = lambda t: torch.cat([t.new_zeros(*t.shape[:-1], 1), t], -1).cuda()[..., 1:]     # odd row length, odd start
    rows, kv_a, q = odd(d["rows"]), odd(d["kv_a"]), odd(d["q"])
    out = ops.mla_rope_append(kv_a[:, :C], kv_a[:, C:C + 64], rows[..., :C], rows[..., C:],
                              torch.tensor(d["lens"], dtype=torch.int32).cuda(), q_pe=q[..., 128:],
                              cu_tokens=torch.tensor([0, 3, 4], dtype=torch.int32).cuda())
    assert torch.equal(rows.cpu(), want[0]) and torch.equal(out.cpu(), want[1])


def test_rows_outside_the_sequences_are_left_alone():
    """Padding before the first and behind the last sequence of cu_tokens."""
    d = _case([2, 3], [4, 70], 8, 64, torch.bfloat16, 64, seed=6)
    N = 5
    pad = lambda t: torch.cat([torch.full_like(t[:2], 7), t, torch.full_like(t[:4], 9)])
    want = _run(d, True)
    e = dict(d, kv_a=pad(d["kv_a"]), q=pad(d["q"]))
    mark = torch.full((N + 6, 8, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    rows, out, err = _run(e, True, cu_tokens=torch.tensor([2, 4, 7], dtype=torch.int32).cuda(), q_out=mark)
    assert err == 0 and torch.equal(rows, want[0]) and torch.equal(out[2:7], want[1])
    assert (out[:2] == 5).all() and (out[7:] == 5).all()


def test_bad_positions_and_pages_are_flagged_and_not_stored():
    d = _case([1, 1, 1], [70, 130, 6], 8, 64, torch.bfloat16, 64, seed=7)
    want = _run(d, False)
    e = dict(d, table=d["table"].clone())
    e["table"][0, 1] = 10 ** 6
    e["table"][2, 0] = -5
    rows, out, err = _run(e, False)
    assert err & 1 and torch.equal(out, want[1])
    only = d["rows"].clone()
    t = d["lens"][1] - 1
    at = (int(d["table"][1, t // 64]), t % 64)
    only[at] = want[0][at]
    assert torch.equal(rows, only)
    # lengths that put a token outside [0, Lk)
    rows, out, err = _run(dict(d, lens=[0, 10 ** 9, -3]), False)
    assert err & 1 and torch.equal(rows, d["rows"])


def test_equal_results_captured_and_on_another_stream():
    from latent_kv_decode_b200 import ops
    d = _case([1] * 4, [0, 3, 63, 64], 16, 64, torch.bfloat16, 64, seed=8)
    want = _run(d, False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _run(d, False, stream=s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    rows, kv_a, q = d["rows"].cuda(), d["kv_a"].cuda(), d["q"].cuda()
    lens, table = torch.tensor(d["lens"], dtype=torch.int32).cuda(), d["table"].cuda()
    run = lambda: ops.mla_rope_append(kv_a[:, None, :C], kv_a[:, None, C:C + 64], rows[..., :C], rows[..., C:], lens,
                                      q_pe=q[:, None, :, 128:], block_table=table)
    run()
    torch.cuda.synchronize()
    rows.copy_(d["rows"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(rows.cpu(), want[0]) and torch.equal(out.cpu(), want[1])


def test_no_tokens():
    from latent_kv_decode_b200 import ops
    d = _case([1, 1], [3, 4], 8, 64, torch.bfloat16, 0, seed=10)
    rows, kv_a, q = d["rows"].cuda(), d["kv_a"].cuda(), d["q"].cuda()
    lens = torch.tensor(d["lens"], dtype=torch.int32).cuda()
    out = ops.mla_rope_append(kv_a[:0, None, :C].expand(0, 1, C).reshape(2, 0, C), kv_a[:0, C:C + 64].reshape(2, 0, 64),
                              rows[..., :C], rows[..., C:], lens, q_pe=q[:0, :, 128:].reshape(2, 0, 8, 64))
    assert out.shape == (2, 8, 0, 64)
    out = ops.mla_rope_append(kv_a[:0, :C], kv_a[:0, C:C + 64], rows[..., :C], rows[..., C:], lens, q_pe=q[:0, :, 128:],
                              cu_tokens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert out.shape == (0, 8, 64) and torch.equal(rows.cpu(), d["rows"])


def test_refusals():
    from latent_kv_decode_b200 import ops
    d = _case([2, 2], [0, 9], 8, 64, torch.bfloat16, 64, seed=9)
    rows, kv_a, q = d["rows"].cuda(), d["kv_a"].cuda(), d["q"].cuda()
    lens, table = torch.tensor(d["lens"], dtype=torch.int32).cuda(), d["table"].cuda()
    c, k, qp = kv_a[:, :C].unflatten(0, (2, 2)), kv_a[:, C:C + 64].unflatten(0, (2, 2)), q[..., 128:].unflatten(0, (2, 2))
    ok = dict(c=c, k=k, kv=rows[..., :C], pe=rows[..., C:], lens=lens, q_pe=qp, block_table=table)

    def call(**kw):
        a = dict(ok, **kw)
        return ops.mla_rope_append(a.pop("c"), a.pop("k"), a.pop("kv"), a.pop("pe"), a.pop("lens"), **a)

    call()
    bad = [dict(c=c.float()), dict(lens=lens.long()), dict(c=c[:1]), dict(k=k[..., :48]), dict(q_pe=qp[..., :32]),
           dict(block_table=table.long()), dict(page_size=32), dict(rope_theta=0.0), dict(kv=rows[..., :256]),
           dict(cu_tokens=torch.tensor([0, 2, 4], dtype=torch.int32).cuda()), dict(lens=lens.cpu()),
           dict(c=c.transpose(0, 1).contiguous().transpose(0, 1)), dict(q_out=torch.empty_like(qp)),
           dict(block_table=table[:1]), dict(k=k.expand(2, 2, 64)[..., ::2])]
    for kw in bad:
        with pytest.raises(ops.MlaError):
            call(**kw)
