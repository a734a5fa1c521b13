"""GPU parity of mla_fp4_linear and mla_fp4_group_wo against a plain fp64
evaluation: decode the entries from the format's definition, multiply, sum.

Tolerance. Weights and (scaled) activations are exact operands, products are
exact and the sums are float32: a sum of K products in the tensor core and of
at most 8 partial sums errs by at most (K + 8) 2^-23 sum |x w| (a rounding or
truncation of at most 2^-23 per addition), usually far less; the output is
rounded once to bf16, at most 2^-8 of its value.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U16 = torch.finfo(torch.bfloat16).eps / 2


def _entries(shape, seed, scale_lo=0x20, scale_hi=0x7F):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (*shape, 256), generator=g, dtype=torch.uint8)
    scales = torch.randint(scale_lo, scale_hi, (*shape, 32), generator=g, dtype=torch.uint8)
    return torch.cat([codes, scales], -1)


def _values(e):
    """(..., blocks, 288) entries as (..., blocks * 512) float64."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    lut = torch.cat([lut, -lut])
    c = e[..., :256].long()
    v = torch.stack([lut[c & 15], lut[c >> 4]], -1).flatten(-2)
    s = e[..., 256:].contiguous().view(torch.float8_e4m3fn).double()
    return (v * s.repeat_interleave(16, -1)).flatten(-2)


def _check(y, x, w, scale):
    """y against x (T, K) fp64 and w (N, K) fp64."""
    want = x @ w.T * scale
    mag = x.abs() @ w.abs().T * abs(scale)
    tol = U16 * want.abs() + (1 + U16) * (x.shape[1] + 8) * 2.0 ** -23 * mag + 1e-40
    err = (y.cpu().double() - want).abs()
    assert (err <= tol).all(), f"worst {(err - tol).max().item():.3e}"


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 65, 130])
@pytest.mark.parametrize("N,K", [(1, 512), (127, 1024), (130, 512), (513, 2560)])
def test_tokens_rows_and_widths(T, N, K):
    from latent_kv_decode_b200 import ops
    w = _entries((N, K // 512), seed=N + K)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(T)).bfloat16()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ops.mla_fp4_linear(x.cuda(), w.cuda(), 0.013, err_flag=err)
    assert y.shape == (T, N) and int(err.item()) == 0
    _check(y, x.double(), _values(w), 0.013)


@pytest.mark.parametrize("T", [1, 3, 8, 9, 16])
@pytest.mark.parametrize("N,K", [(20, 8704), (2500, 4608), (5001, 2560)])
def test_few_tokens_with_many_entries_and_rows(T, N, K):
    """More entries than a CTA has warps; one, two and more CTAs per SM."""
    from latent_kv_decode_b200 import ops
    w = _entries((N, K // 512), seed=N)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(T + 20)).bfloat16()
    y = ops.mla_fp4_linear(x.cuda(), w.cuda(), 0.01)
    _check(y, x.double(), _values(w), 0.01)
    # a token's result does not depend on the tokens beside it
    assert torch.equal(ops.mla_fp4_linear(x[-1:].cuda(), w.cuda(), 0.01)[0], y[-1])


@pytest.mark.parametrize("T", [25, 33, 64, 65, 130])
@pytest.mark.parametrize("N,K", [(21600, 512), (5001, 2560), (1300, 8704)])
def test_larger_products(T, N, K):
    """Ragged token and row blocks, one, five and seventeen entries a row."""
    from latent_kv_decode_b200 import ops
    w = _entries((N, K // 512), seed=N + 1)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(T + 30)).bfloat16()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ops.mla_fp4_linear(x.cuda(), w.cuda(), 0.013, err_flag=err)
    assert int(err.item()) == 0
    _check(y, x.double(), _values(w), 0.013)


def test_magnitudes_and_bad_values_of_larger_products():
    # as the tests of small products, with enough rows for the other kernel
    from latent_kv_decode_b200 import ops
    w = _entries((11000, 2), seed=3)
    base = torch.randn(26, 1024, generator=torch.Generator().manual_seed(4)).bfloat16()
    for k, p in enumerate([-126, -100, -30, 0, 30, 100, 115]):
        base[k] = (base[k].double() * 2.0 ** p).bfloat16()
    base[7, ::2] = 0
    base[8] = 0
    v = _values(w)
    good = ops.mla_fp4_linear(base.cuda(), w.cuda(), 2.0 ** -16)
    _check(good, base.double(), v, 2.0 ** -16)
    assert (good[8] == 0).all()
    base[11, 7], base[13, 9] = math.nan, math.inf
    y = ops.mla_fp4_linear(base.cuda(), w.cuda(), 2.0 ** -16)
    assert torch.isnan(y[11]).all()
    want = torch.where(v[:, 9] == 0, torch.full_like(v[:, 9], math.nan), v[:, 9] * math.inf)
    assert torch.equal(torch.nan_to_num(y[13].cpu().double(), nan=7.0, posinf=8.0, neginf=9.0),
                       torch.nan_to_num(want, nan=7.0, posinf=8.0, neginf=9.0))
    rest = [t for t in range(26) if t not in (11, 13)]
    assert torch.equal(y[rest], good[rest])


@pytest.mark.parametrize("p", [-130, -126, -100, -30, 30, 100, 115])
def test_one_token_over_bf16s_whole_range(p):
    from latent_kv_decode_b200 import ops
    w = _entries((33, 2), seed=3)
    x = (torch.randn(1, 1024, generator=torch.Generator().manual_seed(4)).double() * 2.0 ** p).bfloat16()
    y = ops.mla_fp4_linear(x.cuda(), w.cuda(), 2.0 ** -16 if p > 0 else 1.0)
    _check(y, x.double(), _values(w), 2.0 ** -16 if p > 0 else 1.0)


@pytest.mark.parametrize("B,H,Q,G,R", [(1, 2, 1, 2, 5), (3, 16, 2, 4, 128), (5, 8, 4, 8, 257), (32, 64, 1, 8, 1024)])
def test_groups_and_strided_heads(B, H, Q, G, R):
    from latent_kv_decode_b200 import ops
    w = _entries((G, R, H // G), seed=R)
    g = torch.Generator().manual_seed(B)
    x = torch.randn(B, H, Q, 512, generator=g).bfloat16()
    z = ops.mla_fp4_group_wo(x.cuda(), w.cuda(), scale_a=0.02)
    assert z.shape == (B, Q, G * R)
    wide = torch.randn(B, H, Q, 640, generator=g).bfloat16().cuda()        # the same values in wider rows
    wide[..., :512] = x.cuda()
    assert torch.equal(ops.mla_fp4_group_wo(wide[..., :512], w.cuda(), scale_a=0.02), z)
    u = x.double().reshape(B, G, H // G, Q, 512).permute(1, 0, 3, 2, 4).reshape(G, B * Q, -1)
    for k in range(G):
        _check(z.reshape(B * Q, G, R)[:, k], u[k], _values(w[k]), 0.02)


def test_every_code_and_scale():
    # K = 512: row n holds scale byte n in all groups; token k picks channel k
    from latent_kv_decode_b200 import ops
    e = torch.zeros((256, 1, 288), dtype=torch.uint8)
    lo = torch.arange(256) % 16
    e[:, 0, :256] = (lo + 16 * ((lo + 5) % 16)).to(torch.uint8)            # all sixteen codes, both nibbles
    e[:, 0, 256:] = torch.arange(256, dtype=torch.uint8)[:, None]
    x = torch.eye(512).bfloat16()
    y = ops.mla_fp4_linear(x.cuda(), e.cuda()).cpu().double()
    want = _values(e).T
    nan = torch.isnan(want)                                               # scale bytes 0x7F and 0xFF are NaN
    assert nan[:, 127].all() and nan[:, 255].all() and nan.sum() == 2 * 512
    # a NaN weight meets the other tokens' zeros too: NaN for all of them
    assert torch.isnan(y[:, 127]).all() and torch.isnan(y[:, 255]).all()
    # six significant bits: exact in bf16
    assert torch.equal(y[~nan], want[~nan])


def test_magnitudes_over_bf16s_whole_range():
    from latent_kv_decode_b200 import ops
    w = _entries((64, 2), seed=3)
    g = torch.Generator().manual_seed(4)
    base = torch.randn(12, 1024, generator=g).bfloat16()
    for k, p in enumerate([-126, -100, -30, 0, 30, 100, 115]):
        base[k] = (base[k].double() * 2.0 ** p).bfloat16()
    base[7, ::2] = 0
    base[8] = 0
    base[9] = (torch.randn(1024, generator=g).double() * 2.0 ** torch.randint(-20, 8, (1024,), generator=g)).bfloat16()
    base[10, 5], base[11, 6] = 2.0 ** 20, -2.0 ** -30
    y = ops.mla_fp4_linear(base.cuda(), w.cuda(), 2.0 ** -16)
    _check(y, base.double(), _values(w), 2.0 ** -16)
    assert (y[8] == 0).all()


def test_infinities_and_nan_stay_with_their_token():
    from latent_kv_decode_b200 import ops
    w = _entries((40, 1), seed=5)
    x = torch.randn(5, 512, generator=torch.Generator().manual_seed(6)).bfloat16()
    good = ops.mla_fp4_linear(x.cuda(), w.cuda())
    x[1, 7], x[3, 9] = math.nan, math.inf
    y = ops.mla_fp4_linear(x.cuda(), w.cuda())
    assert torch.isnan(y[1]).all()
    v = _values(w)[:, 9]
    want = torch.where(v == 0, torch.full_like(v, math.nan), v * math.inf)
    assert torch.equal(torch.nan_to_num(y[3].cpu().double(), nan=7.0, posinf=8.0, neginf=9.0),
                       torch.nan_to_num(want, nan=7.0, posinf=8.0, neginf=9.0))
    for t in (0, 2, 4):
        assert torch.equal(y[t], good[t])


def test_the_group_wo_chain_and_packing():
    """pack_fp4_weight -> mla_fp4_group_wo -> mla_fp4_linear, as a user runs them."""
    from latent_kv_decode_b200 import ops
    g = torch.Generator("cuda").manual_seed(8)
    B, H, Q, G, R, D = 3, 16, 2, 4, 256, 384
    x = torch.randn((B, H, Q, 512), generator=g, device="cuda").bfloat16()
    wa = torch.randn((G, R, (H // G) * 512), generator=g, device="cuda") / math.sqrt(2048)
    wb = torch.randn((D, G * R), generator=g, device="cuda") / 32
    ea, sa = ops.pack_fp4_weight(wa)
    eb, sb = ops.pack_fp4_weight(wb)
    assert ea.shape == (G, R, H // G, 288) and eb.shape == (D, G * R // 512, 288)
    qa, qb = _values(ea.cpu()) * sa, _values(eb.cpu()) * sb
    # the packing itself: a weight is off by at most a sixth of its group's largest
    # (E2M1's widest half step, 1 of 6) plus the scale's own half step (2^-4)
    for q, w in ((qa, wa), (qb, wb)):
        w = w.cpu().double()
        top = w.unflatten(-1, (-1, 16)).abs().amax(-1, keepdim=True).expand(*w.shape[:-1], -1, 16).flatten(-2)
        assert ((q - w).abs() <= top * (1 / 6 + 2.0 ** -4) * (1 + 2.0 ** -10)).all()
    z = ops.mla_fp4_group_wo(x, ea, scale_a=sa)
    y = ops.mla_fp4_group_wo(x, ea, eb, scale_a=sa, scale_b=sb)
    assert y.shape == (B, Q, D)
    _check(y.reshape(B * Q, D), z.reshape(B * Q, -1).cpu().double(), qb / sb, sb)
    assert torch.equal(y, ops.mla_fp4_linear(z, eb, sb))


def test_equal_results_on_repeat_and_on_another_stream():
    from latent_kv_decode_b200 import ops
    w = _entries((4096, 8), seed=9).cuda()
    x = torch.randn(3, 4096, generator=torch.Generator().manual_seed(10)).bfloat16().cuda()
    y = ops.mla_fp4_linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = [ops.mla_fp4_linear(x, w, stream=s) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(o, y) for o in out)


def test_inputs_that_need_a_copy():
    """Activations the kernel cannot read in place: copied, on the call's own stream."""
    from latent_kv_decode_b200 import ops
    w = _entries((70, 2), seed=12).cuda()
    x = torch.randn(4, 3, 1024, generator=torch.Generator().manual_seed(13)).bfloat16().cuda()
    want = ops.mla_fp4_linear(x, w)
    assert want.shape == (4, 3, 70)
    odd = torch.zeros((4, 3, 1027), dtype=torch.bfloat16, device="cuda")
    odd[..., 1:1025] = x
    back = x.transpose(0, 1).contiguous().transpose(0, 1)
    packed_off = torch.cat([x.new_zeros(1), x.flatten()])[1:].view(4, 3, 1024)      # contiguous, 2 bytes off
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for v in (odd[..., 1:1025], back, packed_off, x[0, 0]):
        for stream in (None, s):
            y = ops.mla_fp4_linear(v, w, stream=stream)
            s.synchronize()
            torch.cuda.synchronize()
            assert torch.equal(y, want if v.dim() == 3 else want[0, 0])
    wg = _entries((2, 70, 1), seed=14).cuda()
    x4 = torch.randn(2, 2, 3, 512, generator=torch.Generator().manual_seed(15)).bfloat16().cuda()
    want = ops.mla_fp4_group_wo(x4, wg)
    odd = torch.zeros((2, 2, 3, 515), dtype=torch.bfloat16, device="cuda")
    odd[..., 3:] = x4
    torch.cuda.synchronize()
    y = ops.mla_fp4_group_wo(odd[..., 3:], wg, stream=s)
    s.synchronize()
    assert torch.equal(y, want)


def test_no_tokens_and_refusals():
    from latent_kv_decode_b200 import ops
    w = _entries((8, 1), seed=11).cuda()
    x = torch.zeros((0, 512), dtype=torch.bfloat16, device="cuda")
    assert ops.mla_fp4_linear(x, w).shape == (0, 8)
    x = torch.zeros((2, 512), dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: ops.mla_fp4_linear(x.float(), w), lambda: ops.mla_fp4_linear(x, w.float()),
                lambda: ops.mla_fp4_linear(x, w[..., :280]), lambda: ops.mla_fp4_linear(x[:, :256], w),
                lambda: ops.mla_fp4_linear(x.cpu(), w), lambda: ops.mla_fp4_linear(x, w, float("nan")),
                lambda: ops.mla_fp4_linear(x, w, out=torch.empty((2, 9), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ops.MlaError):
            bad()
