"""The new calls run together as a serving step runs them: raw projection outputs
into the paged cache behind a shared prompt (mla_rope_append), the absorbed step
over prompt and own tokens (mla_prefix_decode_step), the output projection with
FP4 weights (mla_fp4_linear); eagerly, captured, on two streams.

Tolerances: the step's outputs against a plain fp64 evaluation on the same bf16
inputs use the parity tests' bf16 bounds (harness), which allow for the roundings
of the cached rows, q_lat, the weights of the softmax, x and out.
"""
import math

import numpy as np
import pytest
import torch

from harness import REL_L2_BF16, TOL_BF16, assert_close

pytestmark = pytest.mark.gpu

C, DR, DN, VD = 512, 64, 128, 128
THETA = 10000.0


def _turn(v, pos):
    j = torch.arange(v.shape[-1] // 2, dtype=torch.float64)
    ang = pos * THETA ** (-2.0 * j / v.shape[-1])
    e, o = v[..., 0::2], v[..., 1::2]
    return torch.stack([e * ang.cos() - o * ang.sin(), e * ang.sin() + o * ang.cos()], -1).flatten(-2)


class Model:
    """One layer's weights and a pool of pages; the prompt sits in pages of its own."""

    def __init__(self, B, H, prompt, steps, seed):
        from latent_kv_decode_b200 import ops
        g = torch.Generator().manual_seed(seed)
        n = lambda *s, scale=1.0: (torch.randn(s, generator=g) * scale).bfloat16()
        self.B, self.H, self.Lp, self.scale = B, H, prompt, 1 / math.sqrt(DN + DR)
        self.wkv_b = n(H, DN + VD, C, scale=1 / math.sqrt(C))
        self.wo = n(256, H * VD, scale=1 / math.sqrt(H * VD)).float()
        self.wo4, self.wo_scale = ops.pack_fp4_weight(self.wo.cuda())
        self.prompt = n(prompt, C + DR)
        self.steps = [dict(kv_a=n(B, C + DR), q=n(B, H, DN + DR)) for _ in range(steps)]
        page, per = 64, -(-steps // 64)
        np_ = -(-prompt // page)
        total = np_ + B * per
        perm = torch.randperm(total, generator=g).to(torch.int32).cuda()
        self.ptable, self.table = perm[:np_].contiguous(), perm[np_:].reshape(B, per).contiguous()
        # stale pages: whatever they hold behind a sequence's end stays out of the sums
        self.pool = torch.full((total, page, C + DR), math.nan, dtype=torch.bfloat16, device="cuda")
        self.kv, self.pe = self.pool[..., :C], self.pool[..., C:]
        self.w_dev = self.wkv_b.cuda()

    def prefill(self):
        from latent_kv_decode_b200 import ops
        p = self.prompt.cuda()
        ops.mla_rope_append(p[:, :C], p[:, C:], self.kv, self.pe,
                            torch.tensor([self.Lp], dtype=torch.int32).cuda(), block_table=self.ptable[None],
                            cu_tokens=torch.tensor([0, self.Lp], dtype=torch.int32).cuda(), rope_theta=THETA)

    def step(self, kv_a, q, lens, err=None, **kw):
        """One token per sequence: lens are the own lengths after it."""
        from latent_kv_decode_b200 import ops
        q_pe = ops.mla_rope_append(kv_a[:, None, :C], kv_a[:, None, C:], self.kv, self.pe, lens,
                                   q_pe=q[:, None, :, DN:], block_table=self.table, pos_offset=self.Lp,
                                   rope_theta=THETA, err_flag=err)
        q_nope = q[:, :, None, :DN].contiguous()
        out = ops.mla_prefix_decode_step(q_nope, q_pe, self.kv, self.pe, self.kv, self.pe, self.w_dev, self.scale,
                                         prefix_len=self.Lp, prefix_table=self.ptable, seq_lens=lens,
                                         block_table=self.table, causal=True, err_flag=err, **kw)
        return ops.mla_fp4_linear(out.reshape(self.B, self.H * VD), self.wo4, self.wo_scale, err_flag=err)

    def expect(self, t):
        """fp64 outputs of step t."""
        keys = [_turn_rows(self.prompt, 0)] * self.B
        w = self.wkv_b.double()
        # the packed weight's values
        e = self.wo4.cpu()
        lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
        lut = torch.cat([lut, -lut])
        c = e[..., :256].long()
        v = torch.stack([lut[c & 15], lut[c >> 4]], -1).flatten(-2)
        s = e[..., 256:].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
        wo = (v * s).flatten(-2) * self.wo_scale
        y = torch.zeros(self.B, 256, dtype=torch.float64)
        for b in range(self.B):
            own = torch.cat([_turn_rows(self.steps[i]["kv_a"][b:b + 1], self.Lp + i) for i in range(t + 1)])
            k = torch.cat([keys[b], own])
            q = self.steps[t]["q"][b].double()
            q_lat = torch.einsum("hd,hdc->hc", q[:, :DN], w[:, :DN])
            logit = (torch.cat([q_lat, _turn(q[:, DN:], self.Lp + t)], -1) @ k.T) * self.scale
            x = torch.softmax(logit, -1) @ k[:, :C]
            out = torch.einsum("hc,hvc->hv", x, w[:, DN:])
            y[b] = wo @ out.flatten()
        return y.numpy()


def _turn_rows(rows, pos0):
    d = rows.double()
    pe = torch.stack([_turn(d[i, C:], pos0 + i) for i in range(len(d))])
    return torch.cat([d[:, :C], pe], -1)


@pytest.mark.parametrize("B,H,prompt,steps", [(3, 16, 200, 5), (2, 128, 64, 3), (9, 8, 129, 66)])
def test_steps_behind_a_prompt(B, H, prompt, steps):
    m = Model(B, H, prompt, steps, seed=B + H)
    m.prefill()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in range(steps):
        lens = torch.full((B,), t + 1, dtype=torch.int32, device="cuda")
        y = m.step(m.steps[t]["kv_a"].cuda(), m.steps[t]["q"].cuda(), lens, err)
        if t in (0, 1, steps - 1):
            torch.cuda.synchronize()
            assert int(err.item()) == 0
            assert_close(y.float().cpu().numpy(), m.expect(t), TOL_BF16, f"step {t}", REL_L2_BF16)


def test_captured_step_follows_its_inputs():
    """A graph of the whole step, replayed with new tokens and lengths, equals the eager step bit for bit."""
    m, ref = (Model(4, 16, 150, 6, seed=1) for _ in range(2))
    m.prefill()
    ref.prefill()
    kv_a, q = m.steps[0]["kv_a"].cuda(), m.steps[0]["q"].cuda()
    lens = torch.ones(4, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step(kv_a, q, lens)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = m.step(kv_a, q, lens)
    for t in range(6):
        kv_a.copy_(m.steps[t]["kv_a"])
        q.copy_(m.steps[t]["q"])
        lens.fill_(t + 1)
        g.replay()
        want = ref.step(ref.steps[t]["kv_a"].cuda(), ref.steps[t]["q"].cuda(), lens.clone())
        torch.cuda.synchronize()
        assert torch.equal(y, want), f"step {t}"
    assert torch.equal(m.pool.view(torch.int16), ref.pool.view(torch.int16))


def test_two_streams_at_once_and_workspaces():
    """Calls that overlap on two streams, each with memory of its own, do not disturb one another;
    a given workspace serves one call after another."""
    from latent_kv_decode_b200 import ops
    g = torch.Generator("cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    B, H, Lp = 8, 16, 2000
    own, prefix = r(B, 100, C + DR), r(Lp, C + DR)
    sets = [(r(B, H, 1, C), r(B, H, 1, DR)) for _ in range(2)]
    lens = torch.arange(1, B + 1, dtype=torch.int32, device="cuda") * 12
    call = lambda k, **kw: ops.mla_prefix_decode(*sets[k], prefix[:, :C], prefix[:, C:], own[..., :C], own[..., C:], 0.07,
                                                 seq_lens=lens, **kw)
    want = [call(k, num_splits=5) for k in range(2)]
    ws = torch.empty(ops.make_prefix_decode(*sets[0], prefix[:, :C], prefix[:, C:], own[..., :C], own[..., C:], 0.07,
                                            seq_lens=lens, num_splits=5).workspace_bytes, dtype=torch.uint8, device="cuda")
    for k in (0, 1, 0):
        x, lse = call(k, num_splits=5, workspace=ws)
        assert torch.equal(x, want[k][0]) and torch.equal(lse, want[k][1])
    with pytest.raises(ops.MlaError):
        call(0, num_splits=5, workspace=ws[:-1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k, s in enumerate(streams):
            got[k].append(call(k, num_splits=5, stream=s))
    torch.cuda.synchronize()
    for k in range(2):
        for x, lse in got[k]:
            assert torch.equal(x, want[k][0]) and torch.equal(lse, want[k][1])


def test_masks_of_any_type():
    from latent_kv_decode_b200 import ops
    g = torch.Generator("cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    q, qp, p, own = r(2, 16, 1, C), r(2, 16, 1, DR), r(100, C + DR), r(2, 40, C + DR)
    mask = torch.rand(140, generator=g, device="cuda") < 0.5
    call = lambda m, **kw: ops.mla_prefix_decode(q, qp, p[:, :C], p[:, C:], own[..., :C], own[..., C:], 0.07, causal_mask=m, **kw)
    want = call(mask)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for m in (mask.to(torch.uint8), mask.float() * 0.25, mask.long().reshape(1, 1, 1, -1), torch.stack([mask, mask], 1)[:, 0]):
        for kw in ({}, dict(stream=s)):
            x, lse = call(m, **kw)
            torch.cuda.synchronize()
            assert torch.equal(x, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(ops.MlaError):
        ops.make_prefix_decode(q, qp, p[:, :C], p[:, C:], own[..., :C], own[..., C:], 0.07, causal_mask=mask.float())


def test_refusals_of_the_prefix_decode():
    from latent_kv_decode_b200 import ops
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")
    ok = dict(q_lat=z(2, 16, 1, C), q_pe=z(2, 16, 1, DR), prefix_kv=z(70, C), prefix_pe=z(70, DR), kv_cache=z(2, 9, C),
              pe_cache=z(2, 9, DR), softmax_scale=0.1)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")

    def call(**kw):
        a = dict(ok, **kw)
        return ops.mla_prefix_decode(a.pop("q_lat"), a.pop("q_pe"), a.pop("prefix_kv"), a.pop("prefix_pe"),
                                     a.pop("kv_cache"), a.pop("pe_cache"), a.pop("softmax_scale"), **a)

    x, lse = call(seq_lens=i32(0, 9))
    assert x.shape == (2, 16, 1, C) and (x == 0).all() and lse.shape == (2, 16, 1)
    assert call(want_lse=False)[1] is None
    pool = z(4, 64, C), z(4, 64, DR)
    bad = [dict(q_lat=z(2, 16, 1, C, dt=torch.float32)), dict(q_lat=z(2, 16, 1, 256)), dict(q_pe=z(2, 16, 1, 48)),
           dict(q_pe=z(2, 8, 1, DR)), dict(prefix_pe=z(69, DR)), dict(prefix_pe=None), dict(prefix_len=71),
           dict(prefix_kv=None, prefix_pe=None, prefix_len=3), dict(kv_cache=z(3, 9, C), pe_cache=z(3, 9, DR)),
           dict(pe_cache=z(2, 8, DR)), dict(pe_cache=None), dict(Lk=10), dict(seq_lens=i32(1, 2).long()),
           dict(seq_lens=i32(1)), dict(causal_mask=torch.ones(78, device="cuda")), dict(sinks=z(16)),
           dict(sinks=z(8, dt=torch.float32)), dict(num_splits=300), dict(num_splits=-1), dict(softmax_scale=0.0),
           dict(x=z(2, 16, 2, C)), dict(lse=z(2, 16, 1)), dict(prefix_kv=pool[0], prefix_pe=pool[1], prefix_table=i32(0)),
           dict(prefix_kv=pool[0], prefix_pe=pool[1], prefix_table=i32(0), prefix_len=65),
           dict(prefix_kv=pool[0], prefix_pe=pool[1], prefix_table=i32(0), prefix_len=64, page_size=32),
           dict(kv_cache=pool[0], pe_cache=pool[1], block_table=i32(0, 1)),
           dict(kv_cache=pool[0], pe_cache=pool[1], block_table=i32(0)[None]),
           dict(kv_cache=pool[0][::2], pe_cache=pool[1][::2], block_table=i32(0, 1)[:, None]), dict(kv_cache=ok["kv_cache"].cpu()),
           dict(q_lat=z(2, 12, 1, C), q_pe=z(2, 12, 1, DR))]
    for kw in bad:
        with pytest.raises(ops.MlaError):
            call(**kw)


def test_tensors_dropped_while_another_stream_still_reads_them():
    # inputs made on the current stream, a call on another that has not reached them
    # yet, the inputs dropped and their memory asked for again
    from latent_kv_decode_b200 import ops
    g = torch.Generator("cuda").manual_seed(31)
    rnd = lambda *sh: torch.randn(sh, generator=g, device="cuda").bfloat16()
    B, H, Lk = 8, 16, 128
    c_kv, k_pe, q_pe = rnd(B, 1, 512), rnd(B, 1, 64), rnd(B, 1, H, 64)
    lens = torch.full((B,), 5, dtype=torch.int32, device="cuda")
    q_lat, q_rot, rows = rnd(B, H, 1, 512), rnd(B, H, 1, 64), rnd(700, 576)
    x = rnd(40, 2048)
    w = torch.randint(0, 120, (300, 4, 288), generator=g, device="cuda", dtype=torch.uint8)
    originals = (c_kv, k_pe, q_pe, lens, q_lat, q_rot, rows, x, w)

    def late(stream):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                torch.cuda._sleep(20_000_000)
        return stream

    def append(stream=None):
        kv, pe = (torch.zeros((B, Lk, n), dtype=torch.bfloat16, device="cuda") for n in (512, 64))
        a = [t.clone() for t in (c_kv, k_pe, lens, q_pe)]
        return ops.mla_rope_append(a[0], a[1], kv, pe, a[2], q_pe=a[3], stream=late(stream)), kv, pe

    def decode(stream=None):
        a = [t.clone() for t in (q_lat, q_rot, rows)]
        return ops.mla_prefix_decode(a[0], a[1], a[2][:, :512], a[2][:, 512:], None, None, 0.07, stream=late(stream))

    def product(stream=None):
        a = [t.clone() for t in (x, w)]
        return (ops.mla_fp4_linear(a[0], a[1], 0.01, stream=late(stream)),)

    s = torch.cuda.Stream()
    for call in (append, decode, product):
        want = call()
        torch.cuda.synchronize()
        got = call(s)
        junk = [torch.full_like(t, 7) for t in originals for _ in range(3)]    # where the dropped inputs were
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), call.__name__
        del junk
