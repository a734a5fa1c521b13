"""The serving-step calls on another stream than the current one: where their memory
comes from and how long their inputs live. Every comparison is of bits: the same
call gives the same result whatever the stream.

A block of memory that was just freed on the current stream may still be written by
work queued there. ``_busy_blocks`` leaves such blocks in the current stream's pool,
of all the sizes that a call may ask for; a call on a stream that does not wait for
that work must not be given one.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

C, DR = 512, 64
SLEEP = 40_000_000          # clock cycles, about 20 ms: longer than any call here takes to enqueue and run


def _inputs():
    g = torch.Generator("cuda").manual_seed(41)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    B, H = 8, 16
    d = dict(c_kv=r(B, 1, C), k_pe=r(B, 1, DR), q_raw=r(B, 1, H, DR), q_lat=r(B, H, 1, C), q_pe=r(B, H, 1, DR),
             rows=r(700, C + DR), x=r(40, 2048), x4=r(40, 8, 1, C))
    d["lens"] = torch.full((B,), 5, dtype=torch.int32, device="cuda")
    d["kv"], d["pe"] = (torch.zeros((B, 128, n), dtype=torch.bfloat16, device="cuda") for n in (C, DR))
    e = lambda *s: torch.randint(0, 120, (*s, 288), generator=g, device="cuda", dtype=torch.uint8)
    # 40 tokens of 4096 x 2048 weights take the kernels with a workspace
    d["w"], d["wa"], d["wb"] = e(6000, 4), e(4, 1024, 2), e(1100, 8)
    return d


def _calls(d):
    from latent_kv_decode_b200 import ops
    prefix = lambda make, **kw: make(d["q_lat"], d["q_pe"], d["rows"][:, :C], d["rows"][:, C:], None, None, 0.07,
                                     num_splits=5, **kw)

    def prepared(stream=None):
        return ops.launch_prefix_decode(prefix(ops.make_prefix_decode), stream=stream)

    return {
        "append": lambda stream=None: (ops.mla_rope_append(d["c_kv"], d["k_pe"], d["kv"], d["pe"], d["lens"],
                                                           q_pe=d["q_raw"], stream=stream), d["kv"], d["pe"]),
        "prefix": lambda stream=None: prefix(ops.mla_prefix_decode, stream=stream),
        "prepared": prepared,
        "product": lambda stream=None: (ops.mla_fp4_linear(d["x"], d["w"], 0.01, stream=stream),),
        "groups": lambda stream=None: (ops.mla_fp4_group_wo(d["x4"], d["wa"], scale_a=0.01, stream=stream),),
        "chain": lambda stream=None: (ops.mla_fp4_group_wo(d["x4"], d["wa"], d["wb"], scale_a=0.01, scale_b=0.01,
                                                           stream=stream),),
    }


def _busy_blocks():
    """Blocks of the current stream's pool that a kernel queued there has yet to write."""
    torch.cuda.synchronize()
    sizes = [512 * 2 ** k for k in range(14)] + [3 * 512 * 2 ** k for k in range(12)]
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda._sleep(SLEEP)
    for b in blocks:
        b.fill_(0x7F)


@pytest.mark.parametrize("name", ["append", "prefix", "prepared", "product", "groups", "chain"])
def test_memory_of_a_call_on_another_stream(name):
    call = _calls(_inputs())[name]
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    _busy_blocks()
    got = call(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["append", "prefix", "prepared", "product", "groups", "chain"])
def test_results_dropped_while_the_current_stream_still_reads_them(name):
    # the current stream waits for the call, reads its results late, and they are dropped;
    # the next call on the same stream must not write over them
    call = _calls(_inputs())[name]
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(SLEEP)
    late = [t.clone() for t in got]
    sizes = [t.numel() * t.element_size() for t in got]
    del got
    with torch.cuda.stream(s):
        junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(late, want))
    del junk


def test_a_prepared_call_in_a_capture():
    # prepared outside, launched inside: the capture takes no dependency on other work
    from latent_kv_decode_b200 import ops
    d = _inputs()
    args = (d["q_lat"], d["q_pe"], d["rows"][:, :C], d["rows"][:, C:], None, None, 0.07)
    want = ops.mla_prefix_decode(*args, num_splits=5)
    c = ops.make_prefix_decode(*args, num_splits=5)
    ops.launch_prefix_decode(c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.launch_prefix_decode(c)
    c.x.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.x, want[0]) and torch.equal(c.lse, want[1])


def _odd(t):
    """The same values in rows that no call reads in place: packed, but two bytes off the wide accesses."""
    wide = torch.zeros((*t.shape[:-1], t.shape[-1] + 3), dtype=t.dtype, device=t.device)
    wide[..., 3:] = t
    return wide[..., 3:]


@pytest.mark.parametrize("name", ["product", "product in blocks", "groups", "chain", "float mask", "strided mask"])
def test_inputs_that_are_copied_and_dropped_while_the_copy_waits(name):
    # the call's stream has not reached the copy when the caller drops the input and
    # asks for its memory again
    from latent_kv_decode_b200 import ops
    d = _inputs()
    g = torch.Generator("cuda").manual_seed(43)
    seen = torch.rand(700, generator=g, device="cuda") < 0.5
    prefix = lambda m, **kw: ops.mla_prefix_decode(d["q_lat"], d["q_pe"], d["rows"][:, :C], d["rows"][:, C:], None, None,
                                                   0.07, causal_mask=m, **kw)
    make, call = {
        "product": (lambda: _odd(d["x"]), lambda x, **kw: ops.mla_fp4_linear(x, d["w"], 0.01, **kw)),
        "product in blocks": (lambda: _odd(d["x"].view(4, 10, 2048)), lambda x, **kw: ops.mla_fp4_linear(x, d["w"], 0.01, **kw)),
        "groups": (lambda: _odd(d["x4"]), lambda x, **kw: ops.mla_fp4_group_wo(x, d["wa"], scale_a=0.01, **kw)),
        "chain": (lambda: _odd(d["x4"]), lambda x, **kw: ops.mla_fp4_group_wo(x, d["wa"], d["wb"], scale_a=0.01, scale_b=0.01, **kw)),
        "float mask": (lambda: seen.float(), prefix),
        "strided mask": (lambda: torch.stack([seen, seen], 1)[:, 0], prefix),
    }[name]
    out = lambda r: r if isinstance(r, tuple) else (r,)
    want = [t.clone() for t in out(call(make()))]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = make()
    size = a.untyped_storage().nbytes()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP)
    got = out(call(a, stream=s))
    del a
    junk = [torch.full((size,), 0x31, dtype=torch.uint8, device="cuda") for _ in range(4)]     # where it was
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del junk
