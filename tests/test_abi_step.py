"""Host-side checks of mla_rope_append, mla_prefix_decode and mla_fp4_linear: bad
arguments are rejected before anything is enqueued, and the binding's structs
mirror the header. No call here reaches a launch: pointers are fake and every
argument set is invalid, or asks for sizes only.
"""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mla.h")
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    from latent_kv_decode_b200 import build, ops
    if not os.path.exists(ops.LIB_PATH):
        build.build()
    return ops.lib()


@pytest.mark.parametrize("name,cls", [("mla_rope_append_args", "RopeAppendArgs"), ("mla_prefix_args", "PrefixArgs"),
                                      ("mla_fp4_linear_args", "Fp4LinearArgs")])
def test_struct_mirrors_header(name, cls):
    """Fields in the header's order, with the header's types."""
    from latent_kv_decode_b200 import ops
    src = open(HEADER).read()
    body = src[src.index(f"typedef struct {name} {{"):src.index(f"}} {name};")]
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    want = []
    for decl in body.split("{", 1)[1].split(";"):
        m = re.match(r"\s*((?:const\s+)?\w+)\s*(.*)", decl.replace("\n", " "))
        if not m or not m.group(2).strip():
            continue
        for f in m.group(2).split(","):
            ptr = f.strip().startswith("*")
            kind = ctypes.c_void_p if ptr else {"int": ctypes.c_int, "mla_dtype_t": ctypes.c_int, "float": ctypes.c_float,
                                                "int64_t": ctypes.c_int64}[m.group(1)]
            want.append((f.strip().lstrip("*").strip(), kind))
    assert want == list(getattr(ops, cls)._fields_)


def _append(**over):
    from latent_kv_decode_b200 import ops
    a = ops.RopeAppendArgs()
    a.B, a.Q, a.N, a.Ckv, a.Dr, a.H, a.dtype = 2, 3, 6, 512, 64, 16, ops.MLA_BF16
    for f in ("c_kv", "k_pe", "q_pe", "q_out", "kv_cache", "pe_cache", "seq_lens"):
        setattr(a, f, FAKE)
    a.c_kv_stride = a.k_pe_stride = 576
    a.q_token_stride, a.q_head_stride = 16 * 192, 192
    a.o_batch_stride, a.o_token_stride, a.o_head_stride = 16 * 3 * 64, 64, 3 * 64
    a.kv_row_stride, a.pe_row_stride = 512, 64
    a.kv_batch_stride, a.pe_batch_stride = 512 * 100, 64 * 100
    a.Lk, a.rope_theta = 100, 10000.0
    for k, v in over.items():
        setattr(a, k, v)
    return a


_PAGED = dict(block_table=FAKE, max_pages=2, page_size=64, num_pages=9)


@pytest.mark.parametrize("over,status", [
    (dict(c_kv=None), 1), (dict(k_pe=None), 1), (dict(q_pe=None), 1), (dict(q_out=None), 1), (dict(kv_cache=None), 1),
    (dict(pe_cache=None), 1), (dict(seq_lens=None), 1), (dict(B=0), 1), (dict(Q=0), 1), (dict(N=5), 1), (dict(N=-1), 1),
    (dict(Lk=0), 1), (dict(H=-1), 1), (dict(dtype=2), 2), (dict(dtype=7), 2), (dict(Ckv=256), 2), (dict(Dr=48), 2),
    (dict(Dr=0), 1), (dict(H=2000), 2), (dict(rope_theta=0.0), 1), (dict(rope_theta=float("inf")), 1),
    (dict(rope_theta=float("nan")), 1), (dict(c_kv=FAKE + 1), 1), (dict(q_out=FAKE + 1), 1), (dict(seq_lens=FAKE + 2), 1),
    (dict(cu_tokens=FAKE + 1), 1), (dict(err_flag=FAKE + 2), 1), (dict(kv_row_stride=500), 1), (dict(pe_row_stride=60), 1),
    (dict(kv_batch_stride=10), 1), (dict(pe_batch_stride=10), 1), (dict(o_head_stride=63), 1),
    (dict(o_token_stride=0), 1), (dict(o_batch_stride=0), 1), (dict(c_kv_stride=-576), 1),
    (dict(_PAGED, page_size=0), 1), (dict(_PAGED, max_pages=1), 1), (dict(_PAGED, num_pages=0), 1),
])
def test_rope_append_rejects(L, over, status):
    assert L.mla_rope_append(ctypes.byref(_append(**over)), None) == status


def test_rope_append_without_tokens_enqueues_nothing(L):
    assert L.mla_rope_append(ctypes.byref(_append(N=0, Q=0, cu_tokens=FAKE, c_kv=None, k_pe=None, q_pe=None, q_out=None)),
                             None) == 0
    assert L.mla_rope_append(None, None) == 1


def _prefix(**over):
    from latent_kv_decode_b200 import ops
    a = ops.PrefixArgs()
    a.B, a.H, a.Q, a.Ckv, a.Dr, a.dtype = 4, 16, 1, 512, 64, ops.MLA_BF16
    for f in ("q_lat", "q_pe", "prefix_kv", "prefix_pe", "kv_cache", "pe_cache", "x"):
        setattr(a, f, FAKE)
    a.prefix_kv_stride, a.prefix_pe_stride, a.prefix_len = 512, 64, 1000
    a.kv_row_stride, a.pe_row_stride = 512, 64
    a.kv_batch_stride, a.pe_batch_stride = 512 * 100, 64 * 100
    a.Lk, a.page_size, a.softmax_scale = 100, 64, 0.07
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(q_lat=None), 1), (dict(q_pe=None), 1), (dict(x=None), 1), (dict(prefix_kv=None), 1), (dict(prefix_pe=None), 1),
    (dict(kv_cache=None), 1), (dict(pe_cache=None), 1), (dict(B=0), 1), (dict(H=12), 2), (dict(H=136), 2), (dict(Q=0), 1),
    (dict(Q=5), 2), (dict(Ckv=256), 2), (dict(Dr=48), 2), (dict(dtype=2), 2), (dict(prefix_len=-1), 1), (dict(Lk=-1), 1),
    (dict(num_splits=-1), 1), (dict(num_splits=257), 1), (dict(softmax_scale=0.0), 1),
    (dict(softmax_scale=float("nan")), 1), (dict(q_lat=FAKE + 8), 1), (dict(prefix_kv=FAKE + 8), 1), (dict(x=FAKE + 4), 1),
    (dict(lse=FAKE + 2), 1), (dict(prefix_kv_stride=511), 1), (dict(prefix_kv_stride=516), 1), (dict(prefix_pe_stride=32), 1),
    (dict(kv_row_stride=508), 1), (dict(kv_batch_stride=512), 1), (dict(kv_batch_stride=512 * 100 + 4), 1),
    (dict(prefix_table=FAKE, prefix_num_pages=0), 1), (dict(prefix_table=FAKE, prefix_num_pages=9, page_size=0), 1),
    (dict(_PAGED, max_pages=1), 1), (dict(_PAGED, num_pages=0), 1),
    (dict(prefix_len=1 << 30), 2), (dict(B=(1 << 20) + 1, num_splits=1), 2),
])
def test_prefix_decode_rejects(L, over, status):
    a = _prefix(**over)
    assert L.mla_prefix_decode(ctypes.byref(a), None, 0, None) == status
    assert L.mla_prefix_decode_num_splits(ctypes.byref(a)) == -1
    assert L.mla_prefix_decode_workspace_size(ctypes.byref(a)) == 0


def test_prefix_decode_workspace(L):
    a = _prefix(num_splits=3)
    rows = 4 * 16
    need = L.mla_prefix_decode_workspace_size(ctypes.byref(a))
    assert need == 3 * rows * 512 * 4 + 3 * rows * 4
    assert L.mla_prefix_decode(ctypes.byref(a), None, 0, None) == 3
    assert L.mla_prefix_decode(ctypes.byref(a), FAKE, need - 1, None) == 3
    assert L.mla_prefix_decode(ctypes.byref(a), FAKE + 16, need, None) == 3     # not 256-byte aligned
    assert L.mla_prefix_decode_workspace_size(ctypes.byref(_prefix(num_splits=1))) == 0
    assert L.mla_prefix_decode(None, None, 0, None) == 1
    # the automatic count: at least 1, at most the block's tiles
    for over in (dict(), dict(prefix_len=0, Lk=1), dict(prefix_len=0, Lk=0, kv_cache=None), dict(prefix_len=131072)):
        assert 1 <= L.mla_prefix_decode_num_splits(ctypes.byref(_prefix(**over))) <= 256


def _linear(**over):
    from latent_kv_decode_b200 import ops
    a = ops.Fp4LinearArgs()
    a.B, a.Q, a.G, a.N, a.K = 3, 2, 4, 100, 1024
    a.x = a.w = a.out = FAKE
    a.x_batch_stride, a.x_token_stride, a.x_group_stride, a.x_block_stride = 8 * 1024, 512, 2048, 1024
    a.scale = 1.0
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(B=0), 1), (dict(Q=0), 1), (dict(G=0), 1),
    (dict(N=0), 1), (dict(K=0), 1), (dict(K=768), 2), (dict(x=FAKE + 8), 1), (dict(w=FAKE + 8), 1), (dict(out=FAKE + 1), 1),
    (dict(x_batch_stride=12), 1), (dict(x_token_stride=-512), 1), (dict(x_block_stride=4), 1), (dict(err_flag=FAKE + 2), 1),
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(B=1 << 20), 2), (dict(N=1 << 29), 2),
    (dict(G=70000, N=1), 2),
])
def test_fp4_linear_rejects(L, over, status):
    a = _linear(**over)
    assert L.mla_fp4_linear(ctypes.byref(a), None, 0, None) == status
    assert L.mla_fp4_linear_workspace_size(ctypes.byref(a)) == 0


def test_fp4_linear_workspace(L):
    assert L.mla_fp4_linear_workspace_size(ctypes.byref(_linear())) == 0     # small products need none
    a = _linear(B=12, N=4096)
    need = L.mla_fp4_linear_workspace_size(ctypes.byref(a))
    assert need == 24 * 4 * 1024 * 2 + 24 * 4 * 4        # float16 activations, an exponent per token and group
    assert L.mla_fp4_linear(ctypes.byref(a), None, 0, None) == 3
    assert L.mla_fp4_linear(ctypes.byref(a), FAKE, need - 1, None) == 3
    assert L.mla_fp4_linear(ctypes.byref(a), FAKE + 16, need, None) == 3


def test_binding_refuses_cpu_tensors():
    import torch
    from latent_kv_decode_b200 import ops
    f = torch.zeros
    with pytest.raises(ops.MlaError):
        ops.mla_prefix_decode(f(1, 8, 1, 512), f(1, 8, 1, 64), f(4, 512), f(4, 64), None, None, 0.1)
    with pytest.raises(ops.MlaError):
        ops.mla_rope_append(f(1, 1, 512), f(1, 1, 64), f(1, 4, 512), f(1, 4, 64), f(1, dtype=torch.int32))
    with pytest.raises(ops.MlaError):
        ops.mla_fp4_linear(f(1, 512, dtype=torch.bfloat16), f(8, 1, 288, dtype=torch.uint8))
    with pytest.raises(ops.MlaError):
        ops.pack_fp4_weight(f(8, 512))
