"""Measured cases of three operators of the decode path.

- append: a step's (or a prompt's) new latent rows and their rotated position
  rows go into the cache, and the queries' position parts are rotated with them.
- prefix: latent attention of a batch whose sequences share a long prefix.
- fp4: products of few tokens with weights held as 4-bit codes and group scales
  (the 288-byte entries of the latent cache: 512 channels, a scale per 16).

``run`` computes the plain form (elementary torch operations in float32, angles
in float64, rounded once), or, where ``own`` is true, calls the package.
Per-sequence lengths are an even spread over a case's range, shuffled by the
seed, so a case's total work does not depend on the seed.
"""
import math

import torch

own = False

CKV = 512          # latent width
ENTRY = 288        # bytes of one 4-bit entry: 256 of codes, 32 scales
THETA = 10000.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one new token for each of two short sequences, float32, few heads: latency
        dict(name="append_tiny_f32", op="append", B=2, Q=1, new_lo=1, new_hi=1, past_lo=0, past_hi=9, H=8, Dr=32,
             dtype="f32", page=0, offset=0),
        # a decode step of the 64-sequence serving batch, all heads, paged cache
        dict(name="append_step_b64", op="append", B=64, Q=1, new_lo=1, new_hi=1, past_lo=0, past_hi=700, H=128, Dr=64,
             dtype="bf16", page=64, offset=4096),
        # prompts of unequal lengths written in one call (a prefill's cache write)
        dict(name="append_prompts", op="append", B=24, Q=0, new_lo=0, new_hi=1021, past_lo=0, past_hi=130, H=128,
             Dr=64, dtype="bf16", page=64, offset=0),
        # the demonstration shape with a shared part: float32, ten cached tokens
        dict(name="prefix_tiny_f32", op="prefix", B=2, H=8, Q=1, Dr=32, dtype="f32", prefix=7, len_lo=1, len_hi=3,
             page=0, causal=0),
        # heads of one of eight cooperating GPUs, a system prompt, ragged answers
        # with two speculative tokens
        dict(name="prefix_b128_h16_q2", op="prefix", B=128, H=16, Q=2, Dr=64, dtype="bf16", prefix=16384, len_lo=2,
             len_hi=511, page=64, causal=1),
        # the 64-sequence serving batch with all heads behind one prompt
        dict(name="prefix_b64_h128", op="prefix", B=64, H=128, Q=1, Dr=64, dtype="bf16", prefix=4096, len_lo=1,
             len_hi=500, page=64, causal=0),
        # few sequences behind one very long document, contiguous storage
        dict(name="prefix_long_b4", op="prefix", B=4, H=128, Q=1, Dr=64, dtype="bf16", prefix=131072, len_lo=17,
             len_hi=129, page=0, causal=0),
        # full float32 precision at a moderate size
        dict(name="prefix_f32_b8_h16", op="prefix", B=8, H=16, Q=1, Dr=64, dtype="f32", prefix=2049, len_lo=0,
             len_hi=99, page=0, causal=0),
        # three tokens, one entry per row, an odd number of rows: latency
        dict(name="fp4_tiny", op="fp4", B=3, H=1, Q=1, G=1, R=200, grouped=0),
        # one token through an output projection (8192 to 4096)
        dict(name="fp4_one_token", op="fp4", B=1, H=16, Q=1, G=1, R=4096, grouped=0),
        # 32 tokens through the groups' own factors: 8 groups of rank 1024, 64 heads
        dict(name="fp4_groups_b32", op="fp4", B=32, H=64, Q=1, G=8, R=1024, grouped=1),
        # 64 tokens through the widest projection (16384 to 7168)
        dict(name="fp4_wide_b64", op="fp4", B=64, H=32, Q=1, G=1, R=7168, grouped=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "prefix", "prefix", "fp4"])
    if op == "append":
        ragged = rng.random() < 0.5
        hi = _log(rng, 1, 1024) if ragged else 0
        q = 0 if ragged else rng.randint(1, 4)
        f32 = rng.random() < 0.3
        return dict(op=op, B=_log(rng, 1, 24 if ragged else 128), Q=q, new_lo=0 if ragged else q,
                    new_hi=hi if ragged else q, past_lo=0, past_hi=_log(rng, 1, 1000), H=8 * rng.randint(1, 16),
                    Dr=rng.choice([32, 64]), dtype="f32" if f32 else "bf16",
                    page=rng.choice([0, 16, 64, 64, 128]), offset=rng.choice([0, _log(rng, 1, 131072)]))
    if op == "prefix":
        f32 = rng.random() < 0.2
        q = rng.randint(1, 4)
        b = _log(rng, 1, 16 if f32 else 128)
        h = 8 * (rng.randint(1, 2) if f32 else _log(rng, 1, 16))
        hi = _log(rng, 1, 100 if f32 else 1024)
        # at most the work of the largest listed case of the type
        cap = 2.5e5 if f32 else 6.0e7
        prefix = max(0, min(_log(rng, 1, 2048 if f32 else 131072), int(cap / (b * h * q)) - hi))
        return dict(op=op, B=b, H=h, Q=q, Dr=rng.choice([32, 64]) if f32 else 64, dtype="f32" if f32 else "bf16",
                    prefix=prefix, len_lo=min(q, hi), len_hi=hi, page=rng.choice([0, 64, 64, 128]),
                    causal=rng.randint(0, 1))
    grouped = rng.random() < 0.4
    if grouped:
        g = rng.choice([2, 4, 8])
        return dict(op=op, B=_log(rng, 1, 32), H=g * rng.randint(1, 8), Q=rng.randint(1, 2), G=g,
                    R=_log(rng, 1, 1024), grouped=1)
    return dict(op=op, B=_log(rng, 1, 64), H=rng.randint(1, 32), Q=1, G=1, R=_log(rng, 1, 7168), grouped=0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], both ends among them."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _shuffled(values, seed, salt):
    g = torch.Generator().manual_seed(seed * 1000003 + salt)
    return [values[i] for i in torch.randperm(len(values), generator=g).tolist()]


def _dt(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _pages(lens, page, perm):
    """(B, most pages) int32 table of the pages perm gives out in turn, -1 where a sequence has none."""
    need = [(n + page - 1) // page for n in lens]
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    k = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[k:k + n]
        k += n
    return table


def _count(lens, page):
    return sum((n + page - 1) // page for n in lens)


def _prepare_append(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt, B, H, Dr = _dt(case), case["B"], case["H"], case["Dr"]
    # new and cached tokens of a sequence, paired before the shuffle: the pool's size is the case's
    pairs = zip(_spread(case["new_lo"], case["new_hi"], B), reversed(_spread(case["past_lo"], case["past_hi"], B)))
    new, past = zip(*_shuffled(list(pairs), seed, 1))
    lens = [p + n for p, n in zip(past, new)]
    N = sum(new)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dt)

    st = dict(case=case, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    # the latent projection's output rows hold the latent, then the position part;
    # the query projection's rows hold each head's content part, then its position part
    st["kv_a"] = normal(N, CKV + Dr)
    st["q"] = normal(N, H, 128 + Dr)
    page = case["page"]
    if page:
        total = max(1, _count(lens, page))
        perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        st["table"] = _pages(lens, page, perm).cuda()
        rows = normal(total, page, CKV + Dr)         # one row per token: latent then position part
    else:
        rows = normal(B, max(1, max(lens)), CKV + Dr)
    st["kv"], st["pe"] = rows[..., :CKV], rows[..., CKV:]
    if not case["Q"]:
        cu = torch.tensor((0,) + new, dtype=torch.int32).cumsum(0).to(torch.int32)
        st["cu"] = cu.cuda()
    return st


def _prepare_prefix(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt, B, H, Q, Dr = _dt(case), case["B"], case["H"], case["Q"], case["Dr"]
    lens = _shuffled(_spread(case["len_lo"], case["len_hi"], B), seed, 2)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dt)

    # an absorbed query (128 products with weights of 1/sqrt(512)) and the usual
    # score scale: logits of standard deviation near 1.5
    st = dict(case=case, scale=1.0 / math.sqrt(128 + Dr), seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
              q_lat=normal(B, H, Q, CKV, scale=0.8), q_pe=normal(B, H, Q, Dr))
    page, Lp = case["page"], case["prefix"]
    if page:
        total = max(1, _count([Lp], page) + _count(lens, page))
        perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        rows = normal(total, page, CKV + Dr)
        st["prefix_table"] = _pages([Lp], page, perm)[0].cuda()
        st["table"] = _pages(lens, page, perm[_count([Lp], page):]).cuda()
        st["pkv"] = st["kv"] = rows[..., :CKV]
        st["ppe"] = st["pe"] = rows[..., CKV:]
    else:
        rows = normal(Lp, CKV + Dr)
        st["pkv"], st["ppe"] = rows[:, :CKV], rows[:, CKV:]
        rows = normal(B, max(1, max(lens)), CKV + Dr)
        st["kv"], st["pe"] = rows[..., :CKV], rows[..., CKV:]
    return st


def _prepare_fp4(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    B, H, Q, G, R = (case[k] for k in ("B", "H", "Q", "G", "R"))
    blocks = H // G
    x = torch.randn((B, H, Q, CKV), generator=gen, device="cuda").to(torch.bfloat16)
    # codes of all sixteen values; scales over the range that group maxima of
    # normal weights take once the largest is brought near the format's end
    codes = torch.randint(0, 256, (G, R, blocks, CKV // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(0x58, 0x7F, (G, R, blocks, CKV // 16), generator=gen, device="cuda", dtype=torch.uint8)
    w = torch.cat([codes, scales], dim=-1)
    scale = 1.0 / (200.0 * 3.0 * math.sqrt(blocks * CKV))
    if not case["grouped"]:
        x, w = x.reshape(B * Q, H * CKV), w[0]
    return dict(case=case, x=x, w=w, scale=scale)


def prepare(case, seed):
    return dict(append=_prepare_append, prefix=_prepare_prefix, fp4=_prepare_fp4)[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _run_append(st):
    case = st["case"]
    B, Q, H, Dr = case["B"], case["Q"], case["H"], case["Dr"]
    kv_a, q_pe = st["kv_a"], st["q"][..., 128:]
    c_kv, k_pe = kv_a[:, :CKV], kv_a[:, CKV:]
    page, table, cu = case["page"], st.get("table"), st.get("cu")
    if own:
        from latent_kv_decode_b200 import ops
        kw = dict(block_table=table, page_size=page or 64, pos_offset=case["offset"], rope_theta=THETA)
        if cu is None:
            q = ops.mla_rope_append(c_kv.unflatten(0, (B, Q)), k_pe.unflatten(0, (B, Q)), st["kv"], st["pe"],
                                    st["seq_lens"], q_pe=q_pe.unflatten(0, (B, Q)), **kw)
        else:
            q = ops.mla_rope_append(c_kv, k_pe, st["kv"], st["pe"], st["seq_lens"], q_pe=q_pe, cu_tokens=cu, **kw)
        return dict(kv=st["kv"], pe=st["pe"], q=q)
    N = kv_a.shape[0]
    n = torch.arange(N, device="cuda")
    if cu is None:
        b = n // Q
        t = st["seq_lens"].long()[b] - Q + n % Q
    else:
        b = torch.searchsorted(cu[1:].long(), n, right=True)
        t = st["seq_lens"].long()[b] - (cu.long()[b + 1] - n)
    freq = THETA ** (-torch.arange(0, Dr, 2, device="cuda", dtype=torch.float64) / Dr)
    ang = (t + case["offset"]).double()[:, None] * freq
    cos, sin = ang.cos().float(), ang.sin().float()

    def rotate(v, c, s):
        e, o = v[..., 0::2].float(), v[..., 1::2].float()
        return torch.stack([e * c - o * s, e * s + o * c], dim=-1).flatten(-2).to(v.dtype)

    if page:
        b, t = table[b, t // page].long(), t % page
    st["kv"][b, t] = c_kv
    st["pe"][b, t] = rotate(k_pe, cos, sin)
    q = rotate(q_pe, cos[:, None], sin[:, None])
    if cu is None:
        q = q.unflatten(0, (B, Q)).transpose(1, 2).contiguous()
    return dict(kv=st["kv"], pe=st["pe"], q=q)


def _rows(pool, table, n, page):
    """Rows 0..n-1 of a paged sequence."""
    t = torch.arange(n, device="cuda")
    return pool[table[t // page].long(), t % page]


def _run_prefix(st):
    case = st["case"]
    B, H, Q, page, Lp = case["B"], case["H"], case["Q"], case["page"], case["prefix"]
    if own:
        from latent_kv_decode_b200 import ops
        x, lse = ops.mla_prefix_decode(st["q_lat"], st["q_pe"], st["pkv"], st["ppe"], st["kv"], st["pe"], st["scale"],
                                       prefix_len=Lp, prefix_table=st.get("prefix_table"), seq_lens=st["seq_lens"],
                                       block_table=st.get("table"), page_size=page or 64, causal=bool(case["causal"]))
        return dict(x=x, lse=lse)
    pk, pp, kv, pe = st["pkv"], st["ppe"], st["kv"], st["pe"]
    L = case["len_hi"] if page else kv.shape[1]
    if page:
        pk, pp = (_rows(t, st["prefix_table"], Lp, page) for t in (pk, pp))
        t = torch.arange(L, device="cuda")
        idx = st["table"][:, t // page].long().clamp(min=0)
        kv, pe = (r[idx, t % page] for r in (kv, pe))
    prefix = torch.cat([pk, pp], -1).float()
    own_rows = torch.cat([kv, pe], -1).float()
    q = torch.cat([st["q_lat"], st["q_pe"]], -1).float().reshape(B, H * Q, -1)
    s = torch.cat([q @ prefix.T, q @ own_rows.transpose(1, 2)], -1) * st["scale"]
    t = torch.arange(Lp + L, device="cuda")
    end = (Lp + st["seq_lens"].long())[:, None, None]
    visible = t < end
    if case["causal"]:
        row_q = torch.arange(H * Q, device="cuda") % Q
        visible = visible & (t <= end - Q + row_q[:, None])
    s = s.masked_fill_(~visible, -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    x = p[..., :Lp] @ prefix[:, :CKV] + p[..., Lp:] @ own_rows[..., :CKV]
    x = (x / total).nan_to_num_(0.0)                      # a row that sees nothing gives zeros
    lse = (top + total.log()).squeeze(-1)
    return dict(x=x.to(_dt(case)).reshape(B, H, Q, CKV), lse=lse.reshape(B, H, Q))


def _weights(w, dtype):
    """The values that (..., blocks, 288) entries stand for, (..., blocks * 512)."""
    code, scale = w[..., :CKV // 2], w[..., CKV // 2:]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device="cuda")
    v = torch.stack([table[(code & 15).int()], table[(code >> 4).int()]], -1)       # channels 2i, 2i + 1
    s = scale.contiguous().view(torch.float8_e4m3fn).to(dtype)
    v = v.reshape(*scale.shape, 16) * s[..., None]
    return v.flatten(-3)


def _run_fp4(st):
    case, x, w = st["case"], st["x"], st["w"]
    if own:
        from latent_kv_decode_b200 import ops
        if case["grouped"]:
            return ops.mla_fp4_group_wo(x, w, scale_a=st["scale"])
        return ops.mla_fp4_linear(x, w, scale=st["scale"])
    wf = _weights(w, torch.float32)
    if not case["grouped"]:
        return (x.float() @ wf.T * st["scale"]).to(x.dtype)
    B, H, Q, G = (case[k] for k in ("B", "H", "Q", "G"))
    u = x.float().reshape(B, G, H // G, Q, CKV).permute(1, 0, 3, 2, 4).reshape(G, B * Q, -1)
    z = (u @ wf.transpose(1, 2) * st["scale"]).to(x.dtype)
    return z.permute(1, 0, 2).reshape(B, Q, -1)


def run(state):
    return dict(append=_run_append, prefix=_run_prefix, fp4=_run_fp4)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "fp4":
        T, G, K, R = case["B"] * case["Q"], case["G"], case["H"] // case["G"] * CKV, case["R"]
        return dict(bytes=G * R * (K // CKV) * ENTRY + 2 * T * G * (K + R), flops=2 * T * G * R * K)
    B, H, Dr, esz = case["B"], case["H"], case["Dr"], 4 if case["dtype"] == "f32" else 2
    if case["op"] == "append":
        N = sum(_spread(case["new_lo"], case["new_hi"], B))
        return dict(bytes=2 * N * (CKV + Dr + H * Dr) * esz, flops=3 * N * Dr * (1 + H))
    Lp, total, rows = case["prefix"], sum(_spread(case["len_lo"], case["len_hi"], B)), H * case["Q"]
    return dict(bytes=(Lp + total) * (CKV + Dr) * esz + B * rows * ((2 * CKV + Dr) * esz + 4),
                flops=2 * rows * (B * Lp + total) * (2 * CKV + Dr))


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_append(case, st):
    kv, pe = st["kv"].double(), st["pe"].double()
    B, Q, H, Dr, page = case["B"], case["Q"], case["H"], case["Dr"], case["page"]
    lens = st["seq_lens"].tolist()
    starts = st["cu"].tolist() if not Q else [Q * b for b in range(B + 1)]
    q = st["q"][..., 128:].double()
    turn = torch.tensor([THETA ** (-2.0 * j / Dr) for j in range(Dr // 2)], dtype=torch.float64, device="cuda")
    out = torch.empty_like(q)
    for b in range(B):
        n0, n1 = starts[b], starts[b + 1]
        if n0 == n1:
            continue
        t = torch.arange(lens[b] - (n1 - n0), lens[b], device="cuda")
        # a pair is a complex number turned by exp(i angle)
        phase = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), (t + case["offset"])[:, None] * turn)
        k = torch.view_as_complex(st["kv_a"][n0:n1, CKV:].double().unflatten(-1, (-1, 2)).contiguous()) * phase
        z = torch.view_as_complex(q[n0:n1].unflatten(-1, (-1, 2)).contiguous()) * phase[:, None]
        out[n0:n1] = torch.view_as_real(z).flatten(-2)
        where = (st["table"][b, t // page].long(), t % page) if page else (torch.full_like(t, b), t)
        kv[where] = st["kv_a"][n0:n1, :CKV].double()
        pe[where] = torch.view_as_real(k).flatten(-2)
    if Q:
        out = out.reshape(B, Q, H, Dr).permute(0, 2, 1, 3)
    return dict(kv=kv, pe=pe, q=out)


def _exact_prefix(case, st):
    B, H, Q, page, Lp = case["B"], case["H"], case["Q"], case["page"], case["prefix"]
    lens = st["seq_lens"].tolist()
    x = torch.zeros((B, H, Q, CKV), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Q), -math.inf, dtype=torch.float64, device="cuda")
    shared = [_rows(st[n], st["prefix_table"], Lp, page) if page else st[n] for n in ("pkv", "ppe")]
    for b in range(B):
        rows = [_rows(st[n], st["table"][b], lens[b], page) if page else st[n][b, :lens[b]] for n in ("kv", "pe")]
        k = torch.cat([torch.cat(r) for r in zip(shared, rows)], -1).double()      # (Lp + len, 512 + Dr)
        for i in range(Q):
            n = k.shape[0] - Q + i + 1 if case["causal"] else k.shape[0]
            if n <= 0:
                continue
            query = torch.cat([st["q_lat"][b, :, i], st["q_pe"][b, :, i]], -1).double()
            logit = torch.einsum("hc,tc->ht", query, k[:n]) * st["scale"]
            lse[b, :, i] = torch.logsumexp(logit, -1)
            x[b, :, i] = torch.exp(logit - lse[b, :, i, None]) @ k[:n, :CKV]
    return dict(x=x, lse=lse)


def _exact_fp4(case, st):
    B, H, Q, G = (case[k] for k in ("B", "H", "Q", "G"))
    w = st["w"] if case["grouped"] else st["w"][None]
    x = st["x"].double().reshape(B, H, Q, CKV)
    z = []
    for g in range(G):
        e = w[g]
        nib = torch.stack([e[..., :CKV // 2] % 16, e[..., :CKV // 2] // 16], -1).flatten(-2).double()
        mag = nib % 8
        # exponent 0 counts halves; above it the value is (1 + m / 2) 2^(e - 1)
        val = torch.where(mag < 2, mag / 2, (1 + (mag % 2) / 2) * 2.0 ** (torch.floor(mag / 2) - 1))
        byte = e[..., CKV // 2:].double()
        m, ex = byte % 8, torch.floor(byte / 8) % 16
        sc = torch.where(ex == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (ex - 7))
        val = torch.where(nib >= 8, -val, val) * torch.where(byte >= 128, -sc, sc).repeat_interleave(16, -1)
        y = 0.0
        for i in range(H // G):
            y = y + torch.einsum("bqc,rc->bqr", x[:, g * (H // G) + i], val[:, i])
        z.append(y * st["scale"])
    z = torch.cat(z, -1)
    return z if case["grouped"] else z.reshape(B * Q, -1)


def exact(case, seed):
    st = prepare(case, seed)
    return dict(append=_exact_append, prefix=_exact_prefix, fp4=_exact_fp4)[case["op"]](case, st)
