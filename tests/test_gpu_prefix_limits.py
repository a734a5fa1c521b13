"""mla_prefix_decode at the ends of its range, against the formula in 64 bits: token
counts beyond 32 bits, long prefixes, sinks and scores of -inf, causal rows that end
before the prefix does.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

C, DR = 512, 64
HALF = torch.finfo(torch.bfloat16).eps / 2     # of a rounding to bf16


def _attend(q, k, scale, sink=None):
    """Rows of q (n, C + DR) over the tokens k (t, C + DR), both float64: x, lse, sum_t p_t |v_t|."""
    s = q @ k.T * scale
    if sink is not None:
        s = torch.cat([s, sink[:, None]], 1)
        k = torch.cat([k, torch.zeros_like(k[:1])])
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    return p @ k[:, :C], lse, p @ k[:, :C].abs()


def test_a_block_of_more_than_2_to_the_31_tokens():
    # sixteen sequences of one block, 2^27 + 2^22 own tokens each, all in one page that their
    # tables repeat; the mask leaves the prefix's first 100 tokens and the last 200
    from latent_kv_decode_b200 import ops
    B, H, page, Lp, n = 16, 8, 4096, 128, 2 ** 27 + 2 ** 22
    g = torch.Generator("cuda").manual_seed(51)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    pool, q = r(2, page, C + DR), r(B, H, 1, C + DR) * 0.8
    mask = torch.zeros(Lp + n, dtype=torch.uint8, device="cuda")
    mask[:100] = 1
    mask[-200:] = 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, lse = ops.mla_prefix_decode(q[..., :C].contiguous(), q[..., C:].contiguous(), pool[..., :C], pool[..., C:],
                                   pool[..., :C], pool[..., C:], 0.07, prefix_len=Lp,
                                   prefix_table=torch.zeros(1, dtype=torch.int32, device="cuda"), page_size=page,
                                   block_table=torch.ones((B, n // page), dtype=torch.int32, device="cuda"),
                                   causal_mask=mask, err_flag=err)
    assert int(err.item()) == 0
    k = torch.cat([pool[0, :100], pool[1, -200:]]).double()
    want, want_lse, size = _attend(q.double().reshape(B * H, -1), k, 0.07)
    # a weight and x are rounded once to bf16; 300 float32 additions of either sum
    tol = HALF * (size + want.abs()) + 300 * 2.0 ** -23 * size
    assert ((x.double().reshape(B * H, C) - want).abs() <= tol).all()
    # scores are float32 sums of 576 products
    at = 576 * 2.0 ** -24 * (q.double().abs().reshape(B * H, -1) @ k.abs().T).amax(1) * 0.07 + 300 * 2.0 ** -24
    assert ((lse.double().reshape(-1) - want_lse).abs() <= at).all()


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sinks_of_minus_infinity(dtype, splits):
    # such a sink adds nothing: rows that see nothing give x = 0 and lse = -inf, the others
    # what they give without it
    from latent_kv_decode_b200 import ops
    B, H = 3, 16
    g = torch.Generator("cuda").manual_seed(52)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    q_lat, q_pe, own = r(B, H, 1, C), r(B, H, 1, DR), r(B, 70, C + DR)
    lens = torch.tensor([0, 70, 1], dtype=torch.int32, device="cuda")
    call = lambda sinks: ops.mla_prefix_decode(q_lat, q_pe, None, None, own[..., :C], own[..., C:], 0.07, seq_lens=lens,
                                               sinks=sinks, num_splits=splits)
    bare = call(None)
    off = call(torch.full((H,), -math.inf, device="cuda"))
    half = torch.randn(H, generator=g, device="cuda")
    some = call(half)
    half[::2] = -math.inf
    both = call(half)
    assert (bare[0][0] == 0).all() and (bare[1][0] == -math.inf).all()
    for got, want in ((off, bare), ([t[:, ::2] for t in both], [t[:, ::2] for t in bare]),
                      ([t[:, 1::2] for t in both], [t[:, 1::2] for t in some])):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_first_score_of_minus_infinity(dtype, splits, page):
    # the prefix's one token has +inf in a position channel: rows with a negative query there
    # give it the weight e^-inf = 0 and go on, rows with a positive one are NaN
    from latent_kv_decode_b200 import ops
    B, H, n = 3, 16, 40
    g = torch.Generator("cuda").manual_seed(53)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    q, own, first = r(B, H, 1, C + DR), r(B, n, C + DR), r(1, C + DR)
    first[0, C + 5] = math.inf
    kw = dict(num_splits=splits)
    if page:
        per = -(-n // page)
        pool = torch.zeros((B * per + 1, page, C + DR), dtype=dtype, device="cuda")
        pool[0, 0] = first[0]
        pool[1:].view(B, per * page, -1)[:, :n] = own
        table = torch.arange(1, B * per + 1, dtype=torch.int32, device="cuda").view(B, per)
        kw.update(prefix_len=1, prefix_table=torch.zeros(1, dtype=torch.int32, device="cuda"), block_table=table,
                  page_size=page, seq_lens=torch.full((B,), n, dtype=torch.int32, device="cuda"))
        prefix = own_rows = pool
    else:
        prefix, own_rows = first, own
    x, lse = ops.mla_prefix_decode(q[..., :C].contiguous(), q[..., C:].contiguous(), prefix[..., :C], prefix[..., C:],
                                   own_rows[..., :C], own_rows[..., C:], 0.07, **kw)
    lost = q[:, :, 0, C + 5] > 0
    assert lost.any() and not lost.all()
    assert torch.isnan(x[:, :, 0][lost]).all() and torch.isnan(lse[..., 0][lost]).all()
    for b in range(B):
        k = own[b].double()
        want, want_lse, size = _attend(q[b, :, 0].double(), k, 0.07)
        # float32 sums of 576 products shift a weight by e^at; bf16 rounds weights and x once more
        at = 2 * 576 * 2.0 ** -24 * (q[b, :, 0].double().abs() @ k.abs().T).amax(1) * 0.07 + n * 2.0 ** -23
        tol = at[:, None] * size + (HALF * (size + want.abs()) if dtype == torch.bfloat16 else 0)
        keep = ~lost[b]
        assert ((x[b, :, 0].double() - want).abs() <= tol)[keep].all()
        assert ((lse[b, :, 0].double() - want_lse).abs() <= at)[keep].all()


@pytest.mark.parametrize("Lp,lens", [(128, [0, 1, 2, 3]), (256, [3, 0, 4, 9]), (256, [2, 4, 9, 200])])
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_bad_last_prefix_row_stays_hidden_from_causal_rows(dtype, bad, splits, page, Lp, lens):
    # fewer own tokens than queries: the first queries do not see the prefix's last row, which
    # ends a full tile and holds NaN or infinity in its latent part; the rows that see it are NaN
    from latent_kv_decode_b200 import ops
    B, H, Q = len(lens), 8, 4
    g = torch.Generator("cuda").manual_seed(54)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    q, own, prefix = r(B, H, Q, C + DR), r(B, max(lens), C + DR), r(Lp, C + DR)
    prefix[-1, 7] = bad
    kw = dict(seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), causal=True, num_splits=splits)
    a, b = prefix, own
    if page:
        n = Lp // page
        per = -(-max(lens) // page)
        pool = torch.zeros((n + B * per, page, C + DR), dtype=dtype, device="cuda")
        pool[:n] = prefix.view(n, page, -1)
        pool[n:].view(B, per * page, -1)[:, :max(lens)] = own
        i32 = lambda t: t.to(torch.int32).cuda()
        kw.update(prefix_len=Lp, prefix_table=i32(torch.arange(n)), page_size=page,
                  block_table=i32(torch.arange(n, n + B * per).view(B, per)))
        a = b = pool
    x, lse = ops.mla_prefix_decode(q[..., :C].contiguous(), q[..., C:].contiguous(), a[..., :C], a[..., C:], b[..., :C],
                                   b[..., C:], 0.07, **kw)
    hidden = 0
    for s in range(B):
        k = torch.cat([prefix, own[s, :lens[s]]]).double()
        for i in range(Q):
            n = Lp + lens[s] - Q + i + 1
            qq = q[s, :, i].double()
            if n >= Lp:
                seen = q[s, :, i, 7] > 0 if bad == math.inf else torch.ones(H, dtype=torch.bool, device="cuda")
                assert torch.isnan(x[s, :, i][seen]).all() and torch.isnan(lse[s, :, i][seen]).all()
                continue
            hidden += 1
            want, want_lse, size = _attend(qq, k[:n], 0.07)
            at = 2 * 576 * 2.0 ** -24 * (qq.abs() @ k[:n].abs().T).amax(1) * 0.07 + n * 2.0 ** -23
            tol = at[:, None] * size + (HALF * (size + want.abs()) if dtype == torch.bfloat16 else 0)
            assert ((x[s, :, i].double() - want).abs() <= tol).all()
            assert ((lse[s, :, i].double() - want_lse).abs() <= at).all()
    assert hidden > 0


@pytest.mark.parametrize("page", [0, 16])
def test_float32_over_a_long_prefix_in_one_range(page):
    # Values of nonzero mean, so that O grows with every one of the 8192 tiles of 16 tokens.
    # Rounded sums: errors of either sign, of which n are within 7 sqrt(n) 2^-24 but for one in
    # 10^10 (Higham and Mary, 2019), for O and for the denominator; a tile's own products, a
    # few truncations of 2^-23 each; the scores, sums of 576 products, are small here.
    from latent_kv_decode_b200 import ops
    H, Lp = 8, 131072
    g = torch.Generator("cuda").manual_seed(55)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    q, rows = r(1, H, 1, C + DR) * 0.01, r(Lp, C + DR) * 0.5 + 1.0
    kw = dict(num_splits=1)
    k = rows
    if page:
        perm = torch.randperm(Lp // page, generator=torch.Generator().manual_seed(5)).cuda()
        pool = torch.empty((Lp // page, page, C + DR), device="cuda")
        pool[perm] = rows.view(-1, page, C + DR)
        kw.update(prefix_len=Lp, prefix_table=perm.to(torch.int32), page_size=page)
        rows = pool
    x, lse = ops.mla_prefix_decode(q[..., :C].contiguous(), q[..., C:].contiguous(), rows[..., :C], rows[..., C:], None,
                                   None, 0.07, **kw)
    qq, k = q[0, :, 0].double(), k.double()
    want, want_lse, size = _attend(qq, k, 0.07)
    at = 576 * 2.0 ** -24 * (qq.abs() @ k.abs().T).amax(1) * 0.07
    sums = 7 * math.sqrt(Lp / 16) * 2.0 ** -24
    tol = (2 * sums + 16 * 2.0 ** -23 + 2 * at)[:, None] * size
    err = (x[0, :, 0].double() - want).abs()
    assert (err <= tol).all(), f"{(err / size).max().item():.2e} of the values"
    assert ((lse[0, :, 0].double() - want_lse).abs() <= at + sums + 2.0 ** -23 * want_lse.abs()).all()


@pytest.mark.parametrize("splits", [0, 1, 5])
@pytest.mark.parametrize("Lp,B,H,Q,lens", [(131072, 1, 128, 1, [130]), (16384, 16, 16, 2, [2, 40, 129, 511] * 4),
                                           (4097, 2, 128, 1, [1, 500])])
def test_bf16_over_long_prefixes(Lp, B, H, Q, lens, splits):
    # the sizes the call is made for, paged, every row against 64 bits. A weight and x are
    # rounded once to bf16; O is a sum of one addition per 16 tokens (at most 2^-23 each, a
    # truncation), the denominator one per tile and thread
    from latent_kv_decode_b200 import ops
    g = torch.Generator("cuda").manual_seed(56)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    page, n, per = 64, -(-Lp // 64), -(-max(lens) // 64)
    perm = torch.randperm(n + B * per, generator=torch.Generator().manual_seed(6)).to(torch.int32).cuda()
    pool, q = r(n + B * per, page, C + DR), r(B, H, Q, C + DR) * 0.8
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, lse = ops.mla_prefix_decode(q[..., :C].contiguous(), q[..., C:].contiguous(), pool[..., :C], pool[..., C:],
                                   pool[..., :C], pool[..., C:], 0.07, prefix_len=Lp, prefix_table=perm[:n],
                                   block_table=perm[n:].view(B, per).contiguous(), causal=True, num_splits=splits,
                                   seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), err_flag=err)
    assert int(err.item()) == 0
    flat = lambda ids, m: pool[ids.long()].flatten(0, 1)[:m].double()
    prefix = flat(perm[:n], Lp)
    for b in range(B):
        k = torch.cat([prefix, flat(perm[n:].view(B, per)[b], lens[b])])
        for i in range(Q):
            seen = Lp + lens[b] - Q + i + 1
            qq = q[b, :, i].double()
            want, want_lse, size = _attend(qq, k[:seen], 0.07)
            at = 576 * 2.0 ** -24 * (qq.abs() @ k.abs().T).amax(1) * 0.07
            tol = HALF * (size + want.abs()) + ((seen / 16) * 2.0 ** -23 + 2 * at[:, None]) * size
            assert ((x[b, :, i].double() - want).abs() <= tol).all()
            assert ((lse[b, :, i].double() - want_lse).abs() <= at + seen / 128 * 2.0 ** -24 + 2.0 ** -22 * want_lse.abs()).all()


@pytest.mark.parametrize("H,B", [(128, 40), (16, 300)])
def test_bf16_sums_over_two_million_tokens(H, B):
    # more blocks of rows than clusters, so that speed alone asks for one range; values of
    # nonzero mean. A weight and x are rounded once to bf16, and O is a sum of at most 2^14
    # additions a range (one per 16 tokens, a truncation of at most 2^-23), merged by rounding ones
    from latent_kv_decode_b200 import ops
    n, pages, page = 2 ** 21, 64, 64
    g = torch.Generator("cuda").manual_seed(57)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    pool, q = (r(pages, page, C + DR) * 0.5 + 1).bfloat16(), (r(B, H, 1, C + DR) * 0.01).bfloat16()
    table = (torch.arange(n // page, device="cuda") % pages).to(torch.int32)
    x, lse = ops.mla_prefix_decode(q[..., :C].contiguous(), q[..., C:].contiguous(), pool[..., :C], pool[..., C:], None,
                                   None, 0.07, prefix_len=n, prefix_table=table)
    k, qq = pool.flatten(0, 1).double(), q.double().reshape(B * H, -1)
    want, want_lse, size = _attend(qq, k, 0.07)                  # every row as often: the same weights
    at = 576 * 2.0 ** -24 * (qq.abs() @ k.abs().T).amax(1) * 0.07
    tol = HALF * (size + want.abs()) + (2.0 ** 14 * 2.0 ** -23 + 2 * at[:, None]) * size
    err = (x.double().reshape(B * H, C) - want).abs()
    assert (err <= tol).all(), f"{(err / size).max().item():.2e} of the values"
    want_lse = want_lse + math.log(n / len(k))
    assert ((lse.double().reshape(-1) - want_lse).abs() <= at + 2.0 ** 14 * 2.0 ** -24 + 2.0 ** -22 * want_lse).all()


@pytest.mark.parametrize("dtype,page", [(torch.float32, 64), (torch.bfloat16, 64), (torch.bfloat16, 16)])
@pytest.mark.parametrize("B,H,Lp,longest", [(4, 8, 256, 500), (4, 16, 100, 3), (3, 128, 700, 130), (40, 128, 300, 200)])
def test_tables_that_allow_more_than_the_lengths_use(B, H, Lp, longest, dtype, page):
    # a block takes the ranges that its lengths ask for, whatever the table allows, and the
    # others leave nothing behind. Some sequences are empty, and the tables' other entries
    # are no pages
    from latent_kv_decode_b200 import ops
    g = torch.Generator("cuda").manual_seed(58)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    lens = [longest * (b % 4) // 3 for b in range(B)]
    n, per = -(-Lp // page), -(-longest // page)
    pool, q_lat, q_pe = r(n + B * per, page, C + DR), r(B, H, 1, C), r(B, H, 1, DR)
    tight = torch.arange(n, n + B * per, dtype=torch.int32, device="cuda").view(B, per)
    prefix_table = torch.arange(n, dtype=torch.int32, device="cuda")

    def call(capacity, **kw):
        table = torch.full((B, capacity // page), -1, dtype=torch.int32, device="cuda")
        table[:, :per] = tight
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = ops.make_prefix_decode(q_lat, q_pe, pool[..., :C], pool[..., C:], pool[..., :C], pool[..., C:], 0.07,
                                    prefix_len=Lp, prefix_table=prefix_table, page_size=page, block_table=table,
                                    seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), err_flag=err, **kw)
        if ws.workspace is not None:
            ws.workspace.fill_(0x7F)                     # what is not written this time must not be read
        ws.x.fill_(math.nan)
        ws.lse.fill_(math.nan)
        x, lse = ops.launch_prefix_decode(ws)
        assert int(err.item()) == 0
        return x, lse

    half = HALF if dtype == torch.bfloat16 else 0
    oracle = {}
    for b in {0, 1, 2, 3 % B, B - 1}:
        k = torch.cat([pool[:n].flatten(0, 1)[:Lp], pool[n + b * per:n + (b + 1) * per].flatten(0, 1)[:lens[b]]]).double()
        q = torch.cat([q_lat[b, :, 0], q_pe[b, :, 0]], -1).double()
        at = 576 * 2.0 ** -24 * (q.abs() @ k.abs().T).amax(1) * 0.07
        oracle[b] = (*_attend(q, k, 0.07), at)
    for capacity in (per * page, 131072, 2 ** 19):
        x, lse = call(capacity)
        assert torch.isfinite(x).all() and torch.isfinite(lse).all()
        for b, (want, want_lse, size, at) in oracle.items():
            # roundings to bf16; float32 sums and exponentials of a few hundred tokens
            tol = half * (size + want.abs()) + (2 * at[:, None] + 2.0 ** -15) * size
            assert ((x[b, :, 0].double() - want).abs() <= tol).all(), f"capacity {capacity}, sequence {b}"
            assert ((lse[b, :, 0].double() - want_lse).abs() <= at + 2.0 ** -15).all()


@pytest.mark.parametrize("dtype,page", [(torch.float32, 64), (torch.bfloat16, 64), (torch.bfloat16, 16)])
@pytest.mark.parametrize("sinks", [False, True])
def test_empty_sequences_with_large_tables(dtype, page, sinks):
    # blocks without a token beside blocks with some: one range each, or several, in one call
    from latent_kv_decode_b200 import ops
    B, H, capacity = 24, 16, 65536
    g = torch.Generator("cuda").manual_seed(59)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    lens = [0] * 16 + [0, 700, 1, 0, 64, 0, 0, 130]
    pool, q_lat, q_pe = r(44 * 64 // page, page, C + DR), r(B, H, 1, C), r(B, H, 1, DR)
    table = torch.full((B, capacity // page), -1, dtype=torch.int32, device="cuda")
    used = 0
    rows = {}
    for b, n in enumerate(lens):
        need = -(-n // page)
        table[b, :need] = torch.arange(used, used + need, device="cuda")
        rows[b] = pool[used:used + need].flatten(0, 1)[:n].double()
        used += need
    sink = torch.randn(H, generator=g, device="cuda") if sinks else None
    x, lse = ops.mla_prefix_decode(q_lat, q_pe, None, None, pool[..., :C], pool[..., C:], 0.07, block_table=table,
                                   page_size=page, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), sinks=sink)
    for b, n in enumerate(lens):
        if n == 0:
            assert (x[b] == 0).all()
            want = sink if sinks else torch.full((H,), -math.inf, device="cuda")
            # e^(sink - sink) and its logarithm, or log2 and back: float32 on either way
            assert torch.allclose(lse[b, :, 0], want, rtol=2.0 ** -21, atol=2.0 ** -21)
            continue
        q = torch.cat([q_lat[b, :, 0], q_pe[b, :, 0]], -1).double()
        want, want_lse, size = _attend(q, rows[b], 0.07, sink.double() if sinks else None)
        at = 576 * 2.0 ** -24 * (q.abs() @ rows[b].abs().T).amax(1) * 0.07
        half = HALF if dtype == torch.bfloat16 else 0
        tol = half * (size + want.abs()) + (2 * at[:, None] + 2.0 ** -15) * size
        assert ((x[b, :, 0].double() - want).abs() <= tol).all(), f"sequence {b}"
        assert ((lse[b, :, 0].double() - want_lse).abs() <= at + 2.0 ** -15).all()


@pytest.mark.parametrize("dtype,page", [(torch.float32, 64), (torch.bfloat16, 64), (torch.bfloat16, 16)])
def test_a_captured_call_follows_its_lengths(dtype, page):
    # the ranges are cut on the device: one graph, replayed while sequences grow from nothing
    # to several tiles, gives the eager call's bits
    from latent_kv_decode_b200 import ops
    B, H, Lp, capacity = 6, 16, 100, 32768
    g = torch.Generator("cuda").manual_seed(60)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    pages = 1024 // page
    pool, q_lat, q_pe = r(B * pages + 128 // page, page, C + DR), r(B, H, 1, C), r(B, H, 1, DR)
    table = torch.full((B, capacity // page), -1, dtype=torch.int32, device="cuda")
    table[:, :pages] = torch.arange(B * pages, device="cuda").view(B, pages)
    prefix_table = torch.arange(B * pages, B * pages + 128 // page, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    call = lambda: ops.mla_prefix_decode(q_lat, q_pe, pool[..., :C], pool[..., C:], pool[..., :C], pool[..., C:], 0.07,
                                         prefix_len=Lp, prefix_table=prefix_table, page_size=page, block_table=table,
                                         seq_lens=lens)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x, lse = call()
    for step in ([0] * 6, [1, 0, 2, 0, 0, 3], [1024, 1, 130, 0, 700, 64], [0, 0, 0, 0, 0, 1], [1024] * 6):
        lens.copy_(torch.tensor(step, dtype=torch.int32))
        graph.replay()
        want, want_lse = call()
        torch.cuda.synchronize()
        assert torch.equal(x, want) and torch.equal(lse, want_lse), str(step)
        for b in range(B):
            k = torch.cat([pool[prefix_table.long()].flatten(0, 1)[:Lp], pool[table[b, :pages].long()].flatten(0, 1)[:step[b]]]).double()
            q = torch.cat([q_lat[b, :, 0], q_pe[b, :, 0]], -1).double()
            v, _, size = _attend(q, k, 0.07)
            at = 576 * 2.0 ** -24 * (q.abs() @ k.abs().T).amax(1) * 0.07
            half = HALF if dtype == torch.bfloat16 else 0
            assert ((x[b, :, 0].double() - v).abs() <= half * (size + v.abs()) + (2 * at[:, None] + 2.0 ** -15) * size).all()
