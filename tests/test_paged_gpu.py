"""GPU tests of the paged-cache calls (sampling step, append, accumulated weight, eviction) against the plain
64-bit implementation of tests/paged_reference.py.  Rows that no entry holds are NaN, table entries past an
entry's rows name no page.  Tolerances are derived there: one rounding to bf16 of the output plus the fp32
arithmetic of the scores; copies and choices are exact."""
import numpy as np
import pytest
import torch

from block_discrete_diffusion_tcgen05_b200 import _lib, attn
import paged_reference as R

pytestmark = pytest.mark.gpu

E2D2_ERR_TIMEOUT, E2D2_ERR_PAGE = 8, 10


def guarded(shape, dtype, fill):
    """A tensor inside a larger one whose margins hold `fill`; returns (tensor, check that they still do)."""
    n = int(np.prod(shape))
    pad = 4096
    big = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    same = big.clone()
    t = big[pad:pad + n].view(shape)

    def check():
        for a, b in ((big[:pad], same[:pad]), (big[pad + n:], same[pad + n:])):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), "written outside the output"

    return t, check


def run_sample(cache, Hq, S, block, seed, sigma=1.0, scale=None, workspace=None):
    B, Hkv, d = cache.B, cache.Hkv, cache.d
    q = R.bf16((B, Hq, S, d), seed, sigma)
    kb, vb = (R.bf16((B, Hkv, S, d), seed + 1, sigma), R.bf16((B, Hkv, S, d), seed + 2)) if block else (None, None)
    k, v, table, P = cache.cuda()
    out, check_o = guarded((B, Hq, S, d), torch.bfloat16, 7.0)
    lse, check_l = guarded((B, Hq, S), torch.float32, 7.0)
    out.fill_(float("nan"))
    lse.fill_(float("nan"))
    got = attn.decoder_sample_paged(q.cuda(), k, v, table, P, None if kb is None else kb.cuda(),
                                    None if vb is None else vb.cuda(), scale=scale, out=out, lse=lse, workspace=workspace)
    torch.cuda.synchronize()
    check_o()
    check_l()
    return got, R.sample(cache, q, kb, vb, scale)


CASES = [
    # B, Hq, Hkv, S, d, page, block, P
    (1, 1, 1, 1, 128, 16, True, [0]),                        # the first token of a sequence: only itself
    (1, 1, 1, 1, 32, 16, False, [1]),
    (2, 8, 2, 1, 128, 64, False, [0, 0]),                    # nothing to see anywhere
    (6, 16, 8, 1, 128, 16, True, [0, 1, 15, 16, 17, 700]),   # page ends on either side of the length
    (5, 8, 8, 1, 128, 64, True, [127, 128, 129, 64, 63]),    # tile ends, one query row per kv head
    (3, 21, 3, 1, 128, 48, True, [47, 48, 1000]),            # 7 query rows, pages of 48
    (2, 32, 2, 1, 128, 32, False, [300, 5]),                 # 16 rows
    (2, 34, 2, 1, 128, 32, True, [300, 5]),                  # 17 rows
    (4, 16, 8, 16, 128, 64, True, [5, 600, 256, 0]),         # blocks: 32 rows
    (2, 32, 8, 16, 128, 128, True, [700, 33]),               # 64 rows
    (2, 12, 4, 11, 128, 16, False, [259, 1]),                # 33 rows
    (2, 16, 2, 13, 128, 48, True, [300, 0]),                 # 104 rows
    (1, 16, 1, 16, 128, 64, True, [513]),                    # 256 rows: two tiles of queries
    (1, 3, 1, 43, 128, 64, True, [100]),                     # 129 rows
    (4, 8, 2, 16, 64, 16, True, [5, 600, 256, 0]),
    (3, 4, 4, 7, 64, 48, False, [299, 1, 130]),
    (2, 16, 2, 9, 64, 128, True, [400, 129]),                # 72 rows
    (3, 4, 4, 7, 32, 16, True, [299, 1, 130]),
    (2, 40, 2, 5, 32, 80, True, [161, 80]),                  # 100 rows
    (3, 16, 8, 1, 128, 0, True, [37, 611, 0]),               # contiguous caches, capacity 613
    (3, 12, 4, 7, 64, 0, False, [37, 613, 1]),
    (2, 8, 2, 16, 32, 0, True, [613, 600]),
    (70, 4, 2, 1, 64, 16, True, [(17 * i) % 97 for i in range(70)]),
    (45, 4, 2, 1, 128, 16, False, [(23 * i) % 301 for i in range(45)]),
    (2, 2, 2, 150, 128, 64, True, [200, 0]),                 # a long block: its own rows take two tiles
    (1, 2, 2, 150, 64, 16, True, [70]),
    (3, 8, 8, 1, 128, 128, True, [512, 512, 512]),           # equal lengths: whole units, or equal parts of them
    (40, 8, 8, 1, 128, 64, False, [128] * 40),               # more equal units than blocks
    (37, 8, 4, 2, 64, 32, True, [96] * 37),
]


@pytest.mark.parametrize("B,Hq,Hkv,S,d,page,block,P", CASES)
def test_sample_matches_the_formula(B, Hq, Hkv, S, d, page, block, P):
    cache = R.Cache(B, Hkv, d, page, P, max(max(P), 613 if page == 0 else 1), 5000 + 7 * B + d)
    got, ref = run_sample(cache, Hq, S, block, 5100 + S)
    R.check_sample(got, ref, f"B{B} Hq{Hq} Hkv{Hkv} S{S} d{d} page{page}")
    assert attn.last_device_error() == 0


@pytest.mark.parametrize("d,S", [(128, 1), (128, 16), (64, 5), (32, 16)])
def test_sample_sharp_softmax_and_large_values(d, S):
    cache = R.Cache(2, 2, d, 32, [400, 77], 400, 5200, sigma_k=4.0, sigma_v=64.0)
    got, ref = run_sample(cache, 8, S, True, 5210, sigma=3.0)
    R.check_sample(got, ref, f"sharp d{d} S{S}")


def test_sample_scale_and_junk_in_the_table():
    for junk in (-1, 2 ** 31 - 1, -2 ** 31, 1000):
        cache = R.Cache(3, 2, 128, 16, [33, 0, 250], 300, 5300, junk=junk)
        got, ref = run_sample(cache, 4, 3, True, 5310, scale=0.03)
        R.check_sample(got, ref, f"junk {junk}")
    assert attn.last_device_error() == 0


def test_sample_long_cache_split_over_the_gpu():
    """One head's cache of 20,011 rows: every SM takes a piece, the pieces are joined."""
    for S, page in ((1, 16), (16, 64)):
        cache = R.Cache(1, 1, 128, page, [20011], 20011, 5400)
        got, ref = run_sample(cache, 2, S, True, 5410)
        R.check_sample(got, ref, f"long S{S}")


def test_sample_matches_the_contiguous_call():
    """The same rows through a table, without one, and in the existing ragged call."""
    B, Hq, Hkv, S, d, cap = 4, 16, 8, 16, 128, 640
    P = [0, 640, 129, 500]
    q, kb, vb = R.bf16((B, Hq, S, d), 5500).cuda(), R.bf16((B, Hkv, S, d), 5501).cuda(), R.bf16((B, Hkv, S, d), 5502).cuda()
    k, v = R.bf16((B, Hkv, cap, d), 5503).cuda(), R.bf16((B, Hkv, cap, d), 5504).cuda()
    Pd = torch.tensor(P, dtype=torch.int32, device="cuda")
    ro, rl = attn.decoder_sample_ragged(q, k, v, Pd, kb, vb)
    co, cl = attn.decoder_sample_paged(q, k, v, None, Pd, kb, vb)
    page = 32
    each = cap // page
    perm = torch.from_numpy(np.random.default_rng(1).permutation(B * each)).cuda()
    kp, vp = (torch.empty(B * each, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for src, dst in ((k, kp), (v, vp)):
        dst[perm] = src.view(B, Hkv, each, page, d).transpose(1, 2).reshape(B * each, Hkv, page, d)
    po, pl = attn.decoder_sample_paged(q, kp, vp, perm.view(B, each).to(torch.int32).contiguous(), Pd, kb, vb)
    torch.cuda.synchronize()
    assert torch.equal(co, po) and torch.equal(cl, pl)   # the same rows in the same order
    assert (ro.float() - co.float()).abs().max().item() <= 2e-2
    assert (rl - cl).abs().max().item() <= 1e-3


def test_sample_lengths_outside_the_capacity_are_clamped():
    cache = R.Cache(3, 2, 64, 16, [64, 0, 64], 64, 5600)
    q = R.bf16((3, 4, 2, 64), 5601)
    k, v, table, _ = cache.cuda()
    P = torch.tensor([65, -3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    got = attn.decoder_sample_paged(q.cuda(), k, v, table, P)
    torch.cuda.synchronize()
    R.check_sample(got, R.sample(cache, q, None, None), "clamped lengths")


def test_bad_pages_are_left_out_and_reported():
    """A page id outside the pool below an entry's length: its rows take no part, nothing faults, and the
    device error names it; the next call is clean."""
    for S, page, bad in ((1, 16, -1), (16, 32, 99), (9, 48, 2 ** 31 - 1)):
        cache = R.Cache(2, 2, 128, page, [200, 150], 200, 5700)
        k, v, table, P = cache.cuda()
        table[0, 2] = bad
        q = R.bf16((2, 8, S, 128), 5701)
        skip = {(0, r) for r in range(2 * page, min(3 * page, 200))}
        got = attn.decoder_sample_paged(q.cuda(), k, v, table, P)
        torch.cuda.synchronize()
        assert attn.last_device_error() == E2D2_ERR_PAGE
        R.check_sample(got, R.sample(cache, q, None, None, skip=skip), f"bad page {bad}")
        w = torch.rand(2, 2, cache.capacity)
        ref_w, tol = R.weigh(cache, q, got[1].cpu(), w, skip=skip)
        out = attn.kv_cache_weigh(q.cuda(), k, table, P, got[1], w.cuda())
        torch.cuda.synchronize()
        assert attn.last_device_error() == E2D2_ERR_PAGE
        assert (np.abs(out.cpu().numpy() - ref_w) <= tol).all()
        kn = torch.ones(2, 2, 8, 128, dtype=torch.bfloat16, device="cuda")
        before = R.bits(k)
        table[0, 2] = bad
        attn.kv_cache_append_paged(k, v, table, torch.tensor([2 * page + 1, 0], dtype=torch.int32, device="cuda"), kn, kn)
        torch.cuda.synchronize()
        assert attn.last_device_error() == E2D2_ERR_PAGE
        after = R.bits(k)
        changed = np.argwhere((before != after).any(axis=(1, 3)))
        assert {tuple(x) for x in changed} <= {(int(cache.table[1, 0]), r) for r in range(8)}
        got = attn.decoder_sample_paged(q.cuda(), k, v, table, torch.tensor([page, 0], dtype=torch.int32, device="cuda"))
        assert attn.last_device_error() == 0


@pytest.mark.parametrize("d,S,P", [(128, 1, 100), (128, 16, 900), (64, 1, 100), (64, 9, 900), (32, 3, 900)])
def test_nan_in_a_row_in_use_reaches_what_uses_it_and_nothing_else(d, S, P):
    cache = R.Cache(2, 2, d, 16, [P, 50], P, 5850)
    pg, i = cache.where(0, 37)
    cache.k[pg, 0, i, 3] = float("nan")     # entry 0, kv head 0: every score against row 37
    cache.v[pg, 1, i, 5] = float("nan")     # entry 0, kv head 1: one column of the values
    q = R.bf16((2, 8, S, d), 5851)
    k, v, table, Pd = cache.cuda()
    out, lse = attn.decoder_sample_paged(q.cuda(), k, v, table, Pd)
    w = attn.kv_cache_weigh(q.cuda(), k, table, Pd, torch.zeros_like(lse), torch.zeros(2, 2, cache.capacity, device="cuda"))
    torch.cuda.synchronize()
    assert out[0, :4].isnan().all() and lse[0, :4].isnan().all()
    assert out[0, 4:, :, 5].isnan().all() and not out[0, 4:, :, :5].isnan().any() and not out[0, 4:, :, 6:].isnan().any()
    assert torch.isfinite(lse[0, 4:]).all() and torch.isfinite(out[1].float()).all() and torch.isfinite(lse[1]).all()
    assert w[0, 0, 37].isnan() and torch.isfinite(w[0, 0, :37]).all() and torch.isfinite(w[0, 0, 38:]).all()
    assert torch.isfinite(w[0, 1]).all() and torch.isfinite(w[1]).all()


def test_shared_pages_are_read_by_both_entries():
    cache = R.Cache(2, 2, 128, 16, [90, 70], 96, 5800)
    cache.table[1, :4] = cache.table[0, :4]   # a common prefix of 64 tokens
    got, ref = run_sample(cache, 4, 1, True, 5801)
    R.check_sample(got, ref, "shared prefix")


def test_sample_is_deterministic_and_leaves_the_workspace_reusable():
    cache = R.Cache(3, 2, 128, 16, [900, 20, 333], 900, 5900)
    q = R.bf16((3, 8, 4, 128), 5901).cuda()
    k, v, table, P = cache.cuda()
    ws = attn.sample_paged_workspace(q, k)
    first = attn.decoder_sample_paged(q, k, v, table, P, workspace=ws)
    for _ in range(5):
        again = attn.decoder_sample_paged(q, k, v, table, P, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert attn.last_device_error() == 0


def test_sample_on_two_streams_at_once():
    caches = [R.Cache(2, 4, 128, 16, [700, 650], 700, 6000 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    args, refs, got = [], [], [None, None]
    for i, c in enumerate(caches):
        q = R.bf16((2, 8, 1, 128), 6010 + i)
        args.append((q.cuda(), *c.cuda()))
        refs.append(R.sample(c, q, None, None))
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = attn.decoder_sample_paged(*args[i])
    torch.cuda.synchronize()
    for g, r in zip(got, refs):
        R.check_sample(g, r, "two streams")


def test_offsets_past_32_bits():
    """A pool of 2^32 + elements each for K and V; the entry's rows lie in its last pages."""
    Hkv, page, d = 8, 128, 128
    pages = (1 << 32) // (Hkv * page * d) + 4
    small = R.Cache(1, Hkv, d, page, [300], 300, 6100, spare=0)
    kp, vp = (torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    last = torch.tensor([pages - 1, pages - 3, pages - 2], dtype=torch.int64)
    for dst, src in ((kp, small.k), (vp, small.v)):
        for i in range(3):
            dst[last[i]] = src[int(small.table[0, i])].cuda()
    table = last.to(torch.int32).view(1, 3).cuda()
    q = R.bf16((1, 16, 2, d), 6101)
    P = torch.tensor([300], dtype=torch.int32, device="cuda")
    got = attn.decoder_sample_paged(q.cuda(), kp, vp, table, P)
    R.check_sample(got, R.sample(small, q, None, None), "past 32 bits")
    w = torch.zeros(1, Hkv, small.capacity)
    ref_w, tol = R.weigh(small, q, got[1].cpu(), w)
    wd, pos = w.cuda(), torch.zeros(1, Hkv, small.capacity, dtype=torch.int32, device="cuda")
    attn.kv_cache_weigh(q.cuda(), kp, table, P, got[1], wd)
    assert (np.abs(wd.cpu().numpy() - ref_w) <= tol).all()
    kn = R.bf16((1, Hkv, 5, d), 6102)
    attn.kv_cache_append_paged(kp, vp, table, P, kn.cuda(), kn.cuda(), weight=wd, pos=pos, tokens=P)
    torch.cuda.synchronize()
    assert np.array_equal(R.bits(kp[pages - 2, :, 44:49]), R.bits(kn[0]))
    w2 = torch.rand(1, Hkv, small.capacity, generator=torch.Generator().manual_seed(3))
    rows_before = torch.cat([kp[int(i)].cpu() for i in last], dim=1)   # [Hkv][384][d]
    wd.copy_(w2)
    attn.kv_cache_evict(kp, vp, table, torch.tensor([305], dtype=torch.int32, device="cuda"), wd, pos, P + 100, 100)
    torch.cuda.synchronize()
    rows_after = torch.cat([kp[int(i)].cpu() for i in last], dim=1)
    for h in range(Hkv):
        moves, _, _ = R.evict(305, w2[0, h].numpy(), pos[0, h].cpu().numpy() * 0, 400, 100, 0)
        want = rows_before[h].clone()
        for s, t in moves:
            want[t] = rows_before[h][s]
        assert np.array_equal(R.bits(rows_after[h][:305]), R.bits(want[:305]))
    assert attn.last_device_error() == 0


# ------------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("d,page,S,P", [(128, 16, 16, [0, 84, 37, 90]), (64, 48, 1, [0, 95, 47, 12]),
                                        (32, 0, 7, [0, 84, 93, 50]), (128, 32, 96, [0, 0, 1, 5])])
@pytest.mark.parametrize("tracked", [True, False])
def test_append_is_bitwise(d, page, S, P, tracked):
    B, Hkv = 4, 3
    cache = R.Cache(B, Hkv, d, page, [96] * B, 96, 6200)
    cap = cache.capacity
    k, v, table, _ = cache.cuda()
    kn, vn = R.bf16((B, Hkv, S, d), 6201), R.bf16((B, Hkv, S, d), 6202)
    Pd = torch.tensor(P, dtype=torch.int32, device="cuda")
    tok = torch.tensor([10, 2000, 0, 77], dtype=torch.int32, device="cuda")
    w = torch.full((B, Hkv, cap), 3.5, device="cuda")
    pos = torch.full((B, Hkv, cap), -9, dtype=torch.int32, device="cuda")
    more = dict(weight=w, pos=pos, tokens=tok) if tracked else {}
    attn.kv_cache_append_paged(k, v, table, Pd, kn.cuda(), vn.cuda(), **more)
    torch.cuda.synchronize()
    want_k, want_v = cache.k.clone(), cache.v.clone()
    want_w, want_p = torch.full((B, Hkv, cap), 3.5), torch.full((B, Hkv, cap), -9, dtype=torch.int32)
    for b in range(B):
        for i in range(S):
            r = P[b] + i
            if r >= cap:
                continue   # rows past the capacity are not written
            pg, j = cache.where(b, r)
            want_k[pg, :, j], want_v[pg, :, j] = kn[b, :, i], vn[b, :, i]
            if tracked:
                want_w[b, :, r], want_p[b, :, r] = 0.0, int(tok[b]) + i
    assert np.array_equal(R.bits(k), R.bits(want_k)) and np.array_equal(R.bits(v), R.bits(want_v))
    assert torch.equal(w.cpu(), want_w) and torch.equal(pos.cpu(), want_p)
    assert attn.last_device_error() == 0


# ------------------------------------------------------------------------------------------------ weigh
@pytest.mark.parametrize("B,Hq,Hkv,S,d,page,P", [
    (1, 1, 1, 1, 128, 16, [1]), (3, 16, 8, 1, 128, 16, [0, 129, 700]), (4, 16, 8, 16, 128, 64, [128, 600, 17, 255]),
    (2, 32, 8, 16, 128, 128, [513, 100]), (2, 12, 4, 7, 64, 48, [299, 1]), (3, 4, 4, 7, 32, 0, [299, 0, 64]),
    (1, 16, 1, 17, 128, 64, [300]), (1, 8, 1, 48, 64, 32, [200]), (1, 8, 1, 70, 32, 16, [140]),
    (40, 2, 1, 3, 64, 16, [(29 * i) % 131 for i in range(40)])])
@pytest.mark.parametrize("in_place", [True, False])
def test_weigh_matches_the_formula(B, Hq, Hkv, S, d, page, P, in_place):
    cache = R.Cache(B, Hkv, d, page, P, max(max(P), 1), 6300 + d)
    cap = cache.capacity
    q = R.bf16((B, Hq, S, d), 6301)
    k, v, table, Pd = cache.cuda()
    lse = torch.from_numpy(R.sample(cache, q, None, None)[1]).float()
    lse[:, 0, 0] = float("-inf")   # a query row that saw nothing adds nothing
    w = torch.rand(B, Hkv, cap, generator=torch.Generator().manual_seed(1))
    out, check = guarded((B, Hkv, cap), torch.float32, -1.0)
    out.copy_(w if in_place else torch.full_like(w, -2.0))
    attn.kv_cache_weigh(q.cuda(), k, table, Pd, lse.cuda(), out if in_place else w.cuda(), out=out)
    torch.cuda.synchronize()
    check()
    ref, tol = R.weigh(cache, q, lse, w)
    got = out.cpu().numpy().astype(np.float64)
    for b in range(B):
        assert (np.abs(got - ref)[b, :, :P[b]] <= tol[b, :, :P[b]]).all(), f"entry {b}: {np.abs(got - ref)[b, :, :P[b]].max()}"
        rest = w[b, :, P[b]:].numpy() if in_place else -2.0
        assert (got[b, :, P[b]:] == rest).all()   # rows past the length are not written
    assert attn.last_device_error() == 0


def test_weigh_rows_sum_to_the_query_count():
    """Every query row's probabilities sum to one: the weights of a fresh cache sum to G S per kv head."""
    cache = R.Cache(2, 4, 128, 16, [777, 50], 800, 6400)
    q = R.bf16((2, 8, 5, 128), 6401).cuda()
    k, v, table, P = cache.cuda()
    _, lse = attn.decoder_sample_paged(q, k, v, table, P)
    w = torch.zeros(2, 4, cache.capacity, device="cuda")
    attn.kv_cache_weigh(q, k, table, P, lse, w)
    first = w.clone()
    assert (w.double().sum(dim=2) - 10).abs().max().item() <= 10 * 2.0 ** -14
    attn.kv_cache_weigh(q, k, table, P, lse, w.zero_())
    assert torch.equal(first, w)


# ------------------------------------------------------------------------------------------------ evict
def run_evict(P, keep, recent, d=64, page=16, Hkv=3, capacity=None, seed=6500, in_place=True, weight=None, shuffle=True):
    B = len(P)
    cache = R.Cache(B, Hkv, d, page, P, capacity or max(max(P), 1), seed)
    cap = cache.capacity
    rng = np.random.default_rng(seed)
    if weight is None:
        weight = np.exp(2 * rng.standard_normal((B, Hkv, cap))).astype(np.float32)
    pos = np.zeros((B, Hkv, cap), np.int32)
    tokens = np.array([p + 11 * b for b, p in enumerate(P)], np.int32)
    for b in range(B):
        for h in range(Hkv):
            line = np.arange(P[b]) + 11 * b
            pos[b, h, :P[b]] = rng.permutation(line) if shuffle else line
    k, v, table, Pd = cache.cuda()
    wd, pd = torch.from_numpy(weight.copy()).cuda(), torch.from_numpy(pos.copy()).cuda()
    td = torch.from_numpy(tokens).cuda()
    if in_place:
        wo, po, Po = wd, pd, Pd
    else:
        wo, po, Po = torch.full_like(wd, -5.0), torch.full_like(pd, -5), torch.full_like(Pd, -5)
    attn.kv_cache_evict(k, v, table, Pd, wd, pd, td, keep, recent=recent, weight_out=wo, pos_out=po, P_out=Po)
    torch.cuda.synchronize()
    assert attn.last_device_error() == 0
    assert Po.tolist() == [min(p, keep) for p in P]
    want_k, want_v = cache.k.clone(), cache.v.clone()
    for b in range(B):
        n = min(P[b], keep)
        for h in range(Hkv):
            moves, w, ps = R.evict(P[b], weight[b, h], pos[b, h], tokens[b], keep, recent)
            for s, t in moves:
                (sp, sr), (tp, tr) = cache.where(b, s), cache.where(b, t)
                want_k[tp, h, tr], want_v[tp, h, tr] = cache.k[sp, h, sr], cache.v[sp, h, sr]
            assert np.array_equal(wo[b, h, :n].cpu().numpy(), w, equal_nan=True), (b, h)
            assert np.array_equal(po[b, h, :n].cpu().numpy(), ps), (b, h)
            rest_w = weight[b, h, n:] if in_place else np.full(cap - n, -5.0, np.float32)
            rest_p = pos[b, h, n:] if in_place else np.full(cap - n, -5, np.int32)
            assert np.array_equal(wo[b, h, n:].cpu().numpy(), rest_w, equal_nan=True)
            assert np.array_equal(po[b, h, n:].cpu().numpy(), rest_p)
    assert np.array_equal(R.bits(k), R.bits(want_k)) and np.array_equal(R.bits(v), R.bits(want_v))


@pytest.mark.parametrize("P,keep,recent", [
    ([0], 5, 0), ([1], 0, 0), ([1], 1, 1), ([7, 6, 5], 6, 2), ([100, 3, 64], 50, 10), ([100, 99], 99, 99), ([300, 17], 0, 0),
    ([1000, 513], 512, 64), ([1025, 1024, 1023], 1, 1), ([2064] * 2, 2048, 64), ([2500, 100], 700, 0),
    ([200, 150], 150, 150)])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict_matches_the_definition(P, keep, recent, in_place):
    run_evict(P, keep, recent, in_place=in_place)


@pytest.mark.parametrize("d,page,capacity", [(128, 64, 900), (32, 48, 777), (64, 0, 777), (128, 0, 901)])
def test_evict_layouts(d, page, capacity):
    run_evict([777, 500, 333], 400, 33, d=d, page=page, capacity=capacity)


def test_evict_ties_and_special_weights():
    """Many equal weights (ties to the lowest row), infinities, both zeros, NaN (below every number), negative
    and denormal weights."""
    rng = np.random.default_rng(3)
    P, cap = [600, 300], 608
    pool = np.array([0.0, -0.0, 1.0, 1.0, np.inf, -np.inf, np.nan, -1.0, 1e-42, -1e-42, 3e38], np.float32)
    for keep in (10, 150, 290, 299):
        w = pool[rng.integers(0, len(pool), size=(2, 3, cap))]
        run_evict(P, keep, 5, weight=w, seed=6600 + keep)
    run_evict(P, 200, 0, weight=np.full((2, 3, cap), 0.25, np.float32), seed=6700)      # all equal: the first 200
    run_evict(P, 200, 20, weight=np.full((2, 3, cap), np.nan, np.float32), seed=6701)
    run_evict(P, 200, 20, weight=np.zeros((2, 3, cap), np.float32), seed=6702, shuffle=False)


def test_evict_long_cache():
    run_evict([40000], 9000, 500, Hkv=2, seed=6800)
    run_evict([40000], 39000, 500, Hkv=1, page=128, seed=6801)


def test_evict_workspace_serves_other_batches():
    """One workspace, zero-filled once, for calls of different batches and heads: the lengths, in place, come out
    right in each (they are written when every head of the call has read them)."""
    ws = None
    for B, Hkv, P in ((5, 3, 300), (1, 1, 90), (40, 8, 300), (1, 1, 90), (5, 3, 300)):
        cache = R.Cache(B, Hkv, 32, 16, [P - 3 * b for b in range(B)], 300, 6950 + B)
        k, v, table, Pd = cache.cuda()
        w = torch.rand(B, Hkv, cache.capacity, device="cuda")
        pos = torch.arange(cache.capacity, dtype=torch.int32, device="cuda").expand(B, Hkv, -1).contiguous()
        if ws is None:
            big = torch.zeros(40, 8, cache.capacity, device="cuda")
            ws = attn.evict_workspace(big)
        tokens = Pd.clone()
        want = torch.minimum(Pd, torch.tensor(200, device="cuda", dtype=torch.int32))
        kept = [torch.topk(w[b, h, : P - 3 * b], min(200, P - 3 * b)).values.sort().values
                for b in range(B) for h in range(Hkv)]
        attn.kv_cache_evict(k, v, table, Pd, w, pos, tokens, 200, recent=0, workspace=ws)
        assert torch.equal(Pd, want)
        got = [w[b, h, : int(want[b])].sort().values for b in range(B) for h in range(Hkv)]
        assert all(torch.equal(x, y) for x, y in zip(got, kept))
    assert attn.last_device_error() == 0


def test_evict_many_protected_rows():
    """More rows at or past the protected position than fit (a caller's positions need not be distinct): the
    lowest of them stay."""
    cap, P, keep = 64, 60, 10
    cache = R.Cache(1, 1, 64, 16, [P], cap, 6900)
    k, v, table, Pd = cache.cuda()
    w = torch.rand(1, 1, cap, device="cuda")
    pos = torch.full((1, 1, cap), 100, dtype=torch.int32, device="cuda")
    w0 = w.clone()
    attn.kv_cache_evict(k, v, table, Pd, w, pos, torch.tensor([100], dtype=torch.int32, device="cuda"), keep, recent=5)
    torch.cuda.synchronize()
    assert Pd.item() == keep and torch.equal(w[0, 0, :keep], w0[0, 0, :keep])


# ------------------------------------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("S,d", [(1, 128), (16, 128), (1, 64), (9, 32)])
def test_waits_that_run_out_are_reported_and_the_next_call_is_clean(S, d):
    """The test hook shortens the waits to 1 ms and holds the loads back for 20 ms: the calls return, the error
    says so, and with a zero-filled workspace the next call is right."""
    lib = _lib.load()
    cache = R.Cache(2, 2, d, 16, [700, 90], 700, 6950)
    q = R.bf16((2, 8, S, d), 6951)
    qd = q.cuda()
    k, v, table, P = cache.cuda()
    ws = attn.sample_paged_workspace(qd, k)
    lse = torch.zeros(2, 8, S, device="cuda")
    w = torch.zeros(2, 2, cache.capacity, device="cuda")
    torch.cuda.synchronize()
    assert attn.last_device_error() == 0
    for call in (lambda: attn.decoder_sample_paged(qd, k, v, table, P, workspace=ws),
                 lambda: attn.kv_cache_weigh(qd, k, table, P, lse, w)):
        try:
            assert lib.e2d2_debug_set_wait_test(1_000_000, 20_000_000) == 0
            call()
            torch.cuda.synchronize()
            assert attn.last_device_error() == E2D2_ERR_TIMEOUT
        finally:
            assert lib.e2d2_debug_set_wait_test(0, 0) == 0
    got = attn.decoder_sample_paged(qd, k, v, table, P, workspace=ws.zero_())
    w.zero_()
    attn.kv_cache_weigh(qd, k, table, P, got[1], w)
    torch.cuda.synchronize()
    assert attn.last_device_error() == 0
    R.check_sample(got, R.sample(cache, q, None, None), "after a timed-out call")
    ref, tol = R.weigh(cache, q, got[1].cpu(), torch.zeros(2, 2, cache.capacity))
    assert (np.abs(w.cpu().numpy() - ref) <= tol).all()


# ------------------------------------------------------------------------------------------------ together
def simulate(B, Hq, Hkv, d, S, keep, recent, blocks, page, graph, seed):
    """A decoding loop: every block attends to the cache and itself, is appended, adds its weights, and the
    cache is cut back to its budget; eager, or one captured block replayed.  The reference keeps its own cache
    (rows in the order of the kernel's) and must agree block by block."""
    cap = keep + S
    each = -(-cap // page)
    W = each * page
    rng = np.random.default_rng(seed)
    n_pages = B * each + 2
    table = torch.from_numpy(rng.permutation(n_pages)[:B * each].reshape(B, each).astype(np.int32))
    dev = dict(device="cuda")
    kp, vp = (torch.full((n_pages, Hkv, page, d), float("nan"), dtype=torch.bfloat16, **dev) for _ in range(2))
    td = table.cuda()
    P, tok = torch.zeros(B, dtype=torch.int32, **dev), torch.zeros(B, dtype=torch.int32, **dev)
    w, pos = torch.full((B, Hkv, W), float("nan"), **dev), torch.full((B, Hkv, W), -1, dtype=torch.int32, **dev)
    q, kb, vb = (torch.zeros(s, dtype=torch.bfloat16, **dev) for s in ((B, Hq, S, d), (B, Hkv, S, d), (B, Hkv, S, d)))
    ws = attn.sample_paged_workspace(q, kp)
    ews = attn.evict_workspace(w)
    out, lse = torch.empty_like(q), torch.empty(B, Hq, S, **dev)
    before = []   # weights, positions and lengths ahead of the eviction

    def block():
        attn.decoder_sample_paged(q, kp, vp, td, P, kb, vb, workspace=ws, out=out, lse=lse)
        attn.kv_cache_append_paged(kp, vp, td, P, kb, vb, weight=w, pos=pos, tokens=tok)
        P.add_(S)
        tok.add_(S)
        attn.kv_cache_weigh(q, kp, td, P, lse, w)
        if not graph:
            before[:] = [w.cpu().numpy(), pos.cpu().numpy(), P.tolist()]
        attn.kv_cache_evict(kp, vp, td, P, w, pos, tok, keep, recent=recent, workspace=ews)

    run = block
    if graph:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            block()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            block()
        for t in (P, tok):
            t.zero_()
        run = g.replay
    K, V = np.zeros((B, Hkv, W, d)), np.zeros((B, Hkv, W, d))
    length = 0
    for i in range(blocks):
        nq, nk, nv = (R.bf16(t.shape, seed + 10 * i + j) for j, t in enumerate((q, kb, vb)))
        q.copy_(nq), kb.copy_(nk), vb.copy_(nv)
        run()
        torch.cuda.synchronize()
        ref = R.Cache.__new__(R.Cache)
        ref.B, ref.Hkv, ref.d, ref.page, ref.table, ref.P = B, Hkv, d, 0, None, [length] * B
        ref.k, ref.v = (torch.from_numpy(x).to(torch.bfloat16) for x in (K, V))
        R.check_sample((out, lse), R.sample(ref, nq, nk, nv), f"block {i}")
        K[:, :, length:length + S], V[:, :, length:length + S] = R.f64(nk), R.f64(nv)
        total = length + S
        length = min(total, keep)
        assert P.tolist() == [length] * B and tok.tolist() == [(i + 1) * S] * B
        # the rows that stayed, by their positions: in the eager loop exactly those that the definition picks
        # from the weights ahead of the eviction, and always distinct and with the newest among them
        ids = pos.cpu().numpy()
        for b in range(B):
            for h in range(Hkv):
                kept = ids[b, h, :length]
                if not graph:
                    _, w_ref, p_ref = R.evict(before[2][b], before[0][b, h], before[1][b, h], tok[b].item(), keep, recent)
                    assert np.array_equal(kept, p_ref) and np.array_equal(w[b, h, :length].cpu().numpy(), w_ref)
                assert len(set(kept.tolist())) == length and kept.max() == tok[b].item() - 1
                if recent:
                    newest = range(max(0, tok[b].item() - recent), tok[b].item())
                    assert set(newest) <= set(kept.tolist())
        rows = torch.empty(B, Hkv, W, d, dtype=torch.bfloat16)
        for x, pool in ((K, kp), (V, vp)):
            pc = pool.cpu()
            for b in range(B):
                rows[b] = pc[table[b].long()].transpose(0, 1).reshape(Hkv, W, d)
            x[:, :, :length] = R.f64(rows[:, :, :length])
        assert torch.isfinite(w[:, :, :length]).all()
    assert attn.last_device_error() == 0
    return kp, vp, w, pos


@pytest.mark.parametrize("graph", [False, True])
def test_decoding_loop_with_a_budget(graph):
    simulate(2, 8, 4, 128, 4, 40, 12, 16, 16, graph, 7000)


def test_decoding_loop_token_by_token():
    simulate(3, 4, 2, 64, 1, 17, 5, 30, 16, False, 7100)


def test_captured_and_eager_loops_agree():
    a = simulate(2, 4, 2, 32, 3, 20, 6, 10, 16, False, 7200)
    b = simulate(2, 4, 2, 32, 3, 20, 6, 10, 16, True, 7200)
    assert torch.equal(a[2][:, :, :20], b[2][:, :, :20]) and torch.equal(a[3][:, :, :20], b[3][:, :, :20])


def test_two_captured_graphs_with_their_own_workspaces():
    cache = R.Cache(2, 4, 128, 16, [900, 333], 900, 7300)
    k, v, table, P = cache.cuda()
    graphs, outs, refs = [], [], []
    for i in range(2):
        q = R.bf16((2, 8, 1 + 3 * i, 128), 7301 + i)
        qd = q.cuda()
        ws = attn.sample_paged_workspace(qd, k)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            attn.decoder_sample_paged(qd, k, v, table, P, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(attn.decoder_sample_paged(qd, k, v, table, P, workspace=ws))
        graphs.append((g, ws, qd))
        refs.append(R.sample(cache, q, None, None))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        R.check_sample(o, r, "captured")
