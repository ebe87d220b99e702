"""GPU tests of the paged-cache calls at their edges: budgets of nothing, values that are no numbers, pages that no pool
holds, every shape of an eviction's launch, and what each call must leave alone.  Every buffer that a call may write lies
inside a larger one whose margins are checked afterwards, the workspace too."""
import numpy as np
import pytest
import torch

from block_discrete_diffusion_tcgen05_b200 import attn
import paged_reference as R

pytestmark = pytest.mark.gpu

PAD = 8192


class Guarded:
    """Tensors with margins of one byte value on either side; check() says whether any margin changed."""

    def __init__(self, fill=0xA5):
        self.fill, self.held = fill, []

    def __call__(self, t):
        n = t.numel() * t.element_size()
        big = torch.full((n + 2 * PAD,), self.fill, dtype=torch.uint8, device="cuda")
        inner = big[PAD:PAD + n].view(t.dtype).view(t.shape)
        inner.copy_(t)
        self.held.append((big, n))
        return inner

    def check(self):
        for i, (big, n) in enumerate(self.held):
            assert (big[:PAD] == self.fill).all() and (big[PAD + n:] == self.fill).all(), f"buffer {i}: written outside"


def raw(t):
    return t.view(torch.int16)


def kept_rows(w, pos, protect, keep):
    """Rows that stay by the definition, as a mask: w, pos numpy [P]."""
    P = len(w)
    kind = np.where(pos >= protect, 2, np.where(np.isnan(w), 0, 1))
    value = np.where(kind == 1, np.where(np.isnan(w), 0, w), 0).astype(np.float64)
    order = np.lexsort((np.arange(P), -value, -kind))
    mask = np.zeros(P, bool)
    mask[order[:keep]] = True
    return mask


def run_evict(P, keep, recent=0, d=64, page=16, Hkv=3, capacity=None, seed=1, in_place=True, weight=None, tokens=None,
              pos=None, bad=(), dirty=False):
    """One eviction of random pools against the definition, bit by bit.  weight: [B][Hkv][capacity] numpy or a function of
    (rng, shape); tokens: one per entry, default P; bad: (entry, page of it) pairs whose table entry names no page;
    dirty: the lists of the workspace hold row numbers past every cache, as a call of other sizes may leave them."""
    B = len(P)
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows = capacity or max(max(P), 1)
    each = -(-rows // page) if page else 1
    cap = each * page if page else rows
    table_h = np.arange(B).reshape(B, 1) if not page else rng.permutation(B * each + 2)[:B * each].reshape(B, each)
    n_pages, per = (B, cap) if not page else (B * each + 2, page)
    guard = Guarded()
    k0, v0 = (torch.randint(-2 ** 15, 2 ** 15, (n_pages, Hkv, per, d), dtype=torch.int16, device="cuda", generator=g)
              .view(torch.bfloat16) for _ in range(2))
    k, v = guard(raw(k0)).view(torch.bfloat16), guard(raw(v0)).view(torch.bfloat16)
    shape = (B, Hkv, cap)
    w0 = np.exp(2 * rng.standard_normal(shape)) if weight is None else (weight(rng, shape) if callable(weight) else weight)
    w0 = np.ascontiguousarray(w0, np.float32)
    if pos is None:
        pos = np.zeros(shape, np.int32)
        for b in range(B):
            for h in range(Hkv):
                pos[b, h, :P[b]] = rng.permutation(P[b])
    tokens = list(P) if tokens is None else tokens
    table = None
    if page:
        named = table_h.astype(np.int32)
        for b, i in bad:
            named[b, i] = n_pages + 5
        table = torch.from_numpy(named).cuda()
    wd, pd = guard(torch.from_numpy(w0).cuda()), guard(torch.from_numpy(pos).cuda())
    Pd, td = guard(torch.tensor(P, dtype=torch.int32, device="cuda")), torch.tensor(tokens, dtype=torch.int32, device="cuda")
    wo, po, Po = (wd, pd, Pd) if in_place else (guard(torch.full_like(wd, -5.0)), guard(torch.full_like(pd, -5)),
                                                guard(torch.full_like(Pd, -5)))
    was_w, was_p = wo.cpu().numpy().copy(), po.cpu().numpy().copy()
    ws = torch.zeros(attn.evict_workspace_bytes(B, Hkv, cap), dtype=torch.uint8, device="cuda")
    if dirty:
        ws[16:].view(torch.int32).fill_(1 << 24)
    ws = guard(ws)
    attn.kv_cache_evict(k, v, table, Pd, wd, pd, td, keep, recent=recent, weight_out=wo, pos_out=po, P_out=Po, workspace=ws)
    torch.cuda.synchronize()
    error = attn.last_device_error()
    guard.check()
    assert ws[:16].eq(0).all(), "the workspace is not reusable"
    assert Po.tolist() == [min(p, keep) for p in P]
    moved = 0
    src, dst, head = [], [], []
    got_w, got_p = wo.cpu().numpy(), po.cpu().numpy()
    for b in range(B):
        n, lost = P[b], {i for e, i in bad if e == b}
        m = min(n, keep)
        for h in range(Hkv):
            want_w, want_p = was_w[b, h].copy(), was_p[b, h].copy()
            want_w[:m], want_p[:m] = w0[b, h, :m], pos[b, h, :m]
            if n > keep:
                mask = kept_rows(w0[b, h, :n], pos[b, h, :n], tokens[b] - recent, keep)
                holes, movers = np.flatnonzero(~mask[:keep]), keep + np.flatnonzero(mask[keep:])
                assert len(holes) == len(movers)
                if page:  # a move whose source or target no page backs is not made
                    ok = ~(np.isin(holes // page, list(lost)) | np.isin(movers // page, list(lost)))
                    holes, movers = holes[ok], movers[ok]
                want_w[holes], want_p[holes] = w0[b, h, movers], pos[b, h, movers]
                moved += len(holes)
                src += [(table_h[b, s // per], s % per) for s in movers]
                dst += [(table_h[b, t // per], t % per) for t in holes]
                head += [h] * len(holes)
            assert np.array_equal(got_w[b, h], want_w, equal_nan=True), (b, h)
            assert np.array_equal(got_p[b, h], want_p), (b, h)
    if moved:
        s, t = (torch.tensor(np.array(x), device="cuda") for x in (src, dst))
        hd = torch.tensor(head, device="cuda")
        for x in (k0, v0):
            raw(x)[t[:, 0], hd, t[:, 1]] = raw(x)[s[:, 0], hd, s[:, 1]]
    assert torch.equal(raw(k), raw(k0)) and torch.equal(raw(v), raw(v0))
    return moved, error


# ------------------------------------------------------------------------------------- a budget of nothing
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("tokens", ["none", "some", "all"])
@pytest.mark.parametrize("P,page,d,Hkv", [([300], 16, 64, 3), ([300, 17, 0, 64], 48, 32, 2), ([1], 16, 128, 1),
                                          ([9000], 0, 64, 1), ([33], 0, 128, 5)])
def test_a_budget_of_nothing_evicts_everything(P, page, d, Hkv, tokens, in_place):
    """keep = 0 with no, some or all of the positions at or past `tokens` (protected, but for the budget): the lengths
    become 0, and not a row, weight or position is written, whatever the workspace's lists hold."""
    tok = {"none": P, "some": [p // 2 for p in P], "all": [0] * len(P)}[tokens]
    assert run_evict(P, 0, d=d, page=page, Hkv=Hkv, tokens=tok, in_place=in_place, dirty=True, seed=11) == (0, 0)


@pytest.mark.parametrize("keep", [1, 2, 149])
def test_protected_rows_past_a_small_budget(keep):
    """As many protected rows as there are, and room for a few of them: the lowest stay."""
    moved, error = run_evict([300, 40], keep, tokens=[0, 20], dirty=True, seed=12)
    assert error == 0


# --------------------------------------------------------------------------- query rows that saw nothing
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("d,Hq,Hkv,S", [(128, 4, 4, 1), (128, 4, 2, 16), (128, 8, 2, 16), (64, 4, 2, 5), (32, 4, 2, 40),
                                        (64, 8, 1, 33)])
def test_a_query_row_that_saw_nothing_adds_nothing_whatever_it_holds(d, Hq, Hkv, S, value):
    """lse = -infinity: the row is padding, its query may hold anything.  The weights are those with any other query in
    its place, bit by bit."""
    B, cap = 3, 400
    g = torch.Generator(device="cuda")
    g.manual_seed(21)
    k = torch.randn(B, Hkv, cap, d, device="cuda", generator=g).bfloat16()
    q = torch.randn(B, Hq, S, d, device="cuda", generator=g).bfloat16()
    P = torch.tensor([400, 0, 131], dtype=torch.int32, device="cuda")
    lse = torch.full((B, Hq, S), 4.0, device="cuda")
    nothing = torch.zeros(B, Hq, S, dtype=torch.bool, device="cuda")
    nothing[0, ::2, S // 2], nothing[0, -1, -1], nothing[2] = True, True, True   # rows here and there, and an entry of padding
    lse[nothing] = float("-inf")
    w0 = torch.rand(B, Hkv, cap, device="cuda", generator=g)
    plain = attn.kv_cache_weigh(q, k, None, P, lse, w0, out=torch.zeros_like(w0))
    q[nothing] = value
    out = attn.kv_cache_weigh(q, k, None, P, lse, w0, out=torch.zeros_like(w0))
    torch.cuda.synchronize()
    assert torch.equal(out, plain) and torch.isfinite(out).all()
    assert torch.equal(out[2, :, :131], w0[2, :, :131])
    assert attn.last_device_error() == 0


# ----------------------------------------------------------------------------------- infinite values
@pytest.mark.parametrize("d,Hq,S", [(128, 4, 1), (128, 4, 16), (128, 4, 32), (128, 4, 50), (64, 4, 1), (64, 4, 9), (64, 4, 16),
                                    (64, 4, 40), (32, 4, 3), (32, 4, 40)])
@pytest.mark.parametrize("P", [100, 900])
@pytest.mark.parametrize("block", [False, True])
def test_an_infinite_value_gives_infinity_in_its_column(d, Hq, S, P, block):
    """Every probability is positive: a row in use whose value is infinite makes its column infinite, of both signs NaN,
    and no other column changes a bit.  In the cached rows, and in the block's own."""
    Hkv = 2
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    normal = lambda *shape: torch.randn(shape, device="cuda", generator=g).bfloat16()  # noqa: E731
    q, k, v = normal(1, Hq, S, d), normal(1, Hkv, P, d), normal(1, Hkv, P, d)
    kb, vb = (normal(1, Hkv, S, d), normal(1, Hkv, S, d)) if block else (None, None)
    Pd = torch.tensor([P], dtype=torch.int32, device="cuda")
    plain, lse0 = attn.decoder_sample_paged(q, k, v, None, Pd, kb, vb)
    v[0, 0, 37, 5] = float("inf")
    v[0, 0, P - 1, 9], v[0, 0, 2, 9] = -float("inf"), float("inf")
    (v if not block else vb)[0, 1, 0, 17] = -float("inf")
    out, lse = attn.decoder_sample_paged(q, k, v, None, Pd, kb, vb)
    torch.cuda.synchronize()
    a, b = out[0, :Hq // 2], out[0, Hq // 2:]
    assert (a[..., 5] == float("inf")).all() and a[..., 9].isnan().all() and (b[..., 17] == -float("inf")).all()
    for got, ref, touched in ((a, plain[0, :Hq // 2], (5, 9)), (b, plain[0, Hq // 2:], (17,))):
        rest = [c for c in range(d) if c not in touched]
        assert torch.equal(got[..., rest], ref[..., rest])
    assert torch.equal(lse, lse0)


# ------------------------------------------------------------------------- page ids outside the pool
E2D2_ERR_PAGE = 10


@pytest.mark.parametrize("bad", [-1, 11, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("d,page", [(128, 16), (64, 48), (32, 32)])
def test_an_append_leaves_rows_without_a_page_alone(d, page, bad):
    """Neither K and V nor the weight and position of such a row are written; the rows around them are, and the error
    is reported."""
    B, Hkv, S, each = 2, 3, 2 * page + 5, 4
    cap, pages = each * page, 11
    rng = np.random.default_rng(41)
    table_h = rng.permutation(pages)[:B * each].reshape(B, each).astype(np.int32)
    guard = Guarded()
    k, v = (guard(torch.full((pages, Hkv, page, d), 3.0, dtype=torch.bfloat16, device="cuda")) for _ in range(2))
    w, pos = guard(torch.full((B, Hkv, cap), 7.0, device="cuda")), guard(torch.full((B, Hkv, cap), -9, dtype=torch.int32, device="cuda"))
    new = torch.arange(1, S + 1, device="cuda", dtype=torch.float32).view(1, 1, S, 1).expand(B, Hkv, S, d).bfloat16().contiguous()
    P, tok = [7, page], [100, 5]
    broken = torch.from_numpy(table_h.copy())
    broken[0, 1] = bad
    attn.kv_cache_append_paged(k, v, broken.cuda(), torch.tensor(P, dtype=torch.int32, device="cuda"), new, -new, weight=w,
                               pos=pos, tokens=torch.tensor(tok, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert attn.last_device_error() == E2D2_ERR_PAGE and attn.last_device_error() == 0
    guard.check()
    want_k, want_w, want_p = torch.full((pages, Hkv, page, d), 3.0), torch.full((B, Hkv, cap), 7.0), torch.full((B, Hkv, cap), -9)
    want_v = want_k.clone()
    for b in range(B):
        for i in range(S):
            r = P[b] + i
            if b == 0 and r // page == 1:
                continue
            value = new[b, 0, i, 0].float().item()
            want_k[table_h[b, r // page], :, r % page], want_v[table_h[b, r // page], :, r % page] = value, -value
            want_w[b, :, r], want_p[b, :, r] = 0.0, tok[b] + i
    assert torch.equal(k.float().cpu(), want_k) and torch.equal(v.float().cpu(), want_v)
    assert torch.equal(w.cpu(), want_w) and torch.equal(pos.cpu().long(), want_p.long())


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("d,page,bad", [(64, 16, [(0, 2)]), (128, 48, [(0, 5)]), (32, 16, [(0, 1), (0, 17), (1, 0)])])
def test_an_eviction_makes_no_move_from_or_to_a_row_without_a_page(d, page, bad, in_place):
    """Where the target's page or the source's is none of the pool, the hole keeps its row, weight and position: the
    three belong together before and after."""
    moved, error = run_evict([300, 290], 150, recent=10, d=d, page=page, bad=bad, in_place=in_place, seed=42)
    assert moved > 0 and error == E2D2_ERR_PAGE


def test_an_append_of_no_rows():
    k, w, pos = torch.ones(2, 3, 64, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(2, 3, 64, device="cuda"), \
        torch.ones(2, 3, 64, dtype=torch.int32, device="cuda")
    P = torch.zeros(2, dtype=torch.int32, device="cuda")
    none = k[:, :, :0].contiguous()
    v = k.clone()
    attn.kv_cache_append_paged(k, v, None, P, none, none, weight=w, pos=pos, tokens=P)
    torch.cuda.synchronize()
    assert all((t == 1).all() for t in (k, v, w, pos)) and attn.last_device_error() == 0


# ------------------------------------------------------------- every shape of an eviction's launch
def few_values(rng, shape):
    """Many rows at the threshold, wherever it falls."""
    return rng.choice(np.array([0.0, 0.25, 0.25, 0.25, 1.0, 3.0], np.float32), size=shape)


LAUNCHES = [
    # P, keep, recent, Hkv, capacity, d, page: blocks per head, threads of a block on 148 SMs
    ([33000], 32500, 100, 80, 33000, 32, 48),          # 1, 1024: more rows than a block's shared memory has ranks for
    ([33000], 16000, 0, 80, 33000, 32, 0),
    ([5000], 2600, 64, 40, 5000, 64, 16),              # 2, 512
    ([9000, 7], 4400, 10, 37, 9000, 32, 48),           # 2, 1024: a block on every SM
    ([9000], 4400, 10, 40, 9000, 32, 48),              # 2, 1024
    ([8192], 5000, 100, 1, 8192, 128, 64),             # 4, 512
    ([8192, 100, 2100, 40], 30, 8, 5, 8200, 64, 16),   # 4, 512: short entries leave a cluster's later blocks without rows
    ([20000, 33, 6000], 5000, 9, 7, 20000, 32, 128),   # 4, 1024
    ([17000, 65], 8500, 0, 8, 17000, 32, 16),          # 8, 512
    ([40000, 31], 20, 20, 4, 40000, 32, 0),            # 8, 1024
]


@pytest.mark.parametrize("P,keep,recent,Hkv,capacity,d,page", LAUNCHES)
@pytest.mark.parametrize("weight", [few_values, None], ids=["ties", "distinct"])
@pytest.mark.parametrize("in_place", [True, False])
def test_every_launch_of_an_eviction(P, keep, recent, Hkv, capacity, d, page, weight, in_place):
    """Clusters of 1, 2, 4 and 8 blocks of 512 and 1024 threads, ranks held in shared memory and read again, rows at the
    threshold in every block of a cluster."""
    moved, error = run_evict(P, keep, recent, d=d, page=page, Hkv=Hkv, capacity=capacity, weight=weight, in_place=in_place,
                             dirty=True, seed=51)
    assert moved > 0 and error == 0


def test_equal_weights_keep_the_lowest_rows_across_a_cluster():
    for Hkv, capacity in ((1, 8192), (40, 5000), (8, 17000)):
        run_evict([capacity], capacity // 2 + 77, Hkv=Hkv, capacity=capacity, d=32, seed=52,
                  weight=lambda rng, shape: np.full(shape, 0.5, np.float32))


# ------------------------------------------------------------- pages that no pool holds, in every sampling kernel
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("rows", [1, 20, 64])
@pytest.mark.parametrize("block", [False, True])
def test_attention_leaves_out_rows_without_a_page(d, page, rows, block):
    """A page in the middle, the one that the length ends in, and all of an entry's pages."""
    each = 3 if page == 128 else 5
    P = [each * page - 7, 2 * page, page + 1]
    cache = R.Cache(3, 2, d, page, P, max(P), 5900 + page)
    lost = [(0, 1), (0, each - 1), (2, 0), (2, 1)]
    k, v, table, Pd = cache.cuda()
    for i, (b, n) in enumerate(lost):
        table[b, n] = (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31)[i]
    skip = {(b, r) for b, n in lost for r in range(n * page, min((n + 1) * page, P[b]))}
    q = R.bf16((3, 2, rows, d), 5910)
    kb, vb = (R.bf16((3, 2, rows, d), 5911), R.bf16((3, 2, rows, d), 5912)) if block else (None, None)
    got = attn.decoder_sample_paged(q.cuda(), k, v, table, Pd, None if kb is None else kb.cuda(), None if vb is None else vb.cuda())
    torch.cuda.synchronize()
    assert attn.last_device_error() == E2D2_ERR_PAGE
    R.check_sample(got, R.sample(cache, q, kb, vb, skip=skip), f"d{d} page{page} rows{rows}")
    w = torch.rand(3, 2, cache.capacity, generator=torch.Generator().manual_seed(1))
    ref, tol = R.weigh(cache, q, got[1].cpu(), w, skip=skip)
    out = attn.kv_cache_weigh(q.cuda(), k, table, Pd, got[1], w.cuda())
    torch.cuda.synchronize()
    assert attn.last_device_error() == E2D2_ERR_PAGE
    assert (np.abs(out.cpu().numpy() - ref) <= tol).all()


# ------------------------------------------------------------- nothing outside the arguments is read
@pytest.mark.parametrize("B,Hq,Hkv,S,d,page,block,P", [
    (1, 1, 1, 1, 128, 0, True, [1]), (2, 6, 2, 5, 128, 16, True, [37, 200]), (1, 16, 2, 8, 128, 48, False, [141]),
    (3, 4, 4, 7, 64, 0, False, [299, 1, 0]), (2, 8, 2, 16, 64, 80, True, [161, 80]), (1, 40, 2, 5, 32, 16, True, [333]),
    (1, 2, 1, 33, 32, 0, True, [45])])
def test_what_lies_around_the_arguments_is_not_read(B, Hq, Hkv, S, d, page, block, P):
    """Every argument and the workspace between NaN: neither the attention nor the weights see it."""
    cache = R.Cache(B, Hkv, d, page, P, max(P), 6000 + d, spare=0)
    guard = Guarded(fill=0xFF)
    k, v, table, Pd = (None if t is None else guard(t) for t in cache.cuda())
    q = R.bf16((B, Hq, S, d), 6001)
    kb, vb = (R.bf16((B, Hkv, S, d), 6002), R.bf16((B, Hkv, S, d), 6003)) if block else (None, None)
    qd, kd, vd = (None if t is None else guard(t.cuda()) for t in (q, kb, vb))
    ws = guard(attn.sample_paged_workspace(qd, k))
    out, lse = guard(torch.zeros_like(qd)), guard(torch.zeros(B, Hq, S, device="cuda"))
    attn.decoder_sample_paged(qd, k, v, table, Pd, kd, vd, workspace=ws, out=out, lse=lse)
    torch.cuda.synchronize()
    R.check_sample((out, lse), R.sample(cache, q, kb, vb), "between NaN")
    w = torch.rand(B, Hkv, cache.capacity, generator=torch.Generator().manual_seed(2))
    ref, tol = R.weigh(cache, q, lse.cpu(), w)
    wd, wo = guard(w.cuda()), guard(w.cuda())
    attn.kv_cache_weigh(qd, k, table, Pd, lse, wd, out=wo)
    torch.cuda.synchronize()
    assert (np.abs(wo.cpu().numpy() - ref) <= tol).all()
    guard.check()
    assert attn.last_device_error() == 0


# ------------------------------------------------------------- captured calls
def test_captured_calls_with_a_workspace_zeroed_ahead_of_them():
    """Two graphs with workspaces of their own, replayed at once on two streams; the warm-up waits for the zero-filling,
    which runs on the stream of the allocation."""
    cache = R.Cache(2, 4, 128, 16, [900, 333], 900, 7400)
    k, v, table, P = cache.cuda()
    made = []
    for i in range(2):
        q = R.bf16((2, 8, 1 + 3 * i, 128), 7401 + i)
        qd = q.cuda()
        ws = attn.sample_paged_workspace(qd, k)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            attn.decoder_sample_paged(qd, k, v, table, P, workspace=ws)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = attn.decoder_sample_paged(qd, k, v, table, P, workspace=ws)
        made.append((g, torch.cuda.Stream(), out, R.sample(cache, q, None, None), ws, qd))
    for _ in range(5):
        for g, s, *_ in made:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, out, ref, *_ in made:
        R.check_sample(out, ref, "captured")
    assert attn.last_device_error() == 0


@pytest.mark.parametrize("B,Hq,Hkv,S,d,page,lo,hi", [(1, 16, 8, 1, 128, 64, 500, 500), (8, 16, 8, 16, 128, 64, 2048, 2048),
                                                     (2, 32, 8, 16, 128, 128, 7000, 8192), (5, 12, 4, 7, 64, 48, 1, 3001)])
def test_repeated_calls_give_the_same_bits(B, Hq, Hkv, S, d, page, lo, hi):
    """Units shared by several blocks are joined in the blocks' order, whichever finishes last."""
    g = torch.Generator(device="cuda")
    g.manual_seed(61)
    normal = lambda *shape: torch.randn(shape, device="cuda", generator=g).bfloat16()  # noqa: E731
    each = -(-hi // page)
    k, v = normal(B * each, Hkv, page, d), normal(B * each, Hkv, page, d)
    table = torch.randperm(B * each, device="cuda", generator=g).view(B, each).int().contiguous()
    P = torch.linspace(lo, hi, B, device="cuda").int()
    q, kb, vb = normal(B, Hq, S, d), normal(B, Hkv, S, d), normal(B, Hkv, S, d)
    ws = attn.sample_paged_workspace(q, k)
    first = attn.decoder_sample_paged(q, k, v, table, P, kb, vb, workspace=ws)
    for _ in range(30):
        again = attn.decoder_sample_paged(q, k, v, table, P, kb, vb, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert attn.last_device_error() == 0


def test_one_workspace_serves_attention_of_other_shapes():
    """Zero-filled once, then calls of other head sizes, rows, batches and lengths on the same stream."""
    shapes = [(2, 16, 2, 8, 128, 16, [900, 333]), (1, 2, 1, 1, 64, 48, [1500]), (3, 8, 2, 16, 128, 64, [700, 0, 129]),
              (2, 4, 4, 7, 32, 16, [299, 800]), (1, 8, 8, 1, 128, 32, [2100])]
    made, ws = [], torch.zeros(max(attn.sample_paged_workspace_bytes(B, Hq, Hkv, d, S) for B, Hq, Hkv, S, d, _, _ in shapes),
                               dtype=torch.uint8, device="cuda")
    for i, (B, Hq, Hkv, S, d, page, P) in enumerate(shapes):
        cache = R.Cache(B, Hkv, d, page, P, max(P), 6200 + i)
        q = R.bf16((B, Hq, S, d), 6210 + i)
        made.append((q.cuda(), *cache.cuda(), R.sample(cache, q, None, None)))
    for _ in range(2):
        got = [attn.decoder_sample_paged(q, k, v, table, P, workspace=ws) for q, k, v, table, P, _ in made]
        torch.cuda.synchronize()
        for g, m in zip(got, made):
            R.check_sample(g, m[-1], "one workspace")
    assert attn.last_device_error() == 0
