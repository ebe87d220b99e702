"""The paged-cache calls without a GPU: what the C ABI refuses, with the status it documents and before
anything touches a device; what the Python front-end refuses; and that the front-end hands every argument to
the parameter of its name."""
import contextlib
import ctypes

import pytest
import torch

from block_discrete_diffusion_tcgen05_b200 import _lib, attn, build
from test_binding_marshalling_cpu import PARAMS, STREAM, WS_BYTES, bf16, check_dims, rec  # noqa: F401

INVALID, UNSUPPORTED, SHAPE, ALIGNMENT, CAPACITY, WORKSPACE = 1, 2, 3, 4, 5, 6
P16 = 0x10000
DIMS = _lib.Dims(2, 4, 2, 64, 0.0)
PAGED = _lib.Pages(9, 32, 4, P16)
FLAT = _lib.Pages(2, 100, 1, None)
MIS = P16 + 8


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def sample_args(**kw):
    a = dict(q=P16, k=P16, v=P16, pages=PAGED, P=P16, kb=P16, vb=P16, out=P16, lse=None, dims=DIMS, S=4, ws=P16,
             n=1 << 30)
    a.update(kw)
    return list(a.values()) + [None]


def append_args(**kw):
    a = dict(k=P16, v=P16, pages=PAGED, P=P16, kn=P16, vn=P16, S=4, w=P16, pos=P16, tok=P16, dims=DIMS)
    a.update(kw)
    return list(a.values()) + [None]


def weigh_args(**kw):
    a = dict(q=P16, k=P16, pages=PAGED, P=P16, lse=P16, w=P16, out=P16, dims=DIMS, S=4)
    a.update(kw)
    return list(a.values()) + [None]


def evict_args(**kw):
    a = dict(k=P16, v=P16, pages=PAGED, P=P16, w=P16, pos=P16, tok=P16, keep=16, recent=4, wo=P16, po=P16, Po=P16,
             dims=DIMS, ws=P16, n=1 << 30)
    a.update(kw)
    return list(a.values()) + [None]


CALLS = [("e2d2_attn_decoder_sample_paged", sample_args), ("e2d2_kv_cache_append_paged", append_args),
         ("e2d2_kv_cache_weigh", weigh_args), ("e2d2_kv_cache_evict", evict_args)]

# what every call refuses alike
COMMON = [
    (dict(k=None), INVALID), (dict(P=None), INVALID), (dict(dims=_lib.Dims(0, 4, 2, 64, 0.0)), INVALID),
    (dict(dims=_lib.Dims(2, 4, 3, 64, 0.0)), INVALID), (dict(dims=_lib.Dims(2, 4, 2, 96, 0.0)), UNSUPPORTED),
    (dict(dims=_lib.Dims(2, 4, 2, 64, float("inf"))), INVALID),
    (dict(pages=_lib.Pages(0, 32, 4, P16)), INVALID), (dict(pages=_lib.Pages(9, 0, 4, P16)), INVALID),
    (dict(pages=_lib.Pages(9, 32, 0, P16)), INVALID), (dict(pages=_lib.Pages(9, -16, 4, P16)), INVALID),
    (dict(pages=_lib.Pages(9, 24, 4, P16)), UNSUPPORTED),            # pages of 24 rows
    (dict(pages=_lib.Pages(9, 32, 4, P16 + 2)), ALIGNMENT),
    (dict(pages=_lib.Pages(3, 100, 1, None)), INVALID),              # no table: one page per entry
    (dict(pages=_lib.Pages(2, 100, 2, None)), INVALID),
    (dict(pages=_lib.Pages(9, 1 << 20, 1 << 12, P16)), SHAPE),       # 2^32 rows per entry
    (dict(pages=_lib.Pages(2, (1 << 31) - 1, 1, None)), SHAPE),
    (dict(pages=_lib.Pages((1 << 31) - 1, 32, 4, P16)), SHAPE),
    (dict(dims=_lib.Dims(1025, 1, 1, 64, 0.0), pages=_lib.Pages(9, 32, 4, P16)), SHAPE),
    (dict(dims=_lib.Dims(1024, 64, 64, 64, 0.0), pages=_lib.Pages(9, 32, 4, P16)), SHAPE),
    (dict(k=MIS), ALIGNMENT), (dict(P=P16 + 2), ALIGNMENT),
]


@pytest.mark.parametrize("name,args", CALLS, ids=[c[0] for c in CALLS])
@pytest.mark.parametrize("change,status", COMMON)
def test_common_refusals(lib, name, args, change, status):
    assert getattr(lib, name)(*args(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID), (dict(kb=None), INVALID),
    # more places in the work stream than 31 bits count
    (dict(dims=_lib.Dims(1024, 64, 32, 64, 0.0), pages=_lib.Pages(9, 1 << 15, 1 << 6, P16), S=1), SHAPE),
    (dict(vb=None), INVALID), (dict(S=0), INVALID), (dict(S=-3), INVALID), (dict(S=1 << 28), SHAPE),
    (dict(q=MIS), ALIGNMENT), (dict(v=MIS), ALIGNMENT), (dict(kb=MIS), ALIGNMENT), (dict(vb=MIS), ALIGNMENT),
    (dict(out=MIS), ALIGNMENT), (dict(lse=P16 + 2), ALIGNMENT), (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE),
    (dict(ws=MIS), ALIGNMENT)])
def test_sample_refusals(lib, change, status):
    assert lib.e2d2_attn_decoder_sample_paged(*sample_args(**change)) == status


def test_sample_workspace_query(lib):
    f = lib.e2d2_attn_decoder_sample_paged_workspace
    assert f(DIMS, 4) > 0
    assert f(DIMS, 0) == 0 and f(_lib.Dims(2, 4, 2, 96, 0.0), 4) == 0


@pytest.mark.parametrize("change,status", [
    (dict(kn=None), INVALID), (dict(vn=None), INVALID), (dict(S=-1), INVALID), (dict(w=None), INVALID),
    (dict(pos=None), INVALID), (dict(tok=None), INVALID), (dict(S=129), CAPACITY),
    (dict(pages=FLAT, S=101), CAPACITY), (dict(kn=MIS), ALIGNMENT), (dict(vn=MIS), ALIGNMENT),
    (dict(w=P16 + 1), ALIGNMENT), (dict(pos=P16 + 2), ALIGNMENT), (dict(tok=P16 + 3), ALIGNMENT),
    (dict(S=0), 0)])
def test_append_refusals(lib, change, status):
    assert lib.e2d2_kv_cache_append_paged(*append_args(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(lse=None), INVALID), (dict(w=None), INVALID), (dict(out=None), INVALID),
    (dict(S=0), INVALID), (dict(S=1 << 28), SHAPE), (dict(q=MIS), ALIGNMENT), (dict(lse=P16 + 2), ALIGNMENT),
    (dict(w=P16 + 2), ALIGNMENT), (dict(out=P16 + 1), ALIGNMENT)])
def test_weigh_refusals(lib, change, status):
    assert lib.e2d2_kv_cache_weigh(*weigh_args(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(v=None), INVALID), (dict(w=None), INVALID), (dict(pos=None), INVALID), (dict(tok=None), INVALID),
    (dict(wo=None), INVALID), (dict(po=None), INVALID), (dict(Po=None), INVALID), (dict(keep=-1), INVALID),
    (dict(recent=-1), INVALID), (dict(recent=17), INVALID), (dict(ws=None), WORKSPACE), (dict(n=64), WORKSPACE),
    (dict(ws=MIS), ALIGNMENT), (dict(v=MIS), ALIGNMENT), (dict(pos=P16 + 2), ALIGNMENT), (dict(wo=P16 + 2), ALIGNMENT),
    (dict(po=P16 + 2), ALIGNMENT), (dict(Po=P16 + 2), ALIGNMENT), (dict(tok=P16 + 2), ALIGNMENT)])
def test_evict_refusals(lib, change, status):
    assert lib.e2d2_kv_cache_evict(*evict_args(**change)) == status


def test_evict_workspace_query(lib):
    f = lib.e2d2_kv_cache_evict_workspace
    assert f(DIMS, PAGED) > 0 and f(DIMS, FLAT) > 0
    assert f(DIMS, _lib.Pages(9, 24, 4, P16)) == 0
    # the front-end's query by row capacity is the pool's, with or without a table
    assert attn.evict_workspace_bytes(2, 2, 128) == f(DIMS, PAGED)
    assert attn.evict_workspace_bytes(2, 2, 100) == f(DIMS, FLAT)


# ------------------------------------------------------------------------------------------ marshalling
B, Hq, Hkv, S, d = 2, 4, 2, 8, 64


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def pool():
    return bf16(9, Hkv, 32, d), bf16(9, Hkv, 32, d), i32(B, 4)


def check_pages(pages, k, table):
    assert (pages.num_pages, pages.page_rows) == (k.shape[0], k.shape[2])
    assert pages.max_pages == (1 if table is None else table.shape[1])
    assert pages.page_table == (None if table is None else table.data_ptr())


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("block", [True, False])
def test_sample_marshalling(rec, paged, block):  # noqa: F811
    k, v, table = pool() if paged else (bf16(B, Hkv, 100, d), bf16(B, Hkv, 100, d), None)
    q, P = bf16(B, Hq, S, d), i32(B)
    kb, vb = (bf16(B, Hkv, S, d), bf16(B, Hkv, S, d)) if block else (None, None)
    ws = torch.zeros(WS_BYTES, dtype=torch.uint8)
    out, lse = attn.decoder_sample_paged(q, k, v, table, P, kb, vb, workspace=ws, scale=0.25)
    c = rec.call("e2d2_attn_decoder_sample_paged")
    assert (c["q_blk"], c["k_pages"], c["v_pages"], c["P_dev"]) == (q.data_ptr(), k.data_ptr(), v.data_ptr(), P.data_ptr())
    assert (c["k_blk"], c["v_blk"]) == ((kb.data_ptr(), vb.data_ptr()) if block else (None, None))
    assert (c["out"], c["lse"], c["S"], c["workspace"], c["ws_bytes"]) == (out.data_ptr(), lse.data_ptr(), S, ws.data_ptr(), WS_BYTES)
    assert c["stream"] == STREAM
    check_pages(c["pages"], k, table)
    check_dims(c["dims"], B, Hq, Hkv, d, 0.25)
    assert out.shape == q.shape and lse.shape == (B, Hq, S)


@pytest.mark.parametrize("tracked", [True, False])
def test_append_marshalling(rec, tracked):  # noqa: F811
    k, v, table = pool()
    kn, vn, P = bf16(B, Hkv, S, d), bf16(B, Hkv, S, d), i32(B)
    w, pos, tok = (torch.zeros(B, Hkv, 128), i32(B, Hkv, 128), i32(B)) if tracked else (None, None, None)
    attn.kv_cache_append_paged(k, v, table, P, kn, vn, weight=w, pos=pos, tokens=tok)
    c = rec.call("e2d2_kv_cache_append_paged")
    assert (c["k_pages"], c["v_pages"], c["P_dev"], c["k_new"], c["v_new"], c["S_new"]) == (
        k.data_ptr(), v.data_ptr(), P.data_ptr(), kn.data_ptr(), vn.data_ptr(), S)
    assert (c["weight"], c["pos"], c["tokens_dev"]) == tuple(None if t is None else t.data_ptr() for t in (w, pos, tok))
    check_pages(c["pages"], k, table)
    check_dims(c["dims"], B, Hkv, Hkv, d, None)


@pytest.mark.parametrize("in_place", [True, False])
def test_weigh_marshalling(rec, in_place):  # noqa: F811
    k, _, table = pool()
    q, P, lse, w = bf16(B, Hq, S, d), i32(B), torch.zeros(B, Hq, S), torch.zeros(B, Hkv, 128)
    out = None if in_place else torch.zeros_like(w)
    got = attn.kv_cache_weigh(q, k, table, P, lse, w, out=out, scale=0.5)
    c = rec.call("e2d2_kv_cache_weigh")
    assert got is (w if in_place else out)
    assert (c["q"], c["k_pages"], c["P_dev"], c["lse"], c["weight"], c["weight_out"], c["S"]) == (
        q.data_ptr(), k.data_ptr(), P.data_ptr(), lse.data_ptr(), w.data_ptr(), got.data_ptr(), S)
    check_pages(c["pages"], k, table)
    check_dims(c["dims"], B, Hq, Hkv, d, 0.5)


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_marshalling(rec, in_place):  # noqa: F811
    k, v, table = pool()
    P, tok, w, pos = i32(B), i32(B), torch.zeros(B, Hkv, 128), i32(B, Hkv, 128)
    more = {} if in_place else dict(weight_out=torch.zeros_like(w), pos_out=torch.zeros_like(pos), P_out=i32(B))
    ws = torch.zeros(WS_BYTES, dtype=torch.uint8)
    got = attn.kv_cache_evict(k, v, table, P, w, pos, tok, 20, recent=3, workspace=ws, **more)
    c = rec.call("e2d2_kv_cache_evict")
    wo, po, Po = (w, pos, P) if in_place else more.values()
    assert got is Po
    assert (c["k_pages"], c["v_pages"], c["P_dev"], c["weight"], c["pos"], c["tokens_dev"]) == tuple(
        t.data_ptr() for t in (k, v, P, w, pos, tok))
    assert (c["weight_out"], c["pos_out"], c["P_out"]) == tuple(t.data_ptr() for t in (wo, po, Po))
    assert (c["keep"], c["recent"], c["workspace"], c["ws_bytes"]) == (20, 3, ws.data_ptr(), WS_BYTES)
    check_pages(c["pages"], k, table)
    check_dims(c["dims"], B, Hkv, Hkv, d, None)


def test_front_end_refusals(rec):  # noqa: F811
    k, v, table = pool()
    q, P, kn = bf16(B, Hq, S, d), i32(B), bf16(B, Hkv, S, d)
    w, pos, lse = torch.zeros(B, Hkv, 128), i32(B, Hkv, 128), torch.zeros(B, Hq, S)
    ws = torch.zeros(WS_BYTES, dtype=torch.uint8)
    bad = [
        lambda: attn.decoder_sample_paged(q, k, v[:8].clone(), table, P, workspace=ws),
        lambda: attn.decoder_sample_paged(q, k, v, None, P, workspace=ws),              # 9 pages, 2 entries
        lambda: attn.decoder_sample_paged(q, k, v, i32(B + 1, 4), P, workspace=ws),
        lambda: attn.decoder_sample_paged(q, k, v, table, i32(B + 1), workspace=ws),
        lambda: attn.decoder_sample_paged(q, k, v, table, P, kn, None, workspace=ws),
        lambda: attn.decoder_sample_paged(q, k, v, table, P, kn[:, :, :4].clone(), kn[:, :, :4].clone(), workspace=ws),
        lambda: attn.decoder_sample_paged(q, k, v, table, P, workspace=ws, out=bf16(B, Hq, S + 1, d)),
        lambda: attn.decoder_sample_paged(bf16(B, Hq, S, 32), k, v, table, P, workspace=ws),
        lambda: attn.kv_cache_append_paged(k, v, table, P, kn, kn[:, :, :4].clone()),
        lambda: attn.kv_cache_append_paged(k, v, table, P, kn, kn, weight=w),
        lambda: attn.kv_cache_append_paged(k, v, table, P, kn, kn, weight=w[:, :, :64].clone(), pos=pos, tokens=i32(B)),
        lambda: attn.kv_cache_weigh(q, k, table, P, lse[:, :, :4].clone(), w),
        lambda: attn.kv_cache_weigh(q, k, table, P, lse, w[:, :1].clone()),
        lambda: attn.kv_cache_weigh(q, k, table, P, lse, w, out=torch.zeros(B, Hkv, 64)),
        lambda: attn.kv_cache_evict(k, v[:8].clone(), table, P, w, pos, i32(B), 20, workspace=ws),
        lambda: attn.kv_cache_evict(k, v, table, P, w, pos[:, :, :64].clone(), i32(B), 20, workspace=ws),
        lambda: attn.kv_cache_evict(k, v, table, P, w, pos, i32(B + 1), 20, workspace=ws),
        lambda: attn.kv_cache_evict(k, v, table, P, w, pos, i32(B), 20, P_out=i32(B + 1), workspace=ws),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    assert not [c for c in rec.calls if not c[0].endswith("_workspace")]


def test_cpu_tensors_are_refused():
    k, v, table = pool()
    with pytest.raises(ValueError, match="CUDA"):
        attn.decoder_sample_paged(bf16(B, Hq, S, d), k, v, table, i32(B))
    with pytest.raises(ValueError, match="CUDA"):
        attn.kv_cache_evict(k, v, table, i32(B), torch.zeros(B, Hkv, 128), i32(B, Hkv, 128), i32(B), 5)


def test_status_of_a_bad_page_has_a_name(lib):
    assert lib.e2d2_status_string(10) == b"E2D2_ERR_PAGE"
    assert ctypes.sizeof(_lib.Pages) == 24


# --------------------------------------------------------------------------------- the reference itself
def test_reference_agrees_with_the_oracle(oracle):
    """tests/paged_reference.py's sampling step is the C oracle's ragged step on the gathered rows; a planted
    mistake (one row more) is seen by its tolerance."""
    import numpy as np
    import paged_reference as R

    cache = R.Cache(3, 2, 64, 16, [37, 0, 90], 96, 11)
    q, kb, vb = R.bf16((3, 4, 5, 64), 12), R.bf16((3, 2, 5, 64), 13), R.bf16((3, 2, 5, 64), 14)
    pad = lambda t, b, h: np.pad(R.f64(cache.rows(t, b, h, cache.P[b])).reshape(-1, 64), ((0, 96 - cache.P[b]), (0, 0)))  # noqa: E731
    full = [np.stack([np.stack([pad(t, b, h) for h in range(2)]) for b in range(3)]) for t in (cache.k, cache.v)]
    want_o, want_l = oracle.decoder_sample_ragged(R.f64(q), full[0], full[1], cache.P, R.f64(kb), R.f64(vb))
    out, lse, tol_o, tol_l = R.sample(cache, q, kb, vb)
    assert np.abs(out - want_o).max() < 1e-9 and np.abs(lse - want_l).max() < 1e-9
    cache.P[0] += 1
    cache.k.nan_to_num_(0.0), cache.v.nan_to_num_(0.0)
    out2, lse2, _, _ = R.sample(cache, q, kb, vb)
    assert (np.abs(lse2[0] - lse[0]) > tol_l[0]).all()


def test_reference_eviction_on_a_case_by_hand():
    import numpy as np
    import paged_reference as R

    w = np.array([5, 1, 3, np.nan, 3, 9], np.float32)
    pos = np.array([4, 1, 2, 3, 0, 5], np.int32)
    # recent = 1 protects row 5 (position 5 of 6 tokens); then rows 0 (5) and 2 (3, before row 4's 3)
    moves, w2, p2 = R.evict(6, w, pos, 6, 3, 1)
    assert moves == [(5, 1)] and w2.tolist() == [5, 9, 3] and p2.tolist() == [4, 5, 2]


def test_a_call_by_keywords_has_its_tensors_device_checked_and_current(monkeypatch):
    class OnDevice(torch.Tensor):
        index = 1
        is_cuda = True

        def get_device(self):
            return self.index

    def tensor(index):
        t = torch.zeros(1).as_subclass(OnDevice)
        t.index = index
        return t

    entered = []

    @contextlib.contextmanager
    def device(idx):
        entered.append(idx)
        yield

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    call = attn._device_guard(lambda q, k: "ran")
    assert call(tensor(1), tensor(1)) == "ran" and entered == [1]
    assert call(q=None, k=tensor(1)) == "ran" and entered == [1, 1]
    for kw in ({"q": tensor(1), "k": tensor(0)}, {"q": tensor(0), "k": torch.zeros(1)}):
        with pytest.raises(ValueError, match="every tensor must be on"):
            call(**kw)
