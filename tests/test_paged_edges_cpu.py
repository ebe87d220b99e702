"""The paged-cache calls' arguments at their edges, without a GPU: counts that 32 bits do not hold, blocks of no rows."""
import pytest
import torch

from block_discrete_diffusion_tcgen05_b200 import _lib, attn, build
from test_binding_marshalling_cpu import WS_BYTES, bf16, rec  # noqa: F401

B, Hkv, d = 2, 2, 64


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.mark.parametrize("keep,recent", [(2 ** 31, 0), (2 ** 32, 0), (2 ** 32 + 20, 3), (20, 2 ** 32 + 3), (-2 ** 32, 0),
                                         (2 ** 63, 0)])
def test_a_budget_that_32_bits_do_not_hold_is_refused(rec, keep, recent):  # noqa: F811
    """Not taken by its low 32 bits: a budget of 2^32 rows would evict everything."""
    k, v, table = bf16(9, Hkv, 32, d), bf16(9, Hkv, 32, d), i32(B, 4)
    ws = torch.zeros(WS_BYTES, dtype=torch.uint8)
    with pytest.raises(ValueError, match="32 bits"):
        attn.kv_cache_evict(k, v, table, i32(B), torch.zeros(B, Hkv, 128), i32(B, Hkv, 128), i32(B), keep, recent=recent,
                            workspace=ws)
    assert not rec.calls


def test_the_largest_budget_is_passed_on(rec):  # noqa: F811
    k, v, table = bf16(9, Hkv, 32, d), bf16(9, Hkv, 32, d), i32(B, 4)
    ws = torch.zeros(WS_BYTES, dtype=torch.uint8)
    attn.kv_cache_evict(k, v, table, i32(B), torch.zeros(B, Hkv, 128), i32(B, Hkv, 128), i32(B), 2 ** 31 - 1,
                        recent=2 ** 31 - 1, workspace=ws)
    c = rec.call("e2d2_kv_cache_evict")
    assert (c["keep"], c["recent"]) == (2 ** 31 - 1, 2 ** 31 - 1)


def test_an_append_of_no_rows_does_nothing():
    """An empty tensor has no address: the C call takes none with S_new = 0, checks the rest and returns."""
    build.build()
    lib = _lib.load()
    p = 0x10000
    pages, dims = _lib.Pages(9, 32, 4, p), _lib.Dims(B, Hkv, Hkv, d, 0.0)
    empty = bf16(B, Hkv, 0, d)
    assert empty.data_ptr() == 0
    assert lib.e2d2_kv_cache_append_paged(p, p, pages, p, None, None, 0, p, p, p, dims, None) == 0
    assert lib.e2d2_kv_cache_append_paged(p, p, pages, None, None, None, 0, p, p, p, dims, None) == 1
    for k, v in ((None, p), (p, None)):
        assert lib.e2d2_kv_cache_append_paged(p, p, pages, p, k, v, 1, p, p, p, dims, None) == 1
