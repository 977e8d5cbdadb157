"""More refusals of the page and 8-bit cache calls, on the host: validation runs before any launch, so nothing here needs a
GPU.  Pointers are made-up addresses that nothing dereferences."""
import ctypes
import os

import pytest
import torch

from paged_block_sparse_kv_b200 import vx

FAKE, FAR = 4096, 1 << 40
INVALID = vx.VX_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(vx.LIB_PATH):
        pytest.skip("libvx.so not built")
    return vx.lib()


def _geo(**kw):
    g = dict(batch=2, num_q_heads=16, num_kv_heads=8, head_dim_qk=128, head_dim_v=128, page_size=16,
             mla_shared_kv=0, num_pool_pages=5000)
    g.update(kw)
    return ctypes.byref(vx.vx_geometry(**g))


def _table(max_pages=10, ptr=256):
    return ctypes.byref(vx.vx_page_table(ptr, ptr, ptr, max_pages))


def _pool(**kw):
    p = dict(k_cache=1 << 30, v_cache=1 << 34, centroids=None, k_scale=None, v_scale=None, elem_bytes=2, num_pages=5000)
    p.update(kw)
    return ctypes.byref(vx.vx_page_pool(**p))


@pytest.mark.parametrize("off", [4, 8, 12])
@pytest.mark.parametrize("pages", [100, 5000])
def test_compaction_counts_apart_and_misaligned(L, off, pages):
    """ref_out is written in 16-byte stores when it is not ref_in: a row of a double buffer of odd length is refused."""
    g = _geo(num_pool_pages=pages)
    n = L.vx_page_workspace_size(g, 1)
    assert L.vx_compact_pages(g, _pool(num_pages=pages), _table(), FAKE, FAKE, FAR + off, FAR + (1 << 20), FAKE, FAKE, n,
                              None, None) == INVALID
    assert b"ref_out" in L.vx_last_error()


def test_more_new_rows_than_31_bits(L):
    c = ctypes.byref(vx.vx_quant_cache(vx.VX_QUANT_INT8, FAKE, FAKE, FAKE, FAKE))
    assert L.vx_quant_update(_geo(), _table(), c, FAKE, FAKE, FAKE, 1 << 31, FAKE, None, None) == vx.VX_ERR_UNSUPPORTED


@pytest.mark.parametrize("pages", [1 << 31, 1 << 60, 1 << 61, (1 << 63) - 1])
def test_pools_of_more_pages_than_31_bits_times_heads(L, pages):
    """Also where the product of pages and heads wraps in 64 bits to a small number."""
    n = L.vx_page_workspace_size(_geo(), 1)
    assert L.vx_copy_pages(_geo(), _pool(num_pages=pages), _pool(k_cache=FAR, v_cache=FAR + (1 << 33)), FAKE, FAKE, 1, FAKE,
                           n, None, None) == INVALID
    assert L.vx_page_workspace_size(_geo(num_pool_pages=pages), 1) == 0


def test_page_workspace_serves_every_batch(L):
    """A workspace for a pool and its new rows is large enough whatever the number of old rows of the call is."""
    n = L.vx_page_workspace_size(_geo(batch=1), 7)
    for batch in (1, 2, 500, 4096):
        g = _geo(batch=batch)
        assert L.vx_page_workspace_size(g, 7) == n
        call = lambda size: L.vx_update_table(g, _pool(), _table(), FAKE, FAKE, FAKE, 7, FAKE, FAR, 100, FAR + 4096, 4, FAKE,
                                              FAKE, size, None, None)
        # (without a GPU the launch fails, after every check of the arguments)
        assert call(n) not in (vx.VX_ERR_WORKSPACE, INVALID) if not torch.cuda.is_available() else True
        assert call(n - 1) == vx.VX_ERR_WORKSPACE


def test_copies_between_pools_that_share_any_array(L):
    """Scales, centroids, and one pool's keys under the other's values: a copy would overwrite what another copy reads."""
    n = L.vx_page_workspace_size(_geo(), 1)

    def copy(**kw):
        src = dict(elem_bytes=1, centroids=1 << 36, k_scale=1 << 37, v_scale=(1 << 37) + (1 << 30))
        dst = dict(elem_bytes=1, k_cache=FAR, v_cache=FAR + (1 << 34), centroids=FAR + (1 << 36), k_scale=FAR + (1 << 37),
                   v_scale=FAR + (1 << 37) + (1 << 30))
        dst.update(kw)
        return L.vx_copy_pages(_geo(), _pool(**src), _pool(**dst), FAKE, FAKE, 0, FAKE, n, None, None)

    assert copy() == vx.VX_OK  # no copies: nothing is launched
    last = 5000 * 8 * 4 - 4  # the last scale
    for kw in (dict(k_scale=1 << 37), dict(v_scale=(1 << 37) + last), dict(k_scale=(1 << 37) + (1 << 30) - last),
               dict(centroids=(1 << 36) + 4096), dict(v_cache=1 << 30), dict(k_cache=(1 << 34) + 16)):
        assert copy(**kw) == INVALID, kw
    assert copy(k_scale=(1 << 37) + last + 4) == vx.VX_OK


def test_binding_refuses_new_tables_in_the_old_ones_memory():
    """The C call knows the old page_indices' start alone; the binding knows its extent."""
    geo = vx.Geometry(2, 4, 2, 64, 64, 16, False, 10)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    codes = torch.zeros(10, 2, 16, 64, dtype=torch.int8)
    pool, both = vx.PagePool(codes, codes.clone()), i32(40)
    old = vx.PageTable(i32(2), both[:24], i32(2), 4)
    call = lambda idx, lens=None: vx.vx_update_table(geo, pool, old, i32(10), i32(2), i32(2),
                                                     vx.PageTable(i32(2), idx, i32(2) if lens is None else lens, 4), i32(10),
                                                     i32(8))
    for idx in (both[16:32], both[23:], both[:24], both[4:8], old.seq_lens):
        with pytest.raises(ValueError, match="old table's memory"):
            call(idx)
    for lens in (both[22:24], old.seq_lens, old.page_ptr):
        with pytest.raises(ValueError, match="old table's memory"):
            call(i32(16), lens)
    with pytest.raises(ValueError, match="CUDA"):  # apart: the next check
        call(both[24:])
    compact = lambda idx: vx.vx_compact_pages(geo, pool, old, i32(10), idx, i32(10), i32(10), i32(1), i32(8))
    with pytest.raises(ValueError, match="apart"):
        compact(both[8:32])
    for idx in (both[:24], i32(24)):
        with pytest.raises(ValueError, match="CUDA"):
            compact(idx)
