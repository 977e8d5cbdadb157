"""Refusals of the 8-bit cache and page calls (no GPU needed: validation runs before any launch), and the plain
implementations the GPU tests compare with, on cases worked by hand."""
import ctypes
import os

import numpy as np
import pytest
import torch

import quant_ref as ref
from paged_block_sparse_kv_b200 import vx

FAKE = 4096  # an aligned non-NULL address; validation fails before anything dereferences it
F0 = ctypes.c_float(0.0)
INVALID, UNSUPPORTED, WORKSPACE = vx.VX_ERR_INVALID_ARG, vx.VX_ERR_UNSUPPORTED, vx.VX_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(vx.LIB_PATH):
        pytest.skip("libvx.so not built")
    return vx.lib()


def _geo(**kw):
    g = dict(batch=2, num_q_heads=16, num_kv_heads=8, head_dim_qk=128, head_dim_v=128, page_size=16,
             mla_shared_kv=0, num_pool_pages=100)
    g.update(kw)
    return ctypes.byref(vx.vx_geometry(**g))


MLA = dict(num_q_heads=16, num_kv_heads=1, head_dim_qk=576, head_dim_v=512, page_size=64, mla_shared_kv=1)


def _table(max_pages=10, ptr=256):
    return ctypes.byref(vx.vx_page_table(ptr, ptr, ptr, max_pages))


def _cache(**kw):
    c = dict(format=vx.VX_QUANT_INT8, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE)
    c.update(kw)
    return ctypes.byref(vx.vx_quant_cache(**c))


def _pool(**kw):
    p = dict(k_cache=1 << 20, v_cache=1 << 30, centroids=None, k_scale=None, v_scale=None, elem_bytes=2, num_pages=100)
    p.update(kw)
    return ctypes.byref(vx.vx_page_pool(**p))


CACHES = [dict(format=0), dict(format=3), dict(k_cache=None), dict(v_cache=FAKE + 8), dict(k_scale=None),
          dict(v_scale=FAKE + 2)]


@pytest.mark.parametrize("kw", CACHES)
def test_bad_caches(L, kw):
    c = _cache(**kw)
    assert L.vx_quant_update(_geo(), _table(), c, FAKE, FAKE, FAKE, 2, None, None, None) == INVALID
    assert L.vx_sparse_decode_quant(_geo(), _table(), FAKE, c, FAKE, 4, F0, 8, FAKE, None, FAKE, 1 << 30, None,
                                    None) == INVALID
    assert L.vx_block_topk_decode_quant(_geo(), _table(), FAKE, c, FAKE, 4, 0, 0, F0, 0, 8, FAKE, None, None, None, FAKE,
                                        1 << 30, None, None) == INVALID
    assert L.vx_block_topk_decode_append_quant(_geo(), _table(), FAKE, c, FAKE, FAKE, FAKE, 4, 0, 0, F0, 0, 8, FAKE,
                                               None, None, None, FAKE, 1 << 30, None, None) == INVALID
    assert L.vx_last_error()


def test_quant_calls_refuse(L):
    c = _cache()
    up = lambda g=None, t=None, cache=c, cen=FAKE, k=FAKE, v=FAKE, n=2, first=None, err=None: \
        L.vx_quant_update(g or _geo(), t or _table(), cache, cen, k, v, n, first, err, None)
    assert up(g=_geo(**MLA)) == UNSUPPORTED
    assert up(g=_geo(head_dim_qk=96, head_dim_v=96)) == UNSUPPORTED
    assert up(t=_table(max_pages=0)) == INVALID
    for kw in (dict(cache=None), dict(cen=None), dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(first=FAKE + 2),
               dict(err=FAKE + 1), dict(n=1), dict(n=-1, first=FAKE)):
        assert up(**kw) == INVALID
    dec = lambda g=None, cache=c, q=FAKE, sel=FAKE, k=4, scale=0.0, out=FAKE, lse=None, ws=FAKE, n=1 << 30, err=None: \
        L.vx_sparse_decode_quant(g or _geo(), _table(), q, cache, sel, k, ctypes.c_float(scale), 8, out, lse, ws, n, err,
                                 None)
    assert dec(g=_geo(**MLA)) == UNSUPPORTED
    for kw in (dict(cache=None), dict(q=None), dict(sel=None), dict(k=0), dict(scale=float("nan")), dict(out=None),
               dict(out=FAKE + 2), dict(lse=FAKE + 4), dict(err=FAKE + 1)):
        assert dec(**kw) == INVALID
    assert dec(ws=None) == WORKSPACE and dec(n=16) == WORKSPACE
    app = lambda cache, k, v, n: L.vx_block_topk_decode_append_quant(
        _geo(), _table(), FAKE, cache, FAKE, k, v, 4, 0, 0, F0, 0, 8, FAKE, None, None, None, FAKE, n, None, None)
    assert app(c, None, FAKE, 1 << 30) == INVALID and app(c, FAKE, None, 1 << 30) == INVALID
    assert app(None, FAKE, FAKE, 1 << 30) == INVALID and app(c, FAKE, FAKE, 16) == WORKSPACE
    assert L.vx_block_topk_decode_quant(_geo(), _table(), FAKE, None, FAKE, 4, 0, 0, F0, 0, 8, FAKE, None, None, None,
                                        FAKE, 1 << 30, None, None) == INVALID


POOLS = [dict(k_cache=None), dict(k_cache=(1 << 20) + 8), dict(v_cache=None), dict(elem_bytes=4), dict(num_pages=0),
         dict(num_pages=1 << 40), dict(k_scale=FAKE), dict(k_scale=FAKE, v_scale=FAKE),
         dict(elem_bytes=1, k_scale=FAKE, v_scale=FAKE + 2), dict(centroids=FAKE + 2), dict(num_pages=99)]


@pytest.mark.parametrize("kw", POOLS)
def test_bad_pools(L, kw):
    p, big = _pool(**kw), 1 << 30
    assert L.vx_copy_pages(_geo(), _pool(), p, FAKE, FAKE, 1, FAKE, big, None, None) == INVALID
    assert L.vx_update_table(_geo(), p, _table(), FAKE, FAKE, FAKE, 2, FAKE, 1 << 25, 10, FAKE, 4, FAKE, FAKE, big, None,
                             None) == INVALID
    assert L.vx_compact_pages(_geo(), p, _table(), FAKE, FAKE, FAKE, 1 << 25, FAKE, FAKE, big, None, None) == INVALID
    assert L.vx_last_error()


def test_copy_refuses(L):
    n = vx.lib().vx_page_workspace_size(_geo(), 1)
    cp = lambda src, dst, s=FAKE, d=FAKE, count=1, ws=FAKE, size=n, g=None: L.vx_copy_pages(
        g or _geo(), src, dst, s, d, count, ws, size, None, None)
    a, far = _pool(), 1 << 40
    other = _pool(k_cache=far, v_cache=far + (1 << 30))
    assert cp(a, other, count=0) == vx.VX_OK  # nothing to do, nothing launched
    assert cp(a, other, count=-1) == INVALID
    assert cp(a, other, s=None) == INVALID and cp(a, other, d=FAKE + 2) == INVALID
    assert cp(a, other, ws=None) == WORKSPACE and cp(a, other, size=n - 1) == WORKSPACE
    assert cp(None, other) == INVALID and cp(a, None) == INVALID
    assert cp(a, other, count=2 ** 31 - 1) == UNSUPPORTED  # more pieces than 31 bits count
    assert cp(a, _pool(k_cache=far, v_cache=far + (1 << 30), centroids=FAKE)) == INVALID      # other arrays
    assert cp(_pool(elem_bytes=1), other) == INVALID                                          # other element size
    assert cp(a, _pool(v_cache=far)) == INVALID                                               # one k_cache, two v_caches
    assert cp(a, _pool(k_cache=(1 << 20) + 4096, v_cache=far)) == INVALID                     # overlapping keys
    assert cp(a, _pool(k_cache=far, v_cache=(1 << 30) - 4096)) == INVALID                     # overlapping values
    mla = dict(k_cache=far, v_cache=None)
    assert cp(_pool(**mla), _pool(), g=_geo(**MLA)) == INVALID                                # v_cache in an MLA pool


def test_update_refuses(L):
    g = _geo()
    n = L.vx_page_workspace_size(g, 2)
    far = 1 << 40

    def up(**kw):
        a = dict(ref=FAKE, parent=FAKE, grow=FAKE, rows=2, ptr=FAKE, idx=far, num=10, lens=far + 4096, top=4, out=FAKE,
                 ws=FAKE, size=n, err=None)
        a.update(kw)
        return L.vx_update_table(g, _pool(), _table(), a["ref"], a["parent"], a["grow"], a["rows"], a["ptr"], a["idx"],
                                 a["num"], a["lens"], a["top"], a["out"], a["ws"], a["size"], a["err"], None)

    for kw in (dict(rows=0), dict(rows=4097), dict(top=0), dict(top=1 << 28), dict(num=0), dict(num=1 << 31),
               dict(ref=None), dict(ref=FAKE + 4), dict(out=FAKE + 4), dict(out=FAKE + 16), dict(parent=None),
               dict(grow=None), dict(ptr=None), dict(idx=None), dict(idx=far + 2), dict(lens=None), dict(err=FAKE + 1),
               dict(idx=256), dict(lens=260)):  # the old table's own memory
        assert up(**kw) == INVALID, kw
    assert up(ws=None) == WORKSPACE and up(size=n - 1) == WORKSPACE


def test_compact_refuses(L):
    n, far = L.vx_page_workspace_size(_geo(), 1), 1 << 40

    def co(**kw):
        a = dict(ref=FAKE, idx=FAKE, out=FAKE, remap=far, live=FAKE, ws=FAKE, size=n)
        a.update(kw)
        return L.vx_compact_pages(_geo(), _pool(), _table(), a["ref"], a["idx"], a["out"], a["remap"], a["live"], a["ws"],
                                  a["size"], None, None)

    for kw in (dict(ref=None), dict(ref=FAKE + 4), dict(idx=None), dict(out=None), dict(out=FAKE + 16), dict(remap=None),
               dict(remap=FAKE), dict(live=None), dict(live=FAKE + 2)):
        assert co(**kw) == INVALID, kw
    assert co(ws=None) == WORKSPACE and co(size=n - 1) == WORKSPACE


def test_page_workspace_size(L):
    assert L.vx_page_workspace_size(_geo(), 0) == 0 and L.vx_page_workspace_size(_geo(), 4097) == 0
    assert L.vx_page_workspace_size(_geo(page_size=8), 1) == 0
    a = L.vx_page_workspace_size(_geo(), 1)
    assert a >= 4 * 100 and L.vx_page_workspace_size(_geo(), 4096) >= a + 16000
    assert L.vx_page_workspace_size(_geo(num_pool_pages=1000), 1) > a


def test_binding_checks_types_shapes_and_devices():
    geo = vx.Geometry(2, 4, 2, 64, 64, 16, False, 10)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    tab = vx.PageTable(i32(2), i32(8), i32(2), 4)
    codes = torch.zeros(10, 2, 16, 64, dtype=torch.int8)
    cache = vx.QuantCache(codes, codes, torch.ones(10, 2), torch.ones(10, 2))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    args = dict(q=bf(2, 4, 64), cache=cache, sel=i32(2, 2, 3), k=3, out=bf(2, 4, 64),
                ws=torch.zeros(8, dtype=torch.uint8))

    def call(**kw):
        a = {**args, **kw}
        vx.vx_sparse_decode_quant(a.get("geo", geo), a.get("tab", tab), a["q"], a["cache"], a["sel"], a["k"], a["out"],
                                  a["ws"])

    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(ValueError, match="sel"):
        call(k=4)
    with pytest.raises(ValueError, match="q has shape"):
        call(q=bf(2, 5, 64))
    with pytest.raises(ValueError, match="contiguous"):
        call(q=bf(2, 64, 4).transpose(1, 2))
    with pytest.raises(TypeError):
        call(q=torch.zeros(2, 4, 64))
    with pytest.raises(TypeError):
        call(cache=vx.QuantCache(codes.to(torch.uint8), codes, torch.ones(10, 2), torch.ones(10, 2)))
    with pytest.raises(TypeError):
        call(cache=vx.QuantCache(codes, codes.view(torch.float8_e4m3fn), torch.ones(10, 2), torch.ones(10, 2)))
    with pytest.raises(ValueError, match="k_scale"):
        call(cache=vx.QuantCache(codes, codes, torch.ones(10, 4), torch.ones(10, 2)))
    with pytest.raises(ValueError, match="seq_lens"):
        call(tab=vx.PageTable(i32(2), i32(8), i32(3), 4))
    pool = vx.PagePool(codes, codes)
    with pytest.raises(ValueError, match="dst_pages"):
        vx.vx_copy_pages(geo, pool, pool, i32(2), i32(3), i32(8))
    with pytest.raises(ValueError, match="centroids"):
        vx.vx_copy_pages(geo, pool, vx.PagePool(codes, codes, bf(10, 2, 32)), i32(2), i32(2), i32(8))
    with pytest.raises(ValueError, match="new_ref"):
        vx.vx_update_table(geo, pool, tab, i32(10), i32(2), i32(2), tab, i32(9), i32(8))
    with pytest.raises(ValueError, match="remap"):
        vx.vx_compact_pages(geo, pool, tab, i32(10), i32(8), i32(10), i32(11), i32(1), i32(8))


# ------------------------------------------------------------------------------------------------ the plain forms

def test_e4m3_against_torch():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    t = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.E4M3, equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 4001), 2.0 ** np.linspace(-12, 8, 2000), [0.0, -0.0, 2.0 ** -10,
                        3 * 2.0 ** -10, -(2.0 ** -10), 448.0, 232.0, 248.0]])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    exact = x.astype(np.float32) == x
    assert np.array_equal(ref.nearest(x.astype(np.float32).astype(np.float64), "e4m3"), want) and exact.any()


def test_int8_and_scales_by_hand():
    assert list(ref.nearest(np.array([0.5, 1.5, -0.5, -2.5, 126.5, 200.0, -200.0]), "int8").view(np.int8)) == \
        [0, 2, 0, -2, 126, 127, -127]
    assert ref.pow2_scale(127.0, "int8") == 1 and ref.pow2_scale(127.5, "int8") == 2 and ref.pow2_scale(63, "int8") == 0.5
    assert ref.pow2_scale(448.0, "e4m3") == 1 and ref.pow2_scale(449.0, "e4m3") == 2
    assert ref.pow2_scale(0.0, "e4m3") == 2.0 ** -126
    x = torch.randn(1000, generator=torch.Generator().manual_seed(0), dtype=torch.float32)
    assert np.array_equal(ref.to_bf16(x.double().numpy()), x.to(torch.bfloat16).double().numpy())


def test_quant_update_by_hand():
    """One head, pages of 2: three tokens arrive one by one; the second doubles the first page's scale."""
    k, ks, cen = np.zeros((2, 1, 2, 1), np.uint8), np.zeros((2, 1)), np.zeros((2, 1, 1))
    for t, x in enumerate([100.0, 200.0, -3.0]):
        ref.quant_update(k, ks, cen, np.array([[[x]]]), [0], [1, 0], [t + 1], [t], "int8")
    assert k.view(np.int8)[1, 0, :, 0].tolist() == [50, 100] and ks[1, 0] == 2 and cen[1, 0, 0] == 150
    assert k.view(np.int8)[0, 0, 0, 0] == -96 and ks[0, 0] == 2.0 ** -5 and cen[0, 0, 0] == -3


def test_attention_against_torch():
    rng = np.random.default_rng(0)
    kv, vv = rng.standard_normal((2, 6, 1, 4, 8))
    q, idx = rng.standard_normal((1, 2, 8)), np.array([3, 1, 5])
    out, lse, *_ = ref.attend(q, kv, vv, [0], idx, [10], np.array([[[0, 2, -1]]]), 0.5)
    K, V = (torch.from_numpy(np.concatenate([a[3, 0], a[5, 0, :2]])) for a in (kv, vv))
    s = 0.5 * torch.from_numpy(q[0]) @ K.T
    assert np.allclose(out[0], (s.softmax(-1) @ V).numpy(), rtol=1e-13)
    assert np.allclose(lse[0], torch.logsumexp(s, -1).numpy(), rtol=1e-13)


def test_table_update_by_hand():
    """Pages of 4; rows of 6 and 4 tokens on pages (5, 2) and (0); page 3 is the caller's."""
    data = np.arange(8)
    refs = np.array([1, 0, 1, 1, 0, 1, 0, 0])
    rows, lens, after = ref.update_table(4, [0, 2], [5, 2, 0], [6, 4], refs, [0, 0, -1], [1, 3, 2], [data])
    # row 0 keeps the last page 2 (7 tokens fit); row 1 shares 5, gets a copy of 2 in page 1 and page 4; row 2 gets 6
    assert rows == [[5, 2], [5, 1, 4], [6]] and lens == [7, 9, 2]
    assert after.tolist() == [0, 1, 1, 1, 1, 2, 1, 0] and data.tolist() == [0, 2, 2, 3, 4, 5, 6, 7]
    assert ref.update_table(4, [0], [0], [4], [1, 0], [0, 0], [4, 4], []) is None


def test_compact_by_hand():
    data = np.arange(6) * 10
    remap, after, n = ref.compact(np.array([0, 2, 0, 0, 1, 3]), [data])
    assert n == 3 and remap.tolist() == [-1, 1, -1, -1, 0, 2] and after.tolist() == [1, 2, 3, 0, 0, 0]
    assert data.tolist() == [40, 10, 50, 30, 40, 50]
