"""8-bit caches on the GPU: the quantising write bit for bit, the attention within bounds derived per element, both against
plain 64-bit implementations; a decode loop of the three together; graphs, streams, far pages."""
import numpy as np
import pytest
import torch

import quant_ref as ref
from paged_block_sparse_kv_b200 import vx

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMTS = ["int8", "e4m3"]


class Case:
    """A quantised cache with a page table: random codes, the worst code in every slot past a length and on every page
    that no row names."""

    def __init__(self, fmt, L, Hq, Hkv, D, P, seed=0, pool=None, at_end=False):
        self.fmt, self.L, self.Hq, self.Hkv, self.D, self.P = fmt, np.asarray(L), Hq, Hkv, D, P
        g = np.random.default_rng(seed)
        B = len(L)
        n = np.maximum(-(-self.L // P), 1)
        self.pool = pool or int(n.sum() * 1.3) + 2
        ids = np.arange(self.pool - n.sum(), self.pool) if at_end else g.permutation(self.pool)[:n.sum()]
        self.idx, self.ptr = g.permutation(ids).astype(np.int32), (np.cumsum(n) - n).astype(np.int32)
        self.max_pages = int(n.max())
        self.geo = vx.Geometry(B, Hq, Hkv, D, D, P, False, self.pool)
        self.table = vx.PageTable(dev(self.ptr), dev(self.idx), dev(self.L), self.max_pages)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.rng = g

    def blank(self):
        bad = 0x7F
        self.k = np.full((self.pool, self.Hkv, self.P, self.D), bad, np.uint8)
        self.v = self.k.copy()
        self.ks = np.full((self.pool, self.Hkv), np.nan, np.float32)
        self.vs = self.ks.copy()
        return self

    def fill(self):
        self.blank()
        for b, n in enumerate(self.L):
            for t0 in range(0, int(n), self.P):
                p, m = self.idx[self.ptr[b] + t0 // self.P], min(self.P, int(n) - t0)
                for c, s in ((self.k, self.ks), (self.v, self.vs)):
                    x = self.rng.standard_normal((self.Hkv, m, self.D)) * (32 if self.fmt == "int8" else 100)
                    c[p, :, :m] = ref.nearest(x, self.fmt)
                    s[p] = 2.0 ** self.rng.integers(-7, -4, self.Hkv) * self.rng.uniform(0.6, 1.4, self.Hkv)
        return self

    def cache(self):
        t = ref.DTYPE[self.fmt]
        return vx.QuantCache(dev(self.k, torch.uint8).view(t), dev(self.v, torch.uint8).view(t),
                             dev(self.ks, torch.float32), dev(self.vs, torch.float32))

    def float_values(self):
        return [ref.values(c, self.fmt) * s.astype(np.float64)[:, :, None, None]
                for c, s in ((self.k, self.ks), (self.v, self.vs))]

    def queries(self, std=1.0):
        return (torch.from_numpy(self.rng.standard_normal((len(self.L), self.Hq, self.D))) * std).to(torch.bfloat16)

    def select(self, k, empty=()):
        sel = np.full((len(self.L), self.Hkv, k), -1, np.int32)
        for b, n in enumerate(self.L):
            m = -(-int(n) // self.P)
            for h in range(self.Hkv):
                if (b, h) not in empty:
                    pick = np.sort(self.rng.permutation(m)[:k])
                    sel[b, h, :len(pick)] = pick
        return sel


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def decode(c, cache, q, sel, num_splits=0, sm_scale=0.0, ws=None, stream=None):
    k = sel.shape[2]
    out = torch.full((len(c.L), c.Hq, c.D), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((len(c.L), c.Hq), float("nan"), dtype=torch.float32, device=DEV)
    if ws is None:
        ws = torch.empty(vx.vx_workspace_size(c.geo, c.max_pages, k, num_splits), dtype=torch.uint8, device=DEV)
    vx.vx_sparse_decode_quant(c.geo, c.table, q, cache, sel, k, out, ws, lse=lse, sm_scale=sm_scale,
                              num_splits=num_splits, err=c.err, stream=stream)
    return out, lse


def check_attention(out, lse, want):
    """Bounds, per output element, against 64 bits:
      * logits: a sum of D products in fp32, at most D / 16 + 4 roundings or truncations of partial sums no larger than
        sum |q_d k_d| (2^-23 each), three products with fp32 scales (2^-24 each), and the difference to the running
        maximum (2^-24 of the largest logit, in base 2): `dx`;
      * weights: exp2 is good to 2^-21, so one is off by dx + 2^-20 relative; P is rounded to fp16 (half a step is 2^-11
        of it, and under the normal range, here 2^-29 of the largest weight, 2^-25 * 2^-15 absolute), each output by the
        sum of |weight * value| (of |value|) times that; the merge adds 2^-20;
      * out is rounded to bf16: half a step is 2^-8 of it."""
    o, l, mass, dot, big, total = want
    D = o.shape[-1]
    dx = (D / 16 + 4) * 2.0 ** -23 * dot + 2.0 ** -22 * (big + dot)
    seen = np.isfinite(l)
    got_l, got_o = lse.double().cpu().numpy(), out.double().cpu().numpy()
    assert np.array_equal(np.isfinite(got_l), seen) and (got_l[~seen] == -np.inf).all()
    assert (got_o[~seen] == 0).all()
    e = np.abs(got_l - np.where(seen, l, 0))[seen]
    assert (e <= (dx + 2.0 ** -20 * (1 + np.abs(np.where(seen, l, 0))))[seen]).all(), e.max()
    bound = mass * (2.0 ** -11 + 2.0 ** -18 + 2 * dx[..., None] + 2.0 ** -20) + 2.0 ** -8 * np.abs(o)
    bound += 2.0 ** -40 * total + 1e-37
    e = np.abs(got_o - o)
    assert (e <= bound).all(), (e / bound).max()


SHAPES = [
    # L, Hq, Hkv, D, P, k, empty rows: one token, odd lengths, whole pages, k above the pages, groups of 1, 2, 5, 9, 16
    ([1], 1, 1, 64, 16, 1, ()),
    ([1024], 4, 1, 64, 16, 8, ()),
    ([37, 16, 1, 700], 16, 8, 128, 16, 12, ((1, 3),)),
    ([129, 64, 63], 9, 1, 128, 64, 4, ()),
    ([300, 33, 31, 32, 5], 20, 4, 128, 32, 5, ((0, 0), (4, 3))),
    ([1000, 20], 32, 2, 64, 32, 40, ()),
    ([777], 16, 16, 64, 64, 3, ()),
    ([2048, 1500], 36, 4, 64, 64, 17, ((1, 0), (1, 1), (1, 2), (1, 3))),
    ([4000, 15], 32, 2, 128, 16, 250, ()),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_decode_matches_64_bits(fmt, shape):
    L, Hq, Hkv, D, P, k, empty = SHAPES[shape]
    c = Case(fmt, L, Hq, Hkv, D, P, seed=shape).fill()
    q, sel = c.queries(), c.select(k, empty)
    want = ref.attend(q.double().numpy(), *c.float_values(), c.ptr, c.idx, c.L, sel, 1 / np.sqrt(D))
    cache = c.cache()
    for splits in (0, 1, 3, 100000):
        out, lse = decode(c, cache, q.to(DEV), dev(sel), num_splits=splits)
        check_attention(out, lse, want)
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_query_range_and_scale(fmt):
    """bf16 queries far outside fp16's range, tiny ones, zeros, a scale argument, scales over many powers of two."""
    c = Case(fmt, [90, 45, 64], 4, 2, 128, 16, seed=5).fill()
    c.ks[:] = np.where(np.isnan(c.ks), c.ks, 2.0 ** c.rng.integers(-60, -20, c.ks.shape))
    c.vs[:] = np.where(np.isnan(c.vs), c.vs, 2.0 ** c.rng.integers(-4, 5, c.vs.shape))
    q = c.queries()
    q[0] *= 2.0 ** 60
    q[1] *= 2.0 ** -100
    q[2, :2] = 0
    # keep the logits of the large queries moderate: their pages have small scales
    for j in range(6):
        c.ks[c.idx[c.ptr[0] + j]] = 2.0 ** -64
    sel = c.select(6)
    want = ref.attend(q.double().numpy(), *c.float_values(), c.ptr, c.idx, c.L, sel, 0.25)
    out, lse = decode(c, c.cache(), q.to(DEV), dev(sel), sm_scale=0.25)
    check_attention(out, lse, want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("exponent", [-110, 112])
def test_decode_values_near_the_ends_of_the_range(fmt, exponent):
    """Value scales that put the output near fp32's largest and smallest normal numbers; short and long rows."""
    c = Case(fmt, [90, 7, 1500], 4, 2, 64, 16, seed=8).fill()
    c.vs[:] = np.where(np.isnan(c.vs), c.vs, 2.0 ** exponent)
    q, sel = c.queries(), c.select(94)
    want = ref.attend(q.double().numpy(), *c.float_values(), c.ptr, c.idx, c.L, sel, 1 / 8)
    cache = c.cache()
    for splits in (0, 5):
        out, lse = decode(c, cache, q.to(DEV), dev(sel), num_splits=splits)
        check_attention(out, lse, want)
    out, lse = decode(c, cache, q.to(DEV), dev(sel[:, :, :6]))
    check_attention(out, lse, ref.attend(q.double().numpy(), *c.float_values(), c.ptr, c.idx, c.L, sel[:, :, :6], 1 / 8))


def test_decode_late_pieces():
    """A share of 64 tiles or more per warp takes the split with late pieces: all of them equal one by one splits."""
    c = Case("e4m3", [32768] * 40, 8, 4, 64, 64, seed=2, pool=64)
    # every row names the same 64 pages, 8 times over
    c.idx = np.tile(np.arange(64, dtype=np.int32), 8 * 40)
    c.ptr = (np.arange(40) * 512).astype(np.int32)
    c.table = vx.PageTable(dev(c.ptr), dev(c.idx), dev(c.L), 512)
    c.blank()
    for a, s in ((c.k, c.ks), (c.v, c.vs)):
        a[:] = ref.nearest(c.rng.standard_normal(a.shape) * 100, "e4m3")
        s[:] = 2.0 ** c.rng.integers(-8, -5, s.shape)
    c.max_pages = 512
    k = 512
    sel = np.broadcast_to(np.arange(512, dtype=np.int32), (40, 4, 512))
    q = c.queries()
    assert vx.vx_planned_splits(c.geo, 512, k) > 148 * 8
    want = ref.attend(q[:3].double().numpy(), *c.float_values(), c.ptr, c.idx, c.L[:3], sel[:3], 1 / 8)
    cache, d_sel = c.cache(), dev(sel)
    out, lse = decode(c, cache, q.to(DEV), d_sel)
    check_attention(out[:3], lse[:3], want)
    again, lse2 = decode(c, cache, q.to(DEV), d_sel)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    # the same from a graph, with the counter reset inside
    ws = torch.empty(vx.vx_workspace_size(c.geo, c.max_pages, k), dtype=torch.uint8, device=DEV)
    d_q, graph = q.to(DEV), torch.cuda.CUDAGraph()
    out3, lse3 = torch.zeros_like(out), torch.zeros_like(lse)
    with torch.cuda.graph(graph):
        vx.vx_sparse_decode_quant(c.geo, c.table, d_q, cache, d_sel, k, out3, ws, lse=lse3)
    for _ in range(3):
        ws.random_(0, 256)
        out3.zero_()
        graph.replay()
        assert torch.equal(out, out3) and torch.equal(lse, lse3)


def test_decode_bad_entries_are_reported_and_skipped():
    c = Case("int8", [100, 60], 4, 2, 64, 16, seed=9).fill()
    q, sel = c.queries(), c.select(4)
    keep = sel.copy()
    sel[0, 0, 3] = 7      # past the request's 7 pages
    keep[0, 0, 3] = -1
    want = ref.attend(q.double().numpy(), *c.float_values(), c.ptr, c.idx, c.L, keep, 1 / 8)
    out, lse = decode(c, c.cache(), q.to(DEV), dev(sel))
    check_attention(out, lse, want)
    assert int(c.err.item()) == vx.VX_DATA_BAD_SELECTION
    c.err.zero_()
    good = c.idx.copy()
    j = keep[1, 1, 0]
    c.table.page_indices[int(c.ptr[1] + j)] = c.pool
    out, lse = decode(c, c.cache(), q.to(DEV), dev(keep))
    keep2 = keep.copy()
    keep2[1][keep2[1] == j] = -1
    want = ref.attend(q.double().numpy(), *c.float_values(), c.ptr, good, c.L, keep2, 1 / 8)
    check_attention(out, lse, want)
    assert int(c.err.item()) == vx.VX_DATA_BAD_PAGE_ID


def test_decode_far_pages():
    """Pages whose bytes lie past 2^32 from the pool's start."""
    pool = 270000  # 270000 x 8 x 16 x 128 bytes = 4.4 GB each for K and V
    c = Case("int8", [200, 77], 8, 8, 128, 16, seed=3, pool=pool, at_end=True)
    g = torch.Generator(DEV).manual_seed(1)
    shape = (pool, 8, 16, 128)
    k = torch.zeros(shape, dtype=torch.int8, device=DEV)
    v = torch.zeros(shape, dtype=torch.int8, device=DEV)
    first = pool - 64
    k[first:] = torch.randint(-127, 128, (64, 8, 16, 128), generator=g, device=DEV).to(torch.int8)
    v[first:] = torch.randint(-127, 128, (64, 8, 16, 128), generator=g, device=DEV).to(torch.int8)
    s = torch.full((pool, 8), 2.0 ** -6, device=DEV)
    cache = vx.QuantCache(k, v, s, s.clone())
    q, sel = c.queries(), c.select(13)
    tail = [a[first:].cpu().numpy().astype(np.float64) * 2.0 ** -6 for a in (k, v)]
    want = ref.attend(q.double().numpy(), *tail, c.ptr, c.idx - first, c.L, sel, 1 / np.sqrt(128))
    out, lse = decode(c, cache, q.to(DEV), dev(sel))
    check_attention(out, lse, want)
    # and written there
    cen = torch.zeros(pool, 8, 128, dtype=torch.bfloat16, device=DEV)
    x = torch.randn(2, 8, 128, generator=g, device=DEV).to(torch.bfloat16)
    vx.vx_quant_update(c.geo, c.table, cache, cen, x, x, err=c.err)
    got = c.idx[c.ptr + (c.L - 1) // 16]
    for b in range(2):
        codes = k[int(got[b]), :, int((c.L[b] - 1) % 16)].double() * s[int(got[b])].double()[:, None]
        half = s[int(got[b])].double()[:, None] / 2
        assert ((codes - x[b].double()).abs() <= half).all()
    assert int(c.err.item()) == 0


# ------------------------------------------------------------------------------------------------ writing

WRITES = [
    # L, first positions, Hkv, D, P
    ([1, 37, 640, 300, 33, 1000], [0, 5, 320, 299, 33, 17], 8, 128, 16),
    ([200, 64, 129, 400], [130, 0, 128, 100], 4, 64, 64),
    ([95, 32, 31, 64], [3, 31, 0, 32], 2, 128, 32),
    ([100, 65], [70, 64], 1, 128, 64),
    ([50, 17, 16], [0, 16, 15], 16, 64, 16),
    ([70], [33], 2, 64, 32),
]


def new_rows(c, n, spread=3):
    """Rows over several powers of two, so that a page's scale grows."""
    x = c.rng.standard_normal((n, c.Hkv, c.D)) * 2.0 ** c.rng.integers(-spread, spread + 1, (n, c.Hkv, 1))
    return torch.from_numpy(x).to(torch.bfloat16)


def check_cache(c, cache, cen, want_cen):
    assert np.array_equal(cache.k_cache.view(torch.uint8).cpu().numpy(), c.k)
    assert np.array_equal(cache.v_cache.view(torch.uint8).cpu().numpy(), c.v)
    assert np.array_equal(cache.k_scale.cpu().numpy(), c.ks, equal_nan=True)
    assert np.array_equal(cache.v_scale.cpu().numpy(), c.vs, equal_nan=True)
    assert np.array_equal(cen.double().cpu().numpy(), want_cen)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", range(len(WRITES)))
def test_prefill_write_bit_for_bit(fmt, case):
    L, first, Hkv, D, P = WRITES[case]
    c = Case(fmt, L, Hkv, Hkv, D, P, seed=case).fill()
    # pages that are partly filled already hold another program's scales (any fp32 number) or powers of two
    if case % 2:
        for s in (c.ks, c.vs):
            s[:] = 2.0 ** np.rint(np.log2(s))
    n = int((np.array(L) - np.array(first)).sum())
    kn, vn = new_rows(c, n), new_rows(c, n)
    cache = c.cache()
    cen = torch.zeros(c.pool, Hkv, D, dtype=torch.bfloat16, device=DEV)
    want = np.zeros((c.pool, Hkv, D))
    vx.vx_quant_update(c.geo, c.table, cache, cen, kn.to(DEV), vn.to(DEV), first_pos=dev(np.array(first)), err=c.err)
    assert int(c.err.item()) == 0
    if case % 2 == 0:
        # scales that are no powers of two: the products are rounded in fp32, so a code may land on the other side of a
        # tie; compare values within half a step plus 2^-22 of the code
        for got, scale, x in ((cache.k_cache, cache.k_scale, kn), (cache.v_cache, cache.v_scale, vn)):
            check_half_step(c, got, scale, x, first)
        return
    ref.quant_update(c.k, c.ks, want, kn.double().numpy(), c.ptr, c.idx, c.L, first, fmt)
    ref.quant_update(c.v, c.vs, None, vn.double().numpy(), c.ptr, c.idx, c.L, first, fmt)
    check_cache(c, cache, cen, want)


def check_half_step(c, codes, scale, x, first):
    raw, s, row = codes.view(torch.uint8).cpu().numpy(), scale.cpu().numpy().astype(np.float64), 0
    for b in range(len(c.L)):
        for t in range(first[b], int(c.L[b])):
            p = c.idx[c.ptr[b] + t // c.P]
            y = x[row].double().numpy() / s[p][:, None]
            got = ref.values(raw[p, :, t % c.P], c.fmt)
            _, e = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))
            step = np.ones_like(y) if c.fmt == "int8" else 2.0 ** (e - 4)
            assert (np.abs(y) <= ref.QMAX[c.fmt]).all()
            assert (np.abs(got - y) <= step / 2 + np.abs(y) * 2.0 ** -22).all()
            row += 1


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("P,D,Hkv", [(16, 128, 8), (32, 64, 1), (64, 128, 2), (64, 64, 4), (32, 128, 16)])
def test_appends_equal_the_plain_ones(fmt, P, D, Hkv):
    """Tokens one by one from empty rows: pages started, grown, filled; each step against the plain write."""
    B, steps = 3, P + 5
    c = Case(fmt, [steps + 2 * b for b in range(B)], Hkv, Hkv, D, P, seed=P + D).blank()
    start = np.array([2 * b for b in range(B)])
    cache, cen = c.cache(), torch.zeros(c.pool, Hkv, D, dtype=torch.bfloat16, device=DEV)
    want = np.zeros((c.pool, Hkv, D))
    if start.sum():
        kn, vn = new_rows(c, int(start.sum())), new_rows(c, int(start.sum()))
        lens = np.maximum(start, 1)
        first = np.where(start > 0, 0, 1)
        t = vx.PageTable(c.table.page_ptr, c.table.page_indices, dev(lens), c.max_pages)
        vx.vx_quant_update(c.geo, t, cache, cen, kn.to(DEV), vn.to(DEV), first_pos=dev(first), err=c.err)
        ref.quant_update(c.k, c.ks, want, kn.double().numpy(), c.ptr, c.idx, lens, first, fmt)
        ref.quant_update(c.v, c.vs, None, vn.double().numpy(), c.ptr, c.idx, lens, first, fmt)
    for step in range(steps):
        lens = start + step + 1
        kn, vn = new_rows(c, B, 6), new_rows(c, B, 6)
        t = vx.PageTable(c.table.page_ptr, c.table.page_indices, dev(lens), c.max_pages)
        vx.vx_quant_update(c.geo, t, cache, cen, kn.to(DEV), vn.to(DEV), err=c.err)
        ref.quant_update(c.k, c.ks, want, kn.double().numpy(), c.ptr, c.idx, lens, lens - 1, fmt)
        ref.quant_update(c.v, c.vs, None, vn.double().numpy(), c.ptr, c.idx, lens, lens - 1, fmt)
    check_cache(c, cache, cen, want)
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("P", [16, 64])
def test_write_of_zeros_tiny_huge_and_non_finite_values(fmt, P):
    D, Hkv = 64, 2
    c = Case(fmt, [P, P + 3, 2 * P, 5], Hkv, Hkv, D, P, seed=11).blank()
    n = int(c.L.sum())
    x = torch.randn(n, Hkv, D, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    x[:P] = 0                                       # a page of zeros
    x[2 * P:2 * P + 3] *= 2.0 ** -130               # a page of subnormal numbers
    x[2 * P + 3:2 * P + 9] *= 2.0 ** 120            # near the largest numbers
    x[2 * P + 10, 0, 5] = float("inf")
    x[2 * P + 10, 1, 6] = float("-inf")
    x[2 * P + 11, 0, 7] = float("nan")
    x[n - 1, 1, 0] = -0.0
    qmax = 127 if fmt == "int8" else 448
    x[n - 5:, 0, 0] = torch.tensor([qmax, qmax * 2, qmax / 2, -qmax, qmax * 2]).to(torch.bfloat16)
    first = np.zeros(4, int)
    cache, cen = c.cache(), torch.zeros(c.pool, Hkv, D, dtype=torch.bfloat16, device=DEV)
    want = np.zeros((c.pool, Hkv, D))
    vx.vx_quant_update(c.geo, c.table, cache, cen, x.to(DEV), x.to(DEV), first_pos=dev(first), err=c.err)
    ref.quant_update(c.k, c.ks, want, x.double().numpy(), c.ptr, c.idx, c.L, first, fmt)
    ref.quant_update(c.v, c.vs, None, x.double().numpy(), c.ptr, c.idx, c.L, first, fmt)
    check_cache(c, cache, cen, want)
    assert int(c.err.item()) == vx.VX_DATA_BAD_VALUE


def test_write_bad_rows_are_reported_and_skipped():
    c = Case("int8", [40, 20, 30], 2, 2, 64, 16, seed=1).blank()
    cache, cen = c.cache(), torch.zeros(c.pool, 2, 64, dtype=torch.bfloat16, device=DEV)
    want = np.zeros((c.pool, 2, 64))
    first = np.array([0, 21, 0])  # request 1: past its length, so it brings no rows
    c.table.page_indices[int(c.ptr[2])] = -1  # request 2's first page
    x = new_rows(c, 70)
    vx.vx_quant_update(c.geo, c.table, cache, cen, x.to(DEV), x.to(DEV), first_pos=dev(first), err=c.err)
    assert int(c.err.item()) == vx.VX_DATA_BAD_SEQ_LEN | vx.VX_DATA_BAD_PAGE_ID
    keep = (c.k.copy(), c.v.copy(), c.ks.copy(), c.vs.copy())
    for a, s, w in ((c.k, c.ks, want), (c.v, c.vs, None)):
        ref.quant_update(a, s, w, x.double().numpy(), c.ptr, c.idx, c.L, [0, 20, 0], "int8")
    p = c.idx[c.ptr[2]]
    for a, old in zip((c.k, c.v, c.ks, c.vs), keep):
        a[p] = old[p]
    want[p] = 0
    check_cache(c, cache, cen, want)


@pytest.mark.parametrize("fmt,P", [("int8", 16), ("e4m3", 64), ("int8", 32)])
def test_prefill_of_many_requests(fmt, P):
    """More requests than a block has threads: chunks of every size, empty ones, some starting inside a page, and two
    requests that are refused."""
    B, rng = 600, np.random.default_rng(P)
    L = rng.integers(1, 3 * P, B)
    first = np.minimum(rng.integers(0, 3 * P, B), L)
    first[::7] = L[::7]
    c = Case(fmt, L, 1, 1, 64, P, seed=P).fill()
    for s in (c.ks, c.vs):
        s[:] = 2.0 ** np.rint(np.log2(s))
    wrong = first.copy()
    wrong[5], wrong[400] = L[5] + 1, -1
    first[5], first[400] = L[5], L[400]  # their rows are not in the input
    n = int((L - first).sum())
    kn, vn = new_rows(c, n), new_rows(c, n)
    cache, cen = c.cache(), torch.zeros(c.pool, 1, 64, dtype=torch.bfloat16, device=DEV)
    want = np.zeros((c.pool, 1, 64))
    vx.vx_quant_update(c.geo, c.table, cache, cen, kn.to(DEV), vn.to(DEV), first_pos=dev(wrong), err=c.err)
    ref.quant_update(c.k, c.ks, want, kn.double().numpy(), c.ptr, c.idx, L, first, fmt)
    ref.quant_update(c.v, c.vs, None, vn.double().numpy(), c.ptr, c.idx, L, first, fmt)
    check_cache(c, cache, cen, want)
    assert int(c.err.item()) == vx.VX_DATA_BAD_SEQ_LEN


def test_largest_batch():
    """4,096 requests: append, prefill and attention."""
    B, P, rng = 4096, 16, np.random.default_rng(1)
    c = Case("int8", rng.integers(2, 40, B), 2, 1, 64, P, seed=9).blank()
    cache, cen = c.cache(), torch.zeros(c.pool, 1, 64, dtype=torch.bfloat16, device=DEV)
    want = np.zeros((c.pool, 1, 64))
    for lo, hi in ((np.zeros(B, int), c.L - 1), (c.L - 1, c.L)):
        t = vx.PageTable(c.table.page_ptr, c.table.page_indices, dev(hi), c.max_pages)
        kn, vn = new_rows(c, int((hi - lo).sum())), new_rows(c, int((hi - lo).sum()))
        vx.vx_quant_update(c.geo, t, cache, cen, kn.to(DEV), vn.to(DEV), first_pos=dev(lo) if lo[0] == 0 else None,
                           err=c.err)
        ref.quant_update(c.k, c.ks, want, kn.double().numpy(), c.ptr, c.idx, hi, lo, "int8")
        ref.quant_update(c.v, c.vs, None, vn.double().numpy(), c.ptr, c.idx, hi, lo, "int8")
    check_cache(c, cache, cen, want)
    q, sel = c.queries(), c.select(3)
    out, lse = decode(c, cache, q.to(DEV), dev(sel))
    check_attention(out, lse, ref.attend(q.double().numpy(), *c.float_values(), c.ptr, c.idx, c.L, sel, 1 / 8))
    assert int(c.err.item()) == 0


def test_two_streams_at_once():
    """The same cache read by two calls that run side by side, each with its own workspace and outputs."""
    c = Case("e4m3", [3000, 500, 77], 16, 8, 128, 16, seed=41).fill()
    sel, cache = c.select(60), c.cache()
    d_sel = dev(sel)
    qs = [c.queries() for _ in range(2)]
    d_qs = [q.to(DEV) for q in qs]
    ws = [torch.empty(vx.vx_workspace_size(c.geo, c.max_pages, 60), dtype=torch.uint8, device=DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = decode(c, cache, d_qs[i], d_sel, ws=ws[i])
    torch.cuda.synchronize()
    for q, (out, lse) in zip(qs, got):
        check_attention(out, lse, ref.attend(q.double().numpy(), *c.float_values(), c.ptr, c.idx, c.L, sel,
                                             1 / np.sqrt(128)))


def test_prefill_rows_past_the_input_are_refused():
    """Fewer new rows than the table says: the requests that would read past them write nothing."""
    c = Case("int8", [20, 30, 5], 2, 2, 64, 16, seed=1).blank()
    cache, cen = c.cache(), torch.zeros(c.pool, 2, 64, dtype=torch.bfloat16, device=DEV)
    want = np.zeros((c.pool, 2, 64))
    x = new_rows(c, 49)
    vx.vx_quant_update(c.geo, c.table, cache, cen, x.to(DEV), x.to(DEV), first_pos=dev(np.zeros(3)), err=c.err)
    assert int(c.err.item()) == vx.VX_DATA_BAD_SEQ_LEN
    for a, s, w in ((c.k, c.ks, want), (c.v, c.vs, None)):
        ref.quant_update(a, s, w, x.double().numpy(), c.ptr, c.idx, [20], [0], "int8")
    check_cache(c, cache, cen, want)


# ------------------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt", FMTS)
def test_decode_loop_of_write_score_select_attend(fmt):
    """A prompt written, then appending steps: selections are those of the step's own scores over the stored centroids,
    outputs those of 64-bit attention over the stored codes; the chained call equals the separate ones bit for bit."""
    from oracle import topk_exact
    B, Hq, Hkv, D, P, k, steps = 4, 8, 4, 128, 16, 5, 20
    c = Case(fmt, [400, 33, 150, 16 + steps], Hq, Hkv, D, P, seed=21).blank()
    start = c.L - steps
    cache, cen = c.cache(), torch.zeros(c.pool, Hkv, D, dtype=torch.bfloat16, device=DEV)
    n = int(start.sum())
    kn, vn = new_rows(c, n, 1).to(DEV), new_rows(c, n, 1).to(DEV)
    t = vx.PageTable(c.table.page_ptr, c.table.page_indices, dev(start), c.max_pages)
    vx.vx_quant_update(c.geo, t, cache, cen, kn, vn, first_pos=dev(np.zeros(B)), err=c.err)
    ws = torch.empty(vx.vx_workspace_size(c.geo, c.max_pages, k), dtype=torch.uint8, device=DEV)
    for step in range(steps):
        lens = start + step + 1
        t = vx.PageTable(c.table.page_ptr, c.table.page_indices, dev(lens), c.max_pages)
        kn, vn, q = new_rows(c, B, 1).to(DEV), new_rows(c, B, 1).to(DEV), c.queries().to(DEV)
        out, out2 = (torch.full((B, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        lse, lse2 = (torch.full((B, Hq), float("nan"), device=DEV) for _ in range(2))
        sc = torch.full((B, Hkv, c.max_pages), float("nan"), device=DEV)
        sel = torch.full((B, Hkv, k), -7, dtype=torch.int32, device=DEV)
        vx.vx_block_topk_decode_append_quant(c.geo, t, q, cache, cen, kn, vn, k, out, ws, lse=lse, scores_out=sc,
                                             sel_out=sel, err=c.err)
        # the steps one by one on the written cache
        sc2, sel2 = torch.full_like(sc, float("nan")), torch.full_like(sel, -7)
        vx.vx_score_pages(c.geo, t, q, cen, sc2)
        vx.vx_topk_pages(c.geo, t, sc2, k, sel2)
        vx.vx_sparse_decode_quant(c.geo, t, q, cache, sel2, k, out2, ws, lse=lse2)
        assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(sel, sel2)
        assert torch.equal(sc.nan_to_num(7), sc2.nan_to_num(7))
        vx.vx_block_topk_decode_quant(c.geo, t, q, cache, cen, k, out2.zero_(), ws, lse=lse2.zero_())
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        c.k, c.v = (x.view(torch.uint8).cpu().numpy() for x in (cache.k_cache, cache.v_cache))
        c.ks, c.vs = cache.k_scale.cpu().numpy(), cache.v_scale.cpu().numpy()
        want = ref.attend(q.double().cpu().numpy(), *c.float_values(), c.ptr, c.idx, lens, sel.cpu().numpy(),
                          1 / np.sqrt(D))
        check_attention(out, lse, want)
        assert np.array_equal(sel.cpu().numpy(), topk_exact(sc.cpu().numpy(), lens, P, k))
    assert int(c.err.item()) == 0


def test_captured_and_replayed_on_another_stream():
    c = Case("e4m3", [300, 80], 8, 4, 128, 16, seed=31).fill()
    sel, q = c.select(9), c.queries().to(DEV)
    cache, d_sel = c.cache(), dev(sel)
    ws = torch.empty(vx.vx_workspace_size(c.geo, c.max_pages, 9), dtype=torch.uint8, device=DEV)
    out = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    vx.vx_sparse_decode_quant(c.geo, c.table, q, cache, d_sel, 9, out, ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        vx.vx_sparse_decode_quant(c.geo, c.table, q, cache, d_sel, 9, out, ws)
    for seed in range(3):
        q.copy_(c.queries())
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        want = ref.attend(q.double().cpu().numpy(), *c.float_values(), c.ptr, c.idx, c.L, sel, 1 / np.sqrt(128))
        lse = torch.from_numpy(want[1])
        check_attention(out, lse, want)
    # a call with a stream argument runs there
    with torch.cuda.stream(side):
        torch.cuda._sleep(1000000)
        q.copy_(c.queries().to(DEV))
    vx.vx_sparse_decode_quant(c.geo, c.table, q, cache, d_sel, 9, out, ws, stream=side)
    side.synchronize()
    want = ref.attend(q.double().cpu().numpy(), *c.float_values(), c.ptr, c.idx, c.L, sel, 1 / np.sqrt(128))
    check_attention(out, torch.from_numpy(want[1]), want)
