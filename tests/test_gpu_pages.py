"""Page calls on the GPU against plain implementations: copy, new rows of a table (fork, free, grow), compaction.  Page data,
tables and reference counts are compared whole."""
import numpy as np
import pytest
import torch

import quant_ref as ref
from paged_block_sparse_kv_b200 import vx

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = ("k_cache", "v_cache", "centroids", "k_scale", "v_scale")


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


class Pool:
    """A pool of `kind` with random contents, on the device and (as raw bytes) on the host."""

    def __init__(self, kind, pages, Hkv=2, D=64, P=16, batch=1, seed=0, extras=True):
        mla = kind == "mla"
        if mla:
            Hkv, D = 1, 576
        self.P, self.geo = P, vx.Geometry(batch, Hkv, Hkv, D, 512 if mla else D, P, mla, pages)
        g = torch.Generator(DEV).manual_seed(seed)

        def draw(shape, dtype):
            n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
            return torch.randint(0, 256, (n,), dtype=torch.uint8, generator=g, device=DEV).view(dtype).view(shape)

        t = {"bf16": torch.bfloat16, "mla": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[kind]
        quant = kind in ("int8", "e4m3")
        self.t = dict(k_cache=draw((pages, Hkv, P, D), t), v_cache=None if mla else draw((pages, Hkv, P, D), t),
                      centroids=draw((pages, Hkv, D), torch.bfloat16) if extras else None,
                      k_scale=draw((pages, Hkv), torch.float32) if quant and extras else None,
                      v_scale=draw((pages, Hkv), torch.float32) if quant and extras else None)
        self.vx = vx.PagePool(**self.t)
        self.host = self.read()

    def read(self):
        return [x.view(torch.uint8).cpu().numpy() for x in (self.t[n] for n in NAMES) if x is not None]

    def check(self):
        for got, want in zip(self.read(), self.host):
            assert np.array_equal(got, want)


def workspace(geo, rows=1):
    return torch.randint(0, 256, (vx.vx_page_workspace_size(geo, rows),), dtype=torch.uint8, device=DEV)


def err_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


KINDS = ["bf16", "int8", "e4m3", "mla"]
SHAPES = {"bf16": dict(Hkv=8, D=128, P=16), "int8": dict(Hkv=1, D=64, P=16), "e4m3": dict(Hkv=4, D=128, P=64),
          "mla": dict(P=64)}


# ------------------------------------------------------------------------------------------------ copy

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [0, 1, 7, 150])
@pytest.mark.parametrize("same", [True, False])
def test_copy(kind, n, same):
    rng = np.random.default_rng(n)
    dst = Pool(kind, 301, seed=1, **SHAPES[kind])
    src = dst if same else Pool(kind, 211, seed=2, **SHAPES[kind])
    ids = rng.permutation(301)
    s, d = (ids[:n], ids[n:2 * n]) if same else (rng.integers(0, 211, n), ids[:n])  # a source may repeat
    err = err_word()
    vx.vx_copy_pages(dst.geo, src.vx, dst.vx, dev(s), dev(d), workspace(dst.geo), err=err)
    for a, b in zip(dst.host, src.host):
        a[d] = b[s]
    dst.check()
    src.check()
    assert int(err.item()) == 0


def test_copy_without_centroids_and_scales():
    dst, src = Pool("int8", 20, extras=False), Pool("int8", 20, seed=3, extras=False)
    vx.vx_copy_pages(dst.geo, src.vx, dst.vx, dev([4, 5]), dev([19, 0]), workspace(dst.geo))
    for a, b in zip(dst.host, src.host):
        a[[19, 0]] = b[[4, 5]]
    dst.check()


def test_copy_refuses_ambiguous_pairs():
    """The first of two copies to one page is made, a copy onto a source is not, bad ids are not."""
    p = Pool("bf16", 40)
    err = err_word()
    s = [1, 2, 3, 4, 5, 6, 40, 7, -1, 8]
    d = [11, 12, 11, 13, 5, 2, 14, 40, 15, -1]  # copy 2: again to 11; 4: onto itself; 5: onto a source; bad ids
    vx.vx_copy_pages(p.geo, p.vx, p.vx, dev(s), dev(d), workspace(p.geo), err=err)
    for a in p.host:
        a[11], a[12], a[13] = a[1], a[2], a[4]
    p.check()
    assert int(err.item()) == vx.VX_DATA_BAD_COPY | vx.VX_DATA_BAD_PAGE_ID
    # between two pools a page may be a source in one and a destination in the other
    q = Pool("bf16", 40, seed=5)
    err.zero_()
    vx.vx_copy_pages(p.geo, q.vx, p.vx, dev([1, 2]), dev([2, 1]), workspace(p.geo), err=err)
    for a, b in zip(p.host, q.host):
        a[2], a[1] = b[1], b[2]
    p.check()
    assert int(err.item()) == 0


@pytest.mark.parametrize("n", [300, 513, 900])
@pytest.mark.parametrize("same", [True, False])
def test_copy_random_pairs(n, same):
    """Pairs with repeated destinations, sources that are destinations and bad ids, fewer and more than a block checks
    by itself."""
    rng = np.random.default_rng(n)
    pages = 800
    dst = Pool("int8", pages, Hkv=1, D=64, P=16, seed=1)
    src = dst if same else Pool("int8", pages, Hkv=1, D=64, P=16, seed=2)
    s, d = rng.integers(-2, pages // 2, n), rng.integers(pages // 4, pages + 2, n)
    err = err_word()
    vx.vx_copy_pages(dst.geo, src.vx, dst.vx, dev(s), dev(d), workspace(dst.geo), err=err)
    named, sources = set(), set(s.tolist()) if same else set()
    before = [a.copy() for a in src.host]
    for x, y in zip(s.tolist(), d.tolist()):
        if 0 <= y < pages and y not in named:
            if 0 <= x < pages and y not in sources:
                for a, b in zip(dst.host, before):
                    a[y] = b[x]
            named.add(y)
    dst.check()
    assert int(err.item()) == vx.VX_DATA_BAD_COPY | vx.VX_DATA_BAD_PAGE_ID


def test_copy_far_pages():
    """Pages whose bytes lie past 2^32 from the pool's start."""
    n = 70000  # x 8 x 32 x 128 x 2 bytes = 4.6 GB each for K and V
    geo = vx.Geometry(1, 8, 8, 128, 128, 32, False, n)
    k = torch.zeros(n, 8, 32, 128, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros(n, 8, 32, 128, dtype=torch.bfloat16, device=DEV)
    k[3], v[3] = 1.5, -2.5
    pool = vx.PagePool(k, v)
    vx.vx_copy_pages(geo, pool, pool, dev([3]), dev([n - 1]), workspace(geo))
    assert (k[n - 1] == 1.5).all() and (v[n - 1] == -2.5).all() and (k[n - 2] == 0).all()
    vx.vx_copy_pages(geo, pool, pool, dev([n - 1]), dev([0]), workspace(geo))
    assert (k[0] == 1.5).all() and (v[0] == -2.5).all()


# ------------------------------------------------------------------------------------------------ new rows

class Rows:
    """A page table over a pool, kept as plain lists too."""

    def __init__(self, kind, pages, lens, max_pages, seed=0, held=0, **shape):
        rng = np.random.default_rng(seed)
        self.pool = Pool(kind, pages, batch=len(lens), seed=seed, **{**SHAPES[kind], **shape})
        P = self.pool.P
        n = [-(-L // P) for L in lens]
        ids = rng.permutation(pages)
        cut = np.cumsum([0] + n)
        self.rows = [list(ids[a:b]) for a, b in zip(cut[:-1], cut[1:])]
        self.lens, self.max_pages = list(lens), max_pages
        self.ref = np.bincount(ids[:cut[-1]], minlength=pages)
        self.ref[ids[cut[-1]:cut[-1] + held]] += 1

    def flat(self, room=1):
        ptr = np.cumsum([0] + [len(r) + room for r in self.rows])
        idx = np.full(ptr[-1], 123456789)
        for p, r in zip(ptr, self.rows):
            idx[p:p + len(r)] = r
        return ptr[:-1], idx

    def update(self, parent, grow, in_place=False, room=2):
        """One call and its plain counterpart; returns the error word."""
        geo = self.pool.geo
        geo.batch = len(self.lens)
        ptr, idx = self.flat()
        table = vx.PageTable(dev(ptr), dev(idx), dev(self.lens), self.max_pages)
        host = [a.copy() for a in self.pool.host]
        want = ref.update_table(self.pool.P, ptr, idx, self.lens, self.ref, parent, grow, host,
                                self.max_pages)
        L2 = [max(0, (self.lens[p] if p >= 0 else 0) + g) for p, g in zip(parent, grow)]
        new_ptr = np.cumsum([0] + [-(-L // self.pool.P) + room for L in L2])
        new = vx.PageTable(dev(new_ptr[:-1]), torch.full((int(new_ptr[-1]),), -5, dtype=torch.int32, device=DEV),
                           torch.full((len(parent),), -5, dtype=torch.int32, device=DEV), self.max_pages)
        old_ref = dev(self.ref)
        new_ref = old_ref if in_place else torch.full_like(old_ref, -5)
        err = err_word()
        vx.vx_update_table(geo, self.pool.vx, table, old_ref, dev(parent), dev(grow), new, new_ref,
                           workspace(geo, len(parent)), err=err)
        got_idx, got_len = new.page_indices.cpu().numpy(), new.seq_lens.cpu().numpy()
        if want is None:
            assert (got_len == 0).all() and (got_idx == -5).all()
            assert np.array_equal(new_ref.cpu().numpy(), self.ref)
        else:
            rows, lens, ref2 = want
            assert list(got_len) == lens
            fill = np.full(len(got_idx), -5)
            for p, r in zip(new_ptr, rows):
                fill[p:p + len(r)] = r
            assert np.array_equal(got_idx, fill)
            assert np.array_equal(new_ref.cpu().numpy(), ref2)
            self.rows, self.lens, self.ref, self.pool.host = rows, lens, ref2, host
        self.pool.check()
        return int(err.item())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("in_place", [False, True])
def test_update_fork_free_grow(kind, in_place):
    P = SHAPES[kind]["P"]
    r = Rows(kind, 400, [1, P, P + 1, 5 * P, 7 * P + 3, 0, 30 * P - 1], 64, seed=1, held=20)
    assert r.update([0, 1, 2, 3, 4, 5, 6], [1] * 7, in_place) == 0           # a decode step
    assert r.update([4, 4, 2, 4, 6, 6, -1, 0], [1, 1, 1, 0, 1, 2 * P, 9, 0], in_place) == 0  # fork, free, create
    assert r.update([0, 1, 2, 3, 4, 5, 6, 7], [1] * 8, in_place) == 0
    assert r.update([7, 6, 5, 4, 3, 2, 1, 0], [0] * 8, in_place) == 0        # reorder alone
    assert r.update([0, 0, 0, 0], [1, 1, 1, 1], in_place) == 0               # everything else is freed
    assert r.update([-1], [0], in_place) == 0                                # and that too
    assert (r.ref > 0).sum() == 20


def test_update_shared_last_page_of_the_caller():
    """A last page that the caller also holds is copied even for the only child, and stays the caller's."""
    r = Rows("int8", 30, [20], 8, seed=2)
    r.ref[r.rows[0][-1]] += 1
    tail = r.rows[0][-1]
    assert r.update([0], [1]) == 0
    assert r.rows[0][-1] != tail and r.ref[tail] == 1


def test_update_random():
    rng = np.random.default_rng(7)
    r = Rows("int8", 700, list(rng.integers(0, 200, 9)), 40, seed=3, held=11)
    for step in range(40):
        n = int(rng.integers(1, 14))
        parent = rng.integers(-1, len(r.lens), n)
        grow = rng.integers(0, 30, n)
        err = r.update(list(parent), list(grow), in_place=bool(step % 2))
        assert err in (0, vx.VX_DATA_NO_PAGES, vx.VX_DATA_BAD_SEQ_LEN)  # out of pages, or of a row's bound of 40


@pytest.mark.parametrize("pages", [128, 129, 255, 40961, 300000])
def test_update_pool_sizes(pages):
    """Ranks over pools smaller and larger than the planner's spans, free pages at both ends."""
    r = Rows("int8", pages, [33, 16 * 60], 64 + pages // 64, seed=pages, held=pages // 3)
    assert r.update([0, 1, -1, 1], [1, 1, 16 * (pages // 64), 40]) == 0


def test_update_many_rows():
    r = Rows("int8", 9000, [17] * 1500, 8, seed=4)
    parent = np.random.default_rng(1).integers(-1, 1500, 4096)
    assert r.update(list(parent), [1] * 4096) == 0


def test_update_refusals_change_nothing():
    r = Rows("bf16", 12, [40, 33], 6, seed=5)  # 6 pages used, 6 free
    assert r.update([0, 1, -1], [8, 15, 6 * 16]) == 0  # every free page
    assert r.update([0, 1], [1, 0]) == vx.VX_DATA_NO_PAGES
    base = (list(r.lens), r.ref.copy())

    def refused(parent, grow, bit, **kw):
        geo, P = r.pool.geo, 16
        geo.batch = len(r.lens)
        ptr, idx = r.flat()
        lens = kw.get("lens", r.lens)
        if "tail" in kw:
            idx[ptr[0] + len(r.rows[0]) - 1] = kw["tail"]
        table = vx.PageTable(dev(ptr), dev(idx), dev(lens), 6)
        new = vx.PageTable(dev(kw.get("ptr", 8 * np.arange(len(parent)))), torch.full((64,), -5, dtype=torch.int32,
                           device=DEV), torch.full((len(parent),), -5, dtype=torch.int32, device=DEV), kw.get("top", 6))
        new_ref, err = torch.full((12,), -5, dtype=torch.int32, device=DEV), err_word()
        vx.vx_update_table(geo, r.pool.vx, table, dev(r.ref), dev(parent), dev(grow), new, new_ref, workspace(geo, 8),
                           err=err)
        assert int(err.item()) == bit
        assert (new.seq_lens == 0).all() and (new.page_indices == -5).all()
        assert np.array_equal(new_ref.cpu().numpy(), base[1])
        r.pool.check()

    refused([3], [0], vx.VX_DATA_BAD_ROW)
    refused([-2], [0], vx.VX_DATA_BAD_ROW)
    refused([0], [-1], vx.VX_DATA_BAD_SEQ_LEN)
    refused([0], [2 ** 31 - 1], vx.VX_DATA_BAD_SEQ_LEN)
    refused([2], [0], vx.VX_DATA_BAD_SEQ_LEN, top=5)
    refused([0], [0], vx.VX_DATA_BAD_SEQ_LEN, lens=[-1, 48, 96])
    refused([0], [0], vx.VX_DATA_BAD_SEQ_LEN, lens=[48, 97, 96])
    refused([0], [0], vx.VX_DATA_BAD_ROW, ptr=np.array([62]))
    refused([0], [0], vx.VX_DATA_BAD_ROW, ptr=np.array([-1]))
    refused([0], [0], vx.VX_DATA_BAD_PAGE_ID, lens=[47, 48, 96], tail=12)
    r.ref[r.rows[0][-1]] = 0  # a last page that its own row holds and the counts call free
    base = (base[0], r.ref.copy())
    refused([0], [0], vx.VX_DATA_BAD_PAGE_ID, lens=[47, 48, 96])


# ------------------------------------------------------------------------------------------------ compaction

def _compact(pool, rows, lens, refs, max_pages, in_place, expect=0):
    geo = pool.geo
    geo.batch = len(rows)
    ptr = np.cumsum([0] + [len(r) + 1 for r in rows])
    idx = np.full(ptr[-1], 55555)
    for p, r in zip(ptr, rows):
        idx[p:p + len(r)] = r
    table = vx.PageTable(dev(ptr[:-1]), dev(idx), dev(lens), max_pages)
    old_ref = dev(refs)
    new_ref = old_ref if in_place else torch.full_like(old_ref, -5)
    new_idx = table.page_indices if in_place else torch.full_like(table.page_indices, 55555)
    remap, live, err = torch.full_like(old_ref, -5), torch.zeros(1, dtype=torch.int32, device=DEV), err_word()
    vx.vx_compact_pages(geo, pool.vx, table, old_ref, new_idx, new_ref, remap, live, workspace(geo), err=err)
    want_map, want_ref, n = ref.compact(refs, pool.host)
    assert int(live.item()) == n
    assert np.array_equal(remap.cpu().numpy(), want_map)
    assert np.array_equal(new_ref.cpu().numpy(), want_ref)
    want_idx = idx.copy()
    for p, r in zip(ptr, rows):
        for j, page in enumerate(r):
            if 0 <= page < len(refs) and want_map[page] >= 0:
                want_idx[p + j] = want_map[page]
    assert np.array_equal(new_idx.cpu().numpy(), want_idx)
    pool.check()
    assert int(err.item()) == expect


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 0.97, 1.0])
def test_compact(kind, in_place, share):
    rng = np.random.default_rng(int(share * 100))
    pages, P = 333, SHAPES[kind]["P"]
    pool = Pool(kind, pages, seed=6, **SHAPES[kind])
    live = rng.permutation(pages)[:int(pages * share)]
    rows = [list(r) for r in np.array_split(live, 5)]
    rows[1] = list(rows[0][:2]) + rows[1]  # shared pages
    refs = np.zeros(pages, int)
    for r in rows:
        for p in r:
            refs[p] += 1
    rows[4], lens = [], [len(r) * P for r in rows]  # the last part is held by the caller alone
    lens[4] = 0
    if lens[2]:
        lens[2] -= P - 1
    _compact(pool, rows, lens, refs, max(1, max(len(r) for r in rows)), in_place)


@pytest.mark.parametrize("pages", [1, 2, 127, 128, 1025, 4095, 4096, 4097, 8193, 33000, 280001])
@pytest.mark.parametrize("share", [0.6, 0.0, 1.0])
def test_compact_pool_sizes(pages, share):
    rng = np.random.default_rng(pages)
    pool = Pool("int8", pages, seed=8, Hkv=1, D=64, P=16)
    refs = (rng.random(pages) < share) * rng.integers(1, 4, pages)
    live = np.flatnonzero(refs)
    rows = [list(live[::2]), list(live[1::2])]
    _compact(pool, rows, [16 * len(r) for r in rows], refs, max(1, pages), False)


def test_compact_bad_entries_are_kept():
    pool = Pool("int8", 50, seed=9, Hkv=1, D=64, P=16)
    refs = np.zeros(50, int)
    refs[[40, 41, 3]] = 1
    _compact(pool, [[40, 7, 50, -1, 41], [3]], [80, 16], refs, 8, False, expect=vx.VX_DATA_BAD_PAGE_ID)


def test_compact_bad_length_keeps_the_row():
    pool = Pool("int8", 10, seed=9, Hkv=1, D=64, P=16)
    geo = pool.geo
    geo.batch = 2
    table = vx.PageTable(dev([0, 2]), dev([9, 8, 7, 6]), dev([33, 32]), 2)  # row 0: longer than max_pages
    refs = dev([0, 0, 0, 0, 0, 0, 1, 1, 1, 1])
    remap, live, err = torch.zeros_like(refs), torch.zeros(1, dtype=torch.int32, device=DEV), err_word()
    vx.vx_compact_pages(geo, pool.vx, table, refs, table.page_indices, refs, remap, live, workspace(geo), err=err)
    assert table.page_indices.tolist() == [9, 8, 1, 0]
    assert remap.tolist() == [-1] * 6 + [0, 1, 2, 3] and refs.tolist() == [1] * 4 + [0] * 6
    assert int(err.item()) == vx.VX_DATA_BAD_SEQ_LEN


# ------------------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_serving_loop_gives_the_same_answers_after_every_page_call(kind):
    """Rows created, written, forked, grown, freed and packed, pages copied to another pool: each row's attention is that
    of its own tokens, kept apart in a second cache whose pages nobody moves."""
    rng, P, Hkv, D, Hq, pages, top = np.random.default_rng(3), 16, 2, 64, 4, 160, 24
    pool = Pool(kind, pages, Hkv=Hkv, D=D, P=P, seed=1)
    quant = kind == "int8"
    g = torch.Generator(DEV).manual_seed(2)
    tokens = []  # of each row: K and V rows [n][Hkv][D]
    lens, refs = dev([0]), torch.zeros(pages, dtype=torch.int32, device=DEV)
    ptr, idx = dev([0]), torch.zeros(top, dtype=torch.int32, device=DEV)
    ws = workspace(pool.geo, 64)
    err = err_word()

    def geometry(batch, n=pages):
        return vx.Geometry(batch, Hq, Hkv, D, D, P, False, n)

    def write(geo, table, first, k, v, p=None):
        t = pool.t if p is None else p
        if quant:
            c = vx.QuantCache(t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"])
            vx.vx_quant_update(geo, table, c, t["centroids"], k, v, first_pos=first, err=err)
        else:
            vx.vx_centroid_update(geo, table, t["k_cache"], t["centroids"], v_cache=t["v_cache"], k_new=k, v_new=v,
                                  first_pos=first, err=err)

    def answers(geo, table, t, q):
        out = torch.empty(geo.batch, Hq, D, dtype=torch.bfloat16, device=DEV)
        w = torch.empty(vx.vx_workspace_size(geo, table.max_pages, top), dtype=torch.uint8, device=DEV)
        sel = torch.arange(top, device=DEV).expand(geo.batch, Hkv, top)
        n = (table.seq_lens + P - 1) // P
        sel = torch.where(sel < n[:, None, None], sel, torch.full_like(sel, -1)).to(torch.int32).contiguous()
        if quant:
            c = vx.QuantCache(t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"])
            vx.vx_sparse_decode_quant(geo, table, q, c, sel, top, out, w, err=err)
        else:
            vx.vx_sparse_decode(geo, table, q, t["k_cache"], t["v_cache"], sel, top, out, w, err=err)
        return out

    plans = [([-1, -1, -1], [40, 17, 100]), ([0, 0, 1, 2, 2], [1, 1, 1, 1, 1]), ([0, 1, 2, 3, 4], [1] * 5),
             ([1, 3, 3, -1], [20, 1, 1, 5]), ([0, 1, 2, 3], [1] * 4), ([2, 1, 0, 0, 3], [1] * 5)]
    for step, (parent, grow) in enumerate(plans):
        geo = geometry(len(lens))
        old = vx.PageTable(ptr, idx, lens, top)
        rows = len(parent)
        new = vx.PageTable(dev(np.arange(rows) * top), torch.zeros(rows * top, dtype=torch.int32, device=DEV),
                           torch.zeros(rows, dtype=torch.int32, device=DEV), top)
        vx.vx_update_table(geo, pool.vx, old, refs, dev(parent), dev(grow), new, refs, ws, err=err)
        ptr, idx, lens = new.page_ptr, new.page_indices, new.seq_lens
        geo = geometry(rows)
        k = torch.randn(sum(grow), Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
        v = torch.randn(sum(grow), Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
        write(geo, new, lens - dev(grow), k, v)
        at, fresh = 0, []
        for p, n in zip(parent, grow):
            base = tokens[p] if p >= 0 else (k[:0], v[:0])
            fresh.append(base + (k[at:at + n], v[at:at + n]) if p >= 0 else (k[at:at + n], v[at:at + n]))
            at += n
        tokens = fresh
        if step % 2:  # pack, and move everything to another pool and back
            remap, live = torch.zeros_like(refs), torch.zeros(1, dtype=torch.int32, device=DEV)
            vx.vx_compact_pages(geo, pool.vx, new, refs, idx, refs, remap, live, ws, err=err)
            n = int(live.item())
            assert bool((refs[:n] > 0).all()) and bool((refs[n:] == 0).all())
            spare = Pool(kind, pages, Hkv=Hkv, D=D, P=P, seed=50 + step)
            ids = torch.arange(n, dtype=torch.int32, device=DEV)
            away = torch.randperm(pages, generator=g, device=DEV)[:n].to(torch.int32)
            vx.vx_copy_pages(geo, pool.vx, spare.vx, ids, away, ws, err=err)
            for x in pool.t.values():
                if x is not None:
                    x.view(torch.uint8)[:n] = 0x7F
            vx.vx_copy_pages(geo, spare.vx, pool.vx, away, ids, ws, err=err)
        # the same rows written, chunk by chunk as they came, into a pool of their own
        apart = Pool(kind, rows * top, Hkv=Hkv, D=D, P=P, seed=99)
        own = vx.PageTable(dev(np.arange(rows) * top), dev(rng.permutation(rows * top)), lens, top)
        geo2 = geometry(rows, rows * top)
        done = torch.zeros_like(lens)
        for part in range(max(len(t) // 2 for t in tokens)):
            ks = [t[2 * part] if len(t) > 2 * part else k[:0] for t in tokens]
            vs = [t[2 * part + 1] if len(t) > 2 * part else k[:0] for t in tokens]
            upto = done + dev([len(x) for x in ks])
            t = vx.PageTable(own.page_ptr, own.page_indices, upto, top)
            write(geo2, t, done, torch.cat(ks), torch.cat(vs), apart.t)
            done = upto
        assert torch.equal(done, lens)
        q = torch.randn(rows, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
        assert torch.equal(answers(geo, new, pool.t, q), answers(geo2, own, apart.t, q))
    assert int(err.item()) == 0


def test_page_calls_captured_and_replayed():
    """The three calls in one graph (they need no host value in between), replayed on new inputs."""
    pool = Pool("int8", 64, Hkv=2, D=64, P=16, seed=4, batch=2)
    geo = vx.Geometry(2, 2, 2, 64, 64, 16, False, 64)
    table = vx.PageTable(dev([0, 8]), dev([60, 61, 62, 0, 0, 0, 0, 0, 50, 51, 0, 0, 0, 0, 0, 0]), dev([40, 20]), 8)
    refs = dev([int(i in (60, 61, 62, 50, 51)) for i in range(64)])
    new = vx.PageTable(dev([0, 8]), torch.zeros(16, dtype=torch.int32, device=DEV),
                       torch.zeros(2, dtype=torch.int32, device=DEV), 8)
    parent, grow = dev([0, 1]), dev([1, 13])
    new_ref, remap = torch.zeros_like(refs), torch.zeros_like(refs)
    live, err, ws = torch.zeros(1, dtype=torch.int32, device=DEV), err_word(), workspace(geo, 2)
    # source and destination of the copy follow from the compaction: page 0 to page 63
    s, d = dev([0]), dev([63])

    def step():
        vx.vx_update_table(geo, pool.vx, table, refs, parent, grow, new, new_ref, ws, err=err)
        vx.vx_compact_pages(geo, pool.vx, new, new_ref, new.page_indices, new_ref, remap, live, ws, err=err)
        vx.vx_copy_pages(geo, pool.vx, pool.vx, s, d, ws, err=err)

    before = [x.clone() for x in pool.t.values() if x is not None]
    graph = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for parent_now, grow_now in (([0, 1], [1, 13]), ([1, 1], [0, 1]), ([-1, 0], [100, 9])):
        for x, y in zip((x for x in pool.t.values() if x is not None), before):
            x.copy_(y)
        parent.copy_(dev(parent_now))
        grow.copy_(dev(grow_now))
        new.page_indices.zero_()
        graph.replay()
        torch.cuda.synchronize()
        host = [x.view(torch.uint8).cpu().numpy() for x in before]
        rows, lens, r2 = ref.update_table(16, [0, 8], [60, 61, 62] + [0] * 5 + [50, 51], [40, 20],
                                          refs.cpu().numpy(), parent_now, grow_now, host)
        remap_w, ref_w, n = ref.compact(r2, host)
        for a in host:
            a[63] = a[0]
        assert int(live.item()) == n and new.seq_lens.tolist() == lens
        assert np.array_equal(new_ref.cpu().numpy(), ref_w) and np.array_equal(remap.cpu().numpy(), remap_w)
        for i, r in enumerate(rows):
            assert new.page_indices[8 * i:8 * i + len(r)].tolist() == [remap_w[p] for p in r]
        for x, y in zip((x for x in pool.t.values() if x is not None), host):
            assert np.array_equal(x.view(torch.uint8).cpu().numpy(), y)
        assert int(err.item()) == 0


def test_pool_of_more_pages_than_prefix_sums():
    """Over 2^20 pages: the ranks' prefix sums then stand for groups of segments."""
    pages, P = 1_100_003, 16
    geo = vx.Geometry(2, 1, 1, 64, 64, P, False, pages)
    g = torch.Generator(DEV).manual_seed(3)
    k = torch.randint(-128, 128, (pages, 1, P, 64), dtype=torch.int8, generator=g, device=DEV)
    pool = vx.PagePool(k, k.clone())
    refs = (torch.rand(pages, generator=g, device=DEV) < 0.7).to(torch.int32)
    live = torch.nonzero(refs)[:, 0].to(torch.int32)
    free = torch.nonzero(refs == 0)[:, 0]
    n = int(live.numel())
    half = n // 2
    table = vx.PageTable(dev([0, half]), live[torch.randperm(n, generator=g, device=DEV)], dev([half * P, (n - half) * P - 5]),
                         n - half)
    ws, err = workspace(geo, 3), err_word()
    # row 0 forked and grown by 200,000 pages, row 1 forked (its last page is copied)
    more = 200_000
    at1, at2 = half + more, n + more
    rows = vx.PageTable(dev([0, at1, at2]), torch.full((2 * n + more,), -5, dtype=torch.int32, device=DEV),
                        torch.zeros(3, dtype=torch.int32, device=DEV), n)
    new_ref = torch.empty_like(refs)
    before = k.clone()
    vx.vx_update_table(geo, pool, table, refs, dev([0, 1, 1]), dev([more * P, 0, 0]), rows, new_ref, ws, err=err)
    assert int(err.item()) == 0
    idx = rows.page_indices
    old0, old1 = table.page_indices[:half], table.page_indices[half:]
    assert torch.equal(idx[:half], old0) and torch.equal(idx[half:half + more], free[:more].to(torch.int32))
    assert torch.equal(idx[at1:at2], old1)
    copied = int(free[more])
    assert int(idx[at2 + n - half - 1]) == copied and torch.equal(idx[at2:at2 + n - half - 1], old1[:-1])
    assert torch.equal(k[copied], before[int(old1[-1])])
    want = refs.clone()
    want[free[:more + 1]] = 1
    want[old1[:-1].long()] += 1
    assert torch.equal(new_ref, want)
    # and packed
    remap, count = torch.empty_like(refs), torch.zeros(1, dtype=torch.int32, device=DEV)
    new_idx, packed = torch.full_like(table.page_indices, -5), torch.empty_like(refs)
    before = k.clone()
    vx.vx_compact_pages(geo, pool, table, new_ref, new_idx, packed, remap, count, ws, err=err)
    m = int((new_ref > 0).sum())
    ids = torch.arange(pages, device=DEV)
    src, dst = ids[(new_ref > 0) & (ids >= m)], ids[(new_ref == 0) & (ids < m)]
    want_map = torch.where(new_ref > 0, ids, torch.full_like(ids, -1))
    want_map[src] = dst
    assert int(count.item()) == m and torch.equal(remap.long(), want_map)
    assert torch.equal(new_idx.long(), want_map[table.page_indices.long()])
    assert torch.equal(k[dst], before[src]) and torch.equal(packed[dst], new_ref[src]) and int(packed[m:].sum()) == 0
    assert int(err.item()) == 0
