"""8-bit caches at the edges of their contract, against plain 64-bit implementations."""
import numpy as np
import pytest
import torch

import quant_ref as ref
from paged_block_sparse_kv_b200 import vx
from test_gpu_quant import DEV, FMTS, WRITES, Case, check_attention, check_cache, decode, dev, new_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("over", [0, 1, 32])
def test_lengths_that_add_up_to_more_than_32_bits(P, over):
    """Two requests of almost 2^31 tokens bring more rows than there are, and so does every request behind them, although
    the sum of the lengths, taken modulo 2^32, is small again: nothing is written."""
    top = 2 ** 31 // P - 1
    huge = top * P  # P tokens short of 2^31, so the two are 2 P short of 2^32
    last = (2 * P + over, 20)
    c = Case("int8", [P, P, *last], 2, 2, 64, P, seed=3).blank()
    cache, cen = c.cache(), torch.zeros(c.pool, 2, 64, dtype=torch.bfloat16, device=DEV)
    x = new_rows(c, 70).to(DEV)
    t = vx.PageTable(c.table.page_ptr, c.table.page_indices, dev(np.array([huge, huge, *last])), top)
    vx.vx_quant_update(c.geo, t, cache, cen, x, x, first_pos=dev(np.zeros(4)), err=c.err)
    check_cache(c, cache, cen, np.zeros((c.pool, 2, 64)))
    assert int(c.err.item()) == vx.VX_DATA_BAD_SEQ_LEN
    # the same behind a request that fits: that one is written
    c = Case("int8", [30, P, P, *last], 2, 2, 64, P, seed=4).blank()
    cache, cen = c.cache(), torch.zeros(c.pool, 2, 64, dtype=torch.bfloat16, device=DEV)
    t = vx.PageTable(c.table.page_ptr, c.table.page_indices, dev(np.array([30, huge, huge, *last])), top)
    c.err.zero_()
    vx.vx_quant_update(c.geo, t, cache, cen, x, x, first_pos=dev(np.zeros(5)), err=c.err)
    want = np.zeros((c.pool, 2, 64))
    for a, s, w in ((c.k, c.ks, want), (c.v, c.vs, None)):
        ref.quant_update(a, s, w, x.double().cpu().numpy(), c.ptr, c.idx, [30], [0], "int8")
    check_cache(c, cache, cen, want)
    assert int(c.err.item()) == vx.VX_DATA_BAD_SEQ_LEN


def bf16_grid(lo, hi):
    """Every positive bf16 number in [lo, hi)."""
    a, b = (np.array([v], np.float32).view(np.uint32)[0] >> 16 for v in (lo, hi))
    return (np.arange(a, b, dtype=np.uint32) << 16).view(np.float32)


def test_int8_codes_under_an_odd_scale_are_the_same_in_an_append_and_a_prefill():
    """Values whose fp32 product with 1 / s rounds onto a tie of two codes that the exact product lies beside."""
    rng, D, P, B = np.random.default_rng(5), 64, 16, 40
    scales, rows = [], []
    x = bf16_grid(0.5, 90.0)
    while len(scales) < B:
        s = rng.uniform(0.75, 1.25, 1).astype(np.float32)[0]
        inv = np.float32(1) / s
        y = x * inv
        split = x[(np.rint(y) != np.rint(x.astype(np.float64) * np.float64(inv))) & (y < 127)]
        if len(split):
            scales.append(s)
            rows.append(np.where(rng.random(D) < 0.5, -1, 1) * rng.choice(np.concatenate([split, split, x[:400]]), D))
    scales, rows = np.array(scales, np.float32), np.array(rows, np.float32)
    got = []
    for prefill in (False, True):
        c = Case("int8", [2] * B, 1, 1, D, P, seed=6).fill()
        first = c.idx[c.ptr]
        c.ks[first, 0] = c.vs[first, 0] = scales
        cache, cen = c.cache(), torch.zeros(c.pool, 1, D, dtype=torch.bfloat16, device=DEV)
        new = torch.from_numpy(rows)[:, None].to(torch.bfloat16).to(DEV)
        vx.vx_quant_update(c.geo, c.table, cache, cen, new, new, first_pos=dev(np.ones(B)) if prefill else None, err=c.err)
        assert int(c.err.item()) == 0
        assert np.array_equal(cache.k_scale.cpu().numpy(), c.ks, equal_nan=True)
        got += [a.cpu().numpy()[first, 0, 1] for a in (cache.k_cache, cache.v_cache)]
    want = np.rint(rows * (np.float32(1) / scales)[:, None])
    for g in got:
        assert np.array_equal(g, want)


@pytest.mark.parametrize("fmt,code,exponent", [("int8", 127, 121), ("int8", -127, 100), ("e4m3", 448, 119), ("e4m3", -448, 112)])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_values_of_one_sign_at_the_end_of_the_range(fmt, code, exponent, D, P):
    """Every value is the same large number, up to bf16's largest: so is every output, however the row is split, though the
    sum of the weighted values before its division by the sum of the weights is far outside fp32's range."""
    c = Case(fmt, [P, 6 * P + 3, 200 * P - 1], 4, 2, D, P, seed=17).fill()
    for b, n in enumerate(c.L):
        for j in range(-(-int(n) // P)):
            c.v[c.idx[c.ptr[b] + j], :, :min(P, int(n) - j * P)] = ref.nearest(np.array([float(code)]), fmt)[0]
    c.vs[:] = 2.0 ** exponent
    q, cache = c.queries(0.25), c.cache()
    for k in (6, 30, 200):  # a block per row; few partials; many
        sel = c.select(k)
        value = code * 2.0 ** exponent
        for splits in (0, 1, 3, 24, 100000):
            out, lse = decode(c, cache, q.to(DEV), dev(sel), num_splits=splits)
            # weights sum to one up to their roundings: fp16 weights (2^-11), the merge's (2^-18), and out's own to bf16
            rel = (out.double() / value - 1).abs()
            assert bool(torch.isfinite(out).all()) and float(rel.max()) <= 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18, (k, splits)
            assert bool(torch.isfinite(lse).all())
    assert int(c.err.item()) == 0


def attend_mixed(c, q, sel, scale):
    """64-bit attention with, per output element, what check_mixed needs: each token's logit is exact to
    (D / 16 + 4) 2^-23 of sum |q_d k_d| and 2^-22 of the largest |logit|."""
    out, lse, tol, ltol = (np.zeros((len(c.L), c.Hq, c.D)), np.full((len(c.L), c.Hq), -np.inf),
                           np.zeros((len(c.L), c.Hq, c.D)), np.zeros((len(c.L), c.Hq)))
    kc, vc = ref.values(c.k, c.fmt), ref.values(c.v, c.fmt)
    for b in range(len(c.L)):
        for h in range(c.Hkv):
            pages = [(c.idx[c.ptr[b] + j], min(c.P, int(c.L[b]) - j * c.P)) for j in sel[b, h] if j >= 0]
            if not pages:
                continue
            K = np.concatenate([kc[p, h, :n] * np.float64(c.ks[p, h]) for p, n in pages])
            C = np.concatenate([vc[p, h, :n] for p, n in pages])
            s = np.concatenate([np.full(n, np.float64(c.vs[p, h])) for p, n in pages])
            for g in range(h * c.Hq // c.Hkv, (h + 1) * c.Hq // c.Hkv):
                x = scale * (K @ q[b, g])
                w = np.exp(x - x.max())
                share = w / w.sum()
                out[b, g], lse[b, g] = (share * s) @ C, x.max() + np.log(w.sum())
                # the logits' error, weighing only what has weight
                dx = (c.D / 16 + 4) * 2.0 ** -23 * scale * (np.abs(K) @ np.abs(q[b, g])) + 2.0 ** -22 * np.abs(x).max()
                lost = 2.0 ** -35 * np.abs(share * s).max()  # an element of P below fp16's normal numbers
                tol[b, g] = (np.abs(share * s) * (2.0 ** -11 + 2.0 ** -17 + 2 * dx)) @ np.abs(C) + lost * np.abs(C).sum(0)
                tol[b, g] += (share * dx).sum() * np.abs(out[b, g]) + 2.0 ** -8 * np.abs(out[b, g]) + 2.0 ** -133
                ltol[b, g] = (share * dx).sum() + 2.0 ** -20 * (1 + abs(lse[b, g]))
    return out, lse, tol, ltol


def check_mixed(out, lse, want):
    o, l, tol, ltol = want
    e = np.abs(out.double().cpu().numpy() - o)
    assert (e <= tol).all(), (e / tol).max()
    e = np.abs(lse.double().cpu().numpy() - l)
    assert (e <= ltol).all(), (e / ltol).max()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hq,Hkv,D,P", [(4, 2, 64, 16), (12, 1, 128, 16), (8, 1, 128, 64)])
@pytest.mark.parametrize("lo,hi,slope", [(-42, 0, 2.0), (-42, 0, -2.0), (-110, 100, 1.4), (-110, 100, -1.4), (-110, 100, 0.0),
                                         (-3, 3, 5.0)])
def test_value_scales_far_apart_in_one_row(fmt, Hq, Hkv, D, P, lo, hi, slope):
    """Pages whose value scales differ by up to 2^210, and whose logits make up for it, or not (slope: logit per power of two,
    in units of -ln 2 / 2): what carries the output is kept, whatever else the row holds."""
    c = Case(fmt, [P, 7 * P - 5, 61 * P + 3, 30 * P], Hq, Hkv, D, P, seed=23).fill()
    exps = c.rng.integers(lo, hi + 1, c.vs.shape)
    exps[c.rng.random(exps.shape) < 0.2] = hi
    exps[c.rng.random(exps.shape) < 0.4] = lo
    c.vs[:] = 2.0 ** exps * c.rng.uniform(1.0, 1.9, exps.shape)
    # keys near a constant direction, so that a page's key scale sets its logits
    base = 32.0
    for b, n in enumerate(c.L):
        for j in range(-(-int(n) // P)):
            p, m = c.idx[c.ptr[b] + j], min(P, int(n) - j * P)
            c.k[p, :, :m] = ref.nearest(base + c.rng.integers(-3, 4, (Hkv, m, D)), fmt)
    q = torch.from_numpy(1 + 0.1 * c.rng.standard_normal((len(c.L), Hq, D))).to(torch.bfloat16)
    logit = -slope * np.log(2) / 2 * exps + c.rng.standard_normal(exps.shape)
    c.ks[:] = logit / (base * np.sqrt(D))
    cache = c.cache()
    for k in (7, 32, 62):
        sel = c.select(k)
        want = attend_mixed(c, q.double().numpy(), sel, 1 / np.sqrt(D))
        for splits in (0, 1, 5, 100000):
            out, lse = decode(c, cache, q.to(DEV), dev(sel), num_splits=splits)
            check_mixed(out, lse, want)
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_pages_of_zeros_and_zero_scales_in_a_row(fmt):
    """A page of zeros has the smallest scale there is, another program's may have scale 0: neither changes its row."""
    c = Case(fmt, [16, 400, 33], 4, 2, 64, 16, seed=29).fill()
    for b in range(3):
        for j in range(0, -(-int(c.L[b]) // 16), 2):
            c.vs[c.idx[c.ptr[b] + j]] = [2.0 ** -126, 0.0][j % 4 // 2]
            if j % 4 == 0:
                c.v[c.idx[c.ptr[b] + j]] = 0
    c.v[c.idx[c.ptr[2]]], c.vs[c.idx[c.ptr[2]]] = 0, 2.0 ** -126
    q, cache = c.queries(), c.cache()
    for k in (3, 25):
        sel = c.select(k)
        want = attend_mixed(c, q.double().numpy(), sel, 1 / 8)
        for splits in (0, 3):
            check_mixed(*decode(c, cache, q.to(DEV), dev(sel), num_splits=splits), want)
    assert int(c.err.item()) == 0


def plain_write(codes, scales, cen, x, c, L, first):
    """vx_quant_update of keys (cen an array) or values (None) from the header's text, page by page: scales in fp32, a code
    the fp32 product x * (1 / s) rounded, older codes times s_old / s when the scale grows, centroids in 64 bits."""
    f32, row = np.float32, 0
    for b in range(len(L)):
        t = int(first[b])
        while t < int(L[b]):
            page, slot = c.idx[c.ptr[b] + t // c.P], t % c.P
            n = min(int(L[b]) - t, c.P - slot)
            for h in range(c.Hkv):
                new = x[row:row + n, h].astype(f32)
                s = f32(ref.pow2_scale(np.abs(new).max(), c.fmt))
                if slot:
                    old = scales[page, h]
                    s = max(s, old)
                    if s > old:
                        was = ref.values(codes[page, h, :slot], c.fmt).astype(f32)
                        codes[page, h, :slot] = ref.nearest((was * (old / s)).astype(np.float64), c.fmt)
                scales[page, h] = s
                codes[page, h, slot:slot + n] = ref.nearest((new * (f32(1) / s)).astype(np.float64), c.fmt)
                if cen is not None:
                    total = ref.values(codes[page, h, :slot + n], c.fmt).sum(0)
                    cen[page, h] = ref.to_bf16(np.float64(s) * total / (slot + n))
            row, t = row + n, t + n


def odd_scales(c):
    """Another program's scales: any fp32 numbers, some of them just under a power of two, some far from ordinary."""
    for s in (c.ks, c.vs):
        wild = c.rng.random(s.shape)
        s[:] = np.where(wild < 0.2, s * f32_pow2(c.rng, s.shape, -90, -80), s)
        s[:] = np.where((wild > 0.2) & (wild < 0.4), np.nextafter(2.0 ** np.rint(np.log2(s)), 0, dtype=np.float32), s)


def f32_pow2(rng, shape, lo, hi):
    return (2.0 ** rng.integers(lo, hi, shape)).astype(np.float32)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", range(len(WRITES)))
@pytest.mark.parametrize("scales", ["powers", "odd"])
def test_prefill_into_filled_pages_is_exact(fmt, case, scales):
    """Scales, all codes (new ones, older ones under a raised scale, untouched slots and pages) and centroids, bit for bit."""
    L, first, Hkv, D, P = WRITES[case]
    c = Case(fmt, L, Hkv, Hkv, D, P, seed=100 + case).fill()
    if scales == "odd":
        odd_scales(c)
    else:
        for s in (c.ks, c.vs):
            s[:] = 2.0 ** np.rint(np.log2(s))
    n = int((np.array(L) - np.array(first)).sum())
    kn, vn = new_rows(c, n), new_rows(c, n)
    cache = c.cache()
    cen = torch.full((c.pool, Hkv, D), 0.5, dtype=torch.bfloat16, device=DEV)
    want = np.full((c.pool, Hkv, D), 0.5)
    vx.vx_quant_update(c.geo, c.table, cache, cen, kn.to(DEV), vn.to(DEV), first_pos=dev(np.array(first)), err=c.err)
    plain_write(c.k, c.ks, want, kn.float().numpy(), c, L, first)
    plain_write(c.v, c.vs, None, vn.float().numpy(), c, L, first)
    check_cache(c, cache, cen, want)
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("P,D,Hkv", [(16, 128, 8), (32, 64, 1), (64, 128, 2), (64, 64, 4), (16, 64, 16)])
def test_appends_under_odd_scales_are_exact(fmt, P, D, Hkv):
    """Tokens appended one by one to pages that another program filled in part, until they are full and others begin."""
    B, steps = 5, P // 2 + 3
    c = Case(fmt, [P // 2 + steps + 3 * b for b in range(B)], Hkv, Hkv, D, P, seed=P + D + Hkv).fill()
    odd_scales(c)
    cache = c.cache()
    cen = torch.full((c.pool, Hkv, D), 0.5, dtype=torch.bfloat16, device=DEV)
    want = np.full((c.pool, Hkv, D), 0.5)
    for step in range(steps):
        lens = c.L - steps + step + 1
        kn, vn = new_rows(c, B, 6), new_rows(c, B, 6)
        t = vx.PageTable(c.table.page_ptr, c.table.page_indices, dev(lens), c.max_pages)
        vx.vx_quant_update(c.geo, t, cache, cen, kn.to(DEV), vn.to(DEV), err=c.err)
        plain_write(c.k, c.ks, want, kn.float().numpy(), c, lens, lens - 1)
        plain_write(c.v, c.vs, None, vn.float().numpy(), c, lens, lens - 1)
        check_cache(c, cache, cen, want)
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("prefill", [False, True])
def test_an_odd_scale_gives_way_to_the_power_of_two_the_token_needs(prefill):
    """0.9 * 127 = 114 would hold a token of 100, whose power of two is 1: the scale becomes 1, the older codes times 0.9."""
    c = Case("int8", [4], 1, 1, 64, 16, seed=1).fill()
    page = c.idx[0]
    c.ks[page] = c.vs[page] = 0.9
    c.k[page, 0, :3] = c.v[page, 0, :3] = np.arange(-96, 96, dtype=np.int64).reshape(3, 64).astype(np.int8).view(np.uint8)
    cache, cen = c.cache(), torch.zeros(c.pool, 1, 64, dtype=torch.bfloat16, device=DEV)
    x = torch.full((1, 1, 64), 100.0, dtype=torch.bfloat16, device=DEV)
    vx.vx_quant_update(c.geo, c.table, cache, cen, x, x, first_pos=dev([3]) if prefill else None, err=c.err)
    assert float(cache.k_scale[page]) == 1 and float(cache.v_scale[page]) == 1
    was = np.arange(-96, 96).astype(np.float32) * np.float32(0.9)  # in fp32, where 95 * 0.9 is the tie 85.5
    for a in (cache.k_cache, cache.v_cache):
        got = a[page, 0].cpu().numpy()
        assert np.array_equal(got[:3].ravel(), np.rint(was)) and (got[3] == 100).all()


@pytest.mark.parametrize("P", [16, 64])
def test_prefill_of_no_rows(P):
    """A step in which no request brings tokens: an empty tensor's pointer is NULL, and nothing is written."""
    c = Case("e4m3", [P, 3 * P + 1, 5], 2, 2, 64, P, seed=7).fill()
    cache, cen = c.cache(), torch.full((c.pool, 2, 64), 0.5, dtype=torch.bfloat16, device=DEV)
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    vx.vx_quant_update(c.geo, c.table, cache, cen, x, x, first_pos=dev(c.L), err=c.err)
    assert int(c.err.item()) == 0
    vx.vx_quant_update(c.geo, c.table, cache, cen, x, x, first_pos=dev(c.L - 1), err=c.err)
    assert int(c.err.item()) == vx.VX_DATA_BAD_SEQ_LEN  # rows that are not there
    check_cache(c, cache, cen, np.full((c.pool, 2, 64), 0.5))


@pytest.mark.parametrize("fmt", FMTS)
def test_tiny_queries_under_large_key_scales(fmt):
    """Queries among bf16's smallest numbers, keys whose scales make up for it, and a small sm_scale: their product is
    ordinary, and so is its precision."""
    c = Case(fmt, [90, 200, 700], 4, 2, 64, 16, seed=31).fill()
    q = (c.queries().double() * torch.tensor([2.0 ** -126, 2.0 ** -112, 2.0 ** -99])[:, None, None]).to(torch.bfloat16)
    for b, e in enumerate((126, 118, 104)):
        pages = c.idx[c.ptr[b]:c.ptr[b] + -(-int(c.L[b]) // 16)]
        c.ks[pages] = 2.0 ** (e - c.rng.integers(0, 3, c.ks[pages].shape)) * c.rng.uniform(0.6, 0.9, c.ks[pages].shape)
    sel, cache = c.select(44), c.cache()
    for sm in (2.0 ** -9, 2.0 ** -14):
        want = attend_mixed(c, q.double().numpy(), sel, sm)
        for splits in (0, 4):
            check_mixed(*decode(c, cache, q.to(DEV), dev(sel), num_splits=splits, sm_scale=sm), want)
    sel = sel[:, :, :5]
    check_mixed(*decode(c, cache, q.to(DEV), dev(sel), sm_scale=2.0 ** -12), attend_mixed(c, q.double().numpy(), sel, 2.0 ** -12))
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("tiles", [1, 2, 3, 40])
def test_a_scale_that_is_no_number_shows_in_its_row_alone(bad, tiles):
    c = Case("int8", [16 * tiles, 16 * tiles], 4, 2, 64, 16, seed=37).fill()
    c.vs[c.idx[c.ptr[0] + tiles // 2], 1] = bad
    q, sel, cache = c.queries(), c.select(tiles), c.cache()
    for splits in (0, 1, 3):
        out, lse = decode(c, cache, q.to(DEV), dev(sel), num_splits=splits)
        assert not bool(torch.isfinite(out[0, 2:]).any()) and bool(torch.isfinite(out[0, :2]).all())
        assert bool(torch.isfinite(out[1]).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("fmt", FMTS)
def test_appending_step_captured_and_replayed(fmt):
    """A graph of the quantising append and the chained step, replayed as the tokens, queries and lengths change: bit for bit
    what the calls give outside of a graph."""
    B, Hq, Hkv, D, P, k, steps = 3, 8, 4, 128, 16, 6, 20
    c = Case(fmt, [300, 40, 16 + steps], Hq, Hkv, D, P, seed=43).fill()
    for s in (c.ks, c.vs):
        s[:] = 2.0 ** np.rint(np.log2(s))
    lens = dev(c.L - steps)
    state = [(c.cache(), torch.randn(c.pool, Hkv, D, generator=torch.Generator(DEV).manual_seed(1), device=DEV).to(torch.bfloat16))
             for _ in range(2)]
    kn, vn, q = (torch.zeros(B, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hkv, Hkv, Hq))
    ws = torch.empty(vx.vx_workspace_size(c.geo, c.max_pages, k), dtype=torch.uint8, device=DEV)
    outs = [(torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=DEV), torch.zeros(B, Hq, device=DEV)) for _ in range(2)]
    t = vx.PageTable(c.table.page_ptr, c.table.page_indices, lens, c.max_pages)

    def step(i):
        vx.vx_block_topk_decode_append_quant(c.geo, t, q, *state[i], kn, vn, k, outs[i][0], ws, lse=outs[i][1], err=c.err)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(0)
    for _ in range(steps):
        lens.add_(1)
        kn.copy_(new_rows(c, B, 2))
        vn.copy_(new_rows(c, B, 2))
        q.copy_(c.queries())
        ws.random_(0, 256)
        graph.replay()
        step(1)
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        (a, ca), (b, cb) = state
        assert torch.equal(ca, cb) and torch.equal(a.k_cache.view(torch.uint8), b.k_cache.view(torch.uint8))
        assert torch.equal(a.v_cache.view(torch.uint8), b.v_cache.view(torch.uint8))
        for x, y in ((a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
            assert torch.equal(x.nan_to_num(), y.nan_to_num())
    assert int(c.err.item()) == 0 and bool(torch.isfinite(outs[0][0]).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lo,hi", [(-8, -4), (-60, 30)])
def test_scales_of_both_signs(fmt, lo, hi):
    """Scales are any finite numbers: negative key and value scales, some zero."""
    c = Case(fmt, [16, 700, 333], 12, 2, 128, 16, seed=41).fill()
    sign = lambda: c.rng.choice([-1.0, 1.0], c.ks.shape)
    c.ks[:] = sign() * 2.0 ** c.rng.integers(-8, -5, c.ks.shape)
    c.vs[:] = sign() * 2.0 ** c.rng.integers(lo, hi, c.vs.shape) * c.rng.uniform(1, 2, c.vs.shape)
    c.ks[c.rng.random(c.ks.shape) < 0.1] = 0
    q, cache = c.queries(), c.cache()
    for k in (5, 44):
        sel = c.select(k)
        want = attend_mixed(c, q.double().numpy(), sel, 1 / np.sqrt(128))
        for splits in (0, 1, 7):
            check_mixed(*decode(c, cache, q.to(DEV), dev(sel), num_splits=splits), want)
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", [1e4, 1e7, 1e9, 1e20, 1e30])
@pytest.mark.parametrize("k", [7, 40])
def test_large_logits_stay_a_mean_of_values(fmt, size, k):
    """Logits so large that fp32 has no digits left behind the point, beside ordinary value scales: the output is still a mean
    of the row's values, so no larger than the largest."""
    c = Case(fmt, [16, 640, 333], 8, 2, 64, 16, seed=47).fill()
    c.vs[:] = 2.0 ** c.rng.integers(-9, 9, c.vs.shape) * c.rng.uniform(1, 2, c.vs.shape)
    q, cache = c.queries(), c.cache()
    sel = c.select(k)
    values = c.float_values()[1]
    for splits in (0, 1, 5):
        out, lse = decode(c, cache, q.to(DEV), dev(sel), num_splits=splits, sm_scale=size)
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
        for b in range(3):
            for h in range(2):
                top = np.max([np.abs(values[c.idx[c.ptr[b] + j], h, :min(16, c.L[b] - 16 * j)]).max((0,)) for j in sel[b, h]
                              if j >= 0], axis=0)
                got = out[b, 4 * h:4 * h + 4].double().abs().cpu().numpy()
                assert (got <= top * (1 + 2.0 ** -7)).all()
