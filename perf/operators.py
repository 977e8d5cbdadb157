"""What is measured of the 8-bit cache and page operators of libvx: cases, inputs, plain forms and 64-bit values.

`own` False: run() computes an operator from elementary torch operations, in fp32; True: run() calls the library.
The pools of a state hold only finite values where a result depends on them; slots that no result may depend on
(past a request's length, pages nobody holds) hold the type's worst value.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
QMAX = {"int8": 127.0, "e4m3": 448.0}
LOG2E = 1.4426950408889634


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one request of the smallest workload (4 query heads on one KV head of 64): latency of a single small call
        dict(name="decode_tiny_int8", op="decode", fmt="int8", B=1, Hq=4, Hkv=1, D=64, P=16, lo=1024, hi=1024, k=8,
             empty=False),
        # the headline layer: 16 query heads on 8 KV heads, 32 requests, 128 pages each
        dict(name="decode_b32_e4m3", op="decode", fmt="e4m3", B=32, Hq=16, Hkv=8, D=128, P=16, lo=4096, hi=32768,
             k=128, empty=False),
        # long context with larger pages and a group of 5 heads; odd lengths, one row without any page
        dict(name="decode_long_odd_int8", op="decode", fmt="int8", B=7, Hq=20, Hkv=4, D=128, P=64, lo=60001, hi=131071,
             k=91, empty=True),
        # continuous batching: 256 requests of very different lengths
        dict(name="decode_b256_e4m3", op="decode", fmt="e4m3", B=256, Hq=32, Hkv=8, D=128, P=16, lo=1024, hi=65536,
             k=64, empty=False),
        # one decode token of each of 256 requests written into the cache, every step
        dict(name="append_b256_int8", op="append", fmt="int8", B=256, Hq=32, Hkv=8, D=128, P=16, lo=1024, hi=16384),
        # prompt chunks of eight requests, the first positions in the middle of a page
        dict(name="prefill_b8_e4m3", op="prefill", fmt="e4m3", B=8, Hq=16, Hkv=8, D=128, P=16, lo=4096, hi=32768),
        # beams of 8 requests reordered: shared prefixes, copies of the last pages, one token more each
        dict(name="table_beam_b64", op="table", fmt="bf16", B=64, Hkv=8, D=128, P=16, lo=1024, hi=4096, beams=8,
             fresh=0),
        # a continuous-batching step: every row grows by a token, finished rows are freed, new prompts get pages;
        # one KV head per GPU (tensor parallel)
        dict(name="table_step_b256", op="table", fmt="int8", B=256, Hkv=1, D=128, P=16, lo=1024, hi=65536, beams=1,
             fresh=5),
        # a small latent-cache pool packed
        dict(name="compact_mla_small", op="compact", fmt="mla", B=5, Hkv=1, D=576, P=64, pages=500, live=0.6),
        # a half empty pool packed, before its upper half is given back
        dict(name="compact_half_bf16", op="compact", fmt="bf16", B=32, Hkv=8, D=128, P=16, pages=32768, live=0.5),
        # a few pages of a shared prefix copied before they are written
        dict(name="copy_5_int8", op="copy", fmt="int8", Hkv=8, D=128, P=16, pages=1024, n=5, same=True),
        # preempted requests' pages brought back from another pool
        dict(name="copy_8192_bf16", op="copy", fmt="bf16", Hkv=8, D=128, P=16, pages=10240, n=8192, same=False),
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "prefill", "table", "compact", "copy"])
    Hkv, D, P = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64])
    fmt = rng.choice(["int8", "e4m3"])
    if op == "decode":
        hi = _log(rng, 16, 131072)
        B = min(_log(rng, 1, 256), max(1, 4000000 // (hi * Hkv // 8 + 1)))
        k = min(_log(rng, 1, 256), max(1, 131072 * 16 // (B * Hkv * P)))
        return dict(op=op, fmt=fmt, B=B, Hq=Hkv * rng.randint(1, 16), Hkv=Hkv, D=D, P=P, lo=_log(rng, 1, hi), hi=hi, k=k,
                    empty=rng.random() < 0.3)
    if op == "append":
        hi = _log(rng, 4, 16384)
        return dict(op=op, fmt=fmt, B=_log(rng, 1, 256), Hq=Hkv, Hkv=Hkv, D=D, P=P, lo=_log(rng, 1, hi), hi=hi)
    if op == "prefill":
        hi = _log(rng, 4, 32768)
        return dict(op=op, fmt=fmt, B=min(_log(rng, 1, 64), 200000 // hi + 1), Hq=Hkv, Hkv=Hkv, D=D, P=P,
                    lo=_log(rng, 1, hi), hi=hi)
    fmt = rng.choice(["int8", "bf16", "mla"])
    if fmt == "mla":
        Hkv, D, P = 1, 576, rng.choice([32, 64])
    if op == "table":
        hi = _log(rng, 16, 16384)
        beams = rng.choice([1, 1, 2, 4, 7])
        groups = min(_log(rng, 1, 256 // beams), 400000 // hi + 1)
        return dict(op=op, fmt=fmt, B=groups * beams, Hkv=Hkv, D=D, P=P, lo=_log(rng, 1, hi), hi=hi, beams=beams,
                    fresh=rng.randint(0, min(8, groups * beams)) if beams == 1 else 0)
    if op == "compact":
        return dict(op=op, fmt=fmt, B=rng.randint(1, 64), Hkv=Hkv, D=D, P=P, pages=_log(rng, 64, 20000),
                    live=rng.uniform(0.05, 0.98))
    n = _log(rng, 1, 6000)
    return dict(op=op, fmt=fmt, Hkv=Hkv, D=D, P=P, pages=2 * n + rng.randint(0, n), n=n, same=rng.random() < 0.5)


def _mean_len(c):
    lo, hi = c["lo"], c["hi"]
    return (hi - lo) / math.log(hi / lo) if hi >= 16 * lo else 0.5 * (lo + hi)


def _page_bytes(c):
    """K, V, centroid and scale bytes of one page."""
    Hkv, D, P = c["Hkv"], c["D"], c["P"]
    if c["fmt"] == "mla":
        return P * D * 2 + D * 2
    e = 2 if c["fmt"] == "bf16" else 1
    return Hkv * (2 * P * D * e + D * 2 + (8 if e == 1 else 0))


def work(c):
    op = c["op"]
    if op == "decode":
        L = _mean_len(c)
        n = L / c["P"]
        toks = c["B"] * c["Hkv"] * min(c["k"] * c["P"], L)
        io = c["B"] * c["Hq"] * (4 * c["D"] + 4)
        table = c["B"] * c["Hkv"] * min(c["k"], n + 1) * (4 + 4 + 8)
        return {"bytes": toks * 2 * c["D"] + io + table, "flops": toks * (c["Hq"] / c["Hkv"]) * c["D"] * 4}
    if op == "append":
        # the new token in and out, the page's key codes for its centroid, the centroid and the scales
        rows = c["B"] * c["Hkv"]
        return {"bytes": rows * (4 * c["D"] + 2 * c["D"] + 0.5 * c["P"] * c["D"] + 2 * c["D"] + 16),
                "flops": rows * c["D"] * (0.5 * c["P"] + 4)}
    if op == "prefill":
        toks = c["B"] * 0.9 * _mean_len(c)
        rows = toks * c["Hkv"]
        return {"bytes": rows * (4 * c["D"] + 2 * c["D"]) + rows / c["P"] * (2 * c["D"] + 8), "flops": rows * c["D"] * 5}
    if op == "table":
        ids = c["B"] * _mean_len(c) / c["P"]
        pool = 1.25 * ids / (c["beams"] if c["beams"] > 1 else 1) + 64
        copies = c["B"] * (1 - 1 / c["beams"])
        return {"bytes": 8 * ids + 8 * pool + copies * 2 * _page_bytes(c), "flops": 0}
    if op == "compact":
        moved = c["pages"] * c["live"] * (1 - c["live"])
        return {"bytes": 2 * moved * _page_bytes(c) + 12 * c["pages"] + 8 * c["live"] * c["pages"], "flops": 0}
    return {"bytes": c["n"] * (2 * _page_bytes(c) + 8), "flops": 0}


# ---------------------------------------------------------------------------------------------- inputs

def _lens(c, rng, n):
    """n lengths spread evenly over [lo, hi] (over its logarithm where it spans more than a factor of 16), shuffled."""
    lo, hi = c["lo"], c["hi"]
    at = (np.arange(n) + 0.5) / max(n, 1)
    lens = lo * (hi / lo) ** at if hi >= 16 * lo else lo + (hi - lo) * at
    return rng.permutation(np.clip(lens.astype(np.int64), lo, max(lo, hi)))


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def _table(rng, lens, P, room=0):
    """page_ptr, page_indices (a permutation of a pool 1.125 times as large as needed) and the pool's size."""
    n = -(-lens // P)
    cap = n + room
    pool = int(math.ceil(1.125 * cap.sum())) + 1
    ids = rng.permutation(pool)[:cap.sum()]
    ptr = np.concatenate([[0], np.cumsum(cap)[:-1]])
    return ptr, ids, pool


def _codes(g, shape, fmt):
    """Codes of values ~ N(0, 1) quantised by a page's largest one."""
    out = torch.empty(shape, dtype=torch.int8 if fmt == "int8" else torch.float8_e4m3fn, device=DEV)
    flat = out.view(torch.uint8).view(-1)
    step = 1 << 27
    for a in range(0, flat.numel(), step):
        x = torch.randn(min(step, flat.numel() - a), generator=g, device=DEV)
        if fmt == "int8":
            y = (x * 32).round_().clamp_(-127, 127).to(torch.int8)
        else:
            y = (x * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
        flat[a:a + step] = y.view(torch.uint8)
    return out


def _scales(g, shape, fmt):
    e = torch.randint(-1, 2, shape, generator=g, device=DEV).float()
    return torch.exp2(e - (5 if fmt == "int8" else 6))


def _worst(t):
    """Fills with the type's worst value: NaN, or the largest code."""
    if t.dtype == torch.int8:
        t.fill_(127)
    elif t.dtype == torch.float8_e4m3fn:
        t.view(torch.uint8).fill_(0x7F)
    else:
        t.fill_(float("nan"))


def prepare(case, seed):
    return globals()["_prepare_" + case["op"]](case, seed)


def _gens(seed):
    return np.random.default_rng(seed), torch.Generator(DEV).manual_seed(seed)


def _geometry(c, batch, pool):
    if not own:
        return None
    from paged_block_sparse_kv_b200 import vx
    mla = c["fmt"] == "mla"
    return vx.Geometry(batch, c.get("Hq", c["Hkv"]), c["Hkv"], c["D"], 512 if mla else c["D"], c["P"], mla, pool)


def _blank(s, c):
    """Slots past a request's length get the worst value."""
    P, L = c["P"], s["lens_host"]
    n = -(-L // P)
    last = torch.as_tensor(s["ids_host"][s["ptr_host"] + n - 1], device=DEV)
    past = torch.arange(P, device=DEV)[None, :] >= _dev(L - (n - 1) * P, torch.int64)[:, None]  # [B][P]
    for name in ("k_cache", "v_cache"):
        raw = s[name].view(torch.uint8)
        bad = 0x7F
        rows = raw[last].transpose(1, 2)  # [B][P][Hkv][D]
        rows = torch.where(past[:, :, None, None], torch.full_like(rows, bad), rows)
        raw[last] = rows.transpose(1, 2)


def _quant_pool(c, g, pool):
    shape = (pool, c["Hkv"], c["P"], c["D"])
    return dict(k_cache=_codes(g, shape, c["fmt"]), v_cache=_codes(g, shape, c["fmt"]),
                k_scale=_scales(g, shape[:2], c["fmt"]), v_scale=_scales(g, shape[:2], c["fmt"]))


def _prepare_decode(c, seed):
    rng, g = _gens(seed)
    B, Hkv, D, P, k = c["B"], c["Hkv"], c["D"], c["P"], c["k"]
    lens = _lens(c, rng, B)
    ptr, ids, pool = _table(rng, lens, P)
    s = dict(case=c, lens_host=lens, ptr_host=ptr, ids_host=ids, **_quant_pool(c, g, pool))
    _blank(s, c)
    n = -(-lens // P)
    # random distinct pages of each (request, KV head), ascending, -1 behind the last
    max_pages = int(n.max())
    key = torch.rand(B, Hkv, max_pages, generator=g, device=DEV)
    key = key.masked_fill(torch.arange(max_pages, device=DEV) >= _dev(n, torch.int64)[:, None, None], -1.0)
    kk = min(k, max_pages)
    top = key.topk(kk, dim=-1)
    sel = torch.where(top.values >= 0, top.indices, torch.full_like(top.indices, 1 << 30)).sort(dim=-1).values
    sel = torch.where(sel == 1 << 30, torch.full_like(sel, -1), sel)
    s["sel"] = torch.full((B, Hkv, k), -1, dtype=torch.int32, device=DEV)
    s["sel"][:, :, :kk] = sel.to(torch.int32)
    if c["empty"]:
        s["sel"][B // 2, Hkv - 1] = -1
    s["q"] = torch.randn(B, c["Hq"], D, generator=g, device=DEV).to(torch.bfloat16)
    s["page_ptr"], s["page_indices"], s["seq_lens"] = _dev(ptr), _dev(ids), _dev(lens)
    s["out"] = torch.empty(B, c["Hq"], D, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty(B, c["Hq"], dtype=torch.float32, device=DEV)
    if own:
        from paged_block_sparse_kv_b200 import vx
        s["geo"] = _geometry(c, B, pool)
        s["table"] = vx.PageTable(s["page_ptr"], s["page_indices"], s["seq_lens"], max_pages)
        s["cache"] = vx.QuantCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        s["ws"] = torch.empty(vx.vx_workspace_size(s["geo"], max_pages, k), dtype=torch.uint8, device=DEV)
    return s


def _prepare_write(c, seed, first_of):
    rng, g = _gens(seed)
    B, Hkv, D, P = c["B"], c["Hkv"], c["D"], c["P"]
    lens = _lens(c, rng, B)
    first = first_of(rng, lens)
    ptr, ids, pool = _table(rng, lens, P)
    s = dict(case=c, lens_host=lens, ptr_host=ptr, ids_host=ids, first_host=first, **_quant_pool(c, g, pool))
    N = int((lens - first).sum())
    s["k_new"] = torch.randn(N, Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
    s["v_new"] = torch.randn(N, Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
    s["centroids"] = torch.zeros(pool, Hkv, D, dtype=torch.bfloat16, device=DEV)
    s["page_ptr"], s["page_indices"], s["seq_lens"] = _dev(ptr), _dev(ids), _dev(lens)
    s["first_pos"] = _dev(first)
    s["max_pages"] = int((-(-lens // P)).max())
    if own:
        from paged_block_sparse_kv_b200 import vx
        s["geo"] = _geometry(c, B, pool)
        s["table"] = vx.PageTable(s["page_ptr"], s["page_indices"], s["seq_lens"], s["max_pages"])
        s["cache"] = vx.QuantCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return s


def _prepare_append(c, seed):
    return _prepare_write(c, seed, lambda rng, lens: lens - 1)


def _prepare_prefill(c, seed):
    return _prepare_write(c, seed, lambda rng, lens: (lens * rng.uniform(0.0, 0.2, len(lens))).astype(np.int64))


def _pool_arrays(c, g, pages):
    """Arrays of a page pool, by name; the last dims of each are one page."""
    Hkv, D, P = c["Hkv"], c["D"], c["P"]
    if c["fmt"] == "int8":
        p = _quant_pool(c, g, pages)
    elif c["fmt"] == "mla":
        p = dict(k_cache=torch.randn(pages, 1, P, D, generator=g, device=DEV).to(torch.bfloat16))
    else:
        shape = (pages, Hkv, P, D)
        p = {n: torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) for n in ("k_cache", "v_cache")}
    p["centroids"] = torch.randn(pages, Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
    return p


def _own_pool(p):
    from paged_block_sparse_kv_b200 import vx
    return vx.PagePool(**p)


def _prepare_table(c, seed):
    rng, g = _gens(seed)
    B, P, beams = c["B"], c["P"], c["beams"]
    if beams > 1:
        # each group of beams shares the whole pages of a prefix and owns the rest
        lens = np.repeat(_lens(c, rng, B // beams), beams)
        shared = np.repeat((lens[::beams] * 0.9).astype(np.int64) // P, beams)
        parent = (np.arange(B) // beams) * beams + rng.integers(0, beams, B)
        grow = np.ones(B, np.int64)
    else:
        lens = _lens(c, rng, B)
        shared = np.zeros(B, np.int64)
        parent = np.arange(B)
        gone = rng.permutation(B)[:c["fresh"]]
        parent[gone] = -1
        grow = np.ones(B, np.int64)
        grow[gone] = _lens(c, rng, len(gone))
    n = -(-lens // P)
    ptr = np.concatenate([[0], np.cumsum(n)[:-1]])
    own_pages = np.where(np.arange(B) % beams == 0, n, n - shared)
    grown = np.where(parent >= 0, lens[parent], 0) + grow
    n2 = -(-grown // P)
    need = int(own_pages.sum())
    coming = int((-(-grow[parent < 0] // P)).sum())  # pages of new prompts
    pool = int(math.ceil(1.1 * need)) + coming + 2 * B + 8
    ids = rng.permutation(pool)
    row, at = [], 0
    for b in range(B):
        head = row[b - b % beams][:shared[b]] if b % beams else np.zeros(0, np.int64)
        row.append(np.concatenate([head, ids[at:at + own_pages[b]]]))
        at += own_pages[b]
    idx = np.concatenate(row)
    ref = np.bincount(idx, minlength=pool)
    held = ids[at:at + (pool - need - B) // 50]  # a prefix cache's own pages
    ref[held] += 1
    # the new rows keep room for a page more than they need
    ptr2 = np.concatenate([[0], np.cumsum(n2 + 1)[:-1]])
    cap2 = int(n.sum()) + coming + 2 * B
    s = dict(case=c, pool=_pool_arrays(c, g, pool), lens_host=lens, ptr_host=ptr, idx_host=idx, parent_host=parent,
             grow_host=grow, ref_host=ref, ptr2_host=ptr2, cap2=cap2, max_pages=int(max(n.max(), n2.max())))
    s["page_ptr"], s["page_indices"], s["seq_lens"] = _dev(ptr), _dev(idx), _dev(lens)
    s["parent"], s["grow"], s["ref"] = _dev(parent), _dev(grow), _dev(ref)
    s["new_ptr"] = _dev(ptr2)
    s["new_indices"] = torch.full((cap2,), -1, dtype=torch.int32, device=DEV)
    s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    s["new_ref"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
    if own:
        from paged_block_sparse_kv_b200 import vx
        s["geo"] = _geometry(c, B, pool)
        s["table"] = vx.PageTable(s["page_ptr"], s["page_indices"], s["seq_lens"], s["max_pages"])
        s["new_table"] = vx.PageTable(s["new_ptr"], s["new_indices"], s["new_lens"], s["max_pages"])
        s["own_pool"] = _own_pool(s["pool"])
        s["ws"] = torch.empty(vx.vx_page_workspace_size(s["geo"], B), dtype=torch.uint8, device=DEV)
    return s


def _prepare_compact(c, seed):
    rng, g = _gens(seed)
    B, P, pages = c["B"], c["P"], c["pages"]
    live = max(1, int(pages * c["live"]))
    held = rng.permutation(pages)[:live]
    # most live pages belong to rows, some are shared by two rows, some are held by a prefix cache alone
    cut = np.sort(rng.integers(0, int(live * 0.95) + 1, B - 1)) if B > 1 else np.zeros(0, np.int64)
    parts = np.split(held[:max(1, int(live * 0.95))], cut)
    parts = [np.concatenate([p, held[:rng.integers(0, 3)]]) for p in parts]
    n = np.array([len(p) for p in parts])
    lens = np.where(n > 0, n * P - rng.integers(0, P, B), 0)
    ptr = np.concatenate([[0], np.cumsum(n)[:-1]])
    idx = np.concatenate(parts)
    ref = np.bincount(idx, minlength=pages)
    idx = np.pad(idx, (0, live + 2 * B - len(idx)))
    ref[held[int(live * 0.95):]] += 1
    ref[held] = np.maximum(ref[held], 1)
    s = dict(case=c, pool=_pool_arrays(c, g, pages), lens_host=lens, ptr_host=ptr, idx_host=idx, ref_host=ref,
             max_pages=int(max(1, n.max())))
    s["page_ptr"], s["page_indices"], s["seq_lens"] = _dev(ptr), _dev(idx), _dev(lens)
    s["ref"] = _dev(ref)
    s["new_indices"] = s["page_indices"].clone()
    s["new_ref"] = torch.zeros_like(s["ref"])
    s["remap"] = torch.zeros_like(s["ref"])
    s["num_live"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if own:
        from paged_block_sparse_kv_b200 import vx
        s["geo"] = _geometry(c, B, pages)
        s["table"] = vx.PageTable(s["page_ptr"], s["page_indices"], s["seq_lens"], s["max_pages"])
        s["own_pool"] = _own_pool(s["pool"])
        s["ws"] = torch.empty(vx.vx_page_workspace_size(s["geo"], B), dtype=torch.uint8, device=DEV)
    return s


def _prepare_copy(c, seed):
    rng, g = _gens(seed)
    pages, n = c["pages"], c["n"]
    s = dict(case=c, pool=_pool_arrays(c, g, pages))
    s["src"] = s["pool"] if c["same"] else _pool_arrays(c, g, pages)
    ids = rng.permutation(pages)
    s["src_pages"] = _dev(ids[:n])
    s["dst_pages"] = _dev(ids[n:2 * n] if c["same"] else rng.permutation(pages)[:n])
    if own:
        from paged_block_sparse_kv_b200 import vx
        s["geo"] = _geometry(c, 1, pages)
        s["own_pool"] = _own_pool(s["pool"])
        s["own_src"] = s["own_pool"] if c["same"] else _own_pool(s["src"])
        s["ws"] = torch.empty(vx.vx_page_workspace_size(s["geo"], 1), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------- passes

def run(s):
    return globals()["_run_" + s["case"]["op"]](s)


def _as_float(codes):
    return codes.to(torch.float32)


def _run_decode(s):
    c = s["case"]
    if own:
        from paged_block_sparse_kv_b200 import vx
        vx.vx_sparse_decode_quant(s["geo"], s["table"], s["q"], s["cache"], s["sel"], c["k"], s["out"], s["ws"],
                                  lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    B, Hq, Hkv, D, P = c["B"], c["Hq"], c["Hkv"], c["D"], c["P"]
    sel = s["sel"].long()
    at = s["page_ptr"].long()[:, None, None] + sel.clamp(min=0)
    phys = s["page_indices"].long()[at]
    head = torch.arange(Hkv, device=DEV)[None, :, None]
    pos = sel[..., None] * P + torch.arange(P, device=DEV)
    ok = ((sel >= 0)[..., None] & (pos < s["seq_lens"].long()[:, None, None, None])).flatten(2)  # [B][Hkv][T]

    def values(cache, scale):
        raw = cache.view(torch.uint8)[phys, head].view(cache.dtype)  # [B][Hkv][k][P][D]
        x = _as_float(raw) * scale[phys, head][..., None, None]
        return torch.where(ok[..., None], x.flatten(2, 3), torch.zeros((), device=DEV))

    q = s["q"].float().view(B, Hkv, Hq // Hkv, D) * (1.0 / math.sqrt(D))
    x = torch.matmul(q, values(s["k_cache"], s["k_scale"]).transpose(-1, -2))
    x = torch.where(ok[:, :, None, :], x, torch.full((), -math.inf, device=DEV))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, values(s["v_cache"], s["v_scale"])) / torch.where(l > 0, l, torch.ones_like(l))
    s["out"].copy_(o.view(B, Hq, D))
    s["lse"].copy_((m + torch.log(l)).view(B, Hq))
    return {"out": s["out"], "lse": s["lse"]}


def _pow2_scale(amax, qmax):
    """The smallest power of two s with amax <= qmax * s, at least 2^-126."""
    f, e = torch.frexp(amax / qmax)  # f in [0.5, 1): amax / qmax = f 2^e
    e = torch.where(f == 0.5, e - 1, e)
    return torch.exp2(torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126).float())


def _run_write(s, append):
    c = s["case"]
    if own:
        from paged_block_sparse_kv_b200 import vx
        vx.vx_quant_update(s["geo"], s["table"], s["cache"], s["centroids"], s["k_new"], s["v_new"],
                           first_pos=None if append else s["first_pos"])
    else:
        P, Hkv, D, qmax = c["P"], c["Hkv"], c["D"], QMAX[c["fmt"]]
        L, first = s["seq_lens"].long(), s["first_pos"].long()
        # every touched page: its request b, logical index j, physical id
        j_all = torch.arange(s["max_pages"], device=DEV)[None, :]
        touched = (j_all >= (first // P)[:, None]) & (j_all < ((L + P - 1) // P)[:, None]) & (first < L)[:, None]
        b, j = torch.nonzero(touched, as_tuple=True)
        phys = s["page_indices"].long()[s["page_ptr"].long()[b] + j]
        pos = j[:, None] * P + torch.arange(P, device=DEV)
        new = (pos >= first[b][:, None]) & (pos < L[b][:, None])  # [M][P]
        old = pos < torch.minimum(first, L)[b][:, None]
        row = (torch.cumsum(L - first, 0) - (L - first))[b][:, None] + pos - first[b][:, None]
        row = torch.where(new, row, torch.zeros_like(row))
        for name in ("k", "v"):
            cache, scale = s[name + "_cache"], s[name + "_scale"]
            x = s[name + "_new"].float()[row].transpose(1, 2)  # [M][Hkv][P][D]
            x = torch.where(new[:, None, :, None], x, torch.zeros((), device=DEV))
            s_old = torch.where(old[:, :1], scale[phys], torch.zeros((), device=DEV))
            sc = torch.maximum(_pow2_scale(x.abs().amax((2, 3)), qmax), s_old)[..., None, None]
            raw = cache.view(torch.uint8)[phys]
            have = _as_float(raw.view(cache.dtype)) * (s_old[..., None, None] / sc)
            y = torch.where(new[:, None, :, None], x / sc, have)
            y = (y.round() if c["fmt"] == "int8" else y).to(cache.dtype)
            keep = (new | old)[:, None, :, None]
            cache.view(torch.uint8)[phys] = torch.where(keep, y.view(torch.uint8), raw)
            scale[phys] = sc[..., 0, 0]
            if name == "k":
                total = torch.where(keep, _as_float(y), torch.zeros((), device=DEV)).sum(2)
                m = (new | old).sum(1)[:, None, None]
                s["centroids"][phys] = (total.double() * sc[..., 0].double() / m).to(torch.bfloat16)
    return {k: s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale", "centroids")}


def _run_append(s):
    return _run_write(s, True)


def _run_prefill(s):
    return _run_write(s, False)


def _move(pool_to, dst, pool_from, src):
    for name, a in pool_to.items():
        a[dst] = pool_from[name][src]


def _run_table(s):
    c = s["case"]
    if own:
        from paged_block_sparse_kv_b200 import vx
        vx.vx_update_table(s["geo"], s["own_pool"], s["table"], s["ref"], s["parent"], s["grow"], s["new_table"],
                           s["new_ref"], s["ws"])
    else:
        P, R = c["P"], c["B"]
        lens, parent, ref = s["seq_lens"].long(), s["parent"].long(), s["ref"]
        idx, ptr, ptr2 = s["page_indices"].long(), s["page_ptr"].long(), s["new_ptr"].long()
        n_old = (lens + P - 1) // P
        par = parent.clamp(min=0)
        L = torch.where(parent >= 0, lens[par], torch.zeros_like(parent))
        n = (L + P - 1) // P
        row = torch.arange(R, device=DEV)
        earlier = (parent[None, :] == parent[:, None]) & (row[None, :] < row[:, None])
        first = ~earlier.any(1)
        tail = idx[(ptr[par] + n - 1).clamp(min=0)]
        copy = (L % P != 0) & ~(first & (ref[tail] == 1))
        L2 = L + s["grow"].long()
        n2 = (L2 + P - 1) // P
        need = copy.long() + n2 - n
        start = torch.cumsum(need, 0) - need
        free = torch.nonzero(ref == 0)[:, 0]
        j = torch.arange(s["max_pages"], device=DEV)[None, :]
        kept = j < (n - copy.long())[:, None]
        fresh = (j >= (n - copy.long())[:, None]) & (j < n2[:, None])
        a = idx[torch.where(kept, ptr[par][:, None] + j, torch.zeros_like(j))]
        f = free[torch.where(fresh, start[:, None] + j - (n - copy.long())[:, None], torch.zeros_like(j))]
        ids = torch.where(kept, a, f)
        put = kept | fresh
        s["new_indices"][(ptr2[:, None] + j)[put]] = ids[put].to(torch.int32)
        s["new_lens"].copy_(L2)
        new_ref = ref.long()
        held = j < n_old[:, None]
        went = idx[(ptr[:, None] + j)[held]]
        new_ref = new_ref.scatter_add(0, went, torch.full_like(went, -1))
        came = ids[put]
        s["new_ref"].copy_(new_ref.scatter_add(0, came, torch.ones_like(came)))
        _move(s["pool"], free[start[copy]], s["pool"], tail[copy])
    return {"new_indices": s["new_indices"], "new_lens": s["new_lens"], "new_ref": s["new_ref"], "pool": s["pool"]}


def _run_compact(s):
    c = s["case"]
    if own:
        from paged_block_sparse_kv_b200 import vx
        vx.vx_compact_pages(s["geo"], s["own_pool"], s["table"], s["ref"], s["new_indices"], s["new_ref"], s["remap"],
                            s["num_live"], s["ws"])
    else:
        P = c["P"]
        ref = s["ref"]
        n_live = (ref > 0).sum()
        page = torch.arange(ref.numel(), device=DEV)
        src = torch.nonzero((ref > 0) & (page >= n_live))[:, 0]
        dst = torch.nonzero((ref == 0) & (page < n_live))[:, 0]
        remap = torch.where(ref > 0, page, torch.full_like(page, -1))
        remap[src] = dst
        s["remap"].copy_(remap)
        new_ref = ref.clone()
        new_ref[dst] = ref[src]
        new_ref[src] = 0
        s["new_ref"].copy_(new_ref)
        n = (s["seq_lens"].long() + P - 1) // P
        j = torch.arange(s["max_pages"], device=DEV)[None, :]
        at = (s["page_ptr"].long()[:, None] + j)[j < n[:, None]]
        s["new_indices"][at] = remap[s["page_indices"].long()[at]].to(torch.int32)
        s["num_live"].copy_(n_live)
        _move(s["pool"], dst, s["pool"], src)
    return {"new_indices": s["new_indices"], "new_ref": s["new_ref"], "remap": s["remap"], "num_live": s["num_live"],
            "pool": s["pool"]}


def _run_copy(s):
    if own:
        from paged_block_sparse_kv_b200 import vx
        vx.vx_copy_pages(s["geo"], s["own_src"], s["own_pool"], s["src_pages"], s["dst_pages"], s["ws"])
    else:
        _move(s["pool"], s["dst_pages"].long(), s["src"], s["src_pages"].long())
    return {"pool": s["pool"]}


# ---------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits; page operations compute no numbers."""
    if case["op"] == "decode":
        return _exact_decode(prepare(case, seed))
    if case["op"] in ("append", "prefill"):
        return _exact_write(prepare(case, seed))
    return None


def _exact_decode(s):
    c = s["case"]
    B, Hq, Hkv, D, P = c["B"], c["Hq"], c["Hkv"], c["D"], c["P"]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
    sel_host = s["sel"].cpu().numpy()
    ids = s["ids_host"]
    kd, vd = s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8)
    for b in range(B):
        L = int(s["lens_host"][b])
        toks, pages = [], []
        width = int((sel_host[b] >= 0).sum(1).max())
        if width == 0:
            continue
        pick = sel_host[b][:, :width]
        phys = torch.as_tensor(ids[s["ptr_host"][b] + np.maximum(pick, 0)], device=DEV)
        h = torch.arange(Hkv, device=DEV)[:, None]
        tok = torch.as_tensor(pick[:, :, None] * P + np.arange(P), device=DEV).reshape(Hkv, -1)
        live = (tok < L) & torch.as_tensor(np.repeat(pick >= 0, P, 1), device=DEV)
        K = kd[phys, h].view(s["k_cache"].dtype).double() * s["k_scale"].double()[phys, h][:, :, None, None]
        V = vd[phys, h].view(s["v_cache"].dtype).double() * s["v_scale"].double()[phys, h][:, :, None, None]
        K, V = K.reshape(Hkv, -1, D), V.reshape(Hkv, -1, D)
        K = K.masked_fill(~live[:, :, None], 0.0)
        V = V.masked_fill(~live[:, :, None], 0.0)
        q = s["q"][b].double().reshape(Hkv, G, D)
        z = torch.einsum("hgd,htd->hgt", q, K) / math.sqrt(D)
        z = z.masked_fill(~live[:, None, :], -math.inf)
        some = live.any(1)
        z = z[some]
        lse_b = torch.logsumexp(z, -1)
        w = torch.exp(z - lse_b[..., None])
        o = torch.zeros(Hkv, G, D, dtype=torch.float64, device=DEV)
        o[some] = torch.einsum("hgt,htd->hgd", w, V[some])
        l = torch.full((Hkv, G), -math.inf, dtype=torch.float64, device=DEV)
        l[some] = lse_b
        out[b], lse[b] = o.reshape(Hq, D), l.reshape(Hq)
    return {"out": out, "lse": lse}


def _exact_write(s):
    """Centroids and scales in 64 bits, page by page of each request; codes are compared with the plain form's."""
    c = s["case"]
    P, qmax = c["P"], QMAX[c["fmt"]]
    cen = s["centroids"].double()
    found = {"k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double()}
    row = 0
    for b in range(c["B"]):
        L, f = int(s["lens_host"][b]), int(s["first_host"][b])
        for name in ("k", "v"):
            cache = s[name + "_cache"]
            x = s[name + "_new"][row:row + L - f].double()
            if L == f:
                continue
            j0, j1 = f // P, -(-L // P)
            pages = torch.as_tensor(s["ids_host"][s["ptr_host"][b] + np.arange(j0, j1)], device=DEV)
            lead = f - j0 * P
            full = torch.zeros(((j1 - j0) * P,) + tuple(x.shape[1:]), dtype=torch.float64, device=DEV)
            full[lead:lead + L - f] = x
            full = full.reshape(j1 - j0, P, c["Hkv"], c["D"])
            top = full.abs().amax((1, 3))
            e = torch.ceil(torch.log2(top / qmax))
            e = torch.where(torch.exp2(e - 1) * qmax >= top, e - 1, e)
            e = torch.where(torch.exp2(e) * qmax < top, e + 1, e).clamp(min=-126)
            sc = torch.exp2(torch.where(top > 0, e, torch.full_like(e, -126)))
            codes = full / sc[:, None, :, None]
            codes = codes.round() if c["fmt"] == "int8" else codes.float().to(torch.float8_e4m3fn).double()
            if lead:
                s0 = found[name + "_scale"][pages[0]]
                grown = torch.maximum(s0, sc[0])
                first = full[0] / grown[None, :, None]
                before = cache.view(torch.uint8)[pages[0]].view(cache.dtype).double() * (s0 / grown)[:, None, None]
                first[:lead] = before.transpose(0, 1)[:lead]
                codes[0] = first.round() if c["fmt"] == "int8" else first.float().to(torch.float8_e4m3fn).double()
                sc[0] = grown
            found[name + "_scale"][pages] = sc
            if name == "k":
                there = torch.arange((j1 - j0) * P, device=DEV).reshape(-1, P) + j0 * P < L
                total = (codes * there[:, :, None, None]).sum(1)
                cen[pages] = total * sc[..., None] / there.sum(1)[:, None, None]
        row += L - f
    return {"k_cache": None, "v_cache": None, **found, "centroids": cen}
