"""Plain implementations of the 8-bit cache and page operators, for the tests: numpy, 64 bits, one loop per row or page,
written from the definitions in include/vx.h."""
import numpy as np
import torch

QMAX = {"int8": 127.0, "e4m3": 448.0}
DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
BF16_MAX = float(torch.finfo(torch.bfloat16).max)


def e4m3_values():
    """The 256 values of e4m3, from its definition: bias 7, 3 mantissa bits, S.1111.111 is NaN."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = np.nan if (c & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -x if c & 128 else x
    return v


E4M3 = e4m3_values()


def values(codes_u8, fmt):
    """Code bytes to float64."""
    return codes_u8.view(np.int8).astype(np.float64) if fmt == "int8" else E4M3[codes_u8]


def nearest(x, fmt):
    """float64 to code bytes: nearest, ties to the even code (e4m3: even mantissa)."""
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(x), 448.0)
    _, e = np.frexp(a)  # a = f 2^e with f in [0.5, 1): steps of 2^(e - 4), 2^-9 below the smallest normal
    step = 2.0 ** np.maximum(e - 4, -9).astype(np.float64)
    r = np.minimum(np.rint(a / step) * step, 448.0)
    pos = E4M3[:127]
    return (np.searchsorted(pos, r) + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def to_bf16(x):
    """float64 rounded once to bf16 (as float64)."""
    _, e = np.frexp(x)
    step = 2.0 ** np.maximum(e - 8, -133).astype(np.float64)
    return np.rint(x / step) * step


def pow2_scale(amax, fmt):
    s = 2.0 ** -126
    while QMAX[fmt] * s < amax:
        s *= 2.0
    return s


def quant_update(k, ks, cen, k_new, ptr, idx, L, first, fmt):
    """One of K or V in place: codes k [N][H][P][D] bytes, scales ks [N][H], rows k_new [n][H][D] float64;
    cen (float64, or None for V)."""
    P, row = k.shape[2], 0
    for b in range(len(L)):
        for t in range(int(first[b]), int(L[b])):
            page, slot = idx[ptr[b] + t // P], t % P
            if slot == 0 or t == first[b]:
                # the rows of this page that arrive now
                n = min(int(L[b]) - t, P - slot)
                x = np.nan_to_num(k_new[row:row + n], nan=0.0, posinf=BF16_MAX, neginf=-BF16_MAX)
                for h in range(k.shape[1]):
                    s = pow2_scale(np.abs(x[:, h]).max(), fmt)
                    if slot:
                        old = float(ks[page, h])
                        if s > old:
                            k[page, h, :slot] = nearest(values(k[page, h, :slot], fmt) * (old / s), fmt)
                        s = max(s, old)
                    ks[page, h] = s
                    k[page, h, slot:slot + n] = nearest(x[:, h] / s, fmt)
                    if cen is not None:
                        cen[page, h] = to_bf16(s * values(k[page, h, :slot + n], fmt).sum(0) / (slot + n))
            row += 1


def attend(q, kv, vv, ptr, idx, L, sel, scale):
    """Attention over float64 values kv, vv [N][H][P][D]: out, lse, and for the error bounds the sums of
    |weight * value|, of |q_d k_d| (largest over tokens), the largest |logit| and the sum of |value|."""
    B, Hq, D = q.shape
    H, P = kv.shape[1], kv.shape[2]
    G = Hq // H
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    mass, dot, big, total = np.zeros((B, Hq, D)), np.zeros((B, Hq)), np.zeros((B, Hq)), np.zeros((B, Hq, D))
    for b in range(B):
        for h in range(H):
            rows = [(idx[ptr[b] + j], min(P, int(L[b]) - j * P)) for j in sel[b, h] if j >= 0]
            if not rows:
                continue
            K = np.concatenate([kv[p, h, :n] for p, n in rows])
            V = np.concatenate([vv[p, h, :n] for p, n in rows])
            for g in range(h * G, (h + 1) * G):
                x = scale * (K @ q[b, g])
                m = x.max()
                w = np.exp(x - m)
                out[b, g], lse[b, g] = w @ V / w.sum(), m + np.log(w.sum())
                mass[b, g] = w @ np.abs(V) / w.sum()
                dot[b, g] = scale * (np.abs(K) @ np.abs(q[b, g])).max()
                big[b, g] = np.abs(x).max()
                total[b, g] = np.abs(V).sum(0)
    return out, lse, mass, dot, big, total


def update_table(P, ptr, idx, L, ref, parent, grow, pools, max_pages=1 << 30):
    """New rows (lists of page ids), lengths and references; pools (numpy arrays) get the copies.  None, when the free
    pages do not suffice or a new row has more than max_pages."""
    old = [list(idx[ptr[b]:ptr[b] + -(-int(L[b]) // P)]) for b in range(len(L))]
    free = [p for p in range(len(ref)) if ref[p] == 0]
    rows, lens, seen, copies = [], [], set(), []
    for p, g in zip(parent, grow):
        row, n = (list(old[p]), int(L[p])) if p >= 0 else ([], 0)
        want = -(-(n + int(g)) // P) - len(row)
        if n % P:
            if p in seen or ref[row[-1]] != 1:
                if not free:
                    return None
                copies.append((row[-1], free[0]))
                row[-1] = free.pop(0)
        seen.add(p)
        if want > len(free) or len(row) + want > max_pages:
            return None
        row += free[:want]
        del free[:want]
        rows.append(row)
        lens.append(n + int(g))
    new_ref = np.array(ref)
    for r in old:
        for p in r:
            new_ref[p] -= 1
    for r in rows:
        for p in r:
            new_ref[p] += 1
    for s, d in copies:
        for a in pools:
            a[d] = a[s]
    return rows, lens, new_ref


def compact(ref, pools):
    """remap and references after it; pools (numpy arrays) get the moves."""
    live = [p for p in range(len(ref)) if ref[p] > 0]
    n = len(live)
    holes = [p for p in range(n) if ref[p] == 0]
    remap, new_ref = np.full(len(ref), -1), np.zeros(len(ref), int)
    for p in live:
        d = p if p < n else holes.pop(0)
        remap[p], new_ref[d] = d, ref[p]
        if d != p:
            for a in pools:
                a[d] = a[p]
    return remap, new_ref, n
