"""Plain CPU oracle of the paged NVFP4 KV cache: the page layout, appending,
attention in 64 bits, and the page pool's bookkeeping as Python loops.

TEST INFRASTRUCTURE ONLY; shares nothing with the CUDA path. Layout: pages
[P][heads][page/16][18*D] bytes; a granule holds K codes [16][D/2], K scales
[16][D/16], V codes, V scales of 16 tokens.
"""
from __future__ import annotations

import numpy as np

from oracle import nvfp4_oracle as o


def granule_views(pages: np.ndarray, page_size: int, D: int):
    """(K codes, K scales, V codes, V scales) views [P, heads, page_size, ...] (writable copies of slices)."""
    P, H, _ = pages.shape
    gr = pages.reshape(P, H, page_size // 16, 18 * D)
    out = []
    for base in (0, 9 * D):
        out.append(gr[..., base:base + 8 * D].reshape(P, H, page_size, D // 2))
        out.append(gr[..., base + 8 * D:base + 9 * D].reshape(P, H, page_size, D // 16))
    return out


def write_token(pages, page, head, slot, D, which, codes, scales):
    """Place one token's packed codes [D/2] and scales [D/16]; which = 0 for K, 1 for V."""
    gr = pages[page, head].reshape(-1, 18 * D)[slot // 16]
    base, r = which * 9 * D, slot % 16
    gr[base + r * (D // 2): base + (r + 1) * (D // 2)] = codes
    gr[base + 8 * D + r * (D // 16): base + 8 * D + (r + 1) * (D // 16)] = scales


def append(pages, k, v, table, cu, kv_len, k_g, v_g, page_size, mode):
    """Quantize rows of k, v [T, heads, D] (FP32 arrays of BF16 values) into pages, in place."""
    D = k.shape[2]
    for which, (x, g) in enumerate(((k, k_g), (v, v_g))):
        T, H, _ = x.shape
        q = o.quantize(x.reshape(T * H, D), mode, np.float32(g))
        codes = o.pack_codes(q["codes"]).reshape(T, H, D // 2)
        scales = q["scales"].reshape(T, H, D // 16)
        for b in range(len(kv_len)):
            n = cu[b + 1] - cu[b]
            for i in range(n):
                pos = kv_len[b] - n + i
                for h in range(H):
                    write_token(pages, table[b][pos // page_size], h, pos % page_size, D, which, codes[cu[b] + i, h],
                                scales[cu[b] + i, h])


def gather(pages, table_row, length, page_size, D, k_g, v_g):
    """K, V [heads, length, D] in FP64."""
    n = -(-length // page_size)
    ids = np.asarray(table_row[:n], np.int64)
    kc, ks, vc, vs = granule_views(pages[ids] if n else pages[:0], page_size, D)
    got = []
    for c, s, g in ((kc, ks, k_g), (vc, vs, v_g)):
        P, H = c.shape[:2]
        val = o.e2m1_decode(o.unpack_codes(c.reshape(-1, D // 2))).astype(np.float64).reshape(P, H, page_size, D)
        sc = o.e4m3_decode(s.reshape(-1)).astype(np.float64).reshape(P, H, page_size, D // 16)
        x = float(np.float32(g)) * np.repeat(sc, 16, -1) * val
        got.append(x.transpose(1, 0, 2, 3).reshape(x.shape[1], P * page_size, D)[:, :length])
    return got


def attention(q, pages, table, cu, kv_len, k_g, v_g, page_size, scale, causal, window, drop=()):
    """out, lse in FP64 and what a tolerance needs: `mass` = sum p |v|, `reach` = the largest scale * sum |q||k| of a
    visible token, `seen` = visible tokens, `big` = largest |v|. drop: (sequence, table index) of pages to leave out."""
    T, HQ, D = q.shape
    H = pages.shape[1]
    group = HQ // H
    out = np.zeros((T, HQ, D))
    lse = np.full((T, HQ), -np.inf)
    mass, reach = np.zeros((T, HQ, D)), np.zeros((T, HQ))
    seen, big = np.zeros((T, HQ)), np.zeros((T, HQ))
    for b in range(len(kv_len)):
        n, L = int(cu[b + 1] - cu[b]), int(kv_len[b])
        if n == 0 or L == 0:
            continue
        K, V = gather(pages, [max(0, min(int(p), pages.shape[0] - 1)) for p in table[b]], L, page_size, D, k_g, v_g)
        j = np.arange(L)
        kept = np.ones(L, bool)
        for bb, page in drop:
            if bb == b:
                kept[page * page_size:(page + 1) * page_size] = False
        for i in range(n):
            pos = L - n + i
            see = kept.copy()
            if causal:
                see &= j <= pos
            if window:
                see &= pos - j < window
            if not see.any():
                continue
            for h in range(HQ):
                k, v = K[h // group][see], V[h // group][see]
                x = q[cu[b] + i, h].astype(np.float64)
                s = scale * (k @ x)
                m = s.max()
                p = np.exp(s - m)
                t = cu[b] + i
                out[t, h] = p @ v / p.sum()
                lse[t, h] = m + np.log(p.sum())
                mass[t, h] = p @ np.abs(v) / p.sum()
                reach[t, h] = scale * (np.abs(k) @ np.abs(x)).max()
                seen[t, h] = see.sum()
                big[t, h] = np.abs(v).max()
    return dict(out=out, lse=lse, mass=mass, reach=reach, seen=seen, big=big)


def attention_tolerance(ref, D):
    """Bounds of |out - ref| and |lse - ref| from the roundings made, first order, added up at their worst.

    A score's error: D products of exact FP16 operands summed in FP32, in any order, (D + 8) half steps of 2^-24 of
    `reach` (the query's own FP16 rounding, 2^-29 of its row's largest, is far inside 8 of them for D <= 128: D * 2^-29
    <= 4 * 2^-24), then two factors and the difference s - m at 2^-24 each of at most 2 * reach; the 2^x function 2^-22.
    A weight p is rounded to FP16: 2^-11 of itself, or 2^-25 absolutely below 2^-14, with the largest p at least 2^7 in
    the running scale: 2^-32 of it. The sums over tokens add (seen + 64) * 2^-24, the output is rounded to BF16: 2^-8 (half of
    eps = 2^-7)."""
    e_s = (D + 16) * 2.0 ** -24 * ref["reach"] + 2.0 ** -21
    e_sum = (ref["seen"] + 64) * 2.0 ** -24
    rel = 2 * e_s + 2.0 ** -11 + 2 * e_sum
    out = 2.0 ** -8 * np.abs(ref["out"]) + rel[..., None] * ref["mass"] * (1 + 2.0 ** -8) \
        + (ref["seen"] * ref["big"] * 2.0 ** -32)[..., None]
    lse = e_s + e_sum + 2.0 ** -22 * (np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0)) + ref["reach"] + 1)
    return out, lse


# ------------------------------------------------------------------ page pool
def held(length, page_size):
    return -(-int(length) // page_size)


def fork(refs, table, seq_len, parent, child, page_size):
    """In place; returns (src, dst, status): status 0, 9 (entries refused) or 10 (too few pages, nothing changed)."""
    n, status = len(parent), 0
    plan, named = [], set()
    start = [int(x) for x in seq_len]
    for a, c in zip(parent, child):
        ok = 0 <= a < len(start) and 0 <= c < len(start) and a != c and start[c] == 0 and c not in named
        if ok:
            named.add(c)
        else:
            status = 9
        plan.append(ok)
    free = [p for p in range(len(refs)) if refs[p] == 0]
    need = sum(1 for i in range(n) if plan[i] and start[parent[i]] % page_size)
    if need > len(free):
        return [-2] * n, [-2] * n, 10
    src, dst = [], []
    for i in range(n):
        if not plan[i]:
            src.append(-2), dst.append(-2)
            continue
        a, c, L = parent[i], child[i], start[parent[i]]
        full = L // page_size
        for j in range(full):
            table[c][j] = table[a][j]
            refs[table[a][j]] += 1
        if L % page_size:
            p = free.pop(0)
            refs[p] = 1
            src.append(int(table[a][full])), dst.append(p)
            table[c][full] = p
        else:
            src.append(-1), dst.append(-1)
        seq_len[c] = L
    return src, dst, status


def free(refs, table, seq_len, which, page_size):
    for s in which:
        for j in range(held(seq_len[s], page_size)):
            refs[table[s][j]] -= 1
            table[s][j] = -1
        seq_len[s] = 0


def compact(refs, table, seq_len, page_size):
    """New (refs, table) and the moves."""
    used = [p for p in range(len(refs)) if refs[p] > 0]
    L = len(used)
    src = [p for p in used if p >= L]
    dst = [p for p in range(L) if refs[p] <= 0]
    to = dict(zip(src, dst))
    new_refs = np.zeros_like(refs)
    for p in used:
        new_refs[to.get(p, p)] = refs[p]
    new_table = table.copy()
    for s in range(len(seq_len)):
        for j in range(held(seq_len[s], page_size)):
            new_table[s][j] = to.get(int(table[s][j]), int(table[s][j]))
    return new_refs, new_table, src, dst, L
