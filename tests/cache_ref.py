"""Plain references for the cache calls, in 64 bits or whole numbers: the page
formats decoded from their definitions, attention row by row, quantisers by
search over every code, and the page operations one row at a time."""
import math

import numpy as np
import torch

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
                 for e in range(16) for m in range(8)])
E4M3[127] = np.nan


def decode_fp4(cache, heads, ps, D):
    """uint8 [P, heads * ps * (D/2 + D/16)] -> float64 [P, heads, ps, D]."""
    c = cache.reshape(cache.shape[0], heads, -1)
    codes = c[..., :ps * D // 2].reshape(-1, heads, ps, D // 2)
    scales = c[..., ps * D // 2:].reshape(-1, heads, ps, D // 16)
    nib = np.stack((codes & 15, codes >> 4), -1).reshape(-1, heads, ps, D)
    val = np.where(nib >= 8, -1.0, 1.0) * E2M1[nib & 7]
    sc = np.where(scales >= 128, -1.0, 1.0) * E4M3[scales & 127]
    return val * np.repeat(sc, 16, -1)


def nearest(table, x):
    """Index of the table value nearest to each x >= 0 (ties to the even index),
    saturating: every midpoint compared in exact arithmetic (float64)."""
    mids = (table[1:] + table[:-1]) / 2
    i = np.searchsorted(mids, x, side="left")       # x == mid stays at the lower index
    tie = (i < len(mids)) & (mids[np.minimum(i, len(mids) - 1)] == x)
    return np.where(tie & (i % 2 == 1), i + 1, i)


def quantise_fp4(x):
    """float64 [..., D] -> (packed codes [..., D/2], scale bytes [..., D/16], values)."""
    b = x.reshape(*x.shape[:-1], -1, 16)
    sc = nearest(E4M3[:127], np.abs(b).max(-1) / 6)
    sc = np.maximum(sc, 1)
    s = E4M3[sc][..., None]
    code = nearest(E2M1, np.abs(b) / s)
    val = np.sign(b) * E2M1[code] * s
    code = np.where((b < 0) & (code > 0), code + 8, code).reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), sc.astype(np.uint8), val.reshape(x.shape)


def quantise_fp8(x):
    """float64 [T, D] -> (code bytes, scales, values)."""
    most = np.abs(x).max(-1)
    s = np.ones_like(most)
    for i, m in enumerate(most):
        if m > 0:
            e = -126
            while m / 2.0 ** e > 448:
                e += 1
            s[i] = 2.0 ** e
    code = nearest(E4M3[:127], np.abs(x) / s[:, None])
    val = np.sign(x) * E4M3[code] * s[:, None]
    neg = np.signbit(x)
    return np.where(neg, code + 128, code).astype(np.uint8), s, val


def token_rows(ctx, offsets, T, per_row=None):
    """(row, position) of each new token, (-1, -1) where it has none."""
    out = []
    for t in range(T):
        if offsets is None:
            b = t // per_row
            out.append((b, ctx[b] - ((b + 1) * per_row - t)))
            continue
        b = max((r for r in range(len(ctx)) if offsets[r] <= t < offsets[r + 1]), default=-1)
        out.append((b, ctx[b] - (offsets[b + 1] - t)) if b >= 0 else (-1, -1))
    return out


def attention(q, k_cache, v_cache, table, ctx, *, heads_kv, ps, scale, indices=None):
    """float64 (out, lse, A, e) for CPU tensors: A = sum p |v| / sum p, the size that
    rounded weights act on; e bounds a score's error from fp32 accumulation:
    scale * max_t sum_d |q k| * 2^-16 (D <= 128 terms of 2^-23 each)."""
    B, nn, H, D = q.shape
    G = H // heads_kv
    K = decode_fp4(k_cache.numpy(), heads_kv, ps, D)
    V = decode_fp4(v_cache.numpy(), heads_kv, ps, D)
    qd = q.double().numpy()
    out, A = np.zeros((B, nn, H, D)), np.zeros((B, nn, H, D))
    lse, err = np.full((B, nn, H), -np.inf), np.zeros((B, nn, H))
    P = k_cache.shape[0]
    for b in range(B):
        c = int(min(max(int(ctx[b]), 0), table.shape[1] * ps))
        for n in range(nn):
            upto = min(max(c - nn + 1 + n, 0), c)
            t = np.arange(upto)
            if indices is not None:
                t = indices[b, n].numpy()
                t = t[(t >= 0) & (t < upto)]
            if not len(t):
                continue
            page = np.clip(table[b].numpy()[t // ps], 0, P - 1)
            for h in range(H):
                k, v = K[page, h // G, t % ps], V[page, h // G, t % ps]
                s = scale * (k @ qd[b, n, h])
                p = np.exp(s - s.max())
                lse[b, n, h] = s.max() + math.log(p.sum())
                p /= p.sum()
                out[b, n, h] = p @ v
                A[b, n, h] = p @ np.abs(v)
                err[b, n, h] = abs(scale) * (np.abs(k) @ np.abs(qd[b, n, h])).max() * 2.0 ** -16
    return out, lse, A, err


def check_attention(got, lse, ref, T, dtype):
    """got against the reference within the roundings that the kernel makes:
    the result to its type (half a step, eps / 2 of |o|); p to f16 (2^-11 of each p,
    2^-25 for those below f16's normal range, where the largest p is at least 1), each
    moving o by p's share of |v - o| <= |v| + |o|; the scores by `err` and exp2's and
    the sums' roundings by 2^-19 together."""
    out, rlse, A, err = ref
    got = got.double().cpu().numpy()
    e = err[..., None] + 2.0 ** -11 + 2.0 ** -19
    big = np.abs(out).max() + A.max()
    bound = torch.finfo(dtype).eps / 2 * np.abs(out) + 2 * e * A + 2 * T * 2.0 ** -25 * big + \
        torch.finfo(dtype).tiny
    bad = ~(np.abs(got - out) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], out[bad][:4], bound[bad][:4])
    if lse is not None:
        lse = lse.double().cpu().numpy()
        fin = np.isfinite(rlse)
        assert np.array_equal(np.isneginf(lse), ~fin)
        # fp32 sums of up to T terms, log2 and the products around it
        tol = err + (T + 64) * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(np.where(fin, rlse, 0)))
        assert (np.abs(lse[fin] - rlse[fin]) <= tol[fin]).all()


def fork(table, lens, parents, refs, ps):
    B, W = table.shape
    P = len(refs)
    cap = W * ps
    ln = np.clip(lens, 0, cap)
    out, olen, refs = np.full((len(parents), W), -1, np.int32), np.zeros(len(parents), np.int32), refs.copy()
    for b in range(B):
        for j in range(-(-int(ln[b]) // ps)):
            if 0 <= table[b, j] < P:
                refs[table[b, j]] -= 1
    for r, p in enumerate(parents):
        if not 0 <= p < B:
            continue
        olen[r] = ln[p]
        for j in range(-(-int(ln[p]) // ps)):
            out[r, j] = table[p, j]
            if 0 <= table[p, j] < P:
                refs[table[p, j]] += 1
    return out, olen, refs


def resize(table, lens, new, refs, ps):
    """(table, lens, refs, src, dst, ran_out), one row after the other."""
    table, refs = table.copy(), refs.copy()
    B, W = table.shape
    P = len(refs)
    old, new = np.clip(lens, 0, W * ps), np.clip(new, 0, W * ps)
    free = [p for p in range(P) if refs[p] == 0]
    src, dst = np.full(B, -1, np.int32), np.full(B, -1, np.int32)
    wanted, ran_out, got = 0, False, np.array(old, np.int32)
    shared = []
    for b in range(B):
        had = -(-int(old[b]) // ps)
        end = table[b, had - 1] if had else -1
        shared.append(bool(new[b] > old[b] and old[b] % ps and 0 <= end < P and refs[end] > 1))
    drop = []
    for b in range(B):
        had, has = -(-int(old[b]) // ps), -(-int(new[b]) // ps)
        need = (has - had if new[b] > old[b] else 0) + shared[b]
        wanted += need
        if need and wanted > len(free):
            ran_out = True
            continue
        mine = free[wanted - need:wanted]
        got[b] = new[b]
        if shared[b]:
            src[b], dst[b] = table[b, had - 1], mine[0]
            drop.append(src[b])
            table[b, had - 1] = mine[0]
            refs[mine[0]] = 1
            mine = mine[1:]
        if new[b] > old[b]:
            for j, p in zip(range(had, has), mine):
                table[b, j] = p
                refs[p] = 1
        else:
            for j in range(has, had):
                if 0 <= table[b, j] < P:
                    drop.append(table[b, j])
                table[b, j] = -1
    for p in drop:
        refs[p] -= 1
    return table, got, refs, src, dst, ran_out


def compact(table, lens, refs, ps):
    table, P = table.copy(), len(refs)
    live = [p for p in range(P) if refs[p] > 0]
    n = len(live)
    src = [p for p in live if p >= n]
    dst = [p for p in range(n) if refs[p] <= 0]
    page_map = np.full(P, -1, np.int32)
    for p in live:
        page_map[p] = p
    for s, d in zip(src, dst):
        page_map[s] = d
    out = np.array(refs)
    for s, d in zip(src, dst):
        out[d], out[s] = refs[s], 0
    ln = np.clip(lens, 0, table.shape[1] * ps)
    for b in range(table.shape[0]):
        for j in range(-(-int(ln[b]) // ps)):
            if 0 <= table[b, j] < P:
                table[b, j] = page_map[table[b, j]]
    pad = [-1] * (P // 2 - len(src))
    return table, out, np.array(src + pad, np.int32), np.array(dst + pad, np.int32), len(src), page_map
