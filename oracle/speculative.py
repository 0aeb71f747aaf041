"""CPU oracle of the speculative decode step's operators -- TEST INFRASTRUCTURE ONLY.

Plain numpy loops in fp64, written from the formulas in include/focr_moe.h and sharing no code with
the CUDA path.  The quantiser is the C oracle's (``oracle.quantize_rows``).
"""
from __future__ import annotations

import math

import numpy as np

import oracle

D, RING = 128, 128


def qk_norm_rope(x, pos, gamma=None, eps=1e-6, theta=10000.0, rot=128, interleaved=False, norm=False):
    """x [T, heads, 128] -> fp64."""
    y = np.array(x, np.float64)
    T, heads, _ = y.shape
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        if gamma is not None:
            y = y * np.asarray(gamma, np.float64)
    out = y.copy()
    for t in range(T):
        for i in range(rot // 2):
            ang = float(pos[t]) * theta ** (-2.0 * i / rot)
            c, s = math.cos(ang), math.sin(ang)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
    return out


def quantise(x, int4: bool):
    """Rows [..., 128] -> (codes as the cache stores them, scales [...])."""
    shape = x.shape[:-1]
    q, s = oracle.quantize_rows(np.ascontiguousarray(x, np.float32).reshape(-1, D), D, 4 if int4 else 8)
    if int4:
        return oracle.nibble_pack(q).reshape(*shape, D // 2), s.reshape(shape)
    return q.reshape(*shape, D), s.reshape(shape)


def values(codes, scales):
    """The fp64 values a cache's rows stand for (exact: a code times a scale)."""
    if codes.dtype == np.uint8:
        lo, hi = (codes & 15).astype(np.int64), (codes >> 4).astype(np.int64)
        q = np.stack((lo, hi), -1).reshape(*codes.shape[:-1], D)
        q = np.where(q > 7, q - 16, q)
    else:
        q = codes.astype(np.int64)
    return q * scales[..., None].astype(np.float64)


def kv_write(cache, k, v, count, start, row0=None, index=None, n_max=None, wrap=False):
    """In place on cache = [k, k_scale, v, v_scale] (numpy)."""
    B, heads, cap = cache[1].shape
    int4 = cache[0].dtype == np.uint8
    for b in range(B):
        n, s0 = int(count[b]), int(start[b])
        if n < 0 or n > n_max or s0 < 0 or (not wrap and s0 + n > cap):
            continue
        for i in range(n):   # in order: a later token overwrites an earlier one in its slot
            r = (b * n_max if row0 is None else int(row0[b])) + (i if index is None else int(index[b][i]))
            slot = (s0 + i) % cap
            last = not any((s0 + j) % cap == slot for j in range(i + 1, n)) if n > cap else True
            if r < 0 or r >= k.shape[0] or not last:
                continue
            for h in range(heads):
                for x, c, s in ((k, cache[0], cache[1]), (v, cache[2], cache[3])):
                    q, sc = quantise(x[r, h][None], int4)
                    c[b, h, slot], s[b, h, slot] = q[0], sc[0]


def tree_lines(parent):
    """Per node: the node and its ancestors, and its depth."""
    lines = []
    for i in range(len(parent)):
        line, j = [], i
        while j >= 0:
            line.append(j)
            j = int(parent[j])
        lines.append(line)
    return lines


def rswa_tree(q, k_new, v_new, ref, ref_len, ring, n_gen, parent=None, n_nodes=None):
    """ref, ring: (k values, v values) fp64 [B, heads, cap, 128].  Returns fp64 [B, N, heads_q, 128]; rows of nodes
    >= n_nodes are NaN."""
    B, N, hq, _ = q.shape
    hk = k_new.shape[2]
    out = np.full(q.shape, np.nan)
    for b in range(B):
        R, n = int(ref_len[b]), int(n_gen[b])
        L = N if n_nodes is None else int(n_nodes[b])
        lines = tree_lines(range(-1, L - 1) if parent is None else parent[b][:L])
        for i in range(L):
            pos = n + len(lines[i]) - 1
            toks = [t for t in range(max(0, n - RING), n) if t > pos - RING]
            slots = [t % RING for t in toks]
            for h in range(hk):
                kk = np.concatenate((ref[0][b, h, :R], ring[0][b, h, slots], k_new[b, lines[i], h].astype(np.float64)))
                vv = np.concatenate((ref[1][b, h, :R], ring[1][b, h, slots], v_new[b, lines[i], h].astype(np.float64)))
                for x in range(h * (hq // hk), (h + 1) * (hq // hk)):
                    s = kk @ q[b, i, x].astype(np.float64) / math.sqrt(D)
                    w = np.exp(s - s.max())
                    out[b, i, x] = w @ vv / w.sum()
    return out


def token_probs(logits, temperature=1.0):
    x = np.asarray(logits, np.float64) / float(np.float32(temperature))
    e = np.exp(x - x.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def spec_verify(target, draft, tokens, parent, n_nodes, u):
    """The recursion as it is usually written: after a rejection the target becomes its normalised residual."""
    B, N = tokens.shape
    n_acc, path, nxt = np.zeros(B, np.int32), np.full((B, N), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        L = N if n_nodes is None else int(n_nodes[b])
        cur, taken = -1, []
        P = target[b, 0].astype(np.float64)
        mass = 1.0
        for i in range(L):
            if (i - 1 if parent is None else int(parent[b][i])) != cur:
                continue
            x = int(tokens[b, i])
            q = None if draft is None else draft[b, cur + 1].astype(np.float64)
            if float(u[b, i]) * (1.0 if q is None else q[x]) * (mass if q is None else 1.0) < P[x]:
                cur = i
                taken.append(i)
                P, mass = target[b, i + 1].astype(np.float64), 1.0
            elif q is None:
                mass -= P[x]
                P[x] = 0.0
            else:
                P = np.maximum(P - q, 0.0)
                if P.sum() > 0.0:
                    P = P / P.sum()
        if not P.sum() > 0.0:
            P = target[b, cur + 1].astype(np.float64)
        c = np.cumsum(P)
        hit = np.nonzero((c > float(u[b, N]) * c[-1]) & (P > 0))[0]
        live = np.nonzero(P > 0)[0]
        nxt[b] = hit[0] if len(hit) else (live[-1] if len(live) else P.size - 1)
        n_acc[b] = len(taken)
        path[b, :len(taken)] = taken
    return n_acc, path, nxt
