"""fp64 statements of the prompt and draft operators, in plain numpy.

They share no code with the CUDA path. Sources: "Gemma 4 E2B on a 4 GB GPU with
pure PyTorch" - the prompt-read paragraph (chunks of a prompt attend to the cache
and themselves), the decode-attention and cache paragraphs (grouped query heads,
full caches, rings that record positions, windows) and Step 2 (logits from the
tied embedding), for several tokens at once.
"""
from __future__ import annotations

import numpy as np


def attend(q, k, v, keep, scale):
    """(out, absout) fp64 [rows][D] of q [rows][D] over k, v [T][D] where keep
    [rows][T]; a row that keeps nothing gives zeros. absout = sum_t w_t |v_t|. What a
    row does not keep is not looked at."""
    q = np.asarray(q, np.float64)
    out = np.zeros(q.shape)
    absout = np.zeros(q.shape)
    for i in range(q.shape[0]):
        t = np.flatnonzero(keep[i])
        if t.size == 0:
            continue
        kk, vv = np.asarray(k[t], np.float64), np.asarray(v[t], np.float64)
        with np.errstate(invalid="ignore", over="ignore"):
            s = scale * (kk @ q[i])
            w = np.exp(s - s.max())
            w = w / w.sum()
            out[i] = w @ vv
            absout[i] = w @ np.abs(vv)
    return out, absout


def attn_prompt(q, k, v, cu_q, cu_k, window, scale):
    """(out, absout) fp64 [total_q][Hq][D]; rows of no sequence are NaN in out."""
    Sq, Hq, D = q.shape
    Hkv = k.shape[1]
    out, ab = np.full((Sq, Hq, D), np.nan), np.zeros((Sq, Hq, D))
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        lq, lk = q1 - q0, k1 - k0
        p = np.arange(lq)[:, None] + lk - lq
        t = np.arange(lk)[None, :]
        keep = t <= p
        if window:
            keep &= t > p - window
        for h in range(Hq):
            g = h // (Hq // Hkv)
            out[q0:q1, h], ab[q0:q1, h] = attend(q[q0:q1, h], k[k0:k1, g], v[k0:k1, g], keep, scale)
    return out, ab


def tree_chain(parents, i):
    """Node i, its parent, and so on; [] for an absent node."""
    if parents[i] == -2:
        return []
    chain = [i]
    while True:
        p = int(parents[chain[-1]])
        if p < 0 or p >= chain[-1]:
            return chain
        chain.append(p)


def tree_keep(parents, pos, kpos, T, window):
    """bool [N][T + N]: what each node keeps of the cache and of the tree."""
    N = len(parents)
    pos = max(int(pos), 0)
    slot = np.arange(T, dtype=np.int64) if kpos is None else np.asarray(kpos, np.int64)
    keep = np.zeros((N, T + N), bool)
    for i in range(N):
        chain = tree_chain(parents, i)
        if not chain:
            continue
        at = pos + len(chain) - 1
        low = at - window if window else -1
        keep[i, :T] = (slot >= 0) & (slot < pos) & (slot > low)
        for d, j in enumerate(chain):
            keep[i, T + j] = at - d > low
    return keep


def attn_tree(q, k, v, k_tree, v_tree, parents, pos, kpos, window, scale):
    """(out, absout) fp64 [B][N][Hq][D]."""
    B, N, Hq, D = q.shape
    T, Hkv = k.shape[1], k.shape[2]
    out, ab = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        keep = tree_keep(parents[b], pos[b], None if kpos is None else kpos[b], T, window)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            kk = np.concatenate([k[b, :, g], k_tree[b, :, g]])
            vv = np.concatenate([v[b, :, g], v_tree[b, :, g]])
            out[b, :, h], ab[b, :, h] = attend(q[b, :, h], kk, vv, keep, scale)
    return out, ab


def logprobs(x, targets, topk):
    """(logprob, entropy, top_logprob, top_id, status) of fp32 rows x [M][V]."""
    x = np.asarray(x, np.float64)
    M, V = x.shape
    lp, ent = np.zeros(M), np.zeros(M)
    top, ids = np.full((M, topk), -np.inf), np.full((M, topk), -1, np.int64)
    status = 0
    for m in range(M):
        r = x[m]
        t = None if targets is None else int(targets[m])
        if t is not None and not 0 <= t < V:
            status, t = 1, None
        n = min(topk, V)
        order = np.lexsort((np.arange(V), -(r + 0.0)))[:n]
        if np.isnan(r).any() or (r == np.inf).any():
            lp[m] = 0.0 if t is None else np.nan
            ent[m] = np.nan
            top[m] = np.nan
            continue
        ids[m, :n] = order
        f = r[np.isfinite(r)]
        if f.size == 0:
            lp[m] = 0.0 if t is None else -np.inf
            continue
        lse = f.max() + np.log(np.exp(f - f.max()).sum())
        p = np.exp(f - lse)
        ent[m] = -(p * (f - lse)).sum()
        top[m, :n] = r[order] - lse
        if t is not None:
            lp[m] = r[t] - lse
    return lp, ent, top, ids, status


def kv_commit(k_cache, v_cache, kpos, k_tree, v_tree, path, count, pos):
    """(k_cache', v_cache', kpos', status) of caches [L][B][T][W]."""
    kc, vc = np.array(k_cache), np.array(v_cache)
    kp = None if kpos is None else np.array(kpos)
    L, B, T, W = kc.shape
    N = k_tree.shape[2]
    status = 0
    for b in range(B):
        for j in range(min(max(int(count[b]), 0), N)):
            node, p = int(path[b][j]), int(pos[b]) + j
            if not 0 <= node < N or p < 0 or p > 2 ** 31 - 1 or (kp is None and p >= T):
                status = 1
                continue
            s = p % T if kp is not None else p
            kc[:, b, s], vc[:, b, s] = k_tree[:, b, node], v_tree[:, b, node]
            if kp is not None:
                kp[b, s] = p
    return kc, vc, kp, status
