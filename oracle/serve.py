"""fp64 statements of the operators that serve several requests at once, in plain numpy.

They share no code with the CUDA path. Sources: "Gemma 4 E2B on a 4 GB GPU with pure
PyTorch" - the decode-attention, cache and prompt-read paragraphs, for several requests
whose caches share one pool of pages, with low-rank adapters beside the projections.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .draft import attend


def norm(x, weight, eps):
    """x [..., D] over its root mean square, times weight; x itself without a weight."""
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


_TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256")
_BITS = 160


def angle(pos, inv_freq):
    """pos [M] * inv_freq [h] (fp32) without its whole turns, from -pi to pi. A frequency is a whole number of
    2^-160 turns (off by half of one), so whole turns of its multiples drop out exactly."""
    one = 1 << _BITS
    f = np.array([round(Fraction(float(x)) * one / _TWO_PI) for x in np.asarray(inv_freq, np.float32)], object)
    t = np.array([int(p) for p in np.asarray(pos)], object)[:, None] * f[None, :]
    t = (t + one // 2) % one - one // 2
    return 2 * np.pi * (t / one).astype(np.float64)


def turn(u, pos, inv_freq, pairs):
    """(turned, size) of heads u [M][H][D] at positions pos [M]: size = |a| + |b| of the
    pair that an element belongs to, |u| where it is not turned."""
    u = np.asarray(u, np.float64)
    out, size = u.copy(), np.abs(u)
    if inv_freq is None or len(inv_freq) == 0:
        return out, size
    h = len(inv_freq)
    t = angle(pos, inv_freq)
    c, s = np.cos(t)[:, None], np.sin(t)[:, None]
    i = np.arange(h) * (2 if pairs else 1)
    j = i + (1 if pairs else h)
    a, b = u[..., i], u[..., j]
    out[..., i], out[..., j] = a * c - b * s, b * c + a * s
    size[..., i] = size[..., j] = np.abs(a) + np.abs(b)
    return out, size


def rows_of(cu_q, lens, M):
    """(sequence, position) of each of M rows; sequence -1 for a row of none."""
    seq, pos = np.full(M, -1), np.zeros(M, np.int64)
    B = len(lens)
    for b in range(B):
        q0, q1 = (b, b + 1) if cu_q is None else (int(cu_q[b]), min(int(cu_q[b + 1]), M))
        for m in range(q0, q1):
            seq[m], pos[m] = b, max(int(lens[b]), 0) - q1 + m
    return seq, pos


def place(table, pages, page, b, p):
    """(page, row) of sequence b's position p, or None where it has none."""
    if p < 0 or p >= table.shape[1] * page:
        return None
    g = int(table[b, p // page])
    return (g, p % page) if 0 <= g < pages else None


def attn_paged(q, k_pages, v_pages, table, lens, cu_q, window, scale):
    """(out, absout) fp64 [M][Hq][D]; rows of no sequence are NaN in out. k_pages, v_pages
    [pages][page][Hkv][D]."""
    M, Hq, D = q.shape
    pages, page, Hkv, _ = k_pages.shape
    out, ab = np.full((M, Hq, D), np.nan), np.zeros((M, Hq, D))
    seq, pos = rows_of(cu_q, lens, M)
    for b in range(len(lens)):
        rows = np.flatnonzero(seq == b)
        if rows.size == 0:
            continue
        at = [place(table, pages, page, b, t) for t in range(min(max(int(lens[b]), 0), table.shape[1] * page))]
        have = np.array([a is not None for a in at], bool)
        g = np.array([a[0] if a else 0 for a in at], np.int64)
        r = np.array([a[1] if a else 0 for a in at], np.int64)
        t = np.arange(len(at))
        keep = have[None, :] & (t[None, :] <= pos[rows][:, None])
        if window:
            keep &= t[None, :] > pos[rows][:, None] - window
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            out[rows, h], ab[rows, h] = attend(q[rows, h], k_pages[g, r, kv], v_pages[g, r, kv], keep, scale)
    return out, ab


def lora(y, x, a, b, ids, scale):
    """(out, size) fp64 [M][N]: size bounds what is added up, |y| + |scale| sum_r |b| sum_k |a x|;
    third: |scale| sum_r |b| |h|, fourth: status."""
    y, x = np.asarray(y, np.float64), np.asarray(x, np.float64)
    out, size, low = y.copy(), np.abs(y), np.zeros(y.shape)
    status = 0
    for m, i in enumerate(int(v) for v in ids):
        if i >= len(a):
            status = 1
        if not 0 <= i < len(a):
            continue
        s = 1.0 if scale is None else float(scale[i])
        aa, bb = np.asarray(a[i], np.float64), np.asarray(b[i], np.float64)
        h = aa @ x[m]
        out[m] += s * (bb @ h)
        size[m] += abs(s) * (np.abs(bb) @ (np.abs(aa) @ np.abs(x[m])))
        low[m] = abs(s) * (np.abs(bb) @ np.abs(h))
    return out, size, low, status
