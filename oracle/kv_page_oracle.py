"""Paged Q3 KV cache, CPU oracle -- TEST INFRASTRUCTURE, not part of the product
(the rules of hlwq_oracle apply).  numpy in fp64, one request, token and head at
a time, on top of kv_oracle's vector encoding.

Of a request's N tokens the last min(N, R) are exact (token i in ring slot
i % R, reading K5 with any R, 0 included), the max(0, N - R) before them are
encoded, P tokens to a page.
"""

from __future__ import annotations

import numpy as np

from .hlwq_oracle import _as_f64, sylvester_hadamard
from .kv_oracle import HEAD_DIM, kv_dequantize, kv_quantize

_H = sylvester_hadamard(HEAD_DIM).astype(np.float64)


def kv_encoded(n: int, R: int) -> int:
    """Encoded tokens among n."""
    return max(0, n - R)


def kv_pages(n: int, P: int, R: int) -> int:
    return -(-kv_encoded(n, R) // P)


def kv_block_tables(n_past, n_new, free, table, P: int, R: int, T: int):
    """(table, cu_new, slot_map, n_free) after one step; free = the stack of
    free pages, last entry first; a page that is not to be had is -1."""
    free = list(free)
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    cu, slots = [0], []
    for b, (p, n) in enumerate(zip(n_past, n_new)):
        for k in range(min(kv_pages(p, P, R), width), min(kv_pages(p + n, P, R), width)):
            table[b, k] = free.pop() if free else -1
        for j in range(n):
            i = p + j - R
            page = -1 if i < 0 or i // P >= width else int(table[b, i // P])
            slots.append(-1 if page < 0 else page * P + i % P)
        cu.append(cu[-1] + n)
    slots = (slots + [-1] * T)[:T]
    return table, np.array(cu), np.array(slots), len(free)


def kv_paged_append(X, slots, cu, n_past, packed, norms, window, R: int):
    """Keys or values X [T][H][256] into (packed [pages][H][P][96], norms float16
    [pages][H][P], window [B][H][R][256]): the new arrays."""
    x = _as_f64(X)
    packed, norms, window = packed.copy(), norms.copy(), window.copy()
    P = packed.shape[2]
    for b, p in enumerate(n_past):
        c0, n = cu[b], cu[b + 1] - cu[b]
        if n == 0:
            continue
        old = range(max(0, p - R), p)
        for h in range(x.shape[1]):
            tokens = {i: window[b, h, i % R] for i in old}
            tokens.update({p + j: x[c0 + j, h] for j in range(n)})
            leave = range(max(0, p - R), kv_encoded(p + n, R))
            if len(leave):
                q = kv_quantize(np.stack([tokens[i] for i in leave]))
                for r, i in enumerate(leave):
                    s = slots[c0 + i + R - p]
                    if s >= 0:
                        packed[s // P, h, s % P] = q["packed"][r]
                        norms[s // P, h, s % P] = q["norms"][r]
            for i in range(max(p, p + n - R), p + n):
                window[b, h, i % R] = tokens[i]
    return packed, norms, window


def _vectors(packed, norms, window, table, b, h, N, R):
    """The N cached vectors of request b, head h, as attention reads them."""
    P, e = packed.shape[2], kv_encoded(N, R)
    i = np.arange(e)
    page = table[b, i // P]
    v = kv_dequantize(packed[page, h, i % P], norms[page, h, i % P]) if e else np.zeros((0, HEAD_DIM))
    w = np.arange(e, N)
    return np.concatenate([v, window[b, h, w % R]]) if N > e else v


def kv_paged_attention(Q, cu, n_past, table, k, v, R: int, scale: float, half_step: float = 2.0 ** -11):
    """(out [T][Hq][256], tol [T][Hq]) in fp64; k, v = (packed, norms, window).

    tol bounds the error's 2-norm for an evaluation in the rotated domain with
    operands rounded to binary16 (relative half step u = 2^-11), fp32 sums and
    one rounding to bf16.  With q~ = q H, k~ = k H:
      - a product q~_d k~_d carries two roundings, each uniform in +-u: the
        score's variance is scale^2 (2 u^2 / 3) sum_d (q~_d k~_d / 256)^2;
      - score errors e_j move o by sum_j p_j e_j (v_j - o): standard deviation
        below s = (sum_j p_j^2 var_j |v_j - o|^2)^(1/2);
      - p_j and the coordinates of v~_j are rounded, and p_j's exponential and
        the sums are in fp32: 2 u per term, independent over j, plus
        2 u |o| for what is common to all terms;
      - the output is off by half a bf16 step, 2^-8 |o|.
    Six standard deviations of the random parts are allowed."""
    q = _as_f64(Q)
    T, Hq = q.shape[0], q.shape[1]
    H = k[0].shape[1]
    G = Hq // H
    u = half_step
    out, tol = np.zeros((T, Hq, HEAD_DIM)), np.zeros((T, Hq))
    for b, p in enumerate(n_past):
        c0, n = cu[b], cu[b + 1] - cu[b]
        if n == 0:
            continue
        for h in range(H):
            K = _vectors(*k, table, b, h, p + n, R)
            V = _vectors(*v, table, b, h, p + n, R)
            Kr = (K @ _H) / HEAD_DIM
            for j in range(n):
                m = p + j + 1
                for g in range(h * G, (h + 1) * G):
                    x = q[c0 + j, g]
                    s = scale * (K[:m] @ x)
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    o = w @ V[:m]
                    var = scale ** 2 * (2 * u * u / 3) * ((Kr[:m] * (x @ _H)) ** 2).sum(1)
                    spread = np.sqrt((w ** 2 * var * ((V[:m] - o) ** 2).sum(1)).sum())
                    terms = np.sqrt((w ** 2 * (V[:m] ** 2).sum(1)).sum())
                    size = np.linalg.norm(o)
                    out[c0 + j, g] = o
                    tol[c0 + j, g] = 2.0 ** -8 * size + 2 * u * size + 6 * (spread + 2 * u * terms)
    return out, tol


__all__ = ["kv_encoded", "kv_pages", "kv_block_tables", "kv_paged_append", "kv_paged_attention"]
