"""Float64 definitions of the operators around the decode step: page maps, cache
appends, prompt attention in the expanded form and the merge of its pieces.

They have no counterpart on the pages, whose harness hands the page table, the
filled cache and the absorbed query over ready made; each function states its
operator's formula plainly, a row or token at a time.
"""
from __future__ import annotations

import numpy as np

from .fp8 import E4M3_MAX


def page_map_ref(kv_lens, new_lens, block_table, free_pages, page_size: int) -> dict:
    """Tables and maps of one step as the loops of its definition (valid steps only)."""
    table = np.array(block_table, dtype=np.int64)
    qo, kv, indices, slots, positions = [0], [0], [], [], []
    used = 0
    for b, (n0, add) in enumerate(zip(kv_lens, new_lens)):
        total = int(n0) + int(add)
        for page in range(-(-int(n0) // page_size), -(-total // page_size)):
            table[b, page] = free_pages[used]
            used += 1
        cells = [int(table[b, j // page_size]) * page_size + j % page_size for j in range(total)]
        indices += cells
        slots += cells[int(n0):]
        positions += range(int(n0), total)
        qo.append(qo[-1] + int(add))
        kv.append(kv[-1] + total)
    return {"table": table, "qo_indptr": np.array(qo), "kv_indptr": np.array(kv),
            "kv_indices": np.array(indices, dtype=np.int64), "slots": np.array(slots, dtype=np.int64),
            "positions": np.array(positions, dtype=np.int64), "pages_used": used}


def rotate_ref(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """Rotation of the 32 pairs of ``x [..., 64]`` by angles given as cos and sin ``[..., 32]``."""
    out = np.empty(x.shape, dtype=np.float64)
    for i in range(32):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        a, b, c, s = x[..., p], x[..., q], cos[..., i], sin[..., i]
        out[..., p] = a * c - b * s
        out[..., q] = b * c + a * s
    return out


def kv_row_ref(kv: np.ndarray, weight: np.ndarray, eps: float, cos, sin, interleaved: bool) -> np.ndarray:
    """Normalised latent and rotated key of each token: float64 ``[T, 576]``."""
    c = kv[:, :512]
    rms = np.sqrt(np.mean(c * c, axis=1, keepdims=True) + eps)
    return np.concatenate([c / rms * weight, rotate_ref(kv[:, 512:], cos, sin, interleaved)], axis=1)


def e4m3_target(row: np.ndarray, scale: float) -> np.ndarray:
    """What the e4m3 codes of a cache row approximate: ``clamp(row / scale, -448, 448)``."""
    return np.clip(row / scale, -E4M3_MAX, E4M3_MAX)


def prefill_ref(q, k_nope, k_rope, v, qo_indptr, kv_indptr, scale: float, causal: bool):
    """``(out [Tq, H, 128], lse [Tq, H], reach [Tq, H, 128], spread [Tq, H])``.

    ``reach`` is the attention-weighted mean of ``|v|`` and ``spread`` the largest
    ``scale * sum |q||k|`` over a query's keys: what rounding errors of the
    probabilities and of the scores are relative to."""
    tq, heads = q.shape[:2]
    out, reach = np.zeros((tq, heads, v.shape[2])), np.zeros((tq, heads, v.shape[2]))
    lse, spread = np.full((tq, heads), -np.inf), np.zeros((tq, heads))
    for b in range(len(qo_indptr) - 1):
        q0, q1, k0, k1 = (int(x) for x in (*qo_indptr[b:b + 2], *kv_indptr[b:b + 2]))
        n, length = q1 - q0, k1 - k0
        if n == 0 or length == 0:
            continue
        sees = np.arange(length)[None, :] < ((length - n + 1 + np.arange(n))[:, None] if causal
                                             else np.full((n, 1), length))
        some = sees.any(axis=1)
        for h in range(heads):
            key = np.concatenate([k_nope[k0:k1, h], k_rope[k0:k1]], axis=1)
            s = np.where(sees, scale * (q[q0:q1, h] @ key.T), -np.inf)
            size = np.where(sees, scale * (np.abs(q[q0:q1, h]) @ np.abs(key).T), 0.0)
            top = np.where(some, s.max(axis=1), 0.0)
            p = np.exp(s - top[:, None])
            total = np.where(some, p.sum(axis=1), 1.0)
            out[q0:q1, h] = (p @ v[k0:k1, h]) / total[:, None]
            reach[q0:q1, h] = (p @ np.abs(v[k0:k1, h])) / total[:, None]
            lse[q0:q1, h] = np.where(some, top + np.log(total), -np.inf)
            spread[q0:q1, h] = size.max(axis=1)
    return out, lse, reach, spread


def merge_ref(parts, lses):
    """``(out, lse, reach)`` of pieces ``[S, ..., dim]`` with log-sum-exps ``[S, ...]``;
    ``reach`` is the weighted mean of the pieces' magnitudes."""
    lses = np.asarray(lses, dtype=np.float64)
    top = lses.max(axis=0)
    top = np.where(np.isneginf(top), 0.0, top)
    w = np.exp(lses - top)
    total = w.sum(axis=0)
    seen = total > 0
    safe = np.where(seen, total, 1.0)
    parts = np.where((w > 0)[..., None], np.asarray(parts, dtype=np.float64), 0.0)
    out = (w[..., None] * parts).sum(axis=0) / safe[..., None]
    reach = (w[..., None] * np.abs(parts)).sum(axis=0) / safe[..., None]
    return out, np.where(seen, top + np.log(safe), -np.inf), reach
