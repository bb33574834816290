"""Float64 definitions of the operators for decode steps over long contexts: attention of
groups of decode queries over shared keys, means of written pages, block scores and the
choice of blocks.

They have no counterpart on the pages; each function states its operator's formula
plainly, a group, page or row at a time.
"""
from __future__ import annotations

import numpy as np


def attend_ref(q: np.ndarray, keys: np.ndarray, seen=None) -> tuple[np.ndarray, np.ndarray]:
    """``q [n, 16, 576]`` over ``keys [L, 576]`` (values their first 512 dims): outputs
    ``[n, 16, 512]`` and natural log-sum-exps ``[n, 16]``.  Query i sees the first ``seen[i]``
    keys (all without it)."""
    n = q.shape[0]
    out, lse = np.zeros((n, 16, 512)), np.full((n, 16), -np.inf)
    for i in range(n):
        k = keys if seen is None else keys[:max(0, seen[i])]
        if len(k) == 0:
            continue
        s = q[i] @ k.T / 24.0
        top = s.max(axis=1, keepdims=True)
        p = np.exp(s - top)
        z = p.sum(axis=1, keepdims=True)
        out[i] = p @ k[:, :512] / z
        lse[i] = (top + np.log(z))[:, 0]
    return out, lse


def shared_ref(q, values, qo_indptr, kv_indptr, kv_indices=None):
    """Groups of query tokens over their groups' keys, ``values [rows, 576]`` the cache."""
    out, lse = np.full((len(q), 16, 512), np.nan), np.full((len(q), 16), np.nan)
    for g in range(len(qo_indptr) - 1):
        a, b = int(qo_indptr[g]), int(qo_indptr[g + 1])
        j = np.arange(kv_indptr[g], kv_indptr[g + 1])
        rows = j if kv_indices is None else np.asarray(kv_indices)[j]
        out[a:b], lse[a:b] = attend_ref(q[a:b], values[rows])
    return out, lse


def written_pages(slots, page_size: int) -> list[tuple[int, int]]:
    """(page, rows that it holds) for every slot that ends its page."""
    ends = []
    for t, s in enumerate(slots):
        after = slots[t + 1] if t + 1 < len(slots) else -1
        if s >= 0 and (after != s + 1 or (s + 1) % page_size == 0):
            ends.append((int(s) // page_size, int(s) % page_size + 1))
    return ends


def block_means_ref(values, slots, means, page_size: int) -> np.ndarray:
    """``means [pages, 576]`` with those of the pages that ``slots`` wrote to renewed."""
    means = np.array(means, dtype=np.float64)
    for page, rows in written_pages(slots, page_size):
        means[page] = values[page * page_size:page * page_size + rows].sum(axis=0) / rows
    return means


def block_scores_ref(q, means, block_table, qo_indptr, kv_indptr, page_size: int) -> np.ndarray:
    """The highest product of each row's queries with each of its pages' means, over 24."""
    scores = np.full(np.shape(block_table), -np.inf)
    for b in range(len(kv_indptr) - 1):
        rows = q[int(qo_indptr[b]):int(qo_indptr[b + 1])].reshape(-1, 576)
        for j in range(-(-int(kv_indptr[b + 1] - kv_indptr[b]) // page_size)):
            if len(rows):
                scores[b, j] = (rows @ means[block_table[b][j]]).max() / 24.0
    return scores


def block_select_ref(scores, block_table, kv_indptr, page_size: int, blocks: int, sink: int, recent: int) -> dict:
    """Chosen pages, and the tokens on them as a page table (valid steps only)."""
    indptr, indices, chosen = [0], [], np.full((len(kv_indptr) - 1, blocks), -1, dtype=np.int64)
    for b in range(len(kv_indptr) - 1):
        tokens = int(kv_indptr[b + 1] - kv_indptr[b])
        pages = -(-tokens // page_size)
        taken = list(range(pages))
        if pages > blocks:
            fixed = set(range(sink)) | set(range(pages - recent, pages))
            rank = sorted((j for j in taken if j not in fixed),
                          key=lambda j: (not np.isnan(scores[b][j]), -np.nan_to_num(scores[b][j], nan=0.0), j))
            taken = sorted(fixed | set(rank[:blocks - len(fixed)]))
        chosen[b, :len(taken)] = taken
        for j in taken:
            first = int(block_table[b][j]) * page_size
            indices += range(first, first + min(page_size, tokens - j * page_size))
        indptr.append(len(indices))
    return {"indptr": np.array(indptr), "indices": np.array(indices, dtype=np.int64), "chosen": chosen}
