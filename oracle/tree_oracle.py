"""Oracle for tree speculation: a plain, slow CPU restatement in fp64 of the block operators for a
tree of drafted tokens.

TEST INFRASTRUCTURE, under the same rule as vfy_oracle.py: the CUDA library shares no code with it and
the product path never calls it.

Readings:
  * Node 0 of a sequence's block is the last committed token; node j > 0 is a drafted token whose
    parent is a node with a lower index, or -1 for a node that continues the prefix itself. Node j's
    K/V row sits at position p0 + j (p0 = L - q); its token sits at p0 + depth_j.
  * A node attends every position before the block (in a window layer those from p0 + depth - W + 1
    on) and the block rows of its mask: by a plan, itself and its ancestors.
  * Acceptance walks from node 0 to the child (lowest index first) whose drafted token is the argmax
    of the node's row, until there is none.
  * Logit rules, in this order: repetition penalty on tokens seen in the prompt, generated, or
    drafted on the row's path; frequency and presence penalties on generated and drafted ones;
    biases; grammar mask.
"""
from __future__ import annotations

import math

import numpy as np

from .vfy_oracle import CHUNK_TOKENS, argmax_row, bf16_to_f64

PROMPT_BIT = 1 << 31


def ancestors(parents):
    """Per node, the set of the node and its ancestors."""
    sets = []
    for i, p in enumerate(parents):
        sets.append({i} | (sets[p] if p >= 0 else set()))
    return sets


def depths(parents):
    return [len(s) - 1 for s in ancestors(parents)]


def mask_words(sets, words: int = 8) -> np.ndarray:
    """Row masks as uint32 [nodes][words]."""
    out = np.zeros((len(sets), words), dtype=np.uint32)
    for i, s in enumerate(sets):
        for j in s:
            out[i, j // 32] |= np.uint32(1 << (j % 32))
    return out


def _attend(q, group, keys, values, see, scale):
    """Attention of q [n][Hq][d] over keys [Hkv][N][d] where see [n][N]. Returns O, LSE and
    sum_j p_j |v_j| (what the rounding of P and of partial rows is relative to)."""
    n, hq, d = q.shape
    out, mag = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse = np.full((n, hq), -math.inf)
    some = see.any(axis=1)
    for g in range(hq):
        h = g // group
        s = np.where(see, scale * (q[:, g] @ keys[h].T), -math.inf)
        m = np.where(some, s.max(axis=1, initial=-math.inf), 0.0)
        w = np.exp(s - m[:, None])
        z = np.where(some, w.sum(axis=1), 1.0)
        w /= z[:, None]
        out[:, g], mag[:, g] = w @ values[h], w @ np.abs(values[h])
        lse[some, g] = (m + np.log(z))[some]
    return out, lse, mag


def attend_tree_full_seq(q, sets, k_pool, v_pool, resident_ids, resident_slots, seq_len: int, scale=None):
    """One sequence of a full layer; `sets`: per node, the block rows it attends."""
    q = bf16_to_f64(q)
    n, hq, d = q.shape
    hkv = k_pool.shape[1]
    p0 = seq_len - n
    ids = np.asarray(resident_ids, dtype=np.int64)
    slots = np.asarray(resident_slots, dtype=np.int64)
    pos = (ids[:, None] * CHUNK_TOKENS + np.arange(CHUNK_TOKENS)).reshape(-1)
    keep = pos < seq_len
    pos = pos[keep]
    kk = bf16_to_f64(k_pool[slots]).transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, keep]
    vv = bf16_to_f64(v_pool[slots]).transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, keep]
    see = np.zeros((n, pos.size), dtype=bool)
    for i in range(n):
        see[i] = (pos < p0) | np.isin(pos, [p0 + j for j in sets[i] if j < n])
    return _attend(q, hq // hkv, kk, vv, see, 1.0 / math.sqrt(d) if scale is None else scale)


def attend_tree_ring_seq(q, sets, depth, k_ring, v_ring, phi: int, seq_len: int, window: int, scale=None):
    """One sequence of a window layer, read from its ring [Hkv][R][d]."""
    q = bf16_to_f64(q)
    n, hq, d = q.shape
    hkv, ring_len, _ = k_ring.shape
    p0 = seq_len - n
    pos = np.arange(max(0, p0 - window + 1), seq_len)
    slots = (pos + phi) % ring_len
    see = np.zeros((n, pos.size), dtype=bool)
    for i in range(n):
        see[i] = (pos < p0) & (pos >= p0 + depth[i] - window + 1)
        see[i] |= np.isin(pos, [p0 + j for j in sets[i] if j < n])
    return _attend(q, hq // hkv, bf16_to_f64(k_ring[:, slots]), bf16_to_f64(v_ring[:, slots]), see,
                   1.0 / math.sqrt(d) if scale is None else scale)


def process_row(row, *, counts=None, path_tokens=(), repetition=1.0, frequency=0.0, presence=0.0, bias=(), allowed=None):
    """One row of logits in fp64. counts: uint32 [vocab] (bit 31: in the prompt); path_tokens: the
    drafted tokens on the row's path; bias: [(token, value)]; allowed: bool [vocab] or None.
    Returns (row, magnitude of the terms)."""
    x = np.asarray(row, dtype=np.float64).copy()
    mag = np.zeros_like(x)
    if counts is not None:
        counts = np.asarray(counts, dtype=np.uint32).astype(np.int64)
        made = (counts & (PROMPT_BIT - 1)).astype(np.float64)
        for t in path_tokens:
            made[t] += 1
        seen = (counts != 0) | (made > 0)
        up = seen & (x > 0)
        down = seen & ~(x > 0)
        x[up] /= float(repetition)
        x[down] *= float(repetition)
        mag = np.abs(x) + abs(float(frequency)) * made + abs(float(presence)) * (made > 0)
        x = x - float(frequency) * made - float(presence) * (made > 0)
    add = np.zeros_like(x)
    for t, v in bias:
        add[t] += float(v)
        mag[t] += abs(float(v))
    x = x + add
    mag = mag + np.abs(x)
    if allowed is not None:
        x[~np.asarray(allowed, dtype=bool)] = -math.inf
    return x, mag


def count_tokens(counts, tokens, as_prompt: bool):
    """counts uint32 [vocab] after `tokens` (-1 skipped)."""
    counts = np.array(counts, dtype=np.uint32, copy=True)
    for t in tokens:
        if t < 0:
            continue
        if as_prompt:
            counts[t] |= np.uint32(PROMPT_BIT)
        else:
            counts[t] += np.uint32(1)
    return counts


def accept_tree_seq(logits, drafts, parents):
    """One sequence: logits [n][V], drafts [n - 1], parents [n] -> (accepted, path, bonus,
    committed), path and committed padded with -1 to n."""
    n = len(parents)
    target = [argmax_row(r) for r in logits]
    node, path = 0, [0]
    while True:
        nxt = [c for c in range(node + 1, n) if parents[c] == node and int(drafts[c - 1]) == target[node]]
        if not nxt:
            break
        node = nxt[0]
        path.append(node)
    k = len(path) - 1
    committed = [int(drafts[c - 1]) for c in path[1:]] + [target[node]] + [-1] * (n - k - 1)
    return k, path + [-1] * (n - k - 1), target[node], committed


def compact_ring(path, accepted, cu_q, seq_len, ring_offset, ring):
    """The accepted path's rows of one ring [B][Hkv][R][d] at their new places."""
    out = np.array(ring, copy=True)
    r = ring.shape[2]
    for b in range(len(cu_q) - 1):
        a = int(cu_q[b])
        p0 = int(seq_len[b]) - (int(cu_q[b + 1]) - a)
        for j in range(1, int(accepted[b]) + 1):
            out[b, :, (p0 + j + int(ring_offset[b])) % r] = ring[b, :, (p0 + int(path[a + j]) + int(ring_offset[b])) % r]
    return out


def compact_full(path, accepted, cu_q, seq_len, cu_chunks, slot_of_chunk, store, pool):
    """The same for one full layer's chunk store and pool. Returns new (store, pool)."""
    new_store, new_pool = np.array(store, copy=True), np.array(pool, copy=True)
    for b in range(len(cu_q) - 1):
        a = int(cu_q[b])
        p0 = int(seq_len[b]) - (int(cu_q[b + 1]) - a)
        for j in range(1, int(accepted[b]) + 1):
            src, dst = p0 + int(path[a + j]), p0 + j
            if src == dst:
                continue
            cs, cd = int(cu_chunks[b]) + src // CHUNK_TOKENS, int(cu_chunks[b]) + dst // CHUNK_TOKENS
            ss, sd = int(slot_of_chunk[cs]), int(slot_of_chunk[cd])
            resident = 0 <= ss < pool.shape[0]
            row = pool[ss, :, src % CHUNK_TOKENS] if resident else store[cs, :, src % CHUNK_TOKENS]
            new_store[cd, :, dst % CHUNK_TOKENS] = row
            if 0 <= sd < pool.shape[0]:
                new_pool[sd, :, dst % CHUNK_TOKENS] = row
    return new_store, new_pool
