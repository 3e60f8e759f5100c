"""Pins of the tree oracle (oracle/tree_oracle.py): against the chain oracle, dense masks, closed forms
and hand-worked cases. No GPU."""
import math

import numpy as np
import pytest

from oracle import tree_oracle as T
from oracle import vfy_oracle as O
from speculative_decode_verify_attn_gb300 import synth


def test_ancestors_hand_case():
    #        0
    #      1   2
    #     3 4   5
    #           6
    parents = [-1, 0, 0, 1, 1, 2, 5]
    assert T.ancestors(parents) == [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {0, 1, 4}, {0, 2, 5}, {0, 2, 5, 6}]
    assert T.depths(parents) == [0, 1, 1, 2, 2, 2, 3]
    w = T.mask_words(T.ancestors(parents))
    assert w[:, 0].tolist() == [1, 3, 5, 11, 19, 37, 101] and not w[:, 1:].any()


def test_mask_words_past_the_first_word():
    w = T.mask_words([{0, 31, 32, 255}])
    assert w[0].tolist() == [(1 << 31) | 1, 1, 0, 0, 0, 0, 0, 1 << 31]


def test_random_trees_are_in_order():
    rng = np.random.default_rng(0)
    for n in (1, 2, 17, 64, 256):
        p = synth.random_tree(rng, n)
        assert len(p) == n and p[0] == -1 and all(0 <= p[i] < i for i in range(1, n))


@pytest.mark.parametrize("nq", [1, 5, 17])
def test_a_chain_is_the_linear_block(nq):
    rng = np.random.default_rng(nq)
    L, hq, hkv, d, chunks = 150, 4, 2, 64, 3
    q = synth.normal_bf16(rng, (nq, hq, d))
    k, v = synth.normal_bf16(rng, (4, hkv, 64, d)), synth.normal_bf16(rng, (4, hkv, 64, d))
    ids, slots = np.arange(chunks), np.array([2, 0, 3])
    sets = T.ancestors(list(range(-1, nq - 1)))
    o, lse, _ = T.attend_tree_full_seq(q, sets, k, v, ids, slots, L)
    ro, rl = O.attend_full_seq(q, k, v, ids, slots, L)
    assert np.allclose(o, ro, atol=1e-13) and np.allclose(lse, rl, atol=1e-13)
    ring_k, ring_v = synth.normal_bf16(rng, (hkv, 128, d)), synth.normal_bf16(rng, (hkv, 128, d))
    o, lse, _ = T.attend_tree_ring_seq(q, sets, T.depths(list(range(-1, nq - 1))), ring_k, ring_v, 77, L, 48)
    ro, rl = O.attend_ring_seq(q, ring_k, ring_v, 77, L, 48)
    assert np.allclose(o, ro, atol=1e-13) and np.allclose(lse, rl, atol=1e-13)


def test_each_path_of_a_tree_is_a_chain_of_its_own():
    """A node's output equals the last row of the linear block made of its path alone."""
    rng = np.random.default_rng(3)
    parents = [-1, 0, 0, 1, 2, 2, 4]
    n, p0, d, hkv, hq = len(parents), 70, 64, 1, 2
    q = synth.normal_bf16(rng, (n, hq, d))
    k, v = synth.normal_bf16(rng, (2, hkv, 64, d)), synth.normal_bf16(rng, (2, hkv, 64, d))
    sets, depth = T.ancestors(parents), T.depths(parents)
    o, lse, _ = T.attend_tree_full_seq(q, sets, k, v, [0, 1], [1, 0], p0 + n)
    rk = np.zeros((hkv, 256, d), np.uint16)
    rv = np.zeros_like(rk)
    for pos in range(p0 + n):
        rk[:, pos], rv[:, pos] = k[1 - pos // 64, :, pos % 64], v[1 - pos // 64, :, pos % 64]
    wo, wl, _ = T.attend_tree_ring_seq(q, sets, depth, rk, rv, 0, p0 + n, 20)
    for i in range(n):
        path = sorted(sets[i])
        flat_k, flat_v = rk.copy(), rv.copy()
        for at, node in enumerate(path):
            flat_k[:, p0 + at], flat_v[:, p0 + at] = rk[:, p0 + node], rv[:, p0 + node]
        L = p0 + len(path)
        ro, rl = O.attend_ring_seq(q[i][None], flat_k, flat_v, 0, L, 10 ** 6)
        assert np.allclose(o[i], ro[0], atol=1e-13) and np.allclose(lse[i], rl[0], atol=1e-13)
        ro, rl = O.attend_ring_seq(q[i][None], flat_k, flat_v, 0, L, 20)
        assert np.allclose(wo[i], ro[0], atol=1e-13) and np.allclose(wl[i], rl[0], atol=1e-13)


def test_a_row_that_attends_nothing():
    q = np.zeros((2, 1, 64), np.uint16)
    k = np.full((1, 1, 64, 64), 0x3F80, np.uint16)
    o, lse, _ = T.attend_tree_full_seq(q, [set(), {0, 1}], k, k, [0], [0], 2)
    assert not o[0].any() and lse[0, 0] == -math.inf
    assert np.allclose(o[1], 1.0) and np.isclose(lse[1, 0], math.log(2))


def test_rules_hand_case():
    row = [2.0, -2.0, 1.0, 0.5, math.inf, math.nan]
    counts = np.array([T.PROMPT_BIT, T.PROMPT_BIT | 2, 0, 3, 0, 0], np.uint32)
    x, _ = T.process_row(row, counts=counts, path_tokens=[2, 2, 3], repetition=2.0, frequency=0.5, presence=0.25,
                         bias=[(0, 1.0), (0, 0.5), (3, -1.0)])
    # 0: prompt only: 2/2 + 1.5; 1: -2*2 - 2*.5 - .25; 2: 1/2 - 2*.5 - .25; 3: .5/2 - 4*.5 - .25 - 1
    assert x[:5].tolist() == [2.5, -5.25, -0.75, -3.0, math.inf] and math.isnan(x[5])
    x, _ = T.process_row(row, allowed=[True, False, True, True, False, False])
    assert x.tolist() == [2.0, -math.inf, 1.0, 0.5, -math.inf, -math.inf]


def test_counts_hand_case():
    c = T.count_tokens(np.zeros(4, np.uint32), [1, 1, -1, 3], False)
    assert c.tolist() == [0, 2, 0, 1]
    c = T.count_tokens(c, [0, 1, 0], True)
    assert c.tolist() == [T.PROMPT_BIT, T.PROMPT_BIT | 2, 0, 1]


def _logits(targets, vocab=16):
    x = np.zeros((len(targets), vocab), np.float32)
    x[np.arange(len(targets)), targets] = 1.0
    return x


def test_accept_hand_cases():
    parents = [-1, 0, 0, 1, 1, 2]
    # target of each row: 0 -> 7, 1 -> 3, 2 -> 9, ...
    lg = _logits([7, 3, 9, 5, 6, 8])
    # node 2 drafts 7 (node 1 does not): path 0, 2, then node 5 drafts 9
    assert T.accept_tree_seq(lg, [4, 7, 3, 3, 9], parents) == (2, [0, 2, 5, -1, -1, -1], 8, [7, 9, 8, -1, -1, -1])
    # both children of 0 draft 7: the lower one is taken, and of its children the lower that drafts 3
    assert T.accept_tree_seq(lg, [7, 7, 2, 3, 9], parents) == (2, [0, 1, 4, -1, -1, -1], 6, [7, 3, 6, -1, -1, -1])
    # nothing matches: the target's own token
    assert T.accept_tree_seq(lg, [1, 1, 3, 3, 9], parents) == (0, [0, -1, -1, -1, -1, -1], 7, [7, -1, -1, -1, -1, -1])
    # a node whose parent is -1 is never reached
    assert T.accept_tree_seq(_logits([7, 7]), [7], [-1, -1]) == (0, [0, -1], 7, [7, -1])


def test_accepting_a_chain_is_the_linear_acceptance():
    rng = np.random.default_rng(5)
    for _ in range(20):
        n = int(rng.integers(1, 9))
        targets = rng.integers(0, 16, n)
        drafts = np.where(rng.random(n - 1) < 0.7, targets[:-1], 15 - targets[:-1])
        k, path, bonus, committed = T.accept_tree_seq(_logits(targets), drafts, list(range(-1, n - 1)))
        rn, rb, rc = O.accept_seq(_logits(targets), drafts)
        assert (k, bonus, committed) == (rn, rb, rc) and path[:k + 1] == list(range(k + 1))


def test_compaction_hand_case():
    """p0 = 62, path 0, 2, 3: rows at 64 and 65 (chunk 1) move to 63 (chunk 0) and 64 (chunk 1). Chunk 1 is
    in slot 0, chunk 0 nowhere."""
    store = np.arange(2 * 64, dtype=np.uint16).reshape(2, 1, 64, 1)
    pool = store[1:] + 1000
    s, p = T.compact_full([0, 2, 3, -1], [2], [0, 4], [66], [0, 2], [-1, 0], store, pool)
    assert s[0, 0, 63, 0] == 1064 and s[1, 0, 0, 0] == 1065 and p[0, 0, 0, 0] == 1065
    changed = np.flatnonzero(s.reshape(-1) != store.reshape(-1))
    assert changed.tolist() == [63, 64] and np.flatnonzero(p.reshape(-1) != pool.reshape(-1)).tolist() == [0]
    ring = np.arange(8, dtype=np.uint16).reshape(1, 1, 8, 1)
    r = T.compact_ring([0, 2, 3, -1], [2], [0, 4], [66], [1], ring)          # slots of 62..65: 7, 0, 1, 2
    assert r.reshape(-1).tolist() == [1, 2, 2, 3, 4, 5, 6, 7]
