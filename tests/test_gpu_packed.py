"""4-bit chunks: the append bit for bit, chunks read back, paging, and attention against fp64.

Attention is compared within 2^-8 |o| (O's rounding to bf16) + (2^-10 + 7e-4) A, A = sum_j p_j |v_j|: weights are rounded to
fp16 at most (half a step, 2^-11, and the next power of two's), scores are fp32 sums of d products of exact values. Codes and
scales are read exactly. fp16's smallest step is 2^-24: a weight is off by at most half of that, 2^-25, where the largest is at
least 2^7 (the reference lies 7 below a maximum, in log2), so that O may be off by 2^-32 sum_j |v_j| more; it shows only in
channels where the heavy keys' values are 0. LSE: 3.1e-4 + 2^-22 |lse|, the scores' part alone."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import vfy_oracle as O
from speculative_decode_verify_attn_gb300 import synth

pytestmark = pytest.mark.gpu

C = 64


@pytest.fixture(scope="module")
def env():
    import __graft_entry__
    __graft_entry__.build()
    from speculative_decode_verify_attn_gb300 import harness, vfy
    torch.cuda.set_device(0)
    return harness, vfy


def u8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def records(rng, n, hkv, d, low=0x20, high=0x39):
    """Random records: any codes, scales of 1/8 .. 1."""
    r = rng.integers(0, 256, (n, hkv, 36 * d)).astype(np.uint8)
    r[..., 32 * d:] = rng.integers(low, high, (n, hkv, 4 * d))
    return r


# ---------------------------------------------------------------------------------------------
# Append, paging, reading back
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("hkv,d", [(4, 128), (1, 64), (3, 64), (8, 128)])
@pytest.mark.parametrize("gk,gv", [(1.0, 1.0), (0.037, 3.0)])
@pytest.mark.parametrize("pinned", [False, True])
def test_append(env, hkv, d, gk, gv, pinned):
    """Codes and scales of every row, in the store and (where resident) the pool; all other bytes stay. The last tokens
    have no chunk and are reported."""
    H, vfy = env
    rng = np.random.default_rng([hkv, d, pinned, int(gk * 1000)])
    counts, lens, chunks = [37, 1, 0, 5], [150, 1, 0, 66], [3, 1, 0, 1]
    T = sum(counts)
    k, v = [rng.standard_normal((T, hkv, d)) * np.exp(rng.uniform(-9, 5, (T, hkv, 1))) for _ in range(2)]
    k[0], v[1, 0, :16] = 0.0, 0.0                               # groups of zeros
    k[2, 0, :16] = 1e-12                                        # a scale that rounds to 0
    k[3, 0, :16] = gk * np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6])   # ties (gk = 1)
    v[4, 0, :16] = 1e6                                          # past the largest scale
    k, v = O.bf16_to_f64(B.to_bf16(k)), O.bf16_to_f64(B.to_bf16(v))
    slot_of = np.array([-1, 3, 0, 2, 1], np.int32)
    store, pool = [records(rng, 5, hkv, d) for _ in range(2)], [records(rng, 4, hkv, d) for _ in range(2)]
    put = (lambda x: torch.from_numpy(x.copy()).pin_memory()) if pinned else u8   # noqa: E731
    sd, pd = [put(x) for x in store], [u8(x) for x in pool]
    cu_chunks = H.cu_from_counts(chunks)
    ctx = vfy.vfy_create(hkv, hkv, d, max_seqs=4, max_queries_per_seq=37, device=0)
    try:
        vfy.vfy_append_full_packed(ctx, H.dev_bf16(B.to_bf16(k)), H.dev_bf16(B.to_bf16(v)), H.dev_i32(H.cu_from_counts(counts)),
                                   H.dev_i32(lens), H.dev_i32(cu_chunks), H.dev_i32(slot_of), *sd, 5, *pd, 4, gk, gv, 4)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT   # position 64 and 65 of the last sequence
        t = 0
        for b, n in enumerate(counts):
            for i in range(n):
                p = lens[b] - n + i
                c = cu_chunks[b] + p // C
                if c < 5:
                    for side, (x, g) in enumerate(((k, gk), (v, gv))):
                        codes, scales = B.pack_rows(x[t], g)
                        for h in range(hkv):
                            B.write_row(store[side][c, h], p % C, codes[h], scales[h])
                            if slot_of[c] >= 0:
                                B.write_row(pool[side][slot_of[c], h], p % C, codes[h], scales[h])
                t += 1
        for got, want in zip(sd + pd, store + pool):
            assert np.array_equal(got.cpu().numpy(), want)
    finally:
        ctx.close()


def test_append_of_what_is_not_finite_gives_finite_values(env):
    H, vfy = env
    d = 64
    x = torch.ones((4, 1, d), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 3], x[1, 0, 3], x[2, 0, 3] = float("inf"), float("nan"), -float("inf")
    x[3, 0, :16] = float("nan")
    rec = [torch.zeros((1, 1, 36 * d), dtype=torch.uint8, device="cuda") for _ in range(4)]
    ctx = vfy.vfy_create(1, 1, d, max_seqs=1, max_queries_per_seq=4, device=0)
    try:
        vfy.vfy_append_full_packed(ctx, x, x, H.dev_i32([0, 4]), H.dev_i32([4]), H.dev_i32([0, 1]), H.dev_i32([0]), *rec[:2], 1,
                                   *rec[2:], 1, 1.0, 1.0, 1)
        got = B.record_values(rec[2].cpu().numpy()[0, 0], d)
        assert np.isfinite(got).all()
        codes, scales = B.pack_rows(np.ones(16, np.float32)[None].repeat(4, 1))    # the other groups are as ever
        assert np.array_equal(got[:4, 16:], np.repeat(np.abs(got[:1, 16:17]), 4, 0).repeat(48, 1))
        assert abs(got[0, 16] - 1) <= 2.0 ** -4
    finally:
        ctx.close()


@pytest.mark.parametrize("hkv,d", [(4, 128), (1, 64)])
@pytest.mark.parametrize("g", [1.0, 0.37])
def test_unpack(env, hkv, d, g):
    """Every code with every finite scale; slots in any order, twice, and out of range (left, reported)."""
    H, vfy = env
    rng = np.random.default_rng(d)
    pools = [records(rng, 9, hkv, d, 0, 127) for _ in range(2)]
    slots = [3, 8, -1, 0, 3, 9, 2 ** 31 - 1, 5]
    ctx = vfy.vfy_create(hkv, hkv, d, device=0)
    out = [torch.full((8, hkv, C, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    try:
        vfy.vfy_unpack_chunks(ctx, *map(u8, pools), 9, H.dev_i32(slots), 8, g, 2 * g, *out)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        for side in range(2):
            got = H.bits_of(out[side])
            for i, s in enumerate(slots):
                if not 0 <= s < 9:
                    assert (out[side][i] == 9).all()
                    continue
                ref = B.record_values(pools[side][s], d) * np.float32(g * (1 + side))
                if g == 1.0:
                    assert np.array_equal(O.bf16_to_f64(got[i]), ref)      # exact
                else:                                                      # one fp32 rounding of s g, one of the value
                    assert np.all(np.abs(O.bf16_to_f64(got[i]) - ref) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(ref))
        vfy.vfy_unpack_chunks(ctx, *map(u8, pools), 9, H.dev_i32([0]), 0, g, g, *out)      # none: nothing to do
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


@pytest.mark.parametrize("hkv,d", [(4, 128), (1, 64), (3, 64)])
@pytest.mark.parametrize("ctas", [0, 1, 4])
def test_page_in(env, hkv, d, ctas):
    H, vfy = env
    rng = np.random.default_rng([hkv, d])
    store, pool = [records(rng, 20, hkv, d) for _ in range(2)], [records(rng, 8, hkv, d) for _ in range(2)]
    pinned = [torch.from_numpy(x).pin_memory() for x in store]
    pd = [u8(x) for x in pool]
    plist = np.full((8, 2), -7, np.int32)
    plist[:3] = [[4, 1], [19, 0], [7, 3]]
    plist[4:6] = [[0, 7], [20, 5]]                              # the last is not in the store
    ctx = vfy.vfy_create(hkv, hkv, d, max_seqs=2, device=0)
    try:
        vfy.vfy_set_pagein_ctas(ctx, ctas)
        vfy.vfy_page_in_packed(ctx, *pinned, 20, *pd, 8, H.dev_i32(plist), H.dev_i32([3, 2]), 2, 4)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        for c, s in ((4, 1), (19, 0), (7, 3), (0, 7)):
            for side in range(2):
                pool[side][s] = store[side][c]
        for got, want in zip(pd, pool):
            assert np.array_equal(got.cpu().numpy(), want)
    finally:
        ctx.close()


# ---------------------------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------------------------

def close(got, lse, ref, rlse, mag, all_v):
    g = O.bf16_to_f64(got)
    off = np.abs(g - ref) - (2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 7e-4) * mag + 2.0 ** -32 * all_v + 1e-30)
    assert off.max(initial=-1) <= 0, (off.max(), np.abs(g - ref).max())
    fin = np.isfinite(rlse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(rlse))
    assert np.all(np.abs(lse[fin] - rlse[fin]) <= 3.1e-4 + np.abs(rlse[fin]) * 2.0 ** -22)


def attend(env, ctx, q, cu_q, pools, ids, slots, cu_res, lens, gk=1.0, gv=1.0, bound=None, with_lse=True):
    H, vfy = env
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda") if with_lse else None
    res = np.diff(cu_res).max() if bound is None else bound
    vfy.vfy_attend_full_packed(ctx, H.dev_bf16(q), H.dev_i32(cu_q), u8(pools[0]), u8(pools[1]), len(pools[0]), H.dev_i32(ids),
                               H.dev_i32(slots), H.dev_i32(cu_res), int(res), H.dev_i32(lens), gk, gv, out, lse, len(lens))
    return H.bits_of(out), None if lse is None else lse.cpu().numpy()


def one(env, heads, n, L, ids=None, splits=0, seed=0, gk=1.0, gv=1.0, spread=1.0, cap=None, scale=0.0):
    """One sequence of n rows and L tokens whose chunks `ids` (all) are resident."""
    H, vfy = env
    hq, hkv, d = heads
    rng = np.random.default_rng([hq, hkv, d, n, L, splits, seed])
    ids = np.arange(-(-L // C)) if ids is None else np.asarray(ids)
    m = max(1, len(ids))
    pools = [records(rng, m + 2, hkv, d) for _ in range(2)]
    slots = rng.permutation(m + 2)[:len(ids)]
    for e, c in enumerate(ids):                                 # what lies behind the last token may be anything
        for side in range(2):
            for t in range(max(0, L - c * C), C):
                pools[side][slots[e], :, 32 * d + t * (d // 16):32 * d + (t + 1) * (d // 16)] = 0x7F
    q = B.to_bf16(rng.standard_normal((n, hq, d)) * spread)
    ctx = vfy.vfy_create(hq, hkv, d, max_seqs=1, max_queries_per_seq=cap or n, softmax_scale=scale, device=0)
    try:
        vfy.vfy_set_splits(ctx, splits, 0)
        i, s = (ids, slots) if len(ids) else ([0], [0])
        got, lse = attend(env, ctx, q, [0, n], pools, i, s, [0, len(ids)], [L], gk, gv)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()
    ref = B.attend_packed_seq(O.bf16_to_f64(q), *pools, ids, slots, L, np.float32(gk), np.float32(gv), scale or None)
    close(got, lse, *ref)


HEADS = [(16, 4, 128), (4, 1, 64), (8, 8, 128), (8, 1, 64), (6, 2, 128), (16, 1, 128)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n", [1, 2, 5, 17, 33])
@pytest.mark.parametrize("extra", [0, 1, 47, 64, 300, 1000])
def test_sizes(env, heads, n, extra):
    one(env, heads, n, n + extra)


@pytest.mark.parametrize("heads", [(16, 4, 128), (4, 1, 64)])
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 16, 40, 64])
@pytest.mark.parametrize("n,L", [(17, 3000), (1, 2048), (17, 100), (4, 64)])
def test_splits(env, heads, splits, n, L):
    """Also more splits than chunks."""
    one(env, heads, n, L, splits=splits)


@pytest.mark.parametrize("heads", [(16, 4, 128), (4, 1, 64), (8, 8, 128), (32, 4, 128)])
@pytest.mark.parametrize("n", [64, 100, 256, 500])
def test_long_blocks(env, heads, n):
    one(env, heads, n, n + 130)


@pytest.mark.parametrize("heads", [(16, 4, 128), (8, 1, 64)])
def test_a_block_smaller_than_its_context(env, heads):
    """Contexts made for many rows, blocks of few."""
    for n, cap in ((1, 17), (3, 64), (17, 256)):
        one(env, heads, n, 700, cap=cap)


@pytest.mark.parametrize("ids", [[0, 3, 4, 9], [9], [8, 9], [0], [5, 0, 9, 2], []])
def test_chunks_that_are_not_resident(env, ids):
    """Any list of chunks in any order; rows that reach none of them give 0 and -inf (position 630 on is the block's)."""
    for splits in (0, 1, 3):
        one(env, (8, 2, 128), 10, 640, ids=ids, splits=splits)
        one(env, (4, 1, 64), 40, 610, ids=ids, splits=splits)    # rows 570 .. 609: chunks 8 and 9


@pytest.mark.parametrize("spread,gk,gv", [(1e-6, 1.0, 1.0), (40.0, 1.0, 1.0), (1e4, 1e-4, 1e4), (1e-30, 1.0, 1e-20), (1e30, 1e-30, 1e20),
                                          (1.0, 0.037, 5.0)])
def test_ranges(env, spread, gk, gv):
    """Queries and scales far from 1: nothing overflows on the way, weights down to the smallest keep their place."""
    one(env, (16, 4, 128), 17, 500, spread=spread, gk=gk, gv=gv)
    one(env, (4, 1, 64), 1, 500, spread=spread, gk=gk, gv=gv)


@pytest.mark.parametrize("splits", [0, 1])
def test_growing_scores(env, splits):
    """Every chunk's scores lie far above the one before (the running maximum moves in every tile), then far below."""
    H, vfy = env
    hq, hkv, d, n, L = 4, 1, 128, 9, 64 * 24
    rng = np.random.default_rng(1)
    pools = [records(rng, 24, hkv, d) for _ in range(2)]
    q = np.abs(rng.standard_normal((n, hq, d)))
    for order in (np.arange(24), np.arange(24)[::-1], rng.permutation(24)):
        for e in range(24):
            pools[0][e][..., :32 * d] = np.where(rng.random(32 * d) < 0.5, 0x22, 0x21)   # positive codes
            pools[0][e][..., 32 * d:] = 0x10 + 2 * order[e]
        bits = B.to_bf16(q)
        ctx = vfy.vfy_create(hq, hkv, d, max_queries_per_seq=n, device=0)
        try:
            vfy.vfy_set_splits(ctx, splits, 0)
            got, lse = attend(env, ctx, bits, [0, n], pools, np.arange(24), np.arange(24), [0, 24], [L])
        finally:
            ctx.close()
        ref = B.attend_packed_seq(O.bf16_to_f64(bits), *pools, np.arange(24), np.arange(24), L)
        # scores of up to 2000: 2^-22 of one is the fp32 sum's error, and that of a weight's exponent
        g = O.bf16_to_f64(got)
        assert np.all(np.abs(g - ref[0]) <= 2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -10 + 4e-3) * ref[2] + 2.0 ** -32 * ref[3])
        assert np.all(np.abs(lse - ref[1]) <= 3.1e-4 + 2.0 ** -20 * np.abs(ref[1]))


def test_a_far_tail_is_not_lost(env):
    """One key 17 nats above 32K others: the others' 1.4e-3 of the sum, each 4e-8 of the largest weight, is kept."""
    H, vfy = env
    d, m = 64, 512
    pools = [np.zeros((m, 1, 36 * d), np.uint8) for _ in range(2)]
    for p in pools:
        p[..., 32 * d:] = 0x38
    pools[0][100, 0, 5 * 16] = 0x07                             # token 5 of chunk 100: 6 in channel 0
    pools[1][..., :32 * d] = 0x22                               # V = 1 everywhere,
    pools[1][100, 0, 5 * 16] = 0x20                             # 0 in that token's channel 0
    q = np.zeros((1, 1, d))
    q[0, 0, 0] = 17 / 6
    bits = B.to_bf16(q)
    ref = B.attend_packed_seq(O.bf16_to_f64(bits), *pools, np.arange(m), np.arange(m), m * C, scale=1.0)
    ctx = vfy.vfy_create(1, 1, d, max_queries_per_seq=1, softmax_scale=1.0, device=0)
    try:
        for splits in (0, 1):
            vfy.vfy_set_splits(ctx, splits, 0)
            got, lse = attend(env, ctx, bits, [0, 1], pools, np.arange(m), np.arange(m), [0, m], [m * C])
            o = O.bf16_to_f64(got)[0, 0, 0]
            assert abs(o - ref[0][0, 0, 0]) <= 2.0 ** -8 * o + 1e-5 and 1.3e-3 < o < 1.6e-3
            assert abs(lse[0, 0] - ref[1][0, 0]) < 1e-5
    finally:
        ctx.close()


@pytest.mark.parametrize("heads", [(16, 4, 128), (4, 1, 64)])
def test_ragged_batches(env, heads):
    """Sequences of different blocks and lengths, an empty one and one that is too long among them; rows behind the last
    stay; the same bits from call to call and without the LSE."""
    H, vfy = env
    hq, hkv, d = heads
    rng = np.random.default_rng(hq)
    counts, lens = [17, 1, 0, 19, 8, 17], [1000, 1, 0, 700, 64, 3000]
    cu = H.cu_from_counts(counts)
    T = int(cu[-1])
    res = [-(-x // C) for x in lens]
    cu_res, total = H.cu_from_counts(res), sum(res)
    pools = [records(rng, total, hkv, d) for _ in range(2)]
    slots = rng.permutation(total)
    ids = np.concatenate([np.arange(r) for r in res])
    q = B.to_bf16(rng.standard_normal((T + 2, hq, d)))
    ctx = vfy.vfy_create(hq, hkv, d, max_seqs=6, max_queries_per_seq=17, device=0)
    try:
        got, lse = attend(env, ctx, q, cu, pools, ids, slots, cu_res, lens)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT   # 19 rows in a context for 17
        again, _ = attend(env, ctx, q, cu, pools, ids, slots, cu_res, lens, with_lse=False)
        assert np.array_equal(got, again)
        vfy.vfy_get_status(ctx)
        seven = B.to_bf16(np.float64(7.0))
        assert (got[T:] == seven).all() and (lse[T:] == 7).all()
        for b in range(6):
            at = slice(cu[b], cu[b + 1])
            if counts[b] == 19:
                assert (got[at] == seven).all() and (lse[at] == 7).all()
            elif counts[b]:
                e = slice(cu_res[b], cu_res[b + 1])
                close(got[at], lse[at], *B.attend_packed_seq(O.bf16_to_f64(q[at]), *pools, ids[e], slots[e], lens[b]))
    finally:
        ctx.close()


def test_bad_chunks_are_left_out_and_reported(env):
    H, vfy = env
    rng = np.random.default_rng(3)
    hq, hkv, d, n, L = 8, 2, 128, 17, 640
    pools = [records(rng, 10, hkv, d) for _ in range(2)]
    q = B.to_bf16(rng.standard_normal((n, hq, d)))
    ctx = vfy.vfy_create(hq, hkv, d, max_queries_per_seq=n, device=0)
    try:
        for splits in (0, 1, 5):
            vfy.vfy_set_splits(ctx, splits, 0)
            ids, slots = np.arange(10), np.array([3, -1, 5, 10, 2 ** 31 - 1, 0, -2 ** 31, 1, 9, 4])
            bad_id = ids.copy()
            bad_id[7] = -5
            got, lse = attend(env, ctx, q, [0, n], pools, bad_id, slots, [0, 10], [L])
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
            close(got, lse, *B.attend_packed_seq(O.bf16_to_f64(q), *pools, bad_id, slots, L))
            for cu, ln in (([-1, 16], [L]), ([0, n + 1], [L]), ([0, n], [n - 1]), ([2 ** 31 - 20, 2 ** 31 - 3], [L])):
                out = attend(env, ctx, q, cu, pools, ids, np.arange(10), [0, 10], ln)
                assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
                assert (out[0] == B.to_bf16(np.float64(7.0))).all() and (out[1] == 7).all()
    finally:
        ctx.close()


def test_the_last_chunk_id(env):
    """A sequence of 2^31 - 1 tokens whose last chunks alone are resident."""
    one(env, (4, 1, 128), 5, 2 ** 31 - 1, ids=[0, 2 ** 25 - 2, 2 ** 25 - 1])


def test_a_pool_past_4_gib(env):
    """Slots whose records lie past 2^32 bytes."""
    H, vfy = env
    hkv, d = 8, 128
    n_slots = (2 ** 32 + 2 ** 28) // (hkv * 36 * d)
    rng = np.random.default_rng(4)
    some = [records(rng, 3, hkv, d) for _ in range(2)]
    slots = [n_slots - 1, 0, n_slots - 2]
    pools = [torch.zeros((n_slots, hkv, 36 * d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for side in range(2):
        for e, s in enumerate(slots):
            pools[side][s] = u8(some[side][e])
    q = B.to_bf16(rng.standard_normal((4, hkv, d)))
    out, lse = torch.zeros((4, hkv, d), dtype=torch.bfloat16, device="cuda"), torch.zeros((4, hkv), device="cuda")
    ctx = vfy.vfy_create(hkv, hkv, d, max_queries_per_seq=4, device=0)
    try:
        vfy.vfy_attend_full_packed(ctx, H.dev_bf16(q), H.dev_i32([0, 4]), *pools, n_slots, H.dev_i32([0, 1, 2]), H.dev_i32(slots),
                                   H.dev_i32([0, 3]), 3, H.dev_i32([180]), 1.0, 1.0, out, lse, 1)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        close(H.bits_of(out), lse.cpu().numpy(), *B.attend_packed_seq(O.bf16_to_f64(q), *some, [0, 1, 2], [0, 1, 2], 180))
        back = [torch.zeros((1, hkv, C, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        vfy.vfy_unpack_chunks(ctx, *pools, n_slots, H.dev_i32([n_slots - 1]), 1, 1.0, 1.0, *back)
        assert np.array_equal(O.bf16_to_f64(H.bits_of(back[0])[0]), B.record_values(some[0][0], d))
    finally:
        ctx.close()
        del pools
        torch.cuda.empty_cache()


def test_refusals(env):
    H, vfy = env
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    rec = lambda: torch.zeros((4, 2, 36 * 64), dtype=torch.uint8, device="cuda")   # noqa: E731
    ctx = vfy.vfy_create(4, 2, 64, max_seqs=1, max_queries_per_seq=4, device=0)
    cu, ln, ids, res = H.dev_i32([0, 4]), H.dev_i32([9]), H.dev_i32([0, 1, 2, 3]), H.dev_i32([0, 1])
    q, k, lse = z(4, 4, 64), z(4, 2, 64), torch.zeros((4, 4), device="cuda")
    a, b = rec(), rec()
    nan, inf = float("nan"), float("inf")
    try:
        before = vfy.vfy_launch_count(ctx)
        calls = []
        for g in (0.0, -1.0, nan, inf):
            calls += [lambda g=g: vfy.vfy_attend_full_packed(ctx, q, cu, a, b, 4, ids, ids, res, 1, ln, g, 1.0, q, lse, 1),
                      lambda g=g: vfy.vfy_attend_full_packed(ctx, q, cu, a, b, 4, ids, ids, res, 1, ln, 1.0, g, q, lse, 1),
                      lambda g=g: vfy.vfy_append_full_packed(ctx, k, k, cu, ln, res, ids, a, b, 4, a, b, 4, g, 1.0, 1),
                      lambda g=g: vfy.vfy_unpack_chunks(ctx, a, b, 4, ids, 1, 1.0, g, k, k)]
        calls += [lambda: vfy.vfy_attend_full_packed(ctx, q, cu, a, b, 0, ids, ids, res, 1, ln, 1.0, 1.0, q, lse, 1),
                  lambda: vfy.vfy_attend_full_packed(ctx, q, cu, a, b, 4, ids, ids, res, -1, ln, 1.0, 1.0, q, lse, 1),
                  lambda: vfy.vfy_attend_full_packed(ctx, q, cu, a, b, 4, ids, ids, res, 1, ln, 1.0, 1.0, q, lse, 2),
                  lambda: vfy.vfy_attend_full_packed(ctx, q, cu, a.view(-1)[8:], b, 1, ids, ids, res, 1, ln, 1.0, 1.0, q, lse, 1),
                  lambda: vfy.vfy_append_full_packed(ctx, k, k, cu, ln, res, ids, a.cpu(), b.cpu(), 4, a, b, 4, 1.0, 1.0, 1),   # pageable
                  lambda: vfy.vfy_append_full_packed(ctx, k, k, cu, ln, res, ids, a, b, 0, a, b, 4, 1.0, 1.0, 1),
                  lambda: vfy.vfy_page_in_packed(ctx, a.cpu(), b.cpu(), 4, a, b, 4, ids, ids, 1, 2),
                  lambda: vfy.vfy_page_in_packed(ctx, a, b, 4, a, b, 4, ids, ids, 1, 0),
                  lambda: vfy.vfy_unpack_chunks(ctx, a, b, 4, ids, -1, 1.0, 1.0, k, k),
                  lambda: vfy.vfy_unpack_chunks(ctx, a, b, 4, None, 1, 1.0, 1.0, k, k)]
        for i, call in enumerate(calls):
            with pytest.raises(vfy.VfyError) as e:
                call()
            assert e.value.status == vfy.VFY_EINVAL, i
        with pytest.raises(TypeError):
            vfy.vfy_attend_full_packed(ctx, q, cu, k, b, 4, ids, ids, res, 1, ln, 1.0, 1.0, q, lse, 1)   # bf16 for bytes
        assert vfy.vfy_launch_count(ctx) == before and vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


def test_a_layer_from_projection_to_output_in_a_graph(env):
    """Selection, paging, rotation, append and attention over the 4-bit pool, captured once and replayed while the context
    grows: each replay against fp64 on the bytes that the pool then holds."""
    H, vfy = env
    hq, hkv, d, n, K = 8, 2, 128, 5, 4
    rng = np.random.default_rng(6)
    ctx = vfy.vfy_create(hq, hkv, d, max_seqs=1, max_queries_per_seq=n, device=0)
    m = 12
    host = [torch.from_numpy(records(rng, m, hkv, d)).pin_memory() for _ in range(2)]
    pool = [torch.zeros((K, hkv, 36 * d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    wide = torch.zeros((n, (hq + 2 * hkv) * d + 8), dtype=torch.bfloat16, device="cuda")
    qd, kd, vd = [wide[:, x * d:y * d].unflatten(1, (-1, d)) for x, y in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv))]
    rope = vfy.Rope(H.dev_f32((10000.0 ** (-np.arange(0, d, 2) / d)).astype(np.float32)))
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    q, k, out, lse = z(n, hq, d), z(n, hkv, d), z(n, hq, d), torch.zeros((n, hq), device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")    # noqa: E731
    cu, ln, cu_c = H.dev_i32([0, n]), H.dev_i32([300]), H.dev_i32([0, m])
    scores = torch.zeros(m, device="cuda")
    slot_of, ids, slots, cu_res, plist, pcount = H.dev_i32(np.full(m, -1)), i32(K), i32(K), i32(2), i32(K, 2), i32(1)

    def step():
        vfy.vfy_select_resident(ctx, scores, cu_c, 1, m, K, slot_of, ids, slots, cu_res, plist, pcount)
        vfy.vfy_page_in_packed(ctx, *host, m, *pool, K, plist, pcount, 1, K)
        vfy.vfy_rope(ctx, rope, qd, kd, cu, ln, None, q, k, 1)
        vfy.vfy_append_full_packed(ctx, k, vd.contiguous(), cu, ln, cu_c, slot_of, *host, m, *pool, K, 0.5, 0.25, 1)
        vfy.vfy_attend_full_packed(ctx, q, cu, *pool, K, ids, slots, cu_res, K, ln, 0.5, 0.25, out, lse, 1)
    try:
        step()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                step()
        for r in range(6):
            L = 300 + n * (r + 1)
            want = rng.standard_normal(m).astype(np.float32)
            want[(L - n) // C:(L - 1) // C + 1] = np.inf        # the block's chunks stay resident
            scores.copy_(torch.from_numpy(want))
            ln.fill_(L)
            wide.copy_(torch.from_numpy(rng.standard_normal(wide.shape)))
            graph.replay()
            torch.cuda.synchronize()
            i, s = ids.tolist(), slots.tolist()
            assert cu_res.tolist() == [0, K] and set((L - n) // C + np.arange((L - 1) // C - (L - n) // C + 1)) <= set(i)
            after = [p.cpu().numpy() for p in pool]
            for e in range(K):                                  # the pool holds what the store holds
                assert np.array_equal(after[0][s[e]], host[0][i[e]].numpy()) and np.array_equal(after[1][s[e]], host[1][i[e]].numpy())
            codes, scales = B.pack_rows(O.bf16_to_f64(H.bits_of(k)), 0.5)
            row = B.record_values(host[0].numpy()[(L - 1) // C, 1], d)[(L - 1) % C]
            assert np.array_equal(row, np.where(codes[-1, 1] >= 8, -1.0, 1.0) * B.E2M1[codes[-1, 1] & 7] * np.repeat(B.E4M3[scales[-1, 1]], 16))
            ref = B.attend_packed_seq(O.bf16_to_f64(H.bits_of(q)), *after, i, s, L, 0.5, 0.25)
            close(H.bits_of(out), lse.cpu().numpy(), *ref)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


def appended(env, counts, lens, hkv, d, g, seed, x=None):
    """Appends the counts and compares every byte of store and pool."""
    H, vfy = env
    rng = np.random.default_rng(seed)
    T, chunks = sum(counts), [-(-n // C) for n in lens]
    k, v = [O.bf16_to_f64(B.to_bf16(rng.standard_normal((T, hkv, d)) * 8.0 * g if x is None else x)) for _ in range(2)]
    m = sum(chunks)
    slot_of = rng.permutation(m + 2)[:m] - 2
    store, pool = [records(rng, m, hkv, d) for _ in range(2)], [records(rng, m, hkv, d) for _ in range(2)]
    sd, pd = [u8(r) for r in store], [u8(r) for r in pool]
    cu_chunks = H.cu_from_counts(chunks)
    ctx = vfy.vfy_create(hkv, hkv, d, max_seqs=len(counts), max_queries_per_seq=max(counts), device=0)
    try:
        vfy.vfy_append_full_packed(ctx, H.dev_bf16(B.to_bf16(k)), H.dev_bf16(B.to_bf16(v)), H.dev_i32(H.cu_from_counts(counts)),
                                   H.dev_i32(lens), H.dev_i32(cu_chunks), H.dev_i32(slot_of), *sd, m, *pd, m, g, g, len(counts))
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()
    seq = np.repeat(np.arange(len(counts)), counts)
    at = np.concatenate([L - n + np.arange(n) for n, L in zip(counts, lens)])
    chunk, row = np.asarray(cu_chunks)[seq] + at // C, at % C
    for side, y in enumerate((k, v)):
        codes, scales = B.pack_rows(y, g)
        pairs = (codes[..., ::2] | codes[..., 1::2] << 4).reshape(T, hkv, d // 32, 16)
        for t in range(T):
            for recs, c in ((store, chunk[t]), (pool, slot_of[chunk[t]])):
                if c >= 0:
                    rec = recs[side][c]
                    rec[:, :32 * d].reshape(hkv, d // 32, C, 16)[:, :, row[t]] = pairs[t]
                    rec[:, 32 * d:].reshape(hkv, C, d // 16)[:, row[t]] = scales[t]
    for got, want in zip(sd + pd, store + pool):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("hkv,d,counts", [(4, 128, [1000, 1, 0, 700, 500]), (1, 64, [1000] * 15 + [1]), (3, 64, [1000, 0, 1000, 1000]),
                                          (32, 128, [300, 200]), (20, 64, [700])])
def test_append_of_many_tokens(env, hkv, d, counts):
    """More tokens than one round of CTAs holds; tokens of more jobs than a CTA has threads."""
    appended(env, counts, [n + 17 if n else 0 for n in counts], hkv, d, 0.037, hkv)


@pytest.mark.parametrize("seqs", [32, 33, 100])
def test_append_to_many_sequences(env, seqs):
    rng = np.random.default_rng(seqs)
    counts = rng.integers(0, 4, seqs)
    counts[-1] = 2
    appended(env, counts.tolist(), (counts + rng.integers(0, 200, seqs)).tolist(), 2, 64, 1.0, seqs)


@pytest.mark.parametrize("g", [1e-37, 1e-33, 2.0 ** -100, 2.0 ** -126, 1e29, 1e33, 2.0 ** 100, 2.0 ** 127])
def test_append_with_extreme_tensor_scales(env, g):
    """Quotients that overflow, underflow, or whose remainders would: the codes of IEEE divisions."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((40, 2, 64)) * np.exp2(np.clip(np.log2(g) + rng.integers(-14, 14, (40, 2, 1)), -130, 125))
    appended(env, [40], [50], 2, 64, float(np.float32(g)), 3, x)


@pytest.mark.parametrize("n", range(1, 17))
@pytest.mark.parametrize("heads", [(1, 1, 64), (2, 2, 128)])
def test_every_number_of_few_rows(env, heads, n):
    one(env, heads, n, 1000 + n, seed=n)
    one(env, heads, n, 1000 + n, seed=n, splits=1)                # (written by the attention kernel itself)


@pytest.mark.parametrize("n", [1, 4, 5, 17, 40])
@pytest.mark.parametrize("splits", [0, 1])
def test_wait_timeout_is_reported_and_recovered(env, n, splits):
    H, vfy = env
    rng = np.random.default_rng(n)
    m, L = 30, 30 * C
    pools = [records(rng, m, 4, 128) for _ in range(2)]
    q = B.to_bf16(rng.standard_normal((n, 16, 128)))
    ctx = vfy.vfy_create(16, 4, 128, max_queries_per_seq=n, device=0)
    try:
        vfy.vfy_set_splits(ctx, splits, 0)
        vfy.vfy_test_wait_timeout(ctx, 2000)
        attend(env, ctx, q, [0, n], pools, np.arange(m), np.arange(m), [0, m], [L])
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_TIMEOUT
        vfy.vfy_test_wait_timeout(ctx, 0)
        got, lse = attend(env, ctx, q, [0, n], pools, np.arange(m), np.arange(m), [0, m], [L])
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        close(got, lse, *B.attend_packed_seq(O.bf16_to_f64(q), *pools, np.arange(m), np.arange(m), L))
    finally:
        ctx.close()


@pytest.mark.parametrize("n", [2, 17])
def test_stable_metadata_and_two_streams(env, n):
    """Two contexts on two streams at once, with metadata that stays: both give what one call alone gives, every time."""
    H, vfy = env
    rng = np.random.default_rng(n)
    m, L = 60, 60 * C
    pools = [u8(records(rng, m, 4, 128)) for _ in range(2)]
    q = H.dev_bf16(B.to_bf16(rng.standard_normal((n, 16, 128))))
    ids, cu, cr, ln = H.dev_i32(np.arange(m)), H.dev_i32([0, n]), H.dev_i32([0, m]), H.dev_i32([L])
    ctxs = [vfy.vfy_create(16, 4, 128, max_queries_per_seq=n, device=0) for _ in range(2)]
    outs, lses = [torch.zeros_like(q) for _ in range(9)], [torch.zeros((n, 16), device="cuda") for _ in range(9)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    try:
        vfy.vfy_attend_full_packed(ctxs[0], q, cu, *pools, m, ids, ids, cr, m, ln, 1.0, 1.0, outs[8], lses[8], 1)
        for c in ctxs:
            vfy.vfy_set_stable_metadata(c, True)
        torch.cuda.synchronize()
        for i in range(8):
            with torch.cuda.stream(streams[i % 2]):
                vfy.vfy_attend_full_packed(ctxs[i % 2], q, cu, *pools, m, ids, ids, cr, m, ln, 1.0, 1.0, outs[i], lses[i], 1)
        torch.cuda.synchronize()
        assert all(torch.equal(o, outs[8]) for o in outs) and all(torch.equal(x, lses[8]) for x in lses)
        assert all(vfy.vfy_get_status(c) == vfy.VFY_OK for c in ctxs)
    finally:
        for c in ctxs:
            c.close()


@pytest.mark.parametrize("seqs", [2, 32, 33, 70])
@pytest.mark.parametrize("cap", [2, 9])
def test_batches_of_many_sequences(env, seqs, cap):
    """Sequences of every length in any order, equal ones and empty lists among them; batches up to 32 are started longest
    first."""
    H, vfy = env
    rng = np.random.default_rng([seqs, cap])
    hq, hkv, d = 4, 2, 64
    counts = rng.integers(1, cap + 1, seqs)
    res = rng.integers(0, 9, seqs)
    lens = np.maximum(res * C - rng.integers(0, C, seqs), counts)
    cu, cu_res, total = H.cu_from_counts(counts), H.cu_from_counts(res), int(res.sum())
    pools = [records(rng, total + 1, hkv, d) for _ in range(2)]
    slots, ids = rng.permutation(total + 1)[:total], np.concatenate([np.arange(r) for r in res])
    q = B.to_bf16(rng.standard_normal((int(cu[-1]), hq, d)))
    ctx = vfy.vfy_create(hq, hkv, d, max_seqs=seqs, max_queries_per_seq=cap, device=0)
    try:
        got, lse = attend(env, ctx, q, cu, pools, ids, slots, cu_res, lens)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()
    for b in range(seqs):
        at, e = slice(cu[b], cu[b + 1]), slice(cu_res[b], cu_res[b + 1])
        close(got[at], lse[at], *B.attend_packed_seq(O.bf16_to_f64(q[at]), *pools, ids[e], slots[e], int(lens[b])))


@pytest.mark.parametrize("heads", [(16, 4, 128), (4, 1, 64)])
@pytest.mark.parametrize("n", [1, 3, 4, 17])
def test_scores_below_every_fp32_value(env, heads, n):
    """Queries and a tensor scale so small that their product is 0: all keys a row attends weigh the same, the others
    nothing."""
    one(env, heads, n, 500 + n, spread=1e-30, gk=1e-30)
    one(env, heads, n, 64 * 9 + n, spread=1e-38, gk=1e-38, splits=1)
