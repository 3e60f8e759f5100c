"""The tree calls at the limits of their arguments: row offsets past a context's capacity, sequences behind one
that is too long, the last chunk id, bias offsets out of order, and what a context's workspace holds.

Attention is compared within 2^-8 (A + |o|) + 2^-16 A + 7e-4 A, A = sum_j p_j |v_j|: P is rounded to bf16 (half a
step, 2^-8, of every weight), then O, of a value that the first rounding moved; the last term is that of fp32 scores
of 128 products of N(0,1) values."""
import numpy as np
import pytest
import torch

from oracle import tree_oracle as T
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


def close(got, lse, ref, rlse, mag):
    g = O.bf16_to_f64(got)
    assert np.all(np.abs(g - ref) <= 2.0 ** -8 * (mag + np.abs(ref)) + (2.0 ** -16 + 7e-4) * mag + 1e-30)
    fin = np.isfinite(rlse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(rlse))
    assert np.all(np.abs(lse[fin] - rlse[fin]) <= 3.1e-4 + np.abs(rlse[fin]) * 2.0 ** -22)


def masks(sets, rows):
    """Row masks of `sets`, then rows of zeros."""
    w = np.zeros((rows, 8), np.uint32)
    w[:len(sets)] = T.mask_words(sets)
    return torch.from_numpy(w.view(np.int32)).cuda()


# ---------------------------------------------------------------------------------------------
# Row offsets past the capacity
# ---------------------------------------------------------------------------------------------

# (nodes a sequence, splits of full layers, of window layers): one and two row tiles; the merge in a cluster, the
# combine kernel, wide tiles and a single split
FORMS = [(32, 0, 0), (32, 40, 20), (32, 3, 1), (32, 1, 1), (64, 12, 3), (64, 1, 20)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,full_splits,swa_splits", FORMS)
def test_rows_past_the_capacity_are_neither_read_nor_written(env, d, cap, full_splits, swa_splits):
    """Offsets that only a 32-bit sum would let pass, a sequence that begins inside the capacity and ends behind it,
    one that begins before the first row: reported and left out whole, by the chain's layers too."""
    H, vfy = env
    ctx = vfy.vfy_create(4, 1, d, max_seqs=1, max_queries_per_seq=cap, device=0)
    q = torch.zeros((cap, 4, d), dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros((64, 1, C, d), dtype=torch.bfloat16, device="cuda")
    ring = torch.zeros((1, 1, 2048, d), dtype=torch.bfloat16, device="cuda")
    words, depth = torch.zeros((cap, 8), dtype=torch.int32, device="cuda"), H.dev_i32(np.zeros(cap))
    ids, cu_res, L, zero = H.dev_i32(np.arange(64)), H.dev_i32([0, 64]), H.dev_i32([64 * C]), H.dev_i32([0])
    out, lse = torch.full_like(q, 3.0), torch.full((cap, 4), 3.0, device="cuda")
    big = 2 ** 31 - 8
    try:
        vfy.vfy_set_splits(ctx, full_splits, swa_splits)
        for offsets in ([big, big + 15 - 2 ** 32], [cap - 4, cap + 11], [cap, cap + 1], [-5, 10]):
            cu = H.dev_i32(offsets)
            calls = [lambda: vfy.vfy_attend_full_tree(ctx, q, cu, words, pool, pool, 64, ids, ids, cu_res, 64, L, out, lse, 1),
                     lambda: vfy.vfy_attend_swa_tree(ctx, q, cu, words, depth, ring, ring, zero, L, out, lse, 1),
                     lambda: vfy.vfy_attend_full(ctx, q, cu, pool, pool, 64, ids, ids, cu_res, 64, L, out, lse, 1),
                     lambda: vfy.vfy_attend_swa(ctx, q, cu, ring, ring, zero, L, out, lse, 1)]
            for i, call in enumerate(calls):
                call()
                assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT, (offsets, i)
                assert (out == 3).all() and (lse == 3).all(), (offsets, i)
    finally:
        ctx.close()


@pytest.mark.parametrize("heads", [(4, 1, 128), (4, 1, 64)])
@pytest.mark.parametrize("splits,bound", [(0, 0), (0, 256), (40, 0), (3, 0)])
def test_a_sequence_behind_one_that_is_too_long(env, heads, splits, bound):
    """A context of 1024 queries: 400 rows are more than a tree may have and are left out, the tree of 200 behind them
    (rows 400 to 599, past 256 a sequence) is planned, attended and compacted."""
    H, vfy = env
    hq, hkv, d = heads
    W, R = 512, 2048
    rng = np.random.default_rng([splits, bound, d])
    n, L = 200, 1000
    cu = [0, 400, 600]
    parents = synth.random_tree(rng, n)
    sets, depth = T.ancestors(parents.tolist()), T.depths(parents.tolist())
    ctx = vfy.vfy_create(hq, hkv, d, max_seqs=2, max_queries_per_seq=1024, window=W, ring_len=R, device=0)
    q = synth.normal_bf16(rng, (600, hq, d))
    m = -(-L // C)
    kp, vp = synth.normal_bf16(rng, (m, hkv, C, d)), synth.normal_bf16(rng, (m, hkv, C, d))
    kr, vr = synth.normal_bf16(rng, (2, hkv, R, d)), synth.normal_bf16(rng, (2, hkv, R, d))
    ids = np.arange(m)
    cu_d, lens = H.dev_i32(cu), H.dev_i32([3000, L])
    dep, words = H.dev_i32(np.full(600, -9)), torch.full((600, 8), -9, dtype=torch.int32, device="cuda")
    try:
        vfy.vfy_set_splits(ctx, splits, min(splits, 20))
        vfy.vfy_tree_plan(ctx, H.dev_i32(np.concatenate([np.arange(-1, 399), parents])), cu_d, dep, words, 2)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        assert (dep[:400] == -9).all() and dep[400:].cpu().tolist() == depth
        assert np.array_equal(words[400:].cpu().numpy().view(np.uint32), T.mask_words(sets))
        dep[:400] = 0
        qd = H.dev_bf16(q)
        for window in (False, True):
            out, lse = torch.full_like(qd, 7.0), torch.full((600, hq), 7.0, device="cuda")
            if window:
                vfy.vfy_attend_swa_tree(ctx, qd, cu_d, words, dep, H.dev_bf16(kr), H.dev_bf16(vr), H.dev_i32([0, 77]), lens,
                                        out, lse, 2)
                ref = T.attend_tree_ring_seq(q[400:], sets, depth, kr[1], vr[1], 77, L, W)
            else:
                vfy.vfy_attend_full_tree(ctx, qd, cu_d, words, H.dev_bf16(kp), H.dev_bf16(vp), m, H.dev_i32(ids),
                                         H.dev_i32(ids), H.dev_i32([0, 0, m]), max(m, bound), lens, out, lse, 2)
                ref = T.attend_tree_full_seq(q[400:], sets, kp, vp, ids, ids, L)
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
            assert (out[:400] == 7).all() and (lse[:400] == 7).all()
            close(H.bits_of(out)[400:], lse[400:].cpu().numpy(), *ref)
        path = np.full(600, -1)
        path[[0, 400, 401, 402]] = [0, 0, 5, 9]
        k, v = H.dev_bf16(kr), H.dev_bf16(vr)
        vfy.vfy_compact_swa(ctx, H.dev_i32(path), H.dev_i32([0, 2]), cu_d, lens, H.dev_i32([0, 77]), [k], [v], 2)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        want = T.compact_ring(path, [0, 2], cu, [3000, L], [0, 77], kr)
        assert np.array_equal(H.bits_of(k), want)
    finally:
        ctx.close()


@pytest.mark.parametrize("bound", [0, 256])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_the_last_chunk_id(env, at, bound):
    """The last chunk that a list may name ends at position 2^31 - 1: behind every short sequence, so that no row
    attends it, wherever it stands in the list, and whatever its slot holds."""
    H, vfy = env
    rng = np.random.default_rng(at)
    n, L = 40, 100
    sets = T.ancestors(synth.random_tree(rng, n).tolist())
    q = synth.normal_bf16(rng, (n, 16, 128))
    kp, vp = synth.normal_bf16(rng, (3, 4, C, 128)), synth.normal_bf16(rng, (3, 4, C, 128))
    kp[2], vp[2] = 0x7FC0, 0x7FC0
    ids, slots = [0, 1], [0, 1]
    ids.insert(at, 2 ** 25 - 1)
    slots.insert(at, 2)
    ctx = vfy.vfy_create(16, 4, 128, max_queries_per_seq=n, device=0)
    qd = H.dev_bf16(q)
    out, lse = torch.full_like(qd, 7.0), torch.full((n, 16), 7.0, device="cuda")
    try:
        vfy.vfy_attend_full_tree(ctx, qd, H.dev_i32([0, n]), masks(sets, n), H.dev_bf16(kp), H.dev_bf16(vp), 3, H.dev_i32(ids),
                                 H.dev_i32(slots), H.dev_i32([0, 3]), max(3, bound), H.dev_i32([L]), out, lse, 1)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        close(H.bits_of(out), lse.cpu().numpy(), *T.attend_tree_full_seq(q, sets, kp, vp, [0, 1], [0, 1], L))
    finally:
        ctx.close()


# ---------------------------------------------------------------------------------------------
# Bias offsets, workspace
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("offsets", [[0, 2, 1], [0, -1, 2], [-3, 0, 2], [0, -2, -1]])
def test_bias_offsets_out_of_order_are_reported(env, rows, offsets):
    """The sequences whose offsets are negative or descend get no bias; the others get theirs."""
    H, vfy = env
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=2, max_queries_per_seq=4, device=0)
    x = torch.arange(2 * rows * 50, device="cuda", dtype=torch.float32).view(2 * rows, 50)
    token, value = [7, 7], [1.0, 2.0]
    try:
        rules = vfy.LogitRules(cu_bias=H.dev_i32(offsets), bias_token=H.dev_i32(token), bias_value=H.dev_f32(value))
        out = torch.full_like(x, 77.0)
        vfy.vfy_process_logits(ctx, x, 50, H.dev_i32([0, rows, 2 * rows]), 2 * rows, rules, out, 2)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        want = x.clone()
        for b in range(2):
            if 0 <= offsets[b] <= offsets[b + 1]:
                want[rows * b:rows * (b + 1), 7] += sum(value[offsets[b]:offsets[b + 1]])
        assert torch.equal(out, want)
    finally:
        ctx.close()


def test_a_context_holds_the_partials_that_its_calls_can_use(env):
    """Only contexts whose trees can go to CTA pairs (d = 128, and two row tiles or four sequences) hold those
    pairs' partials: 256 rows a SM. A chain's context of one sequence holds its splits."""
    H, vfy = env
    n = 16                                             # contexts, so that the allocator's granularity is small beside
    sms = torch.cuda.get_device_properties(0).multi_processor_count

    def each(*shape, **kw):
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        held = [vfy.vfy_create(*shape, device=0, **kw) for _ in range(n)]
        after = torch.cuda.mem_get_info()[0]
        for c in held:
            c.close()
        return (before - after) / n

    each(4, 1, 64, max_queries_per_seq=17)             # (the first context loads the kernels)
    pairs = sms * 256 * (128 + 2) * 4
    slack = 6 << 20                                    # seven allocations, the small ones of at most 2 MB together
    for shape, kw in (((4, 1, 64), dict(max_queries_per_seq=256)), ((4, 1, 128), dict(max_queries_per_seq=17)),
                      ((4, 4, 128), dict(max_queries_per_seq=128, max_seqs=3))):
        hkv, d, seqs = shape[1], shape[2], kw.get("max_seqs", 1)
        tiles = -(-kw["max_queries_per_seq"] * shape[0] // hkv // 128)
        own = seqs * tiles * hkv * 4 * 128 * (d + 2) * 4
        assert own + slack < pairs
        assert each(*shape, max_splits=4, **kw) <= own + slack, (shape, kw)
    assert each(4, 1, 128, max_queries_per_seq=64, max_splits=4) >= pairs
    assert each(4, 1, 128, max_queries_per_seq=17, max_seqs=4, max_splits=4) >= pairs
