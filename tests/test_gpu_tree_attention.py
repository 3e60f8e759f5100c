"""Tree attention through the C ABI against the fp64 oracle: full layers (pool) and window layers
(ring), head layouts, tree sizes from one node to the limit, blocks that cross chunk and ring ends,
sparse residency, arbitrary masks, rows that attend nothing, ragged batches, every split setting.

Tolerance. With p the softmax weights and A = sum_j p_j |v_j|: P is rounded to bf16 (half a step,
2^-8, of every term), partial rows that merge in a cluster are rounded to bf16 once more, and O is:
    |error| <= 2^-8 (2 A + |o|) + fp32 terms.
The fp32 terms: a score is a sum of d <= 128 products in fp32, off by at most (d + 2) 2^-23 times
scale * sum |q k| (below 20 for the N(0,1) inputs here), so by 3.1e-4; the weights follow it
relatively, twice (weight and normaliser): 7e-4 A. The LSE is off by that 3.1e-4 and the roundings
of the log2 units, |lse| 2^-22."""
import numpy as np
import pytest
import torch

from oracle import tree_oracle as T
from oracle import vfy_oracle as O
from speculative_decode_verify_attn_gb300 import synth

pytestmark = pytest.mark.gpu

C = 64
NAN = 0x7FC0


@pytest.fixture(scope="module")
def env():
    import __graft_entry__
    __graft_entry__.build()
    from speculative_decode_verify_attn_gb300 import harness, vfy
    torch.cuda.set_device(0)
    return harness, vfy


def check(got, lse, ref, rlse, mag, what):
    g = O.bf16_to_f64(got)
    assert np.all(np.isfinite(g)), what
    excess = np.abs(g - ref) - (2.0 ** -8 * (2 * mag + np.abs(ref)) + 7e-4 * mag + 1e-30)
    assert excess.max() <= 0, f"{what}: {np.abs(g - ref).max():.3e}"
    fin = np.isfinite(rlse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(rlse)), what
    if fin.any():
        assert np.all(np.abs(lse[fin] - rlse[fin]) <= 3.1e-4 + np.abs(rlse[fin]) * 2.0 ** -22), what


def words_dev(sets_or_words):
    w = sets_or_words if isinstance(sets_or_words, np.ndarray) else T.mask_words(sets_or_words)
    return torch.from_numpy(np.ascontiguousarray(w).view(np.int32)).cuda()


# A host bound on the resident chunks above the longest list: what decides that a block of several row tiles
# (or a batch) goes to the kernel of CTA pairs.
LOOSE = pytest.mark.parametrize("bound", [0, 256])


def attend_full(H, vfy, ctx, q, cu, words, kp, vp, ids, slots, cu_res, lens, stream=None, bound=0):
    qd = H.dev_bf16(q)
    out = torch.full_like(qd, 7.0)
    lse = torch.full(qd.shape[:2], 7.0, device="cuda")
    k, v = H.dev_bf16(kp), H.dev_bf16(vp)
    vfy.vfy_attend_full_tree(ctx, qd, H.dev_i32(cu), words_dev(words), k, v, k.shape[0], H.dev_i32(ids),
                             H.dev_i32(slots), H.dev_i32(cu_res), max(bound, int(np.diff(cu_res).max())), H.dev_i32(lens),
                             out, lse, len(cu) - 1, stream)
    torch.cuda.synchronize()
    return H.bits_of(out), lse.cpu().numpy()


def attend_swa(H, vfy, ctx, q, cu, words, depth, kr, vr, phi, lens):
    qd = H.dev_bf16(q)
    out = torch.full_like(qd, 7.0)
    lse = torch.full(qd.shape[:2], 7.0, device="cuda")
    vfy.vfy_attend_swa_tree(ctx, qd, H.dev_i32(cu), words_dev(words), H.dev_i32(depth), H.dev_bf16(kr), H.dev_bf16(vr),
                            H.dev_i32(phi), H.dev_i32(lens), out, lse, len(cu) - 1)
    torch.cuda.synchronize()
    return H.bits_of(out), lse.cpu().numpy()


def pool_case(rng, hq, hkv, d, n, L, keep=None):
    """Chunks (all, or `keep` of them with the block's), slots in random order in a larger pool whose
    other slots and whose rows past L hold NaN."""
    total = -(-L // C)
    ids = np.arange(total)
    if keep is not None and keep < total:
        block = np.arange((L - n) // C, total)
        rest = np.sort(rng.choice(block[0], max(0, keep - len(block)), replace=False)) if block[0] else []
        ids = np.concatenate([rest, block]).astype(np.int64)
    slots = rng.permutation(len(ids) + 2)[: len(ids)]
    kp = np.full((len(ids) + 2, hkv, C, d), NAN, np.uint16)
    vp = kp.copy()
    kp[slots] = synth.normal_bf16(rng, (len(ids), hkv, C, d))
    vp[slots] = synth.normal_bf16(rng, (len(ids), hkv, C, d))
    if L % C:
        at = slots[np.flatnonzero(ids == total - 1)[0]]
        kp[at, :, L % C:] = NAN
        vp[at, :, L % C:] = NAN
    return synth.normal_bf16(rng, (n, hq, d)), kp, vp, ids, slots


LAYOUTS = [(16, 4, 128), (4, 1, 64), (8, 8, 128), (32, 4, 128), (16, 2, 64)]


@LOOSE
@pytest.mark.parametrize("heads", LAYOUTS)
@pytest.mark.parametrize("n,L", [(1, 1), (1, 64), (2, 65), (17, 17), (17, 1000), (33, 97), (64, 128), (65, 700),
                                 (255, 300), (256, 513)])
def test_full_layer(env, heads, n, L, bound):
    H, vfy = env
    hq, hkv, d = heads
    rng = np.random.default_rng([n, L, hq])
    q, kp, vp, ids, slots = pool_case(rng, hq, hkv, d, n, L)
    sets = T.ancestors(synth.random_tree(rng, n).tolist())
    ref = T.attend_tree_full_seq(q, sets, kp, vp, ids, slots, L)
    ctx = vfy.vfy_create(hq, hkv, d, max_queries_per_seq=n, ring_len=4096, device=0)
    try:
        got = attend_full(H, vfy, ctx, q, [0, n], sets, kp, vp, ids, slots, [0, len(ids)], [L], bound=bound)
        check(*got, *ref, f"{heads} {n} {L}")
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


@LOOSE
@pytest.mark.parametrize("splits", [0, 1, 2, 3, 7, 16, 40])
@pytest.mark.parametrize("n", [9, 47, 64])
def test_full_layer_split_settings(env, splits, n, bound):
    H, vfy = env
    rng = np.random.default_rng([splits, n])
    L, keep = 9000, 41
    q, kp, vp, ids, slots = pool_case(rng, 16, 4, 128, n, L, keep)
    sets = T.ancestors(synth.random_tree(rng, n).tolist())
    ref = T.attend_tree_full_seq(q, sets, kp, vp, ids, slots, L)
    ctx = vfy.vfy_create(16, 4, 128, max_queries_per_seq=64, device=0)
    try:
        vfy.vfy_set_splits(ctx, splits, 0)
        got = attend_full(H, vfy, ctx, q, [0, n], sets, kp, vp, ids, slots, [0, len(ids)], [L], bound=bound)
        check(*got, *ref, f"{splits} {n}")
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


@pytest.mark.parametrize("n,L,phi", [(1, 1, 0), (1, 700, 5), (17, 17, 2040), (17, 5000, 100), (33, 40, 63), (64, 9001, 1900),
                                     (65, 600, -3), (200, 3000, 2047), (256, 256, 1), (256, 70000, 777)])
@pytest.mark.parametrize("heads,splits", [((16, 4, 128), 0), ((4, 1, 64), 0), ((16, 4, 128), 20), ((32, 4, 128), 3)])
def test_window_layer(env, heads, splits, n, L, phi):
    H, vfy = env
    hq, hkv, d = heads
    W, R = 512, 2048
    rng = np.random.default_rng([n, L, hq, splits])
    parents = synth.random_tree(rng, n).tolist()
    sets, depth = T.ancestors(parents), T.depths(parents)
    q = synth.normal_bf16(rng, (n, hq, d))
    kr, vr = np.full((1, hkv, R, d), NAN, np.uint16), np.full((1, hkv, R, d), NAN, np.uint16)
    at = (np.arange(max(0, L - n - W + 1), L) + phi) % R          # the other slots hold NaN
    kr[:, :, at] = synth.normal_bf16(rng, (1, hkv, len(at), d))
    vr[:, :, at] = synth.normal_bf16(rng, (1, hkv, len(at), d))
    ref = T.attend_tree_ring_seq(q, sets, depth, kr[0], vr[0], phi, L, W)
    ctx = vfy.vfy_create(hq, hkv, d, window=W, ring_len=R, max_queries_per_seq=n, device=0)
    try:
        vfy.vfy_set_splits(ctx, 0, splits)
        check(*attend_swa(H, vfy, ctx, q, [0, n], sets, depth, kr, vr, [phi], [L]), *ref, f"{heads} {n} {L} {phi}")
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


@LOOSE
def test_any_mask_is_taken(env, bound):
    """Masks that no plan makes: later nodes, no node at all (with and without a prefix), bits past
    the block (ignored)."""
    H, vfy = env
    rng = np.random.default_rng(8)
    n = 40
    for L in (n, n + 1, 300):
        q, kp, vp, ids, slots = pool_case(rng, 16, 4, 128, n, L)
        bits = rng.random((n, 256)) < 0.3
        bits[3] = False
        bits[7, :n] = False                              # bits past the block only
        bits[11] = True
        sets = [set(np.flatnonzero(r).tolist()) for r in bits]
        ref = T.attend_tree_full_seq(q, sets, kp, vp, ids, slots, L)
        ctx = vfy.vfy_create(16, 4, 128, max_queries_per_seq=n, device=0)
        try:
            got, lse = attend_full(H, vfy, ctx, q, [0, n], sets, kp, vp, ids, slots, [0, len(ids)], [L], bound=bound)
            check(got, lse, *ref, f"L {L}")
            if L == n:
                assert not got[3].any() and np.isneginf(lse[3]).all() and np.isneginf(lse[7]).all()
        finally:
            ctx.close()


@LOOSE
@pytest.mark.parametrize("splits", [0, 2, 5])
def test_ragged_batch(env, splits, bound):
    """Sequences of 1 to 200 nodes, one of them empty, in both layers; rows behind the last sequence
    are left as they were."""
    H, vfy = env
    hq, hkv, d, W, R = 16, 4, 128, 512, 2048
    rng = np.random.default_rng(20 + splits)
    ns, Ls = [17, 0, 200, 1, 64, 33], [1500, 0, 200, 64, 2000, 4000]
    cu = np.concatenate([[0], np.cumsum(ns)])
    q = synth.normal_bf16(rng, (int(cu[-1]) + 5, hq, d))
    words = np.zeros((int(cu[-1]) + 5, 8), np.uint32)
    depth = np.zeros(int(cu[-1]) + 5, np.int64)
    seqs, ids, slots, cu_res = [], [], [], [0]
    total = sum(-(-L // C) for L in Ls)
    order = rng.permutation(total)
    kp, vp = synth.normal_bf16(rng, (total, hkv, C, d)), synth.normal_bf16(rng, (total, hkv, C, d))
    kr, vr = synth.normal_bf16(rng, (len(ns), hkv, R, d)), synth.normal_bf16(rng, (len(ns), hkv, R, d))
    phi = rng.integers(-R, R, len(ns))
    for b, (n, L) in enumerate(zip(ns, Ls)):
        parents = synth.random_tree(rng, n).tolist() if n else []
        sets = T.ancestors(parents)
        m = -(-L // C)
        seqs.append((sets, np.arange(m), order[cu_res[-1]:cu_res[-1] + m], parents))
        ids += list(range(m))
        slots += order[cu_res[-1]:cu_res[-1] + m].tolist()
        cu_res.append(cu_res[-1] + m)
        if n:
            words[cu[b]:cu[b + 1]] = T.mask_words(sets)
            depth[cu[b]:cu[b + 1]] = T.depths(parents)
    ctx = vfy.vfy_create(hq, hkv, d, max_seqs=len(ns), max_queries_per_seq=200, device=0)
    try:
        vfy.vfy_set_splits(ctx, splits, splits)
        got, lse = attend_full(H, vfy, ctx, q, cu, words, kp, vp, ids, slots, cu_res, Ls, bound=bound)
        gotw, lsew = attend_swa(H, vfy, ctx, q, cu, words, depth, kr, vr, phi, Ls)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        for b, (sets, i_b, s_b, parents) in enumerate(seqs):
            rows = slice(cu[b], cu[b + 1])
            if not ns[b]:
                continue
            check(got[rows], lse[rows], *T.attend_tree_full_seq(q[rows], sets, kp, vp, i_b, s_b, Ls[b]), f"full {b}")
            check(gotw[rows], lsew[rows], *T.attend_tree_ring_seq(q[rows], sets, T.depths(parents), kr[b], vr[b],
                                                                  int(phi[b]), Ls[b], W), f"window {b}")
        seven = synth.bf16_bits(np.float32(7.0))
        assert (got[cu[-1]:] == seven).all() and (gotw[cu[-1]:] == seven).all()
        assert (lse[cu[-1]:] == 7).all() and (lsew[cu[-1]:] == 7).all()
    finally:
        ctx.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ns,Ls", [([9, 47, 20, 64, 3], [60000, 50000, 70000, 3000, 130]), ([64, 10], [40000, 190000]),
                                   ([10, 64], [190000, 40000]), ([130, 200, 64], [30000, 64000, 90000])])
def test_long_ragged_batch(env, ns, Ls, d):
    """One KV head, so that a CTA's run holds many tiles and passes from sequences of one row tile to such
    of two and back."""
    H, vfy = env
    rng = np.random.default_rng(sum(Ls))
    hq = 4
    cu = np.concatenate([[0], np.cumsum(ns)])
    counts = [-(-L // C) for L in Ls]
    cu_res = np.concatenate([[0], np.cumsum(counts)])
    total = int(cu_res[-1])
    slots = rng.permutation(total)
    kp, vp = synth.normal_bf16(rng, (total, 1, C, d)), synth.normal_bf16(rng, (total, 1, C, d))
    q = synth.normal_bf16(rng, (int(cu[-1]), hq, d))
    sets = [T.ancestors(synth.random_tree(rng, n).tolist()) for n in ns]
    ids = np.concatenate([np.arange(c) for c in counts])
    ctx = vfy.vfy_create(hq, 1, d, max_seqs=len(ns), max_queries_per_seq=256, device=0)
    try:
        got, lse = attend_full(H, vfy, ctx, q, cu, T.mask_words(sum(sets, [])), kp, vp, ids, slots, cu_res, Ls)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        for b in range(len(ns)):
            rows, at = slice(cu[b], cu[b + 1]), slice(cu_res[b], cu_res[b + 1])
            check(got[rows], lse[rows], *T.attend_tree_full_seq(q[rows], sets[b], kp, vp, ids[at], slots[at], Ls[b]), f"{b}")
    finally:
        ctx.close()


@pytest.mark.parametrize("n", [1, 17, 32])
def test_a_chain_gives_the_bits_of_the_linear_block(env, n):
    """A chain's masks and depths: in a full layer whose splits go through the combine, a block of one
    row tile runs the same arithmetic in the same order. (A window layer merges its splits in fp32 for
    trees and in bf16 for the linear block.)"""
    H, vfy = env
    rng = np.random.default_rng(30 + n)
    L = 3333
    q, kp, vp, ids, slots = pool_case(rng, 16, 4, 128, n, L)
    sets = T.ancestors(list(range(-1, n - 1)))
    kr, vr = synth.normal_bf16(rng, (1, 4, 2048, 128)), synth.normal_bf16(rng, (1, 4, 2048, 128))
    ctx = vfy.vfy_create(16, 4, 128, max_queries_per_seq=n, device=0)
    try:
        got, lse = attend_full(H, vfy, ctx, q, [0, n], sets, kp, vp, ids, slots, [0, len(ids)], [L])
        lin, llse = H.attend_full(ctx, q, [0, n], kp, vp, ids, slots, [0, len(ids)], [L])
        assert np.array_equal(got, lin) and np.array_equal(lse, llse)
        got, lse = attend_swa(H, vfy, ctx, q, [0, n], sets, list(range(n)), kr, vr, [100], [L])
        check(got, lse, *T.attend_tree_ring_seq(q, sets, list(range(n)), kr[0], vr[0], 100, L, 512), "window")
    finally:
        ctx.close()


@pytest.mark.parametrize("ns", [[1], [2], [17], [256], [5, 0, 64, 33, 255, 1]])
def test_plan(env, ns):
    H, vfy = env
    rng = np.random.default_rng(len(ns) + ns[0])
    parents = [synth.random_tree(rng, n) if n else np.zeros(0, np.int32) for n in ns]
    parents[0] = np.arange(-1, ns[0] - 1, dtype=np.int32)          # a chain: as deep as it gets
    if ns[-1] > 2:
        parents[-1][ns[-1] // 2] = -1                              # a second root
    cu = np.concatenate([[0], np.cumsum(ns)])
    n = int(cu[-1])
    depth = torch.full((n + 3,), -9, dtype=torch.int32, device="cuda")
    mask = torch.full((n + 3, 8), -9, dtype=torch.int32, device="cuda")
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=len(ns), max_queries_per_seq=256, device=0)
    try:
        vfy.vfy_tree_plan(ctx, H.dev_i32(np.concatenate(parents)), H.dev_i32(cu), depth, mask, len(ns))
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        want_d = sum((T.depths(p.tolist()) for p in parents), [])
        want_m = T.mask_words(sum((T.ancestors(p.tolist()) for p in parents), []))
        assert depth.cpu().tolist() == want_d + [-9] * 3
        assert np.array_equal(mask.cpu().numpy()[:n].view(np.uint32), want_m) and (mask[n:] == -9).all()
    finally:
        ctx.close()


def test_plan_reports_bad_parents(env):
    H, vfy = env
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=2, max_queries_per_seq=8, device=0)
    depth = torch.full((12,), -9, dtype=torch.int32, device="cuda")
    mask = torch.full((12, 8), -9, dtype=torch.int32, device="cuda")
    try:
        # node 2 names itself, node 3 a later node, node 4 nothing there is: roots of their own
        vfy.vfy_tree_plan(ctx, H.dev_i32([-1, 0, 2, 4, -5]), H.dev_i32([0, 5]), depth, mask, 1)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        assert depth[:5].cpu().tolist() == [0, 1, 0, 0, 0]
        assert mask[:5, 0].cpu().tolist() == [1, 3, 4, 8, 16]
        # a sequence beyond the context's capacity is skipped, the other is planned
        depth.fill_(-9)
        vfy.vfy_tree_plan(ctx, H.dev_i32([-1] + list(range(8)) + [-1, 0]), H.dev_i32([0, 9, 11]), depth, mask, 2)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        assert depth.cpu().tolist() == [-9] * 9 + [0, 1, -9]
    finally:
        ctx.close()


def test_attention_reports_bad_input(env):
    H, vfy = env
    rng = np.random.default_rng(50)
    n, L = 9, 100
    q, kp, vp, ids, slots = pool_case(rng, 16, 4, 128, n, L)
    sets = T.ancestors(synth.random_tree(rng, n).tolist())
    kr, vr = synth.normal_bf16(rng, (1, 4, 2048, 128)), synth.normal_bf16(rng, (1, 4, 2048, 128))
    ctx = vfy.vfy_create(16, 4, 128, max_queries_per_seq=8, device=0)
    try:
        got, _ = attend_full(H, vfy, ctx, q, [0, n], sets, kp, vp, ids, slots, [0, len(ids)], [L])   # 9 nodes of 8
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        # a slot that the pool does not have: its chunk is skipped
        bad = slots.copy()
        bad[0] = 99
        m = 8
        got, lse = attend_full(H, vfy, ctx, q[:m], [0, m], sets[:m], kp, vp, ids, bad, [0, len(ids)], [L - 1])
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        check(got, lse, *T.attend_tree_full_seq(q[:m], sets[:m], kp, vp, ids[1:], slots[1:], L - 1), "bad slot")
        # a depth outside the block counts as its nearest end
        got, lse = attend_swa(H, vfy, ctx, q[:m], [0, m], sets[:m], [-4] + [0] * 6 + [99], kr, vr, [0], [2000])
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        check(got, lse, *T.attend_tree_ring_seq(q[:m], sets[:m], [0] * 7 + [7], kr[0], vr[0], 0, 2000, 512), "bad depth")
    finally:
        ctx.close()


def test_pairs_report_bad_input(env):
    """The same in a context of two row tiles, in the kernel of CTA pairs; a bad sequence leaves the others alone."""
    H, vfy = env
    rng = np.random.default_rng(52)
    n, L = 60, 2000
    q, kp, vp, ids, slots = pool_case(rng, 16, 4, 128, n, L)
    sets = T.ancestors(synth.random_tree(rng, n).tolist())
    ctx = vfy.vfy_create(16, 4, 128, max_seqs=2, max_queries_per_seq=60, device=0)
    both = [0, len(ids), 2 * len(ids)]
    two = [np.concatenate([x, x]) for x in (q, T.mask_words(sets), ids, slots)]
    try:
        bad = slots.copy()
        bad[3] = 99
        got, lse = attend_full(H, vfy, ctx, q, [0, n], sets, kp, vp, ids, bad, [0, len(ids)], [L], bound=256)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        keep = np.arange(len(ids)) != 3
        ref = T.attend_tree_full_seq(q, sets, kp, vp, ids[keep], slots[keep], L)
        check(got, lse, *ref, "bad slot")
        ref = T.attend_tree_full_seq(q, sets, kp, vp, ids, slots, L)
        for cu, lens in (([0, n, 2 * n], [L, n - 1]), ([0, n, 2 * n + 1], [L, L])):    # too short; 61 nodes of 60
            got, lse = attend_full(H, vfy, ctx, two[0], cu, two[1], kp, vp, two[2], two[3], both, lens, bound=256)
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
            check(got[:n], lse[:n], *ref, "the good sequence")
            assert (lse[n:] == 7).all()
    finally:
        ctx.close()


def test_refusals(env):
    """Host-side checks: nothing is launched."""
    H, vfy = env
    ctx = vfy.vfy_create(16, 4, 128, window=100, max_queries_per_seq=101, device=0)
    small = vfy.vfy_create(16, 4, 128, window=100, max_queries_per_seq=100, device=0)
    i = torch.zeros(64, dtype=torch.int32, device="cuda")
    x = torch.zeros((1, 4, 2048, 128), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((1, 16, 128), dtype=torch.bfloat16, device="cuda")
    try:
        def swa(c, mask=i, num=1):
            vfy.vfy_attend_swa_tree(c, q, i, mask, i, x, x, i, i, q, None, num)
        for call in (lambda: swa(ctx),                               # the window is smaller than the block
                     lambda: swa(small, mask=i[1:]),                 # misaligned mask
                     lambda: swa(small, num=2), lambda: swa(small, num=0),
                     lambda: vfy.vfy_attend_full_tree(small, q, i, i[2:], x, x, 32, i, i, i, 1, i, q, None, 1),
                     lambda: vfy.vfy_attend_full_tree(small, q, i, i, x, x, 0, i, i, i, 1, i, q, None, 1),
                     lambda: vfy.vfy_tree_plan(small, i, i, i, i[1:], 1), lambda: vfy.vfy_tree_plan(small, i, i, i, i, 2)):
            before = [vfy.vfy_launch_count(c) for c in (ctx, small)]
            with pytest.raises(vfy.VfyError) as e:
                call()
            assert e.value.status == vfy.VFY_EINVAL
            assert before == [vfy.vfy_launch_count(c) for c in (ctx, small)]
    finally:
        ctx.close()
        small.close()


@LOOSE
def test_plan_and_attention_in_one_graph(env, bound):
    """Captured on a side stream with stable metadata on: every replay attends by the tree that
    stands in `parents` then."""
    H, vfy = env
    rng = np.random.default_rng(60)
    n, L = 40, 2000
    q, kp, vp, ids, slots = pool_case(rng, 16, 4, 128, n, L)
    ctx = vfy.vfy_create(16, 4, 128, max_queries_per_seq=n, device=0)
    qd, kd, vd = H.dev_bf16(q), H.dev_bf16(kp), H.dev_bf16(vp)
    cu, lens, idd, sd, cr = (H.dev_i32(a) for a in ([0, n], [L], ids, slots, [0, len(ids)]))
    parents = torch.zeros(n, dtype=torch.int32, device="cuda")
    depth, mask = torch.zeros_like(parents), torch.zeros((n, 8), dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(qd), torch.zeros((n, 16), device="cuda")
    try:
        vfy.vfy_set_stable_metadata(ctx, True)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()

        def step():
            vfy.vfy_tree_plan(ctx, parents, cu, depth, mask, 1)
            vfy.vfy_attend_full_tree(ctx, qd, cu, mask, kd, vd, kd.shape[0], idd, sd, cr, max(bound, len(ids)), lens, out,
                                     lse, 1)
        with torch.cuda.stream(stream):
            parents.copy_(H.dev_i32(synth.random_tree(rng, n)))
            step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for _ in range(3):
            p = synth.random_tree(rng, n)
            parents.copy_(H.dev_i32(p))
            out.fill_(0)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            ref = T.attend_tree_full_seq(q, T.ancestors(p.tolist()), kp, vp, ids, slots, L)
            check(H.bits_of(out), lse.cpu().numpy(), *ref, "replay")
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


@LOOSE
@pytest.mark.parametrize("n", [9, 64])
def test_wait_timeout_is_reported_and_recovered(env, n, bound):
    H, vfy = env
    rng = np.random.default_rng(70)
    L = 9000
    q, kp, vp, ids, slots = pool_case(rng, 16, 4, 128, n, L)
    sets = T.ancestors(synth.random_tree(rng, n).tolist())
    ctx = vfy.vfy_create(16, 4, 128, max_queries_per_seq=n, device=0)
    try:
        vfy.vfy_test_wait_timeout(ctx, 2000)
        attend_full(H, vfy, ctx, q, [0, n], sets, kp, vp, ids, slots, [0, len(ids)], [L], bound=bound)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_TIMEOUT
        vfy.vfy_test_wait_timeout(ctx, 0)
        got = attend_full(H, vfy, ctx, q, [0, n], sets, kp, vp, ids, slots, [0, len(ids)], [L], bound=bound)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        check(*got, *T.attend_tree_full_seq(q, sets, kp, vp, ids, slots, L), "after a timeout")
    finally:
        ctx.close()
