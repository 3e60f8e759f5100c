"""Tree acceptance and path compaction through the C ABI, bit-exact against the oracle; then a whole tree
step (plan, append, attention, rules, acceptance, compaction, counting) in one captured graph, and the
next step on the cache it left."""
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


def accept(H, vfy, ctx, logits, drafts, parents, cu, max_rows=None):
    B, R = len(cu) - 1, int(cu[-1])
    out = [torch.full((n,), -7, dtype=torch.int32, device="cuda") for n in (B, R + 2, B, R + 2)]
    x = logits if isinstance(logits, torch.Tensor) else H.dev_f32(logits)
    vfy.vfy_accept_tree(ctx, x, x.shape[1], H.dev_i32(drafts if len(drafts) else [0]), H.dev_i32(parents), H.dev_i32(cu),
                        max_rows or R, *out, B)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in out]


def want(logits, drafts, parents, cu):
    res = [], [], [], []
    for b in range(len(cu) - 1):
        a, e = int(cu[b]), int(cu[b + 1])
        for r, x in zip(res, T.accept_tree_seq(logits[a:e], drafts[a - b:e - b - 1], list(parents[a:e]))):
            r.extend(x if isinstance(x, list) else [x])
    return list(res)


@pytest.mark.parametrize("vocab", [1, 3, 31, 1000, 4099, 32001, 131072])
@pytest.mark.parametrize("ns", [[1], [2], [17], [64, 1, 5], [256, 256]])
def test_accept(env, ns, vocab):
    H, vfy = env
    rng = np.random.default_rng([vocab, len(ns), ns[0]])
    cu = np.concatenate([[0], np.cumsum(ns)])
    R = int(cu[-1])
    targets = rng.integers(0, vocab, R)
    logits = synth.planted_logits(rng, targets, vocab)
    trees = [synth.random_tree(rng, n) for n in ns]
    drafts = np.concatenate([synth.tree_drafts_matching(rng, targets[cu[b]:cu[b + 1]], p, 0.7, max(2, vocab))
                             for b, p in enumerate(trees)]).astype(np.int64)
    parents = np.concatenate(trees)
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=len(ns), max_queries_per_seq=256, device=0)
    try:
        ref = want(logits, drafts, parents, cu)
        for _ in range(2):                                   # the workspace is left clean
            got = accept(H, vfy, ctx, logits, drafts, parents, cu)
            assert got[0].tolist() == ref[0] and got[2].tolist() == ref[2]
            assert got[1].tolist() == ref[1] + [-7, -7] and got[3].tolist() == ref[3] + [-7, -7]
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


def test_accept_ties_nan_and_misaligned_rows(env):
    """Equal maxima (the lowest index), -0 == +0, NaN (the maximum), infinities, all equal rows, in a
    vocabulary that puts rows on every 4-byte offset, from a base off the 16-byte grid."""
    H, vfy = env
    V, n = 1031, 9
    rng = np.random.default_rng(1)
    x = np.round(rng.standard_normal((n, V)) * 2).astype(np.float32)
    x[1] = -np.inf
    x[2, 1000:] = np.nan
    x[3] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    x[4, [700, 5, 1030]] = np.inf
    x[5, 1030] = 50
    x[6, 0] = 50
    x[7, [3, 4]] = 50
    base = torch.zeros(n * V + 8, device="cuda")
    parents = np.arange(-1, n - 1)
    targets = [O.argmax_row(r) for r in x]
    ctx = vfy.vfy_create(4, 1, 64, max_queries_per_seq=n, device=0)
    try:
        for off in range(4):
            view = base[off:off + n * V].view(n, V)
            view.copy_(torch.from_numpy(x))
            got = accept(H, vfy, ctx, view, targets[:-1], parents, [0, n])
            assert got[0].tolist() == [n - 1] and got[3][:n].tolist() == targets
    finally:
        ctx.close()


def test_accept_reports_bad_input(env):
    H, vfy = env
    rng = np.random.default_rng(2)
    V = 64
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=3, max_queries_per_seq=300, device=0)

    def clean():
        targets = rng.integers(0, V, 8)
        logits = synth.planted_logits(rng, targets, V)
        parents = np.concatenate([synth.random_tree(rng, 4), synth.random_tree(rng, 4)])
        drafts = np.concatenate([synth.tree_drafts_matching(rng, targets[a:a + 4], parents[a:a + 4], 0.9, V) for a in (0, 4)])
        ref = want(logits, drafts, parents, [0, 4, 8])
        got = accept(H, vfy, ctx, logits, drafts, parents, [0, 4, 8])
        assert [g[:len(r)].tolist() for g, r in zip(got, ref)] == ref
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    try:
        clean()
        # a parent at or behind its node is never reached
        lg = synth.planted_logits(rng, [1, 2, 3], V)
        got = accept(H, vfy, ctx, lg, [1, 2], [-1, 1, 0], [0, 3])
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT and got[0].tolist() == [0]
        clean()
        # an empty sequence, one past max_rows and one of 257 nodes: skipped; the others are accepted
        targets = rng.integers(0, V, 300)
        lg = synth.planted_logits(rng, targets, V)
        chain = np.arange(-1, 2)
        for cu, cap, done in (([0, 3, 3, 6], 6, (0, 2)), ([0, 3, 6, 9], 8, (0, 1)), ([0, 257, 260, 263], 263, (1, 2))):
            parents = np.zeros(300, np.int64)
            drafts = np.zeros(300, np.int64)
            for b in done:
                parents[cu[b]:cu[b] + 3] = chain
                drafts[cu[b] - b:cu[b] - b + 2] = targets[cu[b]:cu[b] + 2]
            got = accept(H, vfy, ctx, lg, drafts, parents, cu, cap)
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
            # (after an empty sequence the packed drafts of the others overlap: the oracle walks what stands there)
            ref = {b: T.accept_tree_seq(lg[cu[b]:cu[b] + 3], drafts[cu[b] - b:cu[b] - b + 2], chain.tolist()) for b in done}
            assert got[0].tolist() == [ref[b][0] if b in done else -7 for b in range(3)]
            for b in done:
                assert got[1][cu[b]:cu[b] + 3].tolist() == ref[b][1] and got[3][cu[b]:cu[b] + 3].tolist() == ref[b][3]
            clean()
        # the first sequence is empty: the second's drafts would start before the first one
        got = accept(H, vfy, ctx, lg, np.zeros(20), np.zeros(20), [0, 0, 3], 3)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT and (got[0] == -7).all()
        clean()
        # offsets out of order: nothing is done
        got = accept(H, vfy, ctx, lg, np.zeros(20), np.zeros(20), [0, 5, 3, 8], 8)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT and (got[0] == -7).all() and (got[1] == -7).all()
        clean()
    finally:
        ctx.close()


def ragged_paths(rng, ns, full=False):
    path, acc = [], []
    for n in ns:
        k = n - 1 if full else int(rng.integers(0, n))
        p = [0] + np.sort(rng.choice(np.arange(1, n), k, replace=False)).tolist()
        path += p + [-1] * (n - k - 1)
        acc.append(k)
    return path, acc


@pytest.mark.parametrize("shape", [(4, 128), (1, 64), (8, 128), (3, 64)])
@pytest.mark.parametrize("layers", [1, 3, 30])
def test_compact_rings(env, shape, layers):
    H, vfy = env
    hkv, d = shape
    rng = np.random.default_rng([hkv, layers])
    ns, lens = [17, 1, 64, 200, 2], [9000, 5, 64, 2050, 2048]
    cu = np.concatenate([[0], np.cumsum(ns)])
    phi = [0, 3, 2040, -100, 2047]
    ctx = vfy.vfy_create(hkv, hkv, d, max_seqs=len(ns), max_queries_per_seq=200, device=0)
    try:
        for full in (False, True):                           # the whole block accepted: nothing moves
            path, acc = ragged_paths(rng, ns, full)
            ks = [synth.normal_bf16(rng, (len(ns), hkv, 2048, d)) for _ in range(layers)]
            vs = [synth.normal_bf16(rng, (len(ns), hkv, 2048, d)) for _ in range(layers)]
            kd, vd = [H.dev_bf16(k) for k in ks], [H.dev_bf16(v) for v in vs]
            vfy.vfy_compact_swa(ctx, H.dev_i32(path), H.dev_i32(acc), H.dev_i32(cu), H.dev_i32(lens), H.dev_i32(phi), kd, vd,
                                len(ns))
            assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
            for x, t in list(zip(ks, kd)) + list(zip(vs, vd)):
                ref = x if full else T.compact_ring(path, acc, cu, lens, phi, x)
                assert np.array_equal(H.bits_of(t), ref)
    finally:
        ctx.close()


def pool_layers(rng, layers, ns, lens, hkv, d, everything):
    chunks = [-(-L // C) for L in lens]
    cu_chunks = np.concatenate([[0], np.cumsum(chunks)])
    total = int(cu_chunks[-1])
    slot_of = np.full(total, -1)
    kept = np.arange(total) if everything else np.sort(rng.choice(total, total // 2, replace=False))
    slot_of[kept] = rng.permutation(len(kept) + 1)[:len(kept)]
    stores = [[synth.normal_bf16(rng, (total, hkv, C, d)) for _ in range(layers)] for _ in range(2)]
    pools = [[synth.normal_bf16(rng, (len(kept) + 1, hkv, C, d)) for _ in range(layers)] for _ in range(2)]
    return cu_chunks, slot_of, stores, pools


@pytest.mark.parametrize("pinned", [False, True])
@pytest.mark.parametrize("everything", [True, False])
def test_compact_pools(env, everything, pinned):
    """Rows from pool slots and (chunks without one) from the store; paths that cross chunks."""
    H, vfy = env
    hkv, d, layers = 4, 128, 3
    rng = np.random.default_rng(40 + everything)
    ns, lens = [17, 64, 200, 1], [70, 64, 1000, 129]
    cu = np.concatenate([[0], np.cumsum(ns)])
    path, acc = ragged_paths(rng, ns)
    cu_chunks, slot_of, stores, pools = pool_layers(rng, layers, ns, lens, hkv, d, everything)
    ctx = vfy.vfy_create(hkv, hkv, d, max_seqs=len(ns), max_queries_per_seq=200, device=0)
    try:
        sd = [[H.host_bf16(x) if pinned else H.dev_bf16(x) for x in s] for s in stores]
        pd = [[H.dev_bf16(x) for x in p] for p in pools]
        vfy.vfy_compact_full(ctx, H.dev_i32(path), H.dev_i32(acc), H.dev_i32(cu), H.dev_i32(lens), H.dev_i32(cu_chunks),
                             H.dev_i32(slot_of), sd[0], sd[1], len(slot_of), pd[0], pd[1], pd[0][0].shape[0], len(ns))
        torch.cuda.synchronize()
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        for kv in range(2):
            for l in range(layers):
                rs, rp = T.compact_full(path, acc, cu, lens, cu_chunks, slot_of, stores[kv][l], pools[kv][l])
                assert np.array_equal(H.bits_of(sd[kv][l]), rs) and np.array_equal(H.bits_of(pd[kv][l]), rp)
    finally:
        ctx.close()


def test_compact_reports_bad_input(env):
    H, vfy = env
    rng = np.random.default_rng(44)
    ring = synth.normal_bf16(rng, (2, 4, 2048, 128))
    ctx = vfy.vfy_create(4, 4, 128, max_seqs=2, max_queries_per_seq=8, device=0)
    cu, lens, phi = [0, 8, 16], [100, 200], [0, 0]
    try:
        def run(path, acc, cu=cu):
            k, v = H.dev_bf16(ring), H.dev_bf16(ring)
            vfy.vfy_compact_swa(ctx, H.dev_i32(path), H.dev_i32(acc), H.dev_i32(cu), H.dev_i32(lens), H.dev_i32(phi), [k], [v], 2)
            return vfy.vfy_get_status(ctx), H.bits_of(k)
        good = [0, 3, 5] + [-1] * 5
        # entries before their place, and past the block: those rows stay, the others move
        for bad in ([0, 2, 1] + [-1] * 5, [0, 2, 8] + [-1] * 5, [0, 2, -1] + [-1] * 5):
            status, got = run(good + bad, [2, 2])
            assert status == vfy.VFY_EDEVICE_INPUT
            assert np.array_equal(got, T.compact_ring(good + [0, 2], [2, 1], cu, lens, phi, ring))
        # lengths out of range: the sequence stays as it was
        for acc in ([2, 8], [2, -1]):
            status, got = run(good + good, acc)
            assert status == vfy.VFY_EDEVICE_INPUT
            assert np.array_equal(got, T.compact_ring(good + good, [2, 0], cu, lens, phi, ring))
        status, got = run(good + good, [2, 2], [0, 8, 17])    # nine nodes of eight
        assert status == vfy.VFY_EDEVICE_INPUT and np.array_equal(got[1], ring[1])
        # a chunk beyond the store
        pool = synth.normal_bf16(rng, (4, 4, C, 128))
        t = [H.dev_bf16(pool) for _ in range(4)]
        vfy.vfy_compact_full(ctx, H.dev_i32(good), H.dev_i32([2]), H.dev_i32([0, 8]), H.dev_i32([330]), H.dev_i32([0, 6]),
                             H.dev_i32([0, 1, 2, 3, 3, 3]), [t[0]], [t[1]], 4, [t[2]], [t[3]], 4, 1)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        assert all(np.array_equal(H.bits_of(x), pool) for x in t)
    finally:
        ctx.close()


def test_refusals(env):
    H, vfy = env
    ctx = vfy.vfy_create(4, 4, 128, max_seqs=2, max_queries_per_seq=8, device=0)
    i = torch.zeros(64, dtype=torch.int32, device="cuda")
    x = torch.zeros((1, 4, 2048, 128), dtype=torch.bfloat16, device="cuda")
    odd = torch.zeros(4 * 2048 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(1, 4, 2048, 128)
    page = torch.zeros((32, 4, C, 128), dtype=torch.bfloat16)             # pageable host memory
    lg = torch.zeros((16, 8), device="cuda")
    try:
        def swa(ks=[x], vs=[x], seqs=1):
            vfy.vfy_compact_swa(ctx, i, i, i, i, i, ks, vs, seqs)

        def full(hk=[x], seqs=1, slots=32, chunks=32):
            vfy.vfy_compact_full(ctx, i, i, i, i, i, i, hk, [x] * len(hk), chunks, [x] * len(hk), [x] * len(hk), slots, seqs)

        def acc(rows=16, vocab=8, seqs=2):
            vfy.vfy_accept_tree(ctx, lg, vocab, i, i, i, rows, i, i, i, i, seqs)
        for f in (lambda: swa([], []), lambda: swa([odd], [x]), lambda: swa([x] * 65, [x] * 65), lambda: swa(seqs=3),
                  lambda: full([page]), lambda: full([odd]), lambda: full([]), lambda: full([x] * 65), lambda: full(seqs=0),
                  lambda: full(slots=0), lambda: full(chunks=0), lambda: acc(rows=17), lambda: acc(rows=0),
                  lambda: acc(vocab=0), lambda: acc(seqs=3)):
            before = vfy.vfy_launch_count(ctx)
            with pytest.raises(vfy.VfyError) as e:
                f()
            assert e.value.status == vfy.VFY_EINVAL and vfy.vfy_launch_count(ctx) == before
        with pytest.raises(ValueError):
            swa([x], [])
    finally:
        ctx.close()


def test_layers_that_overlap_are_refused(env):
    """The layers of one call move their rows at the same time: a buffer in two places would be moved twice."""
    H, vfy = env
    ctx = vfy.vfy_create(4, 4, 128, max_seqs=2, max_queries_per_seq=8, device=0)
    i = torch.zeros(64, dtype=torch.int32, device="cuda")
    ring = torch.zeros((8, 1, 4, 2048, 128), dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros((8, 32, 4, C, 128), dtype=torch.bfloat16, device="cuda")
    host = torch.zeros((8, 32, 4, C, 128), dtype=torch.bfloat16).pin_memory()
    half = ring.view(-1)[ring[0].numel() // 2:][:ring[0].numel()]          # the end of ring 0, the start of ring 1
    try:
        def swa(ks, vs):
            vfy.vfy_compact_swa(ctx, i, i, H.dev_i32([0, 1]), H.dev_i32([9]), i, ks, vs, 1)

        def full(hk, hv, ks, vs):
            vfy.vfy_compact_full(ctx, i, i, H.dev_i32([0, 1]), H.dev_i32([9]), i, i, hk, hv, 32, ks, vs, 32, 1)
        bad = [lambda: swa([ring[0]], [ring[0]]), lambda: swa([ring[0], ring[0]], [ring[1], ring[2]]),
               lambda: swa([ring[0]], [half]),
               lambda: full([host[0]], [host[1]], [pool[0]], [pool[0]]),
               lambda: full([host[0]], [host[0]], [pool[0]], [pool[1]]),
               lambda: full([host[0], host[1]], [host[2], host[3]], [pool[0], pool[1]], [pool[2], pool[0]])]
        for f in bad:
            before = vfy.vfy_launch_count(ctx)
            with pytest.raises(vfy.VfyError) as e:
                f()
            assert e.value.status == vfy.VFY_EINVAL and vfy.vfy_launch_count(ctx) == before
        swa([ring[k] for k in range(0, 8, 2)], [ring[k] for k in range(1, 8, 2)])
        full(list(host[:4]), list(host[4:]), list(pool[:4]), list(pool[4:]))
        full(list(pool[:2]), list(pool[2:4]), list(pool[4:6]), list(pool[6:]))      # a store on the device
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


def test_offsets_past_the_capacity_are_reported(env):
    """Row offsets that only a 32-bit sum would let pass, and ones past the host bound: reported, nothing written."""
    H, vfy = env
    ctx = vfy.vfy_create(4, 1, 128, max_seqs=1, max_queries_per_seq=64, device=0)
    big = 2 ** 31 - 8
    out = torch.full((64, 8), 77, dtype=torch.int32, device="cuda")
    ring = torch.full((2, 1, 1, 2048, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    o = torch.full((64, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    q, pool = torch.zeros_like(o), torch.zeros((256, 1, C, 128), dtype=torch.bfloat16, device="cuda")
    ids = H.dev_i32(range(256))
    try:
        for cu in ([big, big + 15 - 2 ** 32], [60, 75]):
            cu = H.dev_i32(cu)
            vfy.vfy_tree_plan(ctx, out[:, 0].contiguous(), cu, out[:, 1].contiguous(), out, 1)
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
            vfy.vfy_compact_swa(ctx, ids, H.dev_i32([2]), cu, H.dev_i32([100]), H.dev_i32([0]), [ring[0]], [ring[1]], 1)
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
            vfy.vfy_attend_full_tree(ctx, q, cu, out, pool, pool, 256, ids, ids, H.dev_i32([0, 256]), 256,
                                     H.dev_i32([256 * C]), o, None, 1)       # two row tiles: CTA pairs
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        assert (out == 77).all() and (ring == 3).all() and (o == 3).all()
    finally:
        ctx.close()


def test_a_whole_tree_step_in_one_graph(env):
    """Two sequences, one full and one window layer, three steps of one captured graph: every step's trees,
    drafts and K/V are new, the cache, the lengths and the counts are those the last step left. The
    caches are checked bit for bit after every step, so step t + 1 attends what step t committed."""
    H, vfy = env
    hq, hkv, d, R, W, V, B, N = 16, 4, 128, 2048, 512, 1003, 2, 24
    rng = np.random.default_rng(77)
    lens0 = [500, 127]                                        # committed positions before the first block
    cap = [-(-(L + 3 * N + N) // C) for L in lens0]
    cu_chunks = np.concatenate([[0], np.cumsum(cap)])
    total = int(cu_chunks[-1])
    slot_of = rng.permutation(total)
    ids = np.concatenate([np.arange(c) for c in cap])
    store = [synth.normal_bf16(rng, (total, hkv, C, d)) for _ in range(2)]
    pool = [np.zeros_like(s) for s in store]
    for kv in range(2):
        pool[kv][slot_of] = store[kv]
    ring = [synth.normal_bf16(rng, (B, hkv, R, d)) for _ in range(2)]
    phi = [2000, 5]
    ns = [N, 9]
    cu = np.concatenate([[0], np.cumsum(ns)])
    T_ = int(cu[-1])
    ctx = vfy.vfy_create(hq, hkv, d, window=W, ring_len=R, max_seqs=B, max_queries_per_seq=N, device=0)
    dev = {"q": (T_, hq, d), "kn": (T_, hkv, d), "vn": (T_, hkv, d)}
    t = {k: torch.zeros(s, dtype=torch.bfloat16, device="cuda") for k, s in dev.items()}
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")   # noqa: E731
    t.update(parents=i32(T_), drafts=i32(T_ - B), depth=i32(T_), mask=i32(T_, 8), acc=i32(B), path=i32(T_), bonus=i32(B),
             committed=i32(T_), counts=i32(B, V), lens=i32(B), logits=torch.zeros((T_, V), device="cuda"),
             out=torch.zeros((T_, hq, d), dtype=torch.bfloat16, device="cuda"), lse=torch.zeros((T_, hq), device="cuda"),
             wout=torch.zeros((T_, hq, d), dtype=torch.bfloat16, device="cuda"), wlse=torch.zeros((T_, hq), device="cuda"))
    cud, cuc, sod, idd, cur, phid = (H.dev_i32(a) for a in (cu, cu_chunks, slot_of, ids, cu_chunks, phi))
    sk, sv = (H.host_bf16(s) for s in store)
    pk, pv = (H.dev_bf16(p) for p in pool)
    rk, rv = (H.dev_bf16(r) for r in ring)
    par = [np.array([1.2, 1.5], np.float32), np.array([0.3, 0.1], np.float32), np.array([0.2, 0.4], np.float32)]
    grammar = rng.random((T_, V)) < 0.7
    bits = np.zeros((T_, 32 * -(-V // 32)), np.uint8)
    bits[:, :V] = grammar
    words = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32)).cuda()
    rules = vfy.LogitRules(counts=t["counts"], repetition=H.dev_f32(par[0]), frequency=H.dev_f32(par[1]),
                           presence=H.dev_f32(par[2]), drafts=t["drafts"], tree_mask=t["mask"], grammar=words)

    def step():
        vfy.vfy_tree_plan(ctx, t["parents"], cud, t["depth"], t["mask"], B)
        vfy.vfy_append_full(ctx, t["kn"], t["vn"], cud, t["lens"], cuc, sod, sk, sv, total, pk, pv, total, B)
        vfy.vfy_append_swa(ctx, t["kn"], t["vn"], cud, t["lens"], phid, rk, rv, B)
        vfy.vfy_attend_swa_tree(ctx, t["q"], cud, t["mask"], t["depth"], rk, rv, phid, t["lens"], t["wout"], t["wlse"], B)
        vfy.vfy_attend_full_tree(ctx, t["q"], cud, t["mask"], pk, pv, total, idd, sod, cur, max(cap), t["lens"], t["out"],
                                 t["lse"], B)
        vfy.vfy_process_logits(ctx, t["logits"], V, cud, T_, rules, t["logits"], B)
        vfy.vfy_accept_tree(ctx, t["logits"], V, t["drafts"], t["parents"], cud, T_, t["acc"], t["path"], t["bonus"],
                            t["committed"], B)
        vfy.vfy_compact_swa(ctx, t["path"], t["acc"], cud, t["lens"], phid, [rk], [rv], B)
        vfy.vfy_compact_full(ctx, t["path"], t["acc"], cud, t["lens"], cuc, sod, [sk], [sv], total, [pk], [pv], total, B)
        vfy.vfy_count_tokens(ctx, t["committed"], cud, T_, t["counts"], V, B)

    def bf(name, a):
        t[name].copy_(H.dev_bf16(a))

    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        committed_len, counts = list(lens0), np.zeros((B, V), np.uint32)
        for it in range(3):
            trees = [synth.random_tree(rng, n) for n in ns]
            parents = np.concatenate(trees)
            q, kn, vn = (synth.normal_bf16(rng, dev[k]) for k in ("q", "kn", "vn"))
            lens = [c + n for c, n in zip(committed_len, ns)]
            raw = rng.standard_normal((T_, V), dtype=np.float32) * 3
            sets = [T.ancestors(p.tolist()) for p in trees]
            # the drafts decide the rules' path tokens and the rules the targets: plant matches node by node
            drafts, proc = np.zeros(T_ - B, np.int64), np.zeros((T_, V))
            for b, n in enumerate(ns):
                a = cu[b]
                for i in range(n):
                    if i:
                        tgt = int(proc[a + parents[a + i]].argmax())
                        drafts[a - b + i - 1] = tgt if rng.random() < 0.8 else int(rng.integers(0, V))
                    path = [int(drafts[a - b + j - 1]) for j in sorted(sets[b][i]) if j]
                    proc[a + i], _ = T.process_row(raw[a + i], counts=counts[b], path_tokens=path, repetition=par[0][b],
                                                   frequency=par[1][b], presence=par[2][b], allowed=grammar[a + i])
            for name, a in (("parents", parents), ("drafts", drafts), ("lens", lens)):
                t[name].copy_(H.dev_i32(a))
            bf("q", q), bf("kn", kn), bf("vn", vn)
            t["logits"].copy_(torch.from_numpy(raw))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
            # attention over the appended caches
            store[0], store[1], pool[0], pool[1] = O.append_full(kn, vn, cu, lens, cu_chunks, slot_of, *store, *pool)
            ring[0], ring[1] = O.append_ring(kn, vn, cu, lens, phi, *ring)
            for b, n in enumerate(ns):
                rows, at = slice(cu[b], cu[b + 1]), slice(cu_chunks[b], cu_chunks[b + 1])
                full = T.attend_tree_full_seq(q[rows], sets[b], pool[0], pool[1], ids[at], slot_of[at], lens[b])
                win = T.attend_tree_ring_seq(q[rows], sets[b], T.depths(trees[b].tolist()), ring[0][b], ring[1][b], phi[b],
                                             lens[b], W)
                for (ro, rl, mag), o, l in ((full, "out", "lse"), (win, "wout", "wlse")):
                    g = O.bf16_to_f64(H.bits_of(t[o])[rows])
                    assert np.all(np.abs(g - ro) <= 2.0 ** -8 * (2 * mag + np.abs(ro)) + 7e-4 * mag)
                    assert np.all(np.abs(t[l].cpu().numpy()[rows] - rl) <= 3.1e-4 + np.abs(rl) * 2.0 ** -22)
            # acceptance on the library's own processed logits (rounded alike for planted matches)
            lg = t["logits"].cpu().numpy()
            ref = want(lg, drafts, parents, cu)
            assert [t[k].cpu().tolist() for k in ("acc", "path", "bonus", "committed")] == ref
            assert max(ref[0]) >= 1                           # something moves
            for kv, (s_, p_, r_) in enumerate(((sk, pk, rk), (sv, pv, rv))):
                store[kv], pool[kv] = T.compact_full(ref[1], ref[0], cu, lens, cu_chunks, slot_of, store[kv], pool[kv])
                ring[kv] = T.compact_ring(ref[1], ref[0], cu, lens, phi, ring[kv])
                assert np.array_equal(H.bits_of(s_), store[kv]) and np.array_equal(H.bits_of(p_), pool[kv])
                assert np.array_equal(H.bits_of(r_), ring[kv])
            for b in range(B):
                counts[b] = T.count_tokens(counts[b], ref[3][cu[b]:cu[b + 1]], False)
                committed_len[b] += ref[0][b] + 1
            assert np.array_equal(t["counts"].cpu().numpy().view(np.uint32), counts)
    finally:
        ctx.close()
