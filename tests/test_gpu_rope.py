"""Rotation and append against fp64: pairs, partial rotation, norms, strided rows, trees, far positions, every
destination, and what is left as it was.

Tolerance: O is one rounding to bf16, half a step (2^-8 of the value), of an fp32 result. That is off by at most 2^-20 of the
pair's length: mean, root, quotient and weight 2^-22, an angle reduced to a turn of at most 1/2 in fp32 2 pi 2^-26, cosine
and sine 2^-23, two products and a sum 2^-23."""
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


def freqs(rot, base=500000.0):
    return (base ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)


def close(got_bits, ref):
    """Rows [T][H][d] of bf16 bits: within half a step and 2^-20 of the largest of the row's pairs."""
    g = O.bf16_to_f64(got_bits)
    size = np.sqrt(2.0) * np.abs(ref).max(-1, keepdims=True)
    assert np.all(np.abs(g - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * size), np.abs(g - ref).max()


def block(rng, T, hq, hkv, d, extra=8):
    """Rows of one projection: q, k, v side by side and `extra` more values, as bits and as views on the device."""
    wide = synth.normal_bf16(rng, (T, (hq + 2 * hkv) * d + extra))
    dev = torch.from_numpy(wide.view(np.int16)).cuda().view(torch.bfloat16)
    cut = np.cumsum([0, hq * d, hkv * d, hkv * d])
    parts = [wide[:, cut[i]:cut[i + 1]].reshape(T, -1, d) for i in range(3)]
    views = [dev[:, cut[i]:cut[i + 1]].unflatten(1, (-1, d)) for i in range(3)]
    return parts, views


def positions(counts, lens, depth=None):
    p0 = np.repeat(np.asarray(lens) - np.asarray(counts), counts)
    inside = np.concatenate([np.arange(n) for n in counts]) if depth is None else depth
    return p0 + inside


HEADS = [(16, 4, 128), (4, 1, 64), (8, 8, 128), (6, 2, 64), (1, 1, 128)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("rot,interleaved", [(None, False), (None, True), (32, False), (24, True), (8, False), (0, False)])
@pytest.mark.parametrize("norm", [False, True])
def test_rows(env, heads, rot, interleaved, norm):
    H, vfy = env
    hq, hkv, d = heads
    rot = d if rot is None else rot
    rng = np.random.default_rng([hq, d, rot, interleaved, norm])
    counts, lens = [17, 1, 0, 5, 33], [262144, 1, 0, 5, 100000]
    T = sum(counts)
    (q, k, _), (qd, kd, _) = block(rng, T, hq, hkv, d)
    inv = freqs(rot) if rot else None
    wq, wk = [synth.normal_bf16(rng, (d,)) if norm else None for _ in range(2)]
    rope = vfy.Rope(None if inv is None else H.dev_f32(inv), rot, interleaved, 1.25, None if wq is None else H.dev_bf16(wq),
                    None if wk is None else H.dev_bf16(wk), eps=1e-5)
    ctx = vfy.vfy_create(hq, hkv, d, max_seqs=5, max_queries_per_seq=33, device=0)
    qo = torch.full((T + 1, hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((T + 1, hkv, d), 9.0, dtype=torch.bfloat16, device="cuda")
    at = positions(counts, lens)
    val = lambda w: None if w is None else O.bf16_to_f64(w)      # noqa: E731
    try:
        cu, ln = H.dev_i32(H.cu_from_counts(counts)), H.dev_i32(lens)
        vfy.vfy_rope(ctx, rope, qd, kd, cu, ln, None, qo, ko, 5)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        rq = B.rope(O.bf16_to_f64(q), at, inv, interleaved, 1.25, val(wq), 1e-5)
        rk = B.rope(O.bf16_to_f64(k), at, inv, interleaved, 1.25, val(wk), 1e-5)
        close(H.bits_of(qo)[:T], rq)
        close(H.bits_of(ko)[:T], rk)
        assert (qo[T] == 9).all() and (ko[T] == 9).all()
        # only keys, only queries, and in place: the same bits
        ko2, qc = torch.empty_like(ko), qd.contiguous()
        vfy.vfy_rope(ctx, rope, None, kd, cu, ln, None, None, ko2, 5)
        vfy.vfy_rope(ctx, rope, qc, None, cu, ln, None, qc, None, 5)
        assert torch.equal(ko2[:T], ko[:T]) and torch.equal(qc, qo[:T])
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


def test_far_positions(env):
    """Positions up to 2^31 - 2 with frequencies up to 1: the angle is reduced in 64 bits (2^31 2^-53 radians off)."""
    H, vfy = env
    rng = np.random.default_rng(1)
    counts, lens = [2, 2, 2], [2 ** 31 - 1, 2 ** 24 + 3, 999999937]
    (q, k, _), (qd, kd, _) = block(rng, 6, 2, 1, 64)
    inv = freqs(64, 10000.0)
    ctx = vfy.vfy_create(2, 1, 64, max_seqs=3, max_queries_per_seq=2, device=0)
    qo, ko = torch.empty((6, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((6, 1, 64), dtype=torch.bfloat16, device="cuda")
    try:
        vfy.vfy_rope(ctx, vfy.Rope(H.dev_f32(inv)), qd, kd, H.dev_i32([0, 2, 4, 6]), H.dev_i32(lens), None, qo, ko, 3)
        at = positions(counts, lens)
        close(H.bits_of(qo), B.rope(O.bf16_to_f64(q), at, inv))
        close(H.bits_of(ko), B.rope(O.bf16_to_f64(k), at, inv))
    finally:
        ctx.close()


@pytest.mark.parametrize("seqs", [1, 32, 33, 70, 1100])
def test_many_sequences(env, seqs):
    """The search for a row's sequence: one and several rounds of 32, empty sequences among them."""
    H, vfy = env
    rng = np.random.default_rng(seqs)
    counts = rng.integers(0, 4, seqs)
    counts[-1] = 2
    lens = counts + rng.integers(0, 5000, seqs)
    T = int(counts.sum())
    (q, _, _), (qd, _, _) = block(rng, T, 1, 1, 64)
    inv = freqs(64)
    ctx = vfy.vfy_create(1, 1, 64, max_seqs=seqs, max_queries_per_seq=3, max_splits=1, device=0)
    qo = torch.empty((T, 1, 64), dtype=torch.bfloat16, device="cuda")
    try:
        vfy.vfy_rope(ctx, vfy.Rope(H.dev_f32(inv)), qd, None, H.dev_i32(H.cu_from_counts(counts)), H.dev_i32(lens), None, qo, None, seqs)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        close(H.bits_of(qo), B.rope(O.bf16_to_f64(q), positions(counts, lens), inv))
    finally:
        ctx.close()


@pytest.mark.parametrize("heads", [(16, 4, 128), (4, 2, 64)])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("pinned", [False, True])
def test_append_full(env, heads, tree, pinned):
    """K rotated and V as it is in the store and, where resident, the pool: bit for bit the rows that vfy_rope gives.
    Everything else stays, a token whose chunk the store lacks is reported and gets its queries."""
    H, vfy = env
    hq, hkv, d = heads
    rng = np.random.default_rng([hq, tree, pinned])
    counts, lens = [20, 7, 3], [150, 64, 200]
    T, chunks = sum(counts), [3, 1, 3]                          # the last sequence needs four: its last tokens have no place
    (q, k, v), (qd, kd, vd) = block(rng, T, hq, hkv, d)
    depth = np.concatenate([np.sort(rng.integers(0, n, n)) for n in counts]) if tree else None
    inv = freqs(d // 2)
    rope = vfy.Rope(H.dev_f32(inv), k_norm=H.dev_bf16(synth.normal_bf16(rng, (d,))))
    cu_chunks = H.cu_from_counts(chunks)
    slot_of = np.array([-1, 4, 0, 2, 5, -1, 3], dtype=np.int32)
    ctx = vfy.vfy_create(hq, hkv, d, max_seqs=3, max_queries_per_seq=20, device=0)
    sk, sv = [synth.normal_bf16(rng, (7, hkv, C, d)) for _ in range(2)]
    pk, pv = [synth.normal_bf16(rng, (6, hkv, C, d)) for _ in range(2)]
    put = (lambda x: H.host_bf16(x)) if pinned else (lambda x: H.dev_bf16(x))   # noqa: E731
    skd, svd, pkd, pvd = put(sk), put(sv), H.dev_bf16(pk), H.dev_bf16(pv)
    qo, qr = [torch.zeros((T, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kr = torch.zeros((T, hkv, d), dtype=torch.bfloat16, device="cuda")
    try:
        cu, ln = H.dev_i32(H.cu_from_counts(counts)), H.dev_i32(lens)
        dep = None if depth is None else H.dev_i32(depth)
        vfy.vfy_rope(ctx, rope, qd, kd, cu, ln, dep, qr, kr, 3)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        # the store ends where the third sequence's tokens begin that have no chunk
        vfy.vfy_rope_append_full(ctx, rope, qd, kd, vd, cu, ln, dep, H.dev_i32(cu_chunks), H.dev_i32(slot_of), skd, svd, 7,
                                 pkd, pvd, 6, qo, 3)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        assert torch.equal(qo, qr)
        at = positions(counts, lens)
        rk = B.rope(O.bf16_to_f64(k), at if depth is None else positions(counts, lens, depth), inv, norm=O.bf16_to_f64(H.bits_of(rope.tensors[2])), eps=1e-6)
        close(H.bits_of(kr), rk)
        kb = H.bits_of(kr)
        seq = np.repeat(np.arange(3), counts)
        for t in range(T):
            c = cu_chunks[seq[t]] + at[t] // C
            if c >= 7:
                continue
            sk[c, :, at[t] % C], sv[c, :, at[t] % C] = kb[t], v[t]
            if slot_of[c] >= 0:
                pk[slot_of[c], :, at[t] % C], pv[slot_of[c], :, at[t] % C] = kb[t], v[t]
        for got, want in ((skd, sk), (svd, sv), (pkd, pk), (pvd, pv)):
            assert np.array_equal(H.bits_of(got), want)
    finally:
        ctx.close()


@pytest.mark.parametrize("heads", [(16, 4, 128), (4, 2, 64)])
def test_append_swa(env, heads):
    H, vfy = env
    hq, hkv, d = heads
    rng = np.random.default_rng(hq)
    counts, lens, phi, R = [33, 1, 9], [5000, 1, 70], [-37, 2047, 5 * 2048 + 1990], 2048
    T = sum(counts)
    (q, k, v), (qd, kd, vd) = block(rng, T, hq, hkv, d)
    rope = vfy.Rope(H.dev_f32(freqs(d)), interleaved=True)
    depth = np.concatenate([np.arange(n) // 2 for n in counts])
    ctx = vfy.vfy_create(hq, hkv, d, max_seqs=3, max_queries_per_seq=33, ring_len=R, device=0)
    rk, rv = [synth.normal_bf16(rng, (3, hkv, R, d)) for _ in range(2)]
    rkd, rvd = H.dev_bf16(rk), H.dev_bf16(rv)
    qo, qr = [torch.zeros((T, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kr = torch.zeros((T, hkv, d), dtype=torch.bfloat16, device="cuda")
    try:
        cu, ln, dep = H.dev_i32(H.cu_from_counts(counts)), H.dev_i32(lens), H.dev_i32(depth)
        vfy.vfy_rope(ctx, rope, qd, kd, cu, ln, dep, qr, kr, 3)
        vfy.vfy_rope_append_swa(ctx, rope, qd, kd, vd, cu, ln, dep, H.dev_i32(phi), rkd, rvd, qo, 3)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        assert torch.equal(qo, qr)
        kb, at, seq = H.bits_of(kr), positions(counts, lens), np.repeat(np.arange(3), counts)
        for t in range(T):
            place = (at[t] + phi[seq[t]]) % R
            rk[seq[t], :, place], rv[seq[t], :, place] = kb[t], v[t]
        assert np.array_equal(H.bits_of(rkd), rk) and np.array_equal(H.bits_of(rvd), rv)
    finally:
        ctx.close()


def test_rows_out_of_range_are_reported_and_left(env):
    H, vfy = env
    rng = np.random.default_rng(2)
    (_, _, _), (qd, kd, _) = block(rng, 8, 2, 1, 64)
    ctx = vfy.vfy_create(2, 1, 64, max_seqs=2, max_queries_per_seq=4, device=0)
    rope = vfy.Rope(H.dev_f32(freqs(64)))
    try:
        # too many rows; a sequence shorter than its block; rows that start before the first
        for cu, ln, kept in (([0, 5, 8], [9, 9], range(5, 8)), ([0, 4, 8], [9, 3], range(0, 4)), ([-2, 2, 6], [9, 9], range(2, 6))):
            qo = torch.full((8, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
            ko = torch.full((8, 1, 64), 9.0, dtype=torch.bfloat16, device="cuda")
            vfy.vfy_rope(ctx, rope, qd, kd, H.dev_i32(cu), H.dev_i32(ln), None, qo, ko, 2)
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
            written = [t for t in range(8) if not (qo[t] == 9).all()]
            assert written == list(kept) and all((ko[t] == 9).all() for t in range(8) if t not in kept)
    finally:
        ctx.close()


def test_refusals(env):
    H, vfy = env
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    ctx = vfy.vfy_create(4, 2, 64, max_seqs=2, max_queries_per_seq=4, device=0)
    cu, ln, inv = H.dev_i32([0, 4, 8]), H.dev_i32([9, 9]), H.dev_f32(freqs(64))
    q, k = z(8, 4, 64), z(8, 2, 64)
    rope = vfy.Rope(inv)

    def refused(call, kind=None):
        with pytest.raises(kind or vfy.VfyError) as e:
            call()
        if kind is None:
            assert e.value.status == vfy.VFY_EINVAL

    try:
        before = vfy.vfy_launch_count(ctx)
        for bad in (vfy.Rope(H.dev_f32(freqs(60)), 60), vfy.Rope(H.dev_f32(freqs(128)), 128), vfy.Rope(inv, eps=-1.0),
                    vfy.Rope(inv, eps=float("nan")), vfy.Rope(inv, attention_factor=float("inf"))):
            refused(lambda: vfy.vfy_rope(ctx, bad, q, k, cu, ln, None, q, k, 2))
        refused(lambda: vfy.vfy_rope(ctx, rope, q, k, cu, ln, None, None, k, 2))
        refused(lambda: vfy.vfy_rope(ctx, rope, None, None, cu, ln, None, None, None, 2))
        refused(lambda: vfy.vfy_rope(ctx, rope, q, k, cu, ln, None, q, k, 3))
        refused(lambda: vfy.vfy_rope(ctx, rope, q, k, cu, ln, None, q, k, 0))
        wide = z(8, 260)                                        # rows 260 values apart: no multiple of 8
        refused(lambda: vfy.vfy_rope(ctx, rope, wide[:, :256], k, cu, ln, None, q, k, 2))
        wide = z(8, 264)                                        # in place, but rows further apart than packed ones
        assert vfy.lib().vfy_rope(ctx.handle, rope.at, wide.data_ptr(), 264, None, 0, cu.data_ptr(), ln.data_ptr(), None,
                                  wide.data_ptr(), None, 2, None) == vfy.VFY_EINVAL
        refused(lambda: vfy.vfy_rope(ctx, rope, z(8, 5, 64), k, cu, ln, None, q, k, 2), ValueError)
        refused(lambda: vfy.vfy_rope(ctx, rope, z(64, 4, 8).permute(2, 1, 0), k, cu, ln, None, q, k, 2), ValueError)
        refused(lambda: vfy.vfy_rope(ctx, rope, q.float(), k, cu, ln, None, q, k, 2), TypeError)
        refused(lambda: vfy.vfy_rope(ctx, rope, q.cpu(), k, cu, ln, None, q, k, 2), TypeError)
        refused(lambda: vfy.vfy_rope(ctx, vfy.Rope(inv, q_norm=z(128)), q, k, cu, ln, None, q, k, 2), ValueError)
        pageable = torch.zeros((2, 2, C, 64), dtype=torch.bfloat16)
        pool, ids = z(2, 2, C, 64), H.dev_i32([0, 1])
        refused(lambda: vfy.vfy_rope_append_full(ctx, rope, q, k, k, cu, ln, None, cu, ids, pageable, pageable, 2, pool, pool, 2, q, 2))
        refused(lambda: vfy.vfy_rope_append_full(ctx, rope, q, None, k, cu, ln, None, cu, ids, pool, pool, 2, pool, pool, 2, q, 2))
        refused(lambda: vfy.vfy_rope_append_swa(ctx, rope, q, k, None, cu, ln, None, ids, pool, pool, q, 2))
        assert vfy.vfy_launch_count(ctx) == before
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


@pytest.mark.parametrize("window", [False, True])
def test_layer_in_a_graph(env, window):
    """Rotation with append, then the layer's attention, captured once and replayed over a growing context: the replay
    gives what the attention of separately rotated rows gives."""
    H, vfy = env
    hq, hkv, d, n = 8, 2, 128, 5
    rng = np.random.default_rng(window)
    ctx = vfy.vfy_create(hq, hkv, d, max_seqs=1, max_queries_per_seq=n, window=64, ring_len=256, device=0)
    rope = vfy.Rope(H.dev_f32(freqs(d)), q_norm=H.dev_bf16(synth.normal_bf16(rng, (d,))), k_norm=H.dev_bf16(synth.normal_bf16(rng, (d,))))
    _, (qd, kd, vd) = block(rng, n, hq, hkv, d)
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    pool, store, ring = [z(4, hkv, C, d) for _ in range(2)], [z(4, hkv, C, d) for _ in range(2)], [z(1, hkv, 256, d) for _ in range(2)]
    cu, ln, phi = H.dev_i32([0, n]), H.dev_i32([n]), H.dev_i32([100])
    ids, cu_c = H.dev_i32(np.arange(4)), H.dev_i32([0, 4])
    q, out, want, lse = z(n, hq, d), z(n, hq, d), z(n, hq, d), torch.zeros((n, hq), device="cuda")

    def step(append, o):
        if window:
            append and vfy.vfy_rope_append_swa(ctx, rope, qd, kd, vd, cu, ln, None, phi, *ring, q, 1)
            vfy.vfy_attend_swa(ctx, q, cu, *ring, phi, ln, o, lse, 1)
        else:
            append and vfy.vfy_rope_append_full(ctx, rope, qd, kd, vd, cu, ln, None, cu_c, ids, *store, 4, *pool, 4, q, 1)
            vfy.vfy_attend_full(ctx, q, cu, *pool, 4, ids, ids, cu_c, 4, ln, o, lse, 1)
    try:
        step(True, out)
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                step(True, out)
        keys, vals = [], []
        for i in range(1, 8):
            ln.fill_(n * i)
            fresh = synth.normal_bf16(rng, (n, (hq + 2 * hkv) * d + 8))
            qd._base.copy_(torch.from_numpy(fresh.view(np.int16)).cuda().view(torch.bfloat16))
            graph.replay()
            torch.cuda.synchronize()
            k = z(n, hkv, d)
            vfy.vfy_rope(ctx, rope, qd, kd, cu, ln, None, q, k, 1)
            keys.append(k.clone())
            vals.append(vd.clone())
            K, V = torch.cat(keys).transpose(0, 1), torch.cat(vals).transpose(0, 1)
            if window:
                at = (torch.arange(n * i, device="cuda") + 100) % 256
                ring2 = [z(1, hkv, 256, d) for _ in range(2)]
                ring2[0][0, :, at], ring2[1][0, :, at] = K, V
                vfy.vfy_attend_swa(ctx, q, cu, *ring2, phi, ln, want, lse, 1)
            else:
                flat = [torch.nn.functional.pad(x, (0, 0, 0, 256 - n * i)).view(hkv, 4, C, d).transpose(0, 1).contiguous() for x in (K, V)]
                vfy.vfy_attend_full(ctx, q, cu, *flat, 4, ids, ids, cu_c, 4, ln, want, lse, 1)
            torch.cuda.synchronize()
            assert torch.equal(out, want), i
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


@pytest.mark.parametrize("heads", [(16, 4, 128), (4, 1, 64), (6, 3, 64), (1, 1, 128)])
@pytest.mark.parametrize("rot,interleaved", [(None, False), (None, True), (24, True), (8, False)])
def test_a_token_a_warp(env, heads, rot, interleaved):
    """A context with room for many tokens takes one token a warp instead of a CTA: the same bits in every destination,
    with tokens that no multiple of eight divides, and the same rows left as they were."""
    H, vfy = env
    hq, hkv, d = heads
    rot = d if rot is None else rot
    rng = np.random.default_rng([hq, d, rot, interleaved])
    counts, lens, R = [17, 1, 0, 5, 30], [262144, 1, 0, 130, 1000], 512
    T = sum(counts)
    (_, _, _), (qd, kd, vd) = block(rng, T, hq, hkv, d)
    rope = vfy.Rope(H.dev_f32(freqs(rot)), rot, interleaved, 0.75, H.dev_bf16(synth.normal_bf16(rng, (d,))),
                    H.dev_bf16(synth.normal_bf16(rng, (d,))))
    chunks = [-(-x // C) for x in lens]
    cu, ln, phi = H.dev_i32(H.cu_from_counts(counts)), H.dev_i32(lens), H.dev_i32([3, -5, 0, 700, 255])
    dep = H.dev_i32(np.concatenate([np.arange(n) // 2 for n in counts]))
    # (only the block's chunks: the first sequence's others lie before the store)
    first = lens[0] // C - 1
    cu_c = H.dev_i32(np.concatenate([[-first], np.cumsum(chunks)[:-1] - first]))
    n_chunks = sum(chunks) - first
    slot_of = H.dev_i32(rng.permutation(n_chunks + 3)[:n_chunks] - 3)
    results = []
    for cap in (33, 300):
        full = lambda *s: torch.full(s, 9.0, dtype=torch.bfloat16, device="cuda")   # noqa: E731
        ctx = vfy.vfy_create(hq, hkv, d, max_seqs=5, max_queries_per_seq=cap, window=64, ring_len=R, device=0)
        outs = [full(T + 9, hq, d), full(T + 9, hkv, d), full(T + 9, hq, d), *[full(n_chunks, hkv, C, d) for _ in range(4)],
                full(T + 9, hq, d), *[full(5, hkv, R, d) for _ in range(2)]]
        try:
            vfy.vfy_rope(ctx, rope, qd, kd, cu, ln, dep, *outs[:2], 5)
            vfy.vfy_rope_append_full(ctx, rope, qd, kd, vd, cu, ln, dep, cu_c, slot_of, *outs[3:5], n_chunks, *outs[5:7], n_chunks, outs[2], 5)
            vfy.vfy_rope_append_swa(ctx, rope, qd, kd, vd, cu, ln, dep, phi, *outs[8:], outs[7], 5)
            assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        finally:
            ctx.close()
        assert all((o[T:] == 9).all() for o in (outs[0], outs[1], outs[2], outs[7]))
        results.append(outs)
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.equal(results[0][0], results[0][2]) and torch.equal(results[0][0], results[0][7])
