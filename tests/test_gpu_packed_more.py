"""4-bit attention where one CTA of the tensor kernel has little, or much, to do. Tolerances are those of test_gpu_packed."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import vfy_oracle as O
from test_gpu_packed import attend, close, env, records  # noqa: F401

pytestmark = pytest.mark.gpu

C = 64


@pytest.mark.parametrize("heads", [(16, 4, 128), (4, 1, 64)])
@pytest.mark.parametrize("seqs", [3, 40])
def test_batches_of_one_tile(env, heads, seqs):  # noqa: F811
    """Sequences of one or two chunks, one of none, whose blocks have more than 16 rows: each CTA's one tile belongs to the
    first softmax group, and the second, which has none, still writes its rows of O into this sequence's partials."""
    H, vfy = env
    hq, hkv, d = heads
    rng = np.random.default_rng([hq, seqs])
    counts = rng.integers(5, 18, seqs)
    counts[0] = 17
    lens = counts + rng.integers(0, 128 - counts.max(), seqs)
    res = -(-lens // C)
    res[1] = 0                                                  # no chunk resident: 0 and -inf
    cu, cu_res, total = H.cu_from_counts(counts), H.cu_from_counts(res), int(res.sum())
    pools = [records(rng, total, hkv, d) for _ in range(2)]
    slots, ids = rng.permutation(total), np.concatenate([np.arange(r) for r in res])
    q = B.to_bf16(rng.standard_normal((int(cu[-1]), hq, d)))
    ctx = vfy.vfy_create(hq, hkv, d, max_seqs=seqs, max_queries_per_seq=17, device=0)
    try:
        first = None
        for splits in (0, 1, 2, 2):                             # (with two, one of them has the tile)
            vfy.vfy_set_splits(ctx, splits, 0)
            got, lse = attend(env, ctx, q, cu, pools, ids, slots, cu_res, lens)
            assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
            first = (got, lse) if first is None else first
            for b in range(seqs):
                at, e = slice(cu[b], cu[b + 1]), slice(cu_res[b], cu_res[b + 1])
                close(got[at], lse[at], *B.attend_packed_seq(O.bf16_to_f64(q[at]), *pools, ids[e], slots[e], int(lens[b])))
            assert np.array_equal(got, first[0])                # one tile is one tile
    finally:
        ctx.close()


@pytest.mark.parametrize("heads", [(4, 1, 128), (4, 1, 64), (2, 2, 128)])
@pytest.mark.parametrize("n", [1, 2, 4, 5, 17])
@pytest.mark.parametrize("order", ["rising", "falling", "random"])
def test_references_that_move(env, heads, n, order):  # noqa: F811
    """Sixteen levels of scores, each 9.5 (log2) above the one before: in rising order every level moves a row's reference,
    which scales its sums and O. The last three levels' values grow as their weights fall, so that each has a share of the
    output that shows. With one split of 128 chunks a warp of the register kernel takes halves of every level, one after the other."""
    H, vfy = env
    hq, hkv, d = heads
    m = 128
    rng = np.random.default_rng([hq, d, n])
    levels = {"rising": np.arange(m), "falling": np.arange(m)[::-1], "random": rng.permutation(m)}[order] // 8
    pools = [np.zeros((m, hkv, 36 * d), np.uint8) for _ in range(2)]
    for p in pools:
        p[..., :32 * d] = rng.integers(0, 256, (m, hkv, 32 * d))
    pools[1][..., :32 * d] &= 0x77                               # V is not negative
    pools[0][..., :C * 16:16] = (pools[0][..., :C * 16:16] & 0xF0) | 2            # channel 0 of K: 1
    k_scale = np.searchsorted(B.E4M3, np.arange(16.0))
    assert np.array_equal(B.E4M3[k_scale], np.arange(16.0))
    pools[0][..., 32 * d:] = k_scale[levels][:, None, None]
    pools[1][..., 32 * d:] = np.array([1] * 13 + [0x7E, 0x38, 1])[levels][:, None, None]   # 2^-9, 448, 1, 2^-9
    q = rng.standard_normal((n, hq, d)) * 0.02
    q[..., 0] = 9.5 * np.log(2.0)
    bits = B.to_bf16(q)
    ref = B.attend_packed_seq(O.bf16_to_f64(bits), *pools, np.arange(m), np.arange(m), m * C, scale=1.0)
    ctx = vfy.vfy_create(hq, hkv, d, max_queries_per_seq=n, softmax_scale=1.0, device=0)
    try:
        for splits in (0, 1, 2):
            vfy.vfy_set_splits(ctx, splits, 0)
            got, lse = attend(env, ctx, bits, [0, n], pools, np.arange(m), np.arange(m), [0, m], [m * C])
            assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
            close(got, lse, *ref)
    finally:
        ctx.close()


@pytest.mark.parametrize("heads", [(4, 1, 128), (4, 1, 64)])
@pytest.mark.parametrize("n", [5, 17, 40])
@pytest.mark.parametrize("m", [151, 200, 263])
def test_many_tiles_of_one_cta(env, heads, n, m):  # noqa: F811
    """More than 64 tiles of one CTA, whose geometry lies in two buffers of 16: the block's chunks, chunks that are not
    there and a chunk behind the sequence among the third and later sixteens, in lists of no order."""
    H, vfy = env
    hq, hkv, d = heads
    rng = np.random.default_rng([d, n, m])
    L = (m - 1) * C + 20
    pools = [records(rng, m, hkv, d) for _ in range(2)]
    ids = np.concatenate([np.arange(m - 2), [m + 5]])            # (one behind the sequence)
    rng.shuffle(ids)
    for place, chunk in ((2 * 33, m - 2), (2 * 50 + 1, m - 1)):  # where the block lies
        ids = np.insert(ids, place, chunk)
    ids = ids[:m + 1]
    slots = np.append(rng.permutation(m), 0)
    slots[ids == m - 1], slots[ids == m + 5] = m - 1, 3
    slots[[2 * 34, 2 * 49, 2 * 65 + 1]] = [-1, m, 2 ** 31 - 1]   # not in the pool
    for side in range(2):                                        # what lies behind the last token may be anything
        for t in range(20, C):
            pools[side][m - 1, :, 32 * d + t * (d // 16):32 * d + (t + 1) * (d // 16)] = 0x7F
    for e in np.flatnonzero(slots == m - 1):
        if ids[e] != m - 1:
            slots[e] = 1
    q = B.to_bf16(rng.standard_normal((n, hq, d)))
    ref = B.attend_packed_seq(O.bf16_to_f64(q), *pools, ids, slots, L)
    ctx = vfy.vfy_create(hq, hkv, d, max_queries_per_seq=n, device=0)
    try:
        for splits in (1, 2, 0):
            vfy.vfy_set_splits(ctx, splits, 0)
            got, lse = attend(env, ctx, q, [0, n], pools, ids, slots, [0, len(ids)], [L])
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
            close(got, lse, *ref)
    finally:
        ctx.close()


@pytest.mark.parametrize("heads", [(16, 4, 128), (4, 1, 64)])
@pytest.mark.parametrize("n", [1, 4, 17, 40])
def test_the_same_bits_from_call_to_call(env, heads, n):  # noqa: F811
    """Whatever other calls left in the workspace, and in a graph."""
    H, vfy = env
    hq, hkv, d = heads
    rng = np.random.default_rng([hq, n])
    m = 90
    pools = [torch.from_numpy(records(rng, m, hkv, d)).cuda() for _ in range(2)]
    ids, cu, cr, ln, ln2 = H.dev_i32(np.arange(m)), H.dev_i32([0, n]), H.dev_i32([0, m]), H.dev_i32([m * C - 5]), H.dev_i32([m * C - 700])
    q, other = [H.dev_bf16(B.to_bf16(rng.standard_normal((n, hq, d)))) for _ in range(2)]
    new = lambda: (torch.empty_like(q), torch.empty((n, hq), device="cuda"))   # noqa: E731
    ctx = vfy.vfy_create(hq, hkv, d, max_queries_per_seq=n, device=0)
    call = lambda x, l, o: vfy.vfy_attend_full_packed(ctx, x, cu, *pools, m, ids, ids, cr, m, l, 1.0, 1.0, *o, 1)   # noqa: E731
    try:
        first, scratch, got = new(), new(), new()
        call(q, ln, first)
        torch.cuda.synchronize()
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                call(other, ln2, scratch)
                call(q, ln, got)
        for i in range(20):
            got[0].fill_(9.0)
            call(other, ln2, scratch) if i % 2 else call(q, ln, scratch)
            call(q, ln, got) if i % 3 else graph.replay()
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()
