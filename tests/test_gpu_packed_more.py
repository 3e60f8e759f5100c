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
