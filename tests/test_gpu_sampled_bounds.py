"""Sampled acceptance with row lists that pass the host's bound: what the caller does not have is not read."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from test_gpu_sampled import call, check, env, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu,max_rows,arrays,kept", [
    ([0, 2, 5], 2, "no uniform", []),       # a draft although there are as many rows as sequences
    ([0, 2, 9], 2, "none", []),
    ([0, 1, 9], 2, "no uniform", [0]),      # one row, no draft
    ([0, 3, 99], 3, "all", []),             # two drafts where three rows and two sequences allow one
    ([0, 3, 6, 99], 6, "all", [0]),
    ([0, 3, 6, 10], 9, "all", [0, 1]),      # six drafts allow both
    ([0, 1, 1], 2, "all", [0]),             # one row needs no draft, whatever lies behind it
    ([0, 1, 7], 1, "all", [0]),
])
def test_rows_past_the_bound(env, cu, max_rows, arrays, kept):  # noqa: F811
    """Reported; sequences whose rows and drafts lie within the bound are answered, the others' outputs stay."""
    H, vfy = env
    n = len(cu) - 1
    counts = [cu[b + 1] - cu[b] if b in kept else 1 for b in range(n)]
    c = make(np.random.default_rng([max_rows, *cu]), counts, 300)
    want = B.accept_sampled(**c)
    # logits as far as max_rows, drafts as far as max_rows - n: nothing lies behind them
    rows = np.zeros((max_rows, 300), np.float32)
    for b in kept:
        rows[cu[b]:cu[b + 1]] = c["logits"][c["cu_rows"][b]:c["cu_rows"][b + 1]]
    drafts = max(0, max_rows - n)
    bad = dict(c, logits=rows, cu_rows=np.array(cu), drafts=np.zeros(drafts, np.int32), probs=np.zeros((drafts, 300), np.float32),
               uniform=np.zeros(drafts, np.float32))
    for b in kept:
        to, at, k = cu[b] - b, c["cu_rows"][b] - b, cu[b + 1] - cu[b] - 1
        for name in ("drafts", "probs", "uniform"):
            bad[name][to:to + k] = c[name][at:at + k]
    if arrays == "no uniform":
        bad["drafts"] = np.zeros(1, np.int32)
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=n, max_queries_per_seq=max(8, max_rows), device=0)
    try:
        acc, bonus, com = call(env, ctx, bad)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        for b in range(n):
            if b in kept:
                k = cu[b + 1] - cu[b]
                assert (acc[b], bonus[b]) == (want[0][b], want[1][b])
                assert com[cu[b]:cu[b + 1]] == want[2][c["cu_rows"][b]:c["cu_rows"][b] + k].tolist()
            else:
                assert acc[b] == bonus[b] == -7
        check(env, ctx, c)                                      # the workspace is as it was
    finally:
        ctx.close()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("counts", [[5], [1, 4, 2]])
def test_a_bound_above_the_rows(env, counts, bf16):  # noqa: F811
    """max_rows is a bound: a graph made for the most rows serves steps of fewer."""
    c = make(np.random.default_rng(counts), counts, 5000, bf16)
    ctx = env[1].vfy_create(4, 1, 64, max_seqs=len(counts), max_queries_per_seq=40, device=0)
    try:
        check(env, ctx, c, bf16=bf16, max_rows=40 * len(counts))
    finally:
        ctx.close()
