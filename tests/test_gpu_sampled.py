"""Sampled acceptance against fp64: kept lengths, next tokens and committed tokens are equal, for fp32 and bf16 logits, odd
vocabularies and strides, ragged and single-row sequences, greedy ones, masked, infinite and NaN logits.

A decision is left to the inputs: the oracle says how near its nearest decision was (relative), and inputs nearer than 2^-18
are drawn again before the kernel runs. Its own error is 2^-21 in each of a probability's factors (exponential, sum,
quotient)."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import vfy_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import __graft_entry__
    __graft_entry__.build()
    from speculative_decode_verify_attn_gb300 import harness, vfy
    torch.cuda.set_device(0)
    return harness, vfy


def make(rng, counts, V, bf16=False, probs=True, temps=None, spread=2.0):
    """A batch whose decisions are not near."""
    T, n = sum(counts), len(counts)
    while True:
        x = rng.standard_normal((T, V)) * spread
        x = O.bf16_to_f64(B.to_bf16(x)) if bf16 else x.astype(np.float32)
        near = x + rng.standard_normal((T, V)) * 0.5
        q = np.exp(near - near.max(1, keepdims=True))
        q = (q / q.sum(1, keepdims=True)).astype(np.float32)
        drafts, qs = [], []
        for b, c in enumerate(counts):
            r0 = sum(counts[:b])
            for j in range(c - 1):
                drafts.append(rng.choice(V, p=q[r0 + j] / q[r0 + j].sum(dtype=np.float64)) if V > 1 else 0)
                qs.append(q[r0 + j])
        case = {"logits": x, "temperature": np.float32(temps if temps is not None else rng.uniform(0.3, 1.5, n)),
                "drafts": np.array(drafts, np.int32), "probs": np.array(qs, np.float32).reshape(-1, V) if probs else None,
                "uniform": rng.random(T - n).astype(np.float32), "noise": rng.exponential(size=(n, V)).astype(np.float32),
                "cu_rows": np.concatenate([[0], np.cumsum(counts)])}
        if B.accept_sampled(**case)[3] > 2.0 ** -18:
            return case


def call(env, ctx, c, bf16=False, stride=None, offset=0, max_rows=None):
    H, vfy = env
    T, V = c["logits"].shape
    n = len(c["temperature"])
    x = torch.from_numpy(np.ascontiguousarray(c["logits"], dtype=np.float32)).cuda()
    x = x.bfloat16() if bf16 else x
    if stride is not None:
        wide = torch.full((T * stride + offset,), 1e9, device="cuda", dtype=x.dtype)
        view = wide[offset:].view(T, stride)[:, :V]
        view.copy_(x)
        x = view
    e = lambda k: torch.full((k,), -7, device="cuda", dtype=torch.int32)   # noqa: E731
    acc, bonus, com = e(n + 1), e(n + 1), e(T + 1)
    dev = lambda a, f: None if a is None or not len(a) else f(a)           # noqa: E731
    vfy.vfy_accept_sampled(ctx, x, V, H.dev_f32(c["temperature"]), dev(c["drafts"], H.dev_i32), dev(c["probs"], H.dev_f32),
                           dev(c["uniform"], H.dev_f32), H.dev_f32(c["noise"]), H.dev_i32(c["cu_rows"]),
                           T if max_rows is None else max_rows, acc, bonus, com, n)
    torch.cuda.synchronize()
    assert acc[n] == -7 and bonus[n] == -7 and com[T] == -7
    return acc[:n].cpu().tolist(), bonus[:n].cpu().tolist(), com[:T].cpu().tolist()


def check(env, ctx, c, **kw):
    H, vfy = env
    n, bonus, com, _ = B.accept_sampled(**c)
    got = call(env, ctx, c, **kw)
    assert got == (n.tolist(), bonus.tolist(), com.tolist())
    assert vfy.vfy_get_status(ctx) == vfy.VFY_OK


COUNTS = [[17], [1], [1] * 8, [5, 1, 17, 2, 9], [40, 3]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 1025, 4099, 32000])
@pytest.mark.parametrize("bf16,probs", [(False, True), (True, True), (False, False)])
def test_batches(env, counts, V, bf16, probs):
    rng = np.random.default_rng([len(counts), V, bf16, probs])
    ctx = env[1].vfy_create(4, 1, 64, max_seqs=len(counts), max_queries_per_seq=max(counts), device=0)
    try:
        for k in range(3):
            c = make(rng, counts, V, bf16, probs)
            check(env, ctx, c, bf16=bf16)
    finally:
        ctx.close()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("stride,offset", [(1003, 0), (1008, 0), (1001, 1), (1024, 3), (1001, 7)])
def test_rows_apart_and_at_every_alignment(env, bf16, stride, offset):
    rng = np.random.default_rng([stride, offset])
    ctx = env[1].vfy_create(4, 1, 64, max_seqs=3, max_queries_per_seq=9, device=0)
    try:
        check(env, ctx, make(rng, [9, 1, 4], 1001, bf16), bf16=bf16, stride=stride, offset=offset)
    finally:
        ctx.close()


def test_greedy_sequences_are_vfy_accepts(env):
    """T = 0 gives vfy_accept's result, ties, NaN and rows of -inf included; sampled sequences beside them are not touched."""
    H, vfy = env
    rng = np.random.default_rng(3)
    V, counts = 5000, [6, 9, 1, 12]
    c = make(rng, counts, V, temps=[0.0, 0.8, 0.0, 0.0])
    c["logits"] = c["logits"].copy()
    c["logits"][0, [7, 4000]] = 50.0                            # a tie
    c["logits"][16:18, 333] = np.nan
    c["logits"][18] = -np.inf
    for j in range(3):
        c["drafts"][j] = c["logits"][j].argmax()
    c["drafts"][13:16] = [333, 333, 0]
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=4, max_queries_per_seq=12, device=0)
    try:
        check(env, ctx, c)
        n, bonus, com = call(env, ctx, c)
        rn, rb, rc = H.accept(ctx, c["logits"], c["drafts"], c["cu_rows"])
        for b in (0, 2, 3):
            at = slice(c["cu_rows"][b], c["cu_rows"][b + 1])
            assert (n[b], bonus[b], com[at]) == (rn[b], rb[b], rc[at].tolist())
        assert n[0] >= 1 and n[3] == 3
    finally:
        ctx.close()


def test_masked_infinite_and_nan_logits(env):
    H, vfy = env
    rng = np.random.default_rng(4)
    V = 3000
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=8, max_queries_per_seq=4, device=0)
    try:
        while True:
            c = make(rng, [1, 1, 1, 1, 4, 4, 1, 1], V)
            x = c["logits"]
            x[0, rng.permutation(V)[:V - 3]] = -np.inf          # a grammar that lets three tokens follow
            x[1, :] = -np.inf                                   # nothing may follow: token 0
            x[2, [5, 77, 2999]] = np.inf                        # they share the row
            x[3, rng.permutation(V)[:1500]] = np.nan            # as -inf
            x[4:8] = np.where(rng.random((4, V)) < 0.5, -np.inf, x[4:8])   # a drafted token may be masked
            x[8, :] = -np.inf                                   # the drafted row is empty: refused, token 0
            x[12, :] = -3e38                                    # alike, and far from 0
            x[13, 1:] = -3e38
            if B.accept_sampled(**c)[3] > 2.0 ** -18:
                break
        check(env, ctx, c)
        got = call(env, ctx, c)
        assert got[1][1] == 0 and got[1][2] in (5, 77, 2999) and got[1][7] == 0 and got[0][5] == 0 and got[1][5] == 0
    finally:
        ctx.close()


def test_what_nothing_is_left_of(env):
    """p below q everywhere that can be drawn: p itself is drawn from; no token can be drawn: the row's argmax."""
    H, vfy = env
    rng = np.random.default_rng(5)
    V = 700
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=4, max_queries_per_seq=2, device=0)
    try:
        c = make(rng, [2, 2, 1, 2], V)
        c["uniform"][:] = np.float32(1 - 2.0 ** -24)
        c["probs"][0] = 2.0                                     # more than any p: refused, nothing left
        c["probs"][1] = 2.0
        c["noise"][1] = np.where(np.arange(V) % 3 == 0, 0.0, np.where(np.arange(V) % 3 == 1, np.nan, -1.0))
        c["noise"][2] = np.inf
        c["probs"][2] = 0.0                                     # q(d) = 0: any p(d) > 0 is kept
        check(env, ctx, c)
        got = call(env, ctx, c)
        assert got[1][1] == c["logits"][2].argmax() and got[1][2] == c["logits"][4].argmax() and got[0][3] == 1
    finally:
        ctx.close()


@pytest.mark.parametrize("T", [1e-38, 1e-30, 1e-6, 1e-2, 100.0, 3e38])
def test_extreme_temperatures(env, T):
    rng = np.random.default_rng(6)
    ctx = env[1].vfy_create(4, 1, 64, max_seqs=2, max_queries_per_seq=5, device=0)
    try:
        check(env, ctx, make(rng, [5, 1], 999, temps=[T, T]))
    finally:
        ctx.close()


def test_device_errors(env):
    """Bad tokens, temperatures and rows are reported; the others' results stand."""
    H, vfy = env
    rng = np.random.default_rng(7)
    V = 1200
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=3, max_queries_per_seq=6, device=0)
    try:
        c = make(rng, [3, 3, 3], V)
        good = B.accept_sampled(**c)
        for token in (-1, V, 2 ** 31 - 1):
            bad = dict(c, drafts=c["drafts"].copy())
            bad["drafts"][2] = token                            # the second sequence's first draft: refused, p drawn from
            n, bonus, com, gap = B.accept_sampled(**bad)
            assert gap > 2.0 ** -18 and n[1] == 0
            assert call(env, ctx, bad) == (n.tolist(), bonus.tolist(), com.tolist())
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        for t in (-1.0, float("nan"), float("inf")):
            bad = dict(c, temperature=np.float32([c["temperature"][0], t, c["temperature"][2]]))
            want = B.accept_sampled(**dict(c, temperature=np.float32([c["temperature"][0], 0, c["temperature"][2]])))
            assert call(env, ctx, bad) == tuple(x.tolist() for x in want[:3])
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        # a sequence without rows, rows past max_rows, rows before the first
        for cu, kept in (([0, 3, 3, 6], [0]), ([0, 3, 6, 10], [0, 1]), ([-1, 3, 6, 9], [1, 2]), ([0, 0, 3, 6], [])):
            got = call(env, ctx, dict(c, cu_rows=np.array(cu)))
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
            for b in range(3):
                if b in kept and cu[b] == c["cu_rows"][b]:
                    assert got[0][b] == good[0][b] and got[1][b] == good[1][b]
                elif b not in kept and (cu[b + 1] - cu[b] < 1 or cu[b + 1] > 9 or cu[b] < b):
                    assert got[0][b] == -7 and got[1][b] == -7
        check(env, ctx, c)                                      # the workspace is as it was
    finally:
        ctx.close()


def test_refusals(env):
    H, vfy = env
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=2, max_queries_per_seq=4, device=0)
    f = lambda *s: torch.zeros(s, device="cuda")                # noqa: E731
    i = lambda *s: torch.zeros(s, device="cuda", dtype=torch.int32)   # noqa: E731
    args = dict(logits=f(8, 64), vocab=64, temperature=f(2), drafts=i(6), draft_probs=f(6, 64), uniform=f(6), noise=f(2, 64),
                cu_rows=i(3), max_rows=8, accepted_len=i(2), bonus=i(2), committed=i(8), num_seqs=2)
    try:
        before = vfy.vfy_launch_count(ctx)
        for change in (dict(num_seqs=3), dict(num_seqs=0), dict(max_rows=9), dict(max_rows=0), dict(drafts=None), dict(uniform=None),
                       dict(temperature=None), dict(noise=None), dict(bonus=None), dict(vocab=0, noise=f(2, 0), draft_probs=None)):
            with pytest.raises(vfy.VfyError) as e:
                vfy.vfy_accept_sampled(ctx, **{**args, **change})
            assert e.value.status == vfy.VFY_EINVAL
        for change, kind in ((dict(logits=f(8, 64).double()), TypeError), (dict(logits=f(8, 64).cpu()), TypeError),
                             (dict(logits=f(64, 8).T), ValueError), (dict(logits=f(8, 32)), ValueError),
                             (dict(noise=f(2, 65)), ValueError), (dict(draft_probs=f(6, 63)), ValueError),
                             (dict(noise=f(2, 64).cpu()), TypeError), (dict(drafts=f(6)), TypeError)):
            with pytest.raises(kind):
                vfy.vfy_accept_sampled(ctx, **{**args, **change})
        assert vfy.vfy_launch_count(ctx) == before and vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


def test_a_batch_in_a_graph_behind_the_rules(env):
    """vfy_process_logits and the acceptance captured once, replayed with fresh inputs; drafts and random numbers are
    written by kernels right before (the second kernel reads them before it waits)."""
    H, vfy = env
    rng = np.random.default_rng(8)
    V, counts = 4100, [9, 1, 6]
    T, n = sum(counts), 3
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=n, max_queries_per_seq=9, device=0)
    cases = [make(rng, counts, V) for _ in range(5)]
    keys = ("logits", "temperature", "drafts", "probs", "uniform", "noise")
    src = [{k: torch.from_numpy(np.ascontiguousarray(c[k])).cuda() for k in keys} for c in cases]
    now = {k: torch.empty_like(v) for k, v in src[0].items()}
    nxt = {k: torch.empty_like(v) for k, v in src[0].items()}
    cu = H.dev_i32(cases[0]["cu_rows"])
    out = torch.empty_like(now["logits"])
    acc, bonus, com = [torch.empty(k, device="cuda", dtype=torch.int32) for k in (n, n, T)]
    rules = vfy.LogitRules()

    def step():
        for k in keys:
            now[k].copy_(nxt[k])
        vfy.vfy_process_logits(ctx, now["logits"], V, cu, T, rules, out, n)
        vfy.vfy_accept_sampled(ctx, out, V, now["temperature"], now["drafts"], now["probs"], now["uniform"], now["noise"], cu, T,
                               acc, bonus, com, n)
    try:
        for k in keys:
            nxt[k].copy_(src[0][k])
        step()
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                step()
        for c, s in zip(cases, src):
            for k in keys:
                nxt[k].copy_(s[k])
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            want = B.accept_sampled(**c)
            assert acc.tolist() == want[0].tolist() and bonus.tolist() == want[1].tolist() and com.tolist() == want[2].tolist()
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


def test_draws_follow_the_target(env):
    """First committed tokens of 4096 sequences that share one row: their shares are p's within 5 standard deviations."""
    H, vfy = env
    rng = np.random.default_rng(9)
    N, V = 4096, 7
    ctx = vfy.vfy_create(1, 1, 64, max_seqs=N, max_queries_per_seq=2, max_splits=1, device=0)
    x = np.float32([0.1, 1.0, -0.4, 0.8, 0.0, -2.0, 0.5])
    q = np.float32([0.4, 0.02, 0.2, 0.1, 0.1, 0.08, 0.1])
    p = np.exp(x / np.float64(np.float32(0.9)))
    p /= p.sum()
    c = {"logits": np.repeat(x[None], 2 * N, 0), "temperature": np.full(N, 0.9, np.float32),
         "drafts": rng.choice(V, N, p=q / q.sum(dtype=np.float64)).astype(np.int32), "probs": np.repeat(q[None], N, 0),
         "uniform": rng.random(N).astype(np.float32), "noise": rng.exponential(size=(N, V)).astype(np.float32),
         "cu_rows": np.arange(N + 1) * 2}
    try:
        com = np.array(call(env, ctx, c)[2])[::2]
        share = np.bincount(com, minlength=V) / N
        assert np.all(np.abs(share - p) < 5 * np.sqrt(p * (1 - p) / N))
    finally:
        ctx.close()


@pytest.mark.parametrize("counts,V", [([3, 1], 150001), ([1] * 40, 5000), ([2, 1, 3] * 15, 1001), ([50], 2049), ([1], 1 << 20)])
def test_many_sequences_and_long_vocabularies(env, counts, V):
    """More than 32 sequences, segments of several rounds, more draft rows than a CTA has warps."""
    rng = np.random.default_rng([len(counts), V])
    ctx = env[1].vfy_create(4, 1, 64, max_seqs=len(counts), max_queries_per_seq=max(counts), device=0)
    try:
        for bf16 in (False, True):
            check(env, ctx, make(rng, counts, V, bf16), bf16=bf16)
    finally:
        ctx.close()


@pytest.mark.parametrize("small,large", [(1e-38, 1.0), (1e-37, 3e38), (1.0, 1e37), (1e-40, 1e-39)])
def test_noise_of_every_size(env, small, large):
    """Exponentials whose reciprocals leave fp32's normal range: the token with the smallest time is drawn."""
    rng = np.random.default_rng(5)
    ctx = env[1].vfy_create(4, 1, 64, max_seqs=2, max_queries_per_seq=4, device=0)
    try:
        while True:
            c = make(rng, [4, 1], 500)
            for b in range(2):
                c["noise"][b] = np.float32(large) * np.float32(1 + rng.random(500) * 0.1)
                c["noise"][b, rng.integers(0, 500, 3)] = np.float32(small)
            if B.accept_sampled(**c)[3] > 2.0 ** -18:
                break
        check(env, ctx, c)
    finally:
        ctx.close()


@pytest.mark.parametrize("counts,cu", [([1, 1], [0, 2, 2]), ([1, 1], [0, 0, 2]), ([2, 1], [0, 3, 3]), ([2, 1, 1, 1], [0, 5, 5, 5, 5])])
def test_drafts_that_are_not_there_are_not_read(env, counts, cu):
    """Sequences without rows make others need drafts behind the last one (or any, where there are none): reported, and the
    outputs of both stay."""
    H, vfy = env
    c = make(np.random.default_rng(9), counts, 300)
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=len(counts), max_queries_per_seq=8, device=0)
    try:
        acc, bonus, _ = call(env, ctx, dict(c, cu_rows=np.array(cu)))
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        assert acc == bonus == [-7] * len(counts)
        check(env, ctx, c)
    finally:
        ctx.close()


@pytest.mark.parametrize("V", [300, 9000, 40001])
@pytest.mark.parametrize("bf16", [False, True])
def test_nothing_left_in_any_segment(env, V, bf16):
    """A drafter's q that is nowhere below p, and noise that is none: p is drawn from, or the largest logit taken, by whichever
    CTA comes last."""
    rng = np.random.default_rng([V, bf16])
    ctx = env[1].vfy_create(4, 1, 64, max_seqs=3, max_queries_per_seq=4, device=0)
    try:
        c = make(rng, [4, 1, 2], V, bf16)
        c["probs"][:] = 1.0
        c["uniform"][:] = 0.999
        for kind in range(3):
            if kind == 1:
                c["noise"][1:] = 0.0                            # nothing to draw at all
            if kind == 2:
                c["noise"][:] = np.nan
                c["noise"][0, V // 2] = 1.0                     # one token alone
            want = B.accept_sampled(**c)
            if kind or want[3] > 2.0 ** -18:
                check(env, ctx, c, bf16=bf16)
    finally:
        ctx.close()
