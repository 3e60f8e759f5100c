"""Every form of the tree's attention: which kernel and which merge a call takes follows from its sizes, so the sizes here
are chosen for each form. Element by element as tight as two bf16 roundings allow, as a whole as tight as these
two are expected to be, the same bits from call to call.

Elements: |error| <= 2^-8 (A + |o|) + 2^-16 A + 7e-4 A, A = sum_j p_j |v_j| (P to bf16, then O; fp32 scores of 128
products of N(0,1) values).

As a whole: a value in a binade of its own logarithm, rounded to bf16, is off by u^2 / 12 in the mean square, u = 2^-7 of
the binade's start: rho^2 = 2^-14 / 12 * E[1 / m^2] = 2^-14 / 12 * 3 / (8 ln 2) of its square, m log-uniform in
[1, 2). The roundings of P's entries and of O are independent, so the squared error of all outputs is expected to be
rho^2 sum (sum_j p_j^2 v_j^2 + o^2), two terms alike, as E o^2 = sum_j p_j^2 for independent V. The root of the
squared error has to lie within 1.08 of the root of that (some 10^4 outputs spread it by about 1%; it lies below as a
rule, since a row's largest weights may be powers of two, with nothing to round). Partial rows rounded to bf16 before
their merge would add a third such term, sum_s (w_s o_s)^2: 1.22 of the root."""
import math

import numpy as np
import pytest
import torch

from oracle import tree_oracle as T
from oracle import vfy_oracle as O
from speculative_decode_verify_attn_gb300 import synth

pytestmark = pytest.mark.gpu

C = 64
RHO2 = 2.0 ** -14 / 12 * 3 / (8 * math.log(2))


@pytest.fixture(scope="module")
def env():
    import __graft_entry__
    __graft_entry__.build()
    from speculative_decode_verify_attn_gb300 import harness, vfy
    torch.cuda.set_device(0)
    return harness, vfy


class Batch:
    """Sequences of ns[b] nodes and Ls[b] positions, in a pool (slots in random order) and in rings."""

    def __init__(self, seed, ns, Ls, heads, window=512, ring=2048):
        rng = np.random.default_rng(seed)
        self.ns, self.Ls, self.W = ns, Ls, window
        hq, self.hkv, d = self.heads = heads
        self.cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int64)
        rows = int(self.cu[-1])
        self.q = synth.normal_bf16(rng, (rows + 3, hq, d))
        self.trees = [synth.random_tree(rng, n).tolist() if n else [] for n in ns]
        self.sets = [T.ancestors(p) for p in self.trees]
        self.words = np.zeros((rows + 3, 8), np.uint32)
        self.words[:rows] = T.mask_words(sum(self.sets, []))
        self.depth = np.array(sum((T.depths(p) for p in self.trees), []) + [0] * 3)
        chunks = [-(-L // C) for L in Ls]
        self.cu_res = np.concatenate([[0], np.cumsum(chunks)])
        total = int(self.cu_res[-1])
        self.slots, self.ids = rng.permutation(total), np.concatenate([np.arange(m) for m in chunks])
        self.kp, self.vp = (synth.normal_bf16(rng, (total, self.hkv, C, d)) for _ in "kv")
        self.kr, self.vr = (synth.normal_bf16(rng, (len(ns), self.hkv, ring, d)) for _ in "kv")
        self.phi = rng.integers(0, ring, len(ns))

    def context(self, vfy, capacity=None, splits=0):
        ctx = vfy.vfy_create(*self.heads, max_seqs=len(self.ns), max_queries_per_seq=capacity or max(self.ns), window=self.W,
                             device=0)
        vfy.vfy_set_splits(ctx, splits, splits)
        return ctx

    def inputs(self, H):
        self.t = dict(q=H.dev_bf16(self.q), cu=H.dev_i32(self.cu), words=torch.from_numpy(self.words.view(np.int32)).cuda(),
                      depth=H.dev_i32(self.depth), kp=H.dev_bf16(self.kp), vp=H.dev_bf16(self.vp), ids=H.dev_i32(self.ids),
                      slots=H.dev_i32(self.slots), cu_res=H.dev_i32(self.cu_res), L=H.dev_i32(self.Ls),
                      kr=H.dev_bf16(self.kr), vr=H.dev_bf16(self.vr), phi=H.dev_i32(self.phi))

    def run(self, vfy, ctx, window, bound=0):
        t = self.t
        out, lse = torch.full_like(t["q"], 7.0), torch.full(t["q"].shape[:2], 7.0, device="cuda")
        if window:
            vfy.vfy_attend_swa_tree(ctx, t["q"], t["cu"], t["words"], t["depth"], t["kr"], t["vr"], t["phi"], t["L"], out, lse,
                                    len(self.ns))
        else:
            vfy.vfy_attend_full_tree(ctx, t["q"], t["cu"], t["words"], t["kp"], t["vp"], len(self.slots), t["ids"], t["slots"],
                                     t["cu_res"], max(bound, int(np.diff(self.cu_res).max())), t["L"], out, lse, len(self.ns))
        return out, lse

    def expected(self, b, window):
        """Of sequence b: O, LSE, A, and rho^2 (sum_j p_j^2 v_j^2 + o^2) of every output, in fp64."""
        n, L, rows = self.ns[b], self.Ls[b], slice(int(self.cu[b]), int(self.cu[b + 1]))
        hq, hkv, d = self.heads
        q, p0 = O.bf16_to_f64(self.q[rows]), L - n
        pos = np.arange(max(0, p0 - self.W + 1), L) if window else np.arange(L)
        if window:
            at = (pos + self.phi[b]) % self.kr.shape[2]
            k, v = O.bf16_to_f64(self.kr[b][:, at]), O.bf16_to_f64(self.vr[b][:, at])
        else:
            s = self.slots[self.cu_res[b]:self.cu_res[b + 1]]
            k, v = (O.bf16_to_f64(x[s]).transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :L] for x in (self.kp, self.vp))
        see = np.tile(pos < p0, (n, 1))
        for i in range(n):
            if window:
                see[i] &= pos >= p0 + self.depth[rows][i] - self.W + 1
            see[i, [int(p0 + j - pos[0]) for j in self.sets[b][i]]] = True
        o, a, e = (np.zeros((n, hq, d)) for _ in range(3))
        lse = np.zeros((n, hq))
        for g in range(hq):
            h = g // (hq // hkv)
            s = np.where(see, q[:, g] @ k[h].T / math.sqrt(d), -np.inf)
            m = s.max(axis=1, keepdims=True)
            w = np.exp(s - m)
            z = w.sum(axis=1, keepdims=True)
            w /= z
            o[:, g], a[:, g], lse[:, g] = w @ v[h], w @ np.abs(v[h]), (m + np.log(z))[:, 0]
            e[:, g] = RHO2 * ((w * w) @ (v[h] * v[h]) + o[:, g] ** 2)
        return o, lse, a, e

    def check(self, H, out, lse, window, whole=False):
        out, lse = O.bf16_to_f64(H.bits_of(out)), lse.cpu().numpy()
        assert (out[int(self.cu[-1]):] == 7).all() and (lse[int(self.cu[-1]):] == 7).all()
        err, exp = 0.0, 0.0
        for b, n in enumerate(self.ns):
            if not n:
                continue
            rows = slice(int(self.cu[b]), int(self.cu[b + 1]))
            o, l, a, e = self.expected(b, window)
            off = np.abs(out[rows] - o)
            assert np.all(off <= 2.0 ** -8 * (a + np.abs(o)) + (2.0 ** -16 + 7e-4) * a), b
            assert np.all(np.abs(lse[rows] - l) <= 3.1e-4 + np.abs(l) * 2.0 ** -22), b
            err, exp = err + (off ** 2).sum(), exp + e.sum()
        assert not whole or math.sqrt(err / exp) <= 1.08, math.sqrt(err / exp)


# nodes, positions, context's capacity, full layers' bound on resident chunks, splits (0: as the call chooses)
FORMS = {
    "one sequence, a cluster's merge": ([17], [700], 17, 0, 0),
    "one sequence, the combine": ([17], [8192], 17, 0, 0),
    "one sequence, three splits of wide tiles": ([17], [4096], 17, 0, 3),
    "one sequence, one split": ([17], [4096], 17, 0, 1),
    "one sequence, two row tiles": ([64], [2000], 64, 0, 0),
    "one sequence, pairs": ([64], [6000], 64, 256, 0),
    "ragged, below the bound of the pairs": ([17, 0, 200, 1, 64, 33], [1500, 0, 200, 64, 2000, 2900], 200, 0, 0),
    "ragged, pairs of many row tiles": ([17, 0, 200, 1, 64, 33], [1500, 0, 200, 64, 2000, 2900], 200, 256, 0),
    "ragged, pairs of one row tile": ([17, 3, 1, 11, 17], [5000, 900, 1, 70, 3000], 17, 256, 0),
    "ragged, one row tile, split": ([17, 3, 1, 11, 17], [5000, 900, 70, 70, 3000], 17, 0, 0),
}


@pytest.mark.parametrize("heads", [(16, 4, 128), (8, 2, 64)])
@pytest.mark.parametrize("name", FORMS)
def test_full_layers(env, name, heads):
    H, vfy = env
    ns, Ls, capacity, bound, splits = FORMS[name]
    x = Batch(len(name), ns, Ls, heads)
    x.inputs(H)
    ctx = x.context(vfy, capacity, splits)
    try:
        first = x.run(vfy, ctx, False, bound)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        x.check(H, *first, False, whole=True)
        for _ in range(5):
            again = x.run(vfy, ctx, False, bound)
            assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16)) and torch.equal(first[1], again[1])
    finally:
        ctx.close()


@pytest.mark.parametrize("heads", [(16, 4, 128), (8, 2, 64)])
@pytest.mark.parametrize("ns,Ls,capacity,splits", [
    ([17], [5000], 17, 0), ([17], [5000], 17, 20), ([64], [3000], 64, 0), ([17], [600], 256, 0), ([256], [2500], 256, 3),
    ([17, 5, 64, 0, 1, 33, 48], [900, 300, 5000, 0, 1, 70, 1234], 64, 0)])
def test_window_layers(env, ns, Ls, capacity, splits, heads):
    H, vfy = env
    x = Batch(sum(ns), ns, Ls, heads)
    x.inputs(H)
    ctx = x.context(vfy, capacity, splits)
    try:
        first = x.run(vfy, ctx, True)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        x.check(H, *first, True, whole=True)
        for _ in range(5):
            again = x.run(vfy, ctx, True)
            assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16)) and torch.equal(first[1], again[1])
    finally:
        ctx.close()


@pytest.mark.parametrize("bound", [0, 256])
@pytest.mark.parametrize("empty", [(), (31,), (32,), (30, 31, 32, 33), (0, 41), tuple(range(20, 42))])
def test_more_sequences_than_a_warp_has_lanes(env, empty, bound):
    """42 sequences, in the pairs' kernel too, whose work lists run over rounds of 32; some are empty on both sides of
    a round's end."""
    H, vfy = env
    rng = np.random.default_rng(len(empty))
    ns = [0 if b in empty else int(rng.integers(1, 18)) for b in range(42)]
    Ls = [n + int(rng.integers(0, 500)) if n else 0 for n in ns]
    x = Batch(len(empty), ns, Ls, (4, 1, 128))
    x.inputs(H)
    ctx = x.context(vfy, 17)
    try:
        got = x.run(vfy, ctx, False, bound)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        x.check(H, *got, False)
        got = x.run(vfy, ctx, True)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        x.check(H, *got, True)
    finally:
        ctx.close()
