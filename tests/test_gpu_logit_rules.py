"""Logit rules and token counts through the C ABI against the fp64 oracle.

Tolerance: an entry passes one division or product, one product, two subtractions and one addition in
fp32, and its m bias entries m - 1 additions: 4 + m operations, each off by at most 2^-24 of its result,
which is at most the sum of the terms' magnitudes. m is counted from the lists (up to 6 here). Entries
that no rule touches, and the pattern of infinities and NaN, are exact."""
import numpy as np
import pytest
import torch

from oracle import tree_oracle as T
from oracle import vfy_oracle as O
from speculative_decode_verify_attn_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import __graft_entry__
    __graft_entry__.build()
    from speculative_decode_verify_attn_gb300 import harness, vfy
    torch.cuda.set_device(0)
    return harness, vfy


def u32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.uint32).view(np.int32)).cuda()


def check(got, ref, mag, repeats=1):
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(np.isinf(got), np.isinf(ref)) and np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
    fin = np.isfinite(ref)
    assert np.all(np.abs(got[fin] - ref[fin]) <= (4 + max(1, repeats)) * 2.0 ** -24 * mag[fin])


class Case:
    """Rules for a batch of trees, drawn from a seed; `run` calls the library, `want` the oracle."""

    def __init__(self, seed, ns, vocab, *, bf16=False, chain=False, penalties=True, bias=0, grammar=True, indexed=True):
        rng = np.random.default_rng(seed)
        self.ns, self.vocab, self.chain = ns, vocab, chain
        self.cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int64)
        B, R = len(ns), int(self.cu[-1])
        x = rng.standard_normal((R, vocab), dtype=np.float32) * 3
        at = rng.random((R, vocab)) < 0.01
        x[at] = rng.choice(np.array([0.0, -0.0, np.inf, -np.inf, np.nan, 1e38, 1e-38], np.float32), int(at.sum()))
        self.bf16 = bf16
        if bf16:
            self.bits = synth.bf16_bits(x)
            x = O.bf16_to_f64(self.bits).astype(np.float32)
        self.x = x
        self.parents = [np.arange(-1, n - 1) if chain else synth.random_tree(rng, n) for n in ns]
        # drafts from a few tokens only, so that paths repeat them
        few = rng.integers(0, vocab, max(1, max(ns) // 3))
        self.drafts = np.concatenate([rng.choice(few, n - 1) for n in ns]).astype(np.int32)
        self.penalties = penalties
        self.counts = np.where(rng.random((B, vocab)) < 0.2, rng.integers(1, 6, (B, vocab)), 0).astype(np.uint32)
        self.counts |= np.where(rng.random((B, vocab)) < 0.2, T.PROMPT_BIT, 0).astype(np.uint32)
        self.rep = rng.uniform(0.8, 1.5, B).astype(np.float32)
        self.freq = rng.uniform(-0.5, 1, B).astype(np.float32)
        self.pres = rng.uniform(-0.5, 1, B).astype(np.float32)
        self.bias = [[(int(rng.integers(0, vocab)), float(np.float32(rng.uniform(-30, 30)))) for _ in range(bias)] for _ in ns]
        for b in self.bias:
            if len(b) >= 3:
                b[-1] = (b[0][0], b[-1][1])                   # a token listed twice
                b[1] = (b[1][0], -np.inf)
        self.repeats = max([0] + [max(np.bincount([t for t, _ in b])) for b in self.bias if b])
        self.allowed, self.index = None, None
        if grammar:
            n_masks = max(1, R // 2) if indexed else R
            self.allowed = rng.random((n_masks, vocab)) < 0.5
            self.allowed[0] = False                           # lets nothing follow
            self.index = rng.integers(-1, n_masks, R) if indexed else None
            if indexed:
                self.index[0] = 0

    def rules(self, vfy, H):
        kw = {}
        if self.penalties:
            kw.update(counts=u32(self.counts), repetition=H.dev_f32(self.rep), frequency=H.dev_f32(self.freq),
                      presence=H.dev_f32(self.pres), drafts=H.dev_i32(self.drafts if len(self.drafts) else [0]))
            if not self.chain:
                kw["tree_mask"] = u32(np.concatenate([T.mask_words(T.ancestors(p.tolist())) for p in self.parents]))
        if any(self.bias):
            kw.update(cu_bias=H.dev_i32(np.concatenate([[0], np.cumsum([len(b) for b in self.bias])])),
                      bias_token=H.dev_i32([t for b in self.bias for t, _ in b]),
                      bias_value=H.dev_f32([v for b in self.bias for _, v in b]))
        if self.allowed is not None:
            words = -(-self.vocab // 32)
            bits = np.zeros((self.allowed.shape[0], words * 32), np.uint8)
            bits[:, :self.vocab] = self.allowed
            kw["grammar"] = u32(np.packbits(bits, axis=1, bitorder="little").view(np.uint32))
            if self.index is not None:
                kw["mask_index"] = H.dev_i32(self.index)
        return vfy.LogitRules(**kw)

    def logits(self):
        if self.bf16:
            return torch.from_numpy(self.bits.view(np.int16)).cuda().view(torch.bfloat16)
        return torch.from_numpy(self.x).cuda()

    def want(self):
        out, mag = np.zeros(self.x.shape), np.zeros(self.x.shape)
        for b, n in enumerate(self.ns):
            sets = T.ancestors(self.parents[b].tolist())
            for i in range(n):
                row = self.cu[b] + i
                path = [int(self.drafts[self.cu[b] - b + j - 1]) for j in sorted(sets[i]) if j > 0]
                mask = row if self.index is None else self.index[row]
                kw = dict(counts=self.counts[b], path_tokens=path, repetition=self.rep[b], frequency=self.freq[b],
                          presence=self.pres[b]) if self.penalties else {}
                with np.errstate(invalid="ignore", over="ignore"):
                    out[row], mag[row] = T.process_row(
                        self.x[row], bias=self.bias[b],
                        allowed=None if self.allowed is None or mask < 0 else self.allowed[mask], **kw)
        return out, mag


CASES = {
    "one row": dict(ns=[1], vocab=1000),
    "block": dict(ns=[17], vocab=4096),
    "odd vocabulary": dict(ns=[17, 5], vocab=1537, bias=7),
    "vocabulary of one": dict(ns=[3], vocab=1),
    "vocabulary below a word": dict(ns=[4], vocab=31, bias=3),
    "bf16": dict(ns=[9, 33, 1], vocab=2049, bf16=True, bias=40),
    "chain": dict(ns=[17, 3], vocab=1024, chain=True),
    "long chain": dict(ns=[256], vocab=300, chain=True, grammar=False),
    "large trees": dict(ns=[256, 2, 100], vocab=700, bias=300),
    "no penalties": dict(ns=[6, 7], vocab=1025, penalties=False, bias=20),
    "biases only": dict(ns=[6], vocab=5000, penalties=False, bias=600, grammar=False),
    "grammar only": dict(ns=[6], vocab=2048, penalties=False, indexed=False),
    "no rule": dict(ns=[6], vocab=2048, penalties=False, grammar=False),
    "a row each": dict(ns=[1] * 5, vocab=2049, bf16=True, bias=30),
    "a row each, fp32": dict(ns=[1, 1, 1], vocab=4096, bias=3, indexed=False),
    "more sequences than a warp has lanes": dict(ns=[2, 1, 3] * 13, vocab=300, bias=2),
    # enough segments of enough sequences for one CTA to run over all rows of a sequence, more than it stages masks for
    "whole sequences": dict(ns=[40, 1, 2, 33, 70] + [5] * 15, vocab=32001, bf16=True, bias=5),
    "whole sequences, aligned rows": dict(ns=[70, 36, 1, 2] + [5] * 16, vocab=32000, bias=5),
}


@pytest.mark.parametrize("name", CASES)
def test_rules(env, name):
    H, vfy = env
    case = Case(len(name), **CASES[name])
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=len(case.ns), max_queries_per_seq=256, device=0)
    rows = int(case.cu[-1])
    out = torch.full((rows + 2, case.vocab), 77.0, device="cuda")
    try:
        rules = case.rules(vfy, H)
        x = case.logits()
        vfy.vfy_process_logits(ctx, x, case.vocab, H.dev_i32(case.cu), rows, rules, out, len(case.ns))
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
        ref, mag = case.want()
        check(out[:rows].cpu().numpy(), ref, mag, case.repeats)
        assert (out[rows:] == 77).all()
        if name == "no rule":
            assert np.array_equal(out[:rows].cpu().numpy().view(np.uint32), case.x.view(np.uint32))
        # rows further apart than the vocabulary, off the 16-byte grid
        wide = torch.full((rows, case.vocab + 3), 5.0, device="cuda", dtype=x.dtype)
        wide[:, 1:case.vocab + 1] = x
        view = wide[:, 1:case.vocab + 1]
        again = torch.full_like(out, 77.0)
        vfy.vfy_process_logits(ctx, view, case.vocab, H.dev_i32(case.cu), rows, rules, again, len(case.ns))
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int32), again.view(torch.int32))
        if not case.bf16:                                     # in place
            vfy.vfy_process_logits(ctx, x, case.vocab, H.dev_i32(case.cu), rows, rules, x, len(case.ns))
            torch.cuda.synchronize()
            assert torch.equal(out[:rows].view(torch.int32), x.view(torch.int32))
    finally:
        ctx.close()


def test_repeated_biases_add_up_in_list_order(env):
    """1e8 + 1 - 1e8 in fp32: 0 in this order, 1 in others."""
    H, vfy = env
    ctx = vfy.vfy_create(4, 1, 64, max_queries_per_seq=1, device=0)
    n = 700                                                   # entries of one token far apart in the list
    tok = np.arange(n) % 256
    val = np.zeros(n, np.float32)
    for i, v in ((7, 1e8), (7 + 256, 1.0), (7 + 512, -1e8)):
        val[i] = v
    x = torch.zeros((1, 256), device="cuda")
    try:
        rules = vfy.LogitRules(cu_bias=H.dev_i32([0, n]), bias_token=H.dev_i32(tok), bias_value=H.dev_f32(val))
        vfy.vfy_process_logits(ctx, x, 256, H.dev_i32([0, 1]), 1, rules, x, 1)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK and not x.any()
        same = vfy.LogitRules(cu_bias=H.dev_i32([0, 3]), bias_token=H.dev_i32([7, 7, 7]),
                              bias_value=H.dev_f32([1e8, -1e8, 1.0]))
        vfy.vfy_process_logits(ctx, x, 256, H.dev_i32([0, 1]), 1, same, x, 1)
        assert x[0, 7].item() == 1.0
    finally:
        ctx.close()


def test_bad_input_is_reported_and_skipped(env):
    H, vfy = env
    case = Case(3, ns=[4, 4], vocab=512, bias=4)
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=2, max_queries_per_seq=4, device=0)
    ref, mag = case.want()
    try:
        for what in ("draft", "bias", "mask", "rows", "empty"):
            c = Case(3, ns=[4, 4], vocab=512, bias=4)
            cu = c.cu.copy()
            if what == "draft":
                c.drafts = c.drafts.copy()
                c.drafts[3] = 512                              # sequence 1, node 1
            if what == "bias":
                c.bias[1][2] = (-1, 4.0)
            if what == "mask":
                c.index[5] = c.allowed.shape[0]
            if what == "rows":
                cu[2] = 9                                      # more rows than max_rows
            if what == "empty":
                cu = np.array([0, 4, 4])                       # the drafts' packing wants a row of every sequence
            out = torch.full((8, 512), 77.0, device="cuda")
            vfy.vfy_process_logits(ctx, c.logits(), 512, H.dev_i32(cu), 8, c.rules(vfy, H), out, 2)
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT, what
            got = out.cpu().numpy()
            check(got[:4], ref[:4], mag[:4], case.repeats)
            if what in ("rows", "empty"):
                assert (got[4:] == 77).all()
            if what == "mask":
                c.index[5] = -1
                r, m = c.want()
                check(got, r, m, c.repeats)
            if what == "bias":
                del c.bias[1][2]
                r, m = c.want()
                check(got, r, m, c.repeats)
    finally:
        ctx.close()


def test_a_row_each_needs_a_row_each(env):
    """As many rows as sequences, but another sequence has both: reported, and no other row written."""
    H, vfy = env
    case = Case(5, ns=[1, 1], vocab=512)
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=2, max_queries_per_seq=4, device=0)
    try:
        for cu in ([0, 0, 2], [0, 2, 2], [0, 2, 3], [1, 2, 3]):
            out = torch.full((4, 512), 77.0, device="cuda")
            vfy.vfy_process_logits(ctx, case.logits(), 512, H.dev_i32(cu), 2, case.rules(vfy, H), out, 2)
            assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
            assert (out[2:] == 77).all()
    finally:
        ctx.close()


def test_refusals(env):
    H, vfy = env
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=2, max_queries_per_seq=4, device=0)
    x = torch.zeros((10, 64), device="cuda")
    cu = H.dev_i32([0, 4, 8])
    none = vfy.LogitRules()
    i = torch.zeros(64, dtype=torch.int32, device="cuda")
    try:
        def call(logits=x[:8], out=x[:8], vocab=64, rows=8, seqs=2, rules=none):
            vfy.vfy_process_logits(ctx, logits, vocab, cu, rows, rules, out, seqs)
        call()                                                 # in place
        bad = [lambda: call(out=x[1:9]), lambda: call(out=x[2:]), lambda: call(logits=x[:8].view(4, 128), vocab=64),
               lambda: call(rows=9), lambda: call(rows=0), lambda: call(seqs=3), lambda: call(seqs=0),
               lambda: call(logits=x[:8].view(torch.bfloat16)[:, :64], out=x[:8]),
               lambda: call(rules=vfy.LogitRules(cu_bias=i)), lambda: call(rules=vfy.LogitRules(counts=i.view(1, 64), tree_mask=i[1:])),
               lambda: vfy.vfy_count_tokens(ctx, i, cu, 0, i, 64, 1), lambda: vfy.vfy_count_tokens(ctx, i, cu, 8, i, 0, 1),
               lambda: vfy.vfy_count_tokens(ctx, i, cu, 8, i, 64, 3)]
        for f in bad:
            before = vfy.vfy_launch_count(ctx)
            with pytest.raises(vfy.VfyError) as e:
                f()
            assert e.value.status == vfy.VFY_EINVAL and vfy.vfy_launch_count(ctx) == before
        with pytest.raises(ValueError):                        # the counts are for another vocabulary
            call(rules=vfy.LogitRules(counts=torch.zeros((2, 65), dtype=torch.int32, device="cuda")))
        with pytest.raises(ValueError):
            call(rules=vfy.LogitRules(grammar=torch.zeros((8, 3), dtype=torch.int32, device="cuda")))
        with pytest.raises(TypeError):
            call(logits=x[:8].half())
    finally:
        ctx.close()


@pytest.mark.parametrize("vocab,lens", [(1, [1]), (50, [0, 3, 0, 1000]), (1000, [1, 257, 40000])])
def test_counts(env, vocab, lens):
    H, vfy = env
    rng = np.random.default_rng(vocab)
    B = len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    start = rng.integers(0, 5, (B, vocab)).astype(np.uint32)
    tokens = np.concatenate([np.where(rng.random(n) < 0.1, -1, (vocab ** rng.random(n)).astype(np.int64) - 1) for n in lens])
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=B, max_queries_per_seq=4, device=0)
    try:
        for as_prompt in (False, True):
            for reset in (False, True):
                counts = torch.cat([u32(start), u32(start[:1])])
                vfy.vfy_count_tokens(ctx, H.dev_i32(tokens), H.dev_i32(cu), len(tokens), counts, vocab, B,
                                     as_prompt=as_prompt, reset=reset)
                assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
                got = counts.cpu().numpy().view(np.uint32)
                for b in range(B):
                    base = np.zeros_like(start[b]) if reset else start[b]
                    assert np.array_equal(got[b], T.count_tokens(base, tokens[cu[b]:cu[b + 1]], as_prompt))
                assert np.array_equal(got[B], start[0])
    finally:
        ctx.close()


def test_counts_report_bad_tokens(env):
    H, vfy = env
    ctx = vfy.vfy_create(4, 1, 64, max_seqs=1, max_queries_per_seq=4, device=0)
    try:
        counts = torch.zeros((1, 8), dtype=torch.int32, device="cuda")
        vfy.vfy_count_tokens(ctx, H.dev_i32([1, 8, -2, 3]), H.dev_i32([0, 4]), 4, counts, 8, 1)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        assert counts.cpu().tolist() == [[0, 1, 0, 1, 0, 0, 0, 0]]
        vfy.vfy_count_tokens(ctx, H.dev_i32([1, 1, 1, 1]), H.dev_i32([0, 4]), 2, counts, 8, 1)   # more than max_tokens
        assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT and counts[0, 1].item() == 3
    finally:
        ctx.close()
