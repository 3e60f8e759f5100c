"""Cases that time the tree-speculation operators: verification of a tree of drafted tokens.

A drafter may propose a tree instead of a chain: node 0 of a sequence's block is the last committed
token, node j > 0 a drafted token whose parent is an earlier node. One batched target forward
verifies every node; the path the target itself would emit is committed. The operators:

  tree attention    every node attends the cache before the block and, inside the block, its own
                    ancestors (a row mask); over the chunk pool ("full") and the position ring
                    ("swa"). A drafter whose trees change every step also builds the masks on the
                    GPU every step ("dynamic"); a fixed tree's masks are kept ("static").
  logit processing  penalties for tokens that the sequence (and the node's own path) holds already,
                    biases and grammar masks, over every row of the block ("logits"); and the token
                    counts behind the penalties, built from the prompts of new requests ("first").
  tree acceptance   argmax of every row, then the walk from the root along drafted children that
                    equal the target's token ("accept").
  path compaction   the accepted path's K/V rows moved next to the committed prefix, in the rings
                    or in the pools and the chunk store of all layers ("rings", "pools").

`run` computes each in plain torch where `own` is false and calls the library where it is true.
"""
import math
import random

import numpy as np
import torch

own = False

CHUNK = 64
WORDS = 8            # 32-bit words of a node's row mask: 256 nodes
WINDOW, RING = 512, 2048


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def _attention(op, name, seqs, nodes, context, chunks=0, ragged=False, dynamic=False, heads=(16, 4, 128)):
    return {"name": name, "op": op, "seqs": seqs, "nodes": nodes, "context": context, "chunks": chunks,
            "ragged": ragged, "dynamic": dynamic, "q_heads": heads[0], "kv_heads": heads[1], "dim": heads[2]}


def listed():
    return [
        # One sequence at 256K with an 8K resident pool and a fixed tree of 17 nodes: one full layer.
        _attention("full", "full_static17_8k", 1, 17, 262144, chunks=128),
        # The same context all resident on the GPU and a 64-node tree: the largest stream.
        _attention("full", "full_static64_256k", 1, 64, 262144),
        # A serving batch whose drafter grows a new tree for every sequence: masks and first layer.
        _attention("full", "full_dynamic_ragged8", 8, 48, 48000, ragged=True, dynamic=True),
        # One window layer of one sequence, fixed tree: where latency counts.
        _attention("swa", "swa_static17", 1, 17, 262144),
        # One window layer of a batch with new trees.
        _attention("swa", "swa_dynamic_ragged8", 8, 64, 48000, ragged=True, dynamic=True),
        # New requests: count the prompts, then the rules on each request's first row of logits.
        {"name": "first_tokens8", "op": "first", "seqs": 8, "prompt": 32768, "vocab": 131072, "bf16": True},
        # One block of 17 rows with a grammar, as before every acceptance.
        {"name": "logits_block17", "op": "logits", "seqs": 1, "nodes": 17, "ragged": False, "vocab": 131072,
         "bf16": False, "grammar": True, "biases": 32},
        # A batch of trees; bf16 logits, odd vocabulary, half of the requests without a grammar.
        {"name": "logits_batch16", "op": "logits", "seqs": 16, "nodes": 33, "ragged": True, "vocab": 100003,
         "bf16": True, "grammar": True, "biases": 300},
        # Acceptance of one fixed tree.
        {"name": "accept_tree17", "op": "accept", "seqs": 1, "nodes": 17, "ragged": False, "vocab": 131072},
        # Acceptance of a batch of 64-node trees, odd vocabulary.
        {"name": "accept_batch16", "op": "accept", "seqs": 16, "nodes": 64, "ragged": True, "vocab": 32001},
        # The 30 window layers' rings of one sequence after an acceptance.
        {"name": "compact_rings30", "op": "rings", "seqs": 1, "nodes": 17, "layers": 30, "kv_heads": 4, "dim": 128},
        # The 10 full layers' pools and chunk stores of a batch.
        {"name": "compact_pools10", "op": "pools", "seqs": 8, "nodes": 48, "layers": 10, "kv_heads": 4, "dim": 128,
         "context": 8000},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["full", "full", "swa", "first", "logits", "accept", "rings", "pools"])
    seqs = _log(rng, 1, 16)
    if op in ("full", "swa"):
        heads = rng.choice([(16, 4, 128), (4, 1, 64), (8, 8, 128), (32, 4, 128), (16, 2, 64)])
        nodes = _log(rng, 1, 256)
        # rows x keys and K/V elements stay within the largest listed case
        context = _log(rng, nodes + 1, 262144)
        context = min(context, 64 * 16 * 262144 // (nodes * heads[0] * seqs), 4 * 128 * 262144 // (heads[1] * heads[2] * seqs))
        context = max(context, nodes)
        chunks = _log(rng, 1, 512) if op == "full" and rng.random() < 0.4 else 0
        return {k: v for k, v in _attention(op, "", seqs, nodes, context, chunks, seqs > 1, rng.random() < 0.5,
                                            heads).items() if k != "name"}
    vocab = rng.choice([131072, 32000, 100003, _log(rng, 1000, 131072)])
    if op == "first":
        return {"op": op, "seqs": seqs, "prompt": _log(rng, 1, 131072), "vocab": vocab, "bf16": rng.random() < 0.5}
    nodes = _log(rng, 1, 64)
    if op == "logits":
        return {"op": op, "seqs": seqs, "nodes": nodes, "ragged": rng.random() < 0.5, "vocab": vocab,
                "bf16": rng.random() < 0.5, "grammar": rng.random() < 0.6, "biases": rng.choice([0, 1, 32, 300])}
    if op == "accept":
        return {"op": op, "seqs": seqs, "nodes": nodes, "ragged": rng.random() < 0.5, "vocab": vocab}
    case = {"op": op, "seqs": min(seqs, 8), "nodes": max(3, nodes), "layers": _log(rng, 1, 30 if seqs == 1 else 10),
            "kv_heads": rng.choice([1, 4, 8]), "dim": rng.choice([64, 128])}
    if op == "pools":
        case["context"] = _log(rng, 200, 8000)
    return case


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=dtype))).cuda()


def _cu(counts):
    return np.concatenate([[0], np.cumsum(np.asarray(counts, dtype=np.int64))])


def _spread(rng, n, lo, hi):
    """n whole numbers of [lo, hi], hi among them."""
    got = rng.integers(lo, hi + 1, n)
    got[rng.integers(0, n)] = hi
    return [int(x) for x in got]


def _lengths(case):
    """Nodes and context (or prompt) lengths of the sequences: the case's own, whatever the seed."""
    rng = np.random.default_rng([case["seqs"], case.get("nodes", 1), case.get("context", 0), case.get("prompt", 0)])
    B, n, c = case["seqs"], case.get("nodes", 1), case.get("context", 0)
    if case["op"] == "first":
        return [1] * B, _spread(rng, B, max(1, case["prompt"] // 4), case["prompt"])
    nodes = _spread(rng, B, max(1, n // 8), n) if case.get("ragged") else [n] * B
    lens = _spread(rng, B, max(1, c // (12 if case.get("ragged") else 2)), c) if c and B > 1 else [c] * B
    return nodes, [max(x, k) for x, k in zip(lens, nodes)]


def _tree(rng, n):
    """Parents of a random tree in breadth-first order (a parent's index is below its child's)."""
    width = int(rng.integers(3, 9))
    p = np.array([int(rng.integers(max(0, i - width), i)) for i in range(1, n)], dtype=np.int64)
    return np.concatenate([[-1], np.sort(p)]).astype(np.int32)


def _closure(parents):
    """Depth of every node and its row mask: the node itself and its ancestors."""
    depth, mask = [], []
    for i, p in enumerate(parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        mask.append((1 << i) | (0 if p < 0 else mask[p]))
    words = [[(m >> (32 * w)) & 0xFFFFFFFF for w in range(WORDS)] for m in mask]
    return depth, words


def _handles(s, case):
    """What a program that calls the library keeps: its context and, for logits, the rules (which buffers hold what)."""
    from speculative_decode_verify_attn_gb300 import vfy
    s["ctx"] = vfy.vfy_create(case.get("q_heads", case.get("kv_heads", 4)), case.get("kv_heads", 4), case.get("dim", 128),
                              window=WINDOW, ring_len=RING, max_seqs=s["B"], max_queries_per_seq=s["Q"])
    if case["op"] in ("first", "logits"):
        s["rules"] = vfy.LogitRules(counts=s["counts"], repetition=s["rep"], frequency=s["freq"], presence=s["pres"],
                                    drafts=s["drafts"], tree_mask=s["mask"], cu_bias=s.get("cu_bias"),
                                    bias_token=s.get("bias_token"), bias_value=s.get("bias_value"),
                                    grammar=s.get("grammar"), mask_index=s.get("mask_index"))


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": case}
    B = case["seqs"]
    op = case["op"]
    nodes, lens = _lengths(case)
    cu_q = _cu(nodes)
    T = int(cu_q[-1])
    s.update(B=B, T=T, Q=max(nodes), cu_q=_dev(cu_q))
    parents = [_tree(rng, n) for n in nodes]
    s["parents"] = _dev(np.concatenate(parents))
    plans = [_closure(p) for p in parents]
    s["depth"] = _dev(np.concatenate([d for d, _ in plans]))
    s["mask"] = _dev(np.concatenate([np.asarray(w, dtype=np.uint32) for _, w in plans]).view(np.int32))
    if op in ("full", "swa"):
        _attention_inputs(s, case, rng, gen, nodes, lens)
    elif op in ("first", "logits"):
        _logits_inputs(s, case, rng, gen, nodes, lens)
    elif op == "accept":
        _accept_inputs(s, case, rng, gen, nodes, parents, cu_q)
    else:
        _compact_inputs(s, case, rng, gen, nodes, lens)
    if own:
        _handles(s, case)
    return s


def _randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _attention_inputs(s, case, rng, gen, nodes, lens):
    B, T, hq, hkv, d = s["B"], s["T"], case["q_heads"], case["kv_heads"], case["dim"]
    s["seq_len"] = _dev(lens)
    s["q"] = _randn(gen, T, hq, d)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((T, hq), device="cuda", dtype=torch.float32)
    s["depth_out"], s["mask_out"] = torch.empty_like(s["depth"]), torch.empty_like(s["mask"])
    if case["op"] == "swa":
        s["k"], s["v"] = _randn(gen, B, hkv, RING, d), _randn(gen, B, hkv, RING, d)
        s["ring_offset"] = _dev(rng.integers(0, RING, B))
        return
    ids = []
    for n, L in zip(nodes, lens):
        total = -(-L // CHUNK)
        block = np.arange((L - n) // CHUNK, total)
        rest = np.arange(0, block[0])
        if case["chunks"] and len(rest) + len(block) > case["chunks"]:
            rest = np.sort(rng.choice(rest, max(0, case["chunks"] - len(block)), replace=False))
        ids.append(np.concatenate([rest, block]))
    counts = [len(i) for i in ids]
    slots = rng.permutation(sum(counts))
    s.update(ids=_dev(np.concatenate(ids)), slots=_dev(slots), cu_res=_dev(_cu(counts)), max_res=max(counts),
             num_slots=sum(counts))
    s["k"], s["v"] = _randn(gen, sum(counts), hkv, CHUNK, d), _randn(gen, sum(counts), hkv, CHUNK, d)


def _logits_inputs(s, case, rng, gen, nodes, lens):
    B, T, V = s["B"], s["T"], case["vocab"]
    dtype = torch.bfloat16 if case["bf16"] else torch.float32
    s["logits"] = (_randn(gen, T, V, dtype=torch.float32) * 3).to(dtype)
    s["drafts"] = _dev(rng.integers(0, V, max(1, T - B)))
    s["rep"] = _dev(rng.uniform(1.0, 1.3, B), np.float32)
    s["freq"] = _dev(rng.uniform(0.0, 0.5, B), np.float32)
    s["pres"] = _dev(rng.uniform(0.0, 0.8, B), np.float32)
    s["out"] = torch.empty((T, V), device="cuda", dtype=torch.float32)
    s["counts"] = torch.zeros((B, V), device="cuda", dtype=torch.int32)
    if case["op"] == "first":
        cu = _cu(lens)
        # token frequencies of text: a few tokens take most places
        u = torch.rand(int(cu[-1]), generator=gen, device="cuda")
        s["tokens"] = (V ** u - 1).to(torch.int32).clamp(max=V - 1)
        s["cu_tokens"], s["max_tokens"] = _dev(cu), int(cu[-1])
        return
    # what a conversation leaves: some of the vocabulary in the prompt, some of it generated
    u = torch.rand((B, V), generator=gen, device="cuda")
    made = torch.where(u < 0.01, (u * 900).to(torch.int32) + 1, torch.zeros_like(s["counts"]))
    prompt = torch.rand((B, V), generator=gen, device="cuda") < 0.05
    s["counts"] = torch.where(prompt, made | -2 ** 31, made)
    if case["biases"]:
        n = min(case["biases"], V)
        s["cu_bias"] = _dev(np.arange(B + 1) * n)
        s["bias_token"] = _dev(np.concatenate([rng.choice(V, n, replace=False) for _ in range(B)]))
        s["bias_value"] = _dev(rng.uniform(-20, 20, B * n), np.float32)
    if case["grammar"]:
        words = -(-V // 32)
        # every second request (the first of them always) follows a grammar; about half the vocabulary is let through
        seqs = np.repeat(np.arange(B), nodes)
        constrained = seqs % 2 == 0
        index = np.where(constrained, np.cumsum(constrained) - 1, -1)
        s["mask_index"] = _dev(index)
        s["grammar"] = torch.randint(-2 ** 31, 2 ** 31, (int(constrained.sum()), words), generator=gen, device="cuda",
                                     dtype=torch.int64).to(torch.int32)


def _accept_inputs(s, case, rng, gen, nodes, parents, cu_q):
    B, T, V = s["B"], s["T"], case["vocab"]
    s["logits"] = _randn(gen, T, V, dtype=torch.float32)
    targets = rng.integers(0, V, T)
    s["logits"][torch.arange(T, device="cuda"), _dev(targets, np.int64)] = 6.0
    drafts = []
    for b, (n, p) in enumerate(zip(nodes, parents)):
        for j in range(1, n):      # a drafted child is the target's token with probability one half
            drafts.append(targets[cu_q[b] + p[j]] if rng.random() < 0.5 else rng.integers(0, V))
    s["drafts"] = _dev(drafts if drafts else [0])
    e = lambda n: torch.empty(n, device="cuda", dtype=torch.int32)   # noqa: E731
    s.update(accepted=e(B), path=e(T), bonus=e(B), committed=e(T))


def _compact_inputs(s, case, rng, gen, nodes, lens):
    B, T, L, hkv, d = s["B"], s["T"], case["layers"], case["kv_heads"], case["dim"]
    path, accepted = np.full(T, -1, np.int64), []
    cu = _cu(nodes)
    for b, n in enumerate(nodes):
        # an accepted path that starts behind its own length, as in a tree with many children of
        # the root: no row is both moved and written over
        k = int(rng.integers(1, (n - 1) // 2 + 1))
        k = min(k, 12)
        path[cu[b]] = 0
        path[cu[b] + 1: cu[b] + k + 1] = np.sort(rng.choice(np.arange(k + 1, n), k, replace=False))
        accepted.append(k)
    s["path"], s["accepted"] = _dev(path), _dev(accepted)
    if case["op"] == "rings":
        s["seq_len"] = _dev(rng.integers(max(nodes), 262144, B))
        s["ring_offset"] = _dev(rng.integers(0, RING, B))
        s["k"], s["v"] = _randn(gen, L, B, hkv, RING, d), _randn(gen, L, B, hkv, RING, d)
        s["ks"], s["vs"] = list(s["k"].unbind(0)), list(s["v"].unbind(0))
        return
    chunks = [-(-x // CHUNK) for x in lens]
    cu_chunks = _cu(chunks)
    # the last chunks of every sequence are resident, as those of the block are
    slot_of = np.full(int(cu_chunks[-1]), -1)
    kept = np.concatenate([np.arange(max(cu_chunks[b], cu_chunks[b + 1] - 8), cu_chunks[b + 1]) for b in range(B)])
    slot_of[kept] = rng.permutation(len(kept))
    s.update(seq_len=_dev(lens), cu_chunks=_dev(cu_chunks), slot_of=_dev(slot_of), chunks=int(cu_chunks[-1]),
             num_slots=len(kept))
    for name, n in (("k", len(kept)), ("v", len(kept)), ("store_k", s["chunks"]), ("store_v", s["chunks"])):
        s[name] = _randn(gen, L, n, hkv, CHUNK, d)
        s[name + "s"] = list(s[name].unbind(0))


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------

def _row_seq(cu, T):
    """The sequence that every row belongs to, and the row's index within it."""
    row = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu.long(), row, right=True) - 1
    return seq, row - cu.long()[seq]


def _padded(x, cu, Q, fill):
    """Rows of all sequences as [B, Q, ...], `fill` where a sequence has fewer."""
    seq, i = _row_seq(cu, x.shape[0])
    out = x.new_full((cu.numel() - 1, Q) + x.shape[1:], fill)
    out[seq, i] = x
    return out


def _bits(mask, Q):
    """Row masks [..., WORDS] as truth values [..., Q]."""
    j = torch.arange(Q, device=mask.device)
    return ((mask.long()[..., j // 32] >> (j % 32)) & 1).bool()


def _plain_plan(s):
    B, Q, T = s["B"], s["Q"], s["T"]
    parents = _padded(s["parents"], s["cu_q"], Q, -1).long()
    reach = torch.eye(Q, device="cuda").expand(B, Q, Q).clone()
    reach = reach + (parents[..., None] == torch.arange(Q, device="cuda")).float()
    for _ in range(max(1, math.ceil(math.log2(max(2, Q))))):      # paths of 1, 2, 4, ... steps
        reach = (reach @ reach).clamp(max=1)
    seq, i = _row_seq(s["cu_q"], T)
    rows = torch.nn.functional.pad(reach[seq, i].long(), (0, 32 * WORDS - Q))
    words = (rows.view(T, WORDS, 32) << torch.arange(32, device="cuda")).sum(-1)
    depth = rows.sum(-1) - 1
    return depth.int(), torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()


def _plain_softmax(s, keys, values, allowed):
    """Attention of padded queries [B, Q, Hq, d] over [B, Hkv, N, d] where allowed [B, Q, N]."""
    B, Q, hq, d = s["B"], s["Q"], s["case"]["q_heads"], s["case"]["dim"]
    hkv = s["case"]["kv_heads"]
    g = hq // hkv
    q = _padded(s["q"].float(), s["cu_q"], Q, 0.0).view(B, Q, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, Q * g, d)
    x = q @ keys.transpose(-1, -2) / math.sqrt(d)
    x = x.view(B, hkv, Q, g, -1).masked_fill_(~allowed[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = (x - m).exp_()
    total = x.sum(-1, keepdim=True)
    o = x.view(B, hkv, Q * g, -1) @ values
    o = o.view(B, hkv, Q, g, d) / total.clamp(min=1e-38)
    lse = (m + total.log()).squeeze(-1)
    seq, i = _row_seq(s["cu_q"], s["T"])
    o = o.permute(0, 2, 1, 3, 4).reshape(B, Q, hq, d)[seq, i]
    return o.to(torch.bfloat16), lse.permute(0, 2, 1, 3).reshape(B, Q, hq)[seq, i]


def _plain_attention(s):
    case, B, Q = s["case"], s["B"], s["Q"]
    depth, mask = _plain_plan(s) if case["dynamic"] else (s["depth"], s["mask"])
    nodes = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    end = s["seq_len"].long()[:, None]
    start = end - nodes[:, None]                                     # position of node 0
    if case["op"] == "full":
        n = torch.arange(s["max_res"], device="cuda")
        cu = s["cu_res"].long()
        have = n < (cu[1:] - cu[:-1])[:, None]
        at = torch.where(have, cu[:-1, None] + n, 0)
        t = torch.arange(CHUNK, device="cuda")
        pos = (s["ids"].long()[at][..., None] * CHUNK + t).flatten(1)
        valid = have[..., None].expand(-1, -1, CHUNK).flatten(1)
        take = lambda x: x[s["slots"].long()[at]].transpose(1, 2).flatten(2, 3).float()   # noqa: E731
    else:
        pos = end - 1 - torch.arange(WINDOW - 1 + Q, device="cuda")
        valid = pos >= 0
        slot = (pos + s["ring_offset"].long()[:, None]) % RING
        take = lambda x: x.transpose(1, 2)[torch.arange(B, device="cuda")[:, None], slot].transpose(1, 2).float()   # noqa: E731
    inside = (pos - start).clamp(0, Q - 1)                           # block row of a position
    rows = _bits(_padded(mask, s["cu_q"], Q, 0), Q)
    in_block = torch.gather(rows, 2, inside[:, None, :].expand(-1, Q, -1)) & (pos >= start)[:, None, :]
    before = (pos < start)[:, None, :]
    if case["op"] == "swa":
        first = start[..., None] + _padded(depth, s["cu_q"], Q, 0).long()[..., None] - WINDOW + 1
        before = before & (pos[:, None, :] >= first)
    allowed = (before | in_block) & (valid & (pos < end))[:, None, :]
    o, lse = _plain_softmax(s, take(s["k"]), take(s["v"]), allowed)
    return (o, lse, depth, mask) if case["dynamic"] else (o, lse)


def _plain_counts(s):
    """Counts of the prompts: bit 31 marks a token that the prompt holds."""
    seq, _ = _row_seq(s["cu_tokens"], s["max_tokens"])
    counts = torch.zeros_like(s["counts"])
    counts[seq, s["tokens"].long()] = -2 ** 31
    return counts


def _plain_logits(s, counts):
    case, T, B, V, Q = s["case"], s["T"], s["B"], s["case"]["vocab"], s["Q"]
    x = s["logits"].float()
    seq, i = _row_seq(s["cu_q"], T)
    words = counts[seq]
    made = (words & 0x7FFFFFFF).float()
    seen = words != 0
    if Q > 1:
        # the drafted tokens on the node's path count as generated
        node = torch.arange(Q, device="cuda")
        on_path = _bits(s["mask"], Q) & (node > 0)
        at = (s["cu_q"].long()[seq] - seq)[:, None] + node - 1
        token = s["drafts"].long()[torch.where(on_path, at, 0)]
        made = made.scatter_add(1, token, on_path.float())
        seen = seen | (made > 0)
    rep = s["rep"][seq][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["freq"][seq][:, None] * made - s["pres"][seq][:, None] * (made > 0).float()
    if "bias_token" in s:
        bias = torch.zeros((B, V), device="cuda")
        entry_seq, _ = _row_seq(s["cu_bias"], s["bias_token"].numel())
        bias[entry_seq, s["bias_token"].long()] = s["bias_value"]
        x = x + bias[seq]
    if "grammar" in s:
        v = torch.arange(V, device="cuda")
        lets = (s["grammar"][s["mask_index"].long().clamp(min=0)][:, v // 32] >> (v % 32)) & 1
        x = torch.where((lets == 0) & (s["mask_index"] >= 0)[:, None], -math.inf, x)
    return x


def _plain_accept(s):
    B, T, Q, V = s["B"], s["T"], s["Q"], s["case"]["vocab"]
    x = s["logits"]
    v = torch.arange(V, device="cuda")
    target = torch.where(x == x.amax(1, keepdim=True), v, V).amin(1)      # ties to the lowest index
    cu = s["cu_q"].long()
    seq, i = _row_seq(s["cu_q"], T)
    token = torch.where(i > 0, s["drafts"].long()[(cu[seq] - seq + i - 1).clamp(0, s["drafts"].numel() - 1)], -1)
    parent = s["parents"].long()
    good = (i > 0) & (token == target[cu[seq] + parent.clamp(min=0)])
    # of two such children of one node, the lower index is taken
    p_good, p_parent = _padded(good, s["cu_q"], Q, False), _padded(parent, s["cu_q"], Q, -1)
    node = torch.arange(Q, device="cuda")
    earlier = (p_parent[:, :, None] == p_parent[:, None, :]) & (node[:, None] > node) & p_good[:, None, :]
    good = good & ~earlier.any(-1)[seq, i]
    lost = ~_padded(good, s["cu_q"], Q, False) & (node > 0)               # cuts its whole subtree off
    on_path = ~((_bits(s["mask"], Q) & lost[seq]).any(-1))                # rows of the accepted path
    accepted = torch.zeros(B, device="cuda", dtype=torch.int64).index_add_(0, seq, on_path.long()) - 1
    rank = torch.cumsum(on_path.long(), 0)
    rank = rank - 1 - (rank[cu[:-1]] - 1)[seq]
    path = torch.full((T,), -1, device="cuda", dtype=torch.int64)
    committed = path.clone()
    at = cu[seq] + rank
    keep = torch.where(on_path, at, T)
    path = torch.cat([path, path[:1]]).scatter_(0, keep, i)[:T]
    moved = torch.where(on_path & (i > 0), at - 1, T)
    committed = torch.cat([committed, committed[:1]]).scatter_(0, moved, token)[:T]
    last = path[cu[:-1] + accepted]
    bonus = target[cu[:-1] + last]
    committed[cu[:-1] + accepted] = bonus
    return accepted.int(), path.int(), bonus.int(), committed.int()


def _plain_compact(s):
    case, T = s["case"], s["T"]
    cu = s["cu_q"].long()
    seq, j = _row_seq(s["cu_q"], T)
    moves = (j > 0) & (j <= s["accepted"].long()[seq])
    start = s["seq_len"].long()[seq] - (cu[1:] - cu[:-1])[seq]
    src, dst = start + torch.where(moves, s["path"].long(), j), start + j      # the others stay in place
    if case["op"] == "rings":
        phi = s["ring_offset"].long()[seq]
        for name in ("k", "v"):
            x = s[name]
            x[:, seq, :, (dst + phi) % RING] = x[:, seq, :, (src + phi) % RING]
        return s["k"], s["v"]
    c_src, c_dst = s["cu_chunks"].long()[seq] + src // CHUNK, s["cu_chunks"].long()[seq] + dst // CHUNK
    slot_src, slot_dst = s["slot_of"].long()[c_src], s["slot_of"].long()[c_dst]     # all resident
    for name in ("k", "v"):
        rows = s[name][:, slot_src, :, src % CHUNK]
        s["store_" + name][:, c_dst, :, dst % CHUNK] = torch.where(
            moves[:, None, None, None], rows, s["store_" + name][:, c_dst, :, dst % CHUNK])
        s[name][:, slot_dst, :, dst % CHUNK] = rows
    return s["k"], s["v"], s["store_k"], s["store_v"]


def _plain(s):
    op = s["case"]["op"]
    if op in ("full", "swa"):
        return _plain_attention(s)
    if op == "first":
        counts = _plain_counts(s)
        return counts, _plain_logits(s, counts)
    if op == "logits":
        return (_plain_logits(s, s["counts"]),)
    return _plain_accept(s) if op == "accept" else _plain_compact(s)


# ---------------------------------------------------------------------------------------------
# The library's operators
# ---------------------------------------------------------------------------------------------

def _own(s):
    from speculative_decode_verify_attn_gb300 import vfy
    case, ctx, B, T = s["case"], s["ctx"], s["B"], s["T"]
    op = case["op"]
    if op in ("full", "swa"):
        depth, mask = s["depth"], s["mask"]
        if case["dynamic"]:
            depth, mask = s["depth_out"], s["mask_out"]
            vfy.vfy_tree_plan(ctx, s["parents"], s["cu_q"], depth, mask, B)
        if op == "full":
            vfy.vfy_attend_full_tree(ctx, s["q"], s["cu_q"], mask, s["k"], s["v"], s["num_slots"], s["ids"], s["slots"],
                                     s["cu_res"], s["max_res"], s["seq_len"], s["out"], s["lse"], B)
        else:
            vfy.vfy_attend_swa_tree(ctx, s["q"], s["cu_q"], mask, depth, s["k"], s["v"], s["ring_offset"], s["seq_len"],
                                    s["out"], s["lse"], B)
        return (s["out"], s["lse"], depth, mask) if case["dynamic"] else (s["out"], s["lse"])
    if op in ("first", "logits"):
        if op == "first":
            vfy.vfy_count_tokens(ctx, s["tokens"], s["cu_tokens"], s["max_tokens"], s["counts"], case["vocab"], B,
                                 as_prompt=True, reset=True)
        vfy.vfy_process_logits(ctx, s["logits"], case["vocab"], s["cu_q"], T, s["rules"], s["out"], B)
        return (s["counts"], s["out"]) if op == "first" else (s["out"],)
    if op == "accept":
        vfy.vfy_accept_tree(ctx, s["logits"], case["vocab"], s["drafts"], s["parents"], s["cu_q"], T, s["accepted"],
                            s["path"], s["bonus"], s["committed"], B)
        return s["accepted"], s["path"], s["bonus"], s["committed"]
    if op == "rings":
        vfy.vfy_compact_swa(ctx, s["path"], s["accepted"], s["cu_q"], s["seq_len"], s["ring_offset"], s["ks"], s["vs"], B)
        return s["k"], s["v"]
    vfy.vfy_compact_full(ctx, s["path"], s["accepted"], s["cu_q"], s["seq_len"], s["cu_chunks"], s["slot_of"],
                         s["store_ks"], s["store_vs"], s["chunks"], s["ks"], s["vs"], s["num_slots"], B)
    return s["k"], s["v"], s["store_k"], s["store_v"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    nodes, lens = _lengths(case)
    B, rows = len(nodes), sum(nodes)
    if op in ("full", "swa"):
        hq, hkv, d = case["q_heads"], case["kv_heads"], case["dim"]
        if op == "swa":
            keys = [min(x, WINDOW - 1 + n) for n, x in zip(nodes, lens)]
        else:
            keys = [min(x, case["chunks"] * CHUNK or x) for x in lens]
        pairs = sum(n * (min(k, WINDOW) if op == "swa" else k) for n, k in zip(nodes, keys))
        plan = rows * (4 + 4 + 4 * WORDS) if case["dynamic"] else 0
        return {"bytes": sum(keys) * hkv * d * 4 + rows * hq * (d * 4 + 4) + rows * 4 * WORDS + plan,
                "flops": 4 * pairs * hq * d}
    if op in ("first", "logits"):
        V = case["vocab"]
        size = rows * V * ((2 if case["bf16"] else 4) + 4) + B * V * 4
        if op == "first":
            return {"bytes": size + sum(lens) * 4, "flops": rows * V * 5}
        grammar = sum(nodes[::2]) * V / 8 if case["grammar"] else 0
        return {"bytes": size + grammar + B * case["biases"] * 8, "flops": rows * V * 5}
    if op == "accept":
        return {"bytes": rows * (case["vocab"] * 4 + 16), "flops": rows * case["vocab"]}
    moved = sum((1 + min(12, (n - 1) // 2)) / 2 for n in nodes)        # rows, in the mean over seeds
    row = case["layers"] * 2 * case["kv_heads"] * case["dim"] * 2
    return {"bytes": moved * row * (3 if op == "pools" else 2) + rows * 4, "flops": moved}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_attention(s):
    case = s["case"]
    g, d = case["q_heads"] // case["kv_heads"], case["dim"]
    cu, lens = s["cu_q"].tolist(), s["seq_len"].tolist()
    parents, q = s["parents"].tolist(), s["q"].double()
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, device="cuda", dtype=torch.float64)
    for b in range(s["B"]):
        n = cu[b + 1] - cu[b]
        p0 = lens[b] - n
        if case["op"] == "full":
            r0, r1 = s["cu_res"][b].item(), s["cu_res"][b + 1].item()
            pos = (s["ids"][r0:r1].long()[:, None] * CHUNK + torch.arange(CHUNK, device="cuda")).reshape(-1)
            rows = s["slots"][r0:r1].long()
            keys = lambda x, h: x[rows, h].reshape(-1, d).double()          # noqa: E731
        else:
            pos = torch.arange(max(0, p0 - WINDOW + 1), lens[b], device="cuda")
            rows = (pos + s["ring_offset"][b].item()) % RING
            keys = lambda x, h: x[b, h, rows].double()                      # noqa: E731
        see = torch.zeros((n, pos.numel()), dtype=torch.bool, device="cuda")
        for i in range(n):
            chain, a = [], i
            while a >= 0:
                chain.append(a)
                a = parents[cu[b] + a]
            first = p0 + len(chain) - 1 - WINDOW + 1 if case["op"] == "swa" else 0
            see[i] = (pos < p0) & (pos >= first)
            see[i] |= torch.isin(pos, torch.tensor(chain, device="cuda") + p0)
        for h in range(case["kv_heads"]):
            K, V = keys(s["k"], h), keys(s["v"], h)
            for hq in range(h * g, h * g + g):
                x = q[cu[b]:cu[b + 1], hq] @ K.T / math.sqrt(d)
                x = torch.where(see, x, -math.inf)
                lse[cu[b]:cu[b + 1], hq] = torch.logsumexp(x, 1)
                out[cu[b]:cu[b + 1], hq] = torch.softmax(x, 1).nan_to_num() @ V
    return (out, lse, None, None) if case["dynamic"] else (out, lse)


def _exact_logits(s):
    case, V = s["case"], s["case"]["vocab"]
    cu = s["cu_q"].tolist()
    parents, drafts = s["parents"].tolist(), s["drafts"].tolist()
    out = s["logits"].double()
    for b in range(s["B"]):
        if case["op"] == "first":
            t0, t1 = s["cu_tokens"][b].item(), s["cu_tokens"][b + 1].item()
            seen0 = torch.zeros(V, dtype=torch.bool, device="cuda")
            seen0[s["tokens"][t0:t1].long().unique()] = True
            made0 = torch.zeros(V, dtype=torch.float64, device="cuda")
        else:
            made0 = (s["counts"][b].long() % 2 ** 31).double()
            seen0 = s["counts"][b] != 0
        for i in range(cu[b + 1] - cu[b]):
            made, a = made0.clone(), i
            while a > 0:
                made[drafts[cu[b] - b + a - 1]] += 1
                a = parents[cu[b] + a]
            x = out[cu[b] + i]
            seen = seen0 | (made > 0)
            r = s["rep"][b].double()
            x[seen & (x > 0)] /= r
            x[seen & (x < 0)] *= r
            x -= s["freq"][b].double() * made + s["pres"][b].double() * (made > 0)
            if "bias_token" in s:
                e = slice(s["cu_bias"][b].item(), s["cu_bias"][b + 1].item())
                x[s["bias_token"][e].long()] += s["bias_value"][e].double()
            if "grammar" in s and s["mask_index"][cu[b] + i] >= 0:
                words = s["grammar"][s["mask_index"][cu[b] + i].item()].cpu().numpy().view(np.uint8)
                lets = np.unpackbits(words, bitorder="little")[:V]
                x[torch.from_numpy(lets == 0).cuda()] = -math.inf
    return (None, out) if case["op"] == "first" else (out,)


def _exact_compact(s):
    case = s["case"]
    cu, lens, n = s["cu_q"].tolist(), s["seq_len"].tolist(), s["accepted"].tolist()
    names = ["k", "v"] if case["op"] == "rings" else ["k", "v", "store_k", "store_v"]
    out = {x: s[x].clone() for x in names}
    for b in range(s["B"]):
        p0 = lens[b] - (cu[b + 1] - cu[b])
        for j in range(1, n[b] + 1):
            src, dst = p0 + s["path"][cu[b] + j].item(), p0 + j
            for x in ("k", "v"):
                if case["op"] == "rings":
                    phi = s["ring_offset"][b].item()
                    out[x][:, b, :, (dst + phi) % RING] = s[x][:, b, :, (src + phi) % RING]
                else:
                    c0 = s["cu_chunks"][b].item()
                    row = s[x][:, s["slot_of"][c0 + src // CHUNK].item(), :, src % CHUNK]
                    out[x][:, s["slot_of"][c0 + dst // CHUNK].item(), :, dst % CHUNK] = row
                    out["store_" + x][:, c0 + dst // CHUNK, :, dst % CHUNK] = row
    return tuple(out[x].double() for x in names)


def _exact_accept(s):
    cu, parents, drafts = s["cu_q"].tolist(), s["parents"].tolist(), s["drafts"].tolist()
    target = s["logits"].cpu().numpy().argmax(1)                            # the first of equal values
    accepted, bonus = [], []
    path, committed = np.full(s["T"], -1), np.full(s["T"], -1)
    for b in range(s["B"]):
        r0, n = cu[b], cu[b + 1] - cu[b]
        node, k = 0, 0
        path[r0] = 0
        while True:
            token = target[r0 + node]
            committed[r0 + k] = token
            child = [c for c in range(1, n) if parents[r0 + c] == node and drafts[r0 - b + c - 1] == token]
            if not child:
                break
            node, k = child[0], k + 1
            path[r0 + k] = node
        accepted.append(k)
        bonus.append(token)
    return tuple(np.asarray(x, dtype=np.int32) for x in (accepted, path, bonus, committed))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("full", "swa"):
        return _exact_attention(s)
    if case["op"] in ("first", "logits"):
        return _exact_logits(s)
    if case["op"] in ("rings", "pools"):
        return _exact_compact(s)
    return _exact_accept(s)
