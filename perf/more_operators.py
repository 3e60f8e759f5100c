"""Cases that time what a verify block meets around its attention: rotation and append, the 4-bit pool, sampling.

  rotation and append   queries and keys of the block normalised per head and rotated to their positions, in one
                        pass over the projection's output; keys and values go straight to where the layer's
                        attention reads them: rows ("rope_rows"), chunk pool and store ("rope_full") or position
                        ring ("rope_swa").
  4-bit pool            chunks of 4-bit floats (e2m1) with an e4m3 scale for each 16 values. The block's K/V rows
                        are written in that form, and chunks are read back as bf16 ("packed_append"); a full
                        layer attends the 4-bit chunks ("packed_attend").
  sampled verification  drafted tokens accepted with probability min(1, p / q) from given random numbers, the next
                        token drawn from what the drafter left of p ("sampled").

`run` computes each in plain torch where `own` is false and calls the library where it is true.
"""
import math
import random

import numpy as np
import torch

own = False

CHUNK = 64
WINDOW, RING = 512, 2048
# the values of the sixteen 4-bit codes: sign, two exponent bits, one mantissa bit
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def _block(op, name, seqs, nodes, context, heads=(16, 4, 128), ragged=False, **more):
    return {"name": name, "op": op, "seqs": seqs, "nodes": nodes, "context": context, "ragged": ragged,
            "q_heads": heads[0], "kv_heads": heads[1], "dim": heads[2], **more}


def listed():
    return [
        # One full layer's block of 17 tokens at 8K: where latency counts.
        _block("rope_full", "rope_full17", 1, 17, 8192, rot=128, pairs="halves", norm=True, tree=False),
        # One window layer of a batch of trees far into their contexts; half of each head rotated, adjacent pairs.
        _block("rope_swa", "rope_swa_trees8", 8, 33, 262144, ragged=True, rot=64, pairs="adjacent", norm=True, tree=True),
        # A prefill-sized block of eight requests: the largest stream of rows.
        _block("rope_full", "rope_full_8x1024", 8, 1024, 4096, rot=128, pairs="halves", norm=True, tree=False),
        # The block's rows of one layer into the 4-bit pool and store, the chunks that hold them read back.
        _block("packed_append", "packed_append17", 1, 17, 8192, scale=1.0),
        # The same for a prefill-sized block, with scales of its own for K and V.
        _block("packed_append", "packed_append_8x1024", 8, 1024, 4096, scale=0.037),
        # A block over an 8K resident pool of 4-bit chunks: one full layer of a step.
        _block("packed_attend", "packed_attend17_8k", 1, 17, 262144, chunks=128, scale=1.0),
        # One token over 256K tokens, all resident: plain decoding from the 4-bit pool.
        _block("packed_attend", "packed_attend1_256k", 1, 1, 262144, chunks=0, scale=1.0),
        # The verify block over the same context: the largest stream.
        _block("packed_attend", "packed_attend17_256k", 1, 17, 262144, chunks=0, scale=1.0),
        # A serving batch of requests of different lengths and depths.
        _block("packed_attend", "packed_attend_ragged8", 8, 17, 48000, ragged=True, chunks=0, scale=0.25),
        # One block of 17 rows against the drafter's probabilities.
        {"name": "sampled17", "op": "sampled", "seqs": 1, "nodes": 17, "ragged": False, "vocab": 131072, "bf16": False,
         "probs": True},
        # A batch of blocks: bf16 logits, odd vocabulary, ragged depths, some requests greedy.
        {"name": "sampled_batch16", "op": "sampled", "seqs": 16, "nodes": 17, "ragged": True, "vocab": 100003,
         "bf16": True, "probs": True},
        # The first token of eight new requests: sampling from one row each.
        {"name": "sampled_first8", "op": "sampled", "seqs": 8, "nodes": 1, "ragged": False, "vocab": 131072,
         "bf16": True, "probs": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng: random.Random):
    op = rng.choice(["rope_full", "rope_swa", "rope_rows", "packed_append", "packed_attend", "packed_attend", "sampled",
                     "sampled"])
    seqs = _log(rng, 1, 16)
    if op == "sampled":
        return {"op": op, "seqs": seqs, "nodes": _log(rng, 1, 33 if seqs <= 8 else 17), "ragged": rng.random() < 0.5,
                "vocab": rng.choice([131072, 32000, 100003, _log(rng, 1000, 131072)]), "bf16": rng.random() < 0.5,
                "probs": rng.random() < 0.7}
    heads = rng.choice([(16, 4, 128), (4, 1, 64), (8, 8, 128), (32, 4, 128), (16, 2, 64)])
    ragged = seqs > 1 and rng.random() < 0.6
    if op == "packed_attend":
        nodes = _log(rng, 1, 64)
        # rows x keys and K/V elements stay within the largest listed case
        context = _log(rng, nodes + 1, 262144)
        context = min(context, 17 * 16 * 262144 // (nodes * heads[0] * seqs), 4 * 128 * 262144 // (heads[1] * heads[2] * seqs))
        chunks = _log(rng, 1, 512) if rng.random() < 0.4 else 0
        case = _block(op, "", seqs, nodes, max(context, nodes), heads, ragged, chunks=chunks,
                      scale=rng.choice([1.0, 0.25, round(rng.uniform(0.01, 2.0), 3)]))
    else:
        wide = (heads[0] + 2 * heads[1]) * heads[2]
        nodes = _log(rng, 1, min(1024 if op != "rope_swa" else 256, 4096 // max(1, heads[0] // heads[1]),
                                 8 * 1024 * 24 * 128 // (seqs * wide)))
        context = _log(rng, nodes, 262144 if op in ("rope_swa", "rope_rows") else max(nodes, 32768 // seqs))
        if op == "packed_append":
            case = _block(op, "", seqs, nodes, context, heads, ragged, scale=rng.choice([1.0, round(rng.uniform(0.01, 2.0), 3)]))
        else:
            case = _block(op, "", seqs, nodes, context, heads, ragged, rot=rng.choice([heads[2], heads[2] // 2, 32]),
                          pairs=rng.choice(["halves", "adjacent"]), norm=rng.random() < 0.7,
                          tree=nodes <= 256 and rng.random() < 0.3)
    return {k: v for k, v in case.items() if k != "name"}


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
    """Rows and context lengths of the sequences: the case's own, whatever the seed."""
    rng = np.random.default_rng([case["seqs"], case["nodes"], case.get("context", 0), case.get("vocab", 0)])
    B, n, c = case["seqs"], case["nodes"], case.get("context", 0)
    nodes = _spread(rng, B, max(1, n // 8), n) if case["ragged"] else [n] * B
    lens = _spread(rng, B, max(1, c // (12 if case["ragged"] else 2)), c) if c and B > 1 else [c] * B
    return nodes, [max(x, k) for x, k in zip(lens, nodes)]


def _resident(case):
    """How many chunks of each sequence the pool holds."""
    return [min(-(-x // CHUNK), max(case["chunks"], (x - 1) // CHUNK - (x - n) // CHUNK + 1) if case["chunks"] else x)
            for n, x in zip(*_lengths(case))]


def _randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _handles(s, case):
    """What a program that calls the library keeps: its context and the layer's constants."""
    from speculative_decode_verify_attn_gb300 import vfy
    s["ctx"] = vfy.vfy_create(case.get("q_heads", 1), case.get("kv_heads", 1), case.get("dim", 64), window=WINDOW,
                              ring_len=RING, max_seqs=s["B"], max_queries_per_seq=s["Q"])
    if case["op"].startswith("rope"):
        s["rope"] = vfy.Rope(inv_freq=s["inv_freq"], rot_dim=case["rot"], interleaved=case["pairs"] == "adjacent",
                             q_norm=s["q_norm"], k_norm=s["k_norm"], eps=s["eps"])


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    nodes, lens = _lengths(case)
    cu = _cu(nodes)
    s = {"case": case, "B": case["seqs"], "T": int(cu[-1]), "Q": max(nodes), "cu_q": _dev(cu)}
    if case["op"] == "sampled":
        _sampled_inputs(s, case, rng, gen, nodes)
    elif case["op"] == "packed_attend":
        _attend_inputs(s, case, rng, gen, nodes, lens)
    else:
        _append_inputs(s, case, rng, gen, nodes, lens)
    if own:
        _handles(s, case)
    return s


def _tree_depths(rng, n):
    """Depths of a random tree's nodes in breadth-first order."""
    width = int(rng.integers(3, 9))
    depth = [0]
    for i in range(1, n):
        depth.append(depth[int(rng.integers(max(0, i - width), i))] + 1)
    return depth


def _append_inputs(s, case, rng, gen, nodes, lens):
    T, hq, hkv, d = s["T"], case["q_heads"], case["kv_heads"], case["dim"]
    s["seq_len"] = _dev(lens)
    # what one projection gives: queries, keys, values and a gate for each query head, side by side
    s["rows"] = _randn(gen, T, (hq + 2 * hkv) * d + max(8, hq))
    s["q"] = s["rows"][:, :hq * d].unflatten(1, (hq, d))
    s["k"] = s["rows"][:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    s["v"] = s["rows"][:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d))
    if case["op"].startswith("rope"):
        s["inv_freq"] = 500000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float32) / case["rot"])
        s["eps"] = 1e-6
        norm = lambda: (1 + 0.2 * _randn(gen, d)).to(torch.bfloat16) if case["norm"] else None   # noqa: E731
        s["q_norm"], s["k_norm"] = norm(), norm()
        s["depth"] = _dev(np.concatenate([_tree_depths(rng, n) for n in nodes])) if case["tree"] else None
        s["q_out"] = torch.empty((T, hq, d), device="cuda", dtype=torch.bfloat16)
    if case["op"] == "rope_rows":
        s["k_out"] = torch.empty((T, hkv, d), device="cuda", dtype=torch.bfloat16)
        return
    if case["op"] == "rope_swa":
        s["k_dst"], s["v_dst"] = _randn(gen, s["B"], hkv, RING, d), _randn(gen, s["B"], hkv, RING, d)
        s["ring_offset"] = _dev(rng.integers(0, RING, s["B"]))
        return
    chunks = [-(-x // CHUNK) for x in lens]
    cu_chunks = _cu(chunks)
    # the last chunks of every sequence are resident, those that the block reaches among them
    kept = np.concatenate([np.arange(max(cu_chunks[b], cu_chunks[b + 1] - 24), cu_chunks[b + 1]) for b in range(s["B"])])
    slot_of = np.full(int(cu_chunks[-1]), -1)
    slot_of[kept] = rng.permutation(len(kept))
    s.update(cu_chunks=_dev(cu_chunks), slot_of=_dev(slot_of), chunks=int(cu_chunks[-1]), num_slots=len(kept))
    if case["op"] == "rope_full":
        s["k_dst"], s["v_dst"] = _randn(gen, len(kept), hkv, CHUNK, d), _randn(gen, len(kept), hkv, CHUNK, d)
        s["store_k"], s["store_v"] = _randn(gen, s["chunks"], hkv, CHUNK, d), _randn(gen, s["chunks"], hkv, CHUNK, d)
        return
    s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
    for name, n in (("k_dst", len(kept)), ("v_dst", len(kept)), ("store_k", s["chunks"]), ("store_v", s["chunks"])):
        s[name] = _packed_chunks(gen, n, hkv, d)
    # the chunks that hold the block, by their places in the store
    touched = np.concatenate([np.arange(cu_chunks[b] + (x - n) // CHUNK, cu_chunks[b + 1])
                              for b, (n, x) in enumerate(zip(nodes, lens))])
    s["touched"], s["touched_slots"] = _dev(touched), _dev(slot_of[touched])
    for name in ("k_read", "v_read", "k_stored", "v_stored"):
        s[name] = torch.empty((len(touched), hkv, CHUNK, d), device="cuda", dtype=torch.bfloat16)


def _packed_chunks(gen, n, hkv, d):
    """n chunks of hkv records of 36 d bytes: codes [d / 32][64 tokens][16 bytes] (even channels in the low four
    bits), then scales [64 tokens][d / 16]. Codes as Gaussian values give them, scales between 1/8 and 1."""
    x = torch.linspace(-1.0, 1.0, 64, device="cuda").erfinv().clamp(-1.8, 1.8) * 1.41421356 * 6 / 2.55
    one = (x[:, None] - torch.tensor(E2M1, device="cuda")).abs().argmin(1)
    two = (one[:, None] + 16 * one[None, :]).flatten().to(torch.uint8)
    pool = torch.empty((n, hkv, 36 * d), device="cuda", dtype=torch.uint8)
    at = torch.randint(0, 4096, (n, hkv, 32 * d), generator=gen, device="cuda", dtype=torch.int16)
    pool[..., :32 * d] = two[at.int()]
    pool[..., 32 * d:] = torch.randint(0x20, 0x39, (n, hkv, 4 * d), generator=gen, device="cuda", dtype=torch.uint8)
    return pool


def _attend_inputs(s, case, rng, gen, nodes, lens):
    T, hq, hkv, d = s["T"], case["q_heads"], case["kv_heads"], case["dim"]
    s["seq_len"] = _dev(lens)
    s["q"] = _randn(gen, T, hq, d)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((T, hq), device="cuda", dtype=torch.float32)
    ids = []
    for n, x, kept in zip(nodes, lens, _resident(case)):
        total = -(-x // CHUNK)
        block = np.arange((x - n) // CHUNK, total)
        rest = np.sort(rng.choice(block[0], kept - len(block), replace=False)) if kept > len(block) else []
        ids.append(np.concatenate([rest, block]))
    counts = [len(i) for i in ids]
    s.update(ids=_dev(np.concatenate(ids)), slots=_dev(rng.permutation(sum(counts))), cu_res=_dev(_cu(counts)),
             max_res=max(counts), num_slots=sum(counts))
    s["k"], s["v"] = _packed_chunks(gen, sum(counts), hkv, d), _packed_chunks(gen, sum(counts), hkv, d)


def _sampled_inputs(s, case, rng, gen, nodes):
    B, T, V = s["B"], s["T"], case["vocab"]
    dtype = torch.bfloat16 if case["bf16"] else torch.float32
    s["logits"] = (_randn(gen, T, V, dtype=torch.float32) * 3).to(dtype)
    warm = rng.uniform(0.6, 1.2, B)
    warm[1::4] = 0.0                                                   # some requests are greedy
    s["temperature"] = _dev(warm, np.float32)
    seq = np.repeat(np.arange(B), nodes)
    drafted = np.concatenate([np.arange(n) < n - 1 for n in nodes])    # rows that verify a drafted token
    rows, heat = _dev(np.flatnonzero(drafted), np.int64), _dev(np.maximum(warm, 0.3)[seq[drafted]], np.float32)
    s["noise"] = torch.empty((B, V), device="cuda").exponential_(generator=gen)
    s["uniform"] = torch.rand(max(1, T - B), generator=gen, device="cuda")
    # a drafter whose logits are near the target's, and tokens drawn from it
    near = s["logits"][rows].float()
    near = (near + 0.7 * torch.randn(near.shape, generator=gen, device="cuda")) / heat[:, None]
    gumbel = torch.empty(near.shape, device="cuda").exponential_(generator=gen).log()
    s["drafts"] = (near - gumbel).argmax(1).int() if len(rows) else torch.zeros(1, device="cuda", dtype=torch.int32)
    s["probs"] = torch.softmax(near, 1) if case["probs"] and len(rows) else None
    e = lambda n: torch.empty(n, device="cuda", dtype=torch.int32)     # noqa: E731
    s.update(accepted=e(B), bonus=e(B), committed=e(T))


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


def _places(s):
    """Sequence and position of every row of the block."""
    seq, i = _row_seq(s["cu_q"], s["T"])
    cu = s["cu_q"].long()
    return seq, i, s["seq_len"].long()[seq] - (cu[1:] - cu[:-1])[seq] + i


def _plain_rotated(s, x, weight, at):
    """Rows [T, H, d] normalised per head and rotated to the positions `at`, in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()
    angle = at.double()[:, None] * s["inv_freq"].double()              # far positions: in 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    rot = s["case"]["rot"]
    turned, rest = x[..., :rot], x[..., rot:]
    if s["case"]["pairs"] == "adjacent":
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = turned[..., :rot // 2], turned[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, rest], -1).to(torch.bfloat16)


def _plain_rope(s):
    seq, i, pos = _places(s)
    at = pos if s["depth"] is None else pos - i + s["depth"].long()
    s["q_out"] = _plain_rotated(s, s["q"], s["q_norm"], at)
    k = _plain_rotated(s, s["k"], s["k_norm"], at)
    if s["case"]["op"] == "rope_rows":
        return s["q_out"], k
    if s["case"]["op"] == "rope_swa":
        place = (pos + s["ring_offset"].long()[seq]) % RING
        s["k_dst"][seq, :, place] = k
        s["v_dst"][seq, :, place] = s["v"]
        return s["q_out"], s["k_dst"], s["v_dst"]
    chunk = s["cu_chunks"].long()[seq] + pos // CHUNK
    slot = s["slot_of"].long()[chunk]                                  # all resident
    s["store_k"][chunk, :, pos % CHUNK] = k
    s["store_v"][chunk, :, pos % CHUNK] = s["v"]
    s["k_dst"][slot, :, pos % CHUNK] = k
    s["v_dst"][slot, :, pos % CHUNK] = s["v"]
    return s["q_out"], s["k_dst"], s["v_dst"], s["store_k"], s["store_v"]


def _unpacked(records, d, scale):
    """Values [n, hkv, 64, d] of 4-bit chunks, in 32 bits."""
    n, hkv = records.shape[:2]
    codes = records[..., :32 * d].view(n, hkv, d // 32, CHUNK, 16).transpose(2, 3).reshape(n, hkv, CHUNK, d // 2).int()
    values = torch.tensor(E2M1, device="cuda")[torch.stack([codes & 15, codes >> 4], -1)].view(n, hkv, CHUNK, d // 16, 16)
    scales = records[..., 32 * d:].contiguous().view(torch.float8_e4m3fn).view(n, hkv, CHUNK, d // 16, 1).float()
    return (values * scales * scale).view(n, hkv, CHUNK, d)


def _plain_quantised(x, scale):
    """Rows [T, H, d] rounded to 4 bits with a scale for each 16 values, as the values that they stand for."""
    T, H, d = x.shape
    x = (x.float() / scale).view(T, H, d // 16, 16)
    step = (x.abs().amax(-1, keepdim=True) / 6).to(torch.float8_e4m3fn).float()
    y = torch.where(step > 0, x / step, 0.0)
    size = y.abs()
    # to the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6; a value in the middle goes to the even mantissa
    near = torch.where(size <= 2, (size * 2).round() / 2, torch.where(size <= 4, size.round(), (size / 2).round() * 2))
    return (torch.copysign(near.clamp(max=6), y) * step * scale).view(T, H, d)


def _plain_packed_append(s):
    d, scale = s["case"]["dim"], s["case"]["scale"]
    seq, _, pos = _places(s)
    chunk = s["cu_chunks"].long()[seq] + pos // CHUNK
    row = torch.searchsorted(s["touched"].long(), chunk)
    out = []
    for name, rows, source in (("k_dst", s["touched_slots"], s["k"]), ("v_dst", s["touched_slots"], s["v"]),
                               ("store_k", s["touched"], s["k"]), ("store_v", s["touched"], s["v"])):
        read = _unpacked(s[name][rows.long()], d, scale)
        read[row, :, pos % CHUNK] = _plain_quantised(source, scale)
        out.append(read.to(torch.bfloat16))
    return tuple(out)


def _plain_attend(s):
    case, B, Q = s["case"], s["B"], s["Q"]
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["dim"]
    g = hq // hkv
    cu, res = s["cu_q"].long(), s["cu_res"].long()
    n = torch.arange(s["max_res"], device="cuda")
    have = n < (res[1:] - res[:-1])[:, None]
    at = torch.where(have, res[:-1, None] + n, 0)
    pos = (s["ids"].long()[at][..., None] * CHUNK + torch.arange(CHUNK, device="cuda")).flatten(1)
    end = s["seq_len"].long()[:, None]
    first = end - (cu[1:] - cu[:-1])[:, None]
    own_pos = first + torch.arange(Q, device="cuda")
    allowed = (pos[:, None, :] <= own_pos[..., None]) & (have[..., None].expand(-1, -1, CHUNK).flatten(1) & (pos < end))[:, None]
    take = lambda x: _unpacked(x[s["slots"].long()[at].flatten()], d, case["scale"]) \
        .view(B, -1, hkv, CHUNK, d).transpose(1, 2).flatten(2, 3)                       # noqa: E731
    q = _padded(s["q"].float(), s["cu_q"], Q, 0.0).view(B, Q, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, Q * g, d)
    x = q @ take(s["k"]).transpose(-1, -2) / math.sqrt(d)
    x = x.view(B, hkv, Q, g, -1).masked_fill_(~allowed[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = (x - m).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(B, hkv, Q * g, -1) @ take(s["v"])).view(B, hkv, Q, g, d) / total.clamp(min=1e-38)
    lse = (m + total.log()).squeeze(-1)
    seq, i = _row_seq(s["cu_q"], s["T"])
    o = o.permute(0, 2, 1, 3, 4).reshape(B, Q, hq, d)[seq, i]
    return o.to(torch.bfloat16), lse.permute(0, 2, 1, 3).reshape(B, Q, hq)[seq, i]


def _plain_sampled(s):
    B, T, Q, V = s["B"], s["T"], s["Q"], s["case"]["vocab"]
    x = s["logits"].double()                                           # acceptances next to a border: in 64 bits
    cu = s["cu_q"].long()
    seq, i = _row_seq(s["cu_q"], T)
    heat = s["temperature"].double()[seq][:, None]
    v = torch.arange(V, device="cuda")
    top = x.amax(1, keepdim=True)
    best = torch.where(x == top, v, V).amin(1)                         # ties to the lowest index
    p = ((x - top) / torch.where(heat > 0, heat, 1.0)).exp()
    p = torch.where(heat > 0, p / p.sum(1, keepdim=True), (v == best[:, None]).double())
    depth = (cu[1:] - cu[:-1]) - 1
    drafted = i < depth[seq]
    at = torch.where(drafted, cu[seq] - seq + i, 0)
    token = s["drafts"].long()[at]
    q_token = s["probs"][at, token].double() if s["probs"] is not None else torch.ones(T, device="cuda", dtype=torch.float64)
    keeps = drafted & (s["uniform"].double()[at] * q_token < p.gather(1, token[:, None])[:, 0])
    n = _padded(keeps.long(), s["cu_q"], Q, 0).cumprod(1).sum(1)       # the first refused draft
    last = cu[:-1] + n
    p = p[last]
    refused = n < depth
    where = torch.where(refused, cu[:-1] - torch.arange(B, device="cuda") + n, 0)
    q = s["probs"][where].double() if s["probs"] is not None else (v == s["drafts"].long()[where][:, None]).double()
    left = (p - torch.where(refused[:, None], q, 0.0)).clamp(min=0)
    left = torch.where(left.amax(1, keepdim=True) > 0, left, p)
    bonus = (left / s["noise"].double()).argmax(1)
    bonus = torch.where(s["temperature"] > 0, bonus, best[last])
    committed = torch.where(i < n[seq], token, torch.where(i == n[seq], bonus[seq], -1))
    return n.int(), bonus.int(), committed.int()


def _plain(s):
    op = s["case"]["op"]
    if op.startswith("rope"):
        return _plain_rope(s)
    if op == "packed_append":
        return _plain_packed_append(s)
    return _plain_attend(s) if op == "packed_attend" else _plain_sampled(s)


# ---------------------------------------------------------------------------------------------
# The library's operators
# ---------------------------------------------------------------------------------------------

def _own(s):
    from speculative_decode_verify_attn_gb300 import vfy
    case, ctx, B, T = s["case"], s["ctx"], s["B"], s["T"]
    op = case["op"]
    if op == "rope_rows":
        vfy.vfy_rope(ctx, s["rope"], s["q"], s["k"], s["cu_q"], s["seq_len"], s["depth"], s["q_out"], s["k_out"], B)
        return s["q_out"], s["k_out"]
    if op == "rope_swa":
        vfy.vfy_rope_append_swa(ctx, s["rope"], s["q"], s["k"], s["v"], s["cu_q"], s["seq_len"], s["depth"],
                                s["ring_offset"], s["k_dst"], s["v_dst"], s["q_out"], B)
        return s["q_out"], s["k_dst"], s["v_dst"]
    if op == "rope_full":
        vfy.vfy_rope_append_full(ctx, s["rope"], s["q"], s["k"], s["v"], s["cu_q"], s["seq_len"], s["depth"],
                                 s["cu_chunks"], s["slot_of"], s["store_k"], s["store_v"], s["chunks"], s["k_dst"],
                                 s["v_dst"], s["num_slots"], s["q_out"], B)
        return s["q_out"], s["k_dst"], s["v_dst"], s["store_k"], s["store_v"]
    if op == "packed_append":
        g, n = case["scale"], s["touched"].numel()
        vfy.vfy_append_full_packed(ctx, s["k"], s["v"], s["cu_q"], s["seq_len"], s["cu_chunks"], s["slot_of"],
                                   s["store_k"], s["store_v"], s["chunks"], s["k_dst"], s["v_dst"], s["num_slots"], g, g, B)
        vfy.vfy_unpack_chunks(ctx, s["k_dst"], s["v_dst"], s["num_slots"], s["touched_slots"], n, g, g, s["k_read"],
                              s["v_read"])
        vfy.vfy_unpack_chunks(ctx, s["store_k"], s["store_v"], s["chunks"], s["touched"], n, g, g, s["k_stored"],
                              s["v_stored"])
        return s["k_read"], s["v_read"], s["k_stored"], s["v_stored"]
    if op == "packed_attend":
        vfy.vfy_attend_full_packed(ctx, s["q"], s["cu_q"], s["k"], s["v"], s["num_slots"], s["ids"], s["slots"],
                                   s["cu_res"], s["max_res"], s["seq_len"], case["scale"], case["scale"], s["out"],
                                   s["lse"], B)
        return s["out"], s["lse"]
    vfy.vfy_accept_sampled(ctx, s["logits"], case["vocab"], s["temperature"], s["drafts"], s["probs"], s["uniform"],
                           s["noise"], s["cu_q"], T, s["accepted"], s["bonus"], s["committed"], B)
    return s["accepted"], s["bonus"], s["committed"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    nodes, lens = _lengths(case)
    rows = sum(nodes)
    if op == "sampled":
        V, B = case["vocab"], case["seqs"]
        # every row's logits; the noise, and of one drafted row in each sequence the drafter's probabilities
        probs = sum(n > 1 for n in nodes) * V * 4 if case["probs"] else 0
        return {"bytes": rows * (V * (2 if case["bf16"] else 4) + 16) + B * V * 4 + probs, "flops": rows * V * 4}
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["dim"]
    if op == "packed_attend":
        keys = [min(x, c * CHUNK) for x, c in zip(lens, _resident(case))]
        return {"bytes": sum(keys) * hkv * d * 2 * 9 / 16 + rows * hq * (d * 4 + 4),
                "flops": 4 * sum(n * k for n, k in zip(nodes, keys)) * hq * d}
    if op == "packed_append":
        # rows in, 4-bit rows into pool and store; the chunks that hold them read and written as bf16, twice
        touched = sum(-(-x // CHUNK) - (x - n) // CHUNK for n, x in zip(nodes, lens))
        return {"bytes": 2 * hkv * d * (rows * (2 + 2 * 9 / 16) + 2 * touched * CHUNK * (9 / 16 + 2)),
                "flops": rows * 2 * hkv * d * 4}
    copies = {"rope_rows": 0, "rope_swa": 1, "rope_full": 2}[op]
    width = hq * 4 + (hkv * 4 if op == "rope_rows" else hkv * 4 * (1 + copies))
    return {"bytes": rows * width * d, "flops": rows * (hq + hkv) * d * 8}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_turn(s, x, weight, places):
    """Each pair as a complex number, turned by e^(i position frequency)."""
    rot, d = s["case"]["rot"], x.shape[-1]
    x = x.double()
    if weight is not None:
        x = x / ((x * x).sum(-1, keepdim=True) / d + s["eps"]).sqrt() * weight.double()
    pairs = torch.arange(rot, device="cuda")
    pairs = pairs.view(-1, 2) if s["case"]["pairs"] == "adjacent" else pairs.view(2, -1).T
    z = torch.complex(x[..., pairs[:, 0]], x[..., pairs[:, 1]])
    angle = torch.tensor(places, device="cuda", dtype=torch.float64)[:, None, None] * s["inv_freq"].double()
    z = z * torch.polar(torch.ones_like(angle), angle)
    out = x.clone()
    out[..., pairs[:, 0]], out[..., pairs[:, 1]] = z.real, z.imag
    return out


def _block_rows(s):
    """(sequence, index, position) of every row of the block."""
    cu, lens = s["cu_q"].tolist(), s["seq_len"].tolist()
    return [(b, i, lens[b] - (cu[b + 1] - cu[b]) + i) for b in range(s["B"]) for i in range(cu[b + 1] - cu[b])]


def _exact_rope(s):
    rows = _block_rows(s)
    depth = s["depth"].tolist() if s["depth"] is not None else None
    places = [p if depth is None else p - i + depth[t] for t, (_, i, p) in enumerate(rows)]
    q, k = _exact_turn(s, s["q"], s["q_norm"], places), _exact_turn(s, s["k"], s["k_norm"], places)
    if s["case"]["op"] == "rope_rows":
        return q, k
    phi = s["ring_offset"].tolist() if "ring_offset" in s else None
    first = s["cu_chunks"].tolist() if phi is None else None
    slot_of = s["slot_of"].tolist() if phi is None else None
    names = ("k_dst", "v_dst") if phi is not None else ("k_dst", "v_dst", "store_k", "store_v")
    out = [q]
    for name in names:
        x, new = s[name].double(), k if name in ("k_dst", "store_k") else s["v"].double()
        for t, (b, _, p) in enumerate(rows):
            if phi is not None:
                x[b, :, (p + phi[b]) % RING] = new[t]
            else:
                c = first[b] + p // CHUNK
                x[c if name.startswith("store") else slot_of[c], :, p % CHUNK] = new[t]
        out.append(x)
    return tuple(out)


def _exact_values(records, d, scale):
    """4-bit chunks as numpy reads them: sign, exponent and mantissa bits one by one."""
    raw = records.cpu().numpy()
    n, hkv = raw.shape[:2]
    codes = raw[..., :32 * d].reshape(n, hkv, d // 32, CHUNK, 16)
    both = np.empty((n, hkv, d // 32, CHUNK, 32), dtype=np.uint8)
    both[..., 0::2], both[..., 1::2] = codes % 16, codes // 16
    both = np.moveaxis(both, 3, 2).reshape(n, hkv, CHUNK, d)
    e, m = (both >> 1) & 3, both & 1
    size = np.where(e == 0, m * 0.5, (1 + 0.5 * m) * 2.0 ** (e.astype(np.int32) - 1))
    values = np.where(both >= 8, -size, size)
    b = raw[..., 32 * d:].reshape(n, hkv, CHUNK, d // 16).astype(np.int32)
    e, m = b >> 3, b & 7                                               # scales are not negative
    steps = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7))
    return values * np.repeat(steps, 16, -1) * scale


def _exact_rounded(x, scale):
    """4-bit values nearest to x / scale in steps of the group's scale: by distance, ties to the even code."""
    T, H, d = x.shape
    x = x.double().cpu().numpy().reshape(T, H, d // 16, 16) / scale
    e4m3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])

    def nearest(y, table):
        hi = np.clip(np.searchsorted(table, y), 1, len(table) - 1)
        lo = hi - 1
        up = (table[hi] - y < y - table[lo]) | ((table[hi] - y == y - table[lo]) & (hi % 2 == 0))
        return table[np.where(up, hi, lo)]

    step = nearest(np.abs(x).max(-1, keepdims=True) / 6, e4m3)
    y = np.abs(x) / np.where(step > 0, step, 1.0) * (step > 0)
    return (np.sign(x) * nearest(np.minimum(y, 6.0), np.array(E2M1[:8])) * step * scale).reshape(T, H, d)


def _exact_packed_append(s):
    d, scale = s["case"]["dim"], s["case"]["scale"]
    first, touched = s["cu_chunks"].tolist(), s["touched"].tolist()
    out = []
    for name, rows, source in (("k_dst", s["touched_slots"], s["k"]), ("v_dst", s["touched_slots"], s["v"]),
                               ("store_k", s["touched"], s["k"]), ("store_v", s["touched"], s["v"])):
        x, new = _exact_values(s[name][rows.long()], d, scale), _exact_rounded(source, scale)
        place = {c: r for r, c in enumerate(touched)}
        for t, (b, _, p) in enumerate(_block_rows(s)):
            x[place[first[b] + p // CHUNK], :, p % CHUNK] = new[t]
        out.append(x)
    return tuple(out)


def _exact_attend(s):
    case = s["case"]
    g, d = case["q_heads"] // case["kv_heads"], case["dim"]
    cu, lens, q = s["cu_q"].tolist(), s["seq_len"].tolist(), s["q"].double()
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, device="cuda", dtype=torch.float64)
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda", dtype=torch.float64)

    def keys(x, rows, h):
        r = x[rows, h].long()
        c = r[:, :32 * d].view(-1, d // 32, CHUNK, 16).permute(0, 2, 1, 3)
        c = torch.stack([c % 16, c // 16], -1).reshape(-1, d // 16, 16)
        f = r[:, 32 * d:].reshape(-1, d // 16, 1)
        e, m = f // 8, (f % 8).double()
        f = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2(e.double() - 7))
        return (table[c % 8] * torch.where(c >= 8, -1.0, 1.0) * f * case["scale"]).reshape(-1, d)

    for b in range(s["B"]):
        n = cu[b + 1] - cu[b]
        r0, r1 = s["cu_res"][b].item(), s["cu_res"][b + 1].item()
        pos = (s["ids"][r0:r1].long()[:, None] * CHUNK + torch.arange(CHUNK, device="cuda")).reshape(-1)
        rows = s["slots"][r0:r1].long()
        see = pos <= (lens[b] - n + torch.arange(n, device="cuda"))[:, None]
        for h in range(case["kv_heads"]):
            K, V = keys(s["k"], rows, h), keys(s["v"], rows, h)
            for hq in range(h * g, h * g + g):
                x = torch.where(see, q[cu[b]:cu[b + 1], hq] @ K.T / math.sqrt(d), -math.inf)
                lse[cu[b]:cu[b + 1], hq] = torch.logsumexp(x, 1)
                out[cu[b]:cu[b + 1], hq] = torch.softmax(x, 1).nan_to_num() @ V
    return out, lse


def _exact_sampled(s):
    cu, drafts, heat = s["cu_q"].tolist(), s["drafts"].tolist(), s["temperature"].tolist()
    uniform = s["uniform"].double().cpu().numpy()
    accepted, bonus, committed = [], [], np.full(s["T"], -1)
    for b in range(s["B"]):
        x = s["logits"][cu[b]:cu[b + 1]].double().cpu().numpy()
        noise = s["noise"][b].double().cpu().numpy()
        depth = len(x) - 1
        for j in range(depth + 1):
            if heat[b] > 0:
                p = np.exp((x[j] - x[j].max()) / heat[b])
                p /= p.sum()
            else:
                p = (np.arange(x.shape[1]) == x[j].argmax()).astype(np.float64)
            at = cu[b] - b + j
            q = np.zeros_like(p)
            if j < depth:
                if s["probs"] is None:
                    q[drafts[at]] = 1.0
                else:
                    q = s["probs"][at].double().cpu().numpy()
                if uniform[at] * q[drafts[at]] < p[drafts[at]]:
                    committed[cu[b] + j] = drafts[at]
                    continue
            left = np.maximum(p - q, 0)
            left = left if left.max() > 0 else p
            token = (left / noise).argmax() if heat[b] > 0 else p.argmax()
            break
        accepted.append(j)
        bonus.append(token)
        committed[cu[b] + j] = token
    return tuple(np.asarray(a, dtype=np.int32) for a in (accepted, bonus, committed))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rope"):
        return _exact_rope(s)
    if case["op"] == "packed_append":
        return _exact_packed_append(s)
    return _exact_attend(s) if case["op"] == "packed_attend" else _exact_sampled(s)
