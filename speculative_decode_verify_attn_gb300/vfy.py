"""Thin Python binding of libvfy.so (ctypes). The functions carry the C ABI's names and only
marshal arguments: torch tensors become device (or pinned host) pointers, the current torch CUDA
stream becomes the stream handle. Every step of the verify path runs in the library's kernels.
There is no fallback: if the library is not built, or its device is absent, calls raise."""
from __future__ import annotations

import array
import ctypes
import operator
import os

import torch

from . import build as _build

VFY_OK, VFY_EINVAL, VFY_ECUDA, VFY_ENOMEM, VFY_EUNSUPPORTED, VFY_EDEVICE_INPUT, VFY_EDEVICE_TIMEOUT = range(7)

EXPORTS = ("vfy_create", "vfy_destroy", "vfy_get_status", "vfy_strerror", "vfy_set_splits",
           "vfy_select_resident", "vfy_page_in", "vfy_attend_full", "vfy_attend_swa", "vfy_accept",
           "vfy_accept_static", "vfy_launch_count", "vfy_append_full", "vfy_append_swa",
           "vfy_gate_depths", "vfy_test_wait_timeout", "vfy_set_stable_metadata", "vfy_set_pagein_ctas",
           "vfy_tree_plan", "vfy_attend_full_tree", "vfy_attend_swa_tree", "vfy_process_logits",
           "vfy_count_tokens", "vfy_accept_tree", "vfy_compact_full", "vfy_compact_swa")

MAX_TREE_NODES = 256      # VFY_MAX_TREE_NODES
TREE_WORDS = 8            # VFY_TREE_WORDS
MAX_COMPACT_LAYERS = 64   # VFY_MAX_COMPACT_LAYERS


class VfyError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {strerror(status)} (status {status})")


class Config(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("chunk_tokens", ctypes.c_int), ("window", ctypes.c_int), ("ring_len", ctypes.c_int),
                ("max_seqs", ctypes.c_int), ("max_queries_per_seq", ctypes.c_int),
                ("max_splits", ctypes.c_int), ("softmax_scale", ctypes.c_float)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int


def lib_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libvfy.so (built in-tree by build.build())."""
    global _lib
    if _lib is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                               "(or python -m speculative_decode_verify_attn_gb300.build)")
        L = ctypes.CDLL(path)
        L.vfy_create.argtypes = [ctypes.POINTER(Config), _I, ctypes.POINTER(_P)]
        L.vfy_destroy.argtypes = [_P]
        L.vfy_destroy.restype = None
        L.vfy_get_status.argtypes = [_P, _P]
        L.vfy_strerror.argtypes = [_I]
        L.vfy_strerror.restype = ctypes.c_char_p
        L.vfy_set_splits.argtypes = [_P, _I, _I]
        L.vfy_test_wait_timeout.argtypes = [_P, ctypes.c_uint64]
        L.vfy_set_stable_metadata.argtypes = [_P, _I]
        L.vfy_set_pagein_ctas.argtypes = [_P, _I]
        L.vfy_select_resident.argtypes = [_P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]
        L.vfy_page_in.argtypes = [_P, _P, _P, ctypes.c_int64, _P, _P, _I, _P, _P, _I, _I, _P]
        L.vfy_attend_full.argtypes = [_P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _P, _P, _I, _P]
        L.vfy_attend_swa.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P]
        L.vfy_accept.argtypes = [_P, _P, _I, _P, _P, _I, _P, _P, _P, _I, _P]
        L.vfy_accept_static.argtypes = [_P, _I, _P, _P, _I, _I, _P, _P, _P, _P, _P]
        L.vfy_append_full.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int64, _P, _P, _I, _I, _P]
        L.vfy_append_swa.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I, _P]
        L.vfy_gate_depths.argtypes = [_P, _I, _I, _I, _P]
        L.vfy_tree_plan.argtypes = [_P, _P, _P, _P, _P, _I, _P]
        L.vfy_attend_full_tree.argtypes = [_P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _P, _P, _I, _P]
        L.vfy_attend_swa_tree.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P]
        L.vfy_process_logits.argtypes = [_P, _P, _I, ctypes.c_int64, _I, _P, _I, _P, _P, _I, _P]
        L.vfy_count_tokens.argtypes = [_P, _P, _P, ctypes.c_int64, _I, _I, _P, _I, _I, _P]
        L.vfy_accept_tree.argtypes = [_P, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _I, _P]
        L.vfy_compact_full.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _P, _P, ctypes.c_int64, _P, _P, _I, _I, _P]
        L.vfy_compact_swa.argtypes = [_P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _P]
        L.vfy_launch_count.argtypes = [_P]
        L.vfy_launch_count.restype = ctypes.c_ulonglong
        for name in EXPORTS:
            if name not in ("vfy_destroy", "vfy_strerror", "vfy_launch_count"):
                getattr(L, name).restype = _I
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().vfy_strerror(status).decode()


def _check(status: int, what: str):
    if status != VFY_OK:
        raise VfyError(status, what)


# ---------------------------------------------------------------------------------------------
# Pointer marshalling
# ---------------------------------------------------------------------------------------------

def _dev(t: torch.Tensor | None, dtypes, name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _host(t: torch.Tensor, dtypes, name: str):
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise TypeError(f"{name} must be a host tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


BF16 = (torch.bfloat16, torch.int16)
I32 = (torch.int32,)
F32 = (torch.float32,)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# The tree calls run once or more per layer or step, and a call's checks in Python cost more than its
# launch: these helpers take 0.23 us a tensor and 0.1 us for the stream (torch.cuda.current_stream()
# builds a Stream object: 3 us).
_DEVICE_OF, _CONTIGUOUS, _DATA_PTR = torch.Tensor.get_device, torch.Tensor.is_contiguous, torch.Tensor.data_ptr

def _raw_stream(ctx, stream) -> int:
    """The handle of `stream`, or of the current stream of the context's device."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(ctx.device)


def _ptr(ctx, t, dtypes, name: str):
    """Address of a contiguous tensor on the context's device (None for None)."""
    if t is None:
        return None
    try:
        if _DEVICE_OF(t) == ctx.device and t.dtype in dtypes and _CONTIGUOUS(t):
            return _DATA_PTR(t)
    except TypeError:
        pass                           # not a tensor
    _dev(t, dtypes, name)              # says what is wrong with any other tensor
    raise ValueError(f"{name} is on {t.device}, the context on cuda:{ctx.device}")


# ---------------------------------------------------------------------------------------------
# The C ABI, one function each
# ---------------------------------------------------------------------------------------------

class Context:
    """Owns a vfy_ctx (created by vfy_create, freed by vfy_destroy / close())."""

    def __init__(self, handle: ctypes.c_void_p, cfg: Config, device: int):
        self.handle = handle
        self.cfg = cfg
        self.device = device

    def close(self):
        if self.handle:
            lib().vfy_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def vfy_create(num_q_heads: int, num_kv_heads: int, head_dim: int, *, window: int = 512,
               ring_len: int = 2048, max_seqs: int = 1, max_queries_per_seq: int = 17,
               max_splits: int = 64, softmax_scale: float = 0.0, device: int | None = None,
               chunk_tokens: int = 64) -> Context:
    dev = torch.cuda.current_device() if device is None else int(device)
    cfg = Config(num_q_heads, num_kv_heads, head_dim, chunk_tokens, window, ring_len, max_seqs,
                 max_queries_per_seq, max_splits, softmax_scale)
    h = ctypes.c_void_p()
    _check(lib().vfy_create(ctypes.byref(cfg), dev, ctypes.byref(h)), "vfy_create")
    return Context(h, cfg, dev)


def vfy_destroy(ctx: Context):
    ctx.close()


def vfy_get_status(ctx: Context, stream=None) -> int:
    return lib().vfy_get_status(ctx.handle, _stream(stream))


def vfy_launch_count(ctx: Context) -> int:
    return int(lib().vfy_launch_count(ctx.handle))


def vfy_gate_depths(confidence, row_budget: int, max_depth: int) -> list[int]:
    """Host function (no device): confidence-gated draft depths. `confidence` is a sequence of
    per-sequence acceptance probabilities in [0, 1]."""
    import numpy as _np
    c = _np.ascontiguousarray(_np.asarray(confidence, dtype=_np.float32))
    d = _np.zeros(len(c), dtype=_np.int32)
    _check(lib().vfy_gate_depths(c.ctypes.data_as(_P), len(c), int(row_budget), int(max_depth),
                                 d.ctypes.data_as(_P)), "vfy_gate_depths")
    return d.tolist()


def vfy_set_splits(ctx: Context, full_splits: int = 0, swa_splits: int = 0):
    _check(lib().vfy_set_splits(ctx.handle, full_splits, swa_splits), "vfy_set_splits")


def vfy_test_wait_timeout(ctx: Context, limit_ns: int = 0):
    """Test of the timeout path: every attention CTA enqueued afterwards first runs one wait of
    limit_ns that cannot complete (0 turns the test off). See include/vfy.h."""
    _check(lib().vfy_test_wait_timeout(ctx.handle, int(limit_ns)), "vfy_test_wait_timeout")


def vfy_set_pagein_ctas(ctx: Context, ctas_per_chunk: int = 0):
    """CTAs per chunk of the page-ins enqueued afterwards (1-4; 0 = 2). See include/vfy.h."""
    _check(lib().vfy_set_pagein_ctas(ctx.handle, int(ctas_per_chunk)), "vfy_set_pagein_ctas")


def vfy_set_stable_metadata(ctx: Context, stable: bool = True):
    """Declare that this context's per-step attention metadata is final before its kernels start
    (see include/vfy.h); the kernels then read it before waiting for the previous kernel."""
    _check(lib().vfy_set_stable_metadata(ctx.handle, 1 if stable else 0), "vfy_set_stable_metadata")


def vfy_select_resident(ctx: Context, scores, cu_chunks, num_seqs: int, max_chunks_per_seq: int, k: int,
                        slot_of_chunk, resident_ids, resident_slots, cu_resident, pagein_list,
                        pagein_count, stream=None):
    _check(lib().vfy_select_resident(
        ctx.handle, _dev(scores, F32, "scores"), _dev(cu_chunks, I32, "cu_chunks"), num_seqs,
        max_chunks_per_seq, k, _dev(slot_of_chunk, I32, "slot_of_chunk"),
        _dev(resident_ids, I32, "resident_ids"), _dev(resident_slots, I32, "resident_slots"),
        _dev(cu_resident, I32, "cu_resident"), _dev(pagein_list, I32, "pagein_list"),
        _dev(pagein_count, I32, "pagein_count"), _stream(stream)), "vfy_select_resident")


def vfy_page_in(ctx: Context, host_k, host_v, num_host_chunks: int, k_pool, v_pool, num_slots: int,
                pagein_list, pagein_count, num_seqs: int, k: int, stream=None):
    hk = _dev(host_k, BF16, "host_k") if host_k.is_cuda else _host(host_k, BF16, "host_k")
    hv = _dev(host_v, BF16, "host_v") if host_v.is_cuda else _host(host_v, BF16, "host_v")
    _check(lib().vfy_page_in(
        ctx.handle, hk, hv, num_host_chunks, _dev(k_pool, BF16, "k_pool"), _dev(v_pool, BF16, "v_pool"),
        num_slots, _dev(pagein_list, I32, "pagein_list"), _dev(pagein_count, I32, "pagein_count"),
        num_seqs, k, _stream(stream)), "vfy_page_in")


def vfy_append_full(ctx: Context, k_new, v_new, cu_q, seq_len, cu_chunks, slot_of_chunk, host_k, host_v,
                    num_host_chunks: int, k_pool, v_pool, num_slots: int, num_seqs: int, stream=None):
    hk = _dev(host_k, BF16, "host_k") if host_k.is_cuda else _host(host_k, BF16, "host_k")
    hv = _dev(host_v, BF16, "host_v") if host_v.is_cuda else _host(host_v, BF16, "host_v")
    _check(lib().vfy_append_full(
        ctx.handle, _dev(k_new, BF16, "k_new"), _dev(v_new, BF16, "v_new"), _dev(cu_q, I32, "cu_q"),
        _dev(seq_len, I32, "seq_len"), _dev(cu_chunks, I32, "cu_chunks"), _dev(slot_of_chunk, I32, "slot_of_chunk"),
        hk, hv, num_host_chunks, _dev(k_pool, BF16, "k_pool"), _dev(v_pool, BF16, "v_pool"), num_slots, num_seqs,
        _stream(stream)), "vfy_append_full")


def vfy_append_swa(ctx: Context, k_new, v_new, cu_q, seq_len, ring_offset, k_ring, v_ring, num_seqs: int,
                   stream=None):
    _check(lib().vfy_append_swa(
        ctx.handle, _dev(k_new, BF16, "k_new"), _dev(v_new, BF16, "v_new"), _dev(cu_q, I32, "cu_q"),
        _dev(seq_len, I32, "seq_len"), _dev(ring_offset, I32, "ring_offset"), _dev(k_ring, BF16, "k_ring"),
        _dev(v_ring, BF16, "v_ring"), num_seqs, _stream(stream)), "vfy_append_swa")


def vfy_attend_full(ctx: Context, q, cu_q, k_pool, v_pool, num_slots: int, resident_ids, resident_slots,
                    cu_resident, max_resident_per_seq: int, seq_len, out, lse, num_seqs: int, stream=None):
    _check(lib().vfy_attend_full(
        ctx.handle, _dev(q, BF16, "q"), _dev(cu_q, I32, "cu_q"), _dev(k_pool, BF16, "k_pool"),
        _dev(v_pool, BF16, "v_pool"), num_slots, _dev(resident_ids, I32, "resident_ids"),
        _dev(resident_slots, I32, "resident_slots"), _dev(cu_resident, I32, "cu_resident"),
        max_resident_per_seq, _dev(seq_len, I32, "seq_len"), _dev(out, BF16, "out"),
        _dev(lse, F32, "lse"), num_seqs, _stream(stream)), "vfy_attend_full")


def vfy_attend_swa(ctx: Context, q, cu_q, k_ring, v_ring, ring_offset, seq_len, out, lse, num_seqs: int,
                   stream=None):
    _check(lib().vfy_attend_swa(
        ctx.handle, _dev(q, BF16, "q"), _dev(cu_q, I32, "cu_q"), _dev(k_ring, BF16, "k_ring"),
        _dev(v_ring, BF16, "v_ring"), _dev(ring_offset, I32, "ring_offset"), _dev(seq_len, I32, "seq_len"),
        _dev(out, BF16, "out"), _dev(lse, F32, "lse"), num_seqs, _stream(stream)), "vfy_attend_swa")


def vfy_accept(ctx: Context, logits, vocab: int, drafts, cu_rows, max_rows: int, accepted_len, bonus,
               committed, num_seqs: int, stream=None):
    _check(lib().vfy_accept(
        ctx.handle, _dev(logits, F32, "logits"), vocab, _dev(drafts, I32, "drafts"), _dev(cu_rows, I32, "cu_rows"),
        max_rows, _dev(accepted_len, I32, "accepted_len"), _dev(bonus, I32, "bonus"),
        _dev(committed, I32, "committed"), num_seqs, _stream(stream)), "vfy_accept")


def vfy_accept_static(logits, vocab: int, drafts, cu_rows, num_seqs: int, max_rows: int, accepted_len, bonus,
                      committed, device_error=None, stream=None):
    """vfy_accept without a context and without allocating (for callers that cannot allocate
    device memory); max_rows <= 1024. See include/vfy.h."""
    _check(lib().vfy_accept_static(
        _dev(logits, F32, "logits"), vocab, _dev(drafts, I32, "drafts"), _dev(cu_rows, I32, "cu_rows"),
        num_seqs, max_rows, _dev(accepted_len, I32, "accepted_len"), _dev(bonus, I32, "bonus"),
        _dev(committed, I32, "committed"), _dev(device_error, I32, "device_error"), _stream(stream)),
        "vfy_accept_static")


# ---------------------------------------------------------------------------------------------
# Tree speculation
# ---------------------------------------------------------------------------------------------

U32 = (torch.int32, torch.uint32)       # row and grammar masks: 32-bit words
_DTYPE = operator.attrgetter("dtype")
_BF16_SET = frozenset(BF16)


class LogitRules:
    """What vfy_process_logits does to the logits (vfy_logit_rules; every tensor may be None). Keeps
    the tensors alive: build it once for buffers that stay where they are."""

    class _Struct(ctypes.Structure):
        _fields_ = [("counts", _P), ("repetition", _P), ("frequency", _P), ("presence", _P), ("drafts", _P),
                    ("tree_mask", _P), ("cu_bias", _P), ("bias_token", _P), ("bias_value", _P), ("grammar", _P),
                    ("mask_index", _P), ("num_masks", _I)]

    def __init__(self, counts=None, repetition=None, frequency=None, presence=None, drafts=None, tree_mask=None,
                 cu_bias=None, bias_token=None, bias_value=None, grammar=None, mask_index=None):
        self.tensors = (counts, repetition, frequency, presence, drafts, tree_mask, cu_bias, bias_token, bias_value,
                        grammar, mask_index)
        self.struct = LogitRules._Struct(
            _dev(counts, I32, "counts"), _dev(repetition, F32, "repetition"), _dev(frequency, F32, "frequency"),
            _dev(presence, F32, "presence"), _dev(drafts, I32, "drafts"), _dev(tree_mask, U32, "tree_mask"),
            _dev(cu_bias, I32, "cu_bias"), _dev(bias_token, I32, "bias_token"), _dev(bias_value, F32, "bias_value"),
            _dev(grammar, U32, "grammar"), _dev(mask_index, I32, "mask_index"),
            0 if grammar is None else grammar.shape[0])
        self.vocab = None if counts is None else counts.shape[-1]
        self.mask_words = None if grammar is None else grammar.shape[-1]
        self.devices = {t.get_device() for t in self.tensors if t is not None}


def vfy_tree_plan(ctx: Context, parents, cu_q, depth, tree_mask, num_seqs: int, stream=None):
    _check(lib().vfy_tree_plan(
        ctx.handle, _ptr(ctx, parents, I32, "parents"), _ptr(ctx, cu_q, I32, "cu_q"), _ptr(ctx, depth, I32, "depth"),
        _ptr(ctx, tree_mask, U32, "tree_mask"), num_seqs, _raw_stream(ctx, stream)), "vfy_tree_plan")


def vfy_attend_full_tree(ctx: Context, q, cu_q, tree_mask, k_pool, v_pool, num_slots: int, resident_ids,
                         resident_slots, cu_resident, max_resident_per_seq: int, seq_len, out, lse, num_seqs: int,
                         stream=None):
    _check(lib().vfy_attend_full_tree(
        ctx.handle, _ptr(ctx, q, BF16, "q"), _ptr(ctx, cu_q, I32, "cu_q"), _ptr(ctx, tree_mask, U32, "tree_mask"),
        _ptr(ctx, k_pool, BF16, "k_pool"), _ptr(ctx, v_pool, BF16, "v_pool"), num_slots,
        _ptr(ctx, resident_ids, I32, "resident_ids"), _ptr(ctx, resident_slots, I32, "resident_slots"),
        _ptr(ctx, cu_resident, I32, "cu_resident"), max_resident_per_seq, _ptr(ctx, seq_len, I32, "seq_len"),
        _ptr(ctx, out, BF16, "out"), _ptr(ctx, lse, F32, "lse"), num_seqs, _raw_stream(ctx, stream)),
        "vfy_attend_full_tree")


def vfy_attend_swa_tree(ctx: Context, q, cu_q, tree_mask, depth, k_ring, v_ring, ring_offset, seq_len, out, lse,
                        num_seqs: int, stream=None):
    _check(lib().vfy_attend_swa_tree(
        ctx.handle, _ptr(ctx, q, BF16, "q"), _ptr(ctx, cu_q, I32, "cu_q"), _ptr(ctx, tree_mask, U32, "tree_mask"),
        _ptr(ctx, depth, I32, "depth"), _ptr(ctx, k_ring, BF16, "k_ring"), _ptr(ctx, v_ring, BF16, "v_ring"),
        _ptr(ctx, ring_offset, I32, "ring_offset"), _ptr(ctx, seq_len, I32, "seq_len"), _ptr(ctx, out, BF16, "out"),
        _ptr(ctx, lse, F32, "lse"), num_seqs, _raw_stream(ctx, stream)), "vfy_attend_swa_tree")


def vfy_process_logits(ctx: Context, logits, vocab: int, cu_rows, max_rows: int, rules: LogitRules, out,
                       num_seqs: int, stream=None):
    """`logits`: fp32 or bf16 [rows][vocab]; its rows may be further apart than `vocab` entries (a view
    of a wider matrix). `out`: fp32 [rows][vocab], or the logits themselves."""
    if logits.get_device() != ctx.device or logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits must be a float32 or bfloat16 tensor on the context's device, got {logits.dtype} on "
                        f"{logits.device}")
    shape, step = logits.shape, logits.stride()
    if len(shape) != 2 or step[1] != 1 or shape[1] < vocab:
        raise ValueError("logits must be [rows][vocab] with contiguous rows")
    if rules.vocab not in (None, vocab) or rules.mask_words not in (None, (vocab + 31) // 32):
        raise ValueError("the rules' counts or grammar masks are for another vocabulary")
    if not rules.devices <= {ctx.device}:
        raise ValueError(f"the rules are on cuda:{sorted(rules.devices)}, the context on cuda:{ctx.device}")
    _check(lib().vfy_process_logits(
        ctx.handle, logits.data_ptr(), 1 if logits.dtype == torch.bfloat16 else 0,
        step[0] if shape[0] > 1 else shape[1], vocab, _ptr(ctx, cu_rows, I32, "cu_rows"),
        max_rows, ctypes.byref(rules.struct), _ptr(ctx, out, F32, "out"), num_seqs, _raw_stream(ctx, stream)),
        "vfy_process_logits")


def vfy_count_tokens(ctx: Context, tokens, cu_tokens, max_tokens: int, counts, vocab: int, num_seqs: int, *,
                     as_prompt: bool = False, reset: bool = False, stream=None):
    _check(lib().vfy_count_tokens(
        ctx.handle, _ptr(ctx, tokens, I32, "tokens"), _ptr(ctx, cu_tokens, I32, "cu_tokens"), max_tokens,
        1 if as_prompt else 0, 1 if reset else 0, _ptr(ctx, counts, I32, "counts"), vocab, num_seqs,
        _raw_stream(ctx, stream)), "vfy_count_tokens")


def vfy_accept_tree(ctx: Context, logits, vocab: int, drafts, parents, cu_rows, max_rows: int, accepted_len, path,
                    bonus, committed, num_seqs: int, stream=None):
    _check(lib().vfy_accept_tree(
        ctx.handle, _ptr(ctx, logits, F32, "logits"), vocab, _ptr(ctx, drafts, I32, "drafts"),
        _ptr(ctx, parents, I32, "parents"), _ptr(ctx, cu_rows, I32, "cu_rows"), max_rows,
        _ptr(ctx, accepted_len, I32, "accepted_len"), _ptr(ctx, path, I32, "path"), _ptr(ctx, bonus, I32, "bonus"),
        _ptr(ctx, committed, I32, "committed"), num_seqs, _raw_stream(ctx, stream)), "vfy_accept_tree")


def _layers(ctx, name: str, *lists, host_allowed: bool = False):
    """One host array of the addresses of all layers of these lists (keep it while the call runs), and the address of
    each list's part."""
    tensors = [t for ts in lists for t in ts]
    # (in C where possible: a call names up to 256 tensors)
    if (set(map(_DEVICE_OF, tensors)) <= {ctx.device} and all(map(_CONTIGUOUS, tensors))
            and set(map(_DTYPE, tensors)) <= _BF16_SET):
        found = array.array("Q", map(_DATA_PTR, tensors))
    else:
        found = array.array("Q", [_host(t, BF16, name).value or 0 if host_allowed and not t.is_cuda
                                  else _ptr(ctx, t, BF16, name) for t in tensors])
    at, step = found.buffer_info()[0], 8 * len(lists[0])
    return found, *(at + step * i for i in range(len(lists)))


def vfy_compact_full(ctx: Context, path, accepted_len, cu_q, seq_len, cu_chunks, slot_of_chunk, host_k, host_v,
                     num_host_chunks: int, k_pool, v_pool, num_slots: int, num_seqs: int, stream=None):
    """host_k, host_v, k_pool, v_pool: one tensor per layer, in lists of one length."""
    if not len(host_k) == len(host_v) == len(k_pool) == len(v_pool):
        raise ValueError("host_k, host_v, k_pool and v_pool must have one tensor per layer")
    stores, hk, hv = _layers(ctx, "host_k, host_v", host_k, host_v, host_allowed=True)
    pools, kp, vp = _layers(ctx, "k_pool, v_pool", k_pool, v_pool)
    _check(lib().vfy_compact_full(
        ctx.handle, _ptr(ctx, path, I32, "path"), _ptr(ctx, accepted_len, I32, "accepted_len"),
        _ptr(ctx, cu_q, I32, "cu_q"), _ptr(ctx, seq_len, I32, "seq_len"), _ptr(ctx, cu_chunks, I32, "cu_chunks"),
        _ptr(ctx, slot_of_chunk, I32, "slot_of_chunk"), len(k_pool), hk, hv, num_host_chunks, kp, vp, num_slots,
        num_seqs, _raw_stream(ctx, stream)), "vfy_compact_full")


def vfy_compact_swa(ctx: Context, path, accepted_len, cu_q, seq_len, ring_offset, k_ring, v_ring, num_seqs: int,
                    stream=None):
    """k_ring, v_ring: one tensor per layer, in lists of one length."""
    if len(k_ring) != len(v_ring):
        raise ValueError("k_ring and v_ring must have one tensor per layer")
    rings, kr, vr = _layers(ctx, "k_ring, v_ring", k_ring, v_ring)
    _check(lib().vfy_compact_swa(
        ctx.handle, _ptr(ctx, path, I32, "path"), _ptr(ctx, accepted_len, I32, "accepted_len"),
        _ptr(ctx, cu_q, I32, "cu_q"), _ptr(ctx, seq_len, I32, "seq_len"), _ptr(ctx, ring_offset, I32, "ring_offset"),
        len(k_ring), kr, vr, num_seqs, _raw_stream(ctx, stream)), "vfy_compact_swa")
