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
           "vfy_count_tokens", "vfy_accept_tree", "vfy_compact_full", "vfy_compact_swa",
           "vfy_rope", "vfy_rope_append_full", "vfy_rope_append_swa", "vfy_append_full_packed", "vfy_page_in_packed",
           "vfy_unpack_chunks", "vfy_attend_full_packed", "vfy_accept_sampled")

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
        i64, f32 = ctypes.c_int64, ctypes.c_float
        L.vfy_rope.argtypes = [_P, _P, _P, i64, _P, i64, _P, _P, _P, _P, _P, _I, _P]
        L.vfy_rope_append_full.argtypes = [_P, _P, _P, i64, _P, i64, _P, i64, _P, _P, _P, _P, _P, _P, _P, i64, _P, _P, _I, _P,
                                           _I, _P]
        L.vfy_rope_append_swa.argtypes = [_P, _P, _P, i64, _P, i64, _P, i64, _P, _P, _P, _P, _P, _P, _P, _I, _P]
        L.vfy_append_full_packed.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, i64, _P, _P, _I, f32, f32, _I, _P]
        L.vfy_page_in_packed.argtypes = [_P, _P, _P, i64, _P, _P, _I, _P, _P, _I, _I, _P]
        L.vfy_unpack_chunks.argtypes = [_P, _P, _P, _I, _P, _I, f32, f32, _P, _P, _P]
        L.vfy_attend_full_packed.argtypes = [_P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, f32, f32, _P, _P, _I, _P]
        L.vfy_accept_sampled.argtypes = [_P, _P, _I, i64, _I, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P]
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
_NUMEL = torch.Tensor.numel

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
        self.heads = cfg.num_q_heads, cfg.num_kv_heads, cfg.head_dim   # (a field of a Structure costs 0.1 us)
        self.chunk_bytes = cfg.num_kv_heads * packed_bytes(cfg.head_dim)   # of a chunk's 4-bit records

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


# ---------------------------------------------------------------------------------------------
# Position rotation and append
# ---------------------------------------------------------------------------------------------

class Rope:
    """How a layer normalises and rotates its queries and keys (vfy_rotary). Keeps the tensors alive: build it once
    per layer. `inv_freq`: float32 [rot_dim / 2] on the device (None: no rotation); `q_norm`, `k_norm`: bf16 [d]."""

    class _Struct(ctypes.Structure):
        _fields_ = [("inv_freq", _P), ("rot_dim", _I), ("interleaved", _I), ("attention_factor", ctypes.c_float),
                    ("q_norm", _P), ("k_norm", _P), ("eps", ctypes.c_float)]

    def __init__(self, inv_freq=None, rot_dim: int | None = None, interleaved: bool = False, attention_factor: float = 1.0,
                 q_norm=None, k_norm=None, eps: float = 1e-6):
        rot_dim = 2 * (0 if inv_freq is None else inv_freq.numel()) if rot_dim is None else int(rot_dim)
        if inv_freq is not None and inv_freq.numel() != rot_dim // 2:
            raise ValueError(f"inv_freq must have rot_dim / 2 = {rot_dim // 2} entries, got {inv_freq.numel()}")
        self.tensors = (inv_freq, q_norm, k_norm)
        self.norm_dims = {t.numel() for t in (q_norm, k_norm) if t is not None}
        self.struct = Rope._Struct(_dev(inv_freq, F32, "inv_freq"), rot_dim, 1 if interleaved else 0, attention_factor,
                                   _dev(q_norm, BF16, "q_norm"), _dev(k_norm, BF16, "k_norm"), eps)
        self.at = ctypes.addressof(self.struct)
        self.devices = {t.get_device() for t in self.tensors if t is not None}
        self.fits = set()                  # (device, head dim) of contexts that it was found to suit


def _rows(ctx, t, side: int, name: str):
    """Address and row stride of bf16 rows [T][heads][d] (or [T][heads * d]), whose rows may lie further apart. `side`: 0 for
    query heads, 1 for KV heads."""
    if t is None:
        return None, 0
    heads, d = ctx.heads[side], ctx.heads[2]
    shape, step = t.shape, t.stride()
    if t.dtype not in BF16 or _DEVICE_OF(t) != ctx.device:
        raise TypeError(f"{name} must be a bf16 tensor on cuda:{ctx.device}, got {t.dtype} on {t.device}")
    if len(shape) == 3:
        ok = shape[2] == d and shape[1] == heads and step[2] == 1 and (step[1] == d or heads == 1)
    else:
        ok = len(shape) == 2 and shape[1] == heads * d and step[1] == 1
    if not ok:
        raise ValueError(f"{name} must be [rows][{heads}][{d}] with packed rows, got {tuple(shape)} with strides {step}")
    return _DATA_PTR(t), step[0] if shape[0] > 1 else heads * d    # (one row lies apart from no other, whatever the view says)


def _rope_at(ctx, rope: Rope):
    fit = ctx.device, ctx.heads[2]
    if fit not in rope.fits:
        if not rope.devices <= {ctx.device}:
            raise ValueError(f"the rotation is on cuda:{sorted(rope.devices)}, the context on cuda:{ctx.device}")
        if not rope.norm_dims <= {ctx.heads[2]}:
            raise ValueError(f"q_norm and k_norm must have {ctx.heads[2]} entries")
        rope.fits.add(fit)
    return rope.at


def vfy_rope(ctx: Context, rope: Rope, q, k, cu_q, seq_len, depth, q_out, k_out, num_seqs: int, stream=None):
    """q, k: bf16 rows [T][heads][d], which may be views of a wider matrix; q_out, k_out: contiguous, or q, k themselves."""
    _check(lib().vfy_rope(
        ctx.handle, _rope_at(ctx, rope), *_rows(ctx, q, 0, "q"), *_rows(ctx, k, 1, "k"), _ptr(ctx, cu_q, I32, "cu_q"), _ptr(ctx, seq_len, I32, "seq_len"),
        _ptr(ctx, depth, I32, "depth"), _ptr(ctx, q_out, BF16, "q_out"), _ptr(ctx, k_out, BF16, "k_out"), num_seqs,
        _raw_stream(ctx, stream)), "vfy_rope")


def _store(ctx, t, dtypes, name: str):
    """Address of a chunk store: on the context's device, or in (pinned) host memory."""
    return _host(t, dtypes, name) if isinstance(t, torch.Tensor) and not t.is_cuda else _ptr(ctx, t, dtypes, name)


def vfy_rope_append_full(ctx: Context, rope: Rope, q, k, v, cu_q, seq_len, depth, cu_chunks, slot_of_chunk, host_k, host_v,
                         num_host_chunks: int, k_pool, v_pool, num_slots: int, q_out, num_seqs: int, stream=None):
    _check(lib().vfy_rope_append_full(
        ctx.handle, _rope_at(ctx, rope), *_rows(ctx, q, 0, "q"), *_rows(ctx, k, 1, "k"), *_rows(ctx, v, 1, "v"),
        _ptr(ctx, cu_q, I32, "cu_q"), _ptr(ctx, seq_len, I32, "seq_len"), _ptr(ctx, depth, I32, "depth"),
        _ptr(ctx, cu_chunks, I32, "cu_chunks"), _ptr(ctx, slot_of_chunk, I32, "slot_of_chunk"),
        _store(ctx, host_k, BF16, "host_k"), _store(ctx, host_v, BF16, "host_v"), num_host_chunks,
        _ptr(ctx, k_pool, BF16, "k_pool"), _ptr(ctx, v_pool, BF16, "v_pool"), num_slots,
        _ptr(ctx, q_out, BF16, "q_out"), num_seqs, _raw_stream(ctx, stream)), "vfy_rope_append_full")


def vfy_rope_append_swa(ctx: Context, rope: Rope, q, k, v, cu_q, seq_len, depth, ring_offset, k_ring, v_ring, q_out,
                        num_seqs: int, stream=None):
    _check(lib().vfy_rope_append_swa(
        ctx.handle, _rope_at(ctx, rope), *_rows(ctx, q, 0, "q"), *_rows(ctx, k, 1, "k"), *_rows(ctx, v, 1, "v"),
        _ptr(ctx, cu_q, I32, "cu_q"), _ptr(ctx, seq_len, I32, "seq_len"), _ptr(ctx, depth, I32, "depth"),
        _ptr(ctx, ring_offset, I32, "ring_offset"), _ptr(ctx, k_ring, BF16, "k_ring"), _ptr(ctx, v_ring, BF16, "v_ring"),
        _ptr(ctx, q_out, BF16, "q_out"), num_seqs, _raw_stream(ctx, stream)), "vfy_rope_append_swa")


# ---------------------------------------------------------------------------------------------
# The 4-bit pool
# ---------------------------------------------------------------------------------------------

U8 = (torch.uint8,)


def packed_bytes(head_dim: int) -> int:
    """Bytes of one (chunk, KV head) record of K or V (VFY_PACKED_BYTES): pools are uint8 [slots][Hkv][this]."""
    return 36 * head_dim


def _records(ctx, t, count: int, name: str, address=_ptr):
    """Address of `count` chunks' records: uint8 [chunks][Hkv][packed_bytes(d)] (a chunk's records, or all, may be one row of
    bytes), no fewer chunks than `count`: the library knows the address alone."""
    at = address(ctx, t, U8, name)
    if at is not None and _NUMEL(t) != count * ctx.chunk_bytes:        # (as many bytes as that are those records)
        _, hkv, d = ctx.heads
        size, shape = packed_bytes(d), t.shape
        fits = shape[-1] == size or len(shape) == 1 or (len(shape) == 2 and shape[1] == hkv * size)
        if not fits or t.numel() < count * hkv * size:
            raise ValueError(f"{name} must hold {count} chunks of {hkv} records of {size} bytes, got {tuple(shape)}")
    return at


def vfy_append_full_packed(ctx: Context, k_new, v_new, cu_q, seq_len, cu_chunks, slot_of_chunk, host_k, host_v,
                           num_host_chunks: int, k_pool, v_pool, num_slots: int, k_scale: float, v_scale: float,
                           num_seqs: int, stream=None):
    _check(lib().vfy_append_full_packed(
        ctx.handle, _ptr(ctx, k_new, BF16, "k_new"), _ptr(ctx, v_new, BF16, "v_new"), _ptr(ctx, cu_q, I32, "cu_q"),
        _ptr(ctx, seq_len, I32, "seq_len"), _ptr(ctx, cu_chunks, I32, "cu_chunks"),
        _ptr(ctx, slot_of_chunk, I32, "slot_of_chunk"), _records(ctx, host_k, num_host_chunks, "host_k", _store),
        _records(ctx, host_v, num_host_chunks, "host_v", _store), num_host_chunks, _records(ctx, k_pool, num_slots, "k_pool"),
        _records(ctx, v_pool, num_slots, "v_pool"), num_slots, k_scale, v_scale, num_seqs, _raw_stream(ctx, stream)),
        "vfy_append_full_packed")


def vfy_page_in_packed(ctx: Context, host_k, host_v, num_host_chunks: int, k_pool, v_pool, num_slots: int, pagein_list,
                       pagein_count, num_seqs: int, k: int, stream=None):
    _check(lib().vfy_page_in_packed(
        ctx.handle, _records(ctx, host_k, num_host_chunks, "host_k", _store),
        _records(ctx, host_v, num_host_chunks, "host_v", _store), num_host_chunks,
        _records(ctx, k_pool, num_slots, "k_pool"), _records(ctx, v_pool, num_slots, "v_pool"), num_slots,
        _ptr(ctx, pagein_list, I32, "pagein_list"), _ptr(ctx, pagein_count, I32, "pagein_count"), num_seqs, k,
        _raw_stream(ctx, stream)), "vfy_page_in_packed")


def vfy_unpack_chunks(ctx: Context, k_pool, v_pool, num_slots: int, slots, num_chunks: int, k_scale: float, v_scale: float,
                      k_out, v_out, stream=None):
    _check(lib().vfy_unpack_chunks(
        ctx.handle, _records(ctx, k_pool, num_slots, "k_pool"), _records(ctx, v_pool, num_slots, "v_pool"), num_slots,
        _ptr(ctx, slots, I32, "slots"), num_chunks, k_scale, v_scale, _ptr(ctx, k_out, BF16, "k_out"),
        _ptr(ctx, v_out, BF16, "v_out"), _raw_stream(ctx, stream)), "vfy_unpack_chunks")


def vfy_attend_full_packed(ctx: Context, q, cu_q, k_pool, v_pool, num_slots: int, resident_ids, resident_slots, cu_resident,
                           max_resident_per_seq: int, seq_len, k_scale: float, v_scale: float, out, lse, num_seqs: int,
                           stream=None):
    _check(lib().vfy_attend_full_packed(
        ctx.handle, _ptr(ctx, q, BF16, "q"), _ptr(ctx, cu_q, I32, "cu_q"), _records(ctx, k_pool, num_slots, "k_pool"),
        _records(ctx, v_pool, num_slots, "v_pool"), num_slots, _ptr(ctx, resident_ids, I32, "resident_ids"),
        _ptr(ctx, resident_slots, I32, "resident_slots"), _ptr(ctx, cu_resident, I32, "cu_resident"), max_resident_per_seq,
        _ptr(ctx, seq_len, I32, "seq_len"), k_scale, v_scale, _ptr(ctx, out, BF16, "out"), _ptr(ctx, lse, F32, "lse"),
        num_seqs, _raw_stream(ctx, stream)), "vfy_attend_full_packed")


# ---------------------------------------------------------------------------------------------
# Sampled acceptance
# ---------------------------------------------------------------------------------------------

def vfy_accept_sampled(ctx: Context, logits, vocab: int, temperature, drafts, draft_probs, uniform, noise, cu_rows,
                       max_rows: int, accepted_len, bonus, committed, num_seqs: int, stream=None):
    """`logits`: fp32 or bf16 [rows][vocab]; its rows may be further apart than `vocab` entries. `draft_probs` (fp32
    [drafts][vocab], None: certain drafts), `uniform` (fp32, one a draft) and `noise` (fp32 [B][vocab], exponentially
    distributed) are the caller's."""
    if _DEVICE_OF(logits) != ctx.device or logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits must be a float32 or bfloat16 tensor on the context's device, got {logits.dtype} on "
                        f"{logits.device}")
    shape, step = logits.shape, logits.stride()
    if len(shape) != 2 or step[1] != 1 or shape[1] < vocab:
        raise ValueError("logits must be [rows][vocab] with contiguous rows")
    for t, name in ((noise, "noise"), (draft_probs, "draft_probs")):
        if t is not None and t.shape[-1] != vocab:
            raise ValueError(f"{name} must have {vocab} entries a row, got {tuple(t.shape)}")
    _check(lib().vfy_accept_sampled(
        ctx.handle, _DATA_PTR(logits), 1 if logits.dtype == torch.bfloat16 else 0, step[0] if shape[0] > 1 else shape[1],
        vocab, _ptr(ctx, temperature, F32, "temperature"), _ptr(ctx, drafts, I32, "drafts"),
        _ptr(ctx, draft_probs, F32, "draft_probs"), _ptr(ctx, uniform, F32, "uniform"), _ptr(ctx, noise, F32, "noise"),
        _ptr(ctx, cu_rows, I32, "cu_rows"), max_rows, _ptr(ctx, accepted_len, I32, "accepted_len"),
        _ptr(ctx, bonus, I32, "bonus"), _ptr(ctx, committed, I32, "committed"), num_seqs, _raw_stream(ctx, stream)),
        "vfy_accept_sampled")
