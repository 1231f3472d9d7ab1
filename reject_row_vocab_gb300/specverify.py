"""Python binding of libspecverify (ctypes; argument marshalling only).

Every step of the verification runs in the CUDA library; this module only
turns torch tensors into device pointers and sizes, calls the C ABI declared
in include/specverify.h on the current torch stream, and raises on a bad
status.  The library must be built (reject_row_vocab_gb300._build.build());
importing this module without it raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SV_F32, SV_BF16 = 0, 1
STATUS = {0: "SV_OK", 1: "SV_ERR_NULL_ARG", 2: "SV_ERR_BAD_SHAPE", 3: "SV_ERR_BAD_DTYPE", 4: "SV_ERR_MISALIGNED",
          5: "SV_ERR_UNSUPPORTED", 6: "SV_ERR_WORKSPACE_TOO_SMALL", 7: "SV_ERR_CUDA"}
DEV_TOKEN_RANGE, DEV_NONFINITE, DEV_BAD_TREE, DEV_BAD_LAYOUT, DEV_RESIDUAL_EMPTY, DEV_DUP_SIBLING = 1, 2, 4, 8, 16, 32
DEV_TIMEOUT, DEV_SLOT_RANGE = 64, 128

ENTRY_POINTS = ("spec_verify_workspace_bytes", "spec_verify_status_string", "spec_verify_greedy_chain",
                "spec_verify_greedy_tree", "spec_verify_rejection_chain", "spec_verify_rejection_ragged",
                "spec_verify_target_only_tree", "spec_verify_row_stats", "spec_verify_set_stats_events",
                "spec_verify_last_cuda_error", "spec_verify_rejection_chain_noalloc",
                "spec_verify_dspark_workspace_bytes", "spec_verify_dspark_budget", "spec_verify_dspark_verify_lens",
                "spec_verify_sparse_workspace_bytes", "spec_verify_rejection_chain_sparse", "spec_verify_build_tree",
                "spec_verify_sample_match_chain", "spec_verify_attention_workspace_bytes",
                "spec_verify_paged_attention", "spec_verify_kv_commit", "spec_verify_logprobs_workspace_bytes",
                "spec_verify_token_logprobs", "spec_verify_token_logprobs_backward", "spec_verify_kv_append",
                "spec_verify_kv_read", "spec_verify_packed_kv_block_bytes", "spec_verify_packed_kv_append",
                "spec_verify_packed_kv_read", "spec_verify_packed_attention", "spec_verify_packed_kv_commit")


class SpecVerifyError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__("%s returned %s (%d): %s" % (fn, STATUS.get(code, "?"), code, msg))
        self.code = code


class SvOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "accept_len", "num_out", "out_tokens", "bonus", "accept_rows", "commit_cu", "commit_src_slot",
        "commit_dst_pos", "dev_status")]


class SvKvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int), ("layers", ctypes.c_int32),
                ("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("max_pages", ctypes.c_int32), ("ld_table", ctypes.c_int64)]


class SvPackedKvCache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int), ("layers", ctypes.c_int32),
                ("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p), ("max_pages", ctypes.c_int32),
                ("ld_table", ctypes.c_int64)]


class SvRows(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_len", ctypes.c_int32), ("total_rows", ctypes.c_int64),
                ("cu_seqlens", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("row_slots", ctypes.c_void_p)]


class SvRotation(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("pairs", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("magnitude", ctypes.c_float)]


_lib = None


def load_library():
    """Load libspecverify.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libspecverify.so is not built (%s); run reject_row_vocab_gb300._build.build()" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, F, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    OUT = ctypes.POINTER(SvOut)
    sig = {
        "spec_verify_workspace_bytes": ([I64, I32, I32, I32], SZ),
        "spec_verify_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "spec_verify_last_cuda_error": ([], ctypes.c_char_p),
        "spec_verify_greedy_chain": ([P, ctypes.c_int, I64, I32, I32, I32, P, P, P, OUT, P, SZ, P], ctypes.c_int),
        "spec_verify_greedy_tree": ([P, ctypes.c_int, I64, I32, I32, I32, P, P, P, P, P, P, OUT, P, SZ, P],
                                    ctypes.c_int),
        "spec_verify_rejection_chain": ([P, ctypes.c_int, I64, I32, I32, I32, P, P, I64, P, P, P, P, P, OUT, P, SZ,
                                         P], ctypes.c_int),
        "spec_verify_rejection_ragged": ([P, ctypes.c_int, I64, I32, I64, I32, I32, P, P, P, I64, P, P, P, P, P,
                                          OUT, P, SZ, P], ctypes.c_int),
        "spec_verify_target_only_tree": ([P, ctypes.c_int, I64, I32, I32, I32, P, P, P, P, P, F, F, P, P, P, P,
                                          OUT, P, SZ, P], ctypes.c_int),
        "spec_verify_row_stats": ([P, ctypes.c_int, I64, I64, I32, P, P, P, P, P, P, P, P, SZ, P], ctypes.c_int),
        "spec_verify_set_stats_events": ([P, P], ctypes.c_int),
        "spec_verify_sparse_workspace_bytes": ([I64, I32, I32, I32, I32], SZ),
        "spec_verify_rejection_chain_sparse": ([P, ctypes.c_int, I64, I32, I32, I32, P, P, P, I32, I64, P, P, P, P, P,
                                                OUT, P, SZ, P], ctypes.c_int),
        "spec_verify_build_tree": ([P, P, I32, I32, P, P, P, P, P, P, P], ctypes.c_int),
        "spec_verify_sample_match_chain": ([P, ctypes.c_int, I64, I32, I32, I32, P, P, P, P, P, OUT, P, SZ, P],
                                           ctypes.c_int),
        "spec_verify_dspark_workspace_bytes": ([I32], SZ),
        "spec_verify_dspark_budget": ([P, I64, I32, P, I32, F, P], ctypes.c_int),
        "spec_verify_dspark_verify_lens": ([P, I32, I32, I64, I32, I32, I32, F, P, P, SZ, P], ctypes.c_int),
        "spec_verify_attention_workspace_bytes": ([I32, I32, I32, I32, I32], SZ),
        "spec_verify_paged_attention": ([P, I64, I64, I32, P, I32, I32, I64, I32, P, P, P, P, F, P, I64, I64, P, P, P,
                                         SZ, P], ctypes.c_int),
        "spec_verify_kv_commit": ([P, I32, I32, I64, P, P, P, P, P], ctypes.c_int),
        "spec_verify_logprobs_workspace_bytes": ([I64, I32, I32], SZ),
        "spec_verify_token_logprobs": ([P, ctypes.c_int, I64, I64, I32, I64, P, P, I32, I64, P, I32, P, P, P, P, P, P,
                                        P, P, SZ, P], ctypes.c_int),
        "spec_verify_token_logprobs_backward": ([P, ctypes.c_int, I64, I64, I32, P, I32, I64, P, P, P, P, P, I32, P, P,
                                                 P, P, I64, P], ctypes.c_int),
        "spec_verify_kv_append": ([P, I32, P, P, P, P, I64, I64, P, I64, I64, P, I64, I64, I32, P, I64, I64, P, P],
                                  ctypes.c_int),
        "spec_verify_kv_read": ([P, I32, I32, P, P, P, I64, I64, I64, P, P], ctypes.c_int),
        "spec_verify_packed_kv_block_bytes": ([I32, I32], SZ),
    }
    for name in ("kv_append", "kv_read", "kv_commit"):
        sig["spec_verify_packed_" + name] = sig["spec_verify_" + name]
    sig["spec_verify_packed_attention"] = sig["spec_verify_paged_attention"]
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# Argument checks.  The library takes raw device pointers and cannot tell a
# host pointer, a wrong element type or a short array from a good one, and the
# kernels would then read or write outside the arrays.  Every tensor is checked
# here before its pointer is passed: on the logits' device, of the element type
# the call reads, densely laid out (2-D arrays may have a row stride), and at
# least as large as the call reads.  None is passed on as NULL; whether an
# argument may be NULL is the library's decision (it returns SV_ERR_NULL_ARG).


def _require_cuda(t: torch.Tensor, name: str = "logits"):
    """The call's leading 2-D array: a CUDA tensor with dense rows; its device is the call's device."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("%s must be a 2-D torch tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (got %s): the library has no CPU path" % (name, t.device))
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s rows must be dense (stride 1 along a row)" % name)


def _arg(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, numel: int, device) -> Optional[torch.Tensor]:
    """A 1-D (or dense N-D) array argument of at least numel elements."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s; the call runs on %s (the logits' device)" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.numel() < numel:
        raise ValueError("%s has %d elements; the call reads %d" % (name, t.numel(), numel))
    return t


def _rows_arg(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, rows: int, cols: int,
              device) -> Optional[torch.Tensor]:
    """A 2-D array argument [>= rows, >= cols] whose rows are dense (any row stride)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("%s must be a 2-D torch tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s; the call runs on %s (the logits' device)" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape[0] < rows or t.shape[1] < cols:
        raise ValueError("%s is %s; the call reads [%d, %d]" % (name, tuple(t.shape), rows, cols))
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s rows must be dense (stride 1 along a row)" % name)
    return t


def _check_out(out: "VerifyOutputs", batch: int, max_len: int, rows: int, device):
    i32, i64 = torch.int32, torch.int64
    _arg(out.accept_len, "out.accept_len", i32, batch, device)
    _arg(out.num_out, "out.num_out", i32, batch, device)
    _arg(out.out_tokens, "out.out_tokens", i32, batch * max_len, device)
    _arg(out.bonus, "out.bonus", i32, batch, device)
    _arg(out.accept_rows, "out.accept_rows", i32, batch * max_len, device)
    _arg(out.commit_cu, "out.commit_cu", i32, batch + 1, device)
    _arg(out.commit_src_slot, "out.commit_src_slot", i64, rows, device)
    _arg(out.commit_dst_pos, "out.commit_dst_pos", i64, rows, device)
    _arg(out.dev_status, "out.dev_status", i32, batch, device)


def _check_ws(ws: torch.Tensor, device):
    _arg(ws, "ws", torch.uint8, 0, device)


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(logits: torch.Tensor) -> int:
    if logits.dtype == torch.bfloat16:
        return SV_BF16
    if logits.dtype == torch.float32:
        return SV_F32
    raise TypeError("logits must be bfloat16 or float32, got %s" % logits.dtype)


def _check(fn: str, code: int):
    if code != 0:
        lib = load_library()
        msg = lib.spec_verify_status_string(code).decode()
        if code == 7:
            msg += " (%s)" % lib.spec_verify_last_cuda_error().decode()
        raise SpecVerifyError(fn, code, msg)


def set_stats_events(start=None, stop=None):
    """Record torch CUDA events around the row-statistics kernel of later calls (None, None: stop).

    The events must already exist on the device (record them once first)."""
    h = lambda e: None if e is None else ctypes.c_void_p(e.cuda_event)
    _check("spec_verify_set_stats_events", load_library().spec_verify_set_stats_events(h(start), h(stop)))


def workspace_bytes(rows: int, batch: int, vocab: int, max_len: int) -> int:
    return int(load_library().spec_verify_workspace_bytes(rows, batch, vocab, max_len))


def workspace(rows: int, batch: int, vocab: int, max_len: int, device=None) -> torch.Tensor:
    """A zero-filled workspace (the library keeps its counters zero between calls)."""
    n = workspace_bytes(rows, batch, vocab, max_len)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


@dataclass
class VerifyOutputs:
    accept_len: torch.Tensor
    num_out: torch.Tensor
    out_tokens: torch.Tensor
    bonus: torch.Tensor
    accept_rows: torch.Tensor
    commit_cu: torch.Tensor
    commit_src_slot: Optional[torch.Tensor]
    commit_dst_pos: Optional[torch.Tensor]
    dev_status: torch.Tensor  # int32 storage of uint32 bits

    @staticmethod
    def allocate(batch: int, max_len: int, rows: int, device=None, slots: bool = True) -> "VerifyOutputs":
        d = device or "cuda"
        i32 = dict(dtype=torch.int32, device=d)
        return VerifyOutputs(
            accept_len=torch.empty(batch, **i32), num_out=torch.empty(batch, **i32),
            out_tokens=torch.empty(batch, max_len, **i32), bonus=torch.empty(batch, **i32),
            accept_rows=torch.empty(batch, max_len, **i32), commit_cu=torch.empty(batch + 1, **i32),
            commit_src_slot=torch.full((max(rows, 1),), -1, dtype=torch.int64, device=d) if slots else None,
            commit_dst_pos=torch.full((max(rows, 1),), -1, dtype=torch.int64, device=d) if slots else None,
            dev_status=torch.empty(batch, **i32))

    def struct(self) -> SvOut:
        return SvOut(*[None if getattr(self, n) is None else getattr(self, n).data_ptr() for n, _ in SvOut._fields_])

    def to_numpy(self) -> dict:
        out = {}
        for n, _ in SvOut._fields_:
            t = getattr(self, n)
            if t is not None:
                a = t.cpu().numpy()
                out["status" if n == "dev_status" else n] = a.view("uint32") if n == "dev_status" else a
        return out


def _prep(out, ws, batch, max_len, rows, vocab, device, slots):
    if out is None:
        out = VerifyOutputs.allocate(batch, max_len, rows, device, slots)
    if ws is None:
        ws = workspace(rows, batch, vocab, max_len, device)
    _check_out(out, batch, max_len, rows, device)
    _check_ws(ws, device)
    return out, ws


def _chain_args(device, rows, batch, verify_ids, row_slots, seq_lens):
    _arg(verify_ids, "verify_ids", torch.int32, rows, device)
    _arg(row_slots, "row_slots", torch.int64, rows, device)
    _arg(seq_lens, "seq_lens", torch.int64, batch, device)


def greedy_chain(logits, verify_ids, m, *, row_slots=None, seq_lens=None, out=None, ws=None, stream=None):
    """Greedy chain verification of logits [batch*(m+1), V]."""
    lib = load_library()
    _require_cuda(logits)
    rows, V = logits.shape
    batch = rows // (m + 1)
    dev = logits.device
    _chain_args(dev, batch * (m + 1), batch, verify_ids, row_slots, seq_lens)
    out, ws = _prep(out, ws, batch, m + 1, rows, V, logits.device, row_slots is not None)
    st = out.struct()
    _check("spec_verify_greedy_chain", lib.spec_verify_greedy_chain(
        _ptr(logits), _dtype(logits), logits.stride(0), batch, m, V, _ptr(verify_ids), _ptr(row_slots),
        _ptr(seq_lens), ctypes.byref(st), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def rejection_chain(logits, verify_ids, m, q, temperature, u_accept, u_final, *, row_slots=None, seq_lens=None,
                    out=None, ws=None, stream=None):
    """p/q rejection chain verification of logits [batch*(m+1), V] with proposal rows q."""
    lib = load_library()
    _require_cuda(logits)
    rows, V = logits.shape
    batch = rows // (m + 1)
    dev, R = logits.device, batch * (m + 1)
    _chain_args(dev, R, batch, verify_ids, row_slots, seq_lens)
    _rows_arg(q, "q", torch.float32, R, V, dev)
    _arg(temperature, "temperature", torch.float32, batch, dev)
    _arg(u_accept, "u_accept", torch.float32, R, dev)
    _arg(u_final, "u_final", torch.float32, batch, dev)
    out, ws = _prep(out, ws, batch, m + 1, rows, V, logits.device, row_slots is not None)
    st = out.struct()
    _check("spec_verify_rejection_chain", lib.spec_verify_rejection_chain(
        _ptr(logits), _dtype(logits), logits.stride(0), batch, m, V, _ptr(verify_ids), _ptr(q), q.stride(0),
        _ptr(temperature), _ptr(u_accept), _ptr(u_final), _ptr(row_slots), _ptr(seq_lens), ctypes.byref(st),
        _ptr(ws), ws.numel(), _stream(stream)))
    return out


def sample_match_chain(logits, verify_ids, m, temperature, u_sample, *, row_slots=None, seq_lens=None, out=None,
                       ws=None, stream=None):
    """Verification by independent target sampling (u_sample per row) and prefix match."""
    lib = load_library()
    _require_cuda(logits)
    rows, V = logits.shape
    batch = rows // (m + 1)
    dev, R = logits.device, batch * (m + 1)
    _chain_args(dev, R, batch, verify_ids, row_slots, seq_lens)
    _arg(temperature, "temperature", torch.float32, batch, dev)
    _arg(u_sample, "u_sample", torch.float32, R, dev)
    out, ws = _prep(out, ws, batch, m + 1, rows, V, logits.device, row_slots is not None)
    st = out.struct()
    _check("spec_verify_sample_match_chain", lib.spec_verify_sample_match_chain(
        _ptr(logits), _dtype(logits), logits.stride(0), batch, m, V, _ptr(verify_ids), _ptr(temperature),
        _ptr(u_sample), _ptr(row_slots), _ptr(seq_lens), ctypes.byref(st), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def sparse_workspace(rows: int, batch: int, vocab: int, max_len: int, num_cands: int, device=None) -> torch.Tensor:
    lib = load_library()
    n = int(lib.spec_verify_sparse_workspace_bytes(rows, batch, vocab, max_len, num_cands))
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def rejection_chain_sparse(logits, verify_ids, m, cand_ids, cand_probs, temperature, u_accept, u_final, *,
                           row_slots=None, seq_lens=None, out=None, ws=None, stream=None):
    """p/q rejection chain whose q is given by candidate lists cand_ids / cand_probs [rows, K]."""
    lib = load_library()
    _require_cuda(logits)
    rows, V = logits.shape
    batch = rows // (m + 1)
    dev, R = logits.device, batch * (m + 1)
    _chain_args(dev, R, batch, verify_ids, row_slots, seq_lens)
    _rows_arg(cand_ids, "cand_ids", torch.int32, R, 0, dev)
    K = cand_ids.shape[1]
    _rows_arg(cand_probs, "cand_probs", torch.float32, R, K, dev)
    if cand_probs is not None and (cand_probs.shape[1] != K or (K > 1 and cand_probs.stride(0) != cand_ids.stride(0))):
        raise ValueError("cand_probs must have cand_ids' shape and row stride")
    _arg(temperature, "temperature", torch.float32, batch, dev)
    _arg(u_accept, "u_accept", torch.float32, R, dev)
    _arg(u_final, "u_final", torch.float32, batch, dev)
    if ws is None:
        ws = sparse_workspace(rows, batch, V, m + 1, K, logits.device)
    out, ws = _prep(out, ws, batch, m + 1, rows, V, logits.device, row_slots is not None)
    st = out.struct()
    _check("spec_verify_rejection_chain_sparse", lib.spec_verify_rejection_chain_sparse(
        _ptr(logits), _dtype(logits), logits.stride(0), batch, m, V, _ptr(verify_ids), _ptr(cand_ids),
        _ptr(cand_probs), K, cand_ids.stride(0), _ptr(temperature), _ptr(u_accept), _ptr(u_final),
        _ptr(row_slots), _ptr(seq_lens), ctypes.byref(st), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def rejection_ragged(logits, cu_seqlens, max_len, verify_ids, q, temperature, u_accept, u_final, *, row_slots=None,
                     seq_lens=None, out=None, ws=None, stream=None):
    """Ragged p/q rejection verification; cu_seqlens [B+1] int32 (lengths include the anchor)."""
    lib = load_library()
    _require_cuda(logits)
    rows, V = logits.shape
    dev = logits.device
    _arg(cu_seqlens, "cu_seqlens", torch.int32, 1, dev)
    batch = cu_seqlens.numel() - 1
    _chain_args(dev, rows, batch, verify_ids, row_slots, seq_lens)
    _rows_arg(q, "q", torch.float32, rows, V, dev)
    _arg(temperature, "temperature", torch.float32, batch, dev)
    _arg(u_accept, "u_accept", torch.float32, rows, dev)
    _arg(u_final, "u_final", torch.float32, batch, dev)
    out, ws = _prep(out, ws, batch, max_len, rows, V, logits.device, row_slots is not None)
    st = out.struct()
    _check("spec_verify_rejection_ragged", lib.spec_verify_rejection_ragged(
        _ptr(logits), _dtype(logits), logits.stride(0), batch, rows, max_len, V, _ptr(cu_seqlens), _ptr(verify_ids),
        _ptr(q), q.stride(0), _ptr(temperature), _ptr(u_accept), _ptr(u_final), _ptr(row_slots), _ptr(seq_lens),
        ctypes.byref(st), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def _tree_args(device, batch, nodes, tokens, parents, first_child, next_sibling, row_slots, seq_lens):
    n = batch * nodes
    _arg(tokens, "tokens", torch.int32, n, device)
    _arg(parents, "parents", torch.int32, n, device)
    _arg(first_child, "first_child", torch.int32, n, device)
    _arg(next_sibling, "next_sibling", torch.int32, n, device)
    _arg(row_slots, "row_slots", torch.int64, n, device)
    _arg(seq_lens, "seq_lens", torch.int64, batch, device)


def greedy_tree(logits, tokens, parents, *, first_child=None, next_sibling=None, row_slots=None, seq_lens=None,
                out=None, ws=None, stream=None):
    """Greedy tree verification; tokens / parents [batch, nodes], logits [batch*nodes, V]."""
    lib = load_library()
    _require_cuda(logits)
    rows, V = logits.shape
    batch, nodes = tokens.shape
    _tree_args(logits.device, batch, nodes, tokens, parents, first_child, next_sibling, row_slots, seq_lens)
    out, ws = _prep(out, ws, batch, nodes, rows, V, logits.device, row_slots is not None)
    st = out.struct()
    _check("spec_verify_greedy_tree", lib.spec_verify_greedy_tree(
        _ptr(logits), _dtype(logits), logits.stride(0), batch, nodes, V, _ptr(tokens), _ptr(parents),
        _ptr(first_child), _ptr(next_sibling), _ptr(row_slots), _ptr(seq_lens), ctypes.byref(st), _ptr(ws),
        ws.numel(), _stream(stream)))
    return out


def target_only_tree(logits, tokens, parents, temperature, u_accept, u_final, *, threshold_single=1.0,
                     threshold_acc=1.0, first_child=None, next_sibling=None, row_slots=None, seq_lens=None, out=None,
                     ws=None, stream=None):
    """Target-only tree sampling; u_accept [batch*nodes], u_final [batch]."""
    lib = load_library()
    _require_cuda(logits)
    rows, V = logits.shape
    batch, nodes = tokens.shape
    dev = logits.device
    _tree_args(dev, batch, nodes, tokens, parents, first_child, next_sibling, row_slots, seq_lens)
    _arg(temperature, "temperature", torch.float32, batch, dev)
    _arg(u_accept, "u_accept", torch.float32, batch * nodes, dev)
    _arg(u_final, "u_final", torch.float32, batch, dev)
    out, ws = _prep(out, ws, batch, nodes, rows, V, logits.device, row_slots is not None)
    st = out.struct()
    _check("spec_verify_target_only_tree", lib.spec_verify_target_only_tree(
        _ptr(logits), _dtype(logits), logits.stride(0), batch, nodes, V, _ptr(tokens), _ptr(parents),
        _ptr(first_child), _ptr(next_sibling), _ptr(temperature), float(threshold_single), float(threshold_acc),
        _ptr(u_accept), _ptr(u_final), _ptr(row_slots), _ptr(seq_lens), ctypes.byref(st), _ptr(ws), ws.numel(),
        _stream(stream)))
    return out


def row_stats(logits, row_temp=None, probe=None, ws=None, stream=None) -> dict:
    """Row maximum, lowest argmax, Z (fp64), p at probe and flags for every row."""
    lib = load_library()
    _require_cuda(logits)
    rows, V = logits.shape
    d = logits.device
    _arg(row_temp, "row_temp", torch.float32, rows, d)
    _arg(probe, "probe", torch.int32, rows, d)
    res = {"max": torch.empty(rows, dtype=torch.float32, device=d),
           "argmax": torch.empty(rows, dtype=torch.int32, device=d),
           "z": torch.empty(rows, dtype=torch.float64, device=d),
           "p": torch.empty(rows, dtype=torch.float32, device=d) if probe is not None else None,
           "flags": torch.empty(rows, dtype=torch.int32, device=d)}
    if ws is None:
        ws = workspace(rows, 1, V, 1, d)
    _check_ws(ws, d)
    _check("spec_verify_row_stats", lib.spec_verify_row_stats(
        _ptr(logits), _dtype(logits), logits.stride(0), rows, V, _ptr(row_temp), _ptr(probe), _ptr(res["max"]),
        _ptr(res["argmax"]), _ptr(res["z"]), _ptr(res["p"]), _ptr(res["flags"]), _ptr(ws), ws.numel(),
        _stream(stream)))
    return res


def dspark_budget(hist_survival, num_requests: int, sps, eps: float = 0.0) -> int:
    """Host budget K* from historical survival scores and a speed table indexed by target rows."""
    lib = load_library()
    h = np.ascontiguousarray(np.asarray(hist_survival, dtype=np.float32).ravel())
    t = np.ascontiguousarray(np.asarray(sps, dtype=np.float32).ravel())
    k = ctypes.c_int32(-1)
    _check("spec_verify_dspark_budget", lib.spec_verify_dspark_budget(
        ctypes.c_void_p(h.ctypes.data) if h.size else None, h.size, int(num_requests),
        ctypes.c_void_p(t.ctypes.data) if t.size else None, t.size, float(eps), ctypes.byref(k)))
    return int(k.value)


def dspark_workspace(num_requests: int, device=None) -> torch.Tensor:
    lib = load_library()
    return torch.zeros(int(lib.spec_verify_dspark_workspace_bytes(int(num_requests))), dtype=torch.uint8,
                       device=device)


def dspark_verify_lens(survival, budget: int, *, min_len: int = 1, max_len: Optional[int] = None, eps: float = 0.0,
                       out=None, ws=None, stream=None) -> torch.Tensor:
    """verify_lens [R] (int32, on survival's device) from the current survival [R, D]."""
    lib = load_library()
    _require_cuda(survival, "survival")
    R, D = survival.shape
    dev = survival.device
    _rows_arg(survival, "survival", torch.float32, R, D, dev)
    if max_len is None:
        max_len = D + 1
    if out is None:
        out = torch.empty(R, dtype=torch.int32, device=survival.device)
    if ws is None:
        ws = dspark_workspace(R, survival.device)
    _arg(out, "out", torch.int32, R, dev)
    _check_ws(ws, dev)
    _check("spec_verify_dspark_verify_lens", lib.spec_verify_dspark_verify_lens(
        _ptr(survival), R, D, survival.stride(0), int(budget), int(min_len), int(max_len), float(eps), _ptr(out),
        _ptr(ws), ws.numel(), _stream(stream)))
    return out


def build_tree(parents, seq_lens=None, stream=None, out: Optional[dict] = None) -> dict:
    """Positions, ancestor mask, retrieve index and child / sibling links from parents [B, N] (int32, device).

    out: optional preallocated results with the keys and shapes this function returns."""
    lib = load_library()
    _require_cuda(parents, "parents")
    B, N = parents.shape
    d = parents.device
    _arg(parents, "parents", torch.int32, B * N, d)
    _arg(seq_lens, "seq_lens", torch.int64, B, d)
    res = out if out is not None else {
        "positions": torch.empty(B, N, dtype=torch.int64, device=d),
        "mask": torch.empty(B, N, N, dtype=torch.uint8, device=d),
        "retrieve_index": torch.empty(B, N, dtype=torch.int32, device=d),
        "first_child": torch.empty(B, N, dtype=torch.int32, device=d),
        "next_sibling": torch.empty(B, N, dtype=torch.int32, device=d),
        "status": torch.empty(B, dtype=torch.int32, device=d)}
    for k, dt, n in (("positions", torch.int64, B * N), ("mask", torch.uint8, B * N * N),
                     ("retrieve_index", torch.int32, B * N), ("first_child", torch.int32, B * N),
                     ("next_sibling", torch.int32, B * N), ("status", torch.int32, B)):
        if res.get(k) is None:
            raise ValueError("build_tree: out lacks %r" % k)
        _arg(res[k], "out[%r]" % k, dt, n, d)
    _check("spec_verify_build_tree", lib.spec_verify_build_tree(
        _ptr(parents), _ptr(seq_lens), B, N, _ptr(res["positions"]), _ptr(res["mask"]), _ptr(res["retrieve_index"]),
        _ptr(res["first_child"]), _ptr(res["next_sibling"]), _ptr(res["status"]), _stream(stream)))
    return res


# Serving-side operators around the verification: attention over the paged KV
# cache, the KV move of the commit lists, and token log probabilities.


class _NoStream:
    """The current stream: nothing to enter."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_CURRENT = _NoStream()


def _on(stream):
    """Context for the tensors a call allocates: they belong to the stream the call runs on."""
    return _CURRENT if stream is None else torch.cuda.stream(stream)


class _OtherDevice:
    """The call's device, where it is not the current one."""

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        self.was = torch.cuda.current_device()
        torch.cuda.set_device(self.index)

    def __exit__(self, *exc):
        torch.cuda.set_device(self.was)
        return False


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run_on(index, fn, *args):
    """The library's call, on its tensors' device."""
    # (nearly always the current one: a context entered for nothing costs a small call a tenth of its time)
    if index < 0 or _current_device() == index:
        return fn(*args)
    with _OtherDevice(index):
        return fn(*args)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call_stream(stream, device) -> int:
    """The handle of the given stream, or of the device's current one."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)  # the same handle without a stream object around it
    return torch.cuda.current_stream(device).cuda_stream


def _need(t, name: str, dtype, numel: int, device, index: int):
    """_arg for tensors that are used often: the checks in their cheap forms, the full ones only to say what is wrong."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.numel() >= numel
            and t.is_contiguous()):
        return
    _arg(t, name, dtype, numel, device)


def _need_all(args, dtype, device, index: int):
    """_need for (tensor or None, name, numel) arguments of one type."""
    for t, name, numel in args:
        if t is not None and not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index
                                  and t.numel() >= numel and t.is_contiguous()):
            _arg(t, name, dtype, numel, device)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _row_step(t: torch.Tensor) -> int:
    """Row stride of [rows, cols]; of a single row, its own length up to whole 16-byte pieces."""
    if t.shape[0] > 1:
        return t.stride(0)
    per = 16 // t.element_size()
    return -(-t.shape[1] // per) * per


class PagedKvCache:
    """A paged KV cache: k, v [layers, pages, page_size, heads, head_dim] (bf16 or fp32, head_dim dense, any other
    strides, the same for both) and page_table [batch, max_pages] int32 (dense rows).

    Holds the tensors and the library's description of them; make it once and use it for every call."""

    packed = False

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor):
        for t, name in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor) or t.dim() != 5:
                raise ValueError("%s must be a 5-D torch tensor [layers, pages, page_size, heads, head_dim]" % name)
            if t.shape[4] > 1 and t.stride(4) != 1:
                raise ValueError("%s: head_dim must be dense" % name)
        if k.dtype not in (torch.bfloat16, torch.float32) or v.dtype != k.dtype:
            raise TypeError("k and v must both be bfloat16 or float32, got %s and %s" % (k.dtype, v.dtype))
        if v.shape != k.shape or v.stride() != k.stride() or v.device != k.device:
            raise ValueError("k and v must have the same shape, strides and device")
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be a 2-D torch tensor")
        batch, pages = page_table.shape
        _rows_arg(page_table, "page_table", torch.int32, batch, pages, k.device)
        self.k, self.v, self.page_table = k, v, page_table
        self.device, self.dtype, self.batch, self.index = k.device, k.dtype, batch, k.get_device()
        self.layers, self.heads, self.head_dim = k.shape[0], k.shape[3], k.shape[4]
        st = [x if n > 1 else 0 for x, n in zip(k.stride(), k.shape)]  # an axis of one entry has no step
        self.struct = SvKvCache(k.data_ptr(), v.data_ptr(), SV_BF16 if k.dtype == torch.bfloat16 else SV_F32,
                                k.shape[0], k.shape[1], k.shape[2], k.shape[3], k.shape[4], st[0], st[1], st[2], st[3],
                                page_table.data_ptr(), pages, page_table.stride(0) if batch > 1 else max(pages, 1))
        self.ref = ctypes.byref(self.struct)


class PackedKvCache:
    """A paged KV cache held in 4 bits: data [layers, pages, heads, block bytes] uint8 (the last axis dense, other strides
    multiples of 16) and page_table [batch, max_pages] int32 (dense rows).

    A block holds a page's entries of one head: block_bytes(page_size, head_dim) bytes of it are used.  head_dim is a multiple
    of 32.  dtype (bf16 or fp32) is that of the rows that go with the cache: keys and values that kv_append takes and kv_read
    gives back.  paged_attention takes bf16: a cache of fp32 rows cannot be attended to.  Pages of 16, 32, 64 or a multiple of 128
    entries are the fast ones for attention (those that neither divide 128 nor are a multiple of it are gathered row by row).  Stands
    wherever a PagedKvCache does; make it once and use it for every call."""

    packed = True

    def __init__(self, data: torch.Tensor, page_table: torch.Tensor, *, page_size: int, head_dim: int,
                 dtype: torch.dtype = torch.bfloat16):
        if not isinstance(data, torch.Tensor) or data.dim() != 4:
            raise ValueError("data must be a 4-D torch tensor [layers, pages, heads, block bytes]")
        if data.dtype != torch.uint8:
            raise TypeError("data must be torch.uint8, got %s" % data.dtype)
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("dtype must be bfloat16 or float32, got %s" % dtype)
        need = PackedKvCache.block_bytes(page_size, head_dim)
        if data.shape[3] < need or data.stride(3) != 1:
            raise ValueError("data's blocks must be dense and hold %d bytes (got %d)" % (need, data.shape[3]))
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be a 2-D torch tensor")
        batch, pages = page_table.shape
        _rows_arg(page_table, "page_table", torch.int32, batch, pages, data.device)
        self.data, self.page_table = data, page_table
        self.device, self.dtype, self.batch, self.index = data.device, dtype, batch, data.get_device()
        self.layers, self.heads, self.head_dim, self.page_size = data.shape[0], data.shape[2], head_dim, page_size
        st = [x if n > 1 else 0 for x, n in zip(data.stride(), data.shape)]  # an axis of one entry has no step
        self.struct = SvPackedKvCache(data.data_ptr(), SV_BF16 if dtype == torch.bfloat16 else SV_F32, data.shape[0],
                                      data.shape[1], page_size, data.shape[2], head_dim, st[0], st[1], st[2],
                                      page_table.data_ptr(), pages, page_table.stride(0) if batch > 1 else max(pages, 1))
        self.ref = ctypes.byref(self.struct)

    @staticmethod
    def block_bytes(page_size: int, head_dim: int) -> int:
        """Bytes of a page's entries of one head, K and V."""
        n = int(load_library().spec_verify_packed_kv_block_bytes(page_size, head_dim))
        if n == 0:
            raise ValueError("no 4-bit cache of page_size %d and head_dim %d (a multiple of 32, at most 256)"
                             % (page_size, head_dim))
        return n

    @staticmethod
    def allocate(layers: int, pages: int, heads: int, page_size: int, head_dim: int, page_table: torch.Tensor,
                 dtype: torch.dtype = torch.bfloat16) -> "PackedKvCache":
        """A cache of zeros on page_table's device."""
        data = torch.zeros(layers, pages, heads, PackedKvCache.block_bytes(page_size, head_dim), dtype=torch.uint8,
                           device=page_table.device)
        return PackedKvCache(data, page_table, page_size=page_size, head_dim=head_dim, dtype=dtype)


def _require_cache(cache):
    if type(cache) is not PagedKvCache and not isinstance(cache, (PagedKvCache, PackedKvCache)):
        raise TypeError("cache must be a PagedKvCache or a PackedKvCache")
    if cache.index < 0:
        raise ValueError("the cache must be on a CUDA device (got %s): the library has no CPU path" % cache.device)


@dataclass
class AttentionOutputs:
    out: torch.Tensor              # [rows, heads, head_dim], the cache's type
    lse: Optional[torch.Tensor]    # [rows, heads] fp32
    dev_status: torch.Tensor       # [batch] int32 storage of uint32 bits

    @staticmethod
    def allocate(rows: int, heads: int, head_dim: int, batch: int, dtype=torch.bfloat16, device=None,
                 lse: bool = True) -> "AttentionOutputs":
        d = device or "cuda"
        return AttentionOutputs(out=torch.empty(rows, heads, head_dim, dtype=dtype, device=d),
                                lse=torch.empty(rows, heads, dtype=torch.float32, device=d) if lse else None,
                                dev_status=torch.empty(batch, dtype=torch.int32, device=d))


def attention_workspace(batch: int, max_len: int, cache, num_heads: int) -> torch.Tensor:
    """A zero-filled workspace of paged_attention calls (the library keeps its counters zero between calls)."""
    n = int(load_library().spec_verify_attention_workspace_bytes(batch, max_len, num_heads, cache.heads,
                                                                 cache.head_dim))
    return torch.zeros(n, dtype=torch.uint8, device=cache.device)


def _head_rows(t, name, rows, heads, dim, dtype, device, index):
    """Checks t [>= rows, heads, dim]; returns its row and head strides (an axis of one entry has no step)."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.dim() == 3:
        n, h, d = t.shape
        a, b, c = t.stride()
        if n >= rows and h == heads and d == dim and (c == 1 or d == 1):
            return (a if n > 1 else 0), (b if h > 1 else 0)
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError("%s must be a 3-D torch tensor [rows, heads, head_dim]" % name)
    if t.device != device:
        raise ValueError("%s is on %s; the call runs on %s (the cache's device)" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s (the cache's type), got %s" % (name, dtype, t.dtype))
    if t.shape[0] < rows or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError("%s is %s; the call needs [%d, %d, %d]" % (name, tuple(t.shape), rows, heads, dim))
    if dim > 1 and t.stride(2) != 1:
        raise ValueError("%s: head_dim must be dense" % name)


def paged_attention(q, cache, seq_lens, *, layer: int = 0, max_len: Optional[int] = None,
                    cu_seqlens=None, row_slots=None, mask=None, scale: Optional[float] = None, out=None, ws=None,
                    stream=None) -> AttentionOutputs:
    """Attention of each request's new rows q [rows, heads, head_dim] over its committed positions in the cache and
    over the new rows themselves.

    seq_lens [batch] int64: committed positions, without the new rows.  A request has max_len new rows (rows / batch, a
    whole number, when not given; 1 is plain decoding), or cu_seqlens [batch + 1] int32 gives ragged ones of 1..max_len.
    row_slots [rows] int64: where the new rows' K/V lie (None: at positions seq_lens + j).  mask [batch, max_len,
    max_len] uint8: which new rows a row sees (None: itself and earlier ones), as build_tree returns it.
    cache: a PagedKvCache, or a PackedKvCache with bf16 rows.  scale defaults to 1 / sqrt(head_dim)."""
    lib = load_library()
    _require_cache(cache)
    dev, index = cache.device, cache.index
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a 3-D torch tensor [rows, heads, head_dim]")
    rows, heads, dim = q.shape
    q_steps = _head_rows(q, "q", rows, heads, cache.head_dim, cache.dtype, dev, index)
    if seq_lens is None:
        raise ValueError("seq_lens is required")
    _need(seq_lens, "seq_lens", torch.int64, 0, dev, index)
    batch = seq_lens.numel()
    if cache.batch < batch:
        raise ValueError("page_table has %d rows; the call reads %d" % (cache.batch, batch))
    if max_len is None:
        if cu_seqlens is not None:
            raise ValueError("max_len is required with cu_seqlens")
        if batch and (rows % batch or not rows):
            raise ValueError("q's %d rows do not divide among %d requests: max_len is required" % (rows, batch))
        max_len = rows // batch if batch else 1
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, batch + 1, dev, index)
    elif rows < batch * max_len:
        raise ValueError("q has %d rows; the call reads %d" % (rows, batch * max_len))
    if row_slots is not None:
        _need(row_slots, "row_slots", torch.int64, rows, dev, index)
    if mask is not None:
        _need(mask, "mask", torch.uint8, batch * max_len * max_len, dev, index)
    if out is None or ws is None:
        with _on(stream):
            if out is None:
                out = AttentionOutputs.allocate(rows, heads, dim, batch, cache.dtype, dev)
            if ws is None:
                ws = attention_workspace(batch, max_len, cache, heads)
    o, lse, status = out.out, out.lse, out.dev_status
    o_steps = _head_rows(o, "out.out", rows, heads, dim, cache.dtype, dev, index)
    if lse is not None:
        _need(lse, "out.lse", torch.float32, rows * heads, dev, index)
    if status is not None:
        _need(status, "out.dev_status", torch.int32, batch, dev, index)
    _need(ws, "ws", torch.uint8, 0, dev, index)
    fn = lib.spec_verify_packed_attention if cache.packed else lib.spec_verify_paged_attention
    code = _run_on(
        index, fn, q.data_ptr(), q_steps[0], q_steps[1], heads, cache.ref, layer, batch, rows, max_len, _addr(cu_seqlens),
        seq_lens.data_ptr(), _addr(row_slots), _addr(mask), dim ** -0.5 if scale is None else scale,
        o.data_ptr(), o_steps[0], o_steps[1], _addr(lse), _addr(status), ws.data_ptr(), ws.numel(),
        _call_stream(stream, dev))
    if code:
        _check("spec_verify_packed_attention" if cache.packed else "spec_verify_paged_attention", code)
    return out


def kv_commit(cache, commit_cu, commit_src_slot, commit_dst_pos, *, max_len: int, dev_status=None,
              stream=None) -> torch.Tensor:
    """Moves the committed rows' K/V to their positions, in every layer, from a verification's commit lists
    (VerifyOutputs.commit_cu / commit_src_slot / commit_dst_pos).  Returns the requests' status bits [batch].

    Every entry of the cache needs memory of its own: expanded axes, and k and v in the same memory, are refused."""
    lib = load_library()
    _require_cache(cache)
    dev, index = cache.device, cache.index
    if commit_cu is None or commit_src_slot is None or commit_dst_pos is None:
        raise ValueError("commit_cu, commit_src_slot and commit_dst_pos are required")
    _need(commit_cu, "commit_cu", torch.int32, 1, dev, index)
    batch = commit_cu.numel() - 1
    if cache.batch < batch:
        raise ValueError("page_table has %d rows; the call reads %d" % (cache.batch, batch))
    _need(commit_src_slot, "commit_src_slot", torch.int64, 0, dev, index)
    _need(commit_dst_pos, "commit_dst_pos", torch.int64, 0, dev, index)
    if dev_status is None:
        with _on(stream):
            dev_status = torch.empty(batch, dtype=torch.int32, device=dev)
    _need(dev_status, "dev_status", torch.int32, batch, dev, index)
    fn = lib.spec_verify_packed_kv_commit if cache.packed else lib.spec_verify_kv_commit
    code = _run_on(
        index, fn, cache.ref, batch, max_len, min(commit_src_slot.numel(), commit_dst_pos.numel()), commit_cu.data_ptr(),
        commit_src_slot.data_ptr(), commit_dst_pos.data_ptr(), dev_status.data_ptr(), _call_stream(stream, dev))
    if code:
        _check("spec_verify_packed_kv_commit" if cache.packed else "spec_verify_kv_commit", code)
    return dev_status


class Rotation:
    """A rotation by position: pair i of a head's columns turns by position * inv_freq[i] (fp32, on the cache's device).

    A pair is columns (i, i + pairs), or (2 i, 2 i + 1) when interleaved; the rotated columns are multiplied by magnitude, and
    columns from 2 * pairs on are left as they are.  Make it once and use it for every call."""

    def __init__(self, inv_freq: torch.Tensor, *, interleaved: bool = False, magnitude: float = 1.0):
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be a 1-D torch tensor")
        _arg(inv_freq, "inv_freq", torch.float32, 0, inv_freq.device)
        self.inv_freq, self.pairs, self.interleaved, self.magnitude = inv_freq, inv_freq.numel(), interleaved, magnitude
        self.index = inv_freq.get_device()
        self.struct = SvRotation(inv_freq.data_ptr(), self.pairs, 1 if interleaved else 0, magnitude)
        self.ref = ctypes.byref(self.struct)


def _cache_rows(cache, rows, seq_lens, max_len, cu_seqlens, row_slots, positions=None):
    """The rows of a call on a cache: checks their arrays; returns the batch, the rows and the library's description.  rows None:
    as many as the requests have."""
    dev, index = cache.device, cache.index
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, 1, dev, index)
        batch = cu_seqlens.numel() - 1
        if max_len is None:
            raise ValueError("max_len is required with cu_seqlens")
        if rows is None:
            raise ValueError("rows is required with cu_seqlens")
    elif seq_lens is not None:
        _need(seq_lens, "seq_lens", torch.int64, 0, dev, index)
        batch = seq_lens.numel()
        if max_len is None:
            if rows is None:
                raise ValueError("max_len is required")
            if batch and (rows % batch or not rows):
                raise ValueError("%d rows do not divide among %d requests: max_len is required" % (rows, batch))
            max_len = rows // batch if batch else 1
        if rows is None:
            rows = batch * max_len
        elif rows < batch * max_len:
            raise ValueError("there are %d rows; the call reads %d" % (rows, batch * max_len))
    else:
        if rows is None:
            raise ValueError("seq_lens or cu_seqlens is required")
        max_len = 1 if max_len is None else max_len
        if max_len < 1 or rows % max_len:
            raise ValueError("%d rows are no whole number of requests of %d" % (rows, max_len))
        batch = rows // max_len
    _need_all(((seq_lens, "seq_lens", batch), (row_slots, "row_slots", rows), (positions, "positions", rows)), torch.int64, dev,
              index)
    if row_slots is None:
        if seq_lens is None:
            raise ValueError("seq_lens is required without row_slots")
        if cache.batch < batch:
            raise ValueError("page_table has %d rows; the call reads %d" % (cache.batch, batch))
    return batch, rows, SvRows(batch, max_len, rows, None if cu_seqlens is None else cu_seqlens.data_ptr(),
                               None if seq_lens is None else seq_lens.data_ptr(),
                               None if row_slots is None else row_slots.data_ptr())


@dataclass
class KvAppendOutputs:
    q: Optional[torch.Tensor]   # [rows, heads, head_dim], the rotated queries
    dev_status: torch.Tensor    # [batch] int32 storage of uint32 bits, OR-ed into

    @staticmethod
    def allocate(rows: int, heads: int, head_dim: int, batch: int, dtype=torch.bfloat16, device=None) -> "KvAppendOutputs":
        d = device or "cuda"
        return KvAppendOutputs(q=torch.empty(rows, heads, head_dim, dtype=dtype, device=d) if heads else None,
                               dev_status=torch.zeros(batch, dtype=torch.int32, device=d))


def kv_append(cache, k, v, *, layer: int = 0, seq_lens=None, max_len: Optional[int] = None, cu_seqlens=None, row_slots=None,
              positions=None, rotation: Optional[Rotation] = None, q=None, out=None, stream=None) -> KvAppendOutputs:
    """Puts new rows k, v [rows, heads, head_dim] of a layer into the cache, the keys rotated by position, and rotates their
    queries q [rows, query heads, head_dim].

    A request has max_len rows (rows / batch when not given), or cu_seqlens [batch + 1] int32 gives ragged ones of 0..max_len;
    rows behind the last request are left alone.  Row j of request b goes to position seq_lens[b] + j, or to slot row_slots
    [rows] int64; it is rotated by positions [rows] int64, or by seq_lens[b] + j.  Two rows must not have the same place.
    out: KvAppendOutputs; its q may be q itself.  dev_status is OR-ed into: it collects what many calls report until it is
    zeroed.  cache: a PagedKvCache or a PackedKvCache (which takes the rotated values rounded once, to 4 bits)."""
    lib = load_library()
    _require_cache(cache)
    dev, index = cache.device, cache.index
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a 3-D torch tensor [rows, heads, head_dim]")
    rows, dim = k.shape[0], cache.head_dim
    ks = _head_rows(k, "k", rows, cache.heads, dim, cache.dtype, dev, index)
    vs = _head_rows(v, "v", rows, cache.heads, dim, cache.dtype, dev, index)
    batch, _, desc = _cache_rows(cache, rows, seq_lens, max_len, cu_seqlens, row_slots, positions)
    if positions is None and rotation is not None and seq_lens is None:
        raise ValueError("positions are required without seq_lens")
    heads, qs, os = 0, (0, 0), (0, 0)
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be a 3-D torch tensor [rows, heads, head_dim]")
        heads = q.shape[1]
        qs = _head_rows(q, "q", rows, heads, dim, cache.dtype, dev, index)
    if rotation is not None:
        if not isinstance(rotation, Rotation):
            raise TypeError("rotation must be a Rotation")
        if rotation.index != index:
            raise ValueError("rotation is on %s; the call runs on %s (the cache's device)" % (rotation.inv_freq.device, dev))
    if out is None:
        with _on(stream):
            out = KvAppendOutputs.allocate(rows, heads, dim, batch, cache.dtype, dev)
    if q is not None:
        if out.q is None:
            raise ValueError("out.q is required with q")
        os = _head_rows(out.q, "out.q", rows, heads, dim, cache.dtype, dev, index)
    _need(out.dev_status, "out.dev_status", torch.int32, batch, dev, index)
    fn = lib.spec_verify_packed_kv_append if cache.packed else lib.spec_verify_kv_append
    code = _run_on(
        index, fn, cache.ref, layer, ctypes.byref(desc), _addr(positions), None if rotation is None else rotation.ref,
        k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], _addr(q), qs[0], qs[1], heads,
        None if q is None else out.q.data_ptr(), os[0], os[1], out.dev_status.data_ptr(), _call_stream(stream, dev))
    if code:
        _check("spec_verify_packed_kv_append" if cache.packed else "spec_verify_kv_append", code)
    return out


@dataclass
class KvReadOutputs:
    k: torch.Tensor             # [rows, heads, head_dim], or [layers, rows, heads, head_dim]
    v: torch.Tensor
    dev_status: torch.Tensor    # [batch] int32 storage of uint32 bits, OR-ed into

    @staticmethod
    def allocate(rows: int, heads: int, head_dim: int, batch: int, dtype=torch.bfloat16, device=None,
                 layers: Optional[int] = None) -> "KvReadOutputs":
        d = device or "cuda"
        shape = (rows, heads, head_dim) if layers is None else (layers, rows, heads, head_dim)
        return KvReadOutputs(k=torch.empty(shape, dtype=dtype, device=d), v=torch.empty(shape, dtype=dtype, device=d),
                             dev_status=torch.zeros(batch, dtype=torch.int32, device=d))


def _layer_rows(t, name, layers, rows, cache):
    """Checks t [layers, >= rows, heads, dim] of a cache; returns its layer, row and head strides."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4 or t.shape[0] != layers or layers < 1:
        raise ValueError("%s must be [%d layers, rows, heads, head_dim]" % (name, layers))
    _, n, h, d = t.shape
    a, b, c, e = t.stride()
    if not (t.dtype is cache.dtype and t.get_device() == cache.index and n >= rows and h == cache.heads and d == cache.head_dim
            and (e == 1 or d == 1)):
        _head_rows(t[0], name, rows, cache.heads, cache.head_dim, cache.dtype, cache.device, cache.index)
    return (a if layers > 1 else 0), (b if n > 1 else 0), (c if h > 1 else 0)


def kv_read(cache, *, layer: Optional[int] = None, seq_lens=None, max_len: Optional[int] = None, cu_seqlens=None,
            row_slots=None, rows: Optional[int] = None, out=None, stream=None) -> KvReadOutputs:
    """The cache's entries of the given rows' places (as kv_append places rows) as dense rows of the cache's dtype: of one
    layer k, v [rows, heads, head_dim], or, without layer, of every layer [layers, rows, heads, head_dim].

    rows: how many there are (needed with cu_seqlens where neither out nor row_slots tells).  A request's whole history is
    seq_lens of zeros and its lengths in cu_seqlens.  A row whose place lies outside the cache is 0; rows of no request are
    left as they are in out.  dev_status is OR-ed into."""
    lib = load_library()
    _require_cache(cache)
    dev, index = cache.device, cache.index
    if rows is None:
        if out is not None and isinstance(out.k, torch.Tensor):
            rows = out.k.shape[-3]
        elif row_slots is not None and isinstance(row_slots, torch.Tensor):
            rows = row_slots.numel()
    batch, rows, desc = _cache_rows(cache, rows, seq_lens, max_len, cu_seqlens, row_slots)
    layers = cache.layers if layer is None else 1
    if out is None:
        with _on(stream):
            out = KvReadOutputs.allocate(rows, cache.heads, cache.head_dim, batch, cache.dtype, dev,
                                         layers if layer is None else None)
    if layer is None:
        st = _layer_rows(out.k, "out.k", layers, rows, cache)
        same = _layer_rows(out.v, "out.v", layers, rows, cache) == st
    else:
        st = (0,) + _head_rows(out.k, "out.k", rows, cache.heads, cache.head_dim, cache.dtype, dev, index)
        same = (0,) + _head_rows(out.v, "out.v", rows, cache.heads, cache.head_dim, cache.dtype, dev, index) == st
    if not same:
        raise ValueError("out.k and out.v must have the same strides")
    _need(out.dev_status, "out.dev_status", torch.int32, batch, dev, index)
    fn = lib.spec_verify_packed_kv_read if cache.packed else lib.spec_verify_kv_read
    code = _run_on(
        index, fn, cache.ref, 0 if layer is None else layer, layers, ctypes.byref(desc), out.k.data_ptr(), out.v.data_ptr(),
        st[0], st[1], st[2], out.dev_status.data_ptr(), _call_stream(stream, dev))
    if code:
        _check("spec_verify_packed_kv_read" if cache.packed else "spec_verify_kv_read", code)
    return out


@dataclass
class LogprobOutputs:
    logprob: Optional[torch.Tensor]      # [n, num_ids] fp32
    entropy: Optional[torch.Tensor]      # [n] fp32
    row_max: Optional[torch.Tensor]      # [n] fp32, the rows' largest logits
    log_z: Optional[torch.Tensor]        # [n] fp32, ln sum exp((l - row_max) / T)
    top_ids: Optional[torch.Tensor]      # [n, top_k] int32
    top_logprob: Optional[torch.Tensor]  # [n, top_k] fp32
    flags: Optional[torch.Tensor]        # [n] int32 storage of uint32 bits

    @staticmethod
    def allocate(n: int, num_ids: int, top_k: int = 0, device=None) -> "LogprobOutputs":
        f32 = dict(dtype=torch.float32, device=device or "cuda")
        i32 = dict(dtype=torch.int32, device=device or "cuda")
        return LogprobOutputs(logprob=torch.empty(n, num_ids, **f32), entropy=torch.empty(n, **f32),
                              row_max=torch.empty(n, **f32), log_z=torch.empty(n, **f32),
                              top_ids=torch.empty(n, top_k, **i32) if top_k else None,
                              top_logprob=torch.empty(n, top_k, **f32) if top_k else None,
                              flags=torch.empty(n, **i32))


def logprobs_workspace(n: int, vocab: int, top_k: int = 0, device=None) -> torch.Tensor:
    """A zero-filled workspace of token_logprobs calls (the library keeps its counters zero between calls)."""
    b = int(load_library().spec_verify_logprobs_workspace_bytes(n, vocab, top_k))
    return torch.zeros(b, dtype=torch.uint8, device=device or "cuda")


def _given_ids(ids, n, device, index):
    """ids as [n, num_ids] with dense rows (a 1-D array is one id a row): the tensor, num_ids and the row stride."""
    if not isinstance(ids, torch.Tensor) or ids.dim() not in (1, 2):
        raise ValueError("ids must be a 1-D or 2-D torch tensor")
    if ids.dim() == 1:
        ids = ids.unsqueeze(1)
    m, num = ids.shape
    a, b = ids.stride()
    if not (m >= n and (b == 1 or num <= 1) and ids.dtype is torch.int32 and ids.get_device() == index):
        _rows_arg(ids, "ids", torch.int32, n, 0, device)
    return ids, num, (a if n > 1 else num or 1)


def token_logprobs(logits, ids, *, top_k: int = 0, row_index=None, row_temp=None, out=None, ws=None,
                   stream=None) -> LogprobOutputs:
    """Log probabilities of the given tokens ids [n, num_ids] (or [n]) under softmax(logits / T), with each row's
    entropy and its top_k most likely tokens.

    Output i describes logits row row_index[i] (int32, -1 is padding; None: row i), so that a verification's
    accept_rows and out_tokens can be passed as they are.  row_temp [n] fp32 (None: 1)."""
    lib = load_library()
    _require_cuda(logits)
    rows, V = logits.shape
    dev, index = logits.device, logits.get_device()
    if row_index is None:
        n = rows
    else:
        _need(row_index, "row_index", torch.int32, 0, dev, index)
        n = row_index.numel()
    ids, num_ids, ldi = _given_ids(ids, n, dev, index)
    f32, i32 = torch.float32, torch.int32
    if out is None or ws is None:
        with _on(stream):
            if out is None:
                out = LogprobOutputs.allocate(n, num_ids, top_k, dev)
            if ws is None:
                ws = logprobs_workspace(n, V, top_k, dev)
    res = (out.logprob, out.entropy, out.row_max, out.log_z, out.top_ids, out.top_logprob, out.flags)
    _need_all(((row_temp, "row_temp", n), (res[0], "out.logprob", n * num_ids), (res[1], "out.entropy", n),
               (res[2], "out.row_max", n), (res[3], "out.log_z", n), (res[5], "out.top_logprob", n * top_k)),
              f32, dev, index)
    _need_all(((res[4], "out.top_ids", n * top_k), (res[6], "out.flags", n)), i32, dev, index)
    _need(ws, "ws", torch.uint8, 0, dev, index)
    code = lib.spec_verify_token_logprobs(
        logits.data_ptr(), _dtype(logits), _row_step(logits), rows, V, n, _addr(row_index), ids.data_ptr(), num_ids,
        ldi, _addr(row_temp), top_k, *[None if t is None else t.data_ptr() for t in res], ws.data_ptr(), ws.numel(),
        _call_stream(stream, dev))
    if code:
        _check("spec_verify_token_logprobs", code)
    return out


def token_logprobs_backward(logits, ids, kept: LogprobOutputs, g_logprob, *, g_entropy=None, g_top=None, row_temp=None,
                            out=None, stream=None) -> torch.Tensor:
    """The gradient by logits [rows, V] of token_logprobs (called without row_index), given the gradients of its
    logprob [rows, num_ids], entropy [rows] and top_logprob [rows, top_k].

    kept: the forward call's outputs (row_max and log_z; entropy with g_entropy; top_ids with g_top).  out: a tensor
    like logits (rows of a multiple of 16 bytes) that does not overlap them."""
    lib = load_library()
    _require_cuda(logits)
    rows, V = logits.shape
    dev, index, f32 = logits.device, logits.get_device(), torch.float32
    ids, num_ids, ldi = _given_ids(ids, rows, dev, index)
    top_ids, top_k = None, 0
    if g_top is not None:
        if not isinstance(g_top, torch.Tensor) or g_top.dim() != 2:
            raise ValueError("g_top must be a 2-D torch tensor")
        top_ids, top_k = kept.top_ids, g_top.shape[1]
        _need(g_top, "g_top", f32, rows * top_k, dev, index)
        if top_ids is not None:
            _need(top_ids, "kept.top_ids", torch.int32, rows * top_k, dev, index)
            if top_ids.dim() != 2 or top_ids.shape[1] != top_k:
                raise ValueError("kept.top_ids must have g_top's %d columns" % top_k)
    row_max, log_z, entropy = kept.row_max, kept.log_z, kept.entropy
    _need_all(((g_logprob, "g_logprob", rows * num_ids), (g_entropy, "g_entropy", rows), (row_temp, "row_temp", rows),
               (row_max, "kept.row_max", rows), (log_z, "kept.log_z", rows), (entropy, "kept.entropy", rows)),
              f32, dev, index)
    if out is None:
        per = 16 // logits.element_size()
        with _on(stream):
            out = torch.empty(rows, -(-V // per) * per, dtype=logits.dtype, device=dev)[:, :V]
    if not (isinstance(out, torch.Tensor) and out.shape == logits.shape and out.dtype is logits.dtype
            and out.get_device() == index and (out.stride(1) == 1 or V == 1)):
        _rows_arg(out, "out", logits.dtype, rows, V, dev)
    row_temp, row_max, log_z, entropy, top_ids, g_logprob, g_entropy, g_top = [
        None if t is None else t.data_ptr()
        for t in (row_temp, row_max, log_z, entropy, top_ids, g_logprob, g_entropy, g_top)]
    code = lib.spec_verify_token_logprobs_backward(
        logits.data_ptr(), _dtype(logits), _row_step(logits), rows, V, ids.data_ptr(), num_ids, ldi, row_temp,
        row_max, log_z, entropy, top_ids, top_k, g_logprob, g_entropy, g_top, out.data_ptr(), _row_step(out),
        _call_stream(stream, dev))
    if code:
        _check("spec_verify_token_logprobs_backward", code)
    return out
