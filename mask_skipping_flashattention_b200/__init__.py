"""Mask-aware fused attention forward for NVIDIA B200 (sm_100a).

Thin Python binding over the C ABI of ``libbfa.so`` (``include/bfa.h``).  The
binding only marshals torch tensors into device pointers, sizes, strides and the
current CUDA stream; every step of the computation runs in the library's CUDA
kernels.  There is no CPU path: CPU tensors are rejected by the library.

    plan = plan_dense(mask)                      # (Sq, Sk) bool, True = attend
    out, lse = fwd(plan, q, k, v)                # q (B, Sq, H, D), k/v (B, Sk, Hkv, D)

Other mask sources: ``plan_blockids`` (opentau block ids, positions, varlen,
sliding window) and ``plan_bsr`` (BSR routing); ``make_att_block_ids`` builds
block ids from padding and block-opening flags.

``fwd`` and ``bwd`` also take shaped scores (``softcap``, ``slopes``).  Beside the
planned forms, ``fwd_chunk`` attends the newest tokens of each sequence over a
paged cache (decoding included), ``append_paged`` fills that cache, and ``rope``
(frequencies from ``rope_frequencies``) turns queries and keys by their positions.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import math

import numpy as np
import torch

from . import _lib
from ._lib import BfaError, PlanInfo

__all__ = ["Plan", "BfaError", "plan_dense", "plan_blockids", "plan_predicate", "plan_bsr", "plan_bsr_packed",
           "plan_block_bits",
           "fwd", "bwd", "fwd_paged",
           "fwd_chunk", "chunk_device_status", "append_paged", "rope", "rope_frequencies",
           "make_att_block_ids",
           "is_available", "load_error", "set_wait_timeout_ns", "set_bwd_deterministic", "selftest_wait_timeout", "library_path"]

TILE = 128
KIND_NAMES = {1: "dense", 2: "blockids", 3: "positional", 4: "bsr", 5: "predicate"}
_I32_MIN, _I32_MAX = -(2 ** 31), 2 ** 31 - 1

library_path = _lib.LIB_PATH
_L = _lib.load()


def _stream(stream=None):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


@contextlib.contextmanager
def _launch_on(t, stream):
    """The device of ``t`` and ``stream`` as the current ones, so that what is allocated inside
    belongs to the stream that uses it; yields (stream handle, finish).  ``finish`` hands such
    results back to the stream that was current."""
    with torch.cuda.device(t.device):
        ambient = torch.cuda.current_stream()
        if stream is None:
            yield ambient.cuda_stream, _keep
            return
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), t.device) if int(stream) else torch.cuda.default_stream()
        if stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")

        def finish(*results):
            for r in results:
                if r is not None and ambient != stream:
                    r.record_stream(ambient)

        with torch.cuda.stream(stream):
            yield stream.cuda_stream, finish


def _keep(*results):
    pass


def _run_on(t, stream, body):
    """body(stream handle, finish) with the device of ``t`` and ``stream`` current (see
    ``_launch_on``), without a context change where they already are: that costs more than
    a small launch.  CPU tensors are left to the library's refusal."""
    if not t.is_cuda:
        return body(0 if stream is None else _stream(stream), _keep)
    index = t.get_device()
    if stream is None and index == torch._C._cuda_getDevice():
        return body(torch._C._cuda_getCurrentRawStream(index), _keep)
    with _launch_on(t, stream) as (st, finish):
        return body(st, finish)


def _same_device(first, *others):
    want = first.get_device()  # -1: CPU
    for t in others:
        if t is not None and t.get_device() != want:
            raise ValueError(f"tensors on {first.device} and {t.device}")


def _addr(t):
    return None if t is None else t.data_ptr()


_Strides3 = ctypes.c_int64 * 3


@functools.lru_cache(maxsize=4096)
def _strides3_of(st):
    return _Strides3(st[0], st[1], st[2]) if len(st) == 4 else _Strides3(0, st[0], st[1])


def _strides_of(t):
    """{batch, token, head} strides of a (B, S, H, D) or packed (T, H, D) tensor (read-only)."""
    return _strides3_of(t.stride())


def _score_shape(softcap, slopes, q, H):
    """softcap or 0; slopes checked."""
    if slopes is not None:
        if slopes.dtype is not torch.float32:
            raise TypeError("slopes must be float32")
        if slopes.shape != (H,):
            raise ValueError(f"slopes must have one value per query head ({H}), not shape {tuple(slopes.shape)}")
        _same_device(q, slopes)
    return float(softcap) if softcap is not None else 0.0


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _u8(t):
    if t is None:
        return None
    if t.dtype == torch.bool:
        return t
    return (t != 0)


def is_available():
    """True if a B200-class device is present and the kernels load."""
    return bool(_L.bfa_is_available())


def load_error():
    """Message of the last failed library call on this thread, or None."""
    m = _L.bfa_last_error().decode(errors="replace")
    return m or None


def set_wait_timeout_ns(ns):
    _L.bfa_set_wait_timeout_ns(int(ns))


def set_bwd_deterministic(on=True):
    """Two-pass backward for every head dim (bitwise reproducible) when ``on``."""
    _L.bfa_set_bwd_deterministic(1 if on else 0)


def selftest_wait_timeout(stream=None):
    """Run the library's bounded-wait self test; returns the status name."""
    return _lib.STATUS.get(_L.bfa_selftest_wait_timeout(_stream(stream)))


class Plan:
    """A library-owned tile plan; freed when garbage collected or by ``destroy()``."""

    def __init__(self, handle, stream):
        self._h = handle
        self._stream = stream
        info = PlanInfo()
        _lib.check(_L.bfa_plan_get_info(self._h, ctypes.byref(info)))
        self.info = {f: getattr(info, f) for f, _ in PlanInfo._fields_}
        self.kind = KIND_NAMES[self.info["kind"]]

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("plan was destroyed")
        return self._h

    def destroy(self):
        if self._h is not None:
            _L.bfa_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    def stats(self, stream=None):
        f, p, e = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _lib.check(_L.bfa_plan_stats(self.handle, ctypes.byref(f), ctypes.byref(p), ctypes.byref(e),
                                     _stream(stream)))
        return f.value, p.value, e.value

    def device_status(self, stream=None):
        """Raise BfaError(BFA_ERR_TIMEOUT) if a kernel using this plan hit its wait bound."""
        _lib.check(_L.bfa_plan_device_status(self.handle, _stream(stream)))

    def export_cols(self, stream=None):
        """Host copy of the transposed lists of the backward's key-tile pass:
        col_ptr, q_tile, tpart (-1 full, else the fine-word index), col_order."""
        n_full, n_part, _ = self.stats(stream)
        C = self.info["n_cols"]
        nnz = n_full + n_part
        col_ptr = np.zeros(C + 1, np.int32)
        q_tile = np.zeros(max(nnz, 1), np.int32)
        tpart = np.zeros(max(nnz, 1), np.int32)
        col_order = np.zeros(max(C, 1), np.int32)
        P = lambda a: a.ctypes.data_as(ctypes.c_void_p)
        _lib.check(_L.bfa_plan_export_cols(self.handle, P(col_ptr), P(q_tile), P(tpart), P(col_order),
                                           _stream(stream)))
        return dict(col_ptr=col_ptr, q_tile=q_tile[:nnz], tpart=tpart[:nnz], col_order=col_order[:C])

    def export(self, stream=None):
        """Host copy: row_ptr, kv_tile, partial, fine (packed-mask plans), order, classes, pairs."""
        n_full, n_part, _ = self.stats(stream)
        R = self.info["n_rows"]
        nnz = n_full + n_part
        row_ptr = np.zeros(R + 1, np.int32)
        kv_tile = np.zeros(max(nnz, 1), np.int32)
        partial = np.zeros(max(nnz, 1), np.uint8)
        fine = np.zeros((max(n_part, 1), TILE, 4), np.uint32) if self.info["packed_fine"] else None
        order = np.zeros(max(R, 1), np.int32)
        classes = np.zeros(max(self.info["grid_tiles"], 1), np.uint8)
        P = lambda a: a.ctypes.data_as(ctypes.c_void_p) if a is not None else None
        _lib.check(_L.bfa_plan_export(self.handle, P(row_ptr), P(kv_tile), P(partial), P(fine), P(order),
                                      P(classes), _stream(stream)))
        out = dict(row_ptr=row_ptr, kv_tile=kv_tile[:nnz], partial=partial[:nnz], order=order[:R],
                   classes=classes[:self.info["grid_tiles"]])
        n_pairs = self.info["n_pairs"]
        pair_row = np.zeros(max(n_pairs, 1), np.int32)
        pair_order = np.zeros(max(n_pairs, 1), np.int32)
        _lib.check(_L.bfa_plan_export_pairs(self.handle, P(pair_row), P(pair_order), _stream(stream)))
        out["pair_row"] = pair_row[:n_pairs]
        out["pair_order"] = pair_order[:n_pairs]
        if fine is not None:
            out["fine"] = fine[:n_part]
        return out


def make_att_block_ids(pad_masks, att_masks, n_cross_att_tokens=None, cross_att_pad_masks=None, stream=None):
    """(q_blk, k_blk, q_valid, k_valid) from padding and block-opening flags (opentau).

    pad_masks / att_masks: (B, N) bool or integer CUDA tensors; cross columns with
    block id INT32_MIN are prepended when ``n_cross_att_tokens`` is given.
    """
    pad = _u8(pad_masks).contiguous()
    att = _u8(att_masks).contiguous()
    B, N = pad.shape
    nc = int(n_cross_att_tokens or 0)
    cpad = _u8(cross_att_pad_masks).contiguous() if nc else None
    dev = pad.device
    q_blk = torch.empty((B, N), dtype=torch.int32, device=dev)
    k_blk = torch.empty((B, nc + N), dtype=torch.int32, device=dev)
    q_valid = torch.empty((B, N), dtype=torch.bool, device=dev)
    k_valid = torch.empty((B, nc + N), dtype=torch.bool, device=dev)
    _lib.check(_L.bfa_make_block_ids(_ptr(pad), _ptr(att), B, N, nc, _ptr(cpad), _ptr(q_blk), _ptr(k_blk),
                                     _ptr(q_valid), _ptr(k_valid), _stream(stream)))
    return q_blk, k_blk, q_valid, k_valid


def plan_dense(mask, stream=None):
    """Plan from a dense (Sq, Sk) bool CUDA mask (True = attend), shared by all batches/heads."""
    if mask.dim() != 2:
        raise ValueError("mask must be 2-D (Sq, Sk)")
    m = mask if mask.dtype in (torch.bool, torch.uint8) else (mask != 0)
    if m.stride(1) != 1:
        m = m.contiguous()
    h = ctypes.c_void_p()
    st = _stream(stream)
    _lib.check(_L.bfa_plan_dense(_ptr(m), m.stride(0), m.shape[0], m.shape[1], ctypes.byref(h), st))
    return Plan(h, st)


def plan_blockids(q_blk=None, k_blk=None, q_valid=None, k_valid=None, *, B=None, Sq=None, Sk=None,
                  cu_seqlens_q=None, cu_seqlens_k=None, seqused_k=None, max_q=0, max_k=0, window_left=-1,
                  stream=None):
    """Plan from block ids / validity (opentau) or, with ids None, from causal positions.

    Batched: ids (B, Sq) / (B, Sk).  Varlen: ids over packed tokens, ``cu_seqlens_*``
    int32 (B + 1,) starting at 0, ``max_q`` / ``max_k`` >= every sequence length.
    ``seqused_k`` int32 (B,) bounds the usable keys of each batch entry / sequence.
    ``window_left`` > 0 keeps keys with 0 <= q_pos - k_pos < window_left.
    """
    varlen = cu_seqlens_q is not None
    if varlen:
        B = cu_seqlens_q.numel() - 1
        Sq = Sk = 0
    elif q_blk is not None:
        B, Sq = q_blk.shape
        Sk = k_blk.shape[1]
    elif q_valid is not None:
        B, Sq = q_valid.shape
        Sk = k_valid.shape[1] if k_valid is not None else Sk
    for t in (q_blk, k_blk):
        if t is not None and t.dtype != torch.int32:
            raise TypeError("block ids must be int32")
    qv = _u8(q_valid).contiguous() if q_valid is not None else None
    kv = _u8(k_valid).contiguous() if k_valid is not None else None
    qb = q_blk.contiguous() if q_blk is not None else None
    kb = k_blk.contiguous() if k_blk is not None else None
    cq = cu_seqlens_q.to(torch.int32).contiguous() if varlen else None
    ck = (cu_seqlens_k if cu_seqlens_k is not None else cu_seqlens_q).to(torch.int32).contiguous() if varlen else None
    h = ctypes.c_void_p()
    st = _stream(stream)
    su = seqused_k.to(torch.int32).contiguous() if seqused_k is not None else None
    _lib.check(_L.bfa_plan_blockids(_ptr(qb), _ptr(kb), _ptr(qv), _ptr(kv), int(B), int(Sq or 0), int(Sk or 0),
                                    _ptr(cq), _ptr(ck), _ptr(su), int(max_q), int(max_k), int(window_left),
                                    ctypes.byref(h), st))
    return Plan(h, st)


def plan_predicate(terms, *, B=None, Sq=None, Sk=None, cu_seqlens_q=None, cu_seqlens_k=None, seqused_k=None,
                   max_q=0, max_k=0, stream=None):
    """Plan from position terms: attend(i, j) = OR over terms of
    diag_lo <= i - j <= diag_hi AND q_lo <= i < q_hi AND k_lo <= j < k_hi.

    ``terms``: list of dicts with those keys (missing / None = unbounded).  Layout
    as for ``plan_blockids`` (batched B, Sq, Sk or varlen cu_seqlens).
    """
    arr = (_lib.MaskTerm * max(len(terms), 1))()
    for n, t in enumerate(terms):
        get = lambda key, dflt: dflt if t.get(key) is None else int(t[key])
        arr[n] = _lib.MaskTerm(get("diag_lo", _I32_MIN), get("diag_hi", _I32_MAX), get("q_lo", _I32_MIN),
                               get("q_hi", _I32_MAX), get("k_lo", _I32_MIN), get("k_hi", _I32_MAX))
    varlen = cu_seqlens_q is not None
    if varlen:
        B = cu_seqlens_q.numel() - 1
        Sq = Sk = 0
    cq = cu_seqlens_q.to(torch.int32).contiguous() if varlen else None
    ck = (cu_seqlens_k if cu_seqlens_k is not None else cu_seqlens_q).to(torch.int32).contiguous() if varlen else None
    su = seqused_k.to(torch.int32).contiguous() if seqused_k is not None else None
    h = ctypes.c_void_p()
    st = _stream(stream)
    _lib.check(_L.bfa_plan_predicate(ctypes.cast(arr, ctypes.c_void_p), len(terms), int(B), int(Sq or 0),
                                     int(Sk or 0), _ptr(cq), _ptr(ck), _ptr(su), int(max_q), int(max_k),
                                     ctypes.byref(h), st))
    return Plan(h, st)


def plan_bsr(block_indptr, block_indices, Sq, Skv, q_block_size=TILE, kv_block_size=TILE, causal=False,
             kv_valid_bits=None, stream=None):
    """Plan from BSR routing: indptr (B, Hkv, ceil(Sq/q_block)+1) int32, indices int32.

    ``kv_valid_bits`` (B, ceil(Skv/32)) int32/uint32 marks valid key tokens, LSB first.
    """
    ip = block_indptr.to(torch.int32).contiguous()
    ix = block_indices.to(torch.int32).contiguous()
    kv = kv_valid_bits.contiguous() if kv_valid_bits is not None else None
    B, Hkv, _ = ip.shape
    h = ctypes.c_void_p()
    st = _stream(stream)
    _lib.check(_L.bfa_plan_bsr(_ptr(ip), _ptr(ix) if ix.numel() else None, ix.numel(), B, Hkv, int(Sq), int(Skv),
                               int(q_block_size), int(kv_block_size), 1 if causal else 0, _ptr(kv),
                               ctypes.byref(h), st))
    return Plan(h, st)


def plan_bsr_packed(block_indptr, block_indices, Sq, Skv, heads_per_kv, q_block_size=TILE, kv_block_size=TILE,
                    causal=False, kv_valid_bits=None, stream=None):
    """BSR plan with GQA-packed query tiles: each tile holds 128 / heads_per_kv query
    positions of all ``heads_per_kv`` query heads of a kv head (H = Hkv * heads_per_kv
    in the calls that use it, forward and backward)."""
    ip = block_indptr.to(torch.int32).contiguous()
    ix = block_indices.to(torch.int32).contiguous()
    kv = kv_valid_bits.contiguous() if kv_valid_bits is not None else None
    B, Hkv, _ = ip.shape
    h = ctypes.c_void_p()
    st = _stream(stream)
    _lib.check(_L.bfa_plan_bsr_packed(_ptr(ip), _ptr(ix) if ix.numel() else None, ix.numel(), B, Hkv,
                                      int(heads_per_kv), int(Sq), int(Skv), int(q_block_size), int(kv_block_size),
                                      1 if causal else 0, _ptr(kv), ctypes.byref(h), st))
    return Plan(h, st)


def plan_block_bits(exact_block_bits, Sq, Skv, q_block_size=TILE, kv_block_size=TILE, causal=False,
                    kv_valid_bits=None, stream=None):
    """Plan from an exact-block bitmap (B, Hkv, ceil(Sq/q_block), ceil(nkb/32)), LSB first."""
    bits = exact_block_bits.contiguous()
    kv = kv_valid_bits.contiguous() if kv_valid_bits is not None else None
    B, Hkv = bits.shape[:2]
    h = ctypes.c_void_p()
    st = _stream(stream)
    _lib.check(_L.bfa_plan_block_bits(_ptr(bits), B, Hkv, int(Sq), int(Skv), int(q_block_size), int(kv_block_size),
                                      1 if causal else 0, _ptr(kv), ctypes.byref(h), st))
    return Plan(h, st)


def _strides3(t):
    if t.dim() == 4:
        return (ctypes.c_int64 * 3)(t.stride(0), t.stride(1), t.stride(2))
    if t.dim() == 3:
        return (ctypes.c_int64 * 3)(0, t.stride(0), t.stride(1))
    raise ValueError("expected a 4-D (B, S, H, D) or 3-D (T, H, D) tensor")


def fwd(plan, q, k, v, scale=None, out=None, return_lse=True, lse=None, stream=None, softmax_threshold=None,
        softcap=None, slopes=None):
    """Masked attention forward; returns (out, lse or None).

    Batched q (B, Sq, H, D), k/v (B, Sk, Hkv, D); packed (varlen plans) q (Tq, H, D),
    k/v (Tk, Hkv, D).  bf16, last dim contiguous, D in {64, 128}.  A positive
    ``softmax_threshold`` turns on content-based block skipping (approximate).

    Shaped scores: ``softcap * tanh(scale * q.k / softcap) - slopes[h] * |i - j|``, with
    ``softcap`` in [1e-3, 1e6] (None: no cap) and ``slopes`` (H,) float32 (None: no
    distance penalty); positions are those of the plan's masks.  Not with GQA-packed
    plans or block skipping.
    """
    if softcap is not None or slopes is not None:
        if softmax_threshold is not None:
            raise ValueError("softmax_threshold does not go with shaped scores")
        return _fwd_shaped(plan, q, k, v, scale, out, return_lse, lse, stream, softcap, slopes)
    for t in (q, k, v):
        if t.dtype != torch.bfloat16:
            raise TypeError("q, k, v must be bfloat16")
        if t.stride(-1) != 1:
            raise ValueError("the head dim of q, k, v must be contiguous")
    packed = q.dim() == 3
    if packed:
        B = plan.info["batch"]
        _, H, D = q.shape
        Hkv = k.shape[1]
        lse_shape = (H, q.shape[0])
    else:
        B, Sq, H, D = q.shape
        Hkv = k.shape[2]
        lse_shape = (B, H, Sq)
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    if not return_lse:
        lse = None
    sc = float(scale) if scale is not None else 0.0
    if softmax_threshold is None:
        _lib.check(_L.bfa_fwd(plan.handle, _ptr(q), _ptr(k), _ptr(v), _strides3(q), _strides3(k), _strides3(v),
                              int(B), int(H), int(Hkv), int(D), ctypes.c_float(sc), _ptr(out), _strides3(out),
                              _ptr(lse), _stream(stream)))
    else:  # content-based block skipping (an approximation)
        _lib.check(_L.bfa_fwd_approx(plan.handle, _ptr(q), _ptr(k), _ptr(v), _strides3(q), _strides3(k),
                                     _strides3(v), int(B), int(H), int(Hkv), int(D), ctypes.c_float(sc),
                                     ctypes.c_float(float(softmax_threshold)), _ptr(out), _strides3(out), _ptr(lse),
                                     _stream(stream)))
    return out, lse


def _shapes(plan, q, k, v):
    """(B, H, Hkv, D, lse shape) of a batched or packed call, with the forms and types checked."""
    for t in (q, k, v):
        if t.dtype != torch.bfloat16:
            raise TypeError("q, k, v must be bfloat16")
        if t.dim() != q.dim() or t.dim() not in (3, 4):
            raise ValueError("q, k, v must all be (B, S, H, D) or all packed (T, H, D)")
        if t.stride(-1) != 1:
            raise ValueError("the head dim of q, k, v must be contiguous")
    if k.shape != v.shape or k.shape[-1] != q.shape[-1]:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not fit together")
    info = plan.info
    if q.dim() == 3:
        if not info["varlen"]:
            raise ValueError("packed (T, H, D) tensors need a varlen plan")
        B, lse_shape = info["batch"], (q.shape[1], q.shape[0])
    else:
        if info["varlen"]:
            raise ValueError("a varlen plan needs packed (T, H, D) tensors")
        B, lse_shape = q.shape[0], (q.shape[0], q.shape[2], q.shape[1])
        if k.shape[0] != B:
            raise ValueError("q and k must have the same batch size")
    if q.shape[-3] != info["sq"] or k.shape[-3] != info["sk"]:
        raise ValueError(f"the plan is for {info['sq']} queries and {info['sk']} keys, not {q.shape[-3]} and {k.shape[-3]}")
    return int(B), int(q.shape[-2]), int(k.shape[-2]), int(q.shape[-1]), lse_shape


def _like(t, x, name):
    """A caller's result tensor in the form of x, checked, or a new one."""
    if t is None:
        return torch.empty_like(x)
    return _result(t, x, x.shape, x.dtype, name)


def _result(t, x, shape, dtype, name):
    """A caller's result tensor, checked, or a new one beside x."""
    if t is None:
        return x.new_empty(shape, dtype=dtype)
    if t.shape != shape or t.dtype is not dtype or t.device != x.device:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype} on {x.device}")
    if t.dim() and t.stride(-1) != 1:
        raise ValueError(f"the last dim of {name} must be contiguous")
    return t


def _fwd_shaped(plan, q, k, v, scale, out, return_lse, lse, stream, softcap, slopes):
    B, H, Hkv, D, lse_shape = _shapes(plan, q, k, v)
    _same_device(q, k, v)
    cap = _score_shape(softcap, slopes, q, H)
    if lse is not None and return_lse and not lse.is_contiguous():
        raise ValueError("lse must be contiguous")

    def body(st, finish):
        o = _like(out, q, "out")
        l = _result(lse, q, lse_shape, torch.float32, "lse") if return_lse else None
        sl = None if slopes is None else slopes.contiguous()
        _lib.check(_L.bfa_fwd_shaped(plan.handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), _strides_of(q),
                                     _strides_of(k), _strides_of(v), B, H, Hkv, D, scale or 0.0, cap, _addr(sl),
                                     o.data_ptr(), _strides_of(o), _addr(l), st))
        finish(o if out is None else None, l if lse is None else None)
        return o, l

    return _run_on(q, stream, body)


def _bwd_shaped(plan, q, k, v, out, dout, lse, scale, dq, dk, dv, stream, softcap, slopes):
    B, H, Hkv, D, lse_shape = _shapes(plan, q, k, v)
    for t in (out, dout):
        if t.dtype != torch.bfloat16 or t.shape != q.shape or t.stride(-1) != 1:
            raise ValueError("out and dout must be bfloat16 with the shape of q and a contiguous head dim")
    if lse is None or lse.dtype != torch.float32 or lse.shape != lse_shape:
        raise ValueError(f"lse (float32 {tuple(lse_shape)}, from fwd) is required")
    _same_device(q, k, v, out, dout, lse)
    cap = _score_shape(softcap, slopes, q, H)

    def body(st, finish):
        gq = _like(dq, q, "dq")
        gk = _like(dk, k, "dk")
        gv = _like(dv, v, "dv")
        l = lse.contiguous()
        sl = None if slopes is None else slopes.contiguous()
        _lib.check(_L.bfa_bwd_shaped(plan.handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                     dout.data_ptr(), l.data_ptr(), _strides_of(q), _strides_of(k), _strides_of(v),
                                     _strides_of(out), _strides_of(dout), B, H, Hkv, D, scale or 0.0, cap,
                                     _addr(sl), gq.data_ptr(), gk.data_ptr(), gv.data_ptr(), _strides_of(gq),
                                     _strides_of(gk), _strides_of(gv), st))
        finish(gq if dq is None else None, gk if dk is None else None, gv if dv is None else None)
        return gq, gk, gv

    return _run_on(q, stream, body)


def bwd(plan, q, k, v, out, dout, lse, scale=None, dq=None, dk=None, dv=None, stream=None, softcap=None, slopes=None):
    """Gradients (dq, dk, dv) of ``fwd`` for an upstream gradient ``dout`` of ``out``.

    q, k, v, the plan and scale exactly as given to ``fwd``; out and lse as it
    returned them; dout shaped like q.  bf16 outputs shaped like q, k, v (dk and
    dv sum over the query heads of each kv head under GQA).  ``softcap`` and
    ``slopes`` as given to ``fwd``; the slopes are constants, they get no gradient.
    """
    if softcap is not None or slopes is not None:
        return _bwd_shaped(plan, q, k, v, out, dout, lse, scale, dq, dk, dv, stream, softcap, slopes)
    for t in (q, k, v, out, dout):
        if t.dtype != torch.bfloat16:
            raise TypeError("q, k, v, out, dout must be bfloat16")
        if t.stride(-1) != 1:
            raise ValueError("the head dim of q, k, v, out, dout must be contiguous")
    if lse is None or lse.dtype != torch.float32:
        raise TypeError("lse (float32, from fwd) is required")
    if dout.shape != q.shape or out.shape != q.shape:
        raise ValueError("out and dout must have the shape of q")
    packed = q.dim() == 3
    if packed:
        B = plan.info["batch"]
        _, H, D = q.shape
        Hkv = k.shape[1]
    else:
        B, _, H, D = q.shape
        Hkv = k.shape[2]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    sc = float(scale) if scale is not None else 0.0
    _lib.check(_L.bfa_bwd(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse.contiguous()),
                          _strides3(q), _strides3(k), _strides3(v), _strides3(out), _strides3(dout), int(B), int(H),
                          int(Hkv), int(D), ctypes.c_float(sc), _ptr(dq), _ptr(dk), _ptr(dv), _strides3(dq),
                          _strides3(dk), _strides3(dv), _stream(stream)))
    return dq, dk, dv


def fwd_paged(plan, q, k_cache, v_cache, block_table, scale=None, out=None, return_lse=True, lse=None, stream=None):
    """Masked attention forward with keys / values in a paged cache.

    k_cache / v_cache: (num_pages, page_size, Hkv, D) bf16; block_table: (n_seq,
    pages_per_seq) int32 page ids (tensorplay varlen ``block_table``).  q and the
    plan as for ``fwd``.
    """
    if q.dtype != torch.bfloat16 or k_cache.dtype != torch.bfloat16 or v_cache.dtype != torch.bfloat16:
        raise TypeError("q and the caches must be bfloat16")
    if k_cache.stride() != v_cache.stride() or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    packed = q.dim() == 3
    if packed:
        B = plan.info["batch"]
        _, H, D = q.shape
        lse_shape = (H, q.shape[0])
    else:
        B, Sq, H, D = q.shape
        lse_shape = (B, H, Sq)
    num_pages, page_size, Hkv, _ = k_cache.shape
    bt = block_table.to(torch.int32).contiguous()
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    if not return_lse:
        lse = None
    cs = (ctypes.c_int64 * 3)(k_cache.stride(0), k_cache.stride(1), k_cache.stride(2))
    sc = float(scale) if scale is not None else 0.0
    _lib.check(_L.bfa_fwd_paged(plan.handle, _ptr(q), _strides3(q), _ptr(k_cache), _ptr(v_cache), cs, num_pages,
                                page_size, _ptr(bt), bt.shape[1], int(B), int(H), int(Hkv), int(D),
                                ctypes.c_float(sc), _ptr(out), _strides3(out), _ptr(lse), _stream(stream)))
    return out, lse


def _check_cache(k_cache, v_cache, block_table, cu_seqlens, seqused_k):
    """The forms of a paged cache and a ragged batch's integers; (cache shape, cache strides)."""
    if k_cache.dtype is not torch.bfloat16 or v_cache.dtype is not torch.bfloat16:
        raise TypeError("the caches must be bfloat16")
    shape, strides = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or strides != v_cache.stride() or shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must be (num_pages, page_size, Hkv, D) with the same shape and strides")
    if strides[3] != 1:
        raise ValueError("the head dim of the caches must be contiguous")
    used = seqused_k.shape
    if len(used) != 1 or cu_seqlens.shape != (used[0] + 1,):
        raise ValueError("cu_seqlens must hold one entry more than seqused_k")
    table = block_table.shape
    if len(table) != 2 or table[0] != used[0]:
        raise ValueError("block_table must be (sequences, pages per sequence)")
    for t in (block_table, cu_seqlens, seqused_k):
        if t.dtype is not torch.int32 and t.dtype is not torch.int64:
            raise TypeError("block_table, cu_seqlens and seqused_k must be int32 or int64")
    _same_device(k_cache, v_cache, block_table, cu_seqlens, seqused_k)
    # a cache of one page has no page stride of its own
    return shape, _Strides3(strides[0] if shape[0] > 1 else shape[1] * strides[1], strides[1], strides[2])


def _int32(t):
    """t as contiguous int32; called where the launch's stream is current, since it may copy."""
    return t if t.dtype is torch.int32 and t.is_contiguous() else t.to(torch.int32).contiguous()


@functools.lru_cache(maxsize=1024)
def _chunk_workspace(total_q, B, max_q, H, Hkv, D):
    need = _L.bfa_fwd_chunk_workspace(total_q, B, max_q, H, Hkv, D)
    if need < 0:
        _lib.check(-2 if D not in (64, 128) else -1)
    return need


def _check_packed(t, name, heads, D):
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if t.dim() != 3 or t.shape[2] != D or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be (tokens, {'heads' if heads is None else heads}, {D}), not {tuple(t.shape)}")
    if t.stride(-1) != 1:
        raise ValueError(f"the head dim of {name} must be contiguous")


def fwd_chunk(q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k, *, max_q=0, scale=None, window_left=-1,
              softcap=None, slopes=None, out=None, return_lse=True, lse=None, workspace=None, stream=None):
    """Attention of the newest tokens of each sequence over a paged cache; returns (out, lse or None).

    q (T, H, D) bf16 packed by ``cu_seqlens_q`` (B + 1,); ``seqused_k`` (B,) keys of each
    sequence, the new tokens' own included (``append_paged`` writes them).  The last
    new token of a sequence stands at position seqused_k - 1; each attends the keys up
    to its own position, of the last ``window_left`` of them if that is positive.
    Caches and ``block_table`` as for ``fwd_paged``; ``softcap`` and ``slopes`` as for
    ``fwd``.  ``max_q``: the most new tokens of a sequence, if known: it chooses the
    kernels, and decoding without it (1) also launches the one for longer chunks (10 us).
    ``workspace``: a contiguous CUDA tensor to use as scratch, of at least
    ``bfa_fwd_chunk_workspace`` bytes.  Lengths stay on the device: no synchronisation,
    and a captured call follows their contents.  Rows of q behind the last sequence
    are left as they are in out and lse.
    """
    (num_pages, page_size, Hkv, D), cache_strides = _check_cache(k_cache, v_cache, block_table, cu_seqlens_q, seqused_k)
    _check_packed(q, "q", None, D)
    _same_device(q, k_cache, workspace)
    T, H, _ = q.shape
    # to what the library's 32-bit arguments hold, with the same meaning (2^30 keys are all of them)
    max_q, window_left = max(0, min(int(max_q), T)), max(-2, min(int(window_left), 1 << 30))
    B = seqused_k.shape[0]
    cap = _score_shape(softcap, slopes, q, H)
    need = _chunk_workspace(T, B, max_q, H, Hkv, D)
    if lse is not None and return_lse and not lse.is_contiguous():
        raise ValueError("lse must be contiguous")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous: it is used as one run of bytes")

    def body(st, finish):
        table, cu, used = _int32(block_table), _int32(cu_seqlens_q), _int32(seqused_k)
        sl = None if slopes is None else slopes.contiguous()
        o = _like(out, q, "out")
        l = _result(lse, q, (H, T), torch.float32, "lse") if return_lse else None
        ws = q.new_empty(need, dtype=torch.uint8) if workspace is None else workspace
        _lib.check(_L.bfa_fwd_chunk(q.data_ptr(), _strides_of(q), k_cache.data_ptr(), v_cache.data_ptr(), cache_strides,
                                    num_pages, page_size, table.data_ptr(), table.shape[1], cu.data_ptr(),
                                    used.data_ptr(), B, T, max_q, H, Hkv, D, scale or 0.0, window_left, cap, _addr(sl),
                                    o.data_ptr(), _strides_of(o), _addr(l), ws.data_ptr(),
                                    need if workspace is None else ws.numel() * ws.element_size(), st))
        finish(o if out is None else None, l if lse is None else None)
        return o, l

    return _run_on(q, stream, body)


def chunk_device_status(stream=None):
    """Raise BfaError(BFA_ERR_TIMEOUT) if a ``fwd_chunk`` on the current device hit its wait bound."""
    _lib.check(_L.bfa_chunk_device_status(_stream(stream)))


def rope_frequencies(rotary, base=10000.0, *, factor=1.0, ramp=None, device="cuda"):
    """Radians per position of each pair, float64 (rotary / 2,): base ** (-2 i / rotary).

    Long contexts: ``factor`` divides the frequencies (positions are interpolated).  With
    ``ramp = (length, low, high)`` only slow pairs are divided: a pair that makes n turns
    over ``length`` positions keeps the share clamp((n - low) / (high - low), 0, 1) of its
    own frequency and takes the rest of the divided one.
    """
    if rotary <= 0 or rotary % 2:
        raise ValueError("rotary must be a positive even number")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    f = torch.pow(torch.tensor(float(base), dtype=torch.float64),
                  -torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    if ramp is None:
        f = f / factor
    else:
        length, low, high = ramp
        if not (length > 0 and high > low):
            raise ValueError("ramp must be (length > 0, low, high > low)")
        keep = ((length * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f.to(device)


def _check_frequencies(inv_freq, like):
    """rotary of the frequencies (0 without)."""
    if inv_freq is None:
        return 0
    if inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1:
        raise TypeError("inv_freq must be a 1-D float64 tensor (rope_frequencies)")
    _same_device(like, inv_freq)
    return 2 * inv_freq.shape[0]


def rope(x, positions, inv_freq, *, interleaved=False, amplitude=1.0, inverse=False, out=None, stream=None):
    """Rotary positions: x (B, S, H, D) or (T, H, D) bf16 with the first 2 * len(inv_freq)
    values of each head turned in pairs; returns the result (``out=x`` works in place).

    positions: int32 or int64, (B, S), or (S,) for every batch row, or (T,).  Pairs are
    (i, i + rotary / 2), or (2 i, 2 i + 1) with ``interleaved``; ``amplitude`` scales
    what turns.  ``inverse`` turns back: it is the gradient, dx = rope(dout, inverse=True).
    """
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    if x.dim() not in (3, 4) or x.stride(-1) != 1:
        raise ValueError("x must be (B, S, H, D) or (T, H, D) with a contiguous head dim")
    if positions.dtype not in (torch.int32, torch.int64):
        raise TypeError("positions must be int32 or int64")
    B = x.shape[0] if x.dim() == 4 else 1
    S, H, D = x.shape[-3:]
    if positions.shape not in ((S,), x.shape[:-2]):
        raise ValueError(f"positions must be {tuple(x.shape[:-2])} or {(S,)}, not {tuple(positions.shape)}")
    if inv_freq is None:
        raise TypeError("inv_freq is required (rope_frequencies)")
    rotary = _check_frequencies(inv_freq, x)
    _same_device(x, positions)
    if out is not None and out.data_ptr() == x.data_ptr() and out.stride() != x.stride():
        raise ValueError("an in-place result must be x itself")
    if x.numel() == 0:
        return out if out is not None else torch.empty_like(x)

    def body(st, finish):
        y = _like(out, x, "out")
        at, f = positions.contiguous(), inv_freq.contiguous()
        _lib.check(_L.bfa_rope(x.data_ptr(), _strides_of(x), y.data_ptr(), _strides_of(y), at.data_ptr(),
                               1 if at.dtype is torch.int64 else 0, S if at.dim() == 2 else 0, f.data_ptr(), rotary,
                               B, S, H, D, 1 if interleaved else 0, amplitude, 1 if inverse else 0, st))
        finish(y if out is None else None)
        return y

    return _run_on(x, stream, body)


def append_paged(k, v, k_cache, v_cache, block_table, cu_seqlens, seqused_k, *, q=None, q_out=None, inv_freq=None,
                 interleaved=False, amplitude=1.0, stream=None):
    """Write new keys and values (T, Hkv, D) into a paged cache, keys turned by their positions.

    Sequence s owns rows cu_seqlens[s] .. cu_seqlens[s + 1]; ``seqused_k`` (B,) counts its
    keys after the call.  ``q`` (T, H, D) is turned the same way in the same launch and
    returned (into ``q_out``; ``q_out=q`` works in place); without q the result is None.
    ``inv_freq`` None: keys and queries are copied.  Rows behind the last sequence are left
    out.  Lengths and pages stay on the device, as for ``fwd_chunk``.
    """
    (num_pages, page_size, Hkv, D), cache_strides = _check_cache(k_cache, v_cache, block_table, cu_seqlens, seqused_k)
    _check_packed(k, "k", Hkv, D)
    _check_packed(v, "v", Hkv, D)
    T, H = k.shape[0], Hkv
    if v.shape != k.shape:
        raise ValueError("k and v must have the same shape")
    _same_device(k, v, k_cache, q)
    if q is not None:
        _check_packed(q, "q", None, D)
        H = q.shape[1]
        if q.shape[0] != T:
            raise ValueError("q, k and v must hold the same tokens")
        if q_out is not None and q_out.data_ptr() == q.data_ptr() and q_out.stride() != q.stride():
            raise ValueError("an in-place q_out must be q itself")
    elif q_out is not None:
        raise ValueError("q_out without q")
    rotary = _check_frequencies(inv_freq, k)

    def body(st, finish):
        qo = None if q is None else _like(q_out, q, "q_out")
        none3 = _Strides3(0, 0, 0)
        table, cu, used = _int32(block_table), _int32(cu_seqlens), _int32(seqused_k)
        f = None if inv_freq is None else inv_freq.contiguous()
        _lib.check(_L.bfa_append_paged(k.data_ptr(), _strides_of(k), v.data_ptr(), _strides_of(v), _addr(q),
                                       none3 if q is None else _strides_of(q), _addr(qo),
                                       none3 if q is None else _strides_of(qo), k_cache.data_ptr(), v_cache.data_ptr(),
                                       cache_strides, num_pages, page_size, table.data_ptr(), table.shape[1],
                                       cu.data_ptr(), used.data_ptr(), used.shape[0], T, H, Hkv, D, _addr(f),
                                       rotary, 1 if interleaved else 0, amplitude, st))
        finish(qo if q_out is None else None)
        return qo

    return _run_on(k, stream, body)
