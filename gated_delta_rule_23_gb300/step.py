"""Tensor-level binding of the decoder-step operators (argument marshalling only).

A decode or prefill step of a hybrid decoder around ``kda_fwd`` / ``kda_fwd_recurrent``: ``kda_kv_append`` stores
rotated keys and values in a paged cache, ``kda_window_attn`` attends to it through a sliding window with sinks,
``kda_beam_select`` picks the next beams from the logits, ``kda_state_reorder`` moves the states after them.  The
caller passes CUDA tensors and pre-allocated outputs; every step of the computation runs in libkda.so.

Every function first offers its arguments to the compiled binding (csrc/kda_binding.cpp), which makes the call when they
are exactly what it expects and otherwise declines; the code here then checks them one by one, and makes the call (an
empty batch, another device than the current one) or says what is wrong.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Union

import torch

from . import _native
from ._native import KDA_DTYPE_BF16, KDA_DTYPE_FP32, KDA_OK, KDAError
from .api import _check, _ptr

Tensors = Union[torch.Tensor, Sequence[torch.Tensor]]


def _need(t: torch.Tensor, name: str, dtype, shape, dev) -> None:
    """A contiguous tensor of this type, shape and device (the detailed message only where one differs)."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _check(t, name, dtype, shape, dev)


def _rows(t: torch.Tensor, name: str, heads: int, dim: int, lead, dev) -> int:
    """Token stride (elements) of a [B, T, heads, dim] tensor whose tokens are evenly spaced."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
    if t.shape != (*lead, heads, dim):
        raise ValueError(f"{name}: expected shape {(*lead, heads, dim)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name}: expected device {dev}, got {t.device}")
    if t.is_contiguous():
        return heads * dim
    b, n = lead
    s = t.stride()
    step = s[1] if n > 1 else (s[0] if b > 1 else heads * dim)
    if t.numel() and ((dim > 1 and s[3] != 1) or (heads > 1 and s[2] != dim) or (b > 1 and s[0] != n * step)
                      or step % 8 or step < heads * dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous and the tokens evenly spaced "
                         f"(a multiple of 8 elements apart), got strides {s}")
    return step


def _cache(k_cache, v_cache, block_table, kv_lens, cu_seqlens, lead, dev):
    """(cu_seqlens pointer, N, T), (pages, page, max_pages) of a paged cache and its token batch."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, Hkv, page, D]")
    _need(k_cache, "k_cache", torch.bfloat16, k_cache.shape, dev)
    _need(v_cache, "v_cache", torch.bfloat16, k_cache.shape, dev)
    b, t = lead
    n = b
    if cu_seqlens is not None:
        if b != 1:
            raise ValueError("cu_seqlens requires B == 1")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be int64 [N + 1]")
        n = cu_seqlens.numel() - 1
        _need(cu_seqlens, "cu_seqlens", torch.int64, (n + 1,), dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [N, max_pages]")
    _need(block_table, "block_table", torch.int32, (n, block_table.shape[1]), dev)
    _need(kv_lens, "kv_lens", torch.int32, (n,), dev)
    return n, t


def _device(t: torch.Tensor, name: str) -> torch.device:
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name} needs CUDA tensors")
    return dev


def _fit(fn, args) -> None:
    """ctypes keeps the low 32 bits of an int that has more: those are refused here."""
    for a, kind in zip(args, fn.argtypes):
        if kind is ctypes.c_int and not -2 ** 31 <= a < 2 ** 31:
            raise ValueError(f"{fn.__name__}: {a} does not fit the 32 bits of the argument it is for")


def _keys(count) -> int:
    """A window or a number of sinks: 2^31 - 1 and anything above are every key."""
    return min(int(count), 2 ** 31 - 1)


def _call(fn, dev: torch.device, stream: Optional[torch.cuda.Stream], *args) -> None:
    _fit(fn, args)
    if dev.index == torch.cuda.current_device():
        rc = fn(*args, (stream if stream is not None else torch.cuda.current_stream(dev)).cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, (stream if stream is not None else torch.cuda.current_stream(dev)).cuda_stream)
    if rc != KDA_OK:
        raise KDAError(rc)


def _workspace(workspace: torch.Tensor, dev: torch.device) -> int:
    if workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return workspace.numel()


def _raise(rc: int) -> None:
    if rc != KDA_OK:
        raise KDAError(rc)


def kda_kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  block_table: torch.Tensor, kv_lens: torch.Tensor, cos: Optional[torch.Tensor] = None,
                  sin: Optional[torch.Tensor] = None, interleaved: bool = False, q: Optional[torch.Tensor] = None,
                  q_out: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """Rotate and store the new keys and values in the paged cache; rotate the new queries into ``q_out``.

    k, v: bf16 [B, T, Hkv, D], q: bf16 [B, T, Hq, D] (tokens evenly spaced: slices of one projection's rows);
    k_cache, v_cache: bf16 [pages, Hkv, page, D]; block_table: int32 [N, max_pages]; kv_lens: int32 [N], the tokens
    in the cache including these; cos, sin: fp32 [positions, rotary / 2] (None: no rotation); cu_seqlens: int64
    [N + 1] with B = 1.  ``q_out`` may be ``q``.  Runs asynchronously on ``stream`` (default: the current stream).
    """
    rc = _native.binding().kv_append(k, v, k_cache, v_cache, block_table, kv_lens, cos, sin, interleaved, q, q_out,
                                     cu_seqlens, None if stream is None else stream.cuda_stream)
    if rc is not None:
        return _raise(rc)
    dev = _device(k, "kda_kv_append")
    if k.dim() != 4:
        raise ValueError("k must be [B, T, Hkv, D]")
    b, t, hkv, d = k.shape
    lead = (b, t)
    ks = _rows(k, "k", hkv, d, lead, dev)
    vs = _rows(v, "v", hkv, d, lead, dev)
    n, t = _cache(k_cache, v_cache, block_table, kv_lens, cu_seqlens, lead, dev)
    pages, ch, page, cd = k_cache.shape
    if (ch, cd) != (hkv, d):
        raise ValueError(f"k_cache: expected [pages, {hkv}, page, {d}], got {tuple(k_cache.shape)}")
    rotary = positions = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is not None:
        if cos.dim() != 2:
            raise ValueError("cos must be fp32 [positions, rotary / 2]")
        _need(cos, "cos", torch.float32, cos.shape, dev)
        _need(sin, "sin", torch.float32, cos.shape, dev)
        positions, rotary = cos.shape[0], 2 * cos.shape[1]
    hq = qs = 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    if q is not None:
        if q.dim() != 4:
            raise ValueError("q must be [B, T, Hq, D]")
        hq = q.shape[2]
        qs = _rows(q, "q", hq, d, lead, dev)
        _need(q_out, "q_out", torch.bfloat16, q.shape, dev)
    _call(_native.load().kda_kv_append, dev, stream, k.data_ptr(), ks, v.data_ptr(), vs, k_cache.data_ptr(),
          v_cache.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr(), _ptr(cos), _ptr(sin), rotary, positions,
          int(interleaved), _ptr(q), qs, _ptr(q_out), _ptr(cu_seqlens), n, t, hq, hkv, d, pages, page,
          block_table.shape[1])


def kda_window_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    kv_lens: torch.Tensor, out: torch.Tensor, window: int, sinks: int = 0,
                    scale: Optional[float] = None, lse: Optional[torch.Tensor] = None,
                    cu_seqlens: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                    workspace: Optional[torch.Tensor] = None) -> None:
    """Attention over the paged cache: query position p sees key j when j <= p and (j > p - window or j < sinks).

    q, out: bf16 [B, T, Hq, D] (q's tokens evenly spaced); lse: optional fp32 [B, T, Hq]; the cache arguments as for
    ``kda_kv_append``; ``scale`` defaults to D ** -0.5.  Rows that see nothing give out = 0 and lse = -inf.
    ``workspace``: optional uint8 tensor of ``window_attn_workspace_size`` bytes; without it the library's pool
    provides one where the call needs it.
    """
    rc = _native.binding().window_attn(q, k_cache, v_cache, block_table, kv_lens, out, window, sinks, scale, lse,
                                       cu_seqlens, None if stream is None else stream.cuda_stream, workspace)
    if rc is not None:
        return _raise(rc)
    dev = _device(q, "kda_window_attn")
    if q.dim() != 4:
        raise ValueError("q must be [B, T, Hq, D]")
    b, t, hq, d = q.shape
    lead = (b, t)
    qs = _rows(q, "q", hq, d, lead, dev)
    n, t = _cache(k_cache, v_cache, block_table, kv_lens, cu_seqlens, lead, dev)
    pages, hkv, page, cd = k_cache.shape
    if cd != d:
        raise ValueError(f"k_cache: expected head size {d}, got {cd}")
    _need(out, "out", torch.bfloat16, q.shape, dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, (b, t, hq), dev)
    args = (q.data_ptr(), qs, k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr(),
            out.data_ptr(), _ptr(lse), float(d ** -0.5 if scale is None else scale), _keys(window), _keys(sinks),
            _ptr(cu_seqlens), n, t, hq, hkv, d, pages, page, block_table.shape[1])
    if workspace is None:
        _call(_native.load().kda_window_attn, dev, stream, *args)
    else:
        size = _workspace(workspace, dev)
        _call(_native.load().kda_window_attn_ws, dev, stream, *args, workspace.data_ptr(), size)


def window_attn_workspace_size(window: int, sinks: int, N: int, T: int, Hq: int, Hkv: int, D: int, page: int,
                               max_pages: int, varlen: bool = False) -> int:
    """Bytes of workspace a kda_window_attn call of these sizes needs on the current device."""
    fn = _native.load().kda_window_attn_workspace_size
    args = (_keys(window), _keys(sinks), int(varlen), int(N), int(T), int(Hq), int(Hkv), int(D), int(page), int(max_pages))
    _fit(fn, args)
    return int(fn(*args))


def kda_beam_select(logits: torch.Tensor, beam_scores: torch.Tensor, scores: torch.Tensor, tokens: torch.Tensor,
                    parents: torch.Tensor, finished: Optional[torch.Tensor] = None, eos: int = 0,
                    stream: Optional[torch.cuda.Stream] = None, workspace: Optional[torch.Tensor] = None) -> None:
    """The K best continuations of every batch entry: score = beam score + log-softmax of the beam's logits.

    logits: bf16 or fp32 [B, W, V] (rows evenly spaced); beam_scores: fp32 [B, W]; finished: optional uint8 or bool
    [B, W], beams whose one continuation is ``eos`` at their own score.  Writes scores fp32, tokens int32 and parents
    int32 [B, K], best first, ties to the lower (beam, token); parents are rows b * W + w of the batch.  ``scores`` may
    be ``beam_scores`` where K = W; the outputs overlap nothing else.
    """
    rc = _native.binding().beam_select(logits, beam_scores, scores, tokens, parents, finished, eos,
                                       None if stream is None else stream.cuda_stream, workspace)
    if rc is not None:
        return _raise(rc)
    dev = _device(logits, "kda_beam_select")
    if logits.dim() != 3:
        raise ValueError("logits must be [B, W, V]")
    b, w, v = logits.shape
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"logits: expected bf16 or fp32, got {logits.dtype}")
    s = logits.stride()
    step = s[1] if w > 1 else (s[0] if b > 1 else v)
    if (v > 1 and s[2] != 1) or (b > 1 and s[0] != w * step) or step < v:
        raise ValueError(f"logits: the rows must be contiguous and evenly spaced, got strides {s}")
    _need(beam_scores, "beam_scores", torch.float32, (b, w), dev)
    if tokens.dim() != 2:
        raise ValueError("tokens must be int32 [B, K]")
    k = tokens.shape[1]
    _need(tokens, "tokens", torch.int32, (b, k), dev)
    _need(parents, "parents", torch.int32, (b, k), dev)
    _need(scores, "scores", torch.float32, (b, k), dev)
    if finished is not None:
        _need(finished, "finished", torch.bool if finished.dtype == torch.bool else torch.uint8, (b, w), dev)
    args = (logits.data_ptr(), KDA_DTYPE_BF16 if logits.dtype is torch.bfloat16 else KDA_DTYPE_FP32, step,
            beam_scores.data_ptr(), _ptr(finished), int(eos), scores.data_ptr(), tokens.data_ptr(),
            parents.data_ptr(), b, w, v, k)
    if workspace is None:
        _call(_native.load().kda_beam_select, dev, stream, *args)
    else:
        size = _workspace(workspace, dev)
        _call(_native.load().kda_beam_select_ws, dev, stream, *args, workspace.data_ptr(), size)


def beam_select_workspace_size(B: int, W: int, V: int, K: int) -> int:
    """Bytes of workspace a kda_beam_select call of these sizes needs."""
    fn, args = _native.load().kda_beam_select_workspace_size, (int(B), int(W), int(V), int(K))
    _fit(fn, args)
    return int(fn(*args))


def kda_state_reorder(src: Tensors, parents: torch.Tensor, beams: int, dst: Optional[Tensors] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """dst[i][n] = src[i][parents[n]] for every tensor of ``src`` (one tensor or a sequence of them, [N, ...]).

    ``parents``: int32 [N]; rows come in groups of ``beams`` and a row's parent lies in its own group (what
    ``kda_beam_select`` writes).  ``dst`` None (or the same tensors): in place; a destination overlaps no other tensor.
    """
    src = [src] if isinstance(src, torch.Tensor) else list(src)
    dst = src if dst is None else ([dst] if isinstance(dst, torch.Tensor) else list(dst))
    rc = _native.binding().state_reorder(src, dst, parents, beams, None if stream is None else stream.cuda_stream)
    if rc is not None:
        return _raise(rc)
    if len(src) != len(dst):
        raise ValueError(f"dst: expected {len(src)} tensors, got {len(dst)}")
    dev = _device(parents, "kda_state_reorder")
    n = parents.numel()
    _need(parents, "parents", torch.int32, (n,), dev)
    count = len(src)
    pointers, sizes = ctypes.c_void_p * count, ctypes.c_int64 * count
    ps, pd, rows = pointers(), pointers(), sizes()
    for i, (a, b) in enumerate(zip(src, dst)):
        if a.dim() < 1 or a.shape[0] != n:
            raise ValueError(f"src[{i}]: expected {n} rows, got shape {tuple(a.shape)}")
        _need(a, f"src[{i}]", a.dtype, a.shape, dev)
        if b is not a:
            _need(b, f"dst[{i}]", a.dtype, a.shape, dev)
        ps[i], pd[i], rows[i] = a.data_ptr(), b.data_ptr(), (a.numel() // n if n else 0) * a.element_size()
    _call(_native.load().kda_state_reorder, dev, stream, ps, pd, rows, count, parents.data_ptr(), n, int(beams))
