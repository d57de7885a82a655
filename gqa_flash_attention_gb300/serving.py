"""The operators around the attention forward on a serving path.

``qk_norm_rope``: norms and position rotation of the query and key heads in one pass, with
``rope_inv_freq`` and ``rope_table`` for its frequencies. ``Cache4``: a paged cache held in 4 bits,
written by ``cache4_append`` and read back by ``cache4_gather``; ``fwd_cache4``: the attention of each
sequence's last tokens over it. ``fwd_window`` and ``fwd_varlen_window``: prefill attention with a sliding
window and first tokens that stay visible.

As in the rest of the package, these functions check and marshal arguments for the C ABI of
``include/sdp.h`` (which states layouts, ownership and errors), PyTorch supplies memory and
streams, and there is no fallback. They compute forward passes only: a tensor that requires grad
is refused while grad mode is on.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from . import SDP_OK, _check, _DTYPE_CODE, _on, _stream_handle, lib

__all__ = ["rope_inv_freq", "rope_table", "RopeTable", "qk_norm_rope", "Cache4", "cache4_empty", "cache4_append",
           "cache4_gather", "CACHE4_GROUP", "fwd_cache4", "cache4_workspace_bytes",
           "fwd_window", "fwd_varlen_window"]

CACHE4_GROUP = 64  # channels that share one scale and bias

_declared = None


def _lib() -> ctypes.CDLL:
    """libsdp.so with the argument types of this module's calls declared."""
    global _declared
    if _declared is None:
        L = lib()
        vp, i, f, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong
        pool = [vp, vp, vp, vp, i, i, vp, ll, i]
        L.sdp_qk_norm_rope.argtypes = [vp, ll, ll, ll] * 4 + [vp, ll, ll, i, vp, i, f, vp, vp, i, f, i,
                                                              i, i, i, i, i, i, vp]
        L.sdp_qk_norm_rope.restype = i
        L.sdp_cache4_append.argtypes = pool + [vp, ll, ll, vp, ll, ll, vp, vp, i, i, i, i, i, vp]
        L.sdp_cache4_append.restype = i
        L.sdp_cache4_gather.argtypes = pool + [vp, ll, ll, vp, ll, ll, vp, i, i, i, i, i, vp]
        L.sdp_cache4_gather.restype = i
        L.sdp_fwd_cache4_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.sdp_fwd_cache4_workspace_bytes.restype = ll
        L.sdp_fwd_cache4.argtypes = [vp, *pool, vp, vp, vp, i, i, i, i, i, f, i, i, i, vp, ctypes.c_ulonglong, vp]
        L.sdp_fwd_cache4.restype = i
        L.sdp_fwd_window.argtypes = [vp] * 5 + [i] * 6 + [f, i, i, i, vp]
        L.sdp_fwd_window.restype = i
        L.sdp_fwd_varlen_window.argtypes = [vp] * 7 + [i] * 7 + [f, i, i, i, vp]
        L.sdp_fwd_varlen_window.restype = i
        _declared = L
    return _declared


def _no_grad(*tensors) -> None:
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError("forward only: detach the inputs or run under torch.no_grad()")


def _empty(shape, dtype, dev: int, stream) -> torch.Tensor:
    """A new tensor that work on `stream` may write at once: from that stream's own pool (a block of
    the current stream's pool could still be in use there), and safe to free from the current one."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev) if stream else torch.cuda.default_stream(dev)
    now = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    t.record_stream(now)
    return t


def _outputs(q, out, lse, return_lse, lse_shape, dev: int, stream):
    """The output buffers of an attention call: given ones checked, others allocated."""
    if out is None:
        out = _empty(q.shape, q.dtype, dev, stream)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError("out must be a contiguous tensor shaped and typed like q")
    if lse is None:
        if return_lse:
            lse = _empty(lse_shape, torch.float32, dev, stream)
    elif (tuple(lse.shape) != tuple(lse_shape) or lse.dtype != torch.float32 or not lse.is_contiguous()
          or lse.get_device() != dev):
        raise ValueError(f"lse must be a contiguous float32 tensor {tuple(lse_shape)} on q's device")
    return out, lse


# ------------------------------------------------------------------ positions


def rope_inv_freq(dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                  original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Rotation frequencies (rad per position) of `dim` channels as float64 [dim / 2]: base ** (-2 i / dim).

    For contexts `factor` times as long as the model was trained on, `scaling` is one of
    "linear" (every frequency divided by factor), "ntk" (the base raised so that the lowest
    frequency is divided by factor and the highest kept) or "yarn" (frequencies that turn more than
    beta_fast times in original_length kept, those below beta_slow turns divided by factor, a
    linear ramp over the channel index between; its attention factor 0.1 ln(factor) + 1 is the
    table's mscale, see rope_table).
    """
    if dim < 0 or dim % 2:
        raise ValueError("dim must be even")
    if not (base > 0 and factor >= 1):
        raise ValueError("base must be positive and factor at least 1")
    i = torch.arange(dim // 2, dtype=torch.float64, device=device)
    if scaling == "ntk" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    f = torch.exp(-math.log(base) * 2 * i / max(dim, 1))
    if scaling == "linear":
        return f / factor
    if scaling == "yarn":
        if original_length <= 0:
            raise ValueError("yarn scaling needs original_length")

        def index(turns):  # channel pair that turns that many times in original_length
            return dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        low, high = max(0, math.floor(index(beta_fast))), min(dim // 2 - 1, math.ceil(index(beta_slow)))
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp
    if scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f


class RopeTable(NamedTuple):
    """Frequencies laid out for qk_norm_rope: turns per position as 64-bit binary fractions (int64
    [rot_dim / 2] on the device), and the factor of the rotated channels."""
    turns: torch.Tensor
    mscale: float


def rope_table(inv_freq: torch.Tensor, mscale: float = 1.0, device=None) -> RopeTable:
    """The table of frequencies `inv_freq` (rad per position, float64 for far positions), made once.

    Nothing is synchronised when inv_freq is on the device already.
    """
    if inv_freq.dim() != 1 or not inv_freq.is_floating_point():
        raise ValueError("inv_freq must be a 1-D floating-point tensor")
    t = inv_freq.detach().to(device=inv_freq.device if device is None else device, dtype=torch.float64)
    t = t / (2 * math.pi)
    t = t - torch.floor(t)
    high = torch.floor(t * 2.0 ** 32)
    low = torch.floor((t * 2.0 ** 32 - high) * 2.0 ** 32)
    return RopeTable(((high.to(torch.int64) << 32) | low.to(torch.int64)).contiguous(), float(mscale))


def _rows4(t: torch.Tensor, packed: bool):
    """(batch, token, head) strides and sizes of [T, H, D] or [B, H, S, D]."""
    s = t.stride()
    if packed:
        return (0, s[0], s[1]), (1, t.shape[0], t.shape[1])
    return (s[0], s[2], s[1]), (t.shape[0], t.shape[2], t.shape[1])


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor | None,
                 table: RopeTable | None, q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                 eps: float = 1e-6, interleaved: bool = False, q_out: torch.Tensor | None = None,
                 k_out: torch.Tensor | None = None, stream=None):
    """RMS norm of every head's row (where it has a weight), then the rotation by position, in one pass.

    q: [T, Hq, D] or [B, Hq, S, D]; k alike with Hkv heads, or None; fp16 or bf16 on one CUDA
    device, D in {128, 256}; strides of the leading dimensions are free (views of a fused
    projection need no copy), the last dimension is contiguous. The results are contiguous tensors
    of the same shape (what sdp_fwd and sdp_fwd_varlen take) unless q_out / k_out are given, which
    may be q and k themselves. positions: int32 or int64, [T], or [S] or [B, S]; any value. table:
    rope_table's, rotating the first 2 * len(table.turns) channels (a multiple of 16), or None for
    norms only; interleaved pairs channels (2i, 2i+1), else (i, i + half). Weights: [D] of q's dtype or
    float32. Enqueued on `stream` (default: the current stream), not synchronised.
    """
    packed = q.dim() == 3
    if not packed and q.dim() != 4:
        raise ValueError("q must be [T, H, D] or [B, H, S, D]")
    dev = q.get_device()
    dt = _DTYPE_CODE.get(q.dtype)
    if dev < 0 or dt is None:
        raise ValueError("q must be a float16 or bfloat16 CUDA tensor")
    _no_grad(q, k, q_weight, k_weight)
    D = q.shape[-1]
    (qb, qs, qh), (B, S, Hq) = _rows4(q, packed)
    if q.stride(-1) != 1:
        raise ValueError("the last dimension of q must be contiguous")
    if q_out is None:
        q_out = _empty(q.shape, q.dtype, dev, stream)
    elif q_out.shape != q.shape or q_out.dtype != q.dtype or q_out.get_device() != dev or q_out.stride(-1) != 1:
        raise ValueError("q_out must be shaped and typed like q, its last dimension contiguous")
    (ob, os_, oh), _ = _rows4(q_out, packed)
    kb = ks = kh = pb_ = ps_ = ph_ = Hkv = kp = kop = 0
    if k is not None:
        if k.dim() != q.dim() or k.dtype != q.dtype or k.get_device() != dev or k.shape[-1] != D or k.stride(-1) != 1:
            raise ValueError("k must have q's dimensions, dtype, device and head dim, its last dimension contiguous")
        (kb, ks, kh), (Bk, Sk, Hkv) = _rows4(k, packed)
        if (Bk, Sk) != (B, S):
            raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}")
        if k_out is None:
            k_out = _empty(k.shape, k.dtype, dev, stream)
        elif k_out.shape != k.shape or k_out.dtype != k.dtype or k_out.get_device() != dev or k_out.stride(-1) != 1:
            raise ValueError("k_out must be shaped and typed like k, its last dimension contiguous")
        (pb_, ps_, ph_), _ = _rows4(k_out, packed)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need k")
    R = 0
    turns = pos = sb = ss = wide = 0
    mscale = 1.0
    if table is not None:
        R = 2 * table.turns.numel()
        mscale = table.mscale
        if table.turns.get_device() != dev or table.turns.dtype != torch.int64 or not table.turns.is_contiguous():
            raise ValueError("table must be rope_table's, on q's device")
        if positions is None or positions.get_device() != dev or positions.dtype not in (torch.int32, torch.int64):
            raise ValueError("positions must be an int32 or int64 tensor on q's device")
        if positions.dim() == 1 and positions.shape[0] == S:
            ss = positions.stride(0)
        elif not packed and positions.dim() == 2 and tuple(positions.shape) == (B, S):
            sb, ss = positions.stride()
        else:
            raise ValueError("positions must be [T], or [S] or [B, S]")
        turns, pos, wide = table.turns.data_ptr(), positions.data_ptr(), positions.dtype == torch.int64
    wt = None
    for w in (q_weight, k_weight):
        if w is not None:
            if w.shape != (D,) or not w.is_contiguous() or w.get_device() != dev or w.dtype not in (q.dtype, torch.float32):
                raise ValueError("weights must be contiguous [D] tensors of q's dtype or float32 on its device")
            if wt is not None and w.dtype != wt:
                raise ValueError("both weights must have one dtype")
            wt = w.dtype
    with _on(dev):
        rc = _lib().sdp_qk_norm_rope(
            q.data_ptr(), qb, qs, qh, kp, kb, ks, kh, q_out.data_ptr(), ob, os_, oh, kop, pb_, ps_, ph_, pos, sb, ss,
            wide, turns, R, mscale, 0 if q_weight is None else q_weight.data_ptr(),
            0 if k_weight is None else k_weight.data_ptr(), wt == torch.float32, eps, interleaved, B, S, Hq, Hkv, D, dt,
            _stream_handle(stream, dev))
    if rc != SDP_OK:
        _check(rc)
    return q_out, k_out


# ------------------------------------------------------------------ the 4-bit paged cache


class Cache4(NamedTuple):
    """A pool of pages that hold keys and values in 4 bits (4.5 with their scales).

    codes: uint8 [num_pages, Hkv, page_size, D / 2], the lower channel in a byte's low half;
    scales: bfloat16 [num_pages, Hkv, page_size, D / 64, 2], scale and bias of 64 channels: code n
    stands for scale * n + bias. page_size is a multiple of 16. All contiguous on one device.
    """
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


def cache4_empty(num_pages: int, Hkv: int, D: int, page_size: int = 64, device="cuda") -> Cache4:
    """A pool of zeroed pages."""
    if D not in (128, 256) or page_size <= 0 or page_size % 16 or num_pages <= 0 or Hkv <= 0:
        raise ValueError("D must be 128 or 256, page_size a multiple of 16, sizes positive")
    shape = (num_pages, Hkv, page_size)

    def codes():
        return torch.zeros(*shape, D // 2, dtype=torch.uint8, device=device)

    def scales():
        return torch.zeros(*shape, D // CACHE4_GROUP, 2, dtype=torch.bfloat16, device=device)

    return Cache4(codes(), scales(), codes(), scales())


def _pool(cache: Cache4, block_table: torch.Tensor, dev: int):
    """The pool's arguments of a C call, and (nseq, Hkv, D)."""
    kc, ks, vc, vs = cache
    shape = kc.shape
    if len(shape) != 4 or kc.dtype != torch.uint8 or vc.dtype != torch.uint8 or vc.shape != shape:
        raise ValueError("codes must be uint8 [num_pages, Hkv, page_size, D / 2]")
    P, Hkv, page, half = shape
    want = (P, Hkv, page, half // (CACHE4_GROUP // 2), 2)
    if ks.shape != want or vs.shape != want or ks.dtype != torch.bfloat16 or vs.dtype != torch.bfloat16:
        raise ValueError("scales must be bfloat16 [num_pages, Hkv, page_size, D / 64, 2]")
    if not (kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous()):
        raise ValueError("the cache must be contiguous")
    if block_table.dim() != 2 or block_table.dtype != torch.int32 or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be int32 [nseq, max_pages], its last dimension contiguous")
    for t in (kc, ks, vc, vs, block_table):
        if t.get_device() != dev:
            raise ValueError("the cache and the block table must be on the inputs' device")
    nseq, max_pages = block_table.shape
    return ((kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), P, page, block_table.data_ptr(),
             block_table.stride(0), max_pages), nseq, Hkv, 2 * half)


def _int32(name: str, t: torch.Tensor, n: int, dev: int) -> int:
    if t.dim() != 1 or t.shape[0] != n or t.dtype != torch.int32 or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous int32 tensor [{n}] on the inputs' device")
    return t.data_ptr()


def cache4_append(cache: Cache4, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, cache_lens: torch.Tensor,
                  block_table: torch.Tensor, stream=None) -> None:
    """Quantises new rows into the cache.

    k, v: [tokens, Hkv, D] fp16 or bf16 (free token and head strides): rows cu_seqlens[i] ..
    cu_seqlens[i + 1] - 1 become the last tokens of sequence i, whose length with them is
    cache_lens[i]; token t goes to place t % page_size of page block_table[i, t // page_size].
    cu_seqlens, cache_lens: int32 [nseq + 1] and [nseq] on the device. Pages that sequences share
    must not be written. Bad offsets, lengths and pages are skipped and show in poll_status().
    """
    dev = k.get_device()
    dt = _DTYPE_CODE.get(k.dtype)
    if dev < 0 or dt is None or v.dtype != k.dtype or v.get_device() != dev:
        raise ValueError("k and v must be CUDA tensors on one device of one dtype, float16 or bfloat16")
    _no_grad(k, v)
    pool, nseq, Hkv, D = _pool(cache, block_table, dev)
    if k.dim() != 3 or v.shape != k.shape or k.shape[1] != Hkv or k.shape[2] != D:
        raise ValueError(f"k and v must be [tokens, {Hkv}, {D}]")
    if k.stride(2) != 1 or v.stride(2) != 1:
        raise ValueError("the last dimension of k and v must be contiguous")
    cu, lens = _int32("cu_seqlens", cu_seqlens, nseq + 1, dev), _int32("cache_lens", cache_lens, nseq, dev)
    with _on(dev):
        rc = _lib().sdp_cache4_append(*pool, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
                                      v.stride(1), cu, lens, nseq, k.shape[0], Hkv, D, dt, _stream_handle(stream, dev))
    if rc != SDP_OK:
        _check(rc)


def cache4_gather(cache: Cache4, cu_seqlens: torch.Tensor, block_table: torch.Tensor, total: int,
                  dtype: torch.dtype = torch.bfloat16, k_out: torch.Tensor | None = None,
                  v_out: torch.Tensor | None = None, stream=None):
    """Reads sequences back as packed 16-bit rows for the varlen attention calls.

    Rows cu_seqlens[i] .. cu_seqlens[i + 1] - 1 of the returned (k, v), each [total, Hkv, D] of
    `dtype`, are tokens 0, 1, ... of sequence i; rows in no sequence are not written (total is
    cu_seqlens[-1] in plain use). k_out, v_out: buffers to write instead, with free token and head strides.
    """
    dev = cache.k_codes.get_device()
    dt = _DTYPE_CODE.get(dtype)
    if dev < 0 or dt is None:
        raise ValueError("the cache must be on a CUDA device, dtype float16 or bfloat16")
    pool, nseq, Hkv, D = _pool(cache, block_table, dev)
    shape = (int(total), Hkv, D)
    if k_out is None:
        k_out = _empty(shape, dtype, dev, stream)
    if v_out is None:
        v_out = _empty(shape, dtype, dev, stream)
    for t in (k_out, v_out):
        if t.shape != shape or t.dtype != dtype or t.get_device() != dev or t.stride(2) != 1:
            raise ValueError(f"k_out and v_out must be {shape} of dtype, the last dimension contiguous")
    cu = _int32("cu_seqlens", cu_seqlens, nseq + 1, dev)
    with _on(dev):
        rc = _lib().sdp_cache4_gather(*pool, k_out.data_ptr(), k_out.stride(0), k_out.stride(1), v_out.data_ptr(),
                                      v_out.stride(0), v_out.stride(1), cu, nseq, shape[0], Hkv, D, dt,
                                      _stream_handle(stream, dev))
    if rc != SDP_OK:
        _check(rc)
    return k_out, v_out


def cache4_workspace_bytes(nseq: int, rows: int, Hq: int, Hkv: int, D: int, dtype: torch.dtype) -> int:
    """Bytes of workspace that fwd_cache4 needs for these sizes on the current device."""
    rc = _lib().sdp_fwd_cache4_workspace_bytes(nseq, rows, Hq, Hkv, D, _DTYPE_CODE[dtype])
    _check(min(rc, 0))
    return rc


def fwd_cache4(q: torch.Tensor, cache: Cache4, cache_lens: torch.Tensor, block_table: torch.Tensor,
               scale: float | None = None, window: int = 0, sinks: int = 0, out: torch.Tensor | None = None,
               lse: torch.Tensor | None = None, return_lse: bool = True, workspace: torch.Tensor | None = None,
               stream=None):
    """Attention of each sequence's last rows over the 4-bit cache (decoding).

    q: [nseq, Hq, D], or [nseq, rows, Hq, D] with up to 32 rows (drafted tokens): row i of sequence s
    is its token cache_lens[s] - rows + i and sees the keys up to itself, already in the cache; with
    window > 0 only the last `window` of them and the sequence's first `sinks`. Contiguous, fp16 or
    bf16. cache_lens: int32 [nseq]; block_table: int32 [nseq, max_pages]. Returns (o like q, lse fp32
    without the last dimension, or None); a row that sees no key gives 0 and -inf.

    workspace: a contiguous CUDA tensor of cache4_workspace_bytes, not used by another call that may
    overlap; when None it comes from torch's allocator. Enqueued on `stream` (default: the current
    stream), not synchronised; bad lengths and pages show in poll_status().
    """
    shape = q.shape
    if len(shape) == 3:
        nseq, Hq, D = shape
        rows = 1
    elif len(shape) == 4:
        nseq, rows, Hq, D = shape
    else:
        raise ValueError("q must be [nseq, Hq, D] or [nseq, rows, Hq, D]")
    dev = q.get_device()
    dt = _DTYPE_CODE.get(q.dtype)
    if dev < 0 or dt is None or not q.is_contiguous():
        raise ValueError("q must be a contiguous float16 or bfloat16 CUDA tensor")
    _no_grad(q)
    pool, ns, Hkv, Dc = _pool(cache, block_table, dev)
    if ns != nseq or Dc != D:
        raise ValueError(f"shape mismatch: q {tuple(shape)}, {ns} sequences of head dim {Dc} in the cache")
    lens = _int32("cache_lens", cache_lens, nseq, dev)
    out, lse = _outputs(q, out, lse, return_lse, shape[:-1], dev, stream)
    if nseq == 0 or rows == 0:
        return out, lse
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _on(dev):
        if workspace is None:
            need = _lib().sdp_fwd_cache4_workspace_bytes(nseq, rows, Hq, Hkv, D, dt)
            _check(min(need, 0))
            workspace = _empty((need,), torch.uint8, dev, stream)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on q's device")
        rc = _lib().sdp_fwd_cache4(
            q.data_ptr(), *pool, lens, out.data_ptr(), 0 if lse is None else lse.data_ptr(), nseq, rows, Hq, Hkv, D,
            scale, dt, window, sinks, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _stream_handle(stream, dev))
    if rc != SDP_OK:
        _check(rc)
    return out, lse


# ------------------------------------------------------------------ sliding windows


def fwd_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int, sinks: int = 0,
               scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               return_lse: bool = True, stream=None):
    """Causal attention over the last `window` keys and the first `sinks`.

    q: [B, Hq, Sq, D]; k, v: [B, Hkv, Skv, D], contiguous, as sdp_fwd. Row i is at position
    p = Skv - Sq + i and sees keys j <= p with j > p - window or j < sinks. Returns (o like q, lse
    fp32 [B, Hq, Sq] or None); a row that sees no key gives 0 and -inf. Enqueued on `stream`
    (default: the current stream), not synchronised.
    """
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, H, S, D]")
    dev = q.get_device()
    dt = _DTYPE_CODE.get(q.dtype)
    if dev < 0 or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("q, k, v must be CUDA tensors on one device")
    if dt is None or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share one dtype, float16 or bfloat16")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("q, k, v must be contiguous")
    _no_grad(q, k, v)
    B, Hq, Sq, D = q.shape
    kshape = k.shape
    if kshape[0] != B or kshape[3] != D or v.shape != kshape:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    out, lse = _outputs(q, out, lse, return_lse, (B, Hq, Sq), dev, stream)
    with _on(dev):
        rc = _lib().sdp_fwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                   0 if lse is None else lse.data_ptr(), B, Hq, kshape[1], Sq, kshape[2], D,
                                   1.0 / math.sqrt(D) if scale is None else scale, dt, window, sinks,
                                   _stream_handle(stream, dev))
    if rc != SDP_OK:
        _check(rc)
    return out, lse


def fwd_varlen_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                      cu_seqlens_k: torch.Tensor, max_seqlen_q: int, window: int, sinks: int = 0,
                      scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      return_lse: bool = True, stream=None):
    """fwd_window over a variable-length batch packed back to back.

    q: [total_q, Hq, D]; k, v: [total_k, Hkv, D], contiguous; cu_seqlens_q, cu_seqlens_k: int32
    [nseq + 1] offsets on the device; max_seqlen_q: a host int >= every query length, as
    sdp_fwd_varlen. A sequence's query rows are its last positions. Returns (o like q, lse fp32
    [Hq, total_q] or None). Bad offsets show in poll_status().
    """
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be 3-D [tokens, heads, D]")
    dev = q.get_device()
    dt = _DTYPE_CODE.get(q.dtype)
    if dev < 0 or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("q, k, v must be CUDA tensors on one device")
    if dt is None or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share one dtype, float16 or bfloat16")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("q, k, v must be contiguous")
    _no_grad(q, k, v)
    total_q, Hq, D = q.shape
    kshape = k.shape
    if kshape[2] != D or v.shape != kshape:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    n = cu_seqlens_q.shape[0] if cu_seqlens_q.dim() == 1 else 0
    if n < 2:
        raise ValueError("sequence offsets must be 1-D [nseq + 1]")
    cu_q, cu_k = _int32("cu_seqlens_q", cu_seqlens_q, n, dev), _int32("cu_seqlens_k", cu_seqlens_k, n, dev)
    out, lse = _outputs(q, out, lse, return_lse, (Hq, total_q), dev, stream)
    with _on(dev):
        rc = _lib().sdp_fwd_varlen_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                          0 if lse is None else lse.data_ptr(), cu_q, cu_k, n - 1, Hq, kshape[1],
                                          total_q, kshape[0], max_seqlen_q, D,
                                          1.0 / math.sqrt(D) if scale is None else scale, dt, window, sinks,
                                          _stream_handle(stream, dev))
    if rc != SDP_OK:
        _check(rc)
    return out, lse
