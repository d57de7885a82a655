"""The operators around the attention forward on a serving path.

``qk_norm_rope``: norms and position rotation of the query and key heads in one pass, with
``rope_inv_freq`` and ``rope_table`` for its frequencies. ``Cache4``: a paged cache held in 4 bits,
written by ``cache4_append`` and read back by ``cache4_gather``; ``fwd_cache4``: the attention of each
sequence's last tokens over it. ``fwd_window`` and ``fwd_varlen_window``: prefill attention with a sliding
window and first tokens that stay visible.

The work runs in libsdp.so (``include/sdp.h`` states layouts, ownership and errors); PyTorch supplies
memory and streams, and there is no fallback. Arguments are checked, outputs made and the C calls
issued by ``_serving.*.so`` (binding/binding.cpp), built beside the library: a decode step's kernels take
a few microseconds, less than checking their arguments in Python does. These functions compute
forward passes only: a tensor that requires grad is refused while grad mode is on.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
import re
import sysconfig
from typing import NamedTuple

import torch

from . import LIB_PATH, SDP_OK, _check, _DTYPE_CODE, lib

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


def _binding_path(torch_version: str) -> str:
    """The binding built for this Python and that torch. Its name carries both, so that one built for others (before an
    upgrade, or in another environment over the same files) is never loaded: their C++ layouts differ."""
    tag = f"{sysconfig.get_config_var('SOABI')}-torch{torch_version}"
    return os.path.join(os.path.dirname(LIB_PATH), "_serving." + re.sub(r"[^A-Za-z0-9_.+-]", "_", tag) + ".so")


BINDING_PATH = _binding_path(torch.__version__)


class _Binding:
    """The compiled binding's functions, loaded by the first call."""

    def __getattr__(self, name):
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"{BINDING_PATH} is not built: run `python -m gqa_flash_attention_gb300.build` "
                               "(there is no fallback path)")
        lib()
        spec = importlib.util.spec_from_file_location("_serving", BINDING_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        for f in ("qk_norm_rope", "cache4_append", "cache4_gather", "fwd_cache4", "fwd_window", "fwd_varlen_window"):
            setattr(self, f, getattr(module, f))
        return self.__dict__[name]


_binding = _Binding()


# ------------------------------------------------------------------ positions


def rope_inv_freq(dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                  original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Rotation frequencies (rad per position) of `dim` channels as float64 [dim / 2]: base ** (-2 i / dim).

    For contexts `factor` times as long as the model was trained on, `scaling` is one of
    "linear" (every frequency divided by factor), "ntk" (the base raised so that the lowest
    frequency is divided by factor and the highest kept) or "yarn" (frequencies that turn more than
    beta_fast times in original_length kept, those below beta_slow turns divided by factor, a
    linear ramp over the channel index between, its ends rounded outwards to whole pairs; its
    attention factor 0.1 ln(factor) + 1 is the table's mscale, see rope_table).
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

        # the upper end may lie past the last pair, which then is not divided in full
        low, high = max(0, math.floor(index(beta_fast))), min(dim - 1, math.ceil(index(beta_slow)))
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
    rc, q_out, k_out = _binding.qk_norm_rope(q, k, positions, table, q_weight, k_weight, eps, interleaved, q_out, k_out,
                                             stream)
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


def cache4_append(cache: Cache4, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, cache_lens: torch.Tensor,
                  block_table: torch.Tensor, stream=None) -> None:
    """Quantises new rows into the cache.

    k, v: [tokens, Hkv, D] fp16 or bf16 (free token and head strides): rows cu_seqlens[i] ..
    cu_seqlens[i + 1] - 1 become the last tokens of sequence i, whose length with them is
    cache_lens[i]; token t goes to place t % page_size of page block_table[i, t // page_size].
    cu_seqlens, cache_lens: int32 [nseq + 1] and [nseq] on the device. Pages that sequences share
    must not be written. Bad offsets, lengths and pages are skipped and show in poll_status(); a batch
    of no sequences writes nothing.
    """
    rc, = _binding.cache4_append(cache, k, v, cu_seqlens, cache_lens, block_table, stream)
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
    if dtype not in _DTYPE_CODE:
        raise ValueError("dtype must be float16 or bfloat16")
    rc, k_out, v_out = _binding.cache4_gather(cache, cu_seqlens, block_table, total, dtype is torch.bfloat16, k_out, v_out,
                                              stream)
    if rc != SDP_OK:
        _check(rc)
    return k_out, v_out


def cache4_workspace_bytes(nseq: int, rows: int, Hq: int, Hkv: int, D: int, dtype: torch.dtype) -> int:
    """Bytes of workspace that fwd_cache4 needs for these sizes on the current device."""
    if dtype not in _DTYPE_CODE:
        raise ValueError("dtype must be float16 or bfloat16")
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
    bf16. cache_lens: int32 [nseq]; block_table: int32 [nseq, max_pages], of which only entries of pages
    that some row sees are read. Returns (o like q, lse fp32
    without the last dimension, or None); a row that sees no key gives 0 and -inf. The cache is read once
    for each 16 of a KV head's (Hq / Hkv) * rows columns.

    workspace: a contiguous CUDA tensor of cache4_workspace_bytes, not used by another call that may
    overlap; when None it comes from torch's allocator. Enqueued on `stream` (default: the current
    stream), not synchronised; bad lengths and pages show in poll_status().
    """
    rc, out, lse = _binding.fwd_cache4(q, cache, cache_lens, block_table, scale, window, sinks, out, lse, return_lse,
                                       workspace, stream)
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
    rc, out, lse = _binding.fwd_window(q, k, v, window, sinks, scale, out, lse, return_lse, stream)
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
    rc, out, lse = _binding.fwd_varlen_window(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, window, sinks, scale, out,
                                              lse, return_lse, stream)
    if rc != SDP_OK:
        _check(rc)
    return out, lse
