"""libsconv: causal depthwise short convolution on MI355X (gfx950).

Thin Python binding over the C ABI declared in include/sconv.h.  It only
marshals torch tensors into device pointers, element strides and the current
HIP stream; every step of the computation runs in the library's HIP kernels.
There is no fallback: if libsconv.so is missing or a call is rejected, the
binding raises.

Entry points (same names as the C ABI):
  conv1d_fwd_varlen    -- varlen prefill with per-sequence conv state
  conv1d_update_decode -- decode update (state shift), in place allowed
  conv1d_update        -- decode update with speculative-decoding and
                          ring-buffer options
  sconv_paged_fused    -- paged sliding-window cache insert + conv
  sconv_paged_fused_multi -- several conv streams sharing one paged cache
  sconv_seq_metadata   -- per-token (request, first row) buffers
  gdr_fwd_varlen       -- the gated delta rule over a packed varlen batch
  gdr_update           -- its decode update, with the speculative options
  sconv_verify_drafts  -- which drafted tokens stand (num_accepted_tokens)
  ssm_fwd_varlen       -- the selective state space scan over a packed varlen batch
  ssm_update           -- its decode update, with the speculative options
  sconv_group_norm     -- the norm of channel groups, with a gate or activation
bind_fwd_varlen and bind_update_decode marshal a forward or a decode step
once for repeated launches.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

__all__ = ["conv1d_fwd_varlen", "conv1d_update_decode", "conv1d_update", "sconv_paged_fused",
           "sconv_paged_fused_multi", "sconv_seq_metadata", "new_output", "bind_fwd_varlen",
           "bind_update_decode", "gdr_fwd_varlen", "gdr_update", "sconv_verify_drafts",
           "ssm_fwd_varlen", "ssm_update", "sconv_group_norm",
           "SconvError", "library_path", "load_library", "exported_symbols",
           "version", "status_string"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libsconv.so")
_lib = None
_packed = {}              # calls of many arguments: how to pack them, and the entry that takes them so

ACT_NONE, ACT_SILU = 0, 1


class SconvError(RuntimeError):
    """A libsconv call returned a non-zero status."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


def library_path() -> str:
    return _LIB_PATH


def load_library(path: str | None = None):
    """Load libsconv.so (built by causal_depthwise_short_conv1d_amd.build).
    Raises FileNotFoundError when it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise FileNotFoundError(
            f"libsconv not built: {p} is missing "
            "(run python -m causal_depthwise_short_conv1d_amd.build)")
    lib = ctypes.CDLL(p)
    P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    lib.sconv_status_string.argtypes = [ctypes.c_int]
    lib.sconv_status_string.restype = ctypes.c_char_p
    lib.sconv_version.argtypes = []
    lib.sconv_version.restype = ctypes.c_int
    lib.conv1d_fwd_varlen.argtypes = [
        P, I64, I64, P, I64, P, P, I64, I64, I64, I64, P, P, P,
        I32, I64, I32, I32, I32, I32, P, I64, I64, P]
    lib.conv1d_update_decode.argtypes = [
        P, I64, I64, I64, P, I64, P, P, I64, I64, I64, I64, P,
        I32, I32, I32, I32, I32, I32, P, I64, I64, I64, P]
    lib.conv1d_update.argtypes = [
        P, I64, I64, I64, P, I64, P, P, I64, I64, I64, I64, I32, P, P, P,
        P, I64, I64, I64, I64, P, I64, I64,
        I32, I32, I32, I32, I32, I32, P, I64, I64, I64, P]
    lib.sconv_paged_fused.argtypes = [
        P, I64, P, I64, P, P, I64, I64, I64, I64, I32, I32, I32, I32, I32,
        P, P, P, I32, P, I64, I32, I64, I32, I32, I32, P, I64, P]
    lib.sconv_seq_metadata.argtypes = [P, I32, I64, I64, P, I64, P, I64, P]
    lib.sconv_paged_fused_multi.argtypes = [
        I32, P, P, P, P, P, P, P, P, P, P, I64, I64, I64, I64, I32, I32, I32,
        P, P, P, I32, P, I64, I32, I64, I32, I32, I32, P]
    F32 = ctypes.c_float
    lib.gdr_fwd_varlen.argtypes = [
        *([P, I64, I64, I64] * 3), *([P, I64, I64] * 2), P, P, P, I64, I64, I64, I64, I64,
        P, P, P, I32, I64, I32, I32, I32, I32, F32, I32, I32, P, I64, I64, I64, P, I64, P]
    lib.gdr_fwd_workspace_bytes.argtypes = [I32, I64, I32, I32, I32, I32, I32]
    lib.gdr_fwd_workspace_bytes.restype = I64
    lib.gdr_update.argtypes = [
        *([P, I64, I64, I64, I64] * 3), *([P, I64, I64, I64] * 2), P, P, P, I64, I64, I64, I64, I64,
        P, I64, I64, I32, P, P, I64, I64, I32, I32, I32, I32, I32, I32, F32, I32, I32,
        P, I64, I64, I64, I64, P]
    lib.ssm_fwd_varlen.argtypes = [
        *([P, I64, I64, I64] * 2), I32, *([P, I64, I64, I64] * 3), P, I64, I64, P, I64, I64, I64, P, I64, I64, I32, F32, F32,
        P, I64, I64, I64, I64, I64, P, P, P, I32, I64, I32, I32, I32, I32, I32, P, I64, I64, I64, P, I64, P]
    lib.ssm_update.argtypes = [
        *([P, I64, I64, I64, I64] * 2), I32, P, I64, I64, I64, *([P, I64, I64, I64, I64] * 2), P, I64, I64,
        P, I64, I64, I64, I64, P, I64, I64, I32, F32, F32, P, I64, I64, I64, I64, I64, P, I64, I64, I32, P, P, I64, I64,
        I32, I32, I32, I32, I32, I32, I32, P, I64, I64, I64, I64, P]
    lib.ssm_fwd_workspace_bytes.argtypes = [I32, I64, I32, I32, I32, I32, I32]
    lib.ssm_fwd_workspace_bytes.restype = I64
    packed = {}
    for f in (lib.gdr_fwd_varlen, lib.gdr_update, lib.ssm_fwd_varlen, lib.ssm_update):
        words = getattr(lib, f.__name__ + "_packed")
        words.argtypes, words.restype = [ctypes.c_char_p], ctypes.c_int
        # the words of a call as bytes: a float is the low half of its word
        pack = struct.Struct("<" + "".join("f4x" if t is F32 else "q" for t in f.argtypes)).pack
        packed[f.__name__] = (pack, words)
    lib.sconv_verify_drafts.argtypes = [
        P, P, P, I64, P, I64, P, P, I32, I32, I32, I32, P, I64, P, P, I64, P]
    lib.sconv_verify_workspace_bytes.argtypes = [I32, I32]
    lib.sconv_verify_workspace_bytes.restype = I64
    lib.sconv_group_norm.argtypes = [
        *([P, I64, I64, I64] * 2), P, I64, P, I64, I32, I64, I32, I32, I32, I32, I32, F32, P, I64, I64, I64, P]
    for f in (lib.conv1d_fwd_varlen, lib.conv1d_update_decode, lib.conv1d_update,
              lib.sconv_paged_fused, lib.sconv_paged_fused_multi, lib.sconv_seq_metadata,
              lib.gdr_fwd_varlen, lib.gdr_update, lib.sconv_verify_drafts, lib.ssm_fwd_varlen, lib.ssm_update,
              lib.sconv_group_norm):
        f.restype = ctypes.c_int
    if path is None:
        _packed.update(packed)        # before _lib: another thread's call looks there once it finds the library
        _lib = lib
    return lib


def exported_symbols() -> list[str]:
    return ["sconv_status_string", "sconv_version", "conv1d_fwd_varlen",
            "conv1d_update_decode", "conv1d_update", "sconv_paged_fused",
            "sconv_paged_fused_multi", "sconv_seq_metadata", "gdr_fwd_varlen",
            "gdr_fwd_varlen_packed", "gdr_fwd_workspace_bytes", "gdr_update", "gdr_update_packed",
            "sconv_verify_workspace_bytes", "sconv_verify_drafts", "ssm_fwd_varlen", "ssm_fwd_varlen_packed",
            "ssm_fwd_workspace_bytes",
            "ssm_update", "ssm_update_packed", "sconv_group_norm"]


def version() -> tuple[int, int]:
    v = load_library().sconv_version()
    return v >> 16, v & 0xFFFF


def status_string(status: int) -> str:
    try:
        return load_library().sconv_status_string(int(status)).decode()
    except FileNotFoundError:
        return "unknown"


# ------------------------------------------------------------ marshalling --

def _dev(t: torch.Tensor | None, dtype: torch.dtype, name: str, device=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    return ctypes.c_void_p(t.data_ptr()) if t.numel() else None


def _index(t, dtype, name, device, n=None):
    p = _dev(t, dtype, name, device)
    if t is not None:
        if t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1):
            raise ValueError(f"{name} must be a contiguous 1-D tensor")
        if n is not None and t.numel() < n:
            raise ValueError(f"{name} needs at least {n} entries")
    return p


def _act(activation) -> int:
    if activation is True or activation in ("silu", "swish"):
        return ACT_SILU
    if activation in (None, False):
        return ACT_NONE
    raise ValueError(f"unsupported activation {activation!r}")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> ctypes.c_void_p:
    """The current stream of `device` as a raw handle (torch's accessor when
    it has one: no Stream object per call)."""
    if _raw_stream is not None:
        return ctypes.c_void_p(_raw_stream(device.index if device.index is not None
                                           else torch.cuda.current_device()))
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _call(fn: str, *args) -> None:
    rc = getattr(load_library(), fn)(*args)
    if rc != 0:
        raise SconvError(fn, rc)


def _launch(fn: str, dev, args) -> None:
    """Call `fn` with the current stream of `dev` appended, with `dev` made
    the current device for the call (the library launches on the current
    device) unless it already is."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        _call(fn, *args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            _call(fn, *args, _stream(dev))


def _launch_packed(fn: str, dev, args) -> None:
    """_launch for calls of some 50 arguments, which ctypes converts one by one (2.5 us of a call's 12.5): packed into
    words, they are one argument."""
    index = dev.index
    if index is not None and index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _launch_packed(fn, dev, args)
    load_library()
    pack, call = _packed[fn]
    rc = call(pack(*args, _stream(dev).value or 0))
    if rc != 0:
        raise SconvError(fn, rc)


def new_output(x: torch.Tensor) -> torch.Tensor:
    """An uninitialised output in the storage class of x's smaller stride: a
    compact (dim, T) array when tokens are x's closer axis, else (T, pitch)
    storage viewed as (dim, T) with a row pitch rounded up to 8 elements
    (16-byte aligned rows).  Both are layouts the vector kernels take."""
    dim, total = x.shape
    if dim == 1 or (total > 1 and x.stride(1) < x.stride(0)):
        return torch.empty((dim, total), dtype=x.dtype, device=x.device)
    pitch = (dim + 7) // 8 * 8
    return torch.empty((total, pitch), dtype=x.dtype, device=x.device)[:, :dim].t()


def _fwd_varlen_args(x, weight, bias, conv_states, query_start_loc, cache_indices,
                     has_initial_state, activation, pad_slot_id, out):
    """Checked and marshalled arguments of conv1d_fwd_varlen (all but the
    stream), and the output tensor."""
    dev = x.device
    dim, total = x.shape
    width = weight.shape[1]
    batch = query_start_loc.numel() - 1
    if weight.dim() != 2 or weight.shape[0] != dim or weight.stride(1) != 1:
        raise ValueError("weight must be (dim, width) with unit width stride")
    if out is None:
        out = new_output(x)
    if out.shape != x.shape:
        raise ValueError("out must have x's shape")
    if bias is not None and (bias.shape != (dim,) or bias.stride(0) != 1):
        raise ValueError("bias must be a contiguous (dim,) tensor")
    cs = conv_states
    if cs is not None and (cs.dim() != 3 or cs.shape[1] != dim or cs.shape[2] != width - 1):
        raise ValueError("conv_states must be (lines, dim, width-1)")
    bf = torch.bfloat16
    args = (
        _dev(x, bf, "x", dev), x.stride(0), x.stride(1),
        _dev(weight, bf, "weight", dev), weight.stride(0),
        _dev(bias, bf, "bias", dev),
        _dev(cs, bf, "conv_states", dev),
        *(cs.stride() if cs is not None else (0, 0, 0)),
        cs.shape[0] if cs is not None else 0,
        _index(cache_indices, torch.int32, "cache_indices", dev, batch),
        _index(has_initial_state, torch.bool, "has_initial_state", dev, batch),
        _index(query_start_loc, torch.int32, "query_start_loc", dev),
        batch, total, dim, width, _act(activation), pad_slot_id,
        _dev(out, bf, "out", dev), out.stride(0), out.stride(1),
    )
    return args, out


def conv1d_fwd_varlen(x, weight, bias, conv_states, query_start_loc,
                      cache_indices=None, has_initial_state=None,
                      activation="silu", pad_slot_id: int = -1, out=None):
    """Varlen prefill.  x: logical (dim, total_T) bf16 with any strides
    (compact (dim, T) and 16-byte aligned (T, dim) rows take the vector
    kernels); weight (dim, width); bias (dim,) or None; conv_states
    (lines, dim, width-1) or None, updated in place; query_start_loc int32
    (batch+1,); cache_indices int32 (batch,) or None; has_initial_state bool
    (batch,) or None.  Returns out (a new tensor with x's strides unless
    given; see new_output)."""
    args, out = _fwd_varlen_args(x, weight, bias, conv_states, query_start_loc, cache_indices,
                                 has_initial_state, activation, pad_slot_id, out)
    _launch("conv1d_fwd_varlen", x.device, args)
    return out


def bind_fwd_varlen(x, weight, bias, conv_states, query_start_loc, cache_indices=None,
                    has_initial_state=None, activation="silu", pad_slot_id: int = -1,
                    out=None, stream=None):
    """A pre-bound conv1d_fwd_varlen for a caller that runs the same forward
    over and over on fixed buffers (a prefill loop over preallocated
    batches): the tensors are checked and marshalled once, here, and the
    returned function only enqueues the launch on `stream` (default: the
    current stream of x's device now) and raises on a non-zero status.  Its
    `out` attribute is the output tensor.  The tensors must stay alive and
    in place while the function is used."""
    args, out = _fwd_varlen_args(x, weight, bias, conv_states, query_start_loc, cache_indices,
                                 has_initial_state, activation, pad_slot_id, out)
    st = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream(x.device)
    f = load_library().conv1d_fwd_varlen
    full = (*args, st)

    def launch():
        rc = f(*full)
        if rc != 0:
            raise SconvError("conv1d_fwd_varlen", rc)
    launch.out = out
    return launch


def conv1d_update_decode(x, conv_state, weight, bias=None, activation=None,
                         cache_indices=None, pad_slot_id: int = -1, out=None):
    """Decode update.  x: (batch, dim) or (batch, dim, seqlen) bf16;
    conv_state (lines, dim, width-1) updated in place; returns out, which
    may be x itself (pass out=x to compute in place)."""
    dev = x.device
    squeeze = x.dim() == 2
    xv = x.unsqueeze(-1) if squeeze else x
    ov = None
    if out is not None:
        ov = out.unsqueeze(-1) if out.dim() == 2 else out
    else:
        ov = torch.empty_like(xv)
    batch, dim, seqlen = xv.shape
    width = weight.shape[1]
    if weight.dim() != 2 or weight.shape[0] != dim or weight.stride(1) != 1:
        raise ValueError("weight must be (dim, width) with unit width stride")
    if conv_state.dim() != 3 or conv_state.shape[1] != dim or conv_state.shape[2] != width - 1:
        raise ValueError("conv_state must be (lines, dim, width-1)")
    if bias is not None and (bias.shape != (dim,) or bias.stride(0) != 1):
        raise ValueError("bias must be a contiguous (dim,) tensor")
    if ov.shape != xv.shape:
        raise ValueError("out must have x's shape")
    bf = torch.bfloat16
    args = (
        _dev(xv, bf, "x", dev), *xv.stride(),
        _dev(weight, bf, "weight", dev), weight.stride(0),
        _dev(bias, bf, "bias", dev),
        _dev(conv_state, bf, "conv_state", dev), *conv_state.stride(), conv_state.shape[0],
        _index(cache_indices, torch.int32, "cache_indices", dev, batch),
        batch, dim, seqlen, width, _act(activation), pad_slot_id,
        _dev(ov, bf, "out", dev), *ov.stride(),
    )
    _launch("conv1d_update_decode", dev, args)
    if out is not None:
        return out
    return ov.squeeze(-1) if squeeze else ov


def bind_update_decode(x, conv_state, weight, bias=None, activation=None, cache_indices=None,
                       pad_slot_id: int = -1, out=None, stream=None):
    """A pre-bound conv1d_update_decode for a caller that launches the same
    decode step over and over on fixed buffers (a serving loop): the tensors
    are checked and marshalled once, here, and the returned function only
    enqueues the launch on `stream` (default: the current stream of x's
    device now) and raises on a non-zero status.  out=None computes in
    place (x is overwritten, as the page's update does).  The tensors must
    stay alive and in place while the function is used."""
    dev = x.device
    squeeze = x.dim() == 2
    xv = x.unsqueeze(-1) if squeeze else x
    ov = xv if out is None else (out.unsqueeze(-1) if out.dim() == 2 else out)
    batch, dim, seqlen = xv.shape
    width = weight.shape[1]
    if weight.dim() != 2 or weight.shape[0] != dim or weight.stride(1) != 1:
        raise ValueError("weight must be (dim, width) with unit width stride")
    if conv_state.dim() != 3 or conv_state.shape[1] != dim or conv_state.shape[2] != width - 1:
        raise ValueError("conv_state must be (lines, dim, width-1)")
    if bias is not None and (bias.shape != (dim,) or bias.stride(0) != 1):
        raise ValueError("bias must be a contiguous (dim,) tensor")
    if ov.shape != xv.shape:
        raise ValueError("out must have x's shape")
    bf = torch.bfloat16
    st = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream(dev)
    args = (
        _dev(xv, bf, "x", dev), *xv.stride(),
        _dev(weight, bf, "weight", dev), weight.stride(0),
        _dev(bias, bf, "bias", dev),
        _dev(conv_state, bf, "conv_state", dev), *conv_state.stride(), conv_state.shape[0],
        _index(cache_indices, torch.int32, "cache_indices", dev, batch),
        batch, dim, seqlen, width, _act(activation), pad_slot_id,
        _dev(ov, bf, "out", dev), *ov.stride(), st,
    )
    f = load_library().conv1d_update_decode

    def launch():
        rc = f(*args)
        if rc != 0:
            raise SconvError("conv1d_update_decode", rc)
    return launch


def conv1d_update(x, conv_state, weight, bias=None, activation=None, cache_indices=None,
                  cache_seqlens=None, num_accepted_tokens=None, intermediate=None,
                  output_state_indices=None, pad_slot_id: int = -1, out=None):
    """Decode update with the speculative-decoding options
    (num_accepted_tokens (batch,) int32; intermediate (batch, steps, dim,
    width-1) bf16; output_state_indices (batch, seqlen) int32) or ring-buffer
    states (cache_seqlens (batch,) int32).  x: (batch, dim) or
    (batch, dim, seqlen) bf16; conv_state (lines, dim, state_len) bf16,
    state_len >= width-1.  Returns out, which may be x itself."""
    dev = x.device
    squeeze = x.dim() == 2
    xv = x.unsqueeze(-1) if squeeze else x
    if out is not None:
        ov = out.unsqueeze(-1) if out.dim() == 2 else out
    else:
        ov = torch.empty_like(xv)
    batch, dim, seqlen = xv.shape
    width = weight.shape[1]
    if weight.dim() != 2 or weight.shape[0] != dim or weight.stride(1) != 1:
        raise ValueError("weight must be (dim, width) with unit width stride")
    if conv_state.dim() != 3 or conv_state.shape[1] != dim:
        raise ValueError("conv_state must be (lines, dim, state_len)")
    if bias is not None and (bias.shape != (dim,) or bias.stride(0) != 1):
        raise ValueError("bias must be a contiguous (dim,) tensor")
    if ov.shape != xv.shape:
        raise ValueError("out must have x's shape")
    inter = intermediate
    if inter is not None and (inter.dim() != 4 or inter.shape[0] < batch or
                              inter.shape[1] < seqlen or inter.shape[2] != dim or
                              inter.shape[3] != width - 1):
        raise ValueError("intermediate must be (batch, >= seqlen, dim, width-1)")
    osi = output_state_indices
    if osi is not None:
        if osi.dim() != 2 or osi.shape[0] < batch or osi.shape[1] < seqlen:
            raise ValueError("output_state_indices must be (batch, >= seqlen)")
        _dev(osi, torch.int32, "output_state_indices", dev)
    bf = torch.bfloat16
    args = (
        _dev(xv, bf, "x", dev), *xv.stride(),
        _dev(weight, bf, "weight", dev), weight.stride(0),
        _dev(bias, bf, "bias", dev),
        _dev(conv_state, bf, "conv_state", dev), *conv_state.stride(), conv_state.shape[0],
        conv_state.shape[2],
        _index(cache_indices, torch.int32, "cache_indices", dev, batch),
        _index(cache_seqlens, torch.int32, "cache_seqlens", dev, batch),
        _index(num_accepted_tokens, torch.int32, "num_accepted_tokens", dev, batch),
        _dev(inter, bf, "intermediate", dev), *(inter.stride() if inter is not None else (0,) * 4),
        _dev(osi, torch.int32, "output_state_indices", dev),
        *(osi.stride() if osi is not None else (0, 0)),
        batch, dim, seqlen, width, _act(activation), pad_slot_id,
        _dev(ov, bf, "out", dev), *ov.stride(),
    )
    _launch("conv1d_update", dev, args)
    if out is not None:
        return out
    return ov.squeeze(-1) if squeeze else ov


def sconv_paged_fused(x, weight, cache, positions, slot_mapping, query_start_loc,
                      block_table, off_s: int, ws: int, activation=None,
                      use_residual: bool = True, bias=None, out=None):
    """Paged insert + conv.  x (T, H*ws) bf16; weight (H*ws, width); cache
    (num_blocks, H, N, D) bf16 with unit D stride, updated in place;
    positions / slot_mapping int64 (T,); query_start_loc int32 (R+1,);
    block_table int32 (R, max_blocks).  Returns out (T, H*ws)."""
    dev = x.device
    T, C = x.shape
    num_blocks, H, N, D = cache.shape
    width = weight.shape[1]
    num_reqs = query_start_loc.numel() - 1
    if C != H * ws:
        raise ValueError("x's channel count must be cache heads * ws")
    if x.stride(1) != 1 or cache.stride(3) != 1:
        raise ValueError("x channels and cache D must have unit stride")
    if weight.dim() != 2 or weight.shape[0] != C or weight.stride(1) != 1:
        raise ValueError("weight must be (C, width) with unit width stride")
    if bias is not None and (bias.shape != (C,) or bias.stride(0) != 1):
        raise ValueError("bias must be a contiguous (C,) tensor")
    if block_table.dim() != 2 or (block_table.numel() and block_table.stride(1) != 1):
        raise ValueError("block_table must be 2-D with unit column stride")
    if out is None:
        out = torch.empty_like(x)
    if out.shape != x.shape or out.stride(1) != 1:
        raise ValueError("out must be (T, C) with unit channel stride")
    bf = torch.bfloat16
    args = (
        _dev(x, bf, "x", dev), x.stride(0),
        _dev(weight, bf, "weight", dev), weight.stride(0),
        _dev(bias, bf, "bias", dev),
        _dev(cache, bf, "cache", dev), cache.stride(0), cache.stride(1), cache.stride(2),
        num_blocks, H, N, D, off_s, ws,
        _index(positions, torch.int64, "positions", dev, T),
        _index(slot_mapping, torch.int64, "slot_mapping", dev, T),
        _index(query_start_loc, torch.int32, "query_start_loc", dev),
        num_reqs,
        _dev(block_table, torch.int32, "block_table", dev), block_table.stride(0),
        block_table.shape[1],
        T, width, _act(activation), int(bool(use_residual)),
        _dev(out, bf, "out", dev), out.stride(0),
    )
    _launch("sconv_paged_fused", dev, args)
    return out


def sconv_seq_metadata(query_start_loc, num_reqs: int, num_actual_tokens: int,
                       seq_idx_out, query_start_out, num_padded_tokens: int | None = None):
    """Fill seq_idx_out / query_start_out (int32 device tensors) for the
    first num_padded_tokens rows (default num_actual_tokens): owning request
    and its first row for actual rows, 0 / 0 for padded ones."""
    dev = seq_idx_out.device
    for name, t in (("seq_idx_out", seq_idx_out), ("query_start_out", query_start_out)):
        if t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1):
            raise ValueError(f"{name} must be a contiguous 1-D tensor")
    padded = -1 if num_padded_tokens is None else int(num_padded_tokens)
    args = (
        _index(query_start_loc, torch.int32, "query_start_loc", dev, int(num_reqs) + 1),
        int(num_reqs), int(num_actual_tokens), padded,
        _dev(seq_idx_out, torch.int32, "seq_idx_out", dev), seq_idx_out.numel(),
        _dev(query_start_out, torch.int32, "query_start_out", dev), query_start_out.numel(),
    )
    _launch("sconv_seq_metadata", dev, args)


def sconv_paged_fused_multi(xs, weights, cache, positions, slot_mapping, query_start_loc,
                            block_table, offs, ws: int, activation=None,
                            use_residual: bool = True, biases=None, outs=None):
    """Several conv streams sharing one paged cache, in one launch.  xs,
    weights, offs (and biases / outs when given) are lists with one entry per
    stream; every stream has H * ws channels (ws may also be a list).
    Returns the list of outputs."""
    n = len(xs)
    if not (len(weights) == len(offs) == n) or n < 1:
        raise ValueError("xs, weights and offs need one entry per stream")
    wss = list(ws) if isinstance(ws, (list, tuple)) else [int(ws)] * n
    dev = xs[0].device
    num_blocks, H, N, D = cache.shape
    width = weights[0].shape[1]
    num_reqs = query_start_loc.numel() - 1
    T = xs[0].shape[0]
    if outs is None:
        outs = [torch.empty_like(x) for x in xs]
    if biases is None:
        biases = [None] * n
    bf = torch.bfloat16
    for i in range(n):
        x, w, b, o = xs[i], weights[i], biases[i], outs[i]
        if x.dim() != 2 or x.shape != (T, H * wss[i]) or x.stride(1) != 1:
            raise ValueError(f"stream {i}: x must be (T, H*ws) with unit channel stride")
        if o.shape != x.shape or o.stride(1) != 1:
            raise ValueError(f"stream {i}: out must match x")
        if w.dim() != 2 or w.shape != (H * wss[i], width) or w.stride(1) != 1:
            raise ValueError(f"stream {i}: weight must be (C, width) with unit width stride")
        if b is not None and (b.shape != (H * wss[i],) or b.stride(0) != 1):
            raise ValueError(f"stream {i}: bias must be a contiguous (C,) tensor")
    if cache.stride(3) != 1:
        raise ValueError("cache D must have unit stride")
    if block_table.dim() != 2 or (block_table.numel() and block_table.stride(1) != 1):
        raise ValueError("block_table must be (num_reqs, max_blocks) with unit inner stride")
    VP = ctypes.c_void_p * n
    I64A = ctypes.c_int64 * n
    I32A = ctypes.c_int32 * n
    xp = VP(*[_dev(x, bf, f"xs[{i}]", dev) for i, x in enumerate(xs)])
    wp = VP(*[_dev(w, bf, f"weights[{i}]", dev) for i, w in enumerate(weights)])
    bp = VP(*[_dev(b, bf, f"biases[{i}]", dev) for i, b in enumerate(biases)])
    op = VP(*[_dev(o, bf, f"outs[{i}]", dev) for i, o in enumerate(outs)])
    args = (
        n, xp, I64A(*[x.stride(0) for x in xs]), wp, I64A(*[w.stride(0) for w in weights]),
        bp if any(b is not None for b in biases) else None,
        I32A(*[int(o) for o in offs]), I32A(*wss), op, I64A(*[o.stride(0) for o in outs]),
        _dev(cache, bf, "cache", dev), cache.stride(0), cache.stride(1), cache.stride(2),
        num_blocks, H, N, D,
        _index(positions, torch.int64, "positions", dev, T),
        _index(slot_mapping, torch.int64, "slot_mapping", dev, T),
        _index(query_start_loc, torch.int32, "query_start_loc", dev, num_reqs + 1), num_reqs,
        _dev(block_table, torch.int32, "block_table", dev),
        block_table.stride(0) if block_table.dim() == 2 else 0,
        block_table.shape[1] if block_table.dim() == 2 else 0,
        T, width, _act(activation), int(bool(use_residual)),
    )
    _launch("sconv_paged_fused_multi", dev, args)
    return outs


# ------------------------------------------------------- gated delta rule --
#
# These calls take many tensors, and small ones are over in a few
# microseconds: what is checked is checked with few Python calls.

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32


def _ptr(t, dtype, name, dev, index):
    """Address of a checked tensor (0 for None); the failing checks are _dev's."""
    if t is None:
        return 0
    if t.dtype is not dtype or index < 0 or t.get_device() != index:
        _dev(t, dtype, name, dev)
    return t.data_ptr()


def _vec(t, dtype, name, dev, index, n):
    """Address of a checked contiguous 1-D tensor of at least n entries (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or index < 0 or t.get_device() != index or t.dim() != 1 or t.numel() < n or not t.is_contiguous():
        _index(t, dtype, name, dev, n)
    return t.data_ptr()


def _gdr_tensors(q, k, v, g, beta, A_log, dt_bias, state, out, dev, index, step=True):
    """Shapes (num_k_heads, num_v_heads, head_dim_k, head_dim_v) and the marshalled inputs, state and output of a call
    whose tensors have one and the same leading dimensions.  Without `step`, they lack the token dimension that the call
    has: its strides are 0."""
    qs, vs = q.shape, v.shape
    tokens = vs[:-1]
    if k.shape != qs or vs[:-2] != qs[:-2]:
        raise ValueError("q and k need one shape, and v the same tokens")
    hk, dk = qs[-2:]
    hv, dv = vs[-2:]
    if hk < 1 or hv % hk:
        raise ValueError("v's heads must be a multiple of q's")
    if g.shape != tokens or beta.shape != tokens:
        raise ValueError("g and beta need one value per token and value head")
    if out.shape != vs:
        raise ValueError("out must have v's shape")
    gate, layer = _F32, (0, 0)
    if A_log is not None or dt_bias is not None:
        if A_log is None or dt_bias is None:
            raise ValueError("A_log and dt_bias go together")
        gate, one = _BF16, (hv,)
        if A_log.shape != one or dt_bias.shape != one or not (A_log.is_contiguous() and dt_bias.is_contiguous()):
            raise ValueError("A_log and dt_bias must be contiguous (num_v_heads,) tensors")
        layer = (_ptr(A_log, _F32, "A_log", dev, index), _ptr(dt_bias, _F32, "dt_bias", dev, index))
    if state is None:
        st = (0, 0, 0, 0, 0, 0)
    else:
        ss = state.shape
        if ss[1:] != (hv, dv, dk):
            raise ValueError("state must be (lines, num_v_heads, head_dim_v, head_dim_k)")
        st = (_ptr(state, _F32, "state", dev, index), *state.stride(), ss[0])
    if not (index >= 0 and q.dtype is k.dtype is v.dtype is out.dtype is _BF16 and g.dtype is beta.dtype is gate and
            index == k.get_device() == v.get_device() == g.get_device() == beta.get_device() == out.get_device()):
        for t, dtype, name in ((q, _BF16, "q"), (k, _BF16, "k"), (v, _BF16, "v"), (g, gate, "g"), (beta, gate, "beta"),
                               (out, _BF16, "out")):
            _dev(t, dtype, name, dev)
    if step:
        ins = (q.data_ptr(), *q.stride(), k.data_ptr(), *k.stride(), v.data_ptr(), *v.stride(), g.data_ptr(), *g.stride(),
               beta.data_ptr(), *beta.stride(), *layer, *st)
        return (hk, hv, dk, dv), ins, (out.data_ptr(), *out.stride())
    ins = []
    for t in (q, k, v, g, beta, out):
        first, *rest = t.stride()
        ins += (t.data_ptr(), first, 0, *rest)
    return (hk, hv, dk, dv), (*ins[:-5], *layer, *st), ins[-5:]


def gdr_fwd_varlen(q, k, v, g, beta, state, query_start_loc, cache_indices=None,
                   has_initial_state=None, A_log=None, dt_bias=None, scale: float | None = None,
                   use_qk_l2norm: bool = False, pad_slot_id: int = -1, out=None):
    """The gated delta rule over a packed varlen batch: per value head and
    token, S <- e^g S; S <- S + beta (v - S k) k^T; out = S q * scale.

    q, k (T, num_k_heads, head_dim_k) and v (T, num_v_heads, head_dim_v) bf16,
    any strides (views of a convolution's (T, dim) output take the vector
    loads); g, beta (T, num_v_heads) fp32 log decay and write strength, or,
    with A_log and dt_bias (num_v_heads,) fp32, the layer's bf16 projections a
    and b (g = -exp(A_log) softplus(a + dt_bias), beta = sigmoid(b)); state
    (lines, num_v_heads, head_dim_v, head_dim_k) fp32 or None, updated in
    place; query_start_loc int32 (batch+1,), cache_indices int32 (batch,) or
    None, has_initial_state bool (batch,) or None: as for conv1d_fwd_varlen.
    scale defaults to head_dim_k ** -0.5.  Returns out (T, num_v_heads,
    head_dim_v); rows of padded sequences are left as they are.
    Calls of few heads, and layouts without vector loads, take a workspace for
    the time of the call: 19.3 KiB * (T / 64 + batch + 2) * num_v_heads, 1.3 GB
    for 131072 tokens of 32 heads.  Where memory for it is short, a call takes a
    slower form that needs none."""
    dev = q.device
    index = q.get_device()
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be (T, heads, head_dim)")
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=dev)
    (hk, hv, dk, dv), ins, (o, o_tok, o_head, o_dim) = _gdr_tensors(
        q, k, v, g, beta, A_log, dt_bias, state, out, dev, index)
    total = q.shape[0]
    batch = query_start_loc.numel() - 1
    qa, q_tok, q_head, q_dim, ka, k_tok, k_head, k_dim, va, v_tok, v_head, v_dim = ins[:12]
    vector = (q_dim == k_dim == v_dim == o_dim == 1 and not (
        (dk | dv | q_tok | q_head | k_tok | k_head | v_tok | v_head) & 7 or (o_tok | o_head) & 3 or
        (qa | ka | va) & 15 or o & 7) and q_tok >= dk and k_tok >= dk and v_tok >= dv and o_tok >= dv)
    lib = load_library()
    need = lib.gdr_fwd_workspace_bytes(batch, total, hk, hv, dk, dv, vector)
    # the workspace is this stream's until the launch is made: whoever gets its memory next comes after it
    try:
        ws = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=dev) if need else None
    except torch.OutOfMemoryError:
        need = 0                  # (the forms that take none are slower, and right)
    _launch_packed("gdr_fwd_varlen", dev, (
        *ins, _vec(cache_indices, _I32, "cache_indices", dev, index, batch),
        _vec(has_initial_state, torch.bool, "has_initial_state", dev, index, batch),
        _vec(query_start_loc, _I32, "query_start_loc", dev, index, 1),
        batch, total, hk, hv, dk, dv, dk ** -0.5 if scale is None else float(scale),
        1 if use_qk_l2norm else 0, pad_slot_id, o, o_tok, o_head, o_dim,
        ws.data_ptr() if need else 0, need))
    return out


def gdr_update(q, k, v, g, beta, state, cache_indices=None, num_accepted_tokens=None,
               output_state_indices=None, A_log=None, dt_bias=None, scale: float | None = None,
               use_qk_l2norm: bool = False, pad_slot_id: int = -1, out=None):
    """Decode update of the gated delta rule: q, k (batch, num_k_heads,
    head_dim_k) or (batch, seqlen, num_k_heads, head_dim_k), v and the gates
    likewise (types as for gdr_fwd_varlen), state updated in place.

    cache_indices int32 (batch,), or (batch, steps) with num_accepted_tokens
    (batch,) int32: entry b then reads line cache_indices[b,
    num_accepted_tokens[b] - 1].  output_state_indices int32 (batch, seqlen):
    the lines that receive the state after each step, in place of the update
    of the line that was read; the lines of one call are the next call's
    cache_indices.  Returns out, shaped like v."""
    dev = q.device
    index = q.get_device()
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=dev)
    shape = q.shape
    batch, seqlen, step = shape[0] if shape else 0, 1, False
    if len(shape) == 4:
        seqlen, step = shape[1], True
        if v.dim() != 4:
            raise ValueError("q, k and v must be (batch, [seqlen,] heads, head_dim)")
    elif len(shape) != 3:
        raise ValueError("q, k and v must be (batch, [seqlen,] heads, head_dim)")
    elif v.dim() != 3 or g.dim() != 2 or beta.dim() != 2 or out.dim() != 3:
        raise ValueError("q, k, v, g, beta and out must all be without a token dimension, or none")
    if state is None:
        raise ValueError("state is required")
    ci, ci_seq, ci_step, steps, wide = cache_indices, 0, 0, 1, False
    if ci is not None:
        cs = ci.shape
        wide = len(cs) == 2
        if not (wide or len(cs) == 1) or cs[0] < batch:
            raise ValueError("cache_indices must be (batch,) or (batch, steps)")
        if wide:
            steps = cs[1]
            ci_seq, ci_step = ci.stride()
        else:
            ci_seq = ci.stride(0)
    if num_accepted_tokens is not None and not wide:
        raise ValueError("num_accepted_tokens needs cache_indices of (batch, steps)")
    osi, osi_seq, osi_step = output_state_indices, 0, 0
    if osi is not None:
        if osi.dim() != 2 or osi.shape[0] < batch or osi.shape[1] < seqlen:
            raise ValueError("output_state_indices must be (batch, >= seqlen)")
        osi_seq, osi_step = osi.stride()
    (hk, hv, dk, dv), ins, outs = _gdr_tensors(q, k, v, g, beta, A_log, dt_bias, state, out, dev, index, step)
    _launch_packed("gdr_update", dev, (
        *ins, _ptr(ci, _I32, "cache_indices", dev, index), ci_seq, ci_step, steps,
        _vec(num_accepted_tokens, _I32, "num_accepted_tokens", dev, index, batch),
        _ptr(osi, _I32, "output_state_indices", dev, index), osi_seq, osi_step,
        batch, seqlen, hk, hv, dk, dv, dk ** -0.5 if scale is None else float(scale),
        1 if use_qk_l2norm else 0, pad_slot_id, *outs))
    return out


# ----------------------------------------------------- draft verification --

def sconv_verify_drafts(draft_tokens, draft_start_loc, target_probs, draft_probs,
                        accept_uniform, sample_uniform, max_drafts: int, tokens=None,
                        num_accepted_tokens=None):
    """Which drafted tokens stand, and the token drawn after them.

    draft_tokens int32 (num_drafts,), request i's at draft_start_loc[i] ..
    draft_start_loc[i+1] (int32 (batch+1,)), at most max_drafts each;
    target_probs fp32 (num_drafts + batch, vocab), request i's rows at
    draft_start_loc[i] + i; draft_probs fp32 (num_drafts, vocab), or None for
    deterministic drafts; accept_uniform fp32 (num_drafts,) and sample_uniform
    fp32 (batch,) in [0, 1).  Returns (tokens, num_accepted_tokens): int32
    (batch, max_drafts + 1) with the standing drafts, the drawn token, then -1;
    int32 (batch,) with standing drafts + 1, as conv1d_update and gdr_update
    take it."""
    p, q = target_probs, draft_probs
    dev, index = p.device, p.get_device()
    batch = draft_start_loc.numel() - 1
    nd = draft_tokens.numel()
    shape = p.shape
    if len(shape) != 2 or shape[0] < nd + batch:
        raise ValueError("target_probs must be (num_drafts + batch, vocab)")
    vocab = shape[1]
    p_row, p_one = p.stride()
    if vocab > 1 and p_one != 1:
        raise ValueError("target_probs must have a unit vocabulary stride")
    q_row = 0
    if q is not None:
        shape = q.shape
        if len(shape) != 2 or shape[0] < nd or shape[1] != vocab:
            raise ValueError("draft_probs must be (num_drafts, vocab)")
        q_row, q_one = q.stride()
        if vocab > 1 and q_one != 1:
            raise ValueError("draft_probs must have a unit vocabulary stride")
        if nd == 0:
            q = None
    if tokens is None:
        tokens = torch.empty_strided((max(batch, 0), max_drafts + 1), (max_drafts + 1, 1), dtype=_I32, device=dev)
    elif tokens.shape != (batch, max_drafts + 1) or tokens.stride(1) != 1:
        raise ValueError("tokens must be (batch, max_drafts + 1) with a unit inner stride")
    if num_accepted_tokens is None:
        num_accepted_tokens = torch.empty_strided((max(batch, 0),), (1,), dtype=_I32, device=dev)
    ws_bytes = load_library().sconv_verify_workspace_bytes(batch, vocab)
    # the workspace is this stream's until the launch is made: whoever gets its memory next comes after it
    ws = torch.empty_strided((ws_bytes,), (1,), dtype=torch.uint8, device=dev)
    _launch("sconv_verify_drafts", dev, (
        _vec(draft_tokens, _I32, "draft_tokens", dev, index, nd),
        _vec(draft_start_loc, _I32, "draft_start_loc", dev, index, batch + 1),
        _ptr(p, _F32, "target_probs", dev, index), p_row,
        _ptr(q, _F32, "draft_probs", dev, index), q_row,
        _vec(accept_uniform, _F32, "accept_uniform", dev, index, nd),
        _vec(sample_uniform, _F32, "sample_uniform", dev, index, batch),
        batch, nd, vocab, max_drafts, _ptr(tokens, _I32, "tokens", dev, index), tokens.stride(0),
        _vec(num_accepted_tokens, _I32, "num_accepted_tokens", dev, index, batch), ws.data_ptr(),
        ws_bytes))
    return tokens, num_accepted_tokens


# ------------------------------------------------- selective state space scan --

_INF = float("inf")


def _ssm_tensors(x, dt, A, B, C, D, z, dt_bias, state, out, dev, index, lead):
    """Checks and marshals what prefill and decode share.  `lead`: x's leading dimensions (tokens, or entries and maybe
    tokens).  Returns the sizes (heads, groups, head_dim, state_dim), the tensors (x, dt), A, (B, C), D, z, dt_bias, state and
    out, each as its address and strides (the leading dimensions' first), and whether dt is fp32."""
    n = len(lead)
    a_shape, xs, bs = A.shape, x.shape, B.shape
    if C.shape != bs or bs[:n] != lead:
        raise ValueError("B and C need one shape, and x's tokens")
    if out.shape != xs or (z is not None and z.shape != xs):
        raise ValueError("out and z must have x's shape")
    rest = xs[n:]
    if len(a_shape) == 1:              # one decay a head
        if len(rest) != 2 or a_shape[0] != rest[0] or len(bs) != n + 2:
            raise ValueError("A (heads,) needs x (.., heads, head_dim) and B, C (.., groups, state_dim)")
        H, P = rest
        G, N = bs[n:]
        of = (H,)                      # what has a step size
        a_str, d_str = (A.stride(0), 0, 0), (0,)
        whole = (H, P)
    elif len(a_shape) == 2:            # one a channel and state
        if len(rest) != 1 or a_shape[0] != rest[0] or len(bs) not in (n + 1, n + 2) or bs[-1] != a_shape[1]:
            raise ValueError("A (dim, state_dim) needs x (.., dim) and B, C (.., [groups,] state_dim)")
        dim, N = a_shape
        H = G = bs[n] if len(bs) == n + 2 else 1
        if G < 1 or dim % G:
            raise ValueError("dim must be a multiple of B's groups")
        P = dim // G
        of = whole = (dim,)
        a0, a1 = A.stride()
        a_str = (P * a0, a0, a1)
    else:
        raise ValueError("A must be (heads,) or (dim, state_dim)")
    heads = len(a_shape) == 1
    if H < 1 or G < 1 or H % G:
        raise ValueError("x's heads must be a multiple of B's groups")
    if dt.shape != (*lead, *of):
        raise ValueError("dt needs one value per token and head, or per token and channel where A has one decay a channel")

    def weight(t, name):
        if t is None:
            return 0, 0, 0
        if t.shape != of and t.shape != whole:
            raise ValueError(f"{name} must be ({'heads,) or (heads, head_dim' if name == 'D' and heads else 'heads,' if heads else 'dim,'})")
        st = t.stride()
        return (_ptr(t, _F32, name, dev, index), *((st[0], 0) if t.dim() == 1 else st)) if heads else (
            _ptr(t, _F32, name, dev, index), P * st[0], st[0])

    def rows(t):                       # x, z, out
        st = t.stride()
        return st if heads else (*st[:-1], P * st[-1], st[-1])

    if dt_bias is not None and dt_bias.shape != of:
        raise ValueError("dt_bias needs one value per step size of a token")
    if state is None:
        st = (0, 0, 0, 0, 0, 0)
    else:
        ss = state.shape
        if ss[1:] != (*whole, N):
            raise ValueError("state must be (lines, heads, head_dim, state_dim), or (lines, dim, state_dim)")
        s4 = state.stride()
        st = (_ptr(state, _F32, "state", dev, index), *(s4 if heads else (s4[0], P * s4[1], s4[1], s4[2])), ss[0])
    dt_fp32 = dt.dtype is _F32
    if not (index >= 0 and x.dtype is B.dtype is C.dtype is out.dtype is _BF16 and A.dtype is _F32 and
            (dt_fp32 or dt.dtype is _BF16) and (z is None or (z.dtype is _BF16 and z.get_device() == index)) and
            index == B.get_device() == C.get_device() == dt.get_device() == A.get_device() == out.get_device()):
        for t, dtype, name in ((x, _BF16, "x"), (B, _BF16, "B"), (C, _BF16, "C"), (z, _BF16, "z"), (out, _BF16, "out"),
                               (A, _F32, "A"), (dt, _F32 if dt_fp32 else _BF16, "dt")):
            _dev(t, dtype, name, dev)
    d_st = dt.stride()
    d_st = (*d_st, 0) if heads else (*d_st[:-1], P * d_st[-1], d_st[-1])
    b_st, c_st = B.stride(), C.stride()
    if len(bs) == n + 1:
        b_st, c_st = (*b_st[:-1], 0, b_st[-1]), (*c_st[:-1], 0, c_st[-1])
    return ((H, G, P, N), ((x.data_ptr(), *rows(x)), (dt.data_ptr(), *d_st)), (A.data_ptr(), *a_str),
            ((B.data_ptr(), *b_st), (C.data_ptr(), *c_st)), weight(D, "D"),
            (0,) * (n + 3) if z is None else (z.data_ptr(), *rows(z)), weight(dt_bias, "dt_bias"), st,
            (out.data_ptr(), *rows(out)), dt_fp32)


def _limits(dt_limit):
    if dt_limit is None:
        return -_INF, _INF
    lo, hi = dt_limit
    return ctypes.c_float(lo).value, ctypes.c_float(hi).value      # (what fp32 does not hold is no limit)


def ssm_fwd_varlen(x, dt, A, B, C, state, query_start_loc, cache_indices=None, has_initial_state=None, D=None, z=None,
                   dt_bias=None, dt_softplus: bool = False, dt_limit=None, pad_slot_id: int = -1, out=None):
    """The selective state space scan over a packed varlen batch: per channel and token,
    S <- e^(d A) S + d x B; out = (S . C + D x) silu(z), with d = clamp([softplus](dt + dt_bias)).

    One decay a head: A (heads,), x (T, heads, head_dim), dt (T, heads), B, C (T, groups, state_dim), state
    (lines, heads, head_dim, state_dim), D (heads,) or (heads, head_dim), dt_bias (heads,).  One a channel and state:
    A (dim, state_dim), x (T, dim), dt (T, dim), B, C (T, [groups,] state_dim), state (lines, dim, state_dim), D and dt_bias
    (dim,).  x, B, C and z bf16, any strides (views of a convolution's (T, dim) output take the vector loads); dt bf16 or
    fp32; A, D, dt_bias and state fp32; D, z (like x), dt_bias and state may be None.  dt_limit: (least, largest) step size.
    A decay d A above 0 counts as 0.  query_start_loc int32 (batch+1,), cache_indices int32 (batch,) or None,
    has_initial_state bool (batch,) or None: as for conv1d_fwd_varlen.  state is updated in place.  Returns out, like x;
    rows of padded sequences are left as they are.  Calls of few heads and long sequences take a workspace of up to 87 MB for
    the time of the call; where memory for it is short, a call takes a slower form that needs none."""
    dev = x.device
    index = x.get_device()
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    (H, G, P, N), (xa, da), a, (ba, ca), d, za, bias, st, o, dt_fp32 = _ssm_tensors(
        x, dt, A, B, C, D, z, dt_bias, state, out, dev, index, x.shape[:1])
    lo, hi = _limits(dt_limit)
    batch = query_start_loc.numel() - 1
    total = x.shape[0]
    need = load_library().ssm_fwd_workspace_bytes(batch, total, H, G, P, N, A.dim() == 2)
    # the workspace is this stream's until the launch is made: whoever gets its memory next comes after it
    try:
        ws = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=dev) if need else None
    except torch.OutOfMemoryError:
        need = 0                  # (the forms that take none are slower, and right)
    _launch_packed("ssm_fwd_varlen", dev, (
        *xa, *da, dt_fp32, *a, *ba, *ca, *d, *za, *bias, 1 if dt_softplus else 0, lo, hi, *st,
        _vec(cache_indices, _I32, "cache_indices", dev, index, batch),
        _vec(has_initial_state, torch.bool, "has_initial_state", dev, index, batch),
        _vec(query_start_loc, _I32, "query_start_loc", dev, index, 1),
        batch, total, H, G, P, N, pad_slot_id, *o, ws.data_ptr() if need else 0, need))
    return out


def ssm_update(x, dt, A, B, C, state, cache_indices=None, num_accepted_tokens=None, output_state_indices=None, D=None,
               z=None, dt_bias=None, dt_softplus: bool = False, dt_limit=None, pad_slot_id: int = -1, out=None):
    """Decode update of the selective state space scan: x, dt, B, C and z as for ssm_fwd_varlen with (batch,) or
    (batch, seqlen) in place of the tokens, state updated in place.  cache_indices, num_accepted_tokens and
    output_state_indices: as for gdr_update.  Returns out, shaped like x."""
    dev = x.device
    index = x.get_device()
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    n = x.dim() - (2 if A.dim() == 1 else 1)
    if n not in (1, 2):
        raise ValueError("x must be (batch, [seqlen,] heads, head_dim), or (batch, [seqlen,] dim)")
    if state is None:
        raise ValueError("state is required")
    batch, seqlen = x.shape[0], x.shape[1] if n == 2 else 1
    ci, ci_seq, ci_step, steps, wide = cache_indices, 0, 0, 1, False
    if ci is not None:
        cs = ci.shape
        wide = len(cs) == 2
        if not (wide or len(cs) == 1) or cs[0] < batch:
            raise ValueError("cache_indices must be (batch,) or (batch, steps)")
        if wide:
            steps = cs[1]
            ci_seq, ci_step = ci.stride()
        else:
            ci_seq = ci.stride(0)
    if num_accepted_tokens is not None and not wide:
        raise ValueError("num_accepted_tokens needs cache_indices of (batch, steps)")
    osi, osi_seq, osi_step = output_state_indices, 0, 0
    if osi is not None:
        if osi.dim() != 2 or osi.shape[0] < batch or osi.shape[1] < seqlen:
            raise ValueError("output_state_indices must be (batch, >= seqlen)")
        osi_seq, osi_step = osi.stride()
    (H, G, P, N), (xa, da), a, (ba, ca), d, za, bias, st, o, dt_fp32 = _ssm_tensors(
        x, dt, A, B, C, D, z, dt_bias, state, out, dev, index, x.shape[:n])
    if n == 1:                         # (a token dimension of stride 0)
        xa, da, ba, ca, za, o = ((*t[:2], 0, *t[2:]) for t in (xa, da, ba, ca, za, o))
    lo, hi = _limits(dt_limit)
    _launch_packed("ssm_update", dev, (
        *xa, *da, dt_fp32, *a, *ba, *ca, *d, *za, *bias, 1 if dt_softplus else 0, lo, hi, *st,
        _ptr(ci, _I32, "cache_indices", dev, index), ci_seq, ci_step, steps,
        _vec(num_accepted_tokens, _I32, "num_accepted_tokens", dev, index, batch),
        _ptr(osi, _I32, "output_state_indices", dev, index), osi_seq, osi_step,
        batch, seqlen, H, G, P, N, pad_slot_id, *o))
    return out


# -------------------------------------------------------------- group norm --

_NORMS = {"rms": 0, "layer": 1}
_NORM_ACTS = {None: 0, "silu": 1, "swish": 1, "sigmoid": 2}


def sconv_group_norm(x, group_size: int | None = None, weight=None, bias=None, z=None, eps: float = 1e-5,
                     norm: str = "rms", activation=None, gate_first: bool = False, out=None):
    """The norm of every group of channels of every row, with the layer's gate or activation.

    x (rows, channels) bf16 in groups of group_size channels (default: all of them), or (rows, heads, head_dim) with a group a
    head; z like x, or None; weight and bias bf16 or fp32 (one type), of all the channels or of one group (shared by the
    groups), or None.  v = x act(z) with gate_first, else x; v = norm(v) weight + bias over each group ("rms": by its root
    mean square; "layer": its mean is taken out first); then v act(z), or act(v) without z, or v with gate_first.
    activation: None, "silu" or "sigmoid".  Returns out, which may be x or z itself."""
    dev, index = x.device, x.get_device()
    xs = x.shape
    if len(xs) == 3:
        rows, groups, size = xs
        if group_size is not None and group_size != size:
            raise ValueError("x of heads is normalised by heads: group_size must be head_dim")
    elif len(xs) == 2:
        rows, channels = xs
        size = channels if group_size is None else group_size
        if size < 1 or channels % size:
            if channels:
                raise ValueError("channels must be a multiple of group_size")
            size = 1
        groups = channels // size
    else:
        raise ValueError("x must be (rows, channels) or (rows, heads, head_dim)")
    if out is None:
        out = torch.empty(xs, dtype=x.dtype, device=dev)
    if out.shape != xs or (z is not None and z.shape != xs):
        raise ValueError("out and z must have x's shape")
    if norm not in _NORMS or activation not in _NORM_ACTS:
        raise ValueError(f"unsupported norm {norm!r} or activation {activation!r}")
    if gate_first and z is None:
        raise ValueError("gate_first needs z")
    first = bias if weight is None else weight
    w_type, ws = _F32 if first is not None and first.dtype is _F32 else _BF16, []
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            ws += (0, 0)
            continue
        n = t.numel()
        if n not in (size, groups * size) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor of all the channels or of one group's")
        ws += (_ptr(t, w_type, name, dev, index), size if n != size else 0)

    def strides(t):
        st = t.stride()
        return st if len(st) == 3 else (st[0], size * st[1], st[1])

    _launch("sconv_group_norm", dev, (
        _ptr(x, _BF16, "x", dev, index), *strides(x),
        *((_ptr(z, _BF16, "z", dev, index), *strides(z)) if z is not None else (0, 0, 0, 0)), *ws, w_type is _F32,
        rows, groups, size, _NORMS[norm], _NORM_ACTS[activation], 1 if gate_first else 0, eps,
        _ptr(out, _BF16, "out", dev, index), *strides(out)))
    return out
