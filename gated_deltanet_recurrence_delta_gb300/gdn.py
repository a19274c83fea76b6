"""Thin ctypes binding of ``libgdn.so`` (the C-ABI declared in ``include/gdn.h``).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. Tensors are torch CUDA tensors (device memory and streams come from
PyTorch); their data pointers are handed to the C entry points of the same
names. A non-OK status raises :class:`GdnError`. If the library has not been
built, the first call raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import math
from pathlib import Path

import torch

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "_build" / "libgdn.so"

STATUS = {0: "GDN_OK", 1: "GDN_ERR_ARG", 2: "GDN_ERR_SHAPE", 3: "GDN_ERR_MASK", 4: "GDN_ERR_INDEX",
          5: "GDN_ERR_CUDA", 6: "GDN_ERR_WORKSPACE", 7: "GDN_ERR_TIMEOUT", 8: "GDN_ERR_FULL"}
EXPORTS = ("gdn_decode_step", "gdn_verify_with_checkpoints", "gdn_prefill_chunked",
           "gdn_prefill_workspace_size", "gdn_state_copy", "gdn_check_status", "gdn_last_error",
           "gdn_prefill_chunked_static_scratch", "gdn_commit_accepted", "gdn_decode_step_mxfp8",
           "gdn_prefill_chunked_ckpt", "gdn_in_proj", "gdn_out_proj", "gdn_copy_overlapped",
           "gdn_head_norm_rope", "gdn_attn_prefill", "gdn_attn_shared_prefix", "gdn_attn_workspace_size",
           "gdn_accept_draft", "gdn_kv4_store", "gdn_kv4_load", "gdn_attn_kv4", "gdn_attn_kv4_workspace_size",
           "gdn_beam_select", "gdn_beam_workspace_size", "gdn_cache_fork", "gdn_slots_copy")
MAX_OVERLAPPED_COPIES = 8
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8  # 30 ns each when looked up in a call
MAX_SLOT_POOLS = 4
PAGE_TOKENS = 64


class GdnError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code
        self.name = STATUS.get(code, str(code))


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "nk", "nv", "dk", "dv", "conv_k", "n_slots")] + [
        ("scale", ctypes.c_float), ("l2_eps", ctypes.c_float), ("rms_eps", ctypes.c_float)]


class Inputs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "z", "a", "b", "A_log", "dt_bias", "conv_w",
                                               "norm_w", "mask", "cu_seqlens", "state_idx")]


class InputsMxfp8(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "z", "q_scale", "k_scale", "v_scale", "z_scale", "a",
                                               "b", "A_log", "dt_bias", "conv_w", "norm_w", "mask", "state_idx")]


class Copy(ctypes.Structure):
    _fields_ = [("dst", ctypes.c_void_p), ("src", ctypes.c_void_p), ("bytes", ctypes.c_size_t)]


class RopeDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_tokens", "n_q_heads", "n_kv_heads", "head_dim", "rot_dim", "n_axes",
                                              "adjacent")] + [("eps", ctypes.c_float)] + [
        (n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride", "kv_rows")]


class AttnDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "n_tokens", "n_groups", "n_q_heads", "n_kv_heads",
                                              "head_dim")] + [("scale", ctypes.c_float)] + [
        (n, ctypes.c_int64) for n in ("q_stride", "kv_stride", "kv_rows")]


class Kv4Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_tokens", "n_kv_heads", "head_dim", "n_pages", "k_exp", "v_exp")] + [
        (n, ctypes.c_int64) for n in ("k_stride", "v_stride")]


class AttnKv4Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "n_q_heads", "n_kv_heads", "head_dim", "n_pages", "max_pages",
                                              "k_exp", "v_exp")] + [("scale", ctypes.c_float), ("q_stride", ctypes.c_int64)]


class BeamDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_groups", "beams", "vocab", "half", "eos")] + [
        ("row_stride", ctypes.c_int64)]


class ForkDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_rows", "T", "max_pages", "n_pages")]


class SlotPool(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("base", "src", "dst")] + [("slot_bytes", ctypes.c_int64)] + [
        (n, ctypes.c_int32) for n in ("n", "n_layers", "n_slots")]


_pools_of = [SlotPool * max(1, n) for n in range(MAX_SLOT_POOLS + 1)]  # 0.4 us on the host when made in a call


_lib = None


def load_library(path: Path | str | None = None):
    """Load libgdn.so (in-tree build). Raises if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = Path(path) if path else LIB_PATH
    if not p.exists():
        raise RuntimeError(f"{p} is not built; run gated_deltanet_recurrence_delta_gb300.build.build()")
    lib = ctypes.CDLL(str(p))
    P = ctypes.c_void_p
    DP = ctypes.POINTER(Dims)
    IP = ctypes.POINTER(Inputs)
    lib.gdn_decode_step.argtypes = [DP, IP, P, P, P, P]
    lib.gdn_verify_with_checkpoints.argtypes = [DP, IP, P, P, P, P, P, P]
    lib.gdn_prefill_chunked.argtypes = [DP, IP, P, P, P, P, ctypes.c_size_t, P]
    lib.gdn_prefill_chunked_static_scratch.argtypes = [DP, IP, P, P, P, P]
    lib.gdn_prefill_workspace_size.argtypes = [DP, ctypes.c_int]
    lib.gdn_prefill_workspace_size.restype = ctypes.c_size_t
    lib.gdn_state_copy.argtypes = [DP, P, P, P, P, P, P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P]
    lib.gdn_prefill_chunked_ckpt.argtypes = [DP, IP, P, P, P, P, ctypes.c_size_t, P, ctypes.c_int32, P, P,
                                             ctypes.c_int32, P]
    lib.gdn_in_proj.argtypes = [DP, ctypes.c_int32, ctypes.c_int32, P, P, P, P, P, P, P, P, P]
    lib.gdn_out_proj.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, P, P, P]
    lib.gdn_decode_step_mxfp8.argtypes = [DP, ctypes.POINTER(InputsMxfp8), P, P, P, P]
    lib.gdn_commit_accepted.argtypes = [DP, ctypes.c_int32, ctypes.c_int32, P, P, P, P, P, P, P, P]
    lib.gdn_copy_overlapped.argtypes = [ctypes.POINTER(Copy), ctypes.c_int32, P]
    lib.gdn_head_norm_rope.argtypes = [ctypes.POINTER(RopeDims)] + [P] * 13
    AP = ctypes.POINTER(AttnDims)
    lib.gdn_attn_prefill.argtypes = [AP] + [P] * 8
    lib.gdn_attn_shared_prefix.argtypes = [AP] + [P] * 11 + [ctypes.c_size_t, P]
    lib.gdn_attn_workspace_size.argtypes = [AP]
    lib.gdn_attn_workspace_size.restype = ctypes.c_size_t
    lib.gdn_accept_draft.argtypes = [ctypes.c_int32] * 3 + [P] * 8
    lib.gdn_kv4_store.argtypes = [ctypes.POINTER(Kv4Dims)] + [P] * 5
    lib.gdn_kv4_load.argtypes = [ctypes.POINTER(Kv4Dims)] + [P] * 5
    lib.gdn_attn_kv4.argtypes = [ctypes.POINTER(AttnKv4Dims)] + [P] * 7 + [ctypes.c_size_t, P]
    lib.gdn_attn_kv4_workspace_size.argtypes = [ctypes.POINTER(AttnKv4Dims)]
    lib.gdn_attn_kv4_workspace_size.restype = ctypes.c_size_t
    lib.gdn_beam_select.argtypes = [ctypes.POINTER(BeamDims)] + [P] * 8 + [ctypes.c_size_t, P]
    lib.gdn_beam_workspace_size.argtypes = [ctypes.POINTER(BeamDims)]
    lib.gdn_beam_workspace_size.restype = ctypes.c_size_t
    lib.gdn_cache_fork.argtypes = [ctypes.POINTER(ForkDims)] + [P] * 15
    lib.gdn_slots_copy.argtypes = [ctypes.POINTER(SlotPool), ctypes.c_int32, P]
    lib.gdn_check_status.argtypes = [P]
    lib.gdn_last_error.restype = ctypes.c_char_p
    for name in ("gdn_decode_step", "gdn_verify_with_checkpoints", "gdn_prefill_chunked", "gdn_state_copy",
                 "gdn_check_status", "gdn_prefill_chunked_static_scratch", "gdn_commit_accepted",
                 "gdn_decode_step_mxfp8", "gdn_prefill_chunked_ckpt", "gdn_in_proj", "gdn_out_proj",
                 "gdn_copy_overlapped", "gdn_head_norm_rope", "gdn_attn_prefill", "gdn_attn_shared_prefix",
                 "gdn_accept_draft", "gdn_kv4_store", "gdn_kv4_load", "gdn_attn_kv4", "gdn_beam_select",
                 "gdn_cache_fork", "gdn_slots_copy"):
        getattr(lib, name).restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def last_error() -> str:
    return load_library().gdn_last_error().decode()


def _check(code: int):
    if code != 0:
        raise GdnError(code, last_error())


def _ptr(t):
    return t if t is None or isinstance(t, int) else t.data_ptr()


# torch.cuda.current_stream() builds a Stream object (3 us); a small call's kernel takes 5
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _device is not None:
            return _raw_stream(_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _array(x, dtype, size, name):
    """_ptr of an array that a kernel indexes by position alone: refuses a tensor of another type, of fewer than `size`
    bytes or with gaps (0.3 us on the host). What has no tensor to look at (None, a raw address) passes."""
    if x is None or x.__class__ is int:
        return x
    if x.dtype is dtype and x.nbytes >= size and x.is_contiguous():
        return x.data_ptr()
    raise ValueError(f"{name} must be a dense {dtype} tensor of {size // dtype.itemsize} elements or more, it is {x.dtype} "
                     f"{list(x.shape)} with strides {list(x.stride())}")


def _arrays(dtype, size, names, *arrays):
    """_array of each, in one go."""
    return [x if x is None or x.__class__ is int
            else x.data_ptr() if x.dtype is dtype and x.nbytes >= size and x.is_contiguous()
            else _array(x, dtype, size, names[i]) for i, x in enumerate(arrays)]


def _here(x, name):
    """Refuses a tensor that is not on the current device, on which the kernels run."""
    if isinstance(x, torch.Tensor):
        device = x.get_device()
        if device < 0 or device != (_device() if _device is not None else torch.cuda.current_device()):
            raise ValueError(f"{name} must be on the current device, it is on {x.device}")


def _space(workspace):
    """Address and bytes of a workspace tensor, which is dense."""
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be dense")
    return workspace.data_ptr(), workspace.nbytes


def _flags(x):
    """Truth values as the bytes that they are."""
    return x if x is None or x.__class__ is int or x.dtype is not torch.bool else x.view(_U8)


def make_dims(B, T, nk, nv, dk, dv, n_slots, conv_k=4, scale=None, l2_eps=1e-6, rms_eps=1e-6) -> Dims:
    return Dims(B=B, T=T, nk=nk, nv=nv, dk=dk, dv=dv, conv_k=conv_k, n_slots=n_slots,
                scale=dk ** -0.5 if scale is None else scale, l2_eps=l2_eps, rms_eps=rms_eps)


def make_inputs(q, k, v, z, a, b, A_log, dt_bias, conv_w, norm_w, mask=None, cu_seqlens=None,
                state_idx=None) -> Inputs:
    """The inputs struct of raw device pointers. It keeps references to the
    tensors, so they (and their device memory) live as long as the struct."""
    inp = Inputs(q=_ptr(q), k=_ptr(k), v=_ptr(v), z=_ptr(z), a=_ptr(a), b=_ptr(b), A_log=_ptr(A_log),
                 dt_bias=_ptr(dt_bias), conv_w=_ptr(conv_w), norm_w=_ptr(norm_w), mask=_ptr(mask),
                 cu_seqlens=_ptr(cu_seqlens), state_idx=_ptr(state_idx))
    inp._tensors = (q, k, v, z, a, b, A_log, dt_bias, conv_w, norm_w, mask, cu_seqlens, state_idx)
    return inp


def make_inputs_mxfp8(q, k, v, z, q_scale, k_scale, v_scale, z_scale, a, b, A_log, dt_bias, conv_w, norm_w,
                      mask=None, state_idx=None) -> InputsMxfp8:
    """The MXFP8 inputs struct (e4m3 q/k/v/z as uint8 tensors, their E8M0
    block scales as uint8 tensors); keeps references to the tensors."""
    t = (q, k, v, z, q_scale, k_scale, v_scale, z_scale, a, b, A_log, dt_bias, conv_w, norm_w, mask, state_idx)
    inp = InputsMxfp8(*(_ptr(x) for x in t))
    inp._tensors = t
    return inp


def decode_step_mxfp8(dims: Dims, inputs: InputsMxfp8, conv_state, recurrent_state, out, stream=None):
    _check(load_library().gdn_decode_step_mxfp8(ctypes.byref(dims), ctypes.byref(inputs), _ptr(conv_state),
                                                _ptr(recurrent_state), _ptr(out), _stream(stream)))


def copy_overlapped(copies, stream=None):
    """gdn_copy_overlapped: up to MAX_OVERLAPPED_COPIES copies given as
    (dst, src, nbytes) -- tensors or raw addresses, device memory or pinned
    host memory -- done by one kernel that runs alongside the kernel before it
    on the stream and completes after it. The caller keeps the buffers alive
    and untouched until the stream has passed the call."""
    arr = (Copy * max(1, len(copies)))(*[Copy(_ptr(d), _ptr(s), int(n)) for d, s, n in copies])
    _check(load_library().gdn_copy_overlapped(arr, len(copies), _stream(stream)))


def decode_step(dims: Dims, inputs: Inputs, conv_state, recurrent_state, out, stream=None):
    _check(load_library().gdn_decode_step(ctypes.byref(dims), ctypes.byref(inputs), _ptr(conv_state),
                                          _ptr(recurrent_state), _ptr(out), _stream(stream)))


def verify_with_checkpoints(dims: Dims, inputs: Inputs, conv_state, recurrent_state, out, ckpt_state, ckpt_conv,
                            stream=None):
    _check(load_library().gdn_verify_with_checkpoints(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(conv_state), _ptr(recurrent_state), _ptr(out),
        _ptr(ckpt_state), _ptr(ckpt_conv), _stream(stream)))


def prefill_workspace_size(dims: Dims, packed: bool = False) -> int:
    """Workspace bytes of a prefill call: dense rows, or packed rows (cu_seqlens)."""
    return int(load_library().gdn_prefill_workspace_size(ctypes.byref(dims), int(bool(packed))))


def prefill_chunked(dims: Dims, inputs: Inputs, conv_state, recurrent_state, out, workspace, workspace_bytes=None,
                    stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load_library().gdn_prefill_chunked(ctypes.byref(dims), ctypes.byref(inputs), _ptr(conv_state),
                                              _ptr(recurrent_state), _ptr(out), _ptr(workspace),
                                              int(workspace_bytes), _stream(stream)))


def prefill_chunked_ckpt(dims: Dims, inputs: Inputs, conv_state, recurrent_state, out, workspace, ckpt, ckpt_state,
                         ckpt_conv, workspace_bytes=None, stream=None):
    """gdn_prefill_chunked_ckpt: ckpt is a device int32 [n, 3] tensor of (row,
    position, slot); ckpt_state / ckpt_conv the checkpoint slots."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    n = 0 if ckpt is None else int(ckpt.shape[0])
    _check(load_library().gdn_prefill_chunked_ckpt(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(conv_state), _ptr(recurrent_state), _ptr(out),
        _ptr(workspace), int(workspace_bytes), _ptr(ckpt), n, _ptr(ckpt_state), _ptr(ckpt_conv),
        int(ckpt_state.shape[0]) if ckpt_state is not None else 0, _stream(stream)))


def prefill_chunked_static_scratch(dims: Dims, inputs: Inputs, conv_state, recurrent_state, out, stream=None):
    """gdn_prefill_chunked with the library's own 64 MiB static scratch (for
    callers that cannot allocate device memory)."""
    _check(load_library().gdn_prefill_chunked_static_scratch(ctypes.byref(dims), ctypes.byref(inputs),
                                                             _ptr(conv_state), _ptr(recurrent_state), _ptr(out),
                                                             _stream(stream)))


def state_copy(dims: Dims, src_state, src_conv, dst_state, dst_conv, src_slot, dst_slot, n, n_src_slots,
               n_dst_slots, stream=None):
    _check(load_library().gdn_state_copy(ctypes.byref(dims), _ptr(src_state), _ptr(src_conv), _ptr(dst_state),
                                         _ptr(dst_conv), _ptr(src_slot), _ptr(dst_slot), int(n),
                                         int(n_src_slots), int(n_dst_slots), _stream(stream)))


def commit_accepted(dims: Dims, n_layers, paths, ckpt_state, ckpt_conv, state_pool, conv_pool, accept_len, dst_slot,
                    winner=None, stream=None):
    """gdn_commit_accepted: every layer's winning checkpoint into its pool, one launch."""
    _check(load_library().gdn_commit_accepted(ctypes.byref(dims), int(n_layers), int(paths), _ptr(ckpt_state),
                                              _ptr(ckpt_conv), _ptr(state_pool), _ptr(conv_pool), _ptr(accept_len),
                                              _ptr(dst_slot), _ptr(winner), _stream(stream)))


def commit_source_slot(accept_len, T: int) -> tuple[int, int]:
    """The checkpoint to commit after a verify call of len(accept_len) paths x T
    draft tokens: (winner path, checkpoint slot for gdn_state_copy's src_slot).

    generate.py (sparkle, mlx_streaming/mtp), commit_tree_row(row, accepted_len):
    the winner is the first path with the longest accept length (ties go to the
    lower index); its checkpoint slot is winner * T + L - 1, the state after its
    L accepted tokens. L = 0 commits nothing: slot -1 (gdn_state_copy skips it).
    Host arithmetic only."""
    L = [int(x) for x in accept_len]
    if not L or any(x < 0 or x > T for x in L):
        raise ValueError("accept lengths must lie in [0, T] and there must be at least one path")
    win = max(range(len(L)), key=lambda p: (L[p], -p))
    return win, (win * T + L[win] - 1 if L[win] > 0 else -1)


def in_proj(dims: Dims, hidden, w_in, q, k, v, z, a, b, stream=None):
    """gdn_in_proj: hidden [M, H] x w_in [N, H]^T split into q, k, v, z, a, b."""
    H = int(hidden.shape[-1])
    M = hidden.numel() // H
    _check(load_library().gdn_in_proj(ctypes.byref(dims), M, H, _ptr(hidden), _ptr(w_in), _ptr(q), _ptr(k), _ptr(v),
                                      _ptr(z), _ptr(a), _ptr(b), _stream(stream)))


def out_proj(o, w_out, y, stream=None):
    """gdn_out_proj: y [M, H] = o [M, V] x w_out [H, V]^T."""
    V, H = int(o.shape[-1]), int(w_out.shape[0])
    M = o.numel() // V
    _check(load_library().gdn_out_proj(M, H, V, _ptr(o), _ptr(w_out), _ptr(y), _stream(stream)))


def _layout(x, name):
    """(tokens, heads, head_dim, elements between tokens) of a bf16 tensor [tokens, heads, head_dim] or
    [rows, tokens, heads, head_dim] whose heads lie together and whose tokens are evenly spaced."""
    shape, st = x.shape, x.stride()
    rank = len(shape)
    if rank == 3 and st[1:] == (shape[2], 1) and x.dtype is _BF16:  # the usual case: 0.5 us on the host in place of 0.9
        return *shape, st[0]
    if x.dtype is not _BF16 or not 3 <= rank <= 4:
        raise ValueError(f"{name} must be a bf16 tensor [tokens, heads, head_dim] or [rows, tokens, heads, head_dim]")
    heads, d = shape[-2], shape[-1]
    n = shape[0] if rank == 3 else shape[0] * shape[1]
    if st[-1] != 1 or (st[-2] != d and heads > 1) or (rank == 4 and shape[0] > 1 and st[0] != shape[1] * st[1]):
        raise ValueError(f"{name} must have dense heads and evenly spaced tokens")
    return n, heads, d, st[-3]


def _spaced(x, stride, name):
    """Refuses a tensor [.., tokens, heads, head_dim] whose tokens are not `stride` elements apart, as the sizes say."""
    if isinstance(x, torch.Tensor):
        st = x.stride()  # all at once: 0.2 us on the host, one after the other 0.3
        if len(st) >= 3 and st[-3] != stride and x.shape[-3] > 1:
            raise ValueError(f"{name}'s tokens are {st[-3]} elements apart, the sizes say {stride}")


def _tokens(x, n, heads, d, stride, name):
    """_ptr of x, which must be n tokens (or more) of `heads` heads of d, `stride` elements apart, as the sizes say."""
    if x is None or x.__class__ is int:
        return x
    # the usual case at once: 0.3 us on the host in place of 1
    if x.stride() != (stride, d, 1) or x.shape != (n, heads, d) or x.dtype is not _BF16:
        tokens, h, dim, apart = _layout(x, name)
        if tokens < n or h != heads or dim != d or (apart != stride and n > 1):
            raise ValueError(f"{name} is {tokens} tokens of {h} heads of {dim}, {apart} elements apart, the sizes say {n}, "
                             f"{heads}, {d}, {stride}")
    return x.data_ptr()


def make_rope_dims(q, k, rot_dim, n_axes=1, kv_rows=None, adjacent=False, eps=1e-6, v=None) -> RopeDims:
    """Sizes and token strides of a head_norm_rope call on q [n, Hq, d] and k [n, Hk, d]; v's tokens are spaced as
    k's unless v is given. kv_rows: rows of the pools (n when they hold the tokens themselves)."""
    n, hq, d, qs = _layout(q, "q")
    _, hk, _, ks = _layout(k, "k")
    return RopeDims(n, hq, hk, d, rot_dim, n_axes, int(adjacent), eps, qs, ks, ks if v is None else _layout(v, "v")[3],
                    n if kv_rows is None else kv_rows)


def head_norm_rope(dims: RopeDims, q, k, v, q_weight, k_weight, positions, inv_freq, q_out, k_out, v_out, axis=None,
                   kv_index=None, stream=None):
    """gdn_head_norm_rope: per-head norms of q and k, the rotation by positions int32 [axes, n] with inv_freq fp64
    [rot_dim/2] (axis uint8 [rot_dim/2]: each pair's position axis), K and V to the rows kv_index int32 [n] of the
    pools k_out, v_out [kv_rows, Hk, d]."""
    _spaced(v, dims.v_stride, "v")
    _check(load_library().gdn_head_norm_rope(
        ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(q_weight), _ptr(k_weight), _ptr(positions), _ptr(inv_freq),
        _ptr(axis), _ptr(kv_index), _ptr(q_out), _ptr(k_out), _ptr(v_out), _stream(stream)))


def make_attn_dims(q, k, B, T=1, n_groups=0, scale=None) -> AttnDims:
    """Sizes and strides of an attention call: q [n, Hq, d] or [B, T, Hq, d], k (and v, spaced alike) the pool
    [kv_rows, Hk, d]."""
    n, hq, d, qs = _layout(q, "q")
    rows, hk, _, ks = _layout(k, "k")
    return AttnDims(B, T, n, n_groups, hq, hk, d, d ** -0.5 if scale is None else scale, qs, ks, rows)


def attn_prefill(dims: AttnDims, q, k, v, cu_seqlens, out, kv_start=None, kv_len=None, stream=None):
    """gdn_attn_prefill: causal attention of packed prompts over their extents of the pools k, v."""
    _spaced(k, dims.kv_stride, "k")
    _spaced(v, dims.kv_stride, "v")
    _check(load_library().gdn_attn_prefill(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens),
                                           _ptr(kv_start), _ptr(kv_len), _ptr(out), _stream(stream)))


def attn_workspace_size(dims: AttnDims) -> int:
    """Workspace bytes of attn_shared_prefix."""
    return int(load_library().gdn_attn_workspace_size(ctypes.byref(dims)))


def attn_workspace(dims: AttnDims, device="cuda") -> torch.Tensor:
    """A workspace tensor for attn_shared_prefix, reusable from call to call on one stream."""
    return torch.empty(max(attn_workspace_size(dims), 1), dtype=torch.uint8, device=device)


def attn_shared_prefix(dims: AttnDims, q, k, v, group_rows, prefix_start, prefix_len, suffix_start, suffix_len, out,
                       workspace, q_len=None, stream=None):
    """gdn_attn_shared_prefix: q [B, T, Hq, d] over each group's shared prefix extent and each row's own extent."""
    _spaced(k, dims.kv_stride, "k")
    _spaced(v, dims.kv_stride, "v")
    _check(load_library().gdn_attn_shared_prefix(
        ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(group_rows), _ptr(prefix_start), _ptr(prefix_len),
        _ptr(suffix_start), _ptr(suffix_len), _ptr(q_len), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size() if workspace is not None else 0, _stream(stream)))


def accept_draft(tokens, target_probs, draft_probs, uniform, accept_len, next_token, n_tokens=None, stream=None):
    """gdn_accept_draft: tokens int32 [B, T], target_probs fp32 [B, T, V], draft_probs fp32 [B, T-1, V] or None
    (certain drafts), uniform fp32 [B, T] -> accept_len, next_token int32 [B]."""
    B, T, V = target_probs.shape
    _check(load_library().gdn_accept_draft(B, T, V, _ptr(tokens), _ptr(target_probs), _ptr(draft_probs), _ptr(uniform),
                                           _ptr(n_tokens), _ptr(accept_len), _ptr(next_token), _stream(stream)))


def _page_pool(pool, heads, d):
    """(pages, heads) of a pool uint8 [n_pages, heads, 72 d]; heads None: any. Calls look at its strides."""
    shape = pool.shape
    if pool.dtype is not _U8 or len(shape) != 3 or (heads is not None and shape[1] != heads) or shape[2] != 72 * d:
        raise ValueError(f"the pool must be a dense uint8 tensor [n_pages, {heads or 'heads'}, {72 * d}]")
    return shape[0], shape[1]


def kv4_pool(n_pages, n_kv_heads, head_dim, device="cuda") -> torch.Tensor:
    """A pool of n_pages pages of 64 tokens, uint8 [n_pages, n_kv_heads, 72 head_dim]."""
    return torch.zeros((n_pages, n_kv_heads, 72 * head_dim), dtype=torch.uint8, device=device)


def make_kv4_dims(k, pool, v=None, k_exp=0, v_exp=0) -> Kv4Dims:
    """Sizes of a kv4_store / kv4_load call on k [n, Hk, d]; v's tokens are spaced as k's unless v is given."""
    n, hk, d, ks = _layout(k, "k")
    return Kv4Dims(n, hk, d, _page_pool(pool, hk, d)[0], k_exp, v_exp, ks, ks if v is None else _layout(v, "v")[3])


def _kv4_arguments(dims, k, v, kv_index, pool):
    """The four addresses of a kv4_store or kv4_load call."""
    n, heads, d = dims.n_tokens, dims.n_kv_heads, dims.head_dim
    _here(pool, "pool")
    return (_tokens(k, n, heads, d, dims.k_stride, "k"), _tokens(v, n, heads, d, dims.v_stride, "v"),
            _array(kv_index, _I32, 4 * n, "kv_index"), _array(pool, _U8, dims.n_pages * heads * 72 * d, "pool"))


def kv4_store(dims: Kv4Dims, k, v, kv_index, pool, stream=None):
    """gdn_kv4_store: k, v bf16 [n, Hk, d] into the pool rows kv_index int32 [n] (-1: not kept), 4 bits each."""
    args = _kv4_arguments(dims, k, v, kv_index, pool)
    _check(load_library().gdn_kv4_store(ctypes.byref(dims), *args, _stream(stream)))


def kv4_load(dims: Kv4Dims, pool, kv_index, k, v, stream=None):
    """gdn_kv4_load: pool rows kv_index int32 [n] to k, v bf16 [n, Hk, d], exactly as attn_kv4 uses them."""
    to_k, to_v, index, pages = _kv4_arguments(dims, k, v, kv_index, pool)
    _check(load_library().gdn_kv4_load(ctypes.byref(dims), pages, index, to_k, to_v, _stream(stream)))


def _row_tokens(q):
    """(rows, tokens, heads, head_dim, elements between tokens) of a bf16 tensor [rows, tokens, heads, head_dim]."""
    shape, st = q.shape, q.stride()
    if q.dtype is not _BF16 or len(shape) != 4:
        raise ValueError("q must be a bf16 tensor [rows, tokens, heads, head_dim]")
    B, T, hq, d = shape
    qs = st[0] if T == 1 else st[1]  # the stride of a dimension of one token says nothing
    if st[3] != 1 or (st[2] != d and hq > 1) or (T > 1 and B > 1 and st[0] != T * qs):
        raise ValueError("q must have dense heads and evenly spaced tokens")
    return B, T, hq, d, qs


def make_attn_kv4_dims(q, pool, page_table, scale=None, k_exp=0, v_exp=0) -> AttnKv4Dims:
    """Sizes of an attn_kv4 call: q [B, T, Hq, d], one layer's pool, page_table int32 [B, max_pages]."""
    B, T, hq, d, qs = _row_tokens(q)
    pages, hk = _page_pool(pool, None, d)
    table = page_table.shape
    if page_table.dtype is not _I32 or len(table) != 2 or table[0] != B:
        raise ValueError("the page table must be a dense int32 tensor [rows, max_pages]")
    return AttnKv4Dims(B, T, hq, hk, d, pages, table[1], k_exp, v_exp, d ** -0.5 if scale is None else scale, qs)


def attn_kv4_workspace_size(dims: AttnKv4Dims) -> int:
    """Workspace bytes of attn_kv4."""
    return int(load_library().gdn_attn_kv4_workspace_size(ctypes.byref(dims)))


def attn_kv4_workspace(dims: AttnKv4Dims, device="cuda") -> torch.Tensor:
    """A workspace tensor for attn_kv4, reusable from call to call on one stream."""
    return torch.empty(max(attn_kv4_workspace_size(dims), 1), dtype=torch.uint8, device=device)


def attn_kv4(dims: AttnKv4Dims, q, pool, page_table, kv_len, out, workspace, q_len=None, stream=None):
    """gdn_attn_kv4: q [B, T, Hq, d] over the pages of each row, kv_len int32 [B] tokens of it."""
    B, T, hq, hk, d = dims.B, dims.T, dims.n_q_heads, dims.n_kv_heads, dims.head_dim
    if q is not None and q.__class__ is not int:
        qs = dims.q_stride
        if q.stride() != (T * qs, qs, d, 1) or q.shape != (B, T, hq, d) or q.dtype is not _BF16:  # not the usual case
            rows, *sizes, stride = _row_tokens(q)
            if rows < B or sizes != [T, hq, d] or (stride != qs and B * T > 1):
                raise ValueError(f"q is {[rows, *sizes]}, its tokens {stride} elements apart, the sizes say {[B, T, hq, d]}, "
                                 f"{qs}")
    _here(pool, "pool")
    _check(load_library().gdn_attn_kv4(
        ctypes.byref(dims), _ptr(q), _array(pool, _U8, dims.n_pages * hk * 72 * d, "pool"),
        _array(page_table, _I32, 4 * B * dims.max_pages, "page_table"), _array(kv_len, _I32, 4 * B, "kv_len"),
        _array(q_len, _I32, 4 * B, "q_len"), _array(out, _BF16, 2 * B * T * hq * d, "out"), *_space(workspace),
        _stream(stream)))


def make_beam_dims(logits, eos=-1) -> BeamDims:
    """Sizes of a beam_select call on logits [groups, beams, V], fp32 or bf16, rows evenly spaced."""
    shape, st, half = logits.shape, logits.stride(), logits.dtype is _BF16
    if len(shape) != 3 or not (half or logits.dtype is _F32):
        raise ValueError("logits must be fp32 or bf16 [groups, beams, vocab]")
    g, w, v = shape
    stride = st[1] if w > 1 else st[0] if g > 1 else v
    if (v > 1 and st[2] != 1) or (g > 1 and w > 1 and st[0] != w * st[1]):
        raise ValueError("logits must have dense rows, evenly spaced")
    return BeamDims(g, w, v, half, -1 if eos is None else eos, stride)


def beam_workspace(logits) -> torch.Tensor:
    """A workspace tensor for beam_select on logits of this shape, reusable from call to call on one stream."""
    n = int(load_library().gdn_beam_workspace_size(ctypes.byref(make_beam_dims(logits))))
    return torch.empty(max(n, 1), dtype=torch.uint8, device=logits.device)


def beam_select(logits, scores, parent, token, new_scores, workspace, done=None, new_done=None, eos=-1, stream=None):
    """gdn_beam_select: the best continuations of each group's beams; logits [groups, beams, V], scores fp32 and done
    uint8 [groups, beams] -> parent (row numbers), token int32, new_scores, new_done [groups, beams]."""
    dims = make_beam_dims(logits, eos)
    _here(logits, "logits")
    rows = dims.n_groups * dims.beams
    size = 4 * rows
    _check(load_library().gdn_beam_select(
        ctypes.byref(dims), _ptr(logits), _array(scores, _F32, size, "scores"), _array(_flags(done), _U8, rows, "done"),
        _array(parent, _I32, size, "parent"), _array(token, _I32, size, "token"), _array(new_scores, _F32, size, "new_scores"),
        _array(_flags(new_done), _U8, rows, "new_done"), *_space(workspace), _stream(stream)))


_FORK_ROWS = ("parent", "n_new", "kv_len", "kv_len_out", "page_src", "page_dst", "state_idx", "state_idx_out", "state_src",
              "state_dst")


def cache_fork(page_table, kv_len, page_table_out, kv_len_out, kv_index, page_src, page_dst, n_pages, parent=None,
               n_new=None, pinned=None, state_idx=None, state_idx_out=None, state_src=None, state_dst=None, stream=None):
    """gdn_cache_fork: rows become copies of the rows parent int32 [R] and take n_new tokens (kv_index int32 [R, T]);
    page_src / page_dst and state_src / state_dst int32 [R] are slots_copy's."""
    shape = page_table.shape
    if len(shape) != 2 or page_table_out.shape != shape:
        raise ValueError("page_table and page_table_out must be of one shape [rows, max_pages]")
    rows, width = shape
    T = 0 if kv_index is None else kv_index.shape[1]
    dims = ForkDims(rows, T, width, n_pages)
    _here(page_table, "page_table")
    table, table_out = _arrays(_I32, 4 * rows * width, ("page_table", "page_table_out"), page_table, page_table_out)
    parent, n_new, kv_len, kv_len_out, *copies = _arrays(
        _I32, 4 * rows, _FORK_ROWS, parent, n_new, kv_len, kv_len_out, page_src, page_dst, state_idx, state_idx_out, state_src,
        state_dst)
    _check(load_library().gdn_cache_fork(
        ctypes.byref(dims), parent, n_new, table, kv_len, _array(_flags(pinned), _U8, n_pages, "pinned"), table_out, kv_len_out,
        _array(kv_index, _I32, 4 * rows * T, "kv_index"), *copies, _stream(stream)))


def slots_copy(pools, stream=None):
    """gdn_slots_copy: pools (at most MAX_SLOT_POOLS) of (tensor [n_layers, n_slots, ...], src, dst int32 [n]): in every
    layer slot src[i] is copied to slot dst[i]; -1 skips a pair."""
    args = []
    for x, src, dst in pools:
        shape, n = x.shape, src.numel()
        if not x.is_contiguous() or len(shape) < 2 or n != dst.numel():
            raise ValueError("a pool must be a dense tensor [n_layers, n_slots, ...], src and dst of one length")
        layers, slots = shape[0], shape[1]
        slot = x.nbytes // (layers * slots) if layers * slots else x.element_size() * math.prod(shape[2:])
        _here(x, "a pool")
        args.append(SlotPool(x.data_ptr(), _array(src, _I32, 4 * n, "src"), _array(dst, _I32, 4 * n, "dst"), slot, n, layers, slots))
    n = len(args)
    array = _pools_of[n] if n <= MAX_SLOT_POOLS else SlotPool * n
    _check(load_library().gdn_slots_copy(array(*args), n, _stream(stream)))


def check_status(stream=None):
    """Synchronise the stream and raise on a device-detected error."""
    _check(load_library().gdn_check_status(_stream(stream)))


def workspace(dims: Dims, packed: bool = False, device="cuda") -> torch.Tensor:
    """A workspace tensor for gdn_prefill_chunked (torch allocations are
    256-byte aligned); packed: the call passes cu_seqlens."""
    n = prefill_workspace_size(dims, packed)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device)
