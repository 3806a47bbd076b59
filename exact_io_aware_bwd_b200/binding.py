"""ctypes binding of libfa_b200.so: the C ABI of include/fa.h, one Python
function per entry point with the same name, plus two conveniences that
allocate outputs with PyTorch.  Argument marshalling only: every step of the
computation runs in the library's CUDA kernels.  There is no fallback: if the
library cannot be loaded, every call raises.
"""

from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

from .build import LIB_PATH

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_MISALIGNED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(6)
FA_BF16, FA_FP16 = 0, 1

_DTYPES = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16}

_lock = threading.Lock()
_lib = None


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fa_status_string(status)} (status {status})")


def library_path() -> str:
    return os.environ.get("FA_B200_LIB", LIB_PATH)


def load():
    """Load libfa_b200.so (built in-tree by build.build()); raise if absent."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with exact_io_aware_bwd_b200.build.build() "
                    "(there is no fallback implementation)")
            lib = ctypes.CDLL(path)
            vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
            lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
            lib.fa_fwd.restype = i
            lib.fa_bwd_workspace_bytes.argtypes = [i, i, i, i, i]
            lib.fa_bwd_workspace_bytes.restype = ctypes.c_size_t
            lib.fa_bwd.argtypes = ([vp] * 9 + [i, i, i, i, i, f, i, i, vp, ctypes.c_size_t, vp])
            lib.fa_bwd.restype = i
            lib.fa_fwd_window.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
            lib.fa_fwd_window.restype = i
            lib.fa_bwd_window.argtypes = ([vp] * 9 + [i, i, i, i, i, f, i, i, vp, ctypes.c_size_t, vp])
            lib.fa_bwd_window.restype = i
            u64 = ctypes.c_uint64
            lib.fa_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, f, u64, i, vp]
            lib.fa_fwd_dropout.restype = i
            lib.fa_bwd_dropout.argtypes = ([vp] * 9 + [i, i, i, i, i, f, i, f, u64, i, vp,
                                                       ctypes.c_size_t, vp])
            lib.fa_bwd_dropout.restype = i
            lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, f, f, f, i, i, vp]
            lib.fa_fwd_fp8.restype = i
            lib.fa_fwd_blockmask.argtypes = [vp] * 5 + [i] * 5 + [f, i, vp, i, i, vp]
            lib.fa_fwd_blockmask.restype = i
            lib.fa_bwd_blockmask_workspace_bytes.argtypes = [i, i, i, i, i]
            lib.fa_bwd_blockmask_workspace_bytes.restype = ctypes.c_size_t
            lib.fa_bwd_blockmask.argtypes = ([vp] * 9 + [i] * 5 + [f, i, vp, i, i, vp, ctypes.c_size_t, vp])
            lib.fa_bwd_blockmask.restype = i
            lib.fa_decode_workspace_bytes.argtypes = [i, i, i, i, i, i]
            lib.fa_decode_workspace_bytes.restype = ctypes.c_size_t
            lib.fa_decode_paged.argtypes = ([vp] * 7 + [i] * 8 + [f, i, vp, ctypes.c_size_t, vp])
            lib.fa_decode_paged.restype = i
            i64p, sz = ctypes.POINTER(ctypes.c_int64), ctypes.c_size_t
            lib.fa_append_paged.argtypes = [vp, vp, vp, i64p] + [vp] * 8 + [i] * 10 + [i, vp]
            lib.fa_append_paged.restype = i
            lib.fa_fwd_paged_workspace_bytes.argtypes = [i] * 7
            lib.fa_fwd_paged_workspace_bytes.restype = sz
            lib.fa_fwd_paged.argtypes = [vp] * 8 + [i] * 8 + [f, i, vp, sz, vp]
            lib.fa_fwd_paged.restype = i
            lib.fa_decode_prefix_workspace_bytes.argtypes = [i] * 8
            lib.fa_decode_prefix_workspace_bytes.restype = sz
            lib.fa_decode_prefix.argtypes = [vp] * 7 + [i] * 9 + [f, i, vp, sz, vp]
            lib.fa_decode_prefix.restype = i
            lib.fa_get_device_status.argtypes = [vp]
            lib.fa_get_device_status.restype = i
            lib.fa_peek_device_status_word.argtypes = [vp]
            lib.fa_peek_device_status_word.restype = ctypes.c_uint32
            lib.fa_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
            lib.fa_selftest_wait_timeout.restype = i
            lib.fa_set_profile_events.argtypes = [i, vp, vp]
            lib.fa_set_profile_events.restype = i
            lib.fa_set_bwd_max_blocks.argtypes = [i]
            lib.fa_set_bwd_max_blocks.restype = i
            lib.fa_status_string.argtypes = [i]
            lib.fa_status_string.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


def _check(status: int, where: str):
    if status != FA_OK:
        raise FaError(status, where)


def _dims(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"q and k must be 4-D [B, H, N, d], got {tuple(q.shape)} and {tuple(k.shape)}")
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    return B, Hq, Hkv, N, d


_E4M3 = (torch.uint8, torch.float8_e4m3fn)


def _expect(where, *spec):
    """Checks (name, tensor, shape, dtypes) entries before any pointer reaches
    the library: the shape (None: any), the dtype (None: any), a dense
    row-major layout, and one CUDA device for all.  The library reads every
    tensor as dense rows, so a strided view would be read wrongly rather than
    rejected there.  None and raw integer addresses pass through unchecked."""
    spec = [(name, t, shape, dtypes) for name, t, shape, dtypes in spec
            if t is not None and not isinstance(t, int)]
    for name, t, shape, dtypes in spec:
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if dtypes is not None and t.dtype not in dtypes:
            raise TypeError(f"{where}: {name} has dtype {t.dtype}, expected one of {list(dtypes)}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous")
    dev = None
    for name, t, _, _ in spec:
        if not t.is_cuda:
            raise ValueError(f"{where}: {name} must be on a CUDA device")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{where}: all tensors must be on one device ({name} is on {t.device})")


def _expect_attention(where, q, k, v, o, lse, dout=None, dq=None, dk=None, dv=None, workspace=None):
    """_expect for the attention entry points; returns (B, Hq, Hkv, N, d)."""
    B, Hq, Hkv, N, d = _dims(q, k)
    if q.dtype not in _DTYPES:
        raise TypeError(f"{where}: q has dtype {q.dtype}, expected bfloat16 or float16")
    same = (q.dtype,)
    qs, ks = (B, Hq, N, d), (B, Hkv, N, d)
    _expect(where, ("q", q, qs, same), ("k", k, ks, same), ("v", v, ks, same), ("o", o, qs, same),
            ("lse", lse, (B, Hq, N), (torch.float32,)), ("dout", dout, qs, same),
            ("dq", dq, qs, same), ("dk", dk, ks, same), ("dv", dv, ks, same),
            ("workspace", workspace, None, None))
    return B, Hq, Hkv, N, d


def fa_status_string(status: int) -> str:
    return load().fa_status_string(int(status)).decode()


def fa_fwd(q, k, v, o, lse, scale: float, causal: bool, stream=None) -> None:
    """O and lse (natural log) of exact attention into the given tensors.
    q [B,Hq,N,d], k/v [B,Hkv,N,d] (bf16 or fp16, contiguous, on the GPU)."""
    B, Hq, Hkv, N, d = _expect_attention("fa_fwd", q, k, v, o, lse)
    st = load().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d,
                       float(scale), int(bool(causal)), _DTYPES[q.dtype], _stream(stream))
    _check(st, "fa_fwd")


def fa_fwd_window(q, k, v, o, lse, scale: float, window: int, stream=None) -> None:
    """Causal sliding-window forward: query i sees keys i-window+1 .. i."""
    B, Hq, Hkv, N, d = _expect_attention("fa_fwd_window", q, k, v, o, lse)
    st = load().fa_fwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d,
                              float(scale), int(window), _DTYPES[q.dtype], _stream(stream))
    _check(st, "fa_fwd_window")


def fa_bwd_window(q, k, v, o, dout, lse, dq, dk, dv, scale: float, window: int, workspace,
                  stream=None) -> None:
    """Backward of fa_fwd_window with the same window."""
    B, Hq, Hkv, N, d = _expect_attention("fa_bwd_window", q, k, v, o, lse, dout, dq, dk, dv, workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().fa_bwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                              _ptr(dk), _ptr(dv), B, Hq, Hkv, N, d, float(scale), int(window),
                              _DTYPES[q.dtype], _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "fa_bwd_window")


def fa_fwd_dropout(q, k, v, o, lse, scale: float, causal: bool, p_drop: float, seed: int,
                   stream=None) -> None:
    """Forward with dropout on the probabilities (8-bit threshold round(256 p))."""
    B, Hq, Hkv, N, d = _expect_attention("fa_fwd_dropout", q, k, v, o, lse)
    st = load().fa_fwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d,
                               float(scale), int(bool(causal)), float(p_drop),
                               int(seed) & 0xFFFFFFFFFFFFFFFF, _DTYPES[q.dtype], _stream(stream))
    _check(st, "fa_fwd_dropout")


def fa_fwd_fp8(q8, k8, v8, o, lse, scale: float, descale, causal: bool, stream=None) -> None:
    """FP8 forward: q8 [B,Hq,N,128], k8/v8 [B,Hkv,N,128] E4M3 codes (uint8 or
    float8_e4m3fn tensors on the GPU), descale = (delta_q, delta_k, delta_v);
    O (bf16 or fp16, its dtype picks the output type) and lse fp32."""
    B, Hq, Hkv, N, d = _dims(q8, k8)
    if o is None or isinstance(o, int) or o.dtype not in _DTYPES:
        raise TypeError("fa_fwd_fp8: o must be a bfloat16 or float16 tensor (its dtype picks the output type)")
    _expect("fa_fwd_fp8", ("q8", q8, (B, Hq, N, d), _E4M3), ("k8", k8, (B, Hkv, N, d), _E4M3),
            ("v8", v8, (B, Hkv, N, d), _E4M3), ("o", o, (B, Hq, N, d), None),
            ("lse", lse, (B, Hq, N), (torch.float32,)))
    dq, dk, dv = (float(x) for x in descale)
    st = load().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d,
                           float(scale), dq, dk, dv, int(bool(causal)), _DTYPES[o.dtype],
                           _stream(stream))
    _check(st, "fa_fwd_fp8")


def attention_fwd_fp8(q8, k8, v8, descale, scale: float | None = None, causal: bool = False,
                      out_dtype=torch.bfloat16, stream=None):
    """Allocates O (out_dtype) and lse and runs fa_fwd_fp8; returns (O, lse)."""
    B, Hq, Hkv, N, d = _dims(q8, k8)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty((B, Hq, N, d), device=q8.device, dtype=out_dtype)
    lse = torch.empty((B, Hq, N), device=q8.device, dtype=torch.float32)
    fa_fwd_fp8(q8, k8, v8, o, lse, scale, descale, causal, stream)
    return o, lse


def fa_bwd_dropout(q, k, v, o, dout, lse, dq, dk, dv, scale: float, causal: bool, p_drop: float,
                   seed: int, workspace, stream=None) -> None:
    """Backward of fa_fwd_dropout with the same p_drop and seed."""
    B, Hq, Hkv, N, d = _expect_attention("fa_bwd_dropout", q, k, v, o, lse, dout, dq, dk, dv, workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().fa_bwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                               _ptr(dk), _ptr(dv), B, Hq, Hkv, N, d, float(scale),
                               int(bool(causal)), float(p_drop), int(seed) & 0xFFFFFFFFFFFFFFFF,
                               _DTYPES[q.dtype], _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "fa_bwd_dropout")


def _block_mask(where, block_mask, Hq, N, device):
    """(tensor, mask_per_head) of a block mask over 128 x 128 blocks: a bool
    or uint8 CUDA tensor [nb, nb] (every head) or [Hq, nb, nb], nb = ceil(N/128)."""
    nb = -(-N // 128)
    if block_mask is None or isinstance(block_mask, int):
        raise ValueError(f"{where}: a block mask tensor is required")
    if block_mask.dtype not in (torch.uint8, torch.bool):
        raise TypeError(f"{where}: block_mask has dtype {block_mask.dtype}, expected uint8 or bool")
    if tuple(block_mask.shape) == (nb, nb):
        per_head = 0
    elif tuple(block_mask.shape) == (Hq, nb, nb):
        per_head = 1
    else:
        raise ValueError(f"{where}: block_mask has shape {tuple(block_mask.shape)}, expected "
                         f"({nb}, {nb}) or ({Hq}, {nb}, {nb})")
    if not block_mask.is_cuda or block_mask.device != device:
        raise ValueError(f"{where}: block_mask must be on {device}")
    if not block_mask.is_contiguous():
        raise ValueError(f"{where}: block_mask must be contiguous")
    return block_mask.view(torch.uint8) if block_mask.dtype == torch.bool else block_mask, per_head


def fa_fwd_blockmask(q, k, v, o, lse, scale: float, causal: bool, block_mask, stream=None) -> None:
    """Forward under a block mask over 128-row x 128-key blocks (see
    _block_mask for its layout); combined with the causal mask when causal."""
    B, Hq, Hkv, N, d = _expect_attention("fa_fwd_blockmask", q, k, v, o, lse)
    m, per_head = _block_mask("fa_fwd_blockmask", block_mask, Hq, N, q.device)
    st = load().fa_fwd_blockmask(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d,
                                 float(scale), int(bool(causal)), _ptr(m), per_head, _DTYPES[q.dtype],
                                 _stream(stream))
    _check(st, "fa_fwd_blockmask")


def fa_bwd_blockmask_workspace_bytes(B: int, Hq: int, Hkv: int, N: int, d: int) -> int:
    return int(load().fa_bwd_blockmask_workspace_bytes(B, Hq, Hkv, N, d))


def fa_bwd_blockmask(q, k, v, o, dout, lse, dq, dk, dv, scale: float, causal: bool, block_mask,
                     workspace, stream=None) -> None:
    """Backward of fa_fwd_blockmask with the same mask; workspace of at least
    fa_bwd_blockmask_workspace_bytes(...) bytes."""
    B, Hq, Hkv, N, d = _expect_attention("fa_bwd_blockmask", q, k, v, o, lse, dout, dq, dk, dv,
                                         workspace)
    m, per_head = _block_mask("fa_bwd_blockmask", block_mask, Hq, N, q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().fa_bwd_blockmask(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                                 _ptr(dk), _ptr(dv), B, Hq, Hkv, N, d, float(scale), int(bool(causal)),
                                 _ptr(m), per_head, _DTYPES[q.dtype], _ptr(workspace), ws_bytes,
                                 _stream(stream))
    _check(st, "fa_bwd_blockmask")


def fa_bwd_workspace_bytes(B: int, Hq: int, Hkv: int, N: int, d: int) -> int:
    return int(load().fa_bwd_workspace_bytes(B, Hq, Hkv, N, d))


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, scale: float, causal: bool, workspace,
           stream=None) -> None:
    """dQ, dK, dV into the given tensors; workspace: a uint8 GPU tensor of at
    least fa_bwd_workspace_bytes(...) bytes."""
    B, Hq, Hkv, N, d = _expect_attention("fa_bwd", q, k, v, o, lse, dout, dq, dk, dv, workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                       _ptr(dk), _ptr(dv), B, Hq, Hkv, N, d, float(scale), int(bool(causal)),
                       _DTYPES[q.dtype], _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "fa_bwd")


def fa_get_device_status(stream=None) -> int:
    return int(load().fa_get_device_status(_stream(stream)))


def fa_peek_device_status_word(stream=None) -> int:
    return int(load().fa_peek_device_status_word(_stream(stream)))


def fa_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    return int(load().fa_selftest_wait_timeout(int(limit_ns), _stream(stream)))


KERNEL_FWD, KERNEL_BWD_MAIN = 1, 3


def fa_set_profile_events(kernel_id: int, start=None, stop=None) -> None:
    """Bracket every launch of a kernel with two CUDA events (torch.cuda.Event
    objects that have been recorded once, or raw handles); None clears."""
    h = lambda e: None if e is None else ctypes.c_void_p(e.cuda_event if hasattr(e, "cuda_event") else int(e))
    _check(load().fa_set_profile_events(int(kernel_id), h(start), h(stop)), "fa_set_profile_events")


def fa_set_bwd_max_blocks(max_blocks: int) -> None:
    """Cap the persistent blocks of the backward main pass (0: one per SM)."""
    _check(load().fa_set_bwd_max_blocks(int(max_blocks)), "fa_set_bwd_max_blocks")


def fa_decode_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, d: int, max_pages: int) -> int:
    return int(load().fa_decode_workspace_bytes(B, Hq, Hkv, Nq, d, max_pages))


def fa_decode_paged(q, k_cache, v_cache, block_table, seq_lens, o, lse, scale: float, workspace,
                    stream=None) -> None:
    """Decode over a paged cache: q [B,Hq,Nq,d]; caches [pages,Hkv,P,d];
    block_table [B,max_pages] and seq_lens [B] int32 on the GPU."""
    B, Hq, Nq, d = q.shape
    num_pages, Hkv, P, dk = k_cache.shape
    if dk != d or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError(f"incompatible shapes q{tuple(q.shape)} k_cache{tuple(k_cache.shape)}")
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("block_table and seq_lens must be int32")
    if q.dtype not in _DTYPES:
        raise TypeError(f"fa_decode_paged: q has dtype {q.dtype}, expected bfloat16 or float16")
    same = (q.dtype,)
    _expect("fa_decode_paged", ("q", q, None, same), ("k_cache", k_cache, None, same),
            ("v_cache", v_cache, None, same), ("block_table", block_table, (B, block_table.shape[-1]), None),
            ("seq_lens", seq_lens, (B,), None), ("o", o, (B, Hq, Nq, d), same),
            ("lse", lse, (B, Hq, Nq), (torch.float32,)), ("workspace", workspace, None, None))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().fa_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                _ptr(seq_lens), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, d, P,
                                block_table.shape[1], num_pages, float(scale), _DTYPES[q.dtype],
                                _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "fa_decode_paged")


# ------------------------------------------------------------ paged cache
#
# These calls run once per layer and token, so their checks are kept to a few
# microseconds: plain comparisons, one pass over the tensors.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _fits(where, dev, *spec):
    """Says what is wrong: each (name, tensor, shape, dtype) must have the
    shape and dtype (None: any), a dense layout and CUDA device `dev`; those
    that a call may leave out pass as None."""
    for name, t, shape, dtype in spec:
        if t is None and name in ("new_lens", "q_out", "k_out", "inv_freq", "workspace"):
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{where}: {name} must be a tensor")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if dtype is not None and t.dtype is not dtype:
            raise TypeError(f"{where}: {name} has dtype {t.dtype}, expected {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous")
        if t.get_device() != dev:
            if dev < 0 or not t.is_cuda:
                raise ValueError(f"{where}: {name} must be on a CUDA device")
            raise ValueError(f"{where}: all tensors must be on one device ({name} is on {t.device})")
    if dev < 0:
        raise ValueError(f"{where}: the tensors must be on a CUDA device")


def _four_d(where, *named):
    for name, t in named:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{where}: {name} must be a tensor")
        if t.dim() != 4:
            raise ValueError(f"{where}: {name} must be 4-D, got {tuple(t.shape)}")


def _table_width(where, block_table):
    if not isinstance(block_table, torch.Tensor):
        raise TypeError(f"{where}: block_table must be a tensor")
    if block_table.dim() != 2:
        raise ValueError(f"{where}: block_table must be 2-D, got {tuple(block_table.shape)}")
    return block_table.shape[1]


def _handle(dev, stream):
    """The stream of a call: the current one of the tensors' device, whichever
    device is current, when none is given."""
    if stream is None:
        return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _launch(fn, where, dev, *args):
    """fn(*args) with device `dev` current."""
    if dev == _current_device():
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st != FA_OK:
        raise FaError(st, where)


_NineStrides = ctypes.c_int64 * 9


def fa_append_paged(q, k, v, q_out, k_out, k_cache, v_cache, block_table, seq_lens, new_lens, inv_freq,
                    interleaved: bool = False, stream=None) -> None:
    """Appends k, v [B,Hkv,N,d] to a paged cache [pages,Hkv,P,d], k rotated by
    its position; q [B,Hq,N,d] is rotated into q_out (both None: keys and
    values only), and the rotated k also written to k_out when given.  q, k, v
    may be strided (contiguous rows); seq_lens [B] counts the new tokens, of
    which sequence b has new_lens[b] (None: N); inv_freq fp32 [rot/2] or None
    (no rotation)."""
    where = "fa_append_paged"
    try:
        dt, dev, kv = k.dtype, k.get_device(), k.shape
        cache, lens = k_cache.shape, seq_lens.shape
        B, Hkv, N, d = kv
        num_pages, Hc, P, dc = cache
        Bt, max_pages = block_table.shape
        i32, rot, Hq = torch.int32, 0, Hkv
        fine = (dev >= 0 and Hc == Hkv and dc == d and Bt == B and lens == (B,) and v.shape == kv and v.dtype is dt
                and v.get_device() == dev and v_cache.shape == cache and k_cache.dtype is dt and v_cache.dtype is dt
                and k_cache.get_device() == dev and v_cache.get_device() == dev and k_cache.is_contiguous()
                and v_cache.is_contiguous() and block_table.dtype is i32 and seq_lens.dtype is i32
                and block_table.get_device() == dev and seq_lens.get_device() == dev and block_table.is_contiguous()
                and seq_lens.is_contiguous())
        dense = k.is_contiguous() and v.is_contiguous()
        if q is not None:
            Bq, Hq, Nq, dq = qs = q.shape
            fine = (fine and Bq == B and Nq == N and dq == d and q.dtype is dt and q.get_device() == dev
                    and q_out.shape == qs and q_out.dtype is dt and q_out.get_device() == dev and q_out.is_contiguous())
            dense = dense and q.is_contiguous()
        elif q_out is not None:
            fine = False
        if new_lens is not None:
            fine = (fine and new_lens.shape == lens and new_lens.dtype is i32 and new_lens.get_device() == dev
                    and new_lens.is_contiguous())
        if k_out is not None:
            fine = (fine and k_out.shape == kv and k_out.dtype is dt and k_out.get_device() == dev
                    and k_out.is_contiguous())
        if inv_freq is not None:
            rot = 2 * inv_freq.numel()
            fine = (fine and inv_freq.dim() == 1 and inv_freq.dtype is torch.float32 and inv_freq.get_device() == dev
                    and inv_freq.is_contiguous())
        dtype_code = _DTYPES[dt]
    except (AttributeError, KeyError, TypeError, ValueError):  # not a tensor, another type or number of dimensions
        fine = False
    if not fine:
        _refuse_append(where, q, k, v, q_out, k_out, k_cache, v_cache, block_table, seq_lens, new_lens, inv_freq)
    strides = None
    if not dense:
        ks, vs = k.stride(), v.stride()
        qs = ks if q is None else q.stride()
        if (qs[3] != 1 or ks[3] != 1 or vs[3] != 1) and d > 1:
            raise ValueError(f"{where}: the rows of {'q' if qs[3] != 1 else 'k' if ks[3] != 1 else 'v'} must be contiguous")
        strides = _NineStrides(qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2])
    _launch((_lib or load()).fa_append_paged, where, dev,
            None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), strides,
            None if q is None else q_out.data_ptr(), None if k_out is None else k_out.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
            None if new_lens is None else new_lens.data_ptr(), None if inv_freq is None else inv_freq.data_ptr(),
            B, Hq, Hkv, N, d, P, max_pages, num_pages, rot, 1 if interleaved else 0, dtype_code, _handle(dev, stream))


def _refuse_append(where, q, k, v, q_out, k_out, k_cache, v_cache, block_table, seq_lens, new_lens, inv_freq):
    """Raises what is wrong with the arguments of fa_append_paged."""
    if (q is None) != (q_out is None):
        raise ValueError(f"{where}: q and q_out come together")
    named = (("k", k), ("v", v), ("k_cache", k_cache)) + ((("q", q),) if q is not None else ())
    _four_d(where, *named)
    dt, dev = k.dtype, k.get_device()
    if dt not in _DTYPES:
        raise TypeError(f"{where}: k has dtype {dt}, expected bfloat16 or float16")
    B, Hkv, N, d = kv = k.shape
    q_shape = None if q is None else (B, q.shape[1], N, d)
    for name, t, shape in (("q", q, q_shape), ("v", v, kv)):
        if t is not None and t.shape != shape:
            raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t is not None and t.dtype is not dt:
            raise TypeError(f"{where}: {name} has dtype {t.dtype}, expected {dt}")
        if t is not None and t.stride(3) != 1:
            raise ValueError(f"{where}: the rows of {name} must be contiguous")
    if k.stride(3) != 1:
        raise ValueError(f"{where}: the rows of k must be contiguous")
    if inv_freq is not None and (not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1):
        raise ValueError(f"{where}: inv_freq must be a 1-D tensor")
    num_pages, Hc, P, _ = k_cache.shape
    if Hc != Hkv:
        raise ValueError(f"{where}: k has {Hkv} heads, the cache {Hc}")
    max_pages, cache = _table_width(where, block_table), (num_pages, Hkv, P, d)
    _fits(where, dev, ("k_cache", k_cache, cache, dt), ("v_cache", v_cache, cache, dt),
          ("block_table", block_table, (B, max_pages), torch.int32), ("seq_lens", seq_lens, (B,), torch.int32),
          ("new_lens", new_lens, (B,), torch.int32), ("q_out", q_out, q_shape, dt), ("k_out", k_out, kv, dt),
          ("inv_freq", inv_freq, None, torch.float32))
    for name, t in (("q", q), ("v", v)):
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{where}: all tensors must be on one device ({name} is on {t.device})")
    raise ValueError(f"{where}: arguments do not fit together")


def _attention_paged(where, q, k_cache, v_cache, block_table, seq_lens, new_lens, o, lse, workspace):
    """Checks shared by the attention passes over the cache; returns the
    device, the library's pointer and size arguments, and the workspace's."""
    try:
        dt, dev, qs = q.dtype, q.get_device(), q.shape
        cache, lens = k_cache.shape, seq_lens.shape
        B, Hq, N, d = qs
        num_pages, Hkv, P, dc = cache
        Bt, max_pages = block_table.shape
        i32 = torch.int32
        fine = (dev >= 0 and dc == d and Bt == B and lens == (B,) and v_cache.shape == cache and o.shape == qs
                and lse.shape == (B, Hq, N) and k_cache.dtype is dt and v_cache.dtype is dt and o.dtype is dt
                and lse.dtype is torch.float32 and block_table.dtype is i32 and seq_lens.dtype is i32
                and k_cache.get_device() == dev and v_cache.get_device() == dev and block_table.get_device() == dev
                and seq_lens.get_device() == dev and o.get_device() == dev and lse.get_device() == dev
                and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
                and block_table.is_contiguous() and seq_lens.is_contiguous() and o.is_contiguous()
                and lse.is_contiguous())
        if new_lens is not None:
            fine = (fine and new_lens.shape == lens and new_lens.dtype is i32 and new_lens.get_device() == dev
                    and new_lens.is_contiguous())
        ws = (None, 0)
        if workspace is not None:
            fine = fine and workspace.get_device() == dev and workspace.is_contiguous()
            ws = (workspace.data_ptr(), workspace.numel() * workspace.element_size())
        dtype_code = _DTYPES[dt]
    except (AttributeError, KeyError, TypeError, ValueError):  # not a tensor, another type or number of dimensions
        fine = False
    if not fine:
        _four_d(where, ("q", q), ("k_cache", k_cache))
        dt, dev = q.dtype, q.get_device()
        if dt not in _DTYPES:
            raise TypeError(f"{where}: q has dtype {dt}, expected bfloat16 or float16")
        B, Hq, N, d = q.shape
        num_pages, Hkv, P, _ = k_cache.shape
        max_pages, cache = _table_width(where, block_table), (num_pages, Hkv, P, d)
        _fits(where, dev, ("q", q, q.shape, dt), ("k_cache", k_cache, cache, dt), ("v_cache", v_cache, cache, dt),
              ("block_table", block_table, (B, max_pages), torch.int32), ("seq_lens", seq_lens, (B,), torch.int32),
              ("new_lens", new_lens, (B,), torch.int32), ("o", o, q.shape, dt), ("lse", lse, (B, Hq, N), torch.float32),
              ("workspace", workspace, None, None))
        raise ValueError(f"{where}: arguments do not fit together")
    tensors = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr())
    return dev, tensors, (o.data_ptr(), lse.data_ptr()), (B, Hq, Hkv, N, d, P, max_pages, num_pages), dtype_code, ws


def fa_fwd_paged_workspace_bytes(B: int, Hq: int, Hkv: int, N: int, d: int, page_size: int, max_pages: int) -> int:
    return int(load().fa_fwd_paged_workspace_bytes(B, Hq, Hkv, N, d, page_size, max_pages))


def fa_fwd_paged(q, k_cache, v_cache, block_table, seq_lens, new_lens, o, lse, scale: float, workspace,
                 stream=None) -> None:
    """Forward pass of new tokens over a paged cache that already holds them:
    q [B,Hq,N,d], token t < new_lens[b] (None: N) at position
    seq_lens[b] - new_lens[b] + t sees every key up to its own; workspace of
    at least fa_fwd_paged_workspace_bytes(...) bytes."""
    where = "fa_fwd_paged"
    dev, ins, outs, sizes, dt, ws = _attention_paged(where, q, k_cache, v_cache, block_table, seq_lens, new_lens, o, lse,
                                                     workspace)
    _launch((_lib or load()).fa_fwd_paged, where, dev, *ins, None if new_lens is None else new_lens.data_ptr(), *outs,
            *sizes, scale, dt, *ws, _handle(dev, stream))


def fa_decode_prefix_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, d: int, page_size: int, max_pages: int,
                                     prefix_len: int) -> int:
    return int(load().fa_decode_prefix_workspace_bytes(B, Hq, Hkv, Nq, d, page_size, max_pages, prefix_len))


def fa_decode_prefix(q, k_cache, v_cache, block_table, seq_lens, o, lse, scale: float, prefix_len: int, workspace,
                     stream=None) -> None:
    """fa_decode_paged for a batch whose first prefix_len tokens (a multiple of
    the page size) are the same pages in every sequence: they are read once,
    from the pages of sequence 0.  workspace of at least
    fa_decode_prefix_workspace_bytes(...) bytes."""
    where = "fa_decode_prefix"
    dev, ins, outs, sizes, dt, ws = _attention_paged(where, q, k_cache, v_cache, block_table, seq_lens, None, o, lse,
                                                     workspace)
    _launch((_lib or load()).fa_decode_prefix, where, dev, *ins, *outs, *sizes, prefix_len, scale, dt, *ws,
            _handle(dev, stream))


# ------------------------------------------------------------ conveniences

def _allocating(device, stream):
    """Context in which buffers of a call on `stream` are allocated and freed
    in that stream's order."""
    if stream is None:
        return torch.cuda.stream(torch.cuda.current_stream(device))
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                  else torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


def cache_append(q, k, v, k_cache, v_cache, block_table, seq_lens, inv_freq=None, new_lens=None,
                 interleaved: bool = False, stream=None):
    """Allocates the rotated queries and runs fa_append_paged; returns them
    (None when q is None).  Rows behind a sequence's new tokens, and those of
    idle (length 0) and refused sequences, are zero."""
    q_out = None
    if q is not None:
        with _allocating(k.device, stream):
            q_out = torch.zeros(q.shape, device=q.device, dtype=q.dtype)
    fa_append_paged(q, k, v, q_out, None, k_cache, v_cache, block_table, seq_lens, new_lens, inv_freq, interleaved, stream)
    return q_out


def attention_fwd_paged(q, k_cache, v_cache, block_table, seq_lens, new_lens=None, scale: float | None = None,
                        stream=None):
    """Allocates O, lse and the workspace and runs fa_fwd_paged.  Rows behind
    a sequence's new tokens are O = 0, lse = -inf."""
    B, Hq, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    with _allocating(q.device, stream):
        if new_lens is None:
            o = torch.empty_like(q)
            lse = torch.empty((B, Hq, N), device=q.device, dtype=torch.float32)
        else:
            o = torch.zeros_like(q)
            lse = torch.full((B, Hq, N), -math.inf, device=q.device, dtype=torch.float32)
        ws = torch.empty(max(fa_fwd_paged_workspace_bytes(B, Hq, k_cache.shape[1], N, d, k_cache.shape[2],
                                                          block_table.shape[1]), 16),
                         device=q.device, dtype=torch.uint8)
    fa_fwd_paged(q, k_cache, v_cache, block_table, seq_lens, new_lens, o, lse, scale, ws, stream)
    return o, lse


def attention_decode_prefix(q, k_cache, v_cache, block_table, seq_lens, prefix_len: int, scale: float | None = None,
                            stream=None):
    """Allocates O, lse and the workspace and runs fa_decode_prefix."""
    B, Hq, Nq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    with _allocating(q.device, stream):
        o = torch.empty_like(q)
        lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32)
        ws = torch.empty(max(fa_decode_prefix_workspace_bytes(B, Hq, k_cache.shape[1], Nq, d, k_cache.shape[2],
                                                              block_table.shape[1], prefix_len), 16),
                         device=q.device, dtype=torch.uint8)
    fa_decode_prefix(q, k_cache, v_cache, block_table, seq_lens, o, lse, scale, prefix_len, ws, stream)
    return o, lse


def attention_decode_paged(q, k_cache, v_cache, block_table, seq_lens, scale: float | None = None,
                           stream=None):
    """Allocates O, lse and the workspace and runs fa_decode_paged."""
    B, Hq, Nq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32)
    ws = torch.empty(max(fa_decode_workspace_bytes(B, Hq, k_cache.shape[1], Nq, d,
                                                   block_table.shape[1]), 16),
                     device=q.device, dtype=torch.uint8)
    fa_decode_paged(q, k_cache, v_cache, block_table, seq_lens, o, lse, scale, ws, stream)
    return o, lse



def attention_fwd(q, k, v, scale: float | None = None, causal: bool = False, stream=None,
                  window: int = 0, dropout=None, block_mask=None):
    """Allocates O and lse with PyTorch and runs fa_fwd (fa_fwd_window when
    window > 0, which implies causal; fa_fwd_dropout when dropout = (p_drop,
    seed); fa_fwd_blockmask when block_mask is given); returns (O, lse)."""
    if sum((bool(window), bool(dropout), block_mask is not None)) > 1:
        raise ValueError("a sliding window, dropout and a block mask are not combined")
    B, Hq, Hkv, N, d = _dims(q, k)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, N), device=q.device, dtype=torch.float32)
    if block_mask is not None:
        fa_fwd_blockmask(q, k, v, o, lse, scale, causal, block_mask, stream)
    elif window:
        fa_fwd_window(q, k, v, o, lse, scale, window, stream)
    elif dropout:
        fa_fwd_dropout(q, k, v, o, lse, scale, causal, dropout[0], dropout[1], stream)
    else:
        fa_fwd(q, k, v, o, lse, scale, causal, stream)
    return o, lse


def attention_bwd(q, k, v, o, dout, lse, scale: float | None = None, causal: bool = False,
                  workspace=None, stream=None, window: int = 0, dropout=None, block_mask=None):
    """Allocates dQ, dK, dV (and the workspace if not given) and runs fa_bwd
    (fa_bwd_window when window > 0, fa_bwd_dropout with dropout,
    fa_bwd_blockmask with a block mask)."""
    B, Hq, Hkv, N, d = _dims(q, k)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        nbytes = (fa_bwd_blockmask_workspace_bytes(B, Hq, Hkv, N, d) if block_mask is not None
                  else fa_bwd_workspace_bytes(B, Hq, Hkv, N, d))
        workspace = torch.empty(max(nbytes, 16), device=q.device, dtype=torch.uint8)
    if block_mask is not None:
        fa_bwd_blockmask(q, k, v, o, dout, lse, dq, dk, dv, scale, causal, block_mask, workspace, stream)
    elif window:
        fa_bwd_window(q, k, v, o, dout, lse, dq, dk, dv, scale, window, workspace, stream)
    elif dropout:
        fa_bwd_dropout(q, k, v, o, dout, lse, dq, dk, dv, scale, causal, dropout[0], dropout[1],
                       workspace, stream)
    else:
        fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, scale, causal, workspace, stream)
    return dq, dk, dv


def fa_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, scale: float, causal: bool,
                   stream=None) -> None:
    """fa_bwd without a workspace: for callers that cannot allocate device
    memory.  Uses the library's fixed scratch array (FA_BWD_NOALLOC_SCRATCH_BYTES
    per device); raises FaError(FA_ERR_UNSUPPORTED) for problems that need more.
    Calls on one device share that array, so order them on one stream."""
    lib = load()
    fn = lib.fa_bwd_noalloc
    if fn.argtypes is None:
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        fn.argtypes = [vp] * 9 + [i, i, i, i, i, f, i, i, vp]
        fn.restype = i
    B, Hq, Hkv, N, d = _expect_attention("fa_bwd_noalloc", q, k, v, o, lse, dout, dq, dk, dv)
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
            _ptr(dv), B, Hq, Hkv, N, d, float(scale), int(bool(causal)), _DTYPES[q.dtype],
            _stream(stream))
    _check(st, "fa_bwd_noalloc")
