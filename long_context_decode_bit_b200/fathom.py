"""ctypes binding of ``libfathom.so`` (C ABI in ``include/fathom.h``).

Argument marshalling only: every step of the scan runs in the library's
CUDA kernels.  torch tensors supply device memory and the current stream;
outputs are allocated here with torch when the caller does not pass them.
If the library is missing or cannot be loaded, every call raises -- there
is no fallback.

A function runs on the current stream or on the one it is given.  On a given
stream its inputs have to be ready in that stream's order, and the caller's
stream waits for it before it uses the outputs, as with torch's own calls.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfathom.so")

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_CUDA = -3
ERR_WORKSPACE = -4
ERR_TIMEOUT = -5
ERR_OVERFLOW = -6
ERR_BOUNDS = -7   # debug build: a device-side bounds check failed

KEYS_F32 = 0
KEYS_BF16 = 1
SCAN_DENSE = 0
SCAN_CANDIDATE = 1
SCAN_PREPARE = 2
SCAN_FILTER = 3
KV_BF16 = 0
KV_INT8 = 1
KV_E4M3 = 2
KV_BLOCK = 32     # channels that share a power of two

# Every symbol include/fathom.h declares.
EXPORTS = (
    "fathom_version", "fathom_status_string", "fathom_last_cuda_error", "fathom_nb_stride",
    "fathom_pack", "fathom_plan", "fathom_plan_fixed", "fathom_scan_cand_bytes", "fathom_scan",
    "fathom_topk_workspace_bytes", "fathom_topk", "fathom_dequant_rows", "fathom_scan_topk_noalloc",
    "fathom_device_status", "fathom_calibrate_workspace_bytes", "fathom_calibrate",
    "fathom_union_attention_workspace_bytes", "fathom_union_attention",
    "fathom_nibbles_from_planes", "fathom_scan_nibbles", "fathom_layer_budgets_workspace_bytes",
    "fathom_layer_budgets", "fathom_pack_rotated", "fathom_nibbles_tm_from_planes", "fathom_scan_nibbles_tm",
    "fathom_kv_write", "fathom_kv_read", "fathom_paged_attention_workspace_bytes", "fathom_paged_attention",
    "fathom_paged_union_attention_workspace_bytes", "fathom_paged_union_attention",
)

NOALLOC_SCRATCH_BYTES = 16 << 20

_lib = None


class FathomError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {_lib.fathom_status_string(status).decode() if _lib else status}"
        if status == ERR_CUDA and _lib is not None:
            msg += f" (cudaError {_lib.fathom_last_cuda_error()})"
        super().__init__(msg)


def load(path: str | None = None):
    """Load the shared library (raises if it is missing).  ``FATHOM_LIB``
    may name another build of it."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or os.environ.get("FATHOM_LIB") or LIB_PATH
    if not os.path.exists(path):
        raise FileNotFoundError(
            f"{path} is missing: build it with `python -m long_context_decode_bit_b200.build`")
    lib = ctypes.CDLL(path)
    P, I, I64, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "fathom_version": (I, []),
        "fathom_status_string": (ctypes.c_char_p, [I]),
        "fathom_last_cuda_error": (I, []),
        "fathom_nb_stride": (I64, [I64]),
        "fathom_pack": (I, [P, I, I64, I64, I, I64, I64, P, P, I64, P]),
        "fathom_plan": (I, [P, P, I64, I, I, P, ctypes.c_int32, P, P, P, P, P]),
        "fathom_plan_fixed": (I, [P, I64, I, I, I, I, P, P, P, P]),
        "fathom_scan_cand_bytes": (SZ, [I64, I, I64, I]),
        "fathom_scan": (I, [P, P, I64, I, I64, I64, P, P, P, I, I, P, P, SZ, I, P]),
        "fathom_topk_workspace_bytes": (SZ, [I64, I, I64, I]),
        "fathom_topk": (I, [P, P, I64, I, I64, I, P, P, P, P, SZ, P]),
        "fathom_dequant_rows": (I, [P, P, I64, I, I64, I64, P, I64, P, I, P, P]),
        "fathom_scan_topk_noalloc": (I, [P, P, I64, I, I64, I64, P, P, P, I, I, P, P, P, P]),
        "fathom_device_status": (I, [I, P]),
        "fathom_pack_rotated": (I, [P, I, I64, I64, I, I64, I64, P, P, P, I64, P]),
        "fathom_nibbles_tm_from_planes": (I, [P, I64, I, I64, I64, P, P]),
        "fathom_scan_nibbles_tm": (I, [P, P, I64, I, I64, I64, P, P, P, I, I, P, P, SZ, I, P]),
        "fathom_calibrate_workspace_bytes": (SZ, [I64, I, I]),
        "fathom_calibrate": (I, [P, I, I64, I64, I, I64, I64, P, P, P, P, SZ, P]),
        "fathom_union_attention_workspace_bytes": (SZ, [I64, I, I, I64]),
        "fathom_nibbles_from_planes": (I, [P, I64, I, I64, I64, P, P]),
        "fathom_layer_budgets_workspace_bytes": (SZ, [I64, I]),
        "fathom_layer_budgets": (I, [P, P, I64, I, I, I, I64, P, P, SZ, P]),
        "fathom_scan_nibbles": (I, [P, P, I64, I, I64, I64, P, P, P, I, I, P, P, SZ, I, P]),
        "fathom_union_attention": (I, [P, P, I, I64, I64, I, I64, I64, P, I, P, P, I64, ctypes.c_float, P, P, SZ, P]),
        "fathom_kv_write": (I, [P, P, P, P, I, I64, I64, P]),
        "fathom_kv_read": (I, [P, P, P, P, I, I64, I64, P]),
        "fathom_paged_attention_workspace_bytes": (SZ, [I, I, I, I64, I, I64, I64, I]),
        "fathom_paged_attention": (I, [P, P, P, I, I64, I64, I, I64, I64, I, F, P, P, SZ, P]),
        "fathom_paged_union_attention_workspace_bytes": (SZ, [I64, I, I, I64]),
        "fathom_paged_union_attention": (I, [P, P, ctypes.c_int32, I64, P, I, P, P, I64, F, P, P, SZ, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def lib():
    return load()


def _check(st: int, what: str):
    if st != OK:
        raise FathomError(st, what)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The handle of a device's current stream.  torch's own short way makes no Stream object (0.3 us instead of 1.5 on
# the host); it is not part of its public API.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream):
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream


def _scratch(stream, make, *args, **kw):
    """A tensor made (``make(*args, **kw)``) for a call on ``stream``, in that stream's memory: a block of the current
    one's may be free because only the order of that stream's work protects it."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _output(stream, make, *args, **kw):
    """The same, of a tensor that is handed to the caller, whose own stream uses it once ``stream`` is done."""
    t = _scratch(stream, make, *args, **kw)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream())
    return t


def nb_stride(n: int) -> int:
    return int(lib().fathom_nb_stride(int(n)))


def scan_cand_bytes(H: int, G: int, n: int, k: int) -> int:
    return int(lib().fathom_scan_cand_bytes(H, G, n, k))


def topk_workspace_bytes(H: int, G: int, n: int, k: int) -> int:
    return int(lib().fathom_topk_workspace_bytes(H, G, n, k))


def pack(keys: torch.Tensor, nb_stride_words: int | None = None, planes=None, scales=None, stream=None):
    """Bit-plane index of keys [H][n][D] (fp32 or bf16, channels contiguous).
    Returns (planes uint64-as-int64 [H][D][4][nb_stride], scales int16 [H][D][nb_stride])."""
    H, n, D = keys.shape
    if keys.stride(2) != 1:
        raise ValueError("keys must be contiguous along channels")
    dt = {torch.float32: KEYS_F32, torch.bfloat16: KEYS_BF16}[keys.dtype]
    nbs = nb_stride(n) if nb_stride_words is None else int(nb_stride_words)
    dev = keys.device
    if planes is None:
        planes = _output(stream, torch.zeros, (H, D, 4, nbs), dtype=torch.int64, device=dev)
    if scales is None:
        scales = _output(stream, torch.zeros, (H, D, nbs), dtype=torch.int16, device=dev)
    _check(lib().fathom_pack(_p(keys), dt, H, n, D, keys.stride(0), keys.stride(1), _p(planes), _p(scales),
                             nbs, _stream(stream)), "fathom_pack")
    return planes, scales


def pack_rotated(keys: torch.Tensor, U: torch.Tensor, nb_stride_words: int | None = None, planes=None, scales=None,
                 stream=None):
    """Bit-plane index of the keys' coordinates in the basis U [H][D][D]
    (fp32, columns = directions), rotated inside the kernel in a fixed fp32
    fused multiply-add order (see fathom_pack_rotated in include/fathom.h)."""
    H, n, D = keys.shape
    if keys.stride(2) != 1:
        raise ValueError("keys must be contiguous along channels")
    if U.dtype != torch.float32 or tuple(U.shape) != (H, D, D) or not U.is_contiguous():
        raise ValueError("U must be a contiguous fp32 [H][D][D] tensor")
    dt = {torch.float32: KEYS_F32, torch.bfloat16: KEYS_BF16}[keys.dtype]
    nbs = nb_stride(n) if nb_stride_words is None else int(nb_stride_words)
    dev = keys.device
    if planes is None:
        planes = _output(stream, torch.zeros, (H, D, 4, nbs), dtype=torch.int64, device=dev)
    if scales is None:
        scales = _output(stream, torch.zeros, (H, D, nbs), dtype=torch.int16, device=dev)
    _check(lib().fathom_pack_rotated(_p(keys), dt, H, n, D, keys.stride(0), keys.stride(1), _p(U), _p(planes),
                                     _p(scales), nbs, _stream(stream)), "fathom_pack_rotated")
    return planes, scales


def pack_range(keys: torch.Tensor, planes: torch.Tensor, scales: torch.Tensor, block0: int, stream=None):
    """(Re)pack blocks block0.. of an existing index from ``keys`` [H][m][D],
    the keys of tokens 64*block0 .. 64*block0 + m - 1 (appending to the tail
    block during decode).  ``planes``/``scales`` are the whole index."""
    H, m, D = keys.shape
    if keys.stride(2) != 1:
        raise ValueError("keys must be contiguous along channels")
    dt = {torch.float32: KEYS_F32, torch.bfloat16: KEYS_BF16}[keys.dtype]
    nbs = planes.shape[-1]
    if block0 < 0 or block0 + (m + 63) // 64 > nbs:
        raise ValueError("block range outside the index")
    pp = ctypes.c_void_p(planes.data_ptr() + 8 * block0)
    sp = ctypes.c_void_p(scales.data_ptr() + 2 * block0)
    _check(lib().fathom_pack(_p(keys), dt, H, m, D, keys.stride(0), keys.stride(1), pp, sp, nbs, _stream(stream)),
           "fathom_pack")
    return planes, scales


def plan(sigma2: torch.Tensor, q: torch.Tensor, budget, out=None, stream=None):
    """Reverse water-filling plan.  ``budget`` is an int (flat) or an int32
    device tensor [H].  Returns (depth uint8 [H][D], active int16 [H][D],
    n_active int32 [H], theta fp32 [H])."""
    H, G, D = q.shape
    dev = q.device
    if out is None:
        out = (_output(stream, torch.empty, (H, D), dtype=torch.uint8, device=dev),
               _output(stream, torch.empty, (H, D), dtype=torch.int16, device=dev),
               _output(stream, torch.empty, H, dtype=torch.int32, device=dev),
               _output(stream, torch.empty, H, dtype=torch.float32, device=dev))
    depth, active, n_active, theta = out
    if isinstance(budget, torch.Tensor):
        bptr, flat = _p(budget), 0
    else:
        bptr, flat = None, int(budget)
    _check(lib().fathom_plan(_p(sigma2), _p(q), H, G, D, bptr, flat, _p(depth), _p(active), _p(n_active),
                             _p(theta), _stream(stream)), "fathom_plan")
    return depth, active, n_active, theta


def layer_budgets(sigma2: torch.Tensor, q: torch.Tensor, layers: int, total_bits: int, out=None, stream=None):
    """Greedy per-layer split of ``total_bits`` plane bits from calibration
    queries q [H][G][D]: int32 [H] budgets for ``plan``."""
    H, G, D = q.shape
    dev = q.device
    if out is None:
        out = _output(stream, torch.empty, H, dtype=torch.int32, device=dev)
    need = int(lib().fathom_layer_budgets_workspace_bytes(H, D))
    ws = _scratch(stream, torch.empty, max(need, 1), dtype=torch.uint8, device=dev)
    _check(lib().fathom_layer_budgets(_p(sigma2), _p(q), H, G, D, int(layers), int(total_bits), _p(out), _p(ws),
                                      ws.numel(), _stream(stream)), "fathom_layer_budgets")
    return out


def plan_fixed(q: torch.Tensor, r: int, out=None, stream=None, bits: int = 4):
    """Fixed-depth comparator plan: the r channels with the largest
    sum_g |q| read at ``bits`` planes."""
    H, G, D = q.shape
    dev = q.device
    if out is None:
        out = (_output(stream, torch.empty, (H, D), dtype=torch.uint8, device=dev),
               _output(stream, torch.empty, (H, D), dtype=torch.int16, device=dev),
               _output(stream, torch.empty, H, dtype=torch.int32, device=dev))
    depth, active, n_active = out
    _check(lib().fathom_plan_fixed(_p(q), H, G, D, int(r), int(bits), _p(depth), _p(active), _p(n_active),
                                   _stream(stream)),
           "fathom_plan_fixed")
    return depth, active, n_active


def scan(planes, scales, n: int, active, n_active, q, mode: int = SCAN_DENSE, k: int = 0,
         scores=None, cand=None, stream=None, nibbles: bool = False, token_major: bool = False):
    """Scores [H][G][n] (DENSE) or the candidate buffer (CANDIDATE).  With
    ``nibbles`` the first argument is the nibble store (every active channel
    read at 4 bits); with ``token_major`` it is the token-major store of
    ``nibbles_tm_from_planes`` (the same scores)."""
    H, G, D = q.shape
    nbs = scales.shape[-1]
    if token_major:
        fn, name = lib().fathom_scan_nibbles_tm, "fathom_scan_nibbles_tm"
    elif nibbles:
        fn, name = lib().fathom_scan_nibbles, "fathom_scan_nibbles"
    else:
        fn, name = lib().fathom_scan, "fathom_scan"
    if mode == SCAN_DENSE:
        if scores is None:
            scores = _output(stream, torch.empty, (H, G, n), dtype=torch.float32, device=q.device)
        _check(fn(_p(planes), _p(scales), H, D, n, nbs, _p(active), _p(n_active), _p(q), G,
                  SCAN_DENSE, _p(scores), None, 0, int(k), _stream(stream)), name)
        return scores
    nbytes = scan_cand_bytes(H, G, n, k)
    if cand is None:
        cand = _output(stream, torch.empty, nbytes, dtype=torch.uint8, device=q.device)
    _check(fn(_p(planes), _p(scales), H, D, n, nbs, _p(active), _p(n_active), _p(q), G,
              int(mode), None, _p(cand), cand.numel() * cand.element_size(), int(k), _stream(stream)), name)
    return cand


def nibbles_from_planes(planes, n: int, out=None, stream=None):
    """The nibble store [H][D][4][nb_stride] of the codes the planes hold."""
    H, D, _, nbs = planes.shape
    if out is None:
        out = _output(stream, torch.empty_like, planes)
    _check(lib().fathom_nibbles_from_planes(_p(planes), H, D, n, nbs, _p(out), _stream(stream)),
           "fathom_nibbles_from_planes")
    return out


def nibbles_tm_from_planes(planes, n: int, out=None, stream=None):
    """The token-major 4-bit store uint8 [H][64*nb_stride][D/2] of the codes
    the planes hold (two channels per byte, channel 2c in the low nibble)."""
    H, D, _, nbs = planes.shape
    if out is None:
        out = _output(stream, torch.zeros, (H, 64 * nbs, D // 2), dtype=torch.uint8, device=planes.device)
    _check(lib().fathom_nibbles_tm_from_planes(_p(planes), H, D, n, nbs, _p(out), _stream(stream)),
           "fathom_nibbles_tm_from_planes")
    return out


def topk(H: int, G: int, n: int, k: int, scores=None, cand=None, out=None, workspace=None, stream=None):
    """Per-head top-k and per-group union.  Returns (idx int32 [H][G][k],
    union int32 [H][G*k], union_count int32 [H])."""
    dev = (scores if scores is not None else cand).device
    if out is None:
        out = (_output(stream, torch.empty, (H, G, k), dtype=torch.int32, device=dev),
               _output(stream, torch.empty, (H, G * k), dtype=torch.int32, device=dev),
               _output(stream, torch.empty, H, dtype=torch.int32, device=dev))
    idx, uni, cnt = out
    ws_need = topk_workspace_bytes(H, G, n, k)
    if workspace is None and ws_need:
        workspace = _scratch(stream, torch.empty, ws_need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fathom_topk(_p(scores), _p(cand), H, G, n, int(k), _p(idx), _p(uni), _p(cnt), _p(workspace),
                             ws_bytes, _stream(stream)), "fathom_topk")
    return idx, uni, cnt


def dequant_rows(planes, scales, n: int, rows, row_count=None, bits: int = 4, out=None, stream=None):
    """Key rows rebuilt from the index: fp32 [H][M][D] for rows int32 [H][M]
    (e.g. the union of ``topk``), at ``bits`` planes."""
    H, D = planes.shape[0], planes.shape[1]
    M = rows.shape[1]
    if out is None:
        out = _output(stream, torch.empty, (H, M, D), dtype=torch.float32, device=rows.device)
    _check(lib().fathom_dequant_rows(_p(planes), _p(scales), H, D, n, planes.shape[-1], _p(rows), M,
                                     _p(row_count), int(bits), _p(out), _stream(stream)), "fathom_dequant_rows")
    return out


def scan_topk_noalloc(planes, scales, n: int, active, n_active, q, k: int, out=None, stream=None):
    """Candidate scan + top-k + union using the library's own fixed device
    scratch instead of a caller buffer, for callers that cannot allocate
    device memory (see fathom_scan_topk_noalloc in include/fathom.h).  The
    output tensors may be preallocated and passed as ``out``."""
    H, G, D = q.shape
    if out is None:
        dev = q.device
        out = (_output(stream, torch.empty, (H, G, k), dtype=torch.int32, device=dev),
               _output(stream, torch.empty, (H, G * k), dtype=torch.int32, device=dev),
               _output(stream, torch.empty, H, dtype=torch.int32, device=dev))
    idx, uni, cnt = out
    _check(lib().fathom_scan_topk_noalloc(_p(planes), _p(scales), H, D, n, planes.shape[-1], _p(active),
                                          _p(n_active), _p(q), G, int(k), _p(idx), _p(uni), _p(cnt),
                                          _stream(stream)), "fathom_scan_topk_noalloc")
    return idx, uni, cnt


def calibrate_workspace_bytes(H: int, D: int, with_cov: bool) -> int:
    return int(lib().fathom_calibrate_workspace_bytes(H, D, 1 if with_cov else 0))


def calibrate(keys: torch.Tensor, n: int | None = None, with_mean: bool = True, with_cov: bool = False,
              workspace=None, stream=None):
    """Per-group key statistics over the first ``n`` keys of keys [H][n_total][D]
    (fp32 or bf16): (mean [H][D] or None, sigma2 [H][D], cov [H][D][D] or None),
    all fp32."""
    H, nt, D = keys.shape
    n = nt if n is None else int(n)
    if keys.dtype == torch.float32:
        dt = KEYS_F32
    elif keys.dtype == torch.bfloat16:
        dt = KEYS_BF16
    else:
        raise TypeError("keys must be float32 or bfloat16")
    if keys.stride(2) != 1:
        raise ValueError("keys must be contiguous along D")
    dev = keys.device
    sigma2 = _output(stream, torch.empty, (H, D), dtype=torch.float32, device=dev)
    mean = _output(stream, torch.empty, (H, D), dtype=torch.float32, device=dev) if with_mean else None
    cov = _output(stream, torch.empty, (H, D, D), dtype=torch.float32, device=dev) if with_cov else None
    need = calibrate_workspace_bytes(H, D, with_cov)
    if workspace is None or workspace.numel() < need:
        workspace = _scratch(stream, torch.empty, max(need, 1), dtype=torch.uint8, device=dev)
    _check(lib().fathom_calibrate(_p(keys), dt, H, n, D, keys.stride(0), keys.stride(1), _p(mean), _p(sigma2),
                                  _p(cov), _p(workspace), workspace.numel(), _stream(stream)), "fathom_calibrate")
    return mean, sigma2, cov


def union_attention_workspace_bytes(H: int, G: int, D: int, M: int) -> int:
    return int(lib().fathom_union_attention_workspace_bytes(H, G, D, M))


def union_attention(k_cache: torch.Tensor, v_cache: torch.Tensor, q: torch.Tensor, union_idx: torch.Tensor,
                    union_count: torch.Tensor, scale: float | None = None, out=None, workspace=None, stream=None):
    """Softmax attention [H][G][D] (fp32) of each query head over its group's
    union rows of the K/V cache [H][n][D] (fp32 or bf16)."""
    H, n, D = k_cache.shape
    G = q.shape[1]
    M = union_idx.shape[1]
    if k_cache.dtype != v_cache.dtype or k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must share dtype, shape and strides")
    dt = {torch.float32: KEYS_F32, torch.bfloat16: KEYS_BF16}[k_cache.dtype]
    if k_cache.stride(2) != 1:
        raise ValueError("the cache must be contiguous along D")
    if out is None:
        out = _output(stream, torch.empty, (H, G, D), dtype=torch.float32, device=q.device)
    need = int(lib().fathom_union_attention_workspace_bytes(H, G, D, M))
    if workspace is None or workspace.numel() < need:
        workspace = _scratch(stream, torch.empty, max(need, 1), dtype=torch.uint8, device=q.device)
    sc = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check(lib().fathom_union_attention(_p(k_cache), _p(v_cache), dt, H, n, D, k_cache.stride(0), k_cache.stride(1),
                                        _p(q), G, _p(union_idx), _p(union_count), M, sc, _p(out), _p(workspace),
                                        workspace.numel(), _stream(stream)), "fathom_union_attention")
    return out


class _KvCacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
                ("scale_token_stride", ctypes.c_int64), ("H", ctypes.c_int32), ("D", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("format", ctypes.c_int32)]


class _KvRowsStruct(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("cu", ctypes.c_void_p), ("length", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("rows", ctypes.c_int64), ("table_pages", ctypes.c_int32),
                ("B", ctypes.c_int32)]


_KV_ROWS = struct.Struct("PPPqqii").pack   # the bytes of a _KvRowsStruct, made in half the time

_KV_FORMATS = {torch.bfloat16: KV_BF16, torch.int8: KV_INT8, torch.float8_e4m3fn: KV_E4M3}
_KEY_TYPES = {torch.float32: KEYS_F32, torch.bfloat16: KEYS_BF16}


class KVCache:
    """A paged KV cache over the caller's tensors (fathom_kv_cache in
    include/fathom.h): k, v [pages][H][page_tokens][D] in bf16, int8 or
    float8_e4m3fn (any strides, channels contiguous; ``transpose(1, 2)`` of a
    [pages][page_tokens][H][D] tensor, or one layer of a larger one), and for
    the 8-bit formats k_scale, v_scale uint8 [pages][H][page_tokens][D/32].
    Their addresses are taken once, so none of its attributes can be replaced."""

    _FIXED = frozenset(("k", "v", "k_scale", "v_scale", "H", "D", "page_tokens", "format", "_struct", "_ref", "_device"))

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale=None, v_scale=None):
        if k.dtype not in _KV_FORMATS:
            raise TypeError("the cache is bfloat16, int8 or float8_e4m3fn")
        if k.dim() != 4 or v.dtype != k.dtype or v.shape != k.shape or v.stride() != k.stride() or v.device != k.device:
            raise ValueError("k and v must be [pages][H][page_tokens][D] and share dtype, strides and device")
        if k.stride(3) != 1:
            raise ValueError("the cache must be contiguous along D")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.format = _KV_FORMATS[k.dtype]
        pages, self.H, self.page_tokens, self.D = k.shape
        strides = (0, 0, 0)
        if self.format != KV_BF16:
            shape = (pages, self.H, self.page_tokens, self.D // KV_BLOCK)
            for s in (k_scale, v_scale):
                if s is None or s.dtype != torch.uint8 or tuple(s.shape) != shape or s.device != k.device:
                    raise ValueError("an 8-bit cache needs uint8 scales [pages][H][page_tokens][D/32] beside it")
            if k_scale.stride() != v_scale.stride() or k_scale.stride(3) != 1:
                raise ValueError("the scales must share strides and be contiguous along D/32")
            strides = k_scale.stride()[:3]
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bfloat16 cache has no scales")
        scale_ptr = (None, None) if k_scale is None else (k_scale.data_ptr(), v_scale.data_ptr())
        self._struct = _KvCacheStruct(k.data_ptr(), v.data_ptr(), *scale_ptr, pages, k.stride(0), k.stride(1),
                                      k.stride(2), strides[0], strides[1], strides[2], self.H, self.D,
                                      self.page_tokens, self.format)
        self._device = k.get_device()   # -1: not on a GPU
        self._ref = ctypes.byref(self._struct)

    def __setattr__(self, name, value):
        if name in self._FIXED and "_ref" in self.__dict__:
            raise AttributeError(f"{name} is part of what calls use; make another KVCache")
        super().__setattr__(name, value)

    def __delattr__(self, name):
        if name in self._FIXED:
            raise AttributeError(f"{name} is part of what calls use; make another KVCache")
        super().__delattr__(name)

    @classmethod
    def empty(cls, pages: int, H: int, D: int, page_tokens: int = 64, dtype=torch.int8, device="cuda"):
        """A cache of zeros."""
        shape = (pages, H, page_tokens, D)
        if dtype == torch.float8_e4m3fn:
            k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) for _ in range(2))
        else:
            k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype == torch.bfloat16:
            return cls(k, v)
        return cls(k, v, *(torch.zeros(shape[:3] + (D // KV_BLOCK,), dtype=torch.uint8, device=device)
                           for _ in range(2)))


def _kv_here(cache: KVCache, *tensors):
    """Tensors of a cache call live on the cache's device, and that is the current one."""
    dev = cache._device
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError("the tensors of a call must be on the cache's device")
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError("the cache must be on the current CUDA device")


def _kv_rows(cache: KVCache, table, cu, length, rows: int):
    if table.dtype != torch.int32 or cu.dtype != torch.int32 or length.dtype != torch.int32:
        raise TypeError("table, cu and length are int32")
    if length.dim() != 1 or cu.dim() != 1 or table.dim() != 2:
        raise ValueError("table is [B][pages], cu [B+1] and length [B]")
    B, (table_rows, pages) = length.shape[0], table.shape
    if table_rows != B or cu.shape[0] != B + 1:
        raise ValueError("table is [B][pages], cu [B+1] and length [B]")
    stride, step = table.stride()
    if not (cu.is_contiguous() and length.is_contiguous() and (pages < 2 or step == 1)):
        raise ValueError("table rows, cu and length must be contiguous")
    _kv_here(cache, table, cu, length)
    return _KV_ROWS(table.data_ptr(), cu.data_ptr(), length.data_ptr(), stride, rows, pages, B)


def kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, cu: torch.Tensor,
             length: torch.Tensor, stream=None) -> KVCache:
    """Put rows k, v [rows][H][D] (fp32 or bf16) into the cache: the last
    cu[b+1] - cu[b] tokens of each sequence b, up to length[b] (page table
    int32 [B][pages], cu int32 [B+1], length int32 [B])."""
    if k.dtype not in _KEY_TYPES or v.dtype != k.dtype:
        raise TypeError("k and v are float32 or bfloat16")
    shape, strides = k.shape, k.stride()
    if len(shape) != 3 or shape[1] != cache.H or shape[2] != cache.D or v.shape != shape or v.stride() != strides:
        raise ValueError("k and v must be [rows][H][D] and share strides")
    if strides[2] != 1:
        raise ValueError("k and v must be contiguous along D")
    rows = _kv_rows(cache, table, cu, length, shape[0])
    _kv_here(cache, k, v)
    _check(lib().fathom_kv_write(cache._ref, rows, k.data_ptr(), v.data_ptr(), _KEY_TYPES[k.dtype], strides[0],
                                 strides[1], _stream(stream)), "fathom_kv_write")
    return cache


def kv_read(cache: KVCache, table: torch.Tensor, cu: torch.Tensor, length: torch.Tensor, rows: int,
            dtype=torch.bfloat16, out=None, stream=None):
    """Read the same rows back: (K, V), each [H][rows][D] in ``dtype`` (fp32
    or bf16), the layout ``pack`` takes.  ``out`` may give both tensors (any
    strides, channels contiguous), or None in the place of one not wanted."""
    shape = (cache.H, rows, cache.D)
    if out is None:
        if dtype not in _KEY_TYPES:
            raise TypeError("K and V are read back in float32 or bfloat16")
        k, v = _new(cache, shape, dtype, stream), _new(cache, shape, dtype, stream)
    else:
        k, v = out
    first = v if k is None else k
    if first is None:
        raise ValueError("nothing to read")
    strides = first.stride()
    for t in (k, v):
        if t is None:
            continue
        if t.dtype not in _KEY_TYPES or t.dtype != first.dtype:
            raise TypeError("K and V are read back in float32 or bfloat16")
        if t.shape != shape or t.stride() != strides or strides[2] != 1:
            raise ValueError("out must be [H][rows][D] tensors of the same strides, contiguous along D")
        _kv_here(cache, t)
    w = _kv_rows(cache, table, cu, length, rows)
    _check(lib().fathom_kv_read(cache._ref, w, None if k is None else k.data_ptr(), None if v is None else v.data_ptr(),
                                _KEY_TYPES[first.dtype], strides[0], strides[1], _stream(stream)), "fathom_kv_read")
    return k, v


def paged_attention_workspace_bytes(H: int, G: int, D: int, rows: int, B: int, max_new: int, max_len: int,
                                    dtype=torch.bfloat16) -> int:
    return int(lib().fathom_paged_attention_workspace_bytes(H, G, D, rows, B, max_new, max_len, _KEY_TYPES[dtype]))


# Sizes are asked for at every call of a decode loop, mostly the same ones.
_paged_workspace = functools.lru_cache(1024)(lambda *sizes: lib().fathom_paged_attention_workspace_bytes(*sizes))
_union_workspace = functools.lru_cache(1024)(lambda *sizes: lib().fathom_paged_union_attention_workspace_bytes(*sizes))


def _new(cache, shape, dtype, stream):
    """A contiguous [a][b][c] tensor (``empty_strided`` takes the host two
    thirds of the time that ``empty`` takes with a shape)."""
    _, b, c = shape
    if stream is None:
        return torch.empty_strided(shape, (b * c, c, 1), dtype=dtype, device=cache.k.device)
    return _output(stream, torch.empty_strided, shape, (b * c, c, 1), dtype=dtype, device=cache.k.device)


def _workspace(workspace, need: int, like, stream):
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = like.new_empty(need, dtype=torch.uint8) if stream is None else \
            _scratch(stream, like.new_empty, need, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), need
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def paged_attention(cache: KVCache, q: torch.Tensor, table: torch.Tensor, cu: torch.Tensor, length: torch.Tensor,
                    max_new: int, max_len: int, causal: bool = True, scale: float | None = None, out=None,
                    workspace=None, stream=None) -> torch.Tensor:
    """Attention of each sequence's new rows q [rows][H*G][D] (fp32 or bf16;
    head h*G + g belongs to KV head h) over its cached tokens, the rows' own
    among them: a prompt chunk or single tokens.  ``max_new`` and
    ``max_len`` bound the batch's rows and lengths.  Returns [rows][H*G][D]."""
    dt = _KEY_TYPES.get(q.dtype)
    if dt is None:
        raise TypeError("q is float32 or bfloat16")
    shape, strides = q.shape, q.stride()
    if len(shape) != 3 or shape[2] != cache.D or not cache.H or shape[1] % cache.H or strides[2] != 1:
        raise ValueError("q must be [rows][H*G][D], contiguous along D")
    rows, G = shape[0], shape[1] // cache.H
    if out is None:
        out = _new(cache, shape, q.dtype, stream)
    elif out.dtype != q.dtype or out.shape != shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous [rows][H*G][D] tensor of q's type")
    w = _kv_rows(cache, table, cu, length, rows)
    _kv_here(cache, q, out)
    L = lib()
    need = _paged_workspace(cache.H, G, cache.D, rows, length.shape[0], max_new, max_len, dt)
    workspace, ws, ws_bytes = _workspace(workspace, need, q, stream)
    sc = cache.D ** -0.5 if scale is None else float(scale)
    _check(L.fathom_paged_attention(cache._ref, w, q.data_ptr(), dt, strides[0], strides[1], G, max_new, max_len,
                                    int(causal), sc, out.data_ptr(), ws, ws_bytes, _stream(stream)),
           "fathom_paged_attention")
    return out


def paged_union_attention(cache: KVCache, q: torch.Tensor, table: torch.Tensor, n: int, union_idx: torch.Tensor,
                          union_count: torch.Tensor, scale: float | None = None, out=None, workspace=None,
                          stream=None) -> torch.Tensor:
    """``union_attention`` with the winners' rows taken from one sequence of
    the paged cache: q fp32 [H][G][D], table int32 [pages] (or [1][pages]),
    n tokens.  Returns fp32 [H][G][D]."""
    if table.dim() == 2 and table.shape[0] == 1:
        table = table[0]
    shape = q.shape
    if q.dtype != torch.float32 or len(shape) != 3 or shape[0] != cache.H or shape[2] != cache.D or not q.is_contiguous():
        raise ValueError("q must be a contiguous fp32 [H][G][D] tensor")
    if table.dtype != torch.int32 or union_idx.dtype != torch.int32 or union_count.dtype != torch.int32:
        raise TypeError("table, union_idx and union_count are int32")
    if union_idx.dim() != 2 or union_idx.shape[0] != cache.H or union_count.dim() != 1 or union_count.shape[0] != cache.H or \
            not (union_idx.is_contiguous() and union_count.is_contiguous()):
        raise ValueError("union_idx must be [H][M] and union_count [H], as topk writes them")
    if table.dim() != 1 or not table.is_contiguous():
        raise ValueError("table must be the contiguous [pages] of one sequence")
    G, M = shape[1], union_idx.shape[1]
    if out is None:
        out = _new(cache, shape, q.dtype, stream)
    elif out.dtype != q.dtype or out.shape != shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 [H][G][D] tensor")
    _kv_here(cache, q, table, union_idx, union_count, out)
    L = lib()
    workspace, ws, ws_bytes = _workspace(workspace, _union_workspace(cache.H, G, cache.D, M), q, stream)
    sc = cache.D ** -0.5 if scale is None else float(scale)
    _check(L.fathom_paged_union_attention(cache._ref, table.data_ptr(), table.numel(), n, q.data_ptr(), G,
                                          union_idx.data_ptr(), union_count.data_ptr(), M, sc, out.data_ptr(), ws,
                                          ws_bytes, _stream(stream)), "fathom_paged_union_attention")
    return out


def device_status(clear: bool = False, stream=None) -> int:
    """OK, or ERR_TIMEOUT if a library kernel on the current device gave up
    a bounded wait since the fault word was last cleared (synchronises the
    stream)."""
    st = int(lib().fathom_device_status(1 if clear else 0, _stream(stream)))
    if st not in (OK, ERR_TIMEOUT, ERR_BOUNDS):
        _check(st, "fathom_device_status")
    return st


class Step:
    """One decode step of the scan over a resident index: plan -> candidate
    scan -> top-k + union, with the dense rerun for any group whose
    candidate pass could not prove its top-k exact.  Buffers are allocated
    once; ``run`` launches only library kernels.  With ``nibbles`` the scans
    read that nibble store (every active channel whole) instead of the
    planes; with ``token_major`` too, it is the token-major store."""

    def __init__(self, planes, scales, n: int, sigma2, G: int, k: int, budget=48, fixed_r: int | None = None,
                 fixed_bits: int = 4, nibbles=None, token_major: bool = False):
        self.planes, self.scales, self.n, self.sigma2, self.k = planes, scales, n, sigma2, k
        self.nibbles = nibbles
        self.token_major = token_major   # ``nibbles`` is the token-major store
        self.store = planes if nibbles is None else nibbles
        self.H, self.D = sigma2.shape
        self.G = G
        self.budget = budget
        self.fixed_r = fixed_r
        self.fixed_bits = fixed_bits
        dev = sigma2.device
        H, D = self.H, self.D
        self.plan_out = (torch.empty((H, D), dtype=torch.uint8, device=dev),
                         torch.empty((H, D), dtype=torch.int16, device=dev),
                         torch.empty(H, dtype=torch.int32, device=dev),
                         torch.empty(H, dtype=torch.float32, device=dev))
        self.cand = torch.empty(scan_cand_bytes(H, G, n, k), dtype=torch.uint8, device=dev)
        self.topk_out = (torch.empty((H, G, k), dtype=torch.int32, device=dev),
                         torch.empty((H, G * k), dtype=torch.int32, device=dev),
                         torch.empty(H, dtype=torch.int32, device=dev))

    def run_plan(self, q):
        if self.fixed_r is None:
            plan(self.sigma2, q, self.budget, out=self.plan_out)
        else:
            plan_fixed(q, self.fixed_r, out=self.plan_out[:3], bits=self.fixed_bits)
        return self.plan_out

    def run_prepare(self, q):
        _, active, n_active, _ = self.plan_out
        return scan(self.store, self.scales, self.n, active, n_active, q, SCAN_PREPARE, self.k, cand=self.cand,
                    nibbles=self.nibbles is not None, token_major=self.token_major)

    def run_filter(self, q):
        _, active, n_active, _ = self.plan_out
        return scan(self.store, self.scales, self.n, active, n_active, q, SCAN_FILTER, self.k, cand=self.cand,
                    nibbles=self.nibbles is not None, token_major=self.token_major)

    def run_scan(self, q):
        self.run_prepare(q)
        return self.run_filter(q)

    def run_topk(self):
        return topk(self.H, self.G, self.n, self.k, cand=self.cand, out=self.topk_out)

    def run(self, q, check_overflow: bool = True):
        self.run_plan(q)
        self.run_scan(q)
        idx, uni, cnt = self.run_topk()
        if check_overflow:
            self.repair(q)
        return idx, uni, cnt

    def repair(self, q) -> int:
        """Dense rerun of groups whose candidate pass overflowed (host check)."""
        idx, uni, cnt = self.topk_out
        bad = torch.nonzero(cnt < 0).flatten().tolist()
        if not bad:
            return 0
        if int(cnt[bad[0]]) in (ERR_TIMEOUT, ERR_BOUNDS):
            raise FathomError(int(cnt[bad[0]]), "candidate scan (device fault word set)")
        _, active, n_active, _ = self.plan_out
        for h in bad:
            sl = slice(h, h + 1)
            sc = scan(self.store[sl], self.scales[sl], self.n, active[sl], n_active[sl], q[sl], SCAN_DENSE,
                      nibbles=self.nibbles is not None, token_major=self.token_major)
            topk(1, self.G, self.n, self.k, scores=sc, out=(idx[sl], uni[sl], cnt[sl]))
        return len(bad)
