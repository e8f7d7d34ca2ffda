"""ctypes binding of libsidbeam.so: the C ABI of include/sidbeam.h, same names.

Argument marshalling only: device buffers are torch CUDA tensors (their
data_ptr() is passed), streams are torch.cuda.Stream objects (default: the
current stream). Every computation runs in the library's kernels; there is no
CPU fallback, and loading fails loudly when the shared object is missing.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsidbeam.so")

_BF16, _F32, _I32, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn

SIDBEAM_OK = 0
SIDBEAM_ERR_INVALID_ARG = -1
SIDBEAM_ERR_BAD_CATALOG = -2
SIDBEAM_ERR_ALIGNMENT = -3
SIDBEAM_ERR_WORKSPACE = -4
SIDBEAM_ERR_OOM = -5
SIDBEAM_ERR_CUDA = -6
SIDBEAM_ERR_DEVICE_CHECK = -7
SIDBEAM_ERR_TIMEOUT = -8

SIDBEAM_F32 = 0
SIDBEAM_BF16 = 1

LAYOUT_AUTO = 0
LAYOUT_DENSE = 1
LAYOUT_CSR = 2

MAX_DEPTH = 16
MAX_V = 32768
MAX_BEAM = 4096

# Every symbol include/sidbeam.h declares.
EXPORTED = (
    "sid_trie_build", "sid_trie_info", "sid_trie_leaf_rows", "sid_trie_leaf_codes",
    "sid_trie_free", "beam_step_workspace_size", "beam_step", "beam_finalize",
    "catalog_score_workspace_size", "catalog_score_topk", "sidbeam_get_device_status",
    "sidbeam_last_error", "sidbeam_version", "beam_step_noalloc", "lmhead_logits",
    "fused_lmhead_workspace_size", "sidbeam_fused_lmhead_step", "beam_step_ex",
    "beam_step_skipped_rows", "catalog_score_topk_sim", "beam_step_gumbel",
    "beam_step_gumbel_workspace_size", "residual_rmsnorm_fp8", "lmhead_quantize_fp8",
    "lmhead_logits_fp8", "beam_attention",
)

FP8_BLOCK = 128      # SIDBEAM_FP8_BLOCK: elements that share a scale
MAX_HIDDEN = 16384   # SIDBEAM_MAX_HIDDEN

STEP_SKIP_ROWS = 1  # SIDBEAM_STEP_SKIP_ROWS

NOALLOC_SCRATCH_BYTES = 4 << 20


class SidbeamError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"sidbeam status {status}: {message}")
        self.status = status


_lib = None


def load():
    """Load libsidbeam.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing; build it with `python -m trie_constrained_beam_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    L.sid_trie_build.argtypes = [P, I64, I32, P, P, P, ctypes.POINTER(P)]
    L.sid_trie_info.argtypes = [P, I32, ctypes.POINTER(I64), ctypes.POINTER(I32), ctypes.POINTER(SZ)]
    L.sid_trie_leaf_rows.argtypes = [P, P, P]
    L.sid_trie_leaf_codes.argtypes = [P, P, P]
    L.sid_trie_free.argtypes = [P]
    L.sid_trie_free.restype = None
    L.beam_step_workspace_size.argtypes = [I32, I32, I32, I32]
    L.beam_step_workspace_size.restype = SZ
    L.beam_step.argtypes = [P, I32, P, I32, I64, P, P, I32, I32, I32, I32, P, P, P, P, P, SZ, P]
    L.beam_step_noalloc.argtypes = [P, I32, P, I32, I64, P, P, I32, I32, I32, I32, P, P, P, P, P]
    L.beam_step_ex.argtypes = [P, I32, P, I32, I64, P, P, I32, I32, I32, I32, P, P, P, P, P, SZ, P,
                               ctypes.c_uint, P]
    L.beam_step_skipped_rows.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), P]
    L.beam_step_gumbel_workspace_size.argtypes = [I32, I32, I32, I32]
    L.beam_step_gumbel_workspace_size.restype = SZ
    L.beam_step_gumbel.argtypes = [P, I32, P, I32, I64, P, P, I32, I32, I32, I32, ctypes.c_float,
                                   ctypes.c_uint64, P, P, P, P, P, SZ, P]
    L.beam_finalize.argtypes = [I32, I32, I32, P, P, P, P, P, P]
    L.catalog_score_workspace_size.argtypes = [P, I32, I32]
    L.catalog_score_workspace_size.restype = SZ
    L.catalog_score_topk.argtypes = [P, P, I32, I32, P, P, P, SZ, P]
    L.catalog_score_topk_sim.argtypes = [P, P, P, P, I32, I32, I32, P, P, P, SZ, P]
    L.sidbeam_get_device_status.argtypes = [P, P]
    L.lmhead_logits.argtypes = [P, P, I32, I32, I32, P, I64, P, SZ, P]
    L.fused_lmhead_workspace_size.argtypes = [I32, I32, I32, I32]
    L.fused_lmhead_workspace_size.restype = SZ
    L.sidbeam_fused_lmhead_step.argtypes = [P, I32, P, P, I32, P, P, I32, I32, I32, I32, P, P, P,
                                            P, P, SZ, P]
    L.residual_rmsnorm_fp8.argtypes = [P, P, P, ctypes.c_float, I32, I32, P, P, P, P]
    L.lmhead_quantize_fp8.argtypes = [P, I32, I32, P, P, P]
    L.lmhead_logits_fp8.argtypes = [P, P, P, P, I32, I32, I32, P, I32, I64, P, SZ, P]
    L.beam_attention.argtypes = [P, P]
    L.sidbeam_last_error.argtypes = []
    L.sidbeam_last_error.restype = ctypes.c_char_p
    L.sidbeam_version.argtypes = []
    L.sidbeam_version.restype = ctypes.c_char_p
    for name in ("sid_trie_build", "sid_trie_info", "sid_trie_leaf_rows", "sid_trie_leaf_codes",
                 "beam_step", "beam_step_noalloc", "beam_finalize", "catalog_score_topk",
                 "sidbeam_get_device_status", "lmhead_logits", "sidbeam_fused_lmhead_step",
                 "beam_step_ex", "beam_step_skipped_rows", "catalog_score_topk_sim",
                 "beam_step_gumbel", "residual_rmsnorm_fp8", "lmhead_quantize_fp8",
                 "lmhead_logits_fp8", "beam_attention"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def _check(rc: int):
    if rc != SIDBEAM_OK:
        raise SidbeamError(rc, sidbeam_last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    """cudaStream_t of a torch stream; None means torch's current stream
    (or the legacy default stream when torch sees no device)."""
    if stream is None:
        if not torch.cuda.is_available():
            return None
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.float32:
        return SIDBEAM_F32
    if t.dtype == torch.bfloat16:
        return SIDBEAM_BF16
    raise TypeError(f"logits dtype {t.dtype} is not float32 or bfloat16")


def sidbeam_last_error() -> str:
    return load().sidbeam_last_error().decode()


def sidbeam_version() -> str:
    return load().sidbeam_version().decode()


class Trie:
    """Owner of a sidbeam_trie handle (freed with sid_trie_free)."""

    def __init__(self, handle, depth, codes_per_level):
        self.handle = handle
        self.depth = depth
        self.codes_per_level = list(codes_per_level)

    @property
    def _as_parameter_(self):
        return self.handle

    def close(self):
        if self.handle:
            load().sid_trie_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def sid_trie_build(sids, codes_per_level, layout_per_level=None, stream=None) -> Trie:
    """sids: host int array [n_sids, depth]."""
    L = load()
    sids = np.ascontiguousarray(sids, dtype=np.int32)
    n, depth = sids.shape
    cpl = np.ascontiguousarray(codes_per_level, dtype=np.int32)
    lay = None if layout_per_level is None else np.ascontiguousarray(layout_per_level, dtype=np.int32)
    out = ctypes.c_void_p()
    rc = L.sid_trie_build(sids.ctypes.data, n, depth, cpl.ctypes.data,
                          None if lay is None else lay.ctypes.data, _stream(stream),
                          ctypes.byref(out))
    _check(rc)
    return Trie(out, depth, cpl.tolist())


def sid_trie_info(trie: Trie, level: int):
    n = ctypes.c_int64()
    lay = ctypes.c_int()
    nb = ctypes.c_size_t()
    _check(load().sid_trie_info(trie.handle, level, ctypes.byref(n), ctypes.byref(lay),
                                ctypes.byref(nb)))
    return n.value, lay.value, nb.value


def sid_trie_leaf_rows(trie: Trie, out, stream=None):
    _check(load().sid_trie_leaf_rows(trie.handle, _ptr(out), _stream(stream)))


def sid_trie_leaf_codes(trie: Trie, out, stream=None):
    _check(load().sid_trie_leaf_codes(trie.handle, _ptr(out), _stream(stream)))


def beam_step_workspace_size(R: int, B_in: int, n_out: int, V: int) -> int:
    return int(load().beam_step_workspace_size(R, B_in, n_out, V))


def beam_step(trie, step, logits, parent_scores, parent_nodes, R, B_in, n_out, V,
              out_scores, out_parent, out_code, out_node, workspace, stream=None, ld=None,
              skip_rows=False, out_width=None):
    """logits: torch [R*B_in, ld] float32/bfloat16 on the device (row stride = ld).
    skip_rows: do not read rows that cannot contribute (beam_step_ex with
    SIDBEAM_STEP_SKIP_ROWS); the results are the same. out_width: optional
    device int32 [R], beams kept per request (the rest of n_out is padding)."""
    if ld is None:
        ld = logits.stride(0)
    args = (None if trie is None else trie.handle, step, _ptr(logits), _dtype_code(logits), ld,
            _ptr(parent_scores), _ptr(parent_nodes), R, B_in, n_out, V, _ptr(out_scores),
            _ptr(out_parent), _ptr(out_code), _ptr(out_node), _ptr(workspace),
            0 if workspace is None else workspace.numel() * workspace.element_size(),
            _stream(stream))
    if skip_rows or out_width is not None:
        rc = load().beam_step_ex(*args, STEP_SKIP_ROWS if skip_rows else 0,
                                 None if out_width is None else _ptr(out_width))
    else:
        rc = load().beam_step(*args)
    _check(rc)


def beam_step_gumbel_workspace_size(R: int, B_in: int, n_out: int, V: int) -> int:
    return int(load().beam_step_gumbel_workspace_size(R, B_in, n_out, V))


def beam_step_gumbel(trie, step, logits, parent_scores, parent_nodes, R, B_in, n_out, V,
                     temperature, seed, out_scores, out_parent, out_code, out_node, workspace,
                     stream=None, ld=None):
    """Gumbel top-k step at `temperature` (0: the deterministic step); `seed`
    keys the Philox stream. Outputs in draw order; scores unperturbed."""
    if ld is None:
        ld = logits.stride(0)
    rc = load().beam_step_gumbel(None if trie is None else trie.handle, step, _ptr(logits),
                                 _dtype_code(logits), ld, _ptr(parent_scores),
                                 _ptr(parent_nodes), R, B_in, n_out, V, float(temperature),
                                 int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(out_scores),
                                 _ptr(out_parent), _ptr(out_code), _ptr(out_node),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream))
    _check(rc)


def beam_step_skipped_rows(workspace, stream=None) -> int:
    """Rows row skipping left unread since the last call (the counter resets)."""
    c = ctypes.c_uint32(0)
    _check(load().beam_step_skipped_rows(_ptr(workspace), ctypes.byref(c), _stream(stream)))
    return int(c.value)


def beam_step_noalloc(trie, step, logits, parent_scores, parent_nodes, R, B_in, n_out, V,
                      out_scores, out_parent, out_code, out_node, stream=None, ld=None):
    """beam_step with the library's built-in scratch instead of a workspace; for
    callers that cannot allocate device memory. Calls must not overlap on the GPU."""
    if ld is None:
        ld = logits.stride(0)
    rc = load().beam_step_noalloc(None if trie is None else trie.handle, step, _ptr(logits),
                                  _dtype_code(logits), ld, _ptr(parent_scores),
                                  _ptr(parent_nodes), R, B_in, n_out, V, _ptr(out_scores),
                                  _ptr(out_parent), _ptr(out_code), _ptr(out_node),
                                  _stream(stream))
    _check(rc)


def beam_finalize(depth, R, n, bp_parent, bp_code, last_node, out_sids, out_leaf, stream=None):
    _check(load().beam_finalize(depth, R, n, _ptr(bp_parent), _ptr(bp_code), _ptr(last_node),
                                _ptr(out_sids), _ptr(out_leaf), _stream(stream)))


def catalog_score_workspace_size(trie: Trie, R: int, K: int) -> int:
    return int(load().catalog_score_workspace_size(trie.handle, R, K))


def catalog_score_topk(trie, logp, R, K, out_scores, out_leaf, workspace, stream=None):
    rc = load().catalog_score_topk(trie.handle, _ptr(logp), R, K, _ptr(out_scores),
                                   _ptr(out_leaf), _ptr(workspace),
                                   0 if workspace is None else workspace.numel() * workspace.element_size(),
                                   _stream(stream))
    _check(rc)


def catalog_score_topk_sim(trie, logp, user, sid_emb, R, K, out_scores, out_leaf, workspace,
                           stream=None):
    """catalog_score_topk plus <user[r], sid_emb[leaf]>: user f32 [R][d], sid_emb
    bf16 [N][d] (leaf-id order), both on the device."""
    d = int(user.shape[1])
    if int(sid_emb.shape[1]) != d:
        raise ValueError("user and sid_emb disagree on d")
    rc = load().catalog_score_topk_sim(trie.handle, _ptr(logp), _ptr(user), _ptr(sid_emb), d, R,
                                       K, _ptr(out_scores), _ptr(out_leaf), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       _stream(stream))
    _check(rc)


def lmhead_logits(hidden, w_sid, out, workspace, stream=None):
    """out[row][c] = sum_k hidden[row][k] * w_sid[c][k] (bf16 in, fp32 out) on the
    tensor cores. hidden [M][d], w_sid [V][d] bf16; out f32 [M][>= V]."""
    M, d = hidden.shape
    V = w_sid.shape[0]
    _check(load().lmhead_logits(_ptr(hidden), _ptr(w_sid), M, V, d, _ptr(out), out.stride(0),
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream)))


def fused_lmhead_workspace_size(R: int, B_in: int, n_out: int, V: int) -> int:
    return int(load().fused_lmhead_workspace_size(R, B_in, n_out, V))


def fused_lmhead_step(trie, step, hidden, w_sid, parent_scores, parent_nodes, R, B_in, n_out,
                      out_scores, out_parent, out_code, out_node, workspace, stream=None):
    """beam_step on logits = hidden @ w_sid.T made on the tensor cores and never
    written out. hidden bf16 [R*B_in][d], w_sid bf16 [V][d]."""
    d = hidden.shape[1]
    V = w_sid.shape[0]
    rc = load().sidbeam_fused_lmhead_step(
        None if trie is None else trie.handle, step, _ptr(hidden), _ptr(w_sid), d,
        _ptr(parent_scores), _ptr(parent_nodes), R, B_in, n_out, V, _ptr(out_scores),
        _ptr(out_parent), _ptr(out_code), _ptr(out_node), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc)


def _refuse(index, *args):
    """Raises for the first argument (tensor, name, dtype, shape of a contiguous
    tensor or None) that does not fit a call on CUDA device `index`."""
    for t, name, dtype, shape in args:
        if t is None:
            if name in ("residual", "residual_out"):
                continue
            raise ValueError(f"{name} is missing")
        if t.dtype is not dtype:
            raise TypeError(f"{name} dtype {t.dtype} is not {dtype}")
        at = t.get_device()
        if at != index or at < 0:
            raise ValueError(f"{name} is on {t.device}, not on CUDA device {max(index, 0)}")
        if shape is not None and (t.shape != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}, "
                             f"got {tuple(t.shape)} with strides {t.stride()}")
    raise ValueError("arguments do not fit")


def _fits(t, dtype, index, shape):
    """Whether t is a contiguous tensor of that type, device and shape."""
    return (t.dtype is dtype and t.get_device() == index and t.shape == shape
            and t.is_contiguous())


def _run_on(index, stream, fn, *args):
    """Calls a C entry on CUDA device `index`: on `stream`, or on that device's
    current stream. (torch._C's calls, without the wrappers of torch.cuda, are on
    the way of every launch. A torch built without CUDA lacks them: they are looked
    up here, not on import.)"""
    s = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, s)
    if rc != SIDBEAM_OK:
        raise SidbeamError(rc, sidbeam_last_error())


def residual_rmsnorm_fp8(x, residual, weight, eps, residual_out, hidden_q, hidden_scale,
                         stream=None):
    """h = x + residual; y = h / sqrt(mean h^2 + eps) * weight, left in 8 bits:
    hidden_q e4m3 [M][d] with hidden_scale f32 [M][ceil(d/128)], a scale per 128
    columns. x, residual (or None) bf16 [M][d], weight bf16 [d]; residual_out
    (or None) receives h in bf16 and may be x or residual itself."""
    shape = M, d = x.shape
    at = x.get_device()
    scales = (M, (d + FP8_BLOCK - 1) // FP8_BLOCK)
    if not (at >= 0 and x.dtype is _BF16 and x.is_contiguous()
            and (residual is None or _fits(residual, _BF16, at, shape))
            and _fits(weight, _BF16, at, (d,))
            and (residual_out is None or _fits(residual_out, _BF16, at, shape))
            and _fits(hidden_q, _E4M3, at, shape) and _fits(hidden_scale, _F32, at, scales)):
        _refuse(at, (x, "x", _BF16, shape), (residual, "residual", _BF16, shape),
                (weight, "weight", _BF16, (d,)), (residual_out, "residual_out", _BF16, shape),
                (hidden_q, "hidden_q", _E4M3, shape), (hidden_scale, "hidden_scale", _F32, scales))
    _run_on(at, stream, (_lib or load()).residual_rmsnorm_fp8, x.data_ptr(),
            None if residual is None else residual.data_ptr(), weight.data_ptr(), eps, M, d,
            None if residual_out is None else residual_out.data_ptr(), hidden_q.data_ptr(),
            hidden_scale.data_ptr())


def lmhead_quantize_fp8(w_sid, w_q, w_scale, stream=None):
    """The lm_head weight in 8 bits for lmhead_logits_fp8: w_sid bf16 [V][d] ->
    w_q e4m3 [V][d], w_scale f32 [ceil(V/128)][ceil(d/128)]."""
    shape = V, d = w_sid.shape
    at = w_sid.get_device()
    scales = ((V + FP8_BLOCK - 1) // FP8_BLOCK, (d + FP8_BLOCK - 1) // FP8_BLOCK)
    if not (at >= 0 and w_sid.dtype is _BF16 and w_sid.is_contiguous()
            and _fits(w_q, _E4M3, at, shape) and _fits(w_scale, _F32, at, scales)):
        _refuse(at, (w_sid, "w_sid", _BF16, shape), (w_q, "w_q", _E4M3, shape),
                (w_scale, "w_scale", _F32, scales))
    _run_on(at, stream, (_lib or load()).lmhead_quantize_fp8, w_sid.data_ptr(), V, d,
            w_q.data_ptr(), w_scale.data_ptr())


def lmhead_logits_fp8(hidden_q, hidden_scale, w_q, w_scale, out, workspace, stream=None):
    """lmhead_logits on operands in 8 bits: out[row][c] = sum over blocks of 128
    columns of hidden_scale[row][b] * w_scale[c // 128][b] * <hidden_q, w_q>_b
    (fp32 accumulation). out f32 or bf16 [M][V], rows out.stride(0) apart."""
    M, d = hidden_q.shape
    V = w_q.shape[0]
    nb = (d + FP8_BLOCK - 1) // FP8_BLOCK
    at = hidden_q.get_device()
    dtype = _dtype_code(out)
    ld, col = out.stride()
    if out.shape != (M, V) or (V > 1 and col != 1):
        raise ValueError(f"out must be [{M}, {V}] with unit column stride, got "
                         f"{tuple(out.shape)} with strides {out.stride()}")
    if M <= 1:  # the stride of a single row means nothing: any aligned one serves
        ld = (V + 7) // 8 * 8
    vb = (V + FP8_BLOCK - 1) // FP8_BLOCK
    if not (at >= 0 and hidden_q.dtype is _E4M3 and hidden_q.is_contiguous()
            and _fits(hidden_scale, _F32, at, (M, nb)) and _fits(w_q, _E4M3, at, (V, d))
            and _fits(w_scale, _F32, at, (vb, nb)) and out.get_device() == at
            and workspace.get_device() == at):
        _refuse(at, (hidden_q, "hidden_q", _E4M3, (M, d)),
                (hidden_scale, "hidden_scale", _F32, (M, nb)), (w_q, "w_q", _E4M3, (V, d)),
                (w_scale, "w_scale", _F32, (vb, nb)), (out, "out", out.dtype, None),
                (workspace, "workspace", workspace.dtype, None))
    _run_on(at, stream, (_lib or load()).lmhead_logits_fp8, hidden_q.data_ptr(),
            hidden_scale.data_ptr(), w_q.data_ptr(), w_scale.data_ptr(), M, V, d, out.data_ptr(),
            dtype, ld, workspace.data_ptr(), workspace.nbytes)


# The fields of sidbeam_attention in the header's order (native alignment).
_ATTENTION = struct.Struct("PqPPqqiiPPPPPiiiiiiifPqPN").pack


def beam_attention(q, k_cache, v_cache, cache_len, out, workspace, page_table=None, level=0,
                   k_beam=None, v_beam=None, bp_parent=None, scale=None, stream=None):
    """Attention of beam rows over their request's prompt cache and, for level > 0,
    their own ancestors through the back-pointer history.

    q, out      bf16 [R*B, H, D] (rows request-major, any row stride)
    k_cache,    bf16 [R, capacity, Hkv, D], or with page_table int32 [R, pages]
    v_cache     [n_pages, page_size, Hkv, D]; the same strides for both
    cache_len   int32 [R] prompt tokens of each request
    level       steps behind the rows; the first `level` slices of bp_parent
                int32 [depth, R, B] and of k_beam, v_beam bf16 [depth, R*B, Hkv, D]
    scale       default D ** -0.5
    """
    rows, H, D = q.shape
    n_pages, page_size, Hkv, Dk = k_cache.shape
    R = cache_len.shape[0]
    B = rows // R if R else 0
    at = q.get_device()
    if R < 1 or B * R != rows:
        raise ValueError(f"{rows} query rows for {R} requests")
    if v_cache.shape != k_cache.shape or v_cache.stride() != k_cache.stride():
        raise ValueError("k_cache and v_cache differ in shape or strides")
    if out.shape != q.shape or Dk != D:
        raise ValueError(f"shapes of q {tuple(q.shape)}, out {tuple(out.shape)} and k_cache "
                         f"{tuple(k_cache.shape)} do not match")
    q_row, q_head, q_one = q.stride()
    o_row, o_head, o_one = out.stride()
    page, token, k_head, k_one = k_cache.stride()
    if (q_one != 1 or o_one != 1 or k_one != 1 or (H > 1 and (q_head != D or o_head != D))
            or (Hkv > 1 and k_head != D)):
        raise ValueError("the heads of a row must be contiguous in q, out and the caches")
    # Axes of one element: their stride means nothing, the packed one serves.
    if rows == 1:
        q_row = o_row = H * D
    if page_size == 1:
        token = Hkv * D
    if n_pages == 1:
        page = page_size * token
    table = per = kb = vb = bp = 0
    if not (at >= 0 and q.dtype is _BF16 and k_cache.dtype is _BF16 and v_cache.dtype is _BF16
            and out.dtype is _BF16 and k_cache.get_device() == at and v_cache.get_device() == at
            and out.get_device() == at and workspace.get_device() == at
            and _fits(cache_len, _I32, at, (R,))):
        _refuse(at, (q, "q", _BF16, None), (k_cache, "k_cache", _BF16, None),
                (v_cache, "v_cache", _BF16, None), (cache_len, "cache_len", _I32, (R,)),
                (out, "out", _BF16, None), (workspace, "workspace", workspace.dtype, None))
    if page_table is not None:
        per = page_table.shape[-1]
        if not _fits(page_table, _I32, at, (R, per)):
            _refuse(at, (page_table, "page_table", _I32, (R, per)))
        table = page_table.data_ptr()
    if level > 0:
        for t, name in ((bp_parent, "bp_parent"), (k_beam, "k_beam"), (v_beam, "v_beam")):
            if t is None or t.shape[0] < level:
                raise ValueError(f"{name} holds fewer than {level} levels")
        links, beams = (bp_parent.shape[0], R, B), (rows, Hkv, D)
        if not (_fits(bp_parent, _I32, at, links)
                and _fits(k_beam, _BF16, at, (k_beam.shape[0], *beams))
                and _fits(v_beam, _BF16, at, (v_beam.shape[0], *beams))):
            _refuse(at, (bp_parent, "bp_parent", _I32, links),
                    (k_beam, "k_beam", _BF16, (k_beam.shape[0], *beams)),
                    (v_beam, "v_beam", _BF16, (v_beam.shape[0], *beams)))
        bp, kb, vb = bp_parent.data_ptr(), k_beam.data_ptr(), v_beam.data_ptr()
    _run_on(at, stream, (_lib or load()).beam_attention, _ATTENTION(
        q.data_ptr(), q_row, k_cache.data_ptr(), v_cache.data_ptr(), page, token, n_pages,
        page_size, table, cache_len.data_ptr(), bp, kb, vb, per, level, R, B, H, Hkv, D,
        D ** -0.5 if scale is None else scale, out.data_ptr(), o_row, workspace.data_ptr(),
        workspace.nbytes))


def sidbeam_get_device_status(workspace, stream=None) -> int:
    return int(load().sidbeam_get_device_status(_ptr(workspace), _stream(stream)))
