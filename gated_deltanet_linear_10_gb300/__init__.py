"""Python binding of libgdn, the GB300 Gated DeltaNet layer library.

Each function below has the name of a C entry point declared in
``include/gdn.h`` and only marshals arguments: it checks shapes, dtypes and
devices of PyTorch tensors, allocates the outputs that were not passed (with
PyTorch), and calls the C ABI on the current CUDA stream.  Every step of the
computation runs in the library's CUDA kernels; there is no other path.  If
``libgdn.so`` is not built, importing this package raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

(GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_LAUNCH, GDN_ERR_CUDA,
 GDN_ERR_TOO_LARGE) = range(6)
PREFILL_STATIC_SCRATCH_BYTES = 16 << 20
GDN_F32, GDN_BF16, GDN_E4M3 = 0, 1, 2
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
DEVSTAT_BAD_INDEX, DEVSTAT_BAD_SEQLEN, DEVSTAT_TIMEOUT = 0x1, 0x2, 0x4

# Every symbol the header declares (checked by the tests against the .so).
EXPORTS = (
    "gdn_status_string", "gdn_version", "gdn_last_cuda_error", "gdn_gating",
    "causal_conv1d_fwd", "causal_conv1d_update", "gdn_prefill_chunked",
    "gdn_prefill_workspace_size", "gdn_decode_recurrent", "gdn_state_snapshot",
    "gdn_get_device_status", "gdn_prefill_chunked_static", "gdn_gated_rmsnorm",
    "gdn_decode_recurrent_gated", "gdn_decode_step_fused", "gdn_mixed_batch",
    "gdn_debug_set_wait_limit", "gdn_prefill_chunked_gated", "gdn_mtp_step_fused",
    "gdn_decode_step_workspace_size", "gdn_prefill_layer", "gdn_prefill_layer_workspace_size",
    "gdn_prefill_layer_gated", "gdn_add_rmsnorm", "gdn_gated_rmsnorm_quant", "gdn_linear",
    "gdn_linear_block", "gdn_moe_route", "gdn_moe_route_workspace_size", "gdn_block_quant",
    "gdn_grouped_linear", "gdn_moe_combine", "gdn_debug_set_grouped_tile",
)

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built: run `python -c 'import __graft_entry__ as g; "
                      f"g.build()'` (nvcc, sm_103a) first")

_lib = ctypes.CDLL(LIB_PATH)

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_lib.gdn_status_string.restype = ctypes.c_char_p
_lib.gdn_status_string.argtypes = [ctypes.c_int]
_lib.gdn_version.restype = ctypes.c_char_p
_lib.gdn_version.argtypes = []
_lib.gdn_last_cuda_error.restype = ctypes.c_char_p
_lib.gdn_last_cuda_error.argtypes = []
_SIGS = {
    "gdn_gating": [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp, _vp],
    "causal_conv1d_fwd": [_vp, _i64, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _vp, _i64, _vp, _vp,
                          _i32, _vp, _i32, _vp],
    "causal_conv1d_update": [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _vp, _i32,
                             _vp, _i32, _vp],
    "gdn_prefill_chunked": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _i64, _i32,
                            _i32, _i32, _i32, _f32, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _i32,
                            _vp, ctypes.c_size_t, _vp],
    "gdn_decode_recurrent": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _i32,
                             _i32, _i32, _f32, _i32, _vp, _i64, _vp, _vp, _vp, _i32, _vp],
    "gdn_state_snapshot": [_vp, _i64, _i64, _vp, _vp, _i32, _vp],
    "gdn_get_device_status": [ctypes.POINTER(ctypes.c_uint32), _i32, _vp],
    "gdn_decode_step_fused": [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                              _f32, _vp, _i64, _vp, _vp, ctypes.c_size_t, _vp, _vp],
    "gdn_gated_rmsnorm": [_vp, _vp, _i64, _vp, _i64, _i32, _i32, _f32, _vp, _i32, _vp],
    "gdn_add_rmsnorm": [_vp, _i64, _vp, _i64, _vp, _f32, _i64, _i32, _f32, _vp, _i64, _vp, _i64, _vp,
                        _i32, _i32, _vp],
    "gdn_gated_rmsnorm_quant": [_vp, _vp, _i64, _vp, _i64, _i32, _i32, _f32, _vp, _vp, _i32, _vp],
    "gdn_linear": [_vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _i32, _vp,
                   _i64, _i32, _i32, _vp],
    "gdn_linear_block": [_vp, _i64, _vp, _vp, _i64, _vp, _i64, _i32, _i32, _vp, _i64, _i32, _vp],
    "gdn_moe_route": [_vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                      ctypes.c_size_t, _vp],
    "gdn_block_quant": [_vp, _i64, _i64, _i32, _i32, _vp, _i64, _vp, _i32, _vp],
    "gdn_grouped_linear": [_vp, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _i32, _i64, _i32,
                           _i32, _vp, _i64, _i32, _i32, _vp],
    "gdn_moe_combine": [_vp, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp, _i64, _i32, _vp],
    "gdn_debug_set_grouped_tile": [_i32, _i32],
    "gdn_decode_recurrent_gated": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _i32, _i32,
                                   _i32, _i32, _i32, _f32, _i32, _vp, _i64, _vp, _vp, _vp, _i64,
                                   _vp, _f32, _vp, _i32, _vp],
    "gdn_prefill_chunked_static": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _i64,
                                   _i32, _i32, _f32, _i32, _vp, _i64, _vp, _vp, _vp, _vp],
    "gdn_debug_set_wait_limit": [ctypes.c_uint64, _i32, _vp],
    "gdn_prefill_layer": [_vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                          _i64, _i32, _i32, _f32, _vp, _i64, _vp, _vp, _vp, _vp,
                          ctypes.c_size_t, _vp],
    "gdn_prefill_layer_gated": [_vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                _i32, _i64, _i32, _i32, _f32, _vp, _i64, _vp, _vp, _vp, _i64, _vp,
                                _f32, _vp, _vp, ctypes.c_size_t, _vp],
    "gdn_mtp_step_fused": [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                           _f32, _vp, _i64, _vp, _vp, _vp, _vp],
    "gdn_prefill_chunked_gated": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _i64,
                                  _i32, _i32, _i32, _i32, _f32, _i32, _i32, _vp, _i64, _vp, _vp,
                                  _vp, _i64, _vp, _f32, _vp, _i32, _vp, ctypes.c_size_t, _vp],
    "gdn_mixed_batch": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i64, _i32,
                        _i32, _i32, _i32, _f32, _i32, _i32, _vp, _i64, _vp, _vp, _i32, _vp, _i32,
                        _vp, ctypes.c_size_t, _vp],
}
for _name, _args in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = ctypes.c_int
_lib.gdn_prefill_workspace_size.argtypes = [_i32, _i64, _i32, _i32, _i32, _i32, _i32]
_lib.gdn_prefill_workspace_size.restype = ctypes.c_size_t
_lib.gdn_decode_step_workspace_size.argtypes = [_i32, _i32, _i32]
_lib.gdn_decode_step_workspace_size.restype = ctypes.c_size_t
_lib.gdn_prefill_layer_workspace_size.argtypes = [_i32, _i64, _i32, _i32]
_lib.gdn_prefill_layer_workspace_size.restype = ctypes.c_size_t
_lib.gdn_moe_route_workspace_size.argtypes = [_i64, _i32]
_lib.gdn_moe_route_workspace_size.restype = ctypes.c_size_t


class GdnError(RuntimeError):
    pass


def _check(status: int, what: str):
    if status != GDN_OK:
        name = _lib.gdn_status_string(status).decode()
        cuda = _lib.gdn_last_cuda_error().decode()
        raise GdnError(f"{what}: {name}" + (f" ({cuda})" if cuda else ""))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GDN_F32
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    raise GdnError(f"unsupported activation dtype {t.dtype} (fp32 or bf16)")


def _need(cond: bool, msg: str):
    if not cond:
        raise GdnError(msg)


def _cuda(*ts):
    for t in ts:
        if t is not None:
            _need(t.is_cuda, "all tensors must be on a CUDA device")


def _i32_vec(t, name):
    if t is None:
        return None
    _need(t.dtype == torch.int32 and t.is_contiguous(), f"{name} must be contiguous int32")
    return t


def _heads_view(x, heads, d, name):
    """x is [T, heads, d] (or [T, heads*d]) with unit inner strides; returns row stride."""
    if x.dim() == 2:
        _need(x.shape[1] == heads * d and x.stride(1) == 1, f"{name}: bad shape/stride")
        return x.stride(0)
    _need(x.dim() == 3 and x.shape[1] == heads and x.shape[2] == d, f"{name}: shape {tuple(x.shape)}")
    _need(x.stride(2) == 1 and x.stride(1) == d, f"{name}: heads must be packed ({x.stride()})")
    return x.stride(0)


def version() -> str:
    return _lib.gdn_version().decode()


def gdn_gating(a, b, A_log, dt_bias, g=None, beta=None):
    """g = -exp(A_log) softplus(a + dt_bias), beta = sigmoid(b); a, b: [T, hv]."""
    _cuda(a, b, A_log, dt_bias)
    _need(a.shape == b.shape and a.dim() == 2 and a.dtype == b.dtype, "a, b: [T, hv], same dtype")
    _need(a.is_contiguous() and b.is_contiguous(), "a, b must be contiguous")
    T, hv = a.shape
    _need(A_log.dtype == torch.float32 and dt_bias.dtype == torch.float32, "A_log/dt_bias fp32")
    _need(A_log.numel() == hv and dt_bias.numel() == hv, "A_log/dt_bias: [hv]")
    g = torch.empty((T, hv), dtype=torch.float32, device=a.device) if g is None else g
    beta = torch.empty((T, hv), dtype=torch.float32, device=a.device) if beta is None else beta
    _check(_lib.gdn_gating(_ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias), T, hv, _dtype_code(a),
                           _ptr(g), _ptr(beta), _stream(a.device)), "gdn_gating")
    return g, beta


def causal_conv1d_fwd(x, weight, cu_seqlens, conv_state_pool, state_indices,
                      has_initial_state=None, bias=None, silu=True, y=None):
    """Varlen causal conv1d (+SiLU); x [T, C] (row stride free), weight [C, W],
    conv_state_pool [slots, W-1, C]; returns y [T, C]."""
    _cuda(x, weight, cu_seqlens, conv_state_pool, state_indices, has_initial_state, bias)
    _need(x.dim() == 2 and x.stride(1) == 1, "x: [T, C] with unit column stride")
    T, C = x.shape
    _need(weight.shape[0] == C and weight.is_contiguous() and weight.dtype == x.dtype, "weight")
    W = weight.shape[1]
    _need(conv_state_pool.shape[1:] == (W - 1, C) and conv_state_pool.is_contiguous()
          and conv_state_pool.dtype == x.dtype, "conv_state_pool: [slots, W-1, C]")
    _i32_vec(cu_seqlens, "cu_seqlens")
    _i32_vec(state_indices, "state_indices")
    n = cu_seqlens.numel() - 1
    _need(state_indices.numel() == n, "state_indices: [n_seqs]")
    if has_initial_state is not None:
        _need(has_initial_state.dtype == torch.uint8 and has_initial_state.numel() == n,
              "has_initial_state: [n_seqs] uint8")
    y = torch.empty((T, C), dtype=x.dtype, device=x.device) if y is None else y
    _check(_lib.causal_conv1d_fwd(_ptr(x), x.stride(0), _ptr(weight), _ptr(bias), _ptr(cu_seqlens),
                                  n, T, C, W, _ptr(conv_state_pool), conv_state_pool.shape[0],
                                  _ptr(state_indices), _ptr(has_initial_state), int(silu), _ptr(y),
                                  _dtype_code(x), _stream(x.device)), "causal_conv1d_fwd")
    return y


def causal_conv1d_update(x, tokens_per_seq, weight, conv_state_pool, state_indices,
                         snap_indices=None, bias=None, silu=True, y=None):
    """Decode / MTP conv update; x [N*tps, C] contiguous (row i*tps + t)."""
    _cuda(x, weight, conv_state_pool, state_indices, snap_indices, bias)
    _need(x.dim() == 2 and x.is_contiguous(), "x: [N*tps, C] contiguous")
    _i32_vec(state_indices, "state_indices")
    _i32_vec(snap_indices, "snap_indices")
    N = state_indices.numel()
    _need(x.shape[0] == N * tokens_per_seq, "x rows != n_seqs * tokens_per_seq")
    C = x.shape[1]
    W = weight.shape[1]
    _need(conv_state_pool.shape[1:] == (W - 1, C) and conv_state_pool.dtype == x.dtype,
          "conv_state_pool: [slots, W-1, C]")
    if snap_indices is not None:
        _need(snap_indices.numel() == N * tokens_per_seq, "snap_indices: [n_seqs, tps]")
    y = torch.empty_like(x) if y is None else y
    _check(_lib.causal_conv1d_update(_ptr(x), N, tokens_per_seq, C, W, _ptr(weight), _ptr(bias),
                                     _ptr(conv_state_pool), conv_state_pool.shape[0],
                                     _ptr(state_indices), _ptr(snap_indices), int(silu), _ptr(y),
                                     _dtype_code(x), _stream(x.device)), "causal_conv1d_update")
    return y


def gdn_prefill_workspace_size(n_seqs, n_tokens, hv, dk, dv, chunk, dtype=GDN_BF16) -> int:
    return int(_lib.gdn_prefill_workspace_size(n_seqs, n_tokens, hv, dk, dv, chunk, dtype))


def gdn_prefill_chunked(q, k, v, g, beta, cu_seqlens, state_pool, initial_state_indices,
                        final_state_indices, scale, chunk=64, l2norm_qk=True, o=None,
                        workspace=None):
    """Chunked varlen prefill.  q, k [T, hqk, dk]; v [T, hv, dv] (views with a
    free row stride); g, beta [T, hv] fp32; state_pool [slots, hv, dv, dk]
    fp32.  Returns o [T, hv, dv].

    workspace: None allocates the scratch gdn_prefill_workspace_size asks for
    (the bf16 dk = dv = 128 path then runs as a chunk-parallel prep kernel and
    a chain kernel); a uint8 CUDA tensor is used as given; False passes none,
    which selects the single fused kernel."""
    _cuda(q, k, v, g, beta, cu_seqlens, state_pool, initial_state_indices, final_state_indices)
    T, hqk, dk = q.shape
    hv, dv = v.shape[1], v.shape[2]
    qs = _heads_view(q, hqk, dk, "q")
    ks = _heads_view(k, hqk, dk, "k")
    vs = _heads_view(v, hv, dv, "v")
    _need(q.dtype == k.dtype == v.dtype, "q, k, v: one dtype")
    _need(g.dtype == torch.float32 and beta.dtype == torch.float32 and g.is_contiguous()
          and beta.is_contiguous() and g.shape == (T, hv) and beta.shape == (T, hv), "g, beta")
    _need(state_pool.dtype == torch.float32 and state_pool.is_contiguous()
          and state_pool.shape[1:] == (hv, dv, dk), "state_pool: [slots, hv, dv, dk] fp32")
    _i32_vec(cu_seqlens, "cu_seqlens")
    n = cu_seqlens.numel() - 1
    for name, t in (("initial_state_indices", initial_state_indices),
                    ("final_state_indices", final_state_indices)):
        if t is not None:
            _i32_vec(t, name)
            _need(t.numel() == n, f"{name}: [n_seqs]")
    o = torch.empty((T, hv, dv), dtype=q.dtype, device=q.device) if o is None else o
    _need(o.is_contiguous() and o.shape == (T, hv, dv), "o: [T, hv, dv] contiguous")
    dt = _dtype_code(q)
    if workspace is False:
        workspace = None
    elif workspace is None:
        need = gdn_prefill_workspace_size(n, T, hv, dk, dv, chunk, dt)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _cuda(workspace)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.gdn_prefill_chunked(_ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(g), _ptr(beta),
                                    _ptr(cu_seqlens), n, T, hqk, hv, dk, dv, float(scale),
                                    int(l2norm_qk), chunk, _ptr(state_pool), state_pool.shape[0],
                                    _ptr(initial_state_indices), _ptr(final_state_indices),
                                    _ptr(o), dt, _ptr(workspace), wbytes, _stream(q.device)),
           "gdn_prefill_chunked")
    return o


def gdn_prefill_chunked_gated(q, k, v, g, beta, cu_seqlens, state_pool, initial_state_indices,
                              final_state_indices, scale, z, norm_weight, norm_eps=1e-6, chunk=64,
                              l2norm_qk=True, y=None, workspace=None):
    """gdn_prefill_chunked writing y = RMSNorm(o) * norm_weight * SiLU(z) per
    (token, V head) row instead of o.  z: [T, hv, dv] (a view with a free row
    stride); norm_weight [dv] fp32.  Returns y [T, hv, dv].  workspace as for
    gdn_prefill_chunked."""
    _cuda(q, k, v, g, beta, cu_seqlens, state_pool, initial_state_indices, final_state_indices,
          z, norm_weight)
    T, hqk, dk = q.shape
    hv, dv = v.shape[1], v.shape[2]
    qs = _heads_view(q, hqk, dk, "q")
    ks = _heads_view(k, hqk, dk, "k")
    vs = _heads_view(v, hv, dv, "v")
    zs = _heads_view(z, hv, dv, "z")
    _need(q.dtype == k.dtype == v.dtype == z.dtype, "q, k, v, z: one dtype")
    _need(z.shape[0] == T, "z: [T, hv, dv]")
    _need(norm_weight.dtype == torch.float32 and norm_weight.is_contiguous()
          and norm_weight.shape == (dv,), "norm_weight: [dv] fp32")
    _need(g.dtype == torch.float32 and beta.dtype == torch.float32 and g.is_contiguous()
          and beta.is_contiguous() and g.shape == (T, hv) and beta.shape == (T, hv), "g, beta")
    _need(state_pool.dtype == torch.float32 and state_pool.is_contiguous()
          and state_pool.shape[1:] == (hv, dv, dk), "state_pool: [slots, hv, dv, dk] fp32")
    _i32_vec(cu_seqlens, "cu_seqlens")
    n = cu_seqlens.numel() - 1
    for name, t in (("initial_state_indices", initial_state_indices),
                    ("final_state_indices", final_state_indices)):
        if t is not None:
            _i32_vec(t, name)
            _need(t.numel() == n, f"{name}: [n_seqs]")
    y = torch.empty((T, hv, dv), dtype=q.dtype, device=q.device) if y is None else y
    _need(y.is_contiguous() and y.shape == (T, hv, dv), "y: [T, hv, dv] contiguous")
    dt = _dtype_code(q)
    if workspace is False:
        workspace = None
    elif workspace is None:
        need = gdn_prefill_workspace_size(n, T, hv, dk, dv, chunk, dt)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _cuda(workspace)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.gdn_prefill_chunked_gated(
        _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(g), _ptr(beta), _ptr(cu_seqlens), n, T, hqk,
        hv, dk, dv, float(scale), int(l2norm_qk), chunk, _ptr(state_pool), state_pool.shape[0],
        _ptr(initial_state_indices), _ptr(final_state_indices), _ptr(z), zs, _ptr(norm_weight),
        float(norm_eps), _ptr(y), dt, _ptr(workspace), wbytes, _stream(q.device)),
        "gdn_prefill_chunked_gated")
    return y


def gdn_mixed_batch(q, k, v, g, beta, cu_seqlens, n_decode, state_pool, initial_state_indices,
                    final_state_indices, scale, decode_in_place=True, chunk=64, l2norm_qk=True,
                    o=None, workspace=None):
    """A serving step's mixed batch: sequences 0 .. n_decode-1 are one-token
    decode rows (rows 0 .. n_decode-1) continuing the states in
    initial_state_indices (in place, or into final_state_indices when
    decode_in_place is False); the rest go through the chunked prefill with
    both index arrays.  Shapes as gdn_prefill_chunked; workspace as there,
    sized for the prefill sequences."""
    _cuda(q, k, v, g, beta, cu_seqlens, state_pool, initial_state_indices, final_state_indices)
    T, hqk, dk = q.shape
    hv, dv = v.shape[1], v.shape[2]
    qs = _heads_view(q, hqk, dk, "q")
    ks = _heads_view(k, hqk, dk, "k")
    vs = _heads_view(v, hv, dv, "v")
    _need(q.dtype == k.dtype == v.dtype, "q, k, v: one dtype")
    _need(g.dtype == torch.float32 and beta.dtype == torch.float32 and g.is_contiguous()
          and beta.is_contiguous() and g.shape == (T, hv) and beta.shape == (T, hv), "g, beta")
    _need(state_pool.dtype == torch.float32 and state_pool.is_contiguous()
          and state_pool.shape[1:] == (hv, dv, dk), "state_pool: [slots, hv, dv, dk] fp32")
    _i32_vec(cu_seqlens, "cu_seqlens")
    n = cu_seqlens.numel() - 1
    _need(0 <= n_decode <= n and n_decode <= T, "n_decode: 0 .. n_seqs")
    for name, t in (("initial_state_indices", initial_state_indices),
                    ("final_state_indices", final_state_indices)):
        if t is not None:
            _i32_vec(t, name)
            _need(t.numel() == n, f"{name}: [n_seqs]")
    o = torch.empty((T, hv, dv), dtype=q.dtype, device=q.device) if o is None else o
    _need(o.is_contiguous() and o.shape == (T, hv, dv), "o: [T, hv, dv] contiguous")
    dt = _dtype_code(q)
    if workspace is False:
        workspace = None
    elif workspace is None:
        need = gdn_prefill_workspace_size(n - n_decode, T, hv, dk, dv, chunk, dt) if n > n_decode else 0
        # + 512 bytes: room for the work counter of the decode beside the prefill
        workspace = torch.empty(need + 512, dtype=torch.uint8, device=q.device) if need else None
    else:
        _cuda(workspace)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.gdn_mixed_batch(_ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(g), _ptr(beta),
                                _ptr(cu_seqlens), n, int(n_decode), T, hqk, hv, dk, dv,
                                float(scale), int(l2norm_qk), chunk, _ptr(state_pool),
                                state_pool.shape[0], _ptr(initial_state_indices),
                                _ptr(final_state_indices), int(bool(decode_in_place)), _ptr(o),
                                dt, _ptr(workspace), wbytes, _stream(q.device)),
           "gdn_mixed_batch")
    return o


def gdn_prefill_chunked_static(q, k, v, g, beta, cu_seqlens, state_pool, initial_state_indices,
                               final_state_indices, scale, l2norm_qk=True, o=None):
    """gdn_prefill_chunked for bf16, dk = dv = 128, chunk 64, with the
    library's fixed device scratch instead of a workspace: no allocation in
    the library (o is allocated here unless given).  Raises GdnError
    (GDN_ERR_TOO_LARGE) past PREFILL_STATIC_SCRATCH_BYTES of scratch."""
    _cuda(q, k, v, g, beta, cu_seqlens, state_pool, initial_state_indices, final_state_indices)
    T, hqk, dk = q.shape
    hv, dv = v.shape[1], v.shape[2]
    _need(q.dtype == k.dtype == v.dtype == torch.bfloat16 and dk == dv == 128,
          "q, k, v: bf16, head dim 128")
    qs = _heads_view(q, hqk, dk, "q")
    ks = _heads_view(k, hqk, dk, "k")
    vs = _heads_view(v, hv, dv, "v")
    _need(g.dtype == torch.float32 and beta.dtype == torch.float32 and g.is_contiguous()
          and beta.is_contiguous() and g.shape == (T, hv) and beta.shape == (T, hv), "g, beta")
    _need(state_pool.dtype == torch.float32 and state_pool.is_contiguous()
          and state_pool.shape[1:] == (hv, dv, dk), "state_pool: [slots, hv, dv, dk] fp32")
    _i32_vec(cu_seqlens, "cu_seqlens")
    n = cu_seqlens.numel() - 1
    for name, t in (("initial_state_indices", initial_state_indices),
                    ("final_state_indices", final_state_indices)):
        if t is not None:
            _i32_vec(t, name)
            _need(t.numel() == n, f"{name}: [n_seqs]")
    o = torch.empty((T, hv, dv), dtype=q.dtype, device=q.device) if o is None else o
    _need(o.is_contiguous() and o.shape == (T, hv, dv), "o: [T, hv, dv] contiguous")
    _check(_lib.gdn_prefill_chunked_static(_ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(g),
                                           _ptr(beta), _ptr(cu_seqlens), n, T, hqk, hv,
                                           float(scale), int(l2norm_qk), _ptr(state_pool),
                                           state_pool.shape[0], _ptr(initial_state_indices),
                                           _ptr(final_state_indices), _ptr(o),
                                           _stream(q.device)),
           "gdn_prefill_chunked_static")
    return o


def gdn_decode_recurrent(q, k, v, g, beta, tokens_per_seq, state_pool, state_indices,
                         snap_indices=None, scale=None, l2norm_qk=True, o=None):
    """Recurrent decode / MTP decode.  q, k [N*tps, hqk, dk]; v [N*tps, hv, dv];
    g, beta [N*tps, hv] fp32; returns o [N*tps, hv, dv]."""
    _cuda(q, k, v, g, beta, state_pool, state_indices, snap_indices)
    T, hqk, dk = q.shape
    hv, dv = v.shape[1], v.shape[2]
    qs = _heads_view(q, hqk, dk, "q")
    ks = _heads_view(k, hqk, dk, "k")
    vs = _heads_view(v, hv, dv, "v")
    _need(q.dtype == k.dtype == v.dtype, "q, k, v: one dtype")
    _i32_vec(state_indices, "state_indices")
    _i32_vec(snap_indices, "snap_indices")
    N = state_indices.numel()
    _need(T == N * tokens_per_seq, "rows != n_seqs * tokens_per_seq")
    _need(g.shape == (T, hv) and beta.shape == (T, hv) and g.dtype == torch.float32
          and beta.dtype == torch.float32 and g.is_contiguous() and beta.is_contiguous(), "g, beta")
    _need(state_pool.dtype == torch.float32 and state_pool.is_contiguous()
          and state_pool.shape[1:] == (hv, dv, dk), "state_pool: [slots, hv, dv, dk] fp32")
    if snap_indices is not None:
        _need(snap_indices.numel() == T, "snap_indices: [n_seqs, tps]")
    scale = dk ** -0.5 if scale is None else scale
    o = torch.empty((T, hv, dv), dtype=q.dtype, device=q.device) if o is None else o
    _check(_lib.gdn_decode_recurrent(_ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(g), _ptr(beta), N,
                                     tokens_per_seq, hqk, hv, dk, dv, float(scale), int(l2norm_qk),
                                     _ptr(state_pool), state_pool.shape[0], _ptr(state_indices),
                                     _ptr(snap_indices), _ptr(o), _dtype_code(q),
                                     _stream(q.device)), "gdn_decode_recurrent")
    return o


def gdn_decode_recurrent_gated(q, k, v, g, beta, tokens_per_seq, state_pool, state_indices, z,
                               norm_weight, norm_eps=1e-6, snap_indices=None, scale=None,
                               l2norm_qk=True, y=None):
    """gdn_decode_recurrent with the gated RMSNorm fused into the output:
    returns y = o / sqrt(mean(o^2) + eps) * norm_weight * SiLU(z), [N*tps, hv, dv].
    z: [N*tps, hv, dv] (a view with a free row stride), norm_weight [dv] fp32."""
    _cuda(q, k, v, g, beta, state_pool, state_indices, snap_indices, z, norm_weight)
    T, hqk, dk = q.shape
    hv, dv = v.shape[1], v.shape[2]
    qs = _heads_view(q, hqk, dk, "q")
    ks = _heads_view(k, hqk, dk, "k")
    vs = _heads_view(v, hv, dv, "v")
    zs = _heads_view(z, hv, dv, "z")
    _need(q.dtype == k.dtype == v.dtype == z.dtype, "q, k, v, z: one dtype")
    _need(norm_weight.dtype == torch.float32 and norm_weight.is_contiguous()
          and norm_weight.shape == (dv,), "norm_weight: [dv] fp32")
    _i32_vec(state_indices, "state_indices")
    _i32_vec(snap_indices, "snap_indices")
    N = state_indices.numel()
    _need(T == N * tokens_per_seq and z.shape[0] == T, "rows != n_seqs * tokens_per_seq")
    _need(g.shape == (T, hv) and beta.shape == (T, hv) and g.dtype == torch.float32
          and beta.dtype == torch.float32 and g.is_contiguous() and beta.is_contiguous(), "g, beta")
    _need(state_pool.dtype == torch.float32 and state_pool.is_contiguous()
          and state_pool.shape[1:] == (hv, dv, dk), "state_pool: [slots, hv, dv, dk] fp32")
    if snap_indices is not None:
        _need(snap_indices.numel() == T, "snap_indices: [n_seqs, tps]")
    scale = dk ** -0.5 if scale is None else scale
    y = torch.empty((T, hv, dv), dtype=q.dtype, device=q.device) if y is None else y
    _need(y.is_contiguous() and y.shape == (T, hv, dv), "y: [T, hv, dv] contiguous")
    _check(_lib.gdn_decode_recurrent_gated(
        _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(g), _ptr(beta), N, tokens_per_seq, hqk, hv,
        dk, dv, float(scale), int(l2norm_qk), _ptr(state_pool), state_pool.shape[0],
        _ptr(state_indices), _ptr(snap_indices), _ptr(z), zs, _ptr(norm_weight),
        float(norm_eps), _ptr(y), _dtype_code(q), _stream(q.device)), "gdn_decode_recurrent_gated")
    return y


def gdn_decode_step_workspace_size(n_seqs, hqk, hv) -> int:
    return int(_lib.gdn_decode_step_workspace_size(n_seqs, hqk, hv))


def gdn_decode_step_fused(x, conv_weight, conv_state_pool, a, b, A_log, dt_bias, hqk,
                          state_pool, state_indices, scale=None, conv_bias=None, o=None,
                          workspace=None):
    """One decode step: conv update + SiLU of the raw q|k|v stream x [N, C],
    gating from a, b [N, hv], L2 norms and the recurrent update.  Same result
    as causal_conv1d_update + gdn_gating + gdn_decode_recurrent.  bf16,
    dk = dv = 128; both pools use state_indices.  Returns o [N, hv, 128].

    workspace: None allocates the scratch gdn_decode_step_workspace_size asks
    for (the step then runs as the conv / gates kernel and the streaming
    decode behind it); a uint8 CUDA tensor is used as given; False passes
    none, which selects the single fused kernel."""
    _cuda(x, conv_weight, conv_state_pool, a, b, A_log, dt_bias, state_pool, state_indices,
          conv_bias)
    N, C = x.shape
    hv = a.shape[1]
    _need(x.dtype == torch.bfloat16 and x.stride(1) == 1, "x: bf16 rows")
    _need(C == 2 * hqk * 128 + hv * 128, "x: 2*hqk*128 + hv*128 channels")
    _need(conv_weight.shape == (C, 4) and conv_weight.is_contiguous()
          and conv_weight.dtype == torch.bfloat16, "conv_weight: [C, 4] bf16")
    _need(conv_state_pool.dtype == torch.bfloat16 and conv_state_pool.is_contiguous()
          and conv_state_pool.shape[1:] == (3, C), "conv_state_pool: [slots, 3, C] bf16")
    _need(a.shape == (N, hv) and b.shape == (N, hv) and a.is_contiguous() and b.is_contiguous()
          and a.dtype == b.dtype == torch.bfloat16, "a, b: [N, hv] bf16")
    _need(state_pool.dtype == torch.float32 and state_pool.is_contiguous()
          and state_pool.shape[1:] == (hv, 128, 128), "state_pool: [slots, hv, 128, 128] fp32")
    _need(conv_state_pool.shape[0] == state_pool.shape[0], "pools: same slot count")
    _i32_vec(state_indices, "state_indices")
    _need(state_indices.numel() == N, "state_indices: [N]")
    scale = 128 ** -0.5 if scale is None else scale
    o = torch.empty((N, hv, 128), dtype=torch.bfloat16, device=x.device) if o is None else o
    _need(o.is_contiguous() and o.shape == (N, hv, 128), "o: [N, hv, 128] contiguous")
    if workspace is False:
        workspace = None
    elif workspace is None:
        need = gdn_decode_step_workspace_size(N, hqk, hv)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    else:
        _cuda(workspace)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.gdn_decode_step_fused(
        _ptr(x), x.stride(0), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_state_pool), _ptr(a),
        _ptr(b), _ptr(A_log), _ptr(dt_bias), N, hqk, hv, float(scale), _ptr(state_pool),
        state_pool.shape[0], _ptr(state_indices), _ptr(workspace), wbytes, _ptr(o),
        _stream(x.device)), "gdn_decode_step_fused")
    return o


def gdn_prefill_layer_workspace_size(n_seqs, n_tokens, hqk, hv) -> int:
    return int(_lib.gdn_prefill_layer_workspace_size(n_seqs, n_tokens, hqk, hv))


def _layer_args(x, conv_weight, conv_state_pool, conv_state_indices, has_initial_state, a, b,
                A_log, dt_bias, cu_seqlens, hqk, state_pool, initial_state_indices,
                final_state_indices, conv_bias, out, workspace):
    """Checks and marshalling shared by the two layer calls: the leading
    arguments up to the index arrays, the output tensor and the workspace."""
    _cuda(x, conv_weight, conv_state_pool, conv_state_indices, a, b, A_log, dt_bias, cu_seqlens,
          state_pool, initial_state_indices, final_state_indices, conv_bias, has_initial_state)
    T, C = x.shape
    hv = a.shape[1]
    _need(x.dtype == torch.bfloat16 and x.stride(1) == 1, "x: bf16 rows")
    _need(C == 2 * hqk * 128 + hv * 128, "x: 2*hqk*128 + hv*128 channels")
    _need(conv_weight.shape == (C, 4) and conv_weight.is_contiguous()
          and conv_weight.dtype == torch.bfloat16, "conv_weight: [C, 4] bf16")
    _need(conv_state_pool.dtype == torch.bfloat16 and conv_state_pool.is_contiguous()
          and conv_state_pool.shape[1:] == (3, C), "conv_state_pool: [slots, 3, C] bf16")
    _need(a.shape == (T, hv) and b.shape == (T, hv) and a.is_contiguous() and b.is_contiguous()
          and a.dtype == b.dtype == torch.bfloat16, "a, b: [T, hv] bf16")
    _need(state_pool.dtype == torch.float32 and state_pool.is_contiguous()
          and state_pool.shape[1:] == (hv, 128, 128), "state_pool: [slots, hv, 128, 128] fp32")
    _i32_vec(cu_seqlens, "cu_seqlens")
    n = cu_seqlens.numel() - 1
    for name, t in (("conv_state_indices", conv_state_indices),
                    ("initial_state_indices", initial_state_indices),
                    ("final_state_indices", final_state_indices)):
        if t is not None:
            _i32_vec(t, name)
            _need(t.numel() == n, f"{name}: [n_seqs]")
    if has_initial_state is not None:
        _need(has_initial_state.dtype == torch.uint8 and has_initial_state.numel() == n,
              "has_initial_state: [n_seqs] uint8")
    out = torch.empty((T, hv, 128), dtype=torch.bfloat16, device=x.device) if out is None else out
    _need(out.is_contiguous() and out.shape == (T, hv, 128), "output: [T, hv, 128] contiguous")
    if workspace is None:
        need = gdn_prefill_layer_workspace_size(n, T, hqk, hv)
        workspace = torch.empty(need + 1024, dtype=torch.uint8, device=x.device) if need else None
        if workspace is not None:   # 1 KiB alignment
            off = (-workspace.data_ptr()) % 1024
            workspace = workspace[off:off + need]
    else:
        _cuda(workspace)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    lead = (_ptr(x), x.stride(0), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_state_pool),
            conv_state_pool.shape[0], _ptr(conv_state_indices), _ptr(has_initial_state), _ptr(a),
            _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(cu_seqlens), n, T, hqk, hv)
    tail = (_ptr(state_pool), state_pool.shape[0], _ptr(initial_state_indices),
            _ptr(final_state_indices))
    return lead, tail, out, (_ptr(workspace), wbytes, _stream(x.device))


def gdn_prefill_layer(x, conv_weight, conv_state_pool, conv_state_indices, has_initial_state, a, b,
                      A_log, dt_bias, cu_seqlens, hqk, state_pool, initial_state_indices,
                      final_state_indices, scale=None, conv_bias=None, o=None, workspace=None):
    """The prefill side of the layer in one call: the causal conv + SiLU of the
    raw q|k|v stream x [T, C] (conv states as causal_conv1d_fwd), then the
    chunked prefill on its q, k, v with the gates formed from the raw a, b
    [T, hv] inside the prefill.  bf16, dk = dv = 128, chunk 64.  Returns o
    [T, hv, 128].  workspace: None allocates gdn_prefill_layer_workspace_size
    bytes; a uint8 CUDA tensor is used as given."""
    lead, tail, o, ws = _layer_args(x, conv_weight, conv_state_pool, conv_state_indices,
                                    has_initial_state, a, b, A_log, dt_bias, cu_seqlens, hqk,
                                    state_pool, initial_state_indices, final_state_indices,
                                    conv_bias, o, workspace)
    scale = 128 ** -0.5 if scale is None else scale
    _check(_lib.gdn_prefill_layer(*lead, float(scale), *tail, _ptr(o), *ws), "gdn_prefill_layer")
    return o


def gdn_prefill_layer_gated(x, conv_weight, conv_state_pool, conv_state_indices, has_initial_state,
                            a, b, A_log, dt_bias, cu_seqlens, hqk, state_pool,
                            initial_state_indices, final_state_indices, z, norm_weight,
                            norm_eps=1e-6, scale=None, conv_bias=None, y=None, workspace=None):
    """gdn_prefill_layer writing the gated RMSNorm y = o / rms(o) * w *
    SiLU(z) per (token, V head) row instead of o; z [T, hv, 128] or
    [T, hv*128] bf16 (row stride free), norm_weight [128] fp32.  Returns y
    [T, hv, 128]."""
    _cuda(z, norm_weight)
    zs = _heads_view(z, a.shape[1], 128, "z")
    _need(z.dtype == torch.bfloat16 and z.shape[0] == x.shape[0], "z: [T, hv, 128] bf16")
    _need(norm_weight.dtype == torch.float32 and norm_weight.is_contiguous()
          and norm_weight.numel() == 128, "norm_weight: [128] fp32")
    lead, tail, y, ws = _layer_args(x, conv_weight, conv_state_pool, conv_state_indices,
                                    has_initial_state, a, b, A_log, dt_bias, cu_seqlens, hqk,
                                    state_pool, initial_state_indices, final_state_indices,
                                    conv_bias, y, workspace)
    scale = 128 ** -0.5 if scale is None else scale
    _check(_lib.gdn_prefill_layer_gated(*lead, float(scale), *tail, _ptr(z), zs,
                                        _ptr(norm_weight), float(norm_eps), _ptr(y), *ws),
           "gdn_prefill_layer_gated")
    return y


def gdn_mtp_step_fused(x, tokens_per_seq, conv_weight, conv_state_pool, a, b, A_log, dt_bias,
                       hqk, state_pool, state_indices, snap_indices, scale=None, conv_bias=None,
                       o=None):
    """One MTP draft step in one kernel: conv update + SiLU of the raw q|k|v
    stream x [N * tps, C] (row i * tps + t), gating from a, b [N * tps, hv],
    L2 norms and the recurrent update over the tps tokens, with the conv and
    recurrent states after token t written to slot snap_indices[i][t] of
    both pools (the source slots are only read).  Returns o [N * tps, hv, 128]."""
    _cuda(x, conv_weight, conv_state_pool, a, b, A_log, dt_bias, state_pool, state_indices,
          snap_indices, conv_bias)
    T, C = x.shape
    hv = a.shape[1]
    _i32_vec(state_indices, "state_indices")
    _i32_vec(snap_indices, "snap_indices")
    N = state_indices.numel()
    _need(T == N * tokens_per_seq, "x rows != n_seqs * tokens_per_seq")
    _need(snap_indices.numel() == T, "snap_indices: [n_seqs, tps]")
    _need(x.dtype == torch.bfloat16 and x.stride(1) == 1, "x: bf16 rows")
    _need(C == 2 * hqk * 128 + hv * 128, "x: 2*hqk*128 + hv*128 channels")
    _need(conv_weight.shape == (C, 4) and conv_weight.is_contiguous()
          and conv_weight.dtype == torch.bfloat16, "conv_weight: [C, 4] bf16")
    _need(conv_state_pool.dtype == torch.bfloat16 and conv_state_pool.is_contiguous()
          and conv_state_pool.shape[1:] == (3, C), "conv_state_pool: [slots, 3, C] bf16")
    _need(a.shape == (T, hv) and b.shape == (T, hv) and a.is_contiguous() and b.is_contiguous()
          and a.dtype == b.dtype == torch.bfloat16, "a, b: [N*tps, hv] bf16")
    _need(state_pool.dtype == torch.float32 and state_pool.is_contiguous()
          and state_pool.shape[1:] == (hv, 128, 128), "state_pool: [slots, hv, 128, 128] fp32")
    _need(conv_state_pool.shape[0] == state_pool.shape[0], "pools: same slot count")
    scale = 128 ** -0.5 if scale is None else scale
    o = torch.empty((T, hv, 128), dtype=torch.bfloat16, device=x.device) if o is None else o
    _need(o.is_contiguous() and o.shape == (T, hv, 128), "o: [N*tps, hv, 128] contiguous")
    _check(_lib.gdn_mtp_step_fused(
        _ptr(x), x.stride(0), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_state_pool), _ptr(a),
        _ptr(b), _ptr(A_log), _ptr(dt_bias), N, tokens_per_seq, hqk, hv, float(scale),
        _ptr(state_pool), state_pool.shape[0], _ptr(state_indices), _ptr(snap_indices), _ptr(o),
        _stream(x.device)), "gdn_mtp_step_fused")
    return o


def gdn_gated_rmsnorm(o, z, weight, eps=1e-6, y=None):
    """y = o / sqrt(mean(o^2) + eps) * weight * SiLU(z) per (token, head) row.
    o [T, hv, dv] contiguous; z [T, hv, dv] (a view with a free row stride);
    weight [dv] fp32.  y defaults to a new tensor; pass y=o for in place."""
    _cuda(o, z, weight)
    T, hv, dv = o.shape
    _need(o.is_contiguous(), "o: contiguous")
    zs = _heads_view(z, hv, dv, "z")
    _need(z.shape == o.shape and z.dtype == o.dtype, "z: same shape and dtype as o")
    _need(weight.dtype == torch.float32 and weight.is_contiguous() and weight.shape == (dv,),
          "weight: [dv] fp32")
    y = torch.empty_like(o) if y is None else y
    _need(y.is_contiguous() and y.shape == o.shape and y.dtype == o.dtype, "y: like o")
    _check(_lib.gdn_gated_rmsnorm(_ptr(o), _ptr(z), zs, _ptr(weight), T, hv, dv, float(eps),
                                  _ptr(y), _dtype_code(o), _stream(o.device)), "gdn_gated_rmsnorm")
    return y


# The bindings below are on a decode step's critical path (a few microseconds a
# call), so their checks are written out and messages formed only on failure.
_F32, _BF16, _E4M3, _I32 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int32
_CODES = {_F32: GDN_F32, _BF16: GDN_BF16, _E4M3: GDN_E4M3}
# torch's own short forms of its public calls, where it has them (torch.cuda.current_stream
# makes a stream object, a microsecond a call).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _one_device(first, *ts):
    """Every tensor on the CUDA device of the first one; returns its index."""
    dev = first.get_device()
    if dev < 0:
        raise GdnError("all tensors must be on one CUDA device")
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise GdnError("all tensors must be on one CUDA device")
    return dev


def _call(fn, name, dev, *args):
    """fn on the current stream of device `dev`, which is made the current device for the call."""
    if dev == _current_device():
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        _check(status, name)


def _rows(t, shape, name):
    """t has the 2-D shape and unit column stride; returns its row stride (at least a row where there is one)."""
    if t.shape != shape:
        raise GdnError(f"{name}: shape {tuple(t.shape)}, not {list(shape)}")
    if t.is_contiguous():
        return shape[1]
    st, one = t.stride()
    if one != 1 and shape[1] != 1:
        raise GdnError(f"{name}: unit column stride")
    if st < shape[1]:
        if shape[0] > 1:
            raise GdnError(f"{name}: rows must not overlap")
        return shape[1]
    return st


def _f32_vec(t, n, name):
    if t.dtype is not _F32 or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise GdnError(f"{name}: [{n}] fp32, contiguous")
    return t.data_ptr()


def gdn_add_rmsnorm(x, weight, residual=None, eps=1e-6, weight_offset=0.0, y_dtype=None,
                    residual_out=None, y=None, y_scale=None):
    """s = x + residual; y = s / sqrt(mean(s^2) + eps) * (weight_offset + weight)
    per token row.  x, residual [T, H] (views with a free row stride), fp32 or
    bf16; weight [H] fp32.  y_dtype: x's dtype (default) or
    torch.float8_e4m3fn, then with one fp32 scale per token, y * y_scale[:, None]
    being the norm.  Returns (y, y_scale or None, residual_out or None), where
    residual_out [T, H] is s in x's dtype, made when a residual is given (pass
    residual_out=residual to update the stream in place)."""
    dev = _one_device(x, weight, residual, residual_out, y, y_scale)
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2:
        raise GdnError("x: [T, H]")
    if dtype != _BF16 and dtype != _F32:
        raise GdnError(f"unsupported activation dtype {dtype} (fp32 or bf16)")
    T, H = shape
    xs, dt = _rows(x, shape, "x"), _CODES[dtype]
    rs, rp, ros, rop, sp = 0, None, 0, None, None
    if residual is not None:
        if residual.dtype != dtype:
            raise GdnError("residual: x's dtype")
        rs, rp = _rows(residual, shape, "residual"), residual.data_ptr()
        if residual_out is None:
            residual_out = torch.empty((T, H), dtype=dtype, device=x.device)
    if residual_out is not None:
        if residual_out.dtype != dtype:
            raise GdnError("residual_out: x's dtype")
        ros, rop = _rows(residual_out, shape, "residual_out"), residual_out.data_ptr()
    if y is None:
        y = torch.empty((T, H), dtype=dtype if y_dtype is None else y_dtype, device=x.device)
    elif y_dtype is not None and y.dtype != y_dtype:
        raise GdnError("y: y_dtype")
    quant = y.dtype == _E4M3
    if quant:
        if y_scale is None:
            y_scale = torch.empty(T, dtype=_F32, device=x.device)
        sp = _f32_vec(y_scale, T, "y_scale")
    elif y.dtype != dtype:
        raise GdnError("y: x's dtype or float8_e4m3fn")
    elif y_scale is not None:
        raise GdnError("y_scale: only with an 8-bit y")
    _call(_lib.gdn_add_rmsnorm, "gdn_add_rmsnorm", dev, x.data_ptr(), xs, rp, rs,
          _f32_vec(weight, H, "weight"), weight_offset, T, H, eps, rop, ros, y.data_ptr(),
          _rows(y, shape, "y"), sp, dt, GDN_E4M3 if quant else dt)
    return y, y_scale, residual_out


def gdn_gated_rmsnorm_quant(o, z, weight, eps=1e-6, y=None, y_scale=None):
    """gdn_gated_rmsnorm with an 8-bit output: returns y [T, hv, dv]
    float8_e4m3fn and y_scale [T] fp32 (one scale per token), y * y_scale being
    the gated norm.  o [T, hv, dv] contiguous; z [T, hv, dv] or [T, hv*dv] (a
    view with a free row stride); weight [dv] fp32.  y viewed as [T, hv*dv] is
    gdn_linear's 8-bit x."""
    dev = _one_device(o, z, weight, y, y_scale)
    shape, dtype = o.shape, o.dtype
    if len(shape) != 3 or not o.is_contiguous():
        raise GdnError("o: [T, hv, dv] contiguous")
    if dtype != _BF16 and dtype != _F32:
        raise GdnError(f"unsupported activation dtype {dtype} (fp32 or bf16)")
    T, hv, dv = shape
    if z.dtype != dtype:
        raise GdnError("z: o's dtype")
    if z.shape == shape:
        zs, head, one = z.stride()
        if one != 1 or (head != dv and hv != 1):
            raise GdnError("z: heads must be packed")
        if zs < hv * dv:
            if T > 1:
                raise GdnError("z: rows must not overlap")
            zs = hv * dv
    else:
        zs = _rows(z, (T, hv * dv), "z")
    if y is None:
        y = torch.empty((T, hv, dv), dtype=_E4M3, device=o.device)
    elif y.dtype != _E4M3 or y.shape != shape or not y.is_contiguous():
        raise GdnError("y: [T, hv, dv] float8_e4m3fn, contiguous")
    if y_scale is None:
        y_scale = torch.empty(T, dtype=_F32, device=o.device)
    _call(_lib.gdn_gated_rmsnorm_quant, "gdn_gated_rmsnorm_quant", dev, o.data_ptr(), z.data_ptr(),
          zs, _f32_vec(weight, dv, "weight"), T, hv, dv, eps, y.data_ptr(),
          _f32_vec(y_scale, T, "y_scale"), _CODES[dtype])
    return y, y_scale


def gdn_linear(x, weight, x_scale=None, weight_scale=None, bias=None, act="none", residual=None,
               y_dtype=None, y=None):
    """y = act(x_scale weight_scale (x @ weight.T) + bias) + residual.
    x [T, K], weight [N, K]: both bf16, or both float8_e4m3fn with x_scale [T]
    and weight_scale [N] fp32 (None = 1); unit column stride, rows on 16-byte
    boundaries (K itself may be odd).  bias [N] fp32; act "none", "silu" or
    "gelu"; residual [T, N] in y's dtype.  y [T, N] bf16 (default) or fp32,
    columns of a wider buffer if wanted; y may be residual.  Returns y."""
    dev = _one_device(x, weight, x_scale, weight_scale, bias, residual, y)
    shape, wshape, dtype = x.shape, weight.shape, x.dtype
    if len(shape) != 2 or len(wshape) != 2:
        raise GdnError("x: [T, K], weight: [N, K]")
    T, K = shape
    N = wshape[0]
    if dtype != weight.dtype or (dtype != _BF16 and dtype != _E4M3):
        raise GdnError("x, weight: both bf16 or both float8_e4m3fn")
    if wshape[1] != K:
        raise GdnError(f"x {tuple(shape)} and weight {tuple(wshape)} differ in K")
    swp = sxp = bp = rp = None
    rs = 0
    if x_scale is not None or weight_scale is not None:
        if dtype != _E4M3:
            raise GdnError("scales: only with 8-bit x and weight")
        if x_scale is not None:
            sxp = _f32_vec(x_scale, T, "x_scale")
        if weight_scale is not None:
            swp = _f32_vec(weight_scale, N, "weight_scale")
    if bias is not None:
        bp = _f32_vec(bias, N, "bias")
    code = ACTIVATIONS.get(act)
    if code is None:
        raise GdnError(f"act: one of {tuple(ACTIVATIONS)}")
    if y is None:
        y = torch.empty((T, N), dtype=_BF16 if y_dtype is None else y_dtype, device=x.device)
    elif y_dtype is not None and y.dtype != y_dtype:
        raise GdnError("y: y_dtype")
    ydt = y.dtype
    if ydt != _BF16 and ydt != _F32:
        raise GdnError("y: bf16 or fp32")
    if residual is not None:
        if residual.dtype != ydt:
            raise GdnError("residual: y's dtype")
        rs, rp = _rows(residual, (T, N), "residual"), residual.data_ptr()
    _call(_lib.gdn_linear, "gdn_linear", dev, x.data_ptr(), _rows(x, shape, "x"), sxp,
          weight.data_ptr(), _rows(weight, wshape, "weight"), swp, bp, rp, rs, T, K, N, code,
          y.data_ptr(), _rows(y, (T, N), "y"), _CODES[dtype], _CODES[ydt])
    return y


def _vec(t, dtype, shape, name):
    """t is contiguous with this type and shape; returns its address."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise GdnError(f"{name}: {list(shape)} {dtype}, contiguous")
    return t.data_ptr()


def _out(y, y_dtype, shape, device):
    """The products' output: y as given, or a new one; its code and row stride."""
    if y is None and (y_dtype is None or y_dtype in (_BF16, _F32)):
        y_dtype = y_dtype or _BF16
        return torch.empty(shape, dtype=y_dtype, device=device), _CODES[y_dtype], shape[1]
    if y is None:
        raise GdnError("y: bf16 or fp32")
    if y_dtype is not None and y.dtype != y_dtype:
        raise GdnError("y: y_dtype")
    if y.dtype != _BF16 and y.dtype != _F32:
        raise GdnError("y: bf16 or fp32")
    return y, _CODES[y.dtype], _rows(y, shape, "y")


def gdn_linear_block(x, weight, x_scale, weight_scale, y_dtype=None, y=None):
    """y = x @ weight.T for float8_e4m3fn x [T, K] and weight [N, K] with one fp32
    scale for each block of 128 in K: x_scale [T, ceil(K / 128)] (as
    gdn_block_quant gives), weight_scale [ceil(N / 128), ceil(K / 128)].  Unit
    column stride, rows on 16-byte boundaries (K itself may be odd).  y [T, N] bf16
    (default) or fp32, columns of a wider buffer if wanted.  A row's last fp32 bits
    depend on the call's sizes (T among them), not on the other rows.  Returns y."""
    dev = _one_device(x, weight, x_scale, weight_scale, y)
    shape, wshape = x.shape, weight.shape
    if len(shape) != 2 or len(wshape) != 2 or wshape[1] != shape[1]:
        raise GdnError("x: [T, K], weight: [N, K]")
    if x.dtype != _E4M3 or weight.dtype != _E4M3:
        raise GdnError("x, weight: float8_e4m3fn")
    T, K = shape
    N = wshape[0]
    kb = (K + 127) // 128
    y, code, ys = _out(y, y_dtype, (T, N), x.device)
    _call(_lib.gdn_linear_block, "gdn_linear_block", dev, x.data_ptr(), _rows(x, shape, "x"),
          _vec(x_scale, _F32, (T, kb), "x_scale"), weight.data_ptr(), _rows(weight, wshape, "weight"),
          _vec(weight_scale, _F32, ((N + 127) // 128, kb), "weight_scale"), T, K, N, y.data_ptr(), ys, code)
    return y


def gdn_moe_route_workspace_size(n_tokens, n_experts) -> int:
    return int(_lib.gdn_moe_route_workspace_size(n_tokens, n_experts))


def gdn_moe_route(logits, top_k, renormalize=True, ids=None, weights=None, offsets=None, rows=None,
                  slots=None, workspace=None):
    """The top_k experts of each token and the pairs (token, choice) sorted by
    expert.  logits [T, E] fp32 or bf16 (a view with a free row stride).  Returns
    ids [T, top_k] int32 (largest logit first, ties by the lowest index), weights
    [T, top_k] fp32 (their softmax, over all experts or, with renormalize, over
    the chosen), offsets [E + 1], rows [T * top_k] (the token of each sorted row)
    and slots [T, top_k] (the sorted row of each pair), int32.

    workspace: None allocates what gdn_moe_route_workspace_size asks for; a uint8
    CUDA tensor is used as given."""
    dev = _one_device(logits, ids, weights, offsets, rows, slots, workspace)
    shape, dtype, device = logits.shape, logits.dtype, logits.device
    if len(shape) != 2:
        raise GdnError("logits: [T, E]")
    if dtype != _BF16 and dtype != _F32:
        raise GdnError(f"unsupported logits dtype {dtype} (fp32 or bf16)")
    T, E = shape
    if not 0 < top_k <= E:
        raise GdnError("top_k: 1 to E")
    empty, lp, ls = torch.empty, logits.data_ptr(), _rows(logits, shape, "logits")
    # outputs made here need no check
    if ids is None:
        ids = empty((T, top_k), dtype=_I32, device=device)
    else:
        _vec(ids, _I32, (T, top_k), "ids")
    if weights is None:
        weights = empty((T, top_k), dtype=_F32, device=device)
    else:
        _vec(weights, _F32, (T, top_k), "weights")
    if offsets is None:
        offsets = empty(E + 1, dtype=_I32, device=device)
    else:
        _vec(offsets, _I32, (E + 1,), "offsets")
    if rows is None:
        rows = empty(T * top_k, dtype=_I32, device=device)
    else:
        _vec(rows, _I32, (T * top_k,), "rows")
    if slots is None:
        slots = empty((T, top_k), dtype=_I32, device=device)
    else:
        _vec(slots, _I32, (T, top_k), "slots")
    wp = wbytes = None
    if workspace is None:
        need = _lib.gdn_moe_route_workspace_size(T, E)
        if need:
            workspace = empty(need, dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous():
        raise GdnError("workspace: contiguous")
    if workspace is not None:
        wp, wbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call(_lib.gdn_moe_route, "gdn_moe_route", dev, lp, ls, T, E, top_k, 1 if renormalize else 0, ids.data_ptr(),
          weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(), _CODES[dtype], wp, wbytes or 0)
    return ids, weights, offsets, rows, slots


def gdn_block_quant(x, glu=False, y=None, y_scale=None):
    """x, or with glu SiLU(x[:, :n]) * x[:, n:], in 8 bits with one fp32 scale for
    each block of 128 channels.  x [T, n] (glu: [T, 2 n]) fp32 or bf16 (a view with
    a free row stride).  Returns y [T, n] float8_e4m3fn, whose rows start on
    16-byte boundaries (a view of a wider buffer where n is no multiple of 16)
    unless it is given, and y_scale [T, ceil(n / 128)]: the x and x_scale of
    gdn_linear_block and gdn_grouped_linear.  A quotient within fp32's roundings (and,
    with glu, the fast SiLU's) of the middle between two e4m3 values may go to either."""
    dev = _one_device(x, y, y_scale)
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2 or (glu and shape[1] % 2):
        raise GdnError("x: [T, n], with glu [T, 2 n]")
    if dtype != _BF16 and dtype != _F32:
        raise GdnError(f"unsupported activation dtype {dtype} (fp32 or bf16)")
    T, n = shape[0], shape[1] // 2 if glu else shape[1]
    if y is None:
        ys = (n + 15) // 16 * 16
        y = torch.empty_strided((T, n), (ys, 1), dtype=_E4M3, device=x.device)
    elif y.dtype != _E4M3:
        raise GdnError("y: float8_e4m3fn")
    else:
        ys = _rows(y, (T, n), "y")
    if y_scale is None:
        y_scale = torch.empty((T, (n + 127) // 128), dtype=_F32, device=x.device)
    else:
        _vec(y_scale, _F32, (T, (n + 127) // 128), "y_scale")
    _call(_lib.gdn_block_quant, "gdn_block_quant", dev, x.data_ptr(), _rows(x, shape, "x"), T, n, 1 if glu else 0,
          y.data_ptr(), ys, y_scale.data_ptr(), _CODES[dtype])
    return y, y_scale


def gdn_grouped_linear(x, weight, offsets, rows=None, x_scale=None, weight_scale=None, y_dtype=None, y=None):
    """y[r] = weight[e] @ x[rows[r]] for offsets[e] <= r < offsets[e + 1] (rows
    None: x[r]), with offsets [E + 1] and rows [R] int32 as gdn_moe_route gives.
    x [n_x, K], weight [E, N, K]: both bf16, or both float8_e4m3fn with x_scale
    [n_x, ceil(K / 128)] and weight_scale [E, ceil(N / 128), ceil(K / 128)] fp32;
    unit column stride, rows (and experts) on 16-byte boundaries (K itself may be
    odd).  y [R, N] bf16 (default) or fp32; rows from offsets[E] on are left as
    they were, so a y that is not given holds anything there.  A row's last fp32 bits
    depend on the call's sizes, not on the other rows.  Returns y."""
    dev = _one_device(x, weight, offsets, rows, x_scale, weight_scale, y)
    shape, wshape, dtype = x.shape, weight.shape, x.dtype
    if len(shape) != 2 or len(wshape) != 3 or wshape[2] != shape[1]:
        raise GdnError("x: [n_x, K], weight: [E, N, K]")
    if dtype != weight.dtype or (dtype != _BF16 and dtype != _E4M3):
        raise GdnError("x, weight: both bf16 or both float8_e4m3fn")
    n_x, K = shape
    E, N, _ = wshape
    R, rp, sxp, swp = n_x, None, None, None
    if rows is not None:
        R = rows.numel()
        rp = _vec(rows, _I32, (R,), "rows")
    if dtype == _E4M3:
        if x_scale is None or weight_scale is None:
            raise GdnError("x_scale, weight_scale: needed with 8-bit x and weight")
        kb = (K + 127) // 128
        sxp = _vec(x_scale, _F32, (n_x, kb), "x_scale")
        swp = _vec(weight_scale, _F32, (E, (N + 127) // 128, kb), "weight_scale")
    elif x_scale is not None or weight_scale is not None:
        raise GdnError("scales: only with 8-bit x and weight")
    we, ws, one = weight.stride()
    if (one != 1 and K != 1) or (ws < K and N > 1):
        raise GdnError("weight: unit column stride, rows that do not overlap")
    ws = max(ws, K) if N > 1 else K
    if E == 1:
        we = N * ws
    y, code, ys = _out(y, y_dtype, (R, N), x.device)
    _call(_lib.gdn_grouped_linear, "gdn_grouped_linear", dev, x.data_ptr(), _rows(x, shape, "x"), sxp, n_x, rp,
          weight.data_ptr(), ws, we, swp, _vec(offsets, _I32, (E + 1,), "offsets"), E, R, K, N, y.data_ptr(), ys,
          _CODES[dtype], code)
    return y


def gdn_moe_combine(x, slots, weights, residual=None, y=None):
    """y[t] = residual[t] + sum_j weights[t, j] x[slots[t, j]], summed in fp32.
    x [R, H] fp32 or bf16, slots [T, k] int32 (< 0: left out), weights [T, k]
    fp32, residual [T, H] in x's dtype; free row strides.  y [T, H] may be
    residual.  Returns y."""
    dev = _one_device(x, slots, weights, residual, y)
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2 or slots.dim() != 2:
        raise GdnError("x: [R, H], slots: [T, k]")
    if dtype != _BF16 and dtype != _F32:
        raise GdnError(f"unsupported activation dtype {dtype} (fp32 or bf16)")
    T, k = slots.shape
    R, H = shape
    rs, rp = 0, None
    if residual is not None:
        if residual.dtype != dtype:
            raise GdnError("residual: x's dtype")
        rs, rp = _rows(residual, (T, H), "residual"), residual.data_ptr()
    if y is None:
        y, ys = torch.empty((T, H), dtype=dtype, device=x.device), H
    elif y.dtype != dtype:
        raise GdnError("y: x's dtype")
    else:
        ys = _rows(y, (T, H), "y")
    _call(_lib.gdn_moe_combine, "gdn_moe_combine", dev, x.data_ptr(), _rows(x, shape, "x"), R,
          _vec(slots, _I32, (T, k), "slots"), _vec(weights, _F32, (T, k), "weights"), rp, rs, T, k, H,
          y.data_ptr(), ys, _CODES[dtype])
    return y


def gdn_state_snapshot(pool, src, dst):
    """pool[dst[i]] <- pool[src[i]] for whole slots (any pool dtype)."""
    _cuda(pool, src, dst)
    _i32_vec(src, "src")
    _i32_vec(dst, "dst")
    _need(src.numel() == dst.numel(), "src/dst length")
    _need(pool.is_contiguous(), "pool must be contiguous")
    slot_bytes = pool[0].numel() * pool.element_size()
    _check(_lib.gdn_state_snapshot(_ptr(pool), pool.shape[0], slot_bytes, _ptr(src), _ptr(dst),
                                   src.numel(), _stream(pool.device)), "gdn_state_snapshot")


def gdn_get_device_status(clear=True, device=None) -> int:
    """Device status word (DEVSTAT_* bits); synchronises the current stream."""
    out = ctypes.c_uint32(0)
    _check(_lib.gdn_get_device_status(ctypes.byref(out), int(clear), _stream(device)),
           "gdn_get_device_status")
    return int(out.value)


def gdn_debug_set_wait_limit(limit_ns=0, drop_prep_loads=False, device=None, drop_linear_loads=0):
    """Test control of the failure path of the two-kernel prefill and of the
    products (gdn_linear, gdn_linear_block, gdn_grouped_linear): the limit of their
    bounded waits (0 = the default, one second), whether the prep kernel skips its
    K|Q loads, and which loads the products skip (0 none, 1 all, 2 those behind a
    CTA's first block or tile).  Its waits then run out and the call sets
    DEVSTAT_TIMEOUT; its results are undefined.
    Synchronises the stream."""
    _need(drop_linear_loads in (0, 1, 2), "drop_linear_loads: 0, 1 or 2")
    _check(_lib.gdn_debug_set_wait_limit(int(limit_ns), int(bool(drop_prep_loads)) + 2 * drop_linear_loads,
                                         _stream(device)), "gdn_debug_set_wait_limit")


def gdn_debug_set_grouped_tile(rows=0, cut=-1):
    """Test control of the products with block scales and of the grouped ones: tiles
    of 16, 32, 64, 128 or 256 rows in place of the choice by the sizes (0), with the
    sum over k in 2^cut parts (-1: by the sizes)."""
    _check(_lib.gdn_debug_set_grouped_tile(rows, cut), "gdn_debug_set_grouped_tile")
