"""Elastic Attention hybrid-head attention on GB300 (sm_103a).

Thin Python binding over the C ABI declared in ``include/ea.h``; the names match
the C entry points.  This module only marshals arguments (pointers, strides,
streams) from torch tensors: every step of the computation runs in the CUDA
library ``_lib/libea.so``.  If that library is missing, or no CUDA device is
present, the device entry points raise instead of computing anything else.

    ea_route                 router pre-pass (pool -> MLP -> argmax -> mode)
    ea_route_layers          the router pre-pass of many model layers in one launch
    ea_hybrid_attn_prefill   fused FA / SSA / block-sparse prefill, one launch
    ea_hybrid_attn_prefill_host  the prefill on host tensors, copies overlapped
    ea_hybrid_attn_prefill_varlen  sequences of different lengths in one launch
    ea_hybrid_attn_decode    split-KV decode with the prefill-time routing
    ea_hybrid_attn_decode_paged  the same decode over a paged KV cache
    ea_cache_write           new tokens into a KV cache of 8 bits (or bf16), quantised
    ea_hybrid_attn_decode_q8 the decode over an 8-bit cache, with the keys' attention weights
    ea_key_weights           the attention weight that a prefill's queries give its keys
    ea_evict_select          which tokens stay when a cache is cut by those weights
    ea_cache_compact         gathers them into another cache
    ea_rope                  queries and keys rotated by their positions
    ea_cache_write_rope      new tokens into a KV cache, rotated on the way
    ea_tree_plan             depths and ancestors of a tree of drafted tokens
    ea_hybrid_attn_tree      the tree's attention over a cache and over itself
    ea_tree_accept           the path of the tree that the model agrees with
    ea_sparsity_ratios       Omega_MSR / Omega_ESR (host)
    ea_check_errors          read back the device error word of a workspace
"""
import ctypes
import functools
import math
import os

import torch

FULL, SSA, BLOCK = 0, 1, 2
TILE = 128
EA_OK = 0
_STATUS = {0: "EA_OK", 1: "EA_ERR_INVALID_ARG", 2: "EA_ERR_UNSUPPORTED", 3: "EA_ERR_WORKSPACE",
           4: "EA_ERR_CUDA", 5: "EA_ERR_TIMEOUT", 6: "EA_ERR_DEVICE_CHECK"}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libea.so")
_lib = None

# Function names exported by the library (the ones include/ea.h declares).
EXPORTS = ("ea_status_string", "ea_route", "ea_route_layers", "ea_prefill_workspace_size", "ea_hybrid_attn_prefill",
           "ea_prefill_plan", "ea_prefill_attend", "ea_hybrid_attn_prefill_noalloc",
           "ea_prefill_host_buffer_size", "ea_hybrid_attn_prefill_host",
           "ea_prefill_varlen_workspace_size", "ea_hybrid_attn_prefill_varlen",
           "ea_prefill_layers_workspace_size", "ea_hybrid_attn_prefill_layers",
           "ea_decode_workspace_size",
           "ea_hybrid_attn_decode", "ea_hybrid_attn_decode_paged", "ea_xa_workspace_size",
           "ea_xa_estimate", "ea_cache_workspace_size", "ea_cache_write", "ea_evict_select",
           "ea_cache_compact", "ea_decode_q8_workspace_size", "ea_hybrid_attn_decode_q8",
           "ea_key_weights_workspace_size", "ea_key_weights", "ea_rope", "ea_cache_write_rope",
           "ea_tree_plan", "ea_tree_workspace_size", "ea_hybrid_attn_tree", "ea_tree_accept", "ea_sparsity_ratios",
           "ea_check_errors")


class EAError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s failed: %s" % (fn, _STATUS.get(status, status)))


class _Mlp(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("dims", ctypes.POINTER(ctypes.c_int)),
                ("W", ctypes.POINTER(ctypes.c_void_p)), ("b", ctypes.POINTER(ctypes.c_void_p))]


class _PrefillLayer(ctypes.Structure):
    _fields_ = [("Q", ctypes.c_void_p), ("K", ctypes.c_void_p), ("V", ctypes.c_void_p),
                ("O", ctypes.c_void_p), ("LSE", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("block_mask", ctypes.c_void_p)]


class _Cache(ctypes.Structure):
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("kv_str", ctypes.c_int64 * 4),
                ("block_table", ctypes.c_void_p), ("bt_stride", ctypes.c_int64),
                ("outer", ctypes.c_int), ("rows", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("d", ctypes.c_int), ("format", ctypes.c_int),
                ("scale_block", ctypes.c_int)]


MAX_PREFILL_LAYERS = 48


class _Policy(ctypes.Structure):
    _fields_ = [("fa_impl", ctypes.c_uint8), ("sa_impl", ctypes.c_uint8)]


def use_library(path):
    """Route every later call through the library at `path` (for example the
    bounds-checked build, _lib/libea_checked.so); returns the previous path."""
    global _lib, LIB_PATH
    prev = LIB_PATH
    LIB_PATH = path
    _lib = None
    return prev


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libea.so is not built; run __graft_entry__.build() or "
                               "python sparse_head_attention_gb300/build.py")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, sz, f32, f64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float,
                                ctypes.c_double)
        L.ea_status_string.argtypes = [i32]
        L.ea_status_string.restype = ctypes.c_char_p
        L.ea_route.argtypes = [P, P, i32, i32, i32, i32, i32, i32, ctypes.POINTER(_Mlp), _Policy,
                               P, P, P, P]
        L.ea_route_layers.argtypes = [P, i32, P, i32, i32, i32, i32, i32, i32, P, _Policy,
                                      P, P, P, P]
        L.ea_prefill_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.ea_prefill_workspace_size.restype = sz
        L.ea_hybrid_attn_prefill.argtypes = [P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, f32,
                                             P, i32, i32, P, i32, P, sz, P, P]
        L.ea_prefill_plan.argtypes = [i32, i32, i32, i32, i32, P, i32, i32, P, i32, P, sz, P]
        L.ea_prefill_attend.argtypes = list(L.ea_hybrid_attn_prefill.argtypes)
        L.ea_hybrid_attn_prefill_noalloc.argtypes = [P, P, P, P, P, P, P, P, i32, i32, i32, i32,
                                                     i32, f32, P, i32, i32, P, i32, P, P]
        L.ea_hybrid_attn_prefill_noalloc.restype = ctypes.c_int
        L.ea_prefill_host_buffer_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.ea_prefill_host_buffer_size.restype = sz
        L.ea_hybrid_attn_prefill_host.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, f32, P,
                                                  i32, i32, P, i32, P, sz, i32, P]
        L.ea_hybrid_attn_prefill_host.restype = ctypes.c_int
        L.ea_prefill_layers_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.ea_prefill_layers_workspace_size.restype = sz
        L.ea_hybrid_attn_prefill_layers.argtypes = [P, i32, P, P, P, i32, i32, i32, i32, i32, f32,
                                                    i32, i32, i32, P, sz, P]
        L.ea_hybrid_attn_prefill_layers.restype = ctypes.c_int
        L.ea_prefill_varlen_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.ea_prefill_varlen_workspace_size.restype = sz
        L.ea_hybrid_attn_prefill_varlen.argtypes = [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32,
                                                    i32, i32, f32, P, i32, i32, P, i32, P, sz, P]
        L.ea_hybrid_attn_prefill_varlen.restype = ctypes.c_int
        L.ea_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.ea_decode_workspace_size.restype = sz
        L.ea_hybrid_attn_decode.argtypes = [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, f32,
                                            P, i32, i32, P, i32, i32, P, sz, P]
        L.ea_hybrid_attn_decode_paged.argtypes = [P, P, P, P, P, P, P, P, P, ctypes.c_int64, i32,
                                                  i32, i32, P, i32, i32, i32, i32, f32, P, i32,
                                                  i32, P, i32, i32, P, sz, P]
        L.ea_hybrid_attn_decode_paged.restype = ctypes.c_int
        L.ea_xa_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        L.ea_xa_workspace_size.restype = sz
        L.ea_xa_estimate.argtypes = [P, P, P, P, i32, i32, i32, i32, i32, f32, P, i32, f32, i32,
                                     i32, P, P, P, sz, P]
        L.ea_xa_estimate.restype = ctypes.c_int
        L.ea_cache_workspace_size.argtypes = []
        L.ea_cache_workspace_size.restype = sz
        L.ea_cache_write.argtypes = [P, P, P, P, P, P, i32, i32, P, sz, P]
        L.ea_evict_select.argtypes = [P, P, i32, i32, i32, i32, i32, i32, P, P, P, sz, P]
        L.ea_cache_compact.argtypes = [P, P, P, P, i32, i32, P, P, P, sz, P]
        L.ea_decode_q8_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        L.ea_decode_q8_workspace_size.restype = sz
        L.ea_hybrid_attn_decode_q8.argtypes = [P, P, P, P, P, P, P, i32, i32, f32, P, i32, i32, P,
                                               i32, i32, P, i32, P, sz, P]
        L.ea_key_weights_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.ea_key_weights_workspace_size.restype = sz
        L.ea_key_weights.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, f32, P, i32,
                                     i32, P, i32, P, i32, P, sz, P]
        L.ea_rope.argtypes = [P, P, P, P, i32, P, P, P, P, i32, i32, i32, i32, P, i32, i32, f32, P, P, P, sz, P]
        L.ea_cache_write_rope.argtypes = [P, P, P, P, P, P, P, P, i32, P, i32, i32, f32, P, P, P, P, i32, i32,
                                          P, sz, P]
        L.ea_tree_plan.argtypes = [P, P, i32, i32, P, P, P, sz, P]
        L.ea_tree_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.ea_tree_workspace_size.restype = sz
        L.ea_hybrid_attn_tree.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, P, i32, i32, i32, f32, P, i32, i32, P,
                                          i32, P, sz, P]
        L.ea_tree_accept.argtypes = [P, P, P, P, i32, i32, P, P, P, P, sz, P]
        L.ea_sparsity_ratios.argtypes = [P, P, i32, i32, i32, i32, i32, P, i32,
                                         ctypes.POINTER(f64), ctypes.POINTER(f64)]
        L.ea_check_errors.argtypes = [P, P]
        for f in ("ea_route", "ea_route_layers", "ea_hybrid_attn_prefill", "ea_prefill_plan", "ea_prefill_attend",
                  "ea_hybrid_attn_decode", "ea_cache_write", "ea_evict_select", "ea_cache_compact",
                  "ea_hybrid_attn_decode_q8", "ea_key_weights", "ea_rope", "ea_cache_write_rope", "ea_tree_plan",
                  "ea_hybrid_attn_tree", "ea_tree_accept", "ea_sparsity_ratios", "ea_check_errors"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(fn, status):
    if status != EA_OK:
        raise EAError(fn, status)


def _dev(t, name, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t


def _strides(t):
    return (ctypes.c_int64 * t.dim())(*t.stride())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _mlp_struct(weights, biases):
    """(ea_mlp, keep-alive list) for float32 CUDA weights [out, in] and biases [out]."""
    Ws = [_dev(w, "W", torch.float32).contiguous() for w in weights]
    bs = [_dev(b, "b", torch.float32).contiguous() for b in biases]
    dims = [Ws[0].shape[1]] + [w.shape[0] for w in Ws]
    c_dims = (ctypes.c_int * len(dims))(*dims)
    c_W = (ctypes.c_void_p * len(Ws))(*[w.data_ptr() for w in Ws])
    c_b = (ctypes.c_void_p * len(bs))(*[b.data_ptr() for b in bs])
    return _Mlp(len(Ws), c_dims, c_W, c_b), [Ws, bs, c_dims, c_W, c_b]


def ea_route(K, weights, biases, *, pool_head=100, pool_tail=100, policy=(FULL, SSA),
             r_out=None, m_out=None, logits_out=None, stream=None):
    """Router pre-pass on K [B, S, Hkv, d] (bf16, CUDA).  weights/biases: lists of
    float32 CUDA tensors ([out, in] and [out]).  Returns (r, m, logits)."""
    _dev(K, "K", torch.bfloat16)
    B, S, Hkv, d = K.shape
    dev = K.device
    r_out = r_out if r_out is not None else torch.empty(B, Hkv, dtype=torch.uint8, device=dev)
    m_out = m_out if m_out is not None else torch.empty(B, Hkv, dtype=torch.uint8, device=dev)
    if logits_out is None:
        logits_out = torch.empty(B, Hkv, 2, dtype=torch.float64, device=dev)
    mlp, _keep = _mlp_struct(weights, biases)
    st = lib().ea_route(_ptr(K), _strides(K), B, S, Hkv, d, pool_head, pool_tail,
                        ctypes.byref(mlp), _Policy(*policy), _ptr(r_out), _ptr(m_out),
                        _ptr(logits_out), _stream(stream))
    _check("ea_route", st)
    return r_out, m_out, logits_out


def ea_route_layers(K_layers, weights, biases, *, pool_head=100, pool_tail=100,
                    policy=(FULL, SSA), r_out=None, m_out=None, logits_out=None, stream=None):
    """Router pre-pass of L layers at once.  K_layers: L bf16 CUDA tensors
    [B, S, Hkv, d] with equal shapes and strides; weights[l] / biases[l]: layer
    l's MLP as for ea_route.  Returns (r [L, B, Hkv], m [L, B, Hkv],
    logits [L, B, Hkv, 2])."""
    L = len(K_layers)
    if L < 1 or len(weights) != L or len(biases) != L:
        raise ValueError("K_layers, weights and biases need one entry per layer")
    K0 = _dev(K_layers[0], "K", torch.bfloat16)
    for K in K_layers:
        _dev(K, "K", torch.bfloat16)
        if K.shape != K0.shape or K.stride() != K0.stride():
            raise ValueError("every layer's K needs the same shape and strides")
    B, S, Hkv, d = K0.shape
    dev = K0.device
    if r_out is None:
        r_out = torch.empty(L, B, Hkv, dtype=torch.uint8, device=dev)
    if m_out is None:
        m_out = torch.empty(L, B, Hkv, dtype=torch.uint8, device=dev)
    if logits_out is None:
        logits_out = torch.empty(L, B, Hkv, 2, dtype=torch.float64, device=dev)
    built = [_mlp_struct(w, b) for w, b in zip(weights, biases)]
    mlps = (_Mlp * L)(*[m for m, _ in built])
    ptrs = (ctypes.c_void_p * L)(*[K.data_ptr() for K in K_layers])
    st = lib().ea_route_layers(ptrs, L, _strides(K0), B, S, Hkv, d, pool_head, pool_tail, mlps,
                               _Policy(*policy), _ptr(r_out), _ptr(m_out), _ptr(logits_out),
                               _stream(stream))
    _check("ea_route_layers", st)
    return r_out, m_out, logits_out


def ea_prefill_workspace_size(B, S, Hq, Hkv, d=128):
    return int(lib().ea_prefill_workspace_size(B, S, Hq, Hkv, d))


def prefill_workspace(B, S, Hq, Hkv, d=128, device="cuda"):
    """A zeroed workspace buffer of the right size (256-byte aligned by torch)."""
    n = ea_prefill_workspace_size(B, S, Hq, Hkv, d)
    if n == 0:
        raise ValueError("unsupported prefill sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def ea_hybrid_attn_prefill(Q, K, V, m, *, sink, window, block_mask=None, scale=None, O=None,
                           LSE=None, workspace=None, visited_bitmap=None, stream=None,
                           want_lse=True, _entry="ea_hybrid_attn_prefill"):
    """Fused hybrid-head prefill.  Q [B, S, Hq, d], K/V [B, S, Hkv, d] bf16 (CUDA),
    m uint8 [B, Hkv] (CUDA).  Returns (O, LSE)."""
    _dev(Q, "Q", torch.bfloat16)
    _dev(K, "K", torch.bfloat16)
    _dev(V, "V", torch.bfloat16)
    _dev(m, "m", torch.uint8)
    if K.stride() != V.stride():
        raise ValueError("K and V must share strides")
    B, S, Hq, d = Q.shape
    Hkv = K.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    if LSE is None and want_lse:
        LSE = torch.empty(B, Hq, S, dtype=torch.float32, device=Q.device)
    if workspace is None:
        workspace = prefill_workspace(B, S, Hq, Hkv, d, Q.device)
    if block_mask is not None:
        _dev(block_mask, "block_mask", torch.uint8)
        if not block_mask.is_contiguous():
            raise ValueError("block_mask must be contiguous")
    st = getattr(lib(), _entry)(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), _strides(Q), _strides(K), _strides(O),
        B, S, Hq, Hkv, d, float(scale), _ptr(m), int(sink), int(window), _ptr(block_mask), TILE,
        _ptr(workspace), workspace.numel(), _ptr(visited_bitmap), _stream(stream))
    _check(_entry, st)
    return O, LSE


def ea_prefill_plan(B, S, Hq, Hkv, m, *, sink, window, block_mask=None, workspace, d=128,
                    stream=None):
    """Enqueue the planner only (work queue into `workspace`)."""
    _dev(m, "m", torch.uint8)
    st = lib().ea_prefill_plan(B, S, Hq, Hkv, d, _ptr(m), int(sink), int(window), _ptr(block_mask),
                               TILE, _ptr(workspace), workspace.numel(), _stream(stream))
    _check("ea_prefill_plan", st)


def ea_prefill_attend(Q, K, V, m, *, sink, window, workspace, **kw):
    """Enqueue the attention kernel on a plan made by ea_prefill_plan."""
    return ea_hybrid_attn_prefill(Q, K, V, m, sink=sink, window=window, workspace=workspace,
                                  _entry="ea_prefill_attend", **kw)


def ea_hybrid_attn_prefill_noalloc(Q, K, V, m, *, sink, window, block_mask=None, scale=None,
                                   O=None, LSE=None, visited_bitmap=None, stream=None,
                                   want_lse=True):
    """ea_hybrid_attn_prefill without a workspace, for callers that cannot
    allocate device memory for the library: the planner's scratch is a fixed
    4 MiB array inside it, shared by every call (calls that overlap on the GPU
    race).  Returns (O, LSE)."""
    _dev(Q, "Q", torch.bfloat16)
    _dev(K, "K", torch.bfloat16)
    _dev(V, "V", torch.bfloat16)
    _dev(m, "m", torch.uint8)
    if K.stride() != V.stride():
        raise ValueError("K and V must share strides")
    B, S, Hq, d = Q.shape
    Hkv = K.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    if LSE is None and want_lse:
        LSE = torch.empty(B, Hq, S, dtype=torch.float32, device=Q.device)
    if block_mask is not None:
        _dev(block_mask, "block_mask", torch.uint8)
        if not block_mask.is_contiguous():
            raise ValueError("block_mask must be contiguous")
    st = lib().ea_hybrid_attn_prefill_noalloc(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), _strides(Q), _strides(K), _strides(O),
        B, S, Hq, Hkv, d, float(scale), _ptr(m), int(sink), int(window), _ptr(block_mask), TILE,
        _ptr(visited_bitmap), _stream(stream))
    _check("ea_hybrid_attn_prefill_noalloc", st)
    return O, LSE


def ea_prefill_layers_workspace_size(n_layers, B, S, Hq, Hkv, d=128):
    return int(lib().ea_prefill_layers_workspace_size(n_layers, B, S, Hq, Hkv, d))


def prefill_layers_workspace(n_layers, B, S, Hq, Hkv, d=128, device="cuda"):
    n = ea_prefill_layers_workspace_size(n_layers, B, S, Hq, Hkv, d)
    if n == 0:
        raise ValueError("unsupported multi-layer prefill sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def ea_hybrid_attn_prefill_layers(Qs, Ks, Vs, ms, *, sink, window, block_masks=None, scale=None,
                                  Os=None, LSEs=None, workspace=None, stream=None, want_lse=True):
    """Several layers (same shapes and strides) in one planner + one launch.
    Qs/Ks/Vs/ms: lists of per-layer CUDA tensors as for ea_hybrid_attn_prefill;
    block_masks: None or a list (entries may be None).  Returns (Os, LSEs)."""
    L = len(Qs)
    if not (len(Ks) == len(Vs) == len(ms) == L) or L < 1:
        raise ValueError("one Q, K, V and m per layer")
    for t, nm in ((Qs, "Q"), (Ks, "K"), (Vs, "V")):
        for x in t:
            _dev(x, nm, torch.bfloat16)
    for x in ms:
        _dev(x, "m", torch.uint8)
    B, S, Hq, d = Qs[0].shape
    Hkv = Ks[0].shape[2]
    for l in range(L):
        if (Qs[l].shape != Qs[0].shape or Ks[l].shape != Ks[0].shape or Vs[l].shape != Ks[0].shape or
                Qs[l].stride() != Qs[0].stride() or Ks[l].stride() != Ks[0].stride() or
                Vs[l].stride() != Ks[0].stride()):
            raise ValueError("every layer must have the same shapes and strides")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if Os is None:
        Os = [torch.empty_like(Qs[0]) for _ in range(L)]
    if LSEs is None:
        LSEs = [torch.empty(B, Hq, S, dtype=torch.float32, device=Qs[0].device) if want_lse else None
                for _ in range(L)]
    bms = list(block_masks) if block_masks is not None else [None] * L
    for bm in bms:
        if bm is not None:
            _dev(bm, "block_mask", torch.uint8)
            if not bm.is_contiguous():
                raise ValueError("block_mask must be contiguous")
    if workspace is None:
        workspace = prefill_layers_workspace(L, B, S, Hq, Hkv, d, Qs[0].device)
    arr = (_PrefillLayer * L)()
    for l in range(L):
        arr[l] = _PrefillLayer(Qs[l].data_ptr(), Ks[l].data_ptr(), Vs[l].data_ptr(), Os[l].data_ptr(),
                               LSEs[l].data_ptr() if LSEs[l] is not None else None, ms[l].data_ptr(),
                               bms[l].data_ptr() if bms[l] is not None else None)
    st = lib().ea_hybrid_attn_prefill_layers(
        ctypes.cast(arr, ctypes.c_void_p), L, _strides(Qs[0]), _strides(Ks[0]), _strides(Os[0]), B, S,
        Hq, Hkv, d, float(scale), int(sink), int(window), TILE, _ptr(workspace), workspace.numel(),
        _stream(stream))
    _check("ea_hybrid_attn_prefill_layers", st)
    return Os, LSEs


def ea_prefill_host_buffer_size(B, S, Hq, Hkv, d=128, with_block_mask=False):
    return int(lib().ea_prefill_host_buffer_size(B, S, Hq, Hkv, d, 1 if with_block_mask else 0))


def prefill_host_buffer(B, S, Hq, Hkv, d=128, with_block_mask=False, device="cuda"):
    """Device scratch for ea_hybrid_attn_prefill_host (256-byte aligned by torch)."""
    n = ea_prefill_host_buffer_size(B, S, Hq, Hkv, d, with_block_mask)
    if n == 0:
        raise ValueError("unsupported prefill sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _host(t, name, dtype):
    if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError("%s must be a contiguous host %s tensor" % (name, dtype))
    return t


def ea_hybrid_attn_prefill_host(Q, K, V, m, *, sink, window, block_mask=None, scale=None, O=None,
                                LSE=None, device_buffer=None, n_chunks=0, stream=None,
                                want_lse=True):
    """The fused prefill on HOST tensors (contiguous; page-locked for overlap):
    Q [B, S, Hq, d], K/V [B, S, Hkv, d] bf16, m uint8 [B, Hkv], block_mask uint8
    [B, Hkv, nB, nB] or None.  Copies in, attention and copies out run as a
    chunked pipeline on the current CUDA device.  Returns (O, LSE) as host
    tensors, complete once `stream` (default: the current stream) has passed
    the call's work."""
    _host(Q, "Q", torch.bfloat16)
    _host(K, "K", torch.bfloat16)
    _host(V, "V", torch.bfloat16)
    _host(m, "m", torch.uint8)
    if block_mask is not None:
        _host(block_mask, "block_mask", torch.uint8)
    B, S, Hq, d = Q.shape
    Hkv = K.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    pin = Q.is_pinned()
    if O is None:
        O = torch.empty(Q.shape, dtype=torch.bfloat16, pin_memory=pin)
    _host(O, "O", torch.bfloat16)
    if LSE is None and want_lse:
        LSE = torch.empty(B, Hq, S, dtype=torch.float32, pin_memory=pin)
    if LSE is not None:
        _host(LSE, "LSE", torch.float32)
    if device_buffer is None:
        device_buffer = prefill_host_buffer(B, S, Hq, Hkv, d, block_mask is not None)
    _dev(device_buffer, "device_buffer", torch.uint8)
    st = lib().ea_hybrid_attn_prefill_host(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), B, S, Hq, Hkv, d, float(scale), _ptr(m),
        int(sink), int(window), _ptr(block_mask), TILE, _ptr(device_buffer),
        device_buffer.numel(), int(n_chunks), _stream(stream))
    _check("ea_hybrid_attn_prefill_host", st)
    return O, LSE


def ea_prefill_varlen_workspace_size(B, total_tokens, max_seqlen, Hq, Hkv, d=128):
    return int(lib().ea_prefill_varlen_workspace_size(B, total_tokens, max_seqlen, Hq, Hkv, d))


def prefill_varlen_workspace(B, total_tokens, max_seqlen, Hq, Hkv, d=128, device="cuda"):
    n = ea_prefill_varlen_workspace_size(B, total_tokens, max_seqlen, Hq, Hkv, d)
    if n == 0:
        raise ValueError("unsupported variable-length prefill sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def ea_hybrid_attn_prefill_varlen(Q, K, V, cu_seqlens, m, *, max_seqlen, sink, window,
                                  block_mask=None, scale=None, O=None, LSE=None, workspace=None,
                                  stream=None, want_lse=True):
    """Sequences of different lengths packed back to back, one launch.
    Q [total, Hq, d], K/V [total, Hkv, d] bf16; cu_seqlens int32 [B + 1];
    m uint8 [B, Hkv]; block_mask uint8, per sequence [Hkv, nB_b, nB_b] back
    to back (or None); all CUDA.  Returns (O [total, Hq, d], LSE [Hq, total])."""
    _dev(Q, "Q", torch.bfloat16)
    _dev(K, "K", torch.bfloat16)
    _dev(V, "V", torch.bfloat16)
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    _dev(m, "m", torch.uint8)
    if K.stride() != V.stride():
        raise ValueError("K and V must share strides")
    total, Hq, d = Q.shape
    Hkv = K.shape[1]
    B = cu_seqlens.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    if LSE is None and want_lse:
        LSE = torch.empty(Hq, total, dtype=torch.float32, device=Q.device)
    if workspace is None:
        workspace = prefill_varlen_workspace(B, total, max_seqlen, Hq, Hkv, d, Q.device)
    st = lib().ea_hybrid_attn_prefill_varlen(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), _strides(Q), _strides(K), _strides(O),
        _ptr(cu_seqlens), B, total, int(max_seqlen), Hq, Hkv, d, float(scale), _ptr(m), int(sink),
        int(window), _ptr(block_mask), TILE, _ptr(workspace), workspace.numel(), _stream(stream))
    _check("ea_hybrid_attn_prefill_varlen", st)
    return O, LSE


def ea_decode_workspace_size(B, Hq, Hkv, Lmax, num_splits=0, d=128):
    return int(lib().ea_decode_workspace_size(B, Hq, Hkv, d, Lmax, num_splits))


def decode_workspace(B, Hq, Hkv, Lmax, num_splits=0, d=128, device="cuda"):
    n = ea_decode_workspace_size(B, Hq, Hkv, Lmax, num_splits, d)
    if n == 0:
        raise ValueError("unsupported decode sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _block_mask_arg(block_mask, B, Hkv, Lmax):
    if block_mask is None:
        return None
    _dev(block_mask, "block_mask", torch.uint8)
    nB = (Lmax + TILE - 1) // TILE
    if tuple(block_mask.shape) != (B, Hkv, nB, nB) or not block_mask.is_contiguous():
        raise ValueError("block_mask must be a contiguous [B, Hkv, %d, %d] tensor" % (nB, nB))
    return block_mask


def ea_hybrid_attn_decode(q, Kc, Vc, seqlens, m, *, sink, window, block_mask=None, num_splits=0,
                          scale=None, O=None, LSE=None, workspace=None, stream=None, want_lse=True):
    """One decode step.  q [B, Hq, d], Kc/Vc [B, Lmax, Hkv, d] bf16 (CUDA),
    seqlens int32 [B] (CUDA), m uint8 [B, Hkv] (CUDA), block_mask uint8
    [B, Hkv, nB, nB] (nB = ceil(Lmax / 128), CUDA) when a head is BLOCK.
    Returns (O, LSE)."""
    _dev(q, "q", torch.bfloat16)
    _dev(Kc, "Kc", torch.bfloat16)
    _dev(Vc, "Vc", torch.bfloat16)
    _dev(seqlens, "seqlens", torch.int32)
    _dev(m, "m", torch.uint8)
    if Kc.stride() != Vc.stride():
        raise ValueError("Kc and Vc must share strides")
    B, Hq, d = q.shape
    Lmax, Hkv = Kc.shape[1], Kc.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(q)
    if LSE is None and want_lse:
        LSE = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = decode_workspace(B, Hq, Hkv, Lmax, num_splits, d, q.device)
    bm = _block_mask_arg(block_mask, B, Hkv, Lmax)
    st = lib().ea_hybrid_attn_decode(
        _ptr(q), _ptr(Kc), _ptr(Vc), _ptr(O), _ptr(LSE), _strides(q), _strides(Kc), _strides(O),
        _ptr(seqlens), B, Hq, Hkv, d, Lmax, float(scale), _ptr(m), int(sink), int(window),
        _ptr(bm), TILE, int(num_splits), _ptr(workspace), workspace.numel(), _stream(stream))
    _check("ea_hybrid_attn_decode", st)
    return O, LSE


def ea_hybrid_attn_decode_paged(q, K_pages, V_pages, block_table, seqlens, m, *, sink, window,
                                block_mask=None, num_splits=0, scale=None, O=None, LSE=None,
                                workspace=None, stream=None, want_lse=True):
    """One decode step over a paged cache.  q [B, Hq, d]; K_pages/V_pages
    [num_pages, page_size, Hkv, d] bf16; block_table int32 [B, max_pages] (key
    k of sequence b: row k % page_size of page block_table[b, k // page_size]);
    seqlens int32 [B]; m uint8 [B, Hkv]; all CUDA.  Returns (O, LSE)."""
    _dev(q, "q", torch.bfloat16)
    _dev(K_pages, "K_pages", torch.bfloat16)
    _dev(V_pages, "V_pages", torch.bfloat16)
    _dev(block_table, "block_table", torch.int32)
    _dev(seqlens, "seqlens", torch.int32)
    _dev(m, "m", torch.uint8)
    if K_pages.stride() != V_pages.stride() or K_pages.shape != V_pages.shape:
        raise ValueError("K_pages and V_pages must share shapes and strides")
    if block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("block_table must be [B, max_pages] with unit column stride")
    B, Hq, d = q.shape
    num_pages, page_size, Hkv = K_pages.shape[0], K_pages.shape[1], K_pages.shape[2]
    max_pages = block_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(q)
    if LSE is None and want_lse:
        LSE = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = decode_workspace(B, Hq, Hkv, max_pages * page_size, num_splits, d, q.device)
    bm = _block_mask_arg(block_mask, B, Hkv, max_pages * page_size)
    st = lib().ea_hybrid_attn_decode_paged(
        _ptr(q), _ptr(K_pages), _ptr(V_pages), _ptr(O), _ptr(LSE), _strides(q), _strides(K_pages),
        _strides(O), _ptr(block_table), block_table.stride(0), max_pages, page_size, num_pages,
        _ptr(seqlens), B, Hq, Hkv, d, float(scale), _ptr(m), int(sink), int(window),
        _ptr(bm), TILE, int(num_splits), _ptr(workspace), workspace.numel(), _stream(stream))
    _check("ea_hybrid_attn_decode_paged", st)
    return O, LSE


XA_STRIDE = 16


def ea_xa_workspace_size(B, S, Hq, Hkv, max_units, d=128, stride=XA_STRIDE):
    return int(lib().ea_xa_workspace_size(B, S, Hq, Hkv, d, stride, max_units))


def xa_workspace(B, S, Hq, Hkv, max_units, d=128, device="cuda"):
    """A zeroed XA estimation workspace for at most max_units BLOCK (b, KV head) units."""
    n = ea_xa_workspace_size(B, S, Hq, Hkv, max_units, d)
    if n == 0:
        raise ValueError("unsupported XA estimation sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def ea_xa_estimate(Q, K, m, *, threshold=0.9, max_units=None, block_mask=None,
                   block_scores=None, want_scores=False, scale=None, workspace=None,
                   stride=XA_STRIDE, stream=None):
    """XA block-mask estimation (antidiagonal scoring) for the heads whose mode is
    BLOCK.  Q [B, S, Hq, d], K [B, S, Hkv, d] bf16 (CUDA), m uint8 [B, Hkv] (CUDA).
    Returns (block_mask uint8 [B, Hkv, nB, nB], block_scores float32 or None); rows
    of other heads are left as they are in a caller-given block_mask (zeros in a
    new one)."""
    _dev(Q, "Q", torch.bfloat16)
    _dev(K, "K", torch.bfloat16)
    _dev(m, "m", torch.uint8)
    B, S, Hq, d = Q.shape
    Hkv = K.shape[2]
    nB = (S + TILE - 1) // TILE
    if max_units is None:
        max_units = B * Hkv
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if block_mask is None:
        block_mask = torch.zeros(B, Hkv, nB, nB, dtype=torch.uint8, device=Q.device)
    _dev(block_mask, "block_mask", torch.uint8)
    if not block_mask.is_contiguous():
        raise ValueError("block_mask must be contiguous")
    if block_scores is None and want_scores:
        block_scores = torch.zeros(B, Hkv, nB, nB, dtype=torch.float32, device=Q.device)
    if block_scores is not None:
        _dev(block_scores, "block_scores", torch.float32)
        if not block_scores.is_contiguous():
            raise ValueError("block_scores must be contiguous")
    if workspace is None:
        workspace = xa_workspace(B, S, Hq, Hkv, max_units, d, Q.device)
    st = lib().ea_xa_estimate(_ptr(Q), _ptr(K), _strides(Q), _strides(K), B, S, Hq, Hkv, d,
                              float(scale), _ptr(m), int(stride), float(threshold), TILE,
                              int(max_units), _ptr(block_mask), _ptr(block_scores),
                              _ptr(workspace), workspace.numel(), _stream(stream))
    _check("ea_xa_estimate", st)
    return block_mask, block_scores


CACHE_FORMATS = {torch.bfloat16: 0, torch.float8_e4m3fn: 1, torch.int8: 2}
SCALE_BLOCKS = (16, 32, 64, 128)


class KVCache:
    """One layer's KV cache as the cache operators use it: a handle over the
    caller's tensors, made once and kept as long as they are.

    K, V: [B, Lmax, Hkv, 128], or with a block_table (int32 [B, max_pages])
    pages [num_pages, page_size, Hkv, 128]; bfloat16, float8_e4m3fn or int8.
    Sequences may name the same pages, each in a block_table row of its own (an
    expanded row is refused).  Pages hold a multiple of scale_block rows; of 64
    for the decode and, where they are written to, for bfloat16.
    k_scale, v_scale (8-bit formats): float32 [B or num_pages, Hkv,
    ceil(rows / scale_block)], one scale per block of scale_block tokens and
    head.  ``kv_cache`` and ``kv_cache_paged`` allocate an empty one."""

    def __init__(self, K, V, k_scale=None, v_scale=None, *, scale_block=64, block_table=None):
        _dev(K, "K")
        _dev(V, "V", K.dtype)
        if K.dtype not in CACHE_FORMATS:
            raise ValueError("K and V must be bfloat16, float8_e4m3fn or int8, got %s" % K.dtype)
        if K.dim() != 4 or V.shape != K.shape or V.stride() != K.stride():
            raise ValueError("K and V must share 4-dimensional shapes and strides")
        outer, rows, Hkv, d = K.shape
        if outer < 1 or rows < 1 or Hkv < 1:
            raise ValueError("an empty cache")
        self.quantized = K.dtype != torch.bfloat16
        if self.quantized:
            if scale_block not in SCALE_BLOCKS:
                raise ValueError("scale_block must be one of %s" % (SCALE_BLOCKS,))
            shape = (outer, Hkv, -(-rows // scale_block))
            for t, nm in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _dev(t, nm, torch.float32)
                if tuple(t.shape) != shape or not t.is_contiguous():
                    raise ValueError("%s must be a contiguous %s tensor" % (nm, list(shape)))
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bfloat16 cache has no scales")
        if block_table is not None:
            _dev(block_table, "block_table", torch.int32)
            if block_table.dim() != 2 or block_table.shape[1] < 1 or (
                    block_table.shape[1] > 1 and block_table.stride(1) != 1):
                raise ValueError("block_table must be [B, max_pages] with unit column stride")
            if block_table.shape[0] > 1 and block_table.stride(0) < block_table.shape[1]:
                raise ValueError("block_table's rows overlap: sequences that share pages need a row each "
                                 "(block_table.contiguous())")
            if self.quantized and rows % scale_block:
                raise ValueError("pages must hold a multiple of scale_block rows")
        _one_device(K, V, k_scale, v_scale, block_table)
        self.K, self.V, self.k_scale, self.v_scale = K, V, k_scale, v_scale
        self.scale_block, self.block_table = scale_block, block_table
        self.B = outer if block_table is None else block_table.shape[0]
        self.max_pages = 0 if block_table is None else block_table.shape[1]
        self.capacity = rows * max(self.max_pages, 1)
        self.Hkv, self.device = Hkv, K.device
        self._c = _Cache(K.data_ptr(), V.data_ptr(), 0 if k_scale is None else k_scale.data_ptr(),
                         0 if v_scale is None else v_scale.data_ptr(),
                         (ctypes.c_int64 * 4)(*K.stride()),
                         0 if block_table is None else block_table.data_ptr(),
                         # (the row stride of a single row means nothing)
                         block_table.stride(0) if self.B > 1 and block_table is not None else self.max_pages,
                         outer, rows, self.max_pages, Hkv, d, CACHE_FORMATS[K.dtype], scale_block)
        self._ref = ctypes.byref(self._c)


def _alloc_cache(outer, rows, Hkv, dtype, scale_block, device, block_table):
    K = torch.zeros(outer, rows, Hkv, 128, dtype=dtype, device=device)
    scales = [None, None]
    if dtype != torch.bfloat16:
        scales = [torch.zeros(outer, Hkv, -(-rows // scale_block), device=device) for _ in range(2)]
    return KVCache(K, torch.zeros_like(K), *scales, scale_block=scale_block, block_table=block_table)


def kv_cache(B, Lmax, Hkv, *, dtype=torch.float8_e4m3fn, scale_block=64, device="cuda"):
    """An empty contiguous cache [B, Lmax, Hkv, 128]."""
    return _alloc_cache(B, Lmax, Hkv, dtype, scale_block, device, None)


def kv_cache_paged(num_pages, page_size, Hkv, block_table, *, dtype=torch.float8_e4m3fn,
                   scale_block=64):
    """An empty pool of pages [num_pages, page_size, Hkv, 128] read through
    block_table (int32 [B, max_pages], CUDA)."""
    return _alloc_cache(num_pages, page_size, Hkv, dtype, scale_block, block_table.device, block_table)


def _one_device(first, *tensors):
    dev = first.get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors on several devices: %s and %s" % (first.device, t.device))


class _at:
    """Runs a call on the device of its tensors and on the stream it names (the
    device's current one if none), allocations included."""

    __slots__ = ("device", "ctx")

    def __init__(self, device, stream):
        self.device = device
        self.ctx = None
        if stream is not None and stream.device != device:
            raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
        if stream is not None or device.index != torch._C._cuda_getDevice():
            self.ctx = [torch.cuda.device(device)]
            if stream is not None:
                self.ctx.append(torch.cuda.stream(stream))

    def __enter__(self):
        if self.ctx:
            for c in self.ctx:
                c.__enter__()
        # (torch.cuda.current_stream() takes several microseconds to make a Stream)
        return torch._C._cuda_getCurrentRawStream(self.device.index)

    def __exit__(self, *exc):
        if self.ctx:
            for c in reversed(self.ctx):
                c.__exit__(*exc)


_I64 = {n: ctypes.c_int64 * n for n in (3, 4)}


def _like(t, name, shape, dtype):
    _dev(t, name, dtype)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s %s tensor" % (name, dtype, list(shape)))
    return t


def _i32_vec(t, name, B):
    return t if t is None else _like(t, name, (B,), torch.int32)


def ea_cache_workspace_size():
    return int(lib().ea_cache_workspace_size())


def _clear_workspace(n, device):
    # only the header has to be zero, and the decode's stored logits may be large
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def cache_workspace(device="cuda"):
    """A zeroed workspace of ea_cache_write, ea_evict_select, ea_cache_compact,
    ea_rope, ea_cache_write_rope, ea_tree_plan and ea_tree_accept (their error
    word)."""
    return torch.zeros(ea_cache_workspace_size(), dtype=torch.uint8, device=device)


def ea_cache_write(cache, K, V, start=None, n_new=None, *, workspace=None, stream=None):
    """Append K, V [B, T, Hkv, 128] (bf16, CUDA) to the sequences of a KVCache at
    rows start[b] (int32 [B]; None: 0), the first n_new[b] (int32 [B]; None: T)
    tokens of each, quantising them for an 8-bit cache."""
    _dev(K, "K", torch.bfloat16)
    _dev(V, "V", torch.bfloat16)
    if K.dim() != 4 or V.shape != K.shape or V.stride() != K.stride():
        raise ValueError("K and V must share 4-dimensional shapes and strides")
    B, T, Hkv, d = K.shape
    if (B, Hkv, d) != (cache.B, cache.Hkv, 128):
        raise ValueError("K and V must be [%d, T, %d, 128]" % (cache.B, cache.Hkv))
    _i32_vec(start, "start", B)
    _i32_vec(n_new, "n_new", B)
    _one_device(cache.K, K, V, start, n_new, workspace)
    with _at(cache.device, stream) as st:
        if workspace is None:
            workspace = cache_workspace(cache.device)
        _check("ea_cache_write", lib().ea_cache_write(
            cache._ref, K.data_ptr(), V.data_ptr(), _I64[4](*K.stride()), _ptr(start), _ptr(n_new), B, T,
            workspace.data_ptr(), workspace.numel(), st))


def ea_decode_q8_workspace_size(B, Hq, Hkv, Lmax, num_splits=0, weights=False, d=128):
    return int(lib().ea_decode_q8_workspace_size(B, Hq, Hkv, d, Lmax, num_splits, 1 if weights else 0))


def decode_q8_workspace(B, Hq, Hkv, Lmax, num_splits=0, weights=False, d=128, device="cuda"):
    """A workspace of ea_hybrid_attn_decode_q8 (weights: with key_weights), its
    error word zero."""
    n = ea_decode_q8_workspace_size(B, Hq, Hkv, Lmax, num_splits, weights, d)
    if n == 0:
        raise ValueError("unsupported decode sizes")
    return _clear_workspace(n, device)


def ea_hybrid_attn_decode_q8(q, cache, seqlens, m, *, sink, window, block_mask=None, num_splits=0,
                             scale=None, key_weights=None, accumulate=True, O=None, LSE=None,
                             workspace=None, stream=None, want_lse=True):
    """One decode step over an 8-bit KVCache: q [B, Hq, 128] bf16, seqlens int32
    [B], m uint8 [B, Hkv], block_mask uint8 [B, Hkv, nB, nB] (nB =
    ceil(capacity / 128)) when a head is BLOCK; all CUDA.  key_weights (float32
    [B, Hkv, capacity]) receives each cached key's attention weight of this
    step, summed over the group's heads: added (accumulate) or stored.
    Returns (O, LSE)."""
    _dev(q, "q", torch.bfloat16)
    _dev(m, "m", torch.uint8)
    if q.dim() != 3 or q.shape[0] != cache.B or q.shape[2] != 128:
        raise ValueError("q must be [%d, Hq, 128]" % cache.B)
    if not cache.quantized:
        raise ValueError("a bfloat16 cache is read by ea_hybrid_attn_decode")
    B, Hq, d = q.shape
    if seqlens is None:
        raise ValueError("seqlens is needed")
    _i32_vec(seqlens, "seqlens", B)
    _like(m, "m", (B, cache.Hkv), torch.uint8)
    bm = _block_mask_arg(block_mask, B, cache.Hkv, cache.capacity)
    if key_weights is not None:
        _like(key_weights, "key_weights", (B, cache.Hkv, cache.capacity), torch.float32)
    if O is not None:
        _dev(O, "O", torch.bfloat16)
        if O.shape != q.shape:
            raise ValueError("O must have q's shape")
    if LSE is not None:
        _like(LSE, "LSE", (B, Hq), torch.float32)
    _one_device(cache.K, q, seqlens, m, bm, key_weights, O, LSE, workspace)
    with _at(cache.device, stream) as st:
        if O is None:
            O = q.new_empty(q.shape)
        if LSE is None and want_lse:
            LSE = q.new_empty((B, Hq), dtype=torch.float32)
        if workspace is None:
            workspace = decode_q8_workspace(B, Hq, cache.Hkv, cache.capacity, num_splits,
                                            key_weights is not None, d, q.device)
        _check("ea_hybrid_attn_decode_q8", lib().ea_hybrid_attn_decode_q8(
            q.data_ptr(), cache._ref, O.data_ptr(), _ptr(LSE), _I64[3](*q.stride()),
            _I64[3](*O.stride()), seqlens.data_ptr(), B, Hq,
            1.0 / math.sqrt(d) if scale is None else float(scale),
            m.data_ptr(), int(sink), int(window), _ptr(bm), TILE, int(num_splits),
            _ptr(key_weights), 1 if accumulate else 0, workspace.data_ptr(),
            workspace.numel(), st))
    return O, LSE


def ea_key_weights_workspace_size(B, Tq, Lmax, Hq, Hkv, d=128):
    return int(lib().ea_key_weights_workspace_size(B, Tq, Lmax, Hq, Hkv, d))


def key_weights_workspace(B, Tq, Lmax, Hq, Hkv, d=128, device="cuda"):
    """A workspace of ea_key_weights, its error word zero."""
    n = ea_key_weights_workspace_size(B, Tq, Lmax, Hq, Hkv, d)
    if n == 0:
        raise ValueError("unsupported key weight sizes")
    return _clear_workspace(n, device)


def ea_key_weights(Q, K, LSE, m, *, sink, window, seqlens=None, block_mask=None, scale=None,
                   weights=None, accumulate=True, workspace=None, stream=None):
    """The attention weight that the last Tq query rows of each sequence give its
    keys.  Q [B, Tq, Hq, 128], K [B, Lmax, Hkv, 128] bf16; LSE float32 [B, Hq,
    Tq] (the prefill's for those rows, a view of its last columns; unit stride
    along the rows); m uint8 [B, Hkv]; seqlens int32 [B] (None: Lmax; query row
    t sits at position seqlens[b] - Tq + t); block_mask uint8 [B, Hkv, nB, nB]
    (nB = ceil(Lmax / 128)) when a head is BLOCK; all CUDA.  weights (float32
    [B, Hkv, Lmax]) is added to (accumulate) or written for the keys below
    seqlens[b]; zeros are allocated if it is not given.  Returns it."""
    _dev(Q, "Q", torch.bfloat16)
    _dev(K, "K", torch.bfloat16)
    _dev(LSE, "LSE", torch.float32)
    if Q.dim() != 4 or K.dim() != 4 or Q.shape[0] != K.shape[0] or Q.shape[3] != K.shape[3]:
        raise ValueError("Q must be [B, Tq, Hq, d], K [B, Lmax, Hkv, d]")
    B, Tq, Hq, d = Q.shape
    Lmax, Hkv = K.shape[1], K.shape[2]
    if tuple(LSE.shape) != (B, Hq, Tq) or (Tq > 1 and LSE.stride(2) != 1):
        raise ValueError("LSE must be [%d, %d, %d] with unit stride along the rows" % (B, Hq, Tq))
    _like(m, "m", (B, Hkv), torch.uint8)
    _i32_vec(seqlens, "seqlens", B)
    bm = _block_mask_arg(block_mask, B, Hkv, Lmax)
    if weights is not None:
        _like(weights, "weights", (B, Hkv, Lmax), torch.float32)
    _one_device(Q, K, LSE, m, seqlens, bm, weights, workspace)
    with _at(Q.device, stream) as st:
        if weights is None:
            weights = torch.zeros(B, Hkv, Lmax, dtype=torch.float32, device=Q.device)
        if workspace is None:
            workspace = key_weights_workspace(B, Tq, Lmax, Hq, Hkv, d, Q.device)
        _check("ea_key_weights", lib().ea_key_weights(
            Q.data_ptr(), K.data_ptr(), LSE.data_ptr(), _I64[4](*Q.stride()), _I64[4](*K.stride()), _I64[3](*LSE.stride()),
            _ptr(seqlens), B, Tq, Lmax, Hq, Hkv, d, 1.0 / math.sqrt(d) if scale is None else float(scale),
            m.data_ptr(), int(sink), int(window), _ptr(bm), TILE, weights.data_ptr(),
            1 if accumulate else 0, workspace.data_ptr(), workspace.numel(), st))
    return weights


def ea_evict_select(weights, seqlens, *, keep, sink=0, recent=0, index=None, new_seqlens=None,
                    workspace=None, stream=None):
    """The tokens that stay when every sequence is cut to `keep`: the first
    `sink`, the last `recent` and the heaviest of the others by weights (float32
    [B, Hkv, Lmax]), per KV head, ascending.  Returns (index int32 [B, Hkv,
    keep], -1 behind the kept ones; new_seqlens int32 [B])."""
    _dev(weights, "weights", torch.float32)
    if weights.dim() != 3 or not weights.is_contiguous():
        raise ValueError("weights must be a contiguous [B, Hkv, Lmax] tensor")
    B, Hkv, Lmax = weights.shape
    if seqlens is None:
        raise ValueError("seqlens is needed")
    _i32_vec(seqlens, "seqlens", B)
    _i32_vec(new_seqlens, "new_seqlens", B)
    if index is not None:
        _like(index, "index", (B, Hkv, keep), torch.int32)
    _one_device(weights, seqlens, index, new_seqlens, workspace)
    with _at(weights.device, stream) as st:
        if index is None:
            index = torch.empty(B, Hkv, max(int(keep), 0), dtype=torch.int32, device=weights.device)
        if new_seqlens is None:
            new_seqlens = torch.empty(B, dtype=torch.int32, device=weights.device)
        if workspace is None:
            workspace = cache_workspace(weights.device)
        _check("ea_evict_select", lib().ea_evict_select(
            weights.data_ptr(), seqlens.data_ptr(), B, Hkv, Lmax, int(keep), int(sink), int(recent),
            index.data_ptr(), new_seqlens.data_ptr(), workspace.data_ptr(), workspace.numel(), st))
    return index, new_seqlens


def ea_cache_compact(src, dst, index, counts, *, weights=None, weights_out=None, workspace=None,
                     stream=None):
    """Gather rows index[b, h, i] (int32 [B, Hkv, keep]; i < counts[b], int32
    [B]) of KVCache src into rows i of KVCache dst; the formats may differ.
    weights / weights_out (float32 [B, Hkv, capacity]): the tokens' accumulated
    weights move along."""
    B, Hkv = dst.B, dst.Hkv
    if (src.B, src.Hkv) != (B, Hkv):
        raise ValueError("src and dst must have the same sequences and heads")
    _dev(index, "index", torch.int32)
    if index.dim() != 3 or index.shape[:2] != (B, Hkv) or not index.is_contiguous():
        raise ValueError("index must be a contiguous [%d, %d, keep] tensor" % (B, Hkv))
    if counts is None:
        raise ValueError("counts is needed")
    _i32_vec(counts, "counts", B)
    if (weights is None) != (weights_out is None):
        raise ValueError("weights and weights_out go together")
    if weights is not None:
        _like(weights, "weights", (B, Hkv, src.capacity), torch.float32)
        _like(weights_out, "weights_out", (B, Hkv, dst.capacity), torch.float32)
    _one_device(src.K, dst.K, index, counts, weights, weights_out, workspace)
    with _at(dst.device, stream) as st:
        if workspace is None:
            workspace = cache_workspace(dst.device)
        _check("ea_cache_compact", lib().ea_cache_compact(
            src._ref, dst._ref, index.data_ptr(), counts.data_ptr(), B, index.shape[2], _ptr(weights),
            _ptr(weights_out), workspace.data_ptr(), workspace.numel(), st))


_BF16, _I32 = torch.bfloat16, torch.int32


def _fit(t, name, dtype, shape, dev):
    """t is a contiguous CUDA tensor of this kind on device `dev`, or None (these calls
    are short: their checks are made in one place, and told apart when one fails)."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        return
    _like(t, name, shape, dtype)
    raise ValueError("tensors on several devices: %s on %s" % (name, t.device))


def _fit4(t, name, shape, dev):
    """The same for bfloat16 tensors of any strides; returns their strides."""
    if not (t.dtype is _BF16 and t.shape == shape and t.get_device() == dev):
        _dev(t, name, _BF16)
        if tuple(t.shape) != shape:
            raise ValueError("%s must be a %s tensor, got %s" % (name, list(shape), list(t.shape)))
        raise ValueError("tensors on several devices: %s on %s" % (name, t.device))
    return _strides4(t.stride())


@functools.lru_cache(maxsize=256)
def _strides4(strides):
    return _I64[4](*strides)


def _shape4(t, name):
    _dev(t, name, _BF16)
    if t.dim() != 4 or t.shape[3] != 128:
        raise ValueError("%s must be [B, T, heads, 128]" % name)
    return t.shape


def _needed(t, name):
    if t is None:
        raise ValueError("%s is needed" % name)


def _workspace_fits(workspace, dev):
    if workspace is not None and workspace.get_device() != dev:
        raise ValueError("tensors on several devices: workspace on %s" % workspace.device)


MAX_TREE = 128


def ea_rope(Q, K, positions, inv_freq, *, n_new=None, interleaved=False, rope_scale=1.0, Q_out=None,
            K_out=None, workspace=None, stream=None):
    """Rotate queries Q [B, T, Hq, 128] and keys K [B, T, Hkv, 128] (bf16, CUDA;
    either may be None) by positions (int32 [B, T]): the first rot = 2 *
    len(inv_freq) dims in pairs (i, i + rot / 2), or neighbours (interleaved),
    by positions * inv_freq (float32, radians per position), times rope_scale.
    n_new (int32 [B]): rows at or behind it are not written.  Q_out and K_out
    may be Q and K.  Returns (Q_out, K_out)."""
    if Q is None and K is None:
        raise ValueError("Q or K is needed")
    x = Q if Q is not None else K
    B, T = _shape4(x, "Q" if Q is not None else "K")[:2]
    dev = x.get_device()
    _needed(positions, "positions")
    _needed(inv_freq, "inv_freq")
    _fit(positions, "positions", _I32, (B, T), dev)
    half = inv_freq.numel()
    _fit(inv_freq, "inv_freq", torch.float32, (half,), dev)
    _fit(n_new, "n_new", _I32, (B,), dev)
    _workspace_fits(workspace, dev)
    Hq = Hkv = 0
    qs = qos = ks = kos = None
    with _at(x.device, stream) as st:
        if Q is not None:
            Hq = Q.shape[2]
            qs = _fit4(Q, "Q", (B, T, Hq, 128), dev)
            if Q_out is None:
                Q_out = torch.empty_like(Q)
            qos = _fit4(Q_out, "Q_out", (B, T, Hq, 128), dev)
        elif Q_out is not None:
            raise ValueError("Q_out without Q")
        if K is not None:
            Hkv = _shape4(K, "K")[2]
            ks = _fit4(K, "K", (B, T, Hkv, 128), dev)
            if K_out is None:
                K_out = torch.empty_like(K)
            kos = _fit4(K_out, "K_out", (B, T, Hkv, 128), dev)
        elif K_out is not None:
            raise ValueError("K_out without K")
        if workspace is None:
            workspace = cache_workspace(x.device)
        _check("ea_rope", lib().ea_rope(
            _adr(Q), _adr(Q_out), qs, qos, Hq, _adr(K), _adr(K_out), ks, kos, Hkv, B, T, 128, inv_freq.data_ptr(),
            2 * half, 1 if interleaved else 0, rope_scale, positions.data_ptr(), _adr(n_new),
            workspace.data_ptr(), workspace.numel(), st))
    return Q_out, K_out


def _adr(t):
    return None if t is None else t.data_ptr()


def ea_cache_write_rope(cache, K, V, inv_freq, *, Q=None, Q_out=None, start=None, n_new=None, rows=None,
                        positions=None, interleaved=False, rope_scale=1.0, workspace=None, stream=None):
    """ea_cache_write with the rotation of ea_rope on the way: K, V [B, T, Hkv,
    128] (bf16, CUDA, unrotated) go to rows start[b] + i of a KVCache of any
    format, K rotated.  rows (int32 [B, T]): new token i is row rows[b, i] of K
    and V (an accepted path).  positions (int32 [B, T]) of the rows of K (and
    Q); None: start[b] + i.  Q [B, T, Hq, 128] (not with rows) is rotated into
    Q_out (may be Q; allocated if None), which is returned."""
    B, T, Hkv = _shape4(K, "K")[:3]
    _dev(V, "V", _BF16)
    if V.shape != K.shape or V.stride() != K.stride():
        raise ValueError("K and V must share shapes and strides")
    if not isinstance(cache, KVCache) or (B, Hkv) != (cache.B, cache.Hkv):
        raise ValueError("K and V must have the sequences and heads of the KVCache")
    dev = cache.device.index
    ns = _fit4(K, "K", (B, T, Hkv, 128), dev)
    _fit4(V, "V", (B, T, Hkv, 128), dev)
    _needed(inv_freq, "inv_freq")
    half = inv_freq.numel()
    _fit(inv_freq, "inv_freq", torch.float32, (half,), dev)
    _fit(start, "start", _I32, (B,), dev)
    _fit(n_new, "n_new", _I32, (B,), dev)
    _fit(rows, "rows", _I32, (B, T), dev)
    _fit(positions, "positions", _I32, (B, T), dev)
    _workspace_fits(workspace, dev)
    Hq, qs, qos = 0, None, None
    with _at(cache.device, stream) as st:
        if Q is not None:
            if rows is not None:
                raise ValueError("Q and rows do not go together")
            Hq = _shape4(Q, "Q")[2]
            qs = _fit4(Q, "Q", (B, T, Hq, 128), dev)
            if Q_out is None:
                Q_out = torch.empty_like(Q)
            qos = _fit4(Q_out, "Q_out", (B, T, Hq, 128), dev)
        elif Q_out is not None:
            raise ValueError("Q_out without Q")
        if workspace is None:
            workspace = cache_workspace(cache.device)
        _check("ea_cache_write_rope", lib().ea_cache_write_rope(
            cache._ref, K.data_ptr(), V.data_ptr(), ns, _adr(Q), _adr(Q_out), qs, qos, Hq, inv_freq.data_ptr(),
            2 * half, 1 if interleaved else 0, rope_scale, _adr(positions), _adr(start), _adr(n_new), _adr(rows), B,
            T, workspace.data_ptr(), workspace.numel(), st))
    return Q_out


def _tree_shape(t, name):
    _dev(t, name, _I32)
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous [B, T] tensor" % name)
    return t.shape


def ea_tree_plan(parents, n_nodes=None, *, depth=None, mask=None, workspace=None, stream=None):
    """Depth and ancestors of the nodes of drafted trees: parents int32 [B, T]
    (-1 for a root, else a node before it; T <= 128), n_nodes int32 [B] (None:
    T).  Returns (depth int32 [B, T], mask int32 [B, T, 4]: bit u % 32 of word
    u // 32 for the node itself and every ancestor u); zeros behind a
    sequence's last node."""
    B, T = _tree_shape(parents, "parents")
    dev = parents.get_device()
    _fit(n_nodes, "n_nodes", _I32, (B,), dev)
    _fit(depth, "depth", _I32, (B, T), dev)
    _fit(mask, "mask", _I32, (B, T, 4), dev)
    _workspace_fits(workspace, dev)
    with _at(parents.device, stream) as st:
        if depth is None:
            depth = torch.empty_like(parents)
        if mask is None:
            mask = torch.empty((B, T, 4), dtype=_I32, device=parents.device)
        if workspace is None:
            workspace = cache_workspace(parents.device)
        _check("ea_tree_plan", lib().ea_tree_plan(
            parents.data_ptr(), _adr(n_nodes), B, T, depth.data_ptr(), mask.data_ptr(), workspace.data_ptr(),
            workspace.numel(), st))
    return depth, mask


def ea_tree_workspace_size(B, T, Hq, Hkv, Lmax, d=128):
    return int(lib().ea_tree_workspace_size(B, T, Hq, Hkv, d, Lmax))


def tree_workspace(B, T, Hq, Hkv, Lmax, d=128, device="cuda"):
    """A workspace of ea_hybrid_attn_tree for a cache of Lmax rows a sequence, its
    error word zero."""
    n = ea_tree_workspace_size(B, T, Hq, Hkv, Lmax, d)
    if n == 0:
        raise ValueError("unsupported tree sizes")
    return _clear_workspace(n, device)


def ea_hybrid_attn_tree(Q, K, V, cache, seqlens, depth, mask, m, *, sink, window, n_nodes=None, block_mask=None,
                        scale=None, O=None, LSE=None, workspace=None, stream=None, want_lse=True):
    """Attention of every sequence's drafted tokens over its KVCache and over one
    another: Q [B, T, Hq, 128], K, V [B, T, Hkv, 128] bf16 (the drafted tokens',
    rotated; T <= 128), seqlens int32 [B] (tokens in the cache), depth int32 [B,
    T] and mask int32 [B, T, 4] of ea_tree_plan, m uint8 [B, Hkv], n_nodes int32
    [B] (None: T; rows at or behind it are not written), block_mask uint8 [B,
    Hkv, nB, nB] (nB = ceil(capacity / 128)) when a head is BLOCK; all CUDA.
    Returns (O [B, T, Hq, 128], LSE float32 [B, Hq, T])."""
    B, T, Hq = _shape4(Q, "Q")[:3]
    if not isinstance(cache, KVCache) or B != cache.B:
        raise ValueError("Q must have the sequences of the KVCache")
    dev, Hkv = cache.device.index, cache.Hkv
    qs = _fit4(Q, "Q", (B, T, Hq, 128), dev)
    ks = _fit4(K, "K", (B, T, Hkv, 128), dev)
    _fit4(V, "V", (B, T, Hkv, 128), dev)
    if V.stride() != K.stride():
        raise ValueError("K and V must share strides")
    for t, nm in ((seqlens, "seqlens"), (depth, "depth"), (mask, "mask"), (m, "m")):
        if t is None:
            raise ValueError("%s is needed" % nm)
    _fit(seqlens, "seqlens", _I32, (B,), dev)
    _fit(n_nodes, "n_nodes", _I32, (B,), dev)
    _fit(depth, "depth", _I32, (B, T), dev)
    _fit(mask, "mask", _I32, (B, T, 4), dev)
    _fit(m, "m", torch.uint8, (B, Hkv), dev)
    _fit(LSE, "LSE", torch.float32, (B, Hq, T), dev)
    bm = _block_mask_arg(block_mask, B, Hkv, cache.capacity)
    if bm is not None and bm.get_device() != dev:
        raise ValueError("tensors on several devices: block_mask on %s" % bm.device)
    _workspace_fits(workspace, dev)
    with _at(cache.device, stream) as st:
        if O is None:
            O = torch.empty_like(Q)
        os = _fit4(O, "O", (B, T, Hq, 128), dev)
        if LSE is None and want_lse:
            LSE = torch.empty((B, Hq, T), dtype=torch.float32, device=cache.device)
        if workspace is None:
            workspace = tree_workspace(B, T, Hq, Hkv, cache.capacity, 128, cache.device)
        _check("ea_hybrid_attn_tree", lib().ea_hybrid_attn_tree(
            Q.data_ptr(), K.data_ptr(), V.data_ptr(), cache._ref, O.data_ptr(), _adr(LSE), qs, ks, os,
            seqlens.data_ptr(), _adr(n_nodes), depth.data_ptr(), mask.data_ptr(), B, T, Hq,
            _SCALE128 if scale is None else float(scale), m.data_ptr(), int(sink), int(window), _adr(bm),
            TILE, workspace.data_ptr(), workspace.numel(), st))
    return O, LSE


_SCALE128 = 1.0 / math.sqrt(128)


def ea_tree_accept(tokens, parents, targets, n_nodes=None, *, path=None, n_accepted=None, next_token=None,
                   workspace=None, stream=None):
    """The path of each drafted tree that the model agrees with.  tokens, parents
    and targets int32 [B, T]: each node's token, its parent, and the model's
    token after it; node 0 is the token sampled last.  Returns (path int32 [B,
    T], -1 behind the accepted nodes; n_accepted int32 [B]; next_token int32
    [B])."""
    B, T = _tree_shape(tokens, "tokens")
    _needed(parents, "parents")
    _needed(targets, "targets")
    dev = tokens.get_device()
    _fit(parents, "parents", _I32, (B, T), dev)
    _fit(targets, "targets", _I32, (B, T), dev)
    _fit(path, "path", _I32, (B, T), dev)
    _fit(n_nodes, "n_nodes", _I32, (B,), dev)
    _fit(n_accepted, "n_accepted", _I32, (B,), dev)
    _fit(next_token, "next_token", _I32, (B,), dev)
    _workspace_fits(workspace, dev)
    with _at(tokens.device, stream) as st:
        if path is None:
            path = torch.empty_like(tokens)
        if n_accepted is None:
            n_accepted = torch.empty(B, dtype=_I32, device=tokens.device)
        if next_token is None:
            next_token = torch.empty_like(n_accepted)
        if workspace is None:
            workspace = cache_workspace(tokens.device)
        _check("ea_tree_accept", lib().ea_tree_accept(
            tokens.data_ptr(), parents.data_ptr(), targets.data_ptr(), _adr(n_nodes), B, T, path.data_ptr(),
            n_accepted.data_ptr(), next_token.data_ptr(), workspace.data_ptr(), workspace.numel(), st))
    return path, n_accepted, next_token


def ea_sparsity_ratios(r, m, S, *, sink, window, block_masks=None):
    """Host: (Omega_MSR, Omega_ESR) for r, m uint8 [L, Hkv] (CPU tensors or arrays);
    block_masks: None or a list of L uint8 [Hkv, nB, nB] CPU arrays (None entries
    for layers without BLOCK heads)."""
    import numpy as np
    ra = np.ascontiguousarray(np.asarray(r.cpu() if isinstance(r, torch.Tensor) else r), np.uint8)
    ma = np.ascontiguousarray(np.asarray(m.cpu() if isinstance(m, torch.Tensor) else m), np.uint8)
    L, Hkv = ra.shape
    keep = []
    c_masks = None
    if block_masks is not None:
        c_masks = (ctypes.c_void_p * L)()
        for l, bm in enumerate(block_masks):
            if bm is None:
                c_masks[l] = None
                continue
            a = np.ascontiguousarray(np.asarray(bm.cpu() if isinstance(bm, torch.Tensor) else bm),
                                     np.uint8)
            keep.append(a)
            c_masks[l] = a.ctypes.data
    msr, esr = ctypes.c_double(), ctypes.c_double()
    st = lib().ea_sparsity_ratios(ra.ctypes.data, ma.ctypes.data, L, Hkv, S, sink, window,
                                  c_masks, TILE, ctypes.byref(msr), ctypes.byref(esr))
    _check("ea_sparsity_ratios", st)
    return msr.value, esr.value


def ea_check_errors(workspace, stream=None):
    """Synchronise and read/clear the device error word; returns the status code."""
    return lib().ea_check_errors(_ptr(workspace), _stream(stream))
