"""Python binding of the CRISP sparse-prefill C ABI (``include/crisp.h``).

Argument marshalling only: every step runs in the CUDA kernels of
``libcrisp.so``. Tensors are passed by ``data_ptr()``; PyTorch provides the
device memory and the stream. Each wrapper raises :class:`CrispError` when the
library returns a non-OK status. Importing succeeds without a GPU; calling a
step without the built library raises immediately (there is no fallback).
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcrisp.so")
_lib = None

B = 128
D = 128


def num_blocks(n: int) -> int:
    """Blocks of an n-token layer: ceil(n / 128), the last one short when 128 does not divide n."""
    return (n + B - 1) // B


def map_ld(n: int) -> int:
    """Row stride (floats) of the proxy map: 128 * num_blocks(n)."""
    return num_blocks(n) * B

STATUS_NAMES = {0: "CRISP_OK", 1: "CRISP_ERR_INVALID_ARG", 2: "CRISP_ERR_SHAPE", 3: "CRISP_ERR_ALIGN",
                4: "CRISP_ERR_WORKSPACE", 5: "CRISP_ERR_CUDA", 6: "CRISP_ERR_TIMEOUT", 7: "CRISP_ERR_DEVICE",
                8: "CRISP_ERR_BOUNDS", 9: "CRISP_ERR_PAGES"}
PE_GAMMA, PE_NOISE = 0, 1
ROUTE_CSTRUCT, ROUTE_JSD = 0, 1
VS_NOISE, VS_GAMMA = 0, 1


class CrispError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


class Shape(ctypes.Structure):
    _fields_ = [("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("seq_len", ctypes.c_int32), ("block", ctypes.c_int32),
                ("q_head_stride", ctypes.c_int64), ("q_tok_stride", ctypes.c_int64),
                ("kv_head_stride", ctypes.c_int64), ("kv_tok_stride", ctypes.c_int64),
                ("o_head_stride", ctypes.c_int64), ("o_tok_stride", ctypes.c_int64),
                ("scale", ctypes.c_float)]


class Params(ctypes.Structure):
    _fields_ = [("tau_num", ctypes.c_uint32), ("tau_den", ctypes.c_uint32),
                ("alpha_num", ctypes.c_uint32), ("alpha_den", ctypes.c_uint32),
                ("gamma_num", ctypes.c_uint32), ("gamma_den", ctypes.c_uint32),
                ("kmin_blocks", ctypes.c_int32), ("pe_mode", ctypes.c_int32),
                ("route_mode", ctypes.c_int32), ("vs_mode", ctypes.c_int32),
                ("vs_gamma_num", ctypes.c_uint32), ("vs_gamma_den", ctypes.c_uint32),
                ("jsd_tau", ctypes.c_float), ("dense_below", ctypes.c_int32),
                ("sink_tokens", ctypes.c_int32), ("recency_tokens", ctypes.c_int32)]


class LayerViews(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in
                ("vmass", "smass", "rmass", "cstruct", "total", "route", "vbits", "sbits", "pbar", "pebits",
                 "rowbits", "counts", "order")]


class KVCache(ctypes.Structure):
    """A paged 8-bit key/value cache (make_kv_cache); keeps its tensors alive."""
    _fields_ = [("batch", ctypes.c_int32), ("hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p)]


class Tokens(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("tok_stride", ctypes.c_int64)]


class KVStep(ctypes.Structure):
    """What kv_reserve finds out for a step (make_kv_step); cu_new, cu_all, slots,
    positions, runs and all_slots are its int32 tensors."""
    _fields_ = [("max_new", ctypes.c_int32), ("max_all", ctypes.c_int32), ("_cu_new", ctypes.c_void_p),
                ("_cu_all", ctypes.c_void_p), ("_slots", ctypes.c_void_p), ("_positions", ctypes.c_void_p),
                ("_runs", ctypes.c_void_p), ("_all_slots", ctypes.c_void_p)]


class Packed(ctypes.Structure):
    """A batch of packed sequences (make_packed); keeps its tensors alive."""
    _fields_ = [("batch", ctypes.c_int32), ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("total_q", ctypes.c_int32), ("total_k", ctypes.c_int32),
                ("max_k", ctypes.c_int32), ("scale", ctypes.c_float), ("cu_q", ctypes.c_void_p),
                ("cu_k", ctypes.c_void_p)]


def lib():
    """The loaded libcrisp.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with dynamic_sparse_prefill_crisp_gb300.build.build()")
        _lib = load_library(LIB_PATH)
    return _lib


def load_library(path):
    """Loads a build of the library (e.g. the bounds-checking one) with the
    argument types declared; the module's calls keep using lib()."""
    L = ctypes.CDLL(path)
    vp, sz, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p
    P = ctypes.POINTER
    L.crisp_params_default.argtypes = [P(Params)]
    L.crisp_params_default.restype = None
    L.crisp_workspace_size.argtypes = [P(Shape), P(sz)]
    L.crisp_layer_workspace_size.argtypes = [P(Shape), P(sz)]
    L.crisp_workspace_init.argtypes = [vp, sz, st]
    L.crisp_proxy_map.argtypes = [P(Shape), vp, vp, vp, vp, sz, st]
    L.crisp_proxy_map_noalloc.argtypes = [P(Shape), vp, vp, vp, st]
    L.crisp_noalloc_read_status.argtypes = [st, P(ctypes.c_int)]
    L.crisp_block_masses.argtypes = [P(Shape), vp, vp, vp, vp, vp, sz, st]
    L.crisp_proxy_masses.argtypes = [P(Shape), vp, vp, vp, vp, vp, vp, sz, st]
    L.crisp_host_pipeline_create.argtypes = [P(vp)]
    L.crisp_host_pipeline_destroy.argtypes = [vp]
    L.crisp_prefill_layer_host.argtypes = [vp, P(Shape), P(Params)] + [vp] * 9 + [sz, st]
    L.crisp_route_cstruct.argtypes = [P(Shape), P(Params), vp, vp, vp, vp, vp, sz, st]
    L.crisp_route_cstruct_masses.argtypes = [P(Shape), P(Params), vp, vp, vp, vp, vp, vp, sz, st]
    L.crisp_route_jsd.argtypes = [P(Shape), P(Params), vp, vp, vp, vp, vp, sz, st]
    L.crisp_wait_selftest.argtypes = [vp, sz, ctypes.c_int64, st]
    L.crisp_select_vs.argtypes = [P(Shape), P(Params), vp, vp, vp, vp, vp, vp, vp, sz, st]
    L.crisp_select_vs_masses.argtypes = [P(Shape), P(Params), vp, vp, vp, vp, vp, vp, sz, st]
    L.crisp_pe_pool.argtypes = [P(Shape), vp, vp, vp, vp, vp, sz, st]
    L.crisp_select_pe.argtypes = [P(Shape), P(Params), vp, vp, vp, vp, sz, st]
    L.crisp_build_mask.argtypes = [P(Shape), vp, vp, vp, vp, vp, vp, vp, vp, sz, st]
    L.crisp_sparse_prefill.argtypes = [P(Shape), vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, st]
    L.crisp_sparse_prefill_mask.argtypes = [P(Shape), vp, vp, vp, vp, vp, vp, vp, sz, st]
    L.crisp_dense_prefill.argtypes = [P(Shape), vp, vp, vp, vp, vp, sz, st]
    L.crisp_layer_views_get.argtypes = [P(Shape), vp, P(LayerViews)]
    L.crisp_prefill_layer.argtypes = [P(Shape), P(Params), vp, vp, vp, vp, vp, sz, st]
    i32 = ctypes.c_int32
    L.crisp_kv_append_workspace_size.argtypes = [P(KVCache), P(sz)]
    L.crisp_decode_workspace_size.argtypes = [P(KVCache), i32, i32, i32, P(sz)]
    L.crisp_kv_evict_workspace_size.argtypes = [P(KVCache), i32, P(sz)]
    L.crisp_kv_append.argtypes = [P(KVCache), P(Tokens), P(Tokens), i32, vp, vp, sz, st]
    L.crisp_decode_attention.argtypes = [P(KVCache), i32, i32, ctypes.c_float, P(Tokens), P(Tokens), vp, vp, vp, sz,
                                         st]
    L.crisp_kv_evict.argtypes = [P(KVCache), P(KVCache), vp, i32, i32, i32, vp, vp, vp, sz, st]
    # (structures as untyped pointers: addresses, and crisp_tokens as packed bytes)
    L.crisp_kv_reserve.argtypes = [vp] * 8 + [sz, st]
    L.crisp_kv_append_packed.argtypes = [vp, vp, vp, vp, vp, sz, st]
    L.crisp_kv_gather.argtypes = [vp, vp, i32, vp, vp, vp, vp, sz, st]
    L.crisp_packed_workspace_size.argtypes = [P(Packed), P(sz)]
    L.crisp_packed_prefill.argtypes = [vp, vp, vp, vp, vp, vp, sz, st]
    L.crisp_read_status.argtypes = [vp, st, P(ctypes.c_int)]
    L.crisp_status_string.argtypes = [ctypes.c_int]
    L.crisp_status_string.restype = ctypes.c_char_p
    for name in ("crisp_workspace_size", "crisp_layer_workspace_size", "crisp_workspace_init", "crisp_proxy_map",
                 "crisp_proxy_map_noalloc", "crisp_noalloc_read_status", "crisp_block_masses",
                 "crisp_proxy_masses", "crisp_route_cstruct", "crisp_route_cstruct_masses", "crisp_route_jsd",
                 "crisp_select_vs", "crisp_select_vs_masses", "crisp_pe_pool", "crisp_select_pe",
                 "crisp_build_mask", "crisp_sparse_prefill", "crisp_sparse_prefill_mask", "crisp_dense_prefill",
                 "crisp_layer_views_get", "crisp_prefill_layer", "crisp_read_status",
                 "crisp_host_pipeline_create", "crisp_host_pipeline_destroy", "crisp_prefill_layer_host",
                 "crisp_kv_append_workspace_size", "crisp_decode_workspace_size", "crisp_kv_evict_workspace_size",
                 "crisp_kv_append", "crisp_decode_attention", "crisp_kv_evict", "crisp_wait_selftest",
                 "crisp_kv_reserve", "crisp_kv_append_packed", "crisp_kv_gather", "crisp_packed_workspace_size",
                 "crisp_packed_prefill"):
        getattr(L, name).restype = ctypes.c_int
    return L


def status_string(status: int) -> str:
    return lib().crisp_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != 0:
        raise CrispError(rc, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr() if hasattr(t, "data_ptr") else int(t))


_current = None


def _cuda_state():
    """(current device index, its current stream's handle), without building a
    Stream object (3 us a call)."""
    global _current
    if _current is None:
        import torch
        torch.cuda.init()
        dev, raw = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream

        def _current():
            d = dev()
            return d, raw(d)
    return _current()


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(_cuda_state()[1])
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _nbytes(t):
    return t.numel() * t.element_size()


def make_shape(hq, hkv, n, q=None, k=None, out=None, scale=0.0) -> Shape:
    """Shape for [heads][tokens][128] tensors; strides are taken from the
    tensors when given (any layout with the 128 features contiguous)."""
    def strides(t, heads):
        if t is None:
            return n * D, D
        assert t.dim() == 3 and t.shape[0] == heads and t.shape[1] == n and t.shape[2] == D and t.stride(2) == 1
        return t.stride(0), t.stride(1)
    qs, ks, os_ = strides(q, hq), strides(k, hkv), strides(out, hq)
    return Shape(hq, hkv, D, n, B, qs[0], qs[1], ks[0], ks[1], os_[0], os_[1], scale)


def params_default(**overrides) -> Params:
    p = Params()
    lib().crisp_params_default(ctypes.byref(p))
    for key, val in overrides.items():
        if key in ("alpha", "tau", "gamma", "vs_gamma"):
            setattr(p, f"{key}_num", val[0])
            setattr(p, f"{key}_den", val[1])
        else:
            setattr(p, key, val)
    return p


def workspace_size(shape: Shape) -> int:
    n = ctypes.c_size_t()
    _check(lib().crisp_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "crisp_workspace_size")
    return n.value


def layer_workspace_size(shape: Shape) -> int:
    n = ctypes.c_size_t()
    _check(lib().crisp_layer_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "crisp_layer_workspace_size")
    return n.value


def workspace_init(ws, stream=None):
    _check(lib().crisp_workspace_init(_ptr(ws), _nbytes(ws), _stream(stream)), "crisp_workspace_init")


def proxy_map(shape, q, k, pmap, ws, stream=None):
    _check(lib().crisp_proxy_map(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(pmap), _ptr(ws), _nbytes(ws),
                                 _stream(stream)), "crisp_proxy_map")


def proxy_map_noalloc(shape, q, k, pmap, stream=None):
    """crisp_proxy_map with the library's static scratch instead of a workspace
    (for callers that cannot allocate device memory; see include/crisp.h)."""
    _check(lib().crisp_proxy_map_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(pmap), _stream(stream)),
           "crisp_proxy_map_noalloc")


def noalloc_read_status(stream=None) -> int:
    """The status word of proxy_map_noalloc's static scratch (syncs the stream)."""
    s = ctypes.c_int()
    _check(lib().crisp_noalloc_read_status(_stream(stream), ctypes.byref(s)), "crisp_noalloc_read_status")
    return s.value


def block_masses(shape, pmap, vmass, smass, rmass, ws, stream=None):
    _check(lib().crisp_block_masses(ctypes.byref(shape), _ptr(pmap), _ptr(vmass), _ptr(smass), _ptr(rmass), _ptr(ws),
                                    _nbytes(ws), _stream(stream)), "crisp_block_masses")


def proxy_masses(shape, q, k, vmass, smass, rmass, ws, stream=None):
    """Block masses of the proxy map straight from q and k (the map is not stored)."""
    _check(lib().crisp_proxy_masses(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(vmass), _ptr(smass), _ptr(rmass),
                                    _ptr(ws), _nbytes(ws), _stream(stream)), "crisp_proxy_masses")


def route_cstruct(shape, params, pmap, cstruct, total, route, ws, stream=None):
    """A2 from the proxy map (any sink / recency slice widths of params)."""
    _check(lib().crisp_route_cstruct(ctypes.byref(shape), ctypes.byref(params), _ptr(pmap), _ptr(cstruct),
                                     _ptr(total), _ptr(route), _ptr(ws), _nbytes(ws), _stream(stream)),
           "crisp_route_cstruct")


def route_cstruct_masses(shape, params, vmass, rmass, cstruct, total, route, ws, stream=None):
    """A2 from the block masses (both slices one block wide)."""
    _check(lib().crisp_route_cstruct_masses(ctypes.byref(shape), ctypes.byref(params), _ptr(vmass), _ptr(rmass),
                                            _ptr(cstruct), _ptr(total), _ptr(route), _ptr(ws), _nbytes(ws),
                                            _stream(stream)), "crisp_route_cstruct_masses")


def route_jsd(shape, params, vmass, pbar, jsd, route, ws, stream=None):
    """FlexPrefill's divergence routing (comparator); pbar must hold row nb-1 of every head."""
    _check(lib().crisp_route_jsd(ctypes.byref(shape), ctypes.byref(params), _ptr(vmass), _ptr(pbar), _ptr(jsd),
                                 _ptr(route), _ptr(ws), _nbytes(ws), _stream(stream)), "crisp_route_jsd")


def select_vs(shape, params, pmap, route, vmass, smass, vbits, sbits, ws, stream=None):
    """A4 from the proxy map (writes the block masses too)."""
    _check(lib().crisp_select_vs(ctypes.byref(shape), ctypes.byref(params), _ptr(pmap), _ptr(route), _ptr(vmass),
                                 _ptr(smass), _ptr(vbits), _ptr(sbits), _ptr(ws), _nbytes(ws), _stream(stream)),
           "crisp_select_vs")


def select_vs_masses(shape, params, vmass, smass, route, vbits, sbits, ws, stream=None):
    """A4 from the block masses."""
    _check(lib().crisp_select_vs_masses(ctypes.byref(shape), ctypes.byref(params), _ptr(vmass), _ptr(smass),
                                        _ptr(route), _ptr(vbits), _ptr(sbits), _ptr(ws), _nbytes(ws),
                                        _stream(stream)), "crisp_select_vs_masses")


def pe_pool(shape, q, k, route, pbar, ws, stream=None):
    """A5: the pooled estimate of the PE heads (route[h] == 0)."""
    _check(lib().crisp_pe_pool(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(route), _ptr(pbar), _ptr(ws), _nbytes(ws),
                               _stream(stream)), "crisp_pe_pool")


def select_pe(shape, params, pbar, route, pebits, ws, stream=None):
    _check(lib().crisp_select_pe(ctypes.byref(shape), ctypes.byref(params), _ptr(pbar), _ptr(route), _ptr(pebits),
                                 _ptr(ws), _nbytes(ws), _stream(stream)), "crisp_select_pe")


def build_mask(shape, route, vbits, sbits, pebits, rowbits, counts, order, ws, stream=None):
    _check(lib().crisp_build_mask(ctypes.byref(shape), _ptr(route), _ptr(vbits), _ptr(sbits), _ptr(pebits),
                                  _ptr(rowbits), _ptr(counts), _ptr(order), _ptr(ws), _nbytes(ws), _stream(stream)),
           "crisp_build_mask")


def sparse_prefill(shape, q, k, v, route, vbits, sbits, pebits, out, ws, stream=None):
    """A8 from the index sets (the mask and schedule are built in ws)."""
    _check(lib().crisp_sparse_prefill(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(route), _ptr(vbits),
                                      _ptr(sbits), _ptr(pebits), _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream)),
           "crisp_sparse_prefill")


def sparse_prefill_mask(shape, q, k, v, rowbits, order, out, ws, stream=None):
    """A8 over a block mask; order: the schedule from build_mask, or None (the same kv-group-major order)."""
    _check(lib().crisp_sparse_prefill_mask(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(rowbits),
                                           _ptr(order), _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream)),
           "crisp_sparse_prefill_mask")


def dense_prefill(shape, q, k, v, out, ws, stream=None):
    _check(lib().crisp_dense_prefill(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(ws),
                                     _nbytes(ws), _stream(stream)), "crisp_dense_prefill")


def layer_views(shape, ws) -> dict:
    v = LayerViews()
    _check(lib().crisp_layer_views_get(ctypes.byref(shape), _ptr(ws), ctypes.byref(v)), "crisp_layer_views_get")
    return {name: getattr(v, name) for name, _ in LayerViews._fields_}


def prefill_layer(shape, params, q, k, v, out, ws, stream=None):
    _check(lib().crisp_prefill_layer(ctypes.byref(shape), ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                     _ptr(ws), _nbytes(ws), _stream(stream)), "crisp_prefill_layer")


class HostPipeline:
    """Streams and events of crisp_prefill_layer_host (on the current device)."""

    def __init__(self):
        self._h = ctypes.c_void_p()
        _check(lib().crisp_host_pipeline_create(ctypes.byref(self._h)), "crisp_host_pipeline_create")

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            _check(lib().crisp_host_pipeline_destroy(self._h), "crisp_host_pipeline_destroy")
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def prefill_layer_host(pipeline, shape, params, q_host, k_host, v_host, out_host, q, k, v, out, ws, stream=None):
    """crisp_prefill_layer from host buffers (pinned torch CPU tensors), copies
    overlapped with compute; q, k, v, out are the device staging buffers."""
    _check(lib().crisp_prefill_layer_host(pipeline.handle, ctypes.byref(shape), ctypes.byref(params), _ptr(q_host),
                                          _ptr(k_host), _ptr(v_host), _ptr(out_host), _ptr(q), _ptr(k), _ptr(v),
                                          _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream)),
           "crisp_prefill_layer_host")


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def make_kv_cache(k, v, k_scale, v_scale, table, lens) -> KVCache:
    """The cache that these CUDA tensors hold: k, v float8_e4m3fn (or uint8
    codes) [num_pages][hkv][128][128] of the same strides, each head's page
    contiguous; k_scale, v_scale fp32 [num_pages][hkv]; table int32
    [batch][max_pages] of page ids; lens int32 [batch] of tokens held. The
    structure keeps the tensors alive; their contents may change between calls."""
    import torch
    codes = (torch.float8_e4m3fn, torch.uint8)
    _need(k.dim() == 4 and k.shape == v.shape and k.shape[2:] == (B, D) and k.dtype in codes and v.dtype in codes,
          "make_kv_cache: k and v must be 8-bit [num_pages][hkv][128][128]")
    _need(k.stride() == v.stride() and k.stride()[2:] == (D, 1),
          "make_kv_cache: k and v must share their strides and hold each head's page contiguously")
    num, hkv = k.shape[:2]
    for s in (k_scale, v_scale):
        _need(s.shape == (num, hkv) and s.dtype == torch.float32 and s.is_contiguous(),
              "make_kv_cache: the scales must be contiguous fp32 [num_pages][hkv]")
    _need(table.dim() == 2 and table.dtype == torch.int32 and table.is_contiguous(),
          "make_kv_cache: table must be contiguous int32 [batch][max_pages]")
    _need(lens.shape == table.shape[:1] and lens.dtype == torch.int32 and lens.is_contiguous(),
          "make_kv_cache: lens must be contiguous int32 [batch]")
    keep = (k, v, k_scale, v_scale, table, lens)
    _need(all(t.device == k.device for t in keep), "make_kv_cache: the tensors must be on one device")
    c = KVCache(table.shape[0], hkv, D, B, num, table.shape[1], k.stride(0), k.stride(1), k.data_ptr(), v.data_ptr(),
                k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(), lens.data_ptr())
    c.tensors, c.device_index, c.token_dtype = keep, k.get_device(), torch.bfloat16
    c.sizes = table.shape[0], hkv, num, table.data_ptr(), torch.bfloat16, torch.int32
    return c


def _tokens(what, t, cache, heads, tokens):
    if t.shape != (cache.batch, heads, tokens, D) or t.dtype != cache.token_dtype:
        raise ValueError(f"{what} must be bf16 [batch][heads][tokens][128] = "
                         f"{(cache.batch, heads, tokens, D)}: {t.dtype} {tuple(t.shape)}")
    b, h, i, d = t.stride()
    if d != 1:
        raise ValueError(f"{what}: the 128 features must be contiguous")
    return Tokens(t.data_ptr(), b, h, i)


def _rows(what, t, cache, dtype):
    """The address of contiguous [batch][hkv][128 * max_pages] (None: a null pointer)."""
    if t is None:
        return None
    if t.shape != (cache.batch, cache.hkv, cache.max_pages * B) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {dtype} [batch][hkv][128 * max_pages]")
    return t.data_ptr()


def _on_device(cache, stream, *tensors):
    """The handle of the stream to run on (None: the current device's current
    one). Everything has to be on the current device."""
    want = cache.device_index
    if want >= 0:
        dev, handle = _cuda_state()
        if dev == want:
            for t in tensors:
                if t is not None and t.get_device() != want:
                    break
            else:
                if stream is None:
                    return handle
                return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    raise ValueError("the cache and every tensor of the call must be on the current CUDA device")


def kv_append_workspace_size(cache: KVCache) -> int:
    n = ctypes.c_size_t()
    _check(lib().crisp_kv_append_workspace_size(ctypes.byref(cache), ctypes.byref(n)),
           "crisp_kv_append_workspace_size")
    return n.value


def decode_workspace_size(cache: KVCache, hq: int, q_len: int = 1, weights: bool = False) -> int:
    n = ctypes.c_size_t()
    _check(lib().crisp_decode_workspace_size(ctypes.byref(cache), hq, q_len, int(weights), ctypes.byref(n)),
           "crisp_decode_workspace_size")
    return n.value


def kv_evict_workspace_size(cache: KVCache, keep: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().crisp_kv_evict_workspace_size(ctypes.byref(cache), keep, ctypes.byref(n)),
           "crisp_kv_evict_workspace_size")
    return n.value


def kv_append(cache, k_new, v_new, ws, new_lens=None, stream=None):
    """Writes bf16 [batch][hkv][n_new][128] tokens into the cache, the last of
    sequence b at position lens[b] - 1 (advance lens first); new_lens: int32
    [batch], how many of the n_new tokens each sequence has (default: all)."""
    _need(k_new.dim() == 4, "kv_append: k_new must be [batch][hkv][n_new][128]")
    n_new = k_new.shape[2]
    kt = _tokens("kv_append: k_new", k_new, cache, cache.hkv, n_new)
    vt = _tokens("kv_append: v_new", v_new, cache, cache.hkv, n_new)
    if new_lens is not None:
        lens = cache.tensors[5]
        _need(new_lens.shape == lens.shape and new_lens.dtype == lens.dtype and new_lens.is_contiguous(),
              "kv_append: new_lens must be contiguous int32 [batch]")
    st = _on_device(cache, stream, k_new, v_new, ws, new_lens)
    _check(lib().crisp_kv_append(ctypes.byref(cache), ctypes.byref(kt), ctypes.byref(vt), n_new,
                                 None if new_lens is None else new_lens.data_ptr(), ws.data_ptr(), _nbytes(ws), st),
           "crisp_kv_append")


def decode_attention(cache, q, out, ws, weights_in=None, weights_out=None, scale=0.0, stream=None):
    """Attention of the last q_len tokens of every sequence over the cache: q,
    out bf16 [batch][hq][q_len][128]. With weights_out (fp32 [batch][hkv][128 *
    max_pages]) each key's weight, summed over the kv head's rows, is added to
    weights_in's (None: zeros; may be the same tensor). Entries past a length are
    left alone: weights that accumulate start as zeros throughout."""
    _need(q.dim() == 4, "decode_attention: q must be [batch][hq][q_len][128]")
    _, hq, q_len, _ = q.shape
    qt = _tokens("decode_attention: q", q, cache, hq, q_len)
    ot = _tokens("decode_attention: out", out, cache, hq, q_len)
    f32 = cache.tensors[2].dtype
    w_in = _rows("decode_attention: weights_in", weights_in, cache, f32)
    w_out = _rows("decode_attention: weights_out", weights_out, cache, f32)
    st = _on_device(cache, stream, q, out, ws, weights_in, weights_out)
    _check(lib().crisp_decode_attention(ctypes.byref(cache), hq, q_len, scale, ctypes.byref(qt), ctypes.byref(ot),
                                        w_in, w_out, ws.data_ptr(), _nbytes(ws), st), "crisp_decode_attention")


def kv_evict(cache, new_cache, weights, ws, keep, sink=0, recent=0, new_weights=None, kept=None, stream=None):
    """Copies at most `keep` tokens of every sequence and kv head -- the first
    `sink`, the last `recent`, and those of largest weight -- into new_cache's
    pages, in their order, and sets its lens. new_weights (fp32) and kept (int32,
    old positions) are [batch][hkv][128 * new_cache.max_pages], written below the
    new lengths only: new_weights that decoding goes on with start as zeros."""
    f32, i32 = cache.tensors[2].dtype, cache.tensors[5].dtype
    w = _rows("kv_evict: weights", weights, cache, f32)
    new_w = _rows("kv_evict: new_weights", new_weights, new_cache, f32)
    pos = _rows("kv_evict: kept", kept, new_cache, i32)
    st = _on_device(cache, stream, new_cache.tensors[0], weights, ws, new_weights, kept)
    _check(lib().crisp_kv_evict(ctypes.byref(cache), ctypes.byref(new_cache), w, keep, sink, recent, new_w, pos,
                                ws.data_ptr(), _nbytes(ws), st), "crisp_kv_evict")


# The calls on packed sequences come once a layer and step, some of them to run for
# a few microseconds: their checks read each tensor once, and crisp_tokens is packed
# (a quarter of the time of a ctypes structure).
_ELSEWHERE = "the cache, the step or batch, and every tensor of the call must be on the current CUDA device"
_pack, _at = struct.Struct("=4q").pack, ctypes.addressof
_dev = _raw = None


def _here(owner, stream):
    """(current device, handle of the stream to run on); the owner has to be there."""
    global _dev, _raw
    want = owner.device_index
    if want >= 0:
        if _raw is None:
            _cuda_state()
            import torch
            _dev, _raw = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        dev = _dev()
        if dev == want:
            if stream is None:
                return dev, _raw(dev)
            return dev, stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return -1, None  # (a tensor's own fault is told first)


def _packed_tokens(what, t, rows, heads, dtype, dev):
    """The crisp_tokens of packed [rows][heads][128] bf16."""
    if t.dtype is not dtype or t.shape != (rows, heads, D):
        raise ValueError(f"{what} must be bf16 [tokens][heads][128] = {(rows, heads, D)}: {t.dtype} {tuple(t.shape)}")
    i, h, e = t.stride()
    if e != 1:
        raise ValueError(f"{what}: the 128 features must be contiguous")
    if dev < 0 or t.get_device() != dev:
        raise ValueError(_ELSEWHERE)
    return _pack(t.data_ptr(), 0, h, i)


def _ints(what, t, n, dtype, dev):
    """The address of contiguous int32 [n] (None: a null pointer)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous int32 [{n}]")
    if dev < 0 or t.get_device() != dev:
        raise ValueError(_ELSEWHERE)
    return t.data_ptr()


def _space(ws, dev):
    """The address of a workspace."""
    if dev < 0 or ws.get_device() != dev:
        raise ValueError(_ELSEWHERE)
    return ws.data_ptr()


def make_kv_step(cache, max_new, max_all=0) -> KVStep:
    """Room for a step's maps (kv_reserve): at most max_new new tokens of the
    cache's batch, and the slots of all its tokens where max_all is not 0 (the
    most there can be). Allocates int32 tensors on the cache's device."""
    import torch
    _need(0 <= max_new <= 1 << 24 and 0 <= max_all <= 1 << 24, "make_kv_step: max_new and max_all must be 0 .. 2^24")
    runs = min(max_new, max_new // B + 2 * cache.batch)
    sizes = dict(cu_new=cache.batch + 1, cu_all=cache.batch + 1, slots=max_new, positions=max_new, runs=runs + 1,
                 all_slots=max_all)
    s = KVStep(max_new, max_all)
    for name, n in sizes.items():
        t = torch.zeros(n, dtype=torch.int32, device=cache.tensors[5].device)
        setattr(s, name, t)
        setattr(s, "_" + name, t.data_ptr() if n else None)
    s.batch, s.room, s.device_index = cache.batch, max_new, cache.device_index
    return s


def _step_of(what, step, sizes, cache):
    if step.batch != sizes[0] or step.device_index != cache.device_index:
        raise ValueError(f"{what}: the step was made for another batch or device")


def kv_reserve(cache, free_pages, num_free, step, ws, keep=None, new_lens=None, stream=None):
    """Hands out pages for a step: sequence b keeps its first min(keep[b], lens[b])
    tokens (None: all of them) and gets new_lens[b] more (None: none). Pages no
    longer needed go back to the stack of free page ids (free_pages int32
    [num_pages], num_free int32 [1]), missing ones come from it; the cache's table
    and lens are brought up to date and `step` is filled (cu_new, cu_all, slots,
    positions, runs, all_slots). If too few pages are free, or the step or a
    sequence has no room, the status word says so and the step takes no tokens:
    the packed calls behind it do nothing, but decode_attention goes by lens, which
    stay as they were. ws: kv_append_workspace_size bytes."""
    sizes = cache.sizes
    batch, _, pages, table, _, i32 = sizes
    _step_of("kv_reserve", step, sizes, cache)
    dev, st = _here(cache, stream)
    free = _ints("kv_reserve: free_pages", free_pages, pages, i32, dev)
    num = _ints("kv_reserve: num_free", num_free, 1, i32, dev)
    kept = _ints("kv_reserve: keep", keep, batch, i32, dev)
    new = _ints("kv_reserve: new_lens", new_lens, batch, i32, dev)
    rc = lib().crisp_kv_reserve(_at(cache), table, free, num, kept, new, _at(step), _space(ws, dev), ws.nbytes, st)
    if rc:
        _check(rc, "crisp_kv_reserve")


def kv_append_packed(cache, step, k_new, v_new, ws, stream=None):
    """Writes a step's new tokens into the cache: bf16 [max_new][hkv][128], token i
    at slots[i] (rows past the step's total are not read)."""
    sizes = cache.sizes
    _, hkv, _, _, bf16, _ = sizes
    _step_of("kv_append_packed", step, sizes, cache)
    dev, st = _here(cache, stream)
    k = _packed_tokens("kv_append_packed: k_new", k_new, step.room, hkv, bf16, dev)
    v = _packed_tokens("kv_append_packed: v_new", v_new, step.room, hkv, bf16, dev)
    rc = lib().crisp_kv_append_packed(_at(cache), _at(step), k, v, _space(ws, dev), ws.nbytes, st)
    if rc:
        _check(rc, "crisp_kv_append_packed")


def kv_gather(cache, slots, k_out, v_out, ws, count=None, stream=None):
    """Reads cached tokens back: row i of k_out and v_out (bf16 [n][hkv][128]) from
    slot slots[i] (int32 [n], e.g. a step's all_slots), exactly; count: int32 [1],
    how many of the n rows there are (e.g. step.cu_all[-1:]; None: all). Rows of
    negative slots are left alone."""
    _, hkv, _, _, bf16, i32 = cache.sizes
    dev, st = _here(cache, stream)
    n = slots.shape[0] if slots.dim() == 1 else -1
    at = _ints("kv_gather: slots", slots, n, i32, dev)
    num = _ints("kv_gather: count", count, 1, i32, dev)
    k = _packed_tokens("kv_gather: k_out", k_out, n, hkv, bf16, dev)
    v = _packed_tokens("kv_gather: v_out", v_out, n, hkv, bf16, dev)
    rc = lib().crisp_kv_gather(_at(cache), at, n, num, k, v, _space(ws, dev), ws.nbytes, st)
    if rc:
        _check(rc, "crisp_kv_gather")


def make_packed(hq, hkv, cu_q, cu_k, total_q, total_k, max_k=None, scale=0.0) -> Packed:
    """A batch of packed sequences: sequence b has the query rows [cu_q[b], cu_q[b +
    1]) of total_q and the key rows [cu_k[b], cu_k[b + 1]) of total_k (int32 CUDA
    tensors of batch + 1 running sums; the same tensor for whole prompts). max_k:
    about the longest sequence's keys (None: total_k), for how work is split, no
    limit; leaving it out where total_k is the room of many sequences costs
    workspace (packed_workspace_size) and time. The structure keeps the tensors alive; their contents may change
    between calls."""
    import torch
    n = cu_q.shape[0] if cu_q.dim() == 1 else 0
    _need(n >= 1, "make_packed: cu_q must be int32 [batch + 1]")
    for what, t in (("cu_q", cu_q), ("cu_k", cu_k)):
        _need(t.dtype is torch.int32 and t.shape == (n,) and t.is_contiguous(),
              f"make_packed: {what} must be contiguous int32 [{n}]")
    _need(cu_q.device == cu_k.device, "make_packed: the tensors must be on one device")
    _need(max_k is None or max_k >= 0, "make_packed: max_k must not be negative")
    p = Packed(n - 1, hq, hkv, D, total_q, total_k, max_k or 0, scale, cu_q.data_ptr(), cu_k.data_ptr())
    p.tensors, p.device_index = (cu_q, cu_k), cu_q.get_device()
    p.sizes = total_q, total_k, hq, hkv, torch.bfloat16
    return p


def packed_workspace_size(packed: Packed) -> int:
    n = ctypes.c_size_t()
    _check(lib().crisp_packed_workspace_size(ctypes.byref(packed), ctypes.byref(n)), "crisp_packed_workspace_size")
    return n.value


def packed_prefill(packed, q, k, v, out, ws, stream=None):
    """Causal softmax attention of every sequence of a packed batch: q, out bf16
    [total_q][hq][128], k, v bf16 [total_k][hkv][128], features contiguous (any
    token and head strides that are multiples of 8 elements). Query i of a
    sequence of nq queries and nk keys sees its keys j <= nk - nq + i; rows that
    see none become zeros, rows behind the last sequence are left alone. out shares
    no element with the inputs."""
    total_q, total_k, hq, hkv, bf16 = packed.sizes
    dev, st = _here(packed, stream)
    a = _packed_tokens("packed_prefill: q", q, total_q, hq, bf16, dev)
    b = _packed_tokens("packed_prefill: k", k, total_k, hkv, bf16, dev)
    c = _packed_tokens("packed_prefill: v", v, total_k, hkv, bf16, dev)
    d = _packed_tokens("packed_prefill: out", out, total_q, hq, bf16, dev)
    rc = lib().crisp_packed_prefill(_at(packed), a, b, c, d, _space(ws, dev), ws.nbytes, st)
    if rc:
        _check(rc, "crisp_packed_prefill")


def wait_selftest(ws, limit_ns, stream=None):
    """Launches the bounded-wait self-test (a wait that nothing ends)."""
    _check(lib().crisp_wait_selftest(_ptr(ws), _nbytes(ws), int(limit_ns), _stream(stream)), "crisp_wait_selftest")


def read_status(ws, stream=None) -> int:
    s = ctypes.c_int()
    _check(lib().crisp_read_status(_ptr(ws), _stream(stream), ctypes.byref(s)), "crisp_read_status")
    return s.value


def attention(q, k, v, params=None, scale=0.0, stream=None, check=True):
    """One CRISP sparse-prefill layer on torch tensors: q [hq][n][128], k and v
    [hkv][n][128], bf16, on the current CUDA device, features contiguous (any
    head and token strides that are multiples of 8 elements). Allocates the
    output (contiguous [hq][n][128] bf16) and a layer workspace with torch,
    runs crisp_prefill_layer on `stream` and returns the output. params: a
    Params (default: the paper's universal configuration); scale 0 means
    1/sqrt(128). With check=True the stream is synchronised and a device-side
    error raises CrispError."""
    import torch
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape:
        raise ValueError("attention: q must be [hq][n][128], k and v [hkv][n][128]")
    hq, n, _ = q.shape
    hkv = k.shape[0]
    out = torch.empty((hq, n, D), dtype=torch.bfloat16, device=q.device)
    shape = make_shape(hq, hkv, n, q, k, out, scale=scale)
    if k.stride() != v.stride():
        raise ValueError("attention: k and v must share their strides")
    ws = torch.empty(max(layer_workspace_size(shape), 256), dtype=torch.uint8, device=q.device)
    workspace_init(ws, stream)
    prefill_layer(shape, params if params is not None else params_default(), q, k, v, out, ws, stream)
    if check:
        st = read_status(ws, stream)
        if st != 0:
            raise CrispError(st, "crisp_prefill_layer (device)")
    return out
