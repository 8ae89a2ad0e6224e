"""The cache calls' refusals: bad arguments are answered on the host, before
any launch and without a GPU."""
import ctypes

import pytest
import torch

import dynamic_sparse_prefill_crisp_gb300 as crisp
from dynamic_sparse_prefill_crisp_gb300 import build as crisp_build

OK, INVALID, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
vp = ctypes.c_void_p
PAGE = 128 * 128


@pytest.fixture(scope="module")
def L():
    crisp_build.build()
    return crisp.lib()


def cache(**over):
    c = crisp.KVCache(batch=3, hkv=2, head_dim=128, block=128, num_pages=40, max_pages=10, page_stride=2 * PAGE,
                      head_stride=PAGE, k=256, v=256, k_scale=256, v_scale=256, table=256, lens=256)
    for key, val in over.items():
        setattr(c, key, val)
    return c


def tokens(data=256, b=4096, h=128, t=1024):
    return crisp.Tokens(data, b, h, t)


def append(L, c, k=None, v=None, n=4, new_lens=None, ws=256, nbytes=1 << 20):
    k, v = k or tokens(), v or tokens()
    return L.crisp_kv_append(ctypes.byref(c), ctypes.byref(k), ctypes.byref(v), n, new_lens, vp(ws), nbytes, None)


def decode(L, c, hq=8, q_len=2, scale=0.0, q=None, out=None, w_in=None, w_out=None, ws=256, nbytes=1 << 30):
    q, out = q or tokens(), out or tokens()
    return L.crisp_decode_attention(ctypes.byref(c), hq, q_len, scale, ctypes.byref(q), ctypes.byref(out), w_in, w_out,
                                    vp(ws), nbytes, None)


def evict(L, src, dst, weights=vp(512), keep=200, sink=10, recent=20, new_w=None, kept=None, ws=256, nbytes=1 << 20):
    return L.crisp_kv_evict(ctypes.byref(src), ctypes.byref(dst), weights, keep, sink, recent, new_w, kept, vp(ws),
                            nbytes, None)


def other(**over):
    return cache(**{"table": 512, "lens": 512, "max_pages": 2, **over})


BAD_CACHES = [
    ("head_dim", 64, SHAPE), ("block", 64, SHAPE), ("batch", -1, SHAPE), ("batch", 1025, SHAPE), ("hkv", 0, SHAPE),
    ("hkv", 4097, SHAPE), ("num_pages", 0, SHAPE), ("max_pages", 0, SHAPE), ("max_pages", 8193, SHAPE),
    ("page_stride", 0, ALIGN), ("page_stride", 2 * PAGE + 8, ALIGN), ("page_stride", PAGE - 16, SHAPE),
    ("head_stride", -16, ALIGN), ("head_stride", PAGE - 16, SHAPE), ("k", None, INVALID), ("v", None, INVALID),
    ("k_scale", None, INVALID), ("v_scale", None, INVALID), ("table", None, INVALID), ("lens", None, INVALID),
    ("k", 264, ALIGN), ("v", 257, ALIGN), ("k_scale", 258, ALIGN), ("v_scale", 257, ALIGN), ("table", 258, ALIGN),
    ("lens", 257, ALIGN),
]


@pytest.mark.parametrize("field,value,code", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(L, field, value, code):
    c = cache(**{field: value})
    n = ctypes.c_size_t()
    assert L.crisp_kv_append_workspace_size(ctypes.byref(c), ctypes.byref(n)) == code
    assert L.crisp_decode_workspace_size(ctypes.byref(c), 8, 1, 0, ctypes.byref(n)) == code
    assert L.crisp_kv_evict_workspace_size(ctypes.byref(c), 10, ctypes.byref(n)) == code
    assert append(L, c) == code
    assert decode(L, c) == code
    assert evict(L, c, other()) == code
    assert evict(L, cache(), other(**{field: value})) == code


def test_null_structures(L):
    n = ctypes.c_size_t()
    assert L.crisp_kv_append_workspace_size(None, ctypes.byref(n)) == INVALID
    for f in (lambda c, out: L.crisp_kv_append_workspace_size(c, out),
              lambda c, out: L.crisp_decode_workspace_size(c, 8, 1, 1, out),
              lambda c, out: L.crisp_kv_evict_workspace_size(c, 5, out)):
        assert f(ctypes.byref(cache()), None) == INVALID
        assert f(ctypes.byref(cache()), ctypes.byref(n)) == OK and n.value % 256 == 0 and n.value >= 256
    t = tokens()
    assert L.crisp_kv_append(ctypes.byref(cache()), None, ctypes.byref(t), 1, None, vp(256), 1 << 20, None) == INVALID
    assert L.crisp_kv_append(ctypes.byref(cache()), ctypes.byref(t), None, 1, None, vp(256), 1 << 20, None) == INVALID
    assert L.crisp_kv_evict(None, ctypes.byref(other()), vp(512), 5, 0, 0, None, None, vp(256), 1 << 20,
                            None) == INVALID
    assert L.crisp_kv_evict(ctypes.byref(cache()), None, vp(512), 5, 0, 0, None, None, vp(256), 1 << 20,
                            None) == INVALID


def test_append_refusals(L):
    c = cache()
    assert append(L, c, n=-1) == SHAPE and append(L, c, n=1281) == SHAPE
    assert append(L, c, k=tokens(data=None)) == INVALID and append(L, c, v=tokens(data=None)) == INVALID
    assert append(L, c, k=tokens(data=264)) == ALIGN and append(L, c, v=tokens(t=1028)) == ALIGN
    assert append(L, c, k=tokens(h=0)) == ALIGN and append(L, c, k=tokens(b=64)) == SHAPE
    assert append(L, c, new_lens=vp(258)) == ALIGN
    assert append(L, c, ws=None) == WORKSPACE and append(L, c, ws=272) == ALIGN and append(L, c, nbytes=255) == WORKSPACE
    # nothing to write: no buffer is looked at
    assert append(L, c, n=0, k=tokens(data=None), ws=None) == OK
    assert append(L, cache(batch=0, k=None), k=tokens(data=None), ws=None) == OK
    # the stride of an axis of one entry is not used
    assert append(L, cache(batch=1, hkv=1), k=tokens(b=1, h=0, t=7), n=1, ws=None) == WORKSPACE


def test_decode_refusals(L):
    c = cache()
    n = ctypes.c_size_t()
    for hq, q_len in ((0, 1), (7, 1), (4098, 1), (8, 0), (8, 17), (2 * 128, 16)):
        assert decode(L, c, hq=hq, q_len=q_len) == SHAPE
        assert L.crisp_decode_workspace_size(ctypes.byref(c), hq, q_len, 0, ctypes.byref(n)) == SHAPE
    assert decode(L, cache(batch=1024, hkv=256, max_pages=8192), hq=256) == SHAPE  # more tiles than are counted
    assert decode(L, c, scale=-1.0) == INVALID and decode(L, c, scale=float("nan")) == INVALID
    assert decode(L, c, scale=float("inf")) == INVALID
    assert decode(L, c, q=tokens(data=None)) == INVALID and decode(L, c, out=tokens(data=None)) == INVALID
    assert decode(L, c, q=tokens(data=248)) == ALIGN and decode(L, c, out=tokens(h=100)) == ALIGN
    assert decode(L, c, out=tokens(t=64)) == SHAPE
    assert decode(L, c, w_in=vp(256)) == INVALID
    assert decode(L, c, w_in=vp(264), w_out=vp(256)) == ALIGN and decode(L, c, w_out=vp(260)) == ALIGN
    assert decode(L, c, ws=None) == WORKSPACE and decode(L, c, ws=128) == ALIGN
    sizes = []
    for w in (0, 1):
        assert L.crisp_decode_workspace_size(ctypes.byref(c), 8, 2, w, ctypes.byref(n)) == OK
        sizes.append(n.value)
    # scores of every row and key: 3 sequences x 2 heads x 8 rows x 1280 keys
    assert sizes[1] - sizes[0] >= 3 * 2 * 8 * 1280 * 4
    assert decode(L, c, nbytes=sizes[0] - 1) == WORKSPACE
    assert decode(L, c, w_out=vp(256), nbytes=sizes[1] - 1) == WORKSPACE
    assert decode(L, cache(batch=0), q=tokens(data=None), ws=None) == OK


def test_evict_refusals(L):
    c, d = cache(), other()
    assert evict(L, c, other(batch=2)) == SHAPE and evict(L, c, other(hkv=1)) == SHAPE
    for keep, sink, recent in ((0, 0, 0), (257, 0, 0), (200, -1, 0), (200, 0, -1), (200, 150, 51),
                               (200, 2 ** 31 - 1, 2 ** 31 - 1)):
        assert evict(L, c, d, keep=keep, sink=sink, recent=recent) == INVALID
    assert evict(L, c, d, weights=None) == INVALID and evict(L, c, d, new_w=vp(512)) == INVALID
    assert evict(L, c, other(table=256)) == INVALID and evict(L, c, other(lens=256)) == INVALID
    # the same table is refused over any shared pool, and taken over pools of its own (here up to the workspace)
    apart = {"k": 768, "v": 768, "k_scale": 768, "v_scale": 768}
    for field in apart:
        assert evict(L, c, other(table=256, **{**apart, field: 256})) == INVALID
    assert evict(L, c, other(table=256, **apart), nbytes=0) == WORKSPACE
    assert evict(L, c, d, weights=vp(520)) == ALIGN and evict(L, c, d, new_w=vp(260)) == ALIGN
    assert evict(L, c, d, kept=vp(258)) == ALIGN
    n = ctypes.c_size_t()
    assert L.crisp_kv_evict_workspace_size(ctypes.byref(c), 200, ctypes.byref(n)) == OK
    assert evict(L, c, d, nbytes=n.value - 1) == WORKSPACE and evict(L, c, d, ws=None) == WORKSPACE
    assert L.crisp_kv_evict_workspace_size(ctypes.byref(c), 0, ctypes.byref(n)) == INVALID
    assert evict(L, cache(batch=0), other(batch=0), weights=None, ws=None) == OK


def make(**over):
    t = dict(k=torch.zeros((4, 2, 128, 128), dtype=torch.uint8), v=torch.zeros((4, 2, 128, 128), dtype=torch.uint8),
             k_scale=torch.ones((4, 2)), v_scale=torch.ones((4, 2)), table=torch.zeros((3, 2), dtype=torch.int32),
             lens=torch.zeros(3, dtype=torch.int32))
    t.update(over)
    return crisp.make_kv_cache(**t)


@pytest.mark.parametrize("over", [
    dict(k=torch.zeros((4, 2, 128, 64), dtype=torch.uint8)), dict(k=torch.zeros((4, 2, 128, 128))),
    dict(v=torch.zeros((5, 2, 128, 128), dtype=torch.uint8)),
    dict(v=torch.zeros((4, 2, 128, 128), dtype=torch.uint8).transpose(2, 3)),
    dict(v=torch.zeros((4, 4, 128, 128), dtype=torch.uint8)[:, ::2]),
    dict(k_scale=torch.ones((2, 4)).T), dict(v_scale=torch.ones((4, 2), dtype=torch.float64)),
    dict(table=torch.zeros((3, 2), dtype=torch.int64)), dict(table=torch.zeros((3, 4), dtype=torch.int32)[:, ::2]),
    dict(lens=torch.zeros(2, dtype=torch.int32)), dict(lens=torch.zeros(3, dtype=torch.int64))])
def test_make_kv_cache_refuses_other_tensors(over):
    with pytest.raises(ValueError):
        make(**over)


def test_make_kv_cache_takes_strided_pools():
    both = torch.zeros((4, 2, 3, 128, 128), dtype=torch.uint8)
    c = make(k=both[:, 0], v=both[:, 1], k_scale=torch.ones((4, 3)), v_scale=torch.ones((4, 3)))
    assert (c.page_stride, c.head_stride, c.num_pages, c.hkv) == (2 * 3 * PAGE, PAGE, 4, 3)
    assert (c.batch, c.max_pages) == (3, 2) and c.v - c.k == 3 * PAGE


def test_the_binding_checks_tensors_before_the_call():
    c = make()
    ws = torch.zeros(1024, dtype=torch.uint8)
    x = torch.zeros((3, 2, 5, 128), dtype=torch.bfloat16)
    w = torch.zeros((3, 2, 256))
    for bad in (x.float(), x[:2], x[:, :1], x[..., :64], x.transpose(2, 3)):
        with pytest.raises(ValueError):
            crisp.kv_append(c, bad, bad, ws)
    with pytest.raises(ValueError):
        crisp.kv_append(c, x, x[:, :, :4], ws)
    with pytest.raises(ValueError):
        crisp.kv_append(c, x, x, ws, new_lens=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        crisp.decode_attention(c, x, x[:, :, :4], ws)
    for bad in (w[:, :, :128], w.double(), w[:, :1]):
        with pytest.raises(ValueError):
            crisp.decode_attention(c, x, x, ws, bad, w)
        with pytest.raises(ValueError):
            crisp.kv_evict(c, make(), bad, ws, keep=5)
    with pytest.raises(ValueError):
        crisp.kv_evict(c, make(), w, ws, keep=5, kept=w)
    # everything in order but not on a GPU
    for call in (lambda: crisp.kv_append(c, x, x, ws), lambda: crisp.decode_attention(c, x, x, ws),
                 lambda: crisp.kv_evict(c, make(), w, ws, keep=5)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
