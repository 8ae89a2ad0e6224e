"""The packed calls' refusals: bad arguments are answered on the host, before any
launch and without a GPU."""
import ctypes

import pytest
import torch

import dynamic_sparse_prefill_crisp_gb300 as crisp
from dynamic_sparse_prefill_crisp_gb300 import build as crisp_build

OK, INVALID, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
vp, ref = ctypes.c_void_p, ctypes.byref
PAGE = 128 * 128


@pytest.fixture(scope="module")
def L():
    crisp_build.build()
    return crisp.lib()


def with_fields(x, over):
    for key, val in over.items():
        setattr(x, key, val)
    return x


def cache(**over):
    return with_fields(crisp.KVCache(batch=3, hkv=2, head_dim=128, block=128, num_pages=40, max_pages=10,
                                     page_stride=2 * PAGE, head_stride=PAGE, k=256, v=256, k_scale=256, v_scale=256,
                                     table=256, lens=512), over)


def step(**over):
    return with_fields(crisp.KVStep(300, 0, 1024, 1024, 1024, 1024, 1024, None), over)


def packed(**over):
    return with_fields(crisp.Packed(batch=3, hq=8, hkv=2, head_dim=128, total_q=100, total_k=200, max_k=0, scale=0.0,
                                    cu_q=256, cu_k=256), over)


def tokens(data=256, b=0, h=128, t=1024):
    return crisp.Tokens(data, b, h, t)


def reserve(L, c=None, s=None, table=256, free=768, num=768, keep=None, new=None, ws=256, nbytes=256):
    return L.crisp_kv_reserve(ref(c or cache()), vp(table), vp(free), vp(num), vp(keep), vp(new), ref(s or step()), vp(ws),
                              nbytes, None)


def append(L, c=None, s=None, k=None, v=None, ws=256, nbytes=256):
    return L.crisp_kv_append_packed(ref(c or cache()), ref(s or step()), ref(k or tokens()), ref(v or tokens()), vp(ws),
                                    nbytes, None)


def gather(L, c=None, slots=256, n=50, count=None, k=None, v=None, ws=256, nbytes=256):
    return L.crisp_kv_gather(ref(c or cache()), vp(slots), n, vp(count), ref(k or tokens()), ref(v or tokens()), vp(ws),
                             nbytes, None)


def prefill(L, p=None, q=None, k=None, v=None, out=None, ws=256, nbytes=1 << 30):
    return L.crisp_packed_prefill(ref(p or packed()), ref(q or tokens()), ref(k or tokens()), ref(v or tokens()),
                                  ref(out or tokens()), vp(ws), nbytes, None)


def test_every_call_refuses_a_bad_cache(L):
    for field, value, code in (("head_dim", 64, SHAPE), ("batch", 1025, SHAPE), ("hkv", 0, SHAPE), ("max_pages", 0, SHAPE),
                               ("page_stride", 8, ALIGN), ("k", None, INVALID), ("v", 264, ALIGN), ("table", None, INVALID),
                               ("lens", 258, ALIGN)):
        c = cache(**{field: value})
        assert reserve(L, c) == code and append(L, c) == code and gather(L, c) == code
    for f in (lambda: L.crisp_kv_reserve(None, vp(256), vp(256), vp(256), None, None, ref(step()), vp(256), 256, None),
              lambda: L.crisp_kv_reserve(ref(cache()), vp(256), vp(256), vp(256), None, None, None, vp(256), 256, None),
              lambda: L.crisp_kv_append_packed(ref(cache()), None, ref(tokens()), ref(tokens()), vp(256), 256, None),
              lambda: L.crisp_kv_append_packed(ref(cache()), ref(step()), None, ref(tokens()), vp(256), 256, None),
              lambda: L.crisp_kv_gather(ref(cache()), vp(256), 5, None, ref(tokens()), None, vp(256), 256, None),
              lambda: L.crisp_packed_prefill(None, ref(tokens()), ref(tokens()), ref(tokens()), ref(tokens()), vp(256), 256,
                                             None),
              lambda: L.crisp_packed_prefill(ref(packed()), ref(tokens()), None, ref(tokens()), ref(tokens()), vp(256),
                                             1 << 30, None)):
        assert f() == INVALID


def test_reserve_refusals(L):
    for field, value in (("max_new", -1), ("max_new", (1 << 24) + 1), ("max_all", -1), ("max_all", (1 << 24) + 1)):
        assert reserve(L, s=step(**{field: value})) == SHAPE
        assert append(L, s=step(**{field: value})) == SHAPE
    for field in ("_cu_new", "_cu_all", "_slots", "_positions", "_runs"):
        assert reserve(L, s=step(**{field: None})) == INVALID
        assert reserve(L, s=step(**{field: 1026})) == ALIGN
    assert reserve(L, s=step(max_all=7)) == INVALID and reserve(L, s=step(max_all=7, _all_slots=1026)) == ALIGN
    # the table is the cache's own; lengths are not read while they are written
    assert reserve(L, table=None) == INVALID and reserve(L, table=1024) == INVALID
    assert reserve(L, keep=512) == INVALID and reserve(L, new=512) == INVALID
    assert reserve(L, free=None) == INVALID and reserve(L, num=None) == INVALID
    assert reserve(L, free=770) == ALIGN and reserve(L, num=770) == ALIGN
    assert reserve(L, keep=1026) == ALIGN and reserve(L, new=1027) == ALIGN
    assert reserve(L, ws=None) == WORKSPACE and reserve(L, ws=260) == ALIGN and reserve(L, nbytes=255) == WORKSPACE
    # a step of no new tokens has no slots; no sequences: nothing is looked at
    assert reserve(L, s=step(max_new=0, _slots=None, _positions=None), ws=None) == WORKSPACE
    assert reserve(L, cache(batch=0, k=None), free=None, table=None, ws=None) == OK


def test_append_packed_refusals(L):
    assert append(L, s=step(_runs=None)) == INVALID and append(L, s=step(_slots=None)) == INVALID
    assert append(L, s=step(_runs=1025)) == ALIGN and append(L, s=step(_slots=1026)) == ALIGN
    assert append(L, k=tokens(data=None)) == INVALID and append(L, v=tokens(data=264)) == ALIGN
    assert append(L, k=tokens(h=100)) == ALIGN and append(L, v=tokens(t=64)) == SHAPE
    assert append(L, ws=None) == WORKSPACE and append(L, nbytes=100) == WORKSPACE
    assert append(L, s=step(max_new=0, _runs=None), k=tokens(data=None), ws=None) == OK
    assert append(L, cache(batch=0), k=tokens(data=None), ws=None) == OK


def test_gather_refusals(L):
    assert gather(L, n=-1) == SHAPE and gather(L, n=(1 << 24) + 1) == SHAPE
    assert gather(L, slots=None) == INVALID and gather(L, slots=258) == ALIGN and gather(L, count=257) == ALIGN
    assert gather(L, k=tokens(data=None)) == INVALID and gather(L, v=tokens(t=1028)) == ALIGN
    assert gather(L, ws=None) == WORKSPACE and gather(L, ws=128) == ALIGN
    assert gather(L, n=0, slots=None, ws=None) == OK


def test_gather_goes_by_the_pages_alone(L):
    # a cache without sequences has rows to read all the same
    none = dict(batch=0, table=None, lens=None)
    assert gather(L, cache(**none), ws=None) == WORKSPACE and gather(L, cache(**none), slots=None) == INVALID
    for field in ("k", "v", "k_scale", "v_scale"):
        assert gather(L, cache(**none, **{field: None})) == INVALID and gather(L, cache(**none, **{field: 258})) == ALIGN
    assert gather(L, cache(**none, k=None), n=0, slots=None) == OK


def test_packed_prefill_refusals(L):
    n = ctypes.c_size_t()
    for field, value, code in (("head_dim", 64, SHAPE), ("hq", 0, SHAPE), ("hq", 4098, SHAPE), ("hq", 7, SHAPE),
                               ("hkv", 0, SHAPE), ("batch", -1, SHAPE), ("batch", 1025, SHAPE), ("total_q", -1, SHAPE),
                               ("total_q", (1 << 24) + 1, SHAPE), ("total_k", -1, SHAPE), ("total_k", (1 << 24) + 1, SHAPE),
                               ("max_k", -1, SHAPE), ("scale", -1.0, INVALID), ("scale", float("nan"), INVALID),
                               ("scale", float("inf"), INVALID), ("cu_q", None, INVALID), ("cu_k", None, INVALID),
                               ("cu_q", 258, ALIGN), ("cu_k", 257, ALIGN)):
        p = packed(**{field: value})
        assert prefill(L, p) == code and L.crisp_packed_workspace_size(ref(p), ref(n)) == code
    assert L.crisp_packed_workspace_size(ref(packed()), None) == INVALID
    assert L.crisp_packed_workspace_size(ref(packed()), ref(n)) == OK and n.value % 256 == 0 and n.value >= 256
    for name in ("q", "k", "v", "out"):
        assert prefill(L, **{name: tokens(data=None)}) == INVALID
        assert prefill(L, **{name: tokens(data=264)}) == ALIGN and prefill(L, **{name: tokens(h=100)}) == ALIGN
        assert prefill(L, **{name: tokens(t=64)}) == SHAPE
    assert prefill(L, nbytes=n.value - 1) == WORKSPACE and prefill(L, ws=None) == WORKSPACE
    assert prefill(L, ws=128) == ALIGN
    # out is none of the inputs
    for name in ("q", "k", "v"):
        others = {x: tokens(data=512 * i) for i, x in enumerate(("q", "k", "v"), 1)}
        assert prefill(L, **others, out=tokens(data=others[name].data)) == INVALID
    # no queries: nothing is looked at; no keys: k and v are not
    assert prefill(L, packed(total_q=0, cu_q=None), q=tokens(data=None), ws=None) == OK
    assert prefill(L, packed(batch=0, cu_k=None), q=tokens(data=None), ws=None) == OK
    assert prefill(L, packed(total_k=0), k=tokens(data=None), v=tokens(data=None), ws=None) == WORKSPACE
    # the stride of an axis of one entry is not used
    one = packed(batch=1, hq=1, hkv=1, total_q=1, total_k=1)
    assert prefill(L, one, q=tokens(h=1, t=3), k=tokens(h=0, t=0), ws=None) == WORKSPACE


def test_workspaces_hold_unfinished_rows_of_split_tiles_only(L):
    n = ctypes.c_size_t()

    def size(**over):
        assert L.crisp_packed_workspace_size(ref(packed(**over)), ref(n)) == OK
        return n.value

    assert size(batch=1, hq=32, hkv=8, total_q=16384, total_k=16384) == 256
    few = size(batch=1, hq=32, hkv=8, total_q=40, total_k=131072)
    assert few > 2 * 40 * 32 * 128 * 4 and few < 304 * 128 * 130 * 4 + 1024
    assert size(batch=1, hq=32, hkv=8, total_q=40, total_k=131072, max_k=256) == 256


def test_the_longest_sequence_bounds_the_workspace(L):
    # the room of a step is no sequence's length: told the longest one, no tile is split and no rows are held
    n = ctypes.c_size_t()
    p = packed(batch=64, hq=32, hkv=8, total_q=8192, total_k=400_000, max_k=16384)
    assert L.crisp_packed_workspace_size(ref(p), ref(n)) == OK and n.value == 256


def make_cache():
    t = lambda *s, **k: torch.zeros(s, **k)  # noqa: E731
    u8, i32 = torch.uint8, torch.int32
    return crisp.make_kv_cache(t(4, 2, 128, 128, dtype=u8), t(4, 2, 128, 128, dtype=u8), torch.ones(4, 2), torch.ones(4, 2),
                               t(3, 2, dtype=i32), t(3, dtype=i32))


def test_the_binding_checks_tensors_before_the_call():
    c = make_cache()
    s = crisp.make_kv_step(c, 40, 9)
    assert (s.cu_new.shape, s.slots.shape, s.runs.shape, s.all_slots.shape) == ((4,), (40,), (7,), (9,))
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8)
    x = torch.zeros((40, 2, 128), dtype=torch.bfloat16)
    for max_new, max_all in ((-1, 0), (5, -1), ((1 << 24) + 1, 0)):
        with pytest.raises(ValueError):
            crisp.make_kv_step(c, max_new, max_all)
    for free, num, keep, new in ((i32(3), i32(1), None, None), (i32(4), i32(2), None, None), (i32(4), i32(1), i32(2), None),
                                 (i32(4), i32(1), None, torch.zeros(3)), (i32(4).long(), i32(1), None, None)):
        with pytest.raises(ValueError):
            crisp.kv_reserve(c, free, num, s, ws, keep=keep, new_lens=new)
    for bad in (x.float(), x.half(), x[:39], x[:, :1], x[..., :64], x.transpose(0, 1)):
        with pytest.raises(ValueError):
            crisp.kv_append_packed(c, s, bad, x, ws)
        with pytest.raises(ValueError):
            crisp.kv_gather(c, i32(40), x, bad, ws)
    with pytest.raises(ValueError):
        crisp.kv_gather(c, torch.zeros(40), x, x, ws)
    with pytest.raises(ValueError):
        crisp.kv_gather(c, i32(40), x, x, ws, count=i32(2))
    cu = i32(4)
    for args in ((torch.zeros(4), cu), (cu, i32(5)), (cu[:0], cu), (cu.long(), cu)):
        with pytest.raises(ValueError):
            crisp.make_packed(8, 2, *args, 40, 40)
    p = crisp.make_packed(8, 2, cu, cu, 40, 40)
    q = torch.zeros((40, 8, 128), dtype=torch.bfloat16)
    for args in ((x, x, x, q), (q, q, x, q), (q, x, x[:9], q), (q, x, x, x)):
        with pytest.raises(ValueError):
            crisp.packed_prefill(p, *args, ws)
    # everything in order but not on a GPU, or a step of another batch
    other = crisp.make_kv_step(make_cache(), 40, 9)
    other.batch = 2
    for call in (lambda: crisp.kv_reserve(c, i32(4), i32(1), s, ws), lambda: crisp.kv_append_packed(c, s, x, x, ws),
                 lambda: crisp.kv_gather(c, i32(40), x, x, ws), lambda: crisp.packed_prefill(p, q, x, x, q, ws)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    with pytest.raises(ValueError, match="another batch"):
        crisp.kv_append_packed(c, other, x, x, ws)
