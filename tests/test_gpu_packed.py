"""Batches of packed sequences on the GPU against their restatements on the CPU:
causal attention, handing out pages, writing packed tokens, reading them back,
and all of them together over two turns of a batch of requests."""
import os
import re

import numpy as np
import pytest
import torch

import dynamic_sparse_prefill_crisp_gb300 as crisp
from kv_helpers import VALUES, Pools, page_exponent, round_codes
from packed_helpers import B, D, Requests, attention, check, dev32, starts

pytestmark = pytest.mark.gpu

OK, BOUNDS, PAGES = 0, 8, 9
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def workspace(nbytes):
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    crisp.workspace_init(ws)
    return ws


def bf16(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.float32).to(torch.bfloat16)


def inputs(hq, hkv, q_lens, k_lens, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    tq, tk = int(sum(q_lens)), int(sum(k_lens))
    q = bf16(rng.standard_normal((tq, hq, D)) * spread)
    return q, bf16(rng.standard_normal((tk, hkv, D))), bf16(rng.standard_normal((tk, hkv, D)))


def prefill(q, k, v, q_lens, k_lens, max_k=None, scale=0.0, out=None, status=OK, extra=0):
    """q, k, v on the CPU; `extra` rows behind the last sequence, which have to stay."""
    hq, hkv = q.shape[1], k.shape[1]
    pad = lambda t: torch.cat([t, torch.full((extra, *t.shape[1:]), float("nan"), dtype=t.dtype)]).cuda()
    qd, kd, vd = pad(q), pad(k), pad(v)
    out = torch.full_like(qd, float("nan")) if out is None else out
    cu_q, cu_k = dev32(starts(q_lens)), dev32(starts(k_lens))
    p = crisp.make_packed(hq, hkv, cu_q, cu_k, qd.shape[0], kd.shape[0], max_k=max_k, scale=scale)
    ws = workspace(crisp.packed_workspace_size(p))
    ws[256:] = 0xFF  # unfinished rows start as NaN
    crisp.packed_prefill(p, qd, kd, vd, out, ws)
    assert crisp.read_status(ws) == status
    if extra:
        assert torch.isnan(out[q.shape[0]:]).all()
    return out[:q.shape[0]]


def run(hq, hkv, q_lens, k_lens=None, seed=1, spread=1.0, **kw):
    k_lens = q_lens if k_lens is None else k_lens
    q, k, v = inputs(hq, hkv, q_lens, k_lens, seed, spread)
    want, tol = attention(q.double().numpy(), k.double().numpy(), v.double().numpy(), q_lens, k_lens)
    check(prefill(q, k, v, q_lens, k_lens, **kw), want, tol)


# ------------------------------------------------------------------ attention
# name, hq, hkv, q_lens, k_lens (None: whole prompts)
ATTEND = [
    ("one-token", 4, 1, [1], None),
    ("edges", 4, 2, [63, 64, 65, 127, 128, 129, 1, 2], None),
    ("tile-edges-4", 4, 1, [31, 32, 33, 95, 96, 97], None),
    ("empty-between", 8, 2, [0, 5, 0, 0, 200, 0], None),
    ("mha", 3, 3, [300, 64, 129], None),
    ("gqa7", 28, 4, [257, 18, 19, 1], None),
    ("gqa8-ragged", 8, 1, [500, 3, 77, 128], None),
    ("one-group-of-16", 16, 1, [130, 9], None),
    ("group-of-48", 48, 1, [70, 1], None),
    ("group-of-65", 65, 1, [30, 11], None),
    ("group-of-128", 128, 1, [5, 66], None),
    ("group-of-200", 200, 1, [3, 65], None),
    ("chunks", 8, 2, [40, 1, 128, 7], [300, 1, 129, 700]),
    ("chunks-at-block-edges", 4, 1, [64, 65, 63, 1, 1], [128, 129, 127, 64, 65]),
    ("single-tokens", 8, 2, [1] * 9, [1, 2, 63, 64, 65, 127, 128, 129, 1000]),
    ("more-queries-than-keys", 4, 2, [70, 130, 5, 200], [3, 64, 0, 100]),
    ("no-keys-at-all", 4, 2, [7, 3], [0, 0]),
    ("no-queries-some", 4, 2, [0, 6, 0], [50, 60, 70]),
    ("long", 2, 1, [2500], None),
    ("split-chunk", 4, 1, [5], [5000]),
    ("split-chunk-gqa7", 7, 1, [40], [3001]),
    ("split-ragged", 4, 1, [9, 33, 1, 0, 3], [9000, 40, 2222, 100, 1]),
    ("split-short-and-long", 2, 1, [60, 60, 60], [60, 513, 4097]),
    ("split-in-twos", 4, 1, [1], [1001]),
    ("split-many-rows", 7, 1, [1500, 40], [4400, 3001]),
    ("split-whole-prompts", 5, 1, [2100, 130], None),
    ("batch-limit", 2, 1, [i % 3 for i in range(1024)], [i % 3 + i % 7 for i in range(1024)]),
    ("many-short", 4, 1, [(37 * i) % 200 for i in range(300)], None),
]


@pytest.mark.parametrize("name,hq,hkv,q_lens,k_lens", ATTEND, ids=[c[0] for c in ATTEND])
def test_attention_matches_64_bits(name, hq, hkv, q_lens, k_lens):
    run(hq, hkv, q_lens, k_lens, seed=len(name), extra=37)


@pytest.mark.parametrize("max_k", [0, 1, 300, 2000, 5000, 1 << 20])
def test_max_k_is_no_limit(max_k):
    run(4, 1, [5, 3], [2000, 700], max_k=max_k)


@pytest.mark.parametrize("q_len,k_len", [(300, 300), (20, 3000)])
def test_scores_that_grow_and_fall(q_len, k_len):
    # scores up to some hundreds: rows whose first keys are far below or above the others
    rng = np.random.default_rng(5)
    q, k, v = (x.double().numpy() for x in inputs(4, 1, [q_len], [k_len], 6))
    q[:, :, 0] = np.abs(q[:, :, 0]) + 1
    ramp = np.linspace(-900.0, 900.0, k_len)
    for keys in (ramp, -ramp, rng.permutation(ramp)):
        k[:, 0, 0] = keys
        qb, kb, vb = bf16(q), bf16(k), bf16(v)
        want, tol = attention(qb.double().numpy(), kb.double().numpy(), vb.double().numpy(), [q_len], [k_len])
        check(prefill(qb, kb, vb, [q_len], [k_len]), want, tol)


def test_scale_strides_and_a_fused_projection():
    hq, hkv, lens = 8, 2, [130, 77]
    q, k, v = inputs(hq, hkv, lens, lens, 7)
    want, tol = attention(*(x.double().numpy() for x in (q, k, v)), lens, lens, scale=0.25)
    n = sum(lens)
    qkv = torch.full((n + 3, hq + 2 * hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    qkv[:n, :hq], qkv[:n, hq:hq + hkv], qkv[:n, hq + hkv:] = q.cuda(), k.cuda(), v.cuda()
    wide = torch.full((hq, n + 3, 2 * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = wide.transpose(0, 1)[..., D:]  # head-major, every other 128 features
    cu = dev32(starts(lens))
    p = crisp.make_packed(hq, hkv, cu, cu, n + 3, n + 3, scale=0.25)
    ws = workspace(crisp.packed_workspace_size(p))
    crisp.packed_prefill(p, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], out, ws)
    assert crisp.read_status(ws) == OK
    check(out[:n], want, tol)
    assert torch.isnan(out[n:]).all() and torch.isnan(wide[..., :D]).all()


@pytest.mark.parametrize("hq,hkv,q_lens,k_lens", [
    (4, 1, [100, 50, 30], [100, 50, 30]), (4, 1, [33, 5], [900, 70]), (7, 1, [20, 3], [2000, 1000])])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_what_a_row_does_not_see_does_not_reach_it(hq, hkv, q_lens, k_lens, value):
    q, k, v = inputs(hq, hkv, q_lens, k_lens, 8)
    clean = prefill(q, k, v, q_lens, k_lens)
    cq, ck = starts(q_lens), starts(k_lens)
    # the second sequence's keys and values, all of them: the others do not change
    k2, v2 = k.clone(), v.clone()
    k2[ck[1]:ck[2]] = value
    v2[ck[1]:ck[2]] = value
    got = prefill(q, k2, v2, q_lens, k_lens)
    for b in range(len(q_lens)):
        if b != 1:
            assert torch.equal(got[cq[b]:cq[b + 1]], clean[cq[b]:cq[b + 1]])
    assert not torch.isfinite(got[cq[1]:cq[2]]).any()
    # one value of one feature, in the middle of the first sequence's queries
    i = q_lens[0] // 2
    j = k_lens[0] - q_lens[0] + i
    v3 = v.clone()
    v3[j, 0, 77] = value
    got = prefill(q, k, v3, q_lens, k_lens)
    assert torch.equal(got[:i], clean[:i])
    assert torch.equal(got[cq[1]:], clean[cq[1]:])
    hit = got[i:cq[1], :, 77].float()
    assert torch.isnan(hit).all() if value != value else (hit == value).all()
    rest = torch.arange(D, device="cuda") != 77
    assert torch.equal(got[i:cq[1]][..., rest], clean[i:cq[1]][..., rest])
    # a key: the rows that do not see it have the result within its tolerance (an
    # infinite score of another row of their tile may change the rows' reference)
    k3 = k.clone()
    k3[j] = value
    got = prefill(q, k3, v, q_lens, k_lens)
    want, tol = attention(*(x.double().numpy() for x in (q, k, v)), q_lens, k_lens)
    check(got[:i], want[:i], tol[:i])
    assert torch.equal(got[cq[1]:], clean[cq[1]:])


def test_bad_sums_make_a_sequence_empty():
    q_lens = [40, 50, 60]
    q, k, v = (x.cuda() for x in inputs(4, 1, q_lens, q_lens, 9))
    want = prefill(q.cpu(), k.cpu(), v.cpu(), q_lens, q_lens)
    for bad in ([60, 40, 90, 150], [0, 40, 90, 151], [-1, 40, 90, 150], [0, 40, 90, 2 ** 30]):
        for side in ("q", "k"):
            cu, good = dev32(bad), dev32(starts(q_lens))
            p = crisp.make_packed(4, 1, cu if side == "q" else good, good if side == "q" else cu, 150, 150)
            out = torch.full_like(q, float("nan"))
            ws = workspace(crisp.packed_workspace_size(p))
            crisp.packed_prefill(p, q, k, v, out, ws)
            assert crisp.read_status(ws) == BOUNDS
            for b in range(3):
                rows = slice(starts(q_lens)[b], starts(q_lens)[b + 1])
                if list(bad[b:b + 2]) == list(starts(q_lens)[b:b + 2]):
                    assert torch.equal(out[rows], want[rows])


def test_attention_in_a_graph_takes_other_lengths():
    hq, hkv, room = 8, 2, 400
    q = torch.zeros((room, hq, D), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((2 * room, hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cu_q, cu_k = dev32([0, 0, 0, 0]), dev32([0, 0, 0, 0])
    out = torch.empty_like(q)
    p = crisp.make_packed(hq, hkv, cu_q, cu_k, room, 2 * room, max_k=700)
    ws = workspace(crisp.packed_workspace_size(p))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        crisp.packed_prefill(p, q, k, v, out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        crisp.packed_prefill(p, q, k, v, out, ws)
    for seed, (q_lens, k_lens) in enumerate([([100, 0, 300], [100, 5, 300]), ([1, 1, 1], [600, 20, 77]),
                                             ([0, 0, 0], [1, 1, 1]), ([130, 17, 5], [130, 170, 500])]):
        x, y, z = inputs(hq, hkv, q_lens, k_lens, seed)
        want, tol = attention(*(t.double().numpy() for t in (x, y, z)), q_lens, k_lens)
        q[:x.shape[0]], k[:y.shape[0]], v[:y.shape[0]] = x.cuda(), y.cuda(), z.cuda()
        cu_q.copy_(dev32(starts(q_lens)))
        cu_k.copy_(dev32(starts(k_lens)))
        out.fill_(float("nan"))
        g.replay()
        assert crisp.read_status(ws) == OK
        check(out[:x.shape[0]], want, tol)
        assert torch.isnan(out[x.shape[0]:]).all()


def test_two_streams_and_repeats_give_the_same_bits():
    q_lens, k_lens = [300, 40, 1], [300, 2000, 900]
    q, k, v = inputs(8, 2, q_lens, k_lens, 11)
    want = prefill(q, k, v, q_lens, k_lens)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    cu_q, cu_k = dev32(starts(q_lens)), dev32(starts(k_lens))
    p = crisp.make_packed(8, 2, cu_q, cu_k, len(qd), len(kd))
    ws = [workspace(crisp.packed_workspace_size(p)) for _ in range(2)]
    outs = [torch.zeros_like(qd) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for o, w, s in zip(outs, ws, streams):
            crisp.packed_prefill(p, qd, kd, vd, o, w, stream=s)
    torch.cuda.synchronize()
    assert all(crisp.read_status(w) == OK for w in ws)
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_whole_prompts_agree_with_the_dense_step():
    # one sequence of the packed form is the dense step's layer, up to the order of sums
    n, hq, hkv = 700, 8, 2
    q, k, v = inputs(hq, hkv, [n], [n], 12)
    got = prefill(q, k, v, [n], [n]).float()
    qh, kh, vh = (t.cuda().transpose(0, 1) for t in (q, k, v))
    out = torch.empty((hq, n, D), dtype=torch.bfloat16, device="cuda")
    s = crisp.make_shape(hq, hkv, n, qh, kh, out)
    ws = workspace(crisp.workspace_size(s))
    crisp.dense_prefill(s, qh, kh, vh, out, ws)
    assert crisp.read_status(ws) == OK
    want, tol = attention(*(t.double().numpy() for t in (q, k, v)), [n], [n])
    diff = (got - out.transpose(0, 1).float()).abs().cpu().numpy()
    assert (diff <= 2 * tol).all()


# -------------------------------------------------------------------- reserve
class Batch:
    """A cache, its free pages and a step on the GPU beside the lists that restate them."""

    def __init__(self, batch, max_pages, num_pages, max_new, max_all, hkv=1, seed=0, pools=None):
        rng = np.random.default_rng(seed)
        free = rng.permutation(num_pages).tolist()
        self.ref = Requests(batch, max_pages, num_pages, free)
        self.pools = pools or Pools(num_pages, hkv)
        self.cache = self.pools.cache(self.ref.table, self.ref.lens)
        self.free, self.num = dev32(free), dev32([num_pages])
        self.step = crisp.make_kv_step(self.cache, max_new, max_all)
        self.ws = workspace(crisp.kv_append_workspace_size(self.cache))

    def reserve(self, keep, new, status=OK):
        """The call and its restatement; returns what the step holds, or None."""
        for name in ("slots", "positions", "runs", "all_slots", "cu_new", "cu_all"):
            getattr(self.step, name).fill_(-7)
        crisp.workspace_init(self.ws)
        crisp.kv_reserve(self.cache, self.free, self.num, self.step, self.ws, None if keep is None else dev32(keep),
                         None if new is None else dev32(new))
        want = self.ref.reserve(keep, new, self.step.max_new, self.step.max_all)
        assert crisp.read_status(self.ws) == (status if want is None else OK)
        assert (want is None) == (status != OK)
        self.same(want)
        return want

    def same(self, want):
        got = {name: getattr(self.step, name).cpu().numpy() for name in
               ("slots", "positions", "runs", "all_slots", "cu_new", "cu_all")}
        if want is None:
            assert not got["cu_new"].any() and not got["cu_all"].any() and not got["runs"].any()
            want = dict(slots=[], positions=[], all_slots=[])
        else:
            assert np.array_equal(got["cu_new"], want["cu_new"]) and np.array_equal(got["cu_all"], want["cu_all"])
            n = len(want["runs"])
            assert np.array_equal(got["runs"][:n], want["runs"]) and (got["runs"][n:] == len(want["slots"])).all()
        for name in ("slots", "positions", "all_slots"):
            n = min(len(want[name]), len(got[name]))
            assert np.array_equal(got[name][:n], want[name][:n]) and (got[name][n:] == -7).all()
        assert self.cache.tensors[5].tolist() == self.ref.lens
        assert self.cache.tensors[4].tolist() == self.ref.table
        n = int(self.num)
        assert n == len(self.ref.stack) and self.free[:n].tolist() == self.ref.stack


@pytest.mark.parametrize("batch,max_pages,num_pages,most,seed", [
    (1, 9, 9, 900, 0), (5, 12, 40, 500, 1), (33, 8, 150, 700, 2), (64, 3, 192, 300, 3), (1024, 2, 1500, 150, 4),
    (6, 70, 260, 4000, 5), (3, 40, 100, 5120, 6)])
def test_reserve_follows_the_lists(batch, max_pages, num_pages, most, seed):
    rng = np.random.default_rng(100 + seed)
    x = Batch(batch, max_pages, num_pages, max_new=batch * most, max_all=batch * max_pages * B, seed=seed)
    refused = 0
    for turn in range(25):
        lens = np.array(x.ref.lens)
        new = np.minimum(rng.integers(0, most + 1, batch) * (rng.random(batch) < 0.6), B * max_pages - lens)
        if turn % 5 == 0:
            new = np.minimum(1, B * max_pages - lens)  # a decode step
        keep = None
        if turn % 3 == 1:  # some requests done, some drafted tokens taken back
            keep = np.where(rng.random(batch) < 0.4, 0, np.maximum(lens - rng.integers(0, 300, batch), 0))
            keep = np.where(rng.random(batch) < 0.3, lens + 9, keep)  # more than there are: all
        need = sum(-(-(min(int(n), 10 ** 9 if keep is None else int(keep[b])) + int(new[b])) // B)
                   for b, n in enumerate(lens))
        status = PAGES if need > num_pages else OK
        refused += status != OK
        x.reserve(None if keep is None else keep.tolist(), new.tolist(), status)
    assert refused < 25


def test_reserve_undone_leaves_the_stack_as_it_was():
    x = Batch(6, 10, 50, 6 * 600, 0, seed=5)
    x.reserve(None, [500, 128, 0, 129, 1, 600])
    lens, stack, table = list(x.ref.lens), list(x.ref.stack), [list(r) for r in x.ref.table]
    for _ in range(3):
        x.reserve(lens, [7, 300, 400, 0, 127, 1])
    x.reserve(lens, None)
    assert x.ref.stack == stack and x.ref.table == table
    x.reserve([0] * 6, None)
    assert len(x.ref.stack) == 50 and int(x.num) == 50


def test_reserve_without_room_takes_nothing():
    x = Batch(3, 4, 8, 600, 1000, seed=6)
    x.reserve(None, [300, 100, 20])
    x.reserve(None, [0, 0, 600], BOUNDS)          # more than a table row holds
    x.reserve(None, [212, 200, 200], BOUNDS)      # more than max_new
    x.reserve(None, [150, 200, 240], BOUNDS)      # more than max_all
    x.reserve([400, 0, 0], [-1, 5, 5], BOUNDS)
    x.reserve([-1, 0, 0], [5, 5, 5], BOUNDS)
    x.reserve(None, [200, 250, 80])               # 4 + 3 + 1 pages of 8
    y = Batch(3, 4, 8, 600, 1500, seed=6)
    y.reserve(None, [300, 100, 20])
    y.reserve(None, [212, 300, 80], PAGES)        # 4 + 4 + 1 pages of 8
    y.reserve([300, 100, 0], [212, 300, 0])       # and without the third


def test_reserve_refuses_a_broken_state():
    x = Batch(2, 4, 6, 600, 0, seed=7)
    x.reserve(None, [300, 200])
    for broken in ("num_high", "num_low", "len_high", "len_low", "page"):
        num, lens, table = x.num.clone(), x.cache.tensors[5].clone(), x.cache.tensors[4].clone()
        if broken.startswith("num"):
            x.num.fill_(7 if broken == "num_high" else -1)
        elif broken.startswith("len"):
            x.cache.tensors[5][1] = 513 if broken == "len_high" else -1
        else:
            x.cache.tensors[4][0, 1] = 6
        state = x.num.clone(), x.cache.tensors[5].clone(), x.cache.tensors[4].clone(), x.free.clone()
        crisp.workspace_init(x.ws)
        crisp.kv_reserve(x.cache, x.free, x.num, x.step, x.ws, keep=dev32([0, 0]), new_lens=dev32([5, 5]))
        assert crisp.read_status(x.ws) == BOUNDS
        assert not x.step.cu_new.any() and not x.step.runs.any()
        for a, b in zip(state, (x.num, x.cache.tensors[5], x.cache.tensors[4], x.free)):
            assert torch.equal(a, b)
        for t, was in ((x.num, num), (x.cache.tensors[5], lens), (x.cache.tensors[4], table)):
            t.copy_(was)
    x.reserve([0, 0], [5, 5])


# ------------------------------------------------------------- append, gather
def append_reference(host, table, kept, new, k, v):
    """The documented rule in 64 bits, in place on numpy copies of the pools; k, v float64 [tokens][hkv][128]."""
    codes_of = {0: (host[0], host[2]), 1: (host[1], host[3])}
    at = 0
    for b, (old, n) in enumerate(zip(kept, new)):
        for p in range(old // B, -(-(old + n) // B) if n else 0):
            lo = max(old, p * B)
            hi = min(old + n, (p + 1) * B)
            held = lo - p * B
            page = table[b][p]
            for side, x in enumerate((k, v)):
                codes, scales = codes_of[side]
                for g in range(x.shape[1]):
                    fresh = x[at + lo - old:at + hi - old, g]
                    scale = 2.0 ** page_exponent(fresh)
                    if held:
                        had = float(scales[page, g])
                        if had >= scale:
                            scale = had
                        else:
                            codes[page, g, :held] = round_codes(VALUES[codes[page, g, :held]] * had / scale)
                    codes[page, g, held:held + hi - lo] = round_codes(fresh / scale)
                    scales[page, g] = scale
        at += n


def same_values(got, want):
    """Codes agree, -0 and 0 taken for one."""
    sign = np.where(want & 127, 255, 127)
    assert np.array_equal(got & sign, want & sign)


@pytest.mark.parametrize("hkv,interleaved,lens", [
    (1, False, [1]), (2, True, [0, 1, 127, 128, 129, 0, 300]), (4, False, [5, 600, 0, 64]), (3, False, [2] * 40)])
def test_append_packed_and_gather(hkv, interleaved, lens):
    rng = np.random.default_rng(sum(lens) + hkv)
    batch = len(lens)
    num = 8 * batch + 2
    x = Batch(batch, 8, num, sum(lens) * 2 + 70 * batch + 9, 1024 * batch, seed=1,
              pools=Pools(num, hkv, interleaved))
    for turn in range(3):
        new = lens if turn == 0 else rng.integers(0, 70, batch).tolist()
        old = list(x.ref.lens)
        x.reserve(None, new)
        n = sum(new)
        scale = 2.0 ** rng.uniform(-6, 6, (x.step.max_new, 1, 1))
        k, v = (bf16(rng.standard_normal((x.step.max_new, hkv, D)) * scale) for _ in range(2))
        k[n:], v[n:] = float("nan"), float("nan")
        host = x.pools.host()
        append_reference(host, x.ref.table, old, new, k.double().numpy(), v.double().numpy())
        wide = torch.full((x.step.max_new, hkv + 1, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 1:] = k.cuda()
        crisp.kv_append_packed(x.cache, x.step, wide[:, 1:], v.cuda(), x.ws)
        assert crisp.read_status(x.ws) == OK
        got = x.pools.host()
        for a, b in zip(got[:2], host[:2]):
            same_values(a, b)
        for a, b in zip(got[2:], host[2:]):
            assert np.array_equal(a, b, equal_nan=True)
        # everything back, in order, exactly
        total = sum(x.ref.lens)
        outs = [torch.full((x.step.max_all, hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        crisp.kv_gather(x.cache, x.step.all_slots, *outs, x.ws, count=x.step.cu_all[-1:])
        assert crisp.read_status(x.ws) == OK
        slots = np.array([x.ref.table[b][j // B] * B + j % B for b in range(batch) for j in range(x.ref.lens[b])], dtype=int)
        for out, codes, scales in zip(outs, got[:2], got[2:]):
            want = VALUES[codes[slots // B, :, slots % B]] * scales[slots // B].astype(np.float64)[..., None]
            assert np.array_equal(out[:total].double().cpu().numpy(), want)
            assert (out[total:] == 7.0).all()


def test_append_packed_is_append():
    # the same tokens in the padded form: the same pools, bit for bit
    lens, hkv = [300, 5, 128, 77], 2
    rng = np.random.default_rng(21)
    x = Batch(4, 4, 20, 600, 0, hkv=hkv, seed=2)
    y = Pools(20, hkv)
    x.reserve(None, lens)
    cache = y.cache(x.ref.table, lens)
    k, v = (bf16(rng.standard_normal((600, hkv, D)) * 50).cuda() for _ in range(2))
    k[3, 0, 5], v[400, 1, 7] = float("inf"), float("nan")
    crisp.kv_append_packed(x.cache, x.step, k, v, x.ws)
    pads = []
    for t in (k, v):
        pad = torch.zeros((4, 300, hkv, D), dtype=torch.bfloat16, device="cuda")
        for b, (n, at) in enumerate(zip(lens, starts(lens))):
            pad[b, :n] = t[at:at + n]
        pads.append(pad.transpose(1, 2))
    crisp.kv_append(cache, *pads, x.ws, new_lens=dev32(lens))
    assert crisp.read_status(x.ws) == OK
    for a, b in zip(x.pools.host(), y.host()):
        assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f")


@pytest.mark.parametrize("width,shift", [(D + 24, 8), (D + 24, 16), (D + 16, 16), (D + 16, 8), (D + 8, 0)])
def test_append_at_16_byte_addresses(width, shift):
    # rows and heads whose strides or first values are odd multiples of 16 bytes: the same pools as from dense
    # rows, in the packed form and the padded one
    lens, hkv, room = [200, 3, 129], 3, 340
    rng = np.random.default_rng(width + shift)
    k, v = (bf16(rng.standard_normal((room, hkv, D)) * 9).cuda() for _ in range(2))
    parts = []
    for t in (k, v):
        wide = torch.full((room, hkv, width), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[..., shift:shift + D] = t
        parts.append(wide[..., shift:shift + D])
    pools = []
    for pair in ((k, v), parts):
        x = Batch(3, 4, 9, room, 0, hkv=hkv, seed=4)
        x.reserve(None, lens)
        crisp.kv_append_packed(x.cache, x.step, *pair, x.ws)
        assert crisp.read_status(x.ws) == OK
        pools.append(x.pools.host())
        y = Pools(9, hkv)
        for b, at, n in ((0, 0, 200), (2, 200, 140)):  # a sequence at a time, [1][hkv][n][128]
            one = [t[at:at + n].transpose(0, 1)[None] for t in pair]
            crisp.kv_append(y.cache([x.ref.table[b]], [n]), *one, x.ws)
        assert crisp.read_status(x.ws) == OK
        pools.append(y.host())
    for a, b in zip(pools[0] + pools[1], pools[2] + pools[3]):
        assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f")


def test_append_packed_refuses_bad_runs():
    x = Batch(2, 4, 8, 300, 0, hkv=1, seed=3)
    x.reserve(None, [200, 50])
    k = torch.ones((300, 1, D), dtype=torch.bfloat16, device="cuda")
    before = x.pools.host()
    runs, slots = x.step.runs.clone(), x.step.slots.clone()
    for bad_runs, bad_slots in (([-1, 200], None), ([0, 301], None), ([0, 129], None), ([5, 2], None),
                                ([0, 100], -1), ([0, 100], 8 * B), ([0, 100], 2 ** 31 - 1), ([0, 100], 29)):
        x.step.runs.fill_(bad_runs[1])
        x.step.runs[0] = bad_runs[0]
        x.step.slots.copy_(slots)
        if bad_slots is not None:
            x.step.slots[0] = bad_slots
        crisp.workspace_init(x.ws)
        crisp.kv_append_packed(x.cache, x.step, k, k, x.ws)
        assert crisp.read_status(x.ws) == BOUNDS
        for a, b in zip(before, x.pools.host()):
            assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f")
    x.step.runs.copy_(runs)
    x.step.slots.copy_(slots)


def test_gather_takes_any_slots():
    rng = np.random.default_rng(31)
    pools = Pools(5, 3)
    codes = rng.integers(0, 256, (5, 3, B, D)).astype(np.uint8)
    for t in (pools.k, pools.v):
        t.copy_(torch.from_numpy(codes))
    scales = 2.0 ** rng.integers(-100, 100, (5, 3))
    pools.ks.copy_(torch.from_numpy(scales))
    pools.vs.copy_(torch.from_numpy(scales))
    cache = pools.cache([[-1]], [0])
    ws = workspace(crisp.kv_append_workspace_size(cache))
    slots = rng.integers(0, 5 * B, 333)
    slots[[3, 50]], slots[7] = -1, slots[8]
    out = [torch.full((333, 3, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    crisp.kv_gather(cache, dev32(slots), *out, ws)
    assert crisp.read_status(ws) == OK
    want = VALUES[codes[slots // B, :, slots % B]] * scales[slots // B][..., None]
    want[[3, 50]] = 7.0
    for o in out:
        assert np.array_equal(o.double().cpu().numpy(), want, equal_nan=True)
    slots[9] = 5 * B  # past the pool: left alone, and told
    out = [torch.full((333, 3, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    crisp.kv_gather(cache, dev32(slots), *out, ws)
    assert crisp.read_status(ws) == BOUNDS
    want[9] = 7.0
    for o in out:
        assert np.array_equal(o.double().cpu().numpy(), want, equal_nan=True)


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("captured", [False, True])
def test_two_turns_of_a_batch(captured):
    """Three requests' prompts are stored and attended to; the second is replaced and the
    others go on by a chunk, over keys read back from the cache; then each takes a token."""
    hq, hkv, room, room_all = 8, 2, 700, 1500
    rng = np.random.default_rng(41)
    x = Batch(3, 8, 30, room, room_all, hkv=hkv, seed=4)
    step, cache = x.step, x.cache
    new = lambda n, h: torch.zeros((n, h, D), dtype=torch.bfloat16, device="cuda")
    q, out, k, v, ka, va = new(room, hq), new(room, hq), new(room, hkv), new(room, hkv), new(room_all, hkv), new(room_all, hkv)
    whole = crisp.make_packed(hq, hkv, step.cu_new, step.cu_new, room, room)
    going = crisp.make_packed(hq, hkv, step.cu_new, step.cu_all, room, room_all)
    ws = workspace(max(crisp.packed_workspace_size(whole), crisp.packed_workspace_size(going)))
    keep, count = dev32([0, 0, 0]), dev32([0, 0, 0])

    def turn(first):
        crisp.kv_reserve(cache, x.free, x.num, step, ws, keep=keep, new_lens=count)
        crisp.kv_append_packed(cache, step, k, v, ws)
        if first:
            crisp.packed_prefill(whole, q, k, v, out, ws)
        else:
            crisp.kv_gather(cache, step.all_slots, ka, va, ws, count=step.cu_all[-1:])
            crisp.packed_prefill(going, q, ka, va, out, ws)

    graphs = []
    if captured:
        for first in (True, False):
            turn(first)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                turn(first)
            graphs.append(g)
    for first, kept, n in ((True, [0, 0, 0], [300, 17, 200]), (False, [300, 0, 200], [60, 400, 129])):
        keep.copy_(dev32(kept))
        count.copy_(dev32(n))
        for t in (q, k, v):
            t[:] = bf16(rng.standard_normal(t.shape)).cuda()
        out.fill_(float("nan"))
        if captured:
            graphs[0 if first else 1].replay()
        else:
            turn(first)
        assert crisp.read_status(ws) == OK
        want = x.ref.reserve(kept, n, room, room_all)
        assert np.array_equal(step.slots.cpu().numpy()[:sum(n)], want["slots"])
        keys, values = k[:sum(n)], v[:sum(n)]
        k_lens = n
        if not first:
            k_lens = [a + b for a, b in zip(kept, n)]
            keys, values = ka[:sum(k_lens)], va[:sum(k_lens)]
            host = x.pools.host()
            slots = np.array(want["all_slots"])
            back = VALUES[host[0][slots // B, :, slots % B]] * host[2][slots // B].astype(np.float64)[..., None]
            assert np.array_equal(keys.double().cpu().numpy(), back)
        ref, tol = attention(q[:sum(n)].double().cpu().numpy(), keys.double().cpu().numpy(), values.double().cpu().numpy(),
                             n, k_lens)
        check(out[:sum(n)], ref, tol)
        assert torch.isnan(out[sum(n):]).all()
    # a token each by the decode call, over the same pages
    keep.copy_(dev32(x.ref.lens))
    count.fill_(1)
    crisp.kv_reserve(cache, x.free, x.num, step, ws, keep=keep, new_lens=count)
    crisp.kv_append_packed(cache, step, k, v, ws)
    x.ref.reserve(x.ref.lens, [1, 1, 1], room, room_all)
    dws = workspace(crisp.decode_workspace_size(cache, hq))
    one = q[:3].unsqueeze(2)
    got = torch.empty_like(one)
    crisp.decode_attention(cache, one, got, dws)
    crisp.kv_gather(cache, step.all_slots, ka, va, ws, count=step.cu_all[-1:])
    crisp.packed_prefill(going, q, ka, va, out, ws)
    assert crisp.read_status(ws) == OK and crisp.read_status(dws) == OK
    ref, tol = attention(q[:3].double().cpu().numpy(), ka[:sum(x.ref.lens)].double().cpu().numpy(),
                         va[:sum(x.ref.lens)].double().cpu().numpy(), [1, 1, 1], x.ref.lens)
    check(out[:3], ref, tol)
    assert (np.abs(got[:, :, 0].double().cpu().numpy() - ref) <= 2 * tol).all()


# --------------------------------------------------------- the largest, the oddest
def sampled_rows(q, k, v, rows, off):
    """Attention of some rows of one sequence and head in 64 bits on the GPU, and its tolerance."""
    out, tol = [], []
    for i in rows:
        n = off + i + 1
        s = (k[:n, 0].double() @ q[i, 0].double()) * D ** -0.5
        p = torch.softmax(s, 0)
        ds = (D ** -0.5 * 2.0 ** -15.9 * (k[:n, 0].double().abs() @ q[i, 0].double().abs())).max()
        o, a = p @ v[:n, 0].double(), p @ v[:n, 0].double().abs()
        out.append(o)
        tol.append(2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -20 + 2 * (n / 8 + 32) * 2.0 ** -23 + 2 * ds) * a)
    return torch.stack(out), torch.stack(tol)


def test_a_prompt_of_a_million_tokens():
    # a CTA passes more than 2^16 sub-blocks of each of its two slots
    n = 1 << 20
    gen = torch.Generator(device="cuda").manual_seed(51)
    q, k, v = (torch.randn((n, 1, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    cu = dev32([0, n])
    p = crisp.make_packed(1, 1, cu, cu, n, n)
    ws = workspace(crisp.packed_workspace_size(p))
    out = torch.full_like(q, float("nan"))
    crisp.packed_prefill(p, q, k, v, out, ws)
    assert crisp.read_status(ws) == OK
    assert torch.isfinite(out).all()
    rows = [0, 1, 63, 64, 127, 128, 99_999, 500_000, n - 129, n - 128, n - 2, n - 1]
    want, tol = sampled_rows(q, k, v, rows, 0)
    assert ((out[rows, 0].double() - want).abs() <= tol).all()


def test_rows_past_32_bit_offsets():
    # rows 24 k elements apart: the last sequence starts past 2^31 elements (and 2^32 bytes)
    stride, room = 24 * 1024, 90_000
    gen = torch.Generator(device="cuda").manual_seed(52)
    flat = torch.empty(room * stride, dtype=torch.bfloat16, device="cuda")
    rows = flat.view(room, stride // D, D)
    q, k, v, out = rows[:, :4], rows[:, 4:6], rows[:, 6:8], rows[:, 8:12]
    q_lens = [300, room - 700, 400]
    cu = dev32(starts(q_lens))
    first, last = slice(0, 300), slice(room - 400, room)
    for t in (q, k, v, out):
        t.fill_(float("nan"))
        for part in (first, last):
            t[part] = torch.randn(t[part].shape, generator=gen, device="cuda").to(torch.bfloat16)
    out.fill_(float("nan"))
    # the middle sequence's queries are left out (a key sequence of its length, no queries)
    cu_q = dev32([0, 300, 300, 700])
    qs = torch.cat([q[first], q[last]])
    p = crisp.make_packed(4, 2, cu_q, cu, 700, room)
    ws = workspace(crisp.packed_workspace_size(p))
    got = torch.full_like(qs, float("nan"))
    crisp.packed_prefill(p, qs, k, v, got, ws)
    assert crisp.read_status(ws) == OK
    keys, values = (torch.cat([t[first], t[last]]).double().cpu().numpy() for t in (k, v))
    want, tol = attention(qs.double().cpu().numpy(), keys, values, [300, 400], [300, 400])
    check(got, want, tol)
    # and the same rows of q and out where they are
    cu_q = dev32([room - 400, room])
    cu_k = dev32([room - 400, room])
    p = crisp.make_packed(4, 2, cu_q, cu_k, room, room, max_k=400)
    ws = workspace(crisp.packed_workspace_size(p))
    crisp.packed_prefill(p, q, k, v, out, ws)
    assert crisp.read_status(ws) == OK
    check(out[last], want[300:], tol[300:])
    assert torch.isnan(out[:room - 400]).all()


@pytest.mark.parametrize("shift", [0, 8])
def test_rows_at_16_byte_addresses(shift):
    # out rows that start at odd multiples of 16 bytes (and gathered rows)
    lens = [70, 130]
    q, k, v = inputs(4, 2, lens, lens, 53)
    want, tol = attention(*(x.double().numpy() for x in (q, k, v)), lens, lens)
    wide = torch.full((200, 4, D + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = wide[..., 8 + shift:8 + shift + D]
    got = prefill(q, k, v, lens, lens, out=out)
    check(got, want, tol)
    assert torch.isnan(wide[..., :8 + shift]).all() and torch.isnan(wide[..., 8 + shift + D:]).all()
    pools = Pools(2, 3)
    codes = np.random.default_rng(1).integers(0, 127, (2, 3, B, D)).astype(np.uint8)
    for t, s in ((pools.k, pools.ks), (pools.v, pools.vs)):
        t.copy_(torch.from_numpy(codes))
        s.fill_(0.5)
    cache = pools.cache([[0]], [0])
    ws = workspace(256)
    outs = [torch.full((100, 3, D + 24), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    parts = [o[..., 8 + shift:8 + shift + D] for o in outs]
    slots = np.arange(100) * 2 + 7
    crisp.kv_gather(cache, dev32(slots), *parts, ws)
    assert crisp.read_status(ws) == OK
    for o, part in zip(outs, parts):
        assert np.array_equal(part.double().cpu().numpy(), VALUES[codes[slots // B, :, slots % B]] * 0.5)
        assert (o[..., :8 + shift] == 7.0).all() and (o[..., 8 + shift + D:] == 7.0).all()


def test_large_values_do_not_leave_the_range_of_sums():
    # V near 2^100 with scores that grow by up to 60 binary orders from the first keys on: the first
    # reference would take the sums past fp32's largest number
    n = 400
    q, k, v = (x.double().numpy() for x in inputs(4, 1, [n], [n], 54))
    q[:, :, 0] = 1.0
    q[:, :, 1:] *= 0.1
    k[:, 0, 0] = np.where(np.arange(n) < 64, 0.0, 40.0 * np.log(2.0) * np.sqrt(D))
    v *= 2.0 ** 100
    qb, kb, vb = bf16(q), bf16(k), bf16(v)
    want, tol = attention(qb.double().numpy(), kb.double().numpy(), vb.double().numpy(), [n], [n])
    check(prefill(qb, kb, vb, [n], [n]), want, tol)


def test_many_tiles_done_again():
    # every tile of every sequence sums past its range, or holds a NaN that some rows do not see
    lens = [150] * 40
    q, k, v = inputs(8, 2, lens, lens, 55)
    k = k.clone()
    for b in range(40):
        k[150 * b + 100:150 * (b + 1), :, 0] = 300.0
    q[:, :, 0] = q[:, :, 0].abs() + 2
    want, tol = attention(*(x.double().numpy() for x in (q, k, v)), lens, lens)
    check(prefill(q, k, v, lens, lens), want, tol)
    v2 = v.clone()
    for b in range(40):
        v2[150 * b + 140:150 * b + 150] = float("nan")
    got = prefill(q, k, v2, lens, lens).view(40, 150, 8, D)
    seen = got[:, :140].reshape(-1, 8, D)
    rows = [150 * b + i for b in range(40) for i in range(140)]
    check(seen, want[rows], tol[rows])
    assert torch.isnan(got[:, 140:].float()).all()


def test_a_key_of_minus_infinity_is_left_out():
    # the first sub-block's scores are all -inf for some heads: the rows go by the others
    n = 200
    q, k, v = inputs(2, 1, [n], [n], 56)
    q[:, :, 0] = 1.0
    k = k.clone()
    k[:64, 0, 0] = float("-inf")
    k[64:, 0, 0] = -300.0
    want, tol = attention(q[64:].double().numpy(), k[64:].double().numpy(), v[64:].double().numpy(), [n - 64], [n - 64])
    got = prefill(q, k, v, [n], [n])
    check(got[64:], want, tol)


# ------------------------------------------------------------------ checking build
def test_the_checking_build_on_valid_batches():
    # every call between canary regions with both libraries: no status, the same bits
    from dynamic_sparse_prefill_crisp_gb300 import build as crisp_build
    from test_gpu_bounds import Guarded

    i32 = torch.int32
    hq, hkv, room, room_all = 7, 1, 700, 1400
    rng = np.random.default_rng(91)
    values = [bf16(rng.standard_normal((room, h, D))).cuda() for h in (hq, hkv, hkv)]

    def run_all(lib):
        saved, crisp._lib = crisp._lib, lib
        try:
            g = Guarded()
            k8, v8 = g((9, hkv, B, D), torch.uint8), g((9, hkv, B, D), torch.uint8)
            ks, vs = g((9, hkv), torch.float32), g((9, hkv), torch.float32)
            table, lens = g((3, 8), i32, 255), g((3,), i32)
            cache = crisp.make_kv_cache(k8, v8, ks, vs, table, lens)
            free, num = g((9,), i32), g((1,), i32)
            free.copy_(torch.arange(9))
            num.fill_(9)
            step = crisp.make_kv_step(cache, room, room_all)
            for name in ("cu_new", "cu_all", "slots", "positions", "runs", "all_slots"):
                t = g(getattr(step, name).shape, i32)
                setattr(step, name, t)
                setattr(step, "_" + name, t.data_ptr())
            q, k, v = (g(t.shape, torch.bfloat16) for t in values)
            for a, b in zip((q, k, v), values):
                a.copy_(b)
            out, ka, va = g((room, hq, D), torch.bfloat16), g((room_all, hkv, D), torch.bfloat16), g((room_all, hkv, D), torch.bfloat16)
            p = crisp.make_packed(hq, hkv, step.cu_new, step.cu_all, room, room_all)
            ws = g((crisp.packed_workspace_size(p),), torch.uint8)
            crisp.workspace_init(ws)
            got = []
            for keep, new in (([0, 0, 0], [300, 17, 200]), ([300, 0, 190], [60, 333, 1])):
                crisp.kv_reserve(cache, free, num, step, ws, keep=dev32(keep), new_lens=dev32(new))
                crisp.kv_append_packed(cache, step, k, v, ws)
                crisp.kv_gather(cache, step.all_slots, ka, va, ws, count=step.cu_all[-1:])
                crisp.packed_prefill(p, q, ka, va, out, ws)
                got += [t.clone() for t in (out, ka, va, k8, v8, ks, vs, table, lens, free, num, step.slots, step.runs,
                                            step.all_slots, step.positions)]
            assert crisp.read_status(ws) == OK and g.intact()
            return got
        finally:
            crisp._lib = saved

    release = run_all(crisp.lib())
    checking = run_all(crisp.load_library(crisp_build.build(debug=True)))
    for a, b in zip(release, checking):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# --------------------------------------------------------------------- as documented
def test_the_readme_example_of_a_batch():
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), re.S)
    blocks = [b for b in blocks if "make_packed" in b]
    assert len(blocks) == 1
    hq, hkv, max_new, max_all, pages = 8, 2, 600, 900, 20
    gen = torch.Generator(device="cuda").manual_seed(71)
    rand = lambda n, h: torch.randn((n, h, D), generator=gen, device="cuda").to(torch.bfloat16)
    pools = Pools(pages, hkv)
    cache = pools.cache([[-1] * 6] * 3, [0] * 3)
    names = dict(torch=torch, crisp=crisp, cache=cache, pages=pages, hq=hq, hkv=hkv, max_new=max_new, max_all=max_all,
                 keep=dev32([0, 0, 0]), counts=dev32([300, 17, 200]), q=rand(max_new, hq), k=rand(max_new, hkv),
                 v=rand(max_new, hkv), out=torch.zeros((max_new, hq, D), dtype=torch.bfloat16, device="cuda"),
                 k_all=rand(max_all, hkv), v_all=rand(max_all, hkv))
    exec(blocks[0], names)
    assert crisp.read_status(names["ws"]) == OK
    assert cache.tensors[5].tolist() == [300, 17, 200] and int(names["num_free"]) == pages - 3 - 1 - 2
    n = 517
    want, tol = attention(names["q"][:n].double().cpu().numpy(), names["k_all"][:n].double().cpu().numpy(),
                          names["v_all"][:n].double().cpu().numpy(), [300, 17, 200], [300, 17, 200])
    check(names["out"][:n], want, tol)


def test_a_step_that_does_not_fit_leaves_everything():
    x = Batch(2, 4, 5, 600, 1024, hkv=2, seed=8)
    x.reserve(None, [300, 200])
    k = torch.ones((600, 2, D), dtype=torch.bfloat16, device="cuda")
    crisp.kv_append_packed(x.cache, x.step, k, k, x.ws)
    before = x.pools.host()
    x.reserve(None, [10, 300], PAGES)
    q = torch.ones((600, 4, D), dtype=torch.bfloat16, device="cuda")
    out, back = torch.full_like(q, 3.0), torch.full((1024, 2, D), 3.0, dtype=torch.bfloat16, device="cuda")
    crisp.workspace_init(x.ws)
    crisp.kv_append_packed(x.cache, x.step, 2 * k, 2 * k, x.ws)
    crisp.kv_gather(x.cache, x.step.all_slots, back, back.clone(), x.ws, count=x.step.cu_all[-1:])
    p = crisp.make_packed(4, 2, x.step.cu_new, x.step.cu_all, 600, 1024)
    ws = workspace(crisp.packed_workspace_size(p))
    crisp.packed_prefill(p, q, back, back, out, ws)
    assert crisp.read_status(x.ws) == OK and crisp.read_status(ws) == OK
    assert (out == 3.0).all() and (back == 3.0).all()
    for a, b in zip(before, x.pools.host()):
        assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f")


def test_many_slots_and_a_long_request():
    # the maps of many tokens (a launch of their own), requests of no token between long ones
    x = Batch(7, 120, 300, 40_000, 50_000, seed=9)
    x.reserve(None, [0, 15_000, 0, 1, 9_000, 0, 127])
    x.reserve([0, 15_000, 0, 0, 8_900, 0, 127], [1, 100, 0, 12_345, 3, 0, 1])
    x.reserve(None, [0] * 7)
    x.reserve([0] * 7, [5, 6, 7, 8, 9, 10, 11])


def test_host_threads_at_once():
    # the same structures from several host threads, each with its stream and workspace
    import threading
    q_lens, k_lens = [200, 30], [200, 900]
    q, k, v = (t.cuda() for t in inputs(8, 2, q_lens, k_lens, 57))
    cu_q, cu_k = dev32(starts(q_lens)), dev32(starts(k_lens))
    p = crisp.make_packed(8, 2, cu_q, cu_k, len(q), len(k))
    ws = [workspace(crisp.packed_workspace_size(p)) for _ in range(4)]
    outs = [torch.zeros_like(q) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            for _ in range(30):
                crisp.packed_prefill(p, q, k, v, outs[i], ws[i], stream=streams[i])
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and all(crisp.read_status(w) == OK for w in ws)
    assert all(torch.equal(o, outs[0]) for o in outs)
    want, tol = attention(*(t.double().cpu().numpy() for t in (q, k, v)), q_lens, k_lens)
    check(outs[0], want, tol)
