"""The paged 8-bit cache on the GPU against its restatement in 64 bits: writing
tokens, attention over it, eviction, and the three together after a prefilled
layer. Pools start full of NaN codes and NaN scales, table rows end in -1."""
import numpy as np
import pytest
import torch

import dynamic_sparse_prefill_crisp_gb300 as crisp
import synth
from gpu_helpers import to_dev
from kv_helpers import (B, D, VALUES, Pools, attention, fill, page_exponent, round_codes, shuffled_table, tokens_of)

pytestmark = pytest.mark.gpu

CRISP_ERR_BOUNDS = 8


def workspace(nbytes):
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    crisp.workspace_init(ws)
    return ws


def bf16(x):
    return torch.as_tensor(x, dtype=torch.float32).to(torch.bfloat16)


def cut(table, lens):
    """The table with -1 past each sequence's pages."""
    return [[p if j < -(-n // B) else -1 for j, p in enumerate(row)] for row, n in zip(table, lens)]


def make(lens, hkv, seed, spread=0.0, sink=1.0, interleaved=False):
    rng = np.random.default_rng(seed)
    pages = max(1, max(-(-n // B) for n in lens))
    table, num = shuffled_table(rng, len(lens), pages)
    pools = Pools(num, hkv, interleaved)
    fill(pools, table, lens, rng, spread, sink)
    return pools, pools.cache(cut(table, lens), lens), table, rng


def decode(cache, q, weights_in=None, weights_out=None, scale=0.0, status=0):
    """q: CPU bf16 [batch][hq][q_len][128]; the output starts as NaN."""
    qd = q.cuda()
    out = torch.full_like(qd, float("nan"))
    ws = workspace(crisp.decode_workspace_size(cache, q.shape[1], q.shape[2], weights_out is not None))
    crisp.decode_attention(cache, qd, out, ws, weights_in, weights_out, scale=scale)
    assert crisp.read_status(ws) == status
    return out


def check(got, want, tol):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - want) / np.maximum(tol, 1e-300)) if want.size else 0.0
    assert worst <= 1.0, worst


# name, hq, hkv, q_len, lens
DECODE = [
    ("one-key", 4, 1, 1, [1]),
    ("page-edges", 4, 2, 1, [127, 128, 129, 255, 256, 257]),
    ("empty-and-short", 8, 2, 1, [0, 5, 300, 0]),
    ("all-empty", 4, 1, 1, [0, 0]),
    ("mha", 3, 3, 1, [200, 64]),
    ("gqa4-2k", 4, 1, 1, [2048]),
    ("gqa7", 28, 4, 1, [1000, 257]),
    ("rows-16", 16, 1, 1, [700, 129]),
    ("rows-32", 32, 1, 1, [700, 130]),
    ("rows-36-two-chunks", 36, 1, 1, [300, 131]),
    ("drafted-4", 28, 4, 4, [515, 130]),
    ("drafted-edges", 4, 2, 3, [0, 1, 2, 3, 128, 129, 130, 131]),
    ("drafted-16", 2, 1, 16, [7, 16, 135, 400]),
    ("drafted-gqa16", 16, 1, 5, [260, 4]),
    ("drafted-gqa7", 14, 2, 2, [300, 129, 2, 1]),
    ("rows-24", 12, 1, 2, [513]),
    ("batch-limit", 2, 1, 1, [i % 3 * 70 for i in range(1024)]),
    ("many-short", 4, 1, 1, [(37 * i) % 200 for i in range(300)]),
    ("one-long", 4, 1, 1, [45000]),
    ("rows-limit", 1024, 1, 1, [300, 3]),
    ("rows-limit-drafted", 64, 1, 16, [300, 20, 0]),
    # many short sequences, of no page, of an odd and of an even number of pages
    ("short-items", 8, 4, 1, [97 * i % 520 for i in range(160)]),
    ("short-items-12-rows", 12, 1, 1, [0, 0] + [61 * i % 520 for i in range(300)] + [0]),
    ("short-items-two-chunks", 40, 1, 1, [97 * i % 520 // 128 * 128 for i in range(40)] + [300] * 130),
    ("short-items-drafted", 4, 1, 4, [1 + 61 * i % 380 for i in range(330)]),
]


@pytest.mark.parametrize("name,hq,hkv,q_len,lens", DECODE, ids=[c[0] for c in DECODE])
def test_decode_matches_64_bits(name, hq, hkv, q_len, lens):
    pools, cache, table, rng = make(lens, hkv, len(lens) * 1000 + hq, spread=3.0)
    q = bf16(rng.standard_normal((len(lens), hq, q_len, D)))
    want, tol, w, wtol = attention(pools.host(), table, lens, q.double().numpy())
    check(decode(cache, q), want, tol)
    # with weights: the same output bit for bit, the weights added below lens, the rest left
    cap = cache.max_pages * B
    w_in = torch.rand((len(lens), hkv, cap), generator=torch.Generator().manual_seed(1)).cuda()
    w_out = torch.full_like(w_in, -7.0)
    out = decode(cache, q, w_in, w_out)
    assert torch.equal(out, decode(cache, q))
    got, base = w_out.double().cpu().numpy(), w_in.double().cpu().numpy()
    for b, n in enumerate(lens):
        assert (got[b, :, n:] == -7.0).all()
        err = np.abs(got[b, :, :n] - base[b, :, :n] - w[b, :, :n])
        assert (err <= wtol[b, :, :n] + 2.0 ** -24 * np.abs(got[b, :, :n])).all(), err.max()


def test_decode_scale_strides_and_interleaved_pool():
    lens = [300, 130]
    pools, cache, table, rng = make(lens, 2, 5, interleaved=True)
    q = bf16(rng.standard_normal((2, 3, 8, D))).transpose(1, 2)  # token-major [batch][tokens][heads]
    want, tol, _, _ = attention(pools.host(), table, lens, q.double().numpy(), scale=0.25)
    wide = torch.full((2, 3, 11, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = wide[:, :, 2:10, 8:].transpose(1, 2)
    qd = torch.zeros((2, 3, 9, 144), dtype=torch.bfloat16, device="cuda")[:, :, 1:, 16:].transpose(1, 2)
    qd.copy_(q)
    ws = workspace(crisp.decode_workspace_size(cache, 8, 3))
    crisp.decode_attention(cache, qd, out, ws, scale=0.25)
    assert crisp.read_status(ws) == 0
    check(out, want, tol)
    out.fill_(float("nan"))
    assert torch.isnan(wide).all()  # nothing outside out was written


def test_decode_keeps_the_mass_of_many_small_weights():
    # One key about 18 above the rest in base 2, 60000 others alike: their p is
    # 2^-18 of the largest each, and together a fifth of the sum.
    n = 60000
    pools, cache, table, rng = make([n], 1, 7)
    k, v, ks, vs = pools.host()
    q = np.zeros((1, 1, 1, D))
    q[..., 0] = 1.0
    k[:] = 0
    ks[:] = 0.125
    k[table[0][3], 0, 17, 0] = round_codes(np.array([100.0]))[0]
    pools.k.copy_(torch.from_numpy(k))
    pools.ks.copy_(torch.from_numpy(ks))
    v = np.where((v & 127) == 127, v, v & 127)  # values of one sign: the sum does not cancel
    pools.v.copy_(torch.from_numpy(v))
    want, tol, _, _ = attention(pools.host(), table, [n], q, scale=1.0)
    check(decode(cache, bf16(q), scale=1.0), want, tol)


def test_decode_scores_of_any_size():
    # scores in the thousands, of both signs
    pools, cache, table, rng = make([500, 40], 1, 8)
    q = bf16(rng.standard_normal((2, 4, 1, D)) * 50.0)
    want, tol, _, _ = attention(pools.host(), table, [500, 40], q.double().numpy(), scale=1.0)
    check(decode(cache, q, scale=1.0), want, tol)


def test_decode_q_rows_of_any_size():
    # zero rows, rows of subnormal bf16 values, rows up to the largest
    pools, cache, table, rng = make([300], 1, 9, spread=0.0)
    q = rng.standard_normal((1, 6, 1, D))
    for h, m in enumerate((0.0, 1e-39, 1e-20, 1e4, 1.0, 3e-5)):
        q[0, h] *= m
    q = bf16(q)
    want, tol, _, _ = attention(pools.host(), table, [300], q.double().numpy(), scale=1e-3)
    check(decode(cache, q, scale=1e-3), want, tol)


def test_decode_non_finite_values_stay_where_they_are_seen():
    # The newest token's K and V are NaN: only the last query token sees it.
    for n in (130, 129, 128):  # the newest key in a page of its own, in the middle, at the end
        pools, cache, table, rng = make([n, 50], 1, 10)
        k, v, ks, vs = pools.host()
        k[table[0][(n - 1) // B], 0, (n - 1) % B] = 127
        v[table[0][(n - 1) // B], 0, (n - 1) % B] = 255
        pools.k.copy_(torch.from_numpy(k))
        pools.v.copy_(torch.from_numpy(v))
        q = bf16(rng.standard_normal((2, 4, 3, D)))
        out = decode(cache, q).double().cpu().numpy()
        want, tol, _, _ = attention(pools.host(), table, [n, 50], q.double().numpy())
        assert np.isnan(out[0, :, 2]).all()
        seen = np.ones(out.shape, bool)
        seen[0, :, 2] = False
        assert (np.abs(out - want)[seen] <= tol[seen]).all()
    # a NaN (or infinite) query row is that row's alone
    pools, cache, table, rng = make([300], 1, 11)
    q = rng.standard_normal((1, 4, 2, D))
    q[0, 1, 0, 5], q[0, 2, 1, 9] = np.nan, np.inf
    out = decode(cache, bf16(q)).double().cpu().numpy()
    bad = np.zeros((1, 4, 2), bool)
    bad[0, 1, 0] = bad[0, 2, 1] = True
    assert np.isnan(out[bad]).all() and np.isfinite(out[~bad]).all()


def test_decode_bad_pages_and_lengths_are_reported_and_hold_nothing():
    lens = [400, 300, 200]
    pools, cache, table, rng = make(lens, 2, 12)
    q = bf16(rng.standard_normal((3, 4, 1, D)))
    good = decode(cache, q)
    # the middle page of sequence 0 names no page: its keys are not there
    t = pools.table.clone()
    for bad in (-5, pools.num_pages, 2 ** 31 - 1):
        pools.table.copy_(t)
        pools.table[0, 1] = bad
        out = decode(cache, q, status=CRISP_ERR_BOUNDS)
        assert torch.equal(out[1:], good[1:])
        host = pools.host()
        k, v = zip(*(tokens_of(host, table[0], 400, g) for g in range(2)))
        keep = np.r_[0:128, 256:400]
        for h in range(4):
            s = D ** -0.5 * (k[h // 2][keep] @ q[0, h, 0].double().numpy())
            p = np.exp(s - s.max())
            want = p @ v[h // 2][keep] / p.sum()
            assert np.abs(out[0, h, 0].double().cpu().numpy() - want).max() < 0.02
    # the only page of a sequence
    pools.table.copy_(t)
    pools.lens.copy_(torch.tensor([400, 100, 200], dtype=torch.int32))
    pools.table[1, 0] = -1
    assert (decode(cache, q, status=CRISP_ERR_BOUNDS)[1] == 0).all()
    pools.table.copy_(t)
    # lengths outside count as the nearest inside
    pools.lens.copy_(torch.tensor([-3, 300, 200], dtype=torch.int32))
    out = decode(cache, q, status=CRISP_ERR_BOUNDS)
    assert (out[0] == 0).all() and torch.equal(out[1:], good[1:])


def test_decode_on_several_streams_at_once():
    # each stream with a workspace of its own, and inputs made there just before
    lens = [1000, 300, 17, 900]
    pools, cache, table, rng = make(lens, 4, 15)
    qs = [bf16(rng.standard_normal((4, 28, 2, D))).cuda() for _ in range(4)]
    want = [decode(cache, q.cpu()) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    spaces = [workspace(crisp.decode_workspace_size(cache, 28, 2)) for _ in streams]
    torch.cuda.synchronize()
    got = []
    for i in range(24):
        for s, ws in zip(streams, spaces):
            with torch.cuda.stream(s):
                q = qs[i % 4].clone()
                out = torch.empty_like(q)
                crisp.decode_attention(cache, q, out, ws)
                got.append((i % 4, q, out, out.clone()))
    torch.cuda.synchronize()
    assert all(crisp.read_status(ws) == 0 for ws in spaces)
    assert all(torch.equal(want[i], seen) for i, _, _, seen in got)


def test_decode_shared_pages_streams_graphs_and_in_place_weights():
    # Two sequences with the same first pages; the call on a side stream, in a
    # captured graph, and again: the same bits each time.
    lens = [700, 650]
    pools, cache, table, rng = make(lens, 2, 13)
    pools.table[1, :5] = pools.table[0, :5]
    table[1][:5] = table[0][:5]
    q = bf16(rng.standard_normal((2, 8, 1, D)))
    want, tol, w, wtol = attention(pools.host(), table, lens, q.double().numpy())
    ref = decode(cache, q)
    check(ref, want, tol)
    qd = q.cuda()
    weights = torch.zeros((2, 2, cache.max_pages * B), device="cuda")
    ws = workspace(crisp.decode_workspace_size(cache, 8, 1, True))
    out = torch.empty_like(qd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    crisp.decode_attention(cache, qd, out, ws, weights, weights, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    once = weights.clone()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    out2 = torch.empty_like(qd)
    with torch.cuda.graph(g1):
        crisp.decode_attention(cache, qd, out, ws, weights, weights)
    with torch.cuda.graph(g2):  # a second graph over the same workspace
        crisp.decode_attention(cache, qd, out2, ws)
    for _ in range(2):
        out.zero_()
        out2.zero_()
        g1.replay()
        g2.replay()
    torch.cuda.synchronize()
    assert crisp.read_status(ws) == 0
    assert torch.equal(out, ref) and torch.equal(out2, ref)
    n0 = lens[0]
    assert torch.allclose(weights[0, :, :n0], 3 * once[0, :, :n0], rtol=2.0 ** -20)
    # lengths may change between replays
    pools.lens.copy_(torch.tensor([129, 0], dtype=torch.int32))
    g2.replay()
    torch.cuda.synchronize()
    want, tol, _, _ = attention(pools.host(), table, [129, 0], q.double().numpy())
    check(out2, want, tol)


# ------------------------------------------------------------------- writing
def append_reference(host, table, start, new, name):
    """Codes and scales after the new tokens [hkv][n][128] of one sequence."""
    codes, scales = (host[0], host[2]) if name == "k" else (host[1], host[3])
    hkv, n, _ = new.shape
    for g in range(hkv):
        for p in range(start // B, -(-(start + n) // B)):
            lo = max(start, p * B)
            hi = min(start + n, (p + 1) * B)
            x = new[g, lo - start:hi - start]
            e = 2.0 ** page_exponent(x)
            old = lo - p * B
            page = table[p]
            if old > 0:
                had = float(scales[page, g])
                e = max(e, had)
                if e != had:
                    codes[page, g, :old] = round_codes(VALUES[codes[page, g, :old]] * had / e)
            scales[page, g] = e
            codes[page, g, old:old + hi - lo] = round_codes(x / e)


def assert_same_pools(pools, host):
    for got, want in zip(pools.host(), host):
        if got.dtype == np.uint8:  # NaN codes of either sign are one value
            nan = (got & 127) == 127
            assert np.array_equal(nan, (want & 127) == 127)
            # -0 and 0 are one value too
            assert (VALUES[got][~nan] == VALUES[want][~nan]).all()
        else:
            assert np.array_equal(got, want, equal_nan=True)


# name, hkv, [start], [new]
APPEND = [
    ("one-token", 2, [0], [1]),
    ("one-token-each", 1, [0, 1, 127, 128, 300], [1, 1, 1, 1, 1]),
    ("within-a-page", 2, [5], [60]),
    ("page-edges", 1, [0, 0, 128, 100, 1], [128, 129, 128, 28, 127]),
    ("ragged", 3, [0, 77, 256, 10], [0, 400, 131, 1]),
    ("long", 1, [129], [5000]),
]


@pytest.mark.parametrize("name,hkv,start,new", APPEND, ids=[c[0] for c in APPEND])
def test_append_writes_the_codes_of_the_definition(name, hkv, start, new):
    pools, _, _, rng = make([max(s, 0) for s in start], hkv, 21)
    lens = [s + n for s, n in zip(start, new)]
    pages = max(-(-n // B) for n in lens)
    table, num = shuffled_table(rng, len(lens), pages)
    pools = Pools(num, hkv)
    fill(pools, table, start, rng, spread=2.0)
    host = pools.host()
    cache = pools.cache(cut(table, lens), lens)
    n_new = max(new)
    x = {m: bf16(rng.standard_normal((len(lens), hkv, n_new, D)) * 2.0 ** rng.uniform(-3, 3, (len(lens), hkv, n_new, 1)))
         for m in "kv"}
    ws = workspace(crisp.kv_append_workspace_size(cache))
    new_lens = torch.tensor(new, dtype=torch.int32).cuda()
    dev = {m: x[m].transpose(1, 2).contiguous().cuda().transpose(1, 2) for m in "kv"}  # token-major
    for again in range(2):  # a second time changes nothing
        crisp.kv_append(cache, dev["k"], dev["v"], ws, new_lens=new_lens)
        assert crisp.read_status(ws) == 0
        if not again:
            for b in range(len(lens)):
                for m in "kv":
                    append_reference(host, table[b], start[b], x[m][b, :, :new[b]].double().numpy(), m)
        assert_same_pools(pools, host)


def test_append_without_new_lens_and_no_tokens():
    rng = np.random.default_rng(22)
    pools = Pools(4, 2)
    cache = pools.cache([[2], [0]], [40, 40])
    host = pools.host()
    ws = workspace(crisp.kv_append_workspace_size(cache))
    x = bf16(rng.standard_normal((2, 2, 40, D)))
    crisp.kv_append(cache, x[:, :, :0].cuda(), x[:, :, :0].cuda(), ws)
    assert_same_pools(pools, host)
    crisp.kv_append(cache, x.cuda(), (-x).cuda(), ws)
    for b, t in enumerate(([2], [0])):
        append_reference(host, t, 0, x[b].double().numpy(), "k")
        append_reference(host, t, 0, -x[b].double().numpy(), "v")
    assert crisp.read_status(ws) == 0
    assert_same_pools(pools, host)


def test_append_values_of_any_size():
    # zeros, subnormal and huge bf16 values, NaN and infinities; then a page
    # whose scale grows by 2^30, so that what it held becomes zero or tiny
    x = torch.zeros((1, 1, 10, D))
    x[0, 0, 1] = 1e-39
    x[0, 0, 2] = torch.linspace(-1e-38, 1e-38, D)
    x[0, 0, 3, :3] = torch.tensor([float("nan"), float("inf"), -float("inf")])
    x[0, 0, 3, 3:] = 1e-30
    big = torch.full((1, 1, 3, D), 3e38)
    big[0, 0, 1] = torch.linspace(-3e38, 3e38, D)
    pools = Pools(2, 1)
    host = pools.host()
    lens = [0]
    cache = pools.cache([[1]], lens)
    ws = workspace(crisp.kv_append_workspace_size(cache))
    at = 0
    for part in (x[:, :, :1], x[:, :, 1:3], x[:, :, 3:4], x[:, :, 4:], x[:, :, :2] + 1.0, big):
        part = bf16(part)
        pools.lens.copy_(torch.tensor([at + part.shape[2]], dtype=torch.int32))
        crisp.kv_append(cache, part.cuda(), part.cuda(), ws)
        for m in "kv":
            append_reference(host, [1], at, part[0].double().numpy(), m)
        at += part.shape[2]
        assert crisp.read_status(ws) == 0
        assert_same_pools(pools, host)


def test_append_token_by_token_equals_one_append():
    # Powers of two: but for codes below 2^-6 scales the order of writing does not show.
    rng = np.random.default_rng(23)
    x = bf16(rng.choice([-1, 1], (1, 2, 200, D)) * 2.0 ** rng.uniform(-3, 3, (1, 2, 200, D)))
    one, many = Pools(3, 2), Pools(3, 2)
    ws = None
    for pools, steps in ((one, [200]), (many, [1] * 70 + [30] + [1] * 100)):
        cache = pools.cache([[0, 2]], [0])
        ws = workspace(crisp.kv_append_workspace_size(cache)) if ws is None else ws
        at = 0
        for s in steps:
            part = x[:, :, at:at + s].cuda()
            at += s
            pools.lens.fill_(at)
            crisp.kv_append(cache, part, part, ws)
    assert crisp.read_status(ws) == 0
    assert_same_pools(many, one.host())


def test_append_bad_pages_and_lengths_write_nothing_there():
    rng = np.random.default_rng(24)
    pools = Pools(6, 1)
    host = pools.host()
    table = [[0, 6], [3, -1], [5, 4]]
    cache = pools.cache(table, [200, 200, 300])  # sequence 2's length is past its two pages
    x = bf16(rng.standard_normal((3, 1, 200, D)))
    ws = workspace(crisp.kv_append_workspace_size(cache))
    crisp.kv_append(cache, x.cuda(), x.cuda(), ws, new_lens=torch.tensor([200, 300, 256], dtype=torch.int32).cuda())
    assert crisp.read_status(ws) == CRISP_ERR_BOUNDS
    # sequences 0 and 1: their good page, 200 tokens each; sequence 2: 200 tokens that end at 256
    for m in "kv":
        append_reference(host, table[0], 0, x[0, :, :128].double().numpy(), m)
        append_reference(host, table[1], 0, x[1, :, :128].double().numpy(), m)
        append_reference(host, table[2], 56, x[2].double().numpy(), m)
    # sequence 2's first page holds 56 older rows of which nothing was written: its scale was NaN
    got = pools.host()
    for i in (0, 3, 4):
        for a, w in zip(got, host):
            assert np.array_equal(a[i], w[i]), i
    for i in (1, 2):
        assert (got[0][i] == 127).all() and np.isnan(got[2][i]).all()


# ------------------------------------------------------------------ eviction
def evict_reference(weights, n, keep, sink, recent):
    """Kept positions of one sequence and head."""
    if n <= keep:
        return np.arange(n)
    w = np.where(np.isnan(weights[:n]), np.inf, weights[:n]).astype(np.float64)
    w = np.where(np.isnan(weights[:n]), 1e300, np.where(np.isposinf(w), 1e299, w))
    mid = np.arange(sink, n - recent)
    order = mid[np.argsort(-w[mid], kind="stable")][:keep - sink - recent]
    return np.sort(np.r_[np.arange(sink), order, np.arange(n - recent, n)])


# name, hkv, lens, keep, sink, recent, kind of weights
EVICT = [
    ("small", 1, [300], 100, 4, 16, "random"),
    ("edges", 2, [127, 128, 129, 0, 1, 500], 128, 0, 0, "random"),
    ("keep-one", 1, [1, 2, 400], 1, 0, 0, "random"),
    ("all-protected", 2, [600, 90], 130, 30, 100, "random"),
    ("ties", 2, [700, 650], 333, 10, 50, "few"),
    ("all-equal", 1, [1000], 257, 1, 1, "equal"),
    ("odd-values", 1, [900], 300, 2, 3, "odd"),
    ("longer-than-a-turn", 1, [9001, 4096, 4097], 4097, 128, 128, "random"),
    ("chunks", 2, [16390, 20000, 300], 9000, 128, 1024, "random"),
    ("chunks-ties", 1, [40000], 20001, 7, 9, "few"),
    ("chunks-short", 1, [30000, 5], 29999, 0, 1, "equal"),
    ("chunks-odd-values", 1, [33000], 20000, 5, 7, "odd"),
]


@pytest.mark.parametrize("name,hkv,lens,keep,sink,recent,kind", EVICT, ids=[c[0] for c in EVICT])
@pytest.mark.parametrize("shared", [True, False], ids=["one-pool", "two-pools"])
def test_evict_keeps_and_packs_what_the_definition_says(name, hkv, lens, keep, sink, recent, kind, shared):
    batch = len(lens)
    rng = np.random.default_rng(31)
    pages = max(1, max(-(-n // B) for n in lens))
    new_pages = -(-keep // B)
    num = batch * (pages + new_pages) + 2
    ids = rng.permutation(num)
    table = ids[:batch * pages].reshape(batch, pages).tolist()
    new_table = ids[batch * pages:batch * (pages + new_pages)].reshape(batch, new_pages).tolist()
    src = Pools(num, hkv)
    # codes straight from bytes: any finite code, scales of neighbouring pages apart
    gen = torch.Generator(device="cuda").manual_seed(5)
    for t in (src.k, src.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=gen, device="cuda", dtype=torch.uint8))
        t.masked_fill_((t & 127) == 127, 3)
        t.view(-1, D)[::3] &= 0x9F  # rows of small values: pages whose scale changes
    for s in (src.ks, src.vs):
        s.copy_(torch.pow(2.0, torch.randint(-4, 5, s.shape, generator=gen, device="cuda").float()).round(decimals=4))
    dst = src if shared else Pools(num, hkv)
    cap = pages * B
    w = np.exp(rng.standard_normal((batch, hkv, cap)) * 3).astype(np.float32)
    if kind == "few":
        w = rng.choice(np.array([0.0, 0.5, 0.5000001, 2.0], np.float32), w.shape)
    elif kind == "equal":
        w[:] = 1.5
    elif kind == "odd":
        w[..., ::7] = 0.0
        w[..., 1::7] = -0.0
        w[..., 2::50] = np.inf
        w[..., 3::60] = np.nan
        w[..., 4::11] = -1.0
        w[..., 5::13] = 1e-42
        w[..., 6::170] = -np.inf
    host, dhost = src.host(), dst.host()
    cache = src.cache(cut(table, lens), lens)
    new_cache = (Pools.cache(dst, cut(new_table, [min(n, keep) for n in lens]), [-1] * batch))
    wd = torch.from_numpy(w).cuda()
    new_w = torch.full((batch, hkv, new_pages * B), -7.0, device="cuda")
    kept = torch.full((batch, hkv, new_pages * B), -7, dtype=torch.int32, device="cuda")
    ws = workspace(crisp.kv_evict_workspace_size(cache, keep))
    crisp.kv_evict(cache, new_cache, wd, ws, keep=keep, sink=sink, recent=recent, new_weights=new_w, kept=kept)
    assert crisp.read_status(ws) == 0
    new_lens = new_cache.tensors[5].cpu().numpy()
    assert new_lens.tolist() == [min(n, keep) for n in lens]
    kn, wn = kept.cpu().numpy(), new_w.cpu().numpy()
    for b, n in enumerate(lens):
        m = min(n, keep)
        assert (kn[b, :, m:] == -7).all() and (wn[b, :, m:] == -7.0).all()
        for g in range(hkv):
            pos = evict_reference(w[b, g], n, keep, sink, recent)
            assert np.array_equal(kn[b, g, :m], pos)
            assert np.array_equal(wn[b, g, :m], w[b, g, pos], equal_nan=True)
            if m == 0:
                continue
            k, v = tokens_of(host, table[b], n, g)
            for x, codes, scales in ((k, dhost[0], dhost[2]), (v, dhost[1], dhost[3])):
                for p in range(-(-m // B)):
                    rows = x[pos[p * B:(p + 1) * B]]
                    e = 2.0 ** page_exponent(rows)
                    scales[new_table[b][p], g] = e
                    codes[new_table[b][p], g, :len(rows)] = round_codes(rows / e)
    assert_same_pools(dst, dhost)
    if not shared:  # into pages of the same ids, by the same table
        alike = Pools(num, hkv)
        cache2 = crisp.make_kv_cache(alike.k, alike.v, alike.ks, alike.vs, cache.tensors[4],
                                     torch.full((batch,), -1, dtype=torch.int32, device="cuda"))
        if keep <= cache2.max_pages * B:
            crisp.kv_evict(cache, cache2, wd, ws, keep=keep, sink=sink, recent=recent)
            assert crisp.read_status(ws) == 0
            for b, n in enumerate(lens):
                m = min(n, keep)
                for g in range(hkv):
                    for a, c in zip(tokens_of(alike.host(), table[b], m, g), tokens_of(dst.host(), new_table[b], m, g)):
                        assert np.array_equal(a, c, equal_nan=True)
    # without the optional outputs: the same cache
    again = Pools(num, hkv)
    cache2 = Pools.cache(again, cut(new_table, [min(n, keep) for n in lens]), [-1] * batch)
    crisp.kv_evict(cache, cache2, wd, ws, keep=keep, sink=sink, recent=recent)
    assert crisp.read_status(ws) == 0
    for b, n in enumerate(lens):
        m = min(n, keep)
        for g in range(hkv):
            for a, c in zip(tokens_of(again.host(), new_table[b], m, g), tokens_of(dst.host(), new_table[b], m, g)):
                assert np.array_equal(a, c, equal_nan=True)


def test_evict_keeps_non_finite_values_and_reports_bad_pages():
    rng = np.random.default_rng(32)
    src, dst = Pools(4, 1), Pools(4, 1)
    fill(src, [[1, 3]], [200], rng)
    k = src.host()[0]
    k[3, 0, 5, 7] = 255
    src.k.copy_(torch.from_numpy(k))
    w = torch.ones((1, 1, 256), device="cuda")
    cache = src.cache([[1, 3]], [200])
    ws = workspace(crisp.kv_evict_workspace_size(cache, 150))
    new_cache = dst.cache([[2, 0]], [0])
    crisp.kv_evict(cache, new_cache, w, ws, keep=150, sink=10, recent=120)
    assert crisp.read_status(ws) == 0
    host, got = src.host(), dst.host()
    want = tokens_of(host, [1, 3], 200, 0)
    have = tokens_of(got, [2, 0], 150, 0)
    pos = np.r_[0:30, 80:200]
    assert np.isnan(want[0][133]).any()
    assert np.array_equal(have[0], want[0][pos], equal_nan=True) and np.array_equal(have[1], want[1][pos])
    # a bad source page reads as zeros, a bad new page is not written
    src.table[0, 1] = 9
    dst.table[0, 1] = -2
    before = dst.host()
    crisp.kv_evict(cache, new_cache, w, ws, keep=150, sink=10, recent=120)
    assert crisp.read_status(ws) == CRISP_ERR_BOUNDS
    got = dst.host()
    assert np.array_equal(got[0][0], before[0][0]) and np.array_equal(got[1][0], before[1][0])
    have = VALUES[got[0][2, 0]] * float(got[2][2, 0])
    assert (have[30 + 48:] == 0).all()  # positions 128.. are on the bad page
    assert np.array_equal(have[:78], want[0][np.r_[0:30, 80:128]])


def test_evict_replays_from_a_cuda_graph():
    # short and long caches (one launch and a launch per digit); the weights and
    # lengths may change between replays
    for lens, keep in (([3000, 900], 1000), ([20000, 17000], 9000)):
        pools, cache, table, rng = make(lens, 1, 33)
        new_pages = -(-keep // B)
        dst = Pools(2 * new_pages, 1)
        new_cache = dst.cache(np.arange(2 * new_pages).reshape(2, new_pages).tolist(), [0, 0])
        cap = cache.max_pages * B
        w = torch.zeros((2, 1, cap), device="cuda")
        kept = torch.full((2, 1, new_pages * B), -7, dtype=torch.int32, device="cuda")
        ws = workspace(crisp.kv_evict_workspace_size(cache, keep))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            crisp.kv_evict(cache, new_cache, w, ws, keep=keep, sink=3, recent=50, kept=kept)
        for step in range(2):
            wn = rng.random((2, 1, cap)).astype(np.float32)
            w.copy_(torch.from_numpy(wn))
            n = [x - 100 * step for x in lens]
            pools.lens.copy_(torch.tensor(n, dtype=torch.int32))
            g.replay()
            assert crisp.read_status(ws) == 0
            assert new_cache.tensors[5].tolist() == [min(x, keep) for x in n]
            for b in range(2):
                m = min(n[b], keep)
                pos = evict_reference(wn[b, 0], n[b], keep, 3, 50)
                assert np.array_equal(kept[b, 0, :m].cpu().numpy(), pos)
                want = tokens_of(pools.host(), table[b], n[b], 0)
                have = tokens_of(dst.host(), list(range(b * new_pages, (b + 1) * new_pages)), m, 0)
                for x, y in zip(want, have):
                    assert (np.abs(x[pos] - y) <= 2.0 ** -10 * 2.0 ** -3).all()  # subnormal codes may round again


# ------------------------------------------------------------- sizes and edges
def test_offsets_past_32_bits():
    # A pool of 5.2 GB for K and as much for V: pages on both sides of 2^32
    # bytes, written by an append, read by attention, packed to the last pages.
    hkv, num = 8, 40000
    k, v = (torch.empty((num, hkv, B, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((num, hkv), device="cuda") for _ in range(2))
    table = torch.tensor([[5, 32767, 32768, 39990], [39999, 1, 20000, 39000]], dtype=torch.int32).cuda()
    lens = torch.tensor([400, 300], dtype=torch.int32).cuda()
    cache = crisp.make_kv_cache(k, v, ks, vs, table, lens)
    rng = np.random.default_rng(51)
    x = {m: bf16(rng.standard_normal((2, hkv, 400, D))) for m in "kv"}
    ws = workspace(max(crisp.decode_workspace_size(cache, 16, 1, True), crisp.kv_evict_workspace_size(cache, 200)))
    crisp.kv_append(cache, x["k"].cuda(), x["v"].cuda(), ws, new_lens=lens)
    q = bf16(rng.standard_normal((2, 16, 1, D)))
    out, weights = torch.empty_like(q.cuda()), torch.zeros((2, hkv, 4 * B), device="cuda")
    crisp.decode_attention(cache, q.cuda(), out, ws, None, weights)
    new_table = torch.tensor([[39998, 32769], [2, 39997]], dtype=torch.int32).cuda()
    new_lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    new_cache = crisp.make_kv_cache(k, v, ks, vs, new_table, new_lens)
    out2 = torch.empty_like(out)
    crisp.kv_evict(cache, new_cache, weights, ws, keep=200, sink=10, recent=20)
    crisp.decode_attention(new_cache, q.cuda(), out2, ws)
    assert crisp.read_status(ws) == 0

    def read(tab):  # the touched pages only, renumbered
        ids = torch.tensor(sorted({int(i) for i in tab.flatten()}))
        at = {int(p): j for j, p in enumerate(ids)}
        host = tuple(t[ids.cuda()].cpu().numpy() for t in (k, v, ks, vs))
        return host, [[at[int(p)] for p in row] for row in tab.cpu()]
    host, tab = read(table)
    for b, n in enumerate((400, 300)):
        for g in range(hkv):
            for y, m in zip(tokens_of(host, tab[b], n, g), "kv"):
                want = x[m][b, g, :n].double().numpy()
                assert np.abs(y - want).max() <= np.abs(want).max() * 2.0 ** -4
    want, tol, _, _ = attention(host, tab, [400, 300], q.double().numpy())
    check(out, want, tol)
    host, tab = read(new_table)
    want, tol, _, _ = attention(host, tab, [200, 200], q.double().numpy())
    check(out2, want, tol)


def test_a_batch_of_no_sequences_is_nothing_to_do():
    pools = Pools(2, 1)
    cache = pools.cache(torch.zeros((0, 3), dtype=torch.int32), torch.zeros(0, dtype=torch.int32))
    host = pools.host()
    ws = workspace(max(crisp.kv_append_workspace_size(cache), crisp.decode_workspace_size(cache, 4),
                       crisp.kv_evict_workspace_size(cache, 5)))
    x = torch.zeros((0, 1, 7, D), dtype=torch.bfloat16, device="cuda")
    crisp.kv_append(cache, x, x, ws)
    q = torch.zeros((0, 4, 1, D), dtype=torch.bfloat16, device="cuda")
    crisp.decode_attention(cache, q, torch.empty_like(q), ws)
    other = Pools(2, 1).cache(torch.zeros((0, 1), dtype=torch.int32), torch.zeros(0, dtype=torch.int32))
    crisp.kv_evict(cache, other, torch.zeros((0, 1, 3 * B), device="cuda"), ws, keep=5)
    assert crisp.read_status(ws) == 0
    assert_same_pools(pools, host)


# ------------------------------------------------------------------ together
def test_prefill_store_decode_evict_decode():
    """As a program runs them: a layer is prefilled, its K and V are stored, tokens
    are decoded with weights (in a captured graph), the cache is cut and decoding
    goes on. Each step's output against 64 bits over the values the cache holds."""
    hq, hkv, n, steps, keep = 8, 2, 1000, 5, 640
    q, k, v = synth.small("cache", hq, hkv, n, 41).generate()
    out = crisp.attention(to_dev(q), to_dev(k), to_dev(v))
    assert torch.isfinite(out.float()).all()
    rng = np.random.default_rng(42)
    pages = 9
    table, num = shuffled_table(rng, 1, pages + 6)
    pools = Pools(num, hkv)
    cache = pools.cache([table[0][:pages]], [n])
    weights = torch.zeros((1, hkv, pages * B), device="cuda")
    ws = workspace(max(crisp.decode_workspace_size(cache, hq, 1, True), crisp.kv_append_workspace_size(cache),
                       crisp.kv_evict_workspace_size(cache, keep)))
    crisp.kv_append(cache, to_dev(k)[None], to_dev(v)[None], ws)
    # the stored prompt: each value off by at most half an e4m3 step
    host = pools.host()
    for g in range(hkv):
        for got, x, s in zip(tokens_of(host, table[0], n, g), (to_dev(k), to_dev(v)), (host[2], host[3])):
            x = x[g].double().cpu().numpy()
            scale = np.repeat([float(s[p, g]) for p in table[0][:-(-n // B)]], B)[:n, None]
            assert (np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale)).all()

    def step(cache, pools, tab, length, weights, graph=None):
        kn, vn, qn = (bf16(rng.standard_normal((1, h, 1, D))).cuda() for h in (hkv, hkv, hq))
        o = torch.empty_like(qn)

        def body():
            pools.lens.add_(1)
            crisp.kv_append(cache, kn, vn, ws)
            crisp.decode_attention(cache, qn, o, ws, weights, weights)
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                body()
            g.replay()
        else:
            body()
        assert crisp.read_status(ws) == 0
        want, tol, w, _ = attention(pools.host(), tab, [length], qn.double().cpu().numpy())
        check(o, want, tol)
        return w

    total = 0.0
    for i in range(steps):
        w = step(cache, pools, table, n + 1 + i, weights, graph=i == 2)
        total = total + np.pad(w, ((0, 0), (0, 0), (0, pages * B - w.shape[2])))
    length = n + steps
    got = weights.double().cpu().numpy()
    assert np.abs(got - total)[:, :, :length].max() < 1e-4
    assert abs(got[0, :, :length].sum() - steps * hq) < 1e-3  # each row's weights sum to 1
    new_pages = table[0][pages:pages + 6]
    new_pools = Pools(1, 1)
    new_pools.__dict__.update(k=pools.k, v=pools.v, ks=pools.ks, vs=pools.vs, num_pages=num, hkv=hkv)
    new_cache = new_pools.cache([new_pages], [0])
    new_weights = torch.zeros((1, hkv, 6 * B), device="cuda")
    crisp.kv_evict(cache, new_cache, weights, ws, keep=keep, sink=16, recent=64, new_weights=new_weights)
    assert crisp.read_status(ws) == 0 and int(new_pools.lens[0]) == keep
    kept_mass = new_weights[:, :, :keep].sum((0, 2))
    assert (kept_mass >= weights[:, :, :length].sum((0, 2)) * keep / length).all()  # heavier than the mean
    for i in range(steps):
        step(new_cache, new_pools, [new_pages], keep + 1 + i, new_weights, graph=i == 1)
