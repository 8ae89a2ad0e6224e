"""The paged 8-bit cache on the GPU at the edges of its values and of its use."""
import os
import re
import threading

import numpy as np
import pytest
import torch

import dynamic_sparse_prefill_crisp_gb300 as crisp
from kv_helpers import B, D, Pools, attention, fill, page_exponent, round_codes, shuffled_table, tokens_of

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def workspace(nbytes):
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    crisp.workspace_init(ws)
    return ws


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("exponents", [(28, 28), (60, 28), (120, 100), (27, 120), (-100, 120), (-100, -90)])
@pytest.mark.parametrize("beside", ["zeros", "smallest-scale"])
def test_evict_keeps_zeros_of_pages_with_any_scale(exponents, beside):
    # Two old pages at scales 2^exponents: rows of zeros among large ones, and a
    # third page at the smallest scale. What stays is the rows of zeros (of both
    # signs), alone or beside rows of the third page: the new pages' scale is then
    # 2^-100 or near it, whatever their old pages' scales were.
    rng = np.random.default_rng(61)
    src, dst = Pools(3, 1), Pools(3, 1)
    k, v, ks, vs = src.host()
    for codes, scales in ((k, ks), (v, vs)):
        codes[:] = round_codes(rng.standard_normal(codes.shape) * 100.0)
        for p, e in enumerate((*exponents, -100)):
            scales[p] = 2.0 ** e
        codes[:2, 0, ::2] = rng.choice(np.array([0, 128], np.uint8), codes[:2, 0, ::2].shape)
    for t, a in zip((src.k, src.v, src.ks, src.vs), (k, v, ks, vs)):
        t.copy_(torch.from_numpy(a))
    w = torch.zeros((1, 1, 3 * B), device="cuda")
    w[..., :2 * B:4] = 1.0
    keep = B // 2
    if beside == "smallest-scale":  # in the same new page
        w[..., 2 * B + 5::2] = 2.0
        keep += int((w == 2.0).sum())
    pos = torch.nonzero(w[0, 0]).flatten().cpu().numpy()
    assert pos.size == keep
    cache = src.cache([[0, 1, 2]], [3 * B])
    new_cache = dst.cache([[2, 0]], [0])
    ws = workspace(crisp.kv_evict_workspace_size(cache, keep))
    crisp.kv_evict(cache, new_cache, w, ws, keep=keep)
    assert crisp.read_status(ws) == 0
    got = dst.host()
    for x, codes, scales in zip(tokens_of((k, v, ks, vs), [0, 1, 2], 3 * B, 0), got[:2], got[2:]):
        for p, page in enumerate((2, 0)):
            rows = x[pos[p * B:(p + 1) * B]]
            if len(rows) == 0:
                continue
            e = 2.0 ** page_exponent(rows)
            assert float(scales[page, 0]) == e
            want = round_codes(rows / e)
            sign = np.where(want & 127, 255, 127)  # -0 and 0 are one value
            assert np.array_equal(codes[page, 0, :len(rows)] & sign, want & sign)


# ------------------------------------------------------------- host threads
def in_threads(calls):
    """Runs the functions at once, a fresh host thread each; raises what one of them raised."""
    start, errors = threading.Barrier(len(calls)), []

    def run(f):
        try:
            start.wait()
            f()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(f,)) for f in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("own_stream", [False, True])
def test_the_first_call_of_a_host_thread(own_stream):
    # Threads that have called nothing of CUDA's before: no context is current there.
    gen = torch.Generator(device="cuda").manual_seed(63)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)

    pools = Pools(8, 2)
    cache = pools.cache([[0, 3], [5, 1]], [200, 256])
    k, v, q = rand(2, 2, 256, D), rand(2, 2, 256, D), rand(2, 8, 1, D)
    ws = [workspace(crisp.decode_workspace_size(cache, 8)) for _ in range(2)]
    crisp.kv_append(cache, k, v, ws[0], new_lens=cache.tensors[5])
    want = torch.empty_like(q)
    crisp.decode_attention(cache, q, want, ws[0])
    lq, lk, lv = rand(4, 1000, D), rand(1, 1000, D), rand(1, 1000, D)
    layer_want = crisp.attention(lq, lk, lv)
    shape = crisp.make_shape(4, 1, 1000, lq, lk, lq)
    lws = workspace(crisp.layer_workspace_size(shape))
    layer_out, out = torch.zeros_like(lq), torch.zeros_like(q)
    stream = torch.cuda.Stream() if own_stream else None
    params = crisp.params_default()
    torch.cuda.synchronize()
    for call in (lambda: crisp.decode_attention(cache, q, out, ws[1], stream=stream),
                 lambda: crisp.prefill_layer(shape, params, lq, lk, lv, layer_out, lws, stream=stream)):
        in_threads([call])
    torch.cuda.synchronize()
    assert crisp.read_status(ws[1]) == 0 and crisp.read_status(lws) == 0
    assert torch.equal(out, want) and torch.equal(layer_out, layer_want)


def again_and_again(f, args, times):
    """The C call, with its arguments made beforehand: threads meet inside the library as often as they can."""
    def run():
        for _ in range(times):
            rc = f(*args)
            assert rc == 0, rc
    return run


def test_host_threads_decode_batches_of_any_size_at_once():
    # Each thread has a cache, stream, workspace and outputs of its own; only the
    # batch, and with it the shared memory that a launch asks for, differs.
    gen = torch.Generator(device="cuda").manual_seed(62)
    jobs, calls = [], []
    for hq, batch in [(2, 1), (2, 1024)] * 4 + [(16, 1), (16, 1024), (28, 1), (28, 1024)]:
        pools = Pools(batch + 2, 1)
        for t in (pools.k, pools.v):
            t.copy_(torch.randint(0, 127, t.shape, generator=gen, device="cuda", dtype=torch.uint8))
        for t in (pools.ks, pools.vs):
            t.fill_(2.0 ** -8)
        cache = pools.cache([[b + 1] for b in range(batch)], [77] + [0] * (batch - 2) + [5] * (batch > 1))
        q = torch.randn((batch, hq, 1, D), generator=gen, device="cuda").to(torch.bfloat16)
        ws = workspace(crisp.decode_workspace_size(cache, hq))
        want, out, stream = torch.empty_like(q), torch.zeros_like(q), torch.cuda.Stream()
        crisp.decode_attention(cache, q, want, ws)
        qt, ot = (crisp.Tokens(t.data_ptr(), *t.stride()[:3]) for t in (q, out))
        jobs.append((cache, q, out, ws, want, stream))
        calls.append(again_and_again(crisp.lib().crisp_decode_attention,
                                     (cache, hq, 1, 0.0, qt, ot, None, None, ws.data_ptr(), ws.numel(),
                                      stream.cuda_stream), 4000))
    torch.cuda.synchronize()
    in_threads(calls)
    torch.cuda.synchronize()
    for _, _, out, ws, want, _ in jobs:
        assert crisp.read_status(ws) == 0 and torch.equal(out, want)


def test_host_threads_select_blocks_of_any_length_at_once():
    # The prefill's block selection, whose launches ask for shared memory by the length.
    gen = torch.Generator(device="cuda").manual_seed(64)
    jobs, calls, params = [], [], crisp.params_default()
    for n in [256, 128 * 1000] * 4 + [128 * 1100, 128 * 2000]:
        nb = n // B
        x = torch.empty((1, n, D), dtype=torch.bfloat16, device="cuda")
        shape = crisp.make_shape(1, 1, n, x, x, x)
        pbar = torch.softmax(torch.randn((1, nb, nb), generator=gen, device="cuda"), -1)
        route = torch.zeros(1, dtype=torch.uint8, device="cuda")
        ws = workspace(crisp.workspace_size(shape))
        bits = torch.zeros((1, nb, (nb + 31) // 32), dtype=torch.int32, device="cuda")
        want = torch.zeros_like(bits)
        crisp.select_pe(shape, params, pbar, route, want, ws)
        stream = torch.cuda.Stream()
        jobs.append((pbar, route, bits, ws, want, stream))
        calls.append(again_and_again(crisp.lib().crisp_select_pe,
                                     (shape, params, pbar.data_ptr(), route.data_ptr(), bits.data_ptr(),
                                      ws.data_ptr(), ws.numel(), stream.cuda_stream), 4000))
    torch.cuda.synchronize()
    in_threads(calls)
    torch.cuda.synchronize()
    for _, _, bits, ws, want, _ in jobs:
        assert crisp.read_status(ws) == 0 and torch.equal(bits, want)


# ----------------------------------------------------------- non-finite rows
@pytest.mark.parametrize("hq,hkv,q_len,lens", [(4, 2, 3, [130, 129, 128, 2, 1, 0]), (2, 1, 16, [300, 130, 9]),
                                               (32, 1, 2, [257, 1]), (40, 1, 2, [200])])
def test_weights_of_keys_that_a_non_finite_row_does_not_see(hq, hkv, q_len, lens):
    # The first token's first head is NaN (or infinite): its softmax, and with it the
    # weight of every key that it sees, is NaN. The last q_len - 1 keys it does not see.
    rng = np.random.default_rng(65)
    pages = max(1, max(-(-n // B) for n in lens))
    table, num = shuffled_table(rng, len(lens), pages)
    pools = Pools(num, hkv)
    fill(pools, table, lens, rng)
    cache = pools.cache(table, lens)
    q = torch.from_numpy(rng.standard_normal((len(lens), hq, q_len, D))).to(torch.bfloat16)
    _, _, w, wtol = attention(pools.host(), table, lens, q.double().numpy())
    for bad in (float("nan"), float("inf")):
        q[:, 0, 0, 7] = bad
        w_in = torch.rand((len(lens), hkv, cache.max_pages * B), generator=torch.Generator().manual_seed(1)).cuda()
        w_out = torch.full_like(w_in, -7.0)
        qd = q.cuda()
        ws = workspace(crisp.decode_workspace_size(cache, hq, q_len, True))
        crisp.decode_attention(cache, qd, torch.empty_like(qd), ws, w_in, w_out)
        assert crisp.read_status(ws) == 0
        got, base = w_out.double().cpu().numpy(), w_in.double().cpu().numpy()
        for b, n in enumerate(lens):
            seen = max(n - (q_len - 1), 0)
            assert np.isnan(got[b, 0, :seen]).all() and (got[b, :, n:] == -7.0).all()
            for g in range(hkv):
                lo = seen if g == 0 else 0
                err = np.abs(got[b, g, lo:n] - base[b, g, lo:n] - w[b, g, lo:n])
                assert (err <= wtol[b, g, lo:n] + 2.0 ** -24 * np.abs(got[b, g, lo:n])).all()


# ------------------------------------------------------- small weights beside large ones
@pytest.mark.parametrize("n", [3, 128, 200, 256, 1000])
@pytest.mark.parametrize("sink_v", ["zero", "plain"])
def test_decode_small_weights_beside_a_large_one(n, sink_v):
    # Rows whose first key stands 2 to 24 nats above all others, with V = 0 there:
    # what the row puts out comes from the small p alone.
    # Tolerance: kv_helpers.attention's, and for each key 2^-22 of the row's largest p
    # among the keys of its product (256 at most: within 255 positions), times |v|.
    # That is half the smallest step of the second piece: e4m3's 2^-9, over its scale
    # 16, over 2, over the 256 that the largest p is scaled to.
    rng = np.random.default_rng(66)
    gaps = [2, 6, 8, 10, 12, 13, 14, 15, 16, 17, 20, 24]
    hq = len(gaps)
    table, num = shuffled_table(rng, 1, -(-n // B))
    pools = Pools(num, 1)
    fill(pools, table, [n], rng)
    k, v, ks, vs = pools.host()
    first = table[0][0]
    # feature 0 carries the gap: 64 at the first key, 0 elsewhere
    for p in table[0]:
        k[p, 0, :, 0] = 0
        k[p, 0, :, 1:] = round_codes(rng.standard_normal((B, D - 1)))
        ks[p, 0] = 0.25
    k[first, 0, 0, 0] = round_codes(np.array([256.0]))[0]
    k[first, 0, 0, 1:] = 0
    if sink_v == "zero":
        v[first, 0, 0] = 0
    for t, a in zip((pools.k, pools.v, pools.ks, pools.vs), (k, v, ks, vs)):
        t.copy_(torch.from_numpy(a))
    q = rng.standard_normal((1, hq, 1, D)) * 0.25
    q[0, :, 0, 0] = np.array(gaps) / 64.0
    q = torch.from_numpy(q).to(torch.bfloat16)
    cache = pools.cache(table, [n])
    host = pools.host()
    want, tol, w, wtol = attention(host, table, [n], q.double().numpy(), scale=1.0)
    keys, vals = tokens_of(host, table[0], n, 0)
    for h in range(hq):
        s = keys @ q[0, h, 0].double().numpy()
        p = np.exp(s - s.max()) / np.exp(s - s.max()).sum()
        top = np.array([p[max(0, j - 255):j + 256].max() for j in range(n)])
        tol[0, h, 0] += 2.0 ** -22 * (top @ np.abs(vals))
    qd = q.cuda()
    out, weights = torch.full_like(qd, float("nan")), torch.zeros((1, 1, cache.max_pages * B), device="cuda")
    ws = workspace(crisp.decode_workspace_size(cache, hq, 1, True))
    crisp.decode_attention(cache, qd, out, ws, None, weights, scale=1.0)
    assert crisp.read_status(ws) == 0
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    got = weights.double().cpu().numpy()[:, :, :n]  # the weights have no such floor
    assert (np.abs(got - w[:, :, :n]) <= wtol[:, :, :n] + 2.0 ** -24 * np.abs(got)).all()


# ------------------------------------------------------------------ the example
def test_the_documented_example_of_the_cache():
    # The two blocks of the user's guide, as they stand there, with memory that starts
    # as NaN; then a token over the smaller cache. A row's weights sum to 1.
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), re.S)
    blocks = [b for b in blocks if "make_kv_cache" in b]
    assert len(blocks) == 2
    batch, hq, hkv, n, max_pages = 2, 8, 2, 4500, 40
    gen = torch.Generator(device="cuda").manual_seed(67)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)

    names = dict(torch=torch, crisp=crisp, batch=batch, hq=hq, hkv=hkv, n=n, max_pages=max_pages,
                 pages=batch * (max_pages + 50), k=rand(batch, hkv, n, D), v=rand(batch, hkv, n, D),
                 k_new=rand(batch, hkv, 1, D), v_new=rand(batch, hkv, 1, D), q=rand(batch, hq, 1, D))
    names["out"] = torch.empty_like(names["q"])
    torch.use_deterministic_algorithms(True, warn_only=True)  # fills torch.empty
    try:
        for b in blocks:
            exec(b, names)
    finally:
        torch.use_deterministic_algorithms(False)
    weights, small, small_weights, ws = (names[x] for x in ("weights", "small", "small_weights", "ws"))
    rows = hq // hkv
    assert torch.allclose(weights.double().sum(-1), torch.full((), float(rows), dtype=torch.float64, device="cuda"), rtol=1e-5)
    assert (weights[..., n + 1:] == 0).all() and small.tensors[5].tolist() == [4096] * batch
    before = small_weights.double().sum(-1)
    small.tensors[5].add_(1)
    crisp.kv_append(small, names["k_new"], names["v_new"], ws)
    crisp.decode_attention(small, names["q"], names["out"], ws, small_weights, small_weights)
    assert crisp.read_status(ws) == 0 and crisp.read_status(names["ws2"]) == 0
    assert torch.isfinite(names["out"].float()).all()
    assert torch.allclose(small_weights.double().sum(-1), before + rows, rtol=1e-5)
    assert (small_weights[..., 4096] > 0).all() and (small_weights[..., 4097:] == 0).all()
