"""Packed prefill at the edges of its arithmetic and of its lengths, on the GPU against
64 bits."""
import numpy as np
import pytest
import torch

import dynamic_sparse_prefill_crisp_gb300 as crisp
from kv_helpers import VALUES, Pools
from packed_helpers import B, D, attention, check, dev32, starts

pytestmark = pytest.mark.gpu

OK, BOUNDS, PAGES = 0, 8, 9


def workspace(nbytes):
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    crisp.workspace_init(ws)
    return ws


def bf16(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.float32).to(torch.bfloat16)


def call(q, k, v, cu_q, cu_k, status=OK, split=None):
    """out (NaN where nothing was written) of tensors on the CPU; split: whether the plan has to cut tiles."""
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    p = crisp.make_packed(q.shape[1], k.shape[1], dev32(cu_q), dev32(cu_k), q.shape[0], k.shape[0])
    size = crisp.packed_workspace_size(p)
    assert split is None or (size > 256) == split
    ws = workspace(size)
    ws[256:] = 0xFF  # unfinished rows start as NaN
    out = torch.full_like(qd, float("nan"))
    crisp.packed_prefill(p, qd, kd, vd, out, ws)
    assert crisp.read_status(ws) == status
    return out


def inputs(hq, hkv, tq, tk, seed):
    rng = np.random.default_rng(seed)
    return tuple(bf16(rng.standard_normal(s)) for s in ((tq, hq, D), (tk, hkv, D), (tk, hkv, D)))


# ---------------------------------------------------------- the ends of the range
@pytest.mark.parametrize("level", [-960.0, -1000.0, -1040.0, -1400.0])
def test_low_scores_behind_keys_of_minus_infinity(level):
    # the first sub-block's scores are all -inf; the others are around 2^-127 to the base 2 (and on both sides)
    n = 200
    q, k, v = inputs(2, 1, n, n, 81)
    q[:, :, 0] = 1.0
    k[:64, 0, 0] = float("-inf")
    k[64:, 0, 0] = level
    got = call(q, k, v, [0, n], [0, n], split=False)
    want, tol = attention(*(t[64:].double().numpy() for t in (q, k, v)), [n - 64], [n - 64])
    check(got[64:], want, tol)


@pytest.mark.parametrize("tail", [33, 60, 100, 700])
@pytest.mark.parametrize("level", [-960.0, -1000.0, -1040.0])
def test_low_scores_behind_keys_of_minus_infinity_in_parts(level, tail):
    nq, nk = 5, 5000
    q, k, v = inputs(4, 1, nq, nk, 82)
    q[:, :, 0] = 1.0
    k[:nk - tail, 0, 0] = float("-inf")
    k[nk - tail:, 0, 0] = level
    got = call(q, k, v, [0, nq], [0, nk], split=True)
    want, tol = attention(q.double().numpy(), *(t[nk - tail:].double().numpy() for t in (k, v)), [nq], [tail])
    check(got, want, tol)


@pytest.mark.parametrize("nq,nk", [(300, 300), (5, 5000)])
@pytest.mark.parametrize("top", [2.0 ** 104, 2.0 ** 120, 2.0 ** 127])
def test_values_up_to_the_largest(nq, nk, top):
    # sums of p v pass fp32's largest number before they are divided, results do not
    q, k, v = inputs(4, 1, nq, nk, 83)
    v = bf16(torch.sign(v.float()) * (1.0 + 0.9 * torch.frac(v.float().abs())) * top)
    assert torch.isfinite(v).all()
    got = call(q, k, v, [0, nq], [0, nk], split=nk > 1000)
    want, tol = attention(*(t.double().numpy() for t in (q, k, v)), [nq], [nk])
    check(got, want, tol)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_values_that_are_not_finite_beside_sums_out_of_range(value):
    # one feature of one value that every row sees is not finite; the other features' sums leave fp32's range
    # at the first reference: scores grow by 40 binary orders, V is near 2^100
    n = 400
    q, k, v = (x.double().numpy() for x in inputs(4, 1, n, n, 84))
    q[:, :, 0] = 1.0
    q[:, :, 1:] *= 0.1
    k[:, 0, 0] = np.where(np.arange(n) < 64, 0.0, 40.0 * np.log(2.0) * np.sqrt(D))
    v *= 2.0 ** 100
    q, k, v = bf16(q), bf16(k), bf16(v)
    want, tol = attention(*(t.double().numpy() for t in (q, k, v)), [n], [n])
    for key, feature in ((0, 77), (0, 3), (130, 40)):
        w = v.clone()
        w[key, 0, feature] = value
        got = call(q, k, w, [0, n], [0, n])
        rest = [f for f in range(D) if f != feature]
        check(got[..., rest], want[..., rest], tol[..., rest])
        check(got[:key, :, feature], want[:key, :, feature], tol[:key, :, feature])
        hit = got[key:, :, feature].float()
        assert torch.isnan(hit).all() if value != value else (hit == value).all()


@pytest.mark.parametrize("nq,nk", [(300, 300), (5, 5000)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_infinities_beside_sums_out_of_range_of_the_other_sign(nq, nk, value):
    # all of key 130's value is infinite, behind products of p and the values before it, of scores 40 binary
    # orders above the first ones, that pass the largest number with the other sign: not NaN
    q, k, v = inputs(4, 1, nq, nk, 96)
    q[:, :, 0], q[:, :, 1:] = 1.0, 0.1 * q[:, :, 1:]
    k[64:, 0, 0] += 40.0 * np.log(2.0) * np.sqrt(D)
    v = bf16(-np.sign(value) * (1.0 + 0.9 * torch.frac(v.float().abs())) * 2.0 ** 126)
    v[130] = value
    got = call(q, k, v, [0, nq], [0, nk], split=nk > 1000).float()
    first = max(130 - (nk - nq), 0)
    assert (got[first:] == value).all() and torch.isfinite(got[:first]).all()


@pytest.mark.parametrize("nq,nk", [(200, 200), (5, 5000)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("power", [10, 18, 24, 28, 32])
def test_scores_up_to_the_largest(nq, nk, sign, power):
    # scores of one product each, exact, up to the documented 2^30 (2^(power - 2.4)): neighbouring values lie
    # further apart than an exponential reaches, and a row is the mean of its largest score's values
    rng = np.random.default_rng(85 + power)
    q, k, v = inputs(4, 1, nq, nk, 86)
    q[:], k[:] = 0.0, 0.0
    # bf16 keys of 128 magnitudes, each a 2^-8 of the next apart at least
    keys = sign * (128 + rng.integers(0, 128, nk)) / 256.0
    q[:, :, 0] = bf16(2.0 ** (power - power // 2) * (1.0 + rng.integers(0, 128, (nq, 4)) / 128.0))
    k[:, 0, 0] = bf16(keys * 2.0 ** (power // 2))
    got = call(q, k, v, [0, nq], [0, nk], split=nk > 1000)
    x, y, z = (t.double().numpy() for t in (q[:, :, 0], k[:, 0, 0], v[:, 0]))
    want = np.zeros((nq, 4, D))
    tol = np.zeros((nq, 4, D))
    for i in range(nq):
        n = nk - nq + i + 1
        s = x[i][:, None] * y[None, :n] * D ** -0.5
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        want[i] = p @ z[:n]
        # as in attention(), without an error of the scores: a product of 16 bits is exact, and the factor
        # scale * log2 e, off by 2^-23 of itself, changes differences of scores by as much
        tol[i] = 2.0 ** -8 * np.abs(want[i]) + (2.0 ** -8 + 2.0 ** -20 + 2 * (n / 8 + 32) * 2.0 ** -23) * (p @ np.abs(z[:n]))
    check(got, want, tol)


@pytest.mark.parametrize("nq,nk,masked", [(200, 200, 70), (5, 5000, 4998)])
def test_rows_of_minus_infinity_only_become_zeros(nq, nk, masked):
    # the first keys' scores are -inf: rows that see no others are zeros, and the others go by what they see
    q, k, v = inputs(4, 1, nq, nk, 94)
    q[:, :, 0] = 1.0
    k[:masked, 0, 0] = float("-inf")
    got = call(q, k, v, [0, nq], [0, nk], split=nk > 1000)
    zeros = masked - (nk - nq)
    assert not got[:zeros].any()
    want, tol = attention(q[zeros:].double().numpy(), *(t[masked:].double().numpy() for t in (k, v)), [nq - zeros],
                          [nk - masked])
    check(got[zeros:], want, tol)


# ------------------------------------------------------------------- running sums
def rows_of(cu_q, cu_k, total_q, total_k):
    """Which sequences of any sums count, by the documented rule, on plain numbers."""
    n = len(cu_q) - 1
    fine = [0 <= cu_q[b] <= cu_q[b + 1] <= total_q and 0 <= cu_k[b] <= cu_k[b + 1] <= total_k and
            cu_q[b + 1] - cu_q[b] <= 1 << 20 and cu_k[b + 1] - cu_k[b] <= 1 << 20 for b in range(n)]
    return [fine[b] and not any(fine[c] and cu_q[c + 1] > cu_q[b] for c in range(b)) for b in range(n)]


def against_the_rule(q, k, v, cu_q, cu_k, split):
    good = rows_of(cu_q, cu_k, q.shape[0], k.shape[0])
    got = call(q, k, v, cu_q, cu_k, status=OK if all(good) else BOUNDS, split=split)
    left = np.ones(q.shape[0], dtype=bool)
    for b, ok in enumerate(good):
        if not ok or cu_q[b] == cu_q[b + 1]:
            continue
        at, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        want, tol = attention(*(t.double().numpy() for t in (q[at], k[keys], v[keys])), [at.stop - at.start],
                              [keys.stop - keys.start])
        check(got[at], want, tol)
        left[at] = False
    assert torch.isnan(got[torch.from_numpy(left).cuda()]).all()


@pytest.mark.parametrize("cu_q", [[0, 2 ** 30, 40, 120], [0, 2 ** 30, 90, 120], [-5, 30, 40, 120],
                                  [100, 30, 40, 120], [0, 2 ** 31 - 1, 40, 120], [0, 30, 121, 120]])
def test_bad_sums_between_split_sequences(cu_q):
    q, k, v = inputs(4, 1, 120, 6000, 87)
    against_the_rule(q, k, v, cu_q, [0, 2000, 4000, 6000], split=True)


@pytest.mark.parametrize("cu_k", [[0, 2 ** 30, 2000, 6000], [0, 4000, 2000, 6000], [-1, 2000, 4000, 6001],
                                  [0, 3000, 0, 3000]])
def test_bad_key_sums_between_split_sequences(cu_k):
    q, k, v = inputs(4, 1, 120, 6000, 88)
    against_the_rule(q, k, v, [0, 40, 80, 120], cu_k, split=True)


def test_bad_sums_among_many_split_sequences():
    # 75 sequences of 3 queries, each behind 200 keys but two; sums in the middle that are none
    k_lens = [200] * 75
    k_lens[5], k_lens[50] = 9000, 7000
    cu_q, cu_k = starts([3] * 75), starts(k_lens)
    q, k, v = inputs(4, 1, int(cu_q[-1]), int(cu_k[-1]), 89)
    for at, value in ((10, 2 ** 30), (33, -1), (70, 2 ** 31 - 1)):
        sums = cu_q.copy()
        sums[at] = value
        against_the_rule(q, k, v, sums.tolist(), cu_k.tolist(), split=True)


@pytest.mark.parametrize("cu_q,cu_k", [
    ([0, 100, 0, 100], [0, 2000, 4000, 6000]),           # the same rows twice
    ([0, 100, 0, 100, 0, 100, 0, 100], [0, 900, 900, 1800, 1800, 2700, 2700, 6000]),  # more tiles than rows have
    ([0, 40, 20, 120], [0, 2000, 4000, 6000]),           # rows 20 to 39 twice
    ([0, 120, 40, 80], [0, 2000, 4000, 6000]),           # inside an earlier one's
    ([0, 40, 20, 30, 60, 120], [0, 1000, 2000, 3000, 4000, 6000]),  # after one that counts as empty itself
    ([50, 120, 0, 50], [0, 2000, 4000, 6000])])          # apart, the later rows first
def test_sequences_that_share_rows(cu_q, cu_k):
    q, k, v = inputs(4, 1, 120, 6000, 90)
    against_the_rule(q, k, v, cu_q, cu_k, split=True)
    # and where tiles are whole
    against_the_rule(q, k[:120], v[:120], cu_q, [x // 50 for x in cu_k], split=False)


def test_sequences_that_share_rows_among_many():
    k_lens = [200] * 75
    k_lens[5], k_lens[50] = 9000, 7000
    cu_q, cu_k = starts([3] * 75), starts(k_lens)
    q, k, v = inputs(4, 1, int(cu_q[-1]), int(cu_k[-1]), 91)
    for at, value in ((33, 0), (40, 7), (70, 140), (20, 80)):
        sums = cu_q.copy()
        sums[at] = value
        against_the_rule(q, k, v, sums.tolist(), cu_k.tolist(), split=True)


# ------------------------------------------------------------- tiles done again
@pytest.mark.parametrize("q_lens,k_lens", [([900, 300], [900, 300]), ([40, 30], [7000, 3001])])
def test_tiles_done_again_read_what_was_copied(q_lens, k_lens):
    # every tile holds values that are not finite in its last keys and behind them: both slots of V are looked
    # through again and again, and each time the same bits come out
    cu_q, cu_k = starts(q_lens), starts(k_lens)
    q, k, v = inputs(14, 2, int(cu_q[-1]), int(cu_k[-1]), 92)
    clean = call(q, k, v, cu_q, cu_k)
    w = v.clone()
    odd = torch.zeros(v.shape[0], dtype=torch.bool)
    for b, (nq, nk) in enumerate(zip(q_lens, k_lens)):
        odd[cu_k[b] + nk - nq + 5:cu_k[b + 1]:9] = True
    w[odd, :, 5], w[odd, :, 90] = float("inf"), float("nan")
    got = call(q, k, w, cu_q, cu_k)
    rest = [f for f in range(D) if f not in (5, 90)]
    seen = torch.zeros(q.shape[0], dtype=torch.bool)
    for b in range(2):
        first = int(cu_q[b]) + 5
        seen[first:cu_q[b + 1]] = True
    assert torch.equal(got[~seen], clean[~seen]) and torch.equal(got[..., rest], clean[..., rest])
    assert torch.isnan(got[seen][..., 90]).all() and (got[seen][..., 5] == float("inf")).all()
    for _ in range(20):
        again = call(q, k, w, cu_q, cu_k)
        assert torch.equal(again.view(torch.int16), got.view(torch.int16))


# --------------------------------------------------------------------- the cache
def test_rows_of_a_cache_without_sequences():
    pools = Pools(3, 2)
    codes = np.random.default_rng(93).integers(0, 127, (3, 2, B, D)).astype(np.uint8)
    for t, s in ((pools.k, pools.ks), (pools.v, pools.vs)):
        t.copy_(torch.from_numpy(codes))
        s.fill_(2.0)
    cache = crisp.make_kv_cache(pools.k, pools.v, pools.ks, pools.vs, torch.empty((0, 4), dtype=torch.int32, device="cuda"),
                                torch.empty(0, dtype=torch.int32, device="cuda"))
    ws = workspace(crisp.kv_append_workspace_size(cache))
    slots = np.arange(0, 3 * B, 5)
    outs = [torch.full((len(slots), 2, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    crisp.kv_gather(cache, dev32(slots), *outs, ws)
    assert crisp.read_status(ws) == OK
    for out in outs:
        assert np.array_equal(out.double().cpu().numpy(), VALUES[codes[slots // B, :, slots % B]] * 2.0)


def test_decode_behind_a_refused_step_goes_by_the_lengths_from_before():
    hq, hkv = 4, 2
    pools = Pools(5, hkv)
    cache = pools.cache([[-1] * 4] * 2, [0, 0])
    free, num = dev32(range(5)), dev32([5])
    step = crisp.make_kv_step(cache, 600, 1024)
    ws = workspace(crisp.kv_append_workspace_size(cache))
    q, k, v = (t.cuda() for t in inputs(hq, hkv, 2, 600, 95))
    crisp.kv_reserve(cache, free, num, step, ws, new_lens=dev32([300, 200]))
    crisp.kv_append_packed(cache, step, k, v, ws)
    dws = workspace(crisp.decode_workspace_size(cache, hq))
    one = q.unsqueeze(2)
    before, after = torch.empty_like(one), torch.empty_like(one)
    crisp.decode_attention(cache, one, before, dws)
    assert crisp.read_status(ws) == OK
    crisp.kv_reserve(cache, free, num, step, ws, new_lens=dev32([10, 300]))
    assert crisp.read_status(ws) == PAGES and pools.lens.tolist() == [300, 200]
    crisp.kv_append_packed(cache, step, 2 * k, 2 * v, ws)
    crisp.decode_attention(cache, one, after, dws)
    assert crisp.read_status(dws) == OK and torch.equal(before, after)
