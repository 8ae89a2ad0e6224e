"""Packed prefill at the edges of its arithmetic and of its lengths, on the GPU against
64 bits."""
import numpy as np
import pytest
import torch

import dynamic_sparse_prefill_crisp_gb300 as crisp
from packed_helpers import D, attention, check, dev32

pytestmark = pytest.mark.gpu

OK, BOUNDS = 0, 8


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
