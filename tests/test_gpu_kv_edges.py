"""The paged 8-bit cache on the GPU at the edges of its values and of its use."""
import numpy as np
import pytest
import torch

import dynamic_sparse_prefill_crisp_gb300 as crisp
from kv_helpers import B, Pools, page_exponent, round_codes, tokens_of

pytestmark = pytest.mark.gpu


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
