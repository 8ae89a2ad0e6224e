"""The 8-bit cache restated in 64 bits on the CPU (numpy), for its tests."""
import numpy as np
import torch

import dynamic_sparse_prefill_crisp_gb300 as crisp

B, D = 128, 128
MIN_EXP = -100


def code_values():
    """The 256 e4m3 codes' values from the format: 1 sign, 4 exponent (bias 7), 3 mantissa bits; 0x7f is NaN."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


VALUES = code_values()


def round_codes(x):
    """Nearest e4m3 code (even code on a tie) of |x| <= 448; NaN for a non-finite x."""
    mags = VALUES[:127]  # ascending, 0 .. 448
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(mags, a, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = a - mags[lo], mags[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isfinite(x), code, 127)
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def page_exponent(x):
    """The smallest e >= MIN_EXP with every finite |x| <= 448 * 2^e."""
    a = np.abs(x[np.isfinite(x)])
    amax = a.max() if a.size else 0.0
    e = MIN_EXP
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return e


class Pools:
    """A pool on the GPU with every byte set (NaN codes and odd scales where nothing is written)."""

    def __init__(self, num_pages, hkv, interleaved=False, seed=0):
        n = num_pages * hkv * B * D
        if interleaved:  # [page][k, v][head][128][128]
            both = torch.full((num_pages, 2, hkv, B, D), 0x7F, dtype=torch.uint8, device="cuda")
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = (torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda").view(num_pages, hkv, B, D)
                              for _ in range(2))
        self.ks, self.vs = (torch.full((num_pages, hkv), float("nan"), device="cuda") for _ in range(2))
        self.num_pages, self.hkv = num_pages, hkv

    def cache(self, table, lens):
        self.table = torch.as_tensor(table, dtype=torch.int32).cuda().contiguous()
        self.lens = torch.as_tensor(lens, dtype=torch.int32).cuda()
        return crisp.make_kv_cache(self.k, self.v, self.ks, self.vs, self.table, self.lens)

    def host(self):
        """(k codes, v codes, k scales, v scales) as numpy copies."""
        return (self.k.cpu().numpy().copy(), self.v.cpu().numpy().copy(), self.ks.cpu().numpy().copy(),
                self.vs.cpu().numpy().copy())


def fill(pools, table, lens, rng, spread=0.0, sink=1.0):
    """Writes random tokens through the reference rule; page scales differ by up to 2^spread."""
    k, v, ks, vs = pools.host()
    for b, n in enumerate(lens):
        for p in range(-(-n // B)):
            rows = min(B, n - p * B)
            for g in range(pools.hkv):
                for codes, scales, mul in ((k, ks, sink if p == 0 else 1.0), (v, vs, 1.0)):
                    x = rng.standard_normal((rows, D)) * mul * 2.0 ** rng.uniform(-spread, spread)
                    e = page_exponent(x)
                    scales[table[b][p], g] = 2.0 ** e
                    codes[table[b][p], g, :rows] = round_codes(x / 2.0 ** e)
    pools.k.copy_(torch.from_numpy(k))
    pools.v.copy_(torch.from_numpy(v))
    pools.ks.copy_(torch.from_numpy(ks))
    pools.vs.copy_(torch.from_numpy(vs))


def tokens_of(host, table_row, n, g):
    """(keys, values) [n][128] in 64 bits of one sequence and head."""
    k, v, ks, vs = host
    out = []
    for codes, scales in ((k, ks), (v, vs)):
        pages = [VALUES[codes[table_row[p], g]] * float(scales[table_row[p], g]) for p in range(-(-n // B))]
        out.append(np.concatenate(pages)[:n] if pages else np.zeros((0, D)))
    return out


def attention(host, table, lens, q, scale=None):
    """out, sum of weights and their tolerances. q: float64 [batch][hq][q_len][128].

    Tolerances, from the roundings of the documented forms:
      ds, of a score: the 128 products' sums in fp32 (each addition at most 2^-23 of the
          sum of magnitudes when it truncates, 132 of them with the scaling: 2^-15.9) and
          q's two pieces (2^-18 of the row's largest element times sum |k|);
      p: its own rounding 2^-8, the score's error, the exponential's 2^-20;
      out: p's error on sum p |v|, the fp32 sums (2^-16 of it), half a bf16 step 2^-8.
    """
    batch, hq, t, _ = q.shape
    hkv = host[0].shape[1]
    group = hq // hkv
    c = D ** -0.5 if scale is None else scale
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    cap = max(1, max(-(-n // B) for n in lens)) * B
    w, wtol = np.zeros((batch, hkv, cap)), np.zeros((batch, hkv, cap))
    for b, n in enumerate(lens):
        for g in range(hkv):
            k, v = tokens_of(host, table[b], n, g)
            for i in range(t):
                end = n - (t - 1 - i)
                if end <= 0:
                    continue
                for h in range(g * group, (g + 1) * group):
                    row = q[b, h, i]
                    s = c * (k[:end] @ row)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    ds = c * (2.0 ** -15.9 * (np.abs(k[:end]) @ np.abs(row))
                              + 2.0 ** -18 * np.abs(row).max() * np.abs(k[:end]).sum(-1))
                    dp = 2 * ds.max() + 2.0 ** -20  # own score and the sum's
                    a = p @ np.abs(v[:end])
                    out[b, h, i] = p @ v[:end]
                    tol[b, h, i] = 2.0 ** -8 * np.abs(out[b, h, i]) + (2.0 ** -8 + dp + 2.0 ** -16) * a + 1e-30
                    w[b, g, :end] += p
                    wtol[b, g, :end] += p * (dp + 2.0 ** -19)
    return out, tol, w, wtol


def shuffled_table(rng, batch, pages, spare=2):
    """Pages in a random order; returns (table, pages in the pool)."""
    num = batch * pages + spare
    return rng.permutation(num)[:batch * pages].reshape(batch, pages).tolist(), num
