"""Attention over packed sequences and the handing out of pages restated on the
CPU (numpy in 64 bits, and plain lists), for their tests."""
import numpy as np
import torch

import dynamic_sparse_prefill_crisp_gb300 as crisp

B, D = 128, 128


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def dev32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def attention(q, k, v, q_lens, k_lens, scale=None):
    """(out, tolerance) of float64 q [tq][hq][128], k, v [tk][hkv][128].

    Tolerance, from the roundings of the documented form:
      ds, of a score: the 128 products (exact in fp32) summed in fp32, each of 132
          additions off by at most 2^-23 of the sum of magnitudes: 2^-15.9;
      p: the score's error and the sum's, the exponential's 2^-20, its own rounding to
          bf16 2^-8;
      sums over n keys in fp32, at most n / 8 + 32 additions one after another, each
          off by 2^-23 of the sum of magnitudes, for out and for the sum of p;
      out: half a bf16 step, 2^-8.
    """
    hq, hkv = q.shape[1], k.shape[1]
    group = hq // hkv
    c = D ** -0.5 if scale is None else scale
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    cq, ck = starts(q_lens), starts(k_lens)
    for b, (nq, nk) in enumerate(zip(q_lens, k_lens)):
        if nq == 0 or nk == 0:
            continue
        pos = nk - nq + np.arange(nq)
        seen = np.arange(nk)[None] <= pos[:, None]
        some = seen.any(-1)
        sums = (nk / 8 + 32) * 2.0 ** -23
        for h in range(hq):
            x, y, z = q[cq[b]:cq[b + 1], h], k[ck[b]:ck[b + 1], h // group], v[ck[b]:ck[b + 1], h // group]
            s = np.where(seen, c * (x @ y.T), -np.inf)
            m = np.where(some, s.max(-1), 0.0)
            p = np.exp(s - m[:, None])
            p /= np.where(some, p.sum(-1), 1.0)[:, None]
            ds = np.where(seen, c * 2.0 ** -15.9 * (np.abs(x) @ np.abs(y).T), 0.0).max(-1)
            o, a = p @ z, p @ np.abs(z)
            out[cq[b]:cq[b + 1], h] = o
            tol[cq[b]:cq[b + 1], h] = (2.0 ** -8 * np.abs(o)
                                       + (2.0 ** -8 + 2.0 ** -20 + 2 * sums + 2 * ds)[:, None] * a + 1e-30)
    return out, tol


def check(got, want, tol):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - want) / np.maximum(tol, 1e-300)) if want.size else 0.0
    assert worst <= 1.0, worst


class Requests:
    """The documented steps of kv_reserve on plain lists."""

    def __init__(self, batch, max_pages, num_pages, free):
        self.batch, self.max_pages, self.num_pages = batch, max_pages, num_pages
        self.table = [[-1] * max_pages for _ in range(batch)]
        self.lens = [0] * batch
        self.stack = list(free)

    def reserve(self, keep, new, max_new, max_all):
        """None where the step cannot be; else what the step holds."""
        kept = [min(n, n if keep is None else keep[b]) for b, n in enumerate(self.lens)]
        new = [0] * self.batch if new is None else list(new)
        total = [k + c for k, c in zip(kept, new)]
        if min(new) < 0 or (keep is not None and min(keep) < 0) or max(total) > B * self.max_pages:
            return None
        if sum(new) > max_new or (max_all and sum(total) > max_all):
            return None
        back = [(b, p) for b in range(self.batch) for p in range(-(-kept[b] // B), -(-self.lens[b] // B))]
        want = [(b, p) for b in range(self.batch) for p in range(-(-kept[b] // B), -(-total[b] // B))]
        if len(want) > len(self.stack) + len(back):
            return None
        for b, p in reversed(back):
            self.stack.append(self.table[b][p])
            self.table[b][p] = -1
        for b, p in want:
            self.table[b][p] = self.stack.pop()
        self.lens = total
        slots, positions, runs, every = [], [], [], []
        for b in range(self.batch):
            for j in range(total[b]):
                slot = self.table[b][j // B] * B + j % B
                every.append(slot)
                if j >= kept[b]:
                    if j == kept[b] or j % B == 0:
                        runs.append(len(slots))
                    slots.append(slot)
                    positions.append(j)
        return dict(cu_new=starts(new), cu_all=starts(total), slots=slots, positions=positions, runs=runs,
                    all_slots=every)
