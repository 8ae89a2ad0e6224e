"""The operators around a batch of packed sequences as measured: attention over
prompts of different lengths (whole, or going on from what is cached), handing
out cache pages from request lengths, storing packed tokens into those pages,
and reading cached tokens back.

``own = False`` computes each operator in its plain form (elementary torch
operations in 32 bits); ``own = True`` makes the calls a user makes of the
package. ``exact`` restates the computed values from their definition in 64 bits.
"""
import math

import torch

own = False

B = 128  # tokens of a page
D = 128  # features
MIN_EXP = -100  # the smallest exponent of a page's scale


# --------------------------------------------------------------------- cases
def _attend(name, batch, hq, hkv, low, cap, past_low, past_cap):
    return dict(name=name, op="attend", batch=batch, hq=hq, hkv=hkv, low=low, cap=cap, past_low=past_low, past_cap=past_cap)


def _reserve(name, batch, new_low, new_cap, keep_cap, replaced, all_slots):
    return dict(name=name, op="reserve", batch=batch, new_low=new_low, new_cap=new_cap, keep_cap=keep_cap, replaced=replaced,
                all_slots=all_slots)


def _append(name, batch, hkv, low, cap, before):
    return dict(name=name, op="append", batch=batch, hkv=hkv, low=low, cap=cap, before=before)


def _gather(name, batch, hkv, low, cap):
    return dict(name=name, op="gather", batch=batch, hkv=hkv, low=low, cap=cap)


def listed():
    return [
        # one user's short prompt: latency
        _attend("attend-4x1-300", 1, 4, 1, 300, 300, 0, 0),
        # a server's batch of short questions
        _attend("attend-28x4-short", 256, 28, 4, 1, 300, 0, 0),
        # prompts of any length up to 4k, packed
        _attend("attend-32x8-ragged", 16, 32, 8, 1, 4096, 0, 0),
        # one long prompt
        _attend("attend-32x8-16k", 1, 32, 8, 16384, 16384, 0, 0),
        # four long prompts, each going on by a chunk of 512 tokens
        _attend("attend-28x4-chunks", 4, 28, 4, 512, 512, 4001, 49152),
        # the last 40 tokens of a question over a 128k document
        _attend("attend-32x8-question", 1, 32, 8, 40, 40, 131072, 131072),
        # a decode step: a token for each of 64 sequences
        _reserve("reserve-step-64", 64, 1, 1, 8191, 0.0, False),
        # a third of 512 requests done and replaced, the others going on by a chunk; slots of everything held
        _reserve("reserve-turnover-512", 512, 0, 1000, 1500, 0.34, True),
        # the token that a decode step adds to each of 64 sequences
        _append("append-1-of-64", 64, 8, 1, 1, 4100),
        # chunks of 1 to 4096 tokens of 48 sequences at odd offsets
        _append("append-ragged-48", 48, 8, 1, 4096, 3001),
        # a short shared system prompt read back for one request
        _gather("gather-1x700", 1, 4, 700, 700),
        # 16 cached contexts of up to 16k tokens
        _gather("gather-16x16k", 16, 8, 1000, 16384),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    hq, hkv = rng.choice([(4, 1), (32, 8), (28, 4), (16, 1), (8, 8)])
    op = rng.choice(["attend", "attend", "attend", "reserve", "append", "gather"])
    if op == "attend":
        cap, past = log(1, 16384), rng.choice([0, 0, log(1, 131072)])
        # at most the (row, key) pairs of the largest listed case, twice counted
        most = (32 * 16384 ** 2) // hq
        while cap * (cap + 2 * past) > most:
            cap, past = max(1, cap // 2), past // 2
        batch = max(1, min(log(1, 256), most // (cap * (cap + 2 * past)), 400_000 // (cap + past)))
        low = cap if rng.random() < 0.3 else max(1, int(cap * rng.uniform(0.0, 1.0)))
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, low=low, cap=cap, past_low=int(past * rng.uniform(0.0, 1.0)), past_cap=past)
    if op == "reserve":
        batch = log(1, 1024)
        most = 400_000 // batch
        new_cap = rng.choice([1, min(most, log(1, 8000))])
        return dict(op=op, batch=batch, new_low=rng.choice([0, 1]), new_cap=new_cap, keep_cap=min(most, log(1, 8000)),
                    replaced=rng.choice([0.0, rng.random()]), all_slots=rng.random() < 0.5)
    batch = log(1, 128)
    most = 131_072 * 8 // (batch * hkv) if op == "gather" else 98_304 * 8 // (batch * hkv)
    cap = max(1, min(most, log(1, 65536)))
    low = cap if rng.random() < 0.3 else max(1, int(cap * rng.uniform(0.0, 1.0)))
    if op == "append":
        return dict(op=op, batch=batch, hkv=hkv, low=low, cap=cap, before=rng.choice([0, min(most, log(1, 9000))]))
    return dict(op=op, batch=batch, hkv=hkv, low=low, cap=cap)


# -------------------------------------------------------------------- inputs
def _lens(salt, batch, low, cap):
    """Lengths between the bounds, one of them the longest, on the CPU: the same ones for every seed, in another order."""
    gen = torch.Generator()
    gen.manual_seed(salt)
    n = torch.randint(low, cap + 1, (batch,), generator=gen)
    n[0] = cap
    return n


def _order(seed, batch):
    gen = torch.Generator()
    gen.manual_seed(seed)
    return torch.randperm(batch, generator=gen)


def _starts(n):
    """0 and the running sums."""
    return torch.cat([torch.zeros(1, dtype=torch.int64), n.long().cumsum(0)]).to(torch.int32).cuda()


def _pages(n):
    return (n + B - 1) // B


def _keys(shape, gen):
    """Keys [tokens][heads][128] with channels of different strength, as trained layers have."""
    chan = torch.exp(0.5 * torch.randn((shape[1], D), generator=gen, device="cuda"))
    return (torch.randn(shape, generator=gen, device="cuda") * chan).to(torch.bfloat16)


def _exponent(amax):
    """The smallest e >= MIN_EXP with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)


def _pow2(e):
    """2^e in 32 bits, from its bits (a computed power is off in its last place)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise_pages(x):
    """[..., 128, 128] values -> e4m3 codes and a scale for each page."""
    x = x.float()
    s = _pow2(_exponent(x.abs().amax((-1, -2))))
    return (x / s[..., None, None]).to(torch.float8_e4m3fn), s


def _pool(st, num, hkv, gen):
    """A pool of `num` pages with codes in every row."""
    for name in ("k", "v"):
        st[name + "8"] = torch.empty((num, hkv, B, D), dtype=torch.float8_e4m3fn, device="cuda")
        st[name + "_scale"] = torch.empty((num, hkv), device="cuda")
        for at in range(0, num, 512):
            n = min(512, num - at)
            x = torch.randn((n, hkv, B, D), generator=gen, device="cuda") * torch.exp(torch.randn((n, hkv, 1, 1), generator=gen, device="cuda"))
            c, s = _quantise_pages(x)
            st[name + "8"].view(torch.uint8)[at:at + n] = c.view(torch.uint8)
            st[name + "_scale"][at:at + n] = s


def _table(used, width, perm):
    """Rows of page ids, taken from a random order one sequence after the other; -1 past a sequence's pages."""
    before = (used.cumsum(0) - used)[:, None]
    p = torch.arange(width)[None]
    at = (before + p).cuda()
    live = (p < used[:, None]).cuda()
    return torch.where(live, perm[at.clamp(max=perm.numel() - 1)], torch.full_like(at, -1, dtype=torch.int32)).contiguous()


def _prepare_attend(case, seed, gen):
    order = _order(seed, case["batch"])
    n = _lens(1, case["batch"], case["low"], case["cap"])[order]
    total = n + _lens(2, case["batch"], case["past_low"], case["past_cap"])[order]
    tq, tk = int(n.sum()), int(total.sum())
    st = dict(cu_q=_starts(n), cu_k=_starts(total))
    # as a projection leaves them: q, k and v of a token next to one another where all are new
    st["k"] = _keys((tk, case["hkv"], D), gen)
    st["k"][st["cu_k"][:-1].long()] *= 2  # a sequence's first token draws attention (a sink)
    st["v"] = torch.randn((tk, case["hkv"], D), generator=gen, device="cuda").to(torch.bfloat16)
    st["q"] = torch.randn((tq, case["hq"], D), generator=gen, device="cuda").to(torch.bfloat16)
    st["out"] = torch.zeros_like(st["q"])
    return st


def _prepare_reserve(case, seed, gen):
    b = case["batch"]
    order = _order(seed, b)
    keep = _lens(1, b, 0, case["keep_cap"])[order]
    new = _lens(2, b, case["new_low"], case["new_cap"])[order]
    lens = keep.clone()
    done = (_lens(3, b, 0, 999) < 1000 * case["replaced"])[order]
    lens = torch.where(done, lens + 100, lens)  # those done keep nothing of what they hold
    keep = torch.where(done, torch.zeros_like(keep), keep)
    width = int(max(_pages(lens).max(), _pages(keep + new).max())) + 1
    held = int(_pages(lens).sum())
    need = int(_pages(keep + new).sum())
    num = max(held, need) + 64
    perm = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
    st = dict(table=_table(_pages(lens), width, perm), lens=lens.to(torch.int32).cuda(), keep=keep.to(torch.int32).cuda(),
              new=new.to(torch.int32).cuda())
    st["free"] = torch.cat([perm[held:], torch.full((held,), -1, dtype=torch.int32, device="cuda")])
    st["num_free"] = torch.full((1,), num - held, dtype=torch.int32, device="cuda")
    # the room a program has: a fixed number of packed tokens a step
    st["max_new"] = int(new.sum()) + 17
    st["max_all"] = int((keep + new).sum()) + 33 if case["all_slots"] else 0
    for name in ("k", "v"):
        st[name + "8"] = torch.zeros((num, 1, B, D), dtype=torch.float8_e4m3fn, device="cuda")
        st[name + "_scale"] = torch.ones((num, 1), device="cuda")
    return st


def _prepare_append(case, seed, gen):
    b, hkv = case["batch"], case["hkv"]
    order = _order(seed, b)
    new = _lens(1, b, case["low"], case["cap"])[order]
    before = _lens(2, b, 0, case["before"])[order]
    used = _pages(before + new)
    num = int(used.sum()) + 3
    perm = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
    st = dict(table=_table(used, int(used.max()), perm), lens=(before + new).to(torch.int32).cuda(), new=new.to(torch.int32).cuda())
    _pool(st, num, hkv, gen)
    st["max_new"], st["max_all"] = int(new.sum()), 0
    st.update(_plain_maps(st["table"], before.to(torch.int32).cuda(), st["new"], st["max_new"], 0))
    st["k_new"] = _keys((st["max_new"], hkv, D), gen)
    st["v_new"] = torch.randn((st["max_new"], hkv, D), generator=gen, device="cuda").to(torch.bfloat16)
    return st


def _prepare_gather(case, seed, gen):
    b, hkv = case["batch"], case["hkv"]
    lens = _lens(1, b, case["low"], case["cap"])[_order(seed, b)]
    used = _pages(lens)
    num = int(used.sum()) + 3
    perm = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
    st = dict(table=_table(used, int(used.max()), perm), lens=lens.to(torch.int32).cuda())
    _pool(st, num, hkv, gen)
    total = int(lens.sum())
    st["slots"] = _plain_maps(st["table"], torch.zeros_like(st["lens"]), st["lens"], total, 0)["slots"]
    st["k_out"] = torch.zeros((total, hkv, D), dtype=torch.bfloat16, device="cuda")
    st["v_out"] = torch.zeros_like(st["k_out"])
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = {"attend": _prepare_attend, "reserve": _prepare_reserve, "append": _prepare_append, "gather": _prepare_gather}[op](case, seed, gen)
    st["case"] = case
    if own:
        import dynamic_sparse_prefill_crisp_gb300 as crisp

        if op == "attend":
            longest = case["cap"] + case["past_cap"]  # a scheduler knows how long its requests can be
            st["packed"] = crisp.make_packed(case["hq"], case["hkv"], st["cu_q"], st["cu_k"], st["q"].shape[0], st["k"].shape[0],
                                             max_k=longest)
            size = crisp.packed_workspace_size(st["packed"])
        else:
            st["cache"] = crisp.make_kv_cache(st["k8"], st["v8"], st["k_scale"], st["v_scale"], st["table"], st["lens"])
            if op != "gather":
                st["step"] = crisp.make_kv_step(st["cache"], st["max_new"], st["max_all"])
            if op == "append":
                for name in ("cu_new", "cu_all", "slots", "positions", "runs"):
                    getattr(st["step"], name).copy_(st[name])
            size = crisp.kv_append_workspace_size(st["cache"])
        st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        crisp.workspace_init(st["ws"])
    elif op == "reserve":
        b, runs = case["batch"], _max_runs(case["batch"], st["max_new"])
        zeros = dict(dtype=torch.int32, device="cuda")
        st.update(cu_new=torch.zeros(b + 1, **zeros), cu_all=torch.zeros(b + 1, **zeros), slots=torch.zeros(st["max_new"], **zeros),
                  positions=torch.zeros(st["max_new"], **zeros), runs=torch.zeros(runs + 1, **zeros),
                  all_slots=torch.zeros(st["max_all"], **zeros))
    return st


# ----------------------------------------------------------------------- run
def run(st):
    op = st["case"]["op"]
    if own:
        import dynamic_sparse_prefill_crisp_gb300 as crisp

        if op == "attend":
            crisp.packed_prefill(st["packed"], st["q"], st["k"], st["v"], st["out"], st["ws"])
        elif op == "reserve":
            crisp.kv_reserve(st["cache"], st["free"], st["num_free"], st["step"], st["ws"], keep=st["keep"], new_lens=st["new"])
            return {"table": st["table"], "lens": st["lens"], "free": st["free"], "num_free": st["num_free"],
                    **{name: getattr(st["step"], name) for name in STEP}}
        elif op == "append":
            crisp.kv_append_packed(st["cache"], st["step"], st["k_new"], st["v_new"], st["ws"])
        else:
            crisp.kv_gather(st["cache"], st["slots"], st["k_out"], st["v_out"], st["ws"])
    else:
        {"attend": _plain_attend, "reserve": _plain_reserve, "append": _plain_append, "gather": _plain_gather}[op](st)
    if op == "attend":
        return {"out": st["out"]}
    if op == "reserve":
        return {name: st[name] for name in ("table", "lens", "free", "num_free") + STEP}
    if op == "append":
        return {name: st[name] for name in ("k8", "v8", "k_scale", "v_scale")}
    return {"k": st["k_out"], "v": st["v_out"]}


STEP = ("cu_new", "cu_all", "slots", "positions", "runs", "all_slots")


def _plain_attend(st):
    case = st["case"]
    b, hq, hkv = case["batch"], case["hq"], case["hkv"]
    lq, lk = case["cap"], case["cap"] + case["past_cap"]  # the batch padded to its longest
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    nq, nk = cu_q.diff(), cu_k.diff()
    t, j = torch.arange(lq, device="cuda"), torch.arange(lk, device="cuda")
    at_q = (cu_q[:-1, None] + t).clamp(max=st["q"].shape[0] - 1)
    at_k = (cu_k[:-1, None] + j).clamp(max=st["k"].shape[0] - 1)
    q = st["q"][at_q].float().view(b, lq, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, D)
    k = st["k"][at_k].float().permute(0, 2, 3, 1)
    s = (q @ k).view(b, hkv, hq // hkv, lq, lk)
    s *= D ** -0.5
    seen = (j <= (nk - nq)[:, None, None] + t[:, None]) & (j < nk[:, None, None])
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    s -= torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    s.exp_()
    l = s.sum(-1, keepdim=True)
    v = st["v"][at_k].float().transpose(1, 2)
    o = (s.view(b, hkv, -1, lk) @ v).view(b, hkv, hq // hkv, lq, D) / torch.where(l > 0, l, torch.ones_like(l))
    o = o.permute(0, 3, 1, 2, 4).reshape(b, lq, hq, D)
    st["out"][at_q[t < nq[:, None]]] = o[t < nq[:, None]].to(torch.bfloat16)


def _max_runs(batch, max_new):
    """Pages that `max_new` new tokens of `batch` sequences can touch."""
    return min(max_new, max_new // B + 2 * batch)


def _plain_maps(table, keep, new, max_new, max_all):
    """Running sums, slots, positions and page runs of `new` tokens behind `keep` ones, as fresh tensors (zeros past the ends)."""
    table, keep, new = table.long(), keep.long(), new.long()
    lens = keep + new

    def starts(n):
        return torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), n.cumsum(0)])

    def slots(cu, first, room):
        i = torch.arange(room, device="cuda")
        seq = torch.searchsorted(cu[1:], i, right=True).clamp(max=cu.numel() - 2)
        pos = first[seq] + i - cu[seq]
        live = i < cu[-1]
        page = table[seq, (pos // B).clamp(0, table.shape[1] - 1)]
        zero = torch.zeros_like(i)
        return torch.where(live, page * B + pos % B, zero).to(torch.int32), torch.where(live, pos, zero).to(torch.int32)

    cu_new, cu_all = starts(new), starts(lens)
    got = dict(cu_new=cu_new.to(torch.int32), cu_all=cu_all.to(torch.int32))
    got["slots"], got["positions"] = slots(cu_new, keep, max_new)
    got["all_slots"] = slots(cu_all, torch.zeros_like(keep), max_all)[0]
    room = _max_runs(new.numel(), max_new)
    first, count = keep // B, torch.where(new > 0, (lens - 1) // B - keep // B + 1, torch.zeros_like(new))
    before = starts(count)
    r = torch.arange(room + 1, device="cuda")
    seq = torch.searchsorted(before[1:], r, right=True).clamp(max=new.numel() - 1)
    page = first[seq] + r - before[seq]
    at = torch.maximum(page * B, keep[seq]) - keep[seq] + cu_new[seq]
    got["runs"] = torch.where(r < before[-1], at, cu_new[-1]).to(torch.int32)
    return got


def _plain_reserve(st):
    table, lens, new = st["table"].long(), st["lens"].long(), st["new"].long()
    keep = torch.minimum(st["keep"].long(), lens)
    kept, had, want = _pages(keep)[:, None], _pages(lens)[:, None], _pages(keep + new)[:, None]
    p = torch.arange(table.shape[1], device="cuda")[None]
    freed, taken = had - kept, want - kept
    back, fresh = (p >= kept) & (p < had), (p >= kept) & (p < want)
    top = st["num_free"].long() + freed.sum()  # pages go back so that taking them in order finds them again
    free = st["free"].long()
    free[(top - 1 - (freed.cumsum(0) - freed + p - kept))[back]] = table[back]
    at = top - 1 - (taken.cumsum(0) - taken + p - kept)
    table = torch.where(back, torch.full_like(table, -1), table)
    table = torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table)
    st["table"].copy_(table)
    st["free"].copy_(free)
    st["num_free"].copy_(top - taken.sum())
    st["lens"].copy_(keep + new)
    for name, x in _plain_maps(table, keep, new, st["max_new"], st["max_all"]).items():
        st[name].copy_(x)


def _plain_append(st):
    """Pages that the new tokens reach: their old tokens' values and the new ones, one scale, codes rounded again."""
    runs = st["runs"].long()
    runs = runs[:-1][runs[:-1] < runs[1:]]
    ends = torch.cat([runs[1:], torch.full_like(runs[:1], st["max_new"])])
    slot = st["slots"].long()[runs]
    ids, first = slot // B, (slot % B)[:, None]
    row = torch.arange(B, device="cuda")[None]
    is_old, is_new = row < first, (row >= first) & (row < first + (ends - runs)[:, None])
    at = (runs[:, None] + row - first).clamp(0, st["max_new"] - 1)
    for name in ("k", "v"):
        fresh = st[name + "_new"][at].transpose(1, 2).float()  # [n][hkv][128][128]
        codes, scale = st[name + "8"][ids], st[name + "_scale"][ids]
        value = torch.where(is_new[:, None, :, None], fresh, codes.float() * scale[..., None, None])
        need = _pow2(_exponent(torch.where(is_new[:, None, :, None], value.abs(), torch.zeros_like(value)).amax((-1, -2))))
        s = torch.where(first > 0, torch.maximum(need, scale), need)
        out = (value / s[..., None, None]).to(torch.float8_e4m3fn)
        keep = (is_new | is_old)[:, None, :, None]
        st[name + "8"].view(torch.uint8)[ids] = torch.where(keep, out.view(torch.uint8), codes.view(torch.uint8))
        st[name + "_scale"][ids] = s


def _plain_gather(st):
    slot = st["slots"].long()
    page, row = slot // B, slot % B
    for name in ("k", "v"):
        codes = st[name + "8"].view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn)
        st[name + "_out"].copy_((codes.float() * st[name + "_scale"][page][..., None]).to(torch.bfloat16))


# ---------------------------------------------------------------------- work
def _mean(low, cap, batch):
    """The sum of `batch` lengths between the bounds, the first one the longest."""
    return cap + (batch - 1) * (low + cap) / 2


def _mean_square(low, cap, batch):
    return cap * cap + (batch - 1) * (low * low + low * cap + cap * cap) / 3


def work(case):
    b = case["batch"]
    if case["op"] == "attend":
        n, past = _mean(case["low"], case["cap"], b), _mean(case["past_low"], case["past_cap"], b)
        pairs = (_mean_square(case["low"], case["cap"], b) + n) / 2 + n * past / b
        return {"bytes": 2 * D * 2 * (n * case["hq"] + (n + past) * case["hkv"]), "flops": 4 * D * case["hq"] * pairs}
    if case["op"] == "reserve":
        new, keep = _mean(case["new_low"], case["new_cap"], b), _mean(0, case["keep_cap"], b) * (1 - case["replaced"])
        return {"bytes": 28 * b + 8 * new + (4 * (new + keep) if case["all_slots"] else 0) + 8 * new / B, "flops": new}
    n = _mean(case["low"], case["cap"], b) * case["hkv"]
    return {"bytes": n * 2 * (2 * D + D), "flops": n * 2 * D}


# --------------------------------------------------------------------- exact
def _pow2_64(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """Round-half-even of 64-bit values of magnitude <= 448 to 4 significant bits, not below 2^-9."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a))))
    e = torch.where(_pow2_64(e) > a, e - 1, e)
    e = torch.where(_pow2_64(e + 1) <= a, e + 1, e).clamp(min=-6.0)
    step = _pow2_64(e - 3)
    return torch.round(x / step) * step


def _scale_64(amax):
    """By trying exponents one after another from the lowest that can hold amax."""
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -140) / 448.0)) - 1
    for _ in range(3):
        e = torch.where(448.0 * _pow2_64(e) < amax, e + 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, float(MIN_EXP))).clamp(min=float(MIN_EXP))
    return _pow2_64(e)


def exact(case, seed):
    if case["op"] == "reserve":
        return None  # whole numbers
    st = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, st)
    if case["op"] == "append":
        return _exact_append(case, st)
    out = {}
    for name in ("k", "v"):
        rows = []
        for i, n in enumerate(st["lens"].tolist()):
            ids = st["table"][i, :-(-n // B)].long()
            x = st[name + "8"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * st[name + "_scale"][ids].double()[..., None, None]
            rows.append(x.transpose(1, 2).reshape(-1, case["hkv"], D)[:n])
        out[name] = torch.cat(rows)
    return out


def _exact_attend(case, st):
    hq, hkv = case["hq"], case["hkv"]
    group = hq // hkv
    cq, ck = st["cu_q"].tolist(), st["cu_k"].tolist()
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for i in range(case["batch"]):
        k, v = (st[x][ck[i]:ck[i + 1]].double().transpose(0, 1) for x in ("k", "v"))
        past = k.shape[1] - (cq[i + 1] - cq[i])
        for at in range(cq[i], cq[i + 1], 1024):  # rows a thousand at a time, with the keys that they see
            end = min(at + 1024, cq[i + 1])
            last = past + end - cq[i]
            q = st["q"][at:end].double().view(end - at, hkv, group, D).permute(1, 2, 0, 3)
            s = torch.matmul(q.reshape(hkv, -1, D), k[:, :last].transpose(1, 2)).view(hkv, group, end - at, last) / math.sqrt(D)
            hidden = torch.ones((end - at, last), dtype=torch.bool, device="cuda").triu(past + at - cq[i] + 1)
            p = torch.softmax(s.masked_fill_(hidden, float("-inf")), -1)
            o = torch.matmul(p.view(hkv, -1, last), v[:, :last]).view(hkv, group, end - at, D)
            out[at:end] = o.permute(2, 0, 1, 3).reshape(end - at, hq, D)
    return {"out": out}


def _exact_append(case, st):
    got = {name: st[name].double() for name in ("k8", "v8", "k_scale", "v_scale")}
    hkv, at = case["hkv"], 0
    for i in range(case["batch"]):
        end, new = int(st["lens"][i]), int(st["new"][i])
        start = end - new
        p0, p1 = start // B, -(-end // B)
        ids = st["table"][i, p0:p1].long()
        old = start - p0 * B
        for name in ("k", "v"):
            x = torch.zeros((hkv, (p1 - p0) * B, D), dtype=torch.float64, device="cuda")
            x[:, old:old + new] = st[name + "_new"][at:at + new].double().transpose(0, 1)
            scale = _scale_64(x.view(hkv, -1, B, D).abs().amax((-1, -2)))
            if old:
                had = st[name + "_scale"][ids[0]].double()
                x[:, :old] = st[name + "8"][ids[0], :, :old].double() * had[:, None, None]
                scale[:, 0] = torch.maximum(scale[:, 0], had)
            c = _round_e4m3(x.view(hkv, -1, B, D) / scale[..., None, None]).reshape(hkv, -1, D)
            pages = got[name + "8"][ids].transpose(0, 1).reshape(hkv, -1, D)
            pages[:, :old + new] = c[:, :old + new]
            got[name + "8"][ids] = pages.view(hkv, -1, B, D).transpose(0, 1)
            got[name + "_scale"][ids] = scale.T
        at += new
    return got
