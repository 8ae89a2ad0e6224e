"""The cache operators as measured: writing the 8-bit paged key/value cache,
attention of new tokens over it, and eviction from it by accumulated weight.

``own = False`` computes each operator in its plain form (elementary torch
operations in 32 bits); ``own = True`` makes the calls a user makes of the
package. ``exact`` restates each operator from its definition in 64 bits.
"""
import math

import torch

own = False

B = 128  # tokens of a page
D = 128  # features
MIN_EXP = -100  # the smallest exponent of a page's scale


# --------------------------------------------------------------------- cases
def _decode(name, batch, hq, hkv, q_len, cap, low, weights):
    return dict(name=name, op="decode", batch=batch, hq=hq, hkv=hkv, q_len=q_len, cap=cap, low=low, weights=weights)


def _append(name, batch, hkv, new, before, ragged):
    return dict(name=name, op="append", batch=batch, hkv=hkv, new=new, before=before, ragged=ragged)


def _evict(name, batch, hkv, cap, low, keep, sink, recent):
    return dict(name=name, op="evict", batch=batch, hkv=hkv, cap=cap, low=low, keep=keep, sink=sink, recent=recent)


def listed():
    return [
        # one user, one token, a short prompt: latency
        _decode("decode-4x1-2k", 1, 4, 1, 1, 2048, 2048, False),
        # one user, one token, a 32k prompt of a 32/8-head layer
        _decode("decode-32x8-32k", 1, 32, 8, 1, 32768, 32768, False),
        # a server's batch: 32 sequences of any length up to 16k, 28/4 heads
        _decode("decode-28x4-ragged", 32, 28, 4, 1, 16384, 1, False),
        # four drafted tokens checked at once against a 128k cache
        _decode("verify-28x4-128k", 1, 28, 4, 4, 131072, 131071, False),
        # 64 sequences near 8k, with the weights that eviction needs
        _decode("decode-32x8-batch-weights", 64, 32, 8, 1, 8192, 6001, True),
        # one user at 512k tokens, with weights
        _decode("decode-32x8-512k-weights", 1, 32, 8, 1, 524288, 524288, True),
        # the one token a decode step adds to each of 64 sequences
        _append("append-1-batch64", 64, 8, 1, 4100, True),
        # a 32k prompt stored after prefill
        _append("store-32k", 1, 8, 32768, 0, False),
        # chunks of up to 32k tokens added to four sequences at odd offsets
        _append("store-ragged-chunks", 4, 4, 32768, 1007, True),
        # one short sequence cut to its budget: latency
        _evict("evict-4x1-2175", 1, 1, 2175, 2175, 1024, 128, 128),
        # a batch cut from about 8k to 4k tokens
        _evict("evict-batch16-8k", 16, 8, 8192, 3001, 4096, 128, 1024),
        # a 512k cache cut to a quarter
        _evict("evict-512k", 1, 8, 524288, 524288, 131072, 128, 1024),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    hq, hkv = rng.choice([(4, 1), (32, 8), (28, 4), (16, 1), (8, 8)])
    op = rng.choice(["decode", "decode", "append", "evict"])
    batch = log(1, 64)
    # at most the cells (sequences x kv heads x tokens) of the largest listed case of each kind
    most = max(B, (4_194_304 if op != "append" else 524_288) // (batch * hkv))
    cap = log(64, min(524_288, most))
    low = cap if rng.random() < 0.3 else max(1, int(cap * rng.uniform(0.05, 1.0)))
    if op == "decode":
        q_len = rng.choice([1, 1, 1, 2, 3, 4])
        return dict(op="decode", batch=batch, hq=hq, hkv=hkv, q_len=q_len, cap=cap, low=low, weights=rng.random() < 0.5)
    if op == "append":
        return dict(op="append", batch=batch, hkv=hkv, new=rng.choice([1, 1, cap]), before=rng.choice([0, log(1, 9000)]),
                    ragged=rng.random() < 0.5)
    keep = max(1, int(cap * rng.uniform(0.1, 0.9)))
    return dict(op="evict", batch=batch, hkv=hkv, cap=cap, low=low, keep=keep, sink=min(keep // 4, 128),
                recent=min(keep // 4, 1024))


# -------------------------------------------------------------------- inputs
def _lens(case, gen):
    """The lengths after the call (append) or at the call, on the CPU."""
    lo, hi = (case["low"], case["cap"]) if case["op"] != "append" else (1, case["new"])
    n = torch.randint(lo, hi + 1, (case["batch"],), generator=gen)
    n[0] = hi
    return n


def _cpu_gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _keys(shape, gen):
    """Keys with channels of different strength, as trained layers have; values plain."""
    chan = torch.exp(0.5 * torch.randn((shape[1], 1, D), generator=gen, device="cuda"))
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
    s = _pow2(_exponent(torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax((-1, -2))))
    return (x / s[..., None, None]).to(torch.float8_e4m3fn), s


def _filled(case, lens, cap, gen, spare):
    """A pool with `lens` tokens of each sequence in pages of a shuffled order."""
    b, hkv, pages = case["batch"], case["hkv"], -(-cap // B)
    num = b * pages + spare
    perm = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
    used = -(-lens // B)
    table = perm[:b * pages].view(b, pages)
    st = dict(k=torch.zeros((num, hkv, B, D), dtype=torch.float8_e4m3fn, device="cuda"),
              v=torch.zeros((num, hkv, B, D), dtype=torch.float8_e4m3fn, device="cuda"),
              k_scale=torch.ones((num, hkv), device="cuda"), v_scale=torch.ones((num, hkv), device="cuda"))
    pos = torch.arange(pages * B)
    for i in range(b):
        n = int(used[i])
        if n == 0:
            continue
        live = (pos[:n * B] < int(lens[i])).cuda()[None, :, None]
        for name in ("k", "v"):
            shape = (hkv, n * B, D)
            x = _keys((1,) + shape, gen)[0] if name == "k" else torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
            if name == "k":
                x[:, :4] *= 2  # the first tokens draw attention (sinks)
            x = (x * live).view(hkv, n, B, D).transpose(0, 1)
            c, s = _quantise_pages(x)
            at = table[i, :n].long()
            st[name].view(torch.uint8)[at] = c.view(torch.uint8)
            st[name + "_scale"][at] = s
    # entries past a sequence's pages name no page
    table = torch.where(torch.arange(pages, device="cuda")[None] < used[:, None].cuda(), table, torch.full_like(table, -1))
    st.update(table=table.contiguous(), lens=lens.to(torch.int32).cuda(), perm=perm)
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens = _lens(case, _cpu_gen(seed))
    b, hkv = case["batch"], case["hkv"]
    if case["op"] == "append":
        before = torch.randint(0, case["before"] + 1, (b,), generator=_cpu_gen(seed + 1)) if case["ragged"] else torch.full((b,), case["before"])
        new = lens if case["ragged"] else torch.full((b,), case["new"])
        # every page a sequence will reach is in its table, filled up to `before`
        st = _filled(case, before, case["before"] + case["new"], gen, 3)
        st["table"] = st["perm"][:st["table"].numel()].view_as(st["table"]).contiguous()
        st["lens"] = (before + new).to(torch.int32).cuda()
        st["new_lens"] = new.to(torch.int32).cuda()
        # token-major tensors, as a projection leaves them
        st["k_new"] = _keys((b, hkv, case["new"], D), gen).transpose(1, 2).contiguous().transpose(1, 2)
        st["v_new"] = torch.randn((b, case["new"], hkv, D), generator=gen, device="cuda").to(torch.bfloat16).transpose(1, 2)
    elif case["op"] == "decode":
        st = _filled(case, lens, case["cap"], gen, 3)
        st["q"] = torch.randn((b, case["q_len"], case["hq"], D), generator=gen, device="cuda").to(torch.bfloat16).transpose(1, 2)
        st["out"] = torch.zeros((b, case["q_len"], case["hq"], D), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
        if case["weights"]:
            st["weights"] = torch.rand((b, hkv, st["table"].shape[1] * B), generator=gen, device="cuda")
            st["weights_out"] = torch.zeros_like(st["weights"])
    else:
        new_pages = -(-min(case["keep"], case["cap"]) // B)
        st = _filled(case, lens, case["cap"], gen, b * new_pages + 3)
        cap = st["table"].shape[1] * B
        # accumulated weights: a few heavy tokens, a long light tail, some never attended
        w = torch.exp(2.0 * torch.randn((b, hkv, cap), generator=gen, device="cuda") - 4.0)
        w[..., 5::17] = 0.0
        st["weights"] = w
        at = b * st["table"].shape[1]
        st["new_table"] = st["perm"][at:at + b * new_pages].view(b, new_pages).contiguous()
        st["new_lens"] = torch.zeros(b, dtype=torch.int32, device="cuda")
        st["new_weights"] = torch.zeros((b, hkv, new_pages * B), device="cuda")
        st["kept"] = torch.full((b, hkv, new_pages * B), -1, dtype=torch.int32, device="cuda")
    st["case"] = case
    if own:
        import dynamic_sparse_prefill_crisp_gb300 as crisp

        cache = crisp.make_kv_cache(st["k"], st["v"], st["k_scale"], st["v_scale"], st["table"], st["lens"])
        st["cache"] = cache
        if case["op"] == "append":
            size = crisp.kv_append_workspace_size(cache)
        elif case["op"] == "decode":
            size = crisp.decode_workspace_size(cache, case["hq"], case["q_len"], weights=case["weights"])
        else:
            st["new_cache"] = crisp.make_kv_cache(st["k"], st["v"], st["k_scale"], st["v_scale"], st["new_table"], st["new_lens"])
            size = crisp.kv_evict_workspace_size(cache, case["keep"])
        st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        crisp.workspace_init(st["ws"])
    return st


# ----------------------------------------------------------------------- run
def run(st):
    case = st["case"]
    if own:
        import dynamic_sparse_prefill_crisp_gb300 as crisp

        if case["op"] == "append":
            crisp.kv_append(st["cache"], st["k_new"], st["v_new"], st["ws"], new_lens=st["new_lens"])
        elif case["op"] == "decode":
            crisp.decode_attention(st["cache"], st["q"], st["out"], st["ws"], weights_in=st.get("weights"),
                                   weights_out=st.get("weights_out"))
        else:
            crisp.kv_evict(st["cache"], st["new_cache"], st["weights"], st["ws"], keep=case["keep"], sink=case["sink"],
                           recent=case["recent"], new_weights=st["new_weights"], kept=st["kept"])
    else:
        {"append": _plain_append, "decode": _plain_decode, "evict": _plain_evict}[case["op"]](st)
    return _outputs(st)


def _outputs(st):
    op = st["case"]["op"]
    if op == "decode":
        return {"out": st["out"], **({"weights": st["weights_out"]} if "weights" in st else {})}
    got = {name: st[name] for name in ("k", "v", "k_scale", "v_scale")}
    if op == "evict":
        got.update(lens=st["new_lens"], weights=st["new_weights"], kept=st["kept"])
    return got


def _plain_append(st):
    """Pages that the new tokens reach: their old tokens' values and the new ones, one scale, codes rounded again."""
    table, lens, new = st["table"].long(), st["lens"].long(), st["new_lens"].long()
    b, t = st["k_new"].shape[0], st["k_new"].shape[2]
    reach = (t + B - 2) // B + 1  # pages that t tokens can touch
    start = lens - new
    page = start[:, None] // B + torch.arange(reach, device="cuda")[None]
    touched = page * B < lens[:, None]
    ids = table.gather(1, page.clamp(max=table.shape[1] - 1))[touched]  # [n]
    seq = torch.arange(b, device="cuda")[:, None].expand_as(page)[touched]
    pos = page[touched][:, None] * B + torch.arange(B, device="cuda")[None]  # [n][128]
    first, end = start[seq][:, None], lens[seq][:, None]
    is_new = (pos >= first) & (pos < end)
    is_old = pos < first
    at = (pos - first).clamp(0, t - 1)
    for name in ("k", "v"):
        fresh = st[name + "_new"].transpose(1, 2)[seq[:, None], at].transpose(1, 2)  # [n][hkv][128][128]
        codes, scale = st[name][ids], st[name + "_scale"][ids]
        value = torch.where(is_new[:, None, :, None], fresh.float(), codes.float() * scale[..., None, None])
        finite = torch.where(is_new[:, None, :, None] & torch.isfinite(value), value.abs(), torch.zeros_like(value))
        need = _pow2(_exponent(finite.amax((-1, -2))))
        had = is_old.any(-1)[:, None]
        s = torch.where(had, torch.maximum(need, scale), need)
        out = (value / s[..., None, None]).to(torch.float8_e4m3fn)
        keep = (is_new | is_old)[:, None, :, None]
        st[name].view(torch.uint8)[ids] = torch.where(keep, out.view(torch.uint8), codes.view(torch.uint8))
        st[name + "_scale"][ids] = s


def _plain_decode(st):
    q = st["q"].float()
    b, hq, t, _ = q.shape
    ids = st["table"].long().clamp(min=0)
    hkv, cap = st["k"].shape[1], ids.shape[1] * B

    def values(name):
        x = st[name][ids].float() * st[name + "_scale"][ids][..., None, None]
        return x.transpose(1, 2).reshape(b, hkv, cap, D)

    pos = torch.arange(cap, device="cuda")
    vis = st["lens"].long()[:, None] - (t - 1) + torch.arange(t, device="cuda")[None]
    mask = (pos[None, None] < vis[..., None])[:, None, None]  # [b][1][1][t][cap]
    s = torch.einsum("bghtd,bgjd->bghtj", q.view(b, hkv, hq // hkv, t, D), values("k")) * (D ** -0.5)
    s = torch.where(mask, s, torch.full_like(s, float("-inf")))
    m = s.amax(-1, keepdim=True)
    p = torch.where(mask, torch.exp(s - torch.where(torch.isfinite(m), m, torch.zeros_like(m))), torch.zeros_like(s))
    l = p.sum(-1, keepdim=True)
    p = torch.where(l > 0, p / l, torch.zeros_like(p))
    out = torch.einsum("bghtj,bgjd->bghtd", p, values("v"))
    st["out"].copy_(out.reshape(b, hq, t, D).to(torch.bfloat16))
    if "weights" in st:
        live = (pos[None] < st["lens"].long()[:, None])[:, None]
        st["weights_out"].copy_(torch.where(live, st["weights"] + p.sum((2, 3)), st["weights_out"]))


def _plain_evict(st):
    case = st["case"]
    w, ids, lens = st["weights"], st["table"].long().clamp(min=0), st["lens"].long()
    b, hkv, cap = w.shape
    keep, sink, recent = case["keep"], case["sink"], case["recent"]
    pos = torch.arange(cap, device="cuda")
    n = lens[:, None, None]
    key = torch.where((pos < sink) | (pos >= n - recent), torch.full_like(w, float("inf")), w)
    key = torch.where(pos < n, key, torch.full_like(w, float("-inf")))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    width = st["kept"].shape[-1]
    m = lens.clamp(max=keep)
    rank = torch.arange(width, device="cuda")
    live = (rank[None] < m[:, None])[:, None].expand(b, hkv, width)
    take = order[..., :width] if order.shape[-1] >= width else torch.nn.functional.pad(order, (0, width - order.shape[-1]))
    kept = torch.sort(torch.where(live, take, torch.full_like(take, cap)), dim=-1).values
    st["kept"].copy_(torch.where(live, kept.to(torch.int32), st["kept"]))
    st["new_weights"].copy_(torch.where(live, w.gather(-1, kept.clamp(max=cap - 1)), st["new_weights"]))
    st["new_lens"].copy_(m.to(torch.int32))
    src = kept.clamp(max=cap - 1)
    page = ids[:, None].expand(b, hkv, -1).gather(-1, src // B)  # [b][hkv][width]
    head = torch.arange(hkv, device="cuda")[None, :, None]
    used = torch.arange(width // B, device="cuda")[None] * B < m[:, None]
    to = st["new_table"].long()[used]
    tail = live.view(b, hkv, -1, B).transpose(1, 2)[used][..., None]
    for name in ("k", "v"):
        value = st[name][page, head, src % B].float() * st[name + "_scale"][page, head][..., None]
        value = value.view(b, hkv, -1, B, D).transpose(1, 2)[used]
        c, s = _quantise_pages(torch.where(tail, value, torch.zeros_like(value)))
        st[name].view(torch.uint8)[to] = torch.where(tail, c.view(torch.uint8), st[name].view(torch.uint8)[to])
        st[name + "_scale"][to] = s


# ---------------------------------------------------------------------- work
def _case_tokens(case):
    """Tokens held (or added) by a batch whose lengths are uniform between the bounds."""
    lo, hi = (case["low"], case["cap"]) if case["op"] != "append" else ((1, case["new"]) if case["ragged"] else (case["new"], case["new"]))
    return hi + (case["batch"] - 1) * (lo + hi) / 2


def work(case):
    n, hkv = _case_tokens(case), case["hkv"]
    if case["op"] == "append":
        return {"bytes": n * hkv * 2 * (2 * D + D), "flops": n * hkv * 2 * D * 2}
    if case["op"] == "decode":
        rows = case["hq"] * case["q_len"]
        return {"bytes": n * hkv * (2 * D + (8 if case["weights"] else 0)) + case["batch"] * rows * D * 4, "flops": 4 * D * rows * n}
    kept = min(case["keep"], n / case["batch"]) * case["batch"]
    return {"bytes": n * hkv * 4 + kept * hkv * (4 * D + 8), "flops": n * hkv}


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
    st = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(case, st)
    if case["op"] == "append":
        return _exact_append(case, st)
    return _exact_evict(case, st)


def _exact_decode(case, st):
    b, t, hq, hkv = case["batch"], case["q_len"], case["hq"], case["hkv"]
    group = hq // hkv
    out = torch.zeros((b, t, hq, D), dtype=torch.float64, device="cuda").transpose(1, 2)
    w = st["weights_out"].double() if case["weights"] else None
    for i in range(b):
        n = int(st["lens"][i])
        ids = st["table"][i, :-(-n // B)].long()
        for g in range(hkv):
            def side(name):
                return (st[name][ids, g].double() * st[name + "_scale"][ids, g].double()[:, None, None]).reshape(-1, D)[:n]
            k, v = side("k"), side("v")
            total = torch.zeros(n, dtype=torch.float64, device="cuda")
            for x in range(t):
                end = n - (t - 1 - x)
                if end <= 0:
                    continue
                s = st["q"][i, g * group:(g + 1) * group, x].double() @ k[:end].T / math.sqrt(D)
                p = torch.softmax(s, -1)
                out[i, g * group:(g + 1) * group, x] = p @ v[:end]
                total[:end] += p.sum(0)
            if w is not None:
                w[i, g, :n] = st["weights"][i, g, :n].double() + total
    return {"out": out, **({"weights": w} if w is not None else {})}


def _exact_append(case, st):
    got = {name: st[name].double() for name in ("k", "v", "k_scale", "v_scale")}
    for i in range(case["batch"]):
        end, new = int(st["lens"][i]), int(st["new_lens"][i])
        start = end - new
        p0, p1 = start // B, -(-end // B)
        ids = st["table"][i, p0:p1].long()
        old = start - p0 * B
        for name in ("k", "v"):
            hkv = case["hkv"]
            x = torch.zeros((hkv, (p1 - p0) * B, D), dtype=torch.float64, device="cuda")
            x[:, old:old + new] = st[name + "_new"][i, :, :new].double()
            scale = _scale_64(x.view(hkv, -1, B, D).abs().amax((-1, -2)))
            if old:
                had = st[name + "_scale"][ids[0]].double()
                x[:, :old] = st[name][ids[0], :, :old].double() * had[:, None, None]
                scale[:, 0] = torch.maximum(scale[:, 0], had)
            c = _round_e4m3(x.view(hkv, -1, B, D) / scale[..., None, None]).reshape(hkv, -1, D)
            pages = got[name][ids].transpose(0, 1).reshape(hkv, -1, D)
            pages[:, :old + new] = c[:, :old + new]
            got[name][ids] = pages.view(hkv, -1, B, D).transpose(0, 1)
            got[name + "_scale"][ids] = scale.T
    return got


def _exact_evict(case, st):
    got = {name: st[name].double() for name in ("k", "v", "k_scale", "v_scale")}
    got.update(lens=None, kept=None, weights=st["new_weights"].double())
    keep, sink, recent, hkv = case["keep"], case["sink"], case["recent"], case["hkv"]
    for i in range(case["batch"]):
        n = int(st["lens"][i])
        m = min(n, keep)
        ids = st["table"][i].long()
        for g in range(hkv):
            if n <= keep:
                pos = torch.arange(n, device="cuda")
            else:
                mid = st["weights"][i, g, sink:n - recent].double()
                rank = torch.argsort(-mid, stable=True)[:keep - sink - recent] + sink
                pos = torch.cat([torch.arange(sink, device="cuda"), rank.sort().values, torch.arange(n - recent, n, device="cuda")])
            got["weights"][i, g, :m] = st["weights"][i, g, pos].double()
            pages = -(-m // B)
            to = st["new_table"][i, :pages].long()
            for name in ("k", "v"):
                x = torch.zeros((pages * B, D), dtype=torch.float64, device="cuda")
                x[:m] = st[name][ids[pos // B], g, pos % B].double() * st[name + "_scale"][ids[pos // B], g].double()[:, None]
                x = x.view(pages, B, D)
                s = _scale_64(x.abs().amax((-1, -2)))
                c = _round_e4m3(x / s[:, None, None]).view(-1, D)
                flat = got[name][to, g].reshape(-1, D)
                flat[:m] = c[:m]
                got[name][to, g] = flat.view(pages, B, D)
                got[name + "_scale"][to, g] = s
    return got
