"""Target-side cache operators: what is measured, and their plain forms.

The target model of a speculative round keeps a paged key/value cache.  Three operators work on it:

  append   norms of the new rows' queries and keys per head, rotation by position, keys and values written
           to the rows' places in the pages
  attend   the new rows (one token, a drafted block, a prompt) attend over the pages: grouped heads,
           causal, optionally a sliding window with a few first tokens that stay visible, optionally
           by stored positions and with the attention weight that every cached row got added up
  evict    every (sequence, key/value head) is cut down to a budget of rows: the first tokens and the
           most recent ones stay, then the rows with the most weight; kept rows from past the budget move
           into the holes below it

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}


def _append(name, B, rows, Hq, Hkv, dh, page, dtype, rot, interleaved=False, norm=True, past=512, ragged=False):
    return {"name": name, "op": "append", "B": B, "rows": rows, "Hq": Hq, "Hkv": Hkv, "dh": dh, "page": page,
            "dtype": dtype, "rot": rot, "interleaved": interleaved, "norm": norm, "past": past, "ragged": ragged}


def _attend(name, B, rows, L, Hq, Hkv, dh, page, dtype, window=0, sinks=0, ragged=False, weights=False):
    return {"name": name, "op": "attend", "B": B, "rows": rows, "L": L, "Hq": Hq, "Hkv": Hkv, "dh": dh, "page": page,
            "dtype": dtype, "window": window, "sinks": sinks, "ragged": ragged, "weights": weights}


def _evict(name, B, L, budget, Hkv, dh, page, dtype, sinks, recent, ragged=False):
    return {"name": name, "op": "evict", "B": B, "L": L, "budget": budget, "Hkv": Hkv, "dh": dh, "page": page,
            "dtype": dtype, "sinks": sinks, "recent": recent, "ragged": ragged}


def listed():
    return [
        # plain decoding of one conversation: one new row, latency is all
        _append("append_one_row", 1, 1, 32, 8, 128, 64, "bf16", 128),
        # scoring the drafted blocks of a full batch: the last token and 16 drafted ones per sequence
        _append("append_blocks", 64, 17, 32, 8, 128, 16, "bf16", 128, past=1024),
        # a few prompts at once, of odd lengths, a quarter-rotated head, pairs side by side
        _append("append_prompts", 5, 4099, 32, 8, 128, 64, "bf16", 32, interleaved=True, past=0, ragged=True),
        # one conversation's next token over the context of the concurrency-1 workload
        _attend("one_token", 1, 1, 1041, 32, 8, 128, 64, "bf16"),
        # one conversation with a very long context: only a split over its length fills the GPU
        _attend("one_token_long", 1, 1, 131071, 32, 8, 128, 64, "bf16"),
        # a full batch decoding over contexts of mixed lengths, one slot idle; the cache collects weights for eviction
        _attend("batch_weights", 64, 1, 4096, 32, 8, 128, 16, "bf16", ragged=True, weights=True),
        # the fp32 configuration: small heads, a window and sinks, odd lengths
        _attend("window_f32", 7, 17, 1537, 12, 4, 32, 16, "f32", window=500, sinks=5, ragged=True),
        # scoring a drafted block per sequence (the verifier's K + 1 rows) over the batch's contexts
        _attend("score_blocks", 48, 17, 4096, 32, 8, 128, 64, "bf16", ragged=True),
        # a prompt under a sliding window whose first four tokens stay visible
        _attend("prompt_window", 1, 8192, 8192, 32, 8, 128, 64, "bf16", window=2048, sinks=4),
        # a whole causal prompt of odd length after an earlier turn
        _attend("prompt_causal", 2, 2777, 4001, 16, 4, 64, 32, "bf16", ragged=True),
        # after each scored block: a budgeted cache is cut back by the block's rows
        _evict("evict_step", 32, 1041, 1024, 8, 128, 16, "bf16", 4, 128),
        # after the prompts: the cache is cut from the prompt's length to the budget
        _evict("evict_prompts", 8, 16384, 2048, 8, 128, 64, "bf16", 4, 256, ragged=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dh = rng.choice([64, 128] if dtype == "bf16" else [32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
        rows = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(128, 12000 * 48 // (rows * (Hq + 2 * Hkv)))))
        rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= dh])
        c = _append("", B, rows, Hq, Hkv, dh, page, dtype, rot, rng.random() < 0.5, rng.random() < 0.7,
                    rng.choice([0, rng.randint(1, 700)]), rng.random() < 0.5)
    elif op == "evict":
        L = _log(rng, 64, 16384)
        budget = max(32, int(L * rng.choice([rng.uniform(0.05, 0.9), rng.uniform(0.9, 1.0)])))
        B = _log(rng, 1, max(1, min(64, 500000 // (L * Hkv))))
        sinks = rng.randint(0, 8)
        c = _evict("", B, L, budget, Hkv, dh, page, dtype, sinks, rng.randint(0, max(0, budget - sinks) // 2),
                   rng.random() < 0.5)
    else:
        G = rng.choice([1, 2, 4, 5, 8] if dtype == "bf16" else [1, 3, 4])
        Hq = Hkv * G
        kind = rng.choice(["token", "token", "block", "prompt"])
        rows = 1 if kind == "token" else rng.randint(2, 33) if kind == "block" else _log(rng, 100, 4096)
        if dtype == "f32":
            rows = min(rows, 600)
        L = _log(rng, rows, 65536 if kind == "token" and dtype == "bf16" else 8192 if dtype == "bf16" else 4096)
        cost = max(L * Hkv * 6, L * Hq * rows * (1 if dtype == "bf16" else 12) // 30)
        B = _log(rng, 1, max(1, min(96, 7000000 // cost)))
        window = rng.choice([0, rng.randint(1, L)])
        c = _attend("", B, rows, L, Hq, Hkv, dh, page, dtype, window, rng.randint(0, 9) if window else 0,
                    rng.random() < 0.6, kind == "token" and rng.random() < 0.4)
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes that follow from the case alone
def _lens(B, L, ragged, least):
    """Lengths of the sequences: all the same, or spread over the upper half, the second slot nearly empty."""
    if not ragged:
        return [L] * B
    lens = [L - (b * (L // 2)) // max(1, B) for b in range(B)]
    if B > 1:
        lens[1] = 0
    return [max(least, n) for n in lens]


def _rows(c):
    """(new rows, cached rows with the new ones) of every sequence."""
    if c["op"] == "append":
        new = _lens(c["B"], c["rows"], c["ragged"], 0)
        return new, [n + c["past"] for n in new]
    kv = _lens(c["B"], c["L"], c["ragged"], 0)
    return [min(c["rows"], n) for n in kv], kv


def _seen(n, L, window, sinks):
    """(query, row) pairs of a sequence of n new rows among L, and rows that any of them sees."""
    pairs = 0
    if not window:
        pairs = n * L - n * (n - 1) // 2
    else:
        for i in range(n):
            p = L - n + i
            lo = max(0, p - window + 1)
            pairs += p + 1 - lo + min(sinks, lo)
    lo = max(0, L - n - window + 1) if window else 0
    return pairs, (L - lo + min(sinks, lo)) if n else 0


def work(case):
    c, es = case, SIZES[case["dtype"]]
    if c["op"] == "append":
        T = sum(_rows(c)[0])
        return {"bytes": 2 * T * (c["Hq"] + 2 * c["Hkv"]) * c["dh"] * es + 4 * T,
                "flops": 8 * T * (c["Hq"] + c["Hkv"]) * c["dh"]}
    if c["op"] == "attend":
        new, kv = _rows(c)
        seen = [_seen(n, L, c["window"], c["sinks"]) for n, L in zip(new, kv)]
        rows = sum(r for _, r in seen)
        return {"bytes": rows * c["Hkv"] * (2 * c["dh"] * es + (12 if c["weights"] else 0))
                + 2 * sum(new) * c["Hq"] * c["dh"] * es + 4 * sum(new) * c["Hq"],
                "flops": 4 * c["dh"] * c["Hq"] * sum(p for p, _ in seen)}
    kv = _lens(c["B"], c["L"], c["ragged"], 1)
    cut = [L for L in kv if L > c["budget"]]
    # weights and positions of all rows; about (L - budget) budget / L rows move
    moved = sum((L - c["budget"]) * c["budget"] / L for L in cut) * c["Hkv"]
    return {"bytes": 8 * sum(cut) * c["Hkv"] + moved * 2 * (2 * c["dh"] * es + 8) + 8 * c["B"]}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dt)

    B, ps, Hkv, dh = c["B"], c["page"], c["Hkv"], c["dh"]
    if c["op"] == "evict":
        new, kv = None, _lens(B, c["L"], c["ragged"], 1)
    else:
        new, kv = _rows(c)
    pages = [(L + ps - 1) // ps for L in kv]
    n_pages = sum(pages) + 3
    most = max(1, max(pages))
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    host = [[-1] * most for _ in range(B)]
    at = 0
    for b, n in enumerate(pages):
        host[b][:n] = range(at, at + n)
        at += n
    index = torch.tensor(host, device=dev, dtype=torch.int64)
    table = torch.where(index < 0, -1, order[index.clamp(min=0)]).to(torch.int32)
    s = {"case": dict(c), "table": table, "kv": kv, "new": new, "kv_len": torch.tensor(kv, dtype=torch.int32, device=dev),
         "k": normal(n_pages, Hkv, ps, dh), "v": normal(n_pages, Hkv, ps, dh), "pos": None, "weight": None}
    if new is not None:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        T = cu[-1]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["seq"] = torch.tensor([b for b, n in enumerate(new) for _ in range(n)], dtype=torch.int64, device=dev)
        s["off"] = torch.tensor([i for n in new for i in range(n)], dtype=torch.int64, device=dev)
        s["row"] = torch.tensor([L - n + i for n, L in zip(new, kv) for i in range(n)], dtype=torch.int64, device=dev)
    if c["op"] == "append":
        Hq = c["Hq"]
        # one projection's output: queries, keys and values of a row side by side
        s["qkv"] = normal(T, (Hq + 2 * Hkv) * dh, std=2.0)
        # a conversation may begin far into the positions
        start = torch.randint(0, 100000, (B,), generator=g, device=dev)
        s["q_pos"] = (start[s["seq"]] + s["row"]).to(torch.int32)
        s["q_gain"] = s["k_gain"] = None
        if c["norm"]:
            s["q_gain"], s["k_gain"] = normal(dh, std=0.1) + 1, normal(dh, std=0.1) + 1
        i = torch.arange(c["rot"] // 2, device=dev, dtype=torch.float64)
        s["inv_freq"] = torch.exp(-math.log(1e6) * 2 * i / c["rot"])
    elif c["op"] == "attend":
        # heads differ in how peaked their attention is
        sharp = 0.5 + 2.5 * torch.rand(c["Hq"], 1, generator=g, device=dev)
        s["q"] = (torch.randn(T, c["Hq"], dh, generator=g, device=dev) * sharp).to(dt)
        s["scale"] = dh ** -0.5
        if c["weights"]:
            s["weight"] = torch.rand(n_pages, Hkv, ps, generator=g, device=dev)
    else:
        shape = (n_pages, Hkv, ps)
        w = torch.exp(2 * torch.randn(shape, generator=g, device=dev)) / c["L"]
        # rows that got no weight at all tie
        s["weight0"] = torch.where(torch.rand(shape, generator=g, device=dev) < 0.1, torch.zeros_like(w), w)
        s["pos0"] = torch.full(shape, -1, dtype=torch.int32, device=dev)
        # earlier evictions have left the positions out of order
        for b, L in enumerate(kv):
            r = torch.arange(pages[b] * ps, device=dev)
            for h in range(Hkv):
                p = torch.cat([torch.randperm(L, generator=g, device=dev), r[L:]]).to(torch.int32)
                s["pos0"][table[b, :pages[b]].long(), h] = p.reshape(pages[b], ps)
        s["weight"], s["pos"] = s["weight0"].clone(), s["pos0"].clone()
        s["next_pos"] = s["kv_len"].clone()
        keep = [min(L, c["budget"]) for L in kv]
        s["to_seq"] = torch.tensor([b for b, n in enumerate(keep) for _ in range(n)], dtype=torch.int64, device=dev)
        s["to_row"] = torch.cat([torch.arange(n, device=dev) for n in keep])
    if own:
        from step_flow_map_b200.host import PagedCache
        s["cache"] = PagedCache(s["k"], s["v"], table, pos=s["pos"], weight=s["weight"])
    return s


# ------------------------------------------------------------------ the passes
def run(state):
    return {"append": _run_append, "attend": _run_attend, "evict": _run_evict}[state["case"]["op"]](state)


def _split(s):
    c = s["case"]
    Hq, Hkv, dh = c["Hq"], c["Hkv"], c["dh"]
    return (s["qkv"][:, :Hq * dh].unflatten(1, (Hq, dh)), s["qkv"][:, Hq * dh:(Hq + Hkv) * dh].unflatten(1, (Hkv, dh)),
            s["qkv"][:, (Hq + Hkv) * dh:].unflatten(1, (Hkv, dh)))


def _run_append(s):
    c = s["case"]
    q, k, v = _split(s)
    if own:
        q = s["cache"].append(q, k, v, s["cu"], s["kv_len"], q_pos=s["q_pos"], q_gain=s["q_gain"], k_gain=s["k_gain"],
                              eps=1e-6, inv_freq=s["inv_freq"], interleaved=c["interleaved"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    angle = s["q_pos"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    half = c["rot"] // 2

    def turn(x, gain):
        x = x.float()
        if gain is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gain.float()
        if c["interleaved"]:
            a, b = x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:c["rot"]]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., c["rot"]:]], -1)

    page = s["table"][s["seq"], s["row"] // c["page"]].long()
    s["k"][page, :, s["row"] % c["page"]] = turn(k, s["k_gain"]).to(s["k"].dtype)
    s["v"][page, :, s["row"] % c["page"]] = v
    return {"q": turn(q, s["q_gain"]).to(q.dtype), "k": s["k"], "v": s["v"]}


def _run_attend(s):
    c = s["case"]
    most, longest = max(s["new"]), max(s["kv"])
    if own:
        out, lse = s["cache"].attend(s["q"], s["cu"], s["kv_len"], max_rows=most, max_kv=longest, scale=s["scale"],
                                     window=c["window"], sinks=c["sinks"], accumulate=c["weights"], lse=True)
        return {"out": out, "lse": lse, **({"weight": s["weight"]} if c["weights"] else {})}
    B, Hq, Hkv, dh = c["B"], c["Hq"], c["Hkv"], c["dh"]
    G, dev = Hq // Hkv, s["q"].device
    r = torch.arange(longest, device=dev)
    page = s["table"][:, r // c["page"]].clamp(min=0).long()
    k = s["k"][page, :, r % c["page"]].float().permute(0, 2, 1, 3)
    v = s["v"][page, :, r % c["page"]].float().permute(0, 2, 1, 3)
    q = torch.zeros(B, most, Hq, dh, device=dev)
    q[s["seq"], s["off"]] = s["q"].float()
    q = q.reshape(B, most, Hkv, G, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * most, dh)
    new = s["cu"][1:] - s["cu"][:-1]
    p = (s["kv_len"] - new)[:, None] + torch.arange(most, device=dev)
    see = (r <= p[:, :, None]) & (r < s["kv_len"][:, None, None])
    if c["window"]:
        see &= (p[:, :, None] - r < c["window"]) | (r < c["sinks"])
    see = see[:, None, None]
    score = (q @ k.transpose(2, 3) * s["scale"]).unflatten(2, (G, most)).masked_fill_(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    score = score.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = score.sum(-1, keepdim=True)
    score = score.div_(total.masked_fill(total == 0, 1.0))
    out = (score.flatten(2, 3) @ v).unflatten(2, (G, most)).permute(0, 3, 1, 2, 4)[s["seq"], s["off"]]
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2)[s["seq"], s["off"]]
    got = {"out": out.reshape(-1, Hq, dh).to(s["q"].dtype), "lse": lse.reshape(-1, Hq)}
    if c["weights"]:
        # padded rows add nothing
        mine = (r < s["kv_len"][:, None]) & (new > 0)[:, None]
        add = (score * (torch.arange(most, device=dev) < new[:, None])[:, None, None, :, None]).sum((2, 3))
        add = add.permute(0, 2, 1) * mine[:, :, None]
        s["weight"].index_put_((page[:, :, None], torch.arange(Hkv, device=dev), (r % c["page"])[:, None]), add, accumulate=True)
        got["weight"] = s["weight"]
    return got


def _run_evict(s):
    c = s["case"]
    # this pass's weights and positions; keys and values past the budget stay where they are
    s["weight"].copy_(s["weight0"])
    s["pos"].copy_(s["pos0"])
    if own:
        left = s["cache"].evict(s["kv_len"], s["next_pos"], c["budget"], sinks=c["sinks"], recent=c["recent"], max_kv=max(s["kv"]))
        return {"k": s["k"], "v": s["v"], "pos": s["pos"], "weight": s["weight"], "len": left}
    dev, ps, longest = s["k"].device, c["page"], max(s["kv"])
    r = torch.arange(longest, device=dev)
    page = s["table"][:, r // ps].clamp(min=0).long()
    weight = s["weight"][page, :, r % ps].permute(0, 2, 1)
    pos = s["pos"][page, :, r % ps].permute(0, 2, 1)
    live = (r < s["kv_len"][:, None])[:, None]
    kept_by_rule = (pos < c["sinks"]) | (pos >= (s["next_pos"] - c["recent"])[:, None, None])
    key = torch.where(kept_by_rule, math.inf, weight).masked_fill(~live, -1.0)
    rank = torch.sort(key, dim=-1, descending=True, stable=True).indices.argsort(-1)
    limit = s["kv_len"].clamp(max=c["budget"])[:, None, None]
    keep = (rank < limit) & live
    hole, mover = (r < limit) & ~keep, (r >= limit) & keep
    # the n-th hole takes the n-th kept row from past the budget
    first = torch.sort(mover.to(torch.int8), dim=-1, descending=True, stable=True).indices
    come = first.gather(-1, (hole.long().cumsum(-1) - 1).clamp(min=0))
    come = torch.where(hole, come, r)[s["to_seq"], :, s["to_row"]]
    b, h = s["to_seq"][:, None], torch.arange(c["Hkv"], device=dev)
    from_page, from_off = page[b, come], come % ps
    to_page, to_off = page[b, s["to_row"][:, None]], (s["to_row"] % ps)[:, None]
    for name in ("k", "v", "pos", "weight"):
        s[name][to_page, h, to_off] = s[name][from_page, h, from_off]
    return {"k": s["k"], "v": s["v"], "pos": s["pos"], "weight": s["weight"], "len": s["kv_len"].clamp(max=c["budget"])}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "evict": _exact_evict}[case["op"]](s)


def _exact_append(s):
    c = s["case"]
    ps, rot = c["page"], c["rot"]
    cache = {n: s[n].double() for n in ("k", "v")}
    got = []
    # one complex turn per pair of a head's values
    unit = torch.polar(torch.ones((), dtype=torch.float64, device=s["k"].device), s["q_pos"].double()[:, None] * s["inv_freq"])
    parts = [x.double() for x in _split(s)]
    for x, gain in ((parts[0], s["q_gain"]), (parts[1], s["k_gain"])):
        if gain is not None:
            x = x / ((x * x).sum(-1, keepdim=True) / c["dh"] + 1e-6).sqrt() * gain.double()
        turned = x[..., :rot]
        pair = (-1, 2) if c["interleaved"] else (2, -1)
        z = turned.unflatten(-1, pair)
        z = z if c["interleaved"] else z.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * unit[:, None])
        z = z if c["interleaved"] else z.transpose(-1, -2)
        got.append(torch.cat([z.flatten(-2), x[..., rot:]], -1))
    got.append(parts[2])
    at = 0
    for b, n in enumerate(s["new"]):
        for i0 in range(0, n, ps):
            rows = torch.arange(i0, min(n, i0 + ps), device=s["k"].device)
            place = rows + s["kv"][b] - n
            page = s["table"][b, place // ps].long()
            for name, x in (("k", got[1]), ("v", got[2])):
                cache[name][page, :, place % ps] = x[at + rows]
        at += n
    return {"q": got[0], "k": cache["k"], "v": cache["v"]}


def _exact_attend(s):
    c = s["case"]
    Hq, Hkv, dh, ps = c["Hq"], c["Hkv"], c["dh"], c["page"]
    G, dev = Hq // Hkv, s["q"].device
    T = s["q"].shape[0]
    out = torch.zeros(T, Hq, dh, dtype=torch.float64, device=dev)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev)
    weight = s["weight"].double() if c["weights"] else None
    at = 0
    for b, (n, L) in enumerate(zip(s["new"], s["kv"])):
        if n:
            pages = s["table"][b, :(L + ps - 1) // ps].long()
            K = s["k"][pages].transpose(0, 1).reshape(Hkv, -1, dh)[:, :L].double()
            V = s["v"][pages].transpose(0, 1).reshape(Hkv, -1, dh)[:, :L].double()
            got = torch.zeros(Hkv, L, dtype=torch.float64, device=dev)
            for i0 in range(0, n, 512):
                i1 = min(n, i0 + 512)
                where = torch.arange(i0, i1, device=dev) + L - n
                far = where[:, None] - torch.arange(L, device=dev)
                blind = far < 0
                if c["window"]:
                    blind |= (far >= c["window"]) & (torch.arange(L, device=dev) >= c["sinks"])
                Q = s["q"][at + i0:at + i1].double().unflatten(1, (Hkv, G)).permute(1, 2, 0, 3)
                z = torch.matmul(Q, K[:, None].transpose(-1, -2)) * s["scale"]
                z[blind.expand_as(z)] = -math.inf
                logs = torch.logsumexp(z, -1)
                p = torch.exp(z - logs[..., None])
                out[at + i0:at + i1] = torch.matmul(p, V[:, None]).permute(2, 0, 1, 3).flatten(1, 2)
                lse[at + i0:at + i1] = logs.permute(2, 0, 1).flatten(1)
                got += p.sum((1, 2))
            if weight is not None:
                r = torch.arange(L, device=dev)
                weight[pages[r // ps], :, r % ps] += got.T
        at += n
    return {"out": out, "lse": lse, **({"weight": weight} if c["weights"] else {})}


def _exact_evict(s):
    c = s["case"]
    ps = c["page"]
    k, v, weight = (s[n].double() for n in ("k", "v", "weight0"))
    for b, L in enumerate(s["kv"]):
        if L <= c["budget"]:
            continue
        pages = s["table"][b].long()
        for h in range(c["Hkv"]):
            r = torch.arange(L, device=s["k"].device)
            p, w = s["pos0"][pages[r // ps], h, r % ps], weight[pages[r // ps], h, r % ps]
            safe = (p < c["sinks"]) | (p >= L - c["recent"])
            others = r[~safe]
            best = others[torch.sort(w[~safe], descending=True, stable=True).indices]
            kept = torch.cat([r[safe], best])[:c["budget"]].sort().values
            gone = torch.ones(L, dtype=torch.bool, device=r.device)
            gone[kept] = False
            to, come = r[:c["budget"]][gone[:c["budget"]]], kept[kept >= c["budget"]]
            for x in (k, v, weight):
                x[pages[to // ps], h, to % ps] = x[pages[come // ps], h, come % ps]
    return {"k": k, "v": v, "pos": None, "weight": weight, "len": None}
