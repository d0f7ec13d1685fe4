"""Measured cases of the attention operators around the sparse layer: causal attention with a
sliding window and always-visible first tokens (its forward for prompts, its forward and
backward for training), and the serving side over a paged cache held in 8 bits - appending
tokens, windowed attention over it, and sparse edge attention over it.

Each operator has a plain form here (elementary torch operations in fp32), the call a user
makes of the library, and the same result in fp64 from the definition.

Definitions. Query i of a sequence sees key j <= i iff i - j < window or j < sinks; only the
first lens[b] tokens of a sequence exist, other rows give o = 0, lse = -inf and zero gradients.
The cache holds e4m3 values with one power-of-two scale per (page, KV head): 2^e with the
smallest e >= -100 such that the block's largest magnitude is at most 448 * 2^e. A block's scale
never shrinks while it fills; when it grows the block's older values are rounded again.
"""
import math

import torch

own = False

E_MIN = -100  # smallest exponent of a block's scale
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    """The layer shape of most cases (16 query heads, 8 KV heads, head size 128, bf16) and the
    2/1-head, size-64 fp32 shape are the library's own workload configurations."""
    big = {"hq": 16, "hkv": 8, "d": 128, "dtype": "bf16"}
    return [
        # one short user prompt: latency
        {"name": "prefill short", "op": "prefill", "B": 1, "n": 77, "window": 64, "sinks": 4, "ragged": False, **big},
        # a batch of packed prompts through a windowed layer
        {"name": "prefill window", "op": "prefill", "B": 8, "n": 4096, "window": 512, "sinks": 4, "ragged": False, **big},
        # a long prompt through a layer that sees everything (its lse feeds the refresh edges)
        {"name": "prefill full", "op": "prefill", "B": 1, "n": 16384, "window": 16384, "sinks": 0, "ragged": False, **big},
        # the training step of a windowed layer at the training sequence length
        {"name": "train window", "op": "train", "B": 8, "n": 4096, "window": 1024, "sinks": 4, "ragged": False, **big},
        # padded sequences of uneven length, other head shape
        {"name": "train ragged d64", "op": "train", "B": 3, "n": 1531, "window": 200, "sinks": 1, "ragged": True,
         "hq": 8, "hkv": 2, "d": 64, "dtype": "bf16"},
        # the fp32 validation configuration
        {"name": "train fp32", "op": "train", "B": 1, "n": 128, "window": 48, "sinks": 2, "ragged": False,
         "hq": 2, "hkv": 1, "d": 64, "dtype": "fp32"},
        # one decoded token of each of 64 users goes into the cache
        {"name": "append token", "op": "append", "B": 64, "t": 1, "have": 1000, "page": 64, "ragged": True, **big},
        # the prompts of a batch go into the cache
        {"name": "append prompt", "op": "append", "B": 8, "t": 4096, "have": 0, "page": 64, "ragged": False, **big},
        # one user's next token over a long, fully visible context
        {"name": "decode long", "op": "decode", "B": 1, "t": 1, "have": 65536, "page": 64, "window": 1 << 30,
         "sinks": 0, "ragged": False, **big},
        # next tokens of 64 users of uneven length through a windowed layer
        {"name": "decode batch", "op": "decode", "B": 64, "t": 1, "have": 8192, "page": 32, "window": 4096, "sinks": 4,
         "ragged": True, **big},
        # a sparse layer's next tokens
        {"name": "sea token", "op": "sea", "B": 64, "t": 1, "have": 4096, "page": 64, "s": 4, "ragged": True, **big},
        # a sparse layer's whole prompts over the cache
        {"name": "sea prompt", "op": "sea", "B": 8, "t": 4096, "have": 4096, "page": 64, "s": 4, "ragged": False, **big},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["prefill", "train", "append", "decode", "sea"])
    hq, hkv = rng.choice([(16, 8), (16, 8), (8, 8), (8, 2), (2, 1), (6, 2), (8, 1)])
    if op == "sea" and hq == 6:
        hq, hkv = 4, 2  # the sparse attention takes groups of 1, 2, 4 and 8
    case = {"op": op, "hq": hq, "hkv": hkv, "d": rng.choice([64, 128]),
            "dtype": rng.choice(["bf16", "bf16", "bf16", "fp32"]), "ragged": rng.random() < 0.5}
    if op in ("prefill", "train"):
        most = {"prefill": 16384, "train": 4096}[op] if case["dtype"] == "bf16" else 2048
        case["B"] = _between(rng, 1, 8)
        case["n"] = min(_between(rng, 1, most), int(math.sqrt(2.0e9 / (case["B"] * hq))))
        case["window"] = rng.choice([_between(rng, 1, case["n"]), _between(rng, 1, case["n"]), case["n"]])
        case["sinks"] = rng.choice([0, 1, 4, 16, 100])
        return case
    case["page"] = rng.choice([16, 32, 64, 128])
    if op == "append":
        case["B"] = _between(rng, 1, 64)
        case["t"] = min(_between(rng, 1, 4096), 32768 // case["B"])
        case["have"] = rng.choice([0, _between(rng, 1, 2000)])
    elif op == "decode":
        case["t"] = rng.choice([1, 1, 1, 2, 5, 8])
        case["B"] = _between(rng, 1, 64)
        case["have"] = max(case["t"], min(_between(rng, 8, 65536), 400000 // (case["B"] * case["t"])))
        case["window"] = rng.choice([1 << 30, _between(rng, 1, case["have"])])
        case["sinks"] = rng.choice([0, 1, 4, 100])
    else:
        case["B"] = _between(rng, 1, 64)
        case["have"] = min(_between(rng, 1, 16384), 100000 // case["B"])
        case["t"] = rng.choice([1, min(case["have"], 32768 // case["B"])])
        case["s"] = rng.choice([2, 4, 4, 7, 16])
        if case["s"] > 4:
            case["t"] = min(case["t"], 8192 // case["B"])
    return case


# ---- lengths ----------------------------------------------------------------------------------


def _uneven(most, B):
    """Lengths of a ragged batch: the longest is `most`, the others shorter by uneven steps."""
    return [most - (most * ((5 * b) % (B + 1))) // (B + 1) for b in range(B)]


def _lens(case):
    """What each sequence holds: tokens of a padded batch, or tokens in the cache with the new ones."""
    B = case["B"]
    if case["op"] in ("prefill", "train"):
        return _uneven(case["n"], B) if case["ragged"] else [case["n"]] * B
    have = _uneven(case["have"], B) if case["ragged"] else [case["have"]] * B
    if case["op"] == "append":
        return [h + n for h, n in zip(have, _new(case))]
    return [max(h, n) for h, n in zip(have, _new(case))]


def _new(case):
    """How many of a sequence's t rows are its own (the rest is padding)."""
    if case["t"] == 1 or not case["ragged"]:
        return [case["t"]] * case["B"]
    return _uneven(case["t"], case["B"])


# ---- inputs ---------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, hq, hkv, d, dt = case["B"], case["hq"], case["hkv"], case["d"], TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def whole(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    st = {"case": case, "scale": d ** -0.5}
    if case["op"] in ("prefill", "train"):
        n = case["n"]
        st["q"], st["k"], st["v"] = normal(B, n, hq, d).to(dt), normal(B, n, hkv, d).to(dt), normal(B, n, hkv, d).to(dt)
        st["lens"] = whole(_lens(case)) if case["ragged"] else None
        if case["op"] == "train":
            st["dout"] = normal(B, n, hq, d).to(dt)
        return st
    t, page = case["t"], case["page"]
    lens, new = _lens(case), _new(case)
    maxp = -(-max(lens) // page)
    pages = B * maxp + 1
    st["table"] = torch.randperm(pages, generator=g, device="cuda")[: B * maxp].reshape(B, maxp).to(torch.int32)
    # blocks of uneven magnitude, as keys and values of different tokens and heads have
    for name in ("k", "v"):
        size = torch.exp2(torch.randint(-2, 3, (pages, hkv), generator=g, device="cuda").float())
        x = normal(pages, hkv, page, d) * size[:, :, None, None]
        x = torch.where(x.isfinite(), x, 0.0)
        e = _exponent(x.abs().amax((2, 3)))
        st[name + "q"] = (x * torch.exp2(-e)[:, :, None, None]).to(F8)
        st[name + "s"] = torch.exp2(e)
    if case["op"] == "append":
        st["lens"] = whole([a - b for a, b in zip(lens, new)])  # before the call
        st["k"], st["v"] = (normal(B, t, hkv, 1).exp() * normal(B, t, hkv, d)).to(dt), normal(B, t, hkv, d).to(dt)
    else:
        st["lens"] = whole(lens)
        st["q"] = normal(B, t, hq, d).to(dt)
    st["new"] = whole(new) if case["t"] > 1 and case["ragged"] else None
    if case["op"] == "sea":
        # causal targets, weights that sum to one, some slots unused
        s = case["s"]
        pos = (st["lens"] - whole(new))[:, None] + torch.arange(t, device="cuda")[None, :]
        pos = torch.minimum(pos, st["lens"][:, None] - 1)
        u = torch.rand((B, t, hkv, s), generator=g, device="cuda", dtype=torch.float64)
        st["idx"] = (u * (pos.clamp(min=0) + 1)[:, :, None, None]).floor().to(torch.int32)
        w = -torch.rand((B, t, hkv, s), generator=g, device="cuda").clamp(min=1e-7).log() + 1e-6
        w = torch.where(torch.rand((B, t, hkv, s), generator=g, device="cuda") < 0.05, 0.0, w)
        st["w"] = w / w.sum(-1, keepdim=True).clamp(min=1e-6)
    return st


# ---- one pass -------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"prefill": _plain_prefill, "train": _plain_train, "append": _plain_append, "decode": _plain_decode,
            "sea": _plain_sea}[op](state)


def _own(st, op):
    import sparse_dynamic_routing_b200 as gm

    c = st["case"]
    if op in ("prefill", "train"):
        o, lse = gm.gm_window_attention_forward(st["q"], st["k"], st["v"], c["window"], c["sinks"], lens=st["lens"])
        if op == "prefill":
            return {"o": o, "lse": lse}
        dq, dk, dv = gm.gm_window_attention_backward(st["q"], st["k"], st["v"], o, st["dout"], lse, c["window"],
                                                     c["sinks"], lens=st["lens"])
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    cache = (st["kq"], st["vq"], st["ks"], st["vs"], st["table"], st["lens"])
    if op == "append":
        gm.gm_kv8_append(st["k"], st["v"], *cache, new_lens=st["new"])
        return {"kq": st["kq"], "vq": st["vq"], "ks": st["ks"], "vs": st["vs"]}
    if op == "decode":
        o, lse = gm.gm_kv8_attention_forward(st["q"], *cache, c["window"], c["sinks"], q_lens=st["new"])
    else:
        o, lse = gm.gm_kv8_sea_forward(st["q"], st["idx"], st["w"], *cache, q_lens=st["new"])
    return {"o": o, "lse": lse}


# ---- the plain forms ----------------------------------------------------------------------------


def _exponent(amax):
    """Smallest e >= E_MIN with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    return (x - 9 + (m > 0.875)).clamp(min=E_MIN).float()


def _plain_softmax(s, mask):
    """(probabilities, lse) over the last axis of the visible scores; a row with none gives 0 and -inf."""
    s = s.masked_fill_(~mask, float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + m).squeeze(-1)
    return p.div_(torch.where(total > 0, total, 1.0)), lse


def _plain_heads(st):
    """q [B, hkv, G, n, d], k and v [B, hkv, 1, n, d] in fp32, and the visibility [B, 1, 1, n, n]."""
    c = st["case"]
    B, n, hq, hkv, d = c["B"], c["n"], c["hq"], c["hkv"], c["d"]
    q = st["q"].float().reshape(B, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    k = st["k"].float().permute(0, 2, 1, 3)[:, :, None]
    v = st["v"].float().permute(0, 2, 1, 3)[:, :, None]
    i = torch.arange(n, device=q.device)
    see = (i[None, :] <= i[:, None]) & ((i[:, None] - i[None, :] < c["window"]) | (i[None, :] < c["sinks"]))
    see = see[None]
    if st["lens"] is not None:
        see = see & (i[None, :, None] < st["lens"][:, None, None])
    return q, k, v, see[:, None, None]


def _rows(x, dtype):
    """[B, hkv, G, n, d] -> [B, n, hkv * G, d]."""
    B, hkv, G, n, d = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(B, n, hkv * G, d).to(dtype)


def _plain_prefill(st):
    q, k, v, see = _plain_heads(st)
    p, lse = _plain_softmax((q @ k.transpose(-1, -2)).mul_(st["scale"]), see)
    return {"o": _rows(p @ v, st["q"].dtype), "lse": lse.permute(0, 3, 1, 2).flatten(2).contiguous()}


def _plain_train(st):
    q, k, v, see = _plain_heads(st)
    dt = st["q"].dtype
    p, lse = _plain_softmax((q @ k.transpose(-1, -2)).mul_(st["scale"]), see)
    o = p @ v
    do = st["dout"].float().reshape(*st["dout"].shape[:2], k.shape[1], -1, k.shape[-1]).permute(0, 2, 3, 1, 4)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    dp = do @ v.transpose(-1, -2)
    ds = dp.sub_((dp * p).sum(-1, keepdim=True)).mul_(p).mul_(st["scale"])
    dk = (ds.transpose(-1, -2) @ q).sum(2)
    return {"o": _rows(o, dt), "lse": lse.permute(0, 3, 1, 2).flatten(2).contiguous(), "dq": _rows(ds @ k, dt),
            "dk": dk.permute(0, 2, 1, 3).to(dt).contiguous(), "dv": dv.permute(0, 2, 1, 3).to(dt).contiguous()}


def _plain_append(st):
    c = st["case"]
    B, t, page, hkv, d = c["B"], c["t"], c["page"], c["hkv"], c["d"]
    x = torch.arange(t, device="cuda")
    mine = x[None, :] < (st["new"] if st["new"] is not None else torch.full((B,), t, device="cuda"))[:, None]
    pos = st["lens"][:, None].long() + x[None, :]
    table = st["table"].long()
    at = table.gather(1, (pos // page).clamp(max=table.shape[1] - 1))[mine]  # page of each new token
    slot = (pos % page)[mine]
    part = st["lens"].long() % page  # tokens that the first touched page already holds
    first = table.gather(1, (st["lens"].long() // page).clamp(max=table.shape[1] - 1)[:, None]).squeeze(1)
    for name in ("k", "v"):
        val = st[name].float()[mine]  # [tokens, hkv, d]
        amax = torch.zeros_like(st[name + "s"]).index_reduce_(0, at, val.abs().amax(-1), "amax")
        fresh = torch.exp2(_exponent(amax))
        old = st[name + "s"].clone()
        touched = torch.zeros(old.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, at, True)
        keeps = torch.zeros_like(touched).index_fill_(0, first[part > 0], True)
        new = torch.where(touched[:, None], torch.where(keeps[:, None], torch.maximum(fresh, old), fresh), old)
        st[name + "s"].copy_(new)
        pool = st[name + "q"].view(torch.uint8)
        grown = pool[first].view(F8).float() * (old / new)[first][:, :, None, None]
        stays = (part > 0)[:, None] & (torch.arange(page, device="cuda")[None, :] < part[:, None])
        rows, cols = stays.nonzero(as_tuple=True)
        pool[first[rows], :, cols] = grown.to(F8).view(torch.uint8)[rows, :, cols]
        pool[at, :, slot] = (val / new[at][:, :, None]).to(F8).view(torch.uint8)
    return {"kq": st["kq"], "vq": st["vq"], "ks": st["ks"], "vs": st["vs"]}


def _plain_positions(st):
    """Position [B, t] of each query row in its sequence, below 0 where the row is padding."""
    c = st["case"]
    x = torch.arange(c["t"], device="cuda")[None, :]
    new = st["new"][:, None] if st["new"] is not None else c["t"]
    return torch.where(x < new, st["lens"][:, None] - new + x, -1)


def _plain_decode(st):
    c = st["case"]
    B, t, hkv, d, page = c["B"], c["t"], c["hkv"], c["d"], c["page"]
    table = st["table"].long()
    keys, vals = ((st[x + "q"].view(torch.uint8)[table].view(F8).float() * st[x + "s"][table][..., None, None])
                  .permute(0, 2, 1, 3, 4).reshape(B, hkv, 1, -1, d) for x in ("k", "v"))
    q = st["q"].float().reshape(B, t, hkv, -1, d).permute(0, 2, 3, 1, 4)
    i = _plain_positions(st)[:, :, None]
    j = torch.arange(keys.shape[3], device="cuda")[None, None, :]
    see = ((j <= i) & ((i - j < c["window"]) | (j < c["sinks"])))[:, None, None]
    p, lse = _plain_softmax((q @ keys.transpose(-1, -2)).mul_(st["scale"]), see)
    return {"o": _rows(p @ vals, st["q"].dtype), "lse": lse.permute(0, 3, 1, 2).flatten(2).contiguous()}


def _plain_sea(st):
    c = st["case"]
    B, t, hkv, d, page = c["B"], c["t"], c["hkv"], c["d"], c["page"]
    idx = st["idx"].long()
    b = torch.arange(B, device="cuda")[:, None, None, None]
    h = torch.arange(hkv, device="cuda")[None, None, :, None]
    see = (st["w"] > 0) & (_plain_positions(st) >= 0)[:, :, None, None]
    at = st["table"].long()[b, idx // page]
    keys, vals = (st[x + "q"].view(torch.uint8)[at, h, idx % page].view(F8).float() * st[x + "s"][at, h][..., None]
                  for x in ("k", "v"))  # [B, t, hkv, s, d]
    q = st["q"].float().reshape(B, t, hkv, -1, d)
    s = (q @ keys.transpose(-1, -2)).mul_(st["scale"]) + st["w"].log()[:, :, :, None]
    p, lse = _plain_softmax(s, see[:, :, :, None])
    return {"o": (p @ vals).reshape(B, t, -1, d).to(st["q"].dtype), "lse": lse.reshape(B, t, -1)}


# ---- what a pass cannot do without ------------------------------------------------------------


def _seen(first, last, window, sinks):
    """Keys that the queries at positions first .. last - 1 see, summed: window, then sinks outside it."""
    def below(n, w):  # sum over i < n of min(i + 1, w)
        m = min(n, w)
        return m * (m + 1) // 2 + (n - m) * w

    both = min(window + sinks, 1 << 40)
    return below(last, both) - below(first, both)


def _bytes_per(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    B, hq, hkv, d, z = case["B"], case["hq"], case["hkv"], case["d"], _bytes_per(case)
    lens = _lens(case)
    if case["op"] in ("prefill", "train"):
        tokens = sum(lens)
        pairs = hq * sum(_seen(0, n, case["window"], case["sinks"]) for n in lens)
        rows = B * case["n"]
        if case["op"] == "prefill":
            return {"bytes": z * d * (tokens * (hq + 2 * hkv) + rows * hq) + 4 * rows * hq, "flops": 4 * d * pairs}
        return {"bytes": z * d * (tokens * (2 * hq + 2 * hkv) + rows * (2 * hq + 2 * hkv)) + 4 * rows * hq,
                "flops": 14 * d * pairs}
    new = _new(case)
    if case["op"] == "append":
        tokens = sum(new)
        return {"bytes": 2 * tokens * hkv * d * (z + 1), "flops": 4 * tokens * hkv * d}
    rows = B * case["t"]
    ends = rows * hq * (d * z + 4) + sum(new) * hq * d * z  # o and lse, q
    if case["op"] == "decode":
        pairs = hq * sum(_seen(n - x, n, case["window"], case["sinks"]) for n, x in zip(lens, new))
        first = [max(0, n - x + 1 - case["window"]) for n, x in zip(lens, new)]
        kept = sum(n - f + min(f, case["sinks"]) for n, f in zip(lens, first))
        return {"bytes": 2 * kept * hkv * d + ends, "flops": 4 * d * pairs}
    edges = sum(new) * hkv * case["s"]
    reached = min(edges, sum(lens) * hkv)  # K/V rows read, each counted once
    return {"bytes": 2 * reached * d + 8 * edges + ends, "flops": 4 * d * edges * (hq // hkv)}


# ---- the definition in 64 bits ------------------------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("prefill", "train"):
        return _exact_window(case, st)
    if case["op"] == "append":
        return _exact_append(case, st)
    return _exact_cache(case, st)


def _exact_window(case, st):
    n, G = case["n"], case["hq"] // case["hkv"]
    out = {"o": torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"),
           "lse": torch.full(st["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")}
    if case["op"] == "train":
        out |= {"dq": torch.zeros_like(out["o"])} | {
            "d" + x: torch.zeros(st[x].shape, dtype=torch.float64, device="cuda") for x in ("k", "v")}
    step = 2048  # queries at a time
    for b, length in enumerate(_lens(case)):
        for h in range(case["hq"]):
            k, v = (st[x][b, :length, h // G].double() for x in ("k", "v"))
            for first in range(0, length, step):
                last = min(first + step, length)
                i = torch.arange(first, last, device="cuda")[:, None]
                j = torch.arange(last, device="cuda")[None, :]
                hidden = (j > i) | ((j <= i - case["window"]) & (j >= case["sinks"]))
                q = st["q"][b, first:last, h].double()
                z = torch.einsum("id,jd->ij", q, k[:last]) / math.sqrt(case["d"])
                z[hidden] = -math.inf
                lse = torch.logsumexp(z, 1)
                p = torch.exp(z - lse[:, None])
                out["o"][b, first:last, h] = p @ v[:last]
                out["lse"][b, first:last, h] = lse
                if case["op"] == "train":
                    do = st["dout"][b, first:last, h].double()
                    dz = p * (do @ v[:last].T - (do * (p @ v[:last])).sum(1)[:, None]) / math.sqrt(case["d"])
                    out["dq"][b, first:last, h] = dz @ k[:last]
                    out["dk"][b, :last, h // G] += dz.T @ q
                    out["dv"][b, :last, h // G] += p.T @ do
    return out


def _nearest_e4m3(x):
    """x (fp64, magnitude at most 448) rounded to four significant bits, to even, not below 2^-9 steps."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    return torch.round(x * torch.exp2(3 - e)) * torch.exp2(e - 3)


def _exact_append(case, st):
    page = case["page"]
    out = {}
    for x in ("k", "v"):
        pool, scales = st[x + "q"].double(), st[x + "s"].double()
        for b, (n, have) in enumerate(zip(_new(case), st["lens"].tolist())):
            at = have
            while at < have + n:
                stop = min(have + n, (at // page + 1) * page)
                block, off = int(st["table"][b, at // page]), at % page
                val = st[x][b, at - have: stop - have].double().transpose(0, 1)  # [hkv, tokens, d]
                need = torch.ceil(torch.log2(val.abs().amax((1, 2)) / 448)).clamp(min=E_MIN)
                # the logarithm may round across a whole number: settle it by comparison
                need = torch.where(val.abs().amax((1, 2)) > 448 * torch.exp2(need), need + 1, need)
                low = val.abs().amax((1, 2)) <= 448 * torch.exp2(need - 1)
                need = torch.where(low, need - 1, need).clamp(min=E_MIN)
                scale = torch.exp2(need)
                if off:
                    scale = torch.maximum(scale, scales[block])
                    pool[block, :, :off] = _nearest_e4m3(pool[block, :, :off] * (scales[block] / scale)[:, None, None])
                scales[block] = scale
                pool[block, :, off: off + stop - at] = _nearest_e4m3(val / scale[:, None, None])
                at = stop
        out[x + "q"], out[x + "s"] = pool, scales
    return {"kq": out["kq"], "vq": out["vq"], "ks": out["ks"], "vs": out["vs"]}


def _exact_cache(case, st):
    G, page, t = case["hq"] // case["hkv"], case["page"], case["t"]
    out = {"o": torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"),
           "lse": torch.full(st["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")}
    for b, (length, n) in enumerate(zip(_lens(case), _new(case))):
        blocks = st["table"][b, : -(-length // page)].long()
        # [hkv, length, d]
        k, v = ((st[x + "q"].view(torch.uint8)[blocks].view(F8).double() * st[x + "s"][blocks].double()[:, :, None, None])
                .transpose(0, 1).flatten(1, 2)[:, :length] for x in ("k", "v"))
        pos = torch.arange(length - n, length, device="cuda")
        if case["op"] == "decode":
            for h in range(case["hq"]):
                i, j = pos[:, None], torch.arange(length, device="cuda")[None, :]
                z = st["q"][b, :n, h].double() @ k[h // G].T / math.sqrt(case["d"])
                z[(j > i) | ((i - j >= case["window"]) & (j >= case["sinks"]))] = -math.inf
                out["lse"][b, :n, h] = torch.logsumexp(z, 1)
                out["o"][b, :n, h] = torch.softmax(z, 1) @ v[h // G]
        else:
            for h in range(case["hkv"]):
                idx, w = st["idx"][b, :n, h].long(), st["w"][b, :n, h].double()
                qh = st["q"][b, :n, h * G: (h + 1) * G].double()
                z = torch.einsum("igd,isd->igs", qh, k[h][idx]) / math.sqrt(case["d"]) + w.log()[:, None]
                lse = torch.logsumexp(z, 2)
                p = torch.exp(z - torch.where(lse.isfinite(), lse, 0.0)[:, :, None])
                out["lse"][b, :n, h * G: (h + 1) * G] = lse
                out["o"][b, :n, h * G: (h + 1) * G] = torch.einsum("igs,isd->igd", p, v[h][idx])
    return out
