"""What the paged-cache and packed-prompt operators are measured on.

Three operators, all with head_dim 128 and 16-bit keys and values:

* ``prompt``: attention over packed prompts of different lengths, grouped heads, causal or not;
* ``decode``: attention of a batch's newest tokens over the pages of a cache whose leading tokens the batch shares;
* ``cache``: the pages themselves: extended and written, forked, freed and compacted.

``run`` computes them from elementary torch operations in 32 bits, or, where ``own`` is set, calls the library.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
SCORES = 6 << 30          # the plain forms hold at most about this many bytes of scores at a time


def listed():
    return [
        # a handful of short text prompts for a text encoder: latency
        {"name": "prompt text", "op": "prompt", "seqs": 5, "lo": 1, "hi": 77, "past": 0, "hq": 24, "hkv": 24, "type": "fp16", "causal": True, "lens": 1},
        # a batch of prompts of ordinary, ragged lengths, packed
        {"name": "prompt batch", "op": "prompt", "seqs": 13, "lo": 40, "hi": 2048, "past": 0, "hq": 32, "hkv": 8, "type": "bf16", "causal": True, "lens": 2},
        # one long document
        {"name": "prompt long", "op": "prompt", "seqs": 1, "lo": 32768, "hi": 32768, "past": 0, "hq": 40, "hkv": 8, "type": "fp16", "causal": True, "lens": 3},
        # the next chunk of two prompts whose beginnings are there already
        {"name": "prompt chunk", "op": "prompt", "seqs": 2, "lo": 65, "hi": 160, "past": 30000, "hq": 64, "hkv": 8, "type": "bf16", "causal": True, "lens": 4},
        # short clips' tokens attending to each other both ways
        {"name": "prompt both ways", "op": "prompt", "seqs": 3, "lo": 1000, "hi": 5000, "past": 0, "hq": 24, "hkv": 24, "type": "bf16", "causal": False, "lens": 5},
        # one user, one token: latency
        {"name": "decode one", "op": "decode", "seqs": 1, "new": 1, "shared": 0, "lo": 333, "hi": 333, "hq": 24, "hkv": 24, "page": 16, "type": "fp16", "lens": 6},
        # a batch behind one instruction text
        {"name": "decode batch", "op": "decode", "seqs": 61, "new": 1, "shared": 2048, "lo": 1, "hi": 1024, "hq": 32, "hkv": 8, "page": 16, "type": "bf16", "lens": 7},
        # unrelated conversations of very different lengths
        {"name": "decode ragged", "op": "decode", "seqs": 48, "new": 1, "shared": 0, "lo": 1, "hi": 16384, "hq": 40, "hkv": 8, "page": 64, "type": "fp16", "lens": 8},
        # many answers about one long document, three drafted tokens each to verify
        {"name": "decode document", "op": "decode", "seqs": 250, "new": 3, "shared": 32768, "lo": 3, "hi": 700, "hq": 64, "hkv": 8, "page": 128, "type": "bf16", "lens": 9},
        # one step of a serving loop: a token more for each sequence, one layer's keys and values
        {"name": "cache step", "op": "cache", "do": "step", "seqs": 64, "lo": 1, "hi": 4096, "new": 1, "layers": 1, "hkv": 8, "page": 16, "type": "bf16", "lens": 10},
        # a search that keeps 60 continuations of a few texts
        {"name": "cache fork", "op": "cache", "do": "fork", "seqs": 60, "lo": 100, "hi": 3000, "new": 0, "layers": 24, "hkv": 8, "page": 64, "type": "fp16", "lens": 11},
        # every other conversation ends, and the rest move together
        {"name": "cache compact", "op": "cache", "do": "compact", "seqs": 96, "lo": 200, "hi": 6000, "new": 0, "layers": 8, "hkv": 8, "page": 32, "type": "bf16", "lens": 12},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "decode", "decode", "cache"])
    hq, hkv = rng.choice([(24, 24), (32, 8), (40, 8), (64, 8), (28, 4), (16, 1), (6, 2)])
    case = {"op": op, "hkv": hkv, "type": rng.choice(["fp16", "bf16"]), "lens": rng.randrange(1 << 20)}
    if op == "prompt":
        hi = _spread(rng, 1, 8000)
        past = rng.choice([0, 0, _spread(rng, 1, 30000)])
        if past:
            hi = min(hi, 2000)
        seqs = max(1, min(_spread(rng, 1, 64), 24000 // (hi + past)))
        case |= {"hq": hq, "seqs": seqs, "lo": rng.randint(1, hi), "hi": hi, "past": past, "causal": bool(past) or rng.random() < 0.7}
    elif op == "decode":
        new = rng.choice([1, 1, 1, 2, 5])
        page = rng.choice([16, 32, 64, 128])
        hi = new - 1 + _spread(rng, 1, 16000)
        seqs = max(1, min(_spread(rng, 1, 250), 400000 // hi))
        shared = rng.choice([0, _spread(rng, 1, 30000) // page * page])
        case |= {"hq": hq, "seqs": seqs, "new": new, "shared": shared, "lo": rng.randint(new, hi), "hi": hi, "page": page}
    else:
        do = rng.choice(["step", "fork", "compact"])
        hi = _spread(rng, 2, 5000)
        seqs = max(2, min(_spread(rng, 2, 120), 200000 // hi))
        new = _spread(rng, 1, 300) if do == "step" else 0
        case |= {"do": do, "seqs": seqs, "lo": rng.randint(1, hi), "hi": hi, "new": new,
                 "layers": 1 if do == "step" else _spread(rng, 1, 16), "page": rng.choice([16, 32, 64, 128])}
    return case


# ---------------------------------------------------------------- what the cases consist of

def _lengths(case):
    """A length for each sequence: the two ends of the range first, then spread over its logarithm."""
    rng = random.Random(case["lens"])
    return [case["hi"] if i == 0 else case["lo"] if i == 1 else _spread(rng, case["lo"], case["hi"]) for i in range(case["seqs"])]


def _deal(lens, page):
    """Page numbers for sequences that grew side by side: their pages alternate."""
    count = [-(-n // page) for n in lens]
    rows, at = [[] for _ in lens], 0
    for k in range(max(count)):
        for i, c in enumerate(count):
            if k < c:
                rows[i].append(at)
                at += 1
    return rows, at


def _pages(case):
    """{n_pages, rows, lens, max_seqs, max_pages} of the cache that a case starts with."""
    lens, page, n = _lengths(case), case["page"], case["seqs"]
    if case["op"] == "decode":
        own_rows, used = _deal(lens, page)
        lead = case["shared"] // page
        rows = [list(range(used, used + lead)) + r for r in own_rows]
        lens = [case["shared"] + m for m in lens]
        return {"n_pages": used + lead + 3, "rows": rows, "lens": lens, "max_seqs": n + 1, "max_pages": max(map(len, rows)) + 1}
    if case["do"] == "fork":        # the first few sequences are there, the others will continue them
        have = max(1, n // 12)
        lens = lens[:have] + [0] * (n - have)
    rows, used = _deal(lens, page)
    grow = -(-case["new"] // page) + 1
    return {"n_pages": used + n * grow + 7, "rows": rows, "lens": lens, "max_seqs": n + 2, "max_pages": max(map(len, rows)) + grow}


def _up(n):
    return -(-n // 64) * 64         # 256 bytes of int32


def _state(c):
    """The int32 state of a cache as one array: how many rows name each page, each row's length, the table."""
    r, m, w = _up(c["n_pages"]), _up(c["max_seqs"]), c["max_seqs"] * c["max_pages"]
    s = np.zeros(r + m + _up(w), np.int32)
    table = np.full((c["max_seqs"], c["max_pages"]), -1, np.int32)
    for i, row in enumerate(c["rows"]):
        table[i, :len(row)] = row
        np.add.at(s, np.array(row, np.int64), 1)
        s[r + i] = c["lens"][i]
    s[r + m:r + m + w] = table.reshape(-1)
    return s


def _views(s, c):
    r, m, w = _up(c["n_pages"]), _up(c["max_seqs"]), c["max_seqs"] * c["max_pages"]
    return s[:c["n_pages"]], s[r:r + c["max_seqs"]], s[r + m:r + m + w].view(c["max_seqs"], c["max_pages"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = TYPES[case["type"]]

    def normal(*shape, wide=0.0):
        x = torch.randn(*shape, device="cuda", generator=g, dtype=torch.float32 if wide else kind)
        return (x * torch.exp(wide * torch.randn(shape[-1], device="cuda", generator=g))).to(kind) if wide else x

    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "prompt":
        lens = _lengths(case)
        s["cu_q"] = ints([0] + np.cumsum(lens).tolist())
        s["cu_k"] = ints([0] + np.cumsum([n + case["past"] for n in lens]).tolist())
        s["max_q"], s["max_k"] = max(lens), max(lens) + case["past"]
        tq, tk = sum(lens), sum(lens) + case["past"] * case["seqs"]
        s["q"], s["k"], s["v"] = normal(tq, case["hq"], D, wide=0.3), normal(tk, case["hkv"], D, wide=0.3), normal(tk, case["hkv"], D)
        if own:
            from int4_quantized_attention_b200 import api
            s["op"] = api.PackedAttention()
        return s
    c = _pages(case)
    s["dims"] = c
    layers = case.get("layers", 1)
    s["pool"] = normal(2, layers, c["n_pages"], case["hkv"], case["page"], D)
    first = torch.from_numpy(_state(c)).cuda()
    s["first"], s["state"] = first, first.clone()
    n = case["seqs"]
    s["seqs"] = ints(list(range(n)))
    if case["op"] == "decode":
        s["q"] = normal(n * case["new"], case["hq"], D, wide=0.3)
        s["cu_q"] = ints([i * case["new"] for i in range(n + 1)]) if case["new"] > 1 else None
        s["max_own"] = max(c["lens"]) - case["shared"]
    elif case["do"] == "step":
        s["new"] = ints([case["new"]] * n)
        s["cu_new"] = ints([i * case["new"] for i in range(n + 1)]) if case["new"] > 1 else None
        s["k"], s["v"] = normal(n * case["new"], case["hkv"], D), normal(n * case["new"], case["hkv"], D)
    elif case["do"] == "fork":
        have = max(1, n // 12)
        s["parents"], s["children"] = ints([i % have for i in range(have, n)]), ints(list(range(have, n)))
    else:
        s["ended"] = ints(list(range(0, n, 2)))
    if own:
        from int4_quantized_attention_b200 import api
        s["op"] = api.PagedCache(layers, c["n_pages"], case["page"], case["hkv"], c["max_seqs"], c["max_pages"],
                                 dtype=kind, pool=s["pool"], state=s["state"])
    return s


# ---------------------------------------------------------------- the passes

def run(s):
    case = s["case"]
    if case["op"] == "prompt":
        if own:
            o, lse = s["op"].forward(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=case["causal"], return_lse=True)
        else:
            o, lse = _prompt(s)
        return {"o": o, "lse": lse}
    if case["op"] == "decode":
        if own:
            o, lse = s["op"].attention(0, s["q"], s["seqs"], cu_q=s["cu_q"], shared=case["shared"], return_lse=True)
        else:
            o, lse = _decode(s)
        return {"o": o, "lse": lse}
    # the pages are changed in place: each pass begins where the first one did
    s["state"].copy_(s["first"])
    if case["do"] == "step":
        if own:
            s["op"].extend(s["seqs"], s["new"])
            s["op"].write(0, s["seqs"], s["k"], s["v"], cu_new=s["cu_new"])
        else:
            _extend(s)
            _write(s)
    elif case["do"] == "fork":
        if own:
            s["op"].fork(s["parents"], s["children"])
        else:
            _fork(s)
    elif own:
        s["op"].free(s["ended"])
        s["op"].compact()
    else:
        _free(s)
        _compact(s)
    refs, lens, table = _views(s["state"], s["dims"])
    return {"pool": s["pool"], "refs": refs, "lens": lens, "table": table}


def _softmax_(x):
    """exp(x - max) in place, its row sums and its row maxima; rows of -inf give zeros."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(m).exp_()
    return x.sum(-1, keepdim=True), m


def _prompt(s):
    case, q, k, v = s["case"], s["q"], s["k"], s["v"]
    n, hq, hkv, mq, mk = case["seqs"], case["hq"], case["hkv"], s["max_q"], s["max_k"]
    group, dev = hq // hkv, q.device
    lq, lk = (s["cu_q"][1:] - s["cu_q"][:-1]).long(), (s["cu_k"][1:] - s["cu_k"][:-1]).long()
    iq, ik = torch.arange(mq, device=dev), torch.arange(mk, device=dev)
    rows = (s["cu_q"][:-1, None] + iq).clamp(max=q.shape[0] - 1).long()
    keys = (s["cu_k"][:-1, None] + ik).clamp(max=k.shape[0] - 1).long()
    seen = ik < lk[:, None, None]
    if case["causal"]:
        seen = seen & (ik <= iq[:, None] + (lk - lq)[:, None, None])
    hidden = ~seen[:, None, None]                                                      # [n, 1, 1, mq or 1, mk]
    o = torch.empty(n, mq, hkv, group, D, device=dev)
    lse = torch.empty(n, mq, hkv, group, device=dev)
    step = max(1, SCORES // (4 * n * group * mq * mk))
    for h in range(0, hkv, step):                                                      # as many heads at a time as fit
        e = min(hkv, h + step)
        qh = q.view(-1, hkv, group, D)[:, h:e][rows].float().permute(0, 2, 3, 1, 4)    # [n, h, group, mq, D]
        kh, vh = (x[:, h:e][keys].float().permute(0, 2, 1, 3) for x in (k, v))         # [n, h, mk, D]
        x = (qh.reshape(n, e - h, group * mq, D) @ kh.transpose(-1, -2)).mul_(1 / math.sqrt(D)).view(n, e - h, group, mq, mk)
        x.masked_fill_(hidden, -math.inf)
        total, top = _softmax_(x)
        y = (x.view(n, e - h, group * mq, mk) @ vh).view(n, e - h, group, mq, D) / total
        o[:, :, h:e] = y.permute(0, 3, 1, 2, 4)
        lse[:, :, h:e] = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2)
    at = (torch.arange(q.shape[0], device=dev)[:, None] >= s["cu_q"][None, 1:]).sum(1)  # the sequence of each row
    within = torch.arange(q.shape[0], device=dev) - s["cu_q"].long()[at]
    return o[at, within].reshape(-1, hq, D).to(q.dtype), lse[at, within].reshape(-1, hq)


def _decode(s):
    case, q, dev = s["case"], s["q"], s["q"].device
    n, new, hq, hkv, page, shared = case["seqs"], case["new"], case["hq"], case["hkv"], case["page"], case["shared"]
    group, longest, lead = hq // hkv, s["max_own"], case["shared"] // case["page"]
    _, lens, table = _views(s["state"], s["dims"])
    k, v = s["pool"][0, 0], s["pool"][1, 0]                                             # [pages, hkv, page, D]
    qf = q.view(n, new, hkv, group, D).float().permute(2, 0, 3, 1, 4)                   # [hkv, n, group, new, D]
    rows = table[s["seqs"].long(), lead:lead + -(-longest // page)].clamp(min=0).long()
    width = rows.shape[1] * page
    own_len = lens[s["seqs"].long()].long() - shared
    j = torch.arange(width, device=dev)
    seen = j[None, None] < (own_len[:, None] - new + 1 + torch.arange(new, device=dev))[:, :, None]     # [n, new, width]
    o = torch.empty(n, new, hkv, group, D, device=dev)
    lse = torch.empty(n, new, hkv, group, device=dev)
    step = max(1, SCORES // (4 * n * max(group * new * (shared + width), 2 * D * width)))
    for h in range(0, hkv, step):                                                       # as many heads at a time as fit
        e = min(hkv, h + step)
        qh = qf[h:e]
        ko, vo = (x[:, h:e][rows].float().permute(2, 0, 1, 3, 4).reshape(e - h, n, width, D) for x in (k, v))
        own_x = (qh.reshape(e - h, n, group * new, D) @ ko.transpose(-1, -2)).view(e - h, n, group, new, width)
        own_x.masked_fill_(~seen[:, None], -math.inf)
        first = table[s["seqs"][0].long(), :lead].long()
        kp, vp = (x[:, h:e][first].float().permute(1, 0, 2, 3).reshape(e - h, shared, D) for x in (k, v))
        led_x = (qh.reshape(e - h, n * group * new, D) @ kp.transpose(-1, -2)).view(e - h, n, group, new, shared)
        x = torch.cat([led_x, own_x], -1).mul_(1 / math.sqrt(D))
        total, top = _softmax_(x)
        y = (x[..., :shared].reshape(e - h, n * group * new, shared) @ vp).view(e - h, n, group, new, D)
        y = (y + (x[..., shared:].reshape(e - h, n, group * new, width) @ vo).view(e - h, n, group, new, D)) / total
        o[:, :, h:e] = y.permute(1, 3, 0, 2, 4)
        lse[:, :, h:e] = (top + total.log()).squeeze(-1).permute(1, 3, 0, 2)
    return o.view(n * new, hq, D).to(q.dtype), lse.view(n * new, hq)


def _lowest_free(refs):
    """The free pages' numbers in order, padded with the number of pages."""
    free, n = refs == 0, refs.numel()
    ids = torch.arange(n, device=refs.device)
    out = torch.full((n + 1,), n, dtype=torch.long, device=refs.device)
    out[torch.where(free, torch.cumsum(free, 0) - 1, n)] = torch.where(free, ids, n)
    return out[:n]


def _extend(s):
    page, (refs, lens, table) = s["case"]["page"], _views(s["state"], s["dims"])
    seqs, wide = s["seqs"].long(), table.shape[1]
    before = lens[seqs].long()
    have, want = (before + page - 1) // page, (before + s["new"] + page - 1) // page
    need = want - have
    k = torch.arange(-(-s["case"]["new"] // page) + 1, device=refs.device)
    real = k < need[:, None]
    rank = (torch.cumsum(need, 0) - need)[:, None] + k
    pages = _lowest_free(refs)[rank.clamp(max=refs.numel() - 1)]
    flat = torch.cat([table.reshape(-1), table.new_zeros(1)])
    flat[torch.where(real, seqs[:, None] * wide + have[:, None] + k, flat.numel() - 1)] = pages.to(torch.int32)
    table.copy_(flat[:-1].view_as(table))
    more = torch.cat([refs, refs.new_zeros(1)])
    more[torch.where(real, pages, refs.numel())] = 1
    refs.copy_(more[:-1])
    lens[seqs] += s["new"]


def _write(s):
    case, (_, lens, table) = s["case"], _views(s["state"], s["dims"])
    seqs, new = s["seqs"].long(), case["new"]
    at = (lens[seqs].long()[:, None] - new + torch.arange(new, device=lens.device))
    pages = table[seqs[:, None], at // case["page"]].long().reshape(-1)
    off = (at % case["page"]).reshape(-1)
    s["pool"][0, 0][pages, :, off] = s["k"]
    s["pool"][1, 0][pages, :, off] = s["v"]


def _fork(s):
    page, (refs, lens, table) = s["case"]["page"], _views(s["state"], s["dims"])
    parents, children = s["parents"].long(), s["children"].long()
    rows, length = table[parents], lens[parents].long()
    full, rest = length // page, length % page
    col = torch.arange(table.shape[1], device=refs.device)
    keep = col < full[:, None]
    part = rest > 0
    rank = torch.cumsum(part, 0) - part.long()
    last = rows.gather(1, torch.where(part, full, (full - 1).clamp(min=0))[:, None]).squeeze(1).long()
    fresh = torch.where(part, _lowest_free(refs)[rank], last)
    mask = (torch.arange(page, device=refs.device) < rest[:, None])[:, None, :, None]          # [n, 1, page, 1]
    s["pool"][:, :, fresh] = torch.where(mask, s["pool"][:, :, last], s["pool"][:, :, fresh])
    refs.index_add_(0, rows.clamp(min=0).reshape(-1).long(), keep.reshape(-1).to(torch.int32))
    refs.index_add_(0, fresh, part.to(torch.int32))
    table[children] = torch.where(keep, rows, torch.where((col == full[:, None]) & part[:, None], fresh[:, None], -1).to(torch.int32))
    lens[children] = length.to(torch.int32)


def _free(s):
    refs, lens, table = _views(s["state"], s["dims"])
    seqs = s["ended"].long()
    rows = table[seqs]
    refs.index_add_(0, rows.clamp(min=0).reshape(-1).long(), -(rows >= 0).reshape(-1).to(torch.int32))
    table[seqs] = -1
    lens[seqs] = 0


def _compact(s):
    refs, _, table = _views(s["state"], s["dims"])
    ids, live = torch.arange(refs.numel(), device=refs.device), refs > 0
    count = live.sum()
    holes, movers = (~live & (ids < count)).nonzero().squeeze(1), (live & (ids >= count)).nonzero().squeeze(1)
    s["pool"][:, :, holes] = s["pool"][:, :, movers]
    to = ids.clone()
    to[movers] = holes
    refs[holes] = refs[movers]
    refs[movers] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))


# ---------------------------------------------------------------- what they cost, and what is right

def work(case):
    if case["op"] == "prompt":
        lens, past = _lengths(case), case["past"]
        pairs = sum(n * (past + n) - (n * (n - 1) // 2 if case["causal"] else 0) for n in lens)
        tq, tk = sum(lens), sum(lens) + past * len(lens)
        return {"bytes": 2 * D * (2 * tq * case["hq"] + 2 * tk * case["hkv"]) + 4 * tq * case["hq"], "flops": 4 * D * case["hq"] * pairs}
    if case["op"] == "decode":
        lens, new = _lengths(case), case["new"]
        keys = case["shared"] + sum(lens)
        pairs = sum(new * (case["shared"] + n) - new * (new - 1) // 2 for n in lens)
        rows = len(lens) * new * case["hq"]
        return {"bytes": 4 * D * keys * case["hkv"] + (4 * D + 4) * rows + 4 * (keys // case["page"] + len(lens)), "flops": 4 * D * case["hq"] * pairs}
    c, token = _pages(case), 4 * D * case["hkv"] * case["layers"]            # a token's keys and values
    state = 4 * (c["n_pages"] + c["max_seqs"])
    if case["do"] == "step":
        moved = case["seqs"] * case["new"]
    elif case["do"] == "fork":
        have = max(1, case["seqs"] // 12)
        moved = sum(c["lens"][i % have] % case["page"] for i in range(have, case["seqs"]))
    else:
        kept = np.concatenate([np.array(r, np.int64) for r in c["rows"][1::2]])
        moved = int((kept >= kept.size).sum()) * case["page"]
        state += 8 * sum(map(len, c["rows"]))
    return {"bytes": 2 * token * moved + state, "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(s)
    if case["op"] == "decode":
        return _exact_decode(s)
    return _exact_cache(s)


def _attend64(q, k, v, limit):
    """One head in 64 bits: q [rows, D], k and v [keys, D], row i sees the first limit[i] keys."""
    x = q.double() @ k.double().T / math.sqrt(D)
    x[torch.arange(k.shape[0], device=q.device) >= limit[:, None]] = -math.inf
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[:, None]) @ v.double(), lse


def _exact_prompt(s):
    case, q, k, v = s["case"], s["q"], s["k"], s["v"]
    o = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for i in range(case["seqs"]):
        lq, lk = cq[i + 1] - cq[i], ck[i + 1] - ck[i]
        ks, vs = k[ck[i]:ck[i + 1]], v[ck[i]:ck[i + 1]]
        for a in range(0, lq, 4096):
            rows = torch.arange(a, min(lq, a + 4096), device=q.device)
            limit = rows + 1 + lk - lq if case["causal"] else torch.full_like(rows, lk)
            for h in range(case["hq"]):
                kv = h * case["hkv"] // case["hq"]
                at = cq[i] + rows
                o[at, h], lse[at, h] = _attend64(q[at, h], ks[:, kv], vs[:, kv], limit)
    return {"o": o, "lse": lse}


def _exact_decode(s):
    case, c, q = s["case"], s["dims"], s["q"]
    page, new, group = case["page"], case["new"], case["hq"] // case["hkv"]
    o = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    for i in range(case["seqs"]):
        pages, n = torch.tensor(c["rows"][i], device=q.device), c["lens"][i]
        at = torch.arange(i * new, (i + 1) * new, device=q.device)
        limit = torch.arange(n - new + 1, n + 1, device=q.device).repeat(group)
        for h in range(case["hkv"]):
            k, v = (s["pool"][x, 0, pages, h].reshape(-1, D)[:n] for x in (0, 1))
            heads = slice(h * group, (h + 1) * group)
            y, z = _attend64(q[at, heads].transpose(0, 1).reshape(-1, D), k, v, limit)
            o[at, heads], lse[at, heads] = y.view(group, new, D).transpose(0, 1), z.view(group, new).T
    return {"o": o, "lse": lse}


def _exact_cache(s):
    """The pages by the operators' definition, one sequence and one page after another on the host."""
    case, c, page = s["case"], s["dims"], s["case"]["page"]
    rows, lens = [list(r) for r in c["rows"]], list(c["lens"])
    rows += [[] for _ in range(c["max_seqs"] - len(rows))]
    lens += [0] * (c["max_seqs"] - len(lens))
    refs = np.zeros(c["n_pages"], np.int64)
    for r in rows:
        refs[r] += 1
    pool = s["pool"].clone()
    if case["do"] == "step":
        for i in range(case["seqs"]):
            for t in range(case["new"]):
                if lens[i] % page == 0:
                    rows[i].append(int(np.argmin(refs != 0)))
                    refs[rows[i][-1]] = 1
                lens[i] += 1
            first = i * case["new"]
            for a in range(lens[i] - case["new"], lens[i]):
                pool[0, 0, rows[i][a // page], :, a % page] = s["k"][first + a - lens[i] + case["new"]]
                pool[1, 0, rows[i][a // page], :, a % page] = s["v"][first + a - lens[i] + case["new"]]
    elif case["do"] == "fork":
        for p, child in zip(s["parents"].tolist(), s["children"].tolist()):
            full, rest = divmod(lens[p], page)
            rows[child], lens[child] = rows[p][:full], lens[p]
            if rest:
                new = int(np.argmin(refs != 0))
                rows[child].append(new)
                pool[:, :, new, :, :rest] = pool[:, :, rows[p][full], :, :rest]
            for x in rows[child]:
                refs[x] += 1
    else:
        for i in s["ended"].tolist():
            refs[rows[i]] -= 1
            rows[i], lens[i] = [], 0
        count = int((refs > 0).sum())
        moves = dict(zip([i for i in range(count, c["n_pages"]) if refs[i] > 0], [i for i in range(count) if refs[i] == 0]))
        for a, b in moves.items():
            pool[:, :, b] = pool[:, :, a]
            refs[b], refs[a] = refs[a], 0
        rows = [[moves.get(x, x) for x in r] for r in rows]
    table = np.full((c["max_seqs"], c["max_pages"]), -1)
    for i, r in enumerate(rows):
        table[i, :len(r)] = r
    ints = lambda v: torch.tensor(np.array(v), dtype=torch.int32)  # noqa: E731
    return {"pool": pool, "refs": ints(refs), "lens": ints(lens), "table": ints(table)}
