"""Cases and plain forms of the 8-bit integer operators.

Four operators that stand around the quantised linear layers of a decoder:

* ``linear``     the int8 layer: bf16 tokens are (rotated and) quantised per token and
                 multiplied with int8 weights that have a scale per output channel;
* ``norm_rope``  RMS norm of queries and keys for each head with the position rotation;
* ``update``     the same on the way into an int8 paged cache with a scale for each
                 page of tokens and head: K is normed, rotated and quantised, V is
                 quantised, and the pages that were written are read back;
* ``attention``  attention of one or many new tokens per sequence over that cache.

A case is a dict of plain values; lengths of a ragged batch follow from the case alone
(:func:`lengths`).  ``run`` is the plain form in 32-bit torch operations, or, where
``own`` is true, the calls of the framework.  ``exact`` states the same in 64 bits.
"""

import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: the toy layer of the tests, where only latency counts
        {"name": "linear toy", "op": "linear", "m": 4, "k": 512, "n": 256, "rotate": True},
        # one token through the widest projection: the weights are read once
        {"name": "linear one token", "op": "linear", "m": 1, "k": 5120, "n": 17408, "rotate": True},
        # a decode batch on a layer whose width the rotation block does not divide
        {"name": "linear batch odd width", "op": "linear", "m": 45, "k": 4304, "n": 10010, "rotate": False},
        # a prefill chunk through the widest projection
        {"name": "linear prefill", "op": "linear", "m": 4096, "k": 5120, "n": 17408, "rotate": True},
        # a decode batch: a quarter of each head rotated, heads of 256
        {"name": "norm_rope decode", "op": "norm_rope", "t": 16, "hq": 24, "hk": 4, "d": 256, "rot": 64,
         "interleaved": False, "far": 100000},
        # a prefill chunk, interleaved pairs, the whole head rotated
        {"name": "norm_rope prefill", "op": "norm_rope", "t": 8197, "hq": 32, "hk": 8, "d": 128, "rot": 128,
         "interleaved": True, "far": 30000},
        # one new token for each sequence of a decode batch
        {"name": "update decode", "op": "update", "b": 64, "q": 1, "kv": 8192, "hq": 32, "hk": 8, "d": 128, "page": 64,
         "rot": 128, "interleaved": False, "empty": False},
        # a chunk of a few prompts behind what the cache holds of them, pages ending inside it
        {"name": "update prefill", "op": "update", "b": 3, "q": 1500, "kv": 6000, "hq": 24, "hk": 4, "d": 256, "page": 32,
         "rot": 64, "interleaved": False, "empty": True},
        # two short conversations: latency
        {"name": "attention small", "op": "attention", "b": 2, "q": 1, "kv": 300, "hq": 8, "hk": 2, "d": 64, "page": 16,
         "window": 0, "empty": False},
        # a decode batch of ragged lengths
        {"name": "attention decode batch", "op": "attention", "b": 48, "q": 1, "kv": 16384, "hq": 32, "hk": 8, "d": 128,
         "page": 64, "window": 0, "empty": False},
        # one long context, heads of 256
        {"name": "attention long context", "op": "attention", "b": 1, "q": 1, "kv": 131072, "hq": 24, "hk": 4, "d": 256,
         "page": 64, "window": 0, "empty": False},
        # prefill chunks behind a cached prefix
        {"name": "attention prefill", "op": "attention", "b": 2, "q": 2048, "kv": 8192, "hq": 32, "hk": 8, "d": 128,
         "page": 32, "window": 0, "empty": False},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "norm_rope", "update", "attention", "attention"])
    heads = rng.choice([(24, 4), (32, 8), (8, 2), (16, 16), (12, 1), (20, 4), (7, 1)])
    d = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op == "linear":
        rotate = rng.random() < 0.6
        k = 256 * _spread(rng, 1, 68) if rotate else 16 * _spread(rng, 4, 1088)
        n = _spread(rng, 16, 17408)
        m = _spread(rng, 1, min(8192, int(4096 * 5120 * 17408 / (k * n))))
        return {"op": op, "m": m, "k": k, "n": n, "rotate": rotate}
    if op == "norm_rope":
        return {"op": op, "t": _spread(rng, 1, 8192), "hq": heads[0], "hk": heads[1], "d": d,
                "rot": rng.choice([d, d // 2, d // 4]), "interleaved": rng.random() < 0.5,
                "far": _spread(rng, 100, 1000000)}
    kv = _spread(rng, 4, 32768)
    many = rng.random() < 0.4
    q = _spread(rng, 1, min(kv, 2048)) if many else 1
    b = _spread(rng, 1, max(1, min(48, 500000 // kv, 4096 // q)))
    if op == "update":
        return {"op": op, "b": b, "q": q, "kv": kv, "hq": heads[0], "hk": heads[1], "d": d, "page": page,
                "rot": rng.choice([d, d // 2]), "interleaved": rng.random() < 0.5, "empty": rng.random() < 0.3}
    while b > 1 and b * q * kv * heads[0] * d > 2 * 2048 * 8192 * 32 * 128:
        b -= 1
    while q > 1 and b * q * kv * heads[0] * d > 2 * 2048 * 8192 * 32 * 128:
        q -= 1
    return {"op": op, "b": b, "q": q, "kv": kv, "hq": heads[0], "hk": heads[1], "d": d, "page": page,
            "window": rng.choice([0, 0, 128, 1000]), "empty": rng.random() < 0.3}


def lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence: the first has the case's
    full lengths, the others between a third of them and all of them; with ``empty`` one more
    sequence has nothing new."""
    q, kv = [], []
    for i in range(case["b"]):
        part = 1.0 if i == 0 else 1.0 / 3 + 2.0 / 3 * ((0.6180339887 * i) % 1.0)
        kv.append(max(1, int(case["kv"] * part)))
        q.append(max(1, min(kv[-1], int(case["q"] * part))))
    if case["empty"]:
        q.append(0)
        kv.append(max(1, case["kv"] // 2))
    return q, kv


def pages_of(kv, page):
    return [-(-n // page) for n in kv]


def touched(case):
    """How many pages the new tokens of an update lie in."""
    q, kv = lengths(case)
    return sum((n - 1) // case["page"] - (n - c) // case["page"] + 1 for c, n in zip(q, kv) if c)


def work(case):
    op = case["op"]
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2 * m * k + n * k + 4 * n + 2 * m * n, "flops": 2 * m * n * k}
    h, d = case["hq"] + case["hk"], case["d"]
    if op == "norm_rope":
        return {"bytes": 4 * case["t"] * h * d + 4 * case["t"] + 8 * d, "flops": case["t"] * h * (4 * d + 3 * case["rot"])}
    q, kv = lengths(case)
    t, hk = sum(q), case["hk"]
    if op == "update":
        # q read and written, k and v read; each written page's codes read and its values returned in bf16
        return {"bytes": 4 * t * case["hq"] * d + 4 * t * hk * d + touched(case) * case["page"] * hk * d * 2 * 3 + 4 * t,
                "flops": t * (h * (4 * d + 3 * case["rot"]) + hk * d * 4)}
    pairs, seen = 0, 0
    for c, n in zip(q, kv):
        w = case["window"] or n
        pairs += sum(min(w, p + 1) for p in range(n - c, n))
        seen += min(n, w + c - 1) if c else 0
    return {"bytes": 4 * t * case["hq"] * d + seen * hk * 2 * d, "flops": 4 * pairs * case["hq"] * d}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _hadamard():
    h = torch.ones(1, 1, device="cuda")
    for _ in range(8):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _frequencies(rot):
    i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda")
    return BASE ** (-i / rot)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _sequences(case, s, g):
    """The batch's index arrays: pages handed out in random order, entries past a sequence's pages -1."""
    q, kv = lengths(case)
    n = pages_of(kv, case["page"])
    s["pages"] = sum(n) + 5
    order = torch.randperm(s["pages"], generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(q), max(n)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, c in enumerate(n):
        table[i, :c] = order[at:at + c]
        at += c
    s["table"], s["kv_len"] = table, _ints(kv)
    start = [0]
    for c in q:
        start.append(start[-1] + c)
    s["q_start"], s["t"], s["max_q"], s["max_kv"] = _ints(start), start[-1], max(q), max(kv)


def _codes(g, *shape):
    return (_randn(g, *shape) * 36).round_().clamp_(-127, 127).to(torch.int8)


def _cache(case, s, g):
    shape = (s["pages"], case["hk"], case["page"], case["d"])
    s["k"], s["v"] = _codes(g, *shape), _codes(g, *shape)
    s["k_scale"] = (torch.rand(shape[:2], generator=g, device="cuda") + 0.5) / 36
    s["v_scale"] = (torch.rand(shape[:2], generator=g, device="cuda") + 0.5) / 36


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    op = case["op"]
    if op == "linear":
        x = _randn(g, case["m"], case["k"])
        x[:, torch.randperm(case["k"], generator=g, device="cuda")[: max(1, case["k"] // 100)]] *= 20
        s["x"] = x.to(torch.bfloat16)
        s["w"] = _codes(g, case["n"], case["k"])
        s["w_scale"] = (torch.rand(case["n"], generator=g, device="cuda") + 0.5) * 0.002
        s["h"] = _hadamard() if case["rotate"] else None
        return s
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if op == "norm_rope":
        s["t"] = case["t"]
        s["positions"] = torch.randint(0, case["far"], (case["t"],), generator=g, device="cuda", dtype=torch.int32)
    else:
        _sequences(case, s, g)
    t = s["t"]
    if op == "attention":
        s["q"] = (2 * _randn(g, t, hq, d)).to(torch.bfloat16)
        _cache(case, s, g)
        return s
    # the projections' output: q, k and v of a token lie behind each other in one row
    rows = (hq + 2 * hk) * d
    s["qkv"] = (_randn(g, t, rows) * 3).to(torch.bfloat16)
    s["q"], s["k_new"], s["v_new"] = (x.unflatten(1, (-1, d)) for x in s["qkv"].split([hq * d, hk * d, hk * d], 1))
    s["q_weight"] = 1 + 0.3 * _randn(g, d)
    s["k_weight"] = 1 + 0.3 * _randn(g, d)
    s["inv_freq"] = _frequencies(case["rot"])
    if op == "update":
        _cache(case, s, g)
        q, kv = lengths(case)
        # pages that the call writes, in the order of the sequences
        at = [(i, p) for i, (c, n) in enumerate(zip(q, kv)) if c
              for p in range((n - c) // case["page"], (n - 1) // case["page"] + 1)]
        s["written"] = s["table"][_ints([a for a, _ in at]).long(), _ints([p for _, p in at]).long()].contiguous()
    return s


# ---------------------------------------------------------------- plain forms

def _plain_linear(s):
    x = s["x"].float()
    m, k = x.shape
    if s["h"] is not None:
        x = (x.view(m, k // 256, 256) @ s["h"]).view(m, k) / 16
    scale = x.abs().amax(1, keepdim=True) / 127
    codes = torch.where(scale > 0, (x / scale).round().clamp(-127, 127), torch.zeros_like(x))
    y = codes @ s["w"].float().T
    return (y * scale * s["w_scale"]).to(torch.bfloat16)


def _plain_norm_rope(x, weight, positions, inv_freq, interleaved):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    rot = 2 * inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq[None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    part, rest = x[..., :rot], x[..., rot:]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., : rot // 2], part[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    part = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([part, rest], -1)


def _where_tokens(s):
    """Position in its sequence, page and place in the page of every new token."""
    case, start, kv = s["case"], s["q_start"].long(), s["kv_len"].long()
    token = torch.arange(s["t"], device="cuda")
    seq = torch.searchsorted(start[1:], token, right=True)
    pos = kv[seq] - start[seq + 1] + token
    return pos, s["table"].long()[seq, pos // case["page"]], pos % case["page"]


def _plain_store(codes, scales, x, page, slot, fresh, live, written):
    """x [t, heads, d] into the pages: their scales grow to what the new values need, codes that were there are
    rounded anew under a grown scale."""
    need = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(-1) / 127, "amax")
    old = torch.where(fresh[:, None], torch.zeros_like(scales), scales)
    new = torch.maximum(old, need)
    ratio = torch.where(new > 0, old / new, torch.ones_like(new))[written]
    was = codes[written].float()
    keep = live[written][:, None, :, None] & ~fresh[written][:, None, None, None]
    codes[written] = torch.where(keep, (was * ratio[:, :, None, None]).round(), was).to(torch.int8)
    scales[written] = new[written]
    by = new[page][..., None]
    codes[page, :, slot] = torch.where(by > 0, (x / by).round().clamp(-127, 127), torch.zeros_like(x)).to(torch.int8)


def _plain_update(s):
    case = s["case"]
    pos, page, slot = _where_tokens(s)
    q = _plain_norm_rope(s["q"], s["q_weight"], pos, s["inv_freq"], case["interleaved"]).to(torch.bfloat16)
    k = _plain_norm_rope(s["k_new"], s["k_weight"], pos, s["inv_freq"], case["interleaved"])
    v = s["v_new"].float()
    fresh = torch.zeros(s["pages"], dtype=torch.bool, device="cuda")
    fresh[page[slot == 0]] = True
    first = torch.full((s["pages"],), case["page"], dtype=torch.long, device="cuda")
    first.index_reduce_(0, page, slot, "amin")
    live = torch.arange(case["page"], device="cuda")[None, :] < first[:, None]
    written = s["written"].long()
    _plain_store(s["k"], s["k_scale"], k, page, slot, fresh, live, written)
    _plain_store(s["v"], s["v_scale"], v, page, slot, fresh, live, written)
    values = [(c[written].float() * m[written][:, :, None, None]).to(torch.bfloat16)
              for c, m in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"]))]
    return {"q": q, "k": values[0], "v": values[1]}


def _plain_gather(codes, scales, table):
    """Pages of every sequence -> [b, heads, tokens, d] in fp32."""
    at = table.long().clamp(min=0)
    x = codes[at].float() * scales[at][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attention(s):
    case = s["case"]
    hq, hk, d = case["hq"], case["hk"], case["d"]
    group = hq // hk
    start, kv = s["q_start"].long(), s["kv_len"].long()
    count = start[1:] - start[:-1]
    step = torch.arange(s["max_q"], device="cuda")
    row = (start[:-1, None] + step).clamp(max=s["t"] - 1)
    q = s["q"].float()[row].unflatten(2, (hk, group))                      # [b, q, hk, group, d]
    b = q.shape[0]
    q = q.permute(0, 2, 3, 1, 4).reshape(b, hk, group * s["max_q"], d)
    k = _plain_gather(s["k"], s["k_scale"], s["table"])
    v = _plain_gather(s["v"], s["v_scale"], s["table"])
    scores = (q @ k.transpose(2, 3)) / math.sqrt(d)
    pos = (kv - count)[:, None] + step                                      # [b, q]
    key = torch.arange(k.shape[2], device="cuda")
    seen = (key <= pos[..., None]) & (step[None, :, None] < count[:, None, None]) & (key < kv[:, None, None])
    if case["window"]:
        seen &= key > pos[..., None] - case["window"]
    scores = scores.view(b, hk, group, s["max_q"], -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = (scores - torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    out = p.flatten(2, 3) @ v
    out = out.view(b, hk, group, s["max_q"], d) / torch.where(total > 0, total, torch.ones_like(total))
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)                          # [b, q, hq, d]
    return out[step[None, :] < count[:, None]].to(torch.bfloat16)


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from w4a8_codebook_quantized_rotate_b200 import binding as B
        if op == "linear":
            if "workspace" not in s:
                s["workspace"] = B.int8_linear_workspace(case["m"], case["k"], case["n"], "cuda")
            return B.int8_linear(s["x"], s["w"], s["w_scale"], rotate=case["rotate"], workspace=s["workspace"])
        if op == "norm_rope":
            return B.qk_norm_rope(s["q"], s["k_new"], s["positions"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                  eps=EPS, inv_freq=s["inv_freq"], interleaved=case["interleaved"])
        if "cache" not in s:
            s["cache"] = B.KvCache.of(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if op == "update":
            q = B.kv_update(s["cache"], s["k_new"], s["v_new"], s["table"], s["q_start"], s["kv_len"], q=s["q"],
                            q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, inv_freq=s["inv_freq"],
                            interleaved=case["interleaved"])
            k, v = B.kv_dequant(s["cache"], s["written"])
            return {"q": q, "k": k, "v": v}
        if "workspace" not in s:
            s["workspace"] = B.kv_attention_workspace(s["q"].shape[0], case["hq"], case["hk"], case["d"], "cuda")
        return B.kv_attention(s["q"], s["cache"], s["table"], s["q_start"], s["kv_len"], window=case["window"],
                              workspace=s["workspace"])
    if op == "linear":
        return _plain_linear(s)
    if op == "norm_rope":
        return tuple(_plain_norm_rope(x, w, s["positions"], s["inv_freq"], case["interleaved"]).to(torch.bfloat16)
                     for x, w in ((s["q"], s["q_weight"]), (s["k_new"], s["k_weight"])))
    return _plain_update(s) if op == "update" else _plain_attention(s)


# ---------------------------------------------------------------- in 64 bits

def _exact_heads(x, weight, positions, rot, interleaved):
    """Head by head: x / rms(x) * weight, then each pair turned by its angle (as complex numbers)."""
    x = x.double()
    x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    i = torch.arange(rot // 2, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones_like(i)[None, :].expand(positions.numel(), -1).contiguous(),
                       positions.double()[:, None] * torch.pow(BASE, -2 * i / rot)[None, :])[:, None, :]
    y = x.clone()
    re, im = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * turn
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_page(codes, scale, rows, first):
    """One head's page: codes [page, d] and scale with `rows` [n, d] written from place `first` on -> its values."""
    held = codes.double().clone()
    need = rows.abs().max().item() / 127
    new = need if first == 0 else max(scale, need)
    if first and new > scale:
        held[:first] = (held[:first] * (scale / new)).round()
    held[first:first + rows.shape[0]] = (rows / new).round().clamp(-127, 127) if new > 0 else 0.0
    return held * new


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        x = s["x"].double()
        if case["rotate"]:
            i = torch.arange(256, device="cuda")
            both = i[:, None] & i[None, :]
            odd = sum((both >> b) & 1 for b in range(8)) % 2
            x = torch.einsum("mbi,ij->mbj", x.view(x.shape[0], -1, 256), 1.0 - 2.0 * odd.double()).reshape(x.shape) / 16
        top = x.abs().max(1).values
        step = torch.where(top > 0, top / 127, torch.ones_like(top))[:, None]
        return torch.einsum("mk,nk->mn", torch.round(x / step), s["w"].double()) * step * s["w_scale"].double()[None, :]
    if op == "norm_rope":
        return tuple(_exact_heads(x, w, s["positions"], case["rot"], case["interleaved"])
                     for x, w in ((s["q"], s["q_weight"]), (s["k_new"], s["k_weight"])))
    q_len, kv_len = lengths(case)
    page, hk = case["page"], case["hk"]
    if op == "update":
        if touched(case) * hk > 4096:
            return None
        pos = torch.cat([torch.arange(n - c, n) for c, n in zip(q_len, kv_len)]).cuda()
        q = _exact_heads(s["q"], s["q_weight"], pos, case["rot"], case["interleaved"])
        new = (_exact_heads(s["k_new"], s["k_weight"], pos, case["rot"], case["interleaved"]), s["v_new"].double())
        held, scales = (s["k"], s["v"]), (s["k_scale"].tolist(), s["v_scale"].tolist())
        table, out, t = s["table"].tolist(), ([], []), 0
        for i, (c, n) in enumerate(zip(q_len, kv_len)):
            for p in range((n - c) // page, (n - 1) // page + 1 if c else 0):
                lo, hi = max(n - c, p * page), min(n, (p + 1) * page)
                at, rows = table[i][p], slice(t + lo - (n - c), t + hi - (n - c))
                for kind in (0, 1):
                    out[kind].append(torch.stack([
                        _exact_page(held[kind][at, h], scales[kind][at][h], new[kind][rows, h], lo - p * page)
                        for h in range(hk)]))
            t += c
        return {"q": q, "k": torch.stack(out[0]), "v": torch.stack(out[1])}
    group, out, t = case["hq"] // hk, [], 0
    for i, (c, n) in enumerate(zip(q_len, kv_len)):
        if not c:
            continue
        at = s["table"][i, : -(-n // page)].long()
        k, v = ((x[at].double() * m[at].double()[:, :, None, None]).permute(1, 0, 2, 3).reshape(hk, -1, case["d"])[:, :n]
                for x, m in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])))
        mine = torch.arange(n - c, n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")[None, :]
        hidden = (key > mine) | ((key <= mine - case["window"]) if case["window"] else torch.zeros_like(key > mine))
        rows = torch.empty(c, case["hq"], case["d"], dtype=torch.float64, device="cuda")
        for h in range(case["hq"]):
            a = torch.einsum("qd,kd->qk", s["q"][t:t + c, h].double(), k[h // group]) * case["d"] ** -0.5
            rows[:, h] = torch.einsum("qk,kd->qd", torch.softmax(a.masked_fill(hidden, -math.inf), -1), v[h // group])
        out.append(rows)
        t += c
    return torch.cat(out)
