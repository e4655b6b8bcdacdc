"""Cases of the operators that serve several requests at once, their plain forms and their values in 64 bits.

Three operators, in the order in which a layer calls them on a batch of requests:

  lora    w4_lora            low-rank adapters of many requests beside a shared projection
  rope    w4_qk_norm_rope    norms of the query and key heads and the position rotation, one pass;
          w4_qkv_paged       the same with keys and values stored to the pages of a cache
  paged   w4_attn_paged      attention of new tokens (one per request, or chunks) over a paged cache

`own = False` runs the plain forms: elementary torch operations in 32 bits (angles in 64),
rounded once at the end. `own = True` makes the calls that a user of the library makes.
"""
import numpy as np
import torch

own = False

# Most operations that exact() takes on (64-bit products run at about 1 TFLOP/s).
_EXACT_FLOPS = 4e12


def listed():
    return [
        # One request's token on a projection of 2048 x 1536: latency.
        {"name": "lora one", "op": "lora", "M": 1, "N": 2048, "K": 1536, "R": 16, "L": 4, "runs": False},
        # A decode batch, every request with an adapter of its own choice, the long up projection.
        {"name": "lora batch", "op": "lora", "M": 61, "N": 12288, "K": 1536, "R": 64, "L": 16, "runs": False},
        # Prompts of a few requests packed together: rows of one request lie together.
        {"name": "lora prompt", "op": "lora", "M": 4001, "N": 1536, "K": 6144, "R": 32, "L": 8, "runs": True},
        # One token on a full layer (head width 512), stored to its page: latency.
        {"name": "rope one", "op": "rope", "B": 1, "most_q": 1, "past": 5000, "Hq": 8, "Hkv": 1, "D": 512, "R": 512,
         "page": 64, "paged": True, "f32": True, "norm": True, "pairs": False},
        # A decode batch on grouped heads, part of each head rotated, neighbouring elements as pairs.
        {"name": "rope batch", "op": "rope", "B": 61, "most_q": 1, "past": 100000, "Hq": 12, "Hkv": 4, "D": 128, "R": 64,
         "page": 16, "paged": True, "f32": False, "norm": True, "pairs": True},
        # A prompt's queries and keys, far from the beginning.
        {"name": "rope prompt", "op": "rope", "B": 1, "most_q": 8001, "past": 120000, "Hq": 8, "Hkv": 1, "D": 256, "R": 256,
         "page": 0, "paged": False, "f32": True, "norm": True, "pairs": False},
        # Three requests' tokens on a sliding layer (head width 256, window 512): latency.
        {"name": "paged window", "op": "paged", "B": 3, "most_q": 1, "past": 1300, "Hq": 8, "Hkv": 1, "D": 256, "page": 64,
         "window": 512, "step": True},
        # A decode batch of requests of very different lengths, grouped heads, short pages.
        {"name": "paged batch", "op": "paged", "B": 61, "most_q": 1, "past": 16000, "Hq": 8, "Hkv": 2, "D": 128, "page": 16,
         "window": 0, "step": True},
        # One request at the largest context on a full layer (head width 512).
        {"name": "paged long", "op": "paged", "B": 1, "most_q": 1, "past": 130000, "Hq": 8, "Hkv": 1, "D": 512, "page": 128,
         "window": 0, "step": True},
        # Chunks of new tokens and single tokens of several requests packed together.
        {"name": "paged mixed", "op": "paged", "B": 7, "most_q": 1999, "past": 9000, "Hq": 12, "Hkv": 4, "D": 128, "page": 32,
         "window": 0, "step": False},
        # One chunk of a long prompt on a layer of head width 256.
        {"name": "paged chunk", "op": "paged", "B": 1, "most_q": 1024, "past": 60000, "Hq": 8, "Hkv": 1, "D": 256, "page": 64,
         "window": 0, "step": False},
    ]


def _log(rng, lo, hi):
    """A whole number spread over its logarithm."""
    return int(round(lo * (hi / lo) ** rng.random()))


_HEADS = [(8, 1), (8, 2), (4, 4), (12, 4), (6, 2), (7, 1), (16, 2)]


def draw(rng):
    op = rng.choice(["lora", "rope", "paged", "paged"])
    if op == "lora":
        c = {"op": op, "M": _log(rng, 1, 5000), "N": 8 * _log(rng, 8, 1536), "K": 32 * _log(rng, 4, 192),
             "R": 8 * _log(rng, 1, 16), "L": _log(rng, 1, 48), "runs": False}
        c["runs"] = c["M"] > 256 or rng.random() < 0.3
        while c["M"] * (c["N"] + c["K"]) > 30_000_000:
            c["M"] = c["M"] * 3 // 4
        return c
    if op == "rope":
        c = {"op": op, "B": _log(rng, 1, 64), "most_q": rng.choice([1, 1, _log(rng, 1, 4000)]), "past": _log(rng, 1, 130000),
             "Hq": 8, "Hkv": 1, "D": rng.choice([64, 128, 256, 384, 512]), "R": 2, "page": rng.choice([16, 32, 64, 128, 256]),
             "paged": rng.random() < 0.6, "f32": rng.random() < 0.6, "norm": rng.random() < 0.8, "pairs": rng.random() < 0.4}
        c["Hq"], c["Hkv"] = rng.choice(_HEADS)
        c["R"] = rng.choice([c["D"], c["D"], c["D"] // 2, c["D"] // 4])
        while c["B"] * c["most_q"] * (c["Hq"] + 2 * c["Hkv"]) * c["D"] > 18_000_000:
            c["most_q"] = max(1, c["most_q"] // 2)
            c["B"] = max(1, c["B"] * 3 // 4)
        if c["paged"]:
            while c["B"] * (c["past"] + c["most_q"]) * c["Hkv"] * c["D"] > 1 << 27:
                c["past"] = max(1, c["past"] // 2)
                c["B"] = max(1, c["B"] * 7 // 8)
        return c
    c = {"op": op, "B": _log(rng, 1, 64), "most_q": 1, "past": _log(rng, 1, 60000), "Hq": 8, "Hkv": 1,
         "D": rng.choice([64, 128, 256, 256, 384, 512]), "page": rng.choice([16, 16, 32, 64, 128, 256]),
         "window": rng.choice([0, 0, 512, _log(rng, 1, 4000)]), "step": rng.random() < 0.5}
    c["Hq"], c["Hkv"] = rng.choice(_HEADS)
    if not c["step"]:
        c["most_q"] = _log(rng, 1, 4000)
        c["B"] = min(c["B"], 12)
    while (_paged_dense(c) > 5e11 or c["B"] * (c["past"] + c["most_q"]) * c["Hkv"] * c["D"] > 1 << 27 or
           c["B"] * c["most_q"] * (c["past"] + c["most_q"]) * c["Hq"] > 1 << 30):
        c["most_q"] = max(1, c["most_q"] * 3 // 4)
        c["past"] = max(1, c["past"] * 3 // 4)
        c["B"] = max(1, c["B"] * 7 // 8)
    return c


# --------------------------------------------------------------------- inputs

def _lengths(c):
    """New tokens and lengths (with them) of a batch's requests. They belong to the case; the seed changes
    the values."""
    rng = np.random.default_rng([c["B"], c["most_q"], c["past"], c["D"]])
    B = c["B"]
    lq = np.maximum(1, np.round(c["most_q"] ** rng.random(B))).astype(np.int64)
    past = np.round(c["past"] * rng.random(B)).astype(np.int64)
    lq[0], past[0] = c["most_q"], c["past"]
    return lq, past + lq


def _paged_dense(c):
    """Operations of the plain form (it pads every request to the longest)."""
    return 4.0 * c["B"] * c["most_q"] * (c["past"] + c["most_q"]) * c["Hq"] * c["D"]


def _adapters(c):
    """The adapter of each row: any of them or none (-1) for a decode batch, runs of rows for prompts."""
    rng = np.random.default_rng([c["M"], c["L"], c["R"]])
    if not c["runs"]:
        ids = rng.integers(0, c["L"], c["M"])
        ids[rng.random(c["M"]) < 0.1] = -1
        ids[0] = 0
        return ids
    cuts = np.sort(rng.integers(0, c["M"], max(1, min(c["L"], 11)) - 1))
    return rng.integers(-1, c["L"], len(cuts) + 1)[np.searchsorted(cuts, np.arange(c["M"]), side="right")]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _bf16(g, *shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)


def _table(rng, lk, page):
    """Pages of each request, in no order within the pool (-1 past its last), and the pool's pages."""
    n = (lk + page - 1) // page
    table = np.full((len(lk), max(1, int(n.max()))), -1)
    pages = int(n.sum()) + 3
    order = rng.permutation(pages)
    first = np.concatenate([[0], np.cumsum(n)])
    for b in range(len(lk)):
        table[b, :n[b]] = order[first[b]:first[b + 1]]
    return table, pages


def prepare(case, seed):
    c = case
    rng = np.random.default_rng([seed, 23])
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": dict(c)}

    def dev(a, t=np.int32):
        return torch.from_numpy(np.ascontiguousarray(a, t)).cuda()

    if c["op"] == "lora":
        s["ids"] = dev(_adapters(c))
        s["y"] = _randn(g, c["M"], c["N"])
        s["x"] = _bf16(g, c["M"], c["K"])
        s["a"] = (_randn(g, c["L"], c["R"], c["K"]) * c["K"] ** -0.5).bfloat16()
        s["b"] = (_randn(g, c["L"], c["N"], c["R"]) * 0.05).bfloat16()
        s["scale"] = dev(0.5 + rng.random(c["L"]), np.float32)
        return s
    lq, lk = _lengths(c)
    s["lq"], s["lk"] = lq.tolist(), lk.tolist()
    s["cu_q"] = dev(np.concatenate([[0], np.cumsum(lq)]))
    s["lens"] = dev(lk)
    M, Hq, Hkv, D = int(lq.sum()), c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        y = _randn(g, M, (Hq + 2 * Hkv) * D) * 2.0
        y = y if c["f32"] else y.bfloat16()
        s["q"] = y[:, :Hq * D].view(M, Hq, D)
        s["k"] = y[:, Hq * D:(Hq + Hkv) * D].view(M, Hkv, D)
        s["v"] = y[:, (Hq + Hkv) * D:].view(M, Hkv, D)
        s["qw"] = 1.0 + 0.2 * _randn(g, D) if c["norm"] else None
        s["kw"] = 1.0 + 0.2 * _randn(g, D) if c["norm"] else None
        s["inv_freq"] = dev(1e6 ** (-np.arange(0, c["R"], 2) / c["R"]), np.float32)
        s["pos"] = dev(np.concatenate([np.arange(b - a, b) for a, b in zip(lq, lk)]))
        if not c["paged"]:
            return s
    else:
        s["q"] = _bf16(g, M, Hq, D)
        s["scale"] = D ** -0.5
    table, pages = _table(rng, lk, c["page"])
    s["table"] = dev(table)
    s["k_pages"] = _bf16(g, pages, c["page"], Hkv, D)
    s["v_pages"] = _bf16(g, pages, c["page"], Hkv, D)
    return s


# ---------------------------------------------------------------- plain forms

def _plain_lora(s):
    c = s["case"]
    L, R = c["L"], c["R"]
    h = (s["x"].float() @ s["a"].float().view(L * R, -1).T).view(-1, L, R)
    mine = s["ids"].long()[:, None] == torch.arange(L, device="cuda")
    h = torch.where(mine[:, :, None], h * s["scale"][None, :, None], torch.zeros_like(h))
    return s["y"] + h.view(-1, L * R) @ s["b"].float().transpose(1, 2).reshape(L * R, -1)


def _normed(x, w, eps=1e-6):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def _turned(x, cos, sin, pairs):
    h = cos.shape[-1]
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if pairs else (x[..., :h], x[..., h:2 * h])
    u, v = a * cos - b * sin, b * cos + a * sin
    u, v = (torch.stack([u, v], -1).flatten(-2), x[..., :0]) if pairs else (u, v)
    return torch.cat([u, v, x[..., 2 * h:]], -1).bfloat16()


def _plain_rope(s):
    c = s["case"]
    angle = s["pos"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _turned(_normed(s["q"], s["qw"]), cos, sin, c["pairs"])
    k = _turned(_normed(s["k"], s["kw"]), cos, sin, c["pairs"])
    if not c["paged"]:
        return {"q": q, "k": k}
    row = torch.arange(q.shape[0], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu_q"], row, right=True) - 1
    pos = s["pos"].long()
    at = s["table"].long()[seq, pos // c["page"]], pos % c["page"]
    s["k_pages"][at] = k
    s["v_pages"][at] = s["v"].bfloat16()
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_paged(s):
    c = s["case"]
    B, Hkv, G, D = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    n, T = c["most_q"], s["table"].shape[1] * c["page"]
    first, lq = s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    table = s["table"].long().clamp(min=0)
    i = torch.arange(n, device="cuda")
    t = torch.arange(T, device="cuda")
    pos = (s["lens"].long() - lq)[:, None] + i
    keep = (t <= pos[:, :, None]) & (i < lq[:, None])[:, :, None]
    if c["window"]:
        keep &= t > pos[:, :, None] - c["window"]
    k = s["k_pages"][table].view(B, T, Hkv, D).float().permute(0, 2, 3, 1)
    v = s["v_pages"][table].view(B, T, Hkv, D).float().permute(0, 2, 1, 3)
    rows = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[rows].view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    w = ((q @ k) * s["scale"]).view(B, Hkv, G, n, T).masked_fill(~keep[:, None, None], float("-inf"))
    m = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = w.sum(-1, keepdim=True)
    o = (w.view(B, Hkv, G * n, T) @ v).view(B, Hkv, G, n, D) / torch.where(l > 0, l, torch.ones_like(l))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, c["Hq"], D)
    return o[i < lq[:, None]].bfloat16()


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"lora": _plain_lora, "rope": _plain_rope, "paged": _plain_paged}[c["op"]](s)
    import bit_weight_only_w4a16_gb300 as w4
    if c["op"] == "lora":
        return w4.w4_lora(s["y"], s["x"], s["a"], s["b"], s["ids"], scale=s["scale"])
    cu_q = None if c["most_q"] == 1 else s["cu_q"]  # one token of each request
    if c["op"] == "paged":
        return w4.w4_attn_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], cu_q=cu_q, window=c["window"],
                                scale=s["scale"])
    if not c["paged"]:
        q, k = w4.w4_qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], q_weight=s["qw"], k_weight=s["kw"],
                                  pairs=c["pairs"])
        return {"q": q, "k": k}
    q = w4.w4_qkv_paged(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["inv_freq"], cu_q=cu_q,
                        q_weight=s["qw"], k_weight=s["kw"], pairs=c["pairs"])
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# ------------------------------------------------------------------- the work

def work(case):
    c = case
    if c["op"] == "lora":
        ids = _adapters(c)
        M, N, K, R = (float(c[x]) for x in "MNKR")
        rows = float((ids >= 0).sum())
        used = len(set(ids[ids >= 0].tolist()))
        return {"bytes": 8.0 * M * N + 2.0 * rows * K + 2.0 * used * R * (N + K) + 4.0 * M, "flops": 2.0 * rows * R * (N + K)}
    lq, lk = _lengths(c)
    rows = float(lq.sum())
    if c["op"] == "rope":
        heads = c["Hq"] + (2 if c["paged"] else 1) * c["Hkv"]
        return {"bytes": rows * heads * c["D"] * (6.0 if c["f32"] else 4.0), "flops": rows * heads * c["D"] * 8.0}
    pairs, keys = 0, 0
    for a, b in zip(lq.tolist(), lk.tolist()):
        p = np.arange(b - a, b, dtype=np.int64)
        lo = np.maximum(0, p - c["window"] + 1) if c["window"] else np.zeros_like(p)
        pairs += int((p + 1 - lo).sum())
        keys += int(b - lo[0])
    return {"bytes": 4.0 * rows * c["Hq"] * c["D"] + 4.0 * keys * c["Hkv"] * c["D"], "flops": 4.0 * pairs * c["Hq"] * c["D"]}


# -------------------------------------------------------------------- 64 bits

def exact(case, seed):
    c = case
    if work(c)["flops"] > _EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    if c["op"] == "lora":
        out = s["y"].double()
        ids = s["ids"].tolist()
        for i in sorted(set(ids) - {-1}):
            r = torch.tensor([m for m, j in enumerate(ids) if j == i], device="cuda")
            out[r] += float(s["scale"][i]) * ((s["x"][r].double() @ s["a"][i].double().T) @ s["b"][i].double().T)
        return out.cpu().numpy()
    if c["op"] == "rope":
        turn = s["pos"].double().cpu().numpy()[:, None] * s["inv_freq"].double().cpu().numpy()[None, :]
        z = torch.from_numpy(np.exp(1j * turn)).cuda()[:, None, :]
        h = c["R"] // 2
        done = {}
        for name, w in (("q", s["qw"]), ("k", s["kw"])):
            x = s[name].double()
            if w is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()
            first = torch.arange(h, device="cuda") * (2 if c["pairs"] else 1)
            second = first + (1 if c["pairs"] else h)
            y = torch.complex(x[..., first], x[..., second]) * z
            x = x.clone()
            x[..., first], x[..., second] = y.real, y.imag
            done[name] = x
        if not c["paged"]:
            return {n: x.cpu().numpy() for n, x in done.items()}
        k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
        m = 0
        for b, (a, n) in enumerate(zip(s["lq"], s["lk"])):
            p = torch.arange(n - a, n, device="cuda")
            pg = s["table"][b].long()[p // c["page"]]
            k_pages[pg, p % c["page"]] = done["k"][m:m + a]
            v_pages[pg, p % c["page"]] = s["v"][m:m + a].double()
            m += a
        return {"q": done["q"].cpu().numpy(), "k_pages": k_pages.cpu().numpy(), "v_pages": v_pages.cpu().numpy()}
    G, D = c["Hq"] // c["Hkv"], c["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    m = 0
    for b, (a, n) in enumerate(zip(s["lq"], s["lk"])):
        t = torch.arange(n, device="cuda")
        pg = s["table"][b].long()[t // c["page"]]
        k, v = (s[x][pg, t % c["page"]].double() for x in ("k_pages", "v_pages"))
        for i in range(0, a, 512):
            j = min(a, i + 512)
            p = torch.arange(n - a + i, n - a + j, device="cuda")[:, None]
            drop = t > p
            if c["window"]:
                drop |= t <= p - c["window"]
            for h in range(c["Hq"]):
                w = (s["q"][m + i:m + j, h].double() @ k[:, h // G].T) * s["scale"]
                out[m + i:m + j, h] = torch.softmax(w.masked_fill(drop, -np.inf), 1) @ v[:, h // G]
        m += a
    return out.cpu().numpy()
