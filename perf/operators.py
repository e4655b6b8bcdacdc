"""Cases of the prompt and draft operators, their plain forms and their values in 64 bits.

Four operators, as a step with drafted tokens uses them:

  prompt    w4_attn_prompt   causal attention over whole prompts or chunks of them, packed
  tree      w4_attn_tree     attention of a tree of drafted tokens over a cache and the tree itself
  logprobs  w4_logprobs      log probabilities of given tokens, entropy, top alternatives
  commit    w4_kv_commit     the accepted path's key and value rows into the caches

`own = False` runs the plain forms: elementary torch operations in 32 bits, rounded once at the
end. `own = True` makes the calls that a user of the library makes.
"""
import numpy as np
import torch

own = False

# Most operations that exact() takes on (64-bit products run at about 1 TFLOP/s).
_EXACT_FLOPS = 8e12


def listed():
    return [
        # A short prompt on a sliding layer (head width 256, window 512): latency.
        {"name": "prompt short", "op": "prompt", "B": 1, "most_q": 61, "past": 0, "Hq": 8, "Hkv": 1, "D": 256,
         "window": 512, "ragged": False},
        # Nine prompts of very different lengths packed together, grouped heads.
        {"name": "prompt packed", "op": "prompt", "B": 9, "most_q": 4001, "past": 0, "Hq": 12, "Hkv": 4, "D": 128,
         "window": 0, "ragged": True},
        # One 256-token chunk of a long prompt on a full layer (head width 512).
        {"name": "prompt chunk", "op": "prompt", "B": 1, "most_q": 256, "past": 130000, "Hq": 8, "Hkv": 1, "D": 512,
         "window": 0, "ragged": False},
        # A whole prompt at once, eight query heads on one key/value head.
        {"name": "prompt whole", "op": "prompt", "B": 1, "most_q": 16384, "past": 0, "Hq": 8, "Hkv": 1, "D": 256,
         "window": 0, "ragged": False},
        # Eight drafted tokens on a sliding layer's ring of 512 slots: latency.
        {"name": "tree ring", "op": "tree", "B": 1, "N": 8, "T": 512, "pos": 1300, "Hq": 8, "Hkv": 1, "D": 256,
         "window": 512, "ring": True},
        # Sixteen drafted tokens on a full layer at the largest context.
        {"name": "tree long", "op": "tree", "B": 1, "N": 16, "T": 131072, "pos": 130001, "Hq": 8, "Hkv": 1, "D": 512,
         "window": 0, "ring": False},
        # Several sequences at once, each with its own length, a wide tree.
        {"name": "tree batch", "op": "tree", "B": 4, "N": 61, "T": 32768, "pos": 32000, "Hq": 8, "Hkv": 2, "D": 128,
         "window": 0, "ring": False},
        # One drafted token judged after the vocabulary projection.
        {"name": "logprobs one", "op": "logprobs", "M": 1, "V": 262144, "k": 20, "masked": False},
        # A tree of drafted tokens, a constrained decoder's mask on the logits.
        {"name": "logprobs tree", "op": "logprobs", "M": 16, "V": 262144, "k": 20, "masked": True},
        # A 256-token chunk of a prompt scored, an odd vocabulary.
        {"name": "logprobs chunk", "op": "logprobs", "M": 256, "V": 256003, "k": 5, "masked": False},
        # Four accepted tokens into the rings of 28 sliding layers.
        {"name": "commit rings", "op": "commit", "L": 28, "B": 1, "N": 8, "T": 512, "W": 256, "pos": 1300, "ring": True},
        # Accepted paths of 8 sequences into full caches of 7 layers.
        {"name": "commit full", "op": "commit", "L": 7, "B": 8, "N": 61, "T": 4096, "W": 512, "pos": 4000, "ring": False},
    ]


def _log(rng, lo, hi):
    """A whole number spread over its logarithm."""
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "logprobs", "commit"])
    if op == "prompt":
        c = {"op": op, "B": _log(rng, 1, 12), "most_q": 1, "past": rng.choice([0, 0, _log(rng, 1, 60000)]), "Hq": 8,
             "Hkv": 1, "D": rng.choice([64, 128, 256, 256, 384, 512]), "window": rng.choice([0, 0, 512, _log(rng, 1, 4000)]),
             "ragged": True}
        c["Hq"], c["Hkv"] = rng.choice([(8, 1), (8, 2), (4, 4), (12, 4), (6, 2), (7, 1)])
        c["most_q"] = _log(rng, 1, 8000)
        while _prompt_dense(c) > 8e11:
            c["most_q"] = max(1, c["most_q"] * 3 // 4)
            c["past"] = c["past"] * 3 // 4
        return c
    if op == "tree":
        ring = rng.random() < 0.4
        c = {"op": op, "B": _log(rng, 1, 6), "N": _log(rng, 1, 64), "T": 512, "pos": 1, "Hq": 8, "Hkv": 1,
             "D": rng.choice([64, 128, 256, 256, 384, 512]), "window": 0, "ring": ring}
        c["Hq"], c["Hkv"] = rng.choice([(8, 1), (8, 2), (4, 4), (12, 4), (7, 1)])
        if ring:
            c["T"] = c["window"] = rng.choice([512, _log(rng, 16, 2048)])
            c["pos"] = _log(rng, 1, 5000)
        else:
            c["T"] = _log(rng, 64, 131072)
            c["window"] = rng.choice([0, 0, _log(rng, 1, 4000)])
            while c["B"] * c["T"] * c["Hkv"] * c["D"] > 1 << 26 or c["B"] * c["N"] * c["Hq"] * c["T"] > 1 << 26:
                c["T"] = c["T"] * 3 // 4
            c["pos"] = max(1, min(c["T"], _log(rng, 1, c["T"])))
        return c
    if op == "logprobs":
        V = _log(rng, 1000, 262144)
        return {"op": op, "M": max(1, min(_log(rng, 1, 256), 60_000_000 // V)), "V": V, "k": rng.randint(0, 20),
                "masked": rng.random() < 0.3}
    ring = rng.random() < 0.5
    T = 512 if ring else _log(rng, 100, 4096)
    return {"op": op, "L": rng.randint(1, 28), "B": rng.randint(1, 4), "N": _log(rng, 1, 64), "T": T,
            "W": rng.choice([128, 256, 512, 1024]), "pos": _log(rng, 1, 5000) if ring else rng.randint(0, max(0, T - 64)),
            "ring": ring}


# --------------------------------------------------------------------- inputs

def _lengths(c, rng):
    """Query and key lengths of a packed prompt's sequences."""
    B, q = c["B"], c["most_q"]
    if not c["ragged"]:
        lq = np.full(B, q, np.int64)
    else:
        lq = np.maximum(1, np.round(q ** rng.random(B))).astype(np.int64)
        lq[0] = q
    past = np.full(B, c["past"], np.int64)
    if c["ragged"] and c["past"]:
        past = rng.integers(0, c["past"] + 1, B)
        past[0] = c["past"]
    return lq, lq + past


def _prompt_dense(c):
    """Operations of the plain form at most (it forms every score of the packed batch)."""
    q, k = c["B"] * c["most_q"], c["B"] * (c["most_q"] + c["past"])
    return 4.0 * q * k * c["Hq"] * c["D"]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    c = case
    rng = np.random.default_rng([seed, 17])
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": dict(c)}

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()

    if c["op"] == "prompt":
        # A batch's lengths belong to the case; the seed changes the values.
        lq, lk = _lengths(c, np.random.default_rng([c["B"], c["most_q"], c["past"]]))
        s["lq"], s["lk"] = lq.tolist(), lk.tolist()
        s["cu_q"] = dev(np.concatenate([[0], np.cumsum(lq)]))
        s["cu_k"] = dev(np.concatenate([[0], np.cumsum(lk)]))
        s["q"] = _randn(g, int(lq.sum()), c["Hq"], c["D"]).bfloat16()
        s["k"] = _randn(g, int(lk.sum()), c["Hkv"], c["D"]).bfloat16()
        s["v"] = _randn(g, int(lk.sum()), c["Hkv"], c["D"]).bfloat16()
        s["scale"] = c["D"] ** -0.5
        return s
    if c["op"] == "tree":
        B, N, T = c["B"], c["N"], c["T"]
        s["q"] = _randn(g, B, N, c["Hq"], c["D"]).bfloat16()
        s["k"] = torch.empty(B, T, c["Hkv"], c["D"], dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        s["v"] = torch.empty(B, T, c["Hkv"], c["D"], dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        s["kt"] = _randn(g, B, N, c["Hkv"], c["D"]).bfloat16()
        s["vt"] = _randn(g, B, N, c["Hkv"], c["D"]).bfloat16()
        parents = np.stack([_tree(rng, N) for _ in range(B)])
        pos = np.maximum(1, c["pos"] - np.arange(B) * (c["pos"] // (2 * B)))
        s["parents"], s["pos"], s["kpos"] = dev(parents), dev(pos), None
        if c["ring"]:
            last = pos[:, None] - 1
            p = last - (last - np.arange(T)[None, :]) % T
            s["kpos"] = dev(np.where(p >= 0, p, -1))
        s["scale"] = c["D"] ** -0.5
        return s
    if c["op"] == "logprobs":
        x = _randn(g, c["M"], c["V"]) * 3.0
        if c["masked"]:  # a constrained decoder leaves every 64th token and the first ones
            keep = torch.zeros(c["V"], dtype=torch.bool, device="cuda")
            keep[::64] = True
            keep[:8] = True
            x[::2].masked_fill_(~keep, float("-inf"))
        s["logits"] = x
        s["targets"] = dev(rng.integers(0, c["V"], c["M"]) // 64 * 64)
        return s
    L, B, N, T, W = c["L"], c["B"], c["N"], c["T"], c["W"]
    for name, n in (("kc", T), ("vc", T), ("kt", N), ("vt", N)):
        s[name] = torch.empty(L, B, n, W, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    pos = np.full(B, c["pos"]) - (0 if c["ring"] else np.arange(B) % max(1, c["pos"]))
    count = rng.integers(1, min(N, 8) + 1, B)
    path = np.full((B, N), -1)
    for b in range(B):
        path[b, :count[b]] = np.sort(rng.choice(N, count[b], replace=False))
    s["pos"], s["count"], s["path"], s["kpos"] = dev(pos), dev(count), dev(path), None
    if c["ring"]:
        last = pos[:, None] - 1
        p = last - (last - np.arange(T)[None, :]) % T
        s["kpos"] = dev(np.where(p >= 0, p, -1))
    return s


def _tree(rng, N):
    """Parents of a drafted tree in order of its levels: three children at most, parents before children."""
    p = np.full(N, -1)
    used = np.zeros(N, int)
    first = 0
    for i in range(1, N):
        open_ = np.arange(first, i)[used[first:i] < 3]
        p[i] = open_[min(len(open_) - 1, rng.geometric(0.4) - 1)]
        used[p[i]] += 1
        while used[first] >= 3:
            first += 1
    return p


# ---------------------------------------------------------------- plain forms

def _softmax_rows(scores, keep):
    """exp(scores - max) and its sums over the kept entries; a row with none has sum 0."""
    scores = scores.masked_fill(~keep, float("-inf"))
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return p, p.sum(-1, keepdim=True)


def _plain_prompt(s):
    c = s["case"]
    G, D = c["Hq"] // c["Hkv"], c["D"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    iq = torch.arange(q.shape[0], device=q.device, dtype=torch.int32)
    ik = torch.arange(k.shape[0], device=q.device, dtype=torch.int32)
    sq = torch.searchsorted(s["cu_q"], iq, right=True) - 1
    sk = torch.searchsorted(s["cu_k"], ik, right=True) - 1
    pq = iq - s["cu_q"][sq + 1] + (s["cu_k"][sq + 1] - s["cu_k"][sq])
    pk = ik - s["cu_k"][sk]
    keep = (sq[:, None] == sk[None, :]) & (pk[None, :] <= pq[:, None])
    if c["window"]:
        keep &= pk[None, :] > pq[:, None] - c["window"]
    qh = q.view(-1, c["Hkv"], G, D).permute(1, 2, 0, 3).reshape(c["Hkv"], -1, D)
    scores = (qh @ k.permute(1, 2, 0)) * s["scale"]
    p, l = _softmax_rows(scores, keep.repeat(G, 1))
    o = (p @ v.permute(1, 0, 2)) / torch.where(l > 0, l, torch.ones_like(l))
    return o.view(c["Hkv"], G, -1, D).permute(2, 0, 1, 3).reshape(-1, c["Hq"], D).bfloat16()


def _plain_tree(s):
    c = s["case"]
    B, N, T, G, D = c["B"], c["N"], c["T"], c["Hq"] // c["Hkv"], c["D"]
    # Ancestors or self: powers of the parent relation.
    par = s["parents"].long()
    step = (par[:, :, None] == torch.arange(N, device=par.device)).float()
    anc = torch.linalg.matrix_power(torch.eye(N, device=par.device) + step, 64) > 0
    depth = anc.sum(-1) - 1
    pos = s["pos"].long()
    qpos = pos[:, None] + depth
    slot = torch.arange(T, device=par.device).expand(B, T) if s["kpos"] is None else s["kpos"].long()
    keep_c = ((slot >= 0) & (slot < pos[:, None]))[:, None, :].expand(B, N, T)
    keep_t = anc
    if c["window"]:
        keep_c = keep_c & (slot[:, None, :] > qpos[:, :, None] - c["window"])
        keep_t = keep_t & (qpos[:, None, :] > qpos[:, :, None] - c["window"])
    keep = torch.cat([keep_c, keep_t], -1)[:, None, :, None, :]
    keep = keep.expand(B, c["Hkv"], N, G, T + N).reshape(B, c["Hkv"], N * G, T + N)
    q = s["q"].float().view(B, N, c["Hkv"], G, D).permute(0, 2, 1, 3, 4).reshape(B, c["Hkv"], N * G, D)
    k = torch.cat([s["k"], s["kt"]], 1).float().permute(0, 2, 3, 1)
    v = torch.cat([s["v"], s["vt"]], 1).float().permute(0, 2, 1, 3)
    p, l = _softmax_rows((q @ k) * s["scale"], keep)
    o = (p @ v) / torch.where(l > 0, l, torch.ones_like(l))
    return o.view(B, c["Hkv"], N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, c["Hq"], D).bfloat16()


def _plain_logprobs(s):
    x, k = s["logits"], s["case"]["k"]
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    z = e.sum(-1, keepdim=True)
    u = (e * torch.where(torch.isinf(d), torch.zeros_like(d), d)).sum(-1, keepdim=True)
    lse = m + torch.log(z)
    lp = torch.gather(x, 1, s["targets"].long()[:, None]) - lse
    top, ids = torch.sort(x, dim=-1, descending=True, stable=True)  # equal values keep their order
    return {"logprob": lp[:, 0], "entropy": (torch.log(z) - u / z)[:, 0], "top_logprob": top[:, :k] - lse,
            "top_id": ids[:, :k].int()}


def _plain_commit(s):
    c = s["case"]
    j = torch.arange(c["N"], device="cuda")
    b, j = torch.nonzero(j[None, :] < s["count"][:, None], as_tuple=True)
    node = s["path"][b, j].long()
    p = s["pos"][b].long() + j
    slot = p % c["T"]
    s["kc"][:, b, slot] = s["kt"][:, b, node]
    s["vc"][:, b, slot] = s["vt"][:, b, node]
    if s["kpos"] is not None:
        s["kpos"][b, slot] = p.int()
    return _committed(s)


def _committed(s):
    r = {"k": s["kc"], "v": s["vc"]}
    if s["kpos"] is not None:
        r["kpos"] = s["kpos"]
    return r


_PLAIN = {"prompt": _plain_prompt, "tree": _plain_tree, "logprobs": _plain_logprobs, "commit": _plain_commit}


def run(state):
    s, c = state, state["case"]
    if not own:
        return _PLAIN[c["op"]](s)
    import bit_weight_only_w4a16_gb300 as w4
    if c["op"] == "prompt":
        return w4.w4_attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], window=c["window"], scale=s["scale"])
    if c["op"] == "tree":
        return w4.w4_attn_tree(s["q"], s["k"], s["v"], s["kt"], s["vt"], s["parents"], s["pos"], kpos=s["kpos"],
                               window=c["window"], scale=s["scale"])
    if c["op"] == "logprobs":
        lp, ent, top, ids = w4.w4_logprobs(s["logits"], s["targets"], topk=c["k"])
        return {"logprob": lp, "entropy": ent, "top_logprob": top, "top_id": ids}
    w4.w4_kv_commit(s["kc"], s["vc"], s["kt"], s["vt"], s["path"], s["count"], s["pos"], kpos=s["kpos"])
    return _committed(s)


# ------------------------------------------------------------------- the work

def _kept_pairs(lq, lk, window):
    """Kept (query, key) pairs of one sequence, and its keys that any query reads."""
    p = np.arange(lk - lq, lk, dtype=np.int64)
    lo = np.maximum(0, p - window + 1) if window else np.zeros_like(p)
    n = np.maximum(0, p + 1 - lo)
    return int(n.sum()), int(lk - (lo[0] if len(lo) else lk))


def _tree_lengths(c):
    pos = np.maximum(1, c["pos"] - np.arange(c["B"]) * (c["pos"] // (2 * c["B"])))
    n = np.minimum(pos, c["T"])
    if c["window"]:
        n = np.minimum(n, c["window"] - 1)
    return n


def work(case):
    c = case
    if c["op"] == "prompt":
        lq, lk = _lengths(c, np.random.default_rng([c["B"], c["most_q"], c["past"]]))
        pairs = [_kept_pairs(int(a), int(b), c["window"]) for a, b in zip(lq, lk)]
        return {"bytes": 4.0 * int(lq.sum()) * c["Hq"] * c["D"] + 4.0 * sum(k for _, k in pairs) * c["Hkv"] * c["D"],
                "flops": 4.0 * sum(p for p, _ in pairs) * c["Hq"] * c["D"]}
    if c["op"] == "tree":
        n = float(_tree_lengths(c).sum())
        rows = c["B"] * c["N"]
        return {"bytes": 4.0 * (n + rows) * c["Hkv"] * c["D"] + 4.0 * rows * c["Hq"] * c["D"],
                "flops": 4.0 * c["N"] * n * c["Hq"] * c["D"]}
    if c["op"] == "logprobs":
        return {"bytes": 4.0 * c["M"] * c["V"] + c["M"] * (12.0 + 8.0 * c["k"]), "flops": 6.0 * c["M"] * c["V"]}
    rows = 2.0 * c["L"] * c["B"] * min(c["N"], 8) * 0.56  # half of the longest path and one, on average
    return {"bytes": 4.0 * rows * c["W"], "flops": 0.0}


# -------------------------------------------------------------------- 64 bits

def _attend(q, k, v, keep, scale):
    """One sequence and head in 64 bits: rows of q over the kept rows of k and v."""
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for a in range(0, q.shape[0], 512):
        w = (q[a:a + 512].double() @ k.double().T) * scale
        kp = keep(a, min(a + 512, q.shape[0]))
        w[~kp] = -np.inf
        any_ = kp.any(1)
        out[a:a + 512][any_] = torch.softmax(w[any_], 1) @ v.double()
    return out


def exact(case, seed):
    c = case
    if c["op"] in ("prompt", "tree") and work(c)["flops"] * (2 if c["op"] == "prompt" else 1) > _EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    if c["op"] == "prompt":
        G = c["Hq"] // c["Hkv"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        a = b = 0
        for lq, lk in zip(s["lq"], s["lk"]):
            pk = torch.arange(lk, device="cuda")

            def keep(i, j, lq=lq, lk=lk, pk=pk):
                pq = torch.arange(i, j, device="cuda")[:, None] + lk - lq
                kp = pk[None, :] <= pq
                return kp & (pk[None, :] > pq - c["window"]) if c["window"] else kp

            for h in range(c["Hq"]):
                out[a:a + lq, h] = _attend(s["q"][a:a + lq, h], s["k"][b:b + lk, h // G], s["v"][b:b + lk, h // G],
                                           keep, s["scale"])
            a, b = a + lq, b + lk
        return out.cpu().numpy()
    if c["op"] == "tree":
        B, N, T, G = c["B"], c["N"], c["T"], c["Hq"] // c["Hkv"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b in range(B):
            par, pos = s["parents"][b].tolist(), int(s["pos"][b])
            kp = np.zeros((N, T + N), bool)
            slot = np.arange(T) if s["kpos"] is None else s["kpos"][b].cpu().numpy()
            for i in range(N):
                chain = [i]
                while par[chain[-1]] >= 0:
                    chain.append(par[chain[-1]])
                at = pos + len(chain) - 1
                low = at - c["window"] if c["window"] else -1
                kp[i, :T] = (slot >= 0) & (slot < pos) & (slot > low)
                for d, j in enumerate(chain):
                    kp[i, T + j] = at - d > low
            kp = torch.from_numpy(kp).cuda()
            for h in range(c["Hq"]):
                k = torch.cat([s["k"][b, :, h // G], s["kt"][b, :, h // G]])
                v = torch.cat([s["v"][b, :, h // G], s["vt"][b, :, h // G]])
                out[b, :, h] = _attend(s["q"][b, :, h], k, v, lambda i, j: kp[i:j], s["scale"])
        return out.cpu().numpy()
    if c["op"] == "logprobs":
        lp, ent, top = [], [], []
        for i in range(c["M"]):
            x = s["logits"][i].double().cpu().numpy()
            f = x[np.isfinite(x)]
            m = f.max()
            lse = m + np.log(np.exp(f - m).sum())
            p = np.exp(f - lse)
            lp.append(x[int(s["targets"][i])] - lse)
            ent.append(-(p * (f - lse)).sum())
            top.append(np.sort(x)[::-1][:c["k"]] - lse)
        return {"logprob": np.array(lp), "entropy": np.array(ent), "top_logprob": np.array(top).reshape(c["M"], -1),
                "top_id": None}
    return None
