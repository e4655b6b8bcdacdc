"""Decoding with drafted tokens: prompt read, tree attention, judging, commit.

A small one-stack model with 4-bit weights (random ones; the point is the path, not
the text) that alternates a sliding layer (a ring of slots, head width 256) and a
full layer (head width 512), one key/value head under eight query heads:

  prompt   w4_embed_gather -> per layer: w4a16_gemm, w4_attn_prompt, w4a16_gemm;
           the last positions of the keys and values go into the caches
  step     a tree of drafted tokens (its first node is the last accepted token)
           -> per layer: w4a16_gemm, w4_attn_tree, w4a16_gemm -> w4a16_gemm with the
           tied table -> w4_logprobs for the greedy picks and their log probabilities
  accept   walk from the first node to the child that carries the greedy pick, as
           long as there is one; w4_kv_commit stores the path for all layers of a kind

Every step accepts at least one token. The tokens are those of plain decoding (a
tree of one node), whatever was drafted:

  python examples/draft_step.py            # compares the two, prints tokens per step
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bit_weight_only_w4a16_gb300 as w4  # noqa: E402
import synth  # noqa: E402


def _weights(seed, n, k):
    q = torch.from_numpy(synth.gen_qweight(seed, n, k).view(np.int32)).cuda()
    s = torch.from_numpy(synth.gen_scales(seed, n, k).view(np.int16)).cuda()
    return q, s


class Layer:
    def __init__(self, seed, hidden, heads, width, window):
        self.heads, self.width, self.window = heads, width, window
        self.q = _weights(seed, heads * width, hidden)
        self.k = _weights(seed + 1, width, hidden)
        self.v = _weights(seed + 2, width, hidden)
        self.o = _weights(seed + 3, hidden, heads * width)


class Model:
    """Layers of two kinds; each kind has its caches [layers][1][slots][width]."""

    def __init__(self, pairs=2, hidden=512, vocab=2048, heads=8, ring=128, slots=1024, seed=5):
        self.hidden, self.vocab, self.ring, self.slots = hidden, vocab, ring, slots
        self.table = _weights(seed, vocab, hidden)
        self.layers = []
        for i in range(pairs):
            self.layers.append(Layer(seed + 10 * i + 1, hidden, heads, 256, ring))  # sliding
            self.layers.append(Layer(seed + 10 * i + 5, hidden, heads, 512, 0))     # full
        self.caches = {}
        for width, T in ((256, ring), (512, slots)):
            self.caches[width] = [torch.zeros(pairs, 1, T, width, dtype=torch.bfloat16, device="cuda")
                                  for _ in range(2)]
        self.kpos = torch.full((1, ring), -1, dtype=torch.int32, device="cuda")
        self.pos = torch.zeros(1, dtype=torch.int32, device="cuda")

    def project(self, x, w):
        return w4.w4a16_gemm(x, w[0], w[1])

    def norm(self, x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def embed(self, tokens):
        return w4.w4_embed_gather(tokens, *self.table).float() * 8.0

    def qkv(self, x, layer):
        n = x.shape[0]
        q = self.norm(self.project(x, layer.q).view(n, layer.heads, layer.width))
        k = self.norm(self.project(x, layer.k).view(n, 1, layer.width))
        return q, k, self.project(x, layer.v).view(n, 1, layer.width).bfloat16()

    def read_prompt(self, tokens):
        """The prompt's keys and values into the caches; tokens int32 [n], all but the
        last position (the first step's first node) are read."""
        n = tokens.numel() - 1
        self.pos.fill_(n)
        if n == 0:
            return
        h = self.embed(tokens[:n])
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        for i, layer in enumerate(self.layers):
            q, k, v = self.qkv(self.norm(h), layer)
            a = w4.w4_attn_prompt(q, k, v, cu, window=layer.window, scale=layer.width ** -0.5)
            h = h + 0.1 * self.project(a.view(n, -1), layer.o)
            kc, vc = (c[i // 2, 0] for c in self.caches[layer.width])
            if layer.window:
                p = torch.arange(max(0, n - self.ring), n, device="cuda")
                kc[p % self.ring], vc[p % self.ring] = k[p, 0], v[p, 0]
                self.kpos[0, p % self.ring] = p.int()
            else:
                kc[:n], vc[:n] = k[:, 0], v[:, 0]

    def step(self, tokens, parents):
        """Logits [N][vocab] of a tree of tokens at the current position, and the
        nodes' keys and values by head width."""
        N = tokens.numel()
        h = self.embed(tokens)
        new = {w: ([], []) for w in self.caches}
        for i, layer in enumerate(self.layers):
            q, k, v = self.qkv(self.norm(h), layer)
            kc, vc = (c[i // 2].unsqueeze(2) for c in self.caches[layer.width])
            a = w4.w4_attn_tree(q[None], kc, vc, k[None], v[None], parents, self.pos,
                                kpos=self.kpos if layer.window else None, window=layer.window,
                                scale=layer.width ** -0.5)
            h = h + 0.1 * self.project(a.view(N, -1), layer.o)
            new[layer.width][0].append(k[:, 0])
            new[layer.width][1].append(v[:, 0])
        return self.project(self.norm(h), self.table), new

    def commit(self, new, path, count):
        for width, (kc, vc) in self.caches.items():
            k, v = (torch.stack(x).unsqueeze(1) for x in new[width])
            w4.w4_kv_commit(kc, vc, k, v, path, count, self.pos, kpos=self.kpos if width == 256 else None)
        self.pos += count


def decode(model, prompt, n, draft):
    """n tokens after the prompt, with trees from draft(history) -> (tokens, parents)
    (the first node is the history's last token). Returns the tokens and the number of
    steps, with the log probability of each accepted token."""
    history, logps, steps = prompt.tolist(), [], 0
    model.read_prompt(prompt)
    end = len(history) + n
    while len(history) < end:
        tokens, parents = draft(history)
        N = len(tokens)
        dev = torch.tensor(tokens, dtype=torch.int32, device="cuda")
        par = torch.tensor([parents], dtype=torch.int32, device="cuda")
        logits, new = model.step(dev, par)
        _, _, top_lp, top = w4.w4_logprobs(logits, topk=1)
        pick, lp = top[:, 0].tolist(), top_lp[:, 0].tolist()
        node, path = 0, [0]
        while True:
            history.append(pick[node])
            logps.append(lp[node])
            child = [c for c in range(node + 1, N) if parents[c] == node and tokens[c] == pick[node]]
            if not child:
                break
            node = child[0]
            path.append(node)
        count = torch.tensor([len(path)], dtype=torch.int32, device="cuda")
        full = torch.full((1, N), -1, dtype=torch.int32)
        full[0, :len(path)] = torch.tensor(path, dtype=torch.int32)
        model.commit(new, full.cuda(), count)
        steps += 1
    return history[len(prompt):end], logps[:n], steps


def no_draft(history):
    return [history[-1]], [-1]


class TruthDraft:
    """Drafts from a known continuation, with wrong guesses beside and after it: what a
    good draft model would give, without one."""

    def __init__(self, start, truth, vocab, depth=4, seed=0):
        self.start, self.truth, self.vocab, self.depth = start, truth, vocab, depth
        self.rng = np.random.default_rng(seed)

    def __call__(self, history):
        at = len(history) - self.start
        tokens, parents, last = [history[-1]], [-1], 0
        for d in range(self.depth):
            wrong = int(self.rng.integers(self.vocab))
            right = self.truth[at + d] if at + d < len(self.truth) and self.rng.random() < 0.8 else wrong
            tokens += [wrong, right]
            parents += [last, last]
            last = len(tokens) - 1
        return tokens, parents


def main(prompt_len=300, n=48):
    w4.init()
    prompt = torch.from_numpy(synth.gen_ids(3, prompt_len, 2048)).cuda()
    plain, lp, steps = decode(Model(), prompt, n, no_draft)
    drafted, lp2, steps2 = decode(Model(), prompt, n, TruthDraft(prompt_len, plain, 2048))
    same = plain == drafted
    print(f"{n} tokens: {steps} steps plain, {steps2} steps drafted ({n / steps2:.2f} tokens a step), "
          f"same tokens: {same}, largest difference of a log probability "
          f"{max(abs(a - b) for a, b in zip(lp, lp2)):.4f}")
    return same, steps, steps2


if __name__ == "__main__":
    sys.exit(0 if main()[0] else 1)
