"""One token-tree verify step of a small decoder over an 8-bit paged cache.

A decoder of random weights scores drafted trees: per layer a fused projection, rotary
positions (specdec_rope), attention of the tree's nodes over the cached tokens and their
ancestors (specdec_attend), a projection and a gated feed-forward block; its logits go to
specdec_verify_tree, and the accepted nodes' keys and values are appended to each layer's
cache (specdec_kv_append).  Prompts are written through the same calls, as chains.

    python examples/verify_with_cache.py [--steps 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_verification_64_gb300 import binding as sd  # noqa: E402


class Decoder:
    """Random weights in bfloat16; the dense products are torch's."""

    def __init__(self, layers=2, hidden=512, Hq=8, Hkv=2, D=64, V=1000, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(*shape):
            w = torch.randn(shape, generator=g, device=device) * shape[0] ** -0.5
            return w.to(torch.bfloat16)

        self.Hq, self.Hkv, self.D, self.V = Hq, Hkv, D, V
        self.embed = weight(V, hidden) * V ** 0.5
        self.layers = [dict(qkv=weight(hidden, (Hq + 2 * Hkv) * D), out=weight(Hq * D, hidden),
                            up=weight(hidden, 4 * hidden), down=weight(2 * hidden, hidden))
                       for _ in range(layers)]
        self.head = weight(hidden, V) * 4
        self.freq = sd.rope_frequencies(D, device=device)

    @staticmethod
    def norm(x):
        y = x.float()
        return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def forward(self, tokens, caches, parent=None, softcap=30.0):
        """tokens int64 [B, N] -> logits [B, N, V] and each layer's new (k, v)."""
        B, N = tokens.shape
        x, new = self.embed[tokens], []
        for w, cache in zip(self.layers, caches):
            qkv = (self.norm(x) @ w["qkv"]).view(B, N, self.Hq + 2 * self.Hkv, self.D)
            q, k, v = qkv.split((self.Hq, self.Hkv, self.Hkv), 2)
            q, k = sd.rope(q, k, self.freq, base=cache.length, parent=parent)
            a = sd.attend(q, k, v, cache, parent=parent, softcap=softcap)
            x = x + a.out.view(B, N, -1) @ w["out"]
            gate, up = (self.norm(x) @ w["up"]).chunk(2, -1)
            x = x + (torch.nn.functional.silu(gate) * up) @ w["down"]
            new.append((k, v))
        return (self.norm(x) @ self.head), new


def make_caches(model, B, tokens, block=16, device="cuda"):
    """A cache of `tokens` tokens a request for every layer, blocks handed out in a mixed order."""
    per = -(-tokens // block)
    caches = []
    for _ in model.layers:
        c = sd.KVCache.empty(B, per, B * per, block, model.Hkv, model.D, device)
        ids = torch.arange(B * per, dtype=torch.int32, device=device).view(per, B).t()
        c.block_table.copy_(ids)
        caches.append(c)
    return caches


def append(caches, new, **how):
    for cache, (k, v) in zip(caches, new):
        cache.length = sd.kv_append(k, v, cache, **how).length


def run(steps=4, B=3, prompt=37, V=1000, seed=0, trace=None):
    """Generates with drafted trees; returns the emitted tokens of each request."""
    device = "cuda"
    model = Decoder(V=V, seed=seed, device=device)
    g = torch.Generator(device=device)
    g.manual_seed(seed + 1)
    # every step: the last token (node 0), two candidates for the next, two for each of those
    parent = torch.tensor([[-1, 0, 0, 1, 1, 2, 2]], dtype=torch.int32, device=device).repeat(B, 1)
    N, depth = parent.shape[1], 2
    caches = make_caches(model, B, prompt + steps * (depth + 1) + 1)
    tokens = torch.randint(0, V, (B, prompt), generator=g, device=device)
    # the prompt but its last token goes into the caches; the last one is the first root
    _, new = model.forward(tokens[:, :-1], caches)
    append(caches, new)
    last = tokens[:, -1].int()
    temperature = torch.full((B,), 0.8, device=device)
    emitted = [[] for _ in range(B)]
    for _ in range(steps):
        # a uniform draft: q is flat, and the candidates are drawn from it
        q = torch.full((B, N, V), 1.0 / V, device=device, dtype=torch.bfloat16)
        nodes = torch.randint(0, V, (B, N), generator=g, device=device).int()
        nodes[:, 0] = last
        logits, new = model.forward(nodes.long(), caches, parent)
        uniforms = torch.rand((B, N), generator=g, device=device).clamp(1e-6, 1 - 1e-6)
        r = sd.verify_tree(logits.contiguous(), q, nodes, parent, temperature, uniforms, depth)
        append(caches, new, count=r.n_accepted, extra=1, path=r.path_nodes)
        if trace is not None:
            trace.append((logits, r, [c.length.clone() for c in caches]))
        last = r.final_token
        for b in range(B):
            emitted[b] += r.out_tokens[b, :int(r.n_accepted[b]) + 1].tolist()
    return emitted


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    for b, tokens in enumerate(run(a.steps)):
        print(f"request {b}: {tokens}")


if __name__ == "__main__":
    main()
