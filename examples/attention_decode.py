"""Speculative decoding through attention layers with a paged key/value cache.

A small random-weight decoder (rotary grouped-query attention layers only; projections by
torch) answers a batch of prompts, each of them several times:

  prefill   tgdn_rope -> tgdn_prompt_attention, keys and values to pages layer by layer
            (tgdn_pages_reserve, tgdn_pages_append), then tgdn_pages_fork for the other answers
  step      tgdn_pages_reserve -> tgdn_tree_prep, per layer tgdn_rope (cached length + depth) ->
            tgdn_paged_tree_attention -> tgdn_accept -> tgdn_pages_append of the accepted paths
  end       tgdn_pages_free of the finished answers, tgdn_pages_compact

Draft trees hold the last token as the root, a chain of guesses and a wrong sibling beside each;
one-node trees make the same step plain token-by-token decoding, which is what draws the
guesses here.  Run it for the two step times and the tokens per step:

  python examples/attention_decode.py
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tree_speculative_decoding_gated_gb300 import tgdn  # noqa: E402

I32 = torch.int32


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Model:
    """Weights, one paged cache, and the two passes through the layers."""

    def __init__(self, layers=2, H_q=8, H_kv=2, d=64, vocab=512, seqs=8, n_pages=512, page_size=16,
                 max_pages=64, theta=10000.0, dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)
        wide = H_q * d
        new = lambda *s: (torch.randn(s, generator=g) / s[0] ** 0.5).to(dtype).cuda()  # noqa: E731
        self.H_q, self.H_kv, self.d, self.vocab, self.dtype = H_q, H_kv, d, vocab, dtype
        self.embed = new(vocab, wide) * vocab ** 0.5
        self.head = new(wide, vocab)
        self.w_qkv = [new(wide, (H_q + 2 * H_kv) * d) for _ in range(layers)]
        self.w_o = [new(wide, wide) for _ in range(layers)]
        self.freq, self.mscale = tgdn.rope_freqs(d, theta)
        self.freq = self.freq.cuda()
        self.scale = d ** -0.5
        self.pages = tgdn.Pages(seqs, n_pages, page_size, max_pages)
        self.pool = self.pages.pool(layers, H_kv, d, dtype)
        self.ws = tgdn.pages_workspace(self.pages)

    def norm(self, x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(self.dtype)

    def heads(self, qkv):
        return qkv.split([self.H_q, self.H_kv, self.H_kv], dim=1)

    def layer(self, l, x, attend, **position):
        """One layer: rotated q, k and v are views of the fused projection."""
        qkv = (self.norm(x) @ self.w_qkv[l]).view(x.shape[0], -1, self.d)
        q, k, v = self.heads(qkv)
        tgdn.rope(q, k, q, k, self.freq, mscale=self.mscale, **position)
        o = torch.empty((x.shape[0], self.H_q, self.d), dtype=self.dtype, device="cuda")
        attend(q, k, v, o)
        return x + o.view(x.shape[0], -1) @ self.w_o[l], k, v

    def logits(self, x):
        return self.norm(x) @ self.head

    def sound(self, status):
        """(Reads the device; a server would look at its words once per step or later.)"""
        if bool(status.any()):
            raise RuntimeError(f"status {status.tolist()}")

    def prefill(self, prompts):
        """Prompts into the cache's first rows (which hold nothing): the next token of each."""
        tokens = ints([t for p in prompts for t in p])
        cu = [0]
        for p in prompts + [[]] * (self.pages.B - len(prompts)):
            cu.append(cu[-1] + len(p))
        last, cu = [e - 1 for e in cu[1:len(prompts) + 1]], ints(cu)
        tgdn.pages_reserve(self.pages, cu[1:] - cu[:-1], self.ws)
        self.sound(self.pages.status)
        status = torch.empty(self.pages.B, dtype=I32, device="cuda")
        x = self.embed[tokens]
        for l in range(len(self.w_o)):
            x, k, v = self.layer(l, x, lambda q, k, v, o: tgdn.prompt_attention(
                cu, q, k, v, o, self.scale, status), cu=cu)
            self.sound(status)
            tgdn.pages_append(self.pages, cu, k, v, self.pool[l:l + 1],
                              advance=l == len(self.w_o) - 1)
            self.sound(self.pages.status)
        return self.logits(x[last]).argmax(-1).to(I32)

    def fork(self, src, dst):
        status = torch.empty(len(src), dtype=I32, device="cuda")
        tgdn.pages_fork(self.pages, ints(src), ints(dst), self.pool, status, self.ws)
        self.sound(status)

    def step(self, tree, tokens):
        """Verifies draft trees over the cache and appends the accepted paths.  Returns the
        accepted nodes' path [B][depth_max + 1], their number [B] and every node's logits."""
        tgdn.tree_prep(tree)
        tgdn.pages_reserve(self.pages, torch.full_like(self.pages.len, tree.depth_max + 1), self.ws)
        self.sound(self.pages.status)
        n = tgdn.paged_tree_attention_workspace_bytes(tree, self.pages, self.H_q, self.H_kv, self.d)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        x, kept = self.embed[tokens], []
        for l in range(len(self.w_o)):
            x, k, v = self.layer(l, x, lambda q, k, v, o: tgdn.paged_tree_attention(
                tree, self.pages, q, k, v, self.pool[l, 0], self.pool[l, 1], o, self.scale, ws),
                cu=tree.cu_nodes, base=self.pages.len, off=tree.depth)
            kept.append((k, v))
        logits = self.logits(x)
        # node n is accepted when its token is what the verifier answers at its parent
        wanted = logits.argmax(-1).to(I32)
        first = torch.repeat_interleave(tree.cu_nodes[:-1], tree.cu_nodes[1:] - tree.cu_nodes[:-1])
        target = wanted[(first + tree.parent.clamp(min=0)).long()]
        node = torch.empty(tree.B, dtype=I32, device="cuda")
        n_path = torch.empty_like(node)
        path = torch.empty((tree.B, tree.depth_max + 1), dtype=I32, device="cuda")
        tgdn.accept(tree, tokens, target, node, n_path, path)
        for l, (k, v) in enumerate(kept):
            tgdn.pages_append(self.pages, tree.cu_nodes, k, v, self.pool[l:l + 1], path=path,
                              n_path=n_path, advance=l == len(kept) - 1)
        self.sound(tree.status)
        self.sound(self.pages.status)
        return path, n_path, logits

    def finish(self, seqs):
        n_live = torch.empty(1, dtype=I32, device="cuda")
        tgdn.pages_free(self.pages, ints(seqs))
        tgdn.pages_compact(self.pages, self.pool, n_live, self.ws)
        return int(n_live)


def draft(model, roots, guesses, wrong):
    """A tree per sequence: the root, then for every guess the guess and a sibling beside it."""
    cu, parent, tokens = [0], [], []
    for root, chain in zip(roots, guesses):
        parent.append(-1)
        tokens.append(root)
        at = 0
        for t in chain:
            n = len(parent) - cu[-1]
            parent += [at, at]
            tokens += [t, (t + wrong) % model.vocab]
            at = n
        cu.append(len(parent))
    n_max = max(b - a for a, b in zip(cu[:-1], cu[1:]))
    depth = max(len(c) for c in guesses)
    return tgdn.Tree.from_host(cu, parent, n_max, depth), ints(tokens)


def decode(model, first, count, guess, wrong=1):
    """Greedy decoding until every sequence has `count` tokens.  guess(b, n): drafted tokens
    after the n tokens that sequence b has (n counts its root, which is not in the cache yet).
    Returns the tokens, the number of steps and the seconds they took."""
    got = [[t] for t in first.tolist()]
    torch.cuda.synchronize()
    began, steps = time.perf_counter(), 0
    while min(len(t) for t in got) < count:
        tree, tokens = draft(model, [t[-1] for t in got], [guess(b, len(t)) for b, t in enumerate(got)],
                             wrong)
        path, n_path, logits = model.step(tree, tokens)
        answer = logits.argmax(-1).tolist()
        cu, tokens = tree.cu_nodes.tolist(), tokens.tolist()
        for b, (p, n) in enumerate(zip(path.tolist(), n_path.tolist())):
            got[b] += [tokens[cu[b] + i] for i in p[1:n]] + [answer[cu[b] + p[n - 1]]]
        steps += 1
    return got, steps, time.perf_counter() - began


def run(lengths=(300, 37, 1, 170), answers=2, count=48, right=0.8, seed=1, **sizes):
    g = torch.Generator().manual_seed(seed)
    new = len(lengths)
    out = {}
    for name in ("token by token", "draft trees"):
        model = Model(seqs=new * answers, **sizes)
        g.manual_seed(seed)
        prompts = [torch.randint(model.vocab, (n,), generator=g).tolist() for n in lengths]
        first = model.prefill(prompts)
        for i in range(1, answers):
            model.fork(list(range(new)), list(range(i * new, (i + 1) * new)))
        first = first.repeat(answers)
        if name == "token by token":
            guess = lambda b, n: []  # noqa: E731
        else:  # the known answer, each token right with probability `right`
            known = out["token by token"]["tokens"]
            coin = torch.rand((new * answers, count + 16), generator=g)
            guess = lambda b, n: [t if coin[b, n + i] < right else (t + 7) % model.vocab  # noqa: E731
                                  for i, t in enumerate(known[b][n:n + 6])]
        tokens, steps, took = decode(model, first, count, guess)
        live = model.finish(list(range(1, new * answers)))
        out[name] = {"prompts": prompts, "tokens": tokens, "steps": steps, "seconds": took,
                     "live_pages": live, "model": model}
    return out


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--answers", type=int, default=4)
    ap.add_argument("--count", type=int, default=128)
    a = ap.parse_args()
    run(answers=1, count=4)  # (warm-up)
    out = run(answers=a.answers, count=a.count, layers=4, H_q=16, H_kv=4, d=128)
    for name, r in out.items():
        n = sum(len(t) - 1 for t in r["tokens"])
        print(f"{name}: {r['steps']} steps of {1e3 * r['seconds'] / r['steps']:.2f} ms, "
              f"{n / r['steps'] / len(r['tokens']):.2f} tokens per step and sequence, "
              f"{r['live_pages']} pages of the first answer left")


if __name__ == "__main__":
    main()
