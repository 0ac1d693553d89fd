"""A hybrid stack that serves prompts and tokens: KDA layers with a full-attention layer among them.

    python examples/hybrid_serving.py [--layers kkka] [--prompts 37,5,120] [--steps 4] [--drafts 3]

Every letter of ``--layers`` is a layer: ``k`` a KDA layer (its fp32 state per sequence and head), ``a`` a
causal softmax-attention layer with grouped heads (its keys and values in a paged 8-bit cache).  The
prompts arrive packed; then every sequence advances token by token, and at the end a window of
drafted tokens is verified without touching the states.  Weights are random: the example shows how the
calls fit together, and checks that tokens served one at a time agree with the same tokens served as a
prompt.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_attention_recurrence_kda_gb300 import binding as kda  # noqa: E402


class HybridStack:
    """``layers`` (a string of k and a) over ``width`` channels; ``heads`` heads of 128 channels, the attention
    layers' keys and values in ``kv_heads`` heads."""

    D, PAGE = 128, 64

    def __init__(self, layers, width=512, heads=8, kv_heads=2, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.layers, self.heads, self.kv_heads, self.device = layers, heads, kv_heads, device
        r = lambda *s: torch.randn(*s, generator=g, device=device)
        self.w = []
        for kind in layers:
            cols = (4 * heads * self.D + heads) if kind == "k" else (heads + 2 * kv_heads) * self.D
            self.w.append({"in": (r(width, cols) / width ** 0.5).bfloat16(),
                           "out": (r(heads * self.D, width) / (heads * self.D) ** 0.5).bfloat16(),
                           "A": (0.5 * r(heads)).contiguous()})

    def start(self, capacity):
        """States and caches for sequences of at most ``capacity`` tokens (a list)."""
        n = len(capacity)
        need = [-(-c // self.PAGE) for c in capacity]
        table = torch.full((n, max(need)), -1, dtype=torch.int32)  # past a sequence's capacity there is no page
        at = 0
        for i, m in enumerate(need):
            table[i, :m] = torch.arange(at, at + m)
            at += m
        self.begun = False  # do the sequences hold tokens?
        self.table = table.to(self.device)
        self.lengths = torch.zeros(n, dtype=torch.int32, device=self.device)
        self.memory = [torch.zeros(n, self.heads, self.D, self.D, device=self.device) if kind == "k" else
                       kda.kda_cache_alloc(at, self.PAGE, self.kv_heads, self.D, device=self.device)
                       for kind in self.layers]

    def _kda_inputs(self, x, w):
        h, d = self.heads, self.D
        y = x @ w["in"]
        q, k, v, z = (y[:, i * h * d:(i + 1) * h * d].reshape(-1, h, d) for i in range(4))
        unit = lambda t: (t.float() / torch.sqrt((t.float() ** 2).sum(-1, keepdim=True) + 1e-6)).to(t.dtype)
        return unit(q), unit(k), v.contiguous(), z.contiguous(), w["A"], torch.sigmoid(y[:, 4 * h * d:].float()).contiguous()

    def _attention_inputs(self, x, w):
        """Views of one projection: nothing is copied."""
        y = (x @ w["in"]).view(-1, self.heads + 2 * self.kv_heads, self.D)
        return y[:, :self.heads], y[:, self.heads:self.heads + self.kv_heads], y[:, self.heads + self.kv_heads:]

    def _add(self, x, o, w):
        return x + o.reshape(o.shape[0], -1) @ w["out"]

    def prompt(self, x, lens):
        """The packed prompts x [sum(lens), width]; returns the stack's output for every token.  The attention layers'
        prompts attend to their own tokens alone, so that with such layers they must be the sequences' first."""
        if self.begun and "a" in self.layers:
            raise ValueError("the sequences hold tokens that a prompt's attention layers would not see: start() anew, or step()")
        self.begun = True
        cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).to(self.device)
        self.lengths += cu[1:] - cu[:-1]
        for i, (kind, w) in enumerate(zip(self.layers, self.w)):
            if kind == "k":
                o, _ = kda.kda_forward(*self._kda_inputs(x, w), initial_state=self.memory[i], final_state=self.memory[i],
                                       cu_seqlens=cu, max_seqlen=max(lens))
            else:
                q, k, v = self._attention_inputs(x, w)
                o = kda.kda_attention_prefill(q, k, v, cu_seqlens=cu)
                kda.kda_cache_append(k, v, self.memory[i], self.table, self.lengths, cu_seqlens=cu)
            x = self._add(x, o, w)
        return x

    def step(self, x):
        """One token of every sequence, x [n, width]."""
        self.begun = True
        self.lengths += 1
        for i, (kind, w) in enumerate(zip(self.layers, self.w)):
            if kind == "k":
                o = kda.kda_decode_step(*self._kda_inputs(x, w), self.memory[i])
            else:
                q, k, v = self._attention_inputs(x, w)
                kda.kda_cache_append(k, v, self.memory[i], self.table, self.lengths)
                o = kda.kda_attention_decode(q, self.memory[i], self.table, self.lengths)
            x = self._add(x, o, w)
        return x

    def verify(self, x):
        """A window of drafted tokens, x [n * drafts, width]: their outputs.  The KDA states stay as they are;
        the drafts' keys and values lie past ``lengths`` in the caches, where the next tokens replace them."""
        ahead = self.lengths + x.shape[0] // self.lengths.numel()
        for i, (kind, w) in enumerate(zip(self.layers, self.w)):
            if kind == "k":
                o, _ = kda.kda_decode_replay(*self._kda_inputs(x, w), self.memory[i], want_state=False)
            else:
                q, k, v = self._attention_inputs(x, w)
                kda.kda_cache_append(k, v, self.memory[i], self.table, ahead)
                o = kda.kda_attention_decode(q, self.memory[i], self.table, ahead)
            x = self._add(x, o, w)
        return x


def demo(layers="kkka", prompts=(37, 5, 120), steps=4, drafts=3, width=512, seed=0):
    """Serves the prompts, then ``steps`` tokens each, then verifies ``drafts`` more; returns the outputs of the
    tokens after the prompts and what the same tokens give when they arrive as part of the prompts."""
    n = len(prompts)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    total = [p + steps + drafts for p in prompts]
    x = [torch.randn(t, width, generator=g, device="cuda").bfloat16() for t in total]
    served = HybridStack(layers, width, seed=seed)
    served.start(total)
    served.prompt(torch.cat([x[i][:prompts[i]] for i in range(n)]), prompts)
    out = [served.step(torch.stack([x[i][prompts[i] + s] for i in range(n)])) for s in range(steps)]
    out = torch.stack(out, 1)
    window = served.verify(torch.cat([x[i][prompts[i] + steps:] for i in range(n)])).view(n, drafts, width)
    whole = HybridStack(layers, width, seed=seed)
    whole.start(total)
    y = whole.prompt(torch.cat(x), total)
    ends = torch.tensor(total).cumsum(0)
    want = torch.stack([y[e - steps - drafts:e] for e in ends.tolist()])
    return torch.cat([out, window], 1), want


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", default="kkka")
    ap.add_argument("--prompts", default="37,5,120")
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--drafts", type=int, default=3)
    a = ap.parse_args()
    got, want = demo(a.layers, tuple(int(p) for p in a.prompts.split(",")), a.steps, a.drafts)
    err = (got.float() - want.float()).norm() / want.float().norm()
    print(f"{a.layers}: {got.shape[0]} sequences, {a.steps} tokens and {a.drafts} drafts each; "
          f"served one by one against served as a prompt: relative difference {err:.4f}")


if __name__ == "__main__":
    main()
