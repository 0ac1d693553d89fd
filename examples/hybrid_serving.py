"""A hybrid stack that serves prompts and tokens: KDA layers with a full-attention layer among them.

    python examples/hybrid_serving.py [--layers kkka] [--prompts 37,5,120] [--steps 4] [--drafts 3] [--piece 0] [--rotary]

Every letter of ``--layers`` is a layer: ``k`` a KDA layer (its fp32 state per sequence and head), ``a`` a
causal softmax-attention layer with grouped heads (its keys and values in a paged 8-bit cache), with rotary positions
where asked for.  The prompts arrive packed, whole or in pieces that attend to the cache; then every sequence advances token by token, and at the end a window of
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
    layers' keys and values in ``kv_heads`` heads.  ``rotary``: do the attention layers know their tokens' positions?"""

    D, PAGE = 128, 64

    def __init__(self, layers, width=512, heads=8, kv_heads=2, device="cuda", seed=0, rotary=False):
        self.rotary = kda.make_rotary(self.D) if rotary else None
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

    def _remember(self, q, k, v, memory, lengths, cu=None):
        """The tokens' keys and values into the cache, and their queries (if any), both turned where the layers have positions."""
        if self.rotary is None:
            kda.kda_cache_append(k, v, memory, self.table, lengths, cu_seqlens=cu)
            return q
        return kda.kda_rotary_append(self.rotary, k, v, memory, self.table, lengths, q=q, cu_seqlens=cu)

    def _add(self, x, o, w):
        return x + o.flatten(1) @ w["out"]

    def prompt(self, x, lens):
        """The packed prompts x [sum(lens), width]; returns the stack's output for every token.  The attention layers'
        prompts attend to their own tokens alone, so that with such layers they must be the sequences' first (then: more())."""
        if self.begun and "a" in self.layers:
            raise ValueError("the sequences hold tokens that a prompt's attention layers would not see: start() anew, more() or step()")
        self.begun = True
        cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).to(self.device)
        self.lengths += cu[1:] - cu[:-1]
        for i, (kind, w) in enumerate(zip(self.layers, self.w)):
            if kind == "k":
                o, _ = kda.kda_forward(*self._kda_inputs(x, w), initial_state=self.memory[i], final_state=self.memory[i],
                                       cu_seqlens=cu, max_seqlen=max(lens))
            else:
                q, k, v = self._attention_inputs(x, w)
                # (turned keys are rounded once on their way into the cache, as more() and step() have it, so that a prompt's
                # codes are those of its pieces)
                turned = (q, k) if self.rotary is None else kda.kda_rotary(self.rotary, q, k, cu_seqlens=cu)
                o = kda.kda_attention_prefill(*turned, v, cu_seqlens=cu)
                self._remember(None, k, v, self.memory[i], self.lengths, cu)
            x = self._add(x, o, w)
        return x

    def more(self, x, lens):
        """The next pieces of the prompts, packed as in prompt(), of any length each (0: nothing new): the attention
        layers' tokens attend to what the caches hold."""
        self.begun = True
        cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).to(self.device)
        self.lengths += cu[1:] - cu[:-1]
        for i, (kind, w) in enumerate(zip(self.layers, self.w)):
            if kind == "k":
                o, _ = kda.kda_forward(*self._kda_inputs(x, w), initial_state=self.memory[i], final_state=self.memory[i],
                                       cu_seqlens=cu, max_seqlen=max(lens))
            else:
                q = self._remember(*self._attention_inputs(x, w), self.memory[i], self.lengths, cu)
                o = kda.kda_attention_extend(q, self.memory[i], self.table, self.lengths, cu_seqlens=cu)
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
                q = self._remember(*self._attention_inputs(x, w), self.memory[i], self.lengths)
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
                q = self._remember(*self._attention_inputs(x, w), self.memory[i], ahead)
                o = kda.kda_attention_decode(q, self.memory[i], self.table, ahead)
            x = self._add(x, o, w)
        return x


def demo(layers="kkka", prompts=(37, 5, 120), steps=4, drafts=3, width=512, seed=0, piece=0, rotary=False):
    """Serves the prompts (``piece`` > 0: at most so many tokens of each at a time), then ``steps`` tokens each, then verifies ``drafts`` more; returns the outputs of the
    tokens after the prompts and what the same tokens give when they arrive as part of the prompts."""
    n = len(prompts)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    total = [p + steps + drafts for p in prompts]
    x = [torch.randn(t, width, generator=g, device="cuda").bfloat16() for t in total]
    served = HybridStack(layers, width, seed=seed, rotary=rotary)
    served.start(total)
    if piece <= 0:
        served.prompt(torch.cat([x[i][:prompts[i]] for i in range(n)]), prompts)
    else:
        for at in range(0, max(prompts), piece):
            ends = [min(p, at + piece) for p in prompts]
            served.more(torch.cat([x[i][at:ends[i]] for i in range(n)]), [max(e - at, 0) for e in ends])
    out = [served.step(torch.stack([x[i][prompts[i] + s] for i in range(n)])) for s in range(steps)]
    out = torch.stack(out, 1)
    window = served.verify(torch.cat([x[i][prompts[i] + steps:] for i in range(n)])).view(n, drafts, width)
    whole = HybridStack(layers, width, seed=seed, rotary=rotary)
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
    ap.add_argument("--piece", type=int, default=0, help="tokens of every prompt that are served at a time (0: all)")
    ap.add_argument("--rotary", action="store_true", help="rotary positions in the attention layers")
    a = ap.parse_args()
    got, want = demo(a.layers, tuple(int(p) for p in a.prompts.split(",")), a.steps, a.drafts,
                     piece=a.piece, rotary=a.rotary)
    err = (got.float() - want.float()).norm() / want.float().norm()
    print(f"{a.layers}: {got.shape[0]} sequences, {a.steps} tokens and {a.drafts} drafts each; "
          f"served one by one against served as a prompt: relative difference {err:.4f}")


if __name__ == "__main__":
    main()
