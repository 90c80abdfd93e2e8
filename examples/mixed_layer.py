"""A recurrent layer with two kinds of memory, made of this library's operators.

    y = x + Wo group_norm(o) silu(z),   o = (delta rule(q, k, v), linear recurrence(u)),
    q, k, v, u = silu(conv(Wi n)),   z = Wz n,   n = norm(x)

The delta rule's queries and keys are turned by their positions; the linear recurrence keeps one state a channel, with
a decay of its own; each head of either is normalised by itself and gated.  The same parameters
serve three ways:

  train_row(x, lengths)   a row that packs sequences of the given lengths, with gradients
  prefill(x, lengths)     the same without gradients, returning the cache each sequence leaves
  decode(x, cache, ...)   one new token a sequence, the cache advanced in place

Run on a GPU, `python examples/mixed_layer.py` trains a few steps on random data and shows that a
prompt continued token by token gives what the whole sequence gives at once.
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import causal_depthwise_conv1d_amd as ccv  # noqa: E402


class MixedLayer(torch.nn.Module):
    def __init__(self, width=256, key_heads=2, heads=4, head_dim=64, turned=32, linear_heads=2, taps=4, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.hk, self.hv, self.d, self.groups = key_heads, heads, head_dim, heads + linear_heads
        self.split = [key_heads * head_dim, key_heads * head_dim, heads * head_dim, linear_heads * head_dim]
        channels, inner = sum(self.split), self.groups * head_dim
        new = lambda *s: torch.nn.Parameter(torch.randn(*s, device=device, dtype=torch.float32).to(dtype) * s[-1] ** -0.5)  # noqa: E731
        one = lambda n: torch.nn.Parameter(torch.ones(n, device=device))  # noqa: E731
        zero = lambda n: torch.nn.Parameter(torch.zeros(n, device=device))  # noqa: E731
        self.norm_w, self.norm_b = one(width), zero(width)
        self.w_in, self.w_z, self.w_beta = new(channels, width), new(inner, width), new(heads, width)
        self.w_gate, self.w_rate = new(heads, width), new(self.split[3], width)
        self.conv_w = torch.nn.Parameter((torch.randn(channels, taps, device=device) * 0.5).to(dtype))
        self.decay = torch.nn.Parameter(torch.linspace(0.05, 0.5, heads, device=device))
        self.rate = torch.nn.Parameter(torch.linspace(0.01, 0.5, self.split[3], device=device))
        self.out_w, self.out_b = one(inner), zero(inner)
        self.w_out = new(width, inner)
        self.freq, self.scale = ccv.rotary_frequencies(turned, device=device)

    def _project(self, x):
        """The conv's input, the gate, both recurrences' log decays and the write strengths."""
        n = ccv.layer_norm_fn(x, self.norm_w, self.norm_b)
        g = -self.decay * F.softplus(F.linear(n, self.w_gate).float())
        a = -self.rate * F.softplus(F.linear(n, self.w_rate).float())
        return F.linear(n, self.w_in), F.linear(n, self.w_z), g, a, torch.sigmoid(F.linear(n, self.w_beta))

    def _heads(self, c, positions):
        """The conv's output [..., channels] in its parts; queries and keys at unit length and turned."""
        q, k, v, u = c.split(self.split, -1)
        q, k = (F.normalize(t.unflatten(-1, (self.hk, self.d)).float(), dim=-1).to(c.dtype) for t in (q, k))
        q, k = ccv.rotary_fn(q, k, positions, self.freq, scale=self.scale)
        return q, k, v.unflatten(-1, (self.hv, self.d)), u

    def _output(self, x, o, h, z):
        y = ccv.group_norm_fn(torch.cat([o.flatten(-2), h], -1), self.groups, self.out_w, self.out_b, gate=z, activation="silu")
        return x + F.linear(y, self.w_out)

    def _row(self, x, lengths, states):
        cu, seq_idx, positions = ccv.sequence_tables(lengths, x.shape[1])
        c, z, g, a, beta = self._project(x)
        conv = ccv.causal_conv1d_fn(c.transpose(1, 2), self.conv_w, seq_idx=seq_idx, activation="silu").transpose(1, 2)
        q, k, v, u = self._heads(conv, positions.view(1, -1))
        o = ccv.gated_delta_rule_fn(q, k, v, g, beta, cu_seqlens=cu, return_final_state=states)
        h = ccv.gated_linear_recurrence_fn(u, a, cu_seqlens=cu, return_final_state=states, normalize=True)
        o, s = o if states else (o, None)
        h, t = h if states else (h, None)
        return self._output(x, o, h, z), c, cu, s, t

    def train_row(self, x, lengths):
        """x [1, T, width], lengths int32 [N] on the GPU -> [1, T, width]; differentiable."""
        return self._row(x, lengths, False)[0]

    @torch.no_grad()
    def prefill(self, x, lengths):
        """-> (y [1, T, width], cache of every sequence: the conv's last inputs, both states, the next position)."""
        y, c, cu, state, linear = self._row(x, lengths, True)
        back = torch.arange(1 - self.conv_w.shape[1], 0, device=x.device)         # the last taps - 1 inputs
        at = cu[1:, None] + back
        last = torch.where((at >= cu[:-1, None])[..., None], c[0][at.clamp(min=0)], 0)
        return y, {"conv": last.transpose(1, 2).contiguous(), "state": state, "linear": linear, "next": cu[1:] - cu[:-1]}

    @torch.no_grad()
    def decode(self, x, cache, slots=None):
        """x [N, width], one token a sequence -> [N, width].  slots int32 [N]: the states' places
        in larger caches (the conv's history and the positions go with the sequences)."""
        c, z, g, a, beta = self._project(x)
        q, k, v, u = self._heads(ccv.causal_conv1d_update(c, cache["conv"], self.conv_w, activation="silu"), cache["next"])
        o = ccv.gated_delta_rule_update(q, k, v, g, beta, cache["state"], state_indices=slots)
        h = ccv.gated_linear_recurrence_update(u, a, cache["linear"], state_indices=slots, normalize=True)
        cache["next"] += 1
        return self._output(x, o, h, z)


def main():
    torch.manual_seed(0)
    layer, width = MixedLayer(), 256
    lengths = [300, 1, 0, 211]
    x = torch.randn(1, 520, width, device="cuda").bfloat16()
    target = torch.randn_like(x)
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    opt = torch.optim.AdamW(layer.parameters(), lr=3e-3)
    for step in range(5):
        loss = (layer.train_row(x, ln) - target).float().square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        print(f"step {step}: loss {loss.item():.4f}")
    whole, _ = layer.prefill(x, ln)
    ends = [300, 301, 301, 512]
    live = [i for i, n in enumerate(lengths) if n > 0]
    short = torch.tensor([max(n - 1, 0) for n in lengths], dtype=torch.int32, device="cuda")
    rows = torch.cat([x[:, e - n:e - 1] for e, n in zip(ends, lengths) if n > 0], 1)
    _, cache = layer.prefill(rows, short)
    y = layer.decode(torch.stack([x[0, ends[i] - 1] for i in range(len(lengths))]), cache)
    err = max(float((y[i] - whole[0, ends[i] - 1]).float().abs().max()) for i in live)
    print(f"last tokens by decoding and by prefill differ by at most {err:.4f}")


if __name__ == "__main__":
    main()
