"""A recurrent layer of a language model, made of this library's operators.

    y = x + Wo norm(o),   o = gated delta rule(q, k, v),   q, k, v = silu(conv(Wi norm(x)))

with log decays and write strengths from two more projections.  The same parameters serve
three ways, as a model uses them:

  train(x, lengths)      a row that packs sequences of the given lengths, with gradients
  prefill(x, lengths)    the same without gradients, returning the cache each sequence leaves
  decode(x, cache, ...)  one new token a sequence, the cache advanced in place

Run on a GPU, `python examples/delta_layer.py` trains a few steps on random data and shows
that a prompt continued token by token gives what the whole sequence gives at once.
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import causal_depthwise_conv1d_amd as ccv  # noqa: E402


class DeltaLayer(torch.nn.Module):
    def __init__(self, width=256, key_heads=2, heads=4, key_dim=64, value_dim=64, taps=4, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.hk, self.hv, self.dk, self.dv = key_heads, heads, key_dim, value_dim
        self.split = [key_heads * key_dim, key_heads * key_dim, heads * value_dim]
        channels = sum(self.split)
        new = lambda *s: torch.nn.Parameter(torch.randn(*s, device=device, dtype=torch.float32).to(dtype) * s[-1] ** -0.5)  # noqa: E731
        one = lambda n: torch.nn.Parameter(torch.ones(n, device=device))  # noqa: E731
        zero = lambda n: torch.nn.Parameter(torch.zeros(n, device=device))  # noqa: E731
        self.norm_w, self.norm_b = one(width), zero(width)
        self.w_in, self.w_gate, self.w_beta = new(channels, width), new(heads, width), new(heads, width)
        self.conv_w = torch.nn.Parameter((torch.randn(channels, taps, device=device) * 0.5).to(dtype))
        self.decay = torch.nn.Parameter(torch.linspace(0.05, 0.5, heads, device=device))
        self.out_w, self.out_b = one(value_dim), zero(value_dim)
        self.w_out = new(width, heads * value_dim)

    def _project(self, x):
        """The conv's input, the log decays and the write strengths."""
        n = ccv.layer_norm_fn(x, self.norm_w, self.norm_b)
        g = -self.decay * F.softplus(F.linear(n, self.w_gate).float())
        return F.linear(n, self.w_in), g, torch.sigmoid(F.linear(n, self.w_beta))

    def _heads(self, c):
        """Views of the conv's output [..., channels]; queries and keys scaled to unit length."""
        q, k, v = c.split(self.split, -1)
        q, k = (F.normalize(t.unflatten(-1, (self.hk, self.dk)).float(), dim=-1).to(c.dtype) for t in (q, k))
        return q, k, v.unflatten(-1, (self.hv, self.dv))

    def _output(self, x, o):
        return x + F.linear(ccv.layer_norm_fn(o, self.out_w, self.out_b).flatten(-2), self.w_out)

    def _row(self, x, lengths, states):
        cu, seq_idx, _ = ccv.sequence_tables(lengths, x.shape[1])
        c, g, beta = self._project(x)
        conv = ccv.causal_conv1d_fn(c.transpose(1, 2), self.conv_w, seq_idx=seq_idx, activation="silu").transpose(1, 2)
        q, k, v = self._heads(conv)
        o = ccv.gated_delta_rule_fn(q, k, v, g, beta, cu_seqlens=cu, return_final_state=states)
        o, s = o if states else (o, None)
        return self._output(x, o), c, cu, s

    def train_row(self, x, lengths):
        """x [1, T, width], lengths int32 [N] on the GPU -> [1, T, width]; differentiable."""
        return self._row(x, lengths, False)[0]

    @torch.no_grad()
    def prefill(self, x, lengths):
        """-> (y [1, T, width], cache of every sequence: the conv's last inputs and the states)."""
        y, c, cu, states = self._row(x, lengths, True)
        back = torch.arange(1 - self.conv_w.shape[1], 0, device=x.device)         # the last taps - 1 inputs
        at = cu[1:, None] + back
        last = torch.where((at >= cu[:-1, None])[..., None], c[0][at.clamp(min=0)], 0)
        return y, {"conv": last.transpose(1, 2).contiguous(), "state": states}

    @torch.no_grad()
    def decode(self, x, cache, slots=None):
        """x [N, width], one token a sequence -> [N, width].  slots int32 [N]: the states' places
        in a larger cache (the conv's history goes with the sequences)."""
        c, g, beta = self._project(x)
        q, k, v = self._heads(ccv.causal_conv1d_update(c, cache["conv"], self.conv_w, activation="silu"))
        return self._output(x, ccv.gated_delta_rule_update(q, k, v, g, beta, cache["state"], state_indices=slots))


def main():
    torch.manual_seed(0)
    layer, width = DeltaLayer(), 256
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
