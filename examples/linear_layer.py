"""A linear attention layer on the library's operators: prompts, single tokens
and a training step.

    x --W_in--> q, k, v --norm and rotation of q, k--> linear attention with a
    decay for each head --W_out--> y

q, k and v stay slices of one projection; nothing is copied between the
operators.  Run it on a GPU:  python examples/linear_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_delta_rule_49_gb300 import binding  # noqa: E402


class LinearAttention:
    def __init__(self, dim=512, heads=8, key_heads=4, key_width=64, value_width=128,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        self.H, self.Hq, self.K, self.V = heads, key_heads, key_width, value_width
        self.sizes = [key_heads * key_width, key_heads * key_width, heads * value_width]
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, m):
            return (torch.randn(n, m, generator=g, device=device) * m ** -0.5).to(dtype)

        self.w_in = weight(sum(self.sizes), dim)
        self.w_out = weight(dim, heads * value_width)
        self.wq = torch.ones(key_width, device=device)
        self.wk = torch.ones(key_width, device=device)
        # horizons from 8 tokens to 8 thousand
        self.alpha = 1 - 2.0 ** -torch.linspace(3, 13, heads, device=device)
        half = torch.arange(0, key_width, 2, device=device, dtype=torch.float32)
        self.inv_freq = 10000.0 ** (-half / key_width)
        self.scale = key_width ** -0.5

    def _project(self, x):
        q, k, v = (x @ self.w_in.T).split(self.sizes, -1)
        return (q.unflatten(-1, (self.Hq, self.K)), k.unflatten(-1, (self.Hq, self.K)),
                v.unflatten(-1, (self.H, self.V)))

    def prompt(self, x, pos, state=None):
        """x [B, T, dim], pos [B, T] -> (y [B, T, dim], state)."""
        q, k, v = self._project(x)
        q, k = binding.qk_norm_rotate(q, k, pos, self.inv_freq, self.wq, self.wk)
        o, state = binding.linear_prefill(q, k, v, self.alpha, S0=state, scale=self.scale)
        return o.flatten(-2) @ self.w_out.T, state

    def step(self, x, pos, state):
        """One token a sequence: x [B, dim], pos [B]; state is updated in place."""
        q, k, v = self._project(x)
        q, k = binding.qk_norm_rotate(q, k, pos, self.inv_freq, self.wq, self.wk)
        o = binding.linear_decode_step(q, k, v.contiguous(), self.alpha, state, scale=self.scale)
        return o.flatten(-2) @ self.w_out.T

    def gradients(self, x, pos, dy):
        """Gradients of sum(y dy) for a prompt from an empty state: of x and of
        the weights, by name."""
        q, k, v = self._project(x)
        nq, nk = binding.qk_norm_rotate(q, k, pos, self.inv_freq, self.wq, self.wk)
        o, _ = binding.linear_prefill(nq, nk, v, self.alpha, scale=self.scale, want_state=False)
        o, dy = o.flatten(-2), dy.flatten(0, 1)
        do = (dy @ self.w_out).view(v.shape)
        dnq, dnk, dv, _ = binding.linear_backward(nq, nk, v, self.alpha, do, scale=self.scale)
        dq, dk, dwq, dwk = binding.qk_norm_rotate_backward(q, k, pos, self.inv_freq, dnq, dnk,
                                                           self.wq, self.wk)
        d_in = torch.cat([g.flatten(-2) for g in (dq, dk, dv)], -1).flatten(0, 1)
        return {"x": (d_in @ self.w_in).view(x.shape), "w_in": d_in.T @ x.flatten(0, 1),
                "w_out": dy.T @ o.flatten(0, 1), "wq": dwq, "wk": dwk}


def main():
    layer = LinearAttention()
    B, T, new = 2, 300, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(B, T + new, 512, generator=g, device="cuda").bfloat16()
    pos = torch.arange(T + new, device="cuda").repeat(B, 1)
    whole, _ = layer.prompt(x, pos)
    y, state = layer.prompt(x[:, :T].contiguous(), pos[:, :T].contiguous())
    for t in range(T, T + new):
        y = layer.step(x[:, t].contiguous(), pos[:, t].contiguous(), state)
        off = (y - whole[:, t]).float().norm() / whole[:, t].float().norm()
        print(f"token {t}: step against the whole prompt, relative difference {off:.1e}")
    dy = torch.randn(whole.shape, generator=g, device="cuda").bfloat16()
    for name, d in layer.gradients(x, pos, dy).items():
        print(f"gradient of {name}: shape {tuple(d.shape)}, norm {d.float().norm():.3e}")
    assert binding.gdn_get_last_device_status() == binding.GDN_OK


if __name__ == "__main__":
    main()
