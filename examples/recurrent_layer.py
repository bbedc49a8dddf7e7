"""A residual block on the library's operators: prompts, single tokens and a
training step.

    s = x + residual;  n = layer norm of s
    v, g = two halves of one projection of n
    h = gated linear recurrence of v under the gates g
    y = a projection of h, for the next block beside s

v and g stay slices of the projection; nothing is copied between the operators.
Run it on a GPU:  python examples/recurrent_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_delta_rule_49_gb300 import binding  # noqa: E402


class RecurrentBlock:
    def __init__(self, dim=512, width=1024, dtype=torch.bfloat16, device="cuda", seed=0):
        self.width = width
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, m):
            return (torch.randn(n, m, generator=g, device=device) * m ** -0.5).to(dtype)

        self.w_in = weight(2 * width, dim)
        self.w_out = weight(dim, width)
        self.norm_w = torch.ones(dim, device=device)
        self.norm_b = torch.zeros(dim, device=device)
        # gates that forget within a few tokens and within hundreds
        self.b_gate = torch.linspace(0, 6, width, device=device).to(dtype)

    def _inputs(self, n):
        p = n @ self.w_in.T
        p[..., self.width:] += self.b_gate
        return p[..., :self.width], p[..., self.width:]

    def prompt(self, x, residual, state=None):
        """x, residual [B, T, dim], state [B, width] -> (y, s, state)."""
        n, s, _ = binding.layer_norm(x, self.norm_w, self.norm_b, residual=residual)
        h, state, _ = binding.scan_prefill(*self._inputs(n), h0=state)
        return h @ self.w_out.T, s, state

    def packed(self, x, residual, offsets, state=None):
        """x, residual [tokens, dim] of the sequences that offsets [B + 1] cut."""
        n, s, _ = binding.layer_norm(x, self.norm_w, self.norm_b, residual=residual)
        h, state, _ = binding.scan_prefill(*self._inputs(n), h0=state, offsets=offsets)
        return h @ self.w_out.T, s, state

    def step(self, x, residual, state):
        """One token a sequence: x, residual [B, dim]; state is updated in place."""
        n, s, _ = binding.layer_norm(x, self.norm_w, self.norm_b, residual=residual)
        return binding.scan_decode_step(*self._inputs(n), state) @ self.w_out.T, s

    def gradients(self, x, residual, dy, ds):
        """Gradients of sum(y dy) + sum(s ds) for a prompt from an empty state: of x (the
        residual's are the same) and of the weights, by name."""
        n, s, stats = binding.layer_norm(x, self.norm_w, self.norm_b, residual=residual,
                                         want_stats=True)
        v, g = self._inputs(n)
        h, _, states = binding.scan_prefill(v, g, want_state=False, keep_states=True)
        dv, dg, _ = binding.scan_backward(v, g, (dy @ self.w_out).contiguous(), states=states)
        dp = torch.cat([dv, dg], -1)
        dx, dw, db = binding.layer_norm_backward(s, dp @ self.w_in, stats, self.norm_w, ds,
                                                 want_db=True)
        flat = dp.flatten(0, 1)
        return {"x": dx, "w_in": flat.T @ n.flatten(0, 1), "b_gate": dg.flatten(0, 1).sum(0),
                "w_out": dy.flatten(0, 1).T @ h.flatten(0, 1), "norm_w": dw, "norm_b": db}


def main():
    block = RecurrentBlock()
    B, T, new = 2, 300, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(B, T + new, 512, generator=g, device="cuda").bfloat16() for _ in range(2))
    whole, s, _ = block.prompt(x, r)
    _, _, state = block.prompt(x[:, :T].contiguous(), r[:, :T].contiguous())
    for t in range(T, T + new):
        y, _ = block.step(x[:, t].contiguous(), r[:, t].contiguous(), state)
        off = (y - whole[:, t]).float().norm() / whole[:, t].float().norm()
        print(f"token {t}: step against the whole prompt, relative difference {off:.1e}")
    dy, ds = (torch.randn(whole.shape, generator=g, device="cuda").bfloat16() for _ in range(2))
    for name, d in block.gradients(x, r, dy, ds).items():
        print(f"gradient of {name}: shape {tuple(d.shape)}, norm {d.float().norm():.3e}")
    assert binding.gdn_get_last_device_status() == binding.GDN_OK


if __name__ == "__main__":
    main()
