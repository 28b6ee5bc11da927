"""Two token mixers of a hybrid model built from the library's operators: prefill, decode and training.

* ``DeltaMixer``: projection -> short convolution of q, k, v -> unit-norm query and key heads -> gated delta rule -> output.
* ``RecurrentMixer``: projection -> short convolution -> gated linear recurrence -> output.

Both keep what decoding needs in a state (the convolution's last inputs, and the delta rule's or the recurrence's state).
``main`` checks that decoding token by token continues a prefill, then trains the pair for some steps on a synthetic task.

    python examples/hybrid_mixer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_delta_rule_gdn_gb300 as gdn  # noqa: E402


class ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return gdn.gdn_short_conv_fwd(x, weight, bias=bias)[0]

    @staticmethod
    def backward(ctx, d_y):
        x, weight, bias = ctx.saved_tensors
        return gdn.gdn_short_conv_bwd(x, weight, d_y.contiguous(), bias=bias)[:3]


class UnitHeads(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k):
        ctx.save_for_backward(q, k)
        return gdn.gdn_qk_norm_fwd(q, k, norm="l2")

    @staticmethod
    def backward(ctx, d_q, d_k):
        q, k = ctx.saved_tensors
        return gdn.gdn_qk_norm_bwd(q, k, d_q.contiguous(), d_k.contiguous(), norm="l2")[:2]


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, in_gate, A_log, dt_bias):
        o, _, ck = gdn.glr_scan_fwd(x, g, in_gate=in_gate, A_log=A_log, dt_bias=dt_bias, normalize=True,
                                    output_checkpoints=True)
        ctx.save_for_backward(x, g, in_gate, A_log, dt_bias, ck)
        return o

    @staticmethod
    def backward(ctx, d_o):
        x, g, in_gate, A_log, dt_bias, ck = ctx.saved_tensors
        dx, dg, di, _, dA, ddt = gdn.glr_scan_bwd(x, g, d_o.contiguous(), in_gate=in_gate, A_log=A_log, dt_bias=dt_bias,
                                                  normalize=True, checkpoints=ck)
        return dx, dg, di, dA, ddt


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, A_log, dt_bias):
        ctx.save_for_backward(q, k, v, g, beta, A_log, dt_bias)
        return gdn.gdn_chunk_fwd(q, k, v, g, beta, A_log=A_log, dt_bias=dt_bias, beta_sigmoid=True,
                                 o_dtype=torch.bfloat16)[0]

    @staticmethod
    def backward(ctx, d_o):
        q, k, v, g, beta, A_log, dt_bias = ctx.saved_tensors
        dq, dk, dv, dg, dbeta, _, dA, ddt = gdn.gdn_chunk_bwd(q, k, v, g, beta, d_o.contiguous(), A_log=A_log,
                                                              dt_bias=dt_bias, beta_sigmoid=True,
                                                              want_d_initial_state=False)
        return dq.to(q.dtype), dk.to(q.dtype), dv.to(q.dtype), dg, dbeta, dA, ddt


def _param(gen, *shape, std=None, dtype=torch.bfloat16):
    std = shape[-1] ** -0.5 if std is None else std
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype).requires_grad_()


class DeltaMixer:
    def __init__(self, width, heads, gen, W=4, d=128):
        self.H, self.d = heads, d
        n = 3 * heads * d
        self.w_in = _param(gen, n + 2 * heads, width)
        self.conv_w, self.conv_b = _param(gen, n, W, dtype=torch.float32), _param(gen, n, std=0.0, dtype=torch.float32)
        self.A_log = _param(gen, heads, std=0.5, dtype=torch.float32)
        self.dt_bias = _param(gen, heads, std=0.1, dtype=torch.float32)
        self.w_out = _param(gen, width, heads * d)

    def parameters(self):
        return [self.w_in, self.conv_w, self.conv_b, self.A_log, self.dt_bias, self.w_out]

    def _project(self, x):
        p = x @ self.w_in.t()
        n = 3 * self.H * self.d
        return p[..., :n], p[..., n:n + self.H].float().contiguous(), p[..., n + self.H:].float().contiguous()

    def _heads(self, c):
        q, k, v = c.split(self.H * self.d, -1)
        return (t.unflatten(-1, (self.H, self.d)) for t in (q, k, v))

    def train_forward(self, x):
        qkv, g, beta = self._project(x)
        q, k, v = self._heads(ShortConv.apply(qkv, self.conv_w, self.conv_b))
        q, k = UnitHeads.apply(q, k)
        o = DeltaRule.apply(q, k, v.contiguous(), g, beta, self.A_log, self.dt_bias)
        return o.flatten(-2) @ self.w_out.t()

    @torch.no_grad()
    def prefill(self, x):
        qkv, g, beta = self._project(x)
        c, conv = gdn.gdn_short_conv_fwd(qkv, self.conv_w, bias=self.conv_b, output_final_state=True)
        q, k, v = self._heads(c)
        q, k = gdn.gdn_qk_norm_fwd(q, k, norm="l2")
        o, state = gdn.gdn_chunk_fwd(q, k, v.contiguous(), g, beta, output_final_state=True, A_log=self.A_log,
                                     dt_bias=self.dt_bias, beta_sigmoid=True, o_dtype=torch.bfloat16)
        return o.flatten(-2) @ self.w_out.t(), {"conv": conv, "state": state}

    @torch.no_grad()
    def decode(self, x, s):
        qkv, g, beta = self._project(x)
        q, k, v = self._heads(gdn.gdn_short_conv_step(qkv, s["conv"], self.conv_w, self.conv_b))
        q, k = gdn.gdn_qk_norm_fwd(q, k, norm="l2")
        o = gdn.gdn_recurrent_step(q, k, v.contiguous(), g, beta, s["state"], A_log=self.A_log, dt_bias=self.dt_bias,
                                   beta_sigmoid=True, o_dtype=torch.bfloat16)
        return o.flatten(-2) @ self.w_out.t()


class RecurrentMixer:
    def __init__(self, width, inner, gen, W=4):
        self.inner = inner
        self.w_in = _param(gen, 3 * inner, width)
        self.conv_w, self.conv_b = _param(gen, inner, W, dtype=torch.float32), _param(gen, inner, std=0.0, dtype=torch.float32)
        self.A_log = (_param(gen, inner, std=1.0, dtype=torch.float32).detach() - 3).requires_grad_()
        self.dt_bias = _param(gen, inner, std=0.1, dtype=torch.float32)
        self.w_out = _param(gen, width, inner)

    def parameters(self):
        return [self.w_in, self.conv_w, self.conv_b, self.A_log, self.dt_bias, self.w_out]

    def _project(self, x):
        return (x @ self.w_in.t()).split(self.inner, -1)      # token, decay logits, input-gate logits

    def train_forward(self, x):
        u, g, i = self._project(x)
        u = ShortConv.apply(u, self.conv_w, self.conv_b)
        return Recurrence.apply(u, g, i, self.A_log, self.dt_bias) @ self.w_out.t()

    @torch.no_grad()
    def prefill(self, x):
        u, g, i = self._project(x)
        u, conv = gdn.gdn_short_conv_fwd(u, self.conv_w, bias=self.conv_b, output_final_state=True)
        o, state = gdn.glr_scan_fwd(u, g, in_gate=i, A_log=self.A_log, dt_bias=self.dt_bias, normalize=True,
                                    output_final_state=True)
        return o @ self.w_out.t(), {"conv": conv, "state": state}

    @torch.no_grad()
    def decode(self, x, s):
        u, g, i = self._project(x)
        u = gdn.gdn_short_conv_step(u, s["conv"], self.conv_w, self.conv_b)
        o = gdn.glr_step(u, g, s["state"], in_gate=i, A_log=self.A_log, dt_bias=self.dt_bias, normalize=True)
        return o @ self.w_out.t()


def continuation_error(layer, width, B=3, prompt=200, steps=20, seed=1):
    """Largest relative difference between the prefill of prompt + steps tokens and decoding the last ones."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, prompt + steps, width, generator=gen, device="cuda").bfloat16()
    want = layer.prefill(x)[0].float()
    _, s = layer.prefill(x[:, :prompt].contiguous())
    worst = 0.0
    for t in range(prompt, prompt + steps):
        got = layer.decode(x[:, t].contiguous(), s).float()
        worst = max(worst, float((got - want[:, t]).norm() / want[:, t].norm()))
    return worst


def train(layers, width, steps=60, B=4, T=256, lr=3e-3, seed=2):
    """Losses of gradient descent on: the output is the running mean of the inputs so far."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    params = [p for layer in layers for p in layer.parameters()]
    opt = torch.optim.Adam(params, lr=lr)
    losses = []
    for _ in range(steps):
        x = torch.randn(B, T, width, generator=gen, device="cuda").bfloat16()
        target = x.float().cumsum(1) / torch.arange(1, T + 1, device="cuda")[:, None].sqrt()
        y = sum(layer.train_forward(x) for layer in layers).float()
        loss = (y - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def main():
    gen = torch.Generator(device="cuda").manual_seed(0)
    width = 256
    layers = [DeltaMixer(width, 2, gen), RecurrentMixer(width, 512, gen)]
    errors = [continuation_error(layer, width) for layer in layers]
    losses = train(layers, width)
    assert gdn.device_status() == 0
    for layer, e in zip(layers, errors):
        print(f"{type(layer).__name__}: decoding continues a prefill to {e:.1e}")
    print(f"training loss {losses[0]:.3f} -> {losses[-1]:.3f} in {len(losses)} steps")
    return errors, losses


if __name__ == "__main__":
    main()
