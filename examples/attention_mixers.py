"""Two more token mixers of a hybrid model, built from the library's operators.

* ``LinearMixer``: projection -> linear attention with a decay for each head -> output; training, prefill and decoding.
* ``CachedAttention``: the serving side of a softmax attention layer: a prompt's keys and values go into a paged cache with their
  rotation, then tokens one at a time are appended and attend over it.

``main`` checks that decoding token by token continues a prefill, and the linear mixer's gradients against differences.

    python examples/attention_mixers.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_delta_rule_gdn_gb300 as gdn  # noqa: E402


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g):
        ctx.save_for_backward(q, k, v, g)
        return gdn.lin_chunk_fwd(q, k, v, g)[0]

    @staticmethod
    def backward(ctx, d_o):
        q, k, v, g = ctx.saved_tensors
        return gdn.lin_chunk_bwd(q, k, v, g, d_o.contiguous())[:4]


def _param(gen, *shape, std=None, dtype=torch.bfloat16):
    x = torch.randn(shape, generator=gen, device="cuda") * (shape[-1] ** -0.5 if std is None else std)
    return x.to(dtype).requires_grad_()


class LinearMixer:
    """H value heads of size d on H_k query and key heads; a constant decay for each head, exp(-exp(log_decay))."""

    def __init__(self, width, H, H_k, d, gen, dtype=torch.bfloat16):
        self.H, self.H_k, self.d = H, H_k, d
        self.w_in = _param(gen, (2 * H_k + H) * d, width, dtype=dtype)
        self.log_decay = _param(gen, H, std=1.0, dtype=torch.float32)
        self.w_out = _param(gen, width, H * d, dtype=dtype)

    def parameters(self):
        return [self.w_in, self.log_decay, self.w_out]

    def _project(self, x):
        q, k, v = (x @ self.w_in.t()).split((self.H_k * self.d, self.H_k * self.d, self.H * self.d), -1)
        q, k, v = (t.unflatten(-1, (n, self.d)) for t, n in ((q, self.H_k), (k, self.H_k), (v, self.H)))
        return q, k, v, -self.log_decay.exp()

    def train_forward(self, x):
        return LinearAttention.apply(*self._project(x)).flatten(-2) @ self.w_out.t()

    @torch.no_grad()
    def prefill(self, x):
        o, state = gdn.lin_chunk_fwd(*self._project(x), output_final_state=True)
        return o.flatten(-2) @ self.w_out.t(), state

    @torch.no_grad()
    def decode(self, x, state):
        return gdn.lin_recurrent_step(*self._project(x), state).flatten(-2) @ self.w_out.t()


class CachedAttention:
    """Keys and values of N sequences in pages; `lengths` counts each one's tokens."""

    def __init__(self, width, H_q, H_k, d, gen, N, max_pages, page_size=16, dtype=torch.bfloat16):
        self.H_q, self.H_k, self.d = H_q, H_k, d
        self.w_in, self.w_out = _param(gen, (H_q + 2 * H_k) * d, width, dtype=dtype), _param(gen, width, H_q * d, dtype=dtype)
        pool = torch.zeros(N * max_pages, 2, page_size, H_k, d, dtype=dtype, device="cuda")     # both sides of a page together
        self.k_cache, self.v_cache = pool[:, 0], pool[:, 1]
        self.table = torch.randperm(N * max_pages, generator=gen, device="cuda").int().view(N, max_pages)
        self.lengths = torch.zeros(N, dtype=torch.int32, device="cuda")
        angles = torch.arange(max_pages * page_size, device="cuda")[:, None] * 10000.0 ** (-torch.arange(d // 2, device="cuda") * 2 / d)
        self.cos, self.sin = angles.cos(), angles.sin()

    def _project(self, x):
        q, k, v = (x @ self.w_in.t()).split((self.H_q * self.d, self.H_k * self.d, self.H_k * self.d), -1)
        return (t.unflatten(-1, (-1, self.d)) for t in (q, k, v))

    @torch.no_grad()
    def fill(self, x, cu_seqlens):
        """Prompts [tokens, width] of the sequences, packed."""
        _, k, v = self._project(x)
        self.lengths += cu_seqlens[1:] - cu_seqlens[:-1]
        gdn.paged_append(k, v, self.k_cache, self.v_cache, self.table, self.lengths, cu_seqlens=cu_seqlens, cos=self.cos, sin=self.sin)

    @torch.no_grad()
    def decode(self, x):
        q, k, v = self._project(x)
        self.lengths += 1
        q = gdn.paged_append(k, v, self.k_cache, self.v_cache, self.table, self.lengths, q=q, cos=self.cos, sin=self.sin)
        o = gdn.paged_attn_step(q, self.k_cache, self.v_cache, self.table, self.lengths)
        return o.flatten(-2) @ self.w_out.t()


def linear_continuation(layer, width, B=3, prompt=200, steps=10, seed=1):
    """Largest relative difference between the prefill of prompt + steps tokens and decoding the last ones."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, prompt + steps, width, generator=gen, device="cuda").to(layer.w_in.dtype)
    want = layer.prefill(x)[0].float()
    _, state = layer.prefill(x[:, :prompt].contiguous())
    worst = 0.0
    for t in range(prompt, prompt + steps):
        got = layer.decode(x[:, t].contiguous(), state).float()
        worst = max(worst, float((got - want[:, t]).norm() / want[:, t].norm()))
    return worst


def attention_continuation(width, gen, dtype=torch.bfloat16, lens=(40, 1, 77), seed=2):
    """The last token's output after a prompt, against the same layer fed token by token from the start."""
    a = CachedAttention(width, 8, 2, 64, gen, len(lens), 8, dtype=dtype)
    b = CachedAttention(width, 8, 2, 64, gen, len(lens), 8, dtype=dtype)
    b.w_in, b.w_out = a.w_in, a.w_out
    draw = torch.Generator(device="cuda").manual_seed(seed)
    x = [torch.randn(n + 1, width, generator=draw, device="cuda").to(dtype) for n in lens]
    cu = torch.tensor([0] + list(lens), device="cuda").cumsum(0).int()
    a.fill(torch.cat([t[:-1] for t in x]), cu)
    got = a.decode(torch.stack([t[-1] for t in x])).float()
    worst = 0.0
    for n, t in enumerate(x):                             # one sequence at a time: the others repeat their first token
        b.lengths.zero_()
        for i in range(len(t)):
            o = b.decode(t[i].expand(len(lens), width))
        worst = max(worst, float((o[n].float() - got[n]).norm() / got[n].norm()))
    return worst


def gradient_error(width=32, B=2, T=70, seed=3):
    """Largest difference between a parameter's gradient along a random direction and the difference of losses, relative to it (fp32)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer = LinearMixer(width, 4, 2, 16, gen, dtype=torch.float32)
    x = torch.randn(B, T, width, generator=gen, device="cuda")
    y = torch.randn(B, T, width, generator=gen, device="cuda")
    layer.train_forward(x).mul(y).sum().backward()
    worst = 0.0
    for p in layer.parameters():
        d = torch.randn(p.shape, generator=gen, device="cuda")
        d *= p.detach().norm() / d.norm()
        want = float((p.grad * d).sum())
        at = []
        with torch.no_grad():
            for h in (1e-2, -1e-2):
                p += h * d
                at.append(float((layer.train_forward(x) * y).double().sum()))
                p -= h * d
        worst = max(worst, abs((at[0] - at[1]) / 2e-2 - want) / float(p.grad.norm() * d.norm()))
    return worst


def main():
    gen = torch.Generator(device="cuda").manual_seed(0)
    width = 256
    linear = linear_continuation(LinearMixer(width, 8, 4, 64, gen), width)
    attention = attention_continuation(width, gen)
    gradient = gradient_error()
    assert gdn.device_status() == 0
    print(f"LinearMixer: decoding continues a prefill to {linear:.1e}, gradients agree with differences to {gradient:.1e}")
    print(f"CachedAttention: a prompt and tokens one at a time agree to {attention:.1e}")
    return linear, attention, gradient


if __name__ == "__main__":
    main()
