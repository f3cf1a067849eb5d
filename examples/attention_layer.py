"""One attention layer beside the SSM core's, on one GPU:

    x = x + W_o attention(rotated norms of W_qkv norm(x))

over a sliding window with a few first tokens that stay visible: as a prompt
(prefill), token by token over a cache that wraps (decode), and its gradients.
Run it from the repository's root:

    python examples/attention_layer.py

It prints how far decoding the last tokens is from prefilling them, and how far
the gradient of x is from a difference quotient.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from state_space_sequence_03_amd import ops


class Layer:
    """Width D, heads of dim entries, a window with sinks."""

    def __init__(self, D, q_heads, kv_heads, dim, window, sinks, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn((rows, cols), device="cuda", generator=g) * cols ** -0.5).to(dtype)

        self.Hq, self.Hk, self.dim, self.dtype = q_heads, kv_heads, dim, dtype
        self.see = {"window": window, "sinks": sinks}
        self.W_qkv, self.W_o = weight((q_heads + 2 * kv_heads) * dim, D), weight(D, q_heads * dim)
        self.gain, self.bias = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
        self.gain_q, self.gain_k = torch.ones(dim, device="cuda"), torch.ones(dim, device="cuda")
        self.theta = 10000.0 ** (-torch.arange(dim // 2, device="cuda") * 2.0 / dim)

    def heads(self, qkv):
        """Queries, keys and values of a projection's rows (B, L, all heads, dim)."""
        return qkv[:, :, :self.Hq], qkv[:, :, self.Hq:self.Hq + self.Hk], qkv[:, :, self.Hq + self.Hk:]

    def project(self, x, pos=None):
        n, mean, rstd = ops.layer_norm_fwd(x, self.gain, self.bias, want_stats=True)
        qkv, _ = ops.linear_fwd(n, self.W_qkv)
        qkv = qkv.view(*x.shape[:2], -1, self.dim)
        q, k, v = self.heads(qkv)
        q, k = ops.qk_norm_rope_fwd(q, k, self.gain_q, self.gain_k, theta=self.theta, pos=pos)
        return n, mean, rstd, qkv, q, k, v

    def prefill(self, x):
        """x (B, L, D) -> the layer's output and what the backward takes."""
        n, mean, rstd, qkv, q, k, v = self.project(x)
        o, lse = ops.window_attn_fwd(q, k, v, want_lse=True, **self.see)
        y, _ = ops.linear_fwd(o.flatten(2), self.W_o, residual=x)
        return y, (x, n, mean, rstd, qkv, q, k, v, o, lse)

    def cache(self, k, v, capacity):
        """A cache of `capacity` slots that holds what a prompt's (B, L) keys and values leave in it."""
        B, L = k.shape[:2]
        S = self.see["sinks"]
        kc, vc = (torch.zeros((B, capacity, self.Hk, self.dim), dtype=self.dtype, device="cuda") for _ in range(2))
        pos = torch.arange(L, device="cuda")
        pos = pos[(pos < S) | (pos >= L - (capacity - S))]
        at = ops.window_cache_slots(pos, S, capacity)
        kc[:, at], vc[:, at] = k[:, pos], v[:, pos]
        return kc, vc, torch.full((B,), L, device="cuda")

    def decode(self, x, kc, vc, lens):
        """New tokens x (B, T, D) of each sequence; caches and lengths go along."""
        T = x.shape[1]
        *_, q, k, v = self.project(x, lens[:, None] + torch.arange(T, device="cuda"))
        o = ops.window_attn_decode(q, k, v, kc, vc, lens, **self.see)
        lens += T
        return ops.linear_fwd(o.flatten(2), self.W_o, residual=x)[0]

    def backward(self, saved, dy):
        """Gradients of x and of the weights."""
        x, n, mean, rstd, qkv, q, k, v, o, lse = saved
        out = ops.linear_bwd(o.flatten(2), self.W_o, dy, want_dbias=False)
        do = out["dx"].view_as(o)
        dqkv = torch.empty_like(qkv)
        dq, dk, dv = self.heads(dqkv)
        ops.window_attn_bwd(q, k, v, o, lse, do, dq=dq, dk=dk, dv=dv, **self.see)
        q, k, _ = self.heads(qkv)
        turn = ops.qk_norm_rope_bwd(q, k, dq, dk, self.gain_q, self.gain_k, theta=self.theta, dq=dq, dk=dk)
        proj = ops.linear_bwd(n, self.W_qkv, dqkv.flatten(2), want_dbias=False)
        norm = ops.layer_norm_bwd(x, mean, rstd, proj["dx"], self.gain, dskip=dy)
        return {"x": norm["dx"], "W_o": out["dW"], "W_qkv": proj["dW"], "gain": norm["dgain"], "bias": norm["dbias"],
                "gain_q": turn["dgain_q"], "gain_k": turn["dgain_k"]}


def main(B=2, L=200, D=256, q_heads=8, kv_heads=2, dim=64, window=64, sinks=4):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g)
    layer = Layer(D, q_heads, kv_heads, dim, window, sinks)
    x = rand(B, L, D).bfloat16()
    whole, _ = layer.prefill(x)

    # the prompt's first part, then one token at a time and a few at once
    prompt = L - 30
    _, saved = layer.prefill(x[:, :prompt].contiguous())
    caches = layer.cache(saved[6], saved[7], sinks + window + 7)
    parts, at = [], prompt
    for T in (1, 1, 8, 1, 8, 8, 1, 1, 1):
        parts.append(layer.decode(x[:, at:at + T].contiguous(), *caches))
        at += T
    off = float((torch.cat(parts, 1) - whole[:, prompt:at]).abs().max() / whole.abs().max())
    print(f"decode against prefill: {off:.1e} of the largest output")

    # in fp32: sum(y w) along a direction
    layer = Layer(D, q_heads, kv_heads, dim, window, sinks, dtype=torch.float32)
    x, w, d = rand(B, L, D), rand(B, L, D), rand(B, L, D)
    y, saved = layer.prefill(x)
    slope = float((layer.backward(saved, w)["x"].double() * d.double()).sum())
    step = 2.0 ** -8
    up, down = (float((layer.prefill(x + s * step * d)[0].double() * w.double()).sum()) for s in (1, -1))
    quotient = (up - down) / (2 * step)
    error = abs(quotient - slope) / abs(slope)
    print(f"gradient against a difference quotient: {error:.1e}")
    return off, error


if __name__ == "__main__":
    main()
