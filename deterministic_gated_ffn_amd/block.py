"""The FFN half of a transformer layer, composed of the library's calls (no
arithmetic here): the norm before the block, the gated FFN with its activations
saved in 8 bits, or a mixture of experts for a few tokens, and the norm after
it with gate and residual.

Training, one layer over tokens [M, H]:

    h       = norm(x; w_in)                           norm_fwd
    y, ckpt = FFN(h), g and u kept in 8 bits          ffn_fwd_q8
    z       = alpha x + gate norm(y; w_out)           norm_fwd

and back through norm_bwd, ffn_bwd_q8 and norm_bwd.  A layer keeps x, h, y, z
(H wide, 16 bits) and the two checkpoints (I wide, 8.5 bits an element instead
of 16).  Serving replaces the FFN with moe_fwd.

    python -m deterministic_gated_ffn_amd.block       # one training step and one served batch
"""
from __future__ import annotations

import torch

from . import binding as dgf


class FfnBlock:
    """z = alpha x + gate norm(FFN(norm(x))), forward and backward."""

    def __init__(self, w_in, w_gate, w_up, w_down, w_out, gate=None, alpha: float = 1.0, eps: float = 1e-6):
        self.w_in, self.w_out, self.gate, self.alpha, self.eps = w_in, w_out, gate, alpha, eps
        self.w = (w_gate, w_up, w_down)

    def forward(self, x, stream=None):
        """Returns z and what the backward needs."""
        pre = dgf.norm_fwd(x, w_next=self.w_in, eps=self.eps, training=True, stream=stream)
        y, g8, u8 = dgf.ffn_fwd_q8(pre["h"], *self.w, stream=stream)
        post = dgf.norm_fwd(x, y, w_post=self.w_out, gate=self.gate, alpha=self.alpha, eps=self.eps, training=True,
                            stream=stream)
        return post["z"], (x, pre["h"], pre["rstd"], y, g8, u8, post["z"], post["rstd"])

    def backward(self, dz, saved, stream=None):
        """Gradients of the block's parameters, and dx."""
        x, h, rstd_in, y, g8, u8, z, rstd_out = saved
        post = dgf.norm_bwd(dz, None, z, y, w_post=self.w_out, gate=self.gate, alpha=self.alpha, rstd=rstd_out,
                            stream=stream)
        ffn = dgf.ffn_bwd_q8(post["dy"], h, g8, u8, *self.w, stream=stream)
        # the residual's gradient and the norm's meet in one pass: dx = alpha dz + the norm's Jacobian
        pre = dgf.norm_bwd(post["dres"], ffn["dX"], x, w_next=self.w_in, rstd=rstd_in, stream=stream)
        grads = {"dx": pre["dres"], "dw_in": pre["dw_next"], "dw_out": post["dw_post"], "dW_gate": ffn["dW_gate"],
                 "dW_up": ffn["dW_up"], "dW_down": ffn["dW_down"]}
        if self.gate is not None:
            grads["dgate"] = post["dgate"]
        return grads


class MoeBlock:
    """z = alpha x + gate norm(MoE(norm(x))) for a few tokens at a time."""

    def __init__(self, w_in, w_router, w_gate, w_up, w_down, w_out, top_k: int, gate=None, alpha: float = 1.0,
                 eps: float = 1e-6):
        self.w_in, self.w_out, self.gate, self.alpha, self.eps = w_in, w_out, gate, alpha, eps
        self.w, self.top_k = (w_router, w_gate, w_up, w_down), top_k

    def __call__(self, x, w_next=None, stream=None):
        """The new residual z, and with w_next the next block's normed input."""
        h = dgf.norm_fwd(x, w_next=self.w_in, eps=self.eps, stream=stream)["h"]
        y = dgf.moe_fwd(h, *self.w, self.top_k, stream=stream)
        r = dgf.norm_fwd(x, y, w_post=self.w_out, gate=self.gate, alpha=self.alpha, w_next=w_next, eps=self.eps,
                         stream=stream)
        return (r["z"], r["h"]) if w_next is not None else r["z"]


def _demo(M: int = 512, H: int = 1024, I: int = 4096, E: int = 16, k: int = 2) -> None:
    gen = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, scale=1.0, shift=0.0):
        t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        return t.normal_(shift, scale, generator=gen)

    ones = lambda: rand(H, scale=0.05, shift=1.0)  # noqa: E731
    block = FfnBlock(ones(), rand(I, H, scale=0.02), rand(I, H, scale=0.02), rand(H, I, scale=0.02), ones(),
                     gate=rand(H, scale=0.1, shift=0.5))
    x = rand(M, H)
    z, saved = block.forward(x)
    grads = block.backward(rand(M, H, scale=0.1), saved)
    kept = sum(t.codes.nbytes + t.scales.nbytes for t in (saved[4], saved[5]))
    print(f"training step, {M} tokens: |z| = {z.float().norm().item():.1f}, |dx| = {grads['dx'].float().norm().item():.2f}, "
          f"g and u kept in {kept / 1e6:.2f} MB instead of {4 * M * I / 1e6:.2f}")
    moe = MoeBlock(ones(), rand(E, H, scale=0.05), rand(E, I, H, scale=0.02), rand(E, I, H, scale=0.02),
                   rand(E, H, I, scale=0.02), ones(), k)
    z, h = moe(x[:8], w_next=ones())
    print(f"served batch, 8 tokens over {k} of {E} experts: |z| = {z.float().norm().item():.1f}, "
          f"|h| = {h.float().norm().item():.1f}")


if __name__ == "__main__":
    _demo()
