"""A gated recurrent block from the package's operators, for training, prefill
and single-token decode:

    n  = norm(stream)                          8-bit or bf16 rows
    p  = n w_in^T + b_in                       x | g | z side by side
    h  = gated recurrence of x under g, times silu(z)
    s  = stream + h w_out^T                    (added inside the second norm)
    u  = gelu(norm(s) w_up^T + b_up)
    stream <- s + u w_down^T                   (added inside the product)

The residual stream is held in 32 bits, the weights in bf16.  ``forward`` keeps
what ``backward`` needs; ``step`` is one token with the recurrence's state in
place; ``in_8_bits`` gives the same block with the weights behind the norms as
E4M3 values with a scale a row, and the norms writing such rows.

    python -m state_space_model_chunked_gb300.gated_block      # one training step and a few tokens
"""
from __future__ import annotations

import dataclasses

import torch

from .layer_ops import (gated_scan_bwd, gated_scan_fwd, gated_state_update, linear_bwd, linear_fwd,
                        rmsnorm_bwd, rmsnorm_fwd)

E4M3 = torch.float8_e4m3fn


def rows_in_8_bits(w):
    """A weight matrix as E4M3 values and one scale a row (done once, at load time)."""
    w = w.float()
    top = w.abs().amax(dim=1)
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    return (w / scale[:, None]).to(E4M3), scale


@dataclasses.dataclass
class GatedBlock:
    """The block's parameters: matrices [out, in] bf16, vectors f32."""
    norm1: torch.Tensor
    w_in: torch.Tensor
    b_in: torch.Tensor
    w_out: torch.Tensor
    norm2: torch.Tensor
    w_up: torch.Tensor
    b_up: torch.Tensor
    w_down: torch.Tensor
    eps: float = 1e-5
    # of in_8_bits(): the scales of w_in and w_up
    w_in_scale: torch.Tensor | None = None
    w_up_scale: torch.Tensor | None = None

    @classmethod
    def random(cls, d_model, d_inner, d_ff, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def matrix(out, inner):
            w = torch.empty((out, inner), device=device).normal_(0.0, inner ** -0.5, generator=gen)
            return w.to(torch.bfloat16)
        b_in = torch.zeros(3 * d_inner, device=device)
        b_in[d_inner:2 * d_inner] = 2.0         # gates that remember
        return cls(torch.ones(d_model, device=device), matrix(3 * d_inner, d_model), b_in,
                   matrix(d_model, d_inner), torch.ones(d_model, device=device),
                   matrix(d_ff, d_model), torch.zeros(d_ff, device=device), matrix(d_model, d_ff))

    @property
    def d_inner(self):
        return self.w_out.shape[1]

    def in_8_bits(self):
        """The block for serving with 8-bit weights and activations behind the norms."""
        w_in, s_in = rows_in_8_bits(self.w_in)
        w_up, s_up = rows_in_8_bits(self.w_up)
        return dataclasses.replace(self, w_in=w_in, w_in_scale=s_in, w_up=w_up, w_up_scale=s_up)

    def _norm(self, x, weight, residual=None):
        out = E4M3 if self.w_in_scale is not None else torch.bfloat16
        return rmsnorm_fwd(x, weight, residual, eps=self.eps, out_dtype=out)

    def _parts(self, p):
        d = self.d_inner
        return p[..., :d], p[..., d:2 * d], p[..., 2 * d:]

    def forward(self, stream, init_state=None, keep=True):
        """stream [batch, length, d_model] f32, init_state [batch, d_inner] f32
        or None.  Returns (stream, final state, what backward needs or None)."""
        n1, _, rstd1, c1 = self._norm(stream, self.norm1)
        p = linear_fwd(n1, self.w_in, self.b_in, x_scale=c1, w_scale=self.w_in_scale)
        x, g, z = self._parts(p)
        h, final, kept = gated_scan_fwd(x, g, z, init_state, return_checkpoints=True)
        o = linear_fwd(h, self.w_out)
        n2, s, rstd2, c2 = self._norm(o, self.norm2, stream)
        up = linear_fwd(n2, self.w_up, self.b_up, activation="gelu", x_scale=c2,
                        w_scale=self.w_up_scale, return_preact=keep)
        u, preact = up if keep else (up, None)
        out = linear_fwd(u, self.w_down, residual=s, out_dtype=torch.float32)
        saved = (stream, n1, rstd1, p, init_state, kept, h, s, n2, rstd2, preact, u) if keep else None
        return out, final, saved

    def backward(self, saved, dout, dfinal=None):
        """dout [batch, length, d_model] f32: the gradient of forward's stream;
        dfinal of its final state.  Returns (gradient of the stream, gradient of
        the initial state, gradients of the parameters by name)."""
        if self.w_in_scale is not None:
            raise ValueError("the 8-bit block is for serving: train the block it was made from")
        stream, n1, rstd1, p, init, kept, h, s, n2, rstd2, preact, u = saved
        grads = {}
        du, grads["w_down"], _ = linear_bwd(dout.to(torch.bfloat16), u, self.w_down, bias=False)
        dn2, grads["w_up"], grads["b_up"] = linear_bwd(du, n2, self.w_up, preact, activation="gelu")
        do, ds, grads["norm2"] = rmsnorm_bwd(dn2, s, self.norm2, rstd2, dout)
        dh, grads["w_out"], _ = linear_bwd(do, h, self.w_out, bias=False)
        x, g, z = self._parts(p)
        dp = torch.empty_like(p)                # the recurrence writes its three parts side by side
        dx, dg, dz = self._parts(dp)
        _, _, _, dinit = gated_scan_bwd(dh, x, g, kept, z, init, dfinal, dx=dx, dg=dg, dz=dz)
        dn1, grads["w_in"], grads["b_in"] = linear_bwd(dp, n1, self.w_in)
        _, dstream, grads["norm1"] = rmsnorm_bwd(dn1, stream, self.norm1, rstd1, ds)
        return dstream, dinit, grads

    def step(self, stream, state):
        """One token: stream [batch, d_model] f32, state [batch, d_inner] f32
        (updated in place).  Returns the stream."""
        n1, _, _, c1 = self._norm(stream, self.norm1)
        p = linear_fwd(n1, self.w_in, self.b_in, x_scale=c1, w_scale=self.w_in_scale)
        h = gated_state_update(state, *self._parts(p))
        o = linear_fwd(h, self.w_out)
        n2, s, _, c2 = self._norm(o, self.norm2, stream)
        u = linear_fwd(n2, self.w_up, self.b_up, activation="gelu", x_scale=c2,
                       w_scale=self.w_up_scale)
        return linear_fwd(u, self.w_down, residual=s, out_dtype=torch.float32)


def main():
    block = GatedBlock.random(768, 1536, 1536)
    gen = torch.Generator(device="cuda").manual_seed(1)
    stream = torch.empty((2, 512, 768), device="cuda").normal_(generator=gen)
    out, final, saved = block.forward(stream)
    loss = (out * out).mean()
    dstream, _, grads = block.backward(saved, out * (2.0 / out.numel()))
    print(f"loss {loss.item():.4f}, gradient norms: stream {dstream.norm().item():.3e}, " +
          ", ".join(f"{k} {v.float().norm().item():.3e}" for k, v in grads.items()))
    serving = block.in_8_bits()
    _, state, _ = serving.forward(stream, keep=False)
    token = stream[:, -1].contiguous()
    for _ in range(4):
        token = serving.step(token, state)
    print(f"four tokens in 8 bits: norm {token.norm().item():.4f}")


if __name__ == "__main__":
    main()
