"""A feed-forward block on the library's products and row operators: training and decoding.

    out = gate(norm(x + r) · W1ᵀ) · W2ᵀ,    gate([g | u]) = silu(g) * u

Training runs its forward products on block-scaled e4m3 operands (the norm and the gate write them),
keeps g and u in 8 bits, and runs its backward products in bf16.  Decoding runs one to sixteen tokens through the
same weights in 4 bits.

    python examples/feed_forward.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from blackwell_tensor_core_tma_gb300 import gemm  # noqa: E402

EPS = 1e-6


def blocks(k: int) -> int:
    return (k + 31) // 32


def to_e4m3(w: torch.Tensor):
    """N x K fp32 weights as a block-scaled e4m3 operand: codes, UE8M0 scales per 32 of K (K % 32 == 0)."""
    n, k = w.shape
    p = w.view(n, k // 32, 32)
    code = ((p.abs().amax(2).view(torch.int32) + 0x1FFFFF) >> 23).sub_(8).clamp_(min=0)
    q = (p * ((254 - code) << 23).view(torch.float32)[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(n, k).view(torch.uint8), code.to(torch.uint8)


def to_e2m1(w: torch.Tensor):
    """N x K fp32 weights in 4 bits with a UE4M3 scale per 16 of K (K % 32 == 0): packed codes, scales."""
    n, k = w.shape
    p = w.view(n, k // 16, 16)
    sf = (p.abs().amax(2) / 6).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize((p / sf.float()[:, :, None]).abs(), edges).to(torch.uint8) | ((p < 0).to(torch.uint8) << 3)
    code = code.view(n, k // 2, 2)
    return (code[:, :, 0] | (code[:, :, 1] << 4)).contiguous(), sf.view(torch.uint8)


class FeedForward:
    """Weights in fp32 (w1: 2 inner x hidden, w2: hidden x inner, norm: hidden) and the plans of one batch size."""

    def __init__(self, tokens: int, hidden: int, inner: int, seed: int = 0, device: str = "cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.tokens, self.hidden, self.inner = M, H, F = tokens, hidden, inner
        self.w1 = torch.randn(2 * F, H, generator=gen, device=device) * H ** -0.5
        self.w2 = torch.randn(H, F, generator=gen, device=device) * F ** -0.5
        self.norm = torch.ones(H, device=device)

        def new(dtype, *shape):
            return torch.empty(*shape, dtype=dtype, device=device)

        bf16, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
        # kept from the forward pass for the backward pass: h and rstd, g and u in 8 bits
        self.h, self.rstd = new(bf16, M, H), new(f32, M)
        self.ck, self.sfck = new(u8, M, 2 * F), new(u8, M, 2 * blocks(F))
        # passed from one operator to the next
        self.y, self.sfy, self.z = new(u8, M, H), new(u8, M, blocks(H)), new(bf16, M, 2 * F)
        self.a, self.sfa, self.out = new(u8, M, F), new(u8, M, blocks(F)), new(bf16, M, H)
        self.da, self.dz, self.dy, self.dx = new(bf16, M, F), new(bf16, M, 2 * F), new(bf16, M, H), new(bf16, M, H)
        self.a16, self.y16 = new(bf16, M, F), new(bf16, M, H)
        self.dw1, self.dw2, self.dnorm = new(f32, 2 * F, H), new(f32, H, F), new(f32, H)
        self.workspace = new(f32, min(M, gemm.GEMM_NORM_PARTS), H)

        up, keep = gemm.GEMM_SCALE_UE8M0_32, dict(a_row_major=False, b_row_major=True)
        self.up = gemm.Plan(M, 2 * F, H, "e4m3", "bf16", up)
        self.down = gemm.Plan(M, H, F, "e4m3", "bf16", up)
        self.d_down = gemm.Plan(M, F, H, "bf16", "bf16", b_row_major=True)
        self.d_up = gemm.Plan(M, H, 2 * F, "bf16", "bf16", b_row_major=True)
        self.d_w2 = gemm.Plan(H, F, M, "bf16", "f32", **keep)
        self.d_w1 = gemm.Plan(2 * F, H, M, "bf16", "f32", **keep)
        self.prepare()

    def prepare(self):
        """The weights as the products take them; again after every change of w1 and w2."""
        self.w1_q, self.sf1 = to_e4m3(self.w1)
        self.w2_q, self.sf2 = to_e4m3(self.w2)
        self.w1_16, self.w2_16 = self.w1.bfloat16(), self.w2.bfloat16()

    def forward(self, x, r):
        """out of x and the residual stream r (both tokens x hidden bf16); h = x + r is the new stream."""
        M, H, F, s = self.tokens, self.hidden, self.inner, torch.cuda.current_stream()
        gemm.gemm_norm_run(M, H, "bf16", "bf16", "e4m3", EPS, x, r, self.norm, self.h, self.y, self.sfy, self.rstd, s)
        self.up.run(self.y, self.w1_q, None, self.z, self.sfy, self.sf1, s)
        gemm.gemm_gate_run(M, F, "bf16", "e4m3", self.z, self.a, self.sfa, self.ck, self.sfck, s)
        self.down.run(self.a, self.w2_q, None, self.out, self.sfa, self.sf2, s)
        return self.out

    def backward(self, dout, dh):
        """dx (that of x and of r) from the gradients at out and at h; leaves dw1, dw2 and dnorm."""
        M, H, F, s = self.tokens, self.hidden, self.inner, torch.cuda.current_stream()
        self.d_down.run(dout, self.w2_16, None, self.da, None, None, s)
        gemm.gemm_gate_backward(M, F, "bf16", "bf16", "bf16", self.da, self.ck, self.sfck, self.dz, self.a16, s)
        self.d_w2.run(dout, self.a16, None, self.dw2, None, None, s)
        self.d_up.run(self.dz, self.w1_16, None, self.dy, None, None, s)
        gemm.gemm_norm_backward(M, H, "bf16", "bf16", "bf16", self.dy, dh, self.h, self.rstd, self.norm, self.dx, self.dnorm,
                                self.y16, self.workspace, self.workspace.numel() * 4, s)
        self.d_w1.run(self.dz, self.y16, None, self.dw1, None, None, s)
        return self.dx

    def step(self, rate: float):
        self.w1 -= rate * self.dw1
        self.w2 -= rate * self.dw2
        self.norm -= rate * self.dnorm
        self.prepare()

    def close(self):
        for plan in (self.up, self.down, self.d_down, self.d_up, self.d_w1, self.d_w2):
            plan.close()


class Decoder:
    """The same block for a few tokens at a time, weights in 4 bits."""

    def __init__(self, block: FeedForward):
        self.hidden, self.inner, self.norm = block.hidden, block.inner, block.norm
        self.w1, self.sf1 = to_e2m1(block.w1)
        self.w2, self.sf2 = to_e2m1(block.w2)

    def __call__(self, x, r):
        """(out, h) of 1 to 16 rows x and r."""
        m, H, F, s = x.shape[0], self.hidden, self.inner, torch.cuda.current_stream()
        h, y, z = torch.empty_like(r), torch.empty_like(x), x.new_empty(m, 2 * F)
        a, out = x.new_empty(m, F), torch.empty_like(x)
        gemm.gemm_norm_run(m, H, "bf16", "bf16", "bf16", EPS, x, r, self.norm, h, y, None, None, s)
        gemm.gemm_matvec_run(m, 2 * F, H, "bf16", "bf16", gemm.GEMM_SCALE_UE4M3_16, y, self.w1, self.sf1, None, z, s)
        gemm.gemm_gate_run(m, F, "bf16", "bf16", z, a, None, None, None, s)
        gemm.gemm_matvec_run(m, H, F, "bf16", "bf16", gemm.GEMM_SCALE_UE4M3_16, a, self.w2, self.sf2, None, out, s)
        return out, h


def train(tokens=512, hidden=512, inner=1024, steps=20, rate=2.0, seed=0, report=print):
    """Fit the block to another one's outputs; returns the block, the losses and the data."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x, r = (torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16() for _ in range(2))
    teacher = FeedForward(tokens, hidden, inner, seed=seed + 2)
    target = teacher.forward(x, r).float()
    teacher.close()
    block, losses = FeedForward(tokens, hidden, inner, seed=seed), []
    none = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")      # nothing else reads the stream
    for i in range(steps):
        error = block.forward(x, r).float() - target
        losses.append(float(error.square().mean()))
        block.backward((error * (2.0 / error.numel() * tokens)).bfloat16(), none)
        block.step(rate / tokens)
        if i % 5 == 0 or i == steps - 1:
            report(f"step {i}: mean squared error {losses[-1]:.4f}")
    return block, losses, x, r


def main():
    block, _, x, r = train()
    out = block.forward(x, r)[:4].float()
    few, _ = Decoder(block)(x[:4], r[:4])
    rel = float((few.float() - out).norm() / out.norm())
    print(f"4 tokens with 4-bit weights against the 8-bit block: relative difference {rel:.3f}")
    block.close()


if __name__ == "__main__":
    main()
