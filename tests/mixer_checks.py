"""Bars shared by the tests of linear attention and window attention, per
element: |x - ref| <= half a step of the output type at ref + tau * rms(ref).

tau, from how the operands are rounded inside:
* fp32 in and out: sums of a few hundred products, each off by at most a few
  2^-24; sqrt(512) * 2^-24 * 5 (the largest of about 1e5 normal errors is under
  5 sigma) * 3 (chained products) = 2e-5.
* bf16 out: one operand of every product is rounded to bf16, off by 2^-8 at
  most, 2^-8 / sqrt(3) in the mean square; two to three such roundings in a row,
  largest of 1e5 under 5 sigma: 5 * 2^-8 / sqrt(3) * sqrt(3) = 2e-2.
* fp32 sums of bf16 inputs (states): scaled rows as two bf16 numbers, off by
  2^-17: 5 * 2^-17 = 4e-5, with the fp32 part above 6e-5.

`size`, for a result whose elements are sums of terms of very different number
and size (a sink key's gradient has terms from every row, its neighbour's from a
window), or the difference of larger terms (the softmax's gradient, sum_j p (dP -
delta) k): the root of the terms' summed squares, per element. Each term is
rounded by itself, so an element's error is tau times that, however far its terms
cancel and whatever the other elements are: a row that sees one key has p = 1,
dP = delta and a gradient of exactly zero, of which fp32 leaves 2^-24 |dO v| k. An
element is then held to tau times rms(ref) or its size, whichever is larger."""
import torch

STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TAU_F32, TAU_BF16, TAU_STATE = 2e-5, 2e-2, 6e-5


def tau_for(inputs, out):
    if inputs == torch.float32:
        return TAU_F32
    return TAU_BF16 if out == torch.bfloat16 else TAU_STATE


def close(name, x, ref, inputs, tau=None, size=None):
    assert x.shape == ref.shape, name
    if ref.numel() == 0:
        return
    tau = tau_for(inputs, x.dtype) if tau is None else tau
    x, ref, step = x.double(), ref.double().to(x.device), STEP[x.dtype]
    assert torch.isfinite(x).all(), "%s is not finite" % name
    rms = ref.square().mean().sqrt()
    scale = rms if size is None else torch.maximum(rms, size)
    over = ((x - ref).abs() - step * ref.abs()) / scale.clamp_min(1e-300)
    worst = over.max().item() if rms > 0 else (x - ref).abs().max().item()
    assert worst <= tau, "%s off by %.3g of its rms (bar %.3g)" % (name, worst, tau)
