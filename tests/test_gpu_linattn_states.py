"""Linear attention holds its states in 32 bits wherever it keeps them: at segment
boundaries, at blocks of the gradient and while it walks a segment (bf16 inputs).

Each input makes a state the small difference of two large numbers, so that a large
one held or added in 16 bits would leave nothing right of it. Away from there a single
row i of the state is not zero, read one element at a time (q, v and dO of one
nonzero element), so every result is one product.

Bars, per element and relative to the value:
* results in bf16: the state enters the product rounded to bf16, the product is rounded
  to bf16, half a step (2^-8) each, and the fp32 errors below: READ = 2^-7 + 2^-10.
* states in fp32: the difference is of 2^-12 of the terms and up. Decays are products of
  three bf16 numbers, 24 bits, exact. The start state's term is rounded once, the
  token's twice (decayed row; three bf16 parts of it are exact), their sum once, half a
  step (2^-24) of terms of about the same size each, of which the sum's is of the
  difference only: 3 * 2^-24 / 2^-12; and the 64-bit value is that of the same inputs.
  With one more rounding in reserve (the order in which a matrix instruction adds the
  three parts): HELD = 4 * 2^-12 = 2^-10. Two bf16 parts in place of three are off by up
  to 2^-17 / 2^-12 = 2^-5, and more than HELD at nearly every element."""
import pytest
import torch

from oracle import mixers
from test_gpu_linattn import kda  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
READ, HELD = 2.0 ** -7 + 2.0 ** -10, 2.0 ** -10
B, T, H = 1, 520, 64     # segments of two blocks of 64 tokens (forward), of three (gradient)


def tokens_per_segment(kda, dk, dv, grad):
    """From the workspace, which holds each segment's states and, in the gradient, each
    block's."""
    state, blocks = dk * dv, B * ((T + 63) // 64) * H
    if grad:
        segs = (kda.linattn_bwd_workspace_bytes(B, H, T, dk, dv) - blocks * (4 * state + 4)) // (8 * state + 4)
    else:
        segs = kda.linattn_fwd_workspace_bytes(B, H, T, dk, dv) // (4 * state + 4)
    per = segs // (B * H)
    return [L for L in range(64, T + 64, 64) if (T + L - 1) // L == per]


def zeros(dk, dv):
    x = dict(q=torch.zeros(B, T, H, dk), k=torch.zeros(B, T, H, dk), v=torch.zeros(B, T, H, dv), gate=torch.ones(B, T, H))
    x["dO"] = torch.zeros(B, T, H, dv)
    return x


def almost(g, *shape):
    """x in bf16 (|x| in [1, 2), either sign) and y in fp32 with x + y of 2^-12 to 2^-11 of x."""
    x = ((1 + torch.rand(shape, generator=g)) * (1 - 2 * (torch.rand(shape, generator=g) < 0.5).float())).to(BF16)
    return x, (-x.double() * (1 - 2.0 ** -12 * (1 + torch.rand(shape, generator=g, dtype=torch.float64)))).float()


def decays(g):
    """Three neighbouring decays a head, bf16 in (0.5, 1)."""
    return (0.5 + 0.5 * torch.rand(B, 3, H, generator=g)).to(BF16).float()


def one_hot(g, n):
    """[B, T, H, n], one nonzero element a token: element t % n, in +-[1, 2)."""
    x = torch.zeros(B, T, H, n)
    x[:, torch.arange(T), :, torch.arange(T) % n] = almost(g, T, B, H)[0].float()
    return x


def to_gpu(x):
    return {n: (t.cuda() if n in ("S0", "dS_T") else t.to(BF16).cuda()) for n, t in x.items()}


def near(name, x, ref, bar):
    x, ref = x.double(), ref.double()
    assert (ref != 0).any(), name
    worst = ((x - ref).abs() / ref.abs().clamp_min(1e-300)).nan_to_num(float("inf"))
    worst = torch.where(ref == 0, torch.where(x == 0, 0.0, float("inf")), worst).max().item()
    assert worst <= bar, "%s off by %.3g of its value (bar %.3g)" % (name, worst, bar)


SIZES = [(64, 64), (128, 128), (64, 128), (128, 16)]


@pytest.mark.parametrize("dk,dv", SIZES)
def test_start_state_in_32_bits(kda, dk, dv):  # noqa: F811
    """S0 less its rounding to bf16 is what the first block leaves."""
    assert min(tokens_per_segment(kda, dk, dv, False)) >= 128
    g, x, i = torch.Generator().manual_seed(dk + dv), zeros(dk, dv), 5
    x["S0"] = torch.zeros(B, H, dk, dv)
    x["S0"][:, :, i] = 1 + torch.rand(B, H, dv, generator=g)
    x["k"][:, 3, :, i] = 1
    x["v"][:, 3] = -x["S0"][:, :, i].to(BF16).float()
    x["q"][..., i] = one_hot(g, 1)[..., 0]
    x = to_gpu(x)
    o, S_T = kda.linattn_fwd(x["q"], x["k"], x["v"], x["gate"], S0=x["S0"])
    ro, rS, _ = mixers.linattn(x["q"], x["k"], x["v"], x["gate"], x["S0"], mixers.spans(B, T))
    near("S_T", S_T, rS, HELD)   # every step of it is exact
    near("o", o[:, 64:], ro[:, 64:], READ)


@pytest.mark.parametrize("dk,dv", SIZES)
def test_decayed_rows_in_32_bits(kda, dk, dv):  # noqa: F811
    """S0, decayed, and a token's row, decayed by as much, almost cancel."""
    assert min(tokens_per_segment(kda, dk, dv, False)) >= 128
    g, x, i = torch.Generator().manual_seed(dk + dv + 1), zeros(dk, dv), 9
    v, y = almost(g, B, H, dv)
    x["S0"] = torch.zeros(B, H, dk, dv)
    x["S0"][:, :, i] = y
    x["k"][:, 60, :, i] = 1
    x["v"][:, 60] = v.float()
    x["gate"][:, 61:64] = decays(g)
    x["q"][..., i] = one_hot(g, 1)[..., 0]
    x = to_gpu(x)
    o, S_T = kda.linattn_fwd(x["q"], x["k"], x["v"], x["gate"], S0=x["S0"])
    ro, rS, _ = mixers.linattn(x["q"], x["k"], x["v"], x["gate"], x["S0"], mixers.spans(B, T))
    near("S_T", S_T, rS, HELD)
    near("o", o[:, 64:], ro[:, 64:], READ)
    # one short sequence in one launch
    part = {n: t[:, :100].contiguous() for n, t in x.items() if n != "S0"}
    o, S_T = kda.linattn_fwd(part["q"], part["k"], part["v"], part["gate"], S0=x["S0"])
    near("S_T", S_T, rS, HELD)
    near("o", o[:, 64:], ro[:, 64:100], READ)


@pytest.mark.parametrize("dk,dv", SIZES)
def test_gradient_of_queries_in_32_bits(kda, dk, dv):  # noqa: F811
    """The same state, as dq = S dO reads it."""
    assert min(tokens_per_segment(kda, dk, dv, True)) >= 128
    g, x, i = torch.Generator().manual_seed(dk + dv + 2), zeros(dk, dv), 3
    v, y = almost(g, B, H, dv)
    x["S0"] = torch.zeros(B, H, dk, dv)
    x["S0"][:, :, i] = y
    x["k"][:, 60, :, i] = 1
    x["v"][:, 60] = v.float()
    x["gate"][:, 61:64] = decays(g)
    x["dO"] = one_hot(g, dv)
    x["dO"][:, :64] = 0
    x = to_gpu(x)
    r = mixers.linattn_grad(x["q"], x["k"], x["v"], x["gate"], x["dO"], x["S0"], None, mixers.spans(B, T))
    got = kda.linattn_bwd(x["q"], x["k"], x["v"], x["gate"], x["dO"], S0=x["S0"])
    near("dq", got["dq"], r["dq"], READ)


@pytest.mark.parametrize("dk,dv", SIZES)
def test_gradient_of_keys_and_values_in_32_bits(kda, dk, dv):  # noqa: F811
    """The adjoint: dS_T, decayed, and a later token's q dO^T almost cancel."""
    assert min(tokens_per_segment(kda, dk, dv, True)) >= 128
    g, x, i = torch.Generator().manual_seed(dk + dv + 3), zeros(dk, dv), 7
    up, y = almost(g, B, H, dv)
    x["dS_T"] = torch.zeros(B, H, dk, dv)
    x["dS_T"][:, :, i] = y
    x["q"][:, 66, :, i] = 1
    x["dO"][:, 66] = up.float()
    x["gate"][:, 64:67] = decays(g)
    x["v"] = one_hot(g, dv)
    x["k"][..., i] = one_hot(g, 1)[..., 0]
    x = to_gpu(x)
    r = mixers.linattn_grad(x["q"], x["k"], x["v"], x["gate"], x["dO"], None, x["dS_T"], mixers.spans(B, T))
    got = kda.linattn_bwd(x["q"], x["k"], x["v"], x["gate"], x["dO"], dS_T=x["dS_T"])
    near("dk", got["dk"][:, :64], r["dk"][:, :64], READ)
    near("dv", got["dv"][:, :64], r["dv"][:, :64], READ)
    near("dS0", got["dS0"], r["dS0"], HELD)
