"""How far results in bf16 are off, in the mean, beside the error that their own rounding
makes. In each sum of products one operand of a product is exact and the other rounded to
bf16 at most once, off like the rounding of the result by up to 2^-8 of it: the two
together are off by sqrt(2) of one in the root mean square. Bar: 1.5, the rest for the
scatter of a mean over some thousands of values. (The rms over a result's elements of the
difference to 64 bits, over the same of the 64-bit value rounded to bf16.)"""
import pytest
import torch

import test_gpu_linattn as lin
from oracle import mixers
from test_gpu_linattn import kda  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
BAR = 1.5


def check(name, x, ref):
    assert x.dtype == BF16 and x.numel() >= 2000, name
    own = (ref.to(BF16).double() - ref).square().mean().sqrt()
    ratio = ((x.double() - ref).square().mean().sqrt() / own).item()
    print(name, "%.3f" % ratio, flush=True)
    assert ratio <= BAR, "%s off by %.3f of its own rounding" % (name, ratio)


@pytest.mark.parametrize("states", [True, False])
@pytest.mark.parametrize("B,T,H,dk,dv,lens", [
    (1, 700, 8, 128, 128, None), (64, 6, 16, 128, 128, None), (4, 68, 32, 64, 32, None), (2, 1100, 16, 64, 128, None),
    (32, 2, 64, 128, 64, None), (1, 0, 32, 16, 128, [2, 2, 8, 3, 90, 9, 3]), (4, 147, 32, 16, 16, None),
    (1, 0, 16, 32, 32, [112, 137, 59, 97]), (2, 300, 16, 128, 16, None)])
def test_linear(kda, B, T, H, dk, dv, lens, states):  # noqa: F811
    x = lin.make(B, T, H, dk, dv, BF16, "token", lens=lens, states=states, seed=T + dk + dv)
    args, kw = (x["q"], x["k"], x["v"], x["gate"]), dict(S0=x["S0"], cu_seqlens=x["cu"])
    o, _ = kda.linattn_fwd(*args, **kw)
    g = kda.linattn_bwd(*args, x["dO"], dS_T=x["dS_T"], **kw)
    ro, _, _ = mixers.linattn(*args, x["S0"], x["seqs"])
    r = mixers.linattn_grad(*args, x["dO"], x["S0"], x["dS_T"], x["seqs"])
    check("o", o, ro)
    for n in ("dq", "dk", "dv", "dgate"):
        check(n, g[n], r[n])
