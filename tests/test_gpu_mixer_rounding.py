"""How far results in bf16 are off, in the mean, beside the error that their own rounding
makes. In each sum of products one operand of a product is exact and the other rounded to
bf16 at most once, off like the rounding of the result by up to 2^-8 of it: the two
together are off by sqrt(2) of one in the root mean square. Bar: 1.5, the rest for the
scatter of a mean over some thousands of values. (The rms over a result's elements of the
difference to 64 bits, over the same of the 64-bit value rounded to bf16.)"""
import pytest
import torch

import test_gpu_linattn as lin
import test_gpu_swa as swa
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


@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks,lens", [
    (1, 0, 24, 3, 128, 144, 7, [2, 3, 1, 4]), (4, 27, 4, 2, 128, 93, 130, None), (1, 0, 3, 1, 128, 88, 0, [123, 153, 51, 180, 132, 175]),
    (1, 0, 8, 2, 32, 2, 0, [60, 3, 50, 1]), (1, 0, 8, 8, 128, 5, 0, [23, 16, 26, 30]), (1, 0, 9, 3, 64, 101, 64, [213, 36, 88, 244]),
    (2, 92, 4, 2, 64, 357, 7, None), (1, 2231, 3, 1, 32, 2, 0, None), (2, 57, 4, 4, 128, 1, 7, None), (3, 424, 9, 3, 64, 126, 130, None),
    (1, 1050, 32, 8, 128, 300, 4, None), (1, 1400, 4, 1, 64, 1000, 0, None), (1, 600, 32, 32, 128, 3, 1, None)])
def test_window(kda, B, T, Hq, Hkv, d, window, sinks, lens):  # noqa: F811
    x = swa.make(B, T, Hq, Hkv, d, BF16, lens=lens, seed=T + window)
    kw = dict(window=window, sinks=sinks, cu_seqlens=x["cu"])
    o, lse = kda.swa_fwd(x["q"], x["k"], x["v"], **kw)
    g = kda.swa_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], **kw)
    ro, _, r, _ = mixers.swa(x["q"], x["k"], x["v"], window, sinks, d ** -0.5, x["seqs"], x["dO"])
    check("o", o, ro)
    for n in g:
        check(n, g[n], r[n])


@pytest.mark.parametrize("T,window,sinks", [(1024, 1024, 0), (2048, 512, 4)])
def test_window_of_sharp_scores(kda, T, window, sinks):  # noqa: F811
    """Scores of deviation 4: a row's weight lies on few of its keys."""
    x = swa.make(1, T, 4, 1, 128, BF16, seed=T)
    x["q"] = x["q"] * 4
    o, lse = kda.swa_fwd(x["q"], x["k"], x["v"], window=window, sinks=sinks)
    g = kda.swa_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], window=window, sinks=sinks)
    ro, _, r, _ = mixers.swa(x["q"], x["k"], x["v"], window, sinks, 128 ** -0.5, x["seqs"], x["dO"])
    check("o", o, ro)
    for n in g:
        check(n, g[n], r[n])


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("T", [200, 1000])
def test_slow_constant_decays(kda, T, dtype):  # noqa: F811
    """Constant decays from 1/2 to 1 - 2^-12.9, per head: states carry no rounding that adds
    up from token to token. A state is multiplied once a block (32 tokens and more) by a
    product of decays rounded to fp32, half a step off at most and always the same: over
    the mean age of a state's terms, up to T / 2 tokens, (T / 64) 2^-24; besides that fp32
    sums, a few 2^-24, at most 5e-7 in the root mean square (mixer_checks, TAU_F32 / 5 sigma
    would be 4e-6 for single elements). One rounding a token instead: T / 2 of them."""
    H = 24
    x = lin.make(2, T, H, 32, 64, dtype, "head", seed=T)
    x["gate"] = (1 - 2.0 ** -(1 + torch.arange(H, dtype=torch.float64) / 2)).float().cuda()
    args = (x["q"], x["k"], x["v"], x["gate"])
    _, S_T = kda.linattn_fwd(*args, S0=x["S0"])
    g = kda.linattn_bwd(*args, x["dO"], S0=x["S0"], dS_T=x["dS_T"])
    _, rS, _ = mixers.linattn(*args, x["S0"], x["seqs"])
    r = mixers.linattn_grad(*args, x["dO"], x["S0"], x["dS_T"], x["seqs"])
    bar = T / 64 * 2.0 ** -24 + 5e-7
    for name, a, b in (("S_T", S_T, rS), ("dS0", g["dS0"], r["dS0"])):
        off = (a.double() - b).square().mean((0, 2, 3)).sqrt() / b.square().mean((0, 2, 3)).sqrt()
        print(name, ["%.1e" % e for e in off.tolist()], flush=True)
        assert off.max() <= bar, (name, off.max().item(), bar)
