"""Linear attention and window attention in the plans that large inputs take: segments
of several blocks, and workgroups whose waves share no rows (window attention), against
the definitions in 64 bits, at head sizes of 64 and 128. Which plan an input takes is
read off the workspace's size (linear attention) or off the names of the kernels that
ran, so that a change of the rules cannot move these cases to other plans unseen."""
import re

import pytest
import torch

import test_gpu_linattn as lin
import test_gpu_swa as swa
from mixer_checks import STEP, TAU_F32, close, tau_for
from oracle import mixers

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
kda = swa.kda   # the fixture


# ---------------------------------------------------------------- linear attention

def blocks_per_segment(kda, x, grad):
    """At most, by the size of the workspace: fp32 states of every segment and, in the
    gradient, of every block of 64 (fp32: 32) tokens."""
    B, T, H, dk = x["q"].shape
    dv, dt, cu = x["v"].shape[-1], x["q"].dtype, x["cu"]
    N, state, C = len(x["seqs"]), dk * dv, 64 if dt == BF16 else 32
    numbers = lambda L: T // L + N + 1 if cu is not None else B * ((T + L - 1) // L)  # noqa: E731
    if grad:
        size = kda.linattn_bwd_workspace_bytes(B, H, T, dk, dv, N, cu is not None, dt)
        segs = (size - numbers(C) * H * (4 * state + 4)) // (8 * state + 4)
    else:
        segs = kda.linattn_fwd_workspace_bytes(B, H, T, dk, dv, N, cu is not None, dt) // (4 * state + 4)
    return min(L for L in range(64, T + 64, 64) if numbers(L) * H <= segs) // C


def term_sizes(x):
    """Per element of o, dq, dk and dv the root of its terms' summed squares, a term being
    one pair of tokens' or one row's of a boundary state or adjoint. Decays that are zero
    here and there cut some tokens' sums to one term and leave hundreds to others, whose
    values and errors are several times the rms over all: each term is rounded by itself,
    up to 2^-8 of it, so an element is off by tau (five times the root of the mean square
    of three such roundings) times this size, and by less than tau times the rms only where
    the size is below it."""
    q, k, v, dO = (x[n].double() for n in ("q", "k", "v", "dO"))
    a = x["gate"].double().expand(q.shape[:3])
    size = {n: torch.zeros_like(t) for n, t in (("o", v), ("dq", q), ("dk", k), ("dv", v))}
    for s, (b, t0, t1) in enumerate(x["seqs"]):
        n = t1 - t0
        if n == 0:
            continue
        al, qs, ks, vs, gs = (t[b, t0:t1].transpose(0, 1).contiguous() for t in (a, q, k, v, dO))   # [H, n, .]
        D = torch.zeros(q.shape[2], n, n, dtype=torch.float64, device=q.device)   # D[i, j] = a_{j+1} .. a_i
        for i in range(n):
            if i:
                D[:, i] = D[:, i - 1] * al[:, i, None]
            D[:, i, i] = 1.0
        flip = lambda t: t.transpose(1, 2).contiguous()  # noqa: E731
        P, R = ((D * (y @ flip(z))).square() for y, z in ((qs, ks), (gs, vs)))
        first, last = (D[:, :, 0] * al[:, :1]).square()[:, :, None], D[:, n - 1].square()[:, :, None]
        qs, ks, vs, gs, S0, E = (t.square() for t in (qs, ks, vs, gs, x["S0"][s].double(), x["dS_T"][s].double()))
        for m, y in (("o", P @ vs + first * (qs @ S0)), ("dq", R @ ks + first * (gs @ flip(S0))),
                     ("dk", flip(R) @ qs + last * (vs @ flip(E))), ("dv", flip(P) @ gs + last * (ks @ E))):
            size[m][b, t0:t1] = y.sqrt().transpose(0, 1)
    return size


def check_fwd(kda, x):
    o, S_T = kda.linattn_fwd(x["q"], x["k"], x["v"], x["gate"], S0=x["S0"], cu_seqlens=x["cu"])
    ro, rS, _ = mixers.linattn(x["q"], x["k"], x["v"], x["gate"], x["S0"], x["seqs"])
    close("o", o, ro, x["q"].dtype, size=term_sizes(x)["o"])
    close("S_T", S_T, rS, x["q"].dtype)


def check_bwd(kda, x):
    g = kda.linattn_bwd(x["q"], x["k"], x["v"], x["gate"], x["dO"], S0=x["S0"], dS_T=x["dS_T"], cu_seqlens=x["cu"])
    r = mixers.linattn_grad(x["q"], x["k"], x["v"], x["gate"], x["dO"], x["S0"], x["dS_T"], x["seqs"])
    size = term_sizes(x)
    for n in ("dq", "dk", "dv", "dgate", "dS0"):
        if g[n] is not None:
            close(n, g[n], r[n], x["q"].dtype, size=size.get(n))
    assert (g["dgate"] is None) == (x["gate"].dim() == 1)


LONG = [
    # B, T, H, dk, dv, lens; more than 33,280 tokens by heads, 16,640 for the gradient
    (1, 1100, 32, 64, 64, None), (1, 1100, 32, 128, 128, None), (1, 1100, 32, 64, 128, None), (2, 570, 64, 128, 64, None),
    (1, 1100, 32, 32, 128, None), (1, 0, 32, 128, 128, [700, 1, 0, 333, 66]), (1, 0, 32, 64, 64, [65, 1000, 35]),
]
WIDE = [(2, 700, 64, 32, 32, None), (1, 1400, 64, 16, 64, None), (1, 1400, 64, 64, 16, None)]


@pytest.mark.parametrize("gate", ["token", "signed", "head"])
@pytest.mark.parametrize("B,T,H,dk,dv,lens", LONG + WIDE)
def test_linear_forward_in_segments_of_blocks(kda, B, T, H, dk, dv, lens, gate):
    x = lin.make(B, T, H, dk, dv, BF16, gate, lens=lens, seed=T + dk)
    assert blocks_per_segment(kda, x, False) >= 2
    check_fwd(kda, x)


@pytest.mark.parametrize("gate", ["token", "signed", "head"])
@pytest.mark.parametrize("B,T,H,dk,dv,lens", [(b, t, h // 2 if k > 32 or v > 32 else h, k, v, s) for b, t, h, k, v, s in LONG] + WIDE)
def test_linear_gradient_in_segments_of_blocks(kda, B, T, H, dk, dv, lens, gate):
    x = lin.make(B, T, H, dk, dv, BF16, gate, lens=lens, seed=T + dk + 1)
    assert blocks_per_segment(kda, x, True) >= 2
    check_bwd(kda, x)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 32)])
def test_linear_fp32_in_segments_of_blocks(kda, dk, dv):
    x = lin.make(1, 1100, 32, dk, dv, F32, "signed", seed=dk)
    assert blocks_per_segment(kda, x, False) >= 4 and blocks_per_segment(kda, x, True) >= 4
    check_fwd(kda, x)
    check_bwd(kda, x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [None, [300, 0, 1, 299]])
def test_linear_against_the_delta_rule_without_erasing(kda, lens, dtype):
    """kda_chunk_fwd_ew and its gradient with nothing erased and all written, on the same
    inputs. Bars: the sum of both calls' own, 1e-4 (bf16 inputs 2e-2; gradients 1e-4) of
    the rms there."""
    x = lin.make(2, 600, 8, 64, 128, dtype, "token", lens=lens, seed=5)
    args, kw = (x["q"], x["k"], x["v"], x["gate"]), dict(S0=x["S0"], cu_seqlens=x["cu"])
    gates = torch.zeros_like(x["k"]), torch.ones_like(x["v"])
    bar = 1e-4 if dtype == F32 else 2e-2
    o, S_T = kda.linattn_fwd(*args, **kw)
    ro, rS = kda.chunk_fwd_ew(*args, *gates, gate_kind=kda.GATE_SCALAR, **kw)
    close("o", o, ro, dtype, tau_for(dtype, dtype) + bar * (1 + STEP[dtype]))
    close("S_T", S_T, rS, dtype, tau_for(dtype, F32) + bar)
    g = kda.linattn_bwd(*args, x["dO"], dS_T=x["dS_T"], **kw)
    r = kda.chunk_bwd_ew(*args, *gates, x["dO"].float(), dS_T=x["dS_T"], gate_kind=kda.GATE_SCALAR, **kw)
    for n in ("dq", "dk", "dv", "dgate"):
        close(n, g[n], r[n], dtype, tau_for(dtype, dtype) + 1e-4 * (1 + STEP[dtype]))
    close("dS0", g["dS0"], r["dS0"], dtype, tau_for(dtype, F32) + 1e-4)


# ---------------------------------------------------------------- window attention

def kernels(call):
    """Names of the library's kernels that `call` launches, or None without a profiler."""
    from torch.profiler import ProfilerActivity, profile
    call()
    torch.cuda.synchronize()
    try:
        with profile(activities=[ProfilerActivity.CUDA]) as p:
            call()
            torch.cuda.synchronize()
    except RuntimeError as e:
        print("no profiler:", e, flush=True)
        return None
    names = [re.search(r"(\w+_kernel<[^>]*>)", e.name) for e in p.events() if "kda::" in e.name]
    return {n.group(1).replace("unsigned short", "bf16") for n in names if n} or None


MANY = [
    # B, T, Hq, Hkv, d, window, sinks, lens: 256 workgroups of 128 rows by heads and more
    (1, 1050, 32, 8, 128, 300, 4, None), (1, 1050, 32, 8, 64, 300, 4, None), (1, 0, 32, 8, 128, 200, 70, [700, 2, 0, 348]),
    (2, 530, 32, 32, 128, 160, 0, None), (1, 1100, 30, 10, 64, 1000, 1, None), (1, 0, 64, 8, 64, 96, 3, [33, 600, 1]),
]
FEW = [(1, 1050, 8, 2, 128, 300, 4, None), (1, 800, 2, 1, 128, 400, 0, None)]


def check_window(kda, x, window, sinks):
    """As test_gpu_swa.check, with o held to the root of its terms' summed squares p v where
    that is above the rms: a sequence's first rows are a mean of few keys, of the size of v,
    its later ones of hundreds, of a tenth of that and less, and every p is rounded by
    itself, by up to 2^-8 of it."""
    kw = dict(window=window, sinks=sinks, cu_seqlens=x["cu"])
    o, lse = kda.swa_fwd(x["q"], x["k"], x["v"], **kw)
    g = kda.swa_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], **kw)
    scale, dt, group = x["q"].shape[-1] ** -0.5, x["q"].dtype, x["q"].shape[2] // x["k"].shape[2]
    ro, rl, rg, size = mixers.swa(x["q"], x["k"], x["v"], window, sinks, scale, x["seqs"], x["dO"])
    size["o"] = torch.zeros_like(ro)
    for b, t0, t1 in x["seqs"]:
        hidden = ~mixers.visible(t1 - t0, window, sinks, "cuda")
        for h in range(ro.shape[2]):
            y, z = (x[n][b, t0:t1, h // group].double() for n in ("k", "v"))
            s = torch.mm(x["q"][b, t0:t1, h].double(), y.t().contiguous()) * scale
            p = torch.exp(s - rl[b, t0:t1, h, None]).masked_fill(hidden, 0.0)
            size["o"][b, t0:t1, h] = torch.mm(p.square(), z.square()).sqrt()
    close("o", o, ro, dt, size=size["o"])
    close("lse", lse, rl, dt, TAU_F32)
    for n in g:
        close(n, g[n], rg[n], dt, size=size[n])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks,lens", MANY + FEW)
def test_window_wide(kda, B, T, Hq, Hkv, d, window, sinks, lens, dtype):
    """Most tiles of these lie wholly inside the window."""
    check_window(kda, swa.make(B, T, Hq, Hkv, d, dtype, lens=lens, seed=T + window), window, sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks,lens", MANY + FEW)
def test_window_plans(kda, B, T, Hq, Hkv, d, window, sinks, lens, dtype):
    few = (B, T, Hq, Hkv, d, window, sinks, lens) in FEW
    x = swa.make(B, T, Hq, Hkv, d, dtype, lens=lens)
    kw = dict(window=window, sinks=sinks, cu_seqlens=x["cu"])
    o, lse = kda.swa_fwd(x["q"], x["k"], x["v"], **kw)
    ran = kernels(lambda: (kda.swa_fwd(x["q"], x["k"], x["v"], **kw),
                           kda.swa_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], **kw)))
    if ran is None:
        pytest.skip("this profiler shows no kernels")
    print(ran, flush=True)
    for name in ("swa_fwd_kernel", "swa_dq_kernel"):
        alone = "%s<%s, %d, 4, 1>" % (name, "bf16" if dtype == BF16 else "float", d)
        assert (alone in ran) != few, ran


@pytest.mark.parametrize("N,Hq,Hkv,d,window,sinks", [(1, 4, 2, 128, 4000, 3), (3, 16, 4, 64, 1500, 0), (70, 8, 8, 32, 400, 1)])
def test_step_on_full_caches_fp32(kda, N, Hq, Hkv, d, window, sinks):
    """Long caches in full precision, in parts and whole."""
    g = torch.Generator().manual_seed(N)
    rnd = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    slots = window + sinks
    q, k, v, K, V = rnd(N, Hq, d), rnd(N, Hkv, d), rnd(N, Hkv, d), rnd(N, slots, Hkv, d), rnd(N, slots, Hkv, d)
    pos = torch.randint(0, 3 * slots, (N,), generator=g).to(torch.int32)
    o = kda.swa_decode_step(q, k, v, K, V, pos.cuda(), window=window, sinks=sinks)
    torch.cuda.synchronize()
    want = torch.zeros(N, Hq, d, dtype=torch.float64, device="cuda")
    for n, p in enumerate(pos.tolist()):
        slot = p if p < sinks else sinks + (p - sinks) % window
        assert torch.equal(K[n, slot], k[n]) and torch.equal(V[n, slot], v[n])
        m = min(p + 1, slots)
        for h in range(Hq):
            s = (K[n, :m, h // (Hq // Hkv)].double() * q[n, h].double()).sum(1) * d ** -0.5
            want[n, h] = (torch.softmax(s, 0)[:, None] * V[n, :m, h // (Hq // Hkv)].double()).sum(0)
    close("o", o, want, F32)
