"""Window attention with sinks (kda_swa_*) against its definition in 64 bits, on
the GPU."""
import math

import pytest
import torch

from mixer_checks import TAU_F32, close
from oracle import mixers

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_46_amd import kda as m
    m.library()
    return m


def make(B, T, Hq, Hkv, d, dtype=BF16, lens=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    if lens is not None:
        B, T = 1, sum(lens)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64).to(dtype).cuda()  # noqa: E731
    x = dict(q=rnd(B, T, Hq, d), k=rnd(B, T, Hkv, d), v=rnd(B, T, Hkv, d), dO=rnd(B, T, Hq, d), cu=None)
    if lens is not None:
        x["cu"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    x["seqs"] = mixers.spans(B, T, x["cu"])
    print("case B", B, "T", T, "Hq", Hq, "Hkv", Hkv, "d", d, dtype, "lens", lens, flush=True)
    return x


def check(kda, x, window, sinks, scale=None):
    print("window", window, "sinks", sinks, flush=True)
    kw = dict(window=window, sinks=sinks, scale=scale, cu_seqlens=x["cu"])
    o, lse = kda.swa_fwd(x["q"], x["k"], x["v"], **kw)
    g = kda.swa_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], **kw)
    torch.cuda.synchronize()
    scale = x["q"].shape[-1] ** -0.5 if scale is None else scale
    ro, rl, rg, size = mixers.swa(x["q"], x["k"], x["v"], window, sinks, scale, x["seqs"], x["dO"])
    dt = x["q"].dtype
    close("o", o, ro, dt)
    close("lse", lse, rl, dt, TAU_F32)   # a sum of exact products, whatever the inputs
    for n in g:
        close(n, g[n], rg[n], dt, size=size[n])


SIZES = [
    # B, T, Hq, Hkv, d, window, sinks
    (1, 1, 1, 1, 64, 1, 0), (2, 2, 2, 1, 32, 1, 1), (1, 31, 2, 2, 128, 7, 0), (1, 33, 3, 1, 64, 33, 2),
    (2, 64, 2, 1, 128, 64, 0), (1, 65, 4, 2, 64, 16, 4), (1, 128, 2, 2, 32, 200, 0), (1, 129, 2, 1, 128, 100, 1),
    (1, 300, 4, 1, 64, 63, 5), (2, 257, 6, 3, 128, 1, 3), (1, 700, 2, 1, 128, 130, 70), (1, 520, 2, 2, 64, 1000, 9),
    (1, 640, 5, 1, 32, 65, 129), (1, 900, 2, 1, 64, 40, 400),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks", SIZES)
def test_sizes(kda, B, T, Hq, Hkv, d, window, sinks, dtype):
    check(kda, make(B, T, Hq, Hkv, d, dtype, seed=T + window), window, sinks)


LENS = [[5, 1, 0, 64, 70], [0, 0, 1], [128, 129, 1, 200], [0, 333, 0], [1, 2, 3, 4, 5, 6, 7], [500, 63, 0, 65]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("window,sinks", [(40, 3), (1, 0), (500, 150)])
def test_packed(kda, lens, window, sinks, dtype):
    check(kda, make(1, 0, 4, 2, 64, dtype, lens=lens, seed=sum(lens)), window, sinks)


def test_long_with_sinks(kda):
    check(kda, make(1, 3001, 2, 1, 128, BF16, seed=5), 200, 4)
    check(kda, make(1, 3001, 2, 1, 64, BF16, seed=6), 3, 1)


def test_scales(kda):
    x = make(1, 150, 2, 1, 64, F32, seed=9)
    for scale in (0.0, -0.125, 1.0):
        check(kda, x, 60, 2, scale)


def test_window_beyond_the_sequence(kda):
    """Any window that covers the sequence is causal attention, bit for bit."""
    x = make(1, 200, 2, 1, 64, BF16)
    a, la = kda.swa_fwd(x["q"], x["k"], x["v"], window=200)
    for window, sinks in ((201, 0), (2 ** 31 - 1, 0), (2 ** 40, 5), (200, 2 ** 31 - 1)):
        b, lb = kda.swa_fwd(x["q"], x["k"], x["v"], window=window, sinks=sinks)
        assert torch.equal(a, b) and torch.equal(la, lb)
    g = kda.swa_bwd(x["q"], x["k"], x["v"], a, la, x["dO"], window=200)
    g2 = kda.swa_bwd(x["q"], x["k"], x["v"], a, la, x["dO"], window=2 ** 31 - 1, sinks=2 ** 31 - 1)
    for n in g:
        assert torch.equal(g[n], g2[n]), n


def test_large_scores(kda):
    """Scores of some hundreds, where only a shifted exponential survives."""
    x = make(1, 200, 2, 2, 64, F32, seed=3)
    x["q"] = x["q"] * 30
    o, lse = kda.swa_fwd(x["q"], x["k"], x["v"], window=90, sinks=2)
    ro, rl = mixers.swa(x["q"], x["k"], x["v"], 90, 2, 0.125, x["seqs"])
    # scores s with |s| up to 30 * 8 * 5 / 8 * ... are off by 2^-24 sqrt(64) |q||k| scale ~ 1e-4 absolute at most,
    # which moves a probability, and with it o, by as much
    close("o", o, ro, F32, 1e-4)
    close("lse", lse, rl, F32, TAU_F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_bad_values_reach_only_rows_that_see_them(kda, bad, dtype):
    x = make(1, 300, 2, 1, 64, dtype, seed=4)
    window, sinks = 50, 3
    clean, lse = kda.swa_fwd(x["q"], x["k"], x["v"], window=window, sinks=sinks)
    ro, rl = mixers.swa(x["q"], x["k"], x["v"], window, sinks, 0.125, x["seqs"])
    at = 130
    sees = mixers.visible(300, window, sinks, "cuda")[:, at]
    for name in ("k", "v"):
        y = {n: x[n].clone() for n in ("q", "k", "v")}
        y[name][0, at, 0, 5] = bad
        o, l2 = kda.swa_fwd(y["q"], y["k"], y["v"], window=window, sinks=sinks)
        close("o", o[:, ~sees], ro[:, ~sees], dtype)
        close("lse", l2[:, ~sees], rl[:, ~sees], dtype, TAU_F32)
        if name == "v":
            assert torch.equal(l2, lse)
            assert not torch.isfinite(o[0, sees, :, 5]).any()
            keep = [c for c in range(64) if c != 5]
            close("o", o[:, sees][..., keep], ro[:, sees][..., keep], dtype)


def test_rows_behind_the_last_sequence(kda):
    x = make(1, 500, 2, 1, 64)
    lens = [200, 111]
    n = sum(lens)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    seqs = mixers.spans(1, 500, cu)
    out, lse = torch.full_like(x["q"], 7.0), torch.full(x["q"].shape[:3], 7.0, device="cuda")
    x["k"][:, n:], x["v"][:, n:], x["q"][:, n:], x["dO"][:, n:] = (math.nan,) * 4
    kda.swa_fwd(x["q"], x["k"], x["v"], window=60, sinks=4, cu_seqlens=cu, out=out, lse=lse)
    ro, rl, rg, size = mixers.swa(x["q"], x["k"], x["v"], 60, 4, 0.125, seqs, x["dO"])
    close("o", out[:, :n], ro[:, :n], BF16)
    assert (out[:, n:] == 7.0).all() and (lse[:, n:] == 7.0).all()
    g = {m: torch.full_like(x[s], 7.0) for m, s in (("dq", "q"), ("dk", "k"), ("dv", "v"))}
    kda.swa_bwd(x["q"], x["k"], x["v"], out, lse, x["dO"], window=60, sinks=4, cu_seqlens=cu, out=g)
    for m in g:
        close(m, g[m][:, :n], rg[m][:, :n], BF16, size=size[m][:, :n])
        assert (g[m][:, n:] == 7.0).all()


def test_gradient_against_differences(kda):
    """The kernel's gradient against central differences of the definition in 64
    bits (step 1e-4: the third-order remainder is under 1e-8)."""
    x = make(1, 40, 2, 1, 32, F32, seed=3)
    window, sinks, scale = 9, 2, 32 ** -0.5
    o, lse = kda.swa_fwd(x["q"], x["k"], x["v"], window=window, sinks=sinks)
    g = kda.swa_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], window=window, sinks=sinks)
    rng = torch.Generator().manual_seed(1)
    for name in ("q", "k", "v"):
        rms = g["d" + name].double().square().mean().sqrt().item()
        for e in torch.randint(0, x[name].numel(), (10,), generator=rng).tolist():
            d = []
            for sign in (1, -1):
                y = {n: x[n].double() for n in ("q", "k", "v")}
                y[name] = y[name].clone()
                y[name].view(-1)[e] += sign * 1e-4
                ro, _ = mixers.swa(y["q"], y["k"], y["v"], window, sinks, scale, x["seqs"])
                d.append((ro * x["dO"].double()).sum().item())
            got = g["d" + name].view(-1)[e].item()
            assert abs(got - (d[0] - d[1]) / 2e-4) <= 2e-5 * max(rms, abs(got)) + 1e-7, (name, e)


# ---------------------------------------------------------------- one token

def ring(kd, vd, pos, window, sinks):
    """o of the newest token from whole histories kd, vd [T, Hkv, d]."""
    keep = [j for j in range(pos + 1) if pos - j < window or j < sinks]
    return kd[keep], vd[keep]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,d,window,sinks", [(2, 1, 64, 5, 0), (4, 2, 128, 1, 0), (3, 3, 32, 64, 2), (8, 1, 64, 33, 4),
                                                   (40, 1, 64, 50, 1), (66, 2, 32, 7, 9), (4, 1, 128, 300, 4)])
def test_decode_continues_a_prompt(kda, Hq, Hkv, d, window, sinks, dtype):
    """Prompts of several lengths (an empty one too), then steps one by one past
    the wrap of the ring; slots without a token hold NaN."""
    lens = [0, 1, 3, window, window + sinks, 2 * window + sinks + 5]
    N, steps = len(lens), window % 7 + 4
    x = make(1, 0, Hq, Hkv, d, dtype, lens=[n + steps for n in lens], seed=window)
    first = [s[1] for s in x["seqs"]]
    K, V = (torch.full((N, sinks + window, Hkv, d), math.nan, dtype=dtype, device="cuda") for _ in range(2))
    pick = lambda t: torch.cat([t[0, a:a + n] for a, n in zip(first, lens)])[None].contiguous()  # noqa: E731
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    kda.swa_cache_fill(pick(x["k"]), pick(x["v"]), K, V, window=window, sinks=sinks, cu_seqlens=cu)
    pos = torch.tensor(lens, dtype=torch.int32).cuda()
    ro, _ = mixers.swa(x["q"], x["k"], x["v"], window, sinks, d ** -0.5, x["seqs"])
    for t in range(steps):
        rows = [a + n + t for a, n in zip(first, lens)]
        one = lambda m: x[m][0, rows].contiguous()  # noqa: E731
        o = kda.swa_decode_step(one("q"), one("k"), one("v"), K, V, pos, window=window, sinks=sinks)
        close("o at step %d" % t, o, ro[0, rows], dtype)
        pos += 1
    for s in range(N):
        n = lens[s] + steps
        for j in range(n):
            if n - 1 - j < window or j < sinks:
                slot = j if j < sinks else sinks + (j - sinks) % window
                assert torch.equal(K[s, slot], x["k"][0, first[s] + j]) and torch.equal(V[s, slot], x["v"][0, first[s] + j])
        assert torch.isnan(K[s, n:].float()).all() and torch.isnan(V[s, n:].float()).all()


@pytest.mark.parametrize("N,Hq,Hkv,d,window,sinks", [(1, 4, 2, 128, 4000, 3), (3, 16, 4, 64, 1500, 0), (70, 8, 8, 64, 400, 1),
                                                     (2, 48, 1, 128, 2000, 0), (300, 2, 1, 32, 70, 2)])
def test_decode_on_full_caches(kda, N, Hq, Hkv, d, window, sinks):
    """Long caches cut into parts, at any position far beyond the window."""
    g = torch.Generator().manual_seed(N)
    rnd = lambda *s: torch.randn(s, generator=g).to(BF16).cuda()  # noqa: E731
    slots = window + sinks
    q, k, v, K, V = rnd(N, Hq, d), rnd(N, Hkv, d), rnd(N, Hkv, d), rnd(N, slots, Hkv, d), rnd(N, slots, Hkv, d)
    pos = torch.randint(0, 3 * slots, (N,), generator=g).to(torch.int32)
    pos[0] = 2 ** 31 - 1
    if N > 2:
        pos[1] = -1
        K[1], V[1] = math.nan, math.nan
    K0 = K.clone()
    o = kda.swa_decode_step(q, k, v, K, V, pos.cuda(), window=window, sinks=sinks)
    torch.cuda.synchronize()
    want = torch.zeros(N, Hq, d, dtype=torch.float64, device="cuda")
    for n, p in enumerate(pos.tolist()):
        if p < 0:
            assert (o[n] == 0).all() and torch.isnan(K[n].float()).all()
            continue
        slot = p if p < sinks else sinks + (p - sinks) % window
        K0[n, slot] = k[n]
        assert torch.equal(K[n], K0[n]) and torch.equal(V[n, slot], v[n])
        m = min(p + 1, slots)
        for h in range(Hq):
            s = (K[n, :m, h // (Hq // Hkv)].double() * q[n, h].double()).sum(1) * d ** -0.5
            want[n, h] = (torch.softmax(s, 0)[:, None] * V[n, :m, h // (Hq // Hkv)].double()).sum(0)
    close("o", o, want, BF16)


def test_repeats_and_streams(kda):
    x = make(1, 0, 4, 2, 128, BF16, lens=[700, 3, 260], seed=2)
    kw = dict(window=200, sinks=4, cu_seqlens=x["cu"])
    o, lse = kda.swa_fwd(x["q"], x["k"], x["v"], **kw)
    g = kda.swa_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o2, l2 = kda.swa_fwd(x["q"], x["k"], x["v"], stream=st, **kw)
    g2 = kda.swa_bwd(x["q"], x["k"], x["v"], o2, l2, x["dO"], stream=st, **kw)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    for n in g:
        assert torch.equal(g[n], g2[n]), n


def test_graph_replays(kda):
    """Forward, gradient, cache and a step in one captured graph, on new inputs and
    a new split each time, against eager calls, bit for bit."""
    splits = ([300, 0, 155, 90], [1, 2, 270, 272], [545, 0, 0, 0])
    window, sinks = 60, 3
    xs = [make(1, 0, 4, 2, 64, BF16, lens=s, seed=20 + i) for i, s in enumerate(splits)]
    cur = {n: xs[0][n].clone() for n in ("q", "k", "v", "dO", "cu")}
    one = lambda n: cur[n][0, :4].contiguous()  # noqa: E731

    def work(K, V):
        kw = dict(window=window, sinks=sinks)
        o, lse = kda.swa_fwd(cur["q"], cur["k"], cur["v"], cu_seqlens=cur["cu"], **kw)
        g = kda.swa_bwd(cur["q"], cur["k"], cur["v"], o, lse, cur["dO"], cu_seqlens=cur["cu"], **kw)
        K.zero_()
        V.zero_()
        kda.swa_cache_fill(cur["k"], cur["v"], K, V, cu_seqlens=cur["cu"], **kw)
        pos = cur["cu"][1:] - cur["cu"][:-1]
        y = kda.swa_decode_step(one("q"), one("k"), one("v"), K, V, pos, **kw)
        return [o, lse, g["dq"], g["dk"], g["dv"], K, V, y]

    caches = [torch.empty((4, window + sinks, 2, 64), dtype=BF16, device="cuda") for _ in range(4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(*caches[:2])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work(*caches[:2])
    for x in xs + xs[:1]:
        for n in cur:
            cur[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = work(*caches[2:])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_poisoned_lds(kda):
    """The build that fills every workgroup's LDS with NaN first."""
    import os

    from gated_delta_rule_46_amd import build
    assert os.path.exists(build.POISON_LIB)
    with kda.using_library(build.POISON_LIB):
        for dtype in (BF16, F32):
            for d in (32, 64, 128):
                check(kda, make(1, 333, 2, 1, d, dtype, seed=d), 70, 3)
            test_decode_continues_a_prompt(kda, 4, 2, 64, 50, 2, dtype)
        test_decode_on_full_caches(kda, 3, 16, 4, 64, 1500, 0)


def test_a_hybrid_stack(kda):
    """The mixers together, as a model runs them: a prompt through a delta-rule
    layer, a linear-attention layer and a window layer, each fed the sum of the
    ones before, then one token through their states and cache; the step's output
    is what the whole sequence gives at its last token."""
    T, H, d, window, sinks = 200, 2, 64, 48, 2
    g = torch.Generator().manual_seed(11)
    rnd = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    W = [[rnd(d, d) / math.sqrt(d) for _ in range(3)] for _ in range(3)]
    x = rnd(1, T + 1, H, d)
    a = torch.sigmoid(3 + rnd(1, T + 1, H))
    beta = torch.sigmoid(rnd(1, T + 1, H))
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731

    def qkv(i, y):
        q, k, v = (torch.matmul(y, w) for w in W[i])
        return unit(q).contiguous(), unit(k).contiguous(), v.contiguous()

    def prompt(n):
        y = x[:, :n]
        q, k, v = qkv(0, y)
        o, S1 = kda.chunk_fwd(q, k, v, a[:, :n].contiguous(), beta[:, :n].contiguous())
        y = y + o
        q, k, v = qkv(1, y)
        o, S2 = kda.linattn_fwd(q, k, v, a[:, :n].contiguous())
        y = y + o
        q, k, v = qkv(2, y)
        o, _ = kda.swa_fwd(q, k, v, window=window, sinks=sinks)
        return y + o, S1, S2, k, v

    whole, *_ = prompt(T + 1)
    _, S1, S2, k, v = prompt(T)
    K, V = (torch.empty((1, window + sinks, H, d), device="cuda") for _ in range(2))
    kda.swa_cache_fill(k, v, K, V, window=window, sinks=sinks)
    y, an, bn = x[:, T].contiguous(), a[:, T].contiguous(), beta[:, T].contiguous()
    q, k, v = qkv(0, y)
    y = y + kda.decode_step(q, k, v, an, bn, S1)
    q, k, v = qkv(1, y)
    y = y + kda.linattn_decode_step(q, k, v, an, S2)
    q, k, v = qkv(2, y)
    y = y + kda.swa_decode_step(q, k, v, K, V, torch.tensor([T], dtype=torch.int32, device="cuda"), window=window,
                                sinks=sinks)
    err = (y - whole[:, T]).abs().max() / whole[:, T].square().mean().sqrt()
    assert err < 1e-4, err   # the delta rule's own bar for fp32 inputs
