"""Linear attention and window attention on packed batches of very uneven
sequences: work is numbered over the whole batch, so a long sequence next to many
short ones is where those numbers can go wrong."""
import pytest
import torch

import test_gpu_linattn as lin
import test_gpu_swa as swa
from mixer_checks import close
from oracle import mixers

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
kda = swa.kda   # the fixture

UNEVEN = [[900, 1, 0, 65, 300, 334], [0, 1, 2, 1500, 0, 97], [5] * 60 + [1000] + [31] * 9, [256, 256, 512, 128, 448]]


def term_sizes(x):
    """Per element of o, dq, dk and dv the root of its terms' summed squares, a term
    being one pair of tokens' or one row's of a boundary state. With 16 channels a
    single score can be near one, and meet a row of dO of four times its rms: that
    one product's rounding, up to 2^-8 of it, is then 2^-8 * 4 rms = 0.016 rms by
    itself, and no sum of many small ones. Held to its own size instead."""
    q, k, v, dO = (x[n][0].double().transpose(0, 1).contiguous() for n in ("q", "k", "v", "dO"))   # [H, T, .]
    a = x["gate"][0].double().T.contiguous()
    size = {n: torch.zeros_like(t) for n, t in (("o", v), ("dq", q), ("dk", k), ("dv", v))}
    sq = lambda t: t * t  # noqa: E731
    flip = lambda t: t.transpose(1, 2).contiguous()  # noqa: E731
    for s, (_, t0, t1) in enumerate(x["seqs"]):
        n = t1 - t0
        if n == 0:
            continue
        al, qs, ks, vs, gs = (t[:, t0:t1].contiguous() for t in (a, q, k, v, dO))
        D = torch.zeros(len(q), n, n, dtype=torch.float64, device=q.device)   # D[i, j] = a_{j+1} .. a_i
        for i in range(n):
            if i:
                D[:, i] = D[:, i - 1] * al[:, i, None]
            D[:, i, i] = 1.0
        P, B = sq(D * (qs @ flip(ks))), sq(D * (gs @ flip(vs)))
        first = sq(D[:, :, 0] * al[:, :1])[:, :, None]   # decays from before the first token
        last = sq(D[:, n - 1])[:, :, None]               # and to behind the last one
        S0, E = sq(x["S0"][s].double()), sq(x["dS_T"][s].double())
        for m, y in (("o", P @ sq(vs) + first * (sq(qs) @ S0)), ("dq", B @ sq(ks) + first * (sq(gs) @ flip(S0))),
                     ("dk", flip(B) @ sq(qs) + last * (sq(vs) @ flip(E))),
                     ("dv", flip(P) @ sq(gs) + last * (sq(ks) @ E))):
            size[m][:, t0:t1] = y.sqrt()
    return {m: y.transpose(0, 1)[None] for m, y in size.items()}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", UNEVEN)
def test_linear_packed(kda, lens, dtype):
    """64 heads: segments of several blocks, most sequences shorter than one."""
    x = lin.make(1, 0, 64, 16, 16, dtype, "signed", lens=lens, seed=sum(lens))
    args = (x["q"], x["k"], x["v"], x["gate"])
    o, S_T = kda.linattn_fwd(*args, S0=x["S0"], cu_seqlens=x["cu"])
    g = kda.linattn_bwd(*args, x["dO"], S0=x["S0"], dS_T=x["dS_T"], cu_seqlens=x["cu"])
    torch.cuda.synchronize()
    ro, rS, _ = mixers.linattn(*args, x["S0"], x["seqs"])
    r = mixers.linattn_grad(*args, x["dO"], x["S0"], x["dS_T"], x["seqs"])
    size = term_sizes(x)
    close("o", o, ro, dtype, size=size["o"])
    close("S_T", S_T, rS, dtype)
    for n in ("dq", "dk", "dv", "dgate", "dS0"):
        close(n, g[n], r[n], dtype, size=size.get(n))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (6, 2)])   # one head a group, and several
@pytest.mark.parametrize("window,sinks", [(20, 3), (1, 70), (130, 64), (40, 0)])
@pytest.mark.parametrize("lens", UNEVEN)
def test_window_packed(kda, lens, window, sinks, Hq, Hkv, dtype):
    swa.check(kda, swa.make(1, 0, Hq, Hkv, 32, dtype, lens=lens, seed=sum(lens)), window, sinks)


def test_window_many_workgroups(kda):
    """Enough key blocks and kv heads that a group's heads stay together, with the
    far rows of blocks with sinks in parts."""
    swa.check(kda, swa.make(2, 1100, 48, 24, 32, BF16, seed=1), 30, 4)
    swa.check(kda, swa.make(1, 0, 64, 32, 32, BF16, lens=[1200, 3, 0, 500, 400], seed=2), 30, 100)


def test_workspaces_hold_nothing_over(kda):
    """Workspaces full of NaN, exactly as large as asked for, give the same bits, and
    nothing behind them is written."""
    lens = [900, 1, 0, 65, 300]
    x = swa.make(1, 0, 4, 2, 64, BF16, lens=lens, seed=3)
    kw = dict(window=40, sinks=5, cu_seqlens=x["cu"])
    o, lse = kda.swa_fwd(x["q"], x["k"], x["v"], **kw)
    T = sum(lens)

    def guarded(need):
        w = torch.full((need // 4 + 1024,), float("nan"), device="cuda")
        return w, w.view(torch.uint8)[:need]

    g = kda.swa_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], **kw)
    whole, ws = guarded(kda.swa_bwd_workspace_bytes(1, 4, 2, T, 64, 40, 5, N=len(lens), varlen=True))
    g2 = kda.swa_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], workspace=ws, **kw)
    for n in g:
        assert torch.equal(g[n], g2[n]), n
    assert whole[ws.numel() // 4:].isnan().all()

    y = lin.make(1, 0, 64, 16, 32, BF16, lens=lens, seed=4)
    args = (y["q"], y["k"], y["v"], y["gate"])
    g = kda.linattn_bwd(*args, y["dO"], S0=y["S0"], cu_seqlens=y["cu"])
    whole, ws = guarded(kda.linattn_bwd_workspace_bytes(1, 64, T, 16, 32, N=len(lens), varlen=True))
    g2 = kda.linattn_bwd(*args, y["dO"], S0=y["S0"], cu_seqlens=y["cu"], workspace=ws)
    for n in g:
        assert torch.equal(g[n], g2[n]), n
    assert whole[ws.numel() // 4:].isnan().all()
    o, S = kda.linattn_fwd(*args, S0=y["S0"], cu_seqlens=y["cu"])
    whole, ws = guarded(kda.linattn_fwd_workspace_bytes(1, 64, T, 16, 32, N=len(lens), varlen=True))
    o2, S2 = kda.linattn_fwd(*args, S0=y["S0"], cu_seqlens=y["cu"], workspace=ws)
    assert torch.equal(o, o2) and torch.equal(S, S2) and whole[ws.numel() // 4:].isnan().all()


def test_fill_of_a_prompt_shorter_and_longer_than_the_cache(kda):
    for T, window, sinks in ((1, 50, 3), (53, 50, 3), (54, 50, 3), (700, 50, 3), (700, 1, 0), (20, 5, 30), (7, 1000, 0)):
        g = torch.Generator().manual_seed(T)
        k, v = (torch.randn((2, T, 2, 32), generator=g).to(BF16).cuda() for _ in range(2))
        K, V = (torch.full((2, window + sinks, 2, 32), 7.0, dtype=BF16, device="cuda") for _ in range(2))
        wk, wv = K.clone(), V.clone()
        for p in range(T):
            s = p if p < sinks else sinks + (p - sinks) % window
            wk[:, s], wv[:, s] = k[:, p], v[:, p]
        kda.swa_cache_fill(k, v, K, V, window=window, sinks=sinks)
        assert torch.equal(K, wk) and torch.equal(V, wv), (T, window, sinks)
