"""Linear attention with a decay per head (kda_linattn_*) against the
recurrence in 64 bits, on the GPU."""
import pytest
import torch

from mixer_checks import close
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


def make(B, T, H, dk, dv, dtype=BF16, gate="token", lens=None, states=True, seed=0):
    """Inputs. gate: "token" in (0, 1), "signed" with zeros, -0.0, negatives and
    exact ones, "head" one constant per head."""
    g = torch.Generator().manual_seed(seed)

    def rnd(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)

    if lens is not None:
        B, T = 1, sum(lens)
    N = B if lens is None else len(lens)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=unit(rnd(B, T, H, dk)).to(dtype), k=unit(rnd(B, T, H, dk)).to(dtype), v=rnd(B, T, H, dv).to(dtype),
             dO=rnd(B, T, H, dv).to(dtype))
    if gate == "head":
        x["gate"] = (1 - 2.0 ** -(1 + 6 * torch.rand(H, generator=g, dtype=torch.float64))).float()
    else:
        a = torch.sigmoid(3 + rnd(B, T, H))
        if gate == "signed":
            u = torch.rand((B, T, H), generator=g)
            a = torch.where(u < 0.3, -a, a)
            a = torch.where((u >= 0.30) & (u < 0.34), torch.zeros_like(a), a)
            a = torch.where((u >= 0.34) & (u < 0.36), torch.full_like(a, -0.0), a)
            a = torch.where((u >= 0.36) & (u < 0.40), torch.ones_like(a), a)
            a = torch.where((u >= 0.40) & (u < 0.42), torch.full_like(a, -1.0), a)
            a = torch.where((u >= 0.42) & (u < 0.44), torch.full_like(a, 1e-6), a)
        x["gate"] = a.to(dtype)
    x["S0"] = 0.3 * rnd(N, H, dk, dv).float() if states else None
    x["dS_T"] = 0.3 * rnd(N, H, dk, dv).float() if states else None
    cu = None
    if lens is not None:
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    x = {n: t.cuda() if t is not None else None for n, t in x.items()}
    x["cu"] = cu.cuda() if cu is not None else None
    x["seqs"] = mixers.spans(B, T, cu)
    print("case B", B, "T", T, "H", H, "dk", dk, "dv", dv, dtype, gate, "lens", lens, "states", states, flush=True)
    return x


def check_fwd(kda, x, **kw):
    o, S_T = kda.linattn_fwd(x["q"], x["k"], x["v"], x["gate"], S0=x["S0"], cu_seqlens=x["cu"], **kw)
    torch.cuda.synchronize()
    ro, rS, _ = mixers.linattn(x["q"], x["k"], x["v"], x["gate"], x["S0"], x["seqs"])
    dt = x["q"].dtype
    assert o.dtype == dt and S_T.dtype == F32
    close("o", o, ro, dt)
    close("S_T", S_T, rS, dt)


def check_bwd(kda, x):
    g = kda.linattn_bwd(x["q"], x["k"], x["v"], x["gate"], x["dO"], S0=x["S0"], dS_T=x["dS_T"], cu_seqlens=x["cu"])
    torch.cuda.synchronize()
    r = mixers.linattn_grad(x["q"], x["k"], x["v"], x["gate"], x["dO"], x["S0"], x["dS_T"], x["seqs"])
    dt = x["q"].dtype
    for n in ("dq", "dk", "dv", "dgate", "dS0"):
        if n == "dgate" and x["gate"].dim() == 1:
            assert g[n] is None
            continue
        close(n, g[n], r[n], dt)


SIZES = [
    # B, T, H, dk, dv
    (1, 1, 1, 16, 16), (2, 2, 3, 64, 64), (1, 63, 2, 128, 128), (1, 64, 2, 128, 64), (1, 65, 1, 32, 128),
    (2, 129, 2, 128, 128), (1, 257, 3, 64, 128), (1, 300, 2, 128, 16), (3, 513, 1, 16, 64), (1, 700, 2, 32, 32),
]
KINDS = [(BF16, "token"), (BF16, "signed"), (BF16, "head"), (F32, "token"), (F32, "signed"), (F32, "head")]


@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("B,T,H,dk,dv", SIZES)
def test_forward(kda, B, T, H, dk, dv, dtype, gate):
    check_fwd(kda, make(B, T, H, dk, dv, dtype, gate, states=T % 2 == 1, seed=T))


@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("B,T,H,dk,dv", SIZES)
def test_backward(kda, B, T, H, dk, dv, dtype, gate):
    check_bwd(kda, make(B, T, H, dk, dv, dtype, gate, states=T % 2 == 1, seed=T + 1))


@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_every_head_size(kda, dk, dv, dtype):
    x = make(1, 150, 2, dk, dv, dtype, "signed", seed=dk + dv)
    check_fwd(kda, x)
    check_bwd(kda, x)


LENS = [[5, 1, 0, 64, 70], [0, 0, 1], [128, 128, 1, 200], [0, 333, 0], [1, 2, 3, 4, 5, 6, 7], [700, 63, 0, 65]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", LENS)
def test_packed(kda, lens, dtype):
    x = make(1, 0, 2, 64, 128, dtype, "signed", lens=lens, seed=sum(lens))
    check_fwd(kda, x)
    check_bwd(kda, x)


def test_long(kda):
    x = make(1, 2500, 1, 128, 128, BF16, "token", seed=4)
    check_fwd(kda, x)
    check_bwd(kda, x)


def test_no_tokens(kda):
    for dtype in (BF16, F32):
        x = make(2, 0, 2, 32, 64, dtype)
        o, S_T = kda.linattn_fwd(x["q"], x["k"], x["v"], x["gate"], S0=x["S0"])
        assert o.numel() == 0 and torch.equal(S_T, x["S0"])
        g = kda.linattn_bwd(x["q"], x["k"], x["v"], x["gate"], x["dO"], S0=x["S0"], dS_T=x["dS_T"])
        assert torch.equal(g["dS0"], x["dS_T"])


def test_rows_behind_the_last_sequence(kda):
    for T, lens in ((200, [70, 50]), (900, [300, 411])):
        x = make(1, T, 2, 64, 64)
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
        x["S0"] = x["dS_T"] = None
        x["seqs"] = mixers.spans(1, T, cu)
        out = torch.full_like(x["v"], 7.0)
        kda.linattn_fwd(x["q"], x["k"], x["v"], x["gate"], cu_seqlens=cu, out=out)
        ro, _, _ = mixers.linattn(x["q"], x["k"], x["v"], x["gate"], None, x["seqs"])
        n = sum(lens)
        close("o", out[:, :n], ro[:, :n], BF16)
        assert (out[:, n:] == 7.0).all()
        g = {m: torch.full_like(x[s], 7.0) for m, s in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dgate", "gate"))}
        kda.linattn_bwd(x["q"], x["k"], x["v"], x["gate"], x["dO"], cu_seqlens=cu, out=g)
        r = mixers.linattn_grad(x["q"], x["k"], x["v"], x["gate"], x["dO"], None, None, x["seqs"])
        for m in g:
            close(m, g[m][:, :n], r[m][:, :n], BF16)
            assert (g[m][:, n:] == 7.0).all()


def test_state_carries_over(kda):
    """A sequence in two calls, then single steps, is the sequence in one."""
    x = make(1, 600, 2, 128, 128, BF16, "token", seed=8)
    cut = 333
    part = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    _, S = kda.linattn_fwd(*(part(x[n], 0, cut) for n in ("q", "k", "v", "gate")), S0=x["S0"])
    outs = []
    o2, S = kda.linattn_fwd(*(part(x[n], cut, 590) for n in ("q", "k", "v", "gate")), S0=S, S_T=S)   # in place
    for t in range(590, 600):
        outs.append(kda.linattn_decode_step(*(x[n][:, t].contiguous() for n in ("q", "k", "v", "gate")), S))
    ro, rS, _ = mixers.linattn(x["q"], x["k"], x["v"], x["gate"], x["S0"], x["seqs"])
    close("o", torch.cat([o2, torch.stack(outs, 1)], 1), ro[:, cut:], BF16)
    close("S", S, rS, BF16)


@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("N,H,dk,dv", [(1, 1, 16, 16), (3, 5, 32, 128), (1, 16, 128, 128), (2, 3, 128, 64), (7, 2, 64, 32),
                                       (40, 16, 128, 128), (130, 4, 64, 64), (5, 1, 16, 128)])
def test_decode(kda, N, H, dk, dv, dtype, gate):
    x = make(N, 1, H, dk, dv, dtype, gate, seed=N)
    S = x["S0"].clone()
    one = lambda n: x[n][:, 0].contiguous()  # noqa: E731
    o = kda.linattn_decode_step(one("q"), one("k"), one("v"), x["gate"] if gate == "head" else one("gate"), S)
    ro, rS, _ = mixers.linattn(x["q"], x["k"], x["v"], x["gate"], x["S0"], x["seqs"])
    close("o", o, ro[:, 0], dtype)
    close("S", S, rS, F32)


def test_gradient_against_differences(kda):
    """The kernel's gradient against central differences of the recurrence in
    64 bits: L is linear in every single input entry, so they are exact."""
    x = make(1, 37, 1, 16, 16, F32, "signed", seed=3)
    g = kda.linattn_bwd(x["q"], x["k"], x["v"], x["gate"], x["dO"], S0=x["S0"], dS_T=x["dS_T"])

    def loss(y):
        o, S, _ = mixers.linattn(y["q"], y["k"], y["v"], y["gate"], y["S0"], x["seqs"])
        return (o * x["dO"].double()).sum() + (S * x["dS_T"].double()).sum()

    rng = torch.Generator().manual_seed(1)
    for name, gname in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("gate", "dgate"), ("S0", "dS0")):
        rms = g[gname].double().square().mean().sqrt().item()
        for e in torch.randint(0, x[name].numel(), (12,), generator=rng).tolist():
            d = []
            for sign in (1, -1):
                y = {n: x[n].double() for n in ("q", "k", "v", "gate", "S0")}
                y[name] = y[name].clone()
                y[name].view(-1)[e] += sign * 0.5
                d.append(loss(y).item())
            got = g[gname].view(-1)[e].item()
            assert abs(got - (d[0] - d[1])) <= 2e-5 * max(rms, abs(got)), (name, e)


def test_repeats_and_streams(kda):
    x = make(2, 700, 3, 64, 128, BF16, "token", seed=2)
    args = (x["q"], x["k"], x["v"], x["gate"])
    o, S = kda.linattn_fwd(*args, S0=x["S0"])
    g = kda.linattn_bwd(*args, x["dO"], S0=x["S0"], dS_T=x["dS_T"])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o2, S2 = kda.linattn_fwd(*args, S0=x["S0"], stream=st)
    g2 = kda.linattn_bwd(*args, x["dO"], S0=x["S0"], dS_T=x["dS_T"], stream=st)
    with torch.cuda.stream(st):
        o3, _ = kda.linattn_fwd(*args, S0=x["S0"])
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S2) and torch.equal(o, o3)
    for n in g:
        assert torch.equal(g[n], g2[n]), n


def test_graph_replays(kda):
    """Forward, gradient and a step in one captured graph, on new inputs and a new
    split of the packed batch each time, against eager calls, bit for bit."""
    splits = ([300, 0, 155, 90], [1, 2, 270, 272], [545, 0, 0, 0])
    xs = [make(1, 0, 2, 64, 64, BF16, "signed", lens=s, seed=20 + i) for i, s in enumerate(splits)]
    cur = {n: t.clone() for n, t in xs[0].items() if isinstance(t, torch.Tensor)}
    step = lambda n: cur[n][0, :4].contiguous()  # noqa: E731

    def work(S):
        args = (cur["q"], cur["k"], cur["v"], cur["gate"])
        o, S_T = kda.linattn_fwd(*args, S0=cur["S0"], cu_seqlens=cur["cu"])
        g = kda.linattn_bwd(*args, cur["dO"], S0=cur["S0"], dS_T=cur["dS_T"], cu_seqlens=cur["cu"])
        S.copy_(S_T)
        y = kda.linattn_decode_step(step("q"), step("k"), step("v"), step("gate"), S)
        return [o, S_T, S, y] + [g[n] for n in ("dq", "dk", "dv", "dgate", "dS0")]

    S = torch.empty_like(cur["S0"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(S)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work(S)
    for x in xs + xs[:1]:
        for n in cur:
            cur[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = work(torch.empty_like(S))
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
            for dk, dv in ((16, 16), (128, 128), (16, 128), (128, 16)):
                for T in (77, 300):
                    x = make(1, T, 2, dk, dv, dtype, "signed", seed=T)
                    check_fwd(kda, x)
                    check_bwd(kda, x)
        x = make(3, 1, 2, 128, 64)
        S = x["S0"].clone()
        o = kda.linattn_decode_step(*(x[n][:, 0].contiguous() for n in ("q", "k", "v", "gate")), S)
        ro, rS, _ = mixers.linattn(x["q"], x["k"], x["v"], x["gate"], x["S0"], x["seqs"])
        close("o", o, ro[:, 0], BF16)
        close("S", S, rS, F32)
