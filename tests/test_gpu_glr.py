"""The gated linear recurrence on the GPU against its definition in 64 bits.

Bars: an element is off by no more than the roundings on the way of its terms
(each 2^-24 of the term, counted by the oracle) and half a step of its type."""
import pytest
import torch

from oracle import mixers
from oracle import recur_paged as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
TYPES = [(BF16, BF16), (BF16, F32), (F32, F32)]


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_46_amd import kda as k
    k.library()
    return k


def within(name, x, want, bound):
    assert x.shape == want.shape, name
    if x.numel() == 0:
        return
    assert torch.isfinite(x).all(), "%s is not finite" % name
    off = (x.double() - want).abs()
    room = (1 + STEP[x.dtype]) * bound * 2.0 ** -24 + STEP[x.dtype] * want.abs() + 1e-36
    worst = (off / room).max().item()
    assert worst <= 1.0, "%s off by %.3g of its bound" % (name, worst)


def make(B, T, C, x_type, gate_type, kind="slow", lens=None, seed=0, states=True):
    g = torch.Generator().manual_seed(seed)
    cu = None
    if lens is not None:
        B, T = 1, sum(lens)
        cu = torch.tensor([0] + lens).cumsum(0)
    N = B if lens is None else len(lens)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    u = torch.rand(B, T, C, generator=g)
    gate = {"slow": 1 - 0.1 * u, "fast": u, "signed": 2 * u - 1, "zeros": torch.where(u < 0.3, torch.zeros(()), 1 - u / 50)}[kind]
    x = dict(gate=gate.to(gate_type), x=rnd(B, T, C).to(x_type), dh=rnd(B, T, C).to(x_type),
             h0=rnd(N, C) if states else None, dh_T=rnd(N, C) if states else None)
    x = {n: t if t is None else t.cuda() for n, t in x.items()}
    x["cu"] = None if cu is None else cu.to(torch.int32).cuda()
    x["seqs"] = mixers.spans(B, T, cu)
    return x


def check(kda, x, **kw):
    h, h_T = kda.glr_fwd(x["gate"], x["x"], h0=x["h0"], cu_seqlens=x["cu"], **kw)
    g = kda.glr_bwd(x["gate"], x["x"], x["dh"], h0=x["h0"], dh_T=x["dh_T"], cu_seqlens=x["cu"], **kw)
    torch.cuda.synchronize()
    want, want_T, _, bound, bound_T = ref.glr(x["gate"].cpu(), x["x"].cpu(), None if x["h0"] is None else x["h0"].cpu(), x["seqs"])
    cpu = {n: x[n] if x[n] is None else x[n].cpu() for n in ("gate", "x", "h0", "dh", "dh_T")}
    r, rb = ref.glr_grad(cpu["gate"], cpu["x"], cpu["h0"], cpu["dh"], cpu["dh_T"], x["seqs"])
    within("h", h.cpu(), want, bound)
    within("h_T", h_T.cpu(), want_T, bound_T)
    for n in ("dgate", "dx", "dh0"):
        within(n, g[n].cpu(), r[n], rb[n])
    assert h.dtype == x["x"].dtype and g["dgate"].dtype == x["gate"].dtype and g["dx"].dtype == x["x"].dtype


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T", [1, 2, 3, 63, 64, 65, 127, 128, 129, 300, 701])
@pytest.mark.parametrize("C", [8, 72])
def test_lengths(kda, T, C, types):
    check(kda, make(2, T, C, *types, seed=T))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("C", [1, 2, 4, 5, 12, 63, 64, 65, 128, 200, 333])
def test_channels(kda, C, types):
    check(kda, make(1, 150, C, *types, seed=C))
    check(kda, make(3, 70, C, *types, seed=C, states=False))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("kind", ["slow", "fast", "signed", "zeros"])
def test_decays(kda, kind, types):
    check(kda, make(2, 400, 40, *types, kind=kind))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("C", [24, 37])
@pytest.mark.parametrize("lens", [[0, 1, 2, 500, 0, 97], [5] * 60 + [300] + [31] * 9, [128, 128, 64, 256], [0], [0, 0, 3, 0]])
def test_packed(kda, lens, C, types):
    check(kda, make(1, 0, C, *types, lens=lens, seed=len(lens)))
    check(kda, make(1, 0, C, *types, lens=lens, seed=len(lens), states=False))


def test_no_tokens(kda):
    x = make(2, 0, 16, BF16, BF16)
    h, h_T = kda.glr_fwd(x["gate"], x["x"], h0=x["h0"])
    g = kda.glr_bwd(x["gate"], x["x"], x["dh"], h0=x["h0"], dh_T=x["dh_T"])
    assert h.shape == (2, 0, 16) and torch.equal(h_T, x["h0"]) and torch.equal(g["dh0"], x["dh_T"])


def test_many_blocks(kda):
    """A long sequence of few channels: a chain of many blocks."""
    check(kda, make(1, 5000, 3, F32, F32))
    check(kda, make(1, 5000, 8, BF16, F32))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("B,C,T", [(64, 512, 129), (9, 3700, 260), (256, 5, 300)])
def test_batches_that_fill_the_chip(kda, B, C, T, types):
    check(kda, make(B, T, C, *types, seed=C))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("C", [136, 7])
@pytest.mark.parametrize("T", [64 * 64, 64 * 64 + 1, 64 * 128, 64 * 128 + 3])
def test_around_the_longest_walk(kda, T, C, types):
    check(kda, make(1, T, C, *types, seed=T))


def test_packed_long_next_to_short(kda):
    lens = [3, 0, 5000, 1, 700, 0, 128, 64]
    check(kda, make(1, 0, 130, BF16, F32, lens=lens))
    check(kda, make(1, 0, 136, F32, F32, lens=lens, kind="signed"))
    check(kda, make(1, 0, 8, BF16, BF16, lens=[9000, 2, 0, 300]))


@pytest.mark.parametrize("types", TYPES)
def test_step_continues_the_forward(kda, types):
    x = make(3, 40, 56, *types, seed=5)
    _, h_T = kda.glr_fwd(x["gate"][:, :37].contiguous(), x["x"][:, :37].contiguous(), h0=x["h0"])
    state = h_T.clone()
    want, _, _, bound, _ = ref.glr(x["gate"].cpu(), x["x"].cpu(), x["h0"].cpu(), x["seqs"])
    for t in range(37, 40):
        o = kda.glr_decode_step(x["gate"][:, t].contiguous(), x["x"][:, t].contiguous(), state)
        within("o", o.cpu(), want[:, t], bound[:, t])
        within("state", state.cpu(), want[:, t], bound[:, t])


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("N,C", [(1, 1), (1, 8), (3, 5), (2, 1001), (64, 129)])
def test_step_sizes(kda, N, C, types):
    x = make(N, 1, C, *types, seed=C)
    state = x["h0"].clone()
    o = kda.glr_decode_step(x["gate"][:, 0], x["x"][:, 0], state)
    want = x["gate"][:, 0].double() * x["h0"].double() + x["x"][:, 0].double()
    within("state", state, want, want.abs())
    within("o", o, want, want.abs())


@pytest.mark.parametrize("B,T,C", [(2, 100, 64), (2, 200, 64), (1, 3000, 264), (1, 9000, 16), (130, 300, 256)])
def test_state_in_place_and_given_outputs(kda, B, T, C):
    """One block, blocks that form what enters them, a chain of blocks, one workgroup a sequence."""
    x = make(B, T, C, BF16, BF16)
    h, h_T = kda.glr_fwd(x["gate"], x["x"], h0=x["h0"])
    state, out = x["h0"].clone(), torch.empty_like(h)
    a, b = kda.glr_fwd(x["gate"], x["x"], h0=state, h_T=state, out=out)
    assert a is out and b is state and torch.equal(out, h) and torch.equal(state, h_T)
    assert kda.glr_fwd(x["gate"], x["x"], state_out=False)[1] is None
    g = kda.glr_bwd(x["gate"], x["x"], x["dh"], h0=x["h0"])
    given = {n: torch.full_like(t, 7.0) for n, t in g.items()}
    assert kda.glr_bwd(x["gate"], x["x"], x["dh"], h0=x["h0"], out=given) is given
    assert all(torch.equal(given[n], g[n]) for n in g)
    assert kda.glr_bwd(x["gate"], x["x"], x["dh"], want_dh0=False)["dh0"] is None


@pytest.mark.parametrize("C", [16, 5])
def test_rows_behind_the_last_sequence_stay(kda, C):
    x = make(1, 0, C, BF16, BF16, lens=[70, 3, 100])
    pad = lambda t, v: torch.cat([t, torch.full_like(t[:, :40], v)], 1)  # noqa: E731
    big = {n: pad(x[n], float("nan")) for n in ("gate", "x", "dh")}
    out = torch.full_like(big["x"], 3.0)
    g = {n: torch.full_like(big["x"], 3.0) for n in ("dgate", "dx")}
    kda.glr_fwd(big["gate"], big["x"], cu_seqlens=x["cu"], out=out)
    kda.glr_bwd(big["gate"], big["x"], big["dh"], cu_seqlens=x["cu"], out=g)
    h, _ = kda.glr_fwd(x["gate"], x["x"], cu_seqlens=x["cu"])
    r = kda.glr_bwd(x["gate"], x["x"], x["dh"], cu_seqlens=x["cu"])
    for a, b in ((out, h), (g["dgate"], r["dgate"]), (g["dx"], r["dx"])):
        assert torch.equal(a[:, :173], b) and (a[:, 173:] == 3.0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_values_stay_in_their_channel(kda, bad):
    x = make(2, 400, 24, BF16, F32)
    clean, _ = kda.glr_fwd(x["gate"], x["x"], h0=x["h0"])
    clean_g = kda.glr_bwd(x["gate"], x["x"], x["dh"], h0=x["h0"])
    x["x"][1, 150, 9] = bad
    h, h_T = kda.glr_fwd(x["gate"], x["x"], h0=x["h0"])
    g = kda.glr_bwd(x["gate"], x["x"], x["dh"], h0=x["h0"])
    hit = torch.zeros(2, 400, 24, dtype=torch.bool, device="cuda")
    hit[1, 150:, 9] = True
    assert torch.equal(h[~hit], clean[~hit]) and not torch.isfinite(h[hit]).any()
    assert not torch.isfinite(h_T[1, 9]) and torch.isfinite(h_T).sum() == h_T.numel() - 1
    assert torch.equal(g["dx"], clean_g["dx"])
    late = hit.clone()
    late[1, 150, 9] = False
    assert torch.equal(g["dgate"][~late], clean_g["dgate"][~late])


def test_repeats_and_streams_and_graph(kda):
    x = make(2, 700, 100, BF16, BF16)

    def both(**kw):
        h, h_T = kda.glr_fwd(x["gate"], x["x"], h0=x["h0"], **kw)
        g = kda.glr_bwd(x["gate"], x["x"], x["dh"], h0=x["h0"], dh_T=x["dh_T"], **kw)
        return [h, h_T, g["dgate"], g["dx"], g["dh0"]]

    want = both()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = both(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for _ in range(3):
        for t in held:
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        x["x"].mul_(0.5)
        x["x"].mul_(2.0)
    x["x"].neg_()
    want = both()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_calls_at_once(kda):
    """Two streams in turn, a workspace each, over sequences of many blocks."""
    xs = [make(1, 6000, 520, BF16, BF16, seed=i) for i in range(2)]
    args = [(x["gate"], x["x"]) for x in xs]
    want = [kda.glr_fwd(*a, h0=x["h0"]) for a, x in zip(args, xs)]
    side = [torch.cuda.Stream() for _ in xs]
    ws = [torch.empty(kda.glr_fwd_workspace_bytes(1, 6000, 520), dtype=torch.uint8, device="cuda") for _ in xs]
    outs = [[(torch.empty_like(x["x"]), torch.empty_like(x["h0"])) for _ in range(6)] for x in xs]
    torch.cuda.synchronize()
    for n in range(6):
        for i, x in enumerate(xs):
            kda.glr_fwd(*args[i], h0=x["h0"], out=outs[i][n][0], h_T=outs[i][n][1], workspace=ws[i], stream=side[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(h, want[i][0]) and torch.equal(h_T, want[i][1]) for h, h_T in outs[i])


def test_gradient_against_differences(kda):
    """Central differences of the loss in fp32 inputs, formed by the oracle in 64 bits
    so that only the step's own error (its square) is left."""
    x = make(1, 60, 5, F32, F32, kind="signed")
    g = kda.glr_bwd(x["gate"], x["x"], x["dh"], h0=x["h0"], dh_T=x["dh_T"])
    cpu = {n: x[n].double().cpu() for n in ("gate", "x", "h0", "dh", "dh_T")}

    def loss():
        h, h_T, *_ = ref.glr(cpu["gate"], cpu["x"], cpu["h0"], x["seqs"])
        return (h * cpu["dh"]).sum() + (h_T * cpu["dh_T"]).sum()

    pick = torch.Generator().manual_seed(1)
    for name, out in (("gate", "dgate"), ("x", "dx"), ("h0", "dh0")):
        flat = cpu[name].view(-1)
        for e in torch.randint(0, flat.numel(), (12,), generator=pick).tolist():
            keep, eps = flat[e].item(), 1e-4
            flat[e] = keep + eps
            up = loss()
            flat[e] = keep - eps
            slope = (up - loss()) / (2 * eps)
            flat[e] = keep
            # second-order term: eps^2 times third derivatives, which are zero in each input by itself
            assert abs(slope - g[out].view(-1)[e].item()) <= 1e-4 * (1 + abs(slope))


def test_poisoned_lds(kda):
    """The build that fills every workgroup's LDS with NaN first: every kernel."""
    import os

    from gated_delta_rule_46_amd import build
    assert os.path.exists(build.POISON_LIB)
    with kda.using_library(build.POISON_LIB):
        for types in TYPES:
            for C in (24, 5):
                check(kda, make(2, 100, C, *types))
                check(kda, make(1, 0, C, *types, lens=[700, 0, 3, 129]))
            check(kda, make(1, 64 * 128 + 3, 3, *types))
            test_step_sizes(kda, 3, 5, types)
        check(kda, make(130, 270, 256, BF16, BF16))
        test_no_tokens(kda)
