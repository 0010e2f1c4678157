"""The recurrence in the plans that large batches take: which kernel runs, read off the names of
those that ran, and its results against the definition in 64 bits, a channel here and there."""
import pytest
import torch

from oracle import recur_paged as ref
from test_gpu_glr import BF16, F32, TYPES, kda, make, within  # noqa: F401  (kda: the fixture)

pytestmark = pytest.mark.gpu


def kernels(call):
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        call()
        torch.cuda.synchronize()
    return " ".join(e.name for e in prof.events())


def large(B, T, C, x_type, gate_type, seed=0):
    """As make, drawn on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gate = 1 - 0.1 * torch.rand(B, T, C, generator=g, device="cuda")
    return dict(gate=gate.to(gate_type), x=rnd(B, T, C).to(x_type), h0=rnd(B, C), cu=None, seqs=[(b, 0, T) for b in range(B)])


@pytest.mark.parametrize("types,B,T,C,stream", [
    ((BF16, BF16), 16, 700, 2048, True), ((BF16, F32), 16, 700, 2048, True), ((F32, F32), 8, 700, 2048, True),
    ((BF16, F32), 4, 700, 2048, False), ((F32, F32), 16, 1024, 2048, True), ((F32, F32), 16, 1025, 2048, False),
    ((BF16, F32), 32, 193, 1024, True), ((BF16, F32), 32, 192, 1024, False), ((BF16, F32), 256, 300, 7, True)])
def test_forward_of_large_batches(kda, types, B, T, C, stream):  # noqa: F811
    """Either side of 256 pairs, of 2^25 values in fp32 and of a single block; fp32 decays beside
    bf16 x in the streaming kernel's shorter blocks."""
    x = large(B, T, C, *types, seed=T)
    out = []
    ran = kernels(lambda: out.append(kda.glr_fwd(x["gate"], x["x"], h0=x["h0"])))
    assert ("glr_stream_kernel" in ran) == stream and ("glr_pass_kernel" in ran) != stream
    h, h_T = out[0]
    some = torch.arange(0, C, max(1, C // 13))
    rows = torch.arange(0, B, max(1, B // 5))
    cut = lambda t: t[rows.cuda()][..., some.cuda()].cpu()  # noqa: E731
    want, want_T, _, bound, bound_T = ref.glr(cut(x["gate"]), cut(x["x"]), cut(x["h0"]), [(b, 0, T) for b in range(len(rows))])
    within("h", cut(h), want, bound)
    within("h_T", cut(h_T), want_T, bound_T)


def check_forward(kda, x):
    h, h_T = kda.glr_fwd(x["gate"], x["x"], h0=x["h0"], cu_seqlens=x["cu"])
    want, want_T, _, bound, bound_T = ref.glr(x["gate"].cpu(), x["x"].cpu(), x["h0"].cpu(), x["seqs"])
    within("h", h.cpu(), want, bound)
    within("h_T", h_T.cpu(), want_T, bound_T)


def lasting(x, seed=0):
    """Decays of one but for a hundredth of the tokens (2^-8 less) and signs at random, and one
    x in 500: a state carries over thousands of tokens as the largest part of what comes later,
    and its bound (two roundings a token of the terms in it) stays below a hundredth of it."""
    g = torch.Generator().manual_seed(seed)
    u, v, w = (torch.rand(x["x"].shape, generator=g) for _ in range(3))
    gate = torch.where(u < 0.01, 1 - 2.0 ** -8, 1.0) * torch.where(v < 0.1, -1.0, 1.0)
    x["gate"].copy_(gate)
    x["x"].mul_((w < 0.002).to(x["x"].device))
    return x


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("C", [8, 4, 3])
@pytest.mark.parametrize("T", [256 * 65 + 3, 256 * 97])
def test_states_that_come_from_states(kda, T, C, types):  # noqa: F811
    """Every 32nd block of 192 or 256 tokens leaves a state, from the second such on formed from
    the one before: sequences of more than 64 and 96 blocks, in every layout."""
    check_forward(kda, make(1, T, C, *types, seed=C))
    check_forward(kda, lasting(make(1, T, C, *types, seed=C)))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("C", [8, 3])
def test_states_that_come_from_states_packed(kda, C, types):  # noqa: F811
    """The same behind other sequences and before some, so that neither its first token nor its
    first block is a multiple of anything."""
    lens = [77, 0, 1, 256 * 65 + 3, 300, 0, 256 * 33, 5]
    check_forward(kda, make(1, 0, C, *types, lens=lens, seed=C, kind="signed"))
    check_forward(kda, lasting(make(1, 0, C, *types, lens=lens, seed=C)))
