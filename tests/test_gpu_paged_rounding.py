"""How exact attention over a paged cache is in bf16, and a rotation in fp32: what the
results are off by, next to the rounding of the results themselves."""
import pytest
import torch

from test_gpu_paged import BF16, F32, kda, make  # noqa: F401  (kda: the fixture)

pytestmark = pytest.mark.gpu


def definition(x, n, tokens):
    """o [tokens, Hq, d] of sequence n of a batch of causal tokens, in 64 bits."""
    q, Kp, Vp, table = x["q"][n].double(), x["Kp"].double(), x["Vp"].double(), x["table"].long()
    Hq, Hkv, d, page = q.shape[1], Kp.shape[2], q.shape[2], Kp.shape[1]
    L = int(x["ctx"][n]) + tokens
    pages = table[n, :(L + page - 1) // page]
    hidden = torch.zeros(tokens, L, dtype=torch.bool, device="cuda")
    hidden[:, L - tokens:] = torch.ones(tokens, tokens, dtype=torch.bool, device="cuda").triu(1)
    want = torch.empty(tokens, Hq, d, dtype=torch.float64, device="cuda")
    for h in range(Hq):
        K, V = (t[pages].flatten(0, 1)[:L, h // (Hq // Hkv)] for t in (Kp, Vp))
        s = (q[:, h] @ K.t().contiguous() * d ** -0.5).masked_fill(hidden, float("-inf"))
        want[:, h] = torch.softmax(s, -1) @ V
    return want


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("T,G", [(1, 4), (8, 4), (9, 4), (16, 4), (17, 4), (70, 3)])
def test_rows_of_every_block_are_as_exact(kda, T, G, d):  # noqa: F811
    """Blocks of 16, 32, 64 and 128 rows: a token is not less exact for the tokens beside it.
    A probability enters the second product as two bf16 numbers, of which the first takes the
    upper half of its bits (what is left is under 2^-7 of it) and the second rounds the rest
    (2^-8 of that): off by 2^-15 at most, a 64th of the result's own 2^-9 in the mean, so that
    the two together are 1.0002 times the result's own. Scores are sums in fp32. 1.02 leaves
    room for neither of the two numbers alone (1.4 times)."""
    x = make([T] * 2, [2000, 700], 2 * G, 2, d, BF16, 16, packed=False, seed=T + d)
    o, _ = kda.paged_attn(x["q"], x["Kp"], x["Vp"], x["table"], x["ctx"])
    off, own = 0.0, 0.0
    for n in range(2):
        want = definition(x, n, T)
        off += (o[n].double() - want).square().sum().item()
        own += (want.to(BF16).double() - want).square().sum().item()
    ratio = (off / own) ** 0.5
    assert ratio <= 1.02, "%.3f times the rounding of the result" % ratio


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("longest", [100, 10 ** 4, 2 * 10 ** 6])
def test_cosines_and_sines_in_fp32(kda, longest, interleaved):  # noqa: F811
    """Pairs (1, 0) rotated are the cosine and the sine themselves. Each is off by one unit of
    sincospif's (2^-24 below one) and half a unit of the joint with the rest of the angle, 1.5 x
    2^-24 in all; an angle rounded to fp32 first (up to 2^-25 of a half turn, pi 2^-25) would put
    it off by 1.57 more."""
    T, d, page = 65536, 32, 64
    k = torch.zeros(1, T, 1, d, device="cuda")
    one = slice(0, d, 2) if interleaved else slice(0, d // 2)
    k[..., one] = 1
    pages = [torch.zeros(T // page, page, 1, d, device="cuda") for _ in range(2)]
    table = torch.arange(T // page, dtype=torch.int32, device="cuda")[None]
    ctx = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(longest)
    pos = torch.randint(0, longest, (1, T), generator=g).to(torch.int32).cuda()
    freqs = (10000.0 ** (-torch.arange(d // 2) / (d // 2))).to(F32).cuda()
    q = kda.paged_append(k, k, *pages, table, ctx, q=k, pos=pos, freqs=freqs, interleaved=interleaved)[0, :, 0]
    angle = pos[0].double()[:, None] * freqs.double()
    other = slice(1, d, 2) if interleaved else slice(d // 2, d)
    for got, want in ((q[:, one], angle.cos()), (q[:, other], angle.sin())):
        worst = (got.double() - want).abs().max().item() * 2 ** 24
        assert worst <= 1.5, "off by %.3f of 2^-24" % worst
