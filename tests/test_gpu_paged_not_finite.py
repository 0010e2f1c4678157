"""Values that are not finite in rows of a paged cache that some of a block's rows see and
others do not, in blocks of every number of rows, by themselves and with keys shared out."""
import pytest
import torch

from mixer_checks import close
from oracle import recur_paged as ref
from test_gpu_paged import BF16, F32, attend, kda, make  # noqa: F401  (kda: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T", [8, 16, 30, 60])
@pytest.mark.parametrize("ctx", [[7, 101], [7, 3000]])
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_rows_that_see_it_and_rows_that_do_not(kda, kind, ctx, T, bad, dtype):  # noqa: F811
    """2 T rows a kv head: blocks of 16, 32, 64 and 128. A draft of the second sequence has NaN in
    its key for kv head 0 and `bad` in its values for both; so has every page that nothing names.
    o and lse of rows that do not see the draft are as the definition says; of those that do, lse
    for kv head 1 is, lse for kv head 0 is not finite, and o is not."""
    x = make([T, T], ctx, 4, 2, 64, dtype, 16, tree=kind, packed=False, seed=T + len(kind))
    used = torch.zeros(x["Kp"].shape[0] * 16, dtype=torch.bool)
    for n in range(2):
        for r in range(ctx[n] + T):
            used[ref.place(x["table"].cpu(), n, r, 16, len(x["Kp"]))] = True
    for name in ("Kp", "Vp"):
        x[name].view(-1, 2, 64)[~used.cuda()] = bad
    j = 2
    at = ref.place(x["table"].cpu(), 1, ctx[1] + j, 16, len(x["Kp"]))
    x["Vp"].view(-1, 2, 64)[at] = bad
    x["Kp"].view(-1, 2, 64)[at, 0, :3] = float("nan")
    o, lse = (t.cpu() for t in attend(kda, x))
    cpu = {n: t.cpu() if torch.is_tensor(t) else t for n, t in x.items()}
    ro, rl, size, bound = ref.paged_attn(cpu["q"], cpu["Kp"], cpu["Vp"], cpu["table"], cpu["ctx"], cpu["tree"], 0.125, x["seqs"])
    sees = torch.zeros(2, T, dtype=torch.bool)
    sees[1] = torch.tensor([ref.sees(row, i, j) for i, row in enumerate(cpu["tree"][1])])
    assert sees.any() and not sees[1].all()
    close("o", o[~sees], ro[~sees], dtype, size=size[~sees])
    assert not torch.isfinite(o[sees]).any()
    good = torch.isfinite(rl)
    assert not good[sees][:, :2].any() and good[sees][:, 2:].all() and good[~sees].all()
    assert torch.equal(torch.isfinite(lse), good)
    assert ((lse.double() - rl).abs() <= bound)[good].all()
