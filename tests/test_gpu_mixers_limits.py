"""Linear and window attention at the edges of the sizes that they accept."""
import math

import pytest
import torch

from mixer_checks import close
from oracle import mixers
from test_gpu_linattn import kda  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def test_linear_sixteen_million_states(kda):  # noqa: F811
    """2^20 packed sequences of 16 heads, three of them with tokens; more than 256 tokens,
    so that the states go through segments. 2^24 states, 17 GB of them and as much workspace."""
    N, H, d, lens = 2 ** 20, 16, 16, {0: 300, 2 ** 19: 401, 2 ** 20 - 1: 299}
    T = sum(lens.values())
    count = torch.zeros(N, dtype=torch.int32)
    for s, n in lens.items():
        count[s] = n
    cu = torch.cat([torch.zeros(1, dtype=torch.int32), count.cumsum(0).to(torch.int32)]).cuda()
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((1, T, H, d), generator=g).to(BF16).cuda() / 4 for _ in range(3))
    gate = torch.sigmoid(3 + torch.randn((1, T, H), generator=g)).to(BF16).cuda()
    S_T = torch.full((N, H, d, d), math.nan, device="cuda")
    o, _ = kda.linattn_fwd(q, k, v, gate, cu_seqlens=cu, S_T=S_T)
    ends = torch.tensor(list(lens.values())).cumsum(0).tolist()
    ro, rS, _ = mixers.linattn(q, k, v, gate, None, [(0, e - n, e) for e, n in zip(ends, lens.values())])
    close("o", o, ro, BF16)
    close("S_T", S_T[list(lens)], rS, BF16)
    S_T[list(lens)] = 0
    assert all((S_T[i:i + 2 ** 17] == 0).all() for i in range(0, N, 2 ** 17))
    del S_T
    torch.cuda.empty_cache()
