"""A paged cache at the limits of launches: more tokens than one has waves, and no more
workgroups to share the keys than the chip holds at once."""
import pytest
import torch

from test_gpu_paged import BF16, F32, check, kda, make  # noqa: F401  (kda: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[2 ** 26 + 1001], [2 ** 26 - 3, 5, 0, 999]])
def test_more_tokens_than_a_launch_has_waves(kda, lens):  # noqa: F811
    """2^26 tokens are 2^32 threads. All rows arrive; rotated ones are those of small calls."""
    T, N, d, page = sum(lens), len(lens), 32, 4096
    need = [(n + page - 1) // page for n in lens]
    k, v, q = (torch.empty(1, T, 1, d, dtype=BF16, device="cuda").normal_() for _ in range(3))
    pools = [torch.zeros(sum(need), page, 1, d, dtype=BF16, device="cuda") for _ in range(2)]
    table = torch.full((N, max(need)), -1, dtype=torch.int32, device="cuda")
    last = sum(need)
    for n in range(N):   # pages in falling order
        table[n, :need[n]] = torch.arange(last - 1, last - need[n] - 1, -1, dtype=torch.int32, device="cuda")
        last -= need[n]
    ctx = torch.zeros(N, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + lens).cumsum(0)
    freqs = (10000.0 ** (-torch.arange(8) / 8)).to(F32).cuda()
    out = kda.paged_append(k, v, *pools, table, ctx, q=q, freqs=freqs, cu_seqlens=cu.to(torch.int32).cuda() if N > 1 else None)
    torch.cuda.synchronize()

    def rows(pool, n, first, end):
        """Rows first .. end of a sequence as they lie in the cache."""
        pages = pool[table[n, first // page:(end + page - 1) // page].long()].flatten(0, 1)
        return pages[first % page:first % page + end - first]

    for n in range(N):
        t0, most = int(cu[n]), 2 ** 23
        for first in range(0, lens[n], most):   # bit for bit what is not rotated
            end = min(first + most, lens[n])
            assert torch.equal(rows(pools[1], n, first, end), v[0, t0 + first:t0 + end])
            assert torch.equal(rows(pools[0], n, first, end)[..., 16:], k[0, t0 + first:t0 + end, :, 16:])
        for first in sorted({0, max(0, lens[n] - 3000)}):
            end = min(first + 3000, lens[n])
            if end == first:
                continue
            some = slice(t0 + first, t0 + end)
            small = [torch.zeros(1, end - first, 1, d, dtype=BF16, device="cuda") for _ in range(2)]
            pos = torch.arange(first, end, dtype=torch.int32, device="cuda")[None]
            want = kda.paged_append(k[:, some], v[:, some], *small, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                                    ctx[:1], q=q[:, some], pos=pos, freqs=freqs)
            assert torch.equal(out[:, some], want) and torch.equal(rows(pools[0], n, first, end), small[0][0])


@pytest.mark.parametrize("dtype,d,T,wgs", [(F32, 128, 16, 256), (F32, 64, 16, 512), (BF16, 128, 16, 512), (F32, 128, 32, 512),
                                           (F32, 128, 4, 256), (BF16, 64, 4, 256)])
def test_keys_are_shared_by_what_the_chip_holds(kda, dtype, d, T, wgs):  # noqa: F811
    """The first words of a workspace say for each kv head (up to 32 rows: for all that waves
    take side by side, here both) which workgroups have left parts of it. A workgroup of fp32 rows at 128 channels in blocks of 64 takes 135 KB of a CU's 160 KB of
    LDS: one a CU, 256 in all, where the others' are two. Results as ever."""
    x = make([T], [16384], 8, 2, d, dtype, 16, packed=False, seed=d)
    ws = torch.zeros(kda.paged_attn_workspace_bytes(1, T, 8, 2, d), dtype=torch.uint8, device="cuda")
    check(kda, x, workspace=ws)
    spans = ws[:16].view(torch.int32).tolist()
    if T * 4 <= 32:
        assert spans == [0, wgs - 1, 0, 0]
    else:
        assert spans[0] == 0 and spans[3] == wgs - 1 and all(s in (wgs // 2, wgs // 2 - 1) for s in spans[1:3])
