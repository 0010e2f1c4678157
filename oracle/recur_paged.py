"""The gated linear recurrence per channel, rows on their way into a paged cache,
and attention over such a cache, from their definitions in 64 bits, token by token
and row by row (torch, on any device). Test infrastructure only; shares no code
with the kernels.

Sequences are given as (row of the batch, first token, end), as in mixers.py."""
import math

import torch


def glr(gate, x, h0, seqs):
    """h [B,T,C], h_T [N,C], the states before each token, and for h and h_T how
    far rounding can carry them, in units of one rounding: every term a..a x of a
    state passes through no more than two roundings a token that it has been in
    it (its decays are multiplied up once, and the state formed once), and eight
    at the joints."""
    gate, x = gate.double(), x.double()
    N, C = len(seqs), x.shape[-1]
    h, before, bound = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    h_T, bound_T = (torch.zeros(N, C, dtype=torch.float64, device=x.device) for _ in range(2))
    for n, (b, t0, t1) in enumerate(seqs):
        s = torch.zeros(C, dtype=torch.float64, device=x.device) if h0 is None else h0[n].double()
        size, path = s.abs(), 8 * s.abs()
        for t in range(t0, t1):
            before[b, t] = s
            s = gate[b, t] * s + x[b, t]
            path = gate[b, t].abs() * (path + 2 * size) + 10 * x[b, t].abs()
            size = gate[b, t].abs() * size + x[b, t].abs()
            h[b, t], bound[b, t] = s, path
        h_T[n], bound_T[n] = s, path
    return h, h_T, before, bound, bound_T


def glr_grad(gate, x, h0, dh, dh_T, seqs):
    """dict of dgate, dx, dh0 and one of their bounds (as for glr)."""
    _, _, before, reach, _ = glr(gate, x, h0, seqs)
    gate, dh = gate.double(), dh.double()
    N, C = len(seqs), gate.shape[-1]
    out = {"dgate": torch.zeros_like(gate), "dx": torch.zeros_like(gate),
           "dh0": torch.zeros(N, C, dtype=torch.float64, device=gate.device)}
    bound = {n: torch.zeros_like(t) for n, t in out.items()}
    for n, (b, t0, t1) in enumerate(seqs):
        g = torch.zeros(C, dtype=torch.float64, device=gate.device) if dh_T is None else dh_T[n].double()
        size, path = g.abs(), 8 * g.abs()
        for t in range(t1 - 1, t0 - 1, -1):
            lam = dh[b, t] + g
            size, path = size + dh[b, t].abs(), path + 2 * size + 10 * dh[b, t].abs()
            out["dx"][b, t], bound["dx"][b, t] = lam, path
            was = reach[b, t - 1] if t > t0 else (8 * before[b, t].abs())
            out["dgate"][b, t] = lam * before[b, t]
            bound["dgate"][b, t] = path * before[b, t].abs() + was * lam.abs() + 2 * out["dgate"][b, t].abs()
            g = gate[b, t] * lam
            size, path = gate[b, t].abs() * size, gate[b, t].abs() * (path + 2 * size)
        out["dh0"][n], bound["dh0"][n] = g, path
    return out, bound


# ---------------------------------------------------------------- a paged cache

def rotate(x, pos, freqs, interleaved):
    """x [tokens, heads, d] in 64 bits, its first values rotated by pos * freqs."""
    x = x.double().clone()
    half = freqs.shape[0]
    ang = pos.double()[:, None] * freqs.double()[None, :]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = torch.cos(ang[:, i])[:, None], torch.sin(ang[:, i])[:, None]
        u, w = x[:, :, a].clone(), x[:, :, b].clone()
        x[:, :, a], x[:, :, b] = u * c - w * s, u * s + w * c
    return x


def place(table, seq, row, page, pages):
    """Row of the flattened pool where a sequence's row lies, or None."""
    if row < 0 or row // page >= table.shape[1]:
        return None
    at = int(table[seq, row // page])
    return at * page + row % page if 0 <= at < pages else None


def sees(tree_row, i, j):
    """Whether new token i sees new token j (tree_row: its words, or None)."""
    if tree_row is None:
        return j <= i
    return j // 32 < len(tree_row) and bool(int(tree_row[j // 32]) >> (j % 32) & 1)


def paged_attn(q, K_pages, V_pages, table, ctx, tree, scale, seqs):
    """o [B,T,Hq,d], lse [B,T,Hq], per element of o the root of its terms' summed
    squares, and a bound of the error of lse in fp32: a score is a sum of d products
    in some order, (d + 4) roundings of their absolute sum and four of its own, of the
    maximum's and of the result's size, and the sum of the exponentials has no more
    roundings than keys."""
    B, T, Hq, d = q.shape
    pages, page, Hkv, _ = K_pages.shape
    G = Hq // Hkv
    o = torch.zeros(B, T, Hq, d, dtype=torch.float64, device=q.device)
    size = torch.zeros_like(o)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(lse)
    Kf, Vf = K_pages.reshape(pages * page, Hkv, d), V_pages.reshape(pages * page, Hkv, d)
    table, ctx = table.cpu(), [int(c) for c in ctx]
    tree = None if tree is None else tree.cpu()
    for n, (b, t0, t1) in enumerate(seqs):
        if ctx[n] < 0 or t1 == t0:
            continue
        keys = [(r, place(table, n, r, page, pages)) for r in range(ctx[n] + t1 - t0)]
        keys = [(r, at) for r, at in keys if at is not None]
        if not keys:
            continue
        rows = torch.tensor([at for _, at in keys], device=q.device)
        new = [r - ctx[n] for r, _ in keys]
        seen = torch.tensor([[x < 0 or sees(None if tree is None else tree[b, t0 + i], i, x) for x in new]
                             for i in range(t1 - t0)], device=q.device)
        for hk in range(Hkv):
            K, V = Kf[rows, hk].double(), Vf[rows, hk].double()
            for h in range(hk * G, (hk + 1) * G):
                x = q[b, t0:t1, h].double()
                for i in range(t1 - t0):   # a row by itself, from the keys that it sees
                    m = seen[i]
                    if not m.any():
                        continue
                    k, v = K[m], V[m]
                    s = scale * (k @ x[i])
                    top = s.max()
                    e = torch.exp(s - top)
                    p = e / e.sum()
                    o[b, t0 + i, h] = p @ v
                    size[b, t0 + i, h] = (p.square() @ v.square()).sqrt()
                    lse[b, t0 + i, h] = top + e.sum().log()
                    reach = abs(scale) * (k.abs() @ x[i].abs()).max()
                    bound[b, t0 + i, h] = ((d + 4) * reach + 4 * s.abs().max() + 4 * abs(lse[b, t0 + i, h]) + len(s)) * 2.0 ** -24
    return o, lse, size, bound
