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
