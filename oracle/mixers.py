"""Linear attention with a decay per head and window attention with sinks,
from their definitions in 64 bits, token by token and row by row (torch, on any
device). Test infrastructure only; shares no code with the kernels.

Sequences are given as (row of the batch, first token, end)."""
import math

import torch


def spans(B, T, cu=None):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    cu = [int(x) for x in cu]
    return [(0, a, b) for a, b in zip(cu, cu[1:])]


def linattn(q, k, v, gate, S0, seqs):
    """o [B,T,H,dv], S_T [N,H,dk,dv] and every state (a list per sequence)."""
    q, k, v, gate = (x.double() for x in (q, k, v, gate))
    if gate.dim() == 1:
        gate = gate.expand(q.shape[:3])
    H, dk, dv = q.shape[2], q.shape[3], v.shape[3]
    o, finals, states = torch.zeros_like(v), [], []
    for n, (b, t0, t1) in enumerate(seqs):
        S = torch.zeros(H, dk, dv, dtype=torch.float64, device=q.device) if S0 is None else S0[n].double()
        kept = [S]
        for t in range(t0, t1):
            S = gate[b, t][:, None, None] * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = (S * q[b, t][:, :, None]).sum(1)
            kept.append(S)
        finals.append(S)
        states.append(kept)
    return o, torch.stack(finals), states


def linattn_grad(q, k, v, gate, dO, S0, dS_T, seqs):
    """The gradient by the recurrence's adjoint: dict of dq, dk, dv, dgate
    [B,T,H], dS0."""
    _, _, states = linattn(q, k, v, gate, S0, seqs)
    q, k, v, gate, dO = (x.double() for x in (q, k, v, gate, dO))
    if gate.dim() == 1:
        gate = gate.expand(q.shape[:3])
    g = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v),
         "dgate": torch.zeros(q.shape[:3], dtype=torch.float64, device=q.device)}
    first = []
    for n, (b, t0, t1) in enumerate(seqs):
        G = torch.zeros_like(states[n][0]) if dS_T is None else dS_T[n].double()
        for t in range(t1 - 1, t0 - 1, -1):
            S, before = states[n][t - t0 + 1], states[n][t - t0]
            g["dq"][b, t] = (S * dO[b, t][:, None, :]).sum(2)
            G = G + q[b, t][:, :, None] * dO[b, t][:, None, :]
            g["dk"][b, t] = (G * v[b, t][:, None, :]).sum(2)
            g["dv"][b, t] = (G * k[b, t][:, :, None]).sum(1)
            g["dgate"][b, t] = (G * before).sum((1, 2))
            G = gate[b, t][:, None, None] * G
        first.append(G)
    g["dS0"] = torch.stack(first)
    return g


def visible(T, window, sinks, device):
    """[T, T]: whether row i sees key j."""
    i = torch.arange(T, device=device)
    back = i[:, None] - i[None, :]
    return (back >= 0) & ((back < window) | (i[None, :] < sinks))


def swa(q, k, v, window, sinks, scale, seqs, dO=None):
    """o, lse [B,T,Hq] and, with dO, the gradient dict of dq, dk, dv, and for each
    the root of its terms' summed squares: p dO for dv, p (|dP| + |delta|) k (or
    q), the terms whose difference they are, for dq and dk, where |dP| and |delta|
    stand for the same root over the products dO v and dO o that they sum."""
    q, k, v = (x.double() for x in (q, k, v))
    group = q.shape[2] // k.shape[2]
    o = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:3], dtype=torch.float64, device=q.device)
    g = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v)}
    size = {n: torch.zeros_like(t) for n, t in g.items()}
    for b, t0, t1 in seqs:
        seen = visible(t1 - t0, window, sinks, q.device)
        for h in range(q.shape[2]):
            x, y, z = q[b, t0:t1, h], k[b, t0:t1, h // group], v[b, t0:t1, h // group]
            s = torch.where(seen, scale * torch.mm(x, y.t().contiguous()), torch.full((), -math.inf, dtype=torch.float64,
                                                                                     device=q.device))
            m = s.amax(-1, keepdim=True) if t1 > t0 else s.sum(-1, keepdim=True)
            e = torch.exp(s - m)
            tot = e.sum(-1, keepdim=True)
            p = e / tot
            o[b, t0:t1, h] = torch.mm(p, z)
            lse[b, t0:t1, h] = (m + tot.log())[:, 0]
            if dO is not None:
                up = dO[b, t0:t1, h].double()
                dp, delta = torch.mm(up, z.t().contiguous()), (up * o[b, t0:t1, h]).sum(-1, keepdim=True)
                ds = p * (dp - delta) * scale
                parts = torch.mm(up.square(), z.square().t().contiguous()).sqrt()
                parts = parts + (up * o[b, t0:t1, h]).square().sum(-1, keepdim=True).sqrt()
                parts = (p * parts * scale).square()
                size["dq"][b, t0:t1, h] = torch.mm(parts, y.square()).sqrt()
                size["dk"][b, t0:t1, h // group] += torch.mm(parts.t().contiguous(), x.square())
                size["dv"][b, t0:t1, h // group] += torch.mm(p.square().t().contiguous(), up.square())
                g["dq"][b, t0:t1, h] = torch.mm(ds, y)
                g["dk"][b, t0:t1, h // group] += torch.mm(ds.t().contiguous(), x)
                g["dv"][b, t0:t1, h // group] += torch.mm(p.t().contiguous(), up)
    size["dk"], size["dv"] = size["dk"].sqrt(), size["dv"].sqrt()
    return (o, lse) if dO is None else (o, lse, g, size)
