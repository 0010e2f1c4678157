"""The operators that stand beside the gated delta rule, as cases to measure: linear attention with a decay for each
head, and attention with a sliding window and first tokens that stay visible. Each in its three uses: over whole
sequences, its gradient, and one token at a time.

`run` computes a case in plain torch operations, or, where `own` is set, through the library's entry points.

Linear attention, for each sequence and head, with state S in R^{dk x dv} and decay a_t:

    S_t = a_t S_{t-1} + k_t v_t^T,    o_t = S_t^T q_t

Window attention, for each sequence and query head (kv head = head // group):

    o_i = sum_j softmax_j(scale q_i . k_j) v_j   over j <= i with i - j < window or j < sinks
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
CHUNK = 64   # block length of the plain chunked form


# ------------------------------------------------------------------ cases

def _lengths(case):
    """Sequence lengths of a case: `B` of length `T`, or the packed ones in `lens`."""
    if case.get("lens"):
        return [int(x) for x in case["lens"].split(",")]
    return [case["T"]] * case["B"]


def listed():
    return [
        # training on long sequences: the largest forward
        dict(name="lin_fwd_long", op="lin_fwd", dtype="bf16", B=2, T=8192, H=16, dk=128, dv=128, gate="token", s0=False),
        # prompts of a serving batch, packed, that continue from states
        dict(name="lin_fwd_packed", op="lin_fwd", dtype="bf16", lens="1213,64,1,2741,37,1945", H=8, dk=64, dv=128,
             gate="token", s0=True),
        # one short prompt in full precision, a fixed decay per head
        dict(name="lin_fwd_f32", op="lin_fwd", dtype="f32", B=1, T=777, H=4, dk=64, dv=64, gate="head", s0=False),
        # the gradient of a training step
        dict(name="lin_bwd_long", op="lin_bwd", dtype="bf16", B=2, T=4096, H=16, dk=128, dv=128, gate="token", s0=False),
        # the gradient of a packed batch in full precision, states in and out
        dict(name="lin_bwd_packed_f32", op="lin_bwd", dtype="f32", lens="515,1,290,129", H=4, dk=64, dv=32, gate="token",
             s0=True),
        # decoding for a large batch: the state is the traffic
        dict(name="lin_dec_batch", op="lin_dec", dtype="bf16", N=256, H=32, dk=128, dv=128, gate="token"),
        # decoding for one user: latency
        dict(name="lin_dec_one", op="lin_dec", dtype="bf16", N=1, H=16, dk=128, dv=128, gate="head"),
        # a long prompt under a window, shared key heads
        dict(name="win_fwd_long", op="win_fwd", dtype="bf16", B=2, T=8192, Hq=16, Hkv=4, d=128, window=1024, sinks=4),
        # short packed prompts in full precision
        dict(name="win_fwd_packed_f32", op="win_fwd", dtype="f32", lens="301,1,650,73", Hq=6, Hkv=2, d=64, window=100,
             sinks=3),
        # a training step's forward and backward
        dict(name="win_train", op="win_train", dtype="bf16", B=1, T=4096, Hq=16, Hkv=4, d=128, window=512, sinks=4),
        # decoding for a batch with full windows
        dict(name="win_dec_batch", op="win_dec", dtype="bf16", N=64, Hq=32, Hkv=8, d=128, window=2048, sinks=4),
        # decoding for one user: few rows, a long window
        dict(name="win_dec_one", op="win_dec", dtype="bf16", N=1, Hq=16, Hkv=4, d=128, window=4095, sinks=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, total):
    """`total` tokens as one to seven packed sequences of uneven length."""
    n = rng.randint(1, 7)
    w = [rng.uniform(0.02, 1.0) for _ in range(n)]
    lens = [max(1, int(total * x / sum(w))) for x in w]
    return ",".join(str(x) for x in lens)


def draw(rng):
    op = rng.choice(["lin_fwd", "lin_bwd", "lin_dec", "win_fwd", "win_train", "win_dec"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op.startswith("lin"):
        c.update(H=rng.choice([1, 2, 3, 4, 8, 16, 32]), dk=rng.choice([16, 32, 64, 128]), dv=rng.choice([16, 32, 64, 128]),
                 gate=rng.choice(["token", "token", "head"]))
        if op == "lin_dec":
            c["N"] = _log(rng, 1, 256)
            return c
        tokens = _log(rng, 5, min(32768, 131072 // c["H"]) if op == "lin_fwd" else min(16384, 65536 // c["H"]))
        c["s0"] = rng.choice([True, False])
    else:
        c["Hkv"] = rng.choice([1, 2, 3, 4, 8])
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 8])
        c.update(d=rng.choice([32, 64, 128]), window=_log(rng, 1, 2048), sinks=rng.choice([0, 0, 1, 4, 7, 64, 130]))
        if op == "win_dec":
            c["N"] = _log(rng, 1, max(1, 4096 * 64 // c["window"] // c["Hkv"] // 2))
            c["N"] = min(c["N"], 256)
            return c
        tokens = _log(rng, 5, min(8192, 65536 // c["Hq"]) if op == "win_fwd" else min(4096, 32768 // c["Hq"]))
    if rng.random() < 0.5:
        c["lens"] = _split(rng, tokens)
    else:
        c["B"] = rng.choice([1, 1, 2, 3])
        c["T"] = max(1, tokens // c["B"])
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _decay(case, g, shape):
    """Decays: sigmoid of N(3, 1) per token in the inputs' type, or one fp32 value per head, spread from fast to slow."""
    if case["gate"] == "head":
        h = torch.arange(case["H"], device="cuda", dtype=torch.float32)
        u = torch.rand(case["H"], device="cuda", generator=g)
        return 1.0 - torch.exp2(-1.0 - 7.0 * (h + u) / case["H"])
    return torch.sigmoid(3.0 + torch.randn(shape, device="cuda", generator=g)).to(TYPES[case["dtype"]])


def _inputs(case, seed):
    g, dt, op = _gen(seed), TYPES[case["dtype"]], case["op"]

    def rnd(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    if op.startswith("lin"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        if op == "lin_dec":
            lead = (case["N"], H)
        else:
            lens = _lengths(case)
            lead = (1, sum(lens), H) if case.get("lens") else (case["B"], case["T"], H)
        q, k, v = rnd(*lead, dk), rnd(*lead, dk), rnd(*lead, dv)
        s = dict(q=(q / q.norm(dim=-1, keepdim=True)).to(dt), k=(k / k.norm(dim=-1, keepdim=True)).to(dt), v=v.to(dt),
                 gate=_decay(case, g, lead))
        if op == "lin_dec":
            s["S"] = 0.3 * rnd(case["N"], H, dk, dv)
            return s
        s["S0"] = 0.3 * rnd(len(lens), H, dk, dv) if case["s0"] else None
        if op == "lin_bwd":
            s["dO"] = rnd(*lead, dv).to(dt)
            s["dS_T"] = 0.3 * rnd(len(lens), H, dk, dv) if case["s0"] else None
    else:
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        if op == "win_dec":
            N, slots = case["N"], case["sinks"] + case["window"]
            s = dict(q=rnd(N, Hq, d).to(dt), k=rnd(N, Hkv, d).to(dt), v=rnd(N, Hkv, d).to(dt),
                     Kc=rnd(N, slots, Hkv, d).to(dt), Vc=rnd(N, slots, Hkv, d).to(dt))
            # most sequences have filled their window, some have only begun
            far = torch.rand(N, device="cuda", generator=g)
            s["pos"] = torch.where(far < 0.25, far * 4 * slots, slots * (1 + 8 * far)).to(torch.int32)
            return s
        lens = _lengths(case)
        lead = (1, sum(lens)) if case.get("lens") else (case["B"], case["T"])
        s = dict(q=rnd(*lead, Hq, d).to(dt), k=rnd(*lead, Hkv, d).to(dt), v=rnd(*lead, Hkv, d).to(dt))
        if op == "win_train":
            s["dO"] = rnd(*lead, Hq, d).to(dt)
    s["cu"] = None
    if case.get("lens"):
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms

def _token_places(case, s):
    """Of every token (batch and time flattened): its place in an axis where each sequence is padded to whole chunks,
    the sequence of each chunk, and the number of chunks. From the lengths that the program knows."""
    lens = torch.tensor(_lengths(case))
    nc = (lens + CHUNK - 1) // CHUNK
    first = nc.cumsum(0) - nc
    at = torch.arange(int(lens.sum())) - torch.repeat_interleave(lens.cumsum(0) - lens, lens)
    place = torch.repeat_interleave(first * CHUNK, lens) + at
    return place.cuda(), torch.repeat_interleave(torch.arange(len(lens)), nc).cuda(), int(nc.sum())


def _lin_plain(case, q, k, v, logd, S0, place, seq, NC):
    """o and S_T in 32 bits from q, k, v [tokens, H, .] and the logarithms of the decays [tokens, H] (64 bits). Inside
    a chunk by its matrix of scores, between chunks by one product with the chunks' matrix of decays."""
    H, N = q.shape[1], len(_lengths(case))

    def chunks(x):   # [tokens, H, ...] -> [H, NC, CHUNK, ...], zero where a chunk has no token
        p = torch.zeros((NC * CHUNK,) + x.shape[1:], device=x.device, dtype=x.dtype).index_copy(0, place, x)
        return p.reshape((NC, CHUNK) + x.shape[1:]).movedim(2, 0)

    Q, K, V, g = chunks(q), chunks(k), chunks(v), chunks(logd).cumsum(-1)
    causal = torch.ones(CHUNK, CHUNK, device="cuda", dtype=torch.bool).tril()
    D = torch.exp((g[..., :, None] - g[..., None, :]).masked_fill(~causal, -math.inf)).float()
    total = g[..., -1]                                                  # [H, NC]
    Z = (K * torch.exp(total[..., None] - g).float()[..., None]).transpose(-1, -2) @ V
    G = total.cumsum(-1)
    before = G - total
    same = seq[:, None] == seq[None, :]
    c = torch.arange(NC, device="cuda")
    first = torch.searchsorted(seq, torch.arange(N, device="cuda"))     # of each sequence
    last = torch.searchsorted(seq, torch.arange(N, device="cuda"), right=True) - 1
    link = (before[:, :, None] - G[:, None, :]).masked_fill(~(same & (c[:, None] > c[None, :])), -math.inf)
    start = (torch.exp(link).float() @ Z.flatten(2)).reshape(Z.shape)
    if S0 is not None:
        start = start + torch.exp(before - before[:, first[seq]]).float()[..., None, None] * S0.transpose(0, 1)[:, seq]
    o = ((Q @ K.transpose(-1, -2)) * D) @ V + torch.exp(g).float()[..., None] * (Q @ start)
    o = o.movedim(0, 2).reshape(NC * CHUNK, H, -1)[place]
    S_T = torch.exp(total).float()[..., None, None] * start + Z
    return o, S_T[:, last].transpose(0, 1)


def _log_decay(case, gate, lead):
    a = gate.double().log()
    return a.expand(lead).reshape(-1, case["H"]) if case["gate"] == "head" else a.reshape(-1, case["H"])


def _plain_lin_fwd(case, s):
    dt, lead = s["q"].dtype, s["q"].shape[:3]
    q, k, v = (s[x].float().flatten(0, 1) for x in "qkv")
    o, S_T = _lin_plain(case, q, k, v, _log_decay(case, s["gate"], lead), s["S0"], *_token_places(case, s))
    return {"o": o.reshape(*lead, -1).to(dt), "S_T": S_T.contiguous()}


def _plain_lin_bwd(case, s):
    dt, lead = s["q"].dtype, s["q"].shape[:3]
    wanted = {x: s[x].float().detach().requires_grad_() for x in ("q", "k", "v")}
    gate = s["gate"].float().detach().requires_grad_(case["gate"] == "token")
    if case["gate"] == "token":
        wanted["gate"] = gate
    if s["S0"] is not None:
        wanted["S0"] = s["S0"].detach().clone().requires_grad_()
    with torch.enable_grad():
        o, S_T = _lin_plain(case, *(wanted[x].flatten(0, 1) for x in "qkv"), _log_decay(case, gate, lead), wanted.get("S0"),
                            *_token_places(case, s))
        loss = (o.double() * s["dO"].flatten(0, 1)).sum()
        if s["dS_T"] is not None:
            loss = loss + (S_T.double() * s["dS_T"]).sum()
        grads = torch.autograd.grad(loss, list(wanted.values()))
    return {"d" + n: g if n == "S0" else g.to(dt) for n, g in zip(wanted, grads)}


def _plain_lin_dec(case, s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    a = s["gate"].float().expand(q.shape[:2])
    s["S"].copy_(a[..., None, None] * s["S"] + k[..., :, None] * v[..., None, :])
    o = (q[..., :, None] * s["S"]).sum(-2)
    return {"o": o.to(s["q"].dtype), "S": s["S"]}


def _visible(case, T):
    i = torch.arange(T, device="cuda")
    back = i[:, None] - i[None, :]
    return (back >= 0) & ((back < case["window"]) | (i[None, :] < case["sinks"]))


def _win_mask(case, s):
    """Which keys each query of a row of the batch sees."""
    T = s["q"].shape[1]
    if s["cu"] is None:
        return _visible(case, T)
    at = torch.arange(T, device="cuda")
    seq = torch.searchsorted(s["cu"], at, right=True) - 1
    at = at - s["cu"][seq]
    back = at[:, None] - at[None, :]
    return (seq[:, None] == seq[None, :]) & (back >= 0) & ((back < case["window"]) | (at[None, :] < case["sinks"]))


def _win_plain(case, s, q, k, v):
    """o [B, T, Hq, d] and the scores' log-sum-exp [B, T, Hq] in 32 bits."""
    group = case["Hq"] // case["Hkv"]
    Q = q.transpose(1, 2)
    K, V = (x.transpose(1, 2).repeat_interleave(group, 1) for x in (k, v))
    scores = (Q @ K.transpose(-1, -2)) * case["d"] ** -0.5
    scores = scores.masked_fill(~_win_mask(case, s), -math.inf)
    top = scores.amax(-1, keepdim=True).detach()
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ V) / total
    return o.transpose(1, 2), (top + total.log()).squeeze(-1).transpose(1, 2)


def _plain_win_fwd(case, s):
    o, lse = _win_plain(case, s, s["q"].float(), s["k"].float(), s["v"].float())
    return {"o": o.to(s["q"].dtype).contiguous(), "lse": lse.contiguous()}


def _plain_win_train(case, s):
    dt = s["q"].dtype
    q, k, v = (s[x].float().detach().requires_grad_() for x in "qkv")
    with torch.enable_grad():
        o, _ = _win_plain(case, s, q, k, v)
        dq, dk, dv = torch.autograd.grad(o, [q, k, v], s["dO"].float())
    return {"o": o.detach().to(dt).contiguous(), "dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt)}


def _plain_win_dec(case, s):
    W, n_sink, pos = case["window"], case["sinks"], s["pos"].long()
    rows = torch.arange(case["N"], device="cuda")
    slot = torch.where(pos < n_sink, pos, n_sink + (pos - n_sink) % W)
    s["Kc"][rows, slot] = s["k"]
    s["Vc"][rows, slot] = s["v"]
    seen = torch.arange(n_sink + W, device="cuda")[None, :] <= pos[:, None]
    group = case["Hq"] // case["Hkv"]
    q = s["q"].float().reshape(case["N"], case["Hkv"], group, -1)
    K, V = s["Kc"].float().transpose(1, 2), s["Vc"].float().transpose(1, 2)
    scores = (q @ K.transpose(-1, -2)) * case["d"] ** -0.5
    scores = scores.masked_fill(~seen[:, None, None, :], -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    o = (p @ V) / p.sum(-1, keepdim=True)
    return {"o": o.reshape(s["q"].shape).to(s["q"].dtype), "Kc": s["Kc"], "Vc": s["Vc"]}


PLAIN = {"lin_fwd": _plain_lin_fwd, "lin_bwd": _plain_lin_bwd, "lin_dec": _plain_lin_dec, "win_fwd": _plain_win_fwd,
         "win_train": _plain_win_train, "win_dec": _plain_win_dec}


# ------------------------------------------------------------------ the library's calls

def _own(case, s):
    from gated_delta_rule_46_amd import kda

    op = case["op"]
    if op == "lin_fwd":
        o, S_T = kda.linattn_fwd(s["q"], s["k"], s["v"], s["gate"], S0=s["S0"], cu_seqlens=s["cu"])
        return {"o": o, "S_T": S_T}
    if op == "lin_bwd":
        g = kda.linattn_bwd(s["q"], s["k"], s["v"], s["gate"], s["dO"], S0=s["S0"], dS_T=s["dS_T"], cu_seqlens=s["cu"],
                            want_dS0=s["S0"] is not None)
        return {n: g[n] for n in ("dq", "dk", "dv", "dgate", "dS0") if g.get(n) is not None}
    if op == "lin_dec":
        return {"o": kda.linattn_decode_step(s["q"], s["k"], s["v"], s["gate"], s["S"]), "S": s["S"]}
    W, n_sink = case["window"], case["sinks"]
    if op == "win_fwd":
        o, lse = kda.swa_fwd(s["q"], s["k"], s["v"], window=W, sinks=n_sink, cu_seqlens=s["cu"])
        return {"o": o, "lse": lse}
    if op == "win_train":
        o, lse = kda.swa_fwd(s["q"], s["k"], s["v"], window=W, sinks=n_sink, cu_seqlens=s["cu"])
        g = kda.swa_bwd(s["q"], s["k"], s["v"], o, lse, s["dO"], window=W, sinks=n_sink, cu_seqlens=s["cu"])
        return {"o": o, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}
    o = kda.swa_decode_step(s["q"], s["k"], s["v"], s["Kc"], s["Vc"], s["pos"], window=W, sinks=n_sink)
    return {"o": o, "Kc": s["Kc"], "Vc": s["Vc"]}


def run(state):
    if own:
        return _own(state["case"], state)
    return PLAIN[state["case"]["op"]](state["case"], state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    es, op = BYTES[case["dtype"]], case["op"]

    def pairs():
        """(query, key) pairs that a head sees over all sequences."""
        n = 0
        for T in _lengths(case):
            i = torch.arange(T)
            near = torch.clamp(i + 1, max=case["window"])
            n += int((near + torch.clamp(i + 1 - near, max=case["sinks"])).sum())
        return n

    if op.startswith("lin"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        rows = case["N"] * H if op == "lin_dec" else sum(_lengths(case)) * H
        gate = rows * es if case["gate"] == "token" else 4 * H
        if op == "lin_dec":
            return {"bytes": rows * (8 * dk * dv + (2 * dk + 2 * dv) * es) + gate, "flops": rows * 5 * dk * dv}
        states = len(_lengths(case)) * H * dk * dv * 4
        if op == "lin_fwd":
            return {"bytes": rows * (2 * dk + 2 * dv) * es + gate + states * (2 if case["s0"] else 1),
                    "flops": rows * 4 * dk * dv}
        return {"bytes": rows * (4 * dk + 3 * dv) * es + gate * (2 if case["gate"] == "token" else 1)
                + states * (3 if case["s0"] else 0), "flops": rows * 10 * dk * dv}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if op == "win_dec":
        kept = case["N"] * (case["sinks"] + case["window"]) * 0.9
        return {"bytes": kept * Hkv * 2 * d * es + case["N"] * (2 * Hq + 4 * Hkv) * d * es, "flops": kept * Hq * 4 * d}
    rows = sum(_lengths(case))
    if op == "win_fwd":
        return {"bytes": rows * ((2 * Hq + 2 * Hkv) * d * es + 4 * Hq), "flops": pairs() * Hq * 4 * d}
    return {"bytes": rows * (4 * Hq + 4 * Hkv) * d * es, "flops": pairs() * Hq * 14 * d}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]

    def spans():
        """(row of the batch, first token, end) of each sequence."""
        lens = _lengths(case)
        if not case.get("lens"):
            return [(b, 0, case["T"]) for b in range(case["B"])]
        ends = [sum(lens[:n + 1]) for n in range(len(lens))]
        return [(0, e - n, e) for n, e in zip(lens, ends)]

    def linear(keep):
        """The recurrence, token by token. `keep`: every state too, as the gradient needs them."""
        q, k, v, a = (s[x].double() for x in ("q", "k", "v", "gate"))
        if case["gate"] == "head":
            a = a.expand(q.shape[:3])
        o = torch.empty_like(v)
        finals, kept = [], []
        for n, (b, t0, t1) in enumerate(spans()):
            S = s["S0"][n].double() if s["S0"] is not None else torch.zeros(case["H"], case["dk"], case["dv"], device="cuda",
                                                                            dtype=torch.float64)
            all_of_them = [S]
            for t in range(t0, t1):
                S = a[b, t][:, None, None] * S + k[b, t][:, :, None] * v[b, t][:, None, :]
                if keep:
                    all_of_them.append(S)
                else:
                    o[b, t] = torch.matmul(q[b, t][:, None, :], S)[:, 0]
            finals.append(S)
            if keep:
                kept.append(all_of_them)
        return q, k, v, a, o, torch.stack(finals), kept

    def linear_gradient():
        q, k, v, a, _, _, kept = linear(True)
        dO = s["dO"].double()
        dq, dk, dv, da = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(a.contiguous())
        first = []
        for n, (b, t0, t1) in enumerate(spans()):
            G = s["dS_T"][n].double() if s["dS_T"] is not None else torch.zeros_like(kept[n][0])
            for t in range(t1 - 1, t0 - 1, -1):
                S, was = kept[n].pop(), kept[n][-1]
                dq[b, t] = (S * dO[b, t][:, None, :]).sum(-1)
                G = G + q[b, t][:, :, None] * dO[b, t][:, None, :]
                dk[b, t] = (G * v[b, t][:, None, :]).sum(-1)
                dv[b, t] = (G * k[b, t][:, :, None]).sum(-2)
                da[b, t] = (G * was).sum((-1, -2))
                G = a[b, t][:, None, None] * G
            first.append(G)
        out = {"dq": dq, "dk": dk, "dv": dv}
        if case["gate"] == "token":
            out["dgate"] = da
        if s["S0"] is not None:
            out["dS0"] = torch.stack(first)
        return out

    def window():
        """Each sequence and query head by itself; with the gradient where dO is given."""
        group, d = case["Hq"] // case["Hkv"], case["d"]
        q, k, v = (s[x].double() for x in "qkv")
        dO = s["dO"].double() if "dO" in s else None
        o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda", dtype=torch.float64)
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for b, t0, t1 in spans():
            hidden = ~_visible(case, t1 - t0)
            for h in range(case["Hq"]):
                x, y, z = q[b, t0:t1, h], k[b, t0:t1, h // group], v[b, t0:t1, h // group]
                sc = torch.mm(x, y.t()).div_(math.sqrt(d)).masked_fill_(hidden, -math.inf)
                lse[b, t0:t1, h] = torch.logsumexp(sc, -1)
                p = torch.softmax(sc, -1)
                o[b, t0:t1, h] = torch.mm(p, z)
                if dO is not None:
                    up = dO[b, t0:t1, h]
                    ds = p * (torch.mm(up, z.t()) - (up * o[b, t0:t1, h]).sum(-1, keepdim=True)) / math.sqrt(d)
                    dq[b, t0:t1, h] = torch.mm(ds, y)
                    dk[b, t0:t1, h // group] += torch.mm(ds.t(), x)
                    dv[b, t0:t1, h // group] += torch.mm(p.t(), up)
        return {"o": o, "lse": lse} if dO is None else {"o": o, "dq": dq, "dk": dk, "dv": dv}

    if op == "lin_fwd":
        *_, o, S_T, _ = linear(False)
        return {"o": o, "S_T": S_T}
    if op == "lin_bwd":
        return linear_gradient()
    if op == "lin_dec":
        q, k, v = (s[x].double() for x in "qkv")
        a = s["gate"].double().expand(q.shape[:2]) if case["gate"] == "head" else s["gate"].double()
        S = torch.einsum("nh,nhkv->nhkv", a, s["S"].double()) + torch.einsum("nhk,nhv->nhkv", k, v)
        return {"o": torch.matmul(q[:, :, None, :], S)[:, :, 0], "S": S}
    if op in ("win_fwd", "win_train"):
        return window()
    W, n_sink, group = case["window"], case["sinks"], case["Hq"] // case["Hkv"]
    o = torch.empty(s["q"].shape, device="cuda", dtype=torch.float64)
    for n, p in enumerate(s["pos"].tolist()):
        at = p if p < n_sink else n_sink + (p - n_sink) % W
        s["Kc"][n, at], s["Vc"][n, at] = s["k"][n], s["v"][n]
        m = min(p + 1, n_sink + W)
        K, V = s["Kc"][n, :m].double(), s["Vc"][n, :m].double()
        for h in range(case["Hq"]):
            w = torch.softmax(torch.mv(K[:, h // group], s["q"][n, h].double()) / math.sqrt(case["d"]), 0)
            o[n, h] = torch.mv(V[:, h // group].t(), w)
    return {"o": o, "Kc": s["Kc"].double(), "Vc": s["Vc"].double()}
