"""A short, fixed workload to run under rocprofv3.

    python -m gated_delta_rule_46_amd.profile_run [--fwd 3] [--bwd 2] [--bwd-token 0] [--decode 8]
                                                  [--copy-mib 256] [--mixers CASE,CASE|all]
                                                  [--mixer-calls 12] [--rates] [--sizes GROUP,GROUP|all]

Runs, on cuda:0 and with seeded synthetic inputs: --fwd forward calls on the
workload --fwd-workload names (ckda: Complex KDA, B=2, H=16, T=8192, d=128,
bf16, chunk 64, the default; kda: KDA, B=4, H=16, T=4096; gdn: GDN with eight
packed sequences, H=32, T=110,440), --bwd
chunkwise backward calls (kda_chunk_bwd_cw) and --bwd-token token-form
backward calls (kda_chunk_bwd) on the same workload, --decode decode steps on the decode
workload (N=256, H=32, d=128, fp32 state in place), and --copy-mib MiB of
plain device-to-device copy (one read and one write of that many bytes per
call, three calls), whose counter readings calibrate FETCH_SIZE and
WRITE_SIZE against a known byte count.

--mixers runs listed cases of perf/operators.py (linear attention and window
attention) and perf/more_operators.py (gated linear recurrence, paged cache),
--mixer-calls calls of each on three sets of inputs in turn; alone, with --fwd 0
--bwd 0 --decode 0. --rates prints what large copies and large matrix products
reach on this card, and both one-token state updates (decode_step,
linattn_decode_step) on one state and on three in turn. --sizes times the sizes
at which the recurrence's and the paged cache's choices of a kernel, a block or
a split were made (groups: see `sizes`); KDA_LIB names a build with a choice
turned over, for the other side.
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import sys


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def operators(name):
    """perf/<name>.py, set to the library's own calls."""
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "perf", name + ".py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.own = True
    return m


def timed(torch, call, calls):
    """Seconds a call, of `calls` in a row after as many untimed ones."""
    for i in range(calls):
        call(i)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for i in range(calls):
        call(i)
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / 1e3 / calls


def print_rates(torch, kda):
    for gib in (1, 2, 4):
        src = torch.ones(gib << 28, device="cuda")
        dst = torch.empty_like(src)
        for name, call in (("copy_", lambda i: dst.copy_(src)), ("multiplied by one", lambda i: torch.mul(src, 1.0, out=dst))):
            print("copy of %d GiB, %s: %.2f TB/s read and written" % (gib, name, 2 * (gib << 30) / timed(torch, call, 20) / 1e12),
                  flush=True)
        del src, dst
    for dtype, n in ((torch.bfloat16, 8192), (torch.bfloat16, 16384), (torch.float32, 8192)):
        x, y = (torch.randn(n, n, device="cuda", dtype=dtype) for _ in range(2))
        print("product of %d x %d %s: %.0f TFLOP/s" % (n, n, str(dtype)[6:], 2 * n ** 3 / timed(torch, lambda i: x @ y, 10) / 1e12),
              flush=True)
    N, H, d = 256, 32, 128
    sets = [[torch.randn(N, H, d, device="cuda").bfloat16() for _ in range(3)]
            + [torch.rand(N, H, device="cuda").bfloat16() for _ in range(2)] + [torch.randn(N, H, d, d, device="cuda")]
            for _ in range(3)]
    for n in (1, 3):
        for name, call in (("decode_step", lambda i: kda.decode_step(*sets[i % n])),
                           ("linattn_decode_step", lambda i: kda.linattn_decode_step(*sets[i % n][:4], sets[i % n][5]))):
            s = timed(torch, call, 60)
            print("%s, 256 x 32 x 128 x 128, %d state(s) in turn: %.1f us, %.2f TB/s of state"
                  % (name, n, s * 1e6, 8 * N * H * d * d / s / 1e12), flush=True)


def sizes():
    """{group: [case]}: cases of perf/more_operators.py by the choice that they bear on."""
    def attn(N, T, ctx, heads, dtype="bf16", d=128, page=16, tree=False):
        lo, hi = ctx if isinstance(ctx, tuple) else (ctx, ctx)
        return dict(op="attn", dtype=dtype, N=N, T=T, ctx_lo=lo, ctx_hi=hi, tree=tree, Hq=heads[0], Hkv=heads[1], d=d, page=page)

    def recur(B, T, C, dtype="bf16", gate=None, op="glr_fwd", packed=False):
        batch = dict(lens=",".join([str(T)] * B)) if packed else dict(B=B, T=T)
        return dict(op=op, dtype=dtype, gate=gate or dtype, **batch, C=C, h0=False)

    wide, narrow = (32, 8), (16, 4)
    return {
        "share_few": [attn(400, 1, (100, 4096), wide), attn(900, 1, (100, 2048), wide)],
        "share_rows": [attn(64, 32, (100, 8192), wide, tree=True), attn(100, 32, (100, 8192), wide, tree=True),
                       attn(128, 16, 2048, wide, tree=True), attn(16, 512, 0, narrow)],
        "row_blocks": [attn(8, 8, 8192, narrow, page=32, tree=True), attn(64, 8, 4096, wide, tree=True),
                       attn(256, 5, 2048, wide, tree=True), attn(64, 8, 4096, wide, d=64, tree=True),
                       attn(64, 8, 4096, wide, d=32, tree=True), attn(64, 8, 4096, wide, "f32", tree=True)],
        "at_once": [attn(8, 12, 8192, narrow, "f32", tree=True), attn(1, 16, 16384, narrow, "f32", tree=True),
                    attn(64, 16, (100, 4096), wide, "f32", tree=True)],
        "at_once_few": [attn(64, 1, (100, 4096), wide, d=32), attn(8, 8, 8192, narrow, d=32, page=32, tree=True)],
        "two_products": [attn(1, 2048, 6144, narrow, page=128), attn(1, 2048, 0, narrow, page=128),
                         attn(8, 64, (2048, 16384), narrow, page=32, tree=True)],
        "attn_f32": [attn(64, 1, (100, 4096), wide, "f32"), attn(1, 1024, 4096, narrow, "f32", page=128)],
        "stream": [recur(16, T, 2048, *ty) for ty in (("bf16",), ("bf16", "f32"), ("f32",)) for T in (512, 1024, 2048, 4096)]
        + [recur(32, 2048, 1024, "f32"), recur(64, 2048, 509, "f32"), recur(8, 4096, 2048)],
        "states": [recur(1, 131072, 256)],
        "gradients": [recur(2, 4096, 2048, *ty, op="glr_bwd") for ty in (("bf16",), ("bf16", "f32"), ("f32", "f32"))],
        "short": [recur(256, 8, 4096, op=op, packed=p) for op in ("glr_fwd", "glr_bwd") for p in (False, True)],
        "tokens": [recur(2, 8192, 2048), recur(1, 4096, 2048, "f32"), recur(1, 4096, 2049)],
    }


def print_sizes(torch, names):
    m = operators("more_operators")
    for group, cases in sizes().items():
        if names != "all" and group not in names.split(","):
            continue
        for case in cases:
            states = [m.prepare(case, seed) for seed in range(3)]
            s = sorted(timed(torch, lambda i: m.run(states[i % 3]), 60) for _ in range(5))[2]
            print("%s | %s | %.1f us" % (group, " ".join("%s=%.24s" % x for x in case.items() if x[0] != "h0"), s * 1e6), flush=True)
            del states


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--fwd", type=int, default=3)
    ap.add_argument("--fwd-workload", choices=("ckda", "kda", "gdn"), default="ckda")
    ap.add_argument("--bwd", type=int, default=2)
    ap.add_argument("--bwd-token", type=int, default=0)
    ap.add_argument("--decode", type=int, default=8)
    ap.add_argument("--copy-mib", type=int, default=256)
    ap.add_argument("--mixers", default="")
    ap.add_argument("--mixer-calls", type=int, default=12)
    ap.add_argument("--rates", action="store_true")
    ap.add_argument("--sizes", default="")
    args = ap.parse_args(argv)

    sys.path.insert(0, ROOT)
    import torch
    from gated_delta_rule_46_amd import inputs, kda

    dev = torch.device("cuda", 0)
    torch.cuda.set_device(dev)
    kda.library()
    if args.fwd > 0:
        w = {"ckda": inputs.ckda_fwd, "kda": inputs.kda_fwd, "gdn": inputs.gdn_varlen}[args.fwd_workload](seed=0)
        q, k, v, g, b = (t.to(dev) for t in (w.q, w.k, w.v, w.gate, w.beta))
        cu = None if w.cu_seqlens is None else w.cu_seqlens.to(dev)
        N = w.n_seqs
        ws = torch.empty(kda.workspace_bytes(w.B, w.H, w.T, w.dk, w.dv, w.chunk, N, cu is not None, w.dtype),
                         device=dev, dtype=torch.uint8)
        o = torch.empty((w.B, w.T, w.H, w.dv), device=dev, dtype=torch.float32)
        ST = torch.empty((N, w.H, w.dk, w.dv), device=dev, dtype=torch.float32)
        for _ in range(args.fwd):
            kda.chunk_fwd(q, k, v, g, b, cu_seqlens=cu, chunk=w.chunk, gate_kind=w.gate_kind, out=o, S_T=ST,
                          workspace=ws)
        torch.cuda.synchronize()
        print("forward calls: %d (%s)" % (args.fwd, args.fwd_workload), flush=True)
        del q, k, v, g, b, cu, ws, o, ST
    for calls, chunked in ((args.bwd, True), (args.bwd_token, False)):
        if calls <= 0:
            continue
        w = inputs.ckda_fwd(seed=0)
        dO, dST = inputs.cotangents(w, seed=0)
        t = [x.to(dev) for x in (w.q, w.k, w.v, w.gate, w.beta, dO)]
        dST = dST.to(dev)
        need = (kda.bwd_cw_workspace_bytes if chunked else kda.bwd_workspace_bytes)(w.B, w.H, w.T, w.dk, w.dv)
        ws = torch.empty(need, device=dev, dtype=torch.uint8)
        g = kda.chunk_bwd(*t, dS_T=dST, workspace=ws, chunked=chunked)
        for _ in range(calls - 1):
            kda.chunk_bwd(*t, dS_T=dST, workspace=ws, out=g, chunked=chunked)
        torch.cuda.synchronize()
        print("%s backward calls: %d" % ("chunkwise" if chunked else "token-form", calls), flush=True)
        del t, dST, ws, g
    if args.decode > 0:
        dw = inputs.ckda_decode(n_steps=min(args.decode, 16))
        S = dw.S.to(dev)
        steps = [tuple(st[x].to(dev) for x in ("q", "k", "v", "gate", "beta")) for st in dw.steps]
        od = torch.empty((dw.N, dw.H, dw.dv), device=dev, dtype=torch.float32)
        for i in range(args.decode):
            qd, kd, vd, gd, bd = steps[i % len(steps)]
            kda.decode_step(qd, kd, vd, gd, bd, S, out=od, gate_kind=0)
        torch.cuda.synchronize()
        print("decode steps: %d" % args.decode, flush=True)
        del S, steps, od
    if args.mixers:
        files = [operators(name) for name in ("operators", "more_operators")]
        for m, case in [(m, case) for m in files for case in m.listed()]:
            if args.mixers != "all" and case["name"] not in args.mixers.split(","):
                continue
            states = [m.prepare(case, seed) for seed in range(3)]
            for i in range(args.mixer_calls):
                m.run(states[i % 3])
            torch.cuda.synchronize()
            print("%s calls: %d" % (case["name"], args.mixer_calls), flush=True)
            del states
    if args.rates:
        print_rates(torch, kda)
    if args.sizes:
        print_sizes(torch, args.sizes)
    if args.copy_mib > 0:
        src = torch.ones(args.copy_mib << 20, device=dev, dtype=torch.uint8)
        dst = torch.empty_like(src)
        for _ in range(3):
            dst.copy_(src)
        torch.cuda.synchronize()
        print("copy: 3 x %d MiB" % args.copy_mib, flush=True)
    return 0


if __name__ == "__main__":
    sys.exit(main())
