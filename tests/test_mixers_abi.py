"""Refusals of the linear-attention and window-attention calls, in the C ABI
and in the binding, and the sizes of their workspaces (no GPU: every call here
fails its checks)."""
import os

import pytest
import torch

from gated_delta_rule_46_amd import kda

FAKE = 0x10000   # aligned, never dereferenced
OK, EINVAL, ENOTSUP, EALIGN = kda.KDA_OK, kda.KDA_EINVAL, kda.KDA_ENOTSUP, kda.KDA_EALIGN


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_46_amd import build
        build.build()
    return kda.library()


def lin_fwd(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, gate=FAKE, S0=None, o=FAKE, S_T=None, B=2, H=2, T=8, dk=16, dv=32, cu=None,
             N=0, dtype=kda.KDA_BF16, kind=kda.GATE_SCALAR, ws=FAKE, wsb=1 << 40, stream=None)
    a.update(kw)
    return lib.kda_linattn_fwd(*a.values())


def lin_bwd(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, gate=FAKE, S0=None, dO=FAKE, dST=None, gq=FAKE, gk=FAKE, gv=FAKE, gg=FAKE,
             gS0=None, B=2, H=2, T=8, dk=16, dv=32, cu=None, N=0, dtype=kda.KDA_BF16, kind=kda.GATE_SCALAR,
             ws=FAKE, wsb=1 << 40, stream=None)
    a.update(kw)
    return lib.kda_linattn_bwd(*a.values())


@pytest.mark.parametrize("call", [lin_fwd, lin_bwd])
@pytest.mark.parametrize("status,bad", [
    (EINVAL, dict(B=0)), (EINVAL, dict(H=0)), (EINVAL, dict(T=-1)),
    (EINVAL, dict(N=3)), (EINVAL, dict(cu=FAKE, N=2)), (EINVAL, dict(B=1, cu=FAKE, N=0)),
    (EINVAL, dict(q=None)), (EINVAL, dict(k=None)), (EINVAL, dict(v=None)), (EINVAL, dict(gate=None)),
    (EINVAL, dict(ws=None)), (EINVAL, dict(wsb=0)), (EINVAL, dict(wsb=255)),
    (ENOTSUP, dict(dk=24)), (ENOTSUP, dict(dv=256)), (ENOTSUP, dict(dk=0)), (ENOTSUP, dict(dtype=2)),
    (ENOTSUP, dict(kind=kda.GATE_CHANNEL)), (ENOTSUP, dict(kind=3)), (ENOTSUP, dict(H=65536)),
    (ENOTSUP, dict(T=2 ** 30)), (ENOTSUP, dict(B=2 ** 24, T=1, H=1)),
    (EALIGN, dict(q=FAKE + 8)), (EALIGN, dict(k=FAKE + 2)), (EALIGN, dict(v=FAKE + 4)), (EALIGN, dict(gate=FAKE + 1)),
    (EALIGN, dict(gate=FAKE + 2, dtype=kda.KDA_F32)), (EALIGN, dict(S0=FAKE + 2)), (EALIGN, dict(ws=FAKE + 8)),
    (EALIGN, dict(B=1, cu=FAKE + 2, N=2)),
])
def test_linear_refusals(lib, call, status, bad):
    assert call(lib, **bad) == status


def test_linear_refusals_of_each(lib):
    assert lin_fwd(lib, o=None) == EINVAL
    assert lin_fwd(lib, o=FAKE + 8) == EALIGN
    assert lin_fwd(lib, S_T=FAKE + 2) == EALIGN
    assert lin_fwd(lib, kind=kda.GATE_HEAD, gate=FAKE + 2) == EALIGN          # fp32 whatever the dtype
    assert lin_fwd(lib, T=0, q=None, k=None, v=None, gate=None, o=None) == OK   # nothing to do
    for name in ("dO", "gq", "gk", "gv", "gg"):
        assert lin_bwd(lib, **{name: None}) == EINVAL
    for name in ("dO", "gq", "gk", "gv"):
        assert lin_bwd(lib, **{name: FAKE + 8}) == EALIGN
    assert lin_bwd(lib, gg=FAKE + 1) == EALIGN
    assert lin_bwd(lib, dST=FAKE + 1) == EALIGN
    assert lin_bwd(lib, gS0=FAKE + 2) == EALIGN
    assert lin_bwd(lib, kind=kda.GATE_HEAD) == EINVAL                         # a constant has no gradient
    need = kda.linattn_bwd_workspace_bytes(2, 2, 8, 16, 32)
    assert lin_bwd(lib, wsb=need - 1) == EINVAL
    need = kda.linattn_fwd_workspace_bytes(2, 2, 1000, 16, 32)
    assert lin_fwd(lib, T=1000, wsb=need - 1) == EINVAL
    assert lin_bwd(lib, T=0, q=None, k=None, v=None, gate=None, dO=None, gq=None, gk=None, gv=None, gg=None) == OK


def test_linear_step_refusals(lib):
    def step(**kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, gate=FAKE, S=FAKE, o=FAKE, N=2, H=2, dk=16, dv=16, dtype=kda.KDA_BF16,
                 kind=kda.GATE_SCALAR, stream=None)
        a.update(kw)
        return lib.kda_linattn_decode_step(*a.values())
    assert step(N=0) == EINVAL and step(H=-1) == EINVAL
    assert step(dk=8) == ENOTSUP and step(dv=100) == ENOTSUP and step(dtype=5) == ENOTSUP
    assert step(kind=kda.GATE_CHANNEL) == ENOTSUP and step(N=2 ** 30, H=2) == ENOTSUP
    for name in ("q", "k", "v", "gate", "S", "o"):
        assert step(**{name: None}) == EINVAL
    for name in ("q", "k", "v", "gate", "o"):
        assert step(**{name: FAKE + 1}) == EALIGN
    assert step(S=FAKE + 8) == EALIGN
    assert step(kind=kda.GATE_HEAD, gate=FAKE + 2) == EALIGN


def test_linear_workspace(lib):
    for f in (kda.linattn_fwd_workspace_bytes, kda.linattn_bwd_workspace_bytes):
        assert f(0, 2, 8, 16, 16) == 0 and f(1, 2, 8, 16, 48) == 0 and f(2, 2, 8, 16, 16, N=2, varlen=True) == 0
        assert f(1, 2, 8, 16, 16, N=0, varlen=True) == 0
        assert f(1, 2, 0, 16, 16) >= 256
        assert f(1, 2, 5000, 64, 64) <= f(1, 2, 5100, 64, 64) <= f(1, 4, 5100, 64, 64)
    # Packed: what the tokens need, and for each sequence no more than its state at
    # the ends of one segment and one block, in each direction.
    T, N, H, state = 131072, 1024, 16, 128 * 128
    blocks = (T // 64 + N + 1) * H
    segs = (T // 4096 + N + 1) * H
    assert kda.linattn_bwd_workspace_bytes(1, H, T, 128, 128, N=N, varlen=True) <= \
        2 * (blocks * (2 * state + 4) + segs * (6 * state + 4)) + 4096


def swa_fwd(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=None, B=2, Hq=4, Hkv=2, T=8, d=64, window=4, sinks=1, scale=0.125,
             cu=None, N=0, dtype=kda.KDA_BF16, stream=None)
    a.update(kw)
    return lib.kda_swa_fwd(*a.values())


def swa_bwd(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, dO=FAKE, gq=FAKE, gk=FAKE, gv=FAKE, B=2, Hq=4, Hkv=2, T=8,
             d=64, window=4, sinks=1, scale=0.125, cu=None, N=0, dtype=kda.KDA_BF16, ws=FAKE, wsb=1 << 40, stream=None)
    a.update(kw)
    return lib.kda_swa_bwd(*a.values())


@pytest.mark.parametrize("call", [swa_fwd, swa_bwd])
@pytest.mark.parametrize("status,bad", [
    (EINVAL, dict(B=0)), (EINVAL, dict(T=-1)), (EINVAL, dict(Hq=0)), (EINVAL, dict(Hkv=0)), (EINVAL, dict(Hkv=3)),
    (EINVAL, dict(Hq=2, Hkv=4)), (EINVAL, dict(window=0)), (EINVAL, dict(sinks=-1)),
    (EINVAL, dict(scale=float("nan"))), (EINVAL, dict(scale=float("inf"))), (EINVAL, dict(N=1)),
    (EINVAL, dict(cu=FAKE, N=2)), (EINVAL, dict(B=1, cu=FAKE, N=0)),
    (EINVAL, dict(q=None)), (EINVAL, dict(k=None)), (EINVAL, dict(v=None)), (EINVAL, dict(o=None)),
    (ENOTSUP, dict(d=16)), (ENOTSUP, dict(d=256)), (ENOTSUP, dict(dtype=9)), (ENOTSUP, dict(Hq=65536, Hkv=1)),
    (ENOTSUP, dict(B=65536)), (ENOTSUP, dict(T=2 ** 30)), (ENOTSUP, dict(B=65535, T=1, Hq=512)),
    (EALIGN, dict(q=FAKE + 8)), (EALIGN, dict(k=FAKE + 2)), (EALIGN, dict(v=FAKE + 4)), (EALIGN, dict(o=FAKE + 8)),
    (EALIGN, dict(lse=FAKE + 2)), (EALIGN, dict(B=1, cu=FAKE + 2, N=2)),
])
def test_window_refusals(lib, call, status, bad):
    assert call(lib, **bad) == status


def test_window_refusals_of_the_gradient(lib):
    for name in ("lse", "dO", "gq", "gk", "gv", "ws"):
        assert swa_bwd(lib, **{name: None}) == EINVAL
    for name in ("dO", "gq", "gk", "gv", "ws"):
        assert swa_bwd(lib, **{name: FAKE + 8}) == EALIGN
    need = kda.swa_bwd_workspace_bytes(2, 4, 2, 8, 64, 4, 1)
    assert need > 0 and swa_bwd(lib, wsb=need - 1) == EINVAL
    assert swa_fwd(lib, T=0, q=None, k=None, v=None, o=None) == OK
    assert swa_bwd(lib, T=0, q=None, k=None, v=None, o=None, lse=None, dO=None, gq=None, gk=None, gv=None) == OK


def test_window_step_refusals(lib):
    def step(**kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, K=FAKE, V=FAKE, pos=FAKE, o=FAKE, N=2, Hq=4, Hkv=2, d=64, window=4, sinks=1,
                 scale=0.125, dtype=kda.KDA_BF16, ws=FAKE, wsb=1 << 40, stream=None)
        a.update(kw)
        return lib.kda_swa_decode_step(*a.values())
    for bad in (dict(N=0), dict(Hq=3), dict(Hkv=0), dict(window=0), dict(sinks=-2), dict(scale=float("-inf"))):
        assert step(**bad) == EINVAL
    for bad in (dict(N=65536), dict(d=48), dict(dtype=-1), dict(window=2 ** 30, sinks=1)):
        assert step(**bad) == ENOTSUP
    for name in ("q", "k", "v", "K", "V", "pos", "o", "ws"):
        assert step(**{name: None}) == EINVAL
    for name in ("q", "k", "v", "K", "V", "o", "ws"):
        assert step(**{name: FAKE + 8}) == EALIGN
    assert step(pos=FAKE + 2) == EALIGN
    need = kda.swa_decode_workspace_bytes(2, 4, 2, 64, 4000, 1)
    assert need > 0 and step(window=4000, wsb=need - 1) == EINVAL


def test_window_fill_refusals(lib):
    def fill(**kw):
        a = dict(k=FAKE, v=FAKE, K=FAKE, V=FAKE, B=2, Hkv=2, T=8, d=64, window=4, sinks=1, cu=None, N=0,
                 dtype=kda.KDA_BF16, stream=None)
        a.update(kw)
        return lib.kda_swa_cache_fill(*a.values())
    for bad in (dict(B=0), dict(Hkv=0), dict(T=-1), dict(window=0), dict(sinks=-1), dict(N=5), dict(cu=FAKE, N=2),
                dict(k=None), dict(v=None), dict(K=None), dict(V=None)):
        assert fill(**bad) == EINVAL
    for bad in (dict(d=16), dict(dtype=4), dict(window=2 ** 30, sinks=1), dict(B=65536)):
        assert fill(**bad) == ENOTSUP
    for name in ("k", "v", "K", "V"):
        assert fill(**{name: FAKE + 8}) == EALIGN
    assert fill(T=0, k=None, v=None, K=None, V=None) == OK


def test_window_workspace(lib):
    f = kda.swa_bwd_workspace_bytes
    assert f(0, 4, 2, 8, 64, 4) == 0 and f(1, 4, 3, 8, 64, 4) == 0 and f(1, 4, 2, 8, 16, 4) == 0
    assert f(1, 4, 2, 8, 64, 0) == 0 and f(1, 4, 2, 8, 64, 4, -1) == 0 and f(2, 4, 2, 8, 64, 4, N=2, varlen=True) == 0
    assert f(1, 4, 2, 0, 64, 4) > 0
    assert f(1, 4, 2, 500, 64, 2 ** 40, 2 ** 40) == f(1, 4, 2, 500, 64, 500, 500)
    # Packed: one fp32 a row and head, and parts for a bounded number of workgroups
    # or of rows, however many sequences share them.
    T, Hq, Hkv = 65536, 32, 8
    most = max(2048 * 2, T // 64 + 1024 + 64) * Hkv * 2 * 64 * 128 * 4
    for N in (1, 64, 1024):
        assert f(1, Hq, Hkv, T, 128, 512, 4, N=N, varlen=True) <= T * Hq * 4 + 512 + min(most, 256 << 20)
    g = kda.swa_decode_workspace_bytes
    assert g(0, 4, 2, 64, 4) == 0 and g(1, 4, 3, 64, 4) == 0 and g(1, 4, 2, 16, 4) == 0 and g(70000, 4, 2, 64, 4) == 0
    assert g(1, 4, 2, 64, 0) == 0 and g(1, 4, 2, 64, 2 ** 30, 1) == 0
    assert g(1024, 32, 8, 128, 4096) >= 256 and g(1, 32, 8, 128, 4096) > g(1, 32, 8, 128, 100)


def test_binding_refusals():
    """What the binding refuses before it loads the library or asks for a GPU."""
    def t(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype)
    q, k, v, gate = t(1, 4, 2, 16), t(1, 4, 2, 16), t(1, 4, 2, 32), t(1, 4, 2)
    for bad in (dict(q=t(4, 2, 16)), dict(v=t(4, 2, 32))):
        with pytest.raises(ValueError):
            kda.linattn_fwd(**dict(dict(q=q, k=k, v=v, gate=gate), **bad))
    with pytest.raises(ValueError, match="B = 1"):
        kda.linattn_fwd(t(2, 4, 2, 16), t(2, 4, 2, 16), t(2, 4, 2, 32), t(2, 4, 2), cu_seqlens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="GPU"):   # host tensors
        kda.linattn_fwd(q, k, v, gate)
    with pytest.raises(TypeError, match="GPU"):
        kda.linattn_decode_step(q[0], k[0], v[0], gate[0], torch.zeros(4, 2, 16, 32))
    with pytest.raises(ValueError, match="multiple"):
        kda.swa_fwd(t(1, 4, 3, 64), t(1, 4, 2, 64), t(1, 4, 2, 64), window=2)
    for kw in (dict(window=0), dict(window=2, sinks=-1)):
        with pytest.raises(ValueError, match="window"):
            kda.swa_fwd(t(1, 4, 2, 64), t(1, 4, 2, 64), t(1, 4, 2, 64), **kw)
    with pytest.raises(ValueError, match="dims"):
        kda.swa_fwd(t(4, 2, 64), t(4, 2, 64), t(4, 2, 64), window=2)
    with pytest.raises(TypeError, match="GPU"):
        kda.swa_cache_fill(t(1, 4, 2, 64), t(1, 4, 2, 64), t(1, 6, 2, 64), t(1, 6, 2, 64), window=5, sinks=1)
