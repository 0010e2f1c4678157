"""Calls of linear and window attention beyond what one launch takes are refused by
their checks, before anything is enqueued (no GPU: every call here fails its checks)."""
import pytest

from gated_delta_rule_46_amd import kda
from test_mixers_abi import FAKE, lib, lin_bwd, swa_bwd  # noqa: F401 (fixture)


@pytest.mark.parametrize("dk,dv,dtype", [(128, 64, kda.KDA_BF16), (128, 128, kda.KDA_F32), (16, 128, kda.KDA_BF16)])
def test_linear_gradient_of_millions_of_sequences(lib, dk, dv, dtype):  # noqa: F811
    """A workgroup of 512 or 1,024 threads a segment, one segment a sequence at least."""
    for kw in (dict(B=2 ** 23, N=0), dict(B=1, N=2 ** 23, cu=FAKE)):
        assert lin_bwd(lib, T=1, H=1, dk=dk, dv=dv, dtype=dtype, **kw) == kda.KDA_ENOTSUP
        assert lib.kda_linattn_bwd_workspace_bytes(kw["B"], 1, 1, dk, dv, kw["N"], int(kw["N"] > 0), dtype) == 0
        # within the forward's sizes, and within the gradient's for smaller states
        assert lib.kda_linattn_fwd_workspace_bytes(kw["B"], 1, 1, dk, dv, kw["N"], int(kw["N"] > 0), dtype) > 0
        assert lib.kda_linattn_bwd_workspace_bytes(kw["B"], 1, 1, 16, 16, kw["N"], int(kw["N"] > 0), dtype) > 0
    assert lib.kda_linattn_bwd_workspace_bytes(4000000, 1, 1, dk, dv, 0, 0, dtype) > 0


@pytest.mark.parametrize("N,H,dk,dv", [(2 ** 22, 2, 128, 128), (2 ** 23, 1, 16, 128), (2 ** 26, 1, 16, 16), (1, 2 ** 25, 32, 16),
                                       (2 ** 31 - 1, 2 ** 31 - 1, 64, 64)])
def test_linear_step_beyond_a_launch(lib, N, H, dk, dv):  # noqa: F811
    assert lib.kda_linattn_decode_step(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, N, H, dk, dv, kda.KDA_BF16, kda.GATE_SCALAR,
                                       None) == kda.KDA_ENOTSUP


@pytest.mark.parametrize("kw", [dict(B=65535, T=260, N=0), dict(B=65535, T=4096, N=0, Hq=3, Hkv=3)])
def test_window_gradient_beyond_a_launch(lib, kw):  # noqa: F811
    """As many key blocks as the forward takes, and parts of those with sinks besides."""
    kw = dict(dict(Hq=50, Hkv=50, d=32, window=1, sinks=256), **kw)
    assert swa_bwd(lib, **kw) == kda.KDA_ENOTSUP
    size = lambda sinks: lib.kda_swa_bwd_workspace_bytes(kw["B"], kw["Hq"], kw["Hkv"], kw["T"], 32, 1, sinks, 0, 0)  # noqa: E731
    assert size(256) == 0 and size(0) > 0   # without sinks it is within the forward's sizes
