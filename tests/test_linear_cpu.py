"""The linear layer's oracle pinned by differences, its workspaces, and the
entry points' refusals (no GPU: every refused call fails before any HIP call)."""
import math
import os

import numpy as np
import pytest
import torch

import synthetic_inputs as si
from oracle import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sequence_transformer_gemms_amd", "libtpmlp.so")
needs_lib = pytest.mark.skipif(not os.path.exists(LIB), reason="libtpmlp.so not built")
FAKE = 1 << 20  # a non-null, 16-byte-aligned address that is never dereferenced
ACTS = [ops.ACT_NONE, ops.ACT_RELU, ops.ACT_GELU_ERF, ops.ACT_GELU_TANH, ops.ACT_SILU]


@pytest.mark.parametrize("act", ACTS)
def test_oracle_forward_by_scalar_arithmetic(act):
    x, w, b, r = (si.normal_f32(s, k).astype(np.float64) for s, k in (((3, 4), 1), ((4, 5), 2), ((5,), 3), ((3, 5), 4)))
    out = ops.linear_fwd(x, w, b, act, r, scale=0.5)
    for i in range(3):
        for j in range(5):
            z = 0.5 * math.fsum(x[i, k] * w[k, j] for k in range(4)) + b[j]
            y = {ops.ACT_NONE: z, ops.ACT_RELU: max(z, 0.0), ops.ACT_GELU_ERF: 0.5 * z * (1 + math.erf(z / math.sqrt(2))),
                 ops.ACT_GELU_TANH: 0.5 * z * (1 + math.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))),
                 ops.ACT_SILU: z / (1 + math.exp(-z))}[act] + r[i, j]
            assert abs(out["Z"][i, j] - z) < 1e-13 and abs(out["Y"][i, j] - y) < 1e-13


@pytest.mark.parametrize("act", ACTS)
def test_oracle_backward_matches_differences(act):
    # central differences with step 1e-5: truncation of order 1e-10, rounding
    # of order 1e-16 / 1e-5
    x, w, b, dy = (si.normal_f32(s, 20 + k).astype(np.float64) for k, s in enumerate([(4, 3), (3, 5), (5,), (4, 5)]))
    f = ops.linear_fwd(x, w, b, act)
    out = ops.linear_act_bwd(x, w, dy, f["Z"], act)
    loss = lambda *a: float((ops.linear_fwd(a[0], a[1], a[2], act)["Y"] * dy).sum())  # noqa: E731
    for k, name in enumerate(("dX", "dW", "dbias")):
        args = [x, w, b]
        for idx in np.ndindex(args[k].shape):
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[k][idx] += 1e-5
            lo[k][idx] -= 1e-5
            assert abs((loss(*hi) - loss(*lo)) / 2e-5 - out[name][idx]) < 1e-7


def _fwd(**kw):
    from sequence_transformer_gemms_amd import _abi as X
    a = dict(M=256, N=256, K=256, x=FAKE, ldx=256, xs=None, w=FAKE, ldw=256, tw=0, ws=None, dt=X.BF16, b=None, bdt=X.BF16,
             r=None, ldr=0, act=0, z=None, ldz=0, y=FAKE, ldy=256, ydt=X.BF16, C=1, order=None, ready=None, epoch=0,
             wk=None, wkb=0)
    a.update(kw)
    return X.lib.tp_linear_fwd(a["M"], a["N"], a["K"], a["x"], a["ldx"], a["xs"], a["w"], a["ldw"], a["tw"], a["ws"], a["dt"],
                               a["b"], a["bdt"], a["r"], a["ldr"], a["act"], a["z"], a["ldz"], a["y"], a["ldy"], a["ydt"],
                               a["C"], a["order"], a["ready"], a["epoch"], a["wk"], a["wkb"], None)


def _bwd(**kw):
    from sequence_transformer_gemms_amd import _abi as X
    a = dict(M=256, N=256, K=256, x=FAKE, ldx=256, w=FAKE, ldw=256, z=FAKE, ldz=256, dy=FAKE, lddy=256, dt=X.BF16, act=2,
             dw=FAKE, lddw=256, dwdt=X.BF16, dx=FAKE, lddx=256, db=None, wk=FAKE, wkb=1 << 40)
    a.update(kw)
    return X.lib.tp_linear_act_bwd(a["M"], a["N"], a["K"], a["x"], a["ldx"], a["w"], a["ldw"], a["z"], a["ldz"], a["dy"],
                                   a["lddy"], a["dt"], a["act"], a["dw"], a["lddw"], a["dwdt"], a["dx"], a["lddx"], a["db"],
                                   a["wk"], a["wkb"], None)


@needs_lib
def test_forward_refusals():
    from sequence_transformer_gemms_amd import _abi as X
    E, U = X.EINVAL, X.EUNSUPPORTED
    assert _fwd(M=-1) == E and _fwd(N=-1) == E and _fwd(K=-1) == E
    assert _fwd(dt=X.FP8_E5M2) == E and _fwd(dt=7) == E and _fwd(ydt=X.FP8_E4M3) == E
    assert _fwd(b=FAKE, bdt=X.FP8_E4M3) == E and _fwd(act=5) == E and _fwd(act=-1) == E
    assert _fwd(ldx=255) == E and _fwd(ldw=255) == E and _fwd(ldy=255) == E
    assert _fwd(r=FAKE, ldr=255) == E and _fwd(z=FAKE, ldz=255) == E
    assert _fwd(x=None) == E and _fwd(w=None) == E and _fwd(y=None) == E
    assert _fwd(C=3) == E and _fwd(C=2, order=X.int_array([0, 0])) == E
    assert _fwd(dt=X.F32, ydt=X.BF16) == U
    assert _fwd(wk=FAKE + 8, wkb=1 << 20) == E
    assert _fwd(ready=FAKE) == X.EWORKSPACE
    assert _fwd(ready=FAKE, wk=FAKE, wkb=1 << 20, K=260, ldx=260) == U                  # no whole chunks: no gating
    assert _fwd(ready=FAKE, wk=FAKE, wkb=1 << 20, b=FAKE + 2) == U
    assert _fwd(dt=X.FP8_E4M3, tw=0) == U
    assert "tp_linear_fwd" in X.last_error()
    assert _fwd(M=0) == X.OK and _fwd(N=0, ldw=0, ldy=0) == X.OK


@needs_lib
def test_backward_refusals():
    from sequence_transformer_gemms_amd import _abi as X
    E = X.EINVAL
    assert _bwd(M=-1) == E and _bwd(dt=X.FP8_E4M3) == E and _bwd(dwdt=X.FP8_E4M3) == E and _bwd(act=9) == E
    assert _bwd(z=None) == E and "pre-activation" in X.last_error()
    for name in ("x", "w", "dy", "dw", "dx"):
        assert _bwd(**{name: None}) == E, name
    for name in ("ldx", "ldw", "ldz", "lddy", "lddw", "lddx"):
        assert _bwd(**{name: 255}) == E, name
    assert _bwd(dt=X.F32, dwdt=X.BF16) == X.EUNSUPPORTED
    need = X.lib.tpm_workspace_bytes(X.OP_LINEAR_ACT_BWD, 256, 256, 256, 1, 1, X.BF16)
    assert _bwd(wkb=need - 1) == X.EWORKSPACE and _bwd(wk=None) == X.EWORKSPACE and _bwd(wk=FAKE + 4) == E
    assert _bwd(M=0, N=0, K=0, x=None, w=None, z=None, dy=None, dw=None, dx=None, ldx=0, ldw=0, ldz=0, lddy=0, lddw=0, lddx=0) == X.OK


@needs_lib
def test_workspaces():
    from sequence_transformer_gemms_amd import _abi as X
    ws = lambda op, M, N, K, dt: X.lib.tpm_workspace_bytes(op, M, N, K, 1, 1, dt)  # noqa: E731
    # one row: 20 strips of 64 columns, K = 8192 in 32 ranges of one 256-step
    assert ws(X.OP_LINEAR_FWD, 1, 1280, 8192, X.BF16) >= 2048 + 32 * 1280 * 4
    # a full chip of tiles: nothing is split
    assert ws(X.OP_LINEAR_FWD, 8192, 8192, 8192, X.BF16) == 2048
    # the backward keeps dZ
    assert ws(X.OP_LINEAR_ACT_BWD, 4096, 3584, 8192, X.BF16) >= 2048 + 4096 * 3584 * 2
    assert ws(X.OP_LINEAR_ACT_BWD, 4096, 3584, 8192, X.F32) >= 2048 + 4096 * 3584 * 4


@needs_lib
def test_binding_refusals():
    import sequence_transformer_gemms_amd as tpm
    x, w, y = torch.zeros(4, 8), torch.zeros(8, 16), torch.empty(4, 16)
    with pytest.raises(ValueError, match="GPU memory"):
        tpm.tp_linear_fwd(x, w, y)
    with pytest.raises(ValueError, match="W has shape"):
        tpm.tp_linear_fwd(x, w.t().contiguous(), y)
    with pytest.raises(ValueError, match="W has dtype"):
        tpm.tp_linear_fwd(x, w.bfloat16(), y)
    with pytest.raises(ValueError, match="bias has shape"):
        tpm.tp_linear_fwd(x, w, y, bias=torch.zeros(4))
    with pytest.raises(ValueError, match="residual has dtype"):
        tpm.tp_linear_fwd(x, w, y, residual=y.bfloat16())
    with pytest.raises(ValueError, match="unit inner stride"):
        tpm.tp_linear_fwd(x, torch.zeros(16, 8).t(), y)
    with pytest.raises(ValueError, match="dW has shape"):
        tpm.tp_linear_act_bwd(x, w, y, torch.empty(16, 8), torch.empty(4, 8))
    with pytest.raises(ValueError, match="dbias has dtype"):
        tpm.tp_linear_act_bwd(x, w, y, torch.empty(8, 16), torch.empty(4, 8), dbias=torch.empty(16, dtype=torch.bfloat16))


@needs_lib
def test_size_limit():
    from sequence_transformer_gemms_amd import _abi as X
    big = 2**27 + 1
    assert _fwd(M=big) == _fwd(N=big, ldw=big, ldy=big) == _fwd(K=big, ldx=big) == X.EUNSUPPORTED
    assert _bwd(M=big) == _bwd(N=big, ldw=big, ldz=big, lddy=big, lddw=big) == _bwd(K=big, ldx=big, lddx=big) == X.EUNSUPPORTED
