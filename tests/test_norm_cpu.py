"""The token-slice norm's oracle pinned by differences, and the entry
points' refusals (no GPU: every refused call fails before any HIP call)."""
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


def test_oracle_forward_by_scalar_arithmetic():
    p = si.normal_f32((3, 4, 5), 1).astype(np.float64)
    b, r, g = (si.normal_f32(s, k).astype(np.float64) for s, k in (((5,), 2), ((4, 5), 3), ((5,), 4)))
    out = ops.rmsnorm_fwd(p, g, 1e-3, b, r)
    for i in range(4):
        v = [math.fsum([p[0, i, j], p[1, i, j], p[2, i, j], b[j], r[i, j]]) for j in range(5)]
        q = 1.0 / math.sqrt(math.fsum(t * t for t in v) / 5 + 1e-3)
        assert np.allclose(out["h"][i], v, rtol=1e-14)
        assert abs(out["rstd"][i] - q) <= 1e-14 * q
        assert np.allclose(out["y"][i], [v[j] * q * g[j] for j in range(5)], rtol=1e-13)


def test_oracle_backward_matches_differences():
    # the derivative of sum(y * dy) + sum(h * dres) by central differences:
    # step 1e-5 leaves a truncation error of order 1e-10 and a rounding error
    # of order 1e-16 / 1e-5
    T, rows, D, eps = 2, 3, 7, 1e-2
    p, b, r, g, dy, dres = (si.normal_f32(s, 10 + k).astype(np.float64) for k, s in enumerate(
        [(T, rows, D), (D,), (rows, D), (D,), (T, rows, D), (rows, D)]))

    def loss(p_, b_, r_, g_):
        o = ops.rmsnorm_fwd(p_, g_, eps, b_, r_)
        return float((o["y"] * dy.sum(0)).sum() + (o["h"] * dres).sum())

    f = ops.rmsnorm_fwd(p, g, eps, b, r)
    out = ops.rmsnorm_bwd(dy, f["h"], f["rstd"], g, dres)

    def numeric(k):
        args = [p, b, r, g]
        grad = np.zeros_like(args[k])
        for idx in np.ndindex(grad.shape):
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[k][idx] += 1e-5
            lo[k][idx] -= 1e-5
            grad[idx] = (loss(*hi) - loss(*lo)) / 2e-5
        return grad

    dp = numeric(0)
    assert np.allclose(dp[0], out["dh"], atol=1e-8) and np.allclose(dp[1], out["dh"], atol=1e-8)
    assert np.allclose(numeric(1), out["dbias"], atol=1e-8)
    assert np.allclose(numeric(2), out["dh"], atol=1e-8)
    assert np.allclose(numeric(3), out["dgamma"], atol=1e-8)


def _fwd(**kw):
    from sequence_transformer_gemms_amd import _abi as X
    a = dict(T=1, rows=4, D=256, x=FAKE, stride=0, ldx=256, xdt=X.BF16, bias=None, gamma=FAKE, gdt=X.BF16, eps=1e-5,
             res=None, ldr=0, h=None, ldh=0, hdt=X.BF16, rstd=None, y=FAKE, ldy=256, ydt=X.BF16, mx=None, ysc=None, amax=None)
    a.update(kw)
    return X.lib.tp_rmsnorm_fwd(a["T"], a["rows"], a["D"], a["x"], a["stride"], a["ldx"], a["xdt"], a["bias"], a["gamma"],
                                a["gdt"], a["eps"], a["res"], a["ldr"], a["h"], a["ldh"], a["hdt"], a["rstd"], a["y"],
                                a["ldy"], a["ydt"], a["mx"], a["ysc"], a["amax"], None)


def _bwd(**kw):
    from sequence_transformer_gemms_amd import _abi as X
    a = dict(T=1, rows=4, D=256, dy=FAKE, stride=0, lddy=256, dydt=X.BF16, gamma=FAKE, gdt=X.BF16, h=FAKE, ldh=256,
             rstd=FAKE, dres=None, ldr=0, hdt=X.BF16, dh=FAKE, lddh=256, dhdt=X.BF16, dg=None, db=None, ws=None, wsb=0)
    a.update(kw)
    return X.lib.tp_rmsnorm_bwd(a["T"], a["rows"], a["D"], a["dy"], a["stride"], a["lddy"], a["dydt"], a["gamma"], a["gdt"],
                                a["h"], a["ldh"], a["rstd"], a["dres"], a["ldr"], a["hdt"], a["dh"], a["lddh"], a["dhdt"],
                                a["dg"], a["db"], a["ws"], a["wsb"], None)


@needs_lib
def test_forward_refusals():
    from sequence_transformer_gemms_amd import _abi as X
    E, U = X.EINVAL, X.EUNSUPPORTED
    assert _fwd(rows=-1) == E and _fwd(D=-1) == E and _fwd(D=0, ldx=0, ldy=0) == E
    assert _fwd(T=0) == E and _fwd(T=257) == E and _fwd(T=2, stride=-1) == E
    assert _fwd(xdt=X.FP8_E4M3) == E and _fwd(hdt=X.FP8_E4M3) == E and _fwd(gdt=X.FP8_E5M2) == E
    assert _fwd(ydt=X.FP8_E5M2) == E and _fwd(eps=-1.0) == E and _fwd(eps=float("nan")) == E
    assert _fwd(ldx=255) == E and _fwd(ldy=255) == E and _fwd(res=FAKE, ldr=255) == E and _fwd(h=FAKE, ldh=255) == E
    assert _fwd(x=None) == E and _fwd(gamma=None) == E and _fwd(y=None) == E
    assert _fwd(ydt=X.FP8_E4M3) == E                                   # neither scale form
    assert _fwd(ydt=X.FP8_E4M3, mx=FAKE, ysc=FAKE) == E                # both
    assert _fwd(ysc=FAKE) == E and _fwd(mx=FAKE) == E                  # scales without fp8 codes
    assert _fwd(ydt=X.FP8_E4M3, mx=FAKE, amax=FAKE) == E               # an amax goes with a fixed scale
    assert _fwd(ydt=X.FP8_E4M3, mx=FAKE, D=200, ldx=200, ldy=200) == U
    assert _fwd(rows=2**31) == U
    assert "tp_rmsnorm_fwd" in X.last_error()
    assert _fwd(rows=0, x=None, gamma=None, y=None) == X.OK            # nothing to do, nothing enqueued


@needs_lib
def test_backward_refusals():
    from sequence_transformer_gemms_amd import _abi as X
    E = X.EINVAL
    assert _bwd(rows=-1) == E and _bwd(T=0) == E and _bwd(dydt=X.FP8_E4M3) == E and _bwd(dhdt=X.FP8_E4M3) == E
    assert _bwd(lddy=8) == E and _bwd(ldh=8) == E and _bwd(lddh=8) == E and _bwd(dres=FAKE, ldr=8) == E
    for name in ("dy", "gamma", "h", "rstd", "dh"):
        assert _bwd(**{name: None}) == E, name
    need = X.lib.tpm_workspace_bytes(X.OP_RMSNORM_BWD, 4, 256, 0, 1, 1, X.BF16)
    assert need > 0
    assert _bwd(dg=FAKE) == X.EWORKSPACE
    assert _bwd(db=FAKE, ws=FAKE, wsb=need - 1) == X.EWORKSPACE
    assert "tp_rmsnorm_bwd" in X.last_error()
    assert _bwd(rows=0) == X.OK


@needs_lib
def test_binding_refusals():
    import sequence_transformer_gemms_amd as tpm
    x, g = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(ValueError, match="GPU memory"):
        tpm.tp_rmsnorm_fwd(x, g, torch.empty(4, 8))
    with pytest.raises(ValueError, match="gamma has shape"):
        tpm.tp_rmsnorm_fwd(x, torch.ones(7), torch.empty(4, 8))
    with pytest.raises(ValueError, match="y has shape"):
        tpm.tp_rmsnorm_fwd(x, g, torch.empty(4, 9))
    with pytest.raises(ValueError, match="unit inner stride"):
        tpm.tp_rmsnorm_fwd(torch.zeros(8, 4).t(), g, torch.empty(4, 8))
    with pytest.raises(ValueError, match="dtype"):
        tpm.tp_rmsnorm_fwd(x.half(), g, torch.empty(4, 8))
    with pytest.raises(ValueError, match="h has dtype"):
        tpm.tp_rmsnorm_fwd(x, g, torch.empty(4, 8), residual=x, h=torch.empty(4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="mx_scales_bytes"):
        tpm.tp_rmsnorm_fwd(torch.zeros(4, 128), torch.ones(128), torch.empty(4, 128, dtype=torch.uint8),
                           y_scales=torch.empty(4, dtype=torch.uint8))
    with pytest.raises(ValueError, match=r"\[T, rows, D\]"):
        tpm.tp_rmsnorm_fwd(torch.zeros(8), g, torch.empty(8))
    with pytest.raises(ValueError, match="rstd has dtype"):
        tpm.tp_rmsnorm_bwd(x, x, torch.ones(4, dtype=torch.bfloat16), g, torch.empty(4, 8))
    with pytest.raises(ValueError, match="dres has dtype"):
        tpm.tp_rmsnorm_bwd(x, x, torch.ones(4), g, torch.empty(4, 8), dres=torch.zeros(4, 8, dtype=torch.bfloat16))


@needs_lib
def test_limits_and_workspace_alignment():
    """Rows past 2^27 elements and a backward workspace off 16 bytes are
    refused before anything is enqueued."""
    from sequence_transformer_gemms_amd import _abi as X
    D = 2**27 + 1
    assert _fwd(D=D, ldx=D, ldy=D) == X.EUNSUPPORTED
    assert _bwd(D=D, lddy=D, ldh=D, lddh=D) == X.EUNSUPPORTED
    assert _bwd(dg=FAKE, ws=FAKE + 4, wsb=1 << 30) == X.EINVAL and "aligned" in X.last_error()
