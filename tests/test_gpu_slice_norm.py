"""The token-slice norm on the GPU against the float64 oracle, element by
element.

Bounds (u = 2^-24, half a step of fp32; a bf16 rounding is off by at most
2^-8 of the value, an e4m3 one by 2^-4, or half its smallest step 2^-10):
  h     the T + 2 addends are summed in fp32: (T + 2) u sum|addends|, then
        one rounding to h's type
  rstd  v's error enters as its share of the row's length; the sum of D
        squares (all positive) in at most ceil(D / 64) + 32 sequential adds
        per path: n u relative, halved by the square root; the mean, the sum
        with eps, the root and the division round once each
  y     (v, r, gamma): the relative errors of v and r, two products, then
        one rounding to y's type
  sums  a dot product of n terms in fp32 with at most m sequential adds per
        path is off by at most (m + 3) u sum|terms|
"""
import numpy as np
import pytest
import torch

import synthetic_inputs as si
from oracle import formats, ops
from tests._util import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sequence_transformer_gemms_amd as tpm
    from sequence_transformer_gemms_amd import _abi

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
TINY = 2.0 ** -133     # half the smallest bf16 / fp32 subnormal step, and more
B, F = torch.bfloat16, torch.float32


def dev(a, dtype, ld=None, offset=0):
    """a [rows, D] (or [T, rows, D]) on the GPU with row stride ld, `offset`
    elements into its allocation; what lies around the rows is NaN."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype)
    if ld is None:
        return t.cuda()
    lead = a.shape[:-1]
    n = int(np.prod(lead))
    buf = torch.full((offset + n * ld,), float("nan"), dtype=dtype, device="cuda")
    v = buf[offset:].view(*lead, ld)[..., :a.shape[-1]]
    v.copy_(t)
    return v


def empty(rows, D, dtype, ld=None, offset=0):
    """An output with guard elements around its rows, and a check that they
    were left alone."""
    ld = ld or D
    fill = 0x5A if dtype == torch.uint8 else -77.0
    buf = torch.full((offset + rows * ld + 64,), fill, dtype=dtype, device="cuda")
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :D]

    def untouched():
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask[offset:offset + rows * ld].view(rows, ld)[:, :D] = False
        return bool((buf[mask] == fill).all())
    return view, untouched


def inputs(T, rows, D, seed, spread=True):
    chan = np.where(np.arange(D) % 97 == 5, 10.0, 1.0) if spread else 1.0
    return dict(p=si.normal_f32((T, rows, D), seed), r=si.normal_f32((rows, D), seed + 1) * chan,
                g=1 + si.normal_f32((D,), seed + 2, 0.1), b=si.normal_f32((D,), seed + 3, 0.1))


def fwd_bounds(P, G, ref, bias, res, T, D, eps):
    """Bounds of the GPU's unrounded v, rstd and y before the storage roundings."""
    mag = np.abs(P).sum(0) + (0 if bias is None else np.abs(bias)) + (0 if res is None else np.abs(res))
    ev = (T + 2) * U * mag
    ss = (ref["h"] ** 2).sum(1)
    n = -(-D // 64) + 32
    # |d(sum v^2)| <= 2 |v|.|ev| + |ev|^2, relative to sum v^2 + D eps
    rel = (2 * (np.abs(ref["h"]) * ev).sum(1) + (ev ** 2).sum(1) + n * U * ss) / (ss + D * eps)
    er = ref["rstd"] * (0.5 * rel * 1.01 + 5 * U)
    ey = (np.abs(G) * (ev * ref["rstd"][:, None] + (np.abs(ref["h"]) + ev) * er[:, None]) + 3 * U * np.abs(ref["y"]))
    return ev, er, ey


def near(got, want, err, dtype):
    g = f64(got) if isinstance(got, torch.Tensor) else got
    tol = err + HALF[dtype] * (np.abs(want) + err) + TINY
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(g - want) / tol)))


SHAPES = [  # T, rows, D
    (1, 1, 1), (1, 3, 2), (2, 5, 7), (1, 1, 64), (3, 33, 127), (1, 65, 128), (2, 31, 1024), (8, 40, 1032), (1, 1, 8192),
    (1, 300, 2048), (8, 17, 8192), (1, 9, 16384), (2, 3, 20000), (1, 2, 33001), (1, 3, 32768), (1, 700, 96), (4, 600, 8),
    (1, 5, 4104), (5, 260, 520),
]
# many rows: other numbers of chunks per thread, rows per work-group and work-groups
LONG = [(1, 5000, 72), (1, 4100, 1031), (8, 530, 2052), (1, 520, 16390), (2, 515, 9000), (1, 4097, 8200)]


@pytest.mark.parametrize("T,rows,D,xdt,hdt,gdt", [s + t for s in SHAPES for t in [(B, B, B), (F, F, F), (B, F, F), (F, B, B)]]
                         + [s + t for s in LONG for t in [(B, B, B), (F, F, F)]])
def test_forward(T, rows, D, xdt, hdt, gdt):
    i = inputs(T, rows, D, 1000 + D)
    x, res, gamma, bias = dev(i["p"], xdt), dev(i["r"], hdt), dev(i["g"], gdt), dev(i["b"], gdt)
    eps = 1e-5
    for use_b, use_r in ((True, True), (False, True), (True, False), (False, False))[:1 if rows > 512 and D > 96 else 4]:
        P, G = f64(x), f64(gamma)
        bb, rr = (f64(bias) if use_b else None), (f64(res) if use_r else None)
        ref = ops.rmsnorm_fwd(P, G, eps, bb, rr)
        h, h_ok = empty(rows, D, hdt)
        y, y_ok = empty(rows, D, xdt)
        rstd = torch.empty(rows, dtype=F, device="cuda")
        tpm.tp_rmsnorm_fwd(x if T > 1 else x[0], gamma, y, bias=bias if use_b else None, residual=res if use_r else None,
                           h=h, rstd=rstd, eps=eps)
        torch.cuda.synchronize()
        ev, er, ey = fwd_bounds(P, G, ref, bb, rr, T, D, eps)
        near(h, ref["h"], ev, hdt)
        near(rstd, ref["rstd"], er, F)
        near(y, ref["y"], ey, xdt)
        assert h_ok() and y_ok()


@pytest.mark.parametrize("T,rows,D", SHAPES)
@pytest.mark.parametrize("dt", [B, F])
def test_e4m3_output_with_a_fixed_scale(T, rows, D, dt):
    i = inputs(T, rows, D, 2000 + D)
    x, gamma = dev(i["p"], dt), dev(i["g"], dt)
    ref = ops.rmsnorm_fwd(f64(x), f64(gamma), 1e-5)
    _, _, ey = fwd_bounds(f64(x), f64(gamma), ref, None, None, T, D, 1e-5)
    for s in (np.float32(4.0 / 448), np.float32(0.5 / 448)):      # the second saturates
        y, y_ok = empty(rows, D, torch.uint8)
        amax = torch.full((1,), 1e30, device="cuda")
        tpm.tp_rmsnorm_fwd(x if T > 1 else x[0], gamma, y, y_scale=torch.tensor([s], device="cuda"), amax_out=amax)
        torch.cuda.synchronize()
        inv = np.float64(np.float32(1) / s)
        # encoding is monotone: every code is that of a value within the bound
        err = ey * inv + U * np.abs(ref["y"] * inv)
        got = formats.e4m3_to_f64(y.cpu().numpy())
        lo = formats.e4m3_to_f64(formats.e4m3_encode(ref["y"] * inv - err))
        hi = formats.e4m3_to_f64(formats.e4m3_encode(ref["y"] * inv + err))
        assert np.all((got >= lo) & (got <= hi))
        assert abs(float(amax) - np.abs(ref["y"]).max()) <= ey.max() + 2 * U * np.abs(ref["y"]).max()
        assert y_ok()


@pytest.mark.parametrize("T,rows,D", [(1, 1, 128), (2, 33, 256), (8, 64, 1024), (1, 5, 8192), (2, 3, 16384), (1, 3, 32768 + 128)])
@pytest.mark.parametrize("dt", [B, F])
def test_mxfp8_output(T, rows, D, dt):
    i = inputs(T, rows, D, 3000 + D)
    i["p"][:, 0, :32] = 0                                          # a block of zeros
    x, gamma, bias = dev(i["p"], dt), dev(i["g"], dt), None
    ref = ops.rmsnorm_fwd(f64(x), f64(gamma), 1e-5)
    _, _, ey = fwd_bounds(f64(x), f64(gamma), ref, None, None, T, D, 1e-5)
    y, y_ok = empty(rows, D, torch.uint8)
    n = tpm.mx_scales_bytes(rows, D)
    scales = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    tpm.tp_rmsnorm_fwd(x if T > 1 else x[0], gamma, y, bias=bias, y_scales=scales[:n])
    torch.cuda.synchronize()
    assert y_ok() and bool((scales[n:] == 0xA5).all())
    sw = scales[:n].cpu().numpy().reshape(-1, D // 128, 32, 4).transpose(0, 2, 1, 3).reshape(-1, D // 32)
    assert np.all(sw[rows:] == 0)
    e = sw[:rows].astype(np.int64)
    blocks = lambda a: a.reshape(rows, D // 32, 32)                # noqa: E731
    lo_e = formats.mx_e4m3_quantize(np.maximum(np.abs(ref["y"]) - ey, 0))[1].astype(np.int64)
    hi_e = formats.mx_e4m3_quantize(np.abs(ref["y"]) + ey)[1].astype(np.int64)
    zero = blocks(np.abs(ref["y"])).max(2) == 0
    assert np.all(e[zero] == 0)
    assert np.all((e >= lo_e) & (e <= hi_e) | zero)
    X = np.repeat(formats.e8m0_to_f64(e), 32, axis=1)
    got = formats.e4m3_to_f64(y.cpu().numpy())
    assert np.all(got >= formats.e4m3_to_f64(formats.e4m3_encode((ref["y"] - ey) / X)))
    assert np.all(got <= formats.e4m3_to_f64(formats.e4m3_encode((ref["y"] + ey) / X)))


def test_strides_offsets_and_a_rank_slice():
    # rows of a [T, M, D] stack, row strides wider than D, arrays that start
    # off a 16-byte boundary, h written over the residual
    T, M, D, rank = 4, 40, 264, 2
    rows = M // T
    i = inputs(T, M, D, 4001)
    full = dev(i["p"], B)
    part = full[:, rank * rows:(rank + 1) * rows]
    P = f64(part)
    for ld, off in ((D, 0), (D + 8, 0), (D + 3, 0), (D, 1), (D + 8, 8)):
        res = dev(i["r"][:rows], B, ld, off)
        gamma = dev(i["g"], B)
        ref = ops.rmsnorm_fwd(P, f64(gamma), 1e-5, None, f64(res))
        ev, _, ey = fwd_bounds(P, f64(gamma), ref, None, f64(res), T, D, 1e-5)
        y, y_ok = empty(rows, D, B, ld, off)
        tpm.tp_rmsnorm_fwd(part, gamma, y, residual=res, h=res)
        torch.cuda.synchronize()
        near(res, ref["h"], ev, B)
        near(y, ref["y"], ey, B)
        assert y_ok()


def test_rows_that_are_zero_infinite_or_nan():
    rows, D = 6, 1024
    i = inputs(1, rows, D, 4100)
    p = i["p"][0]
    p[1] = 0
    p[2, 7] = np.inf
    p[3, 9] = np.nan
    p[4] *= 1e-30                                       # squares below fp32's range: eps alone
    for D_ in (D, D - 1):                               # both kernels
        x, gamma = dev(p[:, :D_], B), dev(i["g"][:D_], B)
        y = torch.empty(rows, D_, dtype=B, device="cuda")
        rstd = torch.empty(rows, device="cuda")
        tpm.tp_rmsnorm_fwd(x, gamma, y, rstd=rstd, eps=1e-5)
        torch.cuda.synchronize()
        Y, X, G = f64(y), f64(x), f64(gamma)
        assert np.all(Y[1] == 0) and abs(float(rstd[1]) - 1e-5 ** -0.5) < 1e-3
        assert np.isnan(Y[2, 7]) and np.all(np.delete(Y[2], 7) == 0)     # x / inf, inf / inf
        assert np.isnan(Y[3]).all()
        for k in (0, 4, 5):
            r = 1 / np.sqrt((X[k] ** 2).mean() + 1e-5)
            assert np.all(np.abs(Y[k] - X[k] * r * G) <= 2.0 ** -7 * np.abs(X[k] * r * G) + TINY)


# ----------------------------------------------------------------- backward
def bwd_check(T, rows, D, xdt, hdt, gdt, use_r, seed, ld=None, off=0, inplace=False):
    i = inputs(T, rows, D, seed)
    dy, dres, gamma = dev(i["p"], xdt), dev(i["r"], hdt, ld, off), dev(i["g"], gdt)
    h = dev(si.normal_f32((rows, D), seed + 9), hdt, ld, off)
    rstd = torch.from_numpy((0.5 + si.uniform_f32((rows,), seed + 8, 0, 1)).astype(np.float32)).cuda()
    H, R, G, DY, DR = f64(h), f64(rstd), f64(gamma), f64(dy), (f64(dres) if use_r else None)
    ref = ops.rmsnorm_bwd(DY, H, R, G, DR)
    dh, dh_ok = (dres, lambda: True) if inplace else empty(rows, D, hdt, ld, off)
    dgamma, dbias = torch.full((D,), 7.0, device="cuda"), torch.full((D,), 7.0, device="cuda")
    args = dict(dres=dres if use_r else None, dgamma=dgamma, dbias=dbias)
    tpm.tp_rmsnorm_bwd(dy if T > 1 else dy[0], h, rstd, gamma, dh, **args)
    torch.cuda.synchronize()
    x = np.abs(H) * R[:, None]
    mag = np.abs(DY).sum(0)
    edy = (T + 2) * U * mag
    g, eg = mag * np.abs(G), (T + 3) * U * mag * np.abs(G)
    n = -(-D // 64) + 32
    m = (g * x).mean(1, keepdims=True)
    em = (eg * x).mean(1, keepdims=True) * 1.01 + (n + 5) * U * m
    edh = R[:, None] * (eg + x * em + 3 * U * (g + x * m)) + 2 * U * (np.abs(DR) if use_r else 0) + U * np.abs(ref["dh"])
    near(dh, ref["dh"], edh, hdt)
    # column sums: at most `rows` sequential adds on any path
    near(dgamma, ref["dgamma"], (edy * x).sum(0) + (rows + 4) * U * (mag * x).sum(0), F)
    near(dbias, ref["dbias"], edh.sum(0) + (rows + 1) * U * (np.abs(ref["dh"]) + edh).sum(0), F)
    assert dh_ok()
    return dh, dgamma, dbias


@pytest.mark.parametrize("T,rows,D,xdt,hdt,gdt", [s + t for s in SHAPES for t in [(B, B, B), (F, F, F), (B, F, F), (F, B, B)]]
                         + [s + t for s in LONG for t in [(B, B, B), (F, F, F)]])
def test_backward(T, rows, D, xdt, hdt, gdt):
    for use_r in (True, False)[:1 if rows > 512 and D > 96 else 2]:
        bwd_check(T, rows, D, xdt, hdt, gdt, use_r, 5000 + D)


def test_backward_strides_and_in_place():
    for ld, off in ((264, 0), (272, 0), (267, 0), (264, 1)):
        bwd_check(4, 10, 264, B, B, B, True, 6001, ld, off)
        bwd_check(4, 10, 264, B, B, B, True, 6001, ld, off, inplace=True)
    # dh over dy
    i = inputs(1, 50, 520, 6100)
    dy, gamma, h = dev(i["p"][0], B), dev(i["g"], B), dev(i["r"], B)
    rstd = torch.ones(50, device="cuda")
    want = torch.empty_like(dy)
    tpm.tp_rmsnorm_bwd(dy, h, rstd, gamma, want)
    tpm.tp_rmsnorm_bwd(dy, h, rstd, gamma, dy)
    torch.cuda.synchronize()
    assert torch.equal(dy, want)


def test_backward_repeats_bit_for_bit_and_long_columns():
    a = bwd_check(1, 3000, 1024, B, B, B, True, 6200)
    b = bwd_check(1, 3000, 1024, B, B, B, True, 6200)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_no_rows():
    D = 640
    e = torch.empty(0, D, dtype=B, device="cuda")
    gamma = torch.ones(D, dtype=B, device="cuda")
    amax = torch.ones(1, device="cuda")
    tpm.tp_rmsnorm_fwd(e, gamma, torch.empty(0, D, dtype=torch.uint8, device="cuda"), y_scale=torch.ones(1, device="cuda"), amax_out=amax)
    dg, db = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
    tpm.tp_rmsnorm_bwd(e, e, torch.empty(0, device="cuda"), gamma, e.clone(), dgamma=dg, dbias=db)
    torch.cuda.synchronize()
    assert float(amax) == 0 and not dg.any() and not db.any()


def test_forward_then_backward_against_differences():
    # the whole step in fp32: the gradient of sum(y * w) along random
    # directions against central differences of the GPU's own forward.  The
    # loss is of order sqrt(rows D) with fp32 rounding errors of order
    # sqrt(rows D) u per term, the step 2^-7 makes them 2^8 u sqrt(rows D) =
    # 2e-3; the truncation error is of order step^2 times third derivatives
    rows, D, step = 16, 264, 2.0 ** -7
    i = inputs(1, rows, D, 6300, spread=False)
    x, gamma, w = dev(i["p"][0], F), dev(i["g"], F), dev(i["r"], F)

    def fwd(v):
        y, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
        tpm.tp_rmsnorm_fwd(v, gamma, y, h=h, rstd=rstd)
        return y, h, rstd
    y, h, rstd = fwd(x)
    dh = torch.empty_like(x)
    tpm.tp_rmsnorm_bwd(w, h, rstd, gamma, dh)
    for k in range(4):
        d = dev(si.normal_f32((rows, D), 6400 + k), F)
        d /= d.norm()
        hi, lo = fwd(x + step * d)[0], fwd(x - step * d)[0]
        numeric = float(((hi.double() - lo.double()) * w.double()).sum()) / (2 * step)
        assert abs(numeric - float((dh.double() * d.double()).sum())) <= 4e-3


def test_other_streams_and_graph_replays():
    rows, D = 64, 1024
    i = inputs(2, rows, D, 6500)
    x, gamma, res = dev(i["p"], B), dev(i["g"], B), dev(i["r"], B)
    y, h = torch.empty(rows, D, dtype=torch.uint8, device="cuda"), torch.empty(rows, D, dtype=B, device="cuda")
    rstd, amax, sc = torch.empty(rows, device="cuda"), torch.empty(1, device="cuda"), torch.full((1,), 0.01, device="cuda")
    dh, dg = torch.empty(rows, D, dtype=B, device="cuda"), torch.empty(D, device="cuda")
    ws = torch.empty(tpm.workspace_bytes(tpm.OP_RMSNORM_BWD, rows, D, 0, 2), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        tpm.tp_rmsnorm_fwd(x, gamma, y, residual=res, h=h, rstd=rstd, y_scale=sc, amax_out=amax, stream=stream)
        tpm.tp_rmsnorm_bwd(x, h, rstd, gamma, dh, dres=res, dgamma=dg, workspace=ws, stream=stream)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (y, h, rstd, amax, dh, dg)]
    step()
    want = results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dg.zero_()
    torch.cuda.synchronize()
    step(side)                                       # given as an argument
    assert all(torch.equal(a, b) for a, b in zip(results(), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(4):
        x.copy_(dev(si.normal_f32((2, rows, D), 6600 + k), B))
        step()
        eager = results()
        for t in (y, h, rstd, amax, dh, dg):
            t.zero_()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), eager))


@pytest.mark.parametrize("rows,D,dt", [(4097, 1300, B), (4100, 2560, B), (4099, 4099, B), (4096, 5500, B), (4097, 6200, B),
                                       (4097, 2560, F), (4097, 4099, F), (4097, 7000, F)])
def test_backward_of_many_rows_of_every_number_of_waves(rows, D, dt):
    bwd_check(1, rows, D, dt, dt, dt, True, 6300 + D, inplace=D == 2560 or D == 4099)


def test_an_infinite_gamma_saturates_the_8_bit_outputs():
    rows, D, c = 5, 256, 70
    i = inputs(1, rows, D, 6400)
    p = i["p"][0]
    p[:, c] = [1.0, -1.0, 2.0 ** -20, -3.0, 0.5]
    x, gamma = dev(p, B), dev(i["g"], B)
    scale = torch.tensor([4.0 / 448], device="cuda")
    out = []
    for g in (float(gamma[c]), float("inf")):
        gamma[c] = g
        y, mx = torch.empty(rows, D, dtype=torch.uint8, device="cuda"), torch.empty(rows, D, dtype=torch.uint8, device="cuda")
        amax = torch.zeros(1, device="cuda")
        tpm.tp_rmsnorm_fwd(x, gamma, y, y_scale=scale, amax_out=amax)
        tpm.tp_rmsnorm_fwd(x, gamma, mx, y_scales=torch.empty(tpm.mx_scales_bytes(rows, D), dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        out.append((formats.e4m3_to_f64(y.cpu().numpy()), formats.e4m3_to_f64(mx.cpu().numpy()), float(amax)))
    sign = np.sign(p[:, c])
    assert np.array_equal(out[1][0][:, c], 448.0 * sign) and np.array_equal(out[1][1][:, c], 448.0 * sign)
    assert out[1][2] == np.inf and np.isfinite(out[0][2])
    assert np.array_equal(np.delete(out[0][0], c, 1), np.delete(out[1][0], c, 1))
    other = np.arange(D) // 32 != c // 32                       # the other blocks of a row
    assert np.array_equal(out[0][1][:, other], out[1][1][:, other])
