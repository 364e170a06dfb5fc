"""The operators of a rank's layer together, as a training or serving step
uses them: row-parallel products with their bias held back, the token slice's
sum, bias, residual and norm, the next column-parallel product (bf16, e4m3
under delayed scaling, MXFP8), and the way back.  Each step is compared with
the float64 oracle on the values the GPU stored before it, at the bars of the
other parity tests (max |gpu - ref| / (1 + |ref|): 2e-2 bf16, 6e-2 fp8).

The weight and input gradients read dZ as the backward stored it in bf16,
which the call does not return, so they are held to that rounding's bound
instead: dZ is off by e = 2^-8 |dZ| (half a bf16 step) plus the derivative's
own 1e-5 |dZ| + 3e-7 |dY|, a product X^T dZ hence by |X|^T e plus its fp32
summation of n terms, (n + 4) 2^-24 |X|^T (|dZ| + e), and the result's own
rounding by 2^-8 of it."""
import numpy as np
import pytest
import torch

import synthetic_inputs as si
from oracle import formats, ops
from tests._util import TOL, f64, nerr

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sequence_transformer_gemms_amd as tpm
    from sequence_transformer_gemms_amd import _abi

B, F = torch.bfloat16, torch.float32
T, M, D, HID, FF = 4, 256, 512, 512, 2048
SLICE, FT, HT = M // T, FF // T, HID // T


def bf(shape, seed, sigma=1.0):
    return si.to_bf16(si.normal_f32(shape, seed, sigma)).cuda()


def new(*shape, dtype=B):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda") if dtype != torch.uint8 else \
        torch.full(shape, 0x7F, dtype=dtype, device="cuda")


@pytest.fixture(scope="module")
def layer():
    s = dict(att=[bf((M, HT), 10 + t) for t in range(T)], wo=[bf((HT, D), 20 + t, 0.05) for t in range(T)],
             bo=bf((D,), 1, 0.2), res=bf((M, D), 2), gamma=(1 + 0.1 * bf((D,), 3)).to(B), eps=1e-5)
    s["P"] = new(T, M, D)
    for t in range(T):     # every rank's partial of the output projection: no bias, no residual
        tpm.tp_linear_fwd(s["att"][t], s["wo"][t], s["P"][t])
    torch.cuda.synchronize()
    for t in range(T):
        assert nerr(s["P"][t], ops.linear_fwd(f64(s["att"][t]), f64(s["wo"][t]))["Y"]) <= TOL["bf16"]
    return s


def close_products(dW, dX, x, w, dy, back, act):
    e = 2.0 ** -8 * np.abs(back["dZ"]) * 1.0001 + 1e-5 * np.abs(back["dZ"]) + 3e-7 * np.abs(dy)
    if act == ops.ACT_NONE:
        e = 0 * e                                    # dZ is dY as given
    u, big = 2.0 ** -24, np.abs(back["dZ"]) + e
    for got, ref, err in ((dW, back["dW"], np.abs(x).T @ e + (x.shape[0] + 4) * u * (np.abs(x).T @ big)),
                          (dX, back["dX"], e @ np.abs(w).T + (w.shape[1] + 4) * u * (big @ np.abs(w).T))):
        assert np.all(np.abs(f64(got) - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err) + 2.0 ** -133)


def norm(s, rank, y, **fp8):
    rows = slice(rank * SLICE, (rank + 1) * SLICE)
    h, rstd = new(SLICE, D), new(SLICE, dtype=F)
    tpm.tp_rmsnorm_fwd(s["P"][:, rows], s["gamma"], y, bias=s["bo"], residual=s["res"][rows], h=h, rstd=rstd, eps=s["eps"], **fp8)
    ref = ops.rmsnorm_fwd(f64(s["P"][:, rows]), f64(s["gamma"]), s["eps"], f64(s["bo"]), f64(s["res"][rows]))
    torch.cuda.synchronize()
    assert nerr(h, ref["h"]) <= TOL["bf16"] and nerr(rstd, ref["rstd"]) <= TOL["f32"]
    return h, rstd, ref["y"]


def test_slices_make_the_whole_sum_with_one_bias(layer):
    # over all ranks the slices are the residual plus every partial plus the bias once
    hs = [norm(layer, r, new(SLICE, D))[0] for r in range(T)]
    whole = f64(layer["P"]).sum(0) + f64(layer["bo"]) + f64(layer["res"])
    assert nerr(torch.cat(hs), whole) <= TOL["bf16"]


def test_training_step(layer):
    s = layer
    y = new(M, D)                                    # the all-gathered input of the next product
    saved = []
    for r in range(T):
        h, rstd, ref = norm(s, r, y[r * SLICE:(r + 1) * SLICE])
        assert nerr(y[r * SLICE:(r + 1) * SLICE], ref) <= TOL["bf16"]
        saved.append((h, rstd))
    # column-parallel up-projection of each rank with its bias, and the way back to its partial dX
    dX = new(T, M, D)
    for t in range(T):
        w, b, dh = bf((D, FT), 40 + t, 0.05), bf((FT,), 50 + t, 0.2), bf((M, FT), 60 + t)
        Z, H = new(M, FT), new(M, FT)
        tpm.tp_linear_fwd(y, w, H, bias=b, act=tpm.ACT_GELU_ERF, Z=Z)
        dW, db = new(D, FT), new(FT, dtype=F)
        tpm.tp_linear_act_bwd(y, w, dh, dW, dX[t], Z=Z, act=tpm.ACT_GELU_ERF, dbias=db)
        torch.cuda.synchronize()
        ref = ops.linear_fwd(f64(y), f64(w), f64(b), ops.ACT_GELU_ERF)
        assert nerr(Z, ref["Z"]) <= TOL["bf16"] and nerr(H, ref["Y"]) <= TOL["bf16"]
        back = ops.linear_act_bwd(f64(y), f64(w), f64(dh), f64(Z), ops.ACT_GELU_ERF)
        close_products(dW, dX[t], f64(y), f64(w), f64(dh), back, ops.ACT_GELU_ERF)
        assert nerr(db, back["dbias"]) <= TOL["f32"]
    # each rank's slice of the norm's backward, and of the row-parallel products behind it
    dP = new(M, D)
    dgamma, dbias = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
    want = dict(dgamma=0.0, dbias=0.0)
    for r in range(T):
        rows = slice(r * SLICE, (r + 1) * SLICE)
        h, rstd = saved[r]
        dres, dg, db = bf((SLICE, D), 70 + r), new(D, dtype=F), new(D, dtype=F)
        tpm.tp_rmsnorm_bwd(dX[:, rows], h, rstd, s["gamma"], dP[rows], dres=dres, dgamma=dg, dbias=db)
        torch.cuda.synchronize()
        ref = ops.rmsnorm_bwd(f64(dX[:, rows]), f64(h), f64(rstd), f64(s["gamma"]), f64(dres))
        assert nerr(dP[rows], ref["dh"]) <= TOL["bf16"]
        dgamma += dg
        dbias += db
        for k in want:
            want[k] = want[k] + ref[k]
    assert nerr(dgamma, want["dgamma"]) <= TOL["bf16"] and nerr(dbias, want["dbias"]) <= TOL["bf16"]
    for t in range(T):
        dW, dA = new(HT, D), new(M, HT)
        tpm.tp_linear_act_bwd(s["att"][t], s["wo"][t], dP, dW, dA)
        torch.cuda.synchronize()
        back = ops.linear_act_bwd(f64(s["att"][t]), f64(s["wo"][t]), f64(dP))
        close_products(dW, dA, f64(s["att"][t]), f64(s["wo"][t]), f64(dP), back, ops.ACT_NONE)


def test_delayed_scaling_feeds_the_fp8_mlp(layer):
    # two steps: the second step's scale is the library's update from the first one's amax
    s = layer
    wu, wd = si.normal_f32((D, FT), 80, 0.05), si.normal_f32((FT, D), 81, 0.05)
    wuq, su = si.to_e4m3_current(np.ascontiguousarray(wu.T))
    wdq, sd = si.to_e4m3_current(np.ascontiguousarray(wd.T))
    hist = torch.zeros(2, device="cuda")
    x_scale = torch.full((1,), 2.0 ** -6, device="cuda")
    for step in range(2):
        codes = new(M, D, dtype=torch.uint8)
        part = torch.empty(1, device="cuda")
        for r in range(T):
            norm(s, r, codes[r * SLICE:(r + 1) * SLICE], y_scale=x_scale, amax_out=part)
            hist[step] = torch.maximum(hist[step], part[0])
        sx = float(x_scale)
        scales = torch.tensor([sx, su, sd], dtype=F, device="cuda")
        H, P, hs = new(M, FT, dtype=torch.uint8), new(M, D), torch.full((1,), 0.05, device="cuda")
        tpm.tp_mlp_fwd_delayed(codes, wuq.cuda(), wdq.cuda(), H, P, T=T, rank=0, scales=scales, h_scale=hs, act=tpm.ACT_GELU_ERF)
        torch.cuda.synchronize()
        ref = ops.tp_mlp_fwd_fp8_delayed(f64(codes), sx, f64(wuq).T, su, f64(wdq).T, sd, 0.05, ops.ACT_GELU_ERF)
        assert np.mean(H.cpu().numpy() != ref["Hq_codes"]) < 1e-2
        assert nerr(P, ref["P"]) <= TOL["fp8"]
        tpm.fp8_delayed_scale(hist, x_scale)
        torch.cuda.synchronize()
        assert float(x_scale) == float(np.float32(np.float32(float(hist.max())) / np.float32(448)))
    assert np.abs(formats.e4m3_to_f64(codes.cpu().numpy())).max() >= 416        # the updated scale uses the range


def test_mxfp8_feeds_the_mx_mlp(layer):
    s = layer
    codes = new(M, D, dtype=torch.uint8)
    scales = new(tpm.mx_scales_bytes(M, D), dtype=torch.uint8)
    per = tpm.mx_scales_bytes(SLICE, D)                 # a slice of whole 32-row groups is contiguous
    assert SLICE % 32 == 0 and per * T == scales.numel()
    for r in range(T):
        norm(s, r, codes[r * SLICE:(r + 1) * SLICE], y_scales=scales[r * per:(r + 1) * per])
    uc, ue = si.to_mxfp8(si.normal_f32((FT, D), 90, 0.05))
    dc, de = si.to_mxfp8(si.normal_f32((D, FT), 91, 0.05))
    H, Hs, P = new(M, FT, dtype=torch.uint8), new(tpm.mx_scales_bytes(M, FT), dtype=torch.uint8), new(M, D)
    tpm.tp_mlp_fwd_mx(codes, scales, uc.cuda(), tpm.mx_swizzle_scales(ue.cuda(), D), dc.cuda(), tpm.mx_swizzle_scales(de.cuda(), FT),
                      H, Hs, P, T=T, rank=0, act=tpm.ACT_GELU_ERF)
    torch.cuda.synchronize()
    xe = scales.cpu().numpy().reshape(-1, D // 128, 32, 4).transpose(0, 2, 1, 3).reshape(M, D // 32)
    ref = ops.tp_mlp_fwd_mx(codes.cpu().numpy(), xe, uc.numpy(), ue.numpy(), dc.numpy(), de.numpy(), ops.ACT_GELU_ERF)
    assert nerr(P, ref["P"]) <= TOL["fp8"]


def test_decoding_step(layer):
    # one token through the output projection with its bias and residual on
    # one rank (T = 1), the norm, and the next projection
    s = layer
    a, wo = bf((1, HID), 100), bf((HID, D), 101, 0.05)
    h, y, rstd = new(1, D), new(1, D), new(1, dtype=F)
    tpm.tp_linear_fwd(a, wo, h, bias=s["bo"], residual=s["res"][:1])
    tpm.tp_rmsnorm_fwd(h, s["gamma"], y, rstd=rstd, eps=s["eps"])
    w, b, q = bf((D, 3 * HT), 102, 0.05), bf((3 * HT,), 103), new(1, 3 * HT)
    tpm.tp_linear_fwd(y, w, q, bias=b)
    torch.cuda.synchronize()
    assert nerr(h, ops.linear_fwd(f64(a), f64(wo), f64(s["bo"]), residual=f64(s["res"][:1]))["Y"]) <= TOL["bf16"]
    assert nerr(y, ops.rmsnorm_fwd(f64(h)[None], f64(s["gamma"]), s["eps"])["y"]) <= TOL["bf16"]
    assert nerr(q, ops.linear_fwd(f64(y), f64(w), f64(b))["Y"]) <= TOL["bf16"]


def test_two_streams_at_once():
    # two sets of arrays and workspaces, their calls interleaved on two streams
    def make(k):
        d = dict(x=bf((2, 300, D), 200 + k), g=bf((D,), 210 + k), w=bf((D, 264), 220 + k, 0.05), b=bf((264,), 230 + k),
                 h=new(300, D), y=new(300, D), rstd=new(300, dtype=F), Y=new(300, 264), Z=new(300, 264), dW=new(D, 264), dX=new(300, D),
                 db=new(264, dtype=F), dh=new(300, D), dg=new(D, dtype=F))
        d["ws"] = [tpm.alloc_workspace(tpm.OP_LINEAR_FWD, 300, 264, D), tpm.alloc_workspace(tpm.OP_LINEAR_ACT_BWD, 300, 264, D),
                   tpm.alloc_workspace(tpm.OP_RMSNORM_BWD, 300, D, 0)]
        return d

    def step(d, st):
        tpm.tp_rmsnorm_fwd(d["x"], d["g"], d["y"], h=d["h"], rstd=d["rstd"], stream=st)
        tpm.tp_linear_fwd(d["y"], d["w"], d["Y"], bias=d["b"], act=tpm.ACT_SILU, Z=d["Z"], workspace=d["ws"][0], stream=st)
        tpm.tp_linear_act_bwd(d["y"], d["w"], d["Y"], d["dW"], d["dX"], Z=d["Z"], act=tpm.ACT_SILU, dbias=d["db"],
                              workspace=d["ws"][1], stream=st)
        tpm.tp_rmsnorm_bwd(d["dX"], d["h"], d["rstd"], d["g"], d["dh"], dgamma=d["dg"], workspace=d["ws"][2], stream=st)

    keys = ("h", "y", "rstd", "Y", "Z", "dW", "dX", "db", "dh", "dg")
    sets, want = [make(0), make(1)], []
    for d in sets:
        step(d, None)
        torch.cuda.synchronize()
        want.append([d[k].clone() for k in keys])
        for k in keys:
            d[k].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for d, st in zip(sets, streams):
            step(d, st)
    torch.cuda.synchronize()
    for d, ref in zip(sets, want):
        assert all(torch.equal(d[k], r) for k, r in zip(keys, ref))
