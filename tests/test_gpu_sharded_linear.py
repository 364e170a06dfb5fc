"""The linear layer with its fused epilogue on the GPU against the float64
oracle, element by element; bit for bit on integers.

Bounds (u = 2^-24, half a step of fp32; a bf16 rounding is off by at most
2^-8 of the value):
  Z    a dot product of K exact products (bf16 and e4m3 products are exact in
       fp32, fp32 ones round) summed in fp32 in any order, then scale and
       bias: (K + 4) u sum|x w| + 2 u |bias|, then Z's rounding
  Y    |act'| <= 1.13 (the largest slope of the activations) times Z's
       error, the activations' own 1e-5 relative + 3e-7 absolute, the
       residual's addition, then Y's rounding
  dZ   the derivative's own 1e-5 relative + 3e-7 absolute times |dY|, one
       product, then its storage rounding for the two products
  dW, dX   dot products of n terms with inexact dZ: sum|x| |err dZ| + (n + 4)
       u sum|x dZ|, then their rounding
  dbias    sum of err dZ (unrounded) + (M + 4) u sum|dZ|
"""
import numpy as np
import pytest
import torch

import synthetic_inputs as si
from oracle import ops
from tests._util import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sequence_transformer_gemms_amd as tpm
    from sequence_transformer_gemms_amd import _abi

U = 2.0 ** -24
B, F = torch.bfloat16, torch.float32
HALF = {B: 2.0 ** -8, F: U}
TINY = 2.0 ** -133
SLOPE = 1.13
ACTS = [ops.ACT_NONE, ops.ACT_RELU, ops.ACT_GELU_ERF, ops.ACT_GELU_TANH, ops.ACT_SILU]


def dev(a, dtype, ld=None, offset=0):
    """a [rows, cols] on the GPU with row stride ld, `offset` elements into
    its allocation; what lies around the rows is NaN."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype)
    if ld is None and not offset:
        return t.cuda()
    ld = ld or a.shape[-1]
    rows = a.shape[0] if a.ndim == 2 else 1
    buf = torch.full((offset + rows * ld + 16,), float("nan"), dtype=dtype, device="cuda")
    v = buf[offset:offset + rows * ld].view(rows, ld)[:, :a.shape[-1]]
    v.copy_(t)
    return v if a.ndim == 2 else v[0]


def empty(rows, cols, dtype, ld=None, offset=0):
    """An output with guard elements around its rows, and a check that they
    were left alone."""
    ld = ld or cols
    buf = torch.full((offset + rows * ld + 64,), -77.0, dtype=dtype, device="cuda")
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]

    def untouched():
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask[offset:offset + rows * ld].view(rows, ld)[:, :cols] = False
        return bool((buf[mask] == -77.0).all())
    return view, untouched


def near(got, want, err, dtype, what=""):
    g = f64(got)
    tol = err + HALF[dtype] * (np.abs(want) + err) + TINY
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.nanmax(np.abs(g - want) / tol)))


def fwd_check(M, N, K, dt=B, act=ops.ACT_NONE, trans_w=False, bias=True, res=True, save=True, ydt=None, bdt=None, seed=1,
              ld=0, off=0, inplace=False, ws=True, **chunks):
    ydt = ydt or dt
    X = dev(si.normal_f32((M, K), seed), dt, K + ld if ld or off else None, off)
    w = si.normal_f32((K, N), seed + 1, 0.5 / max(K, 1) ** 0.5)
    W = dev(np.ascontiguousarray(w.T) if trans_w else w, dt, (K if trans_w else N) + ld if ld or off else None, off)
    b = dev(si.normal_f32((N,), seed + 2), bdt or dt, None, off) if bias else None
    r = dev(si.normal_f32((M, N), seed + 3), ydt, N + ld if ld or off else None, off) if res else None
    xf, wf = f64(X), (f64(W).T if trans_w else f64(W))
    ref = ops.linear_fwd(xf, wf, None if b is None else f64(b), act, None if r is None else f64(r))
    Y, y_ok = (r, lambda: True) if inplace else empty(M, N, ydt, N + ld, off)
    Z, z_ok = empty(M, N, ydt, N + ld, off)
    work = tpm.alloc_workspace(tpm.OP_LINEAR_FWD, M, N, K, 1, chunks.get("num_chunks", 1), tpm.dtype_code(dt)) if ws else \
        torch.empty(0, dtype=torch.uint8, device="cuda")
    work.fill_(0xFF)                                     # its contents need no preparation
    tpm.tp_linear_fwd(X, W, Y, bias=b, residual=r, act=act, Z=Z if save else None, trans_w=trans_w, workspace=work, **chunks)
    torch.cuda.synchronize()
    ez = (K + 4) * U * (np.abs(xf) @ np.abs(wf)) + (2 * U * np.abs(f64(b)) if bias else 0)
    pre = ops.linear_fwd(xf, wf, None if b is None else f64(b), act)["Y"]
    ey = SLOPE * ez + (1e-5 * np.abs(pre) + 3e-7 if act not in (ops.ACT_NONE, ops.ACT_RELU) else 0)
    ey = ey + 2 * U * np.abs(ref["Y"])
    if save:
        near(Z, ref["Z"], ez, ydt, "Z")
        assert z_ok()
    near(Y, ref["Y"], ey, ydt, "Y")
    assert y_ok()
    return Y


# few rows: every tile height, odd widths, K cut in many ranges
ROWS = [(1, 8, 8), (1, 9, 11), (2, 64, 256), (3, 63, 257), (1, 1280, 8192), (4, 200, 1000), (5, 72, 2057), (8, 130, 520),
        (9, 8, 100), (16, 1288, 264), (17, 77, 300), (33, 264, 512), (64, 100, 1030), (1, 70, 8), (1, 4000, 16)]


@pytest.mark.parametrize("M,N,K", ROWS)
@pytest.mark.parametrize("trans_w", [False, True])
def test_few_rows(M, N, K, trans_w):
    fwd_check(M, N, K, trans_w=trans_w, act=ACTS[(M + N) % 5])
    fwd_check(M, N, K, trans_w=trans_w, act=ACTS[(M + N + 1) % 5], ld=3, off=1, ydt=F, bdt=F)
    fwd_check(M, N, K, trans_w=trans_w, bias=False, res=False, save=False, ws=False)


# whole 16-byte chunks: the 256 x 256 tiles, with split K, a tail split and ragged edges
TILES = [(65, 264, 200), (300, 264, 200), (256, 256, 64), (520, 1288, 1024), (257, 8, 4096), (1000, 512, 8), (4352, 4096, 1024),
         (1100, 1288, 1032), (2056, 520, 2048), (257, 4104, 2048), (2056, 1288, 1032)]


@pytest.mark.parametrize("M,N,K", TILES)
@pytest.mark.parametrize("trans_w", [False, True])
def test_tiles(M, N, K, trans_w):
    for k, (b, r, z) in enumerate(((True, True, True), (True, False, True), (True, True, False), (False, False, False))):
        fwd_check(M, N, K, trans_w=trans_w, act=ACTS[(k + M) % 5], bias=b, res=r, save=z)
        if M > 2000:
            break
    fwd_check(M, N, K, trans_w=trans_w, act=ops.ACT_GELU_ERF, ydt=F, bdt=F, ld=8)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("trans_w", [False, True])
def test_tiles_every_activation(act, trans_w):
    for M, N, K in ((300, 520, 264), (2056, 1288, 1032)):      # small products run on other tiles
        fwd_check(M, N, K, act=act, trans_w=trans_w)
        fwd_check(M, N, K, act=act, trans_w=trans_w, res=False)


# anything else: odd sizes, offsets and strides, fp32
ANY = [(65, 7, 3), (100, 1, 1), (129, 130, 131), (517, 777, 1003), (70, 33, 64), (128, 128, 129), (300, 1001, 72), (1000, 40, 5)]


@pytest.mark.parametrize("M,N,K", ANY)
@pytest.mark.parametrize("dt", [B, F])
@pytest.mark.parametrize("trans_w", [False, True])
def test_any_shape(M, N, K, dt, trans_w):
    fwd_check(M, N, K, dt=dt, trans_w=trans_w, act=ACTS[(M + K) % 5])
    fwd_check(M, N, K, dt=dt, trans_w=trans_w, act=ACTS[(M + K + 2) % 5], ld=5, off=1, bdt=B, ws=False)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 100, 7), (7, 7, 100), (3, 200, 300), (64, 64, 64), (8, 32, 128)])
def test_small_fp32_and_narrow(M, N, K):
    fwd_check(M, N, K, dt=F, act=ops.ACT_SILU)
    fwd_check(M, N, K, dt=B, act=ops.ACT_SILU)


def test_unaligned_arrays_of_whole_chunk_shapes():
    # sizes the tiles take, addresses and strides they do not
    fwd_check(2056, 1288, 1032, off=1)
    fwd_check(2056, 1288, 1032, ld=4, off=4)
    fwd_check(300, 264, 200, off=1)
    fwd_check(300, 264, 200, ld=4, off=4)
    fwd_check(300, 264, 200, ld=1)


def test_empty_contraction_and_empty_outputs():
    fwd_check(5, 24, 0, act=ops.ACT_SILU)
    fwd_check(70, 24, 0, act=ops.ACT_SILU)
    fwd_check(70, 23, 0, dt=F, act=ops.ACT_SILU)
    e = torch.empty(0, 8, dtype=B, device="cuda")
    tpm.tp_linear_fwd(e, torch.empty(8, 16, dtype=B, device="cuda"), torch.empty(0, 16, dtype=B, device="cuda"))
    tpm.tp_linear_fwd(torch.empty(4, 8, dtype=B, device="cuda"), torch.empty(8, 0, dtype=B, device="cuda"),
                      torch.empty(4, 0, dtype=B, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("M,N,K,dt", [(1, 264, 1000, B), (16, 100, 77, B), (300, 264, 200, B), (520, 1288, 1024, B), (2056, 1288, 1032, B), (129, 131, 67, B),
                                      (129, 131, 67, F), (40, 264, 200, F)])
@pytest.mark.parametrize("trans_w", [False, True])
def test_integers_are_exact(M, N, K, dt, trans_w):
    # every product, partial sum and result is an integer below 2^24
    x, w, b, r = (si.small_ints(s, 70 + k) for k, s in enumerate([(M, K), (K, N), (N,), (M, N)]))
    Y, Z = torch.empty(M, N, dtype=F, device="cuda"), torch.empty(M, N, dtype=F, device="cuda")
    tpm.tp_linear_fwd(dev(x, dt), dev(np.ascontiguousarray(w.T) if trans_w else w, dt), Y, bias=dev(b, dt), residual=dev(r, F), Z=Z,
                      act=ops.ACT_RELU, trans_w=trans_w)
    torch.cuda.synchronize()
    ref = ops.linear_fwd(x, w, b, ops.ACT_RELU, r)
    assert np.array_equal(f64(Z), ref["Z"]) and np.array_equal(f64(Y), ref["Y"])


@pytest.mark.parametrize("M,N,K", [(1, 264, 272), (300, 264, 272), (520, 1288, 2048), (4352, 4096, 2048), (1, 1280, 8192), (3, 9, 5),
                                   (33, 70, 250), (129, 131, 67), (1100, 1288, 2064), (1100, 1283, 2061), (2056, 1288, 2064)])
def test_fp8_operands(M, N, K):
    xq, sx = si.to_e4m3_current(si.normal_f32((M, K), 80))
    wq, sw = si.to_e4m3_current(si.normal_f32((N, K), 81, 0.02))
    b, r = dev(si.normal_f32((N,), 82), B), dev(si.normal_f32((M, N), 83), B)
    xf, wf = f64(xq) * float(sx), f64(wq).T * float(sw)
    ref = ops.linear_fwd(xf, wf, f64(b), ops.ACT_GELU_TANH, f64(r))
    Y, y_ok = empty(M, N, B)
    Z, z_ok = empty(M, N, B)
    tpm.tp_linear_fwd(xq.cuda(), wq.cuda(), Y, bias=b, residual=r, act=ops.ACT_GELU_TANH, Z=Z, trans_w=True,
                      x_scale=torch.tensor([sx], device="cuda"), w_scale=torch.tensor([sw], device="cuda"))
    torch.cuda.synchronize()
    # the matrix core may align the products of one instruction to the largest
    # before adding: 2^-13 of the sum of magnitudes covers that step
    ez = (2.0 ** -13 + (K + 6) * U) * (np.abs(xf) @ np.abs(wf)) + 2 * U * np.abs(f64(b))
    near(Z, ref["Z"], ez, B, "Z")
    near(Y, ref["Y"], SLOPE * ez + 1e-5 * np.abs(ref["Y"]) + 3e-7 + 2 * U * np.abs(ref["Y"]), B, "Y")
    assert y_ok() and z_ok()


@pytest.mark.parametrize("M,N,K", [(2, 70, 250), (130, 131, 300), (2056, 1288, 2064)])
def test_fp8_integers_are_exact(M, N, K):
    x, w, b, r = (si.small_ints(s, 85 + k) for k, s in enumerate([(M, K), (N, K), (N,), (M, N)]))
    Y = torch.empty(M, N, dtype=F, device="cuda")
    one = torch.ones(1, device="cuda")
    tpm.tp_linear_fwd(si.to_e4m3_exact(x).cuda(), si.to_e4m3_exact(w).cuda(), Y, bias=dev(b, B), residual=dev(r, F), trans_w=True,
                      x_scale=one, w_scale=one)
    torch.cuda.synchronize()
    assert np.array_equal(f64(Y), ops.linear_fwd(x, w.T, b, ops.ACT_NONE, r)["Y"])


def test_residual_in_place():
    for M, N, K in ((3, 264, 1000), (300, 264, 200), (2056, 1288, 1032), (129, 131, 67)):
        fwd_check(M, N, K, inplace=True, act=ops.ACT_RELU)


def test_chunks_in_any_order_and_gated():
    M, N, K, C = 512, 264, 256, 8
    x = dev(si.normal_f32((M, K), 90), B)
    w, b, r = dev(si.normal_f32((K, N), 91, 0.05), B), dev(si.normal_f32((N,), 92), B), dev(si.normal_f32((M, N), 93), B)
    ws = tpm.alloc_workspace(tpm.OP_LINEAR_FWD, M, N, K, 1, C)
    outs = []
    for order in (None, [7, 6, 5, 4, 3, 2, 1, 0], [3, 1, 4, 0, 5, 7, 2, 6]):
        for gated in (False, True):
            ready = torch.full((C,), 5, dtype=torch.int32, device="cuda") if gated else None
            Y = torch.empty(M, N, dtype=B, device="cuda")
            tpm.tp_linear_fwd(x, w, Y, bias=b, residual=r, act=ops.ACT_SILU, num_chunks=C, chunk_order=order, chunk_ready=ready,
                              epoch=5, workspace=ws)
            torch.cuda.synchronize()
            assert tpm.poll_device_error(ws) == 0
            outs.append(Y)
    assert all(torch.equal(outs[0], y) for y in outs[1:])


@pytest.mark.parametrize("M,N,K", [(4, 264, 1000), (300, 264, 200), (129, 131, 67), (2056, 1288, 1032)])
@pytest.mark.parametrize("trans_w", [False, True])
def test_infinities_and_nans_stay_in_their_row_and_column(M, N, K, trans_w):
    x, w = si.normal_f32((M, K), 95), si.normal_f32((K, N), 96, 0.05)
    x[1, K - 1] = np.nan
    x[2, 0] = np.inf
    w[K - 1, 5] = np.nan
    w[K // 2, N - 1] = np.inf
    X, W = dev(x, B), dev(np.ascontiguousarray(w.T) if trans_w else w, B)
    Y = torch.empty(M, N, dtype=F, device="cuda")
    tpm.tp_linear_fwd(X, W, Y, trans_w=trans_w)
    torch.cuda.synchronize()
    got = f64(Y)
    with np.errstate(invalid="ignore"):
        ref = f64(X) @ (f64(W).T if trans_w else f64(W))
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)) and np.array_equal(np.isnan(got), np.isnan(ref))


# ----------------------------------------------------------------- backward
def bwd_check(M, N, K, dt=B, act=ops.ACT_GELU_ERF, dwdt=None, dbias=True, seed=200, ld=0, off=0):
    dwdt = dwdt or dt
    some = bool(ld or off)
    X = dev(si.normal_f32((M, K), seed), dt, K + ld if some else None, off)
    W = dev(si.normal_f32((K, N), seed + 1, 0.1), dt, N + ld if some else None, off)
    Z = dev(si.normal_f32((M, N), seed + 2), dt, N + ld if some else None, off) if act != ops.ACT_NONE else None
    dY = dev(si.normal_f32((M, N), seed + 3), dt, N + ld if some else None, off)
    dW, w_ok = empty(K, N, dwdt, N + ld, off)
    dX, x_ok = empty(M, K, dt, K + ld, off)
    db = torch.full((N,), 7.0, device="cuda") if dbias else None
    work = tpm.alloc_workspace(tpm.OP_LINEAR_ACT_BWD, M, N, K, 1, 1, tpm.dtype_code(dt))
    work.fill_(0xFF)
    tpm.tp_linear_act_bwd(X, W, dY, dW, dX, Z=Z, act=act, dbias=db, workspace=work)
    torch.cuda.synchronize()
    x, w, dy = f64(X), f64(W), f64(dY)
    ref = ops.linear_act_bwd(x, w, dy, None if Z is None else f64(Z), act)
    smooth = act not in (ops.ACT_NONE, ops.ACT_RELU)
    edz = (1e-5 * np.abs(ref["dZ"]) + 3e-7 * np.abs(dy) if smooth else 0) + 2 * U * np.abs(ref["dZ"])
    stored = edz + (HALF[dt] * (np.abs(ref["dZ"]) + edz) + TINY if act != ops.ACT_NONE else 0)
    adz = np.abs(ref["dZ"]) + stored
    near(dW, ref["dW"], np.abs(x).T @ stored + (M + 4) * U * (np.abs(x).T @ adz), dwdt, "dW")
    near(dX, ref["dX"], stored @ np.abs(w).T + (N + 4) * U * (adz @ np.abs(w).T), dt, "dX")
    if dbias:
        near(db, ref["dbias"], np.asarray(edz).sum(0) + (M + 4) * U * np.abs(ref["dZ"]).sum(0), F, "dbias")
    assert w_ok() and x_ok()
    return dW, dX, db


BWD = [(1, 8, 8), (1, 1, 1), (5, 24, 16), (300, 264, 200), (301, 264, 200), (515, 771, 259), (17, 33, 129), (1000, 512, 264), (64, 1280, 1024),
       (1021, 520, 1032), (3, 600, 7), (2000, 9, 65)]
LARGE = [(2048, 1032, 1096), (2051, 1288, 1024), (4100, 520, 1040)]     # the paired 256 x 256 tiles, whole and ragged rows


@pytest.mark.parametrize("M,N,K", BWD)
@pytest.mark.parametrize("dt", [B, F])
def test_backward(M, N, K, dt):
    bwd_check(M, N, K, dt, ACTS[(M + N) % 5])
    bwd_check(M, N, K, dt, ACTS[(M + N + 2) % 5], dwdt=F, dbias=False)


@pytest.mark.parametrize("M,N,K", LARGE)
def test_backward_large(M, N, K):
    bwd_check(M, N, K, B, ACTS[M % 5])
    bwd_check(M, N, K, B, ops.ACT_GELU_ERF, dwdt=F, ld=8, off=8)


@pytest.mark.parametrize("act", ACTS)
def test_backward_every_activation(act):
    for dt in (B, F):
        bwd_check(200, 136, 72, dt, act)


def test_backward_strides_and_offsets():
    for ld, off in ((8, 0), (8, 8), (3, 0), (4, 4), (0, 1)):
        bwd_check(300, 264, 200, B, ops.ACT_SILU, ld=ld, off=off)
        bwd_check(70, 65, 33, F, ops.ACT_SILU, ld=ld, off=off)


def test_backward_of_empty_sizes():
    z = lambda *s: torch.empty(*s, dtype=B, device="cuda")  # noqa: E731
    dW, dX, db = z(16, 24) + 1, z(0, 16), torch.ones(24, device="cuda")
    tpm.tp_linear_act_bwd(z(0, 16), z(16, 24), z(0, 24), dW, dX, Z=z(0, 24), act=ops.ACT_SILU, dbias=db)
    torch.cuda.synchronize()
    assert not dW.any() and not db.any()
    dX = z(4, 16).fill_(1)
    tpm.tp_linear_act_bwd(z(4, 16), z(16, 0), z(4, 0), z(16, 0), dX)
    torch.cuda.synchronize()
    assert not dX.any()


def test_backward_repeats_bit_for_bit():
    for M, N, K in ((1000, 512, 264), (517, 777, 1003)):
        a, b = bwd_check(M, N, K), bwd_check(M, N, K)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_gradients_against_differences():
    # fp32 throughout: the loss sum(Y * w) along random unit directions of X,
    # W and bias.  Step 2^-6: rounding errors of the loss, about sqrt(M N) u
    # |w| = 2^-24 * 130 * a few, over 2^-5 are below 2e-4; the truncation is
    # step^2 / 6 = 4e-5 times a third derivative of order one
    M, N, K, act = 96, 136, 72, ops.ACT_GELU_ERF
    x, w, b, g = (dev(si.normal_f32(s, 300 + k, v), F) for k, (s, v) in enumerate([((M, K), 1), ((K, N), 0.1), ((N,), 1), ((M, N), 1)]))

    def fwd(x, w, b):
        Y, Z = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
        tpm.tp_linear_fwd(x, w, Y, bias=b, act=act, Z=Z)
        return Y, Z
    Z = fwd(x, w, b)[1]
    dW, dX, db = torch.empty_like(w), torch.empty_like(x), torch.empty_like(b)
    tpm.tp_linear_act_bwd(x, w, g, dW, dX, Z=Z, act=act, dbias=db)
    for k, grad in enumerate((dX, dW, db)):
        d = torch.randn(grad.shape, generator=torch.Generator("cuda").manual_seed(7 + k), device="cuda")
        d /= d.norm()
        hi, lo = [x, w, b], [x, w, b]
        hi[k], lo[k] = hi[k] + 2.0 ** -6 * d, lo[k] - 2.0 ** -6 * d
        numeric = float(((fwd(*hi)[0].double() - fwd(*lo)[0].double()) * g.double()).sum()) * 2.0 ** 5
        assert abs(numeric - float((grad.double() * d.double()).sum())) < 2e-3


def test_other_streams_and_graph_replays():
    M, N, K = 96, 264, 520
    x, w, b, r = (dev(si.normal_f32(s, 400 + k, v), B) for k, (s, v) in enumerate([((M, K), 1), ((K, N), 0.05), ((N,), 1), ((M, N), 1)]))
    Y, Z, y1 = (torch.empty(M, N, dtype=B, device="cuda") for _ in range(3))
    dW, dX, db = torch.empty(K, N, dtype=B, device="cuda"), torch.empty(M, K, dtype=B, device="cuda"), torch.empty(N, device="cuda")
    wf, wb = tpm.alloc_workspace(tpm.OP_LINEAR_FWD, M, N, K), tpm.alloc_workspace(tpm.OP_LINEAR_ACT_BWD, M, N, K)
    w1 = tpm.alloc_workspace(tpm.OP_LINEAR_FWD, 2, N, K)

    def step(stream=None, fresh=False):
        kw = (lambda ws: {}) if fresh else (lambda ws: dict(workspace=ws))
        tpm.tp_linear_fwd(x, w, Y, bias=b, residual=r, act=ops.ACT_SILU, Z=Z, stream=stream, **kw(wf))
        tpm.tp_linear_act_bwd(x, w, Y, dW, dX, Z=Z, act=ops.ACT_SILU, dbias=db, stream=stream, **kw(wb))
        tpm.tp_linear_fwd(x[:2], w, y1[:2], bias=b, stream=stream, **kw(w1))

    outs = (Y, Z, dW, dX, db, y1[:2])

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in outs]
    step()
    want = results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side, fresh=True)
    assert all(torch.equal(p, q) for p, q in zip(results(), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(4):
        x.copy_(dev(si.normal_f32((M, K), 500 + k), B))
        step()
        eager = results()
        for t in outs:
            t.zero_()
        g.replay()
        assert all(torch.equal(p, q) for p, q in zip(results(), eager))
