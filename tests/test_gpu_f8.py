"""GPU parity of linears in 8-bit floating point blocks of 128 (rbq_encode_f8,
rbq_quantize_f8, rbq_gemm_f8, rbq_gemv_f8) against oracle/f8.py.

Codes and scales: equal bits.  Products, per element, with S the sum of the
magnitudes of an output's terms and n = in + 3 T + 16 the roundings a term
can meet (the sums inside a block, the product of the two scales, the fma of
each block, the joining of partial sums), each at most 2^-23 (a matrix
instruction may cut instead of round):
  fp32:  |err| <= n 2^-23 S
  fp16:  the same, and one rounding: 2^-11 (|y| + n 2^-23 S) + 2^-25
More than 32 tokens with fp16 outputs take the 8-bit matrix instruction, which
cuts the products of 8 columns at 2^-13 of the power of two below the largest:
the other 7 lose less than that each, so an output is off by up to 7 2^-13 of
the sum of the groups' largest products more.
"""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
import workloads
from oracle import f8

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def dev():
    return torch.device("cuda:0")


def t_f16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.float16)).to(dev())


def t_f8(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).to(dev()).view(F8)


def t_f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dev())


def np_codes(t):
    return t.view(torch.uint8).cpu().numpy()


def bits32(a):
    return np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)


def same_scales(got, want):
    """Equal bits, any NaN equal to any other."""
    got, want = got.cpu().numpy(), np.asarray(want)
    return np.array_equal(np.isnan(got), np.isnan(want)) and \
        np.array_equal(bits32(np.nan_to_num(got, nan=1.0)), bits32(np.nan_to_num(want, nan=1.0)))


def tolerance(S, y, inf, half, cut=0.0):
    n = inf + 3 * (-(-inf // 128)) + 16
    t = n * 2.0 ** -23 * S + 7 * 2.0 ** -13 * cut
    return 2.0 ** -11 * (np.abs(y) + t) + 2.0 ** -25 + t if half else t


SHAPES = [(1, 32), (128, 128), (129, 160), (300, 96), (17, 4128), (257, 1056)]


@pytest.mark.parametrize("out,inf", SHAPES)
def test_encode_equals_the_oracle(out, inf):
    W = workloads.gaussian_weight(out, inf, out + inf, outliers=True)
    W[0, :3] = [0.0, -0.0, 1e-42]
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    codes, scales = rbq.encode_f8(t_f32(W), status=st)
    torch.cuda.synchronize()
    c, s = f8.encode(W)
    assert np.array_equal(np_codes(codes), c) and same_scales(scales, s)
    assert int(st.item()) == 0


def test_encode_special_blocks():
    W = workloads.gaussian_weight(300, 416, 5)
    W[:128, :128] = 0.0
    W[:128, 128:256] *= np.float32(1e-38)                  # subnormal weights: the floor of the maximum
    W[128:256, :128] *= np.float32(1e36)
    W[130, 140] = np.inf
    W[290, 3] = np.nan
    W[299, 415] = -np.inf                                  # in the smallest corner block
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    codes, scales = rbq.encode_f8(t_f32(W), status=st)
    torch.cuda.synchronize()
    c, s = f8.encode(W)
    assert np.array_equal(np_codes(codes), c) and same_scales(scales, s)
    assert np.isnan(s).sum() == 3 and int(st.item()) == rbq.RBQ_STATUS_NONFINITE_W


@pytest.mark.parametrize("M,inf", [(1, 32), (1, 4096), (16, 128), (17, 160), (33, 4128), (5, 544)])
def test_quantize_equals_the_oracle(M, inf):
    X = workloads.gaussian_activations(M, inf, M + inf).copy()
    X[0, :4] = [0x0000, 0x8000, 0x0001, 0x8001]
    if M > 4:
        X[2] = 0                                           # a padded token
        X[3] &= 0x83FF                                     # a token of subnormals
        X[4, 7] = 0x7BFF
        X[M - 1, inf - 1] = 0xFC00
    codes, scales = rbq.quantize_f8(t_f16(X))
    torch.cuda.synchronize()
    c, s = f8.quantize(X)
    assert np.array_equal(np_codes(codes), c) and same_scales(scales, s)


def test_quantize_every_fp16_value():
    """Every finite fp16 value against maxima that put it next to borders."""
    v = np.concatenate([np.arange(0x7C00), np.arange(0x8000, 0xFC00)]).astype(np.uint16)
    rows = v[np.argsort(v & 0x7FFF, kind="stable")].reshape(-1, 512)   # 124 rows of neighbours
    codes, scales = rbq.quantize_f8(t_f16(rows))
    torch.cuda.synchronize()
    c, s = f8.quantize(rows)
    assert np.array_equal(np_codes(codes), c) and same_scales(scales, s)


def layer(out, inf, M, seed):
    """Random codes of every finite value and scales over several powers of two."""
    rng = np.random.default_rng(seed)
    fin = np.concatenate([np.arange(0x7F), np.arange(0x80, 0xFF)]).astype(np.uint8)
    T = -(-inf // 128)
    w8 = rng.choice(fin, size=(out, inf))
    x8 = rng.choice(fin, size=(M, inf))
    ws = (2.0 ** rng.uniform(-16, -8, (-(-out // 128), T))).astype(np.float32)
    xs = (2.0 ** rng.uniform(-12, -6, (T, M))).astype(np.float32)
    return w8, ws, x8, xs


GEMM = [(1, 1, 32), (16, 16, 128), (130, 3, 160), (33, 17, 416), (300, 64, 1056), (257, 65, 4128), (128, 200, 512),
        (513, 300, 640), (1000, 129, 96), (40, 1000, 288), (272, 530, 1184)]


@pytest.mark.parametrize("half", [True, False], ids=["fp16", "fp32"])
@pytest.mark.parametrize("out,M,inf", GEMM)
def test_gemm_matches_the_oracle(out, M, inf, half):
    w8, ws, x8, xs = layer(out, inf, M, out + M + inf)
    y_ref, S = f8.gemm(w8, ws, x8, xs)
    Y = torch.full((M, out), float("nan"), dtype=torch.float16 if half else torch.float32, device=dev())
    got = rbq.gemm_f8(t_f8(w8), t_f32(ws), t_f8(x8), t_f32(xs), dtype=Y.dtype, Y=Y)
    again = rbq.gemm_f8(t_f8(w8), t_f32(ws), t_f8(x8), t_f32(xs), dtype=Y.dtype)
    torch.cuda.synchronize()
    assert got is Y
    err = np.abs(Y.cpu().numpy().astype(np.float64) - y_ref)
    tol = tolerance(S, y_ref, inf, half, f8.largest_products(w8, ws, x8, xs) if half and M > 32 else 0.0)
    assert (err <= tol).all(), f"{(err / tol).max():.3f} of the tolerance at {np.unravel_index((err / tol).argmax(), err.shape)}"
    assert torch.equal(Y, again)                           # the same bits in every run


# every tile kind, with and without slices: tall and wide, columns of one to
# many blocks, with and without a short last one
TILES = [(5003, 2500, 96), (5003, 2500, 128), (5003, 2500, 288), (5003, 2500, 384), (4999, 2561, 416),
         (5000, 2500, 1184), (4099, 2100, 640), (4099, 2100, 4128), (2050, 1500, 800), (130, 2000, 4128),
         (4096, 100, 4096), (4100, 129, 2080), (1003, 65, 11008), (8200, 300, 544)]


@pytest.mark.parametrize("half", [True, False], ids=["fp16", "fp32"])
@pytest.mark.parametrize("out,M,inf", TILES)
def test_gemm_tiles_match_the_definition_in_64_bits(out, M, inf, half):
    """The same bounds as above, with the sums in 64 bits on the device and
    the cut of the 8-bit instruction bounded by the sum of all products."""
    w8, ws, x8, xs = layer(out, inf, M, out + M + inf)
    dt = torch.float16 if half else torch.float32
    buf = torch.full((M * out + 4096,), float("nan"), dtype=dt, device=dev())
    Y = buf[:M * out].view(M, out)
    args = (t_f8(w8), t_f32(ws), t_f8(x8), t_f32(xs))
    rbq.gemm_f8(*args, dtype=dt, Y=Y)
    again = rbq.gemm_f8(*args, dtype=dt)
    none = rbq.gemm_f8(*args, dtype=dt, workspace=torch.empty(0, dtype=torch.uint8, device=dev()))
    torch.cuda.synchronize()
    assert torch.equal(Y, again) and bool(torch.isnan(buf[M * out:]).all())
    T = -(-inf // 128)
    cols = torch.arange(inf, device=dev()) // 128
    w = args[0].double() * args[1].double()[torch.arange(out, device=dev()) // 128][:, cols]
    x = args[2].double() * args[3].double().t()[:, cols]
    y_ref = x @ w.t().contiguous()
    S = x.abs() @ w.abs().t().contiguous()
    # of 8 products of one group the largest is at least an eighth of their sum and at most all of it
    t = (inf + 3 * T + 16) * 2.0 ** -23 * S + (7 * 2.0 ** -13 * S if half else 0.0)
    if half:
        t = 2.0 ** -11 * (y_ref.abs() + t) + 2.0 ** -25 + t
    for got in (Y, none):
        assert bool(((got.double() - y_ref).abs() <= t).all()), f"{((got.double() - y_ref).abs() / t).max():.3f}"


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_leaves_what_is_behind_its_output(M):
    out, inf = 259, 416
    w8, ws, x8, xs = layer(out, inf, M, 9)
    buf = torch.full((M * out + 4096,), 7.0, dtype=torch.float16, device=dev())
    Y = buf[:M * out].view(M, out)
    rbq.gemm_f8(t_f8(w8), t_f32(ws), t_f8(x8), t_f32(xs), Y=Y)
    torch.cuda.synchronize()
    assert bool((buf[M * out:] == 7.0).all()) and not bool((Y == 7.0).all())


@pytest.mark.parametrize("M", [2, 70, 300])
def test_gemm_non_finite_scales_and_codes_stay_in_their_rows(M):
    out, inf = 300, 544
    w8, ws, x8, xs = layer(out, inf, M, 21)
    x8[1, 5] = 0x7F                                        # a NaN code of token 1
    xs[2, M - 1] = np.nan                                  # a block that held a NaN
    w8[7, 543] = 0xFF
    ws[2, 0] = np.inf                                      # rows 256 .. 299
    Y = rbq.gemm_f8(t_f8(w8), t_f32(ws), t_f8(x8), t_f32(xs), dtype=torch.float32)
    torch.cuda.synchronize()
    bad = ~np.isfinite(Y.cpu().numpy())
    want = np.zeros((M, out), bool)
    want[[1, M - 1], :] = True
    want[:, 7] = True
    want[:, 256:] = True
    assert np.array_equal(bad, want)
    clean, S = f8.gemm(w8[:7], ws[:1], x8, xs)
    err = np.abs(Y.cpu().numpy()[:, :7].astype(np.float64) - clean)
    rows = ~want[:, 0]
    assert (err[rows] <= tolerance(S, clean, inf, False)[rows]).all()


@pytest.mark.parametrize("out,inf", [(1, 32), (16, 128), (130, 160), (1000, 4128), (259, 96), (4096, 4096), (50, 11008)])
def test_gemv_matches_the_oracle_and_the_two_calls(out, inf):
    w8, ws, _, _ = layer(out, inf, 1, out + inf)
    X = workloads.gaussian_activations(1, inf, 3)
    c, s = f8.quantize(X)
    y_ref, S = f8.gemm(w8, ws, c, s)
    y = torch.full((out,), float("nan"), dtype=torch.float16, device=dev())
    assert rbq.gemv_f8(t_f8(w8), t_f32(ws), t_f16(X[0]), y=y) is y
    two = rbq.gemm_f8(t_f8(w8), t_f32(ws), *rbq.quantize_f8(t_f16(X)))
    torch.cuda.synchronize()
    tol = tolerance(S, y_ref, inf, True)[0]
    assert (np.abs(y.cpu().numpy().astype(np.float64) - y_ref[0]) <= tol).all()
    assert (np.abs(two.cpu().numpy()[0].astype(np.float64) - y_ref[0]) <= tol).all()


def test_gemv_special_tokens():
    out, inf = 48, 416
    w8, ws, _, _ = layer(out, inf, 1, 11)
    for place, value, bad in ((0, 0x7E00, True), (415, 0xFC00, True), (200, 0x7BFF, False)):
        X = workloads.gaussian_activations(1, inf, 5).copy()
        X[0, place] = value
        y = rbq.gemv_f8(t_f8(w8), t_f32(ws), t_f16(X[0])).cpu().numpy()
        assert np.isnan(y).all() == bad and (bad or np.isfinite(y).all())
    zero = rbq.gemv_f8(t_f8(w8), t_f32(ws), torch.zeros(inf, dtype=torch.float16, device=dev()))
    assert not zero.cpu().numpy().any()


def test_empty_calls():
    z = torch.zeros(0, 64, dtype=torch.float16, device=dev())
    codes, scales = rbq.quantize_f8(z)
    assert codes.shape == (0, 64) and scales.shape == (1, 0)
    w8, ws, x8, xs = layer(40, 64, 1, 1)
    assert rbq.gemm_f8(t_f8(w8), t_f32(ws), codes, scales).shape == (0, 40)
    e8 = torch.empty(40, 0, dtype=torch.uint8, device=dev()).view(F8)
    es = torch.empty(1, 0, dtype=torch.float32, device=dev())
    for dt in (torch.float16, torch.float32):
        Y = rbq.gemm_f8(e8, es, torch.empty(3, 0, dtype=torch.uint8, device=dev()).view(F8),
                        torch.empty(0, 3, dtype=torch.float32, device=dev()), dtype=dt)
        assert Y.shape == (3, 40) and not Y.any()
    assert not rbq.gemv_f8(e8, es, torch.empty(0, dtype=torch.float16, device=dev())).any()
    c, s = rbq.encode_f8(torch.empty(0, 64, device=dev()))
    assert c.shape == (0, 64) and s.shape == (0, 1)


def test_transposed_layer_is_the_input_gradient():
    """dX = dY W with the transposed codes and scales of the same layer: the
    gradient of the product with respect to its (quantised) input, against the
    formula and against differences of the product itself."""
    out, inf, M = 160, 288, 5
    W = workloads.gaussian_weight(out, inf, 31)
    w8, ws = rbq.encode_f8(t_f32(W))
    dY = workloads.gaussian_activations(M, out, 32)
    d8, dsc = rbq.quantize_f8(t_f16(dY))
    wt = w8.view(torch.uint8).t().contiguous().view(F8)
    dX = rbq.gemm_f8(wt, ws.t().contiguous(), d8, dsc, dtype=torch.float32)
    torch.cuda.synchronize()
    c, s = f8.encode(W)
    w = f8.values(c, s, 128)
    dc, dscale = f8.quantize(dY)
    d = f8.values(dc, np.ascontiguousarray(dscale.T), 1)
    want, S = d @ w, np.abs(d) @ np.abs(w)
    got = dX.cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= tolerance(S, want, out, False)).all()
    # differences: the product is linear in x, so moving code (m, j) from one
    # value to another moves L = sum dY y by dX[m][j] times the step
    rng = np.random.default_rng(33)
    X = workloads.gaussian_activations(M, inf, 34)
    x8, xs = f8.quantize(X)
    for _ in range(6):
        m, j = int(rng.integers(M)), int(rng.integers(inf))
        x8b = x8.copy()
        x8b[m, j] = 0x70                                    # 128 times the scale
        y0 = rbq.gemm_f8(w8, ws, t_f8(x8), t_f32(xs), dtype=torch.float32).cpu().numpy().astype(np.float64)
        y1 = rbq.gemm_f8(w8, ws, t_f8(x8b), t_f32(xs), dtype=torch.float32).cpu().numpy().astype(np.float64)
        step = (f8.e4m3_values(x8b[m, j]) - f8.e4m3_values(x8[m, j])) * float(xs[j // 128, m])
        xv = f8.values(x8b, np.ascontiguousarray(xs.T), 1)
        tol = 2 * (tolerance(np.abs(xv[m]) @ np.abs(w).T + np.abs(f8.values(x8, np.ascontiguousarray(xs.T), 1)[m])
                             @ np.abs(w).T, 0, inf, False) * np.abs(d[m])).sum() + abs(step) * \
            tolerance(S, want, out, False)[m, j]
        assert abs(((y1 - y0)[m] * d[m]).sum() - step * got[m, j]) <= tol


def test_other_stream_and_graph():
    """A run of the operators together: quantise, project, on a side stream,
    then captured and replayed on new inputs, with eager work between."""
    out, inf, M = 300, 416, 33
    W = workloads.gaussian_weight(out, inf, 41)
    w8, ws = rbq.encode_f8(t_f32(W))
    X = [workloads.gaussian_activations(M, inf, 42 + i) for i in range(3)]
    eager = [rbq.gemm_f8(w8, ws, *rbq.quantize_f8(t_f16(x))) for x in X]
    vec = [rbq.gemv_f8(w8, ws, t_f16(x[3])) for x in X]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = rbq.quantize_f8(t_f16(X[0]), stream=side)
    y = rbq.gemm_f8(w8, ws, *q, stream=side)
    y1 = rbq.gemm_f8(w8, ws, *q, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, eager[0]) and torch.equal(y1, eager[0])
    x_in = t_f16(X[0])
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        yg = rbq.gemm_f8(w8, ws, *rbq.quantize_f8(x_in))
        vg = rbq.gemv_f8(w8, ws, x_in[3])
    for rep in range(6):
        x_in.copy_(t_f16(X[rep % 3]))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, eager[rep % 3]) and torch.equal(vg, vec[rep % 3])
        assert torch.equal(rbq.gemm_f8(w8, ws, *rbq.quantize_f8(t_f16(X[1]))), eager[1])


def test_refusals_on_the_device():
    w8, ws, x8, xs = layer(40, 64, 3, 1)
    W8, WS, X8, XS = t_f8(w8), t_f32(ws), t_f8(x8), t_f32(xs)
    with pytest.raises(ValueError):
        rbq.gemm_f8(W8, WS, X8, XS.t().contiguous())
    with pytest.raises(ValueError):
        rbq.gemm_f8(W8, WS[:, :0], X8, XS)
    with pytest.raises(ValueError):
        rbq.gemm_f8(W8, WS, X8[:, :32].contiguous(), XS)
    with pytest.raises(TypeError):
        rbq.gemm_f8(W8, WS, X8, XS, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        rbq.gemm_f8(W8, WS, X8, XS, Y=torch.empty(3, 40, device=dev()))
    with pytest.raises(ValueError):
        rbq.gemm_f8(W8, WS, X8, XS, Y=torch.empty(2, 40, dtype=torch.float16, device=dev()))
    with pytest.raises(ValueError):
        rbq.quantize_f8(torch.empty(64, 64, dtype=torch.float16, device=dev()).t())
    with pytest.raises(rbq.RbqError):
        rbq.quantize_f8(torch.empty(3, 40, dtype=torch.float16, device=dev()))
    with pytest.raises(rbq.RbqError):                       # rows that start 2 bytes off
        rbq.quantize_f8(torch.empty(129, dtype=torch.float16, device=dev())[1:].view(2, 64))
    with pytest.raises(ValueError):                        # a workspace on the host
        rbq.gemm_f8(W8, WS, X8, XS, workspace=torch.empty(64, dtype=torch.uint8))
    with pytest.raises(ValueError):
        rbq.gemv_f8(W8, WS, torch.empty(65, dtype=torch.float16, device=dev()))
