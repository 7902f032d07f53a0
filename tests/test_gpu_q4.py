"""GPU parity of linears in 4 bits (encode_q4, gemm_q4, gemv_q4) against
oracle/q4.py.

Codes, scales, zero points: equal.  Products: with S the sum of the magnitudes of
an output's terms and n = in + 3 T + 24 the roundings a term can meet (the sums of
a group, its scaling, the sum over groups, the joining of waves and slices), each
at most 2^-23 (a matrix instruction may cut instead of round):
  fp32:  |err| <= n 2^-23 S'      fp16:  the same and one rounding
S' counts a term as |c - z| s |x|: the products are exact.
"""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
import workloads
from oracle import q4

pytestmark = pytest.mark.gpu


def dev():
    return torch.device("cuda:0")


def t_of(a, kind):
    return torch.from_numpy(np.ascontiguousarray(a).view(kind)).to(dev())


def layer(out, inf, seed, zeros):
    """Random codes, scales and (or none) zero points, the ends of their ranges among them."""
    rng = np.random.default_rng(seed)
    T = -(-inf // 128)
    codes = rng.integers(0, 16, (out, inf)).astype(np.uint8)
    scales = (rng.random((out, T)) * 0.02 + 0.001).astype(np.float16)
    scales[0, 0] = 2.0 ** -24
    scales[-1, -1] = -0.5
    points = rng.integers(0, 16, (out, T)).astype(np.uint8) if zeros else np.full((out, T), 8, np.uint8)
    return codes, scales.view(np.uint16), points


def to_gpu(codes, scales, points, zeros):
    return t_of(q4.pack(codes), np.uint8), t_of(scales, np.float16), t_of(points, np.uint8) if zeros else None


def check(Y, codes, scales, points, X, what=""):
    y, S = q4.gemm(codes, scales, points, X)
    inf = codes.shape[1]
    tol = (inf + 3 * -(-inf // 128) + 24) * 2.0 ** -23 * S
    if Y.dtype == torch.float16:
        tol = tol + 2.0 ** -11 * (np.abs(y) + tol) + 2.0 ** -25
    err = np.abs(Y.cpu().double().numpy() - y)
    assert (err <= tol).all(), f"{what}: {np.argwhere(~(err <= tol))[:3]}, worst {np.nanmax(err / np.maximum(tol, 1e-300))}"


ENCODE = [(1, 32), (3, 96), (16, 128), (129, 160), (300, 4128), (17, 1056)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("out,inf", ENCODE)
def test_encode_equals_the_oracle(out, inf, zeros):
    W = workloads.gaussian_weight(out, inf, out + inf, outliers=True)
    W[0, :4] = [0.0, -0.0, 1e-42, 0.5]
    W[-1] = 0.0
    if out > 2:
        W[1] = np.abs(W[1]) + 1                 # one sign
        W[2] = np.float32(3e38) * np.sign(W[2]) if out > 20 else W[2]
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    codes, scales, points = rbq.encode_q4(t_of(W, np.float32), zeros=zeros, status=st)
    torch.cuda.synchronize()
    c, s, z = q4.encode(W, zeros)
    assert np.array_equal(scales.cpu().numpy().view(np.uint16), s)
    assert np.array_equal(codes.cpu().numpy(), q4.pack(c))
    assert (points is None) == (not zeros) and (points is None or np.array_equal(points.cpu().numpy(), z))
    assert int(st.item()) == 0


def test_encode_of_non_finite_groups():
    W = workloads.gaussian_weight(5, 288, 2)
    W[1, 130], W[3, 287], W[4, 0] = np.inf, np.nan, -np.inf
    for zeros in (False, True):
        st = torch.zeros(1, dtype=torch.int32, device=dev())
        codes, scales, points = rbq.encode_q4(t_of(W, np.float32), zeros=zeros, status=st)
        c, s, z = q4.encode(W, zeros)
        assert int(st.item()) == rbq.RBQ_STATUS_NONFINITE_W
        s2 = scales.cpu().numpy()
        assert np.array_equal(np.isnan(s2), np.isnan(s.view(np.float16))) and np.isnan(s2).sum() == 3
        assert np.array_equal(codes.cpu().numpy(), q4.pack(c))
        y = rbq.gemv_q4(codes, scales, torch.ones(288, dtype=torch.float16, device=dev()), points)
        assert torch.equal(torch.isnan(y).cpu(), torch.tensor([False, True, False, True, True]))


def test_encode_many_turns():
    """More groups than one turn of the bounded grid takes, sampled."""
    out, inf = 300_000, 544
    W = torch.randn(out, inf, device=dev())
    codes, scales, points = rbq.encode_q4(W, zeros=True)
    rows = [0, 1, 99_999, 299_998, 299_999]
    c, s, z = q4.encode(W[rows].cpu().numpy(), True)
    assert np.array_equal(codes[rows].cpu().numpy(), q4.pack(c))
    assert np.array_equal(scales[rows].cpu().numpy().view(np.uint16), s)
    assert np.array_equal(points[rows].cpu().numpy(), z)


SHAPES = [(1, 32), (5, 64), (16, 128), (17, 160), (40, 288), (130, 1056), (300, 4128), (257, 2080)]
TOKENS = [1, 2, 15, 16, 17, 33, 64, 65, 100, 129, 200, 300]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("out,inf", SHAPES)
def test_products(out, inf, zeros):
    codes, scales, points = layer(out, inf, out + inf, zeros)
    g = to_gpu(codes, scales, points, zeros)
    for M in TOKENS:
        X = workloads.gaussian_activations(M, inf, seed=M + inf)
        x = t_of(X, np.float16)
        for dtype in (torch.float16, torch.float32):
            # (memory behind the output stays as it was)
            buf = torch.full((M * out + 64,), 7.0, dtype=dtype, device=dev())
            Y = rbq.gemm_q4(g[0], g[1], x, g[2], dtype=dtype, Y=buf[:M * out].view(M, out))
            check(Y, codes, scales, points, X, f"{M} tokens {dtype}")
            assert bool((buf[M * out:] == 7).all())
        if M == 1:
            y = rbq.gemv_q4(g[0], g[1], x[0], g[2])
            assert torch.equal(y, rbq.gemm_q4(g[0], g[1], x, g[2])[0])


LARGER = [(1, 4096, 4096), (1, 1000, 11008), (3, 2000, 8192), (16, 512, 11008), (24, 1008, 4096), (48, 1504, 2048),
          (96, 1504, 2048), (150, 700, 4128), (257, 520, 1056), (600, 1030, 512)]


@pytest.mark.parametrize("M,out,inf", LARGER)
def test_larger_products(M, out, inf):
    for zeros in (False, True):
        codes, scales, points = layer(out, inf, M + out, zeros)
        X = workloads.gaussian_activations(M, inf, seed=M)
        g = to_gpu(codes, scales, points, zeros)
        for dtype in (torch.float16, torch.float32):
            Y = rbq.gemm_q4(g[0], g[1], t_of(X, np.float16), g[2], dtype=dtype)
            check(Y, codes, scales, points, X, str(dtype))
            none = torch.empty(0, dtype=torch.uint8, device=dev())
            check(rbq.gemm_q4(g[0], g[1], t_of(X, np.float16), g[2], dtype=dtype, workspace=none), codes, scales,
                  points, X, f"{dtype} without workspace")


@pytest.mark.parametrize("M", [1, 8, 40, 130])
def test_every_column_and_code_has_its_place(M):
    """Unit tokens pick single columns: exact values."""
    out, inf = 19, 416
    codes, scales, points = layer(out, inf, 3, True)
    scales[:] = np.float16(0.25).view(np.uint16)
    g = to_gpu(codes, scales, points, True)
    want = q4.values(codes, scales, points)
    for j0 in range(0, inf, M):
        X = np.zeros((M, inf), np.float16)
        cols = [(j0 + i) % inf for i in range(M)]
        X[np.arange(M), cols] = 1.0
        Y = rbq.gemm_q4(g[0], g[1], t_of(X, np.float16), g[2])
        assert np.array_equal(Y.cpu().double().numpy(), want[:, cols].T)


@pytest.mark.parametrize("M", [1, 5, 20, 70, 140])
def test_non_finite_tokens_stay_in_their_rows(M):
    out, inf = 50, 544
    codes, scales, points = layer(out, inf, 4, False)
    X = workloads.gaussian_activations(M, inf, seed=1).copy()
    clean = X.copy()
    bad = M // 2
    X[bad, 537] = 0x7E00
    clean[bad] = 0
    g = to_gpu(codes, scales, points, False)
    Y = rbq.gemm_q4(g[0], g[1], t_of(X, np.float16), None)
    ref = rbq.gemm_q4(g[0], g[1], t_of(clean, np.float16), None)
    assert torch.isnan(Y[bad]).all()
    keep = [m for m in range(M) if m != bad]
    assert torch.equal(Y[keep], ref[keep])


def test_streams_graphs_and_a_shared_workspace():
    out, inf = 700, 4128
    cases = []
    for M in (1, 16, 70, 200):
        codes, scales, points = layer(out, inf, M, True)
        g = to_gpu(codes, scales, points, True)
        x = t_of(workloads.gaussian_activations(M, inf, seed=M), np.float16)
        cases.append((g, x, rbq.gemm_q4(g[0], g[1], x, g[2], dtype=torch.float32)))
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=dev())
    graphs = []
    torch.cuda.synchronize()
    for g, x, _ in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = rbq.gemm_q4(g[0], g[1], x, g[2], dtype=torch.float32, workspace=ws)
        graphs.append((graph, y))
    for _ in range(3):
        for (graph, y), (_, _, want) in zip(graphs, cases):
            y.zero_()
            graph.replay()
            torch.randn(64, 64, device=dev()).sum()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g, x, want = cases[2]
    got = rbq.gemm_q4(g[0], g[1], x, g[2], dtype=torch.float32, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_empty_products():
    z = (lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device=dev()))
    h = torch.float16
    assert rbq.gemm_q4(z(3, 32), z(3, 1, dtype=h), z(0, 64, dtype=h)).shape == (0, 3)
    assert rbq.gemm_q4(z(0, 32), z(0, 1, dtype=h), z(2, 64, dtype=h)).shape == (2, 0)
    Y = rbq.gemm_q4(z(3, 0), z(3, 0, dtype=h), z(2, 0, dtype=h), Y=torch.ones(2, 3, dtype=h, device=dev()))
    assert not Y.any()
    codes, scales, points = rbq.encode_q4(torch.zeros(0, 64, device=dev()), zeros=True)
    assert codes.shape == (0, 32) and scales.shape == (0, 1) and points.shape == (0, 1)
