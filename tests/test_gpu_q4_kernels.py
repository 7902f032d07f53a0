"""Sizes that reach every kernel behind gemm_q4: one to four tokens, more of them on
one to three row tiles, rows whose scales do not fit LDS, and the tiled kernel with
the columns in one slice and in several.  Bounds as in tests/test_gpu_q4.py; the
oracle's products in float64 on the GPU.  test_q4_plans_cpu.py checks that the sizes
here reach them all."""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
import workloads
from test_gpu_q4 import dev, layer, t_of, to_gpu

pytestmark = pytest.mark.gpu

FEW = [(1, 70, 30016), (4, 40, 28704), (9, 40, 30016), (20, 33, 28736), (16, 4999, 416), (5, 12401, 160), (20, 4111, 1056),
       (13, 9001, 288), (16, 12288, 96), (3, 9001, 288)]
TILED = [(300, 2080, 4128), (17, 30011, 4128), (101, 5003, 4128), (2001, 2001, 544), (5003, 4301, 96), (8200, 8001, 32),
         (1030, 2049, 1056), (70, 1100, 28704)]
KERNELS = FEW + TILED                    # (tokens, out, in)


def weights(codes, scales, points):
    """float64 values on the GPU."""
    c = t_of(codes, np.uint8).double()
    over = (lambda v: v.double().repeat_interleave(128, 1)[:, :codes.shape[1]])
    return (c - over(t_of(points, np.uint8))) * over(t_of(scales, np.float16))


def near(Y, w, x, what=""):
    """tests/test_gpu_q4.py's bound."""
    inf = w.shape[1]
    x = x.double()
    y, S = torch.mm(x, w.t().contiguous()), torch.mm(x.abs(), w.abs().t().contiguous())
    tol = (inf + 3 * -(-inf // 128) + 24) * 2.0 ** -23 * S
    if Y.dtype == torch.float16:
        tol = tol + 2.0 ** -11 * (y.abs() + tol) + 2.0 ** -25
    wrong = ~((Y.double() - y).abs() <= tol)
    assert not bool(wrong.any()), f"{what}: {wrong.nonzero()[:3].tolist()} of {tuple(Y.shape)}"


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,out,inf", KERNELS)
def test_every_kernel(M, out, inf, zeros):
    codes, scales, points = layer(out, inf, M + out, zeros)
    g = to_gpu(codes, scales, points, zeros)
    w = weights(codes, scales, points)
    x = t_of(workloads.gaussian_activations(M, inf, seed=M), np.float16)
    none = torch.empty(0, dtype=torch.uint8, device=dev())
    for dtype in (torch.float16, torch.float32):
        buf = torch.full((M * out + 64,), 7.0, dtype=dtype, device=dev())
        near(rbq.gemm_q4(g[0], g[1], x, g[2], dtype=dtype, Y=buf[:M * out].view(M, out)), w, x, str(dtype))
        assert bool((buf[M * out:] == 7).all())
        near(rbq.gemm_q4(g[0], g[1], x, g[2], dtype=dtype, workspace=none), w, x, f"{dtype} without workspace")


@pytest.mark.parametrize("M,out,inf", [(3, 50, 416), (16, 4200, 416), (1500, 3301, 416), (500, 3301, 1312)])
def test_units_are_exact(M, out, inf):
    """Unit tokens pick single columns: exact values, from the tiled kernel too."""
    codes, scales, points = layer(out, inf, 3, True)
    scales[:] = np.float16(0.25).view(np.uint16)
    scales[:, ::2] = np.float16(2.0).view(np.uint16)
    g = to_gpu(codes, scales, points, True)
    w = weights(codes, scales, points)
    for j0 in range(0, inf, M):
        cols = (torch.arange(M, device=dev()) + j0) % inf
        x = torch.zeros((M, inf), dtype=torch.float16, device=dev())
        x[torch.arange(M, device=dev()), cols] = 1.0
        assert torch.equal(rbq.gemm_q4(g[0], g[1], x, g[2]).double(), w[:, cols].t())


@pytest.mark.parametrize("M,out,inf", [(2, 60, 160), (16, 60, 160), (1200, 3301, 544)])
def test_low_bits_of_zero_points_count(M, out, inf):
    codes, scales, points = layer(out, inf, 5, True)
    g = to_gpu(codes, scales, points, True)
    x = t_of(workloads.gaussian_activations(M, inf, seed=2), np.float16)
    high = g[2] + 16 * torch.randint(0, 16, g[2].shape, dtype=torch.uint8, device=dev())
    assert torch.equal(rbq.gemm_q4(g[0], g[1], x, g[2]), rbq.gemm_q4(g[0], g[1], x, high))
    # no zero points, or 8 everywhere
    eight = torch.full_like(g[2], 8)
    assert torch.equal(rbq.gemm_q4(g[0], g[1], x), rbq.gemm_q4(g[0], g[1], x, eight))


@pytest.mark.parametrize("M", [3, 12, 1300])
def test_broken_rows_and_tokens_stay_apart(M):
    """NaN scales (groups that were not finite) and infinite tokens: their rows and tokens alone."""
    out, inf = 3001, 544
    codes, scales, points = layer(out, inf, 6, True)
    scales[7, 2] = scales[out - 1, 4] = np.float16(np.nan).view(np.uint16)
    g = to_gpu(codes, scales, points, True)
    x = t_of(workloads.gaussian_activations(M, inf, seed=3), np.float16)
    x[M - 2, 500] = float("inf")
    Y = rbq.gemm_q4(g[0], g[1], x, g[2], dtype=torch.float32)
    rows, toks = torch.ones(out, dtype=torch.bool, device=dev()), torch.ones(M, dtype=torch.bool, device=dev())
    rows[7] = rows[out - 1] = toks[M - 2] = False
    assert torch.isnan(Y[:, ~rows]).all() and torch.isfinite(Y[toks][:, rows]).all()
    assert not torch.isfinite(Y[~toks][:, rows]).any() or bool((g[0].int() != 0).all())
    scales[7, 2] = scales[out - 1, 4] = np.float16(1.0).view(np.uint16)
    x[M - 2, 500] = 1.0
    w = weights(codes, scales, points)
    near(Y[toks][:, rows], w[rows], x[toks])


def test_two_graphs_share_a_workspace():
    """Products in several slices, captured, replayed in turn with other work between; a side stream."""
    out, inf = 2500, 4128
    codes, scales, points = layer(out, inf, 8, True)
    g = to_gpu(codes, scales, points, True)
    xs = [t_of(workloads.gaussian_activations(M, inf, seed=M), np.float16) for M in (200, 333)]
    want = [rbq.gemm_q4(g[0], g[1], x, g[2]) for x in xs]
    need = max(int(rbq.lib().rbq_gemm_q4_workspace_bytes(out, inf, x.shape[0], rbq.RBQ_Y_F16)) for x in xs)
    assert need > 0
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=dev())
    graphs = []
    torch.cuda.synchronize()
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = rbq.gemm_q4(g[0], g[1], x, g[2], workspace=ws[:need])
        graphs.append((graph, y))
    for _ in range(3):
        for (graph, y), ref in zip(graphs, want):
            y.zero_()
            graph.replay()
            torch.randn(64, 64, device=dev()).sum()
            torch.cuda.synchronize()
            assert torch.equal(y, ref)
    assert bool((ws[need:] == 255).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rbq.gemm_q4(g[0], g[1], xs[0], g[2], stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])


def test_layers_beyond_32_bit_offsets():
    """More than 2^32 weights and bytes of codes: the last rows are those of the rows alone."""
    out, inf = 2 ** 20 + 5, 8224
    codes = torch.randint(0, 256, (out, inf // 2), dtype=torch.uint8, device=dev())
    scales = (torch.rand(out, 65, device=dev()) * 0.02 + 0.001).half()
    points = torch.randint(0, 16, (out, 65), dtype=torch.uint8, device=dev())
    end = [v[-300:].contiguous() for v in (codes, scales, points)]
    for M in (1, 16):
        x = t_of(workloads.gaussian_activations(M, inf, seed=M), np.float16)
        Y = rbq.gemm_q4(codes, scales, x, points)
        assert torch.equal(Y[:, -300:], rbq.gemm_q4(end[0], end[1], x, end[2]))
    w = weights(np.stack([end[0].cpu().numpy() & 15, end[0].cpu().numpy() >> 4], 2).reshape(300, inf),
                end[1].cpu().numpy().view(np.uint16), end[2].cpu().numpy())
    x = t_of(workloads.gaussian_activations(33, inf, seed=9), np.float16)
    near(rbq.gemm_q4(codes, scales, x, points, dtype=torch.float32)[:, -300:], w, x)
    del codes, scales, points
    W = torch.empty((2 ** 19 + 5, inf), device=dev()).normal_()
    codes, scales, points = rbq.encode_q4(W, zeros=True)
    tail = rbq.encode_q4(W[-300:].contiguous(), zeros=True)
    for a, b in zip((codes, scales, points), tail):
        assert torch.equal(a[-300:], b)


def test_outputs_beyond_32_bit_offsets():
    """More than 2^31 results, and more than 65535 rows of workgroups of tokens."""
    out, inf = 1_100_003, 32
    codes, scales, points = layer(out, inf, 10, True)
    g = to_gpu(codes, scales, points, True)
    M = 2001
    x = t_of(workloads.gaussian_activations(M, inf, seed=1), np.float16)
    Y = rbq.gemm_q4(g[0], g[1], x, g[2])
    w = weights(codes[-70:], scales[-70:], points[-70:])
    near(Y[-70:, -70:], w, x[-70:])
    near(Y[:70, -70:], w, x[:70])
    del Y
    M = 65535 * 16 + 33
    x = torch.randn((M, inf), device=dev()).half()
    small = [v[:3].contiguous() for v in g]
    Y = rbq.gemm_q4(*small[:2], x, small[2], dtype=torch.float32)
    near(Y, weights(codes[:3], scales[:3], points[:3]), x)


def test_refusals():
    codes, scales, points = layer(8, 64, 1, True)
    c, s, z = to_gpu(codes, scales, points, True)
    x = torch.zeros(2, 64, dtype=torch.float16, device=dev())
    f = torch.float32
    for args, kw, what in [
            ((c.int(), s, x), {}, TypeError), ((c, s.float(), x), {}, TypeError), ((c, s, x.float()), {}, TypeError),
            ((c, s, x, z.int()), {}, TypeError), ((c, s, x), {"dtype": torch.bfloat16}, TypeError),
            ((c, s[:, :0], x), {}, (TypeError, ValueError)), ((c, s[:7], x), {}, ValueError),
            ((c, s, x[:, :32].contiguous()), {}, ValueError), ((c, s, x[0]), {}, ValueError),
            ((c, s, x, z[:7]), {}, ValueError), ((c[:, ::2], s, x), {}, (TypeError, ValueError)),
            ((c, s, x.t().contiguous().t()), {}, (TypeError, ValueError)),
            ((c, s, x), {"Y": torch.zeros(2, 9, dtype=torch.float16, device=dev())}, ValueError),
            ((c, s, x), {"Y": torch.zeros(2, 8, dtype=f, device=dev())}, (TypeError, ValueError)),
            ((c, s, x), {"Y": torch.zeros(8, 2, dtype=torch.float16, device=dev()).t()}, (TypeError, ValueError)),
            ((c.cpu(), s, x), {}, TypeError)]:
        with pytest.raises(what):
            rbq.gemm_q4(*args, **kw)
    with pytest.raises(ValueError):
        rbq.gemv_q4(c, s, x)
    with pytest.raises(ValueError):
        rbq.gemv_q4(c, s, x[0], y=torch.zeros(1, 8, dtype=torch.float16, device=dev()))
    W = torch.zeros(4, 64, device=dev())
    for bad in (W.half(), W[:, ::2], W.cpu()):
        with pytest.raises((TypeError, ValueError)):
            rbq.encode_q4(bad)
    with pytest.raises(rbq.RbqError):
        rbq.encode_q4(W[:, :48].contiguous())
    with pytest.raises(ValueError):
        rbq.encode_q4(W[0])
