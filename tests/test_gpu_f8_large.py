"""8-bit linears and checkpoints whose offsets pass 32 bits, against the same
call on the last rows or tokens alone (the same blocks, so the same codes and
scales; sums in another order, within the bounds of test_gpu_f8.py and
test_gpu_qat_ckpt.py), and rows longer than the tiled products take."""
import pytest
import torch

import gemm_rbq_encode_amd as rbq

pytestmark = pytest.mark.gpu
INF = 65536
ROWS = 66000                                     # ROWS * INF > 2^32
LAST = 515 * 128                                 # the first row of the last block of rows


def dev():
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def fill(shape, dtype, seed):
    """Values of mixed sizes, made in pieces."""
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    t = torch.empty(shape, dtype=dtype, device=dev())
    for i in range(0, shape[0], 4096):
        n = min(4096, shape[0] - i)
        t[i:i + n] = torch.randn(n, shape[1], device=dev(), generator=g).to(dtype)
    return t


def values(codes, scales, per_row):
    """fp64 values of 8-bit codes: scales per block of 128 rows, or per row."""
    cols = torch.arange(codes.shape[1], device=dev()) // 128
    s = scales.double()
    s = s.t() if per_row else s[torch.arange(codes.shape[0], device=dev()) // 128]
    return codes.double() * s[:, cols]


@pytest.mark.parametrize("M", [1, 20, 300])
def test_a_weight_beyond_32_bits(M):
    W = fill((ROWS, INF), torch.float32, 1)
    w8, ws = rbq.encode_f8(W)
    tail, tail_s = rbq.encode_f8(W[LAST:].contiguous())
    assert torch.equal(w8[LAST:].view(torch.uint8), tail.view(torch.uint8)) and torch.equal(ws[LAST // 128:], tail_s)
    del W
    X = fill((M, INF), torch.float16, 2)
    x8, xs = rbq.quantize_f8(X)
    w, x = values(tail, tail_s, False), values(x8, xs, True)
    want, S = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()
    T = INF // 128
    t = (INF + 3 * T + 16) * 2.0 ** -23 * S + (7 * 2.0 ** -13 * S if M > 32 else 0.0)
    t = 2.0 ** -11 * (want.abs() + t) + 2.0 ** -25 + t
    Y = rbq.gemm_f8(w8, ws, x8, xs)
    assert bool(((Y[:, LAST:].double() - want).abs() <= t).all())
    if M == 1:
        y = rbq.gemv_f8(w8, ws, X[0])
        assert bool(((y[LAST:].double() - want[0]).abs() <= t[0]).all())


def test_tokens_beyond_32_bits():
    """More than 2^32 codes of tokens, and more than 2^32 outputs."""
    X = fill((ROWS, INF), torch.float16, 3)
    n = 200
    last = X[ROWS - n:].contiguous()
    x8, xs = rbq.quantize_f8(X)
    t8, ts = rbq.quantize_f8(last)
    assert torch.equal(x8[ROWS - n:].view(torch.uint8), t8.view(torch.uint8)) and torch.equal(xs[:, ROWS - n:], ts)
    c, s = rbq.qat_checkpoint(X)
    tc, tsc = rbq.qat_checkpoint(last)
    assert torch.equal(c[ROWS - n:], tc) and torch.equal(s[ROWS - n:], tsc)
    del c, s, X
    w8, ws = rbq.encode_f8(fill((40, INF), torch.float32, 4))
    Y = rbq.gemm_f8(w8, ws, x8, xs, dtype=torch.float32)
    x, w = values(t8, ts, True), values(w8, ws, False)
    want, S = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()
    assert bool(((Y[ROWS - n:].double() - want).abs() <= (INF + 3 * (INF // 128) + 16) * 2.0 ** -23 * S).all())


def test_outputs_beyond_32_bits():
    out, M = 66048, 65540
    w8, ws = rbq.encode_f8(fill((out, 64), torch.float32, 5))
    x8, xs = rbq.quantize_f8(fill((M, 64), torch.float16, 6))
    Y = rbq.gemm_f8(w8, ws, x8, xs)
    n = 128
    x, w = values(x8[M - n:], xs[:, M - n:], True), values(w8[out - n:], ws[out // 128 - 1:], False)
    want, S = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()
    t = (64 + 3 + 16) * 2.0 ** -23 * S + 7 * 2.0 ** -13 * S
    t = 2.0 ** -11 * (want.abs() + t) + 2.0 ** -25 + t
    assert bool(((Y[M - n:, out - n:].double() - want).abs() <= t).all())


def test_rows_longer_than_the_tiles_take():
    """in > 2^23: the few-token kernel serves any number of tokens.  Codes of
    +-1 and scales of 1, so the sums of 2^23 products are exact in fp32."""
    out, M, inf = 33, 40, (1 << 23) + 32
    g = torch.Generator(device=dev())
    g.manual_seed(7)
    one = torch.tensor([0x38, 0xB8], dtype=torch.uint8, device=dev())            # e4m3 +-1
    w8 = one[torch.randint(0, 2, (out, inf), device=dev(), generator=g)].view(torch.float8_e4m3fn)
    x8 = one[torch.randint(0, 2, (M, inf), device=dev(), generator=g)].view(torch.float8_e4m3fn)
    T = -(-inf // 128)
    Y = rbq.gemm_f8(w8, torch.ones(1, T, device=dev()), x8, torch.ones(T, M, device=dev()), dtype=torch.float32)
    want = x8.float().double() @ w8.float().double().t().contiguous()
    assert torch.equal(Y.double(), want)


@pytest.mark.parametrize("out,M", [(64, ROWS), (ROWS, 4), (ROWS, 70)])
def test_backward_beyond_32_bits(out, M):
    """Many tokens (dY zero but for the last ones) and many rows (dX from the
    last ones: the others have scales of zero)."""
    K, n = 2, 40
    g = torch.Generator(device=dev())
    g.manual_seed(8)
    planes = torch.randint(-2 ** 31, 2 ** 31, (K, out, INF // 32), device=dev(), generator=g).int()
    scales = (torch.rand(K, out, 1, device=dev(), generator=g) * 0.02).half()
    X, dY = fill((M, INF), torch.float16, 9), fill((M, out), torch.float16, 10)
    r = min(n, out)
    if M > n:
        dY[:M - n] = 0
    if out > n:
        scales[:, :out - r] = 0
    codes, cs = rbq.qat_checkpoint(X)
    del X
    m = min(n, M)
    lc, ls, ld = codes[M - m:].contiguous(), cs[M - m:].contiguous(), dY[M - m:].contiguous()
    dX, dW, ds = rbq.qat_backward_ckpt(planes, scales, codes, cs, dY)
    # dW's last rows and dX's last tokens, in 64 bits
    x = torch.empty(m, INF, dtype=torch.float64, device=dev())
    cols = torch.arange(INF, device=dev()) // 128
    x[:] = (lc.double() * ls.double()[:, cols]).half().double()
    d = ld[:, out - r:].double()
    want = d.t().contiguous() @ x
    t = 2.0 * M * 2.0 ** -24 * (d.abs().t().contiguous() @ x.abs())
    assert bool(((dW[out - r:].double() - want).abs() <= t + 1e-300).all())
    bits = (planes[:, out - r:, :, None] >> torch.arange(32, device=dev(), dtype=torch.int32)) & 1
    sign = (2 * bits.double() - 1).view(K, r, INF)
    e = ((sign * dW[None, out - r:].double()).sum(2, keepdim=True) - ds[:, out - r:].double()).abs()
    assert bool((e <= 128 * 2.0 ** -24 * dW[None, out - r:].double().abs().sum(2, keepdim=True)
                 + 2.0 ** -23 * ds[:, out - r:].double().abs()).all())
    w = (sign * scales[:, out - r:].double()).sum(0)
    want = d @ w
    a = d.abs() @ w.abs()
    t = d.abs() @ (2.0 ** -21 * w.abs() + 2.0 ** -25) + 4.0 * out * 2.0 ** -24 * a
    assert bool(((dX[M - m:].double() - want).abs() <= t + 1e-300).all())
