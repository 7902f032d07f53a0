"""Host-side checks of the 8-bit block operators: the oracle (oracle/f8.py)
against closed forms and against torch's own e4m3 and fp16 types, and the
arguments that the C ABI and the binding refuse before anything is launched."""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
import workloads
from gemm_rbq_encode_amd import _binding
from oracle import f8

pytestmark = pytest.mark.cpu


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(f8.e4m3_table(), t)


def test_e4m3_rounding_is_torchs():
    rng = np.random.default_rng(1)
    tab = f8.e4m3_table()[:0x7F]
    mids = (tab[1:] + tab[:-1]) / 2                         # every tie
    v = np.concatenate([tab, mids, np.nextafter(mids, 0), np.nextafter(mids, 500), rng.uniform(0, 448, 5000),
                        2.0 ** rng.uniform(-14, 8, 5000)]).astype(np.float32)
    v = np.concatenate([v, -v])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(f8.e4m3_codes(v.astype(np.float64)), want)


def test_block_scale_and_error():
    """The largest entry takes +-448 and every value is within half a step:
    2^-4 of itself, or half of the format's smallest step 2^-9 of the scale
    (plus the fp32 roundings of the two quotients and of the product)."""
    W = workloads.gaussian_weight(130, 288, 3, outliers=True)
    codes, scales = f8.encode(W)
    assert scales.shape == (2, 3) and codes.shape == W.shape
    v = f8.values(codes, scales, 128)
    s = np.repeat(np.repeat(scales, 128, 0)[:130], 128, 1)[:, :288].astype(np.float64)
    assert (np.abs(v - W) <= (1 + 2.0 ** -21) * np.maximum(np.abs(W) * 2.0 ** -4, s * 2.0 ** -10)
            + np.abs(W) * 2.0 ** -21).all()
    for i in range(2):
        for t in range(3):
            b = codes[128 * i:128 * i + 128, 128 * t:128 * t + 128] & 0x7F
            assert b.max() == 0x7E
    zero, sz = f8.encode(np.zeros((3, 32), np.float32))
    assert not zero.any() and sz[0, 0] == np.float32(2.0 ** -100 / 448)
    bad = W.copy()
    bad[0, 130] = np.inf
    c, s2 = f8.encode(bad)
    assert np.isnan(s2[0, 1]) and not c[:128, 128:256].any() and np.isfinite(np.delete(s2.ravel(), 1)).all()


def test_checkpoint_of_every_fp16_maximum():
    """For every finite fp16 maximum: the scale is the smallest allowed one,
    the value restored for it is finite and within half a step of it."""
    A = np.arange(0x7C00, dtype=np.uint16)
    X = np.zeros((len(A), 32), np.uint16)
    X[:, 5] = A
    X[:, 6] = A | 0x8000
    X[:, 7] = A // 2
    codes, scales = f8.checkpoint(X)
    s = scales[:, 0].view(np.float16).astype(np.float64)
    a = A.view(np.float16).astype(np.float64)
    assert (s >= 2.0 ** -24).all() and (s <= 515.5).all()
    capped = a / 127 > 515.5
    assert (s[~capped] * 127 >= a[~capped]).all() and capped.sum() == 2   # 65472, 65504
    x = f8.restore(codes, scales).view(np.float16).astype(np.float64)
    v = X.view(np.float16).astype(np.float64)
    assert np.isfinite(x).all()
    step = np.where(capped, 64.0, s)[:, None]               # beyond the cap: 32 lost, and one rounding
    assert (np.abs(x - v) <= step / 2 + np.abs(v) * 2.0 ** -11 + 2.0 ** -25).all()
    tiny = a <= 127 * 2.0 ** -24
    assert (x[tiny] == v[tiny]).all()


def test_checkpoint_quotients_stay_off_the_borders():
    """A quotient x / s that is no tie is at least 2^-12 from a half-integer:
    the codes do not depend on how the quotient is computed."""
    rng = np.random.default_rng(2)
    s = rng.integers(1, 0x6008, 20000).astype(np.uint16).view(np.float16).astype(np.float64)
    k = rng.integers(0, 127, 20000) + 0.5
    near = (s * k).astype(np.float16).astype(np.float64)
    for v in (near, np.nextafter(near.astype(np.float16), np.float16(0)).astype(np.float64)):
        q = v / s
        ok = (q >= 0.25) & (q <= 127)
        d = np.abs(q - (np.floor(q) + 0.5))[ok]
        assert ((d == 0) | (d >= 2.0 ** -12)).all()


def test_checkpoint_of_non_finite_blocks():
    X = workloads.gaussian_activations(3, 288, 4).copy()
    X[1, 200] = 0x7C00
    X[2, 0] = 0x7E01
    codes, scales = f8.checkpoint(X)
    x = f8.restore(codes, scales).view(np.float16)
    assert np.isnan(x[1, 128:256]).all() and np.isnan(x[2, :128]).all()
    assert np.isfinite(x[0]).all() and np.isfinite(x[1, :128]).all() and np.isfinite(x[1, 256:]).all()


OK = 0x10000   # an aligned stand-in address: checks never dereference it


def test_f8_argument_errors():
    L, E = rbq.lib(), rbq
    bad, al = E.RBQ_ERR_INVALID_ARG, E.RBQ_ERR_ALIGNMENT
    assert L.rbq_encode_f8(None, 8, 64, OK, OK, None, None) == bad
    assert L.rbq_encode_f8(OK, 8, 64, None, OK, None, None) == bad
    assert L.rbq_encode_f8(OK, 8, 64, OK, None, None, None) == bad
    assert L.rbq_encode_f8(OK, -1, 64, OK, OK, None, None) == bad
    assert L.rbq_encode_f8(OK, 8, 48, OK, OK, None, None) == bad
    assert L.rbq_encode_f8(OK, 8, -32, OK, OK, None, None) == bad
    assert L.rbq_encode_f8(OK + 8, 8, 64, OK, OK, None, None) == al
    assert L.rbq_encode_f8(OK, 8, 64, OK + 8, OK, None, None) == al
    assert L.rbq_encode_f8(OK, 8, 64, OK, OK + 2, None, None) == al
    assert L.rbq_encode_f8(OK, 8, 64, OK, OK, OK + 2, None) == al
    assert L.rbq_encode_f8(None, 0, 64, None, None, None, None) == E.RBQ_OK
    assert L.rbq_encode_f8(None, 8, 0, None, None, None, None) == E.RBQ_OK
    assert L.rbq_quantize_f8(None, 2, 64, OK, OK, None) == bad
    assert L.rbq_quantize_f8(OK, -1, 64, OK, OK, None) == bad
    assert L.rbq_quantize_f8(OK, 2, 33, OK, OK, None) == bad
    assert L.rbq_quantize_f8(OK + 2, 2, 64, OK, OK, None) == al
    assert L.rbq_quantize_f8(OK, 2, 64, OK + 4, OK, None) == al
    assert L.rbq_quantize_f8(None, 0, 64, None, None, None) == E.RBQ_OK
    assert L.rbq_gemm_f8(OK, OK, 8, 64, OK, OK, 2, OK, 2, None, 0, None) == bad
    assert L.rbq_gemm_f8(OK, OK, 8, 64, OK, OK, -2, OK, 0, None, 0, None) == bad
    assert L.rbq_gemm_f8(OK, OK, 8, 40, OK, OK, 2, OK, 0, None, 0, None) == bad
    for k in (0, 1, 4, 5, 7):
        a = [OK, OK, 8, 64, OK, OK, 2, OK, 0, None, 0, None]
        a[k] = None
        assert L.rbq_gemm_f8(*a) == bad, k
    for k, off in ((0, 8), (1, 2), (4, 8), (5, 2), (7, 1)):
        a = [OK, OK, 8, 64, OK, OK, 2, OK, 0, None, 0, None]
        a[k] = OK + off
        assert L.rbq_gemm_f8(*a) == al, k
    assert L.rbq_gemm_f8(OK, OK, 8, 64, OK, OK, 2, OK + 2, 1, None, 0, None) == al
    assert L.rbq_gemm_f8(None, None, 8, 64, None, None, 0, None, 0, None, 0, None) == E.RBQ_OK
    assert L.rbq_gemm_f8(None, None, 0, 64, None, None, 3, None, 0, None, 0, None) == E.RBQ_OK
    assert L.rbq_gemm_f8(OK, OK, 8, 64, OK, OK, 2, OK, 0, None, 64, None) == bad
    assert L.rbq_gemm_f8(OK, OK, 8, 64, OK, OK, 2, OK, 0, OK + 2, 64, None) == al
    for a in ((8, 40, 2, 0), (8, 64, -1, 0), (0, 64, 300, 0), (-8, 64, 300, 0), (8, 0, 300, 0), (8, 64, 300, 2)):
        assert L.rbq_gemm_f8_workspace_bytes(*a) == 0, a
    for k in (0, 1, 4, 5):
        a = [OK, OK, 8, 64, OK, OK, None]
        a[k] = None
        assert L.rbq_gemv_f8(*a) == bad, k
    for k, off in ((0, 8), (1, 2), (4, 8), (5, 1)):
        a = [OK, OK, 8, 64, OK, OK, None]
        a[k] = OK + off
        assert L.rbq_gemv_f8(*a) == al, k
    assert L.rbq_gemv_f8(OK, OK, 8, 20, OK, OK, None) == bad
    assert L.rbq_gemv_f8(None, None, 0, 64, None, None, None) == E.RBQ_OK


def test_layers_beyond_the_limit_are_refused():
    L, un, big = rbq.lib(), rbq.RBQ_ERR_UNSUPPORTED, (1 << 25) + 32
    assert L.rbq_encode_f8(OK, big, 64, OK, OK, None, None) == un
    assert L.rbq_encode_f8(OK, 8, big, OK, OK, None, None) == un
    assert L.rbq_quantize_f8(OK, 2, big, OK, OK, None) == un
    assert L.rbq_gemm_f8(OK, OK, big, 64, OK, OK, 2, OK, 0, None, 0, None) == un
    assert L.rbq_gemv_f8(OK, OK, 8, big, OK, OK, None) == un
    assert L.rbq_qat_checkpoint(OK, 2, big, OK, OK, None) == un
    for s in (rbq.shape(big, 64, 2, 0), rbq.shape(8, big, 2, 0)):
        assert L.rbq_qat_backward_ckpt(OK, OK, s, OK, OK, OK, 4, OK, OK, OK, None, 0, None, None) == un
        assert L.rbq_qat_backward_ckpt_workspace_bytes(s, 4) == 0
    assert L.rbq_gemm_f8_workspace_bytes(big, 64, 300, 0) == 0


def test_a_stream_of_another_device_is_refused():
    class Stream:
        cuda_stream, device = 1, torch.device("cuda:1")

    with pytest.raises(ValueError):
        _binding._There(torch.device("cuda:0"), Stream())


def test_workspaces_are_no_larger_than_their_slices():
    """A handful of slices of the outputs at most, for every size."""
    L = rbq.lib()
    for out in (1, 5, 500, 4096, 11008, 1 << 25):
        for inf in (32, 512, 4128, 14336, 1 << 25):
            for M in (1, 33, 128, 2048, 1 << 20, 2 ** 31 - 1):
                for kind in (0, 1):
                    n = L.rbq_gemm_f8_workspace_bytes(out, inf, M, kind)
                    assert n % 16 == 0 and n <= 8 * 4 * -(-M // 256) * 256 * -(-out // 128) * 128 * 1.05
                s = rbq.shape(out, inf, 4, 0)
                n = L.rbq_qat_backward_ckpt_workspace_bytes(s, M)
                assert n <= 4 * (8 * out * inf + 8 * 4 * out * (inf // 128 + 1) + 32 * M * inf)


def test_checkpoint_argument_errors():
    L, E = rbq.lib(), rbq
    bad, al = E.RBQ_ERR_INVALID_ARG, E.RBQ_ERR_ALIGNMENT
    assert L.rbq_qat_checkpoint(None, 2, 64, OK, OK, None) == bad
    assert L.rbq_qat_checkpoint(OK, 2, 64, None, OK, None) == bad
    assert L.rbq_qat_checkpoint(OK, 2, 64, OK, None, None) == bad
    assert L.rbq_qat_checkpoint(OK, 2, 63, OK, OK, None) == bad
    assert L.rbq_qat_checkpoint(OK, -2, 64, OK, OK, None) == bad
    assert L.rbq_qat_checkpoint(OK + 8, 2, 64, OK, OK, None) == al
    assert L.rbq_qat_checkpoint(OK, 2, 64, OK + 8, OK, None) == al
    assert L.rbq_qat_checkpoint(OK, 2, 64, OK, OK + 1, None) == al
    assert L.rbq_qat_checkpoint(None, 0, 64, None, None, None) == E.RBQ_OK
    s = rbq.shape(64, 128, 2, 0)
    ok = [OK, OK, s, OK, OK, OK, 4, OK, OK, OK, None, 0, None, None]

    def call(**change):
        a = list(ok)
        for k, v in change.items():
            a[int(k[1:])] = v
        return L.rbq_qat_backward_ckpt(*a)

    assert call(_2=rbq.shape(64, 100, 2, 0)) == bad
    assert call(_2=rbq.shape(64, 128, 5, 0)) == E.RBQ_ERR_UNSUPPORTED
    assert call(_6=-1) == bad
    assert call(_8=None) == bad                       # dscales without dW
    assert call(_11=64) == bad                        # a workspace size without one
    for k in ("_0", "_1", "_3", "_4", "_5"):
        assert call(**{k: None}) == bad, k
    for k, off in (("_0", 2), ("_1", 1), ("_3", 8), ("_4", 1), ("_5", 1), ("_7", 2), ("_8", 2), ("_9", 2), ("_12", 2)):
        assert call(**{k: OK + off}) == al, k
    assert call(_7=None, _8=None, _9=None) == E.RBQ_OK
    assert L.rbq_qat_backward_ckpt_workspace_bytes(rbq.shape(64, 100, 2, 0), 4) == 0
    assert L.rbq_qat_backward_ckpt_workspace_bytes(s, 0) == 0


def test_binding_refuses_host_tensors_and_types():
    f = torch.zeros(4, 64)
    for call in (lambda: rbq.encode_f8(f), lambda: rbq.quantize_f8(f.half()), lambda: rbq.qat_checkpoint(f.half()),
                 lambda: rbq.gemv_f8(f.to(torch.float8_e4m3fn), f, f.half()),
                 lambda: rbq.gemm_f8(f.to(torch.float8_e4m3fn), f, f.to(torch.float8_e4m3fn), f)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="only meaningful without a GPU")
def test_valid_calls_without_a_device():
    L, none = rbq.lib(), rbq.RBQ_ERR_NO_DEVICE
    assert L.rbq_encode_f8(OK, 8, 64, OK, OK, None, None) == none
    assert L.rbq_quantize_f8(OK, 2, 64, OK, OK, None) == none
    assert L.rbq_gemm_f8(OK, OK, 8, 64, OK, OK, 2, OK, 0, None, 0, None) == none
    assert L.rbq_gemm_f8(None, None, 8, 0, None, None, 2, OK, 1, None, 0, None) == none
    assert L.rbq_gemv_f8(OK, OK, 8, 64, OK, OK, None) == none
    assert L.rbq_qat_checkpoint(OK, 2, 64, OK, OK, None) == none
    s = rbq.shape(64, 128, 2, 0)
    assert L.rbq_qat_backward_ckpt(OK, OK, s, OK, OK, OK, 4, OK, OK, OK, None, 0, None, None) == none


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="only meaningful without a GPU")
def test_a_layer_without_rows_needs_no_output_gradient():
    """dY [M][0] may have no address (an empty tensor's is NULL): dX = 0 is an empty sum."""
    L, s = rbq.lib(), rbq.shape(0, 128, 2, 0)
    for call in (L.rbq_qat_backward_ckpt(None, None, s, None, None, None, 4, OK, None, None, None, 0, None, None),
                 L.rbq_qat_backward(None, None, s, None, None, 4, OK, None, None, None, 0, None, None)):
        assert call == rbq.RBQ_ERR_NO_DEVICE
    s = rbq.shape(8, 128, 2, 0)
    assert L.rbq_qat_backward(OK, OK, s, OK, None, 4, OK, None, None, None, 0, None, None) == rbq.RBQ_ERR_INVALID_ARG


def test_types_of_product_outputs():
    """RBQ_Y_EXACT goes with either type and nothing else does; exact products
    are split alike for both types."""
    L, E = rbq.lib(), rbq
    for kind in (2, 3, 4, 0x101 + 1, 0x200, 0x1000, 0xFFFFFFFF):
        assert L.rbq_gemm_f8(OK, OK, 8, 64, OK, OK, 2, OK, kind, None, 0, None) == E.RBQ_ERR_INVALID_ARG, kind
        assert L.rbq_gemm_f8_workspace_bytes(1024, 8192, 64, kind) == 0
    for kind in (E.RBQ_Y_F16, E.RBQ_Y_F32, E.RBQ_Y_F16 | E.RBQ_Y_EXACT, E.RBQ_Y_F32 | E.RBQ_Y_EXACT):
        assert L.rbq_gemm_f8(OK, OK, 8, 64, OK, OK, 0, OK, kind, None, 0, None) == E.RBQ_OK
        odd = L.rbq_gemm_f8(OK, OK, 8, 64, OK, OK, 2, OK + 2, kind, None, 0, None)
        assert (odd == E.RBQ_ERR_ALIGNMENT) == bool(kind & E.RBQ_Y_F32)
    for M in (33, 300, 777, 2048):
        f32 = L.rbq_gemm_f8_workspace_bytes(5003, 4128, M, E.RBQ_Y_F32)
        assert L.rbq_gemm_f8_workspace_bytes(5003, 4128, M, E.RBQ_Y_F16 | E.RBQ_Y_EXACT) == f32
        assert L.rbq_gemm_f8_workspace_bytes(5003, 4128, M, E.RBQ_Y_F32 | E.RBQ_Y_EXACT) == f32
