"""Calls of the 8-bit operators that their documentation allows and that go
beyond one plain call: scales beyond fp16, outputs inside larger buffers at
any allowed alignment, several streams at once, and graphs that share a
workspace."""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
import test_gpu_f8
from oracle import f8
from test_gpu_qat_ckpt import case, check_grads, dev, t_f16, t_planes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("row", [0, 300, 699])
@pytest.mark.parametrize("M", [3, 100, 200])
def test_overflow_is_flagged_where_a_weight_overflows(row, M):
    """Scales whose sum is beyond fp16: flagged only where planes agree.  700
    rows, in slices and (without a workspace) in one, so that the row is met
    in the first stage, the unchecked ones and the checked last ones."""
    out, inf, K = 700, 160, 2
    planes, s, X, dY = case(out, inf, K, 0, M, 5)
    s = s.copy()
    s[0, row], s[1, row] = (np.array([40000.0, 30000.0], dtype=np.float16)).view(np.uint16)
    planes = planes.copy()
    planes[1, row] = ~planes[0, row]
    codes, cs = rbq.qat_checkpoint(t_f16(X))
    none = torch.empty(0, dtype=torch.uint8, device=dev())

    def flag(p, scales, workspace):
        st = torch.zeros(1, dtype=torch.int32, device=dev())
        got = rbq.qat_backward_ckpt(t_planes(p), t_f16(scales), codes, cs, t_f16(dY), workspace=workspace, status=st)
        torch.cuda.synchronize()
        return got, int(st.item())

    for ws in (None, none):
        got, st = flag(planes, s, ws)
        assert st == 0
        check_grads(got, planes, s, f8.restore(*f8.checkpoint(X)), dY, 0)
        for column in (0, 77, 159):
            p = planes.copy()
            p[1, row, column // 32] ^= np.uint32(1 << (column % 32))
            assert flag(p, s, ws)[1] == rbq.RBQ_STATUS_SCALE_OVERFLOW
        bad = s.copy()
        bad[0, row] = 0x7E00
        assert flag(planes, bad, ws)[1] == rbq.RBQ_STATUS_SCALE_OVERFLOW


def inside(n, offset, fill=-7.0):
    """A float32 buffer of n entries `offset` entries into a larger one."""
    whole = torch.full((n + offset + 300,), fill, dtype=torch.float32, device=dev())
    return whole, whole[offset:]


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("out,inf,K,group,M", [(130, 160, 2, 0, 33), (600, 576, 2, 0, 1100), (100, 256, 4, 128, 70),
                                               (37, 128, 3, 0, 5)])
def test_backward_writes_its_outputs_only(out, inf, K, group, M, offset):
    planes, s, X, dY = case(out, inf, K, group, M, 91)
    a = (t_planes(planes), t_f16(s), *rbq.qat_checkpoint(t_f16(X)), t_f16(dY))
    want = rbq.qat_backward_ckpt(*a, group)
    shape = rbq.shape(out, inf, K, group)
    need = rbq.lib().rbq_qat_backward_ckpt_workspace_bytes(shape, M)
    assert need % 4 == 0
    bufs = [inside(n, offset) for n in (M * inf, out * inf, K * out * (inf // group if group else 1), need // 4)]
    ptr = [b.data_ptr() for _, b in bufs]
    for ws_bytes in (need, max(0, need - 4)):
        st = rbq.lib().rbq_qat_backward_ckpt(a[0].data_ptr(), a[1].data_ptr(), shape, a[2].data_ptr(),
                                             a[3].data_ptr(), a[4].data_ptr(), M, *ptr[:3], ptr[3] if ws_bytes else None,
                                             ws_bytes, None, torch.cuda.current_stream().cuda_stream)
        assert st == rbq.RBQ_OK
        torch.cuda.synchronize()
        for (whole, b), w in zip(bufs, want):
            n = w.numel()
            if ws_bytes == need:
                assert torch.equal(b[:n], w.flatten())
            assert (whole[:offset] == -7).all() and (b[n:] == -7).all()
        whole, b = bufs[3]
        assert (whole[:offset] == -7).all() and (b[need // 4:] == -7).all()
    check_grads([b[:w.numel()].view(w.shape) for (_, b), w in zip(bufs, want)], planes, s,
                f8.restore(*f8.checkpoint(X)), dY, group)


@pytest.mark.parametrize("kind", [torch.float16, torch.float32])
@pytest.mark.parametrize("out,M,inf", [(132, 5, 160), (130, 33, 416), (500, 300, 1056), (1024, 600, 288),
                                       (4096, 64, 1024)])
def test_gemm_writes_its_output_only(out, M, inf, kind):
    W = torch.randn(out, inf, device=dev())
    w8, ws = rbq.encode_f8(W)
    x8, xs = rbq.quantize_f8(torch.randn(M, inf, device=dev()).half())
    want = rbq.gemm_f8(w8, ws, x8, xs, dtype=kind)
    y32 = int(kind == torch.float32)
    need = rbq.lib().rbq_gemm_f8_workspace_bytes(out, inf, M, y32)
    for offset in (0, 1, 2):
        whole = torch.full((M * out + 900,), -7.0, dtype=kind, device=dev())
        y = whole[offset:]
        space, wk = inside(need // 4, offset)
        st = rbq.lib().rbq_gemm_f8(w8.data_ptr(), ws.data_ptr(), out, inf, x8.data_ptr(), xs.data_ptr(), M,
                                   y.data_ptr(), y32, wk.data_ptr() if need else None, need, None)
        assert st == rbq.RBQ_OK
        torch.cuda.synchronize()
        assert torch.equal(y[:M * out], want.flatten())
        assert (whole[:offset] == -7).all() and (y[M * out:] == -7).all()
        assert (space[:offset] == -7).all() and (wk[need // 4:] == -7).all()


def sliced_product(M):
    """Operands of a product whose columns are split through the workspace."""
    w8, ws = rbq.encode_f8(torch.randn(1024, 8192, device=dev()))
    assert rbq.lib().rbq_gemm_f8_workspace_bytes(1024, 8192, M, 0) > 0
    return w8, ws, rbq.quantize_f8(torch.randn(M, 8192, device=dev()).half())


def test_two_streams_at_once():
    """The same inputs on two streams, each with workspaces of its own."""
    out, inf, K, M = 4096, 1024, 2, 64
    planes, s, X, dY = case(out, inf, K, 0, M, 17)
    a = (t_planes(planes), t_f16(s), *rbq.qat_checkpoint(t_f16(X)), t_f16(dY))
    w8, ws, q = sliced_product(M)
    want, y = rbq.qat_backward_ckpt(*a), rbq.gemm_f8(w8, ws, *q)
    assert rbq.lib().rbq_qat_backward_ckpt_workspace_bytes(rbq.shape(out, inf, K, 0), M) > 0
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for st, g in zip(streams, got):
            with torch.cuda.stream(st):
                g.append((*rbq.qat_backward_ckpt(*a), rbq.gemm_f8(w8, ws, *q)))
    torch.cuda.synchronize()
    for g in got:
        for r in g:
            assert all(torch.equal(u, v) for u, v in zip(r, (*want, y)))


def test_graphs_that_share_a_workspace():
    """One workspace for a product and two captured backward passes, replayed
    one after another on one stream, in both orders, between eager calls that
    use it too."""
    out, inf, K, M = 4096, 1024, 2, 64
    planes, s, X, dY = case(out, inf, K, 0, M, 23)
    a = (t_planes(planes), t_f16(s), *rbq.qat_checkpoint(t_f16(X)), t_f16(dY))
    b = (*a[:4], t_f16(dY[::-1].copy()))
    w8, ws, q = sliced_product(M)
    need = max(rbq.lib().rbq_qat_backward_ckpt_workspace_bytes(rbq.shape(out, inf, K, 0), M),
               rbq.lib().rbq_gemm_f8_workspace_bytes(*w8.shape, M, 0))
    space = torch.empty(need, dtype=torch.uint8, device=dev())
    wants = [rbq.qat_backward_ckpt(*a), rbq.qat_backward_ckpt(*b)]
    y = rbq.gemm_f8(w8, ws, *q)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for args in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(rbq.qat_backward_ckpt(*args, workspace=space))
        graphs.append(g)
    for rep in range(6):
        for o in outs:
            for t in o:
                t.fill_(3.0)
        order = (0, 1) if rep % 2 else (1, 0)
        for i in order:
            graphs[i].replay()
            e = rbq.gemm_f8(w8, ws, *q, workspace=space)
        torch.cuda.synchronize()
        assert torch.equal(e, y)
        for o, w in zip(outs, wants):
            assert all(torch.equal(u, v) for u, v in zip(o, w))


def test_the_same_input_twice():
    """One tensor as both operands' source, and one buffer of codes and scales
    read by two products at once."""
    n = 256
    x = torch.randn(n, n, device=dev()).half()
    w8, ws = rbq.encode_f8(x.float())
    q = rbq.quantize_f8(x)
    y = rbq.gemm_f8(w8, ws, *q, dtype=torch.float32)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y1 = rbq.gemm_f8(w8, ws, *q, dtype=torch.float32, stream=st)
    y2 = rbq.gemm_f8(w8, ws, *q, dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(y, y1) and torch.equal(y, y2)
    c = rbq.qat_checkpoint(x)
    planes, scales = rbq.encode(x.float(), 2)
    d = rbq.qat_backward_ckpt(planes, scales, *c, x)
    torch.cuda.synchronize()
    p = planes.cpu().numpy().view(np.uint32)
    xb = x.cpu().numpy().view(np.uint16)
    check_grads(d, p, scales.cpu().numpy().view(np.uint16), f8.restore(*f8.checkpoint(xb)), xb, 0)


@pytest.mark.parametrize("out,M,inf", [(5003, 777, 4128), (7568, 1066, 3040)])
def test_gemm_of_whole_and_sliced_tiles(out, M, inf):
    """More tiles than compute units, the last ones split: within the bounds
    of the other tiles, with the workspace and without."""
    need = rbq.lib().rbq_gemm_f8_workspace_bytes(out, inf, M, rbq.RBQ_Y_F32)
    assert 0 < need < 4 * M * out
    test_gpu_f8.test_gemm_tiles_match_the_definition_in_64_bits(out, M, inf, False)


# one round of tiles of 256, 224 and 192 rows by 256 tokens; no, one and
# several whole blocks of columns, with and without a short last one
HEIGHTS = [(out, M, inf) for out, M in [(8191, 2047), (7168, 2041), (7001, 2048), (6140, 2000), (6144, 2048)]
           for inf in (64, 128, 288, 384, 640)] + [(7167, 2048, 2144), (6143, 2048, 2144), (8190, 2048, 2144)]


@pytest.mark.parametrize("out,M,inf", HEIGHTS)
def test_gemm_tiles_of_every_height(out, M, inf):
    test_gpu_f8.test_gemm_tiles_match_the_definition_in_64_bits(out, M, inf, True)


@pytest.mark.parametrize("out,inf,K,group,M", [(600, 576, 2, 0, 1100), (100, 160, 1, 0, 70), (1030, 640, 4, 128, 300),
                                               (257, 1056, 3, 0, 130), (2050, 2048, 2, 0, 128)])
def test_gradients_asked_for_one_by_one(out, inf, K, group, M):
    """Kernels of their own serve dX alone and dW with or without the scales'
    gradients; with the workspace and without."""
    planes, s, X, dY = case(out, inf, K, group, M, out + 3 * M)
    a = (t_planes(planes), t_f16(s), *rbq.qat_checkpoint(t_f16(X)), t_f16(dY), group)
    x = f8.restore(*f8.checkpoint(X))
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=dev())):
        dx = rbq.qat_backward_ckpt(*a, need_dw=False, need_dscales=False, workspace=ws)
        dw = rbq.qat_backward_ckpt(*a, need_dx=False, need_dscales=False, workspace=ws)
        ds = rbq.qat_backward_ckpt(*a, need_dx=False, workspace=ws)
        both = rbq.qat_backward_ckpt(*a, need_dscales=False, workspace=ws)
        torch.cuda.synchronize()
        assert dx[1:] == (None, None) and (dw[0], dw[2]) == (None, None) and ds[0] is None and both[2] is None
        for got in (dx, dw, ds, both):
            check_grads(got, planes, s, x, dY, group)
