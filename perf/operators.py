"""Measured cases of the 8-bit block operators of rbq: linear layers held in
8-bit floating point with a scale for each block of 128 (encode_f8,
quantize_f8, gemm_f8, gemv_f8), and 8-bit activation checkpoints of the
coupled forward with the backward that reads them (qat_checkpoint,
qat_backward_ckpt).

`own` False computes every case in elementary torch operations in 32 bits;
True makes the calls a user makes of the package.  Sizes are the linears of
workloads.py, and ragged ones around them.
"""
import math

import torch

own = False

BLOCK = 128
TINY = 2.0 ** -100          # the smallest block maximum that f8 scales are made for
F8_MAX = 448.0              # largest e4m3 value
F16_TINY = 2.0 ** -24
CKPT_TOP = 515.5            # largest checkpoint scale: 127 * 515.5 rounds to a finite fp16


# --- cases --------------------------------------------------------------------

def listed():
    return [
        # a frozen linear (gate projection) encoded once when a model is loaded
        dict(name="encode_f8 14336x4096", op="encode_f8", out=14336, inf=4096),
        # the input of one layer at decode, a batch of 4: latency
        dict(name="quantize_f8 4x4096", op="quantize_f8", tokens=4, inf=4096),
        # the input of a down projection in a prefill chunk
        dict(name="quantize_f8 2048x14336", op="quantize_f8", tokens=2048, inf=14336),
        # one decoded token through an up projection: fp16 in, fp16 out, the weight read is all that counts
        dict(name="gemv_f8 11008x4096", op="gemv_f8", out=11008, inf=4096),
        # a decode batch of 16 through a down projection
        dict(name="gemm_f8 16 4096x11008", op="gemm_f8", tokens=16, out=4096, inf=11008, wide=False),
        # a prefill chunk of 2048 tokens through a gate projection
        dict(name="gemm_f8 2048 14336x4096", op="gemm_f8", tokens=2048, out=14336, inf=4096, wide=False),
        # a ragged prompt, rows that fill no tile, a short last block; fp32 outputs (a gradient, logits)
        dict(name="gemm_f8 777 5003x4128 fp32", op="gemm_f8", tokens=777, out=5003, inf=4128, wide=True),
        # the kept input of one layer, a short sequence: latency
        dict(name="checkpoint 16x4096", op="checkpoint", tokens=16, inf=4096),
        # the kept input of a down projection in a training step
        dict(name="checkpoint 4096x11008", op="checkpoint", tokens=4096, inf=11008),
        # few tokens: the write of the weight gradient is what counts
        dict(name="backward 16 4096x4096 K2", op="backward", tokens=16, out=4096, inf=4096, planes=2, group=0),
        # an up projection in a training step of 2048 tokens, scales per row
        dict(name="backward 2048 11008x4096 K2", op="backward", tokens=2048, out=11008, inf=4096, planes=2, group=0),
        # an attention projection, four planes with scales per group, a ragged batch
        dict(name="backward 1003 5120x5120 K4 g128", op="backward", tokens=1003, out=5120, inf=5120, planes=4, group=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["encode_f8", "quantize_f8", "gemv_f8", "gemm_f8", "gemm_f8", "checkpoint", "backward", "backward"])
    inf = 32 * _log(rng, 16, 448)                      # 512 .. 14336, short last blocks among them
    out = _log(rng, 500, 14336)
    if op == "encode_f8":
        return dict(op=op, out=out, inf=inf)
    if op == "gemv_f8":
        return dict(op=op, out=out, inf=inf)
    if op in ("quantize_f8", "checkpoint"):
        return dict(op=op, tokens=_log(rng, 1, 4096), inf=min(inf, 11008))
    if op == "gemm_f8":
        tokens = _log(rng, 1, 2048)
        while tokens * out * inf > 2048 * 14336 * 4096:
            tokens //= 2
        return dict(op=op, tokens=tokens, out=out, inf=inf, wide=rng.random() < 0.5)
    group = rng.choice([0, 128])
    if group:
        inf = max(512, inf // 128 * 128)
    tokens = _log(rng, 1, 2048)
    while tokens * out * inf > 1024 * 11008 * 4096 or out * inf > 11008 * 4096:
        tokens = max(1, tokens // 2)
        out = max(500, out * 3 // 4)
    return dict(op=op, tokens=tokens, out=out, inf=inf, planes=rng.choice([1, 2, 3, 4]), group=group)


# --- inputs -------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *size):
    return torch.randn(size, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, tokens, inf):
    """fp16 activations: unit normal, a few channels 20 times as large, and (in a batch) a padded token of zeros."""
    x = _normal(g, tokens, inf)
    x[:, torch.randint(0, inf, (max(1, inf // 500),), generator=g, device="cuda")] *= 20.0
    if tokens > 8:
        x[tokens // 2] = 0.0
    return x.half()


def _weight(g, out, inf):
    w = _normal(g, out, inf) * 0.02
    pos = torch.randint(0, out * inf, (max(1, out * inf // 1000),), generator=g, device="cuda")
    w.view(-1)[pos] *= 20.0
    return w


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "encode_f8":
        return dict(op=op, w=_weight(g, case["out"], case["inf"]))
    if op in ("quantize_f8", "checkpoint"):
        return dict(op=op, x=_activations(g, case["tokens"], case["inf"]))
    if op == "gemv_f8":
        w8, ws = _encode_f8(_weight(g, case["out"], case["inf"]))
        return dict(op=op, w8=w8, ws=ws, x=_activations(g, 1, case["inf"])[0].contiguous())
    if op == "gemm_f8":
        w8, ws = _encode_f8(_weight(g, case["out"], case["inf"]))
        x8, xs = _quantize_f8(_activations(g, case["tokens"], case["inf"]))
        return dict(op=op, w8=w8, ws=ws, x8=x8, xs=xs, dtype=torch.float32 if case["wide"] else torch.float16)
    K, out, inf, group = case["planes"], case["out"], case["inf"], case["group"]
    planes = torch.randint(-2 ** 31, 2 ** 31, (K, out, inf // 32), generator=g, device="cuda", dtype=torch.int64).int()
    size = (K, out, inf // group if group else 1)
    scales = (torch.rand(size, generator=g, device="cuda") * 0.02 + 0.002).half()
    codes, cs = _checkpoint(_activations(g, case["tokens"], inf))
    dy = (_normal(g, case["tokens"], out) * 0.01).half()
    return dict(op=op, planes=planes, scales=scales, codes=codes, cs=cs, dy=dy, group=group)


# --- the plain forms ----------------------------------------------------------

def _padded(x, dim):
    n = -x.shape[dim] % BLOCK
    if n == 0:
        return x
    size = list(x.shape)
    size[dim] = n
    return torch.cat([x, x.new_zeros(size)], dim)


def _f8_scale(top):
    """(reciprocal scale, scale) of block maxima: each one 64-bit quotient rounded once to 32 bits, as codes next to a
    border go by the last bit."""
    return (F8_MAX / top.double()).float(), (top.double() / F8_MAX).float()


def _encode_f8(w):
    out, inf = w.shape
    p = _padded(_padded(w, 0), 1)
    b = p.view(p.shape[0] // BLOCK, BLOCK, p.shape[1] // BLOCK, BLOCK)
    inv, scales = _f8_scale(b.abs().amax((1, 3)).clamp_min(TINY))
    codes = (b * inv[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(p.shape)[:out, :inf].contiguous(), scales


def _quantize_f8(x):
    M, inf = x.shape
    p = _padded(x.float(), 1)
    b = p.view(M, p.shape[1] // BLOCK, BLOCK)
    inv, scales = _f8_scale(b.abs().amax(2).clamp_min(TINY))
    codes = (b * inv[:, :, None]).to(torch.float8_e4m3fn)
    return codes.view(p.shape)[:, :inf].contiguous(), scales.t().contiguous()


def _over_columns(s, inf):
    """One value per block -> one per column."""
    return s.repeat_interleave(BLOCK, -1)[..., :inf]


def _product_f8(w8, ws, x8, xs):
    out, inf = w8.shape
    w = w8.float() * _over_columns(ws, inf).repeat_interleave(BLOCK, 0)[:out]
    x = x8.float() * _over_columns(xs.t(), inf)
    return x @ w.t()


def _checkpoint(x):
    M, inf = x.shape
    p = _padded(x.float(), 1)
    b = p.view(M, p.shape[1] // BLOCK, BLOCK)
    want = b.abs().amax(2).double() / 127.0
    s = want.half()
    up = (s.view(torch.int16) + 1).view(torch.float16)
    s = torch.where(s.double() < want, up, s).float().clamp(F16_TINY, CKPT_TOP)
    codes = torch.round(b / s[:, :, None]).clamp(-127, 127).to(torch.int8)
    return codes.view(p.shape)[:, :inf].contiguous(), s.half()


def _signs(planes, k, inf):
    bits = torch.arange(32, device=planes.device, dtype=torch.int32)
    return ((planes[k].unsqueeze(-1) >> bits) & 1).view(planes.shape[1], inf).float() * 2 - 1


def _backward(planes, scales, codes, cs, dy, group):
    inf = codes.shape[1]
    K, out, G = scales.shape
    x = (codes.float() * _over_columns(cs.float(), inf)).half().float()
    d = dy.float()
    dw = d.t() @ x
    what, ds = 0.0, []
    for k in range(K):
        b = _signs(planes, k, inf).view(out, G, inf // G)
        what = what + b * scales[k].float().unsqueeze(-1)
        ds.append((b * dw.view(out, G, inf // G)).sum(-1))
    return d @ what.view(out, inf), dw, torch.stack(ds)


def run(s):
    op = s["op"]
    if own:
        import gemm_rbq_encode_amd as rbq
        if op == "encode_f8":
            return rbq.encode_f8(s["w"])
        if op == "quantize_f8":
            return rbq.quantize_f8(s["x"])
        if op == "gemv_f8":
            return rbq.gemv_f8(s["w8"], s["ws"], s["x"])
        if op == "gemm_f8":
            return rbq.gemm_f8(s["w8"], s["ws"], s["x8"], s["xs"], dtype=s["dtype"])
        if op == "checkpoint":
            return rbq.qat_checkpoint(s["x"])
        return rbq.qat_backward_ckpt(s["planes"], s["scales"], s["codes"], s["cs"], s["dy"], s["group"])
    if op == "encode_f8":
        return _encode_f8(s["w"])
    if op == "quantize_f8":
        return _quantize_f8(s["x"])
    if op == "gemv_f8":
        return _product_f8(s["w8"], s["ws"], *_quantize_f8(s["x"].view(1, -1)))[0].half()
    if op == "gemm_f8":
        return _product_f8(s["w8"], s["ws"], s["x8"], s["xs"]).to(s["dtype"])
    if op == "checkpoint":
        return _checkpoint(s["x"])
    return _backward(s["planes"], s["scales"], s["codes"], s["cs"], s["dy"], s["group"])


# --- what a pass has to move and compute --------------------------------------

def work(case):
    op, inf = case["op"], case["inf"]
    T = -(-inf // BLOCK)
    if op == "encode_f8":
        n = case["out"] * inf
        return dict(bytes=5 * n + 4 * T * -(-case["out"] // BLOCK), flops=3 * n)
    if op in ("quantize_f8", "checkpoint"):
        n = case["tokens"] * inf
        return dict(bytes=3 * n + (4 if op == "quantize_f8" else 2) * T * case["tokens"], flops=3 * n)
    out = case["out"]
    if op in ("gemv_f8", "gemm_f8"):
        M = case.get("tokens", 1)
        x = 2 * inf if op == "gemv_f8" else M * inf + 4 * M * T
        y = M * out * (4 if case.get("wide") else 2)
        return dict(bytes=out * inf + 4 * T * -(-out // BLOCK) + x + y, flops=2 * M * out * inf)
    M, K = case["tokens"], case["planes"]
    G = inf // case["group"] if case["group"] else 1
    read = M * inf + 2 * M * T + 2 * M * out + K * out * inf // 8 + 2 * K * out * G
    write = 4 * out * inf + 4 * M * inf + 4 * K * out * G
    return dict(bytes=read + write, flops=4 * M * out * inf + 3 * K * out * inf)


# --- the definitions in 64 bits -----------------------------------------------

def _blocks(n):
    return [slice(i, min(n, i + BLOCK)) for i in range(0, n, BLOCK)]


def _e4m3(v):
    """Nearest e4m3 value of float64 v (|v| <= 448), ties to even: four significant bits, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _f8_of(b):
    """(values, scale) of one block in float64; the scale and its reciprocal are 32-bit values by definition."""
    top = max(float(b.abs().max()), TINY)
    inv, s = torch.tensor([F8_MAX / top, top / F8_MAX], dtype=torch.float64).float().double().tolist()
    return _e4m3((b * inv).float().double()), s


def _f8_rows(x):
    """Per-token blocks of float64 x: (values, scales [T][M])."""
    codes, scales = torch.empty_like(x), []
    for t in _blocks(x.shape[1]):
        top = x[:, t].abs().max(1).values.clamp_min(TINY)
        inv = (F8_MAX / top).float().double()
        codes[:, t] = _e4m3((x[:, t] * inv[:, None]).float().double())
        scales.append((top / F8_MAX).float().double())
    return codes, torch.stack(scales)


def _sum_f8(w, ws, x, xs):
    y = x.new_zeros((x.shape[0], w.shape[0]))
    over = torch.arange(w.shape[0], device=w.device) // BLOCK
    for i, t in enumerate(_blocks(w.shape[1])):
        y += xs[i][:, None] * ws[over, i] * (x[:, t] @ w[:, t].t().contiguous())
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "encode_f8":
        w = s["w"].double()
        codes, scales = torch.empty_like(w), []
        for rows in _blocks(w.shape[0]):
            pairs = [_f8_of(w[rows, t]) for t in _blocks(w.shape[1])]
            codes[rows] = torch.cat([c for c, _ in pairs], 1)
            scales.append([v for _, v in pairs])
        return codes, torch.tensor(scales, dtype=torch.float64)
    if op == "quantize_f8":
        return _f8_rows(s["x"].double())
    if op == "gemv_f8":
        x, xs = _f8_rows(s["x"].double().view(1, -1))
        return _sum_f8(s["w8"].double(), s["ws"].double(), x, xs)[0]
    if op == "gemm_f8":
        return _sum_f8(s["w8"].double(), s["ws"].double(), s["x8"].double(), s["xs"].double())
    if op == "checkpoint":
        x = s["x"].double()
        codes, scales = torch.empty_like(x), []
        for t in _blocks(x.shape[1]):
            want = x[:, t].abs().max(1).values / 127
            # eleven significant bits, steps of 2^-24 below 2^-14, rounded up
            step = torch.exp2(torch.floor(torch.log2(want.clamp_min(2.0 ** -14))) - 10)
            v = (torch.ceil(want / step) * step).clamp(F16_TINY, CKPT_TOP)
            codes[:, t] = torch.round(x[:, t] / v[:, None]).clamp(-127, 127)
            scales.append(v)
        return codes.to(torch.int64), torch.stack(scales, 1)
    inf, out, K = case["inf"], case["out"], case["planes"]
    x = s["codes"].double()
    for i, t in enumerate(_blocks(inf)):
        x[:, t] *= s["cs"][:, i:i + 1].double()
    x = x.half().double()                              # a checkpoint stands for fp16 values
    d = s["dy"].double()
    dw = d.t().contiguous() @ x
    G = inf // case["group"] if case["group"] else 1
    word = s["planes"].to(torch.int64) & 0xFFFFFFFF
    what, ds = torch.zeros_like(dw), []
    for k in range(K):
        b = torch.empty_like(dw)
        for bit in range(32):
            b[:, bit::32] = ((word[k] >> bit) & 1).double() * 2 - 1
        what += (b.view(out, G, -1) * s["scales"][k].double()[:, :, None]).view(out, inf)
        ds.append((b * dw).view(out, G, -1).sum(-1))
    return d @ what, dw, torch.stack(ds)
