"""Measured cases of the operators at the two ends of a binarized model's
output: linears held in 4 bits with group scales (encode_q4, gemm_q4,
gemv_q4), log probabilities of given tokens with entropy and top alternatives
and their gradient (token_logprobs, token_logprobs_backward), and distillation
from a teacher's top log probabilities with its gradient (distill_forward,
distill_backward).

`own` False computes every case in elementary torch operations in 32 bits;
True makes the calls a user makes of the package.  Sizes are the linears of
workloads.py and vocabularies of 32 to 128 thousand tokens, and ragged ones
around them.
"""
import math

import torch

own = False

GROUP = 128
F16_TINY, F16_MAX = 2.0 ** -24, 65504.0
LARGEST = 2048 * 128256                       # logits of the largest case
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# --- cases --------------------------------------------------------------------

def listed():
    return [
        # a down projection put into 4 bits with zero points when a model is loaded
        dict(name="encode_q4 4096x11008 zeros", op="encode_q4", out=4096, inf=11008, zeros=True),
        # a small ragged layer, symmetric, a short last group
        dict(name="encode_q4 1003x4128", op="encode_q4", out=1003, inf=4128, zeros=False),
        # one decoded token through an up projection: the weight read is all that counts
        dict(name="gemv_q4 11008x4096", op="gemv_q4", out=11008, inf=4096, zeros=False, wide=False),
        # a decode batch of 16 through a down projection, zero points
        dict(name="gemm_q4 16 4096x11008 zeros", op="gemm_q4", tokens=16, out=4096, inf=11008, zeros=True, wide=False),
        # a frozen teacher's gate projection on a batch of 2048 tokens
        dict(name="gemm_q4 2048 14336x4096", op="gemm_q4", tokens=2048, out=14336, inf=4096, zeros=False, wide=False),
        # one decoded token with its alternatives: latency
        dict(name="logprobs 1x32000 top20", op="logprobs", rows=1, vocab=32000, type="f16", top=20, temp=1.0),
        # a teacher's pass over a training batch: the alternatives that distillation takes
        dict(name="logprobs 2048x128256 top64", op="logprobs", rows=2048, vocab=128256, type="f16", top=64, temp=1.0),
        # the task loss of a training batch
        dict(name="logprobs step 2048x32000", op="logprobs_step", rows=2048, vocab=32000, type="f16", temp=1.0, entropy=False),
        # a ragged batch, an odd vocabulary (rows start anywhere), a bonus on the entropy
        dict(name="logprobs step 333x50257 bf16", op="logprobs_step", rows=333, vocab=50257, type="bf16", temp=0.7, entropy=True),
        # distillation measured on a short validation batch
        dict(name="distill 64x128256 f32 tail", op="distill", rows=64, vocab=128256, type="f32", slots=64, temp=1.0, tail=True),
        # distillation in training: loss and gradient of the student's logits
        dict(name="distill step 2048x128256 tail", op="distill_step", rows=2048, vocab=128256, type="f16", slots=64, temp=1.0, tail=True),
        # a short ragged batch, the teacher's top 20 taken as all of its mass, a temperature
        dict(name="distill step 77x32001 bf16", op="distill_step", rows=77, vocab=32001, type="bf16", slots=20, temp=2.0, tail=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["encode_q4", "gemv_q4", "gemm_q4", "gemm_q4", "logprobs", "logprobs", "logprobs_step", "distill",
                     "distill_step", "distill_step"])
    if op in ("encode_q4", "gemv_q4", "gemm_q4"):
        case = dict(op=op, out=_log(rng, 500, 14336), inf=32 * _log(rng, 16, 448), zeros=rng.random() < 0.5)
        if op == "encode_q4":
            case["inf"] = min(case["inf"], 11008)
            return case
        case["wide"] = rng.random() < 0.3
        if op == "gemm_q4":
            tokens = _log(rng, 2, 2048)
            while tokens * case["out"] * case["inf"] > 2048 * 14336 * 4096:
                tokens //= 2
            case["tokens"] = tokens
        return case
    kind = rng.choice(["f16", "f16", "bf16", "f32"])
    vocab = _log(rng, 1000, 131072)
    rows = _log(rng, 1, 4096)
    while rows * vocab * (2 if kind == "f32" else 1) > LARGEST:
        rows //= 2
    case = dict(op=op, rows=rows, vocab=vocab, type=kind, temp=rng.choice([1.0, 1.0, 0.7, 2.0]))
    if op == "logprobs":
        return dict(case, top=_log(rng, 1, 128))
    if op == "logprobs_step":
        return dict(case, entropy=rng.random() < 0.5)
    return dict(case, slots=_log(rng, 1, 128), tail=rng.random() < 0.5)


# --- inputs -------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *size):
    return torch.randn(size, generator=g, device="cuda", dtype=torch.float32)


def _weight(g, out, inf):
    w = _normal(g, out, inf) * 0.02
    pos = torch.randint(0, out * inf, (max(1, out * inf // 1000),), generator=g, device="cuda")
    w.view(-1)[pos] *= 10.0
    return w


def _activations(g, tokens, inf):
    """fp16 activations: unit normal, a few channels 20 times as large."""
    x = _normal(g, tokens, inf)
    x[:, torch.randint(0, inf, (max(1, inf // 500),), generator=g, device="cuda")] *= 20.0
    return x.half()


def _logits(g, rows, vocab, kind):
    """Logits as a model gives them: normal, a few dozen likely tokens a row, the last columns (a padded vocabulary) masked."""
    x = _normal(g, rows, vocab) * 2.0
    start = torch.randint(0, vocab, (rows, 1), generator=g, device="cuda")
    hot = (start + torch.arange(48, device="cuda") * (vocab // 48)) % vocab
    x.scatter_(1, hot, _normal(g, rows, 48) * 3.0 + 8.0)
    if vocab >= 2000:
        x[:, vocab - vocab // 500:] = float("-inf")
    return x.to(TYPES[kind])


def _targets(g, x):
    """A token of each row, mostly a likely one; every 17th row has none (padding)."""
    rows, vocab = x.shape
    best = x[:, :vocab - vocab // 500].argmax(1)
    any_ = torch.randint(0, vocab - vocab // 500, (rows,), generator=g, device="cuda")
    t = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.5, best, any_)
    t[16::17] = -1
    return t


def _row_weights(g, rows, scale=256.0):
    """Gradients of the rows' losses: a mean with a loss scale, none for every 17th row (padding)."""
    w = torch.full((rows,), scale / rows, device="cuda")
    w[16::17] = 0.0
    return w


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "encode_q4":
        return dict(case=case, w=_weight(g, case["out"], case["inf"]))
    if op in ("gemv_q4", "gemm_q4"):
        codes, scales, zeros = _encode_q4(_weight(g, case["out"], case["inf"]), case["zeros"])
        x = _activations(g, case.get("tokens", 1), case["inf"])
        return dict(case=case, codes=codes, scales=scales, zeros=zeros, x=x if op == "gemm_q4" else x[0].contiguous(),
                    dtype=torch.float32 if case["wide"] else torch.float16)
    x = _logits(g, case["rows"], case["vocab"], case["type"])
    if op == "logprobs":
        return dict(case=case, x=x, targets=_targets(g, x))
    if op == "logprobs_step":
        a = -_row_weights(g, case["rows"])          # the loss is the mean of -logp
        return dict(case=case, x=x, targets=_targets(g, x), a=a, b=-0.01 * a if case["entropy"] else None)
    near = x.float() + 0.5 * _normal(g, *x.shape)   # a teacher that mostly agrees
    lp, idx = torch.topk(near, case["slots"], 1)
    lp = lp / case["temp"] - torch.logsumexp(near / case["temp"], 1, keepdim=True)
    idx = idx.int()
    if case["slots"] > 4:                           # a shorter list in some rows
        lp[3::7, -2:] = float("-inf")
        idx[3::7, -2:] = -1
    return dict(case=case, x=x, idx=idx, lp=lp, d=_row_weights(g, case["rows"]) * case["temp"] ** 2)


# --- the plain forms ----------------------------------------------------------

def _quotient(a, b):
    """Correctly rounded 32-bit quotients: codes next to a border go by the last bit."""
    return (a.double() / b.double()).float()


def _encode_q4(w, with_zeros):
    out, inf = w.shape
    n = -inf % GROUP
    p = torch.cat([w, w.new_zeros((out, n))], 1) if n else w
    b = p.view(out, -1, GROUP)
    if with_zeros:
        lo, hi = b.amin(2).clamp_max(0.0), b.amax(2).clamp_min(0.0)
        scales = _quotient(hi - lo, torch.full_like(hi, 15.0)).clamp(F16_TINY, F16_MAX).half()
        z = torch.round(_quotient(-lo, scales)).clamp(0, 15)
    else:
        top = b.abs().amax(2)
        scales = _quotient(top, torch.full_like(top, 7.0)).clamp(F16_TINY, F16_MAX).half()
        z = torch.full_like(top, 8.0)
    c = (torch.round(_quotient(b, scales[:, :, None])) + z[:, :, None]).clamp(0, 15).to(torch.uint8)
    c = c.view(out, -1)[:, :inf]
    return c[:, 0::2] | (c[:, 1::2] << 4), scales, z.to(torch.uint8) if with_zeros else None


def _values_q4(codes, scales, zeros):
    out, half = codes.shape
    c = torch.stack([codes & 15, codes >> 4], 2).view(out, 2 * half).float()
    z = torch.full_like(scales, 8.0) if zeros is None else zeros
    over = lambda v: v.float().repeat_interleave(GROUP, 1)[:, :2 * half]
    return (c - over(z)) * over(scales)


def _log_softmax(x, temp):
    z = x.float() / temp
    top = z.amax(1, keepdim=True)
    z = z - top
    return z - torch.log(torch.exp(z).sum(1, keepdim=True))


def _entropy(lp):
    return -torch.where(lp > float("-inf"), torch.exp(lp) * lp, 0.0).sum(1)


def _of_targets(lp, targets):
    got = lp.gather(1, targets.clamp_min(0)[:, None])[:, 0]
    return torch.where(targets >= 0, got, 0.0)


def _ordered(x):
    """Whole numbers in the order of the values, ties by the lowest index: all different."""
    bits = (x.float() + 0.0).view(torch.int32).to(torch.int64)
    bits = torch.where(bits < 0, -2 ** 31 - bits, bits)
    return (bits << 32) + (x.shape[1] - torch.arange(x.shape[1], device=x.device))


def _logprobs(s):
    c, x = s["case"], s["x"]
    lp = _log_softmax(x, c["temp"])
    key = torch.topk(_ordered(x), c["top"], 1).values
    idx = x.shape[1] - (key & 0xFFFFFFFF)
    return _of_targets(lp, s["targets"]), _entropy(lp), lp.gather(1, idx), idx.int()


def _logprobs_step(s):
    c, t = s["case"], s["targets"]
    lp = _log_softmax(s["x"], c["temp"])
    p = torch.exp(lp)
    a = torch.where(t >= 0, s["a"], 0.0)[:, None]
    H = _entropy(lp)
    grad = -a * p
    grad.scatter_add_(1, t.clamp_min(0)[:, None], a)
    if s["b"] is not None:
        grad = grad - s["b"][:, None] * torch.where(p > 0, p * (lp + H[:, None]), 0.0)
    return _of_targets(lp, t), H, (grad / c["temp"]).to(s["x"].dtype)


def _xlogx(p, logq):
    """p (log p - log q), 0 where p is."""
    return torch.where(p > 0, p * (torch.log(p) - logq), 0.0)


def _distill(s, step):
    c, x = s["case"], s["x"]
    lq = _log_softmax(x, c["temp"])
    at = s["idx"].clamp_min(0).long()
    used = (s["idx"] >= 0) & (s["lp"] > float("-inf"))
    t = torch.where(used, s["lp"], float("-inf"))
    p = torch.exp(t) if c["tail"] else torch.exp(t - t.amax(1, keepdim=True))
    if not c["tail"]:
        p = p / p.sum(1, keepdim=True)
    logq = lq.gather(1, at)
    loss = _xlogx(p, logq).sum(1)
    total = p.sum(1, keepdim=True)
    q = torch.exp(lq)
    if c["tail"]:
        rest = (1.0 - total).clamp_min(0.0)
        named = torch.zeros_like(q).scatter_add_(1, at, used.float())
        q_rest = torch.where(named > 0, 0.0, q).sum(1, keepdim=True)
        loss = loss + _xlogx(rest, torch.log(q_rest))[:, 0]
    if not step:
        return loss
    grad = q * (total + rest - torch.where(named > 0, 0.0, rest / q_rest)) if c["tail"] else q * total
    grad.scatter_add_(1, at, -p)
    return loss, (grad * (s["d"][:, None] / c["temp"])).to(x.dtype)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import gemm_rbq_encode_amd as rbq
        if op == "encode_q4":
            codes, scales, zeros = rbq.encode_q4(s["w"], zeros=c["zeros"])
            return (codes, scales, zeros) if c["zeros"] else (codes, scales)
        if op == "gemv_q4":
            return rbq.gemv_q4(s["codes"], s["scales"], s["x"], s["zeros"], dtype=s["dtype"])
        if op == "gemm_q4":
            return rbq.gemm_q4(s["codes"], s["scales"], s["x"], s["zeros"], dtype=s["dtype"])
        if op == "logprobs":
            return rbq.token_logprobs(s["x"], s["targets"], top=c["top"], temperature=c["temp"])
        if op == "logprobs_step":
            grad, logp, H = rbq.token_logprobs_backward(s["x"], s["targets"], s["a"], s["b"], temperature=c["temp"])
            return logp, H, grad
        if op == "distill":
            return rbq.distill_forward(s["x"], s["idx"], s["lp"], temperature=c["temp"], tail=c["tail"])
        grad, loss = rbq.distill_backward(s["x"], s["idx"], s["lp"], s["d"], temperature=c["temp"], tail=c["tail"])
        return loss, grad
    if op == "encode_q4":
        codes, scales, zeros = _encode_q4(s["w"], c["zeros"])
        return (codes, scales, zeros) if c["zeros"] else (codes, scales)
    if op in ("gemv_q4", "gemm_q4"):
        w = _values_q4(s["codes"], s["scales"], s["zeros"])
        y = (s["x"].float().view(-1, c["inf"]) @ w.t()).to(s["dtype"])
        return y if op == "gemm_q4" else y[0]
    if op == "logprobs":
        return _logprobs(s)
    if op == "logprobs_step":
        return _logprobs_step(s)
    return _distill(s, op == "distill_step")


# --- what a pass has to move and compute --------------------------------------

def work(case):
    op = case["op"]
    if op in ("encode_q4", "gemv_q4", "gemm_q4"):
        out, inf = case["out"], case["inf"]
        held = out * inf // 2 + out * -(-inf // GROUP) * (3 if case["zeros"] else 2)
        if op == "encode_q4":
            return dict(bytes=4 * out * inf + held, flops=4 * out * inf)
        M = case.get("tokens", 1)
        return dict(bytes=held + 2 * M * inf + M * out * (4 if case["wide"] else 2), flops=2 * M * out * inf)
    M, V = case["rows"], case["vocab"]
    n = M * V * (4 if case["type"] == "f32" else 2)
    if op == "logprobs":
        return dict(bytes=n + M * (16 + 8 * case["top"]), flops=6 * M * V)
    if op == "logprobs_step":
        return dict(bytes=2 * n + 24 * M, flops=10 * M * V)
    if op == "distill":
        return dict(bytes=n + M * (4 + 8 * case["slots"]), flops=5 * M * V)
    return dict(bytes=2 * n + M * (8 + 8 * case["slots"]), flops=8 * M * V)


# --- the definitions in 64 bits -----------------------------------------------

def _f32(v):
    return v.to(torch.float32).double()


def _f16(v):
    """Nearest binary16 of float64 v >= 0 (in range): eleven significant bits, steps of 2^-24 below 2^-14, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.clamp_min(2.0 ** -14))) - 10)
    return torch.round(v / step) * step


def _exact_q4(w, zeros):
    codes, scales, points = [], [], []
    for i in range(0, w.shape[1], GROUP):
        b = w[:, i:i + GROUP].double()
        if zeros:
            lo, hi = b.min(1).values.clamp(max=0), b.max(1).values.clamp(min=0)
            s = _f16(_f32(_f32(hi - lo) / 15).clamp(F16_TINY, F16_MAX))
            z = torch.round(_f32(-lo / s)).clamp(0, 15)
        else:
            s = _f16(_f32(b.abs().max(1).values / 7).clamp(F16_TINY, F16_MAX))
            z = torch.full_like(s, 8)
        codes.append((torch.round(_f32(b / s[:, None])) + z[:, None]).clamp(0, 15))
        scales.append(s)
        points.append(z)
    c = torch.cat(codes, 1).long()
    packed = c[:, ::2] + 16 * c[:, 1::2]
    return (packed, torch.stack(scales, 1)) + ((torch.stack(points, 1).long(),) if zeros else ())


def _rows(n, at_once=128):
    return [slice(i, min(n, i + at_once)) for i in range(0, n, at_once)]


def _log_p(x, temp):
    z = x.double() / temp
    return z - torch.logsumexp(z, 1, keepdim=True)


def _exact_rows(s, r):
    """One block of rows of a case on logits."""
    c, x = s["case"], s["x"][r]
    op, temp = c["op"], c["temp"]
    lp = _log_p(x, temp)
    p = lp.exp()
    row = torch.arange(lp.shape[0], device=lp.device)
    if op in ("logprobs", "logprobs_step"):
        t = s["targets"][r]
        has = t >= 0
        logp = torch.zeros_like(lp[:, 0])
        logp[has] = lp[row[has], t[has]]
        H = -(p * lp.nan_to_num(neginf=0.0)).sum(1)
        if op == "logprobs":
            order = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :c["top"]]
            return logp, H, lp[row[:, None], order], order
        hot = torch.zeros_like(p)
        hot[row[has], t[has]] = 1.0
        grad = s["a"][r].double()[:, None] * (hot - p) * has[:, None]
        if s["b"] is not None:
            grad -= s["b"][r].double()[:, None] * p * (lp.nan_to_num(neginf=0.0) + H[:, None])
        return logp, H, grad / temp
    idx, t = s["idx"][r].long(), s["lp"][r].double()
    m, k = (idx >= 0).nonzero(as_tuple=True)
    given = torch.zeros_like(t)
    given[m, k] = t[m, k].exp()
    if not c["tail"]:
        given = given / given.sum(1, keepdim=True)
    want, named = torch.zeros_like(p), torch.zeros_like(p, dtype=torch.bool)
    want[m, idx[m, k]] = given[m, k]                  # a row names no token twice
    named[m, idx[m, k]] = True
    rest = (1 - given.sum(1)).clamp(min=0) if c["tail"] else torch.zeros_like(given[:, 0])
    loss = torch.where(want > 0, want * (want.log() - lp), 0.0).sum(1)
    away = torch.where(named, 0.0, p)
    if c["tail"]:
        q = away.sum(1)
        loss += torch.where(rest > 0, rest * (rest.log() - q.log()), 0.0)
        away = away / q[:, None]
    if op == "distill":
        return (loss,)
    # the student's mass against the teacher's: named tokens one by one, the others by their share of the rest
    mass = (given.sum(1) + rest)[:, None]
    grad = mass * p - want - rest[:, None] * away
    return loss, grad * s["d"][r].double()[:, None] / temp


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "encode_q4":
        return _exact_q4(s["w"], case["zeros"])
    if op in ("gemv_q4", "gemm_q4"):
        x = s["x"].double().view(-1, case["inf"])
        y = x.new_zeros((x.shape[0], case["out"]))
        c = torch.empty((case["out"], case["inf"]), dtype=torch.float64, device=x.device)
        c[:, ::2], c[:, 1::2] = (s["codes"] % 16).double(), (s["codes"] // 16).double()
        for t, i in enumerate(range(0, case["inf"], GROUP)):
            z = 8.0 if s["zeros"] is None else s["zeros"][:, t:t + 1].double()
            y += (x[:, i:i + GROUP] @ (c[:, i:i + GROUP] - z).t().contiguous()) * s["scales"][:, t].double()
        return y if op == "gemm_q4" else y[0]
    parts = [_exact_rows(s, r) for r in _rows(case["rows"])]
    out = tuple(torch.cat(v) for v in zip(*parts))
    return out[0] if op == "distill" else out
