"""Cases for timing and checking the operators around the FP8 linear layers.

The operators: layer norm forward and backward, the AdamW step over many
tensors at once (moments in E4M3 or fp32), the per-row int8 quantizer, and
the int8 matrix product with a scale per token and per output channel.

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, with ``own = True``, through this
library's entry points.  ``exact`` is the operators' definition in 64 bits.
"""
import math

import torch
import torch.nn.functional as F

own = False

DEV = "cuda:0"
TILE = 128                      # elements that share one scale of an E4M3 moment
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
FIRST_STEP = 10                 # steps taken before the case's first pass


def listed():
    return [
        # the norm in front of a linear layer while one token is generated: pure latency
        dict(name="norm forward, one token", op="norm_fwd", rows=1, cols=4096, dtype="bf16", wdtype="f32"),
        # the same over a long prompt, the long-K activation shape
        dict(name="norm forward, long prompt", op="norm_fwd", rows=16384, cols=8192, dtype="bf16", wdtype="f32"),
        # training on 4096 tokens with a hidden size of 4096, fp32 master weights
        dict(name="norm backward, training", op="norm_bwd", rows=4096, cols=4096, dtype="bf16", wdtype="f32"),
        # odd sizes in fp32: no row but the first starts on a 16-byte boundary
        dict(name="norm backward, odd fp32", op="norm_bwd", rows=1000, cols=2047, dtype="f32", wdtype="f32"),
        # the weights and the norms of one MLP (4096 <-> 14336), 8-bit moments, bf16 gradients
        dict(name="AdamW E4M3, one MLP", op="adamw", kind="e4m3", gdtype="bf16", count=8, large=14336 * 4096,
             small=4096, larges=2, salt=1),
        # the vectors of a network (biases, norms, odd leftovers), fp32 moments: latency and launches
        dict(name="AdamW fp32, many vectors", op="adamw", kind="f32", gdtype="f32", count=56, large=40000, small=1,
             larges=3, salt=2),
        # activations of a small batch of tokens in generation
        dict(name="int8 rows, 16 tokens", op="quant", rows=16, cols=4096, dtype="bf16"),
        # activations of a long prompt (or, once, a weight)
        dict(name="int8 rows, long prompt", op="quant", rows=16384, cols=8192, dtype="bf16"),
        # MLP up-projection of a single token: the weight is read once
        dict(name="int8 product, one token", op="gemm", M=1, N=14336, K=4096, bias=False, dtype="bf16"),
        # MLP down-projection of a batch of requests
        dict(name="int8 product, 96 tokens", op="gemm", M=96, N=4096, K=14336, bias=False, dtype="bf16"),
        # nothing a multiple of anything, with a bias, fp32 out
        dict(name="int8 product, odd sizes", op="gemm", M=333, N=1001, K=2049, bias=True, dtype="f32"),
        # MLP up-projection of a prompt
        dict(name="int8 product, prompt", op="gemm", M=4096, N=14336, K=4096, bias=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step):
    """A size spread over the logarithm; two in three times a multiple of `step`.  (3072 is left out: no
    configuration of this library has it.)"""
    while True:
        n = _log(rng, lo, hi)
        n = n if rng.random() < 1 / 3 else max(lo, min(hi, -(-n // step) * step))
        if n != 3072:
            return n


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "adamw", "quant", "gemm"])
    if op == "adamw":
        count = _log(rng, 2, 56)
        large = _log(rng, 3000, 14336 * 4096)
        return dict(op=op, kind=rng.choice(["e4m3", "f32"]), gdtype=rng.choice(["bf16", "f32"]), count=count,
                    large=large, small=_log(rng, 1, 3000), larges=min(count, 1 if large > 1 << 25 else 2),
                    salt=rng.randrange(1 << 20))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "gemm":
        while True:
            M, N, K = _size(rng, 1, 4096, 16), _size(rng, 16, 14336, 128), _size(rng, 16, 14336, 128)
            if M * N * K <= 4096 * 14336 * 4096:
                return dict(op=op, M=M, N=N, K=K, bias=rng.random() < 0.5, dtype=dtype)
    while True:
        rows, cols = _size(rng, 1, 16384, 16), _size(rng, 16, 16384, 128)
        if rows * cols <= 16384 * 8192:
            break
    case = dict(op=op, rows=rows, cols=cols, dtype=dtype)
    return case if op == "quant" else dict(case, wdtype=rng.choice(["f32", "f32", "bf16"]))


def _sizes(case):
    """The tensors of an AdamW case: `larges` of the large size, the others between the small one and a
    twentieth of the large one."""
    import random
    rng = random.Random(case["salt"])
    top = max(case["small"], min(case["large"] // 20, 100000))
    rest = [_log(rng, case["small"], top) for _ in range(case["count"] - case["larges"])]
    return [case["large"]] * case["larges"] + rest


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _activations(gen, rows, cols, dtype):
    """Values of a residual stream: rows of different size and mean, one column in 512 far larger."""
    x = torch.randn(rows, cols, device=DEV, generator=gen)
    x *= torch.exp(0.5 * torch.randn(rows, 1, device=DEV, generator=gen))
    x += 0.25 + 0.1 * torch.randn(rows, 1, device=DEV, generator=gen)
    x *= 1 + 19 * (torch.rand(cols, device=DEV, generator=gen) < 1 / 512)
    return x.to(dtype)


def _codes(x):
    """int8 codes and row scales of x, rows padded to 16 bytes as the quantizer allocates them."""
    rows, cols = x.shape
    s = x.abs().amax(1) / 127
    q = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.int8, device=DEV)[:, :cols]
    q.copy_(torch.round(x / s[:, None]))
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    state = dict(case=case)
    if op in ("norm_fwd", "norm_bwd"):
        rows, cols, wt = case["rows"], case["cols"], TYPES[case["wdtype"]]
        x = state["x"] = _activations(gen, rows, cols, TYPES[case["dtype"]])
        state["w"] = (1 + 0.2 * torch.randn(cols, device=DEV, generator=gen)).to(wt)
        state["b"] = (0.1 * torch.randn(cols, device=DEV, generator=gen)).to(wt)
        if op == "norm_bwd":
            state["dy"] = (1e-2 * torch.randn(rows, cols, device=DEV, generator=gen)).to(x.dtype)
            x = x.double()
            mean = x.mean(1)
            state["mean"] = mean.float()
            state["rstd"] = torch.rsqrt((x - mean[:, None]).square().mean(1) + EPS).float()
    elif op == "quant":
        state["x"] = _activations(gen, case["rows"], case["cols"], TYPES[case["dtype"]])
        state["top"] = torch.full((), 127.0, device=DEV)
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        state["a"], state["sa"] = _codes(_activations(gen, M, K, torch.float32))
        state["b"], state["sb"] = _codes(0.02 * torch.randn(N, K, device=DEV, generator=gen))
        state["bias"] = torch.randn(N, device=DEV, generator=gen) if case["bias"] else None
    else:
        sizes = _sizes(case)
        blocks = sum(-(-n // TILE) for n in sizes)
        state["sizes"], state["step"] = sizes, FIRST_STEP
        state["p"] = [0.02 * torch.randn(n, device=DEV, generator=gen) for n in sizes]
        state["g"] = [(1e-3 * torch.randn(n, device=DEV, generator=gen)).to(TYPES[case["gdtype"]]) for n in sizes]
        state["top"] = torch.full((), 448.0, device=DEV)
        # the moments of all tensors in one buffer, each tensor's on a boundary of 128
        live = _flat([torch.ones(n, device=DEV) for n in sizes])
        m = 5e-4 * torch.randn(blocks * TILE, device=DEV, generator=gen) * live
        v = 1e-6 * (0.1 + torch.randn(blocks * TILE, device=DEV, generator=gen).square()) * live
        if case["kind"] == "e4m3":
            state["moments"] = (*_to_e4m3(m, state["top"]), *_to_e4m3(v, state["top"]))
        else:
            state["moments"] = (m, v)
        if own:
            import fp8_precision_quant_amd as fq
            state["plan"] = fq.fp8q_adamw_plan(
                state["p"], fq.STATE_E4M3 if case["kind"] == "e4m3" else fq.STATE_F32, state["moments"])
    return state


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _flat(tensors):
    """All tensors' values in fp32, one behind the other, each padded to a multiple of 128."""
    return torch.cat([F.pad(t.reshape(-1).float(), (0, -t.numel() % TILE)) for t in tensors])


def _from_e4m3(codes, scales):
    return (codes.view(torch.float8_e4m3fn).float().view(-1, TILE) * scales[:, None]).view(-1)


def _to_e4m3(x, top):
    """E4M3 codes and one scale per 128 values: s = amax / 448, code = E4M3(x / s)."""
    x = x.view(-1, TILE)
    s = x.abs().amax(1) / top
    q = torch.where(s[:, None] > 0, x / s[:, None], torch.zeros_like(x))
    return q.to(torch.float8_e4m3fn).view(torch.uint8).view(-1), s


def _plain_norm_fwd(state):
    x = state["x"].float()
    mean = x.mean(1, keepdim=True)
    centred = x - mean
    rstd = torch.rsqrt((centred * centred).mean(1, keepdim=True) + EPS)
    y = centred * rstd * state["w"].float() + state["b"].float()
    return dict(y=y.to(state["x"].dtype), mean=mean[:, 0], rstd=rstd[:, 0])


def _plain_norm_bwd(state):
    x, dy, w = state["x"].float(), state["dy"].float(), state["w"].float()
    xhat = (x - state["mean"][:, None]) * state["rstd"][:, None]
    wdy = dy * w
    dx = (wdy - wdy.mean(1, keepdim=True) - xhat * (wdy * xhat).mean(1, keepdim=True)) * state["rstd"][:, None]
    return dict(dx=dx.to(state["x"].dtype), dw=(dy * xhat).sum(0).to(state["w"].dtype),
                db=dy.sum(0).to(state["w"].dtype))


def _plain_quant(state):
    x = state["x"].float()
    s = x.abs().amax(1) / state["top"]
    q = torch.where(s[:, None] > 0, torch.round(x / s[:, None]), torch.zeros_like(x))
    return dict(q=q.to(torch.int8), s=s)


def _plain_gemm(state):
    c = torch.matmul(state["a"].float(), state["b"].float().t())
    c = c * state["sa"][:, None] * state["sb"]
    if state["bias"] is not None:
        c = c + state["bias"]
    return c.to(TYPES[state["case"]["dtype"]])


def _plain_adamw(state):
    h, t = HYPER, state["step"]
    e4m3 = state["case"]["kind"] == "e4m3"
    p, g, moments = _flat(state["p"]), _flat(state["g"]), state["moments"]
    m, v = (_from_e4m3(*moments[:2]), _from_e4m3(*moments[2:])) if e4m3 else moments
    p = p * (1 - h["lr"] * h["weight_decay"])
    m = m * h["beta1"] + g * (1 - h["beta1"])
    v = v * h["beta2"] + g * (1 - h["beta2"]) * g
    step_size, correction = h["lr"] / (1 - h["beta1"] ** t), math.sqrt(1 - h["beta2"] ** t)
    p = p - m / (v.sqrt() / correction + h["eps"]) * step_size
    parts = p.split([-(-n // TILE) * TILE for n in state["sizes"]])
    torch._foreach_copy_(state["p"], [q[:n] for q, n in zip(parts, state["sizes"])])
    new = (*_to_e4m3(m, state["top"]), *_to_e4m3(v, state["top"])) if e4m3 else (m, v)
    torch._foreach_copy_(list(moments), list(new))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _moments_out(state):
    """The moments as the values they are: E4M3 numbers and their scales, or fp32."""
    if state["case"]["kind"] == "f32":
        m, v = state["moments"]
        return dict(m=m, v=v)
    mq, ms, vq, vs = state["moments"]
    return dict(m=mq.view(torch.float8_e4m3fn), ms=ms, v=vq.view(torch.float8_e4m3fn), vs=vs)


def run(state):
    op = state["case"]["op"]
    if op == "adamw":
        state["step"] += 1
    if not own:
        if op == "adamw":
            _plain_adamw(state)
            return dict(p=state["p"], **_moments_out(state))
        return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "quant": _plain_quant,
                "gemm": _plain_gemm}[op](state)
    import fp8_precision_quant_amd as fq
    if op == "norm_fwd":
        y, mean, rstd = fq.fp8q_layer_norm_forward(state["x"], state["w"], state["b"], eps=EPS)
        return dict(y=y, mean=mean, rstd=rstd)
    if op == "norm_bwd":
        dx, dw, db = fq.fp8q_layer_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], state["w"])
        return dict(dx=dx, dw=dw, db=db)
    if op == "quant":
        q, s = fq.fp8q_int8_quant_rows(state["x"])
        return dict(q=q, s=s)
    if op == "gemm":
        return fq.fp8q_int8_gemm(state["a"], state["sa"], state["b"], state["sb"], bias=state["bias"],
                                 out_dtype=TYPES[state["case"]["dtype"]])
    fq.fp8q_adamw_multi_step(state["plan"], state["g"], step=state["step"], **HYPER)
    return dict(p=state["p"], **_moments_out(state))


def work(case):
    op = case["op"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        out = M * N * SIZE[case["dtype"]]
        return dict(bytes=M * K + N * K + 4 * (M + N) + 4 * N * case["bias"] + out, flops=2 * M * N * K)
    if op == "adamw":
        n = sum(_sizes(case))
        blocks = sum(-(-k // TILE) for k in _sizes(case))
        moments = 4 * n + 16 * blocks if case["kind"] == "e4m3" else 16 * n
        return dict(bytes=8 * n + SIZE[case["gdtype"]] * n + moments, flops=16 * n)
    n, e = case["rows"] * case["cols"], SIZE[case["dtype"]]
    if op == "quant":
        return dict(bytes=n * (e + 1) + 4 * case["rows"], flops=3 * n)
    vectors = case["cols"] * SIZE[case["wdtype"]]
    if op == "norm_fwd":
        return dict(bytes=2 * n * e + 2 * vectors + 8 * case["rows"], flops=7 * n)
    return dict(bytes=3 * n * e + 3 * vectors + 8 * case["rows"], flops=13 * n)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_e4m3(x):
    """(E4M3 value of x / s, s) with s = amax / 448 per 128 values: three fraction bits, the smallest
    normal exponent -6, ties to even."""
    x = x.reshape(-1, TILE)
    s = x.abs().max(dim=1).values / 448
    q = x / s.masked_fill(s == 0, 1)[:, None]
    exponent = torch.frexp(q).exponent.double() - 1
    ulp = torch.exp2(exponent.clamp(min=-6) - 3)
    return (torch.round(q / ulp) * ulp).reshape(-1), s


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        bias = 0 if state["bias"] is None else state["bias"].double()
        scale = torch.outer(state["sa"].double(), state["sb"].double())
        return (state["a"].double() @ state["b"].double().mT) * scale + bias
    if op == "quant":
        # the codes are whole numbers, defined by the fp32 scale and quotient
        return dict(q=None, s=state["x"].double().abs().max(dim=1).values / 127)
    if op == "adamw":
        lr, b1, b2 = HYPER["lr"], HYPER["beta1"], HYPER["beta2"]
        t = FIRST_STEP + 1
        spans, at = [], 0
        for n in state["sizes"]:
            spans.append((at, n))
            at += (n + TILE - 1) // TILE * TILE
        if case["kind"] == "e4m3":
            mq, ms, vq, vs = state["moments"]
            m = mq.view(torch.float8_e4m3fn).double() * ms.double().repeat_interleave(TILE)
            v = vq.view(torch.float8_e4m3fn).double() * vs.double().repeat_interleave(TILE)
        else:
            m, v = (t_.double() for t_ in state["moments"])
        p = []
        for (at, n), p0, g in zip(spans, state["p"], state["g"]):
            g = g.double()
            m[at:at + n] = torch.lerp(g, m[at:at + n], b1)
            v[at:at + n] = torch.lerp(g ** 2, v[at:at + n], b2)
            mhat, vhat = m[at:at + n] / (1 - b1 ** t), v[at:at + n] / (1 - b2 ** t)
            p.append(p0.double() - lr * HYPER["weight_decay"] * p0.double() - lr * mhat / (vhat ** 0.5 + HYPER["eps"]))
        if case["kind"] == "f32":
            return dict(p=p, m=m, v=v)
        (mc, ms), (vc, vs) = _exact_e4m3(m), _exact_e4m3(v)
        return dict(p=p, m=mc, ms=ms, v=vc, vs=vs)
    x, w = state["x"].double(), state["w"].double()
    if op == "norm_fwd":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        y = (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None]
        return dict(y=y * w + state["b"].double(), mean=mean, rstd=(var + EPS) ** -0.5)
    dy, rstd = state["dy"].double(), state["rstd"].double()[:, None]
    z = (x - state["mean"].double()[:, None]) * rstd
    u = dy * w
    n = case["cols"]
    dx = rstd / n * (n * u - u.sum(1, True) - z * (u * z).sum(1, True))
    return dict(dx=dx, dw=torch.einsum("rc,rc->c", dy, z), db=dy.sum(0))
