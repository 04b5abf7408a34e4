"""Cases of the operators around a layer on an FP8 base: the 8-bit linear layer
(activations and weights in E4M3 with a scale per block of 128), the gate that
routes by scores with a balancing bias and groups, and the global gradient norm
with clipping.

`run` computes a case in plain torch operations or, with `own` set, by the
library's entry points; `exact` computes it in FP64.
"""
import math

import torch

own = False

# A case is one of three operators:
#   linear  rows x K hidden states (BF16) through a frozen N x K weight in E4M3
#           with FP32 scales per [128, 128]; the activations are quantised per
#           row and 128 columns; grad: dX of an upstream dY in the same way
#           (dY quantised along N) beside Y; pow2: scales of the activations are
#           powers of two
#   gate    T tokens, E experts, k of them chosen by scores (sigmoid or softmax
#           of the logits) plus a bias, out of the best `top` of `groups` groups
#           (a group counts by its best `gsum` experts); the weights are the
#           scores alone, renormalised or not, times a factor; grad: d_logits
#   clip    n gradients of `lo` to `hi` elements (the sizes spread over their
#           logarithm, or all alike), a share `half` of them BF16, scaled so that
#           their global norm is at most 1; over: the norm is above it


def _li(name, rows, N, K, grad=False, pow2=False):
    return dict(name=name, op="linear", rows=rows, N=N, K=K, grad=grad, pow2=pow2)


def _ga(name, T, E, k, score="sigmoid", bias=True, groups=1, top=1, gsum=2, renorm=True, factor=1.0,
        grad=False):
    return dict(name=name, op="gate", T=T, E=E, k=k, score=score, bias=bias, groups=groups, top=top,
                gsum=gsum, renorm=renorm, factor=factor, grad=grad)


def _cl(name, n, lo, hi, half=0.0, over=True):
    return dict(name=name, op="clip", n=n, lo=lo, hi=hi, half=half, over=over)


def listed():
    return [
        # decoding: one token through a projection of the 7168-wide layer
        _li("linear-token", 1, 4096, 7168),
        # a decode batch through the widest one
        _li("linear-decode64", 64, 7168, 7168),
        # a ragged batch, sizes that end inside a block of 128, scales as powers of two, and dX
        _li("linear-ragged", 333, 1104, 2064, grad=True, pow2=True),
        # a training step: forward and dX
        _li("linear-step", 8192, 4096, 7168, grad=True),
        # the largest batch
        _li("linear-large", 16384, 7168, 7168, grad=True),
        # decoding: one token's experts
        _ga("gate-token", 1, 384, 8, factor=2.5),
        # softmax scores kept as they are, no bias, groups by their best expert, odd sizes
        _ga("gate-odd", 333, 60, 6, score="softmax", bias=False, groups=6, top=3, gsum=1,
            renorm=False, factor=16.0, grad=True),
        # a training batch of the 384-expert layer
        _ga("gate-batch", 8192, 384, 8, factor=2.5, grad=True),
        # a large batch of the 256-expert layer with groups
        _ga("gate-groups", 16384, 256, 8, groups=8, top=4, factor=2.5, grad=True),
        # a small model's gradients: latency, and a norm below the limit
        _cl("clip-small", 24, 1, 4096, over=False),
        # many gradients of all sizes, a head's in BF16 among them
        _cl("clip-many", 60, 7, 40000000, half=0.5),
        # the adapter gradients of one 384-expert layer, two tensors of f32
        _cl("clip-adapter", 2, 384 * 32 * 4096, 384 * 112 * 4096),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "gate", "clip"])
    if op == "linear":
        while True:
            c = _li(None, _logu(rng, 1, 16384), 16 * _logu(rng, 4, 448), 16 * _logu(rng, 4, 448),
                    rng.random() < 0.5, rng.random() < 0.3)
            if c["rows"] * c["N"] * c["K"] <= 16384 * 7168 * 7168:
                break
    elif op == "gate":
        groups = rng.choice([1, 1, 2, 4, 6, 8])
        E = groups * _logu(rng, 2, 1024 // groups)
        top = rng.randint(1, groups)
        c = _ga(None, _logu(rng, 1, 16384), E, rng.randint(1, min(8, top * (E // groups))),
                score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.7, groups=groups,
                top=top, gsum=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                factor=rng.choice([1.0, 2.5]), grad=rng.random() < 0.7)
    else:
        n = _logu(rng, 1, 60)
        hi = _logu(rng, 1, 226492416 // n)
        c = _cl(None, n, _logu(rng, 1, hi), hi, half=rng.choice([0.0, 0.5, 1.0]), over=rng.random() < 0.7)
    del c["name"]
    return c


def _sizes(case):
    """The gradients' sizes and types: spread over the logarithm, in a fixed shuffled order."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    out = []
    for i in range(n):
        j = (i * 7919 + 3) % n if n % 7919 else i
        f = j / (n - 1) if n > 1 else 1.0
        size = int(round(lo * (hi / lo) ** f))
        half = math.floor((i + 1) * case["half"]) > math.floor(i * case["half"])
        out.append((size, torch.bfloat16 if half else torch.float32))
    return out


def _blocks(n):
    return (n + 127) // 128


def work(case):
    if case["op"] == "linear":
        M, N, K = case["rows"], case["N"], case["K"]
        w = N * K + 4 * _blocks(N) * _blocks(K)
        n = 2 * M * K + 2 * M * N + w
        if case["grad"]:
            n += 2 * M * K + 2 * M * N      # the weight is one input of the step
        return {"bytes": n, "flops": 2 * M * N * K * (2 if case["grad"] else 1)}
    if case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        n = 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0)
        if case["grad"]:
            n += 4 * T * k + 4 * T * E
        return {"bytes": n, "flops": 8 * T * E}
    n = f = 0
    for size, t in _sizes(case):
        n += 2 * size * t.itemsize
        f += 3 * size
    return {"bytes": n + 4, "flops": f}


# ---------------------------------------------------------------- inputs

def _inputs(case, seed):
    """Seeded device tensors of a case."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    x = {}
    if case["op"] == "linear":
        M, N, K = case["rows"], case["N"], case["K"]
        # hidden states whose channels and rows differ in size, a few of them by much
        ch = torch.exp(0.5 * randn(K)) * torch.where(rand(K) < 0.01, 8.0, 1.0)
        x["X"] = (randn(M, K) * ch * torch.exp(0.3 * randn(M, 1))).to(torch.bfloat16)
        x["q"] = randn(N, K).to(torch.float8_e4m3fn)
        x["s"] = 0.005 + 0.015 * rand(_blocks(N), _blocks(K))
        if case["grad"]:
            x["dY"] = (randn(M, N) * 0.1 * torch.exp(0.5 * randn(M, 1))).to(torch.bfloat16)
    elif case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        fav = torch.randperm(E, generator=g, device="cuda").float()
        if case["score"] == "softmax":
            x["logits"] = (randn(T, E) - 1.1 * torch.log1p(fav)).contiguous()
        else:
            x["logits"] = (1.5 * randn(T, E) - 0.3 * torch.log1p(fav)).contiguous()
        # a bias as a few thousand steps of balancing leave it: more for rarely chosen experts
        x["bias"] = (0.02 * torch.log1p(fav) + 0.01 * randn(E)) if case["bias"] else None
        x["dw"] = randn(T, k)
    else:
        x["g"] = [randn(n, dtype=t) for n, t in _sizes(case)]
        total = math.sqrt(sum(n for n, _ in _sizes(case)))      # about their norm
        x["max_norm"] = total * (0.4 if case["over"] else 4.0) + (0.0 if case["over"] else 8.0)
    return x


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        if case["op"] == "linear":
            from precision_moe_adapter_gb300.linear import DeviceLinearW8A8
            s["lin"] = DeviceLinearW8A8(s["q"], s["s"], case["rows"], pow2=case["pow2"],
                                        backward=case["grad"])
            s["Y"] = torch.empty((case["rows"], case["N"]), dtype=torch.bfloat16, device="cuda")
            s["dX"] = torch.empty_like(s["X"]) if case["grad"] else None
        elif case["op"] == "gate":
            from precision_moe_adapter_gb300 import pmoe
            T, E, k = case["T"], case["E"], case["k"]
            s["gate"] = pmoe.gate(T, E, k, score=case["score"], groups=case["groups"],
                                  topk_groups=case["top"], group_sum=case["gsum"],
                                  renorm=case["renorm"], factor=case["factor"])
            s["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
            s["w"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
            s["dlogits"] = torch.empty((T, E), dtype=torch.float32, device="cuda") if case["grad"] else None
        else:
            from precision_moe_adapter_gb300.grads import GradList
            s["out"] = [torch.empty_like(t) for t in s["g"]]
            s["list"] = GradList(s["g"], out=s["out"])
            s["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------- passes

def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(s, case):
    if case["op"] == "linear":
        s["lin"].forward(s["X"], s["Y"])
        if not case["grad"]:
            return {"Y": s["Y"]}
        s["lin"].backward(s["X"], s["dY"], s["dX"])
        return {"Y": s["Y"], "dX": s["dX"]}
    if case["op"] == "gate":
        from precision_moe_adapter_gb300 import pmoe
        pmoe.moe_gate_forward(s["gate"], s["logits"], s["bias"], s["idx"], s["w"])
        r = {"idx": s["idx"], "w": s["w"]}
        if case["grad"]:
            pmoe.moe_gate_backward(s["gate"], s["logits"], s["idx"], s["dw"], s["dlogits"])
            r["dlogits"] = s["dlogits"]
        return r
    s["list"].clip(s["max_norm"], s["norm"])
    return {"norm": s["norm"], "out": s["out"]}


def _quantised(X, pow2):
    """The values that X (FP32) has in E4M3 with a scale per row and 128 columns."""
    M, K = X.shape
    nb = _blocks(K)
    P = torch.zeros((M, nb * 128), device=X.device)
    P[:, :K] = X
    P = P.view(M, nb, 128)
    a = P.abs().amax(dim=2, keepdim=True).clamp(min=2.0 ** -100)
    if pow2:
        m, e = torch.frexp(a)                       # a = m 2^e, m in [1/2, 1); 448 = (7/8) 2^9
        e = torch.where(m > 0.875, e - 8, e - 9)
        sc = torch.ldexp(torch.ones_like(a), e)
        v = P / sc
    else:
        sc = a / torch.full_like(a, 448)
        v = P * 448 / a        # (of BF16 values: the quotient in 32 bits rounds to E4M3 as the exact one does)
    return (v.to(torch.float8_e4m3fn).float() * sc).view(M, nb * 128)[:, :K]


def _run_plain(s, case):
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        W = s["s"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K] * s["q"].float()
        r = {"Y": (_quantised(s["X"].float(), case["pow2"]) @ W.t()).to(torch.bfloat16)}
        if case["grad"]:
            r["dX"] = (_quantised(s["dY"].float(), case["pow2"]) @ W).to(torch.bfloat16)
        return r
    if case["op"] == "gate":
        T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
        l = s["logits"].double()                    # in 64 bits: scores next to one another
        if case["score"] == "sigmoid":
            sc = 1 / (1 + torch.exp(-l))
        else:
            e = torch.exp(l - l.amax(dim=1, keepdim=True))
            sc = e / e.sum(dim=1, keepdim=True)
        c = sc if s["bias"] is None else sc + s["bias"].double()
        if case["top"] < G:
            cg = torch.sort(c.view(T, G, E // G), dim=2, descending=True).values
            gs = cg[:, :, :case["gsum"]].sum(dim=2)
            best = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            keep = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, best, True)
            c = torch.where(keep.repeat_interleave(E // G, 1), c, torch.full_like(c, -math.inf))
        idx = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
        sel = sc.gather(1, idx)
        D = sel.sum(dim=1, keepdim=True) + 1e-20 if case["renorm"] else torch.ones_like(sel[:, :1])
        w = case["factor"] * sel / D
        r = {"idx": idx.to(torch.int32), "w": w.float()}
        if case["grad"]:
            ds = case["factor"] * s["dw"].double() / D
            if case["renorm"]:
                ds = ds - (ds * sel).sum(dim=1, keepdim=True) / D
            dl = torch.zeros_like(l)
            if case["score"] == "sigmoid":
                dl.scatter_(1, idx, ds * sel * (1 - sel))
            else:
                dl.scatter_(1, idx, ds * sel)
                dl = dl - sc * (ds * sel).sum(dim=1, keepdim=True)
            r["dlogits"] = dl.float()
        return r
    total = torch.zeros((), dtype=torch.float64, device="cuda")     # long sums in 64 bits
    for t in s["g"]:
        total = total + (t.double() * t.double()).sum()
    norm = torch.sqrt(total)
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return {"norm": norm.float().view(1), "out": [(t.float() * coef).to(t.dtype) for t in s["g"]]}


# ---------------------------------------------------------------- FP64

def _e4m3(v):
    """Doubles rounded to the nearest E4M3 value, ties to even: steps of 2^-9
    below 2^-6, else of an eighth of the power of two below."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(v / step).mul_(step).clamp_(-448, 448)


def _block_values(X, pow2):
    X = X.double()
    out = torch.empty_like(X)
    for c in range(0, X.shape[1], 128):
        x = X[:, c:c + 128]
        a = x.abs().max(dim=1, keepdim=True).values.clamp(min=2.0 ** -100)
        if pow2:
            scale = torch.exp2(torch.ceil(torch.log2(a / 448)))
            q = _e4m3(x / scale)
        else:                                      # (the scale is kept as an FP32 number)
            scale = (a / 448).float().double()
            q = _e4m3(x * 448 / a)
        out[:, c:c + 128] = q * scale
    return out


def exact(case, seed):
    if case["op"] == "linear" and 2 * case["rows"] * case["N"] * case["K"] > 1.2e12:
        return None                       # FP64 products of more than a few seconds
    s = _inputs(case, seed)
    D = torch.float64
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        W = s["q"].to(D)
        for i in range(s["s"].shape[0]):
            for j in range(s["s"].shape[1]):
                W[128 * i:128 * i + 128, 128 * j:128 * j + 128] *= s["s"][i, j].to(D)
        out = {"Y": torch.mm(_block_values(s["X"], case["pow2"]), W.T)}
        if case["grad"]:
            out["dX"] = torch.mm(_block_values(s["dY"], case["pow2"]), W)
        return out
    if case["op"] == "gate":
        T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
        l = s["logits"].to(D).requires_grad_(case["grad"])
        sc = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
        c = sc.detach() + (0 if s["bias"] is None else s["bias"].to(D))
        dead = torch.zeros((T, E), dtype=torch.bool, device="cuda")
        if G > 1:
            gs = c.view(T, G, E // G).topk(min(case["gsum"], E // G), dim=2).values.sum(2)
            # a group is out where as many groups as are taken stand before it
            a, b = gs[:, :, None], gs[:, None, :]
            lower = torch.ones((G, G), device="cuda").tril(-1).bool()
            before = (b > a) | ((b == a) & lower)
            dead = (before.sum(2) >= case["top"])[:, :, None].expand(T, G, E // G).reshape(T, E)
        c = c.masked_fill(dead, -math.inf)
        idx = torch.empty((T, k), dtype=torch.long, device="cuda")
        for j in range(k):                # the largest left, the lowest id among equals
            m = c.max(1, keepdim=True).values
            idx[:, j] = (c == m).to(torch.int8).argmax(1)
            c.scatter_(1, idx[:, j:j + 1], -math.inf)
        w = sc.gather(1, idx)
        if case["renorm"]:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        w = w * case["factor"]
        out = {"idx": idx.to(torch.int32), "w": w.detach()}
        if case["grad"]:
            out["dlogits"] = torch.autograd.grad((w * s["dw"].to(D)).sum(), l)[0]
        return out
    norm = math.sqrt(sum(float(torch.dot(t.to(D), t.to(D))) for t in s["g"]))
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], dtype=D, device="cuda"), "out": [t.to(D) * coef for t in s["g"]]}
