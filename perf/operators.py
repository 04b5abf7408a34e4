"""Cases of the training-loss operators: token log-probabilities through the
vocabulary head, distillation from a teacher's top logits, and the router's
balance loss, each with its gradient.

`run` computes a case in plain torch operations (FP32) or, with `own` set, by
the library's entry points; `exact` computes it in FP64.
"""
import math

import torch

own = False

# A case is one of three operators:
#   logprob  T tokens, hidden size d, vocabulary V; grad "" (scoring only),
#            "x" (frozen head: dX) or "xw" (dX and dW); ignored: share of the
#            tokens without a target (prompt or padding)
#   distill  the same with K teacher entries per token; absent: share of the
#            entries that are missing (id -1); ignored: share of tokens that
#            have none at all
#   balance  T tokens, E experts, k per token, S packed sequences; padded:
#            share of the tokens that do not count


def _lp(name, T, d, V, grad="", ignored=0.0, scale=1.0):
    return dict(name=name, op="logprob", T=T, d=d, V=V, grad=grad, ignored=ignored, scale=scale)


def _di(name, T, d, V, K, grad="", ignored=0.0, absent=0.0, scale=1.0):
    return dict(name=name, op="distill", T=T, d=d, V=V, K=K, grad=grad, ignored=ignored,
                absent=absent, scale=scale)


def _ba(name, T, E, k, S=1, padded=0.0):
    return dict(name=name, op="balance", T=T, E=E, k=k, S=S, padded=padded)


def listed():
    return [
        # one freshly sampled token scored against its own rollout
        _lp("logprob-token", 1, 2048, 32000),
        # a decode batch scored through the widest head
        _lp("logprob-decode512", 512, 7168, 131072, scale=1 / 0.7),
        # a short ragged batch with a prime vocabulary, prompt tokens ignored
        _lp("logprob-ragged", 333, 256, 50021, ignored=0.25),
        # a policy-gradient step through a frozen head
        _lp("policy-frozen", 4096, 2048, 131072, grad="x", ignored=0.1),
        # the same step with the head trained too
        _lp("policy-head", 4096, 2048, 32000, grad="xw"),
        # the largest: a full batch of the 7168-wide layer, frozen head
        _lp("policy-large", 8192, 7168, 131072, grad="x", ignored=0.1),
        # distance to a teacher measured only
        _di("distill-score", 1024, 2048, 65536, 32),
        # a small, odd step with absent entries, empty rows and both gradients
        _di("distill-odd", 77, 256, 1003, 5, grad="xw", ignored=0.1, absent=0.2),
        # a distillation step through a frozen head at temperature 2
        _di("distill-step", 4096, 2048, 131072, 64, grad="x", absent=0.05, scale=0.5),
        # the router of a small layer: latency
        _ba("balance-small", 64, 8, 2),
        # the routers of the large layers: one batch; packed sequences with padding
        _ba("balance-batch", 8192, 384, 8),
        _ba("balance-packed", 16384, 256, 8, S=37, padded=0.1),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MOST = 4 * 8192 * 7168 * 131072          # flops of the largest listed case


def draw(rng):
    op = rng.choice(["logprob", "logprob", "distill", "distill", "balance"])
    if op == "balance":
        E = _logu(rng, 2, 1024)
        T = _logu(rng, 1, 16384)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 8)),
                    S=min(T, _logu(rng, 1, 64)), padded=rng.choice([0.0, 0.3]))
    while True:
        grad = rng.choice(["", "x", "xw"])
        c = dict(op=op, T=_logu(rng, 1, 8192), d=64 * _logu(rng, 1, 112), V=_logu(rng, 100, 131072),
                 grad=grad, ignored=rng.choice([0.0, 0.2]), scale=rng.choice([1.0, 0.5, 1 / 0.7]))
        if op == "distill":
            c["K"] = min(_logu(rng, 1, 128), c["V"])
            c["absent"] = rng.choice([0.0, 0.2])
        if 2 * c["T"] * c["d"] * c["V"] * (1 + len(grad)) <= _MOST:
            return c


def work(case):
    T = case["T"]
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        # logits, ids, weights and their gradients in; dlogits, counts and means out
        return {"bytes": 8 * T * E + 12 * T * k + 8 * S * E + (T if case["padded"] else 0),
                "flops": 10 * T * E}
    d, V, grad = case["d"], case["V"], case["grad"]
    n = 2 * T * d + 2 * V * d + 8 * T
    if case["op"] == "distill":
        n += 8 * T * case["K"]
    else:
        n += 4 * T
    if grad:
        n += 4 * T + 2 * T * d
    if grad == "xw":
        n += 2 * V * d
    return {"bytes": n, "flops": 2 * T * d * V * (1 + len(grad))}


# ---------------------------------------------------------------- inputs

def _inputs(case, seed):
    """Seeded device tensors of a case."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    T = case["T"]
    x = {}
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        # a router's logits with a few favoured experts; top-k by (logit, lowest id)
        fav = torch.randperm(E, generator=g, device="cuda").float()
        x["logits"] = (randn(T, E) - 1.1 * torch.log1p(fav)).contiguous()
        idx = torch.sort(x["logits"], dim=1, descending=True, stable=True).indices[:, :k]
        top = x["logits"].gather(1, idx)
        x["idx"] = idx.to(torch.int32).contiguous()
        x["w"] = torch.softmax(top, dim=1).contiguous()
        x["dw"] = randn(T, k) / T
        x["valid"] = (rand(T) >= case["padded"]).to(torch.uint8) if case["padded"] else None
        cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda")).values
        ends = torch.tensor([0, T], device="cuda")
        x["seq"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32) if S > 1 else None
        x["gl"] = 0.01 * (0.5 + rand(S))
        return x
    d, V = case["d"], case["V"]
    W = randn(V, d, dtype=torch.bfloat16).mul_(0.02)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    # hidden states lean towards a token by 0 to 16 units: from unsure to confident tokens
    lean = 16 * rand(T, 1) / (0.02 * math.sqrt(d))
    X = randn(T, d)
    X += lean * W[y].float() / (0.02 * math.sqrt(d))
    x["X"], x["W"] = X.to(torch.bfloat16), W
    none = rand(T) < case["ignored"]
    if case["op"] == "logprob":
        x["target"] = torch.where(none, torch.full_like(y, -1), y).to(torch.int32)
    else:
        K = case["K"]
        # distinct ids: a start and an odd stride per token, the leaning token first
        step = 1 + torch.randint(0, max(V // K, 1), (T, 1), generator=g, device="cuda")
        ids = (y[:, None] + step * torch.arange(K, device="cuda")) % V
        gone = (rand(T, K) < case["absent"]) | none[:, None]
        x["ids"] = torch.where(gone, torch.full_like(ids, -1), ids).to(torch.int32).contiguous()
        t = randn(T, K) * 2
        t[:, 0] += 6
        x["tl"] = t.contiguous()
    x["g"] = randn(T)                     # one upstream coefficient per token (an advantage)
    return x


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        from precision_moe_adapter_gb300 import pmoe
        T, f32 = case["T"], dict(dtype=torch.float32, device="cuda")
        if case["op"] == "balance":
            E, S = case["E"], case["S"]
            s["dims"] = pmoe.dims(T, 64, E, case["k"], 64, 16)
            n = pmoe.moe_balance_ws_bytes(s["dims"], S)
            s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
            s["counts"] = torch.empty((S, E), dtype=torch.int32, device="cuda")
            s["ntok"] = torch.empty(S, dtype=torch.int32, device="cuda")
            s["pmean"], s["loss"] = torch.empty((S, E), **f32), torch.empty(S, **f32)
            s["dlogits"] = torch.empty((T, E), **f32)
        else:
            from precision_moe_adapter_gb300.head import DeviceHead
            s["head"] = DeviceHead(s["W"], T, K=case.get("K", 0), scale=case["scale"],
                                   backward=bool(case["grad"]))
            s["out"], s["lse"] = torch.empty(T, **f32), torch.empty(T, **f32)
            s["dX"] = torch.empty_like(s["X"]) if case["grad"] else None
            s["dW"] = torch.empty_like(s["W"]) if case["grad"] == "xw" else None
    return s


# ---------------------------------------------------------------- passes

def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(s, case):
    from precision_moe_adapter_gb300 import pmoe
    if case["op"] == "balance":
        pmoe.moe_balance_forward(s["dims"], s["logits"], s["idx"], s["valid"], s["seq"], case["S"],
                                 s["counts"], s["ntok"], s["pmean"], s["loss"], s["ws"])
        pmoe.moe_route_backward(s["dims"], s["logits"], s["idx"], s["w"], s["dw"], s["valid"],
                                s["seq"], case["S"], s["counts"], s["ntok"], s["gl"], s["dlogits"],
                                s["ws"])
        return {n: s[n] for n in ("counts", "pmean", "loss", "dlogits")}
    h = s["head"]
    if case["op"] == "logprob":
        h.logprob(s["X"], s["target"], s["out"], s["lse"])
        if case["grad"]:
            h.logprob_backward(s["X"], s["target"], s["lse"], s["g"], s["dX"], s["dW"])
    else:
        h.distill(s["X"], s["ids"], s["tl"], s["out"], s["lse"])
        if case["grad"]:
            h.distill_backward(s["X"], s["ids"], s["tl"], s["lse"], s["g"], s["dX"], s["dW"])
    r = {"value": s["out"], "lse": s["lse"]}
    if case["grad"]:
        r["dX"] = s["dX"]
    if case["grad"] == "xw":
        r["dW"] = s["dW"]
    return r


def _run_plain(s, case):
    T = case["T"]
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        l, idx = s["logits"], s["idx"].long()
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        v = torch.ones(T, device="cuda") if s["valid"] is None else s["valid"].float()
        if s["seq"] is None:
            sid = torch.zeros(T, dtype=torch.long, device="cuda")
        else:
            sid = (torch.arange(T, device="cuda")[:, None] >= s["seq"][1:][None, :]).sum(dim=1)
        n = torch.zeros(S, device="cuda").index_add_(0, sid, v)
        psum = torch.zeros((S, E), device="cuda").index_add_(0, sid, p * v[:, None])
        ones = v[:, None].expand(T, k).reshape(-1).to(torch.int32)
        c = torch.zeros(S * E, dtype=torch.int32, device="cuda")
        c.index_add_(0, (sid[:, None] * E + idx).reshape(-1), ones)
        c = c.view(S, E)
        n1 = n.clamp(min=1)
        pmean = psum / n1[:, None]
        f = c.float() / (k * n1[:, None])
        loss = E * (f * pmean).sum(dim=1)
        coef = (s["gl"] * E / n1)[sid] * v
        ft = f[sid]
        dl = coef[:, None] * p * (ft - (p * ft).sum(dim=1, keepdim=True))
        dot = (s["w"] * s["dw"]).sum(dim=1, keepdim=True)
        dl = dl.scatter_add(1, idx, s["w"] * (s["dw"] - dot))
        return {"counts": c, "pmean": pmean, "loss": loss, "dlogits": dl}
    X, W, sc = s["X"].float(), s["W"].float(), case["scale"]
    z = (X @ W.t()) * sc
    m = z.amax(dim=1, keepdim=True)
    lse = m[:, 0] + torch.log(torch.exp(z - m).sum(dim=1))
    if case["op"] == "logprob":
        y = s["target"].long()
        has = y >= 0
        y0 = y.clamp(min=0)[:, None]
        value = torch.where(has, z.gather(1, y0)[:, 0] - lse, torch.zeros_like(lse))
        if case["grad"]:
            G = torch.exp(z - lse[:, None])
            G = G.scatter_add(1, y0, torch.full((T, 1), -1.0, device="cuda"))
            G = G * torch.where(has, -s["g"] * sc, torch.zeros_like(lse))[:, None]
    else:
        ids = s["ids"].long()
        has = ids >= 0
        t = torch.where(has, s["tl"] * sc, torch.full_like(s["tl"], -math.inf))
        tm = t.amax(dim=1, keepdim=True)
        q = torch.where(has, torch.exp(t - tm), torch.zeros_like(t))
        qs = q.sum(dim=1, keepdim=True)
        q = torch.where(qs > 0, q / qs, torch.zeros_like(q))
        i0 = ids.clamp(min=0)
        lq = torch.where(q > 0, torch.log(q), torch.zeros_like(q))
        value = (q * (lq - (z.gather(1, i0) - lse[:, None]))).sum(dim=1)
        if case["grad"]:
            G = torch.exp(z - lse[:, None]) * (qs > 0).float()
            G = G.scatter_add(1, i0, -q) * (s["g"] * sc)[:, None]
    r = {"value": value, "lse": lse}
    if case["grad"]:
        r["dX"] = (G @ W).to(torch.bfloat16)
    if case["grad"] == "xw":
        r["dW"] = (G.t() @ X).to(torch.bfloat16)
    return r


# ---------------------------------------------------------------- FP64

def exact(case, seed):
    T = case["T"]
    if case["op"] != "balance" and case["T"] * case["d"] * case["V"] * (1 + len(case["grad"])) > 6e12:
        return None                       # FP64 products of more than about ten seconds
    s = _inputs(case, seed)
    D = torch.float64
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        logits, w, dw = s["logits"].to(D), s["w"].to(D), s["dw"].to(D)
        bounds = [0, T] if s["seq"] is None else s["seq"].tolist()
        counts = torch.zeros((S, E), dtype=torch.int32, device="cuda")
        pmean = torch.zeros((S, E), dtype=D, device="cuda")
        loss = torch.zeros(S, dtype=D, device="cuda")
        dl = torch.zeros((T, E), dtype=D, device="cuda")
        sel = (dw - (w * dw).sum(1, keepdim=True)) * w
        dl.scatter_(1, s["idx"].long(), sel)
        for j in range(S):
            rows = torch.arange(bounds[j], bounds[j + 1], device="cuda")
            if s["valid"] is not None:
                rows = rows[s["valid"][rows] != 0]
            n = rows.numel()
            if n == 0:
                continue
            P = torch.softmax(logits[rows], dim=1)
            c = torch.bincount(s["idx"][rows].reshape(-1).long(), minlength=E)
            counts[j], pmean[j] = c.to(torch.int32), P.mean(0)
            a = E * c.to(D) / (k * n)
            loss[j] = (a * pmean[j]).sum()
            dl[rows] += s["gl"][j].to(D) / n * (P * a - P * (P @ a)[:, None])
        return {"counts": counts, "pmean": pmean, "loss": loss, "dlogits": dl}
    sc, d, V = case["scale"], case["d"], case["V"]
    W = s["W"].to(D)
    value, lse = (torch.empty(T, dtype=D, device="cuda") for _ in range(2))
    dX = torch.empty((T, d), dtype=D, device="cuda") if case["grad"] else None
    dW = torch.zeros((V, d), dtype=D, device="cuda") if case["grad"] == "xw" else None
    for a in range(0, T, 1024):           # by tokens, so that the logits stay small
        r = slice(a, min(T, a + 1024))
        X = s["X"][r].to(D)
        z = sc * torch.mm(X, W.T)
        lse[r] = torch.logsumexp(z, 1)
        logp = z - lse[r][:, None]
        q = torch.zeros_like(z)           # the target distribution of each token
        if case["op"] == "logprob":
            rows = torch.nonzero(s["target"][r] >= 0)[:, 0]
            q[rows, s["target"][r][rows].long()] = 1.0
            value[r] = (q * logp).sum(1)
            sign = -1.0
        else:
            ids, t = s["ids"][r].long(), s["tl"][r].to(D) * sc
            t = t.masked_fill(ids < 0, -math.inf)
            qk = torch.nan_to_num(torch.softmax(t, 1))
            q.scatter_add_(1, ids.clamp(min=0), qk)
            value[r] = torch.xlogy(qk, qk).sum(1) - (q * logp).sum(1)
            sign = 1.0
        if case["grad"]:
            up = sign * sc * s["g"][r].to(D)
            G = (logp.exp() * q.sum(1, keepdim=True) - q) * up[:, None]
            dX[r] = G @ W
            if dW is not None:
                dW += G.T @ X
    out = {"value": value, "lse": lse}
    if dX is not None:
        out["dX"] = dX
    if dW is not None:
        out["dW"] = dW
    return out
