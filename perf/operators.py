"""Cases for measuring the router and FP8 operators of the MoE layer.

Four operators, each in a plain form (elementary torch operations) and as the
call a user makes of the package:

* route      top-k routing with a per-expert bias for load balance: the bias
             takes part in the choice of experts and not in their weights
* route_grad the gradient of the routing weights with respect to the logits
* quant      E4M3 codes and scales per (row, group of 128 columns), of a
             tensor or of SiLU(gate) * up
* matmul     product of E4M3 matrices with a scale per (row, group of 128) of
             the activations and per 128 x 128 block of the weight

`own = False` runs the plain forms, `own = True` the package's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
GROUP = 128
MAX_FLOPS = 2.0 * 8192 * 7168 * 4096


# ------------------------------------------------------------------ cases --
def _route(name, M, E, k, method, renorm, groups, kept, mode, scale, dtype):
    return dict(name=name, op="route", M=M, E=E, k=k, method=method, renorm=renorm, groups=groups,
                kept=kept, mode=mode, scale=scale, dtype=dtype)


def _grad(name, M, E, k, method, renorm, scale, dtype):
    return dict(name=name, op="route_grad", M=M, E=E, k=k, method=method, renorm=renorm,
                scale=scale, dtype=dtype)


def _quant(name, M, K, swiglu):
    return dict(name=name, op="quant", M=M, K=K, swiglu=swiglu)


def _matmul(name, M, K, N, transposed, bias, dtype):
    return dict(name=name, op="matmul", M=M, K=K, N=N, transposed=transposed, bias=bias,
                dtype=dtype)


def listed():
    return [
        # one token of a decode step, DeepSeek-V3 routing: the latency of the call
        _route("route one token", 1, 256, 8, "sigmoid", True, 8, 4, 1, 2.5, "float32"),
        # the same routing over a prefill chunk
        _route("route prefill", 8192, 256, 8, "sigmoid", True, 8, 4, 1, 2.5, "float32"),
        # Qwen-MoE routing of a large batch, router logits in bf16, no groups
        _route("route softmax", 16384, 128, 8, "softmax", False, 1, 1, 0, 1.0, "bfloat16"),
        # a router's training step, softmax without renormalisation: a dense gradient
        _grad("route gradient softmax", 16384, 128, 8, "softmax", False, 1.0, "bfloat16"),
        # the same for sigmoid scores: only the chosen experts' logits have a gradient
        _grad("route gradient sigmoid", 8191, 256, 8, "sigmoid", True, 2.5, "float32"),
        # activations of a small decode batch ahead of the shared expert's first product
        _quant("quantise decode", 64, 7168, False),
        # of a prefill chunk
        _quant("quantise prefill", 8192, 7168, False),
        # between the shared expert's two products: SiLU(gate) * up quantised in one pass
        _quant("quantise swiglu", 8191, 2048, True),
        # shared expert's gate/up product for one token: the weights' bytes
        _matmul("matmul one token", 1, 7168, 4096, False, False, "bfloat16"),
        # its down product for a decode batch, odd count of tokens
        _matmul("matmul decode", 77, 2048, 7168, False, False, "bfloat16"),
        # gate/up product of a prefill chunk: the tensor cores' rate
        _matmul("matmul prefill", 8192, 7168, 4096, False, False, "bfloat16"),
        # weights in the checkpoints' order (rows of K), ragged sizes, bias, fp32 result:
        # a projection beside the experts, or the product of a gradient with the same weights
        _matmul("matmul transposed", 1999, 4096, 2064, True, True, "float32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "quant", "matmul", "matmul"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = groups * rng.randint(max(2, 8 // groups), max(3, 512 // groups))
        kept = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(16, kept * (E // groups)))
        M = _log(rng, 1, min(32768, 4 * 1024 * 1024 // E))
        method = rng.choice(["softmax", "sigmoid"])
        renorm = method == "sigmoid" or rng.random() < 0.5
        scale, dtype = rng.choice([1.0, 2.5]), rng.choice(["float32", "bfloat16"])
        if op == "route":
            c = _route("", M, E, k, method, renorm, groups, kept, rng.randint(0, 1), scale, dtype)
        else:
            # one renormalised weight is constant: its gradient is zero
            c = _grad("", M, E, max(k, 2) if renorm else k, method, renorm, scale, dtype)
    elif op == "quant":
        c = _quant("", _log(rng, 1, 8192), 16 * _log(rng, 2, 448), rng.random() < 0.5)
    else:
        K, N = 16 * _log(rng, 8, 448), 16 * _log(rng, 4, 448)
        M = min(_log(rng, 1, 8192), int(MAX_FLOPS / (2.0 * K * N)))
        c = _matmul("", M, K, N, rng.random() < 0.5, rng.random() < 0.3,
                    rng.choice(["bfloat16", "float32"]))
    del c["name"]
    return c


def _blocks(n):
    return -(-n // GROUP)


def work(case):
    M = case["M"]
    if case["op"] == "route":
        E, k, b = case["E"], case["k"], 2 if case["dtype"] == "bfloat16" else 4
        # scores, bias and weights; the comparisons of a selection are not counted
        return {"bytes": M * E * b + 4 * E + 8 * M * k, "flops": 4.0 * M * E}
    if case["op"] == "route_grad":
        E, k, b = case["E"], case["k"], 2 if case["dtype"] == "bfloat16" else 4
        dense = case["method"] == "softmax" and not case["renorm"]
        read = M * (E if dense else k) * b
        return {"bytes": read + M * E * b + 8 * M * k, "flops": 4.0 * M * (E if dense else k)}
    if case["op"] == "quant":
        K = case["K"]
        return {"bytes": 2 * M * K * (2 if case["swiglu"] else 1) + M * K + 4 * M * _blocks(K),
                "flops": (8.0 if case["swiglu"] else 2.0) * M * K}
    K, N = case["K"], case["N"]
    out = 4 if case["dtype"] == "float32" else 2
    return {"bytes": M * K + K * N + 4 * M * _blocks(K) + 4 * _blocks(K) * _blocks(N)
            + out * M * N + (2 * N if case["bias"] else 0), "flops": 2.0 * M * K * N}


# ----------------------------------------------------------------- inputs --
def _gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 16 + stream)
    return g


def _randn(seed, stream, *shape):
    return torch.randn(*shape, generator=_gen(seed, stream), device=DEV, dtype=torch.float32)


def _expand(scale, rows, cols):
    """A scale per block as one per element, [rows, cols]."""
    s = scale
    if s.shape[0] != rows:
        s = s.repeat_interleave(GROUP, 0)[:rows]
    return s.repeat_interleave(GROUP, 1)[:, :cols]


def prepare(case, seed):
    M = case["M"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        # a learned bias is of the size of the scores' differences
        spread = 0.05 if case["method"] == "sigmoid" else 0.5 / E
        return dict(case=case, logits=_randn(seed, 1, M, E).to(getattr(torch, case["dtype"])),
                    bias=_randn(seed, 2, E) * spread,
                    w=torch.empty(M, k, device=DEV),
                    ids=torch.empty(M, k, device=DEV, dtype=torch.int32))
    if case["op"] == "route_grad":
        E, k = case["E"], case["k"]
        logits = _randn(seed, 1, M, E).to(getattr(torch, case["dtype"]))
        ids = torch.argsort(logits.float() + 0.3 * _randn(seed, 2, M, E), dim=1,
                            descending=True)[:, :k].to(torch.int32).contiguous()
        return dict(case=case, logits=logits, ids=ids, gw=_randn(seed, 3, M, k),
                    out=torch.empty_like(logits))
    K = case["K"]
    if case["op"] == "quant":
        x = _randn(seed, 1, M, K * (2 if case["swiglu"] else 1)).to(torch.bfloat16)
        return dict(case=case, x=x, q=torch.empty(M, K, device=DEV, dtype=E4M3),
                    scale=torch.empty(M, _blocks(K), device=DEV))
    N = case["N"]
    a_q, a_scale = _quantise(_randn(seed, 1, M, K).to(torch.bfloat16).float())
    rows, cols = (N, K) if case["transposed"] else (K, N)
    w_scale = torch.rand(_blocks(rows), _blocks(cols), generator=_gen(seed, 3), device=DEV)
    return dict(case=case, a_q=a_q, a_scale=a_scale, w_q=_randn(seed, 2, rows, cols).to(E4M3),
                w_scale=0.015 + 0.01 * w_scale,
                bias=_randn(seed, 4, N).to(torch.bfloat16) if case["bias"] else None,
                out=torch.empty(M, N, device=DEV, dtype=getattr(torch, case["dtype"])))


# ------------------------------------------------------------ plain forms --
def _scores(logits, method):
    """Scores in 64 bits: the choice of experts compares them, and values
    next to a border have to fall on the right side of it."""
    l = logits.double()
    if method == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    c = s["case"]
    M, E, k, G = c["M"], c["E"], c["k"], c["groups"]
    p = _scores(s["logits"], c["method"])
    choice = p + s["bias"].double()
    if G > 1:
        g = choice.view(M, G, E // G)
        if c["mode"] == 0:
            gs = g.amax(2)
        else:
            top = torch.sort(g, dim=2, descending=True).values
            gs = top[:, :, 0] + top[:, :, 1]
        kept = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros(M, G, dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        choice = torch.where(keep.repeat_interleave(E // G, 1), choice, -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return (w * c["scale"]).float(), ids.to(torch.int32)


def _plain_route_grad(s):
    c = s["case"]
    l, ids, gw = s["logits"].float(), s["ids"].long(), s["gw"]
    if c["method"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    ps = p.gather(1, ids)
    if c["renorm"]:
        total = ps.sum(1, keepdim=True)
        gp = c["scale"] * (gw - (gw * ps).sum(1, keepdim=True) / total) / total
    else:
        gp = c["scale"] * gw
    dense = torch.zeros_like(l).scatter_add_(1, ids, gp)
    if c["method"] == "sigmoid":
        g = dense * p * (1.0 - p)
    else:
        g = p * (dense - (gp * ps).sum(1, keepdim=True))
    return g.to(s["logits"].dtype)


def _quantise(z):
    M, K = z.shape
    amax = torch.nn.functional.pad(z, (0, _blocks(K) * GROUP - K)).view(M, -1, GROUP).abs().amax(2)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    q = (z / _expand(scale, M, K)).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    return q, scale


def _plain_quant(s):
    x = s["x"].float()
    if s["case"]["swiglu"]:
        K = s["case"]["K"]
        gate, up = x[:, :K], x[:, K:]
        x = gate / (1.0 + torch.exp(-gate)) * up
    return _quantise(x)


def _plain_matmul(s):
    a = s["a_q"].float()
    a = a * _expand(s["a_scale"], *a.shape)
    w = s["w_q"].float()
    w = w * _expand(s["w_scale"], *w.shape)
    y = a @ (w.t() if s["case"]["transposed"] else w)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(getattr(torch, s["case"]["dtype"]))


# -------------------------------------------------------------------- run --
def _own(s):
    import mixture_experts_ffn_softmax_gb300 as moe
    c = s["case"]
    if c["op"] == "route":
        return moe.moe_route(s["logits"], c["k"], c["method"], c["renorm"], c["kept"], c["groups"],
                             c["mode"], c["scale"], s["w"], s["ids"], score_bias=s["bias"])
    if c["op"] == "route_grad":
        return moe.moe_route_backward(s["gw"], s["logits"], s["ids"], c["method"], c["renorm"],
                                      c["scale"], grad_logits=s["out"])
    if c["op"] == "quant":
        return moe.moe_quant_groups_fp8(s["x"], swiglu=c["swiglu"], q8=s["q"], scale=s["scale"])
    return moe.moe_matmul_fp8(s["a_q"], s["a_scale"], s["w_q"], s["w_scale"], bias=s["bias"],
                              transposed=c["transposed"], out=s["out"])


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "route_grad": _plain_route_grad, "quant": _plain_quant,
            "matmul": _plain_matmul}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact --
def _exact_log_scores(l, method):
    """Logarithms of the scores in 64 bits."""
    if method == "sigmoid":
        return -torch.logaddexp(torch.zeros_like(l), -l)
    return l - torch.logsumexp(l, 1, keepdim=True)


def _exact_route(s):
    """Expert by expert: rank = how many experts come before it."""
    c = s["case"]
    M, E, G = c["M"], c["E"], c["groups"]
    lp = _exact_log_scores(s["logits"].double(), c["method"])
    choice = lp.exp() + s["bias"].double()
    if G > 1:
        g = choice.view(M, G, -1)
        first = g.amax(2)
        if c["mode"] == 1:
            at = torch.zeros_like(g, dtype=torch.bool).scatter_(2, g.argmax(2, keepdim=True), True)
            first = first + torch.where(at, -math.inf, g).amax(2)
        lower = torch.ones(G, G, dtype=torch.bool, device=DEV).tril(-1)   # [g, h]: h < g
        before = (first[:, None, :] > first[:, :, None]) | (
            (first[:, None, :] == first[:, :, None]) & lower)
        keep = before.sum(2) < c["kept"]
        choice = choice.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    ids = []
    rest = choice.clone()
    for _ in range(c["k"]):
        top = rest.amax(1, keepdim=True)
        i = torch.where(rest == top, torch.arange(E, device=DEV), E).amin(1, keepdim=True)
        ids.append(i)
        rest.scatter_(1, i, -math.inf)
    ids = torch.cat(ids, 1)
    lw = lp.gather(1, ids)
    if c["renorm"]:
        lw = lw - torch.logsumexp(lw, 1, keepdim=True)
    return lw.exp() * c["scale"], ids.to(torch.int32)


def _exact_route_grad(s):
    """Through the logarithms: w_j = scale * exp(u_j) with u the log scores
    (less their log-sum over the chosen ones where renormalised)."""
    c = s["case"]
    l, ids, gw = s["logits"].double(), s["ids"].long(), s["gw"].double()
    lp = _exact_log_scores(l, c["method"])
    u = lp.gather(1, ids)
    if c["renorm"]:
        u = u - torch.logsumexp(u, 1, keepdim=True)
    gu = gw * c["scale"] * u.exp()
    if c["renorm"]:
        gu = gu - u.exp() * gu.sum(1, keepdim=True)
    g = torch.zeros_like(l)
    rows = torch.arange(c["M"], device=DEV)[:, None].expand_as(ids)
    if c["method"] == "sigmoid":
        g.index_put_((rows, ids), gu * torch.sigmoid(-l.gather(1, ids)), accumulate=True)
    else:
        g.index_put_((rows, ids), gu, accumulate=True)
        g -= lp.exp() * gu.sum(1, keepdim=True)
    return g


def _exact_e4m3(v):
    """Nearest E4M3 value, ties to even, of |v| <= 448, in 64 bits."""
    e = torch.frexp(v.abs()).exponent.double() - 1.0
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return torch.round(v / step) * step


def _exact_quant(s):
    c = s["case"]
    K = c["K"]
    x = s["x"].double()
    if c["swiglu"]:
        x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
    q, scale = torch.empty_like(x), []
    for k0 in range(0, K, GROUP):
        part = x[:, k0:k0 + GROUP]
        amax = part.abs().amax(1, keepdim=True)
        sc = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
        scale.append(sc)
        q[:, k0:k0 + GROUP] = _exact_e4m3(part / sc)
    return q, torch.cat(scale, 1)


def _exact_matmul(s):
    c = s["case"]
    y = torch.zeros(c["M"], c["N"], dtype=torch.float64, device=DEV)
    columns = torch.arange(c["N"], device=DEV) // GROUP
    w_q, w_scale = (s["w_q"], s["w_scale"])
    for b, k0 in enumerate(range(0, c["K"], GROUP)):
        a = s["a_q"][:, k0:k0 + GROUP].double() * s["a_scale"][:, b:b + 1].double()
        if c["transposed"]:
            w = w_q[:, k0:k0 + GROUP].double().t() * w_scale[:, b].double()[columns]
        else:
            w = w_q[k0:k0 + GROUP].double() * w_scale[b].double()[columns]
        y += a @ w
    return y if s["bias"] is None else y + s["bias"].double()


def exact(case, seed):
    return {"route": _exact_route, "route_grad": _exact_route_grad, "quant": _exact_quant,
            "matmul": _exact_matmul}[case["op"]](prepare(case, seed))
