"""Cases for measuring the products of rows sorted by expert, with their
gradients, and the 4-bit microscaled ones.

Five operators, each in a plain form (elementary torch operations) and as the
call a user makes of the package:

* product      y[r] = x[r] W[expert of r], rows sorted by expert, experts of any
               number of rows, the weights in either orientation (so that the
               stored weight serves y = x W and dx = dy W^T)
* weight_grad  dW[e] = x_e^T dy_e over the rows of each expert
* swiglu_grad  gradients of z = weight * SiLU(gate) * up: of gate, up and the
               routing weight of each row
* quant4       E2M1 codes with a power-of-two scale per 32 columns (MX FP4), of
               a tensor or of SiLU(gate) * up, with the values that they stand for
* product4     the product of MX FP4 rows and MX FP4 weights, dense or by
               expert, from codes or from bf16 rows that are quantised first

`own = False` runs the plain forms, `own = True` the package's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32                                    # elements of an MX scale
MAX_FLOPS = 2.0 * 8192 * 4096 * 28672         # of the largest listed case
PLAIN_SUM = 4096                              # largest K of a drawn product in fp32


# ------------------------------------------------------------------ cases --
def _product(name, R, E, K, N, transposed, bias, skew, rest, dtype):
    return dict(name=name, op="product", R=R, E=E, K=K, N=N, transposed=transposed, bias=bias,
                skew=skew, rest=rest, dtype=dtype)


def _weight_grad(name, R, E, K, N, skew, dtype):
    return dict(name=name, op="weight_grad", R=R, E=E, K=K, N=N, skew=skew, rest=0, dtype=dtype)


def _swiglu_grad(name, R, I, weighted):
    return dict(name=name, op="swiglu_grad", R=R, I=I, weighted=weighted)


def _quant4(name, R, K, swiglu):
    return dict(name=name, op="quant4", R=R, K=K, swiglu=swiglu)


def _product4(name, R, E, K, N, skew, quantise, dtype):
    """E = 0: one dense weight."""
    return dict(name=name, op="product4", R=R, E=E, K=K, N=N, skew=skew, rest=0,
                quantise=quantise, dtype=dtype)


def listed():
    return [
        # gate/up product of a tiny layer (64 tokens, 2 of 8 experts): the latency of the call
        _product("product tiny", 128, 8, 256, 1024, False, False, 0.0, 0, "bfloat16"),
        # down product of a decode batch, Mixtral-8x7B shape (16 tokens, 2 of 8): the weights' bytes
        _product("product decode", 32, 8, 14336, 4096, False, True, 0.0, 0, "bfloat16"),
        # gate/up product of a prefill chunk of that shape (4096 tokens): the tensor cores' rate
        _product("product prefill", 8192, 8, 4096, 28672, False, False, 0.0, 0, "bfloat16"),
        # gradient of the gate/up product's input, Qwen-MoE shape, skewed experts, the weight as
        # the forward pass has it; 1001 rows behind the last expert's belong to nobody
        _product("product gradient", 131064, 128, 1536, 2048, True, False, 0.8, 1001, "bfloat16"),
        # gradient of the down weight of a Mixtral-8x7B training step, in fp32 for the optimizer
        _weight_grad("weight gradient", 8192, 8, 14336, 4096, 0.0, "float32"),
        # of the gate/up weight, Qwen-MoE shape: many experts, from few rows to many, odd counts
        _weight_grad("weight gradient skewed", 131064, 128, 2048, 1536, 0.8, "bfloat16"),
        # between the two products' gradients: a small batch, one row per routed token
        _swiglu_grad("swiglu gradient decode", 32, 14336, True),
        # of a Qwen-MoE training step
        _swiglu_grad("swiglu gradient", 131064, 768, True),
        # activations of a small batch, for a 4-bit product and the gradients behind it
        _quant4("quantise decode", 64, 7168, False),
        # between the two products of a prefill chunk: SiLU(gate) * up quantised in one pass
        _quant4("quantise swiglu", 8191, 2048, True),
        # experts of a decode batch (64 tokens, 8 of 256 experts, an eighth of them here),
        # rows in bf16 quantised in the call
        _product4("product4 decode", 64, 32, 7168, 4096, 0.0, True, "bfloat16"),
        # shared expert's gate/up product of a prefill chunk: the 4-bit tensor cores' rate
        _product4("product4 prefill", 8192, 0, 7168, 4096, 0.0, False, "bfloat16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "weight_grad", "weight_grad", "swiglu_grad", "quant4",
                     "product4", "product4"])
    if op == "swiglu_grad":
        I = 8 * _log(rng, 4, 1792)
        c = _swiglu_grad("", _log(rng, 1, min(131072, (1 << 27) // I)), I, rng.random() < 0.7)
    elif op == "quant4":
        K = 32 * _log(rng, 1, 448)
        c = _quant4("", _log(rng, 1, min(32768, (1 << 26) // K)), K, rng.random() < 0.5)
    else:
        E = _log(rng, 1, 128)
        R, skew = _log(rng, 1, 65536), rng.choice([0.0, 0.4, 0.8, 1.2])
        dtype = rng.choice(["bfloat16", "float32"])
        unit = 32 if op == "product4" else 8
        K = unit * _log(rng, 64 // unit, 8192 // unit)
        N = 8 * _log(rng, 8, 1024)
        if op == "product" and dtype == "float32":
            K = min(K, PLAIN_SUM)
        while E * K * N > 1 << 30 or 2.0 * R * K * N > MAX_FLOPS / 4:
            E, R = max(1, E // 2), max(1, R // 2)
        if op == "product":
            c = _product("", R, E, K, N, rng.random() < 0.5, rng.random() < 0.3, skew,
                         rng.choice([0, 0, 1, 77]), dtype)
        elif op == "weight_grad":
            c = _weight_grad("", R, E, K, N, skew, dtype)
        else:
            c = _product4("", R, 0 if rng.random() < 0.4 else E, K, N, skew, rng.random() < 0.4,
                          dtype)
    del c["name"]
    return c


def _touched(R, E):
    """Experts that have rows, of E that R rows choose from evenly."""
    return min(E, E * (1.0 - (1.0 - 1.0 / E) ** R))


def work(case):
    op, R = case["op"], case["R"]
    out = 4 if case.get("dtype") == "float32" else 2
    if op == "swiglu_grad":
        I = case["I"]
        return {"bytes": 10 * R * I + (8 * R if case["weighted"] else 0), "flops": 16.0 * R * I}
    if op == "quant4":
        K = case["K"]
        return {"bytes": (4 if case["swiglu"] else 2) * R * K + R * K / 2 + R * K / BLOCK + 2 * R * K,
                "flops": (8.0 if case["swiglu"] else 2.0) * R * K}
    E, K, N = max(1, case["E"]), case["K"], case["N"]
    if op == "product":
        return {"bytes": 2 * R * K + out * R * N + _touched(R, E) * (2 * K * N + (2 * N if case["bias"] else 0)),
                "flops": 2.0 * R * K * N}
    if op == "weight_grad":
        return {"bytes": 2 * R * (K + N) + out * E * K * N, "flops": 2.0 * R * K * N}
    row = 2.0 * K if case["quantise"] else K / 2 + K / BLOCK
    return {"bytes": R * row + out * R * N + _touched(R, E) * N * (K / 2 + K / BLOCK),
            "flops": 2.0 * R * K * N}


# ----------------------------------------------------------------- inputs --
def _gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 16 + stream)
    return g


def _randn(seed, stream, *shape):
    return torch.randn(*shape, generator=_gen(seed, stream), device=DEV, dtype=torch.float32)


def _bounds(seed, R, E, skew):
    """Where each expert's rows begin, and the end: experts by a Zipf law
    over a seeded ranking, a row's expert drawn from it."""
    g = torch.Generator()
    g.manual_seed(seed * 16 + 9)
    p = (torch.randperm(E, generator=g).double() + 1.0) ** -skew
    counts = torch.bincount(torch.multinomial(p, R, replacement=True, generator=g), minlength=E)
    return [0] + torch.cumsum(counts, 0).tolist()


def _weights(seed, stream, E, rows, cols):
    """bf16 [E, rows, cols], expert by expert (a draw in fp32 is twice its size)."""
    w = torch.empty(E, rows, cols, device=DEV, dtype=torch.bfloat16)
    g = _gen(seed, stream)
    for e in range(E):
        w[e] = 0.02 * torch.randn(rows, cols, generator=g, device=DEV)
    return w


def prepare(case, seed):
    op, R = case["op"], case["R"]
    if op == "swiglu_grad":
        I = case["I"]
        return dict(case=case, gate_up=_randn(seed, 1, R, 2 * I).to(torch.bfloat16),
                    dz=_randn(seed, 2, R, I).to(torch.bfloat16),
                    weights=torch.rand(R, generator=_gen(seed, 3), device=DEV) if case["weighted"] else None,
                    d_gate_up=torch.empty(R, 2 * I, device=DEV, dtype=torch.bfloat16),
                    d_weights=torch.empty(R, device=DEV) if case["weighted"] else None)
    K = case["K"]
    if op == "quant4":
        x = _randn(seed, 1, R, K * (2 if case["swiglu"] else 1)).to(torch.bfloat16)
        return dict(case=case, x=x, q=torch.empty(R, K // 2, device=DEV, dtype=torch.uint8),
                    scale=torch.empty(R, K // BLOCK, device=DEV, dtype=torch.uint8),
                    values=torch.empty(R, K, device=DEV, dtype=torch.bfloat16))
    E, N = case["E"], case["N"]
    bounds = _bounds(seed, R, E, case["skew"]) if E else [0, R]
    s = dict(case=case, bounds=bounds,
             offsets=torch.tensor(bounds, dtype=torch.int32, device=DEV) if E else None)
    x = _randn(seed, 1, R + case["rest"], K).to(torch.bfloat16)
    if op == "weight_grad":
        return dict(s, x=x, dy=_randn(seed, 2, R, N).to(torch.bfloat16),
                    out=torch.empty(E, K, N, device=DEV, dtype=getattr(torch, case["dtype"])))
    s["out"] = torch.zeros(R + case["rest"], N, device=DEV, dtype=getattr(torch, case["dtype"]))
    if op == "product":
        w = _weights(seed, 2, E, N, K) if case["transposed"] else _weights(seed, 2, E, K, N)
        return dict(s, x=x, w=w, bias=_randn(seed, 3, E, N).to(torch.bfloat16) if case["bias"] else None)
    # weights as a checkpoint has them: codes of all values, scales around those of N(0, 0.02)
    w_q = torch.randint(0, 256, (max(1, E), N, K // 2), generator=_gen(seed, 2), device=DEV, dtype=torch.uint8)
    w_s = torch.randint(118, 122, (max(1, E), N, K // BLOCK), generator=_gen(seed, 3), device=DEV, dtype=torch.uint8)
    if not E:
        w_q, w_s = w_q[0], w_s[0]
    s.update(w_q=w_q, w_scale=w_s, x=x,
             q=torch.empty(R, K // 2, device=DEV, dtype=torch.uint8),
             scale=torch.empty(R, K // BLOCK, device=DEV, dtype=torch.uint8))
    if not case["quantise"]:
        s["q"], s["scale"], s["x"] = *_quantise(x.float()), None
    return s


# ------------------------------------------------------------ plain forms --
def _plain_product(s):
    c, b = s["case"], s["bounds"]
    out = torch.zeros(s["x"].shape[0], c["N"], device=DEV, dtype=getattr(torch, c["dtype"]))
    for e in range(c["E"]):
        if b[e + 1] > b[e]:
            w = s["w"][e].float()
            y = s["x"][b[e]:b[e + 1]].float() @ (w.t() if c["transposed"] else w)
            if s["bias"] is not None:
                y = y + s["bias"][e].float()
            out[b[e]:b[e + 1]] = y
    return out


def _plain_weight_grad(s):
    c, b = s["case"], s["bounds"]
    out = torch.empty(c["E"], c["K"], c["N"], device=DEV, dtype=getattr(torch, c["dtype"]))
    for e in range(c["E"]):
        out[e] = s["x"][b[e]:b[e + 1]].float().t() @ s["dy"][b[e]:b[e + 1]].float()
    return out


def _plain_swiglu_grad(s):
    I = s["case"]["I"]
    g, u, dz = s["gate_up"][:, :I].float(), s["gate_up"][:, I:].float(), s["dz"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    dw = None
    if s["weights"] is not None:
        dw = (dz * (g * sig * u)).sum(1)
        dz = dz * s["weights"][:, None]
    d = torch.cat([dz * u * sig * (1.0 + g * (1.0 - sig)), dz * g * sig], 1)
    return [d.to(torch.bfloat16), dw]


def _quantise(z):
    """MX FP4 of z fp32 [M, K]: scale 2^(floor(log2 max|z|) - 2) per 32 columns,
    its exponent stored with a bias of 127; codes of sign and magnitude, nearest
    E2M1 value of z / scale, ties to the even code, at most 6; two to a byte."""
    M, K = z.shape
    amax = z.view(M, -1, BLOCK).abs().amax(2)
    biased = (torch.frexp(amax).exponent + 124).clamp(min=0)      # amax = m 2^e, m in [1/2, 1)
    biased = torch.where(amax > 0, biased, 0)
    v = torch.ldexp(z.view(M, -1, BLOCK), (127 - biased)[:, :, None]).view(M, K)
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
            + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int() + 8 * torch.signbit(v).int())
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8), biased.to(torch.uint8)


def _dequantise(q, scale):
    """fp32 values of codes [..., K/2] with scales [..., K/32]."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    table = torch.cat([table, -table])
    v = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], -1).flatten(-2)
    return torch.ldexp(v.unflatten(-1, (-1, BLOCK)), scale.int()[..., None] - 127).flatten(-2)


def _plain_quant4(s):
    x = s["x"].float()
    if s["case"]["swiglu"]:
        K = s["case"]["K"]
        gate, up = x[:, :K], x[:, K:]
        x = gate / (1.0 + torch.exp(-gate)) * up
    return _dequantise(*_quantise(x)).to(torch.bfloat16)


def _plain_product4(s):
    c, b = s["case"], s["bounds"]
    q, scale = _quantise(s["x"].float()) if c["quantise"] else (s["q"], s["scale"])
    out = torch.zeros(c["R"], c["N"], device=DEV, dtype=getattr(torch, c["dtype"]))
    for e in range(max(1, c["E"])):
        if b[e + 1] > b[e]:
            w_q, w_s = (s["w_q"][e], s["w_scale"][e]) if c["E"] else (s["w_q"], s["w_scale"])
            out[b[e]:b[e + 1]] = _dequantise(q[b[e]:b[e + 1]], scale[b[e]:b[e + 1]]) @ _dequantise(w_q, w_s).t()
    return out


# -------------------------------------------------------------------- run --
def _own(s):
    import mixture_experts_ffn_softmax_gb300 as moe
    c = s["case"]
    if c["op"] == "product":
        return moe.moe_grouped_matmul(s["x"], s["w"], s["offsets"], bias=s["bias"],
                                      transposed=c["transposed"], out=s["out"])
    if c["op"] == "weight_grad":
        return moe.moe_grouped_weight_grad(s["x"], s["dy"], s["offsets"], out=s["out"])
    if c["op"] == "swiglu_grad":
        return list(moe.moe_swiglu_backward(s["dz"], s["gate_up"], s["weights"],
                                            grad_gate_up=s["d_gate_up"], grad_weights=s["d_weights"]))
    if c["op"] == "quant4":
        moe.moe_quant_mx_fp4(s["x"], swiglu=c["swiglu"], q4=s["q"], scale=s["scale"], values=s["values"])
        return s["values"]
    if c["quantise"]:
        moe.moe_quant_mx_fp4(s["x"], q4=s["q"], scale=s["scale"])
    return moe.moe_matmul_fp4(s["q"], s["scale"], s["w_q"], s["w_scale"], s["offsets"], out=s["out"])


def run(state):
    if own:
        return _own(state)
    return {"product": _plain_product, "weight_grad": _plain_weight_grad,
            "swiglu_grad": _plain_swiglu_grad, "quant4": _plain_quant4,
            "product4": _plain_product4}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact --
def _exact_e2m1(v):
    """Nearest E2M1 value, ties to the even mantissa, of |v| < 8, in 64 bits."""
    e = (torch.frexp(v.abs()).exponent.double() - 1.0).clamp(min=0.0)
    step = torch.exp2(e - 1.0)
    return (torch.round(v / step) * step).clamp(-6.0, 6.0)


def _exact_values(z):
    """The values that MX FP4 codes of z, in 64 bits, stand for."""
    out = torch.empty_like(z)
    for k in range(0, z.shape[1], BLOCK):
        part = z[:, k:k + BLOCK]
        top = part.abs().amax(1, keepdim=True)
        e = torch.where(top > 0, torch.floor(torch.log2(top)), -125.0)
        # (the logarithm may round up to a power of two that top is below, or the reverse)
        e = torch.where(torch.exp2(e) > top, e - 1.0, e)
        e = torch.where(torch.exp2(e + 1.0) <= top, e + 1.0, e)
        s = torch.exp2(e.clamp(min=-125.0) - 2.0)
        out[:, k:k + BLOCK] = _exact_e2m1(part / s) * s
    return out


def _exact_codes(q, scale):
    """Codes decoded by their bits, in 64 bits."""
    nibble = torch.stack([q & 15, q >> 4], -1).flatten(-2).long()
    exponent, mantissa = (nibble >> 1) & 3, (nibble & 1).double()
    size = torch.where(exponent > 0, (2.0 + mantissa) * torch.exp2(exponent.double() - 2.0), 0.5 * mantissa)
    value = torch.where(nibble >= 8, -size, size)
    return value * torch.exp2(scale.double() - 127.0).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "swiglu_grad":
        g, u = s["gate_up"].double().chunk(2, 1)
        dz, sig = s["dz"].double(), torch.sigmoid(g)
        dw = None
        if s["weights"] is not None:
            dw = torch.einsum("ri,ri->r", dz, g * sig * u)
            dz = s["weights"].double()[:, None] * dz
        return [torch.cat([dz * u * (sig + g * sig * torch.sigmoid(-g)), dz * (g * sig)], 1), dw]
    if op == "quant4":
        z = s["x"].double()
        if case["swiglu"]:
            gate, up = z.chunk(2, 1)
            z = gate * torch.sigmoid(gate) * up
        return _exact_values(z)
    b = s["bounds"]
    if op == "weight_grad":
        return torch.stack([torch.einsum("rk,rn->kn", s["x"][i:j].double(), s["dy"][i:j].double())
                            for i, j in zip(b, b[1:])])
    y = torch.zeros(case["R"] + case["rest"], case["N"], dtype=torch.float64, device=DEV)
    for e, (i, j) in enumerate(zip(b, b[1:])):
        if op == "product":
            x, w = s["x"][i:j].double(), s["w"][e].double()
            w = w if case["transposed"] else w.t()
        else:
            x = _exact_values(s["x"][i:j].double()) if case["quantise"] else _exact_codes(s["q"][i:j], s["scale"][i:j])
            w = _exact_codes(s["w_q"], s["w_scale"]) if not case["E"] else _exact_codes(s["w_q"][e], s["w_scale"][e])
        y[i:j] = torch.einsum("rk,nk->rn", x, w)
        if op == "product" and s["bias"] is not None:
            y[i:j] += s["bias"][e].double()
    return y
