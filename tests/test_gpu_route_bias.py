"""GPU parity of the routing with a bias (ids equal to the 64-bit oracle's,
weights within fp32 rounding) and of the routing gradient."""
import pathlib
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import mixture_experts_ffn_softmax_gb300 as pkg
import oracle
from mixture_experts_ffn_softmax_gb300 import workloads as wl

from helpers import check_out

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24     # half a step of fp32, relative


def weight_rtol(logits, E):
    """Relative error of a weight: expf within 2 U32 of its argument's value
    and its argument l - max rounded (|l - max| U32), twice (numerator and
    sum); the sums of at most E / 32 + 5 positive terms per path; the
    division, the scale and the reciprocal forms, 8 roundings at most."""
    fin = np.where(np.abs(logits) < 1e30, logits, 0.0)   # masked ones take no part
    return (2 * (2 + np.abs(fin).max() * 2) + E / 32 + 6 + 8) * U32


def check_biased(logits, bias, a):
    w, ids = pkg.moe_route(logits, a["k"], a["method"], a["renorm"], a["kg"], a["G"], a["mode"],
                           a["scale"], score_bias=bias)
    torch.cuda.synchronize()
    l = logits.double().cpu().numpy()
    rw, rids = oracle.route_biased(l, bias.double().cpu().numpy(), a["k"], a["method"],
                                   a["renorm"], a["kg"], a["G"], a["mode"], a["scale"])
    assert np.array_equal(ids.cpu().numpy(), rids)
    err = np.abs(w.cpu().double().numpy() - rw)
    # 1e-44: weights below the smallest fp32 numbers
    assert (err <= weight_rtol(l, l.shape[1]) * np.abs(rw) + 1e-44).all(), err.max()
    return w, ids


def args(k=2, method="softmax", renorm=False, kg=1, G=1, mode=0, scale=1.0):
    return dict(k=k, method=method, renorm=renorm, kg=kg, G=G, mode=mode, scale=scale)


CASES = [
    # (M, E, args)
    (1, 1, args(1)),
    (3, 3, args(2, "sigmoid", scale=2.5)),
    (5, 7, args(7, "softmax", True)),
    (1, 8, args(2, "softmax", True)),
    (129, 8, args(2, "softmax", True)),
    (33, 16, args(4, "sigmoid")),
    (65, 24, args(3, "softmax", False, 2, 3, 1)),
    (31, 32, args(8, "softmax", False, 3, 4, 1, 0.5)),
    (17, 33, args(5, "sigmoid")),
    (40, 60, args(6, "sigmoid", True, 2, 5, 1)),
    (64, 64, args(64, "softmax", True)),
    (64, 64, args(33, "sigmoid")),
    (37, 96, args(6, "softmax", True, 2, 3)),
    (50, 128, args(8, "softmax", False)),
    (51, 128, args(8, "sigmoid", True, 4, 16, 1)),
    (70, 160, args(7, "sigmoid", False, 3, 5, 1, 2.5)),
    (1, 256, args(8, "sigmoid", True, 4, 8, 1, 2.5)),
    (300, 256, args(8, "sigmoid", True, 4, 8, 1, 2.5)),
    (300, 256, args(8, "softmax", True, 4, 8, 0, 2.5)),
    (40, 256, args(16, "sigmoid", True, 1, 16, 0)),
    (21, 384, args(6, "sigmoid", True, 1, 1, 0)),
    (20, 512, args(16, "sigmoid", True, 2, 64, 1)),
    (20, 512, args(64, "softmax", False, 128, 256, 1)),
    (9, 1000, args(20, "softmax", True, 4, 10, 1)),
    (9, 1024, args(33, "softmax", True)),
    (9, 1024, args(8, "sigmoid", False, 5, 16, 0, 3.0)),
    (7, 1024, args(64, "sigmoid", False, 512, 1024, 0)),
]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,E,a", CASES)
def test_route_biased(M, E, a, dtype):
    g = torch.Generator(device="cuda").manual_seed(M * 1031 + E)
    logits = torch.randn(M, E, generator=g, device="cuda").to(getattr(torch, dtype))
    bias = torch.randn(E, generator=g, device="cuda") * (0.1 if a["method"] == "sigmoid" else
                                                         1.0 / E)
    check_biased(logits, bias, a)


@pytest.mark.parametrize("method,spread", [("sigmoid", 0.02), ("softmax", 0.0005)])
def test_route_biased_many_tokens(method, spread):
    """Enough tokens that neighbouring scores closer than fp32 rounding occur
    by chance."""
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randn(4096, 256, generator=g, device="cuda")
    bias = torch.randn(256, generator=g, device="cuda") * spread
    check_biased(logits, bias, args(8, method, True, 4, 8, 1, 2.5))


@pytest.mark.parametrize("method", ["sigmoid", "softmax"])
@pytest.mark.parametrize("kg,G,mode", [(1, 1, 0), (2, 4, 1), (3, 8, 0)])
def test_route_biased_ties_and_near_ties(method, kg, G, mode):
    """Exact ties (equal logits and biases), ties of the fp32 scores whose
    64-bit values differ, and saturated scores that agree in 64 bits too."""
    E, k = 64, 8
    rng = np.random.default_rng(3)
    rows = [np.zeros(E), rng.integers(-1, 2, E).astype(float),
            1.0 + rng.integers(0, 4, E) * 2.0 ** -23,         # neighbouring fp32 logits
            rng.permutation(E) * 2.0 ** -22 + 2.0,
            20.0 + rng.integers(0, 3, E),                     # sigmoid rounds to 1 in fp32
            50.0 + rng.integers(0, 3, E),                     # and in 64 bits
            -rng.integers(90, 120, E).astype(float), -700.0 - rng.integers(0, 40, E)]
    logits = torch.tensor(np.stack(rows * 3), dtype=torch.float32, device="cuda")
    for bias in (np.zeros(E), rng.integers(0, 2, E) * 0.5, rng.integers(0, 2, E) * 2.0 ** -25):
        b = torch.tensor(bias, dtype=torch.float32, device="cuda")
        check_biased(logits, b, args(k, method, True, kg, G, mode))
        if method == "softmax":
            check_biased(logits, b, args(k, method, False, kg, G, mode))


@pytest.mark.parametrize("E,kg,G,mode", [(16, 1, 1, 0), (64, 2, 4, 1), (256, 4, 8, 1), (96, 1, 3, 0)])
@pytest.mark.parametrize("method,renorm", [("sigmoid", True), ("softmax", True), ("softmax", False)])
def test_route_biased_masked_experts(E, kg, G, mode, method, renorm):
    """Masked experts (-inf, and the type's lowest value) in all numbers up to
    every expert of the row, with biases that would otherwise choose them."""
    rng = np.random.default_rng(E)
    k = 6
    logits = rng.normal(size=(40, E)).astype(np.float32)
    for t in range(40):
        out = rng.permutation(E)[:[0, E // 2, E - 7, E - 2, E][t % 5]]
        logits[t, out] = -np.inf if t % 2 else np.finfo(np.float32).min
    logits[38] = -np.inf
    bias = torch.tensor(rng.normal(size=E), dtype=torch.float32, device="cuda")
    check_biased(torch.tensor(logits, device="cuda"), bias, args(k, method, renorm, kg, G, mode))


@pytest.mark.parametrize("E,k,G,kg", [(1, 1, 1, 1), (8, 8, 1, 1), (14, 14, 1, 1), (30, 30, 1, 1),
                                      (64, 14, 8, 2), (32, 8, 4, 1), (64, 64, 1, 1)])
@pytest.mark.parametrize("method,renorm", [("sigmoid", True), ("softmax", True), ("softmax", False)])
def test_route_biased_masked_rows_that_choose_every_expert(E, k, G, kg, method, renorm):
    """Every expert (of the kept groups) is chosen, so that nothing is left to
    compare the last one with: none, some or all of them masked."""
    rng = np.random.default_rng(E + k)
    logits = rng.normal(size=(12, E)).astype(np.float32)
    for t in range(12):
        logits[t, rng.permutation(E)[:[0, E // 2, E - 1, E][t % 4]]] = -np.inf
    for bias in (np.zeros(E), rng.normal(size=E)):
        bias = torch.tensor(bias, dtype=torch.float32, device="cuda")
        check_biased(torch.tensor(logits, device="cuda"), bias,
                     args(k, method, renorm, kg, G, 0))


@pytest.mark.parametrize("E,k,G,kg", [(256, 8, 1, 1), (256, 8, 8, 4), (128, 5, 1, 1), (512, 8, 1, 1),
                                      (1024, 3, 1, 1)])
@pytest.mark.parametrize("method", ["sigmoid", "softmax"])
def test_route_biased_scores_in_falling_order_a_few_roundings_apart(E, k, G, kg, method):
    """Scores that rise with the expert's number (against the order of ties) in
    steps from a tenth of an fp32 rounding to thousands of them."""
    M = 96
    step = 2.0 ** np.linspace(-27, -13, M)[:, None]
    rng = np.random.default_rng(E + k)
    jitter = 1 + 0.5 * rng.random((M, E))
    logits = (step * np.cumsum(jitter, 1)).astype(np.float32)
    bias = torch.zeros(E, device="cuda")
    for l in (logits, logits[:, ::-1].copy(), logits[:, rng.permutation(E)].copy()):
        check_biased(torch.tensor(l, device="cuda"), bias, args(k, method, True, kg, G, 0))


@pytest.mark.parametrize("E,k,G,kg,mode", [(256, 8, 8, 4, 1), (256, 14, 1, 1, 0), (128, 8, 1, 1, 0),
                                           (160, 6, 5, 2, 1), (66, 5, 1, 1, 0), (192, 8, 16, 3, 0)])
@pytest.mark.parametrize("method,renorm", [("sigmoid", True), ("softmax", True), ("softmax", False)])
def test_route_biased_many_and_few_tokens(E, k, G, kg, mode, method, renorm):
    """More tokens than a whole warp each is used for: normal rows, masked
    ones, scores a few roundings apart; the same ids in parts of fewer tokens."""
    M = 4097 + 72
    rng = np.random.default_rng(E + k)
    logits = rng.normal(size=(M, E)).astype(np.float32)
    for t in range(64):
        logits[t, rng.permutation(E)[:[1, E // 2, E - 3, E][t % 4]]] = -np.inf
    step = 2.0 ** np.linspace(-27, -13, 256)[:, None]
    logits[100:356] = (step * np.cumsum(1 + 0.5 * rng.random((256, E)), 1)).astype(np.float32)
    logits[400:500] = np.round(logits[400:500] * 4) / 4               # ties
    logits = torch.tensor(logits, device="cuda")
    for spread in (0.0, 0.3):
        bias = torch.tensor(rng.normal(size=E) * spread, dtype=torch.float32, device="cuda")
        a = args(k, method, renorm, kg, G, mode, 2.5)
        w, ids = check_biased(logits, bias, a)
        pos = (a["k"], a["method"], a["renorm"], a["kg"], a["G"], a["mode"], a["scale"])
        for part in (slice(0, 4096), slice(4096, M)):
            assert torch.equal(pkg.moe_route(logits[part], *pos, score_bias=bias)[1], ids[part])


@pytest.mark.parametrize("E,k,G,kg,mode", [(336, 13, 8, 4, 0), (336, 13, 8, 4, 1), (463, 10, 1, 1, 0), (384, 8, 8, 4, 1),
                                           (510, 30, 17, 9, 1), (162, 14, 6, 2, 1), (162, 5, 27, 9, 0), (1000, 8, 4, 2, 1)])
@pytest.mark.parametrize("method,renorm", [("sigmoid", True), ("softmax", False)])
def test_route_biased_near_groups_and_candidates(E, k, G, kg, mode, method, renorm):
    """Group sizes that are no powers of two and rows of odd lengths, with scores
    a few roundings apart in the whole row, in one group, and between groups."""
    rng = np.random.default_rng(E * 3 + k)
    M = 120
    logits = rng.normal(size=(M, E))
    step = 2.0 ** np.linspace(-27, -14, 40)[:, None]
    logits[:40] = step * rng.permutation(E)[None] * (1 + rng.random((40, E)) / 8)
    best = 2.5 + step * rng.random((40, G))                 # every group's best within a step
    for g in range(G):
        logits[40:80, g * (E // G) + 1] = best[:, g]
    for dt in (torch.float32, torch.bfloat16):
        l = torch.tensor(logits, device="cuda").to(dt)
        for spread in (0.0, 0.2):
            bias = torch.tensor(rng.normal(size=E) * spread, dtype=torch.float32, device="cuda")
            check_biased(l, bias, args(k, method, renorm, kg, G, mode))


@pytest.mark.parametrize("E,k,G,kg,mode", [(256, 8, 8, 4, 1), (256, 8, 1, 1, 0), (100, 6, 1, 1, 0), (336, 9, 8, 2, 0)])
@pytest.mark.parametrize("M", [50, 4200])
def test_route_biased_fewer_experts_left_than_chosen(E, k, G, kg, mode, M):
    """Rows with 0 to k + 2 unmasked experts, and biases of -inf and of the
    type's largest numbers beside the masks."""
    rng = np.random.default_rng(M + E)
    logits = rng.normal(size=(M, E)).astype(np.float32)
    for t in range(M):
        logits[t, rng.permutation(E)[t % (k + 3):]] = -np.inf
    bias = rng.normal(size=E).astype(np.float32)
    for special in ((), (-np.inf,), (3e38, -3e38)):
        for i, v in enumerate(special):
            bias[i::7] = v
        check_biased(torch.tensor(logits, device="cuda"), torch.tensor(bias, device="cuda"),
                     args(k, "sigmoid", True, kg, G, mode))


@pytest.mark.parametrize("method", ["sigmoid", "softmax"])
def test_route_biased_non_finite_scores(method):
    """Whatever the logits hold, ids are valid and distinct; other tokens keep
    their results; a NaN is chosen last."""
    E, k = 64, 8
    g = torch.Generator(device="cuda").manual_seed(9)
    logits = torch.randn(12, E, generator=g, device="cuda")
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    w0, i0 = pkg.moe_route(logits, k, method, True, 2, 4, 1, score_bias=bias)
    bad = logits.clone()
    bad[1, 5] = float("nan")
    bad[3] = float("nan")
    bad[5, 60] = float("inf")
    bad[7] = float("inf")
    w, ids = pkg.moe_route(bad, k, method, True, 2, 4, 1, score_bias=bias)
    for t in range(12):
        r = ids[t].tolist()
        assert len(set(r)) == k and all(0 <= e < E for e in r)
        if t not in (1, 3, 5, 7):
            assert torch.equal(w[t], w0[t]) and torch.equal(ids[t], i0[t])
    if method == "sigmoid":
        assert 5 not in ids[1].tolist() and torch.isfinite(w[1]).all()
        assert torch.isnan(w[3]).all()
        assert torch.isfinite(w[5]).all() and torch.isfinite(w[7]).all()
    else:
        assert torch.isnan(w[[1, 3, 5, 7]]).any(1).all()


def test_route_biased_empty_and_untouched_rows():
    bias = torch.zeros(16, device="cuda")
    w, ids = pkg.moe_route(torch.zeros(0, 16, device="cuda"), 4, score_bias=bias)
    assert w.shape == (0, 4) and ids.shape == (0, 4)
    # views of a larger buffer (element-aligned only): the rows around stay
    for M, E, k in ((3, 15, 3), (5, 33, 5), (2, 256, 7)):
        for dt in (torch.float32, torch.bfloat16):
            buf = torch.randn((M + 2) * E + 1, device="cuda").to(dt)
            logits = buf[E + 1:E + 1 + M * E].view(M, E)
            W = torch.full(((M + 2) * k,), -5.0, device="cuda")
            I = torch.full(((M + 2) * k,), -5, dtype=torch.int32, device="cuda")
            b = torch.randn(E + 1, device="cuda")[1:] * 0.1
            pkg.moe_route(logits, k, "sigmoid", topk_weights=W[k:k + M * k].view(M, k),
                          topk_ids=I[k:k + M * k].view(M, k), score_bias=b)
            w, ids = check_biased(logits.contiguous().clone(), b.clone(), args(k, "sigmoid"))
            assert torch.equal(W[k:-k].view(M, k), w) and torch.equal(I[k:-k].view(M, k), ids)
            assert (W[:k] == -5).all() and (W[-k:] == -5).all()
            assert (I[:k] == -5).all() and (I[-k:] == -5).all()


def test_route_biased_zero_bias_is_the_plain_route():
    spec = wl.SMALL_SPECS["deepseek_small"]
    d = wl.make_moe_inputs(spec, device="cuda", weights=False)
    a = (spec.top_k, spec.routing_method, spec.renormalize, spec.k_group, spec.group_count,
         spec.group_select_mode, spec.routed_scaling_factor)
    w0, i0 = pkg.moe_route(d["router_logits"], *a)
    w, i = pkg.moe_route(d["router_logits"], *a,
                         score_bias=torch.zeros(spec.E, device="cuda"))
    assert torch.equal(i, i0)
    assert (w - w0).abs().max() <= 1e-5


def shift_free_rtol(l, ids):
    """Relative error of softmax weights, from each logit's distance to the
    row's largest alone.  Numerator: the distance rounded (|l - max| U32) and
    expf (2).  Sum: 4 for a term's exponential and 2.25 |l - max| for its
    argument (difference and product rounded, the constant's own error), as
    the terms weigh, and the additions of positive terms, one each: at most
    E / 16 in a lane and 5 across them.  Division and scale 2."""
    d = l.max(1, keepdims=True) - l
    p = np.exp(-d)
    p /= p.sum(1, keepdims=True)
    d_mean = (p * d).sum(1, keepdims=True)
    return (np.take_along_axis(d, ids, 1) + 2 + 4 + 2.25 * d_mean + -(-l.shape[1] // 16) + 5 + 2) * U32


@pytest.mark.parametrize("E,k,G,kg,M", [(8, 2, 1, 1, 40), (128, 8, 1, 1, 4200), (256, 8, 8, 4, 40),
                                        (256, 14, 1, 1, 4200), (336, 9, 8, 4, 40), (1000, 8, 1, 1, 20),
                                        (256, 40, 1, 1, 20)])
@pytest.mark.parametrize("dtype,step,shifts", [("float32", 2.0 ** -4, (100.0, -1000.0, 1e4, 2.0 ** 19)),
                                               ("bfloat16", 0.5, (120.0, -120.0))])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_biased_softmax_does_not_see_a_shift(E, k, G, kg, M, dtype, step, shifts, renorm):
    """All logits of a call moved by a number that fp32 adds exactly: the same
    ids and weights, and those within what the distances between logits give."""
    rng = np.random.default_rng(E + M)
    base = np.clip(np.round(rng.normal(size=(M, E)) * 2 / step) * step, -6, 6)
    bias = torch.tensor(rng.normal(size=E) / E, dtype=torch.float32, device="cuda")
    a = (k, "softmax", renorm, kg, G, 0, 2.5)
    dt = getattr(torch, dtype)
    w0, i0 = pkg.moe_route(torch.tensor(base, device="cuda").to(dt), *a, score_bias=bias)
    rw, rids = oracle.route_biased(base, bias.double().cpu().numpy(), *a)
    assert np.array_equal(i0.cpu().numpy(), rids)
    rtol = shift_free_rtol(base, rids)
    for shift in (0.0,) + shifts:
        l = torch.tensor(base + shift, device="cuda").to(dt)
        assert np.array_equal(l.double().cpu().numpy(), base + shift)
        w, ids = pkg.moe_route(l, *a, score_bias=bias)
        assert torch.equal(ids, i0)
        err = np.abs(w.double().cpu().numpy() - rw)
        assert (err <= rtol * rw).all(), (shift, (err / rw).max())
        assert torch.equal(w, w0)


def test_route_biased_softmax_choice_with_large_logits():
    """Logits around 1e8 and 1e9, some equal and the others far below, and
    biases that bring the equal ones' c to the others' within 2^-25 of a
    score: what fp32 says of the order is less than its error."""
    E, n, k = 64, 27, 40
    for part in range(60):
        rng = np.random.default_rng(part)
        base = np.concatenate([rng.integers(1 << 23, 1 << 24, 8) * 8.0,
                               rng.integers(1 << 23, 1 << 24, 8) * 64.0])
        l = np.repeat(base[:, None], E, 1)
        l[:, n:] -= 8192.0
        top = np.float32(-1.0 / n)
        bias = np.full(E, top, dtype=np.float32)
        for e in range(n):
            bias[e] = np.float32(top + rng.integers(0, 3) * 2.0 ** -28)
        c = 1.0 / n + bias[:n].astype(np.float64)
        bias[n:] = c[rng.integers(0, n, E - n)] + rng.uniform(-2e-9, 2e-9, E - n)
        logits = torch.tensor(l, dtype=torch.float32, device="cuda")
        assert np.array_equal(logits.double().cpu().numpy(), l)
        for kk in (8, 28, k):
            _, ids = pkg.moe_route(logits, kk, "softmax", True,
                                   score_bias=torch.tensor(bias, device="cuda"))
            _, rids = oracle.route_biased(l, bias.astype(np.float64), kk, "softmax", True)
            assert np.array_equal(ids.cpu().numpy(), rids), (part, kk)


def biased_ids(logits, bias, k, method, kg, G, mode):
    """The choice in 64 bits, by torch for many tokens (distinct c)."""
    l = logits.double()
    p = torch.softmax(l, 1) if method == "softmax" else torch.sigmoid(l)
    c = p + bias.double()
    M, E = c.shape
    top = c.view(M, G, E // G).sort(dim=2, descending=True).values
    score = top[:, :, 0] + top[:, :, 1] if mode else top[:, :, 0]
    kept = score.sort(dim=1, descending=True, stable=True).indices[:, :kg]
    keep = torch.zeros(M, G, dtype=torch.bool, device=c.device).scatter_(1, kept, True)
    c = c.masked_fill(~keep.repeat_interleave(E // G, 1), -np.inf)
    return c.sort(dim=1, descending=True, stable=True).indices[:, :k].int()


@pytest.mark.parametrize("B", [4.0, 16.0, 64.0, 1000.0])
@pytest.mark.parametrize("E,G,kg,k,M", [(16, 8, 4, 4, 400000), (256, 32, 16, 8, 100000),
                                        (256, 8, 4, 8, 100000), (336, 8, 4, 8, 60000),
                                        (512, 16, 8, 8, 50000), (1024, 32, 16, 8, 30000),
                                        (256, 128, 64, 8, 2000)])
@pytest.mark.parametrize("method", ["softmax", "sigmoid"])
def test_route_biased_groups_with_biases_of_both_signs(E, G, kg, k, M, B, method):
    """Group scores that are small sums of large c of both signs: their
    rounding is the summands'."""
    g = torch.Generator(device="cuda").manual_seed(int(B) + E + G)
    logits = torch.randn(M, E, generator=g, device="cuda")
    bias = torch.full((G, E // G), -B, device="cuda")
    bias[:, 0] = B
    bias = (bias + torch.randn(G, E // G, generator=g, device="cuda") * 1e-3).view(E)
    for part in logits.split(50000):
        ids = pkg.moe_route(part, k, method, True, kg, G, 1, score_bias=bias)[1]
        assert torch.equal(ids, biased_ids(part, bias, k, method, kg, G, 1))
    few = logits[:300]                              # (a whole warp per token)
    assert torch.equal(pkg.moe_route(few, k, method, True, kg, G, 1, score_bias=bias)[1],
                       biased_ids(few, bias, k, method, kg, G, 1))


@pytest.mark.parametrize("E,G,kg,k", [(64, 4, 2, 4), (256, 8, 4, 8), (336, 8, 4, 8), (512, 16, 8, 8),
                                      (160, 5, 2, 6), (1024, 16, 4, 8)])
@pytest.mark.parametrize("method", ["softmax", "sigmoid"])
def test_route_biased_groups_whose_second_experts_are_large_and_near(E, G, kg, k, method):
    """Groups alike but for a few roundings, each with one expert of a small c
    and the others near -80 or -1000, where fp32 cannot order those others:
    their biases differ by steps of fp32, their scores by as much."""
    M, gs = 20000, E // G
    g = torch.Generator(device="cuda").manual_seed(E)
    for B, step in ((80.0, 2.0 ** -17), (1000.0, 2.0 ** -14)):
        bias = -B + step * torch.randint(0, 5, (G, gs), generator=g, device="cuda").float()
        # (not 0: two groups with the same pair of scores would be a tie of real
        # numbers that 64 bits break by their rounding)
        bias[:, 3] = 1e-6 * torch.randn(G, generator=g, device="cuda")
        bias = bias.view(E)
        for steps in (1, 4, 16):
            spread = steps * step * (E / 2 if method == "softmax" else 4)
            row = torch.randn(M, 1, generator=g, device="cuda")
            logits = row + spread * torch.randn(M, E, generator=g, device="cuda")
            for part in (logits, logits[:500]):
                ids = pkg.moe_route(part, k, method, True, kg, G, 1, score_bias=bias)[1]
                ref = biased_ids(part, bias, k, method, kg, G, 1)
                assert torch.equal(ids, ref), (B, steps)


@pytest.mark.parametrize("E,G,kg", [(64, 4, 1), (60, 4, 1), (256, 8, 1), (336, 8, 1), (512, 16, 1)])
def test_route_biased_second_experts_on_both_sides_of_a_rounding(E, G, kg):
    """Two groups, each with one expert of a small c and two near -80 that are
    apart by less than the error of their scores but rounded apart by a whole
    step of fp32 at -80: the step says nothing of their order."""
    M, gs, k, step = 40000, E // G, 2, 2.0 ** -17
    rng = np.random.default_rng(E)
    bias = np.full((G, gs), -1000.0)
    logits = rng.normal(size=(M, G, gs)) * 0.1
    for grp in range(2):
        bias[grp, 0] = 0.0
        logits[:, grp, 0] = 0.25
        for e, p in ((1, 0.5 + step / 2), (2, 0.875 + step / 2)):
            bias[grp, e] = -80.0 - (p - 0.5 - step / 2)            # (c near -79.5 + step / 2)
            exact = p + rng.uniform(-1e-7, 1e-7, M)
            logits[:, grp, e] = np.log(exact / (1 - exact))
    logits = torch.tensor(logits.reshape(M, E), dtype=torch.float32, device="cuda")
    bias = torch.tensor(bias.reshape(E), dtype=torch.float32, device="cuda")
    for part in (logits, logits[:4000]):
        ids = pkg.moe_route(part, k, "sigmoid", True, kg, G, 1, score_bias=bias)[1]
        assert torch.equal(ids, biased_ids(part, bias, k, "sigmoid", kg, G, 1))


@pytest.mark.parametrize("E,k", [(14, 14), (30, 30), (64, 64)])
@pytest.mark.parametrize("top", [80.0, 1.0, -1.0, -17.0, -40.0, -59.0, -60.5, -87.0, -89.0, -300.0])
def test_route_biased_sigmoid_weights_of_far_logits(E, k, top):
    """Chosen experts whose scores are tiny, underflow in fp32, or lie on both
    sides of that: their weights are ratios of the exact scores."""
    rng = np.random.default_rng(k)
    l = np.float32(top - rng.uniform(0, 85, (32, E)))
    l[:, 0] = top
    l[1:4, 1:] = top - np.float32([0.5, 30.0, 80.0])[:, None]
    logits = torch.tensor(l, device="cuda")
    bias = torch.tensor(rng.normal(size=E), dtype=torch.float32, device="cuda")
    w, _ = check_biased(logits, bias, args(k, "sigmoid", scale=2.5))
    assert (w > 0).all()


@pytest.mark.parametrize("E,G,kg,mode", [(256, 8, 4, 1), (256, 8, 4, 0), (336, 8, 4, 1), (128, 4, 2, 1)])
@pytest.mark.parametrize("method", ["sigmoid", "softmax"])
def test_route_biased_masked_groups(E, G, kg, mode, method):
    """Whole groups masked, or (mode 1) all but one of a group's experts: up to
    as many as are dropped, and more, so that some of them are kept."""
    k, gs = 4, E // G
    rng = np.random.default_rng(E + mode)
    logits = rng.normal(size=(300, E)).astype(np.float32)
    for t in range(300):
        for g in rng.permutation(G)[:t % (G + 1)]:
            left = rng.integers(0, 2) if t % 2 else 0
            logits[t, g * gs + left:(g + 1) * gs] = -np.inf
    for spread in (0.0, 0.3):
        bias = torch.tensor(rng.normal(size=E) * spread, dtype=torch.float32, device="cuda")
        check_biased(torch.tensor(logits, device="cuda"), bias, args(k, method, True, kg, G, mode))
    # biases whose sums overflow in fp32 and not in 64 bits, beside masked groups
    big = np.where(np.arange(E) // gs % 3 == 0, -3e38, 0.0) + rng.normal(size=E) * 0.3
    check_biased(torch.tensor(logits, device="cuda"),
                 torch.tensor(big, dtype=torch.float32, device="cuda"),
                 args(k, method, True, kg, G, mode))


def test_route_biased_masked_groups_stay_on_the_fast_path():
    """Rows with masked groups (no -inf is near a finite score, and -inf ties
    are settled by the index) take about the time of rows without: the 64-bit
    choice of every token is 25 times that, the limit 4 times."""
    M, E = 8192, 256
    a = (8, "sigmoid", True, 4, 8, 1, 2.5)
    logits = torch.randn(M, E, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    bias = torch.randn(E, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") * 0.05
    masked = logits.clone()
    masked[:, 64:128] = float("-inf")
    w, ids = torch.empty(M, 8, device="cuda"), torch.empty(M, 8, dtype=torch.int32, device="cuda")

    def best(l):
        times = []
        for _ in range(10):
            t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            t0.record()
            for _ in range(20):
                pkg.moe_route(l, *a, w, ids, score_bias=bias)
            t1.record()
            t1.synchronize()
            times.append(t0.elapsed_time(t1))
        return min(times)
    plain = best(logits)
    assert best(masked) < 4 * plain


@pytest.mark.parametrize("E,k,G,kg,mode,M", [(16, 13, 8, 7, 0, 400), (64, 8, 1, 1, 0, 400), (256, 1, 1, 1, 0, 400),
                                             (24, 9, 8, 3, 0, 400), (256, 8, 8, 4, 1, 400), (256, 8, 8, 4, 0, 4200),
                                             (60, 8, 5, 3, 1, 400), (128, 8, 8, 3, 1, 4200), (336, 9, 8, 4, 1, 300)])
@pytest.mark.parametrize("spread", [8.0, 30.0])
def test_route_biased_near_certain_softmax_and_biases_in_steps(E, k, G, kg, mode, M, spread):
    """Rows whose largest score is 1 but for 1e-5 to 1e-60, and biases in steps of
    a half: 1 - 1e-9 - 0.5 against 0.5 + 1e-40, which an fp32 sum of the exponentials
    calls equal."""
    for seed in range(3):
        rng = np.random.default_rng(seed + E)
        logits = rng.normal(size=(M, E)) * spread
        bias = torch.tensor(np.round(rng.normal(size=E) * 2) / 2, dtype=torch.float32, device="cuda")
        for dt in (torch.float32, torch.bfloat16):
            l = torch.tensor(logits, device="cuda").to(dt)
            # 64 bits define the sum of a row, and with it a score near 1, up to the order
            # of E additions, 1e-13 at most: left out are rows that such an error could
            # change.  Nothing does where all else vanishes beside 1, nor where the largest
            # score lacks more of 1 than the error (the other c are steps of a half plus
            # what they hold of the lack), unless its group's second makes up for it.
            x = l.double().cpu().numpy()
            ex = np.exp(x - x.max(1, keepdims=True))
            rows, best = np.arange(M), x.argmax(1)
            ex[rows, best] = 0.0
            lack = ex.sum(1)
            ex[rows, best] = 1.0
            c = ex / ex.sum(1, keepdims=True) + bias.double().cpu().numpy()
            two = np.sort(c.reshape(M, G, -1), 2)[:, :, -2:].sum(2)
            d = np.abs(two - two[rows, best // (E // G)][:, None])
            d[rows, best // (E // G)] = 1.0
            fine = (lack < 1e-17) | ((lack > 1e-12) & (d > 1e-13).all(1))
            assert fine.sum() > M // 5
            check_biased(l[torch.tensor(fine, device="cuda")], bias, args(k, "softmax", True, kg, G, mode))


@pytest.mark.parametrize("E,k,G,kg,mode", [(80, 14, 5, 5, 0), (160, 14, 5, 3, 0), (128, 4, 8, 7, 1), (200, 14, 2, 2, 0),
                                           (256, 14, 16, 11, 1), (32, 4, 1, 1, 0)])
@pytest.mark.parametrize("method", ["sigmoid", "softmax"])
def test_route_biased_tokens_do_not_see_their_neighbours(E, k, G, kg, mode, method):
    """Two tokens share a warp: one with non-finite scores, or with near ones that
    take further rounds, leaves the other's ids and weights as they are, to the bit."""
    M = 4500
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(M, E, generator=g, device="cuda")
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    a = (k, method, True, kg, G, mode)
    w0, i0 = pkg.moe_route(logits, *a, score_bias=bias)
    rows = torch.arange(M, device="cuda") % 2 == 0
    for other in (torch.full_like(logits, float("nan")), torch.zeros_like(logits), logits * 2.0 ** -22,
                  torch.where(torch.rand(M, E, generator=g, device="cuda") < 0.02, float("inf"), logits)):
        for hit in (rows, ~rows):
            w, ids = pkg.moe_route(torch.where(hit[:, None], other, logits), *a, score_bias=bias)
            assert torch.equal(ids[~hit], i0[~hit]) and torch.equal(w[~hit], w0[~hit])


# ------------------------------------------------------------- gradient --
BACK = [(1, 1, 1), (3, 8, 2), (130, 8, 8), (33, 17, 5), (64, 64, 33), (65, 128, 8), (257, 256, 8),
        (31, 384, 6), (9, 1000, 64), (5, 1024, 16)]


def check_backward(gw, logits, ids, method, renorm, scale):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = pkg.moe_route_backward(gw, logits, ids, method, renorm, scale, error_word=err)
    torch.cuda.synchronize()
    assert got.dtype == logits.dtype and err.item() == 0
    l = logits.double().cpu().numpy()
    ref = oracle.route_backward(gw.double().cpu().numpy(), l, ids.cpu().numpy(), method, renorm,
                                scale)
    # one rounding of the result; before it, terms of at most
    # scale * max|gw| * (1 + k) with the relative error of a weight each
    out = (2.0 ** -8 if logits.dtype == torch.bfloat16 else U32)
    size = scale * gw.abs().max().item() * (1 + ids.shape[1])
    tol = out * np.abs(ref) + 2 * weight_rtol(l, l.shape[1]) * size
    diff = np.abs(got.double().cpu().numpy() - ref)
    assert (diff <= tol).all(), (diff - tol).max()
    return got, ref


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("method,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("M,E,k", BACK)
def test_route_backward(M, E, k, method, renorm, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + E)
    logits = torch.randn(M, E, generator=g, device="cuda").to(getattr(torch, dtype))
    ids = torch.argsort(torch.rand(M, E, generator=g, device="cuda"), 1)[:, :k].int().contiguous()
    gw = torch.randn(M, k, generator=g, device="cuda")
    got, ref = check_backward(gw, logits, ids, method, renorm, 1.5)
    if dtype == "float32" and k > 1:
        # and as a whole, to the accuracy of its terms
        n = np.linalg.norm(ref)
        assert np.linalg.norm(got.double().cpu().numpy() - ref) <= 1e-5 * max(n, 1e-30)


@pytest.mark.parametrize("method,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
def test_route_backward_by_differences(method, renorm):
    """Against differences of the routing itself: the loss sum(gw * w) of
    moe_route's weights when one logit moves by h (choice unchanged).  The
    weights are within weight_rtol, so the quotient's error is at most
    2 k |gw| rtol / (2 h) + O(h^2)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    M, E, k, h = 6, 12, 3, 2.0 ** -6
    logits = torch.randn(M, E, generator=g, device="cuda") * 2
    bias = torch.randn(E, generator=g, device="cuda") * 0.01
    _, ids = pkg.moe_route(logits, k, method, renorm, score_bias=bias)
    gw = torch.randn(M, k, generator=g, device="cuda")
    got = pkg.moe_route_backward(gw, logits, ids, method, renorm)
    steps = []
    for e in range(E):
        loss = []
        for s in (h, -h):
            l = logits.clone()
            l[:, e] += s
            w, i = pkg.moe_route(l, k, method, renorm, score_bias=bias)
            # the weights in the order of the unmoved choice; rows whose choice moved are left out
            same = (i.sort(1).values == ids.sort(1).values).all(1)
            dense = torch.zeros(M, E, device="cuda").scatter_(1, i.long(), w)
            loss.append(((gw * dense.gather(1, ids.long())).sum(1), same))
        steps.append(((loss[0][0] - loss[1][0]) / (2 * h), loss[0][1] & loss[1][1]))
    rtol = weight_rtol(logits.cpu().numpy(), E)
    size = gw.abs().sum(1).max().item()
    tol = size * rtol / h + size * h * h      # third derivatives of a weight are below 1 (1/6 used up to 6)
    checked = 0
    for e, (d, same) in enumerate(steps):
        assert ((d - got[:, e]).abs()[same] <= tol).all()
        checked += int(same.sum())
    assert checked >= M * E // 2


def test_route_backward_repeated_ids_and_bad_ids():
    g = torch.Generator(device="cuda").manual_seed(2)
    M, E, k = 40, 24, 6
    logits = torch.randn(M, E, generator=g, device="cuda")
    gw = torch.randn(M, k, generator=g, device="cuda")
    ids = torch.randint(0, 4, (M, k), generator=g, device="cuda", dtype=torch.int32)
    for method, renorm in (("softmax", False), ("softmax", True), ("sigmoid", True)):
        check_backward(gw, logits, ids, method, renorm, 2.0)
        bad = ids.clone()
        bad[3, 1], bad[5] = -1, E
        bad[7, 0] = 2 ** 31 - 1
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = pkg.moe_route_backward(gw, logits, bad, method, renorm, 2.0, error_word=err)
        ref = oracle.route_backward(gw.double().cpu().numpy(), logits.double().cpu().numpy(),
                                    bad.cpu().numpy(), method, renorm, 2.0)
        np.testing.assert_allclose(out.cpu().numpy(), ref, atol=1e-4)
        assert err.item() == 4 and (out[5] == 0).all()


def test_route_backward_masked_and_extreme_logits():
    g = torch.Generator(device="cuda").manual_seed(4)
    M, E, k = 8, 32, 4
    logits = torch.randn(M, E, generator=g, device="cuda")
    logits[0] = float("-inf")
    logits[1, ::2] = float("-inf")
    logits[2] = -300.0 + logits[2]
    logits[3] = 200.0 + logits[3]
    logits[4] = torch.finfo(torch.float32).min
    gw = torch.randn(M, k, generator=g, device="cuda")
    ids = torch.arange(k, dtype=torch.int32, device="cuda").repeat(M, 1)
    for method, renorm in (("softmax", False), ("softmax", True), ("sigmoid", True)):
        out = pkg.moe_route_backward(gw, logits, ids, method, renorm)
        assert torch.isfinite(out).all(), (method, renorm)
        assert (out[0] == 0).all() and (out[1, ::2] == 0).all()
        # softmax does not change when every logit moves
        if method == "softmax":
            moved = logits.clone()
            moved[2] += 300.0
            moved[3] -= 200.0
            ref = oracle.route_backward(gw.double().cpu().numpy()[1:4],
                                        logits.double().cpu().numpy()[1:4],
                                        ids.cpu().numpy()[1:4], method, renorm)
            np.testing.assert_allclose(out[1:4].cpu().numpy(), ref, atol=1e-5)
        else:
            # far below zero, sigmoid's ratios are the softmax's
            ref = oracle.route_backward(gw.double().cpu().numpy()[2:3],
                                        logits.double().cpu().numpy()[2:3],
                                        ids.cpu().numpy()[2:3], "softmax", True)
            np.testing.assert_allclose(out[2:3].cpu().numpy(), ref, atol=1e-5)


def test_route_backward_views_and_empty():
    assert pkg.moe_route_backward(torch.zeros(0, 2, device="cuda"), torch.zeros(0, 8, device="cuda"),
                                  torch.zeros(0, 2, dtype=torch.int32, device="cuda")).shape == (0, 8)
    for M, E, k in ((3, 15, 3), (5, 33, 5), (3, 256, 7)):
        for dt in (torch.float32, torch.bfloat16):
            buf = torch.randn((M + 2) * E + 1, device="cuda").to(dt)
            logits = buf[E + 1:E + 1 + M * E].view(M, E)
            out = torch.full(((M + 2) * E + 1,), -5.0, device="cuda", dtype=dt)
            gw = torch.randn(M * k + 1, device="cuda")[1:].view(M, k)
            ids = torch.argsort(torch.rand(M, E, device="cuda"), 1)[:, :k].int().contiguous()
            pkg.moe_route_backward(gw, logits, ids, grad_logits=out[E + 1:E + 1 + M * E].view(M, E))
            got, _ = check_backward(gw.clone(), logits.clone(), ids, "softmax", False, 1.0)
            assert torch.equal(out[E + 1:E + 1 + M * E].view(M, E), got)
            assert (out[:E + 1] == -5).all() and (out[E + 1 + M * E:] == -5).all()


@pytest.mark.parametrize("M,E,k", [(5, 32, 4), (40, 256, 8), (7, 500, 20), (6, 128, 40)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("method,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
def test_route_backward_masked_items_take_no_part(M, E, k, dtype, method, renorm):
    """Whatever grad_weights holds for experts that are masked (their weights
    are 0 and nothing made these numbers), the token's gradient is that of the
    others."""
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(M, E, generator=g, device="cuda").to(getattr(torch, dtype))
    ids = torch.argsort(torch.rand(M, E, generator=g, device="cuda"), 1)[:, :k].int().contiguous()
    gw = torch.randn(M, k, generator=g, device="cuda")
    masked = torch.rand(M, k, generator=g, device="cuda") < 0.4
    masked[0], masked[1, 0] = True, True
    logits.scatter_(1, ids.long(), torch.where(masked, float("-inf"), logits.float().gather(
        1, ids.long())).to(logits.dtype))
    clean = torch.where(masked, 0.0, gw)
    ref = pkg.moe_route_backward(clean, logits, ids, method, renorm, 1.5)
    assert torch.isfinite(ref).all() and (ref[0] == 0).all() and (ref != 0).any()
    check_backward(clean, logits, ids, method, renorm, 1.5)
    for junk in (float("nan"), float("inf"), -float("inf"), 3e38):
        got = pkg.moe_route_backward(torch.where(masked, junk, gw), logits, ids, method, renorm, 1.5)
        assert torch.equal(got, ref), junk


@pytest.mark.parametrize("method,renorm,E,k,kg,G", [("sigmoid", True, 256, 8, 4, 8),
                                                    ("softmax", False, 257, 8, 1, 1),
                                                    ("softmax", False, 128, 34, 1, 1)])
def test_route_ops_past_32_bits(method, renorm, E, k, kg, G):
    """More than 2^31 logits: the last rows as in a call of their own (all rows
    but the first and last are of one logit)."""
    M, n = (1 << 31) // E + 5000, 200
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.zeros(M, E, device="cuda", dtype=torch.bfloat16)
    rows = torch.randn(n, E, generator=g, device="cuda").to(torch.bfloat16)
    gw = torch.randn(M, k, generator=g, device="cuda")
    logits[:n], logits[-n:] = rows, rows
    bias = torch.randn(E, generator=g, device="cuda") * 0.05
    a = (k, method, renorm, kg, G, 0, 2.5)
    w, ids = pkg.moe_route(logits, *a, score_bias=bias)
    w0, i0 = check_biased(rows, bias, args(k, method, renorm, kg, G, 0, 2.5))
    # (a few tokens may be summed in another order)
    rtol = 2 * weight_rtol(rows.double().cpu().numpy(), E)
    for part in (slice(0, n), slice(M - n, M)):
        assert torch.equal(ids[part], i0)
        assert ((w[part] - w0).abs() <= rtol * w0).all()
    gl = pkg.moe_route_backward(gw, logits, ids, method, renorm, 2.5)
    for part in (slice(0, n), slice(M - n, M)):
        assert torch.equal(gl[part], pkg.moe_route_backward(gw[part], rows, i0, method, renorm, 2.5))


# ------------------------------------------------- streams, graphs, threads --
def test_route_ops_on_other_streams_in_graphs_and_threads():
    a = (8, "sigmoid", True, 4, 8, 1, 2.5)
    g = torch.Generator(device="cuda").manual_seed(6)
    logits = torch.randn(500, 256, generator=g, device="cuda")
    bias = torch.randn(256, generator=g, device="cuda") * 0.05
    gw = torch.randn(500, 8, generator=g, device="cuda")
    w, ids = pkg.moe_route(logits, *a, score_bias=bias)
    gl = pkg.moe_route_backward(gw, logits, ids, "sigmoid", True, 2.5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    w2, ids2 = pkg.moe_route(logits, *a, score_bias=bias, stream=s)
    gl2 = pkg.moe_route_backward(gw, logits, ids2, "sigmoid", True, 2.5, stream=s)
    s.synchronize()
    assert torch.equal(w, w2) and torch.equal(ids, ids2) and torch.equal(gl, gl2)
    graph = torch.cuda.CUDAGraph()
    static = torch.zeros_like(logits)
    with torch.cuda.graph(graph):
        w3, ids3 = pkg.moe_route(static, *a, score_bias=bias)
        gl3 = pkg.moe_route_backward(gw, static, ids3, "sigmoid", True, 2.5)
    for _ in range(2):
        static.copy_(logits)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(w, w3) and torch.equal(ids, ids3) and torch.equal(gl, gl3)
        static.zero_()
    bad = []

    def run():
        st = torch.cuda.Stream()
        for _ in range(20):
            x = pkg.moe_route(logits, *a, score_bias=bias, stream=st)
            y = pkg.moe_route_backward(gw, logits, x[1], "sigmoid", True, 2.5, stream=st)
            st.synchronize()
            if not (torch.equal(x[1], ids) and torch.equal(y, gl)):
                bad.append(1)
    ts = [threading.Thread(target=run) for _ in range(3)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_layer_with_score_bias():
    """The layer entry points route with the bias."""
    spec = wl.SMALL_SPECS["deepseek_small"]
    d = wl.make_moe_inputs(spec, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    bias = torch.randn(spec.E, generator=g, device="cuda") * 0.2
    a = dict(k_group=spec.k_group, group_count=spec.group_count,
             group_select_mode=spec.group_select_mode, routing_method=spec.routing_method,
             renormalize=spec.renormalize, routed_scaling_factor=spec.routed_scaling_factor)
    w_gate = torch.randn(spec.H, spec.E, generator=g, device="cuda").to(torch.bfloat16) * 0.1
    y = pkg.moe_layer(d["hidden"], w_gate, d["w13"], d["w2"], spec.top_k, score_bias=bias, **a)
    logits = pkg.moe_router_logits(d["hidden"], w_gate)
    y2 = pkg.fused_moe(d["hidden"], logits, d["w13"], d["w2"], spec.top_k, score_bias=bias, **a)
    assert torch.equal(y, y2)
    rw, rids = oracle.route_biased(logits.double().cpu().numpy(), bias.double().cpu().numpy(),
                                   spec.top_k, spec.routing_method, spec.renormalize, spec.k_group,
                                   spec.group_count, spec.group_select_mode,
                                   spec.routed_scaling_factor)
    ref = oracle.forward(wl.to_f64(d["hidden"]), rw, rids, wl.to_f64(d["w13"]), wl.to_f64(d["w2"]))
    check_out(y.double().cpu().numpy(), ref, "layer with score bias")


def test_results_on_a_stream_of_the_callers_come_from_its_memory():
    """A block that the current stream has just given back may still be in use
    by it: a result on another stream must not be put there."""
    logits = torch.randn(512, 256, device="cuda")
    bias = torch.zeros(256, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty(512, 8, device="cuda") for _ in range(4)] + [
        torch.empty(512, 256, device="cuda") for _ in range(2)]
    at = {t.data_ptr() for t in old}
    del old
    w, ids = pkg.moe_route(logits, 8, score_bias=bias, stream=s)
    gl = pkg.moe_route_backward(w, logits, ids, stream=s)
    s.synchronize()
    assert not at & {w.data_ptr(), ids.data_ptr(), gl.data_ptr()}
    assert torch.equal(ids, pkg.moe_route(logits, 8, score_bias=bias)[1])


FIRST_IN_CAPTURE = """
import torch
import mixture_experts_ffn_softmax_gb300 as pkg
E4M3 = torch.float8_e4m3fn
l, b = torch.randn(70, 256, device="cuda"), torch.randn(256, device="cuda") * 0.1
x = torch.randn(600, 512, device="cuda").to(torch.bfloat16)
w13, w2 = torch.ones(512, 768, device="cuda").to(E4M3), torch.ones(384, 512, device="cuda").to(E4M3)
s13, s2 = torch.ones(4, 6, device="cuda") / 64, torch.ones(3, 4, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    w, ids = pkg.moe_route(l, 8, "sigmoid", True, 4, 8, 1, 2.5, score_bias=b)
    gl = pkg.moe_route_backward(w, l, ids, "sigmoid", True, 2.5)
    y = pkg.moe_shared_expert_fp8(x, w13, w2, s13, s2)
    y1 = pkg.moe_shared_expert_fp8(x[:9], w13, w2, s13, s2)
g.replay()
torch.cuda.synchronize()
w_, ids_ = pkg.moe_route(l, 8, "sigmoid", True, 4, 8, 1, 2.5, score_bias=b)
assert torch.equal(ids, ids_) and torch.equal(w, w_)
assert torch.equal(gl, pkg.moe_route_backward(w, l, ids, "sigmoid", True, 2.5))
assert torch.equal(y, pkg.moe_shared_expert_fp8(x, w13, w2, s13, s2))
assert torch.equal(y1, pkg.moe_shared_expert_fp8(x[:9], w13, w2, s13, s2))
"""


def test_first_calls_of_a_process_inside_a_capture():
    root = pathlib.Path(__file__).resolve().parents[1]
    subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], cwd=root, check=True, timeout=300)
