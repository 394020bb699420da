"""CPU tests of the operators beside the expert layer: the oracle's routing
with a bias, its gradient and the block-scaled product against independent
computations, and the refusals of the C ABI and of the binding."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import mixture_experts_ffn_softmax_gb300 as pkg
import oracle

OK, INVALID, NO_DEVICE = 0, 1, 7


# ------------------------------------------------------------- oracle pins --
@pytest.mark.parametrize("seed", range(6))
def test_oracle_biased_route_by_enumeration(seed):
    """Against enumeration of every group subset and expert subset, on scores
    with many exact ties."""
    rng = np.random.default_rng(seed)
    E, G, kg, k, mode = [(6, 1, 1, 3, 0), (6, 3, 2, 2, 0), (8, 4, 2, 3, 1), (8, 2, 1, 4, 1),
                         (6, 2, 2, 6, 0), (8, 4, 3, 5, 1)][seed]
    logits = rng.integers(-1, 2, (20, E)).astype(float)
    bias = rng.integers(-1, 2, E) * 0.25
    w, ids = oracle.route_biased(logits, bias, k, "sigmoid", True, kg, G, mode, 2.0)
    gs = E // G
    for t in range(20):
        p = 1 / (1 + np.exp(-logits[t]))
        c = p + bias
        score = [sorted(c[g * gs:(g + 1) * gs])[-1] + (sorted(c[g * gs:(g + 1) * gs])[-2] if mode
                                                       else 0.0) for g in range(G)]
        kept = max(itertools.combinations(range(G), kg),
                   key=lambda s: (sorted((score[g] for g in s), reverse=True), [-g for g in s]))
        pool = [e for e in range(E) if e // gs in kept]
        best = max(itertools.permutations(pool, k),
                   key=lambda s: ([c[e] for e in s], [-e for e in s]))
        assert list(best) == ids[t].tolist()
        np.testing.assert_allclose(w[t], 2.0 * p[list(best)] / p[list(best)].sum(), rtol=1e-12)


def test_oracle_biased_route_without_bias_is_route():
    rng = np.random.default_rng(0)
    logits = rng.normal(size=(50, 32))
    for method, renorm, kg, G, mode in (("softmax", True, 1, 1, 0), ("softmax", False, 2, 4, 1),
                                        ("sigmoid", True, 2, 4, 1), ("sigmoid", True, 3, 8, 0)):
        w, ids = oracle.route_biased(logits, np.zeros(32), 4, method, renorm, kg, G, mode, 1.5)
        w0, ids0, _ = oracle.route(logits, 4, method, renorm, kg, G, mode, 1.5)
        assert np.array_equal(ids, ids0)
        np.testing.assert_allclose(w, w0, rtol=1e-12)


def test_oracle_biased_route_masks_and_underflow():
    inf = np.inf
    logits = np.array([[-inf, 0.0, -inf, 1.0], [-inf] * 4, [-800.0, -801.0, -900.0, -inf]])
    bias = np.array([9.0, 0.0, 5.0, 0.0])
    w, ids = oracle.route_biased(logits, bias, 3, "sigmoid")
    assert ids.tolist() == [[3, 1, 0], [0, 1, 2], [0, 2, 1]]
    assert w[0, 2] == 0.0 and abs(w[0].sum() - 1) < 1e-12 and w[1].tolist() == [0, 0, 0]
    e = np.exp([0.0, -100.0, -1.0])
    np.testing.assert_allclose(w[2], e / e.sum(), rtol=1e-12)
    w, ids = oracle.route_biased(logits[:2], bias, 2, "softmax", False)
    assert ids.tolist() == [[3, 1], [0, 1]] and w[1].tolist() == [0, 0]


@pytest.mark.parametrize("method,renorm", [("softmax", False), ("softmax", True),
                                           ("sigmoid", True)])
def test_oracle_route_backward_by_differences(method, renorm):
    """Central differences of the weights: error O(h^2) + O(eps / h)."""
    rng = np.random.default_rng(1)
    E, k, h = 7, 3, 1e-5
    logits, gw = rng.normal(size=(4, E)), rng.normal(size=(4, k))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(4)])
    ids[3, 1] = ids[3, 0]                        # an expert named twice
    got = oracle.route_backward(gw, logits, ids, method, renorm, 1.7)
    for t in range(4):
        def loss(l):
            if method == "sigmoid":
                p = 1 / (1 + np.exp(-l))
            else:
                p = np.exp(l) / np.exp(l).sum()
            w = p[ids[t]]
            if method == "sigmoid" or renorm:
                w = w / w.sum()
            return 1.7 * np.dot(gw[t], w)
        for e in range(E):
            d = np.zeros(E)
            d[e] = h
            num = (loss(logits[t] + d) - loss(logits[t] - d)) / (2 * h)
            assert abs(num - got[t, e]) < 1e-8


def test_oracle_matmul_blocks_against_dequantised_product():
    rng = np.random.default_rng(2)
    M, K, N = 5, 272, 144
    a, w = rng.normal(size=(M, K)), rng.normal(size=(K, N))
    sa, sw = rng.uniform(0.5, 2, (M, 3)), rng.uniform(0.5, 2, (3, 2))
    y, size = oracle.matmul_blocks(a, sa, w, sw, bias=np.arange(N))
    da = a * sa[:, np.arange(K) // 128]
    dw = w * sw[np.arange(K) // 128][:, np.arange(N) // 128]
    np.testing.assert_allclose(y, da @ dw + np.arange(N), rtol=1e-12)
    np.testing.assert_allclose(size, np.abs(da) @ np.abs(dw) + np.arange(N), rtol=1e-12)


# --------------------------------------------------------- C ABI refusals --
def _p(v=4096):
    return ctypes.c_void_p(v)


def _biased(M=4, E=8, k=2, method=0, renorm=1, kg=1, G=1, mode=0, scale=1.0, bf16=0, logits=4096,
            bias=4096, w=4096, ids=4096):
    return pkg.lib().moe_route_biased(_p(logits), bf16, _p(bias), M, E, k, method, renorm, kg, G,
                                      mode, scale, _p(w), _p(ids), None)


def test_route_biased_refusals():
    assert _biased(M=-1) == INVALID and _biased(M=1 << 31) == INVALID
    assert _biased(E=0) == INVALID and _biased(E=1025) == INVALID
    assert _biased(k=0) == INVALID and _biased(k=9) == INVALID
    assert _biased(E=128, k=65) == INVALID
    assert _biased(method=2) == INVALID and _biased(mode=2) == INVALID
    assert _biased(G=3) == INVALID and _biased(G=4, kg=5) == INVALID
    assert _biased(G=4, kg=1, k=3) == INVALID and _biased(G=8, kg=2, mode=1) == INVALID
    assert _biased(scale=float("inf")) == INVALID and _biased(bf16=2) == INVALID
    for bad in ("logits", "bias", "w", "ids"):
        assert _biased(**{bad: 0}) == INVALID
        assert _biased(**{bad: 4098}) == INVALID
    assert _biased(logits=4098, bf16=1) in (OK, NO_DEVICE)
    assert _biased(M=0, logits=0) == OK


def _backward(M=4, E=8, k=2, method=0, renorm=1, scale=1.0, bf16=0, gw=4096, logits=4096, ids=4096,
              out=8192, err=0):
    return pkg.lib().moe_route_backward(_p(gw), _p(logits), bf16, _p(ids), M, E, k, method, renorm,
                                        scale, _p(out), _p(err) if err else None, None)


def test_route_backward_refusals():
    assert _backward(M=-1) == INVALID and _backward(M=1 << 31) == INVALID
    assert _backward(E=0) == INVALID and _backward(E=1025) == INVALID
    assert _backward(k=0) == INVALID and _backward(k=65) == INVALID
    assert _backward(method=2) == INVALID and _backward(bf16=-1) == INVALID
    assert _backward(scale=float("nan")) == INVALID and _backward(err=4097) == INVALID
    for bad in ("gw", "logits", "ids", "out"):
        assert _backward(**{bad: 0}) == INVALID
        assert _backward(**{bad: 4097}) == INVALID
    assert _backward(M=0, gw=0) == OK


def test_quant_groups_refusals():
    def q(M=4, K=64, swiglu=0, x=4096, q8=4096, s=4096):
        return pkg.lib().moe_quant_groups_fp8(_p(x), M, K, swiglu, _p(q8), _p(s), None)
    assert q(M=-1) == INVALID and q(M=1 << 31) == INVALID
    for K in (0, 8, 24, -16, (1 << 24) + 16):
        assert q(K=K) == INVALID
    assert q(swiglu=2) == INVALID
    for bad in ("x", "q8"):
        assert q(**{bad: 0}) == INVALID and q(**{bad: 4104}) == INVALID
    assert q(s=0) == INVALID and q(s=4098) == INVALID
    assert q(M=0, x=0) == OK


def test_matmul_fp8_refusals():
    def mm(M=4, K=64, N=64, tr=0, f32=0, err=0, bias=0, **at):
        p = {n: _p(at.get(n, 4096)) for n in ("a", "sa", "w", "sw", "out")}
        return pkg.lib().moe_matmul_fp8(p["a"], p["sa"], p["w"], p["sw"], tr,
                                        _p(bias) if bias else None, M, K, N, f32, p["out"],
                                        _p(err) if err else None, None)
    assert mm(M=-1) == INVALID and mm(M=1 << 31) == INVALID
    for v in (0, 8, 24, -16, 1 << 30):
        assert mm(K=v) == INVALID and mm(N=v) == INVALID
    assert mm(tr=2) == INVALID and mm(f32=3) == INVALID
    assert mm(bias=4104) == INVALID and mm(err=4097) == INVALID
    for bad in ("a", "w", "out"):
        assert mm(**{bad: 0}) == INVALID and mm(**{bad: 4104}) == INVALID
    for bad in ("sa", "sw"):
        assert mm(**{bad: 0}) == INVALID and mm(**{bad: 4097}) == INVALID
    assert mm(M=0, a=0) == OK
    if not torch.cuda.is_available():
        assert mm() == NO_DEVICE


# ------------------------------------------------------- binding refusals --
def test_binding_refuses_wrong_tensors():
    f32, bf = torch.float32, torch.bfloat16
    l, b = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.moe_route(l, 2, score_bias=b)
    with pytest.raises(ValueError, match="score_bias"):
        pkg.moe_route(l, 2, score_bias=torch.zeros(7))
    with pytest.raises(ValueError, match="score_bias"):
        pkg.moe_route(l, 2, score_bias=b.double())
    with pytest.raises(ValueError, match="router_logits"):
        pkg.moe_route(l.double(), 2, score_bias=b)
    with pytest.raises(ValueError, match="router_logits"):
        pkg.moe_route(l[0], 2, score_bias=b)
    with pytest.raises(ValueError, match="contiguous"):
        pkg.moe_route(torch.zeros(8, 4).t(), 2, score_bias=b)
    with pytest.raises(ValueError, match="topk_ids"):
        pkg.moe_route(l, 2, score_bias=b, topk_ids=torch.zeros(4, 2))
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="grad_weights"):
        pkg.moe_route_backward(torch.zeros(4, 3), l, ids)
    with pytest.raises(ValueError, match="topk_ids"):
        pkg.moe_route_backward(torch.zeros(4, 2), l, ids.long())
    with pytest.raises(ValueError, match="grad_logits"):
        pkg.moe_route_backward(torch.zeros(4, 2), l, ids, grad_logits=l.to(bf))
    with pytest.raises(ValueError, match="CUDA"):
        pkg.moe_route_backward(torch.zeros(4, 2), l, ids)
    x = torch.zeros(4, 64, dtype=bf)
    with pytest.raises(ValueError, match="x must"):
        pkg.moe_quant_groups_fp8(x.to(f32))
    with pytest.raises(ValueError, match="even"):
        pkg.moe_quant_groups_fp8(torch.zeros(4, 33, dtype=bf), swiglu=True)
    with pytest.raises(ValueError, match="scale"):
        pkg.moe_quant_groups_fp8(x, scale=torch.zeros(4, 2))
    q = torch.zeros(4, 256, dtype=torch.uint8)
    w, sa, sw = torch.zeros(256, 64, dtype=torch.uint8), torch.ones(4, 2), torch.ones(2, 1)
    with pytest.raises(ValueError, match="w_q has shape"):
        pkg.moe_matmul_fp8(q, sa, w, sw.t().contiguous(), transposed=True)
    with pytest.raises(ValueError, match="w_scale"):
        pkg.moe_matmul_fp8(q, sa, w, torch.ones(2, 2))
    with pytest.raises(ValueError, match="a_scale"):
        pkg.moe_matmul_fp8(q, torch.ones(4, 3), w, sw)
    with pytest.raises(ValueError, match="bias"):
        pkg.moe_matmul_fp8(q, sa, w, sw, bias=torch.zeros(64))
    with pytest.raises(ValueError, match="output"):
        pkg.moe_matmul_fp8(q, sa, w, sw, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out has shape"):
        pkg.moe_matmul_fp8(q, sa, w, sw, out=torch.zeros(4, 32))
    with pytest.raises(ValueError, match="CUDA"):
        pkg.moe_matmul_fp8(q, sa, w, sw)


def test_matmul_fp8_refuses_more_tiles_than_it_counts():
    def mm(M, N):
        p = _p(4096)
        return pkg.lib().moe_matmul_fp8(p, p, p, p, 0, None, M, 64, N, 0, p, None, None)
    assert mm((1 << 31) - 1, 1 << 22) == INVALID
    assert mm((1 << 22) + 1, 1 << 22) == INVALID
    if not torch.cuda.is_available():
        assert mm(1 << 22, 1 << 22) == NO_DEVICE


def test_binding_refuses_sizes_that_32_bits_would_cut():
    def big(rows, cols, dtype):
        return torch.zeros(1, 1, dtype=dtype).expand(rows, cols)
    n = (1 << 32) + 16
    u8 = torch.uint8
    with pytest.raises(ValueError, match="below 2"):
        pkg.moe_matmul_fp8(big(1, n, u8), torch.ones(1, 1), big(n, 16, u8), torch.ones(1, 1))
    with pytest.raises(ValueError, match="below 2"):
        pkg.moe_matmul_fp8(big(1, 16, u8), torch.ones(1, 1), big(16, n, u8), torch.ones(1, 1))
    with pytest.raises(ValueError, match="below 2"):
        pkg.moe_quant_groups_fp8(big(1, n, torch.bfloat16))
    with pytest.raises(ValueError, match="below 2"):
        pkg.moe_route(big(1, n, torch.float32), 2, score_bias=torch.zeros(8))
    with pytest.raises(ValueError, match="below 2"):
        pkg.moe_route_backward(torch.ones(1, 2), big(1, n, torch.float32),
                               torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        pkg.moe_matmul_fp8(torch.zeros(1, 16, dtype=u8), torch.ones(1, 1),
                           torch.zeros(16, 16, dtype=u8), torch.ones(1, 1), out=[0.0])
    with pytest.raises(ValueError):
        pkg.moe_quant_groups_fp8(torch.zeros(1, 16, dtype=torch.bfloat16), q8=[0])
