"""GPU parity of MX FP4: quantisation (bit-exact where its input is) and the
product of codes (bit-exact on codes whose sums are exact)."""
import numpy as np
import pytest
import torch

import mixture_experts_ffn_softmax_gb300 as pkg
import oracle

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U16, U32 = 2.0 ** -8, 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------ quantisation --
QUANT = [(1, 32), (3, 96), (2, 128), (5, 160), (1, 7168), (33, 256), (129, 2048), (17, 1952),
         (1000, 384), (7, 18432)]


@pytest.mark.parametrize("M,K", QUANT)
def test_quant_bit_exact(M, K):
    x = (torch.randn(M, K, generator=gen(M + K), device="cuda") * 3).to(BF16)
    x[0, :32] = 0                                             # a block of zeros
    x[-1] = (torch.randint(-31, 32, (K,), generator=gen(1), device="cuda") / 4).to(BF16)  # ties
    values = torch.full((M + 1, K), 7.0, device="cuda", dtype=BF16)
    q, s = pkg.moe_quant_mx_fp4(x, values=values[:M])
    rc, rs = oracle.quant_mx_fp4(x.double().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), oracle.pack_fp4(rc))
    rv = oracle.mx_fp4_values(q.cpu().numpy(), s.cpu().numpy())
    assert np.array_equal(values[:M].double().cpu().numpy(), rv) and (values[M] == 7).all()
    q2, s2 = pkg.moe_quant_mx_fp4(x)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_quant_every_bf16_value():
    """Every finite bf16 value as its block's only one, and under a largest of 1."""
    bits = torch.arange(0, 1 << 16, device="cuda", dtype=torch.int32)
    v = bits.to(torch.int16).view(BF16)
    v = v[torch.isfinite(v)]
    n = len(v)
    x = torch.zeros(2 * n, 32, device="cuda", dtype=BF16)
    x[:n, 5] = v
    x[n:, 9], x[n:, 5] = 1.0, torch.where(v.abs() <= 1, v, torch.zeros_like(v))
    values = torch.empty_like(x)
    q, s = pkg.moe_quant_mx_fp4(x, values=values)
    rc, rs = oracle.quant_mx_fp4(x.double().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), oracle.pack_fp4(rc))
    assert np.array_equal(values.double().cpu().numpy(), oracle.mx_fp4_values(q.cpu().numpy(), rs))


def test_quant_not_finite():
    x = torch.ones(3, 96, device="cuda", dtype=BF16)
    x[1, 40], x[2, 0] = float("inf"), float("nan")
    values = torch.empty_like(x)
    q, s = pkg.moe_quant_mx_fp4(x, values=values)
    assert s[1].tolist() == [125, 255, 125] and s[2].tolist() == [255, 125, 125]
    assert (q[1, 16:32] == 0).all() and (q[2, :16] == 0).all()
    assert torch.isnan(values[1, 32:64]).all() and torch.isnan(values[2, :32]).all()
    assert (values[0] == 1).all() and (values[1, :32] == 1).all() and (values[2, 32:] == 1).all()


@pytest.mark.parametrize("M,K", QUANT)
def test_quant_swiglu(M, K):
    """The scale is a power of two of max|z|, whose error is 8 * 2^-24: either
    side of a power of two next to it; the code that of z / scale within the
    same error."""
    x = (torch.randn(M, 2 * K, generator=gen(M * 3 + K), device="cuda") * 2).to(BF16)
    values = torch.empty(M, K, device="cuda", dtype=BF16)
    q, s = pkg.moe_quant_mx_fp4(x, swiglu=True, values=values)
    z = oracle.swiglu(x.double().cpu().numpy())
    rel = 8 * U32
    amax = np.abs(z).reshape(M, -1, 32).max(2)
    s = s.cpu().numpy().astype(int)
    floor = lambda v: np.maximum(np.frexp(v)[1] - 1 - 2 + 127, 0)  # noqa: E731
    assert ((s == floor(amax * (1 - rel))) | (s == floor(amax * (1 + rel)))).all()
    scale = np.repeat(np.ldexp(1.0, s - 127), 32, axis=1)
    v = np.abs(z) / scale
    got = oracle.mx_fp4_values(q.cpu().numpy(), s)
    assert np.array_equal(values.double().cpu().numpy(), got)
    lo = np.array([0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    at = np.searchsorted([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.abs(got) / scale)
    hi = np.append(lo[1:], np.inf)
    assert (v >= lo[at] * (1 - 2 * rel)).all() and (v <= hi[at] * (1 + 2 * rel)).all()
    assert (np.sign(got) * np.sign(z) >= 0).all()


def test_quant_past_32_bits():
    K = 2048
    M, n = (1 << 31) // K + 3000, 100
    for swiglu in (False, True):
        x = torch.zeros(M, 2 * K if swiglu else K, device="cuda", dtype=BF16)
        rows = torch.randn(n, x.shape[1], generator=gen(5), device="cuda").to(BF16)
        x[:n], x[-n:] = rows, rows
        q, s = pkg.moe_quant_mx_fp4(x, swiglu)
        q0, s0 = pkg.moe_quant_mx_fp4(rows, swiglu)
        for part in (slice(0, n), slice(M - n, M)):
            assert torch.equal(q[part], q0) and torch.equal(s[part], s0)
