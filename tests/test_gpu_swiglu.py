"""GPU parity of SiLU(gate) * up of routed rows and its gradient."""
import numpy as np
import pytest
import torch

import mixture_experts_ffn_softmax_gb300 as pkg
import oracle

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
U16, U32 = 2.0 ** -8, 2.0 ** -24        # half a step, relative


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(seed, *shape, top=2):
    return torch.randint(-top, top + 1, shape, generator=gen(seed), device="cuda").to(BF16)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("R,I", [(1, 8), (3, 264), (130, 768), (7, 2048), (5, 2056), (2, 14336),
                                 (700, 4096)])
def test_swiglu_and_its_gradient(R, I, weighted):
    """z: sig(g) within 5 * 2^-24, three products and the rounding to bf16.
    dg: sig(g) (1 + g (1 - sig(g))) cancels near g = -1.28, its error is that
    of the summands, at most (2 + |g|) sig(g) times 12 roundings; five more
    products.  dw: a sum of I products, 10 roundings each, and the additions."""
    gu = (torch.randn(R, 2 * I, generator=gen(I), device="cuda") * 2).to(BF16)
    dz = torch.randn(R, I, generator=gen(R), device="cuda").to(BF16)
    w = torch.rand(R, generator=gen(3), device="cuda") if weighted else None
    gu64, dz64 = gu.double().cpu().numpy(), dz.double().cpu().numpy()
    w64 = w.double().cpu().numpy() if weighted else None
    z = pkg.moe_swiglu(gu, w).double().cpu().numpy()
    ref = oracle.swiglu(gu64, w64)
    assert (np.abs(z - ref) <= (U16 * 1.01 + 10 * U32) * np.abs(ref)).all()
    d, dw = pkg.moe_swiglu_backward(dz, gu, w)
    rd, rdw = oracle.swiglu_backward(dz64, gu64, w64)
    g, u = gu64[:, :I], gu64[:, I:]
    s = 1 / (1 + np.exp(-g))
    a = np.abs(dz64 * (1 if w is None else w64[:, None]))
    slack = np.concatenate([a * np.abs(u) * s * (2 + np.abs(g)), a * np.abs(g) * s], 1) * 20 * U32
    assert (np.abs(d.double().cpu().numpy() - rd) <= U16 * 1.01 * np.abs(rd) + slack).all()
    if weighted:
        size = np.abs(dz64 * g * s * u).sum(1)
        adds = -(-I // 256) * 8 + 13       # in a lane, across lanes and warps
        assert (np.abs(dw.double().cpu().numpy() - rdw) <= (adds + 10) * U32 * size).all()
    else:
        assert dw is None
        dw = torch.empty(R, device="cuda")
        assert pkg.moe_swiglu_backward(dz, gu, grad_weights=dw)[1] is dw
        assert np.allclose(dw.double().cpu().numpy(), rdw, rtol=0, atol=1e-5 * np.abs(rdw).max() + 1e-5)
    # in place
    again = gu.clone()
    d2, _ = pkg.moe_swiglu_backward(dz, again, w, grad_gate_up=again)
    assert d2 is again and torch.equal(again, d)


def test_swiglu_far_gates():
    g = torch.tensor([-3e38, -200.0, -90.0, -79.0, 0.0, 79.0, 90.0, 200.0], device="cuda")
    gu = torch.cat([g, torch.full((8,), 2.0, device="cuda")])[None].to(BF16)
    z = pkg.moe_swiglu(gu).double()
    assert torch.equal(z[0, [0, 1, 4]], torch.zeros(3, device="cuda", dtype=torch.float64))
    assert torch.equal(z[0, 5:], 2 * gu[0, 5:8].double())
    d, dw = pkg.moe_swiglu_backward(torch.ones(1, 8, device="cuda", dtype=BF16), gu,
                                    torch.ones(1, device="cuda"))
    assert torch.isfinite(d).all() and torch.isfinite(dw).all()
    assert torch.equal(d[0, [0, 1, 2]].float(), torch.zeros(3, device="cuda"))
    assert torch.equal(d[0, 4:8].float(), torch.tensor([1.0, 2.0, 2.0, 2.0], device="cuda"))


def test_swiglu_nan_rows_stay_alone():
    gu, dz = ints(1, 6, 512), ints(2, 6, 256)
    w = torch.rand(6, generator=gen(1), device="cuda")
    d, dw = pkg.moe_swiglu_backward(dz, gu, w)
    gu2 = gu.clone()
    gu2[3, 17] = float("nan")
    d2, dw2 = pkg.moe_swiglu_backward(dz, gu2, w)
    rows = [0, 1, 2, 4, 5]
    assert torch.isnan(dw2[3]) and torch.isnan(d2[3, 17]) and torch.isnan(d2[3, 256 + 17])
    assert torch.equal(d2[rows], d[rows]) and torch.equal(dw2[rows], dw[rows])
    cols = [c for c in range(512) if c % 256 != 17]
    assert torch.equal(d2[3][cols], d[3][cols])


def test_swiglu_past_32_bits():
    R, I = (1 << 31) // 4096 + 500, 2048
    gu = torch.zeros(R, 2 * I, device="cuda", dtype=BF16)
    dz = torch.zeros(R, I, device="cuda", dtype=BF16)
    gu[-9:], dz[-9:] = ints(1, 9, 2 * I), ints(2, 9, I)
    w = torch.ones(R, device="cuda")
    z, (d, dw) = pkg.moe_swiglu(gu, w), pkg.moe_swiglu_backward(dz, gu, w)
    small = (gu[-9:].clone(), dz[-9:].clone(), w[-9:].clone())
    assert torch.equal(z[-9:], pkg.moe_swiglu(small[0], small[2]))
    sd, sdw = pkg.moe_swiglu_backward(small[1], small[0], small[2])
    assert torch.equal(d[-9:], sd) and torch.equal(dw[-9:], sdw)


INF, NAN = float("inf"), float("nan")
# gates, up and grad_z that meet in one column: not finite, either side of where e^-g and the
# fast form end, products that leave fp32
GATES = [INF, -INF, NAN, 79.0, -79.0, 80.0, -80.0, 88.0, -88.0, 3e38, -3e38, 1e30, 1.0, 0.0, 1.0, 2.0]
UPS = [1.0, 1.0, 1.0, 2.0, 2.0, 2.0, 2.0, 1.5, 1.5, 0.5, 0.5, 1e30, INF, INF, NAN, -INF]


def same_as_formula(got, ref, tol):
    """NaN where the formula has it, the same infinities, finite values within tol."""
    got, ref = got.double(), ref.to(got.dtype).double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)])
    fine = torch.isfinite(ref)
    assert torch.isfinite(got[fine]).all()
    assert ((got - ref)[fine].abs() <= tol * ref[fine].abs() + 2.0 ** -126).all()


@pytest.mark.parametrize("I", [24, 264, 2056])
def test_swiglu_not_finite(I):
    """As the formulas in fp32.  Both sides are rounded to bf16 from values that are apart by
    12 * 2^-24 at most: by a step at most.  The rows beside keep their bits, as do
    the row's columns that are not among the same eight."""
    R = 5
    gu = (torch.randn(R, 2 * I, generator=gen(1), device="cuda")).to(BF16)
    dz = torch.randn(R, I, generator=gen(2), device="cuda").to(BF16)
    w = torch.rand(R, generator=gen(3), device="cuda") + 0.5
    z0, (d0, dw0) = pkg.moe_swiglu(gu, w), pkg.moe_swiglu_backward(dz, gu, w)
    gu2 = gu.clone()
    gu2[2, I - 16:I] = torch.tensor(GATES, device="cuda").to(BF16)
    gu2[2, 2 * I - 16:] = torch.tensor(UPS, device="cuda").to(BF16)
    z, (d, dw) = pkg.moe_swiglu(gu2, w), pkg.moe_swiglu_backward(dz, gu2, w)
    g, u = gu2[:, :I].float(), gu2[:, I:].float()
    s = 1 / (1 + torch.exp(-g))
    silu, dl = g * s, dz.float() * w[:, None]
    tol = 2 * U16 + 12 * U32
    same_as_formula(z[2, -16:], (silu * u * w[:, None])[2, -16:], tol)
    # (the gradient's factor 1 + g (1 - s) of these gates has no cancellation)
    same_as_formula(d[2, I - 16:I], (dl * u * (s * (1 + g * (1 - s))))[2, -16:], tol)
    same_as_formula(d[2, 2 * I - 16:], (dl * silu)[2, -16:], tol)
    assert torch.isnan(dw[2])
    rows, cols = [0, 1, 3, 4], list(range(I - 16)) + list(range(I, 2 * I - 16))
    assert torch.equal(z[rows], z0[rows]) and torch.equal(z[2, :I - 16], z0[2, :I - 16])
    assert torch.equal(d[rows], d0[rows]) and torch.equal(d[2, cols], d0[2, cols])
    assert torch.equal(dw[rows], dw0[rows])


def test_swiglu_backward_sums_that_are_infinite():
    """dw of one infinite summand is infinite, of two opposite ones NaN."""
    gu = torch.ones(3, 32, device="cuda", dtype=BF16)
    dz = torch.ones(3, 16, device="cuda", dtype=BF16)
    gu[1, 3] = INF
    gu[2, 16 + 3], gu[2, 16 + 5] = INF, -INF
    _, dw = pkg.moe_swiglu_backward(dz, gu, torch.ones(3, device="cuda"))
    assert torch.isfinite(dw[0]) and dw[1].item() == INF and torch.isnan(dw[2])
