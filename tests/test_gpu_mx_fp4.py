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


def offsets_of(counts, first=0):
    return torch.tensor([first, *(first + np.cumsum(counts))], dtype=torch.int32, device="cuda")


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


# ----------------------------------------------------------------- product --
TABLE = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                     dtype=torch.float64)


def values64(q, s):
    t = TABLE.to(q.device)
    v = torch.stack([t[(q & 15).long()], t[(q >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(s.double() - 127).repeat_interleave(32, -1)


def codes(seed, lead, K, low=126, high=128):
    """All codes, scales 2^(low - 127)..2^(high - 127): products are multiples of
    2^(2 (low - 127) - 2), so that sums of some thousand are exact in fp32."""
    q = torch.randint(0, 256, (*lead, K // 2), generator=gen(seed), device="cuda", dtype=torch.uint8)
    s = torch.randint(low, high + 1, (*lead, K // 32), generator=gen(seed + 1), device="cuda",
                      dtype=torch.uint8)
    return q, s


def reference(a, w, off, out):
    y = out.double().clone()
    for e, (i, j) in enumerate(zip(off, off[1:])):
        y[i:j] = a[i:j] @ w[e].t()
    return y


@pytest.mark.parametrize("K", [32, 64, 96, 128, 256, 288, 512, 640, 1024, 2080])
@pytest.mark.parametrize("N", [8, 64, 256, 264])
@pytest.mark.parametrize("R", [1, 33, 224, 225, 700])
def test_dense_product_exact(R, N, K):
    a, sa = codes(1, (R,), K)
    w, sw = codes(3, (N,), K)
    ref = values64(a, sa) @ values64(w, sw).t()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt in (F32, BF16):
        out = torch.full((R + 2, N), 7.0, device="cuda", dtype=dt)
        pkg.moe_matmul_fp4(a, sa, w, sw, out=out[1:-1], error_word=err)
        assert torch.equal(out[1:-1], ref.to(dt))
        assert (out[0] == 7).all() and (out[-1] == 7).all()
    assert err.item() == 0


COUNTS = [[1], [0, 3, 0], [31, 32, 33, 1, 0, 16], [223, 224, 225], [0, 0, 1000, 5, 0], [3] * 70]


@pytest.mark.parametrize("K,N", [(32, 8), (288, 264), (1024, 520)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_grouped_product_exact(counts, K, N):
    """Rows of nobody have NaN scales and are not written."""
    E, R = len(counts), sum(counts) + 5
    off = offsets_of(counts, 2)
    a, sa = codes(1, (R,), K)
    sa[:2], sa[-3:] = 255, 255
    w, sw = codes(3, (E, N), K)
    out = torch.full((R, N), 7.0, device="cuda")
    pkg.moe_matmul_fp4(a, sa, w, sw, off, out=out)
    assert torch.equal(out, reference(values64(a, sa), values64(w, sw), off.tolist(),
                                      torch.full_like(out, 7.0)).float())


@pytest.mark.parametrize("N", [8, 24, 136, 520])
@pytest.mark.parametrize("K", [32 * j for j in (1, 3, 7, 10, 13, 17, 24, 27, 31, 33, 36, 39, 62, 65, 97)])
def test_grouped_product_exact_for_any_row_of_scales(K, N):
    """Rows of scales of any length and place in memory; the tensors' last bytes
    are those of a larger one, whose others are NaN scales."""
    counts = [5, 0, 33, 1, 230]
    E, R, KG, off = len(counts), sum(counts), K // 32, offsets_of([5, 0, 33, 1, 230])
    a, sa = codes(1, (R,), K)
    w, sw = codes(3, (E, N), K)
    big = [torch.full((t.numel() + 512,), 255, device="cuda", dtype=torch.uint8) for t in (sa, sw)]
    ga, gw = (b[256:256 + t.numel()].view(t.shape).copy_(t) for b, t in zip(big, (sa, sw)))
    ref = reference(values64(a, sa), values64(w, sw), off.tolist(), torch.zeros(R, N, device="cuda"))
    out = torch.zeros(R, N, device="cuda")
    pkg.moe_matmul_fp4(a, ga, w, gw, off, out=out)
    assert torch.equal(out, ref.float())


@pytest.mark.parametrize("K", [512, 800, 1312])
def test_grouped_product_of_many_tiles_per_expert(K):
    counts, N = [2000, 0, 70, 4100], 1288
    off = offsets_of(counts)
    a, sa = codes(1, (sum(counts),), K)
    w, sw = codes(3, (4, N), K)
    out = torch.zeros(len(a), N, device="cuda")
    assert torch.equal(pkg.moe_matmul_fp4(a, sa, w, sw, off, out=out),
                       reference(values64(a, sa), values64(w, sw), off.tolist(), out * 0).float())


def test_product_every_scale():
    """Scales over their range, of either operand, the other 1: products of normal
    fp32 size scale exactly."""
    K, N = 256, 64
    a, _ = codes(1, (200,), K)
    w, _ = codes(3, (N,), K)
    one_a, one_w = (torch.full((n, K // 32), 127, device="cuda", dtype=torch.uint8) for n in (200, N))
    base = pkg.moe_matmul_fp4(a, one_a, w, one_w, out_dtype=F32).double()
    e = torch.arange(20, 220, device="cuda", dtype=torch.uint8)
    got = pkg.moe_matmul_fp4(a, e[:, None].expand(200, K // 32).contiguous(), w, one_w, out_dtype=F32)
    assert torch.equal(got.double(), base * torch.exp2(e.double() - 127)[:, None])
    e = torch.arange(90, 90 + N, device="cuda", dtype=torch.uint8)
    got = pkg.moe_matmul_fp4(a, one_a, w, e[:, None].expand(N, K // 32).contiguous(), out_dtype=F32)
    assert torch.equal(got.double(), base * torch.exp2(e.double() - 127))


def test_product_nan_scales():
    K, N = 320, 72
    a, sa = codes(1, (50,), K)
    w, sw = codes(3, (N,), K)
    base = pkg.moe_matmul_fp4(a, sa, w, sw)
    sa2, sw2, a2 = sa.clone(), sw.clone(), a.clone()
    sa2[7, 3], sw2[11, 9] = 255, 255
    a2[7, 48:64] = 0                                       # as the quantisation leaves such a block
    y = pkg.moe_matmul_fp4(a2, sa2, w, sw2)
    assert torch.isnan(y[7]).all() and torch.isnan(y[:, 11]).all()
    rows, cols = [r for r in range(50) if r != 7], [c for c in range(N) if c != 11]
    assert torch.equal(y[rows][:, cols], base[rows][:, cols])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,N,K", [(300, 520, 7168), (5, 264, 14336)])
def test_product_within_rounding(R, N, K, dtype):
    """Quantised normals.  An MMA adds 64 products; its sum and addition drop at
    most 2^-23 each of what is there; fp32 outputs add 2048 of K at a time."""
    x = torch.randn(R, K, generator=gen(1), device="cuda").to(BF16)
    v = (torch.randn(N, K, generator=gen(2), device="cuda") * 0.02).to(BF16)
    a, w = pkg.moe_quant_mx_fp4(x), pkg.moe_quant_mx_fp4(v)
    y = pkg.moe_matmul_fp4(*a, *w, out_dtype=dtype).double()
    a64, w64 = values64(*a), values64(*w)
    ref, size = a64 @ w64.t(), a64.abs() @ w64.abs().t()
    adds = 2 * K / 64 if dtype is BF16 else 2 * 32 + K / 2048
    half = U16 if dtype is BF16 else U32
    assert ((y - ref).abs() <= half * ref.abs() * (1 + 1e-3) + (adds + 2) * 2 * U32 * size).all()
    if dtype is F32:
        assert ((y - ref).norm() / ref.norm()).item() < 1e-6


def test_rows_do_not_depend_on_company():
    w, sw = codes(3, (264,), 640, 110, 140)
    a, sa = codes(1, (700,), 640, 110, 140)
    full = pkg.moe_matmul_fp4(a, sa, w, sw)
    for n in (33, 224, 511):
        assert torch.equal(pkg.moe_matmul_fp4(a[:n].clone(), sa[:n].clone(), w, sw), full[:n])
    few = pkg.moe_matmul_fp4(a[:32].clone(), sa[:32].clone(), w, sw)  # (K may be in parts)
    for n in (1, 7, 31):
        assert torch.equal(pkg.moe_matmul_fp4(a[:n].clone(), sa[:n].clone(), w, sw), few[:n])


@pytest.mark.parametrize("counts,K,N,split", [
    ([1], 7168, 4096, True), ([1, 0, 1], 14336, 520, True), ([8, 0, 8, 8, 8], 4096, 264, True),
    ([32], 2080, 2056, True), ([5] * 6, 3104, 1288, True), ([31, 1], 1024, 8, False),
    ([1] * 30, 2048, 520, False), ([33], 7168, 4096, False)])
def test_product_of_few_rows_in_parts_of_K(counts, K, N, split):
    E, R = len(counts), sum(counts)
    off = offsets_of(counts)
    a, sa = codes(1, (R,), K, 127, 128)
    w, sw = codes(3, (E, N), K, 127, 128)
    ref = reference(values64(a, sa), values64(w, sw), off.tolist(), torch.zeros(R, N, device="cuda"))
    for dt in (F32, BF16):
        out = torch.full((R + 2, N), 7.0, device="cuda", dtype=dt)
        for _ in range(5):
            pkg.moe_matmul_fp4(a, sa, w, sw, off, out=out[1:-1])
        assert torch.equal(out[1:-1], ref.to(dt)) and (out[0] == 7).all() and (out[-1] == 7).all()
    pkg.profiler_start()
    pkg.moe_matmul_fp4(a, sa, w, sw, off)
    assert list(pkg.profiler_stop()) == ["matmul_fp4" + "_split" * split]


def test_experts_forward_and_the_gradient_of_their_weight():
    """Rows quantised, multiplied by quantised experts, SiLU * up quantised and
    multiplied again; and the weight gradient from the values the codes stand
    for.  Each step against 64 bits on what the step before gave: bf16 results
    are off by 2^-9 in the mean at most, 0.4 % in the norm with room; a code of a
    z next to a border, 8 * 2^-24 wide, may be its neighbour."""
    E, H, I, counts = 4, 256, 96, [40, 0, 111, 2]
    off = offsets_of(counts)
    x = torch.randn(sum(counts), H, generator=gen(1), device="cuda").to(BF16)
    w13 = (torch.randn(E, 2 * I, H, generator=gen(2), device="cuda") * 0.1).to(BF16)
    w2 = (torch.randn(E, H, I, generator=gen(3), device="cuda") * 0.1).to(BF16)
    q13 = [t.view(E, 2 * I, -1) for t in pkg.moe_quant_mx_fp4(w13.view(-1, H))]
    q2 = [t.view(E, H, -1) for t in pkg.moe_quant_mx_fp4(w2.view(-1, I))]
    xv = torch.empty_like(x)
    xq = pkg.moe_quant_mx_fp4(x, values=xv)
    h = pkg.moe_matmul_fp4(*xq, *q13, off)
    zq = pkg.moe_quant_mx_fp4(h, swiglu=True)
    y = pkg.moe_matmul_fp4(*zq, *q2, off, out_dtype=F32)
    zeros = lambda n: torch.zeros(len(x), n, device="cuda")  # noqa: E731
    o = off.tolist()
    rh = reference(values64(*xq), values64(*q13), o, zeros(2 * I))
    assert ((h.double() - rh).norm() / rh.norm()).item() < 0.004
    # the second product from the library's codes of its own gate and up
    ry = reference(values64(*zq), values64(*q2), o, zeros(H))
    assert ((y.double() - ry).norm() / ry.norm()).item() < 1e-6
    # and the codes those of bf16 gate and up
    code, scale = oracle.quant_mx_fp4(oracle.swiglu(h.double().cpu().numpy()))
    same = (zq[0].cpu().numpy() == oracle.pack_fp4(code)).mean()
    assert same > 0.999 and (zq[1].cpu().numpy() == scale).mean() > 0.999
    dh = torch.randn(len(x), 2 * I, generator=gen(4), device="cuda").to(BF16)
    g = pkg.moe_grouped_weight_grad(xv, dh, off).double()
    rg = torch.stack([xv[i:j].double().t() @ dh[i:j].double() for i, j in zip(o, o[1:])])
    assert ((g - rg).norm() / rg.norm()).item() < 1e-6


def test_captured_calls_replay():
    K, N, counts = 640, 264, [50, 0, 300]
    off = offsets_of(counts)
    x = torch.randn(350, K, generator=gen(1), device="cuda").to(BF16)
    w = codes(3, (3, N), K)
    run = lambda: pkg.moe_matmul_fp4(*pkg.moe_quant_mx_fp4(x), *w, off)  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for seed in (5, 6):
        x.copy_(torch.randn(350, K, generator=gen(seed), device="cuda"))
        off.copy_(offsets_of([3, 300, 47] if seed == 6 else counts))
        g.replay()
        assert torch.equal(out, run())


@pytest.mark.parametrize("R,N,K", [((1 << 31) // 4096 + 700, 4096, 64),      # the output
                                   ((1 << 32) // 8192 + 700, 8, 8192),       # the rows' codes
                                   (40, (1 << 32) // 8192 + 4096, 8192)])    # the weight's
def test_product_past_32_bits(R, N, K):
    a, sa = codes(1, (R,), K, 127, 128)
    w, sw = codes(3, (N,), K, 127, 128)
    y = pkg.moe_matmul_fp4(a, sa, w, sw)
    m, n = min(R, 40), min(N, 136)
    ref = values64(a[-m:], sa[-m:]) @ values64(w[-n:], sw[-n:]).t()
    assert torch.equal(y[-m:, -n:], ref.to(BF16))


@pytest.mark.parametrize("R", [32, 40])
def test_product_of_millions_of_K_to_bf16(R):
    """Positive codes: an accumulation takes 4096 of K, 64 MMAs of a sum and an addition
    that drop at most 2^-23 each; those are added with 2^-24 each.  The mean over rows of
    different lengths, whose sums' mantissas differ, leaves the results' own roundings
    out (2^-8 / sqrt(3) / sqrt(256) = 1.4e-4); a sum of 2^22 in the tensor core alone is
    1e-3 too small."""
    K, N = 1 << 22, 8
    a, sa = codes(1, (R,), K, 127, 128)
    w, sw = codes(3, (N,), K, 127, 128)
    a &= 0x77
    w &= 0x77
    for r in range(R):
        a[r, K // 2 - r * (K // 256):] = 0
    y = pkg.moe_matmul_fp4(a, sa, w, sw).double()
    w64 = values64(w, sw)
    ref = torch.cat([values64(a[r:r + 1], sa[r:r + 1]) @ w64.t() for r in range(R)])
    err = (y - ref) / ref
    assert (err.abs() <= U16 * (1 + 1e-3) + 2 * 64 * 2 * U32 + (K / 4096 + 4) * U32).all()
    assert err.mean().abs().item() < 2.0 ** -11


def name_of(call):
    pkg.profiler_start()
    try:
        call()
    finally:
        took = pkg.profiler_stop()
    return list(took)


@pytest.mark.parametrize("K", [2048, 4128, 7168])
def test_rows_of_calls_in_parts_of_K_agree(K):
    """One weight, up to 32 rows: the parts go by K and N alone, and a row's sum, inexact
    here, is the same in any company."""
    N = 264
    w, sw = codes(3, (N,), K, 100, 150)
    a, sa = codes(1, (32,), K, 100, 150)
    few = pkg.moe_matmul_fp4(a, sa, w, sw, out_dtype=F32)
    ref = values64(a, sa) @ values64(w, sw).t()
    assert not torch.equal(few, ref.float())
    for n in (1, 7, 31, 32):
        got = []
        name = name_of(lambda: got.append(pkg.moe_matmul_fp4(a[:n].clone(), sa[:n].clone(), w, sw,
                                                             out_dtype=F32)))
        assert name == ["matmul_fp4_split"] and torch.equal(got[0], few[:n])


def test_rows_of_several_experts_in_other_numbers_of_parts():
    """Of E experts as many count as have rows at most: the parts, and with them the order
    of a row's sum, go by R too.  Either sum is within its bound (an MMA's 64 products and its
    addition drop at most 2^-23 each, 2048 of K at a time; those sums and the parts'
    are rounded to nearest)."""
    E, N, K = 8, 2056, 7168
    w, sw = codes(3, (E, N), K, 110, 140)
    a, sa = codes(1, (24,), K, 110, 140)
    off = offsets_of([3] * E)
    alone = offsets_of([1] + [0] * (E - 1))
    rows = []
    for r, o in ((24, off), (1, alone)):
        got = []
        name = name_of(lambda: got.append(pkg.moe_matmul_fp4(a[:r].clone(), sa[:r].clone(), w, sw, o,
                                                             out_dtype=F32)))
        assert name == ["matmul_fp4" + "_split" * (r == 1)]
        rows.append(got[0][:1].double())
    a64, w64 = values64(a[:1], sa[:1]), values64(w[0], sw[0])
    ref, size = a64 @ w64.t(), a64.abs() @ w64.abs().t()
    for y in rows:
        assert ((y - ref).abs() <= U32 * ref.abs() + (2 * 32 + K / 2048 + 3 + 2) * 2 * U32 * size).all()


def test_quant_swiglu_not_finite():
    """A block whose SiLU(gate) * up has a NaN or an infinity, from the inputs or by leaving
    fp32, has the NaN scale and codes of 0; blocks with far gates are those of z in 64
    bits; the blocks beside keep theirs."""
    inf, nan = float("inf"), float("nan")
    K, base = 96, 1.0
    bad = [(inf, 1.0), (-inf, 1.0), (nan, 1.0), (1.0, inf), (1.0, nan), (0.0, inf), (1e30, 1e30),
           (3e38, -3e38)]
    far = [(79.0, 2.0), (-79.0, 2.0), (81.0, 2.0), (300.0, 2.0), (-300.0, 2.0), (3e38, 0.5), (-3e38, 3.0),
           (1e30, 2.0)]
    M = len(bad) + len(far)
    x = torch.full((M, 2 * K), base, device="cuda", dtype=BF16)
    clean = pkg.moe_quant_mx_fp4(x, swiglu=True)
    for r, (g, u) in enumerate(bad + far):
        x[r, 40], x[r, K + 40] = g, u
    values = torch.empty(M, K, device="cuda", dtype=BF16)
    q, s = pkg.moe_quant_mx_fp4(x, swiglu=True, values=values)
    for t, c, per in ((q, clean[0], 16), (s, clean[1], 1)):
        assert torch.equal(t[:, :per], c[:, :per]) and torch.equal(t[:, 2 * per:], c[:, 2 * per:])
    n = len(bad)
    assert (s[:n, 1] == 255).all() and (q[:n, 16:32] == 0).all()
    assert torch.isnan(values[:n, 32:64]).all() and torch.isfinite(values[:n, :32]).all()
    # (no z here is within 8 * 2^-24 of a border)
    code, scale = oracle.quant_mx_fp4(oracle.swiglu(x[n:].double().cpu().numpy()))
    assert np.array_equal(s[n:].cpu().numpy(), scale)
    got = oracle.mx_fp4_values(q[n:].cpu().numpy(), scale)
    assert np.array_equal(got, oracle.mx_fp4_values(oracle.pack_fp4(code), scale))
    assert np.array_equal(values[n:].double().cpu().numpy(), got)
