"""GPU parity of the dense FP8 operators: group quantisation (bit-exact where
its input is), the block-scaled product (bit-exact on inputs whose sums are
exact, within its rounding bound otherwise), and the shared expert."""
import threading

import numpy as np
import pytest
import torch

import mixture_experts_ffn_softmax_gb300 as pkg
import oracle
from mixture_experts_ffn_softmax_gb300 import workloads as wl

from helpers import check_out

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def f64(t):
    return t.float().double().cpu().numpy() if t.dtype == E4M3 else t.double().cpu().numpy()


# ------------------------------------------------------------ quantisation --
QUANT = [(1, 16), (3, 112), (2, 128), (5, 144), (1, 7168), (33, 256), (129, 2048), (17, 1936),
         (1000, 384), (7, 18432)]


@pytest.mark.parametrize("M,K", QUANT)
def test_quant_groups_bit_exact(M, K):
    x = (torch.randn(M, K, generator=gen(M + K), device="cuda") * 3).to(torch.bfloat16)
    x[0, :min(K, 128)] = 0                                    # an all-zero group
    x[-1] = torch.randint(-448, 449, (K,), generator=gen(1), device="cuda").to(torch.bfloat16)
    q, s = pkg.moe_quant_groups_fp8(x)
    ref, rs = quantised(f64(x))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(f64(q), ref)


def quantised(z):
    """The oracle's groups, K padded to whole ones."""
    M, K = z.shape
    pad = np.zeros((M, -(-K // 128) * 128))
    pad[:, :K] = z
    codes, scale = oracle.quantize_groups_e4m3(pad)
    return np.asarray(codes, np.float64)[:, :K], np.asarray(scale, np.float32)


def test_quant_groups_extreme_values():
    x = torch.zeros(6, 256, device="cuda", dtype=torch.bfloat16)
    x[0, 0], x[0, 1] = 3e38, 1e30
    x[1, 0], x[1, 130] = 1e-38, 9e-41                          # subnormal scales
    x[2, 5] = float("inf")
    x[2, 6] = 1.0
    x[3, 7] = float("nan")
    x[3, 8] = 2.0
    x[4, 128:] = torch.finfo(torch.bfloat16).max
    q, s = pkg.moe_quant_groups_fp8(x)
    fin = [0, 1, 4, 5]
    ref, rs = quantised(f64(x[fin]))
    assert np.array_equal(s[fin].cpu().numpy(), rs)
    assert np.array_equal(f64(q[fin]), ref)
    assert torch.isinf(s[2, 0]) and torch.isnan(q[2, 5].float()) and q[2, 6].float() == 0
    assert torch.isnan(s[3, 0]) and torch.isnan(q[3, :128].float()).all()
    for t in (2, 3):                                           # the other group is not touched
        assert s[t, 1] == 1 and (q[t, 128:].float() == 0).all()


@pytest.mark.parametrize("M,K", QUANT)
def test_quant_groups_swiglu(M, K):
    x = (torch.randn(M, 2 * K, generator=gen(M * 3 + K), device="cuda") * 2).to(torch.bfloat16)
    q, s = pkg.moe_quant_groups_fp8(x, swiglu=True)
    z = oracle.swiglu_rows(f64(x))
    pad = np.zeros((M, -(-K // 128) * 128))
    pad[:, :K] = np.abs(z)
    amax = pad.reshape(M, -1, 128).max(2)
    scale = np.where(amax > 0, amax / 448.0, 1.0)
    # g / (1 + e) * u: expf 2, the sum, the quotient (its divisor's error
    # counts) and the product 1 each; the scale's own division 1 more
    rel = 8 * U32
    gs = s.double().cpu().numpy()
    assert (np.abs(gs - scale) <= rel * scale).all()
    cols = np.arange(K) // 128
    v = z / gs[:, cols]                 # what the codes stand for, by the scale that was given
    got = f64(q)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    assert (np.abs(got - v) <= step / 2 * (1 + 1e-6) + 2 * rel * np.abs(v)).all()


def test_quant_groups_swiglu_saturated_gates():
    """SiLU of gates far from zero: 0 * up and gate * up, no NaN from exp."""
    g = torch.tensor([-3e38, -200.0, -90.0, 0.0, 90.0, 200.0, 1e30, 1.0], device="cuda")
    x = torch.cat([g.repeat(16), torch.ones(128, device="cuda")])[None].to(torch.bfloat16)
    q, s = pkg.moe_quant_groups_fp8(x, swiglu=True)
    assert torch.isfinite(s).all() and torch.isfinite(q.float()).all()
    v = q.float()[0, :8] * s[0, 0]
    assert (v[:6] == 0).all() and abs(v[6].item() / 1e30 - 1) < 0.01
    x[0, 3], x[0, 130] = float("inf"), 2.0                    # an infinite gate, a finite up
    q, s = pkg.moe_quant_groups_fp8(x, swiglu=True)
    assert torch.isinf(s[0, 0]) and torch.isnan(q.float()[0, 3]) and q.float()[0, 2] == 0


def test_quant_groups_views_and_rows_behind():
    x = torch.randn(6, 272, generator=gen(3), device="cuda").to(torch.bfloat16)
    q = torch.full((6, 272), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((20,), -5.0, device="cuda")
    pkg.moe_quant_groups_fp8(x[1:5], q8=q[1:5], scale=s[1:13].view(4, 3))
    q2, s2 = pkg.moe_quant_groups_fp8(x[1:5].clone())
    assert torch.equal(q[1:5], q2.view(torch.uint8)) and torch.equal(s[1:13].view(4, 3), s2)
    assert (q[0] == 0x55).all() and (q[5] == 0x55).all() and (s[0] == -5) and (s[13:] == -5).all()
    assert pkg.moe_quant_groups_fp8(x[:0])[0].shape == (0, 272)


@pytest.mark.parametrize("top", [1.4e-45, 2.8e-45, 1e-43, 3.1e-43, 3.2e-43, 6e-43, 1e-42, 1e-40])
def test_quant_groups_swiglu_tiny_groups(top):
    """Groups whose largest value over 448 is below the smallest fp32 number,
    or a few of them, with zeros beside: the scale is 1 where it would be 0,
    and nothing is NaN."""
    K = 272
    up = 2.0 ** -133                                       # bf16's smallest number, 9.2e-41
    gate = 2.0 * top / up                                  # SiLU(g) is about g / 2
    x = torch.zeros(3, 2 * K, device="cuda", dtype=torch.bfloat16)
    x[0, [0, 5, 130, 271]] = gate
    x[0, K:] = up
    x[1, :K] = gate
    x[1, K:] = up
    x[1, K + 7::9] = 0.0
    x[2, 3], x[2, K + 3] = -gate, -up
    q, s = pkg.moe_quant_groups_fp8(x, swiglu=True)
    q = q.float()
    assert torch.isfinite(q).all() and torch.isfinite(s).all() and (s > 0).all()
    z = oracle.swiglu_rows(f64(x))
    pad = np.zeros((3, 384))
    pad[:, :K] = z
    amax = np.abs(pad).reshape(3, 3, 128).max(2)
    tiny = 2.0 ** -149
    got = s.double().cpu().numpy()
    sure = amax / 448.0 < 0.45 * tiny                      # 0 whatever z's own rounding
    assert (got[sure] == 1).all() and (q.cpu().numpy().reshape(3, -1)[:, :128][sure[:, 0]] == 0).all()
    # elsewhere within one of the smallest numbers of amax / 448 (z is rounded to them too)
    big = amax / 448.0 > 0.6 * tiny
    assert (np.abs(got[big] - amax[big] / 448.0) <= tiny).all()
    assert ((pad[:, :K] != 0) | (q.cpu().numpy() == 0)).all()
    # and the product of such codes stays finite
    w = torch.ones(K, 16, device="cuda").to(E4M3)
    y = pkg.moe_matmul_fp8(q.to(E4M3), s, w, torch.ones(3, 1, device="cuda"))
    assert torch.isfinite(y).all()


def test_quant_groups_swiglu_of_every_gate():
    """SiLU of every bf16 gate (those whose e^-g fp32 holds), read off the scales
    of groups that hold one gate each, with an up of 1."""
    gate = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    keep = torch.isfinite(gate) & (gate > -86) & (gate.abs() > 1e-30)
    gate = torch.where(keep, gate, torch.ones_like(gate))
    x = torch.zeros(512, 2, 128, 128, device="cuda", dtype=torch.bfloat16)
    x[:, 0, :, 5] = gate.view(512, 128)
    x[:, 1, :, 5] = 1.0
    _, s = pkg.moe_quant_groups_fp8(x.view(512, -1), swiglu=True)
    ref = np.abs(oracle.silu(f64(gate))).reshape(512, 128) / 448.0
    # 2^-h 2.5 (measured: 2.45; its share of 1 + e^-g is below 1), 1 - t, the sum,
    # the quotient and the scale's 1 each; the product with 1 is exact
    assert (np.abs(s.double().cpu().numpy() - ref) <= 6.5 * U32 * ref).all()


# ----------------------------------------------------------------- product --
SHAPES = [
    # (M, K, N)
    (1, 16, 16), (1, 128, 128), (2, 144, 272), (7, 256, 48), (16, 512, 512), (17, 400, 1040),
    (31, 1024, 256), (33, 128, 2064), (64, 2048, 1024), (65, 528, 384), (100, 896, 640),
    (128, 1024, 528), (129, 272, 144), (200, 1536, 304), (255, 384, 512), (257, 640, 272),
    (300, 2048, 1536), (513, 512, 784), (1000, 144, 2048), (1025, 1280, 912),
    (3, 4352, 10256),        # more K blocks per part than scales are held at a time
    (2601, 400, 2064), (4100, 656, 1808),   # several tiles per CTA pair
]


def exact_case(M, K, N, transposed, seed):
    """Small integers and scales that are powers of two: every product and
    partial sum is exact in fp32, so the result is known to the bit."""
    g = gen(seed)
    KB, NB = -(-K // 128), -(-N // 128)
    a = torch.randint(-4, 5, (M, K), generator=g, device="cuda").float()
    w = torch.randint(-4, 5, (K, N), generator=g, device="cuda").float()
    sa = torch.exp2(torch.randint(-2, 3, (M, KB), generator=g, device="cuda").float())
    sw = torch.exp2(torch.randint(-2, 3, (KB, NB), generator=g, device="cuda").float())
    bias = torch.randint(-64, 65, (N,), generator=g, device="cuda").float().to(torch.bfloat16)
    da = a.double() * sa.double().repeat_interleave(128, 1)[:, :K]
    dw = w.double() * sw.double().repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :N]
    y = da @ dw
    assert (y.abs() < 2.0 ** 19).all()       # multiples of 2^-4: 24 bits hold them
    wq, ws = (w.t().contiguous(), sw.t().contiguous()) if transposed else (w, sw)
    return a.to(E4M3), sa, wq.to(E4M3), ws, bias, y


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_matmul_exact_inputs(M, K, N, transposed):
    a, sa, w, sw, bias, y = exact_case(M, K, N, transposed, M + K + N)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        for b in (None, bias):
            ref = y if b is None else y + b.double()
            out = torch.full((M + 2, N), 7.0, device="cuda", dtype=dt)
            pkg.moe_matmul_fp8(a, sa, w, sw, b, transposed, out=out[1:M + 1], error_word=err)
            assert torch.equal(out[1:M + 1], ref.to(dt)), (dt, b is not None)
            assert (out[0] == 7).all() and (out[M + 1] == 7).all()
    assert err.item() == 0


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M,K,N", [(1, 7168, 512), (5, 2048, 272), (48, 1936, 640), (130, 1024, 1040),
                                   (260, 4096, 512), (520, 528, 2064)])
def test_matmul_random(M, K, N, transposed):
    g = gen(M + N)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    a, sa = pkg.moe_quant_groups_fp8(x)
    KB, NB = -(-K // 128), -(-N // 128)
    shape, sshape = ((N, K), (NB, KB)) if transposed else ((K, N), (KB, NB))
    w = torch.randn(*shape, generator=g, device="cuda").to(E4M3)
    sw = torch.rand(*sshape, generator=g, device="cuda") + 0.5
    out = pkg.moe_matmul_fp8(a, sa, w, sw, transposed=transposed, out_dtype=torch.float32)
    w64, s64 = f64(w), f64(sw)
    ref, size = oracle.matmul_blocks(f64(a), f64(sa), w64.T if transposed else w64,
                                     s64.T if transposed else s64)
    # products of E4M3 are exact in fp32; every addition of a block's sum
    # (128 at most), of the blocks and of the scales loses at most one fp32
    # step (2 U32) of a partial sum that |terms| bounds
    err = np.abs(f64(out) - ref)
    assert (err <= (128 + KB + 4) * 2 * U32 * size).all()
    # and far below the result as a whole: the additions' errors are not all of one sign
    assert np.linalg.norm(err) <= 2e-6 * np.linalg.norm(ref)
    half = pkg.moe_matmul_fp8(a, sa, w, sw, transposed=transposed)
    assert torch.equal(half, out.to(torch.bfloat16))


def test_matmul_every_code():
    """All 256 E4M3 codes against one: the value of each, NaN codes included,
    in both operands."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    vals = codes.view(E4M3).float()
    one = torch.tensor([1.0], device="cuda").to(E4M3).view(torch.uint8)
    a = torch.zeros(256, 16, dtype=torch.uint8, device="cuda")
    a[:, 3] = codes
    w = torch.zeros(16, 16, dtype=torch.uint8, device="cuda")
    w[3] = one
    sa, sw = torch.ones(256, 1, device="cuda"), torch.ones(1, 1, device="cuda")
    out = pkg.moe_matmul_fp8(a, sa, w, sw, out_dtype=torch.float32)
    assert torch.equal(torch.nan_to_num(out, nan=1e9),
                       torch.nan_to_num(vals, nan=1e9)[:, None].expand(256, 16))
    for M in (1, 16, 200):
        x = torch.zeros(M, 16, dtype=torch.uint8, device="cuda")
        x[:, 5] = one
        wt = torch.zeros(256, 16, dtype=torch.uint8, device="cuda")
        wt[:, 5] = codes
        out = pkg.moe_matmul_fp8(x, torch.ones(M, 1, device="cuda"), wt,
                                 torch.ones(2, 1, device="cuda"), transposed=True,
                                 out_dtype=torch.float32)
        assert torch.equal(torch.nan_to_num(out, nan=1e9),
                           torch.nan_to_num(vals, nan=1e9)[None].expand(M, 256))


@pytest.mark.parametrize("M", [3, 40, 300])
def test_matmul_non_finite_rows_stay_rows(M):
    a, sa, w, sw, _, y = exact_case(M, 400, 272, False, M)
    sa[1] = float("nan")
    a[2, 300] = float("nan")
    out = pkg.moe_matmul_fp8(a, sa, w, sw, out_dtype=torch.float32)
    keep = [t for t in range(M) if t not in (1, 2)]
    assert torch.isnan(out[1]).all() and torch.isnan(out[2]).all()
    assert torch.equal(out[keep], y[keep].float())


def test_matmul_repeats_to_the_bit():
    for M in (1, 24, 700):
        a, sa = pkg.moe_quant_groups_fp8(
            torch.randn(M, 4096, generator=gen(M), device="cuda").to(torch.bfloat16))
        w = torch.randn(4096, 1024, generator=gen(1), device="cuda").to(E4M3)
        sw = torch.rand(32, 8, generator=gen(2), device="cuda")
        first = pkg.moe_matmul_fp8(a, sa, w, sw, out_dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(first, pkg.moe_matmul_fp8(a, sa, w, sw, out_dtype=torch.float32))


def test_matmul_empty():
    w = torch.zeros(32, 48, dtype=torch.uint8, device="cuda")
    out = pkg.moe_matmul_fp8(torch.zeros(0, 32, dtype=torch.uint8, device="cuda"),
                             torch.zeros(0, 1, device="cuda"), w, torch.ones(1, 1, device="cuda"))
    assert out.shape == (0, 48)


@pytest.mark.parametrize("M", [1, 90, 600])
def test_dense_ops_on_other_streams_in_graphs_and_threads(M):
    H, I = 512, 384
    x = torch.randn(M, H, generator=gen(1), device="cuda").to(torch.bfloat16)
    w13 = torch.randn(H, 2 * I, generator=gen(2), device="cuda").to(E4M3)
    w2 = torch.randn(I, H, generator=gen(3), device="cuda").to(E4M3)
    s13 = torch.rand(4, 6, generator=gen(4), device="cuda") * 0.02
    s2 = torch.rand(3, 4, generator=gen(5), device="cuda") * 0.02

    def layer(h, stream=None):
        return pkg.moe_shared_expert_fp8(h, w13, w2, s13, s2, stream=stream)
    y = layer(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2 = layer(x, s)
    s.synchronize()
    assert torch.equal(y, y2)
    graphs = []
    for _ in range(2):                     # two graphs that live at once
        graph, static = torch.cuda.CUDAGraph(), torch.zeros_like(x)
        with torch.cuda.graph(graph):
            out = layer(static)
        graphs.append((graph, static, out))
    for _ in range(2):
        for graph, static, out in graphs:
            static.copy_(x)
            graph.replay()
        torch.cuda.synchronize()
        for graph, static, out in graphs:
            assert torch.equal(out, y)
            static.zero_()
    bad = []

    def run():
        st = torch.cuda.Stream()
        for _ in range(20):
            z = layer(x, st)
            st.synchronize()
            if not torch.equal(z, y):
                bad.append(1)
    ts = [threading.Thread(target=run) for _ in range(3)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_matmul_with_pdl_off():
    a, sa, w, sw, bias, y = exact_case(70, 640, 528, False, 11)
    try:
        pkg.set_pdl(False)
        out = pkg.moe_matmul_fp8(a, sa, w, sw, bias, out_dtype=torch.float32)
    finally:
        pkg.set_pdl(True)
    assert torch.equal(out, (y + bias.double()).float())


@pytest.mark.parametrize("M,K,N", [(65, 2048, 4112), (96, 1792, 4096), (150, 4096, 2064), (190, 2064, 4112)])
@pytest.mark.parametrize("transposed", [False, True])
def test_matmul_tiles_of_96_rows(M, K, N, transposed):
    a, sa, w, sw, bias, y = exact_case(M, K, N, transposed, M + K)
    out = pkg.moe_matmul_fp8(a, sa, w, sw, bias, transposed, torch.float32)
    assert torch.equal(out, (y + bias.double()).float())
    out = pkg.moe_matmul_fp8(a, sa, w, sw, transposed=transposed)
    assert torch.equal(out, y.to(torch.bfloat16))


@pytest.mark.parametrize("M,K,N", [(384, 2064, 4112), (600, 1104, 2832), (257, 2048, 7168), (1500, 400, 3200)])
@pytest.mark.parametrize("transposed", [False, True])
def test_matmul_pairs_with_narrow_tiles(M, K, N, transposed):
    """Few wide tiles, and (the last) several narrow ones per pair."""
    a, sa, w, sw, bias, y = exact_case(M, K, N, transposed, M + K)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((M + 2, N), 7.0, device="cuda", dtype=dt)
        pkg.moe_matmul_fp8(a, sa, w, sw, bias, transposed, out=out[1:M + 1], error_word=err)
        assert torch.equal(out[1:M + 1], (y + bias.double()).to(dt))
        assert (out[0] == 7).all() and (out[M + 1] == 7).all()
    assert torch.equal(pkg.moe_matmul_fp8(a, sa, w, sw, transposed=transposed), y.to(torch.bfloat16))
    assert err.item() == 0


@pytest.mark.parametrize("N", [256, 512, 1040])
@pytest.mark.parametrize("blocks", range(1, 9))
def test_matmul_pairs_of_few_blocks_back_to_back(blocks, N):
    """Fewer K blocks than stages, as many, and more, so that a pair ends with
    none, some or all of its stages in use; the next call's barriers are in the
    same shared memory at once.  (Above 8192 rows every product is of CTA pairs.)"""
    M, K = 8200, 128 * blocks - 112 * (blocks % 2)
    a, sa, w, sw, bias, y = exact_case(M, K, N, blocks % 2 == 0, blocks)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.full((M, N), 7.0, device="cuda") for _ in range(6)]
    for out in outs:
        pkg.moe_matmul_fp8(a, sa, w, sw, bias, blocks % 2 == 0, out=out, error_word=err)
    ref = (y + bias.double()).float()
    assert all(torch.equal(out, ref) for out in outs) and err.item() == 0


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("kernel,M,K,N", [
    # with more K blocks per part than scales are held at a time (16), except where it says
    ("split16", 13, 4352, 10256), ("split16", 16, 144, 16),           # (few)
    ("split32", 30, 4352, 10256), ("split32", 17, 4336, 10240),
    ("split64", 60, 4352, 10256), ("split64", 61, 2048, 4112),        # (few)
    ("split96", 90, 4592, 9712), ("split96", 96, 8192, 9728), ("split96", 90, 1936, 4112),  # (few)
    ("split128", 125, 8176, 9712), ("split128", 256, 7168, 4096), ("split128", 255, 7152, 4080),
    ("split128", 128, 5120, 9728),
    # K blocks many times the stages; several tiles per pair in the second of each
    ("pairs128", 500, 7152, 4080), ("pairs128", 12790, 2064, 384),
    ("pairs256", 8200, 7184, 512), ("pairs256", 2601, 5136, 4112)])
def test_matmul_exact_inputs_by_kernel(kernel, M, K, N, transposed):
    """Each kernel by its name, over what only many K blocks reach: the scales'
    second helping, the rings of stages and accumulators gone round."""
    a, sa, w, sw, bias, y = exact_case(M, K, N, transposed, M + K)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((M + 2, N), 7.0, device="cuda", dtype=dt)
        pkg.profiler_start()
        try:
            pkg.moe_matmul_fp8(a, sa, w, sw, bias, transposed, out=out[1:M + 1], error_word=err)
        finally:
            took = pkg.profiler_stop()
        assert list(took) == ["matmul_fp8_" + kernel]
        assert torch.equal(out[1:M + 1], (y + bias.double()).to(dt))
        assert (out[0] == 7).all() and (out[M + 1] == 7).all()
    assert err.item() == 0


@pytest.mark.parametrize("swiglu", [False, True])
def test_quant_groups_past_32_bits(swiglu):
    K = 1936
    M, n = (1 << 31) // K + 3000, 100
    x = torch.zeros(M, 2 * K if swiglu else K, device="cuda", dtype=torch.bfloat16)
    rows = torch.randn(n, x.shape[1], generator=gen(5), device="cuda").to(torch.bfloat16)
    x[:n], x[-n:] = rows, rows
    q, s = pkg.moe_quant_groups_fp8(x, swiglu)
    q0, s0 = pkg.moe_quant_groups_fp8(rows, swiglu)
    for part in (slice(0, n), slice(M - n, M)):
        assert torch.equal(q[part].view(torch.uint8), q0.view(torch.uint8))
        assert torch.equal(s[part], s0)


@pytest.mark.parametrize("M,K,N", [((1 << 31) // 4096 + 700, 272, 4096),   # the output, by pairs
                                   ((1 << 31) // 4112 + 300, 4112, 144),   # the activations
                                   (33, 4096, (1 << 19) + 4112),           # the weight, by tiles of few rows
                                   (2600, 528, 1 << 20)])                  # the output, 4096 column tiles
@pytest.mark.parametrize("transposed", [False, True])
def test_matmul_past_32_bits(M, K, N, transposed):
    """Sums that are exact and so do not depend on the kernel: the last rows and
    columns as in calls of their own."""
    g = gen(M)
    KB, NB = -(-K // 128), -(-N // 128)
    codes = torch.arange(-4, 5, device="cuda").float().to(E4M3).view(torch.uint8)

    def some(rows, cols):                      # (in parts: randint makes 64-bit numbers)
        t = torch.empty(rows, cols, device="cuda", dtype=torch.uint8)
        for p in t.split(max(1, (1 << 28) // cols)):
            p.copy_(codes[torch.randint(0, 9, p.shape, generator=g, device="cuda", dtype=torch.int32)])
        return t
    a, sa = some(M, K), torch.exp2(torch.randint(-2, 3, (M, KB), generator=g, device="cuda").float())
    shape, sshape = ((N, K), (NB, KB)) if transposed else ((K, N), (KB, NB))
    w, sw = some(*shape), torch.exp2(torch.randint(-2, 3, sshape, generator=g, device="cuda").float())
    out = pkg.moe_matmul_fp8(a, sa, w, sw, transposed=transposed)
    m, n = min(M, 37), 144
    nb = (N - n) // 128 * 128                  # whole scale blocks of columns
    if transposed:
        wn, sn = w[nb:], sw[nb // 128:]
    else:
        wn, sn = w[:, nb:].contiguous(), sw[:, nb // 128:].contiguous()
    rows = pkg.moe_matmul_fp8(a[-m:].clone(), sa[-m:].clone(), w, sw, transposed=transposed)
    cols = pkg.moe_matmul_fp8(a, sa, wn, sn, transposed=transposed)
    assert torch.equal(out[-m:], rows) and torch.equal(out[:, nb:], cols)
    wd = wn.view(E4M3).double() if not transposed else wn.view(E4M3).double().t()
    sd = (sn if not transposed else sn.t()).double()
    ref = (a[-m:].view(E4M3).double() * sa[-m:].double().repeat_interleave(128, 1)[:, :K]) @ (
        wd * sd.repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :N - nb])
    assert torch.equal(rows[:, nb:], ref.to(torch.bfloat16))


# ----------------------------------------------------------- together --
def shared_oracle(x, w13, w2, s13, s2, b13=None, b2=None):
    q, s = quantised(x)
    h, _ = oracle.matmul_blocks(q, s, w13, s13, b13)
    z = oracle.swiglu_rows(oracle.bf16_round(h))
    zq, zs = quantised(np.asarray(z, np.float32).astype(np.float64))
    return oracle.matmul_blocks(zq, zs, w2, s2, b2)[0]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M", [1, 19, 200, 777])
def test_shared_expert(M, transposed):
    H, I = 640, 272
    x = torch.randn(M, H, generator=gen(M), device="cuda").to(torch.bfloat16)
    w13 = torch.randn(H, 2 * I, generator=gen(2), device="cuda").to(E4M3)
    w2 = torch.randn(I, H, generator=gen(3), device="cuda").to(E4M3)
    s13 = torch.rand(5, 5, generator=gen(4), device="cuda") * 0.04
    s2 = torch.rand(3, 5, generator=gen(5), device="cuda") * 0.04
    b13 = torch.randn(2 * I, generator=gen(6), device="cuda").to(torch.bfloat16) * 0.1
    b2 = torch.randn(H, generator=gen(7), device="cuda").to(torch.bfloat16) * 0.1
    t = (lambda v: v.t().contiguous()) if transposed else (lambda v: v)
    y = pkg.moe_shared_expert_fp8(x, t(w13), t(w2), t(s13), t(s2), b13, b2, transposed)
    ref = shared_oracle(f64(x), f64(w13), f64(w2), f64(s13), f64(s2), f64(b13), f64(b2))
    check_out(y.double().cpu().numpy(), ref, "shared expert")


def test_fp8_layer_with_bias_routing_and_shared_expert():
    """The operators as a DeepSeek-style layer runs them: router logits, the
    biased routing, the routed experts in FP8, the shared expert, and the
    routing's gradient for the router."""
    spec = wl.SMALL_SPECS["deepseek_small"]
    d = wl.make_moe_inputs(spec, device="cuda", weights=False)
    M, H, I, E = spec.M, spec.H, spec.I, spec.E
    g = gen(20)
    w_gate = (torch.randn(H, E, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    bias = torch.randn(E, generator=g, device="cuda") * 0.05
    w13 = torch.randn(E, H, 2 * I, generator=g, device="cuda").to(E4M3)
    w2 = torch.randn(E, I, H, generator=g, device="cuda").to(E4M3)
    s13 = torch.rand(E, H // 128, 2 * I // 128, generator=g, device="cuda") * 0.04
    s2 = torch.rand(E, I // 128, H // 128, generator=g, device="cuda") * 0.04
    x = d["hidden"]
    logits = pkg.moe_router_logits(x, w_gate)
    w, ids = pkg.moe_route(logits, spec.top_k, spec.routing_method, True, spec.k_group,
                           spec.group_count, spec.group_select_mode,
                           spec.routed_scaling_factor, score_bias=bias)
    routed = pkg.moe_forward_fp8(x, w, ids, w13, w2, s13, s2)
    shared = pkg.moe_shared_expert_fp8(x, w13[0], w2[0], s13[0], s2[0])
    rw, rids = oracle.route_biased(f64(logits), f64(bias), spec.top_k, spec.routing_method, True,
                                   spec.k_group, spec.group_count, spec.group_select_mode,
                                   spec.routed_scaling_factor)
    assert np.array_equal(ids.cpu().numpy(), rids)
    used = sorted(set(rids.reshape(-1)))
    local = {e: i for i, e in enumerate(used)}
    lids = np.vectorize(local.get)(rids)
    f = lambda v: f64(v[torch.tensor(used, device="cuda")])  # noqa: E731
    ref = oracle.forward_fp8_block(f64(x), rw, lids, f(w13.float()), f(w2.float()), f(s13), f(s2))
    check_out(routed.double().cpu().numpy(), ref, "routed experts")
    sref = shared_oracle(f64(x), f64(w13[0]), f64(w2[0]), f64(s13[0]), f64(s2[0]))
    check_out(shared.double().cpu().numpy(), sref, "shared expert")
    gw = torch.randn(M, spec.top_k, generator=g, device="cuda")
    gl = pkg.moe_route_backward(gw, logits, ids, spec.routing_method, True,
                                spec.routed_scaling_factor)
    gref = oracle.route_backward(f64(gw), f64(logits), rids, spec.routing_method, True,
                                 spec.routed_scaling_factor)
    assert np.linalg.norm(f64(gl) - gref) <= 1e-5 * np.linalg.norm(gref)
