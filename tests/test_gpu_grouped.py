"""GPU parity of the products of rows sorted by expert and their weight
gradients: bit-exact on integers whose sums are exact, within rounding bounds
otherwise; and the training step of a layer made of them."""
import os
import threading

import numpy as np
import pytest
import torch

import mixture_experts_ffn_softmax_gb300 as pkg

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U16, U32 = 2.0 ** -8, 2.0 ** -24        # half a step, relative


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(seed, *shape, top=2):
    """bf16 integers in -top..top: sums of up to 2^24 / top^2 products are exact."""
    return torch.randint(-top, top + 1, shape, generator=gen(seed), device="cuda").to(BF16)


def offsets_of(counts, first=0):
    return torch.tensor([first, *(first + np.cumsum(counts))], dtype=torch.int32, device="cuda")


def reference(x, w, offsets, out, transposed=False, bias=None):
    y = out.double().clone()
    o = offsets.tolist()
    for e, (a, b) in enumerate(zip(o, o[1:])):
        m = w[e].double()
        y[a:b] = x[a:b].double() @ (m.t() if transposed else m)
        if bias is not None:
            y[a:b] += bias[e].double()
    return y.to(out.dtype)


def weight_reference(x, dy, offsets):
    o = offsets.tolist()
    return torch.stack([x[a:b].double().t() @ dy[a:b].double() for a, b in zip(o, o[1:])])


# no rows, one, either side of what the MMA and a tile take, many experts, one with all rows
COUNTS = [[1], [0, 3, 0], [31, 32, 33, 1, 0, 16], [255, 256, 257], [0, 0, 1000, 5, 0],
          [300, 1, 513], [3] * 70, [0] * 40 + [7]]
SIZES = [(8, 8), (64, 64), (72, 256), (136, 264), (520, 136), (1000, 520)]


# ------------------------------------------------------------------ product --
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("K,N", SIZES)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_product_exact(counts, K, N, transposed):
    """Rows that belong to nobody, before and behind the groups, hold NaN and
    are not written; both output types; with and without a bias."""
    E, R = len(counts), sum(counts) + 5
    off = offsets_of(counts, 2)
    x = ints(1, R, K)
    x[:2], x[-3:] = float("nan"), float("nan")
    w = ints(2, E, N, K) if transposed else ints(2, E, K, N)
    bias = ints(3, E, N)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt, b in ((BF16, None), (F32, bias)):
        out = torch.full((R, N), 7.0, device="cuda", dtype=dt)
        got = pkg.moe_grouped_matmul(x, w, off, bias=b, transposed=transposed, out=out,
                                     error_word=err)
        assert got is out
        ref = reference(x, w, off, torch.full_like(out, 7.0), transposed, b)
        assert torch.equal(out, ref)
    assert err.item() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K,N,counts", [(4096, 512, [700, 0, 90]), (14336, 256, [20, 12]),
                                        (520, 264, [33, 1, 300])])
def test_product_within_rounding(K, N, counts, dtype):
    """fp32 sums: an MMA adds 16 products, whose sum and addition each drop at
    most 2^-23 of what is there (truncation, twice the rounding's half step);
    in fp32 outputs at most 32 such additions follow one another before the sum
    is added in a register with 2^-24."""
    x = torch.randn(sum(counts), K, generator=gen(K), device="cuda").to(BF16)
    w = (torch.randn(len(counts), K, N, generator=gen(N), device="cuda") * 0.02).to(BF16)
    off = offsets_of(counts)
    y = pkg.moe_grouped_matmul(x, w, off, out_dtype=dtype).double()
    z = torch.zeros(len(x), N, device="cuda", dtype=torch.float64)
    ref, size = reference(x, w, off, z), reference(x.abs(), w.abs(), off, z)
    adds = 2 * K / 16 if dtype is BF16 else 2 * 32 + K / 512
    half = U16 if dtype is BF16 else U32
    assert ((y - ref).abs() <= half * ref.abs() * (1 + 1e-3) + (adds + 2) * 2 * U32 * size).all()
    if dtype is F32:
        # the additions' truncation has one sign; 1.0e-9 of the sum per K without the registers
        assert ((y - ref).norm() / ref.norm()).item() < 1e-6


def test_product_of_many_experts_and_ragged_rows():
    rng = np.random.default_rng(0)
    counts = rng.integers(0, 9, 1024) * (rng.random(1024) < 0.4)
    counts[[0, 511, 1023]] = 300, 0, 1
    x, w, off = ints(4, int(counts.sum()), 64), ints(5, 1024, 64, 72), offsets_of(counts)
    out = torch.zeros(len(x), 72, device="cuda")
    assert torch.equal(pkg.moe_grouped_matmul(x, w, off, out=out), reference(x, w, off, out * 0))


@pytest.mark.parametrize("transposed", [False, True])
def test_product_of_many_tiles_per_expert(transposed):
    """Rows and columns past a raster group of 8 row tiles, twice round every pair."""
    counts, K, N = [2400, 0, 70, 4500], 136, 1288
    x, off = ints(1, sum(counts), K), offsets_of(counts)
    w = ints(2, 4, N, K) if transposed else ints(2, 4, K, N)
    out = torch.zeros(len(x), N, device="cuda")
    assert torch.equal(pkg.moe_grouped_matmul(x, w, off, transposed=transposed, out=out),
                       reference(x, w, off, out * 0, transposed))


def test_weight_grad_of_many_tiles_per_expert():
    counts, K, N = [40, 0, 65, 700], 2312, 1032
    x, dy, off = ints(1, sum(counts), K), ints(2, sum(counts), N), offsets_of(counts)
    for dt in (F32, BF16):
        assert torch.equal(pkg.moe_grouped_weight_grad(x, dy, off, out_dtype=dt),
                           weight_reference(x, dy, off).to(dt))


def test_product_rows_do_not_touch_each_other():
    """A row's NaN or infinity stays in its own output row, an expert's weight in
    its own rows."""
    x, w, off = ints(6, 90, 128), ints(7, 3, 128, 64), offsets_of([40, 10, 40])
    y = pkg.moe_grouped_matmul(x, w, off)
    x2, w2 = x.clone(), w.clone()
    x2[41, 3], x2[0, 0] = float("nan"), float("inf")
    w2[1, 5, 7] = float("inf")
    y2 = pkg.moe_grouped_matmul(x2, w2, off)
    assert torch.isnan(y2[41]).all() and not torch.isfinite(y2[0]).any()  # inf * 0 is NaN
    rows = [r for r in range(90) if r not in (0, 41)]
    cols = [c for c in range(64) if c != 7]
    assert torch.equal(y2[rows][:, cols], y[rows][:, cols])
    assert torch.equal(y2[1:40], y[1:40]) and torch.equal(y2[50:], y[50:])


def test_product_same_rows_in_any_company():
    """A row's result does not depend on the rows beside it (as a padded batch
    and its unpadded form have to agree), but for K being summed in parts in
    calls of up to 32 rows in all: those agree among themselves."""
    w = torch.randn(1, 1024, 264, generator=gen(8), device="cuda").to(BF16)
    x = torch.randn(700, 1024, generator=gen(9), device="cuda").to(BF16)
    full = pkg.moe_grouped_matmul(x, w, offsets_of([700]))
    for n in (33, 256, 511):
        assert torch.equal(pkg.moe_grouped_matmul(x[:n].clone(), w, offsets_of([n])), full[:n])
    few = pkg.moe_grouped_matmul(x[:32].clone(), w, offsets_of([32]))
    for n in (1, 7, 31):
        assert torch.equal(pkg.moe_grouped_matmul(x[:n].clone(), w, offsets_of([n])), few[:n])


def name_of(call):
    pkg.profiler_start()
    try:
        call()
    finally:
        took = pkg.profiler_stop()
    return list(took)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts,K,N,split", [
    ([1], 7168, 4096, True), ([1, 0, 1], 14336, 520, True), ([8, 0, 8, 8, 8], 4096, 264, True),
    ([32], 1000, 2056, True), ([5] * 6, 2048, 1288, True), ([31, 1], 264, 8, False),
    ([1] * 30, 1024, 520, False), ([33], 7168, 4096, False)])
def test_product_of_few_rows_in_parts_of_K(counts, K, N, split, transposed):
    E, R = len(counts), sum(counts) + 3
    off = offsets_of(counts, 1)
    x = ints(1, R, K)
    x[0], x[-2:] = float("nan"), float("inf")
    w = ints(2, E, N, K) if transposed else ints(2, E, K, N)
    bias = ints(3, E, N)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # (rows of nobody count among the 32)
    few = split and R <= 32
    for dt, b in ((BF16, None), (F32, bias)):
        out = torch.full((R, N), 7.0, device="cuda", dtype=dt)
        name = name_of(lambda: pkg.moe_grouped_matmul(x, w, off, bias=b, transposed=transposed,
                                                      out=out, error_word=err))
        assert name == ["grouped_matmul" + "_t" * transposed + "_split" * few]
        assert torch.equal(out, reference(x, w, off, torch.full_like(out, 7.0), transposed, b))
    inner = slice(1, R - 2)
    out = torch.full((R - 3, N), 7.0, device="cuda")
    name = name_of(lambda: pkg.moe_grouped_matmul(x[inner].clone(), w, off - 1, transposed=transposed,
                                                  out=out, error_word=err))
    assert name == ["grouped_matmul" + "_t" * transposed + "_split" * split]
    assert torch.equal(out, reference(x[inner], w, off - 1, out, transposed))
    assert err.item() == 0


def test_few_rows_back_to_back():
    """Calls whose clusters follow one another, of other parts and sizes."""
    cases = []
    for i, (counts, K, N) in enumerate([([1], 7168, 4096), ([2, 3], 1024, 264), ([32], 2048, 2056),
                                        ([1, 1], 4096, 1032), ([9], 520, 520)]):
        x, w, off = ints(i, sum(counts), K), ints(9 + i, len(counts), K, N), offsets_of(counts)
        ref = reference(x, w, off, torch.zeros(len(x), N, device="cuda"))
        cases.append((x, w, off, ref, [torch.zeros(len(x), N, device="cuda") for _ in range(8)]))
    for r in range(8):
        for x, w, off, _, outs in cases:
            pkg.moe_grouped_matmul(x, w, off, out=outs[r])
    assert all(torch.equal(o, ref) for _, _, _, ref, outs in cases for o in outs)


def test_empty_calls():
    w, off = ints(1, 2, 64, 32), offsets_of([0, 0])
    assert pkg.moe_grouped_matmul(ints(2, 0, 64), w, off).shape == (0, 32)
    out = torch.full((2, 64, 32), 5.0, device="cuda")
    pkg.moe_grouped_weight_grad(ints(2, 0, 64), ints(3, 0, 32), off, out=out, accumulate=True)
    assert (out == 5).all()
    pkg.moe_grouped_weight_grad(ints(2, 0, 64), ints(3, 0, 32), off, out=out)
    assert (out == 0).all()
    rest = pkg.moe_grouped_matmul(ints(2, 4, 64), w, off, out=torch.full((4, 32), 3.0, device="cuda"))
    assert (rest == 3).all()


@pytest.mark.parametrize("bad", [[0, 5, 3, 8], [-2, 3, 4, 8], [0, 3, 4, 9], [4, 3, 2, 1],
                                 [0, 8, 0, 8], [-2 ** 31, 2 ** 31 - 1, 5, 2 ** 31 - 1]])
def test_offsets_out_of_order_or_range_set_the_error_word(bad):
    x, w, dy = ints(1, 8, 64), ints(2, 3, 64, 32), ints(3, 8, 32)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    guard = torch.full((3, 8, 32), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkg.moe_grouped_matmul(x, w, off, out=guard[1], error_word=err)
    assert err.item() == 1 and (guard[0] == 7).all() and (guard[2] == 7).all()
    # clipped to the rows there are and to the ends of the experts before
    groups, end = [], 0
    for a, b in zip(bad, bad[1:]):
        a = max(min(max(a, 0), 8), end)
        b = max(min(max(b, 0), 8), a)
        end = max(end, b)
        groups.append((a, b))
    ref = torch.full((8, 32), 7.0, device="cuda", dtype=torch.float64)
    for e, (a, b) in enumerate(groups):
        ref[a:b] = x[a:b].double() @ w[e].double()
    assert torch.equal(guard[1].double(), ref)
    err.zero_()
    g = pkg.moe_grouped_weight_grad(x, dy, off, error_word=err)
    assert err.item() == 1
    for e, (a, b) in enumerate(groups):
        assert torch.equal(g[e].double(), x[a:b].double().t() @ dy[a:b].double())


# ---------------------------------------------------------- weight gradient --
@pytest.mark.parametrize("K,N", [(8, 8), (64, 136), (136, 64), (264, 264), (520, 8)])
@pytest.mark.parametrize("counts", [[1], [0, 15, 16, 17], [63, 64, 65, 0, 1], [200, 0, 448, 33],
                                    [3] * 70, [1000]], ids=lambda c: f"{len(c)}x{max(c)}")
def test_weight_grad_exact(counts, K, N):
    """Rows of nobody hold NaN, as do x and dy of other experts' rows in turn:
    neither reaches an expert's sum."""
    E, R = len(counts), sum(counts) + 5
    off = offsets_of(counts, 2)
    x, dy = ints(1, R, K), ints(2, R, N)
    for t in (x, dy):
        t[:2], t[-3:] = float("nan"), float("inf")
    ref = weight_reference(x, dy, off)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt in (F32, BF16):
        out = torch.full((E, K, N), 9.0, device="cuda", dtype=dt)
        pkg.moe_grouped_weight_grad(x, dy, off, out=out, error_word=err)
        assert torch.equal(out, ref.to(dt))
        pkg.moe_grouped_weight_grad(x, dy, off, out=out, accumulate=True, error_word=err)
        assert torch.equal(out, (ref.to(dt).double() + ref).to(dt))
    o = off.tolist()
    for e in range(0, E, max(1, E // 3)):
        if counts[e]:
            x2, dy2 = x.clone(), dy.clone()
            x2[o[e]:o[e + 1]], dy2[o[e + 1] - 1] = float("nan"), float("inf")
            got = pkg.moe_grouped_weight_grad(x2, dy2, off)
            others = [i for i in range(E) if i != e]
            assert torch.isnan(got[e]).all() and torch.equal(got[others].double(), ref[others])
    assert err.item() == 0


@pytest.mark.parametrize("counts,K,N,split", [
    ([1536], 520, 264, True), ([1601], 1000, 1032, True), ([5000, 1, 0], 264, 136, True),
    ([0, 3500], 72, 8, True), ([5, 6000, 77, 500], 512, 520, True), ([1535], 264, 264, False),
    ([4000], 2560, 2048, False), ([4096] * 2, 1536, 768, True)])
def test_weight_grad_of_few_tiles_in_parts_of_the_rows(counts, K, N, split):
    """Sums over rows that the pairs of a cluster share: parts without rows, rows
    that end inside a stage, tiles of 128 columns and of fewer, both output
    types, added to what is there, the same bits in calls one behind the other."""
    E, R = len(counts), sum(counts)
    off = offsets_of(counts, 3)
    x, dy = ints(1, R + 5, K, top=1), ints(2, R + 5, N, top=1)
    for t in (x, dy):
        t[:3], t[-2:] = float("nan"), float("inf")
    ref = weight_reference(x, dy, off)
    name = name_of(lambda: pkg.moe_grouped_weight_grad(x, dy, off))
    # (rows of nobody count among those that decide)
    assert name == ["grouped_weight_grad" + "_split" * (split or R == 1535)]
    x2, dy2, off2 = x[3:-2].clone(), dy[3:-2].clone(), off - 3
    assert name_of(lambda: pkg.moe_grouped_weight_grad(x2, dy2, off2)) == [
        "grouped_weight_grad" + "_split" * split]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt in (F32, BF16):
        outs = [torch.full((E, K, N), 9.0, device="cuda", dtype=dt) for _ in range(6)]
        for i, out in enumerate(outs):
            a = (x, dy, off) if i % 2 else (x2, dy2, off2)
            pkg.moe_grouped_weight_grad(*a, out=out, error_word=err)
        assert all(torch.equal(out, ref.to(dt)) for out in outs)
        pkg.moe_grouped_weight_grad(x, dy, off, out=outs[0], accumulate=True, error_word=err)
        assert torch.equal(outs[0], (ref.to(dt).double() + ref).to(dt))
    assert err.item() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weight_grad_within_rounding(dtype):
    """As for the product, the reduced side being an expert's rows: up to 20000."""
    counts, K, N = [20000, 37, 900], 264, 136
    x = torch.randn(sum(counts), K, generator=gen(1), device="cuda").to(BF16)
    dy = torch.randn(sum(counts), N, generator=gen(2), device="cuda").to(BF16)
    off = offsets_of(counts)
    got = pkg.moe_grouped_weight_grad(x, dy, off, out_dtype=dtype).double()
    ref, size = weight_reference(x, dy, off), weight_reference(x.abs(), dy.abs(), off)
    for e, m in enumerate(counts):
        adds = 2 * m / 16 if dtype is BF16 else 2 * 32 + m / 512
        half = U16 if dtype is BF16 else U32
        bound = half * ref[e].abs() * (1 + 1e-3) + (adds + 2) * 2 * U32 * size[e]
        assert ((got[e] - ref[e]).abs() <= bound).all()
        if dtype is F32:
            assert ((got[e] - ref[e]).norm() / ref[e].norm()).item() < 1e-6


# ----------------------------------------------------------------- together --
def sorted_rows(ids, E):
    """Items sorted by expert and the experts' offsets, as moe_align orders them."""
    plan = pkg.moe_align(ids, E, block_m=1)
    return plan["sorted_token_ids"].long(), plan["expert_offsets"]


@pytest.mark.parametrize("M,H,I,E,k", [(37, 128, 72, 6, 2), (200, 264, 136, 16, 4)])
def test_training_step_of_a_layer(M, H, I, E, k):
    """Routing, the experts forward and backward, the router's gradient: against
    autograd in 64 bits on the same weights.  Intermediate tensors are bf16: gate
    and up, z, dz, their gradients, a rounding of 2^-9 of each element on either
    side of products that average them, so that the relative error of a result
    in the norm is a few times 2^-9 (0.2 %); 1.5 % allows for seven of them."""
    f = lambda s, *shape: (torch.randn(*shape, generator=gen(s), device="cuda") * 0.3).to(BF16)  # noqa: E731
    x, w13, w2, logits, dy = (f(1, M, H), f(2, E, H, 2 * I), f(3, E, I, H), f(4, M, E).float() * 4,
                              f(5, M, H))
    weights, ids = pkg.moe_route(logits, k, "softmax", renormalize=True)
    order, off = sorted_rows(ids, E)
    token = order // k
    row_w = weights.reshape(-1)[order].contiguous()
    xs, dys = x[token], dy[token]
    gate_up = pkg.moe_grouped_matmul(xs, w13, off)
    z = pkg.moe_swiglu(gate_up, row_w)
    y = torch.zeros(M, H, device="cuda").index_add_(0, token, pkg.moe_grouped_matmul(
        z, w2, off, out_dtype=F32))
    dz = pkg.moe_grouped_matmul(dys, w2, off, transposed=True)
    dgu, drow = pkg.moe_swiglu_backward(dz, gate_up, row_w)
    dw2 = pkg.moe_grouped_weight_grad(z, dys, off)
    dw13 = pkg.moe_grouped_weight_grad(xs, dgu, off)
    dx = torch.zeros(M, H, device="cuda").index_add_(0, token, pkg.moe_grouped_matmul(
        dgu, w13, off, transposed=True, out_dtype=F32))
    gw = torch.empty_like(weights)
    gw.view(-1)[order] = drow
    dl = pkg.moe_route_backward(gw, logits, ids, "softmax", renormalize=True)

    t = [v.double().requires_grad_() for v in (x, w13, w2, logits)]
    p = torch.softmax(t[3], 1).gather(1, ids.long())
    p = p / p.sum(1, keepdim=True)
    h = torch.einsum("mh,mkhi->mki", t[0], t[1][ids.long()])
    a = torch.nn.functional.silu(h[..., :I]) * h[..., I:] * p[..., None]
    ry = torch.einsum("mki,mkih->mh", a, t[2][ids.long()])
    (ry * dy.double()).sum().backward()
    for got, ref in ((y, ry.detach()), (dx, t[0].grad), (dw13, t[1].grad), (dw2, t[2].grad),
                     (dl, t[3].grad)):
        assert ((got.double() - ref).norm() / ref.norm()).item() < 0.015
    # the library's own forward of the layer
    own = pkg.moe_forward(x, weights, ids, w13, w2)
    assert ((own.double() - y.double()).norm() / y.double().norm()).item() < 0.015


def step(x, w, dy, off):
    y = pkg.moe_grouped_matmul(x, w, off)
    d = pkg.moe_grouped_matmul(dy, w, off, transposed=True)
    z = pkg.moe_swiglu(y)
    g, _ = pkg.moe_swiglu_backward(z, y)
    return y, d, z, g, pkg.moe_grouped_weight_grad(x, dy, off)


def step_inputs(seed, counts=(40, 0, 300, 7)):
    R = sum(counts)
    return (torch.randn(R, 136, generator=gen(seed), device="cuda").to(BF16),
            torch.randn(len(counts), 136, 272, generator=gen(seed + 1), device="cuda").to(BF16),
            torch.randn(R, 272, generator=gen(seed + 2), device="cuda").to(BF16),
            offsets_of(list(counts)))


def test_captured_steps_replay_on_new_inputs():
    """Two captured graphs of the same calls, replayed in turn and with other
    offsets, equal eager calls bit for bit."""
    a, b = step_inputs(1), step_inputs(50, (0, 347, 0, 0))
    static = [t.clone() for t in a]
    graphs, outs = [], []
    step(*static)
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*static))
        graphs.append(g)
    for inputs in (a, b, a):
        for s, t in zip(static, inputs):
            s.copy_(t)
        for g in graphs:
            g.replay()
        ref = step(*inputs)
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(o, r) for o, r in zip(out, ref))


def test_streams_and_threads():
    """Calls on streams of the caller's and from several host threads."""
    inputs = [step_inputs(10 * i) for i in range(3)]
    refs = [step(*i) for i in inputs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x, w, dy, off = inputs[0]
    s.wait_stream(torch.cuda.current_stream())
    y = pkg.moe_grouped_matmul(x, w, off, stream=s)
    g = pkg.moe_grouped_weight_grad(x, dy, off, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, refs[0][0]) and torch.equal(g, refs[0][4])
    bad = []

    def run(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(20):
                out = step(*inputs[i])
        st.synchronize()
        if not all(torch.equal(o, r) for o, r in zip(out, refs[i])):
            bad.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_repeated_calls_give_the_same_bits():
    inputs = step_inputs(77, (1000, 3, 0, 900))
    ref = step(*inputs)
    for _ in range(10):
        assert all(torch.equal(o, r) for o, r in zip(step(*inputs), ref))


@pytest.mark.parametrize("counts,K,N", [([(1 << 31) // 4096 + 700], 64, 4096),       # the output
                                        ([(1 << 31) // 4096 + 700], 4096, 8),        # the rows
                                        ([5, 300], 4096, (1 << 19) + 4096)])         # the weight
def test_product_past_32_bits(counts, K, N):
    R, off = sum(counts), offsets_of(counts)
    x = torch.empty(R, K, device="cuda", dtype=BF16)
    w = torch.empty(len(counts), K, N, device="cuda", dtype=BF16)
    for t in (x, w):
        for p in t.view(-1).split(1 << 28):
            p.copy_(torch.randint(-1, 2, p.shape, generator=gen(1), device="cuda", dtype=torch.int8))
    y = pkg.moe_grouped_matmul(x, w, off)
    m, n = min(R, 40), min(N, 136)
    e = len(counts) - 1
    ref = x[-m:].double() @ w[e, :, -n:].double()
    assert torch.equal(y[-m:, -n:], ref.to(BF16))


def test_weight_grad_past_32_bits():
    R, K, N = (1 << 31) // 2048 + 100, 2048, 8
    x = torch.zeros(R, K, device="cuda", dtype=BF16)
    dy = torch.zeros(R, N, device="cuda", dtype=BF16)
    x[-50:], dy[-50:] = ints(1, 50, K), ints(2, 50, N)
    off = torch.tensor([0, R - 30, R], dtype=torch.int32, device="cuda")
    got = pkg.moe_grouped_weight_grad(x, dy, off)
    assert torch.equal(got[1].double(), x[-30:].double().t() @ dy[-30:].double())
    assert torch.equal(got[0].double(), x[-50:-30].double().t() @ dy[-50:-30].double())
    E, K, N = 40, 8192, 8192                                    # the output: 2.7e9 elements
    x, dy = ints(3, E * 2, K), ints(4, E * 2, N)
    got = pkg.moe_grouped_weight_grad(x, dy, offsets_of([2] * E), out_dtype=BF16)
    assert torch.equal(got[-1], (x[-2:].double().t() @ dy[-2:].double()).to(BF16))


# --------------------------------------------------------------- long sums --
def long_sum_error(y, ref, adds, rounded):
    """Of a bf16 result whose summands all have one sign: it is the rounded fp32
    sum, whose own error is `adds` additions within an accumulation that drop at
    most 2^-23 each and `rounded` of those behind one another, 2^-24 each.  The mean
    over results of many different mantissas: their roundings, of either sign, go
    out of it (2^-8 / sqrt(3) / sqrt(elements): 4e-5 for 4096, 1.3e-4 for 320)."""
    err = (y.double() - ref) / ref
    slack = adds * 2 * U32 + rounded * U32
    assert (err.abs() <= U16 * (1 + 1e-3) + slack).all()
    assert err.mean().abs().item() < 2.0 ** -10


def positive(seed, *shape):
    """bf16 in [0.5, 1.5), made in pieces."""
    t = torch.empty(*shape, device="cuda", dtype=BF16)
    g = gen(seed)
    for p in t.view(-1).split(1 << 27):
        p.copy_(torch.rand(p.shape, generator=g, device="cuda") + 0.5)
    return t


@pytest.mark.parametrize("counts", [[1 << 23], [1 << 22, 0, (1 << 23) - 77]])
def test_weight_grad_of_millions_of_rows_to_bf16(counts):
    """An accumulation takes 1024 rows, 64 MMAs: the error does not grow with the rows
    as that of the tensor core's truncating sum does (8e-3 for 2^23)."""
    K = N = 64
    x, dy = positive(1, sum(counts), K), positive(2, sum(counts), N)
    x[:, 1::2] *= 0.7109375
    dy[:, 1::2] *= 0.8515625
    off = offsets_of(counts)
    y = pkg.moe_grouped_weight_grad(x, dy, off, out_dtype=BF16)
    o = off.tolist()
    for e, (a, b) in enumerate(zip(o, o[1:])):
        if a == b:
            assert (y[e] == 0).all()
            continue
        ref = sum(x[i:min(i + (1 << 20), b)].double().t() @ dy[i:min(i + (1 << 20), b)].double()
                  for i in range(a, b, 1 << 20))
        long_sum_error(y[e], ref, 2 * 64, counts[e] / 1024 + 4)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("R", [32, 40])
def test_product_of_millions_of_K_to_bf16(R, transposed):
    """As above, K in parts (32 rows) and not; rows of different lengths, so that their
    sums' mantissas differ."""
    K, N = 1 << 22, 8
    x = positive(1, R, K)
    for r in range(R):
        x[r, K - r * (K // 128):] = 0
    w = positive(2, 1, N, K) if transposed else positive(2, 1, K, N)
    y = pkg.moe_grouped_matmul(x, w, offsets_of([R]), transposed=transposed)
    m = w[0].double()
    long_sum_error(y, x.double() @ (m.t() if transposed else m), 2 * 64, K / 1024 + 4)


def test_rows_of_calls_in_parts_of_K_agree():
    """One weight, up to 32 rows: the parts go by K and N alone.  With several experts
    they go by R too; a row's sum is then within its bound (see
    test_product_within_rounding) in either company."""
    K, N = 4096, 520
    w = torch.randn(8, K, N, generator=gen(1), device="cuda").to(BF16)
    x = torch.randn(32, K, generator=gen(2), device="cuda").to(BF16)
    z = torch.zeros(32, N, device="cuda", dtype=torch.float64)
    one = offsets_of([32])
    few = pkg.moe_grouped_matmul(x, w[:1], one, out_dtype=F32)
    ref, size = reference(x, w, one, z), reference(x.abs(), w.abs(), one, z)
    assert not torch.equal(few, ref.float())
    bound = U32 * ref.abs() + (2 * 32 + K / 512 + 3 + 2) * 2 * U32 * size
    for n in (1, 7, 31, 32):
        got = []
        assert name_of(lambda: got.append(pkg.moe_grouped_matmul(
            x[:n].clone(), w[:1], offsets_of([n]), out_dtype=F32))) == ["grouped_matmul_split"]
        assert torch.equal(got[0], few[:n])
    for counts in ([1] + [0] * 7, [2] * 8, [4] * 8):
        y = pkg.moe_grouped_matmul(x[:sum(counts)].clone(), w, offsets_of(counts), out_dtype=F32)
        assert ((y[0].double() - ref[0]).abs() <= bound[0]).all()


def test_training_step_as_documented():
    """The README's step: against autograd in 64 bits (1.5 % in the norm, see
    test_training_step_of_a_layer), and the same bits in every run: a token's rows are
    added in a fixed order, in fp32."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        text = f.read()
    code = text[text.index("# the experts of a training step"):text.index("# rows and weights")]
    M, H, I, E = 70, 136, 72, 32
    f = lambda s, *shape: (torch.randn(*shape, generator=gen(s), device="cuda") * 0.3).to(BF16)  # noqa: E731
    logits = f(4, M, E).float() * 4
    w, ids = pkg.moe_route(logits, 8, "sigmoid", k_group=4, group_count=8, group_select_mode=1,
                           routed_scaling_factor=2.5)
    env = dict(moe=pkg, torch=torch, E=E, hidden=f(1, M, H), w13=f(2, E, H, 2 * I), w2=f(3, E, I, H),
               router_logits=logits, w=w, ids=ids, grad_out=f(5, M, H))
    names = ("y", "grad_hidden", "grad_w13", "grad_w2", "grad_logits")
    runs = []
    for _ in range(3):
        exec(code, dict(env), local := dict(env))
        runs.append([local[n] for n in names])
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))
    t = [env[n].double().requires_grad_() for n in ("hidden", "w13", "w2", "router_logits")]
    p = torch.sigmoid(t[3]).gather(1, ids.long())
    p = 2.5 * p / p.sum(1, keepdim=True)          # (sigmoid weights are divided by their sum)
    assert ((p.detach() - w).abs() < 1e-5).all()
    h = torch.einsum("mh,mkhi->mki", t[0], t[1][ids.long()])
    a = torch.nn.functional.silu(h[..., :I]) * h[..., I:] * p[..., None]
    ry = torch.einsum("mki,mkih->mh", a, t[2][ids.long()])
    (ry * env["grad_out"].double()).sum().backward()
    for got, ref in zip(runs[0], (ry.detach(), *(v.grad for v in t))):
        assert ((got.double() - ref).norm() / ref.norm()).item() < 0.015
