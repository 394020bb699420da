"""CPU tests of the products by expert, their gradients and MX FP4: the oracle
against independent computations, and the refusals of the C ABI and of the
binding."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import mixture_experts_ffn_softmax_gb300 as pkg
import oracle

OK, INVALID, NO_DEVICE = 0, 1, 7


# ------------------------------------------------------------- oracle pins --
def test_oracle_grouped_matmul_and_gradients_by_autograd():
    rng = np.random.default_rng(0)
    offsets, K, N = [1, 4, 4, 9], 5, 3
    x, w, b = rng.normal(size=(11, K)), rng.normal(size=(3, K, N)), rng.normal(size=(3, N))
    y = oracle.grouped_matmul(x, w, offsets, np.full((11, N), 7.0), b)
    assert (y[[0, 9, 10]] == 7).all()
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    expert = torch.tensor([0, 0, 0, 2, 2, 2, 2, 2])
    ty = torch.einsum("rk,rkn->rn", tx[1:9], tw[expert]) + torch.tensor(b)[expert]
    np.testing.assert_allclose(y[1:9], ty.detach().numpy(), rtol=1e-12)
    dy = rng.normal(size=(11, N))
    (ty * torch.tensor(dy[1:9])).sum().backward()
    np.testing.assert_allclose(oracle.grouped_weight_grad(x, dy, offsets), tw.grad.numpy(), rtol=1e-12)
    dx = oracle.grouped_matmul(dy, w.transpose(0, 2, 1), offsets, np.zeros((11, K)))
    np.testing.assert_allclose(dx, tx.grad.numpy(), rtol=1e-12)


def test_oracle_swiglu_backward_by_differences():
    """Central differences: error O(h^2) + O(eps / h)."""
    rng = np.random.default_rng(1)
    gu, dz, w, h = rng.normal(size=(3, 8)), rng.normal(size=(3, 4)), rng.normal(size=3), 1e-5
    d, dw = oracle.swiglu_backward(dz, gu, w)
    loss = lambda a, b: (oracle.swiglu(a, b) * dz).sum()  # noqa: E731
    for i in np.ndindex(gu.shape):
        e = np.zeros_like(gu)
        e[i] = h
        assert abs((loss(gu + e, w) - loss(gu - e, w)) / (2 * h) - d[i]) < 1e-8
    for r in range(3):
        e = np.zeros(3)
        e[r] = h
        assert abs((loss(gu, w + e) - loss(gu, w - e)) / (2 * h) - dw[r]) < 1e-8


def test_oracle_mx_fp4_definition():
    z = np.zeros((5, 32))
    z[0, :10] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -0.25]      # ties, scale 1
    z[1, :3] = [7.9, 4, 0.3]                                            # above 6: held at 6
    z[2, 0] = 2.0 ** 20
    z[3, 0], z[3, 1] = 2.0 ** -126, -2.0 ** -128                        # the scale's lower end
    code, scale = oracle.quant_mx_fp4(z)
    assert scale.ravel().tolist() == [127, 127, 145, 0, 0]
    assert code[0, :10].tolist() == [7, 6, 6, 4, 4, 2, 2, 0, 14, 8]
    assert code[1, :3].tolist() == [7, 6, 1]
    assert code[2, 0] == 6 and code[3, :2].tolist() == [4, 9] and not code[4].any()
    v = oracle.mx_fp4_values(oracle.pack_fp4(code), scale)
    assert v[0, :10].tolist() == [6, 4, 4, 2, 2, 1, 1, 0, -4, 0]
    assert v[2, 0] == 2.0 ** 20 and v[3, :2].tolist() == [2.0 ** -126, -2.0 ** -128]
    # the library's weight-only decoding of the same codes
    packed = oracle.pack_fp4(code)
    assert np.array_equal(oracle.unpack_nibbles(packed), code)


# --------------------------------------------------------- C ABI refusals --
def _p(v=4096):
    return ctypes.c_void_p(v)


def _product(R=8, E=2, K=64, N=64, t=0, f32=0, x=4096, w=4096, off=4096, bias=0, out=4096, err=0):
    return pkg.lib().moe_grouped_matmul(_p(x), _p(w), _p(off), t, _p(bias), R, E, K, N, f32,
                                        _p(out), _p(err), None)


def _grad(R=8, E=2, K=64, N=64, f32=0, acc=0, x=4096, dy=4096, off=4096, out=4096, err=0):
    return pkg.lib().moe_grouped_weight_grad(_p(x), _p(dy), _p(off), R, E, K, N, f32, acc,
                                             _p(out), _p(err), None)


def _fp4(R=8, E=2, K=64, N=64, f32=0, a=4096, sa=4096, w=4096, sw=4096, off=4096, out=4096, err=0):
    return pkg.lib().moe_matmul_fp4(_p(a), _p(sa), _p(w), _p(sw), _p(off), R, E, K, N, f32,
                                    _p(out), _p(err), None)


@pytest.mark.parametrize("call,unit", [(_product, 8), (_grad, 8), (_fp4, 32)])
def test_grouped_refusals(call, unit):
    assert call(R=-1) == INVALID and call(R=(1 << 31) - 1023) == INVALID
    assert call(E=0) == INVALID and call(E=1025) == INVALID
    assert call(K=0) == INVALID and call(K=unit // 2) == INVALID and call(K=64 + unit // 2) == INVALID
    assert call(K=(1 << 22) + 32) == INVALID
    assert call(N=0) == INVALID and call(N=60) == INVALID and call(N=(1 << 22) + 8) == INVALID
    assert call(f32=2) == INVALID
    assert call(R=1 << 30, N=1 << 20) == INVALID                      # R * N
    assert call(E=1024, K=1 << 20, N=1 << 18) == INVALID              # tiles of the weights
    for name in ("x", "w", "out", "off") if call is _product else (
            ("x", "dy", "out", "off") if call is _grad else ("a", "sa", "w", "sw", "out")):
        assert call(**{name: 0}) == INVALID
        assert call(**{name: 4098}) == INVALID                        # alignment
    assert call(err=4098) == INVALID
    if call is _product:
        assert call(t=2) == INVALID and call(bias=4104) == INVALID
    if call is _grad:
        assert call(acc=2) == INVALID and call(R=1 << 30, K=1 << 20) == INVALID
    if call is _fp4:
        assert call(off=0) == INVALID                                 # dense: one weight
    if call is not _grad:
        assert call(R=0, E=1) == OK
    if not torch.cuda.is_available():
        assert call() == NO_DEVICE


def test_swiglu_and_quant_refusals():
    lib, p, odd = pkg.lib(), _p(), _p(4104)
    fwd = lambda R=4, I=64, gu=p, w=None, z=p: lib.moe_swiglu(gu, w, R, I, z, None)  # noqa: E731
    bwd = lambda R=4, I=64, dz=p, gu=p, w=None, d=p, dw=None: lib.moe_swiglu_backward(  # noqa: E731
        dz, gu, w, R, I, d, dw, None)
    for call in (fwd, bwd):
        assert call(R=-1) == INVALID and call(R=1 << 31) == INVALID
        assert call(I=0) == INVALID and call(I=12) == INVALID and call(I=(1 << 22) + 8) == INVALID
        assert call(gu=None) == INVALID and call(gu=odd) == INVALID and call(w=_p(4098)) == INVALID
        assert call(R=0) == OK
    assert fwd(z=None) == INVALID and fwd(z=odd) == INVALID
    assert bwd(dz=None) == INVALID and bwd(d=odd) == INVALID and bwd(dw=_p(4098)) == INVALID

    def quant(M=4, K=64, s=0, x=p, q=p, sc=p, v=None):
        return lib.moe_quant_mx_fp4(x, M, K, s, q, sc, v, None)
    assert quant(M=-1) == INVALID and quant(M=1 << 31) == INVALID
    assert quant(K=0) == INVALID and quant(K=48) == INVALID and quant(K=(1 << 22) + 32) == INVALID
    assert quant(s=2) == INVALID
    assert quant(x=None) == INVALID and quant(q=odd) == INVALID and quant(sc=odd) == INVALID
    assert quant(v=odd) == INVALID
    assert quant(M=0) == OK


# --------------------------------------------------------- binding refusals --
def _raises(text, f, *a, **k):
    with pytest.raises(ValueError, match=text):
        f(*a, **k)


def test_binding_refusals_of_swiglu_and_quant():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    _raises("even number", pkg.moe_swiglu, bf(4, 33))
    _raises("row_weights has shape", pkg.moe_swiglu, bf(4, 32), torch.zeros(3))
    _raises("CUDA device", pkg.moe_swiglu, bf(4, 32))
    _raises("grad_z has shape", pkg.moe_swiglu_backward, bf(4, 32), bf(4, 32))
    _raises("grad_weights has shape", pkg.moe_swiglu_backward, bf(4, 16), bf(4, 32),
            grad_weights=torch.zeros(4, 1))
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    q = pkg.moe_quant_mx_fp4
    _raises("whole blocks", q, bf(4, 48))
    _raises("whole blocks", q, bf(4, 96), swiglu=True)
    _raises("q4 has shape", q, bf(4, 64), q4=u8(4, 31))
    _raises("values must", q, bf(4, 64), values=torch.zeros(4, 64))
    _raises("CUDA device", q, bf(4, 64))


def test_binding_refusals_of_grouped_products():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    off = torch.tensor([0, 3, 8], dtype=torch.int32)
    x, w = bf(8, 64), bf(2, 64, 32)
    f = pkg.moe_grouped_matmul
    _raises("x must be", f, x.float(), w, off)
    _raises("2-dimensional", f, x[0], w, off)
    _raises("w must be a 3-dim", f, x, w[0], off)
    _raises("w has shape", f, x, bf(2, 56, 32), off)
    _raises("w has shape", f, x, w, off, transposed=True)
    _raises("contiguous", f, x, bf(2, 32, 64).transpose(1, 2), off)
    _raises("expert_offsets has shape", f, x, w, off[:2])
    _raises("expert_offsets must", f, x, w, off.long())
    _raises("bias has shape", f, x, w, off, bias=bf(2, 31))
    _raises("the output is", f, x, w, off, out_dtype=torch.float16)
    _raises("out has shape", f, x, w, off, out=bf(8, 31))
    _raises("error_word", f, x, w, off, error_word=off)
    _raises("CUDA device", f, x, w, off)
    g = pkg.moe_grouped_weight_grad
    _raises("dy has shape", g, x, bf(7, 32), off)
    _raises("accumulate needs", g, x, bf(8, 32), off, accumulate=True)
    _raises("at least two", g, x, bf(8, 32), off[:1])
    _raises("expert_offsets must", g, x, bf(8, 32), None)
    _raises("out has shape", g, x, bf(8, 32), off, out=bf(3, 64, 32))
    _raises("CUDA device", g, x, bf(8, 32), off)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    m = pkg.moe_matmul_fp4
    _raises("a_q must", m, u8(4, 32).float(), u8(4, 2), u8(8, 32), u8(8, 2))
    _raises("a_scale has shape", m, u8(4, 32), u8(4, 1), u8(8, 32), u8(8, 2))
    _raises("w_q must be a 2-dim", m, u8(4, 32), u8(4, 2), u8(2, 8, 32), u8(2, 8, 2))
    _raises("w_q must be a 3-dim", m, u8(8, 32), u8(8, 2), u8(8, 32), u8(8, 2), off)
    _raises("w_scale has shape", m, u8(8, 32), u8(8, 2), u8(2, 8, 32), u8(8, 2), off)
    _raises("whole blocks", m, u8(4, 24), u8(4, 1), u8(8, 24), u8(8, 1))
    _raises("CUDA device", m, u8(8, 32), u8(8, 2), u8(2, 8, 32), u8(2, 8, 2), off)


# ------------------------------------------------------ ranges that are read --
SPANS = r"""
#include <algorithm>
#include <cstdio>
#include "raw_scales.cuh"
using namespace gbmoe;
// within the tensor, in whole aligned 16 bytes, every byte of [from, to) and none before
// the 16 that hold the first
static bool good(const RawSpan& s, int64_t from, int64_t to, int64_t total) {
  if (to <= from) return s.bulk == 0 && s.begin + s.bulk >= s.end;
  const int64_t past = s.begin + s.bulk;
  return s.begin % 16 == 0 && s.bulk % 16 == 0 && s.begin <= from && from - s.begin < 16 &&
         past <= total && s.end <= total && std::max(past, s.end) >= to &&
         std::max(past, s.end) < to + 16 && s.end - past < 16;
}
int main() {
  for (int KG = 1; KG <= 32; ++KG) {
    for (int E = 1; E <= 3; ++E)
      for (int N = 8; N <= 528; N += 8)
        for (int e = 0; e < E; ++e)
          for (int n = 0; n < (N + 255) / 256 * 256; n += 128) {
            const int64_t row = int64_t(e) * N + n, rows = std::min(std::max(N - n, 0), 128);
            if (!good(weight_scale_span(E, N, KG, e, n), row * KG, (row + rows) * KG, int64_t(E) * N * KG))
              return std::printf("weight KG=%d E=%d N=%d e=%d n=%d\n", KG, E, N, e, n), 1;
          }
    for (int64_t R : {1, 2, 5, 31, 32, 33, 230, 700, 2147482624})
      for (int64_t c0 : {int64_t(0), int64_t(1), int64_t(7), int64_t(224), R - 1, R - 31, R - 225})
        for (int T = 32; T <= 224 && c0 >= 0 && c0 < R; T += 32)
          if (!good(row_scale_span(R, KG, c0, T), c0 * KG, std::min(c0 + T, R) * KG, R * KG))
            return std::printf("rows KG=%d R=%lld c0=%lld T=%d\n", KG, (long long)R, (long long)c0, T), 1;
  }
  return 0;
}
"""


def test_scales_are_read_inside_their_tensors(tmp_path):
    """The bulk copies of MX FP4 scales for every row length up to 32, both CTAs of a
    tile (the second may have no column at all), every expert."""
    csrc = os.path.join(os.path.dirname(pkg.__file__), "csrc")
    (tmp_path / "spans.cpp").write_text(SPANS)
    exe = str(tmp_path / "spans")
    subprocess.run(["g++", "-std=c++17", "-O1", "-x", "c++", "-I", csrc, str(tmp_path / "spans.cpp"),
                    "-o", exe], check=True, timeout=300)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout
