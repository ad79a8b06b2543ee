"""Weights in 4 bits: quantised and read back to the last bit, and products of a few rows
with them against 64 bits."""
import numpy as np
import pytest
import torch

import hybrid_attention_ssm_hymba_b200 as H
from gpu_util import requires_cuda
from serve_util import DTYPE, HALF_STEP, TINY, TORCH, f64

pytestmark = [pytest.mark.gpu, requires_cuda]


def _codes(w, group):
    """(q in [-8, 7], scales): 7 w / amax to the nearest, ties to even, in 64 bits."""
    w = np.asarray(w, np.float64).reshape(w.shape[0], -1, group)
    most = np.abs(w).max(-1)
    scale = np.maximum((most.astype(np.float32) / np.float32(7)), TINY)
    q = np.rint(7 * w / np.maximum(most, float(TINY))[..., None])
    return q.reshape(w.shape[0], -1), scale


def _pack(q):
    u = (q + 8).astype(np.uint8)
    return u[:, 0::2] | (u[:, 1::2] << 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (3, 64, 64), (5, 128, 128), (129, 96, 32), (64, 1152, 128), (257, 704, 64)])
def test_quantise_and_dequantise(n, k, group, dtype):
    r = np.random.default_rng(n * k)
    w = (r.standard_normal((n, k)) * np.exp(r.uniform(-8, 8, (n, 1)))).astype(np.float32)
    w[0, :group] = 0.0
    if n > 2:
        w[1, :group] = np.arange(group) - group // 2          # exact halves between codes
        w[2, :group] *= np.float32(1e-38)
    t = torch.from_numpy(w).to(TORCH[dtype]).cuda()
    guard = 16
    q4 = torch.full((n * k // 2 + guard,), 0xEE, dtype=torch.uint8, device="cuda")
    sc = torch.full((n * k // group + guard,), 5.0, device="cuda")
    H.check(H.hymba_quantize_w4(t, q4, sc, n, k, group, DTYPE[dtype]), "quantize")
    q, scale = _codes(t.double().cpu().numpy(), group)
    assert np.array_equal(q4[:-guard].cpu().numpy().reshape(n, k // 2), _pack(q))
    assert np.array_equal(sc[:-guard].cpu().numpy().reshape(n, -1), scale)
    assert (q4[-guard:] == 0xEE).all() and (sc[-guard:] == 5.0).all()
    back = torch.zeros(n, k, dtype=TORCH[dtype], device="cuda")
    H.check(H.hymba_dequantize_w4(q4, sc, back, n, k, group, DTYPE[dtype]), "dequantize")
    want = torch.from_numpy(q.astype(np.float32) * np.repeat(scale, group, 1)).to(TORCH[dtype])
    assert torch.equal(back.cpu(), want)


def _product(m, n, k, group, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + m * n + k)
    a = torch.randn(m, k, generator=g).to(TORCH[dtype])
    q4 = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    sc = torch.rand(n, k // group, generator=g) * 0.01
    c = torch.full((m * n + 16,), 3.0, dtype=TORCH[dtype], device="cuda")
    H.check(H.hymba_gemm_w4(a.cuda(), q4.cuda(), sc.cuda(), c, m, n, k, group, DTYPE[dtype]), "gemm_w4")
    q = np.empty((n, k))
    q[:, 0::2], q[:, 1::2] = (q4 & 15).numpy() - 8.0, (q4 >> 4).numpy() - 8.0
    w = q * np.repeat(sc.double().numpy(), group, 1)
    ad = a.double().numpy()
    want, size = ad @ w.T, np.abs(ad) @ np.abs(w).T
    got = f64(c[:-16]).reshape(m, n)
    # fp32 sums of k products (each scaled once), and the output's own rounding
    tol = size * (k + 4) * 2.0 ** -24 + np.abs(want) * HALF_STEP[dtype]
    assert (np.abs(got - want) <= tol).all(), f"worst {(np.abs(got - want) - tol).max():.3e}"
    assert (c[-16:] == 3.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 2, 3, 7, 8, 9, 16])
@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (17, 96, 32), (16, 128, 128), (200, 704, 64), (33, 2048, 128),
                                       (2048, 1152, 32), (15, 5632, 128)])
def test_gemm_w4(m, n, k, group, dtype):
    _product(m, n, k, group, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gemm_w4_wide(dtype):
    _product(5, 11264, 2048, 64, dtype)


@pytest.mark.parametrize("dtype,m", [("bf16", 8), ("bf16", 16), ("f32", 2), ("f32", 8)])
@pytest.mark.parametrize("n,k,group", [(7109, 768, 64), (7109, 2560, 32), (19000, 4352, 128)])
def test_gemm_w4_shares(n, k, group, dtype, m):
    """Several tiles of rows a CTA, whose chunks its warps share across tiles and slabs."""
    _product(m, n, k, group, dtype)


def test_gemm_w4_repeats_and_graph():
    a = torch.randn(8, 2048, device="cuda").bfloat16()
    w = (torch.randn(512, 2048, device="cuda") * 0.02).bfloat16()
    q4 = torch.empty(512, 1024, dtype=torch.uint8, device="cuda")
    sc = torch.empty(512, 16, device="cuda")
    c = torch.empty(8, 512, dtype=torch.bfloat16, device="cuda")
    run = lambda: [H.check(H.hymba_quantize_w4(w, q4, sc, 512, 2048, 128, H.HYMBA_BF16)),  # noqa: E731
                   H.check(H.hymba_gemm_w4(a, q4, sc, c, 8, 512, 2048, 128, H.HYMBA_BF16))]
    run()
    ref = c.clone()
    for _ in range(10):
        run()
        assert torch.equal(c, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    c.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c, ref)
    # against the dequantised weights through hymba_gemm: both round bf16 once
    back = torch.empty(512, 2048, dtype=torch.bfloat16, device="cuda")
    H.check(H.hymba_dequantize_w4(q4, sc, back, 512, 2048, 128, H.HYMBA_BF16))
    full = torch.empty_like(c)
    H.check(H.hymba_gemm(a, back, full, 8, 512, 2048, H.HYMBA_BF16, torch.zeros(256, dtype=torch.uint8, device="cuda")))
    size = a.double().abs() @ back.double().abs().t()
    tol = size * (2.0 ** -8 + 2052 * 2.0 ** -23) + (c.double().abs() + full.double().abs()) * 2.0 ** -8
    assert ((c.double() - full.double()).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gemm_w4_keeps_non_finite_rows_apart(dtype):
    """An infinity or a NaN in one row of A reaches that row of C only; a large finite row stays finite."""
    a = torch.randn(4, 256, dtype=TORCH[dtype], device="cuda")
    a[1, 7], a[2, 9], a[3] = float("inf"), float("nan"), 3e37
    q4 = torch.full((40, 128), 0x99, dtype=torch.uint8, device="cuda")      # every q = 1
    sc = torch.full((40, 4), 1e-3, device="cuda")
    c = torch.empty(4, 40, dtype=TORCH[dtype], device="cuda")
    H.check(H.hymba_gemm_w4(a, q4, sc, c, 4, 40, 256, 64, DTYPE[dtype]))
    assert torch.isfinite(c[0]).all() and torch.isposinf(c[1]).all() and torch.isnan(c[2]).all() and torch.isfinite(c[3]).all()
