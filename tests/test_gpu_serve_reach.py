"""Calls that the serving interface allows at the edges of its sizes: offsets beyond 32 bits, parts
shared over many tiles, many heads a K/V head, padding before the first sequence, one workspace."""
import numpy as np
import pytest
import torch

import hybrid_attention_ssm_hymba_b200 as H
from gpu_util import requires_cuda, status_ok
from serve_util import TORCH, Paged, f64, quantise_e4m3
from test_gpu_paged import _check, _q
from test_gpu_w4 import _product

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.mark.parametrize("m", [9, 16])
@pytest.mark.parametrize("n,k,group", [(7109, 768, 64), (7109, 2560, 32), (19000, 1152, 128)])
def test_gemm_w4_shares_of_many_fp32_rows(n, k, group, m):
    """Nine and more fp32 rows with several tiles of rows a CTA: chunks shared across tiles and slabs."""
    _product(m, n, k, group, "f32")


def test_append_e4m3_beyond_32_bits():
    """Codes and scales at the end of a pool whose V half starts beyond 2^31 elements, to the last
    bit, and the rows next to them as they were."""
    hkv, page = 8, 64
    n_pages = (1 << 31) // (page * hkv * 128) + 40
    c = Paged("bf16", "e4m3", hkv, 128, page, [70, 1], [130, 300], seed=41)
    small = c.n_pages
    c.upload()
    pages = torch.empty((2, n_pages, page, hkv, 128), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((2, n_pages, hkv, page), device="cuda")
    pages.view(torch.uint8)[:, -small:] = c.g_pages.view(torch.uint8)
    pages.view(torch.uint8)[:, -small - 1] = 0x55
    scales[:, -small:] = c.g_scales
    scales[:, -small - 1] = 5.0
    c.g_table += n_pages - small
    c.kv = H.make_paged_kv(pages, c.g_table, page, hkv, 128, c.kv.cache_type, scales=scales)
    x = torch.randn(c.total, 2, hkv, 128, device="cuda").bfloat16()
    status_ok(c.append(x[:, 0], x[:, 1], 2 * hkv * 128))
    xf = x.float().cpu().numpy()
    for b in range(2):
        for w in range(2):
            c.put(w, b, c.lens[b] - c.ns[b], xf[c.first[b]:c.first[b + 1], w])
    assert torch.equal(pages.view(torch.uint8)[:, -small:].cpu(), c.pages.view(torch.uint8))
    assert torch.equal(scales[:, -small:].cpu().view(torch.int32), c.scales.view(torch.int32))
    assert (pages.view(torch.uint8)[:, -small - 1] == 0x55).all() and (scales[:, -small - 1] == 5.0).all()
    codes, scale = quantise_e4m3(xf[0, 1])
    pg, at = c.slots(0, 130, 131)
    assert torch.equal(pages[1, -small + int(pg)][int(at)].view(torch.uint8).cpu(), codes.view(torch.uint8))
    assert np.array_equal(scales[1, -small + int(pg), :, int(at)].cpu().numpy(), scale)


@pytest.mark.parametrize("ns,pasts", [([1], [300]), ([3, 0, 1], [0, 5, 200]), ([70, 130], [500, 0])])
@pytest.mark.parametrize("dtype,cache,hq,hkv,dh,page", [
    ("bf16", "bf16", 128, 1, 128, 128), ("bf16", "e4m3", 128, 1, 128, 384), ("bf16", "e4m3", 65, 1, 128, 8),
    ("bf16", "bf16", 200, 2, 128, 16), ("bf16", "e4m3", 16, 1, 128, 256), ("f32", "f32", 20, 1, 16, 8), ("f32", "e4m3", 33, 3, 112, 64)])
def test_attention_of_many_heads(ns, pasts, dtype, cache, hq, hkv, dh, page):
    c = Paged(dtype, cache, hkv, dh, page, ns, pasts, seed=42).upload()
    q, qd = _q(c, hq)
    out = torch.full((c.total, hq, dh), 7.0, dtype=TORCH[dtype], device="cuda")
    status_ok(c.attend(q, out, hq, 8, 250))
    want, tol = c.attention(qd, hq, 8, 250)
    _check(f64(out), want, tol)
    assert (f64(out)[c.first[-1]:] == 7.0).all()


@pytest.mark.parametrize("dtype,cache,ns", [("bf16", "bf16", [1, 1]), ("bf16", "e4m3", [90, 3]), ("f32", "f32", [5, 2])])
def test_rows_before_the_first_sequence(dtype, cache, ns):
    """q_start[0] > 0: the rows before it are no sequence's, for each of the calls."""
    c = Paged(dtype, cache, 2, 128, 64, ns, [100, 40], seed=43)
    c.first = c.first + 3
    c.total += 3
    c.upload()
    q, qd = _q(c, 4)
    out = torch.full((c.total, 4, 128), 7.0, dtype=TORCH[dtype], device="cuda")
    status_ok(c.attend(q, out, 4, 0, -1))
    want, tol = c.attention(qd, 4, 0, -1)
    _check(f64(out), want, tol)
    assert (out[:3] == 7.0).all() and (out[c.first[-1]:] == 7.0).all()
    back = torch.full((2, c.total, 2, 128), 7.0, dtype=TORCH[dtype], device="cuda")
    status_ok(c.read(back[0], back[1], 256))
    assert (back[:, :3] == 7.0).all() and (back[:, c.first[-1]:] == 7.0).all()
    kv = torch.full((c.total, 2, 256), float("nan"), dtype=TORCH[dtype], device="cuda")
    rows = slice(int(c.first[0]), int(c.first[-1]))
    kv[rows] = back[:, rows].reshape(2, -1, 256).transpose(0, 1)
    status_ok(c.append(kv[:, 0], kv[:, 1], 512))
    again = torch.zeros_like(back)
    status_ok(c.read(again[0], again[1], 256))
    for b in range(2):
        for w in range(2):
            want = c.rows(w, b, c.lens[b] - c.ns[b], c.lens[b])
            got = f64(again[w, c.first[b]:c.first[b + 1]])
            # e4m3: a row's own values quantised again: half a step of the value or of the least code
            bound = 0 if cache != "e4m3" else np.abs(want) * (2.0 ** -4 + 2.0 ** -7) + np.abs(want).max(-1, keepdims=True) / 448 * 2.0 ** -9
            assert (np.abs(got - want) <= bound).all()


def test_one_workspace_for_calls_of_every_size():
    """fp32: a workspace sized for many rows serves a few, which are split over more CTAs."""
    big = Paged("f32", "f32", 2, 64, 64, [200, 150], [300, 700], seed=44).upload()
    ws = big.workspace(4)
    for c in (big, Paged("f32", "f32", 2, 64, 64, [1], [1100], seed=45), Paged("f32", "f32", 2, 64, 64, [3, 1], [900, 5], seed=46)):
        c.upload()
        q, qd = _q(c, 4)
        out = torch.zeros((c.total, 4, 64), device="cuda")
        c.attend(q, out, 4, 0, -1, ws=ws)
        status_ok(ws)
        want, tol = c.attention(qd, 4, 0, -1)
        _check(f64(out), want, tol)


@pytest.mark.parametrize("dtype,cache,ns", [("bf16", "bf16", [1, 1]), ("bf16", "e4m3", [90, 300]), ("f32", "f32", [2, 1])])
def test_two_streams_at_once(dtype, cache, ns):
    """Two streams over one cache, each with its workspace: the bits of a call alone."""
    c = Paged(dtype, cache, 2, 128, 64, ns, [700, 500], seed=47).upload()
    q, _ = _q(c, 8)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [c.workspace(8) for _ in range(2)]
    outs = [torch.zeros((c.total, 8, 128), dtype=TORCH[dtype], device="cuda") for _ in range(2)]
    ref = torch.zeros_like(outs[0])
    c.attend(q, ref, 8, 16, 300, ws=ws[0])
    torch.cuda.synchronize()
    for _ in range(20):
        for o, w, s in zip(outs, ws, streams):
            with torch.cuda.stream(s):
                o.zero_()
                for _ in range(5):
                    c.attend(q, o, 8, 16, 300, ws=w, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    for w in ws:
        status_ok(w)
