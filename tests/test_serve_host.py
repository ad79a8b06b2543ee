"""Refusals of the serving calls: bad arguments return their status before any CUDA call, and
workspace sizes follow (these run on a CPU machine)."""
import numpy as np
import pytest
import torch

import hybrid_attention_ssm_hymba_b200 as H
from serve_util import Paged, quantise_e4m3

P = 1 << 20   # an aligned address that nothing may read
INVALID, UNSUPPORTED, WORKSPACE = H.HYMBA_ERR_INVALID_ARG, H.HYMBA_ERR_UNSUPPORTED, H.HYMBA_ERR_WORKSPACE


def _kv(**kw):
    kv = H.hymba_paged_kv_t()
    src = dict(pages=P, scales=P, page_table=P, n_pages=10, page_size=64, table_ld=4, n_kv_heads=2, head_dim=128,
               cache_type=H.HYMBA_CACHE_E4M3)
    src.update(kw)
    for k, v in src.items():
        setattr(kv, k, v)
    return kv


CACHES = [
    (dict(pages=None), INVALID), (dict(page_table=None), INVALID), (dict(scales=None), INVALID), (dict(n_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(table_ld=0), INVALID), (dict(n_kv_heads=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(cache_type=3), INVALID), (dict(cache_type=-1), INVALID),
    (dict(cache_type=H.HYMBA_CACHE_F32), UNSUPPORTED),             # an fp32 cache with bf16 calls
    (dict(page_size=4), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED), (dict(page_size=192), UNSUPPORTED),
    (dict(head_dim=40), UNSUPPORTED), (dict(head_dim=272), UNSUPPORTED), (dict(pages=P + 8), UNSUPPORTED),
    (dict(scales=P + 4), UNSUPPORTED), (dict(n_pages=1 << 26), UNSUPPORTED), (dict(table_ld=1 << 26), UNSUPPORTED),
]


@pytest.mark.parametrize("bad,status", CACHES)
def test_bad_caches(bad, status):
    kv = _kv(**bad)
    for f in (H.hymba_paged_kv_append, H.hymba_paged_kv_read):
        assert f(kv, P, P, 256, 2, P, P, 5, H.HYMBA_BF16, P, 256, stream=0) == status
    assert H.hymba_paged_attention_workspace_size(kv, 2, 5, 3, 4, H.HYMBA_BF16) == 0
    assert H.hymba_paged_attention(P, 512, kv, P, 512, 2, P, P, 5, 3, 4, 0, -1, H.HYMBA_BF16, P, 1 << 40,
                                   stream=0) == status


@pytest.mark.parametrize("bad,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(ld=255), INVALID), (dict(batch=0), INVALID),
    (dict(q_start=None), INVALID), (dict(kv_len=None), INVALID), (dict(total=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(k=P + 8), UNSUPPORTED), (dict(v=P + 2), UNSUPPORTED), (dict(ld=260), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(wsb=255), WORKSPACE), (dict(ws=P + 16), INVALID)])
def test_bad_copies(bad, status):
    a = dict(k=P, v=P, ld=256, batch=2, q_start=P, kv_len=P, total=5, dtype=H.HYMBA_BF16, ws=P, wsb=256)
    a.update(bad)
    for f in (H.hymba_paged_kv_append, H.hymba_paged_kv_read):
        assert f(_kv(), a["k"], a["v"], a["ld"], a["batch"], a["q_start"], a["kv_len"], a["total"], a["dtype"], a["ws"],
                 a["wsb"], stream=0) == status
    # a call of no rows is complete without a launch
    assert H.hymba_paged_kv_append(_kv(), P, P, 256, 2, P, P, 0, H.HYMBA_BF16, P, 256, stream=0) == H.HYMBA_OK


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q_ld=511), INVALID), (dict(out_ld=511), INVALID),
    (dict(batch=0), INVALID), (dict(q_start=None), INVALID), (dict(kv_len=None), INVALID), (dict(total=-1), INVALID),
    (dict(most=0), INVALID), (dict(hq=0), INVALID), (dict(hq=3), INVALID), (dict(meta=-1), INVALID),
    (dict(window=-2), INVALID), (dict(dtype=5), INVALID), (dict(q=P + 8), UNSUPPORTED), (dict(out=P + 4), UNSUPPORTED),
    (dict(q_ld=516), UNSUPPORTED), (dict(out_ld=516), UNSUPPORTED), (dict(kv=dict(head_dim=64)), UNSUPPORTED),
    (dict(kv=dict(n_kv_heads=1), hq=130, q_ld=130 * 128, out_ld=130 * 128), UNSUPPORTED),
    (dict(kv=dict(head_dim=144), dtype=H.HYMBA_F32, q_ld=1024, out_ld=1024), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(wsb=0), WORKSPACE), (dict(wsb=-1), WORKSPACE), (dict(ws=P + 16), INVALID)])
def test_bad_attention(bad, status):
    a = dict(q=P, q_ld=512, out=P, out_ld=512, batch=2, q_start=P, kv_len=P, total=5, most=3, hq=4, meta=8, window=64,
             dtype=H.HYMBA_BF16, ws=P, wsb=1 << 40, kv={})
    a.update(bad)
    kv = _kv(**a["kv"])
    if a["wsb"] == -1:   # one byte short
        a["wsb"] = H.hymba_paged_attention_workspace_size(kv, 2, 5, 3, 4, H.HYMBA_BF16) - 1
    assert H.hymba_paged_attention(a["q"], a["q_ld"], kv, a["out"], a["out_ld"], a["batch"], a["q_start"], a["kv_len"],
                                   a["total"], a["most"], a["hq"], a["meta"], a["window"], a["dtype"], a["ws"], a["wsb"],
                                   stream=0) == status


@pytest.mark.parametrize("bad,status", [
    (dict(w=None), INVALID), (dict(q4=None), INVALID), (dict(sc=None), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID),
    (dict(group=0), INVALID), (dict(dtype=9), INVALID), (dict(group=48, k=96), UNSUPPORTED), (dict(k=96), UNSUPPORTED),
    (dict(w=P + 8), UNSUPPORTED), (dict(q4=P + 8), UNSUPPORTED), (dict(sc=P + 2), UNSUPPORTED)])
def test_bad_w4(bad, status):
    a = dict(w=P, q4=P, sc=P, n=16, k=128, group=64, dtype=H.HYMBA_BF16)
    a.update(bad)
    rest = (a["n"], a["k"], a["group"], a["dtype"])
    assert H.hymba_quantize_w4(a["w"], a["q4"], a["sc"], *rest, stream=0) == status
    assert H.hymba_dequantize_w4(a["q4"], a["sc"], a["w"], *rest, stream=0) == status
    assert H.hymba_gemm_w4(a["w"], a["q4"], a["sc"], P, 4, *rest, stream=0) == status


def test_bad_w4_rows():
    for m, c, status in ((0, P, INVALID), (17, P, UNSUPPORTED), (1, None, INVALID)):
        assert H.hymba_gemm_w4(P, P, P, c, m, 16, 128, 64, H.HYMBA_BF16, stream=0) == status


def test_pointers_off_their_elements():
    """A load or store of an element at such an address would fault."""
    assert H.hymba_paged_kv_read(_kv(page_table=P + 2), P, P, 256, 2, P, P, 5, H.HYMBA_BF16, P, 256, stream=0) == UNSUPPORTED
    for q_start, kv_len in ((P + 2, P), (P, P + 1)):
        assert H.hymba_paged_kv_append(_kv(), P, P, 256, 2, q_start, kv_len, 5, H.HYMBA_BF16, P, 256, stream=0) == UNSUPPORTED
        assert H.hymba_paged_attention(P, 512, _kv(), P, 512, 2, q_start, kv_len, 5, 3, 4, 8, 64, H.HYMBA_BF16, P, 1 << 40,
                                       stream=0) == UNSUPPORTED
    for c, dtype in ((P + 1, H.HYMBA_BF16), (P + 2, H.HYMBA_F32)):
        assert H.hymba_gemm_w4(P, P, P, c, 4, 16, 128, 64, dtype, stream=0) == UNSUPPORTED


def test_workspace_sizes_are_bounded():
    """The scratch does not grow with the histories, and covers one-row and long chunks."""
    for most, total in ((1, 64), (40, 400), (8192, 20000)):
        n = H.hymba_paged_attention_workspace_size(_kv(n_pages=1 << 20, table_ld=1 << 16), 64, total, most, 16, H.HYMBA_BF16)
        assert 256 <= n <= 256 << 20
    assert H.hymba_paged_attention_workspace_size(_kv(cache_type=H.HYMBA_CACHE_F32), 2, 5, 3, 4, H.HYMBA_F32) >= 256


def test_quantisation_oracle():
    """The tests' own e4m3 steps: half a step of the value, 2^-4, or of the least code, 2^-10 scales."""
    x = np.random.default_rng(0).standard_normal((64, 3, 128)).astype(np.float32)
    codes, scale = quantise_e4m3(x)
    y = codes.float().numpy() * scale[..., None]
    assert (np.abs(y - x) <= np.abs(x) * 2.0 ** -4 * (1 + 1e-6) + scale[..., None] * 2.0 ** -10).all()
    z, s = quantise_e4m3(np.zeros((2, 16)))
    assert (z.float() == 0).all() and (s == 2.0 ** -126).all()


def test_paged_inputs_round_trip_on_the_cpu():
    """The tests' paged container: what is put is what is read, in every layout."""
    for cache in ("f32", "bf16", "e4m3"):
        c = Paged("f32" if cache == "f32" else "bf16", cache, 3, 16, 8, [3, 0, 9], [10, 0, 1], device="cpu")
        assert not np.isnan(c.rows(0, 0, 0, 13)).any() and not np.isnan(c.rows(1, 2, 0, 10)).any()
        used = set(c.table[0, :2]) | set(c.table[2, :2])
        assert len(used) == 4 and torch.isnan(c.pages.float()[0, list(set(range(c.n_pages)) - used)]).all()
