"""The paged K/V cache and its attention on the GPU against 64-bit plain forms: lengths from
one row, empty sequences, pages that end inside a tile, windows with meta rows, head layouts,
strides, NaN in rows nobody sees, bad lengths and page numbers, graphs, streams, and a run of
the calls together."""
import numpy as np
import pytest
import torch

import hybrid_attention_ssm_hymba_b200 as H
from hybrid_attention_ssm_hymba_b200 import host, synth
from gpu_util import requires_cuda, status_ok
from serve_util import TORCH, Paged, f64

pytestmark = [pytest.mark.gpu, requires_cuda]


def _q(c, hq, seed=5):
    q = np.random.default_rng(seed).standard_normal((c.total, hq, c.dh)).astype(np.float32)
    t = torch.from_numpy(q).to(TORCH[c.dtype])
    return t.cuda(), t.double().numpy()


def _check(got, want, tol, what=""):
    rows = ~np.isnan(want).any((1, 2))
    assert np.all(np.isfinite(got[rows])), f"{what}: non-finite values"
    bad = np.abs(got - want)[rows] - tol[rows]
    assert (bad <= 0).all(), f"{what}: {int((bad > 0).sum())} values beyond the tolerance, by up to {bad.max():.3e}"


def _attend(c, hq, meta, window, **kw):
    c.upload()
    q, qd = _q(c, hq)
    out = torch.full((c.total, hq, c.dh), 7.0, dtype=TORCH[c.dtype], device="cuda")
    ws = c.attend(q, out, hq, meta, window, **kw)
    status_ok(ws)
    want, tol = c.attention(qd, hq, meta, window)
    got = f64(out)
    _check(got, want, tol)
    assert (got[c.first[-1]:] == 7.0).all(), "rows behind the last sequence"
    return out


# (ns, pasts): one token alone; boundaries of 128-row tiles; empty sequences; ragged chunks
BATCHES = {
    "first token": ([1], [0]),
    "generation": ([1, 1, 1, 1], [126, 127, 128, 1000]),
    "empty ones": ([0, 3, 0, 1, 0], [5, 0, 0, 300, 70]),
    "ragged": ([5, 130, 1, 64, 17], [0, 257, 700, 64, 1]),
    "one chunk": ([333], [500]),
}


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("dtype,cache,hq,hkv,dh,page", [
    ("bf16", "bf16", 16, 4, 128, 64), ("bf16", "e4m3", 16, 4, 128, 32), ("bf16", "bf16", 5, 1, 128, 16),
    ("bf16", "e4m3", 4, 4, 128, 8), ("bf16", "e4m3", 6, 2, 128, 128), ("bf16", "bf16", 24, 1, 128, 384),
    ("f32", "f32", 4, 2, 32, 16), ("f32", "e4m3", 6, 2, 48, 64), ("f32", "f32", 8, 1, 128, 256),
])
def test_attention_lengths_and_layouts(batch, dtype, cache, hq, hkv, dh, page):
    ns, pasts = BATCHES[batch]
    _attend(Paged(dtype, cache, hkv, dh, page, ns, pasts), hq, 8, -1)


@pytest.mark.parametrize("meta,window", [(0, 0), (8, 0), (0, 1), (128, 63), (16, 200), (40, 129), (4096, 5), (0, 100000)])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
def test_attention_windows(dtype, cache, meta, window):
    c = Paged(dtype, cache, 2, 128, 32, [1, 70, 300, 1], [900, 450, 10, 0], seed=3)
    # pages that no query sees may hold anything and have any number
    for b in range(c.batch):
        seen = c.visible(b, meta, window).any(0)
        for pg in range(-(-c.lens[b] // c.page)):
            if not seen[pg * c.page:(pg + 1) * c.page].any():
                c.table[b, pg] = [-1, 1 << 30, c.n_pages][pg % 3]
    keep = Paged(dtype, cache, 2, 128, 32, [1, 70, 300, 1], [900, 450, 10, 0], seed=3)
    c.rows = keep.rows
    _attend(c, 8, meta, window)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 200])
def test_attention_ignores_rows_outside_every_window(cache, n):
    """NaN in every cache row that no query of the call sees, inside tiles that are read."""
    c = Paged("bf16", cache, 2, 128, 64, [n, n], [600, 333], seed=4)
    for b in range(c.batch):
        for j in np.flatnonzero(~c.visible(b, 24, 100).any(0)):
            pg, at = c.slots(b, j, j + 1)
            for w in range(2):
                if cache == "e4m3":
                    c.pages[w].view(torch.uint8)[pg, at] = 0x7f     # (codes and scales as they come)
                    c.scales[w][pg, :, at] = float("nan")
                else:
                    c.pages[w][pg, at] = float("nan")
    _attend(c, 8, 24, 100)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
def test_attention_strides_leave_other_columns(dtype, cache):
    c = Paged(dtype, cache, 2, 128, 64, [1, 40], [50, 90]).upload()
    hq, wq = 4, 512
    q, qd = _q(c, hq)
    wide_q = torch.full((c.total, wq + 64), float("nan"), dtype=q.dtype, device="cuda")
    wide_q[:, 32:32 + wq] = q.reshape(c.total, wq)
    out = torch.full((c.total, wq + 32), 3.0, dtype=q.dtype, device="cuda")
    ws = c.attend(wide_q[:, 32:], out[:, 16:], hq, 0, -1, q_ld=wq + 64, out_ld=wq + 32)
    status_ok(ws)
    want, tol = c.attention(qd, hq, 0, -1)
    _check(f64(out[:, 16:16 + wq].reshape(c.total, hq, 128)), want, tol)
    assert (out[:, :16] == 3.0).all() and (out[:, 16 + wq:] == 3.0).all()


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
@pytest.mark.parametrize("ns", [[1, 1, 1], [20, 150, 300]])
def test_attention_extreme_scores(dtype, cache, ns):
    """Scores of hundreds: one key takes (nearly) the whole softmax, early or late in the row."""
    c = Paged(dtype, cache, 2, 128, 64, ns, [400, 300, 200], seed=6)
    for b in range(c.batch):
        for j in (3, 130, 250):
            c.put(0, b, j, 40 * c.rng.standard_normal((1, 2, 128)).astype(np.float32))
    _attend(c, 4, 0, -1)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("ns", [[1, 1], [100, 260]])
def test_attention_bad_page_numbers_hide_their_keys(cache, ns):
    c = Paged("bf16", cache, 2, 128, 64, ns, [300, 200], seed=7)
    good = c.table.copy()
    c.upload()
    c.table[0, 1], c.table[1, 0] = -1, c.n_pages
    c.g_table.copy_(torch.from_numpy(c.table))
    c.table = good
    q, qd = _q(c, 4)
    out = torch.zeros((c.total, 4, 128), dtype=torch.bfloat16, device="cuda")
    ws = c.attend(q, out, 4, 0, -1)
    assert H.hymba_workspace_status(ws) == H.HYMBA_ERR_INVALID_ARG
    want, tol = c.attention(qd, 4, 0, -1, hidden=lambda b, j: j // 64 == 1 - b)
    _check(f64(out), want, tol)
    # every page of a sequence bad: its rows are 0
    c.g_table.fill_(-1)
    ws = c.attend(q, out, 4, 0, -1)
    assert H.hymba_workspace_status(ws) == H.HYMBA_ERR_INVALID_ARG
    assert (out[:c.first[-1]] == 0).all()


def test_bad_lengths_skip_their_sequence():
    c = Paged("bf16", "bf16", 2, 128, 64, [3, 4, 5], [100, 20, 60], seed=8).upload()
    q, qd = _q(c, 4)
    want, tol = c.attention(qd, 4, 0, -1)
    for what, lens, first in [("n > len", [103, 3, 65], None), ("len > table", [103, 24, 100000], None),
                              ("n < 0", None, [0, 3, 2, 12]), ("rows > total", None, [0, 3, 7, c.total + 1])]:
        c.g_lens.copy_(torch.tensor(lens if lens else c.lens, dtype=torch.int32))
        c.g_first.copy_(torch.tensor(first if first else c.first, dtype=torch.int32))
        out = torch.full((c.total, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        back = torch.full((2, c.total, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        for ws in (c.attend(q, out, 4, 0, -1), c.read(back[0], back[1], 256), c.append(back[0], back[1], 256)):
            assert H.hymba_workspace_status(ws) == H.HYMBA_ERR_INVALID_ARG, what
        _check(f64(out[:3]), want[:3], tol[:3], what)
    # more rows than the caller promised
    c.upload()
    out.fill_(5.0)
    ws = c.attend(q, out, 4, 0, -1, max_rows=4)
    assert H.hymba_workspace_status(ws) == H.HYMBA_ERR_INVALID_ARG
    _check(f64(out[:7]), want[:7], tol[:7])
    assert (out[7:] == 5.0).all()


@pytest.mark.parametrize("dtype,cache,n", [("bf16", "bf16", 1), ("bf16", "e4m3", 1), ("bf16", "bf16", 300),
                                           ("bf16", "e4m3", 300), ("f32", "f32", 9)])
def test_attention_graph_streams_and_repeats(dtype, cache, n):
    """The same bits eagerly, repeated, on another stream, and from a graph replayed on new lengths."""
    c = Paged(dtype, cache, 2, 128, 64, [n, n, 1], [700, 100, 0], seed=9).upload()
    q, qd = _q(c, 8)
    ws = c.workspace(8)
    out = torch.zeros((c.total, 8, 128), dtype=TORCH[dtype], device="cuda")
    c.attend(q, out, 8, 16, 256, ws=ws)
    ref = out.clone()
    for _ in range(20):
        out.zero_()
        c.attend(q, out, 8, 16, 256, ws=ws)
        assert torch.equal(out, ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.synchronize()
    c.attend(q, out, 8, 16, 256, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend(q, out, 8, 16, 256, ws=ws, stream=torch.cuda.current_stream())
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    # the graph reads the lengths when it runs: fewer rows, shorter sequences
    ns, lens = np.array([max(1, n // 2), 0, 1]), np.array([max(1, n // 2) + 150, 0, 1])
    c.g_first.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)))
    c.g_lens.copy_(torch.from_numpy(lens.astype(np.int32)))
    out.fill_(7.0)
    g.replay()
    status_ok(ws)
    c.ns, c.lens, c.first = ns, lens, np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    want, tol = c.attention(qd, 8, 16, 256)
    _check(f64(out), want, tol)
    assert (out[c.first[-1]:] == 7.0).all()


@pytest.mark.parametrize("dtype,cache,hkv,dh,page", [
    ("bf16", "e4m3", 4, 128, 64), ("bf16", "bf16", 1, 128, 8), ("f32", "e4m3", 3, 48, 16), ("f32", "f32", 2, 16, 32),
    ("bf16", "e4m3", 5, 256, 128), ("bf16", "e4m3", 2, 80, 16), ("f32", "e4m3", 8, 128, 256)])
@pytest.mark.parametrize("batch", BATCHES)
def test_append_and_read(batch, dtype, cache, hkv, dh, page):
    """Codes and scales to the last bit, other rows untouched, and the rows read back."""
    ns, pasts = BATCHES[batch]
    c = Paged(dtype, cache, hkv, dh, page, ns, pasts, seed=10).upload()
    w = hkv * dh
    x = np.random.default_rng(1).standard_normal((c.total, 2, hkv, dh)).astype(np.float32)
    x *= np.exp(np.random.default_rng(2).uniform(-30, 30, (c.total, 2, hkv, 1))).astype(np.float32)
    x[0, 0, 0] = 0.0
    if c.total > 4:
        x[1, 1, 0, 3:] = 0.0
        x[2, 0] *= np.float32(1e-37) / np.abs(x[2, 0]).max()     # subnormal scales
    t = torch.from_numpy(x).to(TORCH[dtype]).cuda()
    status_ok(c.append(t[:, 0], t[:, 1], 2 * w))
    xf = t.float().cpu().numpy()
    for b in range(c.batch):
        for which in range(2):
            c.put(which, b, c.lens[b] - c.ns[b], xf[c.first[b]:c.first[b + 1], which])
    bits = torch.uint8 if cache == "e4m3" else {"bf16": torch.int16, "f32": torch.int32}[cache]
    assert torch.equal(c.g_pages.cpu().view(bits), c.pages.view(bits))
    if cache == "e4m3":
        assert torch.equal(c.g_scales.cpu().view(torch.int32), c.scales.view(torch.int32))
    back = torch.full((2, c.total, w + 16), 9.0, dtype=TORCH[dtype], device="cuda")
    status_ok(c.read(back[0], back[1], w + 16))
    got = f64(back)
    for b in range(c.batch):
        lo, hi = c.first[b], c.first[b + 1]
        for which in range(2):
            want = torch.from_numpy(c.rows(which, b, c.lens[b] - c.ns[b], c.lens[b])).float().to(TORCH[dtype])
            assert np.array_equal(got[which, lo:hi, :w].reshape(-1, hkv, dh), want.double().numpy())
    assert (got[:, c.first[-1]:] == 9.0).all() and (got[:, :, w:] == 9.0).all()


def test_append_special_values():
    """A row with a NaN or an infinity reads back as NaN throughout, and only that row."""
    c = Paged("bf16", "e4m3", 2, 128, 64, [4], [0], pad=0).upload()
    x = torch.randn(4, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    x[1, 0, 1, 7] = float("nan")
    x[2, 1, 0, 9] = -float("inf")
    status_ok(c.append(x[:, 0], x[:, 1], 512))
    back = torch.zeros(2, 4, 2, 128, dtype=torch.bfloat16, device="cuda")
    status_ok(c.read(back[0], back[1], 256))
    nan = torch.isnan(back)
    want = torch.zeros_like(nan)
    want[0, 1, 1] = True
    want[1, 2, 0] = True
    assert torch.equal(nan, want)


def test_append_bad_page_writes_nothing():
    c = Paged("bf16", "bf16", 1, 128, 64, [3, 3], [62, 0], seed=12).upload()
    before = c.g_pages.clone()
    c.g_table[0, 1] = c.n_pages
    x = torch.ones(c.total, 2, 128, dtype=torch.bfloat16, device="cuda")
    assert H.hymba_workspace_status(c.append(x[:, 0], x[:, 1], 256)) == H.HYMBA_ERR_INVALID_ARG
    now = c.g_pages.cpu()
    pg, at = c.slots(1, 0, 3)
    assert (now[:, pg, at] == 1).all()
    pg0, at0 = c.slots(0, 62, 64)
    assert (now[:, pg0, at0] == 1).all()
    now[:, pg, at] = before.cpu()[:, pg, at]
    now[:, pg0, at0] = before.cpu()[:, pg0, at0]
    assert torch.equal(now.view(torch.int16), before.cpu().view(torch.int16))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_offsets_beyond_32_bits(cache):
    """A pool whose V half starts beyond 2^31 elements, with the sequence's pages at its end."""
    hkv, page = 8, 64
    n_pages = (1 << 31) // (page * hkv * 128) + 40
    c = Paged("bf16", cache, hkv, 128, page, [70, 1], [130, 300], seed=13)
    small = c.n_pages
    c.upload()
    pages = torch.empty((2, n_pages, page, hkv, 128), dtype=TORCH[cache], device="cuda")
    pages.view(torch.uint8)[:, -small:] = c.g_pages.view(torch.uint8)
    scales = None
    if cache == "e4m3":
        scales = torch.empty((2, n_pages, hkv, page), device="cuda")
        scales[:, -small:] = c.g_scales
    c.g_table += n_pages - small
    c.g_pages, c.g_scales = pages, scales
    c.kv = H.make_paged_kv(pages, c.g_table, page, hkv, 128, c.kv.cache_type, scales=scales)
    assert c.kv.n_pages == n_pages
    for hq in (8, 16):
        q, qd = _q(c, hq)
        out = torch.zeros((c.total, hq, 128), dtype=torch.bfloat16, device="cuda")
        status_ok(c.attend(q, out, hq, 0, -1))
        want, tol = c.attention(qd, hq, 0, -1)
        _check(f64(out), want, tol)
    back = torch.zeros(2, c.total, hkv, 128, dtype=torch.bfloat16, device="cuda")
    status_ok(c.read(back[0], back[1], hkv * 128))
    for w in range(2):
        for b in range(2):
            want = torch.from_numpy(c.rows(w, b, c.lens[b] - c.ns[b], c.lens[b])).float().bfloat16().double().numpy()
            assert np.array_equal(f64(back[w, c.first[b]:c.first[b + 1]]), want)
    # the round trip through append leaves the rows as they are (the codes of a row's own values)
    status_ok(c.append(back[0], back[1], hkv * 128))
    again = torch.zeros_like(back)
    status_ok(c.read(again[0], again[1], hkv * 128))
    if cache == "bf16":
        assert torch.equal(again, back)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_chunked_prompts_run_together(cache):
    """As a server uses the calls: the layer's Q, K, V projections of two prompts come in chunks,
    each chunk is appended and attended, then generation steps follow; against the plain
    attention of the whole prompt on the K/V the cache then holds."""
    s = synth.workload("hymba1p5b_kvpair", n_layers=1, batch=1, seq_len=8, d_model=256, n_q_heads=8, n_kv_heads=2,
                       window=100).first
    d, wq, wkv, meta, window = s.d_model, s.attn_width, s.kv_width, 16, s.window
    lens, chunks = [333, 150], [[128, 60], [1, 90], [200, 0], [1, 0], [1, 0], [1, 0], [1, 0]]
    page, hkv = 32, s.n_kv_heads
    full = Paged("bf16", cache, hkv, 128, page, lens, [0, 0], seed=14)
    full.upload()
    full.g_pages.view(torch.uint8).fill_(0xff)
    g = torch.Generator("cuda")
    g.manual_seed(3)
    x = [torch.randn(n, d, generator=g, device="cuda").bfloat16() for n in lens]
    w_in = (torch.randn(wq + 2 * wkv, d, generator=g, device="cuda") * 0.06).bfloat16()
    outs, qs, done = [[], []], [[], []], [0, 0]
    ws = None
    for ns in chunks:
        total = sum(ns)
        xs = torch.cat([x[b][done[b]:done[b] + ns[b]] for b in range(2)])
        qkv = torch.empty(total, wq + 2 * wkv, dtype=torch.bfloat16, device="cuda")
        H.check(H.hymba_gemm(xs, w_in, qkv, total, wq + 2 * wkv, d, H.HYMBA_BF16, host.workspace(256)), "gemm")
        full.ns = np.array(ns)
        done = [done[b] + ns[b] for b in range(2)]
        full.lens = np.array(done)
        full.first = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        full.total = total
        full.g_first.copy_(torch.from_numpy(full.first))
        full.g_lens.copy_(torch.from_numpy(full.lens.astype(np.int32)))
        status_ok(full.append(qkv[:, wq:], qkv[:, wq + wkv:], wq + 2 * wkv))
        out = torch.empty(total, wq, dtype=torch.bfloat16, device="cuda")
        status_ok(full.attend(qkv, out, s.n_q_heads, meta, window, q_ld=wq + 2 * wkv))
        for b in range(2):
            outs[b].append(out[full.first[b]:full.first[b + 1]].clone())
            qs[b].append(qkv[full.first[b]:full.first[b + 1], :wq].clone())
    assert done == lens
    # the whole prompts at once, on the rows the cache now holds
    full.pages = full.g_pages.cpu()
    full.scales = None if full.g_scales is None else full.g_scales.cpu()
    full.ns, full.lens, full.total = np.array(lens), np.array(lens), sum(lens)
    full.first = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    q = torch.cat([torch.cat(a) for a in qs]).double().cpu().numpy().reshape(-1, s.n_q_heads, 128)
    want, tol = full.attention(q, s.n_q_heads, meta, window)
    _check(f64(torch.cat([torch.cat(a) for a in outs])).reshape(want.shape), want, tol)
    # what the cache holds is the projections' K and V (e4m3: within half a step of each row's
    # scale, 2^-4 of a value or 2^-10 of the scale for the smallest codes)
    qkv = [f64(x[b]) @ f64(w_in).T for b in range(2)]
    for b in range(2):
        for which in range(2):
            r = qkv[b][:, wq + which * wkv: wq + (which + 1) * wkv].reshape(-1, hkv, 128)
            got = full.rows(which, b, 0, lens[b])
            bound = np.abs(r) * 2.0 ** -8 + 1e-4
            if cache == "e4m3":
                bound = bound + np.abs(r) * 2.0 ** -4 * (1 + 2.0 ** -7) + np.abs(r).max(-1, keepdims=True) / 448 * 2.0 ** -9
            assert (np.abs(got - r) <= bound).all()


def test_a_prefilled_contiguous_cache_is_a_paged_one():
    """hymba_layer_prefill's cache, one page per sequence: the attention of its last rows equals
    the plain attention over the K/V it holds."""
    wl = synth.workload("hymba350m_layer", batch=2, seq_len=224, d_model=512, d_inner=512, dt_rank=32)
    s = wl.first
    x, meta = synth.layer_inputs(wl)
    dev = host.params_to_device(synth.layer_params(wl, 0), "bf16")
    cfg, rows, T = H.make_cfg(s), 384, s.T
    cache = torch.full((2, 2, rows, s.kv_width), float("nan"), dtype=torch.bfloat16, device="cuda")
    state = torch.zeros((2, s.d_inner, s.d_state), device="cuda")
    out = host.empty((2, T, s.d_model), "bf16")
    ws = host.workspace(H.hymba_decode_workspace_size(cfg))
    H.check(H.hymba_layer_prefill(host.to_device(x, "bf16"), host.to_device(meta, "bf16"), H.make_weights(dev), cfg,
                                  cache, rows, state, out, ws), "prefill")
    status_ok(ws)
    c = Paged("bf16", "bf16", s.n_kv_heads, 128, rows, [1, 31], [T - 1, T - 31], spare=0)
    c.table = np.arange(2, dtype=np.int32)[:, None]
    c.pages = cache.cpu().reshape(2, 2, rows, s.n_kv_heads, 128)
    c.n_pages = 2
    _attend(c, s.n_q_heads, s.n_meta, s.window)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_attention_is_the_same_between_other_work(cache):
    """The same bits 300 times between kernels that shift its timing and its caches: a stage freed
    before its reads were done showed in a few of hundreds of calls."""
    c = Paged("bf16", cache, 4, 128, 32, [5, 130, 1, 64, 17], [0, 257, 700, 64, 1], seed=15).upload()
    q, qd = _q(c, 16)
    out = torch.zeros((c.total, 16, 128), dtype=torch.bfloat16, device="cuda")
    ws = c.attend(q, out, 16, 8, -1)
    status_ok(ws)
    want, tol = c.attention(qd, 16, 8, -1)
    _check(f64(out), want, tol)
    ref = out.clone()
    other = torch.empty(1 << 25, device="cuda")
    for k in range(300):
        other[: 1 << (25 if k % 2 else 18)].normal_()
        out.zero_()
        c.attend(q, out, 16, 8, -1, ws=ws)
        assert torch.equal(out, ref), f"call {k}"


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "e4m3")])
@pytest.mark.parametrize("ns", [[1, 1], [40, 200]])
def test_attention_zero_queries_and_tiny_rows(dtype, cache, ns):
    """Rows of Q that are zero (a padded batch's) see the mean of V, beside masked keys and whatever
    the magnitudes of K and V are."""
    c = Paged(dtype, cache, 2, 128, 64, ns, [100, 333], seed=16)
    for b in range(2):
        for w, size in ((0, 1e-9), (1, 1e-12)):
            c.put(w, b, 0, (size * c.rng.standard_normal((c.lens[b], 2, 128))).astype(np.float32))
    c.upload()
    q, qd = _q(c, 4)
    q[::2], qd[::2] = 0, 0
    out = torch.full((c.total, 4, 128), 7.0, dtype=TORCH[dtype], device="cuda")
    status_ok(c.attend(q, out, 4, 8, 50))
    want, tol = c.attention(qd, 4, 8, 50)
    _check(f64(out), want, tol)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 90])
def test_attention_scales_far_apart(cache, n):
    """K and V rows whose magnitudes differ by 2^20 within a head, the large ones early or late."""
    c = Paged("bf16", cache, 2, 128, 64, [n, n], [400, 300], seed=17)
    for b in range(2):
        for j in (5, 200, 290):
            c.put(0, b, j, (2.0 ** -20 * c.rng.standard_normal((1, 2, 128))).astype(np.float32))
            c.put(1, b, j, (2.0 ** (20 if j == 200 else -20) * c.rng.standard_normal((1, 2, 128))).astype(np.float32))
    _attend(c, 8, 0, 64)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_attention_many_parts(cache, n):
    """A tile or a few over a long history: every CTA has a part or two of one."""
    _attend(Paged("bf16", cache, 1, 128, 64, [n], [30000], seed=19), 2, 8, -1)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("batch,n", [(70, 33), (1100, 1)])
def test_attention_large_batches(cache, batch, n):
    """Batches beyond what a CTA plans itself, some sequences empty."""
    r = np.random.default_rng(18)
    ns = r.integers(0, n + 1, batch)
    _attend(Paged("bf16", cache, 1, 128, 16, list(ns), list(r.integers(0, 60, batch)), seed=18), 2, 8, -1)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
def test_sequences_may_share_pages(dtype, cache):
    """The pages of one prompt's beginning in the tables of several sequences."""
    c = Paged(dtype, cache, 2, 128, 64, [1, 1, 20], [200, 250, 300], seed=19)
    c.table[1, :2] = c.table[0, :2]
    c.table[2, :2] = c.table[0, :2]
    _attend(c, 4, 0, -1)


@pytest.mark.parametrize("dtype,cache,most", [("bf16", "bf16", 1), ("bf16", "e4m3", 300), ("f32", "f32", 5)])
def test_attention_of_no_rows(dtype, cache, most):
    c = Paged(dtype, cache, 2, 128, 64, [0, 0], [30, 0], pad=4).upload()
    q, _ = _q(c, 4)
    out = torch.full((4, 4, 128), 7.0, dtype=TORCH[dtype], device="cuda")
    status_ok(c.attend(q, out, 4, 0, -1, max_rows=most))
    assert (out == 7.0).all()


def test_two_graphs_share_a_workspace_in_order():
    """Two captured calls of different shapes on one workspace, replayed one after the other."""
    c = [Paged("bf16", "e4m3", 2, 128, 64, ns, pasts, seed=20 + i).upload()
         for i, (ns, pasts) in enumerate([([200, 1], [300, 40]), ([1, 1, 1], [500, 2, 90])])]
    qs = [_q(x, 8) for x in c]
    outs = [torch.zeros((x.total, 8, 128), dtype=torch.bfloat16, device="cuda") for x in c]
    ws = host.workspace(max(x.workspace(8).numel() for x in c))
    for x, q, o in zip(c, qs, outs):
        x.attend(q[0], o, 8, 0, -1, ws=ws)
    graphs = []
    for x, q, o in zip(c, qs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            x.attend(q[0], o, 8, 0, -1, ws=ws, stream=torch.cuda.current_stream())
    for _ in range(5):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        status_ok(ws)
        for x, q, o in zip(c, qs, outs):
            want, tol = x.attention(q[1], 8, 0, -1)
            _check(f64(o), want, tol)
