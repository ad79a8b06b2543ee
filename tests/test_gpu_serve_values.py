"""Values the serving calls have to keep: weights next to the largest number; NaN in Q and in
visible rows of the cache; rows of K and V whose magnitudes lie far apart."""
import numpy as np
import pytest
import torch

import hybrid_attention_ssm_hymba_b200 as H
from gpu_util import requires_cuda, status_ok
from serve_util import DTYPE, TINY, TORCH, Paged, f64

pytestmark = [pytest.mark.gpu, requires_cuda]


# --------------------------------------------------------------------------- 4-bit weights

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 128])
def test_quantise_w4_of_the_largest_weights(dtype, group):
    """Groups whose largest weight is next to the type's largest number, and on both sides of a
    seventh of it, where 7 w leaves fp32's range."""
    top = torch.finfo(TORCH[dtype]).max
    r = np.random.default_rng(group)
    most = np.array([top, top / 2, top / 6.9, top / 7.0, top / 7.1, 1e37, 1e36])
    w = r.uniform(-1, 1, (len(most), 2 * group)) * most[:, None]
    w[:, 3] = most * np.where(np.arange(len(most)) % 2, -1, 1)
    w[:, group + 5] = most
    t = torch.from_numpy(w).clamp(-top, top).to(TORCH[dtype]).cuda()
    assert torch.isfinite(t).all()
    n, k = t.shape
    q4 = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    sc = torch.empty(n, k // group, device="cuda")
    H.check(H.hymba_quantize_w4(t, q4, sc, n, k, group, DTYPE[dtype]), "quantize")
    x = t.double().cpu().numpy().reshape(n, -1, group)
    amax = np.abs(x).max(-1)
    q = np.rint(7 * x / amax[..., None]).reshape(n, k)
    scale = np.maximum(amax.astype(np.float32) / np.float32(7), TINY)
    got = q4.cpu().numpy()
    assert np.array_equal((got & 15) - 8.0, q[:, 0::2]) and np.array_equal((got >> 4) - 8.0, q[:, 1::2])
    assert np.array_equal(sc.cpu().numpy(), scale)


# --------------------------------------------------------------------------- not finite

def _q(c, hq, seed=5):
    q = np.random.default_rng(seed).standard_normal((c.total, hq, c.dh)).astype(np.float32)
    return torch.from_numpy(q).to(TORCH[c.dtype])


def _row_tolerance(c, q, hq, meta, window):
    """(out, tolerance) in 64 bits as in Paged.attention, with each row's own scores in its
    tolerance (one row's huge scores say nothing about another's), and what 8-bit rows add: P is
    held in 16 bits with a common power of two a row, 2^-25 at least, the largest p_j amax_j / 448
    of the row at 2^8 or more: L 2^-33 max_j p_j amax_j in all, and as much again for its lag."""
    want, _ = c.attention(q, hq, meta, window)
    tol = np.full_like(want, np.nan)
    g = hq // c.hkv
    for b in range(c.batch):
        at = slice(c.first[b], c.first[b + 1])
        see = c.visible(b, meta, window)
        k, v = np.nan_to_num(c.rows(0, b, 0, c.lens[b])), np.nan_to_num(c.rows(1, b, 0, c.lens[b]))
        for h in range(hq):
            qq, kk, vv = q[at, h], k[:, h // g], np.abs(v[:, h // g])
            s = np.where(see, qq @ kk.T / np.sqrt(c.dh), -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            size = np.where(see, np.abs(qq) @ np.abs(kk).T, 0) / np.sqrt(c.dh) * (c.dh + 2) * 2.0 ** -24
            # a score's error matters by its key's weight: 2 ds, and never more than the whole row
            a = p @ vv
            ds = np.minimum(2 * size.max(1, keepdims=True), 1.0)
            t = a * (ds + (c.lens[b] + 16) * 2.0 ** -23) + np.abs(want[at, h]) * 2.0 ** -8 + a * 2.0 ** -8
            tol[at, h] = t + c.lens[b] * 2.0 ** -32 * (p * vv.max(1)[None]).max(1, keepdims=True)
    return want, tol


def _close(got, want, tol, rows=None):
    rows = np.arange(len(want)) if rows is None else np.asarray(rows)
    g, w, t = got[rows], want[rows], tol[rows]
    assert np.isfinite(g).all(), f"{int((~np.isfinite(g)).sum())} values that are not finite"
    bad = np.abs(g - w) - t
    assert (bad <= 0).all(), f"{int((bad > 0).sum())} values beyond the tolerance; worst {np.nanmax(np.abs(g - w) / t):.3e} of it"


FORMS = [("f32", "f32"), ("f32", "e4m3"), ("bf16", "bf16"), ("bf16", "e4m3")]

# one block a tile; tiles of several blocks, which few tiles in a call cut into parts; a row's
# last key alone in its block, or in its piece of the keys
SHAPES = [([1, 1], [32, 0]), ([1, 3], [128, 40]), ([1], [4000]), ([60, 40], [0, 10]), ([20, 129], [237, 128]),
          ([200, 3], [313, 5])]


@pytest.mark.parametrize("dtype,cache", FORMS)
@pytest.mark.parametrize("ns,pasts", SHAPES)
def test_a_nan_query_row_is_a_nan_output_row(ns, pasts, dtype, cache):
    c = Paged(dtype, cache, 2, 128, 64, ns, pasts, seed=31).upload()
    hq = 4
    q = _q(c, hq)
    want, tol = _row_tolerance(c, q.double().numpy(), hq, 0, -1)
    bad = sorted({0, int(c.first[1]) - 1})
    q[bad, 1] = float("nan")
    out = torch.zeros((c.total, hq, 128), dtype=TORCH[dtype], device="cuda")
    status_ok(c.attend(q.cuda(), out, hq, 0, -1))
    got = f64(out)
    assert np.isnan(got[bad, 1]).all(), "a NaN row of Q gave numbers"
    got[bad, 1] = want[bad, 1]
    _close(got[:c.first[-1]], want[:c.first[-1]], tol[:c.first[-1]])


@pytest.mark.parametrize("dtype,cache", FORMS)
@pytest.mark.parametrize("ns,pasts", SHAPES)
@pytest.mark.parametrize("which", [0, 1])
def test_a_nan_token_reaches_its_own_row(which, ns, pasts, dtype, cache):
    """The newest K or V row of a sequence is NaN (as an append of a NaN leaves it): the last row's
    output is NaN for the heads that read it, whole tile or cut; other sequences are as they were."""
    c = Paged(dtype, cache, 2, 128, 64, ns, pasts, seed=32)
    hq = 4
    q = _q(c, hq)
    want, tol = _row_tolerance(c, q.double().numpy(), hq, 0, -1)
    x = np.random.default_rng(3).standard_normal((1, 2, 128)).astype(np.float32)
    x[0, 1] = np.nan
    c.put(which, 0, c.lens[0] - 1, x)
    c.upload()
    out = torch.zeros((c.total, hq, 128), dtype=TORCH[dtype], device="cuda")
    status_ok(c.attend(q.cuda(), out, hq, 0, -1))
    got, last = f64(out), int(c.first[1]) - 1
    assert np.isnan(got[last, 2:]).all(), "the row that sees a NaN gave numbers"
    assert np.isfinite(got[last, :2]).all()
    rest = np.arange(c.first[1], c.first[-1])
    if len(rest):
        _close(got, want, tol, rest)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("ns,pasts", SHAPES)
def test_an_infinite_value_of_no_weight(ns, pasts, cache):
    """A visible V row of infinities (NaN in an e4m3 cache) whose weight is too small for fp32: 0 times
    it is NaN, whole tile or cut."""
    c = Paged("bf16", cache, 2, 128, 64, ns, pasts, seed=37)
    x = np.zeros((1, 2, 128), np.float32)
    c.put(1, 0, 0, np.where(np.arange(2)[:, None] == 1, np.inf, x).astype(np.float32))
    x[:, :, 0] = -400
    c.put(0, 0, 0, x)
    c.upload()
    q = _q(c, 4)
    q[:, :, 0] = 16
    out = torch.zeros((c.total, 4, 128), dtype=torch.bfloat16, device="cuda")
    status_ok(c.attend(q.cuda(), out, 4, 0, -1))
    got, last = f64(out), int(c.first[1]) - 1
    assert np.isnan(got[last, 2:]).all() and np.isfinite(got[last, :2]).all()


# --------------------------------------------------------------------------- far apart

def _largest_score(c, q, hq, b, window):
    """Of each new row of sequence b, over its heads and the keys that it sees."""
    k, g = np.nan_to_num(c.rows(0, b, 0, c.lens[b])), hq // c.hkv
    see = c.visible(b, 0, window)
    qb = q[c.first[b]:c.first[b + 1]]
    return np.max([np.where(see, np.abs(qb[:, h] @ k[:, h // g].T), 0).max(1) for h in range(hq)], 0) / np.sqrt(c.dh)


@pytest.mark.parametrize("up", [24, 30, 45, 60])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_a_large_k_row_that_a_query_does_not_see(n, cache, up):
    """A row of K 2^up times the others, in the window of some queries of a tile and not of the
    rest: those are as exact as without it.  (Rows that see a score beyond 2^20 are outside the
    call's range.)"""
    c = Paged("bf16", cache, 2, 128, 64, [n, n], [400, 300], seed=33)
    window, hq = 64, 8
    for b in range(2):
        lo = c.lens[b] - c.ns[b]
        for j in (lo - window, lo + n // 2):     # the first query's last key; one that appears halfway
            if j < c.lens[b] - 1:
                c.put(0, b, j, (2.0 ** up * c.rng.standard_normal((1, 2, 128))).astype(np.float32))
    c.upload()
    q = _q(c, hq)
    want, tol = _row_tolerance(c, q.double().numpy(), hq, 0, window)
    out = torch.zeros((c.total, hq, 128), dtype=torch.bfloat16, device="cuda")
    status_ok(c.attend(q.cuda(), out, hq, 0, window))
    rows = np.arange(c.first[-1])
    mine = np.concatenate([_largest_score(c, q.double().numpy(), hq, b, window) for b in range(2)]) < 2.0 ** 20
    assert mine.sum() > len(rows) // 3 or n == 1
    _close(f64(out), want, tol, rows[mine])


@pytest.mark.parametrize("up", [12, 21, 24, 30, 45, 80])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,past", [(1, 400), (40, 400), (300, 300), (20, 2000)])
def test_a_large_v_row_that_a_query_does_not_see(n, past, cache, up):
    """The same for V: large rows at the window's far end and halfway through the new rows, and
    small ones between; also with the roles of large and small exchanged."""
    for sign in (1, -1):
        c = Paged("bf16", cache, 2, 128, 64, [n, n], [past, past - 100], seed=34)
        window, hq = 200, 8
        for b in range(2):
            lo = c.lens[b] - c.ns[b]
            for j in (lo - window, lo - window + 1, lo + n // 2):
                if 0 <= j < c.lens[b]:
                    c.put(1, b, j, (2.0 ** (sign * up) * c.rng.standard_normal((1, 2, 128))).astype(np.float32))
        c.upload()
        q = _q(c, hq)
        want, tol = _row_tolerance(c, q.double().numpy(), hq, 0, window)
        out = torch.zeros((c.total, hq, 128), dtype=torch.bfloat16, device="cuda")
        status_ok(c.attend(q.cuda(), out, hq, 0, window))
        _close(f64(out), want, tol, np.arange(c.first[-1]))


@pytest.mark.parametrize("n,past", [(1, 700), (90, 700), (300, 2000)])
def test_v_scales_of_every_magnitude(n, past):
    """V rows over 2^+-50 in random order, zero rows among them (their scale is the least one), in a
    window and in all keys: each output row is exact beside its own largest terms."""
    for window in (-1, 300):
        c = Paged("bf16", "e4m3", 2, 128, 32, [n, 5], [past, 90], seed=35)
        for b in range(2):
            x = c.rng.standard_normal((c.lens[b], 2, 128)) * 2.0 ** c.rng.integers(-50, 50, (c.lens[b], 2, 1))
            x[:: 7] = 0
            c.put(1, b, 0, x.astype(np.float32))
        c.upload()
        q = _q(c, 8)
        want, tol = _row_tolerance(c, q.double().numpy(), 8, 16, window)
        out = torch.zeros((c.total, 8, 128), dtype=torch.bfloat16, device="cuda")
        status_ok(c.attend(q.cuda(), out, 8, 16, window))
        _close(f64(out), want, tol, np.arange(c.first[-1]))


@pytest.mark.parametrize("n,batch", [(1, 200), (90, 3)])
@pytest.mark.parametrize("up", [0, 60, 75])
def test_rising_scores_with_large_values(n, batch, up):
    """Scores that rise by 50 powers of two after the first keys, over V rows of 2^up, in enough
    sequences that a CTA takes several blocks of one: sums that are held relative to an early
    maximum stay finite."""
    c = Paged("bf16", "e4m3", 1, 128, 64, [n] * batch, [600] * batch, seed=36)
    k = np.zeros((c.lens[0], 1, 128), np.float32)
    k[128:, 0, 0] = 50 / (8 * 1.4426950408889634 / np.sqrt(128))
    for b in range(batch):
        c.put(0, b, 0, k)
        c.put(1, b, 0, (2.0 ** up * (2 + c.rng.random((c.lens[b], 1, 128)))).astype(np.float32))
    c.upload()
    q = torch.zeros(c.total, 4, 128, dtype=torch.bfloat16)
    q[:, :, 0] = 8
    want, tol = _row_tolerance(c, q.double().numpy(), 4, 0, -1)
    out = torch.zeros((c.total, 4, 128), dtype=torch.bfloat16, device="cuda")
    status_ok(c.attend(q.cuda(), out, 4, 0, -1))
    _close(f64(out), want, tol, np.arange(c.first[-1]))
