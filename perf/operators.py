"""Cases of the serving operators: the paged K/V cache (written with or without quantisation,
read back, attended over) and the products with 4-bit weights.

Where `own` is false, `run` computes each operator in its plain form with elementary torch
operations; where it is true, it makes the library's calls.  Shapes follow this repository's
workloads: 16 query heads over 4 K/V heads (or 12 over 2, 2 over 1) of 128, window 1024 with
128 meta rows, d_model 2048, FFN 5632.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126          # the smallest normal fp32: the least scale
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "e4m3": 1}


# --------------------------------------------------------------------------- the cases

def listed():
    cache = {"hkv": 4, "dh": 128}
    return [
        # one new token for each of four sequences, as a generation step writes it
        {"name": "append 4 tokens e4m3", "op": "append", "dtype": "bf16", "cache": "e4m3", **cache, "page": 64,
         "batch": 4, "n_lo": 1, "n_hi": 1, "past_lo": 1000, "past_hi": 8320, "lens": 1},
        # the prompts of a batch (8192 tokens and the 128 meta rows each) into the cache
        {"name": "append 4 prompts e4m3", "op": "append", "dtype": "bf16", "cache": "e4m3", **cache, "page": 64,
         "batch": 4, "n_lo": 8320, "n_hi": 8320, "past_lo": 0, "past_hi": 0, "lens": 2},
        # ragged pieces read back in fp32 from an fp32 cache with small pages
        {"name": "read ragged f32", "op": "read", "dtype": "f32", "cache": "f32", "hkv": 2, "dh": 32, "page": 16,
         "batch": 7, "n_lo": 0, "n_hi": 301, "past_lo": 0, "past_hi": 200, "lens": 3},
        # whole quantised histories read back for a layer that wants them in bf16
        {"name": "read 4 prompts e4m3", "op": "read", "dtype": "bf16", "cache": "e4m3", **cache, "page": 64,
         "batch": 4, "n_lo": 8000, "n_hi": 8320, "past_lo": 0, "past_hi": 0, "lens": 4},
        # a generation step's attention in a sliding-window layer: latency counts
        {"name": "decode 4 window bf16", "op": "attention", "dtype": "bf16", "cache": "bf16", "hq": 16, **cache,
         "page": 64, "batch": 4, "n_lo": 1, "n_hi": 1, "past_lo": 8000, "past_hi": 8320, "lens": 5, "meta": 128,
         "window": 1024},
        # a generation step's attention in a global layer over long ragged histories: bandwidth counts
        {"name": "decode 16 long e4m3", "op": "attention", "dtype": "bf16", "cache": "e4m3", "hq": 16, **cache,
         "page": 64, "batch": 16, "n_lo": 1, "n_hi": 1, "past_lo": 4000, "past_hi": 32895, "lens": 6, "meta": 128,
         "window": -1},
        # chunks of prompts beside generating sequences, sliding-window layer, quantised cache
        {"name": "chunks ragged e4m3", "op": "attention", "dtype": "bf16", "cache": "e4m3", "hq": 12, "hkv": 2,
         "dh": 128, "page": 32, "batch": 9, "n_lo": 1, "n_hi": 2048, "past_lo": 0, "past_hi": 6000, "lens": 7,
         "meta": 128, "window": 1024},
        # a long chunk of one prompt in a global layer: the tensor cores count
        {"name": "chunk 4096 of 32K bf16", "op": "attention", "dtype": "bf16", "cache": "bf16", "hq": 16, **cache,
         "page": 128, "batch": 1, "n_lo": 4096, "n_hi": 4096, "past_lo": 28800, "past_hi": 28800, "lens": 8,
         "meta": 128, "window": -1},
        # a square projection's fp32 master weights into 4 bits and back, small groups
        {"name": "w4 weights f32", "op": "w4", "dtype": "f32", "n": 2048, "k": 2048, "group": 32},
        # the FFN's gate and up rows from bf16
        {"name": "w4 weights bf16", "op": "w4", "dtype": "bf16", "n": 11264, "k": 2048, "group": 128},
        # the FFN's down product of one new token
        {"name": "gemm_w4 1 row", "op": "gemm_w4", "dtype": "bf16", "m": 1, "n": 2048, "k": 5632, "group": 128},
        # a wide projection for eight sequences
        {"name": "gemm_w4 8 rows", "op": "gemm_w4", "dtype": "bf16", "m": 8, "n": 16384, "k": 8192, "group": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "attention", "w4", "gemm_w4"])
    if op == "w4":
        group = rng.choice([32, 64, 128])
        return {"op": op, "dtype": rng.choice(["f32", "bf16"]), "n": _log(rng, 1, 8192),
                "k": group * _log(rng, 1, 8192 // group), "group": group}
    if op == "gemm_w4":
        group = rng.choice([32, 64, 128])
        return {"op": op, "dtype": rng.choice(["f32", "bf16", "bf16"]), "m": rng.randint(1, 16),
                "n": _log(rng, 1, 16384), "k": group * _log(rng, 1, 8192 // group), "group": group}
    dtype = rng.choice(["f32", "bf16", "bf16"])
    c = {"op": op, "dtype": dtype, "cache": rng.choice([dtype, "e4m3"]), "hkv": rng.choice([1, 2, 3, 4, 5, 8]),
         "dh": 128 if dtype == "bf16" else rng.choice([32, 64, 128]), "page": rng.choice([8, 16, 32, 64, 128, 256]),
         "batch": _log(rng, 1, 32), "lens": rng.randrange(1 << 20)}
    if op != "attention":
        rows = _log(rng, 1, 16384)          # new rows of the whole batch
        c.update(n_lo=0, n_hi=max(1, 2 * rows // c["batch"]), past_lo=0, past_hi=_log(rng, 1, 8192))
        return c
    group = rng.choice([1, 2, 3, 4, 5, 6, 8])
    c["hkv"] = rng.choice([1, 2, 4])
    c["hq"] = group * c["hkv"]
    # pairs of the whole batch and every head stay below a quarter of the largest listed case
    past = _log(rng, 1, 32768)
    if dtype == "f32":
        past = min(past, 4096)
    most = (5e8 if dtype == "bf16" else 1e7) / (c["batch"] * c["hq"])
    n = max(1, min(4096, int(most / (past + 512))))
    n = _log(rng, 1, n)
    c.update(n_lo=rng.choice([0, 1, n]), n_hi=n, past_lo=0, past_hi=past, meta=8 * rng.randint(0, 16),
             window=rng.choice([-1, -1, 0, rng.randint(1, 2048), 1024]))
    return c


def _lens(case):
    """New rows and cache rows (with the new ones) of each sequence."""
    r = np.random.RandomState(case["lens"])
    n = r.randint(case["n_lo"], case["n_hi"] + 1, case["batch"])
    if n.sum() == 0:
        n[0] = 1
    if case["op"] == "attention" and case["batch"] > 4 and case["n_hi"] > 64:
        n[1::2] = np.minimum(n[1::2], 1)    # every other sequence generates, the rest take a chunk
    past = r.randint(case["past_lo"], case["past_hi"] + 1, case["batch"])
    return n, n + past


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    dt = TORCH[case["dtype"]]
    s = dict(case)
    if case["op"] in ("w4", "gemm_w4"):
        N, K, G = case["n"], case["k"], case["group"]
        if case["op"] == "w4":
            s["w"] = (normal(N, K) * 0.02).to(dt)
            s["codes"] = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(N, K // G, device="cuda")
            s["back"] = torch.empty(N, K, dtype=dt, device="cuda")
        else:
            s["a"] = normal(case["m"], K).to(dt)
            s["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
            s["scales"] = 0.003 + 0.004 * torch.rand(N, K // G, generator=g, device="cuda")
            s["c"] = torch.empty(case["m"], N, dtype=dt, device="cuda")
        return s
    B, hkv, dh, P, ct = case["batch"], case["hkv"], case["dh"], case["page"], case["cache"]
    n, length = _lens(case)
    need = -(-length // P)
    s["n_pages"] = int(need.sum()) + 3
    order = np.random.RandomState(seed % (1 << 31)).permutation(s["n_pages"])
    table = np.full((B, int(need.max()) + 1), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    s["table"] = torch.from_numpy(table).cuda()
    s["q_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
    s["kv_len"] = torch.from_numpy(length.astype(np.int32)).cuda()
    s["most"], s["longest"], s["used"] = int(n.max()), int(length.max()), int(n.sum())
    s["rows"] = s["used"] + (5 if B > 1 else 0)      # a padded batch: rows behind the last sequence
    pool = (2, s["n_pages"], P, hkv, dh)
    if ct == "e4m3":
        # rows of many magnitudes, as the heads of a trained layer have them
        x = normal(*pool[1:]).clamp(-4, 4)
        s["pages"] = torch.stack([(x * (E4M3_MAX / 4)).to(TORCH[ct]), (x.flip(0) * (E4M3_MAX / 4)).to(TORCH[ct])])
        s["scales"] = (4 / E4M3_MAX) * (0.5 + torch.rand(2, s["n_pages"], hkv, P, generator=g, device="cuda"))
    else:
        s["pages"] = torch.stack([normal(*pool[1:]).to(TORCH[ct]), normal(*pool[1:]).to(TORCH[ct])])
        s["scales"] = None
    if case["op"] == "attention":
        w = case["hq"] * dh
        s["q"] = normal(s["rows"], w).to(dt)
        s["out"] = torch.zeros(s["rows"], w, dtype=dt, device="cuda")
    elif case["op"] == "append":
        # K and V as columns of one projection's output
        s["kv"] = (normal(s["rows"], 2, hkv, dh) * (0.25 + 2 * torch.rand(s["rows"], 2, hkv, 1, generator=g, device="cuda"))).to(dt)
    else:
        s["back"] = torch.zeros(2, s["rows"], hkv, dh, dtype=dt, device="cuda")
    s["keep"] = {}
    return s


# --------------------------------------------------------------------------- the library's calls

def _handle(s):
    """What a program makes once for its cache and keeps: the descriptor and the workspace."""
    import hybrid_attention_ssm_hymba_b200 as H
    from hybrid_attention_ssm_hymba_b200 import host
    if "cache" not in s["keep"]:
        ct = {"f32": H.HYMBA_CACHE_F32, "bf16": H.HYMBA_CACHE_BF16, "e4m3": H.HYMBA_CACHE_E4M3}[s["cache"]]
        kv = H.make_paged_kv(s["pages"], s["table"], s["page"], s["hkv"], s["dh"], ct, scales=s["scales"])
        need = 256
        if s["op"] == "attention":
            need = H.hymba_paged_attention_workspace_size(kv, s["batch"], s["rows"], s["most"], s["hq"], _dtype(H, s))
        s["keep"]["cache"], s["keep"]["ws"] = kv, host.workspace(need)
    return H, s["keep"]["cache"], s["keep"]["ws"]


def _dtype(H, s):
    return H.HYMBA_BF16 if s["dtype"] == "bf16" else H.HYMBA_F32


def _run_own(s):
    if s["op"] == "w4":
        import hybrid_attention_ssm_hymba_b200 as H
        N, K, G = s["n"], s["k"], s["group"]
        H.check(H.hymba_quantize_w4(s["w"], s["codes"], s["scales"], N, K, G, _dtype(H, s)), "quantize_w4")
        H.check(H.hymba_dequantize_w4(s["codes"], s["scales"], s["back"], N, K, G, _dtype(H, s)), "dequantize_w4")
        return {"scales": s["scales"], "weights": s["back"]}
    if s["op"] == "gemm_w4":
        import hybrid_attention_ssm_hymba_b200 as H
        H.check(H.hymba_gemm_w4(s["a"], s["codes"], s["scales"], s["c"], s["m"], s["n"], s["k"], s["group"],
                                _dtype(H, s)), "gemm_w4")
        return s["c"]
    H, kv, ws = _handle(s)
    w = s["hkv"] * s["dh"]
    if s["op"] == "append":
        H.check(H.hymba_paged_kv_append(kv, s["kv"][:, 0], s["kv"][:, 1], 2 * w, s["batch"], s["q_start"], s["kv_len"],
                                        s["rows"], _dtype(H, s), ws), "paged_kv_append")
        return {"pages": s["pages"], "scales": s["scales"]}
    if s["op"] == "read":
        H.check(H.hymba_paged_kv_read(kv, s["back"][0], s["back"][1], w, s["batch"], s["q_start"], s["kv_len"],
                                      s["rows"], _dtype(H, s), ws), "paged_kv_read")
        return s["back"]
    wq = s["hq"] * s["dh"]
    H.check(H.hymba_paged_attention(s["q"], wq, kv, s["out"], wq, s["batch"], s["q_start"], s["kv_len"], s["rows"],
                                    s["most"], s["hq"], s["meta"], s["window"], _dtype(H, s), ws), "paged_attention")
    return s["out"]


# --------------------------------------------------------------------------- the plain forms

def run(s):
    if own:
        return _run_own(s)
    return {"append": _append, "read": _read, "attention": _attention, "w4": _w4, "gemm_w4": _gemm_w4}[s["op"]](s)


def _places(s):
    """Page and row in the page of every new row of the batch."""
    q0, length = s["q_start"].long(), s["kv_len"].long()
    row = torch.arange(s["used"], device="cuda")
    b = torch.searchsorted(q0, row, right=True) - 1
    at = length[b] - q0[b + 1] + row                 # the row of the sequence
    return s["table"][b, at // s["page"]].long(), at % s["page"]


def _append(s):
    page, at = _places(s)
    x = s["kv"][:s["used"]].transpose(0, 1)          # [2, rows, hkv, dh]
    if s["cache"] != "e4m3":
        s["pages"][:, page, at] = x.to(s["pages"].dtype)
        return {"pages": s["pages"], "scales": None}
    x = x.float()
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
    code = (x * (1.0 / scale)[..., None]).to(torch.float8_e4m3fn)
    s["pages"].view(torch.uint8)[:, page, at] = code.view(torch.uint8)
    s["scales"][:, page, :, at] = scale.transpose(0, 1)
    return {"pages": s["pages"], "scales": s["scales"]}


def _read(s):
    page, at = _places(s)
    x = s["pages"].view(torch.uint8)[:, page, at].view(TORCH["e4m3"]) if s["cache"] == "e4m3" else s["pages"][:, page, at]
    x = x.float()
    if s["scales"] is not None:
        x = x * s["scales"][:, page, :, at].transpose(0, 1)[..., None]
    s["back"][:, :s["used"]] = x.to(s["back"].dtype)
    return s["back"]


def _attention(s):
    B, hkv, dh, P, L, n = s["batch"], s["hkv"], s["dh"], s["page"], s["longest"], s["most"]
    G = s["hq"] // hkv
    q0, length = s["q_start"].long(), s["kv_len"].long()
    new = q0[1:] - q0[:-1]
    pages = s["table"][:, :-(-L // P)].clamp_min(0).long()
    if s["scales"] is None:
        kv = s["pages"][:, pages].float()                                   # [2, B, pages, P, hkv, dh]
    else:
        kv = s["pages"].view(torch.uint8)[:, pages].view(TORCH["e4m3"]).float()
        kv = kv * s["scales"][:, pages].transpose(-1, -2)[..., None]
    k, v = kv.reshape(2, B, -1, hkv, dh)[:, :, :L].permute(0, 1, 3, 4, 2)     # [B, hkv, dh, L]
    i = torch.arange(n, device="cuda")
    row = (q0[:-1, None] + i).clamp_max(s["rows"] - 1)                       # [B, n]
    q = s["q"][row].float().reshape(B, n, hkv, G, dh).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * n, dh)
    score = (q @ k).reshape(B, hkv, G, n, L) * (1.0 / math.sqrt(dh))
    pos = ((length - new)[:, None] + i)[:, :, None]                           # [B, n, 1]
    j = torch.arange(L, device="cuda")
    see = (j <= pos) & (j < length[:, None, None])
    if s["window"] >= 0:
        see = see & ((pos - j <= s["window"]) | (j < s["meta"]))
    score.masked_fill_(~see[:, None, None], -math.inf)
    score -= score.amax(-1, keepdim=True).clamp_min(-1e30)
    p = score.exp_()
    o = p.reshape(B, hkv, G * n, L) @ v.transpose(-1, -2)
    o = o.reshape(B, hkv, G, n, dh) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * n, hkv * G * dh)
    r = torch.arange(s["used"], device="cuda")
    b = torch.searchsorted(q0, r, right=True) - 1
    out = torch.zeros_like(s["out"])
    out[:s["used"]] = o[b * n + r - q0[b]].to(out.dtype)
    return out


def _w4(s):
    w = s["w"].float().reshape(s["n"], -1, s["group"])
    most = w.abs().amax(-1)
    scale = (most / 7).clamp_min(TINY)
    # in 64 bits: bf16 weights often lie halfway between two codes
    code = (w.double() * 7 / most.clamp_min(TINY)[..., None]).round().float()
    back = (code * scale[..., None]).reshape(s["n"], s["k"]).to(s["back"].dtype)
    return {"scales": scale, "weights": back}


def _gemm_w4(s):
    q = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).reshape(s["n"], -1, s["group"]).float() - 8
    w = (q * s["scales"][..., None]).reshape(s["n"], s["k"])
    return (s["a"].float() @ w.t()).to(s["c"].dtype)


# --------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "w4":
        N, K, G = case["n"], case["k"], case["group"]
        w = s["w"].double()
        most = torch.stack([c.abs().amax(1) for c in w.split(G, dim=1)], 1)
        wide = most.repeat_interleave(G, 1)
        return {"scales": most / 7, "weights": torch.where(wide > 0, torch.round(7 * w / wide), 0.0) * wide / 7}
    if case["op"] == "gemm_w4":
        q = torch.empty(case["n"], case["k"], dtype=torch.float64, device="cuda")
        q[:, 0::2], q[:, 1::2] = (s["codes"] % 16).double(), (s["codes"] // 16).double()
        q = (q - 8) * s["scales"].double().repeat_interleave(case["group"], 1)
        return torch.einsum("mk,nk->mn", s["a"].double(), q)
    n, length = _lens(case)
    table = s["table"].cpu().numpy()
    first = np.concatenate([[0], np.cumsum(n)])
    P = case["page"]

    def slots(b, lo, hi):
        r = np.arange(lo, hi)
        return torch.from_numpy(table[b, r // P].astype(np.int64) * P + r % P).cuda()

    flat = s["pages"].reshape(2, -1, case["hkv"], case["dh"])
    scale = None if s["scales"] is None else s["scales"].transpose(-1, -2).reshape(2, -1, case["hkv"])
    if case["op"] == "append":
        x = s["kv"].double()
        pages = flat.double()
        sc = None if scale is None else scale.double()
        for b in range(case["batch"]):
            at = slots(b, length[b] - n[b], length[b])
            new = x[first[b]:first[b + 1]].transpose(0, 1)
            if sc is None:
                pages[:, at] = new
            else:
                step = new.abs().amax(-1) / E4M3_MAX
                sc[:, at] = step
                pages[:, at] = torch.where(step[..., None] > 0, new / step[..., None], 0.0).to(torch.float8_e4m3fn).double()
        sc = None if sc is None else sc.reshape(2, -1, P, case["hkv"]).transpose(-1, -2).contiguous()
        return {"pages": pages.reshape(s["pages"].shape), "scales": sc}

    def rows(which, b, lo, hi):
        at = slots(b, lo, hi)
        if scale is None:
            return flat[which][at].double()
        return flat[which].view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * scale[which][at].double()[..., None]

    if case["op"] == "read":
        back = torch.zeros(s["back"].shape, dtype=torch.float64, device="cuda")
        for b in range(case["batch"]):
            back[0, first[b]:first[b + 1]] = rows(0, b, length[b] - n[b], length[b])
            back[1, first[b]:first[b + 1]] = rows(1, b, length[b] - n[b], length[b])
        return back
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    dh, G = case["dh"], case["hq"] // case["hkv"]
    for b in range(case["batch"]):
        if n[b] == 0:
            continue
        k, v = rows(0, b, 0, length[b]), rows(1, b, 0, length[b])
        i = torch.arange(length[b] - n[b], length[b], device="cuda")[:, None]
        j = torch.arange(length[b], device="cuda")[None]
        hidden = (j > i) | ((i - j > case["window"]) & (j >= case["meta"]) if case["window"] >= 0 else j < 0)
        for h in range(case["hq"]):
            q = s["q"][first[b]:first[b + 1], h * dh:(h + 1) * dh].double()
            t = (q @ k[:, h // G].t()) / math.sqrt(dh)
            out[first[b]:first[b + 1], h * dh:(h + 1) * dh] = torch.softmax(t.masked_fill_(hidden, -math.inf), -1) @ v[:, h // G]
    return out


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "w4":
        N, K, G = case["n"], case["k"], case["group"]
        return {"bytes": N * K * (2 * es + 0.5) + 4 * N * K / G, "flops": 4 * N * K}
    if case["op"] == "gemm_w4":
        M, N, K, G = case["m"], case["n"], case["k"], case["group"]
        return {"bytes": N * K / 2 + 4 * N * K / G + es * M * (N + K), "flops": 2 * M * N * K}
    n, length = _lens(case)
    row = case["hkv"] * (case["dh"] * BYTES[case["cache"]] + (4 if case["cache"] == "e4m3" else 0))
    new = int(n.sum())
    if case["op"] != "attention":
        return {"bytes": 2 * new * (row + case["hkv"] * case["dh"] * es), "flops": 2 * new * case["hkv"] * case["dh"]}
    W, M, seen, pairs = case["window"], case["meta"], 0, 0
    for a, t in zip(n, length):
        if a == 0:
            continue
        i = np.arange(t - a, t, dtype=np.int64)
        low = np.maximum(0, i - W) if W >= 0 else np.zeros_like(i)
        pairs += int((i + 1 - low + np.minimum(M, low)).sum())
        seen += int(t - low[0] + min(M, low[0]))
    return {"bytes": 2 * seen * row + 2 * new * case["hq"] * case["dh"] * es, "flops": 4 * case["dh"] * case["hq"] * pairs}
