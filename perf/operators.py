"""Cases of the prompt-stage operators: what each computes, in plain torch and
through the library, on inputs a serving loop would hold.

The operators are
  prefill_attention        causal grouped-query attention over packed prompts
  paged_prefill_attention  the same for the newest tokens of sequences whose
                           K/V is in the paged cache (bf16 or FP8 E4M3)
  kv_quant_scales          the per-KV-head scales an FP8 cache is written with
  kv_gather                rows of a paged cache read back as bf16

`own` selects the library's kernels in run(); otherwise run() computes the
plain form (fp32, elementary operations, rounded once at the end).
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -40


# --------------------------------------------------------------------------- #
# Cases                                                                       #
# --------------------------------------------------------------------------- #
def listed():
    return [
        # four short prompts of one small batch: launch latency counts
        {"name": "prefill-tiny", "op": "prefill", "heads": 8, "kv_heads": 2, "dim": 128,
         "lens": "1,17,64,200", "window": 0, "fused": False},
        # prompts of a continuous batch, q/k/v cut from one fused projection
        {"name": "prefill-ragged", "op": "prefill", "heads": 32, "kv_heads": 8, "dim": 128,
         "lens": "33,2999,517,1,1280,764,2048,129", "window": 0, "fused": True},
        # one long prompt: the compute-bound end
        {"name": "prefill-long", "op": "prefill", "heads": 64, "kv_heads": 8, "dim": 128,
         "lens": "8192", "window": 0, "fused": False},
        # wide heads with a sliding window
        {"name": "prefill-wide-window", "op": "prefill", "heads": 32, "kv_heads": 2, "dim": 256,
         "lens": "4096,1500", "window": 1024, "fused": False},
        # one chunk of a long prompt whose prefix is cached: few query rows, a long key axis
        {"name": "chunk-long-prefix", "op": "paged", "heads": 32, "kv_heads": 8, "dim": 128,
         "block": 16, "fp8": False, "q_lens": "512", "ctx": "32768", "window": 0},
        # a mixed step: chunks of some prompts beside sequences that decode one token
        {"name": "mixed-step", "op": "paged", "heads": 32, "kv_heads": 8, "dim": 128,
         "block": 16, "fp8": False, "window": 0,
         "q_lens": "1,1,700,1,1,1,255,1,1,1,1,64,1,1,1,1,1,511,1,1,1,1,1,1",
         "ctx": "513,4096,700,2001,1777,3500,1255,640,2222,3967,1024,800,"
                "95,1600,2750,3003,1111,4095,620,1984,2500,3333,720,1455"},
        # the mixed step on an FP8 cache, with a long context among short ones
        {"name": "mixed-step-fp8", "op": "paged", "heads": 64, "kv_heads": 8, "dim": 128,
         "block": 16, "fp8": True, "window": 0,
         "q_lens": "300,1,17,1,128,1,1,250,1,5,1,33",
         "ctx": "8000,16,17,1023,2048,333,65,250,4097,1500,2900,700"},
        # draft tokens verified against long contexts, wide heads
        {"name": "verify-wide", "op": "paged", "heads": 32, "kv_heads": 2, "dim": 256,
         "block": 32, "fp8": False, "window": 0, "q_lens": "8,8,8,8,8,8,8,8,8,8,8,8,8,8,8,8",
         "ctx": "8192,3011,15999,905,12345,5120,2048,7777,16384,4001,640,9600,1300,11111,6006,82"},
        # scales from the rows of a short prompt, and from a whole calibration batch
        {"name": "scales-short", "op": "scales", "kv_heads": 8, "dim": 128, "tokens": 200},
        {"name": "scales-batch", "op": "scales", "kv_heads": 8, "dim": 128, "tokens": 65536},
        # a short bf16 prefix read back, and a large FP8 one
        {"name": "gather-short", "op": "gather", "kv_heads": 2, "dim": 256, "block": 32,
         "fp8": False, "tokens": 333, "blocks": 64},
        {"name": "gather-fp8", "op": "gather", "kv_heads": 8, "dim": 128, "block": 16,
         "fp8": True, "tokens": 65536, "blocks": 8192},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "paged", "paged", "paged", "scales", "gather"])
    if op == "scales":
        return {"op": op, "kv_heads": rng.choice([1, 2, 3, 4, 8, 16]),
                "dim": rng.choice([128, 256]), "tokens": _log_int(rng, 1, 16384)}
    if op == "gather":
        block, tokens = rng.choice([16, 32, 64]), _log_int(rng, 1, 16384)
        return {"op": op, "kv_heads": rng.choice([1, 2, 3, 4, 8]), "dim": rng.choice([128, 256]),
                "block": block, "fp8": rng.random() < 0.5, "tokens": tokens,
                "blocks": tokens // block + rng.randint(1, 200)}
    dim = rng.choice([128, 128, 256])
    fp8 = op == "paged" and dim == 128 and rng.random() < 0.5
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    kv_heads = rng.choice([1, 2, 4, 8])
    while group * kv_heads > 64:
        kv_heads //= 2
    heads = group * kv_heads
    budget = 1.0e9                       # padded scores of the plain form
    window = _log_int(rng, 16, 2048) if rng.random() < 0.25 else 0
    seqs = _log_int(rng, 1, 48)
    if op == "prefill":
        top = max(8, min(8192, int(math.sqrt(budget / (heads * seqs)))))
        lens = [_log_int(rng, 1, top) for _ in range(seqs)]
        return {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "lens": ",".join(map(str, lens)), "window": window, "fused": rng.random() < 0.5}
    top_ctx = _log_int(rng, 64, 65536 if seqs <= 4 else 16384)
    top_q = max(1, min(1024, int(budget / (heads * seqs * top_ctx))))
    q_lens, ctx = [], []
    for _ in range(seqs):
        q = 1 if rng.random() < 0.4 else _log_int(rng, 1, top_q)
        q_lens.append(q)
        ctx.append(max(q, _log_int(rng, 16, top_ctx)))
    return {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "block": rng.choice([16, 32, 64]), "fp8": fp8, "window": window,
            "q_lens": ",".join(map(str, q_lens)), "ctx": ",".join(map(str, ctx))}


def _ints(text):
    return np.array([int(x) for x in text.split(",")], np.int64)


def _pairs(q_lens, ctx, window):
    """Visible (query, key) pairs, and per sequence the first visible key."""
    total, first = 0, []
    for lq, n in zip(q_lens.tolist(), ctx.tolist()):
        hi = np.maximum(0, np.arange(n - lq + 1, n + 1, dtype=np.int64))
        lo = np.maximum(0, hi - window) if window else np.zeros_like(hi)
        total += int((hi - lo).sum())
        first.append(int(lo[0]))
    return total, np.array(first, np.int64)


def work(case):
    d = case["dim"]
    if case["op"] == "scales":
        n = case["tokens"] * case["kv_heads"] * d
        return {"bytes": 2 * n * 2 + 8 * case["kv_heads"], "flops": 2 * n}
    if case["op"] == "gather":
        n = case["tokens"] * case["kv_heads"] * d
        e = 1 if case["fp8"] else 2
        return {"bytes": 2 * n * (e + 2) + 8 * case["tokens"], "flops": 2 * n if case["fp8"] else 0}
    hq, hkv = case["heads"], case["kv_heads"]
    if case["op"] == "prefill":
        lens = _ints(case["lens"])
        pairs, _ = _pairs(lens, lens, case["window"])
        t = int(lens.sum())
        nbytes = 2 * t * hq * d * 2 + 2 * t * hkv * d * 2 + 4 * t * hq + 4 * (len(lens) + 1)
    else:
        q_lens, ctx = _ints(case["q_lens"]), _ints(case["ctx"])
        pairs, first = _pairs(q_lens, ctx, case["window"])
        t, e, bs = int(q_lens.sum()), 1 if case["fp8"] else 2, case["block"]
        blocks = int(((ctx + bs - 1) // bs - first // bs).sum())
        nbytes = (2 * t * hq * d * 2 + 2 * int((ctx - first).sum()) * hkv * d * e + 4 * t * hq
                  + 4 * blocks + 4 * (2 * len(ctx) + 1) + (8 * hkv if case["fp8"] else 0))
    return {"bytes": nbytes, "flops": 4 * pairs * hq * d}


# --------------------------------------------------------------------------- #
# Inputs                                                                      #
# --------------------------------------------------------------------------- #
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cu(lens):
    return torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device="cuda")


def _cache(g, blocks, hkv, bs, d, fp8):
    """A pool of N(0, 1) rows, and for FP8 the scales it was written with."""
    x = torch.randn((blocks, hkv, bs, d), generator=g, device="cuda")
    if not fp8:
        return x.to(torch.bfloat16), None
    scale = x.abs().amax(dim=(0, 2, 3)) / E4M3_MAX
    return (x / scale[None, :, None, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    d, hkv = case["dim"], case["kv_heads"]
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    if case["op"] == "scales":
        shape = (case["tokens"], hkv, d)
        # heads of different magnitudes, as trained projections have
        size = torch.exp2(2 * torch.randn((1, hkv, 1), generator=g, device="cuda"))
        s["k"] = (torch.randn(shape, generator=g, device="cuda") * size).to(torch.bfloat16)
        s["v"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        s["k_scale"] = torch.empty(hkv, device="cuda")
        s["v_scale"] = torch.empty(hkv, device="cuda")
        return s
    if case["op"] == "gather":
        nb, bs, n = case["blocks"], case["block"], case["tokens"]
        s["k"], s["k_scale"] = _cache(g, nb, hkv, bs, d, case["fp8"])
        s["v"], s["v_scale"] = _cache(g, nb, hkv, bs, d, case["fp8"])
        need = -(-n // bs)
        order = torch.randperm(nb, generator=g, device="cuda")[:need]
        at = torch.arange(n, device="cuda")
        s["slots"] = (order[at // bs] * bs + at % bs).to(torch.int64)
        s["k_out"] = torch.zeros((n, hkv, d), **bf16)
        s["v_out"] = torch.zeros((n, hkv, d), **bf16)
        return s
    hq = case["heads"]
    s["scale"] = 1.0 / math.sqrt(d)
    if case["op"] == "prefill":
        lens = _ints(case["lens"])
        t = int(lens.sum())
        if case["fused"]:
            qkv = torch.randn((t, hq + 2 * hkv, d), generator=g, device="cuda").to(torch.bfloat16)
            s["q"], s["k"], s["v"] = qkv.split([hq, hkv, hkv], dim=1)
        else:
            for name, h in (("q", hq), ("k", hkv), ("v", hkv)):
                s[name] = torch.randn((t, h, d), generator=g, device="cuda").to(torch.bfloat16)
        q_lens = ctx = lens
    else:
        q_lens, ctx, bs = _ints(case["q_lens"]), _ints(case["ctx"]), case["block"]
        t = int(q_lens.sum())
        s["q"] = torch.randn((t, hq, d), generator=g, device="cuda").to(torch.bfloat16)
        need = (ctx + bs - 1) // bs
        nb = int(need.sum()) + 1 + int(need.sum()) // 10
        s["k"], s["k_scale"] = _cache(g, nb, hkv, bs, d, case["fp8"])
        s["v"], s["v_scale"] = _cache(g, nb, hkv, bs, d, case["fp8"])
        order = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        start = torch.from_numpy(np.cumsum(need) - need).cuda()
        col = torch.arange(int(need.max()), device="cuda")
        at = torch.minimum(start[:, None] + col[None, :], torch.tensor(nb - 1, device="cuda"))
        s["table"] = order[at].contiguous()
        s["max_ctx"] = int(ctx.max())
    s["max_q"] = int(q_lens.max())
    s["cu"] = _cu(q_lens)
    s["ctx_lens"] = torch.from_numpy(ctx.astype(np.int32)).cuda()
    s["out"] = torch.zeros((t, hq, d), **bf16)
    s["lse"] = torch.zeros((t, hq), device="cuda")
    return s


# --------------------------------------------------------------------------- #
# One pass                                                                    #
# --------------------------------------------------------------------------- #
def _attend(q, k, v, q_pos, lens, window, scale):
    """Masked attention in fp32.  q [B][Lq][Hkv][g][D], k/v [B][Lk][Hkv][D],
    q_pos [B][Lq] the queries' positions, lens [B] the keys that exist."""
    scores = torch.matmul(q.permute(0, 2, 3, 1, 4).flatten(2, 3),
                          k.permute(0, 2, 3, 1)).mul_(scale)      # [B][Hkv][g*Lq][Lk]
    b, h, lk = scores.shape[0], scores.shape[1], scores.shape[3]
    lq, grp = q.shape[1], q.shape[3]
    key = torch.arange(lk, device=q.device)
    seen = (key <= q_pos[..., None]) & (key < lens[:, None, None])
    if window:
        seen &= key > q_pos[..., None] - window
    scores = scores.view(b, h, grp, lq, lk)
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where((key[None, :] < lens[:, None])[..., None, None], v, 0.0)
    o = torch.matmul(p.view(b, h, grp * lq, lk), v.permute(0, 2, 1, 3)).view(b, h, grp, lq, -1)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + total.log())[..., 0]
    return o.permute(0, 3, 1, 2, 4), lse.permute(0, 3, 1, 2)


def _packed(s, hkv):
    """Index of each (sequence, query) in the packed rows, padded."""
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    col = torch.arange(s["max_q"], device="cuda")
    live = col[None, :] < n[:, None]
    at = torch.where(live, cu[:-1, None] + col[None, :], 0)
    return at, live, n


def _plain_attention(s):
    hq, hkv, d = s["heads"], s["kv_heads"], s["dim"]
    at, live, n = _packed(s, hkv)
    q = s["q"].float().view(-1, hkv, hq // hkv, d)[at]
    ctx = s["ctx_lens"].long()
    if s["op"] == "prefill":
        k, v = s["k"].float()[at], s["v"].float()[at]
    else:
        k, v = s["k"].float(), s["v"].float()
        if s["fp8"]:
            k = k * s["k_scale"][None, :, None, None]
            v = v * s["v_scale"][None, :, None, None]
        table = s["table"].long()
        k = k[table].permute(0, 1, 3, 2, 4).flatten(1, 2)
        v = v[table].permute(0, 1, 3, 2, 4).flatten(1, 2)
    pos = (ctx - n)[:, None] + torch.arange(s["max_q"], device="cuda")[None, :]
    o, lse = _attend(q, k, v, pos, ctx, s["window"], s["scale"])
    out, out_lse = s["out"], s["lse"]
    out[at[live]] = o[live].flatten(1, 2).to(torch.bfloat16)
    out_lse[at[live]] = lse[live].flatten(1, 2)
    return out, out_lse


def _plain(s):
    if s["op"] == "scales":
        return tuple((x.float().abs().amax(dim=(0, 2)) / E4M3_MAX).clamp_min(MIN_SCALE)
                     for x in (s["k"], s["v"]))
    if s["op"] == "gather":
        blk, off = s["slots"] // s["block"], s["slots"] % s["block"]
        k, v = s["k"][blk, :, off].float(), s["v"][blk, :, off].float()
        if s["fp8"]:
            k, v = k * s["k_scale"][:, None], v * s["v_scale"][:, None]
        return k.to(torch.bfloat16), v.to(torch.bfloat16)
    return _plain_attention(s)


def run(s):
    if not own:
        return _plain(s)
    import paged_gqa_decode_07_b200 as pgd
    if s["op"] == "scales":
        return pgd.kv_quant_scales(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if s["op"] == "gather":
        return pgd.kv_gather(s["k"], s["v"], s["slots"], s["k_out"], s["v_out"],
                             k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["op"] == "prefill":
        out = pgd.prefill_attention(s["q"], s["k"], s["v"], s["cu"], s["heads"], s["kv_heads"],
                                    s["dim"], s["scale"], s["out"], window=s["window"],
                                    max_seq_len=s["max_q"], lse_out=s["lse"])
    else:
        out = pgd.paged_prefill_attention(
            s["q"], s["k"], s["v"], s["table"], s["ctx_lens"], s["cu"], s["heads"],
            s["kv_heads"], s["dim"], s["block"], s["scale"], s["out"], window=s["window"],
            max_q_len=s["max_q"], max_context_len=s["max_ctx"], k_scale=s["k_scale"],
            v_scale=s["v_scale"], lse_out=s["lse"])
    return out, s["lse"]


# --------------------------------------------------------------------------- #
# The definitions in 64 bits                                                  #
# --------------------------------------------------------------------------- #
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "scales":
        return tuple(torch.clamp(x.double().abs().amax(2).amax(0) / E4M3_MAX, min=MIN_SCALE)
                     for x in (s["k"], s["v"]))
    if case["op"] == "gather":
        got = []
        for cache, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
            rows = cache.transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"])
            rows = rows.view(torch.uint8)[s["slots"]].view(cache.dtype).double() \
                if case["fp8"] else rows[s["slots"]].double()
            got.append(rows * scale.double()[None, :, None] if case["fp8"] else rows)
        return tuple(got)
    hq, hkv, d, window = case["heads"], case["kv_heads"], case["dim"], case["window"]
    group = hq // hkv
    cu, ctx = s["cu"].tolist(), s["ctx_lens"].tolist()
    out = torch.zeros((cu[-1], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((cu[-1], hq), dtype=torch.float64, device="cuda")
    for b, n in enumerate(ctx):
        lo, hi = cu[b], cu[b + 1]
        if case["op"] == "prefill":
            k, v = s["k"][lo:hi].double(), s["v"][lo:hi].double()
        else:
            pages = s["table"][b, :-(-n // case["block"])].long()
            k, v = ((c[pages].double() * (1.0 if sc is None else sc.double().view(-1, 1, 1)))
                    .transpose(1, 2).reshape(-1, hkv, d)[:n]
                    for c, sc in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])))
        step = max(1, 200_000_000 // (8 * n * group))
        for r0 in range(lo, hi, step):
            r1 = min(hi, r0 + step)
            pos = torch.arange(r0, r1, device="cuda") - lo + n - (hi - lo)
            t = torch.arange(n, device="cuda")
            hide = t[None, :] > pos[:, None]
            if window:
                hide |= t[None, :] <= pos[:, None] - window
            for h in range(hkv):
                x = torch.einsum("rgd,td->grt", s["q"][r0:r1, h * group:(h + 1) * group].double(),
                                 k[:, h]) * s["scale"]
                x[:, hide] = -math.inf
                z = torch.logsumexp(x, -1)
                lse[r0:r1, h * group:(h + 1) * group] = z.T
                w = torch.exp(x - z[..., None])
                out[r0:r1, h * group:(h + 1) * group] = torch.matmul(w, v[:, h]).transpose(0, 1)
    return out, lse
