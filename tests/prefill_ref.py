"""Prompt attention in 64 bits from the definition, and the error each element
of a kernel's output may have.

A rounding is off by at most half a step relative to the value: 2^-8 for
bf16, 2^-11 for f16, 2^-24 for fp32.  For one output element
o = sum_t w_t v_t (sum_t w_t = 1) with A = sum_t w_t |v_t|:

  * the weights enter the product rounded to bf16 or f16:   u_p * A
  * the output is rounded to bf16:                          2^-8 * |o|
  * scores: a dot product of D terms in fp32 is off by at most
    D * 2^-23 * sum |q||k| (each partial sum may be truncated), times the
    scale; a score off by e moves a weight by a factor e^(+-e), numerator and
    normaliser alike:                                       2 * e * A
  * exponentials (2^-21 each, numerator and normaliser), the normaliser's sum
    of n terms and the product's sum of n terms (2^-23 each):
                                                 (2^-20 + 2 n 2^-23) * A

A rounded weight also moves no normaliser (it sums the unrounded ones).  The
log-sum-exp is off by e + 2^-20 + n 2^-23 and the rounding of a value of its
size."""
import math

import torch

U_P = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -11}


def attend(q, k, v, pos, window, scale):
    """q [L][Hq][D], k / v [n][Hkv][D] float64, pos [L] the rows' positions.
    Returns out [L][Hq][D], lse [L][Hq], A and the score bound s [L][Hq]."""
    L, hq, d = q.shape
    n, hkv, _ = k.shape
    g = hq // hkv
    out = torch.zeros((L, hq, d), dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    lse = torch.full((L, hq), -math.inf, dtype=torch.float64, device=q.device)
    sab = torch.zeros((L, hq), dtype=torch.float64, device=q.device)
    t = torch.arange(n, device=q.device)
    seen = t[None, :] <= pos[:, None]
    if window:
        seen &= t[None, :] > pos[:, None] - window
    live = seen.any(1)
    if n == 0 or not bool(live.any()):
        return out, lse, mag, sab
    for h in range(hq):
        x = (q[:, h] @ k[:, h // g].T) * scale
        x = torch.where(seen, x, torch.tensor(-math.inf, dtype=torch.float64, device=q.device))
        m = x.amax(1, keepdim=True)
        m = torch.where(live[:, None], m, torch.zeros_like(m))
        e = torch.where(seen, torch.exp(x - m), torch.zeros_like(x))
        z = e.sum(1, keepdim=True)
        w = torch.where(live[:, None], e / z, torch.zeros_like(e))
        out[:, h] = w @ v[:, h // g]
        mag[:, h] = w @ v[:, h // g].abs()
        lse[:, h] = torch.where(live, m[:, 0] + z[:, 0].log(), lse[:, h])
        sa = (q[:, h].abs() @ k[:, h // g].abs().T) * abs(scale)
        sab[:, h] = torch.where(seen, sa, torch.zeros_like(sa)).amax(1)
    return out, lse, mag, sab


def packed(q, k, v, cu, window, scale):
    """attend() over packed prompts; rows of no sequence stay zero / -inf."""
    T, hq, _ = q.shape
    res = [torch.zeros(q.shape, dtype=torch.float64, device=q.device),
           torch.full((T, hq), -math.inf, dtype=torch.float64, device=q.device),
           torch.zeros(q.shape, dtype=torch.float64, device=q.device),
           torch.zeros((T, hq), dtype=torch.float64, device=q.device)]
    q, k, v = q.double(), k.double(), v.double()
    for a, b in zip(cu[:-1], cu[1:]):
        got = attend(q[a:b], k[a:b], v[a:b], torch.arange(b - a, device=q.device), window, scale)
        for r, x in zip(res, got):
            r[a:b] = x
    return res


def pages(cache, table, n, scale=None):
    """The first n rows [n][Hkv][D] (float64) of a sequence in a paged cache."""
    nb, hkv, bs, d = cache.shape
    need = -(-n // bs)
    x = cache[table[:need].long()].double()
    if scale is not None:
        x = x * scale.double()[None, :, None, None]
    return x.transpose(1, 2).reshape(need * bs, hkv, d)[:n]


def paged(q, k_cache, v_cache, table, ctx, cu, window, scale, k_scale=None, v_scale=None):
    T, hq, _ = q.shape
    res = [torch.zeros(q.shape, dtype=torch.float64, device=q.device),
           torch.full((T, hq), -math.inf, dtype=torch.float64, device=q.device),
           torch.zeros(q.shape, dtype=torch.float64, device=q.device),
           torch.zeros((T, hq), dtype=torch.float64, device=q.device)]
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        n = int(ctx[s])
        k = pages(k_cache, table[s], n, k_scale)
        v = pages(v_cache, table[s], n, v_scale)
        pos = torch.arange(n - (b - a), n, device=q.device)
        got = attend(q[a:b].double(), k, v, pos, window, scale)
        for r, x in zip(res, got):
            r[a:b] = x
    return res


def assert_within(out, lse, ref, n_keys, dim, kv_dtype, what=""):
    """Every element within the error derived above."""
    r_out, r_lse, mag, sab = ref
    e = (dim * 2.0 ** -23 * sab)[..., None]
    tol = (U_P[kv_dtype] * mag + 2.0 ** -8 * r_out.abs()
           + (2 * e + 2.0 ** -20 + 2 * n_keys * 2.0 ** -23) * mag + 1e-30)
    err = (out.double() - r_out).abs()
    bad = ~(err <= tol)
    if bool(bad.any()):
        at = [tuple(int(i) for i in x) for x in bad.nonzero()[:4]]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outputs are off: "
                             + "; ".join(f"{i} got {float(out[i]):.6g} want "
                                         f"{float(r_out[i]):.6g} +- {float(tol[i]):.2g}"
                                         for i in at))
    if lse is not None:
        dead = torch.isneginf(r_lse)
        assert torch.equal(torch.isneginf(lse), dead), f"{what}: rows that see nothing"
        assert bool((out[dead] == 0).all()), f"{what}: rows that see nothing give zero"
        tl = e[..., 0] + 2.0 ** -20 + n_keys * 2.0 ** -23 + 2.0 ** -22 * r_lse.abs()
        el = (lse.double() - r_lse).abs()
        ok = (el <= tl) | dead
        assert bool(ok.all()), (f"{what}: lse off by {float(el[~dead].max()):.3g}, allowed "
                                f"{float(tl[~ok].min()):.3g}")
