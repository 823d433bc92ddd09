"""Prompt attention over long contexts with inputs in which one key tile, or a
handful of keys, decides the output: a tile that is left out, read twice or
taken from the wrong place moves it by far more than the tolerance."""
import math

import pytest
import torch

import paged_gqa_decode_07_b200 as pgd
from tests import prefill_ref
from tests.test_gpu_prefill import cu_of, fp8, make_pages, randn, run_paged, run_packed

pytestmark = pytest.mark.gpu

KINDS = [(128, 16, "bf16"), (256, 64, "bf16"), (128, 32, "e4m3")]
IDS = [f"D{d}-bs{bs}-{dt}" for d, bs, dt in KINDS]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pgd.load_library()
    yield
    assert pgd.get_device_error() == 0


def check(out, lse, ref, n, d, dt, what):
    """prefill_ref's bound with this sequence's own key count, and a closer one
    for the log-sum-exp: the normaliser is two running sums of n / 2 terms, each
    addition off by 2^-24 of a sum that is at most the total, so n * 2^-25."""
    prefill_ref.assert_within(out, lse, ref, n, d, dt, what)
    _, r_lse, _, sab = ref
    tol = d * 2.0 ** -23 * sab + 2.0 ** -20 + n * 2.0 ** -25 + 2.0 ** -22 * r_lse.abs()
    err = (lse.double() - r_lse).abs()
    assert bool((err <= tol).all()), f"{what}: lse off by {float(err.max()):.3g}"


def rows_of(cache, table, pos, bs):
    """Index of a sequence's positions in a cache [blocks][heads][bs][D]."""
    return table[pos // bs].long(), slice(None), pos % bs


@pytest.mark.parametrize("ctas", [0, 1, 7])
@pytest.mark.parametrize("d,bs,dt", KINDS, ids=IDS)
def test_every_key_tile_counts_once(d, bs, dt, ctas):
    """V is zero but for 128 keys, swept over the context: the first, the last,
    those where shares begin, ones that straddle two tiles."""
    hq, hkv, ctx, q_lens = 2, 1, [40001, 20005], [2, 33]
    kc, vc, table, ks, vs = make_pages(ctx, hkv, d, bs, dt, 500)
    cu, cu_t = cu_of(q_lens)
    q = randn((cu[-1], hq, d), 501)
    scale = 1 / math.sqrt(d)
    empty = vc.clone()
    for s, n in enumerate(ctx):
        empty[rows_of(empty, table[s], torch.arange(n, device="cuda"), bs)] = 0
    starts = [[0, 127, n - 129, n // 128 * 128] for n in ctx]
    for s, n in enumerate(ctx):       # where a seventh of the axis ends (keys + 384 a unit)
        total = sum(ctx) + 2 * 384
        at = [total * c // 7 - (0 if s == 0 else ctx[0] + 384) - 384 for c in range(1, 7)]
        starts[s] += [x // 128 * 128 + o for x in at if 0 <= x < n - 256 for o in (-128, 0)
                      if x // 128 * 128 + o > 0]
    for i in range(max(len(x) for x in starts)):
        v = empty.clone()
        for s, n in enumerate(ctx):
            a = starts[s][i % len(starts[s])]
            where = rows_of(v, table[s], torch.arange(a, min(a + 128, n), device="cuda"), bs)
            v[where] = vc[where]
        out, lse = run_paged(q, kc, v, table, ctx, cu_t, hq, hkv, d, bs, scale, ks, vs,
                             max_context_len=max(ctx), num_ctas=ctas)
        for s, n in enumerate(ctx):
            r = slice(cu[s], cu[s + 1])
            ref = prefill_ref.paged(q[r], fp8(kc), fp8(v), table[s:s + 1], [n], [0, q_lens[s]], 0,
                                    scale, ks, vs)
            check(out[r], lse[r], ref, n, d, dt,
                  f"keys {starts[s][i % len(starts[s])]} of {n}, {ctas} CTAs")


def needles(n, bs, shares):
    """Positions at the edges of tiles, blocks and shares."""
    at = {0, 1, 127, 128, bs - 1, bs, n - 1, n // 2 // 128 * 128, n // 2 // 128 * 128 - 1,
          (n - 1) // 128 * 128, (n - 1) // bs * bs - 1}
    for c in range(1, shares):
        x = ((n + 384) * c // shares - 384) // 128 * 128
        at |= {x - 1, x}
    return sorted(t for t in at if 0 <= t < n)


@pytest.mark.parametrize("ctas", [0, 1, 3, 29])
@pytest.mark.parametrize("d,bs,dt", KINDS, ids=IDS)
def test_a_few_keys_decide_the_output(d, bs, dt, ctas):
    """Keys that score 14 above the others share nearly all of the weight."""
    hq, hkv, n, L = 2, 1, 65550, 5
    kc, vc, table, ks, vs = make_pages([n], hkv, d, bs, dt, 510)
    q = randn((1, 1, d), 511).expand(L, hq, d).contiguous()
    scale = 1 / math.sqrt(d)
    at = torch.tensor(needles(n, bs, max(ctas, 2)), device="cuda")
    key = q[0, 0].float() * (14 / (scale * float(q[0, 0].float().square().sum())))
    where = rows_of(kc, table[0], at, bs)
    if dt == "e4m3":
        kc[where] = (key / ks[0]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        kc[where] = key.to(torch.bfloat16)
    out, lse = run_paged(q, kc, vc, table, [n], cu_of([L])[1], hq, hkv, d, bs, scale, ks, vs,
                         max_context_len=n, num_ctas=ctas)
    ref = prefill_ref.paged(q, fp8(kc), fp8(vc), table, [n], [0, L], 0, scale, ks, vs)
    check(out, lse, ref, n, d, dt, f"{ctas} CTAs")
    # each of them is worth many times the tolerance
    assert float(ref[0][0].abs().max()) > 0.1 and len(at) < 80


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("window", [0, 2500])
def test_every_key_tile_of_a_long_prompt_counts_once(d, window):
    hq, hkv, lens = 2, 1, [6000, 1501]
    cu, cu_t = cu_of(lens)
    q, k, v = (randn((cu[-1], h, d), 520 + i) for i, h in enumerate((hq, hkv, hkv)))
    scale = 1 / math.sqrt(d)
    for a in (0, 127, 1280, 2944, 4095, 5872, 5999):
        x = torch.zeros_like(v)
        for s, n in enumerate(lens):
            b = cu[s] + a % n
            x[b:min(b + 128, cu[s + 1])] = v[b:min(b + 128, cu[s + 1])]
        out, lse = run_packed(q, k, x, cu_t, hq, hkv, d, scale, window=window,
                              max_seq_len=max(lens))
        ref = prefill_ref.packed(q, k, x, cu, window, scale)
        for s, n in enumerate(lens):
            r = slice(cu[s], cu[s + 1])
            check(out[r], lse[r], [y[r] for y in ref], n, d, "bf16", f"keys {a} of {n}")
