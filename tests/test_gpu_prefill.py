"""Prompt attention on the GPU (packed and paged) against the definition in 64
bits, element by element within the error derived in tests/prefill_ref.py."""
import math

import pytest
import torch

import paged_gqa_decode_07_b200 as pgd
from tests import prefill_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pgd.load_library()
    yield
    assert pgd.get_device_error() == 0


def randn(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def cu_of(lens, start=0):
    cu = [start]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu, torch.tensor(cu, dtype=torch.int32, device="cuda")


SENTINEL = -7.25


def run_packed(q, k, v, cu, hq, hkv, d, scale, **kw):
    out = torch.full((q.shape[0], hq, d), SENTINEL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], hq), SENTINEL, device="cuda")
    pgd.prefill_attention(q, k, v, cu, hq, hkv, d, scale, out, lse_out=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def check_packed(lens, hq, hkv, d, window=0, seed=0, scale=None, fused=False, gap=0, tail=0, **kw):
    cu, cu_t = cu_of(lens, gap)
    T = cu[-1] + tail
    scale = 1 / math.sqrt(d) if scale is None else scale
    if fused:
        q, k, v = randn((T, hq + 2 * hkv, d), seed).split([hq, hkv, hkv], dim=1)
    else:
        q, k, v = (randn((T, h, d), seed + i) for i, h in enumerate((hq, hkv, hkv)))
    if gap or tail:   # rows of no sequence must not be read
        for x in (q, k, v):
            x[:gap] = math.nan
            x[cu[-1]:] = math.nan
    out, lse = run_packed(q, k, v, cu_t, hq, hkv, d, scale, window=window, **kw)
    a, b = cu[0], cu[-1]
    ref = prefill_ref.packed(q, k, v, cu, window, scale)
    prefill_ref.assert_within(out[a:b], lse[a:b], [r[a:b] for r in ref], max(lens, default=0), d,
                              "bf16", f"lens {lens} {hq}/{hkv} D{d} W{window} {kw}")
    for x in (out, lse):
        assert bool((x[:a] == SENTINEL).all()) and bool((x[b:] == SENTINEL).all())
    return out, lse


LENS = [[1], [1, 17, 64, 200], [0, 5, 0, 0, 129, 1, 0], [127, 128, 129], [255, 256, 257, 33],
        [1000, 3], [513]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 2, 256)])
def test_lengths(lens, hq, hkv, d):
    check_packed(lens, hq, hkv, d)


HEADS = [(1, 1), (4, 4), (2, 1), (3, 1), (12, 3), (20, 4), (7, 1), (16, 2), (16, 1), (30, 2)]


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("hq,hkv", HEADS, ids=[f"{a}over{b}" for a, b in HEADS])
def test_head_layouts(hq, hkv, d):
    check_packed([70, 300, 1, 131], hq, hkv, d, seed=3)


@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 129, 400, 5000])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (6, 2, 256)])
def test_windows(window, hq, hkv, d):
    check_packed([700, 30, 1, 257], hq, hkv, d, window=window, seed=4)


@pytest.mark.parametrize("d", [128, 256])
def test_token_strides_and_rows_of_no_sequence(d):
    check_packed([100, 0, 77], 8, 2, d, fused=True, gap=3, tail=5)
    check_packed([300], 8, 4, d, fused=True, gap=1, tail=200)


def test_strides_larger_than_a_row_each_its_own():
    T, hq, hkv, d = 333, 8, 2, 128
    q = randn((T, hq + 1, d), 1)[:, :hq]
    k = randn((T, 3 * hkv, d), 2)[:, hkv:2 * hkv]
    v = randn((2 * T, hkv, d), 3)[::2]
    cu, cu_t = cu_of([200, 133])
    out, lse = run_packed(q, k, v, cu_t, hq, hkv, d, 0.1)
    prefill_ref.assert_within(out, lse, prefill_ref.packed(q, k, v, cu, 0, 0.1), 200, d, "bf16")


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-4, 2.0, 20.0])
def test_scales(scale):
    # large scales: one key dominates and references move often
    check_packed([400, 65], 8, 2, 128, scale=scale, seed=9)
    check_packed([300], 4, 2, 256, scale=scale, seed=10)


def test_growing_scores_move_the_reference_every_tile():
    """Keys whose scores rise along the sequence: each tile rescales."""
    T, hq, hkv, d = 1500, 4, 2, 128
    q, k, v = (randn((T, h, d), i) for i, h in enumerate((hq, hkv, hkv)))
    q = (q.abs() + 0.5)
    k = (k.abs() * torch.linspace(0.01, 3.0, T, device="cuda")[:, None, None]).to(torch.bfloat16)
    for sc in (1.0, -1.0):
        cu, cu_t = cu_of([T])
        out, lse = run_packed(q, k, v, cu_t, hq, hkv, d, sc)
        prefill_ref.assert_within(out, lse, prefill_ref.packed(q, k, v, cu, 0, sc), T, d, "bf16")


@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 64, 500])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 1, 256)])
def test_cut_work(ctas, hq, hkv, d):
    check_packed([700, 0, 1, 300], hq, hkv, d, num_ctas=ctas, gap=2, tail=3)
    check_packed([1100], hq, hkv, d, num_ctas=ctas, window=200)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("ctas", [1, 2])
def test_masked_keys_have_no_influence(bad, d, ctas):
    """A non-finite key or value reaches the rows that see it and no other."""
    T, hq, hkv, at, window = 300, 8, 2, 137, 90
    q, k, v = (randn((T, h, d), 20 + i) for i, h in enumerate((hq, hkv, hkv)))
    cu, cu_t = cu_of([T - 40, 40])
    ref = prefill_ref.packed(q, k, v, cu, window, 0.09)
    rows = torch.arange(T, device="cuda")
    sees = (rows >= at) & (rows < at + window) & (rows < T - 40)
    for which in ("k", "v"):
        kk, vv = k.clone(), v.clone()
        (kk if which == "k" else vv)[at, 1, 5] = bad
        out, lse = run_packed(q, kk, vv, cu_t, hq, hkv, d, 0.09, window=window, num_ctas=ctas)
        keep = [r[~sees] for r in ref]
        prefill_ref.assert_within(out[~sees], lse[~sees], keep, T, d, "bf16", which)
        other = [r[sees][:, :hq // 2] for r in ref]   # the heads of KV head 0
        prefill_ref.assert_within(out[sees][:, :hq // 2], lse[sees][:, :hq // 2], other, T, d,
                                  "bf16", which)
        if which == "v":
            hit = out[sees][:, hq // 2:]
            assert not bool(torch.isfinite(hit[..., 5]).any())
            rest = [r[sees][:, hq // 2:] for r in ref]
            el = torch.arange(d, device="cuda") != 5
            prefill_ref.assert_within(hit[..., el], None, [rest[0][..., el], rest[1],
                                      rest[2][..., el], rest[3]], T, d, "bf16", which)


@pytest.mark.parametrize("at", [0, 127, 128, 255, 299])
def test_a_later_value_that_is_not_finite(at):
    """The causal mask alone hides it: the diagonal tile's masked weights are
    zero, and zero times infinity must not reach the earlier rows."""
    T, hq, hkv, d = 300, 4, 1, 128
    q, k, v = (randn((T, h, d), 30 + i) for i, h in enumerate((hq, hkv, hkv)))
    cu, cu_t = cu_of([T])
    ref = prefill_ref.packed(q, k, v, cu, 0, 0.09)
    v[at, 0, 77] = math.inf
    out, lse = run_packed(q, k, v, cu_t, hq, hkv, d, 0.09)
    prefill_ref.assert_within(out[:at], lse[:at], [r[:at] for r in ref], T, d, "bf16")
    assert not bool(torch.isfinite(out[at:, :, 77]).any())


def test_queries_that_are_not_finite_stay_in_their_row():
    T, hq, hkv, d = 200, 8, 2, 128
    q, k, v = (randn((T, h, d), 40 + i) for i, h in enumerate((hq, hkv, hkv)))
    cu, cu_t = cu_of([T])
    ref = prefill_ref.packed(q, k, v, cu, 0, 0.09)
    q[50, 3, 0], q[120, 0, 9] = math.nan, math.inf
    out, lse = run_packed(q, k, v, cu_t, hq, hkv, d, 0.09)
    keep = torch.ones((T, hq), dtype=torch.bool, device="cuda")
    keep[50, 3] = keep[120, 0] = False
    prefill_ref.assert_within(out[keep], lse[keep], [r[keep] for r in ref], T, d, "bf16")
    assert bool(torch.isnan(out[50, 3]).all())


# --------------------------------------------------------------------------- #
# Paged                                                                       #
# --------------------------------------------------------------------------- #
def make_pages(ctx, hkv, d, bs, dt, seed, extra=3, width=0):
    """Caches whose unowned rows hold NaN, and a shuffled block table whose
    entries past a context are no block."""
    need = [-(-n // bs) for n in ctx]
    nb = sum(need) + extra
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    W = max(max(need, default=1), 1, width)
    table = torch.full((len(ctx), W), 1 << 30, dtype=torch.int32)
    owned = torch.zeros((nb, bs), dtype=torch.bool)
    at = 0
    for s, n in enumerate(ctx):
        table[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
        for j in range(need[s]):
            owned[table[s, j].long(), :min(bs, n - j * bs)] = True
    kf, vf = (randn((nb, hkv, bs, d), seed + i, torch.float32) for i in (1, 2))
    ks = vs = None
    if dt == "e4m3":
        ks, vs = ((x.abs().amax(dim=(0, 2, 3)) / 448.0) for x in (kf, vf))
        kc, vc = ((x / s[None, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
                  for x, s in ((kf, ks), (vf, vs)))
        for c in (kc, vc):
            c.transpose(1, 2)[~owned.cuda()] = 0x7F
    else:
        kc, vc = kf.to(torch.bfloat16), vf.to(torch.bfloat16)
        for c in (kc, vc):
            c.transpose(1, 2)[~owned.cuda()] = math.nan
    return kc, vc, table.cuda(), ks, vs


def fp8(x):
    return x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x


def run_paged(q, kc, vc, table, ctx, cu, hq, hkv, d, bs, scale, ks, vs, **kw):
    out = torch.full((q.shape[0], hq, d), SENTINEL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], hq), SENTINEL, device="cuda")
    pgd.paged_prefill_attention(q, kc, vc, table,
                                torch.tensor(ctx, dtype=torch.int32, device="cuda"), cu, hq, hkv,
                                d, bs, scale, out, lse_out=lse, k_scale=ks, v_scale=vs, **kw)
    torch.cuda.synchronize()
    return out, lse


def check_paged(q_lens, ctx, hq, hkv, d, bs, dt, window=0, seed=0, gap=0, tail=0, hints=True,
                scale=None, **kw):
    kc, vc, table, ks, vs = make_pages(ctx, hkv, d, bs, dt, seed)
    cu, cu_t = cu_of(q_lens, gap)
    q = randn((cu[-1] + tail, hq, d), seed + 9)
    scale = 1 / math.sqrt(d) if scale is None else scale
    if hints:
        kw.update(max_q_len=max(q_lens), max_context_len=max(ctx))
    out, lse = run_paged(q, kc, vc, table, ctx, cu_t, hq, hkv, d, bs, scale, ks, vs,
                         window=window, **kw)
    ref = prefill_ref.paged(q, fp8(kc), fp8(vc), table, ctx, cu, window, scale, ks, vs)
    a, b = cu[0], cu[-1]
    prefill_ref.assert_within(out[a:b], lse[a:b], [r[a:b] for r in ref], max(ctx), d, dt,
                              f"{q_lens} of {ctx} {hq}/{hkv} D{d} bs{bs} {dt} W{window} {kw}")
    for x in (out, lse):
        assert bool((x[:a] == SENTINEL).all()) and bool((x[b:] == SENTINEL).all())
    return out, lse


CACHES = [(128, 16, "bf16"), (128, 32, "bf16"), (128, 64, "bf16"), (256, 16, "bf16"),
          (256, 32, "bf16"), (256, 64, "bf16"), (128, 16, "e4m3"), (128, 32, "e4m3"),
          (128, 64, "e4m3")]


@pytest.mark.parametrize("d,bs,dt", CACHES, ids=[f"D{a}-bs{b}-{c}" for a, b, c in CACHES])
def test_paged_chunks(d, bs, dt):
    # chunks, whole prompts, single tokens, no tokens, contexts shorter than
    # the chunk (rows that see nothing), an empty context
    check_paged([1, 100, 17, 0, 64, 5, 3, 130, 2],
                [1, 333, 17, 40, 1029, 3, 0, 130, 16], 8, 2, d, bs, dt)


@pytest.mark.parametrize("hq,hkv", HEADS, ids=[f"{a}over{b}" for a, b in HEADS])
@pytest.mark.parametrize("d,dt", [(128, "bf16"), (256, "bf16"), (128, "e4m3")])
def test_paged_head_layouts(hq, hkv, d, dt):
    check_paged([1, 70, 33], [200, 71, 517], hq, hkv, d, 16, dt, seed=5)


@pytest.mark.parametrize("window", [1, 15, 128, 300])
@pytest.mark.parametrize("d,dt", [(128, "bf16"), (256, "bf16"), (128, "e4m3")])
def test_paged_windows(window, d, dt):
    check_paged([40, 1, 260], [700, 333, 260], 8, 2, d, 32, dt, window=window, seed=6)


@pytest.mark.parametrize("ctas", [1, 2, 5, 64, 500])
@pytest.mark.parametrize("d,dt", [(128, "bf16"), (256, "bf16"), (128, "e4m3")])
def test_paged_cut_work(ctas, d, dt):
    check_paged([3, 1, 65, 0], [1500, 16, 700, 9], 8, 2, d, 16, dt, seed=7, num_ctas=ctas,
                gap=1, tail=2)


@pytest.mark.parametrize("dt", ["bf16", "e4m3"])
def test_paged_without_hints_and_automatic_grid(dt):
    check_paged([30], [6000], 8, 1, 128, 16, dt, seed=8, hints=False)
    check_paged([30], [6000], 8, 1, 128, 16, dt, seed=8)


@pytest.mark.parametrize("power", [-20, 0, 17])
def test_fp8_query_magnitudes(power):
    """Query rows far outside f16's range, the softmax scale scaled back."""
    hq, hkv, d, bs = 8, 2, 128, 16
    ctx, q_lens = [500, 70], [60, 70]
    kc, vc, table, ks, vs = make_pages(ctx, hkv, d, bs, "e4m3", 50)
    cu, cu_t = cu_of(q_lens)
    q = (randn((130, hq, d), 51).float() * 2.0 ** power).to(torch.bfloat16)
    q[3] = 0
    scale = 2.0 ** -power / math.sqrt(d)
    out, lse = run_paged(q, kc, vc, table, ctx, cu_t, hq, hkv, d, bs, scale, ks, vs)
    ref = prefill_ref.paged(q, fp8(kc), fp8(vc), table, ctx, cu, 0, scale, ks, vs)
    prefill_ref.assert_within(out, lse, ref, 500, d, "e4m3")


@pytest.mark.parametrize("dt", ["bf16", "e4m3"])
def test_negative_and_zero_scales(dt):
    for sc in (0.0, -0.1):
        check_paged([50, 1], [300, 129], 4, 2, 128, 16, dt, seed=11, scale=sc)


@pytest.mark.parametrize("d,dt", [(128, "bf16"), (128, "e4m3")])
def test_paged_values_that_are_not_finite(d, dt):
    """In a chunk's own rows, behind the causal mask."""
    ctx, q_lens, bs = [400], [150], 16
    kc, vc, table, ks, vs = make_pages(ctx, 1, d, bs, dt, 60)
    cu, cu_t = cu_of(q_lens)
    q = randn((150, 4, d), 61)
    ref = prefill_ref.paged(q, fp8(kc), fp8(vc), table, ctx, cu, 0, 0.09, ks, vs)
    at = 333                                   # the row of query 333 - 250 = 83
    vc[table[0, at // bs].long(), 0, at % bs, 9] = 0x7F if dt == "e4m3" else math.nan
    out, lse = run_paged(q, kc, vc, table, ctx, cu_t, 4, 1, d, bs, 0.09, ks, vs)
    prefill_ref.assert_within(out[:83], lse[:83], [r[:83] for r in ref], 400, d, dt)
    assert bool(torch.isnan(out[83:, :, 9]).all())
    keep = torch.arange(d, device="cuda") != 9
    prefill_ref.assert_within(out[83:][..., keep], None,
                              [ref[0][83:][..., keep], ref[1][83:], ref[2][83:][..., keep],
                               ref[3][83:]], 400, d, dt)


# --------------------------------------------------------------------------- #
# As a serving loop uses them                                                 #
# --------------------------------------------------------------------------- #
def test_chunks_give_what_the_whole_prompt_gives():
    """A prompt in one packed call, and appended and attended chunk by chunk
    through the cache; then one decode step agrees with a chunk of one."""
    n, hq, hkv, d, bs = 900, 8, 2, 128, 16
    q, k, v = (randn((n, h, d), 70 + i) for i, h in enumerate((hq, hkv, hkv)))
    scale = 1 / math.sqrt(d)
    cu, cu_t = cu_of([n])
    whole, whole_lse = run_packed(q, k, v, cu_t, hq, hkv, d, scale)
    ref = prefill_ref.packed(q, k, v, cu, 0, scale)
    nb = 64
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(3))
    table = perm.to(torch.int32)[None, :].cuda()
    kc, vc = (torch.full((nb, hkv, bs, d), math.nan, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    pos = torch.arange(n)
    slots = (perm[pos // bs] * bs + pos % bs).cuda()
    at = 0
    for step in (400, 1, 130, 369):
        rows = slice(at, at + step)
        pgd.kv_append(k[rows], v[rows], slots[rows].contiguous(), kc, vc)
        out, lse = run_paged(q[rows], kc, vc, table, [at + step], cu_of([step])[1], hq, hkv, d, bs,
                             scale, None, None)
        prefill_ref.assert_within(out, lse, [r[rows] for r in ref], n, d, "bf16")
        at += step
    dec = pgd.paged_decode_attention(q[-1:].contiguous(), kc, vc, table,
                                     torch.tensor([n], dtype=torch.int32, device="cuda"), hq, hkv,
                                     d, bs, scale)
    prefill_ref.assert_within(dec, None, [r[-1:] for r in ref], n, d, "bf16")
    prefill_ref.assert_within(whole, whole_lse, ref, n, d, "bf16")


def test_fp8_cache_from_scales_to_decode():
    """Scales from the prompt, the quantising append, a prompt chunk over the
    cache, the cache read back, and a decode step: one FP8 serving path."""
    n, hq, hkv, d, bs = 333, 8, 2, 128, 16
    q, k, v = (randn((n, h, d), 80 + i) for i, h in enumerate((hq, hkv, hkv)))
    ks, vs = pgd.kv_quant_scales(k, v)
    nb = 32
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(4))
    pos = torch.arange(n)
    slots = (perm[pos // bs] * bs + pos % bs).cuda()
    kc, vc = (torch.full((nb, hkv, bs, d), 0x7F, dtype=torch.uint8, device="cuda")
              for _ in range(2))
    pgd.kv_append_quant(k, v, slots, kc, vc, ks, vs)
    kb, vb = pgd.kv_gather(kc, vc, slots, k_scale=ks, v_scale=vs)
    # E4M3 keeps 4 significant bits: half a step is 2^-4 of a normal value,
    # and 2^-10 scales of a subnormal one; then bf16's half step
    for x, y, s in ((k, kb, ks), (v, vb, vs)):
        tol = x.float().abs() * (2.0 ** -4 + 2.0 ** -8 * 1.0625) + 2.0 ** -10 * s[:, None]
        assert bool(((x.float() - y.float()).abs() <= tol * (1 + 2.0 ** -20)).all())
    table = perm.to(torch.int32)[None, :].cuda()
    scale = 1 / math.sqrt(d)
    cu, cu_t = cu_of([n])
    out, lse = run_paged(q, kc, vc, table, [n], cu_t, hq, hkv, d, bs, scale, ks, vs)
    ref = prefill_ref.paged(q, fp8(kc), fp8(vc), table, [n], cu, 0, scale, ks, vs)
    prefill_ref.assert_within(out, lse, ref, n, d, "e4m3")
    dec = pgd.paged_decode_attention(q[-1:].contiguous(), kc, vc, table,
                                     torch.tensor([n], dtype=torch.int32, device="cuda"), hq, hkv,
                                     d, bs, scale, k_scale=ks, v_scale=vs)
    prefill_ref.assert_within(dec, None, [r[-1:] for r in ref], n, d, "e4m3")


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def test_repeats_other_streams_prepared_calls_and_graphs_agree():
    lens, hq, hkv, d = [300, 1, 77], 8, 2, 128
    cu, cu_t = cu_of(lens)
    q, k, v = (randn((cu[-1], h, d), 90 + i) for i, h in enumerate((hq, hkv, hkv)))
    first, first_lse = run_packed(q, k, v, cu_t, hq, hkv, d, 0.09, num_ctas=2)
    again, again_lse = run_packed(q, k, v, cu_t, hq, hkv, d, 0.09, num_ctas=2)
    assert torch.equal(bits(first), bits(again)) and torch.equal(bits(first_lse), bits(again_lse))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = torch.zeros_like(first)
    pgd.prefill_attention(q, k, v, cu_t, hq, hkv, d, 0.09, other, num_ctas=2, stream=s)
    s.synchronize()
    assert torch.equal(bits(first), bits(other))
    out = torch.zeros_like(first)
    call = pgd.prefill_attention(q, k, v, cu_t, hq, hkv, d, 0.09, out, num_ctas=2, prepare=True)
    for _ in range(3):
        out.zero_()
        assert call() is out
        torch.cuda.synchronize()
        assert torch.equal(bits(first), bits(out))
    # two captured graphs, replayed in turn with new inputs
    graphs, outs = [], []
    for _ in range(2):
        o = torch.zeros_like(first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pgd.prefill_attention(q, k, v, cu_t, hq, hkv, d, 0.09, o, num_ctas=2)
        graphs.append(g)
        outs.append(o)
    q.copy_(randn(q.shape, 99))
    want, _ = run_packed(q, k, v, cu_t, hq, hkv, d, 0.09, num_ctas=2)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(bits(o), bits(want))


def test_two_streams_at_once():
    """Two calls in flight, each with its own workspace."""
    hq, hkv, d = 8, 2, 128
    lens = [900]
    cu, cu_t = cu_of(lens)
    data = [[randn((900, h, d), 100 + 5 * j + i) for i, h in enumerate((hq, hkv, hkv))]
            for j in range(2)]
    want = [run_packed(*x, cu_t, hq, hkv, d, 0.09, num_ctas=3)[0] for x in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(10):
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                pgd.prefill_attention(*data[j], cu_t, hq, hkv, d, 0.09, outs[j], num_ctas=3)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(bits(o), bits(w))


def test_block_permutation_does_not_matter():
    ctx, q_lens, hq, hkv, d, bs = [700, 90], [50, 90], 8, 2, 128, 16
    kc, vc, table, _, _ = make_pages(ctx, hkv, d, bs, "bf16", 110)
    cu, cu_t = cu_of(q_lens)
    q = randn((cu[-1], hq, d), 111)
    a, la = run_paged(q, kc, vc, table, ctx, cu_t, hq, hkv, d, bs, 0.09, None, None)
    nb = kc.shape[0]
    perm = torch.randperm(nb, device="cuda")
    kp, vp = torch.empty_like(kc), torch.empty_like(vc)
    kp[perm], vp[perm] = kc, vc
    tp = torch.where(table < nb, perm[table.clamp(max=nb - 1).long()].to(torch.int32), table)
    b, lb = run_paged(q, kp, vp, tp, ctx, cu_t, hq, hkv, d, bs, 0.09, None, None)
    assert torch.equal(bits(a), bits(b)) and torch.equal(bits(la), bits(lb))


def test_workspace_is_checked_and_used():
    lens, hq, hkv, d = [900], 8, 2, 128
    cu, cu_t = cu_of(lens)
    q, k, v = (randn((900, h, d), 120 + i) for i, h in enumerate((hq, hkv, hkv)))
    need = pgd.prefill_workspace_bytes(1, 900, 900, 0, hq, hkv, d, 3)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want, _ = run_packed(q, k, v, cu_t, hq, hkv, d, 0.09, num_ctas=3)
    got, _ = run_packed(q, k, v, cu_t, hq, hkv, d, 0.09, num_ctas=3, workspace=ws)
    assert torch.equal(bits(want), bits(got))
    with pytest.raises(pgd.PGDError) as e:
        run_packed(q, k, v, cu_t, hq, hkv, d, 0.09, num_ctas=3, workspace=ws[:need // 2])
    assert e.value.status == 6
    # without enough of it an automatic call cuts nothing
    out, lse = run_packed(q, k, v, cu_t, hq, hkv, d, 0.09, workspace=ws[:16])
    prefill_ref.assert_within(out, lse, prefill_ref.packed(q, k, v, cu, 0, 0.09), 900, d, "bf16")


def test_bad_lengths_and_blocks_are_flagged_not_read():
    """Out-of-range device inputs raise a flag; every access stays in bounds."""
    hq, hkv, d, bs = 8, 2, 128, 16
    q, k, v = (randn((64, h, d), 130 + i) for i, h in enumerate((hq, hkv, hkv)))
    for cu in ([0, 65], [-1, 30], [40, 20], [0, 1 << 30]):
        out = torch.full((64, hq, d), SENTINEL, dtype=torch.bfloat16, device="cuda")
        pgd.prefill_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), hq, hkv,
                              d, 0.09, out)
        assert pgd.get_device_error() == 2
        assert bool((out == SENTINEL).all())
    kc, vc, table, _, _ = make_pages([100], hkv, d, bs, "bf16", 131)
    cu_t = cu_of([20])[1]
    for bad in (-1, kc.shape[0], 1 << 30):
        t = table.clone()
        t[0, 2] = bad
        run_paged(q, kc, vc, t, [100], cu_t, hq, hkv, d, bs, 0.09, None, None)
        assert pgd.get_device_error() == 1
    for n in (-1, table.shape[1] * bs + 1):
        run_paged(q, kc, vc, table, [n], cu_t, hq, hkv, d, bs, 0.09, None, None)
        assert pgd.get_device_error() & 2


@pytest.mark.parametrize("d", [128, 256])
def test_many_sequences(d):
    """More sequences than a warp has lanes, most of them short or empty."""
    g = torch.Generator().manual_seed(1)
    lens = [int(x) for x in torch.randint(0, 40, (300,), generator=g)]
    lens[::7] = [0] * len(lens[::7])
    lens[150] = 700
    check_packed(lens, 4, 2, d, seed=140)


def test_long_context_rows():
    """Single tokens and a chunk over a context past many tiles."""
    check_paged([1, 33], [40000, 20001], 8, 2, 128, 64, "bf16", seed=150)
    check_paged([1, 33], [40000, 20001], 8, 2, 128, 64, "e4m3", seed=151)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 1, 256)])
def test_longer_prompts(hq, hkv, d):
    check_packed([2500, 1200], hq, hkv, d, seed=160, fused=True)
    check_packed([3333], hq, hkv, d, seed=161, window=700)


def test_outputs_that_start_on_16_bytes():
    """32-byte stores need more: such an output takes 16-byte ones."""
    T, hq, hkv = 150, 8, 2
    for d in (128, 256):
        q, k, v = (randn((T, h, d), 170 + i) for i, h in enumerate((hq, hkv, hkv)))
        cu, cu_t = cu_of([100, 50])
        base = torch.full((T * hq * d + 16,), SENTINEL, dtype=torch.bfloat16, device="cuda")
        out = base[8:8 + T * hq * d].view(T, hq, d)
        assert out.data_ptr() % 32 == 16
        for ctas in (0, 5):
            pgd.prefill_attention(q, k, v, cu_t, hq, hkv, d, 0.09, out, num_ctas=ctas)
            prefill_ref.assert_within(out, None, prefill_ref.packed(q, k, v, cu, 0, 0.09), 100, d,
                                      "bf16", f"{ctas} CTAs")
            assert bool((base[:8] == SENTINEL).all()) and bool((base[-8:] == SENTINEL).all())
            out.fill_(0)


@pytest.mark.parametrize("kw", [{"max_seq_len": 90}, {}, {"num_ctas": 1}, {"num_ctas": 97}],
                         ids=["dealt", "cut", "one", "97"])
@pytest.mark.parametrize("d", [128, 256])
def test_more_sequences_than_a_cta_has_threads(d, kw):
    g = torch.Generator().manual_seed(2)
    lens = [int(x) for x in torch.randint(0, 7, (1300,), generator=g)]
    lens[0] = lens[33] = lens[600] = lens[-1] = 0
    lens[32], lens[511], lens[512], lens[1298] = 90, 40, 33, 77
    check_packed(lens, 4, 2, d, seed=180, **kw)
    check_packed([0] * 700 + [5], 2, 1, d, seed=181, **kw)
    check_packed([0] * 700, 2, 1, d, seed=182, tail=2, **kw)


@pytest.mark.parametrize("dt", ["bf16", "e4m3"])
def test_dealt_and_cut_work_agree_with_the_definition_in_pages(dt):
    """Many short contexts: whole units dealt in turn (hints), or cut."""
    g = torch.Generator().manual_seed(3)
    ctx = [int(x) for x in torch.randint(1, 400, (60,), generator=g)]
    q_lens = [min(n, int(x)) for n, x in zip(ctx, torch.randint(0, 30, (60,), generator=g))]
    check_paged(q_lens, ctx, 8, 2, 128, 16, dt, seed=190)
    check_paged(q_lens, ctx, 8, 2, 128, 16, dt, seed=190, num_ctas=33)


def test_sequences_that_share_blocks():
    """Two sequences over one prefix, and the same block twice in a table."""
    hq, hkv, d, bs = 8, 2, 128, 16
    kc, vc, table, _, _ = make_pages([200], hkv, d, bs, "bf16", 200)
    table = torch.cat([table, table])
    table[1, 3] = table[1, 2]
    cu, cu_t = cu_of([40, 25])
    q = randn((65, hq, d), 201)
    ctx = [200, 180]
    out, lse = run_paged(q, kc, vc, table, ctx, cu_t, hq, hkv, d, bs, 0.09, None, None)
    ref = prefill_ref.paged(q, kc, vc, table, ctx, cu, 0, 0.09)
    prefill_ref.assert_within(out, lse, ref, 200, d, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "e4m3"])
def test_blocks_past_32_bit_offsets(dt):
    """A pool whose last blocks start past 2^32 bytes."""
    hq, hkv, d, bs = 4, 2, 128, 64
    nb = 140000 if dt == "bf16" else 270000
    shape, kind = (nb, hkv, bs, d), torch.bfloat16 if dt == "bf16" else torch.uint8
    small = make_pages([300], hkv, d, bs, dt, 210, extra=0)
    kc, vc = (torch.empty(shape, dtype=kind, device="cuda") for _ in range(2))
    need = small[0].shape[0]
    assert (nb - need) * hkv * bs * d * kc.element_size() > 1 << 32
    kc[nb - need:], vc[nb - need:] = small[0], small[1]
    table = torch.where(small[2] < need, small[2] + (nb - need), small[2])
    cu, cu_t = cu_of([70])
    q = randn((70, hq, d), 211)
    out, lse = run_paged(q, kc, vc, table, [300], cu_t, hq, hkv, d, bs, 0.09, small[3], small[4])
    ref = prefill_ref.paged(q, fp8(small[0]), fp8(small[1]), small[2], [300], cu, 0, 0.09, small[3],
                            small[4])
    prefill_ref.assert_within(out, lse, ref, 300, d, dt)
    # the same rows read back
    pos = torch.arange(300, device="cuda")
    slots = table[0, pos // bs].long() * bs + pos % bs
    ko, _ = pgd.kv_gather(kc, vc, slots, k_scale=small[3], v_scale=small[4])
    want = prefill_ref.pages(fp8(small[0]), small[2][0], 300, small[3])
    assert bool(((ko.double() - want).abs() <= want.abs() * 2.0 ** -8).all())


def test_scores_that_overflow_stay_in_their_rows():
    """A finite query and key whose product is +inf: that row is not finite,
    the others are as if the key were any other."""
    T, hq, hkv, d = 300, 4, 1, 128
    q, k, v = (randn((T, h, d), 220 + i) for i, h in enumerate((hq, hkv, hkv)))
    k[40, 0, :], q[200, 1, :] = 0, 0
    k[40, 0, 7], q[200, 1, 7] = 1e38, 1e38
    q[:, :, 7][torch.arange(T, device="cuda") != 200] = 0
    q[200, [0, 2, 3], 7] = 0
    ref = prefill_ref.packed(q, k, v, [0, T], 0, 0.09)
    cu, cu_t = cu_of([T])
    for ctas in (0, 3):
        out, lse = run_packed(q, k, v, cu_t, hq, hkv, d, 0.09, num_ctas=ctas)
        keep = torch.ones((T, hq), dtype=torch.bool, device="cuda")
        keep[200, 1] = False
        prefill_ref.assert_within(out[keep], lse[keep], [r[keep] for r in ref], T, d, "bf16")
        assert not bool(torch.isfinite(out[200, 1]).any())


def test_contexts_of_sequences_without_rows_are_not_looked_at():
    """A padded batch: no query rows, any context length."""
    kc, vc, table, _, _ = make_pages([60, 60, 60], 2, 128, 16, "bf16", 230)
    cu, cu_t = cu_of([20, 0, 0])
    q = randn((20, 4, 128), 231)
    for kw in ({}, {"max_context_len": 64}):
        out, lse = run_paged(q, kc, vc, table, [60, -5, 1 << 30], cu_t, 4, 2, 128, 16, 0.09, None,
                             None, **kw)
        assert pgd.get_device_error() == 0
        ref = prefill_ref.paged(q, kc, vc, table, [60, 0, 0], cu, 0, 0.09)
        prefill_ref.assert_within(out, lse, ref, 60, 128, "bf16")


def test_a_scale_of_zero_weighs_large_scores_alike():
    q, k, v = (randn((140, h, 128), 240 + i) for i, h in enumerate((4, 2, 2)))
    q, k = q * 1e15, k * 1e15          # scores of up to 1e32
    cu, cu_t = cu_of([140])
    out, lse = run_packed(q, k, v, cu_t, 4, 2, 128, 0.0)
    ref = prefill_ref.packed(q, k, v, cu, 0, 0.0)
    prefill_ref.assert_within(out, lse, ref, 140, 128, "bf16")


@pytest.mark.parametrize("ctas", [0, 7])
@pytest.mark.parametrize("dt", ["bf16", "e4m3"])
def test_a_captured_call_follows_new_lengths(ctas, dt):
    """A serving loop captures one step and replays it as sequences grow,
    begin, end and change their share of the rows."""
    hq, hkv, d, bs = 8, 2, 128, 16
    full = [1700, 300, 1500, 40]
    kc, vc, table, ks, vs = make_pages(full, hkv, d, bs, dt, 190)
    T = 96
    q = randn((T, hq, d), 191)
    scale = 1 / math.sqrt(d)
    cl = torch.tensor(full, dtype=torch.int32, device="cuda")
    cu_t = torch.tensor([0, 40, 41, 90, 96], dtype=torch.int32, device="cuda")
    out = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((T, hq), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pgd.paged_prefill_attention(q, kc, vc, table, cl, cu_t, hq, hkv, d, bs, scale, out,
                                    lse_out=lse, k_scale=ks, v_scale=vs, max_context_len=1700,
                                    num_ctas=ctas)
    for ctx, cu in ((full, [0, 40, 41, 90, 96]), ([1, 300, 0, 7], [0, 1, 90, 90, 94]),
                    ([1699, 0, 1281, 40], [0, 0, 0, 95, 96]), ([0, 0, 0, 0], [0, 0, 0, 0, 0])):
        cl.copy_(torch.tensor(ctx, dtype=torch.int32))
        cu_t.copy_(torch.tensor(cu, dtype=torch.int32))
        out.fill_(SENTINEL)
        lse.fill_(SENTINEL)
        g.replay()
        torch.cuda.synchronize()
        # contexts shorter than the pages: what lies behind them has no influence
        ref = prefill_ref.paged(q, fp8(kc), fp8(vc), table, ctx, cu, 0, scale, ks, vs)
        a, b = cu[0], cu[-1]
        if b > a:
            prefill_ref.assert_within(out[a:b], lse[a:b], [r[a:b] for r in ref], max(ctx), d, dt,
                                      f"{ctx} {cu}")
        for x in (out, lse):
            assert bool((x[b:] == SENTINEL).all())


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n", [1279, 1280, 1281])
def test_lengths_around_where_work_is_cut(n, d):
    assert (pgd.prefill_workspace_bytes(1, n, n, 0, 4, 2, d) > 0) == (n >= 1280)
    check_packed([n], 4, 2, d, seed=n)
    check_paged([3, 0], [n, 0], 4, 2, d, 16, "bf16", seed=n)
