"""Prompt attention at the edges of its tiles, shares and number ranges, against
the definition in 64 bits (tests/prefill_ref.py derives the tolerances)."""
import math

import pytest
import torch

import paged_gqa_decode_07_b200 as pgd
from tests.test_gpu_prefill import (bits, check_packed, check_paged, cu_of, make_pages, randn,
                                    run_packed, run_paged)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pgd.load_library()
    yield
    assert pgd.get_device_error() == 0


# --------------------------------------------------------------------------- #
# Warps whose lanes hold rows and no rows                                     #
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("ctas", [0, 5], ids=["whole", "cut"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 1), (6, 2), (11, 1), (13, 1)])
@pytest.mark.parametrize("d,dt", [(128, "bf16"), (256, "bf16"), (128, "e4m3")])
def test_every_count_of_rows_in_a_warp(d, dt, hq, hkv, ctas):
    """Last tiles with 1, 2, 3 ... rows: some lanes of a warp write, the others
    meet them again at the next 32 columns."""
    lens = list(range(1, 41))
    if dt == "bf16":
        check_packed(lens, hq, hkv, d, seed=300, num_ctas=ctas, tail=3)
    check_paged(lens, [n + 3 * i for i, n in enumerate(lens)], hq, hkv, d, 16, dt, seed=301,
                num_ctas=ctas, tail=3)


# --------------------------------------------------------------------------- #
# More shares than the work is long                                           #
# --------------------------------------------------------------------------- #
def nan_workspace(seqs, tokens, keys, hq, hkv, d, ctas):
    """A workspace in which a slot that nothing wrote shows."""
    need = pgd.prefill_workspace_bytes(seqs, tokens, keys, 0, hq, hkv, d, ctas)
    assert need % 4 == 0 and need > 0
    return torch.full((need // 4,), float("nan"), device="cuda")


@pytest.mark.parametrize("ctas", [600, 700, 1000, 1024])
@pytest.mark.parametrize("d,dt", [(128, "bf16"), (256, "bf16"), (128, "e4m3")])
def test_more_ctas_than_the_axis_is_long(d, dt, ctas):
    """A unit is its keys and a constant long: some CTAs get nothing, and their
    boundaries lie inside a unit that others cut."""
    for ctx in (130, 200, 257, 384, 516, 600, 640, 700):
        check_paged([1], [ctx], 4, 1, d, 16, dt, seed=310 + ctx, num_ctas=ctas,
                    workspace=nan_workspace(1, 1, ctx, 4, 1, d, ctas))
    check_paged([200, 0, 3], [200, 9, 20], 2, 1, d, 16, dt, seed=311, num_ctas=ctas,
                workspace=nan_workspace(3, 203, 200, 2, 1, d, ctas))
    if dt == "bf16":
        check_packed([200], 1, 1, d, seed=312, num_ctas=ctas,
                     workspace=nan_workspace(1, 200, 200, 1, 1, d, ctas))


# --------------------------------------------------------------------------- #
# Values that are not finite                                                  #
# --------------------------------------------------------------------------- #
def paged_case(ctx, q_lens, hq, hkv, d, bs, dt, seed):
    kc, vc, table, ks, vs = make_pages(ctx, hkv, d, bs, dt, seed)
    cu, cu_t = cu_of(q_lens)
    q = randn((cu[-1], hq, d), seed + 9)

    def run(v_cache, **kw):
        return run_paged(q, kc, v_cache, table, ctx, cu_t, hq, hkv, d, bs, 1 / math.sqrt(d), ks,
                         vs, max_context_len=max(ctx), **kw)

    def spoil(places):
        """V with the values of {(sequence, position, head, element): x}."""
        bad = vc.clone()
        for (s, t, h, e), x in places.items():
            bad[table[s, t // bs].long(), h, t % bs, e] = 0x7F if dt == "e4m3" else x
        return bad
    return run, vc, spoil, cu


def assert_only_there(got, clean, spoiled):
    """Bits as with a finite value, but for the outputs `spoiled` [T][Hq][D],
    which are not finite."""
    out, lse = got
    assert torch.equal(bits(lse), bits(clean[1]))
    assert torch.equal(bits(out)[~spoiled], bits(clean[0])[~spoiled])
    assert not bool(torch.isfinite(out[spoiled]).any())


@pytest.mark.parametrize("ctas", [0, 1], ids=["auto", "one"])
@pytest.mark.parametrize("d,dt", [(128, "bf16"), (256, "bf16"), (128, "e4m3")])
def test_a_newest_value_that_is_not_finite_behind_a_long_context(d, dt, ctas):
    """It reaches the newest rows alone, and takes no time that grows with the
    context: nothing gives up waiting, and the work behind it is done."""
    ctx, q_lens = [150001, 70, 90], [5, 70, 3]
    run, vc, spoil, cu = paged_case(ctx, q_lens, 4, 1, d, 64, dt, 400)
    clean = run(vc, num_ctas=ctas)
    got = run(spoil({(0, 149999, 0, 3): math.nan, (0, 149999, 0, d - 1): math.nan}),
              num_ctas=ctas)
    assert pgd.get_device_error() == 0
    spoiled = torch.zeros(clean[0].shape, dtype=torch.bool, device="cuda")
    spoiled[3:5, :, [3, d - 1]] = True           # positions 149999 and 150000
    assert_only_there(got, clean, spoiled)


@pytest.mark.parametrize("d,dt", [(128, "bf16"), (256, "bf16"), (128, "e4m3")])
@pytest.mark.parametrize("window", [0, 1, 77, 300])
def test_many_values_that_are_not_finite(d, dt, window):
    """Every row sees its own ones: behind the causal mask, at the window's
    edge, in every element of a row, in cut pieces; the same bits each time."""
    n, hq, hkv = 611, 2, 1
    run, vc, spoil, cu = paged_case([n, 9], [600, 1], hq, hkv, d, 32, dt, 410)
    g = torch.Generator().manual_seed(5)
    places = {}
    for x in (math.nan, math.inf, -math.inf):
        for t in torch.randint(0, n, (6,), generator=g).tolist():
            places[(0, t, 0, int(torch.randint(0, d, (1,), generator=g)))] = x
    places.update({(0, n - 1, 0, e): math.inf for e in range(d)})
    pos = torch.arange(n - 600, n, device="cuda")
    spoiled = torch.zeros((601, hq, d), dtype=torch.bool, device="cuda")
    for (_, t, _, e) in places:
        sees = (pos >= t) & ((pos < t + window) if window else (pos >= t))
        spoiled[:600, :, e] |= sees[:, None]
    for ctas in (1, 3, 20):
        clean = run(vc, window=window, num_ctas=ctas)
        v = spoil(places)
        first = run(v, window=window, num_ctas=ctas)
        assert_only_there(first, clean, spoiled)
        for _ in range(3):
            again = run(v, window=window, num_ctas=ctas)
            for a, b in zip(first, again):
                assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("d", [128, 256])
def test_infinities_keep_their_sign(d):
    """In tiles that only some rows see, packed."""
    n, hq = 300, 2
    q, k, v = (randn((n, h, d), 420 + i) for i, h in enumerate((hq, 1, 1)))
    cu, cu_t = cu_of([n])
    v[280, 0, 7], v[285, 0, 7], v[290, 0, 9], v[280, 0, d - 2] = math.inf, -math.inf, -math.inf, 1
    out, _ = run_packed(q, k, v, cu_t, hq, 1, d, 0.09)
    assert bool(torch.isfinite(out[:280]).all())
    assert bool((out[280:285, :, 7] == math.inf).all())
    assert bool(torch.isnan(out[285:, :, 7]).all())
    assert bool((out[290:, :, 9] == -math.inf).all()) and bool(torch.isfinite(out[:290, :, 9]).all())


@pytest.mark.parametrize("ctas", [0, 2])
def test_a_bad_value_that_only_the_second_query_tile_sees(ctas):
    """The first tile's rows keep the bits that they have without it, whichever
    warp comes first."""
    n, hq, d = 256, 1, 128                       # one unit: two tiles of 128 tokens
    q, k, v = (randn((n, h, d), 430 + i) for i, h in enumerate((hq, 1, 1)))
    cu_t = cu_of([n])[1]
    clean = run_packed(q, k, v, cu_t, hq, 1, d, 0.09, num_ctas=ctas)
    v[200, 0, 11] = math.nan
    spoiled = torch.zeros((n, hq, d), dtype=torch.bool, device="cuda")
    spoiled[200:, :, 11] = True
    for _ in range(30):
        got = run_packed(q, k, v, cu_t, hq, 1, d, 0.09, num_ctas=ctas)
        assert_only_there(got, clean, spoiled)


# --------------------------------------------------------------------------- #
# The largest windows                                                         #
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("window", [1 << 30, (1 << 31) - 2, (1 << 31) - 1])
@pytest.mark.parametrize("d,dt", [(128, "bf16"), (256, "bf16"), (128, "e4m3")])
def test_windows_longer_than_any_context(d, dt, window):
    """Rows at negative positions see nothing, and the others what they see
    without a window, whatever the window's size."""
    q_lens, ctx = [130, 300, 64, 1], [3, 120, 0, 700]
    for ctas in (0, 1, 3, 40):
        kw = dict(seed=320, num_ctas=ctas, gap=1, tail=2)
        want = check_paged(q_lens, ctx, 6, 2, d, 16, dt, **kw)
        got = check_paged(q_lens, ctx, 6, 2, d, 16, dt, window=window, **kw)
        for a, b in zip(want, got):
            assert torch.equal(bits(a), bits(b))
    if dt == "bf16":
        want = check_packed([400, 1], 6, 2, d, seed=321)
        got = check_packed([400, 1], 6, 2, d, seed=321, window=window)
        for a, b in zip(want, got):
            assert torch.equal(bits(a), bits(b))


# --------------------------------------------------------------------------- #
# Many small weights behind one large one                                     #
# --------------------------------------------------------------------------- #
def dominant_key(n, log2_weight, d, bs, dt):
    """A cache of n rows: the first weighs 1 and its value is zero, the others
    weigh 2^-log2_weight and their values are one.  Returns q, caches, table,
    softmax scale, scales."""
    nb = -(-n // bs)
    if dt == "e4m3":
        kc, vc = (torch.full((nb, 1, bs, d), x, device="cuda").to(torch.float8_e4m3fn)
                  for x in (0.0, 1.0))
        one = torch.ones(1, device="cuda")
        scales = (one, one)
    else:
        kc, vc = (torch.full((nb, 1, bs, d), x, dtype=torch.bfloat16, device="cuda")
                  for x in (0.0, 1.0))
        scales = (None, None)
    kc[..., 0] = -16.0
    kc[0, 0, 0, 0] = 0
    vc[0, 0, 0] = 0
    table = torch.arange(nb, dtype=torch.int32, device="cuda")[None, :].contiguous()
    q = torch.zeros((1, 4, d), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    if dt == "e4m3":
        kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
    return q, kc, vc, table, log2_weight * math.log(2) / 16, scales


@pytest.mark.parametrize("ctas", [1, 0], ids=["one", "auto"])
@pytest.mark.parametrize("e", [14.3, 18.3, 21.3, 24.3, 26.3, 28.3])
def test_small_weights_of_an_fp8_cache_are_not_lost(e, ctas):
    """o = n w / (1 + n w).  Each weight is off by half a step of f16 (2^-11) or
    2^-32 of the largest, the output by half a step, the two sums of n terms by
    2^-23 a term, and the scores by 2^-21 of their size."""
    n, bs = 262145, 64
    q, kc, vc, table, scale, (ks, vs) = dominant_key(n, e, 128, bs, "e4m3")
    out, _ = run_paged(q, kc, vc, table, [n], cu_of([1])[1], 4, 1, 128, bs, scale, ks, vs,
                       max_context_len=n, num_ctas=ctas)
    w = (n - 1) * 2.0 ** -e
    o = w / (1 + w)
    tol = o * (2.0 ** -8 + 2.0 ** -11 + 2 * n * 2.0 ** -23 + e * 2.0 ** -21) + n * 2.0 ** -32
    assert bool(((out.double() - o).abs() <= tol).all()), (float(out[0, 0, 0]), o, tol)


# --------------------------------------------------------------------------- #
# Pieces of no weight                                                         #
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("late", [False, True], ids=["before", "behind"])
@pytest.mark.parametrize("d,dt", [(128, "bf16"), (256, "bf16"), (128, "e4m3")])
def test_a_nan_in_a_piece_whose_weight_vanishes(d, dt, late):
    """Keys of one half score 300 more than the others: e^-300 is zero in fp32.
    A NaN that a row sees there shows, whether the work is cut or not."""
    n, bs = 2048, 16
    q, kc, vc, table, scale, (ks, vs) = dominant_key(n, 300 / math.log(2), d, bs, dt)
    zero, nan = (0, 0x7F) if dt == "e4m3" else (0.0, math.nan)
    half = slice(0, n // 2 // bs) if late else slice(n // 2 // bs, None)
    kc[half, ..., 0] = zero                      # the half that weighs
    at = n * 3 // 4 if late else n // 4
    vc[at // bs, 0, at % bs, 5] = nan
    for ctas in (1, 2, 5, 40):
        out, lse = run_paged(q, kc, vc, table, [n], cu_of([1])[1], 4, 1, d, bs, scale, ks, vs,
                             num_ctas=ctas)
        assert bool(torch.isnan(out[..., 5]).all()), f"{ctas} CTAs"
        keep = torch.arange(d, device="cuda") != 5
        assert bool(torch.isfinite(out[..., keep]).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("d,dt", [(128, "bf16"), (256, "bf16"), (128, "e4m3")])
@pytest.mark.parametrize("window", [0, 300])
def test_no_value_is_finite(d, dt, window):
    """Every element of every tile, with a window of which no tile is seen
    whole: the longest that a unit can take over them, in one CTA too."""
    ctx, q_lens = [3000, 200], [3000, 1]
    run, vc, _, cu = paged_case(ctx, q_lens, 2, 2, d, 16, dt, 440)
    bad = torch.full_like(vc, 0x7F if dt == "e4m3" else math.nan)
    for ctas in (0, 1):
        clean = run(vc, window=window, num_ctas=ctas)
        out, lse = run(bad, window=window, num_ctas=ctas)
        assert pgd.get_device_error() == 0
        assert bool(torch.isnan(out).all()) and torch.equal(bits(lse), bits(clean[1]))
