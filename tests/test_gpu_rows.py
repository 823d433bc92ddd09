"""FP8 scales from K/V rows and cached rows read back, bit for bit against
their definitions."""
import math

import pytest
import torch

import paged_gqa_decode_07_b200 as pgd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pgd.load_library()
    yield
    assert pgd.get_device_error() == 0


def randn(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def want_scale(x):
    """The quotient in 64 bits rounded to fp32: both operands are exact there
    and the 53-bit quotient of an 8-bit by a 3-bit significand rounds as the
    exact one does."""
    a = x.double().abs()
    a = torch.where(torch.isfinite(a), a, torch.zeros_like(a))
    m = a.amax(dim=(0, 2)) if x.shape[0] else torch.zeros(x.shape[1], dtype=torch.float64,
                                                          device=x.device)
    return (m / 448).float().clamp_min(2.0 ** -40)


@pytest.mark.parametrize("n", [0, 1, 2, 7, 200, 256, 257, 5000])
@pytest.mark.parametrize("hkv,d", [(1, 128), (2, 128), (3, 128), (8, 128), (1, 256), (5, 256),
                                   (8, 256), (40, 128), (33, 256)])
def test_scales(n, hkv, d):
    k, v = randn((n, hkv, d), n + 1), randn((n, hkv, d), n + 2) * 3
    ks, vs = pgd.kv_quant_scales(k, v)
    assert torch.equal(ks, want_scale(k)) and torch.equal(vs, want_scale(v))


def test_every_element_counts():
    """The maximum alone, at each corner of a batch, with either sign."""
    n, hkv, d = 77, 3, 128
    for i, (t, h, e) in enumerate([(0, 0, 0), (76, 2, 127), (40, 1, 64), (76, 0, 0), (0, 2, 1)]):
        k = randn((n, hkv, d), 5)
        k[t, h, e] = -100.0 if i % 2 else 100.0
        ks, vs = pgd.kv_quant_scales(k, k)
        assert torch.equal(ks, want_scale(k)) and torch.equal(ks, vs)
        assert float(ks[h]) == float(torch.tensor(100.0) / 448)


def test_zeros_infinities_nan_and_subnormals():
    k = torch.zeros((9, 4, 128), dtype=torch.bfloat16, device="cuda")
    k[3, 1, 5] = math.inf
    k[4, 1, 6] = -2.0
    k[5, 2, 7] = math.nan
    k[6, 3, 8] = 1e-40
    ks, vs = pgd.kv_quant_scales(k, -k)
    floor = 2.0 ** -40
    assert ks.tolist() == [floor, float(torch.tensor(2.0) / 448), floor, floor]
    assert torch.equal(ks, vs)
    big = torch.full((2, 1, 128), 3.3895313892515355e38, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(pgd.kv_quant_scales(big, big)[0], want_scale(big))


def test_accumulate_raises_scales():
    a, b = randn((60, 4, 128), 1), randn((60, 4, 128), 2)
    b[:, 1] *= 9
    a[:, 2] *= 9
    ks, vs = pgd.kv_quant_scales(a, b)
    pgd.kv_quant_scales(b, a, ks, vs, accumulate=True)
    both = want_scale(torch.cat([a, b]))
    assert torch.equal(ks, both) and torch.equal(vs, both)
    pgd.kv_quant_scales(a[:0], b[:0], ks, vs, accumulate=True)
    assert torch.equal(ks, both)
    with pytest.raises(ValueError):
        pgd.kv_quant_scales(a, b, accumulate=True)


def pool(nb, hkv, bs, d, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if dt == "bf16":   # every bit pattern, NaN payloads too
        return torch.randint(-32768, 32768, (nb, hkv, bs, d), generator=g,
                             device="cuda").to(torch.int16).view(torch.bfloat16)
    return torch.randint(0, 256, (nb, hkv, bs, d), generator=g, device="cuda").to(torch.uint8)


@pytest.mark.parametrize("n", [1, 5, 300])
@pytest.mark.parametrize("hkv,d,bs,dt", [
    (2, 128, 16, "bf16"), (8, 128, 32, "bf16"), (3, 256, 64, "bf16"), (1, 256, 16, "bf16"),
    (2, 128, 16, "e4m3"), (8, 128, 64, "e4m3"), (3, 256, 32, "e4m3"), (1, 128, 16, "e4m3")])
def test_gather(n, hkv, d, bs, dt):
    nb = 37
    k, v = pool(nb, hkv, bs, d, dt, 1), pool(nb, hkv, bs, d, dt, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    slots = torch.randint(-3, nb * bs, (n,), generator=g, device="cuda")   # repeats and padding
    slots[0], slots[-1] = nb * bs - 1, 0
    ks = torch.exp2(torch.randn(hkv, generator=g, device="cuda") * 4)
    vs = torch.exp2(torch.randn(hkv, generator=g, device="cuda") * 4)
    ko, vo = (torch.full((n, hkv, d), -7.25, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    pgd.kv_gather(k, v, slots, ko, vo, k_scale=ks, v_scale=vs)
    on = slots >= 0
    at = slots.clamp(min=0)
    for out, cache, sc in ((ko, k, ks), (vo, v, vs)):
        rows = cache.transpose(1, 2).reshape(nb * bs, hkv, d)[at]
        if dt == "e4m3":
            rows = (rows.view(torch.float8_e4m3fn).float() * sc[:, None]).to(torch.bfloat16)
            same = (out == rows) | (torch.isnan(out) & torch.isnan(rows))
        else:
            same = out.view(torch.int16) == rows.view(torch.int16)
        assert bool(same[on].all())
        assert bool((out[~on] == -7.25).all())


def test_gather_flags_slots_past_the_pool():
    k, v = pool(4, 2, 16, 128, "bf16", 1), pool(4, 2, 16, 128, "bf16", 2)
    ko, vo = (torch.full((3, 2, 128), -7.25, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    pgd.kv_gather(k, v, torch.tensor([64, 3, 1 << 40], device="cuda"), ko, vo)
    assert pgd.get_device_error() == 4
    assert bool((ko[0] == -7.25).all()) and bool((vo[2] == -7.25).all())
    assert torch.equal(ko[1].view(torch.int16), k[0, :, 3].view(torch.int16))


def test_append_then_gather_returns_the_rows():
    k, v = randn((100, 2, 128), 1), randn((100, 2, 128), 2)
    kc, vc = (torch.zeros((9, 2, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.randperm(144, device="cuda")[:100]
    pgd.kv_append(k, v, slots, kc, vc)
    ko, vo = pgd.kv_gather(kc, vc, slots)
    assert torch.equal(ko, k) and torch.equal(vo, v)


def test_row_operators_capture_and_prepare():
    k, v = randn((64, 4, 128), 1), randn((64, 4, 128), 2)
    ks, vs = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    call = pgd.kv_quant_scales(k, v, ks, vs, prepare=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pgd.kv_quant_scales(k, v, ks, vs)
    k.copy_(randn((64, 4, 128), 9) * 5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ks, want_scale(k))
    k.mul_(0.5)
    call()
    torch.cuda.synchronize()
    assert torch.equal(ks, want_scale(k)) and torch.equal(vs, want_scale(v))


def test_accumulate_with_few_and_with_many_rows():
    """Both forms of the kernel raise the scales that the other wrote."""
    a, b = randn((256, 3, 128), 11), randn((900, 3, 128), 12)
    a[:, 1] *= 7
    for x, y in ((a, b), (b, a)):
        ks, vs = pgd.kv_quant_scales(x, -x)
        pgd.kv_quant_scales(y, -y, ks, vs, accumulate=True)
        both = want_scale(torch.cat([a, b]))
        assert torch.equal(ks, both) and torch.equal(vs, both)


@pytest.mark.parametrize("hkv,d,bs,dt", [
    (1, 128, 16, "bf16"), (1, 128, 16, "e4m3"), (3, 256, 32, "e4m3"), (40, 128, 16, "bf16")])
@pytest.mark.parametrize("shift", [0, 8])
def test_gather_of_many_rows(hkv, d, bs, dt, shift):
    """Several tokens a CTA, the last CTA not full, padding and slots past the
    pool among them, outputs on 32 and on 16 bytes."""
    nb, n = 53, 5003
    k, v = pool(nb, hkv, bs, d, dt, 4), pool(nb, hkv, bs, d, dt, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    slots = torch.randint(-40, nb * bs, (n,), generator=g, device="cuda")
    slots[100], slots[4999] = nb * bs, 1 << 41
    ks, vs = (torch.exp2(torch.randn(hkv, generator=g, device="cuda")) for _ in range(2))
    base = [torch.full((n * hkv * d + 16,), -7.25, dtype=torch.bfloat16, device="cuda")
            for _ in range(2)]
    ko, vo = (x[shift:shift + n * hkv * d].view(n, hkv, d) for x in base)
    pgd.kv_gather(k, v, slots, ko, vo, k_scale=ks, v_scale=vs)
    assert pgd.get_device_error() == 4
    on = (slots >= 0) & (slots < nb * bs)
    at = torch.where(on, slots, 0)
    for out, cache, sc, x in ((ko, k, ks, base[0]), (vo, v, vs, base[1])):
        rows = cache.transpose(1, 2).reshape(nb * bs, hkv, d)[at]
        if dt == "e4m3":
            rows = (rows.view(torch.float8_e4m3fn).float() * sc[:, None]).to(torch.bfloat16)
            same = (out == rows) | (torch.isnan(out) & torch.isnan(rows))
        else:
            same = out.view(torch.int16) == rows.view(torch.int16)
        assert bool(same[on].all()) and bool((out[~on] == -7.25).all())
        assert bool((x[:shift] == -7.25).all()) and bool((x[shift + n * hkv * d:] == -7.25).all())
