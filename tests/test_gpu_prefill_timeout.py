"""The timeout path of the prompt attention kernels, forced without hanging
anything: the limit of their waits is shortened with the test hook, so that
the roles give up one by one, the copies and products in flight still end, and
the CTA leaves; the next normal call gives the bits of a fresh run."""
import pytest
import torch

import paged_gqa_decode_07_b200 as pgd
from tests.test_gpu_prefill import bits, cu_of, make_pages, randn

pytestmark = pytest.mark.gpu

TIMEOUT_FLAG = 8


@pytest.fixture(autouse=True)
def _restore():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pgd.load_library()
    pgd.debug_set_wait_limit_ns(0)
    assert pgd.get_device_error() == 0
    yield
    pgd.debug_set_wait_limit_ns(0)
    torch.cuda.synchronize()
    pgd.get_device_error()


def exercise(run):
    ref = [bits(t).clone() for t in run()]
    torch.cuda.synchronize()
    assert pgd.get_device_error() == 0
    for limit in (1, 300, 3000):
        pgd.debug_set_wait_limit_ns(limit)
        run()
        torch.cuda.synchronize()
        flags = pgd.get_device_error()
        pgd.debug_set_wait_limit_ns(0)
        assert flags & ~TIMEOUT_FLAG == 0
        assert limit > 1 or flags == TIMEOUT_FLAG, "a 1 ns limit must run out"
        got = run()
        torch.cuda.synchronize()
        assert pgd.get_device_error() == 0
        for a, b in zip(ref, got):
            assert torch.equal(a, bits(b)), f"limit {limit} ns: the next call differs"


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("ctas", [0, 60])
def test_packed(d, ctas):
    hq, hkv = 8, 2
    cu, cu_t = cu_of([700, 64, 1, 300])
    q, k, v = (randn((cu[-1], h, d), i) for i, h in enumerate((hq, hkv, hkv)))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")

    def run():
        pgd.prefill_attention(q, k, v, cu_t, hq, hkv, d, 0.09, out, lse_out=lse, num_ctas=ctas)
        return out, lse
    exercise(run)


@pytest.mark.parametrize("d,dt", [(128, "bf16"), (256, "bf16"), (128, "e4m3")])
def test_paged(d, dt):
    hq, hkv, bs, ctx, q_lens = 8, 2, 16, [3000, 17, 900], [100, 17, 1]
    kc, vc, table, ks, vs = make_pages(ctx, hkv, d, bs, dt, 3)
    cu, cu_t = cu_of(q_lens)
    q = randn((cu[-1], hq, d), 4)
    ctx_t = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")

    def run():
        pgd.paged_prefill_attention(q, kc, vc, table, ctx_t, cu_t, hq, hkv, d, bs, 0.09, out,
                                    lse_out=lse, k_scale=ks, v_scale=vs)
        return out, lse
    exercise(run)
