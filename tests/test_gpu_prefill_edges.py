"""Prompt attention at the edges of its tiles, shares and number ranges, against
the definition in 64 bits (tests/prefill_ref.py derives the tolerances)."""
import pytest
import torch

import paged_gqa_decode_07_b200 as pgd
from tests.test_gpu_prefill import check_packed, check_paged

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
