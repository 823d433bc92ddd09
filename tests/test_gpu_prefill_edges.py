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
