"""CPU checks of the mixture-of-experts host side at its edges."""
import ctypes

import pytest

from persistent_stream_matmul_gb300 import _binding as B
from persistent_stream_matmul_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    B.load()


MOST = 2 ** 31 - 1024


def _work(plan, offsets, unit):
    """The unit's pieces as flat rows of nine values."""
    off = (ctypes.c_int32 * len(offsets))(*offsets)
    n = ctypes.c_int64()
    lib = B.load()
    assert lib.gemm_grouped_plan_units(plan.handle, off, unit, None, 0, ctypes.byref(n)) == B.GEMM_OK
    buf = (ctypes.c_int32 * (9 * max(1, n.value)))()
    assert lib.gemm_grouped_plan_units(plan.handle, off, unit, buf, n.value, ctypes.byref(n)) == B.GEMM_OK
    return [buf[9 * i:9 * i + 9] for i in (*range(min(n.value, 50)), *range(max(0, n.value - 50), n.value))], n.value


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("offsets", [[0, MOST], [5, MOST], [0, 2_140_000_000, MOST], [0, 2_120_000_000], [0, 0, 1, MOST - 1]])
def test_rows_up_to_the_largest_index(offsets, ctas):
    """Groups of more than 2^31 - tile rows: widths and rows stay in range, the
    tiles join without a gap, and every tile is some unit's."""
    plan = B.GroupedPlan(B.GEMM_GROUPED_ROWS, len(offsets) - 1, MOST, 8, 8, B.GEMM_BF16, B.GEMM_ROW_MAJOR,
                         offline_sms=152, ctas=ctas)
    side, tiles = plan.info("tile_n"), 0
    ends = {}
    for unit in (0, 1, plan.info("units") - 1):
        pieces, _ = _work(plan, offsets, unit)
        for tile, g, tm, n0, valid, width, k0, k1, kb in pieces:
            assert 0 < valid <= width <= side and width % (16 * ctas) == 0 and (tm, k0, k1, kb) == (0, 0, 1, 1)
            assert offsets[g] <= n0 and n0 + valid <= offsets[g + 1]
            ends.setdefault(tile, (n0, n0 + valid))
    for tile in ends:
        if tile + 1 in ends:
            assert ends[tile][1] == ends[tile + 1][0]
    tiles = sum(_work(plan, offsets, u)[1] for u in range(plan.info("units")))
    assert tiles == sum(-(-(b - a) // side) for a, b in zip(offsets, offsets[1:]))
    plan.close()


@pytest.mark.parametrize("sms", [2 ** 31 - 2, 2 ** 30])
def test_more_units_than_an_index_holds_twice(sms):
    """A unit's next tile number may pass 2^31; the walk ends there."""
    plan = B.GroupedPlan(B.GEMM_GROUPED_INNER, 3, 100, 256, 256, B.GEMM_BF16, B.GEMM_ROW_MAJOR, offline_sms=sms, ctas=1)
    counts = {u: _work(plan, [0, 50, 60, 100], u)[1] for u in (0, 1, 11, 12, sms - 1)}
    assert counts == {0: 1, 1: 1, 11: 1, 12: 0, sms - 1: 0}
    plan.close()


def test_give_up_hook_refusals():
    plan = B.GroupedPlan(B.GEMM_GROUPED_ROWS, 3, 100, 256, 256, B.GEMM_BF16, B.GEMM_ROW_MAJOR, offline_sms=152)
    for value, status in ((-2, B.GEMM_ERR_UNSUPPORTED), (plan.info("units"), B.GEMM_ERR_UNSUPPORTED), (0, B.GEMM_ERR_NO_DEVICE)):
        with pytest.raises(B.GemmError) as e:
            plan.set_option(B.GEMM_GROUPED_OPT_INJECT_GIVE_UP, value)
        assert e.value.status == status
    plan.close()


def test_layer_refuses_weights_that_are_not_on_a_gpu():
    import torch

    from persistent_stream_matmul_gb300.moe_layer import MoELayer
    w = torch.zeros(8, 16, 24, dtype=torch.float16)
    for up in (w, w.float(), None):
        with pytest.raises(ValueError):
            MoELayer(4, 2, torch.zeros(8, 24, dtype=torch.float16), up, torch.zeros(8, 24, 16, dtype=torch.float16))


@pytest.mark.parametrize("bad", [b"host bytes", "text", 1.5, bytearray(8), ctypes.c_char_p(b"x"), object()])
def test_operands_that_are_no_addresses_are_refused(bad):
    """ctypes takes bytes and str as pointers to host memory."""
    P = 0x1000
    with pytest.raises((AttributeError, TypeError)):
        B.gemm_moe_combine(bad, 16, P, P, 0, 2, 16, 1, P, 16)  # no tokens: nothing would be read
    with pytest.raises((AttributeError, TypeError)):
        B.gemm_moe_combine(P, 16, P, P, 0, 2, 16, 1, P, 16, bad)
    plan = B.Plan(0, 8, 8, B.GEMM_BF16, B.GEMM_ROW_MAJOR, B.GEMM_ROW_MAJOR, "dp", offline_sms=152)
    with pytest.raises((AttributeError, TypeError)):
        plan.run(P, bad, P)
    plan.close()


def test_offsets_for_another_number_of_groups_are_refused():
    """The library reads one offset more than the plan has groups."""
    plan = B.GroupedPlan(B.GEMM_GROUPED_ROWS, 4, 100, 64, 64, B.GEMM_BF16, B.GEMM_ROW_MAJOR, offline_sms=152)
    assert plan.info("groups") == 4 and plan.units([0, 1, 2, 3, 4], 0)
    for offsets in ([], [0], [0, 1, 2, 3], [0, 1, 2, 3, 4, 5]):
        with pytest.raises(ValueError):
            plan.units(offsets, 0)
    plan.close()
