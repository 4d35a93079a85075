"""Arguments that the Python binding refuses by itself (CPU)."""
import os

import pytest

import moe_expert_load_amd as mx

NO_DEVICE = -1                                             # get_device() of a CPU tensor


@pytest.fixture(autouse=True, scope="module")
def _built():
    if not os.path.exists(mx.LIB_PATH):
        from moe_expert_load_amd import build
        build.build()


def test_plan_with_too_few_slots():
    """A plan whose prefix sums are long enough, and whose list of slots is not."""
    c = mx.make_cfg(4, 16, 8, 2, 128, 64, 2)
    other = mx.make_cfg(4, 16, 16, 2, 128, 64, 0, mx.MODE_INFER)
    assert mx._plan_or_none(c, mx.Plan(c, device="cpu"), NO_DEVICE) is not None
    assert mx._plan_or_none(c, None, NO_DEVICE) is None
    plan = mx.Plan(other, device="cpu")
    assert plan.cu_seqlens.numel() >= c.R * (c.E + c.B + 1) and plan.slot_expert.numel() < c.R * c.B
    with pytest.raises(ValueError):
        mx._plan_or_none(c, plan, NO_DEVICE)
    # without slots the list is not read
    bare = mx.make_cfg(4, 16, 8, 2, 128, 64, 0, mx.MODE_INFER)
    assert mx._plan_or_none(bare, plan, NO_DEVICE) is not None


@pytest.mark.parametrize("rows,width", [(1, (1 << 32) + 8), (1, 1 << 31), (1, 8 - (1 << 32)), (1 << 63, 8),
                                        (8 - (1 << 64), 8)])
def test_sizes_that_the_library_cannot_take(rows, width):
    """Numbers beyond the header's int64 and int32 are refused, not cut to their low bits."""
    dc = mx.make_dropout_cfg(0.5)
    for call in (lambda: mx.moe_dropout(dc, rows, width, None, None, None, None),
                 lambda: mx.moe_q8_store(rows, width, None, None, None),
                 lambda: mx.moe_q8_load(rows, width, None, None, None)):
        with pytest.raises(mx.MoeError) as e:
            call()
        assert e.value.code == mx.MOE_ELIMIT
