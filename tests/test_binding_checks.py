"""Arguments that the Python binding refuses by itself (CPU)."""
import pytest

import moe_expert_load_amd as mx

NO_DEVICE = -1                                             # get_device() of a CPU tensor


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
