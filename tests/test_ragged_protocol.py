"""The hand-overs between the warps of the prefill attention kernel hold under any timing, and each
rule that they rest on is needed (modelled on the host: ragged_protocol)."""
import random

import pytest

from ragged_protocol import Block, Broken, random_items


def _run(seed, slots, without=(), give_up=None):
    Block(random_items(random.Random(seed)), seed, slots, without).run(give_up)


@pytest.mark.parametrize("slots", [4, 3])
def test_hand_overs_hold(slots):
    for seed in range(200):
        _run(seed, slots)


@pytest.mark.parametrize("rule,slots", [("q_read", 4), ("pass", 4), ("pass", 3)])
def test_rule_is_needed(rule, slots):
    """Without it the model finds a schedule that breaks."""
    with pytest.raises(Broken):
        for seed in range(200):
            _run(seed, slots, (rule,))
