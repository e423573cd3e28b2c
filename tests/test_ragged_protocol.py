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


def _late(block, running):
    """A wait is given up after the producer has left."""
    return "producer" not in running


def _any_time(at):
    turns = iter(range(10 ** 9))
    return lambda block, running: next(turns) >= at


def test_nothing_in_flight_after_giving_up():
    for seed in range(200):
        _run(seed, 4, give_up=_late)
        _run(seed, 3, give_up=_any_time(random.Random(seed).randint(0, 1500)))
    with pytest.raises(Broken, match="in flight"):
        for seed in range(200):
            _run(seed, 4, ("drain",), give_up=_late)
