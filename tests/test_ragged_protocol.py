"""The hand-overs between the warps of the prefill attention kernel hold under any timing, and each
rule that they rest on is needed (modelled on the host: ragged_protocol)."""
import random

import pytest

from ragged_protocol import Block, Broken, random_items


def _run(seed, f8, without=(), give_up=None):
    Block(random_items(random.Random(seed)), seed, f8, without).run(give_up)


@pytest.mark.parametrize("f8", [False, True])
def test_hand_overs_hold(f8):
    for seed in range(200):
        _run(seed, f8)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("rule", ["q_read", "pass"])
def test_rule_is_needed(rule, f8):
    """Without it the model finds a schedule that breaks."""
    with pytest.raises(Broken):
        for seed in range(200):
            _run(seed, f8, (rule,))


def _late(block, running):
    """A wait is given up after the producer has left."""
    return "producer" not in running


def _any_time(at):
    turns = iter(range(10 ** 9))
    return lambda block, running: next(turns) >= at


def test_nothing_in_flight_after_giving_up():
    for seed in range(200):
        _run(seed, seed % 2 == 0, give_up=_late)
        _run(seed, seed % 2 == 1, give_up=_any_time(random.Random(seed).randint(0, 1500)))
    with pytest.raises(Broken, match="in flight"):
        for seed in range(200):
            _run(seed, False, ("drain",), give_up=_late)
