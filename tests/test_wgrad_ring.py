"""The weight gradient's ring of stages, modelled on the CPU: four groups of warps take the stages in turn, so a group
waits on a barrier whose last phases it has not seen. A wait by parity cannot tell a phase from the one two before it; the
model has the same waits, in the order that the kernel's source has them, and lets copies, decoding and products take any
time. A stage decoded before its codes have come, or while the products still read its operand, is an error."""
import heapq
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "clip_tensor_adamw_gb300", "csrc",
                      "wgrad.cu")


def kernel():
    """(stages, groups, the workers' waits before a stage is decoded, in order)"""
    text = open(SOURCE).read()
    number = lambda name: int(re.search(rf"\b{name} = (\d+)[,;]", text).group(1))  # noqa: E731
    workers = text[text.index("if (whose == group) {"):]
    workers = workers[:workers.index("decode<T>(")]
    waits = re.findall(r"mbar_wait_idle\(&bar\.(\w+)\[s\], turn\.round( \^ 1)?\)", workers)
    return number("kDepths"), number("kGroups"), [(name, bool(flip)) for name, flip in waits]


class Barrier:
    """An mbarrier: a wait for parity p passes when the phase under way has the other parity."""

    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left = self.count
            self.phase += 1

    def passed(self, parity):
        return self.phase % 2 != parity


def run(depths, groups, waits, steps, delay):
    """Runs `steps` stages; delay(kind, step): how long the copy, decoding or products of a step take. The steps that
    were decoded from other codes than their own, or over an operand in use."""
    bars = {name: [Barrier(1) for _ in range(depths)] for name in ("codes_full", "codes_empty", "ready", "used")}
    codes, operand, wrong = [None] * depths, [None] * depths, []  # whose is in the stage; None: on its way, or free
    events, order, now = [], 0, 0.0

    def later(time, action):
        nonlocal order
        order += 1
        heapq.heappush(events, (now + time, order, action))

    def copies():
        for k in range(steps):
            s, turn = k % depths, k // depths
            yield bars["codes_empty"][s], (turn + 1) % 2
            codes[s] = None

            def landed(s=s, k=k):
                codes[s] = k
                bars["codes_full"][s].arrive()
            later(delay("copy", k), landed)

    def group(which):
        for k in range(which, steps, groups):
            s, turn = k % depths, k // depths
            for name, flip in waits:
                yield bars[name][s], (turn + flip) % 2
            if codes[s] != k or operand[s] is not None:
                wrong.append(k)
            operand[s] = k
            done = Barrier(1)
            later(delay("decode", k), done.arrive)
            yield done, 0
            bars["codes_empty"][s].arrive()
            bars["ready"][s].arrive()

    def products():
        for k in range(steps):
            s, turn = k % depths, k // depths
            yield bars["ready"][s], turn % 2
            done = Barrier(1)
            later(delay("products", k), done.arrive)
            yield done, 0
            operand[s] = None
            bars["used"][s].arrive()

    waiting = [(p, next(p)) for p in [copies(), products()] + [group(g) for g in range(groups)]]
    while waiting:
        moved = True
        while moved:
            moved = False
            for i, (process, (bar, parity)) in enumerate(waiting):
                if bar.passed(parity):
                    waiting[i] = (process, next(process, None))
                    moved = True
            waiting = [w for w in waiting if w[1] is not None]
        if wrong or not events:
            break
        now, _, action = heapq.heappop(events)
        action()
    assert wrong or not waiting, "the model came to a stop"
    return wrong


def one_late_copy(late):
    """The codes of step `late` take long, the others a little longer than the products."""
    return lambda kind, step: {"copy": 50.0 if step == late else 3.0, "decode": 1.0, "products": 0.5}[kind]


def random_delays(seed):
    rng = random.Random(seed)
    return lambda kind, step: rng.expovariate(1.0) * rng.choice([0.1, 1.0, 10.0])


def test_the_kernel_waits_for_its_own_codes():
    depths, groups, waits = kernel()
    assert {name for name, _ in waits} == {"codes_full", "used"}
    for late in range(12):
        assert run(depths, groups, waits, 40, one_late_copy(late)) == [], late
    for seed in range(300):
        assert run(depths, groups, waits, 60, random_delays(seed)) == [], seed


def test_the_model_shows_stale_codes():
    """The other order decodes a stage before its codes have come, and without a wait for the products it overwrites
    their operand."""
    depths, groups, _ = kernel()
    codes, used = ("codes_full", False), ("used", True)
    for late in range(12):
        assert run(depths, groups, [codes, used], 40, one_late_copy(late)) == [late + depths]
    assert any(run(depths, groups, [codes], 60, random_delays(seed)) for seed in range(50))


@pytest.mark.parametrize("groups", [1, 2, 3, 4, 5])
def test_the_order_holds_for_other_groups(groups):
    """(with more groups than stages, a group could miss two phases of the products' barrier as well)"""
    depths, _, waits = kernel()
    for seed in range(60):
        assert run(depths, groups, waits, 60, random_delays(seed)) == [], seed
