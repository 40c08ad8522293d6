"""The barriers between the warps of the many-rows decode kernel (csrc/quant_rows.cu), as a model on the CPU: every order in
which its roles may run has to end.  An mbarrier holds one phase at a time, and a wait names a phase by its parity alone: a
role that asks two phases late waits for ever.  The roles' waits and arrivals are those of the kernel, one thread for each
role (the arrival counts are the roles'), the tensor core a role of its own that ends products in their order.
"""
import random

import pytest

TILES = 12
SUMS = 4  # tiles after which the sums are moved


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, parity):
        return self.phase & 1 != parity & 1  # the phase of that parity is not the current one


def _roles(softmax_waits_for_keys):
    b = {"k_full0": 1, "k_full1": 1, "v_full0": 1, "v_full1": 1, "k_empty0": 1, "k_empty1": 1, "v_empty0": 1, "v_empty1": 1,
         "s_full": 1 if softmax_waits_for_keys else 2, "s_free": 2, "p_full": 2, "pv_done": 1}
    bars = {k: Barrier(n) for k, n in b.items()}
    tensor = []  # what a commit arrives on once the products before it have ended

    def unpack():
        for n in range(TILES):
            st, ph = n & 1, (n >> 1 & 1) ^ 1
            yield f"k_empty{st}", ph
            bars[f"k_full{st}"].arrive()
            yield f"v_empty{st}", ph
            bars[f"v_full{st}"].arrive()

    def products():
        def scores(n):
            yield f"k_full{n & 1}", n >> 1 & 1
            if n > 0:
                yield "s_free", (n - 1) & 1
            if not softmax_waits_for_keys:
                bars["s_full"].arrive()
            tensor.extend(("s_full", f"k_empty{n & 1}"))
        yield from scores(0)
        for n in range(TILES):
            if n + 1 < TILES:
                yield from scores(n + 1)
            yield f"v_full{n & 1}", n >> 1 & 1
            yield "p_full", n & 1
            tensor.extend(("pv_done", f"v_empty{n & 1}"))

    def core():
        for _ in range(4 * TILES):
            yield "tensor", 0
            bars[tensor.pop(0)].arrive()

    def softmax():
        for n in range(TILES):
            if n > 0 and n % SUMS == 0:
                yield "pv_done", (n - 1) & 1
            yield "s_full", n & 1
            if softmax_waits_for_keys:
                yield f"k_full{n & 1}", n >> 1 & 1
            bars["s_free"].arrive()
            yield f"v_full{n & 1}", n >> 1 & 1
            if n > 0:
                yield "pv_done", (n - 1) & 1
            bars["p_full"].arrive()
        yield "pv_done", (TILES - 1) & 1

    return bars, tensor, [unpack(), products(), core(), softmax(), softmax()]


def _ends(rng, softmax_waits_for_keys):
    """One run under a random order; roles differ in speed."""
    bars, tensor, roles = _roles(softmax_waits_for_keys)
    waits = {r: next(r) for r in roles}
    speed = {r: rng.choice((1, 1, 3, 20)) for r in roles}
    while waits:
        can = [r for r, (bar, parity) in waits.items() if (tensor if bar == "tensor" else bars[bar].done(parity))]
        if not can:
            return False
        r = rng.choices(can, [speed[x] for x in can])[0]
        try:
            waits[r] = next(r)
        except StopIteration:
            del waits[r]
    return True


@pytest.mark.parametrize("seed", range(4))
def test_every_order_ends(seed):
    rng = random.Random(seed)
    assert all(_ends(rng, False) for _ in range(1500))


def test_the_model_finds_a_wait_that_comes_two_phases_late():
    """Softmax warps that also wait for the key tile's own barrier: a late one finds the tile after the next there."""
    rng = random.Random(9)
    assert not all(_ends(rng, True) for _ in range(1500))
