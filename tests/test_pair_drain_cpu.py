"""The end of a CTA pair's two producers, without a GPU: a model of the ring's
barriers in which each of the two gives up wherever its own waits run out, and
csrc/pair_left.h, which says what has to be waited for before either CTA may
leave."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "post_weight_quantization_accum_b200", "csrc")


@pytest.fixture(scope="module")
def pair_left(tmp_path_factory):
    where = tmp_path_factory.mktemp("pair")
    src, so = where / "shim.cpp", where / "shim.so"
    src.write_text('#include "pair_left.h"\n'
                   'extern "C" void left(uint32_t e, uint32_t o, uint32_t s, uint32_t* r) {\n'
                   '  const gptq::PairLeft l = gptq::pair_left(e, o, s); r[0] = l.first; r[1] = l.both; r[2] = l.most; }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))

    def call(even, odd, stages):
        r = (ctypes.c_uint32 * 3)()
        lib.left(even, odd, stages, r)
        return tuple(r)
    return call


class Barrier:
    """The even CTA's barrier of a stage: an arrival and its expected bytes a phase."""

    def __init__(self):
        self.phase, self.armed, self.bytes = 0, False, 0

    def step(self):
        if self.armed and self.bytes == 0:
            self.phase, self.armed = self.phase + 1, False

    def arm(self, n):
        assert not self.armed
        self.armed, self.bytes = True, self.bytes + n
        self.step()

    def arrive(self, n):
        self.bytes -= n
        self.step()


def _run(rng, stages, total, stop):
    """One run of two producers and the products, in a random order of steps, each
    giving up at its own point.  Returns the barriers, the uses that each producer
    issued and the copies under way, as (use, bytes)."""
    half = [int(rng.integers(1, 5)) * 4096 for _ in range(total)]
    full = [Barrier() for _ in range(stages)]
    issued, used, way = [0, 0], 0, []
    limit = [int(rng.integers(0, total + 1)) if stop[i] else total for i in range(3)]
    while True:
        can = []
        for p in (0, 1):  # a producer goes on when the products have used the stage's last use
            if issued[p] < limit[p] and (issued[p] < stages or used > issued[p] - stages):
                can.append(p)
        if used < limit[2] and full[used % stages].phase > used // stages:
            can.append(2)
        can += [3] * (len(way) > 0)
        if not can or (can == [3] and rng.random() < 0.3):
            return full, half, issued, way
        what = rng.choice(can)
        if what < 2:
            u = issued[what]
            if what == 0:
                full[u % stages].arm(2 * half[u])
            way.append((u, half[u]))
            issued[what] += 1
        elif what == 2:
            used += 1
        else:
            u, n = way.pop(int(rng.integers(len(way))))
            full[u % stages].arrive(n)


@pytest.mark.parametrize("stages", [5, 6])
def test_nothing_is_under_way_when_the_pair_leaves(pair_left, stages):
    rng = np.random.default_rng(stages)
    even_only = odd_only = missed = 0
    for _ in range(4000):
        total = int(rng.integers(0, 25))
        full, half, (even, odd), way = _run(rng, stages, total, rng.random(3) < 0.4)
        first, both, most = pair_left(even, odd, stages)
        assert both == min(even, odd) and most == max(even, odd) and first <= both and most - first <= stages
        even_only += even > odd
        odd_only += odd > even
        # what waiting for the even CTA's own uses alone would leave under way
        missed += any(u >= even for u, _ in way)
        for u in range(first, most):
            bar = full[u % stages]
            if u >= both:
                if most == even:
                    bar.arrive(half[u])
                else:
                    bar.arm(half[u])
            for w in [w for w in way if w[0] % stages == u % stages]:  # (the wait: these copies land meanwhile)
                assert w[0] == u
                way.remove(w)
                bar.arrive(w[1])
            assert bar.phase == u // stages + 1 and bar.bytes == 0  # the wait for this use's phase ends
        assert not way
    assert min(even_only, odd_only, missed) > 50
