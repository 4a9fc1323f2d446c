"""Sizes that the benchmark computes before it touches the GPU."""
import math
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402
from decode_attention_mfa_gb300 import workloads as wl  # noqa: E402


@pytest.mark.parametrize("e2e", [False, True])
@pytest.mark.parametrize("steps,warmup", [(1, 0), (7, 3), (20, 5), (100, 10), (512, 20), (4000, 20)])
@pytest.mark.parametrize("R", [1, 2, 5, 12, 19, 59])
def test_a_cache_copy_has_room_for_every_token_appended_to_it(R, steps, warmup, e2e):
    """Warm-up steps go round the copies; each later phase repeats, region after region, the copies its first region used."""
    tokens = [0] * R
    for i in range(warmup):
        tokens[i % R] += 1
    at, n_ev = warmup, max(2, min(steps, 512))
    phases = [(steps, 81), (n_ev, 1)] + [(steps, 1)] * e2e
    for n, regions in phases:
        for i in range(n):
            tokens[(at + i) % R] += regions
        at += n * regions
    assert bench.steps_per_copy(R, warmup, phases) == max(tokens)


def test_twenty_steps_of_the_ragged_workload_fit():
    """Twelve copies and regions of twenty steps: eight copies take two steps a region, four take one, so the mean of 140
    tokens a copy is not enough room."""
    w = wl.WORKLOADS["ragged"]
    lens = bench.bench_lengths(w)
    regions = math.ceil(0.2 / (20 * bench.est_step_seconds(w, lens)))
    phases = [(20, regions), (20, 1)]
    R = bench.choose_copies(w, lens, 5 + sum(n * r for n, r in phases))
    assert bench.appends(w) and 20 % R
    assert bench.steps_per_copy(R, 5, phases) >= 2 * regions > math.ceil((5 + 20 * (regions + 1)) / R) + 2
