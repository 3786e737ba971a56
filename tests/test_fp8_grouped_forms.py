"""Which by-expert forms the GPU tests' sizes reach (CPU: only the plans are asked for)."""
import random

from fp8_grouped_forms import grouped_form, step_forms
from test_gpu_fp8_block import GROUPED, STEP
from test_gpu_fp8_by_expert import STORED

TEAM = "team waves 2 rows 32 x 16"
FORMS = {TEAM, "64x256", "128x256", "256x256", "64x256 wide", "128x256 wide"}


def size(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def test_every_form_by_expert_is_in_the_gpu_tests():
    reached = {grouped_form(T * topk, E, N, K, f32) for T, topk, E, N, K in GROUPED for f32 in (True, False)}
    assert reached == FORMS
    rng = random.Random(2)
    for _ in range(5000):
        rows, E, N, K = size(rng, 1, 1 << 22), size(rng, 1, 4096), size(rng, 1, 1 << 20), 16 * size(rng, 1, 4096)
        for f32 in (True, False):
            assert grouped_form(rows, E, N, K, f32) in FORMS


def test_every_form_of_the_step_is_in_the_gpu_tests():
    first = {step_forms(T * topk, E, H, F)[0] for T, topk, E, H, F, _ in STEP + STORED}
    second = {step_forms(T * topk, E, H, F)[1] for T, topk, E, H, F, _ in STEP + STORED}
    assert first == {TEAM, "64x256", "128x256", "256x256", "64x256 gated", "128x256 gated", "256x256 gated"}
    assert second == {TEAM, "64x256", "128x256", "256x256"}
    rng = random.Random(3)
    for _ in range(5000):
        rows, E, H, F = size(rng, 1, 1 << 22), size(rng, 1, 4096), 16 * size(rng, 1, 4096), 16 * size(rng, 1, 4096)
        up, down = step_forms(rows, E, H, F)
        assert up in first and down in second
        assert up.endswith(" gated") == (F % 128 == 0 and up != TEAM)
