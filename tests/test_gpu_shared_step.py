"""The example of samples runs tables, writers, fork, copies, attention, release and compaction together."""
import pytest

from examples import shared_prefix_samples as example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompt,samples,steps,budget", [(700, 12, 3, 16), (1, 1, 1, 1), (64, 5, 2, 3), (130, 40, 1, 1000)])
def test_samples(prompt, samples, steps, budget):
    worst, free, extent, pages = example.main(prompt, samples, steps, budget)
    # outputs are at most the largest |v| (below 6 for these draws); a rounding of 2^-8 to bf16, and as much again
    # for the weights' share
    assert worst <= 6 * 2 * 2.0 ** -8
    kept = [b for b in range(samples + 1) if b % 2]
    # pages of the prompt that its samples share, and each one's own behind them
    full, most = prompt // 64, -(-(prompt + steps) // 64)
    used = (full if kept else 0) + len(kept) * (most - full)
    assert pages - free == used and extent == used
