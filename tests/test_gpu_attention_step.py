"""The serving-step example runs the tables, writers, indexer and both attentions together."""
import pytest

from examples import sparse_attention_step as example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompts", [(700, 33, 1500, 128), (1,), (64, 65, 129)])
def test_two_steps(prompts):
    worst, used = example.main(prompts=prompts)
    # outputs are at most the largest |v| (below 6 for these draws); two roundings to bf16 of 2^-8 each
    # and as much again for the weights' share
    assert max(worst) <= 6 * 3 * 2.0 ** -8
    assert used == sum(-(-(p + 1) // 64) for p in prompts)
