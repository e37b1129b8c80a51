"""The absorbed form's row tiles (klt_latent_attend): one by one, and two of a sequence side by side, in
batches that the rule for them takes for what they are and in others."""
import pytest

from test_gpu_latent import _lib, run_attend  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,counts", [
    (64, [2] + [1] * 31),               # one sequence has a second tile
    (64, [4, 1, 1, 2] * 8),             # two queries on average: alike by count alone
    (64, [2] * 32), (64, [3] * 12), (72, [1] * 32), (72, [2, 0] * 16), (192, [1] * 32),
    (100, [1, 2, 1] * 10), (128, [1, 3, 0, 2] * 8), (256, [1] * 20), (40, [4, 2, 3] * 6)])
@pytest.mark.parametrize("many", [1, 4])
def test_row_tiles_of_a_sequence(heads, counts, many):
    counts = counts * many  # fewer items than CTAs, and more
    lens = [(67 * i) % 401 for i in range(len(counts))]
    run_attend(heads, lens, counts, seed=len(counts), rope=32)
