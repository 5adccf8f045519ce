"""The example program's calls together: quantised registry, relocation, attention."""
import pytest

from examples import cached_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("args", [{}, {"chunk_lens": (65, 1), "prompt": 1, "question": 1},
                                  {"chunk_lens": (700, 64, 129), "prompt": 64, "question": 130}])
def test_question_over_relocated_e4m3_chunks(args):
    """A value's e4m3 rounding is at most 2^-4 of it, evenly spread: 2^-4 / sqrt(3) = 0.036
    in the mean square at most.  A score's 512 quantised terms have a standard deviation
    of sqrt(512 / 192) = 1.63, so it moves by 0.059 at most and a weight by that fraction:
    sqrt(0.036^2 + 0.059^2) = 0.069 of the output, and 1.5 times that for small samples.
    A misplaced or wrongly rotated row gives errors near one."""
    errors = cached_attention.run(**args)
    assert len(errors) == 10 and max(errors) < 0.104, errors
