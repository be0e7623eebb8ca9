"""The norms on many rows, where a group of lanes takes several heads of a token (an uneven
number of them at the end) one after another, and on rows that need more registers per lane."""
import pytest

import test_qk_norm as base
from test_qk_norm import kda  # noqa: F401  (the package, or a skip)

CASES = [
    (9000, 37, 5, 64, "rms", 32, False, "bf16"),
    (9000, 37, 5, 64, "l2", 0, False, "f32"),
    (5000, 9, 70, 128, "rms", 128, True, "f32"),
    (7, 3, 2, 300, "rms", 60, False, "bf16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_many_rows_match_definition(kda, case):  # noqa: F811
    base.test_norm_matches_definition(kda, case)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_many_rows_backward_match_definition(kda, case):  # noqa: F811
    base.test_norm_bwd_matches_definition(kda, case)
