"""kda_verify_drafts on the longest rows that an int holds: the walk of a row ends after it, where
a signed index would have passed 2^31 and begun again below zero."""
import pytest

torch = pytest.importorskip("torch")
from test_verify_drafts import kda  # noqa: E402,F401  (the package, or a skip)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [2 ** 31 - 1, 2 ** 31 - 8])
def test_verify_rows_of_almost_2_to_31(kda, V):  # noqa: F811
    target = torch.zeros(1, 1, V, dtype=torch.bfloat16, device="cuda")
    noise = torch.ones(1, V, device="cuda")
    target[0, 0, 5], target[0, 0, V - 2] = 0.25, 0.5
    none = torch.empty(1, 0, dtype=torch.int32, device="cuda")
    accepted, tokens = torch.full((1,), -9, dtype=torch.int32, device="cuda"), torch.full((1, 1), -9, dtype=torch.int32, device="cuda")
    kda.kda_verify_drafts(target, None, none, none.float(), noise, accepted, tokens)
    assert kda.kda_fwd_get_error() == 0
    assert accepted.item() == 0 and tokens.item() == V - 2
    noise[0, V - 2] = 4.0
    kda.kda_verify_drafts(target, None, none, none.float(), noise, accepted, tokens)
    assert tokens.item() == 5


def test_the_walk_needs_more_than_a_signed_index():
    """The largest index that the kernel compares with the row's end, for its narrowest and its
    widest cluster and each access: at most a turn past the row, which an unsigned int holds."""
    for split in (1, 16):
        for vec, at_once in ((1, 8), (8, 1), (8, 2)):
            units = (2 ** 31 - 1) // vec
            largest = units - 1 + at_once * split * 512
            assert largest < 2 ** 32 and (vec > 1 or largest >= 2 ** 31)
