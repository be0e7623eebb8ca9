"""kda_qk_norm and kda_qk_norm_bwd refuse more rows than their 32-bit walk can end on: the last
step of a group of lanes goes up to one stride past the last item."""
import pytest

from test_qk_norm import _c_call

T = 2 ** 31 - 1


@pytest.mark.parametrize("name", ["kda_qk_norm", "kda_qk_norm_bwd"])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 0), (1, 2)])
def test_more_rows_than_a_walk_can_end_on(name, Hq, Hk):
    assert _c_call(name, T=T, Hq=Hq, Hk=Hk, D=2, rotary=0, qs=8, ks=8) == -2


def test_a_stride_is_shorter_than_the_room_that_is_kept():
    """Blocks per SM (at most 3) x SMs x warps of a block x items of a warp."""
    assert 3 * 152 * 8 * 32 < 2 ** 18
