"""The plan of an 8-bit product with an epilogue, on the host."""
import pytest

from fp8_plan import ACT_OF_EACH_PLAN, plan_act


@pytest.mark.parametrize("dtype,M,N,K,want", ACT_OF_EACH_PLAN)
def test_shapes_of_the_gpu_tests_get_the_plans_they_stand_for(dtype, M, N, K, want):
    assert plan_act(M, N, K, dtype) == want
    # an 8-bit output: blocks of 128 columns in a workgroup, or sums that are joined
    bm, bn, splits = plan_act(M, N, K, dtype, to8=True)
    assert bm == 0 or splits > 1 or bn >= 128
    if want[1] >= 128:
        assert (bm, bn, splits) == want
