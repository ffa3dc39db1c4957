"""The plan of an 8-bit product, on the host."""
import pytest

from fp8_plan import OF_EACH_PLAN, plan


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
def test_every_plan_can_be_launched(dtype):
    """A launch holds fewer than 2^32 threads, 256 a tile, in whole rounds of 256 tiles."""
    for M in (97, 1 << 16, (1 << 20) + 1, 1 << 24, (1 << 29) + 5, 1 << 30):
        for N in (1, 64, 65, 200, 1000, 1 << 16, 1 << 22):
            if M * N > 1 << 38:        # outputs that no memory holds
                continue
            for K in (0, 16, 4096):
                bm, bn, splits = plan(M, N, K, dtype)
                if bm:
                    tiles = -(-M // bm) * -(-N // bn) * splits
                    assert -(-tiles // 256) * 256 * 256 < 1 << 32, (M, N, K, bm, bn)


@pytest.mark.parametrize("dtype,M,N,K,want", OF_EACH_PLAN)
def test_shapes_of_the_gpu_tests_get_the_plans_they_stand_for(dtype, M, N, K, want):
    assert plan(M, N, K, dtype) == want
