"""What the equality tests of test_gpu_mxfp4.py rest on: FP32 holds every partial sum of their products, in any order.

Random operands there have scale codes 125 .. 128 (2^-2 .. 2^1) and E2M1 elements, multiples of 1/2: a product of two is a
multiple of (2^-1 2^-2)^2 = 2^-6.  FP32 holds every multiple of 2^-6 up to 2^24 2^-6 = 2^18.  4096 terms of the largest size, 144,
would come to 2^19.2, so it is not their number that bounds the sums: the terms of these very operands do, added by their sizes."""
import numpy as np
import pytest

import _fp4
import test_gpu_mxfp4 as gpu

LIMIT = 2.0 ** 24 * 2.0 ** -6


def _cases(test):
    """The parameter sets of a test's first mark of several names."""
    return next(m.args[1] for m in test.pytestmark if m.name == "parametrize" and "," in m.args[0])


CASES = ([(M, N, K, M + 3 * N + 7 * K) for M, N, K in gpu.PRODUCTS]
         + [(M, N, K, M * N) for M, N, K in _cases(gpu.test_few_tiles_of_many_rows)]
         + [(M, N, K, N) for M, N, K, _ in _cases(gpu.test_ragged_widths_many_times)]
         + [(1291, 2033 + width, 96, width) for width in (0, 15)])


@pytest.mark.parametrize("M,N,K,seed", CASES)
def test_no_partial_sum_leaves_what_fp32_holds(M, N, K, seed):
    rng = np.random.default_rng(seed)
    a, b = ((_fp4.values(codes, scales, K, "e2m1")) for codes, scales in (_fp4.random_operand(rng, R, K) for R in (M, N)))
    for v in (a, b):
        assert (v * 8 == np.round(v * 8)).all()   # multiples of 2^-3
    assert (np.abs(a) @ np.abs(b).T).max() < LIMIT
