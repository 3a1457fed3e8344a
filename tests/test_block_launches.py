"""What the operators around the GEMMs ask of the CUDA runtime (no GPU needed): a recording
stand-in takes its place."""
import itertools

import pytest

import _launches

MAX_DYNAMIC = 8            # cudaFuncAttributeMaxDynamicSharedMemorySize
BLOCK_BYTES = 227 * 1024   # shared memory of a block at most


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    return _launches.load(tmp_path_factory.mktemp("recorder"))


@pytest.mark.parametrize("count", [1, 32, 33, 500, 1024, 1025, 3000])
@pytest.mark.parametrize("scale", [0, 1])
def test_a_refused_launch_is_reported_and_nothing_follows_it(record, count, scale):
    """Clipping: whichever of its launches the runtime refuses, the call says so and launches nothing
    that would read the sums that were never formed."""
    status, launches, _ = record("clip", count, 1000, scale)
    assert status == 0 and len(launches) >= 2
    for n in range(1, len(launches) + 1):
        status, done, _ = record("clip", count, 1000, scale, refuse=n)
        assert status != 0, f"launch {n} of {len(launches)} ({launches[n - 1][0]}) was refused unnoticed"
        assert done == launches[:n - 1]
        assert record.L.rec_launches() == n
    assert record("clip", count, 1000, scale)[0] == 0


@pytest.mark.parametrize("call,args", [("route", (100, 64, 4)), ("plan", (4096, 8, 128)), ("clip", (40, 1000, 0)),
                                       ("clip", (40, 1000, 1)), ("norm", (0, 0, 100, 1024)),
                                       ("norm_backward", (0, 0, 100, 64)), ("norm_backward", (0, 0, 100, 1024)),
                                       ("norm_backward", (0, 0, 100, 20001))])
def test_a_refused_launch_leaves_no_error_for_the_next_call(record, call, args):
    """The runtime keeps the error of a launch for whoever asks next: a good call after a bad one must not
    find it."""
    launches = record(call, *args)[1]
    for n in range(1, len(launches) + 1):
        assert record(call, *args, refuse=n)[0] != 0
        assert record("route", 100, 64, 4, forget=False)[0] == 0, f"the error of launch {n} of {len(launches)} was still there"


SHAPES = {
    "plan": [(t, k, e) for t, k in ((0, 8), (1, 8), (64, 1), (1000, 1), (16384, 8), (2 ** 16, 32)) for e in (1, 8, 128, 511, 1024)],
    "norm": [(f, p, m, c) for f, p in itertools.product((0, 1), (0, 1)) for m in (1, 9, 400, 16384)
             for c in (1, 8, 9, 96, 130, 512, 513, 1111, 2048, 4097, 5120, 7168, 8192, 8999, 16384, 24000, 25999, 40000)],
}
SHAPES["norm_backward"] = SHAPES["norm"]


@pytest.mark.parametrize("call", SHAPES)
def test_the_shared_memory_limit_of_a_kernel_does_not_depend_on_the_shape(record, call):
    """The limit belongs to the kernel, not to the call: were it the size that a call needs, a second
    host thread with a smaller shape could lower it between this one's setting and its launch."""
    limits, needs = {}, {}
    for shape in SHAPES[call]:
        status, launches, attributes = record(call, *shape)
        assert status == 0 and launches, shape
        for kernel, attribute, value in attributes:
            if attribute == MAX_DYNAMIC:
                limits.setdefault(kernel, set()).add(value)
        for kernel, blocks, threads, shared in launches:
            assert blocks >= 1 and 1 <= threads <= 1024, (shape, kernel)
            if shared > 48 * 1024:
                assert any(k == kernel and v >= shared for k, at, v in attributes if at == MAX_DYNAMIC), (shape, kernel)
            needs[kernel] = max(needs.get(kernel, 0), shared)
    assert limits
    for kernel, values in limits.items():
        assert len(values) == 1, (kernel, sorted(values))
        assert needs[kernel] <= max(values) <= BLOCK_BYTES, (kernel, values, needs[kernel])
