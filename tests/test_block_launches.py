"""What the operators around the GEMMs ask of the CUDA runtime (no GPU needed): a recording
stand-in takes its place."""
import pytest

import _launches


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
