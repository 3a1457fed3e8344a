"""Host threads in the C ABI: calls of the same kernels with different shapes at the same time."""
import threading

import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu

CALLS = 10000


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gpu_or_skip()


def _at_once(jobs):
    """Every job, a function of a stream, CALLS times in a thread of its own, all at the same time; the
    statuses that were not 0."""
    bad, start = [], threading.Barrier(len(jobs))

    def work(job):
        stream = torch.cuda.Stream()
        start.wait()
        for _ in range(CALLS):
            status = job(stream.cuda_stream)
            if status != 0:
                bad.append(status)
                return
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    [t.start() for t in threads]
    [t.join() for t in threads]
    return bad


def test_plans_of_few_and_of_many_experts():
    from mxfp8_microscaled_precision_gb300 import mxq
    L, jobs, results = mxq.lib(), [], []
    for tokens, k, experts in ((2048, 8, 1024), (4, 2, 8)):
        ids = torch.randint(0, experts, (tokens, k), device="cuda", dtype=torch.int32)
        want = mxq.moe_plan(ids, experts)
        got = tuple(torch.full_like(t, -7) for t in want)
        results.append((got, want, ids))

        def job(stream, ids=ids, got=got, tokens=tokens, k=k, experts=experts):
            return L.mxq_moe_plan(ids.data_ptr(), tokens, k, experts, got[0].data_ptr(), got[1].data_ptr(), stream)
        jobs.append(job)
    torch.cuda.synchronize()
    assert _at_once(jobs) == []
    for got, want, _ in results:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("shapes", [((64, 7168), (3, 1024)), ((64, 16384), (5, 9000)), ((64, 7167), (400, 1025))],
                         ids=lambda s: "-".join(f"{m}x{c}" for m, c in s))
def test_layer_norm_of_long_and_of_short_rows(shapes):
    """Both directions, FP32 parameters beside BF16 rows: the kernels that ask for more shared memory."""
    from mxfp8_microscaled_precision_gb300 import mxq
    L, jobs, results = mxq.lib(), [], []
    for M, C in shapes:
        x, dy = (torch.randn(M, C, device="cuda").bfloat16() for _ in range(2))
        w = torch.randn(C, device="cuda")
        y, mean, rstd = mxq.layer_norm(x, w)
        want = (y, *mxq.layer_norm_backward(dy, x, w, mean, rstd))
        got = tuple(torch.full_like(t, 7.0) for t in want)
        size = L.mxq_layer_norm_backward_workspace_size(M, C)
        workspace = torch.empty(size, dtype=torch.uint8, device="cuda")
        m2, r2 = torch.empty_like(mean), torch.empty_like(rstd)
        results.append((got, want, x, dy, w, workspace, mean, rstd, m2, r2))

        def job(stream, M=M, C=C, x=x, dy=dy, w=w, mean=mean, rstd=rstd, m2=m2, r2=r2, got=got, workspace=workspace,
                size=size):
            return (L.mxq_layer_norm(x.data_ptr(), 0, M, C, C, w.data_ptr(), None, 1, 1e-5, got[0].data_ptr(), C,
                                     m2.data_ptr(), r2.data_ptr(), stream)
                    or L.mxq_layer_norm_backward(dy.data_ptr(), x.data_ptr(), 0, M, C, C, C, w.data_ptr(), 1,
                                                 mean.data_ptr(), rstd.data_ptr(), got[1].data_ptr(), C,
                                                 got[2].data_ptr(), got[3].data_ptr(), workspace.data_ptr(), size, stream))
        jobs.append(job)
    torch.cuda.synchronize()
    assert _at_once(jobs) == []
    assert mxq.get_device_status() == 0
    for got, want, *_ in results:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
