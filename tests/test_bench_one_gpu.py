"""bench.py's own arm runs on one GPU: ranks of a larger job are told so before anything of the library or the GPU is
touched.  The GEMMs share operand tiles by TMA loads with cluster multicast, which are for single-GPU runs alone."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("what", [[], ["--profile-gemm", "256x256x256"]], ids=["run", "profile"])
@pytest.mark.parametrize("rank", [0, 1])
def test_ranks_of_a_larger_job_are_refused(rank, what):
    # an unimportable package: the refusal comes before the library is built or loaded
    code = ("import sys; sys.modules['mxfp8_microscaled_precision_gb300'] = None; sys.modules['torch'] = None\n"
            "import bench; bench.main(['--gpus', '2', '--steps', '3', '--warmup', '3'] + sys.argv[1:])")
    env = dict(os.environ, RANK=str(rank), LOCAL_RANK=str(rank), WORLD_SIZE="2", MASTER_ADDR="127.0.0.1", MASTER_PORT="1")
    r = subprocess.run([sys.executable, "-c", code, *what], cwd=ROOT, env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 1, r.stderr
    assert "one GPU" in r.stderr and "Traceback" not in r.stderr
    lines = r.stdout.splitlines()
    if rank == 0:
        line = json.loads(lines[-1])
        assert line["n_gpus"] == 2 and "one GPU" in line["unavailable"] and "value" not in line
    else:
        assert lines == []
