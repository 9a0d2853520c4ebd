"""Which processes may run the four-CTA GEMM layout (multicast loads): those alone on one GPU."""
import os
import subprocess
import sys

import pytest

from adjoint_gradients_long_gb300 import build as adj_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("env,allowed", [({}, True), ({"WORLD_SIZE": "1"}, True), ({"WORLD_SIZE": "2"}, False),
                                         ({"WORLD_SIZE": "8", "ADJ_GEMM_QUAD": "1"}, False), ({"ADJ_GEMM_QUAD": "0"}, False)])
def test_multicast_only_in_a_process_of_its_own(env, allowed):
    adj_build.build()
    clean = {n: v for n, v in os.environ.items() if n not in ("WORLD_SIZE", "ADJ_GEMM_QUAD")}
    r = subprocess.run([sys.executable, "-c", "from adjoint_gradients_long_gb300 import lib; print(lib.load().adj_gemm_multicast())"],
                       cwd=ROOT, env={**clean, "CUDA_VISIBLE_DEVICES": "", **env}, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == ("1" if allowed else "0")
