"""The attention plan on the CPU: the device's own code, run under sanitizers by a team
of one thread and followed as the kernels follow it (tests/attn_plan_run.cpp)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANGXX = "/opt/rocm/llvm/bin/clang++"
pytestmark = pytest.mark.skipif(not os.path.exists(CLANGXX), reason="ROCm toolchain not found")


@pytest.fixture(scope="module")
def plan_run(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "plan_run")
    subprocess.run([CLANGXX, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-o", exe, os.path.join(ROOT, "tests", "attn_plan_run.cpp")], check=True, capture_output=True)
    return exe


@pytest.mark.parametrize("kind", ["ordered", "groups", "bad_groups", "bad_lengths", "bad_ends", "bad_bounds", "everything", "long"])
def test_plan(plan_run, kind):
    r = subprocess.run([plan_run, kind, "3000"], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]


@pytest.mark.parametrize("kind", ["bad_ends", "bad_lengths"])
def test_records_of_bad_batches(plan_run, kind):
    """No join reads a record or a partial result that nobody wrote."""
    r = subprocess.run([plan_run, kind, "3000", "records"], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]
