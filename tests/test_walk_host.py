"""How attention deals its work out (csrc/acp_dev_walk.hpp), run on the host with
a thread for each lane of a workgroup: waves that run late at a barrier leave all
lanes at one place, and the shares of random batches have every key once."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "async_copy_pipelining_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_walks_of_late_waves(tmp_path):
    exe = str(tmp_path / "walk_host")
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-w", f"-I{CSRC}", f"-I{ROCM}/include", "-pthread",
                    "-o", exe, os.path.join(ROOT, "tests", "walk_host.cpp")], check=True, timeout=300)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), r.stdout[-2000:] + r.stderr[-2000:]
