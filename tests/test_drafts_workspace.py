"""CPU check of the workspaces of the delta rule and of the check of drafts: handles of
random sizes, calls of random smaller ones, planned by the library's own host code
(tests/drafts_workspace_driver.cpp)."""
import shutil
import subprocess
from pathlib import Path

import pytest

import exact_online_amd as fi
from test_operators_workspace import ROCM, ROOT


@pytest.mark.skipif(shutil.which("g++") is None or not Path(ROCM, "include/hip").is_dir(), reason="g++ or HIP's headers missing")
def test_no_call_uses_more_than_its_handle_holds(tmp_path):
    exe = tmp_path / "drafts_workspace_driver"
    lib = Path(fi.LIB_PATH)
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
                    f"-I{ROOT / 'exact_online_amd' / 'csrc'}", "-o", str(exe), str(ROOT / "tests" / "drafts_workspace_driver.cpp"),
                    str(lib), f"-Wl,-rpath,{lib.parent}", f"-Wl,-rpath,{ROCM}/lib", f"-L{ROCM}/lib", "-lamdhip64"],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
