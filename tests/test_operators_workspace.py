"""CPU check of the operators' workspaces: handles of random sizes, calls of
random smaller ones, planned by the library's own host code
(tests/workspace_driver.cpp): no call uses more than its handle holds."""
import os
import shutil
import subprocess
from pathlib import Path

import pytest

import exact_online_amd as fi

ROOT = Path(__file__).resolve().parents[1]
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None or not Path(ROCM, "include/hip").is_dir(), reason="g++ or HIP's headers missing")
def test_no_call_uses_more_than_its_handle_holds(tmp_path):
    exe = tmp_path / "workspace_driver"
    lib = Path(fi.LIB_PATH)
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
                    f"-I{ROOT / 'exact_online_amd' / 'csrc'}", "-o", str(exe), str(ROOT / "tests" / "workspace_driver.cpp"),
                    str(lib), f"-Wl,-rpath,{lib.parent}", f"-Wl,-rpath,{ROCM}/lib", f"-L{ROCM}/lib", "-lamdhip64"],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
