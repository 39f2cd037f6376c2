"""CPU check of where the parts of the delta rule's workspace lie, by the library's
own host code (tests/delta_workspace_driver.cpp)."""
import shutil
import subprocess
from pathlib import Path

import pytest

import exact_online_amd as fi
from test_operators_workspace import ROCM, ROOT

needs_host_build = pytest.mark.skipif(shutil.which("g++") is None or not Path(ROCM, "include/hip").is_dir(), reason="g++ or HIP's headers missing")


@needs_host_build
def test_parts_lie_apart_and_aligned(tmp_path):
    exe = tmp_path / "delta_workspace_driver"
    lib = Path(fi.LIB_PATH)
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
                    f"-I{ROOT / 'exact_online_amd' / 'csrc'}", "-o", str(exe), str(ROOT / "tests" / "delta_workspace_driver.cpp"),
                    str(lib), f"-Wl,-rpath,{lib.parent}", f"-Wl,-rpath,{ROCM}/lib", f"-L{ROCM}/lib", "-lamdhip64"],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
