"""CPU checks of where the parts of the delta rule's workspace lie, and that handles take no more than the
header says, by the library's own host code (tests/delta_workspace_driver.cpp)."""
import re
import shutil
import subprocess
from pathlib import Path

import pytest

import exact_online_amd as fi
from test_operators_workspace import ROCM, ROOT

needs_host_build = pytest.mark.skipif(shutil.which("g++") is None or not Path(ROCM, "include/hip").is_dir(), reason="g++ or HIP's headers missing")


def run_driver(tmp_path, *args):
    exe = tmp_path / "delta_workspace_driver"
    lib = Path(fi.LIB_PATH)
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
                    f"-I{ROOT / 'exact_online_amd' / 'csrc'}", "-o", str(exe), str(ROOT / "tests" / "delta_workspace_driver.cpp"),
                    str(lib), f"-Wl,-rpath,{lib.parent}", f"-Wl,-rpath,{ROCM}/lib", f"-L{ROCM}/lib", "-lamdhip64"],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe), *args], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr


@needs_host_build
def test_parts_lie_apart_and_aligned(tmp_path):
    run_driver(tmp_path)


@needs_host_build
def test_handles_take_what_the_header_says(tmp_path):
    said = re.search(r"/\* fi_delta_create:.*?Synchronous\.", (ROOT / "include" / "fi.h").read_text(), re.S).group(0)
    said = re.sub(r"\s*\n \*\s*", " ", said)
    assert "more than 8192" in said and "more than 32768 chunks, 4 dk dv bytes for each row and head" in said
    numbers = [re.search(p, said) for p in (r"at most (\d+) MB for the systems", r"(\d+) KB for each row and head", r"at most (\d+) MB for the states of segments")]
    assert all(numbers), said
    run_driver(tmp_path, *(n.group(1) for n in numbers))
