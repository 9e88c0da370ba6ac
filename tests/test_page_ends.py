"""The rule that keeps the products' reads inside their operands' pages, on the
CPU: tests/c_abi/tdg_page_ends.cc, under UndefinedBehaviorSanitizer."""
import os
import subprocess

import tiled_dense_gemm_loop_amd.build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_read_leaves_its_operands_pages(tmp_path):
    exe = str(tmp_path / "page_ends")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                    "-I" + b.CSRC, os.path.join(ROOT, "tests", "c_abi", "tdg_page_ends.cc"), "-o", exe],
                   check=True, timeout=120)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and "page ends passed" in res.stdout, res.stdout + res.stderr
