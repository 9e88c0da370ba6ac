"""Rows past what one grid holds: the steps on the CPU
(tests/c_abi/tdg_row_steps.cc, under UndefinedBehaviorSanitizer), and the
products that take them on the GPU."""
import os
import subprocess

import pytest

import tiled_dense_gemm_loop_amd.build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_piece_of_rows_is_taken_once(tmp_path):
    exe = str(tmp_path / "row_steps")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                    "-I" + b.CSRC, os.path.join(ROOT, "tests", "c_abi", "tdg_row_steps.cc"), "-o", exe],
                   check=True, timeout=120)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and "row steps passed" in res.stdout, res.stdout + res.stderr


@pytest.mark.gpu
@pytest.mark.parametrize("M", [65535 * 16 + 5, 65535 * 32 + 33, 5000000])
@pytest.mark.parametrize("N", [1, 33])
def test_zeros_of_more_rows_than_the_grid_holds(M, N):
    """K = 0: zeros in every row of C, nothing beside them."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import tiled_dense_gemm_loop_amd as tdg
    A = torch.empty(M, 0, dtype=torch.float16, device="cuda")
    codes = torch.empty(0, N, 64, dtype=torch.uint8, device="cuda")
    scales = torch.empty(0, N, dtype=torch.float16, device="cuda")
    C = torch.full((M + 200, N + 1), 7.0, device="cuda")
    tdg.gemm_f16w4f32(A, codes, scales, C=C[100:100 + M, :N])
    assert (C[100:100 + M, :N] == 0).all()
    C[100:100 + M, :N] = 7
    assert (C == 7).all()
