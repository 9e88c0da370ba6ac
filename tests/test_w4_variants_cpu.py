"""Every kernel of the 4-bit products is run by a GPU test, with every length of
sums, with and without zero points: the sizes of those tests through the rule
itself (tests/c_abi/tdg_w4_plan.cc), on the CPU."""
import os
import subprocess

import pytest

import tiled_dense_gemm_loop_amd.build as b

pytest.importorskip("torch")
import test_w4_gpu as first  # noqa: E402
import test_w4_variants_gpu as more  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Sizes (rows, groups, N, K, group, lda) -> the names of their kernels."""
    exe = str(tmp_path_factory.mktemp("plan") / "w4_plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I" + b.CSRC,
                    os.path.join(ROOT, "tests", "c_abi", "tdg_w4_plan.cc"), "-o", exe], check=True, timeout=120)

    def run(sizes):
        res = subprocess.run([exe], input="".join("%d %d %d %d %d %d\n" % s for s in sizes), capture_output=True,
                             text=True, timeout=60, check=True)
        return res.stdout.splitlines()
    return run


FEW = ["few 1 1 16", "few 1 1 8", "few 1 2 8", "few 1 4 8", "few 2 4 8"]
TILES = ["tile 128 512", "tile 64 256", "tile 64 128", "tile 32 128", "tile 32 64"]


def test_every_kernel_is_run(kernels):
    sizes = [(m, g, n, k, group, k) for m, g, n, k in first.TILES + more.MORE for group in more.GROUPS]
    sizes += [(256, len(off) - 1, n, k, group, k) for off, n, k in more.SKEWED for group in more.GROUPS]
    sizes += [(m, g, n, k, group, more.FAR) for m, g, n, k in more.APART for group in more.GROUPS]
    # (each of them runs with and without zero points)
    run = {(name, bool(s[1]), 128 if s[4] % 128 == 0 else 64 if s[4] % 64 == 0 else 32)
           for s, name in zip(sizes, kernels(sizes))}
    want = {(name, grouped, span) for name in FEW + TILES for grouped in (False, True) for span in (32, 64, 128)}
    want -= {("few 1 1 16", True, span) for span in (32, 64, 128)}  # one matrix alone
    want -= {("tile 128 512", grouped, span) for grouped in (False, True) for span in (32, 64)}  # whole blocks alone
    assert run == want, (sorted(want - run), sorted(run - want))


def test_skewed_groups_run_the_kernels_of_few_rows(kernels):
    sizes = [(256, len(off) - 1, n, k, 64, k) for off, n, k in more.SKEWED]
    assert all(off[-1] <= 256 and off == sorted(off) for off, _, _ in more.SKEWED)
    assert {"few 1 1 8", "few 1 2 8", "few 1 4 8"} == set(kernels(sizes))


def test_the_rule_at_its_borders(kernels):
    """Both sides of the sizes at which the rule changes, and none that it has no
    kernel for."""
    at = {(4, 0, 6144, 4096, 128, 4096): "few 1 1 16", (5, 0, 6144, 4096, 128, 4096): "few 1 1 8",
          (5, 0, 6144, 8192, 128, 8192): "few 1 1 16", (5, 0, 6145, 8192, 128, 8192): "few 1 2 8",
          (1, 0, 10240, 4096, 128, 4096): "few 1 2 8", (1, 0, 10241, 4096, 128, 4096): "few 1 4 8",
          (16, 0, 1 << 20, 4096, 128, 4096): "few 1 4 8", (17, 0, 1 << 20, 4096, 128, 4096): "few 2 4 8",
          (32, 0, 1 << 20, 4096, 128, 4096): "few 2 4 8", (33, 0, 1 << 20, 4096, 128, 4096): "tile 32 128",
          (128, 0, 4096, 4096, 128, 4096): "few 2 4 8", (129, 0, 4096, 4096, 128, 4096): "tile 32 64",
          (256, 32, 2048, 2048, 128, 2048): "few 1 4 8", (257, 32, 2048, 2048, 128, 2048): "tile 32 128",
          (4096, 0, 4096, 4096, 128, 4096): "tile 128 512", (4096, 0, 4096, 4096, 64, 4096): "tile 64 256",
          (4096, 0, 4096, 4096, 128, (1 << 24) - 257): "tile 128 512",
          (4096, 0, 4096, 4096, 128, (1 << 24) - 256): "few 2 4 8", (4096, 0, 4096, 0, 128, 1): "few 2 4 8"}
    assert dict(zip(at, kernels(list(at)))) == at
