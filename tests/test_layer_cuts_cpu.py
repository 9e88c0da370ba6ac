"""Every way in which the layer of experts is cut is run by a GPU test: the sizes
of those tests through the plan itself (tests/c_abi/tdg_layer_plan.cc), against
what a wide sweep of sizes meets, on the CPU."""
import os
import subprocess

import pytest

import tiled_dense_gemm_loop_amd as tdg
import tiled_dense_gemm_loop_amd.build as b

pytest.importorskip("torch")
import test_layer_cuts_gpu as cuts  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "layer_plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I" + b.CSRC,
                    os.path.join(ROOT, "tests", "c_abi", "tdg_layer_plan.cc"), "-o", exe], check=True, timeout=120)

    def run(sizes=None):
        text = "" if sizes is None else "".join("%d %d %d %d %d\n" % s for s in sizes)
        return subprocess.run([exe] + ["sweep"] * (sizes is None), input=text, capture_output=True, text=True,
                              timeout=60, check=True).stdout.splitlines()
    return run


def test_every_plan_is_run(plan):
    met = dict(line.split(": ") for line in plan())
    assert len(met) >= 40
    run = set(plan(cuts.CUTS)) | set(plan([s + (0,) for s in cuts.EMPTY]))
    assert run == set(met), {**{k: met[k] for k in set(met) - run}, **{k: "tested, not met" for k in run - set(met)}}


def test_tested_sizes_are_those_that_the_layer_takes():
    for size in cuts.CUTS + [s + (0,) for s in cuts.EMPTY]:
        assert size[1] <= size[2] and tdg.tdg_expert_layer_workspace(*size) > 0
