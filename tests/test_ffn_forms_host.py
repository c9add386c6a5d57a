"""Which forms of the feed-forward block's kernels a shape takes (zk::ffn_plan, on the CPU): the
shapes of the GPU tests reach every form, and those named for a form take it."""
import os
import shutil
import subprocess

import pytest

from ffn_shapes import FEW, LARGE

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    from zero_sharded_optimizer_rank_amd import abi, build
    lib = os.path.dirname(abi.LIB_PATH)
    exe = str(tmp_path_factory.mktemp("forms") / "ffn_forms")
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                    "-I", build.INCLUDE, "-I", build.CSRC, os.path.join(HERE, "ffn_forms.cpp"),
                    abi.LIB_PATH, "-L/opt/rocm/lib", "-lamdhip64", f"-Wl,-rpath,{lib}",
                    "-Wl,-rpath,/opt/rocm/lib", "-o", exe], check=True)

    def run(shapes, odd=False):
        args = [str(int(v)) for s in shapes for v in (*s, odd)]
        out = subprocess.run([exe, *args], check=True, capture_output=True, text=True).stdout
        return [{k: int(v) for k, v in (p.split("=") for p in line.split())}
                for line in out.splitlines()]
    return run


@pytest.mark.parametrize("shapes", [LARGE, FEW], ids=["large", "few"])
def test_named_shapes(plan, shapes):
    for p, (shape, want) in zip(plan(shapes), shapes.items()):
        assert {k: p[k] for k in want} == want, shape


def test_every_form_is_tested(plan):
    pytest.importorskip("torch")
    import test_gpu_ffn as tg
    shapes = tg.SHAPES + [(t, 256, 384) for t in (1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 64)]
    shapes = shapes + [*FEW, *LARGE]
    plans = plan(shapes)
    few = [(p["sets_in"], p["sets_out"], -(-t // 16)) for p, (t, _, _) in zip(plans, shapes)
           if p["few"]]
    assert (1, 1, 1) in few
    for tokens in (1, 2, 3, 4):  # in sixteens: a kernel of its own each
        assert {f[:2] for f in few if f[2] == tokens} >= {(2, 2), (2, 4), (4, 2), (4, 4)}
    assert {p["split_y"] > 1 for p in plans if p["few"]} == {False, True}
    for tile in ("in", "out", "back1", "back2"):
        assert {p["small_" + tile] for p in plans if not p["few"] or "back" in tile} == {0, 1}
    for split, small in (("in", "in"), ("y", "out"), ("dh", "back1"), ("dw1", "back1"),
                         ("dx", "back2"), ("dw2", "back2")):
        seen = {(p["small_" + small], p["split_" + split] > 1) for p in plans
                if not p["few"] or "back" in small}
        assert seen >= {(1, False), (1, True), (0, False)}, split
        assert (0, True) in seen or split not in ("y", "dx"), split
