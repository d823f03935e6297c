"""What the compiler is told about the kernels' memory accesses, looked up on the CPU (device code is compiled and not run)."""
import os
import subprocess

import pytest

from blockwise_scaled_fp8_act_amd import build

SOURCES = [s for s in build.SOURCES if s.endswith(".hip")]


def compile_device(source, *flags):
    return subprocess.run([build.HIPCC, *build.CFLAGS, "--cuda-device-only", *flags, os.path.join(build.CSRC, source)], capture_output=True, text=True)


@pytest.mark.parametrize("source", SOURCES)
def test_no_access_claims_more_alignment_than_its_address_has(source):
    """A pointer to a type of small alignment that goes into a parameter of a larger one: a template's deduced type
    drops the attribute, and the access behind it counts as aligned."""
    r = compile_device(source, "-fsyntax-only", "-Werror=align-mismatch", "-Wno-unused-command-line-argument")
    assert r.returncode == 0, r.stderr[-2000:]


def test_shared_rows_of_sums_declare_the_alignment_of_their_stores():
    """norm_backward_kernel writes them in 16-byte pieces (store8_of of whole pieces)."""
    with open(os.path.join(build.CSRC, "norm.hip")) as f:
        text = f.read()
    assert "store8_of<true>(sums[side]" in text and "__shared__ alignas(16) float sums[" in text


def test_lanes_that_exchange_through_shared_memory_are_ordered(tmp_path):
    """The product's store_block writes a wave's tile to LDS lane by lane and reads other lanes' pieces back: in every
    instance a fence of the wave and a wave barrier stand between the two."""
    out = tmp_path / "gemm_i8.ll"
    r = compile_device("gemm_i8.hip", "-S", "-emit-llvm", "-Xclang", "-disable-llvm-passes", "-o", str(out))
    assert r.returncode == 0, r.stderr[-2000:]
    bodies = {}
    for part in out.read_text().split("\ndefine ")[1:]:
        body = part.split("\n}\n")[0]
        bodies[body.split("@", 1)[1].split("(", 1)[0]] = body
    fence = next(name for name in bodies if "wave_lds_fence" in name)
    assert 'fence syncscope("wavefront") acq_rel' in bodies[fence] and "@llvm.amdgcn.wave.barrier()" in bodies[fence]
    blocks = [body for name, body in bodies.items() if "store_block" in name and "scaled4" in body]
    assert len(blocks) >= 6
    for body in blocks:
        assert body.index("scaled4") < body.index("wave_lds_fence") < body.rindex("load <4 x i32>")
