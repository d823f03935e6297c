"""CPU check of the rules by which the int8 product, the norm's gradient and the calls over gradients are launched
(csrc/schedule.hpp, compiled with the host compiler)."""
import os
import subprocess

import pytest

from tests._i8_cases import BIG, CASES, ROWS, T32X32

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
THREADS = {k: 256 if k <= 2 else 512 for k in range(8)}


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("i8") / "i8_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-I", os.path.join(ROOT, "blockwise_scaled_fp8_act_amd", "csrc"),
                    os.path.join(ROOT, "tests", "i8_check.cpp"), "-o", exe], check=True)

    def run(queries):
        r = subprocess.run([exe], input="\n".join(queries) + "\n", capture_output=True, text=True, check=True)
        return [tuple(int(v) for v in ln.split()) for ln in r.stdout.strip().split("\n")]
    return run


def test_every_kernel_has_cases(ask):
    """The GPU tests' problems reach the kernel that they are listed under, and no kernel is left out."""
    for kernel, past, shapes in CASES:
        for shape, got in zip(shapes, ask([f"i8 {M} {N} {K} 256" for M, N, K in shapes])):
            assert got[:2] == (kernel, past), (shape, got)
    assert {k for k, _, _ in CASES} == set(range(BIG + 1))


def test_choices(ask):
    """The measured best, or one within the fit's error of it."""
    for shape, want in {(1, 14336, 4096): {0}, (4, 5120, 5120): {0}, (16, 5120, 5120): {1}, (16, 14336, 4096): {2}, (64, 14336, 4096): {3}, (256, 4096, 4096): {3},
                        (512, 4096, 4096): {4}, (768, 5120, 5120): {5}, (2048, 4096, 4096): {6}, (4096, 4096, 4096): {7}, (16384, 5120, 5120): {7}}.items():
        assert ask(["i8 %d %d %d 256" % shape])[0][0] in want, shape


def test_launches_stay_below_2_32_lanes(ask):
    """For every problem within the entry point's limits (fewer than 2^22 tiles of 64 x 64)."""
    shapes = []
    for M in (1, 2, 4, 5, 31, 32, 33, 64, 65, 128, 1 << 12, 1 << 17, 1 << 20, (1 << 28) - 64):
        n = ((1 << 22) - 1) // -(-M // 64)
        shapes += [(M, 64 * n, K) for K in (1, 128, 131071)] + [(M, max(1, 64 * n - 63), 256), (M, 1 << 24, 64) if n >= 1 << 18 else (M, 64, 64)]
    for (M, N, K), (kernel, past, bm, bn) in zip(shapes, ask([f"i8 {M} {N} {K} 256" for M, N, K in shapes])):
        tiles = -(-M // bm) * -(-N // bn) if kernel != ROWS else -(-N // bn)
        assert tiles * THREADS[kernel] < 1 << 32 and tiles < 1 << 31, (M, N, K, kernel)
        if past:
            assert M <= bm and T32X32 <= kernel <= 3


def test_rows_and_gradients(ask):
    assert ask(["back 0", "back 1", "back 512", "back 513", "back 16777200"]) == [(0,), (1,), (512,), (512,), (512,)]
    assert ask(["grads 1", "grads 512", "grads 100000"]) == [(1,), (512,), (512,)]
    assert ask(["past 1e6", "past 200e6", "past 201e6"]) == [(0,), (0,), (1,)]
