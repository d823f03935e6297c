"""CPU check that the routed products of tests/_moe_cases.py run, each, the kernel that it names, and together
all of them, by the rule of csrc/schedule.hpp."""
import os
import subprocess

from tests import _moe_cases as cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "blockwise_scaled_fp8_act_amd", "csrc")


def test_products_run_every_kernel(tmp_path):
    src, exe = tmp_path / "rule.cpp", str(tmp_path / "rule")
    src.write_text(r'''
#include <cstdio>
#include "schedule.hpp"
int main() {
    long long M, N, K, E, swiglu;
    while (std::scanf("%lld %lld %lld %lld %lld", &M, &N, &K, &E, &swiglu) == 5)
        switch (bsfp8::sched::routed_kernel(M, N, K, E, swiglu != 0)) {
            case bsfp8::sched::kRoutedRegisters16: std::puts("registers16"); break;
            case bsfp8::sched::kRoutedRegisters32: std::puts("registers32"); break;
            default: std::puts(bsfp8::sched::routed_reads_once(M, N, E, swiglu != 0) ? "lds past the caches" : "lds");
        }
}
''')
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", exe], check=True)
    text = "".join(f"{cases.rows(c)} {c['N']} {c['K']} {cases.experts(c)} {int(c['swiglu'])}\n" for c in cases.PRODUCT_FORMS)
    got = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    assert got == [c["kernel"] for c in cases.PRODUCT_FORMS]
    kernels = ("registers16", "registers32", "lds", "lds past the caches")
    assert {(c["kernel"], c["swiglu"]) for c in cases.PRODUCT_FORMS} == {(k, s) for k in kernels for s in (False, True)}
