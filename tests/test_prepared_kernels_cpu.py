"""The library's record of the kernels whose launch attributes are set
(csrc/clo_prepared.cuh), compiled for the host: the library has more kernels than
such a record may forget, and forgetting one costs two driver calls on each
launch."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "clo_prepared.cuh"
#include <stdio.h>
#include <stdlib.h>
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
static clo::PreparedKernels done;
int main() {
    const uintptr_t base = 0x7f0000001000u;
    auto func = [&](int i) { return reinterpret_cast<const void*>(base + 16 * static_cast<uintptr_t>(i)); };
    // 150 kernels in 3 contexts, of neighbouring 16-byte aligned addresses.
    for (unsigned long long ctx = 1; ctx <= 3; ++ctx)
        for (int i = 0; i < 150; ++i) {
            CHECK(!done.has(func(i), ctx, 0));
            done.add(func(i), ctx, 1000 + i);
        }
    for (unsigned long long ctx = 1; ctx <= 3; ++ctx)
        for (int i = 0; i < 150; ++i) {
            CHECK(done.has(func(i), ctx, 0) && done.has(func(i), ctx, 1000 + i));
            CHECK(!done.has(func(i), ctx, 1001 + i) && !done.has(func(i), ctx + 3, 0));
        }
    done.add(func(7), 2, 5000);  // more shared memory than before
    CHECK(done.has(func(7), 2, 5000) && !done.has(func(7), 1, 5000) && done.has(func(8), 2, 1008));
    // Contexts without end: what was just added is always there, and nothing is
    // there that was not added.
    for (unsigned long long ctx = 10; ctx < 2000; ++ctx) {
        for (int i = 0; i < 100; ++i) {
            CHECK(!done.has(func(i), ctx, 0));
            done.add(func(i), ctx, 1);
            CHECK(done.has(func(i), ctx, 1));
        }
    }
    return 0;
}
"""


def test_every_kernel_is_remembered(tmp_path):
    src = tmp_path / "prepared.cpp"
    src.write_text(PROGRAM)
    exe = str(tmp_path / "prepared")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-O1", "-I",
                    os.path.join(ROOT, "offloaded_kv_decode_gb300", "csrc"), str(src), "-o", exe], check=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout
