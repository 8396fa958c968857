"""The memory of shared-memory limits and occupancy answers (csrc/gqa_limits.h), driven by
a small host program with more kernels than the library has, in place of the runtime."""
import shutil
import subprocess

import pytest

from gqa_decode_attention_kv_gb300 import build as gbuild

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <new>
#include "gqa_limits.h"
static bool no_memory = false;
void* operator new(std::size_t n) {
    if (no_memory) throw std::bad_alloc();
    void* p = std::malloc(n);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
int main() {
    const int kernels = 1000;
    static char fns[kernels];
    gqa::KernelLimits limits;
    std::map<std::pair<int, const void*>, int> runtime;      // what the runtime would hold
    int sets = 0, asks = 0, lowered = 0, failed = 0;
    auto use = [&](int dev, int i, int smem) {
        const void* fn = &fns[i];
        const bool ok = limits.raise(dev, fn, smem, [&](int bytes) {
            ++sets;
            int& now = runtime[{dev, fn}];
            lowered += bytes < now;
            now = bytes;
            return true;
        });
        failed += !ok || runtime[{dev, fn}] < smem;          // a launch at this size would fail
        const int n = limits.ctas(dev, fn, 128, smem, [&] { ++asks; return 1 + smem % 3; });
        failed += n != 1 + smem % 3;
    };
    // sizes that rise and fall, as they do with the batch; every kernel on two devices
    const int size[] = {1000, 9000, 1008, 9000, 5000, 1000};
    for (int s : size)
        for (int dev = 0; dev < 2; ++dev)
            for (int i = 0; i < kernels; ++i) use(dev, i, s);
    // a call that the runtime refuses is not remembered as made
    int tries = 0;
    for (int r = 0; r < 2; ++r) failed += limits.raise(0, &fns[0], 20000, [&](int) { ++tries; return false; });
    for (int r = 0; r < 2; ++r) failed += limits.ctas(0, &fns[0], 1, 7, [&] { ++tries; return 0; }) != 0;
    // without memory for an entry: no limit is set that would be forgotten, no exception
    static char other;
    no_memory = true;
    failed += limits.raise(0, &other, 5000, [&](int) { ++lowered; return true; });
    failed += limits.ctas(0, &other, 128, 5000, [] { return 3; }) != 3;
    failed += !limits.raise(0, &fns[0], 9000, [&](int) { ++lowered; return true; });
    no_memory = false;
    failed += !limits.raise(0, &other, 5000, [](int) { return true; });
    std::printf("%d %d %d %d %d\n", sets, asks, lowered, failed, tries);
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_kernel_keeps_the_largest_limit(tmp_path):
    src, exe = tmp_path / "limits.cpp", tmp_path / "limits"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", gbuild.CSRC, str(src), "-o", str(exe)], check=True)
    sets, asks, lowered, failed, tries = map(int, subprocess.run([str(exe)], capture_output=True, text=True,
                                                                 check=True).stdout.split())
    assert (sets, lowered, failed, tries) == (2 * 1000 * 2, 0, 0, 4)
    assert asks == 2 * 1000 * 4                              # four sizes, each asked for once
