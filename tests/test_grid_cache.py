"""The table behind resident_grid (csrc/grid_cache.h), compiled for the host: it holds every kernel
instance of the library at hundreds of shapes each, and gives no key another's value (no GPU)."""
import os
import subprocess

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include "grid_cache.h"

int main()
{
    static moe::GridCache cache;
    static char code[1 << 16];
    int n = 0, wrong = 0;
    // 200 kernels at ten sizes of shared memory, then one kernel at a thousand
    auto key = [&](int i) {
        return i < 2000 ? moe::GridKey{code + 16 * (i / 10), 0, 256, (size_t)(i % 10) * 1024}
                        : moe::GridKey{code + 8, i % 2, 128, (size_t)(i / 2) * 4};
    };
    for (; n < 3000; n++) {
        wrong += cache.find(key(n)) != -1;
        cache.add(key(n), n + 1);
    }
    for (int i = 0; i < n; i++) wrong += cache.find(key(i)) != i + 1;
    // past its room it keeps what it has, and every search ends
    for (int i = n; i < 10000; i++) cache.add(moe::GridKey{code + 4, 0, i, 0}, i + 1);
    for (int i = 0; i < n; i++) wrong += cache.find(key(i)) != i + 1;
    int held = 0;
    for (int i = n; i < 10000; i++) {
        const int v = cache.find(moe::GridKey{code + 4, 0, i, 0});
        wrong += v != -1 && v != i + 1;
        held += v != -1;
    }
    wrong += held != moe::GridCache::kMost - n;
    std::printf("%d\n", wrong);
}
"""


def test_grid_cache(tmp_path):
    source, program = tmp_path / "cache.cpp", tmp_path / "cache"
    source.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "combine_moe_route_06_gb300", "csrc")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-Wall", "-Werror", "-I", csrc,
                    str(source), "-o", str(program)], check=True)
    assert subprocess.run([str(program)], check=True, capture_output=True, text=True).stdout == "0\n"
