"""Shared memory of the eviction: what a block asks for, over capacities and budgets.  No GPU."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "intra_spatial_pipelining_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <climits>
#include "evict_words.h"

int main() {
    const int fixed = 4488, budgets[] = {1, 255, 256, 1000, 4096, 8192, 8193, 32768, 60000, 1 << 20, INT_MAX};
    const int caps[] = {1, 64, 255, 256, 257, 1024, 4096, 8192, 8193, 16384, 20000, 28000, 30000, 49151, 49152,
                        49153, 100000, 1 << 25, INT_MAX};
    for (int cap : caps)
        for (int b : budgets) {
            const sgp::EvictWords w = sgp::evict_words(cap, b, fixed);
            const long long bytes = 4ll * (w.key + w.list) + fixed, need = cap < b ? cap : b;
            bool ok = bytes <= 227 * 1024 && w.key >= (cap < 49152 ? cap : 49152) && w.key % 256 == 0 &&
                      w.list % 256 == 0;
            // the list holds every position that can stay, and no more than that; or it does not fit
            if (w.list) ok = ok && w.list >= need && w.list < need + 256;
            else ok = ok && 4 * (w.key + need) + fixed > 226 * 1024;
            // two blocks to an SM (228 KB, 1 KB of each taken by the system)
            if (cap <= 8192) ok = ok && 2 * (bytes + 1024) <= 228 * 1024;
            if (!ok) return std::printf("cap %d budget %d: %d + %d words\n", cap, b, w.key, w.list), 1;
        }
    return 0;
}
"""


def test_no_more_than_the_cache_holds(tmp_path):
    src, exe = tmp_path / "words.cpp", tmp_path / "words"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
