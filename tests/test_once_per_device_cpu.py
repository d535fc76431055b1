"""The library's per-device set-up of kernels: a kernel that has run on one device is set up again
on the next, and a set-up that failed is tried again.  The devices and the failing call are fakes."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "intra_spatial_pipelining_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <map>
#include <thread>
#include <utility>
#include <vector>
#include "once.h"

int main() {
    sgp::OncePerDevice once;
    std::map<std::pair<int, const void*>, int> calls;
    int kernel_a, kernel_b;
    auto launch = [&](int dev, const void* f, int status) {
        return once.run(dev, f, [&] { ++calls[{dev, f}]; return status; });
    };
    for (int rep = 0; rep < 3; ++rep)
        for (int dev = 0; dev < 2; ++dev)
            for (const void* f : {(const void*)&kernel_a, (const void*)&kernel_b})
                if (launch(dev, f, 0) != 0) return 1;
    for (auto& c : calls) if (c.second != 1) return 2;
    if (calls.size() != 4) return 3;
    int kernel_c;
    if (launch(1, &kernel_c, 700) != 700) return 4;   // fails: reported, and tried again
    if (launch(1, &kernel_c, 0) != 0 || launch(1, &kernel_c, 700) != 0) return 5;
    if ((calls[{1, &kernel_c}]) != 2) return 6;
    int kernel_d, n = 0;
    std::vector<std::thread> ts;
    for (int i = 0; i < 8; ++i) ts.emplace_back([&] { once.run(3, &kernel_d, [&] { ++n; return 0; }); });
    for (auto& t : ts) t.join();
    return n == 1 ? 0 : 7;
}
"""


def test_set_up_is_remembered_for_each_device(tmp_path):
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
