"""What the library asks of the runtime once per device: csrc/gdn_per_device.h, compiled alone for the host."""
import os
import subprocess

import linear_attention_layer_causal_b200 as gdn

CSRC = os.path.join(os.path.dirname(gdn.__file__), "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <thread>
#include <vector>
#include "gdn_per_device.h"
using namespace gdn;
int main() {
    static PerDevice<int, 4> known;
    int asked = 0, fails = 2;
    const int *v = nullptr;
    auto query = [&](int *out) {
        ++asked;
        if (fails > 0) {
            --fails;
            *out = -1;
            return cudaErrorMemoryAllocation;
        }
        *out = 10 * asked;
        return cudaSuccess;
    };
    // the error of a query is that call's only
    printf("%d ", known.get(1, query, &v) == cudaErrorMemoryAllocation && v == nullptr);
    printf("%d ", known.get(1, query, &v) == cudaErrorMemoryAllocation && v == nullptr);
    printf("%d ", known.get(1, query, &v) == cudaSuccess && *v == 30);
    // what was found stays, and is that device's only
    printf("%d ", known.get(1, query, &v) == cudaSuccess && *v == 30 && asked == 3);
    printf("%d ", known.get(0, query, &v) == cudaSuccess && *v == 40 && asked == 4);
    printf("%d ", known.get(1, query, &v) == cudaSuccess && *v == 30 && asked == 4);
    printf("%d ", known.get(-1, query, &v) == cudaErrorInvalidDevice && known.get(4, query, &v) == cudaErrorInvalidDevice);
    // one query for many threads
    std::vector<std::thread> ts;
    for (int i = 0; i < 8; ++i)
        ts.emplace_back([&] { const int *w; for (int k = 0; k < 1000; ++k) known.get(3, query, &w); });
    for (auto &t : ts)
        t.join();
    printf("%d\n", asked == 5);
}
"""


def test_a_failed_query_is_asked_again_and_devices_are_apart(tmp_path):
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", "/usr/local/cuda/include", str(src), "-o", str(exe), "-lpthread"])
    assert subprocess.check_output([str(exe)], text=True).split() == ["1"] * 8
