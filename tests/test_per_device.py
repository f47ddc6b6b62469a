"""What is done once per device (the shared memory that a kernel may have): on each device, again
after a failure, and not again after a success, from several threads too."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_indexer_tiles_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"
#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
int main() {
    idx::PerDevice once;
    int calls[65] = {};
    auto set = [&](int device, int result) { return once.run(device, [&] { ++calls[device]; return result; }); };
    CHECK(set(0, 0) == 0 && set(0, 0) == 0 && calls[0] == 1)
    CHECK(set(1, 7) == 7 && calls[1] == 1)                    // the second device: not the first one's result
    CHECK(set(1, 0) == 0 && set(1, 9) == 0 && calls[1] == 2)  // after a failure again
    CHECK(set(63, 0) == 0 && set(63, 0) == 0 && calls[63] == 1 && calls[0] == 1)
    CHECK(set(64, 0) == 0 && set(64, 3) == 3 && calls[64] == 2)  // more devices than are remembered
    idx::PerDevice shared;
    std::atomic<int> ran{0}, bad{0};
    std::vector<std::thread> threads;
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([&] {
            for (int i = 0; i < 1000; ++i) {
                const int d = i % 4;
                if (shared.run(d, [&] { ++ran; return 0; }) != 0) ++bad;
            }
        });
    for (auto& t : threads) t.join();
    CHECK(bad == 0 && ran >= 4 && ran <= 32)
    return 0;
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="needs g++")
def test_once_on_every_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_no_kernel_of_the_serving_operators_is_set_up_once_per_process():
    for f in ("attention.cu", "attention_prefix.cu", "evict.cu"):
        text = open(os.path.join(CSRC, f)).read()
        assert "allow_smem(" in text and "call_once" not in text and "cudaFuncSetAttribute" not in text, f
