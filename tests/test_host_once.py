"""What the library looks up once per process (driver entry points, kernel attributes) is kept only when the
lookup worked: after a failure the next call looks again.  Compiled for the host, with a lookup that fails
twice."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "post_weight_quantization_14_b200",
                    "csrc")

PROGRAM = r"""
#include "host_once.h"
#include <cstdio>
#include <thread>
#include <vector>

static int answers[] = {0, 0, 96, 7};
static int asked = 0;
static int look() { return answers[asked++]; }
static void* look_up() { return nullptr; }

int main() {
    gqh::KeepFound<int> k;
    const int got[] = {k.get(look), k.get(look), k.get(look), k.get(look), k.get(look)};
    std::printf("%d %d %d %d %d asked %d\n", got[0], got[1], got[2], got[3], got[4], asked);
    gqh::KeepFound<void*> p;
    const bool none = p.get(look_up) == nullptr;
    std::printf("%d %d\n", none, p.get([] { return (void*)&answers; }) == (void*)&answers);
    gqh::KeepFound<int> shared;
    std::vector<std::thread> t;
    std::atomic<int> wrong{0};
    for (int i = 0; i < 8; ++i)
        t.emplace_back([&] {
            for (int j = 0; j < 1000; ++j) wrong += shared.get([] { return 5; }) != 5;
        });
    for (auto& x : t) x.join();
    std::printf("%d\n", wrong.load());
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_a_failed_lookup_is_tried_again(tmp_path):
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    assert out[0] == "0 0 96 96 96 asked 3"
    assert out[1] == "1 1"
    assert out[2] == "0"
