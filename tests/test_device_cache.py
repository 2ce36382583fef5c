"""The library's per-device facts (csrc/device_cache.h), compiled for the host: a process that uses
two devices must not size one's launches by the other's answer."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "device_cache.h"
int main() {
    static qnf4::DeviceCache c;
    int asked = 0;
    auto get = [&](int dev, int fact) {
        const int v = c.get(dev, [&] { ++asked; return fact; });
        std::printf("%d %d ", v, asked);
    };
    get(0, 132);
    get(1, 148);                // another device: its own answer
    get(0, 7);                  // kept
    get(1, 7);
    get(2, 0);                  // a failed query is not kept
    get(2, 9);
    get(1000, 5);               // past the array: asked each time
    get(1000, 6);
    get(-1, 4);
}
"""


def test_facts_are_kept_per_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "bit_nf4_quantized_double_b200", "csrc"),
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert out == "132 1 148 2 132 2 148 2 0 3 9 4 5 5 6 6 4 7".split()
