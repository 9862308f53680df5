"""What the launch rules keep about a device (csrc/moe_device.h), compiled for the host with stand-ins for the queries."""
import os
import subprocess

import quantized_routed_expert_router_gb300 as moe

CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")

PROGRAM = r"""
#include <cstdio>
#include "moe_device.h"
#define WANT(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
int main() {
    int asked = 0, answer = 0;
    const auto ask = [&] { ++asked; return answer; };
    moe::PerDevice a;
    answer = -1;                                   // a query that fails is not an answer
    WANT(a.get(0, ask) == -1 && a.get(0, ask) == -1 && asked == 2);
    answer = 16;
    WANT(a.get(0, ask) == 16 && asked == 3);
    answer = 9;                                    // another device has its own
    WANT(a.get(1, ask) == 9 && asked == 4);
    WANT(a.get(0, ask) == 16 && a.get(1, ask) == 9 && asked == 4);
    answer = 0;                                    // none fit: an answer too
    WANT(a.get(2, ask) == 0 && a.get(2, ask) == 0 && asked == 5);
    WANT(a.get(63, ask) == 0 && a.get(64, ask) == 0 && a.get(64, ask) == 0 && a.get(-1, ask) == 0 && asked == 9);
    return 0;
}
"""


def test_answers_are_kept_for_each_device_and_failures_are_not(tmp_path):
    src, exe = tmp_path / "answers.cpp", tmp_path / "answers"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_the_products_keep_nothing_about_a_device_elsewhere():
    with open(os.path.join(CSRC, "moe_matmul.cu")) as f:
        text = f.read()
    assert "static const int" not in text and "static const bool" not in text
    assert text.count("static PerDevice") == 2
