"""csrc/device_setup.h: a kernel's set-up on a device that failed is done again by the
next call, whose error it is then, and one that succeeded is not.  And the sources set
their kernels up by nothing else."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_weight_only_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "device_setup.h"

static int fails = 0;
static void want(bool good, const char* what) {
    if (!good) std::printf("%s\n", what), ++fails;
}

int main() {
    static fp8w::DeviceSetup setup;
    int calls = 0;
    want(setup(1, [&] { ++calls; return 7; }) == 7, "its error");
    want(setup(1, [&] { ++calls; return 8; }) == 8, "the next call's error");
    want(setup(1, [&] { ++calls; return 0; }) == 0 && calls == 3, "done again");
    want(setup(1, [&] { ++calls; return 9; }) == 0 && calls == 3, "not once more");
    want(setup(2, [&] { ++calls; return 0; }) == 0 && calls == 4, "another device");
    want(setup(-1, [&] { return 5; }) == 5 && setup(1000, [&] { return 6; }) == 6, "no such device");

    static fp8w::DeviceSetup many;
    std::vector<std::thread> threads;
    int once = 0;
    for (int i = 0; i < 16; ++i)
        threads.emplace_back([&] { for (int j = 0; j < 1000; ++j) many(0, [&] { ++once; return once < 3 ? 1 : 0; }); });
    for (auto& t : threads) t.join();
    want(once == 3, "threads");
    std::printf(fails ? "FAIL\n" : "ok\n");
    return fails;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_a_failed_setup_is_done_again(tmp_path):
    src, exe = tmp_path / "setup.cpp", tmp_path / "setup"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


def test_the_kernels_are_set_up_by_it():
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu"):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        assert "attr_once" not in text, name
        assert ("cudaFuncSetAttribute" in text) == ("DeviceSetup setup" in text), name
