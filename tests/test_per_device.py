"""Per-device set-up of the kernels (host code, compiled and run here): once for each device, and again after an error."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "radixattention_prefix_shared_radix_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "per_device.h"
int main() {
    static sgl::PerDevice state;
    int calls[70] = {}, fail = 0;
    auto on = [&](int dev) { return state.ready(dev, [&] { ++calls[dev < 0 ? 69 : dev]; return fail; }); };
    for (int i = 0; i < 3; ++i) {
        if (on(0) || on(1) || on(63)) return 1;
    }
    if (calls[0] != 1 || calls[1] != 1 || calls[63] != 1) return 2;
    fail = 7;                                   // an error is returned, not kept
    if (on(2) != 7 || on(2) != 7 || calls[2] != 2) return 3;
    if (on(0) || calls[0] != 1) return 4;       // and leaves the others alone
    fail = 0;
    if (on(2) || on(2) || calls[2] != 3) return 5;
    if (on(64) || on(64) || calls[64] != 2 || on(-1) || calls[69] != 1) return 6;   // beyond the record: every time
    sgl::PerDevice other;                       // states are their own
    if (other.ready(0, [&] { return 9; }) != 9) return 7;
    puts("ok");
    return 0;
}
"""


def test_set_up_once_per_device(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe), "-pthread"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.returncode


def test_no_kernel_set_up_is_kept_for_the_process():
    """The opt-in to large shared memory is per device: no launch keeps it in a plain static."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for at, line in enumerate(text.splitlines(), 1):
            if "static const" in line and "attr" in line:
                raise AssertionError("%s:%d: %s" % (name, at, line.strip()))
