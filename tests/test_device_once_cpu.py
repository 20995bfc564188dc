"""CPU-only: what the library sets once per device (the LDS limit of the
distillation kernels) is set on every device, and again after a failure."""

import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weighted_model_update_amd", "csrc")

PROGRAM = r"""
#include <cassert>
#include "device_once.h"

int main()
{
    static fa::DeviceOnce limit;
    int calls = 0, status = 0;
    const auto set = [&] { calls++; return status; };
    status = 7;
    assert(limit.run(0, set) == 7 && calls == 1); // a failure is reported,
    status = 0;
    assert(limit.run(0, set) == 0 && calls == 2); // and not kept
    assert(limit.run(0, set) == 0 && calls == 2);
    assert(limit.run(1, set) == 0 && calls == 3); // another device has its own
    assert(limit.run(1, set) == 0 && limit.run(0, set) == 0 && calls == 3);
    assert(limit.run(63, set) == 0 && limit.run(63, set) == 0 && calls == 4);
    assert(limit.run(64, set) == 0 && limit.run(64, set) == 0 && calls == 6); // beyond the table: every call
    assert(limit.run(-1, set) == 0 && calls == 7);
    return 0;
}
"""


def test_once_per_device(tmp_path):
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(exe), str(src)], check=True, timeout=120)
    subprocess.run([str(exe)], check=True, timeout=60)


def test_no_limit_is_kept_for_the_process():
    """A function attribute in a static initialiser is set for one device only."""
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".hip", ".h")):
            with open(os.path.join(CSRC, name)) as f:
                assert not re.search(r"static\s+const\s+\w+\s+\w+\s*=\s*hipFuncSetAttribute", f.read()), name
