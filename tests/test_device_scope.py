"""The scope that a packed call makes its context's device current for (the
header, compiled here with a stand-in for the runtime)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_draft_depth_gb300", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include "device_scope.h"
static int current, sets, fail_get, fail_set;
struct Fake {
    static int get(int *d) { if (fail_get) return 35; *d = current; return 0; }
    static int set(int d) { ++sets; if (fail_set) return 101; current = d; return 0; }
};
static void show(int want)
{
    sets = 0;
    int err, inside;
    {
        DeviceScope<Fake> s(want);
        err = s.err;
        inside = current;
    }
    printf("%d %d %d %d\n", err, inside, current, sets);
}
int main(void)
{
    current = 0; show(0);
    current = 0; show(3);
    current = 3; show(0);
    current = 1; fail_set = 1; show(2);
    fail_set = 0; fail_get = 1; show(2);
    return 0;
}
"""


def test_the_current_device_comes_back(tmp_path):
    (tmp_path / "a.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-Wall", "-Werror", "-I", CSRC, str(tmp_path / "a.cpp"), "-o", str(tmp_path / "a")], check=True)
    out = subprocess.run([str(tmp_path / "a")], check=True, capture_output=True, text=True).stdout.split("\n")
    # error, device inside, device behind, times it was set
    assert out[:5] == ["0 0 0 0",      # the context's own: nothing to do
                       "0 3 0 2", "0 0 3 2",
                       "101 1 1 1",    # could not be set: nothing to give back
                       "35 1 1 0"]
