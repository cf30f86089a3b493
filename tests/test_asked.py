"""What is asked of the driver once: a failed answer is not kept (csrc/asked.cuh
with a fake of the failing call, on the CPU)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "asked.cuh"
int main() {
    kvc::AskedOnce asked;
    int calls = 0;
    const int answers[] = {0, -2, 168, 7};
    auto fake = [&] { return answers[calls++]; };
    if (asked.get(fake) != 0 || asked.get(fake) != -2) return 1;    // both fail and are told so
    if (asked.get(fake) != 168 || calls != 3) return 2;             // the third is answered
    if (asked.get(fake) != 168 || calls != 3) return 3;             // and not asked again
    return 0;
}
"""


def test_a_failed_answer_is_asked_for_again(tmp_path):
    src, exe = tmp_path / "asked.cpp", tmp_path / "asked"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-I", os.path.join(ROOT, "eviction_kvc_score_gb300", "csrc"), str(src), "-o", str(exe)])
    assert subprocess.run([str(exe)]).returncode == 0

