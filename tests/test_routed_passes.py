"""How an expert's pairs are cut into passes: every pair in one pass, no pass above 128 pairs, passes start at
multiples of 16, and their sizes differ by less than two units of 16 (a pass of one pair beside full ones would read
and convert whole weight tiles for it)."""
import os
import subprocess

from quantized_activation_q4_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "qk_passes.cuh"

static int check(int pairs) {
    const int passes = qk::passes_of(pairs);
    if (passes != (pairs + 127LL) / 128) return 1;
    int at = 0, least = 1 << 30, most = 0;
    const int step = passes > 100000 ? passes / 1000 : 1;   // of very long lists some passes and their successors
    for (int p = 0; p < passes; p += step) {
        const qk::PassRange r = qk::pass_range(pairs, passes, p);
        if (step == 1 && r.start != at) return 2;
        if (r.start % 16 || r.n < 1 || r.n > 128) return 3;
        if (p + 1 < passes ? qk::pass_range(pairs, passes, p + 1).start != r.start + r.n : r.start + r.n != pairs) return 4;
        at = r.start + r.n;
        least = r.n < least ? r.n : least;
        most = r.n > most ? r.n : most;
    }
    return most - least >= 32 ? 5 : 0;
}
int main() {
    for (int pairs = 1; pairs <= 20000; pairs++)
        if (int e = check(pairs)) return printf("%d pairs: rule %d\n", pairs, e), 1;
    for (int shift = 15; shift <= 30; shift++)
        for (int off = -130; off <= 0; off++)
            if (int e = check((1 << shift) + off)) return printf("%d pairs: rule %d\n", (1 << shift) + off, e), 1;
    for (int pairs : {1009, 1153, 2049, 897, 65537, 999983, 123456789})
        if (int e = check(pairs)) return printf("%d pairs: rule %d\n", pairs, e), 1;
    puts("ok");
    return 0;
}
"""


def test_passes_cover_the_pairs_in_nearly_equal_parts(tmp_path):
    src, exe = tmp_path / "passes.cpp", tmp_path / "passes"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", build.CSRC, "-o", os.fspath(exe), os.fspath(src)],
                   check=True)
    r = subprocess.run([os.fspath(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
