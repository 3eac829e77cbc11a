"""How the products' blocks of K are divided into sums (csrc/fp8z_tiles.h), on the
host: whatever the number of blocks, the sums follow one another from the first block
to the last, none is empty, and none is longer than what one sum may hold."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "blockwise_fp8_zero_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "fp8z_tiles.h"

static bool check(int k0, int k1, int most) {
    const int sums = fp8z::sums_of(k0, k1, most);
    if (sums < 1) return false;
    if (k1 == k0) return sums == 1 && fp8z::sum_start(k0, k1, 0, 1) == k0 && fp8z::sum_start(k0, k1, 1, 1) == k1;
    int at = k0;
    for (int i = 0; i < sums; ++i) {
        const int first = fp8z::sum_start(k0, k1, i, sums), end = fp8z::sum_start(k0, k1, i + 1, sums);
        if (first != at || end <= first || (most && end - first > most)) return false;
        at = end;
    }
    return at == k1;
}

int main() {
    const int mosts[] = {0, 1, 8, 24, 64};
    for (int most : mosts) {
        // 2^18 blocks: 2^24 tokens; 2^22: a vocabulary of 2^28 words
        const int large[] = {131071, 131072, 131073, 150001, 262143, 262144, 1 << 20, (1 << 22) - 1, 1 << 22};
        for (int n = 0; n <= 3000; ++n)
            if (!check(0, n, most) || !check(77, 77 + n, most)) return std::printf("%d blocks, %d a sum\n", n, most), 1;
        for (int n : large)
            if (!check(0, n, most) || !check(12345, 12345 + n, most)) return std::printf("%d blocks, %d a sum\n", n, most), 1;
    }
    return 0;
}
"""


def test_sums_cover_every_block_once(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    source, program = tmp_path / "sums.cpp", tmp_path / "sums"
    source.write_text(PROGRAM)
    # signed overflow ends the program instead of passing unseen
    subprocess.run(["g++", "-O1", "-std=c++17", "-ftrapv", "-I", CSRC, str(source), "-o", str(program)], check=True)
    r = subprocess.run([str(program)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout or f"exit {r.returncode}"
