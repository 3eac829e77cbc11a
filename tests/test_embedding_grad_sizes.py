"""The embedding gradient's order of a long list: work that grows with the tokens, not
with their square.  Every block of the sort walks over one row of counts for each
block, so the rows are bounded, as the workspace shows."""
import os
import shutil
import subprocess

import pytest

from blockwise_fp8_zero_gb300 import fp8z

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "blockwise_fp8_zero_gb300", "csrc")


def _counts_bytes(tokens, vocab, hidden):
    """What the workspace holds beside keys and values (two buffers each), the pieces'
    partial sums, tickets and the rows in use: the counts, and under 2 KB of rounding up."""
    piece = 32 if tokens >= 8192 else 16 if tokens >= 2048 else 8
    pieces = -(-tokens // piece)
    rest = 16 * tokens + pieces * 2 * hidden * 4 + 3 * pieces * -(-hidden // 1024) * 4 + (vocab if tokens > 512 else 0)
    return fp8z.fp8z_embedding_grad_workspace(tokens, vocab, hidden) - rest


def test_counts_of_a_long_list_are_bounded():
    from blockwise_fp8_zero_gb300 import build
    build.build()
    row = 4096                                       # 1024 digits of 4 bytes
    for tokens in (1, 2048, 2049, 16384, 500000):
        assert _counts_bytes(tokens, 50000, 8) <= -(-tokens // 2048) * row + 2048
    for tokens in (1 << 20, (1 << 24) + 1, 1 << 28, 1 << 30):
        for vocab in (1, 50000, 1 << 30):
            assert 0 <= _counts_bytes(tokens, vocab, 8) <= 1024 * row


RUNS = r"""
#include <cstdio>
#include "fp8z_tiles.h"

static int looks;

static bool check(int most, int length) {
    looks = 0;
    const int got = fp8z::run_length(most, [&](int from, int step, int end) {
        ++looks;
        int n = 0;
        for (int lane = 0; lane < 32; ++lane) {
            const int q = from + step * lane;
            if (q < end && q < 1) return -1000;              // never outside 1 .. most
            n += q < end && q <= length;
        }
        return n;
    });
    if (got == length && looks <= 7) return true;
    std::printf("%d of %d: %d in %d looks\n", length, most, got, looks);
    return false;
}

int main() {
    for (int most = 0; most <= 300; ++most)
        for (int length = 0; length <= most; ++length)
            if (!check(most, length)) return 1;
    const int large[] = {1023, 1024, 32768, 1000003, (1 << 25) - 1, 1 << 25, 1 << 27};
    for (int most : large) {
        for (long long length = 0; length <= most; length += 1 + length / 3)
            if (!check(most, int(length)) || !check(most, int(most - length))) return 1;
        for (int d = 0; d < 100; ++d)
            if (!check(most, most / 3 + d) || !check(most, 32 + d)) return 1;
    }
    return 0;
}
"""


def test_ends_of_a_run_are_found_in_a_few_looks(tmp_path):
    """A run's block looks for the run's ends: 32 places at a time, not one after the other
    over the whole run, which every block of a run of 2^25 pieces would do."""
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    source, program = tmp_path / "runs.cpp", tmp_path / "runs"
    source.write_text(RUNS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-ftrapv", "-I", CSRC, str(source), "-o", str(program)], check=True)
    r = subprocess.run([str(program)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout or f"exit {r.returncode}"
