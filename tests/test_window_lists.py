"""The window mask's arithmetic (csrc/stream.h) against brute force, compiled for the host: the
keys of a query, the queries of a key, the chunks a run of queries visits and keeps whole, and
the queries that keep a whole block of keys; and the division by numbers known to the host."""
import os
import subprocess

import pytest

from block_sparse_spatio_attn_b200 import build

SOURCE = r"""
#include "stream.h"
#include <algorithm>
#include <cstdio>
#include <cstdlib>
using namespace svga;
static int fdiv(int a, int b) { int q = a / b; return (a % b && a < 0) ? q - 1 : q; }
static bool keep(const Mask &m, int p, int j)
{
    const int bp = fdiv(p, m.block), bj = j / m.block;
    if (m.causal && bj > bp) return false;
    return m.window < 0 || std::abs(bp - bj) <= m.window || j < m.sinks;
}
int main()
{
    srand(1);
    constexpr int T = 8;  // rows and keys of a tile
    long bad = 0, missed = 0, checks = 0;
    for (int t = 0; t < 20000; ++t) {
        const int nq = rand() % 60 + 1, nk = rand() % 60, off = nk - nq;
        const Mask m{rand() % 2, rand() % 4 ? rand() % 12 : -1, rand() % 3 ? rand() % 40 : 0,
                     rand() % 2 ? 1 : rand() % 20 + 1};
        for (int i = 0; i < nq; ++i) {
            const MaskRange r = mask_range(m, i + off, nk);
            for (int j = 0; j < nk; ++j) {
                const bool k = keep(m, i + off, j);
                int a, e;
                mask_rows(m, j, nq, off, a, e);
                bad += k != ((j >= r.lo && j < r.hi) || j < r.sk) || k != (i >= a && i < e);
                ++checks;
            }
        }
        for (int r0 = 0; r0 < nq; r0 += T) {
            const int r1 = std::min(r0 + T, nq);
            const ChunkList c = chunk_list<T>(m, r0 + off, r1 - 1 + off, nk);
            for (int b = 0; b * T < nk + 3 * T; ++b) {
                bool any = false, all = true;
                for (int i = r0; i < r1; ++i)
                    for (int j = b * T; j < (b + 1) * T; ++j) {
                        const bool k = j < nk && keep(m, i + off, j);
                        any |= k;
                        all &= k;
                    }
                bad += any != c.visits(b) || (c.visits(b) && c.full(b) != all);
            }
        }
    }
    const Mask wide{1, 1 << 24, 1 << 24, 1 << 24};  // products past 32 bits
    for (int p : {-(1 << 24), -1, 0, 1, (1 << 24) - 1}) {
        const MaskRange r = mask_range(wide, p, 1 << 24);
        bad += r.lo != 0 || r.hi != (p < 0 ? 0 : 1 << 24) || r.sk != r.hi;
    }
    for (int t = 0; t < 200000; ++t) {  // division by a known number, over the whole range
        const int d = rand() % 3 ? rand() % 5000 + 1 : (int)((unsigned)rand() % 0x7fffffffu) + 1;
        const FastDiv f = fast_div(d);
        const long long k = rand() % (0x7fffffff / d + 1ll);
        for (long long n : {0ll, 1ll, (long long)rand() & 0x7fffffff, k * d, k * d - 1, k * d + d - 1, 0x7fffffffll})
            if (n >= 0 && n <= 0x7fffffff) bad += f.of((int)n) != n / d;
    }
    printf("%ld checks, %ld bad, %ld missed\n", checks, bad, missed);
    return bad != 0;
}
"""


@pytest.mark.skipif(not os.path.exists(build.NVCC), reason="needs nvcc")
def test_mask_arithmetic_against_brute_force(tmp_path):
    src, exe = tmp_path / "lists.cu", tmp_path / "lists"
    src.write_text(SOURCE)
    r = subprocess.run([build.NVCC, *build.ARCH, "-O2", "-std=c++17", "-I", build.CSRC, str(src),
                        "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
