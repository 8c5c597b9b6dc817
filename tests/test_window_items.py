"""What a CTA of the window kernels works out before its first load (csrc/stream.h), against brute
force over random masks, compiled for the host: the merged list of key chunks of two query blocks,
and the queries that keep any, or all, of a block of keys."""
import os
import subprocess

import pytest

from block_sparse_spatio_attn_b200 import build

SOURCE = r"""
#include "stream.h"
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <vector>
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
    srand(2);
    constexpr int T = 8;  // rows and keys of a tile
    long lists = 0, blocks = 0, bad_lists = 0, bad_rows = 0, wrong_full = 0, missed_full = 0;
    for (int t = 0; t < 30000; ++t) {
        const int nq = rand() % 90 + 1, nk = rand() % 90, off = nk - nq;
        const Mask m{rand() % 2, rand() % 4 ? rand() % 14 : -1, rand() % 3 ? rand() % 50 : 0,
                     rand() % 2 ? 1 : rand() % 25 + 1};
        // pairs of query blocks: each chunk that one of them visits once, and no other
        for (int r0 = 0; r0 < nq; r0 += 2 * T) {
            const bool valid1 = r0 + T < nq;
            const ChunkList l0 = chunk_list<T>(m, r0 + off, std::min(r0 + T, nq) - 1 + off, nk);
            ChunkList l1 = l0;
            if (valid1) l1 = chunk_list<T>(m, r0 + T + off, std::min(r0 + 2 * T, nq) - 1 + off, nk);
            int a, skip, end;
            merge_lists(l0, l1, valid1, a, skip, end);
            std::vector<int> seen(nk / T + 3, 0);
            for (int e = 0; e < a + end - skip; ++e) {
                const int c = e < a ? e : skip + e - a;
                if (c < 0 || c >= (int)seen.size())
                    ++bad_lists;
                else
                    ++seen[c];
            }
            for (int c = 0; c < (int)seen.size(); ++c) {
                bool any = false;
                for (int i = r0; i < std::min(r0 + 2 * T, nq); ++i)
                    for (int j = c * T; j < std::min((c + 1) * T, nk); ++j) any |= keep(m, i + off, j);
                bad_lists += seen[c] != any;
            }
            ++lists;
        }
        // blocks of keys
        for (int k0 = 0; k0 < nk; k0 += T) {
            const int k1 = std::min(k0 + T, nk);
            int first[3], end[3];
            for (int e = 0; e < 3; ++e) mask_rows(m, block_key(m, k0, k1, e), nq, off, first[e], end[e]);
            const BlockRows r = block_rows(m, k1, nq, first[0], end[0], first[1], end[1], end[2]);
            int lo = nq, hi = 0;
            for (int i = 0; i < nq; ++i) {
                bool any = false;
                for (int j = k0; j < k1; ++j) any |= keep(m, i + off, j);
                if (any) lo = std::min(lo, i), hi = i + 1;
            }
            bad_rows += hi > lo ? (r.first > lo || r.end < hi || r.first < lo / T * T || r.end > (hi + T - 1) / T * T)
                                : r.end > r.first;
            for (int r0 = r.first / T * T; r0 < r.end; r0 += T) {
                bool all = true;
                for (int i = r0; i < std::min(r0 + T, nq); ++i)
                    for (int j = k0; j < k1; ++j) all &= keep(m, i + off, j);
                const bool full = r0 >= r.all_first && std::min(r0 + T, nq) <= r.all_end;
                wrong_full += full && !all;
                missed_full += all && !full;
            }
            ++blocks;
        }
    }
    printf("%ld lists, %ld bad; %ld blocks, %ld bad rows, %ld wrongly full, %ld full but masked\n", lists, bad_lists,
           blocks, bad_rows, wrong_full, missed_full);
    return bad_lists || bad_rows || wrong_full || missed_full || lists < 10000 || blocks < 10000;
}
"""


def run(tmp_path, source):
    src, exe = tmp_path / "items.cu", tmp_path / "items"
    src.write_text(source)
    r = subprocess.run([build.NVCC, *build.ARCH, "-O2", "-std=c++17", "-I", build.CSRC, str(src),
                        "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return subprocess.run([str(exe)], capture_output=True, text=True)


@pytest.mark.skipif(not os.path.exists(build.NVCC), reason="needs nvcc")
def test_items_against_brute_force(tmp_path):
    r = run(tmp_path, SOURCE)
    assert r.returncode == 0, r.stdout


@pytest.mark.skipif(not os.path.exists(build.NVCC), reason="needs nvcc")
@pytest.mark.parametrize("right,wrong", [
    ("merge_lists(l0, l1, valid1, a, skip, end);", "merge_lists(l0, l1, valid1, a, skip, end); ++end;"),
    ("const BlockRows r = block_rows(", "const BlockRows r = block_rows(Mask{m.causal, m.window, 1 << 20, m.block}, k1, "
     "nq, first[0], end[0], first[1], end[1], end[2]), unused = block_rows(")])
def test_the_comparison_sees_a_wrong_list(tmp_path, right, wrong):
    assert SOURCE.count(right) == 1
    assert run(tmp_path, SOURCE.replace(right, wrong)).returncode == 1
