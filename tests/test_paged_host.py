"""Arithmetic that the paged attention kernels share with the host, compiled and run here.  No GPU is needed."""
import os
import subprocess

from rag_kv_cache_rope_gb300 import build as B

SHARES = r"""
#include <stdio.h>
#include "paged.cuh"
using blend::Shares;
// A line of `total` units in items of `len` (the last one shorter): every unit belongs to one part, a share
// has at most one part that enters it and one that leaves it, and an item that begins in a share is found
// from the share's start.  Walking every item from its first share to its last covers the line.
static int check(int total, int len, int grid, int min_quota, int max_snap) {
    int quota = Shares::parts(total, grid);
    if (quota < min_quota) quota = min_quota;
    const Shares sh(total, quota, max_snap < quota ? max_snap : quota);
    if (sh.n < 1 || sh.n > grid) return 1;
    int at_share = 0;
    for (long long i = 0; i < total; i += len) {
        const int i0 = (int)i, i1 = (int)(i + len < total ? i + len : total);
        const int f = sh.first(i0, i1), l = sh.last(i0, i1);
        if (f < at_share || l < f || l >= sh.n) return 2;
        int at = 0;
        for (int b = f; b <= l; ++b) {
            if (sh.start(b) < 0 || sh.start(b) >= i1) return 3;
            if (sh.begin(b, i0, i1) != at || sh.end(b, i0, i1) <= at || sh.end(b, i0, i1) > i1 - i0) return 4;
            at = sh.end(b, i0, i1);
        }
        if (at != i1 - i0) return 5;
        at_share = l;
    }
    return 0;
}
int main(void) {
    const int totals[] = {1, 2, 303, 304, 305, 9999, 1 << 20, 2147000000, 2147483343, 2147483344, 2147483646, 2147483647};
    const int lens[] = {1, 7, 8, 9, 100, 65537, (1 << 20) - 1, 1 << 20, 2147483647};
    const int grids[] = {456, 304, 76, 1}, snaps[] = {1, 4, 8};
    for (int t : totals)
        for (int len : lens)
            for (int g : grids)
                for (int snap : snaps) {
                    if (t / len > (1 << 20)) continue;
                    const int rc = check(t, len, g, snap / 2 + 1, snap);
                    if (rc) {
                        printf("total %d items of %d grid %d snap %d: %d\n", t, len, g, snap, rc);
                        return 1;
                    }
                }
    return 0;
}
"""


def run_host(tmp_path, source):
    src, exe = tmp_path / "probe.cu", tmp_path / "probe"
    src.write_text(source)
    subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", "-I", B.CSRC, "-I", os.path.join(B.ROOT, "include"), str(src),
                    "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_shares_cover_the_line_up_to_the_largest_total(tmp_path):
    run_host(tmp_path, SHARES)


CAPPED = r"""
#include "paged.cuh"
int main(void) {
    const int cap = blend::PAGED_MAX_UNITS, half = (1 << 30) - 1;
    if (blend::add_capped(3, 4, cap) != 7 || blend::add_capped(cap - 2, 1, cap) != cap - 1) return 1;
    if (blend::add_capped(cap - 1, 1, cap) != cap || blend::add_capped(cap, cap, cap) != cap) return 2;
    if (blend::add_capped(half - 1, 1, half) != half || blend::add_capped(half, half, half) != half) return 3;
    return 0;
}
"""


def test_capped_sums(tmp_path):
    run_host(tmp_path, CAPPED)
