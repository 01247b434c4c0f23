"""The plan of a prefix_attn call over its whole range of sizes, on the host:
compiled by itself with the undefined-behaviour sanitizer."""
import os
import subprocess

from kv_insert_gb300 import _build

MAIN = r"""
#include "prefix_plan.h"
#include <cstdio>
using namespace qkvf;

static uint64_t state = 12345;
static uint64_t next(uint64_t n)   // 0 .. n - 1
{
    state = state * 6364136223846793005ull + 1442695040888963407ull;
    return (state >> 33) % n;
}
static int log_size(int bits) { return (int)next((uint64_t(1) << next(bits + 1)) + 1); }   // 0 .. 2^bits, small ones often

int main()
{
    const int sms[] = {1, 2, 148, 152}, heads[] = {1, 2, 3, 4, 8, 16, 33, 64}, groups[] = {1, 2, 3, 5, 7, 8, 16, 33, 64};
    long checked = 0;
    for (long n = 0; n < 300000; ++n) {
        const int nkv = heads[next(8)], G = groups[next(9)], D = next(2) ? 64 : 128, sm = sms[next(4)];
        const int q = 1 + log_size(10) % 1024, R = n % 50 == 0 ? 0 : log_size(16) % 65536;
        if ((int64_t)R * q * nkv * G > (1 << 24)) continue;
        const int nb = log_size(24), mb = log_size(24);
        const PaPlan p = pa_plan(R, q, nkv * G, nkv, D, nb, mb, sm);
        const PaPlan s = pa_plan(R, q, nkv * G, nkv, D, (int)next(nb + 1), (int)next(mb + 1), sm);   // narrower tables
        const int64_t rows = (int64_t)R * q * nkv * G;
        for (const PaPlan &x : {p, s})
            if (x.sp < 1 || x.ss < 1 || x.sp > x.sp_max || x.ss > x.ss_max || x.sp_max > kPaMaxSplits ||
                x.ss_max > kPaMaxSplits || (int64_t)x.own_rows * x.own_tiles < (int64_t)q * G) {
                std::printf("plan of R %d q %d nkv %d G %d D %d nb %d mb %d sms %d\n", R, q, nkv, G, D, nb, mb, sm);
                return 1;
            }
        if (pa_workspace(s, rows, D) > pa_workspace(p, rows, D)) {
            std::printf("a narrower table needs more: R %d q %d nkv %d G %d D %d nb %d mb %d sms %d\n", R, q, nkv, G, D, nb, mb, sm);
            return 1;
        }
        ++checked;
    }
    std::printf("%ld plans\n", checked);
    return checked > 100000 ? 0 : 1;
}
"""


def test_plans(tmp_path):
    """No size divides by zero (a batch without requests among them) or
    overflows; splits stay within their bounds, and the workspace of some
    table widths serves narrower tables."""
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text("#include <initializer_list>\n" + MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(_build.PKG, "csrc"), "-o", str(exe), str(src)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
