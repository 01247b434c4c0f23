"""The dealing of chunk_attn's and key_weights' work (chunk_plan.h), on the host under
the undefined-behaviour sanitizer: every key step of every item is taken once,
in order, by parts of nearly equal cost, for drawn and extreme batches."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHECK = r"""
#include "chunk_plan.h"
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
using namespace qkvf;
#define NEED(c) do { if (!(c)) { printf("failed: %s (group %d parts %d)\n", #c, group, parts); exit(1); } } while (0)

// One batch: the parts' pieces in order against the list of all items
static void check(const std::vector<ChRequest> &reqs, int nkv, int group, int parts)
{
    const int R = (int)reqs.size();
    std::vector<int64_t> before(R + 1, 0);
    for (int r = 0; r < R; ++r) {
        int64_t sum = 0;
        const int blocks = ch_blocks(reqs[r].n, group);
        for (int b = 0; b < blocks; ++b) {
            if (b < 2000 || b == blocks - 1) NEED(ch_before(reqs[r], group, b) == sum || b >= 2000);
            sum += ch_cost(reqs[r], group, b);
        }
        NEED(blocks == 0 || sum == ch_request_cost(reqs[r], group));
        before[r + 1] = before[r] + nkv * ch_request_cost(reqs[r], group);
    }
    const int64_t total = before[R];
    NEED(total >= 0 && total < (int64_t(1) << 60));
    std::vector<ChPos> pos;
    for (int c = 0; c <= parts; ++c) {
        const int64_t u = ch_part(total, parts, c);
        NEED(u >= 0 && u <= total && (c < parts || u == total));
        ChPos at = {R, 0, 0, 0};
        for (int r = 0; r < R; ++r)
            if (u >= before[r] && u < before[r + 1]) at = ch_locate(reqs[r], group, r, u - before[r]);
        if (at.r < R) {
            NEED(at.g >= 0 && at.g < nkv && at.b >= 0 && at.b < ch_blocks(reqs[at.r].n, group));
            const int steps = ch_steps(ch_keys(reqs[at.r], group, at.b));
            NEED(at.k >= 0 && (steps == 0 ? at.k == 0 : at.k < steps));
        }
        NEED(c == 0 || ch_reached(at, pos.back()));
        pos.push_back(at);
    }
    ChPos want = {0, 0, 0, 0};   // the next step that nobody has taken
    const auto settle = [&] { while (want.r < R && reqs[want.r].n <= 0) want = {want.r + 1, 0, 0, 0}; };
    settle();
    for (int c = 0; c < parts; ++c) {
        ChPos at = pos[c];
        int first = 0, last = 0, count = 0;
        while (!ch_reached(at, pos[c + 1])) {
            if (reqs[at.r].n <= 0) {
                at = {at.r + 1, 0, 0, 0};
                continue;
            }
            ChPiece p;
            const ChRequest &q = reqs[at.r];
            if (!ch_take(q, group, nkv, at, pos[c + 1], p)) continue;
            NEED(ch_same_item(p.at, want) && p.at.k == want.k);
            NEED(p.k1 <= p.steps && p.k1 >= p.at.k);
            first += p.at.k > 0;
            last += p.at.k == 0 && p.k1 < p.steps;
            NEED(p.at.k == 0 || count == 0);   // only a part's first piece continues an item
            ++count;
            want.k = p.k1;
            if (p.k1 == p.steps) {
                want.k = 0;
                if (++want.b == ch_blocks(q.n, group)) {
                    want.b = 0;
                    if (++want.g == nkv) want = {want.r + 1, 0, 0, 0};
                }
                settle();
            }
        }
        NEED(first <= 1 && last <= 1);
    }
    NEED(want.r == R);
}

// The same for key_weights' blocks of keys
static void check_keys(const std::vector<ChRequest> &reqs, int nkv, int group, int parts)
{
    const int R = (int)reqs.size(), tokens = 128 / group > 0 ? 128 / group : 1, over = 3 * tokens;
    std::vector<int64_t> before(R + 1, 0);
    for (int r = 0; r < R; ++r) {
        int64_t sum = 0;
        if (reqs[r].n >= 0 && reqs[r].L > 0) {
            const int blocks = kw_blocks(reqs[r]);
            for (int b = 0; b < blocks; ++b) {
                if (b < 2000 || b == blocks - 1) NEED(kw_before(reqs[r], b, over) == sum);
                NEED(kw_seen(reqs[r], b) >= 0 && kw_seen(reqs[r], b) <= reqs[r].n);
                sum += kw_cost(reqs[r], b, over);
            }
        }
        NEED(sum == kw_request_cost(reqs[r], over));
        before[r + 1] = before[r] + nkv * sum;
    }
    const int64_t total = before[R];
    std::vector<ChPos> pos;
    for (int c = 0; c <= parts; ++c) {
        const int64_t u = ch_part(total, parts, c);
        ChPos at = {R, 0, 0, 0};
        for (int r = 0; r < R; ++r)
            if (u >= before[r] && u < before[r + 1]) at = kw_locate(reqs[r], r, u - before[r], tokens, over);
        if (at.r < R) {
            NEED(at.g >= 0 && at.g < nkv && at.b >= 0 && at.b < kw_blocks(reqs[at.r]));
            const int steps = kw_steps(reqs[at.r], at.b, tokens);
            NEED(at.k >= 0 && (steps == 0 ? at.k == 0 : at.k < steps));
        }
        NEED(c == 0 || ch_reached(at, pos.back()));
        pos.push_back(at);
    }
    ChPos want = {0, 0, 0, 0};
    const auto none = [&](int r) { return reqs[r].n < 0 || reqs[r].L <= 0; };
    const auto settle = [&] { while (want.r < R && none(want.r)) want = {want.r + 1, 0, 0, 0}; };
    settle();
    for (int c = 0; c < parts; ++c) {
        ChPos at = pos[c];
        int count = 0;
        while (!ch_reached(at, pos[c + 1])) {
            if (none(at.r)) {
                at = {at.r + 1, 0, 0, 0};
                continue;
            }
            ChPiece p;
            const ChRequest &q = reqs[at.r];
            if (!kw_take(q, tokens, nkv, at, pos[c + 1], p)) continue;
            NEED(ch_same_item(p.at, want) && p.at.k == want.k && p.k1 <= p.steps);
            NEED(p.at.k == 0 || count == 0);
            ++count;
            want.k = p.k1;
            if (p.k1 == p.steps) {
                want.k = 0;
                if (++want.b == kw_blocks(q)) {
                    want.b = 0;
                    if (++want.g == nkv) want = {want.r + 1, 0, 0, 0};
                }
                settle();
            }
        }
    }
    NEED(want.r == R);
}

int main()
{
    std::mt19937 rng(7);
    const auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    for (int i = 0; i < 3000; ++i) {
        std::vector<ChRequest> reqs;
        const int R = pick(0, 12), most = 1 << pick(0, 12);
        for (int r = 0; r < R; ++r) {
            const int n = pick(0, 3) ? pick(0, most) : 1;
            reqs.push_back({0, n, pick(0, 5) ? n + pick(0, 1 << pick(0, 17)) : pick(0, n)});
        }
        check(reqs, pick(1, 9), pick(1, 64), pick(0, 1) ? 152 : pick(1, 300));
        for (auto &q : reqs)
            if (!pick(0, 5)) q.n = pick(-1, 0);
        check_keys(reqs, pick(1, 9), pick(1, 64), pick(0, 1) ? 152 : pick(1, 300));
    }
    const int far = 1 << 24;
    check({{0, far, far}}, 1, 1, 152);
    check({{0, far, far}}, 64, 1, 152);
    check({{0, 1 << 18, far}}, 4, 64, 152);
    check({{0, 1, far}}, 64, 64, 152);
    check({{0, 1, 1}}, 1, 1, 152);
    check({{0, far, 0}}, 2, 3, 152);
    check({{0, far, 1 << 10}}, 1, 5, 7);
    check(std::vector<ChRequest>(65535, ChRequest{0, 1, far}), 64, 64, 152);
    check(std::vector<ChRequest>(65535, ChRequest{0, 1, 1}), 1, 1, 152);
    check_keys({{0, far, far}}, 64, 1, 152);
    check_keys({{0, 1, far}}, 64, 64, 152);
    check_keys({{0, 0, far}, {0, 1 << 18, far}}, 1, 64, 152);
    check_keys({{0, far, 300}, {0, 256, 512}, {0, 0, 256}}, 1, 1, 152);
    puts("ok");
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="no g++")
def test_plan_on_the_host(tmp_path):
    src = tmp_path / "check.cpp"
    src.write_text(CHECK)
    exe = tmp_path / "check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I",
                    os.path.join(ROOT, "kv_insert_gb300", "csrc"), "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and out.stdout.strip().endswith("ok"), out.stdout + out.stderr


OVERLAP = r"""
#include "chunk_plan.h"
#include <algorithm>
#include <cstdio>
#include <vector>
using namespace qkvf;

// Starts that go up and down, 0, T, 0, T ...: every other request holds all T tokens, and each of them passes by
// itself.  Their costs add up past 64 bits; every part still starts at a place within a request.
static int check(int R, ChRequest q, int nkv, int group)
{
    std::vector<int64_t> before(R + 1, 0);
    for (int r = 0; r < R; ++r)
        before[r + 1] = ch_add(before[r], r % 2 ? 0 : nkv * ch_request_cost(q, group));
    const int64_t total = before[R];
    if (total <= 0 || !std::is_sorted(before.begin(), before.end())) return 1;
    ChPos last = {0, 0, 0, 0};
    for (int c = 0; c <= 152; ++c) {
        const int64_t off = ch_part(total, 152, c);
        ChPos at = {R, 0, 0, 0};
        if (off < total) {
            const int r = (int)(std::upper_bound(before.begin(), before.end(), off) - before.begin()) - 1;
            if (r < 0 || r >= R || r % 2) return 2;
            at = ch_locate(q, group, r, off - before[r]);
            const int steps = ch_steps(ch_keys(q, group, at.b));
            if (at.g < 0 || at.g >= nkv || at.b < 0 || at.b >= ch_blocks(q.n, group) || at.k < 0 || at.k >= steps) return 3;
        }
        if (!ch_reached(at, last)) return 4;
        last = at;
    }
    return 0;
}

int main()
{
    const int far = 1 << 24;
    const int bad = check(65535, {0, far, far}, 1, 64) + check(65535, {0, far, far}, 64, 1) + check(65535, {0, 1 << 18, far}, 64, 64) +
                    check(3, {0, far, far}, 1, 64) + check(2, {0, 1, 1}, 1, 1);
    puts(bad ? "failed" : "ok");
    return bad;
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="no g++")
def test_starts_that_overlap(tmp_path):
    """A sum of costs beyond 64 bits would send a part to a negative place in its table."""
    src = tmp_path / "overlap.cpp"
    src.write_text(OVERLAP)
    exe = tmp_path / "overlap"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I",
                    os.path.join(ROOT, "kv_insert_gb300", "csrc"), "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr
