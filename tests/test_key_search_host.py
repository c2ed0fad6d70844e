"""The search for a row's largest logits (csrc/key_search.h) on the host, with
the kernel's gathering around it: what is left of a row, in whatever order it
comes, are its largest, after no more rounds than the code allows; with NaN
among the logits too, which count as -infinity."""
import os
import shutil
import subprocess

import pytest

from row_reduction_norm_gb300 import build as B

PROGRAM = r"""
#include "key_search.h"
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <functional>
#include <limits>
#include <random>
#include <vector>

using std::vector;
constexpr float kLow = -std::numeric_limits<float>::infinity();

static uint64_t key_of(float x, int place) {
    x = x != x ? kLow : x + 0.f;
    uint32_t u;
    std::memcpy(&u, &x, 4);
    u = u & 0x80000000u ? ~u : u | 0x80000000u;
    return (uint64_t)u << 32 | (uint32_t)~place;
}

static uint64_t nth(vector<uint64_t> v, int top) {
    std::sort(v.rbegin(), v.rend());
    return v[top - 1];
}

enum Order { kInPlace, kBackwards, kShuffled, kUnkind, kOrders };

// Rounds until the row's `top` largest are left, or -1 where others are, or none within `most`.
static int search(const vector<float> &x, int warps, int vec, int top, Order order, std::mt19937 &rng, int most) {
    const int n = (int)x.size(), room = warps < 2 ? 256 : 128 * warps, threads = 32 * warps;
    // which thread saw an element: units of 32 lanes x 8 chunks, a warp each in turn
    auto thread_of = [&](int i) { return i / (256 * vec) % warps * 32 + i / vec % 32; };
    vector<float> seen(threads, kLow);
    for (int i = 0; i < n; ++i)
        if (!(x[i] != x[i])) seen[thread_of(i)] = std::max(seen[thread_of(i)], x[i]);
    vector<float> of_group(32, kLow);
    for (int t = 0; t < threads; ++t) of_group[t % 32] = std::max(of_group[t % 32], seen[t]);
    vector<float> sorted = of_group;
    std::sort(sorted.rbegin(), sorted.rend());
    const float bound = sorted[top - 1];
    const bool lowest = bound == kLow;
    rrn::KeySearch s;
    s.start(key_of(bound, 0) >> 32, key_of(sorted[0], 0) >> 32);
    vector<uint64_t> want;
    for (int i = 0; i < n; ++i) want.push_back(key_of(x[i], i));
    std::partial_sort(want.begin(), want.begin() + top, want.end(), std::greater<>());
    want.resize(top);
    for (int round = 0; round < most; ++round) {
        vector<uint64_t> keys;
        for (int i = 0; i < n; ++i) {
            if (seen[thread_of(i)] < bound || !rrn::reaches(x[i], bound, lowest)) continue;
            if (s.round > 0 && key_of(x[i], i) < s.least) continue;
            keys.push_back(key_of(x[i], i));
        }
        for (uint64_t k : keys)
            if (k < s.least) return -1;
        if (order == kBackwards) std::reverse(keys.begin(), keys.end());
        if (order == kShuffled) std::shuffle(keys.begin(), keys.end(), rng);
        if (order == kUnkind) {   // the lowest first, and so dealt out that a group of 32 has the lowest alone
            std::sort(keys.begin(), keys.end());
            if ((int)keys.size() > room) {
                vector<uint64_t> dealt(keys.begin(), keys.begin() + room);
                const int each = room / 32;
                for (int g = 0; g < 32; ++g)
                    for (int i = 0; i < each; ++i) dealt[i * 32 + g] = keys[g * each + i];
                std::copy(dealt.begin(), dealt.end(), keys.begin());
            }
        }
        const int found = (int)keys.size(), held = std::min(found, room);
        vector<uint64_t> best(32, 0);
        for (int i = 0; i < held; ++i) best[i % 32] = std::max(best[i % 32], keys[i]);
        if (s.enough(found, room, top)) {
            const uint64_t higher = found > 96 ? nth(best, top) : 0;
            vector<uint64_t> left;
            for (uint64_t k : keys)
                if (k >= higher) left.push_back(k);
            std::sort(left.rbegin(), left.rend());
            if ((int)left.size() < top) return -1;
            left.resize(top);
            return left == want ? round + 1 : -1;
        }
        s.next(found, room, nth(best, top));
    }
    return -1;
}

int main(int argc, char **argv) {
    const int most = rrn::kSampledRounds + 64;
    std::mt19937 rng(5);
    std::normal_distribution<float> normal(0.f, 3.f);
    std::uniform_real_distribution<double> uniform(0., 1.);
    int worst = 0, wrong = 0;
    auto run = [&](const char *what, const vector<float> &x, int warps, int vec) {
        for (int top : {1, 5, 20, 32})
            for (int order = 0; order < kOrders; ++order) {
                if (top > (int)x.size()) continue;
                const int rounds = search(x, warps, vec, top, (Order)order, rng, most);
                worst = std::max(worst, rounds);
                if (rounds < 0) {
                    ++wrong;
                    std::printf("%s: %zu logits, %d warps, %d a chunk, top %d, order %d\n", what, x.size(), warps, vec, top, order);
                }
            }
    };
    for (int vec : {4, 8})
        for (int warps : {1, 8})
            for (int n : {33, 256 * vec, 12000}) {
                if (warps == 1 && n > 256 * vec) continue;
                for (double share : {0., .1, .2, .5, .9, .999, 1.}) {
                    vector<float> x(n), y(n), z(n);
                    for (int i = 0; i < n; ++i) {
                        const bool off = uniform(rng) < share;
                        x[i] = off ? NAN : normal(rng);
                        y[i] = off ? NAN : uniform(rng) < .5 ? kLow : std::round(normal(rng));
                        z[i] = off ? NAN : kLow;
                    }
                    run("numbers and NaN", x, warps, vec);
                    run("numbers, masks and NaN", y, warps, vec);
                    run("masks and NaN", z, warps, vec);
                }
                // groups of threads without a large logit, whose bound nearly all reach
                for (int less : {1, 5, 20, 32}) {
                    vector<float> up(n), down(n), mixed(n), equal(n);
                    for (int i = 0; i < n; ++i) {
                        const bool few = i / vec % 32 >= less - 1;
                        up[i] = few ? -1.f : i * 1e-4f;
                        down[i] = few ? -1.f : (n - i) * 1e-4f;
                        mixed[i] = few ? NAN : (float)((long)i * 7919 % n) - n / 2;
                        equal[i] = few ? NAN : 1.f;
                    }
                    run("rising", up, warps, vec);
                    run("falling", down, warps, vec);
                    run("mixed", mixed, warps, vec);
                    run("equal", equal, warps, vec);
                }
            }
    std::printf("%d wrong, %d rounds at most\n", wrong, worst);
    return 0;
}
"""


def test_the_search_ends_with_the_largest(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not installed")
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-I", B.CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert out.startswith("0 wrong, "), out[:2000]


def test_the_kernel_gathers_by_these_rules():
    """Every element that is gathered passed `reaches`, and no other bound is kept beside the search's."""
    with open(os.path.join(B.CSRC, "logprobs_kernels.cuh"), encoding="utf-8") as f:
        text = f.read()
    body = text[text.index("KeySearch search;"):text.index("their order, by counting the larger ones")]
    assert "reaches(x[k], bound, lowest)" in body and "search.enough(" in body and "search.next(" in body
    assert "!(x[k] < bound)" not in body
