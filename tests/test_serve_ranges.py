"""The ranges schedule's arithmetic (the kernels' own header, compiled on the host): every step is
walked once, no two parts share a slot of the partials, the join finds each part where the walk
left it, and each item of a shared unit is joined once."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gqa_exact_attention_b200", "csrc_serve")

# Reads lines "grid min_blocks n steps..." (units' steps); answers each with what is wrong, or "ok".
PROG = r'''
#include <cstdio>
#include <map>
#include <string>
#include <vector>
#define __host__
#define __device__
#include "serve_ranges.h"
using namespace gqa;

std::string walk(int grid, int min_blocks, const std::vector<int>& steps) {
    std::vector<long long> begin{0};
    for (int s : steps) begin.push_back(begin.back() + s);
    const long long all = begin.back();
    const int ctas = range_ctas(all, min_blocks, grid);
    if (ctas < 1 || ctas > grid) return "ctas";
    if (range_start(all, ctas, 0) != 0 || range_start(all, ctas, ctas) != all) return "ends";
    std::vector<char> used(2 * grid, 0);                  // slots
    std::map<size_t, std::vector<int>> parts;             // slots of each shared unit's parts, in order
    std::map<size_t, std::vector<int>> joined;            // times that each item of it is joined
    const int items = 16, blocks = 4;
    size_t u = 0;
    for (int c = 0; c < ctas; ++c) {
        const long long x0 = range_start(all, ctas, c), x_end = range_start(all, ctas, c + 1);
        if (x_end <= x0) return "an empty range";
        if (ctas > 1 && x_end - x0 < min_blocks && all >= min_blocks) return "a short range";
        for (long long x = x0; x < x_end;) {
            while (x >= begin[u + 1]) ++u;
            if (range_cta(all, ctas, x) != c) return "the CTA of a step";
            const long long end = begin[u + 1] < x_end ? begin[u + 1] : x_end;
            const UnitShares s = unit_shares(all, ctas, begin[u], steps[u]);
            if (s.cta0 > c || s.cta0 + s.parts <= c) return "the unit's CTAs";
            const bool whole = x == begin[u] && end == begin[u + 1];
            if (whole != (s.parts == 1)) return "parts";
            if (!whole) {
                const int slot = piece_slot(c, x == x0);
                if (slot < 0 || slot >= 2 * grid || used[slot]++) return "a slot used twice";
                if (part_slot(s.cta0, s.first_slot, (int)parts[u].size()) != slot) return "where the join looks";
                parts[u].push_back(slot);
            }
            if (x == x0 && x > begin[u]) {  // a boundary inside the unit
                auto& j = joined[u];
                j.resize(items);
                for (int b = 0; b < blocks; ++b) {
                    const JoinShare m = join_share(items, c, s.cta0, s.parts, b, blocks);
                    for (int i = m.lo; i < m.hi; ++i) {
                        if (i < 0 || i >= items) return "an item out of range";
                        ++j[i];
                    }
                }
            }
            x = end;
        }
    }
    for (auto& [unit, slots] : parts) {
        if ((int)slots.size() != unit_shares(all, ctas, begin[unit], steps[unit]).parts) return "the number of parts";
        if (joined[unit].empty()) return "a unit that nobody joins";
        for (int n : joined[unit])
            if (n != 1) return "an item joined " + std::to_string(n) + " times";
    }
    if (joined.size() != parts.size()) return "a whole unit is joined";
    return "ok";
}

int main() {
    int grid, min_blocks, n;
    while (std::scanf("%d %d %d", &grid, &min_blocks, &n) == 3) {
        std::vector<int> steps(n);
        for (int& s : steps)
            if (std::scanf("%d", &s) != 1) return 1;
        std::puts(walk(grid, min_blocks, steps).c_str());
    }
    // products around 2^32 and far above against 128-bit arithmetic
    unsigned long long r = 88172645463325252ull, bad = 0;
    for (int i = 0; i < 2000000; ++i) {
        r ^= r << 13, r ^= r >> 7, r ^= r << 17;
        const int b = 1 + (int)((r >> 8) % 296);
        const long long near = (1ll << 32) / b + (long long)(r >> 20) % 5 - 2;
        const long long a = i & 1 ? near : (long long)(r >> (20 + i % 40));
        const long long c = (i % 3 == 0) ? 1 + (long long)(r >> (24 + i % 36)) : 1 + (long long)(r >> 10) % 300;
        if (mul_div(a, b, c) != (long long)((__int128)a * b / c)) ++bad;
    }
    std::printf("%llu\n", bad);
}
'''


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    at = tmp_path_factory.mktemp("ranges")
    (at / "t.cpp").write_text(PROG)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-I", CSRC, str(at / "t.cpp"), "-o", str(at / "t")], check=True)
    return str(at / "t")


def cases():
    r = random.Random(4)
    out = [(296, 2, [1]), (296, 2, [2]), (296, 2, [3, 1]), (1, 2, [5, 7]), (148, 1, [1] * 148), (148, 1, [1] * 149),
           (296, 2, [8192]), (296, 2, [1000000000]), (148, 2, [2 ** 31 - 1] * 40)]
    for _ in range(600):
        grid = r.choice([1, 2, 7, 148, 296])
        n = r.randint(1, 60)
        most = r.choice([1, 3, 20, 300, 20000])
        out.append((grid, r.choice([1, 2]), [r.randint(1, most) for _ in range(n)]))
    return out


def test_schedules(exe):
    given = cases()
    text = "\n".join(" ".join(map(str, (g, m, len(s), *s))) for g, m, s in given)
    got = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    assert got[len(given)] == "0", "mul_div"
    wrong = [(c, a) for c, a in zip(given, got) if a != "ok"]
    assert not wrong, wrong[:3]


@pytest.mark.parametrize("old,new", [
    ("(x + 1) * ctas - 1", "x * ctas"),                    # the CTA of a step
    ("== begin ? 0 : 1", "== begin ? 1 : 0"),              # the first part's slot
    ("2 * (cta0 + i)", "2 * (cta0 + i) + 1"),              # the others'
    ("(cta - cta0 - 1) * blocks", "(cta - cta0) * blocks"),  # the join's shares
    ("(uint32_t)ab / (uint32_t)c", "(uint32_t)ab / (uint32_t)c + (ab > 100)"),
])
def test_mistakes_are_found(tmp_path, old, new):
    """The walk finds a planted mistake of each function."""
    header = open(os.path.join(CSRC, "serve_ranges.h")).read()
    assert header.count(old) == 1
    (tmp_path / "serve_ranges.h").write_text(header.replace(old, new))
    (tmp_path / "t.cpp").write_text(PROG)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", str(tmp_path), str(tmp_path / "t.cpp"), "-o", str(tmp_path / "t")], check=True)
    given = cases()[:40]
    text = "\n".join(" ".join(map(str, (g, m, len(s), *s))) for g, m, s in given)
    got = subprocess.run([str(tmp_path / "t")], input=text, capture_output=True, text=True).stdout.split("\n")
    assert any(a != "ok" for a in got[:len(given)]) or got[-2:-1] != ["0"]
