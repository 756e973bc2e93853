"""The arithmetic of the paged decode step's work list (csrc/pp_paged_shares.cuh), compiled for the host with g++ and
checked on random lists: every job has one warp, every warp that takes part has a job, the division by which a warp finds
its first job agrees with the one by which the second kernel finds a job's warp, and no two records meet or pass the
workspace's end."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "shared_prefix_packed_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <random>
#include <vector>
#include "pp_paged_shares.cuh"
using namespace pp;
struct Item { int row, rows, qrows, nch, u0, j0; };
static int bad = 0;
static void need(bool ok, const char *what) { if (!ok && bad++ < 5) std::printf("%s\n", what); }
int main() {
    std::mt19937 rng(7);
    auto pick = [&](std::initializer_list<int> v) { return *(v.begin() + rng() % v.size()); };
    int lists = 0, cut_items = 0;
    for (int turn = 0; turn < 400; ++turn) {
        const int r = pick({1, 3, 4, 7, 8, 9, 16, 24}), hkv = pick({1, 2, 4}), hq = r * hkv;
        const int warps = pick({PD_WARPS, 2 * PD_WARPS, PD_MAX_CTAS * PD_WARPS});
        std::vector<Item> items;
        int r0 = 0, units = 0, jobs = 0;
        for (int g = 1 + int(rng() % 6); g; --g) {
            const int kg = rng() % 10;
            for (int place = 0; place <= kg; ++place) {
                const bool prefix = place == 0;
                const int qbase = prefix ? r0 : r0 + place - 1, qrows = (prefix ? kg : 1) * r, nch = pick({0, 1, 1, 2, 5, 30, 200});
                const int base = paged_row(prefix, r0, kg, qbase, hq);
                for (int head = 0; head < hkv; ++head)
                    for (int rho = 0; rho < qrows; rho += PD_RB) {
                        if (!nch) continue;
                        items.push_back({base + head * qrows + rho, qrows - rho < PD_RB ? qrows - rho : PD_RB, qrows, nch, units, jobs});
                        units += paged_item(nch, qrows);
                        jobs += nch;
                    }
            }
            r0 += kg;
        }
        if (!units) continue;
        ++lists;
        const PagedShare s(units, warps);
        need(s.many >= 1 && s.many <= warps && s.begin(0) == 0 && s.begin(s.many) == units, "the shares are all units");
        const PagedShare t(s.many, s.per, s.more);
        // the first job of a share, as a warp finds it
        auto from = [&](int u) {
            const int v = u < units ? u : units - 1;
            size_t i = 0;
            while (i + 1 < items.size() && items[i + 1].u0 <= v) ++i;
            return items[i].j0 + paged_job_from(v - items[i].u0 + (u >= units), paged_cost(items[i].qrows));
        };
        std::vector<int> count(s.many, 0), row_of(size_t(paged_rows(r0, hq)), -1);
        for (size_t i = 0; i < items.size(); ++i) {
            const Item &e = items[i];
            int before = -1;
            for (int k = 0; k < e.nch; ++k) {
                const int u = e.u0 + paged_start(k, e.qrows), w = t.warp_of(u);
                need(w >= 0 && w < s.many && s.begin(w) <= u && u < s.begin(w + 1), "a job's warp holds its first unit");
                need(k == 0 || w == before || w == before + 1, "an item's warps follow one another");
                need(from(u) == e.j0 + k && (paged_start(k, e.qrows) == 0 || from(u - 1) <= e.j0 + k), "the first job from a unit");
                if (w != before) {                          // a record
                    cut_items += k > 0;
                    for (int x = 0; x < e.rows; ++x) {
                        const size_t at = size_t(e.row) + size_t(w) * PD_RB + x;
                        need(at < row_of.size() && row_of[at] < 0, "records do not meet");
                        if (at < row_of.size()) row_of[at] = int(i);
                    }
                }
                before = w;
                ++count[w];
            }
            need(from(e.u0) == e.j0, "an item's first unit begins its first job");
        }
        for (int w = 0; w < s.many; ++w) need(count[w] > 0 && count[w] == from(s.begin(w + 1)) - from(s.begin(w)), "a warp's jobs");
    }
    std::printf("%d bad of %d lists, %d cuts\n", bad, lists, cut_items);
    return bad != 0 || lists < 300 || cut_items < 1000;
}
"""


def test_shares_and_records_of_the_decode_step(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ unavailable")
    src = tmp_path / "shares.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "shares"
    subprocess.run([gxx, "-std=c++17", "-O1", "-D__host__=", "-D__device__=", "-D__forceinline__=inline",
                    f"-I{CSRC}", str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
