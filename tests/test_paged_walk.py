"""The walk along paged attention's stage list, compiled for the host (no GPU): places in the list, and that every
place lies inside the call's segments when lengths have changed since the list was counted."""
import os
import subprocess

import pytest

from rotated_quantized_kv_gb300 import build

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>
#include "tq_paged.cuh"
using namespace tqk;
using namespace tqk::paged;

// The list of sequence b as (h, rb, i, st), by counting.
struct Place { int h, rb, i, st, n_st, tokens; };
static std::vector<Place> all(const PagedList &l, const PagedClass &c, int b) {
    std::vector<Place> out;
    for (int h = 0; h < l.H; h++)
        for (int rb = 0; rb < c.n_rb; rb++)
            for (int i = 0; i < c.n; i++) {
                const int len = l.len[c.seg[i]][b], most = l.limit[c.seg[i]];
                const int tokens = len < 0 ? 0 : len > most ? most : len, n = (tokens + c.unit - 1) / c.unit;
                if ((c.heads[i] >> h) & 1)
                    for (int st = 0; st < n; st++) out.push_back({h, rb, i, st, n, tokens});
            }
    return out;
}

int main() {
    int right = 0, moved = 0, wrong = 0, outside = 0;
    std::srand(1);
    for (int run = 0; run < 4000; run++) {
        PagedList l;
        PagedClass c;
        std::memset(&l, 0, sizeof(l));
        std::memset(&c, 0, sizeof(c));
        l.B = 3, l.H = 1 + std::rand() % 16;
        c.n = 1 + (run % 3 ? 0 : std::rand() % 3), c.n_rb = 1 + std::rand() % 3, c.unit = 16 << std::rand() % 3;
        int len[3][3], later[3][3];
        for (int i = 0; i < c.n; i++) {
            c.seg[i] = static_cast<uint8_t>(i);
            c.heads[i] = static_cast<uint16_t>(1 + std::rand() % ((1 << l.H) - 1));
            l.limit[i] = 1000, l.len[i] = len[i];
            for (int b = 0; b < 3; b++) {
                len[i][b] = std::rand() % 1100 - 50;
                later[i][b] = std::rand() % 3 ? std::rand() % 1100 - 50 : std::rand() % 40;
            }
        }
        for (int b = 0; b < 3; b++) {
            const std::vector<Place> want = all(l, c, b);
            for (int at = 0; at < static_cast<int>(want.size()); at++) {
                const Walk w = seek(l, c, b, at);
                const Place &p = want[at];
                const bool ok = w.b == b && w.h == p.h && w.rb == p.rb && w.i == p.i && w.st == p.st && w.n_st == p.n_st &&
                                w.tokens == p.tokens && w.fresh;
                ok ? ++right : ++wrong;
            }
            for (int i = 0; i < c.n; i++) l.len[i] = later[i];
            for (int at = 0; at < static_cast<int>(want.size()); at++) {
                const Walk w = seek(l, c, b, at);
                const bool in = w.b == b && w.h >= 0 && w.h < l.H && w.rb >= 0 && w.rb < c.n_rb && w.i >= 0 && w.i < c.n && w.st >= 0 &&
                                w.st < w.n_st && w.tokens >= 0 && w.tokens <= 1000;
                in ? ++moved : ++outside;
            }
            for (int i = 0; i < c.n; i++) l.len[i] = len[i];
        }
    }
    std::printf("%d %d %d %d\n", right, wrong, moved, outside);
    return 0;
}
"""


@pytest.fixture(scope="module")
def counts(tmp_path_factory):
    d = tmp_path_factory.mktemp("walk")
    (d / "walk.cu").write_text(SOURCE)
    cmd = [build.nvcc(), *build.ARCH, "-std=c++17", "-I" + build.CSRC, "-o", str(d / "walk"), str(d / "walk.cu")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([os.path.join(d, "walk")], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0
    return [int(x) for x in r.stdout.split()]


def test_places(counts):
    assert counts[0] > 100000 and counts[1] == 0


def test_places_when_lengths_have_changed(counts):
    assert counts[2] > 100000 and counts[3] == 0
