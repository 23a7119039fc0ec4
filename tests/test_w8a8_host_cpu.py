"""Arithmetic of the W8A8 kernels and their launches, compiled alone for the
host (csrc/w8a8_plan.h) and checked over its whole range."""
import glob
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_w4a4_quantized_token_b200", "csrc")


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    """Compiles and runs a C++ program beside the header; returns what it prints."""
    where = tmp_path_factory.mktemp("w8a8")

    def compiled(body):
        src, exe = where / "main.cpp", where / "main"
        src.write_text('#include "w8a8_plan.h"\n#include <cstdio>\n#include <vector>\nusing namespace svdq;\n' + body)
        subprocess.check_call([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o",
                               str(exe), str(src)])
        return subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=120).stdout

    return compiled


DRAIN = """
// The ring as the kernel runs it, one barrier per place that counts its finished phases, up to the row whose wait
// runs out: its copy and the later ones are in flight then.
int main() {
    long cases = 0, bad = 0;
    for (int stages = 2; stages <= 8; ++stages)
        for (int step = 1; step <= 148; step += 49)
            for (int first = 0; first < step; first += 16)
                for (int M = first + 1; M < first + 40 * step; M += 1 + step / 3)
                    for (int fail = 0; first + fail * step < M; ++fail) {
                        std::vector<int> done(stages, 0), fill(stages, -1);   // finished phases; copy in flight
                        int ahead = first, n = 0;
                        const auto fetch = [&](int s) {
                            fill[s] = n++;
                            ahead = ahead + (long)step < M ? ahead + step : M;
                        };
                        for (int s = 0; s < stages && ahead < M; ++s) fetch(s);
                        int s = 0;
                        for (int i = 0; i < fail; ++i, s = (s + 1) % stages) {
                            ++done[s], fill[s] = -1;                          // row i has landed and is read
                            if (ahead < M) fetch(s);
                        }
                        std::vector<int> waits(stages, 0);
                        drain_ring(first, step, first + fail * step, ahead, stages, [&](int place, unsigned parity) {
                            ++waits[place];
                            // a wait for the phase that is under way, and not one that returns at once
                            if (fill[place] < 0 || parity != (unsigned)(done[place] & 1)) ++bad;
                        });
                        for (int p = 0; p < stages; ++p) bad += waits[p] != (fill[p] >= 0);
                        ++cases;
                    }
    const int big = 2147483647;   // the largest number of rows
    int waits = 0;
    drain_ring(147, 148, 147 + 148 * 14510000, big, 8, [&](int, unsigned) { ++waits; });
    std::printf("%ld cases, %ld bad, %d\\n", cases, bad, waits);
}
"""


def test_drain_waits_for_the_copies_in_flight_and_no_others(run):
    """After a timeout at any row of any ring: one wait for each copy in flight, in its own phase."""
    out = run(DRAIN).split()
    assert int(out[0]) > 50000 and out[2] == "0", out
    rows = -(-(2147483647 - 147) // 148)
    assert int(out[4]) == rows - 14510000


PLAN = """
// Plans of random shapes (sizes spread over their logarithm) on several chips.
int main() {
    const W8Chip chips[] = {{{148, 74, 33, 15}}, {{148, 74, 30, 12}}, {{132, 66, 28, 12}}, {{160, 80, 40, 20}}};
    unsigned long long seed = 1;
    const auto uniform = [&] { return (double)((seed = seed * 6364136223846793005ull + 1442695040888963407ull) >> 11) / 9007199254740992.0; };
    const auto spread = [&](double hi, int64_t step) {
        int64_t v = 1;
        for (double x = uniform(); x > 0.0 && (double)v < hi; x -= 0.02) v = v + v / 2 + 1;
        v = v - (int64_t)(uniform() * (double)(v / 3));
        return std::max(step, std::min((int64_t)hi, v / step * step));
    };
    long plans = 0, narrow = 0, split = 0, bad = 0;
    for (int i = 0; i < 300000; ++i) {
        const int64_t M = spread(2147483647.0, 1), N = spread(2147483640.0, 8), K = spread(131056.0, 16);
        const int64_t chunks = (K + 127) / 128;
        for (const W8Chip& chip : chips)
            for (int mode = 0; mode < 3; ++mode) {
                const W8Plan p = w8_plan(M, N, K, chip, mode);
                ++plans;
                if (mode == 2 && !p.pair) ++bad;
                if (mode == 1 && p.pair && (M + 127) / 128 <= 65535 && (N + 127) / 128 <= 65535) ++bad;
                if (p.pair) continue;
                ++narrow;
                const int64_t mt = (M + p.nt - 1) / p.nt, nt = (N + p.tile_n - 1) / p.tile_n;
                int l = 0;
                while ((1 << l) < p.split) ++l;
                bad += p.nt != 16 && p.nt != 32 && p.nt != 64 && p.nt != 128;
                bad += p.tile_n < 64 || p.tile_n > 128 || p.tile_n % 8 != 0;
                bad += mt > 65535 || nt > 65535;
                bad += (1 << l) != p.split || p.split > 8 || p.split > chunks;
                // every stage of a CTA's share in one ring place, or places shared evenly by two warps
                const int64_t most = ((chunks + p.split - 1) / p.split + w8n::per(p.nt) - 1) / w8n::per(p.nt);
                bad += p.stages < 1 || p.stages > w8n::kMaxStages || (p.stages == 1 ? most != 1 : p.stages % 2 != 0);
                bad += w8n::fixed_bytes(p.nt, p.split) + p.stages * w8n::stage_bytes(p.nt) > kW8SmemBudget;
                // no cluster waits for another to end
                if (p.split > 1) ++split, bad += mt * nt > chip.clusters[l];
            }
    }
    std::printf("%ld plans, %ld narrow, %ld split, %ld bad\\n", plans, narrow, split, bad);
}
"""


def test_plans_fit_the_chip(run):
    """Grid limits, ring depths, shared memory, and split tiles that are all resident at once, on chips whose clusters
    fit in other numbers."""
    out = run(PLAN).split()
    assert out[6] == "0" and int(out[2]) > 100000 and int(out[4]) > 10000, out


def test_every_wait_site_has_a_number_of_its_own():
    """The device status word names a wait by one byte: two kernels with the same number could not be told apart."""
    sites = {}
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        for name, number in re.findall(r"\b(kSite\w+) = (\d+)", open(path).read()):
            sites.setdefault(int(number), set()).add(name)
    assert len(sites) > 30 and all(0 < n < 256 for n in sites)
    assert all(len(names) == 1 for names in sites.values()), {n: s for n, s in sites.items() if len(s) > 1}
