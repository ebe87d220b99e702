"""The eviction's selection (csrc/evict_select.cuh, the arithmetic that the kernel runs per thread), compiled for
the host and walked as the kernel walks it: ranks by 11, 11 and 10 bits, bins shared out to the threads of a block,
holes and movers counted.  Whatever the ranks, as many rows move as there are holes for them, and neither list is
longer than its place in the workspace."""
import ctypes
import subprocess
from pathlib import Path

import numpy as np
import pytest

CSRC = Path(__file__).resolve().parents[1] / "block_discrete_diffusion_tcgen05_b200" / "csrc"

WALK = r"""
#include <vector>
#include "evict_select.cuh"
using namespace e2d2;

template <int THREADS>
static int walk(const uint32_t* rank, int P, int keep, unsigned char* stay, int* holes, int* movers) {
    constexpr int BINS = kEvictBins / THREADS;
    *holes = *movers = 0;
    if (!evict_selects(P, keep)) {
        for (int j = 0; j < P; ++j) stay[j] = j < keep;
        return 0;
    }
    EvictPick t{0, static_cast<uint32_t>(keep), 0};
    int shift = 0;
    for (int pass = 0;; ++pass) {
        const int bits = evict_pass_bits(pass);
        shift = evict_pass_shift(pass);
        std::vector<uint32_t> hist(kEvictBins, 0);
        for (int j = 0; j < P; ++j)
            if (pass == 0 || (rank[j] >> (shift + bits)) == t.prefix) ++hist[(rank[j] >> shift) & ((1u << bits) - 1u)];
        uint32_t above = 0;
        int picked = 0;
        EvictPick next = t;
        for (int tid = 0; tid < THREADS; ++tid) {
            uint32_t mine[BINS], sum = 0;
            for (int i = 0; i < BINS; ++i) sum += mine[i] = hist[kEvictBins - 1 - BINS * tid - i];
            picked += evict_pick<BINS>(mine, above, sum, t.need, tid, bits, t.prefix, next);
            above += sum;
        }
        if (picked != 1) return 1;
        t = next;
        if (t.need == t.equal || shift == 0) break;
    }
    uint32_t before = 0;
    for (int j = 0; j < P; ++j) {
        const uint32_t leading = rank[j] >> shift;
        stay[j] = leading > t.prefix || (leading == t.prefix && (t.need == t.equal || before < t.need));
        before += leading == t.prefix;
        if (j < keep && !stay[j]) ++*holes;
        if (j >= keep && stay[j]) ++*movers;
    }
    return 0;
}

extern "C" int evict_walk(int threads, const uint32_t* rank, int P, int keep, unsigned char* stay, int* holes, int* movers) {
    return threads == 512 ? walk<512>(rank, P, keep, stay, holes, movers) : walk<1024>(rank, P, keep, stay, holes, movers);
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("evict")
    (d / "walk.cpp").write_text(WALK)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__host__=", "-D__device__=", "-I", str(CSRC),
                    str(d / "walk.cpp"), "-o", str(d / "walk.so")], check=True)
    fn = ctypes.CDLL(str(d / "walk.so")).evict_walk
    vp = ctypes.c_void_p
    fn.argtypes = [ctypes.c_int, vp, ctypes.c_int, ctypes.c_int, vp, vp, vp]

    def run(threads, rank, keep):
        rank = np.ascontiguousarray(rank, np.uint32)
        stay = np.full(len(rank), 2, np.uint8)
        holes, movers = ctypes.c_int(-1), ctypes.c_int(-1)
        assert fn(threads, rank.ctypes.data, len(rank), keep, stay.ctypes.data, ctypes.byref(holes), ctypes.byref(movers)) == 0
        return stay, holes.value, movers.value

    return run


def ranks(weight, pos, protect):
    """Larger for rows that stay: unsigned integers in the order of the floats, -0 as 0, NaN below every number,
    protected rows above all."""
    u = np.where(weight == 0, np.float32(0), weight).astype(np.float32).view(np.uint32)
    r = np.where(u & 0x80000000, ~u, u | 0x80000000).astype(np.uint32)
    r[np.isnan(weight)] = 0
    r[pos >= protect] = 0xFFFFFFFF
    return r


def check(walk, threads, rank, keep):
    P = len(rank)
    stay, holes, movers = walk(threads, rank, keep)
    order = np.lexsort((np.arange(P), -rank.astype(np.int64)))
    want = np.zeros(P, np.uint8)
    want[order[:keep]] = 1
    assert np.array_equal(stay, want), f"P {P} keep {keep}: {int(stay.sum())} rows stay"
    # the lists hold half of the rows that an entry can have, rounded up
    assert holes == movers <= (P // 2 + 4) // 4 * 4, f"P {P} keep {keep}: {holes} holes, {movers} movers"


@pytest.mark.parametrize("threads", [512, 1024])
@pytest.mark.parametrize("protected", ["all", "some", "one", "none"])
@pytest.mark.parametrize("keep", [0, 1, 2, 7, 149, 299, 300, 301])
def test_as_many_rows_move_as_there_are_holes(walk, threads, protected, keep):
    rng = np.random.default_rng(keep)
    for P in (1, 2, 63, 300):
        for weight in (np.exp(2 * rng.standard_normal(P)), np.zeros(P), rng.choice([0.0, -0.0, np.inf, -np.inf, np.nan, 1.0, 1e-42], P)):
            pos = np.arange(P)
            protect = {"all": 0, "some": P // 2, "one": P - 1, "none": P}[protected]
            check(walk, threads, ranks(weight.astype(np.float32), pos, protect), keep)


@pytest.mark.parametrize("threads", [512, 1024])
def test_ranks_that_differ_in_their_last_bits_alone(walk, threads):
    rng = np.random.default_rng(9)
    for base in (0, 0x80000000, 0xBF800000, 0xFFFFFC00):
        rank = (base + rng.integers(0, 900, 700)).astype(np.uint32)
        for keep in (0, 1, 350, 699):
            check(walk, threads, rank, keep)
