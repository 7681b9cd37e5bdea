"""The named barriers of the tile attention's softmax warps in a host model:
with waits for products that run out at any moment, every warp still ends and
no barrier's phase counts a warp twice or mixes the vote with the hand-over."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_weight_quantized_w4a8_gb300", "csrc")

MODEL = """
#include <cstdint>
#include <random>

// Named barriers as the PTX manual has them: a phase ends when `expected`
// warps have arrived; who waits (or reduces) goes on then.
struct Barrier {
    int arrived = 0, phase = 0;
    uint32_t who = 0;
    int kinds = 0;      // 1: reduction, 2: sync or arrive
    bool any = false, result[2] = {false, false};
};

// The slot's eight warps through `jobs` jobs, scheduled at random.  A job of a
// warp: wait for its S (given by the first warp after the hand-over before, until a
// wait has run out somewhere), vote, sync after a vote that says so, hand over.
// 0: all ended; 1: a warp counted twice in a phase; 2: vote and hand-over in one
// phase; 3: nobody can go on.
extern "C" int run(int vote, int hand, int jobs, int fail_after, unsigned seed) {
    std::mt19937 rng(seed);
    constexpr int W = 8;
    Barrier bars[16];
    int job[W] = {}, step[W] = {}, wait_phase[W] = {};
    bool up_result[W] = {}, ok[W];
    for (bool& o : ok) o = true;
    int products = 1;        // S of the jobs below is there
    bool failed = false;     // the abort flag
    long ticks = 0;
    auto arrive = [&](int id, int w, int kind, bool pred) -> int {
        Barrier& b = bars[id];
        if (b.who >> w & 1) return 1;
        if (b.kinds && b.kinds != kind) return 2;
        b.who |= 1u << w;
        b.kinds = kind;
        b.any |= pred;
        if (++b.arrived == W) {
            b.result[b.phase & 1] = b.any;
            b.arrived = 0, b.who = 0, b.kinds = 0, b.any = false, ++b.phase;
        }
        return 0;
    };
    for (;;) {
        int can[W], n = 0, done = 0;
        for (int w = 0; w < W; ++w) {
            if (job[w] == jobs) { ++done; continue; }
            bool go = true;
            if (step[w] == 0) go = !ok[w] || products > job[w] || failed;
            if (step[w] == 2 || step[w] == 4) go = bars[vote].phase != wait_phase[w];
            if (step[w] == 6) go = bars[hand].phase != wait_phase[w];
            if (go) can[n++] = w;
        }
        if (done == W) return 0;
        if (ticks++ == fail_after) { failed = true; continue; }
        if (n == 0) {
            if (!failed) { failed = true; continue; }  // the bounded waits run out
            return 3;
        }
        const int w = can[rng() % n];
        int bad = 0;
        switch (step[w]) {
            case 0:  // the wait for S: with the flag up it may still have come in time
                if (ok[w] && products <= job[w]) ok[w] = false;
                else if (failed && rng() % 2) ok[w] = false;
                step[w] = 1;
                break;
            case 1:
                wait_phase[w] = bars[vote].phase;
                bad = arrive(vote, w, 1, ok[w] && rng() % 4 == 0);
                step[w] = 2;
                break;
            case 2:
                up_result[w] = bars[vote].result[wait_phase[w] & 1];
                step[w] = up_result[w] ? 3 : 5;
                break;
            case 3:
                wait_phase[w] = bars[vote].phase;
                bad = arrive(vote, w, 2, false);
                step[w] = 4;
                break;
            case 4: step[w] = 5; break;
            case 5:
                if (w == 0 && failed && rng() % 4 == 0) ok[w] = false;  // its own waits before the hand-over
                if (w == 0 && failed && rng() % 2) break;               // take their time
                wait_phase[w] = bars[hand].phase;
                bad = arrive(hand, w, 2, false);
                if (w == 0) step[w] = 6;
                else step[w] = 0, ++job[w];
                break;
            case 6:
                if (ok[w]) products = job[w] + 2;
                step[w] = 0, ++job[w];
                break;
        }
        if (bad) return bad;
    }
}
extern "C" int vote_of(int slot) { return w4a8::bar_vote(slot); }
extern "C" int hand_of(int slot) { return w4a8::bar_hand(slot); }
extern "C" int queries() { return w4a8::kBarQueries; }
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    d = tmp_path_factory.mktemp("roles")
    (d / "roles.cpp").write_text('#include "%s"\n' % os.path.join(CSRC, "kvq_roles.h") + MODEL)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-shared", "-fPIC",
                    "-o", str(d / "roles.so"), str(d / "roles.cpp")], check=True)
    return ctypes.CDLL(str(d / "roles.so"))


def outcomes(model, vote, hand):
    return {model.run(vote, hand, jobs, after, seed) for jobs in (1, 2, 7) for after in (0, 5, 17, 40, 90, 10 ** 6)
            for seed in range(300)}


@pytest.mark.parametrize("slot", [0, 1])
def test_every_warp_ends_whatever_runs_out(model, slot):
    assert outcomes(model, model.vote_of(slot), model.hand_of(slot)) == {0}


def test_the_model_finds_a_shared_barrier(model):
    """One barrier for both, as a check of the model: sound only while nothing
    runs out."""
    assert all(model.run(1, 1, 7, 10 ** 6, seed) == 0 for seed in range(300))
    assert outcomes(model, 1, 1) - {0}


def test_barriers_are_distinct_and_are_the_kernels(model):
    ids = [0, model.queries()] + [f(s) for f in (model.vote_of, model.hand_of) for s in (0, 1)]  # 0: the whole CTA
    assert len(set(ids)) == len(ids) and max(ids) < 16
    used = re.findall(r"named_bar_(\w+)\((.*?), kS", open(os.path.join(CSRC, "kvq_tree.cu")).read())
    assert sorted(used) == [("arrive", "bar_hand(slot)"), ("or", "bar_vote(slot)"), ("sync", "bar_hand(slot)"),
                            ("sync", "bar_vote(slot)"), ("sync", "kBarQueries")]
