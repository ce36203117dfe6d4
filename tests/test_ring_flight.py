"""The row rings' account of copies on their way (csrc/ring_flight.cuh), compiled for the host and driven
in the order of the forward and of the backward ring kernels, with copies that land late or never.

The stages' mbarriers are played by a struct that knows when a phase is armed a second time."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <vector>
#include "ring_flight.cuh"

struct Stage { int phase = 0; bool armed = false; int copy = -1; };

// rows: copies to post; stuck: the copy that does not land before the loop is over (-1: none); apart: the
// iteration whose wait for the other blocks runs out, or in which another group's wait does (-1: none);
// ahead: the loop waits for the next row (the backward with both gradients); heed: post only while the
// block's flag is down.
// 0: right; 1: a phase was armed twice; 2: the drain waits for a phase that nothing completes;
// 3: a copy is left out of the drain; 4: an undisturbed run drains or leaves copies out.
extern "C" int run(int rows, int stages, int stuck, int apart, int ahead, int heed) {
    std::vector<Stage> st(stages);
    bl::RingFlight f;
    f.reset();
    const int64_t t0 = 3, step = 5;                // row number n is row t0 + n * step
    bool flag = false;                             // the block's abort flag
    int next = 0;                                  // the next copy to post
    bool twice = false;
    auto post = [&] {
        Stage& s = st[next % stages];
        twice = twice || s.armed;
        s.armed = true;
        s.copy = next++;
    };
    auto wait = [&](int n) {                       // lands what can land; true if copy n is there
        Stage& s = st[n % stages];
        if (s.armed && s.copy == n && n != stuck) {
            s.armed = false;
            ++s.phase;
        }
        return s.phase > n / stages;
    };
    while (next < stages && next < rows) post();
    if (ahead && rows > 0 && !wait(0)) flag = true;
    for (int n = 0; n < rows; ++n) {
        bool landed = true;
        if (!ahead) landed = wait(n);
        else if (n + 1 < rows) landed = wait(n + 1);
        if (!landed || n == apart) flag = true;
        if (n + stages < rows) {
            if (!flag || !heed) post();
            else f.stop(t0 + n * step);
        }
        if (twice) return 1;
    }
    std::vector<bool> waited(rows, false);
    int calls = 0;
    bool bad = false;
    if (flag) f.drain(stages, t0, step, t0 + (rows - 1) * step + 1, [&](int q, unsigned parity) {
        ++calls;
        // what try_wait.parity can find: this phase still open with a copy that will land, or just over
        const Stage& s = st[q];
        const bool open = (unsigned(s.phase) & 1u) == parity && s.armed;
        const bool over = (unsigned(s.phase) & 1u) != parity;
        if (!open && !over) bad = true;
        if (open) waited[s.copy] = true;
    });
    if (bad) return 2;
    for (const Stage& s : st)
        if (s.armed && !waited[s.copy]) return 3;
    if (stuck < 0 && apart < 0 && (calls != 0 || next != rows)) return 4;
    return 0;
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    src, so = d / "ring.cpp", d / "ring.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "bit_ternary_qat_b200", "csrc"), str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so)).run


@pytest.mark.parametrize("ahead", [0, 1])
def test_account(run, ahead):
    for stages in range(1 + ahead, 5):
        for rows in range(0, 15):
            assert run(rows, stages, -1, -1, ahead, 1) == 0
            for stuck in range(rows):
                assert run(rows, stages, stuck, -1, ahead, 1) == 0, (rows, stages, stuck)
                for apart in range(rows):
                    assert run(rows, stages, stuck, apart, ahead, 1) == 0, (rows, stages, stuck, apart)
            for apart in range(rows):
                assert run(rows, stages, -1, apart, ahead, 1) == 0, (rows, stages, apart)


@pytest.mark.parametrize("ahead", [0, 1])
def test_posting_on_is_found(run, ahead):
    """Without heed to the flag a stuck copy's stage is armed again."""
    assert run(12, 3, 4, -1, ahead, 0) == 1
