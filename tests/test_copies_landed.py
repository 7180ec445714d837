"""Copies in flight when a kernel gives up (GDN_DEVERR_TIMEOUT), without a GPU: the loading threads of the
linear attention kernels wait for their own copies whatever ended their work.  The waits' bookkeeping
(wait_copies, gdn_tc.cuh) is compiled for the host and run against barriers with mbarrier phases, and that
each loading role ends in it is read from the source."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decode_gated_gb300",
                    "csrc")
INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")

PROGRAM = r"""
#include <cstdio>
#include "gdn_tc.cuh"

// A barrier of one arrival a phase, and the ring's uses of it whose copies have not landed.
struct Bar { unsigned phase = 0; unsigned in_flight = 0; };

template <unsigned NS>
int run() {
    for (unsigned issued = 0; issued < 3 * NS + 2; ++issued)
        for (unsigned late = 0; late <= NS && late <= issued; ++late) {  // the last `late` uses' copies are in flight
            Bar bars[NS];
            for (unsigned p = 0; p < issued; ++p) {
                if (p + late < issued) ++bars[p % NS].phase;   // landed
                else ++bars[p % NS].in_flight;                 // (a slot has one use in flight at most)
            }
            bool right = true;
            gdn::wait_copies<NS>(issued, [&](unsigned slot, unsigned parity) {
                Bar &b = bars[slot];
                if ((b.phase & 1) != parity) return;           // that phase has completed
                if (!b.in_flight) right = false;               // nothing would ever complete it
                --b.in_flight, ++b.phase;
            });
            for (const Bar &b : bars) right = right && b.in_flight == 0;
            if (!right) { printf("NS %u issued %u late %u\n", NS, issued, late); return 1; }
        }
    return 0;
}

int main() { return run<1>() || run<2>() || run<3>() || run<4>(); }
"""


def test_waits_cover_the_copies_in_flight(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    source, program = tmp_path / "copies.cu", tmp_path / "copies"
    source.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "--extended-lambda", "-gencode", "arch=compute_103a,code=sm_103a", "-I", CSRC,
                    "-I", INCLUDE, str(source), "-o", str(program)], check=True)
    done = subprocess.run([str(program)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout


def body(source, head):
    """The text of the function, or block, whose opening brace follows `head`."""
    at = source.index("{", source.index(head))
    depth = 0
    for i in range(at, len(source)):
        depth += {"{": 1, "}": -1}.get(source[i], 0)
        if depth == 0:
            return source[at:i + 1]
    raise AssertionError(head)


def test_the_drafts_loading_role_ends_in_the_wait():
    with open(os.path.join(CSRC, "gdn_linear_drafts.cu")) as f:
        role = body(f.read(), "void load_role(")
    assert "return" not in role
    assert re.search(r"wait_copies<[^;]*issued[^;]*full[^;]*;\s*\}\);\s*\}$", role)
    # a use counts from when its barrier is armed, the last one (no unit) among them
    assert role.index("wait(bar(s.free") < role.index("++issued") < role.index("arrive(full)")


def test_the_prompts_loading_thread_waits_before_it_leaves():
    with open(os.path.join(CSRC, "gdn_linear_tc.cu")) as f:
        kernel = body(f.read(), "linear_tc_kernel(const __grid_constant__ Launch L)")
    after = kernel[kernel.index("load_role<OUT>("):]
    wait = body(after, "for (uint32_t p = issued > 2 ? issued - 2 : 0; p < issued + (s.dead ? 1 : 0); ++p)")
    assert "return" not in after[:after.index("for (")]
    for name in "qkv":
        assert f"wait_parity(bar(s.b.{name}_full[p & 1]), (p >> 1) & 1)" in wait
