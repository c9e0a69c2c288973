"""The flags of the grouped products' joins, on the host: csrc/joinflag.h compiled
with the C++ compiler, every order of the two sides' steps in every outcome of a
launch, and which flags the kernel's two sides visit (read from the source).

A captured launch has the same epoch on every replay.  So a launch has to leave
its flags at 0 also where a wait ran out: one left at the epoch would hand the
next replay the sums of an earlier one."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rmsnorm_linear_projection_gb300", "csrc")

HARNESS = r"""
#include <cstdio>
#include <initializer_list>
#include "joinflag.h"
using namespace rnl;

// A side is a list of steps on one flag; a step is one access to memory.
//   'P' exchange in the epoch, 'G' exchange in the mark of having given up,
//   'c' the store of 0 that follows an exchange that came second,
//   'W' a look at the flag: goes on to '0' (store 0) if it holds the epoch, else may
//       look again or give up (both are tried)
static const uint64_t E = 0x123456789abcdef0ull;
static int bad = 0, ends = 0, took = 0;

struct Side { char step; bool clear; };   // what comes next; clear: the exchange came second

static void run(uint64_t flag, Side give, Side take, bool published, int looks) {
  if (give.step == 0 && take.step == 0) {
    ++ends;
    if (flag != 0) ++bad;                 // nothing stays
    return;
  }
  if (give.step == 'P' || give.step == 'G') {
    const uint64_t v = give.step == 'P' ? E : join_gave_up(E);
    run(v, {join_is_second(flag, E) ? 'c' : '\0', false}, take, published || give.step == 'P', looks);
  } else if (give.step == 'c') {
    run(0, {0, false}, take, published, looks);
  }
  if (take.step == 'W') {
    if (flag == E) {
      if (!published) ++bad;              // took sums that nobody handed over
      run(flag, give, {'0', false}, published, looks);
    } else if (looks > 0) {
      run(flag, give, {'W', false}, published, looks - 1);
    }
    run(flag, give, {'G', false}, published, looks);  // gives up, for another wait's sake too
  } else if (take.step == '0') {
    ++took;
    run(0, give, {0, false}, published, looks);
  } else if (take.step == 'G') {
    run(join_gave_up(E), give, {join_is_second(flag, E) ? 'c' : '\0', false}, published, looks);
  } else if (take.step == 'c') {
    run(0, give, {0, false}, published, looks);
  }
}

int main() {
  // what the flag holds in front: 0 (a launch before), anything else (a new workspace)
  const uint64_t before[] = {0, 1, 0xA5A5A5A5A5A5A5A5ull, E - 1, E + 1, join_gave_up(E - 1), join_gave_up(E + 1)};
  for (uint64_t b : before)
    for (char g : {'P', 'G'}) run(b, {g, false}, {'W', false}, false, 2);
  printf("%d %d %d\n", ends, bad, took);
  return 0;
}
"""


def test_no_order_of_the_two_sides_leaves_a_flag(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "join.cpp", tmp_path / "join"
    src.write_text(HARNESS)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    ends, bad, took = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert ends > 50 and took > 0 and bad == 0


def test_every_way_out_of_the_epilogue_visits_the_flags():
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "grouped.cu")).read())
    epilogue = text[text.index("const int ew = warp - 2"):]
    epilogue = epilogue[:epilogue.index("if (*abort)")]
    # the one way out of the items in front of their end, and what stands behind the loop for it
    breaks = [m.start() for m in re.finditer(r"\bbreak;", epilogue)]
    assert len(breaks) == 1 and "return" not in epilogue
    behind = epilogue[breaks[0]:]
    assert re.search(r"if \(it < walk\.n\)\s+give_up_joins<", behind) and epilogue.count("give_up_joins<") == 1
    # partial sums are handed over by a visit, too
    assert "flag_release" not in epilogue and epilogue.count("join_visit(") == 1
    helper = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "grouped.cuh")).read())
    helper = helper[helper.index("void give_up_joins("):]
    helper = helper[:helper.index("\n}\n")]
    # the flag of the worker's own partial sums, and those of the parts that it joins
    assert helper.count("join_visit(") == 2 and helper.count("join_gave_up(epoch)") == 2
