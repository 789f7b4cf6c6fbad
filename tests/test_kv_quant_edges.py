"""Properties of the 4-bit key/value cache's sources and binding that no device is
needed for."""
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "token_skipping_sparse_step_b200", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_kernels_that_start_early_do_not_read_by_the_read_only_path():
    """What a kernel reads after griddepcontrol.wait was written while it lived."""
    waiting = []
    for name in sorted(os.listdir(CSRC)):
        if not re.match(r"(kv|attention)_quant.*\.cuh$", name):
            continue
        code = _code(name)
        if "grid_dependency_wait" not in code:
            continue
        waiting.append(name)
        assert not re.search(r"__ldg\s*\(|\.global\.nc\b", code), name
        assert not re.search(r"\bconst\s+\w+\s*\*\s*__restrict__", code), name
    assert waiting == ["attention_quant_rows.cuh", "attention_quant_tc.cuh", "kv_quant.cuh"]


WALK = r"""
#include "copy_window.h"
#include <cstdio>
#include <cstdlib>
#include <set>
#include <algorithm>
// The walk of the expanding warps: K of chunk j + 1 is waited for, its stage may not come free, nor V's of chunk j;
// when both are expanded, the chunk's ring stage takes the copy of chunk j + stages. It gives up at its wait number
// `at`. Prints what is in flight then, and what is drained.
int main(int argc, char** argv) {
  const int nc = atoi(argv[1]), stages = atoi(argv[2]), at = atoi(argv[3]);
  esd::CopyWindow w;
  std::set<int> flying;
  auto copy = [&](int j) { w.start(j); flying.insert(j); };
  int waits = 0;
  auto wait = [&] { return waits++ != at; };
  for (int j = 0; j < std::min(stages, nc); ++j) copy(j);
  bool ok = true;
  for (int j = -1; j < nc && ok; ++j) {
    if (j + 1 < nc) {
      if (!(ok = wait())) break;
      w.land(j + 1);
      flying.erase(j + 1);
      if (j + 1 >= 2 && !(ok = wait())) break;
    }
    if (j >= 0) {
      if (j >= 2 && !(ok = wait())) break;
      if (j + stages < nc) copy(j + stages);
    }
  }
  printf("%d\n", (int)ok);
  for (int j : flying) printf("%d ", j);
  printf("\n");
  w.drain([](int j) { printf("%d ", j); });
  printf("\n");
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("walk")
    (d / "walk.cpp").write_text(WALK)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(d / "walk.cpp"), "-o", str(d / "walk")], check=True)
    return str(d / "walk")


@pytest.mark.parametrize("stages", [2, 3])
@pytest.mark.parametrize("nc", [1, 2, 3, 7])
def test_a_walk_that_gives_up_waits_for_the_copies_in_flight_and_no_others(walk, nc, stages):
    gave_up = 0
    for at in range(3 * nc + 2):
        ok, flying, drained = subprocess.run([walk, str(nc), str(stages), str(at)], capture_output=True, text=True,
                                             check=True).stdout.split("\n")[:3]
        assert flying == drained, (nc, stages, at)
        gave_up += ok == "0"
    assert gave_up >= nc
    # the kernel keeps its copies in the same window
    code = _code("attention_quant_tc.cuh")
    assert "copies.start(j)" in code and "copies.land(jk)" in code and "copies.drain(" in code and "landed" not in code


class _Rows:
    """A tensor of a device that is not here, as far as the checks look."""
    dtype = torch.bfloat16

    def __init__(self, device):
        self.device = device

    def numel(self):
        return 1 << 20

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True


@pytest.mark.parametrize("device", [0, 1])
def test_a_cache_on_another_device_than_the_context_is_refused(device):
    """Its kernels would follow the other device's addresses, on that device's stream."""
    import token_skipping_sparse_step_b200 as esd
    ctx = object.__new__(esd.Context)
    ctx._head_dim, ctx._d, ctx._dtype, ctx._dev = 128, 512, torch.bfloat16, 0
    cache = esd.KVQuant.empty(2, 8, 4, 128, device="cpu")
    cache._dev = device
    rows = _Rows(device)
    if device == 0:
        ctx._check_rows(cache, 2, "k, v", 100, rows, rows, (None, 8))
    else:
        with pytest.raises(ValueError, match="context"):
            ctx._check_rows(cache, 2, "k, v", 100, rows, rows, (None, 8))


def test_a_ring_stage_is_refilled_only_when_what_was_read_of_it_is_written():
    """A copy (asynchronous proxy) is not ordered behind loads whose values nobody has used yet."""
    code = _code("attention_quant_tc.cuh")
    step = code[code.index("auto step = [&]"):]
    step = step[:step.index("constexpr int kSc")]
    reads, written, refill = step.rindex("lds128("), step.index("expand(aV"), step.index("copy(j + kStages)")
    assert reads < written < refill
    expand = code[code.index("auto expand = [&]"):]
    expand = expand[:expand.index("bool ok = true")]
    assert expand.index("sts128(") < expand.index("fence.proxy.async.shared::cta") < expand.index("__syncwarp()")


def test_the_barriers_of_the_first_copies_are_fenced_for_them():
    """They are started by the thread that set the barriers up, ahead of any barrier of the block."""
    code = _code("attention_quant_tc.cuh")
    init, first = code.index("mbar_init(rawfull"), code.index("min(kStages, nc); ++j) copy(j)")
    assert init < code.index("fence.proxy.async.shared::cta", init) < first
