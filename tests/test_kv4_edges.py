"""The 4-bit paged cache on the CPU: what the binding and the library refuse, or decide, on the host."""
import os
import subprocess

import pytest

import random_access_kv_fq_b200 as fq
from random_access_kv_fq_b200 import _lib, build
from tests import kv4_ref as ref
from tests.test_kv4 import _attn_args

torch = pytest.importorskip("torch")


def _call(**kw):
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    cache = torch.zeros(2, 2, 1, ref.unit_bytes(64, 32), dtype=torch.uint8)
    i = torch.zeros(2, dtype=torch.int32)
    return fq.fq_kv4_attn(q, cache, i[:, None], i, 32, **kw)


def test_query_counts_need_their_maximum():
    cu = torch.tensor([0, 1, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="max_q"):
        _call(cu_q=cu)
    for ok in (dict(cu_q=cu, max_q=2), dict(), dict(max_q=1)):  # as far as the tensors, which are not on a GPU
        with pytest.raises(ValueError, match="CUDA"):
            _call(**ok)


DRAIN = r"""
#include <cstdio>
#include <initializer_list>
#include <vector>
#include "kv4.h"

// An mbarrier as far as waits see it: a phase is over for a waiter if the current one's parity is not its own.
struct Bar {
  unsigned phases = 0, filled = 0;  // completed; times that the stage was filled
  bool try_wait(unsigned parity) const { return (phases & 1) != parity; }
};

int main() {
  // Probing both parities of a barrier says "done" of any barrier, and can wait for nothing.
  for (unsigned phases : {0u, 1u, 2u, 3u}) {
    Bar b;
    b.phases = phases;
    if (!b.try_wait(0) && !b.try_wait(1)) return 1;
  }
  // A ring of which the last copies, from any step on, are still in flight: each wait lets its own copy land.
  for (unsigned ring : {2u, 4u, 8u})
    for (unsigned issued = 0; issued <= 5 * ring; ++issued)
      for (unsigned landed = issued > ring ? issued - ring : 0; landed <= issued; ++landed) {
        std::vector<Bar> bars(ring);
        for (unsigned t = 0; t < issued; ++t) {
          ++bars[t % ring].filled;
          if (t < landed) ++bars[t % ring].phases;
        }
        unsigned waits = 0;
        fq::kv4::drain(issued > ring ? issued - ring : 0, issued, ring, [&](unsigned stage, unsigned parity) {
          if (!bars[stage].try_wait(parity)) ++bars[stage].phases, ++waits;
        });
        for (const Bar& b : bars)
          if (b.phases != b.filled) return 2;
        if (waits != issued - landed) return 3;
      }
  return 0;
}
"""


def _run_cpp(tmp_path, source):
    src, exe = tmp_path / "host.cpp", tmp_path / "host"
    src.write_text(source)
    subprocess.run([build.nvcc(), "-std=c++17", "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"), "-o", str(exe), str(src)],
                   check=True, timeout=300)
    return subprocess.run([str(exe)], timeout=60).returncode


def test_every_copy_in_flight_is_waited_for(tmp_path):
    assert _run_cpp(tmp_path, DRAIN) == 0


ITEMS = r"""
#include <random>
#include "kv4.h"

int main() {
  std::mt19937_64 rng(1);
  for (int i = 0; i < 2000000; ++i) {
    const int cost = 4 + (int)(rng() % (1u << (rng() % 27)));
    const int64_t items = 1 + (int64_t)(rng() % (1ull << (rng() % 31)));
    // anywhere, and at an item's two ends
    const int64_t n = (int64_t)(rng() % (uint64_t)items), at[] = {n * cost + (int64_t)(rng() % (uint64_t)cost), n * cost, n * cost + cost - 1};
    for (int64_t place : at)
      if (fq::kv4::item_of(place, cost) != n) return 1;
  }
  return 0;
}
"""


def test_a_place_on_the_line_is_in_its_item(tmp_path):
    assert _run_cpp(tmp_path, ITEMS) == 0


def test_sizes_that_the_attention_refuses_need_no_workspace():
    ws = fq.fq_kv4_attn_workspace_bytes
    assert ws(8192, 32, 8, 128, 1, 1 << 20, 1024) > 0 and ws(8, 1024, 8, 128, 1 << 20, 64, 16) > 0
    assert ws(8193, 32, 8, 128, 1, 64, 16) == 0 and ws(8, 32, 8, 128, 1, (1 << 20) + 1, 1024) == 0
    assert ws(8, 1024, 8, 128, (1 << 20) + 1, 64, 16) == 0


def test_more_query_heads_than_an_items_cost_is_counted_for_are_refused():
    for hq, status in ((1 << 20, 4), ((1 << 20) + 1, 2), (1 << 29, 2)):  # 4: taken, but for a missing workspace
        assert _lib.lib().fq_kv4_attn(*_attn_args(n_q=1, B=1, hq=hq, hkv=1, ws=None)) == status
        assert (fq.fq_kv4_attn_workspace_bytes(1, hq, 1, 64, 1, 4096, 16) > 0) == (status == 4)
