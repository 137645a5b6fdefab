"""Host memory that runs out inside a block-manager call: the call returns PA_ERR_NO_MEMORY, no
exception leaves the C interface, and nothing has changed.  Every allocation of every call fails
once (the manager compiled beside a counting operator new)."""
from __future__ import annotations

import os
import subprocess

from paged_kv_cache_348_b200 import build as pbuild

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <new>
#include <vector>
#include "pagedkv.h"

static long budget = -1;                 // allocations left, -1: no limit
void* operator new(std::size_t n) {
  if (budget == 0) throw std::bad_alloc();
  if (budget > 0) --budget;
  if (void* p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}
void* operator new(std::size_t n, const std::nothrow_t&) noexcept {
  try { return operator new(n); } catch (...) { return nullptr; }
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

static const int kBlocks = 600, kBs = 4, kSeqs = 64;

// everything the interface shows of a manager
static std::vector<long> state(pa_block_manager* bm) {
  const long keep = budget;
  budget = -1;
  std::vector<long> v;
  v.push_back(pa_bm_free_blocks(bm));
  for (int b = 0; b < kBlocks; ++b) v.push_back(pa_bm_refcount(bm, b));
  std::vector<int32_t> row(kBlocks);
  for (int32_t s = 0; s < kSeqs; ++s) {
    int32_t len = -1;
    v.push_back((long)pa_bm_context_len(bm, s));
    v.push_back(pa_bm_num_blocks_of(bm, s));
    const int r = pa_bm_block_tables(bm, &s, 1, kBlocks, -9, row.data(), &len);
    v.push_back(r);
    if (r == PA_OK) v.insert(v.end(), row.begin(), row.end());
  }
  budget = keep;
  return v;
}

static int failures = 0, injected = 0;
// the call with its 1st, 2nd, ... allocation failing until it goes through
static void each(const char* what, pa_block_manager* bm, const std::function<int()>& call) {
  const std::vector<long> before = state(bm);
  for (long k = 0; k < 10000; ++k) {
    budget = k;
    const int r = call();
    budget = -1;
    if (r == PA_OK) return;
    ++injected;
    if (r != PA_ERR_NO_MEMORY || state(bm) != before) {
      std::printf("%s: allocation %ld: status %d, %s\n", what, k, r,
                  state(bm) == before ? "unchanged" : "CHANGED");
      ++failures;
      return;
    }
  }
  std::printf("%s: never went through\n", what);
  ++failures;
}

int main() {
  pa_block_manager* bm = nullptr;
  std::vector<int32_t> order(kBlocks);
  for (int i = 0; i < kBlocks; ++i) order[i] = kBlocks - 1 - i;
  for (long k = 0;; ++k) {
    budget = k;
    const int r = pa_bm_create(kBlocks, kBs, order.data(), &bm);
    budget = -1;
    if (r == PA_OK) break;
    ++injected;
    if (r != PA_ERR_NO_MEMORY || bm) { std::printf("create %ld: %d\n", k, r); return 1; }
  }
  int32_t ids[kSeqs], n = 0;
  auto alloc = [&](int t) { each("allocate", bm, [&] { return pa_bm_allocate(bm, t, &ids[n]); }); ++n; };
  auto fork = [&](int s) { each("fork", bm, [&] { return pa_bm_fork(bm, ids[s], &ids[n]); }); ++n; };
  for (int i = 0; i < 12; ++i) alloc(5 * i);
  fork(11), fork(11), fork(8);
  std::vector<int64_t> slots(400);
  std::vector<int32_t> cow(800), seqs;
  int nc = 0;
  for (int i = 0; i < 200; ++i) seqs.push_back(ids[i % n]);
  each("append", bm, [&] {
    return pa_bm_append_tokens(bm, seqs.data(), (int)seqs.size(), slots.data(), cow.data(), &nc);
  });
  int dropped = 0;
  each("drop_window", bm, [&] { return pa_bm_drop_window(bm, ids[11], 9, 4, &dropped); });
  fork(11);
  std::vector<int32_t> blocks(kBlocks), tables(8 * kBlocks);
  int nb = 0;
  each("swap_out", bm, [&] { return pa_bm_swap_out(bm, ids[11], blocks.data(), &nb); });
  each("swap_in", bm, [&] { return pa_bm_swap_in(bm, ids[11], blocks.data(), &nb); });
  const int32_t some[4] = {ids[11], ids[12], ids[10], ids[3]}, lens[4] = {20, 31, 7, 0};
  each("compact", bm, [&] { return pa_bm_compact(bm, some, lens, 4, kBlocks, -1, tables.data()); });
  const int32_t plan[4] = {ids[12], ids[13], ids[8], ids[14]};
  std::vector<int32_t> pre(4), mem(64), pl(4), ctx(4);
  int chunks = 0, width = 0;
  each("bm_plan_cascade", bm, [&] {
    return pa_bm_plan_cascade(bm, plan, 4, 4, 0, pre.data(), mem.data(), pl.data(), &chunks, &width);
  });
  pa_bm_block_tables(bm, plan, 4, kBlocks, -1, tables.data(), ctx.data());
  each("plan_cascade", bm, [&] {
    return pa_plan_cascade(tables.data(), kBlocks, ctx.data(), 4, kBs, 4, 0, pre.data(), mem.data(),
                           pl.data(), &chunks, &width);
  });
  each("release", bm, [&] { return pa_bm_release(bm, ids[12]); });
  budget = 0;                             // giving everything back needs no memory
  for (int i = 0; i < n; ++i)
    if (i != 12 && pa_bm_release(bm, ids[i]) != PA_OK) ++failures;
  budget = -1;
  if (pa_bm_free_blocks(bm) != kBlocks) { std::printf("blocks lost\n"); ++failures; }
  pa_bm_destroy(bm);
  std::printf("injected %d failures %d\n", injected, failures);
  return failures != 0;
}
"""


def test_every_allocation_may_fail(tmp_path):
    src, exe = tmp_path / "driver.cpp", tmp_path / "driver"
    src.write_text(DRIVER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-I", os.path.join(pbuild.ROOT, "include"),
                    "-o", str(exe), str(src), os.path.join(pbuild.CSRC, "block_manager.cpp")],
                   check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    assert int(r.stdout.split("injected ")[1].split()[0]) > 40, r.stdout
