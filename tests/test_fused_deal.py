"""CPU: how tiles of the products with fused epilogues are dealt out (csrc/fused_deal.h, which the kernel and the
host share): every block of k is done once, and what the joining launch reads of a tile are its parts, each written
once, in the order of k."""
import os
import shutil
import subprocess

import pytest

import mixed_precision_matmul_gb300._build as _build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <vector>

#include "fused_deal.h"

using namespace mpg;

static long g_split = 0, g_parts = 0, g_behind = 0, g_fewer = 0;

#define REQUIRE(x) do { if (!(x)) { std::printf("%s: whole %d workers %d dealers %d tiles %d x %d, %d x %d\n", #x, p.whole_tiles, \
  workers, p.dealers, p.prod[0].num_tiles, p.prod[0].num_k_blk, p.prod[1].num_tiles, p.prod[1].num_k_blk); std::exit(1); } } while (0)

static void product(FusedProduct& x, int m_blk, int n_blk, int kb) {
  x.num_m_blk = m_blk;
  x.num_n_blk = n_blk;
  x.num_k_blk = kb;
  x.num_tiles = m_blk * n_blk;
  x.group_m = 8;
  x.kb_second = x.mb_second = INT32_MAX;
}

// The walks of all workers and the joins of all tiles.
template <bool kMore>
static void run(FusedGemmParams& p, int workers, bool both) {
  p.units_first = (int64_t)(p.prod[0].num_tiles - p.whole_tiles) * p.prod[0].num_k_blk;
  p.units = p.units_first + (both ? (int64_t)p.prod[1].num_tiles * p.prod[1].num_k_blk : 0);
  REQUIRE(p.dealers <= workers && p.units >= p.dealers && (p.units > 0) == (p.dealers > 0));
  struct Part { int which, tile, kb0, kb1, written; };
  std::map<int, Part> slots;
  std::vector<int> done[2];
  std::vector<int> number[2];                     // of the tile at (mb, nb)
  for (int i = 0; i < 2; ++i) {
    const FusedProduct& x = p.prod[i];
    done[i].assign((size_t)x.num_tiles * x.num_k_blk, 0);
    number[i].assign((size_t)x.num_tiles, -1);
    for (int t = 0; t < x.num_tiles; ++t) {
      const FusedTile c = fused_tile(x, t);
      int& n = number[i][(size_t)(c.mb * x.num_n_blk + c.nb)];
      REQUIRE(n == -1);
      n = t;
    }
  }
  for (int w = 0; w < workers; ++w) {
    FusedItems items(p, w, workers);
    FusedItem x;
    while (items.next<kMore>(p, x)) {
      const FusedProduct& pr = p.prod[x.which];
      const int tile = number[x.which][(size_t)(x.mb * pr.num_n_blk + x.nb)];
      REQUIRE(x.kb0 >= 0 && x.kb0 < x.kb1 && x.kb1 <= pr.num_k_blk);
      for (int k = x.kb0; k < x.kb1; ++k) ++done[x.which][(size_t)tile * pr.num_k_blk + k];
      if (x.slot >= 0) {
        REQUIRE(!slots.count(x.slot) && x.slot < 2 * workers);
        slots[x.slot] = Part{x.which, tile, x.kb0, x.kb1, 1};
      } else {
        REQUIRE(x.kb0 == 0 && x.kb1 == pr.num_k_blk);
      }
    }
  }
  for (int i = 0; i < 2; ++i)
    for (int n : done[i]) REQUIRE(n == 1);
  size_t read = 0;
  if (p.units)
    for (int i = 0; i < (both ? 2 : 1); ++i)
      for (int t = i ? 0 : p.whole_tiles; t < p.prod[i].num_tiles; ++t) {
        const int kb = p.prod[i].num_k_blk;
        const int64_t u0 = i ? p.units_first + (int64_t)t * kb : (int64_t)(t - p.whole_tiles) * kb;
        const FusedParts parts(p, u0, u0 + kb);
        REQUIRE(parts.count >= 1);
        if (parts.count == 1) continue;           // (done by one worker: no slot, or the count below is off)
        int at = 0;
        for (int j = 0; j < parts.count; ++j, ++read) {
          const auto s = slots.find(parts.slot(j));
          REQUIRE(s != slots.end());
          REQUIRE(s->second.which == i && s->second.tile == t && s->second.kb0 == at);
          at = s->second.kb1;
        }
        REQUIRE(at == kb);
        ++g_split;
      }
  REQUIRE(read == slots.size());
  g_parts += (long)read;
  if (p.whole_tiles && p.dealers) ++g_behind;
  if (p.whole_tiles && p.dealers && p.units < workers) ++g_fewer;
}

int main() {
  FusedGemmParams p;
  // one product: all small numbers of tiles, blocks and workers, split or not
  for (int most = 1; most <= 13; ++most)
    for (int m = 1; m <= 9; ++m)
      for (int n = 1; n <= 5; ++n)
        for (int kb = 1; kb <= 26; ++kb)
          for (int split = 0; split < 2; ++split) {
            std::memset(static_cast<void*>(&p), 0, sizeof(p));
            product(p.prod[0], m, n, kb);
            const int tiles = m * n, rest = tiles % most;
            if (split && (!rest || kb < 2)) continue;
            p.whole_tiles = split ? tiles - rest : tiles;
            p.dealers = split ? (int)dealers_of(rest, (int64_t)rest * kb, most) : 0;
            run<false>(p, p.whole_tiles ? (tiles < most ? tiles : most) : p.dealers, false);
          }
  // two products whose blocks are all dealt out
  for (int most = 1; most <= 12; ++most)
    for (int a = 1; a <= 9; ++a)
      for (int b = 1; b <= 9; ++b)
        for (int ka = 4; ka <= 20; ++ka)
          for (int kb = 4; kb <= ka; kb += 3) {
            std::memset(static_cast<void*>(&p), 0, sizeof(p));
            product(p.prod[0], a, 1, ka);
            product(p.prod[1], 1, b, kb);
            const int64_t units = (int64_t)a * ka + (int64_t)b * kb;
            p.dealers = (int)std::min<int64_t>(most, std::max<int64_t>(units / kMinUnits, 1));
            run<true>(p, p.dealers, true);
          }
  // two products, the second's whole tiles behind (and beside the last round of) the first's
  for (int most = 1; most <= 12; ++most)
    for (int a = 1; a <= 30; ++a)
      for (int b = 1; b <= 40; b += 3)
        for (int ratio = 1; ratio <= 4; ++ratio) {
          std::memset(static_cast<void*>(&p), 0, sizeof(p));
          product(p.prod[0], a, 1, 6 * ratio);
          product(p.prod[1], 1, b, 6);
          p.whole_tiles = a;
          const int busy = a % most, idle = busy ? most - busy : 0;
          p.late = busy;
          p.late_workers = idle;
          p.late_rounds = std::min(idle ? ratio : 0, idle ? (b + idle - 1) / idle : 0);
          run<true>(p, std::min(most, a + b), false);
        }
  // the choice itself, on 152 CTAs and 76 pairs: sizes with fewer blocks behind whole rounds than workers
  const struct { FusedEpi epi; int64_t m, n, k; bool second_k; } sizes[] = {
      {FusedEpi::kGated, 64, 9856, 2048, false},   {FusedEpi::kGated, 256, 9856, 4096, false},
      {FusedEpi::kGated, 2183, 2131, 2420, false}, {FusedEpi::kGatedGrad, 64, 9856, 2048, false},
      {FusedEpi::kStats, 64, 19500, 2048, false},  {FusedEpi::kStats, 120, 58752, 2304, false},
      {FusedEpi::kStats, 1092, 93248, 2752, false}, {FusedEpi::kProb, 64, 19500, 2048, false},
      {FusedEpi::kPlain, 1792, 2816, 1536, true},  {FusedEpi::kPlain, 2816, 1790, 3001, false}};
  long behind = 0;
  auto choose = [&](const FusedLaunch& l, int64_t tile) {
    const int64_t most = tile == 256 ? 76 : 152;
    const FusedDeal d = deal(l, tile, most, true);
    const FusedShape s = shape_of(l, tile);
    std::memset(static_cast<void*>(&p), 0, sizeof(p));
    product(p.prod[0], (int)s.mb, (int)s.nb, (int)(s.units / s.tiles));
    p.whole_tiles = (int)d.whole;
    p.dealers = (int)d.dealers;
    const long before = g_behind;
    run<false>(p, (int)d.workers, false);
    behind += g_behind > before;
    // the slots fit into what the workspace has for them
    if (d.dealers && (size_t)(2 * d.dealers * tile * tile) * sizeof(float) > fused_slot_bytes(l)) std::exit(2);
  };
  for (const auto& x : sizes)
    for (int64_t tile : {128, 256}) {
      FusedLaunch l;
      l.epi = x.epi; l.m = x.m; l.n = x.n; l.k = x.k; l.second_k = x.second_k;
      choose(l, tile);
    }
  for (int64_t m = 17; m < 2500; m = m * 5 / 4 + 3)
    for (int64_t n = 64; n < 30000; n = n * 6 / 5 + 7)
      for (int64_t k = 64; k < 9000; k = k * 3 / 2 + 5)
        for (FusedEpi e : {FusedEpi::kPlain, FusedEpi::kGated})
          for (int64_t tile : {128, 256}) {
            FusedLaunch l;
            l.epi = e; l.m = m; l.n = n; l.k = k;
            choose(l, tile);
          }
  std::printf("%ld tiles in %ld parts, %ld deals behind whole rounds, %ld of them with fewer blocks than workers, %ld chosen\n",
              g_split, g_parts, g_behind, g_fewer, behind);
  return g_split && g_fewer && behind ? 0 : 3;
}
"""


def test_every_part_is_written_once_and_read_once(tmp_path):
    gxx = shutil.which("g++")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build._nvcc())), "include")
    if gxx is None:
        pytest.skip("no g++")
    source, program = tmp_path / "deal.cpp", tmp_path / "deal"
    # (the slots' size is the launcher's; its function is taken out of its file)
    with open(os.path.join(_build.CSRC, "fused_plan.cu")) as f:
        plan = f.read()
    begin = plan.index("size_t fused_slot_bytes(")
    slots = plan[begin:plan.index("\n}\n", begin) + 3]
    source.write_text(PROGRAM.replace("using namespace mpg;", "namespace mpg {\n" + slots + "}\nusing namespace mpg;", 1))
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-I", _build.CSRC, "-I", _build.INCLUDE, "-I", cuda, str(source), "-o", str(program)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(program)], capture_output=True, text=True)
    assert r.returncode == 0, f"{r.returncode}: {r.stdout}"
