"""The work list of the multi-token attention, compiled with the host compiler and run on
the CPU: the CTAs' walks visit every tile of every unit once, a unit's partial results sit
in the slots that the merge looks up and in nobody else's, and every (entry, query, query
head) has one row in each of its units."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_kv_cache_15_b200", "csrc")

PROGRAM = r'''
#include <cstdio>
#include <map>
#include <random>
#include <set>
#include <vector>
#include "extend.h"
using namespace kvq;
#define CHECK(c) do { if (!(c)) { printf("line %d: %s (case %d)\n", __LINE__, #c, it); return 1; } } while (0)
int main() {
  std::mt19937 rng(1);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int it = 0; it < 1500; ++it) {
    static ExtendParams x;
    x.G = pick(1, 8);
    x.Hkv = pick(1, 4);
    x.Hq = x.G * x.Hkv;
    x.T = pick(0, 3) * 64;
    x.n_entries = it % 50 == 0 ? 256 : pick(1, 12);
    int q = 0;
    for (int e = 0; e < x.n_entries; ++e) {
      x.seq[e] = e;
      x.len[e] = pick(0, 9) == 0 ? pick(0, 3) : pick(0, it % 3 ? 3000 : 400);
      x.nq[e] = std::min(x.len[e], pick(0, 3) == 0 ? pick(0, 100) : pick(0, 5));
      x.q0[e] = q;
      q += x.nq[e];
      x.own0[e] = x.member0[e] = 0;
      x.group[e] = -1;
    }
    x.q0[x.n_entries] = x.total_q = q;
    if (q == 0) continue;
    // groups: some entries share their first positions (whole pages before everyone's new tokens)
    x.n_groups = 0;
    x.g_first[0] = 0;
    int n = 0;
    for (int g = 0; g < 2; ++g) {
      int same = 1 << 30;
      std::vector<int> m;
      for (int e = 0; e < x.n_entries; ++e) {
        const int whole = std::min(ex_paged(x, e), x.len[e] - x.nq[e]) / PAGE * PAGE;
        if (x.group[e] < 0 && x.nq[e] > 0 && whole >= 64 && pick(0, 1)) { m.push_back(e); same = std::min(same, whole); }
      }
      if (m.size() < 2) continue;
      x.g_tok[x.n_groups] = same;
      x.g_nq[x.n_groups] = 0;
      for (int e : m) {
        x.group[e] = (int16_t)x.n_groups;
        x.own0[e] = same;
        x.member0[e] = x.g_nq[x.n_groups];
        x.g_nq[x.n_groups] += x.nq[e];
        x.order[n++] = (uint8_t)e;
      }
      x.g_first[++x.n_groups] = n;
    }
    x.chain = it % 2 ? EX_ALONE : it % 4 ? EX_GROUPS : EX_ENTRIES;
    if (x.chain == EX_GROUPS && x.n_groups == 0) continue;
    const int N = 16 << pick(0, 2);
    CHECK(ex_cut(x, N, it % 4 ? pick(1, 40) : 296));
    std::map<int, std::set<int>> ctas;                 // unit -> CTAs with tiles of it
    std::map<std::pair<int, int>, int> visits;         // (unit, tile)
    std::map<int, ExtendUnit> units;
    std::set<int> slots;
    for (int c = 0; c < x.n_ctas; ++c) {
      ExtendWalk w = ex_walk(x, c);
      ExtendUnit u;
      int k0, k1;
      while (ex_next(x, w, u, k0, k1)) {
        CHECK(0 <= k0 && k0 < k1 && k1 <= u.tiles);
        for (int k = k0; k < k1; ++k) {
          visits[{u.unit, k}]++;
          CHECK(ex_start(x, u, k) / x.per == c);
        }
        units[u.unit] = u;
        ctas[u.unit].insert(c);
        CHECK(slots.insert(c + u.unit).second);
        CHECK(c + u.unit < x.n_ctas + x.e_unit[x.n_entries]);
      }
    }
    for (auto& v : visits) CHECK(v.second == 1);
    std::set<std::vector<int>> rows;                   // kind, entry, query, head
    long tiles = 0;
    for (auto& p : units) {
      const ExtendUnit& u = p.second;
      tiles += u.tiles;
      const ExtendUnit v = ex_unit(x, u.kind, u.index, u.head, u.block);
      CHECK(v.unit == u.unit && v.at == u.at && v.tiles == u.tiles);
      const int c0 = u.at / x.per, c1 = ex_start(x, u, u.tiles - 1) / x.per;   // as the merge looks them up
      CHECK((int)ctas[u.unit].size() == c1 - c0 + 1 && *ctas[u.unit].begin() == c0 && *ctas[u.unit].rbegin() == c1);
      int begin, end;
      ex_range(x, u, &begin, &end);
      CHECK(end - begin > (u.tiles - 1) * EX_TILE && end - begin <= u.tiles * EX_TILE);
      for (int r = 0; r < N; ++r) {
        const ExtendRow w = ex_row(x, u, r);
        if (w.entry < 0) continue;
        CHECK(w.query < x.nq[w.entry] && w.head / x.G == u.head);
        CHECK(rows.insert({u.kind, w.entry, w.query, w.head}).second);
        const int at = (u.kind == EX_SHARED ? x.member0[w.entry] : 0) + w.query;   // the merge's row
        CHECK(at / x.QB == u.block && (at % x.QB) * x.G + w.head % x.G == r);
        CHECK(u.kind == EX_SHARED ? x.group[w.entry] == u.index : u.index == w.entry);
      }
    }
    CHECK(tiles == (long)visits.size());
    for (int e = 0; e < x.n_entries; ++e)
      for (int j = 0; j < x.nq[e]; ++j)
        for (int h = 0; h < x.Hq; ++h) {
          CHECK(rows.count({EX_SHARED, e, j, h}) == (size_t)(x.chain != EX_ENTRIES && x.group[e] >= 0));
          CHECK(rows.count({EX_OWN, e, j, h}) == (size_t)(x.chain != EX_GROUPS && ex_paged(x, e) > x.own0[e]));
          CHECK(rows.count({EX_TAIL, e, j, h}) == (size_t)(x.chain != EX_GROUPS && x.len[e] > ex_paged(x, e)));
        }
  }
  printf("ok\n");
  return 0;
}
'''


def test_walks_cover_the_work_and_slots_are_unique(tmp_path):
    src = tmp_path / "worklist.cpp"
    src.write_text(PROGRAM)
    exe = str(tmp_path / "worklist")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    "-I", "/usr/local/cuda/include", str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-500:]
