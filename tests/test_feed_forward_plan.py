"""The host side of the feed-forward's products, compiled without a device:
how many loads a step's end may leave on their way."""

import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gru_sequence_scan_amd", "csrc")


def _run(tmp_path, body, *args):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text("#include <cstdio>\n#include <cstdlib>\n#include <vector>\n#include \"feed_forward_plan.hpp\"\nusing namespace rnnk;\n" + body)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True, check=True).stdout


# A workgroup's loads in their order, over tiles of any numbers of steps; some
# steps of A and of B go through registers and wait for all that is older.
_PACE = r"""
struct Load { bool b; int step; bool whole; };
int main(int, char** v) {
  const int ahead = atoi(v[1]);
  srand(1);
  long exact = 0, all = 0, last_left = 0;
  for (int round = 0; round < 20000; ++round) {
    std::vector<int> tiles(1 + rand() % 4);
    std::vector<char> whole_a, whole_b;
    const int partial = rand() % 3;  // none, few, many
    for (int& n : tiles) {
      n = 1 + rand() % 9;
      for (int i = 0; i < n; ++i) {
        whole_a.push_back(!(partial && rand() % (partial == 1 ? 8 : 2) == 0));
        whole_b.push_back(!(partial && rand() % (partial == 1 ? 8 : 2) == 0));
      }
    }
    const int n = (int)whole_a.size();
    std::vector<Load> out;  // what may be on its way, oldest first
    auto send = [&](bool b, int step) {
      const bool whole = b ? whole_b[step] : whole_a[step];
      if (whole) out.push_back({b, step, true}); else out.clear();
    };
    for (int i = 0; i < ahead; ++i) {
      if (i < n) send(false, i);
      if (i < ahead - 1 && i < n) send(true, i);
    }
    out.clear();
    int t = 0;
    for (size_t k = 0; k < tiles.size(); ++k)
      for (int i = 0; i < tiles[k]; ++i, ++t) {
        const bool more_b = t + ahead - 1 < n, more_a = t + ahead < n;
        const bool whole = (!more_a || whole_a[t + ahead]) && (!more_b || whole_b[t + ahead - 1]);
        if (more_b) send(true, t + ahead - 1);
        if (more_a) send(false, t + ahead);
        const int later = feed_later(ahead, more_a, more_b, whole, tiles[k] - 1 - i);
        if (later < 0 || later > 2 * ahead - 3) return printf("range %d\n", later), 0;
        // what is newer than the next step's, were all of it still on its way
        int newer = 0;
        for (const Load& l : out) newer += l.step > t + 1;
        const int had = (int)out.size();
        while ((int)out.size() > later) out.erase(out.begin());
        for (const Load& l : out)
          if (l.step <= t + 1) return printf("step %d of %d still loads\n", l.step, n), 0;
        ++all;
        if (k + 1 == tiles.size() && whole && !partial) {
          // nothing newer is waited for in the last tile
          if ((int)out.size() != newer) return printf("waits for %d of %d, %d there\n", newer - (int)out.size(), newer, had), 0;
          ++exact;
          if (!more_a && newer) ++last_left;
        }
      }
    if (!out.empty()) return printf("left\n"), 0;
  }
  printf("ok %d %d %d\n", all > 100000, exact > 10000, last_left > 1000);
}
"""


@pytest.mark.parametrize("ahead", [2, 4])
def test_no_wait_is_too_short_and_the_last_tile_has_none_too_long(tmp_path, ahead):
    # with two steps ahead the last steps have nothing newer than what comes next
    assert _run(tmp_path, _PACE, ahead).strip() == f"ok 1 1 {1 if ahead == 4 else 0}"


# The instance (type, product, tile, divided or not) and the ways out (a tile
# that is whole, one at an edge) of the products that sizes take; of many random
# sizes, those that the given ones leave out.
_COVER = r"""
#include <random>
#include <set>
#include <string>
std::set<std::string> taken(bool bf, int64_t rows, int N, int F, int N_out) {
  const char* ops[] = {"in", "out", "dh", "dx", "dw_in", "dw_out"};
  const char* tiles[] = {"small", "big", "deep"};
  const FeedSizes s(bf, rows, N, F, N_out);
  std::set<std::string> all;
  for (int op = 0; op < kFeedOps; ++op) {
    if (op <= kFeedOut && s.few(true) && s.few(false)) continue;
    const FeedPlan p = s.plan(op, 256);
    const int64_t h = p.tile == kTileBig ? 256 : 128, w = op == kFeedIn ? h / 2 : h;
    const int64_t M = op == kFeedDwIn ? 2 * (int64_t)s.Fp : op == kFeedDwOut ? N_out : rows;
    const int64_t last = op == kFeedIn || op == kFeedDh || op == kFeedDwOut ? F : op == kFeedOut ? N_out : N;
    const std::string name = std::string(bf ? "bf16 " : "f32 ") + ops[op] + " " + tiles[p.tile] + (p.splits > 1 ? " divided" : " undivided");
    if (M >= h && last >= w) all.insert(name + " whole");
    if (M % h || last % w) all.insert(name + " edge");
  }
  return all;
}
int main(int, char** v) {
  std::set<std::string> have, missing;
  FILE* f = fopen(v[1], "r");
  long bf, rows, N, F, N_out;
  while (fscanf(f, "%ld %ld %ld %ld %ld", &bf, &rows, &N, &F, &N_out) == 5)
    for (auto& name : taken(bf, rows, N, F, N_out)) have.insert(name);
  std::mt19937_64 rng(1);
  auto size = [&](double most) { return (int)exp(std::uniform_real_distribution<>(0, log(most))(rng)); };
  for (int i = 0; i < 200000; ++i) {
    const bool b = rng() & 1;
    const int r = size(70000), n = size(20000), h = size(40000), o = rng() & 1 ? n : size(20000);
    if ((double)r * n * h > 3e11) continue;
    for (auto& name : taken(b, r, n, h, o))
      if (!have.count(name)) missing.insert(name);
  }
  for (auto& name : missing) puts(name.c_str());
  printf("%zu\n", have.size());
}
"""


def test_the_gpu_tests_take_every_tile_and_split(tmp_path):
    pytest.importorskip("gru_sequence_scan_amd")
    from feed_plan_shapes import SHAPES
    from test_gpu_feed_forward import SIZES
    sizes = [(t == "bf16",) + tuple(s) for t, *s in SHAPES] + [(bf,) + s for s in SIZES for bf in (False, True)]
    (tmp_path / "sizes").write_text("".join(" ".join(str(int(v)) for v in s) + "\n" for s in sizes))
    out = _run(tmp_path, _COVER, tmp_path / "sizes").split("\n")[:-1]
    assert out[:-1] == [] and int(out[-1]) >= 140
