// A host model of the waits of tc_cross_read_kernel (csrc/tc_cross.cu) under random schedules, with the kernel's own ring
// sizes (csrc/cross_ring.h).  The actors: the warps that share a row (each takes the features of a tile, with its part of the
// row's sum, and then the results of the tile before), the issuing thread, and the copies and products, which end whenever they
// like (products in order).  Checked at every step: a warp that takes features finds that tile in its buffer, and one that
// takes results finds in every part of the sum, and in the tile's buffer, what belongs to that tile.
//
//   cross_ring_check d warps buffers sums tiles runs     (buffers, sums 0: the kernel's)
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "cross_ring.h"

namespace {

struct Model {
  int warps, buffers, sums, tiles;
  std::vector<int> ready, out;      // arrivals of the warps, by tile
  std::vector<char> full, mma;      // a tile has landed; its product is done
  std::vector<int> holds;           // the tile in a buffer
  std::vector<std::vector<int>> den;  // [sums][warps]: the tile that a part belongs to
  std::vector<int> at, part;        // a warp: its step (2 j: features of j, 2 j + 1: results of j - 1), parts that it has read
  std::vector<int> flying;          // tiles on their way
  int issued = 0, step = 0;         // products issued; the issuing thread's step
  int done = 0;                     // products done

  Model(int w, int b, int s, int t)
      : warps(w), buffers(b), sums(s), tiles(t), ready(t), out(t), full(t), mma(t), holds(b, -1), den(s, std::vector<int>(w, -1)),
        at(w), part(w) {
    for (int j = 0; j < t && j < b; ++j) flying.push_back(j);
  }
  // One step of warp w; false: it waits.  bad: it found what is another tile's.
  bool warp(int w, bool* bad) {
    const int j = at[w] / 2;
    if (at[w] % 2 == 0) {
      if (j < tiles) {
        if (!full[j]) return false;
        *bad |= holds[j % buffers] != j;
        den[j % sums][w] = j;
        ++ready[j];
      }
      at[w] += j == 0 ? 2 : 1;  // (nothing goes out before tile 0)
      return true;
    }
    const int t = j - 1;
    if (!mma[t]) return false;
    if (part[w] < warps) {
      *bad |= den[t % sums][part[w]] != t;
      ++part[w];
      return true;
    }
    *bad |= holds[t % buffers] != t;
    part[w] = 0;
    ++out[t];
    ++at[w];
    return true;
  }
  bool finished(int w) const { return at[w] > 2 * tiles + 1; }
  // The issuing thread: step 2 j: the product of tile j; 2 j + 1: the results of tile j - 1 go out, another tile comes in.
  bool issue() {
    const int j = step / 2;
    if (step % 2 == 0 && j < tiles) {
      if (ready[j] < warps) return false;
      ++issued;
    } else if (step % 2 == 1 && j > 0) {
      const int t = j - 1;
      if (out[t] < warps) return false;
      if (t + buffers < tiles) flying.push_back(t + buffers);
    }
    ++step;
    return true;
  }
  bool issue_finished() const { return step > 2 * tiles + 1; }
};

// 0: right; 1: another tile's values; 2: no actor can go on.
int run(int warps, int buffers, int sums, int tiles, std::mt19937& rng) {
  Model m(warps, buffers, sums, tiles);
  std::vector<double> speed(warps + 3);  // some actors lag
  for (double& s : speed) s = rng() % 3 == 0 ? 0.02 : 1.0;
  int idle = 0;
  for (;;) {
    bool end = m.issue_finished();
    for (int w = 0; w < warps; ++w) end = end && m.finished(w);
    if (end) return 0;
    std::discrete_distribution<int> pick(speed.begin(), speed.end());
    const int a = pick(rng);
    bool moved = false, bad = false;
    if (a < warps) {
      moved = !m.finished(a) && m.warp(a, &bad);
    } else if (a == warps) {
      moved = !m.issue_finished() && m.issue();
    } else if (a == warps + 1) {
      if (!m.flying.empty()) {
        const size_t i = rng() % m.flying.size();
        const int t = m.flying[i];
        m.holds[t % buffers] = t;
        m.full[t] = 1;
        m.flying.erase(m.flying.begin() + i);
        moved = true;
      }
    } else if (m.done < m.issued) {
      m.mma[m.done++] = 1;
      moved = true;
    }
    if (bad) return 1;
    idle = moved ? 0 : idle + 1;
    if (idle > 20000) return 2;
  }
}

}  // namespace

int main(int argc, char** argv) {
  if (argc != 7) return 9;
  const int d = std::atoi(argv[1]), warps = std::atoi(argv[2]), tiles = std::atoi(argv[5]), runs = std::atoi(argv[6]);
  const int buffers = std::atoi(argv[3]) ? std::atoi(argv[3]) : mhla::read_buffers(d);
  const int sums = std::atoi(argv[4]) ? std::atoi(argv[4]) : mhla::read_sums(d);
  std::mt19937 rng(7);
  int wrong = 0, stuck = 0;
  for (int i = 0; i < runs; ++i) {
    const int r = run(warps, buffers, sums, tiles, rng);
    wrong += r == 1;
    stuck += r == 2;
  }
  std::printf("%d %d %d %d\n", buffers, sums, wrong, stuck);
  return 0;
}
