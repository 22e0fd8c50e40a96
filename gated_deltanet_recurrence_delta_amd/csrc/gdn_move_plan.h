// The order in which the slots of a pool are moved.  Internal header of the
// host: every definition sits in an unnamed namespace of the including file,
// and nothing in it needs a device.
//
// Every pair writes a slot that no other pair writes, and reads one that may
// be written by another.  Put in an order in which each slot is read before
// it is written, the pairs can run one after the other with no second copy of
// anything: pairs whose target nobody reads come first, and each makes its
// source one reader poorer.  What is left then are plain cycles; one of a
// cycle's slots is kept in registers.  Pairs that neither read what another
// writes nor the other way round are in groups of their own and run side by
// side.
#ifndef GDN_MOVE_PLAN_H
#define GDN_MOVE_PLAN_H

#include <stdint.h>

#include <algorithm>
#include <utility>
#include <vector>

namespace {

constexpr int MAX_STEPS = 320;  // steps of one launch: the list travels as kernel arguments (4 KB at most)
constexpr int STEP_ZERO = -1;   // source: zeros
constexpr int STEP_KEPT = -2;   // source: the registers that a cycle's first slot was kept in; target: keep it there
constexpr int FAN = 8;          // targets that one group takes from one source with a single reading

struct MoveList {
  int src[MAX_STEPS];
  int dst[MAX_STEPS];
  uint16_t begin[MAX_STEPS + 1];
};

// The launches of a plan: lists of steps, and how many groups each has.
struct MovePlan {
  std::vector<std::pair<MoveList, int>> launches;
  MoveList list = {};
  int steps = 0, groups = 0;

  void flush() {
    if (groups) {
      list.begin[groups] = (uint16_t)steps;
      launches.emplace_back(list, groups);
    }
    steps = groups = 0;
  }
  // One group, steps in order; a group longer than a launch goes on in the
  // next one, behind it on the stream.
  void add(const std::vector<std::pair<int, int>>& g) {
    size_t i = 0;
    while (i < g.size()) {
      const size_t room = MAX_STEPS - steps;
      // a full launch opens no group, and a group that fits into one launch is not split
      if (room == 0 || (g.size() - i > room && (i > 0 || g.size() <= MAX_STEPS) && steps > 0)) {
        flush();
        continue;
      }
      const size_t n = std::min(room, g.size() - i);
      list.begin[groups++] = (uint16_t)steps;
      for (size_t j = 0; j < n; ++j, ++steps) {
        list.src[steps] = g[i + j].first;
        list.dst[steps] = g[i + j].second;
      }
      i += n;
      if (i < g.size()) flush();
    }
  }
};

// The plan of n pairs of slots in [0, slots); false: a pair is outside, or a target is named twice.
bool plan_moves(MovePlan& mv, long long slots, const int32_t* src, const int32_t* dst, int n) {
  // (target, source), sorted by target: the writer of a slot is found by bisection
  std::vector<std::pair<int, int>> w;
  w.reserve(n);
  for (int i = 0; i < n; ++i) {
    if (dst[i] < 0 || dst[i] >= slots || src[i] < -1 || src[i] >= slots) return false;
    w.emplace_back(dst[i], src[i]);
  }
  std::sort(w.begin(), w.end());
  for (int i = 1; i < n; ++i)
    if (w[i].first == w[i - 1].first) return false;
  w.erase(std::remove_if(w.begin(), w.end(), [](const std::pair<int, int>& p) { return p.first == p.second; }),
          w.end());
  if (w.empty()) return true;
  n = (int)w.size();
  std::vector<int> writer(n, -1), readers(n, 0), up(n);  // pair -> pair that writes its source; how many read its target
  for (int i = 0; i < n; ++i) {
    up[i] = i;
    if (w[i].second < 0) continue;
    const auto it = std::lower_bound(w.begin(), w.end(), std::make_pair(w[i].second, INT32_MIN));
    if (it != w.end() && it->first == w[i].second) {
      writer[i] = (int)(it - w.begin());
      ++readers[writer[i]];
    }
  }
  std::vector<std::pair<int, int>> g;
  // 1. pairs that no other pair has to wait for or be waited for, those of one source together
  std::vector<std::pair<int, int>> alone;
  for (int i = 0; i < n; ++i)
    if (writer[i] < 0 && readers[i] == 0) alone.emplace_back(w[i].second, w[i].first);
  std::sort(alone.begin(), alone.end());
  for (size_t i = 0; i < alone.size(); ++i) {
    if (!g.empty() && (g.back().first != alone[i].first || g.size() == FAN)) {
      mv.add(g);
      g.clear();
    }
    g.push_back(alone[i]);
  }
  if (!g.empty()) mv.add(g);
  // 2. the others, by connected component
  auto root = [&](int i) {
    while (up[i] != i) i = up[i] = up[up[i]];
    return i;
  };
  for (int i = 0; i < n; ++i)
    if (writer[i] >= 0) up[root(i)] = root(writer[i]);
  std::vector<std::pair<int, int>> of;  // (component, pair)
  for (int i = 0; i < n; ++i)
    if (writer[i] >= 0 || readers[i] > 0) of.emplace_back(root(i), i);
  std::sort(of.begin(), of.end());
  std::vector<std::pair<int, int>> ready;  // (source, pair)
  std::vector<char> done(n, 0);
  for (size_t b = 0; b < of.size();) {
    size_t e = b;
    while (e < of.size() && of[e].first == of[b].first) ++e;
    g.clear();
    ready.clear();
    for (size_t i = b; i < e; ++i)
      if (readers[of[i].second] == 0) ready.emplace_back(w[of[i].second].second, of[i].second);
    std::sort(ready.begin(), ready.end());
    while (!ready.empty()) {
      const int i = ready.back().second;
      ready.pop_back();
      done[i] = 1;
      g.emplace_back(w[i].second, w[i].first);
      const int up_ = writer[i];
      if (up_ >= 0 && --readers[up_] == 0) ready.emplace_back(w[up_].second, up_);
    }
    // What is left is at most one cycle.  A long one is turned in pieces:
    // turning a_0 .. a_k first leaves a_0's old state in a_k, and the rest,
    // a_k among it, is a shorter cycle.
    for (size_t i = b; i < e; ++i) {
      int at = of[i].second;
      if (done[at]) continue;
      std::vector<int> cyc;
      for (; !done[at]; at = writer[at]) {
        done[at] = 1;
        cyc.push_back(w[at].first);
      }
      for (size_t s = 0; s + 1 < cyc.size();) {
        const size_t k = std::min(cyc.size(), s + (size_t)MAX_STEPS - 2);
        if (s > 0 || g.size() + (k - s) + 1 > (size_t)MAX_STEPS) {  // a piece of a cycle stays in one launch
          mv.add(g);
          mv.flush();
          g.clear();
        }
        g.emplace_back(cyc[s], STEP_KEPT);
        for (size_t j = s; j + 1 < k; ++j) g.emplace_back(cyc[j + 1], cyc[j]);
        g.emplace_back(STEP_KEPT, cyc[k - 1]);
        s = k - 1;
      }
    }
    mv.add(g);
    b = e;
  }
  mv.flush();
  return true;
}

}  // namespace

#endif  // GDN_MOVE_PLAN_H
