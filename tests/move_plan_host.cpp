// The launches that move a pool's slots, carried out on the host as
// move_kernel's threads do: one value a slot, the groups of a launch in any order.
#include "gdn_move_plan.h"

#include <cstring>
#include <random>

// 0, or what is wrong: 1 refused, 2 a list out of its bounds, 3 a slot outside the pool,
// 4 two groups of a launch share a slot that one of them writes, 5 a slot read after it was written
extern "C" int move_plan(int slots, const int32_t* src, const int32_t* dst, int n, int* pool, unsigned seed,
                         int* launches) {
  MovePlan plan;
  if (!plan_moves(plan, slots, src, dst, n)) return 1;
  *launches = (int)plan.launches.size();
  std::mt19937 rnd(seed);
  for (const auto& l : plan.launches) {
    const MoveList& m = l.first;
    const int groups = l.second;
    if (groups < 1 || groups > MAX_STEPS || m.begin[0] != 0) return 2;
    for (int i = 0; i < groups; ++i)
      if (m.begin[i] >= m.begin[i + 1] || m.begin[i + 1] > MAX_STEPS) return 2;
    std::vector<int> order(groups), writer(slots, -1);
    for (int i = 0; i < groups; ++i) {
      order[i] = i;
      for (int t = m.begin[i]; t < m.begin[i + 1]; ++t) {
        if (m.src[t] < STEP_KEPT || m.src[t] >= slots || m.dst[t] < STEP_KEPT || m.dst[t] >= slots ||
            m.dst[t] == STEP_ZERO)
          return 3;
        if (m.dst[t] == STEP_KEPT) continue;
        if (writer[m.dst[t]] >= 0) return 4;
        writer[m.dst[t]] = i;
      }
    }
    for (int i = 0; i < groups; ++i)
      for (int t = m.begin[i]; t < m.begin[i + 1]; ++t)
        if (m.src[t] >= 0 && writer[m.src[t]] >= 0 && writer[m.src[t]] != i) return 4;
    std::shuffle(order.begin(), order.end(), rnd);
    for (int g : order) {
      int reg = 0, kept = 0, last = STEP_ZERO;
      std::vector<char> written(slots, 0);
      for (int t = m.begin[g]; t < m.begin[g + 1]; ++t) {
        const int s = m.src[t], d = m.dst[t];
        if (s != last) {
          last = s;
          if (s >= 0 && written[s]) return 5;
          reg = s == STEP_KEPT ? kept : s == STEP_ZERO ? 0 : pool[s];
        }
        if (d == STEP_KEPT) {
          kept = reg;
        } else {
          pool[d] = reg;
          written[d] = 1;
        }
      }
    }
  }
  return 0;
}
