// The places of a packed linear-attention batch, walked through on the host as
// a workgroup's threads do.
#include "gdn_linear_places.h"

namespace {

// found: (sequence, segment, uncut) of each place, and how many times a phase of threads took a place
template <int PASS>
void walk(const int32_t* cu, int B, int T, int rows, int threads, int places, int* found) {
  for (int at = 0; at < places; ++at) {
    const Places<PASS> p = {{cu, B, T}, rows, at};
    PlaceBoard s = {};
    s.n = s.seg = -7;  // what another workgroup left
    int taken = 0;
    for (int t = 0; t < threads; ++t) p.begin(t, s);
    for (int phase = 0; phase < 2; ++phase) {
      int n = s.n, seg = s.seg, here = 0;
      for (int t = 0; t < threads; ++t) {
        s.n = -1;
        if (phase == 0) p.look(t, threads, s);
        else p.settle(t, threads, s);
        if (s.n >= 0) {
          n = s.n;
          seg = s.seg;
          ++here;
        }
      }
      // a phase that finds a falling offset discards what the one before took
      if (phase == 1 && s.falls) {
        taken = here;
        if (!here) n = -1;
      } else {
        taken += here;
      }
      s.n = n;
      s.seg = seg;
    }
    const Place r = p.place(s);
    found[4 * at] = r.n;
    found[4 * at + 1] = r.seg;
    found[4 * at + 2] = r.uncut;
    found[4 * at + 3] = taken;
  }
}

}  // namespace

extern "C" void linear_places(int pass, const int32_t* cu, int B, int T, int rows, int threads, int places, int* found) {
  if (pass == 0) walk<0>(cu, B, T, rows, threads, places, found);
  else walk<1>(cu, B, T, rows, threads, places, found);
}
