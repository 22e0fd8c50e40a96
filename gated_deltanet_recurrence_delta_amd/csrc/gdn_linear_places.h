// Which sequence and segment of a packed batch comes at a place of a linear
// attention launch.  Internal header: every definition sits in an unnamed
// namespace of the including file.  It needs no device, so that a host
// program can walk through it as a workgroup's threads do.
#ifndef GDN_LINEAR_PLACES_H
#define GDN_LINEAR_PLACES_H

#include <stdint.h>

#ifdef __HIPCC__
#define GDN_ANY_SIDE __host__ __device__
#else
#define GDN_ANY_SIDE
#endif

namespace {

// A packed batch: B sequences between offsets that are taken into [0, T].
struct Packed {
  const int32_t* cu;
  int B, T;
  GDN_ANY_SIDE inline int at(int i) const { return cu[i] < 0 ? 0 : cu[i] > T ? T : cu[i]; }
};

// The begin and length of sequence i, within the rows there are; an end before the begin: no rows.
struct Rows {
  int begin, len;
  bool falls;  // the end lies before the begin
};
GDN_ANY_SIDE inline Rows rows_of(const Packed& b, int i) {
  const int begin = b.at(i), end = b.at(i + 1);
  return {begin, end < begin ? 0 : end - begin, end < begin};
}

constexpr int SORTED = 64;  // sequences of a packed batch that are put in order of length

// What a workgroup's threads find out together, in memory they share.
struct PlaceBoard {
  int falls;                        // an offset lies before an earlier one
  int n, seg;                       // what was found; n < 0: nothing
  int whole[SORTED], rest[SORTED];  // sorted order: whole segments, and the rows behind them (-1: none)
  GDN_ANY_SIDE inline void take(int i, int segment) {
    n = i;
    seg = segment;
  }
};

struct Place {
  int n, seg;  // n < 0: there is none
  bool uncut;  // the whole sequence, whatever the segments' length
};

// Place `at` of a packed batch cut into segments of `rows` rows: begin(),
// look() and settle() by every thread of a workgroup, a barrier behind each,
// then place(), and a barrier before the board's memory is used again.
//
// PASS 1 goes by the slots of the segments that others follow: a sequence's
// are floor(begin / rows) and on, as many as whole segments fit in it at most,
// so that the sequences' slots are apart and below floor(T / rows).
//
// PASS 0 takes whole segments first and then the sequences' last ones from
// long to short, so that the workgroups that start late are short ones
// (64,711 rows in 32 sequences of 16 heads, dx = dz = 128: 252 us, in the
// order of the batch 338).  With more sequences the order matters less and
// costs more (50,000 rows in 100: 232 against 225), and sequence i has the
// places floor(begin / rows) + i and on.
//
// All of that needs offsets that ascend: only then are the begins in order,
// no row is in two sequences and T / rows + B places are enough.  Where one
// falls, place i is sequence i, uncut.
template <int PASS>
struct Places {
  Packed b;
  int rows, at;
  static constexpr bool CAN_SORT = PASS == 0;

  GDN_ANY_SIDE inline bool sorted() const { return CAN_SORT && b.B <= SORTED; }
  GDN_ANY_SIDE inline void begin(int tid, PlaceBoard& s) const {
    if (tid == 0) {
      s.falls = 0;
      s.n = -1;
    }
  }
  GDN_ANY_SIDE inline void look(int tid, int threads, PlaceBoard& s) const {
    for (int i = tid; i < b.B; i += threads) {
      const Rows r = rows_of(b, i);
      if (r.falls) s.falls = 1;
      if (sorted()) {
        s.whole[i] = r.len / rows;
        s.rest[i] = r.len % rows > 0 || r.len == 0 ? r.len % rows : -1;
      } else {
        const int segs = (r.len + rows - 1) / rows;
        const int first = r.begin / rows + (PASS == 0 ? i : 0), count = PASS == 0 ? (segs > 1 ? segs : 1) : segs - 1;
        // by several threads only where an offset falls; settle() overrules them there
        if (at >= first && at < first + count) s.take(i, at - first);
      }
    }
  }
  GDN_ANY_SIDE inline void settle(int tid, int threads, PlaceBoard& s) const {
    if (s.falls) {
      if (tid == 0) s.take(PASS == 0 && at < b.B ? at : -1, 0);
    } else if (sorted()) {
      for (int i = tid; i < b.B; i += threads) {
        const int wi = s.whole[i], ri = s.rest[i];
        int before = 0, all = 0, longer = 0;
        for (int j = 0; j < b.B; ++j) {
          const int wj = s.whole[j], rj = s.rest[j];
          all += wj;
          before += j < i ? wj : 0;
          longer += rj > ri || (rj == ri && j < i);
        }
        if (at < all ? at >= before && at < before + wi : ri >= 0 && at - all == longer)
          s.take(i, at < all ? at - before : wi);
      }
    }
  }
  GDN_ANY_SIDE inline Place place(const PlaceBoard& s) const { return {s.n, s.seg, s.falls != 0}; }
};

}  // namespace

#endif  // GDN_LINEAR_PLACES_H
