// Linear attention, chunked forms: how the host plans segments of sequences and how the device
// counts them. Plain C++, so that both sides' arithmetic can be checked without a GPU.
#pragma once

#include <algorithm>

#include "sizes.h"

namespace gdp {
namespace linear {

constexpr int C = 64;  // tokens per chunk
// Most tokens and sequences of a call: positions up to a few chunks past the end, and the number of
// segments, fit an int.
constexpr int64_t kMostTokens = INT32_MAX - 4095, kMostSeqs = 1 << 30;

// A segment of a sequence: t0 = first row, n = rows, pos0 = tokens of the sequence before it
// (paged states: its context included), id = its place in the scratch (cut sequences only).
struct SegRec {
  int t0, n, seq, pos0;
  int first, last, id, pad;
};

// Segments of a launch and the workspace they need.
struct Plan {
  int nseg, Lseg, slices;  // segments per dense sequence, tokens of one
  int64_t bound;           // segments in all at most
  int slots;               // segments of cut sequences at most: a state of scratch each
  size_t recs, seqs, segS, segW, total;
};
// What a kernel's items take, in microseconds: a chunk, a chunk of the state pass, an item's start
// and states, the two extra launches of a split.
struct Cost {
  double chunk, state_chunk, item, split;
};

// Segments of a sequence of n tokens whose first one is `off` positions into its chunk, cut at
// multiples of Lseg positions from that chunk's start.
GDP_HD inline int segment_count(int off, int n, int Lseg) {
  return n > 0 ? (int)(((int64_t)off + n + Lseg - 1) / Lseg) : 1;
}

// Rows of segment j of that sequence.
GDP_HD inline void segment_span(int off, int n, int Lseg, int j, int* lo, int* hi) {
  const int64_t a = (int64_t)j * Lseg - off, b = a + Lseg;
  *lo = j == 0 ? 0 : (int)a;
  *hi = n < b ? n : (int)b;
}

// Segments at most of the sequences that are cut, of N_seq with T tokens in all. A sequence is cut
// when it has more than Lseg positions, of which up to C - 1 may lie before its first token.
inline int64_t cut_bound(int N_seq, int T, int Lseg) {
  const int64_t cut = std::min<int64_t>(N_seq, T / (Lseg + 2 - C));
  return (T + cut * (Lseg + C - 2)) / Lseg;  // segment_count summed
}

// vt: value columns per item; G: multiprocessors.
inline Plan plan_of(int N_seq, int B, int T, int HV, int K, int V, bool packed, int vt, const Cost& cost, int G) {
  Plan x{};
  x.slices = (int)cdiv(V, vt);
  const int chunks = (int)cdiv(T, C);
  const int64_t heads = (int64_t)HV * x.slices;
  x.nseg = 1;
  x.Lseg = std::max(1, chunks) * C;
  if (!packed) {
    // rounds of items over the SMs, of both passes
    const int64_t units = heads * B;
    double best = (double)cdiv(units, G) * (chunks * cost.chunk + cost.item);
    for (int n = 2; n <= chunks && n <= 256; ++n) {
      const int64_t per = cdiv(chunks, n);
      if (cdiv(chunks, per) != n) continue;  // fewer segments of this length do
      const double t = (double)cdiv(units * n, G) * (per * cost.chunk + cost.item) +
                       (double)cdiv(units * (n - 1), G) * (per * cost.state_chunk + cost.item) + cost.split;
      if (t < 0.95 * best) {
        best = t;
        x.nseg = n;
        x.Lseg = (int)per * C;
      }
    }
    x.bound = (int64_t)B * x.nseg;
    x.slots = x.nseg > 1 ? (int)x.bound : 0;
  } else {
    // packed: no more than an SM's share of the whole batch in one item; where a sequence of T tokens
    // fits in one, so it does from any position of a chunk (there is no scratch for a cut then)
    const int64_t share = cdiv(cdiv((int64_t)T * heads, G), C) * C, most = std::max<int64_t>(share, 512);
    x.Lseg = most < T ? (int)most : x.Lseg + C;
    x.bound = ((int64_t)T + (int64_t)N_seq * C) / x.Lseg + N_seq;
    x.slots = x.Lseg < T ? (int)std::min<int64_t>(x.bound, cut_bound(N_seq, T, x.Lseg)) : 0;
  }
  x.recs = kAlign;
  x.seqs = align_up(x.recs + (packed ? (size_t)x.bound * sizeof(SegRec) : 0));
  x.segW = align_up(x.seqs + (packed ? (size_t)N_seq * 2 * sizeof(int32_t) : 0));
  x.segS = align_up(x.segW + (size_t)x.slots * HV * 2 * sizeof(float));
  x.total = align_up(x.segS + (size_t)x.slots * HV * K * V * 4);
  if (x.slots == 0) x.segS = 0;
  return x;
}

}  // namespace linear
}  // namespace gdp
