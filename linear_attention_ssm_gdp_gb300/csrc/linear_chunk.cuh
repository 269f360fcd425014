// Shared by the chunked kernels of linear attention: segments of sequences as work items,
// and the decays of a chunk.
#pragma once

#include "linear_internal.cuh"
#include "linear_plan.h"

namespace gdp {
namespace linear {

constexpr float kGMin = -1e5f;  // e^g is 0 far above this; keeps -inf out of the prefix sums

struct ChunkArgs {
  LinearProblem p;
  const SegRec* recs;   // packed batches; seq = -1 past the last
  const int* split;     // packed batches: whether any sequence is in several segments
  int clear;            // the first launch of a dense call: sets the status word to kDevOk
  int nseg, Lseg;       // dense batches: segments per sequence, tokens per segment
  int slices, vt;       // slices of vt value columns
  int items;            // bound over all CTAs
  float* segS;          // [segments of cut sequences][HV][K][V]: a segment's U, then the state at its start
  float2* segW;         // [the same][HV]: its whole decay factor
};

// The two kernels around the state pass: segment records of a packed batch, and the states at
// the segment starts.
cudaError_t launch_segments(const LinearProblem& p, const Plan& x, SegRec* recs, int2* seqs, int* split);
cudaError_t launch_combine(const ChunkArgs& a, const int2* seqs);

struct Item {
  SegRec r;
  int b, hv, h, v0, off, chunks;
};

// Item `it` of the launch, value slices of a head and heads of a sequence side by side.
__device__ __forceinline__ bool get_item(const ChunkArgs& a, int it, Item& x) {
  const int slice = it % a.slices, rest = it / a.slices;
  x.hv = rest % a.p.HV;
  x.h = x.hv / (a.p.HV / a.p.H);
  x.v0 = slice * a.vt;
  const int s = rest / a.p.HV;
  if (a.recs) {
    const int4 u = reinterpret_cast<const int4*>(a.recs)[2 * s];
    const int4 w = reinterpret_cast<const int4*>(a.recs)[2 * s + 1];
    x.r.t0 = u.x; x.r.n = u.y; x.r.seq = u.z; x.r.pos0 = u.w;
    x.r.first = w.x; x.r.last = w.y; x.r.id = w.z; x.r.pad = 0;
    x.b = 0;
    if (x.r.seq < 0) return false;
  } else {
    const int b = s / a.nseg, j = s - b * a.nseg;
    x.b = b;
    x.r.t0 = j * a.Lseg;
    x.r.n = min(a.Lseg, a.p.T - x.r.t0);
    x.r.seq = b;
    x.r.pos0 = x.r.t0;
    x.r.first = j == 0;
    x.r.last = j == a.nseg - 1;
    x.r.id = s;
    x.r.pad = 0;
  }
  // chunks end where blocks do, so the first one may be short
  x.off = a.p.pool ? x.r.pos0 % C : 0;
  x.chunks = x.r.n > 0 ? (x.off + x.r.n + C - 1) / C : 0;
  return true;
}

// An item that a launch has nothing to do for (the state pass stops before a sequence's last
// segment).
template <bool OUT>
__device__ __forceinline__ bool skip(const Item& x) {
  return !OUT && x.r.last;
}

// ------------------------------------------------------------------ decays of a chunk
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float two_sum(float a, float b, float& e) {
  const float s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
  return s;
}
// Natural-log two-float to base 2, cancellation of the hi parts kept exact.
__device__ __forceinline__ float2 log2e_pair(float hi, float lo) {
  constexpr float kLog2e = 1.44269504088896341f;
  const float p = hi * kLog2e;
  return make_float2(p, fmaf(lo, kLog2e, fmaf(hi, kLog2e, -p)));
}
// e^(hi + lo) as a pair of floats (error ~2^-27): reduction by n ln 2 (a 16-bit head, so
// that n head is exact), Taylor's series for the rest, its leading 1 + r added exactly.
// Below the normal range the result is 0, past the largest float infinite; NaN passes.
__device__ __forceinline__ float2 exp_pair(float hi, float lo) {
  const float n = rintf(hi * 1.44269504f);
  float rl;
  const float r = two_sum(fmaf(-n, 0.693145751953125f, hi), fmaf(-n, 1.42860682e-6f, lo), rl);
  float q = 2.48015873e-5f;                 // 1 / 8!
  q = fmaf(q, r, 1.98412698e-4f);
  q = fmaf(q, r, 1.38888889e-3f);
  q = fmaf(q, r, 8.33333333e-3f);
  q = fmaf(q, r, 4.16666667e-2f);
  q = fmaf(q, r, 1.66666667e-1f);
  q = fmaf(q, r, 0.5f);
  float e, l;
  const float s = two_sum(1.f, r, e);
  const float h = two_sum(s, fmaf(q, r * r, rl) + e, l);
  if (hi < -87.f) return make_float2(0.f, 0.f);
  if (hi > 89.f) return make_float2(__int_as_float(0x7f800000), 0.f);
  // 2^n in two halves: n reaches 128, and 2^128 is past the largest float where h 2^128 is not
  const int m = (int)n, half = m >> 1;
  const float s0 = __int_as_float((half + 127) << 23), s1 = __int_as_float((m - half + 127) << 23);
  return make_float2(h * s0 * s1, l * s0 * s1);
}

// g at position i of the chunk whose position 0 is row `base`; 0 outside the sequence.
__device__ __forceinline__ float load_g(const LinearProblem& p, const Item& x, int base, int i) {
  const int r = base + i;
  if (!p.g || r < x.r.t0 || r >= x.r.t0 + x.r.n) return 0.f;
  return p.g_token ? __ldg(p.g + ((int64_t)x.b * p.T + r) * p.HV + x.hv) : __ldg(p.g + x.hv);
}

// By one warp, lane l with g (as loaded) at positions 2 l and 2 l + 1: writes the chunk's decays,
// g[0..63] and g[64..127] the base-2 prefix sums (hi, lo), g[128..] e^{Gam - Gam_i} (0 outside
// [lo, hi)), g[192..] scale e^{Gam_t}, g[256], g[257] e^{Gam} as a pair. The prefix sums are
// compensated, so differences of them are good however strong the decays before.
__device__ __forceinline__ void chunk_decays(float g0, float g1, float scale, int lo, int hi, int lane, float* g) {
  g0 = g0 < kGMin ? kGMin : g0;
  g1 = g1 < kGMin ? kGMin : g1;
  float e1;
  const float s1 = two_sum(g0, g1, e1);
  float S = s1, E = e1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float S2 = __shfl_up_sync(0xffffffffu, S, o), E2 = __shfl_up_sync(0xffffffffu, E, o);
    if (lane >= o) {
      float e;
      S = two_sum(S2, S, e);
      E = __fadd_rn(__fadd_rn(E2, E), e);
    }
  }
  float pS = __shfl_up_sync(0xffffffffu, S, 1), pE = __shfl_up_sync(0xffffffffu, E, 1);
  if (lane == 0) pS = pE = 0.f;
  float h[2], l[2], e;
  h[0] = two_sum(pS, g0, e);
  l[0] = pE + e;
  h[1] = two_sum(pS, s1, e);
  l[1] = (pE + e1) + e;
  const float hl = __shfl_sync(0xffffffffu, h[1], 31), ll = __shfl_sync(0xffffffffu, l[1], 31);
  const float2 w = exp_pair(hl, ll), bl = log2e_pair(hl, ll);
  float2 b2[2];
  float we[2], ei[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = 2 * lane + u;
    b2[u] = log2e_pair(h[u], l[u]);
    // 2^x is good to 2^-22; a rounded exponent matters less the smaller the factor
    we[u] = i >= lo && i < hi ? ex2_approx((bl.x - b2[u].x) + (bl.y - b2[u].y)) : 0.f;
    ei[u] = scale * ex2_approx(b2[u].x + b2[u].y);
  }
  *reinterpret_cast<float2*>(g + 2 * lane) = make_float2(b2[0].x, b2[1].x);
  *reinterpret_cast<float2*>(g + 64 + 2 * lane) = make_float2(b2[0].y, b2[1].y);
  *reinterpret_cast<float2*>(g + 128 + 2 * lane) = make_float2(we[0], we[1]);
  *reinterpret_cast<float2*>(g + 192 + 2 * lane) = make_float2(ei[0], ei[1]);
  if (lane == 0) *reinterpret_cast<float2*>(g + 256) = w;
}

// A state pass (or the combine kernel) with nothing to do: only the device knows how a packed
// batch's sequences came out.
__device__ __forceinline__ bool no_split(const ChunkArgs& a) { return a.split && __ldcg(a.split) == 0; }

// Where the state after chunk c of an item is kept (null: nowhere), base of [HV, K, V].
template <bool OUT>
__device__ __forceinline__ float* state_dst(const ChunkArgs& a, const Item& x, int c) {
  const LinearProblem& p = a.p;
  const int64_t sz = (int64_t)p.HV * p.K * p.V;
  const bool more = c + 1 < x.chunks;
  if (!OUT) return more ? nullptr : a.segS + x.r.id * sz;
  if (p.pool) {
    uint32_t end = (uint32_t)(x.r.pos0 - x.off) + (uint32_t)(c + 1) * C;
    if (end % (uint32_t)p.block != 0 && (more || !x.r.last)) return nullptr;
    end = min(end, (uint32_t)x.r.pos0 + (uint32_t)x.r.n);
    return p.pool + p.tables[(int64_t)x.r.seq * p.width + (end - 1) / (uint32_t)p.block] * sz;
  }
  return !more && x.r.last && p.sT ? p.sT + x.r.seq * sz : nullptr;
}

// The state that an item starts from (null: zeros), base of [HV, K, V].
template <bool OUT>
__device__ __forceinline__ const float* state_src(const ChunkArgs& a, const Item& x) {
  const LinearProblem& p = a.p;
  const int64_t sz = (int64_t)p.HV * p.K * p.V;
  if (!OUT) return nullptr;
  // a split sequence's states all come from the scratch: its first page may be written by its
  // last segment meanwhile
  if (!(x.r.first && x.r.last)) return a.segS + x.r.id * sz;
  if (p.pool)
    return x.r.pos0 > 0 && x.r.n > 0
               ? p.pool + p.tables[(int64_t)x.r.seq * p.width + (x.r.pos0 - 1) / p.block] * sz
               : nullptr;
  return p.s0 ? p.s0 + x.r.seq * sz : nullptr;
}

// The product of two factors kept as pairs.
__device__ __forceinline__ float2 mul_pair(float2 a, float2 b) {
  const float h = a.x * b.x;
  const float l = fmaf(a.x, b.x, -h) + (a.x * b.y + a.y * b.x);
  const float s = h + l;
  return make_float2(s, l - (s - h));
}

}  // namespace linear
}  // namespace gdp
