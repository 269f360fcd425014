// Linear attention with a decay for each head, chunked form on the tensor cores:
// bf16 inputs, K <= 128, any V in slices of 128 columns.
//
// With Gam_t the sum of g over a chunk's tokens up to t, S the state before the
// chunk and Gam the chunk's whole sum,
//     o_t = scale (e^{Gam_t} S^T q_t + sum_{i <= t} e^{Gam_t - Gam_i} (q_t . k_i) v_i),
//     S  <- e^{Gam} S + sum_i k_i (e^{Gam - Gam_i} v_i)^T.
// Four products per chunk of 64 tokens, with the value columns on the 128 rows of
// the tensor core's accumulator wherever the product has them:
//     QK     [t | i]  = q k^T            (rows 64.. of the A tile are k's: unused)
//     INTER  [v | t]  = S^T q^T          S as bf16
//     INTRA  [v | t]  = v^T P^T          P = masked, decayed scores as bf16
//     U      [v | k]  = v'^T k           v' = e^{Gam - Gam_i} v_i as three bf16 parts
//
// Roundings. q, k, v enter exactly. P and the copy of S that INTER reads are rounded
// to bf16 like o itself (each adds an error of the size of o's own rounding, averaged
// over the sum). The state is kept in fp32 registers and v' in 24 bits (three bf16
// parts), because its error would add up over the chunks; e^{Gam} is a pair of floats
// for the same reason. Decay exponents are differences of compensated prefix sums, so
// a strong decay earlier in the chunk costs no digits.
//
// What bounds it: q, k, v, o are 64 KB per chunk and head, 1.5 us of an SM's share of HBM.
// A product with both operands in shared memory runs at that memory's 128 bytes a clock
// ((A + B) / 128 cycles, measured), more than the tensor pipe needs, so the operands that
// are made on chip (S, v') live in tensor memory, where they cost none of it: about 2300
// cycles of shared memory a chunk with both there, 3200 without. Nothing in the state's
// chain depends on the state but one multiply-add per element (U does not), so a CTA is
// split into groups that meet at mbarriers and work on neighbouring chunks at once:
//     warps 0-7   the state update, S as bf16; o = e^{Gam_t} INTER + INTRA, stores
//     warps 8-11  v' of the next chunk
//     warps 12,13 scores: P; warp 12 issues QK, INTER and INTRA
//     warp 14     TMA loads, decays of the chunk, rows outside the sequence zeroed
//     warp 15     issues U
//
// Sequences are cut into segments when there are too few (sequence, head) pairs to
// fill the GPU: a first launch of the same kernel without its output half (OUT =
// false) forms each segment's own U, a small kernel turns those into the states
// at the segment starts, and the segments then run as independent items.
#include <algorithm>
#include <mutex>

#include "linear_internal.cuh"
#include "ptx.cuh"

namespace gdp {
namespace {

using namespace ptx;
using bf16 = __nv_bfloat16;

constexpr int C = 64;          // tokens per chunk
constexpr int kVT = 128;       // value columns per CTA
constexpr int kThreads = 512;
constexpr float kGMin = -1e5f;  // e^g is 0 far above this; keeps -inf out of the prefix sums

// ------------------------------------------------------------------ arithmetic
typedef unsigned long long f2;
__device__ __forceinline__ f2 pk2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 upk2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 sub2(f2 a, f2 b) {
  f2 d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// bf16x2 of (a, b): a in the low half.
__device__ __forceinline__ uint32_t cvt2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ f2 wide(uint32_t h) {  // the two bf16 as floats
  return pk2(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u));
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
// Below the normal range the result is 0; NaN passes.
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
  if (hi > 88.7f) return make_float2(__int_as_float(0x7f800000), 0.f);
  const float sc = __int_as_float((max(min((int)n, 127), -126) + 127) << 23);
  return make_float2(h * sc, l * sc);
}

// ------------------------------------------------------------------ work items
// A segment of a sequence: t0 = first row, n = rows, pos0 = tokens of the sequence before it
// (paged states: its context included), id = its place among the segments.
struct SegRec {
  int t0, n, seq, pos0;
  int first, last, id, pad;
};

struct ChunkArgs {
  LinearProblem p;
  const SegRec* recs;   // packed batches; seq = -1 past the last
  int nseg, Lseg;       // dense batches: segments per sequence, tokens per segment
  int slices;           // ceil(V / 128)
  int items;            // bound over all CTAs
  float* segS;          // [segments][HV][K][V]: U of a segment, then the state at its start
  float2* segW;         // [segments][HV]: its whole decay factor
};

struct Item {
  SegRec r;
  int b, hv, h, v0, off, chunks;
};

// Item `it` of the launch, value slices of a head and heads of a sequence side by side.
// (Not inlined: the roles' loops together have to fit the instruction cache.)
__device__ __noinline__ bool get_item(const ChunkArgs& a, int it, Item& x) {
  const int slice = it % a.slices, rest = it / a.slices;
  x.hv = rest % a.p.HV;
  x.h = x.hv / (a.p.HV / a.p.H);
  x.v0 = slice * kVT;
  const int s = rest / a.p.HV;
  if (a.recs) {
    const int4 u = reinterpret_cast<const int4*>(a.recs)[2 * s];
    const int4 w = reinterpret_cast<const int4*>(a.recs)[2 * s + 1];
    x.r = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, 0};
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
  }
  // chunks end where blocks do, so the first one may be short
  x.off = a.p.pool ? x.r.pos0 % C : 0;
  x.chunks = x.r.n > 0 ? (x.off + x.r.n + C - 1) / C : 0;
  return true;
}

// The k-th item of this CTA: rows of the grid in alternating directions, so that with items
// sorted by length the CTAs' sums stay close.
__device__ __forceinline__ int nth_item(int k) {
  const int g = (int)gridDim.x, c = (int)blockIdx.x;
  return k * g + ((k & 1) ? g - 1 - c : c);
}

// An item that this launch has nothing to do for (the state pass stops before a sequence's
// last segment).
template <bool OUT>
__device__ __forceinline__ bool skip(const Item& x) {
  return !OUT && x.r.last;
}

// ------------------------------------------------------------------ waits
struct Sync {
  volatile int* dead;  // a wait of this CTA ran out: everybody leaves
  int* status;
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    uint64_t t0 = 0;
    for (int i = 0; !mbar_test(bar, parity); ++i) {
      if ((i & 15) != 15) continue;
      if (*dead) return false;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitBudgetNs) {
        if (status) atomicExch(status, kDevTimeout);
        *dead = 1;
        return false;
      }
    }
    return true;
  }
  // by a whole warp, with one answer for all its lanes
  __device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait(bar, parity));
  }
};

// Barrier over the 256 state threads that combines a flag.
__device__ __forceinline__ bool state_and(bool pred) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 1, 256, p;\n"
               " selp.u32 %0, 1, 0, q;\n}\n" : "=r"(r) : "r"((uint32_t)pred) : "memory");
  return r != 0;
}

// ------------------------------------------------------------------ shared memory
template <int KD, bool OUT>
struct Lay {
  static constexpr int NST = 4;                         // stages of q, k, v
  static constexpr int KH = KD / 64;                    // 64-column halves of q and k
  static constexpr int QK = KH * 16384;                 // [q | k] by half, 64 rows of 128 bytes each
  static constexpr int STG = QK + 16384;                // then v, two halves
  static constexpr int P = NST * STG;                   // scores
  static constexpr int O = P + (OUT ? 8192 : 0);        // output tile, two halves
  // decays: more slots than stages, since the output still reads them when the stage is free
  static constexpr int G = O + (OUT ? 16384 : 0);
  static constexpr int GS = 272 * 4;                    // hi2, lo2, wend, ein [64] each, e^Gam hi, lo
  static constexpr int BAR = G + 8 * GS;
  static constexpr int BYTES = BAR + 256 + 1024;
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};
// full, ready, free by stage; v' ready and free by step; the rest single (B_O: INTER and INTRA)
enum {
  B_FULL = 0, B_READY = 4, B_FREE = 8, B_V = 12, B_VFREE = 16, B_QK = 20, B_O, B_OREAD, B_S, B_U, B_UREAD, B_N
};

// TMEM columns: scores [64], INTER and INTRA [64] each, U [KD], S [KD / 2], v' [3][32]
constexpr uint32_t T_QK = 0, T_INTER = 64, T_INTRA = 128, T_U = 192, T_S = 320, T_V = 384;

template <int KD, bool OUT>
__global__ void __launch_bounds__(kThreads, 1) linear_chunk_kernel(
    const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
    const __grid_constant__ ChunkArgs a) {
  using L = Lay<KD, OUT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + B_N);
  volatile int* s_dead = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_total = reinterpret_cast<int*>(s_tmem + 2);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const LinearProblem& p = a.p;

  if (warp == 0) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < B_N; ++i) {
      int n = 1;
      if (i >= B_FREE && i < B_V) n = OUT ? 2 : 1;                   // both issuing threads
      if (i == B_OREAD || i == B_S || i == B_UREAD) n = 8;           // state warps
      if (i >= B_V && i < B_VFREE) n = 4;                            // v' warps
      mbar_init(&bars[i], n);
    }
    fence_mbar_init();
    *s_dead = 0;
  }
  if (warp == 14 && lane == 0) {
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
    if (OUT) prefetch_tmap(&map_q);
  }
  pdl_wait();
  if (warp == 2) {  // chunks of this CTA over all its items
    int t = 0;
    for (int k = lane;; k += 32) {
      const int it = nth_item(k);
      Item x;
      if (it < a.items && get_item(a, it, x) && !skip<OUT>(x)) t += x.chunks;
      if (__all_sync(0xffffffffu, k * (int64_t)gridDim.x >= a.items)) break;
    }
    t = __reduce_add_sync(0xffffffffu, t);
    if (lane == 0) *s_total = t;
  }
  if (!a.recs && blockIdx.x == 0 && tid == 96 && p.status) *p.status = kDevOk;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int total = *s_total;
  const Sync sy{s_dead, p.status};
  const uint32_t smb = smem_u32(sm);
  auto gates = [&](int n) { return reinterpret_cast<float*>(sm + L::G + (n & 7) * L::GS); };
  // chunk n's tiles have landed, its decays are there and its foreign rows are zeroed
  auto tiles = [&](int n) {
    const uint32_t ph = (n / L::NST) & 1;
    return sy.wait_warp(&bars[B_READY + n % L::NST], ph) && sy.wait_warp(&bars[B_FULL + n % L::NST], ph);
  };
  const int K = p.K, V = p.V;

  if (warp < 8) {
    // ---------------------------------------------------------------- state, output
    constexpr int NC = KD / 2;  // state columns (k) per thread
    const int quarter = warp & 3, half = warp >> 2, cb = half * NC;
    const int row = quarter * 32 + lane;  // value column of the slice
    const uint32_t lb = tmem + ((uint32_t)(quarter * 32) << 16);
    // output tile: this warp's 32 value columns, 16-byte chunks 4 (quarter % 2) .. + 3 of row t in
    // the tile's half quarter / 2, permuted by t % 8; lane l gives row l % 8 of a block of 8 x 8
    const uint32_t orow = smb + L::O + (quarter >> 1) * 8192 + (half * 32 + (lane & 7)) * 128;
    const uint32_t oc = 4 * (quarter & 1) + (lane >> 3);
    float s[NC];
    int n = 0;
    bool ok = true;
    for (int kk = 0; ok && (int64_t)kk * gridDim.x < a.items; ++kk) {
      const int it = nth_item(kk);
      Item got;
      if (it >= a.items || !get_item(a, it, got) || skip<OUT>(got)) continue;
      const Item x = got;
      const bool von = x.v0 + row < V;
      const int64_t page_sz = (int64_t)K * V, at = (int64_t)x.hv * page_sz + x.v0 + row;
      auto page = [&](uint32_t end) {  // page of the state after token end - 1
        return p.pool + (int64_t)p.tables[(int64_t)x.r.seq * p.width + (end - 1) / (uint32_t)p.block] * p.HV * page_sz;
      };
      const float* src = nullptr;
      if (OUT) {
        // a split sequence's states all come from the scratch: its first page may be written by
        // its last segment meanwhile
        if (!(x.r.first && x.r.last)) src = a.segS + (int64_t)x.r.id * p.HV * page_sz;
        else if (p.pool) src = x.r.pos0 > 0 && x.r.n > 0 ? page(x.r.pos0) : nullptr;
        else if (p.s0) src = p.s0 + (int64_t)x.r.seq * p.HV * page_sz;
      }
      {
        const float* q = src ? src + at + (int64_t)cb * V : nullptr;
#pragma unroll
        for (int c = 0; c < NC; ++c, q += V) s[c] = src && von && cb + c < K ? __ldcg(q) : 0.f;
      }
      auto publish = [&] {  // the state as the A operand of INTER (whose last product is done)
#pragma unroll
        for (int q = 0; q < NC / 32; ++q) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = cvt2(s[32 * q + 2 * e], s[32 * q + 2 * e + 1]);
          GDP_TMEM_ST16(lb + T_S + cb / 2 + 16 * q, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_S]);
      };
      if (OUT && x.chunks > 0) publish();
      float2 wseg = make_float2(1.f, 0.f);
      for (int c = 0; c < x.chunks; ++c, ++n) {
        // a failed wait leaves through the barrier below, with the whole group
        ok = sy.wait_warp(&bars[B_U], n & 1);
        if (!OUT && !ok) break;
        tc_fence_after();
        const float* g = gates(n);
        const float wh = g[256], wl = g[257];
        const f2 wh2 = pk2(wh, wh), wl2 = pk2(wl, wl);
#pragma unroll
        for (int q = 0; q < NC / 32; ++q) {
          uint32_t r[32];
          GDP_TMEM_LD32(lb + T_U + cb + 32 * q, r);
          tmem_wait_ld();
          if (q == NC / 32 - 1) {  // the next U may overwrite this one
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_UREAD]);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float* d = s + 32 * q + e;
            const f2 old = pk2(d[0], d[1]);
            const float2 f = upk2(fma2(wh2, old, fma2(wl2, old, pk2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])))));
            d[0] = f.x;
            d[1] = f.y;
          }
        }
        const bool more = c + 1 < x.chunks;
        float* dst = nullptr;  // where the state after this chunk is kept
        if (!OUT) {            // the segment's whole decay, pair by pair
          const float ph = wseg.x * wh;
          const float pl = fmaf(wseg.x, wh, -ph) + (wseg.x * wl + wseg.y * wh);
          wseg.x = ph + pl;
          wseg.y = pl - (wseg.x - ph);
          if (!more) {
            dst = a.segS + (int64_t)x.r.id * p.HV * page_sz;
            if (row == 0 && cb == 0) a.segW[(int64_t)x.r.id * p.HV + x.hv] = wseg;
          }
        } else if (p.pool) {
          const uint32_t end = (uint32_t)(x.r.pos0 - x.off) + (uint32_t)(c + 1) * C;
          if ((!more && x.r.last) || end % (uint32_t)p.block == 0) dst = page(min(end, (uint32_t)x.r.pos0 + (uint32_t)x.r.n));
        } else if (!more && x.r.last && p.sT) {
          dst = p.sT + (int64_t)x.r.seq * p.HV * page_sz;
        }
        if (OUT) {
        ok = sy.wait_warp(&bars[B_O], n & 1) && ok;
        tc_fence_after();
        if (more && ok) publish();
        // o of 16 value columns at a time, as fragments: pairs of rows t in a register
        const float* ein = g + 192 + 32 * half + 2 * (lane & 3);
        uint32_t out[16];  // by t block of 8, value block of 8
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t r[16], w[16];
          GDP_TMEM_LD_16X256_X4(lb + (q << 20) + T_INTER + 32 * half, r);
          GDP_TMEM_LD_16X256_X4(lb + (q << 20) + T_INTRA + 32 * half, w);
          tmem_wait_ld();
          if (q == 1) {  // the next products may overwrite these
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_OREAD]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 e = *reinterpret_cast<const float2*>(ein + 8 * j);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int i = 4 * j + 2 * u;
              const float2 f = upk2(fma2(pk2(e.x, e.y), pk2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])),
                                         pk2(__uint_as_float(w[i]), __uint_as_float(w[i + 1]))));
              out[4 * j + 2 * q + u] = cvt2(f.x, f.y);
            }
          }
        }
        // the previous chunk's stores have read the tile
        if (tid == 0) tma_store_wait_read();
        if (!(ok = state_and(ok))) break;
#pragma unroll
        for (int j = 0; j < 4; ++j)  // rows 8 j .. of this half; lanes 8 m .. address value block m
          stmatrix_x4_trans(orow + j * 1024 + ((oc ^ (lane & 7)) << 4), out[4 * j], out[4 * j + 1], out[4 * j + 2],
                            out[4 * j + 3]);
        // rows of the tile inside the sequence
        const int base = x.r.t0 - x.off + c * C;
        const int lo = max(0, x.r.t0 - base), hi = min(C, x.r.t0 + x.r.n - base);
        const bool whole = lo == 0 && (hi == C || (!a.recs && x.r.last));
        if (whole) {  // rows past a dense batch's end are clipped by the map
          fence_async_smem();
          state_and(true);
          if (tid == 0) {
            tma_store_4d(&map_o, sm + L::O, x.v0, x.hv, base, x.b);
            if (x.v0 + 64 < V) tma_store_4d(&map_o, sm + L::O + 8192, x.v0 + 64, x.hv, base, x.b);
            tma_store_commit();
          }
        } else {
          state_and(true);
          bf16* og = static_cast<bf16*>(p.o) + (((int64_t)x.b * p.T + base) * p.HV + x.hv) * V + x.v0;
          const int j = tid & 15, c8 = 8 * j;  // 16-byte piece of the row (V is a multiple of 8)
          if (x.v0 + c8 < V)
            for (int t = lo + (tid >> 4); t < hi; t += 16)
              *reinterpret_cast<uint4*>(og + (int64_t)t * p.HV * V + c8) =
                  *reinterpret_cast<const uint4*>(sm + L::O + (j >> 3) * 8192 + t * 128 + (((j & 7) ^ (t & 7)) << 4));
          // the next chunk's barrier orders these reads before its writes
        }
        }
        if (dst && von) {
          dst += at + (int64_t)cb * V;
#pragma unroll
          for (int c2 = 0; c2 < NC; ++c2, dst += V)
            if (cb + c2 < K) *dst = s[c2];
        }
      }
      if (!ok) break;
      if (OUT && x.chunks == 0 && p.sT && von && x.r.last) {  // an empty sequence keeps its state
        float* dst = p.sT + (int64_t)x.r.seq * p.HV * page_sz + at;
        src += src ? at : 0;
#pragma unroll 1
        for (int k = cb; k < min(cb + NC, K); ++k) dst[(int64_t)k * V] = src ? __ldcg(src + (int64_t)k * V) : 0.f;
      }
    }
    if (OUT && tid == 0) tma_store_wait_all();
  } else if (warp < 12) {
    // ---------------------------------------------------------------- v'
    const int quarter = warp & 3;
    const uint32_t lb = tmem + ((uint32_t)(quarter * 32) << 16) + T_V;
    // transposing loads: lanes 8 m .. 8 m + 7 address rows i of value block m (16-byte chunk
    // 4 (quarter % 2) + m, permuted by i % 8)
    const uint32_t vrow = L::QK + (quarter >> 1) * 8192 + (lane & 7) * 128 +
                          (((4 * (quarter & 1) + (lane >> 3)) ^ (lane & 7)) << 4);
    bool ok = true;
    for (int n = 0; n < total && ok; ++n) {
      if (!tiles(n)) break;
      uint32_t va = smb + (n % L::NST) * L::STG + vrow;
      const float* g = gates(n) + 128 + 2 * (lane & 3);
      // a step of U (16 positions) at a time, each as soon as U(n - 1) has read its own
#pragma unroll 1
      for (int ks = 0; ks < 4; ++ks, va += 2048, g += 16) {
        // register 4 hh + m: positions 8 hh + 2 (l % 4), + 1 of value column 8 m + l / 4
        uint32_t e[8], h[8], m[8], l[8];
        ldmatrix_x4_trans(va, e);
        ldmatrix_x4_trans(va + 1024, e + 4);
        const float2 w0 = *reinterpret_cast<const float2*>(g), w1 = *reinterpret_cast<const float2*>(g + 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f2 y = mul2(wide(e[i]), i < 4 ? pk2(w0.x, w0.y) : pk2(w1.x, w1.y));
          float2 f = upk2(y);
          h[i] = cvt2(f.x, f.y);
          y = sub2(y, wide(h[i]));
          f = upk2(y);
          m[i] = cvt2(f.x, f.y);
          f = upk2(sub2(y, wide(m[i])));
          l[i] = cvt2(f.x, f.y);
        }
        if (n > 0 && !(ok = sy.wait_warp(&bars[B_VFREE + ks], (n - 1) & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // lanes (value columns) 16 q .. 16 q + 15
          const uint32_t d = lb + (q << 20) + 8 * ks;
          GDP_TMEM_ST_16X128_X2(d, h[2 * q], h[2 * q + 1], h[2 * q + 4], h[2 * q + 5]);
          GDP_TMEM_ST_16X128_X2(d + 32, m[2 * q], m[2 * q + 1], m[2 * q + 4], m[2 * q + 5]);
          GDP_TMEM_ST_16X128_X2(d + 64, l[2 * q], l[2 * q + 1], l[2 * q + 4], l[2 * q + 5]);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_V + ks]);
      }
    }
  } else if (warp < 14) {
    // ---------------------------------------------------------------- scores
    if (OUT) {
      const int t = (warp - 12) * 32 + lane;
      const uint32_t lb = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const f2 sc2 = pk2(p.scale, p.scale);
      const uint32_t id_qk = idesc_bf16(128, 64, false, false);  // and of INTER
      const uint32_t id_a = idesc_bf16(128, 64, true, false);
      auto qk = [&](int n) {  // warp 12
        if (elect_one()) {
          tc_fence_after();
          const uint32_t tl = smb + (n % L::NST) * L::STG;
          mma_run<KD / 16, false, 16384, 32, 16384, 32>(tmem + T_QK, sdesc_sw128(tl, 16, 1024),
                                                        sdesc_sw128(tl + 8192, 16, 1024), id_qk);
          mma_commit(&bars[B_QK]);
        }
        __syncwarp();
      };
      bool ok = true;
      if (warp == 12 && total > 0 && (ok = tiles(0))) qk(0);
      for (int n = 0; n < total; ++n) {
        ok = sy.wait_warp(&bars[B_QK], n & 1) && ok;
        tc_fence_after();
        if (n > 0) ok = sy.wait_warp(&bars[B_O], (n - 1) & 1) && ok;  // INTRA(n - 1) has read P
        const float* g = gates(n);
        const f2 hi = pk2(g[t], g[t]), lo = pk2(g[64 + t], g[64 + t]);
        uint8_t* pt = sm + L::P;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[8];
          if (q >= 2 && warp == 12) {  // columns past every row of this warp
#pragma unroll
            for (int e = 0; e < 8; ++e) pk[e] = 0;
          } else {
            uint32_t r[16];
            GDP_TMEM_LD16(lb + T_QK + 16 * q, r);
            tmem_wait_ld();
            const int ti = t - 16 * q;  // columns i <= ti are this row's
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 h4 = *reinterpret_cast<const float4*>(g + 16 * q + e);
              const float4 l4 = *reinterpret_cast<const float4*>(g + 64 + 16 * q + e);
              const float2 x0 = upk2(add2(sub2(hi, pk2(h4.x, h4.y)), sub2(lo, pk2(l4.x, l4.y))));
              const float2 x1 = upk2(add2(sub2(hi, pk2(h4.z, h4.w)), sub2(lo, pk2(l4.z, l4.w))));
              const float2 y0 = upk2(mul2(mul2(pk2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), sc2),
                                          pk2(ex2_approx(x0.x), ex2_approx(x0.y))));
              const float2 y1 = upk2(mul2(mul2(pk2(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3])), sc2),
                                          pk2(ex2_approx(x1.x), ex2_approx(x1.y))));
              pk[e / 2] = cvt2(e <= ti ? y0.x : 0.f, e + 1 <= ti ? y0.y : 0.f);
              pk[e / 2 + 1] = cvt2(e + 2 <= ti ? y1.x : 0.f, e + 3 <= ti ? y1.y : 0.f);
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
            *reinterpret_cast<uint4*>(pt + sw128_offset(t, (16 * q + 8 * j) * 2)) =
                make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
        }
        fence_async_smem();
        tc_fence_before();
        // both warps have read the scores and written P
        uint32_t all;
        asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 2, 64, p;\n"
                     " selp.u32 %0, 1, 0, q;\n}\n" : "=r"(all) : "r"((uint32_t)ok) : "memory");
        if (!(ok = all != 0)) break;
        if (warp == 12) {
          // the next scores go first if their tiles are there
          bool ahead = n + 1 == total;
          if (!ahead && __all_sync(0xffffffffu, mbar_poll(&bars[B_READY + (n + 1) % L::NST], ((n + 1) / L::NST) & 1))) {
            ok = tiles(n + 1);
            qk(n + 1);
            ahead = true;
          }
          // the state before the chunk is published before the last output is read
          if (n > 0) ok = sy.wait_warp(&bars[B_OREAD], (n - 1) & 1) && ok;
          ok = sy.wait_warp(&bars[B_S], n & 1) && ok;
          if (ok && elect_one()) {
            tc_fence_after();
            mma_run_ts<KD / 16, false, 16384, 32>(tmem + T_INTER, tmem + T_S,
                                                  sdesc_sw128(smb + (n % L::NST) * L::STG, 16, 1024), id_qk);
            mma_run<4, false, 0, 2048, 0, 32>(tmem + T_INTRA, sdesc_sw128(smb + (n % L::NST) * L::STG + L::QK, 8192, 1024),
                                              sdesc_sw128(smb + L::P, 16, 1024), id_a);
            mma_commit(&bars[B_O]);
            mma_commit(&bars[B_FREE + n % L::NST]);
          }
          __syncwarp();
          if (!ahead) {
            ok = tiles(n + 1) && ok;
            if (ok) qk(n + 1);
          }
        }
      }
    }
  } else if (false) {
    // ---------------------------------------------------------------- loads, decays
    int n = 0;
    bool ok = true;
    int nl = 0, lk = -1, lc = 0;  // next load: chunk lc of this CTA's item lk
    Item lx;
    lx.chunks = 0;
    // the tiles of the next chunks, up to a ring ahead of chunk n; a stage that is not free yet is
    // waited for only if chunk n itself is still to load
    auto loads = [&](int now) {
      while (nl < total && nl < now + L::NST) {
        const int st = nl % L::NST;
        if (nl >= L::NST) {
          const uint32_t ph = (nl / L::NST - 1) & 1;
          if (nl > now) {
            if (!__all_sync(0xffffffffu, mbar_poll(&bars[B_FREE + st], ph))) return true;
          } else if (!sy.wait_warp(&bars[B_FREE + st], ph)) {
            return false;
          }
        }
        while (lc >= lx.chunks) {
          ++lk;
          lc = 0;
          const int it = nth_item(lk);
          if (it >= a.items || !get_item(a, it, lx) || skip<OUT>(lx)) lx.chunks = 0;
        }
        if (elect_one()) {
          const int t = lx.r.t0 - lx.off + lc * C;
          const bool two = lx.v0 + 64 < V;
          uint8_t* tile = sm + st * L::STG;
          uint64_t* bar = &bars[B_FULL + st];
          mbar_expect_tx(bar, 8192 * ((OUT ? 2 : 1) * L::KH + (two ? 2 : 1)));
#pragma unroll
          for (int hh = 0; hh < L::KH; ++hh) {
            if (OUT) tma_load_4d(tile + hh * 16384, &map_q, 64 * hh, lx.h, t, lx.b, bar);
            tma_load_4d(tile + hh * 16384 + 8192, &map_k, 64 * hh, lx.h, t, lx.b, bar);
          }
          tma_load_4d(tile + L::QK, &map_v, lx.v0, lx.hv, t, lx.b, bar);
          if (two) tma_load_4d(tile + L::QK + 8192, &map_v, lx.v0 + 64, lx.hv, t, lx.b, bar);
        }
        __syncwarp();
        ++lc;
        ++nl;
      }
      return true;
    };
    loads(0);
    for (int kk = 0; ok && (int64_t)kk * gridDim.x < a.items; ++kk) {
      const int it = nth_item(kk);
      Item got;
      if (it >= a.items || !get_item(a, it, got) || skip<OUT>(got)) continue;
      const Item x = got;
      const float* gb = !p.g ? nullptr : p.g_token ? p.g + (int64_t)x.b * p.T * p.HV + x.hv : p.g + x.hv;
      auto load = [&](int c, int u) {  // g at position 2 lane + u of chunk c
        const int r = x.r.t0 - x.off + c * C + 2 * lane + u;
        if (!gb || r < x.r.t0 || r >= x.r.t0 + x.r.n) return 0.f;
        const float y = p.g_token ? __ldg(gb + (int64_t)r * p.HV) : __ldg(gb);
        return y < kGMin ? kGMin : y;
      };
      float nx0 = load(0, 0), nx1 = load(0, 1);
      for (int c = 0; c < x.chunks; ++c, ++n) {
        const int st = n % L::NST;
        // compensated inclusive prefix of 64 values, two per lane
        float e1;
        const float s0 = nx0, s1 = two_sum(nx0, nx1, e1);
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
        h[0] = two_sum(pS, s0, e);
        l[0] = pE + e;
        h[1] = two_sum(pS, s1, e);
        l[1] = (pE + e1) + e;
        const float hl = __shfl_sync(0xffffffffu, h[1], 31), ll = __shfl_sync(0xffffffffu, l[1], 31);
        if (c + 1 < x.chunks) {
          nx0 = load(c + 1, 0);
          nx1 = load(c + 1, 1);
        }
        const float2 w = exp_pair(hl, ll), bl = log2e_pair(hl, ll);
        const int base = x.r.t0 - x.off + c * C;
        const int lo = max(0, x.r.t0 - base), hi = min(C, x.r.t0 + x.r.n - base);
        float2 b2[2];
        float we[2], ei[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = 2 * lane + u;
          b2[u] = log2e_pair(h[u], l[u]);
          // 2^x is good to 2^-22; a rounded exponent matters less the smaller the factor
          we[u] = i >= lo && i < hi ? ex2_approx((bl.x - b2[u].x) + (bl.y - b2[u].y)) : 0.f;
          ei[u] = p.scale * ex2_approx(b2[u].x + b2[u].y);
        }
        if (!(ok = loads(n) && sy.wait_warp(&bars[B_FULL + st], (n / L::NST) & 1))) break;
        float* g = gates(n);
        *reinterpret_cast<float2*>(g + 2 * lane) = make_float2(b2[0].x, b2[1].x);
        *reinterpret_cast<float2*>(g + 64 + 2 * lane) = make_float2(b2[0].y, b2[1].y);
        *reinterpret_cast<float2*>(g + 128 + 2 * lane) = make_float2(we[0], we[1]);
        *reinterpret_cast<float2*>(g + 192 + 2 * lane) = make_float2(ei[0], ei[1]);
        if (lane == 0) *reinterpret_cast<float2*>(g + 256) = w;
        if (lo > 0 || hi < C) {
          // rows of other sequences, or past the end: k and v as zeros, so that nothing in
          // them (not even a NaN) enters a sum over the rows
          uint8_t* tile = sm + st * L::STG;
          for (int i = lane >> 3; i < C; i += 4)
            if (i < lo || i >= hi) {
              const uint32_t o = i * 128 + (lane & 7) * 16;
#pragma unroll
              for (int hh = 0; hh < L::KH; ++hh)
                *reinterpret_cast<uint4*>(tile + hh * 16384 + 8192 + o) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(tile + L::QK + o) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(tile + L::QK + 8192 + o) = make_uint4(0, 0, 0, 0);
            }
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_READY + st]);
        if (!(ok = loads(n + 1))) break;
      }
    }
    // nothing may still write shared memory when the CTA leaves
    for (int m = max(0, nl - L::NST); m < nl; ++m) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_test(&bars[B_FULL + m % L::NST], (m / L::NST) & 1) && globaltimer_ns() - t0 < kWaitBudgetNs) {}
    }
  } else {
    // ---------------------------------------------------------------- U
    const uint32_t id_u = idesc_bf16(128, KD, false, true);
    for (int n = 0; n < total; ++n) {
      bool ok = tiles(n);
      if (n > 0) ok = sy.wait_warp(&bars[B_UREAD], (n - 1) & 1) && ok;
      const uint64_t kd = sdesc_sw128(smb + (n % L::NST) * L::STG + 8192, 16384, 1024);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        ok = ok && sy.wait_warp(&bars[B_V + ks], n & 1);
        if (!ok) break;
        if (elect_one()) {
          tc_fence_after();
          const uint64_t k = kd + ((ks * 2048) >> 4);
          const uint32_t av = tmem + T_V + 8 * ks;
          if (ks == 0) mma_bf16_ts<false>(tmem + T_U, av + 64, k, id_u);
          else mma_bf16_ts<true>(tmem + T_U, av + 64, k, id_u);
          mma_bf16_ts<true>(tmem + T_U, av + 32, k, id_u);
          mma_bf16_ts<true>(tmem + T_U, av, k, id_u);
          mma_commit(&bars[B_VFREE + ks]);
          if (ks == 3) {
            mma_commit(&bars[B_U]);
            mma_commit(&bars[B_FREE + n % L::NST]);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
    }
  }
  __syncwarp();
  if (*s_dead) {  // products in flight end before their operands and columns go away
    if (warp == 15 && lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) {}  // a chunk's products take microseconds
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ segments
// Segment records of a packed batch (one CTA): offsets and block tables checked as in
// linear_records_kernel, each sequence cut at multiples of Lseg positions, records sorted by
// length, longest first.
constexpr int kRecThreads = 512;
constexpr int kSortMax = 4096;

__device__ __forceinline__ int table_page(const LinearProblem& p, int r, int64_t b) {
  if (b < 0 || b >= p.width) return -1;
  const int pg = p.tables[(int64_t)r * p.width + b];
  return pg >= 0 && pg < p.n_pages ? pg : -1;
}

__global__ void __launch_bounds__(kRecThreads) linear_segments_kernel(const __grid_constant__ LinearProblem p,
                                                                      int Lseg, int bound, SegRec* recs, int2* seqs) {
  pdl_wait();
  __shared__ int lens[kSortMax];
  __shared__ int wsum[kRecThreads / 32 + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  for (int i = tid; i < p.N_seq; i += kRecThreads) {
    const int x = p.cu[i], y = p.cu[i + 1];
    bad |= x < 0 || y < x || y > p.T;
  }
  bad = __syncthreads_or(bad);
  bool any = bad;
  int base = 0;  // segments before this round of sequences
  for (int i0 = 0; i0 < p.N_seq; i0 += kRecThreads) {
    const int i = i0 + tid;
    int t0 = 0, n = 0, pos = 0, cnt = 0;
    if (i < p.N_seq) {
      if (!bad) {
        t0 = p.cu[i];
        n = p.cu[i + 1] - t0;
      }
      if (p.pool && n > 0) {
        pos = p.ctx[i];
        bool off = pos < 0;
        if (!off)
          for (int64_t j = pos > 0 ? (pos - 1) / p.block : 0; j <= ((int64_t)pos + n - 1) / p.block; ++j)
            off |= table_page(p, i, j) < 0;
        if (off) n = pos = 0;
        any |= off;
      }
      cnt = n > 0 ? (int)(((int64_t)pos % C + n + Lseg - 1) / Lseg) : 1;
    }
    int s = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    if (lane == 31) wsum[warp] = s;
    __syncthreads();
    if (tid == 0) {
      int run = 0;
      for (int w = 0; w < kRecThreads / 32; ++w) {
        const int y = wsum[w];
        wsum[w] = run;
        run += y;
      }
      wsum[kRecThreads / 32] = run;
    }
    __syncthreads();
    const int first = base + wsum[warp] + s - cnt;
    base += wsum[kRecThreads / 32];
    if (i < p.N_seq) {
      if (seqs) seqs[i] = make_int2(first, cnt);
      const int off = pos % C;
      for (int j = 0; j < cnt; ++j) {
        const int lo = j == 0 ? 0 : j * Lseg - off, hi = min(n, (j + 1) * Lseg - off);
        SegRec r{t0 + lo, hi - lo, i, p.pool ? pos + lo : lo, j == 0, j == cnt - 1, first + j, 0};
        recs[first + j] = r;
        if (first + j < kSortMax) lens[first + j] = r.n;
      }
    }
    __syncthreads();
  }
  any = __syncthreads_or(any);
  if (tid == 0 && p.status) *p.status = any ? kDevBadSeqlens : kDevOk;
  const int count = base;
  if (count <= kSortMax && count > 1) {  // in place: every thread reads its records first
    SegRec mine[kSortMax / kRecThreads];
    int rank[kSortMax / kRecThreads];
#pragma unroll
    for (int q = 0; q < kSortMax / kRecThreads; ++q) {
      const int i = tid + q * kRecThreads;
      if (i < count) {
        mine[q] = recs[i];
        int r = 0;
        const int len = lens[i];
        for (int j = 0; j < count; ++j) r += lens[j] > len || (lens[j] == len && j < i);
        rank[q] = r;
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSortMax / kRecThreads; ++q)
      if (tid + q * kRecThreads < count) recs[rank[q]] = mine[q];
  }
  for (int i = count + tid; i < bound; i += kRecThreads) recs[i] = SegRec{0, 0, -1, 0, 0, 0, 0, 0};
}

// States at the segment starts: S_0 = the sequence's initial state, S_{j+1} = w_j S_j + U_j,
// in place of the U's. A thread per four state elements.
__global__ void __launch_bounds__(256) linear_combine_kernel(const __grid_constant__ ChunkArgs a, const int2* seqs) {
  pdl_wait();
  const LinearProblem& p = a.p;
  const int64_t sz = (int64_t)p.K * p.V;
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int hv = blockIdx.y, seq = blockIdx.z;
  int first, cnt;
  if (a.recs) {
    const int2 x = seqs[seq];
    first = x.x;
    cnt = x.y;
  } else {
    first = seq * a.nseg;
    cnt = a.nseg;
  }
  if (cnt < 2 || e >= sz) return;
  const float* src = nullptr;
  if (p.pool) {
    const int c = p.ctx[seq];
    if (c > 0) src = p.pool + (int64_t)p.tables[(int64_t)seq * p.width + (c - 1) / p.block] * p.HV * sz;
  } else if (p.s0) {
    src = p.s0 + (int64_t)seq * p.HV * sz;
  }
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (src) s = __ldcg(reinterpret_cast<const float4*>(src + hv * sz + e));
  float4* seg = reinterpret_cast<float4*>(a.segS + ((int64_t)first * p.HV + hv) * sz + e);
  const int64_t step = (int64_t)p.HV * sz / 4;
  const float2* w = a.segW + (int64_t)first * p.HV + hv;
  for (int j0 = 0; j0 + 1 < cnt; j0 += 8) {  // eight segments' loads in flight
    const int m = min(8, cnt - 1 - j0);
    float4 u[8];
    float2 f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < m) {
        u[j] = __ldcg(seg + (j0 + j) * step);
        f[j] = __ldcg(w + (int64_t)(j0 + j) * p.HV);
      }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < m) {
        seg[(j0 + j) * step] = s;
        s.x = fmaf(f[j].x, s.x, fmaf(f[j].y, s.x, u[j].x));
        s.y = fmaf(f[j].x, s.y, fmaf(f[j].y, s.y, u[j].y));
        s.z = fmaf(f[j].x, s.z, fmaf(f[j].y, s.z, u[j].z));
        s.w = fmaf(f[j].x, s.w, fmaf(f[j].y, s.w, u[j].w));
      }
  }
  seg[(int64_t)(cnt - 1) * step] = s;
}

// ------------------------------------------------------------------ host
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

// [B][T][heads][width] with element strides s (batch, token, head); boxes of 64 x 1 x 64 x 1.
bool map4(CUtensorMap* m, const void* base, int width, int heads, int T, int B, const int64_t* s) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
  // the stride of a dimension of one entry is never used; the encoder wants a valid one
  const cuuint64_t some = 16;
  const cuuint64_t st[3] = {heads > 1 ? (cuuint64_t)s[2] * 2 : some, T > 1 ? (cuuint64_t)s[1] * 2 : some,
                            B > 1 ? (cuuint64_t)s[0] * 2 : some};
  const cuuint32_t box[4] = {64, 1, 64, 1}, es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, st, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_ok(const void* base, int heads, int T, int B, const int64_t* s) {
  const auto fits = [](int n, int64_t x) { return n <= 1 || (x > 0 && x % 8 == 0 && x < ((int64_t)1 << 38)); };
  return reinterpret_cast<uintptr_t>(base) % 16 == 0 && fits(heads, s[2]) && fits(T, s[1]) && fits(B, s[0]);
}

struct Plan {
  int nseg, Lseg, bound, slices;  // segments per dense sequence, tokens, segments in all at most
  size_t recs, seqs, segS, segW, total;
};

Plan plan_of(int N_seq, int B, int T, int HV, int K, int V, bool packed) {
  Plan x{};
  const int G = sm_count();
  x.slices = (int)cdiv(V, kVT);
  const int chunks = (int)cdiv(T, C);
  const int64_t heads = (int64_t)HV * x.slices;
  x.nseg = 1;
  x.Lseg = std::max(1, chunks) * C;
  if (!packed) {
    // time in units of a chunk of the second pass: rounds of items over the SMs, with the state
    // pass at 0.6 of that and its two extra launches at about eight chunks
    const int64_t units = heads * B;
    double best = (double)cdiv(units, G) * chunks;
    for (int n = 2; n <= chunks && n <= 64; ++n) {
      const int64_t per = cdiv(chunks, n);
      if (cdiv(chunks, per) != n) continue;  // fewer segments of this length do
      const double t = (double)cdiv(units * n, G) * per + 0.6 * cdiv(units * (n - 1), G) * per + 8.0;
      if (t < 0.95 * best) {
        best = t;
        x.nseg = n;
        x.Lseg = (int)per * C;
      }
    }
    x.bound = B * x.nseg;
  } else {
    // packed: no more than an SM's share of the whole batch in one item
    const int64_t share = cdiv(cdiv((int64_t)T * heads, G), C) * C;
    x.Lseg = (int)std::min<int64_t>(x.Lseg + C, std::max<int64_t>(share, 512));
    x.bound = (int)(((int64_t)T + (int64_t)N_seq * C) / x.Lseg + N_seq);
  }
  const bool split = packed ? x.Lseg < T : x.nseg > 1;
  x.recs = kAlign;
  x.seqs = align_up(x.recs + (packed ? (size_t)x.bound * sizeof(SegRec) : 0));
  x.segW = align_up(x.seqs + (packed ? (size_t)N_seq * sizeof(int2) : 0));
  x.segS = align_up(x.segW + (split ? (size_t)x.bound * HV * sizeof(float2) : 0));
  x.total = align_up(x.segS + (split ? (size_t)x.bound * HV * K * V * 4 : 0));
  if (!split) x.segS = 0;
  return x;
}

template <int KD, bool OUT>
cudaError_t go(const ChunkArgs& a, const CUtensorMap* m) {
  constexpr int smem = Lay<KD, OUT>::BYTES;
  auto kern = linear_chunk_kernel<KD, OUT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(std::min(a.items, sm_count())), dim3(kThreads), smem, a.p.stream, m[0], m[1], m[2],
                    m[3], a);
}

}  // namespace

bool linear_tc_shape(int K, int V, gdp_dtype dt) { return dt == GDP_BF16 && K <= 128 && K % 8 == 0 && V % 8 == 0; }

size_t linear_tc_workspace(int N_seq, int B, int T, int HV, int K, int V) {
  // the query does not say whether the batch is packed
  const size_t d = N_seq == B ? plan_of(N_seq, B, T, HV, K, V, false).total : 0;
  return std::max(d, B == 1 ? plan_of(N_seq, B, T, HV, K, V, true).total : 0);
}

bool linear_tc_ok(const LinearProblem& p) {
  return linear_tc_shape(p.K, p.V, p.dt) && map_ok(p.q, p.H, p.T, p.B, p.qs) && map_ok(p.k, p.H, p.T, p.B, p.ks) &&
         map_ok(p.v, p.HV, p.T, p.B, p.vs) && p.N_seq <= 65535 && p.HV <= 65535 && reinterpret_cast<uintptr_t>(p.o) % 16 == 0;
}

cudaError_t launch_linear_tc(const LinearProblem& p, uint8_t* ws) {
  const Plan x = plan_of(p.N_seq, p.B, p.T, p.HV, p.K, p.V, p.cu != nullptr);
  ChunkArgs a{};
  a.p = p;
  a.nseg = x.nseg;
  a.Lseg = x.Lseg;
  a.slices = x.slices;
  if ((int64_t)x.bound * p.HV * x.slices > INT32_MAX - 65536) return cudaErrorInvalidValue;
  a.items = x.bound * p.HV * x.slices;
  if (a.items == 0) return cudaSuccess;
  int2* seqs = nullptr;
  if (p.cu) {
    SegRec* recs = reinterpret_cast<SegRec*>(ws + x.recs);
    seqs = reinterpret_cast<int2*>(ws + x.seqs);
    a.recs = recs;
    cudaError_t e = launch_pdl(linear_segments_kernel, dim3(1), dim3(kRecThreads), 0, p.stream, p, x.Lseg, x.bound,
                               recs, seqs);
    if (e != cudaSuccess) return e;
  }
  CUtensorMap m[4];
  const int64_t os[3] = {(int64_t)p.T * p.HV * p.V, (int64_t)p.HV * p.V, p.V};
  if (!map4(&m[0], p.q, p.K, p.H, p.T, p.B, p.qs) || !map4(&m[1], p.k, p.K, p.H, p.T, p.B, p.ks) ||
      !map4(&m[2], p.v, p.V, p.HV, p.T, p.B, p.vs) || !map4(&m[3], p.o, p.V, p.HV, p.T, p.B, os))
    return cudaErrorInvalidValue;
  if (x.segS) {
    a.segS = reinterpret_cast<float*>(ws + x.segS);
    a.segW = reinterpret_cast<float2*>(ws + x.segW);
    cudaError_t e = p.K > 64 ? go<128, false>(a, m) : go<64, false>(a, m);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)cdiv((int64_t)p.K * p.V, 1024), p.HV, p.N_seq);
    e = launch_pdl(linear_combine_kernel, grid, dim3(256), 0, p.stream, a, (const int2*)seqs);
    if (e != cudaSuccess) return e;
  }
  return p.K > 64 ? go<128, true>(a, m) : go<64, true>(a, m);
}

}  // namespace gdp
