// Linear attention with a decay for each head, chunked form on the tensor cores:
// bf16 inputs, K <= 128, any V in slices of 128 columns.
//
// With Gam_t the sum of g over a chunk's tokens up to t, S the state before the
// chunk and Gam the chunk's whole sum,
//     o_t = scale (e^{Gam_t} S^T q_t + sum_{i <= t} e^{Gam_t - Gam_i} (q_t . k_i) v_i),
//     S  <- e^{Gam} S + sum_i k_i (e^{Gam - Gam_i} v_i)^T.
// Four products per chunk of 64 tokens, with the value columns on the 128 rows of
// the tensor core's accumulator wherever the product has them:
//     QK     [t | i]  = q k^T            (64 rows: 16 in each warp's quarter of the lanes)
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
// What bounds it: q, k, v, o are 64 KB per chunk and head, 1.5 us of an SM's share of HBM (36 KB, 0.8
// us, where eight items of a key head share its q and k through the L2).
// A product with both operands in shared memory runs at that memory's 128 bytes a clock
// ((A + B) / 128 cycles, measured), more than the tensor pipe needs, so the operands that
// are made on chip (S, v') live in tensor memory, where they cost none of it. Nothing in the
// state's chain depends on the state but one multiply-add per element (U does not), so a CTA is
// split into groups that meet at mbarriers and work on neighbouring chunks at once:
//     8 state warps   the state update, S as bf16; o = e^{Gam_t} INTER + INTRA, stores
//     4 v' warps      v' of the next chunk
//     4 score warps   P
//     1 warp          decays of the chunk, rows outside the sequence zeroed
//     1 warp          TMA loads, issues QK
//     2 warps         issue U, and INTER with INTRA
// The roles' loops are rolled where they can be: together they have to fit the 32 KB
// first-level instruction cache, or the SMs of a GPC wait for their common next level (with
// them unrolled a third of the warps' time went there, at 80 % of that cache's bandwidth).
// Measured: 1.8 us a chunk (K = V = 128), 1.2 in the state pass, 9.4 us for a call of one chunk;
// 2 x 4096 tokens, 16 heads: 70 us with the state pass and the combine kernel. What is left above
// the bytes is a stage's round trip over its three places: 1.4 us for a load to land, as long
// again for v' at the rate that four warps reach beside the others, then U and INTRA. Measured in
// place of it: four stages with one P buffer, 73 us; a step of v' on the score warps, 72; sixteen
// state and four output warps at 64 registers, 78 (as eight then were).
//
// Sequences are cut into segments when there are too few (sequence, head) pairs to
// fill the GPU: a first launch of the same kernel without its output half (OUT =
// false) forms each segment's own U, a small kernel turns those into the states
// at the segment starts, and the segments then run as independent items.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "linear_chunk.cuh"
#include "ptx.cuh"

namespace gdp {
namespace {

using namespace ptx;
using namespace linear;
using bf16 = __nv_bfloat16;

constexpr int kVT = 128;       // value columns per CTA
constexpr int kSW = 8;             // state warps; then the v' warps
constexpr int kScore = kSW + 4;    // first of the four score warps
constexpr int kDecay = kScore + 4;  // decays; then the issuers of U, of loads and QK, of INTER and INTRA
constexpr int kThreads = (kDecay + 4) * 32;

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
// bf16x2 of (a, b): a in the low half.
__device__ __forceinline__ uint32_t cvt2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ f2 wide(uint32_t h) {  // the two bf16 as floats
  return pk2(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u));
}
// 4 bytes to shared memory, zeros unless `on` (src is not read then).
__device__ __forceinline__ void cp_async4(float* dst, const float* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// ------------------------------------------------------------------ work items
// (Kept in shared memory, not in registers: with 220 KB of that in use the first-level cache is
// too small for anything that would spill to local memory.)
__device__ __noinline__ bool fill_item(const ChunkArgs& a, int it, Item* px) {
  Item x;
  if (!get_item(a, it, x)) return false;
  *px = x;
  return true;
}

// The item in a warp's own slot, filled by its first lane.
__device__ __forceinline__ bool warp_item(const ChunkArgs& a, int it, Item* slot) {
  __syncwarp();
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = it < a.items && fill_item(a, it, slot);
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// The k-th item of this CTA: rows of the grid in alternating directions, so that with items
// sorted by length the CTAs' sums stay close.
__device__ __forceinline__ int nth_item(int k) {
  const int g = (int)gridDim.x, c = (int)blockIdx.x;
  return k * g + ((k & 1) ? g - 1 - c : c);
}

// Chunks of item `it` in this launch.
template <bool OUT>
__device__ __forceinline__ int chunks_of(const ChunkArgs& a, int it) {
  const int s = it / (a.slices * a.p.HV);
  int n, off = 0, last;
  if (a.recs) {
    const SegRec& r = a.recs[s];
    n = r.seq < 0 ? 0 : r.n;
    last = r.last;
    if (a.p.pool) off = r.pos0 % C;
  } else {
    const int j = s % a.nseg;
    n = min(a.Lseg, a.p.T - j * a.Lseg);
    last = j == a.nseg - 1;
  }
  return n > 0 && (OUT || !last) ? (off + n + C - 1) / C : 0;
}

// ------------------------------------------------------------------ waits
// (The loop is not inlined: it would be a third of the kernel's code.)
// (The limit stands beside `dead` in shared memory, in units of 1024 ns: read from device memory it cost
// the packed prompts 4 %.)
__device__ __forceinline__ bool past_budget(uint64_t ns, volatile int* dead) { return (ns >> 10) > (uint32_t)dead[2]; }
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* dead, int* status) {
  uint64_t t0 = 0;
  while (!mbar_test_for(bar, parity, 20000)) {
    if (*dead) return false;
    const uint64_t t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    if (past_budget(t - t0, dead)) {
      if (status) atomicExch(status, kDevTimeout);
      *dead = 1;
      return false;
    }
  }
  return true;
}
struct Sync {
  volatile int* dead;  // a wait of this CTA ran out: everybody leaves
  int* status;
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    return mbar_test(bar, parity) || wait_slow(bar, parity, dead, status);
  }
  // by a whole warp, with one answer for all its lanes
  __device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait(bar, parity));
  }
};

// Barrier over the state threads that combines a flag.
__device__ __forceinline__ bool state_and(bool pred) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 1, %2, p;\n"
               " selp.u32 %0, 1, 0, q;\n}\n" : "=r"(r) : "r"((uint32_t)pred), "n"(kSW * 32) : "memory");
  return r != 0;
}

// ------------------------------------------------------------------ shared memory
struct TcArgs : ChunkArgs {
  int k_halves, v_halves;  // 64-column halves in the boxes of q and k, and of v and o
  int budget;              // limit of a wait, in units of 1024 ns
  int fault;               // test hook (gdp_debug_wait_fault): CTA 0 waits for a commit more of its first U
};

template <int KD, bool OUT>
struct Lay {
  static constexpr int NST = 3;                         // stages of q, k, v
  static constexpr int KH = KD / 64;                    // 64-column halves of q and k
  // q, k and v by halves of 64 columns: 64 rows of 128 bytes each
  static constexpr int KT = KH * 8192, VT = 2 * KT, STG = VT + 16384;
  static constexpr int P = NST * STG;                   // scores, two buffers
  static constexpr int O = P + (OUT ? 16384 : 0);       // output tile, two halves
  // decays: more slots than stages, since the output still reads them when the stage is free
  static constexpr int G = O + (OUT ? 16384 : 0);
  static constexpr int GS = 272 * 4;                    // hi2, lo2, wend, ein [64] each, e^Gam hi, lo
  static constexpr int BAR = G + 8 * GS;
  static constexpr int RAW = BAR + 256;                 // g as loaded, four chunks
  static constexpr int ITEM = RAW + 1024;               // work items, one slot per state warp and two more
  static constexpr int BYTES = ITEM + (kSW + 2) * 64 + 1024;
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};
// full, ready, free by stage; v' ready and free by step; INTER and INTRA done, P done by parity;
// U done and read by buffer; the rest single
enum {
  B_FULL = 0, B_READY = 3, B_FREE = 6, B_V = 9, B_VFREE = 13, B_O = 17, B_P = 19, B_QK = 21, B_SREAD, B_OREAD, B_S, B_U,
  B_UREAD = B_U + 2, B_N = B_UREAD + 2
};

// TMEM columns: scores [64], INTER and INTRA [64] each, U [KD], S [KD / 2], v' [3][32]
constexpr uint32_t T_QK = 0, T_INTER = 64, T_INTRA = 128, T_U = 192, T_S = 320, T_V = 384;
// (the state pass has no scores and outputs: two U's [128] in their place, so that one is formed while
// the other is read)

template <int KD, bool OUT>
__global__ void __launch_bounds__(kThreads, 1) linear_chunk_kernel(
    const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
    const __grid_constant__ TcArgs a) {
  using L = Lay<KD, OUT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + B_N);
  volatile int* s_dead = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_total = reinterpret_cast<int*>(s_tmem + 2);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const LinearProblem& p = a.p;

  if (!OUT) {
    pdl_wait();
    if (no_split(a)) return;
  }
  if (warp == 0) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < B_N; ++i) {
      int n = 1;
      if (i >= B_FREE && i < B_V) n = OUT ? 2 : 1;                   // both issuing warps
      if (i == B_OREAD || i == B_S || i >= B_UREAD) n = kSW;         // state warps
      if ((i >= B_V && i < B_VFREE) || i == B_P || i == B_P + 1 || i == B_SREAD) n = 4;  // v' or score warps
      if (i == B_U && a.fault && blockIdx.x == 0) n = 2;
      mbar_init(&bars[i], n);
    }
    fence_mbar_init();
    *s_dead = 0;
    s_dead[2] = a.budget;
  }
  if (warp == kDecay && lane == 0) {
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
    if (OUT) prefetch_tmap(&map_q);
  }
  pdl_wait();
  if (warp == 2) {  // chunks of this CTA over all its items
    int t = 0;
    for (int k = lane;; k += 32) {
      const int it = nth_item(k);
      if (it < a.items) t += chunks_of<OUT>(a, it);
      if (__all_sync(0xffffffffu, k * (int64_t)gridDim.x >= a.items)) break;
    }
    t = __reduce_add_sync(0xffffffffu, t);
    if (lane == 0) *s_total = t;
  }
  if (a.clear && blockIdx.x == 0 && tid == 96) *p.status = kDevOk;
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
  constexpr int NU = OUT ? 1 : 2;  // U's
  auto u_at = [&](int n) { return tmem + (OUT ? T_U : (uint32_t)(128 * (n & 1))); };

  if (warp < kSW) {
    // ---------------------------------------------------------------- state, output
    constexpr int NP = kSW / 4, NC = KD / NP;  // parts of k and of t; state columns (k) per thread
    const int quarter = warp & 3, part = warp >> 2, cb = part * NC;
    const int row = quarter * 32 + lane;  // value column of the slice
    const uint32_t lb = tmem + ((uint32_t)(quarter * 32) << 16);
    // output tile: this warp's 32 value columns, 16-byte chunks 4 (quarter % 2) .. + 3 of rows t =
    // 64 / NP part .. in the tile's half quarter / 2, permuted by t % 8; lane l gives row l % 8 of
    // a block of 8 x 8
    const uint32_t orow = smb + L::O + (quarter >> 1) * 8192 + (part * (64 / NP) + (lane & 7)) * 128;
    const uint32_t oc = 4 * (quarter & 1) + (lane >> 3);
    float s[NC];
    int n = 0;
    bool ok = true;
    for (int kk = 0; ok && (int64_t)kk * gridDim.x < a.items; ++kk) {
      const int it = nth_item(kk);
      Item& x = *reinterpret_cast<Item*>(sm + L::ITEM + warp * 64);
      if (!warp_item(a, it, &x) || skip<OUT>(x)) continue;
      const int chunks = x.chunks;
      const bool von = x.v0 + row < V;
      const int64_t at = ((int64_t)x.hv * K + cb) * V + x.v0 + row;
      {
        const float* src = state_src<OUT>(a, x);
        const float* q = src ? src + at : nullptr;
#pragma unroll
        for (int c = 0; c < NC; ++c, q += V) s[c] = src && von && cb + c < K ? __ldcg(q) : 0.f;
      }
      auto publish = [&] {  // the state as the A operand of INTER (whose last product is done)
#pragma unroll
        for (int q = 0; q < NC; q += 16) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = cvt2(s[q + 2 * e], s[q + 2 * e + 1]);
          GDP_TMEM_ST8(lb + T_S + (cb + q) / 2, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_S]);
      };
      if (OUT && chunks > 0) publish();
      float2 wseg = make_float2(1.f, 0.f);
      for (int c = 0; c < chunks; ++c, ++n) {
        // a failed wait leaves through the barrier below, with the whole group
        ok = sy.wait_warp(&bars[B_U + n % NU], (n / NU) & 1);
        if (!OUT && !ok) break;
        tc_fence_after();
        const float* g = gates(n);
        const float wh = g[256], wl = g[257];
        const f2 wh2 = pk2(wh, wh), wl2 = pk2(wl, wl);
#pragma unroll
        for (int q = 0; q < NC; q += 16) {
          uint32_t r[16];
          GDP_TMEM_LD16(u_at(n) + ((uint32_t)(quarter * 32) << 16) + cb + q, r);
          tmem_wait_ld();
          if (q + 16 == NC) {
            tc_fence_before();  // the next U may overwrite this one
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_UREAD + n % NU]);
          }
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float* d = s + q + e;
            const f2 old = pk2(d[0], d[1]);
            const float2 f = upk2(fma2(wh2, old, fma2(wl2, old, pk2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])))));
            d[0] = f.x;
            d[1] = f.y;
          }
        }
        if (!OUT) wseg = mul_pair(wseg, make_float2(wh, wl));
        if (OUT) {
          ok = sy.wait_warp(&bars[B_O + (n & 1)], (n >> 1) & 1) && ok;
          tc_fence_after();
          if (ok && c + 1 < chunks) publish();
          // the previous chunk's stores have read the tile
          if (tid == 0) tma_store_wait_read();
          if (!(ok = state_and(ok))) break;
          // eight rows t at a time, as fragments: pairs of rows in a register, by value block of 8
          const float* ein = g + 192 + (64 / NP) * part + 2 * (lane & 3);
#pragma unroll 1
          for (int z = 0; z < 8 / NP; ++z) {
            const uint32_t col = (64 / NP) * part + 8 * z;
            uint32_t r[8], w[8], out[4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              GDP_TMEM_LD_16X256_X1(lb + (q << 20) + T_INTER + col, (r + 4 * q));
              GDP_TMEM_LD_16X256_X1(lb + (q << 20) + T_INTRA + col, (w + 4 * q));
            }
            const float2 e = *reinterpret_cast<const float2*>(ein + 8 * z);
            tmem_wait_ld();
            if (z == 8 / NP - 1) {  // the next products may overwrite these
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars[B_OREAD]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float2 f = upk2(fma2(pk2(e.x, e.y), pk2(__uint_as_float(r[2 * u]), __uint_as_float(r[2 * u + 1])),
                                         pk2(__uint_as_float(w[2 * u]), __uint_as_float(w[2 * u + 1]))));
              out[u] = cvt2(f.x, f.y);
            }
            // lanes 8 m .. address value block m
            stmatrix_x4_trans(orow + z * 1024 + ((oc ^ (lane & 7)) << 4), out[0], out[1], out[2], out[3]);
          }
          // rows of the tile inside the sequence
          const int base = x.r.t0 - x.off + c * C;
          const int lo = max(0, x.r.t0 - base), hi = min(C, x.r.t0 + x.r.n - base);
          const bool whole = lo == 0 && (hi == C || (!a.recs && x.r.last));
          if (whole) {  // rows past a dense batch's end are clipped by the map
            fence_async_smem();
            state_and(true);
            if (tid == 0) {
              if (a.v_halves == 1) {
                tma_store_5d(&map_o, sm + L::O, x.v0, x.hv, base, x.b, 0);
                if (x.v0 + 64 < V) tma_store_5d(&map_o, sm + L::O + 8192, x.v0 + 64, x.hv, base, x.b, 0);
              } else {
                tma_store_5d(&map_o, sm + L::O, 0, x.hv, base, x.b, x.v0 >> 6);
              }
              tma_store_commit();
            }
          } else {
            state_and(true);
            bf16* og = static_cast<bf16*>(p.o) + (((int64_t)x.b * p.T + base) * p.HV + x.hv) * V + x.v0;
            const int j = tid & 15, c8 = 8 * j;  // 16-byte piece of the row (V is a multiple of 8)
            if (x.v0 + c8 < V)
              for (int t = lo + (tid >> 4); t < hi; t += 2 * kSW)
                *reinterpret_cast<uint4*>(og + (int64_t)t * p.HV * V + c8) =
                    *reinterpret_cast<const uint4*>(sm + L::O + (j >> 3) * 8192 + t * 128 + (((j & 7) ^ (t & 7)) << 4));
            // the next chunk's barrier orders these reads before its writes
          }
        }
        if (float* dst = state_dst<OUT>(a, x, c)) {
          if (von) {
            dst += at;
#pragma unroll
            for (int c2 = 0; c2 < NC; ++c2, dst += V)
              if (cb + c2 < K) *dst = s[c2];
          }
        }
      }
      if (!ok) break;
      if (!OUT && chunks > 0 && row == 0 && cb == 0) a.segW[(int64_t)x.r.id * p.HV + x.hv] = wseg;
      if (OUT && chunks == 0 && !p.pool && p.sT && von && x.r.last) {  // an empty sequence keeps its state
        float* dst = p.sT + (int64_t)x.r.seq * p.HV * K * V + at;
#pragma unroll
        for (int c2 = 0; c2 < NC; ++c2, dst += V)
          if (cb + c2 < K) *dst = s[c2];
      }
    }
    if (OUT && tid == 0) tma_store_wait_all();
  } else if (warp < (OUT ? kScore : kDecay)) {
    // ---------------------------------------------------------------- v'
    // (in the state pass by the score warps too, two of a chunk's four steps each)
    constexpr int KS = OUT ? 4 : 2;
    const int quarter = warp & 3, ks0 = (warp - kSW) / 4 * KS;
    const uint32_t lb = tmem + ((uint32_t)(quarter * 32) << 16) + T_V;
    // transposing loads: lanes 8 m .. 8 m + 7 address rows i of value block m (16-byte chunk
    // 4 (quarter % 2) + m, permuted by i % 8)
    const uint32_t vrow = L::VT + (quarter >> 1) * 8192 + (lane & 7) * 128 +
                          (((4 * (quarter & 1) + (lane >> 3)) ^ (lane & 7)) << 4);
    bool ok = true;
    for (int n = 0; n < total && ok; ++n) {
      if (!tiles(n)) break;
      uint32_t va = smb + (n % L::NST) * L::STG + vrow + ks0 * 2048;
      const float* g = gates(n) + 128 + ks0 * 16 + 2 * (lane & 3);
      // a step of U (16 positions) at a time, each as soon as U(n - 1) has read its own
#pragma unroll 1
      for (int ks = ks0; ks < ks0 + KS; ++ks, va += 2048, g += 16) {
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
  } else if (warp < kDecay) {
    // ---------------------------------------------------------------- scores
    if (OUT) {
      // rows t0 + l / 4 (+ 8) of the chunk, columns 2 (l % 4) (+ 1) of a block of 8, as fragments
      const int quarter = warp & 3, t0 = 16 * quarter + (lane >> 2), i0 = 2 * (lane & 3);
      const uint32_t lb = tmem + ((uint32_t)(quarter * 32) << 16) + T_QK;
      // stores: lanes 8 m .. address rows 8 (m % 2) .. of the warp's 16 and 16-byte chunk m / 2
      const int srow = 16 * quarter + 8 * ((lane >> 3) & 1) + (lane & 7);
      const uint32_t prow = smb + L::P + srow * 128;
      const f2 sc2 = pk2(p.scale, p.scale);
      for (int n = 0; n < total; ++n) {
        // INTRA(n - 2) has read this P buffer
        if (n >= 2 && !sy.wait_warp(&bars[B_O + (n & 1)], ((n >> 1) - 1) & 1)) break;
        if (!sy.wait_warp(&bars[B_QK], n & 1)) break;
        tc_fence_after();
        const float* g = gates(n);
        const f2 hi0 = pk2(g[t0], g[t0]), lo0 = pk2(g[64 + t0], g[64 + t0]);
        const f2 hi1 = pk2(g[t0 + 8], g[t0 + 8]), lo1 = pk2(g[72 + t0], g[72 + t0]);
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[4] = {0, 0, 0, 0};
          if (q <= quarter) {  // else columns past every row of this warp
            uint32_t r[8];
            GDP_TMEM_LD_16X256_X2(lb + 16 * q, r);
            const float* gq = g + 16 * q + i0;
            const float2 h0 = *reinterpret_cast<const float2*>(gq), h1 = *reinterpret_cast<const float2*>(gq + 8);
            const float2 l0 = *reinterpret_cast<const float2*>(gq + 64), l1 = *reinterpret_cast<const float2*>(gq + 72);
            tmem_wait_ld();
            if (q == quarter) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars[B_SREAD]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {  // block u / 2 of 8 columns, rows + 8 (u % 2)
              const f2 h = u < 2 ? pk2(h0.x, h0.y) : pk2(h1.x, h1.y), l = u < 2 ? pk2(l0.x, l0.y) : pk2(l1.x, l1.y);
              const float2 x = upk2(add2(sub2(u & 1 ? hi1 : hi0, h), sub2(u & 1 ? lo1 : lo0, l)));
              const float2 y = upk2(mul2(mul2(pk2(__uint_as_float(r[2 * u]), __uint_as_float(r[2 * u + 1])), sc2),
                                         pk2(ex2_approx(x.x), ex2_approx(x.y))));
              const int d = t0 + 8 * (u & 1) - 16 * q - 8 * (u >> 1) - i0;  // t - i
              pk[u] = cvt2(d >= 0 ? y.x : 0.f, d >= 1 ? y.y : 0.f);
            }
          }
          stmatrix_x4(prow + (n & 1) * 8192 + (((2 * q + (lane >> 4)) ^ (lane & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_P + (n & 1)]);
      }
    }
  } else if (warp == kDecay) {
    // ---------------------------------------------------------------- decays
    float* ring = reinterpret_cast<float*>(sm + L::RAW) + 2 * lane;  // g as loaded, four chunks
    int n = 0;
    bool ok = true;
    for (int kk = 0; ok && (int64_t)kk * gridDim.x < a.items; ++kk) {
      Item& x = *reinterpret_cast<Item*>(sm + L::ITEM + kSW * 64);
      if (!warp_item(a, nth_item(kk), &x) || skip<OUT>(x)) continue;
      const int chunks = x.chunks, base0 = x.r.t0 - x.off, t1 = x.r.t0 + x.r.n;
      auto fetch = [&](int c) {  // zeros outside the sequence
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int t = base0 + c * C + 2 * lane + u;
          const bool on = p.g && t >= x.r.t0 && t < t1;
          const int64_t at = p.g_token ? ((int64_t)x.b * p.T + t) * p.HV + x.hv : x.hv;
          cp_async4(ring + (c & 3) * C + u, on ? p.g + at : static_cast<const float*>(p.k), on);
        }
        cp_async_commit();
      };
      fetch(0);
      fetch(1);
      for (int c = 0; c < chunks; ++c, ++n) {
        const int st = n % L::NST, base = base0 + c * C;
        const int lo = max(0, x.r.t0 - base), hi = min(C, t1 - base);
        fetch(c + 2);
        // chunk n - 3's products are done, so the decays of chunk n - 8 have been used
        if (n >= L::NST && !(ok = sy.wait_warp(&bars[B_FREE + st], (n / L::NST - 1) & 1))) break;
        cp_async_wait<2>();
        const float2 g = *reinterpret_cast<const float2*>(ring + (c & 3) * C);
        chunk_decays(g.x, g.y, p.scale, lo, hi, lane, gates(n));
        if (!(ok = sy.wait_warp(&bars[B_FULL + st], (n / L::NST) & 1))) break;
        if (lo > 0 || hi < C) {
          // rows of other sequences, or past the end: k and v as zeros, so that nothing in
          // them (not even a NaN) enters a sum over the rows
          uint8_t* tile = sm + st * L::STG;
          for (int i = lane >> 3; i < C; i += 4)
            if (i < lo || i >= hi) {
              const uint32_t o = i * 128 + (lane & 7) * 16;
#pragma unroll
              for (int hh = 0; hh < L::KH; ++hh)
                *reinterpret_cast<uint4*>(tile + L::KT + hh * 8192 + o) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(tile + L::VT + o) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(tile + L::VT + 8192 + o) = make_uint4(0, 0, 0, 0);
            }
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_READY + st]);
      }
      cp_async_wait<0>();
    }
  } else if (warp == kDecay + 1) {
    // ---------------------------------------------------------------- U
    const uint32_t id_u = idesc_bf16(128, KD, false, true);
    for (int n = 0; n < total; ++n) {
      bool ok = tiles(n);
      if (n >= NU) ok = sy.wait_warp(&bars[B_UREAD + n % NU], (n / NU - 1) & 1) && ok;
      const uint64_t kd = sdesc_sw128(smb + (n % L::NST) * L::STG + L::KT, 8192, 1024);
#pragma unroll 1
      for (int ks = 0; ks < 4; ++ks) {
        ok = ok && sy.wait_warp(&bars[B_V + ks], n & 1);
        if (!ok) break;
        if (elect_one()) {
          tc_fence_after();
          const uint64_t k = kd + (uint64_t)(ks * (2048 >> 4));
          const uint32_t av = tmem + T_V + 8 * ks;
          mma_bf16_ts(u_at(n), av + 64, k, id_u, ks > 0);
          mma_bf16_ts(u_at(n), av + 32, k, id_u, 1);
          mma_bf16_ts(u_at(n), av, k, id_u, 1);
          mma_commit(&bars[B_VFREE + ks]);
          if (ks == 3) {
            mma_commit(&bars[B_U + n % NU]);
            mma_commit(&bars[B_FREE + n % L::NST]);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
    }
  } else if (warp == kDecay + 2) {
    // ---------------------------------------------------------------- loads, QK
    const uint32_t id = idesc_bf16(64, 64, false, false);
    int next = 0, kk = -1, c = 0, chunks = 0;  // the next load: chunk c of the CTA's item kk
    Item& x = *reinterpret_cast<Item*>(sm + L::ITEM + (kSW + 1) * 64);
    auto load = [&] {
      const int st = next % L::NST;
      while (c >= chunks) {
        c = 0;
        chunks = warp_item(a, nth_item(++kk), &x) && !skip<OUT>(x) ? x.chunks : 0;
      }
      if (elect_one()) {
          const int t = x.r.t0 - x.off + c * C;
          uint8_t* tile = sm + st * L::STG;
          uint64_t* bar = &bars[B_FULL + st];
          // a tensor whose width is whole halves comes by one load, both halves in its box; of
          // another the second half is its own load (zeros past the width), if there is one
          const bool two = a.v_halves == 1 && x.v0 + 64 < V, twok = KD == 128 && a.k_halves == 1;
          mbar_expect_tx(bar, (OUT ? 2 : 1) * L::KT + 8192 * (two ? 2 : a.v_halves));
          if (OUT) tma_load_5d(tile, &map_q, 0, x.h, t, x.b, 0, bar);
          tma_load_5d(tile + L::KT, &map_k, 0, x.h, t, x.b, 0, bar);
          if (a.v_halves == 1) tma_load_5d(tile + L::VT, &map_v, x.v0, x.hv, t, x.b, 0, bar);
          else tma_load_5d(tile + L::VT, &map_v, 0, x.hv, t, x.b, x.v0 >> 6, bar);
          if (twok) {
            if (OUT) tma_load_5d(tile + 8192, &map_q, 64, x.h, t, x.b, 0, bar);
            tma_load_5d(tile + L::KT + 8192, &map_k, 64, x.h, t, x.b, 0, bar);
          }
          if (two) tma_load_5d(tile + L::VT + 8192, &map_v, x.v0 + 64, x.hv, t, x.b, 0, bar);
      }
      __syncwarp();
      ++c;
      ++next;
    };
    // loads and scores as each becomes possible, whichever is first
    auto all = [](bool yes) { return __all_sync(0xffffffffu, yes); };
    uint64_t since = 0;  // nothing was possible since then
    for (int n = 0, spins = 0; OUT ? n < total : next < total;) {
      const bool qk = OUT && n < next && all(mbar_poll(&bars[B_READY + n % L::NST], (n / L::NST) & 1) &&
                                             mbar_poll(&bars[B_FULL + n % L::NST], (n / L::NST) & 1) &&
                                             (n == 0 || mbar_poll(&bars[B_SREAD], (n - 1) & 1)));
      if (qk) {
        if (elect_one()) {
          tc_fence_after();
          const uint32_t tl = smb + (n % L::NST) * L::STG;
          const uint64_t qd = sdesc_sw128(tl, 16, 1024), kd = sdesc_sw128(tl + L::KT, 16, 1024);
#pragma unroll 1
          for (int i = 0; i < KD / 16; ++i) {
            const uint64_t o = (uint64_t)((i >> 2) * (8192 >> 4) + (i & 3) * 2);
            mma_bf16(tmem + T_QK, qd + o, kd + o, id, i > 0);
          }
          mma_commit(&bars[B_QK]);
        }
        __syncwarp();
        ++n;
      } else if (next < total && (next < L::NST || all(mbar_poll(&bars[B_FREE + next % L::NST], (next / L::NST - 1) & 1)))) {
        load();
      } else {
        if ((++spins & 63) == 0) {  // a bounded wait like the others
          const uint64_t t = globaltimer_ns();
          if (spins == 64) since = t;
          if (__any_sync(0xffffffffu, *sy.dead || past_budget(t - since, sy.dead))) {
            if (lane == 0 && !*sy.dead) {
              if (p.status) atomicExch(p.status, kDevTimeout);
              *sy.dead = 1;
            }
            break;
          }
        }
        continue;
      }
      spins = 0;
    }
    // nothing may still write shared memory when the CTA leaves
    for (int m = max(0, next - L::NST); m < next; ++m) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_test(&bars[B_FULL + m % L::NST], (m / L::NST) & 1) && !past_budget(globaltimer_ns() - t0, s_dead)) {}
    }
  } else if (OUT) {
    // ---------------------------------------------------------------- INTER, INTRA
    const uint32_t id_i = idesc_bf16(128, 64, false, false), id_a = idesc_bf16(128, 64, true, false);
    for (int n = 0; n < total; ++n) {
      if (!tiles(n)) break;
      // the state before the chunk, its scores, and the last output out of the way
      if (!sy.wait_warp(&bars[B_S], n & 1)) break;
      if (!sy.wait_warp(&bars[B_P + (n & 1)], (n >> 1) & 1)) break;
      if (n > 0 && !sy.wait_warp(&bars[B_OREAD], (n - 1) & 1)) break;
      if (elect_one()) {
        tc_fence_after();
        const uint32_t tl = smb + (n % L::NST) * L::STG;
        const uint64_t qd = sdesc_sw128(tl, 16, 1024);
#pragma unroll 1
        for (int i = 0; i < KD / 16; ++i)
          mma_bf16_ts(tmem + T_INTER, tmem + T_S + 8 * i, qd + (uint64_t)((i >> 2) * (8192 >> 4) + (i & 3) * 2), id_i, i > 0);
        const uint64_t vd = sdesc_sw128(tl + L::VT, 8192, 1024);
        const uint64_t pd = sdesc_sw128(smb + L::P + (n & 1) * 8192, 16, 1024);
#pragma unroll 1
        for (int i = 0; i < 4; ++i) mma_bf16(tmem + T_INTRA, vd + i * (2048 >> 4), pd + i * 2, id_a, i > 0);
        mma_commit(&bars[B_O + (n & 1)]);
        mma_commit(&bars[B_FREE + n % L::NST]);
      }
      __syncwarp();
    }
  }
  __syncwarp();
  if (*s_dead) {  // products in flight end before their operands and columns go away
    if (warp == kDecay + 1 && lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) {}  // a chunk's products take microseconds
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ host
// Test hook state (gdp_debug_wait_fault): armed for the next launch only.
std::atomic<int> g_fault{0};
std::atomic<unsigned long long> g_budget_ns{kWaitBudgetNs};

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

// [B][T][heads][width] with element strides s (batch, token, head); boxes of 64 x 1 x 64 x 1,
// `halves` of them side by side where the width is a multiple of 64 (1: any width).
bool map5(CUtensorMap* m, const void* base, int width, int halves, int heads, int T, int B, const int64_t* s) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const bool split = halves > 1;
  const cuuint64_t dims[5] = {(cuuint64_t)(split ? 64 : width), (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B,
                              (cuuint64_t)(split ? width / 64 : 1)};
  // the stride of a dimension of one entry is never used; the encoder wants a valid one
  const cuuint64_t some = 16;
  const cuuint64_t st[4] = {heads > 1 ? (cuuint64_t)s[2] * 2 : some, T > 1 ? (cuuint64_t)s[1] * 2 : some,
                            B > 1 ? (cuuint64_t)s[0] * 2 : some, split ? (cuuint64_t)128 : some};
  const cuuint32_t box[5] = {64, 1, 64, 1, (cuuint32_t)halves}, es[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, st, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_ok(const void* base, int heads, int T, int B, const int64_t* s) {
  const auto fits = [](int n, int64_t x) { return n <= 1 || (x > 0 && x % 8 == 0 && x < ((int64_t)1 << 38)); };
  return reinterpret_cast<uintptr_t>(base) % 16 == 0 && fits(heads, s[2]) && fits(T, s[1]) && fits(B, s[0]);
}

template <int KD, bool OUT>
cudaError_t go(const TcArgs& a, const CUtensorMap* m) {
  constexpr int smem = Lay<KD, OUT>::BYTES;
  auto kern = linear_chunk_kernel<KD, OUT>;
  cudaError_t e = allow_smem<linear_chunk_kernel<KD, OUT>>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(std::min(a.items, sm_count())), dim3(kThreads), smem, a.p.stream, m[0], m[1], m[2],
                    m[3], a);
}

}  // namespace

// As measured at K = V = 128 (smaller ones take as long: the roles' steps, not the bytes, set it); an
// item's and a split's fixed times are the best of a sweep over 16 sizes from 16 heads x 192 tokens to
// 32 x 16384 (1 x 700 tokens, 16 heads: 20.4 us, against 25.8 with 5 and 9).
constexpr Cost kCost = {1.85, 1.2, 3.0, 6.0};

bool linear_tc_shape(int K, int V, gdp_dtype dt) { return dt == GDP_BF16 && K <= 128 && K % 8 == 0 && V % 8 == 0; }

size_t linear_tc_workspace(int N_seq, int B, int T, int HV, int K, int V) {
  // the query does not say whether the batch is packed
  const size_t d = N_seq == B ? plan_of(N_seq, B, T, HV, K, V, false, kVT, kCost, sm_count()).total : 0;
  return std::max(d, B == 1 ? plan_of(N_seq, B, T, HV, K, V, true, kVT, kCost, sm_count()).total : 0);
}

bool linear_tc_ok(const LinearProblem& p) {
  return linear_tc_shape(p.K, p.V, p.dt) && map_ok(p.q, p.H, p.T, p.B, p.qs) && map_ok(p.k, p.H, p.T, p.B, p.ks) &&
         map_ok(p.v, p.HV, p.T, p.B, p.vs) && reinterpret_cast<uintptr_t>(p.o) % 16 == 0;
}

void linear_wait_fault(int arm, unsigned long long budget_ns) {
  g_fault.store(arm);
  g_budget_ns.store(budget_ns);
}

cudaError_t launch_linear_tc(const LinearProblem& p, uint8_t* ws) {
  const Plan x = plan_of(p.N_seq, p.B, p.T, p.HV, p.K, p.V, p.cu != nullptr, kVT, kCost, sm_count());
  TcArgs a{};
  a.p = p;
  a.clear = !p.cu;  // (the segment kernel does it for a packed batch)
  a.nseg = x.nseg;
  a.Lseg = x.Lseg;
  a.slices = x.slices;
  a.vt = kVT;
  if (x.bound * p.HV * x.slices > INT32_MAX - 65536) return cudaErrorInvalidValue;
  a.items = (int)(x.bound * p.HV * x.slices);
  if (a.items == 0) return cudaMemsetAsync(p.status, 0, sizeof(int32_t), p.stream);  // kDevOk
  int2* seqs = nullptr;
  if (p.cu) {
    SegRec* recs = reinterpret_cast<SegRec*>(ws + x.recs);
    seqs = reinterpret_cast<int2*>(ws + x.seqs);
    a.recs = recs;
    int* split = reinterpret_cast<int*>(ws) + 1;  // beside the status word
    a.split = split;
    const cudaError_t e = launch_segments(p, x, recs, seqs, split);
    if (e != cudaSuccess) return e;
  }
  CUtensorMap m[4];
  const int64_t os[3] = {(int64_t)p.T * p.HV * p.V, (int64_t)p.HV * p.V, p.V};
  a.k_halves = p.K == 128 ? 2 : 1;
  a.v_halves = p.V % 128 == 0 ? 2 : 1;
  if (!map5(&m[0], p.q, p.K, a.k_halves, p.H, p.T, p.B, p.qs) || !map5(&m[1], p.k, p.K, a.k_halves, p.H, p.T, p.B, p.ks) ||
      !map5(&m[2], p.v, p.V, a.v_halves, p.HV, p.T, p.B, p.vs) || !map5(&m[3], p.o, p.V, a.v_halves, p.HV, p.T, p.B, os))
    return cudaErrorInvalidValue;
  a.budget = (int)(g_budget_ns.load() >> 10);
  a.fault = g_fault.exchange(0);
  if (x.segS) {
    a.segS = reinterpret_cast<float*>(ws + x.segS);
    a.segW = reinterpret_cast<float2*>(ws + x.segW);
    cudaError_t e = p.K > 64 ? go<128, false>(a, m) : go<64, false>(a, m);
    if (e == cudaSuccess) e = launch_combine(a, seqs);
    if (e != cudaSuccess) return e;
    a.fault = a.clear = 0;
  }
  return p.K > 64 ? go<128, true>(a, m) : go<64, true>(a, m);
}

}  // namespace gdp
