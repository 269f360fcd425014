// Attention of new tokens over a paged cache on the tensor cores: bf16 and fp16, heads of up to 256
// elements in steps of 8.
//
// A CTA walks the pieces of its share (attention.cuh) with two slots, each with four warps of its own,
// two buffers of 64 columns of scores and KD of outputs in tensor memory:
//   more than 128 rows: the slots are two tiles of 128 rows that read the same keys;
//   fewer: both slots have the same rows and take the tiles of 64 keys in turn, and their two bases, sums
//   and outputs are joined at the piece's end (they lie in the same lanes of tensor memory).
// Heads above 128 have one slot, whose outputs take the second one's columns.
// So one slot's softmax runs beside the other's products either way, and a decode step's few rows cost
// what streaming their keys costs: the products of a padded tile of 128 rows keep the tensor pipe busy a
// third of the time that HBM needs for its keys.
//
// A tile: S = Q K^T (tcgen05, K-major operands), then a thread per row takes its 64 scores from tensor
// memory, forms p = 2^(c s - b) in registers and puts them back as 16-bit pairs over S, and O += P V takes
// P from there and V as it lies (MN-major). The base b only follows the row's maximum when that has grown by more
// than 2^8 (then O is scaled in tensor memory): p stays below 2^8, and a 16-bit p keeps its relative
// precision, half a step of the type, which is what the output's own rounding costs (fp16's begins 2^7 higher, see
// kUp). Sums are fp32.
//
// Roles: warps 0 to 7 softmax, 8 and 9 load K and V, 10 and 11 issue the products. Loads are boxes of 64
// columns and `g` keys, g the largest power of two that divides both the page and the tile, through tensor
// maps of the whole caches (both halves of 128 columns in one box where it holds a whole tile); pages that
// are not there are boxes past the last page, which arrive as zeros, and so are boxes behind the last key;
// what remains of the last box is zeroed in shared memory before it is multiplied (weights of 0 times NaN
// are not 0). Pages whose size is not a multiple of 8 come by 16-byte cp.async.
//
// Measured: 256 requests of up to 8192 keys, 32 heads over 8, 128 columns: 610 us, 98 % of the measured copy
// rate, bound by HBM. Pieces of prompts, 8 of up to 1024 tokens on up to 4096: 137 us, 0.91 PFLOP/s, 47 % of
// the measured bf16 rate: a tile of 2 x 128 rows takes 1830 cycles, where its products fill 1024 and its
// exponentials 1024 (16 a cycle and SM); the rest is the chain scores, softmax, weights, outputs, scores, which
// two buffers a slot overlap but once. One slot: 16 requests of up to 9000 keys, 16 heads over 4, 256 columns: 68 us,
// where HBM needs 50; pieces of prompts of 16 heads over 4, 256 columns: 311 us, 0.81 PFLOP/s. Pages by cp.async (of
// 100): the decode batch 1450 us, the prompts 262. Beginning a share 4 us, queries in and outputs out 6 us a piece.
#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "attention.cuh"
#include "ptx.cuh"

namespace gdp {
namespace attn {
namespace {
using namespace ptx;

constexpr int kKeys = 64;
constexpr int kLoad = 8, kScores = 10, kOutputs = 11;  // warps; 0 to 3 and 4 to 7 are the slots', 8 and 9 load K and V
constexpr int kThreads = 384;
// Shares are of equal cost, in units of about 0.3 us as measured: up to 128 rows 3 us to begin and end an item and
// 0.6 a tile, more rows 6.5 and 0.95; heads above 128, with twice the bytes, 3 and 1.5. (With tiles alone the slowest CTA of a decode batch took 870 us, the median
// 566, and 216 and 130 of pieces of prompts; now 610 and 588, 132 and 122.)
constexpr Cost kCost = {10, 2, 22, 3}, kCostWide = {10, 5, 10, 5};
// log2 of a factor of all weights, which their sum has too: fp16's reach from 2^15 down to 2^-14 in full precision, so
// that only those 2^21 times smaller than the largest lose some. The base is the row's maximum less this.
template <typename T> constexpr float kUp = std::is_same_v<T, __half> ? 7.f : 0.f;
template <typename T> constexpr float kGrow = kUp<T> + 8.f;  // log2 of how far the maximum may lie above the base
// From here on (powers of two) a score's steps are a half and more. One multiply-add of a score and its base would then
// give the largest weight anything from 2^-half a step to 2^half a step, in 16 bits as far as 0 and infinity. So such a
// row's scores are rounded as their maximum was before the base, that maximum itself, is taken off: by a second pass over
// the tile's scores in tensor memory, so that other tiles pay a vote (pieces of prompts 137 us, 136 without; 138 to 151
// with the rounding in the first pass, in a function, or in more columns a step).
constexpr float kFar = 4194304.f;

template <int KD>
struct Lay {
  // Buffers of K and of V. A tile of K is free when its scores are formed, one of V two thousand cycles later:
  // with as many of V as of K in common stages a decode step had too few loads in flight.
  static constexpr int NK = KD == 256 ? 2 : KD == 128 ? 4 : 8, NV = KD == 256 ? 3 : KD == 128 ? 6 : 12;
  static constexpr int SLOTS = KD == 256 ? 1 : 2, ROWS = 128 * SLOTS;
  static constexpr int HALF = kKeys * 128;       // 64 columns of a tile: 64 rows of 128 bytes
  static constexpr int TILE = KD / 64 * HALF;
  static constexpr int QT = KD / 64 * 16384;     // 128 rows of queries
  static constexpr int Q = 0, K = SLOTS * QT, V = K + NK * TILE;
  static constexpr int BAR = V + NV * TILE;
  static constexpr int ML = BAR + 704;           // bases and sums [2][128]
  static constexpr int START = ML + 2048;        // the share, and the sums that lead to it
  static constexpr int BYTES = START + 192;
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};
// by buffer: K full, empty, V full, empty, absent keys known; by slot and buffer of its scores: scores, weights,
// outputs (a waiter may be two tiles behind, which one barrier's parity cannot tell from none); by slot: queries;
// a piece's two slots have left their bases, have read each other's outputs
enum {
  B_KFULL = 0, B_KEMPTY = 8, B_VFULL = 16, B_VEMPTY = 28, B_META = 40, B_S = 52, B_P = 56, B_O = 60, B_Q = 64,
  B_JOIN = 66, B_DONE, B_END, B_N = B_END + 2
};
constexpr uint32_t T_S = 0, T_O = 256;  // columns: scores [2][2][64], weights over them; outputs [2][128] or [256]

struct TcArgs : Args {
  int g;          // keys of a box
  int halves;     // of 64 columns in a box
  int budget;     // limit of a wait, in units of 1024 ns
  int fault;      // test hook (gdp_debug_wait_fault): every CTA waits for a commit more of its first scores
};

// ------------------------------------------------------------------ waits
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* dead, int budget, int* status) {
  uint64_t t0 = 0;
  while (!mbar_test_for(bar, parity, 20000)) {
    if (*dead) return false;
    const uint64_t t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    if (((t - t0) >> 10) > (uint32_t)budget) {
      report(status, kDevTimeout);
      *dead = 1;
      return false;
    }
  }
  return true;
}
struct Sync {
  volatile int* dead;  // a wait of this CTA ran out: everybody leaves
  int budget;
  int* status;
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait1(bar, parity));
  }
  // by one thread
  __device__ __forceinline__ bool wait1(uint64_t* bar, uint32_t parity) const {
    return mbar_test(bar, parity) || wait_slow(bar, parity, dead, budget, status);
  }
};

template <typename T> __device__ __forceinline__ uint32_t pack(float a, float b);
template <> __device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
template <> __device__ __forceinline__ uint32_t pack<__half>(float a, float b) {
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
// kind::f16 with operands of type T (fp16 is format 0)
template <typename T>
__device__ constexpr uint32_t idesc(int M, int N, bool b_mn) {
  return sizeof(T) == 2 && std::is_same<T, __half>::value ? idesc_bf16(M, N, false, b_mn) & ~((1u << 7) | (1u << 10))
                                                          : idesc_bf16(M, N, false, b_mn);
}
// The lowest n of 64 bits (n outside 0 .. 64 is held to it).
__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull; }

// How a piece's tiles are spread over the slots.
template <int SLOTS>
struct Spread {
  bool two;       // tiles of rows of their own, the same keys
  int n, rows, row0;
  __device__ __forceinline__ Spread(const Piece& x, int slot) {
    two = SLOTS == 2 && x.rows > 128;
    n = two ? x.j1 - x.j0 : SLOTS == 2 ? (x.j1 - x.j0 + 1 - slot) / 2 : slot ? 0 : x.j1 - x.j0;
    rows = two ? (slot ? x.rows - 128 : 128) : x.rows;
    row0 = x.row0 + (two ? 128 * slot : 0);
  }
};

template <typename T, int KD, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ TcArgs a) {
  using L = Lay<KD>;
  extern __shared__ __align__(1024) uint8_t sm[];  // (nothing static beside it: the array begins on a swizzle atom)
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint64_t* s_absent = bars + B_N;                                     // [NV]: keys of a tile that are not there
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_absent + L::NV);
  volatile int* s_dead = reinterpret_cast<volatile int*>(s_tmem + 1);
  float2* s_ml = reinterpret_cast<float2*>(sm + L::ML);                // [2][128]
  Start& s_start = *reinterpret_cast<Start*>(sm + L::START);
  long long* s_scan = reinterpret_cast<long long*>(sm + L::START + 96);  // [kThreads / 32]
  static_assert(sizeof(Start) <= 96 && kThreads / 32 * 8 <= 96 && B_N * 8 + L::NV * 8 + 8 <= 704, "shared memory");
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const Problem& p = a.p;

  if (warp == kScores) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (tid < B_N) {
    int n = 1;
    if ((tid >= B_P && tid < B_O) || (tid >= B_Q && tid < B_JOIN)) n = 4;                // warps of the slot
    if (tid == B_JOIN || tid == B_DONE) n = 8;
    if (tid == B_S && a.fault) n = 2;
    mbar_init(&bars[tid], n);
    fence_mbar_init();
  }
  if (tid == 96) *s_dead = 0;
  if (TMA && warp == kLoad && lane == 0) {
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  pdl_wait();
  pdl_trigger();
  find_start<L::ROWS, kKeys, kThreads>(a, &s_start, s_scan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const Sync sy{s_dead, a.budget, p.status};
  Walk<L::ROWS, kKeys> walk(s_start, a.cost);
  Piece x;
  bool ok = true;

  if (warp < kLoad) {
    // ---------------------------------------------------------------- softmax, outputs
    const int slot = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lanes + T_S + 128 * slot, to = tmem + lanes + T_O;
    // a scale of 0 as the least that keeps 0 times -inf (not seen) at -inf
    const float c = fmaxf(fabsf(p.c), 1e-37f);
    uint8_t* sq = sm + L::Q + slot * L::QT;
    const uint32_t sqa = smem_u32(sq);
    uint32_t n = 0, tile0 = 0, joins = 0, other = 0;  // tiles of this slot, of the CTA; joins; tiles of the other slot
    bool rec = false, owe = false;
#pragma unroll 1
    while (ok && walk.next(p, x)) {
      const Spread<L::SLOTS> d(x, slot);
      if (d.n > 0) {  // Q: 16-byte chunks of the rows, zero behind the head's end
        const int ch = tid % (KD / 8);
        const T* q0 = static_cast<const T*>(p.q) + (p.cu ? x.first * p.qs[1] : x.r * p.qs[0]) + x.head * p.G * p.qs[2] +
                      (8 * ch < p.D ? 8 * ch : 0);
#pragma unroll 4
        for (int r = (tid & 127) / (KD / 8); r < d.rows; r += 128 / (KD / 8)) {
          const int R = d.row0 + r, t = (int)quot(R, p.by_G);
          const T* src = q0 + t * p.qs[1] + (R - t * p.G) * p.qs[2];
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           sqa + (ch >> 3) * 16384 + sw128_offset(r, (ch & 7) * 16)),
                       "l"(src), "r"(8 * ch < p.D ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_Q + slot]);
      }
      const bool live = quarter * 32 < d.rows;
      const int t = (int)quot(d.row0 + min(row, d.rows - 1), p.by_G);
      const uint64_t bits = p.tree && x.x.live ? (uint64_t)p.tree[x.first + t] : 0ull;
      float b = -INFINITY, off = 0.f, l = 0.f;  // off: what is taken off a score: b, or 0 while nothing is seen
      bool far = false;                         // b lies beyond kFar
#pragma unroll 1
      for (int k = 0; ok && k < d.n; ++k, ++n) {
        const int j = d.two || L::SLOTS == 1 ? k : 2 * k + slot, key0 = (x.j0 + j) * kKeys;
        const uint32_t stage = (tile0 + j) % L::NV, turn = (tile0 + j) / L::NV;
        const uint32_t buf = n & 1, tb = ts + 64 * buf;
        ok = sy.wait(&bars[B_S + 2 * slot + buf], n >> 1 & 1) && (!live || sy.wait(&bars[B_META + stage], turn & 1));
        if (!ok) break;
        tc_fence_after();
        const uint64_t absent = live ? s_absent[stage] : 0ull;
        if (live) {
          uint32_t s[kKeys];
          GDP_TMEM_LD32(tb, s);
          GDP_TMEM_LD32(tb + 32, (s + 32));
          tmem_wait_ld();
          uint64_t see = ~0ull;
          if (key0 + kKeys > x.x.ctx || absent) {  // some of the keys are not seen by some row
            if (p.tree) {
              const int back = key0 - x.x.ctx;
              see = low_bits(-back);
              if (back > -kKeys && back < 64) see |= back >= 0 ? bits >> back : bits << -back;
            } else {
              see = low_bits(x.x.ctx + t + 1 - key0);
            }
            see &= low_bits(x.keys - key0) & ~absent;
#pragma unroll
            for (int e = 0; e < kKeys; ++e) {
              const uint32_t half = (uint32_t)(see >> (e & 32));
              s[e] = half >> (e & 31) & 1 ? s[e] : __float_as_uint(-INFINITY);
            }
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kKeys; ++e) top[e & 3] = fmaxf(top[e & 3], __uint_as_float(s[e]));
          const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
          const bool grow = mt - b > kGrow<T>;  // (from -inf: as soon as anything is seen)
          if (__any_sync(0xffffffffu, grow || far)) {
            const float bn = grow ? mt - (fabsf(mt) < kFar ? kUp<T> : 0.f) : b, f = grow ? ex2(b - bn) : 1.f;
            b = bn;
            l *= f;
            far = row < d.rows && fabsf(b) >= kFar && b != -INFINITY;
            off = b == -INFINITY ? 0.f : b;
            if (k > 0 && __any_sync(0xffffffffu, grow)) {  // the last product into O is done, then O is scaled
              ok = sy.wait(&bars[B_O + 2 * slot + (buf ^ 1)], (n - 1) >> 1 & 1);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < KD; q += 8) {
                uint32_t o[8];
                GDP_TMEM_LD8(to + 128 * slot + q, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                GDP_TMEM_ST8(to + 128 * slot + q, o);
              }
            }
          }
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float p0 = ex2(fmaf(__uint_as_float(s[2 * e]), c, -off));
            const float p1 = ex2(fmaf(__uint_as_float(s[2 * e + 1]), c, -off));
            sum[2 * (e & 1)] += p0;
            sum[2 * (e & 1) + 1] += p1;
            w[e] = pack<T>(p0, p1);
          }
          if (__any_sync(0xffffffffu, far)) {  // again, from rounded scores, in place: word e is formed of columns 2 e, 2 e + 1
            float all = 0.f;
#pragma unroll 1
            for (int e = 0; e < 32; ++e) {
              uint32_t u[2];
              tmem_ld2(tb + 2 * e, u);
              tmem_wait_ld();
              const float s0 = see >> (2 * e) & 1 ? __uint_as_float(u[0]) : -INFINITY;
              const float s1 = see >> (2 * e + 1) & 1 ? __uint_as_float(u[1]) : -INFINITY;
              const float p0 = ex2(far ? __fmul_rn(s0, c) - off : fmaf(s0, c, -off));
              const float p1 = ex2(far ? __fmul_rn(s1, c) - off : fmaf(s1, c, -off));
              all += p0 + p1;
              tmem_st1(tb + e, pack<T>(p0, p1));
              tmem_wait_st();
            }
            l += all;
          } else {
            GDP_TMEM_ST32(tb, w);
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          }
          tmem_wait_st();
        }
        const int z0 = x.keys - key0;
        if (z0 > 0 && z0 < kKeys && z0 % a.g) {  // rows of V behind the last key, in the last box
          ok = sy.wait(&bars[B_VFULL + stage], turn & 1);
          if (!ok) break;
          uint8_t* sv = sm + L::V + stage * L::TILE;
          const int z1 = (z0 + a.g - 1) / a.g * a.g;
#pragma unroll 1
          for (int e = tid & 127; e < (z1 - z0) * (KD / 8); e += 128) {
            const int r = z0 + e / (KD / 8), ch = e % (KD / 8);
            *reinterpret_cast<uint4*>(sv + (ch >> 3) * L::HALF + sw128_offset(r, (ch & 7) * 16)) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_async_smem();
        }
        if (owe) {  // the other slot has read this one's outputs of the last piece
          owe = false;
          ok = sy.wait(&bars[B_DONE], (joins - 1) & 1);
          if (!ok) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_P + 2 * slot + buf]);
      }
      const int nt = x.j1 - x.j0;
      tile0 += nt;
      other += d.two ? nt : nt - d.n;
      if (!ok) break;
      // Two slots on the same rows: each leaves its bases and sums, then joins half of the columns. (Both
      // slots' outputs lie in the same lanes of tensor memory.)
      const bool join = L::SLOTS == 2 && !d.two && nt > 1;
      float f0 = 1.f, f1 = 0.f;  // of this slot's and of the other's outputs
      if (d.n > 0) ok = sy.wait(&bars[B_O + 2 * slot + ((n - 1) & 1)], (n - 1) >> 1 & 1);
      if (join) {
        s_ml[slot * 128 + row] = make_float2(b, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_JOIN]);
        ok = ok && sy.wait(&bars[B_JOIN], joins & 1) && 
             sy.wait(&bars[B_O + 2 * (slot ^ 1) + ((other - 1) & 1)], (other - 1) >> 1 & 1);
        if (!ok) break;
        ++joins;
        owe = true;
        const float2 u = s_ml[(slot ^ 1) * 128 + row];
        const float bn = fmaxf(b, u.x), base = bn == -INFINITY ? 0.f : bn;
        f0 = ex2(b - base);
        f1 = ex2(u.x - base);
        b = bn;
        l = f0 * l + f1 * u.y;
      }
      if (!ok) break;
      tc_fence_after();
      if ((join || d.n > 0) && live) {
        const bool on = row < d.rows;
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        const int at = d.row0 - x.row0 + row;  // of the item's rows
        const int64_t cut = (int64_t)blockIdx.x * 2 + x.slot;
        const bool whole = x.slot < 0;
        if (!whole && on && (slot == 0 || d.two)) a.ml[cut * a.cap + at] = make_float2(b, l);
        float4* part = reinterpret_cast<float4*>(a.part + (whole ? 0 : cut * a.cap * a.dvp)) + at;
        T* dst = static_cast<T*>(p.o) + out_at(p, x.first, x.head, d.row0 + min(row, d.rows - 1));
        if (whole) { f0 *= inv; f1 *= inv; }
        const int q0 = join && slot ? KD / 2 : 0, q1 = join && !slot ? KD / 2 : KD;
        __syncwarp();
#pragma unroll 1
        for (int q = q0; q < q1; q += 32) {
          uint32_t o[32];
          GDP_TMEM_LD32(to + 128 * slot + q, o);
          if (join) {
            uint32_t u[32];
            GDP_TMEM_LD32(to + 128 * (slot ^ 1) + q, u);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(fmaf(f1, __uint_as_float(u[e]), __uint_as_float(o[e]) * f0));
          } else {
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            const float* y = reinterpret_cast<const float*>(o + e);
            if (on && q + e < p.DV) {
              if (whole) {
                *reinterpret_cast<uint4*>(dst + q + e) = make_uint4(pack<T>(y[0], y[1]), pack<T>(y[2], y[3]),
                                                                    pack<T>(y[4], y[5]), pack<T>(y[6], y[7]));
              } else {  // quads of columns outermost: lanes are side by side
                part[((q + e) >> 2) * a.cap] = make_float4(y[0], y[1], y[2], y[3]);
                part[(((q + e) >> 2) + 1) * a.cap] = make_float4(y[4], y[5], y[6], y[7]);
              }
            }
          }
          __syncwarp();  // (the loads from tensor memory are the whole warp's)
        }
      }
      tc_fence_before();
      if (join) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_DONE]);
      }
      if (x.slot == 1) {
        rec = true;
        if (tid == 0) write_rec(a, s_start, &x);
      }
    }
    if (!rec && tid == 0) write_rec(a, s_start, nullptr);
  } else if (warp < kScores) {
    // ---------------------------------------------------------------- loads
    // (One warp for K and V took 1350 cycles for a tile, longer than HBM's 1130.)
    const bool v = warp > kLoad;
    const int n = v ? L::NV : L::NK, empty = v ? B_VEMPTY - B_VFULL : B_KEMPTY - B_KFULL;
    uint64_t* full = &bars[v ? B_VFULL : B_KFULL];
    uint8_t* tiles = sm + (v ? L::V : L::K);
    int stage = 0;
    uint32_t turn = 1, loads = 0;
    // keys of the tile that are not there: known before its values are
    auto tell = [&](uint64_t absent) {
      if (!v) return;
      s_absent[stage] = absent;
      mbar_arrive(&bars[B_META + stage]);
    };
    if (TMA) {
      const int subs = kKeys / a.g;  // boxes of a tile and half: 1 to 8, so a lane's is the same in every round
      const int sub = lane % subs, boxes = subs * (KD / 64) / a.halves, col = lane / subs * 64;
      const CUtensorMap* map = v ? &map_v : &map_k;
      uint8_t* dst = tiles + sub * a.g * 128 + lane / subs * L::HALF;
#pragma unroll 1
      while (ok && walk.next(p, x)) {
        const int32_t* table = p.tables + (int64_t)x.r * p.width;
        // page of this lane's box in tile j; -1: none
        auto page_of = [&](int j) {
          const int key = j * kKeys + sub * a.g;
          return j < x.j1 && key < x.keys ? table[quot(key, p.by_block)] : -1;
        };
        int page = page_of(x.j0);
#pragma unroll 1
        for (int j = x.j0; j < x.j1; ++j) {
          const int next = page_of(j + 1), key = j * kKeys + sub * a.g;
          ok = sy.wait(full + empty + stage, turn);
          if (!ok) break;
          if (page >= p.n_pages) report(p.status, GDP_ERR_INVALID_ARG);
          const bool there = (uint32_t)page < (uint32_t)p.n_pages;
          const uint32_t gone = ~__ballot_sync(0xffffffffu, there) & ((1u << subs) - 1u);
          if (lane == 0) {
            uint64_t absent = 0;
            if (gone)
              for (int b = 0; b < subs; ++b)
                if (gone >> b & 1) absent |= low_bits(a.g) << (b * a.g);
            tell(absent);
            mbar_expect_tx(full + stage, L::TILE);
          }
          __syncwarp();
          if (lane < boxes)  // (a box past the last page arrives as zeros)
            tma_load_5d(dst + stage * L::TILE, map, col, x.head, key - (int)quot(key, p.by_block) * p.block,
                        there ? page : p.n_pages, 0, full + stage);
          if (++stage == n) { stage = 0; turn ^= 1; }
          ++loads;
          page = next;
        }
      }
    } else {
      // Pages whose size is not a multiple of 8: 16-byte copies, a row to KD / 8 lanes, three tiles in flight; a
      // tile is told full once its copies are done and visible to the tensor cores.
      constexpr int kLag = L::NK > 3 ? 3 : L::NK - 1, kRow = KD / 8, kBeside = 32 / kRow;  // tiles; lanes of a row, rows beside each other
      static_assert(kLag < L::NK, "a tile is told full before the wait for its buffer's next use");
      const T* base = static_cast<const T*>(v ? p.v : p.k);
      const int64_t s0 = v ? p.vs[0] : p.ks[0], s1 = v ? p.vs[1] : p.ks[1], s2 = v ? p.vs[2] : p.ks[2];
      const int ch = lane % kRow, width = v ? p.DV : p.D;
      int told = 0;       // stage of the next tile to be told
      uint32_t tell_of = 0;
      auto tell_full = [&]() {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full + told);
        if (++told == n) told = 0;
        ++tell_of;
      };
#pragma unroll 1
      while (ok && walk.next(p, x)) {
        const int32_t* table = p.tables + (int64_t)x.r * p.width;
        auto page_of = [&](int j, int half) {  // of key j kKeys + 32 half + lane
          const int key = j * kKeys + 32 * half + lane;
          return j < x.j1 && key < x.keys ? table[quot(key, p.by_block)] : -1;
        };
        int page0 = page_of(x.j0, 0), page1 = page_of(x.j0, 1);
#pragma unroll 1
        for (int j = x.j0; j < x.j1; ++j) {
          const int next0 = page_of(j + 1, 0), next1 = page_of(j + 1, 1), key0 = j * kKeys + lane, key1 = key0 + 32;
          ok = sy.wait(full + empty + stage, turn);
          if (!ok) break;
          if (page0 >= p.n_pages || page1 >= p.n_pages) report(p.status, GDP_ERR_INVALID_ARG);
          const bool there0 = (uint32_t)page0 < (uint32_t)p.n_pages, there1 = (uint32_t)page1 < (uint32_t)p.n_pages;
          const uint64_t gone = ~(__ballot_sync(0xffffffffu, there0) | (uint64_t)__ballot_sync(0xffffffffu, there1) << 32);
          if (lane == 0) tell(gone);
          const long long at0 = there0 ? page0 * s0 + (key0 - (int)quot(key0, p.by_block) * p.block) * s1 : -1;
          const long long at1 = there1 ? page1 * s0 + (key1 - (int)quot(key1, p.by_block) * p.block) * s1 : -1;
          const uint32_t dst = smem_u32(tiles + stage * L::TILE) + (ch >> 3) * L::HALF;
#pragma unroll 4
          for (int i = 0; i < kKeys; i += kBeside) {
            const int r = i + lane / kRow;
            const long long a0 = __shfl_sync(0xffffffffu, i < 32 ? at0 : at1, r & 31);
            const bool in = a0 >= 0 && 8 * ch < width;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + sw128_offset(r, (ch & 7) * 16)),
                         "l"(base + (in ? a0 + x.head * s2 + 8 * ch : 0)), "r"(in ? 16 : 0)
                         : "memory");
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (++stage == n) { stage = 0; turn ^= 1; }
          if (++loads > kLag) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
            tell_full();
          }
          page0 = next0;
          page1 = next1;
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      while (tell_of < loads) tell_full();
    }
    // the last buffers' commits land before the CTA leaves, and so do copies in flight where a wait ran out
    for (uint32_t b = loads > n ? loads - n : 0; ok && b < loads; ++b) ok = sy.wait(full + empty + b % n, (b / n) & 1);
    if (TMA && *s_dead)
      for (uint32_t b = loads > n ? loads - n : 0; b < loads; ++b)
        for (int tries = 0; tries < 1000 && !mbar_test_for(full + b % n, (b / n) & 1, 20000); ++tries) {}
  } else {
    // ---------------------------------------------------------------- products
    // One thread forms the scores, another the outputs, each tile by tile for both slots in turn: with both in one
    // warp a tile of 2 x 128 rows took 2800 cycles, its waits and issues one after another, and votes and elections
    // in every step cost a tenth.
    const bool pv = warp == kOutputs;
    const uint32_t id_s = idesc<T>(128, kKeys, false) | (p.c < 0.f ? 1u << 13 : 0u);  // (-Q)
    constexpr uint32_t id_o = idesc<T>(128, KD, true);
    const uint32_t base = smem_u32(sm);
    if (elect_one()) {
      uint32_t stage = 0, turn = 0, n0 = 0, n1 = 0;  // buffer of the next tile; tiles of the slots
      if (!pv) {
        const uint64_t qd = sdesc_sw128(base + L::Q, 16, 1024), kd = sdesc_sw128(base + L::K, 16, 1024);
        uint32_t nq0 = 0, nq1 = 0;
#pragma unroll 1
        while (ok && walk.next(p, x)) {
          const int nt = x.j1 - x.j0;
          const bool two = L::SLOTS == 2 && x.rows > 128;
          const int steps = two ? 2 * nt : nt;
#pragma unroll 1
          for (int i = 0; i < steps; ++i) {
            const int s = L::SLOTS == 2 ? i & 1 : 0;
            const uint32_t n = s ? n1 : n0, buf = n & 1;
            // Scores go over the weights of two tiles before, once those have been multiplied; in a piece's first
            // two tiles they have been, and its queries are there.
            if (i < L::SLOTS) {
              ok = sy.wait1(&bars[B_Q + s], (s ? nq1 : nq0) & 1);
              if (s) ++nq1; else ++nq0;
            } else if (i >= 2 * L::SLOTS) {
              ok = sy.wait1(&bars[B_O + 2 * s + buf], (n >> 1) - 1 & 1);
            }
            ok = ok && ((two && s) || sy.wait1(&bars[B_KFULL + stage], turn));
            if (!ok) break;
            tc_fence_after();
            mma_run<KD / 16, false, 16384, 32, L::HALF, 32>(tmem + T_S + 128 * s + 64 * buf, qd + s * (L::QT >> 4),
                                                            kd + stage * (L::TILE >> 4), id_s);
            mma_commit(&bars[B_S + 2 * s + buf]);
            if (s) ++n1; else ++n0;
            if (!two || s) {  // the last step of the tile
              mma_commit(&bars[B_KEMPTY + stage]);
              if (++stage == L::NK) { stage = 0; turn ^= 1; }
            }
          }
        }
      } else {
        const uint64_t vd = sdesc_sw128(base + L::V, L::HALF, 1024);
#pragma unroll 1
        while (ok && walk.next(p, x)) {
          const int nt = x.j1 - x.j0;
          const bool two = L::SLOTS == 2 && x.rows > 128;
          const int steps = two ? 2 * nt : nt;
#pragma unroll 1
          for (int i = 0; i < steps; ++i) {
            const int s = L::SLOTS == 2 ? i & 1 : 0;
            const uint32_t n = s ? n1 : n0;
            ok = sy.wait1(&bars[B_P + 2 * s + (n & 1)], n >> 1 & 1) &&
                 ((two && s) || sy.wait1(&bars[B_VFULL + stage], turn));
            if (!ok) break;
            tc_fence_after();
            const uint64_t v = vd + stage * (L::TILE >> 4);
#pragma unroll
            for (int e = 0; e < kKeys / 16; ++e)
              mma_bf16_ts(tmem + T_O + 128 * s, tmem + T_S + 128 * s + 64 * (n & 1) + 8 * e, v + e * (2048 >> 4),
                          id_o, i >= L::SLOTS || e > 0);
            mma_commit(&bars[B_O + 2 * s + (n & 1)]);
            if (s) ++n1; else ++n0;
            if (!two || s) {
              mma_commit(&bars[B_VEMPTY + stage]);
              if (++stage == L::NV) { stage = 0; turn ^= 1; }
            }
          }
        }
      }
      if (!ok) {  // products in flight end before their operands and columns go away
        mma_commit(&bars[B_END + pv]);
        for (int tries = 0; tries < 1000 && !mbar_test_for(&bars[B_END + pv], 0, 20000); ++tries) {}
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kScores) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ host
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

// [pages][places][heads][D] with element strides s (page, place, head); boxes of 64 columns of g places, or of
// both halves of 128 columns side by side.
bool map5(CUtensorMap* m, const Problem& p, const void* base, int D, const int64_t* s, int g, int halves) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const bool both = halves == 2;
  const cuuint64_t dims[5] = {(cuuint64_t)(both ? 64 : D), (cuuint64_t)p.HKV, (cuuint64_t)p.block, (cuuint64_t)p.n_pages,
                              (cuuint64_t)(both ? 2 : 1)};
  // the stride of a dimension of one entry is never used; the encoder wants a valid one
  const cuuint64_t some = 16;
  const cuuint64_t st[4] = {p.HKV > 1 ? (cuuint64_t)s[2] * 2 : some, p.block > 1 ? (cuuint64_t)s[1] * 2 : some,
                            p.n_pages > 1 ? (cuuint64_t)s[0] * 2 : some, both ? (cuuint64_t)128 : some};
  const cuuint32_t box[5] = {64, 1, (cuuint32_t)g, 1, (cuuint32_t)halves}, es[5] = {1, 1, 1, 1, 1};
  return fn(m, p.dt == GDP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
            const_cast<void*>(base), dims, st, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int KD, bool TMA>
cudaError_t go(const TcArgs& a, const CUtensorMap* m) {
  const cudaError_t e = allow_smem<attention_kernel<T, KD, TMA>>(Lay<KD>::BYTES);
  return e != cudaSuccess ? e
                          : launch_pdl(attention_kernel<T, KD, TMA>, dim3(a.ctas), dim3(kThreads), Lay<KD>::BYTES,
                                       a.p.stream, m[0], m[1], a);
}
template <typename T>
cudaError_t go(const TcArgs& a, const CUtensorMap* m, bool tma) {
  if (a.p.D > 128 || a.p.DV > 128) return tma ? go<T, 256, true>(a, m) : go<T, 256, false>(a, m);
  if (a.p.D > 64 || a.p.DV > 64) return tma ? go<T, 128, true>(a, m) : go<T, 128, false>(a, m);
  return tma ? go<T, 64, true>(a, m) : go<T, 64, false>(a, m);
}

}  // namespace

bool tc_shape(int D, int DV, gdp_dtype dt) {
  return (dt == GDP_BF16 || dt == GDP_F16) && D <= 256 && DV <= 256 && D % 8 == 0 && DV % 8 == 0;
}

bool tc_ok(const Problem& p) {
  const auto fits = [](int n, int64_t x) { return n <= 1 || (x > 0 && x % 8 == 0 && x < ((int64_t)1 << 38)); };
  const auto even = [](const void* x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; };
  if (!tc_shape(p.D, p.DV, p.dt) || p.n_pages < 1) return false;
  if (!even(p.q) || !even(p.k) || !even(p.v) || !even(p.o)) return false;
  const int qn[3] = {p.B, p.T, p.H}, cn[3] = {p.n_pages, p.block, p.HKV};
  for (int i = 0; i < 3; ++i)
    if ((qn[i] > 1 && p.qs[i] % 8) || !fits(cn[i], p.ks[i]) || !fits(cn[i], p.vs[i])) return false;
  return true;
}

static Layout tc_layout(int64_t rows, int D, int DV) {
  return layout(sm_count(), rows, D > 128 || DV > 128 ? Lay<256>::ROWS : Lay<128>::ROWS, DV);
}
size_t tc_workspace(int64_t rows, int D, int DV) { return tc_layout(rows, D, DV).total; }

void wait_fault(int arm, unsigned long long budget_ns) {
  g_fault.store(arm);
  g_budget_ns.store(budget_ns);
}

cudaError_t launch_tc(const Problem& p, uint8_t* ws) {
  TcArgs a{};
  a.p = p;
  set_layout(a, tc_layout((int64_t)p.T * p.G, p.D, p.DV), ws, sm_count());
  a.cost = p.D > 128 || p.DV > 128 ? kCostWide : kCost;
  a.budget = (int)(g_budget_ns.load() >> 10);
  a.fault = g_fault.exchange(0);
  CUtensorMap m[2] = {};
  const bool tma = p.block % 8 == 0;  // (swizzled boxes begin on 8 rows)
  a.g = tma ? 8 : 1;
  while (tma && a.g < kKeys && p.block % (2 * a.g) == 0) a.g *= 2;
  // (a box of both halves needs its rows to be a whole half's)
  a.halves = a.g == kKeys && p.D == 128 && p.DV == 128 ? 2 : 1;
  if (tma && (!map5(&m[0], p, p.k, p.D, p.ks, a.g, a.halves) || !map5(&m[1], p, p.v, p.DV, p.vs, a.g, a.halves)))
    return cudaErrorInvalidValue;
  const cudaError_t e = p.dt == GDP_BF16 ? go<__nv_bfloat16>(a, m, tma) : go<__half>(a, m, tma);
  return e != cudaSuccess ? e : launch_combine(a);
}

}  // namespace attn
}  // namespace gdp
