// Attention of new tokens over a paged cache on the tensor cores: bf16 and fp16, heads of up to 128
// elements, pages whose size is a multiple of 8.
//
// A CTA walks the pieces of its share (attention.cuh) with two slots, each with four warps of its own,
// 128 columns of scores and KD of outputs in tensor memory:
//   more than 128 rows: the slots are two tiles of 128 rows that read the same keys;
//   fewer: both slots have the same rows and take the key tiles in turn, and their two maxima, sums and
//   outputs are joined at the piece's end.
// So one slot's softmax runs beside the other's products either way, and a decode step's few rows cost
// what streaming their keys costs: the products of a padded tile of 128 rows take a fifth of the time
// that HBM needs for its keys.
//
// A key tile: S = Q K^T (tcgen05, K-major operands), then a thread per row takes its 128 scores from
// tensor memory, forms p = 2^(c s - m) in registers and puts them back as 16-bit pairs over S, and
// O += P V takes P from there and V as it lies (MN-major). m only follows the row's maximum when that
// has grown by more than 2^8 (then O is scaled in tensor memory): p stays below 2^8, and a 16-bit p
// keeps its relative precision. Sums are fp32.
//
// One warp loads: boxes of 64 columns and `g` keys, g the largest power of two that divides both the
// page and the tile, through tensor maps of the whole caches. Pages that are not there are boxes past
// the last page, which arrive as zeros, and so are boxes behind the last key; what remains of the
// last box is zeroed in shared memory before it is multiplied (weights of 0 times NaN are not 0).
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

constexpr int kRows = 256, kKeys = 64;
constexpr int kLoad = 8, kMma = 9;  // warps; 0 to 3 and 4 to 7 are the slots', 9 and 10 issue their products
constexpr int kThreads = 352;
constexpr float kGrow = 8.f;        // log2 of how far the maximum may lie above m

template <int KD>
struct Lay {
  static constexpr int NB = KD == 128 ? 5 : 10;  // stages of the ring, a tile of K and one of V each
  static constexpr int HALF = kKeys * 128;       // 64 columns of a tile: 64 rows of 128 bytes
  static constexpr int TILE = KD / 64 * HALF;
  static constexpr int QT = KD / 64 * 16384;     // 128 rows of queries
  static constexpr int Q = 0, RING = 2 * QT;
  static constexpr int BAR = RING + NB * 2 * TILE;
  static constexpr int ML = BAR + 384;           // maxima and sums [2][128]
  static constexpr int START = ML + 2048;        // the share, and the sums that lead to it
  static constexpr int BYTES = START + 192;
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};
// by stage: full, empty; by slot and buffer: scores, weights, outputs (of the buffer's tile: a waiter may be two
// tiles behind, which one barrier's parity cannot tell from none); by slot: queries; a piece's two slots have left
// their maxima, have read each other's outputs
enum { B_FULL = 0, B_EMPTY = 10, B_S = 20, B_P = 24, B_O = 28, B_Q = 32, B_JOIN = 34, B_DONE, B_END, B_N = B_END + 2 };
constexpr uint32_t T_S = 0, T_O = 256;  // columns: S [2][2][64], O [2][128]

struct TcArgs : Args {
  int g;          // keys of a box
  int budget;     // limit of a wait, in units of 1024 ns
  int fault;      // test hook (gdp_debug_wait_fault): CTA 0 waits for a commit more of its first scores
};

// ------------------------------------------------------------------ waits
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* dead, int budget, int* status) {
  uint64_t t0 = 0;
  while (!mbar_test_for(bar, parity, 20000)) {
    if (*dead) return false;
    const uint64_t t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    if (((t - t0) >> 10) > (uint32_t)budget) {
      if (status) atomicExch(status, kDevTimeout);
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
    const bool ok = mbar_test(bar, parity) || wait_slow(bar, parity, dead, budget, status);
    return __all_sync(0xffffffffu, ok);
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
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
// The lowest n bits (n outside 0 .. 32 is held to it).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// How a piece's tiles are spread over the slots.
struct Spread {
  bool two;       // tiles of rows of their own, the same keys
  int n, rows, row0;
  __device__ __forceinline__ Spread(const Piece& x, int slot) {
    two = x.rows > 128;
    n = two ? x.j1 - x.j0 : (x.j1 - x.j0 + 1 - slot) / 2;
    rows = two ? (slot ? x.rows - 128 : 128) : x.rows;
    row0 = x.row0 + (two ? 128 * slot : 0);
  }
};

template <typename T, int KD>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ TcArgs a) {
  using L = Lay<KD>;
  extern __shared__ __align__(1024) uint8_t sm[];  // (nothing static beside it: the array begins on a swizzle atom)
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + B_N);
  volatile int* s_dead = reinterpret_cast<volatile int*>(s_tmem + 1);
  uint32_t* s_absent = s_tmem + 2;                                     // [NB]
  float2* s_ml = reinterpret_cast<float2*>(sm + L::ML);                // [2][128]
  Start& s_start = *reinterpret_cast<Start*>(sm + L::START);
  long long* s_scan = reinterpret_cast<long long*>(sm + L::START + 96);  // [kThreads / 32]
  static_assert(sizeof(Start) <= 96 && kThreads / 32 * 8 <= 96 && B_N * 8 + 8 + L::NB * 4 <= 384, "shared memory");
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const Problem& p = a.p;

  if (warp == kMma) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (tid < B_N) {
    int n = 1;
    if (tid >= B_P && tid < B_O) n = 4;                                // warps of the slot
    if (tid >= B_Q && tid < B_JOIN) n = 4;
    if (tid == B_JOIN || tid == B_DONE) n = 8;
    if (tid >= B_EMPTY && tid < B_S) n = 2;                            // both slots
    if (tid == B_S && a.fault && blockIdx.x == 0) n = 2;
    mbar_init(&bars[tid], n);
    fence_mbar_init();
  }
  if (tid == 64) *s_dead = 0;
  if (warp == kLoad && lane == 0) {
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  pdl_wait();
  find_start<kRows, kKeys, kThreads>(a, &s_start, s_scan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const Sync sy{s_dead, a.budget, p.status};
  Walk<kRows, kKeys> walk(s_start);
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
      const Spread d(x, slot);
      if (d.n > 0) {  // Q: 16-byte chunks of the rows, zero behind the head's end
#pragma unroll 1
        for (int i = tid & 127; i < d.rows * (KD / 8); i += 128) {
          const int r = i / (KD / 8), ch = i % (KD / 8), R = d.row0 + r, t = (int)quot(R, p.by_G);
          const int h = x.head * p.G + R - t * p.G;
          const int64_t at = p.cu ? (x.first + t) * p.qs[1] : x.r * p.qs[0] + t * p.qs[1];
          const T* src = static_cast<const T*>(p.q) + at + h * p.qs[2] + (8 * ch < p.D ? 8 * ch : 0);
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
      const uint64_t bits = p.tree && x.x.ok ? (uint64_t)p.tree[x.first + t] : 0ull;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int k = 0; ok && k < d.n; ++k, ++n) {
        const int j = d.two ? k : 2 * k + slot, key0 = (x.j0 + j) * kKeys;
        const uint32_t stage = (tile0 + j) % L::NB, turn = (tile0 + j) / L::NB;
        const uint32_t buf = n & 1, tb = ts + 64 * buf;
        ok = sy.wait(&bars[B_S + 2 * slot + buf], (n >> 1) & 1) && sy.wait(&bars[B_FULL + stage], turn & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t absent = s_absent[stage];
        if (live) {
          if (key0 + kKeys > x.x.ctx || absent) {  // some of the keys are not seen by some row
#pragma unroll 1
            for (int q = 0; q < kKeys; q += 8) {
              const int k0 = key0 + q;
              uint32_t see;
              if (p.tree) {
                const int back = k0 - x.x.ctx;
                see = low_bits(-back);
                if (back > -8 && back < 64) see |= (uint32_t)(back >= 0 ? bits >> back : bits << -back);
              } else {
                see = low_bits(x.x.ctx + t + 1 - k0);
              }
              see &= low_bits(x.keys - k0);
              if (absent >> (q / a.g) & 1) see = 0;
              uint32_t s[8];
              GDP_TMEM_LD8(tb + q, s);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) s[e] = see >> e & 1 ? s[e] : __float_as_uint(-INFINITY);
              GDP_TMEM_ST8(tb + q, s);
            }
            tmem_wait_st();
          }
          uint32_t s[kKeys];
          GDP_TMEM_LD32(tb, s);
          GDP_TMEM_LD32(tb + 32, (s + 32));
          tmem_wait_ld();
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kKeys; ++e) top[e & 3] = fmaxf(top[e & 3], __uint_as_float(s[e]));
          const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
          const bool grow = mt > m + kGrow;  // (from -inf: as soon as anything is seen)
          if (__any_sync(0xffffffffu, grow)) {
            const float mn = grow ? mt : m, f = grow ? ex2(m - mn) : 1.f;
            m = mn;
            l *= f;
            if (k > 0) {  // the last product into O is done, then O is scaled
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
          const float base = m == -INFINITY ? 0.f : m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float p0 = ex2(fmaf(__uint_as_float(s[2 * e]), c, -base));
            const float p1 = ex2(fmaf(__uint_as_float(s[2 * e + 1]), c, -base));
            sum[2 * (e & 1)] += p0;
            sum[2 * (e & 1) + 1] += p1;
            w[e] = pack<T>(p0, p1);
          }
          GDP_TMEM_ST32(tb, w);
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        const int z0 = x.keys - key0;
        if (z0 > 0 && z0 < kKeys && z0 % a.g) {  // rows of V behind the last key, in the last box
          uint8_t* sv = sm + L::RING + stage * 2 * L::TILE + L::TILE;
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
      // Two slots on the same rows: each leaves its maxima and sums, then joins half of the columns. (Both
      // slots' outputs lie in the same lanes of tensor memory.)
      const bool join = !d.two && nt > 1;
      float f0 = 1.f, f1 = 0.f;  // of this slot's and of the other's outputs
      if (d.n > 0) ok = sy.wait(&bars[B_O + 2 * slot + ((n - 1) & 1)], (n - 1) >> 1 & 1);
      if (join) {
        s_ml[slot * 128 + row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_JOIN]);
        ok = ok && sy.wait(&bars[B_JOIN], joins & 1) && 
             sy.wait(&bars[B_O + 2 * (slot ^ 1) + ((other - 1) & 1)], (other - 1) >> 1 & 1);
        if (!ok) break;
        ++joins;
        owe = true;
        const float2 u = s_ml[(slot ^ 1) * 128 + row];
        const float mn = fmaxf(m, u.x), base = mn == -INFINITY ? 0.f : mn;
        f0 = ex2(m - base);
        f1 = ex2(u.x - base);
        m = mn;
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
        if (!whole && on && (slot == 0 || d.two)) a.ml[cut * a.cap + at] = make_float2(m, l);
        float4* part = reinterpret_cast<float4*>(a.part + (whole ? 0 : cut * a.cap * a.dvp)) + at;
        T* dst = static_cast<T*>(p.o) + out_at(p, x.first, x.head, d.row0 + min(row, d.rows - 1));
        if (whole) { f0 *= inv; f1 *= inv; }
        const int q0 = join && slot ? KD / 2 : 0, q1 = join && !slot ? KD / 2 : KD;
        __syncwarp();
#pragma unroll 1
        for (int q = q0; q < q1; q += 8) {
          uint32_t o[8], u[8];
          GDP_TMEM_LD8(to + 128 * slot + q, o);
          if (join) GDP_TMEM_LD8(to + 128 * (slot ^ 1) + q, u);
          tmem_wait_ld();
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] = __uint_as_float(o[e]) * f0;
            if (join) y[e] = fmaf(f1, __uint_as_float(u[e]), y[e]);
          }
          if (on && q < p.DV) {
            if (whole) {
              *reinterpret_cast<uint4*>(dst + q) = make_uint4(pack<T>(y[0], y[1]), pack<T>(y[2], y[3]),
                                                              pack<T>(y[4], y[5]), pack<T>(y[6], y[7]));
            } else {  // quads of columns outermost: lanes are side by side
              part[(q >> 2) * a.cap] = make_float4(y[0], y[1], y[2], y[3]);
              part[((q >> 2) + 1) * a.cap] = make_float4(y[4], y[5], y[6], y[7]);
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
        if (tid == 0) write_rec(a, s_start, &x, walk.at - nt);
      }
    }
    if (!rec && tid == 0) write_rec(a, s_start, nullptr, 0);
  } else if (warp == kLoad) {
    // ---------------------------------------------------------------- loads
    const int subs = kKeys / a.g;  // boxes of a tile and half: 1 to 8, so a lane's is the same in every round
    const int sub = lane % subs;
    uint32_t i = 0;
#pragma unroll 1
    while (ok && walk.next(p, x)) {
      const int32_t* table = p.tables + (int64_t)x.r * p.width;
      auto page_of = [&](int j, int& place) {  // n_pages: a box of zeros
        const int key = j * kKeys + sub * a.g;
        place = 0;
        if (j >= x.j1 || key >= x.keys) return p.n_pages;
        const int b = (int)quot(key, p.by_block), page = table[b];
        place = key - b * p.block;
        if (page >= p.n_pages && p.status) *p.status = GDP_ERR_INVALID_ARG;
        return page >= 0 && page < p.n_pages ? page : p.n_pages;
      };
      int place, page = page_of(x.j0, place);
#pragma unroll 1
      for (int j = x.j0; j < x.j1; ++j, ++i) {
        int place1;
        const int page1 = page_of(j + 1, place1);
        const uint32_t absent = __ballot_sync(0xffffffffu, page == p.n_pages) & low_bits(subs);
        const uint32_t stage = i % L::NB;
        ok = sy.wait(&bars[B_EMPTY + stage], ((i / L::NB) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          s_absent[stage] = absent;
          mbar_expect_tx(&bars[B_FULL + stage], 2 * L::TILE);
        }
        __syncwarp();
        uint8_t* dst = sm + L::RING + stage * 2 * L::TILE + sub * a.g * 128;
#pragma unroll 1
        for (int b = lane; b < subs * (KD / 32); b += 32) {  // halves of K, then of V
          const int half = b / subs;
          const bool v = half >= KD / 64;
          tma_load_4d(dst + half * L::HALF, v ? &map_v : &map_k, (v ? half - KD / 64 : half) * 64, x.head, place, page,
                      &bars[B_FULL + stage]);
        }
        page = page1;
        place = place1;
      }
    }
    // the last stages' commits land before the CTA leaves, and so do copies in flight where a wait ran out
    for (uint32_t b = i > L::NB ? i - L::NB : 0; ok && b < i; ++b)
      ok = sy.wait(&bars[B_EMPTY + b % L::NB], (b / L::NB) & 1);
    if (*s_dead)
      for (uint32_t b = i > L::NB ? i - L::NB : 0; b < i; ++b)
        for (int tries = 0; tries < 1000 && !mbar_test_for(&bars[B_FULL + b % L::NB], (b / L::NB) & 1, 20000); ++tries) {}
  } else {
    // ---------------------------------------------------------------- products
    // A warp for each slot (a step of its loop, four waits and twelve products, takes 1000 cycles: with one
    // warp for both a tile of 2 x 128 rows took 2800, and a decode step's tile 1400). Scores are formed up to two
    // tiles ahead of the outputs, whichever of the two can be first.
    const int slot = warp - kMma;
    const uint32_t id_s = idesc<T>(128, kKeys, false) | (p.c < 0.f ? 1u << 13 : 0u);  // (-Q)
    constexpr uint32_t id_o = idesc<T>(128, KD, true);
    const uint32_t base = smem_u32(sm), ts = tmem + T_S + 128 * slot, to = tmem + T_O + 128 * slot;
    const uint64_t qd = sdesc_sw128(base + L::Q + slot * L::QT, 16, 1024);
    const uint64_t kd = sdesc_sw128(base + L::RING, 16, 1024);
    const uint64_t vd = sdesc_sw128(base + L::RING + L::TILE, L::HALF, 1024);
    auto poll = [](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_poll(bar, parity)); };
    uint32_t tile0 = 0, ns = 0, np = 0, nq = 0;  // tiles of the CTA; this slot's scores, weights, queries
#pragma unroll 1
    while (ok && walk.next(p, x)) {
      const Spread d(x, slot);
      const int nt = x.j1 - x.j0;
      // stages of the next tile and of the next outputs
      uint32_t ks = tile0 % L::NB, kt = tile0 / L::NB & 1, os = (tile0 + (d.two ? 0 : slot)) % L::NB;
      int k = 0, is = 0, io = 0, done = 0;  // tiles whose scores and outputs are under way, whose outputs are complete
      bool queries = false;
      uint64_t t0 = 0;
      int spins = 0;
#pragma unroll 1
      while (io < d.n || k < nt) {
        bool moved = false, seen = false;
        // (products into different columns may overtake one another: scores go over weights only once those
        // have been multiplied)
        if (done < io && poll(&bars[B_O + 2 * slot + ((np - 1) & 1)], (np - 1) >> 1 & 1)) done = io;
        // Every tile is waited for in turn, the other slot's too, and both slots release its stage: a warp that
        // skipped tiles could take a stage's last but one load for the last (a parity tells only two apart).
        if (k < nt && (!d.two && (k & 1) != slot)) {
          if (poll(&bars[B_FULL + ks], kt)) {
            if (lane == 0) mbar_arrive(&bars[B_EMPTY + ks]);
            seen = true;
          }
        } else if (k < nt && is < done + 2) {
          if (!queries) queries = poll(&bars[B_Q + slot], nq & 1);
          if (queries && poll(&bars[B_FULL + ks], kt)) {
            __syncwarp();
            tc_fence_after();
            if (elect_one()) {
              mma_run<KD / 16, false, 16384, 32, L::HALF, 32>(ts + 64 * (ns & 1), qd, kd + ks * (2 * L::TILE >> 4), id_s);
              mma_commit(&bars[B_S + 2 * slot + (ns & 1)]);
            }
            __syncwarp();
            ++ns;
            ++is;
            seen = true;
          }
        }
        if (seen) {
          ++k;
          if (++ks == L::NB) { ks = 0; kt ^= 1; }
          moved = true;
        }
        if (io < is && done == io && poll(&bars[B_P + 2 * slot + (np & 1)], np >> 1 & 1)) {
          __syncwarp();
          tc_fence_after();
          if (elect_one()) {
            const uint64_t v = vd + os * (2 * L::TILE >> 4);
#pragma unroll
            for (int e = 0; e < kKeys / 16; ++e)
              mma_bf16_ts(to, ts + 64 * (np & 1) + 8 * e, v + e * (2048 >> 4), id_o, io > 0 || e > 0);
            mma_commit(&bars[B_O + 2 * slot + (np & 1)]);
            mma_commit(&bars[B_EMPTY + os]);
          }
          __syncwarp();
          ++np;
          ++io;
          os += d.two ? 1 : 2;
          if (os >= L::NB) os -= L::NB;
          moved = true;
        }
        if (moved) {
          spins = 0;
          t0 = 0;
        } else if (++spins > 256) {
          spins = 0;
          const uint64_t now = globaltimer_ns();
          if (t0 == 0) t0 = now;
          const bool over = *s_dead || ((now - t0) >> 10) > (uint32_t)a.budget;
          if (__any_sync(0xffffffffu, over)) {
            if (lane == 0 && !*s_dead) {
              if (p.status) atomicExch(p.status, kDevTimeout);
              *s_dead = 1;
            }
            ok = false;
            break;
          }
        }
      }
      if (queries) ++nq;
      tile0 += nt;
    }
    if (!ok) {  // products in flight end before their operands and columns go away
      if (elect_one()) mma_commit(&bars[B_END + slot]);
      for (int tries = 0; tries < 1000 && !mbar_test_for(&bars[B_END + slot], 0, 20000); ++tries) {}
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, 512);
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

// [pages][places][heads][D] with element strides s (page, place, head); boxes of 64 x 1 x g x 1.
bool map4(CUtensorMap* m, const Problem& p, const void* base, int D, const int64_t* s, int g) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)p.HKV, (cuuint64_t)p.block, (cuuint64_t)p.n_pages};
  // the stride of a dimension of one entry is never used; the encoder wants a valid one
  const cuuint64_t some = 16;
  const cuuint64_t st[3] = {p.HKV > 1 ? (cuuint64_t)s[2] * 2 : some, p.block > 1 ? (cuuint64_t)s[1] * 2 : some,
                            p.n_pages > 1 ? (cuuint64_t)s[0] * 2 : some};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)g, 1}, es[4] = {1, 1, 1, 1};
  return fn(m, p.dt == GDP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(base), dims, st, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int KD>
cudaError_t go(const TcArgs& a, const CUtensorMap* m) {
  const cudaError_t e = allow_smem<attention_kernel<T, KD>>(Lay<KD>::BYTES);
  return e != cudaSuccess ? e
                          : launch_pdl(attention_kernel<T, KD>, dim3(a.ctas), dim3(kThreads), Lay<KD>::BYTES,
                                       a.p.stream, m[0], m[1], a);
}

}  // namespace

bool tc_shape(int D, int DV, gdp_dtype dt) {
  return (dt == GDP_BF16 || dt == GDP_F16) && D <= 128 && DV <= 128 && D % 8 == 0 && DV % 8 == 0;
}

bool tc_ok(const Problem& p) {
  const auto fits = [](int n, int64_t x) { return n <= 1 || (x > 0 && x % 8 == 0 && x < ((int64_t)1 << 38)); };
  const auto even = [](const void* x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; };
  if (!tc_shape(p.D, p.DV, p.dt) || p.block % 8 || p.n_pages < 1) return false;
  if (!even(p.q) || !even(p.k) || !even(p.v) || !even(p.o)) return false;
  const int qn[3] = {p.B, p.T, p.H}, cn[3] = {p.n_pages, p.block, p.HKV};
  for (int i = 0; i < 3; ++i)
    if ((qn[i] > 1 && p.qs[i] % 8) || !fits(cn[i], p.ks[i]) || !fits(cn[i], p.vs[i])) return false;
  return true;
}

size_t tc_workspace(int64_t rows, int DV) { return layout(sm_count(), rows, kRows, DV).total; }

void wait_fault(int arm, unsigned long long budget_ns) {
  g_fault.store(arm);
  g_budget_ns.store(budget_ns);
}

cudaError_t launch_tc(const Problem& p, uint8_t* ws) {
  TcArgs a{};
  a.p = p;
  set_layout(a, layout(sm_count(), (int64_t)p.T * p.G, kRows, p.DV), ws, sm_count());
  a.g = 8;
  while (a.g < kKeys && p.block % (2 * a.g) == 0) a.g *= 2;
  a.budget = (int)(g_budget_ns.load() >> 10);
  a.fault = g_fault.exchange(0);
  CUtensorMap m[2];
  if (!map4(&m[0], p, p.k, p.D, p.ks, a.g) || !map4(&m[1], p, p.v, p.DV, p.vs, a.g)) return cudaErrorInvalidValue;
  const bool wide = p.D > 64 || p.DV > 64;
  cudaError_t e;
  if (p.dt == GDP_BF16)
    e = wide ? go<__nv_bfloat16, 128>(a, m) : go<__nv_bfloat16, 64>(a, m);
  else
    e = wide ? go<__half, 128>(a, m) : go<__half, 64>(a, m);
  return e != cudaSuccess ? e : launch_combine(a);
}

}  // namespace attn
}  // namespace gdp
