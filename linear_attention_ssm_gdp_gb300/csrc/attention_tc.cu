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

constexpr int kRows = 256, kKeys = 128;
constexpr int kLoad = 8, kMma = 9;  // warps; 0 to 3 and 4 to 7 are the slots'
constexpr int kThreads = 320;
constexpr int kMeta = 8;            // tiles whose absent boxes are on record
constexpr float kGrow = 8.f;        // log2 of how far the maximum may lie above m

template <int KD>
struct Lay {
  static constexpr int NB = KD == 128 ? 5 : 8;   // buffers of the ring, each a tile of K or of V
  static constexpr int TILE = KD / 64 * 16384;   // halves of 64 columns: 128 rows of 128 bytes
  static constexpr int Q = 0;                    // two tiles of rows
  static constexpr int RING = 2 * TILE;
  static constexpr int BAR = RING + NB * TILE;
  static constexpr int BYTES = BAR + 1536 + 1024;       // (barriers, maxima and sums; alignment)
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};
enum { B_FULL = 0, B_EMPTY = 8, B_S = 16, B_P = 18, B_O = 20, B_Q = 22, B_META = 24, B_JOIN = 32, B_END, B_N };
constexpr uint32_t T_S = 0, T_O = 256;  // columns: S [2][128], O [2][128]

struct TcArgs : Args {
  int g;          // keys of a box
  int box_bytes;
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
  int first, step, n, rows, row0;
  __device__ __forceinline__ Spread(const Piece& x, int slot) {
    two = x.rows > 128;
    first = two ? x.j0 : x.j0 + slot;
    step = two ? 1 : 2;
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
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + B_N);
  volatile int* s_dead = reinterpret_cast<volatile int*>(s_tmem + 1);
  uint32_t* s_absent = s_tmem + 2;                               // [kMeta]
  float2* s_ml = reinterpret_cast<float2*>(sm + L::BAR + 384);   // [128]: the second slot's
  __shared__ Start s_start;
  __shared__ long long s_scan[kThreads / 32 + 1];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const Problem& p = a.p;

  if (warp == kMma) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < B_N; ++i) {
      int n = 1;
      if (i >= B_P && i < B_O) n = 4;                            // warps of the slot
      if (i >= B_Q && i < B_META) n = 4;
      if (i == B_JOIN) n = 8;
      if (i == B_S && a.fault && blockIdx.x == 0) n = 2;
      mbar_init(&bars[i], n);
    }
    fence_mbar_init();
    *s_dead = 0;
  }
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
    const uint32_t ts = tmem + lanes + T_S + 128 * slot, to = tmem + lanes + T_O + 128 * slot;
    const float c = fabsf(p.c);
    const uint32_t flip = p.c < 0.f ? 0x80008000u : 0u;
    uint8_t* sq = sm + L::Q + slot * L::TILE;
    float* so = reinterpret_cast<float*>(sm + L::Q);             // [KD][128]: the second slot's outputs
    uint32_t n = 0, tile0 = 0, joins = 0;  // this slot's tiles so far, the CTA's at the piece's start
    bool rec = false;
    while (ok && walk.next(p, x)) {
      const Spread d(x, slot);
      if (d.n > 0) {  // Q: 16-byte chunks of the rows, zero behind the head's end
        for (int i = tid & 127; i < d.rows * (KD / 8); i += 128) {
          const int r = i / (KD / 8), ch = i % (KD / 8), R = d.row0 + r, t = R / p.G, h = x.head * p.G + R - t * p.G;
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (8 * ch < p.D) {
            const int64_t at = p.cu ? (x.first + t) * p.qs[1] : x.r * p.qs[0] + t * p.qs[1];
            v = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + at + h * p.qs[2] + 8 * ch);
            v.x ^= flip; v.y ^= flip; v.z ^= flip; v.w ^= flip;
          }
          *reinterpret_cast<uint4*>(sq + (ch >> 3) * 16384 + sw128_offset(r, (ch & 7) * 16)) = v;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_Q + slot]);
      }
      const bool live = quarter * 32 < d.rows;
      const int t = (d.row0 + min(row, d.rows - 1)) / p.G;
      const uint64_t bits = p.tree && x.x.ok ? (uint64_t)p.tree[x.first + t] : 0ull;
      float m = -INFINITY, l = 0.f;
      for (int k = 0; ok && k < d.n; ++k, ++n) {
        const int j = d.first + k * d.step, key0 = j * kKeys;
        const uint32_t tile = tile0 + (uint32_t)(j - x.j0);
        ok = sy.wait(&bars[B_META + tile % kMeta], (tile / kMeta) & 1);
        const uint32_t absent = s_absent[tile % kMeta];
        ok = ok && sy.wait(&bars[B_S + slot], n & 1);
        if (!ok) break;
        tc_fence_after();
        if (live) {
          uint32_t s[kKeys];
#pragma unroll
          for (int q = 0; q < kKeys; q += 32) GDP_TMEM_LD32(ts + q, (s + q));
          tmem_wait_ld();
          float ce = c;
          if (key0 + kKeys > x.x.ctx || absent) {  // some of the keys are not seen by some row
            ce = 1.f;
#pragma unroll
            for (int q = 0; q < kKeys; q += 32) {
              const int k0 = key0 + q;
              uint32_t see;
              if (p.tree) {
                const int back = k0 - x.x.ctx;
                see = low_bits(-back);
                if (back > -32 && back < 64) see |= (uint32_t)(back >= 0 ? bits >> back : bits << -back);
              } else {
                see = low_bits(x.x.ctx + t + 1 - k0);
              }
              see &= low_bits(x.keys - k0);
              if (absent)
                for (int b = 0; b < 32; b += 8)
                  if (absent >> ((q + b) / a.g) & 1) see &= ~(0xffu << b);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                s[q + e] = __float_as_uint(see >> e & 1 ? __uint_as_float(s[q + e]) * c : -INFINITY);
            }
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kKeys; ++e) top[e & 3] = fmaxf(top[e & 3], __uint_as_float(s[e]));
          const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          const float mt = most == -INFINITY ? -INFINITY : most * ce;
          const bool grow = mt > m + kGrow;  // (from -inf: as soon as anything is seen)
          if (__any_sync(0xffffffffu, grow)) {
            const float mn = grow ? mt : m, f = grow ? ex2(m - mn) : 1.f;
            m = mn;
            l *= f;
            if (k > 0) {  // the last product into O is done, then O is scaled
              ok = sy.wait(&bars[B_O + slot], (n - 1) & 1);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < KD; q += 16) {
                uint32_t o[16];
                GDP_TMEM_LD16(to + q, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                GDP_TMEM_ST8(to + q, o);
                GDP_TMEM_ST8(to + q + 8, (o + 8));
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < kKeys; q += 64) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float p0 = ex2(fmaf(__uint_as_float(s[q + 2 * e]), ce, -base));
              const float p1 = ex2(fmaf(__uint_as_float(s[q + 2 * e + 1]), ce, -base));
              sum[2 * (e & 1)] += p0;
              sum[2 * (e & 1) + 1] += p1;
              w[e] = pack<T>(p0, p1);
            }
            GDP_TMEM_ST32(ts + q / 2, w);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        if (key0 + kKeys > x.keys && x.keys > 0) {  // rows of V behind the last key, in the last box
          const int z0 = x.keys - key0, z1 = (z0 + a.g - 1) / a.g * a.g;
          if (z0 > 0 && z1 > z0) {
            const uint32_t i = 2 * tile + 1;
            ok = sy.wait(&bars[B_FULL + i % L::NB], (i / L::NB) & 1);
            if (!ok) break;
            uint8_t* sv = sm + L::RING + (i % L::NB) * L::TILE;
            for (int e = tid & 127; e < (z1 - z0) * (KD / 8); e += 128) {
              const int r = z0 + e / (KD / 8), ch = e % (KD / 8);
              *reinterpret_cast<uint4*>(sv + (ch >> 3) * 16384 + sw128_offset(r, (ch & 7) * 16)) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async_smem();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_P + slot]);
      }
      tile0 += x.j1 - x.j0;
      if (!ok) break;
      if (d.n > 0) {
        ok = sy.wait(&bars[B_O + slot], (n - 1) & 1);
        if (!ok) break;
        tc_fence_after();
      }
      // Two slots on the same rows: the second leaves its results in the first ones' shared memory
      // (no product reads Q any more), column by column so that lanes are side by side.
      const bool join = !d.two && x.j1 - x.j0 > 1;
      auto meet = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_JOIN]);
        const bool met = sy.wait(&bars[B_JOIN], joins & 1);
        ++joins;
        return met;
      };
      float f0 = 1.f, f1 = 0.f;
      if (join) {
        ok = meet();
        if (!ok) break;
        if (slot == 1 && live) {
#pragma unroll 1
          for (int q = 0; q < KD; q += 16) {
            uint32_t o[16];
            GDP_TMEM_LD16(to + q, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) so[(q + e) * 128 + row] = __uint_as_float(o[e]);
          }
          s_ml[row] = make_float2(m, l);
        }
        ok = meet();
        if (!ok) break;
        if (slot == 0 && live) {
          const float2 u = s_ml[row];
          const float mn = fmaxf(m, u.x), base = mn == -INFINITY ? 0.f : mn;
          f0 = ex2(m - base);
          f1 = ex2(u.x - base);
          m = mn;
          l = f0 * l + f1 * u.y;
        }
      }
      if ((d.two || slot == 0) && live) {
        const bool on = row < d.rows;
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        const int at = d.row0 - x.row0 + row;  // of the item's rows
        float* part = x.slot >= 0 && on ? a.part + (((int64_t)blockIdx.x * 2 + x.slot) * a.cap + at) * a.dvp : nullptr;
        T* dst = on ? static_cast<T*>(p.o) + out_at(p, x.first, x.head, d.row0 + row) : nullptr;
        if (part) a.ml[((int64_t)blockIdx.x * 2 + x.slot) * a.cap + at] = make_float2(m, l);
        const float f = part ? f0 : f0 * inv, g = part ? f1 : f1 * inv;
#pragma unroll 1
        for (int q = 0; q < KD; q += 16) {
          uint32_t o[16];
          GDP_TMEM_LD16(to + q, o);
          tmem_wait_ld();
          if (!on) continue;
          float y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            y[e] = __uint_as_float(o[e]) * f;
            if (join) y[e] = fmaf(g, so[(q + e) * 128 + row], y[e]);
          }
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            if (q + e >= p.DV) break;
            if (part) {
              *reinterpret_cast<float4*>(part + q + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
              *reinterpret_cast<float4*>(part + q + e + 4) = make_float4(y[e + 4], y[e + 5], y[e + 6], y[e + 7]);
            } else {
              *reinterpret_cast<uint4*>(dst + q + e) =
                  make_uint4(pack<T>(y[e], y[e + 1]), pack<T>(y[e + 2], y[e + 3]), pack<T>(y[e + 4], y[e + 5]),
                             pack<T>(y[e + 6], y[e + 7]));
            }
          }
        }
      }
      tc_fence_before();
      if (join) {
        ok = meet();
        if (!ok) break;
      }
      if (x.slot == 1) {
        rec = true;
        if (tid == 0) write_rec(a, s_start, &x, walk.at - (x.j1 - x.j0));
      }
    }
    if (!rec && tid == 0) write_rec(a, s_start, nullptr, 0);
  } else if (warp == kLoad) {
    // ---------------------------------------------------------------- loads
    const int subs = kKeys / a.g;  // boxes of a tile and half: 1 to 16, so a lane's is the same in every round
    const int sub = lane % subs;
    uint32_t i = 0, tile = 0;
    while (ok && walk.next(p, x)) {
      auto page_of = [&](int j, int& place) {  // n_pages: a box of zeros
        const int key = j * kKeys + sub * a.g;
        place = 0;
        if (j >= x.j1 || key >= x.keys) return p.n_pages;
        const int b = key / p.block, page = p.tables[(int64_t)x.r * p.width + b];
        place = key - b * p.block;
        if (page >= p.n_pages && p.status) *p.status = GDP_ERR_INVALID_ARG;
        return page >= 0 && page < p.n_pages ? page : p.n_pages;
      };
      int place, page = page_of(x.j0, place);
      for (int j = x.j0; ok && j < x.j1; ++j, ++tile) {
        int place1;
        const int page1 = page_of(j + 1, place1);
        const uint32_t absent = __ballot_sync(0xffffffffu, page == p.n_pages) & low_bits(subs);
#pragma unroll
        for (int v = 0; v < 2; ++v, ++i) {
          uint64_t* bar = &bars[B_FULL + i % L::NB];
          ok = sy.wait(&bars[B_EMPTY + i % L::NB], ((i / L::NB) & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) {
            if (v == 0) {
              s_absent[tile % kMeta] = absent;
              mbar_arrive(&bars[B_META + tile % kMeta]);
            }
            mbar_expect_tx(bar, L::TILE);
          }
          __syncwarp();
          uint8_t* dst = sm + L::RING + (i % L::NB) * L::TILE + sub * a.g * 128;
          for (int b = lane; b < subs * (KD / 64); b += 32) {
            const int half = b / subs;
            tma_load_4d(dst + half * 16384, v ? &map_v : &map_k, half * 64, x.head, place, page, bar);
          }
        }
        page = page1;
        place = place1;
      }
    }
    if (*s_dead)  // copies in flight land before the CTA leaves
      for (uint32_t b = i > L::NB ? i - L::NB : 0; b < i; ++b)
        for (int tries = 0; tries < 1000 && !mbar_test_for(&bars[B_FULL + b % L::NB], (b / L::NB) & 1, 20000); ++tries) {}
  } else {
    // ---------------------------------------------------------------- products
    constexpr uint32_t id_s = idesc<T>(128, kKeys, false), id_o = idesc<T>(128, KD, true);
    const uint32_t base = smem_u32(sm);
    uint32_t i0 = 0, np[2] = {0, 0}, nq[2] = {0, 0};  // ring at the piece's start; weights and queries taken
    while (ok && walk.next(p, x)) {
      const int nt = x.j1 - x.j0;
      const bool two = x.rows > 128;
      for (int s = 0; ok && s < 2; ++s)
        if (two || s < nt) ok = sy.wait(&bars[B_Q + s], nq[s]++ & 1);
      auto scores = [&](int s, int k) {  // of the piece's tile k in slot s
        const uint32_t i = i0 + 2 * k;
        ok = ok && sy.wait(&bars[B_FULL + i % L::NB], (i / L::NB) & 1);
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          mma_run<KD / 16, false, 16384, 32, 16384, 32>(
              tmem + T_S + 128 * s, sdesc_sw128(base + L::Q + s * L::TILE, 16, 1024),
              sdesc_sw128(base + L::RING + (i % L::NB) * L::TILE, 16, 1024), id_s);
          mma_commit(&bars[B_S + s]);
          if (!two || s == 1) mma_commit(&bars[B_EMPTY + i % L::NB]);
        }
        __syncwarp();
      };
      auto outputs = [&](int s, int k) {
        const uint32_t i = i0 + 2 * k + 1;
        ok = ok && sy.wait(&bars[B_P + s], np[s] & 1);
        ok = ok && sy.wait(&bars[B_FULL + i % L::NB], (i / L::NB) & 1);
        if (!ok) return;
        ++np[s];
        tc_fence_after();
        if (elect_one()) {
          const uint64_t vd = sdesc_sw128(base + L::RING + (i % L::NB) * L::TILE, 16384, 1024);
          const bool add = two ? k > 0 : k > 1;
#pragma unroll
          for (int e = 0; e < kKeys / 16; ++e)
            mma_bf16_ts(tmem + T_O + 128 * s, tmem + T_S + 128 * s + 8 * e, vd + e * (2048 >> 4), id_o, add || e > 0);
          mma_commit(&bars[B_O + s]);
          if (!two || s == 1) mma_commit(&bars[B_EMPTY + i % L::NB]);
        }
        __syncwarp();
      };
      if (two) {
        scores(0, 0);
        scores(1, 0);
        for (int k = 0; ok && k < nt; ++k)
          for (int s = 0; ok && s < 2; ++s) {
            outputs(s, k);
            if (k + 1 < nt) scores(s, k + 1);
          }
      } else {
        scores(0, 0);
        if (nt > 1) scores(1, 1);
        for (int k = 0; ok && k < nt; ++k) {
          outputs(k & 1, k);
          if (k + 2 < nt) scores(k & 1, k + 2);
        }
      }
      i0 += 2 * nt;
    }
    if (*s_dead) {  // products in flight end before their operands and columns go away
      if (elect_one()) mma_commit(&bars[B_END]);
      for (int tries = 0; tries < 1000 && !mbar_test_for(&bars[B_END], 0, 20000); ++tries) {}
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
  set_layout(a, layout(sm_count(), (int64_t)p.T * p.G, kRows, p.DV), ws, sm_count(), 1);
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
