// Attention of new tokens over a paged cache: entry points, the kernel for any type and size, and
// the kernel that joins cut items.
//
// o = sum_j p_j v_j / sum_j p_j with p_j = e^(scale q k_j - m) over the keys j that a row sees, in one
// pass with a running maximum m and sum (in base 2, the factor log2 e in the scale).
#include <algorithm>
#include <cmath>

#include "attention.cuh"

namespace gdp {
namespace attn {
namespace {

// ------------------------------------------------------------------ any type and size
// fp32, and 16-bit heads that are not steps of 8 or not on a grid of 16 bytes. A CTA of eight warps takes up to 8 rows
// of an item against tiles of 32 keys, which arrive in their own type by cp.async of the widest size that the rows
// allow (16, 8 or 4 bytes; odd 16-bit rows by elements), up to three tiles ahead. Products are fp32 multiply-adds: for
// the scores a thread has two keys and every 16th chunk of the head (a chunk of Q is read for both), for the outputs
// four columns (eight above 128) and every eighth key, whose sums meet at the item's end. Bound by the latency of its
// steps between three barriers a tile (half of the issue slots used): 64 requests of up to 4000 keys, 16 heads over 4,
// 128 columns, fp32: 122 us, where HBM needs 65; 32 drafted tokens on up to 4000 keys, 8 requests, 64 columns: 309 us;
// pieces of prompts, 8 of up to 256 tokens on up to 1024, 128 columns: 747 us; 16 requests of up to 9000 keys, 100
// columns, bf16, 8 bytes a copy: 115 us, HBM 20 (by elements 738; 54 bytes a thread spill in 16 bits). Not kept: one
// key a thread (129 and 327 us), four (126 and 376); keys and maxima of its own for each warp with no barrier in a
// tile (185 us: its sums of a score over lanes and its rescaling are every warp's); three CTAs of 80 registers an SM
// (with one key a thread 123 us, but small calls 22 for 20 and trees 334).
constexpr int kRows = 8, kKeys = 32, kThreads = 256, kWarps = kThreads / 32;
constexpr int kScores = kKeys + 1;  // stride of a row of scores: eight rows in other banks
constexpr Cost kCost = {8, 3, 8, 3};

// Of any sizes: two stages of fp32 and 256 columns are the most, smaller ones have more stages within 105 KB.
constexpr int kMostSmem = 144 * 1024;

struct SimpleSmem {
  int ks, vs;                 // bytes of a row of K and of V
  int stage, stages;
  int q, s, p, off, bytes;    // offsets past the stages
};
inline SimpleSmem simple_smem(int D, int DV, int esz) {
  SimpleSmem x;
  x.ks = (D * esz + 15) / 16 * 16;
  x.vs = (DV * esz + 15) / 16 * 16;
  x.stage = kKeys * (x.ks + x.vs);
  x.stages = std::max(2, std::min(4, 105 * 1024 / x.stage));  // (two CTAs an SM)
  x.q = std::max(x.stages * x.stage, kWarps * kRows * 512 * (DV > 128 ? 2 : 1));  // (the warps' outputs meet there)
  x.s = x.q + 4 * kRows * (x.ks / esz);                            // Q, fp32
  x.p = x.s + 4 * kRows * kScores;                                 // scores [row][key], weights [key][row]
  x.off = x.p + 4 * kRows * kKeys + 4 * kRows * 2;                 // factors and sums of the rows
  x.bytes = x.off + 2 * kKeys * 16 + 16 + 4 * 4;                   // offsets of two tiles' rows; seen keys by stage
  return x;
}

template <typename T> struct alignas(16) Chunk { T e[16 / sizeof(T)]; };
template <typename T> struct alignas(4 * sizeof(T)) Quad { T e[4]; };

struct SimpleArgs : Args {
  SimpleSmem L;
  int k_wide, v_wide;         // bytes of a copy: 16, 8 or 4, as the rows and their grid allow; 0: by elements
  int by_k, by_v;             // logarithm of the threads of a row
};

// N bytes; of what is not there, zeros.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool there) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? N : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(there ? N : 0)
                 : "memory");
}

// The tiles [j0, j1) of one piece for R rows (x.rows of them in use), outputs of NQ quads a thread.
template <typename T, int R, int NQ>
__device__ __forceinline__ void simple_piece(const SimpleArgs& a, uint8_t* sm, const Piece& x) {
  constexpr int VN = 16 / sizeof(T);
  const Problem& p = a.p;
  const SimpleSmem& L = a.L;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, NST = L.stages;
  float* sq = reinterpret_cast<float*>(sm + L.q);
  float* ss = reinterpret_cast<float*>(sm + L.s);                  // [kRows][kScores]
  float* sp = reinterpret_cast<float*>(sm + L.p);                  // [kKeys][kRows]
  float* s_alpha = sp + kRows * kKeys;
  float* s_sum = s_alpha + kRows;
  longlong2* s_off = reinterpret_cast<longlong2*>(sm + L.off);     // [2][kKeys]
  uint32_t* s_ok = reinterpret_cast<uint32_t*>(s_off + 2 * kKeys); // [stages]
  const int qs = L.ks / (int)sizeof(T);
  const T *k0 = static_cast<const T*>(p.k) + x.head * p.ks[2], *v0 = static_cast<const T*>(p.v) + x.head * p.vs[2];

  // where the rows of tile j lie (by the last warp; -1: not there), from page numbers that were asked for a tile before
  int page = -1;
  auto ask = [&](int j) {
    const int key = j * kKeys + lane;
    if (warp == kWarps - 1) page = j < x.j1 && key < x.keys ? p.tables[(int64_t)x.r * p.width + quot(key, p.by_block)] : -1;
  };
  auto find = [&](int j) {
    if (warp != kWarps - 1) return;
    const int key = j * kKeys + lane, in = key - (int)quot(key, p.by_block) * p.block;
    if (page >= p.n_pages) report(p.status, GDP_ERR_INVALID_ARG);
    const bool there = (uint32_t)page < (uint32_t)p.n_pages;
    s_off[(j & 1) * kKeys + lane] =
        there ? make_longlong2(page * p.ks[0] + in * p.ks[1], page * p.vs[0] + in * p.vs[1]) : make_longlong2(-1, -1);
    const uint32_t ok = __ballot_sync(0xffffffffu, there);
    if (lane == 0) s_ok[j % NST] = ok;
    ask(j + 1);
  };
  // tile j into its stage; rows that are not there are 0
  auto load = [&](int j) {
    if (j < x.j1) {
      uint8_t* st = sm + (j % NST) * L.stage;
      const longlong2* off = s_off + (j & 1) * kKeys;
      auto rows = [&](uint8_t* dst, int stride, const T* src, int D, int wide, int by, bool k) {
        auto copy = [&](auto n) {
          constexpr int N = decltype(n)::value, E = N / (int)sizeof(T);
          const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
          const int c0 = tid & ((1 << by) - 1);
#pragma unroll 4
          for (int key = tid >> by; key < kKeys; key += kThreads >> by) {
            const int64_t o = k ? off[key].x : off[key].y;
            for (int c = c0; c < stride / N; c += 1 << by) {
              const bool there = o >= 0 && c * E < D;
              cp_async<N>(to + key * stride + N * c, src + (there ? o + c * E : 0), there);
            }
          }
        };
        if (wide == 16) copy(std::integral_constant<int, 16>());
        else if (wide == 8) copy(std::integral_constant<int, 8>());
        else if (wide == 4) copy(std::integral_constant<int, 4>());
        else
          for (int key = warp; key < kKeys; key += kWarps) {
            const int64_t o = k ? off[key].x : off[key].y;
            for (int d = lane; d < stride / (int)sizeof(T); d += 32)
              reinterpret_cast<T*>(dst + key * stride)[d] = o >= 0 && d < D ? src[o + d] : from_f<T>(0.f);
          }
      };
      rows(st, L.ks, k0, p.D, a.k_wide, a.by_k, true);
      rows(st + kKeys * L.ks, L.vs, v0, p.DV, a.v_wide, a.by_v, false);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");           // (one for each tile, empty ones too)
  };

  ask(x.j0);
  __syncthreads();  // (the last piece's reads are over)
  for (int i = tid; i < R * qs; i += kThreads) {
    const int row = i / qs, d = i - row * qs;
    float f = 0.f;
    if (row < x.rows && d < p.D) {
      const int at = x.row0 + row, t = (int)quot(at, p.by_G), h = x.head * p.G + at - t * p.G;
      const int64_t base = p.cu ? (x.first + t) * p.qs[1] : x.r * p.qs[0] + t * p.qs[1];
      f = to_f(static_cast<const T*>(p.q)[base + h * p.qs[2] + d]);
    }
    sq[i] = f;
  }
  for (int i = 0; i + 1 < NST; ++i) {
    find(x.j0 + i);
    __syncthreads();
    load(x.j0 + i);
  }
  find(x.j0 + NST - 1);
  float4 acc[R][NQ];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int n = 0; n < NQ; ++n) acc[i][n] = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;                                    // of row `warp`

  for (int j = x.j0; j < x.j1; ++j) {
    if (NST == 2) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (NST == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
    __syncthreads();                                               // tile j is there, tile j - 1 has been read
    load(j + NST - 1);
    const uint8_t* st = sm + (j % NST) * L.stage;
    {  // scores of two keys: chunks part, + 16, ..
      constexpr int NK = 2, PARTS = 8 * NK;
      float s[NK * R];                                             // [key][row]
#pragma unroll
      for (int i = 0; i < NK * R; ++i) s[i] = 0.f;
      const int part = lane % PARTS, key0 = tid / PARTS;           // keys key0, + kThreads / PARTS
      const uint8_t* kp = st + key0 * L.ks;
      for (int c = part; c * VN < p.D; c += PARTS) {
        Chunk<T> kk[NK];
#pragma unroll
        for (int k = 0; k < NK; ++k) kk[k] = reinterpret_cast<const Chunk<T>*>(kp + k * (kThreads / PARTS) * L.ks)[c];
#pragma unroll
        for (int e = 0; e < VN; e += 4)
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const float4 q = *reinterpret_cast<const float4*>(sq + i * qs + c * VN + e);
#pragma unroll
            for (int k = 0; k < NK; ++k)
              s[k * R + i] = fmaf(q.x, to_f(kk[k].e[e]), fmaf(q.y, to_f(kk[k].e[e + 1]),
                             fmaf(q.z, to_f(kk[k].e[e + 2]), fmaf(q.w, to_f(kk[k].e[e + 3]), s[k * R + i]))));
          }
      }
      // the parts' sums: each exchange halves the scores that a lane goes on with, to number part % (NK R)
#pragma unroll
      for (int h = NK * R / 2; h > 0; h >>= 1)
#pragma unroll
        for (int i = 0; i < h; ++i) {
          const bool up = part & h;
          const float give = up ? s[i] : s[i + h], keep = up ? s[i + h] : s[i];
          s[i] = keep + __shfl_xor_sync(0xffffffffu, give, h);
        }
      if (R == 4) s[0] += __shfl_xor_sync(0xffffffffu, s[0], PARTS / 2);
      const int i = part % R, key = key0 + kThreads / PARTS * (part / R);
      if (part < NK * R) {
        const int back = j * kKeys + key - x.x.ctx;
        bool sees = (s_ok[j % NST] >> key & 1) && i < x.rows;
        if (sees && back >= 0) {
          const int t = (int)quot(x.row0 + i, p.by_G);
          sees = p.tree ? (p.tree[x.first + t] >> back) & 1 : back <= t;
        }
        ss[i * kScores + key] = sees ? s[0] * p.c : -INFINITY;
      }
    }
    __syncthreads();
    find(j + NST);                                                 // (its offsets' place was tile j + NST - 2's)
    if (warp < R) {                                                // running maximum and sum of row `warp`
      const float s = ss[warp * kScores + lane];
      float top = s;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
      const float w = ex2(s - base), f = ex2(m - base);
      sp[lane * kRows + warp] = w;
      l = l * f + w;                                               // (each lane its own keys' sum)
      m = mn;
      if (lane == 0) s_alpha[warp] = f;
    }
    __syncthreads();
    // outputs: columns 4 lane .. + 3 (+ 128), keys warp, + 8, ..
    float f[R];
#pragma unroll
    for (int i = 0; i < R; ++i) f[i] = s_alpha[i];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        acc[i][n].x *= f[i]; acc[i][n].y *= f[i]; acc[i][n].z *= f[i]; acc[i][n].w *= f[i];
      }
    const uint8_t* sv = st + kKeys * L.ks;
#pragma unroll 2
    for (int key = warp; key < kKeys; key += kWarps) {
      float w[R];
#pragma unroll
      for (int i = 0; i < R; i += 4) {
        const float4 u = *reinterpret_cast<const float4*>(sp + key * kRows + i);
        w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n)
        if (4 * lane + 128 * n < p.DV) {
          const Quad<T> u = *reinterpret_cast<const Quad<T>*>(sv + key * L.vs + (4 * lane + 128 * n) * sizeof(T));
          const float4 v = make_float4(to_f(u.e[0]), to_f(u.e[1]), to_f(u.e[2]), to_f(u.e[3]));
#pragma unroll
          for (int i = 0; i < R; ++i) {
            acc[i][n].x = fmaf(w[i], v.x, acc[i][n].x);
            acc[i][n].y = fmaf(w[i], v.y, acc[i][n].y);
            acc[i][n].z = fmaf(w[i], v.z, acc[i][n].z);
            acc[i][n].w = fmaf(w[i], v.w, acc[i][n].w);
          }
        }
    }
  }

  // the warps' sums meet, in their order; outputs of a whole item, or a piece's share of them
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float4* so = reinterpret_cast<float4*>(sm);                      // [warp][R][NQ][32]
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int n = 0; n < NQ; ++n) so[((warp * R + i) * NQ + n) * 32 + lane] = acc[i][n];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (warp < R && lane == 0) {
    s_sum[warp] = l;
    if (x.slot >= 0 && warp < x.rows) a.ml[((int64_t)blockIdx.x * 2 + x.slot) * a.cap + warp] = make_float2(m, l);
  }
  __syncthreads();
  for (int e = tid; e < x.rows * NQ * 32; e += kThreads) {
    const int c = e % 32, n = e / 32 % NQ, row = e / (32 * NQ), col = 4 * c + 128 * n;
    if (col >= p.DV) continue;
    float4 y = so[(row * NQ + n) * 32 + c];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 u = so[((w * R + row) * NQ + n) * 32 + c];
      y.x += u.x; y.y += u.y; y.z += u.z; y.w += u.w;
    }
    if (x.slot >= 0) {
      float4* dst = reinterpret_cast<float4*>(a.part) + ((int64_t)blockIdx.x * 2 + x.slot) * a.cap * (a.dvp / 4);
      dst[(int64_t)(col / 4) * a.cap + row] = y;
    } else {
      const float sum = s_sum[row], g = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      T* dst = static_cast<T*>(p.o) + out_at(p, x.first, x.head, x.row0 + row) + col;
      const float u[4] = {y.x, y.y, y.z, y.w};
      for (int k = 0; k < 4; ++k)
        if (col + k < p.DV) dst[k] = from_f<T>(u[k] * g);
    }
  }
}

template <typename T, int NQ>
__global__ void __launch_bounds__(kThreads, NQ == 1 ? 2 : 1) simple_kernel(const __grid_constant__ SimpleArgs a) {
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ Start s_start;
  __shared__ long long s_scan[kThreads / 32 + 1];
  pdl_wait();
  pdl_trigger();
  find_start<kRows, kKeys, kThreads>(a, &s_start, s_scan);
  Walk<kRows, kKeys> walk(s_start, a.cost);
  Piece x;
  bool rec = false;
  while (walk.next(a.p, x)) {
    if (x.rows <= 4)
      simple_piece<T, 4, NQ>(a, sm, x);
    else
      simple_piece<T, 8, NQ>(a, sm, x);
    if (x.slot == 1) {
      rec = true;
      if (threadIdx.x == 0) write_rec(a, s_start, &x);
    }
  }
  if (!rec && threadIdx.x == 0) write_rec(a, s_start, nullptr);
}

// ------------------------------------------------------------------ joining cut items
// A CTA per record and RB rows, a thread per row, two quads of columns and every groups-th piece: batches of
// four pieces, their loads in flight together, are added under a running maximum, in the order of the pieces;
// then the groups' results in the order of the groups. Rows lie side by side, so a warp reads whole lines.
constexpr int kJoin = 256, kBatch = 4;

struct Joined {
  float m, l;
  float4 acc[2];
  __device__ __forceinline__ void add(float xm, float xl, const float4& x0, const float4& x1) {
    const float mn = fmaxf(m, xm), base = mn == -INFINITY ? 0.f : mn;
    const float f0 = ex2(m - base), f1 = ex2(xm - base);
    m = mn;
    l = f0 * l + f1 * xl;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float4& x = n ? x1 : x0;
      acc[n].x = fmaf(f1, x.x, f0 * acc[n].x);
      acc[n].y = fmaf(f1, x.y, f0 * acc[n].y);
      acc[n].z = fmaf(f1, x.z, f0 * acc[n].z);
      acc[n].w = fmaf(f1, x.w, f0 * acc[n].w);
    }
  }
};

template <typename T, int RB>
__global__ void __launch_bounds__(kJoin) join_kernel(const __grid_constant__ Args a) {
  constexpr int kSlots = kJoin / RB;
  __shared__ Joined s_part[kJoin];
  pdl_wait();
  const Rec r = a.recs[blockIdx.x];
  const int tid = threadIdx.x, row = blockIdx.y * RB + tid % RB;
  if ((int)blockIdx.y * RB >= r.rows) return;
  const Problem& p = a.p;
  const int pieces = r.more + 1, quads = a.dvp / 4;
  int span = 1;  // slots of a group, for two quads each: a power of two
  while (2 * span < quads && span < kSlots) span *= 2;
  const int slot = tid / RB, group = slot / span, groups = kSlots / span;
  const bool even = p.DV % 4 == 0 && reinterpret_cast<uintptr_t>(p.o) % sizeof(Quad<T>) == 0;
  // piece i: slot 1 of this CTA, slot 0 of the next ones
  auto at = [&](int i) { return ((int64_t)(blockIdx.x + i) * 2 + (i == 0)) * a.cap; };
  for (int q0 = 0; q0 < quads; q0 += 2 * span) {
    const int q = q0 + slot % span;
    const bool on = row < r.rows && q < quads, both = q + span < quads;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    Joined x = {-INFINITY, 0.f, {zero, zero}};
    if (on)
      for (int i0 = group; i0 < pieces; i0 += kBatch * groups) {
        float2 ml[kBatch];
        float4 v[kBatch][2];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int i = i0 + k * groups;
          if (i < pieces) {
            const float4* src = reinterpret_cast<const float4*>(a.part) + at(i) * quads + (int64_t)q * a.cap + row;
            ml[k] = a.ml[at(i) + row];
            v[k][0] = src[0];
            v[k][1] = both ? src[(int64_t)span * a.cap] : zero;
          }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (i0 + k * groups < pieces) x.add(ml[k].x, ml[k].y, v[k][0], v[k][1]);
      }
    if (groups > 1) {
      __syncthreads();
      s_part[tid] = x;
      __syncthreads();
      if (group == 0)
        for (int g = 1; g < groups; ++g) {
          const Joined& y = s_part[tid + g * span * RB];
          x.add(y.m, y.l, y.acc[0], y.acc[1]);
        }
    }
    if (on && group == 0) {
      const float f = x.l > 0.f || x.l != x.l ? 1.f / x.l : 0.f;
      T* dst = static_cast<T*>(p.o) + out_at(p, r.first, r.head, r.row0 + row);
      for (int n = 0; n < 1 + both; ++n) {
        const float4 u = n ? x.acc[1] : x.acc[0];
        const int col = 4 * (q + n * span);
        const Quad<T> y = {from_f<T>(u.x * f), from_f<T>(u.y * f), from_f<T>(u.z * f), from_f<T>(u.w * f)};
        if (even)
          *reinterpret_cast<Quad<T>*>(dst + col) = y;
        else
          for (int k = 0; k < 4; ++k)
            if (col + k < p.DV) dst[col + k] = y.e[k];
      }
    }
  }
}

template <typename T>
cudaError_t join(const Args& a) {
  // (few rows a CTA where an item may be cut often; more where that would be thousands of CTAs)
  if (a.cap <= 64) return launch_pdl(join_kernel<T, 8>, dim3(a.ctas, (a.cap + 7) / 8), dim3(kJoin), 0, a.p.stream, a);
  return launch_pdl(join_kernel<T, 16>, dim3(a.ctas, (a.cap + 15) / 16), dim3(kJoin), 0, a.p.stream, a);
}

template <typename T, int NQ>
cudaError_t go(const SimpleArgs& a) {
  const cudaError_t e = allow_smem<simple_kernel<T, NQ>>(kMostSmem);
  return e != cudaSuccess ? e
                          : launch_pdl(simple_kernel<T, NQ>, dim3(a.ctas), dim3(kThreads), a.L.bytes, a.p.stream, a);
}
template <typename T>
cudaError_t go(const SimpleArgs& a) {
  return a.p.DV > 128 ? go<T, 2>(a) : go<T, 1>(a);
}

constexpr int kResident = 2;  // CTAs of an SM at most

// The widest asynchronous copy that the rows of a cache are whole multiples of, on its grid; 0: none.
int widest(const Problem& p, const void* base, const int64_t* s, int D, int esz) {
  const int n[3] = {p.n_pages, p.block, p.HKV};
  for (int w = 16; w >= 4; w /= 2) {
    bool all = reinterpret_cast<uintptr_t>(base) % w == 0 && D * esz % w == 0;
    for (int i = 0; i < 3; ++i) all = all && (n[i] <= 1 || s[i] * esz % w == 0);
    if (all) return w;
  }
  return 0;
}

}  // namespace

size_t simple_workspace(int64_t rows, int DV) { return layout(kResident * sm_count(), rows, kRows, DV).total; }

cudaError_t launch_combine(const Args& a) {
  switch (a.p.dt) {
    case GDP_BF16: return join<__nv_bfloat16>(a);
    case GDP_F16: return join<__half>(a);
    default: return join<float>(a);
  }
}

void set_layout(Args& a, const Layout& x, uint8_t* ws, int ctas) {
  a.recs = reinterpret_cast<Rec*>(ws + x.recs);
  a.ml = reinterpret_cast<float2*>(ws + x.ml);
  a.part = reinterpret_cast<float*>(ws + x.part);
  a.ctas = ctas;
  a.cap = x.cap;
  a.dvp = x.dvp;
}

cudaError_t launch_simple(const Problem& p, uint8_t* ws) {
  SimpleArgs a{};
  a.p = p;
  const int esz = p.dt == GDP_F32 ? 4 : 2;
  a.L = simple_smem(p.D, p.DV, esz);
  // as many CTAs as are resident (a kilobyte of each one's shared memory is the system's)
  const int ctas = sm_count() * std::max(1, std::min(kResident, (228 * 1024) / (a.L.bytes + 1280)));
  set_layout(a, layout(ctas, (int64_t)p.T * p.G, kRows, p.DV), ws, ctas);
  a.cost = kCost;
  a.k_wide = widest(p, p.k, p.ks, p.D, esz);
  a.v_wide = widest(p, p.v, p.vs, p.DV, esz);
  auto threads_of = [](int copies) {
    int l = 0;
    while (l < 5 && 1 << l < copies) ++l;
    return l;
  };
  a.by_k = threads_of(a.L.ks / std::max(4, a.k_wide));
  a.by_v = threads_of(a.L.vs / std::max(4, a.v_wide));
  cudaError_t e;
  switch (p.dt) {
    case GDP_BF16: e = go<__nv_bfloat16>(a); break;
    case GDP_F16: e = go<__half>(a); break;
    default: e = go<float>(a);
  }
  return e != cudaSuccess ? e : launch_combine(a);
}

}  // namespace attn
}  // namespace gdp

using namespace gdp;

namespace {

constexpr int kMostHead = 256;

bool sizes_ok(int N_seq, int B, int T, int H, int HKV, int D, int DV) {
  return N_seq >= 0 && B >= 0 && T >= 0 && H > 0 && HKV > 0 && H % HKV == 0 && D > 0 && DV > 0;
}
// Sizes that the kernels take: rows of a request and rows of tokens are counted in 32 bits.
bool sizes_built(int B, int T, int H, int HKV, int D, int DV, gdp_dtype dt) {
  return (dt == GDP_BF16 || dt == GDP_F16 || dt == GDP_F32) && D <= kMostHead && DV <= kMostHead &&
         (int64_t)B * T <= INT32_MAX && (int64_t)T * (H / HKV) <= INT32_MAX - 1024;
}
// (the same for every stride, so the larger of the two kernels' where both may run)
size_t workspace_of(int T, int H, int HKV, int D, int DV, gdp_dtype dt) {
  const int64_t rows = (int64_t)T * (H / HKV);
  const size_t s = attn::simple_workspace(rows, DV);
  return attn::tc_shape(D, DV, dt) ? std::max(s, attn::tc_workspace(rows, D, DV)) : s;
}

}  // namespace

extern "C" {

size_t gdp_attention_paged_workspace_size(int B, int T, int N_seq, int H, int HKV, int D, int DV, gdp_dtype dt) {
  if (!sizes_ok(N_seq, B, T, H, HKV, D, DV) || !sizes_built(B, T, H, HKV, D, DV, dt)) return 0;
  return workspace_of(T, H, HKV, D, DV, dt);
}

gdp_status gdp_attention_paged(const void* q, const int64_t* q_strides, const void* k_cache,
                               const int64_t* k_cache_strides, const void* v_cache, const int64_t* v_cache_strides,
                               int n_pages, int block_size, const int32_t* block_tables, int max_blocks,
                               const int32_t* context_lens, const int32_t* cu_seqlens, int N_seq,
                               const int64_t* tree_mask, int B, int T, int H, int HKV, int D, int DV, float scale,
                               gdp_dtype dt, void* o, int32_t* status, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  if (!sizes_ok(N_seq, B, T, H, HKV, D, DV) || n_pages < 0 || block_size <= 0 || max_blocks < 0)
    return GDP_ERR_INVALID_ARG;
  if (!sizes_built(B, T, H, HKV, D, DV, dt)) return GDP_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks * block_size > INT32_MAX - 65536) return GDP_ERR_UNSUPPORTED;
  const float c = scale * 1.44269504088896341f;  // scores in powers of two
  if (!std::isfinite(c) || (cu_seqlens ? B != 1 : N_seq != B)) return GDP_ERR_INVALID_ARG;
  if ((int64_t)B * T == 0 || N_seq == 0) return GDP_OK;
  if (!q || !o || !q_strides || !k_cache_strides || !v_cache_strides || !context_lens) return GDP_ERR_INVALID_ARG;
  if ((max_blocks > 0 && !block_tables) || (n_pages > 0 && (!k_cache || !v_cache))) return GDP_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (q_strides[i] < 0 || k_cache_strides[i] < 0 || v_cache_strides[i] < 0) return GDP_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % kAlign != 0 ||
      workspace_bytes < workspace_of(T, H, HKV, D, DV, dt))
    return GDP_ERR_WORKSPACE;
  attn::Problem p{};
  p.q = q; p.k = k_cache; p.v = v_cache;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = q_strides[i];
    p.ks[i] = k_cache_strides[i];
    p.vs[i] = v_cache_strides[i];
  }
  p.n_pages = n_pages; p.block = block_size; p.tables = block_tables; p.width = max_blocks; p.ctx = context_lens;
  p.cu = cu_seqlens; p.n = N_seq; p.B = B; p.T = T; p.H = H; p.HKV = HKV; p.G = H / HKV; p.D = D; p.DV = DV;
  p.by_G = div_by(p.G); p.by_block = div_by(block_size);
  p.tree = tree_mask; p.c = c; p.dt = dt; p.o = o; p.status = status; p.stream = stream;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const cudaError_t e = attn::tc_ok(p) ? attn::launch_tc(p, ws) : attn::launch_simple(p, ws);
  return e == cudaSuccess ? GDP_OK : GDP_ERR_CUDA;
}

}  // extern "C"
