// Group norm with an activation, channels last: x [N, L, C], G groups of C / G
// neighbouring channels, statistics over (L, C / G) of each sample and group,
//     z = (x - mean) / sqrt(var + eps) * weight + bias,
//     y = act(z),  or with a gate  y = z * act(gate).
// L = 1 is the norm of a token's heads (the output norm and gate of a linear
// attention layer).
//
// The bound is HBM: x (and the gate) read once, y written once. norm_rows keeps what it has
// read in registers and norm_map in shared memory, where it fits, while they form the
// mean and then the squared distances from it: the variance is the two-pass one, in
// fp32. norm_elements, norm_map without room and the slices of norm_map read x again, from a
// cache where it still is there. Sums run in a fixed order.
#include <algorithm>
#include <type_traits>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gdp_internal.cuh"

namespace cg = cooperative_groups;

namespace gdp {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }

// n neighbouring elements as one or two vector accesses (p aligned to min(16, n sizeof(T))).
template <typename T, int n>
struct alignas(n * sizeof(T) < 16 ? n * sizeof(T) : 16) Pack {
  T e[n];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// a / (1 + e^-a): 2^x by the hardware (2^-22; the exponent's rounding adds |a| 2^-24 where e^-a
// counts at all, |a| below ~20) and an approximate division (2 ulp; 0 for a denominator above
// 2^126, where the quotient is below 1e-36).
__device__ __forceinline__ float silu(float a) { return __fdividef(a, 1.f + ex2(-1.44269504f * a)); }

// Means are products by __fmul_rn: contracted into the differences from them, they would not be the
// rounded ones whose rest is taken out below.
struct NormArgs {
  const void *x, *gate;
  int64_t x_sn, x_sl, g_sn, g_sl;
  const float *w, *b;
  void* y;
  int64_t N, L;
  int C, G, Cg;
  float eps;
  int silu;
  int GS, sets;   // groups per CTA, CTAs along the groups
  int rows;       // positions per CTA
  int resident;   // the CTA's elements stay in shared memory
  int slices;     // runs of positions per set of groups, where they meet through memory
  float pow2, nn, inv_nn, var_of;  // rows: power of two below 1 / Cg, Cg times it, 1 / nn, 1 / (Cg nn^2)
  float4* part;   // [sample, set][slice][GS]: a slice's mean, what its rounding left, squared distances, elements
};

template <bool GATE>
__device__ __forceinline__ float finish(const NormArgs& a, float z, float gt) {
  const float u = GATE ? gt : z;
  const float act = a.silu ? silu(u) : u;
  return GATE ? z * act : act;
}

// ---------------------------------------------------------------- one position per sample
// TG lanes hold one (sample, group): NV 16-byte vectors each; U samples per lane group are in
// flight at once, far apart in N so that they share their channels' weights. 8192 x 4096 bf16
// with a gate, 32 groups: 37.8 us, 201 MB at 5.3 TB/s, 78 % of a plain copy; issue slots are 73 %
// used (scalar weight loads and an exact exponential made it issue-bound, 77 us).
template <typename TX, typename TO, int TG, int NV, int U, bool GATE>
__global__ void __launch_bounds__(256) norm_rows_kernel(const __grid_constant__ NormArgs a, int64_t Nu) {
  pdl_wait();
  constexpr int VEC = 16 / sizeof(TX);
  using PX = Pack<TX, VEC>;
  using PO = Pack<TO, VEC>;
  const int sub = threadIdx.x % TG;
  const int64_t item = (int64_t)blockIdx.x * (256 / TG) + threadIdx.x / TG;  // of the first Nu samples
  const int64_t n0 = item / a.G;
  const int c = (int)(item - n0 * a.G) * a.Cg, nvec = a.Cg / VEC;
  PX x[U][NV];
  PO gt[GATE ? U : 1][GATE ? NV : 1];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t n = n0 + u * Nu;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int vi = sub + j * TG;
      if (n0 < Nu && n < a.N && vi < nvec) {
        x[u][j] = *reinterpret_cast<const PX*>(static_cast<const TX*>(a.x) + n * a.x_sn + c + vi * VEC);
        if (GATE)
          gt[u][j] = *reinterpret_cast<const PO*>(static_cast<const TO*>(a.gate) + n * a.g_sn + c + vi * VEC);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) put(&x[u][j].e[e], 0.f);
      }
    }
  }
  float w[NV][VEC], bi[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int vi = sub + j * TG, cc = c + vi * VEC;
    const bool on = n0 < Nu && vi < nvec;
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {  // (C is a multiple of VEC; the host checks the 16-byte bases)
      const float4 w4 = on && a.w ? __ldg(reinterpret_cast<const float4*>(a.w + cc + e)) : make_float4(1.f, 1.f, 1.f, 1.f);
      const float4 b4 = on && a.b ? __ldg(reinterpret_cast<const float4*>(a.b + cc + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
      w[j][e] = w4.x; w[j][e + 1] = w4.y; w[j][e + 2] = w4.z; w[j][e + 3] = w4.w;
      bi[j][e] = b4.x; bi[j][e + 1] = b4.y; bi[j][e + 2] = b4.z; bi[j][e + 3] = b4.w;
    }
  }
  // Distances from the mean without its rounding, which a group of equal or close values would show:
  // z = (n x - sum x) / (n std), with n scaled by a power of two (a.nn, below 1) so that nothing
  // overflows that did not, is one exact multiply-add where the sum is exact. It is for 16-bit values
  // of one size (n is at most 1024 here); 32-bit ones are taken from one of the group's, which makes
  // the differences of close values exact: the middle one of three, since an outlier k stds away would
  // cost the others k 2^-24 of a std.
  constexpr bool kPivot = sizeof(TX) == 4;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t n = n0 + u * Nu;
    float f[NV][VEC], s = 0.f;
    float x0 = 0.f;
    if (kPivot) {
      const float p0 = __shfl_sync(0xffffffffu, to_f(x[u][0].e[0]), 0, TG);
      const float p1 = __shfl_sync(0xffffffffu, to_f(x[u][0].e[VEC - 1]), 0, TG);
      const float p2 = __shfl_sync(0xffffffffu, to_f(x[u][0].e[1]), min(TG, nvec) - 1, TG);
      x0 = fmaxf(fminf(p0, p1), fminf(fmaxf(p0, p1), p2));
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        f[j][e] = to_f(x[u][j].e[e]);
        if (kPivot) f[j][e] = sub + j * TG < nvec ? f[j][e] - x0 : 0.f;
        s += f[j][e];
      }
#pragma unroll
    for (int o = TG / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float sn = s * a.pow2;
    float m2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (sub + j * TG < nvec)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          f[j][e] = fmaf(a.nn, f[j][e], -sn);
          m2 = fmaf(f[j][e], f[j][e], m2);
        }
#pragma unroll
    for (int o = TG / 2; o > 0; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
    const float rstd = rsqrtf(fmaf(m2, a.var_of, a.eps)) * a.inv_nn;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int vi = sub + j * TG;
      if (n0 >= Nu || n >= a.N || vi >= nvec) continue;
      PO out;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        put(&out.e[e], finish<GATE>(a, fmaf(f[j][e], rstd * w[j][e], bi[j][e]),
                                    GATE ? to_f(gt[GATE ? u : 0][GATE ? j : 0].e[e]) : 0.f));
      *reinterpret_cast<PO*>(static_cast<TO*>(a.y) + n * a.C + c + vi * VEC) = out;
    }
  }
}

// The same for groups or rows that are not whole vectors: TG lanes read one (sample, group) element
// by element, three times (the second and third reads come from the first-level cache). A CTA per
// sample, as below, made 138485 x 6 fp16 in 2 groups 760 us; 4.1 us with a lane per group. Groups of 9 to
// 31 leave lanes idle: 200000 x 160 bf16 in groups of 10 takes 758 us, 128 MB that could be read and
// written in 19.
template <typename TX, typename TO, int TG, bool GATE>
__global__ void __launch_bounds__(256) norm_elements_kernel(const __grid_constant__ NormArgs a) {
  pdl_wait();
  const int sub = threadIdx.x % TG;
  const int64_t item = (int64_t)blockIdx.x * (256 / TG) + threadIdx.x / TG;
  const int64_t n = item / a.G;
  const int c0 = (int)(item - n * a.G) * a.Cg;
  const int len = n < a.N ? a.Cg : 0;  // (lanes past the end take part in the shuffles)
  const TX* x = static_cast<const TX*>(a.x) + n * a.x_sn + c0;
  const TO* gate = static_cast<const TO*>(a.gate) + (GATE ? n * a.g_sn + c0 : 0);
  TO* y = static_cast<TO*>(a.y) + n * a.C + c0;
  const float inv = 1.f / (float)a.Cg;
  float t = 0.f;
  for (int i = sub; i < len; i += TG) t += to_f(x[i]);
#pragma unroll
  for (int o = TG / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const float mean = __fmul_rn(t, inv);
  // (the mean's own rounding, which a group of a few close values would show, is taken out again)
  float rest = 0.f;
  t = 0.f;
  for (int i = sub; i < len; i += TG) {
    const float d = to_f(x[i]) - mean;
    rest += d;
    t = fmaf(d, d, t);
  }
#pragma unroll
  for (int o = TG / 2; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
  rest *= inv;
#pragma unroll
  for (int o = TG / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const float rstd = rsqrtf(fmaf(-rest, rest, t * inv) + a.eps);
  for (int i = sub; i < len; i += TG) {
    const float w = a.w ? a.w[c0 + i] : 1.f, b = a.b ? a.b[c0 + i] : 0.f;
    put(y + i, finish<GATE>(a, fmaf((to_f(x[i]) - mean) - rest, rstd * w, b), GATE ? to_f(gate[i]) : 0.f));
  }
}

// ---------------------------------------------------------------- many positions per sample
// A cluster of CTAs takes one sample and a set of GS neighbouring groups (enough that its row
// segments fill whole sectors), each CTA a run of positions; the group sums meet through
// distributed shared memory. A thread keeps one vector column, so that its channels' groups
// are fixed, and walks down the positions. 4 x 4096 x 320 fp16 in 32 groups, 21 MB: 13.2 us;
// what it waits for is latency: two reductions over a cluster and the loads of a few warps.
constexpr int kMapThreads = 256;
constexpr int kMaxGS = 128;
constexpr int kMapSmem = 200 * 1024;  // most that a CTA keeps

//
// The second walk sums the distances from the rounded mean beside their squares: what the mean's
// rounding has left (`rest`) is taken out of the variance and of the elements.
//
// PART: a slice's own mean and squared distances from it go to memory, and a second launch (APPLY)
// merges the slices' in order (Chan's formula) and normalises: as many CTAs per group as it takes.
enum { WHOLE, PART, APPLY };

// (a variance of nearly equal values may come out just below zero)
__device__ __forceinline__ float rstd_of(float var, float eps) { return rsqrtf((var < 0.f ? 0.f : var) + eps); }

template <typename TX, typename TO, int VEC, bool GATE, int STAGE>
__global__ void __launch_bounds__(kMapThreads) norm_map_kernel(const __grid_constant__ NormArgs a) {
  pdl_wait();
  extern __shared__ __align__(16) uint8_t raw[];
  using PX = Pack<TX, VEC>;
  using PO = Pack<TO, VEC>;
  __shared__ float part[2][kMapThreads * (VEC + 1)];  // rows of W + 1 (W is at least a vector)
  __shared__ float total[2][kMaxGS];                  // the cluster's group sums
  __shared__ float gsum[3][kMaxGS];                   // this CTA's: elements, squared distances, distances
  cg::cluster_group cl = cg::this_cluster();
  const int CL = (int)cl.num_blocks(), runs = STAGE == WHOLE ? CL : a.slices;
  const int rank = STAGE == WHOLE ? (int)cl.block_rank() : (int)(blockIdx.x % runs);
  const int64_t unit = blockIdx.x / runs;
  const int64_t n = unit / a.sets;
  const int set = (int)(unit - n * a.sets);
  const int g0 = set * a.GS, gs = min(a.GS, a.G - g0);
  const int c0 = g0 * a.Cg, W = gs * a.Cg, cols = W / VEC;
  const int64_t l0 = (int64_t)rank * a.rows, l1 = min(l0 + a.rows, a.L);
  const int nrow = (int)max((int64_t)0, l1 - l0);
  // thread -> (first vector column, column step, row, row step)
  const int tc = min(cols, kMapThreads), ty = threadIdx.x / tc, tx = threadIdx.x % tc;
  const int nty = kMapThreads / tc;
  const bool on = ty < nty;
  PX* keep = reinterpret_cast<PX*>(raw);
  bool kept = false;  // the elements are in shared memory
  const TX* xb = static_cast<const TX*>(a.x) + n * a.x_sn + l0 * a.x_sl + c0;
  const float inv = 1.f / ((float)(STAGE == PART ? max(nrow, 1) : a.L) * (float)a.Cg);

  float mean_of[VEC];  // per channel of the thread's column (one group: all the same)
  float acc[VEC], dev[VEC];
  // this CTA's sums of acc (and of dev, with two) by group, in a fixed order, then the cluster's: into
  // gsum[which ..] and total
  auto reduce = [&](int which, auto two) {
    constexpr int S = decltype(two)::value;
    if (gs == 1) {
      float t[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        t[0] += on ? acc[e] : 0.f;
        if (S == 2) t[1] += on ? dev[e] : 0.f;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < S; ++i) t[i] += __shfl_xor_sync(0xffffffffu, t[i], o);
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < S; ++i) part[i][threadIdx.x >> 5] = t[i];
      __syncthreads();
      if (threadIdx.x < S) {
        float u = 0.f;
        for (int i = 0; i < kMapThreads / 32; ++i) u += part[threadIdx.x][i];
        gsum[which + threadIdx.x][0] = u;
      }
    } else {  // one pass of columns: a warp per group, lanes over the rows of W channel sums
      if (on)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          part[0][ty * (W + 1) + tx * VEC + e] = acc[e];
          if (S == 2) part[1][ty * (W + 1) + tx * VEC + e] = dev[e];
        }
      __syncthreads();
      const int lane = threadIdx.x & 31;
      for (int g = threadIdx.x >> 5; g < gs; g += kMapThreads / 32) {
        float t[2] = {0.f, 0.f};
        for (int y = lane; y < nty; y += 32)
          for (int i = 0; i < a.Cg; ++i)
#pragma unroll
            for (int j = 0; j < S; ++j) t[j] += part[j][y * (W + 1) + g * a.Cg + i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int j = 0; j < S; ++j) t[j] += __shfl_xor_sync(0xffffffffu, t[j], o);
        if (lane < S) gsum[which + lane][g] = lane == 0 ? t[0] : t[1];
      }
    }
    cl.sync();
    for (int g = threadIdx.x >> 3; g < gs; g += kMapThreads / 8) {  // eight lanes, a rank each
      const int r = threadIdx.x & 7;
      const uint32_t m = 0xffu << (threadIdx.x & 24);
#pragma unroll
      for (int j = 0; j < S; ++j) {
        float t = r < CL ? cl.map_shared_rank(&gsum[which + j][0], r)[g] : 0.f;
        t += __shfl_xor_sync(m, t, 1);
        t += __shfl_xor_sync(m, t, 2);
        t += __shfl_xor_sync(m, t, 4);
        if (r == 0) total[j][g] = t;  // the cluster's sums
      }
    }
    __syncthreads();
  };
  auto group_of = [&](int col, int e) { return gs == 1 ? 0 : (col * VEC + e) / a.Cg; };
  // rows ty, ty + nty, .. of column c: D loads in flight; `use` gets the row's index from ty and its data
  auto walk = [&](int c, auto use) {
    constexpr int D = 4;
    const TX* src = xb + (int64_t)ty * a.x_sl + c * VEC;
    const int64_t step = (int64_t)nty * a.x_sl;
    const PX* kp = keep + ty * cols + c;
    const int kstep = nty * cols;
    for (int r = ty; r < nrow; r += D * nty) {
      PX x[D];
#pragma unroll
      for (int d = 0; d < D; ++d)
        if (r + d * nty < nrow) x[d] = kept ? kp[d * kstep] : *reinterpret_cast<const PX*>(src + d * step);
#pragma unroll
      for (int d = 0; d < D; ++d)
        if (r + d * nty < nrow) use(r + d * nty, x[d]);
      src += D * step;
      kp += D * kstep;
    }
  };

  if constexpr (STAGE != APPLY) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
    if (on)
      for (int c = tx; c < cols; c += tc)
        walk(c, [&](int r, const PX& x) {
          if (a.resident) keep[r * cols + c] = x;
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[e] += to_f(x.e[e]);
        });
    kept = a.resident;
    reduce(0, std::integral_constant<int, 1>());
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      mean_of[e] = __fmul_rn(total[0][group_of(tx, e)], inv);
      acc[e] = dev[e] = 0.f;
    }
    __syncthreads();
    if (on)
      for (int c = tx; c < cols; c += tc)
        walk(c, [&](int, const PX& x) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float d = to_f(x.e[e]) - mean_of[e];
            dev[e] += d;
            acc[e] = fmaf(d, d, acc[e]);
          }
        });
    reduce(1, std::integral_constant<int, 2>());
    if constexpr (STAGE == PART) {
      for (int g = threadIdx.x; g < gs; g += kMapThreads) {
        const float r = gsum[2][g] * inv;
        a.part[(unit * runs + rank) * a.GS + g] = make_float4(__fmul_rn(gsum[0][g], inv), r, fmaf(-r, gsum[2][g], gsum[1][g]),
                                                             (float)nrow * (float)a.Cg);
      }
      return;
    }
  } else {
    for (int g = threadIdx.x >> 5; g < gs; g += kMapThreads / 32) {  // a warp per group, lanes over the slices
      const float4* q = a.part + unit * runs * a.GS + g;
      const int lane = threadIdx.x & 31;
      float t = 0.f, m2 = 0.f, rest = 0.f;
      for (int i = lane; i < runs; i += 32) {
        const float4 x = __ldcg(q + (int64_t)i * a.GS);
        t = fmaf(x.w, x.x, t);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      const float mean = __fmul_rn(t, inv);
      for (int i = lane; i < runs; i += 32) {
        const float4 x = __ldcg(q + (int64_t)i * a.GS);
        const float d = (x.x - mean) + x.y, cd = x.w * d;
        rest += cd;
        m2 += fmaf(cd, d, x.z);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        m2 += __shfl_xor_sync(0xffffffffu, m2, o);
        rest += __shfl_xor_sync(0xffffffffu, rest, o);
      }
      if (lane == 0) {
        gsum[0][g] = mean;
        total[0][g] = m2;
        total[1][g] = rest;
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) mean_of[e] = gsum[0][group_of(tx, e)];
  }
  const TO* gb = static_cast<const TO*>(a.gate);
  if (GATE) gb += n * a.g_sn + l0 * a.g_sl + c0;
  TO* yb = static_cast<TO*>(a.y) + (n * a.L + l0) * a.C + c0;
  if (on)
    for (int c = tx; c < cols; c += tc) {
      float ww[VEC], bb[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int g = group_of(c, e);
        const float rest = total[1][g] * inv, rstd = rstd_of(fmaf(-rest, rest, total[0][g] * inv), a.eps);
        ww[e] = rstd * (a.w ? a.w[c0 + c * VEC + e] : 1.f);
        bb[e] = fmaf(-rest, ww[e], a.b ? a.b[c0 + c * VEC + e] : 0.f);
      }
      walk(c, [&](int r, const PX& x) {
        PO gt, out;
        if (GATE) gt = *reinterpret_cast<const PO*>(gb + (int64_t)r * a.g_sl + c * VEC);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          put(&out.e[e], finish<GATE>(a, fmaf(to_f(x.e[e]) - mean_of[e], ww[e], bb[e]),
                                      GATE ? to_f(gt.e[e]) : 0.f));
        *reinterpret_cast<PO*>(yb + (int64_t)r * a.C + c * VEC) = out;
      });
    }
  if (STAGE == WHOLE) cl.sync();  // no CTA leaves while another may still read its sums
}

template <typename TX, typename TO, int TG, int NV, int U>
cudaError_t go_rows(const NormArgs& a, cudaStream_t s) {
  const int64_t Nu = cdiv(a.N, U), grid = cdiv(Nu * a.G, 256 / TG);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return a.gate ? launch_pdl(norm_rows_kernel<TX, TO, TG, NV, U, true>, dim3((unsigned)grid), dim3(256), 0, s, a, Nu)
                : launch_pdl(norm_rows_kernel<TX, TO, TG, NV, U, false>, dim3((unsigned)grid), dim3(256), 0, s, a, Nu);
}

template <typename TX, typename TO, int TG>
cudaError_t go_elements(const NormArgs& a, cudaStream_t s) {
  const int64_t grid = cdiv(a.N * a.G, 256 / TG);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return a.gate ? launch_pdl(norm_elements_kernel<TX, TO, TG, true>, dim3((unsigned)grid), dim3(256), 0, s, a)
                : launch_pdl(norm_elements_kernel<TX, TO, TG, false>, dim3((unsigned)grid), dim3(256), 0, s, a);
}

template <typename TX, typename TO, int VEC, bool GATE, int STAGE>
cudaError_t go_map2(const NormArgs& a, int CL, size_t smem, cudaStream_t s) {
  auto kern = norm_map_kernel<TX, TO, VEC, GATE, STAGE>;
  if (smem > 24 * 1024) {  // beside up to 21 KB of static shared memory
    const cudaError_t e = allow_smem<norm_map_kernel<TX, TO, VEC, GATE, STAGE>>(kMapSmem);
    if (e != cudaSuccess) return e;
  }
  const int64_t grid = a.N * a.sets * (STAGE == WHOLE ? CL : a.slices);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kMapThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = CL;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// How a norm over positions is laid out: GS groups per set, and either clusters of CL CTAs (slices =
// 0) or slices that meet through memory.
struct MapPlan {
  int GS, sets, CL, slices, rows;
  int64_t seg, part_bytes;
};
MapPlan plan_map(int64_t N, int64_t L, int G, int Cg, int size, int vec, bool split) {
  MapPlan m{};
  auto sets_of = [&](int64_t least) {  // row segments of whole vectors and at least so many bytes
    m.GS = 1;
    while (m.GS < G && m.GS < kMaxGS && ((int64_t)m.GS * Cg * size < least || (m.GS * Cg) % vec != 0)) ++m.GS;
    // a thread's channels must keep their groups, so a set of several groups is one pass of columns
    m.sets = (int)cdiv(G, m.GS);
    m.seg = (int64_t)m.GS * Cg * size;
  };
  // Row segments of 128 bytes; half and a quarter of that where even clusters of 8 would leave SMs
  // idle or a CTA with more than 48 KB (4 x 4096 x 320 in 32 groups, fp16: 13.2 us, against 18.2
  // with 128 bytes), but not beyond (16 x 256 x 1280, 32 groups: 16.2 us with 64 bytes, 12.4 with 128).
  for (const int64_t least : {128, 64, 32}) {
    sets_of(least);
    if (N * m.sets * 8 >= sm_count() && cdiv(L, 8) * m.seg <= 48 * 1024) break;
  }
  // Slices where that still leaves a CTA with much: the same work on more SMs, for a second read of
  // x and a launch. 1 x 16384 x 128 fp16 in one group: 17.7 us / 71.3 in a cluster of 8;
  // 2 x 9000 x 512 fp32 in four: 21.4 / 46.5. Sets of several small groups cost more to reduce, so
  // they stay with clusters longer (1 x 16384 x 128, 32 groups: 43 us in slices, 15.3 in clusters).
  const int64_t much = N * m.sets * 8 >= sm_count() ? 96 : m.GS > 1 ? 64 : 32;
  if (split && cdiv(L, 8) * m.seg > much * 1024) {
    sets_of(128);
    const int64_t units = N * m.sets, most = std::max<int64_t>(1, L * m.seg / 8192);
    const int64_t want = std::max(cdiv(4 * sm_count(), units), cdiv(L * m.seg, 64 * 1024));
    m.rows = (int)cdiv(L, std::min<int64_t>(1024, std::min(want, most)));
    m.slices = (int)cdiv(L, m.rows);
    m.CL = 1;
    m.part_bytes = units * m.slices * m.GS * (int64_t)sizeof(float4);
    return m;
  }
  // CTAs per cluster: until every SM has one, or 8 KB of work are left each (clusters of 16 found
  // few places: 4 x 4096 x 320 took 34 us)
  m.CL = 1;
  while (m.CL < 8 && N * m.sets * m.CL < sm_count() && L * m.seg > (int64_t)m.CL * 8192) m.CL *= 2;
  while (m.CL < 8 && cdiv(L, m.CL) * m.seg > 96 * 1024) m.CL *= 2;
  m.rows = (int)cdiv(L, m.CL);
  return m;
}

template <typename TX, typename TO, int VEC>
cudaError_t go_map(NormArgs a, cudaStream_t s) {
  const MapPlan m = plan_map(a.N, a.L, a.G, a.Cg, sizeof(TX), VEC, a.part != nullptr);
  a.GS = m.GS;
  a.sets = m.sets;
  a.rows = m.rows;
  a.slices = m.slices;
  const int64_t bytes = (int64_t)m.rows * m.seg;
  a.resident = bytes <= kMapSmem;
  const size_t smem = a.resident ? (size_t)bytes : 0;
  if (m.slices > 0) {
    const cudaError_t e = go_map2<TX, TO, VEC, false, PART>(a, 1, smem, s);
    if (e != cudaSuccess) return e;
    return a.gate ? go_map2<TX, TO, VEC, true, APPLY>(a, 1, 0, s) : go_map2<TX, TO, VEC, false, APPLY>(a, 1, 0, s);
  }
  return a.gate ? go_map2<TX, TO, VEC, true, WHOLE>(a, m.CL, smem, s) : go_map2<TX, TO, VEC, false, WHOLE>(a, m.CL, smem, s);
}

bool aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <typename TX, typename TO>
cudaError_t run(NormArgs a, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(TX);
  // vectors: 16 bytes of x, as many elements of the gate and of y
  constexpr int GA = std::min<int>(16, VEC * sizeof(TO));
  const bool rows_ok = a.x_sn % VEC == 0 && a.x_sl % VEC == 0 && aligned(a.x, 16) &&
                       aligned(a.y, GA) && a.C % VEC == 0 &&
                       (!a.gate || (a.g_sn % VEC == 0 && a.g_sl % VEC == 0 && aligned(a.gate, GA)));
  if (a.L == 1 && rows_ok && a.Cg % VEC == 0 && aligned(a.w, 16) && aligned(a.b, 16)) {
    const int nvec = a.Cg / VEC;
    if (nvec <= 1) return go_rows<TX, TO, 1, 1, 2>(a, s);
    if (nvec <= 2) return go_rows<TX, TO, 2, 1, 2>(a, s);
    if (nvec <= 4) return go_rows<TX, TO, 4, 1, 2>(a, s);
    if (nvec <= 8) return go_rows<TX, TO, 8, 1, 2>(a, s);
    if (nvec <= 16) return go_rows<TX, TO, 16, 1, 2>(a, s);
    if (nvec <= 32) return go_rows<TX, TO, 32, 1, 2>(a, s);
    if (nvec <= 64) return go_rows<TX, TO, 32, 2, 1>(a, s);
    if (nvec <= 128) return go_rows<TX, TO, 32, 4, 1>(a, s);
    // fp32 groups of 516 to 1024 channels: one read where a lane's eight vectors are mostly used, or
    // where there are few groups and latency counts; else single elements, whose reads overlap
    // better (us of rows / elements, 4 groups: 400 x 2560 3.3 / 6.6, 32768 x 2560 141.8 / 127.1,
    // 400 x 3584 3.6 / 8.5, 32768 x 3584 163.0 / 189.7)
    if constexpr (VEC == 4)
      if (nvec <= 256 && (nvec > 192 || a.N * a.G <= 16 * sm_count())) return go_rows<TX, TO, 32, 8, 1>(a, s);
  }
  if (a.L == 1 && a.Cg <= 8) return go_elements<TX, TO, 1>(a, s);
  if (a.L == 1 && a.Cg <= 1024) return go_elements<TX, TO, 32>(a, s);
  // several groups share a vector only where the set of groups ends on one
  if (rows_ok && (a.Cg % VEC == 0 || a.Cg * sizeof(TX) < 128)) return go_map<TX, TO, VEC>(a, s);
  return go_map<TX, TO, 1>(a, s);
}

}  // namespace
}  // namespace gdp

using namespace gdp;

namespace {

gdp_status norm(const void* x, int64_t x_sn, int64_t x_sl, const void* gate, int64_t gate_sn, int64_t gate_sl,
                const float* weight, const float* bias, int64_t N, int64_t L, int C, int G, float eps,
                gdp_activation activation, gdp_dtype dt, gdp_dtype dt_out, void* y, float4* part, cudaStream_t stream) {
  if (N < 0 || L < 0 || C <= 0 || G <= 0 || C % G != 0 || !(eps >= 0.f)) return GDP_ERR_INVALID_ARG;
  if (activation != GDP_ACT_NONE && activation != GDP_ACT_SILU) return GDP_ERR_UNSUPPORTED;
  if (N == 0 || L == 0) return GDP_OK;
  if (!x || !y) return GDP_ERR_INVALID_ARG;
  if ((L > 1 && (x_sl < C || (gate && gate_sl < C))) ||
      (N > 1 && (x_sn < C || (gate && gate_sn < C))))
    return GDP_ERR_INVALID_ARG;
  if (L > INT32_MAX) return GDP_ERR_UNSUPPORTED;
  if (L == 1) x_sl = gate_sl = 0;  // the stride of a single position or sample means nothing
  if (N == 1) x_sn = gate_sn = 0;
  float pow2 = 1.f;
  while (pow2 * (float)(C / G) > 1.f) pow2 *= 0.5f;
  const float nn = pow2 * (float)(C / G);
  NormArgs a{x, gate, x_sn, x_sl, gate_sn, gate_sl, weight, bias, y, N, L, C, G, C / G, eps,
             activation == GDP_ACT_SILU, 0, 0, 0, 0, 0, pow2, nn, 1.f / nn, 1.f / ((float)(C / G) * nn * nn), part};
  cudaError_t e;
  if (dt == GDP_BF16 && dt_out == GDP_BF16) e = run<__nv_bfloat16, __nv_bfloat16>(a, stream);
  else if (dt == GDP_F16 && dt_out == GDP_F16) e = run<__half, __half>(a, stream);
  else if (dt == GDP_F32 && dt_out == GDP_F32) e = run<float, float>(a, stream);
  else if (dt == GDP_F32 && dt_out == GDP_BF16) e = run<float, __nv_bfloat16>(a, stream);
  else if (dt == GDP_F32 && dt_out == GDP_F16) e = run<float, __half>(a, stream);
  else return GDP_ERR_UNSUPPORTED;
  return e == cudaSuccess ? GDP_OK : GDP_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t gdp_group_norm_workspace_size(int64_t N, int64_t L, int C, int G, gdp_dtype dt) {
  if (N <= 0 || L <= 1 || L > INT32_MAX || C <= 0 || G <= 0 || C % G != 0) return 0;
  const int size = dt == GDP_F32 ? 4 : 2;
  // the strides, which this does not know, decide between vectors and single elements
  return std::max(plan_map(N, L, G, C / G, size, 16 / size, true).part_bytes,
                  plan_map(N, L, G, C / G, size, 1, true).part_bytes);
}

gdp_status gdp_group_norm(const void* x, int64_t x_sn, int64_t x_sl, const void* gate, int64_t gate_sn,
                          int64_t gate_sl, const float* weight, const float* bias, int64_t N, int64_t L, int C,
                          int G, float eps, gdp_activation activation, gdp_dtype dt, gdp_dtype dt_out, void* y,
                          cudaStream_t stream) {
  return norm(x, x_sn, x_sl, gate, gate_sn, gate_sl, weight, bias, N, L, C, G, eps, activation, dt, dt_out, y, nullptr,
              stream);
}

gdp_status gdp_group_norm_ws(const void* x, int64_t x_sn, int64_t x_sl, const void* gate, int64_t gate_sn,
                             int64_t gate_sl, const float* weight, const float* bias, int64_t N, int64_t L, int C,
                             int G, float eps, gdp_activation activation, gdp_dtype dt, gdp_dtype dt_out, void* y,
                             void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const size_t need = gdp_group_norm_workspace_size(N, L, C, G, dt);
  if (need > 0 && (!workspace || reinterpret_cast<uintptr_t>(workspace) % kAlign != 0 || workspace_bytes < need))
    return GDP_ERR_WORKSPACE;
  return norm(x, x_sn, x_sl, gate, gate_sn, gate_sl, weight, bias, N, L, C, G, eps, activation, dt, dt_out, y,
              need > 0 ? static_cast<float4*>(workspace) : nullptr, stream);
}

}  // extern "C"
