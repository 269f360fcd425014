// Linear attention with a decay for each head, recurrent form (single tokens and
// short runs of draft tokens):
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
// with the fp32 state S [K, V] of each (request, value head) read once and
// written once per call; value head hv reads key/query head hv / (HV / H).
//
// The work is the state's read and write (8 bytes per element and call, against
// 5 operations), so the kernel is an HBM stream: a CTA of 256 threads takes one
// (request, value head, slice of up to 64 columns) and holds it in registers,
// four columns (16 bytes) by R rows per thread, all loads in flight at once.
// The sum over K of a read-out is in-thread over R rows, then shuffles across
// the lanes of equal columns, then the eight warps through shared memory in a
// fixed order. Sums and states are fp32; o alone is rounded, to the inputs' type.
// The decay factor is a pair of floats: a decay that stays the same from token to token,
// rounded to 24 bits, would drift from e^{n g} by n roundings in one direction.
//
// Measured at K = V = 128, bf16: 256 requests of 32 heads 178 us, 1.07 GB of states at 6.0 TB/s,
// 89 % of a plain copy; one request of 16 heads 3.2 us in a captured graph, its launch and two
// dependent trips to memory. The state's loads issued before everything else and four CTAs per
// SM instead of two took the batch (paged, each call waited for) from 234 to 199 us.
#include <algorithm>

#include "linear_chunk.cuh"

namespace gdp {
namespace {

constexpr int kThreads = 256;
constexpr int kStep = 16;  // most steps of a call

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }

struct WalkArgs {
  LinearProblem p;
  int VS;      // value columns per CTA
  int slices;  // CTAs along V
};

// Page of block b of request r, or -1 when it has none in the pool.
__device__ __forceinline__ int page_of(const LinearProblem& p, int r, uint32_t b) {
  if (b >= (uint32_t)p.width) return -1;
  const int pg = p.tables[(int64_t)r * p.width + b];
  return pg >= 0 && pg < p.n_pages ? pg : -1;
}

template <typename T, int VEC, int R>
__global__ void __launch_bounds__(kThreads, R <= 8 ? 4 : R <= 16 ? 2 : 1)
    linear_walk_kernel(const __grid_constant__ WalkArgs a) {
  pdl_wait();
  extern __shared__ __align__(16) float sm[];
  const LinearProblem& p = a.p;
  const int K = p.K, V = p.V, VS = a.VS, tid = threadIdx.x, len = p.T;
  float* sq = sm;                    // [len][K]
  float* sk = sq + len * K;          // [len][K]
  float* sv = sk + len * K;          // [len][VS]
  float* sw = sv + len * VS;         // [2][kStep] decay factors, hi and lo
  float* red = sw + 2 * kStep;       // [2][8][VS]
  const int slice = blockIdx.x % a.slices, rest = blockIdx.x / a.slices;
  const int hv = rest % p.HV, seq = rest / p.HV;
  const int v0 = slice * VS, h = hv / (p.HV / p.H);
  const int CG = VS / VEC, RG = kThreads / CG;   // column groups, row groups
  const int cg = tid % CG, rg = tid / CG, c0 = v0 + cg * VEC;
  const bool col_ok = c0 < V;                    // VEC divides V

  // A padded request names no page for its last token; one with a page outside the pool or a
  // negative context is ill-defined and treated the same (and reported).
  const float* src = p.s0 ? p.s0 + ((int64_t)seq * p.HV + hv) * K * V : nullptr;
  uint32_t ctx = 0, b0 = 0, w0 = 0, w1 = 0;  // blocks read and written: [b0, w1], [w0, w1]
  bool live = true, bad = false;
  if (p.pool) {
    const int c = p.ctx[seq];
    ctx = (uint32_t)max(c, 0);
    b0 = (max(ctx, 1u) - 1) / (uint32_t)p.block;
    w0 = ctx / (uint32_t)p.block;
    w1 = (ctx + (uint32_t)len - 1) / (uint32_t)p.block;
    live = c < 0 || w1 >= (uint32_t)p.width || p.tables[(int64_t)seq * p.width + w1] != -1;
    if (live) {
      bad = c < 0;
      for (uint32_t j = b0; j <= w1 && !bad; ++j) bad = page_of(p, seq, j) < 0;
    }
    if (live && !bad && ctx > 0) src = p.pool + ((int64_t)page_of(p, seq, b0) * p.HV + hv) * K * V;
  }
  // the state's loads go out first; everything up to the first step runs behind them
  float s[R][VEC];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = rg + RG * i;
    if (src && live && !bad && col_ok && row < K) {
      if (VEC == 4) {
        const float4 x = __ldcs(reinterpret_cast<const float4*>(src + (int64_t)row * V + c0));
        s[i][0] = x.x; s[i][1 % VEC] = x.y; s[i][2 % VEC] = x.z; s[i][3 % VEC] = x.w;
      } else {
        s[i][0] = src[(int64_t)row * V + c0];
      }
    } else {
#pragma unroll
      for (int c = 0; c < VEC; ++c) s[i][c] = 0.f;
    }
  }
  if (p.pool && live && !bad) {
    // a request that writes a page which another one reads or writes would race with it (every CTA
    // looks at all requests: harmless at 256, 19 us in place of 13 for 8 heads of 64 x 64; 750 in place
    // of 180 at 4096)
    for (int r = tid; r < p.N_seq && !bad; r += kThreads) {
      const int rc = p.ctx[r];
      if (r == seq || rc < 0) continue;
      const uint32_t r1 = ((uint32_t)rc + (uint32_t)len - 1) / (uint32_t)p.block;
      if (page_of(p, r, r1) < 0) continue;
      for (uint32_t i = (max((uint32_t)rc, 1u) - 1) / (uint32_t)p.block; i <= r1; ++i) {
        const int pg = page_of(p, r, i);
        for (uint32_t j = w0; j <= w1; ++j) bad |= pg >= 0 && pg == page_of(p, seq, j);
      }
    }
  }
  const T* q = static_cast<const T*>(p.q) + seq * p.qs[0] + h * p.qs[2];
  const T* k = static_cast<const T*>(p.k) + seq * p.ks[0] + h * p.ks[2];
  const T* v = static_cast<const T*>(p.v) + seq * p.vs[0] + hv * p.vs[2];
  for (int t = 0; t < len; ++t) {
    for (int c = tid; c < K; c += kThreads) {
      sq[t * K + c] = to_f(q[t * p.qs[1] + c]);
      sk[t * K + c] = to_f(k[t * p.ks[1] + c]);
    }
    if (tid < VS) sv[t * VS + tid] = v0 + tid < V ? to_f(v[t * p.vs[1] + v0 + tid]) : 0.f;
  }
  if (tid < len) {
    const float g = !p.g ? 0.f : p.g_token ? p.g[((int64_t)seq * len + tid) * p.HV + hv] : p.g[hv];
    const float2 w = linear::exp_pair(g, 0.f);
    sw[tid] = w.x;
    sw[kStep + tid] = w.y;
  }
  T* o = static_cast<T*>(p.o) + (int64_t)seq * len * p.HV * V + (int64_t)hv * V;
  const int64_t orow = (int64_t)p.HV * V;
  if (__syncthreads_or(bad)) {
    if (tid == 0 && p.status) atomicExch(p.status, 1);
    live = false;
  }
  if (!live) {
    for (int i = tid; i < len * VS; i += kThreads) {
      const int c = v0 + i % VS;
      if (c < V) put(o + (i / VS) * orow + c, 0.f);
    }
    return;
  }
  auto store = [&](float* dst) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int row = rg + RG * i;
      if (col_ok && row < K) {
        if (VEC == 4)
          __stcs(reinterpret_cast<float4*>(dst + (int64_t)row * V + c0),
                 make_float4(s[i][0], s[i][1 % VEC], s[i][2 % VEC], s[i][3 % VEC]));
        else
          dst[(int64_t)row * V + c0] = s[i][0];
      }
    }
  };
  for (int t = 0; t < len; ++t) {
    const float w = sw[t], wl = sw[kStep + t];
    float vv[VEC], acc[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      vv[c] = sv[t * VS + cg * VEC + c];
      acc[c] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int row = rg + RG * i;
      if (row < K) {
        const float kk = sk[t * K + row], qq = sq[t * K + row];
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          s[i][c] = fmaf(w, s[i][c], fmaf(wl, s[i][c], kk * vv[c]));
          acc[c] = fmaf(qq, s[i][c], acc[c]);
        }
      }
    }
    float* keep = nullptr;  // where the state after this step goes
    if (p.pool) {
      const uint32_t end = ctx + (uint32_t)t + 1;
      if (end % (uint32_t)p.block == 0 || t + 1 == len)
        keep = p.pool + ((int64_t)page_of(p, seq, (end - 1) / (uint32_t)p.block) * p.HV + hv) * K * V;
    } else if (t + 1 == len) {
      keep = p.sT + ((int64_t)seq * p.HV + hv) * K * V;
    }
    if (keep) store(keep);
    // lanes of equal columns are CG apart inside a warp
    for (int off = CG; off < 32; off <<= 1)
#pragma unroll
      for (int c = 0; c < VEC; ++c) acc[c] += __shfl_xor_sync(0xffffffffu, acc[c], off);
    float* rb = red + (t & 1) * 8 * VS;
    if ((tid & 31) < CG)
#pragma unroll
      for (int c = 0; c < VEC; ++c) rb[(tid >> 5) * VS + cg * VEC + c] = acc[c];
    __syncthreads();
    if (tid < VS && v0 + tid < V) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x += rb[i * VS + tid];
      put(o + t * orow + v0 + tid, x * p.scale);
    }
  }
}

template <typename T, int VEC, int R>
cudaError_t go(const WalkArgs& a, int smem) {
  const int64_t grid = (int64_t)a.p.N_seq * a.p.HV * a.slices;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(linear_walk_kernel<T, VEC, R>, dim3((unsigned)grid), dim3(kThreads), smem,
                    a.p.stream, a);
}

template <typename T>
cudaError_t pick(const LinearProblem& p) {
  WalkArgs a{p, 0, 0};
  const bool vec = p.V % 4 == 0;  // 16-byte state columns (the API checks the base's alignment)
  // 64 columns: 8 rows of K = 128 per thread, four CTAs per SM; fewer where that leaves SMs idle
  int VS = vec ? 64 : 32;
  while (vec && VS > 32 && (VS / 2 >= p.V ||
         (int64_t)p.N_seq * p.HV * cdiv(p.V, VS) < 2 * sm_count()))
    VS /= 2;
  a.VS = VS;
  a.slices = (int)cdiv(p.V, VS);
  const int RG = kThreads / (vec ? VS / 4 : VS), rows = (int)cdiv(p.K, RG);
  const int smem = (2 * p.T * p.K + p.T * VS + 2 * kStep + 16 * VS) * 4;  // 40 KB for K = 256, 16 steps
  if (!vec) return rows <= 16 ? go<T, 1, 16>(a, smem) : go<T, 1, 32>(a, smem);
  if (rows <= 4) return go<T, 4, 4>(a, smem);
  if (rows <= 8) return go<T, 4, 8>(a, smem);
  return go<T, 4, 16>(a, smem);  // K <= 256: 16 rows at most
}

}  // namespace

cudaError_t launch_linear_walk(const LinearProblem& p) {
  if (p.N_seq == 0) return cudaSuccess;
  switch (p.dt) {
    case GDP_BF16: return pick<__nv_bfloat16>(p);
    case GDP_F16: return pick<__half>(p);
    default: return pick<float>(p);
  }
}

}  // namespace gdp
