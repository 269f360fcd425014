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
constexpr int kRows = 16, kKeys = 64, kThreads = 256;

struct SimpleSmem {
  int sd, sv;  // row strides of q and k, and of v, in floats
  size_t k, v, s, bytes;
};
// sd = 4 mod 8, so that eight keys' vectors fall into different banks
__host__ __device__ inline SimpleSmem simple_smem(int D, int DV) {
  SimpleSmem x;
  x.sd = (D + 7) / 8 * 8 + 4;
  x.sv = (DV + 3) / 4 * 4;
  x.k = sizeof(float) * kRows * x.sd;
  x.v = x.k + sizeof(float) * kKeys * x.sd;
  x.s = x.v + sizeof(float) * kKeys * x.sv;
  x.bytes = x.s + sizeof(float) * kRows * (kKeys + 1) + sizeof(float) * kRows * 2 + sizeof(int64_t) * kKeys * 2;
  return x;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) simple_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ Start s_start;
  __shared__ long long s_scan[kThreads / 32 + 1];
  const Problem& p = a.p;
  const SimpleSmem L = simple_smem(p.D, p.DV);
  float* sq = reinterpret_cast<float*>(sm);
  float* sk = reinterpret_cast<float*>(sm + L.k);
  float* sv = reinterpret_cast<float*>(sm + L.v);
  float* ss = reinterpret_cast<float*>(sm + L.s);        // [kRows][kKeys + 1]
  float* s_alpha = ss + kRows * (kKeys + 1);
  float* s_sum = s_alpha + kRows;
  int64_t* s_ko = reinterpret_cast<int64_t*>(s_sum + kRows);
  int64_t* s_vo = s_ko + kKeys;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  find_start<kRows, kKeys, kThreads>(a, &s_start, s_scan);
  Walk<kRows, kKeys> walk(s_start, a.cost);
  Piece x;
  bool rec = false;
  const int quads = L.sv / 4;
  // outputs: a thread holds the quad of columns tid % 64 of rows tid / 64 + 4 i
  constexpr int RG = kThreads / 64, RN = kRows / RG;
  while (walk.next(p, x)) {
    float4 acc[RN];
#pragma unroll
    for (int i = 0; i < RN; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows 2 warp, 2 warp + 1
    __syncthreads();  // (the last piece's reads of sq are over)
    for (int i = tid; i < kRows * L.sd; i += kThreads) {
      const int row = i / L.sd, d = i - row * L.sd;
      float f = 0.f;
      if (row < x.rows && d < p.D) {
        const int R = x.row0 + row, t = (int)quot(R, p.by_G), h = x.head * p.G + R - t * p.G;
        const int64_t at = p.cu ? (x.first + t) * p.qs[1] : x.r * p.qs[0] + t * p.qs[1];
        f = to_f(static_cast<const T*>(p.q)[at + h * p.qs[2] + d]);
      }
      sq[i] = f;
    }
    for (int j = x.j0; j < x.j1; ++j) {
      __syncthreads();  // (the last tile's reads are over)
      if (tid < kKeys) {
        const int key = j * kKeys + tid;
        int64_t ko = -1, vo = -1;
        if (key < x.keys) {
          const int b = (int)quot(key, p.by_block), page = p.tables[(int64_t)x.r * p.width + b];
          if (page >= p.n_pages && p.status) *p.status = GDP_ERR_INVALID_ARG;
          if (page >= 0 && page < p.n_pages) {
            ko = page * p.ks[0] + (key - b * p.block) * p.ks[1] + x.head * p.ks[2];
            vo = page * p.vs[0] + (key - b * p.block) * p.vs[1] + x.head * p.vs[2];
          }
        }
        s_ko[tid] = ko;
        s_vo[tid] = vo;
      }
      __syncthreads();
      // a warp per key row; what is not there is 0
      for (int key = warp; key < kKeys; key += kThreads / 32) {
        const int64_t ko = s_ko[key], vo = s_vo[key];
        for (int d = lane; d < L.sd; d += 32)
          sk[key * L.sd + d] = ko >= 0 && d < p.D ? to_f(static_cast<const T*>(p.k)[ko + d]) : 0.f;
        for (int d = lane; d < L.sv; d += 32)
          sv[key * L.sv + d] = vo >= 0 && d < p.DV ? to_f(static_cast<const T*>(p.v)[vo + d]) : 0.f;
      }
      __syncthreads();
      {  // scores of key tid % 64, rows 4 (tid / 64) .. + 3
        const int key = tid % kKeys, r0 = tid / kKeys * 4;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const float4* kp = reinterpret_cast<const float4*>(sk + key * L.sd);
        for (int d = 0; d < (p.D + 3) / 4; ++d) {
          const float4 kk = kp[d];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 q = *reinterpret_cast<const float4*>(sq + (r0 + i) * L.sd + 4 * d);
            s[i] = fmaf(q.x, kk.x, fmaf(q.y, kk.y, fmaf(q.z, kk.z, fmaf(q.w, kk.w, s[i]))));
          }
        }
        const int at = j * kKeys + key, back = at - x.x.ctx;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bool sees = s_ko[key] >= 0 && r0 + i < x.rows;
          if (sees && back >= 0) {
            const int t = (int)quot(x.row0 + r0 + i, p.by_G);
            sees = p.tree ? (p.tree[x.first + t] >> back) & 1 : back <= t;
          }
          ss[(r0 + i) * (kKeys + 1) + key] = sees ? s[i] * p.c : -INFINITY;
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // running maximum and sum, two rows a warp
        float* row = ss + (2 * warp + i) * (kKeys + 1);
        const float s0 = row[lane], s1 = row[lane + 32];
        float top = fmaxf(s0, s1);
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float mn = fmaxf(m[i], top), base = mn == -INFINITY ? 0.f : mn;
        const float p0 = ex2(s0 - base), p1 = ex2(s1 - base), alpha = ex2(m[i] - base);
        row[lane] = p0;
        row[lane + 32] = p1;
        float sum = p0 + p1;
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = l[i] * alpha + sum;
        m[i] = mn;
        if (lane == 0) s_alpha[2 * warp + i] = alpha;
      }
      __syncthreads();
      const int c = tid % 64, rg = tid / 64;
      if (c < quads) {
#pragma unroll
        for (int i = 0; i < RN; ++i) {
          const float f = s_alpha[rg + RG * i];
          acc[i].x *= f; acc[i].y *= f; acc[i].z *= f; acc[i].w *= f;
        }
        for (int key = 0; key < kKeys; ++key) {
          const float4 vv = *reinterpret_cast<const float4*>(sv + key * L.sv + 4 * c);
#pragma unroll
          for (int i = 0; i < RN; ++i) {
            const float f = ss[(rg + RG * i) * (kKeys + 1) + key];
            acc[i].x = fmaf(f, vv.x, acc[i].x);
            acc[i].y = fmaf(f, vv.y, acc[i].y);
            acc[i].z = fmaf(f, vv.z, acc[i].z);
            acc[i].w = fmaf(f, vv.w, acc[i].w);
          }
        }
      }
    }
    // outputs of a whole item, or a piece's share of them
    if (lane < 2) s_sum[2 * warp + lane] = lane == 0 ? l[0] : l[1];
    if (x.slot >= 0 && lane < 2 && 2 * warp + lane < x.rows)
      a.ml[((int64_t)blockIdx.x * 2 + x.slot) * a.cap + 2 * warp + lane] =
          lane == 0 ? make_float2(m[0], l[0]) : make_float2(m[1], l[1]);
    __syncthreads();
    const int c = tid % 64, rg = tid / 64;
    if (c < quads)
#pragma unroll
      for (int i = 0; i < RN; ++i) {
        const int row = rg + RG * i;
        if (row >= x.rows) continue;
        if (x.slot >= 0) {
          float4* dst = reinterpret_cast<float4*>(a.part) + ((int64_t)blockIdx.x * 2 + x.slot) * a.cap * quads;
          dst[c * a.cap + row] = acc[i];
          continue;
        }
        const float sum = s_sum[row], f = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        T* dst = static_cast<T*>(p.o) + out_at(p, x.first, x.head, x.row0 + row) + 4 * c;
        const float y[4] = {acc[i].x, acc[i].y, acc[i].z, acc[i].w};
        for (int e = 0; e < 4; ++e)
          if (4 * c + e < p.DV) dst[e] = from_f<T>(y[e] * f);
      }
    if (x.slot == 1) {
      rec = true;
      if (tid == 0) write_rec(a, s_start, &x);
    }
  }
  if (!rec && tid == 0) write_rec(a, s_start, nullptr);
}

// ------------------------------------------------------------------ joining cut items
// A CTA per record and RB rows, a thread per row, quad of columns and every groups-th piece: batches of
// pieces, their loads in flight together, are added under a running maximum, in the order of the pieces;
// then the groups' results in the order of the groups. Rows lie side by side, so a warp reads whole lines.
constexpr int kJoin = 256, kBatch = 8;

template <typename T>
struct alignas(4 * sizeof(T)) Quad {
  T e[4];
};

struct Joined {
  float m, l;
  float4 acc;
  // f0 of this, f1 of x
  __device__ __forceinline__ void add(float xm, float xl, const float4& x) {
    const float mn = fmaxf(m, xm), base = mn == -INFINITY ? 0.f : mn;
    const float f0 = ex2(m - base), f1 = ex2(xm - base);
    m = mn;
    l = f0 * l + f1 * xl;
    acc.x = fmaf(f1, x.x, f0 * acc.x);
    acc.y = fmaf(f1, x.y, f0 * acc.y);
    acc.z = fmaf(f1, x.z, f0 * acc.z);
    acc.w = fmaf(f1, x.w, f0 * acc.w);
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
  int span = 1;  // slots of a group: a power of two
  while (span < quads && span < kSlots) span *= 2;
  const int slot = tid / RB, group = slot / span, groups = kSlots / span;
  const bool even = p.DV % 4 == 0 && reinterpret_cast<uintptr_t>(p.o) % sizeof(Quad<T>) == 0;
  // piece i: slot 1 of this CTA, slot 0 of the next ones
  auto at = [&](int i) { return ((int64_t)(blockIdx.x + i) * 2 + (i == 0)) * a.cap; };
  for (int q0 = 0; q0 < quads; q0 += span) {
    const int q = q0 + slot % span;
    const bool on = row < r.rows && q < quads;
    Joined x = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (on)
      for (int i0 = group; i0 < pieces; i0 += kBatch * groups) {
        float2 ml[kBatch];
        float4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int i = i0 + k * groups;
          if (i < pieces) {
            ml[k] = a.ml[at(i) + row];
            v[k] = reinterpret_cast<const float4*>(a.part)[at(i) * quads + (int64_t)q * a.cap + row];
          }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (i0 + k * groups < pieces) x.add(ml[k].x, ml[k].y, v[k]);
      }
    if (groups > 1) {
      __syncthreads();
      s_part[tid] = x;
      __syncthreads();
      if (group == 0)
        for (int g = 1; g < groups; ++g) {
          const Joined& y = s_part[tid + g * span * RB];
          x.add(y.m, y.l, y.acc);
        }
    }
    if (on && group == 0) {
      const float f = x.l > 0.f || x.l != x.l ? 1.f / x.l : 0.f;
      T* dst = static_cast<T*>(p.o) + out_at(p, r.first, r.head, r.row0 + row) + 4 * q;
      const Quad<T> y = {from_f<T>(x.acc.x * f), from_f<T>(x.acc.y * f), from_f<T>(x.acc.z * f), from_f<T>(x.acc.w * f)};
      if (even)
        *reinterpret_cast<Quad<T>*>(dst) = y;
      else
        for (int k = 0; k < 4; ++k)
          if (4 * q + k < p.DV) dst[k] = y.e[k];
    }
  }
}

template <typename T>
cudaError_t join(const Args& a) {
  // (few rows a CTA where an item may be cut often; more where that would be thousands of CTAs)
  if (a.cap <= 64) return launch_pdl(join_kernel<T, 8>, dim3(a.ctas, (a.cap + 7) / 8), dim3(kJoin), 0, a.p.stream, a);
  return launch_pdl(join_kernel<T, 16>, dim3(a.ctas, (a.cap + 15) / 16), dim3(kJoin), 0, a.p.stream, a);
}

template <typename T>
cudaError_t go(const Args& a) {
  const int smem = (int)simple_smem(a.p.D, a.p.DV).bytes;
  const cudaError_t e = allow_smem<simple_kernel<T>>((int)simple_smem(256, 256).bytes);
  return e != cudaSuccess ? e : launch_pdl(simple_kernel<T>, dim3(a.ctas), dim3(kThreads), smem, a.p.stream, a);
}

int simple_ctas() { return 2 * sm_count(); }

}  // namespace

size_t simple_workspace(int64_t rows, int DV) { return layout(simple_ctas(), rows, kRows, DV).total; }

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
  Args a{};
  a.p = p;
  set_layout(a, layout(simple_ctas(), (int64_t)p.T * p.G, kRows, p.DV), ws, simple_ctas());
  a.cost = {4, 8, 4, 8};
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
  return attn::tc_shape(D, DV, dt) ? std::max(s, attn::tc_workspace(rows, DV)) : s;
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
  if (!std::isfinite(scale) || (cu_seqlens ? B != 1 : N_seq != B)) return GDP_ERR_INVALID_ARG;
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
  p.tree = tree_mask; p.c = scale * 1.44269504088896341f; p.dt = dt; p.o = o; p.status = status; p.stream = stream;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const cudaError_t e = attn::tc_ok(p) ? attn::launch_tc(p, ws) : attn::launch_simple(p, ws);
  return e == cudaSuccess ? GDP_OK : GDP_ERR_CUDA;
}

}  // extern "C"
