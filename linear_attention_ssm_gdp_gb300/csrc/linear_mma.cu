// Linear attention with a decay for each head, chunked form for every type, size and stride
// that the tensor-memory kernel does not take: fp32 and fp16 inputs, K up to 256, odd sizes.
//
// The same algebra on chunks of 64 tokens (see linear_chunk.cu), one CTA of sixteen warps per
// (segment, value head, slice of value columns), the products with mma.sync in tf32: an
// operand that has more than tf32's 11 bits goes in as two parts (x = hi + lo to 2^-22)
// and a product of two such operands takes three instructions, so that sums are fp32 to a few
// 2^-22 whatever the input type. 16-bit inputs are exact in one part, and their scores q k^T come
// from 16-bit instructions (exact products, fp32 sums). The state stays in registers as the
// accumulator fragments of U, in fp32. What several warps read as an operand (the state for
// the read-out q S, the decayed values v') is split into its parts once, into shared memory.
//
// What bounds it: mma.sync's own rate, 16 cycles of an SM quarter per m16n8k8 in tf32
// (measured: 12,000 cycles a chunk for fp16 K = V = 64, 17,500 for fp32, the same with eight
// warps, with sixteen and with the loops unrolled). Tiles of the next chunk stream in by
// cp.async meanwhile where two fit in shared memory. 16384 tokens, 4 heads, K = V = 64, fp16: 66 us
// with the state pass; 3 x 333 tokens, 6 value heads over 2, K = 48, V = 80, fp32: 31 us.
#include <algorithm>
#include <type_traits>

#include "linear_chunk.cuh"
#include "ptx.cuh"

namespace gdp {
namespace {

using namespace linear;

constexpr int kThreads = 512;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void zero(float* p) { *p = 0.f; }
__device__ __forceinline__ void zero(__nv_bfloat16* p) { *p = __float2bfloat16_rn(0.f); }
__device__ __forceinline__ void zero(__half* p) { *p = __float2half_rn(0.f); }

__device__ __forceinline__ uint32_t tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
// D += A B, one m16n8k8 step.
__device__ __forceinline__ void mma(float* d, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// The same for 16-bit operands, m16n8k16.
template <typename T>
__device__ __forceinline__ void mma16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t saddr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
// An operand fragment of N registers: hi, and lo unless EXACT.
template <int N, bool EXACT>
struct Frag {
  uint32_t hi[N], lo[EXACT ? 1 : N];
  __device__ __forceinline__ void set(int i, float x) {
    if (EXACT) {
      hi[i] = __float_as_uint(x);
    } else {
      hi[i] = tf32(x);
      lo[EXACT ? 0 : i] = tf32(x - __uint_as_float(hi[i]));
    }
  }
};
// N products with the same A, the small terms first; neighbouring instructions have accumulators
// of their own. The instruction cuts its sum off instead of rounding it, which over K = 128 made
// fp32 outputs 1.1e-6 off (2-norm); with STEP each step's sum starts from zero and is added to the
// rest by the fp32 units, rounded: 1.7e-7, for 3 % of the time.
template <bool STEP, bool EA, bool EB, int N>
__device__ __forceinline__ void mma_parts(float (*d)[4], const Frag<4, EA>& a, const Frag<2, EB> (&b)[N]) {
  float z[N][4] = {};
  float(*t)[4] = STEP ? z : d;
  if (!EA)
#pragma unroll
    for (int j = 0; j < N; ++j) mma(t[j], a.lo, b[j].hi);
  if (!EB)
#pragma unroll
    for (int j = 0; j < N; ++j) mma(t[j], a.hi, b[j].lo);
#pragma unroll
  for (int j = 0; j < N; ++j) mma(t[j], a.hi, b[j].hi);
  if (STEP)
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[j][e] += t[j][e];
}

template <typename T, int KD>
struct MmaLay {
  static constexpr int VS = KD <= 128 ? 64 : 32;  // value columns per CTA
  static constexpr int LK = KD + 16 / sizeof(T);  // row lengths in elements: rows spread over the banks
  static constexpr int LV = VS + 8;
  static constexpr int Q = 0, Kt = Q + C * LK * (int)sizeof(T), Vt = Kt + C * LK * (int)sizeof(T);
  static constexpr int TILE = Vt + C * LV * (int)sizeof(T);
  // the state as hi and lo parts where they fit, v' as hi and lo, P, decays
  static constexpr bool SPLIT = KD <= 128;
  static constexpr int SB = KD * LV * 4, VB = C * LV * 4;
  static constexpr int REST = (SPLIT ? 2 : 1) * SB + 2 * VB + C * (C + 4) * 4 + 2 * 272 * 4;
  static constexpr int STAGES = 2 * TILE + REST <= 227 * 1024 ? 2 : 1;
  static constexpr int S = STAGES * TILE, W = S + (SPLIT ? 2 : 1) * SB, P = W + 2 * VB, G = P + C * (C + 4) * 4;
  static constexpr int BYTES = G + 2 * 272 * 4;
  static_assert(BYTES <= 227 * 1024, "shared memory of one CTA");
};

template <typename T, int KD, bool OUT>
__global__ void __launch_bounds__(kThreads) linear_mma_kernel(const __grid_constant__ ChunkArgs a, int vec) {
  pdl_wait();
  using L = MmaLay<T, KD>;
  constexpr bool EX = sizeof(T) == 2;  // inputs are exact in tf32
  constexpr int VS = L::VS, LK = L::LK, LV = L::LV, LP = C + 4;
  extern __shared__ __align__(16) uint8_t sm[];
  const LinearProblem& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tq = lane & 3;
  if (!OUT && no_split(a)) return;
  if (a.clear && blockIdx.x == 0 && tid == 0) *p.status = kDevOk;
  Item x;
  if (!get_item(a, blockIdx.x, x) || skip<OUT>(x)) return;
  float* sS = reinterpret_cast<float*>(sm + L::S);
  float* sP = reinterpret_cast<float*>(sm + L::P);
  uint32_t* sW = reinterpret_cast<uint32_t*>(sm + L::W);  // v' parts: hi, then lo
  constexpr int SL = L::SB / 4, WL = L::VB / 4;
  const int K = p.K, V = p.V;
  const T* gq = static_cast<const T*>(p.q) + x.b * p.qs[0] + x.h * p.qs[2];
  const T* gk = static_cast<const T*>(p.k) + x.b * p.ks[0] + x.h * p.ks[2];
  const T* gv = static_cast<const T*>(p.v) + x.b * p.vs[0] + x.hv * p.vs[2] + x.v0;
  const int nv = min(VS, V - x.v0);

  // tile rows of `cols` elements (the rest of the tile's width and rows outside the sequence zero)
  auto tile = [&](int off, int ld, auto wide, const T* src, int64_t step, int cols, int base) {
    T* dst = reinterpret_cast<T*>(sm + off);
    constexpr int VEC = 16 / sizeof(T), width = decltype(wide)::value;
    if (vec) {
      constexpr int per = width / VEC;
#pragma unroll
      for (int i = tid; i < C * per; i += kThreads) {
        const int r = i / per, c = (i - r * per) * VEC, row = base + r;
        T* d = dst + r * ld + c;
        const bool in = row >= x.r.t0 && row < x.r.t0 + x.r.n && c < cols;
        // a short copy is zero-filled: cols is a multiple of VEC here
        const int bytes = in ? 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(d)),
                     "l"(in ? src + row * step + c : src), "r"(bytes)
                     : "memory");
      }
    } else {
#pragma unroll 1
      for (int i = tid; i < C * width; i += kThreads) {
        const int r = i / width, c = i - r * width, row = base + r;
        if (row >= x.r.t0 && row < x.r.t0 + x.r.n && c < cols) dst[r * ld + c] = src[row * step + c];
        else zero(dst + r * ld + c);
      }
    }
  };
  auto load = [&](int c) {
    const int base = x.r.t0 - x.off + c * C, o = (c % L::STAGES) * L::TILE;
    if (OUT) tile(o + L::Q, LK, std::integral_constant<int, KD>(), gq, p.qs[1], K, base);
    tile(o + L::Kt, LK, std::integral_constant<int, KD>(), gk, p.ks[1], K, base);
    tile(o + L::Vt, LV, std::integral_constant<int, VS>(), gv, p.vs[1], nv, base);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // state fragments: U's accumulators, one 16-row tile of k and NT 8-column tiles of v per warp
  constexpr int MW = KD / 16 < 16 ? KD / 16 : 16;  // warps along k, the rest along v
  constexpr int NT = VS / 8 * MW / 16;
  const int m0 = 16 * (warp % MW), n0 = 8 * NT * (warp / MW);
  float s[NT][4];
  const int64_t at = (int64_t)x.hv * K * V + x.v0;
  auto each_state = [&](auto f) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = m0 + gr + 8 * (e >> 1), v = n0 + 8 * j + 2 * tq + (e & 1);
        f(s[j][e], k, v, k < K && v < nv);
      }
  };
  {
    const float* src = state_src<OUT>(a, x);
    each_state([&](float& y, int k, int v, bool in) { y = src && in ? __ldcg(src + at + (int64_t)k * V + v) : 0.f; });
  }
  float2 wseg = make_float2(1.f, 0.f);
  // the decays of a chunk, a chunk ahead, by a warp that has no scores (its tile is above the diagonal)
  constexpr int kDecay = 12;
  float* sG = reinterpret_cast<float*>(sm + L::G);
  float g0 = 0.f, g1 = 0.f;
  auto fetch_g = [&](int c) {
    g0 = load_g(p, x, x.r.t0 - x.off + c * C, 2 * lane);
    g1 = load_g(p, x, x.r.t0 - x.off + c * C, 2 * lane + 1);
  };
  auto decays = [&](int c) {
    const int base = x.r.t0 - x.off + c * C;
    chunk_decays(g0, g1, p.scale, max(0, x.r.t0 - base), min(C, x.r.t0 + x.r.n - base), lane, sG + (c & 1) * 272);
  };
  if (x.chunks > 0) load(0);
  if (warp == kDecay && x.chunks > 0) {
    fetch_g(0);
    decays(0);
    fetch_g(1);
  }
  for (int c = 0; c < x.chunks; ++c) {
    const int base = x.r.t0 - x.off + c * C;
    const int lo = max(0, x.r.t0 - base), hi = min(C, x.r.t0 + x.r.n - base);
    const float* g = sG + (c & 1) * 272;
    if (L::STAGES == 1 && c > 0) {
      __syncthreads();  // the last chunk's readers are done with the tiles
      load(c);
    }
    if (OUT)  // the state before the chunk, for the read-out
      each_state([&](float& y, int k, int v, bool) {
        if (L::SPLIT) {
          const uint32_t y0 = tf32(y);
          sS[k * LV + v] = __uint_as_float(y0);
          sS[SL + k * LV + v] = __uint_as_float(tf32(y - __uint_as_float(y0)));
        } else {
          sS[k * LV + v] = y;
        }
      });
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    if (L::STAGES == 2 && c + 1 < x.chunks) load(c + 1);  // its stage was last read before this barrier
    const uint8_t* st = sm + (c % L::STAGES) * L::TILE;
    const T* tQ = reinterpret_cast<const T*>(st + L::Q);
    const T* tK = reinterpret_cast<const T*>(st + L::Kt);
    const T* tV = reinterpret_cast<const T*>(st + L::Vt);
    const int kk = (K + 7) / 8;  // steps over K
#pragma unroll
    for (int i = tid; i < C * VS; i += kThreads) {  // v' = e^{Gam - Gam_i} v_i in two parts
      const int t = i / VS, v = i % VS;
      const float y = g[128 + t] * to_f(tV[t * LV + v]);
      const uint32_t y0 = tf32(y);
      sW[t * LV + v] = y0;
      sW[WL + t * LV + v] = tf32(y - __uint_as_float(y0));
    }
    if (warp == kDecay && c + 1 < x.chunks) {
      decays(c + 1);
      fetch_g(c + 2);
    }
    if (OUT) {
      // scores: rows 16 (warp % 4), columns 16 (warp / 4), only tiles that reach the diagonal
      const int r0 = 16 * (warp & 3), c0 = 16 * (warp >> 2);
      float d[2][4] = {};
      if (c0 <= r0 + 15) {
        if constexpr (EX) {
          // lanes 8 m ..: rows 8 (m % 2) .. of the A tile, columns 8 (m / 2); of B rows 8 (m / 2) ..
          const uint32_t qa = ptx::smem_u32(tQ + (r0 + (lane & 15)) * LK + 8 * (lane >> 4));
          const uint32_t kb = ptx::smem_u32(tK + (c0 + (lane & 7) + 8 * (lane >> 4)) * LK + 8 * ((lane >> 3) & 1));
#pragma unroll 1
          for (int k0 = 0; k0 < (K + 15) / 16; ++k0) {
            uint32_t fa[4], fb[4];
            ldmatrix_x4(qa + 32 * k0, fa);
            ldmatrix_x4(kb + 32 * k0, fb);
            mma16<T>(d[0], fa, fb[0], fb[1]);
            mma16<T>(d[1], fa, fb[2], fb[3]);
          }
        } else {
#pragma unroll 1
          for (int k0 = 0; k0 < 8 * kk; k0 += 8) {
            Frag<4, EX> fa;
            const T* qa = tQ + (r0 + gr) * LK + k0 + tq;
            fa.set(0, to_f(qa[0]));
            fa.set(1, to_f(qa[8 * LK]));
            fa.set(2, to_f(qa[4]));
            fa.set(3, to_f(qa[8 * LK + 4]));
            Frag<2, EX> fb[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const T* kb = tK + (c0 + 8 * j + gr) * LK + k0 + tq;
              fb[j].set(0, to_f(kb[0]));
              fb[j].set(1, to_f(kb[4]));
            }
            mma_parts<!EX>(d, fa, fb);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = r0 + gr + 8 * (e >> 1), i = c0 + 8 * j + 2 * tq + (e & 1);
          const float f = ex2_approx((g[t] - g[i]) + (g[64 + t] - g[64 + i]));
          sP[t * LP + i] = i <= t ? d[j][e] * (p.scale * f) : 0.f;
        }
    }
    __syncthreads();
    if (OUT) {
      const int r0 = 16 * (warp & 3);
      // o: rows r0, value columns of this warp's quarter
      constexpr int NO = VS / 32;
      const int v0 = (VS / 4) * (warp >> 2);
      float o[NO][4] = {};
#pragma unroll 1
      for (int k0 = 0; k0 < 8 * kk; k0 += 8) {
        Frag<4, EX> fa;
        const T* qa = tQ + (r0 + gr) * LK + k0 + tq;
        fa.set(0, to_f(qa[0]));
        fa.set(1, to_f(qa[8 * LK]));
        fa.set(2, to_f(qa[4]));
        fa.set(3, to_f(qa[8 * LK + 4]));
        Frag<2, false> fb[NO];
#pragma unroll
        for (int j = 0; j < NO; ++j) {
          const float* sb = sS + (k0 + tq) * LV + v0 + 8 * j + gr;
          if (L::SPLIT) {
            fb[j].hi[0] = __float_as_uint(sb[0]);
            fb[j].hi[1] = __float_as_uint(sb[4 * LV]);
            fb[j].lo[0] = __float_as_uint(sb[SL]);
            fb[j].lo[1] = __float_as_uint(sb[SL + 4 * LV]);
          } else {
            fb[j].set(0, sb[0]);
            fb[j].set(1, sb[4 * LV]);
          }
        }
        mma_parts<!EX>(o, fa, fb);
      }
      const float e0 = g[192 + r0 + gr], e1 = g[192 + r0 + gr + 8];
#pragma unroll
      for (int j = 0; j < NO; ++j) {
        o[j][0] *= e0;
        o[j][1] *= e0;
        o[j][2] *= e1;
        o[j][3] *= e1;
      }
#pragma unroll 1
      for (int i0 = 0; i0 < r0 + 16; i0 += 8) {
        Frag<4, false> fa;
        const float* pa = sP + (r0 + gr) * LP + i0 + tq;
        fa.set(0, pa[0]);
        fa.set(1, pa[8 * LP]);
        fa.set(2, pa[4]);
        fa.set(3, pa[8 * LP + 4]);
        Frag<2, EX> fb[NO];
#pragma unroll
        for (int j = 0; j < NO; ++j) {
          const T* vb = tV + (i0 + tq) * LV + v0 + 8 * j + gr;
          fb[j].set(0, to_f(vb[0]));
          fb[j].set(1, to_f(vb[4 * LV]));
        }
        mma_parts<!EX>(o, fa, fb);
      }
      T* og = static_cast<T*>(p.o) + (((int64_t)x.b * p.T + base) * p.HV + x.hv) * V + x.v0;
#pragma unroll
      for (int j = 0; j < NO; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = r0 + gr + 8 * (e >> 1), v = v0 + 8 * j + 2 * tq + (e & 1);
          if (t >= lo && t < hi && v < nv) put(og + (int64_t)t * p.HV * V + v, o[j][e]);
        }
    }
    // U = k^T (w v), then S = e^Gam S + U
    const float wh = g[256], wl = g[257];
    {
      float u[NT][4] = {};
#pragma unroll 1
      for (int t0 = 0; t0 < C; t0 += 8) {
        Frag<4, EX> fa;
        const T* ka = tK + (t0 + tq) * LK + m0 + gr;
        fa.set(0, to_f(ka[0]));
        fa.set(1, to_f(ka[8]));
        fa.set(2, to_f(ka[4 * LK]));
        fa.set(3, to_f(ka[4 * LK + 8]));
        Frag<2, false> fb[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint32_t* wb = sW + (t0 + tq) * LV + n0 + 8 * j + gr;
          fb[j].hi[0] = wb[0];
          fb[j].hi[1] = wb[4 * LV];
          fb[j].lo[0] = wb[WL];
          fb[j].lo[1] = wb[WL + 4 * LV];
        }
        mma_parts<!EX>(u, fa, fb);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = fmaf(wh, s[j][e], fmaf(wl, s[j][e], u[j][e]));
    }
    if (!OUT) wseg = mul_pair(wseg, make_float2(wh, wl));
    if (float* dst = state_dst<OUT>(a, x, c))
      each_state([&](float& y, int k, int v, bool in) {
        if (in) dst[at + (int64_t)k * V + v] = y;
      });
    __syncthreads();  // S, P and v' are rewritten next
  }
  if (!OUT && tid == 0) a.segW[(int64_t)x.r.id * p.HV + x.hv] = wseg;
  if (OUT && x.chunks == 0 && x.r.last && !p.pool && p.sT)  // an empty sequence keeps its state
    each_state([&](float& y, int k, int v, bool in) {
      if (in) p.sT[x.r.seq * (int64_t)p.HV * K * V + at + (int64_t)k * V + v] = y;
    });
}

template <typename T, int KD, bool OUT>
cudaError_t go(const ChunkArgs& a, int vec) {
  constexpr int smem = MmaLay<T, KD>::BYTES;
  cudaError_t e = allow_smem<linear_mma_kernel<T, KD, OUT>>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(linear_mma_kernel<T, KD, OUT>, dim3((unsigned)a.items), dim3(kThreads), smem, a.p.stream, a, vec);
}
template <typename T, bool OUT>
cudaError_t go_k(const ChunkArgs& a, int vec) {
  return a.p.K <= 64 ? go<T, 64, OUT>(a, vec) : a.p.K <= 128 ? go<T, 128, OUT>(a, vec) : go<T, 256, OUT>(a, vec);
}
template <bool OUT>
cudaError_t go_t(const ChunkArgs& a, int vec) {
  switch (a.p.dt) {
    case GDP_BF16: return go_k<__nv_bfloat16, OUT>(a, vec);
    case GDP_F16: return go_k<__half, OUT>(a, vec);
    default: return go_k<float, OUT>(a, vec);
  }
}

// Measured at K = V = 64: 5.9 us a chunk for 16-bit inputs, 8.7 for fp32; products over K grow with it.
Cost cost_of(int K, gdp_dtype dt) {
  const double k = K / 64.0;
  return dt == GDP_F32 ? Cost{3.0 + 5.5 * k, 1.3 + 2.2 * k, 4.0, 8.0} : Cost{2.5 + 3.2 * k, 1.0 + 1.3 * k, 4.0, 8.0};
}
int slice_of(int K) { return K <= 128 ? 64 : 32; }
Plan plan(int N_seq, int B, int T, int HV, int K, int V, gdp_dtype dt, bool packed) {
  return plan_of(N_seq, B, T, HV, K, V, packed, slice_of(K), cost_of(K, dt), sm_count());
}

}  // namespace

size_t linear_mma_workspace(int N_seq, int B, int T, int HV, int K, int V, gdp_dtype dt) {
  // the query does not say whether the batch is packed
  const size_t d = N_seq == B ? plan(N_seq, B, T, HV, K, V, dt, false).total : 0;
  return std::max(d, B == 1 ? plan(N_seq, B, T, HV, K, V, dt, true).total : 0);
}

cudaError_t launch_linear_mma(const LinearProblem& p, uint8_t* ws) {
  const Plan x = plan(p.N_seq, p.B, p.T, p.HV, p.K, p.V, p.dt, p.cu != nullptr);
  ChunkArgs a{};
  a.p = p;
  a.clear = !p.cu;  // (the segment kernel does it for a packed batch)
  a.nseg = x.nseg;
  a.Lseg = x.Lseg;
  a.slices = x.slices;
  a.vt = slice_of(p.K);
  if (x.bound * p.HV * x.slices > INT32_MAX) return cudaErrorInvalidValue;
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
  // 16-byte copies: rows and bases on 16-byte steps, whole vectors in a row
  const int n = p.dt == GDP_F32 ? 4 : 8;
  const auto fits = [n](const void* b, const int64_t* s) {
    return reinterpret_cast<uintptr_t>(b) % 16 == 0 && s[0] % n == 0 && s[1] % n == 0 && s[2] % n == 0;
  };
  const int vec = p.K % n == 0 && p.V % n == 0 && fits(p.q, p.qs) && fits(p.k, p.ks) && fits(p.v, p.vs);
  if (x.segS) {
    a.segS = reinterpret_cast<float*>(ws + x.segS);
    a.segW = reinterpret_cast<float2*>(ws + x.segW);
    cudaError_t e = go_t<false>(a, vec);
    if (e == cudaSuccess) e = launch_combine(a, seqs);
    if (e != cudaSuccess) return e;
    a.clear = 0;
  }
  return go_t<true>(a, vec);
}

}  // namespace gdp
