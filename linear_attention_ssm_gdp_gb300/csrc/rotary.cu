// Position rotation of heads, and appending keys and values to a paged cache with the rotation on
// the way.
//
// Pair i of a head's R rotated elements turns by pos f_i: (a, b) -> A (a c - b s, a s + b c) with
// c = cos(pos f_i), s = sin(pos f_i) and an amplitude A; the gradient's pass turns by the opposite
// angle. Pairs are (i, i + R / 2) or neighbours (2 i, 2 i + 1).
//
// Angles. A position times a frequency in 32 bits is off by pos 2^-24 of a turn's radians (0.06 at a
// position of 10^6), so angles are counted in turns as 64-bit integers: F_i = frac(f_i / 2 pi) 2^64
// once per CTA from the fp64 frequency, and the phase of a position is the integer product pos F_i
// mod 2^64, exact for every int32 position. Its nearest quarter turn picks the quadrant, the rest (at
// most an eighth of a turn) goes to sincospif as a float.
//
// Bound by HBM: every element is read and written once. A CTA takes a few tokens at a time: its
// threads form the tokens' cosines and sines in shared memory (one thread per token and pair), then
// walk the tokens' vectors of all heads of q, k and v, two 16-byte vectors of a pair (or one vector
// of neighbours) per step. Elements whose sizes, strides or addresses are not whole 16-byte vectors
// go one by one in the same walk.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "fast_div.cuh"
#include "gdp_internal.cuh"

namespace gdp {
namespace {

constexpr int kThreads = 256;
constexpr int kMostDim = 1024;  // of a head

// One tensor [B, T, H, D] of a call: rows of `per_head` steps, the first `pairs` of them rotated.
struct Rows {
  const void* x;
  void* y;
  int64_t xs[3], ys[3];  // batch (cache: page), token, head, in elements
  int H, D, pairs;
  uint32_t per_head, units;  // steps of a head, of a token
  Div by_head;
};

struct RotaryArgs {
  Rows r[3];
  int cached;  // tensors from this one on are written to the cache (3: none)
  const int32_t* pos;
  const double* freq;
  const int64_t* slot;
  int64_t n_slots;
  Div by_block;
  int32_t* status;
  int half, offset;  // R / 2, first rotated element
  float amplitude;
  int backward;
  int64_t tokens;
  int T, group;      // tokens per batch entry, per step of a CTA
  Div by_T, by_units;
  uint32_t units;    // steps of a token over all tensors
};

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

template <typename T, int VN>
struct alignas(sizeof(T) * VN) Vec {
  T e[VN];
};

template <typename T, int VN, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  using V = Vec<T, VN>;
  extern __shared__ unsigned long long sm[];
  unsigned long long* turns = sm;                                    // [half]
  long long* dst = reinterpret_cast<long long*>(sm + a.half);        // [2][group][2]: cache rows of k and v
  float2* cs = reinterpret_cast<float2*>(dst + 4 * a.group);         // [2][group][half]
  const int tid = threadIdx.x;
  pdl_wait();
  for (int i = tid; i < a.half; i += kThreads) {
    double t = a.freq[i] * 0.15915494309189533577;                   // 1 / 2 pi
    t -= floor(t);
    turns[i] = __double2ull_rn(t * 18446744073709551616.0);
  }
  __syncthreads();
  const int64_t groups = (a.tokens + a.group - 1) / a.group;
  int buf = 0;
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x, buf ^= 1) {
    const int64_t t0 = g * a.group;
    const int here = (int)min((int64_t)a.group, a.tokens - t0);
    float2* c = cs + buf * a.group * a.half;
    long long* d = dst + buf * a.group * 2;
    for (int i = tid; i < here * a.half; i += kThreads) {
      const int tok = i / a.half;
      const unsigned long long ph = (unsigned long long)(long long)a.pos[t0 + tok] * turns[i - tok * a.half];
      const unsigned q = (unsigned)((ph + (1ull << 61)) >> 62);      // nearest quarter turn
      float s, k;
      sincospif((float)(long long)(ph - ((unsigned long long)q << 62)) * 0x1p-63f, &s, &k);
      if (q & 1) {
        const float x = s;
        s = k;
        k = -x;
      }
      if (q & 2) { s = -s; k = -k; }
      if (a.backward) s = -s;
      c[i] = make_float2(k * a.amplitude, s * a.amplitude);
    }
    if (a.cached < 3 && tid < here) {
      const int64_t slot = a.slot[t0 + tid];
      const bool in = slot >= 0 && slot < a.n_slots;
      if (!in && slot != -1 && a.status) *a.status = GDP_ERR_INVALID_ARG;
      const int64_t page = in ? slot / a.by_block.d : 0, at = slot - page * a.by_block.d;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        d[2 * tid + j] = in ? page * a.r[1 + j].ys[0] + at * a.r[1 + j].ys[1] : -1;
    }
    __syncthreads();  // (the other buffer is free: every thread has passed the barrier after its use)

    // a step's addresses and data: x1 (and y1) only where it is a pair of two vectors
    struct Step {
      const T *x0, *x1;
      T *y0, *y1;
      const float2* c;
      int first;  // INTER: pair of the vector's first element (may be negative); pairs: >= 0 rotated
      bool on, two, turn;
      V v0, v1;
    };
    const uint32_t all = (uint32_t)here * a.units;
    auto load = [&](uint32_t u, Step& s) {
      s.on = u < all;
      if (!s.on) return;
      const uint32_t tok = quot(u, a.by_units);
      uint32_t w = u - tok * a.units;
      int j = 0;
      if (w >= a.r[0].units) {
        w -= a.r[0].units;
        j = 1;
        if (w >= a.r[1].units) { w -= a.r[1].units; j = 2; }
      }
      const Rows& r = a.r[j];
      const uint32_t h = quot(w, r.by_head);
      const int i = (int)(w - h * r.per_head);
      const uint32_t t = (uint32_t)(t0 + tok), b = quot(t, a.by_T);
      const uint32_t tb = t - b * a.T;
      int e0, e1 = 0;
      s.two = false;
      if (INTER && VN > 1) {
        e0 = i * VN;
        s.first = (e0 - a.offset) >> 1;  // (the offset is even here)
        s.turn = r.pairs > 0 && e0 + VN > a.offset && s.first < a.half;
      } else {
        s.turn = i < r.pairs;
        if (s.turn) {
          s.two = true;
          s.first = i * VN;
          e0 = a.offset + (INTER ? 2 * i : i * VN);
          e1 = e0 + (INTER ? 1 : a.half);
        } else {
          e0 = (i - r.pairs) * VN;
          if (r.pairs > 0 && e0 >= a.offset) e0 += 2 * a.half;
        }
      }
      const T* x = static_cast<const T*>(r.x) + b * r.xs[0] + tb * r.xs[1] + h * r.xs[2];
      int64_t row;
      if (j >= a.cached) {
        row = d[2 * tok + j - 1];
        if (row < 0) { s.on = false; return; }
      } else {
        row = b * r.ys[0] + tb * r.ys[1];
      }
      T* y = static_cast<T*>(r.y) + row + h * r.ys[2];
      s.x0 = x + e0;
      s.y0 = y + e0;
      s.y1 = y + e1;
      s.c = c + tok * a.half;
      s.v0 = *reinterpret_cast<const V*>(s.x0);
      if (s.two) s.v1 = *reinterpret_cast<const V*>(x + e1);
    };
    auto finish = [&](Step& s) {
      if (!s.on) return;
      if (s.two) {
#pragma unroll
        for (int n = 0; n < VN; ++n) {
          const float2 k = s.c[s.first + n];
          const float p = to_f(s.v0.e[n]), q = to_f(s.v1.e[n]);
          s.v0.e[n] = from_f<T>(p * k.x - q * k.y);
          s.v1.e[n] = from_f<T>(p * k.y + q * k.x);
        }
        *reinterpret_cast<V*>(s.y0) = s.v0;
        *reinterpret_cast<V*>(s.y1) = s.v1;
        return;
      }
      if (INTER && VN > 1 && s.turn) {
#pragma unroll
        for (int n = 0; n + 1 < VN; n += 2) {
          const int i = s.first + n / 2;
          if (i >= 0 && i < a.half) {
            const float2 k = s.c[i];
            const float p = to_f(s.v0.e[n]), q = to_f(s.v0.e[n + 1]);
            s.v0.e[n] = from_f<T>(p * k.x - q * k.y);
            s.v0.e[n + 1] = from_f<T>(p * k.y + q * k.x);
          }
        }
      }
      *reinterpret_cast<V*>(s.y0) = s.v0;
    };
    // two steps' loads in flight
    for (uint32_t u = tid; u < all; u += 2 * kThreads) {
      Step s0, s1;
      load(u, s0);
      load(u + kThreads, s1);
      finish(s0);
      finish(s1);
    }
  }
}

template <typename T, int VN>
cudaError_t go(const RotaryArgs& a, bool inter, cudaStream_t stream) {
  const int64_t groups = cdiv(a.tokens, a.group);
  const int grid = (int)std::min<int64_t>(groups, (int64_t)sm_count() * 6);
  const size_t smem = (size_t)a.half * 8 + (size_t)a.group * 32 + (size_t)a.group * a.half * 16;
  return inter ? launch_pdl(rotary_kernel<T, VN, true>, dim3(grid), dim3(kThreads), smem, stream, a)
               : launch_pdl(rotary_kernel<T, VN, false>, dim3(grid), dim3(kThreads), smem, stream, a);
}

bool dtype_ok(gdp_dtype dt) { return dt == GDP_BF16 || dt == GDP_F16 || dt == GDP_F32; }

// Whether a tensor's rows are whole 16-byte vectors.
bool whole(const void* p, const int64_t* s, const int* n, int D, int vn) {
  if (reinterpret_cast<uintptr_t>(p) % 16 || D % vn) return false;
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && s[i] % vn) return false;
  return true;
}

// `dst`: extents of the destination's first two dimensions where they are not B and T.
struct Side {
  const void* x;
  const int64_t* xs;
  void* y;
  const int64_t* ys;
  int H, D, rotated;
  int dst[2];
};

cudaError_t launch(RotaryArgs& a, const Side* sides, int n, int B, int T, int R, bool inter, gdp_dtype dt,
                   cudaStream_t stream) {
  const int esz = dt == GDP_F32 ? 4 : 2, vn = 16 / esz;
  bool vec = true;
  for (int i = 0; i < n; ++i) {
    const Side& s = sides[i];
    if (s.H == 0) continue;
    const int xn[3] = {B, T, s.H}, yn[3] = {s.dst[0], s.dst[1], s.H};
    vec = vec && whole(s.x, s.xs, xn, s.D, vn) && whole(s.y, s.ys, yn, s.D, vn);
    if (s.rotated && R > 0)
      vec = vec && (inter ? a.offset % 2 == 0 : a.offset % vn == 0 && (R / 2) % vn == 0);
  }
  const int w = vec ? vn : 1;
  a.half = R / 2;
  a.units = 0;
  for (int i = 0; i < 3; ++i) {
    Rows& r = a.r[i];
    r = Rows{};
    r.by_head = div_by(1);
    if (i >= n || sides[i].H == 0) continue;
    const Side& s = sides[i];
    r.x = s.x;
    r.y = s.y;
    for (int j = 0; j < 3; ++j) { r.xs[j] = s.xs[j]; r.ys[j] = s.ys[j]; }
    r.H = s.H;
    r.D = s.D;
    const int rot = s.rotated ? R : 0;
    r.pairs = rot / 2 / w;
    if (inter && vec) {
      r.pairs = rot > 0;  // (only whether any pair of the head turns)
      r.per_head = s.D / w;
    } else {
      r.per_head = r.pairs + (s.D - rot) / w;
    }
    r.units = r.per_head * s.H;
    r.by_head = div_by(r.per_head);
    a.units += r.units;
  }
  a.T = T;
  a.by_T = div_by(T);
  a.by_units = div_by(a.units);
  // tokens per step: a cosine and sine per thread, but work for every SM first (and steps that fit 31 bits)
  const int most = std::max(1, std::min(64, kThreads / std::max(1, a.half)));
  a.group = (int)std::max<int64_t>(1, std::min<int64_t>({most, cdiv(a.tokens, (int64_t)sm_count() * 4),
                                                         INT32_MAX / a.units}));
  switch (dt) {
    case GDP_BF16: return vec ? go<__nv_bfloat16, 8>(a, inter, stream) : go<__nv_bfloat16, 1>(a, inter, stream);
    case GDP_F16: return vec ? go<__half, 8>(a, inter, stream) : go<__half, 1>(a, inter, stream);
    default: return vec ? go<float, 4>(a, inter, stream) : go<float, 1>(a, inter, stream);
  }
}

// Shared checks of sizes and of the rotation.
gdp_status check(int B, int T, int D, gdp_dtype dt, const int32_t* pos, const double* freq, int R, int offset,
                 float amplitude) {
  if (!dtype_ok(dt)) return GDP_ERR_UNSUPPORTED;
  if (B < 0 || T < 0 || D <= 0 || R < 0 || R % 2 || offset < 0 || R > D || offset > D - R) return GDP_ERR_INVALID_ARG;
  if (!std::isfinite(amplitude)) return GDP_ERR_INVALID_ARG;
  if (D > kMostDim || (int64_t)B * T > INT32_MAX) return GDP_ERR_UNSUPPORTED;
  if (R > 0 && (int64_t)B * T > 0 && (!pos || !freq)) return GDP_ERR_INVALID_ARG;
  return GDP_OK;
}

bool strides_ok(const int64_t* s, int n) {
  if (!s) return false;
  for (int i = 0; i < n; ++i)
    if (s[i] < 0) return false;
  return true;
}

}  // namespace
}  // namespace gdp

using namespace gdp;

extern "C" {

gdp_status gdp_rotary_frequencies(int rotary_dim, double base, gdp_rotary_scaling scaling, double factor,
                                  double original_length, double low, double high, double* frequencies,
                                  double* amplitude) {
  const int R = rotary_dim;
  if (R < 0 || R % 2 || !(base > 0) || !std::isfinite(base) || (R > 0 && !frequencies)) return GDP_ERR_INVALID_ARG;
  if (scaling < GDP_ROTARY_NONE || scaling > GDP_ROTARY_WAVELENGTH) return GDP_ERR_UNSUPPORTED;
  if (scaling != GDP_ROTARY_NONE && (!(factor > 0) || !std::isfinite(factor))) return GDP_ERR_INVALID_ARG;
  const bool ranged = scaling == GDP_ROTARY_RAMP || scaling == GDP_ROTARY_WAVELENGTH;
  if (ranged && (!(original_length > 0) || !(low > 0) || !(high > low) || !std::isfinite(high) ||
                 !std::isfinite(original_length)))
    return GDP_ERR_INVALID_ARG;
  if (scaling == GDP_ROTARY_RAMP && !(base > 1)) return GDP_ERR_INVALID_ARG;
  const double tau = 6.283185307179586476925;
  double first = 0, last = 0;
  if (scaling == GDP_ROTARY_RAMP) {
    const auto pair_of = [&](double turns) { return R * std::log(original_length / (turns * tau)) / (2 * std::log(base)); };
    first = std::max(std::floor(pair_of(high)), 0.0);
    last = std::min(std::ceil(pair_of(low)), R - 1.0);
  }
  for (int i = 0; i < R / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / R);
    double keep = 1;  // share of the unscaled frequency
    if (scaling == GDP_ROTARY_LINEAR) keep = 0;
    if (scaling == GDP_ROTARY_RAMP) keep = 1 - std::min(std::max((i - first) / std::max(last - first, 1e-3), 0.0), 1.0);
    if (scaling == GDP_ROTARY_WAVELENGTH)
      keep = std::min(std::max((original_length * f / tau - low) / (high - low), 0.0), 1.0);
    frequencies[i] = scaling == GDP_ROTARY_NONE ? f : keep * f + (1 - keep) * (f / factor);
  }
  if (amplitude) *amplitude = scaling == GDP_ROTARY_RAMP && factor > 1 ? 0.1 * std::log(factor) + 1 : 1;
  return GDP_OK;
}

gdp_status gdp_rotary(const void* x, const int64_t* x_strides, const int32_t* positions, const double* frequencies,
                      int rotary_dim, int offset, int interleaved, float amplitude, int backward, int B, int T, int H,
                      int D, gdp_dtype dt, void* y, const int64_t* y_strides, cudaStream_t stream) {
  const gdp_status st = check(B, T, D, dt, positions, frequencies, rotary_dim, offset, amplitude);
  if (st != GDP_OK) return st;
  if (H < 0) return GDP_ERR_INVALID_ARG;
  if ((int64_t)H * D > INT32_MAX / 2) return GDP_ERR_UNSUPPORTED;
  if ((int64_t)B * T * H == 0) return GDP_OK;
  if (!x || !y || !strides_ok(x_strides, 3) || !strides_ok(y_strides, 3)) return GDP_ERR_INVALID_ARG;
  if (y == x)  // in place: every element is written where it was read
    for (int i = 0; i < 3; ++i)
      if ((i == 0 ? B : i == 1 ? T : H) > 1 && x_strides[i] != y_strides[i]) return GDP_ERR_INVALID_ARG;
  RotaryArgs a{};
  a.cached = 3;
  a.pos = positions;
  a.freq = frequencies;
  a.offset = offset;
  a.amplitude = amplitude;
  a.backward = backward != 0;
  a.tokens = (int64_t)B * T;
  a.by_block = div_by(1);
  const Side s{x, x_strides, y, y_strides, H, D, 1, {B, T}};
  return launch(a, &s, 1, B, T, rotary_dim, interleaved != 0, dt, stream) == cudaSuccess ? GDP_OK : GDP_ERR_CUDA;
}

gdp_status gdp_cache_append(const void* q, const void* k, const void* v, const int64_t* strides,
                            const int32_t* positions, const double* frequencies, int rotary_dim, int offset,
                            int interleaved, float amplitude, int B, int T, int H, int HKV, int D, int DV,
                            gdp_dtype dt, const int64_t* slot_map, void* k_cache, const int64_t* k_cache_strides,
                            void* v_cache, const int64_t* v_cache_strides, int n_pages, int block_size, void* q_out,
                            int32_t* status, cudaStream_t stream) {
  const gdp_status st = check(B, T, D, dt, positions, frequencies, rotary_dim, offset, amplitude);
  if (st != GDP_OK) return st;
  if (H < 0 || HKV <= 0 || DV <= 0 || n_pages < 0 || block_size <= 0) return GDP_ERR_INVALID_ARG;
  if (DV > kMostDim || (int64_t)H * D > INT32_MAX / 4 || (int64_t)HKV * D > INT32_MAX / 4 ||
      (int64_t)HKV * DV > INT32_MAX / 4)
    return GDP_ERR_UNSUPPORTED;
  if ((int64_t)B * T == 0) return GDP_OK;
  if (!k || !v || !slot_map || (n_pages > 0 && (!k_cache || !v_cache)) || !strides_ok(strides, 9) || !strides_ok(k_cache_strides, 3) ||
      !strides_ok(v_cache_strides, 3))
    return GDP_ERR_INVALID_ARG;
  const int QH = q ? H : 0;
  const int64_t qo[3] = {(int64_t)T * H * D, (int64_t)H * D, D};
  if (q && H > 0) {
    if (!q_out) return GDP_ERR_INVALID_ARG;
    if (q_out == q)  // in place: every element is written where it was read
      for (int i = 0; i < 3; ++i)
        if ((i == 0 ? B : i == 1 ? T : H) > 1 && strides[i] != qo[i]) return GDP_ERR_INVALID_ARG;
  }
  RotaryArgs a{};
  a.cached = 1;
  a.pos = positions;
  a.freq = frequencies;
  a.slot = slot_map;
  a.n_slots = (int64_t)n_pages * block_size;
  a.by_block = div_by(block_size);
  a.status = status;
  a.offset = offset;
  a.amplitude = amplitude;
  a.tokens = (int64_t)B * T;
  const Side s[3] = {{q, strides, q_out, qo, QH, D, 1, {B, T}},
                     {k, strides + 3, k_cache, k_cache_strides, HKV, D, 1, {n_pages, block_size}},
                     {v, strides + 6, v_cache, v_cache_strides, HKV, DV, 0, {n_pages, block_size}}};
  return launch(a, s, 3, B, T, rotary_dim, interleaved != 0, dt, stream) == cudaSuccess ? GDP_OK : GDP_ERR_CUDA;
}

}  // extern "C"
