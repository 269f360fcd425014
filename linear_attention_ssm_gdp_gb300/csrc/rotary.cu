// Position rotation of heads, and appending keys and values to a paged cache with the rotation on
// the way.
//
// Pair i of a head's R rotated elements turns by pos f_i: (a, b) -> A (a c - b s, a s + b c) with
// c = cos(pos f_i), s = sin(pos f_i) and an amplitude A; the gradient's pass turns by the opposite
// angle. Pairs are (i, i + R / 2) or neighbours (2 i, 2 i + 1).
//
// Angles. A position times a frequency in 32 bits is off by pos 2^-24 of a turn's radians (0.06 at a
// position of 10^6), so angles are counted in turns as 64-bit integers: F_i = frac(f_i / 2 pi) 2^64
// once per CTA from the fp64 frequency (off by 2^-52 of a frequency and 2^-65 of a turn), and the phase of a
// position is the integer product pos F_i mod 2^64, itself exact for every int32 position. Its nearest quarter turn picks the quadrant, the rest (at
// most an eighth of a turn) goes to sincospif as a float.
//
// Bound by HBM: every element is read and written once. A warp takes a token (or a share of its heads, where
// tokens are few): its lanes form the token's cosines and sines in shared memory, and each keeps those of one
// place in the head, eight pairs of two 16-byte vectors or one vector of neighbours, in registers for all the
// heads that it then walks, two heads' loads in flight. Where sizes, strides or addresses are not whole
// 16-byte vectors, smaller ones or single elements go in the same walk, more heads at a time. 8192 tokens of 32
// heads of 128 in bf16: 24 us, 84 % of the copy rate (35 with a CTA for a few tokens and the cosines read from
// shared memory for every head).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "fast_div.cuh"
#include "gdp_internal.cuh"

namespace gdp {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kResident = 4;  // CTAs of an SM
constexpr int kMostDim = 1024;  // of a head

// One tensor [B, T, H, D] of a call: `places` of a head are walked, the first `pairs` of them rotated.
struct Rows {
  const void* x;
  void* y;
  int64_t xs[3], ys[3];  // batch (cache: page), token, head, in elements
  int H, places, pairs, heads;  // heads: side by side in a warp
  Div by_places;
};

struct RotaryArgs {
  Rows r[3];
  int cached;  // tensors from this one on are written to the cache (3: none)
  const int32_t* pos;
  const double* freq;
  const int64_t* slot;
  int64_t n_slots;
  int block;
  int32_t* status;
  int half, offset;  // R / 2, first rotated element
  float amplitude;
  int backward;
  int64_t tokens;
  int T, log_parts;  // tokens per batch entry; warps that share a token
  Div by_T;
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
// Pairs (a, b) -> (a x - b y, a y + b x), two at a time where the type packs two to a register.
template <typename T>
__device__ __forceinline__ void turn1(T& a, T& b, const float2& w) {
  const float p = to_f(a), q = to_f(b);
  a = from_f<T>(p * w.x - q * w.y);
  b = from_f<T>(p * w.y + q * w.x);
}
__device__ __forceinline__ float2 two(const __nv_bfloat16* e) { return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(e)); }
__device__ __forceinline__ float2 two(const __half* e) { return __half22float2(*reinterpret_cast<const __half2*>(e)); }
__device__ __forceinline__ void put(__nv_bfloat16* e, float x, float y) { *reinterpret_cast<__nv_bfloat162*>(e) = __floats2bfloat162_rn(x, y); }
__device__ __forceinline__ void put(__half* e, float x, float y) { *reinterpret_cast<__half2*>(e) = __floats2half2_rn(x, y); }
// (a0, b0), (a1, b1) apart
template <typename T>
__device__ __forceinline__ void turn2(T* a, T* b, const float2& w0, const float2& w1) {
  if constexpr (sizeof(T) == 4) {
    turn1(a[0], b[0], w0);
    turn1(a[1], b[1], w1);
  } else {
    const float2 p = two(a), q = two(b);
    put(a, p.x * w0.x - q.x * w0.y, p.y * w1.x - q.y * w1.y);
    put(b, p.x * w0.y + q.x * w0.x, p.y * w1.y + q.y * w1.x);
  }
}
// neighbours
template <typename T>
__device__ __forceinline__ void turn_next(T* a, const float2& w) {
  if constexpr (sizeof(T) == 4) {
    turn1(a[0], a[1], w);
  } else {
    const float2 p = two(a);
    put(a, p.x * w.x - p.y * w.y, p.x * w.y + p.y * w.x);
  }
}

template <typename T, int VN, bool INTER>
__global__ void __launch_bounds__(kThreads, kResident) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  using V = Vec<T, VN>;
  constexpr bool kPairs = !(INTER && VN > 1);    // a rotated place is two vectors
  constexpr int kTurns = kPairs ? VN : VN / 2;   // pairs of a place
  constexpr int kBatch = sizeof(V) >= 16 ? 2 : sizeof(V) >= 8 ? 4 : 8;  // heads whose loads are in flight
  extern __shared__ unsigned long long sm[];
  unsigned long long* turns = sm;                // [half]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float2* cs = reinterpret_cast<float2*>(sm + a.half) + warp * a.half;
  pdl_wait();
  const int64_t items = a.tokens << a.log_parts, stride = (int64_t)gridDim.x * kWarps;
  int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  // position and slot of the next item, on their way beside this one
  int pos1 = 0;
  int64_t slot1 = -1;
  auto fetch = [&](int64_t i) {
    if (i >= items) return;
    if (a.half > 0) pos1 = a.pos[i >> a.log_parts];
    if (a.cached < 3) slot1 = a.slot[i >> a.log_parts];
  };
  fetch(item);
  for (int i = tid; i < a.half; i += kThreads) {
    double t = a.freq[i] * 0.15915494309189533577;                   // 1 / 2 pi
    t -= floor(t);
    turns[i] = __double2ull_rn(t * 18446744073709551616.0);
  }
  __syncthreads();
  for (; item < items; item += stride) {
    const uint32_t t = (uint32_t)(item >> a.log_parts), b = quot(t, a.by_T), tb = t - b * a.T;
    const int part = (int)(item & ((1 << a.log_parts) - 1));
    int64_t page = -1, place = 0;
    const unsigned long long pos = (unsigned long long)(long long)pos1;
    const int64_t slot = slot1;
    fetch(item + stride);
    if (a.cached < 3) {
      if (slot >= 0 && slot < a.n_slots) {
        page = slot / a.block;
        place = slot - page * a.block;
      } else if (slot != -1 && lane == 0) {
        report(a.status, GDP_ERR_INVALID_ARG);
      }
    }
    if (a.half > 0) {
      __syncwarp();  // (the last token's cosines have been read)
      for (int i = lane; i < a.half; i += 32) {
        const unsigned long long ph = pos * turns[i];
        const unsigned q = (unsigned)((ph + (1ull << 61)) >> 62);    // nearest quarter turn
        float s, k;
        sincospif((float)(long long)(ph - ((unsigned long long)q << 62)) * 0x1p-63f, &s, &k);
        if (q & 1) {
          const float x = s;
          s = k;
          k = -x;
        }
        if (q & 2) { s = -s; k = -k; }
        if (a.backward) s = -s;
        cs[i] = make_float2(k * a.amplitude, s * a.amplitude);
      }
      __syncwarp();
    }
#pragma unroll 1
    for (int j = 0; j < 3; ++j) {
      const Rows& r = a.r[j];
      if (r.H == 0) continue;
      const T* x = static_cast<const T*>(r.x) + b * r.xs[0] + tb * r.xs[1];
      T* y = static_cast<T*>(r.y);
      if (j >= a.cached) {
        if (page < 0) continue;
        y += page * r.ys[0] + place * r.ys[1];
      } else {
        y += b * r.ys[0] + tb * r.ys[1];
      }
      const int beside = (int)quot(lane, r.by_places);  // head of this lane among those of the warp
#pragma unroll 1
      for (int i0 = 0; i0 < r.places; i0 += 32) {
        const int i = r.heads > 1 ? lane - beside * r.places : i0 + lane;
        if (i >= r.places || (r.heads > 1 && beside >= r.heads)) continue;
        // elements from e0 on and the pairs' others from e1 on; `turn`: rotated
        int e0, e1 = 0, first;
        bool turn;
        if (kPairs) {
          turn = i < r.pairs;
          first = i * VN;
          if (turn) {
            e0 = a.offset + (INTER ? 2 * i : i * VN);
            e1 = e0 + (INTER ? 1 : a.half);
          } else {
            e0 = (i - r.pairs) * VN;
            if (r.pairs > 0 && e0 >= a.offset) e0 += 2 * a.half;
          }
        } else {
          e0 = i * VN;
          first = (e0 - a.offset) >> 1;  // (the offset is even here; may be negative)
          turn = r.pairs > 0 && e0 + VN > a.offset && first < a.half;
        }
        float2 w[kTurns];
        if (turn)
#pragma unroll
          for (int n = 0; n < kTurns; ++n)  // (a vector's neighbours outside the rotated part stay as they are)
            w[n] = kPairs || (first + n >= 0 && first + n < a.half) ? cs[first + n] : make_float2(0.f, 0.f);
        const int step = r.heads << a.log_parts;
#pragma unroll 1
        for (int h0 = part * r.heads + (r.heads > 1 ? beside : 0); h0 < r.H; h0 += kBatch * step) {
          V v0[kBatch], v1[kBatch];
#pragma unroll
          for (int n = 0; n < kBatch; ++n)
            if (h0 + n * step < r.H) {
              const T* src = x + (h0 + n * step) * r.xs[2];
              v0[n] = *reinterpret_cast<const V*>(src + e0);
              if (kPairs && turn) v1[n] = *reinterpret_cast<const V*>(src + e1);
            }
#pragma unroll
          for (int n = 0; n < kBatch; ++n)
            if (h0 + n * step < r.H) {
              T* dst = y + (h0 + n * step) * r.ys[2];
              if (turn) {
                if constexpr (VN == 1) {
                  turn1(v0[n].e[0], v1[n].e[0], w[0]);
                } else if constexpr (kPairs) {
#pragma unroll
                  for (int m = 0; m < VN; m += 2) turn2(v0[n].e + m, v1[n].e + m, w[m], w[m + 1]);
                } else {
#pragma unroll
                  for (int m = 0; m < kTurns; ++m)
                    if (first + m >= 0 && first + m < a.half) turn_next(v0[n].e + 2 * m, w[m]);
                }
                if (kPairs) *reinterpret_cast<V*>(dst + e1) = v1[n];
              }
              *reinterpret_cast<V*>(dst + e0) = v0[n];
            }
        }
      }
    }
  }
}

template <typename T, int VN>
cudaError_t go(const RotaryArgs& a, bool inter, cudaStream_t stream) {
  const int64_t ctas = cdiv(a.tokens << a.log_parts, kWarps);
  const int grid = (int)std::min<int64_t>(ctas, (int64_t)sm_count() * kResident);
  const size_t smem = (size_t)a.half * 8 * (1 + kWarps);
  return inter ? launch_pdl(rotary_kernel<T, VN, true>, dim3(grid), dim3(kThreads), smem, stream, a)
               : launch_pdl(rotary_kernel<T, VN, false>, dim3(grid), dim3(kThreads), smem, stream, a);
}

template <typename T>
cudaError_t go16(const RotaryArgs& a, int vn, bool inter, cudaStream_t stream) {
  return vn == 8   ? go<T, 8>(a, inter, stream)
         : vn == 4 ? go<T, 4>(a, inter, stream)
         : vn == 2 ? go<T, 2>(a, inter, stream)
                   : go<T, 1>(a, inter, stream);
}

bool dtype_ok(gdp_dtype dt) { return dt == GDP_BF16 || dt == GDP_F16 || dt == GDP_F32; }

// Whether a tensor's rows are whole vectors of vn elements on their grid.
bool whole(const void* p, const int64_t* s, const int* n, int D, int vn, int esz) {
  if (reinterpret_cast<uintptr_t>(p) % (vn * esz) || D % vn) return false;
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
  // vectors of up to 16 bytes, as sizes, strides and addresses allow (72 elements with a rotated half of 18 in bf16:
  // vectors of 2)
  const int esz = dt == GDP_F32 ? 4 : 2;
  int w = 16 / esz;
  const auto fits = [&](int vn) {
    for (int i = 0; i < n; ++i) {
      const Side& s = sides[i];
      if (s.H == 0) continue;
      const int xn[3] = {B, T, s.H}, yn[3] = {s.dst[0], s.dst[1], s.H};
      if (!whole(s.x, s.xs, xn, s.D, vn, esz) || !whole(s.y, s.ys, yn, s.D, vn, esz)) return false;
      if (s.rotated && R > 0 && (inter ? a.offset % 2 != 0 : a.offset % vn != 0 || (R / 2) % vn != 0)) return false;
    }
    return true;
  };
  while (w > 1 && !fits(w)) w /= 2;
  a.half = R / 2;
  int walks = 1;  // batches of heads that a token's longest walk takes
  for (int i = 0; i < 3; ++i) {
    Rows& r = a.r[i];
    r = Rows{};
    r.by_places = div_by(1);
    if (i >= n || sides[i].H == 0) continue;
    const Side& s = sides[i];
    r.x = s.x;
    r.y = s.y;
    for (int j = 0; j < 3; ++j) { r.xs[j] = s.xs[j]; r.ys[j] = s.ys[j]; }
    r.H = s.H;
    const int rot = s.rotated ? R : 0;
    r.pairs = rot / 2 / w;
    r.places = r.pairs + (s.D - rot) / w;
    if (inter && w > 1) {
      r.pairs = rot > 0;  // (only whether any pair of the head turns)
      r.places = s.D / w;
    }
    r.by_places = div_by(r.places);
    r.heads = r.places <= 32 ? 32 / r.places : 1;
    walks = std::max(walks, (int)std::min<int64_t>(cdiv(s.H, r.heads), 64));
  }
  a.T = T;
  a.by_T = div_by(T);
  // warps that share a token: none where tokens fill the SMs, up to one for each step of its walk
  a.log_parts = 0;
  while ((a.tokens << a.log_parts) < 4ll * sm_count() && (1 << a.log_parts) < walks) ++a.log_parts;
  switch (dt) {
    case GDP_BF16: return go16<__nv_bfloat16>(a, w, inter, stream);
    case GDP_F16: return go16<__half>(a, w, inter, stream);
    default: return w == 4 ? go<float, 4>(a, inter, stream) : w == 2 ? go<float, 2>(a, inter, stream) : go<float, 1>(a, inter, stream);
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

// No two elements of a destination in one place, as far as a stride alone says.
bool apart(const int64_t* s, int n0, int n1, int n2) {
  return (n0 <= 1 || s[0] > 0) && (n1 <= 1 || s[1] > 0) && (n2 <= 1 || s[2] > 0);
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
  if (!x || !y || !strides_ok(x_strides, 3) || !strides_ok(y_strides, 3) || !apart(y_strides, B, T, H))
    return GDP_ERR_INVALID_ARG;
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
  a.block = 1;
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
      !strides_ok(v_cache_strides, 3) || !apart(k_cache_strides, n_pages, block_size, HKV) ||
      !apart(v_cache_strides, n_pages, block_size, HKV))
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
  a.block = block_size;
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
