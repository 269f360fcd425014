// Linear attention, chunked forms: how sequences are cut into segments, the segment records of
// packed batches, and the states at the segment starts.
//
// A segment is a work item of its own when there are too few (sequence, head) pairs to fill the
// GPU: the state pass of a chunked kernel forms each segment's own U from a zero state, the
// combine kernel here turns those into the states at the segment starts, and the whole pass then
// runs over all segments at once. Reading k and v twice costs less than idle SMs: 2 x 4096 tokens of
// 16 heads (K = V = 128) take 70 us in four segments each, as long as half their tokens would in one.
#include <algorithm>

#include "linear_chunk.cuh"

namespace gdp {
namespace linear {
namespace {

// Segment records of a packed batch (one CTA): each sequence cut at multiples of Lseg positions,
// records sorted by length, longest first (by counting ranks, so up to kSortMax of them; 6 to
// 8 us for 16 sequences with their tables).
// Checked on the way: offsets that decrease or leave [0, T] make every sequence empty; a negative
// context or a page outside the pool makes that sequence empty; either sets the status.
constexpr int kRecThreads = 512;
constexpr int kSortMax = 4096;

__device__ __forceinline__ int table_page(const LinearProblem& p, int r, int64_t b) {
  if (b < 0 || b >= p.width) return -1;
  const int pg = p.tables[(int64_t)r * p.width + b];
  return pg >= 0 && pg < p.n_pages ? pg : -1;
}

__global__ void __launch_bounds__(kRecThreads) linear_segments_kernel(const __grid_constant__ LinearProblem p,
                                                                      int Lseg, int bound, SegRec* recs, int2* seqs,
                                                                      int* split) {
  pdl_wait();
  __shared__ int lens[kSortMax];
  __shared__ int2 wsum[kRecThreads / 32 + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  for (int i = tid; i < p.N_seq; i += kRecThreads) {
    const int x = p.cu[i], y = p.cu[i + 1];
    bad |= x < 0 || y < x || y > p.T;
  }
  bad = __syncthreads_or(bad);
  bool any = bad, cut = false;
  int base = 0, sbase = 0;  // segments before this round of sequences, those of cut ones
  for (int i0 = 0; i0 < p.N_seq; i0 += kRecThreads) {
    const int i = i0 + tid;
    int t0 = 0, n = 0, pos = 0, cnt = 0;
    if (i < p.N_seq) {
      if (!bad) {
        t0 = p.cu[i];
        n = p.cu[i + 1] - t0;
      }
      if (p.pool && n > 0) {
        pos = p.ctx[i];
        bool off = pos < 0;
        if (!off)
          for (int64_t j = pos > 0 ? (pos - 1) / p.block : 0; j <= ((int64_t)pos + n - 1) / p.block; ++j)
            off |= table_page(p, i, j) < 0;
        if (off) n = pos = 0;
        any |= off;
      }
      cnt = segment_count(pos % C, n, Lseg);
    }
    cut |= cnt > 1;
    const int slots = cnt > 1 ? cnt : 0;
    int s = cnt, z = slots;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o), w = __shfl_up_sync(0xffffffffu, z, o);
      if (lane >= o) {
        s += y;
        z += w;
      }
    }
    if (lane == 31) wsum[warp] = make_int2(s, z);
    __syncthreads();
    if (tid == 0) {
      int2 run = make_int2(0, 0);
      for (int w = 0; w < kRecThreads / 32; ++w) {
        const int2 y = wsum[w];
        wsum[w] = run;
        run.x += y.x;
        run.y += y.y;
      }
      wsum[kRecThreads / 32] = run;
    }
    __syncthreads();
    const int first = base + wsum[warp].x + s - cnt, slot = sbase + wsum[warp].y + z - slots;
    base += wsum[kRecThreads / 32].x;
    sbase += wsum[kRecThreads / 32].y;
    if (i < p.N_seq) {
      if (seqs) seqs[i] = make_int2(slot, cnt);
      const int off = pos % C;
      for (int j = 0; j < cnt; ++j) {
        int lo, hi;
        segment_span(off, n, Lseg, j, &lo, &hi);
        // (a position past 2^31 stays one of 32 bits; chunks and pages count it unsigned)
        SegRec r{t0 + lo, hi - lo, i, p.pool ? (int)((uint32_t)pos + (uint32_t)lo) : lo, j == 0, j == cnt - 1, slots ? slot + j : 0, 0};
        recs[first + j] = r;
        if (first + j < kSortMax) lens[first + j] = r.n;
      }
    }
    __syncthreads();
  }
  any = __syncthreads_or(any);
  cut = __syncthreads_or(cut);
  if (tid == 0) {
    *split = cut;
    if (p.status) *p.status = any ? kDevBadSeqlens : kDevOk;
  }
  const int count = base;
  if (count <= kSortMax && count > 1) {  // in place: every thread reads its records first
    SegRec mine[kSortMax / kRecThreads];
    int rank[kSortMax / kRecThreads];
#pragma unroll
    for (int q = 0; q < kSortMax / kRecThreads; ++q) {
      const int i = tid + q * kRecThreads;
      if (i < count) {
        mine[q] = recs[i];
        int r = 0;
        const int len = lens[i];
        for (int j = 0; j < count; ++j) r += lens[j] > len || (lens[j] == len && j < i);
        rank[q] = r;
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSortMax / kRecThreads; ++q)
      if (tid + q * kRecThreads < count) recs[rank[q]] = mine[q];
  }
  for (int i = count + tid; i < bound; i += kRecThreads) recs[i] = SegRec{0, 0, -1, 0, 0, 0, 0, 0};
}

// States at the segment starts: S_0 = the sequence's initial state, S_{j+1} = w_j S_j + U_j,
// in place of the U's. A thread per VEC state elements. A read and a write of the scratch,
// bound by the trips to memory of eight segments' loads at a time: 13 us alone with cold caches for 32
// heads of four segments (15 MB). With four at a time a sequence of 37 segments takes 2 us longer.
template <int VEC>
__global__ void __launch_bounds__(256, 4) linear_combine_kernel(const __grid_constant__ ChunkArgs a, const int2* seqs) {
  pdl_wait();
  if (no_split(a)) return;
  const LinearProblem& p = a.p;
  const int64_t sz = (int64_t)p.K * p.V;
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;
  if (e >= sz) return;
  for (int64_t pair = blockIdx.y; pair < (int64_t)p.N_seq * p.HV; pair += gridDim.y) {
    const int seq = (int)(pair / p.HV), hv = (int)(pair - (int64_t)seq * p.HV);
    int first, cnt;
    if (a.recs) {
      const int2 x = seqs[seq];
      first = x.x;
      cnt = x.y;
    } else {
      first = seq * a.nseg;
      cnt = a.nseg;
    }
    if (cnt < 2) continue;
    const float* src = nullptr;
    if (p.pool) {
      const int c = p.ctx[seq];
      if (c > 0) src = p.pool + (int64_t)p.tables[(int64_t)seq * p.width + (c - 1) / p.block] * p.HV * sz;
    } else if (p.s0) {
      src = p.s0 + (int64_t)seq * p.HV * sz;
    }
    float s[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) s[i] = 0.f;
    auto load = [](float* d, const float* q) {
      if (VEC == 4) *reinterpret_cast<float4*>(d) = __ldcg(reinterpret_cast<const float4*>(q));
      else *d = __ldcg(q);
    };
    if (src) load(s, src + hv * sz + e);
    float* seg = a.segS + ((int64_t)first * p.HV + hv) * sz + e;
    const int64_t step = (int64_t)p.HV * sz;
    const float2* w = a.segW + (int64_t)first * p.HV + hv;
    for (int j0 = 0; j0 < cnt; j0 += 8) {  // eight segments' loads in flight
      const int m = min(8, cnt - 1 - j0);
      alignas(16) float u[8][VEC];
      float2 f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < m) {
          load(u[j], seg + (j0 + j) * step);
          f[j] = __ldcg(w + (int64_t)(j0 + j) * p.HV);
        }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < cnt) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) seg[(j0 + j) * step + i] = s[i];
          if (j < m)
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[i] = fmaf(f[j].x, s[i], fmaf(f[j].y, s[i], u[j][i]));
        }
    }
  }
}

}  // namespace

cudaError_t launch_segments(const LinearProblem& p, const Plan& x, SegRec* recs, int2* seqs, int* split) {
  return launch_pdl(linear_segments_kernel, dim3(1), dim3(kRecThreads), 0, p.stream, p, x.Lseg, (int)x.bound, recs, seqs,
                    split);
}

cudaError_t launch_combine(const ChunkArgs& a, const int2* seqs) {
  const int64_t sz = (int64_t)a.p.K * a.p.V;
  const bool vec = sz % 4 == 0;
  // what is resident: a packed batch's CTAs may all have nothing to do
  const int64_t gx = cdiv(sz, vec ? 1024 : 256), gy = std::max<int64_t>(1, 4 * sm_count() / gx);
  const dim3 grid((unsigned)gx, (unsigned)std::min<int64_t>((int64_t)a.p.N_seq * a.p.HV, gy));
  return vec ? launch_pdl(linear_combine_kernel<4>, grid, dim3(256), 0, a.p.stream, a, seqs)
             : launch_pdl(linear_combine_kernel<1>, grid, dim3(256), 0, a.p.stream, a, seqs);
}

}  // namespace linear
}  // namespace gdp
