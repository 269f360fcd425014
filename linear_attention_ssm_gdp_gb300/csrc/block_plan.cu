// Block plan of a serving step, built on the device from request lengths: offsets
// of the packed tokens, each token's request, position and cache slot, and the new
// entries of the block tables, taken in request order from a list of free pages.
//
// With blocks(x) = ceil(x / block): request r needs blocks(ctx + query) -
// blocks(ctx) new pages; exclusive prefix sums over the requests give the token
// offsets and the places in the free list. The token at position p sits in the
// page of block p / block, at p % block.
//
// The work is a few bytes per token, so a call is bound by its launch and by three
// dependent trips to memory. One launch does it all: every CTA scans the lengths
// of all requests by itself (they are few, and stay in shared memory), then fills
// its share of the tokens and table rows; no CTA waits for another, and no entry
// of a block table that one CTA writes is read by another (a token in a new block
// takes its page from the free list). 256 requests of one token: 6.2 us in a captured
// graph; 64 requests of up to 2048 tokens (131072 in all at most): 8.5 us.
#include <algorithm>

#include "gdp_internal.cuh"

namespace gdp {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanMax = 16384;  // requests: 8 bytes each of shared memory

struct PlanArgs {
  const int32_t *ctx, *query;
  int n;
  int32_t* tables;
  int width;
  const int32_t* free_pages;
  int n_free;
  const int32_t* free_used;
  int block, max_tokens;
  int32_t *cu, *req, *pos;
  int64_t* slot;
  int32_t *used_out, *status;
};

__global__ void __launch_bounds__(kPlanThreads) block_plan_kernel(const __grid_constant__ PlanArgs a) {
  pdl_wait();
  extern __shared__ int sm[];
  int* cu = sm;               // [n + 1] token offsets
  int* first = sm + a.n + 1;  // [n] first new page's place in the free list
  __shared__ long long wq[17], wn[17];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int used_in = *a.free_used;
  const int used = used_in < 0 ? a.n_free : used_in;
  const int per = (a.n + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(tid * per, a.n), r1 = min(r0 + per, a.n);
  int flags = used_in < 0 ? 1 : 0;

  // a request's tokens and new pages; {0, 0} (and a flag) where its lengths are not valid
  auto lengths = [&](int r, int& q, int& need) {
    const int64_t c = a.ctx[r], m = a.query[r];
    q = need = 0;
    if (c < 0 || m < 0 || c + m > (int64_t)a.width * a.block) return false;
    q = (int)m;
    need = (int)((c + m + a.block - 1) / a.block - (c + a.block - 1) / a.block);
    return true;
  };
  long long sq = 0, sn = 0;
  for (int r = r0; r < r1; ++r) {
    int q, need;
    if (!lengths(r, q, need)) flags |= 1;
    sq += q;
    sn += need;
  }
  long long iq = sq, in = sn;  // inclusive scan over the block
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, iq, o), y = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) { iq += x; in += y; }
  }
  if (lane == 31) { wq[warp] = iq; wn[warp] = in; }
  __syncthreads();
  long long eq = iq - sq, en = in - sn;
  for (int w = 0; w < warp; ++w) { eq += wq[w]; en += wn[w]; }
  // requests are admitted in order while their pages and tokens fit; sums only grow,
  // so the admitted ones are the leading ones, and offsets stay flat after them
  long long cq = eq, cn = en;
  __syncthreads();
  if (tid == 0) { wq[16] = 0; wn[16] = 0; }
  __syncthreads();
  long long fq = 0, fn = 0;  // totals admitted through this thread's requests
  bool mine = false;
  for (int r = r0; r < r1; ++r) {
    int q, need;
    lengths(r, q, need);
    const bool fits = (cn + need == 0 || used + cn + need <= a.n_free) && cq + q <= a.max_tokens;
    if (!fits) flags |= 2;
    first[r] = fits ? used + (int)cn : -1;
    cq += q;
    cn += need;
    cu[r + 1] = fits ? (int)cq : -1;
    if (fits) { fq = cq; fn = cn; mine = true; }
  }
  if (mine) {  // integers: the order does not matter
    atomicMax(&wq[16], fq);
    atomicMax(&wn[16], fn);
  }
  if (tid == 0) cu[0] = 0;
  flags = __syncthreads_or(flags & 1) ? 1 : 0;
  const int total = (int)wq[16], pages = (int)wn[16];
  bool left_out = false;
  for (int r = r0; r < r1; ++r)
    if (cu[r + 1] < 0) {
      cu[r + 1] = total;
      left_out = true;
    }
  flags |= __syncthreads_or(left_out) ? 2 : 0;

  if (blockIdx.x == 0) {
    for (int r = tid; r <= a.n; r += kPlanThreads) a.cu[r] = cu[r];
    if (tid == 0) {
      *a.used_out = used_in < 0 ? used_in : used + pages;
      if (a.status) *a.status = flags;
    }
  }
  // new table entries: a warp per request
  for (int r = blockIdx.x * (kPlanThreads / 32) + warp; r < a.n; r += gridDim.x * (kPlanThreads / 32)) {
    if (first[r] < 0) continue;
    int q, need;
    lengths(r, q, need);
    if (need == 0) continue;
    const int have = (int)(((int64_t)a.ctx[r] + a.block - 1) / a.block);
    for (int j = lane; j < need; j += 32)
      a.tables[(int64_t)r * a.width + have + j] = a.free_pages[first[r] + j];
  }
  // (64 bits: the last step of the loop passes max_tokens by up to a grid)
  for (int64_t t64 = blockIdx.x * kPlanThreads + tid; t64 < a.max_tokens; t64 += gridDim.x * kPlanThreads) {
    const int t = (int)t64;
    int rr = -1, pp = -1;
    int64_t ss = -1;
    if (t < total) {
      int lo = 0, hi = a.n - 1;  // first request whose end is past t
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid + 1] > t) hi = mid; else lo = mid + 1;
      }
      const int c = a.ctx[lo];
      rr = lo;
      pp = c + (t - cu[lo]);
      const int b = pp / a.block, have = (int)(((int64_t)c + a.block - 1) / a.block);
      const int page = b < have ? a.tables[(int64_t)lo * a.width + b] : a.free_pages[first[lo] + b - have];
      if (page >= 0) ss = (int64_t)page * a.block + (pp - b * a.block);
    }
    a.req[t] = rr;
    a.pos[t] = pp;
    a.slot[t] = ss;
  }
}

}  // namespace
}  // namespace gdp

using namespace gdp;

extern "C" gdp_status gdp_block_plan(const int32_t* context_lens, const int32_t* query_lens, int n,
                                     int32_t* block_tables, int max_blocks,
                                     const int32_t* free_pages, int n_free,
                                     const int32_t* free_used, int block_size, int max_tokens,
                                     int32_t* cu_seqlens, int32_t* token_req, int32_t* token_pos,
                                     int64_t* slot_map, int32_t* free_used_out, int32_t* status,
                                     cudaStream_t stream) {
  if (n < 0 || max_blocks < 0 || n_free < 0 || block_size <= 0 || max_tokens < 0)
    return GDP_ERR_INVALID_ARG;
  // (one CTA writes free_used_out while others read free_used)
  if (!cu_seqlens || !free_used || !free_used_out || free_used == free_used_out) return GDP_ERR_INVALID_ARG;
  if (n > 0 && (!context_lens || !query_lens)) return GDP_ERR_INVALID_ARG;
  if (n > 0 && max_blocks > 0 && !block_tables) return GDP_ERR_INVALID_ARG;
  if (n_free > 0 && !free_pages) return GDP_ERR_INVALID_ARG;
  if (max_tokens > 0 && (!token_req || !token_pos || !slot_map)) return GDP_ERR_INVALID_ARG;
  if (n > kPlanMax || (int64_t)max_blocks * block_size > INT32_MAX) return GDP_ERR_UNSUPPORTED;
  const PlanArgs a{context_lens, query_lens, n, block_tables, max_blocks, free_pages, n_free,
                   free_used, block_size, max_tokens, cu_seqlens, token_req, token_pos, slot_map,
                   free_used_out, status};
  const int smem = (2 * n + 1) * 4;
  // (48 KB unasked, the kernel's static part among them)
  if (smem > 40 * 1024 && allow_smem<block_plan_kernel>((2 * kPlanMax + 1) * 4) != cudaSuccess)
    return GDP_ERR_CUDA;
  const int64_t want = std::max(cdiv(max_tokens, kPlanThreads), cdiv(n, kPlanThreads / 32));
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(want, sm_count()));
  return launch_pdl(block_plan_kernel, dim3(grid), dim3(kPlanThreads), smem, stream, a) == cudaSuccess
             ? GDP_OK
             : GDP_ERR_CUDA;
}
