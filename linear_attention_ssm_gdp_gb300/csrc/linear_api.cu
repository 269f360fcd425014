// C ABI entry points of the linear-attention operators: argument validation and
// dispatch. Every validation runs before anything is launched; nothing here
// allocates device memory or synchronises.
#include <algorithm>

#include "linear_internal.cuh"
#include "linear_plan.h"

using namespace gdp;

namespace {

bool dtype_ok(gdp_dtype dt) { return dt == GDP_BF16 || dt == GDP_F16 || dt == GDP_F32; }

// Workspace: status word, then what the kernel that takes the problem lays out. The size does
// not depend on the strides, so it is the larger of the two kernels' where both may.
size_t linear_ws(int N_seq, int B, int T, int HV, int K, int V, gdp_dtype dt) {
  const size_t m = linear_mma_workspace(N_seq, B, T, HV, K, V, dt);
  return linear_tc_shape(K, V, dt) ? std::max(m, linear_tc_workspace(N_seq, B, T, HV, K, V)) : m;
}

// Lengths that the chunked kernels count in 32 bits.
bool lengths_ok(int N_seq, int B, int T) {
  return (int64_t)B * T <= linear::kMostTokens && N_seq <= linear::kMostSeqs;
}

bool sizes_ok(int N_seq, int B, int T, int H, int HV, int K, int V) {
  return N_seq >= 0 && B >= 0 && T >= 0 && H > 0 && HV > 0 && K > 0 && V > 0 && HV % H == 0;
}

gdp_status check(const LinearProblem& p, const int64_t* strides) {
  if (!dtype_ok(p.dt)) return GDP_ERR_UNSUPPORTED;
  if (!sizes_ok(p.N_seq, p.B, p.T, p.H, p.HV, p.K, p.V)) return GDP_ERR_INVALID_ARG;
  if (p.K > 256 || p.V > 1024) return GDP_ERR_UNSUPPORTED;
  if ((int64_t)p.B * p.T > INT32_MAX) return GDP_ERR_UNSUPPORTED;
  const bool work = (int64_t)p.B * p.T > 0;
  if (work && (!p.q || !p.k || !p.v || !p.o || !strides)) return GDP_ERR_INVALID_ARG;
  if (work)
    for (int i = 0; i < 9; ++i)
      if (strides[i] < 0) return GDP_ERR_INVALID_ARG;
  const auto off16 = [](const void* x) { return reinterpret_cast<uintptr_t>(x) % 16 != 0; };
  if (off16(p.s0) || off16(p.sT) || off16(p.pool)) return GDP_ERR_INVALID_ARG;
  if (p.pool) {
    if (p.n_pages <= 0 || p.width <= 0 || p.block <= 0) return GDP_ERR_INVALID_ARG;
    if (p.N_seq > 0 && (!p.tables || !p.ctx)) return GDP_ERR_INVALID_ARG;
  }
  return GDP_OK;
}

void set_strides(LinearProblem& p, const int64_t* s) {
  if (!s) return;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = s[i];
    p.ks[i] = s[3 + i];
    p.vs[i] = s[6 + i];
  }
}

gdp_status chunk(LinearProblem& p, const int64_t* strides, void* workspace, size_t bytes) {
  const gdp_status st = check(p, strides);
  if (st != GDP_OK) return st;
  if (!lengths_ok(p.N_seq, p.B, p.T)) return GDP_ERR_UNSUPPORTED;
  if (p.cu ? p.B != 1 : p.N_seq != p.B) return GDP_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % kAlign != 0 ||
      bytes < linear_ws(p.N_seq, p.B, p.T, p.HV, p.K, p.V, p.dt))
    return GDP_ERR_WORKSPACE;
  set_strides(p, strides);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.status = reinterpret_cast<int32_t*>(ws);
  const cudaError_t e = (int64_t)p.B * p.T > 0 && linear_tc_ok(p) ? launch_linear_tc(p, ws) : launch_linear_mma(p, ws);
  return e == cudaSuccess ? GDP_OK : GDP_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t gdp_linear_chunk_fwd_workspace_size(int B, int T, int N_seq, int H, int HV, int K, int V,
                                           gdp_dtype dt) {
  if (!sizes_ok(N_seq, B, T, H, HV, K, V) || K > 256 || V > 1024 || !dtype_ok(dt) ||
      !lengths_ok(N_seq, B, T))
    return 0;
  return linear_ws(N_seq, B, T, HV, K, V, dt);
}

gdp_status gdp_linear_chunk_fwd(const void* q, const void* k, const void* v, const int64_t* strides,
                                const float* g, int g_per_token, const float* initial_state,
                                const int32_t* cu_seqlens, int N_seq, int B, int T, int H, int HV,
                                int K, int V, float scale, gdp_dtype dt, void* o,
                                float* final_state, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
  LinearProblem p{};
  p.q = q; p.k = k; p.v = v; p.g = g; p.g_token = g_per_token; p.s0 = initial_state;
  p.sT = final_state; p.cu = cu_seqlens; p.N_seq = N_seq; p.B = B; p.T = T; p.H = H; p.HV = HV;
  p.K = K; p.V = V; p.scale = scale; p.dt = dt; p.o = o; p.stream = stream;
  return chunk(p, strides, workspace, workspace_bytes);
}

gdp_status gdp_linear_chunk_fwd_paged(const void* q, const void* k, const void* v,
                                      const int64_t* strides, const float* g, int g_per_token,
                                      const int32_t* cu_seqlens, int N_seq, int T, int H, int HV,
                                      int K, int V, float scale, gdp_dtype dt, float* state_pool,
                                      int n_pages, const int32_t* block_tables, int max_blocks,
                                      const int32_t* context_lens, int block_size, void* o,
                                      void* workspace, size_t workspace_bytes,
                                      cudaStream_t stream) {
  if (!cu_seqlens || !state_pool) return GDP_ERR_INVALID_ARG;
  if (block_size > 0 && block_size % 64 != 0) return GDP_ERR_UNSUPPORTED;
  LinearProblem p{};
  p.q = q; p.k = k; p.v = v; p.g = g; p.g_token = g_per_token; p.cu = cu_seqlens; p.N_seq = N_seq;
  p.B = 1; p.T = T; p.H = H; p.HV = HV; p.K = K; p.V = V; p.scale = scale; p.dt = dt;
  p.pool = state_pool; p.n_pages = n_pages; p.tables = block_tables; p.width = max_blocks;
  p.ctx = context_lens; p.block = block_size; p.o = o; p.stream = stream;
  return chunk(p, strides, workspace, workspace_bytes);
}

gdp_status gdp_linear_recurrent_update(const void* q, const void* k, const void* v,
                                       const int64_t* strides, const float* g, int g_per_token,
                                       float* state, int n, int S, int H, int HV, int K, int V,
                                       float scale, gdp_dtype dt, void* o, cudaStream_t stream) {
  if (S < 1 || S > 16) return GDP_ERR_INVALID_ARG;
  LinearProblem p{};
  p.q = q; p.k = k; p.v = v; p.g = g; p.g_token = g_per_token; p.s0 = state; p.sT = state;
  p.N_seq = n; p.B = n; p.T = S; p.H = H; p.HV = HV; p.K = K; p.V = V; p.scale = scale; p.dt = dt;
  p.o = o; p.stream = stream;
  if (n > 0 && !state) return GDP_ERR_INVALID_ARG;
  const gdp_status st = check(p, strides);
  if (st != GDP_OK || n == 0) return st;
  set_strides(p, strides);
  return launch_linear_walk(p) == cudaSuccess ? GDP_OK : GDP_ERR_CUDA;
}

gdp_status gdp_linear_recurrent_update_paged(const void* q, const void* k, const void* v,
                                             const int64_t* strides, const float* g,
                                             int g_per_token, float* state_pool, int n_pages,
                                             const int32_t* block_tables, int max_blocks,
                                             const int32_t* context_lens, int block_size, int n,
                                             int S, int H, int HV, int K, int V, float scale,
                                             gdp_dtype dt, void* o, int32_t* status,
                                             cudaStream_t stream) {
  if (S < 1 || S > 16 || !state_pool) return GDP_ERR_INVALID_ARG;
  LinearProblem p{};
  p.q = q; p.k = k; p.v = v; p.g = g; p.g_token = g_per_token; p.N_seq = n; p.B = n; p.T = S;
  p.H = H; p.HV = HV; p.K = K; p.V = V; p.scale = scale; p.dt = dt; p.pool = state_pool;
  p.n_pages = n_pages; p.tables = block_tables; p.width = max_blocks; p.ctx = context_lens;
  p.block = block_size; p.o = o; p.status = status; p.stream = stream;
  const gdp_status st = check(p, strides);
  if (st != GDP_OK || n == 0) return st;
  set_strides(p, strides);
  return launch_linear_walk(p) == cudaSuccess ? GDP_OK : GDP_ERR_CUDA;
}

}  // extern "C"
