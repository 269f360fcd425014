// Internal declarations of the linear-attention operators (per-head decay, no
// delta rule): one problem description shared by the recurrent and the chunked
// kernels. Nothing here is part of the C ABI (include/gdp.h is).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gdp_internal.cuh"

namespace gdp {

// One linear-attention problem, as validated by the API layer. Element strides of
// q, k, v: batch, token, head (the last dimension is contiguous). States are
// [.., K, V] fp32: dense (s0 -> sT, one entry per sequence, may be the same
// buffer) or pages of `pool` addressed by block tables.
struct LinearProblem {
  const void *q, *k, *v;
  int64_t qs[3], ks[3], vs[3];
  const float* g;   // null: no decay
  int g_token;      // 1: g [B, T, HV], 0: g [HV]
  const float* s0;  // may be null (zero states)
  float* sT;        // may be null
  float* pool;      // non-null: paged states
  int n_pages;
  const int32_t* tables;  // [N_seq, width]
  int width;
  const int32_t* ctx;     // [N_seq] tokens before this call
  int block;
  const int32_t* cu;      // may be null: N_seq == B sequences of T tokens
  int N_seq, B, T, H, HV, K, V;
  float scale;
  gdp_dtype dt;
  void* o;                // [B, T, HV, V] contiguous, dtype dt
  int32_t* status;        // may be null
  cudaStream_t stream;
};

// The recurrent form: one walk over a few tokens with the state in registers.
cudaError_t launch_linear_walk(const LinearProblem& p);

// The chunked form for any type, size and stride.
size_t linear_mma_workspace(int N_seq, int B, int T, int HV, int K, int V, gdp_dtype dt);
cudaError_t launch_linear_mma(const LinearProblem& p, uint8_t* ws);

// The chunked form on the tensor cores: whether sizes and type fit it, whether the
// tensors' addresses and strides do too (16-byte steps, for TMA), its workspace.
bool linear_tc_shape(int K, int V, gdp_dtype dt);
bool linear_tc_ok(const LinearProblem& p);
size_t linear_tc_workspace(int N_seq, int B, int T, int HV, int K, int V);
cudaError_t launch_linear_tc(const LinearProblem& p, uint8_t* ws);

}  // namespace gdp
