// linrec.cuh -- arguments and workspace layout of the gated linear recurrence, shared by
// the C entry points and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// A kernel that reads what the launch before it wrote, launched while that one still runs: its
// blocks come in as the other's leave, and wait in wait_for_launch() for the rest of them.
__device__ __forceinline__ void wait_for_launch() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
inline cudaLaunchAttribute early_launch() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr[1] = {early_launch()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

constexpr int kLinrecChunk = 64;  // tokens of a chunk (GDN_LINREC_CHUNK of the C ABI)

// One batch: B rows of T tokens, or (cu != NULL) B packed sequences over T tokens.
// ld*: elements between the tokens of a tensor.
struct LinrecArgs {
  const void *x, *a, *b;  // b NULL: no write gate
  const float *A_log, *dt_bias, *h0;
  const long long* cu;    // HOST
  int B, T, D, dtype, flags;
  long long ldx, lda, ldb;
  // forward
  void* h;  // NULL: states only
  long long ldh;
  float *ht, *states_out;
  // backward
  const void* dh;
  long long lddh;
  const float *dht, *states;
  void *dx, *da, *db;
  long long lddx, ldda, lddb;
  float *dA_log, *ddt_bias, *dh0;
};

// Chunks of the batch (each sequence's chunks start at its first token).
long long linrec_chunks(const long long* cu, int B, int T);
size_t linrec_workspace_bytes(const long long* cu, int B, int T, int D);
size_t linrec_bwd_workspace_bytes(const long long* cu, int B, int T, int D, bool states_given,
                                  int flags);
cudaError_t launch_linrec_fwd(const LinrecArgs& a, void* workspace, cudaStream_t s);
cudaError_t launch_linrec_bwd(const LinrecArgs& a, void* workspace, cudaStream_t s);
cudaError_t launch_linrec_step(const LinrecArgs& a, float* state, cudaStream_t s);

// Arguments of the norm-and-rotation of q and k.
struct QkRopeArgs {
  const void *q, *k;
  const long long* positions;
  const float *inv_freq, *q_weight, *k_weight;
  long long tokens;
  int Hq, Hk, d, rot, dtype, flags;
  long long ldq, ldk;
  float eps, scale;
  void *q_out, *k_out;  // outputs, or the gradients dq, dk
  long long ldqo, ldko;
  // backward
  const void *gq, *gk;  // gradients at the outputs
  long long ldgq, ldgk;
  float *dqw, *dkw;
};
size_t qk_rope_bwd_workspace_bytes(long long tokens, int Hq, int Hk, int d, int flags);
cudaError_t launch_qk_rope(const QkRopeArgs& a, cudaStream_t s);
cudaError_t launch_qk_rope_bwd(const QkRopeArgs& a, void* workspace, cudaStream_t s);

}  // namespace gdn
