// linrec_launch.cuh -- host side shared by the scan and the backward of the gated linear
// recurrence: workspace layout, choice of the kernel by type, the persistent launch.
#pragma once

#include "linrec_chain.cuh"

namespace gdn {

constexpr unsigned kLinrecSpin = 1u << 21;  // polls of a neighbour's flag before giving up (> 1 s)

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
inline size_t seq_table_bytes(int B) {
  return align256((size_t)(B + 1) * sizeof(long long)) + align256((size_t)(B + 1) * sizeof(int));
}
inline size_t flags_bytes(long long tiles) { return align256(256 + (size_t)tiles * sizeof(int)); }
inline size_t carry_bytes(long long chunks, int D) {
  return align256((size_t)chunks * D * sizeof(float));
}
inline size_t chain_bytes(const long long* cu, int B, int T, int D) {
  const long long chunks = linrec_chunks(cu, B, T), tiles = chunks * ((D + kTileC - 1) / kTileC);
  return (cu ? seq_table_bytes(B) : 0) + flags_bytes(tiles) +
         (size_t)tiles * 32 * sizeof(float4) + carry_bytes(chunks, D);
}

// Lays the chain's arrays out in the workspace, writes the sequence table (`table`) and
// clears the flags.  carry: where the tiles' carries go (NULL: into the workspace).
cudaError_t make_chain(const LinrecArgs& a, void* workspace, float* carry, bool table,
                       cudaStream_t s, Chain* ch);
// The forward scan on a chain; wide_flag: the call's flag for float32 outputs.
cudaError_t launch_linrec_scan(const LinrecArgs& a, const Chain& ch, int wide_flag,
                               cudaStream_t s);
// Rows of dst that belong to empty sequences: src's (zeros where NULL).
cudaError_t copy_empty(const LinrecArgs& a, const Chain& ch, const float* src, float* dst,
                       cudaStream_t s);

// Rows that start on 16 bytes; rows whose element pairs are aligned.
inline int rows16(const void* p, long long ld, int es) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * es)) & 15) == 0;
}
inline int pairs(const void* p, long long ld, int es) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * es)) & (2 * es - 1)) == 0;
}

// One block a slot of the machine (or a tile, where those are fewer).
template <typename K, typename... More>
cudaError_t launch_chain(K kernel, size_t smem, const LinrecArgs& p, const Chain& ch, int vec,
                         cudaStream_t s, More... more) {
  int dev = 0, sms = 0, per = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kLinrecThreads, smem);
  if (e != cudaSuccess) return e;
  const long long most = (long long)sms * (per > 0 ? per : 1);
  kernel<<<(unsigned)(ch.tiles < most ? ch.tiles : most), kLinrecThreads, smem, s>>>(p, ch, vec, more...);
  return cudaGetLastError();
}

// Calls f.template run<TX, TG, GIVEN, SCALE, WIDE>() for the call's types: x in TX, the gates
// in TG (GIVEN: g and beta themselves, float32), WIDE: outputs (forward) or gradients
// (backward) in float32.
template <typename F, typename TX, typename TG, bool GIVEN, bool WIDE>
cudaError_t by_scale(const LinrecArgs& p, const F& f) {
  if (p.flags & GDN_LINREC_TIED) return f.template run<TX, TG, GIVEN, kScaleTied, WIDE>();
  if (p.flags & GDN_LINREC_UNIT) return f.template run<TX, TG, GIVEN, kScaleUnit, WIDE>();
  return f.template run<TX, TG, GIVEN, kScaleNone, WIDE>();
}
template <typename F>
cudaError_t by_type(const LinrecArgs& p, int wide_flag, const F& f) {
  using bf16 = __nv_bfloat16;
  const bool given = p.flags & GDN_GATES_PRECOMPUTED;
  if (p.dtype == GDN_F32)
    return given ? by_scale<F, float, float, true, true>(p, f)
                 : by_scale<F, float, float, false, true>(p, f);
  if (p.flags & wide_flag)
    return given ? by_scale<F, bf16, float, true, true>(p, f)
                 : by_scale<F, bf16, bf16, false, true>(p, f);
  return given ? by_scale<F, bf16, float, true, false>(p, f)
               : by_scale<F, bf16, bf16, false, false>(p, f);
}
template <typename TX, bool WIDE> struct Wide { using type = TX; };
template <typename TX> struct Wide<TX, true> { using type = float; };

}  // namespace gdn
