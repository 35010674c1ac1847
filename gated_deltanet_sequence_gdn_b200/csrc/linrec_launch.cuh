// linrec_launch.cuh -- host side shared by the scan and the backward of the gated linear
// recurrence: workspace layout, choice of the kernel by type, the launch.
#pragma once

#include <atomic>

#include "linrec_tile.cuh"

namespace gdn {

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
inline size_t seq_table_bytes(int B) {
  return align256((size_t)(B + 1) * sizeof(long long)) +
         2 * align256((size_t)(B + 1) * sizeof(int));
}

// Fills in what every launch of a call shares and writes the table of a packed batch.
cudaError_t make_chains(const LinrecArgs& a, void* workspace, cudaStream_t s, Chains* ch);
// The forward scan; wide_flag: the call's flag for float32 outputs.
cudaError_t launch_linrec_scan(const LinrecArgs& a, const Chains& ch, int wide_flag,
                               cudaStream_t s);

// The map of a tensor's tiles, where its rows start on 16 bytes.
template <int SPLIT, typename T>
bool map_tiles(CUtensorMap* m, const LinrecArgs& p, const void* base, long long ld) {
  if (((reinterpret_cast<uintptr_t>(base) | (uintptr_t)(ld * (long long)sizeof(T))) & 15) != 0)
    return false;
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t rows = p.cu ? 1 : p.B;
  const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.T, rows};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * sizeof(T), (cuuint64_t)p.T * ld * sizeof(T)};
  const cuuint32_t box[3] = {Shape<SPLIT>::kC, Shape<SPLIT>::kT, 1}, es[3] = {1, 1, 1};
  return enc(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
             3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Element pairs that are aligned.
inline int pairs(const void* p, long long ld, int es) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * es)) & (2 * es - 1)) == 0;
}

// Tokens of the longest sequence.
inline long long longest(const LinrecArgs& p) {
  if (p.cu == nullptr) return p.T;
  long long n = 0;
  for (int i = 0; i < p.B; ++i) n = p.cu[i + 1] - p.cu[i] > n ? p.cu[i + 1] - p.cu[i] : n;
  return n;
}
// The most blocks that one chain can use.
inline int most_blocks(const LinrecArgs& p) {
  const long long n = (longest(p) + kLinrecChunk - 1) / kLinrecChunk;
  return n < 1 ? 1 : n < kMaxCluster ? (int)n : kMaxCluster;
}

// What the runtime says of one kernel on one device, asked once: at[cs] clusters of cs blocks
// run at once (at[1]: 0 until asked).
struct KernelSlots {
  std::atomic<int> at[64][kMaxCluster + 1];
};
// A shape's kernels: of blocks that are alone on their chains (nothing of the exchange in their
// registers), and of clusters.
template <typename K>
struct ChainKernel {
  K alone, cluster;
  K of(int cs) const { return cs > 1 ? cluster : alone; }
};
// smem: of the call; most_smem: the most that any call of the kernel takes (its limit is set to
// that once and for all), both without the cluster's folds.
template <typename K>
cudaError_t kernel_slots(const ChainKernel<K>& k, size_t smem, size_t most_smem, KernelSlots* known,
                         const std::atomic<int>** slots) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::atomic<int>* at = known->at[dev];
  *slots = at;
  if (at[1].load(std::memory_order_acquire) != 0) return cudaSuccess;
  int sms = 0, per = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const size_t most = most_smem + 2 * kMaxCluster * sizeof(FoldRow);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k.alone, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k.cluster, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k.cluster, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, k.alone, kLinrecThreads, smem);
  if (e != cudaSuccess) return e;
  for (int cs = 2; cs <= kMaxCluster; ++cs) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms * 8 / cs * cs));
    cfg.blockDim = dim3(kLinrecThreads);
    cfg.dynamicSmemBytes = smem + 2 * cs * sizeof(FoldRow);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, k.cluster, &cfg);
    if (e != cudaSuccess) return e;
    at[cs].store(n, std::memory_order_relaxed);
  }
  at[1].store(sms * (per > 0 ? per : 1), std::memory_order_release);
  return cudaSuccess;
}

// How a call is cut: chunks of a tile, blocks of a cluster.
struct Split {
  int split, cs;
};
inline long long chains_of(const LinrecArgs& p, int split) {
  return (long long)p.B * ((p.D * (long long)split + 63) / 64);
}
// The shape that keeps the most of the machine at useful work: blocks at work at once times
// the share of a tile's channels that exist.  Chains that fill the machine run without
// clusters (608 to 704 chains of 4096 tokens take the same 286 us; in clusters, which end in a
// smaller last wave, 286 to 341); fewer run in the largest cluster whose launch still runs at
// once, and the smaller cluster (fewer exchanges) is taken where shapes are equal.  That is
// not always the faster of the equal ones: 32768 x 2048 would gain 8% from 2x6, where 8192 x
// 4096 and 8192 x 12288 lose or gain nothing by the larger cluster; what an exchange costs is
// not weighed against the longer rows of a wider tile.  Forward, us by shape (chunks of a tile
// x blocks of a cluster):
//   8192 tokens x 12288 channels  1x2 200, 1x3 224, 2x1 185, 2x2 192, 4x1 183 (taken, 768 blocks)
//   8192 x 8192                   1x3 143, 2x2 129, 4x1 123 (taken)
//   8192 x 4096                   1x6 80, 2x3 80, 4x1 80, 4x2 78 (taken)
//   32768 x 2048                  1x8 174, 2x6 153, 4x3 166 (taken), 4x6 178
//   131072 x 1024, tied           1x16 440, 2x8 363, 4x6 319, 4x8 297 (taken, 280 by now)
//   43 x 3699 x 14                53 in tiles of 64 channels, 22 of 16 (taken)
template <typename K>
cudaError_t choose_split(const LinrecArgs& p, const ChainKernel<K> (&ks)[3], size_t smem,
                         size_t most_smem, KernelSlots* known, Split* out) {
  *out = Split{1, 1};
  const long long chunks = (longest(p) + kLinrecChunk - 1) / kLinrecChunk;
  const long long mean = p.cu ? linrec_chunks(p.cu, p.B, p.T) / p.B : chunks;
  double best = 0.0;
  for (int j = 0; j < 3; ++j) {
    const int split = 1 << j;
    if (j > 0 && mean < split) break;  // tiles of more chunks than a sequence has
    const std::atomic<int>* slots = nullptr;
    cudaError_t e = kernel_slots(ks[j], smem, most_smem, known + j, &slots);
    if (e != cudaSuccess) return e;
    const long long n = chains_of(p, split), tiles = (chunks + split - 1) / split;
    const long long room = slots[1].load(std::memory_order_relaxed);
    int cs = 1;
    for (int i = 2; i <= kMaxCluster && i <= tiles; ++i)
      if (n <= slots[i].load(std::memory_order_relaxed)) cs = i;
    const double used = (double)p.B * p.D * split / (64.0 * n);
    const double work = used * (double)(n > room ? room : n * cs);
    if (work > 1.02 * best || (work > 0.98 * best && cs < out->cs)) {
      best = work > best ? work : best;
      *out = Split{split, cs};
    }
  }
  return cudaSuccess;
}

template <int SPLIT, typename K, typename... More>
cudaError_t launch_chains(K kernel, size_t smem, const LinrecArgs& p, const Chains& chains, int cs,
                          int vec, cudaStream_t s, More... more) {
  Chains ch = chains;
  ch.cs = cs;
  ch.nblk = (p.D + Shape<SPLIT>::kC - 1) / Shape<SPLIT>::kC;
  cudaLaunchAttribute attr[2];
  unsigned attrs = 0;
  if (cs > 1) {
    attr[attrs].id = cudaLaunchAttributeClusterDimension;
    attr[attrs].val.clusterDim.x = (unsigned)cs;
    attr[attrs].val.clusterDim.y = 1;
    attr[attrs++].val.clusterDim.z = 1;
  }
  if (ch.after) attr[attrs++] = early_launch();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p.B * ch.nblk * cs));
  cfg.blockDim = dim3(kLinrecThreads);
  cfg.dynamicSmemBytes = smem + (cs > 1 || SPLIT > 1 ? 2 * cs * sizeof(FoldRow) : 0);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = attrs;
  return cudaLaunchKernelEx(&cfg, kernel, p, ch, vec, more...);
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
