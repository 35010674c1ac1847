// linrec_tile.cuh -- what the scan of the gated linear recurrence and the reverse scan of
// its backward share: tiles of tokens x channels, their rows copied to shared memory ahead of
// use, and the carry from tile to tile.
//
// A chain is one sequence's 64 channels (or 32, or 16: Shape); its tiles are taken in turn by the
// blocks of one thread-block cluster (1 to 16 blocks: as many as it takes to fill the
// machine).  A lane holds 2 adjacent channels of 8 tokens.  Each thread folds its 8 tokens
// into (A, H): carry_out = A carry_in + H; the folds of a chunk's 8 groups of tokens meet in
// shared memory, so that within a chunk the recurrence is 8 + 8 steps instead of 64.  The
// blocks of a cluster send their chunks' (A, H) to one another through distributed shared
// memory, counted on the receiver's mbarrier, and each runs the same carry through the chunks
// of the round.  The carry is folded chunk by chunk in order whatever the cluster's size and
// the tile's shape, so the result does not depend on them.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "linrec.cuh"
#include "linrec_math.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace gdn {

constexpr int kWarps = 8;   // of a block
constexpr int kPer = 8;     // tokens of a thread
constexpr int kLinrecThreads = kWarps * 32;
constexpr int kMaxCluster = 16;
constexpr int kGroup = 4;   // tokens whose gates are formed together
constexpr int kTile = 64 * 64;  // elements of a tile

// A tile's shape: one chunk of 64 channels, or 2 of 32 or 4 of 16 where there are few chains
// to share the machine (half the channels are twice the chains and half the rounds of a
// cluster; their rows are 64 or 32 bytes of bf16 instead of 128).
template <int SPLIT>
struct Shape {
  static constexpr int kChunks = SPLIT;
  static constexpr int kT = SPLIT * kLinrecChunk, kC = 64 / SPLIT;
  static constexpr int kLanes = kC / 2;  // of one group of tokens
};
// A thread's place in it.
template <int SPLIT>
struct Spot {
  int lane, warp, cl, part, first;  // channel pair, which of the warp's groups, first token
  __device__ __forceinline__ Spot() {
    constexpr int kLanes = Shape<SPLIT>::kLanes;
    lane = threadIdx.x & 31;
    warp = threadIdx.x / 32;
    cl = lane % kLanes;
    part = lane / kLanes;
    first = (threadIdx.x / kLanes) * kPer;
  }
  // first element of the thread in a tile
  __device__ __forceinline__ int mine() const { return first * Shape<SPLIT>::kC + 2 * cl; }
  // For the joining warps, each part of which takes one of the tile's chunks: where group w of
  // the lane's chunk has its fold.
  __device__ __forceinline__ int group(int w) const {
    return (part * 8 + w) * Shape<SPLIT>::kLanes + cl;
  }
};

// Packed batches: each sequence's first token and first chunk, entry B the totals.
struct SeqTab {
  const long long* cu;  // NULL: dense rows
  const int* chunk0;
  const int* order;     // the sequences, long ones first (they would else end the launch alone)
};

// Maps of the inputs' tiles.
struct LinrecMaps {
  CUtensorMap x, a, b, dh;
};

// One launch: the chains by cluster, row by row of the batch.
struct Chains {
  SeqTab tab;
  int nblk;  // chains of a sequence
  int cs;    // blocks of a cluster
  int* status;
  unsigned spin;  // polls before a wait gives up
  int fault;      // test hook (WaitFaultSite): the first block of a cluster keeps its folds to
                  // itself, or the tiles' copies are not asked for
  bool tma;       // the inputs come by TMA
  bool after;     // the launch before it is the call's own and writes what this one reads
};

// One chain, as a block of its cluster sees it.
struct Chain {
  long long tok;   // the sequence's first token (row of the tensors)
  long long len;   // its tokens
  long long chunk0;
  int row, c0;     // sequence, first channel
  int chunks, tiles, rank;
};
template <int SPLIT, bool CLUSTER>
__device__ __forceinline__ Chain chain_of(const LinrecArgs& p, const Chains& ch) {
  Chain k;
  const int cs = CLUSTER ? ch.cs : 1, id = blockIdx.x / cs;
  k.rank = blockIdx.x % cs;
  k.row = id / ch.nblk;
  k.c0 = (id - k.row * ch.nblk) * Shape<SPLIT>::kC;
  if (ch.tab.cu != nullptr) k.row = ch.tab.order[k.row];
  if (ch.tab.cu == nullptr) {
    k.tok = (long long)k.row * p.T;
    k.len = p.T;
    k.chunk0 = (long long)k.row * ((p.T + (long long)kLinrecChunk - 1) / kLinrecChunk);
  } else {
    k.tok = ch.tab.cu[k.row];
    k.len = ch.tab.cu[k.row + 1] - k.tok;
    k.chunk0 = ch.tab.chunk0[k.row];
  }
  k.chunks = (int)((k.len + kLinrecChunk - 1) / kLinrecChunk);
  k.tiles = (k.chunks + Shape<SPLIT>::kChunks - 1) / Shape<SPLIT>::kChunks;
  return k;
}

// Shared memory of the carry: each thread's fold, and behind the kernel's own shared memory
// the cluster's folds, [2 rounds][cs][32].
struct CarrySmem {
  float4 fold[kLinrecThreads];  // (A, A', H, H') of each thread's two channels
  uint64_t full[2];             // the round's folds have arrived
  uint64_t loaded[2];           // the stage's tiles have
};
using FoldRow = float4[32];

__device__ __forceinline__ float2 first2(float4 v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 last2(float4 v) { return make_float2(v.z, v.w); }
__device__ __forceinline__ float4 join4(float2 a, float2 b) {
  return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void st_async_peer(uint32_t addr, float4 v, uint32_t bar_addr) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
          addr),
      "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar_addr)
      : "memory");
}

// (A, H) of the lane's chunk, from the folds of its 8 groups of tokens; BACK: (A, R).
template <int SPLIT, bool BACK>
__device__ __forceinline__ float4 chunk_fold(const Spot<SPLIT>& at, const CarrySmem& sm,
                                             const float2* back) {
  float2 A = both(1.f), H = both(0.f);
#pragma unroll 4
  for (int i = 0; i < 8; ++i) {
    const int j = at.group(BACK ? 7 - i : i);
    const float4 f = sm.fold[j];
    H = fma2(first2(f), H, BACK ? back[j] : last2(f));
    A = mul2(A, first2(f));
  }
  return join4(A, H);
}
// Runs v through the folds of blocks r0 .. r1 - 1 of the round; where `in` is given, it is set
// to what enters the lane's chunk of the last of them.  BACK: a tile's last chunk comes first.
template <int SPLIT, bool BACK>
__device__ __forceinline__ float2 carry_through(const FoldRow* row, int r0, int r1, float2 v,
                                                float2* in) {
  constexpr int kLanes = Shape<SPLIT>::kLanes;
  const int lane = threadIdx.x & 31, part = lane / kLanes, cl = lane % kLanes;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    float4 f[SPLIT];
#pragma unroll
    for (int i = 0; i < SPLIT; ++i) f[i] = row[r][kLanes * i + cl];
#pragma unroll
    for (int i = 0; i < SPLIT; ++i) {
      const int h = BACK ? SPLIT - 1 - i : i;
      if (in && h == part) *in = v;
      v = fma2(first2(f[h]), v, last2(f[h]));
    }
  }
  return v;
}
// One round of the carry, by one warp: own is the (A, H) of the lane's chunk of this block's
// tile.  Returns what enters that chunk and moves `carry` behind this block's tile; carry_rest
// moves it behind the round's other tiles, when nobody waits for it any more.  `lost`: a wait
// has expired, later ones are not tried.
template <int SPLIT, bool CLUSTER, bool BACK>
__device__ __forceinline__ float2 carry_round(const Chains& ch, int rank, int round, float4 own,
                                              CarrySmem& sm, FoldRow* folds, float2* carry,
                                              bool* lost) {
  float2 in = *carry;
  const int lane = threadIdx.x & 31, buf = round & 1;
  FoldRow* row = folds + (CLUSTER ? buf * ch.cs : buf);
  if (CLUSTER) {
    // Once a wait has expired its phase stays open: nothing is armed on it again (an arrival in
    // a phase that expects none is undefined), nothing sent, nothing waited for.
    if (!*lost) {
      if (lane == 0)
        tc::mbar_arrive_expect_tx(&sm.full[buf], (uint32_t)(ch.cs * 32 * sizeof(float4)));
      __syncwarp();
      if (!(ch.fault == kFaultLinrec && rank == 0))
        for (int r = 0; r < ch.cs; ++r)
          st_async_peer(tc::map_peer(&row[rank][lane], r), own, tc::map_peer(&sm.full[buf], r));
      const bool ok = tc::mbar_wait(&sm.full[buf], (round >> 1) & 1, nullptr, 0, ch.spin);
      *lost = !__all_sync(0xffffffffu, ok);
      if (*lost && lane == 0) report_timeout(ch.status, 0x4c52);
    }
  } else {  // the parts' chunks
    row[0][lane] = own;
    __syncwarp();
  }
  const float2 v = CLUSTER ? carry_through<SPLIT, BACK>(row, 0, rank, in, nullptr) : in;
  *carry = carry_through<SPLIT, BACK>(row, rank, rank + 1, v, &in);
  return in;
}
template <int SPLIT, bool CLUSTER, bool BACK>
__device__ __forceinline__ void carry_rest(const Chains& ch, int rank, int round,
                                           const FoldRow* folds, float2* carry) {
  if (CLUSTER)
    *carry = carry_through<SPLIT, BACK>(folds + (round & 1) * ch.cs, rank + 1, ch.cs, *carry,
                                        nullptr);
}

template <bool CLUSTER>
__device__ __forceinline__ void carry_begin(CarrySmem& sm) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.loaded[i], 1);
    }
    tc::fence_mbar_init();
  }
  __syncthreads();
  if (CLUSTER) tc::cluster_sync();  // the barriers are there before a peer counts on them
}
// No block leaves while a peer may still send to it.
template <bool CLUSTER>
__device__ __forceinline__ void carry_end() {
  __syncwarp();
  if (CLUSTER) tc::cluster_sync();
}

// Tiles of one tensor to shared memory [tokens][channels].  Tensors whose rows start on 16 bytes
// come by TMA, one instruction a tile, through a map over [channels][tokens][rows of the batch]
// (zeros behind the last token of a dense row and behind the last channel); the tokens behind
// a packed sequence are the next one's and are cleared by the caller.
__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, uint64_t* bar, int c0,
                                            int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(tc::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// The others by element: asynchronous copies of 4 bytes, or plain loads of 2.
__device__ __forceinline__ void cp_async4(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int SPLIT, typename T>
__device__ __forceinline__ void load_elements(T* dst, const void* base, long long ld,
                                              long long tok, int n, int c0, int D) {
  constexpr int kTileC = Shape<SPLIT>::kC, kTileT = Shape<SPLIT>::kT;
  constexpr int kStep = kLinrecThreads / kTileC;  // rows at once
  const int r0 = threadIdx.x / kTileC, c = threadIdx.x % kTileC;
  const bool in = c < D - c0;
  const T* src = static_cast<const T*>(base) + (tok + r0) * ld + c0 + (in ? c : 0);
  dst += threadIdx.x;
#pragma unroll 8
  for (int r = 0; r < kTileT; r += kStep) {
    const bool here = in && r0 + r < n;
    if (sizeof(T) == 4)
      cp_async4(dst + r * kTileC, here ? static_cast<const void*>(src) : base, here ? 4 : 0);
    else
      dst[r * kTileC] = here ? *src : from_f32<T>(0.f);
    src += kStep * ld;
  }
}
// Clears the rows of a tile behind its n tokens.
template <int SPLIT, typename T>
__device__ __forceinline__ void clear_rows(T* tile, int n) {
  for (int i = n * Shape<SPLIT>::kC + threadIdx.x; i < kTile; i += kLinrecThreads)
    tile[i] = from_f32<T>(0.f);
}

// A lane's two channels.
__device__ __forceinline__ float2 get2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 get2(const __nv_bfloat16* p) {
  const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ void put2(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
__device__ __forceinline__ void put2(__nv_bfloat16* p, float2 v) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}
// `cols` of them are inside, and a pair may not be aligned.
template <typename T>
__device__ __forceinline__ void put2(T* p, float2 v, int cols) {
  if (cols > 0) p[0] = from_f32<T>(v.x);
  if (cols > 1) p[1] = from_f32<T>(v.y);
}
// An output tensor of a block: a 64-bit base that moves from tile to tile, the same for all
// threads, and 32-bit byte offsets inside a tile (256 rows of at most 2^21 elements).
template <typename T>
struct Rows {
  char* base;
  uint32_t off, ld;  // bytes: of the thread's first element, from token to token
  __device__ __forceinline__ void begin(void* p, long long row_elems, long long tok, int c0,
                                        int first, int lane2) {
    base = static_cast<char*>(p) + (tok * row_elems + c0) * (long long)sizeof(T);
    ld = (uint32_t)row_elems * (uint32_t)sizeof(T);
    off = (uint32_t)first * ld + (uint32_t)lane2 * (uint32_t)sizeof(T);
  }
  __device__ __forceinline__ T* at(int i) const {
    return reinterpret_cast<T*>(base + (off + (uint32_t)i * ld));
  }
  __device__ __forceinline__ void advance(int tokens) { base += (long long)tokens * ld; }
};
// Two floats of a [.., D] array at channel c (0 outside, or where the array is NULL).
__device__ __forceinline__ float2 read2(const float* base, long long row, int c, int D) {
  if (base == nullptr) return both(0.f);
  base += row * D + c;
  return make_float2(c < D ? base[0] : 0.f, c + 1 < D ? base[1] : 0.f);
}
__device__ __forceinline__ void write2(float* base, long long row, int c, int D, float2 v) {
  if (base == nullptr) return;
  base += row * D + c;
  if (c < D) base[0] = v.x;
  if (c + 1 < D) base[1] = v.y;
}

}  // namespace gdn
