// linrec_chain.cuh -- what the scan of the gated linear recurrence and the reverse scan of
// its backward share: tiles of 64 tokens x 64 channels handed out by ticket, their rows
// copied to shared memory ahead of use, and the carry handed from tile to tile.
//
// A tile is 8 warps x 8 tokens; a lane holds 2 adjacent channels.  Each thread folds its 8
// tokens into (A, H): carry_out = A carry_in + H; the folds of the 8 warps meet in shared
// memory, so that within a tile the recurrence is 8 + 8 steps instead of 64.  A ninth warp
// joins tiles: it publishes a tile's (A, H) where the carry is not known yet, reads the
// neighbours' until it meets a known carry, and publishes its own.  The carry of a tile is
// always A carry_in + H of its predecessor's carry, folded tile by tile in order, whichever
// of the two it was read from: the result does not depend on the schedule.
//
// Tickets are taken in the order of the carries, so a tile only waits for tiles that a
// running block already holds: the smallest ticket not finished is never waiting.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "linrec.cuh"
#include "linrec_math.cuh"

namespace gdn {

constexpr int kTileT = kLinrecChunk;  // tokens of a tile
constexpr int kTileC = 64;            // channels of a tile
constexpr int kWorkWarps = 8;         // compute warps, 8 tokens each
constexpr int kPer = kTileT / kWorkWarps;
constexpr int kWorkThreads = kWorkWarps * 32;
constexpr int kLinrecThreads = kWorkThreads + 32;  // and the joining warp

// Packed batches: each sequence's first token and first chunk, entry B the totals.
struct SeqTab {
  const long long* cu;  // NULL: dense rows
  const int* chunk0;
};

// The work of one launch: tiles by ticket, and the arrays that join them.
struct Chain {
  SeqTab tab;
  int B, T, D, nblk;
  int per_row;     // chunks of a dense row
  int tiles;
  int* ticket;     // NULL: no tile has a neighbour; tiles by block index
  int* flags;      // [tile] 0, 1 (aggregate published), 2 (carry published)
  float4* agg;     // [tile][32 lanes] (A, H) of two channels
  float* carry;    // [chunk][D]: what enters the chunk
  int* status;
  unsigned spin;   // polls before a wait gives up
  bool fault;      // test hook: first tiles do not publish
};

struct Tile {
  long long tok;  // first token (row of the tensors)
  int row;        // sequence
  int chunk;      // its number in `carry` and `flags`
  int n;          // tokens, 1..64
  int c0;         // first channel
  int before, after;  // chunks of the sequence before and after this one
};

// Tile of a ticket; REV: later chunks first.
template <bool REV>
__device__ __forceinline__ Tile tile_of(const Chain& ch, int k) {
  if (REV) k = ch.tiles - 1 - k;
  Tile t;
  const int f = k / ch.nblk;
  t.c0 = (k - f * ch.nblk) * kTileC;
  int tt, cnt;
  long long len;
  if (ch.tab.cu == nullptr) {  // chunk by chunk over all rows: their chains advance together
    tt = f / ch.B;
    t.row = f - tt * ch.B;
    cnt = ch.per_row;
    len = ch.T;
    t.chunk = t.row * cnt + tt;
    t.tok = (long long)t.row * ch.T;
  } else {  // the last sequence that starts at or before chunk f
    int lo = 0, hi = ch.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (ch.tab.chunk0[mid] <= f) lo = mid; else hi = mid;
    }
    t.row = lo;
    tt = f - ch.tab.chunk0[lo];
    cnt = ch.tab.chunk0[lo + 1] - ch.tab.chunk0[lo];
    t.tok = ch.tab.cu[lo];
    len = ch.tab.cu[lo + 1] - t.tok;
    t.chunk = f;
  }
  t.tok += (long long)tt * kTileT;
  const long long left = len - (long long)tt * kTileT;
  t.n = left < kTileT ? (int)left : kTileT;
  t.before = tt;
  t.after = cnt - 1 - tt;
  return t;
}

// Takes the next ticket's tile into slot k % 3 (the joining warp's lane 0).
template <bool REV, typename S>
__device__ __forceinline__ void next_tile(const Chain& ch, S& sm, int k) {
  const int id = ch.ticket ? atomicAdd(ch.ticket, 1) : (int)(blockIdx.x + k * gridDim.x);
  sm.more[k % 3] = id < ch.tiles;
  if (id < ch.tiles) sm.tile[k % 3] = tile_of<REV>(ch, id);
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src),
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

// A tile's rows of one tensor to shared memory [64][64], zeros outside the sequence and
// behind the last channel; `vec`: rows start on 16 bytes and move in 16-byte pieces.  Called
// by the compute warps.
template <typename T>
__device__ __forceinline__ void load_tile(T* dst, const void* base, long long ld, const Tile& t,
                                          int D, bool vec) {
  const T* src = static_cast<const T*>(base) + t.tok * ld + t.c0;
  const int cols = D - t.c0 < kTileC ? D - t.c0 : kTileC;
  if (vec) {
    constexpr int E = 16 / sizeof(T), P = kTileC / E;  // elements of a piece, pieces of a row
#pragma unroll
    for (int i = 0; i < kTileT * P / kWorkThreads; ++i) {
      const int k = threadIdx.x + i * kWorkThreads, r = k / P, c = (k % P) * E;
      const int in = r < t.n && c < cols ? (cols - c < E ? cols - c : E) : 0;
      cp_async16(dst + r * kTileC + c, in ? src + r * ld + c : static_cast<const T*>(base),
                 in * (int)sizeof(T));
    }
  } else {
#pragma unroll 4
    for (int i = 0; i < kTileT * kTileC / kWorkThreads; ++i) {
      const int k = threadIdx.x + i * kWorkThreads, r = k / kTileC, c = k % kTileC;
      const bool in = r < t.n && c < cols;
      if (sizeof(T) == 4)
        cp_async4(dst + r * kTileC + c, in ? src + r * ld + c : static_cast<const T*>(base),
                  in ? 4 : 0);
      else
        dst[r * kTileC + c] = in ? src[r * ld + c] : from_f32<T>(0.f);
    }
  }
}

// A lane's two channels.
__device__ __forceinline__ float2 get2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 get2(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}
// `cols` of them are inside; `pair`: the two may be stored at once.
__device__ __forceinline__ void put2(float* p, float a, float b, int cols, bool pair) {
  if (pair && cols == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
  } else {
    if (cols > 0) p[0] = a;
    if (cols > 1) p[1] = b;
  }
}
__device__ __forceinline__ void put2(__nv_bfloat16* p, float a, float b, int cols, bool pair) {
  if (pair && cols == 2) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
  } else {
    if (cols > 0) p[0] = __float2bfloat16_rn(a);
    if (cols > 1) p[1] = __float2bfloat16_rn(b);
  }
}
// Two floats of a [.., D] array at channel c (0 outside).
__device__ __forceinline__ float2 read2(const float* row, int c, int D) {
  return make_float2(c < D ? __ldcg(row + c) : 0.f, c + 1 < D ? __ldcg(row + c + 1) : 0.f);
}
__device__ __forceinline__ void write2(float* row, int c, int D, float2 v) {
  if (c < D) __stcg(row + c, v.x);
  if (c + 1 < D) __stcg(row + c + 1, v.y);
}

__device__ __forceinline__ int load_flag(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_flag(int* p, int v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// The joining warp's part of a tile: what enters it, given the tile's own (A, H) of the
// lane's two channels.  STEP: +1 where the carry comes from the chunk before, -1 after.
// edge: what enters the sequence's first tile of the chain.
template <int STEP>
__device__ __forceinline__ float2 chain_in(const Chain& ch, const Tile& t, float4 own,
                                           const float* edge_row) {
  const int lane = threadIdx.x & 31, c = t.c0 + 2 * lane, blk = t.c0 / kTileC;
  const int reach = STEP > 0 ? t.before : t.after;  // tiles the carry has come through
  if (reach == 0) {
    return edge_row ? read2(edge_row, c, ch.D) : make_float2(0.f, 0.f);
  }
  bool published = false;
  unsigned polls = 0;
  for (;;) {
    const int f = lane < reach ? load_flag(ch.flags + (t.chunk - STEP * (1 + lane)) * ch.nblk + blk) : 0;
    const unsigned known = __ballot_sync(0xffffffffu, f == 2);
    const unsigned some = __ballot_sync(0xffffffffu, f != 0);
    const int j = known ? __ffs(known) - 1 : 32;
    if (j < 32 && ((~some) & ((1u << j) - 1u)) == 0) {
      __syncwarp();
      float2 v = read2(ch.carry + (long long)(t.chunk - STEP * j) * ch.D, c, ch.D);
      for (int l = j - 1; l >= 0; --l) {
        const float4 g =
            __ldcg(ch.agg + ((long long)(t.chunk - STEP * (1 + l)) * ch.nblk + blk) * 32 + lane);
        v.x = fmaf(g.x, v.x, g.y);
        v.y = fmaf(g.z, v.y, g.w);
      }
      return v;
    }
    if (!published) {
      __stcg(ch.agg + ((long long)t.chunk * ch.nblk + blk) * 32 + lane, own);
      __threadfence();
      __syncwarp();
      if (lane == 0) store_flag(ch.flags + t.chunk * ch.nblk + blk, 1);
      published = true;
    }
    if (++polls > ch.spin) {
      if (lane == 0) report_timeout(ch.status, 0x4c52);
      return make_float2(0.f, 0.f);
    }
  }
}
// What leaves the tile: the next one's carry (entering chunk + STEP).
template <int STEP>
__device__ __forceinline__ void chain_out(const Chain& ch, const Tile& t, float2 v) {
  const int lane = threadIdx.x & 31, c = t.c0 + 2 * lane, blk = t.c0 / kTileC;
  write2(ch.carry + (long long)(t.chunk + STEP) * ch.D, c, ch.D, v);
  __threadfence();
  __syncwarp();
  if (lane == 0 && !(ch.fault && (STEP > 0 ? t.before : t.after) == 0))
    store_flag(ch.flags + t.chunk * ch.nblk + blk, 2);
}

}  // namespace gdn
