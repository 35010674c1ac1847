// qk_rope.cu -- norm of each head of q and k and the position rotation, one pass:
//   n = x / sqrt(mean(x^2) + eps) * w    (GDN_QK_RMSNORM)
//   n = x / sqrt(sum(x^2) + eps)         (GDN_QK_L2NORM), or n = x,
//   (p, q) -> (p cos - q sin, q cos + p sin) over pairs of the first `rot` channels,
//   angle = position * inv_freq[i],
// queries times `scale`; and its backward.
//
// HBM-bound: every row is read once and written once.  A head is held by a group of 8, 16
// or 32 lanes, 8 consecutive channels a lane (16 bytes of bf16), so the sums are shuffles
// inside the group and a pair's partner is in the same lane or one shuffle away.  A warp
// takes one token at a time and runs over its heads, so that the token's angles are
// evaluated once per warp and shared by them.
//
// Angles: position * inv_freq in float32 is off by 2^-24 of the angle, which is 0.01 rad
// at position 10^5.  A turn is held as a 64-bit fraction instead: phase = position *
// round(2^64 inv_freq / 2 pi) modulo 2^64 is exact but for that one rounding, for every
// 64-bit position, and its top 32 bits go to sincospi.
#include "common.cuh"
#include "linrec.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxHalf = 128;  // rotated pairs of a head (d <= 256)

enum Pairs { kPairShuffle = 0, kPairLane = 1, kPairShared = 2 };

struct Smem {
  float2 cs[kWarps][kMaxHalf];    // cos, sin of the warp's token
  float swap[kWarps][32 * 8 + 8];  // kPairShared: the warp's rows
};

// 8 elements from / to one lane's place of a row; `cnt` of them are inside the head.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int cnt, float* f) {
  if (VEC) {
    if (cnt > 0) {
      if (sizeof(T) == 2) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = __uint_as_float(w[i] << 16);
          f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      } else {
        const float4 v0 = reinterpret_cast<const float4*>(p)[0];
        const float4 v1 = reinterpret_cast<const float4*>(p)[1];
        f[0] = v0.x; f[1] = v0.y; f[2] = v0.z; f[3] = v0.w;
        f[4] = v1.x; f[5] = v1.y; f[6] = v1.z; f[7] = v1.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < cnt ? to_f32(p[i]) : 0.f;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int cnt, const float* f) {
  if (VEC) {
    if (cnt > 0) {
      if (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) p[i] = from_f32<T>(f[i]);
  }
}

// One turn of inv_freq as a 64-bit fraction.
__device__ __forceinline__ unsigned long long turn_fraction(float inv_freq) {
  const double t = (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}

// What a lane knows of its 8 channels.
struct Lane {
  int e0, cnt;       // first channel, channels inside the head
  int pairs;         // Pairs
  int half, rot;
  int src;           // kPairShuffle: the partner's lane
};

// Rotates the lane's 8 values (the whole warp calls it); BACK: by the opposite angle.
template <bool BACK>
__device__ __forceinline__ void rotate(const Lane& L, const float* c, const float* s, float* swap,
                                       float* y) {
  if (L.rot == 0) return;
  if (L.pairs == kPairLane) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float p = y[i], q = y[i + 1];
      if (L.e0 + i < L.rot) {
        const float sn = BACK ? -s[i] : s[i];
        y[i] = p * c[i] - q * sn;
        y[i + 1] = q * c[i] + p * sn;
      }
    }
    return;
  }
  float o[8];
  if (L.pairs == kPairShuffle) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, y[i], L.src);
  } else {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 8; ++i) swap[lane * 8 + i] = y[i];
    __syncwarp();
    const int row = lane * 8 - L.e0;  // the head's first value
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = L.e0 + i;
      o[i] = e < L.rot ? swap[row + (e < L.half ? e + L.half : e - L.half)] : 0.f;
    }
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = L.e0 + i;
    const bool lo = e < L.half;
    if (e < L.rot) y[i] = (lo != BACK) ? y[i] * c[i] - o[i] * s[i] : y[i] * c[i] + o[i] * s[i];
  }
}

template <int GROUP>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = GROUP / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int GROUP>
__device__ __forceinline__ Lane lane_of(const QkRopeArgs& p, int pairs) {
  Lane L;
  const int lane = threadIdx.x & 31;
  L.e0 = (lane % GROUP) * 8;
  L.cnt = p.d - L.e0 < 8 ? (p.d - L.e0 < 0 ? 0 : p.d - L.e0) : 8;
  L.pairs = pairs;
  L.half = p.rot / 2;
  L.rot = p.rot;
  const int step = L.half / 8;
  L.src = L.e0 < L.half ? lane + step : L.e0 < L.rot ? lane - step : lane;
  return L;
}

// The angles of one position into the warp's row of shared memory, and from there to the
// lane's registers.
struct Turns {
  unsigned long long u[kMaxHalf / 32];
};
__device__ __forceinline__ Turns load_turns(const QkRopeArgs& p) {
  Turns t;
#pragma unroll
  for (int j = 0; j < kMaxHalf / 32; ++j) {
    const int i = (threadIdx.x & 31) + 32 * j;
    t.u[j] = i < p.rot / 2 ? turn_fraction(p.inv_freq[i]) : 0ull;
  }
  return t;
}
__device__ __forceinline__ void angles(const QkRopeArgs& p, const Lane& L, const Turns& t,
                                       long long pos, float2* cs, float* c, float* s) {
  if (L.rot == 0) return;
  __syncwarp();  // the last token's reads are done
#pragma unroll
  for (int j = 0; j < kMaxHalf / 32; ++j) {
    const int i = (threadIdx.x & 31) + 32 * j;
    if (i < L.half) {
      const unsigned long long ph = (unsigned long long)pos * t.u[j];
      float sn, cn;
      sincospif((float)(int)(ph >> 32) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31 half turns
      cs[i] = make_float2(cn, sn);
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = L.e0 + i;
    const int k = L.pairs == kPairLane ? e / 2 : e < L.half ? e : e - L.half;
    const float2 v = e < L.rot ? cs[k] : make_float2(1.f, 0.f);
    c[i] = v.x;
    s[i] = v.y;
  }
}

template <typename T, int GROUP, bool VEC>
__global__ void __launch_bounds__(kThreads)
qk_rope_kernel(QkRopeArgs p, int pairs, int splits, int heads_per) {
  __shared__ Smem sm;
  constexpr int NH = 32 / GROUP;  // heads a warp holds at once
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const Lane L = lane_of<GROUP>(p, pairs);
  const Turns turns = load_turns(p);
  const bool rms = p.flags & GDN_QK_RMSNORM, l2 = p.flags & GDN_QK_L2NORM;
  float qw[8], kw[8], c[8], s[8];
  load8<float, false>(p.q_weight + L.e0, p.q_weight ? L.cnt : 0, qw);
  load8<float, false>(p.k_weight + L.e0, p.k_weight ? L.cnt : 0, kw);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (!p.q_weight) qw[i] = 1.f;
    if (!p.k_weight) kw[i] = 1.f;
    qw[i] *= p.scale;
  }
  const int H = p.Hq + p.Hk;
  const long long items = p.tokens * splits;
  for (long long it = blockIdx.x * (long long)kWarps + warp; it < items;
       it += (long long)gridDim.x * kWarps) {
    const long long t = it / splits;
    const int h0 = (int)(it % splits) * heads_per;
    const int h1 = h0 + heads_per < H ? h0 + heads_per : H;
    angles(p, L, turns, p.positions[t], sm.cs[warp], c, s);
    for (int hb = h0; hb < h1; hb += NH) {
      const int h = hb + lane / GROUP;
      const bool isq = h < p.Hq;
      const int cnt = h < h1 ? L.cnt : 0;
      const T* src = isq ? static_cast<const T*>(p.q) + t * p.ldq + (long long)h * p.d + L.e0
                         : static_cast<const T*>(p.k) + t * p.ldk +
                               (long long)(h - p.Hq) * p.d + L.e0;
      float x[8];
      load8<T, VEC>(src, cnt, x);
      if (rms || l2) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        ss = group_sum<GROUP>(ss);
        const float inv = rsqrtf(rms ? ss / (float)p.d + p.eps : ss + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= inv;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= isq ? qw[i] : kw[i];
      rotate<false>(L, c, s, sm.swap[warp], x);
      T* dst = isq ? static_cast<T*>(p.q_out) + t * p.ldqo + (long long)h * p.d + L.e0
                   : static_cast<T*>(p.k_out) + t * p.ldko + (long long)(h - p.Hq) * p.d + L.e0;
      store8<T, VEC>(dst, cnt, x);
    }
  }
}

// dw of a block: [q | k][256] partial sums.
constexpr int kWRow = 512;

template <typename T, typename TG, int GROUP, bool VEC>
__global__ void __launch_bounds__(kThreads)
qk_rope_bwd_kernel(QkRopeArgs p, int pairs, int splits, int heads_per, float* partial) {
  __shared__ Smem sm;
  __shared__ float wsum[kWarps][kWRow];
  constexpr int NH = 32 / GROUP;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const Lane L = lane_of<GROUP>(p, pairs);
  const Turns turns = load_turns(p);
  const bool rms = p.flags & GDN_QK_RMSNORM, l2 = p.flags & GDN_QK_L2NORM;
  float qw[8], kw[8], c[8], s[8], dqw[8], dkw[8];
  load8<float, false>(p.q_weight + L.e0, p.q_weight ? L.cnt : 0, qw);
  load8<float, false>(p.k_weight + L.e0, p.k_weight ? L.cnt : 0, kw);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (!p.q_weight) qw[i] = 1.f;
    if (!p.k_weight) kw[i] = 1.f;
    dqw[i] = dkw[i] = 0.f;
  }
  const int H = p.Hq + p.Hk;
  const long long items = p.tokens * splits;
  for (long long it = blockIdx.x * (long long)kWarps + warp; it < items;
       it += (long long)gridDim.x * kWarps) {
    const long long t = it / splits;
    const int h0 = (int)(it % splits) * heads_per;
    const int h1 = h0 + heads_per < H ? h0 + heads_per : H;
    angles(p, L, turns, p.positions[t], sm.cs[warp], c, s);
    for (int hb = h0; hb < h1; hb += NH) {
      const int h = hb + lane / GROUP;
      const bool isq = h < p.Hq;
      const int cnt = h < h1 ? L.cnt : 0;
      const long long hk = (long long)(h - p.Hq) * p.d + L.e0, hq = (long long)h * p.d + L.e0;
      float x[8], g[8];
      load8<T, VEC>(isq ? static_cast<const T*>(p.q) + t * p.ldq + hq
                        : static_cast<const T*>(p.k) + t * p.ldk + hk, cnt, x);
      load8<TG, VEC>(isq ? static_cast<const TG*>(p.gq) + t * p.ldgq + hq
                         : static_cast<const TG*>(p.gk) + t * p.ldgk + hk, cnt, g);
      rotate<true>(L, c, s, sm.swap[warp], g);
      const float sc = isq ? p.scale : 1.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] *= sc;
      if (rms || l2) {
        float ss = 0.f, xd = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(x[i], x[i], ss);
          xd = fmaf(x[i], g[i] * (isq ? qw[i] : kw[i]), xd);
        }
        ss = group_sum<GROUP>(ss);
        xd = group_sum<GROUP>(xd);
        const float inv = rsqrtf(rms ? ss / (float)p.d + p.eps : ss + p.eps);
        const float m = xd * inv * (rms ? 1.f / (float)p.d : 1.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = x[i] * inv;
          if (h < h1) {  // a group past the last head holds no row
            if (isq) dqw[i] = fmaf(g[i], n, dqw[i]);
            else dkw[i] = fmaf(g[i], n, dkw[i]);
          }
          g[i] = inv * fmaf(-n, m, g[i] * (isq ? qw[i] : kw[i]));
        }
      }
      store8<TG, VEC>(isq ? static_cast<TG*>(p.q_out) + t * p.ldqo + hq
                          : static_cast<TG*>(p.k_out) + t * p.ldko + hk, cnt, g);
    }
  }
  if (partial == nullptr) return;  // no weights
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = GROUP; o < 32; o <<= 1) {
      dqw[i] += __shfl_xor_sync(0xffffffffu, dqw[i], o);
      dkw[i] += __shfl_xor_sync(0xffffffffu, dkw[i], o);
    }
    if (lane < GROUP) {
      wsum[warp][L.e0 + i] = dqw[i];
      wsum[warp][256 + L.e0 + i] = dkw[i];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kWRow; e += kThreads) {
    if (e % 256 >= GROUP * 8) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += wsum[w][e];
    partial[(size_t)blockIdx.x * kWRow + e] = v;
  }
}

// The blocks' partial sums, in block order: a warp a channel.
__global__ void __launch_bounds__(kThreads)
qk_rope_sums_kernel(const float* partial, int blocks, int d, float* dqw, float* dkw) {
  const int w = blockIdx.x * kWarps + threadIdx.x / 32, lane = threadIdx.x & 31;
  const int e = w % d;
  if (w >= 2 * d) return;
  float v = 0.f;
  for (int b = lane; b < blocks; b += 32)
    v += partial[(size_t)b * kWRow + (w >= d ? 256 : 0) + e];
  v = warp_sum(v);
  if (lane == 0) {
    if (w < d) { if (dqw) dqw[e] = v; }
    else { if (dkw) dkw[e] = v; }
  }
}

bool vec_ok(const void* p, long long ld, int es) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * es)) & 15) == 0;
}

struct Plan {
  int blocks, splits, heads_per, pairs;
};
constexpr int kMaxBlocks = 148 * 4;
Plan plan_of(const QkRopeArgs& p, int group) {
  const int H = p.Hq + p.Hk, nh = 32 / group;
  const int steps = (H + nh - 1) / nh;
  // enough warps for the machine: a token's heads are split over several where there are
  // few tokens
  const long long want = (long long)kMaxBlocks * kWarps;
  long long splits = (want + p.tokens - 1) / p.tokens;
  if (splits > steps) splits = steps;
  const int per = (int)((steps + splits - 1) / splits) * nh;
  Plan q;
  q.heads_per = per;
  q.splits = (H + per - 1) / per;
  const long long blocks = (p.tokens * q.splits + kWarps - 1) / kWarps;
  q.blocks = (int)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
  q.pairs = (p.flags & GDN_ROPE_INTERLEAVED) ? kPairLane
            : (p.rot / 2) % 8 == 0           ? kPairShuffle
                                             : kPairShared;
  return q;
}
int group_of(int d) { return d <= 64 ? 8 : d <= 128 ? 16 : 32; }

template <typename T, int GROUP>
cudaError_t run_fwd(const QkRopeArgs& p, cudaStream_t s) {
  const Plan q = plan_of(p, GROUP);
  const int es = sizeof(T);
  const bool vec = p.d % 8 == 0 && vec_ok(p.q, p.ldq, es) && vec_ok(p.k, p.ldk, es) &&
                   vec_ok(p.q_out, p.ldqo, es) && vec_ok(p.k_out, p.ldko, es);
  if (vec)
    qk_rope_kernel<T, GROUP, true><<<q.blocks, kThreads, 0, s>>>(p, q.pairs, q.splits, q.heads_per);
  else
    qk_rope_kernel<T, GROUP, false><<<q.blocks, kThreads, 0, s>>>(p, q.pairs, q.splits, q.heads_per);
  return cudaGetLastError();
}
template <typename T, typename TG, int GROUP>
cudaError_t run_bwd(const QkRopeArgs& p, float* partial, cudaStream_t s) {
  const Plan q = plan_of(p, GROUP);
  const int es = sizeof(T), eg = sizeof(TG);
  const bool vec = p.d % 8 == 0 && vec_ok(p.q, p.ldq, es) && vec_ok(p.k, p.ldk, es) &&
                   vec_ok(p.q_out, p.ldqo, eg) && vec_ok(p.k_out, p.ldko, eg) &&
                   vec_ok(p.gq, p.ldgq, eg) && vec_ok(p.gk, p.ldgk, eg);
  if (p.dqw == nullptr && p.dkw == nullptr) partial = nullptr;
  if (vec)
    qk_rope_bwd_kernel<T, TG, GROUP, true>
        <<<q.blocks, kThreads, 0, s>>>(p, q.pairs, q.splits, q.heads_per, partial);
  else
    qk_rope_bwd_kernel<T, TG, GROUP, false>
        <<<q.blocks, kThreads, 0, s>>>(p, q.pairs, q.splits, q.heads_per, partial);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || partial == nullptr) return e;
  qk_rope_sums_kernel<<<(2 * p.d + kWarps - 1) / kWarps, kThreads, 0, s>>>(partial, q.blocks, p.d,
                                                                         p.dqw, p.dkw);
  return cudaGetLastError();
}
template <typename T, typename TG>
cudaError_t bwd_by_group(const QkRopeArgs& p, float* partial, cudaStream_t s) {
  switch (group_of(p.d)) {
    case 8: return run_bwd<T, TG, 8>(p, partial, s);
    case 16: return run_bwd<T, TG, 16>(p, partial, s);
    default: return run_bwd<T, TG, 32>(p, partial, s);
  }
}

}  // namespace

cudaError_t launch_qk_rope(const QkRopeArgs& p, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  const int g = group_of(p.d);
  if (p.dtype == GDN_BF16)
    return g == 8 ? run_fwd<bf16, 8>(p, s) : g == 16 ? run_fwd<bf16, 16>(p, s)
                                                      : run_fwd<bf16, 32>(p, s);
  return g == 8 ? run_fwd<float, 8>(p, s) : g == 16 ? run_fwd<float, 16>(p, s)
                                                    : run_fwd<float, 32>(p, s);
}

size_t qk_rope_bwd_workspace_bytes(long long tokens, int Hq, int Hk, int d, int flags) {
  if (!(flags & GDN_QK_RMSNORM)) return 0;
  QkRopeArgs p{};
  p.tokens = tokens; p.Hq = Hq; p.Hk = Hk; p.d = d; p.flags = flags;
  return (size_t)plan_of(p, group_of(d)).blocks * kWRow * sizeof(float);
}

cudaError_t launch_qk_rope_bwd(const QkRopeArgs& p, void* workspace, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  float* partial = static_cast<float*>(workspace);
  if (p.dtype == GDN_F32) return bwd_by_group<float, float>(p, partial, s);
  if (p.flags & GDN_GRAD_F32) return bwd_by_group<bf16, float>(p, partial, s);
  return bwd_by_group<bf16, bf16>(p, partial, s);
}

}  // namespace gdn
