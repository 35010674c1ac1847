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
// brings in several heads of one token at a time before it works on the first.  The angles
// of a block's tokens are evaluated once, into shared memory, and a lane keeps those of its
// channels for all the heads that its warp takes.
//
// Angles: position * inv_freq in float32 is off by 2^-24 of the angle, which is 0.01 rad
// at position 10^5.  A turn is held as a 64-bit fraction instead: phase = position *
// round(2^64 inv_freq / 2 pi) modulo 2^64 is exact but for that one rounding, for every
// 64-bit position, and its top 32 bits go to sincospi.
#include "common.cuh"
#include "linrec.cuh"
#include "linrec_math.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxHalf = 128;  // rotated pairs of a head (d <= 256)

enum Pairs { kPairShuffle = 0, kPairLane = 1, kPairShared = 2 };

// How a block's warps share its tokens.
struct Plan {
  int blocks;
  int warps;  // of a token (1, 2, 4 or 8); the block takes kWarps / warps tokens at a time
  int pairs;  // Pairs
};

struct Smem {
  float2 cs[kWarps][kMaxHalf];     // cos, sin of the block's tokens
  float w[2][256];                 // weights of q (times scale, forward) and k
  float swap[kWarps][32 * 8 + 8];  // kPairShared: the warp's rows
};

// One lane's 8 elements of a row as they come from memory.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void get(float2* f) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void set(const float2* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 q = __floats2bfloat162_rn(f[i].x, f[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&q);
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Raw<float> {
  float4 v[2];
  __device__ __forceinline__ void get(float2* f) const {
    f[0] = make_float2(v[0].x, v[0].y); f[1] = make_float2(v[0].z, v[0].w);
    f[2] = make_float2(v[1].x, v[1].y); f[3] = make_float2(v[1].z, v[1].w);
  }
  __device__ __forceinline__ void set(const float2* f) {
    v[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    v[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  }
};
// cnt of the 8 are inside the head; VEC: rows move in 16-byte pieces (all or none).
template <bool VEC, typename T>
__device__ __forceinline__ Raw<T> load8(const T* p, int cnt) {
  Raw<T> r{};
  if (VEC) {
    if (cnt > 0) r = *reinterpret_cast<const Raw<T>*>(p);
  } else {
    float2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = make_float2(2 * i < cnt ? to_f32(p[2 * i]) : 0.f,
                         2 * i + 1 < cnt ? to_f32(p[2 * i + 1]) : 0.f);
    r.set(f);
  }
  return r;
}
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, int cnt, const float2* f) {
  if (VEC) {
    Raw<T> r;
    r.set(f);
    if (cnt > 0) *reinterpret_cast<Raw<T>*>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * i < cnt) p[2 * i] = from_f32<T>(f[i].x);
      if (2 * i + 1 < cnt) p[2 * i + 1] = from_f32<T>(f[i].y);
    }
  }
}

// One turn of inv_freq as a 64-bit fraction.
__device__ __forceinline__ unsigned long long turn_fraction(float inv_freq) {
  const double t = (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}

// What a lane knows of its 8 channels: cos and +-sin for each (1 and 0 where it is not
// rotated), and where the partners are.
struct Lane {
  int e0, cnt;  // first channel, channels inside the head
  int src;      // kPairShuffle: the partner's lane
  bool turned;  // kPairShuffle, kPairLane: the lane's channels are rotated
  float2 c[4], s[4];
};
template <int GROUP>
__device__ __forceinline__ void lane_begin(const QkRopeArgs& p, Lane& L) {
  const int lane = threadIdx.x & 31, half = p.rot / 2;
  L.e0 = (lane % GROUP) * 8;
  L.cnt = p.d - L.e0 < 8 ? (p.d - L.e0 < 0 ? 0 : p.d - L.e0) : 8;
  L.src = L.e0 < half ? lane + half / 8 : L.e0 < p.rot ? lane - half / 8 : lane;
}

// Evaluates the angles of the block's tokens from t0 on (every thread calls it).
__device__ __forceinline__ void block_angles(const QkRopeArgs& p, const Plan& plan, long long t0,
                                             Smem& sm) {
  const int half = p.rot / 2, toks = kWarps / plan.warps;
  for (int j = threadIdx.x; j < half * toks; j += kThreads) {
    const int tk = j / half, i = j - tk * half;
    if (t0 + tk >= p.tokens) break;
    const unsigned long long ph =
        (unsigned long long)p.positions[t0 + tk] * turn_fraction(p.inv_freq[i]);
    float sn, cn;
    sincospif((float)(int)(ph >> 32) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31 half turns
    sm.cs[tk][i] = make_float2(cn, sn);
  }
}
// The lane's own of one token; back: of the opposite rotation.
__device__ __forceinline__ void lane_angles(const QkRopeArgs& p, const Plan& plan,
                                            const float2* cs, bool back, Lane& L) {
  const int half = p.rot / 2;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = L.e0 + i;
    const int k = plan.pairs == kPairLane ? e / 2 : e < half ? e : e - half;
    const float2 v = e < p.rot ? cs[k] : make_float2(1.f, 0.f);
    // the first of a pair loses its partner's sine, the second gains it
    const bool lo = plan.pairs == kPairLane ? (e & 1) == 0 : e < half;
    c[i] = v.x;
    s[i] = lo != back ? -v.y : v.y;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    L.c[i] = make_float2(c[2 * i], c[2 * i + 1]);
    L.s[i] = make_float2(s[2 * i], s[2 * i + 1]);
  }
  L.turned = L.e0 < p.rot;
}

// Rotates the lane's 8 values (the whole warp calls it).
__device__ __forceinline__ void rotate(const QkRopeArgs& p, const Plan& plan, const Lane& L,
                                       float* swap, float2* y) {
  if (p.rot == 0) return;
  float2 o[4];
  if (plan.pairs == kPairLane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = make_float2(y[i].y, y[i].x);
  } else if (plan.pairs == kPairShuffle) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = make_float2(__shfl_sync(0xffffffffu, y[i].x, L.src),
                         __shfl_sync(0xffffffffu, y[i].y, L.src));
  } else {
    const int lane = threadIdx.x & 31, half = p.rot / 2;
    const int row = lane * 8 - L.e0;  // the head's first value
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(swap + lane * 8 + 2 * i) = y[i];
    __syncwarp();
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = L.e0 + i;
      v[i] = e < p.rot ? swap[row + (e < half ? e + half : e - half)] : 0.f;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = make_float2(v[2 * i], v[2 * i + 1]);
  }
  // a channel that is not rotated stays as it is, whatever its neighbour holds
  const int whole = (L.e0 + 8 <= p.rot) ? 8 : p.rot - L.e0;
  if (whole == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = fma2(o[i], L.s[i], mul2(y[i], L.c[i]));
  } else if (L.turned) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = fma2(o[i], L.s[i], mul2(y[i], L.c[i]));
      if (2 * i < whole) y[i].x = t.x;
      if (2 * i + 1 < whole) y[i].y = t.y;
    }
  }
}

template <int GROUP>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = GROUP / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void load_weights(const QkRopeArgs& p, float qscale, Smem& sm) {
  for (int i = threadIdx.x; i < 256; i += kThreads) {
    const bool in = i < p.d;
    sm.w[0][i] = (in && p.q_weight ? p.q_weight[i] : 1.f) * qscale;
    sm.w[1][i] = in && p.k_weight ? p.k_weight[i] : 1.f;
  }
}
__device__ __forceinline__ void lane_weights(const float* w, float2* f) {
  const float4 a = reinterpret_cast<const float4*>(w)[0], b = reinterpret_cast<const float4*>(w)[1];
  f[0] = make_float2(a.x, a.y); f[1] = make_float2(a.z, a.w);
  f[2] = make_float2(b.x, b.y); f[3] = make_float2(b.z, b.w);
}

template <typename T, int GROUP, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) qk_rope_kernel(QkRopeArgs p, Plan plan) {
  __shared__ Smem sm;
  constexpr int NH = 32 / GROUP;           // heads a warp holds at once
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // of them on the way at once
  const int warp = threadIdx.x / 32, grp = (threadIdx.x & 31) / GROUP;
  const int toks = kWarps / plan.warps, tk = warp / plan.warps, part = warp % plan.warps;
  const long long t0 = (long long)blockIdx.x * toks, t = t0 + tk;
  const bool rms = p.flags & GDN_QK_RMSNORM, norm = p.flags & (GDN_QK_RMSNORM | GDN_QK_L2NORM);
  const float unit = rms ? 1.f / (float)p.d : 1.f;
  const int H = p.Hq + p.Hk;
  Lane L;
  lane_begin<GROUP>(p, L);
  block_angles(p, plan, t0, sm);
  load_weights(p, p.scale, sm);
  __syncthreads();
  if (t >= p.tokens) return;
  lane_angles(p, plan, sm.cs[tk], false, L);
  const T* qrow = static_cast<const T*>(p.q) + t * p.ldq + L.e0;
  const T* krow = static_cast<const T*>(p.k) + t * p.ldk + L.e0;
  T* qout = static_cast<T*>(p.q_out) + t * p.ldqo + L.e0;
  T* kout = static_cast<T*>(p.k_out) + t * p.ldko + L.e0;
  for (int hb = part * NH * U; hb < H; hb += plan.warps * NH * U) {
    Raw<T> raw[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int h = hb + j * NH + grp, cnt = h < H ? L.cnt : 0;
      raw[j] = load8<VEC>(h < p.Hq ? qrow + h * p.d : krow + (h - p.Hq) * p.d, cnt);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (hb + j * NH >= H) break;
      const int h = hb + j * NH + grp, cnt = h < H ? L.cnt : 0;
      float2 x[4], w[4];
      raw[j].get(x);
      lane_weights(sm.w[h < p.Hq ? 0 : 1] + L.e0, w);
      if (norm) {
        float2 ss = mul2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) ss = fma2(x[i], x[i], ss);
        const float inv = rsqrtf(fmaf(group_sum<GROUP>(ss.x + ss.y), unit, p.eps));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], both(inv));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], w[i]);
      rotate(p, plan, L, sm.swap[warp], x);
      store8<VEC>(h < p.Hq ? qout + h * p.d : kout + (h - p.Hq) * p.d, cnt, x);
    }
  }
}

// dw of a block: [q | k][256] partial sums.
constexpr int kWRow = 512;

template <typename T, typename TG, int GROUP, bool VEC>
__global__ void __launch_bounds__(kThreads, 2)
qk_rope_bwd_kernel(QkRopeArgs p, Plan plan, float* partial) {
  __shared__ Smem sm;
  __shared__ float wsum[kWarps][kWRow];
  constexpr int NH = 32 / GROUP;
  constexpr int U = 2;
  const int warp = threadIdx.x / 32, grp = (threadIdx.x & 31) / GROUP;
  const int toks = kWarps / plan.warps, tk = warp / plan.warps, part = warp % plan.warps;
  const bool rms = p.flags & GDN_QK_RMSNORM, norm = p.flags & (GDN_QK_RMSNORM | GDN_QK_L2NORM);
  const float unit = rms ? 1.f / (float)p.d : 1.f;
  const int H = p.Hq + p.Hk;
  Lane L;
  lane_begin<GROUP>(p, L);
  load_weights(p, 1.f, sm);
  float2 dqw[4], dkw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dqw[i] = dkw[i] = both(0.f);
  for (long long t0 = (long long)blockIdx.x * toks; t0 < p.tokens;
       t0 += (long long)gridDim.x * toks) {
    __syncthreads();  // the last tokens' angles are read
    block_angles(p, plan, t0, sm);
    __syncthreads();
    const long long t = t0 + tk;
    if (t >= p.tokens) continue;
    lane_angles(p, plan, sm.cs[tk], true, L);
    const T* qrow = static_cast<const T*>(p.q) + t * p.ldq + L.e0;
    const T* krow = static_cast<const T*>(p.k) + t * p.ldk + L.e0;
    const TG* gqrow = static_cast<const TG*>(p.gq) + t * p.ldgq + L.e0;
    const TG* gkrow = static_cast<const TG*>(p.gk) + t * p.ldgk + L.e0;
    TG* qout = static_cast<TG*>(p.q_out) + t * p.ldqo + L.e0;
    TG* kout = static_cast<TG*>(p.k_out) + t * p.ldko + L.e0;
    for (int hb = part * NH * U; hb < H; hb += plan.warps * NH * U) {
      Raw<T> rx[U];
      Raw<TG> rg[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int h = hb + j * NH + grp, cnt = h < H ? L.cnt : 0;
        const bool isq = h < p.Hq;
        const int off = (isq ? h : h - p.Hq) * p.d;
        rg[j] = load8<VEC>((isq ? gqrow : gkrow) + off, cnt);
        if (norm) rx[j] = load8<VEC>((isq ? qrow : krow) + off, cnt);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (hb + j * NH >= H) break;
        const int h = hb + j * NH + grp, cnt = h < H ? L.cnt : 0;
        const bool isq = h < p.Hq;
        float2 g[4];
        rg[j].get(g);
        rotate(p, plan, L, sm.swap[warp], g);
        const float2 sc = both(isq ? p.scale : 1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = mul2(g[i], sc);
        if (norm) {
          float2 x[4], w[4];
          rx[j].get(x);
          lane_weights(sm.w[isq ? 0 : 1] + L.e0, w);
          float2 ss = mul2(x[0], x[0]), xd = mul2(x[0], mul2(g[0], w[0]));
#pragma unroll
          for (int i = 1; i < 4; ++i) {
            ss = fma2(x[i], x[i], ss);
            xd = fma2(x[i], mul2(g[i], w[i]), xd);
          }
          const float inv = rsqrtf(fmaf(group_sum<GROUP>(ss.x + ss.y), unit, p.eps));
          const float m = group_sum<GROUP>(xd.x + xd.y) * inv * unit;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 n = mul2(x[i], both(inv));
            if (h < H && partial) {  // a group past the last head holds no row
              if (isq) dqw[i] = fma2(g[i], n, dqw[i]);
              else dkw[i] = fma2(g[i], n, dkw[i]);
            }
            g[i] = mul2(fma2(n, both(-m), mul2(g[i], w[i])), both(inv));
          }
        }
        store8<VEC>((isq ? qout : kout) + (isq ? h : h - p.Hq) * p.d, cnt, g);
      }
    }
  }
  if (partial == nullptr) return;  // no weights
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = GROUP; o < 32; o <<= 1) {
      dqw[i].x += __shfl_xor_sync(0xffffffffu, dqw[i].x, o);
      dqw[i].y += __shfl_xor_sync(0xffffffffu, dqw[i].y, o);
      dkw[i].x += __shfl_xor_sync(0xffffffffu, dkw[i].x, o);
      dkw[i].y += __shfl_xor_sync(0xffffffffu, dkw[i].y, o);
    }
    if (lane < GROUP) {
      *reinterpret_cast<float2*>(&wsum[warp][L.e0 + 2 * i]) = dqw[i];
      *reinterpret_cast<float2*>(&wsum[warp][256 + L.e0 + 2 * i]) = dkw[i];
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

bool rows16(const void* p, long long ld, int es) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * es)) & 15) == 0;
}
int group_of(int d) { return d <= 64 ? 8 : d <= 128 ? 16 : 32; }

constexpr int kMostBlocks = 148 * 2;  // of the backward, whose blocks loop over the tokens
// u: heads that a warp brings in at once.
Plan plan_of(const QkRopeArgs& p, int u) {
  const int step = 32 / group_of(p.d) * u, H = p.Hq + p.Hk;
  Plan q;
  q.warps = 1;
  while (q.warps < kWarps && q.warps * step < H) q.warps *= 2;
  const int toks = kWarps / q.warps;
  const long long blocks = (p.tokens + toks - 1) / toks;
  q.blocks = (int)(blocks < 0x7fffffff ? blocks : 0x7fffffff);
  q.pairs = (p.flags & GDN_ROPE_INTERLEAVED) ? kPairLane
            : (p.rot / 2) % 8 == 0           ? kPairShuffle
                                             : kPairShared;
  return q;
}
int bwd_blocks(const Plan& q) { return q.blocks < kMostBlocks ? q.blocks : kMostBlocks; }

template <typename T, int GROUP>
cudaError_t run_fwd(const QkRopeArgs& p, cudaStream_t s) {
  const Plan q = plan_of(p, sizeof(T) == 2 ? 4 : 2);
  const int es = sizeof(T);
  if (p.d % 8 == 0 && rows16(p.q, p.ldq, es) && rows16(p.k, p.ldk, es) &&
      rows16(p.q_out, p.ldqo, es) && rows16(p.k_out, p.ldko, es))
    qk_rope_kernel<T, GROUP, true><<<q.blocks, kThreads, 0, s>>>(p, q);
  else
    qk_rope_kernel<T, GROUP, false><<<q.blocks, kThreads, 0, s>>>(p, q);
  return cudaGetLastError();
}
template <typename T, typename TG, int GROUP>
cudaError_t run_bwd(const QkRopeArgs& p, float* partial, cudaStream_t s) {
  const Plan q = plan_of(p, 2);
  const int es = sizeof(T), eg = sizeof(TG), blocks = bwd_blocks(q);
  if (p.dqw == nullptr && p.dkw == nullptr) partial = nullptr;
  if (p.d % 8 == 0 && rows16(p.q, p.ldq, es) && rows16(p.k, p.ldk, es) &&
      rows16(p.q_out, p.ldqo, eg) && rows16(p.k_out, p.ldko, eg) && rows16(p.gq, p.ldgq, eg) &&
      rows16(p.gk, p.ldgk, eg))
    qk_rope_bwd_kernel<T, TG, GROUP, true><<<blocks, kThreads, 0, s>>>(p, q, partial);
  else
    qk_rope_bwd_kernel<T, TG, GROUP, false><<<blocks, kThreads, 0, s>>>(p, q, partial);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || partial == nullptr) return e;
  qk_rope_sums_kernel<<<(2 * p.d + kWarps - 1) / kWarps, kThreads, 0, s>>>(partial, blocks, p.d,
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
  return (size_t)bwd_blocks(plan_of(p, 2)) * kWRow * sizeof(float);
}

cudaError_t launch_qk_rope_bwd(const QkRopeArgs& p, void* workspace, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  float* partial = static_cast<float*>(workspace);
  if (p.dtype == GDN_F32) return bwd_by_group<float, float>(p, partial, s);
  if (p.flags & GDN_GRAD_F32) return bwd_by_group<bf16, float>(p, partial, s);
  return bwd_by_group<bf16, bf16>(p, partial, s);
}

}  // namespace gdn
