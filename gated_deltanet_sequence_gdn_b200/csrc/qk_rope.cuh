// qk_rope.cuh -- norm of each head of q and k and the position rotation, one pass:
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
// 64-bit position (off by |position| 2^-65 turns: 2^-22 rad at 2^40), and its top 32 bits go
// to sincospi.
#pragma once

#include "common.cuh"
#include "linrec.cuh"
#include "linrec_math.cuh"

namespace gdn {
namespace rope {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxHalf = 128;  // rotated pairs of a head (d <= 256)

// Where a pair's partner is: a whole number of lanes away, in the same lane, or anywhere in the
// head (through shared memory).
enum Pairs { kPairShuffle = 0, kPairLane = 1, kPairShared = 2 };

// One of q and k.
struct Side {
  const void *x, *g;  // the rows; backward: the gradient at their results
  void* out;          // the results, or the gradient at the rows
  long long ldx, ldg, ldo;
  const float* weight;
  float scale;
  int H;
  int warps;  // that share a token's heads
};
struct Sides {
  Side s[2];
  int warps;   // of both, 1, 2, 4 or 8: a block takes kWarps / warps tokens at a time
  int blocks;  // of the launch
  const long long* positions;
  const float* inv_freq;
  long long tokens;
  int d, rot, pairs;  // Pairs
  float eps, unit;    // of the norm: x / sqrt(unit * sum(x^2) + eps)
  bool norm;
};

struct Smem {
  float cs[kWarps][kMaxHalf], sn[kWarps][kMaxHalf];  // of the block's tokens
  float w[2][256];                                  // the weights (times scale, forward)
  float swap[kWarps][32 * 8 + 8];                   // kPairShared: the warp's rows
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

// One turn of inv_freq as a 64-bit fraction, rounded once: inv_freq / 2 pi as an unevaluated
// sum of two doubles (1 / 2 pi is one, to 2^-108), whose whole turns drop out of the larger.
__device__ __forceinline__ unsigned long long turn_fraction(float inv_freq) {
  constexpr double kHi = 0.15915494309189534561, kLo = -9.8393383375912434e-18;
  constexpr double k64 = 18446744073709551616.0;
  const double f = fabs((double)inv_freq), hi = f * kHi;
  const double lo = fma(f, kLo, fma(f, kHi, -hi));
  const double part = (hi - floor(hi)) * k64, whole = floor(part);
  const unsigned long long turn =
      __double2ull_rz(whole) + (unsigned long long)__double2ll_rn((part - whole) + lo * k64);
  return inv_freq < 0.f ? 0 - turn : turn;
}

// What a lane knows of its 8 channels: cos and the partner's factor +-sin for each, and where
// the partners are.
struct Lane {
  int e0, cnt;  // first channel, channels inside the head
  int turned;   // of its channels, how many are rotated
  int src;      // kPairShuffle: the partner's lane
  float2 c[4], s[4];
};
template <int GROUP>
__device__ __forceinline__ void lane_begin(const Sides& p, Lane& L) {
  const int lane = threadIdx.x & 31, half = p.rot / 2;
  L.e0 = (lane % GROUP) * 8;
  L.cnt = p.d - L.e0 < 8 ? (p.d - L.e0 < 0 ? 0 : p.d - L.e0) : 8;
  L.turned = p.rot - L.e0 < 8 ? (p.rot - L.e0 < 0 ? 0 : p.rot - L.e0) : 8;
  L.src = L.e0 < half ? lane + half / 8 : L.e0 < p.rot ? lane - half / 8 : lane;
}

// Evaluates the angles of `toks` tokens from t0 on (every thread calls it); turn(i): pair i's
// turn_fraction.
template <typename Turn>
__device__ __forceinline__ void block_angles(const Sides& p, int toks, long long t0, Smem& sm,
                                             const Turn& turn) {
  const int half = p.rot / 2;
  for (int j = threadIdx.x; j < half * toks; j += kThreads) {
    const int tk = j / half, i = j - tk * half;
    if (t0 + tk >= p.tokens) break;
    const unsigned long long ph = (unsigned long long)p.positions[t0 + tk] * turn(i);
    float sn, cn;
    sincospif((float)(int)(ph >> 32) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31 half turns
    sm.cs[tk][i] = cn;
    sm.sn[tk][i] = sn;
  }
}
__device__ __forceinline__ void take8(const float* at, float2* f) {
  const float4 a = reinterpret_cast<const float4*>(at)[0], b = reinterpret_cast<const float4*>(at)[1];
  f[0] = make_float2(a.x, a.y); f[1] = make_float2(a.z, a.w);
  f[2] = make_float2(b.x, b.y); f[3] = make_float2(b.z, b.w);
}
// The lane's own of one token; back: of the opposite rotation.  The first of a pair loses its
// partner's sine, the second gains it.
template <int PAIRS>
__device__ __forceinline__ void lane_angles(const Sides& p, const float* cs, const float* sn,
                                            bool back, Lane& L) {
  const int half = p.rot / 2;
  if (PAIRS == kPairShuffle) {  // 8 consecutive pairs
    const bool lo = L.e0 < half;
    const int k = L.turned == 0 ? 0 : lo ? L.e0 : L.e0 - half;
    const float2 sign = both(lo != back ? -1.f : 1.f);
    take8(cs + k, L.c);
    take8(sn + k, L.s);
#pragma unroll
    for (int i = 0; i < 4; ++i) L.s[i] = mul2(L.s[i], sign);
  } else if (PAIRS == kPairLane) {  // 4 (what is behind the last pair is not used: rotate)
    const float sign = back ? 1.f : -1.f;
    const int k = L.turned == 0 ? 0 : L.e0 / 2;
    const float4 c = *reinterpret_cast<const float4*>(cs + k);
    const float4 s = *reinterpret_cast<const float4*>(sn + k);
    L.c[0] = both(c.x); L.c[1] = both(c.y); L.c[2] = both(c.z); L.c[3] = both(c.w);
    L.s[0] = make_float2(sign * s.x, -sign * s.x);
    L.s[1] = make_float2(sign * s.y, -sign * s.y);
    L.s[2] = make_float2(sign * s.z, -sign * s.z);
    L.s[3] = make_float2(sign * s.w, -sign * s.w);
  } else {
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = L.e0 + i;
      const bool lo = e < half;
      const int k = i < L.turned ? (lo ? e : e - half) : 0;
      c[i] = cs[k];
      s[i] = lo != back ? -sn[k] : sn[k];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      L.c[i] = make_float2(c[2 * i], c[2 * i + 1]);
      L.s[i] = make_float2(s[2 * i], s[2 * i + 1]);
    }
  }
}

// Rotates the lane's 8 values (the whole warp calls it).  A channel that is not rotated stays
// as it is, whatever its neighbours hold.
template <int PAIRS>
__device__ __forceinline__ void rotate(const Sides& p, const Lane& L, float* swap, float2* y) {
  if (p.rot == 0) return;
  float2 o[4];
  if (PAIRS == kPairShuffle) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = make_float2(__shfl_sync(0xffffffffu, y[i].x, L.src),
                         __shfl_sync(0xffffffffu, y[i].y, L.src));
  } else if (PAIRS == kPairLane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = make_float2(y[i].y, y[i].x);
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
      v[i] = i < L.turned ? swap[row + (e < half ? e + half : e - half)] : 0.f;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = make_float2(v[2 * i], v[2 * i + 1]);
  }
  // A whole head's turn needs no look at the lane, where the head fills its lanes' channels: in a
  // lane that it ends in, the angles behind the last pair are not there, and 0 (the channels
  // behind the head) times what the shared memory holds may be NaN, which the backward's sums
  // would take to the rest of the head.  kPairShuffle takes whole lanes only.
  if ((p.rot == p.d && (PAIRS == kPairShuffle || p.d % 8 == 0)) || L.turned == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = fma2(o[i], L.s[i], mul2(y[i], L.c[i]));
  } else if (PAIRS != kPairShuffle && L.turned > 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = fma2(o[i], L.s[i], mul2(y[i], L.c[i]));
      if (2 * i < L.turned) y[i].x = t.x;
      if (2 * i + 1 < L.turned) y[i].y = t.y;
    }
  }
}

// Sums over the lanes of a head, N of them at once.
template <int GROUP, int N>
__device__ __forceinline__ void group_sums(float* v) {
#pragma unroll
  for (int o = GROUP / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}
// Both weights, times the scale where `scaled`.
__device__ __forceinline__ void load_weights(const Sides& p, bool scaled, Smem& sm) {
  for (int i = threadIdx.x; i < 256; i += kThreads)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const Side& q = p.s[j];
      sm.w[j][i] = (i < p.d && q.weight ? q.weight[i] : 1.f) * (scaled ? q.scale : 1.f);
    }
}

// A warp's place: which of the block's tokens, which side, which of the side's warps.
struct Place {
  int warp, token, side, part;
};
__device__ __forceinline__ Place place_of(const Sides& p) {
  Place a;
  a.warp = threadIdx.x / 32;
  a.token = a.warp / p.warps;
  a.part = a.warp - a.token * p.warps;
  a.side = a.part >= p.s[0].warps;
  if (a.side) a.part -= p.s[0].warps;
  return a;
}

inline bool rows16(const void* p, long long ld, int es) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * es)) & 15) == 0;
}
inline int group_of(int d) { return d <= 64 ? 8 : d <= 128 ? 16 : 32; }

// How warps share a token: as many as leave each `rounds` of the u heads that it brings in
// at once, so that what a warp does once a token (its angles) stays small beside its heads; q
// and k get them as they have heads.
inline void plan_warps(Sides* p, int u, int rounds) {
  Side &q = p->s[0], &k = p->s[1];
  const int step = 32 / group_of(p->d) * u, H = q.H + k.H;
  int w = q.H > 0 && k.H > 0 ? 2 : 1;
  while (w < kWarps && w * step * rounds < H) w *= 2;
  k.warps = k.H == 0 ? 0 : (int)((2LL * w * k.H + H) / (2 * H));
  if (k.H > 0 && k.warps == 0) k.warps = 1;
  if (q.H > 0 && k.warps == w) k.warps = w - 1;
  q.warps = w - k.warps;
  p->warps = w;
  const int toks = kWarps / w;
  p->blocks = (int)((p->tokens + toks - 1) / toks);
}
inline Sides sides_of(const QkRopeArgs& p) {
  Sides s{};
  s.s[0] = Side{p.q, p.gq, p.q_out, p.ldq, p.ldgq, p.ldqo, p.q_weight, p.scale, p.Hq, 0};
  s.s[1] = Side{p.k, p.gk, p.k_out, p.ldk, p.ldgk, p.ldko, p.k_weight, 1.f, p.Hk, 0};
  s.positions = p.positions;
  s.inv_freq = p.inv_freq;
  s.tokens = p.tokens;
  s.d = p.d;
  s.rot = p.rot;
  s.pairs = (p.flags & GDN_ROPE_INTERLEAVED) ? kPairLane
            : (p.rot / 2) % 8 == 0           ? kPairShuffle
                                             : kPairShared;
  s.norm = p.flags & (GDN_QK_RMSNORM | GDN_QK_L2NORM);
  s.unit = (p.flags & GDN_QK_RMSNORM) ? 1.f / (float)p.d : 1.f;
  s.eps = p.eps;
  return s;
}
inline bool vec_ok(const Sides& p, int ex, int eg) {
  bool ok = p.d % 8 == 0;
  for (const Side& q : p.s)
    if (q.H > 0)
      ok = ok && rows16(q.x, q.ldx, ex) && rows16(q.g, q.ldg, eg) && rows16(q.out, q.ldo, eg);
  return ok;
}

// Calls f.template run<GROUP, PAIRS, VEC>() for the call's sizes.
template <typename F, int GROUP>
cudaError_t by_pairs(const Sides& p, bool vec, const F& f) {
  if (!vec) return p.pairs == kPairLane ? f.template run<GROUP, kPairLane, false>()
                                        : f.template run<GROUP, kPairShared, false>();
  return p.pairs == kPairLane      ? f.template run<GROUP, kPairLane, true>()
         : p.pairs == kPairShuffle ? f.template run<GROUP, kPairShuffle, true>()
                                   : f.template run<GROUP, kPairShared, true>();
}
template <typename F>
cudaError_t by_size(const Sides& p, bool vec, const F& f) {
  const int g = group_of(p.d);
  return g == 8 ? by_pairs<F, 8>(p, vec, f) : g == 16 ? by_pairs<F, 16>(p, vec, f)
                                                       : by_pairs<F, 32>(p, vec, f);
}

}  // namespace rope
}  // namespace gdn
