// qk_rope.cu -- norm and rotation of q and k (qk_rope.cuh), forward.
//
// What bounds it: 15.7 instructions an element against 4 bytes of bf16 (the time of 22), at 57%
// of the issue slots with 21 warps an SM, which wait for their loads between rounds of heads.
// Measured, 16 + 16 heads of 128, bf16: 8192 tokens 31 us, 4.3 TB/s; 65536 tokens 206 us, 5.2
// TB/s.  A head at a time took 77 us at 8192 tokens; four on the way 49; q and k by warps of
// the same block, the kind of pairs at compile time and the loads ahead of the angles 31.
// Eight on the way with two blocks an SM take 35, two with four blocks 36.
#include "qk_rope.cuh"

namespace gdn {
namespace {
using namespace rope;

template <typename T, int GROUP, int PAIRS, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) qk_rope_kernel(const __grid_constant__ Sides p) {
  __shared__ __align__(16) Smem sm;
  constexpr int NH = 32 / GROUP;             // heads a warp holds at once
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // of them on the way at once
  const Place a = place_of(p);
  const Side& q = p.s[a.side];
  const int H = q.H, warps = q.warps, grp = (threadIdx.x & 31) / GROUP, toks = kWarps / p.warps;
  const long long t0 = (long long)blockIdx.x * toks, t = t0 + a.token;
  Lane L;
  lane_begin<GROUP>(p, L);
  const int off = grp * p.d + L.e0;
  const T* in = static_cast<const T*>(q.x) + t * q.ldx + off;
  auto load = [&](int hb, Raw<T>* raw) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int h = hb + j * NH;
      raw[j] = load8<VEC>(in + h * p.d, t < p.tokens && h + grp < H ? L.cnt : 0);
    }
  };
  int hb = a.part * NH * U;
  Raw<T> raw[U];
  load(hb, raw);  // on the way while the angles are evaluated
  block_angles(p, toks, t0, sm, [&](int i) { return turn_fraction(p.inv_freq[i]); });
  load_weights(p, true, sm);
  __syncthreads();
  if (t >= p.tokens) return;
  lane_angles<PAIRS>(p, sm.cs[a.token], sm.sn[a.token], false, L);
  float2 w[4];
  take8(sm.w[a.side] + L.e0, w);
  T* out = static_cast<T*>(q.out) + t * q.ldo + off;
  while (true) {
    float inv[U];
    if (p.norm) {  // the sums of all of them together: their shuffles follow one another
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float2 x[4];
        raw[j].get(x);
        float2 ss = mul2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) ss = fma2(x[i], x[i], ss);
        inv[j] = ss.x + ss.y;
      }
      group_sums<GROUP, U>(inv);
#pragma unroll
      for (int j = 0; j < U; ++j) inv[j] = rsqrtf(fmaf(inv[j], p.unit, p.eps));
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int h = hb + j * NH;
      float2 x[4];
      raw[j].get(x);
      if (p.norm) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], both(inv[j]));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], w[i]);
      rotate<PAIRS>(p, L, sm.swap[a.warp], x);
      store8<VEC>(out + h * p.d, h + grp < H ? L.cnt : 0, x);
    }
    hb += warps * NH * U;
    if (hb >= H) return;
    load(hb, raw);
  }
}

template <typename T>
struct FwdRun {
  const Sides& p;
  cudaStream_t s;
  template <int GROUP, int PAIRS, bool VEC>
  cudaError_t run() const {
    qk_rope_kernel<T, GROUP, PAIRS, VEC><<<p.blocks, kThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
};
template <typename T>
cudaError_t run_fwd(const QkRopeArgs& a, cudaStream_t s) {
  Sides p = sides_of(a);
  plan_warps(&p, sizeof(T) == 2 ? 4 : 2, 2);
  return by_size(p, vec_ok(p, sizeof(T), sizeof(T)), FwdRun<T>{p, s});
}

}  // namespace

cudaError_t launch_qk_rope(const QkRopeArgs& p, cudaStream_t s) {
  return p.dtype == GDN_BF16 ? run_fwd<__nv_bfloat16>(p, s) : run_fwd<float>(p, s);
}

}  // namespace gdn
