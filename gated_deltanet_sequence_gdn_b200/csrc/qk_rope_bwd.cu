// qk_rope_bwd.cu -- norm and rotation of q and k (qk_rope.cuh), backward.  With n the
// normalised row and inv its factor:
//   dy = scale R^T dout, dw = sum dy n, dn = dy w, dx = inv (dn - n <n, dn>)
// (the product's mean with the RMS norm).
//
// What bounds it: 25 instructions an element against 6 bytes of bf16 (the time of 33), at 55% of
// the issue slots with the 15 warps an SM that 123 registers leave.  Measured, 16 + 16 heads of
// 128, bf16, with the launch that joins the weights' gradients: 8192 tokens 51 us, 3.9 TB/s;
// 65536 tokens 328 us, 4.9 TB/s.  Three blocks an SM spill (69 against 61 us at the time).
#include "qk_rope.cuh"

namespace gdn {
namespace {
using namespace rope;

// Writes partial[block][q, k][256], the block's sums for dw (NULL: no weights).
template <typename T, typename TG, int GROUP, int PAIRS, bool VEC>
__global__ void __launch_bounds__(kThreads, 2)
qk_rope_bwd_kernel(const __grid_constant__ Sides p, float* partial) {
  __shared__ __align__(16) Smem sm;
  __shared__ float wsum[kWarps][256];
  __shared__ unsigned long long turns[kMaxHalf];  // formed once: the block takes many tokens
  constexpr int NH = 32 / GROUP;
  constexpr int U = 2;
  const Place a = place_of(p);
  const Side& q = p.s[a.side];
  const int H = q.H, warps = q.warps, toks = kWarps / p.warps;
  const int warp = a.warp, lane = threadIdx.x & 31, grp = lane / GROUP;
  Lane L;
  lane_begin<GROUP>(p, L);
  load_weights(p, false, sm);
  for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) turns[i] = turn_fraction(p.inv_freq[i]);
  const int off = grp * p.d + L.e0;
  float2 dw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dw[i] = both(0.f);
  for (long long t0 = (long long)blockIdx.x * toks; t0 < p.tokens;
       t0 += (long long)gridDim.x * toks) {
    const long long t = t0 + a.token;
    const T* in = static_cast<const T*>(q.x) + t * q.ldx + off;
    const TG* gin = static_cast<const TG*>(q.g) + t * q.ldg + off;
    TG* out = static_cast<TG*>(q.out) + t * q.ldo + off;
    auto load = [&](int hb, Raw<T>* rx, Raw<TG>* rg) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int h = hb + j * NH, cnt = t < p.tokens && h + grp < H ? L.cnt : 0;
        rg[j] = load8<VEC>(gin + h * p.d, cnt);
        if (p.norm) rx[j] = load8<VEC>(in + h * p.d, cnt);
      }
    };
    int hb = a.part * NH * U;
    Raw<T> rx[U];
    Raw<TG> rg[U];
    load(hb, rx, rg);  // on the way while the angles are evaluated
    __syncthreads();   // the turns are there, the last tokens' angles read
    block_angles(p, toks, t0, sm, [&](int i) { return turns[i]; });
    __syncthreads();
    if (t >= p.tokens) continue;
    lane_angles<PAIRS>(p, sm.cs[a.token], sm.sn[a.token], true, L);
    while (hb < H) {
      const int next = hb + warps * NH * U;
      Raw<T> mx[U];
      Raw<TG> mg[U];
      if (next < H) load(next, mx, mg);
      float2 g[U][4];
      float sums[2 * U];  // of x^2, and of x dn
#pragma unroll
      for (int j = 0; j < U; ++j) {
        rg[j].get(g[j]);
        rotate<PAIRS>(p, L, sm.swap[warp], g[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[j][i] = mul2(g[j][i], both(q.scale));
        if (p.norm) {
          float2 x[4], w[4], ss = both(0.f), xd = both(0.f);
          rx[j].get(x);
          take8(sm.w[a.side] + L.e0, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ss = fma2(x[i], x[i], ss);
            xd = fma2(x[i], mul2(g[j][i], w[i]), xd);
          }
          sums[2 * j] = ss.x + ss.y;
          sums[2 * j + 1] = xd.x + xd.y;
        }
      }
      if (p.norm) group_sums<GROUP, 2 * U>(sums);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int h = hb + j * NH;
        const bool live = h + grp < H;  // a group past the last head holds no row
        if (p.norm) {
          float2 x[4], w[4];
          rx[j].get(x);
          take8(sm.w[a.side] + L.e0, w);
          const float inv = rsqrtf(fmaf(sums[2 * j], p.unit, p.eps));
          const float2 m = both(-sums[2 * j + 1] * inv * p.unit), iv = both(inv);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 n = mul2(x[i], iv);
            if (live) dw[i] = fma2(g[j][i], n, dw[i]);
            g[j][i] = mul2(fma2(n, m, mul2(g[j][i], w[i])), iv);
          }
        }
        store8<VEC>(out + h * p.d, live ? L.cnt : 0, g[j]);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        rx[j] = mx[j];
        rg[j] = mg[j];
      }
      hb = next;
    }
  }
  if (partial == nullptr) return;  // no weights
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = GROUP; o < 32; o <<= 1) {
      dw[i].x += __shfl_xor_sync(0xffffffffu, dw[i].x, o);
      dw[i].y += __shfl_xor_sync(0xffffffffu, dw[i].y, o);
    }
    if (lane < GROUP) *reinterpret_cast<float2*>(&wsum[warp][L.e0 + 2 * i]) = dw[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * 256; e += kThreads) {
    const int side = e / 256, c = e % 256;
    if (c >= GROUP * 8) continue;
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w)  // each warp holds one side's
      if ((w % p.warps >= p.s[0].warps) == side) v += wsum[w][c];
    partial[((size_t)blockIdx.x * 2 + side) * 256 + c] = v;
  }
}

// The blocks' partial sums, in block order: a warp a channel.
__global__ void __launch_bounds__(kThreads)
qk_rope_sums_kernel(const float* partial, int blocks, int d, float* dqw, float* dkw) {
  const int w = blockIdx.x * kWarps + threadIdx.x / 32, lane = threadIdx.x & 31;
  wait_for_launch();
  if (w >= 2 * d) return;
  const int side = w >= d, e = w - side * d;
  float* to = side ? dkw : dqw;
  if (to == nullptr) return;
  float v = 0.f;
  for (int b = lane; b < blocks; b += 32) v += partial[((size_t)b * 2 + side) * 256 + e];
  v = warp_sum(v);
  if (lane == 0) to[e] = v;
}

// The backward's blocks loop over the tokens (they keep their share of the weights'
// gradients): two on each of the 148 multiprocessors of the chip that this is built for.  The
// workspace's size goes by them, and is asked for without a device.
constexpr int kBwdBlocks = 148 * 2;
void plan_bwd(Sides* p) {
  plan_warps(p, 2, 4);
  if (p->blocks > kBwdBlocks) p->blocks = kBwdBlocks;
}
template <typename T, typename TG>
struct BwdRun {
  const Sides& p;
  float* partial;
  cudaStream_t s;
  template <int GROUP, int PAIRS, bool VEC>
  cudaError_t run() const {
    qk_rope_bwd_kernel<T, TG, GROUP, PAIRS, VEC>
        <<<p.blocks, kThreads, 0, s>>>(p, partial);
    return cudaGetLastError();
  }
};
template <typename T, typename TG>
cudaError_t run_bwd(const QkRopeArgs& a, float* partial, cudaStream_t s) {
  Sides p = sides_of(a);
  plan_bwd(&p);
  if (a.dqw == nullptr && a.dkw == nullptr) partial = nullptr;
  cudaError_t e =
      by_size(p, vec_ok(p, sizeof(T), sizeof(TG)), BwdRun<T, TG>{p, partial, s});
  if (e != cudaSuccess || partial == nullptr) return e;
  return launch_after(qk_rope_sums_kernel, dim3((2 * p.d + kWarps - 1) / kWarps), dim3(kThreads),
                      s, partial, p.blocks, p.d, a.dqw, a.dkw);
}

}  // namespace

size_t qk_rope_bwd_workspace_bytes(long long tokens, int Hq, int Hk, int d, int flags) {
  if (!(flags & GDN_QK_RMSNORM)) return 0;
  Sides p{};
  p.tokens = tokens;
  p.d = d;
  p.s[0].H = Hq;
  p.s[1].H = Hk;
  plan_bwd(&p);
  return (size_t)p.blocks * 2 * 256 * sizeof(float);
}

cudaError_t launch_qk_rope_bwd(const QkRopeArgs& p, void* workspace, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  float* partial = static_cast<float*>(workspace);
  if (p.dtype == GDN_F32) return run_bwd<float, float>(p, partial, s);
  if (p.flags & GDN_GRAD_F32) return run_bwd<bf16, float>(p, partial, s);
  return run_bwd<bf16, bf16>(p, partial, s);
}

}  // namespace gdn
