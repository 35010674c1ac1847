// linrec_bwd.cu -- the backward of the gated linear recurrence.  With c the gradient that
// arrives at a state from later tokens,
//   lambda_t = dh_t + c_t,  c_{t-1} = alpha_t lambda_t,
//   dx = lambda f beta,  dbeta = lambda f x,  dg = alpha lambda h_{t-1} + lambda beta x f'(g),
// c runs over the tiles from the last to the first as the forward's state does from the
// first to the last (linrec_chain.cuh).  The states h_{t-1} of a tile are recomputed in
// float32 from the state before it, which the forward kept.
#include "linrec_launch.cuh"

namespace gdn {
namespace {

template <typename TX, typename TG, typename TD>
struct BwdStage {
  alignas(16) TX x[kTileT * kTileC];
  alignas(16) TG a[kTileT * kTileC];
  alignas(16) TG b[kTileT * kTileC];
  alignas(16) TD dh[kTileT * kTileC];
};
template <typename TX, typename TG, typename TD>
struct BwdSmem {
  BwdStage<TX, TG, TD> stage[2];
  float4 fold[kWorkWarps][32];   // (A, H) of each warp's tokens, forward
  float2 back[kWorkWarps][32];   // R: c_out = A c_in + R
  float4 sums[kWorkWarps][32];   // of dg g and dz
  float2 in[32];                 // the gradient that enters the tile
  Tile tile[3];
  int more[3];
};

template <typename TX, typename TG, bool GIVEN, int SCALE, typename TD, typename TDG>
__global__ void __launch_bounds__(kLinrecThreads)
linrec_bwd_kernel(LinrecArgs p, Chain ch, int vec, const float* states, float2* sums) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<BwdSmem<TX, TG, TD>*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const bool work = warp < kWorkWarps;
  if (threadIdx.x == kWorkThreads) {
    next_tile<true>(ch, sm, 0);
    next_tile<true>(ch, sm, 1);
  }
  __syncthreads();
  auto load = [&](int k) {
    if (sm.more[k % 3]) {
      const Tile& t = sm.tile[k % 3];
      BwdStage<TX, TG, TD>& st = sm.stage[k & 1];
      load_tile(st.x, p.x, p.ldx, t, p.D, vec & 1);
      load_tile(st.a, p.a, p.lda, t, p.D, vec & 2);
      if (p.b) load_tile(st.b, p.b, p.ldb, t, p.D, vec & 4);
      load_tile(st.dh, p.dh, p.lddh, t, p.D, vec & 8);
    }
    cp_async_commit();
  };
  if (work) load(0);
  GateConst k0{0.f, 0.f}, k1{0.f, 0.f};
  int c0 = -1;
  for (int k = 0;; ++k) {
    cp_async_wait<0>();
    __syncthreads();
    if (!sm.more[k % 3]) return;
    const Tile t = sm.tile[k % 3];
    const int c = t.c0 + 2 * lane, first = warp * kPer;
    float al[kPer][2], be[kPer][2], f[kPer][2];
    float2 hs = make_float2(0.f, 0.f);
    const BwdStage<TX, TG, TD>& st = sm.stage[k & 1];
    if (work) {
      load(k + 1);
      hs = read2(states + (long long)t.chunk * p.D, c, p.D);
      if (!GIVEN && c0 != t.c0) {
        c0 = t.c0;
        if (c < p.D) k0 = gate_const(p.A_log, p.dt_bias, c);
        if (c + 1 < p.D) k1 = gate_const(p.A_log, p.dt_bias, c + 1);
      }
      float A0 = 1.f, A1 = 1.f, H0 = 0.f, H1 = 0.f, R0 = 0.f, R1 = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = (first + i) * kTileC + 2 * lane;
        const float2 av = get2(st.a + at), xv = get2(st.x + at);
        const float g0 = log_decay<GIVEN>(av.x, k0), g1 = log_decay<GIVEN>(av.y, k1);
        al[i][0] = ex2_f(g0 * kLog2e);
        al[i][1] = ex2_f(g1 * kLog2e);
        f[i][0] = input_scale<SCALE>(g0);
        f[i][1] = input_scale<SCALE>(g1);
        be[i][0] = be[i][1] = 1.f;
        if (p.b) {
          const float2 bv = get2(st.b + at);
          be[i][0] = write_gate<GIVEN>(bv.x);
          be[i][1] = write_gate<GIVEN>(bv.y);
        }
        if (first + i >= t.n) al[i][0] = al[i][1] = 1.f;  // behind the sequence (x, dh are 0)
        H0 = fmaf(al[i][0], H0, xv.x * f[i][0] * be[i][0]);
        H1 = fmaf(al[i][1], H1, xv.y * f[i][1] * be[i][1]);
        A0 *= al[i][0];
        A1 *= al[i][1];
      }
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i) {
        const float2 d = get2(st.dh + (first + i) * kTileC + 2 * lane);
        R0 = al[i][0] * (d.x + R0);
        R1 = al[i][1] * (d.y + R1);
      }
      sm.fold[warp][lane] = make_float4(A0, H0, A1, H1);
      sm.back[warp][lane] = make_float2(R0, R1);
    } else if (lane == 0) {
      next_tile<true>(ch, sm, k + 2);
    }
    __syncthreads();
    float4 ex = make_float4(1.f, 0.f, 1.f, 0.f);  // c through the tile's later tokens
    if (work) {
      for (int w = 0; w < warp; ++w) {
        const float4 q = sm.fold[w][lane];
        hs.x = fmaf(q.x, hs.x, q.y);
        hs.y = fmaf(q.z, hs.y, q.w);
      }
      for (int w = kWorkWarps - 1; w > warp; --w) {
        const float4 q = sm.fold[w][lane];
        const float2 r = sm.back[w][lane];
        ex.y = fmaf(q.x, ex.y, r.x);
        ex.w = fmaf(q.z, ex.w, r.y);
        ex.x *= q.x;
        ex.z *= q.z;
      }
    } else {
      float4 own = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
      for (int w = kWorkWarps - 1; w >= 0; --w) {
        const float4 q = sm.fold[w][lane];
        const float2 r = sm.back[w][lane];
        own.y = fmaf(q.x, own.y, r.x);
        own.w = fmaf(q.z, own.w, r.y);
        own.x *= q.x;
        own.z *= q.z;
      }
      const float2 in = chain_in<-1>(ch, t, own, p.dht ? p.dht + (long long)t.row * p.D : nullptr);
      sm.in[lane] = in;
      const float2 out = make_float2(fmaf(own.x, in.x, own.y), fmaf(own.z, in.y, own.w));
      if (t.before > 0) chain_out<-1>(ch, t, out);
      else if (p.dh0) write2(p.dh0 + (long long)t.row * p.D, c, p.D, out);
    }
    __syncthreads();
    if (work) {
      float hp[kPer][2];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float2 xv = get2(st.x + (first + i) * kTileC + 2 * lane);
        hp[i][0] = hs.x;
        hp[i][1] = hs.y;
        hs.x = fmaf(al[i][0], hs.x, xv.x * f[i][0] * be[i][0]);
        hs.y = fmaf(al[i][1], hs.y, xv.y * f[i][1] * be[i][1]);
      }
      const float2 in = sm.in[lane];
      float cc[2] = {fmaf(ex.x, in.x, ex.y), fmaf(ex.z, in.y, ex.w)};
      float sA[2] = {0.f, 0.f}, sb[2] = {0.f, 0.f};
      const int cols = p.D - c < 2 ? p.D - c : 2;
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i) {
        const int at = (first + i) * kTileC + 2 * lane;
        const float2 x2 = get2(st.x + at), a2 = get2(st.a + at), d2 = get2(st.dh + at);
        const float xv[2] = {x2.x, x2.y}, av[2] = {a2.x, a2.y}, dv[2] = {d2.x, d2.y};
        float bv[2] = {0.f, 0.f};
        if (p.b) {
          const float2 b2 = get2(st.b + at);
          bv[0] = b2.x;
          bv[1] = b2.y;
        }
        float dx[2], da[2], db[2];
        const bool live = first + i < t.n;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const GateConst& kc = j ? k1 : k0;
          const float lam = dv[j] + cc[j];
          cc[j] = al[i][j] * lam;
          const float lx = lam * xv[j];
          float dg = cc[j] * hp[i][j];
          if (SCALE != kScaleNone)
            dg = fmaf(lx * be[i][j], input_scale_slope<SCALE>(al[i][j], f[i][j]), dg);
          dx[j] = lam * f[i][j] * be[i][j];
          db[j] = lx * f[i][j];
          if (!GIVEN) db[j] *= be[i][j] * sigmoid_sfu(-bv[j]);
          da[j] = dg;
          if (!GIVEN) {
            da[j] = dg * kc.neg_A * sigmoid_sfu(av[j] + kc.bias);
            if (live) {
              const float g = log_decay<false>(av[j], kc);
              sb[j] += da[j];
              sA[j] += dg == 0.f ? 0.f : dg * g;  // g = -inf where alpha = 0
            }
          }
        }
        if (live) {
          const long long r = t.tok + first + i;
          put2(static_cast<TD*>(p.dx) + r * p.lddx + c, dx[0], dx[1], cols, vec & 16);
          put2(static_cast<TDG*>(p.da) + r * p.ldda + c, da[0], da[1], cols, vec & 32);
          if (p.b) put2(static_cast<TDG*>(p.db) + r * p.lddb + c, db[0], db[1], cols, vec & 64);
        }
      }
      if (!GIVEN) sm.sums[warp][lane] = make_float4(sA[0], sb[0], sA[1], sb[1]);
    }
    if (!GIVEN) {
      __syncthreads();
      if (!work) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWorkWarps; ++w) {
          const float4 q = sm.sums[w][lane];
          v.x += q.x; v.y += q.y; v.z += q.z; v.w += q.w;
        }
        float2* row = sums + (long long)t.chunk * p.D;
        if (c < p.D) row[c] = make_float2(v.x, v.y);
        if (c + 1 < p.D) row[c + 1] = make_float2(v.z, v.w);
      }
    }
  }
}

// dA_log and ddt_bias: the chunks' sums of a channel, in a fixed order (32 rows of threads,
// each every 32nd chunk), in 64 bits.
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows)
linrec_sums_kernel(const float2* sums, long long chunks, int D, float* dA_log, float* ddt_bias) {
  __shared__ double2 part[kSumRows][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  double A = 0.0, b = 0.0;
  if (c < D)
    for (long long r = threadIdx.y; r < chunks; r += kSumRows) {
      const float2 v = sums[r * D + c];
      A += v.x;
      b += v.y;
    }
  part[threadIdx.y][threadIdx.x] = make_double2(A, b);
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    for (int r = 1; r < kSumRows; ++r) {
      A += part[r][threadIdx.x].x;
      b += part[r][threadIdx.x].y;
    }
    dA_log[c] = (float)A;
    ddt_bias[c] = (float)b;
  }
}

struct BwdRun {
  const LinrecArgs& p;
  const Chain& ch;
  const float* states;
  float2* sums;
  cudaStream_t s;
  template <typename TX, typename TG, bool GIVEN, int SCALE, bool WIDE>
  cudaError_t run() const {
    using TD = typename Wide<TX, WIDE>::type;
    using TDG = typename Wide<TD, GIVEN>::type;
    const int vec = rows16(p.x, p.ldx, sizeof(TX)) | rows16(p.a, p.lda, sizeof(TG)) << 1 |
                    rows16(p.b, p.ldb, sizeof(TG)) << 2 | rows16(p.dh, p.lddh, sizeof(TD)) << 3 |
                    pairs(p.dx, p.lddx, sizeof(TD)) << 4 | pairs(p.da, p.ldda, sizeof(TDG)) << 5 |
                    pairs(p.db, p.lddb, sizeof(TDG)) << 6;
    return launch_chain(linrec_bwd_kernel<TX, TG, GIVEN, SCALE, TD, TDG>,
                        sizeof(BwdSmem<TX, TG, TD>), p, ch, vec, s, states, sums);
  }
};

}  // namespace

// Workspace: the chain's (linrec_workspace_bytes); the states, where the call does not pass
// the forward's; the chunks' sums of the gate parameters' gradients.
size_t linrec_bwd_workspace_bytes(const long long* cu, int B, int T, int D, bool states_given,
                                  int flags) {
  const long long chunks = linrec_chunks(cu, B, T);
  return chain_bytes(cu, B, T, D) + (states_given ? 0 : carry_bytes(chunks, D)) +
         (flags & GDN_GATES_PRECOMPUTED ? 0 : align256((size_t)chunks * D * sizeof(float2)));
}

cudaError_t launch_linrec_bwd(const LinrecArgs& a, void* workspace, cudaStream_t s) {
  const long long chunks = linrec_chunks(a.cu, a.B, a.T);
  char* more = static_cast<char*>(workspace) + chain_bytes(a.cu, a.B, a.T, a.D);
  Chain ch{};
  const float* states = a.states;
  cudaError_t e;
  if (states == nullptr) {
    float* own = reinterpret_cast<float*>(more);
    more += carry_bytes(chunks, a.D);
    LinrecArgs f = a;
    f.states_out = own;
    e = make_chain(f, workspace, own, true, s, &ch);
    if (e == cudaSuccess) e = launch_linrec_scan(f, ch, GDN_GRAD_F32, s);
    if (e != cudaSuccess) return e;
    states = own;
  }
  e = make_chain(a, workspace, nullptr, a.states != nullptr, s, &ch);
  float2* sums = reinterpret_cast<float2*>(more);
  if (e == cudaSuccess) e = by_type(a, GDN_GRAD_F32, BwdRun{a, ch, states, sums, s});
  if (e == cudaSuccess && !(a.flags & GDN_GATES_PRECOMPUTED)) {
    linrec_sums_kernel<<<(a.D + 31) / 32, dim3(32, kSumRows), 0, s>>>(sums, chunks, a.D, a.dA_log,
                                                                     a.ddt_bias);
    e = cudaGetLastError();
  }
  return e != cudaSuccess ? e : copy_empty(a, ch, a.dht, a.dh0, s);
}

}  // namespace gdn
