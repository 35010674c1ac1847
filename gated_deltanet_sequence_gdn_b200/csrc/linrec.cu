// linrec.cu -- the scan of the gated linear recurrence,
//   h_t = alpha_t h_{t-1} + f(alpha_t) beta_t x_t  per channel
// (linrec_math.cuh for the gates, linrec_chain.cuh for the split along time), and its
// one-token step.  Host side of the scan and of the backward (linrec_bwd.cu).
#include "linrec_chain.cuh"
#include "linrec_launch.cuh"

namespace gdn {

long long linrec_chunks(const long long* cu, int B, int T) {
  if (cu == nullptr) return B * (((long long)T + kLinrecChunk - 1) / kLinrecChunk);
  long long n = 0;
  for (int i = 0; i < B; ++i) n += (cu[i + 1] - cu[i] + kLinrecChunk - 1) / kLinrecChunk;
  return n;
}

namespace {

template <typename TX, typename TG>
struct FwdStage {
  alignas(16) TX x[kTileT * kTileC];
  alignas(16) TG a[kTileT * kTileC];
  alignas(16) TG b[kTileT * kTileC];
};
template <typename TX, typename TG>
struct FwdSmem {
  FwdStage<TX, TG> stage[2];
  float4 fold[kWorkWarps][32];  // (A, H) of each warp's tokens
  float2 in[32];                // what enters the tile
  Tile tile[3];                 // this tile's, the next one's, the one after
  int more[3];
};

template <typename TX, typename TG, bool GIVEN, int SCALE, typename TO>
__global__ void __launch_bounds__(kLinrecThreads)
linrec_fwd_kernel(LinrecArgs p, Chain ch, int vec) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<FwdSmem<TX, TG>*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const bool work = warp < kWorkWarps;
  const bool pair = vec & 8;
  if (threadIdx.x == kWorkThreads) {
    next_tile<false>(ch, sm, 0);
    next_tile<false>(ch, sm, 1);
  }
  __syncthreads();
  auto load = [&](int k) {
    if (sm.more[k % 3]) {
      const Tile& t = sm.tile[k % 3];
      FwdStage<TX, TG>& st = sm.stage[k & 1];
      load_tile(st.x, p.x, p.ldx, t, p.D, vec & 1);
      load_tile(st.a, p.a, p.lda, t, p.D, vec & 2);
      if (p.b) load_tile(st.b, p.b, p.ldb, t, p.D, vec & 4);
    }
    cp_async_commit();
  };
  if (work) load(0);
  GateConst k0{0.f, 0.f}, k1{0.f, 0.f};
  int c0 = -1;
  for (int k = 0;; ++k) {
    cp_async_wait<0>();
    __syncthreads();  // the stage is complete, the other one free, the tiles' numbers known
    if (!sm.more[k % 3]) return;
    const Tile t = sm.tile[k % 3];
    const int c = t.c0 + 2 * lane;
    float al[kPer][2], u[kPer][2];
    if (work) {
      load(k + 1);
      if (!GIVEN && c0 != t.c0) {
        c0 = t.c0;
        if (c < p.D) k0 = gate_const(p.A_log, p.dt_bias, c);
        if (c + 1 < p.D) k1 = gate_const(p.A_log, p.dt_bias, c + 1);
      }
      const FwdStage<TX, TG>& st = sm.stage[k & 1];
      float A0 = 1.f, A1 = 1.f, H0 = 0.f, H1 = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = (warp * kPer + i) * kTileC + 2 * lane;
        const float2 av = get2(st.a + at), xv = get2(st.x + at);
        const float g0 = log_decay<GIVEN>(av.x, k0), g1 = log_decay<GIVEN>(av.y, k1);
        al[i][0] = ex2_f(g0 * kLog2e);
        al[i][1] = ex2_f(g1 * kLog2e);
        u[i][0] = xv.x * input_scale<SCALE>(g0);
        u[i][1] = xv.y * input_scale<SCALE>(g1);
        if (p.b) {
          const float2 bv = get2(st.b + at);
          u[i][0] *= write_gate<GIVEN>(bv.x);
          u[i][1] *= write_gate<GIVEN>(bv.y);
        }
      }
      if (t.n < kTileT) {  // behind the sequence: the state passes through
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (warp * kPer + i >= t.n) {
            al[i][0] = al[i][1] = 1.f;
            u[i][0] = u[i][1] = 0.f;
          }
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        H0 = fmaf(al[i][0], H0, u[i][0]);
        H1 = fmaf(al[i][1], H1, u[i][1]);
        A0 *= al[i][0];
        A1 *= al[i][1];
      }
      sm.fold[warp][lane] = make_float4(A0, H0, A1, H1);
    } else if (lane == 0) {
      next_tile<false>(ch, sm, k + 2);
    }
    __syncthreads();
    float4 ex = make_float4(1.f, 0.f, 1.f, 0.f);  // what the tile's tokens before do
    if (work) {
      if (p.h) {
        for (int w = 0; w < warp; ++w) {
          const float4 f = sm.fold[w][lane];
          ex.y = fmaf(f.x, ex.y, f.y);
          ex.w = fmaf(f.z, ex.w, f.w);
          ex.x *= f.x;
          ex.z *= f.z;
        }
      }
    } else {
      float4 own = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWorkWarps; ++w) {
        const float4 f = sm.fold[w][lane];
        own.y = fmaf(f.x, own.y, f.y);
        own.w = fmaf(f.z, own.w, f.w);
        own.x *= f.x;
        own.z *= f.z;
      }
      const float2 in = chain_in<1>(ch, t, own, p.h0 ? p.h0 + (long long)t.row * p.D : nullptr);
      sm.in[lane] = in;
      const float2 out = make_float2(fmaf(own.x, in.x, own.y), fmaf(own.z, in.y, own.w));
      if (t.before == 0 && p.states_out) write2(p.states_out + (long long)t.chunk * p.D, c, p.D, in);
      if (t.after > 0) chain_out<1>(ch, t, out);
      else if (p.ht) write2(p.ht + (long long)t.row * p.D, c, p.D, out);
    }
    __syncthreads();
    if (work && p.h) {
      const float2 in = sm.in[lane];
      float h0 = fmaf(ex.x, in.x, ex.y), h1 = fmaf(ex.z, in.y, ex.w);
      TO* out = static_cast<TO*>(p.h) + (t.tok + warp * kPer) * p.ldh + c;
      const int cols = p.D - c;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        h0 = fmaf(al[i][0], h0, u[i][0]);
        h1 = fmaf(al[i][1], h1, u[i][1]);
        if (warp * kPer + i < t.n) put2(out, h0, h1, cols < 2 ? cols : 2, pair);
        out += p.ldh;
      }
    }
  }
}

template <typename TX, typename TG, bool GIVEN, int SCALE, typename TO>
__global__ void __launch_bounds__(128) linrec_step_kernel(LinrecArgs p, float* state) {
  const int blocks = (p.D + 127) / 128;
  const long long r = blockIdx.x / blocks;
  const int c = (blockIdx.x % blocks) * 128 + threadIdx.x;
  if (c >= p.D) return;
  const GateConst k = GIVEN ? GateConst{0.f, 0.f} : gate_const(p.A_log, p.dt_bias, c);
  const float g = log_decay<GIVEN>(to_f32(static_cast<const TG*>(p.a)[r * p.lda + c]), k);
  float u = to_f32(static_cast<const TX*>(p.x)[r * p.ldx + c]) * input_scale<SCALE>(g);
  if (p.b) u *= write_gate<GIVEN>(to_f32(static_cast<const TG*>(p.b)[r * p.ldb + c]));
  const float st = fmaf(ex2_f(g * kLog2e), state[r * p.D + c], u);
  state[r * p.D + c] = st;
  static_cast<TO*>(p.h)[r * p.ldh + c] = from_f32<TO>(st);
}

constexpr int kPiece = 240;  // entries of a table piece passed by value (< 4 KB of arguments)
struct TabPiece {
  long long cu[kPiece];
  int chunk0[kPiece];
  int first, n;
};
__global__ void seq_table_kernel(TabPiece p, long long* cu, int* chunk0) {
  for (int i = threadIdx.x; i < p.n; i += blockDim.x) {
    cu[p.first + i] = p.cu[i];
    chunk0[p.first + i] = p.chunk0[i];
  }
}
cudaError_t fill_seq_table(const long long* cu, int B, const SeqTab& tab, cudaStream_t s) {
  long long chunks = 0;
  TabPiece p;
  for (int i0 = 0; i0 <= B; i0 += kPiece) {
    p.first = i0;
    p.n = B + 1 - i0 < kPiece ? B + 1 - i0 : kPiece;
    for (int i = 0; i < p.n; ++i) {
      const int j = i0 + i;
      p.cu[i] = cu[j];
      p.chunk0[i] = (int)chunks;
      if (j < B) chunks += (cu[j + 1] - cu[j] + kLinrecChunk - 1) / kLinrecChunk;
    }
    seq_table_kernel<<<1, 256, 0, s>>>(p, const_cast<long long*>(tab.cu),
                                       const_cast<int*>(tab.chunk0));
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// What an empty sequence's chain starts with is what it ends with.
__global__ void copy_empty_kernel(const long long* cu, int D, const float* src, float* dst) {
  const int r = blockIdx.x;
  if (cu[r + 1] != cu[r]) return;
  for (int c = threadIdx.x; c < D; c += blockDim.x)
    dst[(long long)r * D + c] = src ? src[(long long)r * D + c] : 0.f;
}

struct FwdRun {
  const LinrecArgs& p;
  const Chain& ch;
  cudaStream_t s;
  template <typename TX, typename TG, bool GIVEN, int SCALE, bool WIDE>
  cudaError_t run() const {
    using TO = typename Wide<TX, WIDE>::type;
    const int vec = rows16(p.x, p.ldx, sizeof(TX)) | rows16(p.a, p.lda, sizeof(TG)) << 1 |
                    rows16(p.b, p.ldb, sizeof(TG)) << 2 | pairs(p.h, p.ldh, sizeof(TO)) << 3;
    return launch_chain(linrec_fwd_kernel<TX, TG, GIVEN, SCALE, TO>, sizeof(FwdSmem<TX, TG>), p,
                        ch, vec, s);
  }
};
struct StepRun {
  const LinrecArgs& p;
  float* state;
  cudaStream_t s;
  template <typename TX, typename TG, bool GIVEN, int SCALE, bool WIDE>
  cudaError_t run() const {
    const long long blocks = (long long)p.B * ((p.D + 127) / 128);
    linrec_step_kernel<TX, TG, GIVEN, SCALE, typename Wide<TX, WIDE>::type>
        <<<(unsigned)blocks, 128, 0, s>>>(p, state);
    return cudaGetLastError();
  }
};

bool any_neighbours(const LinrecArgs& a) {
  if (a.cu == nullptr) return a.T > kLinrecChunk;
  for (int i = 0; i < a.B; ++i)
    if (a.cu[i + 1] - a.cu[i] > kLinrecChunk) return true;
  return false;
}

}  // namespace

// Workspace: the sequence table; the ticket and a flag a tile; the tiles' aggregates; the
// chunks' carries.
size_t linrec_workspace_bytes(const long long* cu, int B, int T, int D) {
  return chain_bytes(cu, B, T, D);
}

cudaError_t make_chain(const LinrecArgs& a, void* workspace, float* carry, bool table,
                       cudaStream_t s, Chain* ch) {
  char* ws = static_cast<char*>(workspace);
  const long long chunks = linrec_chunks(a.cu, a.B, a.T);
  ch->B = a.B; ch->T = a.T; ch->D = a.D;
  ch->nblk = (a.D + kTileC - 1) / kTileC;
  ch->per_row = (int)(((long long)a.T + kTileT - 1) / kTileT);
  ch->tiles = (int)(chunks * ch->nblk);
  if (a.cu) {
    ch->tab.cu = reinterpret_cast<const long long*>(ws);
    ch->tab.chunk0 =
        reinterpret_cast<const int*>(ws + align256((size_t)(a.B + 1) * sizeof(long long)));
    if (table) {
      cudaError_t e = fill_seq_table(a.cu, a.B, ch->tab, s);
      if (e != cudaSuccess) return e;
    }
    ws += seq_table_bytes(a.B);
  }
  const size_t flag_bytes = flags_bytes(ch->tiles);
  ch->ticket = any_neighbours(a) ? reinterpret_cast<int*>(ws) : nullptr;
  ch->flags = reinterpret_cast<int*>(ws) + 64;
  ch->agg = reinterpret_cast<float4*>(ws + flag_bytes);
  ch->carry = carry ? carry
                    : reinterpret_cast<float*>(ws + flag_bytes + (size_t)ch->tiles * 32 * sizeof(float4));
  ch->status = status_word();
  if (ch->status == nullptr) return cudaErrorUnknown;
  const WaitFault wf = wait_fault();
  ch->spin = wf.spin < kLinrecSpin ? wf.spin : kLinrecSpin;
  ch->fault = wf.site == kFaultLinrec;
  return ch->ticket ? cudaMemsetAsync(ws, 0, flag_bytes, s) : cudaSuccess;
}

cudaError_t copy_empty(const LinrecArgs& a, const Chain& ch, const float* src, float* dst,
                       cudaStream_t s) {
  if (a.cu == nullptr || dst == nullptr || src == dst) return cudaSuccess;
  bool any = false;
  for (int i = 0; i < a.B; ++i) any |= a.cu[i + 1] == a.cu[i];
  if (!any) return cudaSuccess;
  copy_empty_kernel<<<a.B, 128, 0, s>>>(ch.tab.cu, a.D, src, dst);
  return cudaGetLastError();
}

cudaError_t launch_linrec_scan(const LinrecArgs& a, const Chain& ch, int wide_flag,
                               cudaStream_t s) {
  return by_type(a, wide_flag, FwdRun{a, ch, s});
}

cudaError_t launch_linrec_fwd(const LinrecArgs& a, void* workspace, cudaStream_t s) {
  Chain ch{};
  cudaError_t e = make_chain(a, workspace, a.states_out, true, s, &ch);
  if (e == cudaSuccess) e = launch_linrec_scan(a, ch, GDN_OUT_F32, s);
  return e != cudaSuccess ? e : copy_empty(a, ch, a.h0, a.ht, s);
}

cudaError_t launch_linrec_step(const LinrecArgs& a, float* state, cudaStream_t s) {
  return by_type(a, GDN_OUT_F32, StepRun{a, state, s});
}

}  // namespace gdn
