// linrec.cu -- the scan of the gated linear recurrence,
//   h_t = alpha_t h_{t-1} + f(alpha_t) beta_t x_t  per channel
// (linrec_math.cuh for the gates, linrec_tile.cuh for the split along time), and its
// one-token step.  Host side of the scan and of the backward (linrec_bwd.cu).
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
  CarrySmem carry;
};

template <typename TX, typename TG, bool GIVEN, int SCALE, typename TO>
__global__ void __launch_bounds__(kLinrecThreads, sizeof(TX) + sizeof(TG) == 4 ? 4 : 2)
linrec_fwd_kernel(LinrecArgs p, Chains ch, int vec) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<FwdSmem<TX, TG>*>(smem_raw);
  FoldRow* folds = reinterpret_cast<FoldRow*>(smem_raw + sizeof(FwdSmem<TX, TG>));
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const Chain k = chain_of(p, ch);
  const int c = k.c0 + 2 * lane, cols = p.D - c;
  auto load = [&](int round) {
    const int tt = round * ch.cs + k.rank;
    if (tt < k.chunks) {
      const long long left = k.len - (long long)tt * kTileT, tok = k.tok + (long long)tt * kTileT;
      const int n = left < kTileT ? (int)left : kTileT;
      FwdStage<TX, TG>& st = sm.stage[round & 1];
      load_tile(st.x, p.x, p.ldx, tok, n, k.c0, p.D, vec & 1);
      load_tile(st.a, p.a, p.lda, tok, n, k.c0, p.D, vec & 2);
      if (p.b) load_tile(st.b, p.b, p.ldb, tok, n, k.c0, p.D, vec & 4);
    }
    cp_async_commit();
  };
  load(0);
  carry_begin(ch, sm.carry);
  GateConst gc{both(0.f), both(0.f)};
  if (!GIVEN) gc = gate_const(p.A_log, p.dt_bias, c, p.D);
  float2 carry = read2(p.h0, k.row, c, p.D);  // before the round's first tile (warp 0's)
  bool lost = false;
  const int rounds = (k.chunks + ch.cs - 1) / ch.cs;
  for (int round = 0; round < rounds; ++round) {
    cp_async_wait<0>();
    __syncthreads();  // the stage is complete, the other one free
    if (round + 1 < rounds) load(round + 1);
    const int tt = round * ch.cs + k.rank;
    const long long left = k.len - (long long)tt * kTileT;
    const int n = left < kTileT ? (left < 0 ? 0 : (int)left) : kTileT;
    const FwdStage<TX, TG>& st = sm.stage[round & 1];
    const int mine = warp * kPer * kTileC + 2 * lane;
    float2 al[kPer], u[kPer];
    float2 A = both(1.f), H = both(0.f);
#pragma unroll
    for (int i0 = 0; i0 < kPer; i0 += kGroup) {
      float2 e[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) e[i] = get2(st.a + mine + (i0 + i) * kTileC);
      decay_exponents<GIVEN, kGroup>(e, gc);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        al[i0 + i] = ex2_2(e[i]);
        u[i0 + i] = get2(st.x + mine + (i0 + i) * kTileC);
        if (SCALE != kScaleNone)
          u[i0 + i] = mul2(u[i0 + i], input_scale<SCALE>(e[i], al[i0 + i]));
      }
      if (p.b)
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
          u[i0 + i] = mul2(u[i0 + i], write_gate<GIVEN>(get2(st.b + mine + (i0 + i) * kTileC)));
    }
    if (n < kTileT) {  // behind the sequence: the state passes through
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (warp * kPer + i >= n) {
          al[i] = both(1.f);
          u[i] = both(0.f);
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      H = fma2(al[i], H, u[i]);
      A = mul2(A, al[i]);
    }
    sm.carry.fold[warp][lane] = join4(A, H);
    __syncthreads();
    A = both(1.f);  // what the tile's tokens before the warp's do
    H = both(0.f);
    if (warp == 0) {
      float2 tA = both(1.f), tH = both(0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 f = sm.carry.fold[w][lane];
        tH = fma2(first2(f), tH, last2(f));
        tA = mul2(tA, first2(f));
      }
      const float2 in = carry_round(ch, k.rank, round, join4(tA, tH), sm.carry, folds, &carry, &lost);
      sm.carry.in[lane] = in;
      if (n > 0) write2(p.states_out, k.chunk0 + tt, c, p.D, in);
    } else {
      for (int w = 0; w < warp; ++w) {
        const float4 f = sm.carry.fold[w][lane];
        H = fma2(first2(f), H, last2(f));
        A = mul2(A, first2(f));
      }
    }
    __syncthreads();
    if (p.h) {
      float2 h = fma2(A, sm.carry.in[lane], H);
      TO* out = static_cast<TO*>(p.h) + (k.tok + (long long)tt * kTileT + warp * kPer) * p.ldh + c;
      if (n == kTileT && cols > 1 && (vec & 8)) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          h = fma2(al[i], h, u[i]);
          put2(out, h);
          out += p.ldh;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          h = fma2(al[i], h, u[i]);
          if (warp * kPer + i < n) put2(out, h, cols);
          out += p.ldh;
        }
      }
    }
  }
  if (k.rank == 0 && warp == 0) write2(p.ht, k.row, c, p.D, carry);
  carry_end(ch);
}

// Two channels from anywhere a row has them.
template <typename T>
__device__ __forceinline__ float2 take2(const void* base, long long at, int cols) {
  const T* p = static_cast<const T*>(base) + at;
  return make_float2(to_f32(p[0]), cols > 1 ? to_f32(p[1]) : 0.f);
}
template <typename TX, typename TG, bool GIVEN, int SCALE, typename TO>
__global__ void __launch_bounds__(128) linrec_step_kernel(LinrecArgs p, float* state) {
  const int blocks = (p.D + 255) / 256;
  const long long r = blockIdx.x / blocks;
  const int c = (blockIdx.x % blocks) * 256 + 2 * threadIdx.x, cols = p.D - c;
  if (cols <= 0) return;
  GateConst gc{both(0.f), both(0.f)};
  if (!GIVEN) gc = gate_const(p.A_log, p.dt_bias, c, p.D);
  float2 e = take2<TG>(p.a, r * p.lda + c, cols);
  decay_exponents<GIVEN, 1>(&e, gc);
  const float2 al = ex2_2(e);
  float2 u = mul2(take2<TX>(p.x, r * p.ldx + c, cols), input_scale<SCALE>(e, al));
  if (p.b) u = mul2(u, write_gate<GIVEN>(take2<TG>(p.b, r * p.ldb + c, cols)));
  const float2 st = fma2(al, read2(state, r, c, p.D), u);
  write2(state, r, c, p.D, st);
  put2(static_cast<TO*>(p.h) + r * p.ldh + c, st, cols);
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

struct FwdRun {
  const LinrecArgs& p;
  const Chains& ch;
  cudaStream_t s;
  template <typename TX, typename TG, bool GIVEN, int SCALE, bool WIDE>
  cudaError_t run() const {
    using TO = typename Wide<TX, WIDE>::type;
    const int vec = rows16(p.x, p.ldx, sizeof(TX)) | rows16(p.a, p.lda, sizeof(TG)) << 1 |
                    rows16(p.b, p.ldb, sizeof(TG)) << 2 | pairs(p.h, p.ldh, sizeof(TO)) << 3;
    int cs = 1;
    return launch_chains(linrec_fwd_kernel<TX, TG, GIVEN, SCALE, TO>, sizeof(FwdSmem<TX, TG>), p,
                         ch, vec, &cs, s);
  }
};
struct StepRun {
  const LinrecArgs& p;
  float* state;
  cudaStream_t s;
  template <typename TX, typename TG, bool GIVEN, int SCALE, bool WIDE>
  cudaError_t run() const {
    const long long blocks = (long long)p.B * ((p.D + 255) / 256);
    linrec_step_kernel<TX, TG, GIVEN, SCALE, typename Wide<TX, WIDE>::type>
        <<<(unsigned)blocks, 128, 0, s>>>(p, state);
    return cudaGetLastError();
  }
};

}  // namespace

// Workspace: the table of a packed batch.
size_t linrec_workspace_bytes(const long long* cu, int B, int T, int D) {
  return cu ? seq_table_bytes(B) : 0;
}

cudaError_t make_chains(const LinrecArgs& a, void* workspace, bool table, cudaStream_t s,
                        Chains* ch) {
  ch->nblk = (a.D + kTileC - 1) / kTileC;
  if (a.cu) {
    char* ws = static_cast<char*>(workspace);
    ch->tab.cu = reinterpret_cast<const long long*>(ws);
    ch->tab.chunk0 =
        reinterpret_cast<const int*>(ws + align256((size_t)(a.B + 1) * sizeof(long long)));
    if (table) {
      cudaError_t e = fill_seq_table(a.cu, a.B, ch->tab, s);
      if (e != cudaSuccess) return e;
    }
  }
  ch->status = status_word();
  if (ch->status == nullptr) return cudaErrorUnknown;
  const WaitFault wf = wait_fault();
  ch->spin = wf.spin;
  ch->fault = wf.site == kFaultLinrec;
  return cudaSuccess;
}

cudaError_t launch_linrec_scan(const LinrecArgs& a, const Chains& ch, int wide_flag,
                               cudaStream_t s) {
  return by_type(a, wide_flag, FwdRun{a, ch, s});
}

cudaError_t launch_linrec_fwd(const LinrecArgs& a, void* workspace, cudaStream_t s) {
  Chains ch{};
  cudaError_t e = make_chains(a, workspace, true, s, &ch);
  return e != cudaSuccess ? e : launch_linrec_scan(a, ch, GDN_OUT_F32, s);
}

cudaError_t launch_linrec_step(const LinrecArgs& a, float* state, cudaStream_t s) {
  return by_type(a, GDN_OUT_F32, StepRun{a, state, s});
}

}  // namespace gdn
