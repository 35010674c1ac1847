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
  alignas(128) TX x[kTile];
  alignas(128) TG a[kTile];
  alignas(128) TG b[kTile];
};
template <typename TX, typename TG>
struct FwdSmem {
  FwdStage<TX, TG> stage[2];
  CarrySmem carry;
};

template <typename TX, typename TG, bool GIVEN, int SCALE, typename TO, bool NARROW>
__global__ void __launch_bounds__(kLinrecThreads, sizeof(TX) + sizeof(TG) == 4 ? 4 : 2)
linrec_fwd_kernel(LinrecArgs p, Chains ch, int vec, const __grid_constant__ LinrecMaps maps) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<FwdSmem<TX, TG>*>(smem_raw);
  FoldRow* folds = reinterpret_cast<FoldRow*>(smem_raw + sizeof(FwdSmem<TX, TG>));
  constexpr int kTileT = Shape<NARROW>::kT, kC = Shape<NARROW>::kC, kTileChunks = kTileT / kLinrecChunk;
  const Spot<NARROW> at;
  const Chain k = chain_of<NARROW>(p, ch);
  const int c = k.c0 + 2 * at.cl, cols = p.D - c;
  const int step = ch.cs * kTileT;
  const int tokens = (int)k.len - k.rank * kTileT;  // from the block's first tile on
  auto length = [&](int round) {
    const int left = tokens - round * step;
    return left < kTileT ? (left < 0 ? 0 : left) : kTileT;
  };
  auto load = [&](int round) {
    const int n = length(round), t = (round * ch.cs + k.rank) * kTileT;
    FwdStage<TX, TG>& st = sm.stage[round & 1];
    if (ch.tma) {
      if (n > 0 && threadIdx.x == 0) {
        uint64_t* bar = &sm.carry.loaded[round & 1];
        const int y = ch.tab.cu ? (int)k.tok + t : t, z = ch.tab.cu ? 0 : k.row;
        tc::mbar_arrive_expect_tx(bar, sizeof(st.x) + sizeof(st.a) + (p.b ? sizeof(st.b) : 0));
        tma_load_3d(st.x, &maps.x, bar, k.c0, y, z);
        tma_load_3d(st.a, &maps.a, bar, k.c0, y, z);
        if (p.b) tma_load_3d(st.b, &maps.b, bar, k.c0, y, z);
      }
    } else {
      if (n > 0) {
        load_elements<NARROW>(st.x, p.x, p.ldx, k.tok + t, n, k.c0, p.D);
        load_elements<NARROW>(st.a, p.a, p.lda, k.tok + t, n, k.c0, p.D);
        if (p.b) load_elements<NARROW>(st.b, p.b, p.ldb, k.tok + t, n, k.c0, p.D);
      }
      cp_async_commit();
    }
  };
  carry_begin(ch, sm.carry);
  load(0);
  GateConst gc{both(0.f), both(0.f)};
  if (!GIVEN) gc = gate_const(p.A_log, p.dt_bias, c, p.D);
  float2 carry = read2(p.h0, k.row, c, p.D);  // before the round's first tile (warp 0's)
  bool lost = false;
  Rows<TO> out;
  out.begin(p.h, p.ldh, k.tok + k.rank * kTileT, k.c0, at.first, 2 * at.cl);
  const int rounds = (k.tiles + ch.cs - 1) / ch.cs;
  for (int round = 0; round < rounds; ++round) {
    const int n = length(round);
    if (!ch.tma) {
      cp_async_wait<0>();
    } else if (n > 0 && !tc::mbar_wait(&sm.carry.loaded[round & 1], (round >> 1) & 1, nullptr, 0)) {
      report_timeout(ch.status, 0x4c54);
    }
    __syncthreads();  // the stage is complete, the other one free
    if (round + 1 < rounds) load(round + 1);
    const FwdStage<TX, TG>& st = sm.stage[round & 1];
    const int mine = at.mine();
    float2 al[kPer], u[kPer];
#pragma unroll
    for (int i0 = 0; i0 < kPer; i0 += kGroup) {
      float2 e[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) e[i] = get2(st.a + mine + (i0 + i) * kC);
      decay_exponents<GIVEN, kGroup>(e, gc);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        al[i0 + i] = ex2_2(e[i]);
        u[i0 + i] = get2(st.x + mine + (i0 + i) * kC);
      }
      if (SCALE != kScaleNone) {
        float2 f[kGroup];
        input_scales<SCALE, kGroup>(e, al + i0, f);
#pragma unroll
        for (int i = 0; i < kGroup; ++i) u[i0 + i] = mul2(u[i0 + i], f[i]);
      }
      if (p.b) {
        float2 b[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) b[i] = get2(st.b + mine + (i0 + i) * kC);
        write_gates<GIVEN, kGroup>(b);
#pragma unroll
        for (int i = 0; i < kGroup; ++i) u[i0 + i] = mul2(u[i0 + i], b[i]);
      }
    }
    if (n < kTileT) {  // behind the sequence: the state passes through
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (at.first + i >= n) {
          al[i] = both(1.f);
          u[i] = both(0.f);
        }
    }
    float2 A = al[0], H = u[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) {
      H = fma2(al[i], H, u[i]);
      A = mul2(A, al[i]);
    }
    sm.carry.fold[threadIdx.x] = join4(A, H);
    __syncthreads();
    if (at.warp == 0) {
      A = both(1.f);
      H = both(0.f);
#pragma unroll 4
      for (int w = 0; w < 8; ++w) {
        const float4 f = sm.carry.fold[at.group(w)];
        H = fma2(first2(f), H, last2(f));
        A = mul2(A, first2(f));
      }
      float2 v = carry_round<NARROW, false>(ch, k.rank, round, join4(A, H), sm.carry, folds, &carry,
                                            &lost);
      if (n > at.half * kLinrecChunk)
        write2(p.states_out,
               k.chunk0 + (long long)(round * ch.cs + k.rank) * kTileChunks + at.half, c, p.D, v);
#pragma unroll 4
      for (int w = 0; w < 8; ++w) {
        sm.carry.start[at.group(w)] = v;
        const float4 f = sm.carry.fold[at.group(w)];
        v = fma2(first2(f), v, last2(f));
      }
    }
    __syncthreads();
    if (p.h) {
      float2 h = sm.carry.start[threadIdx.x];
      if (n == kTileT && cols > 1 && vec) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          h = fma2(al[i], h, u[i]);
          put2(out.at(i), h);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          h = fma2(al[i], h, u[i]);
          if (at.first + i < n) put2(out.at(i), h, cols);
        }
      }
      out.advance(step);
    }
  }
  if (k.rank == 0 && at.warp == 0 && at.half == 0) write2(p.ht, k.row, c, p.D, carry);
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
  float2 u = take2<TX>(p.x, r * p.ldx + c, cols);
  if (SCALE != kScaleNone) {
    float2 f;
    input_scales<SCALE, 1>(&e, &al, &f);
    u = mul2(u, f);
  }
  if (p.b) {
    float2 b = take2<TG>(p.b, r * p.ldb + c, cols);
    write_gates<GIVEN, 1>(&b);
    u = mul2(u, b);
  }
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
  int vec;  // the rows of h take pairs
  cudaStream_t s;
  template <typename TX, typename TG, bool GIVEN, int SCALE, bool WIDE>
  cudaError_t run() const {
    using TO = typename Wide<TX, WIDE>::type;
    static KernelSlots known, known_narrow;
    const auto kernel = linrec_fwd_kernel<TX, TG, GIVEN, SCALE, TO, false>;
    const std::atomic<int>* slots = nullptr;
    int cs = 1;
    cudaError_t e = kernel_slots(kernel, sizeof(FwdSmem<TX, TG>), &known, &slots);
    if (e != cudaSuccess) return e;
    return narrow_tiles(p, slots[0].load(std::memory_order_relaxed))
               ? launch<TX, TG, true>(linrec_fwd_kernel<TX, TG, GIVEN, SCALE, TO, true>,
                                      &known_narrow, &cs)
               : launch<TX, TG, false>(kernel, &known, &cs);
  }
  template <typename TX, typename TG, bool NARROW, typename K>
  cudaError_t launch(K kernel, KernelSlots* known, int* cs) const {
    LinrecMaps maps;
    Chains c = ch;
    c.tma = map_tiles<NARROW, TX>(&maps.x, p, p.x, p.ldx) &&
            map_tiles<NARROW, TG>(&maps.a, p, p.a, p.lda) &&
            (!p.b || map_tiles<NARROW, TG>(&maps.b, p, p.b, p.ldb));
    return launch_chains<NARROW>(kernel, sizeof(FwdSmem<TX, TG>), p, c, known, vec, cs, s, maps);
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
  const int wide = a.dtype == GDN_F32 || (a.flags & wide_flag);
  return by_type(a, wide_flag, FwdRun{a, ch, pairs(a.h, a.ldh, wide ? 4 : 2), s});
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
