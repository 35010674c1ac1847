// linrec.cu -- the scan of the gated linear recurrence,
//   h_t = alpha_t h_{t-1} + f(alpha_t) beta_t x_t  per channel
// (linrec_math.cuh for the gates, linrec_tile.cuh for the split along time), and its
// one-token step.  Host side of the scan and of the backward (linrec_bwd.cu).
//
// What bounds the scan: an element of bf16 with both gates moves 8 bytes and takes 33
// instructions, most of them softplus, two exponentials and a sigmoid, against the 44 that an
// SM issues while 8 bytes cross its share of the HBM at the measured copy rate; 60% of the
// issue slots and of the XU pipe are in use at 27 warps an SM.  float32 (16 bytes) is bound by
// the HBM alone.  Measured: 64 sequences of 512 x 4096 bf16 181 us, 5.9 TB/s (copy: 6.6);
// float32 of 512 x 2048 160 us, 6.7 TB/s.  Where there are few chains, their blocks do not
// share evenly among the SMs and wait more for their own carry: one sequence of 8192 x 12288
// 184 us on the same inputs again and 197 on others each time (4.4 and 4.1 TB/s); 131072 x
// 1024, tied, without a write gate (6 bytes), in clusters 280 us, 2.9 TB/s.
//
// Three barriers a tile: the stage is there; the folds are; the start states are.  One warp
// joins the folds while the others wait.  Every warp finding its own start state takes one
// barrier less but spills and adds 2 to 3 instructions an element (a packed batch of 20011 x
// 4096 174 against 164 us).  The 64 registers of four blocks an SM hold the tile's alpha and
// u; blocks alone on their chains have a kernel without the exchange (187 against 183 us).
#include "linrec_launch.cuh"

namespace gdn {

long long linrec_chunks(const long long* cu, int B, int T) {
  if (cu == nullptr) return B * (((long long)T + kLinrecChunk - 1) / kLinrecChunk);
  long long n = 0;
  for (int i = 0; i < B; ++i) n += (cu[i + 1] - cu[i] + kLinrecChunk - 1) / kLinrecChunk;
  return n;
}

namespace {

// Shared memory: the carry, then two stages of x, a and (where there is a write gate) b, then
// the cluster's folds.
template <typename TX, typename TG>
constexpr size_t stage_bytes(bool gate) {
  return kTile * (sizeof(TX) + sizeof(TG) * (gate ? 2 : 1));
}
constexpr size_t kCarryBytes = (sizeof(CarrySmem) + 127) / 128 * 128;
template <typename TX, typename TG>
constexpr size_t fwd_smem(bool gate) {
  return kCarryBytes + 2 * stage_bytes<TX, TG>(gate);
}
template <typename TX, typename TG>
struct FwdStage {
  TX* x;
  TG *a, *b;
};

template <typename TX, typename TG, bool GIVEN, int SCALE, typename TO, int SPLIT, bool CLUSTER>
__global__ void __launch_bounds__(kLinrecThreads, sizeof(TX) + sizeof(TG) == 4 ? 4 : 2)
linrec_fwd_kernel(LinrecArgs p, Chains ch, int vec, const __grid_constant__ LinrecMaps maps) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  CarrySmem& carry_sm = *reinterpret_cast<CarrySmem*>(smem_raw);
  const uint32_t stage_size = stage_bytes<TX, TG>(p.b != nullptr);
  FoldRow* folds = reinterpret_cast<FoldRow*>(smem_raw + kCarryBytes + 2 * stage_size);
  auto stage = [&](int round) {
    unsigned char* s = smem_raw + kCarryBytes + (round & 1) * stage_size;
    TG* a = reinterpret_cast<TG*>(s + kTile * sizeof(TX));
    return FwdStage<TX, TG>{reinterpret_cast<TX*>(s), a, a + kTile};
  };
  constexpr int kTileT = Shape<SPLIT>::kT, kC = Shape<SPLIT>::kC;
  constexpr int kTileChunks = kTileT / kLinrecChunk;
  const Spot<SPLIT> at;
  wait_for_launch();
  const Chain k = chain_of<SPLIT, CLUSTER>(p, ch);
  const int c = k.c0 + 2 * at.cl, cols = p.D - c;
  const int cs = CLUSTER ? ch.cs : 1, step = cs * kTileT;
  const int tokens = (int)k.len - k.rank * kTileT;  // from the block's first tile on
  auto length = [&](int round) {
    const int left = tokens - round * step;
    return left < kTileT ? (left < 0 ? 0 : left) : kTileT;
  };
  int late = -1;  // the round whose tiles have not come in time: no more are asked for
  auto load = [&](int round) {
    const int n = length(round), t = (round * cs + k.rank) * kTileT;
    const FwdStage<TX, TG> st = stage(round);
    if (ch.tma) {
      if (n > 0 && threadIdx.x == 0 && late < 0) {
        uint64_t* bar = &carry_sm.loaded[round & 1];
        const int y = ch.tab.cu ? (int)k.tok + t : t, z = ch.tab.cu ? 0 : k.row;
        tc::mbar_arrive_expect_tx(bar, stage_size);
        if (ch.fault == kFaultLinrecTiles) return;
        tma_load_3d(st.x, &maps.x, bar, k.c0, y, z);
        tma_load_3d(st.a, &maps.a, bar, k.c0, y, z);
        if (p.b) tma_load_3d(st.b, &maps.b, bar, k.c0, y, z);
      }
    } else {
      if (n > 0) {
        load_elements<SPLIT>(st.x, p.x, p.ldx, k.tok + t, n, k.c0, p.D);
        load_elements<SPLIT>(st.a, p.a, p.lda, k.tok + t, n, k.c0, p.D);
        if (p.b) load_elements<SPLIT>(st.b, p.b, p.ldb, k.tok + t, n, k.c0, p.D);
      }
      cp_async_commit();
    }
  };
  carry_begin<CLUSTER>(carry_sm);
  load(0);
  GateConst gc{both(0.f), both(0.f)};
  if (!GIVEN) gc = gate_const(p.A_log, p.dt_bias, c, p.D);
  float2 carry = read2(p.h0, k.row, c, p.D);  // before the round's first tile (warp 0's)
  bool lost = false;
  Rows<TO> out;
  out.begin(p.h, p.ldh, k.tok + k.rank * kTileT, k.c0, at.first, 2 * at.cl);
  constexpr bool alone = SPLIT == 1 && !CLUSTER;  // what enters a tile is known before it is folded
  const int rounds = (k.tiles + cs - 1) / cs;
  for (int round = 0; round < rounds; ++round) {
    const int n = length(round);
    if (!ch.tma) {
      cp_async_wait<0>();
    } else if (n > 0 && late < 0 &&
               !tc::mbar_wait(&carry_sm.loaded[round & 1], (round >> 1) & 1, nullptr, 0, ch.spin)) {
      report_timeout(ch.status, 0x4c54);
      late = round;
    }
    __syncthreads();  // the stage is complete, the other one free
    if (round + 1 < rounds) load(round + 1);
    const FwdStage<TX, TG> st = stage(round);
    const int mine = at.mine();
    float2 al[kPer], u[kPer];
#pragma unroll
    for (int i0 = 0; i0 < kPer; i0 += kGroup) {
      float2 e[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        e[i] = get2(st.a + mine + (i0 + i) * kC);
        u[i0 + i] = get2(st.x + mine + (i0 + i) * kC);
      }
      decay_exponents<GIVEN, kGroup>(e, gc);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) al[i0 + i] = ex2_2(e[i]);
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
    carry_sm.fold[threadIdx.x] = join4(A, H);
    __syncthreads();
    if (at.warp == 0) {
      float2 v = carry;
      if (!alone)
        v = carry_round<SPLIT, CLUSTER, false>(
            ch, k.rank, round, chunk_fold<SPLIT, false>(at, carry_sm, nullptr), carry_sm, folds,
            &carry, &lost);
      if (n > at.part * kLinrecChunk)
        write2(p.states_out,
               k.chunk0 + (long long)(round * cs + k.rank) * kTileChunks + at.part, c, p.D, v);
      A = both(1.f);
      H = both(0.f);
#pragma unroll 4
      for (int w = 0; w < 8; ++w) {
        const float4 f = carry_sm.fold[at.group(w)];
        // in the fold's place: 2 KB that let clusters of 2 and 3 keep four blocks an SM
        put2(&carry_sm.fold[at.group(w)].x, v);
        v = fma2(first2(f), v, last2(f));
        H = fma2(first2(f), H, last2(f));
        A = mul2(A, first2(f));
      }
      // what leaves the tile, as it is formed elsewhere: from the chunk's own (A, H)
      if (alone) carry = fma2(A, carry, H);
    }
    __syncthreads();
    if (p.h) {
      float2 h = get2(&carry_sm.fold[threadIdx.x].x);
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
    if (at.warp == 0) carry_rest<SPLIT, CLUSTER, false>(ch, k.rank, round, folds, &carry);
  }
  // no copy is to be on its way when the block leaves: once more, with a limit
  if (late >= 0 && threadIdx.x == 0)
    tc::mbar_wait(&carry_sm.loaded[late & 1], (late >> 1) & 1, nullptr, 0, 1u << 20);
  carry_end<CLUSTER>();
  // ht may be h0, which every block of the cluster has read by now
  if (k.rank == 0 && at.warp == 0 && at.part == 0) write2(p.ht, k.row, c, p.D, carry);
}

// The step: HBM-bound on the float32 state, read and written once.  A thread takes 4 channels
// of one sequence, in pieces of 4 elements (VEC: the rows are aligned to them) or one by one.
// 16 bytes a bf16 channel with a write gate: 4096 x 4096 44 us, 6.1 TB/s; 256 x 12288 10.4 us
// in a graph, 4.8 TB/s (6144 blocks, 2.6 times what runs at once: the launch, the first loads'
// latency and the unfilled last wave count); two channels a thread took 2.6 us more.
template <bool VEC, typename T>
__device__ __forceinline__ void take4(const void* base, long long at, int cols, float2* f) {
  const T* p = static_cast<const T*>(base) + at;
  if (!VEC) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < cols ? to_f32(p[i]) : 0.f;
    f[0] = make_float2(v[0], v[1]);
    f[1] = make_float2(v[2], v[3]);
  } else if (sizeof(T) == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    f[0] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
    f[1] = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  } else {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = make_float2(v.x, v.y);
    f[1] = make_float2(v.z, v.w);
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void leave4(void* base, long long at, int cols, const float2* f) {
  T* p = static_cast<T*>(base) + at;
  if (!VEC) {
    const float v[4] = {f[0].x, f[0].y, f[1].x, f[1].y};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < cols) p[i] = from_f32<T>(v[i]);
  } else if (sizeof(T) == 2) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0].x, f[0].y);
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[1].x, f[1].y);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  }
}
constexpr int kStepThreads = 128;
template <typename TX, typename TG, bool GIVEN, int SCALE, typename TO, bool VEC>
__global__ void __launch_bounds__(kStepThreads) linrec_step_kernel(LinrecArgs p, float* state) {
  const int blocks = (p.D + 4 * kStepThreads - 1) / (4 * kStepThreads);
  const long long r = blockIdx.x / blocks;
  const int c = (blockIdx.x % blocks) * 4 * kStepThreads + 4 * threadIdx.x, cols = p.D - c;
  if (cols <= 0) return;
  float2 e[2], x[2], b[2], st[2], al[2], f[2];
  take4<VEC, TG>(p.a, r * p.lda + c, cols, e);
  take4<VEC, TX>(p.x, r * p.ldx + c, cols, x);
  take4<VEC, float>(state, r * p.D + c, cols, st);
  if (p.b) take4<VEC, TG>(p.b, r * p.ldb + c, cols, b);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    GateConst gc{both(0.f), both(0.f)};
    if (!GIVEN) gc = gate_const(p.A_log, p.dt_bias, c + 2 * i, p.D);
    decay_exponents<GIVEN, 1>(e + i, gc);
    al[i] = ex2_2(e[i]);
  }
  if (SCALE != kScaleNone) {
    input_scales<SCALE, 2>(e, al, f);
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = mul2(x[i], f[i]);
  }
  if (p.b) {
    write_gates<GIVEN, 2>(b);
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = mul2(x[i], b[i]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) st[i] = fma2(al[i], st[i], x[i]);
  leave4<VEC, float>(state, r * p.D + c, cols, st);
  leave4<VEC, TO>(p.h, r * p.ldh + c, cols, st);
}

constexpr int kPiece = 240;  // entries of a table piece passed by value (< 4 KB of arguments)
struct TabPiece {
  long long cu[kPiece];
  int chunk0[kPiece], order[kPiece];
  int first, n;
};
__global__ void seq_table_kernel(TabPiece p, long long* cu, int* chunk0, int* order) {
  for (int i = threadIdx.x; i < p.n; i += blockDim.x) {
    cu[p.first + i] = p.cu[i];
    chunk0[p.first + i] = p.chunk0[i];
    order[p.first + i] = p.order[i];
  }
}
// The sequences' order: by eighths of the longest one's length, from the last to the first,
// each in the order of the batch.
struct Order {
  const long long* cu;
  int B, eighth, next;
  long long most;
  int take() {
    for (; eighth >= 0; --eighth, next = 0)
      while (next < B) {
        const int i = next++;
        const long long e = (cu[i + 1] - cu[i]) * 8 / most;
        if ((e < 7 ? e : 7) == eighth) return i;
      }
    return 0;  // entry B, which is not a sequence
  }
};
cudaError_t fill_seq_table(const LinrecArgs& a, const SeqTab& tab, cudaStream_t s) {
  const long long most = longest(a);
  Order order{a.cu, a.B, 7, 0, most > 0 ? most : 1};
  long long chunks = 0;
  TabPiece p;
  for (int i0 = 0; i0 <= a.B; i0 += kPiece) {
    p.first = i0;
    p.n = a.B + 1 - i0 < kPiece ? a.B + 1 - i0 : kPiece;
    for (int i = 0; i < p.n; ++i) {
      const int j = i0 + i;
      p.cu[i] = a.cu[j];
      p.chunk0[i] = (int)chunks;
      p.order[i] = order.take();
      if (j < a.B) chunks += (a.cu[j + 1] - a.cu[j] + kLinrecChunk - 1) / kLinrecChunk;
    }
    seq_table_kernel<<<1, 256, 0, s>>>(p, const_cast<long long*>(tab.cu),
                                       const_cast<int*>(tab.chunk0), const_cast<int*>(tab.order));
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
    static KernelSlots known[2][3];  // with and without a write gate
    KernelSlots* k = known[p.b != nullptr];
    using Kernel = void (*)(LinrecArgs, Chains, int, LinrecMaps);
    const ChainKernel<Kernel> ks[3] = {{linrec_fwd_kernel<TX, TG, GIVEN, SCALE, TO, 1, false>,
                                        linrec_fwd_kernel<TX, TG, GIVEN, SCALE, TO, 1, true>},
                                       {linrec_fwd_kernel<TX, TG, GIVEN, SCALE, TO, 2, false>,
                                        linrec_fwd_kernel<TX, TG, GIVEN, SCALE, TO, 2, true>},
                                       {linrec_fwd_kernel<TX, TG, GIVEN, SCALE, TO, 4, false>,
                                        linrec_fwd_kernel<TX, TG, GIVEN, SCALE, TO, 4, true>}};
    Split sp;
    cudaError_t e = choose_split(p, ks, fwd_smem<TX, TG>(p.b != nullptr), fwd_smem<TX, TG>(true), k,
                                 &sp);
    if (e != cudaSuccess) return e;
    return sp.split == 4   ? launch<TX, TG, 4>(ks[2].of(sp.cs), sp.cs)
           : sp.split == 2 ? launch<TX, TG, 2>(ks[1].of(sp.cs), sp.cs)
                           : launch<TX, TG, 1>(ks[0].of(sp.cs), sp.cs);
  }
  template <typename TX, typename TG, int SPLIT, typename K>
  cudaError_t launch(K kernel, int cs) const {
    LinrecMaps maps;
    Chains c = ch;
    c.tma = map_tiles<SPLIT, TX>(&maps.x, p, p.x, p.ldx) &&
            map_tiles<SPLIT, TG>(&maps.a, p, p.a, p.lda) &&
            (!p.b || map_tiles<SPLIT, TG>(&maps.b, p, p.b, p.ldb));
    return launch_chains<SPLIT>(kernel, fwd_smem<TX, TG>(p.b != nullptr), p, c, cs, vec, s, maps);
  }
};
struct StepRun {
  const LinrecArgs& p;
  float* state;
  cudaStream_t s;
  template <typename TX, typename TG, bool GIVEN, int SCALE, bool WIDE>
  cudaError_t run() const {
    using TO = typename Wide<TX, WIDE>::type;
    const long long blocks =
        (long long)p.B * ((p.D + 4 * kStepThreads - 1) / (4 * kStepThreads));
    const bool vec = p.D % 4 == 0 && fours(p.x, p.ldx, sizeof(TX)) &&
                     fours(p.a, p.lda, sizeof(TG)) && fours(p.b, p.ldb, sizeof(TG)) &&
                     fours(p.h, p.ldh, sizeof(TO)) && fours(state, p.D, sizeof(float));
    if (vec)
      linrec_step_kernel<TX, TG, GIVEN, SCALE, TO, true>
          <<<(unsigned)blocks, kStepThreads, 0, s>>>(p, state);
    else
      linrec_step_kernel<TX, TG, GIVEN, SCALE, TO, false>
          <<<(unsigned)blocks, kStepThreads, 0, s>>>(p, state);
    return cudaGetLastError();
  }
  // rows whose pieces of 4 elements are aligned
  static bool fours(const void* q, long long ld, int es) {
    return ((reinterpret_cast<uintptr_t>(q) | (uintptr_t)(ld * es)) & (4 * es - 1)) == 0;
  }
};

}  // namespace

// Workspace: the table of a packed batch.
size_t linrec_workspace_bytes(const long long* cu, int B, int T, int D) {
  return cu ? seq_table_bytes(B) : 0;
}

cudaError_t make_chains(const LinrecArgs& a, void* workspace, cudaStream_t s, Chains* ch) {
  if (a.cu) {
    char* ws = static_cast<char*>(workspace);
    ch->tab.cu = reinterpret_cast<const long long*>(ws);
    ws += align256((size_t)(a.B + 1) * sizeof(long long));
    ch->tab.chunk0 = reinterpret_cast<const int*>(ws);
    ws += align256((size_t)(a.B + 1) * sizeof(int));
    ch->tab.order = reinterpret_cast<const int*>(ws);
    cudaError_t e = fill_seq_table(a, ch->tab, s);
    if (e != cudaSuccess) return e;
    ch->after = true;
  }
  ch->status = status_word();
  if (ch->status == nullptr) return cudaErrorUnknown;
  const WaitFault wf = wait_fault();
  ch->spin = wf.spin;
  ch->fault = wf.site;
  return cudaSuccess;
}

cudaError_t launch_linrec_scan(const LinrecArgs& a, const Chains& ch, int wide_flag,
                               cudaStream_t s) {
  const int wide = a.dtype == GDN_F32 || (a.flags & wide_flag);
  return by_type(a, wide_flag, FwdRun{a, ch, pairs(a.h, a.ldh, wide ? 4 : 2), s});
}

cudaError_t launch_linrec_fwd(const LinrecArgs& a, void* workspace, cudaStream_t s) {
  Chains ch{};
  cudaError_t e = make_chains(a, workspace, s, &ch);
  return e != cudaSuccess ? e : launch_linrec_scan(a, ch, GDN_OUT_F32, s);
}

cudaError_t launch_linrec_step(const LinrecArgs& a, float* state, cudaStream_t s) {
  return by_type(a, GDN_OUT_F32, StepRun{a, state, s});
}

}  // namespace gdn
