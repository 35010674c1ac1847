// linrec_bwd.cu -- the backward of the gated linear recurrence.  With c the gradient that
// arrives at a state from later tokens,
//   lambda_t = dh_t + c_t,  c_{t-1} = alpha_t lambda_t,
//   dx = lambda f beta,  dbeta = lambda f x,  dg = alpha lambda h_{t-1} + lambda beta x f'(g),
// c runs over the tiles from the last to the first as the forward's state does from the
// first to the last (linrec_tile.cuh).  The states h_{t-1} of a tile are recomputed in
// float32 from the state before it, which the forward kept (4 bytes for 64 elements).
//
// Two passes over a tile in shared memory.  The first forms the gates and folds both chains,
// (A, H) and (A, R); the exponents, the slopes of softplus and beta stay in registers (48 of
// the 128 that two blocks an SM leave).  The second walks the states forward and the gradients
// back, four tokens at a time: the later four start from the state that the fold of the first
// four gives.  All eight at once spilled (sqrt(1 - alpha^2), 64 x 512 x 4096: 561 against 500
// us).  dA_log and ddt_bias are summed by the lanes that hold their channels, rounding errors
// kept, and joined over the blocks in a fixed order.
//
// What bounds it: 66 instructions an element against 14 bytes of bf16, at 56% of the issue
// slots with 15 warps an SM.  Measured: 64 sequences of 512 x 4096 bf16 421 us, 4.5 TB/s;
// float32 of 512 x 2048 360 us, 5.2 TB/s; 131072 x 1024 without a write gate 461 us, 2.9 TB/s.
#include "linrec_launch.cuh"

namespace gdn {
namespace {

template <typename TX, typename TG, typename TD>
struct BwdStage {
  alignas(128) TX x[kTile];
  alignas(128) TG a[kTile];
  alignas(128) TG b[kTile];
  alignas(128) TD dh[kTile];
};
// Two stages where they leave room for two blocks on a multiprocessor, else one.
template <typename TX, typename TG, typename TD>
struct BwdSmem {
  static constexpr int kStages = sizeof(BwdStage<TX, TG, TD>) <= 48 * 1024 ? 2 : 1;
  BwdStage<TX, TG, TD> stage[kStages];
  CarrySmem carry;
  float2 start[kLinrecThreads];  // the state that enters each thread's tokens
  float2 back[kLinrecThreads];   // R of each thread's tokens: c_out = A c_in + R
  float4 sums[kLinrecThreads];
};

// sum += v with the rounding error kept in err.
__device__ __forceinline__ void add_kept(float2* sum, float2* err, float2 v) {
  const float2 minus = both(-1.f), y = fma2(*err, minus, v), t = add2(*sum, y);
  *err = fma2(y, minus, fma2(*sum, minus, t));
  *sum = t;
}

template <typename TX, typename TG, bool GIVEN, int SCALE, typename TD, typename TDG, int SPLIT,
          bool CLUSTER>
__global__ void __launch_bounds__(kLinrecThreads, 2)
linrec_bwd_kernel(LinrecArgs p, Chains ch, int vec, const __grid_constant__ LinrecMaps maps,
                  const float* states, float2* sums) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  using Smem = BwdSmem<TX, TG, TD>;
  constexpr int kStages = Smem::kStages;
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  FoldRow* folds = reinterpret_cast<FoldRow*>(smem_raw + sizeof(Smem));
  constexpr int kTileT = Shape<SPLIT>::kT, kC = Shape<SPLIT>::kC;
  constexpr int kTileChunks = kTileT / kLinrecChunk;
  const Spot<SPLIT> at;
  wait_for_launch();
  const int first = at.first;
  const Chain k = chain_of<SPLIT, CLUSTER>(p, ch);
  const int c = k.c0 + 2 * at.cl, cols = p.D - c;
  const int cs = CLUSTER ? ch.cs : 1, step = cs * kTileT;
  const int last = k.tiles - 1 - k.rank;  // the block's first tile; may be before the sequence
  const long long tok0 = k.tok + last * (long long)kTileT;
  const int tokens = (int)k.len - last * kTileT;  // from there to the sequence's end
  auto tile = [&](int round) { return last - round * cs; };
  auto length = [&](int round) {  // of the round's tile: only the sequence's last is short
    return tile(round) < 0 ? 0 : round == 0 && tokens < kTileT ? tokens : kTileT;
  };
  int late = -1;  // the round whose tiles have not come in time: no more are asked for
  auto load = [&](int round) {
    const int n = length(round), t = tile(round) * kTileT;
    BwdStage<TX, TG, TD>& st = sm.stage[round % kStages];
    if (ch.tma) {
      if (n > 0 && threadIdx.x == 0 && late < 0) {
        uint64_t* bar = &sm.carry.loaded[round % kStages];
        const int y = ch.tab.cu ? (int)k.tok + t : t, z = ch.tab.cu ? 0 : k.row;
        tc::mbar_arrive_expect_tx(bar, sizeof(st.x) + sizeof(st.a) + (p.b ? sizeof(st.b) : 0) +
                                           sizeof(st.dh));
        if (ch.fault == kFaultLinrecTiles) return;
        tma_load_3d(st.x, &maps.x, bar, k.c0, y, z);
        tma_load_3d(st.a, &maps.a, bar, k.c0, y, z);
        if (p.b) tma_load_3d(st.b, &maps.b, bar, k.c0, y, z);
        tma_load_3d(st.dh, &maps.dh, bar, k.c0, y, z);
      }
    } else {
      if (n > 0) {
        load_elements<SPLIT>(st.x, p.x, p.ldx, k.tok + t, n, k.c0, p.D);
        load_elements<SPLIT>(st.a, p.a, p.lda, k.tok + t, n, k.c0, p.D);
        if (p.b) load_elements<SPLIT>(st.b, p.b, p.ldb, k.tok + t, n, k.c0, p.D);
        load_elements<SPLIT>(st.dh, p.dh, p.lddh, k.tok + t, n, k.c0, p.D);
      }
      cp_async_commit();
    }
  };
  carry_begin<CLUSTER>(sm.carry);
  load(0);
  GateConst gc{both(0.f), both(0.f)};
  if (!GIVEN) gc = gate_const(p.A_log, p.dt_bias, c, p.D);
  float2 carry = read2(p.dht, k.row, c, p.D);  // behind the round's last tile (warp 0's)
  bool lost = false;
  auto state = [&](int tt) {  // before the lane's chunk of a tile
    const int j = tt * kTileChunks + at.part;
    return tt >= 0 && j < k.chunks ? read2(states, k.chunk0 + j, c, p.D) : both(0.f);
  };
  float2 hnext = both(0.f);
  if (at.warp == 1) hnext = state(last);
  float2 sA = both(0.f), eA = both(0.f), sb = both(0.f), eb = both(0.f);
  Rows<TD> odx;
  Rows<TDG> oda, odb;
  odx.begin(p.dx, p.lddx, tok0, k.c0, first, 2 * at.cl);
  oda.begin(p.da, p.ldda, tok0, k.c0, first, 2 * at.cl);
  odb.begin(p.db, p.lddb, tok0, k.c0, first, 2 * at.cl);
  constexpr bool alone = SPLIT == 1 && !CLUSTER;  // what enters a tile is known before it is folded
  const int rounds = (k.tiles + cs - 1) / cs;
  for (int round = 0; round < rounds; ++round) {
    const int tt = tile(round), n = length(round);
    if (!ch.tma) {
      cp_async_wait<0>();
    } else if (n > 0 && late < 0 &&
               !tc::mbar_wait(&sm.carry.loaded[round % kStages], (round / kStages) & 1, nullptr,
                              0, ch.spin)) {
      report_timeout(ch.status, 0x4c54);
      late = round;
    }
    __syncthreads();  // the stage is complete, the other one free
    if (kStages > 1 && round + 1 < rounds) load(round + 1);
    // The next tile's state is on its way during both passes, or where the carry needs its
    // registers (128K tokens in clusters: spills, 516 against 455 us) during the second.
    float2 hs = hnext;  // warp 1's
    if (alone && at.warp == 1) hnext = state(tt - cs);
    BwdStage<TX, TG, TD>& st = sm.stage[round % kStages];
    if (n > 0 && n < kTileT && ch.tab.cu) {  // the next sequence's tokens
      clear_rows<SPLIT>(st.x, n);
      tc::fence_proxy_async_smem();  // the stage's next tiles come by TMA
      __syncthreads();
    }
    const int mine = at.mine();
    float2 e[kPer], slope[kPer], be[kPer];
    float2 Am, Hm;  // of the first kGroup tokens
    {
      float2 al[kPer], A = both(1.f), H = both(0.f), R = both(0.f);
#pragma unroll
      for (int i0 = 0; i0 < kPer; i0 += kGroup) {
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          e[i0 + i] = get2(st.a + mine + (i0 + i) * kC);
          be[i0 + i] = p.b ? get2(st.b + mine + (i0 + i) * kC) : both(1.f);
        }
        if (GIVEN) decay_exponents<true, kGroup>(e + i0, gc);
        else decay_exponents_slope<kGroup>(e + i0, gc, slope + i0);
        if (p.b) write_gates<GIVEN, kGroup>(be + i0);
      }
      if (n < kTileT) {  // behind the sequence: both states pass through
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (first + i >= n) e[i] = be[i] = both(0.f);
      }
#pragma unroll
      for (int i0 = 0; i0 < kPer; i0 += kGroup) {
        float2 f[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) al[i0 + i] = ex2_2(e[i0 + i]);
        if (SCALE != kScaleNone) input_scales<SCALE, kGroup>(e + i0, al + i0, f);
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          float2 u = mul2(get2(st.x + mine + (i0 + i) * kC), be[i0 + i]);
          if (SCALE != kScaleNone) u = mul2(u, f[i]);
          H = fma2(al[i0 + i], H, u);
          A = mul2(A, al[i0 + i]);
        }
        if (i0 == 0) {
          Am = A;
          Hm = H;
        }
      }
      // lambda from token to token, R = alpha lambda of the first.  dh + alpha lambda is written as
      // the fma that the compiler makes of it in some of these loops and not in others: the
      // gradients' last bits would go by the loop, that is by the tile's shape.
      if (n == kTileT) {
        R = get2(st.dh + mine + (kPer - 1) * kC);
#pragma unroll
        for (int i = kPer - 2; i >= 0; --i)
          R = fma2(al[i + 1], R, get2(st.dh + mine + i * kC));
      } else {
#pragma unroll
        for (int i = kPer - 1; i >= 0; --i) {
          const float2 dh = first + i < n ? get2(st.dh + mine + i * kC) : both(0.f);
          R = i == kPer - 1 ? dh : fma2(al[i + 1], R, dh);
        }
      }
      R = mul2(al[0], R);
      sm.carry.fold[threadIdx.x] = join4(A, H);
      sm.back[threadIdx.x] = R;
    }
    __syncthreads();
    if (at.warp == 1) {  // the state through the lane's chunk
      if (!alone) hnext = state(tt - cs);
#pragma unroll 4
      for (int w = 0; w < 8; ++w) {
        sm.start[at.group(w)] = hs;
        const float4 q = sm.carry.fold[at.group(w)];
        hs = fma2(first2(q), hs, last2(q));
      }
    } else if (at.warp == 0) {  // its gradient
      float2 v = carry, A = both(1.f), R = both(0.f);
      if (!alone)
        v = carry_round<SPLIT, CLUSTER, true>(
            ch, k.rank, round, chunk_fold<SPLIT, true>(at, sm.carry, sm.back), sm.carry, folds,
            &carry, &lost);
#pragma unroll 4
      for (int w = 7; w >= 0; --w) {
        const float2 r = sm.back[at.group(w)], a = first2(sm.carry.fold[at.group(w)]);
        sm.back[at.group(w)] = v;
        v = fma2(a, v, r);
        R = fma2(a, R, r);
        A = mul2(A, a);
      }
      // what leaves the tile, as it is formed elsewhere: from the chunk's own (A, R)
      if (alone) carry = fma2(A, carry, R);
    }
    __syncthreads();
    hs = sm.start[threadIdx.x];
    // lambda, and alpha, of the token behind (of none: what arrives from there)
    float2 lam = sm.back[threadIdx.x], behind = both(1.f);
    float2 tA = both(0.f), tb = both(0.f);
    // The later group of tokens first; its states from the one in front of it.
#pragma unroll
    for (int i0 = kPer - kGroup; i0 >= 0; i0 -= kGroup) {
      float2 al[kGroup], f[kGroup], hp[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) al[i] = ex2_2(e[i0 + i]);
      if (SCALE != kScaleNone) input_scales<SCALE, kGroup>(e + i0, al, f);
      hp[0] = i0 == 0 ? hs : fma2(Am, hs, Hm);
#pragma unroll
      for (int i = 0; i + 1 < kGroup; ++i) {
        float2 u = mul2(get2(st.x + mine + (i0 + i) * kC), be[i0 + i]);
        if (SCALE != kScaleNone) u = mul2(u, f[i]);
        hp[i + 1] = fma2(al[i], hp[i], u);
      }
      auto token = [&](int j, float2* dx, float2* da, float2* db) {
        const int i = i0 + j, el = mine + i * kC;
        lam = fma2(behind, lam, get2(st.dh + el));
        behind = al[j];
        const float2 cc = mul2(al[j], lam);
        const float2 lx = mul2(lam, get2(st.x + el));
        float2 dg = mul2(cc, hp[j]);
        *dx = mul2(lam, be[i]);
        *db = lx;
        if (SCALE != kScaleNone) {
          const float2 q = make_float2(input_scale_slope<SCALE>(al[j].x, f[j].x),
                                       input_scale_slope<SCALE>(al[j].y, f[j].y));
          dg = fma2(mul2(lx, be[i]), q, dg);
          *dx = mul2(*dx, f[j]);
          *db = mul2(*db, f[j]);
        }
        *da = dg;
        if (!GIVEN) {
          if (p.b) *db = mul2(mul2(*db, be[i]), write_gate_rest(get2(st.b + el), be[i]));
          *da = mul2(dg, slope[i]);
          tb = fma2(dg, slope[i], tb);
          // dg log2(e) times e, which is -inf where alpha = 0
          tA = fma2(dg, make_float2(fmaxf(e[i].x, -3e38f), fmaxf(e[i].y, -3e38f)), tA);
        }
      };
      float2 dx, da, db;
      if (n == kTileT && cols > 1 && vec) {
#pragma unroll
        for (int j = kGroup - 1; j >= 0; --j) {
          token(j, &dx, &da, &db);
          put2(odx.at(i0 + j), dx);
          put2(oda.at(i0 + j), da);
          if (p.b) put2(odb.at(i0 + j), db);
        }
      } else {
#pragma unroll
        for (int j = kGroup - 1; j >= 0; --j) {
          if (first + i0 + j >= n) continue;
          token(j, &dx, &da, &db);
          put2(odx.at(i0 + j), dx, cols);
          put2(oda.at(i0 + j), da, cols);
          if (p.b) put2(odb.at(i0 + j), db, cols);
        }
      }
    }
    if (at.warp == 0) carry_rest<SPLIT, CLUSTER, true>(ch, k.rank, round, folds, &carry);
    odx.advance(-step);
    oda.advance(-step);
    odb.advance(-step);
    if (!GIVEN) {  // a lane keeps its channels: their sums run through the rounds
      add_kept(&sA, &eA, tA);
      add_kept(&sb, &eb, tb);
    }
    if (kStages == 1 && round + 1 < rounds) {
      __syncthreads();  // the stage is read
      load(round + 1);
    }
  }
  if (!GIVEN) {
    sm.sums[threadIdx.x] = join4(mul2(sA, both(kLn2)), sb);
    __syncthreads();
    if (at.warp == 0 && at.part == 0) {
      float2 vA = both(0.f), vb = both(0.f);
      for (int i = at.cl; i < kLinrecThreads; i += Shape<SPLIT>::kLanes) {
        const float4 q = sm.sums[i];
        vA = add2(vA, first2(q));
        vb = add2(vb, last2(q));
      }
      if (sums == nullptr) {  // the only block of its channels
        write2(p.dA_log, 0, c, p.D, vA);
        write2(p.ddt_bias, 0, c, p.D, vb);
      } else {
        float2* to = sums + ((long long)k.row * cs + k.rank) * p.D + c;
        if (cols > 0) to[0] = make_float2(vA.x, vb.x);
        if (cols > 1) to[1] = make_float2(vA.y, vb.y);
      }
    }
  }
  // no copy is to be on its way when the block leaves: once more, with a limit
  if (late >= 0 && threadIdx.x == 0)
    tc::mbar_wait(&sm.carry.loaded[late % kStages], (late / kStages) & 1, nullptr, 0, 1u << 20);
  carry_end<CLUSTER>();
  // dh0 may be dht, which every block of the cluster has read by now
  if (k.rank == 0 && at.warp == 0 && at.part == 0) write2(p.dh0, k.row, c, p.D, carry);
}

// dA_log and ddt_bias: a channel's sums of all blocks, in a fixed order (32 rows of threads,
// each every 32nd block), in 64 bits.
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows)
linrec_sums_kernel(const float2* sums, long long rows, int D, float* dA_log, float* ddt_bias) {
  __shared__ double2 part[kSumRows][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  double A = 0.0, b = 0.0;
  wait_for_launch();
  if (c < D)
    for (long long r = threadIdx.y; r < rows; r += kSumRows) {
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
  const Chains& ch;
  const float* states;
  float2* sums;
  cudaStream_t s;
  template <typename TX, typename TG, bool GIVEN, int SCALE, bool WIDE>
  cudaError_t run() const {
    using TD = typename Wide<TX, WIDE>::type;
    using TDG = typename Wide<TD, GIVEN>::type;
    static KernelSlots known[3];
    using Kernel = void (*)(LinrecArgs, Chains, int, LinrecMaps, const float*, float2*);
    const ChainKernel<Kernel> ks[3] = {
        {linrec_bwd_kernel<TX, TG, GIVEN, SCALE, TD, TDG, 1, false>,
         linrec_bwd_kernel<TX, TG, GIVEN, SCALE, TD, TDG, 1, true>},
        {linrec_bwd_kernel<TX, TG, GIVEN, SCALE, TD, TDG, 2, false>,
         linrec_bwd_kernel<TX, TG, GIVEN, SCALE, TD, TDG, 2, true>},
        {linrec_bwd_kernel<TX, TG, GIVEN, SCALE, TD, TDG, 4, false>,
         linrec_bwd_kernel<TX, TG, GIVEN, SCALE, TD, TDG, 4, true>}};
    Split sp;
    constexpr size_t smem = sizeof(BwdSmem<TX, TG, TD>);
    cudaError_t e = choose_split(p, ks, smem, smem, known, &sp);
    if (e != cudaSuccess) return e;
    return sp.split == 4   ? launch<TX, TG, GIVEN, TD, TDG, 4>(ks[2].of(sp.cs), sp.cs)
           : sp.split == 2 ? launch<TX, TG, GIVEN, TD, TDG, 2>(ks[1].of(sp.cs), sp.cs)
                           : launch<TX, TG, GIVEN, TD, TDG, 1>(ks[0].of(sp.cs), sp.cs);
  }
  template <typename TX, typename TG, bool GIVEN, typename TD, typename TDG, int SPLIT, typename K>
  cudaError_t launch(K kernel, int cs) const {
    LinrecMaps maps;
    Chains c = ch;
    c.tma = map_tiles<SPLIT, TX>(&maps.x, p, p.x, p.ldx) &&
            map_tiles<SPLIT, TG>(&maps.a, p, p.a, p.lda) &&
            (!p.b || map_tiles<SPLIT, TG>(&maps.b, p, p.b, p.ldb)) &&
            map_tiles<SPLIT, TD>(&maps.dh, p, p.dh, p.lddh);
    const bool alone = p.B == 1 && cs == 1;  // one block a channel: no sums to join
    const int vec = pairs(p.dx, p.lddx, sizeof(TD)) && pairs(p.da, p.ldda, sizeof(TDG)) &&
                    pairs(p.db, p.lddb, sizeof(TDG));
    cudaError_t e = launch_chains<SPLIT>(kernel, sizeof(BwdSmem<TX, TG, TD>), p, c, cs, vec, s,
                                         maps, states, alone ? nullptr : sums);
    if (e != cudaSuccess || GIVEN || alone) return e;
    return launch_after(linrec_sums_kernel, dim3((p.D + 31) / 32), dim3(32, kSumRows), s, sums,
                        (long long)p.B * cs, p.D, p.dA_log, p.ddt_bias);
  }
};

size_t states_bytes(const LinrecArgs& a) {
  return align256((size_t)linrec_chunks(a.cu, a.B, a.T) * a.D * sizeof(float));
}

}  // namespace

// Workspace: the table of a packed batch; the states, where the call does not pass the
// forward's; the blocks' sums of the gate parameters' gradients.
size_t linrec_bwd_workspace_bytes(const long long* cu, int B, int T, int D, bool states_given,
                                  int flags) {
  LinrecArgs a{};
  a.cu = cu; a.B = B; a.T = T; a.D = D;
  return (cu ? seq_table_bytes(B) : 0) + (states_given ? 0 : states_bytes(a)) +
         (flags & GDN_GATES_PRECOMPUTED
              ? 0
              : align256((size_t)B * most_blocks(a) * D * sizeof(float2)));
}

cudaError_t launch_linrec_bwd(const LinrecArgs& a, void* workspace, cudaStream_t s) {
  char* ws = static_cast<char*>(workspace);
  Chains ch{};
  cudaError_t e = make_chains(a, ws, s, &ch);
  if (e != cudaSuccess) return e;
  if (a.cu) ws += seq_table_bytes(a.B);
  const float* states = a.states;
  if (states == nullptr) {
    LinrecArgs f = a;
    f.states_out = reinterpret_cast<float*>(ws);
    ws += states_bytes(a);
    e = launch_linrec_scan(f, ch, GDN_GRAD_F32, s);
    if (e != cudaSuccess) return e;
    states = f.states_out;
    ch.after = true;
  }
  return by_type(a, GDN_GRAD_F32, BwdRun{a, ch, states, reinterpret_cast<float2*>(ws), s});
}

}  // namespace gdn
