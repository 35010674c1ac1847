// linrec.cu -- the gated linear recurrence, per channel
//   h_t = alpha_t h_{t-1} + f(alpha_t) beta_t x_t
// (linrec_math.cuh for the gates), over dense or packed batches, its backward and its
// one-token step.  One thread per (sequence, channel) walks the tokens in order.
#include "linrec.cuh"
#include "linrec_math.cuh"

namespace gdn {

long long linrec_chunks(const long long* cu, int B, int T) {
  if (cu == nullptr) return B * (((long long)T + kLinrecChunk - 1) / kLinrecChunk);
  long long n = 0;
  for (int i = 0; i < B; ++i) n += (cu[i + 1] - cu[i] + kLinrecChunk - 1) / kLinrecChunk;
  return n;
}

namespace {

constexpr int kT = 128;

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Packed batches: each sequence's first token and first chunk, entry B the totals.
struct SeqTab {
  const long long* cu;
  const int* chunk0;
};
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
size_t seq_table_bytes(int B) {
  return align256((size_t)(B + 1) * sizeof(long long)) + align256((size_t)(B + 1) * sizeof(int));
}
cudaError_t fill_seq_table(const long long* cu, int B, void* at, SeqTab* tab, cudaStream_t s) {
  long long* dcu = static_cast<long long*>(at);
  int* dch = reinterpret_cast<int*>(static_cast<char*>(at) +
                                    align256((size_t)(B + 1) * sizeof(long long)));
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
    seq_table_kernel<<<1, 256, 0, s>>>(p, dcu, dch);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  tab->cu = dcu;
  tab->chunk0 = dch;
  return cudaSuccess;
}

template <typename TX, typename TG, bool GIVEN, int SCALE, typename TO>
__global__ void __launch_bounds__(kT)
linrec_fwd_kernel(LinrecArgs p, SeqTab tab, float* states) {
  const int c = blockIdx.x * kT + threadIdx.x, r = blockIdx.y;
  if (c >= p.D) return;
  const bool packed = tab.cu != nullptr;
  const long long t0 = packed ? tab.cu[r] : (long long)r * p.T;
  const int n = packed ? (int)(tab.cu[r + 1] - t0) : p.T;
  const long long chunk0 =
      packed ? tab.chunk0[r] : (long long)r * ((p.T + kLinrecChunk - 1) / kLinrecChunk);
  const TX* x = static_cast<const TX*>(p.x) + t0 * p.ldx + c;
  const TG* a = static_cast<const TG*>(p.a) + t0 * p.lda + c;
  const TG* b = p.b ? static_cast<const TG*>(p.b) + t0 * p.ldb + c : nullptr;
  TO* h = p.h ? static_cast<TO*>(p.h) + t0 * p.ldh + c : nullptr;
  const GateConst k = GIVEN ? GateConst{0.f, 0.f} : gate_const(p.A_log, p.dt_bias, c);
  float st = p.h0 ? p.h0[(size_t)r * p.D + c] : 0.f;
  for (int t = 0; t < n; ++t) {
    if (states != nullptr && t % kLinrecChunk == 0)
      states[(chunk0 + t / kLinrecChunk) * p.D + c] = st;
    const float g = log_decay<GIVEN>(to_f32(a[t * p.lda]), k);
    float u = to_f32(x[t * p.ldx]) * input_scale<SCALE>(g);
    if (b) u *= write_gate<GIVEN>(to_f32(b[t * p.ldb]));
    st = fmaf(ex2_f(g * kLog2e), st, u);
    if (h) h[t * p.ldh] = from_f32<TO>(st);
  }
  if (p.ht) p.ht[(size_t)r * p.D + c] = st;
}

template <typename TX, typename TG, bool GIVEN, int SCALE, typename TD, typename TDG>
__global__ void __launch_bounds__(kT)
linrec_bwd_kernel(LinrecArgs p, SeqTab tab, const float* states, float2* sums) {
  const int c = blockIdx.x * kT + threadIdx.x, r = blockIdx.y;
  if (c >= p.D) return;
  const bool packed = tab.cu != nullptr;
  const long long t0 = packed ? tab.cu[r] : (long long)r * p.T;
  const int n = packed ? (int)(tab.cu[r + 1] - t0) : p.T;
  const long long chunk0 =
      packed ? tab.chunk0[r] : (long long)r * ((p.T + kLinrecChunk - 1) / kLinrecChunk);
  const TX* x = static_cast<const TX*>(p.x) + t0 * p.ldx + c;
  const TG* a = static_cast<const TG*>(p.a) + t0 * p.lda + c;
  const TG* b = p.b ? static_cast<const TG*>(p.b) + t0 * p.ldb + c : nullptr;
  const TD* dh = static_cast<const TD*>(p.dh) + t0 * p.lddh + c;
  TD* dx = static_cast<TD*>(p.dx) + t0 * p.lddx + c;
  TDG* da = static_cast<TDG*>(p.da) + t0 * p.ldda + c;
  TDG* db = b ? static_cast<TDG*>(p.db) + t0 * p.lddb + c : nullptr;
  const GateConst k = GIVEN ? GateConst{0.f, 0.f} : gate_const(p.A_log, p.dt_bias, c);
  float carry = p.dht ? p.dht[(size_t)r * p.D + c] : 0.f;
  double sum_A = 0.0, sum_b = 0.0;
  float prev[kLinrecChunk];
  for (int j = (n + kLinrecChunk - 1) / kLinrecChunk - 1; j >= 0; --j) {
    const int lo = j * kLinrecChunk, m = n - lo < kLinrecChunk ? n - lo : kLinrecChunk;
    float st = states[(chunk0 + j) * p.D + c];
    for (int i = 0; i < m; ++i) {
      prev[i] = st;
      const float g = log_decay<GIVEN>(to_f32(a[(lo + i) * p.lda]), k);
      float u = to_f32(x[(lo + i) * p.ldx]) * input_scale<SCALE>(g);
      if (b) u *= write_gate<GIVEN>(to_f32(b[(lo + i) * p.ldb]));
      st = fmaf(ex2_f(g * kLog2e), st, u);
    }
    for (int i = m - 1; i >= 0; --i) {
      const int t = lo + i;
      const float av = to_f32(a[t * p.lda]), xv = to_f32(x[t * p.ldx]);
      const float g = log_decay<GIVEN>(av, k), alpha = ex2_f(g * kLog2e);
      const float f = input_scale<SCALE>(g);
      const float beta = b ? write_gate<GIVEN>(to_f32(b[t * p.ldb])) : 1.f;
      const float lam = to_f32(dh[t * p.lddh]) + carry;
      carry = alpha * lam;
      const float dg = fmaf(carry, prev[i], lam * xv * beta * input_scale_slope<SCALE>(alpha, f));
      dx[t * p.lddx] = from_f32<TD>(lam * f * beta);
      if (b) {
        const float dbeta = lam * f * xv;
        db[t * p.lddb] =
            from_f32<TDG>(GIVEN ? dbeta : dbeta * beta * sigmoid_sfu(-to_f32(b[t * p.ldb])));
      }
      if (GIVEN) {
        da[t * p.ldda] = from_f32<TDG>(dg);
      } else {
        const float dz = dg * k.neg_A * sigmoid_sfu(av + k.bias);
        da[t * p.ldda] = from_f32<TDG>(dz);
        sum_b += dz;
        sum_A += dg == 0.f ? 0.f : dg * g;  // g = -inf where alpha = 0
      }
    }
  }
  if (p.dh0) p.dh0[(size_t)r * p.D + c] = carry;
  if (!GIVEN) sums[(size_t)r * p.D + c] = make_float2((float)sum_A, (float)sum_b);
}

__global__ void linrec_sums_kernel(const float2* sums, long long rows, int D, float* dA_log,
                                   float* ddt_bias) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= D) return;
  double A = 0.0, b = 0.0;
  for (long long r = 0; r < rows; ++r) {
    const float2 v = sums[r * D + c];
    A += v.x;
    b += v.y;
  }
  dA_log[c] = (float)A;
  ddt_bias[c] = (float)b;
}

template <typename TX, typename TG, bool GIVEN, int SCALE, typename TO>
__global__ void __launch_bounds__(kT) linrec_step_kernel(LinrecArgs p, float* state) {
  const int c = blockIdx.x * kT + threadIdx.x;
  const long long r = blockIdx.y;
  if (c >= p.D) return;
  const GateConst k = GIVEN ? GateConst{0.f, 0.f} : gate_const(p.A_log, p.dt_bias, c);
  const float g = log_decay<GIVEN>(to_f32(static_cast<const TG*>(p.a)[r * p.lda + c]), k);
  float u = to_f32(static_cast<const TX*>(p.x)[r * p.ldx + c]) * input_scale<SCALE>(g);
  if (p.b) u *= write_gate<GIVEN>(to_f32(static_cast<const TG*>(p.b)[r * p.ldb + c]));
  const float st = fmaf(ex2_f(g * kLog2e), state[r * p.D + c], u);
  state[r * p.D + c] = st;
  static_cast<TO*>(p.h)[r * p.ldh + c] = from_f32<TO>(st);
}

// Calls f.template run<TX, TG, GIVEN, SCALE, wide>() for the call's types: x in TX, the
// gates in TG, `wide`: the outputs (forward) or gradients (backward) in float32.
template <typename F, typename TX, typename TG, bool GIVEN, bool WIDE>
cudaError_t by_scale(const LinrecArgs& p, F f) {
  if (p.flags & GDN_LINREC_TIED) return f.template run<TX, TG, GIVEN, kScaleTied, WIDE>();
  if (p.flags & GDN_LINREC_UNIT) return f.template run<TX, TG, GIVEN, kScaleUnit, WIDE>();
  return f.template run<TX, TG, GIVEN, kScaleNone, WIDE>();
}
template <typename F>
cudaError_t by_type(const LinrecArgs& p, int wide_flag, F f) {
  using bf16 = __nv_bfloat16;
  const bool given = p.flags & GDN_GATES_PRECOMPUTED;
  if (p.dtype == GDN_F32)
    return given ? by_scale<F, float, float, true, true>(p, f)
                 : by_scale<F, float, float, false, true>(p, f);
  if (p.flags & wide_flag)
    return given ? by_scale<F, bf16, float, true, true>(p, f)
                 : by_scale<F, bf16, bf16, false, true>(p, f);
  return given ? by_scale<F, bf16, float, true, false>(p, f)
               : by_scale<F, bf16, bf16, false, false>(p, f);
}
template <typename TX, bool WIDE> struct Wide { using type = TX; };
template <typename TX> struct Wide<TX, true> { using type = float; };

struct FwdRun {
  const LinrecArgs& p;
  SeqTab tab;
  float* states;
  cudaStream_t s;
  template <typename TX, typename TG, bool GIVEN, int SCALE, bool WIDE>
  cudaError_t run() {
    linrec_fwd_kernel<TX, TG, GIVEN, SCALE, typename Wide<TX, WIDE>::type>
        <<<dim3((p.D + kT - 1) / kT, p.B), kT, 0, s>>>(p, tab, states);
    return cudaGetLastError();
  }
};
struct BwdRun {
  const LinrecArgs& p;
  SeqTab tab;
  const float* states;
  float2* sums;
  cudaStream_t s;
  template <typename TX, typename TG, bool GIVEN, int SCALE, bool WIDE>
  cudaError_t run() {
    using TD = typename Wide<TX, WIDE>::type;
    linrec_bwd_kernel<TX, TG, GIVEN, SCALE, TD, typename Wide<TD, GIVEN>::type>
        <<<dim3((p.D + kT - 1) / kT, p.B), kT, 0, s>>>(p, tab, states, sums);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || GIVEN) return e;
    linrec_sums_kernel<<<(p.D + 127) / 128, 128, 0, s>>>(sums, p.B, p.D, p.dA_log, p.ddt_bias);
    return cudaGetLastError();
  }
};
struct StepRun {
  const LinrecArgs& p;
  float* state;
  cudaStream_t s;
  template <typename TX, typename TG, bool GIVEN, int SCALE, bool WIDE>
  cudaError_t run() {
    linrec_step_kernel<TX, TG, GIVEN, SCALE, typename Wide<TX, WIDE>::type>
        <<<dim3((p.D + kT - 1) / kT, p.B), kT, 0, s>>>(p, state);
    return cudaGetLastError();
  }
};

}  // namespace

size_t linrec_workspace_bytes(const long long* cu, int B, int T, int D) {
  return cu ? seq_table_bytes(B) : 0;
}
size_t linrec_bwd_workspace_bytes(const long long* cu, int B, int T, int D, bool states_given,
                                  int flags) {
  size_t n = cu ? seq_table_bytes(B) : 0;
  if (!states_given) n += align256((size_t)linrec_chunks(cu, B, T) * D * sizeof(float));
  if (!(flags & GDN_GATES_PRECOMPUTED)) n += align256((size_t)B * D * sizeof(float2));
  return n;
}

cudaError_t launch_linrec_fwd(const LinrecArgs& a, void* workspace, cudaStream_t s) {
  SeqTab tab{nullptr, nullptr};
  if (a.cu) {
    cudaError_t e = fill_seq_table(a.cu, a.B, workspace, &tab, s);
    if (e != cudaSuccess) return e;
  }
  return by_type(a, GDN_OUT_F32, FwdRun{a, tab, a.states_out, s});
}

cudaError_t launch_linrec_bwd(const LinrecArgs& a, void* workspace, cudaStream_t s) {
  SeqTab tab{nullptr, nullptr};
  char* ws = static_cast<char*>(workspace);
  if (a.cu) {
    cudaError_t e = fill_seq_table(a.cu, a.B, ws, &tab, s);
    if (e != cudaSuccess) return e;
    ws += seq_table_bytes(a.B);
  }
  const float* states = a.states;
  if (states == nullptr) {
    float* own = reinterpret_cast<float*>(ws);
    ws += align256((size_t)linrec_chunks(a.cu, a.B, a.T) * a.D * sizeof(float));
    LinrecArgs f = a;
    f.h = nullptr;
    f.ht = nullptr;
    cudaError_t e = by_type(f, GDN_GRAD_F32, FwdRun{f, tab, own, s});
    if (e != cudaSuccess) return e;
    states = own;
  }
  return by_type(a, GDN_GRAD_F32,
                 BwdRun{a, tab, states, reinterpret_cast<float2*>(ws), s});
}

cudaError_t launch_linrec_step(const LinrecArgs& a, float* state, cudaStream_t s) {
  return by_type(a, GDN_OUT_F32, StepRun{a, state, s});
}

}  // namespace gdn
