// ttt_delta.cu -- gated delta rule (linear fast weight trained on the squared
// binding loss), float32 on CUDA cores: every type and every dim up to 128,
// the single-token form, and the backward pass of these.
//
//   a_t = exp(g_t);  e_t = v_t - a_t S^T k_t;  S <- a_t S + beta_t k_t e_t^T;  o_t = scale S^T q_t
//
// The value columns of S never mix, so a column of S and its entry of e, v
// and o live in 8 neighbouring lanes (up to 16 rows each, in registers) for
// the whole sequence, and a CTA of 16 columns needs no other CTA.  Tokens go
// four at a time: with s the state before them, A_t the product of the decays
// up to t and R_ti that of the decays behind i up to t,
//   u_t = beta_t (v_t - A_t k_t.s - sum_{i<t} R_ti (k_t.k_i) u_i)
//   o_t = scale (A_t q_t.s + sum_{i<=t} R_ti (q_t.k_i) u_i),  s <- A_3 s + sum_i R_3i k_i u_i
// so one reduction over the lanes serves eight dot products, and the products
// of tokens with one another are shared by the CTA's columns.  Bound by the
// latency of that chain; the chunked tensor-core kernels (delta_umma.cu) take
// the sizes where it matters.
#include <algorithm>
#include <type_traits>

#include "kernels.h"

namespace ttt {

namespace {

constexpr int L = 8;            // lanes of one column
constexpr int COLS = 16;        // columns of a CTA
constexpr int THREADS = L * COLS;
constexpr int TT = 32;          // tokens staged at a time, and between kept states
constexpr int NB = TT / 4;      // blocks of four tokens
constexpr int DMAX = 128;

TTT_DEVICE_INLINE float to_f(float x) { return x; }
TTT_DEVICE_INLINE float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
TTT_DEVICE_INLINE T from_f(float x) {
  if constexpr (std::is_same<T, float>::value) return x;
  else return __float2bfloat16_rn(x);
}

// This thread's rows 4 (lane + 8 i) + 0..3, i < R4, of a column of a [dk][dv] matrix.
template <int R4>
struct Column {
  int l, c, dk, dv;
  bool live;
  TTT_DEVICE_INLINE int row(int i, int j) const { return 4 * (l + L * i) + j; }
  TTT_DEVICE_INLINE void load(const float* S, float (&s)[4 * R4]) const {
#pragma unroll
    for (int i = 0; i < R4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[4 * i + j] = (live && row(i, j) < dk) ? S[(size_t)row(i, j) * dv + c] : 0.f;
  }
  TTT_DEVICE_INLINE void store(float* S, const float (&s)[4 * R4]) const {
#pragma unroll
    for (int i = 0; i < R4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (live && row(i, j) < dk) S[(size_t)row(i, j) * dv + c] = s[4 * i + j];
  }
};

// Tokens [t0, t0 + TT) as zero-padded float rows (k, q), the CTA's columns of
// a value tensor (w), the gates, and the coefficients of every block of four
// tokens; rows 4 floats longer than the dims, so that a column of rows lies in
// different banks.
template <int R4>
struct Stage {
  static constexpr int PITCH = 32 * R4 + 4;
  float k[TT][PITCH], q[TT][PITCH], w[TT][COLS], a[TT], b[TT];
  float A[TT], R[TT];            // A_t, R_3t
  float kk[TT][4], qk[TT][4];    // R_ti k_t.k_i (i < t), R_ti q_t.k_i (i <= t); else 0
  float os[TT][COLS];
};

// The next tile's tokens wait in registers while this one is worked on.
template <typename Tin, int R4>
struct Fetch {
  static constexpr int NX = TT * 32 * R4 / THREADS, NW = TT * COLS / THREADS;
  Tin k[NX], q[NX], w[NW], g, b;
  int t0;
  TTT_DEVICE_INLINE void load(const Tin* kp, const Tin* qp, const Tin* wp, const Tin* gp, const Tin* bp,
                              size_t bh, int t0_, int N, int dk, int dv, int c0, int tid) {
    t0 = t0_;
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int e = i * THREADS + tid, t = t0 + e / (32 * R4), r = e % (32 * R4);
      const bool in = t >= 0 && t < N && r < dk;
      const size_t at = (bh * N + t) * dk + r;
      k[i] = in ? kp[at] : from_f<Tin>(0.f);
      q[i] = in && qp != nullptr ? qp[at] : from_f<Tin>(0.f);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int e = i * THREADS + tid, t = t0 + e / COLS, c = c0 + e % COLS;
      w[i] = t >= 0 && t < N && c < dv ? wp[(bh * N + t) * dv + c] : from_f<Tin>(0.f);
    }
    g = b = from_f<Tin>(0.f);   // no decay, no step: a padding token
    const int t = t0 + tid;
    if (tid < TT && t >= 0 && t < N) {
      if (gp != nullptr) g = gp[bh * N + t];
      b = bp[bh * N + t];
    }
  }
  TTT_DEVICE_INLINE void put(Stage<R4>& st, float wscale, int tid) const {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int e = i * THREADS + tid;
      st.k[e / (32 * R4)][e % (32 * R4)] = to_f(k[i]);
      st.q[e / (32 * R4)][e % (32 * R4)] = to_f(q[i]);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) (&st.w[0][0])[i * THREADS + tid] = wscale * to_f(w[i]);
    if (tid < TT) {
      st.a[tid] = expf(to_f(g));
      st.b[tid] = to_f(b);
    }
  }
};

// Coefficients of the staged tokens: thread 16 b + d takes one of the 16
// products within block b.
template <int R4>
TTT_DEVICE_INLINE void coefficients(Stage<R4>& st, int tid) {
  const int base = tid / 16 * 4, d = tid % 16;
  // d: 0..9 q.k with (t, i) in lower-triangle order, 10..15 k.k below the diagonal
  constexpr unsigned long long TS = 0x3332213333222110ull, IS = 0x2101003210210100ull;
  const int t = (int)(TS >> (4 * d) & 15), i = (int)(IS >> (4 * d) & 15);
  const float* x = d < 10 ? st.q[base + t] : st.k[base + t];
  const float* y = st.k[base + i];
  float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
  for (int r = 0; r < 32 * R4; r += 4) {
    const float4 u = *reinterpret_cast<const float4*>(x + r), v = *reinterpret_cast<const float4*>(y + r);
    a0 = fmaf(u.x, v.x, a0);
    a1 = fmaf(u.y, v.y, a1);
    a2 = fmaf(u.z, v.z, a2);
    a3 = fmaf(u.w, v.w, a3);
  }
  float f = (a0 + a1) + (a2 + a3);
  for (int m = i + 1; m <= t; ++m) f *= st.a[base + m];
  if (d < 10) st.qk[base + t][i] = f;
  else st.kk[base + t][i] = f;
  if (tid < TT) {
    const int b0 = tid & ~3;
    float A = 1.f, R = 1.f;
    for (int m = b0; m < b0 + 4; ++m) {
      if (m <= tid) A *= st.a[m];
      else R *= st.a[m];
    }
    st.A[tid] = A;
    st.R[tid] = R;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (m > (tid & 3)) st.qk[tid][m] = 0.f;
      if (m >= (tid & 3)) st.kk[tid][m] = 0.f;
    }
  }
}

template <int R4>
TTT_DEVICE_INLINE void load_rows(const float* row, int l, float (&x)[4 * R4]) {
#pragma unroll
  for (int i = 0; i < R4; ++i) {
    const float4 t = *reinterpret_cast<const float4*>(row + 4 * (l + L * i));
    x[4 * i] = t.x; x[4 * i + 1] = t.y; x[4 * i + 2] = t.z; x[4 * i + 3] = t.w;
  }
}
template <int R4>
TTT_DEVICE_INLINE float part_dot(const float (&x)[4 * R4], const float (&y)[4 * R4]) {
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int i = 0; i < 4 * R4; i += 2) {
    a = fmaf(x[i], y[i], a);
    b = fmaf(x[i + 1], y[i + 1], b);
  }
  return a + b;
}

// ------------------------------------------------------------------ forward
// out may be null (the backward pass's replay); then e and the state at every
// chunk border (TT tokens) are kept: ev [BH][N][dv], Sc [BH][nch + 1][dk][dv].
template <typename Tin, typename Tout, int R4>
__global__ void __launch_bounds__(THREADS)
    delta_rec_kernel(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
                     const Tin* __restrict__ g, const Tin* __restrict__ beta, const float* S_in,
                     float* S_out, Tout* __restrict__ out, float* __restrict__ ev,
                     float* __restrict__ Sc, int N, int dk, int dv, float scale) {
  __shared__ __align__(16) Stage<R4> st;
  const size_t bh = blockIdx.x;
  const int c0 = blockIdx.y * COLS, tid = threadIdx.x, cl = tid / L;
  const Column<R4> col{tid % L, c0 + cl, dk, dv, c0 + cl < dv};
  const int l = col.l, lt = l & 3;
  const size_t mat = (size_t)dk * dv;
  float s[4 * R4];
  if (S_in != nullptr) {
    col.load(S_in + bh * mat, s);
  } else {
#pragma unroll
    for (int i = 0; i < 4 * R4; ++i) s[i] = 0.f;
  }
  const int nch = (N + TT - 1) / TT;
  Fetch<Tin, R4> f;
  const Tin* qp = out != nullptr ? q : nullptr;
  f.load(k, qp, v, g, beta, bh, 0, N, dk, dv, c0, tid);
  for (int t0 = 0; t0 < N; t0 += TT) {
    f.put(st, 1.f, tid);
    __syncthreads();
    f.load(k, qp, v, g, beta, bh, t0 + TT, N, dk, dv, c0, tid);
    coefficients(st, tid);
    if (Sc != nullptr) col.store(Sc + (bh * (nch + 1) + t0 / TT) * mat, s);
    __syncthreads();
    const int n = min(TT, N - t0), nb = (n + 3) / 4;
    for (int b = 0; b < nb; ++b) {
      float kv[4][4 * R4], d[8];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        load_rows<R4>(st.k[4 * b + t], l, kv[t]);
        d[t] = part_dot<R4>(kv[t], s);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float qv[4 * R4];
        load_rows<R4>(st.q[4 * b + t], l, qv);
        d[4 + t] = part_dot<R4>(qv, s);
      }
      // eight sums over eight lanes, halving the values a lane holds: k_t.s
      // ends in lane t, q_t.s in lane 4 + t
      float h[4], p2[2], mine;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        h[t] = ((l & 4) ? d[4 + t] : d[t]) + __shfl_xor_sync(0xffffffffu, (l & 4) ? d[t] : d[4 + t], 4);
#pragma unroll
      for (int t = 0; t < 2; ++t)
        p2[t] = ((l & 2) ? h[2 + t] : h[t]) + __shfl_xor_sync(0xffffffffu, (l & 2) ? h[t] : h[2 + t], 2);
      mine = ((l & 1) ? p2[1] : p2[0]) + __shfl_xor_sync(0xffffffffu, (l & 1) ? p2[0] : p2[1], 1);
      float p[4], e[4], u[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) p[t] = __shfl_sync(0xffffffffu, mine, t, 8);
#pragma unroll
      for (int t = 0; t < 4; ++t) e[t] = fmaf(-st.A[4 * b + t], p[t], st.w[4 * b + t][cl]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int i = 0; i < t; ++i) e[t] = fmaf(-st.kk[4 * b + t][i], u[i], e[t]);
        u[t] = st.b[4 * b + t] * e[t];
      }
      if (out != nullptr) {
        const float4 c = *reinterpret_cast<const float4*>(st.qk[4 * b + lt]);
        const float o = fmaf(c.x, u[0], fmaf(c.y, u[1], fmaf(c.z, u[2], fmaf(c.w, u[3], st.A[4 * b + lt] * mine))));
        if (l & 4) st.os[4 * b + lt][cl] = scale * o;
      } else if (l < 4) {
        st.os[4 * b + l][cl] = l == 0 ? e[0] : l == 1 ? e[1] : l == 2 ? e[2] : e[3];
      }
      const float A3 = st.A[4 * b + 3];
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] *= st.R[4 * b + t];
#pragma unroll
      for (int i = 0; i < 4 * R4; ++i)
        s[i] = fmaf(kv[3][i], u[3], fmaf(kv[2][i], u[2], fmaf(kv[1][i], u[1], fmaf(kv[0][i], u[0], A3 * s[i]))));
    }
    __syncthreads();
    for (int i = tid; i < n * COLS; i += THREADS) {
      const int t = t0 + i / COLS, c = c0 + i % COLS;
      if (c >= dv) continue;
      const size_t at = (bh * N + t) * dv + c;
      if (out != nullptr) out[at] = from_f<Tout>(st.os[i / COLS][i % COLS]);
      else ev[at] = st.os[i / COLS][i % COLS];
    }
  }
  if (Sc != nullptr) col.store(Sc + (bh * (nch + 1) + nch) * mat, s);
  if (S_out != nullptr) col.store(S_out + bh * mat, s);
}

// ------------------------------------------------------------------ reverse
// X = dL/dS from the last token back:  X += scale q do^T;  du = X^T k;
// X <- a (X - beta k du^T).  Four tokens at a time, with X the value behind
// them and f = beta du:
//   du_t = R_3t k_t.X + sum_{s>=t} R_st (q_s.k_t) do_s - sum_{s>t} R_st (k_s.k_t) f_s
//   X <- A_3 X + sum_s A_s (q_s do_s - k_s f_s)
// Kept: du [BH][N][dv], and X at the end of every chunk of TT tokens, Xc
// [BH][nch][dk][dv].
template <typename Tin, int R4>
__global__ void __launch_bounds__(THREADS)
    delta_rev_kernel(const Tin* __restrict__ q, const Tin* __restrict__ k,
                     const Tin* __restrict__ dout, const Tin* __restrict__ g,
                     const Tin* __restrict__ beta, const float* __restrict__ dS_end,
                     float* __restrict__ dS0, float* __restrict__ duv, float* __restrict__ Xc, int N,
                     int dk, int dv, float scale) {
  __shared__ __align__(16) Stage<R4> st;
  const size_t bh = blockIdx.x;
  const int c0 = blockIdx.y * COLS, tid = threadIdx.x, cl = tid / L;
  const Column<R4> col{tid % L, c0 + cl, dk, dv, c0 + cl < dv};
  const int l = col.l;
  const size_t mat = (size_t)dk * dv;
  float x[4 * R4];
  if (dS_end != nullptr) {
    col.load(dS_end + bh * mat, x);
  } else {
#pragma unroll
    for (int i = 0; i < 4 * R4; ++i) x[i] = 0.f;
  }
  const int nch = (N + TT - 1) / TT;
  Fetch<Tin, R4> f;
  f.load(k, q, dout, g, beta, bh, (nch - 1) * TT, N, dk, dv, c0, tid);
  for (int ch = nch - 1; ch >= 0; --ch) {
    const int t0 = ch * TT;
    f.put(st, scale, tid);
    __syncthreads();
    f.load(k, q, dout, g, beta, bh, t0 - TT, N, dk, dv, c0, tid);
    coefficients(st, tid);
    col.store(Xc + (bh * nch + ch) * mat, x);
    __syncthreads();
    const int n = min(TT, N - t0);
    for (int b = (n + 3) / 4 - 1; b >= 0; --b) {
      float kv[4][4 * R4], d[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        load_rows<R4>(st.k[4 * b + t], l, kv[t]);
        d[t] = part_dot<R4>(kv[t], x);
      }
      float h[2], mine;
#pragma unroll
      for (int t = 0; t < 2; ++t)
        h[t] = ((l & 2) ? d[2 + t] : d[t]) + __shfl_xor_sync(0xffffffffu, (l & 2) ? d[t] : d[2 + t], 2);
      mine = ((l & 1) ? h[1] : h[0]) + __shfl_xor_sync(0xffffffffu, (l & 1) ? h[0] : h[1], 1);
      mine += __shfl_xor_sync(0xffffffffu, mine, 4);
      float du[4], w[4], fu[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) w[t] = st.w[4 * b + t][cl];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        du[t] = st.R[4 * b + t] * __shfl_sync(0xffffffffu, mine, t, 8);
#pragma unroll
        for (int s = t; s < 4; ++s) du[t] = fmaf(st.qk[4 * b + s][t], w[s], du[t]);
      }
#pragma unroll
      for (int t = 3; t >= 0; --t) {
#pragma unroll
        for (int s = 3; s > t; --s) du[t] = fmaf(-st.kk[4 * b + s][t], fu[s], du[t]);
        fu[t] = st.b[4 * b + t] * du[t];
      }
      if (l < 4) st.os[4 * b + l][cl] = l == 0 ? du[0] : l == 1 ? du[1] : l == 2 ? du[2] : du[3];
      const float A3 = st.A[4 * b + 3];
#pragma unroll
      for (int i = 0; i < 4 * R4; ++i) x[i] *= A3;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float A = st.A[4 * b + t], wt = A * w[t], ft = -A * fu[t];
        float qv[4 * R4];
        load_rows<R4>(st.q[4 * b + t], l, qv);
#pragma unroll
        for (int i = 0; i < 4 * R4; ++i) x[i] = fmaf(qv[i], wt, fmaf(kv[t][i], ft, x[i]));
      }
    }
    __syncthreads();
    for (int i = tid; i < n * COLS; i += THREADS) {
      const int c = c0 + i % COLS;
      if (c < dv) duv[(bh * N + t0 + i / COLS) * dv + c] = st.os[i / COLS][i % COLS];
    }
  }
  col.store(dS0 + bh * mat, x);
}

// ------------------------------------------------------------------ a chunk's gradients
// With the states S0 at the chunk's start and S1 at its end, X1 = dL/dS at
// its end, and every token's e and du, the chunk's gradients need no
// recurrence.  G: the decay's running sum in the chunk, Gam_ij = exp(G_i -
// G_j), gam_i = exp(G_i), rho_j = exp(G_end - G_j), U = beta e, R = beta du:
//   Mq_ij = (scale do_i . U_j) Gam_ij (j <= i),  Mk_ij = -(R_i . U_j) Gam_ij (j < i)
//   dq_i = gam_i S0 (scale do_i) + sum_j Mq_ij k_j
//   dk_i = [-gam_i S0 R_i + sum_j Mk_ij k_j] + [sum_j (Mq_ji q_j + Mk_ji k_j) + rho_i X1 U_i]
//   dv_i = R_i,  dbeta_i = du_i . e_i
//   dg_t = sum_{i >= t} (q_i . dq_i + k_i . [read part of dk_i] - k_i . [write part]) + <X1, S1>
// One CTA per chunk and head, every matrix in shared memory.
constexpr int CB = TT;          // tokens of a chunk
constexpr int GTHREADS = 256;

template <typename Tin>
struct ChunkArgs {
  const Tin *q, *k, *dout, *g, *beta;
  const float *ev, *duv, *Sc, *Xc;
  Tin *dq, *dk, *dv, *dg, *dbeta;
  int N, dk_, dv_;
  float scale;
};

template <typename Tin>
__global__ void __launch_bounds__(GTHREADS) delta_chunk_grad_kernel(ChunkArgs<Tin> p) {
  extern __shared__ float sm[];
  const int dk = p.dk_, dv = p.dv_, N = p.N, tid = threadIdx.x;
  float* M = sm;                    // [dk][dv + 1]: S0, then X1
  const int ms = dv + 1;
  float* Q = M + dk * ms;           // [CB][dk]
  float* K = Q + CB * dk;
  float* D = K + CB * dk;           // [CB][dv] scale * dout
  float* U = D + CB * dv;           // beta e
  float* R = U + CB * dv;           // beta du
  float* Mq = R + CB * dv;          // [CB][CB + 1]
  float* Mk = Mq + CB * (CB + 1);
  float* dKr = Mk + CB * (CB + 1);  // [CB]: row sums for dg
  __shared__ double G[CB];
  __shared__ float red[GTHREADS / 32];
  const size_t bh = blockIdx.y;
  const int ch = blockIdx.x, t0 = ch * CB, n = min(CB, N - t0), nch = gridDim.x;
  const size_t mat = (size_t)dk * dv, tok = bh * N + t0;
  const float* S0 = p.Sc + (bh * (nch + 1) + ch) * mat;
  const float* S1 = S0 + mat;
  const float* X1 = p.Xc + (bh * nch + ch) * mat;

  if (tid == 0) {
    double acc = 0;
    for (int i = 0; i < n; ++i) {
      // exp(-200) is 0 in float32: a cleared state keeps G finite
      const float gi = p.g != nullptr ? to_f(p.g[tok + i]) : 0.f;
      acc += gi < -200.f ? -200.0 : (double)gi;   // NaN stays
      G[i] = acc;
    }
  }
  if (tid < CB) dKr[tid] = 0.f;
  for (int i = tid; i < n * dk; i += GTHREADS) {
    Q[i] = to_f(p.q[tok * dk + i]);
    K[i] = to_f(p.k[tok * dk + i]);
  }
  for (int i = tid; i < n * dv; i += GTHREADS) {
    const float b = to_f(p.beta[tok + i / dv]);
    const float r = b * p.duv[tok * dv + i];
    D[i] = p.scale * to_f(p.dout[tok * dv + i]);
    U[i] = b * p.ev[tok * dv + i];
    R[i] = r;
    p.dv[tok * dv + i] = from_f<Tin>(r);
  }
  float xs = 0.f;   // <X1, S1>
  for (int i = tid; i < dk * dv; i += GTHREADS) {
    M[i / dv * ms + i % dv] = S0[i];
    xs = fmaf(X1[i], S1[i], xs);
  }
  for (int o = 16; o > 0; o >>= 1) xs += __shfl_xor_sync(0xffffffffu, xs, o);
  if ((tid & 31) == 0) red[tid / 32] = xs;
  __syncthreads();
  // dbeta, Mq, Mk
  for (int i = tid / 32; i < n; i += GTHREADS / 32) {
    float acc = 0.f;
    for (int c = tid & 31; c < dv; c += 32)
      acc = fmaf(p.duv[(tok + i) * dv + c], p.ev[(tok + i) * dv + c], acc);
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if ((tid & 31) == 0) p.dbeta[tok + i] = from_f<Tin>(acc);
  }
  for (int e = tid; e < CB * CB; e += GTHREADS) {
    const int i = e / CB, j = e % CB;
    float mq = 0.f, mk = 0.f;
    if (i < n && j <= i) {
      for (int c = 0; c < dv; ++c) {
        mq = fmaf(D[i * dv + c], U[j * dv + c], mq);
        mk = fmaf(R[i * dv + c], U[j * dv + c], mk);
      }
      const float f = expf((float)(G[i] - G[j]));
      mq *= f;
      mk = j < i ? -mk * f : 0.f;
    }
    Mq[i * (CB + 1) + j] = mq;
    Mk[i * (CB + 1) + j] = mk;
  }
  __syncthreads();
  // a thread holds row r of four tokens' dq and dk at a time; lanes of a warp
  // share the tokens, so the sums for dg are warp sums
  const int warp = tid / 32, lane = tid & 31;
  constexpr int ROWS = DMAX / 32;
  static_assert(CB == 4 * (GTHREADS / 32), "a warp takes four tokens");
  const int i0 = warp * 4;
  float dqv[4][ROWS], dkr[4][ROWS];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < ROWS; ++b) { dqv[a][b] = 0.f; dkr[a][b] = 0.f; }
  for (int c = 0; c < dv; ++c) {
    float m[ROWS];
#pragma unroll
    for (int b = 0; b < ROWS; ++b) m[b] = lane + 32 * b < dk ? M[(lane + 32 * b) * ms + c] : 0.f;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int i = i0 + a;
      const float d = i < n ? D[i * dv + c] : 0.f, r = i < n ? R[i * dv + c] : 0.f;
#pragma unroll
      for (int b = 0; b < ROWS; ++b) {
        dqv[a][b] = fmaf(d, m[b], dqv[a][b]);
        dkr[a][b] = fmaf(-r, m[b], dkr[a][b]);
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < dk * dv; i += GTHREADS) M[i / dv * ms + i % dv] = X1[i];
  __syncthreads();
  float dkw[4][ROWS];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < ROWS; ++b) dkw[a][b] = 0.f;
  for (int c = 0; c < dv; ++c) {
    float m[ROWS];
#pragma unroll
    for (int b = 0; b < ROWS; ++b) m[b] = lane + 32 * b < dk ? M[(lane + 32 * b) * ms + c] : 0.f;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float u = i0 + a < n ? U[(i0 + a) * dv + c] : 0.f;
#pragma unroll
      for (int b = 0; b < ROWS; ++b) dkw[a][b] = fmaf(u, m[b], dkw[a][b]);
    }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int i = i0 + a;
    const float gam = i < n ? expf((float)G[i]) : 0.f;
    const float rho = i < n ? expf((float)(G[n - 1] - G[i])) : 0.f;
#pragma unroll
    for (int b = 0; b < ROWS; ++b) { dqv[a][b] *= gam; dkr[a][b] *= gam; dkw[a][b] *= rho; }
  }
  for (int j = 0; j < n; ++j) {
    float kj[ROWS], qj[ROWS];
#pragma unroll
    for (int b = 0; b < ROWS; ++b) {
      kj[b] = lane + 32 * b < dk ? K[j * dk + lane + 32 * b] : 0.f;
      qj[b] = lane + 32 * b < dk ? Q[j * dk + lane + 32 * b] : 0.f;
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int i = i0 + a;   // rows behind n read zeros written above
      const float mq = Mq[i * (CB + 1) + j], mk = Mk[i * (CB + 1) + j];
      const float wq = Mq[j * (CB + 1) + i], wk = Mk[j * (CB + 1) + i];
#pragma unroll
      for (int b = 0; b < ROWS; ++b) {
        dqv[a][b] = fmaf(mq, kj[b], dqv[a][b]);
        dkr[a][b] = fmaf(mk, kj[b], dkr[a][b]);
        dkw[a][b] = fmaf(wq, qj[b], fmaf(wk, kj[b], dkw[a][b]));
      }
    }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int i = i0 + a;
    float acc = 0.f;
    if (i < n) {
#pragma unroll
      for (int b = 0; b < ROWS; ++b) {
        const int r = lane + 32 * b;
        if (r >= dk) continue;
        p.dq[(tok + i) * dk + r] = from_f<Tin>(dqv[a][b]);
        p.dk[(tok + i) * dk + r] = from_f<Tin>(dkr[a][b] + dkw[a][b]);
        acc = fmaf(Q[i * dk + r], dqv[a][b], fmaf(K[i * dk + r], dkr[a][b] - dkw[a][b], acc));
      }
    }
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) dKr[i] = acc;
  }
  __syncthreads();
  if (tid == 0 && p.dg != nullptr) {
    float acc = 0.f;
    for (int w = 0; w < GTHREADS / 32; ++w) acc += red[w];
    for (int i = n - 1; i >= 0; --i) {
      acc += dKr[i];
      p.dg[tok + i] = from_f<Tin>(acc);
    }
  }
}

size_t chunk_grad_smem(int dk, int dv) {
  return sizeof(float) * ((size_t)dk * (dv + 1) + 2 * CB * dk + 3 * CB * dv + 2 * CB * (CB + 1) + CB);
}

// ------------------------------------------------------------------ single tokens
// One token per row; a CTA takes `vc` columns of one row's head: lanes cover
// the columns four at a time, the other threads split dk.  The state slice is
// read into registers in one sweep, the two dot products over dk (S^T k, and
// q.S' from q.S and q.k) are joined through shared memory in one exchange,
// and the slice is written back: bound by the state's bytes.
constexpr int STHREADS = 128;
constexpr int SROWS = 32;       // most rows of dk a thread holds

template <typename Tin, typename Tout>
__global__ void __launch_bounds__(STHREADS)
    delta_step_kernel(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
                      const Tin* __restrict__ g, const Tin* __restrict__ beta,
                      const int* __restrict__ slots, int n_slots, float* __restrict__ S,
                      Tout* __restrict__ out, int B, int H, int dk, int dv, int vc, float scale) {
  __shared__ float ks[DMAX], qs[DMAX];
  __shared__ float part[2][STHREADS][4];   // partial S^T k and S^T q of four columns
  __shared__ float qk_s;
  __shared__ int again;
  const int h = blockIdx.y, c0 = blockIdx.z * vc, tid = threadIdx.x;
  int b = blockIdx.x;
  const int slot = slots != nullptr ? slots[b] : b;
  if (slot < 0 || slot >= n_slots) return;
  if (slots != nullptr) {   // a sequence's first row takes all of its rows, in order
    int dup = 0;
    for (int j = tid; j < b; j += STHREADS) dup |= slots[j] == slot;
    if (__syncthreads_or(dup)) return;
  }
  const int lanes = vc / 4, groups = STHREADS / lanes;
  const int cl = tid % lanes, gr = tid / lanes, c = c0 + 4 * cl;
  const bool vec = (dv & 3) == 0;
  float* Sm = S + ((size_t)slot * H + h) * dk * dv;
  float4 s[SROWS];
#pragma unroll
  for (int i = 0; i < SROWS; ++i) {
    const int r = gr + groups * i;
    s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < dk && c < dv) {
      const float* src = Sm + (size_t)r * dv + c;
      if (vec) {
        s[i] = *reinterpret_cast<const float4*>(src);
      } else {
        s[i].x = src[0];
        if (c + 1 < dv) s[i].y = src[1];
        if (c + 2 < dv) s[i].z = src[2];
        if (c + 3 < dv) s[i].w = src[3];
      }
    }
  }
  for (;;) {
    const size_t tok = (size_t)b * H + h;
    for (int i = tid; i < DMAX; i += STHREADS) {
      ks[i] = i < dk ? to_f(k[tok * dk + i]) : 0.f;
      qs[i] = i < dk ? to_f(q[tok * dk + i]) : 0.f;
    }
    __syncthreads();
    const float a = g != nullptr ? expf(to_f(g[tok])) : 1.f, bt = to_f(beta[tok]);
    float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
    for (int i = 0; i < SROWS; ++i) {
      const int r = gr + groups * i;
      if (r < dk) {
        const float kr = ks[r], qr = qs[r];
        pk.x = fmaf(kr, s[i].x, pk.x); pk.y = fmaf(kr, s[i].y, pk.y);
        pk.z = fmaf(kr, s[i].z, pk.z); pk.w = fmaf(kr, s[i].w, pk.w);
        pq.x = fmaf(qr, s[i].x, pq.x); pq.y = fmaf(qr, s[i].y, pq.y);
        pq.z = fmaf(qr, s[i].z, pq.z); pq.w = fmaf(qr, s[i].w, pq.w);
      }
    }
    *reinterpret_cast<float4*>(part[0][tid]) = pk;
    *reinterpret_cast<float4*>(part[1][tid]) = pq;
    if (tid < 32) {
      float x = 0.f;
      for (int i = tid; i < dk; i += 32) x = fmaf(qs[i], ks[i], x);
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (tid == 0) qk_s = x;
    }
    __syncthreads();
    pk = pq = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < groups; ++j) {
      const float4 x = *reinterpret_cast<const float4*>(part[0][j * lanes + cl]);
      pk.x += x.x; pk.y += x.y; pk.z += x.z; pk.w += x.w;
      if (gr == 0) {
        const float4 y = *reinterpret_cast<const float4*>(part[1][j * lanes + cl]);
        pq.x += y.x; pq.y += y.y; pq.z += y.z; pq.w += y.w;
      }
    }
    float u[4] = {0.f, 0.f, 0.f, 0.f};
    const float pks[4] = {pk.x, pk.y, pk.z, pk.w}, pqs[4] = {pq.x, pq.y, pq.z, pq.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c + j < dv) {
        u[j] = bt * (to_f(v[tok * dv + c + j]) - a * pks[j]);
        // S'^T q = a S^T q + (q.k) u
        if (gr == 0) out[tok * dv + c + j] = from_f<Tout>(scale * fmaf(qk_s, u[j], a * pqs[j]));
      }
    }
#pragma unroll
    for (int i = 0; i < SROWS; ++i) {
      const int r = gr + groups * i;
      if (r < dk) {
        const float kr = ks[r];
        s[i].x = fmaf(kr, u[0], a * s[i].x); s[i].y = fmaf(kr, u[1], a * s[i].y);
        s[i].z = fmaf(kr, u[2], a * s[i].z); s[i].w = fmaf(kr, u[3], a * s[i].w);
      }
    }
    if (slots == nullptr) break;
    // the next row of the same sequence
    if (tid == 0) again = B;
    __syncthreads();
    int next = B;
    for (int j = b + 1 + tid; j < B; j += STHREADS)
      if (slots[j] == slot) { next = j; break; }
    if (next < B) atomicMin(&again, next);
    __syncthreads();
    if (again >= B) break;
    b = again;
    __syncthreads();   // `again`, ks and qs are written again above
  }
#pragma unroll
  for (int i = 0; i < SROWS; ++i) {
    const int r = gr + groups * i;
    if (r < dk && c < dv) {
      float* dst = Sm + (size_t)r * dv + c;
      if (vec) {
        *reinterpret_cast<float4*>(dst) = s[i];
      } else {
        dst[0] = s[i].x;
        if (c + 1 < dv) dst[1] = s[i].y;
        if (c + 2 < dv) dst[2] = s[i].z;
        if (c + 3 < dv) dst[3] = s[i].w;
      }
    }
  }
}

#define TTT_BY_ROWS(CALL)                     \
  switch ((p.dk + 31) / 32) {                 \
    case 1: CALL(1); break;                   \
    case 2: CALL(2); break;                   \
    case 3: CALL(3); break;                   \
    default: CALL(4); break;                  \
  }

template <typename Tin, typename Tout>
int rec_launch(const DeltaLaunch& p, float* S_out, const float* S_in, Tout* out, float* ev, float* Sc,
               cudaStream_t stream) {
  const dim3 grid((unsigned)(p.B * p.H), (unsigned)((p.dv + COLS - 1) / COLS));
  prof_before(K_DELTA_REC, stream);
#define TTT_REC(R4)                                                                            \
  delta_rec_kernel<Tin, Tout, R4><<<grid, THREADS, 0, stream>>>(                               \
      (const Tin*)p.q, (const Tin*)p.k, (const Tin*)p.v, (const Tin*)p.g, (const Tin*)p.beta,  \
      S_in, S_out, out, ev, Sc, p.N, p.dk, p.dv, p.scale)
  TTT_BY_ROWS(TTT_REC)
#undef TTT_REC
  prof_after(K_DELTA_REC, stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <typename Tin>
int bwd_launch(const DeltaBwdLaunch& L, cudaStream_t stream) {
  const DeltaLaunch& p = L.f;
  const int BH = p.B * p.H, nch = (p.N + CB - 1) / CB;
  const DeltaBwdWorkspace w = delta_rec_bwd_layout(BH, p.N, p.dk, p.dv);
  float* ev = reinterpret_cast<float*>(L.ws + w.ev);
  float* du = reinterpret_cast<float*>(L.ws + w.du);
  float* Sc = reinterpret_cast<float*>(L.ws + w.Sc);
  float* Xc = reinterpret_cast<float*>(L.ws + w.Xc);
  if (rec_launch<Tin, float>(p, nullptr, L.S0, nullptr, ev, Sc, stream)) return -1;
  const dim3 grid((unsigned)BH, (unsigned)((p.dv + COLS - 1) / COLS));
  prof_before(K_DELTA_REV, stream);
#define TTT_REV(R4)                                                                               \
  delta_rev_kernel<Tin, R4><<<grid, THREADS, 0, stream>>>(                                        \
      (const Tin*)p.q, (const Tin*)p.k, (const Tin*)L.dout, (const Tin*)p.g, (const Tin*)p.beta,  \
      L.dS_end, L.dS0, du, Xc, p.N, p.dk, p.dv, p.scale)
  TTT_BY_ROWS(TTT_REV)
#undef TTT_REV
  prof_after(K_DELTA_REV, stream);
  if (cudaGetLastError() != cudaSuccess) return -1;
  const size_t smem = chunk_grad_smem(p.dk, p.dv);
  auto kfn = delta_chunk_grad_kernel<Tin>;
  static std::atomic<uint64_t> attr{0};
  if (allow_dynamic_smem(kfn, (int)chunk_grad_smem(DMAX, DMAX), attr)) return -1;
  ChunkArgs<Tin> a{(const Tin*)p.q, (const Tin*)p.k, (const Tin*)L.dout, (const Tin*)p.g,
                   (const Tin*)p.beta, ev, du, Sc, Xc, (Tin*)L.dq, (Tin*)L.dk, (Tin*)L.dv,
                   (Tin*)L.dg, (Tin*)L.dbeta, p.N, p.dk, p.dv, p.scale};
  if (nch == 0) return 0;
  // grid.y is limited to 65535: more heads go in slices
  for (int b0 = 0; b0 < BH; b0 += 65535) {
    const int nb = std::min(65535, BH - b0);
    ChunkArgs<Tin> s = a;
    const size_t t = (size_t)b0 * p.N, mat = (size_t)p.dk * p.dv;
    s.q += t * p.dk; s.k += t * p.dk; s.dq += t * p.dk; s.dk += t * p.dk;
    s.dout += t * p.dv; s.dv += t * p.dv; s.ev += t * p.dv; s.duv += t * p.dv;
    s.beta += t; s.dbeta += t;
    if (s.g != nullptr) { s.g += t; s.dg += t; }
    s.Sc += (size_t)b0 * (nch + 1) * mat;
    s.Xc += (size_t)b0 * nch * mat;
    prof_before(K_DELTA_GRAD, stream);
    kfn<<<dim3((unsigned)nch, (unsigned)nb), GTHREADS, smem, stream>>>(s);
    prof_after(K_DELTA_GRAD, stream);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

int launch_delta_rec(const DeltaLaunch& p, cudaStream_t stream) {
  if (p.in_bf16) {
    if (p.out_bf16) return rec_launch<__nv_bfloat16, __nv_bfloat16>(p, p.S, p.S, (__nv_bfloat16*)p.out, nullptr, nullptr, stream);
    return rec_launch<__nv_bfloat16, float>(p, p.S, p.S, (float*)p.out, nullptr, nullptr, stream);
  }
  if (p.out_bf16) return rec_launch<float, __nv_bfloat16>(p, p.S, p.S, (__nv_bfloat16*)p.out, nullptr, nullptr, stream);
  return rec_launch<float, float>(p, p.S, p.S, (float*)p.out, nullptr, nullptr, stream);
}

DeltaBwdWorkspace delta_rec_bwd_layout(int BH, int N, int dk, int dv) {
  DeltaBwdWorkspace w{};
  size_t at = 256;
  auto take = [&](size_t floats) {
    const size_t o = at;
    at += (floats * sizeof(float) + 255) / 256 * 256;
    return o;
  };
  const size_t nch = (N + CB - 1) / CB, mat = (size_t)dk * dv;
  w.ev = take((size_t)BH * N * dv);
  w.du = take((size_t)BH * N * dv);
  w.Sc = take((size_t)BH * (nch + 1) * mat);
  w.Xc = take((size_t)BH * nch * mat);
  w.total = at;
  return w;
}

int launch_delta_rec_bwd(const DeltaBwdLaunch& L, cudaStream_t stream) {
  return L.f.in_bf16 ? bwd_launch<__nv_bfloat16>(L, stream) : bwd_launch<float>(L, stream);
}

int launch_delta_step(const DeltaLaunch& p, const int* slots, int n_slots, cudaStream_t stream) {
  // columns of a CTA: all of them where rows and heads fill the device, fewer
  // where they do not (a slice of 16 columns is 64 bytes of every state row)
  int vc = 16;
  while (vc < 128 && vc < p.dv) vc *= 2;
  while (vc > 16 && (long long)p.B * p.H * ((p.dv + vc - 1) / vc) < 4 * 148) vc /= 2;
  const dim3 grid((unsigned)p.B, (unsigned)p.H, (unsigned)((p.dv + vc - 1) / vc));
#define TTT_STEP(TI, TO)                                                                          \
  delta_step_kernel<TI, TO><<<grid, STHREADS, 0, stream>>>(                                        \
      (const TI*)p.q, (const TI*)p.k, (const TI*)p.v, (const TI*)p.g, (const TI*)p.beta, slots,    \
      n_slots, p.S, (TO*)p.out, p.B, p.H, p.dk, p.dv, vc, p.scale)
  prof_before(K_DELTA_STEP, stream);
  if (p.in_bf16) {
    if (p.out_bf16) TTT_STEP(__nv_bfloat16, __nv_bfloat16);
    else TTT_STEP(__nv_bfloat16, float);
  } else {
    if (p.out_bf16) TTT_STEP(float, __nv_bfloat16);
    else TTT_STEP(float, float);
  }
#undef TTT_STEP
  prof_after(K_DELTA_STEP, stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace ttt
