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
// latency of that chain (0.28 us a step in heads of 32, 0.4 of 64, 0.6 of 128);
// the chunked tensor-core kernels (delta_umma.cu) take the sizes where it
// matters.
#include <algorithm>
#include <type_traits>

#include "kernels.h"

namespace ttt {

namespace {

constexpr int L = 8;            // lanes of one column
constexpr int COLS = 16;        // columns of a CTA
constexpr int THREADS = L * COLS;
constexpr int TT = 32;          // tokens staged at a time, and between kept states
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

// The next tile's tokens wait in registers while this one is worked on.  A
// thread keeps its row of k and q and its column of the value tensor.  Without Q
// (the replay, which reads nothing out) there are no queries.
template <typename Tin, int R4, bool Q>
struct Fetch {
  static constexpr int RW = R4 == 3 ? 128 : 32 * R4;      // threads of a token's row
  static constexpr int TS = THREADS / RW, NX = TT / TS;   // tokens side by side, and of a thread
  static constexpr int WS = THREADS / COLS, NW = TT / WS;
  Tin k[NX], q[Q ? NX : 1], w[NW], g, b;
  const Tin *kp, *qp, *wp, *gp, *bp;
  int N, dk, dv, r, tr, tw, tid;
  bool row, col;
  TTT_DEVICE_INLINE Fetch(const Tin* k_, const Tin* q_, const Tin* w_, const Tin* g_, const Tin* b_, size_t bh,
                          int N_, int dk_, int dv_, int c0, int tid_)
      : N(N_), dk(dk_), dv(dv_), r(tid_ % RW), tr(tid_ / RW), tw(tid_ / COLS), tid(tid_) {
    row = r < dk;
    col = c0 + tid % COLS < dv;
    const size_t tok = bh * N;
    kp = k_ + tok * dk + r;
    if constexpr (Q) qp = q_ + tok * dk + r;
    wp = w_ + tok * dv + c0 + tid % COLS;
    gp = g_ != nullptr ? g_ + tok : nullptr;
    bp = b_ + tok;
  }
  TTT_DEVICE_INLINE void load(int t0) {
    const Tin zero = from_f<Tin>(0.f);
    const int n = N - t0;
    const size_t x0 = ((size_t)t0 + tr) * dk, w0 = ((size_t)t0 + tw) * dv;
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const bool in = row && tr + i * TS < n;
      k[i] = in ? kp[x0 + (size_t)(i * TS * dk)] : zero;
      if constexpr (Q) q[i] = in ? qp[x0 + (size_t)(i * TS * dk)] : zero;
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = col && tw + i * WS < n ? wp[w0 + (size_t)(i * WS * dv)] : zero;
    g = b = zero;   // no decay, no step: a padding token
    if (tid < TT && tid < n) {
      if (gp != nullptr) g = gp[t0 + tid];
      b = bp[t0 + tid];
    }
  }
  TTT_DEVICE_INLINE void put(Stage<R4>& st, float wscale) const {
    if (R4 != 3 || r < 96) {
#pragma unroll
      for (int i = 0; i < NX; ++i) {
        st.k[tr + i * TS][r] = to_f(k[i]);
        if constexpr (Q) st.q[tr + i * TS][r] = to_f(q[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) st.w[tw + i * WS][tid % COLS] = wscale * to_f(w[i]);
    if (tid < TT) {
      st.a[tid] = expf(to_f(g));
      st.b[tid] = to_f(b);
    }
  }
};
// st.os to global memory, n tokens of 16 columns
template <typename T, int R4>
TTT_DEVICE_INLINE void write_os(const Stage<R4>& st, T* dst, int n, int dv, int c0, int tid) {
  const int c = tid % COLS, t = tid / COLS;
  constexpr int WS = THREADS / COLS;
  T* p = dst + (size_t)t * dv + c0 + c;
#pragma unroll
  for (int i = 0; i < TT / WS; ++i)
    if (c0 + c < dv && t + i * WS < n) p[(size_t)(i * WS * dv)] = from_f<T>(st.os[t + i * WS][c]);
}

// Coefficients of the staged tokens: thread 16 b + d takes one of the 16
// products within block b, the first ten of them with queries.
template <int R4, bool Q>
TTT_DEVICE_INLINE void coefficients(Stage<R4>& st, int tid) {
  const int base = tid / 16 * 4, d = tid % 16;
  // d: 0..9 q.k with (t, i) in lower-triangle order, 10..15 k.k below the diagonal
  constexpr unsigned long long TS = 0x3332213333222110ull, IS = 0x2101003210210100ull;
  const int t = (int)(TS >> (4 * d) & 15), i = (int)(IS >> (4 * d) & 15);
  const float* x = d < 10 ? st.q[base + t] : st.k[base + t];
  const float* y = st.k[base + i];
  float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
  if (Q || d >= 10) {
#pragma unroll
    for (int r = 0; r < 32 * R4; r += 4) {
      const float4 u = *reinterpret_cast<const float4*>(x + r), v = *reinterpret_cast<const float4*>(y + r);
      a0 = fmaf(u.x, v.x, a0);
      a1 = fmaf(u.y, v.y, a1);
      a2 = fmaf(u.z, v.z, a2);
      a3 = fmaf(u.w, v.w, a3);
    }
  }
  float f = (a0 + a1) + (a2 + a3);
  const float4 av = *reinterpret_cast<const float4*>(st.a + base);
  if (i < 1 && t >= 1) f *= av.y;
  if (i < 2 && t >= 2) f *= av.z;
  if (i < 3 && t >= 3) f *= av.w;
  if (d >= 10) st.kk[base + t][i] = f;
  else if (Q) st.qk[base + t][i] = f;
  if (d < 4) {   // token d of the block
    st.A[base + d] = av.x * (d >= 1 ? av.y : 1.f) * (d >= 2 ? av.z : 1.f) * (d >= 3 ? av.w : 1.f);
    st.R[base + d] = (d < 1 ? av.y : 1.f) * (d < 2 ? av.z : 1.f) * (d < 3 ? av.w : 1.f);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (Q && m > d) st.qk[base + d][m] = 0.f;
      if (m >= d) st.kk[base + d][m] = 0.f;
    }
  }
}

// A block's coefficients in registers, read ahead of its chain.
struct BlockCoef {
  float A[4], R[4], b[4], w[4], kk[4][4];
  template <int R4>
  TTT_DEVICE_INLINE BlockCoef(const Stage<R4>& st, int blk, int cl) {
    auto get = [](const float* p, float (&x)[4]) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    };
    get(st.A + 4 * blk, A);
    get(st.R + 4 * blk, R);
    get(st.b + 4 * blk, b);
#pragma unroll
    for (int t = 0; t < 4; ++t) w[t] = st.w[4 * blk + t][cl];
#pragma unroll
    for (int t = 1; t < 4; ++t) get(st.kk[4 * blk + t], kk[t]);
  }
};

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

// ------------------------------------------------------------------ tiles
// A CTA's 128 state threads walk tiles of TT tokens.  With HELP, 128 more
// threads stage the next tile, form its coefficients and write the last one's
// values meanwhile, in two buffers: what is left between tiles is one barrier.
template <typename Tin, int R4, bool Q, bool HELP, typename K, typename W, typename F>
TTT_DEVICE_INLINE void walk_tiles(Stage<R4>* st, Fetch<Tin, R4, Q>& f, int nch, bool down, float wscale, int tid,
                                  K keep, W work, F write) {
  if (nch == 0) return;
  // the i-th tile of the walk starts at token t0(i)
  auto t0 = [&](int i) { return (down ? nch - 1 - i : i) * TT; };
  if constexpr (HELP) {
    const bool helper = tid >= THREADS;
    const int h = tid - THREADS;
    auto stage = [&](int i) {   // by the helpers: tile i, whose values they hold
      Stage<R4>& s = st[i & 1];
      f.put(s, wscale);
      named_bar_sync(1, THREADS);
      if (i + 1 < nch) f.load(t0(i + 1));
      coefficients<R4, Q>(s, h);
    };
    if (helper) {
      f.load(t0(0));
      stage(0);
    }
    __syncthreads();
    for (int i = 0; i < nch; ++i) {
      if (!helper) {
        keep(t0(i));
        work(st[i & 1], t0(i));
      } else {
        if (i > 0) write(st[(i - 1) & 1], t0(i - 1), h);
        if (i + 1 < nch) stage(i + 1);
      }
      __syncthreads();
    }
    if (helper) write(st[(nch - 1) & 1], t0(nch - 1), h);
  } else {
    f.load(t0(0));
    for (int i = 0; i < nch; ++i) {
      f.put(st[0], wscale);
      __syncthreads();
      if (i + 1 < nch) f.load(t0(i + 1));
      coefficients<R4, Q>(st[0], tid);
      keep(t0(i));
      __syncthreads();
      work(st[0], t0(i));
      __syncthreads();
      write(st[0], t0(i), tid);
    }
  }
}
template <int R4, bool HELP>
constexpr size_t stage_bytes() { return (HELP ? 2 : 1) * sizeof(Stage<R4>); }

// ------------------------------------------------------------------ forward
// The state over one tile of n tokens; READS: out of every token into st.os,
// else e.
template <int R4, bool READS>
TTT_DEVICE_INLINE void rec_tile(Stage<R4>& st, float (&s)[4 * R4], int n, float scale, int l, int cl) {
  constexpr int U = R4 == 1 ? 4 : 2;
  const int lt = l & 3, nb = (n + 3) / 4;
  // U blocks to a turn, so that one block's loads pass under the chain of
  // the one before (results are kept back, as a store would stop the loads);
  // padding tokens change nothing
  for (int b0 = 0; b0 < nb; b0 += U) {
    float keep[U];
#pragma unroll
    for (int ub = 0; ub < U; ++ub) {
      const int b = b0 + ub;
      const BlockCoef c4(st, b, cl);
      float kv[4][4 * R4], d[4], dq[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        load_rows<R4>(st.k[4 * b + t], l, kv[t]);
        d[t] = part_dot<R4>(kv[t], s);
      }
      // eight sums over eight lanes, halving the values a lane holds: k_t.s
      // ends in lane t, q_t.s in lane 4 + t
      if constexpr (READS) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float qv[4 * R4];
          load_rows<R4>(st.q[4 * b + t], l, qv);
          dq[t] = part_dot<R4>(qv, s);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
          d[t] = ((l & 4) ? dq[t] : d[t]) + __shfl_xor_sync(0xffffffffu, (l & 4) ? d[t] : dq[t], 4);
      }
      float p2[2], mine;
#pragma unroll
      for (int t = 0; t < 2; ++t)
        p2[t] = ((l & 2) ? d[2 + t] : d[t]) + __shfl_xor_sync(0xffffffffu, (l & 2) ? d[t] : d[2 + t], 2);
      mine = ((l & 1) ? p2[1] : p2[0]) + __shfl_xor_sync(0xffffffffu, (l & 1) ? p2[0] : p2[1], 1);
      if constexpr (!READS) mine += __shfl_xor_sync(0xffffffffu, mine, 4);
      float p[4], e[4], u[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) p[t] = __shfl_sync(0xffffffffu, mine, t, 8);
#pragma unroll
      for (int t = 0; t < 4; ++t) e[t] = fmaf(-c4.A[t], p[t], c4.w[t]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int i = 0; i < t; ++i) e[t] = fmaf(-c4.kk[t][i], u[i], e[t]);
        u[t] = c4.b[t] * e[t];
      }
      if constexpr (READS) {
        const float4 c = *reinterpret_cast<const float4*>(st.qk[4 * b + lt]);
        // (selected, not multiplied by zero: a later token may hold NaN)
        float o = fmaf(c.x, u[0], st.A[4 * b + lt] * mine);
        o = lt >= 1 ? fmaf(c.y, u[1], o) : o;
        o = lt >= 2 ? fmaf(c.z, u[2], o) : o;
        o = lt >= 3 ? fmaf(c.w, u[3], o) : o;
        keep[ub] = scale * o;
      } else {
        keep[ub] = lt == 0 ? e[0] : lt == 1 ? e[1] : lt == 2 ? e[2] : e[3];
      }
      const float A3 = c4.A[3];
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] *= c4.R[t];
#pragma unroll
      for (int i = 0; i < 4 * R4; ++i)
        s[i] = fmaf(kv[3][i], u[3], fmaf(kv[2][i], u[2], fmaf(kv[1][i], u[1], fmaf(kv[0][i], u[0], A3 * s[i]))));
    }
    if (l & 4)
#pragma unroll
      for (int ub = 0; ub < U; ++ub) st.os[4 * (b0 + ub) + lt][cl] = keep[ub];
  }
}

// One CTA's 16 columns over the whole sequence.  KEEP: the backward pass's
// replay, whose rows are e (ev [BH][N][dv]) in place of out, and which keeps
// the state at the start of every chunk (TT tokens), Sc [BH][nch][dk][dv].
template <typename Tin, typename Tout, int R4, bool HELP, bool KEEP>
TTT_DEVICE_INLINE void rec_cta(Stage<R4>* st, const Tin* __restrict__ q, const Tin* __restrict__ k,
                               const Tin* __restrict__ v, const Tin* __restrict__ g,
                               const Tin* __restrict__ beta, const float* S_in, float* S_out,
                               Tout* __restrict__ rows, float* __restrict__ Sc, int N, int dk, int dv,
                               float scale) {
  const size_t bh = blockIdx.x;
  const int c0 = blockIdx.y * COLS, tid = threadIdx.x, cl = tid % THREADS / L;
  const Column<R4> col{tid % L, c0 + cl, dk, dv, c0 + cl < dv};
  const bool state = tid < THREADS;
  const size_t mat = (size_t)dk * dv;
  float s[4 * R4];
  if (state && S_in != nullptr) {
    col.load(S_in + bh * mat, s);
  } else {
#pragma unroll
    for (int i = 0; i < 4 * R4; ++i) s[i] = 0.f;
  }
  const int nch = tiles_of(N, TT);
  Fetch<Tin, R4, !KEEP> f(k, q, v, g, beta, bh, N, dk, dv, c0, tid % THREADS);
  walk_tiles<Tin, R4, !KEEP, HELP>(
      st, f, nch, false, 1.f, tid,
      [&](int t0) {
        if constexpr (KEEP) col.store(Sc + (bh * nch + t0 / TT) * mat, s);
      },
      [&](Stage<R4>& t, int t0) { rec_tile<R4, !KEEP>(t, s, min(TT, N - t0), scale, col.l, cl); },
      [&](const Stage<R4>& t, int t0, int h) {
        write_os(t, rows + (bh * N + t0) * dv, min(TT, N - t0), dv, c0, h);
      });
  if constexpr (!KEEP)
    if (state) col.store(S_out + bh * mat, s);
}
template <typename Tin, typename Tout, int R4, bool HELP>
__global__ void __launch_bounds__(HELP ? 2 * THREADS : THREADS)
    delta_rec_kernel(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
                     const Tin* __restrict__ g, const Tin* __restrict__ beta, float* S,
                     Tout* __restrict__ out, int N, int dk, int dv, float scale) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  rec_cta<Tin, Tout, R4, HELP, false>(reinterpret_cast<Stage<R4>*>(smem_raw), q, k, v, g, beta, S, S, out,
                                      nullptr, N, dk, dv, scale);
}

// ------------------------------------------------------------------ reverse
// X = dL/dS from the last token back:  X += scale q do^T;  du = X^T k;
// X <- a (X - beta k du^T).  Four tokens at a time, with X the value behind
// them and f = beta du:
//   du_t = R_3t k_t.X + sum_{s>=t} R_st (q_s.k_t) do_s - sum_{s>t} R_st (k_s.k_t) f_s
//   X <- A_3 X + sum_s A_s (q_s do_s - k_s f_s)
template <int R4>
TTT_DEVICE_INLINE void rev_tile(Stage<R4>& st, float (&x)[4 * R4], int n, int l, int cl) {
  constexpr int U = R4 == 1 ? 4 : 2;
  for (int b0 = (n + 4 * U - 1) / (4 * U) * U - 1; b0 >= 0; b0 -= U) {
    float keep[U];
#pragma unroll
    for (int ub = 0; ub < U; ++ub) {
      const int b = b0 - ub;
      const BlockCoef c4(st, b, cl);
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
      for (int t = 0; t < 4; ++t) w[t] = c4.w[t];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        du[t] = c4.R[t] * __shfl_sync(0xffffffffu, mine, t, 8);
#pragma unroll
        for (int s = t; s < 4; ++s) du[t] = fmaf(st.qk[4 * b + s][t], w[s], du[t]);
      }
#pragma unroll
      for (int t = 3; t >= 0; --t) {
#pragma unroll
        for (int s = 3; s > t; --s) du[t] = fmaf(-c4.kk[s][t], fu[s], du[t]);
        fu[t] = c4.b[t] * du[t];
      }
      keep[ub] = (l & 3) == 0 ? du[0] : (l & 3) == 1 ? du[1] : (l & 3) == 2 ? du[2] : du[3];
      const float A3 = c4.A[3];
#pragma unroll
      for (int i = 0; i < 4 * R4; ++i) x[i] *= A3;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float A = c4.A[t], wt = A * w[t], ft = -A * fu[t];
        float qv[4 * R4];
        load_rows<R4>(st.q[4 * b + t], l, qv);
#pragma unroll
        for (int i = 0; i < 4 * R4; ++i) x[i] = fmaf(qv[i], wt, fmaf(kv[t][i], ft, x[i]));
      }
    }
    if (l & 4)
#pragma unroll
      for (int ub = 0; ub < U; ++ub) st.os[4 * (b0 - ub) + (l & 3)][cl] = keep[ub];
  }
}

// Kept: du [BH][N][dv], and X at the end of every chunk of TT tokens, Xc
// [BH][nch][dk][dv].
template <typename Tin, int R4, bool HELP>
TTT_DEVICE_INLINE void rev_cta(Stage<R4>* st, const Tin* __restrict__ q, const Tin* __restrict__ k,
                               const Tin* __restrict__ dout, const Tin* __restrict__ g,
                               const Tin* __restrict__ beta, const float* __restrict__ dS_end,
                               float* __restrict__ dS0, float* __restrict__ duv, float* __restrict__ Xc,
                               int N, int dk, int dv, float scale) {
  const size_t bh = blockIdx.x;
  const int c0 = blockIdx.y * COLS, tid = threadIdx.x, cl = tid % THREADS / L;
  const Column<R4> col{tid % L, c0 + cl, dk, dv, c0 + cl < dv};
  const bool state = tid < THREADS;
  const size_t mat = (size_t)dk * dv;
  float x[4 * R4];
  if (state && dS_end != nullptr) {
    col.load(dS_end + bh * mat, x);
  } else {
#pragma unroll
    for (int i = 0; i < 4 * R4; ++i) x[i] = 0.f;
  }
  const int nch = tiles_of(N, TT);
  Fetch<Tin, R4, true> f(k, q, dout, g, beta, bh, N, dk, dv, c0, tid % THREADS);
  walk_tiles<Tin, R4, true, HELP>(
      st, f, nch, true, scale, tid,
      [&](int t0) { col.store(Xc + (bh * nch + t0 / TT) * mat, x); },
      [&](Stage<R4>& t, int t0) { rev_tile<R4>(t, x, min(TT, N - t0), col.l, cl); },
      [&](const Stage<R4>& t, int t0, int h) {
        write_os(t, duv + (bh * N + t0) * dv, min(TT, N - t0), dv, c0, h);
      });
  if (state) col.store(dS0 + bh * mat, x);
}

// Neither direction needs the other: the forward replay (z = 0) and the
// reverse (z = 1) are CTAs of one launch.
template <typename Tin>
struct StatesArgs {
  const Tin *q, *k, *v, *dout, *g, *beta;
  const float *S0, *dS_end;
  float *dS0, *ev, *du, *Sc, *Xc;
  int N, dk, dv;
  float scale;
};
template <typename Tin, int R4, bool HELP>
__global__ void __launch_bounds__(HELP ? 2 * THREADS : THREADS) delta_states_kernel(const StatesArgs<Tin> a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Stage<R4>* st = reinterpret_cast<Stage<R4>*>(smem_raw);
  if (blockIdx.z == 0)
    rec_cta<Tin, float, R4, HELP, true>(st, a.q, a.k, a.v, a.g, a.beta, a.S0, nullptr, a.ev, a.Sc, a.N, a.dk,
                                        a.dv, a.scale);
  else
    rev_cta<Tin, R4, HELP>(st, a.q, a.k, a.dout, a.g, a.beta, a.dS_end, a.dS0, a.du, a.Xc, a.N, a.dk, a.dv,
                           a.scale);
}

// ------------------------------------------------------------------ a chunk's gradients
// With the state S0 at the chunk's start, X1 = dL/dS at its end, and every
// token's e and du, the chunk's gradients need no recurrence.  G: the decay's running sum in the chunk, Gam_ij = exp(G_i -
// G_j), gam_i = exp(G_i), rho_j = exp(G_end - G_j), U = beta e, R = beta du:
//   Mq_ij = (scale do_i . U_j) Gam_ij (j <= i),  Mk_ij = -(R_i . U_j) Gam_ij (j < i)
//   dq_i = gam_i S0 (scale do_i) + sum_j Mq_ij k_j
//   dk_i = [-gam_i S0 R_i + sum_j Mk_ij k_j] + [sum_j (Mq_ji q_j + Mk_ji k_j) + rho_i X1 U_i]
//   dv_i = R_i,  dbeta_i = du_i . e_i
//   dg_t = sum_{i >= t} gam_i (q_i . S0 (scale do_i) - k_i . S0 R_i)
//          + sum_{i >= t > j} (Mq_ij q_i . k_j + Mk_ij k_i . k_j)
//          + sum_{i < t} rho_i k_i . X1 U_i + gam_end <X1, S0>
// (every term of dg_t holds the decay of token t.  The sums over dq and dk of
// the tokens i >= t less those of dk as a written key are the same, but pairs of
// tokens behind t then enter with both signs, and where the decays are strong
// what is left of them is larger than dg_t.)
// One CTA per chunk and head, every matrix in shared memory, whose reads and
// the latency of the phases bound it: 12 us for one chunk of heads of 64, 2 of
// them for dg.
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

// Shared memory: pitches are 4 (mod 8) floats, so that 16-byte reads down a
// column of rows meet different banks; everything behind dv or dk in a row is zero.
struct GradSmem {
  int ms;                                  // pitch of a value row
  int ks;                                  // pitch of a key row
  size_t S0, X1, Q, K, D, U, R, Mq, Mk, floats;
  __host__ __device__ GradSmem(int dk, int dv) {
    ms = (dv + 7) / 8 * 8 + 4;
    ks = (dk + 7) / 8 * 8 + 4;
    S0 = 0;
    X1 = S0 + (size_t)dk * ms;
    D = X1 + (size_t)dk * ms;
    U = D + CB * ms;
    R = U + CB * ms;
    Mq = R + CB * ms;
    Mk = Mq + CB * MP;
    Q = Mk + CB * MP;
    K = Q + CB * ks;
    floats = K + CB * ks;
  }
  static constexpr int MP = CB + 4;        // pitch of Mq, Mk
};

TTT_DEVICE_INLINE void copy_async4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
TTT_DEVICE_INLINE void copy_async16(float* dst, const float* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
TTT_DEVICE_INLINE float dot4(const float4& a, const float4& b, float acc) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, acc))));
}

// n values' sums over the warp, halving the values a lane holds: value v ends in
// x[0] of the 32 / n lanes from v 32 / n on.
template <int n>
TTT_DEVICE_INLINE void lane_sums(float (&x)[n], int lane) {
#pragma unroll
  for (int o = 16, h = n / 2; o > 0; o >>= 1, h >>= 1) {
    if (h > 0) {
#pragma unroll
      for (int v = 0; v < h; ++v)
        x[v] = ((lane & o) ? x[v + h] : x[v]) + __shfl_xor_sync(0xffffffffu, (lane & o) ? x[v] : x[v + h], o);
    } else {
      x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
    }
  }
}

template <typename Tin, int R4>   // R4: groups of 32 rows of dk and columns of dv
__global__ void __launch_bounds__(GTHREADS) delta_chunk_grad_kernel(ChunkArgs<Tin> p) {
  extern __shared__ __align__(16) float sm[];
  constexpr int WARPS = GTHREADS / 32, MP = GradSmem::MP;
  static_assert(CB == 4 * WARPS && CB == 32, "a warp takes four tokens, the gates are one warp's");
  const int dk = p.dk_, dv = p.dv_, N = p.N, tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const GradSmem L_(dk, dv);
  const int ms = L_.ms, ks = L_.ks;
  float *S0s = sm + L_.S0, *X1s = sm + L_.X1, *Q = sm + L_.Q, *K = sm + L_.K;
  float *D = sm + L_.D, *U = sm + L_.U, *R = sm + L_.R, *Mq = sm + L_.Mq, *Mk = sm + L_.Mk;
  __shared__ double G[CB];
  __shared__ float red[WARPS], rows[2][CB], psum[WARPS][CB], corner[CB];
  const size_t bh = blockIdx.y;
  const int ch = blockIdx.x, t0 = ch * CB, n = min(CB, N - t0), nch = gridDim.x;
  const size_t mat = (size_t)dk * dv, tok = bh * N + t0;
  const float* S0 = p.Sc + (bh * nch + ch) * mat;
  const float* X1 = p.Xc + (bh * nch + ch) * mat;

  if (dv % 4 == 0) {   // (four floats at a time: 128 x 128 alone take 33,000 copies of one)
    const int vecs = dv / 4, rows = GTHREADS / vecs, rest = GTHREADS - rows * vecs;
    int r = tid / vecs, c = tid - r * vecs;
    for (int e = tid; e < dk * vecs; e += GTHREADS) {
      copy_async16(S0s + r * ms + 4 * c, S0 + 4 * e);
      copy_async16(X1s + r * ms + 4 * c, X1 + 4 * e);
      r += rows;
      c += rest;
      if (c >= vecs) { c -= vecs; ++r; }
    }
    for (int r = tid; r < dk; r += GTHREADS)
      for (int c = dv; c < ms; ++c) S0s[r * ms + c] = X1s[r * ms + c] = 0.f;
  } else {
    for (int r = warp; r < dk; r += WARPS)
      for (int c = lane; c < ms; c += 32) {
        if (c < dv) {
          copy_async4(S0s + r * ms + c, S0 + (size_t)r * dv + c);
          copy_async4(X1s + r * ms + c, X1 + (size_t)r * dv + c);
        } else {
          S0s[r * ms + c] = X1s[r * ms + c] = 0.f;
        }
      }
  }
  // tokens warp + 8 i: every load before the first use
  Tin qv[4][R4], kv[4][R4], dov[4][R4], bv[4];
  float evv[4][R4], duv[4][R4];
  const Tin zero = from_f<Tin>(0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = warp + WARPS * i;
    const bool in = t < n;
    bv[i] = in ? p.beta[tok + t] : zero;
#pragma unroll
    for (int b = 0; b < R4; ++b) {
      const int r = lane + 32 * b;
      const size_t ak = (tok + t) * dk + r, av = (tok + t) * dv + r;
      qv[i][b] = in && r < dk ? p.q[ak] : zero;
      kv[i][b] = in && r < dk ? p.k[ak] : zero;
      dov[i][b] = in && r < dv ? p.dout[av] : zero;
      evv[i][b] = in && r < dv ? p.ev[av] : 0.f;
      duv[i][b] = in && r < dv ? p.duv[av] : 0.f;
    }
  }
  const Tin gv = p.g != nullptr && lane < n ? p.g[tok + lane] : zero;
  constexpr int UX = R4 == 4 ? 4 : 8;   // loads in flight, beside the rows in registers
  float xs = 0.f;   // <X1, S0>
  if (mat % 4 == 0) {
#pragma unroll UX
    for (int e = 4 * tid; e < (int)mat; e += 4 * GTHREADS)
      xs = dot4(*reinterpret_cast<const float4*>(X1 + e), *reinterpret_cast<const float4*>(S0 + e), xs);
  } else {
#pragma unroll 8
    for (int e = tid; e < (int)mat; e += GTHREADS) xs = fmaf(X1[e], S0[e], xs);
  }
  if (warp == 0) {
    // exp(-200) is 0 in float32: a cleared state keeps G finite
    const float gi = to_f(gv);
    double acc = gi < -200.f ? -200.0 : (double)gi;   // NaN stays
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, acc, o);
      if (lane >= o) acc += y;
    }
    G[lane] = acc;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = warp + WARPS * i;
    const float bt = to_f(bv[i]);
    float db = 0.f;
#pragma unroll
    for (int b = 0; b < R4; ++b) {
      const int r = lane + 32 * b;
      if (r < ks) {
        Q[t * ks + r] = to_f(qv[i][b]);
        K[t * ks + r] = to_f(kv[i][b]);
      }
      if (r < ms) {
        const float rv = bt * duv[i][b];
        D[t * ms + r] = p.scale * to_f(dov[i][b]);
        U[t * ms + r] = bt * evv[i][b];
        R[t * ms + r] = rv;
        if (t < n && r < dv) p.dv[(tok + t) * dv + r] = from_f<Tin>(rv);
      }
      db = fmaf(duv[i][b], evv[i][b], db);
    }
    for (int o = 16; o > 0; o >>= 1) db += __shfl_xor_sync(0xffffffffu, db, o);
    if (lane == 0 && t < n) p.dbeta[tok + t] = from_f<Tin>(db);
    // a full last group leaves the row's last four floats to this
    if (32 * R4 + lane < ks) Q[t * ks + 32 * R4 + lane] = K[t * ks + 32 * R4 + lane] = 0.f;
    if (32 * R4 + lane < ms) D[t * ms + 32 * R4 + lane] = U[t * ms + 32 * R4 + lane] = R[t * ms + 32 * R4 + lane] = 0.f;
  }
  for (int o = 16; o > 0; o >>= 1) xs += __shfl_xor_sync(0xffffffffu, xs, o);
  if (lane == 0) red[warp] = xs;
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  auto at4 = [](const float* x) { return *reinterpret_cast<const float4*>(x); };
  const int i0 = warp * 4;
  float pairs[4];   // the pairs' terms of dg
  {   // Mq, Mk: row i = lane, columns j = i0 + a; all zero where those lie behind n
    const int i = lane, dv_in = i0 < n ? dv : 0, dk_in = i0 < n ? dk : 0;
    float mq[4] = {0.f, 0.f, 0.f, 0.f}, mk[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int c = 0; c < dv_in; c += 4) {
      const float4 d = at4(D + i * ms + c), r = at4(R + i * ms + c);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const float4 u = at4(U + (i0 + a) * ms + c);
        mq[a] = dot4(d, u, mq[a]);
        mk[a] = dot4(r, u, mk[a]);
      }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int j = i0 + a;
      const float f = j <= i ? expf((float)(G[i] - G[j])) : 0.f;
      mq[a] = j <= i ? mq[a] * f : 0.f;
      mk[a] = j < i ? -mk[a] * f : 0.f;
    }
    *reinterpret_cast<float4*>(Mq + i * MP + i0) = make_float4(mq[0], mq[1], mq[2], mq[3]);
    *reinterpret_cast<float4*>(Mk + i * MP + i0) = make_float4(mk[0], mk[1], mk[2], mk[3]);
    if (p.dg != nullptr) {
      float qk[4] = {0.f, 0.f, 0.f, 0.f}, kk[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
      for (int c = 0; c < dk_in; c += 4) {
        const float4 x = at4(Q + i * ks + c), y = at4(K + i * ks + c);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const float4 k = at4(K + (i0 + a) * ks + c);
          qk[a] = dot4(x, k, qk[a]);
          kk[a] = dot4(y, k, kk[a]);
        }
      }
#pragma unroll
      for (int a = 0; a < 4; ++a) pairs[a] = i0 + a < i ? fmaf(mq[a], qk[a], mk[a] * kk[a]) : 0.f;
      psum[warp][i] = (pairs[0] + pairs[1]) + (pairs[2] + pairs[3]);
    }
  }
  __syncthreads();
  if (p.dg != nullptr) {   // the sums over j < t = i0 + a of row i = lane, then over the rows from t on
    float below = 0.f;
    for (int w = 0; w < warp; ++w) below += psum[w][lane];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float x = pairs[a];
      pairs[a] = lane >= i0 + a ? below : 0.f;
      below += x;
    }
    lane_sums<4>(pairs, lane);
    if ((lane & 7) == 0) corner[i0 + lane / 8] = pairs[0];
  }
  // a lane holds rows lane + 32 b of four tokens' gradients
  float dqv[4][R4], dkr[4][R4], dkw[4][R4];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < R4; ++b) dqv[a][b] = dkr[a][b] = dkw[a][b] = 0.f;
#pragma unroll 2
  for (int c = 0; c < dv; c += 4) {
    float4 m[R4], x[R4];
#pragma unroll
    for (int b = 0; b < R4; ++b) {
      const int r = min(lane + 32 * b, dk - 1);   // rows behind dk are not stored
      m[b] = at4(S0s + r * ms + c);
      x[b] = at4(X1s + r * ms + c);
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float4 d = at4(D + (i0 + a) * ms + c), r = at4(R + (i0 + a) * ms + c), u = at4(U + (i0 + a) * ms + c);
#pragma unroll
      for (int b = 0; b < R4; ++b) {
        dqv[a][b] = dot4(d, m[b], dqv[a][b]);
        dkr[a][b] = dot4(r, m[b], dkr[a][b]);
        dkw[a][b] = dot4(u, x[b], dkw[a][b]);
      }
    }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const float gam = expf((float)G[i0 + a]), rho = expf((float)(G[CB - 1] - G[i0 + a]));
#pragma unroll
    for (int b = 0; b < R4; ++b) { dqv[a][b] *= gam; dkr[a][b] *= -gam; dkw[a][b] *= rho; }
  }
  if (p.dg != nullptr) {   // the states' part of dg: reads of the four tokens, then their writes
    float x[8];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      x[a] = x[4 + a] = 0.f;
#pragma unroll
      for (int b = 0; b < R4; ++b) {
        const int r = lane + 32 * b;
        if (r >= dk) continue;
        const float k = K[(i0 + a) * ks + r];
        x[a] = fmaf(Q[(i0 + a) * ks + r], dqv[a][b], fmaf(k, dkr[a][b], x[a]));
        x[4 + a] = fmaf(k, dkw[a][b], x[4 + a]);
      }
    }
    lane_sums<8>(x, lane);
    if ((lane & 3) == 0) rows[lane / 16][i0 + (lane >> 2 & 3)] = x[0];
  }
#pragma unroll 2
  for (int j = 0; j < n; ++j) {   // rows and columns of Mq and Mk behind n are zero
    float kj[R4], qj[R4];
#pragma unroll
    for (int b = 0; b < R4; ++b) {
      const int r = min(lane + 32 * b, dk - 1);
      kj[b] = K[j * ks + r];
      qj[b] = Q[j * ks + r];
    }
    const float4 wq4 = at4(Mq + j * MP + i0), wk4 = at4(Mk + j * MP + i0);
    const float wq[4] = {wq4.x, wq4.y, wq4.z, wq4.w}, wk[4] = {wk4.x, wk4.y, wk4.z, wk4.w};
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float mq = Mq[(i0 + a) * MP + j], mk = Mk[(i0 + a) * MP + j];
#pragma unroll
      for (int b = 0; b < R4; ++b) {
        dqv[a][b] = fmaf(mq, kj[b], dqv[a][b]);
        dkr[a][b] = fmaf(mk, kj[b], dkr[a][b]);
        dkw[a][b] = fmaf(wq[a], qj[b], fmaf(wk[a], kj[b], dkw[a][b]));
      }
    }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int i = i0 + a;
#pragma unroll
    for (int b = 0; b < R4; ++b) {
      const int r = lane + 32 * b;
      if (r >= dk || i >= n) continue;
      p.dq[(tok + i) * dk + r] = from_f<Tin>(dqv[a][b]);
      p.dk[(tok + i) * dk + r] = from_f<Tin>(dkr[a][b] + dkw[a][b]);
    }
  }
  __syncthreads();
  if (warp == 0 && p.dg != nullptr) {
    float x1s0 = 0.f;
    for (int w = 0; w < WARPS; ++w) x1s0 += red[w];
    // reads of the tokens from this one on, writes of those before it
    float reads = rows[0][lane], writes = rows[1][lane];
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_down_sync(0xffffffffu, reads, o), y = __shfl_up_sync(0xffffffffu, writes, o);
      if (lane + o < 32) reads += x;
      if (lane >= o) writes += y;
    }
    writes = __shfl_up_sync(0xffffffffu, writes, 1);
    if (lane == 0) writes = 0.f;
    if (lane < n) p.dg[tok + lane] = from_f<Tin>((reads + corner[lane]) + fmaf(expf((float)G[CB - 1]), x1s0, writes));
  }
}

size_t chunk_grad_smem(int dk, int dv) { return sizeof(float) * GradSmem(dk, dv).floats; }

// ------------------------------------------------------------------ single tokens
// One token per row; a CTA takes VC columns of one row's head: lanes cover the
// columns four at a time, the other threads split dk.  The state slice is
// read into registers in one sweep, the two dot products over dk (S^T k, and
// q.S' from q.S and q.k) are joined through shared memory in one exchange,
// and the slice is written back: bound by the state's bytes (247 rows of 16
// heads of 128: 522 MB in 95 us, 5.5 TB/s).  To find the rows that share a
// state every CTA reads all B slots, from L2: 1 KB beside 32 KB of state at 256
// rows, as much as the state at 8192.
constexpr int STHREADS = 128;

template <typename Tin, typename Tout, int VC>
__global__ void __launch_bounds__(STHREADS, 7)
    delta_step_kernel(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
                      const Tin* __restrict__ g, const Tin* __restrict__ beta,
                      const int* __restrict__ slots, int n_slots, float* __restrict__ S,
                      Tout* __restrict__ out, int B, int H, int dk, int dv, float scale) {
  constexpr int lanes = VC / 4, groups = STHREADS / lanes, SROWS = DMAX / groups;   // SROWS: rows of a thread
  __shared__ float ks[DMAX], qs[DMAX];
  __shared__ float part[2][STHREADS][4];   // partial S^T k and S^T q of four columns
  __shared__ float qk_s;
  __shared__ int next_s;
  static_assert(DMAX == STHREADS, "a thread brings one row of k and q");
  const int h = blockIdx.y, c0 = blockIdx.z * VC, tid = threadIdx.x;
  int b = blockIdx.x;
  const int slot = slots != nullptr ? slots[b] : b;
  if (slot < 0 || slot >= n_slots) return;
  const int cl = tid % lanes, gr = tid / lanes, c = c0 + 4 * cl;
  const bool vec = (dv & 3) == 0;
  // every load of the row before the first wait
  Tin kr_, qr_, vr_[4], gr_, br_;
  const Tin zero = from_f<Tin>(0.f);
  auto fetch = [&]() {
    const size_t tok = (size_t)b * H + h;
    kr_ = tid < dk ? k[tok * dk + tid] : zero;
    qr_ = tid < dk ? q[tok * dk + tid] : zero;
#pragma unroll
    for (int j = 0; j < 4; ++j) vr_[j] = c + j < dv ? v[tok * dv + c + j] : zero;
    gr_ = g != nullptr ? g[tok] : zero;
    br_ = beta[tok];
  };
  fetch();
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
  int next = B;
  if (slots != nullptr) {   // a sequence's first row takes all of its rows, in order
    if (tid == 0) next_s = B;
    __syncthreads();
    int before = 0, after = B;
    for (int j = tid; j < B; j += STHREADS) {
      if (slots[j] != slot) continue;
      if (j < b) before = 1;
      else if (j > b) after = min(after, j);
    }
    if (after < B) atomicMin(&next_s, after);
    if (__syncthreads_or(before)) return;
    next = next_s;
  }
  for (;;) {
    const size_t tok = (size_t)b * H + h;
    ks[tid] = to_f(kr_);
    qs[tid] = to_f(qr_);
    __syncthreads();
    const float a = expf(to_f(gr_)), bt = to_f(br_);
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
        u[j] = bt * (to_f(vr_[j]) - a * pks[j]);
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
    if (next >= B) break;
    // the next row of the same sequence
    b = next;
    fetch();
    if (tid == 0) next_s = B;
    __syncthreads();   // every thread is behind its reads of ks, qs and next_s
    int after = B;
    for (int j = b + 1 + tid; j < B && after == B; j += STHREADS)
      if (slots[j] == slot) after = j;
    if (after < B) atomicMin(&next_s, after);
    __syncthreads();
    next = next_s;
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

#define TTT_BY_ROWS(ROWS, CALL)               \
  switch (((ROWS) + 31) / 32) {               \
    case 1: CALL(1); break;                   \
    case 2: CALL(2); break;                   \
    case 3: CALL(3); break;                   \
    default: CALL(4); break;                  \
  }

// Helpers pay while every CTA has an SM for itself: forward over 1,024 float32
// tokens, 8 heads of 32 / 64 / 128: 97 / 130 / 201 us alone, 75 / 102 / 159
// helped.  Beyond that they take issue slots from the second CTA: 64 heads of
// 64 / 128: 177 / 575 us alone, 203 / 631 helped (64 heads of 32 are 128 CTAs).
template <int R4, bool HELP, typename... KArgs, typename... Args>
int launch_cols(void (*kernel)(KArgs...), dim3 grid, cudaStream_t stream, Args... args) {
  constexpr size_t smem = stage_bytes<R4, HELP>();
  static std::atomic<uint64_t> attr{};
  if (smem > 48 * 1024 && allow_dynamic_smem(kernel, (int)smem, attr)) return -1;
  return launch_plain(kernel, grid, dim3(HELP ? 2 * THREADS : THREADS), smem, stream, args...) == cudaSuccess ? 0 : -1;
}
// heads x slices of columns x directions
dim3 cols_grid(const DeltaLaunch& p, int directions) {
  return dim3((unsigned)(p.B * p.H), (unsigned)((p.dv + COLS - 1) / COLS), (unsigned)directions);
}
bool helped(const DeltaLaunch& p, const dim3& g) { return (long long)g.x * g.y * g.z <= p.sms; }

template <typename Tin, typename Tout>
int rec_launch(const DeltaLaunch& p, cudaStream_t stream) {
  const dim3 grid = cols_grid(p, 1);
  const bool help = helped(p, grid);
  int err = 0;
  prof_before(K_DELTA_REC, stream);
#define TTT_REC(R4)                                                                                \
  err = help ? launch_cols<R4, true>(delta_rec_kernel<Tin, Tout, R4, true>, grid, stream,          \
                                     TTT_REC_ARGS)                                                 \
             : launch_cols<R4, false>(delta_rec_kernel<Tin, Tout, R4, false>, grid, stream,        \
                                      TTT_REC_ARGS)
#define TTT_REC_ARGS                                                                               \
  (const Tin*)p.q, (const Tin*)p.k, (const Tin*)p.v, (const Tin*)p.g, (const Tin*)p.beta, p.S,     \
      (Tout*)p.out, p.N, p.dk, p.dv, p.scale
  TTT_BY_ROWS(p.dk, TTT_REC)
#undef TTT_REC_ARGS
#undef TTT_REC
  prof_after(K_DELTA_REC, stream);
  return err;
}

template <typename Tin>
int bwd_launch(const DeltaBwdLaunch& L, cudaStream_t stream) {
  const DeltaLaunch& p = L.f;
  const int BH = p.B * p.H, nch = tiles_of(p.N, CB);
  const DeltaBwdWorkspace w = delta_rec_bwd_layout(BH, p.N, p.dk, p.dv);
  float* ev = reinterpret_cast<float*>(L.ws + w.ev);
  float* du = reinterpret_cast<float*>(L.ws + w.du);
  float* Sc = reinterpret_cast<float*>(L.ws + w.Sc);
  float* Xc = reinterpret_cast<float*>(L.ws + w.Xc);
  const StatesArgs<Tin> states{(const Tin*)p.q, (const Tin*)p.k, (const Tin*)p.v, (const Tin*)L.dout,
                               (const Tin*)p.g, (const Tin*)p.beta, L.S0, L.dS_end, L.dS0, ev, du, Sc, Xc,
                               p.N, p.dk, p.dv, p.scale};
  const dim3 grid = cols_grid(p, 2);
  const bool help = helped(p, grid);
  int err = 0;
  prof_before(K_DELTA_STATES, stream);
#define TTT_STATES(R4)                                                                             \
  err = help ? launch_cols<R4, true>(delta_states_kernel<Tin, R4, true>, grid, stream, states)     \
             : launch_cols<R4, false>(delta_states_kernel<Tin, R4, false>, grid, stream, states)
  TTT_BY_ROWS(p.dk, TTT_STATES)
#undef TTT_STATES
  prof_after(K_DELTA_STATES, stream);
  if (err) return -1;
  const size_t smem = chunk_grad_smem(p.dk, p.dv);
  void (*kfn)(ChunkArgs<Tin>) = nullptr;
  static std::atomic<uint64_t> attr[4] = {};
  const int widest = std::max(p.dk, p.dv);
#define TTT_GRAD(R4) kfn = delta_chunk_grad_kernel<Tin, R4>
  TTT_BY_ROWS(widest, TTT_GRAD)
#undef TTT_GRAD
  if (allow_dynamic_smem(kfn, (int)chunk_grad_smem(DMAX, DMAX), attr[(widest - 1) / 32])) return -1;
  ChunkArgs<Tin> a{(const Tin*)p.q, (const Tin*)p.k, (const Tin*)L.dout, (const Tin*)p.g,
                   (const Tin*)p.beta, ev, du, Sc, Xc, (Tin*)L.dq, (Tin*)L.dk, (Tin*)L.dv,
                   (Tin*)L.dg, (Tin*)L.dbeta, p.N, p.dk, p.dv, p.scale};
  if (nch == 0) return 0;
  // grid.y is limited to 65535: more heads go in slices (b0 ends at BH: a step
  // of 65535 would pass 2^31 behind the last heads that an int counts)
  for (int b0 = 0, nb; b0 < BH; b0 += nb) {
    nb = std::min(65535, BH - b0);
    ChunkArgs<Tin> s = a;
    const size_t t = (size_t)b0 * p.N, mat = (size_t)p.dk * p.dv;
    s.q += t * p.dk; s.k += t * p.dk; s.dq += t * p.dk; s.dk += t * p.dk;
    s.dout += t * p.dv; s.dv += t * p.dv; s.ev += t * p.dv; s.duv += t * p.dv;
    s.beta += t; s.dbeta += t;
    if (s.g != nullptr) { s.g += t; s.dg += t; }
    s.Sc += (size_t)b0 * nch * mat;
    s.Xc += (size_t)b0 * nch * mat;
    prof_before(K_DELTA_GRAD, stream);
    const cudaError_t e = launch_plain(kfn, dim3((unsigned)nch, (unsigned)nb), dim3(GTHREADS), smem, stream, s);
    prof_after(K_DELTA_GRAD, stream);
    if (e != cudaSuccess) return -1;
  }
  return 0;
}

}  // namespace

int launch_delta_rec(const DeltaLaunch& p, cudaStream_t stream) {
  if (p.in_bf16) {
    if (p.out_bf16) return rec_launch<__nv_bfloat16, __nv_bfloat16>(p, stream);
    return rec_launch<__nv_bfloat16, float>(p, stream);
  }
  if (p.out_bf16) return rec_launch<float, __nv_bfloat16>(p, stream);
  return rec_launch<float, float>(p, stream);
}

DeltaBwdWorkspace delta_rec_bwd_layout(int BH, int N, int dk, int dv) {
  DeltaBwdWorkspace w{};
  size_t at = 256;
  auto take = [&](size_t floats) {
    const size_t o = at;
    at += (floats * sizeof(float) + 255) / 256 * 256;
    return o;
  };
  const size_t nch = tiles_of(N, CB), mat = (size_t)dk * dv;
  w.ev = take((size_t)BH * N * dv);
  w.du = take((size_t)BH * N * dv);
  w.Sc = take((size_t)BH * nch * mat);
  w.Xc = take((size_t)BH * nch * mat);
  w.total = at;
  return w;
}

int launch_delta_rec_bwd(const DeltaBwdLaunch& L, cudaStream_t stream) {
  return L.f.in_bf16 ? bwd_launch<__nv_bfloat16>(L, stream) : bwd_launch<float>(L, stream);
}

int launch_delta_step(const DeltaLaunch& p, const int* slots, int n_slots, cudaStream_t stream) {
  // columns of a CTA: a slice of 32 is one 128-byte line of every state row and
  // 16 KB in all, so that a dozen CTAs of an SM keep loads and stores mixed;
  // half of it where rows and heads do not fill the device
  const int vc = (long long)p.B * p.H * ((p.dv + 31) / 32) < 4 * p.sms ? 16 : 32;
  const dim3 grid((unsigned)p.B, (unsigned)p.H, (unsigned)((p.dv + vc - 1) / vc));
#define TTT_STEP_VC(TI, TO, VC)                                                                    \
  e = launch_plain(delta_step_kernel<TI, TO, VC>, grid, dim3(STHREADS), 0, stream, (const TI*)p.q,  \
                   (const TI*)p.k, (const TI*)p.v, (const TI*)p.g, (const TI*)p.beta, slots,        \
                   n_slots, p.S, (TO*)p.out, p.B, p.H, p.dk, p.dv, p.scale)
#define TTT_STEP(TI, TO)                     \
  do {                                       \
    if (vc == 16) TTT_STEP_VC(TI, TO, 16);   \
    else TTT_STEP_VC(TI, TO, 32);            \
  } while (0)
  cudaError_t e = cudaSuccess;
  prof_before(K_DELTA_STEP, stream);
  if (p.in_bf16) {
    if (p.out_bf16) TTT_STEP(__nv_bfloat16, __nv_bfloat16);
    else TTT_STEP(__nv_bfloat16, float);
  } else {
    if (p.out_bf16) TTT_STEP(float, __nv_bfloat16);
    else TTT_STEP(float, float);
  }
#undef TTT_STEP
#undef TTT_STEP_VC
  prof_after(K_DELTA_STEP, stream);
  return e == cudaSuccess ? 0 : -1;
}

}  // namespace ttt
