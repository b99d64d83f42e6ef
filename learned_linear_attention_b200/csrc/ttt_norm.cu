// ttt_norm.cu -- row norm with weight, gate and scaled residual, and its
// backward pass:  out = res + scale * x r(x) * w * act(z), row by row.
//
// A row belongs to a group of T threads (4 to 32 lanes of a warp, or a whole
// CTA of 256), each holding the same V 16-byte vectors of every row it meets,
// so a row is read once, its sum of squares is a few shuffles, and the
// weight's gradient is summed in registers over the CTA's rows.  Bound by
// memory: 262,144 rows of 128 bf16 with gate and residual 45 us, 6.0 TB/s, their
// gradients 68 us, 5.0.
#include <algorithm>
#include <type_traits>

#include "kernels.h"

namespace ttt {

namespace {

constexpr int THREADS = 256;

template <typename T>
struct Vec;   // 16 bytes of T; kept as they are until they are worked on
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static TTT_DEVICE_INLINE void get(const uint4& t, float* x) {
    x[0] = __uint_as_float(t.x); x[1] = __uint_as_float(t.y); x[2] = __uint_as_float(t.z); x[3] = __uint_as_float(t.w);
  }
  static TTT_DEVICE_INLINE void store(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static TTT_DEVICE_INLINE void get(const uint4& t, float* x) {
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[2 * i] = bf16lo(w[i]); x[2 * i + 1] = bf16hi(w[i]); }
  }
  static TTT_DEVICE_INLINE void store(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
};
template <typename E>
TTT_DEVICE_INLINE uint4 raw(const void* p, size_t at) {
  return *reinterpret_cast<const uint4*>(static_cast<const E*>(p) + at);
}

// Sum over the T threads of a row (several warps: through shared memory, by
// the whole CTA together).
template <int T>
TTT_DEVICE_INLINE float row_sum(float x, float* red) {
#pragma unroll
  for (int o = 1; o < (T < 32 ? T : 32); o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if constexpr (T > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.f;
    const float* mine = red + threadIdx.x / T * (T / 32);
#pragma unroll
    for (int w = 0; w < T / 32; ++w) x += mine[w];
  }
  return x;
}

// float32 rows take expf, with which the sigmoid is good to a few 2^-24.  bf16 ones
// take __expf, off by (2 + 1.16 |z|) 2^-23 at most (3.7e-6 of the sigmoid at |z| =
// 80), which the 2^-9 of their results hides: with expf they take 49 us in the
// place of 45 (262,144 rows of 128 with gate and residual), their gradients 78 in
// the place of 68.  __fdividef(1, y) is 0 for y > 2^126, where sigmoid is below
// float32's normal range; z = -inf gives 0 and NaN stays.
template <typename E>
TTT_DEVICE_INLINE float sigmoidf(float z) {
  const float e = std::is_same<E, float>::value ? expf(-z) : __expf(-z);
  return __fdividef(1.f, 1.f + e);
}

struct NormArgs {
  const void *x, *z, *res, *dout;
  const float* w;
  void *out, *dx, *dz;
  float* part;   // partial sums of dw [gridDim.x][D]
  long long rows;
  int D, kind, gate;
  float eps, scale, inv_d;
};

// r of a row with sum of squares ss; `fixed` where r does not depend on x
TTT_DEVICE_INLINE float row_r(const NormArgs& a, float ss, bool& fixed) {
  if (a.kind == 0) {
    fixed = false;
    // rsqrtf with one Newton step, which an infinite sum would make NaN
    const float m = fmaf(ss, a.inv_d, a.eps), y = rsqrtf(m);
    return m < 3e38f ? fmaf(0.5f * y, fmaf(-m * y, y, 1.f), y) : y;
  }
  const float len = sqrtf(ss);
  fixed = !(len > a.eps);
  return 1.f / (fixed && len == len ? a.eps : len);
}

// A thread's vectors of a row of up to three tensors.  Where it holds one or
// two, the next row's are on their way while this one is worked on: the work
// (two or three transcendental functions an element) takes as long as the
// loads, and four CTAs an SM alone would leave the memory idle meanwhile.
template <typename E, int T, int V>
struct Row {
  uint4 v[3][V];
  TTT_DEVICE_INLINE void load(const NormArgs& a, const void* p0, const void* p1, const void* p2, long long row,
                              int t) {
    constexpr int N = Vec<E>::N;
    const size_t at = (size_t)row * a.D;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * T + t) * N;
      v[0][i] = v[1][i] = v[2][i] = make_uint4(0, 0, 0, 0);
      if (row >= a.rows || c >= a.D) continue;
      v[0][i] = raw<E>(p0, at + c);
      if (p1 != nullptr) v[1][i] = raw<E>(p1, at + c);
      if (p2 != nullptr) v[2][i] = raw<E>(p2, at + c);
    }
  }
};
template <typename E, int T, int V, typename F>
TTT_DEVICE_INLINE void for_rows(const NormArgs& a, const void* p0, const void* p1, const void* p2, F work) {
  constexpr int GROUPS = THREADS / T;
  const int t = threadIdx.x % T, gr = threadIdx.x / T;
  // a warp's groups leave the loop together: the bound is on the CTA's first row
  const long long step = (long long)gridDim.x * GROUPS;
  long long r0 = (long long)blockIdx.x * GROUPS;
  Row<E, T, V> cur;
  if constexpr (V <= 2) {
    if (r0 < a.rows) cur.load(a, p0, p1, p2, r0 + gr, t);
    for (; r0 < a.rows; r0 += step) {
      Row<E, T, V> next;
      next.load(a, p0, p1, p2, r0 + step + gr, t);
      work(cur, r0 + gr);
      cur = next;
    }
  } else {
    for (; r0 < a.rows; r0 += step) {
      cur.load(a, p0, p1, p2, r0 + gr, t);
      work(cur, r0 + gr);
    }
  }
}
template <int V>
constexpr int ctas() { return V == 1 ? 4 : 1; }

template <typename E, int T, int V>
__global__ void __launch_bounds__(THREADS, ctas<V>()) norm_fwd_kernel(NormArgs a) {
  constexpr int N = Vec<E>::N;
  __shared__ float red[THREADS / 32];
  const int t = threadIdx.x % T;
  float w[V][N];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * T + t) * N;
#pragma unroll
    for (int i = 0; i < N; ++i) w[v][i] = a.scale * (a.w != nullptr && c < a.D ? a.w[c + i] : 1.f);
  }
  for_rows<E, T, V>(a, a.x, a.gate != 0 ? a.z : nullptr, a.res, [&](const Row<E, T, V>& in, long long row) {
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float x[N];
      Vec<E>::get(in.v[0][v], x);
#pragma unroll
      for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
    }
    bool fixed;
    const float r = row_r(a, row_sum<T>(ss, red), fixed);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * T + t) * N;
      if (row >= a.rows || c >= a.D) continue;
      float x[N], z[N], rs[N];
      Vec<E>::get(in.v[0][v], x);
      Vec<E>::get(in.v[1][v], z);
      Vec<E>::get(in.v[2][v], rs);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float y = x[i] * r * w[v][i];
        if (a.gate != 0) {
          const float s = sigmoidf<E>(z[i]);
          y *= a.gate == 1 ? z[i] * s : s;
        }
        x[i] = a.res != nullptr ? y + rs[i] : y;
      }
      Vec<E>::store(static_cast<E*>(a.out) + (size_t)row * a.D + c, x);
    }
  });
}

// With n = x r, p = scale dout:  dz = p n w act'(z),  dw = sum p act(z) n,
// dn = p w act(z),  dx = r (dn - n mean(dn n))  (RMS; for L2 the sum instead
// of the mean, and no such term where r is 1 / eps).
template <typename E, int T, int V>
__global__ void __launch_bounds__(THREADS, V == 1 ? 3 : 1) norm_bwd_kernel(NormArgs a) {
  constexpr int N = Vec<E>::N, GROUPS = THREADS / T;
  __shared__ float red[THREADS / 32];
  extern __shared__ float acc_s[];   // [GROUPS][D] where dw is wanted
  const int t = threadIdx.x % T, gr = threadIdx.x / T;
  float dw[V][N], w[V][N];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * T + t) * N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dw[v][i] = 0.f;
      w[v][i] = a.w != nullptr && c < a.D ? a.w[c + i] : 1.f;
    }
  }
  for_rows<E, T, V>(a, a.x, a.dout, a.gate != 0 ? a.z : nullptr, [&](const Row<E, T, V>& in, long long row) {
    float ss = 0.f, dot = 0.f, dn[V][N];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float x[N];
      Vec<E>::get(in.v[0][v], x);
#pragma unroll
      for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
    }
    bool fixed;
    const float r = row_r(a, row_sum<T>(ss, red), fixed);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * T + t) * N;
      float x[N], z[N], d[N];
      Vec<E>::get(in.v[0][v], x);
      Vec<E>::get(in.v[1][v], d);
      Vec<E>::get(in.v[2][v], z);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float n = x[i] * r;
        float p = a.scale * d[i];
        if (a.gate != 0) {
          const float s = sigmoidf<E>(z[i]);
          // act' is s (1 + z (1 - s)) for silu, s (1 - s) for the sigmoid
          const float act = a.gate == 1 ? z[i] * s : s;
          const float dact = a.gate == 1 ? fmaf(act, 1.f - s, s) : fmaf(-s, s, s);
          z[i] = p * n * w[v][i] * dact;
          p *= act;
        }
        dw[v][i] = fmaf(p, n, dw[v][i]);
        dn[v][i] = p * w[v][i];
        dot = fmaf(dn[v][i], n, dot);
      }
      if (a.gate != 0 && row < a.rows && c < a.D) Vec<E>::store(static_cast<E*>(a.dz) + (size_t)row * a.D + c, z);
    }
    dot = row_sum<T>(dot, red);
    const float m = fixed ? 0.f : a.kind == 0 ? dot * a.inv_d : dot;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * T + t) * N;
      if (row >= a.rows || c >= a.D) continue;
      float x[N];
      Vec<E>::get(in.v[0][v], x);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = r * fmaf(-m, x[i] * r, dn[v][i]);
      Vec<E>::store(static_cast<E*>(a.dx) + (size_t)row * a.D + c, x);
    }
  });
  if (a.part == nullptr) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * T + t) * N;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c < a.D) acc_s[(size_t)gr * a.D + c + i] = dw[v][i];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.D; c += THREADS) {
    float s = 0.f;
    for (int j = 0; j < GROUPS; ++j) s += acc_s[(size_t)j * a.D + c];
    a.part[(size_t)blockIdx.x * a.D + c] = s;
  }
}

// dw[c] = sum of the CTAs' partial sums, in their order: 32 columns and 32
// interleaved runs of partial sums to a CTA.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int n, int D,
                                                       float* __restrict__ dw) {
  __shared__ float s[32][33];
  const int l = threadIdx.x % 32, j0 = threadIdx.x / 32, c = blockIdx.x * 32 + l;
  float acc = 0.f;
  if (c < D)
#pragma unroll 8
    for (int j = j0; j < n; j += 32) acc += part[(size_t)j * D + c];
  s[j0][l] = acc;
  __syncthreads();
  if (j0 == 0 && c < D) {
#pragma unroll
    for (int j = 1; j < 32; ++j) acc += s[j][l];
    dw[c] = acc;
  }
}

struct Shape { int T, V; };
// Threads of a row and vectors of a thread: few threads keep several rows'
// loads in flight in a warp, one vector a thread keeps accesses whole and the
// next row in registers.  A warp takes a row of up to four float32 vectors a
// thread (65,536 rows of 512 with gate and residual 82 us, against 97 for 128
// threads a row; without them 50 against 70; gradients 120 against 113 and 82
// against 84).  bf16 vectors hold twice the values: up to two a thread (65,536
// rows of 512 with gate and residual 47 us against 64, gradients 79 against 133);
// rows of more go to several warps (32,768 rows of 1024 45 us, against 68 for a
// warp a row with four; gradients 76 against 95).
Shape norm_shape(int D, int per_vec) {
  const int nv = (D + per_vec - 1) / per_vec, most = per_vec == 4 ? 128 : 64;
  int T = 4;
  while (T < 32 && T < nv) T *= 2;
  while (T < 256 && nv > most && T < nv) T *= T == 32 ? 4 : 2;
  int V = 1;
  while (T * V < nv) V *= 2;
  return {T, V};
}

// `per_sm` CTAs an SM, 4 forward and 3 backward: as many as are resident where a
// thread holds one vector (see __launch_bounds__), so that all take the same
// number of rows.  With more vectors fewer are resident and the others follow.
int norm_grid(long long rows, int T, int sms, int per_sm) {
  const long long groups = THREADS / T;
  return (int)std::max<long long>(1, std::min<long long>((rows + groups - 1) / groups, (long long)sms * per_sm));
}

template <typename E, bool BWD>
int launch_t(const NormArgs& a, int grid, size_t smem, cudaStream_t stream) {
  const Shape s = norm_shape(a.D, Vec<E>::N);
#define TTT_NORM(T_, V_)                                                              \
  if (s.T == T_ && s.V == V_) {                                                       \
    const auto kernel = BWD ? norm_bwd_kernel<E, T_, V_> : norm_fwd_kernel<E, T_, V_>; \
    return launch_plain(kernel, dim3(grid), dim3(THREADS), smem, stream, a) == cudaSuccess ? 0 : -1; \
  }
  TTT_NORM(4, 1) TTT_NORM(8, 1) TTT_NORM(16, 1) TTT_NORM(32, 1) TTT_NORM(32, 2)
  TTT_NORM(256, 1) TTT_NORM(256, 2) TTT_NORM(256, 4)
  if constexpr (Vec<E>::N == 4) {   // the others that norm_shape gives for the type
    TTT_NORM(32, 4) TTT_NORM(256, 8)
  } else {
    TTT_NORM(128, 1)
  }
#undef TTT_NORM
  return -1;
}

NormArgs args_of(const NormLaunch& L) {
  NormArgs a{};
  a.x = L.x; a.z = L.z; a.res = L.res; a.dout = L.dout; a.w = L.w;
  a.out = L.out; a.dx = L.dx; a.dz = L.dz;
  a.rows = L.rows; a.D = L.D; a.kind = L.kind; a.gate = L.gate; a.eps = L.eps; a.scale = L.scale;
  a.inv_d = 1.f / (float)L.D;
  return a;
}

}  // namespace

int norm_bwd_parts(long long rows, int D, int bf16, int sms) {
  return norm_grid(rows, norm_shape(D, bf16 ? 8 : 4).T, sms, 3);
}

int launch_norm_fwd(const NormLaunch& L, int sms, cudaStream_t stream) {
  const NormArgs a = args_of(L);
  const int grid = norm_grid(L.rows, norm_shape(L.D, L.bf16 ? 8 : 4).T, sms, 4);
  prof_before(K_NORM, stream);
  const int r = L.bf16 ? launch_t<__nv_bfloat16, false>(a, grid, 0, stream)
                       : launch_t<float, false>(a, grid, 0, stream);
  prof_after(K_NORM, stream);
  return r;
}

int launch_norm_bwd(const NormLaunch& L, int sms, cudaStream_t stream) {
  NormArgs a = args_of(L);
  const int T = norm_shape(L.D, L.bf16 ? 8 : 4).T;
  const int grid = norm_bwd_parts(L.rows, L.D, L.bf16, sms);
  a.part = L.dw != nullptr ? L.part : nullptr;
  const size_t smem = a.part != nullptr ? (size_t)(THREADS / T) * L.D * sizeof(float) : 0;
  prof_before(K_NORM_BWD, stream);
  int r = L.bf16 ? launch_t<__nv_bfloat16, true>(a, grid, smem, stream) : launch_t<float, true>(a, grid, smem, stream);
  if (r == 0 && L.dw != nullptr &&
      launch_plain(norm_dw_kernel, dim3((L.D + 31) / 32), dim3(1024), 0, stream, a.part, grid, L.D, L.dw) != cudaSuccess)
    r = -1;
  prof_after(K_NORM_BWD, stream);
  return r;
}

}  // namespace ttt
