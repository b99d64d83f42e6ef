// delta_umma.cu -- gated delta rule on tensor cores: bf16, dk = dv = D = 64
// or 128, chunks of 128 tokens.
//
// With G the running sum of g in a chunk, gam_i = exp(G_i), Gam_ij = exp(G_i
// - G_j) and rho_i = exp(G_last - G_i), the recurrence of a chunk is
//   A_ij = beta_i Gam_ij k_i.k_j (j < i),   T = (I + A)^-1
//   W = T diag(beta gam) K,  Ut = T diag(beta) V,  U = Ut - W S0
//   O = scale (gam Q S0 + (Gam . Q K^T) U)          (lower triangle, with the diagonal)
//   S1 = gam_last S0 + (rho K)^T U = (gam_last I + Mc) S0 + Hc
//   Mc = -(rho K)^T W [D, D],  Hc = (rho K)^T Ut [D, D]
// so only the D x D recurrence S1 = gam_last S0 + Mc S0 + Hc runs in order
// (one product a chunk), and everything else is parallel over the chunks:
//   delta_prep_kernel   K, V -> W, Ut, Mc, Hc
//   delta_chain_kernel  Mc, Hc -> every chunk's start state, end state
//   delta_out_kernel    Q, K, W, Ut, start states -> O
#include <algorithm>

#include "delta_umma.cuh"

namespace ttt {

using namespace dl;

namespace {

// ------------------------------------------------------------------ inverse
// (I + A)^-1 in place, A strictly lower triangular [128][128] float32 in
// shared memory (rows LDA floats apart), by 256 threads: 16 x 16 diagonal
// blocks by substitution, one column a thread, then blocks of 16, 32 and 64
// joined two by two, T21 = -T22 (A21 T11).  Every factor is itself an
// inverse, so the intermediate values stay of the size of the result (the
// powers of A of a Neumann product do not).  A21 T11 waits in the unused
// block above the diagonal, so what is above the diagonal is not zero at the
// end.
constexpr int LDA = 132;

template <int S>
TTT_DEVICE_INLINE void join_blocks(float* A, int tid) {
  constexpr int RT = S / 16, CG = S / 4;
  const int p = tid / (4 * S), t = tid % (4 * S), cg = t % CG, r0 = t / CG * RT;
  float* T11 = A + p * 2 * S * (LDA + 1);
  float* A21 = T11 + S * LDA;
  float* T22 = A21 + S;
  float* Z = T11 + S;
  float4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto step = [&](const float* X, const float* Y, int k, float sign) {
    float4 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = *reinterpret_cast<const float4*>(Y + (k + i) * LDA + 4 * cg);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float4 x = *reinterpret_cast<const float4*>(X + (r0 + r) * LDA + k);
      const float xs[4] = {sign * x.x, sign * x.y, sign * x.z, sign * x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[r].x = fmaf(xs[i], y[i].x, acc[r].x);
        acc[r].y = fmaf(xs[i], y[i].y, acc[r].y);
        acc[r].z = fmaf(xs[i], y[i].z, acc[r].z);
        acc[r].w = fmaf(xs[i], y[i].w, acc[r].w);
      }
    }
  };
  // rows of T11 above a column are zero (its own upper part was zeroed with
  // its 16-blocks, or holds an earlier Z: skipped either way)
  auto tri = [&](const float* X, int k, int row) {   // X[row][k..k+3] with what is above the diagonal as 0
    float4 x = *reinterpret_cast<const float4*>(X + row * LDA + k);
    if (k > row) x.x = 0.f;
    if (k + 1 > row) x.y = 0.f;
    if (k + 2 > row) x.z = 0.f;
    if (k + 3 > row) x.w = 0.f;
    return x;
  };
  // Z = A21 T11, k from the column group's first row on
  for (int k = 4 * cg; k < S; k += 4) {
    float4 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = *reinterpret_cast<const float4*>(T11 + (k + i) * LDA + 4 * cg);
      if (k == 4 * cg) {   // the diagonal's own 4 x 4: above it may be anything
        if (i < 1) y[i].y = 0.f;
        if (i < 2) y[i].z = 0.f;
        if (i < 3) y[i].w = 0.f;
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float4 x = *reinterpret_cast<const float4*>(A21 + (r0 + r) * LDA + k);
      const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[r].x = fmaf(xs[i], y[i].x, acc[r].x);
        acc[r].y = fmaf(xs[i], y[i].y, acc[r].y);
        acc[r].z = fmaf(xs[i], y[i].z, acc[r].z);
        acc[r].w = fmaf(xs[i], y[i].w, acc[r].w);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    *reinterpret_cast<float4*>(Z + (r0 + r) * LDA + 4 * cg) = acc[r];
    acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  // T21 = -T22 Z, k up to the row group's last row; whole 4-steps below the
  // group's first row need no mask
  const int kd = r0 & ~3;
  for (int k = 0; k < kd; k += 4) step(T22, Z, k, -1.f);
  for (int k = kd; k < r0 + RT; k += 4) {
    float4 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = *reinterpret_cast<const float4*>(Z + (k + i) * LDA + 4 * cg);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float4 x = tri(T22, k, r0 + r);
      const float xs[4] = {-x.x, -x.y, -x.z, -x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[r].x = fmaf(xs[i], y[i].x, acc[r].x);
        acc[r].y = fmaf(xs[i], y[i].y, acc[r].y);
        acc[r].z = fmaf(xs[i], y[i].z, acc[r].z);
        acc[r].w = fmaf(xs[i], y[i].w, acc[r].w);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) *reinterpret_cast<float4*>(A21 + (r0 + r) * LDA + 4 * cg) = acc[r];
  __syncthreads();
}

TTT_DEVICE_INLINE void invert(float* A, int tid) {
  float x[16];
  if (tid < C) {
    const float* B = A + (tid >> 4) * 16 * (LDA + 1);
    const int j = tid & 15;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float acc = i == j ? 1.f : 0.f;
#pragma unroll
      for (int k = 0; k < i; ++k) acc = fmaf(-B[i * LDA + k], x[k], acc);
      x[i] = acc;
    }
  }
  __syncthreads();
  if (tid < C) {
    float* B = A + (tid >> 4) * 16 * (LDA + 1);
#pragma unroll
    for (int i = 0; i < 16; ++i) B[i * LDA + (tid & 15)] = x[i];
  }
  __syncthreads();
  join_blocks<16>(A, tid);
  join_blocks<32>(A, tid);
  join_blocks<64>(A, tid);
}

// ------------------------------------------------------------------ prep
struct PrepArgs {
  const __nv_bfloat16 *g, *beta;
  float* gend;             // [BH nch] exp(G_last)
  float* H;                // [BH nch][D / 64][16][D][4]: columns in groups of four
  __nv_bfloat16* M;        // [BH nch][2][D][D] hi, lo
  __nv_bfloat16* T;        // nullable: [BH nch][2][128][128] hi, lo
  int N, nch;
  DevStatus st;
};

template <int D>
struct PrepSmem {
  static constexpr uint32_t OP = D / 64 * ATOM;          // a [128][D] operand
  static constexpr uint32_t K = 0, V = OP, T = 2 * OP;   // T: A in float32, then operand tiles
  static constexpr uint32_t TBYTES = (C * LDA * 4 + 1023) / 1024 * 1024;
  static constexpr uint32_t GATES = T + TBYTES;
  static constexpr uint32_t BAR = GATES + sizeof(Gates);
  static constexpr uint32_t TOTAL = BAR + 64;
};

template <int D>
__global__ void __launch_bounds__(256)
    delta_prep_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                      const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapU,
                      PrepArgs a) {
  using SM = PrepSmem<D>;
  constexpr int DA = D / 64;
  constexpr uint32_t TM_A = 0, TM_U = 128, TM_W = 128 + D, TM_COLS = D == 64 ? 256 : 512;
  // Hc takes the place of A; Mc follows it (D = 64) or takes the last columns
  constexpr uint32_t TM_H = 0, TM_M = D == 64 ? 64 : 384;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* load = reinterpret_cast<uint64_t*>(smem + SM::BAR);
  uint64_t* mma = load + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma + 1);
  uint32_t* abort_flag = tmem_slot + 1;
  Gates& gates = *reinterpret_cast<Gates*>(smem + SM::GATES);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ch = blockIdx.x % a.nch;
  const size_t bh = blockIdx.x / a.nch, ci = blockIdx.x;
  const int t0 = ch * C, n = min(C, a.N - t0);

  if (tid == 0) {
    mbar_init(load, 1);
    mbar_init(mma, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sb = smem_u32(smem);
  Phase ph{Waiter{abort_flag, a.st, 1000}, mma, 0};
  const int q4 = warp & 3, hf = warp >> 2, row = q4 * 32 + lane;
  const uint32_t lanes = (uint32_t)(q4 * 32) << 16;

  if (tid == 0) {
    mbar_arrive_expect_tx(load, 2 * SM::OP);
    for (int i = 0; i < DA; ++i) {
      tma_load_3d(smem + SM::K + i * ATOM, &mapK, load, 64 * i, t0, (int)bh);
      tma_load_3d(smem + SM::V + i * ATOM, &mapV, load, 64 * i, t0, (int)bh);
    }
  }
  if (warp == 2) {
    const size_t tok = bh * a.N + t0;
    load_gates(gates, a.g ? a.g + tok : nullptr, a.beta + tok, n, lane);
    if (lane == 31) a.gend[ci] = gate_decay(gates, C - 1);
  }
  auto work = [&]() {
    if (!ph.wait(load, 0, 1)) return;
    const Op K{sb + SM::K, ATOM, false}, Kmn{sb + SM::K, ATOM, true}, Vmn{sb + SM::V, ATOM, true};
    if (tid == 0) {
      product(tmem + TM_A, K, K, 128, 128, D / 16, false);
      mma_commit(mma);
    }
    if (!ph.mma_done(2)) return;
    // A = beta_i Gam_ij k_i.k_j below the diagonal, float32
    float* A = reinterpret_cast<float*>(smem + SM::T);
    {
      const float bi = gates.beta[row], gh = gates.hi[row], gl = gates.lo[row];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int c0 = hf * 64 + b * 16;
        float x[16];
        const bool any = c0 <= q4 * 32 + 31;   // the warp's last row
        if (any) {
          tmem_ld16(tmem + lanes + TM_A + c0, x);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float d = (gh - gates.hi[c0 + j]) + (gl - gates.lo[c0 + j]);
            x[j] = c0 + j < row ? bi * x[j] * gate_exp(d) : 0.f;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          *reinterpret_cast<float4*>(A + row * LDA + c0 + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
      }
    }
    tc_fence_before();
    __syncthreads();
    invert(A, tid);
    // this thread's half row of T
    float t[64];
#pragma unroll
    for (int j = 0; j < 64; j += 4) {
      const int c0 = hf * 64 + j;
      float4 x = *reinterpret_cast<const float4*>(A + row * LDA + c0);
      t[j] = c0 <= row ? x.x : 0.f;
      t[j + 1] = c0 + 1 <= row ? x.y : 0.f;
      t[j + 2] = c0 + 2 <= row ? x.z : 0.f;
      t[j + 3] = c0 + 3 <= row ? x.w : 0.f;
    }
    if (a.T != nullptr) {
      uint4* d0 = reinterpret_cast<uint4*>(a.T + (ci * 2 * C + row) * C + hf * 64);
      uint4* d1 = reinterpret_cast<uint4*>(a.T + (ci * 2 * C + C + row) * C + hf * 64);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split2(t[8 * j + 2 * i], t[8 * j + 2 * i + 1], h[i], l[i]);
        d0[j] = make_uint4(h[0], h[1], h[2], h[3]);
        d1[j] = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
    __syncthreads();
    // operand tiles [hi atom 0, hi atom 1, lo atom 0, lo atom 1] of T with scaled columns
    const uint32_t tb = sb + SM::T;
    const Pair Tp{{tb, ATOM, false}, 2 * ATOM};
    auto put_t = [&](bool with_gam) {
#pragma unroll
      for (int j = 0; j < 64; j += 8) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = hf * 64 + j + i;
          x[i] = t[j + i] * (with_gam ? gates.beta[c] * gate_decay(gates, c) : gates.beta[c]);
        }
        store8_split(tb + hf * ATOM, tb + (2 + hf) * ATOM, row, j, x);
      }
    };
    put_t(false);
    ph.publish();
    if (tid == 0) {
      product(tmem + TM_U, Tp.hi, Vmn, 128, D, 8, false);
      product(tmem + TM_U, Tp.lo(), Vmn, 128, D, 8, true);
      mma_commit(mma);
    }
    if (!ph.mma_done(3)) return;
    put_t(true);
    ph.publish();
    if (tid == 0) {
      product(tmem + TM_W, Tp.hi, Kmn, 128, D, 8, false);
      product(tmem + TM_W, Tp.lo(), Kmn, 128, D, 8, true);
      mma_commit(mma);
    }
    if (!ph.mma_done(4)) return;
    // rho K as hi (in K's place) and lo (in V's)
    {
      const float rho = gate_exp((gates.hi[C - 1] - gates.hi[row]) + (gates.lo[C - 1] - gates.lo[row]));
#pragma unroll
      for (int j = 0; j < D / 2; j += 8) {
        const int c = hf * (D / 2) + j;
        const uint32_t at = (uint32_t)(c >> 6) * ATOM;
        float x[8];
        load8(sb + SM::K + at, row, c & 63, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= rho;
        store8_split(sb + SM::K + at, sb + SM::V + at, row, c & 63, x);
      }
    }
    // Ut and W as operand tiles, stored to the workspace and multiplied
    auto put = [&](uint32_t tm, int col0, int cols, uint32_t hi, uint32_t lo) {
      for (int j = 0; j < cols; j += 16) {
        float x[16];
        tmem_ld16(tmem + lanes + tm + col0 + j, x);
        const int c = col0 + j;
        const uint32_t at = (uint32_t)(c >> 6) * ATOM;
        store8_split(hi + at, lo + at, row, c & 63, x);
        store8_split(hi + at, lo + at, row, (c & 63) + 8, x + 8);
      }
    };
    const Pair Kr{{sb + SM::K, ATOM, true}, SM::OP};
    if constexpr (D == 64) {
      // [Ut hi, W hi, Ut lo, W lo]: a 128-column operand
      if (hf == 0) put(TM_U, 0, 64, tb, tb + 2 * ATOM);
      else put(TM_W, 0, 64, tb + ATOM, tb + 3 * ATOM);
      ph.publish();
      if (tid == 0) {
        const Pair B{{tb, ATOM, true}, 2 * ATOM};
        product3(tmem + TM_H, Kr, B, 64, 128, 8, false);
        mma_commit(mma);
        for (int h = 0; h < 2; ++h) {
          tma_store_3d(&mapU, smem + SM::T + 2 * h * ATOM, 0, 0, (int)(2 * ci + h));
          tma_store_3d(&mapW, smem + SM::T + (2 * h + 1) * ATOM, 0, 0, (int)(2 * ci + h));
        }
        bulk_commit();
      }
      if (!ph.mma_done(5)) return;
    } else {
      for (int m = 0; m < 2; ++m) {
        put(m ? TM_W : TM_U, hf * 64, 64, tb, tb + 2 * ATOM);
        ph.publish();
        if (tid == 0) {
          const Pair B{{tb, ATOM, true}, 2 * ATOM};
          product3(tmem + (m ? TM_M : TM_H), Kr, B, 128, 128, 8, false);
          mma_commit(mma);
          for (int h = 0; h < 2; ++h)
            for (int i = 0; i < 2; ++i)
              tma_store_3d(m ? &mapW : &mapU, smem + SM::T + (2 * h + i) * ATOM, 64 * i, 0, (int)(2 * ci + h));
          bulk_commit();
          bulk_wait_read();
        }
        if (!ph.mma_done(5 + m)) return;
      }
    }
    // Hc in float32, Mc as hi and lo; for D = 64 the 64 rows sit in the first
    // 16 lanes of each quadrant
    const int r = D == 64 ? q4 * 16 + lane : row;
    const bool own = D == 128 || lane < 16;
    const int cols = D / 2;   // of each, this half
    for (int j = 0; j < cols; j += 16) {
      const int c = hf * cols + j;
      float h[16], m[16];
      tmem_ld16(tmem + lanes + TM_H + c, h);
      tmem_ld16(tmem + lanes + TM_M + c, m);
      if (!own) continue;
      store_h16(a.H + ci * D * D, D, r, c, h);
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) split2(-m[2 * i], -m[2 * i + 1], hi[i], lo[i]);
      uint4* d0 = reinterpret_cast<uint4*>(a.M + (ci * 2 * D + r) * D + c);
      uint4* d1 = reinterpret_cast<uint4*>(a.M + (ci * 2 * D + D + r) * D + c);
      d0[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      d0[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
      d1[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      d1[1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
    }
    if (tid == 0) bulk_wait_all();
  };
  work();
  if (tid == 0 && ph.W.aborted()) {   // nothing in flight may outlive the CTA
    ph.W.drain(load, 0);
    bulk_wait_all();
    mma_commit(mma);
    ph.W.drain(mma, 0);
    ph.W.drain(mma, 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
}

// ------------------------------------------------------------------ chain
// X <- e_c X + H_c + Mc X over the chunks of one head and 64 value columns
// (backward: Mc^T, from the last chunk); X in float32 registers (16 values a
// thread), its hi + lo copy in shared memory as the operand of the next
// chunk's product and in the workspace as the chunk's border state.
struct ChainArgs {
  const float* gend;
  DeltaChain dir[2];       // forward, backward
  int nch, BH, first;      // the first CTAs take dir[first]
  DevStatus st;
};

template <int D>
struct ChainSmem {
  static constexpr int STAGES = D == 64 ? 4 : 2;
  static constexpr uint32_t SA = D * 128;                 // bytes of a [D][64] atom
  static constexpr uint32_t STAGE = 2 * (D / 64) * SA;    // Mc hi, lo
  static constexpr uint32_t X = STAGES * STAGE;           // [hi, lo]
  static constexpr uint32_t BAR = X + 2 * SA;
  static constexpr uint32_t TOTAL = BAR + 128;
};

template <int D>
__global__ void __launch_bounds__(512, 1)
    delta_chain_kernel(const __grid_constant__ CUtensorMap mapM, ChainArgs a) {
  using SM = ChainSmem<D>;
  constexpr int DA = D / 64, STAGES = SM::STAGES;
  constexpr uint32_t TM_COLS = 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::BAR);
  uint64_t* mma = full + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma + 1);
  uint32_t* abort_flag = tmem_slot + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slice = blockIdx.x % DA;
  const bool rev = a.first + blockIdx.x / (DA * a.BH) == 1;
  const DeltaChain& dir = a.dir[rev ? 1 : 0];
  const size_t bh = blockIdx.x / DA % a.BH, c0 = bh * a.nch;
  auto chunk = [&](int i) { return c0 + (rev ? a.nch - 1 - i : i); };

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(&full[s], 1);
    mbar_init(mma, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot, sb = smem_u32(smem);
  Phase ph{Waiter{abort_flag, a.st, 1100}, mma, 0};
  const int q4 = warp & 3, cg = warp >> 2;    // 16 columns of the slice
  const int r = D == 64 ? q4 * 16 + lane : q4 * 32 + lane;
  const bool own = D == 128 || lane < 16;
  const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
  const int col = slice * 64 + cg * 16;
  int issued = 0;
  auto fetch = [&]() {   // by thread 0: the next chunk's Mc
    if (issued >= a.nch) return;
    const int s = issued % STAGES;
    mbar_arrive_expect_tx(&full[s], SM::STAGE);
    for (int h = 0; h < 2; ++h)
      for (int i = 0; i < DA; ++i)
        tma_load_3d(smem + s * SM::STAGE + (h * DA + i) * SM::SA, &mapM, &full[s], 64 * i, 0,
                    (int)(2 * chunk(issued) + h));
    ++issued;
  };
  if (tid == 0)
    for (int s = 0; s < STAGES; ++s) fetch();
  float x[16];
#pragma unroll
  for (int j = 0; j < 16; j += 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (own && dir.S_in != nullptr) v = *reinterpret_cast<const float4*>(dir.S_in + (bh * D + r) * D + col + j);
    x[j] = v.x; x[j + 1] = v.y; x[j + 2] = v.z; x[j + 3] = v.w;
  }
  // the operand copy, and the border state of chunk c
  auto put_x = [&](int c) {
    if (!own) return;
    uint32_t h[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) split2(x[2 * i], x[2 * i + 1], h[i], l[i]);
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const uint32_t o = sw128_offset(r, cg * 16 + 2 * i);
      st_shared_v4(sb + SM::X + o, h[i], h[i + 1], h[i + 2], h[i + 3]);
      st_shared_v4(sb + SM::X + SM::SA + o, l[i], l[i + 1], l[i + 2], l[i + 3]);
    }
    uint4* g0 = reinterpret_cast<uint4*>(dir.X + (chunk(c) * 2 * D + r) * D + col);
    uint4* g1 = reinterpret_cast<uint4*>(dir.X + (chunk(c) * 2 * D + D + r) * D + col);
    g0[0] = make_uint4(h[0], h[1], h[2], h[3]);
    g0[1] = make_uint4(h[4], h[5], h[6], h[7]);
    g1[0] = make_uint4(l[0], l[1], l[2], l[3]);
    g1[1] = make_uint4(l[4], l[5], l[6], l[7]);
  };
  auto load_h = [&](int c, float4 (&h)[4]) {
    const float* p = dir.H + chunk(c) * D * D + (size_t)slice * 64 * D + ((size_t)cg * 4 * D + r) * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = own ? *reinterpret_cast<const float4*>(p + (size_t)j * D * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 h[4];
  float e = 0.f;
  load_h(0, h);
  e = a.gend[chunk(0)];
  for (int c = 0; c < a.nch; ++c) {
    put_x(c);
    ph.publish();
    if (tid == 0) {
      const int s = c % STAGES;
      if (ph.W.wait(&full[s], (c / STAGES) & 1, 1)) {
        const Pair A{{sb + s * SM::STAGE, SM::SA, rev}, DA * SM::SA};
        const Pair B{{sb + SM::X, SM::SA, true}, SM::SA};
        product3(tmem, A, B, D, 64, D / 16, false);
        mma_commit(mma);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[4 * j] = fmaf(e, x[4 * j], h[j].x);
      x[4 * j + 1] = fmaf(e, x[4 * j + 1], h[j].y);
      x[4 * j + 2] = fmaf(e, x[4 * j + 2], h[j].z);
      x[4 * j + 3] = fmaf(e, x[4 * j + 3], h[j].w);
    }
    if (c + 1 < a.nch) {
      load_h(c + 1, h);
      e = a.gend[chunk(c + 1)];
    }
    if (!ph.mma_done(2)) break;
    float d[16];
    tmem_ld16(tmem + lanes + cg * 16, d);
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] += d[j];
    if (tid == 0) fetch();   // the stage that this chunk's product has read
  }
  if (!ph.W.aborted() && own && dir.S_out != nullptr) {
    float* dst = dir.S_out + (bh * D + r) * D + col;
#pragma unroll
    for (int j = 0; j < 16; j += 4)
      *reinterpret_cast<float4*>(dst + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
  }
  if (tid == 0 && ph.W.aborted()) {
    for (int i = max(0, issued - STAGES); i < issued; ++i) ph.W.drain(&full[i % STAGES], (i / STAGES) & 1);
    mma_commit(mma);
    ph.W.drain(mma, 0);
    ph.W.drain(mma, 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
}

// ------------------------------------------------------------------ outputs
// O = scale (gam Q S0 + (Gam . Q K^T) (Ut - W S0)) of one chunk and 64 value columns.
struct OutArgs {
  const __nv_bfloat16 *g, *beta;
  void* out;
  int N, nch, out_bf16;
  float scale;
  DevStatus st;
};

template <int D>
struct OutSmem {
  static constexpr int DA = D / 64;
  static constexpr uint32_t OP = DA * ATOM, SA = D * 128;
  static constexpr uint32_t Q = 0, K = OP, W = 2 * OP;             // W hi, lo
  static constexpr uint32_t P = 0;                                  // 4 atoms, over Q, K (and W for D = 64)
  static constexpr uint32_t U = 4 * OP;                             // Ut, then U: hi, lo
  static constexpr uint32_t S = U + 2 * ATOM;                       // S0 hi, lo
  static constexpr uint32_t GATES = S + 2 * SA;
  static constexpr uint32_t BAR = GATES + sizeof(Gates);
  static constexpr uint32_t TOTAL = BAR + 64;
};

template <int D>
__global__ void __launch_bounds__(256)
    delta_out_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                     const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapU,
                     const __grid_constant__ CUtensorMap mapS, OutArgs a) {
  using SM = OutSmem<D>;
  constexpr int DA = D / 64;
  constexpr uint32_t TM_P = 0, TM_W = 128, TM_Q = 192, TM_COLS = 256;   // P U takes W S0's place
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* load = reinterpret_cast<uint64_t*>(smem + SM::BAR);
  uint64_t* mma = load + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma + 1);
  uint32_t* abort_flag = tmem_slot + 1;
  Gates& gates = *reinterpret_cast<Gates*>(smem + SM::GATES);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slice = blockIdx.x % DA;
  const size_t ci = blockIdx.x / DA, bh = ci / a.nch;
  const int t0 = (int)(ci % a.nch) * C, n = min(C, a.N - t0);

  if (tid == 0) {
    mbar_init(load, 1);
    mbar_init(mma, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot, sb = smem_u32(smem);
  Phase ph{Waiter{abort_flag, a.st, 1200}, mma, 0};
  const int q4 = warp & 3, hf = warp >> 2, row = q4 * 32 + lane;
  const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
  if (tid == 0) {
    mbar_arrive_expect_tx(load, 4 * SM::OP + 2 * ATOM + 2 * SM::SA);
    for (int i = 0; i < DA; ++i) {
      tma_load_3d(smem + SM::Q + i * ATOM, &mapQ, load, 64 * i, t0, (int)bh);
      tma_load_3d(smem + SM::K + i * ATOM, &mapK, load, 64 * i, t0, (int)bh);
      for (int h = 0; h < 2; ++h)
        tma_load_3d(smem + SM::W + (h * DA + i) * ATOM, &mapW, load, 64 * i, 0, (int)(2 * ci + h));
    }
    for (int h = 0; h < 2; ++h) {
      tma_load_3d(smem + SM::U + h * ATOM, &mapU, load, 64 * slice, 0, (int)(2 * ci + h));
      tma_load_3d(smem + SM::S + h * SM::SA, &mapS, load, 64 * slice, 0, (int)(2 * ci + h));
    }
  }
  if (warp == 2) {
    const size_t tok = bh * a.N + t0;
    load_gates(gates, a.g ? a.g + tok : nullptr, a.beta + tok, n, lane);
  }
  auto work = [&]() {
    if (!ph.wait(load, 0, 1)) return;
    const Op Q{sb + SM::Q, ATOM, false}, K{sb + SM::K, ATOM, false};
    const Pair Wp{{sb + SM::W, ATOM, false}, SM::OP}, S{{sb + SM::S, SM::SA, true}, SM::SA};
    if (tid == 0) {
      product(tmem + TM_P, Q, K, 128, 128, D / 16, false);
      product3(tmem + TM_W, Wp, S, 128, 64, D / 16, false);
      product(tmem + TM_Q, Q, S.hi, 128, 64, D / 16, false);
      product(tmem + TM_Q, Q, S.lo(), 128, 64, D / 16, true);
      mma_commit(mma);
    }
    if (!ph.mma_done(2)) return;
    // U = Ut - W S0, in place; this half's 32 columns
    {
      float w[32];
      tmem_ld32(tmem + lanes + TM_W + hf * 32, w);
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        float u[8];
        load8_split(sb + SM::U, sb + SM::U + ATOM, row, hf * 32 + j, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] -= w[j + i];
        store8_split(sb + SM::U, sb + SM::U + ATOM, row, hf * 32 + j, u);
      }
    }
    // P = Gam . Q K^T on and below the diagonal: [hi 0, hi 1, lo 0, lo 1]
    {
      const float gh = gates.hi[row], gl = gates.lo[row];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int c0 = hf * 64 + b * 16;
        float x[16];
        if (c0 <= q4 * 32 + 31) {
          tmem_ld16(tmem + lanes + TM_P + c0, x);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float d = (gh - gates.hi[c0 + j]) + (gl - gates.lo[c0 + j]);
            x[j] = c0 + j <= row ? x[j] * gate_exp(d) : 0.f;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = 0.f;
        }
        store8_split(sb + SM::P + hf * ATOM, sb + SM::P + (2 + hf) * ATOM, row, b * 16, x);
        store8_split(sb + SM::P + hf * ATOM, sb + SM::P + (2 + hf) * ATOM, row, b * 16 + 8, x + 8);
      }
    }
    ph.publish();
    if (tid == 0) {
      const Pair P{{sb + SM::P, ATOM, false}, 2 * ATOM}, U{{sb + SM::U, ATOM, true}, ATOM};
      product3(tmem + TM_W, P, U, 128, 64, 8, false);
      mma_commit(mma);
    }
    if (!ph.mma_done(3)) return;
    float o[32], qs[32];
    tmem_ld32(tmem + lanes + TM_W + hf * 32, o);
    tmem_ld32(tmem + lanes + TM_Q + hf * 32, qs);
    if (row < n) {
      const float gam = a.scale * gate_decay(gates, row);
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = fmaf(gam, qs[j], a.scale * o[j]);
      const size_t at = (bh * a.N + t0 + row) * D + slice * 64 + hf * 32;
      if (a.out_bf16) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          dst[j] = make_uint4(pack_bf16x2(o[8 * j], o[8 * j + 1]), pack_bf16x2(o[8 * j + 2], o[8 * j + 3]),
                              pack_bf16x2(o[8 * j + 4], o[8 * j + 5]), pack_bf16x2(o[8 * j + 6], o[8 * j + 7]));
      } else {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
#pragma unroll
        for (int j = 0; j < 8; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
      }
    }
  };
  work();
  if (tid == 0 && ph.W.aborted()) {
    ph.W.drain(load, 0);
    mma_commit(mma);
    ph.W.drain(mma, 0);
    ph.W.drain(mma, 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
}

template <int D>
int prep_launch(const DeltaLaunch& p, const DeltaPrepOut& o, cudaStream_t stream) {
  const int BH = p.B * p.H, nch = (p.N + C - 1) / C;
  const uint64_t nc = (uint64_t)BH * nch, rs = D * 2;
  CUtensorMap mk, mv, mw, mu;
  if (make_tmap_bf16_3d(&mk, p.k, D, p.N, BH, rs, p.N * rs, 64, C) ||
      make_tmap_bf16_3d(&mv, p.v, D, p.N, BH, rs, p.N * rs, 64, C) ||
      make_tmap_bf16_3d(&mw, o.W, D, C, 2 * nc, rs, C * rs, 64, C) ||
      make_tmap_bf16_3d(&mu, o.U, D, C, 2 * nc, rs, C * rs, 64, C))
    return -1;
  static std::atomic<uint64_t> attr{0};
  if (allow_dynamic_smem(delta_prep_kernel<D>, (int)PrepSmem<D>::TOTAL, attr)) return -1;
  const PrepArgs a{(const __nv_bfloat16*)p.g, (const __nv_bfloat16*)p.beta, o.gend, o.H, o.M, o.T, p.N, nch, p.st};
  prof_before(K_DELTA_PREP, stream);
  delta_prep_kernel<D><<<(unsigned)nc, 256, PrepSmem<D>::TOTAL, stream>>>(mk, mv, mw, mu, a);
  prof_after(K_DELTA_PREP, stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <int D>
int chain_launch(const DeltaLaunch& p, const float* gend, const __nv_bfloat16* M, const DeltaChain* fwd,
                 const DeltaChain* rev, cudaStream_t stream) {
  const int BH = p.B * p.H, nch = (p.N + C - 1) / C;
  const uint64_t nc = (uint64_t)BH * nch, rs = D * 2;
  CUtensorMap mm;
  if (make_tmap_bf16_3d(&mm, M, D, D, 2 * nc, rs, D * rs, 64, D)) return -1;
  static std::atomic<uint64_t> attr{0};
  if (allow_dynamic_smem(delta_chain_kernel<D>, (int)ChainSmem<D>::TOTAL, attr)) return -1;
  ChainArgs a{gend, {}, nch, BH, fwd ? 0 : 1, p.st};
  if (fwd) a.dir[0] = *fwd;
  if (rev) a.dir[1] = *rev;
  const unsigned dirs = (fwd ? 1 : 0) + (rev ? 1 : 0);
  prof_before(K_DELTA_CHAIN, stream);
  delta_chain_kernel<D><<<dirs * (unsigned)(BH * (D / 64)), 512, ChainSmem<D>::TOTAL, stream>>>(mm, a);
  prof_after(K_DELTA_CHAIN, stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <int D>
int fwd_launch(const DeltaLaunch& p, cudaStream_t stream) {
  const int BH = p.B * p.H, nch = (p.N + C - 1) / C;
  const DeltaUmmaWorkspace w = delta_umma_layout(BH, p.N, D);
  const uint64_t nc = (uint64_t)BH * nch, rs = D * 2;
  auto bf = [&](size_t at) { return reinterpret_cast<__nv_bfloat16*>(p.ws + at); };
  auto f32 = [&](size_t at) { return reinterpret_cast<float*>(p.ws + at); };
  const DeltaPrepOut o{f32(w.gend), f32(w.H), bf(w.W), bf(w.U), bf(w.M), nullptr};
  const DeltaChain chain{o.H, p.S, p.S, bf(w.X)};
  if (prep_launch<D>(p, o, stream) || chain_launch<D>(p, o.gend, o.M, &chain, nullptr, stream)) return -1;
  CUtensorMap mq, mk, mw, mu, ms;
  if (make_tmap_bf16_3d(&mq, p.q, D, p.N, BH, rs, p.N * rs, 64, C) ||
      make_tmap_bf16_3d(&mk, p.k, D, p.N, BH, rs, p.N * rs, 64, C) ||
      make_tmap_bf16_3d(&mw, o.W, D, C, 2 * nc, rs, C * rs, 64, C) ||
      make_tmap_bf16_3d(&mu, o.U, D, C, 2 * nc, rs, C * rs, 64, C) ||
      make_tmap_bf16_3d(&ms, chain.X, D, D, 2 * nc, rs, D * rs, 64, D))
    return -1;
  static std::atomic<uint64_t> attr{0};
  if (allow_dynamic_smem(delta_out_kernel<D>, (int)OutSmem<D>::TOTAL, attr)) return -1;
  const OutArgs a{(const __nv_bfloat16*)p.g, (const __nv_bfloat16*)p.beta, p.out, p.N, nch, p.out_bf16, p.scale, p.st};
  prof_before(K_DELTA_OUT, stream);
  delta_out_kernel<D><<<(unsigned)(nc * (D / 64)), 256, OutSmem<D>::TOTAL, stream>>>(mq, mk, mw, mu, ms, a);
  prof_after(K_DELTA_OUT, stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

bool delta_uses_umma(int bf16, int dk, int dv) { return bf16 && dk == dv && (dk == 64 || dk == 128); }

DeltaUmmaWorkspace delta_umma_layout(int BH, int N, int D) {
  DeltaUmmaWorkspace w{};
  const size_t nc = (size_t)BH * ((N + C - 1) / C);
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  w.gend = take(nc * 4);
  w.W = take(nc * 2 * C * D * 2);
  w.U = take(nc * 2 * C * D * 2);
  w.M = take(nc * 2 * D * D * 2);
  w.H = take(nc * D * D * 4);
  w.X = take(nc * 2 * D * D * 2);
  w.total = at;
  return w;
}

int launch_delta_prep(const DeltaLaunch& p, const DeltaPrepOut& o, cudaStream_t stream) {
  return p.dk == 64 ? prep_launch<64>(p, o, stream) : prep_launch<128>(p, o, stream);
}
int launch_delta_chain(const DeltaLaunch& p, const float* gend, const __nv_bfloat16* M, const DeltaChain* fwd,
                       const DeltaChain* rev, cudaStream_t stream) {
  return p.dk == 64 ? chain_launch<64>(p, gend, M, fwd, rev, stream)
                    : chain_launch<128>(p, gend, M, fwd, rev, stream);
}
int launch_delta_umma(const DeltaLaunch& p, cudaStream_t stream) {
  return p.dk == 64 ? fwd_launch<64>(p, stream) : fwd_launch<128>(p, stream);
}

}  // namespace ttt
