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
//   prep_cta   K, V -> W, Ut, Mc, Hc
//   chain_cta  Mc, Hc -> every chunk's start state, end state
//   out_cta    Q, K, W, Ut, start states -> O
#include <algorithm>

#include "delta_umma.cuh"

namespace ttt {

using namespace dl;

namespace {

constexpr int THREADS = 512;   // of every CTA: four column groups of 128 rows

// ------------------------------------------------------------------ inverse
// (I + A)^-1 in place, A strictly lower triangular [128][128] float32 in
// shared memory (rows LDA floats apart): 16 x 16 diagonal blocks by
// substitution, one column a thread, then blocks of 16, 32 and 64 joined two
// by two, T21 = -T22 (A21 T11).  Every factor is itself an inverse, so the
// intermediate values stay of the size of the result (the powers of A of a
// Neumann product do not).  A21 T11 waits in the unused block above the
// diagonal, so what is above the diagonal may be anything, before and after.
//
// The joins are warp-level tensor products, a tile of 16 x 16 a warp, with
// every float32 value as a sum of two tf32 ones (three products).  hi is rounded
// to nearest, so lo is at most 2^-11 of the value and of either sign; lo's own
// lowest bits, which the product does not read, are below 2^-21 of it, and lo lo,
// which is left out, below 2^-22: a product of two values is off by 2^-20 + 2^-22
// at most (1.2e-6; 4.6e-7 the largest of four million random ones, and no bias.
// A hi cut off instead of rounded: 1.6e-6, all towards zero).  With
// FFMA, what the register tiles read from shared memory bound them: 4 x 4 a
// thread took 8100 cycles for blocks of 64, two CTAs an SM.  (The blocks are
// too small for tcgen05: its operands would have to be split into planes and
// stored first.)
constexpr int LDA = 132;

struct Tf32 {
  uint32_t hi, lo;
  TTT_DEVICE_INLINE explicit Tf32(float x) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;   // NaN and infinity leave NaN in lo
    lo = __float_as_uint(x - __uint_as_float(hi));
  }
};
TTT_DEVICE_INLINE void mma_16x8x8(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// acc = X Y of a 16 x 16 tile: X at its first row, Y at its first column, k in
// [k0, k1).  xd, yd: the tile's first row or column where X or Y is lower
// triangular (what lies above the diagonal counts as zero), -1 where not.  The
// three products have sums of their own, so that a step waits for one of them.
// Lane (g, t) holds columns 2t and 2t + 1 of X's rows tile_row(g) and 8 below,
// and those rows of Y: with LDA = 4 (mod 32) no two lanes meet in a bank.
TTT_DEVICE_INLINE int tile_row(int g) { return 2 * (g & 3) + (g >> 2); }
TTT_DEVICE_INLINE void tile_product(const float* X, const float* Y, int k0, int k1, int xd, int yd, int lane,
                                    float (&acc)[2][4]) {
  const int g = lane >> 2, t = lane & 3, gr = tile_row(g);
  float s1[2][4], s2[2][4];
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = s1[n][i] = s2[n][i] = 0.f;
  auto step = [&](int k, bool diag) {
    uint32_t ah[4], al[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = gr + i * 8, c = k + 2 * t;
      const float2 x = *reinterpret_cast<const float2*>(X + r * LDA + c);
      const Tf32 v(diag && xd >= 0 && c > xd + r ? 0.f : x.x), w(diag && xd >= 0 && c + 1 > xd + r ? 0.f : x.y);
      ah[i] = v.hi;
      al[i] = v.lo;
      ah[i + 2] = w.hi;
      al[i + 2] = w.lo;
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      uint32_t bh[2], bl[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = k + 2 * t + i, c = 8 * n + g;
        const float y = Y[r * LDA + c];
        const Tf32 v(diag && yd >= 0 && r < yd + c ? 0.f : y);
        bh[i] = v.hi;
        bl[i] = v.lo;
      }
      mma_16x8x8(s1[n], al, bh);
      mma_16x8x8(s2[n], ah, bl);
      mma_16x8x8(acc[n], ah, bh);
    }
  };
  // the 16 columns (rows) on the diagonal, then the others: at most 48
  const int d0 = xd >= 0 ? xd : yd;
  step(d0, true);
  step(d0 + 8, true);
  const int e0 = xd >= 0 ? k0 : k0 + 16, e1 = xd >= 0 ? k1 - 16 : k1;
#pragma unroll 2
  for (int k = e0; k < e1; k += 8) step(k, false);
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] += s1[n][i] + s2[n][i];
}
TTT_DEVICE_INLINE void store_tile(float* C_, float sign, int lane, const float (&acc)[2][4]) {
  const int g = tile_row(lane >> 2), t = lane & 3;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    *reinterpret_cast<float2*>(C_ + g * LDA + 8 * n + 2 * t) = make_float2(sign * acc[n][0], sign * acc[n][1]);
    *reinterpret_cast<float2*>(C_ + (g + 8) * LDA + 8 * n + 2 * t) = make_float2(sign * acc[n][2], sign * acc[n][3]);
  }
}

template <int S>
TTT_DEVICE_INLINE void join_blocks(float* A, int warp, int lane) {
  constexpr int TILES = S / 16, WARPS = TILES * TILES * (C / (2 * S));
  static_assert(WARPS <= THREADS / 32, "a tile a warp");
  // (the columns turn from row to row, and rows from pair to pair, as a tile's
  // depth goes with them and an SM's quarter runs every fourth warp)
  const int p = warp / (TILES * TILES), r0 = (warp / TILES + p) % TILES * 16;
  const int n0 = (warp + warp / 4) % TILES * 16;
  float* T11 = A + p * 2 * S * (LDA + 1);
  float* A21 = T11 + S * LDA;
  float* T22 = A21 + S;
  float* Z = T11 + S;
  float acc[2][4];
  if (warp < WARPS) {   // Z = A21 T11: nothing above T11's columns
    tile_product(A21 + r0 * LDA, T11 + n0, n0, S, -1, n0, lane, acc);
    store_tile(Z + r0 * LDA + n0, 1.f, lane, acc);
  }
  __syncthreads();
  if (warp < WARPS) {   // -T22 Z: nothing right of T22's rows
    tile_product(T22 + r0 * LDA, Z + n0, 0, r0 + 16, r0, -1, lane, acc);
    store_tile(A21 + r0 * LDA + n0, -1.f, lane, acc);
  }
  __syncthreads();
}

TTT_DEVICE_INLINE void invert(float* A, int warp, int lane) {
  const int tid = warp * 32 + lane;
  float x[16];
  if (tid < C) {
    const float* B = A + (tid >> 4) * 16 * (LDA + 1);
    const int j = tid & 15;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float b[16], acc = i == j ? 1.f : 0.f;
#pragma unroll
      for (int k = 0; k < i; k += 4) *reinterpret_cast<float4*>(b + k) = *reinterpret_cast<const float4*>(B + i * LDA + k);
#pragma unroll
      for (int k = 0; k < i; ++k) acc = fmaf(-b[k], x[k], acc);
      x[i] = acc;
    }
    __syncwarp();   // a block's 16 threads are in one warp
    float* W = A + (tid >> 4) * 16 * (LDA + 1);
#pragma unroll
    for (int i = 0; i < 16; ++i) W[i * LDA + (tid & 15)] = x[i];
  }
  __syncthreads();
  join_blocks<16>(A, warp, lane);
  join_blocks<32>(A, warp, lane);
  join_blocks<64>(A, warp, lane);
}

// ------------------------------------------------------------------ prep
// A chunk takes about 22 us with two CTAs an SM (heads of 64), a third of it
// the inverse, the rest the latency of two rounds of products, splits and
// stores: 2048 chunks 166 us, and no unit is more than half busy.
struct PrepArgs {
  const __nv_bfloat16 *g, *beta;
  float* gend;             // [BH nch] exp(G_last)
  float* H;                // [BH nch] float32 tiles [D][D]
  float* U;                // [BH nch] float32 tiles [128][D]: Ut
  __nv_bfloat16* W;        // [BH nch][2][128][D] hi, lo
  __nv_bfloat16* M;        // [BH nch][2][D][D] hi, lo
  __nv_bfloat16* T;        // nullable: [BH nch][2][128][128] hi, lo
  int N;
  Slab slab;
  DevStatus st;
};

template <int D>
struct PrepSmem {
  static constexpr uint32_t OP = D / 64 * ATOM;          // a [128][D] operand
  static constexpr uint32_t K = 0, V = OP, T = 2 * OP;   // T: A in float32, then gam K
  static constexpr uint32_t TBYTES = (C * LDA * 4 + 1023) / 1024 * 1024;
  static constexpr uint32_t GATES = T + TBYTES;
  static constexpr uint32_t COL = GATES + sizeof(Gates);   // gam, rho
  static constexpr uint32_t BAR = COL + 2 * C * 4;
  static constexpr uint32_t TOTAL = BAR + 80;
};

template <int D>
TTT_DEVICE_INLINE void prep_cta(uint8_t* smem, const CUtensorMap& mapK, const CUtensorMap& mapV,
                                const PrepArgs& a, unsigned block) {
  using SM = PrepSmem<D>;
  constexpr int DA = D / 64;
  constexpr uint32_t TM_A = 0, TM_T = 0, TM_U = 128, TM_W = 128 + D, TM_COLS = D == 64 ? 256 : 512;
  // Hc takes the place of T; Mc follows it (D = 64) or takes the last columns
  constexpr uint32_t TM_H = 0, TM_M = D == 64 ? 64 : 384;
  Bars& bars = *reinterpret_cast<Bars*>(smem + SM::BAR);
  Gates& gates = *reinterpret_cast<Gates*>(smem + SM::GATES);
  float* gams = reinterpret_cast<float*>(smem + SM::COL);
  float* rhos = gams + C;
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const ChunkId id(block, 1, a.slab, a.N);
  const size_t ci = id.ci;
  const uint32_t sb = smem_u32(smem);
  const uint32_t tmem = cta_begin(bars, TM_COLS, warp, [&]() {
    mbar_arrive_expect_tx(&bars.load[0], 2 * SM::OP);
    for (int i = 0; i < DA; ++i) {
      tma_load_3d(smem + SM::K + i * ATOM, &mapK, &bars.load[0], 64 * i, id.t0, (int)id.bh);
      tma_load_3d(smem + SM::V + i * ATOM, &mapV, &bars.load[0], 64 * i, id.t0, (int)id.bh);
    }
  });
  Phase ph{Waiter{&bars.abort, a.st, 1000}, &bars.mma, 0};
  const int q4 = warp & 3, cg = warp >> 2, row = q4 * 32 + lane;
  const uint32_t lanes = (uint32_t)(q4 * 32) << 16;

  if (cg == 1) {
    load_gates(gates, a.g ? a.g + id.tok : nullptr, a.beta + id.tok, id.n, row, gams[row], rhos[row]);
    if (row == C - 1) a.gend[ci] = gams[row];
  }
  auto work = [&]() {
    const Op K{sb + SM::K, ATOM, false};
    if (warp == 0 && ph.W.wait_warp(&bars.load[0], 0, 1) && elect_one()) {
      products<D / 16>(Prod(tmem + TM_A, K, K, 128, 128, false));
      mma_commit(&bars.mma);
    }
    if (!ph.mma_done(2)) return;
    // A = beta_i Gam_ij k_i.k_j below the diagonal, float32; what lies in
    // blocks of 16 above it is read by nobody
    float* A = reinterpret_cast<float*>(smem + SM::T);
    {
      const float bi = gates.beta[row];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int c0 = cg * 32 + b * 16;
        if (c0 > q4 * 32 + 31) continue;
        float x[16];
        tmem_ld16(tmem + lanes + TM_A + c0, x);
        weigh16<false>(gates, q4 * 32, row, c0, bi, x);
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          *reinterpret_cast<float4*>(A + row * LDA + c0 + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
      }
    }
    tc_fence_before();
    __syncthreads();
    invert(A, warp, lane);
    // this thread's 32 columns of a row of T
    const bool some = cg <= q4;   // the others lie above the diagonal
    float t[32];
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const int c0 = cg * 32 + j;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (some) x = *reinterpret_cast<const float4*>(A + row * LDA + c0);
      t[j] = c0 <= row ? x.x : 0.f;
      t[j + 1] = c0 + 1 <= row ? x.y : 0.f;
      t[j + 2] = c0 + 2 <= row ? x.z : 0.f;
      t[j + 3] = c0 + 3 <= row ? x.w : 0.f;
    }
    if (a.T != nullptr) {
      __nv_bfloat16* d = a.T + (ci * 2 * C + row) * C + cg * 32;
#pragma unroll
      for (int j = 0; j < 32; j += 16) store16_pair(d + j, d + C * C + j, t + j);
    }
    // T diag(beta), hi and lo, becomes an operand in TMEM in A's place; hi + lo
    // is off by 2^-18 at most, and what T adds to the diagonal is a part of U
    // and W only.  S comes out to 5.1e-7; with a third plane to 1.2e-7, but the call
    // takes 2 % longer (64 heads of 64, 32K tokens: 1747 us against 1711), and where
    // the last chunk is short, M and X leave more (8e-7 in the place of 9e-7)
    {
      uint32_t h[16], l[16];
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 b = *reinterpret_cast<const float4*>(gates.beta + cg * 32 + j);
        split2(t[j] * b.x, t[j + 1] * b.y, h[j / 2], l[j / 2]);
        split2(t[j + 2] * b.z, t[j + 3] * b.w, h[j / 2 + 1], l[j / 2 + 1]);
      }
      tmem_st16_issue(tmem + lanes + TM_T + cg * 16, h);
      tmem_st16_issue(tmem + lanes + TM_T + 64 + cg * 16, l);
    }
    __syncthreads();   // all of A has been read
    // gam K, hi and lo, in A's place
    const uint32_t tb = sb + SM::T;
    {
      const float gam = gams[row];
      constexpr int cols = D / 4;
#pragma unroll
      for (int j = 0; j < cols; j += 8) {
        const int c = cg * cols + j;
        const uint32_t at = (uint32_t)(c >> 6) * ATOM;
        float x[8];
        load8(sb + SM::K + at, row, c & 63, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= gam;
        store8_split(tb + at, tb + SM::OP + at, row, c & 63, x);
      }
    }
    tmem_wait_st();
    ph.publish();
    if (warp == 0 && elect_one()) {
      // V and the hi plane of gam K lie side by side, as Ut and W do: one operand
      const Op VK{sb + SM::V, ATOM, true}, gKlo{tb + SM::OP, ATOM, true};
      const uint32_t hi = tmem + TM_T, lo = hi + 64;
      products<8>(Prod(tmem + TM_U, lo, VK, 2 * D, false));
      products<8>(Prod(tmem + TM_W, hi, gKlo, D, true));
      products<8>(Prod(tmem + TM_U, hi, VK, 2 * D, true));
      mma_commit(&bars.mma);
    }
    // Ut goes out in float32, W as hi + lo; rho Ut (three planes: Hc is the
    // state's own term, and hi + lo alone would leave 4e-6 of it) and rho W
    // (two: Mc multiplies what the decay left of the last state) are operands
    // in the place of V and T, against the exact K
    const float rho = rhos[row];
    // (planes `second` bytes apart)
    auto out_u = [&](int c, uint32_t second) {   // 16 columns
      float x[16];
      tmem_ld16(tmem + lanes + TM_U + c, x);
      store_tile16(a.U + ci * C * D, C, row, c, x);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= rho;
      const uint32_t at = sb + SM::V + (uint32_t)(c >> 6) * ATOM;
#pragma unroll
      for (int i = 0; i < 16; i += 8)
        store8_split3(at, at + second, at + 2 * second, row, (c & 63) + i, x + i);
    };
    auto out_w = [&](int c, uint32_t hi, uint32_t second) {
      float x[16];
      tmem_ld16(tmem + lanes + TM_W + c, x);
      __nv_bfloat16* d = a.W + (ci * 2 * C + row) * D + c;
      store16_pair(d, d + C * D, x);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= rho;
      const uint32_t at = hi + (uint32_t)(c >> 6) * ATOM;
#pragma unroll
      for (int i = 0; i < 16; i += 8) store8_split(at, at + second, row, (c & 63) + i, x + i);
    };
    if (!ph.mma_done(3)) return;
    const Op Kt{sb + SM::K, ATOM, true};
    const uint32_t vb = sb + SM::V;
    if constexpr (D == 64) {
      // atoms [Ut hi, W hi, Ut lo, W lo, Ut rest]: Ut and W are one operand of 128 columns
#pragma unroll
      for (int c = 0; c < 32; c += 16) {
        if (cg < 2) out_u(cg * 32 + c, 2 * ATOM);
        else out_w((cg - 2) * 32 + c, vb + ATOM, 2 * ATOM);
      }
      ph.publish();
      if (warp == 0 && elect_one()) {
        products<8>(Prod(tmem + TM_H, Kt, Op{vb + 2 * ATOM, ATOM, true}, 64, 128, false));
        products<8>(Prod(tmem + TM_H, Kt, Op{vb + 4 * ATOM, ATOM, true}, 64, 64, true));
        products<8>(Prod(tmem + TM_H, Kt, Op{vb, ATOM, true}, 64, 128, true));
        mma_commit(&bars.mma);
      }
      if (!ph.mma_done(5)) return;
    } else {
#pragma unroll
      for (int c = 0; c < 32; c += 16) out_u(cg * 32 + c, SM::OP);
      ph.publish();
      if (warp == 0 && elect_one()) {
        const Pair U{{vb, ATOM, true}, SM::OP};
        for (int i = 2; i >= 0; --i) products<8>(Prod(tmem + TM_H, Kt, U.plane(i), 128, 128, i < 2));
        mma_commit(&bars.mma);
      }
      if (!ph.mma_done(5)) return;
#pragma unroll
      for (int c = 0; c < 32; c += 16) out_w(cg * 32 + c, vb, SM::OP);
      ph.publish();
      if (warp == 0 && elect_one()) {
        const Pair W{{vb, ATOM, true}, SM::OP};
        products<8>(Prod(tmem + TM_M, Kt, W.lo(), 128, 128, false));
        products<8>(Prod(tmem + TM_M, Kt, W.hi, 128, 128, true));
        mma_commit(&bars.mma);
      }
      if (!ph.mma_done(6)) return;
    }
    // Hc in float32, Mc = -K^T rho W as hi and lo; for D = 64 the 64 rows sit
    // in the first 16 lanes of each quadrant
    const int r = D == 64 ? q4 * 16 + lane : row;
    const bool own = D == 128 || lane < 16;
    constexpr int cols = D / 4;   // of each, this group
#pragma unroll
    for (int j = 0; j < cols; j += 16) {
      const int c = cg * cols + j;
      float h[16], m[16];
      tmem_ld16(tmem + lanes + TM_H + c, h);
      tmem_ld16(tmem + lanes + TM_M + c, m);
      if (!own) continue;
      store_tile16(a.H + ci * D * D, D, r, c, h);
#pragma unroll
      for (int i = 0; i < 16; ++i) m[i] = -m[i];
      __nv_bfloat16* d = a.M + (ci * 2 * D + r) * D + c;
      store16_pair(d, d + D * D, m);
    }
  };
  work();
  cta_end(bars, ph, 1, tmem, TM_COLS, warp);
}

// ------------------------------------------------------------------ chain
// X <- e_c X + H_c + Mc X over the chunks of one head and 64 value columns
// (backward: Mc^T, from the last chunk); X in float32 registers, its hi + lo
// copy in shared memory as the operand of the chunk's product and, by TMA, in
// the workspace as its border state.
//
// Bound by latency, a chunk after another, so the work is split by warps that
// meet at mbarriers and nowhere else: 0 issues the products, 1 the loads, 2
// the stores, 4 to 11 hold X (32 columns of a row a thread; the others rest).
// While the tensor core works, those add e X + H.  With sixteen warps that did
// everything between two CTA barriers, the warps beside the issuing ones
// were last to every barrier.  A chunk takes 1.0 us at D = 64 and 1.7 at 128
// (that form: 1.5 and 2.1).
struct ChainArgs {
  const float* gend;
  DeltaChain dir[2];       // forward; backward, by the CTAs behind the forward ones
  int BH;
  Slab slab;
  DevStatus st;
};

template <int D>
struct ChainSmem {
  static constexpr int MS = 2, HS = D == 64 ? 2 : 1;      // slots of Mc and of H
  static constexpr uint32_t SA = D * 128;                 // bytes of a [D][64] atom
  static constexpr uint32_t M = 0, MB = 2 * (D / 64) * SA;   // Mc hi, lo
  static constexpr uint32_t H = MS * MB, HB = D * 64 * 4;
  static constexpr uint32_t X = H + HS * HB;              // two of [hi, lo], in turn
  static constexpr uint32_t BAR = X + 4 * SA;
  static constexpr uint32_t TOTAL = BAR + 256;
};
// Every barrier belongs to a slot, which is filled again only behind the wait
// of its reader: nobody can be a phase behind without being noticed.
struct ChainBars {
  uint64_t m_full[2], m_free[2], h_full[2], h_free[2], x_ready[2], x_free[2], mma, fin;
  uint32_t tmem, abort;
};

template <int D>
TTT_DEVICE_INLINE void chain_cta(uint8_t* smem, const CUtensorMap& mapM, const CUtensorMap& mapXf,
                                 const CUtensorMap& mapXr, const ChainArgs& a, unsigned block) {
  using SM = ChainSmem<D>;
  constexpr int DA = D / 64, MS = SM::MS, HS = SM::HS, XWARPS = 8;
  constexpr uint32_t TM_COLS = 64;
  ChainBars& bars = *reinterpret_cast<ChainBars*>(smem + SM::BAR);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const int slice = block % DA, nch = a.slab.len;
  const bool rev = block >= (unsigned)(DA * a.BH);
  const float* H = rev ? a.dir[1].H : a.dir[0].H;
  const float* S_in = rev ? a.dir[1].S_in : a.dir[0].S_in;
  float* S_out = rev ? a.dir[1].S_out : a.dir[0].S_out;
  const size_t bh = block / DA % a.BH, c0 = a.slab.w0 + bh * nch;
  auto chunk = [&](int i) { return c0 + (rev ? nch - 1 - i : i); };

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.m_full[i], 1);
      mbar_init(&bars.m_free[i], 1);
      mbar_init(&bars.h_full[i], 1);
      mbar_init(&bars.h_free[i], XWARPS);
      mbar_init(&bars.x_ready[i], XWARPS);
      mbar_init(&bars.x_free[i], 1);
    }
    mbar_init(&bars.mma, 1);
    mbar_init(&bars.fin, 1);
    bars.abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars.tmem, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem, 0), sb = smem_u32(smem);
  const Waiter W{&bars.abort, a.st, 1100};

  if (warp == 0) {
    for (int c = 0; c < nch; ++c) {
      const int s = c % MS, b = c & 1;
      if (!W.wait_warp(&bars.m_full[s], (c / MS) & 1, 1) || !W.wait_warp(&bars.x_ready[b], (c >> 1) & 1, 2)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t xb = sb + SM::X + b * 2 * SM::SA, m = sb + SM::M + s * SM::MB, mlo = m + DA * SM::SA;
        const Op X{xb, SM::SA, true}, Xlo{xb + SM::SA, SM::SA, true};
        products<D / 16>(Prod(tmem, Op{mlo, SM::SA, rev}, X, D, 64, false));
        products<D / 16>(Prod(tmem, Op{m, SM::SA, rev}, Xlo, D, 64, true));
        products<D / 16>(Prod(tmem, Op{m, SM::SA, rev}, X, D, 64, true));
        mma_commit(&bars.mma);
        mma_commit(&bars.m_free[s]);
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(&bars.fin);   // nothing in flight outlives the CTA
    __syncwarp();
    W.drain(&bars.fin, 0);
  } else if (warp == 1) {
    int c = 0;
    for (; c < nch; ++c) {
      const int s = c % MS, hs = c % HS;
      if (c >= MS && !W.wait_warp(&bars.m_free[s], (c / MS - 1) & 1, 3)) break;
      if (elect_one()) {
        const int z = (int)(2 * chunk(c));
        mbar_arrive_expect_tx(&bars.m_full[s], SM::MB);
        for (int h = 0; h < 2; ++h)
          for (int k = 0; k < DA; ++k)
            tma_load_3d(smem + SM::M + s * SM::MB + (h * DA + k) * SM::SA, &mapM, &bars.m_full[s], 64 * k, 0, z + h);
      }
      __syncwarp();
      if (c >= HS && !W.wait_warp(&bars.h_free[hs], (c / HS - 1) & 1, 4)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&bars.h_full[hs], SM::HB);
        bulk_load_1d(smem + SM::H + hs * SM::HB, H + chunk(c) * D * D + (size_t)slice * 64 * D, SM::HB, &bars.h_full[hs]);
      }
      __syncwarp();
    }
    if (W.aborted()) {   // the loads of the last rounds, if they were issued
      for (int i = max(0, c - MS); i <= min(c, nch - 1); ++i) W.drain(&bars.m_full[i % MS], (i / MS) & 1);
      for (int i = max(0, c - HS); i < c; ++i) W.drain(&bars.h_full[i % HS], (i / HS) & 1);
    }
  } else if (warp == 2) {
    for (int c = 0; c < nch; ++c) {
      const int b = c & 1;
      if (!W.wait_warp(&bars.x_ready[b], (c >> 1) & 1, 5)) break;
      if (elect_one()) {   // chunk c's border state
        for (int h = 0; h < 2; ++h)
          tma_store_3d(rev ? &mapXr : &mapXf, smem + SM::X + (2 * b + h) * SM::SA, 64 * slice, 0,
                       (int)(2 * chunk(c) + h));
        bulk_commit();
        bulk_wait_read();
        mbar_arrive(&bars.x_free[b]);
      }
      __syncwarp();
    }
    if (elect_one()) bulk_wait_all();   // the same thread: an election has one outcome
    __syncwarp();
  } else if (warp >= 4 && warp < 4 + XWARPS) {
    const int q4 = warp & 3, cg = (warp - 4) >> 2;    // 32 columns of the slice
    const int r = D == 64 ? q4 * 16 + lane : q4 * 32 + lane;
    const bool own = D == 128 || lane < 16;
    const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
    const size_t at = (bh * D + r) * D + slice * 64 + cg * 32;
    float x[32];
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (own && S_in != nullptr) v = *reinterpret_cast<const float4*>(S_in + at + j);
      x[j] = v.x; x[j + 1] = v.y; x[j + 2] = v.z; x[j + 3] = v.w;
    }
    float e = a.gend[chunk(0)];
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
      const int b = c & 1, hs = c % HS;
      ok = c < 2 || W.wait_warp(&bars.x_free[b], ((c >> 1) - 1) & 1, 6);
      if (!ok) break;
      if (own) {
        const uint32_t xb = sb + SM::X + b * 2 * SM::SA;
#pragma unroll
        for (int j = 0; j < 32; j += 8) store8_split(xb, xb + SM::SA, r, cg * 32 + j, x + j);
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.x_ready[b]);
      ok = W.wait_warp(&bars.h_full[hs], (c / HS) & 1, 7);
      if (!ok) break;
      if (own) {
        const float4* h = reinterpret_cast<const float4*>(smem + SM::H + hs * SM::HB) + cg * 8 * D + r;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 v = h[j * D];
          x[4 * j] = fmaf(e, x[4 * j], v.x);
          x[4 * j + 1] = fmaf(e, x[4 * j + 1], v.y);
          x[4 * j + 2] = fmaf(e, x[4 * j + 2], v.z);
          x[4 * j + 3] = fmaf(e, x[4 * j + 3], v.w);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.h_free[hs]);
      if (c + 1 < nch) e = a.gend[chunk(c + 1)];
      ok = W.wait_warp(&bars.mma, c & 1, 8);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < 32; j += 16) {
        float d[16];
        tmem_ld16(tmem + lanes + cg * 32 + j, d);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[j + i] += d[i];
      }
    }
    if (ok && own && S_out != nullptr) {
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4*>(S_out + at + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    }
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
  const float* U;
  void* out;
  int N, out_bf16;
  Slab slab;
  float scale;
  DevStatus st;
};

template <int D>
struct OutSmem {
  static constexpr int DA = D / 64;
  static constexpr uint32_t OP = DA * ATOM, SA = D * 128;
  static constexpr uint32_t Q = 0, K = OP, W = 2 * OP;              // W hi, lo
  static constexpr uint32_t S = 4 * OP;                             // S0 hi, lo
  static constexpr uint32_t U = 0, QS = 3 * ATOM;                   // behind the first products: three planes, Q S0
  static_assert(QS + C * 64 * 4 <= S + 2 * SA, "in the place of the operands");
  static constexpr uint32_t GATES = S + 2 * SA, BAR = GATES + sizeof(Gates), TOTAL = BAR + 80;
};

template <int D>
TTT_DEVICE_INLINE void out_cta(uint8_t* smem, const CUtensorMap& mapQ, const CUtensorMap& mapK,
                               const CUtensorMap& mapW, const CUtensorMap& mapS, const OutArgs& a,
                               unsigned block) {
  using SM = OutSmem<D>;
  constexpr int DA = D / 64;
  constexpr uint32_t TM_P = 0, TM_W = 128, TM_Q = 192, TM_COLS = 256;   // P U takes Q S0's place
  Bars& bars = *reinterpret_cast<Bars*>(smem + SM::BAR);
  Gates& gates = *reinterpret_cast<Gates*>(smem + SM::GATES);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const ChunkId id(block, DA, a.slab, a.N);
  const int slice = id.slice;
  const size_t ci = id.ci;
  const uint32_t sb = smem_u32(smem);
  const uint32_t tmem = cta_begin(bars, TM_COLS, warp, [&]() {
    mbar_arrive_expect_tx(&bars.load[0], 4 * SM::OP + 2 * SM::SA);
    for (int i = 0; i < DA; ++i) {
      tma_load_3d(smem + SM::Q + i * ATOM, &mapQ, &bars.load[0], 64 * i, id.t0, (int)id.bh);
      tma_load_3d(smem + SM::K + i * ATOM, &mapK, &bars.load[0], 64 * i, id.t0, (int)id.bh);
      for (int h = 0; h < 2; ++h)
        tma_load_3d(smem + SM::W + (h * DA + i) * ATOM, &mapW, &bars.load[0], 64 * i, 0, (int)(2 * ci + h));
    }
    for (int h = 0; h < 2; ++h)
      tma_load_3d(smem + SM::S + h * SM::SA, &mapS, &bars.load[0], 64 * slice, 0, (int)(2 * ci + h));
  });
  Phase ph{Waiter{&bars.abort, a.st, 1200}, &bars.mma, 0};
  const int q4 = warp & 3, cg = warp >> 2, row = q4 * 32 + lane;
  const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
  if (cg == 1) {
    load_gates(gates, a.g ? a.g + id.tok : nullptr, a.beta + id.tok, id.n, row);
  }
  // this thread's 16 values of Ut, while the operands travel
  float u[16];
  load_tile16(a.U + ci * C * D, C, row, slice * 64 + cg * 16, u);
  auto work = [&]() {
    const Op Q{sb + SM::Q, ATOM, false}, K{sb + SM::K, ATOM, false};
    const Pair Wp{{sb + SM::W, ATOM, false}, SM::OP}, S{{sb + SM::S, SM::SA, true}, SM::SA};
    if (warp == 0 && ph.W.wait_warp(&bars.load[0], 0, 1) && elect_one()) {
      products<D / 16>(Prod(tmem + TM_W, Wp.lo(), S.hi, 128, 64, false), Prod(tmem + TM_P, Q, K, 128, 128, false),
                       Prod(tmem + TM_Q, Q, S.lo(), 128, 64, false));
      products<D / 16>(Prod(tmem + TM_W, Wp.hi, S.lo(), 128, 64, true), Prod(tmem + TM_Q, Q, S.hi, 128, 64, true));
      products<D / 16>(Prod(tmem + TM_W, Wp.hi, S.hi, 128, 64, true));
      mma_commit(&bars.mma);
    }
    if (!ph.mma_done(2)) return;
    // U = Ut - W S0, and Q S0 into shared memory (this thread's values stay its own)
    float* qs = reinterpret_cast<float*>(smem + SM::QS) + (cg * 4 * C + row) * 4;
    {
      float w[16];
      tmem_ld16(tmem + lanes + TM_W + cg * 16, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] -= w[i];
#pragma unroll
      for (int i = 0; i < 16; i += 8)
        store8_split3(sb + SM::U, sb + SM::U + ATOM, sb + SM::U + 2 * ATOM, row, cg * 16 + i, u + i);
      tmem_ld16(tmem + lanes + TM_Q + cg * 16, w);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(qs + i * C * 4) = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    // P = Gam . Q K^T on and below the diagonal becomes an operand in tensor memory
    // in the place of Q K^T and W S0, three planes of 64 columns
    float x[32];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int c0 = cg * 32 + b * 16;
      if (c0 <= q4 * 32 + 31) {
        tmem_ld16(tmem + lanes + TM_P + c0, x + 16 * b);
        weigh16<true>(gates, q4 * 32, row, c0, 1.f, x + 16 * b);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[16 * b + j] = 0.f;
      }
    }
    tc_fence_before();
    __syncthreads();   // all of Q K^T and W S0 has been read
    tc_fence_after();
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float *v = x + 16 * b + 2 * j;
          h[j] = pack_bf16x2(v[0], v[1]);
          v[0] -= bf16lo(h[j]);
          v[1] -= bf16hi(h[j]);
        }
        tmem_st8_issue(tmem + lanes + TM_P + 64 * p + cg * 16 + 8 * b, h);
      }
    tmem_wait_st();
    ph.publish();
    if (warp == 0 && elect_one()) {
      // two planes would leave 2.6e-6 of the outputs for P and for U each, and lo lo
      // 2.8e-6 (together 4.7e-6); these leave 4e-8, and the outputs are as far off as S0
      // and W S0, 9e-7.  It takes 2 to 3 % of the call (64 heads of 64, 32K tokens: 1689
      // us against 1653)
      const Pair U{{sb + SM::U, ATOM, true}, ATOM};
      const uint32_t hi = tmem + TM_P, lo = hi + 64, rest = hi + 128, o = tmem + TM_Q;
      products<8>(Prod(o, rest, U.hi, 64, false));
      products<8>(Prod(o, hi, U.plane(2), 64, true));
      products<8>(Prod(o, lo, U.lo(), 64, true));
      products<8>(Prod(o, lo, U.hi, 64, true));
      products<8>(Prod(o, hi, U.lo(), 64, true));
      products<8>(Prod(o, hi, U.hi, 64, true));
      mma_commit(&bars.mma);
    }
    if (!ph.mma_done(3)) return;
    const float gam = a.scale * gate_decay(gates, row);
    float o[16];
    tmem_ld16(tmem + lanes + TM_Q + cg * 16, o);
    if (row >= id.n) return;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(qs + i * C);
      o[i] = fmaf(gam, v.x, a.scale * o[i]);
      o[i + 1] = fmaf(gam, v.y, a.scale * o[i + 1]);
      o[i + 2] = fmaf(gam, v.z, a.scale * o[i + 2]);
      o[i + 3] = fmaf(gam, v.w, a.scale * o[i + 3]);
    }
    const size_t at = (id.tok + row) * D + slice * 64 + cg * 16;
    if (a.out_bf16) {
      store_bf16_row16(static_cast<__nv_bfloat16*>(a.out) + at, o);
    } else {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    }
  };
  work();
  cta_end(bars, ph, 1, tmem, TM_COLS, warp);
}

// ------------------------------------------------------------------ kernels
template <int D>
__global__ void __launch_bounds__(THREADS, D == 64 ? 2 : 1)
    delta_prep_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                      PrepArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  prep_cta<D>(smem, mapK, mapV, a, blockIdx.x);
}
template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    delta_chain_kernel(const __grid_constant__ CUtensorMap mapM, const __grid_constant__ CUtensorMap mapXf,
                       const __grid_constant__ CUtensorMap mapXr, ChainArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  chain_cta<D>(smem, mapM, mapXf, mapXr, a, blockIdx.x);
}

// The forward pass goes over the sequence in slabs, one launch after another:
// the recurrence over slab i, the outputs of slab i - 1 and the preparation of
// slab i + 1 share a launch, so the recurrence, which keeps a CTA a head and
// 64 columns busy with latency, costs next to nothing, and the workspace is
// that of three slabs.  No CTA waits for another one of its launch.
struct FwdMaps {
  CUtensorMap q, k, v, w, m, x;   // x as the chain stores it and the outputs read it
};
struct FwdArgs {
  ChainArgs chain;
  OutArgs out;
  PrepArgs prep;
  unsigned n_chain, n_out;        // CTAs of these roles, first in the grid; the others prepare
};
template <int D>
struct FwdSmem {
  static constexpr uint32_t most(uint32_t a, uint32_t b) { return a > b ? a : b; }
  static constexpr uint32_t TOTAL = most(PrepSmem<D>::TOTAL, most(ChainSmem<D>::TOTAL, OutSmem<D>::TOTAL));
};
static_assert(2 * (FwdSmem<64>::TOTAL + 1024) <= 233472, "two CTAs an SM");

template <int D>
__global__ void __launch_bounds__(THREADS, D == 64 ? 2 : 1)
    delta_fwd_kernel(const __grid_constant__ FwdMaps maps, const __grid_constant__ FwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const unsigned b = blockIdx.x;
  if (b < a.n_chain) chain_cta<D>(smem, maps.m, maps.x, maps.x, a.chain, b);
  else if (b < a.n_chain + a.n_out) out_cta<D>(smem, maps.q, maps.k, maps.w, maps.x, a.out, b - a.n_chain);
  else prep_cta<D>(smem, maps.k, maps.v, a.prep, b - a.n_chain - a.n_out);
}

template <int D>
int prep_launch(const DeltaLaunch& p, const DeltaPrepOut& o, cudaStream_t stream) {
  const int BH = p.B * p.H, nch = tiles_of(p.N, C);
  const uint64_t nc = (uint64_t)BH * nch, rs = D * 2;
  CUtensorMap mk, mv;
  if (make_tmap_bf16_3d(&mk, p.k, D, p.N, BH, rs, p.N * rs, 64, C) ||
      make_tmap_bf16_3d(&mv, p.v, D, p.N, BH, rs, p.N * rs, 64, C))
    return -1;
  static std::atomic<uint64_t> attr{0};
  if (allow_dynamic_smem(delta_prep_kernel<D>, (int)PrepSmem<D>::TOTAL, attr)) return -1;
  const PrepArgs a{(const __nv_bfloat16*)p.g, (const __nv_bfloat16*)p.beta, o.gend, o.H, o.U, o.W, o.M, o.T,
                   p.N, Slab{0, nch, 0}, p.st};
  prof_before(K_DELTA_PREP, stream);
  const cudaError_t err = launch_pdl(
      delta_prep_kernel<D>, dim3((unsigned)nc), dim3(THREADS), PrepSmem<D>::TOTAL, stream,
      mk, mv, a);
  prof_after(K_DELTA_PREP, stream);
  return err == cudaSuccess ? 0 : -1;
}

template <int D>
int chain_launch(const DeltaLaunch& p, const float* gend, const __nv_bfloat16* M, const DeltaChain& fwd,
                 const DeltaChain& rev, cudaStream_t stream) {
  const int BH = p.B * p.H, nch = tiles_of(p.N, C);
  const uint64_t nc = (uint64_t)BH * nch, rs = D * 2;
  CUtensorMap mm, mf, mr;
  if (make_tmap_bf16_3d(&mm, M, D, D, 2 * nc, rs, D * rs, 64, D) ||
      make_tmap_bf16_3d(&mf, fwd.X, D, D, 2 * nc, rs, D * rs, 64, D) ||
      make_tmap_bf16_3d(&mr, rev.X, D, D, 2 * nc, rs, D * rs, 64, D))
    return -1;
  static std::atomic<uint64_t> attr{0};
  if (allow_dynamic_smem(delta_chain_kernel<D>, (int)ChainSmem<D>::TOTAL, attr)) return -1;
  const ChainArgs a{gend, {fwd, rev}, BH, Slab{0, nch, 0}, p.st};
  prof_before(K_DELTA_CHAIN, stream);
  const cudaError_t err = launch_pdl(
      delta_chain_kernel<D>, dim3(2u * (unsigned)(BH * (D / 64))), dim3(THREADS), ChainSmem<D>::TOTAL, stream,
      mm, mf, mr, a);
  prof_after(K_DELTA_CHAIN, stream);
  return err == cudaSuccess ? 0 : -1;
}

// Chunks of a slab: about a sixth of the sequence, and whole rounds of preparing
// CTAs on the device (two at least; where the recurrence keeps few SMs, on the
// others), but four chunks at least.  64 heads of 64, 32K tokens: 4 slabs 1755
// us, 6 1784, 8 1828, 16 1914; the workspace is three slabs.  8 heads of 128,
// 32749 tokens: slabs of 2.6 rounds 650 us, of whole ones 614.
int slab_chunks(int BH, int nch, int D, int sms) {
  const int all = sms * (D == 64 ? 2 : 1), chain = BH * (D / 64);
  const int free = chain <= all / 4 ? all - chain : all;
  const long long rounds = std::max(2ll, ((long long)BH * ((nch + 5) / 6) + free - 1) / free);
  return std::min(nch, std::max((int)(rounds * free / BH), 4));
}

template <int D>
int fwd_launch(const DeltaLaunch& p, cudaStream_t stream) {
  const int BH = p.B * p.H, nch = tiles_of(p.N, C), len = slab_chunks(BH, nch, D, p.sms);
  const int slabs = (nch + len - 1) / len;
  const DeltaUmmaWorkspace w = delta_umma_layout(BH, p.N, D, p.sms);
  const uint64_t nc = w.chunks, rs = D * 2;
  uint8_t* ws = delta_ws_base(p.ws);
  auto bf = [&](size_t at) { return reinterpret_cast<__nv_bfloat16*>(ws + at); };
  auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
  FwdMaps maps;
  if (make_tmap_bf16_3d(&maps.q, p.q, D, p.N, BH, rs, p.N * rs, 64, C) ||
      make_tmap_bf16_3d(&maps.k, p.k, D, p.N, BH, rs, p.N * rs, 64, C) ||
      make_tmap_bf16_3d(&maps.v, p.v, D, p.N, BH, rs, p.N * rs, 64, C) ||
      make_tmap_bf16_3d(&maps.w, bf(w.W), D, C, 2 * nc, rs, C * rs, 64, C) ||
      make_tmap_bf16_3d(&maps.m, bf(w.M), D, D, 2 * nc, rs, D * rs, 64, D) ||
      make_tmap_bf16_3d(&maps.x, bf(w.X), D, D, 2 * nc, rs, D * rs, 64, D))
    return -1;
  static std::atomic<uint64_t> attr{0};
  if (allow_dynamic_smem(delta_fwd_kernel<D>, (int)FwdSmem<D>::TOTAL, attr)) return -1;
  const __nv_bfloat16 *g = (const __nv_bfloat16*)p.g, *beta = (const __nv_bfloat16*)p.beta;
  auto slab = [&](int i) {
    return Slab{i * len, std::min(len, nch - i * len), (size_t)(i % 3) * BH * len};
  };
  for (int j = 0; j < slabs + 2; ++j) {   // prepare slab j, recur over j - 1, outputs of j - 2
    FwdArgs a{};
    unsigned n_prep = 0;
    if (j < slabs) {
      a.prep = PrepArgs{g, beta, f32(w.gend), f32(w.H), f32(w.U), bf(w.W), bf(w.M), nullptr, p.N, slab(j), p.st};
      n_prep = (unsigned)BH * a.prep.slab.len;
    }
    if (j >= 1 && j <= slabs) {
      // every slab's recurrence starts from S and leaves its end there
      const DeltaChain dir{f32(w.H), p.S, p.S, nullptr};
      a.chain = ChainArgs{f32(w.gend), {dir, {}}, BH, slab(j - 1), p.st};
      a.n_chain = (unsigned)(BH * (D / 64));
    }
    if (j >= 2) {
      a.out = OutArgs{g, beta, f32(w.U), p.out, p.N, p.out_bf16, slab(j - 2), p.scale, p.st};
      a.n_out = (unsigned)(BH * (D / 64)) * a.out.slab.len;
    }
    prof_before(K_DELTA_FWD, stream);
    const cudaError_t err = launch_pdl(
      delta_fwd_kernel<D>, dim3(a.n_chain + a.n_out + n_prep), dim3(THREADS), FwdSmem<D>::TOTAL, stream,
      maps, a);
    prof_after(K_DELTA_FWD, stream);
    if (err != cudaSuccess) return -1;
  }
  return 0;
}

}  // namespace

// Short sequences go token by token: the chunk kernels' latency is that of a
// whole chunk and of three launches (23 us forward, 52 us backward at D = 64;
// 32 and 64 at 128), the recurrent ones' 0.1 us a token at D = 64 and 0.14 at 128
// (backward the same behind 24 and 40), times the rounds that their CTAs of 16
// value columns take on the device.  Both grow alike with the heads once the
// chunks too fill it, so rounds count up to 5.  Token by token against chunks, us:
// forward 8 heads of 64, 128 tokens 17 / 24, 256 tokens 29 / 23; of 128, 128 tokens
// 25 / 32, 256 tokens 43 / 33; 128 heads of 64, 32 tokens 16 / 24, 64 tokens 27 /
// 24.  Backward 8 heads of 64, 256 tokens 47 / 51, 300 tokens 51 / 53, 512 tokens
// 72 / 54; of 128, 128 tokens 59 / 64, 200 tokens 72 / 65; 128 heads of 64, 32
// tokens 41 / 55, 64 tokens 69 / 56.  Heads of other sizes, or of two, go token by
// token at every length: the tiles, the operands' layouts and the D x D recurrence
// are written for one D.
bool delta_uses_umma(int bf16, int dk, int dv, long long BH, int N, int sms, bool backward) {
  if (!bf16 || dk != dv || (dk != 64 && dk != 128)) return false;
  const double rounds = (double)BH * (dv / 16) * (backward ? 2 : 1) / sms;
  return N * std::min(std::max(rounds, 1.0), 5.0) > (!backward ? 190 : dk == 64 ? 270 : 150);
}

DeltaUmmaWorkspace delta_umma_layout(int BH, int N, int D, int sms) {
  DeltaUmmaWorkspace w{};
  const int nch = tiles_of(N, C), len = slab_chunks(BH, nch, D, sms);
  const size_t nc = (size_t)BH * std::min(nch, 3 * len);
  w.chunks = nc;
  size_t at = 512;   // see delta_ws_base
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  w.gend = take(nc * 4);
  w.W = take(nc * 2 * C * D * 2);
  w.U = take(nc * C * D * 4);
  w.M = take(nc * 2 * D * D * 2);
  w.H = take(nc * D * D * 4);
  w.X = take(nc * 2 * D * D * 2);
  w.total = at;
  return w;
}

int launch_delta_prep(const DeltaLaunch& p, const DeltaPrepOut& o, cudaStream_t stream) {
  return p.dk == 64 ? prep_launch<64>(p, o, stream) : prep_launch<128>(p, o, stream);
}
int launch_delta_chain(const DeltaLaunch& p, const float* gend, const __nv_bfloat16* M, const DeltaChain& fwd,
                       const DeltaChain& rev, cudaStream_t stream) {
  return p.dk == 64 ? chain_launch<64>(p, gend, M, fwd, rev, stream)
                    : chain_launch<128>(p, gend, M, fwd, rev, stream);
}
int launch_delta_umma(const DeltaLaunch& p, cudaStream_t stream) {
  return p.dk == 64 ? fwd_launch<64>(p, stream) : fwd_launch<128>(p, stream);
}

}  // namespace ttt
