// delta_umma_bwd.cu -- gradients of the gated delta rule on tensor cores:
// bf16, dk = dv = D = 64 or 128, chunks of 128 tokens.
//
// With the chunk's matrices of the forward pass (delta_umma.cu; Gam, gam, rho,
// T, W, Ut, U, S0 its start state), X1 = dL/dS at its end and P = Gam . Q K^T:
//   dU = scale P^T dO + rho K X1,   Y = T^T dU          (of T's right-hand side)
//   X0 = gam_last X1 + Q^T (scale gam dO) - W^T dU
//      = (gam_last I + Mc^T) X1 + Hb,  Hb = Q^T (scale gam dO) - W^T (scale P^T dO)
//   dV = beta Y
//   Mq = Gam . scale dO U^T (j <= i),   Mk = -beta_i Gam . Y U^T (j < i)
//   dQ = scale gam dO S0^T + Mq K
//   dK = [Mk K - gam beta Y S0^T] + [Mq^T Q + Mk^T K] + [rho U X1^T]
//   dbeta_i = Y_i . (V_i - gam_i S0^T k_i) - sum_j Gam_ij (Y_i . U_j) (k_i . k_j)
// and, with r_i = gam_i (q_i . scale S0 dO_i - beta_i k_i . S0 Y_i), V_ij = Mq_ij
// q_i . k_j + Mk_ij k_i . k_j (j < i) and w_i = k_i . [third part of dk_i],
//   dg_t = sum_{i >= t} r_i + sum_{i >= t > j} V_ij + sum_{i < t} w_i + gam_last <X1, S0>
// where every term holds the decay of token t (sums of q_i . dq_i and k_i . dk_i
// over i >= t would hold the V_ij of i, j >= t with both signs, and where the
// decays are strong what rounding leaves of them is larger than dg_t).  So the
// reverse recurrence runs over the same Mc, side
// by side with the forward one:
//   delta_prep_kernel      K, V -> W, Ut, T, Mc, Hc
//   delta_hb_kernel        Q, K, dO, W -> Hb, Z = -scale P^T dO
//   delta_chain_kernel     S0 and X1 of every chunk, dS0
//   delta_vals_kernel      U, Y, dV, first part of dbeta; 64 value columns a CTA
//   delta_keys_kernel      dQ, dK, r, w, sums of V, second part of dbeta; 64 key columns a CTA
//   delta_gate_grad_kernel dg, dbeta
#include <algorithm>

#include "delta_umma.cuh"

namespace ttt {

using namespace dl;

namespace {

constexpr int THREADS = 512;        // four column groups of 128 rows

TTT_DEVICE_INLINE void zero16(float* x) {
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = 0.f;
}
// 16 columns of a row into a matrix of two column atoms: [hi 0, hi 1, lo 0, lo 1]
TTT_DEVICE_INLINE void store16_square(uint32_t base, int row, int c0, const float* x) {
  const uint32_t hi = base + (uint32_t)(c0 >> 6) * ATOM, lo = hi + 2 * ATOM;
  store8_split(hi, lo, row, c0 & 63, x);
  store8_split(hi, lo, row, (c0 & 63) + 8, x + 8);
}
// the same, and a third plane [0, 1] at `rest`
TTT_DEVICE_INLINE void store16_square3(uint32_t base, uint32_t rest, int row, int c0, const float* x) {
  const uint32_t at = (uint32_t)(c0 >> 6) * ATOM;
#pragma unroll
  for (int i = 0; i < 16; i += 8)
    store8_split3(base + at, base + at + 2 * ATOM, rest + at, row, (c0 & 63) + i, x + i);
}
// the column groups' sums of a row, [group][row]
TTT_DEVICE_INLINE float row_total(const float* red, int row) {
  return (red[row] + red[C + row]) + (red[2 * C + row] + red[3 * C + row]);
}

// ------------------------------------------------------------------ Hb
// Hb is what dS0 is made of, in float32: its operands are carried in three
// planes (hi + lo alone left 3e-6 of dS0, mostly by scale gam dO).  Its shared
// memory leaves one CTA an SM, whose phases' latency bounds it: 2048 chunks of
// heads of 64 118 us.
struct HbArgs {
  const __nv_bfloat16 *g, *beta;
  float *H, *Z;            // Z = -scale P^T dO: [BH nch][D / 64] float32 tiles [128][64]
  int N, nch;
  float scale;
  DevStatus st;
};

template <int D>
struct HbSmem {
  static constexpr int DA = D / 64;
  // three planes of P over K; then three each of -scale P^T dO, scale gam dO
  static constexpr uint32_t Q = 0, P = DA * ATOM;
  static constexpr uint32_t W = P + 6 * ATOM, DO = W + 2 * DA * ATOM;
  static constexpr uint32_t GATES = DO + ATOM, BAR = GATES + sizeof(Gates), TOTAL = BAR + 80;
};

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    delta_hb_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                    const __grid_constant__ CUtensorMap mapD, const __grid_constant__ CUtensorMap mapW, HbArgs a) {
  using SM = HbSmem<D>;
  constexpr int DA = D / 64;
  constexpr uint32_t TM_P = 0, TM_U = 128, TM_COLS = 256;   // Hb's accumulators take their places
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + SM::BAR);
  Gates& gates = *reinterpret_cast<Gates*>(smem + SM::GATES);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const ChunkId id(blockIdx.x, DA, Slab{0, a.nch, 0}, a.N);
  const uint32_t sb = smem_u32(smem);
  const uint32_t tmem = cta_begin(bars, TM_COLS, warp, [&]() {
    mbar_arrive_expect_tx(&bars.load[0], 4 * DA * ATOM + ATOM);
    for (int i = 0; i < DA; ++i) {
      tma_load_3d(smem + SM::Q + i * ATOM, &mapQ, &bars.load[0], 64 * i, id.t0, (int)id.bh);
      tma_load_3d(smem + SM::P + i * ATOM, &mapK, &bars.load[0], 64 * i, id.t0, (int)id.bh);
      for (int h = 0; h < 2; ++h)
        tma_load_3d(smem + SM::W + (h * DA + i) * ATOM, &mapW, &bars.load[0], 64 * i, 0, (int)(2 * id.ci + h));
    }
    tma_load_3d(smem + SM::DO, &mapD, &bars.load[0], 64 * id.slice, id.t0, (int)id.bh);
  });
  Phase ph{Waiter{&bars.abort, a.st, 1300}, &bars.mma, 0};
  const int q4 = warp & 3, cg = warp >> 2, row = q4 * 32 + lane;
  const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
  if (cg == 1) load_gates(gates, a.g ? a.g + id.tok : nullptr, a.beta + id.tok, id.n, row);
  auto work = [&]() {
    const Op dOmn{sb + SM::DO, ATOM, true}, Qmn{sb + SM::Q, ATOM, true};
    if (warp == 0 && ph.W.wait_warp(&bars.load[0], 0, 1) && elect_one()) {
      products<D / 16>(Prod(tmem + TM_P, Op{sb + SM::Q, ATOM, false}, Op{sb + SM::P, ATOM, false}, 128, 128, false));
      mma_commit(&bars.mma);
    }
    if (!ph.mma_done(2)) return;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int c0 = cg * 32 + b * 16;
      float x[16];
      if (c0 <= q4 * 32 + 31) {
        tmem_ld16(tmem + lanes + TM_P + c0, x);
        weigh16<true>(gates, q4 * 32, row, c0, 1.f, x);
      } else {
        zero16(x);
      }
      const uint32_t at = sb + SM::P + (uint32_t)(cg >> 1) * ATOM;   // [plane][column atom]
#pragma unroll
      for (int i = 0; i < 16; i += 8)
        store8_split3(at, at + 2 * ATOM, at + 4 * ATOM, row, (c0 & 63) + i, x + i);
    }
    ph.publish();
    if (warp == 0 && elect_one()) {
      const Pair Pt{{sb + SM::P, ATOM, true}, 2 * ATOM};
      for (int i = 2; i >= 0; --i) products<8>(Prod(tmem + TM_U, Pt.plane(i), dOmn, 128, 64, i < 2));
      mma_commit(&bars.mma);
    }
    if (!ph.mma_done(3)) return;
    float u[16];
    tmem_ld16(tmem + lanes + TM_U + cg * 16, u);
    {
      const float f = a.scale * gate_decay(gates, row);
#pragma unroll
      for (int j = 0; j < 16; j += 8) {
        float d[8];
        load8(sb + SM::DO, row, cg * 16 + j, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[j + i] *= -a.scale;
          d[i] *= f;
        }
        const uint32_t at = sb + SM::P;
        store8_split3(at, at + ATOM, at + 2 * ATOM, row, cg * 16 + j, u + j);
        store8_split3(at + 3 * ATOM, at + 4 * ATOM, at + 5 * ATOM, row, cg * 16 + j, d);
      }
    }
    ph.publish();
    if (warp == 0 && elect_one()) {
      const Pair U{{sb + SM::P, ATOM, true}, ATOM}, G{{sb + SM::P + 3 * ATOM, ATOM, true}, ATOM};
      const Pair Wt{{sb + SM::W, ATOM, true}, DA * ATOM};
      // the three planes side by side are one operand of 192 columns: an
      // accumulator each, of which the first holds the large terms
      products<8>(Prod(tmem, Wt.hi, U.hi, D, 192, false));
      products<8>(Prod(tmem + 64, Wt.lo(), U.hi, D, 128, true));
      products<8>(Prod(tmem, Qmn, G.hi, D, 192, true));
      mma_commit(&bars.mma);
    }
    store_tile16(a.Z + (id.ci * DA + id.slice) * C * 64, C, row, cg * 16, u);
    if (!ph.mma_done(4)) return;
    const int r = D == 64 ? q4 * 16 + lane : row;
    float h[16];
    tmem_ld16(tmem + lanes + 128 + cg * 16, h);
#pragma unroll
    for (int p = 1; p >= 0; --p) {
      float y[16];
      tmem_ld16(tmem + lanes + 64 * p + cg * 16, y);
#pragma unroll
      for (int i = 0; i < 16; ++i) h[i] += y[i];
    }
    if (D == 128 || lane < 16) store_tile16(a.H + id.ci * D * D, D, r, id.slice * 64 + cg * 16, h);
  };
  work();
  cta_end(bars, ph, 1, tmem, TM_COLS, warp);
}

// ------------------------------------------------------------------ values
// Reads T, W, Ut, the border states and what Hb left and writes U and Y, 0.64 GB in
// 140 us for 2048 chunks of heads of 64: 4.6 TB/s, 70 % of what HBM gives.  Bound by
// the latency of the loads, which one CTA an SM (its shared memory) does not hide.
struct ValsArgs {
  const __nv_bfloat16 *g, *beta, *v;
  const float *Ut, *Z;     // Z in the memory that Y takes
  __nv_bfloat16* dv;
  float* bpart;            // [D / 64][BH N]
  int N, nch;
  size_t tokens;
  DevStatus st;
};

template <int D>
struct ValsSmem {
  static constexpr int DA = D / 64;
  static constexpr uint32_t SA = D * 128;
  static constexpr uint32_t T = 0;                            // W first
  static constexpr uint32_t K = 4 * ATOM, S = K + DA * ATOM, X = S + 2 * SA, U = X + 2 * SA, Y = U + 2 * ATOM;
  static constexpr uint32_t RED = K;                          // behind the first products
  static constexpr uint32_t GATES = Y + 2 * ATOM, BAR = GATES + sizeof(Gates), TOTAL = BAR + 80;
};

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    delta_vals_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapW,
                      const __grid_constant__ CUtensorMap mapU, const __grid_constant__ CUtensorMap mapY,
                      const __grid_constant__ CUtensorMap mapT, const __grid_constant__ CUtensorMap mapS,
                      const __grid_constant__ CUtensorMap mapX, ValsArgs a) {
  using SM = ValsSmem<D>;
  constexpr int DA = D / 64;
  constexpr uint32_t TM_W = 0, TM_Z = 64, TM_X = 128, TM_Y = 192, TM_COLS = 256;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + SM::BAR);
  Gates& gates = *reinterpret_cast<Gates*>(smem + SM::GATES);
  float* red = reinterpret_cast<float*>(smem + SM::RED);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const ChunkId id(blockIdx.x, DA, Slab{0, a.nch, 0}, a.N);
  const uint32_t sb = smem_u32(smem);
  const uint32_t tmem = cta_begin(bars, TM_COLS, warp, [&]() {
    mbar_arrive_expect_tx(&bars.load[0], 3 * DA * ATOM + 4 * SM::SA);
    for (int i = 0; i < DA; ++i) {
      tma_load_3d(smem + SM::K + i * ATOM, &mapK, &bars.load[0], 64 * i, id.t0, (int)id.bh);
      for (int h = 0; h < 2; ++h)
        tma_load_3d(smem + SM::T + (h * DA + i) * ATOM, &mapW, &bars.load[0], 64 * i, 0, (int)(2 * id.ci + h));
    }
    for (int h = 0; h < 2; ++h) {
      const int z = (int)(2 * id.ci + h), x = 64 * id.slice;
      tma_load_3d(smem + SM::S + h * SM::SA, &mapS, &bars.load[0], x, 0, z);
      tma_load_3d(smem + SM::X + h * SM::SA, &mapX, &bars.load[0], x, 0, z);
    }
  });
  Phase ph{Waiter{&bars.abort, a.st, 1400}, &bars.mma, 0};
  const int q4 = warp & 3, cg = warp >> 2, row = q4 * 32 + lane;
  const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
  if (cg == 1) load_gates(gates, a.g ? a.g + id.tok : nullptr, a.beta + id.tok, id.n, row);
  // this thread's 16 values of Ut and Z, while the operands travel
  const size_t at_slice = id.ci * DA + id.slice;
  float u[16], y[16];
  load_tile16(a.Ut + id.ci * C * D, C, row, id.slice * 64 + cg * 16, u);
  load_tile16(a.Z + at_slice * C * 64, C, row, cg * 16, y);
  int loads = 1;
  auto work = [&]() {
    const Op K{sb + SM::K, ATOM, false};
    const Pair W{{sb + SM::T, ATOM, false}, DA * ATOM};
    const Pair S{{sb + SM::S, SM::SA, true}, SM::SA}, X{{sb + SM::X, SM::SA, true}, SM::SA};
    if (warp == 0 && ph.W.wait_warp(&bars.load[0], 0, 1) && elect_one()) {
      products<D / 16>(Prod(tmem + TM_W, W.lo(), S.hi, 128, 64, false), Prod(tmem + TM_Z, K, S.lo(), 128, 64, false),
                       Prod(tmem + TM_X, K, X.lo(), 128, 64, false));
      products<D / 16>(Prod(tmem + TM_W, W.hi, S.lo(), 128, 64, true), Prod(tmem + TM_Z, K, S.hi, 128, 64, true),
                       Prod(tmem + TM_X, K, X.hi, 128, 64, true));
      products<D / 16>(Prod(tmem + TM_W, W.hi, S.hi, 128, 64, true));
      mma_commit(&bars.mma);
    }
    if (!ph.mma_done(2)) return;
    if (warp == 2 && elect_one()) {   // T takes W's place
      mbar_arrive_expect_tx(&bars.load[1], 4 * ATOM);
      for (int h = 0; h < 2; ++h)
        for (int i = 0; i < 2; ++i)
          tma_load_3d(smem + SM::T + (2 * h + i) * ATOM, &mapT, &bars.load[1], 64 * i, 0, (int)(2 * id.ci + h));
    }
    loads = 3;
    // U = Ut - W S0;  dU = rho K X1 - Z; their third planes take the places of S0 and X1
    // (two planes, and lo lo left out, would be 3e-6 of dV, and 2.6e-6 of dQ and dK)
    {
      const float rho = gate_ratio(gates, C - 1, row);
      const int c = cg * 16;
      float w[16], x[16];
      tmem_ld16(tmem + lanes + TM_W + c, w);
      tmem_ld16(tmem + lanes + TM_X + c, x);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        u[i] -= w[i];
        y[i] = fmaf(rho, x[i], -y[i]);
      }
#pragma unroll
      for (int b = 0; b < 16; b += 8) {
        store8_split3(sb + SM::U, sb + SM::U + ATOM, sb + SM::S, row, c + b, u + b);
        store8_split3(sb + SM::Y, sb + SM::Y + ATOM, sb + SM::X, row, c + b, y + b);
      }
    }
    ph.publish();
    if (warp == 1 && elect_one()) {
      for (int h = 0; h < 3; ++h)
        tma_store_3d(&mapU, smem + (h < 2 ? SM::U + h * ATOM : SM::S), 0, 0, (int)(3 * at_slice + h));
      bulk_commit();
    }
    if (warp == 0 && ph.W.wait_warp(&bars.load[1], 0, 3) && elect_one()) {
      const Pair Tt{{sb + SM::T, ATOM, true}, 2 * ATOM}, dU{{sb + SM::Y, ATOM, true}, ATOM};
      products<8>(Prod(tmem + TM_Y, Tt.hi, Op{sb + SM::X, ATOM, true}, 128, 64, false));
      products<8>(Prod(tmem + TM_Y, Tt.lo(), dU.lo(), 128, 64, true));
      products<8>(Prod(tmem + TM_Y, Tt.lo(), dU.hi, 128, 64, true));
      products<8>(Prod(tmem + TM_Y, Tt.hi, dU.lo(), 128, 64, true));
      products<8>(Prod(tmem + TM_Y, Tt.hi, dU.hi, 128, 64, true));
      mma_commit(&bars.mma);
    }
    if (!ph.mma_done(4)) return;
    {
      float acc = 0.f;
      const float beta = gates.beta[row], gam = gate_decay(gates, row);
      const size_t at = (id.tok + row) * D + id.slice * 64 + cg * 16;
      float z[16];
      tmem_ld16(tmem + lanes + TM_Y + cg * 16, y);
      tmem_ld16(tmem + lanes + TM_Z + cg * 16, z);
#pragma unroll
      for (int j = 0; j < 16; j += 8) store8_split(sb + SM::Y, sb + SM::Y + ATOM, row, cg * 16 + j, y + j);
      if (row < id.n) {
        const uint4* vp = reinterpret_cast<const uint4*>(a.v + at);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 t = vp[j];
          const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc = fmaf(y[8 * j + 2 * i], bf16lo(w[i]) - gam * z[8 * j + 2 * i], acc);
            acc = fmaf(y[8 * j + 2 * i + 1], bf16hi(w[i]) - gam * z[8 * j + 2 * i + 1], acc);
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] *= beta;
        store_bf16_row16(a.dv + at, y);
      }
      red[cg * C + row] = acc;
    }
    ph.publish();
    if (warp == 1 && elect_one()) {
      for (int h = 0; h < 2; ++h)
        tma_store_3d(&mapY, smem + SM::Y + h * ATOM, 0, 0, (int)(2 * at_slice + h));
      bulk_commit();
    }
    if (cg == 0 && row < id.n) a.bpart[id.slice * a.tokens + id.tok + row] = row_total(red, row);
  };
  work();
  cta_end(bars, ph, loads, tmem, TM_COLS, warp);
}

// ------------------------------------------------------------------ keys
// One CTA an SM, by its shared memory; bound by the latency of its four rounds
// of products: 2048 chunks of heads of 64 211 us (188 without the pairs' part of dg,
// of which only what the last round does not hide counts, and without the third
// planes of U and Mq).
struct KeysArgs {
  const __nv_bfloat16 *g, *beta;
  __nv_bfloat16 *dq, *dk;
  float *rpart, *wpart;    // [D / 64][BH N]
  float* cpart;            // [D / 64][BH N]: sum_{i >= t > j} V_ij; nullable: dg not wanted
  float* xpart;            // [D / 64][BH nch]: <X1, S0>
  float* bkey;             // [BH N]
  int N, nch;
  size_t tokens, chunks;
  float scale;
  DevStatus st;
};

template <int D>
struct KeysSmem {
  static constexpr int DA = D / 64;
  static constexpr uint32_t HA = 64 * 128;                    // a [64][64] atom
  // for the first products: dO; S0 and X1, hi and lo (rows of this slice); U, three
  // planes; Y, whose hi plane comes into dO's place where D = 128
  static constexpr uint32_t DO = 0, YHI = D == 64 ? ATOM : 0, S = 2 * ATOM, X = 4 * ATOM, UR = 6 * ATOM;
  static constexpr uint32_t U = 8 * ATOM, YLO = 12 * ATOM;
  // behind them: K, Q (this slice), sums; Mq, three planes, and Mk, hi and lo
  // (heads of 64 have room for K and Q beside the first operands; but loaded with
  // those, they hold up the first products: 694 us against 688 for the gradients of
  // 2048 chunks)
  static constexpr uint32_t K = 0, Q = 12 * ATOM, RED = 13 * ATOM;
  static constexpr uint32_t MQ = 4 * ATOM, MQR = 2 * ATOM, MK = 8 * ATOM;
  static constexpr uint32_t GATES = 14 * ATOM, XS = GATES + sizeof(Gates), BAR = XS + 64, TOTAL = BAR + 80;
};

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    delta_keys_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                      const __grid_constant__ CUtensorMap mapD, const __grid_constant__ CUtensorMap mapU,
                      const __grid_constant__ CUtensorMap mapY, const __grid_constant__ CUtensorMap mapS,
                      const __grid_constant__ CUtensorMap mapX, KeysArgs a) {
  using SM = KeysSmem<D>;
  constexpr int DA = D / 64;
  constexpr uint32_t TM_P = 0, TM_A = 128, TM_QS = 256, TM_YS = 320, TM_UX = 384, TM_KW = 448, TM_COLS = 512;
  constexpr uint32_t TM_QK = TM_A, TM_KR = TM_A + 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + SM::BAR);
  Gates& gates = *reinterpret_cast<Gates*>(smem + SM::GATES);
  float *red = reinterpret_cast<float*>(smem + SM::RED), *xs = reinterpret_cast<float*>(smem + SM::XS);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const ChunkId id(blockIdx.x, DA, Slab{0, a.nch, 0}, a.N);
  const uint32_t sb = smem_u32(smem);
  const uint32_t tmem = cta_begin(bars, TM_COLS, warp, [&]() {
    // what the first products read, then the others' operands
    mbar_arrive_expect_tx(&bars.load[0], 4 * DA * ATOM + 2 * DA * SM::HA);
    for (int i = 0; i < DA; ++i) {
      tma_load_3d(smem + SM::DO + i * ATOM, &mapD, &bars.load[0], 64 * i, id.t0, (int)id.bh);
      for (int h = 0; h < 3; ++h)
        tma_load_3d(smem + (h < 2 ? SM::U + 2 * h * ATOM : SM::UR) + i * ATOM, &mapU, &bars.load[0], 0, 0,
                    (int)(3 * (id.ci * DA + i)) + h);
      for (int h = 0; h < 2; ++h)
        tma_load_3d(smem + SM::S + (h * DA + i) * SM::HA, &mapS, &bars.load[0], 64 * i, 64 * id.slice, (int)(2 * id.ci + h));
    }
    mbar_arrive_expect_tx(&bars.load[3], (D == 64 ? 2 : 1) * DA * ATOM + 2 * DA * SM::HA);
    for (int i = 0; i < DA; ++i) {
      const int zs = (int)(2 * (id.ci * DA + i));
      tma_load_3d(smem + SM::YLO + i * ATOM, &mapY, &bars.load[3], 0, 0, zs + 1);
      for (int h = 0; h < 2; ++h)
        tma_load_3d(smem + SM::X + (h * DA + i) * SM::HA, &mapX, &bars.load[3], 64 * i, 64 * id.slice, (int)(2 * id.ci + h));
      if (D == 64) tma_load_3d(smem + SM::YHI, &mapY, &bars.load[3], 0, 0, zs);
    }
  });
  Phase ph{Waiter{&bars.abort, a.st, 1500}, &bars.mma, 0};
  const int q4 = warp & 3, cg = warp >> 2, row = q4 * 32 + lane;
  const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
  if (cg == 1) load_gates(gates, a.g ? a.g + id.tok : nullptr, a.beta + id.tok, id.n, row);
  int loads = D == 64 ? 9 : 13;
  auto work = [&]() {
    if (warp == 0) {
      bool ok = ph.W.wait_warp(&bars.load[0], 0, 1);
      const Op dO{sb + SM::DO, ATOM, false}, Ylo{sb + SM::YLO, ATOM, false}, Yhi{sb + SM::YHI, ATOM, false};
      const Pair U{{sb + SM::U, ATOM, false}, 2 * ATOM};
      const Pair S{{sb + SM::S, SM::HA, false}, DA * SM::HA}, X{{sb + SM::X, SM::HA, false}, DA * SM::HA};
      auto prod = [&](uint32_t d, const Op& x, const Op& y, int N, bool add) { return Prod(tmem + d, x, y, 128, N, add); };
      if (ok && elect_one()) {
        // those of dO first: its place is free for Y's hi plane while the others run
        products<D / 16>(prod(TM_P, dO, Op{sb + SM::UR, ATOM, false}, 128, false), prod(TM_QS, dO, S.lo(), 64, false));
        products<D / 16>(prod(TM_P, dO, U.lo(), 128, true), prod(TM_QS, dO, S.hi, 64, true));
        products<D / 16>(prod(TM_P, dO, U.hi, 128, true));
        if (D == 128) mma_commit(&bars.half);
      }
      __syncwarp();
      ok = ok && ph.W.wait_warp(&bars.load[3], 0, 9);
      if (ok && elect_one()) {
        products<D / 16>(prod(TM_A, Ylo, U.lo(), 128, false), prod(TM_YS, Ylo, S.hi, 64, false),
                         prod(TM_UX, U.lo(), X.lo(), 64, false));
        products<D / 16>(prod(TM_A, Ylo, U.hi, 128, true), prod(TM_UX, U.lo(), X.hi, 64, true));
        products<D / 16>(prod(TM_UX, U.hi, X.lo(), 64, true));
        products<D / 16>(prod(TM_UX, U.hi, X.hi, 64, true));
      }
      __syncwarp();
      if (D == 128) ok = ok && ph.W.wait_warp(&bars.load[2], 0, 7);
      if (ok && elect_one()) {
        products<D / 16>(prod(TM_A, Yhi, U.lo(), 128, true), prod(TM_YS, Yhi, S.lo(), 64, true));
        products<D / 16>(prod(TM_A, Yhi, U.hi, 128, true), prod(TM_YS, Yhi, S.hi, 64, true));
        mma_commit(&bars.mma);
      }
      __syncwarp();
    }
    if (ph.W.wait_warp(&bars.load[0], 0, 1) && ph.W.wait_warp(&bars.load[3], 0, 9)) {   // <X1, S0> of this slice's rows, while they are still here
      float acc = 0.f;
      for (int e = tid; e < 64 * D / 8; e += THREADS) {
        const int r = e / (D / 8), c = e % (D / 8) * 8;
        const uint32_t at = (uint32_t)(c >> 6) * SM::HA;
        float s[8], x[8];
        load8_split(sb + SM::S + at, sb + SM::S + DA * SM::HA + at, r, c & 63, s);
        load8_split(sb + SM::X + at, sb + SM::X + DA * SM::HA + at, r, c & 63, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = fmaf(s[i], x[i], acc);
      }
      for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
      if (lane == 0) xs[warp] = acc;
    }
    if (D == 128 && warp == 2) {
      if (ph.W.wait_warp(&bars.half, 0, 8) && elect_one()) {
        mbar_arrive_expect_tx(&bars.load[2], DA * ATOM);
        for (int i = 0; i < DA; ++i)
          tma_load_3d(smem + SM::YHI + i * ATOM, &mapY, &bars.load[2], 0, 0, (int)(2 * (id.ci * DA + i)));
      }
      __syncwarp();
    }
    if (!ph.mma_done(2)) return;
    if (warp == 2 && elect_one()) {   // K and Q take the places of dO and Y
      mbar_arrive_expect_tx(&bars.load[1], (DA + 1) * ATOM);
      for (int i = 0; i < DA; ++i)
        tma_load_3d(smem + SM::K + i * ATOM, &mapK, &bars.load[1], 64 * i, id.t0, (int)id.bh);
      tma_load_3d(smem + SM::Q, &mapQ, &bars.load[1], 64 * id.slice, id.t0, (int)id.bh);
    }
    if (tid == 96) {
      float acc = 0.f;
      for (int w = 0; w < THREADS / 32; ++w) acc += xs[w];
      a.xpart[id.slice * a.chunks + id.ci] = acc;
    }
    loads |= 2;
    // Mq in three planes (two would be 2.5e-6 of dQ and dK)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int c0 = cg * 32 + b * 16;
      float x[16];
      if (c0 <= q4 * 32 + 31) {
        tmem_ld16(tmem + lanes + TM_P + c0, x);
        weigh16<true>(gates, q4 * 32, row, c0, a.scale, x);
      } else {
        zero16(x);
      }
      store16_square3(sb + SM::MQ, sb + SM::MQR, row, c0, x);
    }
    ph.publish();
    const Op K{sb + SM::K, ATOM, false};
    if (warp == 0 && ph.W.wait_warp(&bars.load[1], 0, 3) && elect_one()) {
      products<D / 16>(Prod(tmem + TM_P, K, K, 128, 128, false));
      mma_commit(&bars.mma);
    }
    if (!ph.mma_done(4)) return;
    // Mk, and its row sums against k_i . k_j without beta; v: those terms
    float db = 0.f, v[32];
    const float beta = gates.beta[row];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int c0 = cg * 32 + b * 16;
      float x[16];
      if (c0 <= q4 * 32 + 31) {
        float kk[16];
        tmem_ld16(tmem + lanes + TM_A + c0, x);
        tmem_ld16(tmem + lanes + TM_P + c0, kk);
        weigh16<false>(gates, q4 * 32, row, c0, -1.f, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          v[16 * b + j] = c0 + j < row ? x[j] * kk[j] : 0.f;
          db += v[16 * b + j];
          x[j] *= beta;
        }
      } else {
        zero16(x);
        zero16(v + 16 * b);
      }
      store16_square(sb + SM::MK, row, c0, x);
    }
    red[cg * C + row] = db;
    ph.publish();
    const Op Kmn{sb + SM::K + id.slice * ATOM, ATOM, true}, Qmn{sb + SM::Q, ATOM, true};
    // (by a warp whose pairs all lie above the diagonal: issuing takes as long as
    // the products, and the other warps' sums go on meanwhile)
    constexpr int ISSUER = 4;
    if (warp == ISSUER && elect_one()) {
      const Pair Mq{{sb + SM::MQ, ATOM, false}, 2 * ATOM}, Mk{{sb + SM::MK, ATOM, false}, 2 * ATOM};
      const Pair Mqt{{sb + SM::MQ, ATOM, true}, 2 * ATOM}, Mkt{{sb + SM::MK, ATOM, true}, 2 * ATOM};
      if (a.cpart != nullptr) {   // q_i . k_j over this slice's columns, first: it is waited for alone
        products<4>(Prod(tmem + TM_P, Op{sb + SM::Q, ATOM, false}, Op{sb + SM::K + id.slice * ATOM, ATOM, false}, 128,
                         128, false));
        mma_commit(&bars.aux);
      }
      products<8>(Prod(tmem + TM_QK, Op{sb + SM::MQR, ATOM, false}, Kmn, 128, 64, false),
                  Prod(tmem + TM_KW, Op{sb + SM::MQR, ATOM, true}, Qmn, 128, 64, false));
      products<8>(Prod(tmem + TM_QK, Mq.lo(), Kmn, 128, 64, true), Prod(tmem + TM_KR, Mk.lo(), Kmn, 128, 64, false),
                  Prod(tmem + TM_KW, Mqt.lo(), Qmn, 128, 64, true));
      products<8>(Prod(tmem + TM_KW, Mkt.lo(), Kmn, 128, 64, true));
      products<8>(Prod(tmem + TM_QK, Mq.hi, Kmn, 128, 64, true), Prod(tmem + TM_KR, Mk.hi, Kmn, 128, 64, true),
                  Prod(tmem + TM_KW, Mqt.hi, Qmn, 128, 64, true));
      products<8>(Prod(tmem + TM_KW, Mkt.hi, Kmn, 128, 64, true));
      mma_commit(&bars.mma);
    }
    if (cg == 0 && id.slice == 0 && row < id.n) a.bkey[id.tok + row] = row_total(red, row);
    // c_t = sum_{i >= t > j} V_ij while the other products run: the sums over j < t
    // of a row, then over the rows from t on
    float *vsum = red + 8 * C, *csum = red + 12 * C;   // [column group][row], [32 rows][column]
    bool ok = true;
    if (a.cpart != nullptr && cg > q4) {
      csum[q4 * C + cg * 32 + lane] = 0.f;
    } else if (a.cpart != nullptr) {
      ok = ph.W.wait_warp(&bars.aux, 0, 6);
      tc_fence_after();
      const float fk = id.slice == 0 ? beta : 0.f;   // k_i . k_j is whole in every slice
      float total = 0.f;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int c0 = cg * 32 + b * 16;
        float qk[16], mq[16];
        tmem_ld16(tmem + lanes + TM_P + c0, qk);
        const uint32_t at = sb + SM::MQ + (uint32_t)(c0 >> 6) * ATOM;
        load8_split(at, at + 2 * ATOM, row, c0 & 63, mq);
        load8_split(at, at + 2 * ATOM, row, (c0 & 63) + 8, mq + 8);
        float rest[16];
        const uint32_t rat = sb + SM::MQR + (uint32_t)(c0 >> 6) * ATOM;
        load8(rat, row, c0 & 63, rest);
        load8(rat, row, (c0 & 63) + 8, rest + 8);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float& x = v[16 * b + j];
          x = c0 + j < row ? fmaf(mq[j] + rest[j], qk[j], fk * x) : 0.f;
          total += x;
        }
      }
      vsum[cg * C + row] = total;
      named_bar_sync(3, 10 * 32);   // the warps on and below the diagonal
      float below = 0.f;
      for (int g = 0; g < cg; ++g) below += vsum[g * C + row];
#pragma unroll
      for (int j = 0; j < 32; ++j) {   // t = 32 cg + j
        const float x = v[j];
        v[j] = row >= cg * 32 + j ? below : 0.f;
        below += x;
      }
      // 32 sums over 32 lanes, halving the values a lane holds: column j ends in lane j
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int j = 0; j < o; ++j)
          v[j] = ((lane & o) ? v[j + o] : v[j]) + __shfl_xor_sync(0xffffffffu, (lane & o) ? v[j] : v[j + o], o);
      csum[q4 * C + cg * 32 + lane] = v[0];
    }
    if (!ph.mma_done(5, ok)) {
      if (warp == ISSUER && elect_one()) {   // nothing in flight outlives the CTA (cta_end knows warp 0's)
        mma_commit(&bars.fin);
        ph.W.drain(&bars.fin, 0);
      }
      return;
    }
    const float gam = gate_decay(gates, row), rho = gate_ratio(gates, C - 1, row);
    const float fq = a.scale * gam, fy = -gam * beta;
    const int c = cg * 16;
    const size_t at = (id.tok + row) * D + id.slice * 64 + c;
    float rs = 0.f, ws = 0.f;
    float x[16], y[16], z[16], t[16];
    // dq
    tmem_ld16(tmem + lanes + TM_QS + c, x);
    tmem_ld16(tmem + lanes + TM_QK + c, y);
    load8(sb + SM::Q, row, c, t);
    load8(sb + SM::Q, row, c + 8, t + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] *= fq;
      rs = fmaf(t[i], x[i], rs);
      x[i] += y[i];
    }
    if (row < id.n) store_bf16_row16(a.dq + at, x);
    // dk: the state's part of the first for rs, third for ws
    load8(sb + SM::K + id.slice * ATOM, row, c, t);
    load8(sb + SM::K + id.slice * ATOM, row, c + 8, t + 8);
    tmem_ld16(tmem + lanes + TM_KR + c, x);
    tmem_ld16(tmem + lanes + TM_YS + c, y);
    tmem_ld16(tmem + lanes + TM_KW + c, z);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      y[i] *= fy;
      rs = fmaf(t[i], y[i], rs);
      x[i] += y[i] + z[i];
    }
    tmem_ld16(tmem + lanes + TM_UX + c, y);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float w = rho * y[i];
      ws = fmaf(t[i], w, ws);
      x[i] += w;
    }
    if (row < id.n) store_bf16_row16(a.dk + at, x);
    float* wred = red + 4 * C;
    red[cg * C + row] = rs;
    wred[cg * C + row] = ws;
    __syncthreads();
    if (cg == 0 && row < id.n) {
      const size_t o = id.slice * a.tokens + id.tok + row;
      a.rpart[o] = row_total(red, row);
      a.wpart[o] = row_total(wred, row);
      if (a.cpart != nullptr) a.cpart[o] = row_total(csum, row);
    }
  };
  work();
  cta_end(bars, ph, loads, tmem, TM_COLS, warp);
}

// ------------------------------------------------------------------ gates
struct GateArgs {
  const float *gend, *rpart, *wpart, *cpart, *xpart, *bpart, *bkey;
  __nv_bfloat16 *dg, *dbeta;   // dg nullable
  int N, nch, slices;
  size_t tokens, chunks;
};

TTT_DEVICE_INLINE float sum_below(float x, float* buf, int tid, float& total) {   // over threads 0..tid-1 of 128
  float pre = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_up_sync(0xffffffffu, pre, o);
    if ((tid & 31) >= o) pre += y;
  }
  if ((tid & 31) == 31) buf[tid >> 5] = pre;
  __syncthreads();
  float base = 0.f;
  total = 0.f;
#pragma unroll
  for (int w = 0; w < C / 32; ++w) {
    if (w < tid >> 5) base += buf[w];
    total += buf[w];
  }
  __syncthreads();
  // the shifted lane, not pre - x: that would cancel
  const float y = __shfl_up_sync(0xffffffffu, pre, 1);
  return base + ((tid & 31) ? y : 0.f);
}

__global__ void __launch_bounds__(C) delta_gate_grad_kernel(GateArgs a) {
  __shared__ float buf[C / 32];
  const int tid = threadIdx.x;
  const size_t ci = blockIdx.x, bh = ci / a.nch;
  const int t0 = (int)(ci % a.nch) * C, n = min(C, a.N - t0);
  const size_t tok = bh * a.N + t0;
  const bool live = tid < n;
  pdl_wait();
  pdl_launch_dependents();
  float r = 0.f, w = 0.f, c = 0.f, b = 0.f, x = 0.f;
  for (int s = 0; s < a.slices; ++s) {
    const size_t at = s * a.tokens + tok + tid;
    if (live) {
      r += a.rpart[at];
      w += a.wpart[at];
      if (a.dg != nullptr) c += a.cpart[at];
      b += a.bpart[at];
    }
    x += a.xpart[s * a.chunks + ci];
  }
  if (live) a.dbeta[tok + tid] = __float2bfloat16_rn(b + a.bkey[tok + tid]);
  if (a.dg == nullptr) return;
  // the sum over i >= t is a prefix sum of the reversed order
  __shared__ float rev[C];
  rev[C - 1 - tid] = r;
  __syncthreads();
  float total, wt;
  const float below = sum_below(rev[tid], buf, tid, total) + rev[tid];
  const float wpre = sum_below(w, buf, tid, wt);
  rev[tid] = below;   // every thread has read its own entry
  __syncthreads();
  if (live) a.dg[tok + tid] = __float2bfloat16_rn((rev[C - 1 - tid] + c) + fmaf(a.gend[ci], x, wpre));
}

template <int D>
int bwd_launch(const DeltaBwdLaunch& L, cudaStream_t stream) {
  const DeltaLaunch& p = L.f;
  const int BH = p.B * p.H, nch = tiles_of(p.N, C);
  constexpr int DA = D / 64;
  const DeltaUmmaBwdWorkspace w = delta_umma_bwd_layout(BH, p.N, D);
  const uint64_t nc = (uint64_t)BH * nch, rs = D * 2;
  const size_t tokens = (size_t)BH * p.N;
  uint8_t* ws = delta_ws_base(L.ws);
  auto bf = [&](size_t at) { return reinterpret_cast<__nv_bfloat16*>(ws + at); };
  auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
  const __nv_bfloat16 *g = (const __nv_bfloat16*)p.g, *beta = (const __nv_bfloat16*)p.beta;
  const DeltaPrepOut o{f32(w.gend), f32(w.H), f32(w.Ut), bf(w.W), bf(w.M), bf(w.T)};
  const DeltaChain fwd{o.H, L.S0, nullptr, bf(w.X)}, rev{f32(w.Hb), L.dS_end, L.dS0, bf(w.X1)};
  CUtensorMap mq, mk, md, mw, mu, my, mt, ms, mx, ms64, mx64;
  if (make_tmap_bf16_3d(&mq, p.q, D, p.N, BH, rs, p.N * rs, 64, C) ||
      make_tmap_bf16_3d(&mk, p.k, D, p.N, BH, rs, p.N * rs, 64, C) ||
      make_tmap_bf16_3d(&md, L.dout, D, p.N, BH, rs, p.N * rs, 64, C) ||
      make_tmap_bf16_3d(&mw, o.W, D, C, 2 * nc, rs, C * rs, 64, C) ||
      make_tmap_bf16_3d(&mu, ws + w.U, 64, C, 3 * DA * nc, 128, ATOM, 64, C) ||   // [BH nch][D / 64][three planes][128][64]
      make_tmap_bf16_3d(&my, ws + w.Y, 64, C, 2 * DA * nc, 128, ATOM, 64, C) ||   // [BH nch][D / 64][hi, lo][128][64]
      make_tmap_bf16_3d(&mt, o.T, C, C, 2 * nc, 2 * C, 2 * C * C, 64, C) ||
      make_tmap_bf16_3d(&ms, fwd.X, D, D, 2 * nc, rs, D * rs, 64, D) ||
      make_tmap_bf16_3d(&mx, rev.X, D, D, 2 * nc, rs, D * rs, 64, D) ||
      make_tmap_bf16_3d(&ms64, fwd.X, D, D, 2 * nc, rs, D * rs, 64, 64) ||
      make_tmap_bf16_3d(&mx64, rev.X, D, D, 2 * nc, rs, D * rs, 64, 64))
    return -1;
  static std::atomic<uint64_t> a0{0}, a1{0}, a2{0};
  if (allow_dynamic_smem(delta_hb_kernel<D>, (int)HbSmem<D>::TOTAL, a0) ||
      allow_dynamic_smem(delta_vals_kernel<D>, (int)ValsSmem<D>::TOTAL, a1) ||
      allow_dynamic_smem(delta_keys_kernel<D>, (int)KeysSmem<D>::TOTAL, a2))
    return -1;
  if (launch_delta_prep(p, o, stream)) return -1;
  const unsigned grid = (unsigned)(nc * DA);
  prof_before(K_DELTA_HB, stream);
  const cudaError_t e_hb = launch_pdl(
      delta_hb_kernel<D>, dim3(grid), dim3(THREADS), HbSmem<D>::TOTAL, stream,
      mq, mk, md, mw, HbArgs{g, beta, f32(w.Hb), f32(w.Y), p.N, nch, p.scale, p.st});
  prof_after(K_DELTA_HB, stream);
  if (launch_delta_chain(p, o.gend, o.M, fwd, rev, stream)) return -1;
  prof_before(K_DELTA_VALS, stream);
  const cudaError_t e_vals = launch_pdl(
      delta_vals_kernel<D>, dim3(grid), dim3(THREADS), ValsSmem<D>::TOTAL, stream,
      mk, mw, mu, my, mt, ms, mx,
      ValsArgs{g, beta, (const __nv_bfloat16*)p.v, o.U, f32(w.Y), (__nv_bfloat16*)L.dv, f32(w.bpart), p.N, nch, tokens, p.st});
  prof_after(K_DELTA_VALS, stream);
  prof_before(K_DELTA_KEYS, stream);
  const cudaError_t e_keys = launch_pdl(
      delta_keys_kernel<D>, dim3(grid), dim3(THREADS), KeysSmem<D>::TOTAL, stream,
      mq, mk, md, mu, my, ms64, mx64,
      KeysArgs{g, beta, (__nv_bfloat16*)L.dq, (__nv_bfloat16*)L.dk, f32(w.rpart), f32(w.wpart),
               L.dg != nullptr ? f32(w.cpart) : nullptr, f32(w.xpart), f32(w.bkey), p.N, nch, tokens, nc, p.scale, p.st});
  prof_after(K_DELTA_KEYS, stream);
  prof_before(K_DELTA_GATES, stream);
  const cudaError_t e_gates = launch_pdl(
      delta_gate_grad_kernel, dim3((unsigned)nc), dim3(C), 0, stream,
      GateArgs{o.gend, f32(w.rpart), f32(w.wpart), f32(w.cpart), f32(w.xpart), f32(w.bpart), f32(w.bkey),
               (__nv_bfloat16*)L.dg, (__nv_bfloat16*)L.dbeta, p.N, nch, DA, tokens, nc});
  prof_after(K_DELTA_GATES, stream);
  const bool ok = e_hb == cudaSuccess && e_vals == cudaSuccess && e_keys == cudaSuccess && e_gates == cudaSuccess;
  return ok ? 0 : -1;
}

}  // namespace

DeltaUmmaBwdWorkspace delta_umma_bwd_layout(int BH, int N, int D) {
  DeltaUmmaBwdWorkspace w{};
  const size_t nc = (size_t)BH * tiles_of(N, C), tokens = (size_t)BH * N, DA = D / 64;
  size_t at = 512;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t tile = nc * 2 * C * D * 2, mat = nc * 4 * D * D;
  w.gend = take(nc * 4);
  w.W = take(tile);
  w.U = take(tile / 2 * 3);
  w.Ut = take(tile);
  w.Y = take(tile);
  w.T = take(nc * 2 * C * C * 2);
  w.M = take(mat);
  w.H = take(mat);
  w.Hb = take(mat);
  w.X = take(mat);
  w.X1 = take(mat);
  w.rpart = take(DA * tokens * 4);
  w.wpart = take(DA * tokens * 4);
  w.cpart = take(DA * tokens * 4);
  w.bpart = take(DA * tokens * 4);
  w.bkey = take(tokens * 4);
  w.xpart = take(DA * nc * 4);
  w.total = at;
  return w;
}

int launch_delta_umma_bwd(const DeltaBwdLaunch& L, cudaStream_t stream) {
  return L.f.dk == 64 ? bwd_launch<64>(L, stream) : bwd_launch<128>(L, stream);
}

}  // namespace ttt
