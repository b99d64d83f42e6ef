// delta_umma.cuh -- shared pieces of the tensor-core kernels of the gated
// delta rule (bf16, dk = dv = 64 or 128, chunks of 128 tokens).
//
// Tiles: [rows][64] bf16 with 128-byte rows and 128-byte swizzle ("atoms");
// a 128-row atom is 16 KB.  A derived matrix is a pair of atoms rows, hi =
// bf16(x) and lo = bf16(x - hi): off by at most 2^-18 of the value, where one
// bf16 alone would be off by 2^-9 and show in the float32 state.  Three products
// join two pairs (lo lo, at most 2^-18, is left out).  What would be most of a
// result's error is carried in three planes, errors by their norm: H and Hb, which S
// and dS0 consist of where the state decays (off by 5e-7 and 1e-6; 2.7e-6 and 3e-6
// with two planes); P and U of the outputs (9e-7; 4.7e-6); dU, U and Mq of the
// gradients (1e-6 to 1.5e-6 before they are rounded to bf16; 4e-6).  Without decay
// the two planes of T, W, M and X leave 4.4e-6 of S, where float32 operands would
// leave 5e-7: three planes of all four would take twice the products and half as
// much memory again, three of any of them leave 1.2e-6 or more.
#pragma once

#include "kernels.h"

namespace ttt {
namespace dl {

constexpr int C = 128;                  // tokens of a chunk
constexpr uint32_t ATOM = C * 128;      // bytes of a 128-row atom

// ----------------------------------------------------------------- gates
// Running sum G of the log decays of a chunk, as hi + lo: hi sums multiples of
// 2^-9 that float32 holds exactly (|G| <= 128 * 200 < 2^15), lo the rests
// (below 2^-10 each), so a difference of two sums keeps the precision of its
// own size and not that of G.  A single log decay is held to +-200 (exp(-200)
// is 0 in float32), which keeps G finite where a state is cleared; NaN stays.
struct Gates {
  float hi[C], lo[C], beta[C];
  float down[C];           // exp(G_e - G_j), e the last token of j's block of 16
  float part[8];
};
// Off by (2 + 1.16 |d|) 2^-23 of exp(d) at most, so for d <= 0 by 2^-22 = 2.4e-7 of
// the largest factor 1.  With expf S comes out 2 % nearer to 64 bits (5.0e-7 of
// its norm in the place of 5.1e-7, 1024 tokens of heads of 64) and the calls take 5
// to 9 % longer (64 heads of 64, 32K tokens: 1742 us against 1652).
TTT_DEVICE_INLINE float gate_exp(float d) { return __expf(d); }
TTT_DEVICE_INLINE float gate_clamp(float g) { return g < -200.f ? -200.f : g > 200.f ? 200.f : g; }

// By the 128 threads t = 0..127 of four whole warps (barrier 2); tokens behind
// n have beta = 0 and no decay.  gam = exp(G_t), rho = exp(G_last - G_t).
TTT_DEVICE_INLINE void load_gates(Gates& s, const __nv_bfloat16* g, const __nv_bfloat16* beta, int n, int t,
                                  float& gam, float& rho) {
  const int lane = t & 31, w = t >> 5, at = min(t, n - 1);
  const __nv_bfloat16 bv = beta[at];
  float x = g != nullptr ? gate_clamp(__bfloat162float(g[at])) : 0.f;
  if (t >= n) x = 0.f;
  float hi = rintf(x * 512.f) * (1.f / 512.f), lo = x - hi;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float h = __shfl_up_sync(0xffffffffu, hi, o), l = __shfl_up_sync(0xffffffffu, lo, o);
    if (lane >= o) { hi += h; lo += l; }
  }
  if (lane == 31) { s.part[w] = hi; s.part[4 + w] = lo; }
  named_bar_sync(2, C);
  float hl = 0.f, ll = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i == w) { hi += hl; lo += ll; }
    hl += s.part[i];
    ll += s.part[4 + i];
  }
  const float he = __shfl_sync(0xffffffffu, hi, lane | 15), le = __shfl_sync(0xffffffffu, lo, lane | 15);
  s.hi[t] = hi;
  s.lo[t] = lo;
  s.beta[t] = t < n ? __bfloat162float(bv) : 0.f;
  s.down[t] = gate_exp((he - hi) + (le - lo));
  gam = gate_exp(hi + lo);
  rho = gate_exp((hl - hi) + (ll - lo));
}
TTT_DEVICE_INLINE void load_gates(Gates& s, const __nv_bfloat16* g, const __nv_bfloat16* beta, int n, int t) {
  float gam, rho;
  load_gates(s, g, beta, n, t, gam, rho);
}
// exp(G_i - G_j)
TTT_DEVICE_INLINE float gate_ratio(const Gates& s, int i, int j) {
  return gate_exp((s.hi[i] - s.hi[j]) + (s.lo[i] - s.lo[j]));
}
TTT_DEVICE_INLINE float gate_decay(const Gates& s, int i) { return gate_exp(s.hi[i] + s.lo[i]); }

// x_j <- f Gam_ij x_j of 16 columns of a row, lower triangle with the diagonal
// or without.  `warp_row` is the first row of the warp (uniform branch): blocks
// below all of its rows take one exponential, exp(G_i - G_e) exp(G_e - G_j) with
// e the block's last token, the others one an element.
template <bool DIAG>
TTT_DEVICE_INLINE void weigh16(const Gates& s, int warp_row, int row, int c0, float f, float* x) {
  if (c0 < warp_row) {
    const float a = f * gate_ratio(s, row, c0 + 15);
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const float4 d = *reinterpret_cast<const float4*>(s.down + c0 + j);
      x[j] *= a * d.x; x[j + 1] *= a * d.y; x[j + 2] *= a * d.z; x[j + 3] *= a * d.w;
    }
  } else {
    const float gh = s.hi[row], gl = s.lo[row];
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const float4 h = *reinterpret_cast<const float4*>(s.hi + c0 + j);
      const float4 l = *reinterpret_cast<const float4*>(s.lo + c0 + j);
      const float d[4] = {(gh - h.x) + (gl - l.x), (gh - h.y) + (gl - l.y), (gh - h.z) + (gl - l.z),
                          (gh - h.w) + (gl - l.w)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + j + i;
        x[j + i] = (DIAG ? c <= row : c < row) ? f * x[j + i] * gate_exp(d[i]) : 0.f;
      }
    }
  }
}

// ----------------------------------------------------------------- hi + lo
TTT_DEVICE_INLINE void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  lo = pack_bf16x2(a - bf16lo(hi), b - bf16hi(hi));
}
// 8 columns (col a multiple of 8) of a row of two atoms
TTT_DEVICE_INLINE void store8_split(uint32_t hi_atom, uint32_t lo_atom, int row, int col, const float* x) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2(x[2 * i], x[2 * i + 1], h[i], l[i]);
  const uint32_t o = sw128_offset(row, col);
  st_shared_v4(hi_atom + o, h[0], h[1], h[2], h[3]);
  st_shared_v4(lo_atom + o, l[0], l[1], l[2], l[3]);
}
TTT_DEVICE_INLINE void load8(uint32_t atom, int row, int col, float* x) {
  uint32_t w[4];
  ld_shared_v4(atom + sw128_offset(row, col), w[0], w[1], w[2], w[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) { x[2 * i] = bf16lo(w[i]); x[2 * i + 1] = bf16hi(w[i]); }
}
TTT_DEVICE_INLINE void load8_split(uint32_t hi_atom, uint32_t lo_atom, int row, int col, float* x) {
  float l[8];
  load8(hi_atom, row, col, x);
  load8(lo_atom, row, col, l);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] += l[i];
}

// three planes: what is left of 24 bits after hi and lo
TTT_DEVICE_INLINE void store8_split3(uint32_t hi_atom, uint32_t lo_atom, uint32_t rest_atom, int row, int col,
                                     const float* x) {
  uint32_t h[4], l[4], r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    const float a = x[2 * i] - bf16lo(h[i]), b = x[2 * i + 1] - bf16hi(h[i]);
    split2(a, b, l[i], r[i]);
  }
  const uint32_t o = sw128_offset(row, col);
  st_shared_v4(hi_atom + o, h[0], h[1], h[2], h[3]);
  st_shared_v4(lo_atom + o, l[0], l[1], l[2], l[3]);
  st_shared_v4(rest_atom + o, r[0], r[1], r[2], r[3]);
}
// 16 columns of a row of the caller's (16-byte aligned) bf16 tensor
TTT_DEVICE_INLINE void store_bf16_row16(__nv_bfloat16* p, const float* x) {
  uint4* d = reinterpret_cast<uint4*>(p);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    d[i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                      pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
}
// 16 columns of a row as hi and lo rows of the workspace (32-byte aligned)
TTT_DEVICE_INLINE void store16_pair(__nv_bfloat16* hi, __nv_bfloat16* lo, const float* x) {
  uint32_t h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split2(x[2 * i], x[2 * i + 1], h[i], l[i]);
  st_global_v8(hi, h);
  st_global_v8(lo, l);
}

// ----------------------------------------------------------------- products
// Operands by shared address: K-major (rows are the M or N index, the 64
// columns of an atom are K; further atoms of K `astride` bytes on) or MN-major
// (rows are K, the columns M or N; further atoms of M or N `astride` on).
struct Op {
  uint32_t addr, astride;
  bool mn;
};
TTT_DEVICE_INLINE uint64_t op_desc(const Op& o) {
  return o.mn ? make_sdesc(o.addr, o.astride, 1024) : make_sdesc(o.addr, 16, 1024);
}
// D (+)= A B^T over K, 16 at a step, by one elected thread (see elect_one): one
// descriptor an operand, an addition a step.  A step of M = 128, N = 64 takes
// about 50 cycles, what its 6 KB of operands take to leave shared memory.
// products() takes a step of each of several products in turn.  The tensor core
// truncates its running sum, so small terms go first.
struct Prod {
  uint32_t d, id, a_stride, b_stride, ta;
  uint64_t da, db;
  bool add, a_mn, b_mn, ts;
  TTT_DEVICE_INLINE Prod(uint32_t d_, const Op& a, const Op& b, int M, int N, bool add_)
      : d(d_), id(make_idesc(M, N, a.mn, b.mn)), a_stride(a.astride), b_stride(b.astride), ta(0),
        da(op_desc(a)), db(op_desc(b)), add(add_), a_mn(a.mn), b_mn(b.mn), ts(false) {}
  // A in TMEM: lane = row, two bf16 of K to a column
  TTT_DEVICE_INLINE Prod(uint32_t d_, uint32_t a_tmem, const Op& b, int N, bool add_)
      : d(d_), id(make_idesc(128, N, false, b.mn)), a_stride(0), b_stride(b.astride), ta(a_tmem), da(0),
        db(op_desc(b)), add(add_), a_mn(false), b_mn(b.mn), ts(true) {}
  TTT_DEVICE_INLINE static uint32_t at(bool mn, uint32_t stride, int ks) {   // bytes to K step ks
    return mn ? ks * 2048 : (ks >> 2) * stride + (ks & 3) * 32;
  }
  TTT_DEVICE_INLINE void step(int ks) const {
    const uint32_t acc = add || ks > 0;
    const uint64_t b = sdesc_add(db, at(b_mn, b_stride, ks));
    if (ts) mma_bf16_ts(d, ta + 8 * ks, b, id, acc);
    else mma_bf16(d, sdesc_add(da, at(a_mn, a_stride, ks)), b, id, acc);
  }
};
template <int STEPS, typename... P>
TTT_DEVICE_INLINE void products(const P&... p) {
#pragma unroll
  for (int ks = 0; ks < STEPS; ++ks) (p.step(ks), ...);
}
// The hi + lo pair of an operand: lo is `second` bytes after hi.  A product of
// two pairs is lo hi + hi lo + hi hi (lo lo, at most 2^-18 of it, is left out).
struct Pair {
  Op hi;
  uint32_t second;
  TTT_DEVICE_INLINE Op lo() const { return plane(1); }
  TTT_DEVICE_INLINE Op plane(int i) const { return Op{hi.addr + i * second, hi.astride, hi.mn}; }
};

// ----------------------------------------------------------------- float32 tiles in global memory
// [rows][D] in 64-column slices, columns in groups of four: a row's 16 columns
// (c a multiple of 16) are four 16-byte accesses, each whole across the rows
// of a warp.
TTT_DEVICE_INLINE float* tile_at(float* p, int rows, int r, int c) {
  return p + (size_t)(c >> 6) * 64 * rows + ((size_t)((c & 63) >> 2) * rows + r) * 4;
}
TTT_DEVICE_INLINE void store_tile16(float* p, int rows, int r, int c, const float* x) {
  float* t = tile_at(p, rows, r, c);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4*>(t + (size_t)i * rows * 4) = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
TTT_DEVICE_INLINE void load_tile16(const float* p, int rows, int r, int c, float* x) {
  const float* t = tile_at(const_cast<float*>(p), rows, r, c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(t + (size_t)i * rows * 4);
    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
  }
}

// ----------------------------------------------------------------- phases
// A CTA that works in phases: every thread waits for the same barrier and
// learns whether all of them saw it complete; after a wait that ran out they
// leave together.
struct Phase {
  Waiter W;
  uint64_t* mma;       // completed by mma_commit, one phase per product group
  uint32_t parity;
  TTT_DEVICE_INLINE bool mma_done(uint32_t site, bool before = true) {   // before: this thread's waits so far
    const bool done = W.wait(mma, parity, site);
    const bool ok = __syncthreads_or(!done || !before) == 0;
    parity ^= 1;
    tc_fence_after();
    return ok;
  }
  // generic writes of this phase become visible to the tensor cores
  TTT_DEVICE_INLINE void publish() const {
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
};

// ----------------------------------------------------------------- CTA
// Chunks [c0, c0 + len) of every head; their buffers in the workspace are those
// from w0 on, head by head.
struct Slab {
  int c0, len;
  size_t w0;
};
// The chunk (and 64-column slice) of a CTA; ci counts in the workspace.
struct ChunkId {
  int slice, t0, n;
  size_t ci, bh, tok;
  TTT_DEVICE_INLINE ChunkId(unsigned block, int slices, const Slab& s, int N) {
    slice = block % slices;
    const unsigned r = block / slices;
    ci = s.w0 + r;
    bh = r / s.len;
    t0 = (s.c0 + (int)(r % s.len)) * C;
    n = min(C, N - t0);
    tok = bh * N + t0;
  }
};
struct Bars {
  uint64_t load[4], mma, aux, fin, half;   // aux, fin, half: of product groups waited for beside those of mma
  uint32_t tmem, abort;
};
static_assert(sizeof(Bars) <= 80, "the layouts leave 80 bytes");
// Barriers and `cols` TMEM columns, before the first phase; returns the TMEM
// base.  An elected thread of warp 0 issues the first loads (on load[0]) as
// soon as the barriers stand and the launch before this one is complete (every
// kernel here is launched to start while its predecessor drains, and waits
// before it touches global memory) (elected: an address that the whole warp knows
// costs a TMA instruction a few cycles, one in a thread's registers about 100).
template <typename F>
TTT_DEVICE_INLINE uint32_t cta_begin(Bars& b, uint32_t cols, int warp, F loads) {
  if (warp == 0 && elect_one()) {
    for (int i = 0; i < 4; ++i) mbar_init(&b.load[i], 1);
    mbar_init(&b.mma, 1);
    mbar_init(&b.aux, 1);
    mbar_init(&b.fin, 1);
    mbar_init(&b.half, 1);
    b.abort = 0;
    fence_barrier_init();
    pdl_wait();
    loads();
  }
  if (warp == 1) {
    tmem_alloc(&b.tmem, cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_launch_dependents();   // every CTA has its tensor memory by then
  return __shfl_sync(0xffffffffu, b.tmem, 0);
}
// After the last phase, or an aborted one: nothing in flight outlives the CTA.
// `loads` has a bit for each load barrier in use.  Warp 0's elected thread issues the
// products, warp 1's the stores: an election has one outcome, so the threads
// that wait here are the same ones.
TTT_DEVICE_INLINE void cta_end(Bars& b, const Phase& ph, int loads, uint32_t tmem, uint32_t cols, int warp) {
  if (warp == 0 && ph.W.aborted() && elect_one()) {
    for (int i = 0; i < 4; ++i)
      if (loads >> i & 1) ph.W.drain(&b.load[i], 0);
    mma_commit(&b.mma);
    ph.W.drain(&b.mma, 0);
    ph.W.drain(&b.mma, 1);
  }
  if (warp == 1 && elect_one()) bulk_wait_all();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, cols);
  }
}

}  // namespace dl

// ----------------------------------------------------------------- launches shared by both passes
// Offsets of the workspace layouts count from here: 256-byte aligned and less
// than 256 bytes before the caller's 16-byte aligned pointer, so offset 512 is
// behind its status block.
inline uint8_t* delta_ws_base(uint8_t* ws) {
  return reinterpret_cast<uint8_t*>(reinterpret_cast<uintptr_t>(ws) & ~uintptr_t(255));
}
struct DeltaPrepOut {       // device buffers, per chunk of all heads
  float *gend, *H, *U;              // U: Ut, float32 tiles
  __nv_bfloat16 *W, *M, *T;         // hi, lo; T nullable
};
struct DeltaChain {         // one direction of the state recurrence
  const float *H, *S_in;    // S_in nullable (zeros)
  float* S_out;             // nullable
  __nv_bfloat16* X;         // [BH nch][2][D][D] hi, lo: the state at every chunk's start (its end, backward)
};
// All chunks at once, each with buffers of its own.
int launch_delta_prep(const DeltaLaunch& p, const DeltaPrepOut& o, cudaStream_t stream);
// both directions side by side; rev: X <- exp(G_last) X + M^T X + H, from the last chunk
int launch_delta_chain(const DeltaLaunch& p, const float* gend, const __nv_bfloat16* M, const DeltaChain& fwd,
                       const DeltaChain& rev, cudaStream_t stream);
}  // namespace ttt
