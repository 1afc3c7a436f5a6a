// Gradients of the Mamba2 sequence scan with respect to B, C, dt and the
// head parameters, from the states before each block of 128 tokens and the
// gradients of the states after it (both written by the walks of
// gdn_m2scan.hip, which also give dx and the initial states' gradient).
//
// In a block, with c_i the prefix sums of the log-decays g in it, S the state
// before it, dS' the gradient after it, W_ij = dy_i.x_j, G_ij = C_i.B_j and
// L_ij = e^{c_i - c_j} (j <= i):
//     dC_i = sum_heads sum_{j<=i} L_ij dt'_j W_ij B_j  +  e^{c_i} S^T dy_i
//     dB_j = sum_heads sum_{i>=j} L_ij dt'_j W_ij C_i  +  dt'_j e^{c_last - c_j} dS'^T x_j
//     dg_t = sum_{j<t<=i} dt'_j L_ij W_ij G_ij + sum_{i>=t} e^{c_i} dy_i.(S C_i)
//            + sum_{j<t} dt'_j e^{c_last-c_j} x_j.(dS' B_j) + e^{c_last} <S, dS'>
//     ddt'_t = sum_{i>=t} L_it W_it G_it + e^{c_last-c_t} x_t.(dS' B_t) - exp(A_log) dg_t
// One workgroup takes a block and a group and goes over the group's heads, so
// the sums over heads stay in registers: the sum over heads of L dt' W (16
// rows a wave) and the state parts of dC and dB (16 columns n a wave).  The
// products with B and C follow once, after the last head.  dC's state part
// dotted with C_i is also dg's, and dB's with B_j.
//
// dg's first sum is taken without differences of larger sums: tiles of 16 x 16
// with a whole block of rows after t and of columns before t count whole, those
// that share t's rows or columns by sums from the far side, and inside the
// diagonal tile each row's sum of the columns before t counts where the row is
// not.  So where a step clears the state its dg is as small as the decay, and
// what stands behind it leaves nothing there.  Diagonal elements do not enter.
//
// A decay multiplies last and is the square of a root that the hardware's
// exponential does not flush, so that one close to the smallest numbers costs
// two roundings there.  The states are split in three bf16 terms (bf16 inputs), so all sums that end
// in dt's gradient and the head parameters' are FP32 sums of FP32 products.
// Parameter sums go through one partial row a block and are added in a fixed
// order, in 64 bits.
//
// Measured (bf16, heads of 64 x 128, 16 heads a group): 16,384 tokens x 128
// heads 806 us in a kernel trace, 2.7 GB read and 0.13 written, 3.5 TB/s.  One workgroup of eight
// waves fits a compute unit, as the summed products and C.B of a block lie in
// LDS; its parts (products of a head, the state parts, the sums that close a
// head) wait for memory and LDS in turn.  Matrix units are busy 13% of the time.
#include "gdn_m2scan.h"

namespace gdn {

template <bool BF, int D, int NN>
struct GradGeom {
  typedef typename Frag<BF>::E E;
  static constexpr int T = kGradBlock, NT = NN / 16;
  static constexpr int DK = D < 32 ? 32 : D, DB = DK / 32;
  static constexpr int LDX = DK + (BF ? 8 : 4);   // x and dy [128][LDX]
  static constexpr int LDN = T + (BF ? 8 : 4);    // the summed products [128][LDN], over x and dy after the last head
  static constexpr int ELEMS = 2 * T * LDX > T * LDN ? 2 * T * LDX : T * LDN;
  static constexpr bool BOTH = NT == 8;           // each wave has a column tile of dC and of dB; else one wave has one of them
  static constexpr bool G_LDS = BF || D < 128;    // C_i.B_j in LDS, in registers where that is full
  static constexpr bool N_LDS = BF;               // the heads' summed products too
  static constexpr bool LATE = BF && D < 128;     // a head's sums are closed while the next head is under way
  static constexpr int XV = T * DK / 8 / 512;     // vectors of 8 elements of x (and of dy) that a thread stages
  // a head's results: column sums [8][128], row sums in two parts, the diagonal tiles' part of dg and column sums, the diagonal, the state
  // parts [NT][128] twice, the waves' parts of <S, dS'> and of sum dy.x
  static constexpr int RES = (8 + 5 + 2 * NT) * T + 16;
  // a head's gates: c / 2 (two), e^{c_i}, dt' e^{c_last - c_j}, dt', exp(A_log), e^{c_last}; of the head under way, the one
  // before it, which is being closed, and the next
  static constexpr int GATES = 5 * T + 4, RING = LATE ? 3 : 1;
  static constexpr int TILES = 36 * 64 * 16;      // bytes of the tiles on and below the diagonal
  static_assert(!BF || 2 * T * LDN * 2 <= ELEMS * 2 + TILES, "both terms of the summed products fit over x, dy and C.B");
  static constexpr size_t LDS = (size_t)ELEMS * sizeof(E) + (G_LDS ? TILES : 0) + (N_LDS ? TILES : 0) + (RING * GATES + (LATE ? 2 : 1) * RES) * 4;
};

// Sums over a 16-lane row's lanes at or after, and at or before, each lane.
template <int CTRL>
__device__ __forceinline__ float row_shift(float x) {  // zero from outside the row
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_suffix(float x) {
  x += row_shift<0x101>(x);
  x += row_shift<0x102>(x);
  x += row_shift<0x104>(x);
  x += row_shift<0x108>(x);
  return x;
}
__device__ __forceinline__ float row_prefix(float x) {
  x += row_shift<0x111>(x);
  x += row_shift<0x112>(x);
  x += row_shift<0x114>(x);
  x += row_shift<0x118>(x);
  return x;
}

template <bool BF, int D, int NN>
__global__ void __launch_bounds__(512, 2) gdn_m2s_grad_kernel(const M2GradArgs a) {
  using W = GradGeom<BF, D, NN>;
  typedef typename W::E E;
  constexpr int T = W::T, NT = W::NT, LDX = W::LDX, LDN = W::LDN, DB = W::DB, Q = kScanChunk;
  constexpr bool BOTH = W::BOTH;
  extern __shared__ __align__(16) unsigned char smem[];
  E* const s_x = reinterpret_cast<E*>(smem);
  E* const s_y = s_x + T * LDX;
  E* const s_n = s_x;
  int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int tile0 = wave * (wave + 1) / 2 * 64 + lane;  // tile (i, j <= i) is the i (i + 1) / 2 + j-th, a lane's four values together
  f32x4* const s_gt = reinterpret_cast<f32x4*>(smem + (size_t)W::ELEMS * sizeof(E));
  f32x4* const s_ns = s_gt + (W::G_LDS ? 36 * 64 : 0);
  float* const s_gates = reinterpret_cast<float*>(smem + (size_t)W::ELEMS * sizeof(E) + (W::G_LDS ? W::TILES : 0) + (W::N_LDS ? W::TILES : 0));
  float* const s_res = s_gates + W::RING * W::GATES;

  const int hpg = a.H / a.G;
  const int slot = blockIdx.x / (a.G * a.splits), rest = blockIdx.x - slot * (a.G * a.splits), g = rest / a.splits, split = rest - g * a.splits;
  const int h_lo = (int)((int64_t)hpg * split / a.splits), h_hi = (int)((int64_t)hpg * (split + 1) / a.splits);
  const Piece pc = find_piece(a.cu, a.N, a.total, slot, T);
  const int64_t t0 = pc.begin + (int64_t)pc.index * T;
  const int len = pc.seq < 0 ? 0 : (int)min((int64_t)T, pc.begin + pc.len - t0);
  const bool live = len > 0 && state_live(a.live, a.live_slots, pc.seq);

  if (!live) {  // an unused slot, or a padded sequence: zero gradients
    for (int i = tid; i < (h_hi - h_lo) * 3; i += 512) a.part[((int64_t)slot * a.H + g * hpg + h_lo) * 3 + i] = 0.f;
    for (int i = tid; i < len * (h_hi - h_lo); i += 512)
      store_elem(a.ddt, (t0 + i / (h_hi - h_lo)) * a.H + g * hpg + h_lo + i % (h_hi - h_lo), 0.f, a.dt_in);
    for (int i = tid; i < len * NN; i += 512) {
      const int64_t at = ((t0 + i / NN) * a.G + g) * NN + i % NN;
      if (a.splits > 1) {
        a.part_bc[(int64_t)(2 * split) * a.total * a.G * NN + at] = 0.f;
        a.part_bc[(int64_t)(2 * split + 1) * a.total * a.G * NN + at] = 0.f;
      } else {
        store_elem(a.dB, at, 0.f, a.dt_in);
        store_elem(a.dC, at, 0.f, a.dt_in);
      }
    }
    return;
  }
  const int64_t slot64 = pc.seq + pc.begin / Q + 2 * pc.index;  // its first chunk's slot
  const int tiles = (len + 15) >> 4;

  // which part of the column work this wave has
  const int nt = wave % NT, n16 = 16 * nt;
  const bool do_c = BOTH || wave < NT, do_b = BOTH || (wave >= NT && wave < 2 * NT);

  // the next head's operands travel in registers while this head's are used
  Frag<BF> vx[W::XV], vy[W::XV];
  f32x4 vs[2 * DB];
  float vr[8 * DB];
  float vg[3], tot[5];  // a token's c (two) and dt'; the chunks' totals (two each) and A_log
  auto fetch_tokens = [&](int h) {
    constexpr int VPR = W::DK / 8;
    if constexpr (BF) {
      const auto wx = window(a.x, t0 * a.x_ts + (int64_t)h * D, 2, 2 * ((len - 1) * a.x_ts + D));
      const auto wy = window(a.dy, (t0 * a.H + h) * D, 2, 2 * ((len - 1) * (int64_t)(a.H * D) + D));
      const int t = tid / VPR, p0 = tid % VPR * 8;
      // (of d = 16, the vectors past the row's end lie outside the window's rows)
#pragma unroll
      for (int k = 0; k < W::XV; ++k) {
        const int tk = t + k * (512 / VPR);
        vx[k] = vy[k] = Frag<BF>::zero();
        if (D >= 32 || p0 < D) {
          vx[k].v = __builtin_amdgcn_raw_buffer_load_b128(wx, 2 * (tk * (int)a.x_ts + p0), 0, 0);
          vy[k].v = __builtin_amdgcn_raw_buffer_load_b128(wy, 2 * (tk * a.H * D + p0), 0, 0);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < W::XV; ++k) {
        const int i = tid + 512 * k, t = i / VPR, p0 = (i - t * VPR) * 8;
        vx[k] = vy[k] = Frag<BF>::zero();
        if (t < len && p0 < D) {
          vx[k] = frag_from<BF>(a.x, t0 * a.x_ts + (int64_t)h * D, t * (uint32_t)a.x_ts + p0, a.dt_in);
          vy[k] = frag_from<BF>(a.dy, (t0 * a.H + h) * D, t * (uint32_t)(a.H * D) + p0, a.dt_in);
        }
      }
    }
  };
  auto fetch_gates = [&](int h) {
    if (wave < 2) {  // the first wave has the first chunk's tokens, the second the second's, where there is one
      const float* g0 = a.gates + (slot64 * a.H + h) * 3 * Q;
      const float* g1 = g0 + (len > Q ? (int64_t)a.H * 3 * Q : 0);
      const auto w = window(wave == 0 ? g0 : g1, 0, 4, 12 * Q);
      vg[0] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(w, 4 * lane, 0, 0));
      vg[1] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(w, 4 * lane + 4 * Q, 0, 0));
      vg[2] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(w, 4 * lane + 8 * Q, 0, 0));
      tot[0] = scalar_read(g0 + Q - 1);
      tot[1] = scalar_read(g0 + 2 * Q - 1);
      tot[2] = scalar_read(g1 + Q - 1);
      tot[3] = scalar_read(g1 + 2 * Q - 1);
      tot[4] = scalar_read(a.A_log + h);
    }
  };
  auto commit_tokens = [&]() {
#pragma unroll
    for (int k = 0; k < W::XV; ++k) {
      const int at = (tid / (W::DK / 8) + k * (512 / (W::DK / 8))) * LDX + tid % (W::DK / 8) * 8;
      *reinterpret_cast<Frag<BF>*>(s_x + at) = vx[k];
      *reinterpret_cast<Frag<BF>*>(s_y + at) = vy[k];
    }
  };
  auto store_gates = [&](float* out) {
    if (wave < 2) {
      // prefix sums over the block: the second chunk's follow the first's total
      const double tot0 = (double)tot[0] + (double)tot[1];
      const double last = len > Q ? tot0 + ((double)tot[2] + (double)tot[3]) : tot0;
      double c = (double)vg[0] + (double)vg[1];
      float dtp = vg[2];
      if (wave == 1) {
        c = len > Q ? tot0 + c : tot0;
        dtp = len > Q ? dtp : 0.f;
      }
      const float ch = (float)c;
      out[tid] = 0.5f * ch;
      out[T + tid] = 0.5f * (float)(c - (double)ch);
      out[2 * T + tid] = exp2f((float)c);
      out[3 * T + tid] = dtp * exp2f((float)(last - c));
      out[4 * T + tid] = dtp;
      if (tid == 0) {
        out[5 * T] = expf(tot[4]);
        out[5 * T + 1] = exp2f((float)last);
      }
    }
  };
  // a state's column n of this wave's, 8 rows p at a time: from [n][p], or from [p][n]
  auto fetch_fwd = [&](int h) {
    const auto w = window(a.fwd, ((int64_t)slot * a.H + h) * (D * NN), 4, 4 * D * NN);
#pragma unroll
    for (int k = 0; k < 2 * DB; ++k) {
      vs[k] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (D >= 32 || 8 * q < D)
        vs[k] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(w, 4 * (l16 * D + 8 * q) + 4 * (32 * (k >> 1) + 4 * (k & 1)), 4 * n16 * D, 0));
    }
  };
  auto fetch_rev = [&](int h) {
    const auto w = window(a.rev, ((int64_t)slot * a.H + h) * (D * NN), 4, 4 * D * NN);
#pragma unroll
    for (int k = 0; k < 8 * DB; ++k) {
      vr[k] = 0.f;
      if (D >= 32 || 8 * q < D)
        vr[k] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(w, 4 * (8 * q * NN + l16) + 4 * (32 * (k >> 3) + (k & 7)) * NN, 4 * n16, 0));
    }
  };
  // four 16-token tiles of x or dy times a split state, their terms apart: a product never follows the one it adds to
  auto products = [&](const E* rows, int i0, const Split<BF> (&st)[DB], f32x4 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < DB; ++k) {
      Frag<BF> f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = Frag<BF>::load(rows + (16 * (i0 + i) + l16) * LDX + 32 * k + 8 * q);
#pragma unroll
      for (int t = Split<BF>::K - 1; t >= 0; --t)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = frag_mma(v[i], f[i], st[k].t[t]);
    }
  };

  // G for the wave's 16 rows: C_i . B_j.  bf16: both rows through LDS, over the places of x and dy and of the summed
  // products; FP32: straight from memory
  f32x4 G[W::G_LDS ? 1 : 8], Ns[W::N_LDS ? 1 : 8];
  constexpr int KB = (NN + 31) / 32, LDC = KB * 32 + 8;
  if constexpr (BF) {
    E* const s_c = s_x;
    E* const s_b = reinterpret_cast<E*>(s_ns);
    static_assert(T * LDC <= W::ELEMS && 2 * T * LDC <= W::TILES, "the rows of C and of B fit");
    const auto wc = window(a.Cm, t0 * a.c_ts + g * NN, 2, 2 * ((len - 1) * a.c_ts + NN));
    const auto wb = window(a.Bm, t0 * a.b_ts + g * NN, 2, 2 * ((len - 1) * a.b_ts + NN));
    Frag<BF> c[KB], b[KB];
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int t = (tid + 512 * k) / (KB * 4), n0 = (tid + 512 * k) % (KB * 4) * 8;
      c[k] = b[k] = Frag<BF>::zero();
      if (NN >= 32 || n0 < NN) {
        c[k].v = __builtin_amdgcn_raw_buffer_load_b128(wc, 2 * (t * (int)a.c_ts + n0), 0, 0);
        b[k].v = __builtin_amdgcn_raw_buffer_load_b128(wb, 2 * (t * (int)a.b_ts + n0), 0, 0);
      }
    }
    fetch_gates(g * hpg + h_lo);
    fetch_fwd(g * hpg + h_lo);
    fetch_rev(g * hpg + h_lo);
    fetch_tokens(g * hpg + h_lo);
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int at = (tid + 512 * k) / (KB * 4) * LDC + (tid + 512 * k) % (KB * 4) * 8;
      *reinterpret_cast<Frag<BF>*>(s_c + at) = c[k];
      *reinterpret_cast<Frag<BF>*>(s_b + at) = b[k];
    }
    __syncthreads();
    for (int jt = 0; jt <= wave; ++jt) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        acc = frag_mma(acc, Frag<BF>::load(s_c + (16 * wave + l16) * LDC + 32 * kb + 8 * q), Frag<BF>::load(s_b + (16 * jt + l16) * LDC + 32 * kb + 8 * q));
      s_gt[tile0 + jt * 64] = acc;
    }
    __syncthreads();
    for (int jt = 0; jt <= wave; ++jt) s_ns[tile0 + jt * 64] = f32x4{0.f, 0.f, 0.f, 0.f};
  } else {
    const int i = 16 * wave + l16;
#pragma unroll
    for (int jt = 0; jt < 8; ++jt) {
      Ns[jt] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (jt > wave) continue;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const int n0 = 32 * kb + 8 * q, j = 16 * jt + l16;
        Frag<BF> cf = Frag<BF>::zero(), bf = cf;
        if (i < len && n0 < NN) cf = frag_from<BF>(a.Cm, t0 * a.c_ts + g * NN, i * (uint32_t)a.c_ts + n0, a.dt_in);
        if (j < len && n0 < NN) bf = frag_from<BF>(a.Bm, t0 * a.b_ts + g * NN, j * (uint32_t)a.b_ts + n0, a.dt_in);
        acc = frag_mma(acc, cf, bf);
      }
      if constexpr (W::G_LDS) s_gt[tile0 + jt * 64] = acc;
      else G[jt] = acc;
    }
  }
  // four tiles of the wave's columns of C or B in the accumulators' order, from the transposed copies where the input is
  // bf16 (four tokens together; past the second chunk there is nothing to read)
  struct Columns {
    u32x2 w[BF ? 8 : 1];
  };
  auto load_columns = [&](const void* transposed, Columns& c) {
    if constexpr (BF)
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const auto w = window(transposed, (((slot64 + (it >> 2)) * a.G + g) * NN + n16) * Q, 2, it < 4 || len > Q ? 2 * 16 * Q : 0);
        c.w[it] = __builtin_amdgcn_raw_buffer_load_b64(w, 2 * (l16 * Q + 4 * q) + 32 * (it & 3), 0, 0);
      }
  };
  auto column_of = [&](const void* m, int64_t ts, const Columns& c, int it, float (&v)[4]) {
    if constexpr (BF) {
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = (r & 1) ? unpack_hi<GDN_BF16>(c.w[it][r >> 1]) : unpack_lo<GDN_BF16>(c.w[it][r >> 1]);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * it + 4 * q + r;
        v[r] = t < len ? load_elem(at_bytes(m, t0 * ts + g * NN + n16, t * (uint32_t)ts + l16, a.dt_in != GDN_F32 ? 2 : 4), 0, a.dt_in) : 0.f;
      }
    }
  };
  auto pick4 = [&](float v0, float v1, float v2, float v3) {
    const float lo = (l16 & 4) ? v1 : v0, hi = (l16 & 4) ? v3 : v2;
    return (l16 & 8) ? hi : lo;
  };
  // 2^(2 x) for x = half an exponent: the square of a root that the hardware's exponential does not flush
  auto decay_half = [](float x) {
    const float r = __builtin_amdgcn_exp2f(x);
    return r * r;
  };

  // closes a head: dt's gradient for the block's tokens and the head's parameter sums (one wave)
  auto close_head = [&](int h, const float* res, const float* gates) {
    const float *r_col = res, *r_row = res + 8 * T, *r_rd = r_row + T, *r_cd = r_rd + T, *r_dg = r_cd + T, *r_help = r_dg + T, *r_cs = r_help + T,
                *r_cv = r_cs + NT * T, *r_q = r_cv + NT * T, *r_dd = r_q + 8;
    // whole tiles with rows after block b and columns before it: 8 lanes a block
    float whole = 0.f;
    {
      const int b = lane >> 3, sub = lane & 7;
      for (int j = sub; j < 16 * b; j += 8)
        for (int i = b + 1; i < tiles; ++i) whole += r_col[i * T + j];
      whole += dpp_mov<0xB1>(whole);
      whole += dpp_mov<0x4E>(whole);
      whole += __shfl_xor(whole, 4, 64);
    }
    float qs = 0.f, dd = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      qs += i < NT ? r_q[i] : 0.f;
      dd += i < tiles ? r_dd[i] : 0.f;
    }
    // token 64 k + lane, in the block of 16 tokens 4 k + q
    float cv[2], co[2], dtp[2], pre[2], suf[2], cs_suf[2], cv_pre[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = 64 * k + lane, b = 4 * k + q;
      const bool in = t < 16 * tiles;
      float cs = 0.f;
      cv[k] = co[k] = 0.f;
      dtp[k] = gates[4 * T + t];
      if (in) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          cs += r_cs[i * T + t];
          cv[k] += r_cv[i * T + t];
        }
        for (int i = b + 1; i < tiles; ++i) co[k] += r_col[i * T + t];
      }
      // inside the block: earlier columns of later rows, and later rows of earlier columns
      const float r0 = in ? r_row[t] + (W::N_LDS && b > 4 ? r_help[t] : 0.f) : 0.f;
      pre[k] = row_shift<0x111>(row_prefix(co[k]));  // before t, not at it
      suf[k] = row_suffix(r0);
      cs_suf[k] = row_suffix(cs);
      cv_pre[k] = row_prefix(cv[k]);
      pre[k] += row_shift<0x111>(cv_pre[k]);
    }
    // the blocks' totals of the state parts, from both sides
    float after = 0.f, before = 0.f;
#pragma unroll
    for (int k = 1; k >= 0; --k)
#pragma unroll
      for (int r = 3; r >= 0; --r) {
        const float tot = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, cs_suf[k]), 16 * r));
        if (q == r) suf[k] += cs_suf[k] + after;
        after += tot;
      }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float tot = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, cv_pre[k]), 16 * r + 15));
        if (q == r) pre[k] += before;
        before += tot;
      }
    const float A = gates[5 * T], eq = qs * gates[5 * T + 1];
    float sa = 0.f, sb = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = 64 * k + lane;
      const float wh = __shfl(whole, 8 * (4 * k + q), 64);
      if (t < len) {
        const float dg = ((wh + pre[k]) + (suf[k] + r_rd[t])) + eq;
        // dt' x_t.X_t over dt'; a step that underflows to zero has a slope of zero with it
        const float own = dtp[k] > 0.f ? ((co[k] + r_cd[t]) + (r_dg[t] + cv[k])) / dtp[k] : 0.f;
        const float d = (own - A * dg) * -expm1f(-dtp[k]);  // softplus' = sigmoid = 1 - e^-softplus
        store_elem(a.ddt, (t0 + t) * a.H + h, d, a.dt_in);
        sa -= A * dtp[k] * dg;
        sb += d;
      }
    }
    sa = wave_sum(sa);
    sb = wave_sum(sb);
    if (lane == 0) {
      float* o = a.part + ((int64_t)slot * a.H + h) * 3;
      o[0] = sa;
      o[1] = sb;
      o[2] = dd;
    }
  };

  f32x4 dC[8], dB[8];
#pragma unroll
  for (int it = 0; it < 8; ++it) dC[it] = dB[it] = f32x4{0.f, 0.f, 0.f, 0.f};

  if constexpr (!BF) {
    fetch_tokens(g * hpg + h_lo);
    fetch_gates(g * hpg + h_lo);
    fetch_fwd(g * hpg + h_lo);
    fetch_rev(g * hpg + h_lo);
  }
  float *g_before = nullptr, *g_now = s_gates, *g_next = s_gates + (W::LATE ? W::GATES : 0);
  if constexpr (W::LATE) store_gates(g_now);
  for (int hi = h_lo; hi < h_hi; ++hi) {
    const int h = g * hpg + hi, h_next = min(h + 1, g * hpg + h_hi - 1);
    // the lane's places are not known to be the ones of the head before: what follows from them is formed anew, in a few
    // instructions, where it would otherwise be kept in registers that the loop has not got
    asm volatile("" : "+v"(tid), "+v"(lane), "+v"(l16), "+v"(q), "+v"(tile0));
    float* const res = s_res + (W::LATE ? (hi & 1) * W::RES : 0);
    float *r_col = res, *r_row = res + 8 * T, *r_rd = r_row + T, *r_cd = r_rd + T, *r_dg = r_cd + T, *r_help = r_dg + T, *r_cs = r_help + T,
          *r_cv = r_cs + NT * T, *r_q = r_cv + NT * T, *r_dd = r_q + 8;
    __syncthreads();  // the head before is done with LDS
    commit_tokens();
    if constexpr (!W::LATE) store_gates(g_now);
    const float *s_ch = g_now, *s_cl = s_ch + T, *s_er = s_cl + T, *s_wd = s_er + T, *s_dt = s_wd + T;
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    Columns cc, bb;
    if (do_c) load_columns(a.ct, cc);
    __builtin_amdgcn_sched_barrier(0);

    // state parts of dC and dB for the wave's 16 columns; row l16 / 4 of four tiles, token 4 q + l16 % 4 of it
    const int own = 16 * (l16 >> 2) + 4 * q + (l16 & 3);
    if (do_c) {
      Split<BF> sc[DB];
#pragma unroll
      for (int k = 0; k < DB; ++k) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = vs[2 * k + (e >> 2)][e & 3];
        sc[k] = Split<BF>::of(f);
      }
#pragma unroll
      for (int i0 = 0; i0 < 8; i0 += 4) {
        if (i0 >= tiles) continue;
        f32x4 v[4];
        products(s_y, i0, sc, v);
        float dots[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float col[4];
          column_of(a.Cm, a.c_ts, cc, i0 + i, col);
          dots[i] = row16_sum4(v[i][0] * col[0], v[i][1] * col[1], v[i][2] * col[2], v[i][3] * col[3]);
          dC[i0 + i] += v[i] * *reinterpret_cast<const f32x4*>(s_er + 16 * (i0 + i) + 4 * q);
        }
        r_cs[nt * T + 16 * i0 + own] = s_er[16 * i0 + own] * pick4(dots[0], dots[1], dots[2], dots[3]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (do_c) {
      float qs = 0.f;
#pragma unroll
      for (int k = 0; k < 8 * DB; ++k) qs += vs[k >> 2][k & 3] * vr[k];
      qs = wave_sum(qs);
      if (lane == 0) r_q[wave] = qs;
    }
    if (do_b) load_columns(a.bt, bb);  // before the next head's loads: these are waited for in order
    Split<BF> sb[DB];
#pragma unroll
    for (int k = 0; k < DB; ++k) {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = vr[8 * k + e];
      sb[k] = Split<BF>::of(f);
    }
    __builtin_amdgcn_sched_barrier(0);
    fetch_fwd(h_next);
    fetch_tokens(h_next);
    __builtin_amdgcn_sched_barrier(0);
    if (do_b) {
#pragma unroll
      for (int i0 = 0; i0 < 8; i0 += 4) {
        if (i0 >= tiles) continue;
        f32x4 v[4];
        products(s_x, i0, sb, v);
        float dots[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float col[4];
          column_of(a.Bm, a.b_ts, bb, i0 + i, col);
          dots[i] = row16_sum4(v[i][0] * col[0], v[i][1] * col[1], v[i][2] * col[2], v[i][3] * col[3]);
          dB[i0 + i] += v[i] * *reinterpret_cast<const f32x4*>(s_wd + 16 * (i0 + i) + 4 * q);
        }
        r_cv[nt * T + 16 * i0 + own] = s_wd[16 * i0 + own] * pick4(dots[0], dots[1], dots[2], dots[3]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    fetch_rev(h_next);
    if constexpr (W::LATE) fetch_gates(h_next);

    // products of dy and x, a row of 16 x 16 tiles a wave; off the diagonal tile the decay is that down to the rows'
    // first token times that from there
    auto tile_row = [&](int it, int j_lo, int j_hi, bool owner) {
      Frag<BF> yf[DB];
#pragma unroll
      for (int k = 0; k < DB; ++k) yf[k] = Frag<BF>::load(s_y + (16 * it + l16) * LDX + 32 * k + 8 * q);
      const int i0 = 16 * it + 4 * q, base = it * (it + 1) / 2 * 64 + lane;
      const f32x4 ih = *reinterpret_cast<const f32x4*>(s_ch + i0), il = *reinterpret_cast<const f32x4*>(s_cl + i0);
      const float mh = s_ch[16 * it], ml = s_cl[16 * it];
      f32x4 rowo = {0.f, 0.f, 0.f, 0.f}, down;
#pragma unroll
      for (int r = 0; r < 4; ++r) down[r] = decay_half((ih[r] - mh) + (il[r] - ml));
      auto product = [&](int j) {
        f32x4 w = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < DB; ++k) w = frag_mma(w, yf[k], Frag<BF>::load(s_x + j * LDX + 32 * k + 8 * q));
        return w;
      };
      auto below = [&](int jt, f32x4& ns, const f32x4& gt) {
        const int j = 16 * jt + l16;
        const f32x4 w = product(j);
        const float from = s_dt[j] * decay_half((mh - s_ch[j]) + (ml - s_cl[j]));
        float col = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = down[r] * from, m = e * (w[r] * gt[r]);
          ns[r] += e * w[r];
          col += m;
          rowo[r] += m;
        }
        col = xor_sum_from<16>(col);
        if (q == 0) r_col[it * T + j] = col;
      };
      auto diagonal = [&](f32x4& ns, const f32x4& gt) {
        const int j = 16 * it + l16;
        const f32x4 w = product(j);
        const float jh = s_ch[j], jl = s_cl[j], dtj = s_dt[j];
        f32x4 off;
        float diag = 0.f, wd = 0.f, cd = 0.f, dg = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = dtj * decay_half(j <= i0 + r ? (ih[r] - jh) + (il[r] - jl) : -INFINITY), m = e * (w[r] * gt[r]);
          ns[r] += e * w[r];
          diag = j == i0 + r ? m : diag;
          wd = j == i0 + r ? w[r] : wd;
          off[r] = j == i0 + r ? 0.f : m;
          cd += off[r];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // the columns before j, of j's row and later ones
          const float before = row_prefix(row_shift<0x111>(off[r]));
          dg += j <= i0 + r ? before : 0.f;
        }
        const float z = rows_sum4(cd, diag, wd, dg);  // the rows of 16 lanes get the four sums over the tile's rows
        if (q != 2) (q == 0 ? r_cd : q == 1 ? r_dg : r_rd)[j] = z;
        const float dd = row16_sum(z);
        if (lane == 32) r_dd[it] = dd;
      };
      if constexpr (W::N_LDS) {
        f32x4 ns;
#pragma unroll 1
        for (int jt = j_lo; jt < j_hi; ++jt) {
          ns = s_ns[base + jt * 64];
          below(jt, ns, s_gt[base + jt * 64]);
          s_ns[base + jt * 64] = ns;
        }
        if (owner) {
          ns = s_ns[base + it * 64];
          diagonal(ns, s_gt[base + it * 64]);
          s_ns[base + it * 64] = ns;
        }
      } else {
#pragma unroll
        for (int jt = 0; jt < 8; ++jt) {
          f32x4 gt = {0.f, 0.f, 0.f, 0.f};
          if (jt <= it) {
            if constexpr (W::G_LDS) gt = s_gt[base + jt * 64];
            else gt = G[jt];
          }
          if (jt < it) below(jt, Ns[jt], gt);
          else if (jt == it) diagonal(Ns[jt], gt);
        }
      }
      const float ro = row16_sum4(rowo[0], rowo[1], rowo[2], rowo[3]);
      if (l16 < 4) (owner ? r_row : r_help)[i0 + l16] = ro;
    };
    // Rows 5, 6 and 7 give their first 1, 2 and 3 tiles to waves 3, 2 and 1, which leaves five tiles a wave and one for
    // the first, which closes heads (where the tiles' sums are in registers every wave keeps its row).
    const int given = W::N_LDS && wave > 4 ? wave - 4 : 0;
    if (wave < tiles) tile_row(wave, given, wave, true);
    if (W::N_LDS && wave >= 1 && wave < 4 && 8 - wave < tiles) tile_row(8 - wave, 0, 4 - wave, false);
    if constexpr (W::LATE) {
      store_gates(g_next);
      if (wave == 0 && hi > h_lo) close_head(h - 1, s_res + ((hi - 1) & 1) * W::RES, g_before);
      g_before = g_now;
      g_now = g_next;
      g_next = s_gates + ((hi - h_lo + 2) % 3) * W::GATES;
    } else {
      __syncthreads();
      if (wave == 0) close_head(h, res, g_now);
      fetch_gates(h_next);
    }
  }
  if constexpr (W::LATE) {
    __syncthreads();
    if (wave == 0) close_head(g * hpg + h_hi - 1, s_res + ((h_hi - 1) & 1) * W::RES, g_before);
  }

  // the heads' summed products with B and C, in two bf16 terms (bf16 inputs): as [i][j] for dC, as [j][i] for dB
#pragma unroll
  for (int turn = 0; turn < 2; ++turn) {
    constexpr int TERMS = BF ? 2 : 1;
    Frag<BF> f[4];
    if (turn == 0 ? do_c : do_b)
#pragma unroll
      for (int kb = 0; kb < 4; ++kb)
        f[kb] = 32 * kb >= len ? Frag<BF>::zero()
                               : Frag<BF>::load(reinterpret_cast<const E*>(at_bytes(
                                     turn == 0 ? a.bt : a.ct, (((slot64 + (kb >> 1)) * a.G + g) * NN + n16) * Q + 32 * (kb & 1), l16 * Q + 8 * q, sizeof(E))));
    __syncthreads();
#pragma unroll
    for (int jt = 0; jt < 8; ++jt) {
      f32x4 ns = {0.f, 0.f, 0.f, 0.f};
      if (jt <= wave) {
        if constexpr (W::N_LDS) ns = s_ns[tile0 + jt * 64];
        else ns = Ns[jt];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * wave + 4 * q + r, j = 16 * jt + l16;
        E* d = s_n + (turn == 0 ? i * LDN + j : j * LDN + i);
        if constexpr (BF) {
          const uint32_t hi = pack2<GDN_BF16>(ns[r], 0.f) & 0xffffu;
          d[0] = (E)hi;
          d[T * LDN] = (E)pack2<GDN_BF16>(ns[r] - bf16_bits_to_f32(hi), 0.f);
        } else {
          d[0] = ns[r];
        }
      }
    }
    __syncthreads();
    if (turn == 0 ? do_c : do_b) {
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        if (32 * kb >= len) continue;
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          if (turn == 0 ? 2 * kb > it : 2 * kb + 1 < it) continue;  // no pair j <= i in the tile
#pragma unroll
          for (int k = TERMS - 1; k >= 0; --k) {
            const Frag<BF> nf = Frag<BF>::load(s_n + k * T * LDN + (16 * it + l16) * LDN + 32 * kb + 8 * q);
            if (turn == 0) dC[it] = frag_mma(dC[it], nf, f[kb]);
            else dB[it] = frag_mma(dB[it], nf, f[kb]);
          }
        }
      }
    }
  }
  auto write = [&](const f32x4 (&v)[8], void* out, int which) {
    const int64_t at = (t0 * a.G + g) * NN + n16;
    const int64_t part = (int64_t)(2 * split + which) * a.total * a.G * NN + at;
#pragma unroll
    for (int it = 0; it < 8; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * it + 4 * q + r;
        const uint32_t off = t * (uint32_t)(a.G * NN) + l16;
        if (t >= len) continue;
        if (a.splits > 1) *reinterpret_cast<float*>(const_cast<char*>(at_bytes(a.part_bc, part, off, 4))) = v[it][r];
        else if constexpr (BF) *reinterpret_cast<__bf16*>(const_cast<char*>(at_bytes(out, at, off, 2))) = (__bf16)v[it][r];
        else store_elem(out, at + off, v[it][r], a.dt_in);
      }
  };
  if (do_b) write(dB, a.dB, 0);
  if (do_c) write(dC, a.dC, 1);
}

// dB and dC from the splits' parts, in order.
__global__ void __launch_bounds__(256) gdn_m2s_join_kernel(const float* part, int splits, int64_t each, void* dB, void* dC, int dt) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= 2 * each) return;
  float s = part[i];
  for (int k = 1; k < splits; ++k) s += part[(int64_t)2 * k * each + i];
  if (i < each) store_elem(dB, i, s, dt);
  else store_elem(dC, i - each, s, dt);
}

// The head parameters' gradients: a workgroup a head, its blocks in a fixed order.
__global__ void __launch_bounds__(256) gdn_m2s_params_kernel(const float* part, int64_t slots, int H, float* dA_log, float* ddt_bias, float* dD) {
  __shared__ double s[3][256];
  const int h = blockIdx.x;
  double t[3] = {0.0, 0.0, 0.0};
  for (int64_t i = threadIdx.x; i < slots; i += 256)
#pragma unroll
    for (int k = 0; k < 3; ++k) t[k] += part[(i * H + h) * 3 + k];
#pragma unroll
  for (int k = 0; k < 3; ++k) s[k][threadIdx.x] = t[k];
  for (int off = 128; off > 0; off >>= 1) {
    __syncthreads();
    if (threadIdx.x < off)
#pragma unroll
      for (int k = 0; k < 3; ++k) s[k][threadIdx.x] += s[k][threadIdx.x + off];
  }
  if (threadIdx.x == 0) {
    dA_log[h] = (float)s[0][0];
    ddt_bias[h] = (float)s[1][0];
    dD[h] = (float)s[2][0];
  }
}

// ------------------------------------------------------------------ host
namespace {

template <bool BF, int D, int NN>
hipError_t grad(const M2GradArgs& a, int64_t slots, hipStream_t s) {
  using W = GradGeom<BF, D, NN>;
  auto* k = gdn_m2s_grad_kernel<BF, D, NN>;
  static std::atomic<uint64_t> allowed{0};
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(k), W::LDS, allowed);
  if (e != hipSuccess) return e;
  k<<<(unsigned)(slots * a.G * a.splits), 512, W::LDS, s>>>(a);
  return hipGetLastError();
}

template <bool BF, int D>
hipError_t grad_n(const M2GradArgs& a, int n, int64_t slots, hipStream_t s) {
  if (n == 16) return grad<BF, D, 16>(a, slots, s);
  if (n == 64) return grad<BF, D, 64>(a, slots, s);
  return grad<BF, D, 128>(a, slots, s);
}

template <bool BF>
hipError_t grad_dn(const M2GradArgs& a, int d, int n, int64_t slots, hipStream_t s) {
  if (d == 16) return grad_n<BF, 16>(a, n, slots, s);
  if (d == 64) return grad_n<BF, 64>(a, n, slots, s);
  return grad_n<BF, 128>(a, n, slots, s);
}

}  // namespace

// Workgroups that share a group's heads: more than one where blocks and groups
// alone would leave compute units idle.
int grad_splits(int64_t N, int64_t total, int H, int G) {
  const int64_t units = ((total + kGradBlock - 1) / kGradBlock) * G;
  int64_t s = units > 0 ? 512 / units : 1;
  if (s > H / G) s = H / G;
  return s < 1 ? 1 : (int)s;
}

int64_t grad_work_items(int64_t N, int64_t total, int H, int G) {
  return scan_slots(N, total, kGradBlock) * G * grad_splits(N, total, H, G) * 512;
}

hipError_t launch_scan_grad(const M2GradArgs& a, bool bf, int d, int n, hipStream_t s) {
  const int64_t slots = scan_slots(a.N, a.total, kGradBlock);
  if (a.total > 0) {
    hipError_t e = bf ? grad_dn<true>(a, d, n, slots, s) : grad_dn<false>(a, d, n, slots, s);
    if (e != hipSuccess) return e;
    if (a.splits > 1) {
      const int64_t each = a.total * a.G * n;
      gdn_m2s_join_kernel<<<(unsigned)((2 * each + 255) / 256), 256, 0, s>>>(a.part_bc, a.splits, each, a.dB, a.dC, a.dt_in);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  gdn_m2s_params_kernel<<<a.H, 256, 0, s>>>(a.part, a.total > 0 ? slots : 0, a.H, a.dA_log, a.ddt_bias, a.dD);
  return hipGetLastError();
}

}  // namespace gdn
