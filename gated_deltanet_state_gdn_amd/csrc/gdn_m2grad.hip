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
// that share t's rows or columns by sums from the far side, and only inside
// the diagonal tile row sums and column sums are subtracted.  Diagonal
// elements do not enter.
//
// A decay multiplies last, so that one close to the smallest numbers costs one
// rounding there.  The states are split in three bf16 terms (bf16 inputs), so all sums that end
// in dt's gradient and the head parameters' are FP32 sums of FP32 products.
// Parameter sums go through one partial row a block and are added in a fixed
// order, in 64 bits.
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
  // floats: c (two), dt', read and write factors; row and column sums; the waves' parts
  static constexpr int FLOATS = 5 * T + 8 * T + 4 * T + 2 * NT * T + 8 + 8;
  static constexpr size_t LDS = (size_t)ELEMS * sizeof(E) + FLOATS * 4;
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
__global__ void __launch_bounds__(512) gdn_m2s_grad_kernel(const M2GradArgs a) {
  using W = GradGeom<BF, D, NN>;
  typedef typename W::E E;
  constexpr int T = W::T, NT = W::NT, LDX = W::LDX, LDN = W::LDN, DB = W::DB, Q = kScanChunk;
  constexpr bool BOTH = W::BOTH;
  extern __shared__ __align__(16) unsigned char smem[];
  E* const s_x = reinterpret_cast<E*>(smem);
  E* const s_y = s_x + T * LDX;
  E* const s_n = s_x;
  float* const s_ch = reinterpret_cast<float*>(smem + (size_t)W::ELEMS * sizeof(E));
  float* const s_cl = s_ch + T;
  float* const s_dt = s_cl + T;
  float* const s_er = s_dt + T;      // e^{c_i}
  float* const s_ew = s_er + T;      // e^{c_last - c_j}
  float* const s_col = s_ew + T;     // [8][128] column sums of the tiles below the diagonal, by row block
  float* const s_row = s_col + 8 * T;  // row sums of them
  float* const s_rd = s_row + T;     // row and column sums inside the diagonal tiles
  float* const s_cd = s_rd + T;
  float* const s_dg = s_cd + T;      // the diagonal
  float* const s_cs = s_dg + T;      // [NT][128]
  float* const s_cv = s_cs + NT * T;
  float* const s_q = s_cv + NT * T;  // [8] parts of <S, dS'>
  float* const s_dd = s_q + 8;       // [8] parts of sum dy.x

  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
  const bool do_c = wave < NT, do_b = BOTH || (wave >= NT && wave < 2 * NT);

  // G for the wave's 16 rows: C_i . B_j
  f32x4 G[8], Ns[8];
#pragma unroll
  for (int jt = 0; jt < 8; ++jt) G[jt] = Ns[jt] = f32x4{0.f, 0.f, 0.f, 0.f};
  {
    const int i = 16 * wave + l16;
#pragma unroll
    for (int kb = 0; kb < (NN + 31) / 32; ++kb) {
      const int n0 = 32 * kb + 8 * q;
      Frag<BF> cf = Frag<BF>::zero();
      if (i < len && n0 < NN) cf = frag_from<BF>(a.Cm, (t0 + i) * a.c_ts + g * NN + n0, a.dt_in);
#pragma unroll
      for (int jt = 0; jt < 8; ++jt) {
        if (jt > wave) continue;
        const int j = 16 * jt + l16;
        Frag<BF> bf = Frag<BF>::zero();
        if (j < len && n0 < NN) bf = frag_from<BF>(a.Bm, (t0 + j) * a.b_ts + g * NN + n0, a.dt_in);
        G[jt] = frag_mma(G[jt], cf, bf);
      }
    }
  }
  // the wave's columns of C and B in the accumulators' order, kept in the input's width
  constexpr int CW = BF ? 2 : 4;
  uint32_t cc[8][CW], bb[8][CW];
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    float cv[4], bv[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t t = t0 + 16 * it + 4 * q + r;
      const bool in = 16 * it + 4 * q + r < len;
      cv[r] = in ? load_elem(a.Cm, t * a.c_ts + g * NN + n16 + l16, a.dt_in) : 0.f;
      bv[r] = in ? load_elem(a.Bm, t * a.b_ts + g * NN + n16 + l16, a.dt_in) : 0.f;
    }
    if constexpr (BF) {
      cc[it][0] = pack2<GDN_BF16>(cv[0], cv[1]);
      cc[it][1] = pack2<GDN_BF16>(cv[2], cv[3]);
      bb[it][0] = pack2<GDN_BF16>(bv[0], bv[1]);
      bb[it][1] = pack2<GDN_BF16>(bv[2], bv[3]);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        cc[it][r] = __float_as_uint(cv[r]);
        bb[it][r] = __float_as_uint(bv[r]);
      }
    }
  }
  auto value = [](const uint32_t (&w)[CW], int r) {
    if constexpr (BF) return (r & 1) ? unpack_hi<GDN_BF16>(w[r >> 1]) : unpack_lo<GDN_BF16>(w[r >> 1]);
    else return __uint_as_float(w[r]);
  };

  f32x4 dC[8], dB[8];
#pragma unroll
  for (int it = 0; it < 8; ++it) dC[it] = dB[it] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int hi = h_lo; hi < h_hi; ++hi) {
    const int h = g * hpg + hi;
    __syncthreads();  // the head before is done with LDS
    constexpr int VPR = W::DK / 8;
    for (int i = tid; i < T * VPR; i += 512) {
      const int t = i / VPR, p0 = (i - t * VPR) * 8;
      Frag<BF> xv = Frag<BF>::zero(), yv = xv;
      if (t < len && p0 < D) {
        xv = frag_from<BF>(a.x, (t0 + t) * a.x_ts + (int64_t)h * D + p0, a.dt_in);
        yv = frag_from<BF>(a.dy, ((t0 + t) * a.H + h) * D + p0, a.dt_in);
      }
      *reinterpret_cast<Frag<BF>*>(s_x + t * LDX + p0) = xv;
      *reinterpret_cast<Frag<BF>*>(s_y + t * LDX + p0) = yv;
    }
    if (tid < T) {
      // prefix sums over the block: the second chunk's follow the first's total
      const float* g0 = a.gates + (slot64 * a.H + h) * 3 * Q;
      const float* g1 = g0 + (int64_t)a.H * 3 * Q;
      const double tot0 = (double)g0[Q - 1] + (double)g0[2 * Q - 1];
      double c = tot0, last = tot0;
      float dtp = 0.f;
      if (len > Q) last = tot0 + ((double)g1[Q - 1] + (double)g1[2 * Q - 1]);
      if (tid < Q) {
        c = (double)g0[tid] + (double)g0[Q + tid];
        dtp = g0[2 * Q + tid];
      } else if (len > Q) {
        c = tot0 + ((double)g1[tid - Q] + (double)g1[tid]);
        dtp = g1[Q + tid];
      }
      const float ch = (float)c;
      s_ch[tid] = ch;
      s_cl[tid] = (float)(c - (double)ch);
      s_dt[tid] = dtp;
      s_er[tid] = expf((float)c);
      s_ew[tid] = expf((float)(last - c));
    }
    // the states' rows n of this wave's columns: S^T[n][p]
    Split<BF> sc[DB], sb[DB];
    float qs = 0.f;
    {
      const int64_t at = ((int64_t)slot * a.H + h) * (D * NN) + (n16 + l16) * D;
#pragma unroll
      for (int k = 0; k < DB; ++k) {
        float f[8], r[8];
        const int p0 = 32 * k + 8 * q;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = r[e] = 0.f;
        if (p0 < D) {
          load_vec<8>(a.fwd, at + p0, GDN_F32, f);
          load_vec<8>(a.rev, at + p0, GDN_F32, r);
        }
        if (do_c)
#pragma unroll
          for (int e = 0; e < 8; ++e) qs += f[e] * r[e];
        sc[k] = Split<BF>::of(f);
        sb[k] = Split<BF>::of(r);
      }
    }
    __syncthreads();

    // products of dy and x for the wave's 16 rows
    if (wave < tiles) {
      Frag<BF> yf[DB];
#pragma unroll
      for (int k = 0; k < DB; ++k) yf[k] = Frag<BF>::load(s_y + (16 * wave + l16) * LDX + 32 * k + 8 * q);
      const int i0 = 16 * wave + 4 * q;
      float ih[4], il[4], rowo[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        ih[r] = s_ch[i0 + r];
        il[r] = s_cl[i0 + r];
      }
#pragma unroll
      for (int jt = 0; jt < 8; ++jt) {
        if (jt > wave) continue;
        f32x4 w = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < DB; ++k) w = frag_mma(w, yf[k], Frag<BF>::load(s_x + (16 * jt + l16) * LDX + 32 * k + 8 * q));
        const int j = 16 * jt + l16;
        const float jh = s_ch[j], jl = s_cl[j], dtj = s_dt[j];
        if (jt < wave) {
          float col = 0.f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float e = decay_between(ih[r], il[r], jh, jl), dw = dtj * w[r];
            Ns[jt][r] += e * dw;
            const float m = e * (dw * G[jt][r]);
            col += m;
            rowo[r] += m;
          }
          col = xor_sum_from<16>(col);
          if (q == 0) s_col[wave * T + j] = col;
        } else {
          float col = 0.f, rowd[4], diag = 0.f, wd = 0.f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = i0 + r;
            const float e = j <= i ? decay_between(ih[r], il[r], jh, jl) : 0.f, dw = dtj * w[r];
            Ns[jt][r] += e * dw;
            const float m = e * (dw * G[jt][r]);
            if (i == j) {
              diag = m;
              wd = w[r];
            }
            const float off = i == j ? 0.f : m;
            col += off;
            rowd[r] = row16_sum(off);
            rowo[r] = row16_sum(rowo[r]);
          }
          col = xor_sum_from<16>(col);
          diag = xor_sum_from<16>(diag);
          wd = wave_sum(wd);
          if (q == 0) {
            s_cd[j] = col;
            s_dg[j] = diag;
          }
          if (lane == 0) s_dd[wave] = wd;
          if (l16 < 4) {
            const float v = l16 == 0 ? rowd[0] : l16 == 1 ? rowd[1] : l16 == 2 ? rowd[2] : rowd[3];
            const float o = l16 == 0 ? rowo[0] : l16 == 1 ? rowo[1] : l16 == 2 ? rowo[2] : rowo[3];
            s_rd[i0 + l16] = v;
            s_row[i0 + l16] = o;
          }
        }
      }
    }
    // state parts of dC and dB for the wave's 16 columns
    if (do_c) {
      qs = wave_sum(qs);
      if (lane == 0) s_q[wave] = qs;
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        if (it >= tiles) continue;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < DB; ++k) v = sc[k].mma_right(v, Frag<BF>::load(s_y + (16 * it + l16) * LDX + 32 * k + 8 * q));
        float s[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = s_er[16 * it + 4 * q + r];
          s[r] = e * row16_sum(v[r] * value(cc[it], r));
          v[r] *= e;
        }
        dC[it] += v;
        if (l16 < 4) s_cs[nt * T + 16 * it + 4 * q + l16] = l16 == 0 ? s[0] : l16 == 1 ? s[1] : l16 == 2 ? s[2] : s[3];
      }
    }
    if (do_b) {
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        if (it >= tiles) continue;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < DB; ++k) v = sb[k].mma_right(v, Frag<BF>::load(s_x + (16 * it + l16) * LDX + 32 * k + 8 * q));
        float s[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * it + 4 * q + r;
          const float e = s_ew[j], dtj = s_dt[j];
          s[r] = e * (dtj * row16_sum(v[r] * value(bb[it], r)));
          v[r] *= e * dtj;
        }
        dB[it] += v;
        if (l16 < 4) s_cv[nt * T + 16 * it + 4 * q + l16] = l16 == 0 ? s[0] : l16 == 1 ? s[1] : l16 == 2 ? s[2] : s[3];
      }
    }
    __syncthreads();

    if (wave == 0) {
      // dg: token 64 k + lane, its block of 16 b = 4 k + q
      // whole tiles with rows after block b and columns before it: 8 lanes a block
      float whole = 0.f;
      {
        const int b = lane >> 3, sub = lane & 7;
        for (int j = sub; j < 16 * b; j += 8) {
          float c = 0.f;
          for (int i = b + 1; i < tiles; ++i) c += s_col[i * T + j];
          whole += c;
        }
        whole += dpp_mov<0xB1>(whole);
        whole += dpp_mov<0x4E>(whole);
        whole += __shfl_xor(whole, 4, 64);
      }
      float qs_ = 0.f, dd = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        qs_ += i < NT ? s_q[i < NT ? i : 0] : 0.f;
        dd += i < tiles ? s_dd[i] : 0.f;
      }
      float cs[2], cv[2], co[2], dtp[2], pre[2], suf[2], cs_suf[2], cv_pre[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = 64 * k + lane, b = 4 * k + q;
        const bool in = t < 16 * tiles;
        cs[k] = cv[k] = co[k] = 0.f;
        dtp[k] = s_dt[t];
        if (in) {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            cs[k] += s_cs[i * T + t];
            cv[k] += s_cv[i * T + t];
          }
          for (int i = b + 1; i < tiles; ++i) co[k] += s_col[i * T + t];
        }
        // inside the block: earlier columns of later rows, later rows of earlier columns, and the diagonal tile
        const float r0 = in ? s_row[t] + (s_rd[t] - s_cd[t]) : 0.f;
        pre[k] = row_shift<0x111>(row_prefix(co[k]));  // before t, not at it
        suf[k] = row_suffix(r0);
        cs_suf[k] = row_suffix(cs[k]);
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
      const float A = expf(a.A_log[h]), bias = a.dt_bias[h], eq = qs_ * s_er[len - 1];
      float sa = 0.f, sb_ = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = 64 * k + lane;
        const float wh = __shfl(whole, 8 * (4 * k + q), 64);
        if (t < len) {
          const float dg = ((wh + pre[k]) + suf[k]) + eq;
          // dt' x_t.X_t over dt'; a step that underflows to zero has a slope of zero with it
          const float own = dtp[k] > 0.f ? ((co[k] + s_cd[t]) + (s_dg[t] + cv[k])) / dtp[k] : 0.f;
          const float raw = load_elem(a.dt, (t0 + t) * a.dt_ts + h, a.dt_in) + bias;
          const float d = (own - A * dg) * sigmoid_f(raw);
          store_elem(a.ddt, (t0 + t) * a.H + h, d, a.dt_in);
          sa -= A * dtp[k] * dg;
          sb_ += d;
        }
      }
      sa = wave_sum(sa);
      sb_ = wave_sum(sb_);
      if (lane == 0) {
        float* o = a.part + ((int64_t)slot * a.H + h) * 3;
        o[0] = sa;
        o[1] = sb_;
        o[2] = dd;
      }
    }
  }

  // the heads' summed products with B and C, in two bf16 terms (bf16 inputs): as [i][j] for dC, as [j][i] for dB
#pragma unroll
  for (int turn = 0; turn < 2; ++turn) {
    f32x4 left[8];
#pragma unroll
    for (int jt = 0; jt < 8; ++jt) left[jt] = Ns[jt];
#pragma unroll
    for (int term = 0; term < (BF ? 2 : 1); ++term) {
      __syncthreads();
#pragma unroll
      for (int jt = 0; jt < 8; ++jt) {
        E e[4];
        if constexpr (BF) {
          const uint32_t w0 = pack2<GDN_BF16>(left[jt][0], left[jt][1]), w1 = pack2<GDN_BF16>(left[jt][2], left[jt][3]);
          e[0] = (E)w0;
          e[1] = (E)(w0 >> 16);
          e[2] = (E)w1;
          e[3] = (E)(w1 >> 16);
#pragma unroll
          for (int r = 0; r < 4; ++r) left[jt][r] -= bf16_bits_to_f32(e[r]);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) e[r] = left[jt][r];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * wave + 4 * q + r, j = 16 * jt + l16;
          s_n[turn == 0 ? i * LDN + j : j * LDN + i] = e[r];
        }
      }
      __syncthreads();
      const bool mine = turn == 0 ? do_c : do_b;
      if (mine) {
        const E* src = static_cast<const E*>(turn == 0 ? a.bt : a.ct);
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          if (32 * kb >= len) continue;
          const Frag<BF> f = Frag<BF>::load(src + (((slot64 + (kb >> 1)) * a.G + g) * NN + n16 + l16) * Q + 32 * (kb & 1) + 8 * q);
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            if (turn == 0 ? 2 * kb > it : 2 * kb + 1 < it) continue;  // no pair j <= i in the tile
            const Frag<BF> nf = Frag<BF>::load(s_n + (16 * it + l16) * LDN + 32 * kb + 8 * q);
            if (turn == 0) dC[it] = frag_mma(dC[it], nf, f);
            else dB[it] = frag_mma(dB[it], nf, f);
          }
        }
      }
    }
  }
#pragma unroll
  for (int it = 0; it < 8; ++it)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * it + 4 * q + r;
      if (t >= len) continue;
      const int64_t at = ((t0 + t) * a.G + g) * NN + n16 + l16;
      if (a.splits > 1) {
        const int64_t each = a.total * a.G * NN;
        if (do_b) a.part_bc[(int64_t)(2 * split) * each + at] = dB[it][r];
        if (do_c) a.part_bc[(int64_t)(2 * split + 1) * each + at] = dC[it][r];
      } else {
        if (do_b) store_elem(a.dB, at, dB[it][r], a.dt_in);
        if (do_c) store_elem(a.dC, at, dC[it][r], a.dt_in);
      }
    }
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
  if (W::LDS > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, (int)W::LDS);
    if (e != hipSuccess) return e;
  }
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
