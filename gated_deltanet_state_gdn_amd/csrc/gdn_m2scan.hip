// Mamba2 recurrence over packed sequences, and its reverse (the sequence form
// of the state update of gdn_mamba2.hip, Dao and Gu's selective state-space
// model; AREX ReplaySSM article, "bottleneck" section, for the state's shape).
//
// Per head, with g = -exp(A_log) dt' and dt' = softplus(dt + dt_bias):
//     S_t = e^{g_t} S_{t-1} + dt'_t x_t B_t^T,   y_t = S_t C_t + D x_t.
// Over a chunk of 64 tokens with c_i = g_1 + .. + g_i in it and S before it:
//     y_i = e^{c_i} S C_i + sum_{j<=i} e^{c_i-c_j} dt'_j (C_i.B_j) x_j + D x_i
//     S'  = e^{c_last} S + sum_j e^{c_last-c_j} dt'_j x_j B_j^T
// and in reverse, with dS' the gradient of the state after the chunk:
//     X_j  = e^{c_last-c_j} dS' B_j + sum_{i>=j} e^{c_i-c_j} (C_i.B_j) dy_i
//     dx_j = dt'_j X_j + D dy_j,   dS = e^{c_last} dS' + sum_i e^{c_i} dy_i C_i^T
// One kernel does both: tokens have a read vector (C, or B in reverse), a
// write vector (B, or C) and an input (x, or dy).  Exponents are never positive.
//
// Kernels: the prep forms, once for all heads of a group, the products of read
// and write vectors and the transposed write vectors, and each head's dt' and
// c.  The walk keeps the states of 128 rows (two heads of 64; 64 rows, one head,
// where walks are few) in accumulators and goes over the chunks; the state meets the read vectors straight from its
// accumulators, whose layout is that of an operand once the read vectors'
// columns are stored in the same order.  Where there are too few walks for the
// chip, sequences are cut into segments: a first walk finds each segment's own
// end state, a small kernel chains them, the second walk starts every segment
// from its true state.
//
// Rounding (bf16 inputs and outputs): products of two inputs are exact in FP32.  The state
// is FP32, and its updates multiply e^{..} dt' x in three bf16 terms, all its
// 24 bits, with exact B.  For the output alone the state and the decay-weighted
// products of read and write vectors are taken in two bf16 terms, off by 2^-16 of
// each, where y's own rounding is 2^-8: 99.8% of y then is the exact value's
// rounding, against half of it with one term.  (The prefill below takes 663 us
// with two terms, 604 with one.)
// Any other types take the FP32 MFMA throughout.
//
// Measured (bf16, heads of 64 x 128): prompts of 1024, 3000 and twice 8192
// tokens through 128 heads 663 us a call, of which the prep takes 50, 1.2 TB/s of
// what has to move: the chain of 128 chunks, 4.8 us each, is what bounds it.
// Matrix units are busy 15% of the time, vector units 27%.  In a kernel trace,
// 16,384 tokens, states only, 222 us; in reverse with dx 451.
#include <algorithm>

#include "gdn_m2scan.h"

namespace gdn {

// ------------------------------------------------------------------ prep
// One workgroup a (chunk slot, group): gm[r][c] = read_r . write_c in FP32,
// wt = write vectors transposed [n][64], rt = read vectors transposed (only
// where asked for), and for the group's heads c as two floats and dt'.
// Tokens past the sequence's end count as zero vectors with dt' = g = 0.
template <bool BF, int NN>
__global__ void __launch_bounds__(256) gdn_m2s_prep_kernel(const M2ScanArgs a) {
  typedef typename Frag<BF>::E E;
  constexpr int KB = (NN + 31) / 32, LD = KB * 32 + (BF ? 8 : 4);
  __shared__ __align__(16) E s_r[kScanChunk * LD];
  __shared__ __align__(16) E s_w[kScanChunk * LD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, q = lane >> 4;
  const Piece pc = find_piece(a.cu, a.N, a.total, blockIdx.x, kScanChunk);
  const int64_t t0 = pc.begin + (int64_t)pc.index * kScanChunk;
  const int len = pc.seq < 0 ? 0 : (int)min((int64_t)kScanChunk, pc.begin + pc.len - t0);
  if (len <= 0) return;
  const int g = blockIdx.y;
  constexpr int VPR = KB * 4;  // 8-element vectors of a row, zeros past NN
  for (int u = tid; u < kScanChunk * VPR; u += 256) {
    const int t = u / VPR, n0 = (u - t * VPR) * 8;
    Frag<BF> r = Frag<BF>::zero(), w = r;
    if (t < len && n0 < NN) {
      r = frag_from<BF>(a.read, t0 * a.read_ts + g * NN, t * (uint32_t)a.read_ts + n0, a.in_dt);
      w = frag_from<BF>(a.write, t0 * a.write_ts + g * NN, t * (uint32_t)a.write_ts + n0, a.in_dt);
    }
    *reinterpret_cast<Frag<BF>*>(s_r + t * LD + n0) = r;
    *reinterpret_cast<Frag<BF>*>(s_w + t * LD + n0) = w;
  }
  // gates: a head a wave, a token a lane
  const int hpg = a.H / a.G;
  for (int hi = wave; hi < hpg; hi += 4) {
    const int h = g * hpg + hi;
    float dtp = 0.f;
    double c = 0.0;
    if (lane < len) {
      dtp = softplus_f(load_elem(a.dt, (t0 + lane) * a.dt_ts + h, a.in_dt) + a.dt_bias[h]);
      c = -(double)(expf(a.A_log[h]) * dtp) * 1.4426950408889634;  // in powers of two
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double o = __shfl_up(c, off, 64);
      if (lane >= off) c += o;
    }
    float* gt = a.gates + ((int64_t)blockIdx.x * a.H + h) * 3 * kScanChunk;
    const float ch = (float)c;
    gt[lane] = ch;
    gt[kScanChunk + lane] = (float)(c - (double)ch);
    gt[2 * kScanChunk + lane] = dtp;
  }
  __syncthreads();
  const int64_t cg = (int64_t)blockIdx.x * a.G + g;
  if (a.gm != nullptr) {
    float* gm = a.gm + cg * kScanChunk * kScanChunk;
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        acc = frag_mma(acc, Frag<BF>::load(s_r + (16 * wave + l16) * LD + 32 * kb + 8 * q),
                       Frag<BF>::load(s_w + (16 * ct + l16) * LD + 32 * kb + 8 * q));
#pragma unroll
      for (int r = 0; r < 4; ++r) gm[(16 * wave + 4 * q + r) * kScanChunk + 16 * ct + l16] = acc[r];
    }
  }
  for (int u = tid; u < NN * 8; u += 256) {
    const int n = u % NN, tb = (u / NN) * 8;
    Frag<BF> f;
    E* e = reinterpret_cast<E*>(&f);
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = s_w[(tb + k) * LD + n];
    *reinterpret_cast<Frag<BF>*>(static_cast<E*>(a.wt) + (cg * NN + n) * kScanChunk + tb) = f;
    if (a.rt != nullptr) {
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = s_r[(tb + k) * LD + n];
      *reinterpret_cast<Frag<BF>*>(static_cast<E*>(a.rt) + (cg * NN + n) * kScanChunk + tb) = f;
    }
  }
}

// ------------------------------------------------------------------ walk
// Four waves over 128 state rows (two heads of 64), two workgroups on a compute
// unit, or 64, three: one's vector work then runs beside the other's matrix work.  Eight
// waves over 256 rows, one workgroup, share the read and write vectors of a
// chunk among twice the heads but keep in step: a prefill of 20,408 tokens
// through 128 heads took 789 us that way, 678 us this way (the read-out with one
// bf16 term in both).
template <bool BF, int D, int NN, int PT_, bool OUT>
struct WalkGeom {
  typedef typename Frag<BF>::E E;
  static constexpr int NW = 4;
  static constexpr int THREADS = 64 * NW;
  static constexpr int PT = PT_;                       // 16-row tiles of a wave
  static constexpr int ROWS = 16 * PT * NW;            // state rows of the workgroup
  static constexpr int HB = ROWS / D;                  // its heads
  static constexpr int WPH = NW / HB;                  // waves of a head
  static constexpr int NT = NN / 16, KB = (NN + 31) / 32;
  static constexpr int LDF = KB * 32 + (BF ? 8 : 4);   // read vectors [64][LDF], columns in accumulator order
  static constexpr int LDK = kScanChunk + (BF ? 0 : 4);  // write vectors [NN][LDK] (16-bit form: groups of 8 tokens permuted by the row)
  static constexpr int LDT = kScanChunk + (BF ? 8 : 4);  // inputs [ROWS][LDT], products [HB][64][LDT]
  // the products' second bf16 terms lie over the read vectors
  static constexpr int PE = HB * kScanChunk * LDT, FE = BF && PE > kScanChunk * LDF ? PE : kScanChunk * LDF;
  static constexpr int F0 = 0, K0 = F0 + (OUT ? FE : 0), X0 = K0 + NN * LDK, P0 = X0 + ROWS * LDT;
  static constexpr int ELEMS = P0 + (OUT ? PE : 0);
  // floats a head: c (two), dt', the input's weight, the read factor
  static constexpr size_t LDS = ((size_t)ELEMS * sizeof(E) + 15) / 16 * 16 + (size_t)HB * 5 * kScanChunk * 4;
  // vectors of 8 elements that a thread stages
  static constexpr int FV = (kScanChunk * NN / 8 + THREADS - 1) / THREADS;
  static constexpr int XV = kScanChunk * ROWS / 8 / THREADS;
};

// Where (row p, token t) of the transposed inputs lies: in 16-bit form groups
// of 8 tokens are permuted by the row's block of 8, so that the transposing
// stores of a wave meet all banks.
template <bool BF, int LDT>
__device__ __forceinline__ int xt_at(int p, int t) {
  return p * LDT + (BF ? ((((t >> 3) ^ (p >> 3)) & 7) << 3 | (t & 7)) : t);
}

template <bool BF, int LDK>
__device__ __forceinline__ int kt_at(int n, int t) {
  return n * LDK + (BF ? ((t >> 3) ^ (n & 7)) << 3 : t);  // t: a multiple of 8
}

template <bool BF, int D, int NN, int PT, bool REV, bool OUT>
__global__ void __launch_bounds__(256, BF ? 2 : 1) gdn_m2s_walk_kernel(const M2ScanArgs a) {
  using W = WalkGeom<BF, D, NN, PT, OUT>;
  typedef typename W::E E;
  constexpr int HB = W::HB, NT = W::NT, KB = W::KB, LDF = W::LDF, LDT = W::LDT, ROWS = W::ROWS, Q = kScanChunk;
  constexpr int THREADS = W::THREADS, WPH = W::WPH, PB = ROWS / 8;
  extern __shared__ __align__(16) unsigned char smem[];
  E* const s_f = reinterpret_cast<E*>(smem) + W::F0;
  E* const s_k = reinterpret_cast<E*>(smem) + W::K0;
  E* const s_x = reinterpret_cast<E*>(smem) + W::X0;
  E* const s_p = reinterpret_cast<E*>(smem) + W::P0;
  float* const s_g = reinterpret_cast<float*>(smem + ((size_t)W::ELEMS * sizeof(E) + 15) / 16 * 16);  // [HB][5][64]

  int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hpg = a.H / a.G, hbs = (hpg + HB - 1) / HB;
  // Whole sequences: each XCD takes a run of them, so that a chunk's heads share its L2.  Segments: round the XCDs, as the
  // slots behind a sequence that is not cut have no work, and runs of them would leave some XCDs with half the others' (10
  // x 500 to 1000 tokens x 64 heads 117 us round, 151 in runs; equal lengths, 20 x 500 x 32 heads, 82 and 80).
  const int u = a.seg_chunks > 0 ? blockIdx.x : xcd_unit(blockIdx.x, gridDim.x);
  const int slot = u / (a.G * hbs), gh = u - slot * (a.G * hbs), g = gh / hbs, hb = gh - g * hbs;
  Piece sg;
  if (a.seg_chunks > 0) {
    sg = find_piece(a.cu, a.N, a.total, slot, a.seg_chunks * Q);
    if (sg.seq < 0) return;
    if (sg.count <= a.whole) {  // its first segment's workgroup takes it whole
      if (sg.index > 0) return;
      sg.count = 1;
    }
  } else {
    sg.seq = slot;
    sg.begin = token_at(a.cu, slot, a.total);
    sg.len = max(token_at(a.cu, slot + 1, a.total) - sg.begin, (int64_t)0);
    sg.index = 0;
    sg.count = 1;
  }
  const bool last_seg = REV ? sg.index == 0 : sg.index == sg.count - 1;
  if (a.local && last_seg) return;  // nothing starts from this segment's end
  const int chunks = (int)((sg.len + Q - 1) / Q);
  const int c_lo = sg.index * a.seg_chunks;
  const int c_hi = sg.count > 1 ? min(chunks, c_lo + a.seg_chunks) : chunks;
  const int64_t slot0 = sg.seq + sg.begin / Q;  // chunk slot of the sequence's first chunk

  const int p0 = wave * 16 * PT;                // the wave's rows of the workgroup's
  const int hl = wave / WPH, hw = hb * HB + hl; // its head of the workgroup's, and of the group's
  const int rows_in = min(ROWS, (hpg - hb * HB) * D);
  const bool mine = hw < hpg;
  const int64_t col0 = ((int64_t)g * hpg + hb * HB) * D;  // the workgroup's first column of a token's inputs
  const int h = g * hpg + min(hw, hpg - 1);
  const int pd = p0 - hl * D;                   // the wave's rows within its head

  if (!state_live(a.live, a.live_slots, sg.seq)) {  // a padded sequence: zero outputs, no state
    if (OUT)
      for (int64_t i = tid; i < (int64_t)(c_hi - c_lo) * Q * rows_in; i += THREADS) {
        const int64_t t = sg.begin + (int64_t)c_lo * Q + i / rows_in;
        if (t < sg.begin + sg.len) store_elem(a.out, t * a.H * D + col0 + i % rows_in, 0.f, a.out_dt);
      }
    if (OUT && a.fin.base != nullptr && a.fin.slots == nullptr && last_seg)
      for (int i = tid; i < rows_in * NN; i += THREADS) store_elem(a.fin.base, ((int64_t)sg.seq * a.H * D + col0) * NN + i, 0.f, a.fin.dtype);
    return;
  }

  // The state in accumulators.  With outputs it is transposed, S[nt][pt][r] = (n = 16 nt + 4 q + r, p = 16 pt + l16), the
  // order in which it meets the read vectors; without, (n = 16 nt + l16, p = 16 pt + 4 q + r), which gives blocks [n][p]
  // four values at a time.  In memory a state is [p][n].
  f32x4 S[NT][PT];
  auto load_as = [&](const void* base, int64_t unit, auto type) {  // all loads before the first use
    constexpr int DT = decltype(type)::value, EB = DT == GDN_F32 ? 4 : 2;
    const int64_t at = ((unit * a.H + h) * D + pd) * NN;
    InVec<DT, 4> v[OUT ? NT : 1][PT];
    uint32_t e[OUT ? 1 : NT][PT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        if constexpr (OUT) {
          v[nt][pt].load(at_bytes(base, at + 16 * pt * NN + 16 * nt, l16 * NN + 4 * q, EB), 0);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) e[nt][pt][r] = in_bits<DT>(at_bytes(base, at + (16 * pt + r) * NN + 16 * nt, 4 * q * NN + l16, EB), 0);
        }
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        float f[4];
        if constexpr (OUT) v[nt][pt].widen(f);
        else
#pragma unroll
          for (int r = 0; r < 4; ++r) f[r] = in_value<DT>(e[nt][pt][r]);
        S[nt][pt] = f32x4{f[0], f[1], f[2], f[3]};
      }
  };
  auto load_state = [&](const void* base, int64_t unit, int dt) {
    if (dt == GDN_F32) load_as(base, unit, std::integral_constant<int, GDN_F32>{});
    else if (dt == GDN_BF16) load_as(base, unit, std::integral_constant<int, GDN_BF16>{});
    else load_as(base, unit, std::integral_constant<int, GDN_F16>{});
  };
  auto store_state = [&](void* base, int64_t unit, int dt) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        const int64_t at = ((unit * a.H + h) * D + pd + 16 * pt) * NN + 16 * nt;
        const float f[4] = {S[nt][pt][0], S[nt][pt][1], S[nt][pt][2], S[nt][pt][3]};
        if constexpr (OUT) store_vec<4>(base, at + l16 * NN + 4 * q, f, dt, true);
        else
#pragma unroll
          for (int r = 0; r < 4; ++r) store_elem(base, at + (4 * q + r) * NN + l16, f[r], dt);
      }
  };
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int pt = 0; pt < PT; ++pt) S[nt][pt] = f32x4{0.f, 0.f, 0.f, 0.f};
  double total_g = 0.0;
  const float Dh = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, a.Dskip[h])));

  // A chunk's operands are fetched a chunk ahead, in registers.  What a thread stages: vectors of 8 along n of the read
  // vectors (token t, and t + 256 / (NN / 8) for the next), of 8 tokens of the transposed write vectors, and of 8 columns of
  // the inputs, in 16-bit form for two neighbouring tokens (eight column blocks, then eight pairs, a wave).
  constexpr int VPR = NN / 8, FSTEP = 256 / VPR;
  static_assert(256 % VPR == 0 && NN * 8 % 64 == 0, "whole rows of vectors");
  Frag<BF> vf[OUT ? W::FV : 1], vk[W::FV], vx[W::XV];
  float vg[3];
  // the products of read and write vectors: the 16 x 16 tiles on and below the diagonal (above it in reverse) and the two
  // beyond it that share a 32-token operand with one on it go round the head's waves; lane: row lane / 4, four columns
  constexpr int PER = 12 / WPH;
  f32x4 gm[OUT ? PER : 1];
  int rts[PER], cts[PER];
  const int sub = wave & (WPH - 1);
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int t = sub + k * WPH;
    const int i = t >= 10 ? 2 * (t - 10) : t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0, j = t >= 10 ? i + 1 : t - i * (i + 1) / 2;
    rts[k] = REV ? j : i;
    cts[k] = REV ? i : j;
  }
  auto fetch = [&](int c) {
    const int64_t t0 = sg.begin + (int64_t)c * Q;
    const int len = (int)min((int64_t)Q, sg.begin + sg.len - t0);
    const int64_t cs = slot0 + c, cg = cs * a.G + g;
    const char* pk = static_cast<const char*>(a.wt) + cg * (NN * Q * (int)sizeof(E));
#pragma unroll
    for (int k = 0; k < W::FV; ++k)
      if (NN * 8 % 256 == 0 || tid + 256 * k < NN * 8)
        vk[k] = Frag<BF>::load(reinterpret_cast<const E*>(pk + k * 256 * 8 * sizeof(E) + (uint32_t)(tid * 8 * sizeof(E))));
    if constexpr (OUT && BF) {
      const auto w = window(a.read, t0 * a.read_ts + g * NN, 2, 2 * ((len - 1) * a.read_ts + NN));
      const int off = 2 * (tid / VPR * (int)a.read_ts + tid % VPR * 8);
#pragma unroll
      for (int k = 0; k < W::FV; ++k) vf[k].v = __builtin_amdgcn_raw_buffer_load_b128(w, off + 2 * k * FSTEP * (int)a.read_ts, 0, 0);
    } else if constexpr (OUT) {
      const int t = tid / VPR;
      const uint32_t off = t * (uint32_t)a.read_ts + tid % VPR * 8;
      const int64_t at = t0 * a.read_ts + g * NN;
#pragma unroll
      for (int k = 0; k < W::FV; ++k) {
        vf[k] = Frag<BF>::zero();
        if (t + k * FSTEP < len) vf[k] = frag_from<BF>(a.read, at + k * FSTEP * a.read_ts, off, a.in_dt);
      }
    }
    if constexpr (BF) {
      // rows past the group's heads read what lies there, or zero: no output depends on them
      const auto w = window(a.in, t0 * a.in_ts + col0, 2, 2 * ((len - 1) * a.in_ts + rows_in));
      const int off = 2 * (2 * (tid >> 3 & 31) * (int)a.in_ts + 8 * (tid & 7));
#pragma unroll
      for (int k = 0; k < W::XV; ++k)  // 2 k and 2 k + 1 are two tokens of the same block of columns
        vx[k].v = __builtin_amdgcn_raw_buffer_load_b128(w, off + 2 * ((k & 1) * (int)a.in_ts + 64 * (k >> 1)), 0, 0);
    } else {
      const int t = tid / PB, pb = tid % PB;
      const uint32_t off = t * (uint32_t)a.in_ts + 8 * pb;
      const int64_t at = t0 * a.in_ts + col0;
#pragma unroll
      for (int k = 0; k < W::XV; ++k) {
        const int dt = k * (256 / PB);
        vx[k] = Frag<BF>::zero();
        if (t + dt < len && 8 * pb < rows_in) vx[k] = frag_from<BF>(a.in, at + dt * a.in_ts, off, a.in_dt);
      }
    }
    if (wave < HB) {  // a wave a head, a token a lane
      const char* gt = reinterpret_cast<const char*>(a.gates + (cs * a.H + g * hpg + min(hb * HB + wave, hpg - 1)) * 3 * Q);
      vg[0] = *reinterpret_cast<const float*>(gt + (uint32_t)(4 * lane));
      vg[1] = *reinterpret_cast<const float*>(gt + 4 * Q + (uint32_t)(4 * lane));
      vg[2] = *reinterpret_cast<const float*>(gt + 8 * Q + (uint32_t)(4 * lane));
    }
  };
  auto fetch_products = [&](int c) {
    const char* pg = reinterpret_cast<const char*>(a.gm + ((slot0 + c) * a.G + g) * Q * Q);
#pragma unroll
    for (int k = 0; k < PER; ++k)
      gm[k] = *reinterpret_cast<const f32x4*>(pg + (16 * rts[k] * Q + 16 * cts[k]) * 4 + (uint32_t)(((lane >> 2) * Q + (lane & 3) * 4) * 4));
  };
  auto commit = [&](int len) {
    {
      E* d = s_k + kt_at<BF, W::LDK>(tid >> 3, (tid & 7) * 8);  // 32 rows on, the same place in the permutation
#pragma unroll
      for (int k = 0; k < W::FV; ++k)
        if (NN * 8 % 256 == 0 || tid + 256 * k < NN * 8) *reinterpret_cast<Frag<BF>*>(d + k * 32 * W::LDK) = vk[k];
    }
    if constexpr (OUT) {
      // n = 32 k + 16 b + 4 s + r is stored at 32 k + 8 s + 4 b + r
      const int t = tid / VPR, n0 = tid % VPR * 8;
      E* d = s_f + t * LDF + (n0 & ~31) + 2 * (n0 & 15) + ((n0 >> 4) & 1) * 4;
#pragma unroll
      for (int k = 0; k < W::FV; ++k)
        if (Q * VPR % 256 == 0 || t + k * FSTEP < Q) {
          vf[k].store_halves(d + k * FSTEP * LDF, d + k * FSTEP * LDF + 8);
          if (NN == 16) Frag<BF>::zero().store_halves(d + k * FSTEP * LDF + 4, d + k * FSTEP * LDF + 12);
        }
    }
    if constexpr (BF) {
      // 64 rows on, a row's block of 8 has the same place in the permutation
      E* d = s_x + xt_at<BF, LDT>(8 * (tid & 7), 2 * (tid >> 3 & 31));
#pragma unroll
      for (int k = 0; k < W::XV / 2; ++k) {
        const u32x4 v0 = vx[2 * k].v, v1 = vx[2 * k + 1].v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          *reinterpret_cast<uint32_t*>(d + (64 * k + 2 * e) * LDT) = __builtin_amdgcn_perm(v1[e], v0[e], 0x05040100u);
          *reinterpret_cast<uint32_t*>(d + (64 * k + 2 * e + 1) * LDT) = __builtin_amdgcn_perm(v1[e], v0[e], 0x07060302u);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < W::XV; ++k) {
        const int pb = tid % PB, t = tid / PB + k * (256 / PB);
        float f[8];
        vx[k].widen(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s_x[xt_at<BF, LDT>(8 * pb + e, t)] = (E)f[e];
      }
    }
    if (wave < HB) {
      const float end_h = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, vg[0]), 63));
      const float end_l = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, vg[1]), 63));
      const float to_end = exp2f((end_h - vg[0]) + (end_l - vg[1])), from_start = exp2f(vg[0] + vg[1]);
      float* o = s_g + wave * 5 * Q + lane;
      o[0] = vg[0];
      o[Q] = vg[1];
      o[2 * Q] = vg[2];
      o[3 * Q] = lane < len ? (REV ? from_start : to_end * vg[2]) : 0.f;
      o[4 * Q] = REV ? to_end : from_start;
    }
  };

  const int steps = c_hi - c_lo;
  if (steps > 0) {
    fetch(REV ? c_hi - 1 : c_lo);
    if constexpr (OUT) fetch_products(REV ? c_hi - 1 : c_lo);
  }
  if (!a.local && mine) {
    if (sg.count > 1) load_state(a.seg, slot, GDN_F32);
    else if (a.init.base != nullptr) load_state(a.init.base, a.init.slots != nullptr ? a.init.slots[sg.seq] : sg.seq, a.init.dtype);
  }
  const float* const gh_ = s_g + hl * 5 * Q;

  for (int step = 0; step < steps; ++step) {
    const int c = REV ? c_hi - 1 - step : c_lo + step;
    const int64_t t0 = sg.begin + (int64_t)c * Q;
    const int len = (int)min((int64_t)Q, sg.begin + sg.len - t0);
    // the lane's places are not known to be the ones of the chunk before: what follows from them is formed anew, in a few
    // instructions, where it would otherwise be kept in registers that the loop has not got
    asm volatile("" : "+v"(tid), "+v"(lane), "+v"(l16), "+v"(q));

    __syncthreads();  // the chunk before is done with LDS
    commit(len);
    __syncthreads();

    // Memory operations are waited for in order: the inputs once more (for D x) first, then the next chunk's operands,
    // which have the whole chunk to arrive, then, once this chunk's are used, the next products, and last the stores.
    const int c_next = min(max(REV ? c - 1 : c + 1, c_lo), c_hi - 1);
    f32x4 acc[PT][4];
    InVec<BF ? GDN_BF16 : GDN_F32, 4> vin[PT][4];
    if constexpr (OUT) {
      if constexpr (BF) {
        const auto w = window(a.in, t0 * a.in_ts + (int64_t)h * D + pd, 2, 2 * ((len - 1) * a.in_ts + 16 * PT));
        const int off = 2 * (l16 * (int)a.in_ts + 4 * q);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) {
            const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(w, off + 2 * (16 * rt * (int)a.in_ts + 16 * pt), 0, 0);
            vin[pt][rt].w[0] = v[0];
            vin[pt][rt].w[1] = v[1];
          }
      } else {
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) {
            const int64_t at = (t0 + 16 * rt) * a.in_ts + (int64_t)h * D + pd + 16 * pt;
            float f[4] = {0.f, 0.f, 0.f, 0.f};
            if (16 * rt + l16 < len) load_vec<4>(at_bytes(a.in, at, l16 * (uint32_t)a.in_ts + 4 * q, a.in_dt == GDN_F32 ? 4 : 2), 0, a.in_dt, f);
#pragma unroll
            for (int r = 0; r < 4; ++r) vin[pt][rt].w[r] = __float_as_uint(f[r]);
          }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    fetch(c_next);
    __builtin_amdgcn_sched_barrier(0);
    Frag<BF> xf[2][PT];  // the wave's inputs
    if constexpr (OUT) {
      u32x2 low[BF ? PER : 1];  // the products' second terms
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int r = 16 * rts[k] + (lane >> 2), c0 = 16 * cts[k] + 4 * (lane & 3);
        // c of the column less that of the row
        const f32x4 x = (*reinterpret_cast<const f32x4*>(gh_ + c0) - gh_[r]) + (*reinterpret_cast<const f32x4*>(gh_ + Q + c0) - gh_[Q + r]);
        f32x4 w = gm[k];
        if constexpr (!REV) w *= *reinterpret_cast<const f32x4*>(gh_ + 2 * Q + c0);
        E* d = s_p + (hl * Q + r) * LDT + c0;
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool on = REV ? c0 + e >= r : c0 + e <= r;
          const float v = __builtin_amdgcn_exp2f(REV ? x[e] : -x[e]) * w[e];
          f[e] = on ? v : 0.f;
        }
        if constexpr (BF) {
          const u32x2 high = {pack2<GDN_BF16>(f[0], f[1]), pack2<GDN_BF16>(f[2], f[3])};
          *reinterpret_cast<u32x2*>(d) = high;
          bf16_rest(high[0], f[0], f[1]);
          bf16_rest(high[1], f[2], f[3]);
          low[k] = u32x2{pack2<GDN_BF16>(f[0], f[1]), pack2<GDN_BF16>(f[2], f[3])};
        } else {
          *reinterpret_cast<f32x4*>(d) = f32x4{f[0], f[1], f[2], f[3]};
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      // the state's part of the output
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) acc[pt][rt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        typedef Split<BF, 2> Terms;
        Terms sf[PT];
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[e] = S[2 * kb][pt][e];
            f[4 + e] = 2 * kb + 1 < NT ? S[2 * kb + 1 < NT ? 2 * kb + 1 : 0][pt][e] : 0.f;
          }
          sf[pt] = Terms::of(f);
        }
        Frag<BF> ff[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) ff[rt] = Frag<BF>::load(s_f + (16 * rt + l16) * LDF + 32 * kb + 8 * q);
#pragma unroll
        for (int k = Terms::K - 1; k >= 0; --k)
#pragma unroll
          for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) acc[pt][rt] = frag_mma(acc[pt][rt], sf[pt].t[k], ff[rt]);
      }
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        const float f = gh_[4 * Q + 16 * rt + l16];
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) acc[pt][rt] *= f;
      }

      __builtin_amdgcn_sched_barrier(0);
      fetch_products(c_next);
      __builtin_amdgcn_sched_barrier(0);
      auto take_products = [&](const E* p) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) {
            if (REV ? (ks == 0 && rt >= 2) : (ks == 1 && rt < 2)) continue;  // all beyond the diagonal
            const Frag<BF> pf = Frag<BF>::load(p + (hl * Q + 16 * rt + l16) * LDT + 32 * ks + 8 * q);
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) acc[pt][rt] = frag_mma(acc[pt][rt], xf[ks][pt], pf);
          }
        }
      };
      __syncthreads();  // the products are there, and the read vectors done with
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) xf[ks][pt] = Frag<BF>::load(s_x + xt_at<BF, LDT>(p0 + 16 * pt + l16, 32 * ks + 8 * q));
      if constexpr (BF)
#pragma unroll
        for (int k = 0; k < PER; ++k)
          *reinterpret_cast<u32x2*>(s_f + (hl * Q + 16 * rts[k] + (lane >> 2)) * LDT + 16 * cts[k] + 4 * (lane & 3)) = low[k];
      take_products(s_p);
      if constexpr (BF) {
        __syncthreads();  // and their second terms
        take_products(s_f);
      }
      if constexpr (BF) {
        const auto w = window(a.out, (t0 * a.H + h) * D + pd, 2, mine ? 2 * ((len - 1) * (a.H * D) + 16 * PT) : 0);
        const int off = 2 * (l16 * (a.H * D) + 4 * q);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          const float sc = REV ? gh_[2 * Q + 16 * rt + l16] : 1.f;
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) {
            float v[4];
            vin[pt][rt].widen(v);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = acc[pt][rt][r] * sc + Dh * v[r];
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack2<GDN_BF16>(v[0], v[1]), pack2<GDN_BF16>(v[2], v[3])}, w,
                                                  off + 2 * (16 * rt * (a.H * D) + 16 * pt), 0, 0);
          }
        }
      } else if (mine) {
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          const int t = 16 * rt + l16;
          if (t < len) {
            const float sc = REV ? gh_[2 * Q + t] : 1.f;
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) {
              float v[4];
              vin[pt][rt].widen(v);
#pragma unroll
              for (int r = 0; r < 4; ++r) v[r] = acc[pt][rt][r] * sc + Dh * v[r];
              store_vec<4>(const_cast<char*>(at_bytes(a.out, (t0 + 16 * rt) * a.H * D + (int64_t)h * D + pd + 16 * pt,
                                                      l16 * (uint32_t)(a.H * D) + 4 * q, a.out_dt != GDN_F32 ? 2 : 4)), 0, v, a.out_dt, true);
            }
          }
        }
      }
    }

    if (a.blocks != nullptr && mine && (REV ? ((c & 1) || c == chunks - 1) : !(c & 1))) {
      // the state that meets this block of two chunks: [p][n] in reverse, [n][p] forward
      float* o = a.blocks + ((sg.seq + sg.begin / kGradBlock + (c >> 1)) * a.H + h) * (int64_t)(D * NN);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) {
          const int64_t at = OUT ? (pd + 16 * pt) * NN + 16 * nt : 16 * nt * D + pd + 16 * pt;
          *reinterpret_cast<f32x4*>(const_cast<char*>(at_bytes(o, at, l16 * (OUT ? NN : D) + 4 * q, 4))) = S[nt][pt];
        }
    }
    // the state after the chunk
    const float end_h = gh_[Q - 1], end_l = gh_[2 * Q - 1], dec = exp2f(end_h + end_l);
    total_g += (double)end_h + (double)end_l;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) S[nt][pt] *= dec;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (32 * ks >= len) continue;
      Split<BF> xs[PT];
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        float f[8];
        if constexpr (OUT) xf[ks][pt].widen(f);
        else Frag<BF>::load(s_x + xt_at<BF, LDT>(p0 + 16 * pt + l16, 32 * ks + 8 * q)).widen(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= gh_[3 * Q + 32 * ks + 8 * q + e];
        xs[pt] = Split<BF>::of(f);
      }
      // four tiles of n at a time, their terms apart: a product never follows the one it adds to
      constexpr int NG = NT < 4 ? NT : 4;
#pragma unroll
      for (int ng = 0; ng < NT; ng += NG) {
        Frag<BF> kf[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i) kf[i] = Frag<BF>::load(s_k + kt_at<BF, W::LDK>(16 * (ng + i) + l16, 32 * ks + 8 * q));
#pragma unroll
        for (int k = Split<BF>::K - 1; k >= 0; --k)
#pragma unroll
          for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt)
              S[ng + i][pt] = OUT ? frag_mma(S[ng + i][pt], kf[i], xs[pt].t[k]) : frag_mma(S[ng + i][pt], xs[pt].t[k], kf[i]);
      }
    }
  }

  if (!mine) return;
  if (a.local) {
    store_state(a.seg, slot, GDN_F32);
    if (pd == 0 && lane == 0) a.seg_g[(int64_t)slot * a.H + h] = total_g;
  } else if (a.fin.base != nullptr && last_seg && (REV || sg.len > 0)) {
    store_state(a.fin.base, a.fin.slots != nullptr ? a.fin.slots[sg.seq] : sg.seq, a.fin.dtype);
  }
}

// ------------------------------------------------------------------ chain
// Turns the segments' own end states into the states they start from, in
// place: per (sequence, head), four state elements a thread.
template <bool REV>
__global__ void __launch_bounds__(256) gdn_m2s_chain_kernel(const M2ScanArgs a, int elems) {
  const int seq = blockIdx.z, h = blockIdx.y;
  const int i = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= elems || !state_live(a.live, a.live_slots, seq)) return;
  const int P = a.seg_chunks * kScanChunk;
  const int64_t b = token_at(a.cu, seq, a.total), e = token_at(a.cu, seq + 1, a.total);
  const int count = (int)max((e - b + P - 1) / P, (int64_t)1);
  if (count <= a.whole) return;
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (a.init.base != nullptr) {
    float f[4];
    load_vec<4>(a.init.base, ((a.init.slots != nullptr ? a.init.slots[seq] : (int64_t)seq) * a.H + h) * elems + i, a.init.dtype, f);
    S = f32x4{f[0], f[1], f[2], f[3]};
  }
  const int64_t s0 = seq + b / P;
  for (int k = 0; k < count; ++k) {
    const int64_t unit = (s0 + (REV ? count - 1 - k : k)) * a.H + h;
    f32x4* p = reinterpret_cast<f32x4*>(a.seg + unit * elems + i);
    if (k + 1 < count) {
      const f32x4 own = *p;
      const float dec = (float)exp2(a.seg_g[unit]);
      *p = S;
      S = S * dec + own;
    } else {
      *p = S;
    }
  }
}

// ------------------------------------------------------------------ host
int64_t scan_slots(int64_t N, int64_t total, int64_t P) { return N + (total + P - 1) / P; }

namespace {

template <bool BF, int D, int NN, int PT, bool REV, bool OUT>
hipError_t walk(const M2ScanArgs& a, hipStream_t s) {
  using W = WalkGeom<BF, D, NN, PT, OUT>;
  const int hpg = a.H / a.G, hbs = (hpg + W::HB - 1) / W::HB;
  const int64_t slots = a.seg_chunks > 0 ? scan_slots(a.N, a.total, (int64_t)a.seg_chunks * kScanChunk) : a.N;
  auto* k = gdn_m2s_walk_kernel<BF, D, NN, PT, REV, OUT>;
  static std::atomic<uint64_t> allowed{0};
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(k), W::LDS, allowed);
  if (e != hipSuccess) return e;
  k<<<(unsigned)(slots * a.G * hbs), W::THREADS, W::LDS, s>>>(a);
  return hipGetLastError();
}

template <bool BF, int D, int NN, int PT>
hipError_t walk_kind(const M2ScanArgs& a, bool rev, bool out, hipStream_t s) {
  if (rev) return out ? walk<BF, D, NN, PT, true, true>(a, s) : walk<BF, D, NN, PT, true, false>(a, s);
  return out ? walk<BF, D, NN, PT, false, true>(a, s) : walk<BF, D, NN, PT, false, false>(a, s);
}

template <bool BF, int D, int NN>
hipError_t walk_pt(const M2ScanArgs& a, bool rev, bool out, hipStream_t s) {
  if constexpr (D == 64) return a.narrow ? walk_kind<BF, D, NN, 1>(a, rev, out, s) : walk_kind<BF, D, NN, 2>(a, rev, out, s);
  else return walk_kind<BF, D, NN, D == 16 ? 1 : 2>(a, rev, out, s);
}

template <bool BF, int D>
hipError_t walk_n(const M2ScanArgs& a, int n, bool rev, bool out, hipStream_t s) {
  if (n == 16) return walk_pt<BF, D, 16>(a, rev, out, s);
  if (n == 64) return walk_pt<BF, D, 64>(a, rev, out, s);
  return walk_pt<BF, D, 128>(a, rev, out, s);
}

template <bool BF>
hipError_t walk_dn(const M2ScanArgs& a, int d, int n, bool rev, bool out, hipStream_t s) {
  if (d == 16) return walk_n<BF, 16>(a, n, rev, out, s);
  if (d == 64) return walk_n<BF, 64>(a, n, rev, out, s);
  return walk_n<BF, 128>(a, n, rev, out, s);
}

template <bool BF>
hipError_t prep(const M2ScanArgs& a, int n, hipStream_t s) {
  const dim3 grid((unsigned)scan_slots(a.N, a.total, kScanChunk), (unsigned)a.G);
  if (n == 16) gdn_m2s_prep_kernel<BF, 16><<<grid, 256, 0, s>>>(a);
  else if (n == 64) gdn_m2s_prep_kernel<BF, 64><<<grid, 256, 0, s>>>(a);
  else gdn_m2s_prep_kernel<BF, 128><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

// Sizes decide two things (bf16, d = 64, n = 128; us for the whole call, whole
// sequences unless a number of chunks is given):
//  - Waves of 16 state rows, a head a workgroup, where the waves of 32 would be
//    fewer than two workgroups a compute unit: four prompts (20,408 tokens) x
//    128 heads 665 narrow, 767 wide; 32 x 1024 tokens x 128 heads 713 and 685.
//  - Segments only where there are few walks, as they cost a second walk and the
//    states' way through memory: backward of 4 x 4096 tokens x 128 heads (512
//    walks) 1415 whole, 1910 in segments of 58; the four prompts 665 and 917; of
//    16,385 tokens x 32 heads (32 walks) 1745 whole, 558 in segments of 12.
//    Their length leaves 704 workgroups, close to three a compute unit.
//    Walks enough for that, but not for two workgroups of 128 rows a compute
//    unit, and of little work (3 to 12 chunks a workgroup of the 704, sequences
//    that average a chunk or more): if they are ragged, the longest sequence
//    decides, so sequences of more than two segments are cut.  The lengths lie
//    on the device.  Whole and cut: 20 sequences of 0 to 1500 tokens x 32 heads
//    106 and 75; 12 of 1 to 3000 x 64 heads 244 and 114; 8 of 1 to 6000 x 32
//    heads 310 and 142; 30 of 1 to 4000 x 32 heads 202 and 208.  Where nothing
//    is cut the two launches more cost 5 to 11: 10 of 500 to 1000 x 64 heads 112
//    and 117, 20 of 245 x 32 heads 45 and 55, 20 of 500 71 and 82.  With more
//    walks: 24 of 0 to 800 x 48 heads 164 and 200, 16 of 100 to 1500 x 64 heads
//    213 and 226, so those stay whole.
ScanPlan scan_plan(int64_t N, int64_t total, int H, int G, int d) {
  const int hpg = H / G, wide_heads = (d == 16 ? 64 : 128) / d;
  const int64_t chunks = (total + kScanChunk - 1) / kScanChunk, wide = (int64_t)G * ((hpg + wide_heads - 1) / wide_heads);
  ScanPlan p;
  p.narrow = d == 64 && N * wide < 512;
  const int64_t walks = p.narrow ? H : wide;
  p.seg_chunks = 0;
  const bool few = N * walks < 384;
  p.whole = few ? 1 : 2;
  if (chunks > 8 && (few || (N * wide < 512 && N <= chunks && chunks * walks >= 3 * 704 && chunks * walks <= 12 * 704))) {
    const int64_t per = (chunks * walks / 704 + 1) / 2 * 2;
    p.seg_chunks = per < 4 ? 4 : (int)per;
  }
  return p;
}

int64_t scan_work_items(int64_t N, int64_t total, int H, int G, int d) {
  const ScanPlan p = scan_plan(N, total, H, G, d);
  const int heads = p.narrow ? 1 : (d == 16 ? 64 : 128) / d;  // a workgroup's
  const int64_t slots = p.seg_chunks > 0 ? scan_slots(N, total, (int64_t)p.seg_chunks * kScanChunk) : N;
  return std::max(scan_slots(N, total, kScanChunk), slots * G * ((H / G + heads - 1) / heads)) * 256;
}

hipError_t launch_scan_prep(const M2ScanArgs& a, bool bf, int n, hipStream_t s) {
  return bf ? prep<true>(a, n, s) : prep<false>(a, n, s);
}

// The walk over all sequences, with the segments' first walk and their chain
// where a.seg_chunks is set.  out: write outputs (else states only).
hipError_t launch_scan_walk(M2ScanArgs a, bool bf, int d, int n, bool rev, bool out, hipStream_t s) {
  auto go = [&](const M2ScanArgs& b, bool o) { return bf ? walk_dn<true>(b, d, n, rev, o, s) : walk_dn<false>(b, d, n, rev, o, s); };
  if (a.seg_chunks > 0) {
    M2ScanArgs b = a;
    b.local = 1;
    b.blocks = nullptr;
    hipError_t e = go(b, false);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((d * n + 1023) / 1024), (unsigned)a.H, (unsigned)a.N);
    if (rev) gdn_m2s_chain_kernel<true><<<grid, 256, 0, s>>>(a, d * n);
    else gdn_m2s_chain_kernel<false><<<grid, 256, 0, s>>>(a, d * n);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  a.local = 0;
  return go(a, out);
}

}  // namespace gdn
