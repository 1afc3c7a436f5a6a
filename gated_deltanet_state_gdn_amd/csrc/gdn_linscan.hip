// Linear attention with a fixed decay a head over packed sequences, forward
// and backward.
//
// Per head, S_t = e^g S_{t-1} + k_t v_t^T and o_t = scale S_t^T q_t.  Over a
// chunk of 64 tokens (i, j from 0) with S before it and p[m] = e^{g m}:
//     o_i = scale (p[i+1] S^T q_i + sum_{j<=i} p[i-j] (q_i.k_j) v_j)
//     S'  = p[64] S + sum_j p[63-j] k_j v_j^T.
// The gradients are walks of the same form with the tensors in other places:
// with do the gradient of o and dS that of the state behind a chunk,
//     dq_i = scale (p[i+1] S do_i + sum_{j<=i} p[i-j] (do_i.v_j) k_j)
//     dv_j = p[63-j] dS^T k_j + scale sum_{i>=j} p[i-j] (k_j.q_i) do_i
//     dk_j = p[63-j] dS  v_j + scale sum_{i>=j} p[i-j] (v_j.do_i) q_i
//     dS  <- p[64] dS + scale sum_i p[i+1] q_i do_i^T.
// So one kernel has a read, a write and an input tensor (q, k, v for o) and a
// direction, and a backward pass runs three of these walks side by side.  The
// p[m] are a table of 65 numbers for all chunks; exponents never grow.
//
// A workgroup walks one head of a sequence (or segment) with the state in
// accumulators, transposed so that it meets the read vectors straight from
// them: lane l holds the rows 8 (l / 16) + .. of column l % 16.  All operands
// of a chunk lie in LDS as they do in memory, row by row; operands that run
// over tokens are read transposed (the 16-bit transposing LDS reads), so nothing
// is stored twice.  Blocks of 8 values of a row are permuted by the row's number
// so that both kinds of reads meet all banks (464 cycles of conflicts a chunk of
// 128 x 128; rows permuted for 16 lanes in a row have some 650 more).  The chunk
// behind the next is fetched into registers, and the next one put into LDS, under
// the work on this one: two barriers a chunk.  80 KB of LDS, so that two
// workgroups fit a compute unit.
//
// Where there are too few walks for the chip, sequences are cut into segments:
// a first walk finds each segment's own end state, a small kernel chains them,
// and the second walk starts every segment from its true state.
//
// What bounds it: 16 sequences of 2048 tokens x 32 heads of 128 in BF16 take 318
// us, 3.4 TB/s of inputs and outputs where a large copy reaches 4.7.  No unit is at
// its limit (matrix units busy 39% of the time, vector units 45%, LDS 26%): the
// four waves of a workgroup meet at two barriers a chunk, which takes 10 us, and
// two workgroups on a compute unit do not lay all loads, splits and products under
// one another.  That is this schedule's bound, not a floor.  Heads of 64 reach 3.8
// TB/s (64 x 2048 tokens x 32 heads 572 us).  In FP32 one workgroup fits a compute
// unit from heads of 64 on and the matrix units are busy 52%: 16 x 1024 tokens x
// 32 heads of 64 take 202 us, 16 x 2048 x 32 of 128 956.  FP16 runs as FP32, its
// values widened as they come: 1384 us for those.  Eight waves of 16 columns, in
// place of four of 32, took 362 us for 324 (the read vectors are then read twice
// as often); three workgroups a compute unit in the segments' first walk, with
// one buffer each, gained nothing.
//
// Rounding (bf16 inputs and outputs): products of two inputs are exact in FP32.
// The state is FP32.  Wherever the matrix instructions take an FP32 number, that
// is the weighted inputs of an update, the state and the weighted products that
// an output reads, they take it in three bf16 terms, all its 24 bits, beside
// exact inputs.  (Two terms of what outputs read take 7% less for prompts and 11%
// for gradients, but outputs are then 1.0e-4 of their size from an FP32 scan's,
// where the order of sums alone leaves 0.3e-4, and sums over shared heads have 16
// bits.)  The wave that forms a product also splits it, once for the four that
// read it.  Any other types take the FP32 MFMA throughout.
#include <algorithm>

#include "gdn_m2scan.h"

namespace gdn {

namespace {

constexpr int Q = kScanChunk;

template <bool BF, int D, bool OUT>
struct LinGeom {
  typedef typename Frag<BF>::E E;
  static constexpr int PT = D < 128 ? 1 : 2;           // 16-column tiles of a wave
  static constexpr int NW = D / (16 * PT);             // waves
  static constexpr int THREADS = 64 * NW;
  static constexpr int NT = D / 16, KB = (D + 31) / 32;
  static constexpr int LD = BF ? D : D + 4;            // rows of the operands
  // The weighted products: ten tiles of 16 x 16, each as 32 cells of 8 writing tokens of one reading token, in three bf16 terms or in
  // FP32.  Cells are 48 bytes apart, 12 banks, so that 16 of them meet all banks.
  static constexpr int CELL = 48, TILE = 32 * CELL, PB = OUT ? 10 * TILE : 0;
  static constexpr int TPW = (10 + NW - 1) / NW;       // 16 x 16 tiles of them that a wave forms
  // read vectors, inputs (twice without outputs), write vectors twice, products
  static constexpr int X0 = OUT ? Q * LD : 0, W0 = X0 + (OUT ? 1 : 2) * Q * LD, ELEMS = W0 + 2 * Q * LD;
  static constexpr int TABLE = 64 + 64 + 16 + 68;      // floats: p[63], .., p[0]; scale p[63], .., scale p[0]; zeros; scale p[0..64]
  static constexpr size_t LDS = (size_t)ELEMS * sizeof(E) + PB + TABLE * 4;
  static constexpr int VPR = D / 8;                    // 8-element vectors of a row
  static constexpr int SV = Q * VPR / THREADS;         // and those that a thread stages of an operand
  static_assert(SV * THREADS == Q * VPR && ELEMS * sizeof(E) % 16 == 0, "whole vectors");
};

// Where the 8-value block c of row t lies: blocks are permuted by the row, so
// that 16 rows of one block, and 4 rows of 4 blocks, meet all banks.
template <bool BF, int D>
__device__ __forceinline__ int block_at(int t, int c) {
  if constexpr (!BF) return t * (D + 4) + 8 * c;
  const int g = ((t >> 2 ^ t >> 3) & 1) << 1 | (t >> 3 & 1);
  const int f = D == 128 ? (t & 3) << 2 | g : D == 64 ? (t >> 1 & 1) << 2 | g : D == 32 ? g : t >> 3 & 1;
  return t * D + ((c ^ f) << 3);
}

// Four 16-bit values of one column, from four rows of 16 columns of which lane
// l of 16 points at row l / 4, columns 4 (l % 4) and on.
__device__ __forceinline__ u32x2 read_transposed(const uint16_t* p) {
  typedef short i16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) i16x4* Lds;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(const_cast<uint16_t*>(p))));
}

// A decay in powers of two; an infinite one is left finite, so that over 0 tokens it is 0.
__device__ __forceinline__ double log2_of_decay(float g) { return 1.4426950408889634 * (g == -INFINITY ? -1e300 : (double)g); }

// Segments behind a sequence's first: segment c > 0 of sequence s has the slot floor(cu[s] / P) + c - 1, distinct for all
// sequences, since P (ceil(len / P) - 1) < len.  A slot's sequence, if it has one, is the last with floor(cu[s] / P) <= slot.
// Slots in front of the first sequence come out with an index below 1.
__device__ __forceinline__ Piece whole_sequence(const int32_t* cu, int64_t total, int seq) {
  Piece p;
  p.seq = seq;
  p.begin = token_at(cu, seq, total);
  p.len = max(token_at(cu, seq + 1, total) - p.begin, (int64_t)0);
  p.index = 0;
  p.count = 1;
  return p;
}

__device__ __forceinline__ Piece find_other_segment(const int32_t* cu, int N, int64_t total, int slot, int P) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = N;  // the answer lies in [lo, hi), or is s = 0
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) >> 6;
    const int s = lo + lane * step;
    const int n = __popcll(__ballot(s < hi && cu[min(s, N)] / P <= slot));
    const int nlo = lo + max(n - 1, 0) * step;  // the condition holds on a prefix
    hi = __builtin_amdgcn_readfirstlane(min(hi, nlo + step));
    lo = __builtin_amdgcn_readfirstlane(nlo);
  }
  Piece p = whole_sequence(cu, total, lo);
  p.index = slot - (int)(p.begin / P) + 1;
  return p;
}

template <bool BF, int D, bool OUT>
__global__ void __launch_bounds__((LinGeom<BF, D, OUT>::THREADS), (BF || D < 128 ? 2 : 1)) gdn_linear_walk_kernel(const LinScanArgs a) {
  using W = LinGeom<BF, D, OUT>;
  typedef typename W::E E;
  constexpr int PT = W::PT, NW = W::NW, NT = W::NT, KB = W::KB, LD = W::LD, THREADS = W::THREADS, VPR = W::VPR, SV = W::SV, TPW = W::TPW;
  extern __shared__ __align__(16) unsigned char smem[];
  E* const s_r = reinterpret_cast<E*>(smem);
  E* const s_x = reinterpret_cast<E*>(smem) + W::X0;
  E* const s_w = reinterpret_cast<E*>(smem) + W::W0;  // [2]
  unsigned char* const s_p = smem + (size_t)W::ELEMS * sizeof(E);
  // tables: s_a[m] = scale p[m] for m to 64, and zero for -16 <= m < 0; s_b[i] = p[63 - i], and numbers that meet zeros alone behind
  // them; s_c[i] = scale p[63 - i], and zero for 64 <= i < 80
  float* const s_b = reinterpret_cast<float*>(s_p + W::PB);
  float* const s_c = s_b + 64;
  float* const s_a = s_c + 80;

  // Places: all sequences' first segments (or the sequences whole), then the other segments.  The roles, and the heads that
  // share a tensor's head, are neighbours on one XCD (workgroup i of a launch goes to XCD i mod 8).  Of whole sequences each
  // XCD takes a run, whose heads' tokens share its L2 (256 x 512 tokens x 32 heads of 32 263 us, round the XCDs 332, of 64 498 and
  // 520; of 128, and 64 x 2048 of 64, no difference).  Segments, whose places are not all used, go round the XCDs.
  const int inner = a.bunch * a.roles, groups = a.H / a.bunch;
  int u;
  if (a.seg_chunks == 0) {
    const int units = a.N * a.H * a.roles;
    if ((int)blockIdx.x >= units) return;
    u = xcd_unit(blockIdx.x, units);
  } else {
    const int k = blockIdx.x >> 3;
    u = ((k / inner) * 8 + (blockIdx.x & 7)) * inner + k % inner;
  }
  const int group = u / inner, in_group = u - group * inner;
  const int place = group / groups;
  if (place >= a.N + a.extras) return;
  const bool first = place < a.N;
  const int h = (group - place * groups) * a.bunch + in_group / a.roles;
  const LinRole& ro = a.role[in_group % a.roles];
  int tid = threadIdx.x, l16 = tid & 15, q = tid >> 4 & 3;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool rev = ro.rev;
  Piece sg = first ? whole_sequence(a.cu, a.total, place) : find_other_segment(a.cu, a.N, a.total, place - a.N, a.seg_chunks * Q);
  if (a.seg_chunks > 0) {
    sg.count = (int)((sg.len + a.seg_chunks * Q - 1) / (a.seg_chunks * Q));
    if (!first && (sg.index < 1 || sg.index >= sg.count)) return;
  }
  const bool last_seg = rev ? sg.index == 0 : sg.index == sg.count - 1;
  if (!OUT && last_seg) return;  // nothing starts from this segment's end
  const int chunks = (int)((sg.len + Q - 1) / Q);
  const int c_lo = sg.index * a.seg_chunks;
  const int c_hi = sg.count > 1 ? min(chunks, c_lo + a.seg_chunks) : chunks;
  const int p0 = wave * 16 * PT;  // the wave's columns
  const int64_t out_ts = (int64_t)a.H * D;

  if (!state_live(a.live, a.live_slots, sg.seq)) {  // a padded sequence: zero outputs, no state
    if (OUT)
      for (int64_t i = tid; i < (int64_t)(c_hi - c_lo) * Q * D; i += THREADS) {
        const int64_t t = sg.begin + (int64_t)c_lo * Q + i / D;
        if (t < sg.begin + sg.len) store_elem(ro.out, t * out_ts + h * D + i % D, 0.f, ro.out_dt);
      }
    if (OUT && ro.fin.base != nullptr && ro.fin.slots == nullptr && last_seg)
      for (int i = tid; i < D * D; i += THREADS) store_elem(ro.fin.base, ((int64_t)sg.seq * a.H + h) * D * D + i, 0.f, ro.fin.dtype);
    return;
  }

  // ---- a chunk's operands: from memory two chunks ahead, in registers, then to LDS one chunk ahead
  Frag<BF> vr[OUT ? SV : 1], vw[SV], vx[SV];
  auto fetch_one = [&](auto& v, const void* base, int64_t ts, int64_t t0, int head, int len) __attribute__((always_inline)) {
    const int st = tid / VPR, sc = tid % VPR;  // the thread's first row, and its block of the row
    if constexpr (BF) {
      const auto w = window(base, t0 * ts + head * D, 2, 2 * ((len - 1) * ts + D));
      const int off = 2 * (st * (int)ts + 8 * sc);
#pragma unroll
      for (int k = 0; k < SV; ++k) v[k].v = __builtin_amdgcn_raw_buffer_load_b128(w, off + 2 * k * (THREADS / VPR) * (int)ts, 0, 0);
    } else {
#pragma unroll
      for (int k = 0; k < SV; ++k) {
        const int t = st + k * (THREADS / VPR);
        v[k] = Frag<BF>::zero();
        if (t < len) v[k] = frag_from<BF>(base, t0 * ts + head * D, t * (uint32_t)ts + 8 * sc, a.in_dt);
      }
    }
  };
  const int steps = c_hi - c_lo;
  const int hr = h / ro.read_share, hw = h / ro.write_share, hx = h / ro.in_share;
  auto chunk_of = [&](int step) { return rev ? c_hi - 1 - step : c_lo + step; };
  auto fetch = [&](int step) __attribute__((always_inline)) {
    if (step >= steps) return;
    const int64_t t0 = sg.begin + (int64_t)chunk_of(step) * Q;
    const int len = (int)min((int64_t)Q, sg.begin + sg.len - t0);
    if constexpr (OUT) fetch_one(vr, ro.read, ro.read_ts, t0, hr, len);
    fetch_one(vw, ro.write, ro.write_ts, t0, hw, len);
    fetch_one(vx, ro.in, ro.in_ts, t0, hx, len);
  };
  auto commit = [&](int step) __attribute__((always_inline)) {
    if (step >= steps) return;
    E* const w = s_w + (step & 1) * Q * LD;
    E* const x = s_x + (OUT ? 0 : (step & 1) * Q * LD);
    const int st = tid / VPR, sc = tid % VPR;
#pragma unroll
    for (int k = 0; k < SV; ++k) {
      const int at = block_at<BF, D>(st + k * (THREADS / VPR), sc);
      if constexpr (OUT) *reinterpret_cast<Frag<BF>*>(s_r + at) = vr[k];
      *reinterpret_cast<Frag<BF>*>(w + at) = vw[k];
      *reinterpret_cast<Frag<BF>*>(x + at) = vx[k];
    }
  };
  fetch(0);

  const double log2_decay = log2_of_decay(a.log_decay[h]);
  auto power = [&](int m) __attribute__((always_inline)) {  // p[m]: the exponent's whole part apart, so the rest loses nothing
    const double x = log2_decay * m, n = fmin(fmax(rint(x), -400.0), 400.0);
    return ldexpf(exp2f((float)(x - n)), (int)n);
  };
  // Powers past the sequence's length meet rows of zeros alone, and are zero: where the state grows they may be infinite.
  const int most = (int)min((int64_t)Q, sg.len);
  for (int m = tid - 16; m <= Q; m += THREADS) {
    const float p = m >= 0 && m <= most ? power(m) : 0.f;
    s_a[m] = a.scale * p;
    if (m >= 0 && m < Q) {
      s_b[Q - 1 - m] = p;
      s_c[Q - 1 - m] = a.scale * p;
    }
  }
  const float whole_decay = power(Q);

  // The state S[nt][pt][r]: its row (a value of the write vector) is row_of(nt, 4 q + r), its column column_of(pt, l16): eight
  // neighbours of a row or column in a lane's registers, where a head has so many.
  f32x4 S[NT][PT];
  auto row_of = [&](int nt, int m) { return D == 16 ? m : 32 * (nt >> 1) + 8 * (m >> 2) + 4 * (nt & 1) + (m & 3); };
  auto column_of = [&](int pt, int m) { return p0 + (PT == 1 ? m : 8 * (m >> 2) + 4 * pt + (m & 3)); };
  // its elements in memory: one lane offset, and a uniform one an element
  const int sn = ro.transposed ? 1 : D, sp = ro.transposed ? D : 1;
  const int state_at = row_of(0, 4 * q) * sn + column_of(0, l16) * sp;
  auto load_as = [&](const void* base, int64_t unit, auto type) __attribute__((always_inline)) {
    constexpr int DT = decltype(type)::value, EB = DT == GDN_F32 ? 4 : 2;
    const auto w = window(base, (unit * a.H + h) * D * D, EB, EB * D * D);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        float f[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = EB * (row_of(nt, r) * sn + 4 * pt * sp);
          if constexpr (EB == 4) f[r] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(w, EB * state_at, at, 0));
          else f[r] = in_value<DT>(__builtin_amdgcn_raw_buffer_load_b16(w, EB * state_at, at, 0));
        }
        S[nt][pt] = f32x4{f[0], f[1], f[2], f[3]};
      }
  };
  auto store_as = [&](void* base, int64_t unit, auto type) __attribute__((always_inline)) {
    constexpr int DT = decltype(type)::value, EB = DT == GDN_F32 ? 4 : 2;
    const auto w = window(base, (unit * a.H + h) * D * D, EB, EB * D * D);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = EB * (row_of(nt, r) * sn + 4 * pt * sp);
          const float f = S[nt][pt][r];
          if constexpr (EB == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, f), w, EB * state_at, at, 0);
          else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack2<DT == GDN_F32 ? GDN_BF16 : DT>(f, 0.f), w, EB * state_at, at, 0);
        }
  };
  if (OUT && (sg.count > 1 || ro.init.base != nullptr)) {
    const bool cut = sg.count > 1;
    const void* const base = cut ? ro.seg : ro.init.base;
    const int64_t unit = cut ? place : ro.init.slots != nullptr ? ro.init.slots[sg.seq] : sg.seq;
    const int dt = cut ? (int)GDN_F32 : ro.init.dtype;
    if (dt == GDN_F32) load_as(base, unit, std::integral_constant<int, GDN_F32>{});
    else if (dt == GDN_BF16) load_as(base, unit, std::integral_constant<int, GDN_BF16>{});
    else load_as(base, unit, std::integral_constant<int, GDN_F16>{});
  } else {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) S[nt][pt] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // ---- fragments.  The lane's places in the first block of 32 columns (see block_at); `along` goes on by whole such blocks.
  auto along = [](int at, int kb) __attribute__((always_inline)) { return BF ? at ^ (32 * kb) : at + 32 * kb; };
  // row 16 rt + l16, the values of block kb in the order of the state's rows
  auto row_frag = [&](const E* s, int rt, int kb) __attribute__((always_inline)) {
    if constexpr (D >= 32) return Frag<BF>::load(s + 16 * rt * LD + along(block_at<BF, D>(l16, q), kb));
    Frag<BF> f = Frag<BF>::zero();
    const E* p = s + 16 * rt * LD + block_at<BF, D>(l16, q >> 1) + 4 * (q & 1);
    if constexpr (BF) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(p);
      f.v[0] = v[0];
      f.v[1] = v[1];
    } else {
      f.a = *reinterpret_cast<const f32x4*>(p);
    }
    return f;
  };
  // tokens 32 ks + 8 q and on of a column a lane: l16's of sixteen, of which lanes point at four each.  A tile of the state's rows:
  auto write_frag = [&](const E* s, int nt, int ks) __attribute__((always_inline)) {
    if constexpr (BF) {
      const int t = 8 * q + (l16 >> 2), c = l16 & 3;
      u32x2 v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = D == 16 ? block_at<BF, D>(t + 4 * h, c >> 1) + 4 * (c & 1) : along(block_at<BF, D>(t + 4 * h, c), nt >> 1) + 4 * (nt & 1);
        v[h] = read_transposed(s + 32 * ks * LD + at);
      }
      return Frag<BF>{u32x4{v[0][0], v[0][1], v[1][0], v[1][1]}};
    } else {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = s[(32 * ks + 8 * q + e) * LD + row_of(nt, l16)];
      return Frag<BF>::round(f);
    }
  };
  // and of the wave's columns
  auto in_frag = [&](int step, int pt, int ks) __attribute__((always_inline)) {
    const E* const s = s_x + (OUT ? 0 : (step & 1) * Q * LD) + 32 * ks * LD;
    if constexpr (BF) {
      const int t = 8 * q + (l16 >> 2), c = l16 & 3;
      u32x2 v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = PT == 1 ? block_at<BF, D>(t + 4 * h, 2 * wave + (c >> 1)) + 4 * (c & 1) : along(block_at<BF, D>(t + 4 * h, c), wave) + 4 * pt;
        v[h] = read_transposed(s + at);
      }
      return Frag<BF>{u32x4{v[0][0], v[0][1], v[1][0], v[1][1]}};
    } else {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = s[(8 * q + e) * LD + column_of(pt, l16)];
      return Frag<BF>::round(f);
    }
  };

  // ---- the weighted products: the wave's 16 x 16 tiles on and below the diagonal (above it in reverse).  A lane has four writing
  // tokens of one reading token.  The last tile goes to several waves where the tiles do not go round.
  // Tiles lie in the order in which they are read (see below), whose rows and columns stand in two bits a tile.
  const int turn = rev ? 1 : 0;
  int prt[TPW], pct[TPW];
#pragma unroll
  for (int k = 0; k < TPW; ++k) {
    const int t = 2 * min(wave + k * NW, 9);
    prt[k] = (rev ? 0x4143a : 0xfbe94) >> t & 3;  // forward 0 1 1 2 2 3 3 2 3 3, in reverse 2 2 3 0 0 1 1 0 0 1
    pct[k] = (rev ? 0x53bbe : 0xe9110) >> t & 3;  // forward 0 0 1 0 1 0 1 2 2 3, in reverse 2 3 3 2 3 2 3 0 1 1
  }
  auto products = [&](int step) __attribute__((always_inline)) {
    if (step >= steps) return;
    const E* const w = s_w + (step & 1) * Q * LD;
    f32x4 acc[TPW];
#pragma unroll
    for (int k = 0; k < TPW; ++k) acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int k = 0; k < TPW; ++k) acc[k] = frag_mma(acc[k], row_frag(w, pct[k], kb), row_frag(s_r, prt[k], kb));
#pragma unroll
    for (int k = 0; k < TPW; ++k) {
      const int rt = prt[k], ct = pct[k], m0 = 16 * rt + l16 - 16 * ct - 4 * q;
      const float* const p = (rev ? s_a : s_c + Q - 1) - m0;  // scale p[|m0 - r|] on the diagonal and to its one side, zero on the other
      float f[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) f[r] = acc[k][r] * p[r];
      unsigned char* const cell = s_p + min(wave + k * NW, 9) * W::TILE + (16 * (q >> 1) + l16) * W::CELL;
      if constexpr (BF) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const u32x2 term = {pack2<GDN_BF16>(f[0], f[1]), pack2<GDN_BF16>(f[2], f[3])};
          *reinterpret_cast<u32x2*>(cell + 16 * i + 8 * (q & 1)) = term;
          if (i < 2) {
            bf16_rest(term[0], f[0], f[1]);
            bf16_rest(term[1], f[2], f[3]);
          }
        }
      } else {
        *reinterpret_cast<f32x4*>(cell + 16 * (q & 1)) = f32x4{f[0], f[1], f[2], f[3]};
      }
    }
  };

  if (steps > 0) {
    commit(0);
    fetch(1);
    __syncthreads();
    if constexpr (OUT) products(0);
  }
  for (int step = 0; step < steps; ++step) {
    const int64_t t0 = sg.begin + (int64_t)chunk_of(step) * Q;
    const int len = (int)min((int64_t)Q, sg.begin + sg.len - t0);
    // the lane's places are not known to be the ones of the chunk before: what follows from them is formed anew, in a few
    // instructions, where it would otherwise be kept in registers that the loop has not got
    asm volatile("" : "+v"(tid));
    tid &= THREADS - 1;
    l16 = tid & 15;
    q = tid >> 4 & 3;
    // what tokens see of the state, and how much of their input reaches the next
    const float* const tell = rev ? s_b + Q - len : s_a + 1;
    const float* const keep = rev ? s_a + 1 : s_b + Q - len;
    // In reverse blocks of 16 tokens and halves of 32 go in the order 2 3 0 1 and 1 0, so that the half of the writing tokens
    // that reading tokens do not meet has the same place.
    Frag<BF> xf[2][PT];
    if constexpr (OUT) {
      // the state's part of the output, transposed: acc[pt][i][r] = (column column_of(pt, 4 q + r), token 16 (i ^ 2 turn) + l16)
      f32x4 acc[PT][4];
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) acc[pt][rt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        typedef Split<BF> Terms;
        Frag<BF> rf[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) rf[rt] = row_frag(s_r, rt ^ 2 * turn, kb);
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
#pragma unroll
        for (int k = Terms::K - 1; k >= 0; --k)
#pragma unroll
          for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) acc[pt][rt] = frag_mma(acc[pt][rt], sf[pt].t[k], rf[rt]);
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) xf[ks][pt] = in_frag(step, pt, ks ^ turn);
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        const float f = tell[16 * (rt ^ 2 * turn) + l16];
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) acc[pt][rt] *= f;
      }
      __syncthreads();  // the products are there, and read vectors and inputs done with
      commit(step + 1);
      __builtin_amdgcn_sched_barrier(0);
      fetch(step + 2);
      __builtin_amdgcn_sched_barrier(0);
      // Blocks 0 to 3 of reading tokens with the first half of the writing ones, 2 and 3 with the second: 12 pairs of a block and 16
      // writing tokens, of which two lie beyond the diagonal.  They have no tile, and their lanes read zeros.
      const unsigned char* const at = s_p + (q >> 1) * W::TILE + (16 * (q & 1) + l16) * W::CELL;
      const unsigned char* const zeros = reinterpret_cast<const unsigned char*>(s_a - 16);
#pragma unroll
      for (int i = 0; i < 6; i += 2) {  // two blocks at a time, so that a product never follows the one it adds to
        const int ks = i >= 4, rt = i - 2 * ks;
        constexpr int first[6] = {0, 1, 3, 5, 7, 8}, K = Split<BF>::K;
        Frag<BF> pf[2][K];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool none = i != 2 && (j == 0 ? !rev && q >= 2 : rev && q < 2);
          const unsigned char* const p = none ? zeros : at + first[i + j] * W::TILE;
#pragma unroll
          for (int k = 0; k < K; ++k) pf[j][k] = Frag<BF>::load(reinterpret_cast<const E*>(p + 16 * k));
        }
#pragma unroll
        for (int k = K - 1; k >= 0; --k)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) acc[pt][rt + j] = frag_mma(acc[pt][rt + j], xf[ks][pt], pf[j][k]);
      }
      if (BF && ro.out_dt == GDN_BF16) {
        const auto w = window(ro.out, t0 * out_ts + h * D + p0, 2, 2 * ((len - 1) * out_ts + 16 * PT));
        const int off = 2 * (l16 * (int)out_ts + 4 * PT * q);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          uint32_t v[2 * PT];
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) {
            v[2 * pt] = pack2<GDN_BF16>(acc[pt][rt][0], acc[pt][rt][1]);
            v[2 * pt + 1] = pack2<GDN_BF16>(acc[pt][rt][2], acc[pt][rt][3]);
          }
          if constexpr (PT == 2) __builtin_amdgcn_raw_buffer_store_b128(u32x4{v[0], v[1], v[2], v[3]}, w, off + 32 * (rt ^ 2 * turn) * (int)out_ts, 0, 0);
          else __builtin_amdgcn_raw_buffer_store_b64(u32x2{v[0], v[1]}, w, off + 32 * (rt ^ 2 * turn) * (int)out_ts, 0, 0);
        }
      } else {
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          const int t = 16 * (rt ^ 2 * turn) + l16;
          if (t < len)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) {
              const float v[4] = {acc[pt][rt][0], acc[pt][rt][1], acc[pt][rt][2], acc[pt][rt][3]};
              store_vec<4>(ro.out, (t0 + t) * out_ts + h * D + p0 + 4 * PT * q + 4 * pt, v, ro.out_dt, true);
            }
        }
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) xf[ks][pt] = in_frag(step, pt, ks ^ turn);
      commit(step + 1);
      __builtin_amdgcn_sched_barrier(0);
      fetch(step + 2);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (OUT) {
      __syncthreads();  // the next operands are there, and the products done with
      products(step + 1);
    }

    // the state after the chunk
    const E* const w = s_w + (step & 1) * Q * LD;
    const float dec = len == Q ? whole_decay : s_b[Q - 1 - len];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) S[nt][pt] *= dec;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      float wt[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) wt[e] = keep[32 * (ks ^ turn) + 8 * q + e];
      Split<BF> xs[PT];
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        float f[8];
        xf[ks][pt].widen(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= wt[e];
        xs[pt] = Split<BF>::of(f);
      }
      constexpr int NG = NT < 4 ? NT : 4;  // tiles at a time, their terms apart: a product never follows the one it adds to
#pragma unroll
      for (int ng = 0; ng < NT; ng += NG) {
        Frag<BF> wf[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i) wf[i] = write_frag(w, ng + i, ks ^ turn);
#pragma unroll
        for (int k = Split<BF>::K - 1; k >= 0; --k)
#pragma unroll
          for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) S[ng + i][pt] = frag_mma(S[ng + i][pt], wf[i], xs[pt].t[k]);
      }
    }
    if constexpr (!OUT) __syncthreads();  // the next operands are there, and these done with
  }

  if (!OUT || (ro.fin.base != nullptr && last_seg && (rev || sg.len > 0))) {
    void* const base = OUT ? ro.fin.base : ro.seg;
    const int64_t unit = !OUT ? place : ro.fin.slots != nullptr ? ro.fin.slots[sg.seq] : sg.seq;
    const int dt = OUT ? ro.fin.dtype : (int)GDN_F32;
    if (dt == GDN_F32) store_as(base, unit, std::integral_constant<int, GDN_F32>{});
    else if (dt == GDN_BF16) store_as(base, unit, std::integral_constant<int, GDN_BF16>{});
    else store_as(base, unit, std::integral_constant<int, GDN_F16>{});
  }
}

// ------------------------------------------------------------------ chain
// Turns the segments' own end states into the states they start from, in
// place: per (sequence, head), four state elements a thread.
__global__ void __launch_bounds__(256) gdn_linear_chain_kernel(const LinScanArgs a, int elems, int parts) {
  const LinRole& ro = a.role[blockIdx.y];
  const int unit = blockIdx.x / parts, seq = unit / a.H, h = unit - seq * a.H;
  const int i = ((blockIdx.x - unit * parts) * 256 + threadIdx.x) * 4;
  if (i >= elems || !state_live(a.live, a.live_slots, seq)) return;
  const int P = a.seg_chunks * Q;
  const int64_t b = token_at(a.cu, seq, a.total), e = token_at(a.cu, seq + 1, a.total);
  const int count = (int)max((e - b + P - 1) / P, (int64_t)1);
  if (count <= 1) return;
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (ro.init.base != nullptr) {
    float f[4];
    load_vec<4>(ro.init.base, ((ro.init.slots != nullptr ? ro.init.slots[seq] : (int64_t)seq) * a.H + h) * elems + i, ro.init.dtype, f);
    S = f32x4{f[0], f[1], f[2], f[3]};
  }
  const double g = log2_of_decay(a.log_decay[h]);
  const float whole = (float)exp2(g * P);
  const float tail = (float)exp2(g * (double)(e - b - (int64_t)(count - 1) * P));  // the sequence's last segment
  for (int k = 0; k < count; ++k) {
    const int at = ro.rev ? count - 1 - k : k;
    f32x4* p = reinterpret_cast<f32x4*>(ro.seg + ((at == 0 ? seq : a.N + b / P + at - 1) * a.H + h) * elems + i);
    if (k + 1 < count) {
      const f32x4 own = *p;
      *p = S;
      S = S * (at == count - 1 ? tail : whole) + own;
    } else {
      *p = S;
    }
  }
}

// ------------------------------------------------------------------ shared heads
__global__ void __launch_bounds__(256) gdn_linear_sum_kernel(const LinSumArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.items) return;
  const int v = a.D / 4;
  const int64_t head = i / v;  // of all tokens
  if (head / a.heads < a.cu[0] || head / a.heads >= a.cu[a.N]) return;  // in no sequence
  const float* p = a.each + head * a.share * a.D + (i - head * v) * 4;
  f32x4 sum = *reinterpret_cast<const f32x4*>(p);
  for (int k = 1; k < a.share; ++k) sum += *reinterpret_cast<const f32x4*>(p + (int64_t)k * a.D);
  const float f[4] = {sum[0], sum[1], sum[2], sum[3]};
  store_vec<4>(a.out, i * 4, f, a.out_dt, true);
}

template <bool BF, int D, bool OUT>
hipError_t walk(const LinScanArgs& a, hipStream_t s) {
  using W = LinGeom<BF, D, OUT>;
  auto* k = gdn_linear_walk_kernel<BF, D, OUT>;
  static std::atomic<uint64_t> allowed{0};
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(k), W::LDS, allowed);
  if (e != hipSuccess) return e;
  const int64_t all = ((int64_t)a.N + a.extras) * a.H * a.roles, ways = 8 * (a.seg_chunks > 0 ? a.bunch * a.roles : 1);
  k<<<(unsigned)((all + ways - 1) / ways * ways), W::THREADS, W::LDS, s>>>(a);
  return hipGetLastError();
}

template <bool OUT>
hipError_t walk_any(const LinScanArgs& a, bool bf, int D, hipStream_t s) {
  if (bf) return D == 16 ? walk<true, 16, OUT>(a, s) : D == 32 ? walk<true, 32, OUT>(a, s) : D == 64 ? walk<true, 64, OUT>(a, s) : walk<true, 128, OUT>(a, s);
  return D == 16 ? walk<false, 16, OUT>(a, s) : D == 32 ? walk<false, 32, OUT>(a, s) : D == 64 ? walk<false, 64, OUT>(a, s) : walk<false, 128, OUT>(a, s);
}

}  // namespace

// The host knows how many sequences and tokens there are, not how long each sequence is.  In steps of a chunk, `room`
// workgroups at a time, sequences of equal lengths take `whole`; cut in segments of `per` chunks, of which ragged ones make a
// few more, `cut`: a start and end of some three steps among them, and two fifths for the segments' first walk and the chain.
// A lone workgroup on a compute unit takes 0.65 of the time that each of two takes.  In FP32 from 64 on one fits, and 224 leave
// some for what ragged lengths add (256 places filled exactly took 219 to 342 us from call to call, with room 255 to 270).
// Measured, us whole / cut: forward in heads of 128, 4 x 4096 tokens x 32 heads 350 / 258, prompts of 1024 to 8192 x 32 660 / 299
// (segments of 23 chunks; of 16 325, of 32 400), 8 x 2048 x 32 181 / 209, so whole; one of 16,384 x 16 heads of 64 666 / 79, 4 x 960 x 8
// 44 / 30; backward in heads of 128, 4 x 4096 x 32 523 / 545 and more, one of 16,385 x 16 1483 / 400 (segments of 16: 370); FP32, one
// of 4099 x 24 heads of 64 345 / 82, 4 x 2048 x 16 of 128 462 / 261.
// Several sequences that would stay whole by that may be long ones among short.  They are cut at a quarter above their mean
// length, which leaves nearly equal ones whole (16 of 905 to 1150 tokens x 32 heads of 64: 86 us, whole 77, at the mean length
// 105), or at five chunks where the chip is empty.  Whole / so: 16 of 33 to 8192 x 32 heads of 128 689 / 301, 16 of 100 to 2300 x 32 of
// 128 239 / 230 and of 64 backward x 16 136 / 126, 20 of 0 to 1500 x 32 of 64 73 / 56 and x 8 67 / 33, 6 of 60 to 1600 x 16 70 / 35.
// Equal lengths pay for two launches that find nothing to do: 20 of 215 tokens x 8 heads 18 / 24, 16 x 1024 x 32 of 64 78 / 88, 8 x 2048
// x 32 of 128 181 / 191, backward 4 x 4096 x 32 of 128 523 / 526.
// Above four times `room` walks, or below two chunks a sequence, batches stay whole, and a long sequence among many short ones is one
// walk: forward in 32 heads of 128 one of 8192 tokens with 63 of 200 takes 326 us (whole 705), with 64 of them 704 (394 in segments of
// 23 chunks), in 8 heads one of 8192 with 64 single tokens 635 (139 in segments of 16); backward one of 16,384 with 20 of 100 822 (whole
// 3169), with 21 of them 3166 (816 in segments of 26).
int linear_plan(int64_t N, int64_t total, int H, int D, bool bf, int roles) {
  int seg_chunks = 0;
  const int64_t chunks = (total + Q - 1) / Q, walks = N * H * roles;
  if (chunks <= 8) return 0;
  const int64_t room = !bf && D >= 64 ? 224 : 512;
  const int64_t length = (chunks + N - 1) / N;
  auto rounds = [&](int64_t w) { return (w + room - 1) / room; };
  double best = (double)(rounds(walks) * length) * (2 * walks <= room ? 0.65 : 1.0);
  for (int64_t per = std::max<int64_t>(4, length / 128); per < length; per += per / 32 + 1) {
    const int64_t segs = std::max(N * ((length + per - 1) / per), (4 * chunks + N * per + 4 * per - 1) / (4 * per));
    const double cut = rounds(segs * H * roles) * (per + 3.5) * (2 * segs * H * roles <= room ? 0.65 : 1.0) * 1.4;
    if (cut < best) {
      best = cut;
      seg_chunks = (int)per;
    }
  }
  if (seg_chunks == 0 && N > 1 && walks <= 4 * room && chunks >= 2 * N)
    seg_chunks = (int)(4 * walks <= room ? 5 : std::max<int64_t>(5, length + length / 4));
  return seg_chunks;
}

// The walks of roles 0 and on; backward, roles 1 and 2 go the same way over the
// same states, so the segments' first walk and the chain take roles 0 and 1.
hipError_t launch_linear_scan(LinScanArgs a, bool bf, int D, int roles, hipStream_t s) {
  a.extras = a.seg_chunks > 0 ? (int32_t)(a.total / (a.seg_chunks * Q)) : 0;
  if (a.extras == 0) a.seg_chunks = 0;  // no sequence is longer than a segment
  a.bunch = 1;
  for (int i = 0; i < roles; ++i) a.bunch = std::max({a.bunch, a.role[i].read_share, a.role[i].write_share, a.role[i].in_share});
  if (a.seg_chunks > 0) {
    const int passes = a.roles = std::min(roles, 2);
    hipError_t e = walk_any<false>(a, bf, D, s);
    if (e != hipSuccess) return e;
    const int parts = (D * D + 1023) / 1024;
    gdn_linear_chain_kernel<<<dim3((unsigned)((int64_t)a.N * a.H * parts), (unsigned)passes), 256, 0, s>>>(a, D * D, parts);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  a.roles = roles;
  return walk_any<true>(a, bf, D, s);
}

hipError_t launch_linear_sum(const LinSumArgs& a, hipStream_t s) {
  gdn_linear_sum_kernel<<<(unsigned)((a.items + 255) / 256), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace gdn
