// Layer and RMS norm of the slices of a row, forward and backward.
//
// A row of N values is `groups` slices of n = N / groups, each normalised on
// its own.  With u = x, or x silu(z) when the gate comes before the norm:
//     m = mean(u)  (0 in the RMS form),  r = (mean((u - m)^2) + eps)^-1/2,
//     h = (u - m) r,  v = h w + b,  y = v, or v silu(z) with the gate after.
// Backward, with dv = dy (or dy silu(z)) and e = dv w:
//     du = r (e - mean(e) [layer form only] - h mean(e h)),
//     dw = sum over rows of dv h,  db = sum over rows of dv,
// and the product rule at the gate, silu'(z) = s (1 + z (1 - s)), s = sigmoid(z).
//
// Both directions move each tensor once: a slice stays in registers from its
// load to its store, so they are bound by HBM.  LPU lanes (16 to 1024) hold a
// slice, a vector of 8 values each (two above 8192 values); a workgroup walks
// rows with its weights (and, backward, its part of dw and db) in registers.
// Rows start at any element: vectors are read and written at the element's own
// alignment, and one that would pass the slice's end is read from its last
// eight values and moved.  Measured, layer form with a bias in
// bf16 where not said (a copy reaches 5.1 to 5.4 TB/s): forward 20,408 rows of
// 4096 values 65 us, 5.2 TB/s, and of 8 slices of 1024, RMS with the gate
// before, 205 us, 4.9 TB/s; backward 16,384 rows of 4096 84 us, 4.8 TB/s;
// backward 16,384 rows of 8 slices of 1024, RMS with the gate before, 268 us,
// 5.0 TB/s; backward 40,001 rows of 128, RMS in FP32 with the gate behind, 22 us,
// 4.6 TB/s; backward 20,001 rows of 2047, which no vector fits, 63 us, 3.9 TB/s;
// backward 4000 rows of 16,384 with the gate before 255 us, 2.6 TB/s (its
// arithmetic spills); three rows of 8 slices: the call's latency, 13 us.
// The variance is taken from the deviations, not from a difference of sums.
// All sums are FP32.  The backward pass writes one row of partial dw and db a
// workgroup, and a second kernel adds them in a fixed order: no atomics, so
// equal calls give equal bits.
#include "gdn_device.h"
#include "gdn_launch.h"

namespace gdn {

constexpr int kNormMaxSlice = 16384;  // 1024 lanes x 2 vectors of 8
enum : int { kGateNone = 0, kGateBefore = 1, kGateAfter = 2 };
constexpr int norm_threads(int lpu) { return lpu > 64 ? lpu : 256; }

// ------------------------------------------------------------------ vectors at element alignment
typedef u32x4 u32x4_e2 __attribute__((aligned(2)));
typedef u32x4 u32x4_e4 __attribute__((aligned(4)));

// 8 values as they lie in memory.
template <int DT>
struct NormRaw {
  u32x4 v[DT == GDN_F32 ? 2 : 1];
};

// Values e0 to e0 + 7 of the slice of n values at element i.  One load without
// a branch: a vector that would pass the slice's end is taken to end there, and
// norm_open moves its values down.
template <int DT>
__device__ __forceinline__ NormRaw<DT> norm_fetch(const void* p, int64_t i, int e0, int n) {
  NormRaw<DT> r;
  if (n >= 8) {
    i += e0 < n - 8 ? e0 : n - 8;
    if constexpr (DT == GDN_F32) {
      const auto* q = reinterpret_cast<const u32x4_e4*>(static_cast<const float*>(p) + i);
      r.v[0] = q[0];
      r.v[1] = q[1];
    } else {
      r.v[0] = *reinterpret_cast<const u32x4_e2*>(static_cast<const uint16_t*>(p) + i);
    }
  } else {
#pragma unroll
    for (int e = 0; e < (DT == GDN_F32 ? 8 : 4); ++e) {
      uint32_t t = 0;
      if constexpr (DT == GDN_F32) {
        if (e0 + e < n) t = static_cast<const uint32_t*>(p)[i + e0 + e];
      } else {
        const auto* q = static_cast<const uint16_t*>(p) + i + e0;
        if (e0 + 2 * e < n) t = q[2 * e];
        if (e0 + 2 * e + 1 < n) t |= (uint32_t)q[2 * e + 1] << 16;
      }
      r.v[e >> 2][e & 3] = t;
    }
  }
  return r;
}

// The values of a fetched vector; those past the slice's end are zero.
template <int DT>
__device__ __forceinline__ void norm_open(const NormRaw<DT>& r, int e0, int n, float (&f)[8]) {
  constexpr int W = DT == GDN_F32 ? 8 : 4;
  uint32_t w[W];
#pragma unroll
  for (int e = 0; e < W; ++e) w[e] = r.v[e >> 2][e & 3];
  if (n >= 8 && e0 > n - 8) {
    const int by = e0 - (n - 8);  // values to move down
#pragma unroll
    for (int e = 0; e < W; ++e) w[e] = by < 8 ? w[e] : 0;
    const int words = DT == GDN_F32 ? by : by >> 1;
#pragma unroll
    for (int k = 1; k < W; k *= 2)
#pragma unroll
      for (int e = 0; e < W; ++e) w[e] = words & k ? (e + k < W ? w[e + k] : 0) : w[e];
    if (DT != GDN_F32 && (by & 1)) {
#pragma unroll
      for (int e = 0; e < W; ++e) w[e] = w[e] >> 16 | (e + 1 < W ? w[e + 1] << 16 : 0);
    }
  }
#pragma unroll
  for (int e = 0; e < W; ++e) {
    if constexpr (DT == GDN_F32) {
      f[e] = __uint_as_float(w[e]);
    } else {
      f[2 * e] = unpack_lo<DT>(w[e]);
      f[2 * e + 1] = unpack_hi<DT>(w[e]);
    }
  }
}

template <int DT>
__device__ __forceinline__ void norm_load(const void* p, int64_t i, int e0, int n, float (&f)[8]) {
  norm_open<DT>(norm_fetch<DT>(p, i, e0, n), e0, n, f);
}

// The first `left` of 8 values to element i, rounded once to nearest even.
template <int DT>
__device__ __forceinline__ void norm_store(void* p, int64_t i, int left, const float (&f)[8]) {
  if (left >= 8) {
    if constexpr (DT == GDN_F32) {
      auto* q = reinterpret_cast<u32x4_e4*>(static_cast<float*>(p) + i);
      u32x4 a, b;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = __float_as_uint(f[e]);
        b[e] = __float_as_uint(f[4 + e]);
      }
      q[0] = a;
      q[1] = b;
    } else {
      u32x4 a;
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = pack2<DT>(f[2 * e], f[2 * e + 1]);
      *reinterpret_cast<u32x4_e2*>(static_cast<uint16_t*>(p) + i) = a;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) store_elem(p, i + e, f[e], DT);
  }
}

__device__ __forceinline__ void norm_store_as(void* p, int64_t i, int left, const float (&f)[8], int dt) {
  if (dt == GDN_F32) norm_store<GDN_F32>(p, i, left, f);
  else if (dt == GDN_BF16) norm_store<GDN_BF16>(p, i, left, f);
  else norm_store<GDN_F16>(p, i, left, f);
}

// Sum over the LPU lanes of a slice, to every one of them.  Where they are
// several waves, those meet in `part` (one barrier; each call of a row has its
// own place, and rows alternate between two sets, so no second one is needed).
template <int LPU>
__device__ __forceinline__ float slice_sum(float x, float* part) {
  if constexpr (LPU == 16) {
    x += dpp_mov<0xB1>(x);
    x += dpp_mov<0x4E>(x);
    x += dpp_mov<0x128>(x);
    x += dpp_mov<0x124>(x);
    return x;
  } else if constexpr (LPU == 64) {
    return wave_sum(x);
  } else {
    x = wave_sum(x);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    float t = part[0];
#pragma unroll
    for (int w = 1; w < LPU / 64; ++w) t += part[w];
    return t;
  }
}

// sigmoid from a = e^-|x|, which cannot overflow: 1 / (1 + a), or a / (1 + a) for
// x < 0.  Without expf's steps for its range: a = (2^t 2^lo)^2, t + lo = -|x| log2 e / 2,
// 2^lo to first order; the hardware's exponential does not flush this root, so a
// keeps to the smallest numbers.  From 110 on a is zero.
__device__ __forceinline__ float norm_sigmoid(float x) {
  const float v = fmaxf(-fabsf(x), -110.f), t = v * 0.72134752f;
  const float lo = fmaf(v, 0.72134752f, -t) + v * 9.62981514e-9f;  // log2 e / 2 = 0.72134752 (in FP32) + 9.630e-9
  const float root = __builtin_amdgcn_exp2f(t), p = root * root;
  const float a = fmaf(p, lo * 1.38629436f, p), s = __builtin_amdgcn_rcpf(1.f + a);
  return x < 0.f ? a * s : s;
}

template <int IDT, int LPU, int CH, int GATE>
__global__ void __launch_bounds__(norm_threads(LPU)) gdn_norm_fwd_kernel(const NormArgs a) {
  constexpr int UPW = norm_threads(LPU) / LPU;
  __shared__ float part[2][2][16];
  const int sub = threadIdx.x / LPU, l = threadIdx.x % LPU;
  const int n = a.N / a.groups, g = blockIdx.y, col0 = g * n;
  float w[CH][8], b[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e0 = (c * LPU + l) * 8;
    norm_load<GDN_F32>(a.w, col0, e0, n, w[c]);
    if (a.b != nullptr) norm_load<GDN_F32>(a.b, col0, e0, n, b[c]);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) b[c][e] = 0.f;
  }
  const float inv = 1.f / (float)n;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * UPW + sub; row < a.rows; row += (int64_t)gridDim.x * UPW, turn ^= 1) {
    float u[CH][8], z[GATE ? CH : 1][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * LPU + l) * 8;
      norm_load<IDT>(a.x, row * a.x_stride + col0, e0, n, u[c]);
      if constexpr (GATE) norm_load<IDT>(a.z, row * a.z_stride + col0, e0, n, z[c]);
    }
    if constexpr (GATE) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          z[c][e] *= norm_sigmoid(z[c][e]);
          if constexpr (GATE == kGateBefore) u[c][e] *= z[c][e];
        }
    }
    float m = 0.f;
    if (!a.rms) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) m += u[c][e];
      m = slice_sum<LPU>(m, part[turn][0]) * inv;
    }
    float q = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[c][e] -= m;
        if ((c * LPU + l) * 8 + e < n) q += u[c][e] * u[c][e];
      }
    const float r = 1.f / sqrtf(slice_sum<LPU>(q, part[turn][1]) * inv + a.eps);
    if (l == 0 && a.rstd != nullptr) {
      a.mean[row * a.groups + g] = m;
      a.rstd[row * a.groups + g] = r;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * LPU + l) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[c][e] = u[c][e] * r * w[c][e] + b[c][e];
        if constexpr (GATE == kGateAfter) u[c][e] *= z[c][e];
      }
      norm_store_as(a.y, row * a.y_stride + col0 + e0, n - e0, u[c], a.out_dt);
    }
  }
}

template <int IDT, int LPU, int CH, int GATE>
__global__ void __launch_bounds__(norm_threads(LPU), 4) gdn_norm_bwd_kernel(const NormArgs a) {
  constexpr int UPW = norm_threads(LPU) / LPU;
  // Two vectors a lane: dw and db lie in LDS and the weights are read again for
  // each row, since 1024 lanes have 128 registers each.
  constexpr bool LEAN = CH == 2;
  // Whether a row is fetched while the one before it is worked on: where the
  // 128 registers hold it (20,001 rows of 2047 values 64 us with; 130 without
  // and with their last values read one by one; 40,001 gated rows of 128 in
  // FP32 32 us with, 26 without).
  constexpr bool AHEAD = !LEAN && !(GATE && (IDT == GDN_F32 || LPU >= 512));
  __shared__ float part[2][2][16];
  __shared__ float s_acc[UPW > 1 ? 4 : 1][UPW > 1 ? LPU * 8 : 1];
  __shared__ f32x4 s_sum[LEAN ? CH * 4 : 1][LEAN ? LPU : 1];
  const int sub = threadIdx.x / LPU, l = threadIdx.x % LPU, wave = threadIdx.x >> 6;
  const int n = a.N / a.groups, g = blockIdx.y, col0 = g * n;
  float w[CH][8], dw[CH][8], db[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    norm_load<GDN_F32>(a.w, col0, (c * LPU + l) * 8, n, w[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[c][e] = db[c][e] = 0.f;
    if constexpr (LEAN)
#pragma unroll
      for (int k = 0; k < 4; ++k) s_sum[c * 4 + k][l] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const float inv = 1.f / (float)n;
  int turn = 0;
  int64_t row = (int64_t)blockIdx.x * UPW + sub;
  const int64_t step = (int64_t)gridDim.x * UPW;
  NormRaw<IDT> rx[CH], rdy[CH], rz[GATE ? CH : 1];
  float m_next = 0.f, r_next = 0.f;
  auto fetch = [&](int64_t at) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * LPU + l) * 8;
      rx[c] = norm_fetch<IDT>(a.x, at * a.x_stride + col0, e0, n);
      rdy[c] = norm_fetch<IDT>(a.dy, at * a.dy_stride + col0, e0, n);
      if constexpr (GATE) rz[c] = norm_fetch<IDT>(a.z, at * a.z_stride + col0, e0, n);
    }
    if (!a.rms) m_next = a.mean[at * a.groups + g];
    r_next = a.rstd[at * a.groups + g];
  };
  if (AHEAD && row < a.rows) fetch(row);
  for (; row < a.rows; row += step, turn ^= 1) {
    if constexpr (!AHEAD) fetch(row);
    const float m = m_next, r = r_next;
    float h[CH][8], v[CH][8], x[GATE ? CH : 1][8], z[GATE ? CH : 1][8];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * LPU + l) * 8;
      norm_open<IDT>(rx[c], e0, n, h[c]);
      norm_open<IDT>(rdy[c], e0, n, v[c]);
      if constexpr (GATE) norm_open<IDT>(rz[c], e0, n, z[c]);
      if constexpr (LEAN) norm_load<GDN_F32>(a.w, col0, e0, n, w[c]);
    }
    // the next row is under way while this one is worked on
    if (AHEAD && row + step < a.rows) fetch(row + step);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * LPU + l) * 8;
      float bias[8];
      if constexpr (GATE == kGateAfter)
        if (a.b != nullptr) norm_load<GDN_F32>(a.b, col0, e0, n, bias);
      if constexpr (LEAN)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dw[c][e] = s_sum[c * 4 + (e >> 2)][l][e & 3];
          db[c][e] = s_sum[c * 4 + 2 + (e >> 2)][l][e & 3];
        }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float gate = 1.f, slope = 0.f;
        if constexpr (GATE) {
          const float zz = z[c][e], s = norm_sigmoid(zz);
          gate = zz * s;
          slope = s * (1.f + zz * (1.f - s));
          x[c][e] = h[c][e];
          if constexpr (GATE == kGateBefore) h[c][e] *= gate;
        }
        h[c][e] = (h[c][e] - m) * r;  // past the slice's end dy is zero, and with it what h adds
        if constexpr (GATE) {
          if constexpr (GATE == kGateAfter) {
            // z's gradient is complete here: dy v silu'(z)
            const float vv = h[c][e] * w[c][e] + (a.b != nullptr ? bias[e] : 0.f);
            z[c][e] = v[c][e] * vv * slope;
            v[c][e] *= gate;
          } else {
            z[c][e] = slope * x[c][e];  // du times this is z's gradient, du times the gate x's
            x[c][e] = gate;
          }
        }
        dw[c][e] += v[c][e] * h[c][e];
        db[c][e] += v[c][e];
        v[c][e] *= w[c][e];
        s1 += v[c][e];
        s2 += v[c][e] * h[c][e];
        // values two at a time: side by side their gates' steps take 100 registers more
        if (GATE && (e & 1)) __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (LEAN)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          s_sum[c * 4 + k][l] = f32x4{dw[c][4 * k], dw[c][4 * k + 1], dw[c][4 * k + 2], dw[c][4 * k + 3]};
          s_sum[c * 4 + 2 + k][l] = f32x4{db[c][4 * k], db[c][4 * k + 1], db[c][4 * k + 2], db[c][4 * k + 3]};
        }
    }
    s2 = slice_sum<LPU>(s2, part[turn][1]) * inv;
    s1 = a.rms ? 0.f : slice_sum<LPU>(s1, part[turn][0]) * inv;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * LPU + l) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[c][e] = r * (v[c][e] - s1 - h[c][e] * s2);
        if constexpr (GATE == kGateBefore) {
          z[c][e] *= v[c][e];
          v[c][e] *= x[c][e];
        }
      }
      norm_store<IDT>(a.dx, row * a.dx_stride + col0 + e0, n - e0, v[c]);
      if constexpr (GATE) norm_store<IDT>(a.dz, row * a.dz_stride + col0 + e0, n - e0, z[c]);
    }
  }
  // this workgroup's row of partial sums: dw then db, N values each
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.N + col0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * LPU + l) * 8;
      float(&acc)[8] = k == 0 ? dw[c] : db[c];
      if constexpr (LEAN)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = s_sum[c * 4 + 2 * k + (e >> 2)][l][e & 3];
      if constexpr (LPU == 16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = xor_sum_from<16>(acc[e]);
      }
      if constexpr (UPW > 1) {
        __syncthreads();
        if ((threadIdx.x & 63) < LPU)
#pragma unroll
          for (int e = 0; e < 8; ++e) s_acc[wave][l * 8 + e] = acc[e];
        __syncthreads();
        if (threadIdx.x < LPU)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = (s_acc[0][l * 8 + e] + s_acc[1][l * 8 + e]) + (s_acc[2][l * 8 + e] + s_acc[3][l * 8 + e]);
      }
      if (UPW == 1 || threadIdx.x < LPU) norm_store<GDN_F32>(out + (int64_t)k * a.N, e0, n - e0, acc);
    }
  }
}

// dw and db from the workgroups' partial rows: 32 columns a workgroup, its 32
// half waves over the rows, each adding its rows in order, then the half waves
// in order.  Columns [0, N) are dw, [N, 2 N) db.  Few workgroups and long
// chains: the eight loads in flight are what it lives on (2048 rows of 2 x 1000
// sums: a backward pass over 20,000 rows of 1000 values takes 30 us with them,
// 38 with 64 columns, 16 waves and four).
__global__ void __launch_bounds__(1024) gdn_norm_sum_kernel(const float* part, int blocks, int N, float* dw, float* db) {
  __shared__ float s[32][32];
  const int lane = threadIdx.x & 31, line = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float t = 0.f;
  if (col < 2 * N) {
#pragma unroll 8
    for (int i = line; i < blocks; i += 32) t += part[(int64_t)i * 2 * N + col];
  }
  s[line][lane] = t;
  __syncthreads();
  if (line != 0 || col >= 2 * N) return;
  t = s[0][lane];
#pragma unroll
  for (int i = 1; i < 32; ++i) t += s[i][lane];
  if (col < N) dw[col] = t;
  else if (db != nullptr) db[col - N] = t;
}

// ------------------------------------------------------------------ host
namespace {

struct NormGeom {
  int lpu, ch;
};
// Lanes for a slice of n: one vector of 8 a lane while a workgroup has the
// lanes.  A vector takes about 90 of the backward kernel's registers, 130 with a
// gate, of the 128 that leave 16 waves on a compute unit.  One vector against
// two: slices of 1024 with a gate 262 against 342 us, slices of 4096 84 against
// 92 (16,384 rows each).
NormGeom norm_geom(int n) {
  if (n <= 128) return {16, 1};
  if (n <= 512) return {64, 1};
  if (n <= 1024) return {128, 1};
  if (n <= 2048) return {256, 1};
  if (n <= 4096) return {512, 1};
  if (n <= 8192) return {1024, 1};
  return {1024, 2};
}

int64_t row_blocks(int64_t rows, int lpu, int groups, int64_t most) {
  const int64_t upw = norm_threads(lpu) / lpu, need = (rows + upw - 1) / upw;
  const int64_t cap = most / groups > 0 ? most / groups : 1;
  return need < cap ? need : cap;
}

}  // namespace

bool norm_slice_fits(int n) { return n <= kNormMaxSlice; }

// Workgroups of the backward kernel a group: over all groups as many as the
// card holds at 16 waves a compute unit, which its registers allow, so that all
// start together and take equal shares, and no more, since each writes 2 N floats.
int norm_bwd_blocks(int64_t rows, int N, int groups) {
  const int lpu = norm_geom(N / groups).lpu;
  return (int)row_blocks(rows, lpu, groups, 262144 / norm_threads(lpu));
}

#define GDN_NORM_LAUNCH(KERNEL, IDT, LPU, CH)                                               \
  do {                                                                                      \
    if (a.z == nullptr) KERNEL<IDT, LPU, CH, kGateNone><<<grid, norm_threads(LPU), 0, s>>>(a);    \
    else if (a.gate_after) KERNEL<IDT, LPU, CH, kGateAfter><<<grid, norm_threads(LPU), 0, s>>>(a); \
    else KERNEL<IDT, LPU, CH, kGateBefore><<<grid, norm_threads(LPU), 0, s>>>(a);                 \
  } while (0)
#define GDN_NORM_GEOM(KERNEL, IDT)                                                          \
  do {                                                                                      \
    if (q.lpu == 16) GDN_NORM_LAUNCH(KERNEL, IDT, 16, 1);                                   \
    else if (q.lpu == 64) GDN_NORM_LAUNCH(KERNEL, IDT, 64, 1);                 \
    else if (q.lpu == 128) GDN_NORM_LAUNCH(KERNEL, IDT, 128, 1);                            \
    else if (q.lpu == 256) GDN_NORM_LAUNCH(KERNEL, IDT, 256, 1);                            \
    else if (q.lpu == 512) GDN_NORM_LAUNCH(KERNEL, IDT, 512, 1);                            \
    else if (q.ch == 1) GDN_NORM_LAUNCH(KERNEL, IDT, 1024, 1);                              \
    else GDN_NORM_LAUNCH(KERNEL, IDT, 1024, 2);                                             \
  } while (0)
#define GDN_NORM_TYPE(KERNEL)                                                               \
  do {                                                                                      \
    if (a.in_dt == GDN_F32) GDN_NORM_GEOM(KERNEL, GDN_F32);                                 \
    else if (a.in_dt == GDN_BF16) GDN_NORM_GEOM(KERNEL, GDN_BF16);                          \
    else GDN_NORM_GEOM(KERNEL, GDN_F16);                                                    \
  } while (0)

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  const NormGeom q = norm_geom(a.N / a.groups);
  // workgroups over all groups: 20,408 rows of 8 slices of 1024 with a gate take 201 us with 2048 and 223 with 4096, 10,000
  // rows of 8192 85 and 89; 4096 is the better for 40,000 rows of 512 (16.1 and 14.7) and 20,408 of 2048 (33 and 28), and
  // other widths from 96 to 4096 take the same
  const dim3 grid((unsigned)row_blocks(a.rows, q.lpu, a.groups, 2048), (unsigned)a.groups);
  GDN_NORM_TYPE(gdn_norm_fwd_kernel);
  return hipGetLastError();
}

int64_t norm_sum_work_items(int N) { return (2 * (int64_t)N + 31) / 32 * 1024; }

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  const NormGeom q = norm_geom(a.N / a.groups);
  const int blocks = norm_bwd_blocks(a.rows, a.N, a.groups);
  if (blocks > 0) {
    const dim3 grid((unsigned)blocks, (unsigned)a.groups);
    GDN_NORM_TYPE(gdn_norm_bwd_kernel);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  gdn_norm_sum_kernel<<<(unsigned)(norm_sum_work_items(a.N) / 1024), 1024, 0, s>>>(a.part, blocks, a.N, a.dw, a.db);
  return hipGetLastError();
}

}  // namespace gdn
