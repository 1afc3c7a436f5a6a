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
// slice, at most 2 vectors of 8 values each; a workgroup walks rows with its
// weights (and, backward, its part of dw and db) in registers.  Rows start at
// any element: vectors are read and written at the element's own alignment.
// The variance is taken from the deviations, not from a difference of sums.
// All sums are FP32.  The backward pass writes one row of partial dw and db a
// workgroup, and a second kernel adds them in a fixed order: no atomics, so
// equal calls give equal bits.
#include "gdn_device.h"
#include "gdn_launch.h"

namespace gdn {

constexpr int kNormMaxSlice = 16384;  // 1024 lanes x 2 vectors of 8
constexpr int norm_threads(int lpu) { return lpu > 256 ? lpu : 256; }

// ------------------------------------------------------------------ vectors at element alignment
typedef u32x4 u32x4_e2 __attribute__((aligned(2)));
typedef u32x4 u32x4_e4 __attribute__((aligned(4)));

// 8 values from element i; those at or past `left` read as zero.
template <int DT>
__device__ __forceinline__ void norm_load(const void* p, int64_t i, int left, float (&f)[8]) {
  if (left >= 8) {
    if constexpr (DT == GDN_F32) {
      const auto* q = reinterpret_cast<const u32x4_e4*>(static_cast<const float*>(p) + i);
      const u32x4 a = q[0], b = q[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = __uint_as_float(a[e]);
        f[4 + e] = __uint_as_float(b[e]);
      }
    } else {
      const u32x4 a = *reinterpret_cast<const u32x4_e2*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] = unpack_lo<DT>(a[e]);
        f[2 * e + 1] = unpack_hi<DT>(a[e]);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e < left ? load_elem(p, i + e, DT) : 0.f;
  }
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

template <int IDT, int LPU, int CH, bool GATE>
__global__ void __launch_bounds__(norm_threads(LPU)) gdn_norm_fwd_kernel(const NormArgs a) {
  constexpr int UPW = norm_threads(LPU) / LPU;
  __shared__ float part[2][2][16];
  const int sub = threadIdx.x / LPU, l = threadIdx.x % LPU;
  const int n = a.N / a.groups, g = blockIdx.y, col0 = g * n;
  float w[CH][8], b[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e0 = (c * LPU + l) * 8;
    norm_load<GDN_F32>(a.w, col0 + e0, n - e0, w[c]);
    if (a.b != nullptr) norm_load<GDN_F32>(a.b, col0 + e0, n - e0, b[c]);
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
      norm_load<IDT>(a.x, row * a.x_stride + col0 + e0, n - e0, u[c]);
      if constexpr (GATE) norm_load<IDT>(a.z, row * a.z_stride + col0 + e0, n - e0, z[c]);
    }
    if constexpr (GATE) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          z[c][e] *= sigmoid_f(z[c][e]);
          if (!a.gate_after) u[c][e] *= z[c][e];
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
        if constexpr (GATE)
          if (a.gate_after) u[c][e] *= z[c][e];
      }
      norm_store_as(a.y, row * a.y_stride + col0 + e0, n - e0, u[c], a.out_dt);
    }
  }
}

template <int IDT, int LPU, int CH, bool GATE>
__global__ void __launch_bounds__(norm_threads(LPU)) gdn_norm_bwd_kernel(const NormArgs a) {
  constexpr int UPW = norm_threads(LPU) / LPU;
  __shared__ float part[2][2][16];
  __shared__ float s_acc[UPW > 1 ? 4 : 1][UPW > 1 ? LPU * 8 : 1];
  const int sub = threadIdx.x / LPU, l = threadIdx.x % LPU, wave = threadIdx.x >> 6;
  const int n = a.N / a.groups, g = blockIdx.y, col0 = g * n;
  float w[CH][8], dw[CH][8], db[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e0 = (c * LPU + l) * 8;
    norm_load<GDN_F32>(a.w, col0 + e0, n - e0, w[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[c][e] = db[c][e] = 0.f;
  }
  const float inv = 1.f / (float)n;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * UPW + sub; row < a.rows; row += (int64_t)gridDim.x * UPW, turn ^= 1) {
    const float m = a.rms ? 0.f : a.mean[row * a.groups + g], r = a.rstd[row * a.groups + g];
    float h[CH][8], v[CH][8], x[GATE ? CH : 1][8], z[GATE ? CH : 1][8];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * LPU + l) * 8;
      norm_load<IDT>(a.x, row * a.x_stride + col0 + e0, n - e0, h[c]);
      norm_load<IDT>(a.dy, row * a.dy_stride + col0 + e0, n - e0, v[c]);
      if constexpr (GATE) norm_load<IDT>(a.z, row * a.z_stride + col0 + e0, n - e0, z[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * LPU + l) * 8;
      float bias[8];
      if constexpr (GATE)
        if (a.gate_after && a.b != nullptr) norm_load<GDN_F32>(a.b, col0 + e0, n - e0, bias);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float gate = 1.f, slope = 0.f;
        if constexpr (GATE) {
          const float zz = z[c][e], s = sigmoid_f(zz);
          gate = zz * s;
          slope = s * (1.f + zz * (1.f - s));
          x[c][e] = h[c][e];
          if (!a.gate_after) h[c][e] *= gate;
        }
        h[c][e] = e0 + e < n ? (h[c][e] - m) * r : 0.f;
        if constexpr (GATE) {
          if (a.gate_after) {
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
        if constexpr (GATE)
          if (!a.gate_after) {
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

// dw and db from the workgroups' partial rows: 64 columns a workgroup, its 16
// waves over the rows, each adding its rows in order, then the waves in order.
// Columns [0, N) are dw, [N, 2 N) db.
__global__ void __launch_bounds__(1024) gdn_norm_sum_kernel(const float* part, int blocks, int N, float* dw, float* db) {
  __shared__ float s[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  float t = 0.f;
  if (col < 2 * N) {
#pragma unroll 4
    for (int i = wave; i < blocks; i += 16) t += part[(int64_t)i * 2 * N + col];
  }
  s[wave][lane] = t;
  __syncthreads();
  if (wave != 0 || col >= 2 * N) return;
  t = s[0][lane];
#pragma unroll
  for (int i = 1; i < 16; ++i) t += s[i][lane];
  if (col < N) dw[col] = t;
  else if (db != nullptr) db[col - N] = t;
}

// ------------------------------------------------------------------ host
namespace {

struct NormGeom {
  int lpu, ch;
};
// Lanes for a slice of n: at most 2 vectors of 8 a lane, which leaves the
// backward kernel's weights, sums and up to three tensors in its registers.
NormGeom norm_geom(int n) {
  if (n <= 128) return {16, 1};
  if (n <= 512) return {64, 1};
  if (n <= 1024) return {64, 2};
  if (n <= 2048) return {256, 1};
  if (n <= 4096) return {256, 2};
  if (n <= 8192) return {512, 2};
  return {1024, 2};
}

int64_t row_blocks(int64_t rows, int lpu, int groups, int64_t most) {
  const int64_t upw = norm_threads(lpu) / lpu, need = (rows + upw - 1) / upw;
  const int64_t cap = most / groups > 0 ? most / groups : 1;
  return need < cap ? need : cap;
}

}  // namespace

bool norm_slice_fits(int n) { return n <= kNormMaxSlice; }

// Workgroups of the backward kernel a group: enough to fill 256 compute units
// four deep over all groups, no more, since each writes 2 N floats.
int norm_bwd_blocks(int64_t rows, int N, int groups) {
  return (int)row_blocks(rows, norm_geom(N / groups).lpu, groups, 1024);
}

#define GDN_NORM_LAUNCH(KERNEL, IDT, LPU, CH)                                               \
  do {                                                                                      \
    if (a.z != nullptr) KERNEL<IDT, LPU, CH, true><<<grid, norm_threads(LPU), 0, s>>>(a);        \
    else KERNEL<IDT, LPU, CH, false><<<grid, norm_threads(LPU), 0, s>>>(a);                      \
  } while (0)
#define GDN_NORM_GEOM(KERNEL, IDT)                                                          \
  do {                                                                                      \
    if (q.lpu == 16) GDN_NORM_LAUNCH(KERNEL, IDT, 16, 1);                                   \
    else if (q.lpu == 64 && q.ch == 1) GDN_NORM_LAUNCH(KERNEL, IDT, 64, 1);                 \
    else if (q.lpu == 64) GDN_NORM_LAUNCH(KERNEL, IDT, 64, 2);                              \
    else if (q.ch == 1) GDN_NORM_LAUNCH(KERNEL, IDT, 256, 1);                               \
    else if (q.lpu == 256) GDN_NORM_LAUNCH(KERNEL, IDT, 256, 2);                              \
    else if (q.lpu == 512) GDN_NORM_LAUNCH(KERNEL, IDT, 512, 2);                            \
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
  const dim3 grid((unsigned)row_blocks(a.rows, q.lpu, a.groups, 2048), (unsigned)a.groups);
  GDN_NORM_TYPE(gdn_norm_fwd_kernel);
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  const NormGeom q = norm_geom(a.N / a.groups);
  const int blocks = norm_bwd_blocks(a.rows, a.N, a.groups);
  if (blocks > 0) {
    const dim3 grid((unsigned)blocks, (unsigned)a.groups);
    GDN_NORM_TYPE(gdn_norm_bwd_kernel);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  gdn_norm_sum_kernel<<<(2 * a.N + 63) / 64, 1024, 0, s>>>(a.part, blocks, a.N, a.dw, a.db);
  return hipGetLastError();
}

}  // namespace gdn
