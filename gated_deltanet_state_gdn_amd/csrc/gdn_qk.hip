// RMS norm of every head of the queries and keys and the rotation by the
// token's position behind it, in one pass, and its reverse.
//
// Per head of d values, with r = (mean x^2 + eps)^-1/2 and n = x r w, pair i of
// the first `rot` values turns by the angle p f_i:
//     (a, b) -> (a cos - b sin, b cos + a sin).
// In reverse the gradient turns back, dn = rot(dy, -angle), and with xh = x r
//     dw = sum dn xh,   dx = r (dn w - xh mean(dn w xh)),
// where mean(dn w xh) = r mean(dn w x): both sums of a row are taken at once.
//
// A row (one head of one token) lies on d / 8 lanes rounded up to a power of
// two, 8 values a lane as two vectors of 4: those of four pairs, so a rotation
// never leaves its lane.  A workgroup takes a few tokens at a time: first its
// threads form the tokens' cosines and sines, one pair a thread, in LDS (the
// angle's turns as a sum of two FP64 numbers, reduced to a quarter turn before
// they are rounded to FP32), then
// its rows of lanes go over all heads of these tokens, so that a token's angles
// are formed once for all its heads.  A row is fetched under the one before it.
//
// What bounds it is memory: 20,408 tokens of 32 and 16 heads of 128 take 95 us,
// 5.3 TB/s, and back 16,384 of 32 and 32 take 153, 5.3 TB/s, where a large copy
// reaches 4.7 (vector units are active 77 and 68% of the time).  Four and two
// rows in flight in place of one took 104 and 177 us (registers, so fewer
// waves); rows are never kept for a second pass.  Three tokens take 4.5 us, all
// latency: loads, the angles and the barrier behind them, a row, its store.
#include <algorithm>

#include "gdn_device.h"
#include "gdn_launch.h"

namespace gdn {

namespace {

constexpr int kQkThreads = 256;

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// Sum over LPR neighbouring lanes, in every one of them.
template <int LPR>
__device__ __forceinline__ float lanes_sum(float x) {
  if constexpr (LPR >= 2) x = dpp_add<0xB1>(x);    // lane ^ 1
  if constexpr (LPR >= 4) x = dpp_add<0x4E>(x);    // lane ^ 2
  if constexpr (LPR >= 8) x = dpp_add<0x141>(x);   // mirrored in 8: the other quad
  if constexpr (LPR >= 16) x = dpp_add<0x140>(x);  // mirrored in 16: the other half
  if constexpr (LPR >= 32) {
    const unsigned a = __builtin_bit_cast(unsigned, x);
    const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    unsigned r0 = r[0], r1 = r[1];
    asm volatile("" : "+v"(r0), "+v"(r1));
    x = __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
  }
  return x;
}

// cos and sin of p f: turns, of which the whole and then the quarter ones are
// dropped exactly; what is left, at most an eighth, is rounded to FP32.  The
// product and 1 / (2 pi) are sums of two FP64 numbers each: single ones would be
// off by up to 2^-22 radians where p f is 2^31, several steps of a sine.  (No
// product may be fused with the subtraction behind it here: its rest is added
// apart.)
__device__ __forceinline__ void cos_sin(int p, float f, float& c, float& s) {
#pragma clang fp contract(off)
  constexpr double kTurns = 0x1.45f306dc9c883p-3, kTurnsRest = -0x1.6b01ec5417056p-57;  // 1 / (2 pi), and what it leaves
  const double x = (double)p * (double)f, x_rest = fma((double)p, (double)f, -x);
  double t = x * kTurns;
  const double t_rest = fma(x, kTurns, -t) + fma(x_rest, kTurns, x * kTurnsRest);
  t = 4.0 * ((t - rint(t)) + t_rest);
  const double quarter = rint(t);
  float sr, cr;
  sincospif(0.5f * (float)(t - quarter), &sr, &cr);
  const int k = (int)quarter;
  c = k & 1 ? sr : cr;
  s = k & 1 ? cr : sr;
  if ((k + 1) & 2) c = -c;
  if (k & 2) s = -s;
}

template <int IDT, int LPR, bool NB, bool BWD>
__global__ void __launch_bounds__(kQkThreads) gdn_qk_kernel(const QkArgs a) {
  constexpr int G = kQkThreads / LPR;  // rows at a time
  extern __shared__ __align__(16) float s_turn[];  // [tokens][2][rot / 2]; backward also [G][d]
  const int tid = threadIdx.x, r = tid % LPR, row0 = tid / LPR + G * blockIdx.y, step = G * gridDim.y;
  const int half = a.rot / 2, d = a.d;
  const bool on = 8 * r < d, turned = 8 * r < a.rot;
  // the lane's two vectors of 4
  const int o1 = !on ? 0 : NB || !turned ? 8 * r : 4 * r, o2 = !on ? 4 : NB || !turned ? 8 * r + 4 : half + 4 * r;
  float acc[BWD ? 2 : 1][8];
  if constexpr (BWD)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[s][e] = 0.f;
  float w[2][8];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[s][e] = a.w[s][o1 + e];
      w[s][4 + e] = a.w[s][o2 + e];
    }
  const float inv_d = 1.f / (float)d;

  const int64_t turns = (a.T + a.tokens - 1) / a.tokens;
  const int dt0 = step / a.heads[0], dh0 = step - dt0 * a.heads[0], dt1 = step / a.heads[1], dh1 = step - dt1 * a.heads[1];
  for (int64_t turn_at = blockIdx.x; turn_at < turns; turn_at += gridDim.x) {
    const int64_t t0 = turn_at * a.tokens;
    const int n = (int)min((int64_t)a.tokens, a.T - t0);
    struct Row {
      int t, h;
      InVec<IDT, 4> x1, x2, g1, g2;
    } row, next;
    auto load = [&](Row& q, int s) __attribute__((always_inline)) {
      const int64_t xo = (t0 + q.t) * a.x_ts[s] + (int64_t)q.h * d;
      q.x1.load(a.x[s], xo + o1);
      q.x2.load(a.x[s], xo + o2);
      if constexpr (BWD) {
        const int64_t go = (t0 + q.t) * a.dy_ts[s] + (int64_t)q.h * d;
        q.g1.load(a.dy[s], go + o1);
        q.g2.load(a.dy[s], go + o2);
      }
    };
    next.t = row0 / a.heads[0];
    next.h = row0 - next.t * a.heads[0];
    if (row0 < n * a.heads[0]) load(next, 0);  // on its way while the angles are formed
    if (turn_at != blockIdx.x) __syncthreads();  // the tokens before are done with
    for (int i = tid; i < n * half; i += kQkThreads) {
      const int k = i / half, p = i - k * half;
      const int axis = (a.axis[p >> 4] >> (2 * (p & 15))) & 3;
      float c, s;
      cos_sin(a.pos[axis * a.T + t0 + k], a.freq[p], c, s);
      s_turn[2 * k * half + p] = c;
      s_turn[(2 * k + 1) * half + p] = BWD ? -s : s;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int rows = n * a.heads[s];
      if (s == 1) {
        next.t = row0 / a.heads[1];
        next.h = row0 - next.t * a.heads[1];
        if (row0 < rows) load(next, 1);
      }
      for (int i = row0; i < rows; i += step) {
        row = next;
        next.t += s == 0 ? dt0 : dt1;
        next.h += s == 0 ? dh0 : dh1;
        if (next.h >= a.heads[s]) {
          next.h -= a.heads[s];
          ++next.t;
        }
        if (i + step < rows) load(next, s);
        float x[8], y[8];
        {
          float f[4], f2[4];
          row.x1.widen(f);
          row.x2.widen(f2);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = on ? f[e] : 0.f;
            x[4 + e] = on ? f2[e] : 0.f;
          }
        }
        const float* cs = s_turn + 2 * row.t * half + 4 * (turned ? r : 0);
        float c[4], sn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c[e] = turned ? cs[e] : 1.f;
          sn[e] = turned ? cs[half + e] : 0.f;
        }
        auto turn = [&](float (&v)[8]) __attribute__((always_inline)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = NB ? 2 * e : e, j = NB ? 2 * e + 1 : 4 + e;
            const float p = v[i], q = v[j];
            v[i] = p * c[e] - q * sn[e];
            v[j] = q * c[e] + p * sn[e];
          }
        };
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
        if constexpr (!BWD) {
          const float rstd = rsqrtf(lanes_sum<LPR>(sum) * inv_d + a.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e] * rstd * w[s][e];
          turn(y);
        } else {
          float f[4], f2[4];
          row.g1.widen(f);
          row.g2.widen(f2);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] = on ? f[e] : 0.f;
            y[4 + e] = on ? f2[e] : 0.f;
          }
          turn(y);
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) dot = fmaf(y[e] * w[s][e], x[e], dot);
          const float rstd = rsqrtf(lanes_sum<LPR>(sum) * inv_d + a.eps);
          const float m = lanes_sum<LPR>(dot) * rstd * inv_d;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float xh = x[e] * rstd;
            acc[BWD ? s : 0][e] = fmaf(y[e], xh, acc[BWD ? s : 0][e]);
            y[e] = rstd * fmaf(-xh, m, y[e] * w[s][e]);
          }
        }
        if (on) {
          const int64_t yo = (t0 + row.t) * a.y_ts[s] + (int64_t)row.h * d;
          const float lo[4] = {y[0], y[1], y[2], y[3]}, hi[4] = {y[4], y[5], y[6], y[7]};
          store_vec<4>(a.y[s], yo + o1, lo, IDT, true);
          store_vec<4>(a.y[s], yo + o2, hi, IDT, true);
        }
      }
    }
  }
  if constexpr (BWD) {
    // the workgroup's sums over its rows of lanes, in order
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      __syncthreads();
      float* row = s_turn + (tid / LPR) * d;
      if (on)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          row[o1 + e] = acc[s][e];
          row[o2 + e] = acc[s][4 + e];
        }
      __syncthreads();
      if (tid < d) {
        float sum = 0.f;
        for (int g = 0; g < G; ++g) sum += s_turn[g * d + tid];
        a.part[((int64_t)blockIdx.x * 2 + s) * d + tid] = sum;
      }
    }
  }
}

// Adds the workgroups' partial weight gradients in a fixed order: 16 columns a
// workgroup, a 64th of the workgroups' sums a row of threads, four in flight.
__global__ void __launch_bounds__(1024) gdn_qk_sum_kernel(const QkArgs a, int blocks) {
  __shared__ float s_sum[64][17];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4, col = blockIdx.x * 16 + x, d = a.d;
  float sum = 0.f;
  if (col < 2 * d) {
    const float* p = a.part + col;
    for (int b = y; b < blocks; b += 4 * 64) {
      float f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = b + 64 * k < blocks ? p[(int64_t)(b + 64 * k) * 2 * d] : 0.f;
      sum += (f[0] + f[1]) + (f[2] + f[3]);
    }
  }
  s_sum[y][x] = sum;
  __syncthreads();
  if (threadIdx.x < 64) {  // a column a row of 16 lanes' place, 16 sums each
    const int c = threadIdx.x & 15, k0 = threadIdx.x >> 4;
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) sum += s_sum[k0 + 4 * k][c];
    sum = xor_sum_from<16>(sum);
    if (k0 == 0 && col < 2 * d) (col < d ? a.dw[0] : a.dw[1])[col < d ? col : col - d] = sum;
  }
}

int lanes_of_row(int d) {
  int l = 2;
  while (8 * l < d) l *= 2;
  return l;
}

// Tokens of a workgroup's turn: eight rounds of its rows, so that angles and
// the barrier behind them are shared, but as many workgroups as given.
int turn_tokens(int64_t T, int heads, int d, int workgroups) {
  const int rows = kQkThreads / lanes_of_row(d);
  const int64_t t = std::min<int64_t>(16, std::max(1, 8 * rows / heads));
  return (int)std::max<int64_t>(1, std::min(t, (T + workgroups - 1) / workgroups));
}
// Forward (4096 tokens of 32 and 8 heads of 128: 19.9 us with 2048 workgroups, 21.3 with 4096, 18.9 with 1024, but 2500 tokens
// 12.9, 13.7 and 13.7; 16,384 tokens of 64 and 8 heads take 113 with any).  Backward, four a compute unit, which are all there
// at once (16,384 tokens: 178 us with 1024, 190 with 768, 199 with 1536, 182 with 2048).
constexpr int kQkForward = 2048, kQkBackward = 1024;

template <int IDT, int LPR, bool BWD>
hipError_t launch(const QkArgs& a, dim3 grid, size_t lds, hipStream_t s) {
  if (a.neighbours) gdn_qk_kernel<IDT, LPR, true, BWD><<<grid, kQkThreads, lds, s>>>(a);
  else gdn_qk_kernel<IDT, LPR, false, BWD><<<grid, kQkThreads, lds, s>>>(a);
  return hipGetLastError();
}

template <int IDT, bool BWD>
hipError_t launch_lanes(const QkArgs& a, dim3 grid, size_t lds, hipStream_t s) {
  switch (lanes_of_row(a.d)) {
    case 2: return launch<IDT, 2, BWD>(a, grid, lds, s);
    case 4: return launch<IDT, 4, BWD>(a, grid, lds, s);
    case 8: return launch<IDT, 8, BWD>(a, grid, lds, s);
    case 16: return launch<IDT, 16, BWD>(a, grid, lds, s);
    default: return launch<IDT, 32, BWD>(a, grid, lds, s);
  }
}

template <bool BWD>
hipError_t launch_type(const QkArgs& a, dim3 grid, size_t lds, hipStream_t s) {
  if (a.in_dt == GDN_F32) return launch_lanes<GDN_F32, BWD>(a, grid, lds, s);
  if (a.in_dt == GDN_BF16) return launch_lanes<GDN_BF16, BWD>(a, grid, lds, s);
  return launch_lanes<GDN_F16, BWD>(a, grid, lds, s);
}

}  // namespace

hipError_t launch_qk(QkArgs a, hipStream_t s) {
  const int heads = a.heads[0] + a.heads[1], rows = kQkThreads / lanes_of_row(a.d);
  a.tokens = turn_tokens(a.T, heads, a.d, kQkForward);
  dim3 grid((unsigned)std::min<int64_t>((a.T + a.tokens - 1) / a.tokens, 1 << 20));
  // few tokens: their heads on several workgroups (32 and 8 heads of 128: one token 3.4 us and without 3.8, 511 tokens 5.6 and
  // 6.0, but 1024 tokens 8.5 and 7.8)
  if (a.T < 512) grid.y = (unsigned)std::min((std::max(a.heads[0], a.heads[1]) + rows - 1) / rows, 64);
  return launch_type<false>(a, grid, (size_t)a.tokens * a.rot * 4, s);
}

// Workgroups of the backward pass, each with a partial sum of the weights'
// gradients.
int qk_bwd_blocks(int64_t T, int heads, int d) {
  const int t = turn_tokens(T, heads, d, kQkBackward);
  return (int)std::min<int64_t>((T + t - 1) / t, kQkBackward);
}

hipError_t launch_qk_bwd(QkArgs a, hipStream_t s) {
  const int blocks = a.T > 0 ? qk_bwd_blocks(a.T, a.heads[0] + a.heads[1], a.d) : 0;
  if (blocks > 0) {
    a.tokens = turn_tokens(a.T, a.heads[0] + a.heads[1], a.d, kQkBackward);
    const size_t lds = std::max((size_t)a.tokens * a.rot * 4, (size_t)(kQkThreads / lanes_of_row(a.d)) * a.d * 4);
    const hipError_t e = launch_type<true>(a, dim3((unsigned)blocks), lds, s);
    if (e != hipSuccess) return e;
  }
  gdn_qk_sum_kernel<<<(2 * a.d + 15) / 16, 1024, 0, s>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace gdn
