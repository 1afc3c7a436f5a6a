// One token of linear attention with a fixed decay a head, for every sequence
// of a batch: S <- e^g S + k v^T and o = scale S^T q, the state read and
// written once.
//
// A workgroup takes CW columns of a D x D tile (D, or fewer where there are few
// tiles, as columns never meet): each lane owns VEC neighbouring columns, a
// wave RPW rows a pass, and the whole part is in flight before any arithmetic.
// q and k are staged in LDS while it comes.
//
// What bounds it is the state's way from and to memory: 256 sequences of 32
// heads of 128 x 128 in FP32 take 195 us, 5.5 TB/s of states read and written
// where a large copy reaches 4.7.  One sequence of 32 heads is all latency,
// 3.3 us of which the launch alone is some 2.
#include "gdn_device.h"
#include "gdn_launch.h"

namespace gdn {

namespace {

template <int SDT, int D, int CW>
struct StepGeom {
  static constexpr int MAXW = SDT == GDN_F32 ? 4 : 8;
  static constexpr int VEC0 = 16 / StateElem<SDT>::BYTES;
  static constexpr int VEC = 64 / (CW / VEC0) > D || CW < VEC0 ? VEC0 / 2 : VEC0;
  static constexpr int LPR = CW / VEC, RPW = 64 / LPR;
  static constexpr int NW = D / RPW < MAXW ? D / RPW : MAXW;
  static constexpr int PASSES = D / (RPW * NW);
  static_assert(LPR * VEC == CW && LPR * RPW == 64 && PASSES * RPW * NW == D, "tile geometry");
};

template <int SDT, int D, int CW, int IDT, bool NTL, bool NTS>
__global__ void __launch_bounds__((StepGeom<SDT, D, CW>::NW * 64)) gdn_linear_step_kernel(const LinStepArgs a) {
  using G = StepGeom<SDT, D, CW>;
  constexpr int VEC = G::VEC, LPR = G::LPR, RPW = G::RPW, NW = G::NW, PASSES = G::PASSES, NTH = NW * 64;
  using IO = TileIO<SDT, VEC, NTL>;
  using OUT = TileIO<SDT, VEC, NTS>;
  using ST = typename StateElem<SDT>::T;
  __shared__ __align__(16) float s_q[D], s_k[D], s_o[NW][CW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int u = blockIdx.x / (D / CW), part = blockIdx.x - u * (D / CW);
  const int b = u / a.H, h = u - b * a.H;
  const int c0 = part * CW + (lane % LPR) * VEC, r0 = wave * RPW + lane / LPR;
  const int64_t ob = ((int64_t)b * a.H + h) * D + part * CW;
  const int slot = a.slot_map[b];
  if (slot < 0 || (int64_t)slot >= a.num_slots) {  // padded row
    for (int i = tid; i < CW; i += NTH) store_elem(a.out, ob + i, 0.f, a.out_dt);
    return;
  }
  // the small loads first: loads complete in order, so their waits do not cover the tile
  constexpr int QV = D / 8;  // threads that stage q, and as many k
  static_assert(2 * QV <= NTH, "q and k in one go");
  const bool is_k = tid >= QV;
  const int qi = 8 * min(is_k ? tid - QV : tid, QV - 1);
  InVec<IDT, 8> qk;
  qk.load(is_k ? a.k : a.q, (is_k ? b * a.k_ts + (int64_t)(h / a.k_share) * D : b * a.q_ts + (int64_t)(h / a.q_share) * D) + qi);
  InVec<IDT, VEC> vv;
  vv.load(a.v, b * a.v_ts + (int64_t)(h / a.v_share) * D + c0);
  const float alpha = expf(a.log_decay[h]);
  ST* tile = static_cast<ST*>(a.pool) + ((int64_t)slot * a.H + h) * (int64_t)(D * D);
  typename IO::Raw raw[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) raw[p] = IO::load_raw(tile + (r0 + p * NW * RPW) * D + c0);
  if (tid < 2 * QV) {
    float f[8];
    qk.widen(f);
    float* o = (is_k ? s_k : s_q) + qi;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = f[e];
  }
  float v[VEC], acc[VEC];
  vv.widen(v);
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  __syncthreads();
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r = r0 + p * NW * RPW;
    const float k = s_k[r], q = s_q[r];
    float s[VEC];
    IO::widen(raw[p], s);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      s[e] = fmaf(alpha, s[e], k * v[e]);
      acc[e] = fmaf(q, s[e], acc[e]);
    }
    OUT::store(tile + r * D + c0, s);
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    if constexpr (LPR < 64) acc[e] = xor_sum_from<LPR>(acc[e]);
    if (lane < LPR) s_o[wave][lane * VEC + e] = acc[e];
  }
  __syncthreads();
  if (tid < CW) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += s_o[w][tid];
    store_elem(a.out, ob + tid, a.scale * sum, a.out_dt);
  }
}

template <int SDT, int D, int CW, int IDT>
hipError_t launch_part(const LinStepArgs& a, hipStream_t s) {
  using G = StepGeom<SDT, D, CW>;
  const long long bytes = (long long)a.B * a.H * D * D * StateElem<SDT>::BYTES;
  const unsigned grid = (unsigned)((int64_t)a.B * a.H * (D / CW));
  const bool ntl = SDT == GDN_F32 || stream_tile_reads(bytes), nts = SDT == GDN_F32 || stream_tile_writes(bytes);
  if (nts) gdn_linear_step_kernel<SDT, D, CW, IDT, true, true><<<grid, G::NW * 64, 0, s>>>(a);
  else if (ntl) gdn_linear_step_kernel<SDT, D, CW, IDT, true, SDT == GDN_F32><<<grid, G::NW * 64, 0, s>>>(a);
  else gdn_linear_step_kernel<SDT, D, CW, IDT, SDT == GDN_F32, SDT == GDN_F32><<<grid, G::NW * 64, 0, s>>>(a);
  return hipGetLastError();
}

template <int SDT, int D>
hipError_t launch_in(const LinStepArgs& a, hipStream_t s) {
  auto go = [&](auto type) -> hipError_t {
    constexpr int IDT = decltype(type)::value;
    // Up to a tile for every second compute unit, parts of rows that are still 128 bytes: 32 FP32 tiles in four parts 3.3 us
    // and whole 4.4, 128 tiles 4.5 and 5.2, 192 tiles 5.8 and 5.7; 32 BF16 tiles in two parts 3.5 and whole 3.8, 128 tiles 4.2
    // and 4.4, 192 tiles 5.1 both.  Shorter parts lose (64 x 64 tiles in four parts: 32 tiles 2.6 whole, 3.5).
    if constexpr (D == 128) {
      int cus = 0;
      const hipError_t e = device_cus(&cus);
      if (e != hipSuccess) return e;
      if (2 * (int64_t)a.B * a.H <= cus) return launch_part<SDT, D, SDT == GDN_F32 ? D / 4 : D / 2, IDT>(a, s);
    }
    return launch_part<SDT, D, D, IDT>(a, s);
  };
  if (a.in_dt == GDN_F32) return go(std::integral_constant<int, GDN_F32>{});
  if (a.in_dt == GDN_BF16) return go(std::integral_constant<int, GDN_BF16>{});
  return go(std::integral_constant<int, GDN_F16>{});
}

template <int SDT>
hipError_t launch_d(const LinStepArgs& a, int D, hipStream_t s) {
  if (D == 16) return launch_in<SDT, 16>(a, s);
  if (D == 32) return launch_in<SDT, 32>(a, s);
  if (D == 64) return launch_in<SDT, 64>(a, s);
  return launch_in<SDT, 128>(a, s);
}

}  // namespace

hipError_t launch_linear_step(const LinStepArgs& a, int state_dt, int D, hipStream_t s) {
  if (state_dt == GDN_F32) return launch_d<GDN_F32>(a, D, s);
  if (state_dt == GDN_BF16) return launch_d<GDN_BF16>(a, D, s);
  return launch_d<GDN_F16>(a, D, s);
}

}  // namespace gdn
