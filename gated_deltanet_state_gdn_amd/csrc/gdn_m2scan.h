// Device pieces shared by the Mamba2 sequence scan's kernels (gdn_m2scan.hip,
// gdn_m2grad.hip): where chunks lie, operand fragments, and the exact split of
// an FP32 operand into bf16 terms.
#pragma once

#include <atomic>

#include "gdn_device.h"
#include "gdn_launch.h"

namespace gdn {

constexpr int kScanChunk = 64;   // tokens of a chunk
constexpr int kGradBlock = 128;  // tokens of a block of the gradient kernel, two chunks

// Lets a kernel take more than 64 KiB of dynamic LDS, once a device (`done`: a
// bit a device; a device past 63 is asked every time).
inline hipError_t allow_lds(const void* kernel, size_t bytes, std::atomic<uint64_t>& done) {
  if (bytes <= 65536) return hipSuccess;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// ------------------------------------------------------------------ where chunks lie
// Sequence s of a packed batch, cut into pieces of P tokens, owns the slots
// s + floor(cu[s] / P) + c, c < max(1, ceil(len / P)): distinct for all
// sequences, and below sequences + ceil(total / P).  A workgroup of slot i finds its
// sequence as the last s with s + floor(cu[s] / P) <= i.
struct Piece {
  int seq;          // -1: the slot is not used
  int index, count; // this piece, and the pieces of its sequence
  int64_t begin;    // the sequence's first token
  int64_t len;      // and its tokens
};

// cu[i], inside the batch, in a scalar register (i is uniform).
__device__ __forceinline__ int64_t token_at(const int32_t* cu, int i, int64_t total) {
  return __builtin_amdgcn_readfirstlane((int)min((int64_t)cu[i], total));
}

// The lanes of a wave test 64 sequences at a time.
__device__ __forceinline__ Piece find_piece(const int32_t* cu, int N, int64_t total, int64_t slot, int P) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = N;  // the answer lies in [lo, hi): s = 0 always qualifies
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) >> 6;
    const int s = lo + lane * step;
    const bool in = s < hi && (int64_t)s + cu[s] / P <= slot;
    const int n = __popcll(__ballot(in));
    const int nlo = lo + (n - 1) * step;  // the condition holds on a prefix, and for lane 0
    hi = __builtin_amdgcn_readfirstlane(min(hi, nlo + step));
    lo = __builtin_amdgcn_readfirstlane(nlo);  // the same in every lane, and in scalar registers with all that follows from it
  }
  Piece p;
  const int64_t b = token_at(cu, lo, total), e = token_at(cu, lo + 1, total);
  p.begin = b;
  p.len = max(e - b, (int64_t)0);
  p.index = (int)(slot - lo - b / P);
  p.count = (int)max((p.len + P - 1) / P, (int64_t)1);
  p.seq = p.index < p.count ? lo : -1;
  return p;
}

__device__ __forceinline__ bool state_live(const int32_t* slots, int64_t num_slots, int seq) {
  if (slots == nullptr) return true;
  const int32_t s = slots[seq];
  return s >= 0 && (int64_t)s < num_slots;
}

// ------------------------------------------------------------------ addresses
// A uniform 64-bit base and a 32-bit lane offset, in elements of `EB` bytes: a
// load then takes its base from scalar registers, and a loop over many
// addresses keeps one vector register each instead of two.
__device__ __forceinline__ const char* at_bytes(const void* base, int64_t uniform, uint32_t lane, int eb) {
  return static_cast<const char*>(base) + uniform * eb + (uint32_t)(lane * (uint32_t)eb);
}

// A window of `bytes` from a uniform element: reads past its end give zero and
// writes past it are dropped, so a chunk's last tokens need no branches, and
// the number of memory operations in flight is known to the compiler.  All of
// an access's offset goes into its lane offset, which is what is compared with
// the window's size.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const void* base, int64_t elem, int eb, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(base)) + eb * elem, 0, (int)bytes, 0x00027000);
}

// A uniform read through the scalar cache, of what no kernel writes meanwhile.
__device__ __forceinline__ float scalar_read(const float* p) {
  return *reinterpret_cast<const float __attribute__((address_space(4)))*>(reinterpret_cast<uintptr_t>(p));
}

// ------------------------------------------------------------------ fragments
// A fragment is the 8 values that a lane gives a 16 x 16 product over 32 k's:
// lane l holds row (or column) l % 16 and the k's stored at 8 (l / 16) .. + 7.
// bf16: one 16x16x32 MFMA.  FP32: eight 16x16x4 ones, the e-th on every lane's
// e-th value; any order of the k's does, as both operands use the same.
template <bool BF>
struct Frag;
template <>
struct Frag<true> {
  typedef uint16_t E;
  u32x4 v;
  __device__ __forceinline__ static Frag load(const E* p) { return Frag{*reinterpret_cast<const u32x4*>(p)}; }
  __device__ __forceinline__ static Frag zero() { return Frag{u32x4{0u, 0u, 0u, 0u}}; }
  __device__ __forceinline__ void widen(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = unpack_lo<GDN_BF16>(v[j]);
      f[2 * j + 1] = unpack_hi<GDN_BF16>(v[j]);
    }
  }
  __device__ __forceinline__ static Frag round(const float (&f)[8]) {
    Frag r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = pack2<GDN_BF16>(f[2 * j], f[2 * j + 1]);
    return r;
  }
  // values 0..3 to p and 4..7 to p2
  __device__ __forceinline__ void store_halves(E* p, E* p2) const {
    *reinterpret_cast<u32x2*>(p) = u32x2{v[0], v[1]};
    *reinterpret_cast<u32x2*>(p2) = u32x2{v[2], v[3]};
  }
};
template <>
struct Frag<false> {
  typedef float E;
  f32x4 a, b;
  __device__ __forceinline__ static Frag load(const E* p) {
    return Frag{*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4)};
  }
  __device__ __forceinline__ static Frag zero() { return Frag{f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}}; }
  __device__ __forceinline__ void widen(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = a[j];
      f[4 + j] = b[j];
    }
  }
  __device__ __forceinline__ static Frag round(const float (&f)[8]) {
    return Frag{f32x4{f[0], f[1], f[2], f[3]}, f32x4{f[4], f[5], f[6], f[7]}};
  }
  __device__ __forceinline__ void store_halves(E* p, E* p2) const {
    *reinterpret_cast<f32x4*>(p) = a;
    *reinterpret_cast<f32x4*>(p2) = b;
  }
};

__device__ __forceinline__ f32x4 frag_mma(f32x4 acc, const Frag<true>& a, const Frag<true>& b) {
  typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), acc, 0, 0, 0);
}
__device__ __forceinline__ f32x4 frag_mma(f32x4 acc, const Frag<false>& a, const Frag<false>& b) {
#pragma unroll
  for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[j], b.a[j], acc, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b[j], b.b[j], acc, 0, 0, 0);
  return acc;
}

// What two bf16 roundings leave of a and b, exactly: a dot product with (-1, 0)
// and (0, -1), one instruction each in place of an unpacking and a subtraction
// (prefill of 20,408 tokens x 128 heads 663 us so, 678 with those; backward of
// 16,384 tokens 1404 and 1411).
// (The factors come from registers, since the immediate -1.0 would stand for
// the second one in both.  An infinity or NaN reaches its neighbour's rest too.)
__device__ __forceinline__ void bf16_rest(uint32_t pair, float& a, float& b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  uint32_t first = 0x0000bf80u, second = 0xbf800000u;
  asm("" : "+s"(first), "+s"(second));
  a = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, first), a, false);
  b = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, second), b, false);
}

// FP32 values as a sum of bf16 terms, each the rounding of what the ones
// before leave: three hold the 24 bits, so a product with exact bf16 values is
// that of the FP32 values; two are off by at most 2^-16 of it.  FP32 mode needs
// one.
template <bool BF, int TERMS = 3>
struct Split {
  static constexpr int K = BF ? TERMS : 1;
  Frag<BF> t[K];
  __device__ __forceinline__ static Split of(float (&f)[8]) {
    Split s;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      s.t[k] = Frag<BF>::round(f);
      if constexpr (BF)
        if (k + 1 < K)
#pragma unroll
          for (int j = 0; j < 4; ++j) bf16_rest(s.t[k].v[j], f[2 * j], f[2 * j + 1]);
    }
    return s;
  }
};

// 8 consecutive input elements from element (uniform + lane) as a fragment
// (16-byte aligned; BF: the input is bf16).
template <bool BF>
__device__ __forceinline__ Frag<BF> frag_from(const void* p, int64_t uniform, uint32_t lane, int dt) {
  if constexpr (BF) {
    return Frag<true>::load(reinterpret_cast<const uint16_t*>(at_bytes(p, uniform, lane, 2)));
  } else {
    float f[8];
    load_vec<8>(at_bytes(p, uniform, lane, dt == GDN_F32 ? 4 : 2), 0, dt, f);
    return Frag<false>::round(f);
  }
}

// ------------------------------------------------------------------ sums across lanes
// x from the lane that CTRL names, in a form that folds into the addition
// that uses it.
template <int CTRL>
__device__ __forceinline__ float dpp_zero(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row16_sum(float x) {
  x += dpp_zero<0xB1>(x);
  x += dpp_zero<0x4E>(x);
  x += dpp_zero<0x128>(x);
  x += dpp_zero<0x124>(x);
  return x;
}
// Sums of four values over each row of 16 lanes: lane l gets that of value l % 4.
__device__ __forceinline__ float row16_sum4(float a, float b, float c, float d) {
  const int l = threadIdx.x;
  const bool odd = l & 1, two = l & 2;
  const float p = (odd ? b : a) + dpp_zero<0xB1>(odd ? a : b);
  const float r = (odd ? d : c) + dpp_zero<0xB1>(odd ? c : d);
  float x = (two ? r : p) + dpp_zero<0x4E>(two ? p : r);
  x += dpp_zero<0x128>(x);
  x += dpp_zero<0x124>(x);
  return x;
}
// Sums of four values over the four rows of 16 lanes: lane l gets, for its
// place l % 16, that of value l / 16.
__device__ __forceinline__ float rows_sum4(float a, float b, float c, float d) {
  auto join = [](float x, float y, auto wide) {  // halves (pairs of rows) of x, then of y, added
    const unsigned p = __builtin_bit_cast(unsigned, x), r = __builtin_bit_cast(unsigned, y);
    unsigned u, v;
    if constexpr (decltype(wide)::value) {
      const auto t = __builtin_amdgcn_permlane32_swap(p, r, false, false);
      u = t[0];
      v = t[1];
    } else {
      const auto t = __builtin_amdgcn_permlane16_swap(p, r, false, false);
      u = t[0];
      v = t[1];
    }
    return __builtin_bit_cast(float, u) + __builtin_bit_cast(float, v);
  };
  // after the 32-lane swap the low half holds the first value's sum over halves, the high half the second's
  const float x = join(a, c, std::true_type{}), y = join(b, d, std::true_type{});
  return join(x, y, std::false_type{});
}

}  // namespace gdn
