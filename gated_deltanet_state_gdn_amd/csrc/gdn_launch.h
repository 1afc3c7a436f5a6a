// Internal launch interface between the C ABI (gdn_api.cpp) and the kernels.
// Arguments here are already validated by the ABI layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

struct DecodeArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* a;
  const void* b;
  const float* A_log;
  const float* dt_bias;
  void* pool;
  const int32_t* slot_map;
  void* out;
  int64_t num_slots;
  int32_t B, Hk, Hv;
  int32_t in_dt, out_dt;
  float scale;
};

struct RingArgs {
  void* k;
  void* v;
  float* g;
  float* beta;
  int32_t* start;
  int32_t* count;
  int32_t L;
};

struct ReplayArgs {
  DecodeArgs d;  // q, k, v, a, b laid out [B, T, H, d]; pool is the checkpoint pool
  RingArgs ring;
  int32_t T;     // 1..L; 0 selects the flush-only kernel
  const int32_t* num_rejected;
  void* read_pool;  // dual-precision mode: the 16-bit read copy of the fp32 checkpoint (else null)
  int32_t read_dt;
  int32_t* rec;     // [B * Hv][4] unit records (slot or -1, start and count after any fold), written by
                    // the fold's check for the one-wave prep; null when that prep is not used
};

struct SpecArgs {
  DecodeArgs d;  // q, k, v, a, b laid out [B, T, H, d]; slot_map holds the source slots
  const int32_t* dst_slots;  // [B, T]
  int32_t T;
};

struct CopyArgs {
  const gdn_state_ref* refs;  // [P], device
  const int32_t* src;         // [n], device
  const int32_t* dst;         // [n], device
  int32_t P, n;
};
constexpr int kCopyThreads = 256;
constexpr uint64_t kCopyChunk = 64 * 1024;  // bytes of a slot per workgroup

struct M2Args {
  const void* x;      // [B, T, H, P] (decode: T = 1)
  const void* Bm;     // [B, T, G, N]
  const void* Cm;     // [B, T, G, N]
  const void* dt;     // [B, T, H]
  const float* A_log;
  const float* dt_bias;
  const float* Dskip;
  void* pool;         // [num_slots, H, P, N]
  const int32_t* slot_map;
  void* y;            // [B, T, H, P]
  int64_t num_slots;
  int32_t B, H, G, in_dt, out_dt;
  int32_t T, L;       // replay window and ring length
  void* rx;           // ring x [num_slots, H, L, P]
  void* rB;           // ring B [num_slots, G, L, N]
  float* rg;          // ring g [num_slots, H, L]
  float* rdtp;        // ring dt' [num_slots, H, L]
  int32_t* start;     // [num_slots]
  int32_t* count;     // [num_slots]
  const int32_t* num_rejected;
};

struct PrefillArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* a;
  const void* b;
  const float* A_log;
  const float* dt_bias;
  void* pool;
  const int32_t* slot_map;
  const int32_t* cu_seqlens;
  void* out;
  int64_t num_slots;
  int64_t total_tokens;
  int32_t N, Hk, Hv;
  int32_t in_dt, out_dt;
  float scale;
};

// States that a scan starts from or ends in: a pool's slots, or (slots null)
// one state a sequence.
struct ScanStates {
  void* base;  // or null: zero states, or none written
  const int32_t* slots;
  int32_t dtype;
};

// The walk of the sequence scan, forward (read C, write B, in x) or in reverse
// (read B, write C, in dy).  Strides are in elements between tokens.
struct M2ScanArgs {
  const void* read;   // [T, G, n]
  const void* write;  // [T, G, n]
  const void* in;     // [T, H, d]
  const void* dt;     // [T, H]
  const float* A_log;
  const float* dt_bias;
  const float* Dskip;
  const int32_t* cu;    // [N + 1]
  const int32_t* live;  // slot of each sequence: outside [0, live_slots) marks a padded one; or null
  int64_t live_slots;
  int64_t read_ts, write_ts, in_ts, dt_ts;
  int64_t total;
  int32_t N, H, G, in_dt, out_dt;
  void* out;        // y, or dx
  ScanStates init, fin;
  float* gates;     // [chunk slots][H][3][64]: prefix sums of log-decays (two floats), dt'
  void* wt;         // [chunk slots][G][n][64] transposed write vectors
  void* rt;         // the same of the read vectors, or null
  float* gm;        // [chunk slots][G][64][64] read . write, or null
  float* seg;       // [segment slots][H][d][n] states at the segments' starts
  double* seg_g;    // [segment slots][H] the segments' summed log-decays
  float* blocks;    // states that meet each 128-token block, [block slots][H] of [n][d] (in reverse [d][n]), or null
  int32_t seg_chunks, whole, narrow;  // ScanPlan
  int32_t local;       // the segments' first walk
};

// The gradient kernel over blocks of 128 tokens.
struct M2GradArgs {
  const void* x;
  const void* Bm;
  const void* Cm;
  const void* dy;
  const float* A_log;
  const int32_t* cu;
  const int32_t* live;
  int64_t live_slots;
  int64_t x_ts, b_ts, c_ts;
  int64_t total;
  int32_t N, H, G, dt_in, splits;  // dt_in: dtype of the inputs and their gradients; splits: workgroups a group
  const float* gates;
  const void* bt;      // transposed B and C [chunk slots][G][n][64]
  const void* ct;
  const float* fwd;    // [block slots][H][n][d] states before each block
  const float* rev;    // [block slots][H][d][n] gradients of the states after it
  void* dB;            // [T, G, n]
  void* dC;
  void* ddt;           // [T, H]
  float* part_bc;      // [splits][2][T][G][n] where splits > 1
  float* part;         // [block slots][H][3] sums for dA_log, ddt_bias, dD
  float* dA_log;
  float* ddt_bias;
  float* dD;
};

struct NormArgs {
  const void* x;
  const void* z;       // the gate, or null
  const float* w;
  const float* b;      // or null
  void* y;
  float* mean;         // [rows, groups], or null
  float* rstd;
  const void* dy;
  void* dx;
  void* dz;
  float* part;         // [blocks][2][N] partial dw and db
  float* dw;
  float* db;           // or null
  int64_t rows, x_stride, z_stride, y_stride, dy_stride, dx_stride, dz_stride;
  int32_t N, groups, rms, gate_after, in_dt, out_dt;
  float eps;
};

// Each returns hipSuccess or the launch error.
hipError_t launch_decode(const DecodeArgs& a, int state_dt, int D, hipStream_t s);
// state_dt: dtype of the checkpoint pool a.d.pool; with a.read_pool set the
// checkpoint is the fp32 master and outputs read the read_dt copy.
hipError_t launch_replay(const ReplayArgs& a, int state_dt, int D, float* ws, hipStream_t s);
hipError_t launch_replay_flush(const ReplayArgs& a, int state_dt, int D, hipStream_t s);
hipError_t launch_replay_rollback(const ReplayArgs& a, hipStream_t s);
hipError_t launch_prefill(const PrefillArgs& a, int state_dt, int D, int chunk, float* ws, hipStream_t s);
hipError_t launch_spec(const SpecArgs& a, int state_dt, int D, hipStream_t s);
hipError_t launch_copy_blocks(const CopyArgs& a, uint64_t max_slot_bytes, hipStream_t s);
hipError_t launch_m2_decode(const M2Args& a, int state_dt, int P, int N, hipStream_t s);
// fold, step (T > 0) and pointer advance; T == 0 is the flush
hipError_t launch_m2_replay(const M2Args& a, int state_dt, int P, int N, hipStream_t s);
hipError_t launch_m2_rollback(const M2Args& a, hipStream_t s);
// Slots of a packed batch cut into pieces of P tokens.
int64_t scan_slots(int64_t N, int64_t total, int64_t P);
// How a walk is cut: chunks a segment (even, so that blocks of two chunks do not straddle; 0 for whole sequences), the
// most segments that a sequence may have and stay whole, and whether a wave has 16 state rows (narrow; d = 64 only) or 32.
struct ScanPlan {
  int seg_chunks, whole, narrow;
};
ScanPlan scan_plan(int64_t N, int64_t total, int H, int G, int d);
// Threads along x of the largest launch of a scan, and of the gradient kernel; a launch takes fewer than 2^32.
int64_t scan_work_items(int64_t N, int64_t total, int H, int G, int d);
int64_t grad_work_items(int64_t N, int64_t total, int H, int G);
hipError_t launch_scan_prep(const M2ScanArgs& a, bool bf, int n, hipStream_t s);
hipError_t launch_scan_walk(M2ScanArgs a, bool bf, int d, int n, bool rev, bool out, hipStream_t s);
int grad_splits(int64_t N, int64_t total, int H, int G);
hipError_t launch_scan_grad(const M2GradArgs& a, bool bf, int d, int n, hipStream_t s);
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s);
bool norm_slice_fits(int n);
int norm_bwd_blocks(int64_t rows, int N, int groups);
int64_t norm_sum_work_items(int N);  // threads of the kernel that adds dw and db: fewer than 2^32
size_t m2_lds_bytes(int P, int N, int L, int T, int heads_per_group);

// Dynamic LDS of the speculative-decode kernel; launches need <= kSpecMaxLds.
size_t spec_lds_bytes(int D, int T);
constexpr size_t kSpecMaxLds = 49152;

// Compute units of the current device (cached per device).
hipError_t device_cus(int* cus);
// Workgroups of `kernel` resident on one compute unit at this block size and
// dynamic LDS (cached per device, kernel, block and LDS size).
hipError_t resident_blocks(const void* kernel, int block, size_t lds, int* per_cu);

// Largest LDS footprint of the replay kernels for this shape; launches need <= 64 KiB.
size_t replay_lds_total(int D, int L, int T);
constexpr size_t kMaxLds = 65536;

// Workspace of gdn_replay_decode: w_t and acc_t (dv floats each) per
// (sequence, value head, window position).
size_t replay_workspace_bytes(int64_t B, int Hv, int T, int D);

// Fixed device scratch that gdn_replay_decode_noalloc uses in place of a caller
// workspace: one array per GPU the library runs on, kept until the process
// ends.  kReplayScratchBytes holds the workspace of 512 rows x 32 value heads
// x 5-token windows at head dim 128 (81.25 MiB).  replay_scratch() returns its
// device address on the current device, looked up once per device.
constexpr size_t kReplayScratchBytes = (size_t)96 << 20;
hipError_t replay_scratch(void** ptr);

// Workspace of the chunked prefill for chunks of C tokens: per (chunk slot,
// value head) the inverse T, the causal decay-weighted Q K^T, gamma and beta
// of one chunk.
size_t prefill_workspace_bytes(int N, int64_t total, int Hv, int C);
bool prefill_chunk_slots_fit(int N, int64_t total, int Hk, int Hv, int C);

}  // namespace gdn
