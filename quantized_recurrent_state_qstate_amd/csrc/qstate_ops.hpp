// Internal interface of the operators around the decode step (convolution,
// query/key norm and rotation, slot copies, prompt scan): kernel arguments
// and launchers, and what their host code needs of a handle.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qstate.h"

namespace qs {

// Error reporting of the C ABI (the thread's last error text).
qs_status op_fail(qs_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
qs_status op_ok();

// What a handle holds, for host code outside qstate_host.cpp.
struct HandleView {
  const qstate_config* cfg;
  const qstate_sizes* sizes;
};
HandleView op_view(const qstate_handle* h);
qs_status op_check_tensors(const qstate_handle* h, const qstate_tensors* st);
qs_status op_check_device(const qstate_handle* h);

// A launch has fewer than 2^32 threads: the runtime takes the number modulo
// 2^32, silently unless it is 0.  Launchers split what needs more, or their host
// code refuses it.
constexpr int64_t max_blocks(int threads) { return 0xFFFFFFFFll / threads; }

// ---- short causal convolution ---------------------------------------------
struct ConvArgs {
  const void* x;
  void* out;
  const float* weight;     // [W][C]
  const float* bias;       // [C] or null
  void* window;            // [slots][W-1][C] or null
  const int32_t* slot;     // [n] or null (sequence i uses slot i)
  const int32_t* offsets;  // [n+1] (prompt form)
  int64_t x_stride, out_stride;   // elements between tokens
  int32_t bf16, T, C, W, n, slots, silu;
  int32_t vec;             // 16-byte accesses possible
};
hipError_t launch_conv(const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t s);

// ---- norm and rotation of queries and keys ---------------------------------
struct QkArgs {
  const void* x[2];        // q, k
  void* y[2];
  const float* w[2];       // [dim] or null
  const int32_t* position; // [T] (rot > 0)
  const double* frequency; // [rot/2] (rot > 0)
  int64_t xs[2], ys[2];    // elements between tokens
  int32_t bf16, T, heads[2], dim, rot, norm, interleaved;
  float eps, scale[2];
};
hipError_t launch_qk(const QkArgs& a, hipStream_t s);

// ---- slot copies -------------------------------------------------------------
constexpr int kMaxSlotBuffers = 12;
struct SlotBuffer {
  const uint8_t* src;
  uint8_t* dst;
  uint64_t bytes;          // per slot
  uint32_t unit;           // 16, 4, 2 or 1: the widest access its size and bases allow
  uint32_t first;          // index of its first piece within a slot
};
struct SlotArgs {
  SlotBuffer buf[kMaxSlotBuffers];
  int32_t nbuf;
  uint32_t pieces;         // pieces of one slot over all buffers
  int32_t src_slots, dst_slots, n;
  const int32_t* src_slot; // copy: [n]
  const int32_t* dst_slot;
  const uint8_t* live;     // compact: [dst_slots]
  int32_t* where;
};
hipError_t launch_copy_slots(const SlotArgs& a, hipStream_t s);
hipError_t launch_compact_slots(const SlotArgs& a, hipStream_t s);
constexpr int kSlotPiece = 16384;        // bytes of a piece
constexpr int kMaxCompactSlots = 16384;  // the moves of one call fit LDS

// ---- prompt scan ---------------------------------------------------------------
struct ScanArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* decay;
  const float* beta;       // or null
  const float* skip;       // [H] or null
  const float* initial;    // [n][H][dv][dk] or null
  float* final;
  void* out;
  const int32_t* offsets;  // [n+1] or null (one sequence of T tokens)
  int64_t qs, ks, vs, ds, bs, os;   // elements between tokens
  int32_t T, n, H, G, dk, dv;
  int32_t least, most;     // a launch takes the sequences of least .. most tokens, and leaves the others alone
  int32_t bf16, delta, key;
  int32_t vec;             // 16-byte accesses: 2 to q, k, v and out rows, 1 to q and k, 0 to none
};

// Segments of the scans: cells of `seg` tokens of the packed axis,
// cut again where sequences begin; `count` bounds their number.  Delta rule:
// sequences of more than two cells of `cut` tokens (0: none) are cut, total has
// for each piece L and M, [dv + dk][dk] a head; in chunks, seg is a chunk's 64
// tokens and states its prepared matrices.
struct ScanSegs {
  int32_t seg, count, cut;
  float* states;           // [count][H][dv][dk], null: no sequence is cut; delta rule: [count][H] kScanPrepBytes
  float* total;            // [count][H] or [count][H][dk]: a segment's whole decay; delta rule: L and M
  int32_t* uncut;          // [n][H] where sequences are cut: not 0 if this one's outputs are made in one piece
};
constexpr int kScanPrepBytes = 1024 + 18 * 1024 + 12 * 1024;
hipError_t launch_scan_key(const ScanArgs& a, const ScanSegs& g, hipStream_t s);
hipError_t launch_scan_join(const ScanArgs& a, const ScanSegs& g, hipStream_t s);
hipError_t launch_delta_join(const ScanArgs& a, const ScanSegs& g, hipStream_t s);
hipError_t launch_scan_delta(const ScanArgs& a, const ScanSegs& g, hipStream_t s);
hipError_t launch_scan(const ScanArgs& a, const ScanSegs& g, hipStream_t s);
hipError_t launch_scan_chunk(const ScanArgs& a, const ScanSegs& g, hipStream_t s);

}  // namespace qs
