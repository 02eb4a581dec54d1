// Copies of whole state slots (fork, move, clear) and the compaction of a
// pool.  A slot is its bytes in every buffer of the state, so a call is one
// launch over (move, piece of a slot); bound by HBM: each byte is read once
// and written once.  64 slots of 540 KB moved by a compaction of 256: 14 us
// (4.9 TB/s, the listing of the moves included); 7 forks of 336 KB: 3.8 us.
#include <hip/hip_runtime.h>

#include "qstate_ops.hpp"

namespace qs {
namespace {

// Nontemporal: a slot is far larger than what the next launch would find in
// the L2, and the copy's destination is not read by this launch.
template <typename V>
__device__ __forceinline__ void copy_units(const uint8_t* src, uint8_t* dst, uint32_t bytes, bool zero) {
  const uint32_t units = bytes / (uint32_t)sizeof(V);
  for (uint32_t i = threadIdx.x; i < units; i += 256u * 4u) {
    V v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = V{};
      const uint32_t k = i + 256u * (uint32_t)j;
      if (!zero && k < units) v[j] = __builtin_nontemporal_load((const V*)src + k);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t k = i + 256u * (uint32_t)j;
      if (k < units) __builtin_nontemporal_store(v[j], (V*)dst + k);
    }
  }
}

using U4 = uint32_t __attribute__((ext_vector_type(4)));

// Piece `piece` of a slot: from slot `from` (or zeros when from < 0) to slot `to`.
__device__ __forceinline__ void copy_piece(const SlotArgs& a, uint32_t piece, int from, int to) {
  int b = 0;
  for (int i = 1; i < a.nbuf; ++i)
    if (piece >= a.buf[i].first) b = i;
  const SlotBuffer& f = a.buf[b];
  const uint64_t at = (uint64_t)(piece - f.first) * kSlotPiece;
  const uint32_t bytes = (uint32_t)min((uint64_t)kSlotPiece, f.bytes - at);
  const bool zero = from < 0;
  const uint8_t* src = zero ? nullptr : f.src + (uint64_t)from * f.bytes + at;
  uint8_t* dst = f.dst + (uint64_t)to * f.bytes + at;
  if (f.unit == 16) copy_units<U4>(src, dst, bytes, zero);
  else if (f.unit == 4) copy_units<uint32_t>(src, dst, bytes, zero);
  else if (f.unit == 2) copy_units<uint16_t>(src, dst, bytes, zero);
  else copy_units<uint8_t>(src, dst, bytes, zero);
}

__global__ __launch_bounds__(256) void k_copy_slots(const SlotArgs a) {
  const int i = (int)(blockIdx.x / a.pieces);
  const int from = a.src_slot[i], to = a.dst_slot[i];
  if (to < 0 || to >= a.dst_slots || from < -1 || from >= a.src_slots) return;
  if (from == to && a.buf[0].src == a.buf[0].dst) return;
  copy_piece(a, blockIdx.x % a.pieces, from, to);
}

// Compaction: with F live slots, the i-th live slot at or behind F moves to
// the i-th free slot before F, so sources and destinations never meet.  Every
// workgroup lists the moves itself (one pass over the B flags) and takes its
// share of (move, piece): one launch, nothing to wait for between workgroups.
__global__ __launch_bounds__(256) void k_compact_slots(const SlotArgs a) {
  extern __shared__ uint16_t move[];        // [B/2] sources, [B/2] destinations
  __shared__ int counts[4], base[2];
  const int B = a.dst_slots, half = (B + 1) / 2;
  const int tid = (int)threadIdx.x, wave = tid >> 6, lane = tid & 63;
  int n = 0;
  for (int i = tid; i < B; i += 256) n += a.live[i] != 0;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) n += __shfl_xor(n, m);
  if (lane == 0) counts[wave] = n;
  if (tid < 2) base[tid] = 0;
  __syncthreads();
  const int F = counts[0] + counts[1] + counts[2] + counts[3];
  for (int i0 = 0; i0 < B; i0 += 256) {
    const int i = i0 + tid;
    const bool live = i < B && a.live[i] != 0;
    const bool is_src = live && i >= F, is_dst = i < F && !live;
    const uint64_t ms = __ballot(is_src), md = __ballot(is_dst);
    __syncthreads();                        // counts and base of the round before are read
    if (lane == 0) counts[wave] = (int)__popcll(ms) | ((int)__popcll(md) << 16);
    __syncthreads();
    int s = base[0], d = base[1];
    for (int w = 0; w < 4; ++w)
      if (w < wave) {
        s += counts[w] & 0xFFFF;
        d += counts[w] >> 16;
      }
    const uint64_t below = (1ull << lane) - 1ull;
    if (is_src) move[s + (int)__popcll(ms & below)] = (uint16_t)i;
    if (is_dst) move[half + d + (int)__popcll(md & below)] = (uint16_t)i;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < 4; ++w) {
        base[0] += counts[w] & 0xFFFF;
        base[1] += counts[w] >> 16;
      }
    }
  }
  __syncthreads();
  const int moves = base[0];                // as many live slots behind F as free ones before it
  if (blockIdx.x == 0) {
    for (int i = tid; i < B; i += 256)
      if (a.live[i] == 0 || i < F) a.where[i] = a.live[i] ? i : -1;
    for (int i = tid; i < moves; i += 256) a.where[move[i]] = (int)move[half + i];
  }
  const uint32_t tasks = (uint32_t)moves * a.pieces;
  for (uint32_t t = blockIdx.x; t < tasks; t += gridDim.x) {
    const uint32_t m = t / a.pieces;
    copy_piece(a, t % a.pieces, (int)move[m], (int)move[half + m]);
  }
}

}  // namespace

hipError_t launch_copy_slots(const SlotArgs& a, hipStream_t s) {
  const int64_t most = max_blocks(256) / a.pieces;   // copies of a launch; the host refuses slots of more pieces
  for (int64_t i = 0; i < a.n; i += most) {
    SlotArgs part = a;
    part.n = (int32_t)(a.n - i < most ? a.n - i : most);
    part.src_slot = a.src_slot + i;
    part.dst_slot = a.dst_slot + i;
    k_copy_slots<<<dim3((uint32_t)part.n * a.pieces), 256, 0, s>>>(part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_compact_slots(const SlotArgs& a, hipStream_t s) {
  // at most half of the slots move; eight workgroups a compute unit are resident
  const uint64_t most = (uint64_t)(a.dst_slots / 2) * a.pieces;
  const uint32_t grid = (uint32_t)(most < 2048 ? (most ? most : 1) : 2048);
  const uint32_t lds = (uint32_t)((a.dst_slots + 1) / 2) * 2u * (uint32_t)sizeof(uint16_t);
  k_compact_slots<<<dim3(grid), 256, lds, s>>>(a);
  return hipGetLastError();
}

}  // namespace qs
