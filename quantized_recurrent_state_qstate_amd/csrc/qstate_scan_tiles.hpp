// Device helpers of the chunked scans: bf16 and fp32 matrix instructions,
// fp32 numbers as sums of bf16 ones, tiles of rows from global memory and in
// LDS, sums over a wave, segments of packed tokens.
#pragma once
#include <hip/hip_runtime.h>

#include "qstate_ops.hpp"

namespace qs {
namespace {

using BF8 = __bf16 __attribute__((ext_vector_type(8)));
using BF4 = __bf16 __attribute__((ext_vector_type(4)));
using F4 = float __attribute__((ext_vector_type(4)));
using S4 = short __attribute__((ext_vector_type(4)));
using U4 = uint32_t __attribute__((ext_vector_type(4)));

constexpr int kL = 64;   // tokens of a chunk

__device__ __forceinline__ F4 mfma(BF8 a, BF8 b, F4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ F4 mfma1(float a, float b, F4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// Four rows of one column for every lane: in each group of 16 lanes, lane l
// points at columns 4 (l & 3).. of row l >> 2 and gets column l of the rows.
__device__ __forceinline__ BF4 read_tr(const uint16_t* p) {
  typedef __attribute__((address_space(3))) S4* L;
  return __builtin_bit_cast(BF4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((L)p));
}

// Floats as a sum of bf16 numbers, each the rest rounded: three hold all 24 bits,
// the second is at most 2^-9 of the number, the third 2^-18.
__device__ __forceinline__ uint32_t round2(float a, float b) {
  using F2 = float __attribute__((ext_vector_type(2)));
  using B2 = __bf16 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(((F2){a, b}), B2));
}
// The next piece of two numbers, which are left with the rest.
__device__ __forceinline__ uint32_t take2(float& a, float& b) {
  const uint32_t d = round2(a, b);
  a -= __uint_as_float(d << 16);
  b -= __uint_as_float(d & 0xFFFF0000u);
  return d;
}
template <int N>
__device__ __forceinline__ void split(const float (&f)[8], BF8 (&out)[N]) {
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = f[j];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    uint32_t d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = n + 1 < N ? take2(r[2 * j], r[2 * j + 1]) : round2(r[2 * j], r[2 * j + 1]);
    out[n] = __builtin_bit_cast(BF8, (U4){d[0], d[1], d[2], d[3]});
  }
}

// Six products of three pieces by three; the other three are at most 2^-27 of
// the whole each.  Product p takes pieces first_of(p) and second_of(p).
__device__ constexpr int first_of(int p) { return p == 2 || p == 3 ? 1 : p == 5 ? 2 : 0; }
__device__ constexpr int second_of(int p) { return p == 1 || p == 3 ? 1 : p == 4 ? 2 : 0; }

__device__ __forceinline__ BF8 join(BF4 a, BF4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Inclusive sums over the wave's 64 lanes, by DPP moves of the two halves:
// shifts within rows of 16, then the last lane of a row, of a half, on.
template <int CTRL, int ROWS>
__device__ __forceinline__ double shifted(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
__device__ __forceinline__ double wave_sums(double x) {
  x += shifted<0x111, 0xF>(x);
  x += shifted<0x112, 0xF>(x);
  x += shifted<0x114, 0xF>(x);
  x += shifted<0x118, 0xF>(x);
  x += shifted<0x142, 0xA>(x);
  x += shifted<0x143, 0xC>(x);
  return x;
}

// Segment s of the packed tokens.  Segment s = (sequence i, cell c) with
// s = i + c: cells are seg tokens of the packed axis, and each sequence or
// cell boundary moves s on by one, so (i, c) follows from s and the offsets.
struct Segment {
  int seq, t0, t1;      // tokens
  bool first, last, none;
  int end;              // the sequence's
};
// The last sequence i > 0 with `le(i)`, which holds up to some i and not behind; else 0.
template <class F>
__device__ __forceinline__ int last_sequence(const ScanArgs& a, F le) {
  const int lane = (int)(threadIdx.x & 63u);
  int lo = 0, len = a.n - 1;
  while (len > 0) {
    const int step = (len + 63) >> 6;
    const int i = lo + (lane + 1) * step;
    const int c = (int)__popcll(__ballot(i <= lo + len && le(i)));
    lo += c * step;
    len = min(len - c * step, step - 1);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}
__device__ __forceinline__ Segment find_segment(const ScanArgs& a, int seg, int s) {
  Segment r{0, 0, 0, true, true, false, 0};
  int start = 0, end = a.T;
  if (a.offsets) {
    r.seq = last_sequence(a, [&](int i) { return min(max(a.offsets[i], 0), a.T) / seg + i <= s; });
    start = min(max(a.offsets[r.seq], 0), a.T);
    end = min(max(a.offsets[r.seq + 1], start), a.T);
  }
  const int c = s - r.seq, c0 = start / seg, c1 = end > start ? (end - 1) / seg : c0;
  r.none = c < c0 || c > c1 || end - start < a.least || end - start > a.most;
  r.first = c == c0;
  r.last = c == c1;
  r.t0 = r.first ? start : c * seg;
  r.t1 = r.last ? end : (c + 1) * seg;
  r.end = end;
  return r;
}

// Piece s of the delta rule's scans.  A sequence of more than two cells of `cut`
// tokens (of the packed axis) is cut where cells begin, any other is one piece:
// whether it is depends on the offsets, which the host does not know.  Piece
// s < n is the first of sequence s, piece n + c - 1 the one from cell c on, if
// cell c begins inside a sequence that is cut: what there may be none of comes
// last in a grid, or it leaves the rest badly dealt to the compute units (4
// sequences of 512 tokens of 16 heads token by token: 127 us, 179 with
// find_segment's order, 121 with no pieces).
struct Piece {
  int seq, t0, t1;
  bool first, last, none;
  int end;
};
__device__ __forceinline__ bool long_enough(int start, int end, int cut) { return cut > 0 && (end - start + 1) / 2 > cut; }
__device__ __forceinline__ Piece find_piece(const ScanArgs& a, int cut, int s) {
  const int x = s < a.n ? 0 : (s - a.n + 1) * cut;
  const int seq = s < a.n ? s : a.offsets ? last_sequence(a, [&](int i) { return a.offsets[i] <= x; }) : 0;
  const int start = a.offsets ? min(max(a.offsets[seq], 0), a.T) : 0;
  const int end = a.offsets ? min(max(a.offsets[seq + 1], start), a.T) : a.T;
  const bool many = long_enough(start, end, cut), none = end - start < a.least || end - start > a.most;
  if (s < a.n) return {seq, start, many ? (start / cut + 1) * cut : end, true, !many, none, end};
  return {seq, x, min(x + cut, end), false, x + cut >= end, none || !(many && start < x && x < end), end};
}

// A sequence that is cut needs its segments' whole decays (the delta rule's M) to
// be numbers: decays above one may leave fp32 where the state, zero or small, does
// not.  Where one is not, the join says so for that head, and the outputs are made
// in one piece: by the workgroups of the first one, which take the whole sequence.
template <class P>
__device__ __forceinline__ void outputs_of(P& p, const ScanArgs& a, const ScanSegs& g, int h) {
  if ((p.first && p.last) || !__builtin_amdgcn_readfirstlane(g.uncut[(int64_t)p.seq * a.H + h])) return;
  p.none |= !p.first;
  p.t1 = p.end;
  p.last = true;
}
__device__ __forceinline__ bool finite(F4 x) {
  return fabsf(x[0]) < INFINITY && fabsf(x[1]) < INFINITY && fabsf(x[2]) < INFINITY && fabsf(x[3]) < INFINITY;
}

// 16 bytes a lane from a buffer at `offset` to LDS, lane after lane from `to` on
// (the same in all lanes); beyond the buffer's bound they are zeros.
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t rsrc, uint16_t* to, int offset) {
  typedef __attribute__((address_space(3))) void* L;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (L)to, 16, offset, 0, 0, 0);
}

template <int N>
__device__ __forceinline__ int flip(int r);

// 64 rows of a bf16 tensor from row t0's element `p` on, `n` of them real: 16-byte
// pieces of `width` elements, zeros behind the last row and from column `width` on
// (what lies there is another head's, or not of the tensor).  VEC: buffer loads,
// whose bound is the last real row's end (rows are at most 2^24 elements
// apart, so offsets fit; a piece that begins in a row begins in front of the
// bound, and pieces are 16-byte aligned within it).
template <bool VEC>
struct Tile {
  const uint16_t* p;
  __amdgpu_buffer_rsrc_t rsrc;
  int32_t stride, n, width;
  Tile() = default;
  __device__ __forceinline__ Tile(const void* base, int64_t at, int64_t row, int n_, int width_)
      : p((const uint16_t*)base + at), stride((int32_t)row), n(n_), width(width_) {
    if constexpr (VEC)
      rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, n > 0 ? ((n - 1) * stride + width) * 2 : 0, 0x00027000);
  }
  // Byte offset of (r, c); beyond every bound, whatever rows are added, from column `width` on.
  __device__ __forceinline__ uint32_t offset(int r, int c) const {
    return c < width ? (uint32_t)((r * stride + c) * 2) : 0x80000000u;
  }
  __device__ __forceinline__ U4 load(int r, int c) const {
    if constexpr (VEC) {
      return __builtin_bit_cast(U4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, offset(r, c), 0, 0));
    } else {
      uint32_t d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t e = (int64_t)r * stride + c + 2 * j;
        const uint32_t lo = r < n && c + 2 * j < width ? p[e] : 0u, hi = r < n && c + 2 * j + 1 < width ? p[e + 1] : 0u;
        d[j] = lo | (hi << 16);
      }
      return (U4){d[0], d[1], d[2], d[3]};
    }
  }
  // Piece i of several that lie `step` rows apart from row r on: one product, then sums.
  __device__ __forceinline__ U4 load_step(int r, int c, int i, int step) const {
    if constexpr (VEC) {
      const uint32_t at = offset(r, c) + (uint32_t)(i * (step * stride * 2));
      return __builtin_bit_cast(U4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, 0, 0));
    } else {
      return load(r + i * step, c);
    }
  }
  // The same way back; nothing at or behind the bound, or from column `width` on.
  __device__ __forceinline__ void store_step(int r, int c, int i, int step, U4 y) const {
    if constexpr (VEC) {
      __builtin_amdgcn_raw_buffer_store_b128(y, rsrc, offset(r, c) + (uint32_t)(i * (step * stride * 2)), 0, 0);
    } else {
      uint16_t* o = (uint16_t*)p + (int64_t)(r + i * step) * stride + c;
      if (r + i * step < n)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < width) o[j] = (uint16_t)(y[j >> 1] >> (16 * (j & 1)));
    }
  }
  // Elements e .. e + 511 of an LDS tile with rows of N, as at<N>() lays them, by one wave.
  template <int N>
  __device__ __forceinline__ void bring(uint16_t* tile, int e, int lane) const {
    const int r = (e + lane * 8) / N, c = (((lane * 8) % N / 8) ^ flip<N>(r)) * 8;
    if constexpr (VEC) to_lds(rsrc, tile + e, (int)offset(r, c));
    else *(U4*)(tile + e + lane * 8) = load(r, c);
  }
};

// The largest exponents (as 15-bit patterns without sign) of 8 bf16 numbers, by halves.
using H2 = uint16_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ H2 largest(H2 x, U4 u) {
#pragma unroll
  for (int j = 0; j < 4; ++j) x = __builtin_elementwise_max(x, __builtin_bit_cast(H2, u[j] & 0x7FFF7FFFu));
  return x;
}
__device__ __forceinline__ bool odd(H2 x) { return x[0] >= 0x7F80 || x[1] >= 0x7F80; }   // infinity or NaN

// The largest magnitude of fp32 numbers, as bits; NaN is the largest.  From kHuge
// (2^120) on a chunk's numbers count as out of fp32's range.
constexpr uint32_t kHuge = (120u + 127u) << 23;
__device__ __forceinline__ uint32_t highest(uint32_t top, F4 x) {
#pragma unroll
  for (int r = 0; r < 4; ++r) top = max(top, __float_as_uint(x[r]) & 0x7FFFFFFFu);
  return top;
}

// Whether the lane's column of a state (in the scans' tiles, below) has a value that
// is not finite: then all its later outputs are not, in whichever way they are made.
template <int N>
__device__ __forceinline__ bool spoiled(const F4 (&S)[N]) {
  uint32_t top = 0;
#pragma unroll
  for (int y = 0; y < N; ++y) top = highest(top, S[y]);
  uint64_t b = __ballot(top >= 0x7F800000u);
  b |= b >> 32;
  b |= b >> 16;
  return (b >> (threadIdx.x & 15u) & 1u) != 0;
}

// Element (r, c) of an LDS tile with rows of N elements.  The 16-byte pieces of
// a row are exchanged by the row's low bits, so that both ways of reading, 8
// channels of 16 rows and (transposed) 4 rows of 4 x 4 channels, meet every
// bank once.  Rows of 32 elements need no exchange.
template <int N>
__device__ __forceinline__ int flip(int r) {
  return N >= 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : N == 64 ? ((r & 3) << 1) | ((r >> 2) & 1) : 0;
}
template <int N>
__device__ __forceinline__ int at(int r, int c) {
  return r * N + (((c >> 3) ^ flip<N>(r)) << 3) + (c & 7);
}

// A chunk token by token, for one with a value that is not finite, or that is
// not in the products of a whole chunk: there a zero times such a value would
// reach the tokens before it.  The state tiles are those of the scans (lane m, q4: column m,
// channels 32 i + 8 q4 .. + 7); K(i, c) and Q(i, c) give 8 channels from c on
// of token i, V(i) the lane's v, and O(i, o) takes the output.
template <int DK, bool DELTA, class FK, class FQ, class FV, class FO>
__device__ __forceinline__ void by_token(const ScanArgs& a, int t, int n, int h, FK K, FQ Q, FV V, FO O, F4 (&S)[DK / 16]) {
  const int lane = (int)threadIdx.x & 63, q4 = lane >> 4;
  const float skip = a.skip ? a.skip[h] : 0.0f;
  for (int i = 0; i < n; ++i) {
    const float d = a.decay[(int64_t)(t + i) * a.ds + h], beta = a.beta ? a.beta[(int64_t)(t + i) * a.bs + h] : 1.0f;
    const float v = V(i);
    float w = 0.0f, o = 0.0f;
#pragma unroll
    for (int c = 0; c < DK / 32; ++c) {
      const BF8 k = K(i, 32 * c + 8 * q4);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = S[2 * c + (j >> 2)][j & 3] * d;
        S[2 * c + (j >> 2)][j & 3] = x;
        if constexpr (DELTA) w = fmaf(x, (float)k[j], w);
      }
    }
    if constexpr (DELTA) {
      w += __shfl_xor(w, 16);
      w += __shfl_xor(w, 32);
    }
    const float u = beta * (v - w);
#pragma unroll
    for (int c = 0; c < DK / 32; ++c) {
      const BF8 k = K(i, 32 * c + 8 * q4), q = Q(i, 32 * c + 8 * q4);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = fmaf(u, (float)k[j], S[2 * c + (j >> 2)][j & 3]);
        S[2 * c + (j >> 2)][j & 3] = x;
        o = fmaf(x, (float)q[j], o);
      }
    }
    o += __shfl_xor(o, 16);
    o += __shfl_xor(o, 32);
    if (a.skip) o = fmaf(skip, v, o);
    if (q4 == 0) O(i, o);
  }
}

}  // namespace
}  // namespace qs
