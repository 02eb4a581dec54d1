// Short causal convolution over the tokens of each channel (the input path of
// the recurrence's q, k, v), for packed prompts and for single tokens.
//
//   y[t][c] = act(bias[c] + sum_{j<W} w[j][c] x[t - (W-1) + j][c]),
//   act(y) = y / (1 + e^-y) or y; rows before a sequence's first token are
//   its window (the last W-1 rows of what it has seen), which the call
//   replaces by the new last W-1 rows.
//
// Sums in fp32, one rounding to the output type.  Bound by HBM: every x row is
// read once (the W-1 rows that neighbouring runs share come from the cache),
// every y row written once.  A thread keeps 8 (fp32: 4) channels and their
// weights over a run of tokens, so a wave reads and writes 1 KB a row.  16384
// tokens of 12288 channels in bf16: 172 us, 4.7 TB/s where a copy of 1 GiB
// reaches 5.2; 4011 of 2304 in fp32: 15 us, 4.9 TB/s.  One token for 8 sequences
// of 2304 channels: 3.9 us, a launch and one trip to memory.
#include <hip/hip_runtime.h>

#include "qstate_ops.hpp"

namespace qs {
namespace {

template <int BF16>
struct Elem;
template <>
struct Elem<1> {
  using type = uint16_t;
  static __device__ __forceinline__ float get(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
  static __device__ __forceinline__ uint16_t put(float f) {
    const __bf16 b = (__bf16)f;
    return __builtin_bit_cast(uint16_t, b);
  }
};
template <>
struct Elem<0> {
  using type = float;
  static __device__ __forceinline__ float get(float f) { return f; }
  static __device__ __forceinline__ float put(float f) { return f; }
};

// V consecutive elements in one access.
template <int BF16, int V>
struct Vec {
  using E = typename Elem<BF16>::type;
  struct __attribute__((aligned(sizeof(E) * V))) type {
    E e[V];
  };
};

// The bare 2^x: a subnormal e^-y would vanish in the sum anyway.
__device__ __forceinline__ float silu(float y) {
  return y * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(y * -1.44269504088896341f));
}

// The sequence that token t belongs to: the number of offsets[1..n] <= t.
// The wave searches together, 64 probes a round.
__device__ __forceinline__ int find_seq(const int32_t* off, int n, int t) {
  const int lane = (int)(threadIdx.x & 63u);
  int lo = 0, len = n;                       // the answer lies in [lo, lo + len]
  while (len > 0) {
    const int step = (len + 63) >> 6;
    const int i = lo + (lane + 1) * step;    // offsets[i] is the end of sequence i-1
    const bool le = i <= lo + len && off[i] <= t;
    const int c = (int)__popcll(__ballot(le));
    lo += c * step;
    len = min(len - c * step, step - 1);
  }
  return lo;
}

constexpr int kRows = 4;   // tokens a thread has in registers at a time; the next ones are on their way

// Blocks [0, tiles): runs of kRows * steps tokens x 64*V channels a wave.  The
// other blocks: one sequence (from seq0 on) x 256*V channels: its first W-1
// outputs, which read the window, and the new window.  Only they touch the
// window, so no block waits for another.
template <int BF16, int V, int W>
__global__ __launch_bounds__(256) void k_conv(const ConvArgs a, int ctiles, int tiles, int sctiles, int steps, int seq0) {
  using E = typename Elem<BF16>::type;
  using VT = typename Vec<BF16, V>::type;
  const E* x = (const E*)a.x;
  E* out = (E*)a.out;
  const int b = (int)blockIdx.x;
  float w[W][V], bias[V];
  if (b < tiles) {
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int ct = b % ctiles;
    const int64_t run = (int64_t)(b / ctiles * 4 + wave) * kRows * steps;
    const int c = (ct * 64 + (int)(threadIdx.x & 63u)) * V;
    if (run >= a.T) return;
    const int t0 = (int)run, t1 = (int)min(run + kRows * steps, (int64_t)a.T);
    int seq = __builtin_amdgcn_readfirstlane(find_seq(a.offsets, a.n, t0));
    if (c >= a.C) return;
    VT r[W - 1 + kRows], next[kRows];
    auto row = [&](int t) {
      VT y;
      if (t >= 0 && t < t1) {
        y = *(const VT*)(x + (int64_t)t * a.x_stride + c);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) y.e[e] = 0;
      }
      return y;
    };
#pragma unroll
    for (int i = 0; i < W - 1; ++i) r[i] = row(t0 - (W - 1) + i);
#pragma unroll
    for (int i = 0; i < kRows; ++i) next[i] = row(t0 + i);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) w[j][i] = a.weight[(int64_t)j * a.C + c + i];
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = a.bias ? a.bias[c + i] : 0.0f;
    int start = seq < a.n ? a.offsets[seq] : 0x7FFFFFFF;
    int end = seq < a.n ? a.offsets[seq + 1] : 0x7FFFFFFF;
    auto skipped = [&](int s) {
      if (!a.window) return false;
      const int sl = a.slot ? a.slot[s] : s;
      return sl < 0 || sl >= a.slots;
    };
    bool skip = seq < a.n && skipped(seq);
    for (int tb = t0; tb < t1; tb += kRows) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) r[W - 1 + i] = next[i];
#pragma unroll
      for (int i = 0; i < kRows; ++i) next[i] = row(tb + kRows + i);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int t = tb + i;
        if (t < t1) {
          while (seq < a.n && t >= end) {     // the next sequence that is not empty
            ++seq;
            start = end;
            end = seq < a.n ? a.offsets[seq + 1] : 0x7FFFFFFF;
            if (seq < a.n) skip = skipped(seq);
          }
          const int seen = t - start;         // tokens of the sequence before this one
          if (seq < a.n && seen >= (a.window ? W - 1 : 0) && !skip) {
            VT y;
            float s[V];
#pragma unroll
            for (int e = 0; e < V; ++e) s[e] = bias[e];
            if (seen >= W - 1) {
#pragma unroll
              for (int j = 0; j < W; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) s[e] = fmaf(w[j][e], Elem<BF16>::get(r[i + j].e[e]), s[e]);
            } else {
#pragma unroll
              for (int j = 0; j < W; ++j)
                if (seen >= W - 1 - j)
#pragma unroll
                  for (int e = 0; e < V; ++e) s[e] = fmaf(w[j][e], Elem<BF16>::get(r[i + j].e[e]), s[e]);
            }
            if (a.silu) {
#pragma unroll
              for (int e = 0; e < V; ++e) s[e] = silu(s[e]);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) y.e[e] = Elem<BF16>::put(s[e]);
            VT* to = (VT*)(out + (int64_t)t * a.out_stride + c);
            // nontemporal: a long prompt's outputs are more than the caches hold
            // (16384 x 12288 bf16: 3% faster; 4011 x 2304 fp32: 6%)
            if constexpr (sizeof(VT) == 16) {
              using N4 = uint32_t __attribute__((ext_vector_type(4)));
              __builtin_nontemporal_store(__builtin_bit_cast(N4, y), (N4*)to);
            } else {
              *to = y;
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < W - 1; ++i) r[i] = r[i + kRows];
    }
    return;
  }
  // one sequence's beginning and its window
  const int sb = b - tiles;
  const int seq = seq0 + sb / sctiles;
  const int c = ((sb % sctiles) * 256 + (int)threadIdx.x) * V;
  if (c >= a.C) return;
  const int sl = a.slot ? a.slot[seq] : seq;
  if (sl < 0 || sl >= a.slots) return;
  const int start = min(max(a.offsets[seq], 0), a.T), end = min(max(a.offsets[seq + 1], start), a.T);
  const int len = end - start;
  if (len == 0) return;
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) w[j][i] = a.weight[(int64_t)j * a.C + c + i];
#pragma unroll
  for (int i = 0; i < V; ++i) bias[i] = a.bias ? a.bias[c + i] : 0.0f;
  E* win = (E*)a.window + (int64_t)sl * (W - 1) * a.C + c;
  VT r[2 * (W - 1)], last[W - 1];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) r[i] = *(const VT*)(win + (int64_t)i * a.C);
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    r[W - 1 + i] = r[0];
    if (i < len) r[W - 1 + i] = *(const VT*)(x + (int64_t)(start + i) * a.x_stride + c);
  }
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {         // row i of the new window: token len - (W-1) + i
    const int t = len - (W - 1) + i;
    last[i] = r[0];
    if (t >= 0) last[i] = *(const VT*)(x + (int64_t)(start + t) * a.x_stride + c);
    else
#pragma unroll
      for (int m = 0; m < W - 1; ++m)
        if (W - 1 + t == m) last[i] = r[m];
  }
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    if (i < len) {
      VT y;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float s = bias[e];
#pragma unroll
        for (int j = 0; j < W; ++j) s = fmaf(w[j][e], Elem<BF16>::get(r[i + j].e[e]), s);
        y.e[e] = Elem<BF16>::put(a.silu ? silu(s) : s);
      }
      *(VT*)(out + (int64_t)(start + i) * a.out_stride + c) = y;
    }
  }
#pragma unroll
  for (int i = 0; i < W - 1; ++i) *(VT*)(win + (int64_t)i * a.C) = last[i];
}

// One token of each of n sequences: a thread holds V channels of one sequence,
// reads the window and the token, writes the output and the shifted window.
template <int BF16, int V, int W>
__global__ __launch_bounds__(64) void k_conv_step(const ConvArgs a, int ctiles, int seq0) {
  using E = typename Elem<BF16>::type;
  using VT = typename Vec<BF16, V>::type;
  const int seq = seq0 + (int)blockIdx.x / ctiles;
  const int c = (((int)blockIdx.x % ctiles) * 64 + (int)threadIdx.x) * V;
  if (c >= a.C) return;
  const int sl = a.slot ? a.slot[seq] : seq;
  if (sl < 0 || sl >= a.slots) return;
  E* win = (E*)a.window + (int64_t)sl * (W - 1) * a.C + c;
  VT r[W];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) r[i] = *(const VT*)(win + (int64_t)i * a.C);
  r[W - 1] = *(const VT*)((const E*)a.x + (int64_t)seq * a.x_stride + c);
  VT y;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float s = a.bias ? a.bias[c + e] : 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) s = fmaf(a.weight[(int64_t)j * a.C + c + e], Elem<BF16>::get(r[j].e[e]), s);
    y.e[e] = Elem<BF16>::put(a.silu ? silu(s) : s);
  }
  *(VT*)((E*)a.out + (int64_t)seq * a.out_stride + c) = y;
#pragma unroll
  for (int i = 0; i < W - 1; ++i) *(VT*)(win + (int64_t)i * a.C) = r[i + 1];
}

template <int BF16, int V, int W>
hipError_t conv(const ConvArgs& a, hipStream_t s) {
  const int ctiles = (a.C + 64 * V - 1) / (64 * V);
  // Long runs read fewer rows twice and load the weights less often; short
  // ones keep the device full: at least about 8192 waves (16384 x 12288 bf16: 224 us with one
  // step, 182 with four, 178 with eight, 198 with sixteen and a quarter of the waves).
  int steps = 1;
  while (steps < 8 && (int64_t)ctiles * (a.T / (kRows * 2 * steps)) >= 8192) steps *= 2;
  auto runs = [&] { return ctiles * (((int64_t)a.T + 4 * kRows * steps - 1) / (4 * kRows * steps)); };
  while (runs() > max_blocks(256) / 2) steps *= 2;
  const int sctiles = (a.C + 256 * V - 1) / (256 * V);
  const int64_t most = max_blocks(256) / 2 / sctiles;   // sequences of a launch
  int64_t tiles = runs(), seq = 0;
  do {
    const int64_t n = !a.window ? 0 : a.n - seq < most ? a.n - seq : most;
    if (tiles + n == 0) break;
    k_conv<BF16, V, W><<<dim3((uint32_t)(tiles + n * sctiles)), 256, 0, s>>>(a, ctiles, (int)tiles, sctiles, steps, (int)seq);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    tiles = 0;
    seq += n;
  } while (a.window && seq < a.n);
  return hipSuccess;
}

template <int BF16, int V, int W>
hipError_t conv_step(const ConvArgs& a, hipStream_t s) {
  const int ctiles = (a.C + 64 * V - 1) / (64 * V);
  const int64_t most = max_blocks(64) / ctiles;         // sequences of a launch
  for (int64_t seq = 0; seq < a.n; seq += most) {
    const int64_t n = a.n - seq < most ? a.n - seq : most;
    k_conv_step<BF16, V, W><<<dim3((uint32_t)(n * ctiles)), 64, 0, s>>>(a, ctiles, (int)seq);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

#define QS_CONV_PICK(fn)                                                        \
  if (a.bf16) {                                                                 \
    if (a.vec) return a.W == 4 ? fn<1, 8, 4>(a, s) : a.W == 3 ? fn<1, 8, 3>(a, s) : fn<1, 8, 2>(a, s); \
    return a.W == 4 ? fn<1, 1, 4>(a, s) : a.W == 3 ? fn<1, 1, 3>(a, s) : fn<1, 1, 2>(a, s);            \
  }                                                                             \
  if (a.vec) return a.W == 4 ? fn<0, 4, 4>(a, s) : a.W == 3 ? fn<0, 4, 3>(a, s) : fn<0, 4, 2>(a, s);   \
  return a.W == 4 ? fn<0, 1, 4>(a, s) : a.W == 3 ? fn<0, 1, 3>(a, s) : fn<0, 1, 2>(a, s);

}  // namespace

hipError_t launch_conv(const ConvArgs& a, hipStream_t s) { QS_CONV_PICK(conv) }
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t s) { QS_CONV_PICK(conv_step) }

}  // namespace qs
