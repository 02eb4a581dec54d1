// Scan of packed bf16 prompts, additive with a decay for every key channel, 16
// tokens at a time on the matrix cores.
//
// With D_i the product of a channel's decays from the block's first token to
// token i (a vector over channels), S the state before the block, u = beta v,
//   S_i = S diag(D_i) + sum_{j<=i} v_j (beta_j k_j D_i / D_j)^T,
//   o_i = S (q_i D_i) + sum_{j<=i} P_ij v_j,  P_ij = (q_i D_i).(beta_j k_j / D_j),
// and the state after the block is the last S_i, whose keys beta_j k_j D_last / D_j
// are formed with the products of the decays behind j, not by division.
//
// A block is 16 tokens because 1 / D_j has to stay in range: blocks in which D
// leaves [2^-100, 2^20] (decays below 1/64 all along), beta k / D or q D leaves what
// three bf16 pieces hold, or a value is not finite go token by token.  No
// logarithms: they would cost a rounding a token that adds up over the state's memory.
//
// Precision: v is bf16; the other operands (the state's keys, q D, k / D, S and
// P) are cut into three bf16 pieces, which hold their 24 bits; products of three
// by three leave out the last three, at most 2^-27 of the whole each.  All sums
// are fp32; an output is rounded to bf16 once.
//
// A workgroup holds 64 NV value columns of one (segment, head), each wave 16 NV
// in accumulators [dk][v].  Each wave prepares 4 of the block's 16 tokens.
//
// 2048 tokens of 32 heads of 128 x 128: 126 us with operands from HBM, 109 from the
// Infinity Cache, of which (then, under a trace) the local states 34, the states
// between segments 12, the outputs 73.  Vector instructions fill 32% of the
// outputs' time (splitting S into pieces every 16 tokens, and the block's
// operands), matrix instructions 19%; the rest is waiting, with two waves a SIMD.
#include <hip/hip_runtime.h>

#include "qstate_scan_tiles.hpp"

namespace qs {
namespace {

constexpr int kB = 16;   // tokens of a block

__device__ __forceinline__ F4 mfma16(BF4 a, BF4 b, F4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(S4, a), __builtin_bit_cast(S4, b), c, 0, 0, 0);
}

// N consecutive bf16 or fp32 numbers as fp32.
template <int N, bool VEC>
__device__ __forceinline__ void get_bf16(const void* p, int64_t i, float (&f)[N]) {
  const uint16_t* x = (const uint16_t*)p + i;
  if constexpr (VEC && N == 4) {
    const uint2 u = *(const uint2*)x;
    f[0] = __uint_as_float(u.x << 16);
    f[1] = __uint_as_float(u.x & 0xFFFF0000u);
    f[2] = __uint_as_float(u.y << 16);
    f[3] = __uint_as_float(u.y & 0xFFFF0000u);
  } else if constexpr (VEC && N == 2) {
    const uint32_t u = *(const uint32_t*)x;
    f[0] = __uint_as_float(u << 16);
    f[1] = __uint_as_float(u & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = __uint_as_float((uint32_t)x[j] << 16);
  }
}

// N numbers as three bf16 pieces, `next` elements apart.
template <int N>
__device__ __forceinline__ void put_pieces(uint16_t* to, int next, float (&f)[N]) {
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    if constexpr (N == 1) {
      const __bf16 b = (__bf16)f[0];
      to[p * next] = __builtin_bit_cast(uint16_t, b);
      f[0] -= (float)b;
    } else {
#pragma unroll
      for (int j = 0; j < N; j += 2) *(uint32_t*)(to + p * next + j) = take2(f[j], f[j + 1]);
    }
  }
}

template <int DK, int NV, bool OUT, int VEC>
__global__ __launch_bounds__(256, DK <= 128 && VEC > 0 ? 2 : 1) void k_scan_key(const ScanArgs a, const ScanSegs g, int vchunks) {
  constexpr int kDV = 64 * NV, kKS = DK / 32, kC = DK / 64, kR = DK + 8, kVR = kDV + 8;
  constexpr int kVP = kB * kDV / 8;                                    // 16-byte pieces of v
  __shared__ __attribute__((aligned(16))) uint16_t sq[OUT ? 3 : 1][OUT ? kB * kR : 8];   // q D
  __shared__ __attribute__((aligned(16))) uint16_t sk[OUT ? 3 : 1][OUT ? kB * kR : 8];   // beta k / D
  __shared__ __attribute__((aligned(16))) uint16_t su[3][kB * kR];                       // the state's keys
  __shared__ __attribute__((aligned(16))) uint16_t sv[kB * kVR];
  __shared__ __attribute__((aligned(16))) uint16_t so[OUT ? kB * kVR : 8];
  __shared__ __attribute__((aligned(16))) float part[4][DK], all[DK];  // products over 4 tokens, over the block
  __shared__ int sodd[2];
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, q4 = lane >> 4;
  const int per = a.H * vchunks;
  const int s = (int)(blockIdx.x / (uint32_t)per), hv = (int)(blockIdx.x % (uint32_t)per);
  const int h = hv % a.H, v0 = hv / a.H * kDV, kh = h / (a.H / a.G);
  Segment sg = find_segment(a, g.seg, s);
  if (OUT && !sg.none) outputs_of(sg, a, g, h);
  if (sg.none || (!OUT && sg.last)) return;
  const int64_t head = (int64_t)h * a.dv;
  const float skip = a.skip ? a.skip[h] : 0.0f;

  F4 S[NV][2 * kKS];
  const int col = (wave * NV) * 16 + m;
  const float* from = !OUT ? nullptr
                      // a sequence in one piece; of several, the first one's state is kept with the
                      // others, since the last one may write it over (final may be initial)
                      : sg.first && sg.last ? (a.initial ? a.initial + (int64_t)sg.seq * a.H * a.dv * DK : nullptr)
                                            : g.states + (int64_t)s * a.H * a.dv * DK;
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int t = 0; t < 2 * kKS; ++t) {
      S[n][t] = (F4){0, 0, 0, 0};
      if (from && v0 + col + 16 * n < a.dv)
        S[n][t] = *(const F4*)(from + (head + v0 + col + 16 * n) * DK + 32 * (t >> 1) + 8 * q4 + 4 * (t & 1));
    }

  // what this thread brings: channels kC lane .. of tokens 4 wave .. + 3; a piece of v
  const int ch = kC * lane;
  float nd[4][kC], nq[OUT ? 4 : 1][kC], nk[4][kC], nb[4];
  U4 nv = (U4){0, 0, 0, 0};
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t tt = t + 4 * wave + i;
      nb[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        nd[i][j] = 1.0f;
        nk[i][j] = 0.0f;
        if constexpr (OUT) nq[i][j] = 0.0f;
      }
      if (tt < sg.t1) {
#pragma unroll
        for (int j = 0; j < kC; ++j) nd[i][j] = a.decay[tt * a.ds + (int64_t)h * DK + ch + j];
        get_bf16<kC, (VEC > 0)>(a.k, tt * a.ks + (int64_t)kh * DK + ch, nk[i]);
        if constexpr (OUT) get_bf16<kC, (VEC > 0)>(a.q, tt * a.qs + (int64_t)kh * DK + ch, nq[i]);
        nb[i] = a.beta ? a.beta[tt * a.bs + h] : 1.0f;
      }
    }
    if (tid < kVP) {
      const Tile<VEC == 2> tv(a.v, (int64_t)t * a.vs + head + v0, a.vs, min(kB, sg.t1 - t), min(kDV, a.dv - v0));
      nv = tv.load(tid / (kDV / 8), tid % (kDV / 8) * 8);
    }
  };

  float whole[kC];                           // the segment's decay of channels ch ..
#pragma unroll
  for (int j = 0; j < kC; ++j) whole[j] = 1.0f;
  if (tid < 2) sodd[tid] = 0;
  if (sg.t0 < sg.t1) fetch(sg.t0);
  __syncthreads();
  int turn = 0;
  for (int t = sg.t0; t < sg.t1; t += kB, turn ^= 1) {
    const int n = min(kB, sg.t1 - t);
    // ---- products of the decays within 4 tokens
    float pre[4][kC], suf[4][kC];
    bool bad = OUT && odd(largest((H2){0, 0}, nv));
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      pre[0][j] = nd[0][j];
      suf[3][j] = 1.0f;
#pragma unroll
      for (int i = 1; i < 4; ++i) pre[i][j] = pre[i - 1][j] * nd[i][j];
#pragma unroll
      for (int i = 2; i >= 0; --i) suf[i][j] = suf[i + 1][j] * nd[i + 1][j];
      part[wave][ch + j] = pre[3][j];
    }
    if (tid < kVP) *(U4*)&sv[tid / (kDV / 8) * kVR + tid % (kDV / 8) * 8] = nv;
    __syncthreads();                         // products are there; the block before has been read
    // ---- the operands
    uint32_t far = 0, low = 0xFFFFFFFFu;
    int32_t high = 0;
    float before[kC], behind[kC];
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      before[j] = behind[j] = 1.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float x = part[w][ch + j];
        if (w < wave) before[j] *= x;
        if (w > wave) behind[j] *= x;
      }
      const float x = before[j] * pre[3][j] * behind[j];
      if (wave == 0) all[ch + j] = x;
      whole[j] *= x;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * wave + i;
      float x[kC], y[kC], z[kC];
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        const float D = before[j] * pre[i][j], kb = nk[i][j] * nb[i];
        if constexpr (OUT) {
          // On the bits, whose sums and differences are products and quotients to a factor
          // of 2: D in [2^-100, 2^20]; |kb| / D up to 2^100, which a kb that is not finite exceeds;
          // |q| D from 2^-100 on where q is not zero, so that its third piece is a normal number.
          const uint32_t bits = __float_as_uint(D);
          far = max(far, bits - (27u << 23));
          high = max(high, (int32_t)((__float_as_uint(kb) & 0x7FFFFFFFu) - bits));
          low = min(low, __builtin_elementwise_add_sat((__float_as_uint(nq[i][j]) & 0x7FFFFFFFu) - 1u, bits));
          x[j] = nq[i][j] * D;
          const float inv = __builtin_amdgcn_rcpf(D);     // within 1 ulp; one Newton step
          y[j] = kb * fmaf(fmaf(-D, inv, 1.0f), inv, inv);
        }
        const float rest = suf[i][j] * behind[j];
        if constexpr (!OUT) bad |= !(D <= 0x1p100f && rest <= 0x1p100f);
        z[j] = kb * rest;
      }
      if constexpr (OUT) {
        put_pieces<kC>(&sq[0][r * kR + ch], kB * kR, x);
        put_pieces<kC>(&sk[0][r * kR + ch], kB * kR, y);
      }
      put_pieces<kC>(&su[0][r * kR + ch], kB * kR, z);
    }
    if (bad || (OUT && (far > 120u << 23 || high > 100 << 23 || low < 154u << 23))) sodd[turn] = 1;
    if (tid == 0) sodd[turn ^ 1] = 0;        // read in the block before, next written in the next
    __syncthreads();
    if (t + kB < sg.t1) fetch(t + kB);
    if (!OUT && sodd[turn])                  // decays that grow out of fp32: the sequence is not cut
#pragma unroll
      for (int j = 0; j < kC; ++j) whole[j] = NAN;
    if (OUT && sodd[turn]) {
      // ---- token by token, q, k and the decays from memory
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        auto rows = [&](const void* p, int64_t stride, int i, int c) {
          BF8 f;
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = ((const __bf16*)p)[(int64_t)(t + i) * stride + (int64_t)kh * DK + c + j];
          return f;
        };
        for (int i = 0; i < n; ++i) {
          const float beta = a.beta ? a.beta[(int64_t)(t + i) * a.bs + h] : 1.0f;
          const float vv = __uint_as_float((uint32_t)sv[i * kVR + col + 16 * v] << 16), u = beta * vv;
          float o = 0.0f;
#pragma unroll
          for (int c = 0; c < kKS; ++c) {
            const BF8 k = rows(a.k, a.ks, i, 32 * c + 8 * q4), q = rows(a.q, a.qs, i, 32 * c + 8 * q4);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float d = a.decay[(int64_t)(t + i) * a.ds + (int64_t)h * DK + 32 * c + 8 * q4 + j];
              const float x = fmaf(u, (float)k[j], S[v][2 * c + (j >> 2)][j & 3] * d);
              S[v][2 * c + (j >> 2)][j & 3] = x;
              o = fmaf(x, (float)q[j], o);
            }
          }
          o += __shfl_xor(o, 16);
          o += __shfl_xor(o, 32);
          if (a.skip) o = fmaf(skip, vv, o);
          const __bf16 y = (__bf16)o;
          if (q4 == 0) so[i * kVR + col + 16 * v] = __builtin_bit_cast(uint16_t, y);
        }
      }
    } else {
      BF4 vf[NV];                            // v: rows 4 q4 .. of the lane's column
#pragma unroll
      for (int v = 0; v < NV; ++v) vf[v] = read_tr(&sv[(4 * q4 + (m >> 2)) * kVR + (wave * NV + v) * 16 + 4 * (m & 3)]);
      if constexpr (OUT) {
        // ---- P (transposed: a lane gets 4 j of one i, which is the next product's operand)
        F4 p = (F4){0, 0, 0, 0}, O[NV];
        BF8 qf[kKS][3];
#pragma unroll
        for (int c = 0; c < kKS; ++c)
#pragma unroll
          for (int x = 0; x < 3; ++x) qf[c][x] = *(const BF8*)&sq[x][m * kR + 32 * c + 8 * q4];
#pragma unroll
        for (int c = 0; c < kKS; ++c) {
          BF8 kd[3];
#pragma unroll
          for (int x = 0; x < 3; ++x) kd[x] = *(const BF8*)&sk[x][m * kR + 32 * c + 8 * q4];
#pragma unroll
          for (int x = 0; x < 6; ++x) p = mfma(kd[first_of(x)], qf[c][second_of(x)], p);
        }
        // ---- products with the state
#pragma unroll
        for (int v = 0; v < NV; ++v) O[v] = (F4){0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < kKS; ++c) {
          BF8 sp[NV][3];
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = S[v][2 * c + (j >> 2)][j & 3];
            split(f, sp[v]);
          }
#pragma unroll
          for (int x = 0; x < 6; ++x)
#pragma unroll
            for (int v = 0; v < NV; ++v) O[v] = mfma(qf[c][first_of(x)], sp[v][second_of(x)], O[v]);
        }
        float f[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) f[r] = 4 * q4 + r <= m ? p[r] : 0.0f;
        uint2 pp[3];
#pragma unroll
        for (int x = 0; x < 3; ++x) pp[x] = make_uint2(take2(f[0], f[1]), take2(f[2], f[3]));
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
          for (int x = 0; x < 3; ++x) O[v] = mfma16(__builtin_bit_cast(BF4, pp[x]), vf[v], O[v]);
          if (a.skip)
#pragma unroll
            for (int r = 0; r < 4; ++r) O[v][r] = fmaf(skip, (float)vf[v][r], O[v][r]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const __bf16 y = (__bf16)O[v][r];
            so[(4 * q4 + r) * kVR + col + 16 * v] = __builtin_bit_cast(uint16_t, y);
          }
        }
      }
      // ---- the state
#pragma unroll
      for (int x = 0; x < 2 * kKS; ++x) {
        const F4 d = *(const F4*)&all[32 * (x >> 1) + 8 * q4 + 4 * (x & 1)];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[v][x][r] *= d[r];
      }
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int x = 0; x < 2 * kKS; ++x) {
          const BF4 kt = read_tr(&su[p][(4 * q4 + (m >> 2)) * kR + 32 * (x >> 1) + 8 * (m & 3) + 4 * (x & 1)]);
#pragma unroll
          for (int v = 0; v < NV; ++v) S[v][x] = mfma16(kt, vf[v], S[v][x]);
        }
    }
    __syncthreads();                         // outputs are in LDS, the block has been read
    if constexpr (OUT) {
      if (tid < kVP) {
        const int r = tid / (kDV / 8), c = tid % (kDV / 8) * 8;
        const Tile<VEC == 2> to(a.out, (int64_t)t * a.os + head + v0, a.os, n, min(kDV, a.dv - v0));
        to.store_step(r, c, 0, 0, *(const U4*)&so[r * kVR + c]);
      }
    }
  }

  float* to = OUT ? (sg.last ? a.final + (int64_t)sg.seq * a.H * a.dv * DK : nullptr)
                  : g.states + (int64_t)s * a.H * a.dv * DK;
  if (to) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (v0 + col + 16 * v < a.dv)
#pragma unroll
        for (int t = 0; t < 2 * kKS; ++t)
          *(F4*)(to + (head + v0 + col + 16 * v) * DK + 32 * (t >> 1) + 8 * q4 + 4 * (t & 1)) = S[v][t];
  }
  if (!OUT && wave == 0 && v0 == 0)
#pragma unroll
    for (int j = 0; j < kC; ++j) g.total[((int64_t)s * a.H + h) * DK + ch + j] = whole[j];
  if (!OUT && tid == 0 && v0 == 0 && sg.first) g.uncut[(int64_t)sg.seq * a.H + h] = 0;   // until the join finds otherwise
}

template <int DK, int NV, int VEC>
hipError_t key(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  const int vchunks = (a.dv + 64 * NV - 1) / (64 * NV);
  const uint32_t grid = (uint32_t)(g.count * a.H * vchunks);
  if (g.states) {
    k_scan_key<DK, NV, false, VEC><<<dim3(grid), 256, 0, s>>>(a, g, vchunks);
    const hipError_t e = launch_scan_join(a, g, s);
    if (e != hipSuccess) return e;
  }
  k_scan_key<DK, NV, true, VEC><<<dim3(grid), 256, 0, s>>>(a, g, vchunks);
  return hipGetLastError();
}

template <int DK>
hipError_t key_dk(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  // 128 columns a workgroup halve the operands' preparation; 256 channels leave
  // no registers for them
  if constexpr (DK < 256)
    if (a.dv > 64) return a.vec == 2 ? key<DK, 2, 2>(a, g, s) : a.vec ? key<DK, 2, 1>(a, g, s) : key<DK, 2, 0>(a, g, s);
  return a.vec == 2 ? key<DK, 1, 2>(a, g, s) : a.vec ? key<DK, 1, 1>(a, g, s) : key<DK, 1, 0>(a, g, s);
}

}  // namespace

hipError_t launch_scan_key(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  return a.dk == 64 ? key_dk<64>(a, g, s) : a.dk == 128 ? key_dk<128>(a, g, s) : key_dk<256>(a, g, s);
}

}  // namespace qs
