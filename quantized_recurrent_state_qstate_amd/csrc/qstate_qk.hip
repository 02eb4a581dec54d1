// Norm of queries and keys for each head with the position rotation, in one
// pass: the rows are read once and written once.
//
//   y = x / sqrt(sum x^2 + eps)            (norm 1, L2: the delta rule's keys)
//   y = x / sqrt(mean x^2 + eps) * w       (norm 2, RMS; w optional)
//   pairs (a, b) of y's first `rot` channels -> (a cos - b sin, a sin + b cos),
//   angle = position * frequency[pair], pairs (i, i + rot/2) or (2i, 2i+1);
//   out = y * scale.
//
// Everything in fp32 but the angle: position * frequency / 2 pi is formed in
// fp64 and reduced to (-1/2, 1/2] turns there, so a position of 2^20 loses
// nothing; sine and cosine of the reduced turn are fp32.  A workgroup takes
// heads of one token and computes the token's cos and sin once, into LDS,
// while its first rows are on their way.  Bound by HBM: 8192 tokens of 64 heads
// of 128 in bf16 take 52-54 us, 5.0-5.2 TB/s, as a copy; 64 tokens 3.9 us.
#include <hip/hip_runtime.h>

#include "qstate_ops.hpp"

namespace qs {
namespace {

template <int BF16>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&f)[8]) {
  if constexpr (BF16) {
    const uint4 u = *(const uint4*)((const uint16_t*)p + i);
    const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(d[j] << 16);
      f[2 * j + 1] = __uint_as_float(d[j] & 0xFFFF0000u);
    }
  } else {
    const float4 a = *(const float4*)((const float*)p + i), b = *(const float4*)((const float*)p + i + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}

template <int BF16>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&f)[8]) {
  if constexpr (BF16) {
    uint32_t d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __bf16 lo = (__bf16)f[2 * j], hi = (__bf16)f[2 * j + 1];
      d[j] = (uint32_t)__builtin_bit_cast(uint16_t, lo) | ((uint32_t)__builtin_bit_cast(uint16_t, hi) << 16);
    }
    *(uint4*)((uint16_t*)p + i) = make_uint4(d[0], d[1], d[2], d[3]);
  } else {
    *(float4*)((float*)p + i) = make_float4(f[0], f[1], f[2], f[3]);
    *(float4*)((float*)p + i + 4) = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// L lanes (a power of two, 8 channels each, 8 L >= dim) hold one head.
template <int BF16, int L>
__global__ __launch_bounds__(256) void k_qk(const QkArgs a, int splits, int per) {
  __shared__ float cs[2][256];             // cos, sin of the token's pairs (rot <= 512)
  const int t = (int)blockIdx.x / splits;
  const int h0 = ((int)blockIdx.x % splits) * per;
  const int nh = a.heads[0] + a.heads[1];
  const int h1 = min(h0 + per, nh);
  const int lane = (int)threadIdx.x & (L - 1);
  const int c = lane * 8;
  const bool in = c < a.dim;
  constexpr int kHeads = 256 / L;          // heads the workgroup holds at a time
  int h = h0 + (int)threadIdx.x / L;
  auto load = [&](int hh, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    if (in && hh < h1) {
      const int s = hh >= a.heads[0];
      const int64_t i = (int64_t)t * a.xs[s] + (int64_t)(hh - (s ? a.heads[0] : 0)) * a.dim + c;
      load8<BF16>(a.x[s], i, f);
    }
  };
  float f[8];
  load(h, f);
  const int half = a.rot >> 1;
  if (a.rot) {
    for (int p = (int)threadIdx.x; p < half; p += 256) {
      const double turns = (double)a.position[t] * (a.frequency[p] * 0.15915494309189533577);
      float sn, cn;
      sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cn);
      cs[0][p] = cn;
      cs[1][p] = sn;
    }
    __syncthreads();
  }
  for (int hb = h0; hb < h1; hb += kHeads) {
    h = hb + (int)threadIdx.x / L;
    float next[8];
    load(h + kHeads, next);                // the next heads' rows are on their way meanwhile
    const int s = h >= a.heads[0];
    if (a.norm) {
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
#pragma unroll
      for (int m = 1; m < L; m <<= 1) ss += __shfl_xor(ss, m);
      float inv = 1.0f / sqrtf((a.norm == 2 ? ss / (float)a.dim : ss) + a.eps);
      // Squares beyond fp32, or (where eps is not above what they could add) subnormal
      // ones: again with x 2^-70, where eps is nothing, or x 2^100.
      const bool large = ss > 0x1p126f, tiny = a.eps < 0x1p-70f && ss < 0x1p-100f;
      if (__ballot(large || tiny)) {
        const float by = large ? 0x1p-70f : tiny ? 0x1p100f : 1.0f;
        float s2 = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = f[j] * by;
          s2 = fmaf(x, x, s2);
        }
#pragma unroll
        for (int m = 1; m < L; m <<= 1) s2 += __shfl_xor(s2, m);
        if (large || tiny) {
          inv = 1.0f / sqrtf((a.norm == 2 ? s2 / (float)a.dim : s2) + a.eps * by * by);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] *= by;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= inv;
      const float* w = a.w[s];
      if (w && in) {
        float g[8];
        load8<0>(w, c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= g[j];
      }
    }
    if (a.rot) {
      if (a.interleaved) {
        if (c < a.rot) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float cn = cs[0][(c >> 1) + j], sn = cs[1][(c >> 1) + j];
            const float x = f[2 * j], y = f[2 * j + 1];
            f[2 * j] = fmaf(-y, sn, x * cn);
            f[2 * j + 1] = fmaf(y, cn, x * sn);
          }
        }
      } else {
        // the partner of channel c + j is c + j +- rot/2: rot/16 lanes away
        const bool low = c < half;
        const int from = ((int)threadIdx.x & 63) + (low ? (half >> 3) : -(half >> 3));
        float g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = __shfl(f[j], from & 63);
        if (c < a.rot) {
          const int p = low ? c : c - half;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float cn = cs[0][p + j], sn = cs[1][p + j];
            f[j] = low ? fmaf(-g[j], sn, f[j] * cn) : fmaf(f[j], cn, g[j] * sn);
          }
        }
      }
    }
    if (in && h < h1) {
      const float scale = a.scale[s];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= scale;
      store8<BF16>(a.y[s], (int64_t)t * a.ys[s] + (int64_t)(h - (s ? a.heads[0] : 0)) * a.dim + c, f);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = next[j];
  }
}

template <int BF16, int L>
hipError_t qk(const QkArgs& a, hipStream_t s) {
  // A few tokens alone would leave most compute units empty: their heads are
  // split over workgroups, down to one round of heads each.
  const int nh = a.heads[0] + a.heads[1], round = 256 / L;
  int splits = 1;
  while (a.T * splits < 512 && (nh + splits - 1) / splits > round) splits *= 2;
  const int per = ((nh + splits - 1) / splits + round - 1) / round * round;
  splits = (nh + per - 1) / per;
  const int64_t most = max_blocks(256) / splits, es = BF16 ? 2 : 4;   // tokens of a launch
  for (int64_t t = 0; t < a.T; t += most) {
    QkArgs part = a;
    part.T = (int32_t)(a.T - t < most ? a.T - t : most);
    for (int i = 0; i < 2; ++i) {
      if (!a.heads[i]) continue;
      part.x[i] = (const char*)a.x[i] + t * a.xs[i] * es;
      part.y[i] = (char*)a.y[i] + t * a.ys[i] * es;
    }
    if (a.position) part.position = a.position + t;
    k_qk<BF16, L><<<dim3((uint32_t)(part.T * splits)), 256, 0, s>>>(part, splits, per);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_qk(const QkArgs& a, hipStream_t s) {
  const int lanes = (a.dim + 7) / 8;
#define QS_QK_PICK(B)                                  \
  return lanes <= 8 ? qk<B, 8>(a, s)                   \
         : lanes <= 16 ? qk<B, 16>(a, s)               \
         : lanes <= 32 ? qk<B, 32>(a, s) : qk<B, 64>(a, s);
  if (a.bf16) {
    QS_QK_PICK(1)
  }
  QS_QK_PICK(0)
}

}  // namespace qs
