// Scan of packed prompts into states: the recurrence of the decode step, token
// by token, with the state in registers.
//
//   D = S diag(d_t);  u = beta (v - D k) (delta rule) or beta v (additive);
//   S = D + u k^T;    o = S q (+ skip v)
//
// A workgroup holds 16 * RPL value rows of one (sequence, head): 16 lanes a
// row group, each with dk/16 key channels of RPL rows.  Tokens come in stages
// of kStage: while one stage runs from LDS, the next is on its way into
// registers.  Sums over channels are 16-lane DPP reductions.  Everything is
// fp32.
//
// It carries fp32 prompts, short ones, and the delta rule with a decay a
// channel.  Bound by the chain from token to token (a reduction in it by the
// delta rule): 0.15 us a token of 64 channels, 0.19 of 128; 315 us for 2048 tokens
// of 8 heads of 64 x 64 in one piece.  So long sequences are cut.  Additive: one
// pass for the states that the segments add (no queries, no outputs), the join,
// one pass for the outputs; 45 us against 285 uncut for the same sizes.  Delta
// rule, of few heads: the first pass makes L and M of each piece, which maps the
// state before it to S M + L (M's rows: the state's of an identity with values of
// zero); 5120 tokens of 8 heads of 64 x 64: 128 us against 780.
#include <hip/hip_runtime.h>

#include "qstate_scan_tiles.hpp"

namespace qs {
namespace {

constexpr int kStage = 16;   // tokens staged in LDS at a time

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
}
// Sum over the 16 lanes of a DPP row; every lane gets the same bits.
__device__ __forceinline__ float sum16(float x) {
  x += dpp<0xB1>(x);    // lane ^ 1
  x += dpp<0x4E>(x);    // lane ^ 2
  x += dpp<0x141>(x);   // the other quad of the half row
  x += dpp<0x140>(x);   // the other half row
  return x;
}

template <int BF16>
__device__ __forceinline__ float get1(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  else return ((const float*)p)[i];
}

// N consecutive elements (N a multiple of 4) from global memory as fp32.
template <int BF16, int N>
__device__ __forceinline__ void get(const void* p, int64_t i, bool vec, float (&f)[N]) {
  if (vec) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      if constexpr (BF16) {
        const uint2 u = *(const uint2*)((const uint16_t*)p + i + j);
        f[j] = __uint_as_float(u.x << 16);
        f[j + 1] = __uint_as_float(u.x & 0xFFFF0000u);
        f[j + 2] = __uint_as_float(u.y << 16);
        f[j + 3] = __uint_as_float(u.y & 0xFFFF0000u);
      } else {
        const float4 u = *(const float4*)((const float*)p + i + j);
        f[j] = u.x; f[j + 1] = u.y; f[j + 2] = u.z; f[j + 3] = u.w;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = get1<BF16>(p, i + j);
  }
}

template <int BF16, int DK, bool DELTA, bool KEY, int RPL, bool OUT>
__global__ __launch_bounds__(256) void k_scan(const ScanArgs a, const ScanSegs gs, int rchunks) {
  constexpr int kRows = 16 * RPL;
  constexpr int kEl = kStage * DK / 256;   // staged elements a thread brings, of each of q, k, decay
  constexpr int kTh = DK / kEl;            // threads a token's row takes (16)
  constexpr int kM = DK / 64;              // groups of 4 channels a lane holds
  constexpr int kV = kStage * kRows / 256; // staged elements of v a thread brings
  static_assert(kTh == 16, "16 threads bring one token");
  __shared__ float sk[kStage][DK], sq[OUT ? kStage : 1][OUT ? DK : 1], sd[KEY ? kStage : 1][KEY ? DK : 1];
  __shared__ float sv[kStage][kRows], so[OUT ? kStage : 1][OUT ? kRows : 1], sg[kStage], sb[kStage];
  const int tid = (int)threadIdx.x;
  const int per = a.H * (DELTA && !OUT ? rchunks + DK / kRows : rchunks);
  const int sid = (int)(blockIdx.x / (uint32_t)per), hr = (int)(blockIdx.x % (uint32_t)per);
  const int h = hr / (per / a.H), rc = hr % (per / a.H);
  const int g = h / (a.H / a.G);
  Piece seg;
  if constexpr (DELTA) {
    seg = find_piece(a, gs.cut, sid);
  } else {
    const Segment x = find_segment(a, gs.seg, sid);
    seg = {x.seq, x.t0, x.t1, x.first, x.last, x.none, x.end};
  }
  const bool matrix = DELTA && !OUT && rc >= rchunks;   // rows of M
  if (OUT && !seg.none) outputs_of(seg, a, gs, h);
  if (seg.none || (!OUT && (seg.last || (matrix && seg.first)))) return;
  const int t0 = seg.t0, t1 = seg.t1;
  const int sub = tid & 15, row = (tid >> 4) * RPL;   // this lane's channels and first row
  const int r0 = (matrix ? rc - rchunks : rc) * kRows, rows = matrix ? DK : a.dv;
  // a sequence in one piece begins with its own state; of several pieces all
  // states are kept in the workspace (final may be initial)
  const int64_t own = ((int64_t)seg.seq * a.H + h) * a.dv * DK;
  float* kept = DELTA ? gs.total + (((int64_t)sid * a.H + h) * (a.dv + DK) + (matrix ? a.dv : 0)) * DK
                      : gs.states + ((int64_t)sid * a.H + h) * a.dv * DK;
  const bool whole = seg.first && seg.last;
  const float* from = OUT && !whole                                    ? kept
                      : (OUT || DELTA) && seg.first && a.initial ? a.initial + own
                                                                       : nullptr;
  float* to = !OUT ? kept : seg.last ? a.final + own : nullptr;

  float s[RPL][kM][4];
#pragma unroll
  for (int r = 0; r < RPL; ++r)
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      float4 x = make_float4(0, 0, 0, 0);
      if (from && !matrix && r0 + row + r < rows)
        x = *(const float4*)(from + (int64_t)(r0 + row + r) * DK + m * 64 + sub * 4);
      s[r][m][0] = x.x; s[r][m][1] = x.y; s[r][m][2] = x.z; s[r][m][3] = x.w;
      if (matrix)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[r][m][e] = m * 64 + sub * 4 + e == r0 + row + r ? 1.0f : 0.0f;
    }

  // what this thread brings of a stage: token bt, channels bc..; v: rows of token vt
  const int bt = tid >> 4, bc = (tid & 15) * kEl;
  float nk[kEl], nq[OUT ? kEl : 1], nd[KEY ? kEl : 1], nv[kV], ng = 1.0f, nb = 1.0f;
  auto fetch = [&](int t) {
    const bool in = t + bt < t1;
    const int64_t tt = t + bt;
#pragma unroll
    for (int j = 0; j < kEl; ++j) {
      nk[j] = 0.0f;
      if constexpr (OUT) nq[j] = 0.0f;
    }
    if (in) {
      get<BF16>(a.k, tt * a.ks + (int64_t)g * DK + bc, a.vec, nk);
      if constexpr (OUT) get<BF16>(a.q, tt * a.qs + (int64_t)g * DK + bc, a.vec, nq);
    }
    if constexpr (KEY) {
#pragma unroll
      for (int j = 0; j < kEl; ++j) nd[j] = in ? a.decay[tt * a.ds + (int64_t)h * DK + bc + j] : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int e = tid * kV + j, vt = e / kRows, vr = e % kRows;
      nv[j] = (!matrix && t + vt < t1 && r0 + vr < rows) ? get1<BF16>(a.v, (int64_t)(t + vt) * a.vs + (int64_t)h * a.dv + r0 + vr)
                                              : 0.0f;
    }
    ng = nb = 1.0f;
    if (tid < kStage && t + tid < t1) {
      if constexpr (!KEY) ng = a.decay[(int64_t)(t + tid) * a.ds + h];
      nb = a.beta ? a.beta[(int64_t)(t + tid) * a.bs + h] : 1.0f;
    }
  };

  [[maybe_unused]] float all[KEY ? kM : 1][4];
#pragma unroll
  for (int m = 0; m < (KEY ? kM : 1); ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) all[m][e] = 1.0f;
  fetch(t0);
  const float skip = a.skip ? a.skip[h] : 0.0f;
  for (int t = t0; t < t1; t += kStage) {
    __syncthreads();                       // the stage before has been read
#pragma unroll
    for (int j = 0; j < kEl; j += 4) {
      *(float4*)&sk[bt][bc + j] = make_float4(nk[j], nk[j + 1], nk[j + 2], nk[j + 3]);
      if constexpr (OUT) *(float4*)&sq[bt][bc + j] = make_float4(nq[j], nq[j + 1], nq[j + 2], nq[j + 3]);
      if constexpr (KEY) *(float4*)&sd[bt][bc + j] = make_float4(nd[j], nd[j + 1], nd[j + 2], nd[j + 3]);
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) (&sv[0][0])[tid * kV + j] = nv[j];
    if (tid < kStage) {
      if constexpr (!KEY) sg[tid] = ng;
      sb[tid] = nb;
    }
    __syncthreads();
    fetch(t + kStage);                     // reads nothing at or behind t1
    const int n = min(kStage, t1 - t);
    auto token = [&](int i) {
      float kk[kM][4], qq[OUT ? kM : 1][4], dd[KEY ? kM : 1][4];
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const float4 x = *(const float4*)&sk[i][m * 64 + sub * 4];
        kk[m][0] = x.x; kk[m][1] = x.y; kk[m][2] = x.z; kk[m][3] = x.w;
        if constexpr (OUT) {
          const float4 y = *(const float4*)&sq[i][m * 64 + sub * 4];
          qq[m][0] = y.x; qq[m][1] = y.y; qq[m][2] = y.z; qq[m][3] = y.w;
        }
        if constexpr (KEY) {
          const float4 z = *(const float4*)&sd[i][m * 64 + sub * 4];
          dd[m][0] = z.x; dd[m][1] = z.y; dd[m][2] = z.z; dd[m][3] = z.w;
        }
      }
      const float d = KEY ? 1.0f : sg[i], beta = sb[i];
      float o[RPL];
#pragma unroll
      for (int r = 0; r < RPL; ++r) {
        float w = 0.0f;
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[r][m][e] *= KEY ? dd[KEY ? m : 0][e] : d;
            if constexpr (DELTA) w = fmaf(s[r][m][e], kk[m][e], w);
          }
        float u = sv[i][row + r];
        if constexpr (DELTA) u -= sum16(w);
        u *= beta;
        o[r] = 0.0f;
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[r][m][e] = fmaf(u, kk[m][e], s[r][m][e]);
            if constexpr (OUT) o[r] = fmaf(s[r][m][e], qq[OUT ? m : 0][e], o[r]);
          }
        if constexpr (OUT) o[r] = sum16(o[r]);
      }
      if constexpr (OUT)
#pragma unroll
        for (int r = 0; r < RPL; ++r)
          if (sub == r) so[i][row + r] = o[r];
      if constexpr (!OUT && !DELTA) {        // the segment's whole decay
        if constexpr (KEY) {
#pragma unroll
          for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) all[m][e] *= dd[m][e];
        } else {
          all[0][0] *= d;
        }
      }
    };
    // four tokens at a time, so that the next ones' channels are read meanwhile
    int i = 0;
    for (; i + 4 <= n; i += 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) token(i + j);
    }
    for (; i < n; ++i) token(i);
    if constexpr (!OUT) continue;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int e = j * 256 + tid, vt = e / kRows, vr = e % kRows;
      if (vt < n && r0 + vr < a.dv) {
        const float y = fmaf(skip, sv[vt][vr], so[OUT ? vt : 0][OUT ? vr : 0]);
        const int64_t at = (int64_t)(t + vt) * a.os + (int64_t)h * a.dv + r0 + vr;
        if constexpr (BF16) {
          const __bf16 b = (__bf16)y;
          ((uint16_t*)a.out)[at] = __builtin_bit_cast(uint16_t, b);
        } else {
          ((float*)a.out)[at] = y;
        }
      }
    }
  }
  if (to)
#pragma unroll
    for (int r = 0; r < RPL; ++r)
      if (r0 + row + r < rows)
#pragma unroll
        for (int m = 0; m < kM; ++m)
          *(float4*)(to + (int64_t)(r0 + row + r) * DK + m * 64 + sub * 4) =
              make_float4(s[r][m][0], s[r][m][1], s[r][m][2], s[r][m][3]);
  if (!OUT && seg.first && rc == 0 && tid == 0) gs.uncut[(int64_t)seg.seq * a.H + h] = 0;   // until the join finds otherwise
  if (!OUT && !DELTA && rc == 0 && tid < 16) {
    if constexpr (KEY) {
#pragma unroll
      for (int m = 0; m < kM; ++m)
        *(float4*)&gs.total[((int64_t)sid * a.H + h) * DK + m * 64 + sub * 4] =
            make_float4(all[m][0], all[m][1], all[m][2], all[m][3]);
    } else if (tid == 0) {
      gs.total[(int64_t)sid * a.H + h] = all[0][0];
    }
  }
}

template <int BF16, int DK, bool DELTA, bool KEY, int RPL>
hipError_t scan_rows(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  const int rchunks = (a.dv + 16 * RPL - 1) / (16 * RPL);
  const int pieces = !DELTA ? g.count : a.n + (g.cut > 0 ? (a.T - 1) / g.cut : 0);
  const uint32_t grid = (uint32_t)(pieces * a.H * rchunks);
  if constexpr (DELTA) {
    if (g.cut > 0) {
      const uint32_t both = (uint32_t)(pieces * a.H * (rchunks + DK / (16 * RPL)));
      k_scan<BF16, DK, DELTA, KEY, RPL, false><<<dim3(both), 256, 0, s>>>(a, g, rchunks);
      const hipError_t e = launch_delta_join(a, g, s);
      if (e != hipSuccess) return e;
    }
  } else {
    if (g.states) {
      k_scan<BF16, DK, DELTA, KEY, RPL, false><<<dim3(grid), 256, 0, s>>>(a, g, rchunks);
      const hipError_t e = launch_scan_join(a, g, s);
      if (e != hipSuccess) return e;
    }
  }
  k_scan<BF16, DK, DELTA, KEY, RPL, true><<<dim3(grid), 256, 0, s>>>(a, g, rchunks);
  return hipGetLastError();
}

// One row a lane has the shorter chain, two read the channels half as often.
// Up to 16384 rows in all (1024 workgroups of one row a lane) the chain counts:
// delta rule, one decay a head, 2048 tokens of 8 heads of 64 x 64: 378 us with
// one, 548 us with two; of 32 heads of 128 x 128: 381, 551; 8 times 256 tokens
// of 32 heads of 128 x 128 (32768 rows): 194, 179.
template <int BF16, int DK, bool DELTA, bool KEY>
hipError_t scan(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  return (int64_t)g.count * a.H * a.dv <= 16384 ? scan_rows<BF16, DK, DELTA, KEY, 1>(a, g, s)
                                                : scan_rows<BF16, DK, DELTA, KEY, 2>(a, g, s);
}

template <int BF16, int DK>
hipError_t scan_dk(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  if (a.delta) return a.key ? scan<BF16, DK, true, true>(a, g, s) : scan<BF16, DK, true, false>(a, g, s);
  return a.key ? scan<BF16, DK, false, true>(a, g, s) : scan<BF16, DK, false, false>(a, g, s);
}

template <int BF16>
hipError_t scan_in(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  return a.dk == 64 ? scan_dk<BF16, 64>(a, g, s)
                    : a.dk == 128 ? scan_dk<BF16, 128>(a, g, s) : scan_dk<BF16, 256>(a, g, s);
}

}  // namespace

hipError_t launch_scan(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  return a.bf16 ? scan_in<1>(a, g, s) : scan_in<0>(a, g, s);
}

}  // namespace qs
