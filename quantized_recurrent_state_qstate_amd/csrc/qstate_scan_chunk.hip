// Scan of packed bf16 prompts, additive with one decay a head, 64 tokens at a
// time on the matrix cores.
//
// With c_i the sum of log2 decays from a chunk's first token to token i, u = beta v
// and S the state before the chunk,
//   S_i = 2^{c_i} S + sum_{j<=i} 2^{c_i - c_j} u_j k_j^T,
//   o_i = 2^{c_i} S q_i + sum_{j<=i} P_ij v_j,   P_ij = 2^{c_i - c_j} beta_j k_j.q_i,
// and the state after the chunk is the last S_i.
//
// Precision: q, k and v are bf16, so a product with one of them is exact when
// the other operand, w v in the state's update, S and P in the outputs, is cut
// into three bf16 pieces, which hold its 24 bits.  All sums are fp32; an output
// is rounded to bf16 once.  c is summed in fp64:
// differences of long sums of logs would lose the decays between neighbours;
// a decay of zero counts as 2^-10000.
//
// A workgroup holds 16 NV WAVES value columns of one (segment, head): each wave
// keeps the state of its columns in accumulators [dk][v], which are the second
// operand of S q as they are (the tiles' rows are dealt so that a lane holds 8
// channels in a row); k, q, v and P go through LDS.
//
// Segments: sequences may be cut at multiples of `seg` tokens.  Then three
// launches: the state each segment adds by itself, the states between
// segments, and the outputs; so that few long sequences fill the device.
//
// 16384 tokens of 32 heads of 128 x 64 in 16 segments: 156 us.  Under a trace,
// which makes them longer (171 in all), the local states take 41, the states
// between 13, the outputs 117, of which vector instructions fill 30%, matrix
// instructions 23%: what is left is LDS and waiting, with the two waves a SIMD that
// 73 KB of LDS and 223 registers allow.  With outputs of two pieces, 142 us in all
// then, chunks of 32 tokens (three waves) measured 145-149, and LDS rows whose
// pieces are exchanged against bank conflicts the same 142.
#include <hip/hip_runtime.h>

#include "qstate_scan_tiles.hpp"

namespace qs {
namespace {

template <int DK, int NV, int WAVES, bool OUT, int VEC>
__global__ __launch_bounds__(64 * WAVES, DK <= 128 && VEC > 0 ? 2 : 1) void k_scan_chunk(const ScanArgs a, const ScanSegs g, int vchunks) {
  constexpr int kT = 64 * WAVES;            // threads
  constexpr int kDV = 16 * NV * WAVES;      // value columns
  constexpr int kKS = DK / 32;              // steps of 32 channels
  constexpr int kKR = DK + 8, kVR = kDV + 8, kPR = kL + 8;   // LDS rows: 16 bytes more than they need
  constexpr int kKP = kL * DK / 8 / kT, kVP = kL * kDV / 8 / kT;           // 16-byte pieces a thread brings
  __shared__ __attribute__((aligned(16))) uint16_t sk[kL * kKR];
  __shared__ __attribute__((aligned(16))) uint16_t sq[OUT ? kL * kKR : 8];
  __shared__ __attribute__((aligned(16))) uint16_t sv[kL * kVR];           // v, then the outputs
  __shared__ __attribute__((aligned(16))) uint16_t sp[OUT ? 3 : 1][OUT ? kL * kPR : 8];   // P's three pieces
  __shared__ __attribute__((aligned(16))) float sc[2][kL];                 // c_i as a sum of two floats
  __shared__ __attribute__((aligned(16))) float se[kL], sw[kL], sb[kL];    // 2^{c_i}, weight in the update, beta
  __shared__ int sgrow;

  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, q4 = lane >> 4;
  const int per = a.H * vchunks;
  const int s = (int)(blockIdx.x / (uint32_t)per), hv = (int)(blockIdx.x % (uint32_t)per);
  const int h = hv / vchunks, v0 = (hv % vchunks) * kDV;
  const int kh = h / (a.H / a.G);
  Segment sg = find_segment(a, g.seg, s);
  if (OUT && !sg.none) outputs_of(sg, a, g, h);
  if (sg.none || (!OUT && sg.last)) return;
  const int64_t head = (int64_t)h * a.dv;

  // state tiles: row 4 q4 + r of tile 2 i + j is channel 32 i + 8 q4 + 4 j + r, column m is value v0 + ...
  F4 S[NV][2 * kKS];
  const int vcol = (wave * NV) * 16 + m;
  const float* from = !OUT ? nullptr
                      // a sequence in one piece; of several, the first one's state is kept with the
                      // others, since the last one may write it over (final may be initial)
                      : sg.first && sg.last ? (a.initial ? a.initial + (int64_t)sg.seq * a.H * a.dv * DK : nullptr)
                                            : g.states + (int64_t)s * a.H * a.dv * DK;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int v = v0 + vcol + 16 * n;
#pragma unroll
    for (int t = 0; t < 2 * kKS; ++t) {
      S[n][t] = (F4){0, 0, 0, 0};
      if (from && v < a.dv) S[n][t] = *(const F4*)(from + (head + v) * DK + 32 * (t >> 1) + 8 * q4 + 4 * (t & 1));
    }
  }
  // the pieces this thread brings: rows kr, kr + kKStep, ..., column kc on; the same for v
  constexpr int kKStep = kT * 8 / DK, kVStep = kT * 8 / kDV;
  const int kr = tid / (DK / 8), kc = tid % (DK / 8) * 8, vr = tid / (kDV / 8), vc = tid % (kDV / 8) * 8;
  U4 nk[kKP], nq[OUT ? kKP : 1], nv[kVP];
  float nd = 1.0f, nb = 0.0f;
  auto fetch = [&](int t, int t1) {
    const int rows = min(kL, t1 - t);
    const Tile<(VEC > 0)> tk(a.k, (int64_t)t * a.ks + (int64_t)kh * DK, a.ks, rows, DK);
    const Tile<(VEC > 0)> tq(OUT ? a.q : a.k, OUT ? (int64_t)t * a.qs + (int64_t)kh * DK : 0, a.qs, rows, DK);
    const Tile<VEC == 2> tv(a.v, (int64_t)t * a.vs + head + v0, a.vs, rows, min(kDV, a.dv - v0));
#pragma unroll
    for (int i = 0; i < kKP; ++i) {
      nk[i] = tk.load_step(kr, kc, i, kKStep);
      if constexpr (OUT) nq[i] = tq.load_step(kr, kc, i, kKStep);
    }
#pragma unroll
    for (int i = 0; i < kVP; ++i) nv[i] = tv.load_step(vr, vc, i, kVStep);
    nd = 1.0f;
    nb = 0.0f;
    if (tid < kL && t + tid < t1) {
      nd = a.decay[(int64_t)(t + tid) * a.ds + h];
      nb = a.beta ? a.beta[(int64_t)(t + tid) * a.bs + h] : 1.0f;
    }
  };
  // S = 2^{c of the last token} S + sum_j k_j (w_j u_j)^T, four tiles at a time
  auto update = [&](const BF8 (&wu)[NV][2][3], float eall) {
#pragma unroll
    for (int t4 = 0; t4 < 2 * kKS; t4 += 4) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int t = t4; t < t4 + 4; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[v][t][r] *= eall;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        BF8 kt[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint16_t* x =
              &sk[(32 * c + 4 * q4 + (m >> 2)) * kKR + 32 * ((t4 + t) >> 1) + 8 * (m & 3) + 4 * (t & 1)];
          kt[t] = join(read_tr(x), read_tr(x + 16 * kKR));
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int t = 0; t < 4; ++t) S[v][t4 + t] = mfma(kt[t], wu[v][c][p], S[v][t4 + t]);
      }
    }
  };

  double total = 0.0;
  [[maybe_unused]] bool lost[NV] = {};       // this lane's columns whose state is not finite any more
  fetch(sg.t0, sg.t1);
  for (int t = sg.t0; t < sg.t1;) {
    const int n = min(kL, sg.t1 - t);
    // ---- this chunk into LDS; gates
    __syncthreads();                         // the chunk before has been read
#pragma unroll
    for (int i = 0; i < kKP; ++i) {
      *(U4*)&sk[kr * kKR + kc + i * (kKStep * kKR)] = nk[i];
      if constexpr (OUT) *(U4*)&sq[kr * kKR + kc + i * (kKStep * kKR)] = nq[i];
    }
#pragma unroll
    for (int i = 0; i < kVP; ++i) *(U4*)&sv[vr * kVR + vc + i * (kVStep * kVR)] = nv[i];
    if (wave == 0) {
      const double c = wave_sums(nd == 0.0f ? -10000.0 : (double)log2f(nd));
      const double all = __shfl(c, 63);
      sc[0][lane] = (float)c;
      sc[1][lane] = (float)(c - (double)(float)c);
      sb[lane] = nb;
      const float e = __builtin_amdgcn_exp2f((float)c), w = __builtin_amdgcn_exp2f((float)(all - c));
      se[lane] = e;
      sw[lane] = w * nb;
      const bool grow = __ballot(e >= 0x1p100f || w >= 0x1p100f) != 0;
      if constexpr (OUT) sgrow = grow;
      else if (grow) total = NAN;            // the sequence is not cut
    }
    __syncthreads();
    const int next = t + n;
    if (next < sg.t1) fetch(next, sg.t1);
    if constexpr (!OUT) total += (double)sc[0][kL - 1] + (double)sc[1][kL - 1];
    const float eall = se[kL - 1];

    if constexpr (OUT) {
      // ---- P (transposed tiles: a lane gets 4 j of one i)
#pragma unroll
      for (int x = 0; x < 4 / WAVES; ++x) {
        const int it = WAVES == 4 ? wave : (x ? 3 - wave : wave);
        const int i = 16 * it + m;
        const float ci = sc[0][i], di = sc[1][i];
        // two tiles at a time, to the end of the step of 32 that the products below
        // read: right of the diagonal they become zeros
        for (int jp = 0; jp <= it; jp += 2) {
          F4 p[2] = {(F4){0, 0, 0, 0}, (F4){0, 0, 0, 0}};
#pragma unroll
          for (int c = 0; c < kKS; ++c) {
            const BF8 qi = *(const BF8*)&sq[i * kKR + 32 * c + 8 * q4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const BF8 kj = *(const BF8*)&sk[(16 * (jp + y) + m) * kKR + 32 * c + 8 * q4];
              p[y] = mfma(kj, qi, p[y]);
            }
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int j = 16 * (jp + y) + 4 * q4;
            const F4 bj = *(const F4*)&sb[j];
            const F4 cj = *(const F4*)&sc[0][j], dj = *(const F4*)&sc[1][j];
            float f[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float e = __builtin_amdgcn_exp2f((ci - cj[r]) + (di - dj[r]));
              const float w = p[y][r] * e * bj[r];
              f[r] = j + r <= i ? w : 0.0f;
            }
            *(uint2*)&sp[0][i * kPR + j] = make_uint2(take2(f[0], f[1]), take2(f[2], f[3]));
            *(uint2*)&sp[1][i * kPR + j] = make_uint2(take2(f[0], f[1]), take2(f[2], f[3]));
            *(uint2*)&sp[2][i * kPR + j] = make_uint2(round2(f[0], f[1]), round2(f[2], f[3]));
          }
        }
      }
      __syncthreads();
      // ---- products with the state
      F4 O[NV][4];
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) O[v][i] = (F4){0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < kKS; ++c) {
        BF8 sp_[NV][3];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = S[v][2 * c + (j >> 2)][j & 3];
          split(f, sp_[v]);
        }
        BF8 qf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[i] = *(const BF8*)&sq[(16 * i + m) * kKR + 32 * c + 8 * q4];
        // products on one accumulator are kept apart: each takes several issue slots
#pragma unroll
        for (int x = 0; x < 3; ++x)
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i) O[v][i] = mfma(qf[i], sp_[v][x], O[v][i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F4 e = *(const F4*)&se[16 * i + 4 * q4];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int r = 0; r < 4; ++r) O[v][i][r] *= e[r];
      }
      // ---- outputs: P u on top
      BF8 ub[2][NV];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const uint16_t* x = &sv[(32 * c + 4 * q4 + (m >> 2)) * kVR + (wave * NV + v) * 16 + 4 * (m & 3)];
          ub[c][v] = join(read_tr(x), read_tr(x + 16 * kVR));
        }
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          BF8 p[4];
#pragma unroll
          for (int i = 2 * c; i < 4; ++i) {
            const uint16_t* y = &sp[x][(16 * i + m) * kPR + 32 * c + 4 * q4];
            p[i] = join(*(const BF4*)y, *(const BF4*)(y + 16));
          }
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 2 * c; i < 4; ++i) O[v][i] = mfma(p[i], ub[c][v], O[v][i]);
        }
      }
      // ---- weighted v; then the outputs take v's place
      BF8 wu[NV][2][3];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        F4 W[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) W[j] = *(const F4*)&sw[32 * c + 16 * j + 4 * q4];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = W[j >> 2][j & 3] * (float)ub[c][v][j];
          split(f, wu[v][c]);
        }
      }
      if (a.skip) {
        const float skip = a.skip[h];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              O[v][2 * c + (j >> 2)][j & 3] = fmaf(skip, (float)ub[c][v][j], O[v][2 * c + (j >> 2)][j & 3]);
      }
      // ---- An output that is not finite, or nearly so: a value that was not, which the
      // zeros in P bring to earlier tokens, or products that leave fp32 where the
      // recurrence does not.  Then the outputs are made token by token; the state too, if
      // it is v or decays that grow, else (a query) it is taken back from its place in memory.
      bool out_of_range = false;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = highest(top, O[v][i]);
        out_of_range |= top >= kHuge && !lost[v];
      }
      if (sgrow || __ballot(out_of_range)) {
        H2 most = (H2){0, 0};
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int v = 0; v < NV; ++v) most = largest(most, __builtin_bit_cast(U4, ub[c][v]));
        const bool anew = sgrow || __ballot(odd(most));
        float* kept = sg.last ? a.final + (int64_t)sg.seq * a.H * a.dv * DK : g.states + (int64_t)s * a.H * a.dv * DK;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int col = v0 + vcol + 16 * v;
          if (!anew && col < a.dv)
#pragma unroll
            for (int y = 0; y < 2 * kKS; ++y)
              *(F4*)(kept + (head + col) * DK + 32 * (y >> 1) + 8 * q4 + 4 * (y & 1)) = S[v][y];
          by_token<DK, false>(
              a, t, n, h, [&](int i, int c) { return *(const BF8*)&sk[i * kKR + c]; },
              [&](int i, int c) { return *(const BF8*)&sq[i * kKR + c]; },
              [&](int i) { return __uint_as_float((uint32_t)sv[i * kVR + (wave * NV + v) * 16 + m] << 16); },
              [&](int i, float o) {
                const __bf16 y = (__bf16)o;
                sv[i * kVR + (wave * NV + v) * 16 + m] = __builtin_bit_cast(uint16_t, y);
              },
              S[v]);
          lost[v] = spoiled(S[v]);
          if (!anew && col < a.dv)
#pragma unroll
            for (int y = 0; y < 2 * kKS; ++y)
              S[v][y] = *(const F4*)(kept + (head + col) * DK + 32 * (y >> 1) + 8 * q4 + 4 * (y & 1));
        }
        if (!anew) update(wu, eall);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const __bf16 y = (__bf16)O[v][i][r];
              sv[(16 * i + 4 * q4 + r) * kVR + (wave * NV + v) * 16 + m] = __builtin_bit_cast(uint16_t, y);
            }
        update(wu, eall);
      }
    } else {
      BF8 wu[NV][2][3];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const uint16_t* x = &sv[(32 * c + 4 * q4 + (m >> 2)) * kVR + (wave * NV + v) * 16 + 4 * (m & 3)];
          const BF8 y = join(read_tr(x), read_tr(x + 16 * kVR));
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = sw[32 * c + 16 * (j >> 2) + 4 * q4 + (j & 3)] * (float)y[j];
          split(f, wu[v][c]);
        }
      update(wu, eall);
    }
    if constexpr (OUT) {
      __syncthreads();                       // outputs are in LDS, the chunk has been read
      const Tile<VEC == 2> to(a.out, (int64_t)t * a.os + head + v0, a.os, n, min(kDV, a.dv - v0));
#pragma unroll
      for (int i = 0; i < kVP; ++i) to.store_step(vr, vc, i, kVStep, *(const U4*)&sv[vr * kVR + vc + i * (kVStep * kVR)]);
    }
    t = next;
  }

  float* to = OUT ? (sg.last ? a.final + (int64_t)sg.seq * a.H * a.dv * DK : nullptr)
                  : g.states + (int64_t)s * a.H * a.dv * DK;
  if (to) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = v0 + vcol + 16 * v;
      if (col < a.dv)
#pragma unroll
        for (int t = 0; t < 2 * kKS; ++t)
          *(F4*)(to + (head + col) * DK + 32 * (t >> 1) + 8 * q4 + 4 * (t & 1)) = S[v][t];
    }
  }
  if (!OUT && tid == 0 && v0 == 0) {
    g.total[(int64_t)s * a.H + h] = __builtin_amdgcn_exp2f((float)total);
    if (sg.first) g.uncut[(int64_t)sg.seq * a.H + h] = 0;   // until the join finds otherwise
  }
}

// States between segments: for each sequence, S = initial, then S = decay S + local
// from segment to segment; segment s's place takes the state before it.  Of the
// long sequences alone there is at most one that begins in a cell of `least`
// tokens, the last that does, so there are as many workgroups as cells need: one
// for each short one that does nothing cost 40 us (256 of 32 heads of 128 x 64).
__global__ __launch_bounds__(256) void k_scan_join(const ScanArgs a, const ScanSegs g, int blocks) {
  int seq = (int)blockIdx.x / blocks;
  if (a.least > 0) {
    const int cell = seq;
    seq = last_sequence(a, [&](int i) { return min(max(a.offsets[i], 0), a.T) / a.least <= cell; });
    if (min(max(a.offsets[seq], 0), a.T) / a.least != cell) return;
  }
  const int64_t per = (int64_t)a.dv * a.dk / 4, all = per * a.H;
  const int64_t e = (int64_t)((int)blockIdx.x % blocks) * 256 + threadIdx.x;
  if (e >= all) return;
  const int h = (int)(e / per);
  const int start = a.offsets ? min(max(a.offsets[seq], 0), a.T) : 0;
  const int end = a.offsets ? min(max(a.offsets[seq + 1], start), a.T) : a.T;
  if (end <= start || end - start < a.least || end - start > a.most) return;
  const int c0 = start / g.seg, c1 = (end - 1) / g.seg;
  if (c0 == c1) return;                      // not cut
  bool numbers = true;
  F4* st = (F4*)g.states;
  F4 S = (F4){0, 0, 0, 0};
  if (a.initial) S = ((const F4*)a.initial)[(int64_t)seq * all + e];
  // kAhead segments' states are asked for at a time: one by one, their latency
  // is the launch (16 segments of 32 heads of 128 x 64: 9.9 us)
  constexpr int kAhead = 8;
  for (int c = c0; c < c1; c += kAhead) {
    F4 L[kAhead], d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (c + i >= c1) break;
      const int64_t s = c + i + seq;
      L[i] = st[s * all + e];
      if (a.key) {
        d[i] = *(const F4*)&g.total[(s * a.H + h) * a.dk + e * 4 % a.dk];
      } else {
        const float x = g.total[s * a.H + h];
        d[i] = (F4){x, x, x, x};
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (c + i >= c1) break;
      st[(int64_t)(c + i + seq) * all + e] = S;   // what was there is in L
#pragma unroll
      for (int r = 0; r < 4; ++r) S[r] = fmaf(d[i][r], S[r], L[i][r]);
      numbers &= finite(d[i]);
    }
  }
  if (!numbers) g.uncut[(int64_t)seq * a.H + h] = 1;
  st[(int64_t)(c1 + seq) * all + e] = S;
}

template <int DK, int NV, int WAVES, int VEC>
hipError_t chunk(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  const int vchunks = (a.dv + 16 * NV * WAVES - 1) / (16 * NV * WAVES);
  const uint32_t grid = (uint32_t)(g.count * a.H * vchunks);
  if (g.states) {
    k_scan_chunk<DK, NV, WAVES, false, VEC><<<dim3(grid), 64 * WAVES, 0, s>>>(a, g, vchunks);
    const hipError_t e = launch_scan_join(a, g, s);
    if (e != hipSuccess) return e;
  }
  k_scan_chunk<DK, NV, WAVES, true, VEC><<<dim3(grid), 64 * WAVES, 0, s>>>(a, g, vchunks);
  return hipGetLastError();
}

template <int DK>
hipError_t chunk_dk(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  return a.vec == 2 ? chunk<DK, 1, 4, 2>(a, g, s) : a.vec ? chunk<DK, 1, 4, 1>(a, g, s) : chunk<DK, 1, 4, 0>(a, g, s);
}

}  // namespace

hipError_t launch_scan_join(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  const int blocks = (int)(((int64_t)a.H * a.dv * a.dk / 4 + 255) / 256);
  const int sequences = a.least > 0 ? a.T / a.least : a.n;
  k_scan_join<<<dim3((uint32_t)(sequences * blocks)), 256, 0, s>>>(a, g, blocks);
  return hipGetLastError();
}

hipError_t launch_scan_chunk(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  return a.dk == 64 ? chunk_dk<64>(a, g, s) : a.dk == 128 ? chunk_dk<128>(a, g, s) : chunk_dk<256>(a, g, s);
}

}  // namespace qs
