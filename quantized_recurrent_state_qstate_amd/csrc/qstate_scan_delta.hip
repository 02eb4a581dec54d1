// Scan of packed bf16 prompts by the delta rule with one decay a head, 64
// tokens at a time on the matrix cores.
//
// With c_i the sum of log2 decays from a chunk's first token to token i and S
// the state before the chunk, u_i = beta_i (v_i - 2^{c_i} S k_i
// - sum_{j<i} 2^{c_i - c_j} (k_j.k_i) u_j) is a unit lower triangular system:
//   (I + A) U = R,  A_ij = beta_i 2^{c_i - c_j} k_j.k_i (j < i),
//   R_i = beta_i (v_i - 2^{c_i} S k_i),  so U = T R with T = (I + A)^-1,
//   o_i = 2^{c_i} S q_i + sum_{j<=i} P_ij u_j,  P_ij = 2^{c_i - c_j} k_j.q_i,
//   S'  = 2^{c_last} S + sum_j 2^{c_last - c_j} u_j k_j^T.
// T and P do not depend on the state.  A first launch makes them for all
// chunks at once, in the layout in which the second one's lanes take them;
// the second goes through a sequence's chunks one after the other.  That
// chain bounds a long prompt: with T at hand a chunk is four products.
//
// Precision: q, k and v are bf16, so a product with one of them is exact when
// the other operand, S or u, is cut into three bf16 pieces, which hold its 24
// bits.  T is fp32, made by fp32 matrix instructions: its diagonal blocks of 16
// by substitution, the others from them.  T R and P u are products of three
// pieces by three without the last three, at most 2^-27 of the whole each.
// All sums are fp32, c's fp64; a decay of zero counts as 2^-10000; an output is
// rounded to bf16 once.
//
// Where few heads leave compute units idle, long sequences go in pieces at once:
// a pass for what each piece does to the state before it, a short chain over
// the pieces, a pass for the outputs.  One sequence of 7868 tokens, 32 heads of
// 128 x 128, in 3 pieces: 350 us; under a trace, which makes them longer (422 in
// all), 56 for the first launch, 127, 13 and 226 for the others, 5.5 us a chunk at the
// outputs, of which 216 matrix instructions of a wave (16 cycles each) are 26% and
// 1190 vector instructions (4 cycles; most split operands into pieces) 36%, one
// after the other in the one wave a SIMD has.  8192 tokens 375 us, in one piece
// 610; of 2 heads, in 16 pieces, 112, in one 560.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "qstate_scan_tiles.hpp"

namespace qs {
namespace {

// What the first launch leaves for a chunk of a head.
constexpr int kGate = 256;                    // floats: 2^{c_i}, 2^{c_last - c_i}, beta_i, 2^{c_last}, oddness
constexpr int kTile = 64 * 8 / 2;             // floats of a 16 x 32 tile in bf16, 8 elements a lane
constexpr int kTri = 6 * 3 * kTile;           // T's lower tiles in three pieces
constexpr int kPairs = 6 * 2 * kTile;         // P's lower tiles in fp32
constexpr int kPrepFloats = kGate + kTri + kPairs;
static_assert(kPrepFloats * 4 == kScanPrepBytes, "workspace a chunk and head");

// The lower 16 x 32 tiles of a 64 x 64 matrix: rows 16 i .., columns 32 c ...
// A lane (m, q4) has row m's columns 4 q4 .. + 3 and 16 + 4 q4 .. + 3: the
// order in which accumulators of 16 x 16 tiles are the other operand.
__device__ __forceinline__ int piece(int i, int c) { return i < 2 ? i : 2 * i - 2 + c; }

template <int DK, bool VEC>
__global__ __launch_bounds__(256) void k_delta_prep(const ScanArgs a, float* prep, int32_t* uncut) {
  constexpr int kKS = DK / 32, kKR = DK + 8, kAR = kL + 4, kKP = kL * DK / 8 / 256;
  __shared__ __attribute__((aligned(16))) uint16_t sk[kL * kKR], sq[kL * kKR];
  __shared__ __attribute__((aligned(16))) float sa[kL * kAR];   // minus A; then T
  __shared__ double sc[kL];
  __shared__ float sb[kL], sodd;
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, q4 = lane >> 4;
  const int s = (int)(blockIdx.x / (uint32_t)a.H), h = (int)(blockIdx.x % (uint32_t)a.H);
  const int kh = h / (a.H / a.G);
  const Segment sg = find_segment(a, kL, s);
  if (sg.none || sg.t1 <= sg.t0) return;
  const int n = sg.t1 - sg.t0;
  float* out = prep + (int64_t)blockIdx.x * kPrepFloats;
  const Tile<VEC> tk(a.k, (int64_t)sg.t0 * a.ks + (int64_t)kh * DK, a.ks, n, DK);
  const Tile<VEC> tq(a.q, (int64_t)sg.t0 * a.qs + (int64_t)kh * DK, a.qs, n, DK);
  if (tid == 0) sodd = 0.0f;
  if (uncut && sg.first && tid == 0) uncut[(int64_t)sg.seq * a.H + h] = 0;   // until the join finds otherwise
  __syncthreads();
  H2 most = (H2){0, 0};
#pragma unroll
  for (int i = 0; i < kKP; ++i) {
    const int p = i * 256 + tid, r = p / (DK / 8), c = p % (DK / 8) * 8;
    const U4 k = tk.load(r, c);
    most = largest(most, k);
    *(U4*)&sk[r * kKR + c] = k;
    *(U4*)&sq[r * kKR + c] = tq.load(r, c);
  }
  if (odd(most)) sodd = 1.0f;
  if (wave == 0) {
    float d = 1.0f, b = 0.0f;
    if (lane < n) {
      d = a.decay[(int64_t)(sg.t0 + lane) * a.ds + h];
      b = a.beta ? a.beta[(int64_t)(sg.t0 + lane) * a.bs + h] : 1.0f;
    }
    const double c = wave_sums(d == 0.0f ? -10000.0 : (double)log2f(d));
    const double all = __shfl(c, 63);
    sc[lane] = c;
    sb[lane] = b;
    const float e = __builtin_amdgcn_exp2f((float)c), w = __builtin_amdgcn_exp2f((float)(all - c));
    out[lane] = e;
    out[64 + lane] = w;
    out[128 + lane] = b;
    if (!(fabsf(d) < INFINITY && fabsf(b) < INFINITY && e < 0x1p100f && w < 0x1p100f)) sodd = 1.0f;
    if (lane == 0) out[192] = __builtin_amdgcn_exp2f((float)all);
  }
  __syncthreads();
  if (tid == 0) out[193] = sodd;            // k or a gate is not finite, or the decays grow out of fp32
  // ---- P and A, transposed tiles: a lane gets 4 j of one i; wave i takes rows 16 i ..
  {
    const int i = 16 * wave + m;
    const double ci = sc[i];
    const float bi = sb[i];
    for (int jp = 0; jp <= wave; jp += 2) {
      F4 p[2] = {(F4){0, 0, 0, 0}, (F4){0, 0, 0, 0}}, kk[2] = {(F4){0, 0, 0, 0}, (F4){0, 0, 0, 0}};
#pragma unroll
      for (int c = 0; c < kKS; ++c) {
        const BF8 qi = *(const BF8*)&sq[i * kKR + 32 * c + 8 * q4], ki = *(const BF8*)&sk[i * kKR + 32 * c + 8 * q4];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const BF8 kj = *(const BF8*)&sk[(16 * (jp + y) + m) * kKR + 32 * c + 8 * q4];
          p[y] = mfma(kj, qi, p[y]);
          kk[y] = mfma(kj, ki, kk[y]);
        }
      }
      F4* to = (F4*)(out + kGate + kTri) + piece(wave, jp >> 1) * 128 + lane;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int j = 16 * (jp + y) + 4 * q4;
        F4 f, neg;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = __builtin_amdgcn_exp2f((float)(ci - sc[j + r]));
          const float w = p[y][r] * e, z = -(bi * e * kk[y][r]);
          f[r] = j + r <= i ? w : 0.0f;
          neg[r] = j + r < i ? z : 0.0f;
        }
        *(F4*)&sa[i * kAR + j] = neg;
        to[64 * y] = f;                       // columns j .. j + 3
      }
    }
  }
  __syncthreads();
  // ---- the diagonal blocks of I + A inverted, a column each lane
  if (wave == 0) {
    float x[16];
    float* blk = &sa[(16 * q4) * kAR + 16 * q4];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float y = i == m ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < i; ++j) y = fmaf(blk[i * kAR + j], x[j], y);
      x[i] = y;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) blk[i * kAR + m] = x[i];
  }
  __syncthreads();
  // ---- T's column of blocks `wave`: T_ba = T_bb sum_{a<=x<b} (-A_bx) T_xa
  F4 X[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) X[b] = (F4){0, 0, 0, 0};
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (b == wave) {
#pragma unroll
      for (int r = 0; r < 4; ++r) X[b][r] = sa[(16 * b + 4 * q4 + r) * kAR + 16 * b + m];
    } else if (b > wave) {
      F4 acc = (F4){0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < b; ++x) {            // blocks before the column are zero
        const F4 ab = *(const F4*)&sa[(16 * b + m) * kAR + 16 * x + 4 * q4];
        if (x >= wave)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc = mfma1(ab[r], X[x][r], acc);
      }
      const F4 tb = *(const F4*)&sa[(16 * b + m) * kAR + 16 * b + 4 * q4];
#pragma unroll
      for (int r = 0; r < 4; ++r) X[b] = mfma1(tb[r], acc[r], X[b]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (b > wave)
#pragma unroll
      for (int r = 0; r < 4; ++r) sa[(16 * b + 4 * q4 + r) * kAR + 16 * wave + m] = X[b][r];
  __syncthreads();
  for (int c = 0; c <= wave >> 1; ++c) {
    const F4 x = *(const F4*)&sa[(16 * wave + m) * kAR + 32 * c + 4 * q4];
    const F4 y = *(const F4*)&sa[(16 * wave + m) * kAR + 32 * c + 16 + 4 * q4];
    const float f[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    BF8 t[3];
    split(f, t);
#pragma unroll
    for (int p = 0; p < 3; ++p) *(BF8*)(out + kGate + (3 * piece(wave, c) + p) * kTile + lane * 4) = t[p];
  }
}

// A chunk of a workgroup's columns in LDS.
template <int DK, int DV>
struct Chunk {
  uint16_t k[kL * DK], q[kL * DK], v[kL * DV];   // rows as at<>() lays them
  float prep[kPrepFloats];
};

// A sequence's chunks in order; a workgroup holds 16 WAVES value columns of a
// head, each wave 16 in accumulators [dk][v] (rows dealt so that a lane holds 8
// channels in a row, the second operand of S k and S q as it is).  While a
// chunk is worked on, the next one is on its way into the other buffer, from
// memory to LDS directly; a chunk costs one barrier.
//
// Where few heads leave compute units idle, long sequences are cut into pieces.
// A piece maps the state before it to S M + L.  The !OUT pass makes L (state
// rows, from zero or the first piece's initial state) and M (further dk rows:
// values of zero, from the identity) into `carry`, k_delta_join goes from
// piece to piece, and the OUT pass makes the outputs of all pieces at once.
template <int DK, int WAVES, int VEC, bool OUT>
__global__ __launch_bounds__(64 * WAVES, 1) void k_delta_scan(const ScanArgs a, const ScanSegs g, int vchunks) {
  const float* prep = g.states;
  float* carry = g.total;
  constexpr int kDV = 16 * WAVES, kKS = DK / 32;
  using Buf = Chunk<DK, kDV>;
  constexpr bool kTwo = 2 * sizeof(Buf) + WAVES * kL * 32 <= 160 * 1024;   // room for two buffers
  __shared__ __attribute__((aligned(1024))) Buf buf0;
  __shared__ __attribute__((aligned(1024))) typename std::conditional<kTwo, Buf, int>::type buf1;
  __shared__ __attribute__((aligned(16))) uint16_t so[WAVES][kL * 16];     // a wave's outputs
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, q4 = lane >> 4;
  const int per = a.H * (OUT ? vchunks : vchunks + DK / kDV);
  const int hv = (int)(blockIdx.x % (uint32_t)per), h = hv % a.H, kh = h / (a.H / a.G);
  const int part = (int)(blockIdx.x / (uint32_t)per);
  Piece piece_of = find_piece(a, g.cut, part);
  const bool matrix = !OUT && hv / a.H >= vchunks;   // columns of M
  const int v0 = matrix ? 0 : hv / a.H * kDV, m0 = matrix ? (hv / a.H - vchunks) * kDV : 0;
  if (OUT && !piece_of.none) outputs_of(piece_of, a, g, h);
  if (piece_of.none || (!OUT && (piece_of.last || (matrix && piece_of.first)))) return;
  const int seq = piece_of.seq, start = piece_of.t0, end = piece_of.t1;
  const int64_t head = (int64_t)h * a.dv, st = (int64_t)seq * a.H * a.dv;
  const int col = wave * 16 + m, v = v0 + col;
  const float skip = a.skip ? a.skip[h] : 0.0f;
  // this lane's row of the states given and kept, channels 8 q4 .. of every 32
  const int64_t at_state = (st + head + v) * DK + 8 * q4;
  const int64_t at_carry =
      (((int64_t)part * a.H + h) * (a.dv + DK) + (matrix ? a.dv + m0 + col : v)) * DK + 8 * q4;
  const bool real = matrix || v < a.dv;
  const float* from = OUT && !(piece_of.first && piece_of.last) ? carry + at_carry
                      : piece_of.first && a.initial             ? a.initial + at_state
                                                                : nullptr;
  float* to = !OUT ? carry + at_carry : piece_of.last ? a.final + at_state : nullptr;

  F4 S[2 * kKS];
#pragma unroll
  for (int t = 0; t < 2 * kKS; ++t) {
    S[t] = (F4){0, 0, 0, 0};
    if (matrix)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[t][r] = 32 * (t >> 1) + 8 * q4 + 4 * (t & 1) + r == m0 + col ? 1.0f : 0.0f;
    else if (from && real) S[t] = *(const F4*)(from + 32 * (t >> 1) + 4 * (t & 1));
  }

  // The next chunk's pieces of 1 KB, `kPieces` for each wave, brought one by one.
  constexpr int kK = kL * DK / 512 / WAVES, kV = kL * kDV / 512 / WAVES, kQ = OUT ? kK : 0;
  constexpr int kUsed = OUT ? kPrepFloats : kGate + kTri, kP = (kUsed / 256 + WAVES - 1) / WAVES;
  constexpr int kPieces = kK + kQ + kV + kP;
  auto bringing = [&](Buf& b, int t, int t1) {   // piece i of the chunk from t to t1 into b
    const int rows = t1 - t;
    return [&b, wave, lane, tk = Tile<(VEC > 0)>(a.k, (int64_t)t * a.ks + (int64_t)kh * DK, a.ks, rows, DK),
            tq = Tile<(VEC > 0)>(a.q, (int64_t)t * a.qs + (int64_t)kh * DK, a.qs, rows, DK),
            tv = Tile<VEC == 2>(a.v, (int64_t)t * a.vs + head + v0, a.vs, matrix ? 0 : rows, min(kDV, a.dv - v0)),
            tp = Tile<true>(prep, 2 * ((int64_t)(t / kL + seq) * a.H + h) * kPrepFloats, 0, min(rows, 1), kPrepFloats * 2)](
               int i) {
      if (i < kK) tk.template bring<DK>(b.k, (i * WAVES + wave) * 512, lane);
      else if (i < kK + kQ) tq.template bring<DK>(b.q, ((i - kK) * WAVES + wave) * 512, lane);
      else if (i < kK + kQ + kV) tv.template bring<kDV>(b.v, ((i - kK - kQ) * WAVES + wave) * 512, lane);
      else if (i < kPieces) {
        const int e = (i - kK - kQ - kV) * WAVES + wave;
        if (e < kUsed / 256) to_lds(tp.rsrc, (uint16_t*)b.prep + e * 512, e * 1024 + lane * 16);
      }
    };
  };

  bool lost = false;                         // this lane's column has a state that is not finite any more
  int done_t = 0, done_n = 0;                // the chunk whose outputs wait in `so`
  auto put_out = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 32 * i + (lane >> 1), c = 8 * (lane & 1);
      if (r < done_n) {
        const U4 y = *(const U4*)&so[wave][r * 16 + c];
        uint16_t* o = (uint16_t*)a.out + (int64_t)(done_t + r) * a.os + head + v0 + wave * 16 + c;
        if constexpr (VEC == 2) {
          if (v0 + wave * 16 + c < a.dv) *(U4*)o = y;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (v0 + wave * 16 + c + j < a.dv) o[j] = (uint16_t)(y[j >> 1] >> (16 * (j & 1)));
        }
      }
    }
  };

  // A chunk; the next one's pieces are asked for on the way, a few at each of
  // kPoints places: asked for at once they would hold the wave up.
  constexpr int kPoints = kKS + 6, kEach = (kPieces + kPoints - 1) / kPoints;
  auto work = [&](Buf& b, auto& bring, int t, int n) {
    auto point = [&](int i) {
      if constexpr (kTwo)
#pragma unroll
        for (int j = 0; j < kEach; ++j) bring(i * kEach + j);
    };
    // ---- v of the wave's columns; a value that is not finite
    BF4 x[4];
    H2 most = (H2){0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = read_tr(&b.v[at<kDV>(16 * i + 4 * q4 + (m >> 2), wave * 16 + 4 * (m & 3))]);
      const uint2 u = __builtin_bit_cast(uint2, x[i]);
      most = largest(most, (U4){u.x, u.y, 0, 0});
    }
    const bool odd_in = b.prep[193] != 0.0f || __ballot(odd(most)) != 0;
    // ---- products with the state
    F4 O[4], R[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) O[i] = R[i] = (F4){0, 0, 0, 0};
    BF8 qf[2][4], kf[2][4];
    auto rows = [&](int c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kf[c & 1][i] = *(const BF8*)&b.k[at<DK>(16 * i + m, 32 * c + 8 * q4)];
        if constexpr (OUT) qf[c & 1][i] = *(const BF8*)&b.q[at<DK>(16 * i + m, 32 * c + 8 * q4)];
      }
    };
    BF8 sp[2][3];
    auto pieces = [&](int c) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = S[2 * c + (j >> 2)][j & 3];
      split(f, sp[c & 1]);
    };
    rows(0);
    pieces(0);
#pragma unroll
    for (int c = 0; c < kKS; ++c) {
      if (c + 1 < kKS) rows(c + 1);
      point(c);
      // products on one accumulator are kept apart: each takes several issue slots
#pragma unroll
      for (int y = 0; y < 3; ++y)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          R[i] = mfma(kf[c & 1][i], sp[c & 1][y], R[i]);
          if constexpr (OUT) O[i] = mfma(qf[c & 1][i], sp[c & 1][y], O[i]);
        }
      if (c + 1 < kKS) pieces(c + 1);
    }
    // ---- U = T R
    F4 U[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) U[i] = (F4){0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      BF8 T[4][3];
#pragma unroll
      for (int i = 2 * c; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < 3; ++p) T[i][p] = *(const BF8*)&b.prep[kGate + (3 * piece(i, c) + p) * kTile + lane * 4];
      float f[8];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = 2 * c + y;
        const F4 e = *(const F4*)&b.prep[16 * i + 4 * q4], bt = *(const F4*)&b.prep[128 + 16 * i + 4 * q4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f[4 * y + r] = bt[r] * fmaf(-e[r], R[i][r], (float)x[i][r]);
          O[i][r] *= e[r];
          if (a.skip) O[i][r] = fmaf(skip, (float)x[i][r], O[i][r]);
        }
      }
      BF8 rp[3];
      split(f, rp);
      point(kKS + c);
#pragma unroll
      for (int p = 0; p < 6; ++p)
#pragma unroll
        for (int i = 2 * c; i < 4; ++i) U[i] = mfma(T[i][first_of(p)], rp[second_of(p)], U[i]);
    }
    // ---- outputs: P u on top
    BF8 wu[2][3], kt[2][4];
    auto columns = [&](int z) {              // k transposed: tokens 32 (z & 1) .., tiles 4 (z >> 1) ..
      const int c = z & 1, t4 = 4 * (z >> 1);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint16_t* p =
            &b.k[at<DK>(32 * c + 4 * q4 + (m >> 2), 32 * ((t4 + y) >> 1) + 8 * (m & 3) + 4 * (y & 1))];
        kt[z & 1][y] = join(read_tr(p), read_tr(p + 16 * DK));
      }
    };
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      BF8 P[4][3];
#pragma unroll
      for (int i = 2 * c; OUT && i < 4; ++i) {
        const float* from = &b.prep[kGate + kTri + 2 * piece(i, c) * kTile + lane * 4];
        const F4 lo = *(const F4*)from, hi = *(const F4*)(from + 256);
        const float p[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        split(p, P[i]);
      }
      if (c == 1) columns(0);
      float f[8], g[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const F4 w = *(const F4*)&b.prep[64 + 32 * c + 16 * j + 4 * q4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f[4 * j + r] = U[2 * c + j][r];
          g[4 * j + r] = U[2 * c + j][r] * w[r];
        }
      }
      BF8 ub[3];
      split(f, ub);
      point(kKS + 2 + c);
#pragma unroll
      for (int y = 0; y < 6; ++y)
#pragma unroll
        for (int i = 2 * c; OUT && i < 4; ++i) O[i] = mfma(P[i][first_of(y)], ub[second_of(y)], O[i]);
      split(g, wu[c]);
    }
    // ---- A chunk with a value that is not finite, or nearly so, is made again token
    // by token: a zero in T or P times it would reach earlier tokens, and products may
    // leave fp32 where the recurrence does not.  If it is the outputs alone (a query),
    // the state is taken back from its place in memory.
    uint32_t top = 0, otop = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      top = highest(top, U[i]);
      if constexpr (OUT) otop = highest(otop, O[i]);
    }
    const bool anew = odd_in || __ballot(top >= kHuge && !lost), again = anew || __ballot(otop >= kHuge && !lost);
    if (again) {
      float* kept = OUT && piece_of.last ? a.final + at_state : carry + at_carry;
      if (!anew && real)
#pragma unroll
        for (int y = 0; y < 2 * kKS; ++y) *(F4*)(kept + 32 * (y >> 1) + 4 * (y & 1)) = S[y];
      by_token<DK, true>(
          a, t, n, h, [&](int i, int c) { return *(const BF8*)&b.k[at<DK>(i, c)]; },
          [&](int i, int c) { return *(const BF8*)&(OUT ? b.q : b.k)[at<DK>(i, c)]; },
          [&](int i) { return __uint_as_float((uint32_t)b.v[at<kDV>(i, col)] << 16); },
          [&](int i, float o) {
            const __bf16 y = (__bf16)o;
            so[wave][i * 16 + m] = __builtin_bit_cast(uint16_t, y);
          },
          S);
      lost = spoiled(S);
      if (anew) {
        point(kKS + 4);
        point(kKS + 5);
        return;
      }
      if (real)
#pragma unroll
        for (int y = 0; y < 2 * kKS; ++y) S[y] = *(const F4*)(kept + 32 * (y >> 1) + 4 * (y & 1));
    }
    // ---- the state
    const float eall = b.prep[192];
#pragma unroll
    for (int z = 0; z < kKS; ++z) {
      const int c = z & 1, t4 = 4 * (z >> 1);
      if (z + 1 < kKS) columns(z + 1);
      if (c == 0)
#pragma unroll
        for (int y = t4; y < t4 + 4; ++y)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[y][r] *= eall;
      if (z < 2) point(kKS + 4 + z);
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int y = 0; y < 4; ++y) S[t4 + y] = mfma(kt[z & 1][y], wu[c][p], S[t4 + y]);
      if (OUT && z < 2 && !again)            // the outputs, behind the products that made them
#pragma unroll
        for (int i = 2 * z; i < 2 * z + 2; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const __bf16 y = (__bf16)O[i][r];
            so[wave][(16 * i + 4 * q4 + r) * 16 + m] = __builtin_bit_cast(uint16_t, y);
          }
    }
  };

  int t = start;
  auto step = [&](auto& b, auto& other) {
    const int next = min((t / kL + 1) * kL, end);
    __builtin_amdgcn_s_waitcnt(0x0F70);      // vmcnt 0: what this wave brings is in LDS
    __syncthreads();                         // this chunk is in LDS, and the one before has been read
    // behind the last chunk this is an empty one: the other buffer gets zeros
    const auto bring = bringing(other, next, min(next + kL, end));
    if constexpr (OUT) put_out();
    work(b, bring, t, next - t);
    done_t = t;
    done_n = next - t;
    if constexpr (!kTwo) {
      __syncthreads();
#pragma unroll
        for (int i = 0; i < kPieces; ++i) bring(i);
    }
    t = next;
  };
  if (start < end) {
    const auto bring = bringing(buf0, start, min((start / kL + 1) * kL, end));
#pragma unroll
    for (int i = 0; i < kPieces; ++i) bring(i);
  }
  while (t < end) {
    if constexpr (kTwo) {
      step(buf0, buf1);
      if (t < end) step(buf1, buf0);
    } else {
      step(buf0, buf0);
    }
  }
  if constexpr (OUT) put_out();
  if (to && real)
#pragma unroll
    for (int y = 0; y < 2 * kKS; ++y) *(F4*)(to + 32 * (y >> 1) + 4 * (y & 1)) = S[y];
}

// From piece to piece of a sequence that is cut: the place of a piece's L takes
// the state before it.  A workgroup has kJoinRows value rows of a head; its
// groups of dk threads share the sum over S M's inner channel.  A piece waits
// for the one before it, so its M and L are asked for one piece ahead: 16
// pieces of 2 heads of 128 x 128 take 35 us (87 without, by 16 rows).
constexpr int kJoinRows = 8;
template <int DK>
__global__ __launch_bounds__(512) void k_delta_join(const ScanArgs a, const ScanSegs g, int rchunks) {
  const int cut = g.cut;
  float* carry = g.total;
  constexpr int kGroups = 512 / DK, kJ = DK / kGroups, kE = kJoinRows * DK / 512;
  __shared__ __attribute__((aligned(16))) float ss[kJoinRows][DK], sums[kGroups][kJoinRows * DK];
  const int tid = (int)threadIdx.x;
  const int per = a.H * rchunks;
  const int seq = (int)(blockIdx.x / (uint32_t)per), hr = (int)(blockIdx.x % (uint32_t)per);
  const int h = hr / rchunks, r0 = hr % rchunks * kJoinRows;
  const int start = a.offsets ? min(max(a.offsets[seq], 0), a.T) : 0;
  const int end = a.offsets ? min(max(a.offsets[seq + 1], start), a.T) : a.T;
  if (!long_enough(start, end, cut) || end - start < a.least || end - start > a.most) return;
  const int c0 = start / cut, c1 = (end - 1) / cut;
  auto piece_at = [&](int c) { return carry + ((int64_t)(c == c0 ? seq : a.n + c - 1) * a.H + h) * (a.dv + DK) * DK; };
  // this thread's elements of the rows, tid + 512 e, and its part of M: a channel, kJ rows
  const int ch = tid % DK, j0 = tid / DK * kJ;
  const int rows = min(kJoinRows, a.dv - r0) * DK;   // elements there are
  float S[kE], L[kE], w[kJ];
  auto ask = [&](int c) {
    typedef const __attribute__((address_space(1))) float* G;
    G p = (G)piece_at(c);
    asm("" : "+s"(p));                      // one base, or each load keeps an address of its own from piece to piece
    const G M = p + (int64_t)a.dv * DK;
#pragma unroll
    for (int e = 0; e < kE; ++e) L[e] = tid + 512 * e < rows ? p[(int64_t)r0 * DK + tid + 512 * e] : 0.0f;
#pragma unroll
    for (int j = 0; j < kJ; ++j) w[j] = (M + j * DK)[(uint32_t)(j0 * DK + ch)];
  };
  auto keep = [&](int c, int e, float x) {
    if (tid + 512 * e < rows) piece_at(c)[(int64_t)r0 * DK + tid + 512 * e] = x;
  };
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const bool in = tid + 512 * e < rows;
    const int64_t at = (((int64_t)seq * a.H + h) * a.dv + r0) * DK + tid + 512 * e;
    S[e] = in ? piece_at(c0)[(int64_t)r0 * DK + tid + 512 * e] : 0.0f;   // began with the initial state
    keep(c0, e, a.initial && in ? a.initial[at] : 0.0f);
  }
  bool numbers = true;
  ask(c0 + 1);
  for (int c = c0 + 1; c < c1; ++c) {
    float next[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      next[e] = L[e];
      keep(c, e, S[e]);
      (&ss[0][0])[tid + 512 * e] = S[e];
    }
    __syncthreads();
    float acc[kJoinRows];
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) acc[r] = 0.0f;
#pragma unroll
    for (int j = 0; j < kJ; j += 4) {
#pragma unroll
      for (int r = 0; r < kJoinRows; ++r) {
        const F4 x = *(const F4*)&ss[r][j0 + j];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r] = fmaf(x[e], w[j + e], acc[r]);
      }
      // or all rows are read first, into more registers than there are
#pragma unroll
      for (int r = 0; r < kJoinRows; ++r) asm volatile("" : "+v"(acc[r]) : : "memory");
    }
    float zero = 0.0f;                      // or NaN
#pragma unroll
    for (int j = 0; j < kJ; ++j) zero = fmaf(w[j], 0.0f, zero);
    numbers &= zero == 0.0f;
    ask(min(c + 1, c1 - 1));
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) sums[tid / DK][r * DK + ch] = acc[r];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kE; ++e) {
#pragma unroll
      for (int i = 0; i < kGroups; ++i) next[e] += sums[i][tid + 512 * e];
      S[e] = next[e];
    }
  }
#pragma unroll
  for (int e = 0; e < kE; ++e) keep(c1, e, S[e]);
  if (!numbers) g.uncut[(int64_t)seq * a.H + h] = 1;
}

template <int DK>
hipError_t join(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  const int rchunks = (a.dv + kJoinRows - 1) / kJoinRows;
  k_delta_join<DK><<<dim3((uint32_t)(a.n * a.H * rchunks)), 512, 0, s>>>(a, g, rchunks);
  return hipGetLastError();
}

template <int DK, int VEC>
hipError_t delta(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  // 64 columns a workgroup: with 32, twice as many workgroups bring the same
  // keys (measured with outputs of two pieces, in one piece a sequence: one of 7868
  // tokens, 32 heads of 128 x 128: 493 against 506 us in all; sixteen of 256: 107, 172).
  constexpr int WAVES = 4;
  const int vchunks = (a.dv + 16 * WAVES - 1) / (16 * WAVES);
  k_delta_prep<DK, (VEC > 0)><<<dim3((uint32_t)(g.count * a.H)), 256, 0, s>>>(a, g.states, g.uncut);
  const int pieces = a.n + (g.cut > 0 ? (a.T - 1) / g.cut : 0);
  if (g.cut > 0) {
    k_delta_scan<DK, WAVES, VEC, false><<<dim3((uint32_t)(pieces * a.H * (vchunks + DK / (16 * WAVES)))), 64 * WAVES, 0, s>>>(
        a, g, vchunks);
    const hipError_t e = join<DK>(a, g, s);
    if (e != hipSuccess) return e;
  }
  k_delta_scan<DK, WAVES, VEC, true><<<dim3((uint32_t)(pieces * a.H * vchunks)), 64 * WAVES, 0, s>>>(a, g, vchunks);
  return hipGetLastError();
}

template <int DK>
hipError_t delta_dk(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  return a.vec == 2 ? delta<DK, 2>(a, g, s) : a.vec ? delta<DK, 1>(a, g, s) : delta<DK, 0>(a, g, s);
}

}  // namespace

hipError_t launch_delta_join(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  return a.dk == 64 ? join<64>(a, g, s) : a.dk == 128 ? join<128>(a, g, s) : join<256>(a, g, s);
}

hipError_t launch_scan_delta(const ScanArgs& a, const ScanSegs& g, hipStream_t s) {
  return a.dk == 64 ? delta_dk<64>(a, g, s) : a.dk == 128 ? delta_dk<128>(a, g, s) : delta_dk<256>(a, g, s);
}

}  // namespace qs
