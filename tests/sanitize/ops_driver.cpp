// CPU driver of the host code of the operators around the decode step under
// AddressSanitizer and UndefinedBehaviorSanitizer (built by
// tests/test_ops_host.py with g++, no GPU): argument checks, plans and
// workspace sizes over good and bad calls.  HIP runtime calls are host-memory
// stand-ins, the kernel launchers stubs that count.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "qstate.h"
#include "qstate_internal.hpp"
#include "qstate_ops.hpp"

static int g_device = 0;
extern "C" {
hipError_t hipGetDevice(int* d) {
  *d = g_device;
  return hipSuccess;
}
hipError_t hipMalloc(void** p, size_t n) {
  *p = std::malloc(n ? n : 1);
  return *p ? hipSuccess : hipErrorOutOfMemory;
}
hipError_t hipFree(void* p) {
  std::free(p);
  return hipSuccess;
}
hipError_t hipMemcpy(void* d, const void* s, size_t n, hipMemcpyKind) {
  std::memcpy(d, s, n);
  return hipSuccess;
}
const char* hipGetErrorString(hipError_t) { return "stand-in"; }
}

static int g_launches = 0, g_chunked = 0;
static qs::ScanSegs g_segs;
static qs::SlotArgs g_slots;
namespace qs {
hipError_t launch_step(int, int, int, int, const Args&, hipStream_t) { return hipSuccess; }
hipError_t launch_quantize(const Args&, hipStream_t) { return hipSuccess; }
hipError_t launch_dequantize(const Args&, hipStream_t) { return hipSuccess; }
const char* step_kernel_name(int, int, int, int, int) { return "stand-in"; }
hipError_t launch_conv(const ConvArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_conv_step(const ConvArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_qk(const QkArgs&, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_scan(const ScanArgs&, const ScanSegs& s, hipStream_t) { ++g_launches; g_chunked = 0; g_segs = s; return hipSuccess; }
hipError_t launch_scan_join(const ScanArgs&, const ScanSegs&, hipStream_t) { return hipSuccess; }
hipError_t launch_scan_chunk(const ScanArgs&, const ScanSegs& s, hipStream_t) { ++g_launches; g_chunked = 1; g_segs = s; return hipSuccess; }
hipError_t launch_scan_key(const ScanArgs&, const ScanSegs& s, hipStream_t) { ++g_launches; g_chunked = 2; g_segs = s; return hipSuccess; }
hipError_t launch_scan_delta(const ScanArgs&, const ScanSegs& s, hipStream_t) { ++g_launches; g_chunked = 3; g_segs = s; return hipSuccess; }
hipError_t launch_copy_slots(const SlotArgs& a, hipStream_t) { ++g_launches; g_slots = a; return hipSuccess; }
hipError_t launch_compact_slots(const SlotArgs& a, hipStream_t) { ++g_launches; g_slots = a; return hipSuccess; }
}  // namespace qs

static int g_fail = 0, g_checks = 0;
#define CHECK(c)                                                        \
  do {                                                                  \
    ++g_checks;                                                         \
    if (!(c)) {                                                         \
      std::fprintf(stderr, "check failed line %d: %s (%s)\n", __LINE__, #c, qstate_last_error()); \
      ++g_fail;                                                         \
    }                                                                   \
  } while (0)

static qstate_config config(int kind, int decay, int B, int H, int dk, int dv, int dtype) {
  qstate_config c;
  std::memset(&c, 0, sizeof(c));
  c.abi_version = QSTATE_ABI_VERSION;
  c.kind = kind;
  c.decay_mode = decay;
  c.B = B;
  c.H = H;
  c.dk = dk;
  c.dv = dv;
  c.qbits = 8;
  c.hp_dtype = QS_BF16;
  c.in_dtype = dtype;
  c.rounding = QS_ROUND_STOCHASTIC;
  c.sr_bits = 16;
  return c;
}

static char* at(uint64_t x) { return reinterpret_cast<char*>(x); }   // never read

static qstate_scan_args scan_args(const qstate_config& c, int T, int n, int G) {
  qstate_scan_args a;
  std::memset(&a, 0, sizeof(a));
  const uint64_t G1 = 1ull << 32;
  a.q = at(1 * G1);
  a.k = at(2 * G1);
  a.v = at(3 * G1);
  a.decay = (const float*)at(4 * G1);
  a.beta = (const float*)at(5 * G1);
  a.initial = (const float*)at(6 * G1);
  a.final = (float*)at(7 * G1);
  a.out = at(8 * G1);
  a.offsets = (const int32_t*)at(9 * G1);
  a.q_stride = a.k_stride = (int64_t)G * c.dk;
  a.v_stride = a.out_stride = (int64_t)c.H * c.dv;
  a.decay_stride = (int64_t)c.H * (c.decay_mode == QS_DECAY_KEY ? c.dk : 1);
  a.beta_stride = c.H;
  a.tokens = T;
  a.n = n;
  a.k_heads = G;
  return a;
}

int main() {
  char* ws = at(32ull << 32);
  const uint64_t big = 1ull << 40;
  for (int kind = 0; kind < 2; ++kind)
    for (int decay = 0; decay < 2; ++decay)
      for (int dtype : {QS_BF16, QS_FP32}) {
        const qstate_config c = config(kind, decay, 4, 8, 128, 64, dtype);
        qstate_handle* h = nullptr;
        CHECK(qstate_init(&c, &h, nullptr) == QS_OK);
        uint64_t need = 1;
        qstate_scan_args a = scan_args(c, 4096, 2, 4);
        CHECK(qstate_scan_workspace(h, &a, &need) == QS_OK);
        CHECK(qstate_scan(h, &a, ws, need, nullptr) == QS_OK);
        const bool chunked = dtype == QS_BF16 && !(kind == QS_KIND_DELTA && decay == QS_DECAY_KEY);
        CHECK((g_chunked != 0) == chunked);
        CHECK(need > 0 && (kind == QS_KIND_ADDITIVE || chunked) == (g_segs.states != nullptr));
        CHECK((g_segs.cut > 0) == (kind == QS_KIND_DELTA));
        if (need) {
          CHECK(qstate_scan(h, &a, nullptr, need, nullptr) == QS_EINVAL);
          CHECK(qstate_scan(h, &a, ws + 16, need, nullptr) == QS_EINVAL);
          CHECK(qstate_scan(h, &a, ws, need - 1, nullptr) == QS_EINVAL);
          CHECK(qstate_scan(h, &a, (void*)a.v, need, nullptr) == QS_EINVAL);
          CHECK(qstate_scan(h, &a, a.final, need, nullptr) == QS_EINVAL);
        }
        a = scan_args(c, 8, 2, 4);                    // short sequences run token by token
        CHECK(qstate_scan(h, &a, nullptr, 0, nullptr) == QS_OK && g_chunked == 0);
#define BAD(code, ...)                                           \
  do {                                                           \
    a = scan_args(c, 4096, 2, 4);                                \
    __VA_ARGS__;                                                 \
    const int before = g_launches;                               \
    CHECK(qstate_scan(h, &a, ws, big, nullptr) == (code));       \
    CHECK(g_launches == before);                                 \
  } while (0)
        BAD(QS_EINVAL, a.q = nullptr);
        BAD(QS_EINVAL, a.v = nullptr);
        BAD(QS_EINVAL, a.decay = nullptr);
        BAD(QS_EINVAL, a.out = nullptr);
        BAD(QS_EINVAL, a.final = nullptr);
        BAD(QS_EINVAL, a.offsets = nullptr);
        BAD(QS_EINVAL, a.tokens = -1);
        BAD(QS_EINVAL, a.n = -1);
        BAD(QS_EINVAL, a.k_heads = 3);
        BAD(QS_EINVAL, a.k_heads = 0);
        BAD(QS_EINVAL, a.q_stride -= 1);
        BAD(QS_EINVAL, a.v_stride = 0);
        BAD(QS_EINVAL, a.out_stride = -a.out_stride);
        BAD(QS_EINVAL, a.decay_stride -= 1);
        BAD(QS_EINVAL, a.beta_stride = 1);
        BAD(QS_EINVAL, a.q = at((1ull << 32) + 1));
        BAD(QS_EINVAL, a.final = (float*)at((7ull << 32) + 4));
        BAD(QS_EINVAL, a.initial = (float*)at((6ull << 32) + 8));
        BAD(QS_EINVAL, a.out = (void*)a.v);
        BAD(QS_EINVAL, a.out = (char*)a.q + 64);
        BAD(QS_EINVAL, a.final = (float*)((char*)a.initial + 64));
        BAD(QS_EINVAL, a.final = (float*)a.out);
        if (chunked) BAD(QS_EUNSUPPORTED, a.q = at(1000ull << 32); a.q_stride = (1 << 24) + 8);
        a = scan_args(c, 4096, 2, 4);
        a.final = (float*)a.initial;                  // in place
        a.beta = nullptr;
        CHECK(qstate_scan(h, &a, ws, big, nullptr) == QS_OK);
        a = scan_args(c, 4096, 2, 4);                 // q, k and v as slices of one tensor
        a.q_stride = a.k_stride = a.v_stride = a.v_stride + 2 * a.q_stride;
        a.k = (char*)a.v + 8 * 64 * (dtype == QS_BF16 ? 2 : 4);
        a.q = (char*)a.k + 4 * 128 * (dtype == QS_BF16 ? 2 : 4);
        CHECK(qstate_scan(h, &a, ws, big, nullptr) == QS_OK);
        a = scan_args(c, 0, 2, 4);                    // no tokens: only the states
        a.q = a.k = a.v = nullptr;
        a.out = nullptr;
        a.decay = nullptr;
        CHECK(qstate_scan(h, &a, nullptr, 0, nullptr) == QS_OK);
        a = scan_args(c, 100, 0, 4);
        const int before = g_launches;
        CHECK(qstate_scan(h, &a, nullptr, 0, nullptr) == QS_OK && g_launches == before);
        a = scan_args(c, 4096, 1, 4);
        a.offsets = nullptr;
        CHECK(qstate_scan(h, &a, ws, big, nullptr) == QS_OK);
        g_device = 1;                                 // another device is current
        CHECK(qstate_scan(h, &a, ws, big, nullptr) == QS_EINVAL);
        g_device = 0;
        // any sizes: the plan holds every segment, and the workspace is what it says
        std::mt19937 r(7 + kind * 4 + decay * 2);
        for (int i = 0; i < 500; ++i) {
          const int n = 1 + (int)(r() % 3000), T = (int)(r() % 2000000);
          a = scan_args(c, T, n, 1 << (r() % 4));
          a.out = at(1000ull << 32);
          a.v = at(2000ull << 32);
          a.k = at(3000ull << 32);
          a.decay = (const float*)at(4000ull << 32);
          a.final = (float*)at(5000ull << 32);
          a.initial = nullptr;
          CHECK(qstate_scan_workspace(h, &a, &need) == QS_OK);
          CHECK(qstate_scan(h, &a, at(6000ull << 32), need, nullptr) == QS_OK);
          {
            const int64_t seg = g_segs.seg;
            CHECK(seg > 0 && g_segs.count >= ((seg < T ? (T - 1) / seg : 0) + n));
            if (g_segs.states) {
              const uint64_t per = g_chunked == 3 ? (uint64_t)qs::kScanPrepBytes : 64ull * 128 * 4;
              CHECK((char*)g_segs.states + (uint64_t)g_segs.count * 8 * per <= at(6000ull << 32) + need);
            }
            if (g_segs.states ? g_chunked != 3 : g_segs.cut > 0)
              CHECK(g_segs.uncut != nullptr);
            if (g_segs.uncut) {                       // a word for each head of a sequence, behind all else
              const uint64_t per = g_chunked == 3 ? (uint64_t)qs::kScanPrepBytes : 64ull * 128 * 4;
              CHECK((char*)(g_segs.uncut + (int64_t)n * 8) <= at(6000ull << 32) + need);
              if (g_segs.states) CHECK((char*)g_segs.states + (uint64_t)g_segs.count * 8 * per <= (char*)g_segs.uncut);
            }
            if (g_segs.cut > 0) {                     // pieces: L and M in front of the prepared chunks
              const uint64_t pieces = (uint64_t)((T - 1) / g_segs.cut + n);
              CHECK((char*)g_segs.total + pieces * 8 * (64 + 128) * 128 * 4 <=
                    (g_segs.states ? (char*)g_segs.states : at(6000ull << 32) + need));
            }
          }
        }
        // a launch has fewer than 2^32 threads
        for (int n : {1 << 20, 1 << 21, 1 << 22}) {
          a = scan_args(c, 100, n, 1);
          a.final = (float*)at(5000ull << 32);
          a.initial = nullptr;
          const int before = g_launches;
          const qs_status s = qstate_scan(h, &a, at(6000ull << 32), 1ull << 44, nullptr);
          CHECK(s == ((int64_t)n * 8 * (64 * 128 / 1024) < (1 << 24) ? QS_OK : QS_EUNSUPPORTED));
          CHECK(g_launches - before == (s == QS_OK));
        }
        // many short sequences, of which one may be long: two parts, by length
        {
          const bool by_length = chunked || kind == QS_KIND_ADDITIVE;
          for (int T : {600, 4095, 12000}) {
            a = scan_args(c, T, 900, 4);
            a.final = (float*)at(5000ull << 32);
            a.initial = nullptr;
            CHECK(qstate_scan_workspace(h, &a, &need) == QS_OK);
            const int before = g_launches;
            CHECK(qstate_scan(h, &a, need ? at(6000ull << 32) : nullptr, need, nullptr) == QS_OK);
            const bool split = by_length && T > 600;
            CHECK(g_launches - before == (split ? 2 : 1));
            CHECK((g_chunked != 0) == (split && chunked) && (need > 0) == split);
          }
          if (chunked) {                              // rows too far apart for chunks: token by token, as in one part
            a = scan_args(c, 12000, 900, 4);
            a.final = (float*)at(5000ull << 32);
            a.initial = nullptr;
            a.q = at(1000ull << 32);
            a.q_stride = (1 << 24) + 8;
            const int before = g_launches;
            CHECK(qstate_scan(h, &a, at(6000ull << 32), big, nullptr) == QS_OK);
            CHECK(g_launches - before == 1 && g_chunked == 0);
          }
        }
        // slots
        qstate_sizes z;
        CHECK(qstate_plan(&c, &z) == QS_OK);
        qstate_tensors p{at(1ull << 32), at(2ull << 32), nullptr, nullptr, nullptr, nullptr};
        qstate_tensors o{at(3ull << 32), at(4ull << 32), nullptr, nullptr, nullptr, nullptr};
        const int32_t *src = (const int32_t*)at(5ull << 32), *dst = (const int32_t*)at(6ull << 32);
        CHECK(qstate_copy_slots(h, &p, &p, 4, 3, src, dst, nullptr, 0, nullptr) == QS_OK);
        CHECK(g_slots.nbuf == 2 && g_slots.buf[0].bytes == z.codes / 4 && g_slots.buf[1].bytes == z.scales / 4);
        CHECK(g_slots.pieces == (z.codes / 4 + 16383) / 16384 + (z.scales / 4 + 16383) / 16384);
        CHECK(qstate_copy_slots(h, &p, &o, 9, 3, src, dst, nullptr, 0, nullptr) == QS_OK);
        CHECK(qstate_copy_slots(h, &p, &p, 4, 0, nullptr, nullptr, nullptr, 0, nullptr) == QS_OK);
        CHECK(qstate_copy_slots(h, &p, &p, 4, -1, src, dst, nullptr, 0, nullptr) == QS_EINVAL);
        CHECK(qstate_copy_slots(h, &p, &p, -1, 1, src, dst, nullptr, 0, nullptr) == QS_EINVAL);
        CHECK(qstate_copy_slots(h, &p, &p, 4, 1, nullptr, dst, nullptr, 0, nullptr) == QS_EINVAL);
        CHECK(qstate_copy_slots(h, &p, nullptr, 4, 1, src, dst, nullptr, 0, nullptr) == QS_EINVAL);
        // the pool as its own source has no more slots than the pool
        {
          const int before = g_launches;
          CHECK(qstate_copy_slots(h, &p, &p, 5, 1, src, dst, nullptr, 0, nullptr) == QS_EINVAL);
          qstate_tensors again = p;
          CHECK(qstate_copy_slots(h, &p, &again, 1 << 20, 1, src, dst, nullptr, 0, nullptr) == QS_EINVAL);
          CHECK(g_launches == before);
          CHECK(qstate_copy_slots(h, &p, &p, 3, 1, src, dst, nullptr, 0, nullptr) == QS_OK && g_slots.src_slots == 3);
        }
        qstate_tensors shifted = p, mixed = o;
        shifted.codes = at((1ull << 32) + 16);
        CHECK(qstate_copy_slots(h, &p, &shifted, 4, 1, src, dst, nullptr, 0, nullptr) == QS_EINVAL);
        mixed.codes = p.codes;
        CHECK(qstate_copy_slots(h, &p, &mixed, 4, 1, src, dst, nullptr, 0, nullptr) == QS_EINVAL);
        qstate_slot_buffer e[7];
        for (auto& x : e) x = {at(7ull << 32), at(7ull << 32), 222};
        CHECK(qstate_copy_slots(h, &p, &p, 4, 1, src, dst, e, 6, nullptr) == QS_OK);
        CHECK(g_slots.nbuf == 8 && g_slots.buf[2].unit == 2 && g_slots.buf[7].first == g_slots.pieces - 1);
        CHECK(qstate_copy_slots(h, &p, &p, 4, 1, src, dst, e, 7, nullptr) == QS_EINVAL);
        CHECK(qstate_copy_slots(h, &p, &p, 4, 1, src, dst, nullptr, 1, nullptr) == QS_EINVAL);
        e[1].src = nullptr;
        CHECK(qstate_copy_slots(h, &p, &p, 4, 1, src, dst, e, 2, nullptr) == QS_EINVAL);
        e[1] = {at(8ull << 32), at(9ull << 32), 64};
        CHECK(qstate_copy_slots(h, &p, &p, 4, 1, src, dst, e, 2, nullptr) == QS_EINVAL);   // only one of two pools
        CHECK(qstate_compact_slots(h, &p, (uint8_t*)src, (int32_t*)dst, e, 2, nullptr) == QS_EINVAL);
        CHECK(qstate_compact_slots(h, &p, (uint8_t*)src, (int32_t*)dst, e, 1, nullptr) == QS_OK);
        CHECK(qstate_compact_slots(h, &p, nullptr, (int32_t*)dst, nullptr, 0, nullptr) == QS_EINVAL);
        CHECK(qstate_compact_slots(h, &p, (uint8_t*)src, (int32_t*)(at(6ull << 32) + 2), nullptr, 0, nullptr) == QS_EINVAL);
        CHECK(qstate_compact_slots(h, nullptr, (uint8_t*)src, (int32_t*)dst, nullptr, 0, nullptr) == QS_EINVAL);
        qstate_destroy(h);
      }
  {
    const qstate_config c = config(0, 0, 20000, 1, 64, 8, QS_BF16);
    qstate_handle* h = nullptr;
    CHECK(qstate_init(&c, &h, nullptr) == QS_OK);
    qstate_tensors p{at(1ull << 32), at(2ull << 32), nullptr, nullptr, nullptr, nullptr};
    CHECK(qstate_compact_slots(h, &p, (uint8_t*)at(4096), (int32_t*)at(8192), nullptr, 0, nullptr) == QS_EUNSUPPORTED);
    qstate_destroy(h);
  }
  // a launch that fails is reported
  qstate_qk k;
  std::memset(&k, 0, sizeof(k));
  k.q = at(1ull << 32);
  k.q_out = at(2ull << 32);
  k.q_stride = k.q_out_stride = 64;
  k.dtype = QS_FP32;
  k.tokens = 3;
  k.q_heads = 1;
  k.dim = 64;
  CHECK(qstate_qk_norm_rotate(&k, nullptr) == QS_EHIP);
  std::printf("%d checks, %d failed checks\n", g_checks, g_fail);
  return g_fail ? 1 : 0;
}
