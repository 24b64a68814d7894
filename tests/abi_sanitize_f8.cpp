// Host-side checks of dropout's call and the six of the linear layer in 8-bit
// floating point under AddressSanitizer and UndefinedBehaviorSanitizer (built
// host-only by test_sanitize_f8.py; no kernel is launched): refusals, the plans
// and workspace arithmetic up to the largest sizes, and plausible arguments,
// which stop at the device check where there is no GPU.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <initializer_list>

#include "sg.h"

// No kernel is registered: the host-only objects hold none.
extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* handle;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
}

static int failures = 0;

static void expect(sg_status got, sg_status want, const char* what) {
  const char* msg = sg_last_error_message();
  const bool no_device = want == SG_ERR_HIP && (got == SG_ERR_HIP || got == SG_ERR_UNSUPPORTED) && msg && strstr(msg, "device");
  if (!(got == want || no_device) || (got != SG_OK && (msg == nullptr || msg[0] == '\0'))) {
    fprintf(stderr, "FAIL %s: status %d (want %d), message '%s'\n", what, got, want, msg ? msg : "(null)");
    ++failures;
  }
}

template <typename T>
static T* at(uintptr_t a) {  // device-looking, never dereferenced on the host
  return reinterpret_cast<T*>(a);
}
static int64_t up(int64_t v, int64_t to) { return v < INT64_MAX - to ? (v + to - 1) / to * to : INT64_MAX - INT64_MAX % to; }

int main() {
  const int64_t top = ((int64_t)1 << 31) - 1, far = (int64_t)1 << 23, wide = (int64_t)1 << 31;
  const int64_t ms[] = {-1, 0, 1, 33, 64, 1000, 4096, 11008, 1 << 20, (1 << 20) + 1};
  const int64_t ns[] = {-1, 0, 1, 127, 128, 1000, 4096, 28672, 65536, 65537, 1 << 20, INT64_MAX};
  const int64_t ts[] = {INT64_MIN, -1, 0, 1, 16, 64, 512, 70000, far, far + 1, 34000000, top, top + 1, INT64_MAX};
  const int32_t ops[] = {SG_OP_LINEAR_F8, SG_OP_F8_GRAD_INPUT, SG_OP_F8_GRAD_WEIGHT};
  for (int32_t op : ops)
    for (int64_t m : ms)
      for (int64_t n : ns)
        for (int64_t T : ts) {
          const size_t b = sg_workspace_bytes(op, m, n, T, 0);
          const bool ok = m >= 1 && m <= 1 << 20 && n >= 1 && n <= 65536 && T >= 0 && T <= top;
          if ((!ok || T == 0) && b != 0) ++failures, fprintf(stderr, "FAIL workspace of refused sizes\n");
          if (b % 256 != 0) ++failures, fprintf(stderr, "FAIL workspace alignment\n");
        }

  uint8_t *q = at<uint8_t>(0x10000), *s = at<uint8_t>(0x20000), *w = at<uint8_t>(0x30000), *v = at<uint8_t>(0x40000);
  void *x = at<void>(0x50000), *ws = at<void>(0x100000);
  const size_t big = (size_t)1 << 60;
  const sg_drop drop = {0.3, UINT64_MAX, UINT64_MAX, nullptr};

  for (int64_t m : ms)
    for (int64_t n : ns)
      for (int64_t T : ts) {
        const bool t_ok = T >= 0 && T <= top, m_ok = m >= 1 && m <= 1 << 20;
        auto want = [](bool ok) { return ok ? SG_ERR_HIP : SG_ERR_INVALID_ARGUMENT; };
        const bool product = m_ok && n >= 1 && n <= 65536 && t_ok, rows = n >= 1 && n <= 1 << 20 && t_ok;
        expect(sg_dropout(x, 1 << 20, x, SG_BF16, 1 << 20, x, 1 << 20, T, n, &drop, nullptr), want(rows), "dropout");
        expect(sg_quantize_f8(q, far, s, wide, nullptr, 0, nullptr, 0, SG_E5M2, x, SG_F32, T, n, 1 << 20, &drop, nullptr),
               want(rows), "quantize");
        expect(sg_quantize_f8(q, far, s, wide, w, far, v, wide, SG_E4M3, x, SG_BF16, T, n, 1 << 20, nullptr, nullptr),
               want(rows && T <= far), "quantize both");
        expect(sg_dequantize_f8(x, SG_F32, far, q, far, s, wide, SG_E4M3, T, n, nullptr),
               (T == 0 || n == 0) && t_ok && n >= 0 && n <= far ? SG_ERR_HIP : want(t_ok && n >= 0 && n <= far), "read back");
        expect(sg_pack_f8(q, far, s, wide, w, far, v, wide, x, SG_BF16, m, n, 65536, nullptr), want(m_ok && n >= 1 && n <= 65536), "pack");
        expect(sg_linear_f8(x, SG_BF16, 1 << 20, q, far, s, wide, SG_E4M3, T, w, far, v, wide, m, n, ws, big, nullptr),
               want(product), "linear");
        expect(sg_linear_f8_grad_input(x, SG_F32, 65536, q, far, s, wide, SG_E5M2, T, w, far, v, wide, m, n, &drop, ws, big, nullptr),
               want(product), "grad_input");
        expect(sg_linear_f8_grad_weight(x, SG_F32, 65536, 1, q, far, s, wide, SG_E5M2, w, far, v, wide, T, q, m, n, ws, big, nullptr),
               want(product && T <= far), "grad_weight");
      }

  for (int64_t ld : {INT64_MIN, (int64_t)-128, (int64_t)0, (int64_t)1, (int64_t)100, far + 128, INT64_MAX - 127}) {
    expect(sg_quantize_f8(q, ld, s, 16, nullptr, 0, nullptr, 0, 0, x, SG_BF16, 4, 100, 100, nullptr, nullptr), SG_ERR_INVALID_ARGUMENT, "pitch");
    expect(sg_quantize_f8(q, 128, s, ld | 1, nullptr, 0, nullptr, 0, 0, x, SG_BF16, 4, 100, 100, nullptr, nullptr), SG_ERR_INVALID_ARGUMENT,
           "scale pitch");
    expect(sg_linear_f8(x, SG_BF16, 200, q, ld, s, 16, 0, 4, w, 128, v, up(200, 16), 200, 100, ws, big, nullptr), SG_ERR_INVALID_ARGUMENT, "pitch");
  }
  for (int64_t ld : {INT64_MIN, (int64_t)0, (int64_t)99}) {
    expect(sg_quantize_f8(q, 128, s, 16, nullptr, 0, nullptr, 0, 0, x, SG_BF16, 4, 100, ld, nullptr, nullptr), SG_ERR_INVALID_ARGUMENT, "ldx");
    expect(sg_dropout(x, 100, x, SG_F32, ld, nullptr, 0, 4, 100, &drop, nullptr), SG_ERR_INVALID_ARGUMENT, "ldx");
    expect(sg_dequantize_f8(x, SG_F32, ld, q, 128, s, 16, 0, 4, 100, nullptr), SG_ERR_INVALID_ARGUMENT, "ldx");
  }
  expect(sg_quantize_f8(q, 128, s, 16, nullptr, 0, nullptr, 0, 0, x, SG_BF16, 4, 100, INT64_MAX, nullptr, nullptr), SG_ERR_UNSUPPORTED, "ldx");
  for (double p : {-1.0, -1e-300, 1.0, 1.0 - 0x1p-34, (double)INFINITY, (double)NAN}) {
    const sg_drop bad = {p, 0, 0, nullptr};
    expect(sg_dropout(x, 100, x, SG_F32, 100, nullptr, 0, 4, 100, &bad, nullptr), SG_ERR_INVALID_ARGUMENT, "p");
  }
  for (double p : {0.0, -0.0, 1e-300, 0.5, 1.0 - 0x1p-31}) {
    const sg_drop good = {p, 0, 0, nullptr};
    expect(sg_dropout(x, 100, x, SG_F32, 100, nullptr, 0, 4, 100, &good, nullptr), SG_ERR_HIP, "p");
  }
  expect(sg_linear_f8(x, SG_BF16, 4489, q, 35968, s, 80, 0, 77, w, 35968, v, 4496, 4489, 35851, nullptr, 0, nullptr), SG_ERR_WORKSPACE, "workspace");

  if (failures) {
    fprintf(stderr, "%d failure(s)\n", failures);
    return 1;
  }
  printf("f8 host checks passed\n");
  return 0;
}
