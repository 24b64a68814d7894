// Host-side checks of the 8-bit linear layer's six calls under
// AddressSanitizer and UndefinedBehaviorSanitizer (built host-only by
// test_sanitize_linear8.py; no kernel is launched): refusals, the plans and
// workspace arithmetic up to the largest sizes, and plausible arguments, which
// stop at the device check where there is no GPU.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

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

int main() {
  const int64_t top = ((int64_t)1 << 31) - 1;
  const int64_t ms[] = {-1, 0, 1, 33, 64, 1000, 4096, 11008, 1 << 20, (1 << 20) + 1};
  const int64_t ns[] = {-1, 0, 1, 63, 64, 1000, 4096, 28672, 65536, 65537, INT64_MAX};
  const int64_t ts[] = {INT64_MIN, -1, 0, 1, 64, 512, 70000, 8388608, 8388609, 34000000, top, top + 1, INT64_MAX};
  const int32_t ops[] = {SG_OP_LINEAR_W8A8, SG_OP_GRAD_INPUT, SG_OP_GRAD_WEIGHT};
  for (int32_t op : ops)
    for (int64_t m : ms)
      for (int64_t n : ns)
        for (int64_t T : ts) {
          const size_t b = sg_workspace_bytes(op, m, n, T, 0);
          const bool ok = m >= 1 && m <= 1 << 20 && n >= 1 && n <= 65536 && T >= 0 && T <= top;
          if ((!ok || T == 0) && b != 0) ++failures, fprintf(stderr, "FAIL workspace of refused sizes\n");
          if (b % 256 != 0) ++failures, fprintf(stderr, "FAIL workspace alignment\n");
        }

  int8_t* q = at<int8_t>(0x10000);
  float* s = at<float>(0x20000);
  int32_t* i = at<int32_t>(0x30000);
  void* x = at<void>(0x40000);
  uint8_t* u = at<uint8_t>(0x50000);
  void* ws = at<void>(0x100000);
  const size_t big = (size_t)1 << 60;

  for (int64_t m : ms)
    for (int64_t n : ns)
      for (int64_t T : ts) {
        const bool ok = m >= 1 && m <= 1 << 20 && n >= 1 && n <= 65536 && T >= 0 && T <= top;
        const sg_status want = ok ? SG_ERR_HIP : SG_ERR_INVALID_ARGUMENT;
        const sg_status rows = n >= 1 && n <= 65536 && T >= 0 && T <= top ? SG_ERR_HIP : SG_ERR_INVALID_ARGUMENT;
        const sg_status pack = m >= 1 && m <= 1 << 20 && n >= 1 && n <= 65536 ? SG_ERR_HIP : SG_ERR_INVALID_ARGUMENT;
        expect(sg_quantize_tokens(q, 65536, s, i, x, SG_BF16, T, n, 65536, nullptr), rows, "quantize");
        expect(sg_dequantize_tokens(x, SG_F32, 65536, q, 65536, s, T, n, nullptr), rows, "dequantize");
        expect(sg_pack_w8(q, 65536, i, s, u, s, s, m, n, nullptr), pack, "pack");
        expect(sg_linear_w8a8(x, SG_BF16, 1 << 20, q, 65536, s, i, T, q, 65536, i, s, m, n, ws, big, nullptr), want, "linear");
        expect(sg_linear_w8_grad_input(x, SG_F32, 65536, x, SG_BF16, 1 << 20, T, q, 65536, i, s, m, n, ws, big, nullptr),
               want, "grad_input");
        expect(sg_linear_w8_grad_weight(x, SG_F32, 65536, 0, x, SG_BF16, 1 << 20, q, 65536, s, T, u, m, n, ws, big, nullptr),
               want, "grad_weight");
      }

  expect(sg_quantize_tokens(q, INT64_MAX - 63, s, i, x, SG_BF16, 4, 100, 100, nullptr), SG_ERR_INVALID_ARGUMENT, "pitch");
  expect(sg_quantize_tokens(q, INT64_MIN, s, i, x, SG_BF16, 4, 100, 100, nullptr), SG_ERR_INVALID_ARGUMENT, "pitch");
  expect(sg_quantize_tokens(q, 128, s, i, x, SG_BF16, 4, 100, INT64_MIN, nullptr), SG_ERR_INVALID_ARGUMENT, "ldx");
  expect(sg_quantize_tokens(q, 128, s, i, x, SG_BF16, 4, 100, INT64_MAX, nullptr), SG_ERR_UNSUPPORTED, "ldx");
  expect(sg_linear_w8_grad_input(x, SG_F32, 100, x, SG_BF16, 1000, 40, q, 128, i, s, 1000, 100, nullptr, 0, nullptr),
         SG_ERR_WORKSPACE, "workspace");
  expect(sg_linear_w8_grad_weight(x, SG_F32, 100, 0, x, SG_BF16, 1000, q, 128, s, 40, u, 1000, 100, ws, 1, nullptr),
         SG_ERR_WORKSPACE, "workspace");

  if (failures) {
    fprintf(stderr, "%d failure(s)\n", failures);
    return 1;
  }
  printf("linear8 host checks passed\n");
  return 0;
}
