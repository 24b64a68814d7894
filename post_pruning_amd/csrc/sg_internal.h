// Internal declarations of the gfx950 SparseGPT layer solver library.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/sg.h"
#include "hessian.h"

namespace sg {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// the same at any address that its elements have: vector memory takes it (rows of
// 4095 bf16 are dropped out 2.6 times as fast as element by element)
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_bytes __attribute__((ext_vector_type(4), aligned(1)));

constexpr int kNumCU = 256;       // MI355X compute units (launch sizing only)
constexpr int kFactorNB = 128;    // factorisation panel width
constexpr int kGemmTile = 128;    // fp32 MFMA update tile edge
constexpr int kSelBins = 2048;    // radix-select histogram bins
constexpr int kRecTile = 128;     // reconstruction-error output tile edge

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

__device__ inline float bf16_to_f32(uint16_t h) {
  return __uint_as_float(static_cast<uint32_t>(h) << 16);
}

// ---------------------------------------------------------------------------
// Host-side error reporting (thread-local message).
// ---------------------------------------------------------------------------
sg_status set_error(sg_status s, const char* fmt, ...);
sg_status check_launch(const char* what);

// ---------------------------------------------------------------------------
// Factorisation
// ---------------------------------------------------------------------------
size_t factor_ws_bytes(int64_t n);
sg_status launch_prepare_hinv(float* Hinv, const float* H, int64_t n, double damp,
                              int32_t* info, void* ws, hipStream_t st, hipStream_t side,
                              hipEvent_t ev_a, hipEvent_t ev_b);
// nl layers of order n in one set of launches; layer L's part of the workspace
// starts factor_ws_bytes(n) * L bytes in; info[L] is its status.
sg_status launch_prepare_hinv_batched(float* const* Hinv, const float* const* H, int nl, int64_t n,
                                      double damp, int32_t* info, void* ws, hipStream_t st,
                                      hipStream_t side, hipEvent_t ev_a, hipEvent_t ev_b);

// ---------------------------------------------------------------------------
// Prune
// ---------------------------------------------------------------------------
struct PruneArgs {
  float* W_out;
  uint8_t* mask_out;
  const void* W;
  int w_dtype;
  int64_t m, n, ldw;
  const float* U;
  // seg_u: every stacked matrix has a factor of its own, Useg[p] (else all
  // share U)
  bool seg_u;
  const float* Useg[SG_MAX_SEGMENTS];
  int kind;
  double sparsity;
  int n_keep, m_group;
  int blocksize;
  const uint8_t* mask_in;
  // row segments: W stacks nseg matrices that share the input (and U);
  // unstructured selection is per segment
  int nseg;
  int64_t seg_rows[SG_MAX_SEGMENTS + 1];
  // vector-level removal: 1 = column by column, 16 = joint per 16 columns
  int vec;
  // joint quantization (bits == 0: pruning only)
  int bits;
  uint8_t* codes_out;
  float* qscale;
  float* qzero;
};
size_t prune_ws_bytes(int64_t m, int64_t n, int blocksize);
// The no-allocation prune entry point's scratch array (per device; its size
// is SG_NOALLOC_SCRATCH_BYTES): its device address on the current device.
constexpr size_t kNoAllocScratchBytes = SG_NOALLOC_SCRATCH_BYTES;
sg_status noalloc_scratch(void** ptr);
sg_status launch_prune(const PruneArgs& a, void* ws, hipStream_t st);

// ---------------------------------------------------------------------------
// 2:4 compressed export
// ---------------------------------------------------------------------------
sg_status launch_pack_two_four(void* values, int v_dtype, uint8_t* meta, int32_t* bad,
                               const float* W_hat, const uint8_t* mask, int64_t m, int64_t n,
                               hipStream_t st);

// ---------------------------------------------------------------------------
// Reconstruction error
// ---------------------------------------------------------------------------
size_t recon_ws_bytes(int64_t m, int64_t T);
sg_status launch_recon(double* err, int accumulate, const void* W, int w_dtype,
                       int64_t ldw, const float* W_hat, int64_t m, int64_t n,
                       const void* X, int x_dtype, int64_t T, int64_t ldx,
                       void* ws, hipStream_t st);

// ---------------------------------------------------------------------------
// 8-bit linear layer
// ---------------------------------------------------------------------------
sg_status launch_quantize_tokens(int8_t* Q, int64_t ldq, float* scale, int32_t* sum, const void* X,
                                 int x_dtype, int64_t T, int64_t n, int64_t ldx, hipStream_t st);
sg_status launch_dequantize_tokens(void* X, int x_dtype, int64_t ldx, const int8_t* Q, int64_t ldq,
                                   const float* scale, int64_t T, int64_t n, hipStream_t st);
sg_status launch_pack_w8(int8_t* Wq, int64_t ldw, int32_t* offset, float* w_scale, const uint8_t* codes,
                         const float* scale, const float* zero, int64_t m, int64_t n, hipStream_t st);

struct LinearArgs {
  void* Y;
  int y_dtype;
  int64_t ldy;
  const int8_t* Q;
  int64_t ldq;
  const float* x_scale;
  const int32_t* x_sum;
  int64_t T;
  const int8_t* Wq;
  int64_t ldw;
  const int32_t* w_offset;
  const float* w_scale;
  int64_t m, n;
};
size_t linear_ws_bytes(int64_t m, int64_t n, int64_t T);
sg_status launch_linear_w8a8(const LinearArgs& a, void* ws, hipStream_t st);

struct GradInputArgs {
  void* dX;
  int dx_dtype;
  int64_t lddx;
  const uint16_t* dY;
  int64_t lddy;
  int64_t T;
  const int8_t* Wq;
  int64_t ldw;
  const int32_t* w_offset;
  const float* w_scale;
  int64_t m, n;
};
size_t grad_input_ws_bytes(int64_t m, int64_t n, int64_t T);
sg_status launch_grad_input(const GradInputArgs& a, void* ws, hipStream_t st);

struct GradWeightArgs {
  void* dW;
  int dw_dtype;
  int64_t lddw;
  int accumulate;
  const uint16_t* dY;
  int64_t lddy;
  const int8_t* Q;
  int64_t ldq;
  const float* x_scale;
  int64_t T;
  const uint8_t* mask;
  int64_t m, n;
};
size_t grad_weight_ws_bytes(int64_t m, int64_t n, int64_t T);
sg_status launch_grad_weight(const GradWeightArgs& a, void* ws, hipStream_t st);

// ---------------------------------------------------------------------------
// Dropout and the linear layer in 8-bit floating point
// ---------------------------------------------------------------------------
struct DropArgs {
  uint32_t threshold;     // kept: words from here on
  float grow;             // 1 / (1 - p)
  uint64_t seed, offset;  // state[0] and state[1] are added where there is one
  const uint64_t* state;
};
sg_status launch_dropout(void* Y, int64_t ldy, const void* X, int dtype, int64_t ldx, const void* R, int64_t ldr,
                         int64_t T, int64_t n, const DropArgs& d, hipStream_t st);
sg_status launch_quantize_f8(uint8_t* Q, int64_t ldq, uint8_t* q_scale, int64_t ldqs, uint8_t* Qt, int64_t ldqt,
                             uint8_t* qt_scale, int64_t ldqts, int format, const void* X, int x_dtype, int64_t T,
                             int64_t n, int64_t ldx, const DropArgs* drop, hipStream_t st);
sg_status launch_dequantize_f8(void* X, int x_dtype, int64_t ldx, const uint8_t* Q, int64_t ldq,
                               const uint8_t* scale, int64_t lds, int format, int64_t T, int64_t n, hipStream_t st);
sg_status launch_pack_f8(uint8_t* Wq, int64_t ldw, uint8_t* w_scale, int64_t ldws, uint8_t* Wt, int64_t ldwt,
                         uint8_t* wt_scale, int64_t ldwts, const void* W, int w_dtype, int64_t m, int64_t n,
                         int64_t ld, hipStream_t st);

// out[nb x na] = B A^T over a contraction of k
struct F8LinearArgs {
  const uint8_t* A;  // e4m3
  int64_t lda;
  const uint8_t* a_scale;
  int64_t a_lds, na;
  const uint8_t* B;
  int b_format;
  int64_t ldb;
  const uint8_t* b_scale;
  int64_t b_lds, nb;
  int64_t k;
  void* out;
  int out_dtype;
  int64_t ldo;
  const uint8_t* mask;
  int accumulate;
  const DropArgs* drop;
};
size_t linear_f8_ws_bytes(int64_t na, int64_t nb, int64_t k);
sg_status launch_linear_f8(const F8LinearArgs& a, void* ws, const char* what, hipStream_t st);

}  // namespace sg
