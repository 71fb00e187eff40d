// Internal declarations shared by the HIP kernels and the C ABI of libconvrot.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convrot {

// Code formats of the rotate+quantize kernel.
constexpr int kFmtInt4 = 4;  // int4 codes, K'/2 bytes per row, row scale s = max/7
constexpr int kFmtInt8 = 8;  // int8 codes, K' bytes per row, row scale s = max/127
constexpr int kFmtMx4 = 1;   // MXFP4: E2M1 codes, K'/2 bytes per row, E8M0 bytes bs[M][S]
                             // with S = 4 ceil(K'/128) (K'/32 blocks, zero padding)

// Launches the fused pad + group-wise RHT + absmax + quantize + pack kernel on rows [0, M)
// of x (row stride ldx elements).  g in {16, 64, 256, 1024} (MXFP4: 64, 256, 1024);
// Kp = K' <= 65536.  x_dtype: 0 = fp32, 1 = bf16.  fmt: a kFmt* value; s is used by the
// integer formats, bs by MXFP4.  vec_bytes: bytes per input load, 16 (every element dword
// aligned) or 2 (bf16 rows at odd element offsets).
hipError_t launch_rotate_quant(const void* x, int x_dtype, int64_t M, int64_t K, int64_t ldx,
                               int g, int64_t Kp, int fmt, int vec_bytes, uint8_t* q, float* s,
                               uint8_t* bs, float* xrot, hipStream_t stream);

// Launches the W4A4 GEMM with the fused dequant epilogue.  Kp must be a multiple of 16
// (packed rows of a multiple of 8 bytes).
hipError_t launch_w4a4_gemm(const uint8_t* xq, const float* xs, const uint8_t* wq,
                            const float* ws, const uint16_t* bias, int64_t M, int64_t N,
                            int64_t Kp, uint16_t* y, int32_t* acc_dbg, hipStream_t stream);

// Launches the W8A8 GEMM (int8 codes, K' bytes per row, exact int32 sums) with the same
// fused dequant epilogue.  Kp must be a multiple of 16.
hipError_t launch_w8a8_gemm(const uint8_t* xq, const float* xs, const uint8_t* wq,
                            const float* ws, const uint16_t* bias, int64_t M, int64_t N,
                            int64_t Kp, uint16_t* y, int32_t* acc_dbg, hipStream_t stream);

// Launches the MXFP4 GEMM: packed E2M1 codes (K'/2 bytes per row) with E8M0 block scales
// (rows of 4 ceil(K'/128) bytes), fp32 accumulation on the scaled FP4 matrix instructions,
// y = bf16(sum + bias).  Kp must be a multiple of 64.  acc_dbg: the fp32 sums, or NULL.
hipError_t launch_mxfp4_gemm(const uint8_t* xq, const uint8_t* xbs, const uint8_t* wq,
                             const uint8_t* wbs, const uint16_t* bias, int64_t M, int64_t N,
                             int64_t Kp, uint16_t* y, float* acc_dbg, hipStream_t stream);

// Compute units of the current device (cached per device; 256 if the query fails).
int device_cus();

// The fused single-launch ConvLinear4bit (bf16 rows, g = 256 or 1024, int4 codes): whether a
// shape is supported, and the launch.  xq / xs: the workspace's codes and scales; fail: a word
// of device memory that the kernel sets to nonzero if its grid barrier timed out.
bool fused_linear_supported(int x_dtype, int g, int64_t M, int64_t N, int64_t K, int64_t Kp);
hipError_t launch_fused_linear(const void* x, int64_t M, int64_t K, int g, int64_t Kp,
                               uint8_t* xq, float* xs, const uint8_t* wq, const float* ws,
                               const uint16_t* bias, int64_t N, uint16_t* y, unsigned* fail,
                               hipStream_t stream);

// Small launch helper that returns the launch status instead of relying on hipGetLastError.
template <typename... KArgs, typename... Args>
inline hipError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t shmem,
                                hipStream_t stream, Args... args) {
  static_assert(sizeof...(KArgs) == sizeof...(Args), "argument count mismatch");
  return [&](KArgs... typed) {
    void* argv[] = {(void*)&typed...};
    return hipLaunchKernel((const void*)kernel, grid, block, argv, shmem, stream);
  }(static_cast<KArgs>(args)...);
}

// Analysis helpers (rowquant.hip): per-row int4 quantization without rotation, dequantization.
hipError_t launch_quant_rows_int4(const float* y, int64_t M, int64_t K, int64_t ldy, uint8_t* q,
                                  float* s, hipStream_t stream);
hipError_t launch_dequant_int4(const uint8_t* q, const float* s, int64_t M, int64_t K,
                               double* out, hipStream_t stream);

// Offline weights with group scales (w4a16.hip): rotate rows of w [N][K] (padded to Kp) in
// windows of g (0: no rotation), one bf16 scale per sg values, 4-bit codes.
hipError_t launch_quant_weight_g4(const void* w, int w_dtype, int64_t N, int64_t K, int g, int sg, int64_t Kp,
                                  uint8_t* wq, uint16_t* ws, hipStream_t stream);

// How the W4A16 product of M rows runs, and the workspace it needs.
struct W4A16Plan {
  int64_t units;        // of 256 columns of the padded depth
  int vector_units;     // one or two rows: of a wave, all of its part of K at once (1, 2, 4 or 8); 0: more of them
  int64_t rows_padded;  // activation rows of the prepared operand; 0: one launch, no workspace
  size_t operand_bytes, factor_bytes;
};
W4A16Plan plan_w4a16(int64_t M, int64_t Kp, int g);
hipError_t launch_w4a16_linear(const void* x, int x_dtype, int64_t M, int64_t K, int64_t ldx, int g, int sg,
                               int64_t Kp, const uint8_t* wq, const uint16_t* ws, int64_t N,
                               const uint16_t* bias, uint16_t* y, void* workspace, hipStream_t stream);

// Rotary positions (rotary.hip): strides in elements; heads 0: no such tensor.
struct RotaryPart {
  const void* in;
  void* out;
  int64_t in_t, in_h, out_t, out_h;
  int heads;
};
struct RotaryArgs {
  RotaryPart q, k;
  const int64_t* pos;
  const float* inv_freq;
  float factor;
  int D, R, interleaved, inverse;
};
hipError_t launch_rotary(const RotaryArgs& a, int dtype, int64_t T, hipStream_t stream);

// The paged 8-bit key/value cache (kv8.hip).
struct Kv8Batch {
  const int32_t* cu;     // [B + 1]: first row of each sequence among the T rows
  const int32_t* lens;   // [B]: tokens of each sequence, the rows' own included
  const int32_t* table;  // [B][table_ld]: pages of each sequence
  int64_t B, T, table_ld, max_pages;
};
struct Kv8Cache {
  int8_t* kc;   // [num_pages][H][page][D]
  float* ks;    // [num_pages][H]
  int8_t* vc;   // [num_pages][H][D][page]
  float* vs;    // [num_pages][H]
  int64_t num_pages;
  int page, H, D;
};
hipError_t launch_kv8_append(const void* k, const void* v, int dtype, int64_t k_t, int64_t k_h, int64_t v_t,
                             int64_t v_h, const Kv8Batch& b, const Kv8Cache& c, int g, int64_t max_new,
                             hipStream_t stream);
hipError_t launch_kv8_read(const Kv8Batch& b, const Kv8Cache& c, int g, int64_t max_new, uint16_t* k,
                           uint16_t* v, hipStream_t stream);

// Attention over it: how the work is split, and the workspace that needs.
struct Kv8Plan {
  int row_tiles;       // 16-row tiles of a workgroup: 1, 2 or 4 (few rows), 8 or 16 (many)
  int64_t row_blocks;  // per sequence and cached head
  int splits;          // of a sequence's tokens
  size_t bytes;
};
Kv8Plan plan_kv8_attention(int64_t B, int64_t T, int64_t Hq, int64_t H, int64_t D, int64_t max_new,
                           int64_t max_len);
hipError_t launch_kv8_attention(const void* q, int dtype, int64_t q_t, int64_t q_h, int64_t Hq,
                                const Kv8Batch& b, const Kv8Cache& c, int g, float scale, const Kv8Plan& p,
                                uint16_t* out, void* workspace, hipStream_t stream);

}  // namespace convrot
