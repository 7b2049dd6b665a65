// Host-side launchers of the gfx950 kernels (one per kernel family).  Each returns
// hipGetLastError() after queuing its launch on `s`; arguments are checked by the
// C-ABI layer before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// Devices the library keeps per-device state for (compute-unit counts, kernel attributes).
constexpr int kMaxDevices = 64;

// Raises a kernel's dynamic LDS limit to `bytes` on the current device, once per device
// (`done` is the caller's per-kernel record); a no-op after the first call there.
hipError_t set_dynamic_lds_once(const void* kernel, int bytes, bool (&done)[kMaxDevices]);

// A linear's epilogue with activation and residual: from z = alpha * acc + bias in fp32,
// preact [m][n] = bf16(z) when not NULL and out = bf16(act(z) + residual), act one of
// NVFP4_ACT_*: nothing is rounded in between.  residual [m][n] bf16, NULL, or out itself:
// every element is read by the thread that writes it, just before.
struct Epilogue {
  const uint16_t* residual = nullptr;
  uint16_t* preact = nullptr;
  int act = 0;
  bool active() const { return residual != nullptr || preact != nullptr || act != 0; }
};

// Upper bound on the number of per-block partial maxima of the amax pass, and on the
// number of segments (row blocks with their own scale) of one call.
constexpr int kMaxAmaxPartials = 8192;
constexpr int kMaxSegments = 1024;

// Partial maxima of `segments` consecutive row blocks of seg_rows rows each (one
// segment for a plain call): partials[seg * (*n_partials) + i].  With `up` not NULL the
// input is the bf16 SwiGLU product of x (gate) and up, computed on the fly and, if
// xout is not NULL, stored there.
hipError_t launch_amax_partials(const uint16_t* x, const uint16_t* up, uint16_t* xout, int64_t seg_rows, int64_t k,
                                int segments, int group, float inv_sqrt_g, float* partials, int* n_partials,
                                hipStream_t s);

// Quantizes rows x [rows][k]; with static_gsf NULL, segment s (rows [s*seg_rows,
// (s+1)*seg_rows)) takes its global scale from its n_partials partial maxima and
// gsf_out[s] receives it.  With a16 not NULL, a16 [rows][k] also receives every
// quantized value as the exact fp16 code * scale * 2^-8 (the operand form of the GEMMs,
// for gemm_decode_a16).
hipError_t launch_quantize(const uint16_t* x, const uint16_t* up, int64_t rows, int64_t k, int group,
                           float inv_sqrt_g, const float* static_gsf, const float* partials, int n_partials,
                           int64_t seg_rows, int segments, uint8_t* codes, uint8_t* scales, float* gsf_out,
                           hipStream_t s, uint16_t* a16 = nullptr);

// Dynamic-scale quantize of a small input (rows * k within quantize_small_supported) in
// one launch: the same codes, scales, global scale (*gsf_out) and a16 as
// launch_amax_partials followed by launch_quantize with one segment.
bool quantize_small_supported(int64_t rows, int64_t k);
hipError_t launch_quantize_small(const uint16_t* x, int64_t rows, int64_t k, int group, float inv_sqrt_g,
                                 uint8_t* codes, uint8_t* scales, float* gsf_out, hipStream_t s,
                                 uint16_t* a16 = nullptr);

// x [rows][k] = bf16 SwiGLU product of gate and up.
hipError_t launch_swiglu(const uint16_t* gate, const uint16_t* up, uint16_t* x, int64_t rows, int64_t k, hipStream_t s);

// NVFP4 [rows][k] (codes + scales in the library layout) -> bf16 or fp32 values
// fp32(code * scale) / gsf.
hipError_t launch_dequant(const uint8_t* packed, const uint8_t* scales, int64_t rows, int64_t k, const float* gsf,
                          void* out, bool out_bf16, hipStream_t s);

// *amax = max of n_partials partial maxima (accumulate: max with the value already there).
hipError_t launch_amax_finalize(const float* partials, int n_partials, float* amax, bool accumulate, hipStream_t s);

// *gsf = 2688 / max(fp32(*amax * margin), 1e-12).
hipError_t launch_static_scale(const float* amax, float margin, float* gsf, hipStream_t s);

hipError_t launch_rotate(const void* x, bool x_bf16, void* y, bool y_bf16, int64_t rows, int64_t k, int group,
                         float inv_sqrt_g, hipStream_t s);

hipError_t launch_scale_layout(const uint8_t* src, uint8_t* dst, int64_t rows, int64_t k, bool to_canonical,
                               hipStream_t s);

// alpha = 1 / (gsf_a * gsf_b); with a_seg_rows > 0, row r of A takes gsf_a[r / a_seg_rows]
// (one global scale per block of a_seg_rows rows; not with an active epilogue), otherwise
// gsf_a[0] for every row.
hipError_t launch_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m, int64_t k,
                       const uint8_t* b_codes, const uint8_t* b_scales, int64_t n,
                       const float* gsf_a, const float* gsf_b, int64_t a_seg_rows, const uint16_t* bias,
                       const Epilogue& ep, uint16_t* out, void* workspace, size_t workspace_bytes, hipStream_t s);

// Compute units of the current device (cached per device).
int compute_units();

// The software-pipelined 256 x 256-tile GEMM (gemm_pipe.hip): K a multiple of 32 and
// every operand pointer 16-byte aligned.  Tiles beyond the
// last whole round (one tile per compute unit) are split along K when the workspace
// (gemm_pipe_workspace_bytes) allows; without it they run unsplit.
bool gemm_pipe_supported(int64_t m, int64_t k, int64_t n, const void* a_codes, const void* a_scales,
                         const void* b_codes, const void* b_scales, int cus);
size_t gemm_pipe_workspace_bytes(int64_t m, int64_t k, int64_t n, int cus);
hipError_t launch_gemm_pipe(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m, int64_t k,
                            const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, const float* gsf_a,
                            const float* gsf_b, int64_t a_seg_rows, const uint16_t* bias, const Epilogue& ep,
                            uint16_t* out, void* workspace, size_t workspace_bytes, int cus, hipStream_t s);

// The decode GEMM for m <= kDecodeA16Rows activation rows given as the fp16 operand
// form a16 [m][k] (launch_quantize's a16 output) instead of codes and scales, so the
// kernel expands only the weight.  One activation scale (gsf_a[0]).  K a multiple of
// 32, b_codes 16-byte and b_scales 4-byte aligned, a16 16-byte aligned.
constexpr int kDecodeA16Rows = 4;
bool gemm_decode_a16_supported(int64_t m, int64_t k, const void* a16, const void* b_codes, const void* b_scales);
hipError_t launch_gemm_decode_a16(const uint16_t* a16, int64_t m, int64_t k, const uint8_t* b_codes,
                                  const uint8_t* b_scales, int64_t n, const float* gsf_a, const float* gsf_b,
                                  const uint16_t* bias, const Epilogue& ep, uint16_t* out, void* workspace,
                                  size_t workspace_bytes, int cus, hipStream_t s);

// The weight-streaming GEMM for m <= 128 (gemm_skinny.hip): K a multiple of 32, code
// pointers 16-byte and scale pointers 4-byte aligned.  Splits K across blocks when the
// workspace (gemm_skinny_workspace_bytes) allows.
bool gemm_skinny_supported(int64_t m, int64_t k, const void* a_codes, const void* a_scales, const void* b_codes,
                           const void* b_scales);
size_t gemm_skinny_workspace_bytes(int64_t m, int64_t k, int64_t n, int cus);
hipError_t launch_gemm_skinny(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m, int64_t k,
                              const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, const float* gsf_a,
                              const float* gsf_b, int64_t a_seg_rows, const uint16_t* bias, const Epilogue& ep,
                              uint16_t* out, void* workspace, size_t workspace_bytes, int cus, hipStream_t s);

// The whole linear for up to 16 activation rows with a static scale, in the
// weight-streaming kernel: each block quantizes its K range of the bf16 rows x [m][k]
// into LDS (same codes and scales as launch_quantize) instead of a separate pass.
// Needs the workspace of gemm_skinny_workspace_bytes (hipErrorInvalidValue without).
// The linear at one activation row in one launch: each wave of the decode GEMM quantizes
// its K range of the bf16 row itself (bit-identical to the quantize pass then the GEMM).
// gsf_x: the static scale, or NULL for the dynamic one, which every block forms from the
// row's abs-max.  gsf_used (NULL allowed only with a static scale) receives the scale
// used.  Needs the split-K partials of gemm_workspace_bytes when the decode plan splits
// K, else runs unsplit while every wave's range fits its LDS region.
bool linear_decode_fused_supported(int64_t m, int64_t k, int64_t n, bool dynamic, const void* x,
                                   const void* b_codes, const void* b_scales, size_t workspace_bytes, int cus);
hipError_t launch_linear_decode_fused(const uint16_t* x, int64_t k, const uint8_t* b_codes, const uint8_t* b_scales,
                                      int64_t n, const float* gsf_x, float* gsf_used, const float* gsf_w,
                                      const uint16_t* bias, const Epilogue& ep, uint16_t* out, void* workspace,
                                      size_t workspace_bytes, int cus, hipStream_t s);

// RMS norm (norm.hip), k a multiple of 16 up to kNormMaxK.  x is bf16 or (x_f32) fp32;
// with a residual (bf16, or fp32 with stream_f32; an fp32 x takes an fp32 one) r receives
// the rounded sum.  kNormOut writes y (bf16) and, with codes not NULL, its checkpoint;
// kNormStatic and kNormDynamic write NVFP4 codes and scales under *gsf or the dynamic
// scale (gsf_out: the scale used); dynamic takes rstd [rows] and partials [kNormPartials].
constexpr int64_t kNormMaxK = 16384;
constexpr int kNormPartials = 1280;   // workgroups of the statistics pass at most
enum NormMode { kNormOut, kNormStatic, kNormDynamic, kNormOneRow, kNormStats };   // the last two: internal
struct NormForward {
  const void* x;
  const void* residual;
  const void* w;
  void* r;
  int64_t rows, k;
  double eps;
  bool x_f32, stream_f32, w_f32;
  int mode;
  uint16_t* y;
  uint8_t *codes, *scales;
  const float* gsf;
  float *gsf_out, *rstd, *partials;
  int lanes;   // set by the launcher
};
hipError_t launch_rmsnorm(NormForward a, hipStream_t s);

// Its gradient: grad_r [rows][k] (the stream's type; grad_residual, of that type, is added
// when not NULL) and, when not NULL, grad_w [k] fp32 through partials.
struct NormBackward {
  const uint16_t* gy;
  const void *r, *w, *grad_residual;
  int64_t rows, k;
  double eps;
  bool stream_f32, w_f32;
  void* grad_r;
  float *grad_w, *partials;
  int lanes;   // set by the launcher
};
size_t rmsnorm_backward_partial_floats(int64_t rows, int64_t k);
hipError_t launch_rmsnorm_backward(NormBackward a, hipStream_t s);

// 8-bit checkpoints (checkpoint.hip): codes [rows][k], scales [rows][ceil(k / 32)].
hipError_t launch_checkpoint_pack(const uint16_t* x, int64_t rows, int64_t k, int group, float inv_sqrt_g,
                                  uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_checkpoint_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t k, void* out,
                                    bool out_bf16, hipStream_t s);
hipError_t launch_swiglu_checkpoint(const uint16_t* gate, const uint16_t* up, int64_t rows, int64_t k, uint16_t* x,
                                    uint8_t* gate_codes, uint8_t* gate_scales, uint8_t* up_codes, uint8_t* up_scales,
                                    hipStream_t s);
// Saved operands are checkpoint codes, or bf16 where their scales are NULL.
hipError_t launch_swiglu_backward(const uint16_t* gy, const void* gate, const uint8_t* gate_scales, const void* up,
                                  const uint8_t* up_scales, int64_t rows, int64_t k, uint16_t* grad_gate,
                                  uint16_t* grad_up, hipStream_t s);
hipError_t launch_activation_backward(const uint16_t* gy, const void* z, const uint8_t* z_scales, int64_t rows,
                                      int64_t k, int act, uint16_t* grad_z, hipStream_t s);

// grad_w [n][k] (fp32, or bf16) = sum over rows of gy [rows][n] x checkpoint [rows][k]
// (weight_grad.hip).  partial: fp32 split sums, weight_grad_workspace_bytes of them, or
// NULL (unsplit).
size_t weight_grad_workspace_bytes(int64_t m, int64_t n, int64_t k, int cus);
hipError_t launch_weight_grad(const uint16_t* gy, int64_t m, int64_t n, const uint8_t* codes, const uint8_t* scales,
                              int64_t k, void* grad_w, bool out_bf16, void* workspace, size_t workspace_bytes,
                              int cus, hipStream_t s);

// Workspace the GEMM dispatcher can use for an [m, k] x [n, k] product (0 if none).
size_t gemm_workspace_bytes(int64_t m, int64_t k, int64_t n);

}  // namespace nvfp4
