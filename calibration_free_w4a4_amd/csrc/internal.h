// Internal declarations shared by the host layer and the kernels of liborbq.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/orbq.h"

namespace orbq {

// api.cpp: records the detail that orbq_last_error returns (of this host thread) and gives back
// `status`; set_ok clears it and gives back ORBQ_OK.
int set_error(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int set_ok();

constexpr int kMaxPosBoundaries = 31;  // 6-bit codebooks: N/2 - 1 positive decision boundaries
constexpr int kMaxTableHalf = 256;     // quantizer table holds buckets -J..J-1, J <= 256
// 2-, 3- and 4-bit codebooks: the quantize kernel's table covers every bucket of t' in
// [-2^k, 2^k] (2^(k+1) + 4 entries of 8 bytes), so 2^k is capped at 1024 (16 KB of LDS).  Every
// Lloyd-Max codebook of f_d up to d = 16384 needs 2^k <= 1024.
constexpr int kMaxFullScale = 1024;

// Decision thresholds of one codebook in the scaled coordinate t' = t * 2^k.
//
// Positive centroids c_{N/2+p} (p = 0..N/2-1) are separated by the exact midpoints
// B_p = (c_{N/2+p} + c_{N/2+p+1}) / 2.  For fp32 t':
//   t' > 0 : rank = #{p : t' > B_p}            (ties -> lower index -> lower rank)
//   t' <= 0: rank = #{p : |t'| >= B_p}         (ties -> lower index -> higher rank)
// thr_gt[p] = largest float <= B_p * 2^k, so  t' > B_p  <=>  t' > thr_gt[p];
// thr_ge[p] = largest float <  B_p * 2^k, so  u >= B_p  <=>  u > thr_ge[p].
// 2^k is chosen so that neighbouring thresholds are at least 1.5 apart: every unit
// bucket of t' then holds at most one threshold, which lets the kernels decide with one
// table lookup and one compare per coordinate.
struct QuantParams {
  float scale;  // 2^k
  int32_t J;    // buckets j = floor(-t') are clamped to [-J, J-1]
  int32_t nb;   // number of positive boundaries, N/2 - 1
  int32_t bits;
  float thr_gt[kMaxPosBoundaries + 1];
  float thr_ge[kMaxPosBoundaries + 1];
  uint16_t vals[64];  // bf16 of the signed centroid of each code (QuantMode::kDecoded only)
};

// Host: builds QuantParams from an ascending, antisymmetric fp32 codebook.
// Returns 0 on success, nonzero when no power-of-two scale separates the thresholds.
int build_quant_params(const float* centroids, int bits, QuantParams* qp);

// Host: float64 Lloyd-Max for f_d (codebook.cpp).
int lloyd_max_host(int d, int bits, double* out);

// Decode tables for the product: bf16 bit patterns of the centroid magnitudes, by rank.
struct DecodeParams {
  int32_t bits;
  uint16_t mag[32];  // bf16(|c_{N/2+r}|), r = 0..N/2-1
};
void build_decode_params(const float* centroids, int bits, DecodeParams* dp);

uint16_t f32_to_bf16_rne(float x);

// Launchers (return hipError_t as int).
struct RotArgs {
  int32_t d, block;
  const int32_t* perm;
  const int8_t* signs;
  int32_t passes;  // composed passes (1..3); perm and signs hold passes * d entries
};

// kDecoded: activations written as the bf16 centroids of their codes (qp.vals), [n][d] bf16 with
// the 8 values of each aligned group of 8 positions in the order 0,2,4,6,1,3,5,7 (the order in
// which the product stages its operands), for a product that stages them without decoding.
// kRotateBf16: the rotated rows x' = Pi x (no quantization) as bf16, rounded to nearest even,
// in the same order within each group of 8 positions, for the weight-only product.
enum class QuantMode { kActivations, kWeights, kRotateOnly, kDecoded, kRotateBf16 };

int launch_rpbh_quantize(QuantMode mode, const uint16_t* X, int64_t n, int64_t ldx, const RotArgs& rot,
                         const QuantParams* qp, float eps, uint8_t* codes, void* norms, float* x_rot,
                         hipStream_t stream);

// The current device's compute-unit count (256 if the runtime cannot say), cached per device
// and host thread.
int device_cus();

// Weight-only product (bf16 activations, rotated in fp32): K-range splits and launcher.
// x_rot [nt][d] bf16 (QuantMode::kRotateBf16) with nt <= 16; d % 128 == 0.
void a16_splits(int64_t d, int* splits, int* ss_per_split);
int launch_a16_gemm(const uint16_t* x_rot, int nt, int64_t d, const uint8_t* w_codes, const uint16_t* w_norms,
                    const DecodeParams& dw, int64_t m, void* Y, int y_bf16, int64_t ldy, hipStream_t stream);

int launch_flatness(const uint16_t* X, int64_t n, int32_t d, int64_t ldx, float* rho3, float* rhoinf,
                    hipStream_t stream);

int launch_quantize_t(const float* t, int64_t count, const QuantParams& qp, uint8_t* codes,
                      hipStream_t stream);

// The current device's fixed workspace for orbq_linear_noalloc (noalloc.hip).
int noalloc_scratch(void** ptr);

int launch_lut_gemm(const uint8_t* x_codes, const float* x_norms, const DecodeParams& da,
                    const uint8_t* w_codes, const uint16_t* w_norms, const DecodeParams& dw,
                    int64_t n, int64_t m, int64_t d, void* Y, int y_bf16, int64_t ldy,
                    int act, hipStream_t stream);

// The checks and steps of the layer's entry points (api.cpp); each returns a status and says what it is about.
namespace layer {
int check_dim(int64_t d, const char* what);
int check_rot(const orbq_rpbh* rot, int64_t d, const char* what);
int check_codebook(const orbq_codebook* cb, int64_t d, const char* what);
int check_product(const uint8_t* x_codes, const float* x_norms, const orbq_codebook* cb_a, const uint8_t* w_codes,
                  const void* w_norms, const orbq_codebook* cb_w, int64_t n, int64_t m, int64_t d, void* Y,
                  orbq_dtype y_type, int64_t ldy, const char* what, bool check_x);
int check_layer(const orbq_rpbh* rot, const orbq_codebook* cb_a, const uint8_t* w_codes, const void* w_norms,
                const orbq_codebook* cb_w, int64_t n, int64_t m, int64_t d, int64_t ldx, void* Y, orbq_dtype y_type,
                int64_t ldy, const char* what);
int check_a16(const void* X, int64_t n, int64_t d, int64_t ldx, const orbq_rpbh* rot, const uint8_t* w_codes, const void* w_norms,
              const orbq_codebook* cb_w, int64_t m, void* workspace, size_t ws_bytes, void* Y, orbq_dtype y_type, int64_t ldy,
              const char* what);
int quantize_rows(QuantMode mode, const void* X, int64_t n, int64_t d, int64_t ld, const orbq_rpbh* rot,
                  const orbq_codebook* cb, float eps, uint8_t* codes, void* norms, size_t norm_align, void* stream,
                  const char* what);
// the layer keeps its activations' bf16 centroids instead of their codes
bool keeps_centroids(int32_t bits_a, int64_t m);
size_t codes_bytes(int64_t n, int64_t d, int32_t bits);  // of the codes in the layer's workspace
constexpr int64_t kA16Tokens = 16;                       // tokens per weight-only launch
size_t a16_tokens_bytes(int64_t n, int64_t d);           // of the rotated tokens in its workspace
}  // namespace layer

// What the fused products do behind the scaled product: Y = residual + gate[group] act(. + bias).
struct ProductEpilogue {
  int act;
  const void* bias;
  const void* gate;
  const void* residual;  // of Y's type
  int64_t gate_ld, residual_ld;
  int bias_f32, gate_f32;  // else bf16
  const int32_t* cu;
  int32_t groups;
};

// the rows of a call that a launch of at most 16 has
struct FusedRows {
  const ProductEpilogue& ep;
  int64_t row0, rows;  // the launch's first, and how many the call has
};
int launch_a16_gemm_fused(const uint16_t* x_rot, int nt, int64_t d, const uint8_t* w_codes, const uint16_t* w_norms,
                          const DecodeParams& dw, int64_t m, void* Y, int y_bf16, int64_t ldy, const FusedRows& fused,
                          hipStream_t stream);
int launch_a16_gemm_rot_fused(const uint16_t* X, int64_t ldx, int nt, int64_t d, const int32_t* perm, const int8_t* signs,
                              int32_t h, const uint8_t* w_codes, const uint16_t* w_norms, const DecodeParams& dw, int64_t m,
                              void* Y, int y_bf16, int64_t ldy, const FusedRows& fused, hipStream_t stream);

int launch_lut_gemm_fused(const uint8_t* x_codes, const float* x_norms, const DecodeParams& da, const uint8_t* w_codes,
                          const uint16_t* w_norms, const DecodeParams& dw, int64_t n, int64_t m, int64_t d, void* Y,
                          int y_bf16, int64_t ldy, const ProductEpilogue& ep, hipStream_t stream);

// The form for few token rows, whose sums are in another order.
bool takes_few_rows(int64_t n, int64_t m, int64_t d);
int launch_lut_gemm_few(const uint8_t* x_codes, const float* x_norms, const DecodeParams& da, const uint8_t* w_codes,
                        const uint16_t* w_norms, const DecodeParams& dw, int64_t n, int64_t m, int64_t d, void* Y,
                        int y_bf16, int64_t ldy, const ProductEpilogue& ep, hipStream_t stream);

}  // namespace orbq
