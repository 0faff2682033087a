// Internal declarations of the gated delta rule kernels.
//
// For one head, with the state S [dk, dv] (fp32) and a_t = exp(gate_t):
//
//   w_t = v_t - a_t S_{t-1}^T k_t
//   S_t = a_t S_{t-1} + beta_t k_t w_t^T
//   o_t = scale S_t^T q_t
//
// a damped row-action sweep for the dense system k_t^T S = v_t (beta the
// relaxation; with unit keys, beta = 1 and a = 1 every token projects S on
// its row).  Value head h reads query and key head h / (Hv / Hk).
//
// The recurrent kernel (delta_step.hip) walks tokens.  The chunked kernels
// (delta_prep.hip, delta_scan.hip, delta_grad.hip) take kChunk tokens at a time,
// with G_i the chunk's running sum of gates and D_ij = exp(G_i - G_j):
//
//   (I + L) W = V - Gamma K S     L_ij = D_ij (k_i . k_j) beta_j,  j < i
//   O  = scale (Gamma Q S + P' W)  P'_ij = D_ij (q_i . k_j) beta_j, j <= i
//   S' = exp(G_C) S + sum_j exp(G_C - G_j) beta_j k_j w_j^T
//
// so one unit lower triangular system is solved per chunk; its backward
// pass solves the transposed one.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sla.h"

namespace sla {

void set_last_error(hipError_t e);

constexpr int kChunk = 64;       // tokens of a chunk: one per lane of a wavefront
constexpr int kMaxDk = 128;      // largest key size: state rows held by one wavefront
constexpr int kSlice = 16;       // state columns of one wavefront of the chunk scans
constexpr float kMinGate = -1000.f;  // exp underflows to 0 far above: -inf acts like this

// Whole sequences answer NaN where a run of gates within a chunk sums to more
// than this.  A chunk's products hold decays between any two of its tokens, and
// where tokens correct what grew between them (equal unit keys, beta = 1) the
// grown terms cancel: a run of 2 loses a factor of 3 in accuracy, of 8 a factor
// of 300, and 64 gates of 1 all digits.
constexpr float kMaxGrowth = 2.f;

// What every kernel of the rule reads; strides in elements, the last
// dimension of each array contiguous.
struct DeltaArgs {
    const void *q, *k, *v;
    const float *beta, *gate;
    int64_t qb, qt, qh, kb, kt, kh, vb, vt, vh;
    int64_t bb, bt, bh, gb, gt, gh;
    const int32_t *lengths;  // [B] or null: all T
    int32_t B, T, Hk, Hv, dk, dv;
    float scale;
};

__device__ inline int seq_len(const DeltaArgs &a, int b) {
    if (!a.lengths) return a.T;
    const int n = a.lengths[b];
    return n < 0 ? 0 : n > a.T ? a.T : n;
}

template <typename T>
__device__ inline float to_f32(T x);
template <>
__device__ inline float to_f32<float>(float x) { return x; }
template <>
__device__ inline float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ inline float to_f32<__hip_bfloat16>(__hip_bfloat16 x) {
    return __uint_as_float((uint32_t)__builtin_bit_cast(uint16_t, x) << 16);
}

// Rounding to nearest even; the outputs' last step.
template <typename T>
__device__ inline T from_f32(float x);
template <>
__device__ inline float from_f32<float>(float x) { return x; }
template <>
__device__ inline __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ inline __hip_bfloat16 from_f32<__hip_bfloat16>(float x) {
    return __builtin_bit_cast(__hip_bfloat16, (__bf16)x);
}

hipError_t launch_delta_step(int dtype, const DeltaArgs &a, const float *s_in, float *s_out,
                             const int32_t *slots, int64_t n_slots, void *o, int64_t ob,
                             int64_t ot, int64_t oh, float max_growth, hipStream_t s);

}  // namespace sla
