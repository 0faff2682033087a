// Launches of the chunked gated delta rule (delta_prep.hip, delta_scan.hip,
// delta_grad.hip).
#pragma once

#include "delta_tile.h"

namespace sla {

// The chunks that one round of launches works on; workspace is sized for
// them, so a long sequence goes in several rounds.
struct ChunkRange {
    int32_t first, count;
    __host__ __device__ int64_t key_chunk(const DeltaArgs &a, int b, int hk, int i) const {
        return ((int64_t)b * a.Hk + hk) * count + i;
    }
    __host__ __device__ int64_t chunk(const DeltaArgs &a, int b, int h, int i) const {
        return ((int64_t)b * a.Hv + h) * count + i;
    }
};

__host__ __device__ inline int num_chunks(const DeltaArgs &a) {
    return (a.T + kChunk - 1) / kChunk;
}
__host__ __device__ inline int padded_dv(int dv) { return (dv + 31) / 32 * 32; }

// A training pass keeps the state at every chunk's start, and W, as the scans
// hold them: for each chunk and slice of 16 columns the accumulator tiles (of
// DK / 16 and of 4 row tiles), 4 rows a lane.  The backward scan leaves dS and
// dR so.  All heads' parts of a chunk stand together: the scans write them at about
// the same time, and with a head's chunks together they would be whole powers
// of 2 apart.
__host__ __device__ inline int64_t saved_chunk(const DeltaArgs &a, int b, int h, int n) {
    return ((int64_t)n * a.B + b) * a.Hv + h;
}

// Whether the rows of q and k can be read four elements at a time.
inline bool rows_aligned(const DeltaArgs &a, int size) {
    const int64_t s = a.qb | a.qt | a.qh | a.kb | a.kt | a.kh | a.dk;
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k);
    return s % 4 == 0 && p % (4 * size) == 0;
}

struct DeltaForward {
    const float *s_in;  // null: zero
    float *s_out;       // null: not wanted (may be s_in)
    void *o;
    int64_t ob, ot, oh;
    float *save_s, *save_w;  // null: no backward pass follows
};

struct DeltaBackward {
    const void *grad_o;
    int64_t ob, ot, oh;
    const float *ds_in;  // gradient of the last state; null: zero
    float *ds_out;       // gradient of the first state, and of the state between rounds; null: not wanted
    void *dq, *dk, *dv;  // contiguous
    float *dbeta, *dgate;
    const float *save_s, *save_w;
    float *ws_ds, *ws_dr;  // per chunk of a round: dS, dR
};

// fn<T, DK>(...) of the call's type and key size (padded to 64 or 128).
#define SLA_DELTA_DISPATCH(fn, ...)                                                     \
    (a.dk <= 64 ? (dtype == SLA_F32   ? fn<float, 64>(__VA_ARGS__)                      \
                   : dtype == SLA_F16 ? fn<__half, 64>(__VA_ARGS__)                     \
                                      : fn<__hip_bfloat16, 64>(__VA_ARGS__))            \
                : (dtype == SLA_F32   ? fn<float, 128>(__VA_ARGS__)                     \
                   : dtype == SLA_F16 ? fn<__half, 128>(__VA_ARGS__)                    \
                                      : fn<__hip_bfloat16, 128>(__VA_ARGS__)))

hipError_t launch_delta_prep(int dtype, const DeltaArgs &a, const ChunkRange &cr, bool back,
                             unsigned char *ws_key, unsigned char *ws_head, hipStream_t s);
hipError_t launch_delta_scan(int dtype, const DeltaArgs &a, const ChunkRange &cr,
                             const DeltaForward &f, const unsigned char *ws_key,
                             const unsigned char *ws_head, hipStream_t s);
hipError_t launch_delta_scan_back(int dtype, const DeltaArgs &a, const ChunkRange &cr,
                                  const DeltaBackward &f, const unsigned char *ws_key,
                                  const unsigned char *ws_head, hipStream_t s);
hipError_t launch_delta_grad(int dtype, const DeltaArgs &a, const ChunkRange &cr,
                             const DeltaBackward &f, const unsigned char *ws_key,
                             const unsigned char *ws_head, hipStream_t s);

}  // namespace sla
