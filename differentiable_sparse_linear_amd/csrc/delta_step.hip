// The gated delta rule token by token: single tokens on a server, and short
// sequences.
#include "delta.h"

namespace sla {

namespace {

constexpr int kThreads = 256;

struct StepArgs {
    DeltaArgs a;
    const float *s_in;
    float *s_out;
    const int32_t *slots;
    int64_t n_slots;
    void *o;
    int64_t ob, ot, oh;
    float max_growth;  // of a run of gates: kMaxGrowth or infinity
};

// One workgroup holds CL * VEC columns of one head's state in registers:
// thread (rg, c) rows rg, rg + RG, ... of columns c * VEC ...  Both products
// of a token are taken in the pass that reads S,
//   S_t^T q = a (S^T q) + (q . k) beta w,
// so a token costs one reduction over the row groups, and one token reads
// and writes each state once: 8 dk dv bytes a head, which bounds it: 6144 heads
// of 128 x 128 (bf16 rows) take 162 us, 5.0 TB/s; 16 heads 5.3 us, little more
// than a launch.
template <typename T, int CL, int RPT, int VEC>
__global__ __launch_bounds__(kThreads) void delta_step_kernel(StepArgs p) {
    constexpr int RG = kThreads / CL, COLS = CL * VEC;
    const DeltaArgs &a = p.a;
    const int tid = threadIdx.x, c = tid % CL, rg = tid / CL, wave = tid / 64;
    const int h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hv / a.Hk);
    const int col = blockIdx.x * COLS + c * VEC;
    const int len = seq_len(a, b);
    T *o = reinterpret_cast<T *>(p.o) + b * p.ob + h * p.oh;
    int64_t slot = b;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.n_slots) {  // no request: the answer is 0
            for (int t = 0; t < a.T; ++t)
                for (int e = 0; e < VEC; ++e)
                    if (rg == 0 && col + e < a.dv) o[t * p.ot + col + e] = from_f32<T>(0.f);
            return;
        }
    }
    const int64_t base = (slot * a.Hv + h) * a.dk * (int64_t)a.dv;
    const T *q = reinterpret_cast<const T *>(a.q) + b * a.qb + hk * a.qh;
    const T *k = reinterpret_cast<const T *>(a.k) + b * a.kb + hk * a.kh;
    const T *v = reinterpret_cast<const T *>(a.v) + b * a.vb + h * a.vh;
    const float *beta = a.beta + b * a.bb + h * a.bh;
    const float *gate = a.gate + b * a.gb + h * a.gh;

    __shared__ float kq[2][kMaxDk][2];  // k and q of a token, double buffered
    __shared__ float red[2][kThreads / 64][2 * COLS + 1];

    float s[RPT][VEC];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int row = rg + RG * i;
        const bool in = p.s_in && row < a.dk;
        const float *src = p.s_in + base + (int64_t)row * a.dv + col;
        if constexpr (VEC == 4) {  // dv a multiple of 4: all four columns or none
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in && col < a.dv) x = *reinterpret_cast<const float4 *>(src);
            s[i][0] = x.x, s[i][1] = x.y, s[i][2] = x.z, s[i][3] = x.w;
        } else {
            s[i][0] = in && col < a.dv ? *src : 0.f;
        }
    }
    const int d = tid & (kMaxDk - 1);  // threads 0-127 read k, 128-255 q
    auto fetch = [&](int t) -> float {
        if (d >= a.dk) return 0.f;
        return tid < kMaxDk ? to_f32<T>(k[t * a.kt + d]) : to_f32<T>(q[t * a.qt + d]);
    };
    float next = len > 0 ? fetch(0) : 0.f, run = 0.f;
    for (int t = 0; t < len; ++t) {
        float(*x)[2] = kq[t & 1];
        x[d][tid / kMaxDk] = next;
        float vt[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            vt[e] = col + e < a.dv ? to_f32<T>(v[t * a.vt + col + e]) : 0.f;
        const float bt = beta[t * a.bt], gt = gate[t * a.gt];
        run = fmaxf(run, 0.f) + gt;
        const float at = run > p.max_growth ? __builtin_nanf("") : expf(gt);
        __syncthreads();
        if (t + 1 < len) next = fetch(t + 1);
        float sk[VEC] = {}, sq[VEC] = {}, dot = 0.f;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int row = rg + RG * i;
            const float kr = x[row][0], qr = x[row][1];
            dot = fmaf(kr, qr, dot);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                sk[e] = fmaf(s[i][e], kr, sk[e]);
                sq[e] = fmaf(s[i][e], qr, sq[e]);
            }
        }
#pragma unroll
        for (int off = CL; off < 64; off <<= 1) {
            dot += __shfl_xor(dot, off, 64);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                sk[e] += __shfl_xor(sk[e], off, 64);
                sq[e] += __shfl_xor(sq[e], off, 64);
            }
        }
        float *mine = red[t & 1][wave];
        if ((tid & 63) < CL) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                mine[c * VEC + e] = sk[e];
                mine[COLS + c * VEC + e] = sq[e];
            }
            if (c == 0) mine[2 * COLS] = dot;
        }
        __syncthreads();
        dot = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) dot += red[t & 1][w][2 * COLS];
        float u[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float xk = 0.f, xq = 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 64; ++w) {
                xk += red[t & 1][w][c * VEC + e];
                xq += red[t & 1][w][COLS + c * VEC + e];
            }
            u[e] = bt * (vt[e] - at * xk);
            const float ot = a.scale * fmaf(dot, u[e], at * xq);
            if (rg == 0 && col + e < a.dv) o[t * p.ot + col + e] = from_f32<T>(ot);
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float kr = x[rg + RG * i][0];
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                s[i][e] = fmaf(kr, u[e], at * s[i][e]);
        }
    }
    if (rg == 0)
        for (int t = len; t < a.T; ++t)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (col + e < a.dv) o[t * p.ot + col + e] = from_f32<T>(0.f);
    if (!p.s_out) return;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int row = rg + RG * i;
        if (row >= a.dk || col >= a.dv) continue;
        float *dst = p.s_out + base + (int64_t)row * a.dv + col;
        if constexpr (VEC == 4)
            *reinterpret_cast<float4 *>(dst) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
        else
            *dst = s[i][0];
    }
}

template <typename T, int CL, int VEC>
hipError_t launch_cl(const StepArgs &p, hipStream_t s) {
    constexpr int RG = kThreads / CL;
    const dim3 grid((p.a.dv + CL * VEC - 1) / (CL * VEC), p.a.Hv, p.a.B);
    if (p.a.dk <= kMaxDk / 2)
        delta_step_kernel<T, CL, kMaxDk / 2 / RG, VEC><<<grid, kThreads, 0, s>>>(p);
    else
        delta_step_kernel<T, CL, kMaxDk / RG, VEC><<<grid, kThreads, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const StepArgs &p, hipStream_t s) {
    const bool vec = p.a.dv % 4 == 0 && (reinterpret_cast<uintptr_t>(p.s_in) & 15) == 0 &&
                     (reinterpret_cast<uintptr_t>(p.s_out) & 15) == 0;
    if (!vec) return launch_cl<T, 16, 1>(p, s);
    // 32 columns a workgroup, or 128 where that gives two workgroups a CU: one
    // token of 32 heads of 128 x 128 takes 4.6 us and 7.0, of 256 8.6 and 9.0, of
    // 512 14.0 and 12.1, of 1024 26.5 and 23.8.
    const int64_t wide = (int64_t)p.a.B * p.a.Hv * ((p.a.dv + 127) / 128);
    if (wide >= 512) return launch_cl<T, 32, 4>(p, s);
    return launch_cl<T, 8, 4>(p, s);
}

}  // namespace

hipError_t launch_delta_step(int dtype, const DeltaArgs &a, const float *s_in, float *s_out,
                             const int32_t *slots, int64_t n_slots, void *o, int64_t ob,
                             int64_t ot, int64_t oh, float max_growth, hipStream_t s) {
    const StepArgs p{a, s_in, s_out, slots, n_slots, o, ob, ot, oh, max_growth};
    return dtype == SLA_F32   ? launch_t<float>(p, s)
           : dtype == SLA_F16 ? launch_t<__half>(p, s)
                              : launch_t<__hip_bfloat16>(p, s);
}

}  // namespace sla
