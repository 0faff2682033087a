// Operators on lists of tensors: the gradients' norm, clipping by it, and the
// AdamW step that clips as it reads.
//
// A list goes in launches whose tables of pointers travel as kernel
// arguments: nothing is copied to the device and nothing is kept from
// one call to the next.  Each tensor is cut into chunks and each workgroup
// takes a chunk or a run of them.  The norm's partial sums, one per
// workgroup, are added in one fixed order by whoever needs the norm (every
// workgroup of the clipping and AdamW kernels, or one finishing kernel): no
// atomics, and results that do not depend on scheduling.
//
// Every kernel is bound by the bytes it streams (a 4 GiB copy moves 4.75 TB/s
// on the same card).  200M gradients, bf16 and fp32: the norm reads 402 MB in
// 88-91 us (120 us through the caches), clipping reads and writes them in 150-168
// us (246 us with 2048 workgroups that each walk a long run of chunks instead of
// one workgroup a chunk).  AdamW on 150M parameters, 4.2 GB: 757 us, 5.5 TB/s
// (1260 us with 2048 workgroups).
#include <cmath>
#include <type_traits>

#include "delta.h"

namespace sla {

namespace {

constexpr int kThreads = 256;
// Values of a workgroup's chunk.  The norm reads one array and scaling reads and
// writes one: there long chunks pay (a list of 200M values: scaled in 148 us with
// 8192, 166 with 4096, 502 with 1024; the norm of 4M in 7 us against 12).  AdamW's
// workgroups have five arrays each, and one vector of four of each a thread is
// enough in flight: 150M values in 732 us with 1024, 816 with 4096, 844 with
// 8192; 64k values in 3.2 us against 7.4 (all without the counters of skipped
// steps in the table).
constexpr int kGradElems = 8192, kStepElems = 1024;
constexpr int kMaxSums = 2048;       // partial sums of one table: 8 workgroups a CU
constexpr int kMaxBlocks = 1 << 20;  // workgroups of an updating launch
constexpr int kDirect = kThreads;    // partial sums that every workgroup adds up for itself

// A table of tensors as a kernel argument (within 4 KB).  Entries name the
// chunks of the table that come before them; vec: every array of the tensor
// starts at a multiple of 16 bytes.
struct GradEntry {
    void *grad;
    int64_t n;
    int32_t first;
    uint8_t grad_type, vec;
};
struct AdamEntry {
    void *grad, *param, *exp_avg, *exp_avg_sq, *master;
    int64_t n, step, *skipped;
    double rate, root;  // lr / (1 - b1^step), 1 / sqrt(1 - b2^step), with no step skipped
    int32_t first;
    uint8_t grad_type, param_type, vec;
};
template <typename E>
struct Table {
    static constexpr int kMost = (4096 - 256) / sizeof(E);
    int32_t count, chunks, elems;  // elems: values of a chunk
    E e[kMost];
};
template <typename T>
struct alignas(4 * sizeof(T) < 16 ? 4 * sizeof(T) : 16) Four {
    T x[4];
};

// 16 bytes, or 8 of a 2-byte type; NT: past the caches, for what is not used
// again before it would be gone from them.
template <bool NT, typename T>
__device__ inline void move_part(const T *from, T *to) {
    typedef uint32_t Part __attribute__((ext_vector_type(sizeof(T) == 2 ? 2 : 4)));
    const Part *f = reinterpret_cast<const Part *>(from);
    Part *t = reinterpret_cast<Part *>(to);
    if constexpr (NT)
        *t = __builtin_nontemporal_load(f);
    else
        *t = *f;
}

// Four values from p, in the vector case by accesses of up to 16 bytes.
template <bool NT, typename T>
__device__ inline Four<T> load4(const T *p, bool vec) {
    Four<T> y;
    if (vec) {
        move_part<NT>(p, y.x);
        if constexpr (sizeof(T) == 8) move_part<NT>(p + 2, y.x + 2);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) y.x[e] = p[e];
    }
    return y;
}

template <bool NT, typename T>
__device__ inline void store4(T *p, const Four<T> &y, bool vec) {
    if (vec) {
        typedef uint32_t Part __attribute__((ext_vector_type(sizeof(T) == 2 ? 2 : 4)));
        const Part *f = reinterpret_cast<const Part *>(y.x);
        Part *t = reinterpret_cast<Part *>(p);
#pragma unroll
        for (int i = 0; i < (sizeof(T) == 8 ? 2 : 1); ++i) {
            if constexpr (NT)
                __builtin_nontemporal_store(f[i], t + i);
            else
                t[i] = f[i];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = y.x[e];
    }
}

// In the type that a tensor is computed in: fp64 for fp64, else fp32.
template <typename T>
using Wide = std::conditional_t<std::is_same_v<T, double>, double, float>;
template <typename T>
__device__ inline Wide<T> widen(T x) {
    if constexpr (std::is_same_v<T, double>)
        return x;
    else
        return to_f32<T>(x);
}
template <typename T, typename W>
__device__ inline T narrow(W x) {
    if constexpr (std::is_same_v<T, double>)
        return x;
    else
        return from_f32<T>(x);
}

__device__ inline double wave_sum(double x) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, 64);
    return x;
}

__device__ inline double block_sum(double x) {
    __shared__ double part[kThreads / 64];
    x = wave_sum(x);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) x += part[w];
    __syncthreads();
    return x;
}

// sqrt of the sum of all partial sums, the same in every thread of every
// workgroup.
__device__ inline double norm_of(const double *part, int n) {
    double x = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) x += part[i];
    return sqrt(block_sum(x));
}

__device__ inline void put_norm(void *out, int type, double x) {
    if (type == SLA_F64)
        *reinterpret_cast<double *>(out) = x;
    else
        *reinterpret_cast<float *>(out) = (float)x;
}

// Calls f(entry, begin, end) for each piece of a tensor in this workgroup's
// run of chunks.
template <typename E, typename F>
__device__ inline void for_pieces(const Table<E> &tb, F &&f) {
    const int64_t n = tb.chunks;
    int chunk = (int)(n * blockIdx.x / gridDim.x);
    const int stop = (int)(n * (blockIdx.x + 1) / gridDim.x);
    int lo = 0, hi = tb.count - 1;  // the last tensor that begins at or before the run
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (tb.e[mid].first <= chunk) lo = mid; else hi = mid - 1;
    }
    for (; chunk < stop; ++lo) {
        const E &e = tb.e[lo];
        const int end = lo + 1 < tb.count ? tb.e[lo + 1].first : tb.chunks;
        const int upto = end < stop ? end : stop;
        const int64_t b = (int64_t)(chunk - e.first) * tb.elems;
        int64_t z = (int64_t)(upto - e.first) * tb.elems;
        if (z > e.n) z = e.n;
        f(e, b, z);
        chunk = upto;
    }
}

// Squares are taken and added in fp64: no fp32 gradient's square leaves its
// range, and the sum of 2^31 of them keeps more than fp32's digits.
template <typename T>
__device__ double square_sum(const T *g, int64_t b, int64_t z, bool vec) {
    double s0 = 0.0, s1 = 0.0;
    constexpr int kUnroll = 4;
    int64_t i = b + 4 * threadIdx.x;
    for (; i + 4 * kThreads * (kUnroll - 1) + 4 <= z; i += 4 * kThreads * kUnroll) {
        Four<T> y[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) y[u] = load4<true>(g + i + 4 * kThreads * u, vec);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const double a = widen(y[u].x[e]), c = widen(y[u].x[e + 1]);
                s0 = fma(a, a, s0);
                s1 = fma(c, c, s1);
            }
    }
    for (; i < z; i += 4 * kThreads)
        for (int e = 0; e < 4; ++e)
            if (i + e < z) {
                const double a = widen(g[i + e]);
                s0 = fma(a, a, s0);
            }
    return s0 + s1;
}

__global__ __launch_bounds__(kThreads) void square_sum_kernel(Table<GradEntry> tb, double *part) {
    double s = 0.0;
    for_pieces(tb, [&](const GradEntry &e, int64_t b, int64_t z) {
        switch (e.grad_type) {
            case SLA_F64: s += square_sum(static_cast<const double *>(e.grad), b, z, e.vec); break;
            case SLA_F32: s += square_sum(static_cast<const float *>(e.grad), b, z, e.vec); break;
            case SLA_F16: s += square_sum(static_cast<const __half *>(e.grad), b, z, e.vec); break;
            default:
                s += square_sum(static_cast<const __hip_bfloat16 *>(e.grad), b, z, e.vec);
        }
    });
    s = block_sum(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The sum of all partial sums, for lists so long that each workgroup of the
// next launch would take longer over them than this launch does.
__global__ __launch_bounds__(kThreads) void total_kernel(const double *part, int n, double *out) {
    double x = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) x += part[i];
    x = block_sum(x);
    if (threadIdx.x == 0) *out = x;
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const double *part, int n, void *out,
                                                        int type) {
    const double norm = norm_of(part, n);
    if (threadIdx.x == 0) put_norm(out, type, norm);
}

__device__ inline double clip_factor(double norm, double max_norm) {
    const double c = max_norm / (norm + 1e-6);
    return c < 1.0 || c != c ? c : 1.0;
}

template <typename T>
__device__ void scale(T *g, int64_t b, int64_t z, bool vec, Wide<T> c) {
    int64_t i = b + 4 * threadIdx.x;
    for (; i + 4 <= z; i += 4 * kThreads) {
        Four<T> y = load4<false>(g + i, vec);
#pragma unroll
        for (int e = 0; e < 4; ++e) y.x[e] = narrow<T>(widen(y.x[e]) * c);
        store4<false>(g + i, y, vec);
    }
    for (int e = 0; e < 4; ++e)
        if (i + e < z) g[i + e] = narrow<T>(widen(g[i + e]) * c);
}

__global__ __launch_bounds__(kThreads) void clip_kernel(Table<GradEntry> tb, const double *part,
                                                        int n, double max_norm, void *out, int type) {
    const double norm = norm_of(part, n), c = clip_factor(norm, max_norm);
    if (out && blockIdx.x == 0 && threadIdx.x == 0) put_norm(out, type, norm);
    if (c == 1.0) return;
    for_pieces(tb, [&](const GradEntry &e, int64_t b, int64_t z) {
        switch (e.grad_type) {
            case SLA_F64: scale(static_cast<double *>(e.grad), b, z, e.vec, c); break;
            case SLA_F32: scale(static_cast<float *>(e.grad), b, z, e.vec, (float)c); break;
            case SLA_F16: scale(static_cast<__half *>(e.grad), b, z, e.vec, (float)c); break;
            default:
                scale(static_cast<__hip_bfloat16 *>(e.grad), b, z, e.vec, (float)c);
        }
    });
}

struct AdamArgs {
    double lr, b1, b2, eps, keep, max_norm;  // keep = 1 - lr weight_decay
    double rate, root;                       // of the tensor at hand
};

// b^n, n >= 1, by squaring.
__device__ inline double power(double b, int64_t n) {
    double y = 1.0;
    for (; n > 0; n >>= 1, b *= b)
        if (n & 1) y *= b;
    return y;
}

// A value that is the same in all lanes, in scalar registers.
__device__ inline double uniform(double x) {
    const uint64_t y = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)y),
                   hi = __builtin_amdgcn_readfirstlane((uint32_t)(y >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The tensor's rate and root: the host's where no step was skipped (134M bf16
// values with masters: 206 us a launch of three; from then on 225).
__device__ inline void set_rates(const AdamEntry &t, AdamArgs &o) {
    o.rate = t.rate, o.root = t.root;
    const int64_t skipped = t.skipped ? *t.skipped : 0;
    if (skipped == 0) return;
    const int64_t step = t.step - skipped > 1 ? t.step - skipped : 1;
    o.rate = uniform(o.lr / (1.0 - power(o.b1, step)));
    o.root = uniform(1.0 / sqrt(1.0 - power(o.b2, step)));
}

// P the params' type, M the master's (P: there is none), G the gradients'.
template <typename P, typename M, typename G>
__device__ void adamw(const AdamEntry &t, int64_t b, int64_t z, const AdamArgs &o,
                      double factor) {
    using W = Wide<M>;
    const W b1 = (W)o.b1, b2 = (W)o.b2, n1 = (W)(1.0 - o.b1), n2 = (W)(1.0 - o.b2),
            eps = (W)o.eps, keep = (W)o.keep, rate = (W)o.rate, root = (W)o.root, c = (W)factor;
    const bool vec = t.vec;
    P *p = static_cast<P *>(t.param);
    M *master = static_cast<M *>(std::is_same_v<P, M> ? t.param : t.master);
    const G *g = static_cast<const G *>(t.grad);
    W *m = static_cast<W *>(t.exp_avg), *v = static_cast<W *>(t.exp_avg_sq);
    auto one = [&](W gx, W &mx, W &vx, W &px) {
        gx *= c;
        mx = b1 * mx + n1 * gx;
        vx = b2 * vx + n2 * (gx * gx);
        px = keep * px - rate * mx / (sqrt(vx) * root + eps);
    };
    int64_t i = b + 4 * threadIdx.x;
    for (; i + 4 <= z; i += 4 * kThreads) {
        const Four<G> gx = load4<true>(g + i, vec);
        Four<W> mx = load4<true>(m + i, vec), vx = load4<true>(v + i, vec);
        Four<M> px = load4<true>(master + i, vec);
        Four<P> low;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            W x = widen(px.x[e]);
            one((W)widen(gx.x[e]), mx.x[e], vx.x[e], x);
            px.x[e] = narrow<M>(x);
            low.x[e] = narrow<P>(x);
        }
        store4<true>(m + i, mx, vec);
        store4<true>(v + i, vx, vec);
        store4<!std::is_same_v<P, M>>(master + i, px, vec);
        if constexpr (!std::is_same_v<P, M>) store4<false>(p + i, low, vec);
    }
    for (int e = 0; e < 4; ++e)
        if (i + e < z) {
            W x = widen(master[i + e]);
            one((W)widen(g[i + e]), m[i + e], v[i + e], x);
            master[i + e] = narrow<M>(x);
            if constexpr (!std::is_same_v<P, M>) p[i + e] = narrow<P>(x);
        }
}

template <typename P>
__device__ void adamw_low(const AdamEntry &t, int64_t b, int64_t z, const AdamArgs &o,
                          double c) {
    if (t.master) {
        if (t.grad_type == SLA_F32) adamw<P, float, float>(t, b, z, o, c);
        else adamw<P, float, P>(t, b, z, o, c);
    } else {
        if (t.grad_type == SLA_F32) adamw<P, P, float>(t, b, z, o, c);
        else adamw<P, P, P>(t, b, z, o, c);
    }
}

__global__ __launch_bounds__(kThreads) void adamw_kernel(Table<AdamEntry> tb, const double *part,
                                                         int n, AdamArgs o, void *out, int type) {
    double c = 1.0;
    if (o.max_norm > 0.0) {
        const double norm = norm_of(part, n);
        if (out && blockIdx.x == 0 && threadIdx.x == 0) put_norm(out, type, norm);
        if (!isfinite(norm)) {  // counted by whoever has a tensor's first chunk
            for_pieces(tb, [&](const AdamEntry &t, int64_t b, int64_t) {
                if (b == 0 && t.skipped && threadIdx.x == 0) ++*t.skipped;
            });
            return;
        }
        c = clip_factor(norm, o.max_norm);
    }
    for_pieces(tb, [&](const AdamEntry &t, int64_t b, int64_t z) {
        set_rates(t, o);
        switch (t.param_type) {
            case SLA_F64: adamw<double, double, double>(t, b, z, o, c); break;
            case SLA_F32:
                if (t.grad_type == SLA_F32) adamw<float, float, float>(t, b, z, o, c);
                else if (t.grad_type == SLA_F16) adamw<float, float, __half>(t, b, z, o, c);
                else adamw<float, float, __hip_bfloat16>(t, b, z, o, c);
                break;
            case SLA_F16: adamw_low<__half>(t, b, z, o, c); break;
            default: adamw_low<__hip_bfloat16>(t, b, z, o, c);
        }
    });
}

bool known(int type) {
    return type == SLA_F64 || type == SLA_F32 || type == SLA_F16 || type == SLA_BF16;
}

sla_status check(const sla_tensor *t, int64_t count, bool grads_only) {
    if (count < 0 || (count > 0 && !t)) return SLA_ERR_ARG;
    int64_t chunks = 0;  // kernels count them in 32 bits
    for (int64_t i = 0; i < count; ++i) {
        const sla_tensor &x = t[i];
        if (x.n < 0 || x.n > (int64_t)kStepElems << 30 || !known(x.grad_type)) return SLA_ERR_ARG;
        chunks += (x.n + kStepElems - 1) / kStepElems;
        if (chunks > 0x7fffffff) return SLA_ERR_ARG;
        if (x.n > 0 && !x.grad) return SLA_ERR_ARG;
        if (grads_only) continue;
        const bool low = x.param_type == SLA_F16 || x.param_type == SLA_BF16;
        if (!known(x.param_type) || (x.master && !low) || x.step < 1) return SLA_ERR_ARG;
        if (x.param_type == SLA_F64 || x.grad_type == SLA_F64) {
            if (x.param_type != x.grad_type) return SLA_ERR_ARG;
        } else if (low && x.grad_type != SLA_F32 && x.grad_type != x.param_type) {
            return SLA_ERR_ARG;
        }
        if (x.n > 0 && (!x.param || !x.exp_avg || !x.exp_avg_sq)) return SLA_ERR_ARG;
    }
    return SLA_OK;
}

inline bool aligned(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Calls f(table, blocks) for the list's non-empty tensors, a table at a time;
// fill(entry, tensor) sets what the chunks do not.
template <typename E, typename Fill, typename F>
hipError_t for_tables(const sla_tensor *t, int64_t count, int elems, int most, Fill &&fill, F &&f) {
    Table<E> tb;
    tb.count = tb.chunks = 0, tb.elems = elems;
    auto flush = [&]() -> hipError_t {
        if (tb.count == 0) return hipSuccess;
        const int blocks = tb.chunks < most ? tb.chunks : most;
        const hipError_t e = f(tb, blocks);
        tb.count = tb.chunks = 0;
        return e;
    };
    for (int64_t i = 0; i < count; ++i) {
        if (t[i].n == 0) continue;
        const int64_t chunks = (t[i].n + tb.elems - 1) / tb.elems;
        if (tb.count == Table<E>::kMost) {
            const hipError_t e = flush();
            if (e != hipSuccess) return e;
        }
        E &x = tb.e[tb.count++];
        x.n = t[i].n;
        x.grad = t[i].grad;
        x.grad_type = (uint8_t)t[i].grad_type;
        x.first = tb.chunks;
        fill(x, t[i]);
        tb.chunks += (int32_t)chunks;
    }
    return flush();
}

void fill_grad(GradEntry &x, const sla_tensor &t) { x.vec = aligned(t.grad); }

// The partial sums of the whole list: *n of them at *part.
hipError_t square_sums(const sla_tensor *t, int64_t count, double *work, const double **part,
                       int *n, hipStream_t s) {
    *n = 0;
    *part = work + 1;
    hipError_t e = for_tables<GradEntry>(
        t, count, kGradElems, kMaxSums, fill_grad, [&](const Table<GradEntry> &tb, int blocks) {
            square_sum_kernel<<<blocks, kThreads, 0, s>>>(tb, work + 1 + *n);
            *n += blocks;
            return hipGetLastError();
        });
    if (e != hipSuccess || *n <= kDirect) return e;
    total_kernel<<<1, kThreads, 0, s>>>(*part, *n, work);
    *part = work;
    *n = 1;
    return hipGetLastError();
}

hipError_t finish(const double *part, int n, void *d_norm, int type, hipStream_t s) {
    norm_kernel<<<1, kThreads, 0, s>>>(part, n, d_norm, type);
    return hipGetLastError();
}

bool norm_type_ok(int type) { return type == SLA_F32 || type == SLA_F64; }

}  // namespace

}  // namespace sla

using namespace sla;

#define TRAIN_TRY(...)                 \
    do {                               \
        hipError_t e_ = (__VA_ARGS__); \
        if (e_ != hipSuccess) {        \
            set_last_error(e_);        \
            return SLA_ERR_DEVICE;     \
        }                              \
    } while (0)

extern "C" {

int64_t sla_grad_workspace_bytes(int64_t count) {
    if (count <= 0) return count < 0 ? -1 : 0;
    return 8 + 8 * kMaxSums * ((count + Table<GradEntry>::kMost - 1) / Table<GradEntry>::kMost);
}

sla_status sla_grad_norm(const sla_tensor *tensors, int64_t count, void *d_norm,
                         int32_t norm_type, void *d_work, void *stream) {
    if (check(tensors, count, true) != SLA_OK || !d_norm || !norm_type_ok(norm_type))
        return SLA_ERR_ARG;
    if (count > 0 && !d_work) return SLA_ERR_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const double *part;
    int n;
    TRAIN_TRY(square_sums(tensors, count, static_cast<double *>(d_work), &part, &n, s));
    TRAIN_TRY(finish(part, n, d_norm, norm_type, s));
    return SLA_OK;
}

sla_status sla_clip_grads(const sla_tensor *tensors, int64_t count, double max_norm,
                          void *d_norm, int32_t norm_type, void *d_work, void *stream) {
    if (check(tensors, count, true) != SLA_OK || !d_norm || !norm_type_ok(norm_type) ||
        !(max_norm >= 0.0))
        return SLA_ERR_ARG;
    if (count > 0 && !d_work) return SLA_ERR_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const double *part;
    int n;
    TRAIN_TRY(square_sums(tensors, count, static_cast<double *>(d_work), &part, &n, s));
    if (n == 0) {
        TRAIN_TRY(finish(part, 0, d_norm, norm_type, s));
        return SLA_OK;
    }
    void *out = d_norm;
    TRAIN_TRY(for_tables<GradEntry>(tensors, count, kGradElems, kMaxBlocks, fill_grad, [&](const Table<GradEntry> &tb, int blocks) {
        clip_kernel<<<blocks, kThreads, 0, s>>>(tb, part, n, max_norm, out, norm_type);
        out = nullptr;  // the first launch wrote it
        return hipGetLastError();
    }));
    return SLA_OK;
}

sla_status sla_adamw(const sla_tensor *tensors, int64_t count, const sla_adamw_opts *opts,
                     void *d_norm, int32_t norm_type, void *d_work, void *stream) {
    if (check(tensors, count, false) != SLA_OK || !opts) return SLA_ERR_ARG;
    const sla_adamw_opts &q = *opts;
    if (!(q.beta_one >= 0.0 && q.beta_one < 1.0) ||
        !(q.beta_two >= 0.0 && q.beta_two < 1.0) || !(q.eps >= 0.0) || !std::isfinite(q.lr) ||
        !std::isfinite(q.weight_decay) || !(q.max_norm >= 0.0))
        return SLA_ERR_ARG;
    const bool clip = q.max_norm > 0.0;
    if (clip && (!d_norm || !norm_type_ok(norm_type) || (count > 0 && !d_work))) return SLA_ERR_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    AdamArgs o;
    o.lr = q.lr, o.b1 = q.beta_one, o.b2 = q.beta_two, o.eps = q.eps;
    o.keep = 1.0 - q.lr * q.weight_decay;
    o.max_norm = q.max_norm;
    const double *part = nullptr;
    int n = 0;
    void *out = d_norm;
    if (clip) {
        TRAIN_TRY(square_sums(tensors, count, static_cast<double *>(d_work), &part, &n, s));
        if (n == 0) TRAIN_TRY(finish(part, 0, d_norm, norm_type, s));
    }
    int64_t step = 0;
    double rate = 0.0, root = 0.0;
    auto fill = [&](AdamEntry &x, const sla_tensor &t) {
        if (t.step != step) {
            step = t.step;
            rate = q.lr / (1.0 - std::pow(q.beta_one, (double)step));
            root = 1.0 / std::sqrt(1.0 - std::pow(q.beta_two, (double)step));
        }
        x.param = t.param, x.exp_avg = t.exp_avg, x.exp_avg_sq = t.exp_avg_sq;
        x.master = t.master;
        x.param_type = (uint8_t)t.param_type;
        x.rate = rate, x.root = root, x.step = step, x.skipped = t.d_skipped;
        x.vec = aligned(t.grad) && aligned(t.param) && aligned(t.exp_avg) &&
                aligned(t.exp_avg_sq) && aligned(t.master);
    };
    TRAIN_TRY(for_tables<AdamEntry>(tensors, count, kStepElems, kMaxBlocks, fill, [&](const Table<AdamEntry> &tb, int blocks) {
        adamw_kernel<<<blocks, kThreads, 0, s>>>(tb, part, n, o, out, norm_type);
        out = nullptr;
        return hipGetLastError();
    }));
    return SLA_OK;
}

}  // extern "C"
