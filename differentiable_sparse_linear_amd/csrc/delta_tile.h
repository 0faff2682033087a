// Matrix tiles of the chunked gated delta rule.
//
// All products run on v_mfma_f32_16x16x32_bf16 and are still exact to about
// 24 bits: a value x is held as bf16 planes x = x0 + x1 + x2 of 8 bits each
// (one plane holds a bf16 input exactly, two an fp16 input, three an fp32
// value), and a product keeps the plane pairs (i, j) with i + j <= 2, the
// smaller first.  Six such products cost 6/16 of the fp32 matrix
// instructions' time, three (an exact bf16 input against fp32) 3/16.
//
// Layouts, with lane l = 16 g + c of a wavefront:
//   accumulator tile  element (row 4 g + r, column c) in register r
//   operand fragment  8 bf16: row c of A (or column c of B) at the
//                     contraction indexes 4 g + {0..3} and 16 + 4 g + {0..3}
// The fragment's order of the contraction is chosen so that two accumulator
// tiles, one over the other, are after rounding a fragment of B as they
// stand: results feed the next product without leaving their lane.
#pragma once

#include <type_traits>

#include "delta.h"

namespace sla {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <typename T>
struct Planes;  // bf16 planes that hold a T exactly
template <>
struct Planes<__hip_bfloat16> { static constexpr int n = 1; };
template <>
struct Planes<__half> { static constexpr int n = 2; };
template <>
struct Planes<float> { static constexpr int n = 3; };

template <int N>
struct Frag {
    u32x4 p[N];
};

// The leading N planes of a pair.  A remainder a - bf16(a) is exact in fp32,
// and one two-term bf16 dot product takes it off the packed pair as it is.
template <int N>
__device__ inline void split_pair(float a, float b, uint32_t (&out)[N]) {
    // (-1, 0) and (0, -1) as register values: an inline constant stands for
    // another pair
    uint32_t minus_first = 0x0000bf80u, minus_second = 0xbf800000u;
    asm("" : "+s"(minus_first));
    asm("" : "+s"(minus_second));
    const bf16x2 first = __builtin_bit_cast(bf16x2, minus_first),
                 second = __builtin_bit_cast(bf16x2, minus_second);
#pragma unroll
    for (int p = 0; p < N; ++p) {
        const bf16x2 y = {(__bf16)a, (__bf16)b};
        out[p] = __builtin_bit_cast(uint32_t, y);
        if (p + 1 < N) {
            a = __builtin_amdgcn_fdot2_f32_bf16(y, first, a, false);
            b = __builtin_amdgcn_fdot2_f32_bf16(y, second, b, false);
        }
    }
}

template <int N>
__device__ inline Frag<N> split(const float (&x)[8]) {
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t y[N];
        split_pair<N>(x[2 * i], x[2 * i + 1], y);
#pragma unroll
        for (int p = 0; p < N; ++p) f.p[p][i] = y[p];
    }
    return f;
}

template <int N>
__device__ inline Frag<N> split(const f32x4 &lo, const f32x4 &hi) {
    const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return split<N>(x);
}

__device__ inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// c + a b, the plane pairs (i, j) with i + j <= 2: 24 bits.
template <int NA, int NB>
__device__ inline f32x4 mac(const Frag<NA> &a, const Frag<NB> &b, f32x4 c) {
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) c = mfma(a.p[i], b.p[s - i], c);
    return c;
}

// c0 + a0 b0 and c1 + a1 b1, their steps in turn: a step waits for the one
// before it in its own sum.
template <int NA, int NB>
__device__ inline void mac_pair(const Frag<NA> &a0, const Frag<NB> &b0, f32x4 &c0,
                                const Frag<NA> &a1, const Frag<NB> &b1, f32x4 &c1) {
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) {
                c0 = mfma(a0.p[i], b0.p[s - i], c0);
                c1 = mfma(a1.p[i], b1.p[s - i], c1);
            }
}

// Buffers: addresses are a descriptor, a lane's offset and constants, and
// what lies at or past `bytes` reads as 0 and is not written.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ inline Buffer buffer(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, bytes, 0x00027000);
}
constexpr uint32_t kNowhere = 0x80000000u;  // a lane offset that no buffer reaches

// 16 bytes at lane + at; `at` a constant within the buffer, whose multiple of
// 4096 rides in a scalar register.
__device__ inline u32x4 load16(Buffer b, uint32_t lane, uint32_t at) {
    return __builtin_amdgcn_raw_buffer_load_b128(b, lane + (at & 4095u), at & ~4095u, 0);
}
// A store keeps its offset in the vector register alone.  An instruction after a
// store of 16 bytes may overwrite its data before all of it is taken; the
// compiler puts a wait state between unless a scalar register holds part of the
// offset, which it takes to make up for it, and here it did not: the last
// lanes of fragments were an address computed next, where several workgroups
// shared a CU.
__device__ inline void store16(u32x4 x, Buffer b, uint32_t lane, uint32_t at) {
    __builtin_amdgcn_raw_buffer_store_b128(x, b, lane + at, 0, 0);
}
// The same for what is read much later: not kept in the caches.
__device__ inline void store16_later(u32x4 x, Buffer b, uint32_t lane, uint32_t at) {
    __builtin_amdgcn_raw_buffer_store_b128(x, b, lane + at, 0, 2);
}
template <typename T>
__device__ inline T load_one(Buffer b, uint32_t at) {
    if constexpr (sizeof(T) == 4)
        return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(b, at, 0, 0));
    else
        return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(b, at, 0, 0));
}
template <typename T>
__device__ inline void store_one(T x, Buffer b, uint32_t at) {
    if constexpr (sizeof(T) == 4)
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), b, at, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, x), b, at, 0, 0);
}

// 64 rows of a strided array: element (token, column) of a chunk's first
// `rows` tokens, whose stride is at most kMaxStride.  A lane keeps the offsets
// of its rows 4 g + {0..3} and adds a multiple of the stride for a row tile.
// (Not as the buffer instruction's scalar offset: that is taken off the
// buffer's length unchecked, and may be more than it here.)
constexpr int64_t kMaxStride = 1 << 22;
template <typename T>
struct Rows {
    uint32_t lane[4], tile;
    __device__ void set(int64_t stride, int g, int col, bool in) {
        tile = 16 * (uint32_t)stride * sizeof(T);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            lane[r] = in ? ((4 * g + r) * (uint32_t)stride + col) * sizeof(T) : kNowhere;
    }
    // the rows of one chunk: those at and past `rows` are out of reach
    static __device__ Buffer chunk(const T *first, int64_t stride, int rows) {
        return buffer(first, (rows < kChunk ? rows : kChunk) * (uint32_t)stride * sizeof(T));
    }
    __device__ T load(Buffer b, int it, int r, int m = 0) const {
        return load_one<T>(b, lane[r] + it * tile + 16 * m * sizeof(T));
    }
    __device__ void store(T x, Buffer b, int it, int r, int m = 0) const {
        store_one<T>(x, b, lane[r] + it * tile + 16 * m * sizeof(T));
    }
};

// 8 values of row `x` at d0 + {0..3} and d0 + 16 + {0..3}, 0 past `n` and
// where the row is not live.  vec: rows start at 4-element boundaries and n
// is a multiple of 4.
template <typename T>
__device__ inline void load8(const T *x, int d0, int n, bool live, bool vec, float (&out)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int d = d0 + 16 * h;
        if (vec) {
            T y[4] = {};
            if (live && d < n) {
                if constexpr (sizeof(T) == 4)
                    *reinterpret_cast<float4 *>(y) = *reinterpret_cast<const float4 *>(x + d);
                else
                    *reinterpret_cast<uint2 *>(y) = *reinterpret_cast<const uint2 *>(x + d);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) out[4 * h + e] = to_f32<T>(y[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                out[4 * h + e] = live && d + e < n ? to_f32<T>(x[d + e]) : 0.f;
        }
    }
}

// load8 as a fragment.
template <typename T>
__device__ inline Frag<Planes<T>::n> load_frag(const T *x, int d0, int n, bool live, bool vec) {
    if constexpr (Planes<T>::n == 1) {
        if (vec) {  // the values are the plane
            uint2 lo = make_uint2(0u, 0u), hi = lo;
            if (live && d0 < n) lo = *reinterpret_cast<const uint2 *>(x + d0);
            if (live && d0 + 16 < n) hi = *reinterpret_cast<const uint2 *>(x + d0 + 16);
            Frag<1> f;
            f.p[0] = u32x4{lo.x, lo.y, hi.x, hi.y};
            return f;
        }
    }
    float y[8];
    load8<T>(x, d0, n, live, vec, y);
    return split<Planes<T>::n>(y);
}

// Values 4 half + {0..3} of a fragment.
template <int N>
__device__ inline f32x4 values(const Frag<N> &f, int half) {
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = N - 1; p >= 0; --p) {
        const uint32_t lo = half ? f.p[p][2] : f.p[p][0], hi = half ? f.p[p][3] : f.p[p][1];
        y[0] += __uint_as_float(lo << 16);
        y[1] += __uint_as_float(lo & 0xffff0000u);
        y[2] += __uint_as_float(hi << 16);
        y[3] += __uint_as_float(hi & 0xffff0000u);
    }
    return y;
}

// exp of a difference of gate sums, which are kept in units of log 2: one
// rounding of the difference and one instruction.
constexpr double kLog2e = 1.4426950408889634;
__device__ inline float decay(double x) { return __builtin_amdgcn_exp2f((float)x); }

// Planes in LDS, by tiles of 16 x 16 that are written as accumulator tiles
// stand (column c, rows 4 g + {0..3} in one 8-byte access) and read back
// transposed by ds_read_b64_tr_b16: lane (g, c) gets row c at columns
// 4 g + {0..3}, half an operand fragment whose contraction runs over the
// columns.
constexpr int kTileBytes = 512;
typedef short s16x4 __attribute__((ext_vector_type(4)));
template <int N>
__device__ inline void put_tile(unsigned char *lds, int plane_stride, const f32x4 &x, int g, int c) {
    uint32_t lo[N], hi[N];
    split_pair<N>(x[0], x[1], lo);
    split_pair<N>(x[2], x[3], hi);
#pragma unroll
    for (int p = 0; p < N; ++p)
        *reinterpret_cast<uint2 *>(lds + p * plane_stride + 32 * c + 8 * g) = make_uint2(lo[p], hi[p]);
}
// The fragment over two tiles' columns (tiles `next` bytes apart).
template <int N>
__device__ inline Frag<N> get_transposed(const unsigned char *lds, int plane_stride, int next, int l) {
    Frag<N> f;
#pragma unroll
    for (int p = 0; p < N; ++p)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            typedef __attribute__((address_space(3))) s16x4 *LdsPtr;
            const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (LdsPtr)(lds + p * plane_stride + e * next + 8 * l));
            const uint2 u = __builtin_bit_cast(uint2, y);
            f.p[p][2 * e] = u.x;
            f.p[p][2 * e + 1] = u.y;
        }
    return f;
}

// The operand fragments of a chunk, in the order in which a wavefront uses
// them, held in registers D ahead of their use.  Positions are compile-time
// constants once the chunk's loops are unrolled; N is their number, rounded up
// to a multiple of D.
template <int N, int D>
struct Ring {
    static_assert(N % D == 0, "a chunk takes whole turns of the ring");
    u32x4 x[D];
    template <typename F>
    __device__ void fill(F &&fetch) {
#pragma unroll
        for (int j = 0; j < D; ++j) x[j] = fetch(j, false);
    }
    __device__ u32x4 at(int j) const { return x[j % D]; }
    // After the last use of the N positions from j: fetches those D further on
    // (of the next chunk where that is past the end) in their place.  (Fetched
    // before that use they would stand in other registers, and copying them into
    // these at the loop's end would wait for all of them.)
    template <typename F>
    __device__ void next(int j, int n, F &&fetch) {
        __builtin_amdgcn_sched_barrier(0x0386);  // products stay on their side, LDS may pass
#pragma unroll
        for (int i = j; i < j + n; ++i)
            x[i % D] = i + D < N ? fetch(i + D, false) : fetch(i + D - N, true);
        __builtin_amdgcn_sched_barrier(0x000f);  // arithmetic may pass, loads stay here
    }
};

// Values {0..3} and 16 + {0..3} from a lane's offset in a buffer as a fragment; 0
// where fewer than that are `left` (or where the buffer ends).  vec: offsets and
// `left` are multiples of four elements.
template <typename T>
__device__ inline Frag<Planes<T>::n> row_frag(Buffer b, uint32_t at, int left, bool vec) {
    T x[8];
    if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t from = 16 * h < left ? at + 16 * h * sizeof(T) : kNowhere;
            if constexpr (sizeof(T) == 4) {
                const u32x4 y = __builtin_amdgcn_raw_buffer_load_b128(b, from, 0, 0);
                __builtin_memcpy(x + 4 * h, &y, sizeof(y));
            } else {
                const auto y = __builtin_amdgcn_raw_buffer_load_b64(b, from, 0, 0);
                __builtin_memcpy(x + 4 * h, &y, sizeof(y));
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int d = 16 * (e >> 2) + (e & 3);
            x[e] = load_one<T>(b, d < left ? at + d * sizeof(T) : kNowhere);
        }
    }
    if constexpr (Planes<T>::n == 1) {  // the values are the plane
        Frag<1> f;
        __builtin_memcpy(&f.p[0], x, sizeof(x));
        return f;
    } else {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = to_f32<T>(x[e]);
        return split<Planes<T>::n>(y);
    }
}

// The sum over the 16 lanes that share g, in each of them.
__device__ inline float sum16(float x) {
    auto add = [&](auto ror) {
        x += __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(x),
                                                         0x120 + decltype(ror)::value, 0xf, 0xf, false));
    };
    add(std::integral_constant<int, 8>{});
    add(std::integral_constant<int, 4>{});
    add(std::integral_constant<int, 2>{});
    add(std::integral_constant<int, 1>{});
    return x;
}

// A barrier for exchanges through LDS: what was put there is there, what was
// read is in registers.  Unlike __syncthreads() it orders LDS alone, so it does
// not wait for loads that run ahead, nor for stores.
__device__ inline void exchange() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Tiles of the lower triangle of a 64 x 64 matrix as A operand (row tile i,
// contraction block kb <= i / 2), and of the upper one (kb >= i / 2).
constexpr int kTriTiles = 6;
__host__ __device__ constexpr int lower_tile(int i, int kb) { return i + (i == 3 ? 1 : 0) + kb; }
__host__ __device__ constexpr int upper_tile(int i, int kb) {
    return i < 2 ? 2 * i + kb : 2 + i;
}

// Gates of a chunk, one token a lane: the running sum in 64 bits and units of
// log 2 (differences keep 32 bits whatever was summed before them); NaN where
// the gates of a run of tokens sum to more than kMaxGrowth.
__device__ inline double gate_sum(float gate, int lane) {
    double x = (gate < kMinGate ? kMinGate : gate) * kLog2e;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const double y = __shfl_up(x, off, 64);
        if (lane >= off) x += y;
    }
    float low = fminf((float)x, 0.f);  // the least sum up to here
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const float y = __shfl_up(low, off, 64);
        if (lane >= off) low = fminf(low, y);
    }
    const bool grows = (float)x - low > (float)(kMaxGrowth * kLog2e);
    return __any(grows) ? (double)__builtin_nanf("") : x;
}

// What the preparation of a chunk leaves for the scans and the gradients, in
// fragments of 1 KB.  Everything is padded with zeros to whole tiles (keys to
// DK, tokens to 64).  K and Q: [DK / 32][4 row tiles][planes]; K^T and Q^T:
// [planes][DK / 16][2]; a triangle: [3 planes][kTriTiles].
template <int NP, int DK>
struct PrepLayout {
    static constexpr int kKey = NP * 4 * (DK / 32) * 64 * 16;    // K or Q, rows tokens
    static constexpr int kKeyT = NP * (DK / 16) * 2 * 64 * 16;   // K^T or Q^T, rows keys
    static constexpr int kTri = 3 * kTriTiles * 64 * 16;         // a triangle's planes
    static constexpr int kScalars = 3 * 64 * 4;                  // since, until, beta
    // per chunk and key head; the third is Q (forward) or Q^T (backward)
    static constexpr int kPerKeyHead = kKey + 2 * kKeyT;
    static constexpr int kPerHead = 2 * kTri + kScalars;
};

}  // namespace sla
