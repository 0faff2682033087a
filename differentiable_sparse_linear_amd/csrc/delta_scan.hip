// The scans of the chunked gated delta rule: one chunk after another, forward
// and back.
//
// A workgroup carries 16 NC columns of one head's state.  Four wavefronts
// divide the rows: wavefront w has a quarter of the keys (tiles of the state)
// and the w-th 16 tokens of every chunk (tiles of R and W), so it needs only its
// rows of the operands, which it loads a chunk ahead into registers.  What all
// rows need, the state, R and W as planes, goes through LDS: three barriers a
// chunk.  The tiles stand in LDS as operand fragments, so writing one is its
// lane's own 8 bytes a plane.  Forward, four more wavefronts form the output from
// the same planes, beside the chain of products that carries the state.
//
// Bound by that chain: 1.4 us a chunk with 16 columns (bf16, 128 keys, 16 heads,
// half of the CUs at work), 1.6 with 64 keys and what the gradients need; 2.9 with
// one wavefront a workgroup and nothing exchanged, which alone on a SIMD issues
// one instruction in four cycles.  64 heads, 32 columns: 2.7 us a chunk, 4.0 with
// what the gradients need, 96 KB a chunk and head, stored at 1.6 TB/s; back 4.4.
// The output's products in 24 bits instead of 16 are 0.1 us of a chunk, with 64
// keys 0.2.
#include <type_traits>

#include "delta_chunk.h"

namespace sla {

namespace {

// The workgroup's head and part of its columns: all workgroups of a head on
// one XCD (workgroups go to the XCDs in turn), whose L2 then holds one copy of
// what they share.
__device__ inline bool head_and_part(const DeltaArgs &a, int &b, int &h, int &part) {
    const int heads = a.B * a.Hv, stride = (heads + 7) & ~7;
    const int head = blockIdx.x % stride;
    part = blockIdx.x / stride;
    b = head / a.Hv, h = head % a.Hv;
    return head < heads;
}

// Chunks of this round that have tokens.
__device__ inline int live_chunks(const ChunkRange &cr, int len) {
    const int n = (len + kChunk - 1) / kChunk - cr.first;
    return n < 0 ? 0 : n > cr.count ? cr.count : n;
}

// exp(G_C), the last of the chunk's `since`.  One word: registers of a wider load
// that nobody reads would be used for something else, after a wait for it.
template <typename L>
__device__ inline u32x4 load_whole(Buffer head) {
    return u32x4{load_one<uint32_t>(head, 2 * L::kTri + 252), 0u, 0u, 0u};
}

// A matrix of 32 K rows and 16 columns in LDS, as the planes of its fragments
// for a B operand: [N planes][K][64 lanes].
template <int N, int K>
struct Shared {
    u32x4 x[N * K * 64];
    // rows 16 tile + ..., from an accumulator tile
    __device__ void put(int tile, const f32x4 &y, int l) {
        uint32_t lo[N], hi[N];
        split_pair<N>(y[0], y[1], lo);
        split_pair<N>(y[2], y[3], hi);
#pragma unroll
        for (int p = 0; p < N; ++p)
            reinterpret_cast<uint2 *>(&x[(p * K + (tile >> 1)) * 64 + l])[tile & 1] =
                make_uint2(lo[p], hi[p]);
    }
    __device__ Frag<N> get(int kb, int l) const {
        Frag<N> f;
#pragma unroll
        for (int p = 0; p < N; ++p) f.p[p] = x[(p * K + kb) * 64 + l];
        return f;
    }
};

// A wavefront's fragments of a chunk, in the order of their use.
template <int NP, int DK>
struct StateOrder {
    static constexpr int KB = DK / 32, TW = DK / 64;       // TW: state tiles of a wavefront
    static constexpr int kSince = KB * NP, kX = kSince + 1, kEnd = kX + 6, kKT = kEnd + 2,
                         kTotal = kKT + TW * 2 * NP;
    static constexpr int D = NP == 3 ? (kTotal + 1) / 2 : kTotal, N = (kTotal + D - 1) / D * D;
};
template <int NP, int DK>
struct OutputOrder {
    static constexpr int KB = DK / 32;
    static constexpr int kSince = KB * NP, kP = kSince + 1, kTotal = kP + 6;
    static constexpr int D = kTotal, N = kTotal;
};

template <typename T, int DK, int NC, bool SAVE>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void
delta_scan_kernel(DeltaArgs a, ChunkRange cr, const unsigned char *ws_key,
                  const unsigned char *ws_head, const float *s_in, float *s_out, T *o, int64_t ob,
                  int64_t ot, int64_t oh, float *save_s, float *save_w) {
    constexpr int NP = Planes<T>::n;
    using L = PrepLayout<NP, DK>;
    using Y = OutputOrder<NP, DK>;
    using Z = StateOrder<NP, DK>;
    constexpr int KB = Z::KB, TW = Z::TW, KT = DK / 16;
    __shared__ Shared<3, KB> Sx[NC];   // S
    __shared__ Shared<3, 2> Rx[NC];    // R
    __shared__ Shared<3, 2> Ux[NC];    // until beta W
    __shared__ Shared<3, 2> Wx[NC];    // W, for the output
    int b, h, part;
    if (!head_and_part(a, b, h, part)) return;
    const int hk = h / (a.Hv / a.Hk), len = seq_len(a, b), live = live_chunks(cr, len);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave & 3,
              l = threadIdx.x & 63, g = l >> 4, c = l & 15, col0 = kSlice * NC * part,
              dvp = padded_dv(a.dv);
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const uint32_t lane16 = 16 * l;
    using Inputs = std::integral_constant<int, NP>;
    using Three = std::integral_constant<int, 3>;

    // this chunk's workspace and the next one's; a head's chunks follow one another
    const unsigned char *key_at = ws_key + cr.key_chunk(a, b, hk, 0) * L::kPerKeyHead,
                        *head_at = ws_head + cr.chunk(a, b, h, 0) * L::kPerHead;
    Buffer key0 = buffer(key_at, L::kPerKeyHead), key1 = key0,
           head0 = buffer(head_at, L::kPerHead), head1 = head0;
    auto advance = [&](int i) {  // after the last chunk: read again, not used
        if (i + 1 < live) {
            key_at += L::kPerKeyHead;
            head_at += L::kPerHead;
        }
        key1 = buffer(key_at, L::kPerKeyHead), head1 = buffer(head_at, L::kPerHead);
    };
    // this wavefront's rows: of K and Q, of a triangle, of K^T, of the scalars.
    // Rows of a triangle's first two tiles end with the first block: what is
    // read in place of the second is not used.
    const uint32_t k_lane = lane16 + w * NP * 1024, x_lane = lane16 + lower_tile(w, 0) * 1024,
                   kt_lane = lane16 + w * TW * 2048, s_lane = 16 * g + 64 * w;
    auto rows_of_key = [&](Buffer key, int base, int j) {
        return load16(key, k_lane, base + (j / NP * 4 * NP + j % NP) * 1024);
    };

    // o = scale (Gamma Q S + P' W), to 24 bits for every type: the two parts cancel
    // where a token reads what it has just corrected
    if (wave >= 4) {
        T *oc = o + b * ob + h * oh + col0;
        Rows<T> o_rows[NC];  // of this wavefront's tokens; lanes past the columns reach nothing
#pragma unroll
        for (int m = 0; m < NC; ++m) o_rows[m].set(ot, 4 * w + g, c, col0 + 16 * m + c < a.dv);
        auto fetch = [&](int j, bool next) -> u32x4 {
            const Buffer key = next ? key1 : key0, head = next ? head1 : head0;
            if (j < Y::kSince) return rows_of_key(key, L::kKey + L::kKeyT, j);
            if (j == Y::kSince) return load16(head, s_lane, 2 * L::kTri);
            return load16(head, x_lane,
                          L::kTri + ((j - Y::kP) % 3 * kTriTiles + (j - Y::kP) / 3) * 1024);
        };
        Ring<Y::N, Y::D> ring;
        auto frag = [&](auto n, int j) {
            Frag<decltype(n)::value> f;
#pragma unroll
            for (int p = 0; p < decltype(n)::value; ++p) f.p[p] = ring.at(j + p);
            return f;
        };
        if (live > 0) ring.fill(fetch);
        for (int i = 0; i < live; ++i) {
            const int t0 = (cr.first + i) * kChunk;
            advance(i);
            f32x4 O[NC];
#pragma unroll
            for (int m = 0; m < NC; ++m) O[m] = zero;
            exchange();  // S is there
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const Frag<NP> q = frag(Inputs{}, kb * NP);
#pragma unroll
                for (int m = 0; m < NC; ++m) O[m] = mac(q, Sx[m].get(kb, l), O[m]);
                ring.next(kb * NP, NP, fetch);
            }
            const f32x4 since = __builtin_bit_cast(f32x4, ring.at(Y::kSince));
#pragma unroll
            for (int m = 0; m < NC; ++m) O[m] *= since;
            ring.next(Y::kSince, 1, fetch);
            exchange();
            exchange();  // W is there
            const Frag<3> p0 = frag(Three{}, Y::kP), p1 = frag(Three{}, Y::kP + 3);
            const Buffer dst = Rows<T>::chunk(oc + t0 * ot, ot, a.T - t0);
#pragma unroll
            for (int m = 0; m < NC; ++m) {
                O[m] = mac(p0, Wx[m].get(0, l), O[m]);
                if (w >= 2) O[m] = mac(p1, Wx[m].get(1, l), O[m]);
            }
            ring.next(Y::kP, 6, fetch);
#pragma unroll
            for (int m = 0; m < NC; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool past = t0 + 16 * w + 4 * g + r >= len;  // answers 0
                    o_rows[m].store(from_f32<T>(past ? 0.f : a.scale * O[m][r]), dst, 0, r, m);
                }
            key0 = key1, head0 = head1;
        }
        for (int t = (cr.first + live) * kChunk + 4 * w + g;
             t < a.T && t < (cr.first + cr.count) * kChunk; t += 16)
#pragma unroll
            for (int m = 0; m < NC; ++m)
                if (t >= len && col0 + 16 * m + c < a.dv) oc[t * ot + 16 * m + c] = from_f32<T>(0.f);
        return;
    }

    f32x4 S[TW][NC];  // rows 16 (TW w + t) + 4 g + r
    const int64_t state = (int64_t)(b * a.Hv + h) * a.dk;
#pragma unroll
    for (int t = 0; t < TW; ++t)
#pragma unroll
        for (int m = 0; m < NC; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * (TW * w + t) + 4 * g + r, col = col0 + 16 * m + c;
                S[t][m][r] = s_in && col < a.dv && row < a.dk ? s_in[(state + row) * a.dv + col]
                                                              : 0.f;
            }
    const T *v = reinterpret_cast<const T *>(a.v) + b * a.vb + h * a.vh + col0;
    Rows<T> v_rows[NC];
#pragma unroll
    for (int m = 0; m < NC; ++m) v_rows[m].set(a.vt, 4 * w + g, c, col0 + 16 * m + c < a.dv);
    auto keep = [&](int n) {  // this wavefront's tiles of the state
#pragma unroll
        for (int m = 0; m < NC; ++m) {
            if (col0 + 16 * m >= dvp) break;
            const Buffer dst = buffer(save_s + (saved_chunk(a, b, h, n) * dvp + col0 + 16 * m) * DK,
                                      DK * kSlice * 4);
#pragma unroll
            for (int t = 0; t < TW; ++t)
                store16_later(__builtin_bit_cast(u32x4, S[t][m]), dst, lane16 + 1024 * TW * w, 1024 * t);
        }
    };
    auto fetch = [&](int j, bool next) -> u32x4 {
        const Buffer key = next ? key1 : key0, head = next ? head1 : head0;
        if (j < Z::kSince) return rows_of_key(key, 0, j);
        if (j == Z::kSince) return load16(head, s_lane, 2 * L::kTri);
        if (j < Z::kEnd) return load16(head, x_lane, ((j - Z::kX) % 3 * kTriTiles + (j - Z::kX) / 3) * 1024);
        if (j == Z::kEnd) return load16(head, s_lane, 2 * L::kTri + 256);
        if (j == Z::kEnd + 1) return load_whole<L>(head);
        if (j < Z::kTotal)
            return load16(key, kt_lane,
                          L::kKey + ((j - Z::kKT) % NP * KT * 2 + (j - Z::kKT) / NP) * 1024);
        return u32x4{0u, 0u, 0u, 0u};
    };
    T vt[NC][4];
    auto fetch_v = [&](int i) {
        const int t0 = (cr.first + i) * kChunk;
        const Buffer src = Rows<T>::chunk(v + t0 * a.vt, a.vt, len - t0);
#pragma unroll
        for (int m = 0; m < NC; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) vt[m][r] = v_rows[m].load(src, 0, r, m);
    };
    auto put_state = [&]() {
#pragma unroll
        for (int t = 0; t < TW; ++t)
#pragma unroll
            for (int m = 0; m < NC; ++m) Sx[m].put(TW * w + t, S[t][m], l);
    };
    Ring<Z::N, Z::D> ring;
    auto frag = [&](auto n, int j) {
        Frag<decltype(n)::value> f;
#pragma unroll
        for (int p = 0; p < decltype(n)::value; ++p) f.p[p] = ring.at(j + p);
        return f;
    };
    if (live > 0) {
        // in the loop's order: waits count the loads that were issued since
        fetch_v(0);
        ring.fill(fetch);
        put_state();
    }
    for (int i = 0; i < live; ++i) {
        const int n = cr.first + i;
        advance(i);
        if (SAVE) keep(n);
        exchange();
        // R = V - Gamma K S (in two sums, since a sum's products wait for one another)
        f32x4 R[NC], R2[NC], W[NC];
#pragma unroll
        for (int m = 0; m < NC; ++m) R[m] = R2[m] = W[m] = zero;
#pragma unroll
        for (int kb = 0; kb < KB; kb += 2) {
            const Frag<NP> k0 = frag(Inputs{}, kb * NP), k1 = frag(Inputs{}, (kb + 1) * NP);
#pragma unroll
            for (int m = 0; m < NC; ++m)
                mac_pair(k0, Sx[m].get(kb, l), R[m], k1, Sx[m].get(kb + 1, l), R2[m]);
            ring.next(kb * NP, 2 * NP, fetch);
        }
        const f32x4 since = __builtin_bit_cast(f32x4, ring.at(Z::kSince));
#pragma unroll
        for (int m = 0; m < NC; ++m) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                R[m][r] = to_f32<T>(vt[m][r]) - since[r] * (R[m][r] + R2[m][r]);
            Rx[m].put(w, R[m], l);
        }
        ring.next(Z::kSince, 1, fetch);
        if (i + 1 < live) fetch_v(i + 1);
        exchange();
        // W = X R
        const Frag<3> x0 = frag(Three{}, Z::kX), x1 = frag(Three{}, Z::kX + 3);
#pragma unroll
        for (int m = 0; m < NC; ++m) {
            if (w >= 2) {
                f32x4 y = zero;
                mac_pair(x0, Rx[m].get(0, l), W[m], x1, Rx[m].get(1, l), y);
                W[m] += y;
            } else {
                W[m] = mac(x0, Rx[m].get(0, l), W[m]);
            }
        }
        ring.next(Z::kX, 6, fetch);
        const f32x4 end = __builtin_bit_cast(f32x4, ring.at(Z::kEnd));
        const float whole = __uint_as_float(ring.at(Z::kEnd + 1)[0]);
#pragma unroll
        for (int m = 0; m < NC; ++m) {
            Ux[m].put(w, W[m] * end, l);
            Wx[m].put(w, W[m], l);
        }
        exchange();
        // S <- exp(G_C) S + K^T (until beta W)
#pragma unroll
        for (int m = 0; m < NC; ++m) {
            const Frag<3> u0 = Ux[m].get(0, l), u1 = Ux[m].get(1, l);
#pragma unroll
            for (int t = 0; t < TW; ++t) {
                f32x4 y = zero;
                S[t][m] *= whole;
                mac_pair(frag(Inputs{}, Z::kKT + 2 * t * NP), u0, S[t][m],
                         frag(Inputs{}, Z::kKT + (2 * t + 1) * NP), u1, y);
                S[t][m] += y;
            }
        }
        ring.next(Z::kEnd, Z::N - Z::kEnd, fetch);
        put_state();
        if (SAVE)
#pragma unroll
            for (int m = 0; m < NC; ++m) {
                if (col0 + 16 * m >= dvp) break;
                const Buffer dst = buffer(
                    save_w + (saved_chunk(a, b, h, n) * dvp + col0 + 16 * m) * kChunk,
                    kChunk * kSlice * 4);
                store16_later(__builtin_bit_cast(u32x4, W[m]), dst, lane16 + 1024 * w, 0);
            }
        key0 = key1, head0 = head1;
    }
    if (s_out)
#pragma unroll
        for (int t = 0; t < TW; ++t)
#pragma unroll
            for (int m = 0; m < NC; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * (TW * w + t) + 4 * g + r, col = col0 + 16 * m + c;
                    if (row < a.dk && col < a.dv) s_out[(state + row) * a.dv + col] = S[t][m][r];
                }
}

template <int NP, int DK>
struct BackwardOrder {
    static constexpr int KB = DK / 32, TW = DK / 64;
    static constexpr int kUntil = KB * NP, kP = kUntil + 1, kBeta = kP + 6, kX = kBeta + 1,
                         kSince = kX + 6, kT = kSince + 2, kTotal = kT + TW * 4 * NP;
    static constexpr int D = NP == 1 ? kTotal : (kTotal + 1) / 2, N = (kTotal + D - 1) / D * D;
};

// The scan's backward pass, chunks from last to first, dS the gradient at
// the chunk's end: dW = beta (P^T dO + until K dS), dR = X^T dW (which is
// dV), dS <- exp(G_C) dS + Q~^T Gamma dO - K^T Gamma dR.  It leaves dS and dR
// of every chunk for the gradients.  Rows are divided as in the forward scan.
template <typename T, int DK, int NC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void
delta_scan_back_kernel(DeltaArgs a, ChunkRange cr, const unsigned char *ws_key,
                       const unsigned char *ws_head, const T *grad_o, int64_t ob, int64_t ot,
                       int64_t oh, const float *ds_in, float *ds_out, T *dv, float *ws_ds,
                       float *ws_dr) {
    constexpr int NP = Planes<T>::n;
    using L = PrepLayout<NP, DK>;
    using Z = BackwardOrder<NP, DK>;
    constexpr int KB = Z::KB, TW = Z::TW, KT = DK / 16;
    __shared__ Shared<3, KB> Sx[NC];   // dS
    __shared__ Shared<NP, 2> Ox[NC];   // dO
    __shared__ Shared<3, 2> Wx[NC];    // dW
    __shared__ Shared<3, 2> Rx[NC];    // -Gamma dR
    __shared__ Shared<3, 2> Gx[NC];    // scale Gamma dO
    int b, h, part;
    if (!head_and_part(a, b, h, part)) return;
    const int hk = h / (a.Hv / a.Hk), len = seq_len(a, b), live = live_chunks(cr, len);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, g = l >> 4,
              c = l & 15, col0 = kSlice * NC * part, dvp = padded_dv(a.dv);
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const uint32_t lane16 = 16 * l;

    f32x4 S[TW][NC];
    const int64_t state = (int64_t)(b * a.Hv + h) * a.dk;
#pragma unroll
    for (int t = 0; t < TW; ++t)
#pragma unroll
        for (int m = 0; m < NC; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * (TW * w + t) + 4 * g + r, col = col0 + 16 * m + c;
                S[t][m][r] = ds_in && col < a.dv && row < a.dk ? ds_in[(state + row) * a.dv + col]
                                                               : 0.f;
            }
    const int64_t dvt = (int64_t)a.Hv * a.dv;
    const T *go = grad_o + b * ob + h * oh + col0;
    T *dvc = dv + ((int64_t)b * a.T * a.Hv + h) * a.dv + col0;
    Rows<T> o_rows[NC], v_rows[NC];
#pragma unroll
    for (int m = 0; m < NC; ++m) {
        o_rows[m].set(ot, 4 * w + g, c, col0 + 16 * m + c < a.dv);
        v_rows[m].set(dvt, 4 * w + g, c, col0 + 16 * m + c < a.dv);
    }
    for (int t = (cr.first + live) * kChunk + 4 * w + g; t < a.T && t < (cr.first + cr.count) * kChunk;
         t += 16)
#pragma unroll
        for (int m = 0; m < NC; ++m)
            if (t >= len && col0 + 16 * m + c < a.dv) dvc[t * dvt + 16 * m + c] = from_f32<T>(0.f);

    const int last = live > 0 ? live - 1 : 0;
    const unsigned char *key_at = ws_key + cr.key_chunk(a, b, hk, last) * L::kPerKeyHead,
                        *head_at = ws_head + cr.chunk(a, b, h, last) * L::kPerHead;
    Buffer key0, key1, head0, head1;
    // rows of a transposed triangle: their last block always, the first one
    // for the first two tiles (elsewhere what is read for it is not used)
    const uint32_t k_lane = lane16 + w * NP * 1024, x_lane = lane16 + upper_tile(w, 1) * 1024,
                   kt_lane = lane16 + w * TW * 2048, s_lane = 16 * g + 64 * w;
    const uint32_t x_first = lane16 + (w < 2 ? upper_tile(w, 0) : 0) * 1024;
    auto fetch = [&](int j, bool next) -> u32x4 {
        const Buffer key = next ? key1 : key0, head = next ? head1 : head0;
        auto triangle = [&](int i, int base) {  // [first block, last block][3]
            return load16(head, i < 3 ? x_first : x_lane, base + i % 3 * kTriTiles * 1024);
        };
        if (j < Z::kUntil) return load16(key, k_lane, (j / NP * 4 * NP + j % NP) * 1024);
        if (j == Z::kUntil) return load16(head, s_lane, 2 * L::kTri + 256);
        if (j < Z::kBeta) return triangle(j - Z::kP, L::kTri);
        if (j == Z::kBeta) return load16(head, s_lane, 2 * L::kTri + 512);
        if (j < Z::kSince) return triangle(j - Z::kX, 0);
        if (j == Z::kSince) return load16(head, s_lane, 2 * L::kTri);
        if (j == Z::kSince + 1) return load_whole<L>(head);
        if (j < Z::kTotal) {
            const int i = j - Z::kT, p = i % NP, q = i / NP % 2, at = i / (2 * NP);
            return load16(key, kt_lane, L::kKey + q * L::kKeyT + (p * KT * 2 + at) * 1024);
        }
        return u32x4{0u, 0u, 0u, 0u};
    };
    T ov[NC][4];
    auto fetch_o = [&](int i) {
        const int t0 = (cr.first + i) * kChunk;
        const Buffer src = Rows<T>::chunk(go + t0 * ot, ot, len - t0);
#pragma unroll
        for (int m = 0; m < NC; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) ov[m][r] = o_rows[m].load(src, 0, r, m);
    };
    f32x4 dO[NC];
    auto put_inputs = [&]() {  // dS, and dO of the chunk that is next
#pragma unroll
        for (int m = 0; m < NC; ++m) {
#pragma unroll
            for (int t = 0; t < TW; ++t) Sx[m].put(TW * w + t, S[t][m], l);
#pragma unroll
            for (int r = 0; r < 4; ++r) dO[m][r] = to_f32<T>(ov[m][r]);
            Ox[m].put(w, dO[m], l);
        }
    };
    Ring<Z::N, Z::D> ring;
    auto frag = [&](auto n, int j) {
        Frag<decltype(n)::value> f;
#pragma unroll
        for (int p = 0; p < decltype(n)::value; ++p) f.p[p] = ring.at(j + p);
        return f;
    };
    using Inputs = std::integral_constant<int, NP>;
    using Three = std::integral_constant<int, 3>;
    if (live > 0) {
        // in the loop's order: waits count the loads that were issued since
        key0 = buffer(key_at, L::kPerKeyHead), head0 = buffer(head_at, L::kPerHead);
        fetch_o(live - 1);
        ring.fill(fetch);
        put_inputs();
    }
    for (int i = live - 1; i >= 0; --i) {
        const int t0 = (cr.first + i) * kChunk;
        if (i > 0) {  // before the first chunk: read again, not used
            key_at -= L::kPerKeyHead;
            head_at -= L::kPerHead;
        }
        key1 = buffer(key_at, L::kPerKeyHead), head1 = buffer(head_at, L::kPerHead);
        const int64_t at = cr.chunk(a, b, h, i);
        if (i > 0) fetch_o(i - 1);
        exchange();
        // dW = beta (until K dS + P^T dO)
        f32x4 dW[NC], dW2[NC], dR[NC];
#pragma unroll
        for (int m = 0; m < NC; ++m) dW[m] = dW2[m] = dR[m] = zero;
#pragma unroll
        for (int kb = 0; kb < KB; kb += 2) {
            const Frag<NP> k0 = frag(Inputs{}, kb * NP), k1 = frag(Inputs{}, (kb + 1) * NP);
#pragma unroll
            for (int m = 0; m < NC; ++m)
                mac_pair(k0, Sx[m].get(kb, l), dW[m], k1, Sx[m].get(kb + 1, l), dW2[m]);
            ring.next(kb * NP, 2 * NP, fetch);
        }
        const f32x4 until = __builtin_bit_cast(f32x4, ring.at(Z::kUntil));
        const Frag<3> p0 = frag(Three{}, Z::kP), p1 = frag(Three{}, Z::kP + 3);
        const f32x4 beta = __builtin_bit_cast(f32x4, ring.at(Z::kBeta));
#pragma unroll
        for (int m = 0; m < NC; ++m) {
            dW[m] = (dW[m] + dW2[m]) * until;
            if (w < 2) dW[m] = mac(p0, Ox[m].get(0, l), dW[m]);
            dW[m] = mac(p1, Ox[m].get(1, l), dW[m]);
            Wx[m].put(w, dW[m] * beta, l);
        }
        ring.next(Z::kUntil, Z::kBeta + 1 - Z::kUntil, fetch);
        // what the gradients need of dS
#pragma unroll
        for (int m = 0; m < NC; ++m) {
            if (col0 + 16 * m >= dvp) break;
            const Buffer ds = buffer(ws_ds + (at * dvp + col0 + 16 * m) * DK, DK * kSlice * 4);
#pragma unroll
            for (int t = 0; t < TW; ++t)
                store16(__builtin_bit_cast(u32x4, S[t][m]), ds, lane16 + 1024 * TW * w, 1024 * t);
        }
        exchange();
        // dR = X^T dW
        const Frag<3> x0 = frag(Three{}, Z::kX), x1 = frag(Three{}, Z::kX + 3);
        const f32x4 since = __builtin_bit_cast(f32x4, ring.at(Z::kSince));
        const float whole = __uint_as_float(ring.at(Z::kSince + 1)[0]);
#pragma unroll
        for (int m = 0; m < NC; ++m) {
            if (w < 2) {
                f32x4 y = zero;
                mac_pair(x0, Wx[m].get(0, l), y, x1, Wx[m].get(1, l), dR[m]);
                dR[m] += y;
            } else {
                dR[m] = mac(x1, Wx[m].get(1, l), dR[m]);
            }
            Rx[m].put(w, dR[m] * -since, l);
            Gx[m].put(w, dO[m] * (since * a.scale), l);
        }
        ring.next(Z::kX, 6, fetch);
        exchange();
        // dS <- exp(G_C) dS + Q~^T Gamma dO - K^T Gamma dR
#pragma unroll
        for (int t = 0; t < TW; ++t)
#pragma unroll
            for (int m = 0; m < NC; ++m) S[t][m] *= whole;
#pragma unroll
        for (int t = 0; t < TW; ++t)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const Frag<NP> k = frag(Inputs{}, Z::kT + ((t * 2 + kb) * 2) * NP),
                               q = frag(Inputs{}, Z::kT + ((t * 2 + kb) * 2 + 1) * NP);
#pragma unroll
                for (int m = 0; m < NC; ++m) {
                    f32x4 y = zero;
                    mac_pair(k, Rx[m].get(kb, l), S[t][m], q, Gx[m].get(kb, l), y);
                    S[t][m] += y;
                }
                ring.next(Z::kT + (t * 2 + kb) * 2 * NP, 2 * NP, fetch);
            }
        ring.next(Z::kSince, 2, fetch);
        if (Z::N > Z::kTotal) ring.next(Z::kTotal, Z::N - Z::kTotal, fetch);
        put_inputs();
        // rows past the length are 0: X^T is the identity there, and dW 0
        const Buffer dst = Rows<T>::chunk(dvc + t0 * dvt, dvt, a.T - t0);
#pragma unroll
        for (int m = 0; m < NC; ++m) {
#pragma unroll
            for (int r = 0; r < 4; ++r) v_rows[m].store(from_f32<T>(dR[m][r]), dst, 0, r, m);
            if (col0 + 16 * m >= dvp) break;
            store16(__builtin_bit_cast(u32x4, dR[m]),
                    buffer(ws_dr + (at * dvp + col0 + 16 * m) * kChunk, kChunk * kSlice * 4),
                    lane16 + 1024 * w, 0);
        }
        key0 = key1, head0 = head1;
    }
    if (ds_out)
#pragma unroll
        for (int t = 0; t < TW; ++t)
#pragma unroll
            for (int m = 0; m < NC; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * (TW * w + t) + 4 * g + r, col = col0 + 16 * m + c;
                    if (row < a.dk && col < a.dv) ds_out[(state + row) * a.dv + col] = S[t][m][r];
                }
}

// 32 columns a workgroup where that still leaves one for every CU: 64 heads of
// 128 x 128 over 2048 tokens take 86 us against 108 with 16 (bf16), 119 against
// 153 with what the gradients need, and back 142 against 148; 96 heads of 96 x 112
// over 1000 tokens 134 against 153 (fp32).  16 heads, which would leave three
// quarters of the CUs idle: 281 against 195 (8192 tokens of 128 x 128), training on
// 64 x 128 298 against 219, back 333 against 196.
bool two_slices(const DeltaArgs &a, int slices) {
    return (int64_t)a.B * a.Hv * ((slices + 1) / 2) >= 256;
}

int grid_of(const DeltaArgs &a, int slices, int nc) {
    return (a.B * a.Hv + 7) / 8 * 8 * ((slices + nc - 1) / nc);
}

template <typename T, int DK, int NC>
hipError_t scan_nc(const DeltaArgs &a, const ChunkRange &cr, const DeltaForward &f, int slices,
                   const unsigned char *ws_key, const unsigned char *ws_head, hipStream_t s) {
    const int grid = grid_of(a, slices, NC);
    T *o = reinterpret_cast<T *>(f.o);
    if (f.save_s)
        delta_scan_kernel<T, DK, NC, true><<<grid, 512, 0, s>>>(
            a, cr, ws_key, ws_head, f.s_in, f.s_out, o, f.ob, f.ot, f.oh, f.save_s, f.save_w);
    else
        delta_scan_kernel<T, DK, NC, false><<<grid, 512, 0, s>>>(
            a, cr, ws_key, ws_head, f.s_in, f.s_out, o, f.ob, f.ot, f.oh, nullptr, nullptr);
    return hipGetLastError();
}

template <typename T, int DK>
hipError_t scan_t(const DeltaArgs &a, const ChunkRange &cr, const DeltaForward &f,
                  const unsigned char *ws_key, const unsigned char *ws_head, hipStream_t s) {
    const int slices = (f.save_s ? padded_dv(a.dv) : a.dv + kSlice - 1) / kSlice;
    return two_slices(a, slices) ? scan_nc<T, DK, 2>(a, cr, f, slices, ws_key, ws_head, s)
                                 : scan_nc<T, DK, 1>(a, cr, f, slices, ws_key, ws_head, s);
}

template <typename T, int DK, int NC>
hipError_t scan_back_nc(const DeltaArgs &a, const ChunkRange &cr, const DeltaBackward &f,
                        const unsigned char *ws_key, const unsigned char *ws_head, hipStream_t s) {
    const int grid = grid_of(a, padded_dv(a.dv) / kSlice, NC);
    delta_scan_back_kernel<T, DK, NC><<<grid, 256, 0, s>>>(
        a, cr, ws_key, ws_head, reinterpret_cast<const T *>(f.grad_o), f.ob, f.ot, f.oh, f.ds_in,
        f.ds_out, reinterpret_cast<T *>(f.dv), f.ws_ds, f.ws_dr);
    return hipGetLastError();
}

template <typename T, int DK>
hipError_t scan_back_t(const DeltaArgs &a, const ChunkRange &cr, const DeltaBackward &f,
                       const unsigned char *ws_key, const unsigned char *ws_head, hipStream_t s) {
    return two_slices(a, padded_dv(a.dv) / kSlice)
               ? scan_back_nc<T, DK, 2>(a, cr, f, ws_key, ws_head, s)
               : scan_back_nc<T, DK, 1>(a, cr, f, ws_key, ws_head, s);
}

}  // namespace

hipError_t launch_delta_scan(int dtype, const DeltaArgs &a, const ChunkRange &cr,
                             const DeltaForward &f, const unsigned char *ws_key,
                             const unsigned char *ws_head, hipStream_t s) {
    return SLA_DELTA_DISPATCH(scan_t, a, cr, f, ws_key, ws_head, s);
}

hipError_t launch_delta_scan_back(int dtype, const DeltaArgs &a, const ChunkRange &cr,
                                  const DeltaBackward &f, const unsigned char *ws_key,
                                  const unsigned char *ws_head, hipStream_t s) {
    return SLA_DELTA_DISPATCH(scan_back_t, a, cr, f, ws_key, ws_head, s);
}

}  // namespace sla
