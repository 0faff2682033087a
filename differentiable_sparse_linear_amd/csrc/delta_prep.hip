// The gated delta rule in chunks: what the scans over the chunks need of each,
// prepared for all of them at once.
#include "delta_chunk.h"

namespace sla {

namespace {

// acc + A B of 16 x 16 fp32 blocks in LDS (v_mfma_f32_16x16x4_f32).
__device__ inline f32x4 block_mac(const float *A, const float *B, int ld, f32x4 acc, int g, int c) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(A[c * ld + 4 * k + g], B[(4 * k + g) * ld + c],
                                                   acc, 0, 0, 0);
    return acc;
}

// A fragment's 16 bytes of each lane.
__device__ inline void put16(u32x4 x, unsigned char *to, uint32_t lane16) {
    *reinterpret_cast<u32x4 *>(to + lane16) = x;
}

// One workgroup prepares one chunk of one key head and of its value heads:
// the fragments of K, K^T and Q (backward: Q^T), and for each value head
// those of X = (I + L)^-1 and P' (backward: of X^T and P^T, P_ij =
// scale D_ij (q_i . k_j)).
//
// The inverse is taken in fp32 by 16 x 16 blocks: those on the diagonal by
// substitution, then the two blocks that complete 32 x 32 inverses, then the
// four that complete the whole, each [A 0; C B]^-1 = [A^-1 0; -B^-1 C A^-1 B^-1].
//
// A workgroup waits on the latency of its loads, barriers and short products
// for most of its time, so four of them share a CU where the planes allow (128
// registers): 112 chunks of 16 heads (bf16) take 50 us with 128 keys, 155 MB
// written at 3.1 TB/s, and 49 with 256 registers; 128 chunks of 16 heads with 64
// keys 39.4 and 40.3, for the backward pass 22.4 and 22.9 a launch of 64.
template <typename T, int DK, bool BWD>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(Planes<T>::n == 1 ? 4 : 2))) void
delta_prep_kernel(DeltaArgs a, ChunkRange cr, bool vec, unsigned char *ws_key,
                  unsigned char *ws_head) {
    constexpr int NP = Planes<T>::n, KB = DK / 32, KT = DK / 16, LD = 68;
    using L = PrepLayout<NP, DK>;
    const int n = cr.first + blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
    const int len = seq_len(a, b);
    if (n * kChunk >= len) return;
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    int g = l >> 4, c = l & 15;

    // the planes' tiles of K (then of Q, backward), then the triangles
    constexpr int kPlane = 4 * KT * kTileBytes, kTriBytes = 2 * 64 * LD * 4;
    __shared__ __align__(16) unsigned char lds[NP * kPlane > kTriBytes ? NP * kPlane : kTriBytes];
    __shared__ double Gs[64];
    __shared__ float Bs[64];
    float *Lb = reinterpret_cast<float *>(lds), *Pb = Lb + 64 * LD;

    unsigned char *key = ws_key + cr.key_chunk(a, b, hk, blockIdx.x) * L::kPerKeyHead;
    const uint32_t lane16 = 16 * l;

    const int t = n * kChunk + 16 * w + c;
    const bool live = t < len;
    const T *krow = reinterpret_cast<const T *>(a.k) + b * a.kb + t * a.kt + hk * a.kh;
    const T *qrow = reinterpret_cast<const T *>(a.q) + b * a.qb + t * a.qt + hk * a.qh;
    Frag<NP> kf[KB], qf[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        kf[kb] = load_frag<T>(krow, 32 * kb + 4 * g, a.dk, live, vec);
        qf[kb] = load_frag<T>(qrow, 32 * kb + 4 * g, a.dk, live, vec);
    }
    // rows in tiles: row c of tile (w, 2 kb + e), four keys from 4 g
    auto put_rows = [&](const Frag<NP> (&f)[KB]) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<uint2 *>(lds + p * kPlane + (w * KT + 2 * kb + e) * kTileBytes +
                                               32 * c + 8 * g) =
                        make_uint2(f[kb].p[p][2 * e], f[kb].p[p][2 * e + 1]);
    };
    // transposed: rows d of K^T, contraction over the tokens
    auto transpose = [&](int base) {
#pragma unroll
        for (int i = 0; i < KT / 2; ++i) {
            const int rt = (4 * i + w) >> 1, kb = w & 1;
            const Frag<NP> f = get_transposed<NP>(lds + (2 * kb * KT + rt) * kTileBytes, kPlane,
                                                  KT * kTileBytes, l);
#pragma unroll
            for (int p = 0; p < NP; ++p)
                put16(f.p[p], key + base + (p * KT + rt) * 2048 + kb * 1024, lane16);
        }
    };
    put_rows(kf);
    exchange();
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        kk[j] = qk[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (j > w) continue;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            Frag<NP> f;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const unsigned char *tile = lds + p * kPlane + (j * KT + 2 * kb) * kTileBytes + 32 * c + 8 * g;
                const uint2 lo = *reinterpret_cast<const uint2 *>(tile),
                            hi = *reinterpret_cast<const uint2 *>(tile + kTileBytes);
                f.p[p] = u32x4{lo.x, lo.y, hi.x, hi.y};
            }
            mac_pair(kf[kb], f, kk[j], qf[kb], f, qk[j]);
        }
    }
    transpose(L::kKey);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            unsigned char *to = key + ((kb * 4 + w) * NP + p) * 1024;
            put16(kf[kb].p[p], to, lane16);
            if (!BWD) put16(qf[kb].p[p], to + L::kKey + L::kKeyT, lane16);
        }
    if (BWD) {
        exchange();
        put_rows(qf);
        exchange();
        transpose(L::kKey + L::kKeyT);
    }

    const int group = a.Hv / a.Hk;
    for (int m = 0; m < group; ++m) {
        // not known to be the same in every turn, or all addresses in LDS would
        // be kept in registers between them
        asm volatile("" : "+v"(g), "+v"(c));
        const int h = hk * group + m;
        unsigned char *at = ws_head + cr.chunk(a, b, h, blockIdx.x) * L::kPerHead;
        float *scalars = reinterpret_cast<float *>(at + 2 * L::kTri);
        // every wavefront sums the gates; the first keeps them
        const int tl = n * kChunk + l;
        const bool in = tl < len;
        const float be = in ? a.beta[b * a.bb + tl * a.bt + h * a.bh] : 0.f;
        const double G = gate_sum(in ? a.gate[b * a.gb + tl * a.gt + h * a.gh] : 0.f, l);
        exchange();  // the tiles, or the last head's triangles, are done with
        if (w == 0) {
            Gs[l] = G;
            Bs[l] = be;
            scalars[l] = decay(G);
            const float until = decay(__shfl(G, 63, 64) - G);
            scalars[64 + l] = BWD ? until : until * be;
            scalars[128 + l] = be;
        }
        exchange();
        double Gi[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) Gi[r] = Gs[16 * w + 4 * g + r];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = 16 * j + c;
            const double Gj = Gs[col];
            const float bj = Bs[col];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * w + 4 * g + r;
                const float D = row >= col ? decay(Gi[r] - Gj) : 0.f;
                Lb[row * LD + col] = row > col ? D * kk[j][r] * bj : 0.f;
                Pb[row * LD + col] = BWD ? a.scale * D * qk[j][r] : D * qk[j][r] * bj;
            }
        }
        exchange();
        // a triangle to its fragments
        auto fragments = [&](const float *M, int base) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                if (BWD ? kb < (w >> 1) : kb > (w >> 1)) continue;
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = 16 * w + c, j = 32 * kb + 16 * (e >> 2) + 4 * g + (e & 3);
                    x[e] = BWD ? M[j * LD + i] : M[i * LD + j];
                }
                const Frag<3> f = split<3>(x);
                const int tile = BWD ? upper_tile(w, kb) : lower_tile(w, kb);
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    put16(f.p[p], at + base + (p * kTriTiles + tile) * 1024, lane16);
            }
        };
        fragments(Pb, L::kTri);
        // X takes P's place: diagonal blocks by substitution, column c
        float x[16];
        const float *Ld = Lb + 16 * w * LD + 16 * w;
        int from = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            // four rows at a time, tied to the ones before: all 120 values at
            // once would fill the registers
            if (q) asm volatile("" : "+v"(x[4 * q - 1]), "+v"(from));
            f32x4 rows[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j <= q; ++j)
                    rows[r][j] = *reinterpret_cast<const f32x4 *>(Ld + from + (4 * q + r) * LD + 4 * j);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 4 * q + r;
                x[i] = i == c ? 1.f : 0.f;
#pragma unroll
                for (int j = 0; j < i; ++j) x[i] = fmaf(-rows[r][j >> 2][j & 3], x[j], x[i]);
            }
        }
        exchange();
        if (g == 0)
#pragma unroll
            for (int i = 0; i < 16; ++i) Pb[(16 * w + i) * LD + 16 * w + c] = x[i];
#pragma unroll
        for (int j = 1; j < 4; ++j)  // nothing stands above the diagonal blocks
            if (j > w)
#pragma unroll
                for (int r = 0; r < 4; ++r) Pb[(16 * w + 4 * g + r) * LD + 16 * j + c] = 0.f;
        exchange();
        auto block = [&](float *M, int i, int j) { return M + 16 * i * LD + 16 * j; };
        auto put_block = [&](float *to, const f32x4 &y, float sign) {
#pragma unroll
            for (int r = 0; r < 4; ++r) to[(4 * g + r) * LD + c] = sign * y[r];
        };
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        if (w & 1) {  // blocks (1, 0) and (3, 2); L's upper blocks hold what is between
            float *between = block(Lb, w - 1, w);
            put_block(between, block_mac(block(Lb, w, w - 1), block(Pb, w - 1, w - 1), LD, zero, g, c), 1.f);
            put_block(block(Pb, w, w - 1), block_mac(block(Pb, w, w), between, LD, zero, g, c), -1.f);
        }
        exchange();
        const int bi = 2 + (w >> 1), bj = w & 1;  // the block of this wavefront
        f32x4 y = block_mac(block(Lb, bi, 1), block(Pb, 1, bj), LD, zero, g, c);
        if (bj == 0) y = block_mac(block(Lb, bi, 0), block(Pb, 0, 0), LD, y, g, c);
        put_block(block(Lb, bj, bi), y, 1.f);
        exchange();
        y = block_mac(block(Pb, bi, 2), block(Lb, bj, 2), LD, zero, g, c);
        if (bi == 3) y = block_mac(block(Pb, 3, 3), block(Lb, bj, 3), LD, y, g, c);
        put_block(block(Pb, bi, bj), y, -1.f);
        exchange();
        fragments(Pb, 0);
    }
}

template <typename T, int DK>
hipError_t prep_t(const DeltaArgs &a, const ChunkRange &cr, bool back, unsigned char *ws_key,
                  unsigned char *ws_head, hipStream_t s) {
    if (cr.count == 0) return hipSuccess;
    const bool vec = rows_aligned(a, sizeof(T));
    const dim3 grid(cr.count, a.Hk, a.B);
    if (back)
        delta_prep_kernel<T, DK, true><<<grid, 256, 0, s>>>(a, cr, vec, ws_key, ws_head);
    else
        delta_prep_kernel<T, DK, false><<<grid, 256, 0, s>>>(a, cr, vec, ws_key, ws_head);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_prep(int dtype, const DeltaArgs &a, const ChunkRange &cr, bool back,
                             unsigned char *ws_key, unsigned char *ws_head, hipStream_t s) {
    return SLA_DELTA_DISPATCH(prep_t, a, cr, back, ws_key, ws_head, s);
}

}  // namespace sla
