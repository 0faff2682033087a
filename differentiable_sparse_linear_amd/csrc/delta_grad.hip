// Gradients of q, k, beta and gate of the gated delta rule, all chunks at
// once, from what the forward scan (S, W) and the backward scan (dS, dR) left.
#include "delta_chunk.h"

namespace sla {

namespace {

// With z_ij = D_ij dO_i . w_j (j <= i) and y_ij = -D_ij dR_i . w_j (j < i):
//
//   dq~_i   = Gamma_i S dO_i + sum_j beta_j z_ij k_j
//   dk_i    = r_i + beta_i h_i
//   r_i     = -Gamma_i S dR_i + sum_j beta_j y_ij k_j        (k read the state)
//   h_j     = until_j dS w_j + sum_i (y_ij k_i + z_ij q~_i)   (k wrote it)
//   dbeta_j = k_j . h_j
//
// A gate acts on everything that passes its token t:
//
//   dgate_t = sum_(i >= t) A_i + sum_(j < t) B_j + sum_(j < t <= i) E_ij + exp(G_C) <S, dS>
//     A_i  = Gamma_i (q~_i . S dO_i - k_i . S dR_i)
//     B_j  = beta_j until_j k_j . dS w_j
//     E_ij = beta_j (z_ij q~_i . k_j + y_ij k_i . k_j)
//
// Each term has a_t as a factor, so a strong decay's gradient is as exact as a weak
// one's.  (As the sum of q~_i . dq~_i + k_i . r_i - beta_i dbeta_i from t on it would
// be a difference of terms that have not.)
//
// One workgroup takes one chunk of one key head and sums over the value
// heads that share it, so no sum depends on the order of workgroups.  Wavefront
// (w, half) has 16 tokens and half of the keys; half 0 also forms z, half 1 y.
// What several need (S, dS, W, dR, as the scans left them) is split into planes
// once, staged in LDS 32 value columns at a time and read back transposed; the
// next columns' tiles are loaded meanwhile.
//
// 64 heads of 128 x 128 over 1024 tokens (bf16) take 124 us, 1.7 TB/s of the 208 KB
// a chunk and head; 16 heads of 64 x 128 over 4096 tokens 91: two wavefronts a SIMD
// wait in turn for loads, LDS and each other (48 % of their cycles; matrix
// instructions busy 16 % of the time).  The pairs' part of the gates' gradient is
// 16 and 10 us of it; before it was there, four wavefronts a SIMD (1024 threads,
// 128 registers, which spill) took 142 and 85 us against 106 and 75, a double
// stage 104 and 83.
template <typename T, int DK, bool GROUP>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void
delta_grad_kernel(DeltaArgs a, ChunkRange cr, bool vec_q, bool vec_o, const unsigned char *ws_key,
                  const unsigned char *ws_head, const T *grad_o, int64_t ob, int64_t ot,
                  int64_t oh, T *dq, T *dk, float *dbeta, float *dgate, const float *save_s,
                  const float *save_w, const float *ws_ds, const float *ws_dr) {
    constexpr int NP = Planes<T>::n, KT = DK / 16, HT = KT / 2, KB = DK / 32, LD = 68;
    constexpr int kThreads = 512;
    using L = PrepLayout<NP, DK>;
    const int n = cr.first + blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
    const int len = seq_len(a, b), group = a.Hv / a.Hk, dvp = padded_dv(a.dv);
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3, half = wave >> 2;
    const int l = tid & 63, g = l >> 4, c = l & 15;
    const int t0 = n * kChunk, tile0 = HT * half;

    if (t0 >= len) {  // nothing here was read
        for (int i = tid; i < kChunk * a.dk; i += kThreads) {
            const int t = t0 + i / a.dk, d = i % a.dk;
            if (t >= a.T) break;
            const int64_t at = (((int64_t)b * a.T + t) * a.Hk + hk) * a.dk + d;
            dq[at] = dk[at] = from_f32<T>(0.f);
        }
        for (int i = tid; i < kChunk * group; i += kThreads) {
            const int t = t0 + i / group;
            if (t >= a.T) break;
            const int64_t at = ((int64_t)b * a.T + t) * a.Hv + hk * group + i % group;
            dbeta[at] = dgate[at] = 0.f;
        }
        return;
    }

    // stage: planes of S and dS [3][KT][2 slices], of W and dR [3][4][2]
    constexpr int kStateBytes = 3 * KT * 2 * kTileBytes, kRowBytes = 3 * 4 * 2 * kTileBytes;
    constexpr int kStatePlane = KT * 2 * kTileBytes, kRowPlane = 4 * 2 * kTileBytes;
    constexpr int kStage = 2 * kStateBytes + 2 * kRowBytes, kTri = 2 * 64 * LD * 4;
    __shared__ __align__(16) unsigned char lds[kStage > kTri ? kStage : kTri];
    __shared__ double Gs[64];
    __shared__ float Bs[64], dots[2][4][64];    // of a token: A, dbeta, B, its rows' E
    __shared__ float below[2][4][64], ends[8];  // E's sums over a row tile; <S, dS>
    unsigned char *Sp = lds, *Dp = lds + kStateBytes, *Wp = lds + 2 * kStateBytes,
                  *Rp = Wp + kRowBytes;
    float *Zb = reinterpret_cast<float *>(lds), *Yb = Zb + 64 * LD;

    const unsigned char *key = ws_key + cr.key_chunk(a, b, hk, blockIdx.x) * L::kPerKeyHead;
    const Buffer kq = buffer(key, L::kPerKeyHead);
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const uint32_t lane16 = 16 * l;

    f32x4 dq_sum[HT], dk_sum[HT];
#pragma unroll
    for (int t = 0; t < HT; ++t) dq_sum[t] = dk_sum[t] = zero;

    for (int m = 0; m < group; ++m) {
        const int h = hk * group + m;
        const int64_t at = cr.chunk(a, b, h, blockIdx.x);
        const uint32_t state_bytes = DK * dvp * 4, row_bytes = kChunk * dvp * 4;
        const Buffer S = buffer(save_s + saved_chunk(a, b, h, n) * DK * dvp, state_bytes),
                     dS = buffer(ws_ds + at * DK * dvp, state_bytes),
                     rows = half ? buffer(ws_dr + at * kChunk * dvp, row_bytes)
                                 : buffer(save_w + saved_chunk(a, b, h, n) * kChunk * dvp, row_bytes);
        const float *scalars =
            reinterpret_cast<const float *>(ws_head + at * L::kPerHead + 2 * L::kTri);
        const int rows_here = len - t0 < kChunk ? len - t0 : kChunk;
        const Buffer o_rows = buffer(grad_o + b * ob + t0 * ot + h * oh,
                                     rows_here * (uint32_t)ot * sizeof(T));
        const uint32_t o_lane = ((16 * w + c) * (uint32_t)ot + 4 * g) * sizeof(T);

        // what this wavefront stages of two slices: with DK 128 one tile of S
        // and of dS each, with 64 one of either; and one of W (half 0) or dR
        constexpr int kMine = KT == 8 ? 2 : 1;
        f32x4 st[kMine][2], rw[2];
        Frag<NP> of_next;
        auto tile_of = [&](Buffer from, uint32_t i) {
            return __builtin_bit_cast(
                f32x4, __builtin_amdgcn_raw_buffer_load_b128(from, lane16, i * 1024, 0));
        };
        auto load_tiles = [&](int v0) {
            const int sl = v0 / kSlice;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    st[i][e] = tile_of((KT == 8 ? i : half) ? dS : S,
                                       (sl + e) * KT + (KT == 8 ? wave : w));
                rw[e] = tile_of(rows, (sl + e) * 4 + w);
            }
            of_next = row_frag<T>(o_rows, o_lane + v0 * sizeof(T), a.dv - v0 - 4 * g, vec_o);
        };

        f32x4 zy[4], aq[HT], ar[HT], hh[HT];
#pragma unroll
        for (int j = 0; j < 4; ++j) zy[j] = zero;
#pragma unroll
        for (int t = 0; t < HT; ++t) aq[t] = ar[t] = hh[t] = zero;
        float inner = 0.f;  // this lane's part of <S, dS>
        load_tiles(0);
        for (int v0 = 0; v0 < dvp; v0 += 32) {
            exchange();  // the stage (or Z and Y of the last head) is done with
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    put_tile<3>(((KT == 8 ? i : half) ? Dp : Sp) +
                                    ((KT == 8 ? wave : w) * 2 + e) * kTileBytes,
                                kStatePlane, st[i][e], g, c);
                put_tile<3>((half ? Rp : Wp) + (w * 2 + e) * kTileBytes, kRowPlane, rw[e], g, c);
                if constexpr (KT == 8)
#pragma unroll
                    for (int r = 0; r < 4; ++r) inner = fmaf(st[0][e][r], st[1][e][r], inner);
            }
            const Frag<NP> of = of_next;
            if constexpr (KT != 8) {  // S's owner reads dS of the same tile
                if (!half)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const f32x4 y = tile_of(dS, (v0 / kSlice + e) * KT + w);
#pragma unroll
                        for (int r = 0; r < 4; ++r) inner = fmaf(st[0][e][r], y[r], inner);
                    }
            }
            exchange();
            if (v0 + 32 < dvp) load_tiles(v0 + 32);
            const Frag<3> rf = get_transposed<3>(Rp + w * 2 * kTileBytes, kRowPlane, kTileBytes, l);
            const Frag<3> wf = get_transposed<3>(Wp + w * 2 * kTileBytes, kRowPlane, kTileBytes, l);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j > w) continue;
                const Frag<3> f = get_transposed<3>(Wp + j * 2 * kTileBytes, kRowPlane, kTileBytes, l);
                zy[j] = half ? mac(rf, f, zy[j]) : mac(of, f, zy[j]);
            }
#pragma unroll
            for (int t = 0; t < HT; ++t) {
                const int at_t = (tile0 + t) * 2 * kTileBytes;
                Frag<3> f = get_transposed<3>(Sp + at_t, kStatePlane, kTileBytes, l);
                aq[t] = mac(of, f, aq[t]);
                ar[t] = mac(rf, f, ar[t]);
                f = get_transposed<3>(Dp + at_t, kStatePlane, kTileBytes, l);
                hh[t] = mac(wf, f, hh[t]);
            }
        }
        const int tl = t0 + l;
        const float be = tl < len ? a.beta[b * a.bb + tl * a.bt + h * a.bh] : 0.f;
        if (wave == 0) {
            Gs[l] = gate_sum(tl < len ? a.gate[b * a.gb + tl * a.gt + h * a.gh] : 0.f, l);
            Bs[l] = be;
        }
        exchange();
        // q (half 0) or k (half 1) of this wavefront's tokens, for E
        Frag<NP> xf[KB];
        if (half) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    xf[kb].p[p] = load16(kq, lane16 + w * NP * 1024, (kb * 4 * NP + p) * 1024);
        } else {
            const int t = t0 + 16 * w + c;
            const T *x = reinterpret_cast<const T *>(a.q) + b * a.qb + t * a.qt + hk * a.qh;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
                xf[kb] = load_frag<T>(x, 32 * kb + 4 * g, a.dk, t < len, vec_q);
        }
        float f[4] = {0.f, 0.f, 0.f, 0.f};  // of rows t: E_ij of j < t <= i, i in this tile
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = 16 * j + c;
            f32x4 e = zero;
            if (j <= w) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    Frag<NP> kf;
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        kf.p[p] = load16(kq, lane16, ((kb * 4 + j) * NP + p) * 1024);
                    e = mac(xf[kb], kf, e);
                }
                e *= half ? Bs[col] : a.scale * Bs[col];
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * w + 4 * g + r;
                const float D = row >= col ? decay(Gs[row] - Gs[col]) : 0.f;
                const float y = half ? row > col ? -D * zy[j][r] : 0.f : D * zy[j][r];
                (half ? Yb : Zb)[row * LD + col] = y;
                e[r] = row > col ? e[r] * y : 0.f;
            }
            // sums from a row to the tile's end
#pragma unroll
            for (int r = 2; r >= 0; --r) e[r] += e[r + 1];
            float later = 0.f;
#pragma unroll
            for (int d = 1; d < 4; ++d) {
                const float y = __shfl_down(e[0], 16 * d, 64);
                later += g + d < 4 ? y : 0.f;
            }
            if (g == 0) below[half][w][col] = e[0] + later;
#pragma unroll
            for (int r = 0; r < 4; ++r) f[r] += 16 * w + 4 * g + r > col ? e[r] + later : 0.f;
        }
        const f32x4 since = *reinterpret_cast<const f32x4 *>(scalars + 16 * w + 4 * g);
        const f32x4 until = *reinterpret_cast<const f32x4 *>(scalars + 64 + 16 * w + 4 * g);
        const f32x4 beta = *reinterpret_cast<const f32x4 *>(scalars + 128 + 16 * w + 4 * g);
#pragma unroll
        for (int t = 0; t < HT; ++t) {
            aq[t] *= since;
            ar[t] *= -since;
            hh[t] *= until;
        }
        // q and k where the accumulators have their products' rows and keys:
        // values of the transposed fragments of this wavefront's tokens
        f32x4 qv[HT], kv[HT];
#pragma unroll
        for (int t = 0; t < HT; ++t) {
            Frag<NP> f, q;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const uint32_t at_t = L::kKey + ((p * KT + t) * 2) * 1024;
                const uint32_t lane = lane16 + tile0 * 2048 + (w >> 1) * 1024;
                f.p[p] = load16(kq, lane, at_t);
                q.p[p] = load16(kq, lane, L::kKeyT + at_t);
            }
            kv[t] = values(f, w & 1);
            qv[t] = values(q, w & 1) * a.scale;
        }
        // A and B, before the pairs' terms come to aq, ar and hh
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float A = 0.f, B = 0.f;
#pragma unroll
            for (int i = 0; i < HT; ++i) {
                A = fmaf(qv[i][r], aq[i][r], fmaf(kv[i][r], ar[i][r], A));
                B = fmaf(kv[i][r], hh[i][r], B);
            }
            A = sum16(A), B = sum16(beta[r] * B);
            const float F = sum16(f[r]);
            if (c == 0) {
                dots[half][0][16 * w + 4 * g + r] = A;
                dots[half][2][16 * w + 4 * g + r] = B;
                dots[half][3][16 * w + 4 * g + r] = F;
            }
        }
        inner *= scalars[63];
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) inner += __shfl_xor(inner, off, 64);
        if (l == 0) ends[wave] = inner;
        exchange();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if (kb <= (w >> 1)) {  // rows i of Z and Y
                float x1[8], x2[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = 16 * w + c, j = 32 * kb + 16 * (e >> 2) + 4 * g + (e & 3);
                    x1[e] = Bs[j] * Zb[i * LD + j];
                    x2[e] = Bs[j] * Yb[i * LD + j];
                }
                const Frag<3> zf = split<3>(x1), yf = split<3>(x2);
#pragma unroll
                for (int t = 0; t < HT; ++t) {
                    Frag<NP> f;
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        f.p[p] = load16(kq, lane16 + tile0 * 2048, L::kKey + ((p * KT + t) * 2 + kb) * 1024);
                    aq[t] = mac(zf, f, aq[t]);
                    ar[t] = mac(yf, f, ar[t]);
                }
            }
            if (kb >= (w >> 1)) {  // columns j
                float x1[8], x2[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = 16 * w + c, i = 32 * kb + 16 * (e >> 2) + 4 * g + (e & 3);
                    x1[e] = a.scale * Zb[i * LD + j];
                    x2[e] = Yb[i * LD + j];
                }
                const Frag<3> zf = split<3>(x1), yf = split<3>(x2);
#pragma unroll
                for (int t = 0; t < HT; ++t) {
                    Frag<NP> f, q;
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        const uint32_t at_t = L::kKey + ((p * KT + t) * 2 + kb) * 1024;
                        f.p[p] = load16(kq, lane16 + tile0 * 2048, at_t);
                        q.p[p] = load16(kq, lane16 + tile0 * 2048, L::kKeyT + at_t);
                    }
                    hh[t] = mac(zf, q, hh[t]);
                    hh[t] = mac(yf, f, hh[t]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float db = 0.f;
#pragma unroll
            for (int i = 0; i < HT; ++i) db = fmaf(kv[i][r], hh[i][r], db);
            db = sum16(db);
            if (c == 0) dots[half][1][16 * w + 4 * g + r] = db;
        }
        exchange();
        if (wave == 0) {  // lane t
            float A = dots[0][0][l] + dots[1][0][l], B = dots[0][2][l] + dots[1][2][l],
                  dg = dots[0][3][l] + dots[1][3][l], end = 0.f, past[3];
#pragma unroll
            for (int i = 0; i < 8; ++i) end += ends[i];
            // past[i]: of rows beyond tile i, then of columns up to this lane's
#pragma unroll
            for (int i = 2; i >= 0; --i)
                past[i] = (i < 2 ? past[i + 1] : 0.f) + below[0][i + 1][l] + below[1][i + 1][l];
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const float later = __shfl_down(A, off, 64), earlier = __shfl_up(B, off, 64);
                A += l + off < 64 ? later : 0.f;
                B += l >= off ? earlier : 0.f;
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const float y = __shfl_up(past[i], off, 64);
                    past[i] += l >= off ? y : 0.f;
                }
            }
            B = __shfl_up(B, 1, 64);  // of tokens before this one
#pragma unroll
            for (int i = 0; i < 3; ++i) past[i] = __shfl_up(past[i], 1, 64);
            dg += A + end + (l > 0 ? B : 0.f) +
                  (l >= 48 || l == 0 ? 0.f : l >= 32 ? past[2] : l >= 16 ? past[1] : past[0]);
            if (tl < a.T) {
                const int64_t out = ((int64_t)b * a.T + tl) * a.Hv + h;
                dbeta[out] = tl < len ? dots[0][1][l] + dots[1][1][l] : 0.f;
                dgate[out] = tl < len ? dg : 0.f;
            }
        }
#pragma unroll
        for (int t = 0; t < HT; ++t) {
            if (GROUP) {
                dq_sum[t] += a.scale * aq[t];
                dk_sum[t] += ar[t] + beta * hh[t];
            } else {
                dq_sum[t] = a.scale * aq[t];
                dk_sum[t] = ar[t] + beta * hh[t];
            }
        }
    }
    // rows past the length are 0, since nothing there was read
    const int64_t stride = (int64_t)a.Hk * a.dk, out = ((int64_t)b * a.T + t0) * stride + hk * a.dk;
    const Buffer dq_rows = Rows<T>::chunk(dq + out, stride, a.T - t0),
                 dk_rows = Rows<T>::chunk(dk + out, stride, a.T - t0);
#pragma unroll
    for (int i = 0; i < HT; ++i) {
        const int d = 16 * (tile0 + i) + c;
        Rows<T> rows;
        rows.set(stride, 4 * w + g, d, d < a.dk);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            rows.store(from_f32<T>(dq_sum[i][r]), dq_rows, 0, r);
            rows.store(from_f32<T>(dk_sum[i][r]), dk_rows, 0, r);
        }
    }
}

template <typename T, int DK>
hipError_t grad_t(const DeltaArgs &a, const ChunkRange &cr, const DeltaBackward &f,
                  const unsigned char *ws_key, const unsigned char *ws_head, hipStream_t s) {
    if (cr.count == 0) return hipSuccess;
    const bool vec_o = ((f.ob | f.ot | f.oh | a.dv) % 4 == 0) &&
                       reinterpret_cast<uintptr_t>(f.grad_o) % (4 * sizeof(T)) == 0;
    const dim3 grid(cr.count, a.Hk, a.B);
    auto kernel = a.Hv > a.Hk ? delta_grad_kernel<T, DK, true> : delta_grad_kernel<T, DK, false>;
    kernel<<<grid, 512, 0, s>>>(
        a, cr, rows_aligned(a, sizeof(T)), vec_o, ws_key, ws_head, reinterpret_cast<const T *>(f.grad_o), f.ob, f.ot, f.oh,
        reinterpret_cast<T *>(f.dq), reinterpret_cast<T *>(f.dk), f.dbeta, f.dgate, f.save_s,
        f.save_w, f.ws_ds, f.ws_dr);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grad(int dtype, const DeltaArgs &a, const ChunkRange &cr,
                             const DeltaBackward &f, const unsigned char *ws_key,
                             const unsigned char *ws_head, hipStream_t s) {
    return SLA_DELTA_DISPATCH(grad_t, a, cr, f, ws_key, ws_head, s);
}

}  // namespace sla
