// C entry points of the gated delta rule: argument checks, the workspace's
// layout, and the rounds of launches.
#include <cmath>

#include "delta_chunk.h"

namespace sla {

namespace {

// Without a backward pass to follow, few tokens are walked by the recurrent
// kernel, whose time grows with them, where one chunk's hardly does, but with the
// states' size and the inputs' planes.  Tokens at which the two meet (GPU time; in
// brackets us for 8 tokens, walked and as a chunk):
//
//   heads                  16               128               512
//   128 x 128, bf16    7.1 (15.1, 13.2)  12 (18.0, 24.3)   28 (29.8, 72.7)
//    64 x  64, bf16    6.6 (13.4, 11.3)   8 (13.9, 13.7)   17 (18.6, 32.7)
//    32 x  32, bf16    6.5 (13.2, 11.2)   7 (13.4, 12.1)   11 (17.1, 21.6)
//   128 x 128, fp32    12  (12.8, 17.5)  20 (16.0, 31.7)   58 (26.7, 119)
//    64 x  64, fp32    9.3 (12.0, 13.4)  12 (12.3, 16.6)   28 (17.2, 44.5)
//    32 x  32, fp32    9.2 (11.8, 13.3)  11 (12.0, 14.6)   19 (15.6, 30.2)
bool few_tokens(const DeltaArgs &a, int dtype) {
    const int planes = dtype == SLA_F32 ? 3 : dtype == SLA_F16 ? 2 : 1;
    const double states = (double)a.B * a.Hv * a.dk * a.dv / (kMaxDk * kMaxDk);
    const double most = 4.5 + 1.5 * planes + states * (planes + 1) / 40;
    return a.T <= (most < 24 ? most : 24);
}

// A round's workspace is kept near this, so that what one launch leaves the
// next one finds in the 256 MB Infinity Cache, and yet a launch is long.  16384
// tokens of 16 heads of 128 x 128: 479 us, with 80 MB 511 and with 400 MB 583;
// training on 8192 tokens of 16 heads of 64 x 128: 648, 683 and 704 us, on 4 x 2048
// of 128 x 128 560, 617 and 554.
constexpr int64_t kRoundBytes = 160 << 20;

int64_t align256(int64_t x) { return (x + 255) & ~(int64_t)255; }

bool valid(const sla_delta_args *p) {
    return p && p->batch >= 0 && p->batch <= 65535 && p->tokens >= 0 && p->tokens <= (1 << 30) &&
           p->key_heads >= 1 && p->value_heads >= 1 && p->value_heads <= 65535 &&
           p->value_heads % p->key_heads == 0 && p->dk >= 1 && p->dk <= kMaxDk && p->dv >= 1 &&
           (int64_t)p->value_heads * p->dv <= kMaxStride &&
           (int64_t)p->key_heads * p->dk <= kMaxStride &&
           (p->dtype == SLA_F32 || p->dtype == SLA_F16 || p->dtype == SLA_BF16);
}

bool has_data(const sla_delta_args *p, bool back = false) {
    return p->batch * p->tokens == 0 ||
           (p->d_q && p->d_k && (p->d_v || back) && p->d_beta && p->d_gate);
}

// The scans address a chunk's rows of v and o in 32 bits and tell a row past
// the end by its offset.
bool valid_rows(const sla_delta_args *p, const int64_t *stride) {
    return p->tokens <= 1 || (stride[1] >= p->dv && stride[1] <= kMaxStride);
}

DeltaArgs args_of(const sla_delta_args *p) {
    DeltaArgs a;
    a.q = p->d_q, a.k = p->d_k, a.v = p->d_v, a.beta = p->d_beta, a.gate = p->d_gate;
    a.qb = p->q_stride[0], a.qt = p->q_stride[1], a.qh = p->q_stride[2];
    a.kb = p->k_stride[0], a.kt = p->k_stride[1], a.kh = p->k_stride[2];
    a.vb = p->v_stride[0], a.vt = p->v_stride[1], a.vh = p->v_stride[2];
    a.bb = p->beta_stride[0], a.bt = p->beta_stride[1], a.bh = p->beta_stride[2];
    a.gb = p->gate_stride[0], a.gt = p->gate_stride[1], a.gh = p->gate_stride[2];
    a.lengths = p->d_lengths;
    if (p->tokens <= 1) a.vt = p->dv;
    a.B = (int32_t)p->batch, a.T = (int32_t)p->tokens;
    a.Hk = p->key_heads, a.Hv = p->value_heads, a.dk = p->dk, a.dv = p->dv;
    a.scale = p->scale;
    return a;
}

int padded_dk(int dk) { return dk <= 64 ? 64 : 128; }

template <int NP, int DK>
int64_t key_bytes() { return PrepLayout<NP, DK>::kPerKeyHead; }

// Bytes of one key head's chunk and of one value head's (PrepLayout).
int64_t key_chunk_bytes(const DeltaArgs &a, int dtype) {
    const bool big = a.dk > 64;
    return dtype == SLA_F32   ? (big ? key_bytes<3, 128>() : key_bytes<3, 64>())
           : dtype == SLA_F16 ? (big ? key_bytes<2, 128>() : key_bytes<2, 64>())
                              : (big ? key_bytes<1, 128>() : key_bytes<1, 64>());
}
constexpr int64_t kHeadChunkBytes = PrepLayout<1, 64>::kPerHead;

// Where the parts of a call's workspace begin.
struct Work {
    int per_round;  // chunks
    int64_t key, head, state, ds, dr, bytes;
};

Work layout(const DeltaArgs &a, int dtype, bool back) {
    if (a.B == 0) return Work{};
    const int N = num_chunks(a), dvp = padded_dv(a.dv);
    const int64_t heads = (int64_t)a.B * a.Hv;
    const int64_t key = a.B * (int64_t)a.Hk * key_chunk_bytes(a, dtype);
    const int64_t ds = heads * padded_dk(a.dk) * dvp * 4, dr = heads * kChunk * dvp * 4;
    const int64_t chunk = key + heads * kHeadChunkBytes + (back ? ds + dr : 0);
    Work w;
    // whole turns of the chip for the kernels that take a chunk of a key head
    // per workgroup (256 CUs), at least one
    int64_t turn = (256 + (int64_t)a.B * a.Hk - 1) / ((int64_t)a.B * a.Hk), fit = kRoundBytes / chunk;
    if (turn < 8) turn = 8;
    fit = fit < turn ? turn : fit / turn * turn;
    w.per_round = (int)(fit < N ? fit : N);
    const int64_t n = w.per_round;
    w.key = 0;
    w.head = w.key + align256(n * key);
    w.state = w.head + align256(n * heads * kHeadChunkBytes);
    w.ds = w.state + (n < N ? align256(heads * a.dk * a.dv * 4) : 0);
    w.dr = w.ds + (back ? align256(n * ds) : 0);
    w.bytes = w.dr + (back ? align256(n * dr) : 0);
    return w;
}

int64_t saved_state_bytes(const DeltaArgs &a) {
    return align256((int64_t)a.B * a.Hv * num_chunks(a) * padded_dk(a.dk) * padded_dv(a.dv) * 4);
}

}  // namespace

}  // namespace sla

using namespace sla;

#define DELTA_TRY(...)                 \
    do {                               \
        hipError_t e_ = (__VA_ARGS__); \
        if (e_ != hipSuccess) {        \
            set_last_error(e_);        \
            return SLA_ERR_DEVICE;     \
        }                              \
    } while (0)

extern "C" {

int64_t sla_delta_workspace_bytes(const sla_delta_args *args, int32_t backward) {
    if (!valid(args)) return -1;
    return layout(args_of(args), args->dtype, backward != 0).bytes;
}

int64_t sla_delta_saved_bytes(const sla_delta_args *args) {
    if (!valid(args)) return -1;
    const DeltaArgs a = args_of(args);
    return saved_state_bytes(a) +
           align256((int64_t)a.B * a.Hv * num_chunks(a) * kChunk * padded_dv(a.dv) * 4);
}

sla_status sla_delta_forward(const sla_delta_args *args, const float *d_state_in,
                             float *d_state_out, void *d_o, const int64_t *o_stride,
                             void *d_saved, void *d_work, int64_t work_bytes, void *stream) {
    if (!valid(args) || !has_data(args) || !o_stride || !valid_rows(args, o_stride) ||
        !valid_rows(args, args->v_stride))
        return SLA_ERR_ARG;
    if (args->batch == 0) return SLA_OK;
    if (!d_o && args->tokens > 0) return SLA_ERR_ARG;
    const DeltaArgs a = args_of(args);
    const int dtype = args->dtype;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (!d_saved && few_tokens(a, dtype)) {
        DELTA_TRY(launch_delta_step(dtype, a, d_state_in, d_state_out, nullptr, 0, d_o, o_stride[0],
                                    o_stride[1], o_stride[2], kMaxGrowth, s));
        return SLA_OK;
    }
    const Work w = layout(a, dtype, false);
    if (work_bytes < w.bytes || (!d_work && w.bytes)) return SLA_ERR_ARG;
    unsigned char *work = static_cast<unsigned char *>(d_work);
    DeltaForward f;
    f.o = d_o, f.ob = o_stride[0], f.ot = a.T == 1 ? a.dv : o_stride[1], f.oh = o_stride[2];
    f.save_s = reinterpret_cast<float *>(d_saved);
    f.save_w = d_saved ? reinterpret_cast<float *>(static_cast<char *>(d_saved) +
                                                   saved_state_bytes(a))
                       : nullptr;
    const int N = num_chunks(a);
    float *carry = d_state_out ? d_state_out : reinterpret_cast<float *>(work + w.state);
    for (int first = 0; first < N || first == 0; first += w.per_round) {
        const ChunkRange cr{first, N - first < w.per_round ? N - first : w.per_round};
        const bool last = first + cr.count >= N;
        f.s_in = first ? carry : d_state_in;
        f.s_out = last ? d_state_out : carry;
        DELTA_TRY(launch_delta_prep(dtype, a, cr, false, work + w.key, work + w.head, s));
        DELTA_TRY(launch_delta_scan(dtype, a, cr, f, work + w.key, work + w.head, s));
        if (last) break;
    }
    return SLA_OK;
}

sla_status sla_delta_backward(const sla_delta_args *args, const void *d_saved,
                              const void *d_grad_o, const int64_t *o_stride,
                              const float *d_grad_state, void *d_dq, void *d_dk, void *d_dv,
                              float *d_dbeta, float *d_dgate, float *d_dstate, void *d_work,
                              int64_t work_bytes, void *stream) {
    if (!valid(args) || !has_data(args, true) || !o_stride || !valid_rows(args, o_stride))
        return SLA_ERR_ARG;
    if (d_dstate && d_dstate == d_grad_state) return SLA_ERR_ARG;
    if (args->batch == 0) return SLA_OK;
    if (args->tokens > 0 &&
        (!d_saved || !d_grad_o || !d_dq || !d_dk || !d_dv || !d_dbeta || !d_dgate))
        return SLA_ERR_ARG;
    const DeltaArgs a = args_of(args);
    const int dtype = args->dtype;
    const Work w = layout(a, dtype, true);
    if (work_bytes < w.bytes || (!d_work && w.bytes)) return SLA_ERR_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    unsigned char *work = static_cast<unsigned char *>(d_work);
    DeltaBackward f;
    f.grad_o = d_grad_o, f.ob = o_stride[0], f.ot = a.T == 1 ? a.dv : o_stride[1], f.oh = o_stride[2];
    f.dq = d_dq, f.dk = d_dk, f.dv = d_dv, f.dbeta = d_dbeta, f.dgate = d_dgate;
    f.save_s = reinterpret_cast<const float *>(d_saved);
    f.save_w = reinterpret_cast<const float *>(static_cast<const char *>(d_saved) +
                                               saved_state_bytes(a));
    f.ws_ds = reinterpret_cast<float *>(work + w.ds);
    f.ws_dr = reinterpret_cast<float *>(work + w.dr);
    const int N = num_chunks(a);
    float *carry = d_dstate ? d_dstate : reinterpret_cast<float *>(work + w.state);
    const int rounds = N ? (N + w.per_round - 1) / w.per_round : 1;
    for (int i = rounds - 1; i >= 0; --i) {
        const int first = i * w.per_round;
        const ChunkRange cr{first, N - first < w.per_round ? N - first : w.per_round};
        f.ds_in = i == rounds - 1 ? d_grad_state : carry;
        f.ds_out = i ? carry : d_dstate;
        DELTA_TRY(launch_delta_prep(dtype, a, cr, true, work + w.key, work + w.head, s));
        DELTA_TRY(launch_delta_scan_back(dtype, a, cr, f, work + w.key, work + w.head, s));
        DELTA_TRY(launch_delta_grad(dtype, a, cr, f, work + w.key, work + w.head, s));
    }
    return SLA_OK;
}

sla_status sla_delta_step(const sla_delta_args *args, float *d_state, int64_t n_slots,
                          const int32_t *d_slots, void *d_o, const int64_t *o_stride,
                          void *stream) {
    if (!valid(args) || !has_data(args) || !o_stride || n_slots < 0) return SLA_ERR_ARG;
    if (!d_slots && n_slots < args->batch) return SLA_ERR_ARG;
    if (args->batch == 0 || args->tokens == 0) return SLA_OK;
    if (!d_state || !d_o) return SLA_ERR_ARG;
    DELTA_TRY(launch_delta_step(args->dtype, args_of(args), d_state, d_state, d_slots, n_slots, d_o,
                                o_stride[0], o_stride[1], o_stride[2], HUGE_VALF,
                                reinterpret_cast<hipStream_t>(stream)));
    return SLA_OK;
}

}  // extern "C"
