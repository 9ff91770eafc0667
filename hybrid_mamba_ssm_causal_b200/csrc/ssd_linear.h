// ssd_linear.h -- linear attention with a decay per head: one scan serves the prefill and all
// three gradients.
//
// With l = exp(log_decay[h]), a scan over the n tokens of a row keeps a state S [DV][DK] fp32:
//   forwards:   S <- l S + u v_t k_t^T;   o_t = c S q_t          (t = 0 .. n-1, S entering)
//   backwards:  S <- S + u v_t k_t^T;     o_t = c S q_t;   S <- l S   (t = n-1 .. 0)
// The prefill is the forward scan of (q, k, v). Its gradients are scans too: with dS_t = R_t,
//   dq_t = c S_t^T do_t                              forwards on (do, v, k), state S^T
//   R_t = l R_{t+1} + c do_t q_t^T, dv_t = R_t k_t   backwards on (k, q, do), state R
//   dk_t = R_t^T v_t                                 backwards on (v, do, q), state R^T
// and the state that leaves the backward scan of R is the gradient of the initial state.
#pragma once

#include "ssd_internal.h"

namespace ssd {

// One scan over every (sequence, head). Operand x of head h, token row t starts at
// x + t * x_ld + (h / x_share) * width elements.
struct LinearScan {
    const void *q, *k, *v;
    int64_t q_ld, k_ld, v_ld;
    int q_share, k_share, v_share;
    void* o;
    int64_t o_ld;
    bool o_f32;          // o is fp32 (partial gradients of shared heads), else the activation type
    int DK, DV;
    bool reverse;
    float u_scale, out_scale;
    const float* init;   // element (d, e) of head h at slot * H * DK * DV + h * DK * DV + d * init_rs + e * init_cs
    int init_rs, init_cs;
    float* final_state;  // [slot][H][DV][DK], or nullptr when not wanted; may be init itself
    float* seg_states;   // workspace: [item][H][DV][DK], used when rows are split
};

// Scans of one shape, which run in the same launches.
constexpr int kMaxScans = 3;
struct LinearScans {
    LinearScan s[kMaxScans];
    int n;
};

// What the scans of one call share.
struct LinearCall {
    int64_t b, L, T;     // sequences, tokens per row (fixed length), token rows in all
    int H, act;
    const float* log_decay;
    const int32_t *cu_seqlens, *slot_idx;   // packed sequences on slots when cu_seqlens is given
    const uint8_t* has_init;
    int64_t nslots;
    // Rows are cut into segments of seg_tokens; segment t of sequence i is item
    // i + floor(start_i / seg_tokens) + t of a packed call (distinct for any lengths), i * nseg + t
    // of a fixed-length one.
    int64_t seg_tokens, nseg, items;
    bool split;          // some row may have more than one segment
    // The states' pass of fixed-length rows works on pieces of seg_tokens / sub tokens, to fill SMs that
    // few segments would leave idle: linear_pieces(c) is the call that it sees, and seg_states is laid
    // out by those pieces.
    int sub;
    // The first 256 bytes of the workspace: the status word, and (tensor cores) how many segments the CTAs
    // have taken beyond their first, by launch. Where the counts are needed all of it is cleared
    // beforehand; otherwise the first kernel's block 0 clears the status word as it starts: a block can
    // only set it seconds later, when a wait gives up, or at its start for the reason that block 0 meets
    // too.
    int* status;
    int* taken;
    bool clear_status;
    // A packed call on the tensor cores works off lists of (sequence, segment), the longest first, made
    // by launch_linear_list: `items` entries of the main pass, then of the states' pass, and their counts.
    int2* list;
    int* counts;
};

// Who clears the status word. In the bounds-checked build blocks may set it from their start on, before block
// 0 of the same kernel would clear it.
inline cudaError_t set_clear_status(LinearCall* c, cudaStream_t st)
{
#ifdef SSD_DEBUG_BOUNDS
    c->clear_status = false;
    return clear_device_status(c->status, st);
#else
    (void)st;
    c->clear_status = true;
    return cudaSuccess;
#endif
}

SSD_HD inline LinearCall linear_pieces(const LinearCall& c)
{
    LinearCall f = c;
    if (c.sub > 1) {
        f.seg_tokens = c.seg_tokens / c.sub;
        f.nseg = (c.L + f.seg_tokens - 1) / f.seg_tokens;
        f.items = c.b * f.nseg;
    }
    return f;
}

// Longest supported per-call counts keep every index in 32-bit grid dimensions.
bool linear_tc_supported(const LinearScan& s, int act);
// nscans scans (1, or the 3 of a backward pass) in as few launches as the split allows.
cudaError_t launch_linear_tc(const LinearCall& c, const LinearScan* scans, int nscans, cudaStream_t st);
cudaError_t launch_linear_simt(const LinearCall& c, const LinearScan* scans, int nscans, cudaStream_t st);
// The states entering every segment of rows that have more than one, from the pieces' own states; c as
// linear_pieces gives it.
cudaError_t launch_linear_pass(const LinearCall& c, const LinearScans& scans, cudaStream_t st);   // follows a launch
// (follows a launch)
cudaError_t launch_linear_group_sum(const float* in, void* out, int64_t ld, int64_t rows, int G, int r, int D, int act,
                                    cudaStream_t st);
// Forward scans of rows of at most kLinearShort tokens (one: of exactly one token each) on CUDA cores;
// in a packed call, of those rows alone. Rows of 8 tokens (9: the tensor-core scan's whole block): 64
// sequences of 32 heads of 128 99 us (123), of 64 23 (80); 1 sequence of 8 heads of 64 6.0 (8.7).
constexpr int kLinearShort = 8;
cudaError_t launch_linear_list(const LinearCall& c, cudaStream_t st);
// `follows`: it comes after another kernel of the call.
cudaError_t launch_linear_short(const LinearCall& c, const LinearScan& s, bool one, bool follows, cudaStream_t st);
// Segment length of a call's scans, and the pieces of a segment in the states' pass.
int64_t linear_segment_tokens(bool tc, int64_t b, int64_t L, int64_t T, bool packed, int H, int nscans, int DK, int DV, int sms,
                              int* sub);

#ifdef __CUDACC__

// lambda = exp(log_decay): -inf (no memory) is taken as exp(-1e4) = 0 so that 0 * log_decay is 0. NaN stays
// NaN (fmaxf would drop it).
__device__ __forceinline__ float linear_log_decay(const float* log_decay, int h)
{
    const float g = log_decay[h];
    return g < -1e4f ? -1e4f : g;
}

// One step of a decayed sum, S <- l S + add. A slow decay (l > 1/2) is taken as S + (l - 1) S: l
// itself rounded to fp32 would be off by up to 2^-25 in every step, the same way each time, 3e-3
// over the 1e5 steps that l = 1 - 1e-5 remembers. A fast one is taken as it stands, where S + add
// would lose what is small next to the forgotten S.
struct LinearDecay {
    bool slow;
    float f;       // l - 1, or l
    __device__ __forceinline__ explicit LinearDecay(float log_l) : slow(log_l > -0.6931472f), f(slow ? expm1f(log_l) : expf(log_l)) {}
    __device__ __forceinline__ float step(float S, float add) const { return fmaf(f, S, slow ? S + add : add); }
};

// The segment that `item` stands for: sequence, its state slot, first token row, tokens, position
// in the row. False: the item stands for none (or its slot is outside 0 .. nslots-1).
struct LinearItem {
    int64_t seq, slot, row0;
    int64_t n, seg, nseg;
};
// Segment `seg` of sequence `seq` of a packed call. The rows are clamped to the packed ones, so that no
// cu_seqlens can reach outside them.
__device__ __forceinline__ bool linear_packed_item(const LinearCall& c, int64_t seq, int64_t seg, LinearItem* it)
{
    int64_t start = c.cu_seqlens[seq], end = c.cu_seqlens[seq + 1];
    it->slot = c.slot_idx ? (int64_t)c.slot_idx[seq] : seq;
    start = start < 0 ? 0 : (start > c.T ? c.T : start);
    end = end < start ? start : (end > c.T ? c.T : end);
    const int64_t len = end - start;
    it->seq = seq;
    it->seg = seg;
    it->nseg = len > 0 ? (len + c.seg_tokens - 1) / c.seg_tokens : 1;
    it->row0 = start + seg * c.seg_tokens;
    const int64_t left = len - seg * c.seg_tokens;
    it->n = left < c.seg_tokens ? left : c.seg_tokens;
    return seg >= 0 && seg < it->nseg && it->slot >= 0 && it->slot < c.nslots;
}
__device__ __forceinline__ int64_t linear_packed_first(const LinearCall& c, int64_t seq)   // item of its segment 0
{
    int64_t s = c.cu_seqlens[seq];
    s = s < 0 ? 0 : (s > c.T ? c.T : s);
    return seq + s / c.seg_tokens;
}
__device__ __forceinline__ bool linear_item(const LinearCall& c, int64_t item, LinearItem* it)
{
    if (c.cu_seqlens) {
        // the largest i with i + floor(start_i / seg_tokens) <= item
        int64_t lo = 0, hi = c.b - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (linear_packed_first(c, mid) <= item) lo = mid;
            else hi = mid - 1;
        }
        return linear_packed_item(c, lo, item - linear_packed_first(c, lo), it);
    }
    it->seq = it->slot = item / c.nseg;
    it->seg = item - it->seq * c.nseg;
    it->nseg = c.nseg;
    it->row0 = it->seq * c.L + it->seg * c.seg_tokens;
    const int64_t left = c.L - it->seg * c.seg_tokens;
    it->n = left < c.seg_tokens ? left : c.seg_tokens;
    return it->seg < it->nseg;
}
// Its rows and its slot lie inside the call's.
__device__ __forceinline__ bool linear_in_bounds(const LinearCall& c, const LinearItem& it)
{
    return it.n >= 0 && it.row0 >= 0 && it.row0 + it.n <= c.T && it.slot >= 0 && it.slot < c.nslots;
}
// Whether the sequence continues from the state in its slot.
__device__ __forceinline__ bool linear_has_init(const LinearCall& c, const LinearScan& s, int64_t seq)
{
    return s.init && !(c.has_init && c.has_init[seq] == 0);
}

#endif

}  // namespace ssd
