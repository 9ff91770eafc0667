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
    // 256 bytes at the start of the workspace: the status word, and (tensor cores, more segments than
    // SMs) how many segments the CTAs of the states' and of the main pass have taken beyond their first.
    // Those calls clear all of it beforehand; others leave the status word to the first kernel's block 0,
    // as it starts: a block can only set it seconds later, when a wait gives up, or at its start for the
    // reason that block 0 meets too.
    int* status;
    int* taken;
    bool clear_status;
};

// Longest supported per-call counts keep every index in 32-bit grid dimensions.
bool linear_tc_supported(const LinearScan& s, int act);
// nscans scans (1, or the 3 of a backward pass) in as few launches as the split allows.
cudaError_t launch_linear_tc(const LinearCall& c, const LinearScan* scans, int nscans, cudaStream_t st);
cudaError_t launch_linear_simt(const LinearCall& c, const LinearScan& s, cudaStream_t st);
// The states entering every segment of rows that have more than one, from the segments' own states.
cudaError_t launch_linear_pass(const LinearCall& c, const LinearScan& s, cudaStream_t st);
cudaError_t launch_linear_group_sum(const float* in, void* out, int64_t ld, int64_t rows, int G, int r, int D, int act,
                                    cudaStream_t st);
cudaError_t launch_linear_decode(int64_t b, int H, int share, int DK, int DV, float scale, int act, const void* q,
                                 int64_t q_ld, const void* k, int64_t k_ld, const void* v, int64_t v_ld,
                                 const float* log_decay, float* state, int64_t nslots, const int32_t* slot_idx, void* o,
                                 int64_t o_ld, cudaStream_t st);
// Segment length of a call's scans.
int64_t linear_segment_tokens(bool tc, int64_t b, int64_t L, int64_t T, bool packed, int H, int nscans, int sms);

#ifdef __CUDACC__

// lambda = exp(log_decay): -inf (no memory) is taken as exp(-1e4) = 0 so that 0 * log_decay is 0.
__device__ __forceinline__ float linear_log_decay(const float* log_decay, int h) { return fmaxf(log_decay[h], -1e4f); }

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
__device__ __forceinline__ bool linear_item(const LinearCall& c, int64_t item, LinearItem* it)
{
    int64_t start, len;
    if (c.cu_seqlens) {
        // the largest i with i + floor(start_i / seg_tokens) <= item; the lengths are clamped to the
        // packed rows, so that no cu_seqlens can reach outside them
        int64_t lo = 0, hi = c.b - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            int64_t s = c.cu_seqlens[mid];
            s = s < 0 ? 0 : (s > c.T ? c.T : s);
            if (mid + s / c.seg_tokens <= item) lo = mid;
            else hi = mid - 1;
        }
        start = c.cu_seqlens[lo];
        start = start < 0 ? 0 : (start > c.T ? c.T : start);
        int64_t end = c.cu_seqlens[lo + 1];
        end = end < start ? start : (end > c.T ? c.T : end);
        len = end - start;
        it->seq = lo;
        it->seg = item - (lo + start / c.seg_tokens);
        it->nseg = len > 0 ? (len + c.seg_tokens - 1) / c.seg_tokens : 1;
        it->slot = c.slot_idx ? (int64_t)c.slot_idx[lo] : lo;
        if (it->slot < 0 || it->slot >= c.nslots) return false;
    } else {
        it->seq = it->slot = item / c.nseg;
        it->seg = item - it->seq * c.nseg;
        it->nseg = c.nseg;
        start = it->seq * c.L;
        len = c.L;
    }
    if (it->seg < 0 || it->seg >= it->nseg) return false;
    it->row0 = start + it->seg * c.seg_tokens;
    const int64_t left = len - it->seg * c.seg_tokens;
    it->n = left < c.seg_tokens ? left : c.seg_tokens;
    return true;
}
// Whether the sequence continues from the state in its slot.
__device__ __forceinline__ bool linear_has_init(const LinearCall& c, const LinearScan& s, int64_t seq)
{
    return s.init && !(c.has_init && c.has_init[seq] == 0);
}

#endif

}  // namespace ssd
