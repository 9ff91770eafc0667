// ssd_linear_tc.cu -- the scan of linear attention on tcgen05 (bf16, DK and DV of 64 or 128).
//
// A CTA walks one segment of one (sequence, head) row in blocks of 128 tokens. With l the head's
// decay, i and j tokens of the block counted in scan order, n its tokens and S [DV][DK] the state
// that enters it:
//   o_i = c sum_{j <= i} l^{i-j} u (q_i . k_j) v_j + c l^{i+1} S q_i
//   S  <- l^n S + sum_j l^{n-1-j} u v_j k_j^T
// (backwards the entering state has had its decay already: l^i S q_i, and l^n S + sum l^{n-j} u v_j k_j^T
// leaves, decayed for the next block). Four products a block, all M = 128:
//   QK     [i][j]  = Q K^T                       A, B: the TMA tiles, K-major
//   inter  [i][d]  = Q S^T                       B: S in two bf16 terms, written by the state warps
//   U      [d][e]  = (w V)^T K                   A: w V transposed, in TMEM; B: the K tile, MN-major
//   intra  [i][d]  = P V                         A: the decayed scores P in TMEM; B: the V tile, MN-major
// S stays in fp32 registers, S = l^n S + U, and w V is taken as the sum of three bf16 (24 bits), so
// that the state is as exact as its fp32 sums. P and the operand copy of S are sums of two bf16 (16
// bits): o is rounded once, when it is stored. With one term each, o's error against 64 bits was 1.4
// times that of its rounding (rms 2.35e-3 of the values, now 1.66e-3); the second costs a third more matrix
// instructions (1 x 2048 x 148 heads of 128 69 -> 82 us).
//
// One CTA per SM, which takes segment after segment; a row that is cut into several has their own
// states computed first (the same kernel without q and o) and joined by a small kernel between.
// Five warpgroups, so that the next block's (and the next segment's) loads, w V and scores are under
// way while this one's state and outputs are finished; registers are moved to the one that holds a
// tile in them (setmaxnreg):
//   0    outputs, a row i each: scores -> P; inter times c l^{i+1}, in place, for intra to add to; then
//        o, staged over the block's own tiles for a TMA store
//   1    state, a row d each: S += U, and its operand copy, 32 columns at a time in two slots in turn
//   2, 3 w V: V's tile transposed by ldmatrix, times w, into TMEM, 32 tokens at a time in a slot each
//   4    a warp for the list of segments (where each lies and its head's powers of l, one segment ahead)
//        and their TMA loads, one for the stores, one for the MMAs of the outputs and one for those of the
//        state, which would otherwise wait for one another
// TMEM columns: QK and, in its place, both terms of P; one output tile; U; the two slots of w V. The loops are
// kept rolled where registers allow: the warpgroups' code competes for the instruction cache (scores
// unrolled by four: 106 us where 72 are). Nothing may spill: beside 227 KB of shared memory the L1 has some
// 16 KB left, and a reload waits behind the tiles.
//
// Measured: 1 x 2048 tokens x 148 heads of 128, a row per SM, 84 us (3.9 TB/s of operands): 5.2 us a block,
// of which 2.3 are matrix instructions and 2.5 HBM. With few rows the chain of one block bounds it, 3.8-3.9
// us (2.9 for 64 x 64), and a segment's start and end, some 6. Tried: S's copy made column by column as U
// is added (1 x 8192 x 32 heads on 8, backward: 346 us, 327 as it is); with one term of P and S, when it
// took 69 us: P in columns of its own with w V in slots of 16 tokens, the next block's QK before this one's
// intra (82 us); scores and outputs on two warpgroups, w V on one (82).
//
// No decay factor is ever above 1: every score is multiplied by its own l^{i-j}, from a table.
//
// Scores of tokens that do not see one another are selected away, whatever q and k hold; but their zeros meet v in
// P V. w V's warps, which look at every value of v, tell the outputs' of a block with values that are not finite,
// and those keep them out of the product (one packed product for each pair of values and a barrier a block: 82 ->
// 84 us in the case above, 64 x 64 57 -> 61).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>

#include "../../include/ssd_mixer.h"
#include "ssd_common.cuh"
#include "ssd_linear.h"
#include "ssd_pdl.cuh"
#include "ssd_profile.h"
#include "ssd_tc_util.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kB = 128;                  // tokens per block
constexpr int kThreads = 640;
constexpr uint32_t kAtom = 128 * 128;    // one [128 rows][128 bytes] swizzled tile
constexpr uint32_t kSmemMax = 232448;
constexpr long long kWait = 4000000000LL;   // ~2 s at 2 GHz
constexpr uint32_t kColP = 0, kColO = 128, kColU = 256, kColV = 384;
constexpr int kSub = 32;                 // tokens of one slot of w V
constexpr uint32_t kSlotCols = 64;       // its TMEM columns: three terms of 16, and 16 unused
// Registers per thread of the warpgroups (outputs; state; the two of w V; the last); they share what
// the launch gave them (640 x 96).
constexpr int kRegsOut = 88, kRegsState = 200, kRegsV = 72, kRegsCtl = 48;
static_assert(kRegsOut + kRegsState + 2 * kRegsV + kRegsCtl <= 5 * 96, "more registers than the launch's");

template <int DK, int DV, bool STATES>
struct Cfg {
    static constexpr uint32_t kQ = STATES ? 0 : kAtom * (DK / 64), kK = kAtom * (DK / 64), kV = kAtom * (DV / 64);
    static constexpr uint32_t kStage = kQ + kK + kV;
    static constexpr uint32_t kSlot = DV * 128;  // operand copy of 32 columns of S
    static constexpr uint32_t kS = STATES ? DV * DK * 2 : 2 * kSlot;   // two slots; staging of whole states
    static_assert(kS >= (uint32_t)DV * DK * 2, "staging");
    static constexpr uint32_t kTail = 2688;      // the segments' powers and places, barriers, what is not finite
    static constexpr int kFit = (int)((kSmemMax - kS - kTail) / kStage);
    static constexpr int kStages = kFit > 4 ? 4 : kFit;
    static_assert(kStages >= 2, "two stages");
    static constexpr uint32_t kOffS = kStages * kStage, kOffWork = kOffS + kS, kOffBar = kOffWork + 2 * 1072;
    static constexpr uint32_t kSmem = kOffWork + kTail;
};

// One segment of one scan, as the list warp leaves it for the others.
struct Work {
    float pow[256];      // l^{|e - 127|}
    float log_l;
    int n;               // tokens; -1: the list has ended
    int row0, scan, head, slot;
    int flags;
    int item;            // seg_states index
};
enum : int { kFirstInit = 1, kSplit = 2, kFinal = 4 };   // from an initial state; one of several segments; the scan's last
static_assert(sizeof(Work) <= 1072, "room for two");

struct ScanMaps {
    CUtensorMap q, k, v, o;
};
struct TcArgs {
    LinearCall c;
    LinearScan s[kMaxScans];
    int nscans;
    // o of every scan fits over q's tiles, so that k's and v's are free as soon as the block's MMAs are
    // done; otherwise o takes k's and v's place too, and the state's MMAs stay a block behind the outputs
    bool early;
};
struct TcMaps {
    ScanMaps m[kMaxScans];
};

// MN-major operand in the 128-byte swizzled layout: rows of 64 elements along M or N (128 bytes), one
// per K index. 8 rows make an atom of 1024 bytes; the next 64 elements along M or N start kAtom on.
__device__ __forceinline__ uint64_t sdesc_sw128_mn(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(kAtom >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}
// Barrier `id` of n threads; true if `p` is in all of them.
__device__ __forceinline__ bool named_all(int id, int n, bool p)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbarrier.cta.red.and.pred b, %2, %3, a;\n\tselp.u32 %0, 1, 0, b;\n\t}\n"
                 : "=r"(r)
                 : "r"((uint32_t)p), "r"(id), "r"(n)
                 : "memory");
    return r != 0;
}
// Two fp32 numbers as the sum of two pairs of bf16 each (what the first leaves is exact in fp32).
__device__ __forceinline__ void split2(float2 t, uint32_t* hi, uint32_t* lo)
{
    *hi = pack_f2(t);
    const float2 h = bf2_to_f2(*hi);
    *lo = pack_bf16x2(t.x - h.x, t.y - h.y);
}
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// Four 8 x 8 matrices of 16-bit elements, transposed: thread t holds, of each, column t / 4's
// elements in rows 2 (t % 4) and 2 (t % 4) + 1. Thread 8 m + r gives the address of matrix m's row r.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t* r)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16 TMEM lanes x 16 columns: in each group of 4 columns, thread t writes column t % 4 of lanes t / 4
// (first of the group's two registers) and t / 4 + 8 (second).
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t* v)
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// A warp's 32 rows of a state: row-major fp32 in global memory, a row a lane in registers, through 32
// rows of DK * 2 bytes of shared memory (half of the columns at a time, chunks of 16 bytes permuted by
// the row) so that the global side is coalesced.
template <int DK>
__device__ __forceinline__ void load_state(const float* p, unsigned char* buf, int lane, float* S)
{
    constexpr int kC = DK / 8;                    // 16-byte chunks of half a row
    // all loads first, into the registers that the rows will take: one latency, not one for every few
#pragma unroll
    for (int x = 0; x < 2 * kC; ++x) {
        const int at = (x % kC) * 32 + lane, r = at / kC, ch = at % kC;
        const float4 v = *reinterpret_cast<const float4*>(p + (int64_t)r * DK + (x / kC) * (DK / 2) + ch * 4);
        S[4 * x] = v.x; S[4 * x + 1] = v.y; S[4 * x + 2] = v.z; S[4 * x + 3] = v.w;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float* o = S + half * (DK / 2);
#pragma unroll
        for (int x = 0; x < kC; ++x) {
            const int at = x * 32 + lane, r = at / kC, ch = at % kC;
            *reinterpret_cast<float4*>(buf + r * (DK * 2) + ((ch ^ (r & 7)) << 4)) = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
        __syncwarp();
#pragma unroll
        for (int ch = 0; ch < kC; ++ch) {
            const float4 v = *reinterpret_cast<const float4*>(buf + lane * (DK * 2) + ((ch ^ (lane & 7)) << 4));
            o[4 * ch] = v.x; o[4 * ch + 1] = v.y; o[4 * ch + 2] = v.z; o[4 * ch + 3] = v.w;
        }
        __syncwarp();
    }
}
template <int DK>
__device__ __forceinline__ void store_state(float* p, unsigned char* buf, int lane, const float* S)
{
    constexpr int kC = DK / 8;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int ch = 0; ch < kC; ++ch) {
            const float* v = S + half * (DK / 2) + ch * 4;
            *reinterpret_cast<float4*>(buf + lane * (DK * 2) + ((ch ^ (lane & 7)) << 4)) = make_float4(v[0], v[1], v[2], v[3]);
        }
        __syncwarp();
#pragma unroll 4
        for (int x = lane; x < 32 * kC; x += 32) {
            const int r = x / kC, ch = x % kC;
            *reinterpret_cast<float4*>(p + (int64_t)r * DK + half * (DK / 2) + ch * 4) =
                *reinterpret_cast<const float4*>(buf + r * (DK * 2) + ((ch ^ (r & 7)) << 4));
        }
        __syncwarp();
    }
}

template <int DK, int DV, bool STATES>
__global__ void __launch_bounds__(kThreads, 1) linear_tc_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ TcMaps maps)
{
    using C = Cfg<DK, DV, STATES>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const LinearCall& c = a.c;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // warp: uniform, as the compiler sees
    const uint32_t sb = smem_u32(smem);
    if (sb & 1023u) {
        pdl_follow();
        if (c.clear_status && blockIdx.x == 0 && tid == 0) *c.status = kDevOk;
        if (tid == 0) set_device_status(c.status, kDevSmemMisaligned);
        return;
    }
    Work* works = reinterpret_cast<Work*>(smem + C::kOffWork);
    static_assert(C::kOffBar >= C::kOffWork + 2 * sizeof(Work) && C::kOffBar % 8 == 0, "work slots");
    const uint32_t bar0 = sb + C::kOffBar;
    auto q_full = [&](int i) { return bar0 + 8 * i; };
    auto q_empty = [&](int i) { return bar0 + 32 + 8 * i; };
    auto kv_full = [&](int i) { return bar0 + 64 + 8 * i; };
    auto kv_empty = [&](int i) { return bar0 + 96 + 8 * i; };
    auto v_ready = [&](int i) { return bar0 + 128 + 8 * i; };
    auto v_free = [&](int i) { return bar0 + 144 + 8 * i; };
    auto w_full = [&](int i) { return bar0 + 160 + 8 * i; };
    auto w_empty = [&](int i) { return bar0 + 176 + 8 * i; };
    // by stage, as the warp that waits may be more than a block behind
    auto o_staged = [&](int i) { return bar0 + 264 + 8 * i; };
    const uint32_t qk_done = bar0 + 192, p_ready = bar0 + 200, inter_done = bar0 + 208, inter_read = bar0 + 216,
                   intra_done = bar0 + 224, o_free = bar0 + 232, u_done = bar0 + 240, u_free = bar0 + 248;
    // by slot of S's operand copy
    auto s_ready = [&](int i) { return bar0 + 296 + 8 * i; };
    auto s_free = [&](int i) { return bar0 + 312 + 8 * i; };
    // by stage: w V's warps may be some blocks ahead of the outputs
    auto v_seen = [&](int i) { return bar0 + 328 + 8 * i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 360);
    // bad[i & 7] = i + 1: v of block i has values that are not finite. They are at most kStages + 1 blocks ahead of
    // its reader. from[d]: where in the block column d's first lies.
    int* bad = reinterpret_cast<int*>(smem + C::kOffBar + 368);
    unsigned char* from = smem + C::kOffBar + 400;
    const uint32_t from_full = bar0 + 528, from_read = bar0 + 536;
    static_assert(C::kOffBar + 544 <= C::kSmem && C::kStages + 1 < 8, "barriers");
    constexpr int kReaders = STATES ? 13 : 19;   // warps that read a work slot

    if (tid == 0) {
        for (int i = 0; i < 8; ++i) bad[i] = 0;
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(q_full(i), 1);
            mbar_init(q_empty(i), 1);
            mbar_init(kv_full(i), 1);
            mbar_init(o_staged(i), 128);
            mbar_init(v_seen(i), 256);
            mbar_init(kv_empty(i), STATES ? 1 : 2);   // U's MMAs, and intra's or the stores
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(v_ready(i), 128);
            mbar_init(v_free(i), 1);
            mbar_init(w_full(i), 1);
            mbar_init(w_empty(i), kReaders);
            mbar_init(s_ready(i), 128);
            mbar_init(s_free(i), 1);
        }
        mbar_init(from_full, 128);
        mbar_init(from_read, 128);
        mbar_init(qk_done, 1);
        mbar_init(p_ready, 128);
        mbar_init(inter_done, 1);
        mbar_init(inter_read, 128);
        mbar_init(intra_done, 1);
        mbar_init(o_free, 128);
        mbar_init(u_done, 1);
        mbar_init(u_free, 128);
        fence_mbar_init();
    }
    if (warp == 17) tmem_alloc(smem_u32(tmem_slot), 512);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    pdl_follow();
    if (c.clear_status && blockIdx.x == 0 && tid == 0) *c.status = kDevOk;
    // segments of this launch, of every head and scan
    const int64_t total = (c.list ? (int64_t)c.counts[STATES ? 1 : 0] : c.items) * c.H * a.nscans;
    bool ok = true;
    // The barrier's n-th completion (from 0). A wait tells a completion from the one before it only, so
    // nobody may be two ahead of a wait for it: each barrier's next but one completion needs an arrival
    // that comes after the wait.
    auto wait = [&](uint32_t bar, int n) {
        if (ok && !mbar_wait_bounded(bar, (uint32_t)(n & 1), kWait)) ok = false;
    };
    // The k-th segment of this CTA; nullptr: there are no more, or a wait gave up, in which case all
    // the warps that meet at named barriers (`group` threads at barrier `id`) leave together.
    auto open = [&](int k, int id, int group) -> const Work* {
        wait(w_full(k & 1), k >> 1);
        ok = group > 32 ? named_all(id, group, ok) : __all_sync(0xffffffffu, ok);
        const Work* w = works + (k & 1);
        return ok && w->n >= 0 ? w : nullptr;
    };
    auto close = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive_local(w_empty(k & 1));
    };
    // Blocks of a segment in scan order: block x of it, and that block's tokens.
    auto block = [&](bool rev, int nb, int x) { return rev ? nb - 1 - x : x; };
    auto tokens = [&](int n, int b) { return min(n - b * kB, kB); };

    if (warp >= 8 && warp < 16) {
        // ------------------------------------------------------------------ w V
        // two warpgroups, every other sub-block (and slot) each
        regs_down<kRegsV>();
        const int first = warp < 12 ? 0 : 1;
        const int q = warp & 3;                                    // TMEM lanes, and rows d, 32 q ..
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + kColV;
        const bool mine = 32 * q < DV;
        if (!mine) {                                               // lanes past DV: zeros, once
            uint32_t zero[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) zero[x] = 0;
#pragma unroll
            for (uint32_t x = 0; x < 2 * kSlotCols; x += 16) tmem_st16(lanes + x, zero);
            tmem_wait_st();
        }
        int i = 0;                                                 // blocks so far
        for (int k = 0;; ++k) {
            const Work* wk = open(k, 3, 256);
            if (!wk) break;
            const bool rev = a.s[wk->scan].reverse;
            const float us = a.s[wk->scan].u_scale;
            const int nall = wk->n, nb = (nall + kB - 1) / kB;
            for (int x0 = 0; x0 < nb; ++x0, ++i) {
                const int st = i % C::kStages;
                const int n = tokens(nall, block(rev, nb, x0));
                const uint32_t k_off = (uint32_t)st * C::kStage + C::kQ, v_off = k_off + C::kK;
                wait(kv_full(st), i / C::kStages);
                if (n < kB && first == 0) {   // rows behind the sequence: whatever they hold must not meet a zero weight
                    for (int id = tid & 127; id < (kB - n) * 8; id += 128) {
                        const int rr = n + (id >> 3), ch = (id & 7) << 4;
#pragma unroll
                        for (int x = 0; x < DK / 64; ++x) *reinterpret_cast<uint4*>(smem + k_off + x * kAtom + rr * 128 + ch) = make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int x = 0; x < DV / 64; ++x) *reinterpret_cast<uint4*>(smem + v_off + x * kAtom + rr * 128 + ch) = make_uint4(0, 0, 0, 0);
                    }
                    named_sync(2, 128);
                    fence_async_smem();
                }
                if (n < kB) named_sync(3, 256);
                float2 seen = splat2(0.0f);          // NaN once one of v's values is infinite or NaN
#pragma unroll 1
                for (int u = first; u < kB / kSub; u += 2) {
                    const int kk = i * (kB / kSub) + u;
                    if (kk >= 2) wait(v_free(kk & 1), (kk >> 1) - 1);
                    fence_after_sync();
                    if (mine) {
                        // thread t's tokens of 8-token group x: j0 + 8 x, and the next. A short block ends a
                        // row; rows behind it are zeros by now, whatever weight they meet.
                        const int j0 = u * kSub + 2 * (lane & 3);
                        float2 w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int j = j0 + 8 * x, e = rev ? j + 1 : n - 1 - j, e1 = rev ? j + 2 : n - 2 - j;
                            w[x] = make_float2(us * wk->pow[127 + max(e, 0)], us * wk->pow[127 + max(e1, 0)]);
                        }
                        // addresses: matrix m = lane / 8 is token group m, its row lane % 8 a token
                        const uint32_t row = (uint32_t)(u * kSub + lane);
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {          // 16 rows d
                            uint32_t raw[2][4], a0[8], a1[8], a2[8];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint32_t ch = (uint32_t)(q * 4 + half * 2 + y);     // 8-column group of d
                                ldmatrix_x4_trans(sb + v_off + (ch >> 3) * kAtom + row * 128 + (((ch & 7) ^ (row & 7)) << 4), raw[y]);
                            }
#pragma unroll
                            for (int x = 0; x < 4; ++x)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const float2 v = bf2_to_f2(raw[y][x]);
                                    if (!STATES) seen = fma2(v, splat2(0.0f), seen);
                                    float2 t = mul2(v, w[x]);
                                    const uint32_t h0 = pack_f2(t);
                                    float2 b0 = bf2_to_f2(h0);
                                    t = make_float2(t.x - b0.x, t.y - b0.y);
                                    const uint32_t h1 = pack_f2(t);
                                    b0 = bf2_to_f2(h1);
                                    a0[2 * x + y] = h0;
                                    a1[2 * x + y] = h1;
                                    a2[2 * x + y] = pack_bf16x2(t.x - b0.x, t.y - b0.y);
                                }
                            const uint32_t at = lanes + ((uint32_t)(half * 16) << 16) + (uint32_t)(kk & 1) * kSlotCols;
                            tmem_st_16x128b_x4(at, a0);
                            tmem_st_16x128b_x4(at + 16, a1);
                            tmem_st_16x128b_x4(at + 32, a2);
                        }
                        tmem_wait_st();
                    }
                    fence_before_sync();
                    mbar_arrive_local(v_ready(kk & 1));
                }
                if (!STATES) {
                    if (!(seen.x == 0.0f && seen.y == 0.0f)) bad[i & 7] = i + 1;
                    mbar_arrive_local(v_seen(st));
                }
            }
            close(k);
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------------ scores and outputs
        regs_down<kRegsOut>();
        if constexpr (!STATES) {
            const int r = tid;                                     // row i of the block = TMEM lane
            const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
            int i = 0, rare = 0;                                   // blocks, and those with values that are not finite
            for (int k = 0;; ++k) {
                const Work* wk = open(k, 1, 128);
                if (!wk) break;
                const LinearScan& s = a.s[wk->scan];
                const bool rev = s.reverse, o_f32 = s.o_f32;
                const float out_scale = s.out_scale, ps = s.out_scale * s.u_scale;
                const float* tab = wk->pow + 127;                 // l^{|e|}
                const int nall = wk->n, nb = (nall + kB - 1) / kB;
                for (int x0 = 0; x0 < nb; ++x0, ++i) {
                    const int st = i % C::kStages;
                    const int b = block(rev, nb, x0), n = tokens(nall, b);
                    wait(qk_done, i);
                    fence_after_sync();
#pragma unroll 1
                    for (int m = 0; m < 4; ++m) {                  // 32 score columns at a time
                        float v[32];
                        tmem_ld32(lanes + kColP + 32 * m, v);
                        // columns x <= g forwards, x >= g that are tokens backwards, times c u l^{|g - x|}: one code
                        // for every tile and direction
                        const int g = r - 32 * m, left = n - 32 * m;
                        const uint32_t from = g <= 0 ? 0xffffffffu : (g < 32 ? 0xffffffffu << g : 0u);       // x >= g
                        const uint32_t to = g < 0 ? 0u : (g < 31 ? (2u << g) - 1u : 0xffffffffu);             // x <= g
                        const uint32_t in = left <= 0 ? 0u : (left < 32 ? (1u << left) - 1u : 0xffffffffu);
                        const uint32_t mask = rev ? from & in : to;
                        const float* t = tab + g;
                        uint32_t hi[16], lo[16];
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            const float y = v[x] * t[-x];
                            v[x] = mask >> x & 1u ? y : 0.0f;
                        }
#pragma unroll
                        for (int x = 0; x < 16; ++x) split2(mul2(splat2(ps), make_float2(v[2 * x], v[2 * x + 1])), &hi[x], &lo[x]);
                        tmem_st16(lanes + kColP + 32 * m, hi);
                        tmem_st16(lanes + kColP + 32 * m + 16, lo);
                    }
                    if (n < kB) {     // P's zeros must not meet what rows behind the sequence hold
                        unsigned char* sv = smem + (size_t)st * C::kStage + C::kQ + C::kK + (n + r) * 128;
                        if (n + r < kB)
                            for (int x = 0; x < 8 * (DV / 64); ++x) *reinterpret_cast<uint4*>(sv + (x >> 3) * kAtom + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
                        fence_async_smem();
                    }
                    tmem_wait_st();
                    fence_before_sync();
                    mbar_arrive_local(p_ready);

                    // inter's row times c l^{i+1}, back as what intra adds to
                    const int e = rev ? n - 1 - r : r + 1;
                    const float2 f = splat2(out_scale * tab[max(e, 0)]);     // rows past the sequence are not stored
                    wait(inter_done, i);
                    fence_after_sync();
#pragma unroll 1
                    for (int x = 0; x < DV; x += 32) {
                        float v[32];
                        tmem_ld32(lanes + kColO + x, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int y = 0; y < 32; y += 2) {
                            const float2 t = mul2(f, make_float2(v[y], v[y + 1]));
                            v[y] = t.x;
                            v[y + 1] = t.y;
                        }
                        tmem_st32(lanes + kColO + x, v);
                    }
                    tmem_wait_st();
                    wait(v_seen(st), i / C::kStages);
                    if (__all_sync(0xffffffffu, bad[i & 7] == i + 1)) {
                        // Zeros of P must not meet what is not finite: its place in the V tile becomes zero (w V has read
                        // it), and its column of o NaN from its token on, in scan order, for intra to add to.
                        if (rare > 0) wait(from_read, rare - 1);
                        if (r < DV) {
                            unsigned char* sv = smem + (size_t)st * C::kStage + C::kQ + C::kK + (r >> 6) * kAtom + (r & 7) * 2;
                            int at = rev ? 0 : 255;
#pragma unroll 1
                            for (int j = 0; j < n; ++j) {
                                unsigned short* v = reinterpret_cast<unsigned short*>(sv + j * 128 + ((((r & 63) >> 3) ^ (j & 7)) << 4));
                                if ((*v & 0x7f80) != 0x7f80) continue;
                                *v = 0;
                                at = rev ? j + 1 : min(at, j);
                            }
                            from[r] = (unsigned char)at;
                        }
                        fence_async_smem();
                        mbar_arrive_local(from_full);
                        wait(from_full, rare);
#pragma unroll 1
                        for (int x = 0; x < DV; x += 16) {
                            float v[16];
                            tmem_ld16(lanes + kColO + x, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int y = 0; y < 16; ++y)
                                if (rev ? r < from[x + y] : r >= from[x + y]) v[y] = __int_as_float(0x7fffffff);
                            tmem_st16(lanes + kColO + x, reinterpret_cast<const uint32_t*>(v));
                        }
                        tmem_wait_st();
                        mbar_arrive_local(from_read);
                        ++rare;
                    }
                    fence_before_sync();
                    mbar_arrive_local(inter_read);
                    wait(intra_done, i);
                    if (!a.early) wait(u_done, i);               // k and v too have been read
                    fence_after_sync();
                    unsigned char* so = smem + (size_t)st * C::kStage + r * 128;   // over the block's tiles, which are done with
#pragma unroll 1
                    for (int x = 0; x < DV; x += 32) {
                        float v[32];
                        tmem_ld32(lanes + kColO + x, v);
                        tmem_wait_ld();
                        if (o_f32) {                               // tiles of 32 columns
#pragma unroll
                            for (int y = 0; y < 8; ++y)
                                *reinterpret_cast<float4*>(so + (x / 32) * kAtom + ((y ^ (r & 7)) << 4)) =
                                    make_float4(v[4 * y], v[4 * y + 1], v[4 * y + 2], v[4 * y + 3]);
                        } else {                                   // tiles of 64
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                *reinterpret_cast<uint4*>(so + (x / 64) * kAtom + (((y + (x & 32) / 8) ^ (r & 7)) << 4)) =
                                    make_uint4(pack_bf16x2(v[8 * y], v[8 * y + 1]), pack_bf16x2(v[8 * y + 2], v[8 * y + 3]),
                                               pack_bf16x2(v[8 * y + 4], v[8 * y + 5]), pack_bf16x2(v[8 * y + 6], v[8 * y + 7]));
                        }
                    }
                    fence_before_sync();
                    mbar_arrive_local(o_free);
                    if (n < kB) {   // rows behind the sequence may be another's: plain stores of its own rows
                        named_sync(1, 128);
                        const int64_t row = wk->row0 + (int64_t)b * kB;
                        const int es = o_f32 ? 4 : 2, chunks = DV * es / 16;
                        unsigned char* dst = (unsigned char*)s.o;
                        for (int id = tid; id < n * chunks; id += 128) {
                            const int rr = id / chunks, ch = id % chunks;
                            *reinterpret_cast<uint4*>(dst + ((row + rr) * s.o_ld + (int64_t)wk->head * DV) * es + ch * 16) =
                                *reinterpret_cast<const uint4*>(so + (ch >> 3) * kAtom + (rr - r) * 128 + (((ch & 7) ^ (rr & 7)) << 4));
                        }
                    }
                    fence_async_smem();
                    mbar_arrive_local(o_staged(st));
                }
                close(k);
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------------ the state
        regs_up<kRegsState>();
        const int d = tid - 128;                                   // state row = TMEM lane
        const uint32_t lanes = tmem + ((uint32_t)((warp - 4) * 32) << 16);
        const bool mine = d < DV;
        const int64_t hs = (int64_t)DK * DV;
        unsigned char* buf = smem + C::kOffS + (size_t)(warp - 4) * 32 * (DK * 2);   // this warp's rows of the operand copy's room
        // The operand copies of the first n blocks have been read. (Not by inter_done: its last but one completion
        // is not waited for here.)
        auto copy_read = [&](int n) {
            if (n > 0)
                for (int x = 0; x < 2; ++x) wait(s_free(x), n * (DK / 64) - 1);
        };
        int i = 0;
        for (int k = 0;; ++k) {
            const Work* wk = open(k, 4, 128);
            if (!wk) break;
            const LinearScan& s = a.s[wk->scan];
            const int flags = wk->flags, nall = wk->n, nb = (nall + kB - 1) / kB;
            const bool rev = s.reverse;
            if (!STATES) copy_read(i);
            float S[DK];
#pragma unroll
            for (int e = 0; e < DK; ++e) S[e] = 0.0f;
            if (!STATES && mine) {
                if (flags & kSplit) {    // never the slot itself: the row's last segment may be rewriting it
                    load_state<DK>(s.seg_states + ((int64_t)wk->item * c.H + wk->head) * hs + (int64_t)(d - lane) * DK, buf, lane, S);
                } else if (flags & kFirstInit) {
                    const float* p = s.init + ((int64_t)wk->slot * c.H + wk->head) * hs;
                    if (s.init_cs == 1) {
                        load_state<DK>(p + (int64_t)(d - lane) * DK, buf, lane, S);
                    } else {
                        p += (int64_t)d * s.init_rs;
#pragma unroll
                        for (int e = 0; e < DK; e += 8) {   // 8 addresses at a time: more would not fit in registers
#pragma unroll
                            for (int x = 0; x < 8; ++x) S[e + x] = p[x * s.init_cs];
                            p += 8 * s.init_cs;
                            asm volatile("" : "+l"(p)::"memory");
                        }
                    }
                }
            }
            // a warp's room for whole states holds other warps' rows of the operand copy
            if (!STATES) named_sync(4, 128);
            const float g = wk->log_l;
            for (int x0 = 0; x0 < nb; ++x0, ++i) {
                if constexpr (!STATES) {     // the K-major operand of inter: rows of 32 columns of S, high terms, then low
#pragma unroll
                    for (int ch = 0; ch < DK / 32; ++ch) {
                        const int use = i * (DK / 64) + (ch >> 1);           // of slot ch & 1
                        if (use > 0) wait(s_free(ch & 1), use - 1);
                        if (mine) {
                            unsigned char* row = smem + C::kOffS + (ch & 1) * C::kSlot + d * 128;
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                uint32_t hi[4], lo[4];
#pragma unroll
                                for (int z = 0; z < 4; ++z) {
                                    const int e = 32 * ch + 8 * y + 2 * z;
                                    split2(make_float2(S[e], S[e + 1]), &hi[z], &lo[z]);
                                }
                                *reinterpret_cast<uint4*>(row + ((y ^ (d & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                                *reinterpret_cast<uint4*>(row + (((4 + y) ^ (d & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                            }
                        }
                        fence_async_smem();
                        mbar_arrive_local(s_ready(ch & 1));
                    }
                }
                const LinearDecay dec(g * (float)tokens(nall, block(rev, nb, x0)));
                const float2 f2 = splat2(dec.f), keep2 = splat2(dec.slow ? 1.0f : 0.0f);
                wait(u_done, i);
                fence_after_sync();
                float u2[2][16];
                tmem_ld16(lanes + kColU, u2[0]);
#pragma unroll
                for (int e = 0; e < DK; e += 16) {
                    float* u = u2[(e >> 4) & 1];
                    tmem_wait_ld();
                    if (e + 16 < DK) tmem_ld16(lanes + kColU + e + 16, u2[((e >> 4) + 1) & 1]);
#pragma unroll
                    for (int x = 0; x < 16; x += 2) {          // LinearDecay::step, both kinds in one code
                        const float2 S2 = make_float2(S[e + x], S[e + x + 1]);
                        const float2 t = fma2(f2, S2, fma2(keep2, S2, make_float2(u[x], u[x + 1])));
                        S[e + x] = t.x;
                        S[e + x + 1] = t.y;
                    }
                }
                fence_before_sync();
                mbar_arrive_local(u_free);
            }
            float* out = nullptr;
            if (STATES) out = s.seg_states + ((int64_t)wk->item * c.H + wk->head) * hs;
            else if ((flags & kFinal) && s.final_state) out = s.final_state + ((int64_t)wk->slot * c.H + wk->head) * hs;
            if (out) {
                if (!STATES) copy_read(i);
                if (mine) store_state<DK>(out + (int64_t)(d - lane) * DK, buf, lane, S);
            }
            close(k);
        }
    } else {
        // ------------------------------------------------------------------ one warp each
        regs_down<kRegsCtl>();
        if (warp == 16) {                                          // the list of segments, and their loads
            int64_t w = blockIdx.x;
            // The CTA's next segment: its first, then whichever no CTA has taken (lengths differ).
            auto next = [&]() {
                int64_t t = total;
                if (gridDim.x < total) {
                    if (lane == 0) t = (int64_t)gridDim.x + atomicAdd(c.taken + (STATES ? 0 : 1), 1);
                    t = __shfl_sync(0xffffffffu, t, 0);
                }
                return t;
            };
            // the CTA's k-th segment into its slot; false after the last
            auto list = [&](int k) {
                LinearItem it{};
                int z = 0, h = 0;
                int64_t item = 0;
                bool rev = false;
                for (;; w = next()) {
                    if (w >= total) break;
                    z = (int)(w % a.nscans);
                    h = (int)(w / a.nscans % c.H);
                    rev = a.s[z].reverse;
                    item = w / a.nscans / c.H;
                    if (c.list) {
                        const int2 e = c.list[(STATES ? c.items : 0) + item];
                        linear_packed_item(c, e.x, e.y, &it);
                        item = linear_packed_first(c, e.x) + e.y;
                    } else {
                        linear_item(c, item, &it);
                        // pieces of the scan's last segment: nothing follows it
                        if (STATES && (rev ? it.seg < c.sub : it.seg / c.sub == (it.nseg - 1) / c.sub)) continue;
                        if (!STATES && c.sub > 1) {        // the first in scan order of the segment's pieces
                            const int64_t piece = c.seg_tokens / c.sub, pieces = (c.L + piece - 1) / piece;
                            const int64_t p = it.seg * c.sub + (rev ? c.sub - 1 : 0);
                            item = it.seq * pieces + (p < pieces ? p : pieces - 1);
                        }
                    }
                    break;
                }
                // segment states: pieces of this launch, or of the states' pass before it
                const bool end = w >= total ||
                                 !SSD_IN_BOUNDS(c.status, linear_in_bounds(c, it) && (it.nseg == 1 || item < (STATES ? c : linear_pieces(c)).items));
                if (k >= 2) wait(w_empty(k & 1), (k >> 1) - 1);
                ok = __all_sync(0xffffffffu, ok);
                Work* wk = works + (k & 1);
                if (!end) {
                    // l^e in fp32: g e as the sum of a product and its rounding error
                    const float g = linear_log_decay(c.log_decay, h);
                    auto power = [&](int e) {
                        const float p = g * (float)e;
                        return expf(p) * (1.0f + fmaf(g, (float)e, -p));
                    };
#pragma unroll 1
                    for (int e = lane; e < 256; e += 32) wk->pow[e] = power(abs(e - 127));
                    if (lane == 0) {
                        const bool init = linear_has_init(c, a.s[z], it.seq), split = it.nseg > 1;
                        wk->log_l = g;
                        wk->row0 = (int)it.row0;
                        wk->scan = z;
                        wk->head = h;
                        wk->slot = (int)it.slot;
                        wk->item = (int)item;
                        wk->flags = (init ? kFirstInit : 0) | (split ? kSplit : 0) |
                                    ((rev ? it.seg == 0 : it.seg == it.nseg - 1) ? kFinal : 0);
                        if (!STATES && (init || split)) {      // the state that enters, on its way to L2 by the time it is wanted
                            const float* p = split ? a.s[z].seg_states + (item * c.H + h) * (int64_t)(DK * DV)
                                                   : a.s[z].init + (it.slot * c.H + h) * (int64_t)(DK * DV);
                            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(DK * DV * 4) : "memory");
                        }
                    }
                }
                if (lane == 0) wk->n = end ? -1 : (int)it.n;
                __syncwarp();
                if (lane == 0) mbar_arrive_local(w_full(k & 1));
                if (!end) w = next();
                return !end && ok;
            };
            int i = 0;
            for (int k = 0; list(k); ++k) {
                if (lane == 0) {
                    const Work* wk = works + (k & 1);
                    const LinearScan& s = a.s[wk->scan];
                    const ScanMaps& m = maps.m[wk->scan];
                    const int nb = (wk->n + kB - 1) / kB, h = wk->head, row0 = wk->row0;
                    const int cq = h / s.q_share * DK, ck = h / s.k_share * DK, cv = h / s.v_share * DV;
                    for (int x0 = 0; x0 < nb; ++x0, ++i) {
                        const int st = i % C::kStages;
                        const uint32_t dst = sb + (uint32_t)st * C::kStage;
                        const int row = row0 + block(s.reverse, nb, x0) * kB;
                        if (i >= C::kStages) wait(kv_empty(st), i / C::kStages - 1);
                        if (!ok) break;
                        mbar_arrive_expect_tx(kv_full(st), C::kK + C::kV);
                        for (int x = 0; x < DV / 64; ++x)
                            tma_load_3d(dst + C::kQ + C::kK + x * kAtom, &m.v, cv + 64 * x, row, 0, kv_full(st));
                        for (int x = 0; x < DK / 64; ++x)
                            tma_load_3d(dst + C::kQ + x * kAtom, &m.k, ck + 64 * x, row, 0, kv_full(st));
                        if constexpr (!STATES) {
                            if (i >= C::kStages) wait(q_empty(st), i / C::kStages - 1);
                            if (!ok) break;
                            mbar_arrive_expect_tx(q_full(st), C::kQ);
                            for (int x = 0; x < DK / 64; ++x)
                                tma_load_3d(dst + x * kAtom, &m.q, cq + 64 * x, row, 0, q_full(st));
                        }
                    }
                }
                __syncwarp();
            }
            // nothing is in flight when the block ends, whatever gave up
            if (lane == 0)
                for (int x = max(0, i - C::kStages); x < i; ++x) {
                    mbar_wait_bounded(kv_full(x % C::kStages), (uint32_t)(x / C::kStages & 1), kWait);
                    if (!STATES) mbar_wait_bounded(q_full(x % C::kStages), (uint32_t)(x / C::kStages & 1), kWait);
                }
        } else if (warp == 17 && !STATES) {                        // MMAs of the outputs: the warp waits, one lane issues
            const bool leader = elect_one();
            int i = 0;
            for (int k = 0;; ++k) {
                const Work* wk = open(k, 0, 32);
                if (!wk) break;
                const int nb = (wk->n + kB - 1) / kB;
                close(k);
                for (int x0 = 0; x0 < nb; ++x0, ++i) {
                    const int st = i % C::kStages;
                    const uint32_t sq = sb + (uint32_t)st * C::kStage, sk = sq + C::kQ, sv = sk + C::kK;
                    // descriptors count addresses in 16 bytes
                    const uint64_t qd = sdesc_sw128(sq), kd = sdesc_sw128(sk), vmn = sdesc_sw128_mn(sv);
                    wait(kv_full(st), i / C::kStages);
                    wait(q_full(st), i / C::kStages);
                    fence_after_sync();
                    if (leader) {
#pragma unroll
                        for (int x = 0; x < DK / 16; ++x) {
                            const uint64_t at = ((x >> 2) * kAtom + (x & 3) * 32) >> 4;
                            mma_bf16(tmem + kColP, qd + at, kd + at, idesc_bf16(128, 128, 0, 0), x > 0);
                        }
                        mma_commit(qk_done);
                    }
                    __syncwarp();
                    if (i > 0) wait(o_free, i - 1);
#pragma unroll
                    for (int ch = 0; ch < DK / 32; ++ch) {
                        wait(s_ready(ch & 1), i * (DK / 64) + (ch >> 1));
                        fence_after_sync();
                        if (leader) {
                            const uint64_t sd = sdesc_sw128(sb + C::kOffS + (ch & 1) * C::kSlot);
#pragma unroll
                            for (int y = 0; y < 4; ++y) {                    // two steps of 16 columns, high terms and low
                                const int x = 2 * ch + (y & 1);
                                mma_bf16(tmem + kColO, qd + (((x >> 2) * kAtom + (x & 3) * 32) >> 4), sd + (y * 32 >> 4),
                                         idesc_bf16(128, DV, 0, 0), ch + y > 0);
                            }
                            mma_commit(s_free(ch & 1));
                            if (ch == DK / 32 - 1) mma_commit(inter_done);
                        }
                        __syncwarp();
                    }
                    wait(p_ready, i);
                    wait(inter_read, i);
                    fence_after_sync();
                    if (leader) {
#pragma unroll
                        for (int x = 0; x < kB / 16; ++x)
#pragma unroll
                            for (int t = 0; t < 2; ++t)
                                mma_bf16_ts(tmem + kColO, tmem + kColP + (x >> 1) * 32 + t * 16 + (x & 1) * 8, vmn + (uint64_t)(x * 2048 >> 4),
                                            idesc_bf16(128, DV, 0, 1), 1);
                        mma_commit(intra_done);
                        if (a.early) mma_commit(kv_empty(st));
                    }
                    __syncwarp();
                }
            }
            if (i > 0) mbar_wait_bounded(intra_done, (uint32_t)((i - 1) & 1), kWait);
        } else if (warp == 18 && !STATES) {                        // stores
            int i = 0;
            for (int k = 0;; ++k) {
                const Work* wk = open(k, 0, 32);
                if (!wk) break;
                if (lane == 0) {
                    const LinearScan& s = a.s[wk->scan];
                    const CUtensorMap* m = &maps.m[wk->scan].o;
                    const int per = s.o_f32 ? 32 : 64, nb = (wk->n + kB - 1) / kB, c0 = wk->head * DV;
                    for (int x0 = 0; x0 < nb; ++x0, ++i) {
                        const int st = i % C::kStages, b = block(s.reverse, nb, x0);
                        wait(o_staged(st), i / C::kStages);
                        if (tokens(wk->n, b) == kB) {
                            for (int x = 0; x < DV / per; ++x)
                                tma_store_3d(m, sb + (uint32_t)st * C::kStage + x * kAtom, c0 + per * x, wk->row0 + b * kB, 0);
                            bulk_commit();
                            bulk_wait_read_all();
                        }
                        mbar_arrive_local(q_empty(st));
                        if (!a.early) mbar_arrive_local(kv_empty(st));
                    }
                }
                close(k);
            }
            if (lane == 0) bulk_wait_all();
        } else if (warp == 19) {                                   // MMAs of the state, whenever their operands are there
            const bool leader = elect_one();
            int i = 0;
            for (int k = 0;; ++k) {
                const Work* wk = open(k, 0, 32);
                if (!wk) break;
                const int nb = (wk->n + kB - 1) / kB;
                close(k);
                for (int x0 = 0; x0 < nb; ++x0, ++i) {
                    const int st = i % C::kStages;
                    const uint64_t kmn = sdesc_sw128_mn(sb + (uint32_t)st * C::kStage + C::kQ);
                    wait(kv_full(st), i / C::kStages);
                    if (i > 0) wait(u_free, i - 1);
                    if (!STATES && !a.early && i > 0) wait(o_free, i - 1);
#pragma unroll 1
                    for (int u = 0; u < kB / kSub; ++u) {
                        const int kk = i * (kB / kSub) + u;
                        wait(v_ready(kk & 1), kk >> 1);
                        fence_after_sync();
                        const uint32_t at = tmem + kColV + (uint32_t)(kk & 1) * kSlotCols;
                        if (leader) {
#pragma unroll
                            for (int x = 0; x < kSub / 16; ++x)
#pragma unroll
                                for (int t = 0; t < 3; ++t)
                                    mma_bf16_ts(tmem + kColU, at + t * 16 + x * 8, kmn + (uint64_t)((u * kSub + x * 16) * 128 >> 4),
                                                idesc_bf16(128, DK, 0, 1), u + x + t > 0);
                            mma_commit(v_free(kk & 1));
                            if (u == kB / kSub - 1) {
                                mma_commit(u_done);
                                mma_commit(kv_empty(st));
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            if (i > 0) mbar_wait_bounded(u_done, (uint32_t)((i - 1) & 1), kWait);
        }
    }
    if (!ok) set_device_status(c.status, kDevTimeout);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 17) tmem_dealloc(tmem, 512);
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn()
{
    static EncodeFn fn = []() -> EncodeFn {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// rows x cols of bf16 (or fp32), in boxes of 128 rows x 128 bytes, 128-byte swizzled.
bool encode_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, bool f32)
{
    EncodeFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t es = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, 1};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * es, (cuuint64_t)(rows * ld) * es};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / es), kB, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, bool STATES>
cudaError_t launch_one(const TcArgs& a, const TcMaps& m, bool follows, cudaStream_t st)
{
    using C = Cfg<DK, DV, STATES>;
    cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel<DK, DV, STATES>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    LaunchScope ls(STATES ? "linear_tc_states" : "linear_tc", st);
    const int64_t total = a.c.items * a.c.H * a.nscans, sms = device_sm_count();
    return pdl_launch(follows, linear_tc_kernel<DK, DV, STATES>, dim3((unsigned)(total < sms ? total : sms)), kThreads, C::kSmem, st, a, m);
}

template <int DK, int DV>
cudaError_t launch_shape(const TcArgs& a, const TcMaps& m, bool follows, cudaStream_t st)
{
    if (a.c.split) {
        TcArgs fine = a;
        fine.c = linear_pieces(a.c);
        cudaError_t e = launch_one<DK, DV, true>(fine, m, follows, st);
        if (e == cudaSuccess) {
            LinearScans all{};
            for (int i = 0; i < a.nscans; ++i) all.s[all.n++] = a.s[i];
            e = launch_linear_pass(fine.c, all, st);
        }
        if (e != cudaSuccess) return e;
        TcArgs after = a;
        after.c.clear_status = false;
        return launch_one<DK, DV, false>(after, m, true, st);
    }
    return launch_one<DK, DV, false>(a, m, follows, st);
}

}  // namespace

bool linear_tc_supported(const LinearScan& s, int act)
{
    return act == SSD_BF16 && (s.DK == 64 || s.DK == 128) && (s.DV == 64 || s.DV == 128);
}

cudaError_t launch_linear_tc(const LinearCall& c, const LinearScan* scans, int nscans, cudaStream_t st)
{
    if (c.items == 0) return cudaSuccess;
    if (c.cu_seqlens) {
        cudaError_t e = launch_linear_list(c, st);
        if (e == cudaSuccess) e = launch_linear_short(c, scans[0], false, true, st);
        if (e != cudaSuccess) return e;
    }
    const bool queue = linear_pieces(c).items * c.H * nscans > device_sm_count();   // of any launch below
    bool done[kMaxScans] = {};
    for (int i = 0; i < nscans; ++i) {   // scans of one shape run in the same launches
        if (done[i]) continue;
        TcArgs a{};
        TcMaps m;
        memset(&m, 0, sizeof(m));
        a.c = c;
        a.c.clear_status = c.clear_status && !queue && i == 0 && !c.list;
        a.c.taken = c.taken + 2 * i;
        if (queue && i == 0 && !c.list) {
            const cudaError_t e = cudaMemsetAsync(c.status, 0, 256, st);
            if (e != cudaSuccess) return e;
        }
        a.early = true;
        for (int j = i; j < nscans; ++j) {
            const LinearScan& s = scans[j];
            if (done[j] || s.DK != scans[i].DK || s.DV != scans[i].DV) continue;
            done[j] = true;
            if (s.DV > s.DK || s.o_f32) a.early = false;
            a.s[a.nscans] = s;
            ScanMaps& x = m.m[a.nscans++];
            if (c.T > 0 && (!encode_rows(&x.q, s.q, c.T, (int64_t)(c.H / s.q_share) * s.DK, s.q_ld, false) ||
                            !encode_rows(&x.k, s.k, c.T, (int64_t)(c.H / s.k_share) * s.DK, s.k_ld, false) ||
                            !encode_rows(&x.v, s.v, c.T, (int64_t)(c.H / s.v_share) * s.DV, s.v_ld, false) ||
                            !encode_rows(&x.o, s.o, c.T, (int64_t)c.H * s.DV, s.o_ld, s.o_f32)))
                return cudaErrorInvalidValue;
        }
        const int dk = scans[i].DK, dv = scans[i].DV;
        const bool follows = i > 0 || c.list;    // after the call's own kernel
        const cudaError_t e = dk == 64 ? (dv == 64 ? launch_shape<64, 64>(a, m, follows, st) : launch_shape<64, 128>(a, m, follows, st))
                                       : (dv == 64 ? launch_shape<128, 64>(a, m, follows, st) : launch_shape<128, 128>(a, m, follows, st));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace ssd
