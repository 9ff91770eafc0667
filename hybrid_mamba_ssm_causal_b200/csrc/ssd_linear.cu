// ssd_linear.cu -- linear attention with a decay per head on CUDA cores: the scan for any
// supported shape and type, the state pass between segments, the sum over shared heads' gradients
// and the decode step. The tensor-core scan is ssd_linear_tc.cu.
#include <math.h>

#include <type_traits>

#include "../../include/ssd_mixer.h"
#include "ssd_common.cuh"
#include "ssd_linear.h"
#include "ssd_pdl.cuh"
#include "ssd_profile.h"
#include "ssd_tc_util.cuh"

namespace ssd {
namespace {

using tc::fma2;
using tc::mul2;
using tc::splat2;

// ---------------------------------------------------------------------------- the scan
// Token by token: the recurrence needs 4 DK DV flops a token, fewer than any chunked form, and
// keeps fp32 throughout, so fp32 activations and the shapes without a tensor-core variant use it.
// A CTA owns one segment of one (sequence, head) row; a warp owns 8 state rows (16 when DK = 16)
// in registers, its lanes along DK. Tokens come in tiles of 16 through shared memory, the next
// tile's loads in flight while the present one is used. The products S q are summed over the lanes
// by a butterfly that halves the values with each of its first three steps (9 shuffles for 8 rows).
// A token takes a warp 0.25 us (its chain of loads, sums and shuffles) and, from some three warps to a
// scheduler on, issue slots and the pipe that shared loads and shuffles have in common: 2 x 777 x 12 heads
// 64 x 32 fp32 34 us, 1 x 16384 x 32 heads of 128 2.6 ms (18 % of the rate of fp32 products).
constexpr int kTile = 16;

template <int DK>
struct SimtShape {
    static constexpr int kCols = DK >= 32 ? DK / 32 : 1;      // state columns per lane
    static constexpr int kLanes = DK / kCols;                 // lanes per state row (32, or 16)
    static constexpr int kRows = 8;                           // state rows per lane
    static constexpr int kWarpRows = kRows * (32 / kLanes);
};

// N neighbouring values of a row, aligned to their own size
template <int N>
__device__ __forceinline__ void load_row(const float* p, float* out)
{
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(p + i);
            out[i] = x.x; out[i + 1] = x.y; out[i + 2] = x.z; out[i + 3] = x.w;
        }
    } else if constexpr (N == 2) {
        const float2 x = *reinterpret_cast<const float2*>(p);
        out[0] = x.x; out[1] = x.y;
    } else {
        out[0] = *p;
    }
}
template <int N>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float* out)
{
    uint32_t w[N > 1 ? N / 2 : 1];
    if constexpr (N == 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (N == 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x; w[1] = x.y;
    } else if constexpr (N == 2) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
        out[0] = __bfloat162float(*p);
        return;
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        out[2 * i] = __uint_as_float(w[i] << 16);
        out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v)
{
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}
template <int N>
__device__ __forceinline__ void store_row(float* p, const float* v)
{
    if constexpr (N == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else if constexpr (N == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    else *p = v[0];
}

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(32 * (DV / SimtShape<DK>::kWarpRows > 0 ? DV / SimtShape<DK>::kWarpRows : 1))
    linear_scan_kernel(const LinearCall c, const LinearScans scans, bool state_only)
{
    const LinearScan& s = scans.s[blockIdx.y];
    using Sh = SimtShape<DK>;
    constexpr int kWarps = DV / Sh::kWarpRows > 0 ? DV / Sh::kWarpRows : 1;
    constexpr int kThr = 32 * kWarps;
    constexpr int kVec = Act<T>::kVec;
    constexpr int kRowVecs = (2 * DK + DV) / kVec;            // 16-byte vectors of one token's k, q, v
    constexpr int kTileVecs = kTile * kRowVecs;
    constexpr int kPer = (kTileVecs + kThr - 1) / kThr;
    __shared__ __align__(16) T s_in[kTile][2 * DK + DV];      // k, then q, then v
    __shared__ __align__(16) float s_o[kTile][DV];
    pdl_wait();
    if (c.clear_status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *c.status = kDevOk;

    const int h = blockIdx.x % c.H;
    const int64_t item = blockIdx.x / c.H;
    LinearItem it;
    if (!linear_item(c, item, &it) || !SSD_IN_BOUNDS(c.status, linear_in_bounds(c, it) && item < c.items)) return;
    // segments in scan order; the state-only pass covers all but the last of a row
    const bool last = s.reverse ? it.seg == 0 : it.seg == it.nseg - 1;
    if (state_only && last) return;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sub = lane / Sh::kLanes, l = lane % Sh::kLanes;
    const int d0 = warp * Sh::kWarpRows + sub * Sh::kRows;    // this lane's first state row
    const int e0 = l * Sh::kCols;                             // and first column
    const LinearDecay decay(linear_log_decay(c.log_decay, h));
    const int64_t hs = (int64_t)DK * DV;

    constexpr int kPairs = Sh::kRows / 2;
    float2 S[kPairs][Sh::kCols];             // two neighbouring rows in a pair: two roundings an instruction
#pragma unroll
    for (int r = 0; r < kPairs; ++r)
#pragma unroll
        for (int e = 0; e < Sh::kCols; ++e) S[r][e] = splat2(0.0f);
    const auto load_state = [&](const float* p) {    // [DV][DK]
#pragma unroll
        for (int r = 0; r < kPairs; ++r) {
            float x[Sh::kCols], y[Sh::kCols];
            load_row<Sh::kCols>(p + (d0 + 2 * r) * DK + e0, x);
            load_row<Sh::kCols>(p + (d0 + 2 * r + 1) * DK + e0, y);
#pragma unroll
            for (int e = 0; e < Sh::kCols; ++e) S[r][e] = make_float2(x[e], y[e]);
        }
    };
    if (!state_only) {
        if (it.nseg > 1) {   // never the slot itself: the row's last segment may be rewriting it
            load_state(s.seg_states + (item * c.H + h) * hs);
        } else if (linear_has_init(c, s, it.seq)) {
            const float* p = s.init + (it.slot * c.H + h) * hs;
            if (s.init_cs == 1) {
                load_state(p);                       // rows of DK
            } else {
#pragma unroll
                for (int r = 0; r < kPairs; ++r)
#pragma unroll
                    for (int e = 0; e < Sh::kCols; ++e)
                        S[r][e] = make_float2(p[(d0 + 2 * r) * s.init_rs + (e0 + e) * s.init_cs],
                                              p[(d0 + 2 * r + 1) * s.init_rs + (e0 + e) * s.init_cs]);
            }
        }
    }

    const T* kp = (const T*)s.k + (int64_t)(h / s.k_share) * DK;
    const T* qp = (const T*)s.q + (int64_t)(h / s.q_share) * DK;
    const T* vp = (const T*)s.v + (int64_t)(h / s.v_share) * DV;
    const int ntiles = (int)((it.n + kTile - 1) / kTile);
    uint4 next[kPer];
    // tile i of the segment in scan order: tokens kTile * ti ..
    auto tile_of = [&](int i) { return s.reverse ? ntiles - 1 - i : i; };
    auto fetch = [&](int i) {
        const int64_t t0 = (int64_t)tile_of(i) * kTile;
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            const int id = tid + x * kThr;
            const int tt = id / kRowVecs, w = (id % kRowVecs) * kVec;
            next[x] = make_uint4(0, 0, 0, 0);
            if (id < kTileVecs && t0 + tt < it.n) {
                const int64_t row = it.row0 + t0 + tt;
                const T* p = w < DK ? kp + row * s.k_ld + w
                                    : w < 2 * DK ? qp + row * s.q_ld + (w - DK) : vp + row * s.v_ld + (w - 2 * DK);
                next[x] = *reinterpret_cast<const uint4*>(p);
            }
        }
    };
    if (ntiles > 0) fetch(0);
    bool fresh = s.reverse;      // the first backward step has no decay
    for (int i = 0; i < ntiles; ++i) {
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            const int id = tid + x * kThr;
            if (id < kTileVecs) *reinterpret_cast<uint4*>(&s_in[id / kRowVecs][(id % kRowVecs) * kVec]) = next[x];
        }
        __syncthreads();
        if (i + 1 < ntiles) fetch(i + 1);
        const int64_t t0 = (int64_t)tile_of(i) * kTile;
        const int nt = it.n - t0 < kTile ? (int)(it.n - t0) : kTile;
        // one token; `slow` is a constant of each of the two loops below, f its factor
        const auto token = [&](int tt, auto slow_c, float f) {
            constexpr bool slow = decltype(slow_c)::value;
            float kk[Sh::kCols], v[Sh::kRows];
            load_row<Sh::kCols>(&s_in[tt][e0], kk);
            load_row<Sh::kRows>(&s_in[tt][2 * DK + d0], v);
#pragma unroll
            for (int e = 0; e < Sh::kCols; ++e) {
                const float2 ke = splat2(s.u_scale * kk[e]), ff = splat2(f);
#pragma unroll
                for (int r = 0; r < kPairs; ++r) {
                    const float2 vr = make_float2(v[2 * r], v[2 * r + 1]);
                    S[r][e] = slow ? fma2(ff, S[r][e], fma2(vr, ke, S[r][e])) : fma2(ff, S[r][e], mul2(vr, ke));
                }
            }
            if (!state_only) {
                float qq[Sh::kCols], o[Sh::kRows];
                load_row<Sh::kCols>(&s_in[tt][DK + e0], qq);
#pragma unroll
                for (int r = 0; r < kPairs; ++r) {
                    float2 x = mul2(S[r][0], splat2(qq[0]));
#pragma unroll
                    for (int e = 1; e < Sh::kCols; ++e) x = fma2(S[r][e], splat2(qq[e]), x);
                    o[2 * r] = x.x;
                    o[2 * r + 1] = x.y;
                }
                // lanes with the offset's bit set keep the upper half of the rows, the others the lower
                int row = 0;
#pragma unroll
                for (int half = Sh::kRows / 2, off = Sh::kLanes / 2; half > 0; half >>= 1, off >>= 1) {
                    const bool up = (l & off) != 0;
#pragma unroll
                    for (int r = 0; r < half; ++r) {
                        const float give = up ? o[r] : o[r + half];
                        const float keep = up ? o[r + half] : o[r];
                        o[r] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                    }
                    row += up ? half : 0;
                }
#pragma unroll
                for (int off = Sh::kLanes / 16; off > 0; off >>= 1) o[0] += __shfl_xor_sync(0xffffffffu, o[0], off);
                if ((l & (Sh::kLanes / 8 - 1)) == 0) s_o[tt][d0 + row] = s.out_scale * o[0];
            }
        };
        const auto walk = [&](auto slow_c) {
            constexpr bool slow = decltype(slow_c)::value;
            int x = 0;
            if (fresh && nt > 0) {               // the first backward step has no decay
                token(s.reverse ? nt - 1 : 0, slow_c, slow ? 0.0f : 1.0f);
                fresh = false;
                x = 1;
            }
#pragma unroll 4
            for (; x < nt; ++x) token(s.reverse ? nt - 1 - x : x, slow_c, decay.f);
        };
        if (decay.slow) walk(std::true_type{});
        else walk(std::false_type{});
        if (!state_only) {
            __syncthreads();
            for (int id = tid; id < nt * (DV / 4); id += kThr) {
                const int tt = id / (DV / 4), d = id % (DV / 4) * 4;
                const int64_t at = (it.row0 + t0 + tt) * s.o_ld + (int64_t)h * DV + d;
                const float4 y = *reinterpret_cast<const float4*>(&s_o[tt][d]);
                if (s.o_f32) *reinterpret_cast<float4*>((float*)s.o + at) = y;
                else store4((T*)s.o + at, y);
            }
        }
    }
    pdl_release();      // not earlier: a successor's blocks, placed beside unfinished ones, crowd some SMs (42 -> 37 us)
    if (s.reverse && it.n > 0) {
#pragma unroll
        for (int r = 0; r < kPairs; ++r)
#pragma unroll
            for (int e = 0; e < Sh::kCols; ++e) S[r][e] = make_float2(decay.step(S[r][e].x, 0.0f), decay.step(S[r][e].y, 0.0f));
    }
    float* out = nullptr;
    if (state_only) out = s.seg_states + (item * c.H + h) * hs;
    else if (last && s.final_state) out = s.final_state + (it.slot * c.H + h) * hs;
    if (out) {
#pragma unroll
        for (int r = 0; r < kPairs; ++r) {
            float x[Sh::kCols], y[Sh::kCols];
#pragma unroll
            for (int e = 0; e < Sh::kCols; ++e) {
                x[e] = S[r][e].x;
                y[e] = S[r][e].y;
            }
            store_row<Sh::kCols>(out + (d0 + 2 * r) * DK + e0, x);
            store_row<Sh::kCols>(out + (d0 + 2 * r + 1) * DK + e0, y);
        }
    }
}

template <typename T, int DK, int DV>
void launch_scan_shape(const LinearCall& c, const LinearScans& s, bool state_only, bool follows, cudaStream_t st)
{
    constexpr int kWarps = DV / SimtShape<DK>::kWarpRows > 0 ? DV / SimtShape<DK>::kWarpRows : 1;
    LaunchScope ls(state_only ? "linear_states" : "linear_scan", st);
    pdl_launch(follows, linear_scan_kernel<T, DK, DV>, dim3((unsigned)(c.items * c.H), (unsigned)s.n), 32 * kWarps, 0,
                  st, c, s, state_only);
}
template <typename T, int DK>
void launch_scan_dv(const LinearCall& c, const LinearScans& s, bool so, bool follows, cudaStream_t st)
{
    switch (s.s[0].DV) {
    case 16: return launch_scan_shape<T, DK, 16>(c, s, so, follows, st);
    case 32: return launch_scan_shape<T, DK, 32>(c, s, so, follows, st);
    case 64: return launch_scan_shape<T, DK, 64>(c, s, so, follows, st);
    default: return launch_scan_shape<T, DK, 128>(c, s, so, follows, st);
    }
}
template <typename T>
void launch_scan_dk(const LinearCall& c, const LinearScans& s, bool so, bool follows, cudaStream_t st)
{
    switch (s.s[0].DK) {
    case 16: return launch_scan_dv<T, 16>(c, s, so, follows, st);
    case 32: return launch_scan_dv<T, 32>(c, s, so, follows, st);
    case 64: return launch_scan_dv<T, 64>(c, s, so, follows, st);
    default: return launch_scan_dv<T, 128>(c, s, so, follows, st);
    }
}

// ------------------------------------------------------------- states between segments
// Rows of one segment are left alone. Before: seg_states[t] holds piece t's own state from a zero start
// (the pieces of the scan's last segment have none). After: at each segment's first piece in scan order,
// the state entering it. A block takes 1024 elements of one (sequence, head), a thread four of them, with
// the loads of the next kPassAhead pieces under way: a piece then costs 0.07 us, with one load ahead
// it is the load's latency, 0.5.
constexpr int kPassElems = 1024, kPassAhead = 8;
// The n-th of a packed call's sequences that have more than one segment (of which there are at most
// T / seg_tokens), found by a block of 256 threads; false: there is none.
__device__ bool nth_long(const LinearCall& c, int n, int64_t* seq)
{
    __shared__ int longs[8], found;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t base = 0; base < c.b && n >= 0; base += 256) {
        const int64_t i = base + threadIdx.x;
        LinearItem it;
        it.nseg = 0;
        if (i < c.b) linear_packed_item(c, i, 0, &it);     // of its rows, not its offsets: those may lie outside 0 .. T
        const bool is = it.nseg > 1;
        const unsigned all = __ballot_sync(0xffffffffu, is);
        if (lane == 0) longs[warp] = __popc(all);
        __syncthreads();
        int before = __popc(all & ((1u << lane) - 1)), total = 0;
        for (int w = 0; w < 8; ++w) {
            before += w < warp ? longs[w] : 0;
            total += longs[w];
        }
        if (is && before == n) found = (int)i;
        n -= total;
        __syncthreads();
    }
    *seq = found;
    return n < 0;
}
__global__ void __launch_bounds__(256) linear_pass_kernel(const LinearCall c, const LinearScans scans, int parts)
{
    const LinearScan& s = scans.s[blockIdx.x / parts];
    __shared__ LinearItem first;
    __shared__ int64_t item0;
    const int h = blockIdx.y;
    int64_t seq = blockIdx.z;
    const int hs = s.DK * s.DV, e0 = blockIdx.x % parts * kPassElems + 4 * threadIdx.x;
    pdl_follow();
    if (c.cu_seqlens && !nth_long(c, blockIdx.z, &seq)) return;
    if (threadIdx.x == 0) {
        item0 = c.cu_seqlens ? linear_packed_first(c, seq) : seq * c.nseg;
        const bool is = c.cu_seqlens ? linear_packed_item(c, seq, 0, &first) : linear_item(c, item0, &first);
        if (!is || item0 + first.nseg > c.items) first.nseg = 0;
    }
    __syncthreads();
    const int64_t nseg = first.nseg;
    if (nseg > 0 && !SSD_IN_BOUNDS(c.status, linear_in_bounds(c, first) && item0 >= 0 && item0 + nseg <= c.items)) return;
    // pieces before the scan's last segment, whose entering state ends the walk
    const int64_t before = s.reverse ? nseg - c.sub : (nseg - 1) / c.sub * c.sub;
    if (before < 1) return;
    const float g = linear_log_decay(c.log_decay, h);
    const bool init = linear_has_init(c, s, seq);
    const float* ip = s.init ? s.init + (first.slot * c.H + h) * (int64_t)hs : nullptr;
    if (e0 >= hs) return;
    // pieces in scan order (the short one is the row's last): p is the present one, `to_start` counts the
    // pieces to the next one that starts a segment
    const int64_t step = (s.reverse ? -1 : 1) * (int64_t)c.H * hs;
    float* p = s.seg_states + ((item0 + (s.reverse ? nseg - 1 : 0)) * c.H + h) * (int64_t)hs + e0;
    int to_start = 0;
    const int short_first = s.reverse ? (int)(nseg % c.sub) : 0;    // pieces of the scan's first segment, if not all
    float4 S = make_float4(0.0f, 0.0f, 0.0f, 0.0f), own[kPassAhead];
#pragma unroll
    for (int x = 0; x < kPassAhead; ++x) own[x] = x < before ? *reinterpret_cast<const float4*>(p + x * step) : S;
    if (init) {
        const float* q = ip + (int64_t)(e0 / s.DK) * s.init_rs + (int64_t)(e0 % s.DK) * s.init_cs;   // four of one row
        S = make_float4(q[0], q[s.init_cs], q[2 * s.init_cs], q[3 * s.init_cs]);
    }
    const LinearDecay whole(g * (float)c.seg_tokens);
    for (int64_t k0 = 0; k0 <= before; k0 += kPassAhead) {
#pragma unroll
        for (int x = 0; x < kPassAhead; ++x) {
            const int64_t k = k0 + x;
            if (k > before) break;
            if (to_start == 0) {
                *reinterpret_cast<float4*>(p) = S;
                to_start = k == 0 && short_first > 0 ? short_first : c.sub;
            }
            --to_start;
            // backwards the short piece comes first (only fixed-length rows run backwards)
            const LinearDecay d = s.reverse && k == 0 ? LinearDecay(g * (float)(c.L - (nseg - 1) * c.seg_tokens)) : whole;
            S = make_float4(d.step(S.x, own[x].x), d.step(S.y, own[x].y), d.step(S.z, own[x].z), d.step(S.w, own[x].w));
            if (k + kPassAhead < before) own[x] = *reinterpret_cast<const float4*>(p + kPassAhead * step);
            p += step;
        }
    }
}

// ------------------------------------------------------------- gradients of shared heads
// out[row][g][d] = sum of the r heads of group g, in fp32, rounded once. Bound by memory: 8192 tokens of 32
// heads of 128 on 8, 151 MB, 30 us (5 TB/s).
template <typename T>
__global__ void __launch_bounds__(256) linear_group_sum_kernel(const float* __restrict__ in, T* __restrict__ out, int64_t ld,
                                                               int64_t n, int G, int r, int D)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    pdl_follow();
    if (i >= n) return;
    const int64_t w = (int64_t)G * D, row = i / w;
    const int col = (int)(i - row * w), g = col / D, d = col - g * D;
    const float* p = in + (row * G + g) * (int64_t)r * D + d;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k = 0; k < r; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(p + (int64_t)k * D);
        a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
    }
    store4(out + row * ld + col, a);
}

// ------------------------------------------------------------------- lists of segments
// One block: the packed call's segments, sorted by their blocks of 128 tokens (a counting sort, the
// longest first, so that no CTA starts a long one last); those the recurrence does are left out. The
// order of equals is left to chance: it decides which CTA takes which, not what is computed. Some 4 us, its
// chain of a few loads, two barriers and a scan over the buckets.
constexpr int kListThreads = 1024, kBuckets = 256;
__global__ void __launch_bounds__(kListThreads) linear_list_kernel(const LinearCall c)
{
    __shared__ int start[2][kBuckets];
    pdl_follow();
    if (threadIdx.x < 64) c.status[threadIdx.x] = 0;          // the status word, the counts, what is taken
    for (int i = threadIdx.x; i < 2 * kBuckets; i += kListThreads) (&start[0][0])[i] = 0;
    __syncthreads();
    // bucket 0 holds the longest; z = 0: every segment, z = 1: those with one after them
    const auto each = [&](auto use) {
        for (int64_t seq = threadIdx.x; seq < c.b; seq += kListThreads) {
            LinearItem it;
            if (!linear_packed_item(c, seq, 0, &it) || (it.nseg == 1 && it.n <= kLinearShort)) continue;
            for (int64_t seg = 0; seg < it.nseg; ++seg) {
                linear_packed_item(c, seq, seg, &it);
                const int64_t blocks = (it.n + 127) / 128;
                const int bucket = kBuckets - 1 - (int)(blocks < kBuckets ? blocks : kBuckets - 1);
                use(0, bucket, seq, seg);
                if (seg + 1 < it.nseg) use(1, bucket, seq, seg);
            }
        }
    };
    each([&](int z, int bucket, int64_t, int64_t) { atomicAdd(&start[z][bucket], 1); });
    __syncthreads();
    if (threadIdx.x < 64) {                    // a warp per list, 8 buckets a lane: counts -> first places
        const int z = threadIdx.x >> 5, lane = threadIdx.x & 31;
        int n[kBuckets / 32], own = 0;
        for (int i = 0; i < kBuckets / 32; ++i) own += n[i] = start[z][lane * (kBuckets / 32) + i];
        int sum = own;
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) c.counts[z] = sum < c.items ? sum : (int)c.items;
        sum -= own;
        for (int i = 0; i < kBuckets / 32; ++i) {
            start[z][lane * (kBuckets / 32) + i] = sum;
            sum += n[i];
        }
    }
    __syncthreads();
    each([&](int z, int bucket, int64_t seq, int64_t seg) {
        const int at = atomicAdd(&start[z][bucket], 1);
        if (at < c.items) c.list[z * c.items + at] = make_int2((int)seq, (int)seg);
    });
}

// ---------------------------------------------------------------------------- decode and short rows
// Up to kLinearShort tokens of each row, token by token: the fp32 state is read once and written once,
// which for a few tokens is nearly all of the bytes. Lanes along DK (a float4 each), kRif state rows in
// flight per lane, so a CTA's whole part of the state is on its way before the first product.
// 256 sequences of 128 heads of 128 x 64: 324 us a step, 6.7 TB/s; one token of 32 heads of 128: 2.6 us.
constexpr int kShortThreads = 128, kRif = 8;

struct LinearShort {
    const void *q, *k, *v;
    int64_t q_ld, k_ld, v_ld, o_ld;
    const float* log_decay;
    const float* init;          // [slot][H][DV][DK] or nullptr; may be final_state
    float* final_state;
    const int32_t *cu_seqlens, *slot_idx;
    const uint8_t* has_init;
    int64_t nslots, L, T;
    void* o;
    int H, share, DV, parts;
    float scale;
    int* status;                // cleared by the kernel where it is the call's only one
};

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p)
{
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}

// ONE: rows of exactly one token (decode).
template <typename T, int DK, bool ONE>
__global__ void __launch_bounds__(kShortThreads) linear_short_kernel(const LinearShort p)
{
    constexpr int kLanes = DK / 4, kRows = kShortThreads / kLanes;   // rows of one pass of the CTA
    constexpr int kTokens = ONE ? 1 : kLinearShort;
    const int64_t seq = blockIdx.y;
    const int h = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
    if (!ONE) pdl_follow();
    if (!ONE && p.status && blockIdx.x == 0 && seq == 0 && threadIdx.x == 0) *p.status = kDevOk;
    int64_t row = seq * p.L, n = p.L;
    if (!ONE && p.cu_seqlens) {
        row = p.cu_seqlens[seq];
        row = row < 0 ? 0 : (row > p.T ? p.T : row);
        const int64_t end = p.cu_seqlens[seq + 1];
        n = (end < row ? row : (end > p.T ? p.T : end)) - row;
        if (n > kLinearShort) return;                                // the scan's
    }
    const int64_t slot = p.slot_idx ? (int64_t)p.slot_idx[seq] : seq;
    if (slot < 0 || slot >= p.nslots) return;
    const int l = threadIdx.x % kLanes, r0 = part * kRows * kRif + threadIdx.x / kLanes;
    const int64_t at = ((slot * p.H + h) * p.DV) * DK + 4 * l;
    const bool init = p.init && !(p.has_init && p.has_init[seq] == 0);
    float4 s[kRif];
#pragma unroll
    for (int i = 0; i < kRif; ++i) {
        const int r = r0 + i * kRows;
        s[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (init && r < p.DV) s[i] = *reinterpret_cast<const float4*>(p.init + at + (int64_t)r * DK);
    }
    const LinearDecay decay(linear_log_decay(p.log_decay, h));
    const T* kp = (const T*)p.k + row * p.k_ld + (int64_t)(h / p.share) * DK;
    const T* qp = (const T*)p.q + row * p.q_ld + (int64_t)h * DK;
    const T* vp = (const T*)p.v + row * p.v_ld + (int64_t)(h / p.share) * p.DV;
    T* op = (T*)p.o + row * p.o_ld + (int64_t)h * p.DV;
    // several tokens come into shared memory together, with the state's loads: token after token from
    // global memory is a load's latency each (1.4 us)
    __shared__ __align__(16) float sk[kTokens][DK], sq[kTokens][DK], sv[kTokens][kRows * kRif];
    if (!ONE) {
        for (int id = threadIdx.x; id < (int)n * kLanes; id += kShortThreads) {
            const int t = id / kLanes, e = id % kLanes * 4;
            *reinterpret_cast<float4*>(&sk[t][e]) = load4(kp + t * p.k_ld + e);
            *reinterpret_cast<float4*>(&sq[t][e]) = load4(qp + t * p.q_ld + e);
        }
        const int v0 = part * kRows * kRif, vecs = (p.DV - v0 < kRows * kRif ? p.DV - v0 : kRows * kRif) / 4;
        for (int id = threadIdx.x; id < (int)n * vecs; id += kShortThreads) {
            const int t = id / vecs, e = id % vecs * 4;
            *reinterpret_cast<float4*>(&sv[t][e]) = load4(vp + t * p.v_ld + v0 + e);
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int t = 0; t < (ONE ? 1 : (int)n); ++t) {
        const float4 k = ONE ? load4(kp + 4 * l) : *reinterpret_cast<const float4*>(&sk[t][4 * l]);
        const float4 q = ONE ? load4(qp + 4 * l) : *reinterpret_cast<const float4*>(&sq[t][4 * l]);
        float o[kRif];
#pragma unroll
        for (int i = 0; i < kRif; ++i) {
            const int r = r0 + i * kRows;
            o[i] = 0.0f;
            if (r < p.DV) {
                const float v = ONE ? ld_f(vp + r) : sv[t][threadIdx.x / kLanes + i * kRows];
                s[i].x = decay.step(s[i].x, v * k.x);
                s[i].y = decay.step(s[i].y, v * k.y);
                s[i].z = decay.step(s[i].z, v * k.z);
                s[i].w = decay.step(s[i].w, v * k.w);
                o[i] = s[i].x * q.x + s[i].y * q.y + s[i].z * q.z + s[i].w * q.w;
                if (ONE) *reinterpret_cast<float4*>(p.final_state + at + (int64_t)r * DK) = s[i];
            }
        }
        // lanes with the offset's bit set keep the upper half of the rows, the others the lower
        int first = 0;
#pragma unroll
        for (int half = kRif / 2, off = kLanes / 2; half > 0 && off > 0; half >>= 1, off >>= 1) {
            const bool up = (l & off) != 0;
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const float give = up ? o[i] : o[i + half];
                const float keep = up ? o[i + half] : o[i];
                o[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
            }
            first += up ? half : 0;
        }
#pragma unroll
        for (int off = kLanes / 16; off > 0; off >>= 1) o[0] += __shfl_xor_sync(0xffffffffu, o[0], off);
        if (kLanes <= 8 || (l & (kLanes / 8 - 1)) == 0) {
#pragma unroll
            for (int i = 0; i < (kLanes < 8 ? 8 / kLanes : 1); ++i) {
                const int r = r0 + (first + i) * kRows;
                if (r < p.DV) op[r] = Act<T>::from_f(p.scale * o[i]);
            }
        }
        op += p.o_ld;
    }
    if (!ONE) {
#pragma unroll
        for (int i = 0; i < kRif; ++i) {
            const int r = r0 + i * kRows;
            if (r < p.DV) *reinterpret_cast<float4*>(p.final_state + at + (int64_t)r * DK) = s[i];
        }
    }
}

template <typename T, bool ONE>
cudaError_t launch_short(LinearShort p, int DK, int64_t b, bool follows, cudaStream_t st)
{
    const int rows = kShortThreads / (DK / 4) * kRif;
    p.parts = (p.DV + rows - 1) / rows;
    LaunchScope ls(ONE ? "linear_decode" : "linear_short", st);
    const dim3 grid((unsigned)(p.H * p.parts), (unsigned)b);
    switch (DK) {
    case 16: return pdl_launch(follows, linear_short_kernel<T, 16, ONE>, grid, kShortThreads, 0, st, p);
    case 32: return pdl_launch(follows, linear_short_kernel<T, 32, ONE>, grid, kShortThreads, 0, st, p);
    case 64: return pdl_launch(follows, linear_short_kernel<T, 64, ONE>, grid, kShortThreads, 0, st, p);
    default: return pdl_launch(follows, linear_short_kernel<T, 128, ONE>, grid, kShortThreads, 0, st, p);
    }
}

}  // namespace

cudaError_t launch_linear_simt(const LinearCall& c, const LinearScan* scans, int nscans, cudaStream_t st)
{
    if (c.items == 0) return cudaSuccess;
    LinearCall call = c;
    bool follows = false, done[kMaxScans] = {};
    for (int i = 0; i < nscans; ++i) {
        if (done[i]) continue;
        LinearScans s{};
        for (int j = i; j < nscans; ++j) {
            if (done[j] || scans[j].DK != scans[i].DK || scans[j].DV != scans[i].DV) continue;
            done[j] = true;
            s.s[s.n++] = scans[j];
        }
        const auto run = [&](bool state_only) {
            if (c.act == SSD_BF16) launch_scan_dk<__nv_bfloat16>(call, s, state_only, follows, st);
            else launch_scan_dk<float>(call, s, state_only, follows, st);
            follows = true;
            call.clear_status = false;
            return cudaGetLastError();
        };
        cudaError_t e = cudaSuccess;
        if (c.split) {
            e = run(true);
            if (e == cudaSuccess) e = launch_linear_pass(c, s, st);
        }
        if (e == cudaSuccess) e = run(false);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_linear_pass(const LinearCall& c, const LinearScans& scans, cudaStream_t st)
{
    LaunchScope ls("linear_pass", st);
    const int64_t rows = c.cu_seqlens && c.T / c.seg_tokens < c.b ? c.T / c.seg_tokens : c.b;
    const int parts = (scans.s[0].DK * scans.s[0].DV + kPassElems - 1) / kPassElems;
    return pdl_launch(true, linear_pass_kernel, dim3((unsigned)(parts * scans.n), (unsigned)c.H, (unsigned)rows), 256, 0, st, c,
                         scans, parts);
}

// Splitting rows into segments fills SMs that whole rows would leave idle, at the price of a pass over
// k and v before the main one and of the segments' states.
namespace {
// Tensor cores, in units of one block of 128 tokens of the main pass (some 3.8 us for 128 x 128): a CTA
// per SM takes segment after segment, each some 1.6 to start and to end; a block of the states' pass is
// 0.5; the two more launches 1.8, and every segment's state goes through memory four times.
int64_t segment_tc(int64_t b, int64_t L, int64_t T, bool packed, int H, int nscans, int sms, int* sub)
{
    const int64_t rows = b * H * nscans;
    const double start = 1.6, states = 0.5, join = 1.8, each = 0.009;
    const int64_t blocks = ((packed ? T : L) + 127) / 128;
    if (blocks <= 1 || b == 0) return 256;                 // nothing to split: longer than any row
    if (packed && b > 1) {
        // The lengths are not known here. Segments are twice an SM's even share of all blocks (and 8 at
        // least): shorter rows, which find their place among the others, stay whole, and one long prompt
        // among many short rows does not keep a few SMs busy alone.
        const int64_t share = (blocks * H * nscans + sms - 1) / sms;
        return (2 * share > 8 ? 2 * share : 8) * 128;
    }
    const auto rounds = [&](int64_t n) { return (double)((n + sms - 1) / sms); };
    double best = rounds(rows) * ((double)blocks + start);   // whole rows
    int64_t best_seg = blocks + 1;
    for (int64_t nseg = 2; nseg <= blocks && nseg <= 256; ++nseg) {
        for (int m = 1; m <= (packed ? 1 : 4); ++m) {
            const int64_t piece = (blocks + nseg * m - 1) / (nseg * m), seg = piece * m;
            const int64_t n = rows * ((blocks + seg - 1) / seg), pieces = (n - rows) * m;
            if (n == rows) continue;
            const double cost = rounds(n) * ((double)seg + start) + rounds(pieces) * (states * (double)piece + start) + join +
                                each * (double)pieces * 148.0 / (double)sms;
            if (cost < best) {
                best = cost;
                best_seg = seg;
                *sub = m;
            }
        }
    }
    return best_seg * 128;
}

// CUDA cores, in us. A token costs a warp's latency (0.25; states alone 0.12) or, with w warps to a
// scheduler, w times its issue slots (0.066 + 0.0004 dk; states half of it), and a little more where the two
// are near: so segments are cut until the schedulers have some three warps each. A CTA's state comes and goes
// at some 15 KB a us of its SM; the pass that joins the segments takes 0.07 a segment of a row.
int64_t segment_simt(int64_t b, int64_t L, int64_t T, bool packed, int H, int nscans, int DK, int DV, int sms)
{
    const int64_t tiles = ((packed ? T : L) + kTile - 1) / kTile;
    if (tiles <= 1 || b == 0) return 2 * kTile;
    const int rows_per_warp = DK == 16 ? 16 : 8;
    const double warps = DV > rows_per_warp ? DV / rows_per_warp : 1, slots = 0.066 + 0.0004 * DK;
    const double state_kb = 4.0 * DK * DV / 1024.0;
    const auto pass = [&](int64_t n, double seg, double latency, double issue) {
        // a few CTAs to an SM: the fullest SM counts; many: their average
        const double each = n > 8 * (int64_t)sms ? (double)n / sms : (double)((n + sms - 1) / sms), w = each * warps / 4.0;
        return 3.0 + each * state_kb / 15.0 + seg * kTile * pow(pow(latency, 4.0) + pow(w * issue, 4.0), 0.25);
    };
    if (packed && b > 1) {
        // The lengths are not known here: an SM's even share of all tokens with three warps to a
        // scheduler, and 64 tokens at least.
        const double ctas = sms * (12.0 / warps > 1.0 ? 12.0 / warps : 1.0);
        const int64_t share = (int64_t)((double)tiles * H / ctas) + 1;
        return (share > 4 ? share : 4) * kTile;
    }
    // the three scans of a backward pass run together where their shapes are one, else two and one
    const int64_t rows = b * H * (nscans < 2 || DK == DV ? nscans : 2);
    double best = pass(rows, (double)tiles, 0.25, slots);    // whole rows
    int64_t best_seg = tiles + 1;
    for (int64_t nseg = 2; nseg <= tiles && nseg <= 512; ++nseg) {
        const int64_t seg = (tiles + nseg - 1) / nseg, n = rows * ((tiles + seg - 1) / seg);
        const double cost = pass(n, (double)seg, 0.25, slots) + pass(n - rows, (double)seg, 0.12, 0.5 * slots) +
                            3.0 + 0.07 * (double)nseg + 2.0 * state_kb * (double)n / 6400.0;
        if (cost < best) {
            best = cost;
            best_seg = seg;
        }
    }
    return best_seg * kTile;
}
}  // namespace

int64_t linear_segment_tokens(bool tc, int64_t b, int64_t L, int64_t T, bool packed, int H, int nscans, int DK, int DV, int sms,
                              int* sub)
{
    *sub = 1;
    return tc ? segment_tc(b, L, T, packed, H, nscans, sms, sub) : segment_simt(b, L, T, packed, H, nscans, DK, DV, sms);
}

cudaError_t launch_linear_group_sum(const float* in, void* out, int64_t ld, int64_t rows, int G, int r, int D, int act,
                                    cudaStream_t st)
{
    const int64_t n = rows * G * (int64_t)D;
    if (n == 0) return cudaSuccess;
    LaunchScope ls("linear_group_sum", st);
    const unsigned grid = (unsigned)((n / 4 + 255) / 256);
    return act == SSD_BF16 ? pdl_launch(true, linear_group_sum_kernel<__nv_bfloat16>, dim3(grid), 256, 0, st, in, (__nv_bfloat16*)out, ld, n, G, r, D)
                           : pdl_launch(true, linear_group_sum_kernel<float>, dim3(grid), 256, 0, st, in, (float*)out, ld, n, G, r, D);
}

cudaError_t launch_linear_list(const LinearCall& c, cudaStream_t st)
{
    LaunchScope ls("linear_list", st);
    linear_list_kernel<<<1, kListThreads, 0, st>>>(c);
    return cudaGetLastError();
}

cudaError_t launch_linear_short(const LinearCall& c, const LinearScan& s, bool one, bool follows, cudaStream_t st)
{
    LinearShort p{};
    p.q = s.q; p.k = s.k; p.v = s.v; p.o = s.o;
    p.q_ld = s.q_ld; p.k_ld = s.k_ld; p.v_ld = s.v_ld; p.o_ld = s.o_ld;
    p.log_decay = c.log_decay;
    p.init = s.init;
    p.final_state = s.final_state;
    p.cu_seqlens = c.cu_seqlens; p.slot_idx = c.slot_idx; p.has_init = c.has_init;
    p.nslots = c.nslots; p.L = c.L; p.T = c.T;
    p.H = c.H; p.share = s.k_share; p.DV = s.DV;
    p.scale = s.out_scale;
    p.status = c.clear_status && !c.cu_seqlens ? c.status : nullptr;
    if (c.act == SSD_BF16)
        return one ? launch_short<__nv_bfloat16, true>(p, s.DK, c.b, follows, st) : launch_short<__nv_bfloat16, false>(p, s.DK, c.b, follows, st);
    return one ? launch_short<float, true>(p, s.DK, c.b, follows, st) : launch_short<float, false>(p, s.DK, c.b, follows, st);
}

}  // namespace ssd
