// ssd_layer_norm.cu -- layer norm over contiguous groups of a row's channels, and its gradients.
//
//   y = (x - m) r w + b,   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps)
//   with xh = (x - m) r and dh = dy w:
//   dx = r (dh - mean(dh) - xh mean(dh xh)),   dw = sum over rows of dy xh,   db = sum of dy
// All sums in fp32, the variance around the mean (no difference of large sums).
//
// Both passes are bound by memory in principle, x (and dy) read once and y (dx) written once, and by
// instructions in practice: few operations an element and few shuffles a row decide. A thread holds NV
// vectors of 16 (or, for rows that only 8 divides, 8) bytes of a row; a group is summed by a team,
// either a power of two of lanes of one warp (head norms: no barrier at all) or the whole block.
// Rows that are not so aligned are read element by element, forwards into registers too; teams that would
// not fit, and gradients of such rows, take a loop of one warp per (row, group).
//   Forwards, block teams: a block per row, many on an SM, so that one's barriers are the others' time.
//   All others walk down the rows on one set of columns, the coming rows on their way into shared
//   memory, where each thread copies and reads its own vectors only: several rows in flight without a
//   register or a barrier for them. Backwards the columns' weight gradients stay in registers over all
//   rows and each block leaves one partial sum; a second kernel adds those in a fixed order.
#include "../../include/ssd_mixer.h"
#include "ssd_common.cuh"
#include "ssd_layer_norm.h"
#include "ssd_pdl.cuh"
#include "ssd_profile.h"

namespace ssd {
namespace {

constexpr int kWarps = 8;

// One warp per (row, group), three readings of the row: for rows too wide for registers.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) layer_norm_kernel(const LayerNorm p)
{
    const int64_t seg = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (seg >= p.rows * p.groups) return;
    const int lane = threadIdx.x & 31, g = (int)(seg % p.groups);
    const int64_t row = seg / p.groups;
    const T* x = (const T*)p.x + row * p.x_ld + (int64_t)g * p.width;
    T* y = (T*)p.y + row * p.y_ld + (int64_t)g * p.width;
    const float* w = p.weight ? p.weight + (int64_t)g * p.width : nullptr;
    const float* b = p.bias ? p.bias + (int64_t)g * p.width : nullptr;
    float s = 0.0f;
    for (int i = lane; i < p.width; i += 32) s += ld_f(x + i);
    const float m = warp_sum(s) / p.width;
    s = 0.0f;
    for (int i = lane; i < p.width; i += 32) {
        const float d = ld_f(x + i) - m;
        s = fmaf(d, d, s);
    }
    const float r = 1.0f / sqrtf(warp_sum(s) / p.width + p.eps);
    for (int i = lane; i < p.width; i += 32)
        y[i] = Act<T>::from_f(fmaf((ld_f(x + i) - m) * r, w ? w[i] : 1.0f, b ? b[i] : 0.0f));
    if (lane == 0) {
        if (p.mean) p.mean[seg] = m;
        if (p.rstd) p.rstd[seg] = r;
    }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) layer_norm_dx_kernel(const LayerNorm p)
{
    const int64_t seg = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (seg >= p.rows * p.groups) return;
    const int lane = threadIdx.x & 31, g = (int)(seg % p.groups);
    const int64_t row = seg / p.groups;
    const T* x = (const T*)p.x + row * p.x_ld + (int64_t)g * p.width;
    const T* dy = (const T*)p.dy + row * p.dy_ld + (int64_t)g * p.width;
    T* dx = (T*)p.y + row * p.y_ld + (int64_t)g * p.width;
    const float* w = p.weight ? p.weight + (int64_t)g * p.width : nullptr;
    const float m = p.mean[seg], r = p.rstd[seg];
    float s1 = 0.0f, s2 = 0.0f;
    for (int i = lane; i < p.width; i += 32) {
        const float dh = ld_f(dy + i) * (w ? w[i] : 1.0f);
        s1 += dh;
        s2 = fmaf(dh, (ld_f(x + i) - m) * r, s2);
    }
    s1 = warp_sum(s1) / p.width;
    s2 = warp_sum(s2) / p.width;
    for (int i = lane; i < p.width; i += 32) {
        const float dh = ld_f(dy + i) * (w ? w[i] : 1.0f);
        dx[i] = Act<T>::from_f(r * (dh - s1 - (ld_f(x + i) - m) * r * s2));
    }
}

// Partial sums over a slice of the rows, a thread per channel (4096 x 12 groups of 333 bf16: 32 us, after 41 for
// dx by a warp per group, against some 15 in all that the bytes would take).
template <typename T>
__global__ void __launch_bounds__(256) layer_norm_dw_kernel(const LayerNorm p, int parts)
{
    const int64_t C = p.channels(), c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= C) return;
    const int g = (int)(c / p.width), part = blockIdx.y;
    float dw = 0.0f, db = 0.0f;
    for (int64_t row = part; row < p.rows; row += parts) {
        const float dy = ld_f((const T*)p.dy + row * p.dy_ld + c);
        const float xh = (ld_f((const T*)p.x + row * p.x_ld + c) - p.mean[row * p.groups + g]) * p.rstd[row * p.groups + g];
        dw = fmaf(dy, xh, dw);
        db += dy;
    }
    p.part[((int64_t)part * 2 + 0) * C + c] = dw;
    p.part[((int64_t)part * 2 + 1) * C + c] = db;
}

// ------------------------------------------------------------------ vectors
// VB bytes of a row (16, 8, or a single element): the raw words, and how many elements they are.
template <typename T, int VB>
struct RowVec {
    static constexpr int kN = VB / (int)sizeof(T), kW = VB < 4 ? 1 : VB / 4;   // elements, words
    uint32_t w[kW];
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (VB == 16) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (kN == 1) {
            w[0] = __float_as_uint(ld_f(p));
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x; w[1] = v.y;
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kW; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float at(int i) const
    {
        if constexpr (sizeof(T) == 4 || kN == 1) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ void set(const float* f)
    {
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            if constexpr (sizeof(T) == 4 || kN == 1) {
                w[i] = __float_as_uint(f[i]);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
    __device__ __forceinline__ void store(T* p) const
    {
        if constexpr (VB == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kN == 1) *p = Act<T>::from_f(__uint_as_float(w[0]));
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
};
// N parameters from column c (aligned to 4 N bytes), or a constant. Eight come as one load of 32 bytes a lane:
// as two of 16 a warp's loads would pass through the L1 with gaps, at half its rate, which is what bound wide
// rows of bf16 (16384 x 8192: 127 us, now 104).
template <int N>
__device__ __forceinline__ void load_params(const float* p, int64_t c, float none, float* f)
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = none;
    } else if constexpr (N == 1) {
        f[0] = p[c];
    } else if constexpr (N == 2) {
        const float2 v = *reinterpret_cast<const float2*>(p + c);
        f[0] = v.x; f[1] = v.y;
    } else if constexpr (N == 8) {
        asm("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
            : "l"(p + c));
    } else {
        static_assert(N == 4, "");
        const float4 v = *reinterpret_cast<const float4*>(p + c);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    }
}

// N floats from an address that 4 N bytes (at most 16) divide: one by one, a warp's stores would touch each
// sector several times (256 blocks of 2 x 2688: 12.8 us for the call, in vectors 6.8).
template <int N>
__device__ __forceinline__ void store_params(float* p, const float* v)
{
    if constexpr (N == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    else
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
// Sum over a team of TEAM lanes, or (TEAM = 0) over the block, in a fixed order. One barrier a call,
// so successive calls take different `red` (32 values).
template <int TEAM>
__device__ __forceinline__ float team_sum1(float v, float* red)
{
#pragma unroll
    for (int o = (TEAM ? TEAM : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TEAM == 0) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < (int)(blockDim.x >> 5) ? red[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}
// Two sums at the price of one and a bit (an SM's warps share one shuffle unit): after the first
// exchange the lower half of the team's lanes carries a, the upper half b. red: 64 floats.
template <int TEAM>
__device__ __forceinline__ float2 team_sum2(float a, float b, float* red)
{
    constexpr int H = (TEAM ? TEAM : 32) / 2;
    const int lane = threadIdx.x & 31;
    const bool up = (lane & H) != 0;
    float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, H);
#pragma unroll
    for (int o = H / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TEAM == 0) {
        if ((lane & 15) == 0) red[(up ? 32 : 0) + (threadIdx.x >> 5)] = v;
        __syncthreads();
        const int w = 2 * (lane & 15), warps = blockDim.x >> 5;
        const float2 x = *reinterpret_cast<const float2*>(red + (up ? 32 : 0) + w);
        v = (w < warps ? x.x : 0.0f) + (w + 1 < warps ? x.y : 0.0f);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    const float other = __shfl_xor_sync(0xffffffffu, v, H);
    return up ? make_float2(other, v) : make_float2(v, other);
}

// VB bytes global -> shared, asynchronously; and all but the newest N groups of this thread's copies.
template <int VB>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src)
{
    if constexpr (VB == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The columns of a block and the ring of its rows: OPS operands (x, or x and dy), kRing rows deep.
// Lane teams: the block's columns are blockDim.x vectors from blockIdx.x * blockDim.x; block teams:
// group blockIdx.x. Rows blockIdx.y, blockIdx.y + gridDim.y, ..
SSD_HD constexpr int ring_rows(int nv, int ops) { return nv == 4 && ops == 2 ? 3 : 4; }   // at most 192 KB a block
template <typename T, int VB, int NV, int TEAM, int OPS>
struct RowWalk {
    using V = RowVec<T, VB>;
    static constexpr int kRing = ring_rows(NV, OPS);
    unsigned char* ring;
    uint32_t ring0;
    int step, tid, vecs, g, slot;
    int64_t c0, row, stride, rows;
    const T *x, *dy;            // this thread's first vector of the next row to fetch

    __device__ __forceinline__ RowWalk(const LayerNorm& p, unsigned char* r)
        : ring(r), ring0((uint32_t)__cvta_generic_to_shared(r)), step(blockDim.x), tid(threadIdx.x), slot(0), row(blockIdx.y),
          stride(gridDim.y), rows(p.rows)
    {
        const int64_t C = p.channels();
        c0 = TEAM ? (int64_t)blockIdx.x * blockDim.x * V::kN : (int64_t)blockIdx.x * p.width;
        vecs = TEAM ? (int)((C - c0) / V::kN < step ? (C - c0) / V::kN : step) : p.width / V::kN;
        g = TEAM ? (int)((c0 + (int64_t)(tid < vecs ? tid : 0) * V::kN) / p.width) : (int)blockIdx.x;
        x = (const T*)p.x + row * p.x_ld + col(0);
        if (OPS == 2) dy = (const T*)p.dy + row * p.dy_ld + col(0);
#pragma unroll
        for (int a = 0; a < kRing - 1; ++a) fetch(p, row + a * stride, a);
    }
    __device__ __forceinline__ bool in(int i) const { return tid + i * step < vecs; }
    __device__ __forceinline__ int64_t col(int i) const { return c0 + (int64_t)(tid + i * step) * V::kN; }
    __device__ __forceinline__ uint32_t at(int a, int o, int i) const
    {
        return (uint32_t)((((a * OPS + o) * NV + i) * step + tid) * VB);
    }
    __device__ __forceinline__ void fetch(const LayerNorm& p, int64_t r, int a)
    {
        if (r < rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in(i)) {
                    copy_async<VB>(ring0 + at(a, 0, i), x + i * step * V::kN);
                    if (OPS == 2) copy_async<VB>(ring0 + at(a, 1, i), dy + i * step * V::kN);
                }
            x += stride * p.x_ld;
            if (OPS == 2) dy += stride * p.dy_ld;
        }
        copy_commit();
    }
    // The present row's vectors (zeros past the columns), and on to the next row: the slot read one
    // row ago takes the row kRing - 1 further on.
    __device__ __forceinline__ void take(const LayerNorm& p, V (*v)[NV])
    {
        copy_wait<kRing - 2>();
#pragma unroll
        for (int o = 0; o < OPS; ++o)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                v[o][i].zero();
                if (in(i)) v[o][i].load(reinterpret_cast<const T*>(ring + at(slot, o, i)));
            }
        fetch(p, row + (kRing - 1) * stride, slot == 0 ? kRing - 1 : slot - 1);
        slot = slot == kRing - 1 ? 0 : slot + 1;
    }
};

// Lane teams, down the rows. 32768 x 64 groups of 128 bf16: 195 us, 5.5 TB/s, 78 % of the issue slots taken
// (two sums over 16 lanes for 8 elements a lane).
template <typename T, int VB, int TEAM>
__global__ void __launch_bounds__(256) layer_norm_lanes_kernel(const LayerNorm p)
{
    using W = RowWalk<T, VB, 1, TEAM, 1>;
    using V = typename W::V;
    extern __shared__ __align__(16) unsigned char ring[];
    W it(p, ring);
    const float inv = 1.0f / (float)p.width;
    float w[V::kN], b[V::kN];
    load_params<V::kN>(it.in(0) ? p.weight : nullptr, it.col(0), 1.0f, w);
    load_params<V::kN>(it.in(0) ? p.bias : nullptr, it.col(0), 0.0f, b);
    for (; it.row < p.rows; it.row += it.stride) {
        V v[1][1];
        it.take(p, v);
        float f[V::kN], s = 0.0f;
#pragma unroll
        for (int e = 0; e < V::kN; ++e) s += f[e] = v[0][0].at(e);
        const float m = team_sum1<TEAM>(s, nullptr) * inv;
        s = 0.0f;
#pragma unroll
        for (int e = 0; e < V::kN; ++e) {
            f[e] -= m;
            s = fmaf(f[e], f[e], s);
        }
        const float rs = 1.0f / sqrtf(team_sum1<TEAM>(s, nullptr) * inv + p.eps);
        if (it.in(0)) {
#pragma unroll
            for (int e = 0; e < V::kN; ++e) f[e] = fmaf(f[e] * rs, w[e], b[e]);
            V o;
            o.set(f);
            o.store((T*)p.y + it.row * p.y_ld + it.col(0));
            if (it.tid % TEAM == 0) {
                const int64_t seg = it.row * p.groups + it.g;
                if (p.mean) p.mean[seg] = m;
                if (p.rstd) p.rstd[seg] = rs;
            }
        }
    }
    copy_wait<0>();
}

// A block, or (TEAM = 32) each warp of it, per (row, group). 16384 x 8192 bf16: 103 us, 5.2 TB/s (what bounds
// it: the parameters' way through the L1, then a row's chain of load, two sums and store); fp32 164 us, 6.5.
template <typename T, int VB, int NV, int TEAM>
__global__ void __launch_bounds__(TEAM ? 128 : (NV > 4 ? 512 : 1024)) layer_norm_block_kernel(const LayerNorm p)
{
    using V = RowVec<T, VB>;
    __shared__ float red[2][32];
    const int64_t seg = TEAM ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
    if (TEAM && seg >= p.rows * p.groups) return;
    const int t = TEAM ? threadIdx.x & 31 : threadIdx.x, step = TEAM ? 32 : blockDim.x, vecs = p.width / V::kN;
    const int g = (int)(seg % p.groups);
    const int64_t row = seg / p.groups, c0 = (int64_t)g * p.width + t * V::kN;
    const T* x = (const T*)p.x + row * p.x_ld + c0;
    const float inv = 1.0f / (float)p.width;
    float f[NV][V::kN];
    {
        V v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i].zero();
            if (t + i * step < vecs) v[i].load(x + i * step * V::kN);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V::kN; ++e) f[i][e] = v[i].at(e);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V::kN; ++e) s += f[i][e];
    const float m = team_sum1<TEAM>(s, red[0]) * inv;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (t + i * step < vecs)
#pragma unroll
            for (int e = 0; e < V::kN; ++e) {
                f[i][e] -= m;
                s = fmaf(f[i][e], f[i][e], s);
            }
    const float rs = 1.0f / sqrtf(team_sum1<TEAM>(s, red[1]) * inv + p.eps);
    T* y = (T*)p.y + row * p.y_ld + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (t + i * step < vecs) {
            float w[V::kN], b[V::kN];
            load_params<V::kN>(p.weight, c0 + i * step * V::kN, 1.0f, w);
            load_params<V::kN>(p.bias, c0 + i * step * V::kN, 0.0f, b);
#pragma unroll
            for (int e = 0; e < V::kN; ++e) f[i][e] = fmaf(f[i][e] * rs, w[e], b[e]);
            V o;
            o.set(f[i]);
            o.store(y + i * step * V::kN);
        }
    if (t == 0) {
        if (p.mean) p.mean[seg] = m;
        if (p.rstd) p.rstd[seg] = rs;
    }
}

// dx = rs dy w + (A xh + B), A = -rs mean(dh xh), B = -rs mean(dh): three operations an element. xh = (x - m) rs
// takes the difference first: of close numbers it is exact, where the rounding of m rs in x rs - m rs is the
// same over a whole row (dweight of rows at 1000 spreads from zero was off by 2e-5 of its size, now 4e-8). Block
// teams keep xh in registers for dx where there is room (16384 x 8192 bf16: 177 us, 210 without); lane teams
// take x - m again (32768 x 64 groups of 128: 280 us, 296 with it kept).
// 16384 x 8192 bf16: 177 us, 4.6 TB/s: one block to an SM, whose rows follow one another through a barrier and
// two sums; 32768 x 64 groups of 128 280 us, 5.8; 2048 x 2688 fp32 some 14 us: 14 rows a block in the same way.
template <typename T, int VB, int NV, int TEAM>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) layer_norm_grad_kernel(const LayerNorm p)
{
    using W = RowWalk<T, VB, NV, TEAM, 2>;
    using V = typename W::V;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ __align__(16) float red[2][64];
    W it(p, ring);
    const int64_t C = p.channels();
    const float inv = 1.0f / (float)p.width;
    float dw[NV][V::kN], db[NV][V::kN], w[V::kN];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V::kN; ++e) dw[i][e] = db[i][e] = 0.0f;
    if (NV == 1) load_params<V::kN>(it.in(0) ? p.weight : nullptr, it.col(0), 1.0f, w);
    const float *mp = p.mean + it.row * p.groups + it.g, *rp = p.rstd + it.row * p.groups + it.g;
    const int64_t sstep = it.stride * p.groups;
    float m_next = 0.0f, r_next = 0.0f;
    if (it.row < p.rows) {
        m_next = *mp;
        r_next = *rp;
    }
    T* dx = (T*)p.y + it.row * p.y_ld + it.col(0);
    for (int k = 0; it.row < p.rows; it.row += it.stride, k ^= 1) {
        const float rs = r_next, m = m_next;
        if (it.row + it.stride < p.rows) {
            m_next = *(mp += sstep);
            r_next = *(rp += sstep);
        }
        V v[2][NV];
        it.take(p, v);
        float s1 = 0.0f, s2 = 0.0f, xhs[NV][V::kN];
        constexpr bool kKeep = TEAM == 0 && (NV == 1 || sizeof(T) == 4);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (it.in(i)) {
                if (NV > 1) load_params<V::kN>(p.weight, it.col(i), 1.0f, w);
#pragma unroll
                for (int e = 0; e < V::kN; ++e) {
                    const float d = v[1][i].at(e), xh = (v[0][i].at(e) - m) * rs, dh = d * w[e];
                    dw[i][e] = fmaf(d, xh, dw[i][e]);
                    db[i][e] += d;
                    s1 += dh;
                    s2 = fmaf(dh, xh, s2);
                    if (kKeep) xhs[i][e] = xh;
                }
            }
        const float2 s = team_sum2<TEAM>(s1, s2, red[k]);
        const float A = -rs * (s.y * inv), B = -rs * (s.x * inv);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (it.in(i)) {
                if (NV > 1) load_params<V::kN>(p.weight, it.col(i), 1.0f, w);
                float f[V::kN];
#pragma unroll
                for (int e = 0; e < V::kN; ++e)
                    f[e] = fmaf(v[1][i].at(e), rs * w[e], kKeep ? fmaf(xhs[i][e], A, B) : fmaf(v[0][i].at(e) - m, A * rs, B));
                V o;
                o.set(f);
                o.store(dx + i * it.step * V::kN);
            }
        dx += it.stride * p.y_ld;
    }
    copy_wait<0>();
    pdl_release();
    if (!p.part) return;
    float* part = p.part + (int64_t)blockIdx.y * 2 * C;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (it.in(i)) {
            store_params<V::kN>(part + it.col(i), dw[i]);
            store_params<V::kN>(part + C + it.col(i), db[i]);
        }
}

// Sums of the partial sums, 32 channels a block, its 8 warps sharing the parts: each in order, then
// the warps in order. 148 parts of 2 x 8192, from L2: 4 us.
__global__ void __launch_bounds__(256) layer_norm_parts_kernel(const LayerNorm p, int parts)
{
    __shared__ float s[8][32];
    const int64_t C = p.channels(), c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const int warp = threadIdx.x >> 5;
    pdl_wait();
    float a = 0.0f;
    if (c < C)
#pragma unroll 8
        for (int i = warp; i < parts; i += 8) a += p.part[((int64_t)i * 2 + blockIdx.y) * C + c];
    s[warp][threadIdx.x & 31] = a;
    __syncthreads();
    float* out = blockIdx.y ? p.dbias : p.dweight;
    if (warp == 0 && c < C && out) {
#pragma unroll
        for (int i = 1; i < 8; ++i) a += s[i][threadIdx.x];
        out[c] = a;
    }
}

// ------------------------------------------------------------------ which kernel
// The widest vector that divides every row's address and the width; 0: none.
template <typename T>
int vector_bytes(const LayerNorm& p)
{
    for (int vb = 16; vb >= 8; vb -= 8) {
        const int n = vb / (int)sizeof(T);
        const uintptr_t par = n * 4;
        if (p.width % n || (uintptr_t)p.x % vb || (uintptr_t)p.y % vb || (uintptr_t)p.dy % vb || p.x_ld % n || p.y_ld % n ||
            p.dy_ld % n || (uintptr_t)p.weight % par || (uintptr_t)p.bias % par)
            continue;
        return vb;
    }
    return 0;
}
bool lane_team(int vecs) { return vecs >= 2 && vecs <= 32 && (vecs & (vecs - 1)) == 0; }
int round32(int64_t v) { return (int)((v + 31) / 32 * 32); }

// Blocks of the kernels that walk down the rows: threads, vectors a thread, blocks across the columns,
// and blocks resident on an SM together (1024 threads of 64 registers, or 512 of 128).
struct RowShape {
    int threads, nv, cols, per_sm;
};
RowShape row_shape(int groups, int width, int vec)
{
    const int vecs = width / vec;
    RowShape s{};
    if (lane_team(vecs)) {
        const int64_t all = (int64_t)groups * vecs;
        s.threads = all >= 256 ? 256 : round32(all);
        s.nv = 1;
        s.cols = (int)((all + s.threads - 1) / s.threads);
    } else {
        if (vecs < 1 || vecs > 2048) return s;
        s.nv = vecs <= 1024 ? 1 : 4;
        s.threads = round32((vecs + s.nv - 1) / s.nv);
        s.cols = groups;
    }
    s.per_sm = (s.nv == 1 ? 1024 : 512) / s.threads;
    s.per_sm = s.per_sm < 1 ? 1 : s.per_sm;
    return s;
}
int64_t rows_at_a_time(const RowShape& s, int sms) { return ((int64_t)sms * s.per_sm + s.cols - 1) / s.cols; }

template <typename K>
cudaError_t launch_rows(K kernel, const LayerNorm& p, const RowShape& s, int ops, int vb, int64_t rows, cudaStream_t st)
{
    const int smem = ring_rows(s.nv, ops) * ops * s.nv * s.threads * vb;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<dim3((unsigned)s.cols, (unsigned)rows), s.threads, smem, st>>>(p);
    return cudaGetLastError();
}

// False: not a shape that the vector kernels take.
template <typename T, int VB>
bool forward_vec(const LayerNorm& p, cudaStream_t st, cudaError_t* e)
{
    const int vecs = p.width / RowVec<T, VB>::kN;
    if constexpr (RowVec<T, VB>::kN > 1) {
        if (lane_team(vecs)) {
            const RowShape s = row_shape(p.groups, p.width, RowVec<T, VB>::kN);
            int64_t rows = rows_at_a_time(s, device_sm_count());
            rows = rows < p.rows ? rows : p.rows;
            const auto go = [&](auto kernel) { *e = launch_rows(kernel, p, s, 1, VB, rows < 65535 ? rows : 65535, st); };
            switch (vecs) {
            case 2: go(layer_norm_lanes_kernel<T, VB, 2>); break;
            case 4: go(layer_norm_lanes_kernel<T, VB, 4>); break;
            case 8: go(layer_norm_lanes_kernel<T, VB, 8>); break;
            case 16: go(layer_norm_lanes_kernel<T, VB, 16>); break;
            default: go(layer_norm_lanes_kernel<T, VB, 32>); break;
            }
            return true;
        }
    }
    const unsigned grid = (unsigned)(p.rows * p.groups), warps = (unsigned)((p.rows * p.groups + 3) / 4);
    // Rows of up to 256 vectors of eight elements, or 384 smaller ones: a warp each (51 against 54 us for
    // 65536 x 1024 bf16, 28 against 51 for 4096 x 12 groups of 333; 32768 x 2688 bf16, 336 vectors, 79
    // against 75), but a block where there are too few of them to fill the device (8.8 against
    // 11 us for 1200 x 1024). Blocks hold 32 elements a thread (16384 x 8192 bf16 104 us, 5.1 TB/s; x 4096
    // 54, with half of that 76), with few rows half of that.
    constexpr bool kEights = RowVec<T, VB>::kN >= 8;
    constexpr int kNV = kEights ? 4 : 8;
    const bool many = p.rows * p.groups >= (int64_t)device_sm_count() * 8;
    if (many && vecs <= (kEights ? 256 : 384)) {
        if (vecs <= 64) layer_norm_block_kernel<T, VB, 2, 32><<<warps, 128, 0, st>>>(p);
        else if (vecs <= 128) layer_norm_block_kernel<T, VB, 4, 32><<<warps, 128, 0, st>>>(p);
        else if (kEights || vecs <= 256) layer_norm_block_kernel<T, VB, 8, 32><<<warps, 128, 0, st>>>(p);
        else layer_norm_block_kernel<T, VB, kEights ? 8 : 12, 32><<<warps, 128, 0, st>>>(p);
    } else if (!many && vecs <= 512) layer_norm_block_kernel<T, VB, 2, 0><<<grid, round32((vecs + 1) / 2), 0, st>>>(p);
    else if (vecs <= 4096) layer_norm_block_kernel<T, VB, kNV, 0><<<grid, round32((vecs + kNV - 1) / kNV), 0, st>>>(p);
    else return false;
    *e = cudaGetLastError();
    return true;
}
template <typename T, int VB>
bool backward_vec(const LayerNorm& p, int parts, cudaStream_t st, cudaError_t* e)
{
    const RowShape s = row_shape(p.groups, p.width, RowVec<T, VB>::kN);
    if (!s.threads) return false;
    const int vecs = p.width / RowVec<T, VB>::kN;
    const auto go = [&](auto kernel) { *e = launch_rows(kernel, p, s, 2, VB, parts, st); };
    if (lane_team(vecs)) {
        switch (vecs) {
        case 2: go(layer_norm_grad_kernel<T, VB, 1, 2>); break;
        case 4: go(layer_norm_grad_kernel<T, VB, 1, 4>); break;
        case 8: go(layer_norm_grad_kernel<T, VB, 1, 8>); break;
        case 16: go(layer_norm_grad_kernel<T, VB, 1, 16>); break;
        default: go(layer_norm_grad_kernel<T, VB, 1, 32>); break;
        }
    } else if (s.nv == 1) go(layer_norm_grad_kernel<T, VB, 1, 0>);
    else go(layer_norm_grad_kernel<T, VB, 4, 0>);
    return true;
}

template <typename T>
cudaError_t forward(const LayerNorm& p, cudaStream_t st)
{
    LaunchScope ls("layer_norm", st);
    const int vb = vector_bytes<T>(p);
    cudaError_t e = cudaSuccess;
    if (vb == 16 ? forward_vec<T, 16>(p, st, &e) : vb == 8 ? forward_vec<T, 8>(p, st, &e) : forward_vec<T, sizeof(T)>(p, st, &e)) return e;
    const int64_t segs = p.rows * p.groups;
    layer_norm_kernel<T><<<(unsigned)((segs + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const LayerNorm& p, int parts, cudaStream_t st)
{
    const int64_t segs = p.rows * p.groups;
    const bool params = p.dweight || p.dbias;
    bool done = false;
    if (segs > 0) {
        LaunchScope ls("layer_norm_grad", st);
        const int vb = vector_bytes<T>(p);
        cudaError_t e = cudaSuccess;
        done = vb == 16 ? backward_vec<T, 16>(p, parts, st, &e) : vb == 8 && backward_vec<T, 8>(p, parts, st, &e);
        if (e != cudaSuccess) return e;
        if (!done) layer_norm_dx_kernel<T><<<(unsigned)((segs + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(p);
    }
    if (params) {
        if (!done) {
            LaunchScope ls("layer_norm_dw", st);
            layer_norm_dw_kernel<T><<<dim3((unsigned)((p.channels() + 255) / 256), (unsigned)parts), 256, 0, st>>>(p, parts);
        }
        LaunchScope ls("layer_norm_parts", st);
        const cudaError_t e = pdl_launch(true, layer_norm_parts_kernel, dim3((unsigned)((p.channels() + 31) / 32), 2), 256, 0,
                                         st, p, parts);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

}  // namespace

// Rows a backward pass works on at a time: as many blocks as are resident on the device, but no fewer than
// four rows to each (its partial sums cost as much as some rows; 256 x 2688 bf16 6.2 us, one row each 6.8;
// 512 x 32 groups of 128 6.5 and 9.4) unless that leaves fewer than 64. The vector's width follows from
// addresses that are not known here, so the larger of the two counts is kept.
int layer_norm_parts(int64_t rows, int groups, int width, int act, int sms)
{
    int64_t parts = 64;
    for (int vb = 8; vb <= 16; vb += 8) {
        const int n = vb / (act == SSD_BF16 ? 2 : 4);
        if (width % n) continue;
        const RowShape s = row_shape(groups, width, n);
        if (!s.threads) continue;
        const int64_t fit = rows_at_a_time(s, sms);
        parts = parts > fit ? parts : fit;
    }
    const int64_t four = (rows + 3) / 4, few = four > 64 ? four : (rows < 64 ? rows : 64);
    return (int)(few < 1 ? 1 : (few < parts ? few : parts));
}

cudaError_t launch_layer_norm(const LayerNorm& p, cudaStream_t st)
{
    if (p.rows == 0) return cudaSuccess;
    return p.act == SSD_BF16 ? forward<__nv_bfloat16>(p, st) : forward<float>(p, st);
}

cudaError_t launch_layer_norm_backward(const LayerNorm& p, int parts, cudaStream_t st)
{
    return p.act == SSD_BF16 ? backward<__nv_bfloat16>(p, parts, st) : backward<float>(p, parts, st);
}

}  // namespace ssd

namespace {

ssd_status check_norm(int64_t rows, int32_t groups, int32_t width, int32_t act)
{
    if (rows < 0 || groups <= 0 || width <= 0) return SSD_ERR_INVALID_ARG;
    if (act != SSD_F32 && act != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if ((int64_t)groups * width > (1LL << 24) || rows > 0x7fffff00LL / groups) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}
bool elems_ok(const void* p, int64_t ld, int64_t width, int32_t act)
{
    return ld >= width && ((uintptr_t)p & (act == SSD_BF16 ? 1u : 3u)) == 0;
}
bool floats_ok(const void* p) { return ((uintptr_t)p & 3u) == 0; }

}  // namespace

extern "C" {

ssd_status ssd_mixer_layer_norm(int64_t rows, int32_t groups, int32_t width, float eps, int32_t act, const void* x,
                                int64_t x_ld, const float* weight, const float* bias, void* y, int64_t y_ld, float* mean,
                                float* rstd, void* stream)
{
    const ssd_status cs = check_norm(rows, groups, width, act);
    if (cs != SSD_OK) return cs;
    if (!(eps >= 0.0f)) return SSD_ERR_INVALID_ARG;
    if (rows == 0) return SSD_OK;
    if (!x || !y) return SSD_ERR_INVALID_ARG;
    const int64_t C = (int64_t)groups * width;
    if (!elems_ok(x, x_ld, C, act) || !elems_ok(y, y_ld, C, act) || !floats_ok(weight) || !floats_ok(bias) ||
        !floats_ok(mean) || !floats_ok(rstd))
        return SSD_ERR_UNSUPPORTED;
    ssd::LayerNorm p{};
    p.rows = rows; p.groups = groups; p.width = width; p.act = act; p.eps = eps;
    p.x = x; p.x_ld = x_ld; p.weight = weight; p.bias = bias;
    p.y = y; p.y_ld = y_ld; p.mean = mean; p.rstd = rstd;
    return ssd::launch_layer_norm(p, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_mixer_layer_norm_backward_workspace_size(int64_t rows, int32_t groups, int32_t width, int32_t act)
{
    if (check_norm(rows, groups, width, act) != SSD_OK) return 0;
    return (size_t)ssd::layer_norm_parts(rows, groups, width, act, ssd::device_sm_count()) * 2 * groups * width * 4;
}

ssd_status ssd_mixer_layer_norm_backward(int64_t rows, int32_t groups, int32_t width, int32_t act, const void* dy,
                                         int64_t dy_ld, const void* x, int64_t x_ld, const float* weight, const float* mean,
                                         const float* rstd, void* dx, int64_t dx_ld, float* dweight, float* dbias,
                                         void* workspace, size_t workspace_bytes, void* stream)
{
    const ssd_status cs = check_norm(rows, groups, width, act);
    if (cs != SSD_OK) return cs;
    const int parts = ssd::layer_norm_parts(rows, groups, width, act, ssd::device_sm_count());
    const int64_t C = (int64_t)groups * width;
    if (dweight || dbias) {
        if (!workspace || workspace_bytes < (size_t)parts * 2 * C * 4 || ((uintptr_t)workspace & 255u)) return SSD_ERR_INVALID_ARG;
    }
    if (rows > 0) {
        if (!dy || !x || !mean || !rstd || !dx) return SSD_ERR_INVALID_ARG;
        if (!elems_ok(dy, dy_ld, C, act) || !elems_ok(x, x_ld, C, act) || !elems_ok(dx, dx_ld, C, act) || !floats_ok(mean) ||
            !floats_ok(rstd))
            return SSD_ERR_UNSUPPORTED;
    }
    if (!floats_ok(weight) || !floats_ok(dweight) || !floats_ok(dbias)) return SSD_ERR_UNSUPPORTED;
    ssd::LayerNorm p{};
    p.rows = rows; p.groups = groups; p.width = width; p.act = act;
    p.x = x; p.x_ld = x_ld; p.dy = dy; p.dy_ld = dy_ld; p.weight = weight;
    p.y = dx; p.y_ld = dx_ld;
    p.mean = const_cast<float*>(mean); p.rstd = const_cast<float*>(rstd);
    p.dweight = dweight; p.dbias = dbias;
    p.part = dweight || dbias ? (float*)workspace : nullptr;   // checked above only where it is wanted
    return ssd::launch_layer_norm_backward(p, parts, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
