// ssd_layer_norm.cu -- layer norm over contiguous groups of a row's channels, and its gradients.
//
//   y = (x - m) r w + b,   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps)
//   with xh = (x - m) r and dh = dy w:
//   dx = r (dh - mean(dh) - xh mean(dh xh)),   dw = sum over rows of dy xh,   db = sum of dy
// All sums in fp32, the variance around the mean (no difference of large sums).
//
// Both passes are bound by memory: x (and dy) are read once into registers and y (dx) written once.
// A thread holds NV vectors of 16 (or, for rows that only 8 divides, 8) bytes of its row; a group is
// summed by a team, either a power of two of lanes of one warp (head norms: no barrier at all) or
// the whole block. Rows that are not so aligned, and teams that would not fit, take a loop of one
// warp per (row, group).
// Forwards a block runs one row, or (lane teams) four rows whose loads are all in flight before the
// first sum; the other blocks of the SM hide its latency. Backwards a block keeps its columns'
// weight gradients in registers over many rows, the coming rows on their way into shared memory,
// and leaves one partial sum; a second kernel adds those in a fixed order.
#include "../../include/ssd_mixer.h"
#include "ssd_common.cuh"
#include "ssd_layer_norm.h"
#include "ssd_profile.h"

namespace ssd {
namespace {

constexpr int kWarps = 8;

// One warp per (row, group).
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

// Partial sums over a slice of the rows, a thread per channel.
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
// VB bytes of a row: the raw words, and how many elements they are.
template <typename T, int VB>
struct RowVec {
    static constexpr int kN = VB / (int)sizeof(T), kW = VB / 4;
    uint32_t w[kW];
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (VB == 16) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
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
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ void set(const float* f)
    {
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            if constexpr (sizeof(T) == 4) {
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
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
};
// kN parameters from column c (aligned to kN * 4 bytes, at most 16), or a constant.
template <int N>
__device__ __forceinline__ void load_params(const float* p, int64_t c, float none, float* f)
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = none;
    } else if constexpr (N == 2) {
        const float2 v = *reinterpret_cast<const float2*>(p + c);
        f[0] = v.x; f[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + c + i);
            f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
        }
    }
}

// Sum over a team of TEAM lanes, or (TEAM = 0) over the block: red holds 32 values a call, and calls
// alternate between two of them, so that one barrier a call is enough.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float* red)
{
#pragma unroll
    for (int o = (TEAM ? TEAM : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TEAM == 0) {
        const int warps = (blockDim.x + 31) >> 5, lane = threadIdx.x & 31;
        if (lane == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? red[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}
template <int TEAM>
__device__ __forceinline__ float2 team_sum2(float2 v, float2* red)
{
#pragma unroll
    for (int o = (TEAM ? TEAM : 32) / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (TEAM == 0) {
        const int warps = (blockDim.x + 31) >> 5, lane = threadIdx.x & 31;
        if (lane == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
    }
    return v;
}

// TEAM lanes per group and R rows at a time (NV = 1), or the block on one group of one row (R = 1).
template <typename T, int VB, int NV, int TEAM, int R>
__global__ void __launch_bounds__(TEAM ? 256 : 1024) layer_norm_vec_kernel(const LayerNorm p)
{
    using V = RowVec<T, VB>;
    static_assert(TEAM == 0 ? R == 1 : NV == 1, "lane teams hold one vector a lane, blocks one row");
    __shared__ float red[2][32];
    int64_t row0;
    int g, t;
    if constexpr (TEAM != 0) {
        const int64_t id = ((int64_t)blockIdx.x * 256 + threadIdx.x) / TEAM;   // rows R to a team, groups fastest
        g = (int)(id % p.groups);
        row0 = id / p.groups * R;
        t = threadIdx.x % TEAM;
    } else {
        g = (int)(blockIdx.x % p.groups);
        row0 = blockIdx.x / p.groups;
        t = threadIdx.x;
    }
    const int step = TEAM ? TEAM : blockDim.x, vecs = p.width / V::kN;
    const float inv = 1.0f / (float)p.width;
    const T* x = (const T*)p.x + (int64_t)g * p.width;
    T* y = (T*)p.y + (int64_t)g * p.width;
    V v[R][NV];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[r][i].zero();
            if (t + i * step < vecs && row0 + r < p.rows) v[r][i].load(x + (row0 + r) * p.x_ld + (int64_t)(t + i * step) * V::kN);
        }
    float w[NV][V::kN], b[NV][V::kN];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (t + i * step < vecs && NV <= 2) {
            load_params<V::kN>(p.weight, (int64_t)g * p.width + (t + i * step) * V::kN, 1.0f, w[i]);
            load_params<V::kN>(p.bias, (int64_t)g * p.width + (t + i * step) * V::kN, 0.0f, b[i]);
        }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V::kN; ++e) s += v[r][i].at(e);
        const float m = team_sum<TEAM>(s, red[0]) * inv;
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t + i * step < vecs)
#pragma unroll
                for (int e = 0; e < V::kN; ++e) {
                    const float d = v[r][i].at(e) - m;
                    s = fmaf(d, d, s);
                }
        const float rs = 1.0f / sqrtf(team_sum<TEAM>(s, red[1]) * inv + p.eps);
        if (row0 + r >= p.rows) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t + i * step < vecs) {
                if constexpr (NV > 2) {      // many vectors: the parameters would not fit beside them
                    load_params<V::kN>(p.weight, (int64_t)g * p.width + (t + i * step) * V::kN, 1.0f, w[i]);
                    load_params<V::kN>(p.bias, (int64_t)g * p.width + (t + i * step) * V::kN, 0.0f, b[i]);
                }
                float f[V::kN];
#pragma unroll
                for (int e = 0; e < V::kN; ++e) f[e] = fmaf((v[r][i].at(e) - m) * rs, w[i][e], b[i][e]);
                V o;
                o.set(f);
                o.store(y + (row0 + r) * p.y_ld + (int64_t)(t + i * step) * V::kN);
            }
        if (t == 0) {
            const int64_t seg = (row0 + r) * p.groups + g;
            if (p.mean) p.mean[seg] = m;
            if (p.rstd) p.rstd[seg] = rs;
        }
    }
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

// dx, and this block's share of dweight and dbias. Lane teams: the block's columns are blockDim.x
// vectors from blockIdx.x * blockDim.x; block teams: group blockIdx.x. Rows blockIdx.y, blockIdx.y +
// gridDim.y, .. The coming rows wait in shared memory, where each thread copies and reads its own
// vectors only: several rows deep without a register or a barrier for it (two rows ahead in registers
// spilled, one row was not enough in flight).
constexpr int ring_rows(int nv) { return nv == 1 ? 4 : 3; }   // 128 KB of 1024 threads, 192 KB of 512 with four vectors
template <typename T, int VB, int NV, int TEAM>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) layer_norm_grad_kernel(const LayerNorm p)
{
    using V = RowVec<T, VB>;
    constexpr int kRing = ring_rows(NV);
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ float2 red[2][32];
    const int step = blockDim.x, tid = threadIdx.x;
    const int64_t C = p.channels();
    const int64_t c0 = TEAM ? (int64_t)blockIdx.x * blockDim.x * V::kN : (int64_t)blockIdx.x * p.width;   // first column
    const int vecs = TEAM ? (int)((C - c0) / V::kN < step ? (C - c0) / V::kN : step) : p.width / V::kN;
    const int g = TEAM ? (int)((c0 + (int64_t)(tid < vecs ? tid : 0) * V::kN) / p.width) : (int)blockIdx.x;
    const float inv = 1.0f / (float)p.width;
    const T* x = (const T*)p.x + c0;
    const T* dy = (const T*)p.dy + c0;
    T* dx = (T*)p.y + c0;
    const uint32_t ring0 = (uint32_t)__cvta_generic_to_shared(ring);
    // slot a, operand o, vector i of this thread
    auto at = [&](int a, int o, int i) { return (uint32_t)((((a * 2 + o) * NV + i) * step + tid) * VB); };
    auto fetch = [&](int64_t row, int a) {
        if (row < p.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (tid + i * step < vecs) {
                    copy_async<VB>(ring0 + at(a, 0, i), x + row * p.x_ld + (int64_t)(tid + i * step) * V::kN);
                    copy_async<VB>(ring0 + at(a, 1, i), dy + row * p.dy_ld + (int64_t)(tid + i * step) * V::kN);
                }
        }
        copy_commit();
    };
    float dw[NV][V::kN], db[NV][V::kN], w[V::kN];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V::kN; ++e) dw[i][e] = db[i][e] = 0.0f;
    int64_t row = blockIdx.y;
    const int64_t stride = gridDim.y;
#pragma unroll
    for (int a = 0; a < kRing - 1; ++a) fetch(row + a * stride, a);
    if (NV == 1) load_params<V::kN>(tid < vecs ? p.weight : nullptr, c0 + tid * V::kN, 1.0f, w);
    float m_next = 0.0f, r_next = 0.0f;
    if (row < p.rows) {
        m_next = p.mean[row * p.groups + g];
        r_next = p.rstd[row * p.groups + g];
    }
    int slot = 0;
    for (int k = 0; row < p.rows; row += stride, ++k) {
        const float m = m_next, rs = r_next;
        if (row + stride < p.rows) {
            m_next = p.mean[(row + stride) * p.groups + g];
            r_next = p.rstd[(row + stride) * p.groups + g];
        }
        copy_wait<kRing - 2>();
        V vx[NV], vd[NV];
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            vx[i].zero();
            vd[i].zero();
            if (tid + i * step < vecs) {
                vx[i].load(reinterpret_cast<const T*>(ring + at(slot, 0, i)));
                vd[i].load(reinterpret_cast<const T*>(ring + at(slot, 1, i)));
                if (NV > 1) load_params<V::kN>(p.weight, c0 + (tid + i * step) * V::kN, 1.0f, w);
#pragma unroll
                for (int e = 0; e < V::kN; ++e) {
                    const float d = vd[i].at(e), xh = (vx[i].at(e) - m) * rs, dh = d * w[e];
                    dw[i][e] = fmaf(d, xh, dw[i][e]);
                    db[i][e] += d;
                    s.x += dh;
                    s.y = fmaf(dh, xh, s.y);
                }
            }
        }
        // this thread has read the slot that the row kRing - 1 further on goes to one row ago
        fetch(row + (kRing - 1) * stride, slot == 0 ? kRing - 1 : slot - 1);
        slot = slot == kRing - 1 ? 0 : slot + 1;
        s = team_sum2<TEAM>(s, red[k & 1]);
        const float s1 = s.x * inv, s2 = s.y * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (tid + i * step < vecs) {
                if (NV > 1) load_params<V::kN>(p.weight, c0 + (tid + i * step) * V::kN, 1.0f, w);
                float f[V::kN];
#pragma unroll
                for (int e = 0; e < V::kN; ++e) f[e] = rs * (vd[i].at(e) * w[e] - s1 - (vx[i].at(e) - m) * rs * s2);
                V o;
                o.set(f);
                o.store(dx + row * p.y_ld + (int64_t)(tid + i * step) * V::kN);
            }
    }
    copy_wait<0>();
    if (!p.part) return;
    float* part = p.part + (int64_t)blockIdx.y * 2 * C + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (tid + i * step < vecs)
#pragma unroll
            for (int e = 0; e < V::kN; ++e) {
                part[(tid + i * step) * V::kN + e] = dw[i][e];
                part[C + (tid + i * step) * V::kN + e] = db[i][e];
            }
}

// Sums of the partial sums, 32 channels a block, its 8 warps sharing the parts: each in order, then
// the warps in order.
__global__ void __launch_bounds__(256) layer_norm_parts_kernel(const LayerNorm p, int parts)
{
    __shared__ float s[8][32];
    const int64_t C = p.channels(), c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const int warp = threadIdx.x >> 5;
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
        const uintptr_t par = n * 4 < 16 ? n * 4 : 16;
        if (p.width % n || (uintptr_t)p.x % vb || (uintptr_t)p.y % vb || (uintptr_t)p.dy % vb || p.x_ld % n || p.y_ld % n ||
            p.dy_ld % n || (uintptr_t)p.weight % par || (uintptr_t)p.bias % par)
            continue;
        return vb;
    }
    return 0;
}
bool lane_team(int vecs) { return vecs >= 2 && vecs <= 32 && (vecs & (vecs - 1)) == 0; }
int round32(int64_t v) { return (int)((v + 31) / 32 * 32); }

template <typename T, int VB>
bool forward_vec(const LayerNorm& p, cudaStream_t st)
{
    const int vecs = p.width / RowVec<T, VB>::kN;
    if (lane_team(vecs)) {
        constexpr int R = 4;
        const int64_t teams = (p.rows + R - 1) / R * p.groups;
        const unsigned grid = (unsigned)((teams * vecs + 255) / 256);
        switch (vecs) {
        case 2: layer_norm_vec_kernel<T, VB, 1, 2, R><<<grid, 256, 0, st>>>(p); break;
        case 4: layer_norm_vec_kernel<T, VB, 1, 4, R><<<grid, 256, 0, st>>>(p); break;
        case 8: layer_norm_vec_kernel<T, VB, 1, 8, R><<<grid, 256, 0, st>>>(p); break;
        case 16: layer_norm_vec_kernel<T, VB, 1, 16, R><<<grid, 256, 0, st>>>(p); break;
        default: layer_norm_vec_kernel<T, VB, 1, 32, R><<<grid, 256, 0, st>>>(p); break;
        }
        return true;
    }
    if (vecs < 32 || vecs > 4096) return false;
    const unsigned grid = (unsigned)(p.rows * p.groups);
    if (vecs <= 256) layer_norm_vec_kernel<T, VB, 1, 0, 1><<<grid, round32(vecs), 0, st>>>(p);
    else if (vecs <= 512) layer_norm_vec_kernel<T, VB, 2, 0, 1><<<grid, round32((vecs + 1) / 2), 0, st>>>(p);
    else layer_norm_vec_kernel<T, VB, 4, 0, 1><<<grid, round32((vecs + 3) / 4), 0, st>>>(p);
    return true;
}

// Blocks of the gradient kernel: threads, vectors a thread, blocks across the columns.
struct GradShape {
    int threads, nv, cols;
};
GradShape grad_shape(int groups, int width, int vec)
{
    const int vecs = width / vec;
    if (lane_team(vecs)) {
        const int64_t all = (int64_t)groups * vecs;
        const int th = all >= 512 ? 512 : round32(all);
        return {th, 1, (int)((all + th - 1) / th)};
    }
    if (vecs < 32 || vecs > 4096) return {0, 0, 0};
    if (vecs <= 1024) return {round32(vecs), 1, groups};
    if (vecs <= 2048) return {round32((vecs + 3) / 4), 4, groups};
    return {0, 0, 0};
}

template <typename T, int VB, int NV, int TEAM>
cudaError_t launch_grad(const LayerNorm& p, const GradShape& s, int parts, cudaStream_t st)
{
    const int smem = ring_rows(NV) * 2 * NV * s.threads * VB;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(layer_norm_grad_kernel<T, VB, NV, TEAM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    layer_norm_grad_kernel<T, VB, NV, TEAM><<<dim3((unsigned)s.cols, (unsigned)parts), s.threads, smem, st>>>(p);
    return cudaGetLastError();
}

// False: not a shape that the vector kernel takes.
template <typename T, int VB>
bool backward_vec(const LayerNorm& p, int parts, cudaStream_t st, cudaError_t* e)
{
    const GradShape s = grad_shape(p.groups, p.width, RowVec<T, VB>::kN);
    if (!s.threads) return false;
    const int vecs = p.width / RowVec<T, VB>::kN;
    if (lane_team(vecs)) {
        switch (vecs) {
        case 2: *e = launch_grad<T, VB, 1, 2>(p, s, parts, st); break;
        case 4: *e = launch_grad<T, VB, 1, 4>(p, s, parts, st); break;
        case 8: *e = launch_grad<T, VB, 1, 8>(p, s, parts, st); break;
        case 16: *e = launch_grad<T, VB, 1, 16>(p, s, parts, st); break;
        default: *e = launch_grad<T, VB, 1, 32>(p, s, parts, st); break;
        }
    } else {
        *e = s.nv == 1 ? launch_grad<T, VB, 1, 0>(p, s, parts, st) : launch_grad<T, VB, 4, 0>(p, s, parts, st);
    }
    return true;
}

template <typename T>
cudaError_t forward(const LayerNorm& p, cudaStream_t st)
{
    LaunchScope ls("layer_norm", st);
    const int vb = vector_bytes<T>(p);
    if (vb == 16 ? forward_vec<T, 16>(p, st) : vb == 8 && forward_vec<T, 8>(p, st)) return cudaGetLastError();
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
        layer_norm_parts_kernel<<<dim3((unsigned)((p.channels() + 31) / 32), 2), 256, 0, st>>>(p, parts);
    }
    return cudaGetLastError();
}

}  // namespace

// Rows a backward pass works on at a time: as many blocks as fit on the device at 64 registers a
// thread (1024 threads an SM). The vector's width follows from addresses that are not known here, so
// the larger of the two counts is kept.
int layer_norm_parts(int64_t rows, int groups, int width, int act, int sms)
{
    int64_t parts = 64;
    for (int vb = 8; vb <= 16; vb += 8) {
        const int n = vb / (act == SSD_BF16 ? 2 : 4);
        if (width % n) continue;
        const GradShape s = grad_shape(groups, width, n);
        if (!s.threads) continue;
        const int64_t fit = (int64_t)sms * (1024 / s.threads > 1 ? 1024 / s.threads : 1) / s.cols;
        parts = parts > fit ? parts : fit;
    }
    return (int)(rows < 1 ? 1 : (rows < parts ? rows : parts));
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
    p.dweight = dweight; p.dbias = dbias; p.part = (float*)workspace;
    return ssd::launch_layer_norm_backward(p, parts, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
