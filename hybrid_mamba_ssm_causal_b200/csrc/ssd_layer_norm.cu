// ssd_layer_norm.cu -- layer norm over contiguous groups of a row's channels, and its gradients.
//
//   y = (x - m) r w + b,   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps)
//   with xh = (x - m) r and dh = dy w:
//   dx = r (dh - mean(dh) - xh mean(dh xh)),   dw = sum over rows of dy xh,   db = sum of dy
// All sums in fp32, the variance around the mean (no difference of large sums).
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

// The partial sums in a fixed order.
__global__ void __launch_bounds__(256) layer_norm_sum_kernel(const LayerNorm p, int parts)
{
    const int64_t C = p.channels(), c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= C) return;
    float dw = 0.0f, db = 0.0f;
    for (int i = 0; i < parts; ++i) {
        dw += p.part[((int64_t)i * 2 + 0) * C + c];
        db += p.part[((int64_t)i * 2 + 1) * C + c];
    }
    if (p.dweight) p.dweight[c] = dw;
    if (p.dbias) p.dbias[c] = db;
}

template <typename T>
cudaError_t forward(const LayerNorm& p, cudaStream_t st)
{
    LaunchScope ls("layer_norm", st);
    const int64_t segs = p.rows * p.groups;
    layer_norm_kernel<T><<<(unsigned)((segs + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const LayerNorm& p, int parts, cudaStream_t st)
{
    const int64_t segs = p.rows * p.groups;
    const unsigned cols = (unsigned)((p.channels() + 255) / 256);
    if (segs > 0) {
        LaunchScope ls("layer_norm_dx", st);
        layer_norm_dx_kernel<T><<<(unsigned)((segs + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(p);
    }
    if (p.dweight || p.dbias) {
        {
            LaunchScope ls("layer_norm_dw", st);
            layer_norm_dw_kernel<T><<<dim3(cols, (unsigned)parts), 256, 0, st>>>(p, parts);
        }
        LaunchScope ls("layer_norm_sum", st);
        layer_norm_sum_kernel<<<cols, 256, 0, st>>>(p, parts);
    }
    return cudaGetLastError();
}

}  // namespace

int layer_norm_parts(int64_t rows, int groups, int width, int act, int sms)
{
    return (int)(rows < 1 ? 1 : (rows < 64 ? rows : 64));
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
