// ssd_layer_norm.h -- launch parameters of the grouped layer norm and its backward pass.
#pragma once

#include "ssd_internal.h"

namespace ssd {

// Each row's groups * width channels are normalised in contiguous groups of width.
struct LayerNorm {
    int64_t rows;
    int groups, width, act;
    float eps;
    const void *x, *dy;
    int64_t x_ld, dy_ld;
    const float *weight, *bias;     // [groups * width], or nullptr: ones, zeros
    void* y;                        // y, or dx in the backward pass
    int64_t y_ld;
    float *mean, *rstd;             // [rows][groups]; written forwards (nullptr: not wanted), read backwards
    float *dweight, *dbias;         // [groups * width], or nullptr: not wanted
    float* part;                    // workspace: [layer_norm_parts][2][groups * width]; nullptr: no parameter gradients wanted

    SSD_HD int64_t channels() const { return (int64_t)groups * width; }
};

// Partial sums of the parameter gradients that a backward pass keeps.
int layer_norm_parts(int64_t rows, int groups, int width, int act, int sms);
cudaError_t launch_layer_norm(const LayerNorm& p, cudaStream_t st);
cudaError_t launch_layer_norm_backward(const LayerNorm& p, int parts, cudaStream_t st);

}  // namespace ssd
