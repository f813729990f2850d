// Layer norm over rows of D elements, its residual form and its backward pass. RetNet's
// blocks normalise the residual stream before the retention sub-layer and before the
// feed-forward one ("Retentive Network (RetNet) 详解", section 3.2's module inside its block).
//   s = x (+ residual),  mu = mean_c s,  r = 1 / sqrt(mean_c (s - mu)^2 + eps),
//   xh = (s - mu) r,     y = w xh + b
//   dx = r (u - mean_c u - xh mean_c (u xh)) (+ dsum),  u = w dy
//   dw = sum_rows dy xh,  db = sum_rows dy
// Statistics and sums are fp32; the variance is of centred values (two passes over the row),
// so a mean far from zero costs no digits. With a residual the statistics and y are of the
// fp32 sum, not of its rounded copy: one rounding less, at no cost.
#pragma once

#include "common.cuh"

namespace ret {

constexpr int kLnThreads = 256;

// Sum over the block, in every thread. `sm` holds one float per warp and may be reused at once.
__device__ __forceinline__ float block_sum(float x, float* sm) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) t += sm[i];
    __syncthreads();
    return t;
}

template <typename W>
__device__ __forceinline__ float ln_weight(const W* w, int c, float none) { return w ? ld_elem(w + c) : none; }

// Any D: one block per row, three passes (the later ones from L1/L2). x, residual, y and
// sum_out may alias element by element: an element is read by the thread that writes it.
template <typename T, typename W>
__global__ void __launch_bounds__(kLnThreads)
ln_forward_rows_kernel(const T* x, const T* res, const W* __restrict__ weight, const W* __restrict__ bias, T* y,
                       T* sum_out, float* __restrict__ mean, float* __restrict__ rstd, size_t rows, int D, float eps) {
    __shared__ float sm[kLnThreads / 32];
    for (size_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const size_t at = r * D;
        auto value = [&](int c) { return ld_elem(x + at + c) + (res ? ld_elem(res + at + c) : 0.f); };
        float s = 0.f;
        for (int c = threadIdx.x; c < D; c += kLnThreads) s += value(c);
        const float mu = block_sum(s, sm) / (float)D;
        float v = 0.f;
        for (int c = threadIdx.x; c < D; c += kLnThreads) {
            const float z = value(c) - mu;
            v = fmaf(z, z, v);
        }
        const float rs = rsqrtf(block_sum(v, sm) / (float)D + eps);
        for (int c = threadIdx.x; c < D; c += kLnThreads) {
            const float z = value(c);
            if (sum_out) st_elem(sum_out + at + c, z);
            st_elem(y + at + c, fmaf((z - mu) * rs, ln_weight(weight, c, 1.f), ln_weight(bias, c, 0.f)));
        }
        if (threadIdx.x == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

// dx of any D: one block per row, two passes.
template <typename T, typename W>
__global__ void __launch_bounds__(kLnThreads)
ln_backward_rows_kernel(const T* dy, const T* x, const W* __restrict__ weight, const float* __restrict__ mean,
                        const float* __restrict__ rstd, const T* dsum, T* dx, size_t rows, int D) {
    __shared__ float sm[kLnThreads / 32];
    for (size_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const size_t at = r * D;
        const float mu = mean[r], rs = rstd[r];
        float a = 0.f, b = 0.f;
        for (int c = threadIdx.x; c < D; c += kLnThreads) {
            const float u = ld_elem(dy + at + c) * ln_weight(weight, c, 1.f);
            a += u;
            b = fmaf(u, (ld_elem(x + at + c) - mu) * rs, b);
        }
        const float ma = block_sum(a, sm) / (float)D, mb = block_sum(b, sm) / (float)D;
        for (int c = threadIdx.x; c < D; c += kLnThreads) {
            const float u = ld_elem(dy + at + c) * ln_weight(weight, c, 1.f);
            const float z = rs * (u - ma - (ld_elem(x + at + c) - mu) * rs * mb);
            st_elem(dx + at + c, dsum ? z + ld_elem(dsum + at + c) : z);
        }
    }
}

// Partial sums of dw and db over every gridDim.y-th row, one column per thread, in
// part [gridDim.y, 2, D]; ln_reduce_kernel adds them in row order, so calls agree bit for bit.
template <typename T>
__global__ void __launch_bounds__(kLnThreads)
ln_backward_columns_kernel(const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ mean,
                           const float* __restrict__ rstd, float* __restrict__ part, size_t rows, int D) {
    const int c = blockIdx.x * kLnThreads + threadIdx.x;
    if (c >= D) return;
    float dw = 0.f, db = 0.f;
    for (size_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const float g = ld_elem(dy + r * D + c);
        dw = fmaf(g, (ld_elem(x + r * D + c) - mean[r]) * rstd[r], dw);
        db += g;
    }
    part[(size_t)blockIdx.y * 2 * D + c] = dw;
    part[((size_t)blockIdx.y * 2 + 1) * D + c] = db;
}

template <typename W>
__global__ void __launch_bounds__(kLnThreads)
ln_reduce_kernel(const float* __restrict__ part, int parts, W* __restrict__ dweight, W* __restrict__ dbias, int D) {
    const int c = blockIdx.x * kLnThreads + threadIdx.x;
    if (c >= D) return;
    float dw = 0.f, db = 0.f;
    for (int p = 0; p < parts; ++p) {
        dw += part[(size_t)p * 2 * D + c];
        db += part[((size_t)p * 2 + 1) * D + c];
    }
    if (dweight) st_elem(dweight + c, dw);
    if (dbias) st_elem(dbias + c, db);
}

}  // namespace ret
