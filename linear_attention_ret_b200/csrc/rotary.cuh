// Rotary prologue of retention: q and k as the projections give them, token-major
// [B, N, H, d] with strides, rotated by their positions and written where retention reads
// them (head-major [B, H, N, d], or any other strides); RetNet rotates its queries and keys
// by e^{i n theta} before retention ("RetNet retention mechanism" page, 保留机制初识).
// For the pair (a, b) at frequency i of a token at position p, with t = p * freqs[i]:
//   a' = s m (a cos t - b sin t),   b' = s m (a sin t + b cos t)
// and s x for the d - rot elements behind the rotated part. The inverse (the gradient, as a
// rotation's transpose is its inverse) takes -t.
//
// The angle is formed in 64 bits: at p = 2^20 a product in fp32 is off by up to 2^-4 rad.
#pragma once

#include "common.cuh"

namespace ret {

constexpr int kRotThreads = 256;

struct RotView {  // strides in elements of batch, token and head; the head dimension is contiguous
    const void* in;
    void* out;
    long long ib, in_, ih, ob, on, oh;
    int H;
    float scale;
};

struct RotArgs {
    RotView x[2];  // q, k
    const double* freqs;
    const long long* positions;  // [B, N] or null
    const long long* starts;     // [B] or null
    long long offset;
    int B, N, d, rot;
    float amplitude;
    float sign;  // -1 for the inverse
};

__device__ __forceinline__ long long rot_position(const RotArgs& a, int b, int n) {
    return a.offset + (a.positions ? a.positions[(size_t)b * a.N + n] : n + (a.starts ? a.starts[b] : 0));
}

// cos and sin of p * f, times the amplitude. The product and its reduction to (-1/2, 1/2]
// turns are in 64 bits, so the fp32 argument of sincospif is off by at most 2^-25 of a half
// turn plus p * f * 2^-53.
__device__ __forceinline__ void rot_angle(const RotArgs& a, long long p, int i, float& c, float& s) {
    double t = (double)p * a.freqs[i] * 0.15915494309189533577;  // 1 / (2 pi)
    t -= rint(t);
    sincospif((float)(2.0 * t), &s, &c);
    c *= a.amplitude;
    s *= a.amplitude * a.sign;
}

// One thread per pair, or element behind the rotated part, of q and k.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotArgs a, size_t total) {
    const int units = a.d - a.rot / 2, H = a.x[0].H + a.x[1].H;
    for (size_t w = (size_t)blockIdx.x * kRotThreads + threadIdx.x; w < total; w += (size_t)gridDim.x * kRotThreads) {
        const int u = (int)(w % units);
        const size_t r = w / units;
        int h = (int)(r % H);
        const size_t bn = r / H;
        const int n = (int)(bn % a.N), b = (int)(bn / a.N);
        const bool second = h >= a.x[0].H;
        const RotView& v = a.x[second];
        if (second) h -= a.x[0].H;
        const T* x = static_cast<const T*>(v.in) + b * v.ib + n * v.in_ + h * v.ih;
        T* y = static_cast<T*>(v.out) + b * v.ob + n * v.on + h * v.oh;
        if (u < a.rot / 2) {
            const int i = HALF ? u : 2 * u, j = HALF ? u + a.rot / 2 : 2 * u + 1;
            float c, s;
            rot_angle(a, rot_position(a, b, n), u, c, s);
            const float p = ld_elem(x + i), q = ld_elem(x + j);
            st_elem(y + i, v.scale * (p * c - q * s));
            st_elem(y + j, v.scale * (p * s + q * c));
        } else {
            const int i = u + a.rot / 2;
            st_elem(y + i, v.scale * ld_elem(x + i));
        }
    }
}

}  // namespace ret
