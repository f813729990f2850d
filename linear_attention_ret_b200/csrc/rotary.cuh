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

// Vectors of VE elements: the items (token, head, unit) of a block's `tokens` tokens are spread
// over its threads, unit fastest, so that a warp reads and writes whole stretches of a head's
// row. A unit is VE consecutive elements (VE / 2 pairs) in the interleaved layout, and in the
// half layout the two vectors whose elements pair up, or one vector behind the rotated part.
// cos and sin of a token are formed once per block, in shared memory, and serve all heads of
// q and k (16 rows in a 1.3B-shaped layer); a block's first loads are in flight meanwhile.
struct RotPlan {
    FastDiv units, heads, N;  // units of a head; heads of q and k together; tokens of a batch
    int tokens;            // of a block
    int half_units;        // half layout: units of two vectors
    int stride;            // of a token's cos (or sin) in shared memory, in floats
};

template <typename T, int VE, bool HALF, int ITEMS>
__global__ void __launch_bounds__(kRotThreads) rotary_vec_kernel(const RotArgs a, const RotPlan pl) {
    using V = Vec<T, VE>;
    constexpr int P = HALF ? VE : VE / 2;  // frequencies of a unit
    extern __shared__ float4 rot_sm[];
    float* cs = reinterpret_cast<float*>(rot_sm);
    float* sn = cs + pl.tokens * pl.stride;
    const unsigned all = (unsigned)a.B * a.N, first = blockIdx.x * (unsigned)pl.tokens;  // below 2^31
    const int tokens = (int)min((unsigned)pl.tokens, all - first);
    const unsigned total = (unsigned)tokens * pl.heads.d * pl.units.d;
    const int half = a.rot / 2;
    struct Item {
        T* y;
        float scale;
        int t, u;
        typename V::Raw lo, hi;
    };
    for (unsigned w0 = 0; w0 < total; w0 += kRotThreads * ITEMS) {
        Item it[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const unsigned w = w0 + i * kRotThreads + threadIdx.x;
            if (w >= total) continue;
            unsigned r, u, t, h, b, n;
            pl.units.divmod(w, r, u);
            pl.heads.divmod(r, t, h);
            const bool second = (int)h >= a.x[0].H;
            const RotView& v = a.x[second];
            if (second) h -= a.x[0].H;
            pl.N.divmod(first + t, b, n);
            const int at = HALF && (int)u >= pl.half_units ? a.rot + ((int)u - pl.half_units) * VE : (int)u * VE;
            const T* x = static_cast<const T*>(v.in) + b * v.ib + n * v.in_ + h * v.ih + at;
            it[i].y = static_cast<T*>(v.out) + b * v.ob + n * v.on + h * v.oh + at;
            it[i].scale = v.scale;
            it[i].t = (int)t;
            it[i].u = (int)u;
            it[i].lo = V::load_cs(x);
            if (HALF && (int)u < pl.half_units) it[i].hi = V::load_cs(x + half);
        }
        if (w0 == 0) {
            for (int j = threadIdx.x; j < tokens * half; j += kRotThreads) {
                const int t = j / half, i = j - t * half;
                unsigned b, n;
                pl.N.divmod(first + t, b, n);
                float c, s;
                rot_angle(a, rot_position(a, (int)b, (int)n), i, c, s);
                cs[t * pl.stride + i] = c;
                sn[t * pl.stride + i] = s;
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const unsigned w = w0 + i * kRotThreads + threadIdx.x;
            if (w >= total) continue;
            const float* c = cs + it[i].t * pl.stride + it[i].u * P;
            const float* s = sn + it[i].t * pl.stride + it[i].u * P;
            const float m = it[i].scale;
            float lo[VE];
            V::unpack(it[i].lo, lo);
            if (HALF) {
                if (it[i].u < pl.half_units) {
                    float hi[VE];
                    V::unpack(it[i].hi, hi);
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float p = lo[e], q = hi[e];
                        lo[e] = m * (p * c[e] - q * s[e]);
                        hi[e] = m * (p * s[e] + q * c[e]);
                    }
                    V::store(it[i].y + half, hi);
                } else {
#pragma unroll
                    for (int e = 0; e < VE; ++e) lo[e] *= m;
                }
            } else {
                const int live = min(P, half - it[i].u * P);  // pairs of this unit that are rotated
                auto turn = [&](int e) {
                    const float p = lo[2 * e], q = lo[2 * e + 1];
                    lo[2 * e] = m * (p * c[e] - q * s[e]);
                    lo[2 * e + 1] = m * (p * s[e] + q * c[e]);
                };
                if (live == P) {
#pragma unroll
                    for (int e = 0; e < P; ++e) turn(e);
                } else {
#pragma unroll
                    for (int e = 0; e < P; ++e) {
                        if (e < live) {
                            turn(e);
                        } else {
                            lo[2 * e] *= m;
                            lo[2 * e + 1] *= m;
                        }
                    }
                }
            }
            V::store(it[i].y, lo);
        }
    }
}

// Any width and alignment. One thread per pair, or element behind the rotated part, of q and k.
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
