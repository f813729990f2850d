// Multi-scale retention output epilogue: per-head RMSNorm without affine weights,
// times the swish of the gate projection ("Retentive Network (RetNet) 详解",
// section 3.2: multi-scale retention adds a gate and a normalisation to
// retention; the Gated RetNet page's GateRetention module: subln normalises
// each head over its dimension, g_proj feeds a swish gate):
//   y[b, n, h, :] = swish(gate[b, n, h, :]) * o[b, h, n, :] * rsqrt(mean_c o[b, h, n, c]^2 + eps),
//   swish(x) = x / (1 + e^-x).
// o is the retention output [B, H, N, dv]; gate and y are token-major
// [B, N, H, dv], the layout the module's projections use, so the transpose
// happens here on the way through.
//
// One pass over HBM: every row's O and gate are read once and y written once.
// A group of LPR lanes takes one row; each lane holds CH 16-byte chunks of O
// and of the gate in registers, so all of a row's loads are in flight before
// the sum of squares is reduced across the group with shuffles.
#pragma once

#include "common.cuh"

namespace ret {

constexpr int kNormThreads = 256;

template <typename T> struct Vec16;
template <> struct Vec16<float> {
    static constexpr int kE = 4;
    static __device__ __forceinline__ void unpack(const uint4& u, float* f) {
        f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct Vec16<__nv_bfloat16> {
    static constexpr int kE = 8;
    static __device__ __forceinline__ void unpack(const uint4& u, float* f) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 b;
            memcpy(&b, &w[i], 4);
            const float2 x = __bfloat1622float2(b);
            f[2 * i] = x.x;
            f[2 * i + 1] = x.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            memcpy(&w[i], &b, 4);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// swish(x) = x / (1 + e^-x) = x * rcp(1 + 2^(-x log2 e)) with the hardware ex2 and rcp
// (flush-to-zero forms; relative errors about 2^-22 and 1 ulp): five instructions. The
// flushes only touch e^-x below 2^-126 (where 1 + e^-x rounds to 1 anyway) and results
// below 2^-126 in magnitude (x < -87, where swish(x) is under 1e-36).
__device__ __forceinline__ float swish(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-x * kLog2e));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return x * r;
}

// Source row of o and destination row of y for token-major row index r = (b N + n) H + h.
__device__ __forceinline__ void norm_rows(size_t r, int H, int N, size_t& o_row, size_t& y_row) {
    const int h = (int)(r % H);
    const size_t bn = r / H;
    const int n = (int)(bn % N);
    const size_t b = bn / N;
    o_row = (b * H + h) * N + n;
    y_row = r;
}

// Vector path: dv * sizeof(T) a multiple of 16 and all pointers 16-byte aligned.
// LPR lanes per row (a power of two dividing 32), CH chunks per lane.
template <typename T, int LPR, int CH>
__global__ void __launch_bounds__(kNormThreads)
norm_gate_vec_kernel(const T* __restrict__ o, const T* gate, T* y, int H, int N, int dv, float eps, size_t rows) {
    constexpr int kE = Vec16<T>::kE;
    constexpr int kRowsPerWarp = 32 / LPR;
    const int lane = threadIdx.x & 31, sub = lane % LPR;
    const int chunks = dv / kE;
    const float inv_dv = 1.f / (float)dv;
    const size_t warps = (size_t)gridDim.x * (kNormThreads / 32);
    for (size_t w = (size_t)blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5); w * kRowsPerWarp < rows;
         w += warps) {
        const size_t r = w * kRowsPerWarp + lane / LPR;
        const bool live = r < rows;
        size_t o_row = 0, y_row = 0;
        if (live) norm_rows(r, H, N, o_row, y_row);
        const uint4* op = reinterpret_cast<const uint4*>(o + o_row * dv);
        const uint4* gp = reinterpret_cast<const uint4*>(gate + y_row * dv);
        uint4 ov[CH], gv[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int idx = sub + c * LPR;
            if (live && idx < chunks) {
                ov[c] = __ldcs(op + idx);
                gv[c] = __ldcs(gp + idx);
            } else {
                ov[c] = make_uint4(0, 0, 0, 0);
                gv[c] = make_uint4(0, 0, 0, 0);
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float f[kE];
            Vec16<T>::unpack(ov[c], f);
#pragma unroll
            for (int e = 0; e < kE; ++e) ss = fmaf(f[e], f[e], ss);
        }
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float inv_rms = rsqrtf(ss * inv_dv + eps);
        uint4* yp = reinterpret_cast<uint4*>(y + y_row * dv);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int idx = sub + c * LPR;
            if (live && idx < chunks) {
                float f[kE], g[kE];
                Vec16<T>::unpack(ov[c], f);
                Vec16<T>::unpack(gv[c], g);
#pragma unroll
                for (int e = 0; e < kE; ++e) f[e] = swish(g[e]) * (f[e] * inv_rms);
                yp[idx] = Vec16<T>::pack(f);
            }
        }
    }
}

// Any dv and alignment: one warp per row, two passes over the row (the second
// from L1/L2).
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
norm_gate_scalar_kernel(const T* __restrict__ o, const T* gate, T* y, int H, int N, int dv, float eps, size_t rows) {
    const int lane = threadIdx.x & 31;
    const size_t warps = (size_t)gridDim.x * (kNormThreads / 32);
    for (size_t r = (size_t)blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5); r < rows; r += warps) {
        size_t o_row, y_row;
        norm_rows(r, H, N, o_row, y_row);
        const T* op = o + o_row * dv;
        float ss = 0.f;
        for (int c = lane; c < dv; c += 32) {
            const float x = ld_elem(op + c);
            ss = fmaf(x, x, ss);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float inv_rms = rsqrtf(ss / (float)dv + eps);
        for (int c = lane; c < dv; c += 32)
            st_elem(y + y_row * dv + c, swish(ld_elem(gate + y_row * dv + c)) * (ld_elem(op + c) * inv_rms));
    }
}

// Backward of the epilogue: with r = rsqrt(mean_c o^2 + eps), sig = 1 / (1 + e^-g) and
// u = dy swish(g),
//   do = r u - o r^3 mean_c (u o),   dg = dy o r (sig + swish(g) (1 - sig)).
// sig as in swish() above.
__device__ __forceinline__ float sigmoid(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-x * kLog2e));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// LPR lanes per row, each with CH vectors of VE elements of dy, o and gate in registers, so a
// row is read once and all of its loads are in flight before the two sums are reduced.
// swish(gate) is formed again for the outputs: two more special-function instructions per element
// cost less than the registers. VE = 1 serves rows that are not whole 16-byte chunks: neighbouring
// lanes still read neighbouring elements. A row's place takes two 32-bit divisions by
// multiplication: rows are fewer than 2^31. dgate may be gate or dy, and dout o: an element is
// read by the thread that writes it.
//
// Blocks per SM: left alone, the two-vector form (dv = 512) keeps the first pass's unpacked
// values, 93 registers and two blocks: 60.2 us at the 1.3B-shaped output (336 MB), 55.3 us with three
// blocks (6.07 TB/s), 59.8 us with four, which spill.
template <typename T, int VE, int LPR, int CH>
__global__ void __launch_bounds__(kNormThreads, VE * CH * sizeof(T) <= 32 ? 3 : VE * CH * sizeof(T) <= 64 ? 2 : 1)
norm_gate_backward_vec_kernel(const T* dy, const T* o, const T* gate, T* dout, T* dgate, FastDiv H, FastDiv N, int dv,
                              float eps, unsigned rows) {
    using V = Vec<T, VE>;
    constexpr unsigned kRowsPerWarp = 32 / LPR;
    const int lane = threadIdx.x & 31, sub = lane % LPR;
    const int chunks = dv / VE;
    const float inv_dv = 1.f / (float)dv;
    const unsigned warps = gridDim.x * (kNormThreads / 32);
    wait_previous_kernel();
    for (unsigned w = blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5); w * kRowsPerWarp < rows; w += warps) {
        const unsigned r = w * kRowsPerWarp + lane / LPR;
        const bool live = r < rows;
        unsigned bn, h, b, n;
        H.divmod(live ? r : 0, bn, h);
        N.divmod(bn, b, n);
        const size_t o_row = ((size_t)(b * H.d + h) * N.d + n) * dv, y_row = (size_t)(live ? r : 0) * dv;
        typename V::Raw ov[CH], gv[CH], yv[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int idx = sub + c * LPR;
            ov[c] = gv[c] = yv[c] = V::zero();
            if (live && idx < chunks) {
                ov[c] = V::load_cs(o + o_row + idx * VE);
                gv[c] = V::load_cs(gate + y_row + idx * VE);
                yv[c] = V::load_cs(dy + y_row + idx * VE);
            }
        }
        float ss = 0.f, uo = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float x[VE], g[VE], d[VE];
            V::unpack(ov[c], x);
            V::unpack(gv[c], g);
            V::unpack(yv[c], d);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                ss = fmaf(x[e], x[e], ss);
                uo = fmaf(d[e] * (g[e] * sigmoid(g[e])), x[e], uo);
            }
        }
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, off);
            uo += __shfl_xor_sync(0xffffffffu, uo, off);
        }
        const float inv_rms = rsqrtf(ss * inv_dv + eps);
        const float k = inv_rms * inv_rms * (uo * inv_dv);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int idx = sub + c * LPR;
            if (live && idx < chunks) {
                float x[VE], g[VE], d[VE];
                V::unpack(ov[c], x);
                V::unpack(gv[c], g);
                V::unpack(yv[c], d);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float sig = sigmoid(g[e]), sw = g[e] * sig, z = x[e], t = d[e];
                    x[e] = inv_rms * (t * sw - z * k);
                    d[e] = t * (z * inv_rms) * (sig + sw * (1.f - sig));
                }
                V::store(dout + o_row + idx * VE, x);
                V::store(dgate + y_row + idx * VE, d);
            }
        }
    }
}

// Any dv and alignment: one warp per row, two passes over the row (the second from L1/L2).
// dgate may be gate or dy, and dout o: an element is read by the thread that writes it.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
norm_gate_backward_scalar_kernel(const T* dy, const T* o, const T* gate, T* dout, T* dgate, int H, int N, int dv,
                                 float eps, size_t rows) {
    const int lane = threadIdx.x & 31;
    const size_t warps = (size_t)gridDim.x * (kNormThreads / 32);
    for (size_t r = (size_t)blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5); r < rows; r += warps) {
        size_t o_row, y_row;
        norm_rows(r, H, N, o_row, y_row);
        float ss = 0.f, uo = 0.f;
        for (int c = lane; c < dv; c += 32) {
            const float x = ld_elem(o + o_row * dv + c);
            ss = fmaf(x, x, ss);
            uo = fmaf(ld_elem(dy + y_row * dv + c) * swish(ld_elem(gate + y_row * dv + c)), x, uo);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, off);
            uo += __shfl_xor_sync(0xffffffffu, uo, off);
        }
        const float inv_rms = rsqrtf(ss / (float)dv + eps);
        const float k = inv_rms * inv_rms * (uo / (float)dv);
        for (int c = lane; c < dv; c += 32) {
            const float x = ld_elem(o + o_row * dv + c), g = ld_elem(gate + y_row * dv + c);
            const float d = ld_elem(dy + y_row * dv + c), sig = sigmoid(g);
            st_elem(dout + o_row * dv + c, inv_rms * (d * (g * sig) - x * k));
            st_elem(dgate + y_row * dv + c, d * (x * inv_rms) * (sig + g * sig * (1.f - sig)));
        }
    }
}

}  // namespace ret
