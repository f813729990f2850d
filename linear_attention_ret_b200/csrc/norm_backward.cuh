// Backward of the output epilogue (norm.cuh): with r = rsqrt(mean_c o^2 + eps),
// sig = 1 / (1 + e^-g) and u = dy swish(g),
//   do = r u - o r^3 mean_c (u o),   dg = dy o r (sig + swish(g) (1 - sig)).
// dy, gate and dgate are token-major [B, N, H, dv], o and do head-major [B, H, N, dv]. Five tensors cross HBM
// once each, about 30 instructions per element: HBM-bound.
#pragma once

#include "norm.cuh"
#include "vec.cuh"

namespace ret {

// sig as in swish() (norm.cuh): relative errors about 2^-22 and 1 ulp.
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
// values, 93 registers and two blocks: 60.2 us at the 1.3B-shaped output (336 MB), 54.8 us with three
// blocks (6.13 TB/s; 80 registers, 16 bytes spilled), 59.8 us with four, which spill more. Longer bf16 rows
// spill 80 to 92 bytes at their one or two blocks.
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

// Any dv and alignment: one warp per row, two passes over the row (the second from L1/L2). An
// ordinary launch: it has no wait for the kernel before it (likewise the general kernels of the other
// operators around retention).
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
