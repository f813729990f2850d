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

// VE weights as floats (vector path: the pointer is aligned to the vector, at most 16 bytes).
template <typename W, int VE>
__device__ __forceinline__ void ln_weights(const W* w, float* f) {
    constexpr int kPart = VE * (int)sizeof(W) <= 16 ? VE : 16 / (int)sizeof(W);
#pragma unroll
    for (int e = 0; e < VE; e += kPart) Vec<W, kPart>::unpack(Vec<W, kPart>::load(w + e), f + e);
}

// A row's threads: `lanes` lanes of a warp (a power of two), or the whole block. The sums of K
// values over them, in every one of them; sm (block form) holds K rows of 32 and is not reused
// before the next barrier.
template <bool WARP, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], int lanes, float (*sm)[32]) {
    for (int off = WARP ? lanes >> 1 : 16; off > 0; off >>= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
    }
    if (!WARP) {
        const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
        if ((threadIdx.x & 31) < K) {
            float mine = v[0];
#pragma unroll
            for (int k = 1; k < K; ++k) mine = (threadIdx.x & 31) == k ? v[k] : mine;
            sm[threadIdx.x & 31][warp] = mine;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float t = 0.f;
            for (int i = 0; i < warps; i += 4) {
                const float4 q = *reinterpret_cast<const float4*>(&sm[k][i]);
                t += q.x;
                if (i + 1 < warps) t += q.y;
                if (i + 2 < warps) t += q.z;
                if (i + 3 < warps) t += q.w;
            }
            v[k] = t;
        }
    }
}

// One row per `lanes` lanes of a warp (WARP), or per block; a thread keeps EPT elements of it, in
// vectors of VE, as floats: the row is read once, and the mean and then the centred squares are
// summed from registers.
template <typename T, typename W, int VE, int EPT, bool WARP>
__global__ void __launch_bounds__(WARP ? kLnThreads : 1024)
ln_forward_kernel(const T* x, const T* res, const W* __restrict__ weight, const W* __restrict__ bias, T* y, T* sum_out,
                  float* __restrict__ mean, float* __restrict__ rstd, unsigned rows, int D, float eps, int lanes) {
    using V = Vec<T, VE>;
    constexpr int CH = EPT / VE;
    __shared__ __align__(16) float sm[2][1][32];
    const int sub = WARP ? threadIdx.x & (lanes - 1) : threadIdx.x;
    const unsigned r = WARP ? (unsigned)((blockIdx.x * (size_t)kLnThreads + threadIdx.x) / lanes) : blockIdx.x;
    const bool live = r < rows;
    const size_t at = (size_t)r * D;
    const int chunks = D / VE;
    float v[CH][VE];
    {
        typename V::Raw xr[CH], rr[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = sub + c * lanes;
            xr[c] = rr[c] = V::zero();
            if (live && i < chunks) {
                xr[c] = V::load_cs(x + at + i * VE);
                if (res) rr[c] = V::load_cs(res + at + i * VE);
            }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            V::unpack(xr[c], v[c]);
            if (res) {
                float f[VE];
                V::unpack(rr[c], f);
#pragma unroll
                for (int e = 0; e < VE; ++e) v[c][e] += f[e];
            }
        }
    }
    const float inv = 1.f / (float)D;
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < VE; ++e) s[0] += v[c][e];
    row_sums<WARP>(s, lanes, sm[0]);
    const float mu = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (sub + c * lanes < chunks) {
#pragma unroll
            for (int e = 0; e < VE; ++e) s[0] = fmaf(v[c][e] - mu, v[c][e] - mu, s[0]);
        }
    }
    row_sums<WARP>(s, lanes, sm[1]);
    const float rs = rsqrtf(s[0] * inv + eps);
    if (!live) return;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = sub + c * lanes;
        if (i >= chunks) continue;
        if (sum_out) V::store(sum_out + at + i * VE, v[c]);
        float w[VE], b[VE];
        if (weight) ln_weights<W, VE>(weight + i * VE, w);
        if (bias) ln_weights<W, VE>(bias + i * VE, b);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            float z = (v[c][e] - mu) * rs;
            if (weight) z *= w[e];
            if (bias) z += b[e];
            v[c][e] = z;
        }
        V::store(y + at + i * VE, v[c]);
    }
    if (sub == 0) {
        if (mean) mean[r] = mu;
        if (rstd) rstd[r] = rs;
    }
}

// dx and the column sums in one pass: blocks stay, and a thread keeps the same EPT columns of
// every row it takes, their dw and db sums in registers. The next row's loads are issued before
// the current row's two sums are reduced. Each block ends with one row of partial sums, part
// [gridDim.x, 2, D]; ln_reduce_kernel adds those in block order.
template <typename T, typename W, int VE, int EPT, bool WARP>
__global__ void __launch_bounds__(WARP ? kLnThreads : (EPT <= 8 ? 1024 : 512))
ln_backward_kernel(const T* dy, const T* x, const W* __restrict__ weight, const float* __restrict__ mean,
                   const float* __restrict__ rstd, const T* dsum, T* dx, float* __restrict__ part, unsigned rows, int D,
                   int lanes) {
    using V = Vec<T, VE>;
    constexpr int CH = EPT / VE;
    extern __shared__ float ln_sm[];  // WARP: [2, D] for joining the warps' column sums
    __shared__ __align__(16) float sm[2][2][32];
    const int sub = WARP ? threadIdx.x & (lanes - 1) : threadIdx.x;
    const unsigned per_block = WARP ? kLnThreads / lanes : 1, mine = WARP ? threadIdx.x / lanes : 0;
    const unsigned step = gridDim.x * per_block;
    const int chunks = D / VE;
    const float inv = 1.f / (float)D;
    float w[CH][VE], dw[CH][VE], db[CH][VE];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            w[c][e] = 1.f;
            dw[c][e] = db[c][e] = 0.f;
        }
        if (weight && sub + c * lanes < chunks) ln_weights<W, VE>(weight + (sub + c * lanes) * VE, w[c]);
    }
    struct Row {
        typename V::Raw g[CH], x[CH], s[CH];
        float mu, rs;
    };
    auto load = [&](Row& q, unsigned r) {
        const size_t at = (size_t)r * D;
        const bool live = r < rows;
        q.mu = live ? mean[r] : 0.f;
        q.rs = live ? rstd[r] : 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = sub + c * lanes;
            q.g[c] = q.x[c] = q.s[c] = V::zero();
            if (live && i < chunks) {
                q.g[c] = V::load_cs(dy + at + i * VE);
                q.x[c] = V::load_cs(x + at + i * VE);
                if (dsum) q.s[c] = V::load_cs(dsum + at + i * VE);
            }
        }
    };
    Row cur;
    unsigned base = blockIdx.x * per_block;  // every thread of a block makes the same trips
    load(cur, base + mine);
    for (int flip = 0; base < rows; base += step, flip ^= 1) {
        const unsigned r = base + mine;
        Row next;
        load(next, r + step);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float g[VE], z[VE];
            V::unpack(cur.g[c], g);
            V::unpack(cur.x[c], z);
            const bool on = sub + c * lanes < chunks;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float xh = on ? (z[e] - cur.mu) * cur.rs : 0.f, u = g[e] * w[c][e];
                s[0] += u;
                s[1] = fmaf(u, xh, s[1]);
                dw[c][e] = fmaf(g[e], xh, dw[c][e]);
                db[c][e] += g[e];
            }
        }
        row_sums<WARP>(s, lanes, sm[flip]);
        const float m0 = s[0] * inv, m1 = s[1] * inv;
        const size_t at = (size_t)r * D;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = sub + c * lanes;
            if (r >= rows || i >= chunks) continue;
            float g[VE], z[VE], a[VE];
            V::unpack(cur.g[c], g);
            V::unpack(cur.x[c], z);
            V::unpack(cur.s[c], a);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float xh = (z[e] - cur.mu) * cur.rs;
                z[e] = cur.rs * (g[e] * w[c][e] - m0 - xh * m1) + (dsum ? a[e] : 0.f);
            }
            V::store(dx + at + i * VE, z);
        }
        cur = next;
    }
    if (!part) return;
    float* out = part + (size_t)blockIdx.x * 2 * D;
    if (WARP) {  // the groups of a warp, then the warps one after another
        for (int off = 16; off >= lanes; off >>= 1) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    dw[c][e] += __shfl_xor_sync(0xffffffffu, dw[c][e], off);
                    db[c][e] += __shfl_xor_sync(0xffffffffu, db[c][e], off);
                }
        }
        for (int q = 0; q < kLnThreads / 32; ++q) {
            if ((int)(threadIdx.x >> 5) == q && (threadIdx.x & 31) < lanes) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const int i = sub + c * lanes;
                    if (i >= chunks) continue;
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        float* a = ln_sm + i * VE + e;
                        a[0] = q ? a[0] + dw[c][e] : dw[c][e];
                        a[D] = q ? a[D] + db[c][e] : db[c][e];
                    }
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * D; c += kLnThreads) out[c] = ln_sm[c];
    } else {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = sub + c * lanes;
            if (i >= chunks) continue;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                out[i * VE + e] = dw[c][e];
                out[D + i * VE + e] = db[c][e];
            }
        }
    }
}

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

// dw and db from `parts` rows of partial sums [2, D]: 32 columns per block, eight threads per
// column over every eighth row, then those eight one after another.
constexpr int kReduceSlices = kLnThreads / 32;
template <typename W>
__global__ void __launch_bounds__(kLnThreads)
ln_reduce_kernel(const float* __restrict__ part, int parts, W* __restrict__ dweight, W* __restrict__ dbias, int D) {
    __shared__ float sm[kReduceSlices][32];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const long long c = blockIdx.x * 32LL + lane;  // of 2 D
    float t = 0.f;
    if (c < 2LL * D) {
#pragma unroll 8
        for (int p = slice; p < parts; p += kReduceSlices) t += part[(size_t)p * 2 * D + c];
    }
    sm[slice][lane] = t;
    __syncthreads();
    if (slice == 0 && c < 2LL * D) {
#pragma unroll
        for (int i = 1; i < kReduceSlices; ++i) t += sm[i][lane];
        W* out = c < D ? dweight : dbias;
        if (out) st_elem(out + (c < D ? c : c - D), t);
    }
}

}  // namespace ret
