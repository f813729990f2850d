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

// A thread's EPT elements of a row: vectors sub, sub + lanes, ... of VE elements, as they are in
// memory, and as pairs of floats.
template <typename T, int VE, int EPT>
struct RowPart {
    using V = Vec<T, VE>;
    static constexpr int CH = EPT / VE;
    typename V::Raw q[CH];

    __device__ __forceinline__ void load(const T* row, int sub, int lanes, int chunks, bool live) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = sub + c * lanes;
            q[c] = V::zero();
            if (live && i < chunks) q[c] = V::load_cs(row + i * VE);
        }
    }
    __device__ __forceinline__ void pairs(F2 (&f)[EPT / 2]) const {
        float e[EPT];
#pragma unroll
        for (int c = 0; c < CH; ++c) V::unpack(q[c], e + c * VE);
#pragma unroll
        for (int i = 0; i < EPT / 2; ++i) f[i] = F2(e[2 * i], e[2 * i + 1]);
    }
    static __device__ __forceinline__ void store(T* row, const F2 (&f)[EPT / 2], int sub, int lanes, int chunks) {
        float e[EPT];
#pragma unroll
        for (int i = 0; i < EPT / 2; ++i) {
            e[2 * i] = f[i].lo();
            e[2 * i + 1] = f[i].hi();
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = sub + c * lanes;
            if (i < chunks) V::store(row + i * VE, e + c * VE);
        }
    }
};

// Pairs of a thread's columns of a weight, `none` where there is no weight or no column.
template <typename W, int VE, int EPT>
__device__ __forceinline__ void column_weights(const W* w, float none, F2 (&f)[EPT / 2], int sub, int lanes,
                                               int chunks) {
    float e[EPT];
#pragma unroll
    for (int c = 0; c < EPT / VE; ++c) {
        const int i = sub + c * lanes;
#pragma unroll
        for (int k = 0; k < VE; ++k) e[c * VE + k] = none;
        if (w && i < chunks) ln_weights<W, VE>(w + i * VE, e + c * VE);
    }
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) f[i] = F2(e[2 * i], e[2 * i + 1]);
}

// One row per `lanes` lanes of a warp (WARP), or per block; a thread keeps EPT elements of it: the
// row is read once, and the mean and then the centred squares are summed from registers. Blocks
// stay and take every gridDim.x-th row; the next row's loads are issued before the current
// row's sums are reduced. HOLD: the thread's columns of weight and bias stay in registers too, else they
// are read from L1 for every row.
template <typename T, typename W, int VE, int EPT, bool WARP, bool HOLD>
__global__ void __launch_bounds__(WARP ? kLnThreads : 512)
ln_forward_kernel(const T* x, const T* res, const W* __restrict__ weight, const W* __restrict__ bias, T* y, T* sum_out,
                  float* __restrict__ mean, float* __restrict__ rstd, unsigned rows, int D, float eps, int lanes) {
    using Part = RowPart<T, VE, EPT>;
    __shared__ __align__(16) float sm[2][2][1][32];
    const int sub = WARP ? threadIdx.x & (lanes - 1) : threadIdx.x;
    const unsigned per_block = WARP ? kLnThreads / lanes : 1, mine = WARP ? threadIdx.x / lanes : 0;
    const unsigned step = gridDim.x * per_block;
    const int chunks = D / VE;
    const float inv = 1.f / (float)D;
    F2 w[EPT / 2], b[EPT / 2];
    if (HOLD) {
        column_weights<W, VE, EPT>(weight, 1.f, w, sub, lanes, chunks);
        column_weights<W, VE, EPT>(bias, 0.f, b, sub, lanes, chunks);
    }
    Part cur, cur_res;
    unsigned base = blockIdx.x * per_block;  // every thread of a block makes the same trips
    auto load = [&](Part& p, Part& pr, unsigned r) {
        p.load(x + (size_t)r * D, sub, lanes, chunks, r < rows);
        if (res) pr.load(res + (size_t)r * D, sub, lanes, chunks, r < rows);
    };
    load(cur, cur_res, base + mine);
    for (int flip = 0; base < rows; base += step, flip ^= 1) {
        const unsigned r = base + mine;
        F2 v[EPT / 2];
        cur.pairs(v);
        if (res) {
            F2 f[EPT / 2];
            cur_res.pairs(f);
#pragma unroll
            for (int i = 0; i < EPT / 2; ++i) v[i] = add2(v[i], f[i]);
        }
        load(cur, cur_res, r + step);
        F2 t = v[0];
#pragma unroll
        for (int i = 1; i < EPT / 2; ++i) t = add2(t, v[i]);
        float s[1] = {t.sum()};
        row_sums<WARP>(s, lanes, sm[flip][0]);
        const float mu = s[0] * inv;
        const F2 minus = F2(-mu, -mu);
        t = F2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < Part::CH; ++c) {
            if (sub + c * lanes < chunks) {
                if (VE == 1) {
                    const float z = (c & 1 ? v[c / 2].hi() : v[c / 2].lo()) - mu;
                    t = add2(t, F2(z * z, 0.f));
                } else {
#pragma unroll
                    for (int i = c * VE / 2; i < (c + 1) * VE / 2; ++i) {
                        const F2 z = add2(v[i], minus);
                        t = fma2(z, z, t);
                    }
                }
            }
        }
        s[0] = t.sum();
        row_sums<WARP>(s, lanes, sm[flip][1]);
        const float rs = rsqrtf(s[0] * inv + eps);
        if (r < rows) {
            const size_t at = (size_t)r * D;
            if (sum_out) Part::store(sum_out + at, v, sub, lanes, chunks);
            if (!HOLD) {
                column_weights<W, VE, EPT>(weight, 1.f, w, sub, lanes, chunks);
                column_weights<W, VE, EPT>(bias, 0.f, b, sub, lanes, chunks);
            }
            const F2 scale = F2(rs, rs);
#pragma unroll
            for (int i = 0; i < EPT / 2; ++i) v[i] = fma2(mul2(add2(v[i], minus), scale), w[i], b[i]);
            Part::store(y + at, v, sub, lanes, chunks);
            if (sub == 0) {
                if (mean) mean[r] = mu;
                if (rstd) rstd[r] = rs;
            }
        }
    }
}

// dx and the column sums in one pass: blocks stay, and a thread keeps the same EPT columns of
// every row it takes, their dw and db sums in registers. The next row's loads are issued before
// the current row's two sums are reduced. Each block ends with one row of partial sums, part
// [gridDim.x, 2, D]; ln_reduce_kernel adds those in block order.
template <typename T, typename W, int VE, int EPT, bool WARP>
__global__ void __launch_bounds__(WARP ? kLnThreads : 512)
ln_backward_kernel(const T* dy, const T* x, const W* __restrict__ weight, const float* __restrict__ mean,
                   const float* __restrict__ rstd, const T* dsum, T* dx, float* __restrict__ part, unsigned rows, int D,
                   int lanes) {
    using Part = RowPart<T, VE, EPT>;
    constexpr int P = EPT / 2;
    extern __shared__ float ln_sm[];  // WARP: [2, D] for joining the warps' column sums
    __shared__ __align__(16) float sm[2][2][32];
    const int sub = WARP ? threadIdx.x & (lanes - 1) : threadIdx.x;
    const unsigned per_block = WARP ? kLnThreads / lanes : 1, mine = WARP ? threadIdx.x / lanes : 0;
    const unsigned step = gridDim.x * per_block;
    const int chunks = D / VE;
    const float inv = 1.f / (float)D;
    F2 w[P], dw[P], db[P];
    column_weights<W, VE, EPT>(weight, 1.f, w, sub, lanes, chunks);
#pragma unroll
    for (int i = 0; i < P; ++i) dw[i] = db[i] = F2(0.f, 0.f);
    Part dyp, xp, sp;
    float mu, rs;
    auto load = [&](unsigned r) {
        const bool live = r < rows;
        mu = live ? mean[r] : 0.f;
        rs = live ? rstd[r] : 0.f;
        dyp.load(dy + (size_t)r * D, sub, lanes, chunks, live);
        xp.load(x + (size_t)r * D, sub, lanes, chunks, live);
        if (dsum) sp.load(dsum + (size_t)r * D, sub, lanes, chunks, live);
    };
    unsigned base = blockIdx.x * per_block;  // every thread of a block makes the same trips
    load(base + mine);
    for (int flip = 0; base < rows; base += step, flip ^= 1) {
        const unsigned r = base + mine;
        F2 u[P], xh[P], add[P];
        dyp.pairs(u);
        xp.pairs(xh);
        if (dsum) sp.pairs(add);
        const float scale = rs, shift = -mu * rs;
        load(r + step);
        // columns behind the row: dy is 0 there, so whatever xh holds (finite) adds nothing
        F2 s0 = F2(0.f, 0.f), s1 = s0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            xh[i] = fma2(xh[i], F2(scale, scale), F2(shift, shift));
            dw[i] = fma2(u[i], xh[i], dw[i]);
            db[i] = add2(db[i], u[i]);
            u[i] = mul2(u[i], w[i]);
            s0 = add2(s0, u[i]);
            s1 = fma2(u[i], xh[i], s1);
        }
        float s[2] = {s0.sum(), s1.sum()};
        row_sums<WARP>(s, lanes, sm[flip]);
        if (r < rows) {
            const float m0 = -scale * (s[0] * inv), m1 = -scale * (s[1] * inv);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                u[i] = fma2(xh[i], F2(m1, m1), fma2(u[i], F2(scale, scale), F2(m0, m0)));
                if (dsum) u[i] = add2(u[i], add[i]);
            }
            Part::store(dx + (size_t)r * D, u, sub, lanes, chunks);
        }
    }
    if (!part) return;
    float* out = part + (size_t)blockIdx.x * 2 * D;
    if (WARP) {  // the groups of a warp, then the warps one after another
        float* acc = ln_sm;
        for (int off = 16; off >= lanes; off >>= 1) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                F2 q;
                q.v = __shfl_xor_sync(0xffffffffu, dw[i].v, off);
                dw[i] = add2(dw[i], q);
                q.v = __shfl_xor_sync(0xffffffffu, db[i].v, off);
                db[i] = add2(db[i], q);
            }
        }
        for (int q = 0; q < kLnThreads / 32; ++q) {
            if ((int)(threadIdx.x >> 5) == q && (threadIdx.x & 31) < lanes) {
#pragma unroll
                for (int e = 0; e < EPT; ++e) {
                    const int i = (sub + e / VE * lanes) * VE + e % VE;
                    if (i >= D) continue;
                    const float a = e & 1 ? dw[e / 2].hi() : dw[e / 2].lo(), d = e & 1 ? db[e / 2].hi() : db[e / 2].lo();
                    acc[i] = q ? acc[i] + a : a;
                    acc[D + i] = q ? acc[D + i] + d : d;
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * D; c += kLnThreads) out[c] = acc[c];
    } else {
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            const int i = (sub + e / VE * lanes) * VE + e % VE;
            if (i >= D) continue;
            out[i] = e & 1 ? dw[e / 2].hi() : dw[e / 2].lo();
            out[D + i] = e & 1 ? db[e / 2].hi() : db[e / 2].lo();
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
