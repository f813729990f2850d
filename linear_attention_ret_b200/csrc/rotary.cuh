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

#include "vec.cuh"

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

// Vectors of VE elements. A thread owns one unit of every `split`-th head of a token's q or k: a
// unit is VE consecutive elements (VE / 2 pairs) in the interleaved layout, and in the half layout
// two vectors, those whose elements pair up or two neighbours behind the rotated part. With VE = 1
// (odd sizes and alignments) a unit is two elements in either layout. Threads of neighbouring
// units and heads lie side by side, so a warp reads whole stretches of a token-major row. A block
// holds `tokens` tokens of `split` head groups of q and of k each. With one or two heads
// (MANY) each has its thread, and the thread's rows are of BATCH tokens, `at_once` apart: BATCH rows
// are in flight either way, and what a block costs once is spread over as many.
// cos and sin of a token are formed once per block, in shared memory, and serve all heads of q and
// k; a thread's first BATCH rows are in flight meanwhile. HBM-bound; index arithmetic is once per
// thread, as divisions per vector bound the kernel by instruction issue (1.3B-shaped, 134 MB:
// 40.6 us, now 23.0 us, 5.8 TB/s; batches of two rows 25.9 us).
struct RotPlan {
    FastDiv units, split, N;  // units of a head; head groups of a token's q (or k); tokens of a batch
    int tensors;              // 2: q and k, 1: q alone
    int tokens, at_once;      // of a block; neighbouring threads' tokens
    int half_units;           // half layout, or VE = 1: units that are rotated
    int apart;                // and elements from the first of a pair to the second
    int stride;               // of a token's cos (or sin) in shared memory, in floats
};

template <typename T, int VE, bool HALF, int BATCH>
struct RotUnit {
    using V = Vec<T, VE>;
    static constexpr int P = HALF ? VE : VE / 2;  // frequencies of a unit
    typename V::Raw lo[BATCH], hi[HALF ? BATCH : 1];

    // row i at x; the second vector `second` elements on (half layout, 0: there is none)
    __device__ __forceinline__ void load(int i, const T* x, int second) {
        lo[i] = V::load_cs(x);
        if (HALF && second) hi[HALF ? i : 0] = V::load_cs(x + second);
    }

    // live: how many of the unit's frequencies are rotated; c and s carry the scale m. Elements
    // that are not rotated are selected, not multiplied by 0: a neighbour may be infinite.
    __device__ __forceinline__ void turn_store(int i, T* y, int second, int live, const float (&c)[P],
                                               const float (&s)[P], float m) {
        float f[VE];
        V::unpack(lo[i], f);
        if (HALF) {
            float g[VE];
            V::unpack(hi[HALF ? i : 0], g);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float p = f[e], q = g[e];
                f[e] = live ? p * c[e % P] - q * s[e % P] : p * m;
                g[e] = live ? p * s[e % P] + q * c[e % P] : q * m;
            }
            if (second) V::store(y + second, g);
        } else {
#pragma unroll
            for (int e = 0; e < VE / 2; ++e) {
                const float p = f[2 * e], q = f[2 * e + 1];
                f[2 * e] = e < live ? p * c[e % P] - q * s[e % P] : p * m;
                f[2 * e + 1] = e < live ? p * s[e % P] + q * c[e % P] : q * m;
            }
        }
        V::store(y, f);
    }
};

// The half layout of bf16 takes vectors of 8 bytes, two per unit: units of 16 bytes need twice the
// registers and leave three blocks on an SM instead of four (134 MB, 4 heads of 128: 26.9 us against
// 25.9 us), and with eight heads or more a thread takes eight rows at once (gradient at the gated
// layer's shapes, 268 MB: 47.0 us with four, 44.6 us with eight, 6.0 TB/s; the interleaved layout gains nothing).
// fp32 keeps 16-byte vectors in both layouts: 268 MB, 4 heads of 128 42.5 us interleaved (6.3 TB/s) and
// 44.2 us half (6.1 TB/s), although the half layout's four rows of two vectors spill 48 bytes at 64 registers.
template <typename T, int VE, bool HALF, int BATCH, bool MANY>
__global__ void __launch_bounds__(kRotThreads, BATCH > 4 ? 3 : 4) rotary_vec_kernel(const RotArgs a, const RotPlan pl) {
    using Unit = RotUnit<T, VE, HALF, BATCH>;
    constexpr int P = Unit::P;
    extern __shared__ float4 rot_sm[];
    float* cs = reinterpret_cast<float*>(rot_sm);
    float* sn = cs + pl.tokens * pl.stride;
    const unsigned all = (unsigned)a.B * a.N, first = blockIdx.x * (unsigned)pl.tokens;  // below 2^31
    const int tokens = (int)min((unsigned)pl.tokens, all - first), half = a.rot / 2;
    unsigned group, u, t, g, b, n;
    pl.units.divmod(threadIdx.x, group, u);
    pl.split.divmod(group, t, g);
    const bool second = pl.tensors == 2 && (t & 1);
    if (pl.tensors == 2) t >>= 1;
    const RotView& v = a.x[second];
    const int split = (int)pl.split.d, H = v.H;
    const bool pair = HALF && (int)u < pl.half_units;
    // pairs next to each other lie like what is behind the rotated part: VE = 1, interleaved
    const int at = !HALF || (pair && pl.apart != 1) ? (int)u * VE
                                                    : (pair ? 0 : a.rot - 2 * VE * pl.half_units) + (int)u * 2 * VE;
    const int second_at = !HALF ? 0 : pair ? pl.apart : at + VE < a.d ? VE : 0;
    const int live = HALF ? (pair ? P : 0) : min(max(half - (int)u * P, 0), P);
    const long long si = split * v.ih, so = split * v.oh;
    const float m = v.scale;
    // threads behind the last group have no rows; t: MANY the first of the thread's tokens, else its only one
    const bool on = (int)t < (MANY ? pl.at_once : tokens) && (!MANY || (int)g < H);
    auto in_row = [&](unsigned token) {
        pl.N.divmod(first + token, b, n);
        return static_cast<const T*>(v.in) + b * v.ib + n * v.in_ + g * v.ih + at;
    };
    auto out_row = [&](unsigned token) {
        pl.N.divmod(first + token, b, n);
        return static_cast<T*>(v.out) + b * v.ob + n * v.on + g * v.oh + at;
    };
    const T* x = in_row(t);
    T* y = out_row(t);
    wait_previous_kernel();
    Unit r;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
        if (MANY) {
            if (on && (int)t + i * pl.at_once < tokens) r.load(i, in_row(t + i * pl.at_once), second_at);
        } else if (on && (int)g + i * split < H) {
            r.load(i, x + i * si, second_at);
        }
    }
    for (int j = threadIdx.x; j < tokens * half; j += kRotThreads) {
        const int tj = j / half, f = j - tj * half;
        unsigned bj, nj;
        pl.N.divmod(first + tj, bj, nj);
        rot_angle(a, rot_position(a, (int)bj, (int)nj), f, cs[tj * pl.stride + f], sn[tj * pl.stride + f]);
    }
    __syncthreads();
    if (!on) return;
    float c[P], s[P];
    auto angles = [&](unsigned token) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
            c[e] = e < live ? m * cs[token * pl.stride + u * P + e] : 0.f;
            s[e] = e < live ? m * sn[token * pl.stride + u * P + e] : 0.f;
        }
    };
    if (MANY) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const unsigned token = t + i * pl.at_once;
            if ((int)token >= tokens) break;
            angles(token);
            r.turn_store(i, out_row(token), second_at, live, c, s, m);
        }
        return;
    }
    angles(t);
    for (int h = (int)g;;) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (h + i * split < H) r.turn_store(i, y + i * so, second_at, live, c, s, m);
        }
        h += BATCH * split;
        if (h >= H) break;
        x += BATCH * si;
        y += BATCH * so;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (h + i * split < H) r.load(i, x + i * si, second_at);
        }
    }
}

// Any width and alignment. One thread per pair, or element behind the rotated part, of q and k. An
// ordinary launch: it has no wait for the kernel before it.
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
