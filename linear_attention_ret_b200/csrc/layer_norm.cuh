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

#include <cfloat>
#include <cooperative_groups.h>
#include <type_traits>

#include "vec.cuh"

namespace ret {

constexpr int kLnThreads = 256;
constexpr int kLnMaxShared = 220 * 1024;  // of a block: what its rows in flight may take

// VE weights as floats (vector path: the pointer is aligned to the vector, at most 16 bytes).
template <typename W, int VE>
__device__ __forceinline__ void ln_weights(const W* w, float* f) {
    constexpr int kPart = VE * (int)sizeof(W) <= 16 ? VE : 16 / (int)sizeof(W);
#pragma unroll
    for (int e = 0; e < VE; e += kPart) Vec<W, kPart>::unpack(Vec<W, kPart>::load(w + e), f + e);
}

// A row's threads: `lanes` lanes of a warp (WARP; a power of two), or `lanes` / 32 whole warps, up
// to 16; a block holds `groups` of them, each with a row of its own. row_sum adds a value over a
// row's threads, row_sums two at once; every thread gets the sums. Whole warps meet at a barrier
// and take `sm`, one float per warp and value, zero behind the row's warps and not written again
// before the next barrier. PAIR: the row's threads are two blocks of a cluster; each warp's sums go
// to both blocks' sm, and the cluster's barrier takes the place of the block's.
// row_sum is for blocks of one group. row_sums' groups meet at barriers of their own (number
// group + 1); a kernel with numbered barriers holds 16 of an SM's for each block, too many where
// blocks are small (8192 x 1024 forward: 24.5 us against 13.6 us).
struct RowThreads {
    int sub, lanes, group, groups;
    __device__ __forceinline__ void meet() const {
        if (groups == 1) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");
    }
};
constexpr int kLnWarps = 16;   // most warps of a row
constexpr int kLnGroups = 8;   // most groups of whole warps in a block
using RowShared = float[2][kLnWarps];

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int off = lanes >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int off = LANES >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

template <bool WARP, bool PAIR>
__device__ __forceinline__ float row_sum(float v, const RowThreads& t, RowShared& sm) {
    if (WARP) return lanes_sum(v, t.lanes);
    v = lanes_sum<32>(v);
    const int lane = threadIdx.x & 31, place = lane & (kLnWarps - 1);
    if (PAIR) {
        const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        if (lane == 0) {
            float* mine = &sm[cluster.block_rank()][t.sub >> 5];
            *mine = v;
            *cluster.map_shared_rank(mine, cluster.block_rank() ^ 1) = v;
        }
        cluster.sync();
        return lanes_sum<kLnWarps>(sm[0][place] + sm[1][place]);
    }
    if (lane == 0) sm[0][t.sub >> 5] = v;
    __syncthreads();
    return lanes_sum<kLnWarps>(sm[0][place]);
}

// Two sums for little more than the shuffles of one: after the first exchange the lower half of
// a warp carries a and the upper half b.
template <bool WARP, bool PAIR>
__device__ __forceinline__ void row_sums(float& a, float& b, const RowThreads& t, RowShared (&sm)[PAIR ? 2 : 1]) {
    if (WARP && t.lanes < 32) {
        a = lanes_sum(a, t.lanes);
        b = lanes_sum(b, t.lanes);
        return;
    }
    const int lane = threadIdx.x & 31;
    const bool upper = lane >= 16;
    float v = upper ? b : a;
    v += __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
    v = lanes_sum<16>(v);
    if (!WARP) {
        const int warp = t.sub >> 5, place = lane & (kLnWarps - 1);
        if (PAIR) {
            const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
            if ((lane & 15) == 0) {
                float* mine = &sm[cluster.block_rank()][upper][warp];
                *mine = v;
                *cluster.map_shared_rank(mine, cluster.block_rank() ^ 1) = v;
            }
            cluster.sync();
            v = sm[0][upper][place] + sm[PAIR][upper][place];
        } else {
            if ((lane & 15) == 0) sm[0][upper][warp] = v;
            t.meet();
            v = sm[0][upper][place];
        }
        v = lanes_sum<kLnWarps>(v);
    }
    const float other = __shfl_xor_sync(0xffffffffu, v, 16);
    a = upper ? other : v;
    b = upper ? v : other;
}

__device__ __forceinline__ RowThreads row_threads(int lanes) {
    RowThreads t;
    t.lanes = lanes;
    t.groups = blockDim.x / lanes;
    t.group = t.groups == 1 ? 0 : threadIdx.x / lanes;
    t.sub = threadIdx.x - t.group * lanes;
    return t;
}

// A thread's EPT elements of a row: CH vectors of VE elements, 32 vectors apart, the first of them
// number row_first. A warp's vectors lie together, so the distances are known when the kernel is
// compiled (fewer than 32 lanes of a warp hold at most one vector each).
template <int CH>
__device__ __forceinline__ int row_first(const RowThreads& t) {
    return (t.sub >> 5) * 32 * CH + (t.sub & 31);
}

template <typename T, int VE, int EPT>
struct RowPart {
    using V = Vec<T, VE>;
    using Raw = typename V::Raw;
    static constexpr int CH = EPT / VE;

    static __device__ __forceinline__ void pairs(const Raw (&q)[CH], F2 (&f)[EPT / 2]) {
        float e[EPT];
#pragma unroll
        for (int c = 0; c < CH; ++c) V::unpack(q[c], e + c * VE);
#pragma unroll
        for (int i = 0; i < EPT / 2; ++i) f[i] = F2(e[2 * i], e[2 * i + 1]);
    }
};

// The rows that a thread works through: `row`, row + step, ... below `rows`, kAhead of them in
// flight. Each thread copies its own parts of N tensors' rows into slots of shared memory that no
// other thread reads, so it waits for its own copies alone, and registers hold no row in flight but
// its N_STAT statistics, loaded two rows ahead. 2-byte accesses have no asynchronous copy: those
// wait in registers, one row ahead. Vectors behind the row read as zero; rows behind the last one
// are not copied, and taking one gives whatever an earlier row left.
template <typename T, int VE, int EPT, int N, int N_STAT>
struct RowStream {
    using Part = RowPart<T, VE, EPT>;
    using Raw = typename Part::Raw;
    static constexpr int CH = Part::CH;
    static constexpr bool kAsync = sizeof(Raw) >= 4;
    // rows in slots: four of up to 64 bytes per thread, three of up to 128, two of more
    static constexpr int kRowBytes = N * CH * (int)sizeof(Raw);
    static constexpr int kSlots = !kAsync ? 0 : kRowBytes <= 64 ? 4 : kRowBytes <= 128 ? 3 : 2;
    static constexpr int kAhead = kAsync ? kSlots - 1 : 1;
    // [slot][tensor][vector][thread]: neighbouring threads' copies lie side by side. A thread's own
    // slots side by side, threads an odd number of 16-byte units apart, met no bank twice either but
    // was a third slower (fp32 8192 x 2048 forward 32.4 us against 24.3 us).
    static constexpr size_t bytes(int threads) { return (size_t)kSlots * threads * kRowBytes; }

    const T* src[N];  // of this thread's first vector of the next row to copy
    const float* stat[N_STAT > 0 ? N_STAT : 1];
    unsigned next, step, rows;            // the next row to copy
    long long stride;                     // elements from a row to the next of this thread
    static constexpr int kGap = 32 * VE;  // elements from a vector to the next of this thread
    bool has[CH];
    unsigned char* slots;  // this thread's place in slot 0
    int put, get;          // the slot to fill and the slot to read next
    int pitch;             // bytes from a vector to the thread's next
    Raw held[kAsync ? 1 : N][CH];
    float stats[2][N_STAT > 0 ? N_STAT : 1];  // of the current row and the next
    unsigned next_stat;

    __device__ __forceinline__ Raw* at(int slot, int t, int c) const {
        return reinterpret_cast<Raw*>(slots + (slot * N * CH + t * CH + c) * pitch);
    }

    __device__ __forceinline__ void issue() {
        if (next < rows) {
#pragma unroll
            for (int t = 0; t < N; ++t) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    if (!has[c]) continue;
                    if (kAsync) copy_async<kAsync ? (int)sizeof(Raw) : 4>(at(put, t, c), src[t] + c * kGap);
                    else held[kAsync ? 0 : t][c] = Part::V::load_cs(src[t] + c * kGap);
                }
                src[t] += stride;
            }
            next += step;
        }
        if (kAsync) {
            copy_commit();
            put = put == kSlots - 1 ? 0 : put + 1;
        }
    }
    __device__ __forceinline__ void load_stats(float (&s)[N_STAT > 0 ? N_STAT : 1]) {
#pragma unroll
        for (int k = 0; k < N_STAT; ++k) s[k] = next_stat < rows ? stat[k][next_stat] : 0.f;
        next_stat += step;
    }
    // src and stat are set; issues the first kAhead rows. The stream is of the first `width` of
    // rows of D elements.
    __device__ __forceinline__ void start(void* smem, const RowThreads& t, unsigned row, unsigned step_, unsigned rows_,
                                          int D, int width, int) {
        const int chunks = width / VE;
        next = row;
        step = step_;
        rows = rows_;
        stride = (long long)step * D;
        const int first = row_first<CH>(t);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            src[k] += row < rows ? (size_t)row * D + first * VE : 0;
        }
        pitch = blockDim.x * (int)sizeof(Raw);
        slots = static_cast<unsigned char*>(smem) + threadIdx.x * sizeof(Raw);
        next_stat = row;
#pragma unroll
        for (int k = 0; k < 2; ++k) load_stats(stats[k]);
        put = get = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            has[c] = first + c * 32 < chunks;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if (!kAsync) held[kAsync ? 0 : k][c] = Part::V::zero();
                else if (!has[c])
                    for (int q = 0; q < kSlots; ++q) *at(q, k, c) = Part::V::zero();
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) issue();
    }
    // the current row's parts; then the row that its slot's turn comes to is issued
    __device__ __forceinline__ void take(F2 (&f)[N][EPT / 2], float (&s)[N_STAT > 0 ? N_STAT : 1]) {
        if (N_STAT > 0) {
#pragma unroll
            for (int k = 0; k < N_STAT; ++k) {
                s[k] = stats[0][k];
                stats[0][k] = stats[1][k];
            }
            load_stats(stats[1]);
        }
        if (kAsync) copy_wait<kAhead - 1>();
#pragma unroll
        for (int t = 0; t < N; ++t) {
            Raw q[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) q[c] = kAsync ? *at(get, t, c) : held[kAsync ? 0 : t][c];
            Part::pairs(q, f[t]);
        }
        if (kAsync) {
            get = get == kSlots - 1 ? 0 : get + 1;
        }
        issue();
    }
    static constexpr bool full = false;
    __device__ __forceinline__ bool in_row(int e) const { return has[e / VE]; }  // this thread's element e
    __device__ __forceinline__ void store(T* row, const F2 (&f)[EPT / 2]) const {  // row: this thread's first vector
        float e[EPT];
#pragma unroll
        for (int i = 0; i < EPT / 2; ++i) {
            e[2 * i] = f[i].lo();
            e[2 * i + 1] = f[i].hi();
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (has[c]) Part::V::store(row + c * kGap, e + c * VE);
        }
    }
};

// The same for single elements (VE = 1): a warp copies the 16-byte units that cover its stretch of 32
// EPT elements, and its threads then read single elements of them, neighbouring lanes neighbouring
// elements. Copies are wide and asynchronous whatever a row starts on; a unit that reaches over
// either end of the tensor is filled element by element. Units hold neighbours' elements too, which
// an in-place call may be writing: they are copied and never looked at.
template <typename T, int EPT, int N, int N_STAT>
struct RowSpan {
    static constexpr bool kAsync = true;
    static constexpr int E = 16 / (int)sizeof(T);  // elements of a unit
    static constexpr int kRowBytes = N * EPT * (int)sizeof(T);
    static constexpr int kSlots = kRowBytes <= 64 ? 4 : kRowBytes <= 128 ? 3 : 2;
    static constexpr int kAhead = kSlots - 1;
    static constexpr int kUnits = 32 * EPT / E + 1;  // most units that a warp's stretch touches
    static constexpr size_t bytes(int threads) { return (size_t)kSlots * N * (threads / 32) * kUnits * 16; }

    const T* src[N];  // of this warp's first element of the next row to copy (start: of the tensors)
    const float* stat[N_STAT > 0 ? N_STAT : 1];
    unsigned next, step, rows;  // the next row to copy
    long long stride;           // elements from a row to the next of this warp
    int left;                   // this thread's element c is in the row where 32 c < left
    bool full;                  // all of the warp's elements are (asked first: one test for sixteen)
    const T *begin[N], *end[N];  // of the tensors
    T* slots;                    // this warp's place in slot 0
    int put, get;                // the slot to fill and the slot to read next
    int pitch;                   // elements from a slot's tensor to the next
    int count;                   // elements of this warp's stretch
    int skip[N];                 // elements before the current row's first in its first unit
    float stats[2][N_STAT > 0 ? N_STAT : 1];  // of the current row and the next
    unsigned next_stat;

    static __device__ __forceinline__ int off_unit(const T* p) {
        return (int)(reinterpret_cast<uintptr_t>(p) / sizeof(T)) & (E - 1);
    }
    __device__ __forceinline__ void issue() {
        if (next < rows) {
            const int lane = threadIdx.x & 31;
            // rows whose units may reach over an end (they may be shorter than a unit)
            const bool edge = next < (unsigned)E || next + E >= rows;
#pragma unroll
            for (int t = 0; t < N; ++t) {
                const int off = off_unit(src[t]), units = count > 0 ? (off + count + E - 1) / E : 0;
                const T* from = src[t] - off;
                T* to = slots + (put * N + t) * pitch;
#pragma unroll
                for (int j = 0; j < (kUnits + 31) / 32; ++j) {
                    const int u = j * 32 + lane;
                    if (u >= units) continue;
                    const T* p = from + u * E;
                    if (edge && (p < begin[t] || p + E > end[t])) {
                        for (int e = 0; e < E; ++e)
                            if (p + e >= begin[t] && p + e < end[t]) to[u * E + e] = p[e];
                    } else {
                        copy_async<16>(to + u * E, p);
                    }
                }
                src[t] += stride;
            }
            next += step;
        }
        copy_commit();
        put = put == kSlots - 1 ? 0 : put + 1;
    }
    __device__ __forceinline__ void load_stats(float (&s)[N_STAT > 0 ? N_STAT : 1]) {
#pragma unroll
        for (int k = 0; k < N_STAT; ++k) s[k] = next_stat < rows ? stat[k][next_stat] : 0.f;
        next_stat += step;
    }
    // tensors: src as given, rows_ rows of D elements from `before` elements before src on
    __device__ __forceinline__ void start(void* smem, const RowThreads& t, unsigned row, unsigned step_, unsigned rows_,
                                          int D, int width, int before) {
        next = row;
        step = step_;
        rows = rows_;
        stride = (long long)step * D;
        const int first = (t.sub >> 5) * 32 * EPT;
        count = min(32 * EPT, width - first);
        pitch = (blockDim.x / 32) * kUnits * E;
        slots = static_cast<T*>(smem) + (threadIdx.x >> 5) * kUnits * E;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            begin[k] = src[k] - before;
            end[k] = begin[k] + (size_t)rows * D;
            src[k] += row < rows ? (size_t)row * D + first : 0;
            skip[k] = off_unit(src[k]);
        }
        next_stat = row;
#pragma unroll
        for (int k = 0; k < 2; ++k) load_stats(stats[k]);
        put = get = 0;
        left = count - (t.sub & 31);
        full = count == 32 * EPT;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) issue();
    }
    __device__ __forceinline__ void take(F2 (&f)[N][EPT / 2], float (&s)[N_STAT > 0 ? N_STAT : 1]) {
        if (N_STAT > 0) {
#pragma unroll
            for (int k = 0; k < N_STAT; ++k) {
                s[k] = stats[0][k];
                stats[0][k] = stats[1][k];
            }
            load_stats(stats[1]);
        }
        copy_wait<kAhead - 1>();
        __syncwarp();  // every lane's copies have landed, and every lane has read the slot that is filled next
#pragma unroll
        for (int t = 0; t < N; ++t) {
            const T* from = slots + (get * N + t) * pitch + skip[t] + (threadIdx.x & 31);
            float e[EPT];
            if (full) {
#pragma unroll
                for (int c = 0; c < EPT; ++c) e[c] = ld_elem(from + c * 32);
            } else {
#pragma unroll
                for (int c = 0; c < EPT; ++c) e[c] = 32 * c < left ? ld_elem(from + c * 32) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < EPT / 2; ++i) f[t][i] = F2(e[2 * i], e[2 * i + 1]);
            skip[t] = (skip[t] + (int)(stride & (E - 1))) & (E - 1);
        }
        get = get == kSlots - 1 ? 0 : get + 1;
        issue();
    }
    __device__ __forceinline__ bool in_row(int e) const { return 32 * e < left; }
    __device__ __forceinline__ void store(T* row, const F2 (&f)[EPT / 2]) const {  // row: this thread's first element
        if (full) {
#pragma unroll
            for (int c = 0; c < EPT; ++c) st_elem(row + c * 32, c & 1 ? f[c / 2].hi() : f[c / 2].lo());
        } else {
#pragma unroll
            for (int c = 0; c < EPT; ++c)
                if (32 * c < left) st_elem(row + c * 32, c & 1 ? f[c / 2].hi() : f[c / 2].lo());
        }
    }
};

// Single elements are read through spans where that was faster: the forward of fp32 (9189 x 1023 with a
// residual: 27.5 us against 32.2 us), the backward of fp32 with three tensors (16400 x 1023: 51.2 us
// against 61.9 us; with two 55.7 us against 51.2 us) and, of either type, the backward's rows above 4,096
// elements (2048 x 8191 in bf16: 38.9 us against 62.7 us). Elsewhere bf16 waits in registers (forward of
// 16400 x 1023 26.8 us against 30.8 us, of 2048 x 8191 30.6 against 32.7 and of 1365 x 12289 53.9 against
// 62.9, with a residual 34.2 against 34.6, 43.6 against 41.7 and 73.9 against 106; backward of 16400 x 1023
// 33.4 us against 55.5 us). The backward's widest form by spans with three tensors spills 80 to 104 bytes.
template <typename T, int VE, int EPT, int N, int N_STAT>
constexpr bool by_span() {
    if (VE > 1) return false;
    return N_STAT == 0 ? sizeof(T) == 4 : EPT > 8 || (sizeof(T) == 4 && N == 3);
}
template <typename T, int VE, int EPT, int N, int N_STAT>
using Rows = std::conditional_t<by_span<T, VE, EPT, N, N_STAT>(), RowSpan<T, EPT, N, N_STAT>,
                                RowStream<T, VE, EPT, N, N_STAT>>;

// Pairs of a thread's columns of a weight, `none` where there is no weight or no column.
template <typename W, int VE, int EPT>
__device__ __forceinline__ void column_weights(const W* w, float none, F2 (&f)[EPT / 2], const RowThreads& t,
                                               int chunks) {
    float e[EPT];
#pragma unroll
    for (int c = 0; c < EPT / VE; ++c) {
        const int i = row_first<EPT / VE>(t) + c * 32;
#pragma unroll
        for (int k = 0; k < VE; ++k) e[c * VE + k] = none;
        if (w && i < chunks) ln_weights<W, VE>(w + i * VE, e + c * VE);
    }
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) f[i] = F2(e[2 * i], e[2 * i + 1]);
}

// One row per `lanes` lanes of a warp (WARP), per block, or per pair of blocks of a cluster (PAIR,
// each block with its columns); a thread keeps EPT elements of it: the row is read once, and the
// mean and then the centred squares are summed from registers. Blocks stay and take every
// gridDim.x-th row, with the next rows in flight and (EPT up to 16) their columns of weight and bias
// in registers. HBM-bound at large sizes: 8192 x 2048 in bf16 (67 MB) 13.6 us, 4.9 TB/s; one row
// per block and unpacked arithmetic took 23.9 us, two thirds of it instruction issue.
// Above 8,192 elements a block of 512 threads takes EPT = 32 (1024 x 16384 in bf16: 20 us; a pair of
// blocks, which meet twice a row, 35 us), or a pair does where the rows of EPT = 32 do not fit shared
// memory (fp32 with a residual).
template <typename T, typename W, int VE, int EPT, bool WARP, bool RES, bool PAIR>
__global__ void __launch_bounds__(WARP ? kLnThreads : 512)
ln_forward_kernel(const T* x, const T* res, const W* weight, const W* bias, T* y, T* sum_out, float* mean, float* rstd,
                  unsigned rows, int D, float eps, int lanes) {
    extern __shared__ uint4 ln_ring[];
    __shared__ RowShared sm[2][2];  // one group of whole warps
    const RowThreads t = row_threads(lanes);
    const unsigned blocks = PAIR ? gridDim.x / 2 : gridDim.x, block = PAIR ? blockIdx.x / 2 : blockIdx.x;
    const unsigned per_block = t.groups, mine = t.group, step = blocks * per_block;
    const float inv = 1.f / (float)D;
    // this block's columns
    const int half = (D / VE + 1) / 2 * VE, left = PAIR ? (int)(blockIdx.x & 1) * half : 0;
    const int width = !PAIR ? D : left ? D - half : half;
    if (!WARP) {
        for (int i = t.sub; i < 4 * 2 * kLnWarps; i += lanes) (&sm[0][0][0][0])[i] = 0.f;
    }
    wait_previous_kernel();
    unsigned base = block * per_block;  // every group of a block makes the same trips
    Rows<T, VE, EPT, RES ? 2 : 1, 0> in;
    in.src[0] = x + left;
    if (RES) in.src[RES] = res + left;
    in.start(ln_ring, t, base + mine, step, rows, D, width, left);
    size_t at = (size_t)(base + mine) * D + left + row_first<EPT / VE>(t) * VE;
    F2 w[EPT / 2], b[EPT / 2];
    auto columns = [&] {
        column_weights<W, VE, EPT>(weight ? weight + left : weight, 1.f, w, t, width / VE);
        column_weights<W, VE, EPT>(bias ? bias + left : bias, 0.f, b, t, width / VE);
    };
    if (EPT <= 16) columns();
    if (PAIR) cooperative_groups::this_cluster().sync();
    else if (!WARP) __syncthreads();
    for (int flip = 0; base < rows; base += step, at += in.stride, flip ^= 1) {
        const unsigned r = base + mine;
        F2 f[RES ? 2 : 1][EPT / 2];
        float none[1];
        in.take(f, none);
        F2(&v)[EPT / 2] = f[0];
        if (RES) {
#pragma unroll
            for (int i = 0; i < EPT / 2; ++i) v[i] = add2(v[i], f[RES][i]);
        }
        F2 q = v[0];
#pragma unroll
        for (int i = 1; i < EPT / 2; ++i) q = add2(q, v[i]);
        const float mu = row_sum<WARP, PAIR>(q.sum(), t, sm[flip][0]) * inv;
        const F2 minus = F2(-mu, -mu);
        if (RES && sum_out && r < rows) in.store(sum_out + at, v);
        q = F2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < EPT / 2; ++i) {  // elements behind the row stay out of the sum of centred squares
            v[i] = add2(v[i], minus);
            if (VE > 1 || in.full) {
                if (in.full || in.in_row(2 * i)) q = fma2(v[i], v[i], q);
            } else {
                const F2 z = F2(in.in_row(2 * i) ? v[i].lo() : 0.f, in.in_row(2 * i + 1) ? v[i].hi() : 0.f);
                q = fma2(z, z, q);
            }
        }
        const float rs = rsqrtf(row_sum<WARP, PAIR>(q.sum(), t, sm[flip][1]) * inv + eps);
        if (r < rows) {
            if (EPT > 16) columns();
            const F2 scale = F2(rs, rs);
#pragma unroll
            for (int i = 0; i < EPT / 2; ++i) v[i] = fma2(mul2(v[i], scale), w[i], b[i]);
            in.store(y + at, v);
            if (t.sub == 0 && left == 0) {
                if (mean) mean[r] = mu;
                if (rstd) rstd[r] = rs;
            }
        }
    }
    if (PAIR) cooperative_groups::this_cluster().sync();  // the other block may still write its sums here
}

// Floats of one row of column sums: a multiple of four, so that rows start on 16 bytes.
__host__ __device__ constexpr int ln_pitch(int D) { return (D + 3) / 4 * 4; }

// dx and the column sums in one pass: blocks stay, and a thread keeps the same EPT columns of
// every row it takes, their dw and db sums in registers; the next rows are in flight. Groups of
// whole warps share a block of 512 threads, one row each, and join their column sums at the end:
// each block leaves one row of partial sums, part [blocks, 2, ln_pitch(D)], which ln_reduce_kernel
// adds in order. HBM-bound: 8192 x 4096 in bf16 with the sum's gradient (269 MB) 48.9 us with the
// reduction, 5.5 TB/s; dx and the column sums in a pass each took 228 us. Joining partial sums over
// clusters instead was slower (8192 x 2048: 38.4 us against 27.7 us).
// PAIR: rows too wide for the registers of one block are split over the two blocks of a cluster, each
// with its columns (1024 x 16384 in bf16, 100 MB: 39 us, bound by the cluster's barrier in every
// row; 95 us with a second pass for the column sums).
template <typename T, typename W, int VE, int EPT, bool WARP, bool SUM, bool PAIR>
__global__ void __launch_bounds__(WARP ? kLnThreads : 512)
ln_backward_kernel(const T* dy, const T* x, const W* weight, const float* mean, const float* rstd, const T* dsum, T* dx,
                   float* part, unsigned rows, int D, int lanes) {
    constexpr int P = EPT / 2;
    extern __shared__ uint4 ln_ring[];  // rows in flight, and at the end column sums
    __shared__ RowShared sm_all[WARP || PAIR ? 1 : kLnGroups][2][PAIR ? 2 : 1];
    const RowThreads t = row_threads(lanes);
    RowShared(&sm)[2][PAIR ? 2 : 1] = sm_all[WARP || PAIR ? 0 : t.group];
    const unsigned blocks = PAIR ? gridDim.x / 2 : gridDim.x, block = PAIR ? blockIdx.x / 2 : blockIdx.x;
    const unsigned per_block = t.groups, mine = t.group, step = blocks * per_block;
    const float inv = 1.f / (float)D;
    // this block's columns
    const int half = (D / VE + 1) / 2 * VE, left = PAIR ? (int)(blockIdx.x & 1) * half : 0;
    const int width = !PAIR ? D : left ? D - half : half;
    if (!WARP) {
        for (int i = t.sub; i < (PAIR ? 4 : 2) * 2 * kLnWarps; i += lanes) (&sm[0][0][0][0])[i] = 0.f;
    }
    allow_next_kernel();
    wait_previous_kernel();
    unsigned base = block * per_block;  // every group of a block makes the same trips
    Rows<T, VE, EPT, SUM ? 3 : 2, 2> in;
    in.src[0] = dy + left;
    in.src[1] = x + left;
    if (SUM) in.src[SUM ? 2 : 0] = dsum + left;
    in.stat[0] = mean;
    in.stat[1] = rstd;
    in.start(ln_ring, t, base + mine, step, rows, D, width, left);
    size_t at = (size_t)(base + mine) * D + left + row_first<EPT / VE>(t) * VE;
    F2 w[P], dw[P], db[P];
    column_weights<W, VE, EPT>(weight ? weight + left : weight, 1.f, w, t, width / VE);
#pragma unroll
    for (int i = 0; i < P; ++i) dw[i] = db[i] = F2(0.f, 0.f);
    if (PAIR) cooperative_groups::this_cluster().sync();
    else if (!WARP) __syncthreads();
    for (int flip = 0; base < rows; base += step, at += in.stride, flip ^= 1) {
        const unsigned r = base + mine;
        F2 f[SUM ? 3 : 2][P];
        float st[2];
        in.take(f, st);
        F2(&u)[P] = f[0];
        F2(&xh)[P] = f[1];
        // Centred before it is scaled: x - mean is exact where they are close, so a mean far from zero
        // costs no digits. Columns behind the row: x and dy read as 0 there, so what xh holds adds nothing
        // as long as it is finite. (0 - mean) rstd is not where the product overflows; the elements of a
        // row with such statistics are all its mean (the next fp32 value would be 10^31 deviations away),
        // so there xh is 0 throughout.
        const float scale = st[1], minus = -st[0];
        const float scale_x = fabsf(minus * scale) <= FLT_MAX ? scale : 0.f;
        F2 s0 = F2(0.f, 0.f), s1 = s0;
        if (r < rows) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                xh[i] = mul2(add2(xh[i], F2(minus, minus)), F2(scale_x, scale_x));
                dw[i] = fma2(u[i], xh[i], dw[i]);
                db[i] = add2(db[i], u[i]);
                u[i] = mul2(u[i], w[i]);
                s0 = add2(s0, u[i]);
                s1 = fma2(u[i], xh[i], s1);
            }
        }
        float a = s0.sum(), c = s1.sum();
        row_sums<WARP, PAIR>(a, c, t, sm[flip]);
        if (r < rows) {
            const float m0 = -scale * (a * inv), m1 = -scale * (c * inv);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                u[i] = fma2(xh[i], F2(m1, m1), fma2(u[i], F2(scale, scale), F2(m0, m0)));
                if (SUM) u[i] = add2(u[i], f[SUM ? 2 : 0][i]);
            }
            in.store(dx + at, u);
        }
    }
    if (PAIR) cooperative_groups::this_cluster().sync();  // the other block may still write its sums here
    if (!part) return;
    // column sums to shared memory, [2, Dp]: the groups of a warp (WARP) joined first, then one warp
    // or group after another
    __syncthreads();  // no copy is in flight: every row that was issued has been taken
    float* acc = reinterpret_cast<float*>(ln_ring);
    const int Dp = ln_pitch(D);
    if (WARP) {
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
    }
    const int turn = WARP ? threadIdx.x >> 5 : t.group, turns = WARP ? kLnThreads / 32 : t.groups;
    for (int q = 0; q < turns; ++q) {
        if (turn == q && (!WARP || (int)(threadIdx.x & 31) < lanes)) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int e = 2 * i + k, at_col = (row_first<EPT / VE>(t) + e / VE * 32) * VE + e % VE;
                    if (!in.in_row(e)) continue;
                    const float a = k ? dw[i].hi() : dw[i].lo(), d = k ? db[i].hi() : db[i].lo();
                    acc[at_col] = q ? acc[at_col] + a : a;
                    acc[Dp + at_col] = q ? acc[Dp + at_col] + d : d;
                }
            }
        }
        __syncthreads();
    }
    float* out = part + (size_t)block * 2 * Dp + left;
    if (PAIR) {
        for (int q = threadIdx.x; q < width; q += blockDim.x) {
            out[q] = acc[q];
            out[Dp + q] = acc[Dp + q];
        }
    } else {
        for (int q = threadIdx.x; q < Dp / 2; q += blockDim.x)
            reinterpret_cast<float4*>(out)[q] = reinterpret_cast<const float4*>(acc)[q];
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

// Any D, and a sum without a residual: one block per row, three passes (the later ones from L1/L2). x,
// residual, y and sum_out may alias element by element: an element is read by the thread that writes it.
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

// dx of any D: one block per row, two passes. This kernel, the one above and the one below are ordinary
// launches and have no wait for the kernel before them: __restrict__ is safe in them for that reason alone.
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
// part [gridDim.y, 2, ln_pitch(D)].
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
    part[(size_t)blockIdx.y * 2 * ln_pitch(D) + c] = dw;
    part[((size_t)blockIdx.y * 2 + 1) * ln_pitch(D) + c] = db;
}

// dw and db from `parts` rows of partial sums: 16 columns per block, four per thread, 64 threads per
// column over every 64th row; those are joined in a fixed order, so equal calls agree bit for bit.
constexpr int kReduceColumns = 16, kReduceQuads = kReduceColumns / 4;
template <typename W>
__global__ void __launch_bounds__(kLnThreads)
ln_reduce_kernel(const float* part, int parts, W* dweight, W* dbias, int D) {
    __shared__ float4 sm[kLnThreads / 32][kReduceQuads];
    const int Dp = ln_pitch(D), quad = threadIdx.x % kReduceQuads, slice = threadIdx.x / kReduceQuads;
    const int c = blockIdx.x * kReduceColumns + 4 * quad;  // of 2 Dp
    wait_previous_kernel();
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& z) { t = make_float4(t.x + z.x, t.y + z.y, t.z + z.z, t.w + z.w); };
    if (c < 2 * Dp) {
#pragma unroll 4
        for (int p = slice; p < parts; p += kLnThreads / kReduceQuads)
            add(*reinterpret_cast<const float4*>(part + (size_t)p * 2 * Dp + c));
    }
#pragma unroll
    for (int off = kReduceQuads; off < 32; off <<= 1) {
        add(make_float4(__shfl_xor_sync(0xffffffffu, t.x, off), __shfl_xor_sync(0xffffffffu, t.y, off),
                        __shfl_xor_sync(0xffffffffu, t.z, off), __shfl_xor_sync(0xffffffffu, t.w, off)));
    }
    if ((threadIdx.x & 31) < kReduceQuads) sm[threadIdx.x >> 5][quad] = t;
    __syncthreads();
    const int mine = blockIdx.x * kReduceColumns + threadIdx.x;
    if (threadIdx.x >= kReduceColumns || mine >= 2 * Dp) return;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kLnThreads / 32; ++i) v += reinterpret_cast<const float*>(sm[i])[threadIdx.x];
    const int col = mine < Dp ? mine : mine - Dp;
    W* out = mine < Dp ? dweight : dbias;
    if (out && col < D) st_elem(out + col, v);
}

}  // namespace ret
