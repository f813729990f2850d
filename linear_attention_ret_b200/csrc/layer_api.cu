// C ABI of libret.so, second part (declared in include/ret.h): the operators around retention, that is
// the rotary prologue, layer norm with its gradients and the gradients of the output epilogue. Host-side
// validation, kernel selection and launch. A translation unit of its own: these kernels have
// no waits that could run out, so they share nothing with the retention kernels' error word.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <initializer_list>
#include <utility>

#include "layer_norm.cuh"
#include "norm_backward.cuh"
#include "rotary.cuh"

using namespace ret;

namespace {

constexpr int kMaxDevices = 64;

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline ret_status status(cudaError_t e) {
    if (e == cudaSuccess) return RET_OK;
    cudaGetLastError();  // reported by the status: nobody else's next check finds it
    return RET_ERR_CUDA;
}
inline ret_status launch_status() { return status(cudaGetLastError()); }

inline int current_device() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

inline int sm_count() {
    static std::atomic<int> known[kMaxDevices];
    const int dev = current_device();
    const bool keep = dev >= 0 && dev < kMaxDevices;
    int n = keep ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (dev < 0 || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            return 148;
        if (keep) known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Inside, this thread may make calls that a stream capture forbids: what is set up once per process
// is also set up when the first call is captured.
struct RelaxedCapture {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
    ~RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

// Stream-ordered scratch from the device's default pool, which keeps freed memory for the next call.
inline cudaError_t scratch_alloc(float** p, size_t floats, cudaStream_t st) {
    static std::atomic<bool> done[kMaxDevices];
    const int dev = current_device();
    if (dev >= 0 && dev < kMaxDevices && !done[dev].exchange(true)) {
        RelaxedCapture relaxed;
        cudaMemPool_t pool;
        uint64_t threshold = UINT64_MAX;
        if (cudaDeviceGetDefaultMemPool(&pool, dev) == cudaSuccess)
            cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &threshold);
    }
    return cudaMallocAsync(reinterpret_cast<void**>(p), sizeof(float) * floats, st);
}

// A programmatic dependent launch in clusters of `cluster` blocks: the kernel's blocks may be placed
// while the previous kernel in the stream drains, and wait for it (wait_previous_kernel) before they
// read or write anything.
template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), unsigned grid, int cluster, int threads, size_t smem, cudaStream_t st,
                            A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t st,
                             A&&... args) {
    return launch_clusters(kernel, grid, 1, threads, smem, st, std::forward<A>(args)...);
}

// Most elements of one tensor: more than any device holds, few enough that byte counts fit.
constexpr long long kMaxElements = 1LL << 46;
// Longest row (layer norm's D, a head's d or dv): column numbers, a step of the general kernels' loops past
// the last one, and a row of both column sums (2 D floats) are counted in 31 bits.
constexpr int kMaxRow = 1 << 29;
inline size_t elt_size(ret_dtype dt) { return dt == RET_BF16 ? 2 : 4; }
inline bool valid_dtype(int dt) { return dt == RET_F32 || dt == RET_BF16; }

// Whether [a, a + na) and [b, b + nb) share a byte; a null pointer shares none.
inline bool bytes_overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), z = reinterpret_cast<uintptr_t>(b);
    return a && b && x < z + nb && z < x + na;
}
inline bool ranges_overlap(const void* a, const void* b, size_t bytes) {
    return bytes_overlap(a, bytes, b, bytes);
}

// ------------------------------------------------------------------ rotary prologue (see rotary.cuh)

// A strided [B, N, H, d] tensor: byte address, strides in elements, head dimension contiguous.
struct Strided {
    uintptr_t base;
    long long st[3];  // batch, token, head
    int n[3];
    int d;
    size_t elt;
    // one past the last element, in elements from the base
    long long extent() const {
        long long e = d;
        for (int i = 0; i < 3; ++i) e += st[i] * (long long)(n[i] - 1);
        return e;
    }
    bool same(const Strided& o) const {
        for (int i = 0; i < 3; ++i)
            if (n[i] != o.n[i] || (n[i] > 1 && st[i] != o.st[i])) return false;
        return base == o.base && d == o.d;
    }
};

// No two indices of `v` share an element: taken by increasing stride, each dimension steps over all
// of those below it.
bool writes_once(const Strided& v) {
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return v.st[a] < v.st[b]; });
    long long span = v.d;
    for (int i : order) {
        if (v.n[i] == 1) continue;
        if (v.st[i] < span) return false;
        span += v.st[i] * (long long)(v.n[i] - 1);
    }
    return true;
}

// Whether a and b are seen to share no element: their address ranges are disjoint, or they are
// column blocks of one row-strided buffer (slices of a fused projection): the same row stride,
// and heads at distinct places of each row.
bool disjoint(const Strided& a, const Strided& b) {
    const uintptr_t ea = a.base + (uintptr_t)a.extent() * a.elt, eb = b.base + (uintptr_t)b.extent() * b.elt;
    if (ea <= b.base || eb <= a.base) return true;
    long long row = 0;  // the stride of rows; batches of both must be whole rows apart
    for (int i = 1; i >= 0; --i) {
        if (a.n[i] == 1 && b.n[i] == 1) continue;
        const long long s = a.n[i] > 1 ? a.st[i] : b.st[i];
        if ((a.n[i] > 1 && a.st[i] != s) || (b.n[i] > 1 && b.st[i] != s)) return false;
        if (row == 0) row = s;
        else if (s % row != 0) return false;
    }
    const long long bytes = (long long)(b.base - a.base), elt = (long long)a.elt;
    if (row <= 0 || bytes % elt != 0) return false;
    const long long wa = a.st[2] * (a.n[2] - 1) + a.d, wb = b.st[2] * (b.n[2] - 1) + b.d;
    const long long at = ((bytes / elt) % row + row) % row;
    return at >= wa && at + wb <= row;
}

inline int rotary_units(const RotArgs& a, bool half, int ve) {
    return half ? a.rot / 2 / ve + ((a.d - a.rot) / ve + 1) / 2 : a.d / ve;
}

template <typename T, int VE, bool HALF, int BATCH, bool MANY>
ret_status launch_rotary_batch(const RotArgs& a, int apart, cudaStream_t st) {
    constexpr int kTableBytes = 32 * 1024;  // most shared memory for cos and sin
    RotPlan pl;
    pl.half_units = HALF ? a.rot / 2 / VE : 0;
    pl.apart = apart;
    pl.tensors = a.x[1].H > 0 ? 2 : 1;
    const int units = rotary_units(a, HALF, VE), heads = std::max(a.x[0].H, a.x[1].H);
    const int groups = std::max(1, kRotThreads / (units * pl.tensors));  // head groups of a block's q (or k)
    pl.stride = (a.rot / 2 + VE - 1) / VE * VE;  // whole vectors
    const long long all = (long long)a.B * a.N;
    // head groups of a token: one batch of rows per thread, or as many threads as there are heads
    // where that leaves SMs idle (decode)
    int split = MANY ? heads : std::min(groups, (heads + BATCH - 1) / BATCH);
    if (all * split < (long long)groups * 2 * sm_count()) split = std::min(groups, heads);
    const int table = pl.stride ? std::max(1, kTableBytes / (8 * pl.stride)) : kRotThreads * BATCH;  // tokens it holds
    pl.at_once = std::min(groups / split, MANY ? std::max(1, table / BATCH) : table);
    pl.tokens = (int)std::min<long long>(MANY ? std::min(pl.at_once * BATCH, table) : pl.at_once, all);
    pl.units = FastDiv((unsigned)units);
    pl.split = FastDiv((unsigned)split);
    pl.N = FastDiv((unsigned)a.N);
    const size_t smem = (size_t)8 * pl.tokens * pl.stride;
    return status(launch_dependent(rotary_vec_kernel<T, VE, HALF, BATCH, MANY>,
                                   (unsigned)((all + pl.tokens - 1) / pl.tokens), kRotThreads, smem, st, a, pl));
}

template <typename T, int VE, bool HALF>
ret_status launch_rotary_vec(const RotArgs& a, int apart, cudaStream_t st) {
    const int heads = std::max(a.x[0].H, a.x[1].H), units = rotary_units(a, HALF, VE) * (a.x[1].H > 0 ? 2 : 1);
    // One or two heads, a thread for each, and tokens enough for two blocks per SM all the same (134 MB of bf16
    // heads of 128, one 48.6 us against 65.7 us, two 35.4 against 36.4; three 32.7 against 27.2 and four 29.1
    // against 23.5 the other way; 64 and 256 alike).
    if (heads < 3 && heads * units <= kRotThreads &&
        (long long)a.B * a.N >= (long long)4 * (kRotThreads / (heads * units)) * 2 * sm_count())
        return launch_rotary_batch<T, VE, HALF, 4, true>(a, apart, st);
    // Eight rows at once from eight heads on: 134 MB, half layout, twelve heads of 128 23.9 us against
    // 25.5 us with four rows, eight and sixteen heads within 2% (six heads of 256 would take it too: 24.1 against 25.6).
    if constexpr (HALF && VE > 1 && VE * sizeof(T) <= 8)
        if (heads >= 8) return launch_rotary_batch<T, VE, HALF, 8, false>(a, apart, st);
    return launch_rotary_batch<T, VE, HALF, 4, false>(a, apart, st);
}

// The widest vectors that every row of every view starts on and that the layout's parts are whole
// numbers of, else single elements; a thread per pair where a head's units outnumber a block.
template <typename T, bool HALF>
ret_status launch_rotary(const RotArgs& a, cudaStream_t st) {
    constexpr int kE = 16 / (int)sizeof(T);
    auto fits = [&](int ve) {
        const size_t bytes = ve * sizeof(T);
        if (a.d % ve != 0 || (HALF && a.rot / 2 % ve != 0) ||
            rotary_units(a, HALF, ve) * (a.x[1].H > 0 ? 2 : 1) > kRotThreads)
            return false;
        for (const RotView& v : a.x) {
            if (v.H == 0) continue;
            for (const void* p : {v.in, static_cast<const void*>(v.out)})
                if (reinterpret_cast<uintptr_t>(p) % bytes != 0) return false;
            const long long st3[3][2] = {{v.ib, v.ob}, {v.in_, v.on}, {v.ih, v.oh}};
            const int n[3] = {a.B, a.N, v.H};
            for (int i = 0; i < 3; ++i)
                if (n[i] > 1 && (st3[i][0] % ve != 0 || st3[i][1] % ve != 0)) return false;
        }
        return true;
    };
    const bool small = (long long)a.B * a.N < (1LL << 31);  // tokens are counted in 31 bits
    if constexpr (!(HALF && sizeof(T) == 2))
        if (small && fits(kE)) return launch_rotary_vec<T, kE, HALF>(a, a.rot / 2, st);
    if (small && fits(kE / 2)) return launch_rotary_vec<T, kE / 2, HALF>(a, a.rot / 2, st);
    if (sizeof(T) == 2 && small && fits(2)) return launch_rotary_vec<T, 2, HALF>(a, a.rot / 2, st);
    if (small && (a.d + 1) / 2 * (a.x[1].H > 0 ? 2 : 1) <= kRotThreads)
        return launch_rotary_vec<T, 1, true>(a, HALF ? a.rot / 2 : 1, st);
    const size_t total = (size_t)a.B * a.N * (size_t)(a.x[0].H + a.x[1].H) * (size_t)(a.d - a.rot / 2);
    const unsigned grid = (unsigned)std::min<size_t>((total + kRotThreads - 1) / kRotThreads, (size_t)32 * sm_count());
    rotary_kernel<T, HALF><<<grid, kRotThreads, 0, st>>>(a, total);
    return launch_status();
}

// ------------------------------------------------------------------ layer norm (see layer_norm.cuh)

inline unsigned block_rows(long long rows) {
    return (unsigned)std::min<long long>(rows, (long long)32 * sm_count());
}

// Elements of one access: 16 bytes where every row (and weight) starts on 16 bytes, pairs of
// 2-byte elements where on 4, else single elements.
inline int norm_vector(size_t elt, size_t welt, int D, std::initializer_list<const void*> rows,
                       std::initializer_list<const void*> weights) {
    auto fits = [&](int ve) {
        if (D % ve != 0) return false;
        for (const void* p : rows)
            if (!aligned_to(p, ve * elt)) return false;
        for (const void* p : weights)
            if (!aligned_to(p, std::min<size_t>(16, ve * welt))) return false;
        return true;
    };
    const int widest = 16 / (int)elt;
    return fits(widest) ? widest : elt == 2 && fits(2) ? 2 : 1;
}
inline int lanes_for(int chunks) {  // a power of two up to 32
    int n = 1;
    while (n < chunks && n < 32) n *= 2;
    return n;
}
inline int warp_threads(int n) { return (n + 31) / 32 * 32; }

// Blocks that stay: as many as fit the device at once, or as many as the rows need. A kernel's
// occupancy (its shared memory limit raised first) is asked for once per device and block size.
struct StayingBlocks {
    std::atomic<int> per_sm[kMaxDevices][17];
};
template <typename Kernel>
int staying_blocks(Kernel kernel, StayingBlocks& known, int threads, size_t smem, long long blocks) {
    const int dev = current_device();
    std::atomic<int>* k = dev >= 0 && dev < kMaxDevices ? &known.per_sm[dev][threads / 32] : nullptr;
    int per_sm = k ? k->load(std::memory_order_relaxed) : 0;
    if (per_sm == 0) {
        RelaxedCapture relaxed;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLnMaxShared) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1)
            return 0;
        if (k) k->store(per_sm, std::memory_order_relaxed);
    }
    return (int)std::min<long long>(blocks, (long long)per_sm * sm_count());
}

template <typename T, typename W, int VE, int EPT, bool WARP, bool RES, bool PAIR>
ret_status launch_ln_forward(const T* x, const T* res, const W* w, const W* b, T* y, T* sum_out, float* mean,
                             float* rstd, long long rows, int D, float eps, cudaStream_t st) {
    static StayingBlocks known;
    const int chunks = PAIR ? (D / VE + 1) / 2 : D / VE;  // of a block
    const int lanes = WARP ? (VE == 1 ? 32 : lanes_for(chunks)) : warp_threads((chunks + EPT / VE - 1) / (EPT / VE));
    const int threads = WARP ? kLnThreads : lanes;
    const long long per_block = WARP ? threads / lanes : 1;
    const size_t smem = Rows<T, VE, EPT, RES ? 2 : 1, 0>::bytes(threads);
    const auto kernel = ln_forward_kernel<T, W, VE, EPT, WARP, RES, PAIR>;
    int grid = staying_blocks(kernel, known, threads, smem, (rows + per_block - 1) / per_block * (PAIR ? 2 : 1));
    if (grid == 0) return RET_ERR_CUDA;
    if (PAIR) grid = grid / 2 * 2;
    return status(launch_clusters(kernel, (unsigned)grid, PAIR ? 2 : 1, threads, smem, st, x, res, w, b, y, sum_out,
                                  mean, rstd, (unsigned)rows, D, eps, lanes));
}

template <typename T, typename W, int VE, bool RES>
ret_status launch_ln_forward_width(const T* x, const T* res, const W* w, const W* b, T* y, T* sum_out, float* mean,
                                   float* rstd, long long rows, int D, float eps, cudaStream_t st) {
#define RET_LN_FORWARD(LANES, EPT, WARP, PAIR) \
    if (D <= LANES * EPT)                      \
    return launch_ln_forward<T, W, VE, EPT, WARP, RES, PAIR>(x, res, w, b, y, sum_out, mean, rstd, rows, D, eps, st)
    RET_LN_FORWARD(32, 8, true, false);
    RET_LN_FORWARD(32, 16, true, false);
    RET_LN_FORWARD(512, 16, false, false);
    using Wide = Rows<T, VE, 32, RES ? 2 : 1, 0>;
    if constexpr (Wide::kAsync && Wide::bytes(512) <= kLnMaxShared) {
        RET_LN_FORWARD(512, 32, false, false);
    } else {
        RET_LN_FORWARD(1024, 16, false, true);
    }
#undef RET_LN_FORWARD
    return RET_ERR_UNSUPPORTED;  // not reached: wider rows are not sent here
}

// Rows of up to 16,384 elements are read once, in the vectors of norm_vector; longer rows (and 2^30
// rows and more) in three passes. So is a sum without a residual, which is x: the one-pass kernels store
// a sum only where they form one. With that store in those without a residual too, calls that ask for no
// sum took longer above 8,192 elements (2046 x 8200 in bf16: 24.8 us against 20.2 us).
template <typename T, typename W>
ret_status launch_layer_norm(const void* x_, const void* res_, const void* w_, const void* b_, void* y_,
                             void* sum_out_, float* mean, float* rstd, long long rows, int D, float eps,
                             cudaStream_t st) {
    constexpr int kE = 16 / (int)sizeof(T);
    const T *x = static_cast<const T*>(x_), *res = static_cast<const T*>(res_);
    const W *w = static_cast<const W*>(w_), *b = static_cast<const W*>(b_);
    T *y = static_cast<T*>(y_), *sum_out = static_cast<T*>(sum_out_);
    if (D <= 1024 * 16 && rows < (1LL << 30) && (res || !sum_out)) {
        auto go = [&](auto plain, auto with_residual) {
            return (res ? with_residual : plain)(x, res, w, b, y, sum_out, mean, rstd, rows, D, eps, st);
        };
        const int ve = norm_vector(sizeof(T), sizeof(W), D, {x, res, y, sum_out}, {w, b});
        if (ve == kE) return go(launch_ln_forward_width<T, W, kE, false>, launch_ln_forward_width<T, W, kE, true>);
        if constexpr (sizeof(T) == 2)
            if (ve == 2) return go(launch_ln_forward_width<T, W, 2, false>, launch_ln_forward_width<T, W, 2, true>);
        return go(launch_ln_forward_width<T, W, 1, false>, launch_ln_forward_width<T, W, 1, true>);
    }
    ln_forward_rows_kernel<T, W><<<block_rows(rows), kLnThreads, 0, st>>>(x, res, w, b, y, sum_out, mean, rstd,
                                                                          (size_t)rows, D, eps);
    return launch_status();
}

template <typename W>
ret_status launch_ln_reduce(const float* part, int parts, W* dw, W* db, int D, cudaStream_t st) {
    const unsigned blocks = (unsigned)((2LL * ln_pitch(D) + kReduceColumns - 1) / kReduceColumns);
    return status(launch_dependent(ln_reduce_kernel<W>, blocks, kLnThreads, 0, st, part, parts, dw, db, D));
}

template <typename T, typename W, int VE, int EPT, bool WARP, bool SUM, bool PAIR>
ret_status launch_ln_backward(const T* dy, const T* x, const W* w, const float* mean, const float* rstd, const T* dsum,
                              T* dx, W* dw, W* db, long long rows, int D, cudaStream_t st) {
    const int chunks = PAIR ? (D / VE + 1) / 2 : D / VE;  // of a block
    const int lanes = WARP ? (VE == 1 ? 32 : lanes_for(chunks)) : warp_threads((chunks + EPT / VE - 1) / (EPT / VE));
    // rows at once: a warp's groups of lanes, one row per pair of blocks, or groups of whole warps up
    // to 512 threads as far as there are rows for them
    int groups = WARP ? kLnThreads / lanes : 1;
    if (!WARP && !PAIR)
        groups = (int)std::max<long long>(1, std::min<long long>(std::min(kLnGroups, 512 / lanes), rows / sm_count()));
    const int threads = groups * lanes;
    const size_t ring = Rows<T, VE, EPT, SUM ? 3 : 2, 2>::bytes(threads);
    const size_t smem = std::max(ring, sizeof(float) * 2 * ln_pitch(D));
    static StayingBlocks known;
    const auto kernel = ln_backward_kernel<T, W, VE, EPT, WARP, SUM, PAIR>;
    // A block leaves a row of partial sums, 8 D bytes written and read again: four rows or more
    // each, unless that would leave SMs idle.
    const long long most = (rows + groups - 1) / groups;
    const long long sets = sm_count() / (PAIR ? 2 : 1);
    int grid = staying_blocks(kernel, known, threads, smem, std::max((most + 3) / 4, std::min(most, sets)));
    if (grid == 0) return RET_ERR_CUDA;
    if (PAIR) grid = (int)std::min<long long>(grid, sets);
    float* part = nullptr;
    ret_status r = RET_OK;
    if (dw || db) r = status(scratch_alloc(&part, 2 * (size_t)grid * ln_pitch(D), st));
    if (r != RET_OK) return r;
    r = status(launch_clusters(kernel, (unsigned)(PAIR ? 2 * grid : grid), PAIR ? 2 : 1, threads, smem, st, dy, x, w,
                               mean, rstd, dsum, dx, part, (unsigned)rows, D, lanes));
    if (part) {
        if (r == RET_OK) r = launch_ln_reduce(part, grid, dw, db, D, st);
        if (cudaFreeAsync(part, st) != cudaSuccess && r == RET_OK) r = RET_ERR_CUDA;
    }
    return r;
}

template <typename T, typename W, int VE, bool SUM>
ret_status launch_ln_backward_width(const T* dy, const T* x, const W* w, const float* mean, const float* rstd,
                                    const T* dsum, T* dx, W* dw, W* db, long long rows, int D, cudaStream_t st) {
#define RET_LN_BACKWARD(LANES, EPT, WARP) \
    if (D <= LANES * EPT)                 \
    return launch_ln_backward<T, W, VE, EPT, WARP, SUM, false>(dy, x, w, mean, rstd, dsum, dx, dw, db, rows, D, st)
    RET_LN_BACKWARD(32, 8, true);
    RET_LN_BACKWARD(32, 16, true);
    if constexpr (VE <= 2) RET_LN_BACKWARD(512, 8, false);
    RET_LN_BACKWARD(512, 16, false);
#undef RET_LN_BACKWARD
    return launch_ln_backward<T, W, VE, 16, false, SUM, true>(dy, x, w, mean, rstd, dsum, dx, dw, db, rows, D, st);
}

// Up to 16,384 columns in one pass; wider (and 2^30 rows and more): the column sums and dx in a
// pass of their own each.
template <typename T, typename W>
ret_status launch_layer_norm_backward(const void* dy_, const void* x_, const void* w_, const float* mean,
                                      const float* rstd, const void* dsum_, void* dx_, void* dw_, void* db_,
                                      long long rows, int D, cudaStream_t st) {
    constexpr int kE = 16 / (int)sizeof(T);
    const T *dy = static_cast<const T*>(dy_), *x = static_cast<const T*>(x_), *dsum = static_cast<const T*>(dsum_);
    const W* w = static_cast<const W*>(w_);
    T* dx = static_cast<T*>(dx_);
    W *dw = static_cast<W*>(dw_), *db = static_cast<W*>(db_);
    if (D <= 1024 * 16 && rows < (1LL << 30)) {
        auto go = [&](auto plain, auto with_sum) {
            return (dsum ? with_sum : plain)(dy, x, w, mean, rstd, dsum, dx, dw, db, rows, D, st);
        };
        const int ve = norm_vector(sizeof(T), sizeof(W), D, {dy, x, dsum, dx}, {w});
        if (ve == kE) return go(launch_ln_backward_width<T, W, kE, false>, launch_ln_backward_width<T, W, kE, true>);
        if constexpr (sizeof(T) == 2)
            if (ve == 2) return go(launch_ln_backward_width<T, W, 2, false>, launch_ln_backward_width<T, W, 2, true>);
        return go(launch_ln_backward_width<T, W, 1, false>, launch_ln_backward_width<T, W, 1, true>);
    }
    ret_status r = RET_OK;
    if (dw || db) {
        const unsigned cols = (unsigned)((D + kLnThreads - 1) / kLnThreads);
        const unsigned parts = (unsigned)std::min<long long>(rows, std::max(1u, 8u * sm_count() / cols));
        float* part = nullptr;
        r = status(scratch_alloc(&part, 2 * (size_t)parts * ln_pitch(D), st));
        if (r != RET_OK) return r;
        ln_backward_columns_kernel<T><<<dim3(cols, parts), kLnThreads, 0, st>>>(dy, x, mean, rstd, part, (size_t)rows,
                                                                               D);
        r = launch_status();
        if (r == RET_OK) r = launch_ln_reduce(part, (int)parts, dw, db, D, st);
        if (cudaFreeAsync(part, st) != cudaSuccess && r == RET_OK) r = RET_ERR_CUDA;
        if (r != RET_OK) return r;
    }
    // last: dx may take dy's place
    ln_backward_rows_kernel<T, W><<<block_rows(rows), kLnThreads, 0, st>>>(dy, x, w, mean, rstd, dsum, dx, (size_t)rows,
                                                                           D);
    return launch_status();
}

template <typename T, int VE, int LPR, int CH>
ret_status launch_norm_backward_vec(const T* dy, const T* o, const T* gate, T* dout, T* dgate, int H, int N, int dv,
                                    float eps, size_t rows, cudaStream_t st) {
    const size_t rows_per_block = (size_t)(kNormThreads / 32) * (32 / LPR);
    const size_t blocks = std::min<size_t>((rows + rows_per_block - 1) / rows_per_block, (size_t)32 * sm_count());
    return status(launch_dependent(norm_gate_backward_vec_kernel<T, VE, LPR, CH>, (unsigned)blocks, kNormThreads, 0, st,
                                   dy, o, gate, dout, dgate, FastDiv((unsigned)H), FastDiv((unsigned)N), dv, eps,
                                   (unsigned)rows));
}

// Rows in registers: whole 16-byte chunks on up to 32 lanes, or the narrower accesses of norm_vector
// on 32 lanes; longer rows (and 2^30 rows and more) in two passes.
template <typename T>
ret_status launch_norm_gate_backward(const void* dy_, const void* o_, const void* gate_, void* dout_, void* dgate_,
                                     int B, int H, int N, int dv, float eps, cudaStream_t st) {
    constexpr int kE = 16 / (int)sizeof(T);
    const T *dy = static_cast<const T*>(dy_), *o = static_cast<const T*>(o_), *gate = static_cast<const T*>(gate_);
    T *dout = static_cast<T*>(dout_), *dgate = static_cast<T*>(dgate_);
    const size_t rows = (size_t)B * N * H;
    const int ve = norm_vector(sizeof(T), 1, dv, {dy, o, gate, dout, dgate}, {});
#define RET_NORM_BACKWARD(VE, LPR, CH) \
    if (dv <= VE * LPR * CH)           \
    return launch_norm_backward_vec<T, VE, LPR, CH>(dy, o, gate, dout, dgate, H, N, dv, eps, rows, st)
    if (rows < (1u << 30) && ve == kE) {
        RET_NORM_BACKWARD(kE, 1, 1);
        RET_NORM_BACKWARD(kE, 2, 1);
        RET_NORM_BACKWARD(kE, 4, 1);
        RET_NORM_BACKWARD(kE, 8, 1);
        RET_NORM_BACKWARD(kE, 16, 1);
        RET_NORM_BACKWARD(kE, 32, 1);
        RET_NORM_BACKWARD(kE, 32, 2);
        RET_NORM_BACKWARD(kE, 32, 4);
        RET_NORM_BACKWARD(kE, 32, 8);
    } else if (rows < (1u << 30)) {
        if constexpr (sizeof(T) == 2) {
            if (ve == 2) {
                RET_NORM_BACKWARD(2, 32, 1);
                RET_NORM_BACKWARD(2, 32, 2);
                RET_NORM_BACKWARD(2, 32, 4);
                RET_NORM_BACKWARD(2, 32, 8);
                RET_NORM_BACKWARD(2, 32, 16);
            }
        }
        RET_NORM_BACKWARD(1, 32, 2);
        RET_NORM_BACKWARD(1, 32, 4);
        RET_NORM_BACKWARD(1, 32, 8);
        RET_NORM_BACKWARD(1, 32, 16);
        RET_NORM_BACKWARD(1, 32, 32);
    }
#undef RET_NORM_BACKWARD
    const size_t blocks = std::min<size_t>((rows + kNormThreads / 32 - 1) / (kNormThreads / 32),
                                           (size_t)32 * sm_count());
    norm_gate_backward_scalar_kernel<T><<<(unsigned)blocks, kNormThreads, 0, st>>>(dy, o, gate, dout, dgate, H, N, dv,
                                                                                  eps, rows);
    return launch_status();
}

}  // namespace

extern "C" {

ret_status ret_msr_norm_gate_backward(const void* dy, const void* o, const void* gate, void* dout, void* dgate, int B,
                                      int H, int N, int dv, float eps, ret_dtype dt, void* stream) {
    if (!valid_dtype(dt)) return RET_ERR_DTYPE;
    if (B <= 0 || H <= 0 || N < 0 || dv <= 0) return RET_ERR_SHAPE;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return RET_ERR_SHAPE;
    if (dv > kMaxRow || (__int128)B * H * N > kMaxElements / dv) return RET_ERR_UNSUPPORTED;
    if (N == 0) return RET_OK;
    if (!dy || !o || !gate || !dout || !dgate) return RET_ERR_NULL;
    const size_t bytes = (size_t)B * H * N * dv * elt_size(dt);
    for (const void* p : {dy, o, gate, static_cast<const void*>(dout), static_cast<const void*>(dgate)})
        if (!aligned_to(p, elt_size(dt))) return RET_ERR_ALIGN;
    // dout may take o's place, dgate that of gate or dy; any other overlap would race
    if (ranges_overlap(dout, dgate, bytes) || ranges_overlap(dout, gate, bytes) || ranges_overlap(dout, dy, bytes) ||
        (dout != o && ranges_overlap(dout, o, bytes)) || ranges_overlap(dgate, o, bytes) ||
        (dgate != gate && ranges_overlap(dgate, gate, bytes)) || (dgate != dy && ranges_overlap(dgate, dy, bytes)))
        return RET_ERR_UNSUPPORTED;
    cudaStream_t st = as_stream(stream);
    if (dt == RET_BF16) return launch_norm_gate_backward<__nv_bfloat16>(dy, o, gate, dout, dgate, B, H, N, dv, eps, st);
    return launch_norm_gate_backward<float>(dy, o, gate, dout, dgate, B, H, N, dv, eps, st);
}

ret_status ret_rotary(const void* q, const void* k, void* q_out, void* k_out, const long long* q_strides,
                      const long long* k_strides, const long long* q_out_strides, const long long* k_out_strides,
                      const double* freqs, const long long* positions, const long long* starts, long long offset,
                      int B, int N, int Hq, int Hk, int d, int rot, ret_rotary_layout layout, int inverse,
                      float amplitude, float q_scale, float k_scale, ret_dtype dt, void* stream) {
    if (!valid_dtype(dt)) return RET_ERR_DTYPE;
    if (B <= 0 || N < 0 || Hq <= 0 || Hk < 0 || d <= 0 || rot < 0 || rot > d || rot % 2 != 0) return RET_ERR_SHAPE;
    if (!std::isfinite(amplitude) || !std::isfinite(q_scale) || !std::isfinite(k_scale)) return RET_ERR_SHAPE;
    if (layout != RET_ROTARY_INTERLEAVED && layout != RET_ROTARY_HALF) return RET_ERR_UNSUPPORTED;
    if (d > kMaxRow) return RET_ERR_UNSUPPORTED;
    if (N == 0) return RET_OK;
    if (!q || !q_out || !q_strides || !q_out_strides || (rot > 0 && !freqs)) return RET_ERR_NULL;
    if (Hk > 0 && (!k || !k_out || !k_strides || !k_out_strides)) return RET_ERR_NULL;
    if (positions && starts) return RET_ERR_UNSUPPORTED;
    if (rot > 0 && !aligned_to(freqs, 8)) return RET_ERR_ALIGN;
    if (!aligned_to(positions, 8) || !aligned_to(starts, 8)) return RET_ERR_ALIGN;
    const size_t elt = elt_size(dt);
    RotArgs a{};
    Strided in[2], out[2];
    const void* src[2] = {q, k};
    void* dst[2] = {q_out, k_out};
    const long long* ss[2] = {q_strides, k_strides};
    const long long* ds[2] = {q_out_strides, k_out_strides};
    const int heads[2] = {Hq, Hk}, T = Hk > 0 ? 2 : 1;
    const float scale[2] = {q_scale, k_scale};
    const size_t tokens = (size_t)B * N;
    for (int t = 0; t < T; ++t) {
        for (int i = 0; i < 3; ++i)
            if (ss[t][i] < 0 || ds[t][i] < 0) return RET_ERR_SHAPE;
        if (!aligned_to(src[t], elt) || !aligned_to(dst[t], elt)) return RET_ERR_ALIGN;
        for (const long long* x : {ss[t], ds[t]})
            if ((__int128)x[0] * B + (__int128)x[1] * N + (__int128)x[2] * heads[t] + d > kMaxElements)
                return RET_ERR_UNSUPPORTED;
        in[t] = {reinterpret_cast<uintptr_t>(src[t]), {ss[t][0], ss[t][1], ss[t][2]}, {B, N, heads[t]}, d, elt};
        out[t] = {reinterpret_cast<uintptr_t>(dst[t]), {ds[t][0], ds[t][1], ds[t][2]}, {B, N, heads[t]}, d, elt};
        a.x[t] = {src[t], dst[t], ss[t][0], ss[t][1], ss[t][2], ds[t][0], ds[t][1], ds[t][2], heads[t], scale[t]};
    }
    // each output element is written once and read by nobody else; an output may be its own input
    for (int t = 0; t < T; ++t) {
        if (!writes_once(out[t])) return RET_ERR_UNSUPPORTED;
        const size_t bytes = (size_t)out[t].extent() * elt;
        if (bytes_overlap(dst[t], bytes, freqs, sizeof(double) * (size_t)(rot / 2)) ||
            bytes_overlap(dst[t], bytes, positions, 8 * tokens) || bytes_overlap(dst[t], bytes, starts, 8 * (size_t)B))
            return RET_ERR_UNSUPPORTED;
        for (int i = 0; i < T; ++i)
            if (!disjoint(out[t], in[i]) && !(i == t && out[t].same(in[t]))) return RET_ERR_UNSUPPORTED;
    }
    if (T == 2 && !disjoint(out[0], out[1])) return RET_ERR_UNSUPPORTED;
    a.freqs = freqs;
    a.positions = positions;
    a.starts = starts;
    a.offset = offset;
    a.B = B;
    a.N = N;
    a.d = d;
    a.rot = rot;
    a.amplitude = amplitude;
    a.sign = inverse ? -1.f : 1.f;
    cudaStream_t st = as_stream(stream);
    if (dt == RET_BF16)
        return layout == RET_ROTARY_HALF ? launch_rotary<__nv_bfloat16, true>(a, st)
                                         : launch_rotary<__nv_bfloat16, false>(a, st);
    return layout == RET_ROTARY_HALF ? launch_rotary<float, true>(a, st) : launch_rotary<float, false>(a, st);
}

ret_status ret_layer_norm(const void* x, const void* residual, const void* weight, const void* bias, void* y,
                          void* sum_out, float* mean, float* rstd, long long rows, int D, float eps, ret_dtype dt,
                          ret_dtype wdt, void* stream) {
    if (!valid_dtype(dt) || !valid_dtype(wdt)) return RET_ERR_DTYPE;
    if (wdt != dt && wdt != RET_F32) return RET_ERR_DTYPE;
    if (rows < 0 || D <= 0) return RET_ERR_SHAPE;
    if (D > kMaxRow || rows > kMaxElements / D) return RET_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return RET_ERR_SHAPE;
    if (rows == 0) return RET_OK;
    if (!x || !y) return RET_ERR_NULL;
    const size_t elt = elt_size(dt), welt = elt_size(wdt);
    if (!aligned_to(x, elt) || !aligned_to(residual, elt) || !aligned_to(y, elt) || !aligned_to(sum_out, elt) ||
        !aligned_to(weight, welt) || !aligned_to(bias, welt) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return RET_ERR_ALIGN;
    // y and sum_out may each take the place of x or residual; any other overlap would race
    const size_t bytes = (size_t)rows * D * elt, wb = (size_t)D * welt, sb = (size_t)rows * 4;
    for (const void* out : {static_cast<const void*>(y), static_cast<const void*>(sum_out)}) {
        if ((out != x && bytes_overlap(out, bytes, x, bytes)) ||
            (out != residual && bytes_overlap(out, bytes, residual, bytes)) || bytes_overlap(out, bytes, weight, wb) ||
            bytes_overlap(out, bytes, bias, wb) || bytes_overlap(out, bytes, mean, sb) ||
            bytes_overlap(out, bytes, rstd, sb))
            return RET_ERR_UNSUPPORTED;
    }
    if (bytes_overlap(y, bytes, sum_out, bytes) || bytes_overlap(mean, sb, rstd, sb)) return RET_ERR_UNSUPPORTED;
    for (const void* stat : {static_cast<const void*>(mean), static_cast<const void*>(rstd)})
        if (bytes_overlap(stat, sb, x, bytes) || bytes_overlap(stat, sb, residual, bytes) ||
            bytes_overlap(stat, sb, weight, wb) || bytes_overlap(stat, sb, bias, wb))
            return RET_ERR_UNSUPPORTED;
    cudaStream_t st = as_stream(stream);
    if (dt == RET_F32)
        return launch_layer_norm<float, float>(x, residual, weight, bias, y, sum_out, mean, rstd, rows, D, eps, st);
    if (wdt == RET_F32)
        return launch_layer_norm<__nv_bfloat16, float>(x, residual, weight, bias, y, sum_out, mean, rstd, rows, D, eps,
                                                       st);
    return launch_layer_norm<__nv_bfloat16, __nv_bfloat16>(x, residual, weight, bias, y, sum_out, mean, rstd, rows, D,
                                                           eps, st);
}

ret_status ret_layer_norm_backward(const void* dy, const void* x, const void* weight, const float* mean,
                                   const float* rstd, const void* dsum, void* dx, void* dweight, void* dbias,
                                   long long rows, int D, ret_dtype dt, ret_dtype wdt, void* stream) {
    if (!valid_dtype(dt) || !valid_dtype(wdt)) return RET_ERR_DTYPE;
    if (wdt != dt && wdt != RET_F32) return RET_ERR_DTYPE;
    if (rows < 0 || D <= 0) return RET_ERR_SHAPE;
    if (D > kMaxRow || rows > kMaxElements / D) return RET_ERR_UNSUPPORTED;
    cudaStream_t st = as_stream(stream);
    const size_t elt = elt_size(dt), welt = elt_size(wdt);
    const size_t bytes = (size_t)rows * D * elt, wb = (size_t)D * welt, sb = (size_t)rows * 4;
    if (rows == 0) {  // sums over no rows
        for (void* p : {dweight, dbias})
            if (p && cudaMemsetAsync(p, 0, wb, st) != cudaSuccess) return RET_ERR_CUDA;
        return RET_OK;
    }
    if (!dy || !x || !mean || !rstd || !dx) return RET_ERR_NULL;
    if (!aligned_to(dy, elt) || !aligned_to(x, elt) || !aligned_to(dsum, elt) || !aligned_to(dx, elt) ||
        !aligned_to(weight, welt) || !aligned_to(dweight, welt) || !aligned_to(dbias, welt) || !aligned_to(mean, 4) ||
        !aligned_to(rstd, 4))
        return RET_ERR_ALIGN;
    // dx may take the place of dy, x or dsum; any other overlap would race
    for (const void* in : {dy, x, dsum})
        if ((in != dx && bytes_overlap(dx, bytes, in, bytes)) || bytes_overlap(dweight, wb, in, bytes) ||
            bytes_overlap(dbias, wb, in, bytes))
            return RET_ERR_UNSUPPORTED;
    const struct { const void* p; size_t n; } outs[] = {{dx, bytes}, {dweight, wb}, {dbias, wb}};
    for (const auto& o : outs)
        if (bytes_overlap(o.p, o.n, weight, wb) || bytes_overlap(o.p, o.n, mean, sb) ||
            bytes_overlap(o.p, o.n, rstd, sb))
            return RET_ERR_UNSUPPORTED;
    if (bytes_overlap(dx, bytes, dweight, wb) || bytes_overlap(dx, bytes, dbias, wb) ||
        bytes_overlap(dweight, wb, dbias, wb))
        return RET_ERR_UNSUPPORTED;
    if (dt == RET_F32)
        return launch_layer_norm_backward<float, float>(dy, x, weight, mean, rstd, dsum, dx, dweight, dbias, rows, D,
                                                        st);
    if (wdt == RET_F32)
        return launch_layer_norm_backward<__nv_bfloat16, float>(dy, x, weight, mean, rstd, dsum, dx, dweight, dbias,
                                                                rows, D, st);
    return launch_layer_norm_backward<__nv_bfloat16, __nv_bfloat16>(dy, x, weight, mean, rstd, dsum, dx, dweight,
                                                                    dbias, rows, D, st);
}

}  // extern "C"
