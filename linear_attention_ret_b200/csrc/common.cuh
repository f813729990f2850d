// Shared device helpers for the retention kernels (sm_100a).
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>
#include <string.h>

#include "ret.h"

namespace ret {

// Device error word. A kernel whose bounded wait runs out ORs a code in here;
// ret_last_device_error() reads and clears it. One per device (module scope).
__device__ unsigned int g_error_word;

enum : unsigned int {
    kErrWaitTimeout = 1u,  // an mbarrier / flag wait exceeded its iteration limit
};

__device__ __forceinline__ void raise_error(unsigned int code) { atomicOr(&g_error_word, code); }

// ---------------------------------------------------------------- element IO

template <typename T> struct Elem;
template <> struct Elem<float> {
    static __device__ __forceinline__ float load(const float* p) { return *p; }
    static __device__ __forceinline__ void store(float* p, float x) { *p = x; }
};
template <> struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
};

template <typename T>
__device__ __forceinline__ float ld_elem(const T* p) { return Elem<T>::load(p); }
template <typename T>
__device__ __forceinline__ void st_elem(T* p, float x) { Elem<T>::store(p, x); }

// VE consecutive elements moved as one access of VE * sizeof(T) bytes (2, 4, 8 or 16), the
// address a multiple of that. load_cs evicts first: for tensors that are read once.
template <int BYTES> struct RawBytes;
template <> struct RawBytes<2> { using type = unsigned short; };
template <> struct RawBytes<4> { using type = unsigned int; };
template <> struct RawBytes<8> { using type = uint2; };
template <> struct RawBytes<16> { using type = uint4; };

template <typename T, int VE>
struct Vec {
    using Raw = typename RawBytes<VE * (int)sizeof(T)>::type;
    static __device__ __forceinline__ Raw load_cs(const T* p) { return __ldcs(reinterpret_cast<const Raw*>(p)); }
    static __device__ __forceinline__ Raw load(const T* p) { return *reinterpret_cast<const Raw*>(p); }
    static __device__ __forceinline__ Raw zero() {
        Raw r;
        memset(&r, 0, sizeof(r));
        return r;
    }
    static __device__ __forceinline__ void unpack(const Raw& u, float* f) {
        if constexpr (sizeof(T) == 2 && VE > 1) {
            // a bf16 is the upper half of its fp32 value: one shift or one mask per element
            unsigned int w[VE / 2];
            memcpy(w, &u, sizeof(u));
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            T e[VE];
            memcpy(e, &u, sizeof(u));
#pragma unroll
            for (int i = 0; i < VE; ++i) f[i] = ld_elem(e + i);
        }
    }
    static __device__ __forceinline__ void store(T* p, const float* f) {
        Raw r;
        if constexpr (sizeof(T) == 2 && VE > 1) {
            unsigned int w[VE / 2];
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                memcpy(&w[i], &b, 4);
            }
            memcpy(&r, w, sizeof(r));
        } else {
            T e[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) st_elem(e + i, f[i]);
            memcpy(&r, e, sizeof(r));
        }
        *reinterpret_cast<Raw*>(p) = r;
    }
};

// One asynchronous copy of BYTES (4, 8 or 16) from global to shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    const unsigned at = (unsigned)__cvta_generic_to_shared(to);
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest LEFT groups of this thread's copies have landed (in the thread's own view).
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Programmatic dependent launch: a kernel launched with the attribute waits here for the one
// before it in the stream, and may let the next one's blocks be placed early.
__device__ __forceinline__ void wait_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next_kernel() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Two floats that one instruction adds, multiplies or fuses (fma.rn.f32x2 and its kin, sm_100):
// each half is rounded as the scalar operation rounds it.
struct F2 {
    unsigned long long v;
    F2() = default;
    __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
    __device__ __forceinline__ float lo() const { return halves(true); }
    __device__ __forceinline__ float hi() const { return halves(false); }
    __device__ __forceinline__ float sum() const { return lo() + hi(); }

  private:
    __device__ __forceinline__ float halves(bool low) const {
        float a, b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
        return low ? a : b;
    }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// Division of a 32-bit number by a fixed 32-bit d >= 1, exact for every n < 2^31: with
// l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d = (umulhi(m, n) + n) >> l
// (Granlund and Montgomery, Division by invariant integers using multiplication, 1994).
struct FastDiv {
    unsigned d, m, l;
    FastDiv() = default;
    explicit FastDiv(unsigned d_) : d(d_), l(0) {
        while ((1ull << l) < d) ++l;
        m = (unsigned)(((1ull << 32) * ((1ull << l) - d)) / d + 1);
    }
    __device__ __forceinline__ unsigned div(unsigned n) const { return (__umulhi(m, n) + n) >> l; }
    __device__ __forceinline__ void divmod(unsigned n, unsigned& q, unsigned& r) const {
        q = div(n);
        r = n - q * d;
    }
};

// gamma^n for an integer n >= 0 given log2(gamma); gamma^0 = 1 even for gamma = 0
// (log2(0) = -inf and exp2(-inf) = 0 give the n > 0 cases).
__device__ __forceinline__ float pow_int_log2(float log2g, int n) {
    return n == 0 ? 1.0f : exp2f(log2g * (float)n);
}

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace ret
