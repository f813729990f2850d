// Device helpers of the operators around retention: vector accesses, asynchronous copies,
// dependent launches, packed fp32 arithmetic and division by a fixed number.
#pragma once

#include <string.h>

#include "common.cuh"

namespace ret {

// One access of 2, 4, 8 or 16 bytes. load_cs evicts first, for tensors that are read once; it is
// volatile so that it stays behind the wait of a dependent launch (the same reason keeps
// __restrict__ and read-only loads out of the kernels that are launched that way).
template <int BYTES> struct RawBytes;
template <> struct RawBytes<2> {
    using type = unsigned short;
    static __device__ __forceinline__ type load_cs(const void* p) {
        type r;
        asm volatile("ld.global.cs.u16 %0, [%1];" : "=h"(r) : "l"(p));
        return r;
    }
};
template <> struct RawBytes<4> {
    using type = unsigned int;
    static __device__ __forceinline__ type load_cs(const void* p) {
        type r;
        asm volatile("ld.global.cs.u32 %0, [%1];" : "=r"(r) : "l"(p));
        return r;
    }
};
template <> struct RawBytes<8> {
    using type = uint2;
    static __device__ __forceinline__ type load_cs(const void* p) {
        type r;
        asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
        return r;
    }
};
template <> struct RawBytes<16> {
    using type = uint4;
    static __device__ __forceinline__ type load_cs(const void* p) {
        type r;
        asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                     : "l"(p));
        return r;
    }
};

// VE consecutive elements moved as one access, the address a multiple of its size.
template <typename T, int VE>
struct Vec {
    using Raw = typename RawBytes<VE * (int)sizeof(T)>::type;
    static __device__ __forceinline__ Raw load_cs(const T* p) { return RawBytes<VE * (int)sizeof(T)>::load_cs(p); }
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

}  // namespace ret
