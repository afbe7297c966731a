// Helpers of the operators around the recurrence (short convolution, selective scan,
// norms): 8-element vectors of either element type, activations, the sum of partial
// rows, argument checks, and the status word shared with the rest of the library.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "comba.h"

namespace comba {

// Device address of the current device's status word (see common.cuh); nullptr if the
// runtime cannot give it.
int* status_word();

namespace blk {

using bf16 = __nv_bfloat16;

constexpr int kVec = 8;          // elements a thread handles at a time on the vector path
constexpr int kSMs = 148;        // B200; sizes grids only, results do not depend on it

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ bf16 from_f<bf16>(float x) { return __float2bfloat16_rn(x); }

// V consecutive elements at p, as floats.  V == 8 needs 16-byte alignment.
template <int V>
__device__ __forceinline__ void load_v(const bf16* __restrict__ p, float (&x)[V]) {
    if constexpr (V == 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else if constexpr (V == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        x[0] = __uint_as_float(u.x << 16); x[1] = __uint_as_float(u.x & 0xffff0000u);
        x[2] = __uint_as_float(u.y << 16); x[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = to_f(p[i]);
    }
}
template <int V>
__device__ __forceinline__ void load_v(const float* __restrict__ p, float (&x)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 u = reinterpret_cast<const float4*>(p)[i];
            x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = u.z; x[4 * i + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = p[i];
    }
}

// Brings the line at p into L2 while nothing waits for it.
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

template <int V>
__device__ __forceinline__ void store_v(bf16* __restrict__ p, const float (&x)[V]) {
    if constexpr (V == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                  pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = __float2bfloat16_rn(x[i]);
    }
}
template <int V>
__device__ __forceinline__ void store_v(float* __restrict__ p, const float (&x)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = x[i];
    }
}

// Pairs of fp32 values in a 64-bit register: one instruction for two products or sums.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float a, float b) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(Pair v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
constexpr float kLog2e = 1.44269504088896340736f;

// 2^v and 1 / v by the hardware's approximations (relative errors 2^-22 and 2^-23).
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// sigmoid(v) = 1 / (1 + exp(-v)); where the exponential overflows, 0.
__device__ __forceinline__ float sigmoid(float v) { return rcp_fast(1.f + exp2_fast(-kLog2e * v)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
// d silu / dv
__device__ __forceinline__ float dsilu(float v) {
    const float s = sigmoid(v);
    return s * (1.f + v * (1.f - s));
}

// softplus(v) = log(1 + e), e = exp(v); above 20 it is v to fp32 precision, -inf gives 0, and
// NaN stays NaN (a token must not pass for one with dt = -inf).  The exponent v log2(e) is taken in two parts, since its rounding alone would be 3e-7 of e at
// v = -7, where time steps of 1e-3 lie.  Up to e = 1/2 as 2 atanh(s) with s = e / (2 + e) <=
// 1/5, by atanh's series up to s^11 (the next term is 6e-10 of the sum), which keeps the
// relative precision of small results; above, from the hardware's logarithm of 1 + e, whose
// absolute error of 2^-22 is 6e-7 of results of at least 0.4.
__device__ __forceinline__ float softplus(float v) {
    const float w = fmaxf(v, -126.f);   // below, e is 0 to every sum it enters, and -inf has no rest
    const float t = kLog2e * w, rest = fmaf(w, kLog2e, -t);
    float e = exp2_fast(t);
    e = v < -100.f ? 0.f : fmaf(e, rest * 0.693147181f, e);
    const float s = e * rcp_fast(2.f + e), q = s * s;
    float r = fmaf(q, 1.f / 11.f, 1.f / 9.f);
    r = fmaf(q, r, 1.f / 7.f);
    r = fmaf(q, r, 1.f / 5.f);
    r = fmaf(q, r, 1.f / 3.f);
    r = 2.f * fmaf(q * s, r, s);
    r = e > 0.5f ? __logf(1.f + e) : r;
    return v <= 20.f ? r : v;   // NaN too: fmaxf has dropped it from r
}

// Sequence bounds on the joint token axis: N uniform sequences of T tokens, or packed
// ones with device bounds over T tokens in all.  A packed sequence is well formed if its
// bounds lie in [0, T] in order; others are skipped.
struct Seqs {
    const int* cu;      // nullptr: uniform
    int N;
    int T;              // tokens per sequence (uniform) or in all (packed)
    __host__ __device__ long tokens() const { return cu ? (long)T : (long)N * T; }
    __device__ __forceinline__ bool bounds(int n, long& s, long& e) const {
        if (!cu) {
            s = (long)n * T;
            e = s + T;
            return true;
        }
        s = cu[n];
        e = cu[n + 1];
        return s >= 0 && s <= e && e <= T;
    }
    // The last sequence that starts at or before token t (0 if none does).  Whatever the
    // bounds hold, the answer is in [0, N).
    __device__ __forceinline__ int find(long t) const {
        if (!cu) return (int)(t / T);
        int lo = 0, hi = N - 1;
        while (lo < hi) {
            const int mid = hi - ((hi - lo) >> 1);   // the upper middle; lo + hi may pass 2^31
            if (cu[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
};

// out[k][c] = sum over rows of part[k][row][c] for k = blockIdx.y (where out[k] is given), in
// double and in a fixed order: 32 columns by 8 row lanes a block.
struct SumRows {
    const float* part;
    float* out[3];
    long rows, cols;
};
__global__ void __launch_bounds__(256)
sum_rows_kernel(const __grid_constant__ SumRows p) {
    __shared__ double s[8][33];
    float* out = p.out[blockIdx.y];
    if (!out) return;
    const float* part = p.part + blockIdx.y * p.rows * p.cols;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const long c = (long)blockIdx.x * 32 + lane;
    double acc = 0.0;
    if (c < p.cols) {
#pragma unroll 8
        for (long r = w; r < p.rows; r += 8) acc += (double)part[r * p.cols + c];
    }
    s[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < p.cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) acc += s[i][lane];
        out[c] = (float)acc;
    }
}

// ------------------------------------------------------------------ host side
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// One tensor argument of an entry point: its bytes, the alignment it needs and whether it
// may be null.
struct Arg {
    const void* p;
    size_t bytes;
    size_t align;
    bool optional;
};

// Every argument present (unless optional or empty) and aligned; no output overlaps an
// input or another output.
template <int NI, int NO>
inline bool args_ok(const Arg (&ins)[NI], const Arg (&outs)[NO]) {
    for (const Arg& a : ins)
        if ((!a.p && !a.optional && a.bytes) || !aligned(a.p, a.align)) return false;
    for (const Arg& a : outs)
        if ((!a.p && !a.optional && a.bytes) || !aligned(a.p, a.align)) return false;
    for (int i = 0; i < NO; ++i) {
        for (const Arg& a : ins)
            if (overlap(outs[i].p, outs[i].bytes, a.p, a.bytes)) return false;
        for (int j = i + 1; j < NO; ++j)
            if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return false;
    }
    return true;
}

inline int launched() { return cudaGetLastError() == cudaSuccess ? COMBA_OK : COMBA_ECUDA; }
inline long ceil_div(long a, long b) { return (a + b - 1) / b; }

}  // namespace blk
}  // namespace comba
