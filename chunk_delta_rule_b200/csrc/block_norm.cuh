// RMS norms at the two ends of a mixer block, fused with what surrounds them:
//
//   gated norm     out = x r(x) w silu(gate),              r(v) = 1 / sqrt(mean v^2 + eps)
//   residual norm  h = residual + scale u,  out = h r(h) w,  u = x, or x r(x) w_post
//
// with x r(x) over the last dimension (a head's values, or the model width).  Each row is
// read and written once and its statistics are two sums, so the kernels are bound by HBM
// bandwidth.  A row lies in the registers of the 8 .. 1024 threads that share it, 8 values
// each: 8 consecutive ones where the rows allow 16-byte accesses, else every TPR-th one,
// so that any width up to 8192 runs.
#pragma once

#include "block_common.cuh"

namespace comba {
namespace norm {

using namespace blk;

constexpr int kMaxWidth = 8192;

// A thread's 8 columns of its row: consecutive (VECTOR), or tid, tid + TPR, ...
template <bool VECTOR>
struct Cols {
    int tid, tpr, D;
    __device__ __forceinline__ bool on(int i) const { return VECTOR ? tid * 8 < D : tid + i * tpr < D; }
    __device__ __forceinline__ int at(int i) const { return VECTOR ? tid * 8 + i : tid + i * tpr; }
    template <typename T>
    __device__ __forceinline__ void load(const T* __restrict__ row, float (&v)[8]) const {
        if constexpr (VECTOR) {
            if (tid * 8 < D) load_v<8>(row + tid * 8, v);
            else
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = 0.f;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = on(i) ? to_f(row[at(i)]) : 0.f;
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* __restrict__ row, const float (&v)[8]) const {
        if constexpr (VECTOR) {
            if (tid * 8 < D) store_v<8>(row + tid * 8, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (on(i)) row[at(i)] = from_f<T>(v[i]);
        }
    }
    // A row of parameters; `other` where there is none.
    __device__ __forceinline__ void param(const float* __restrict__ p, float other, float (&v)[8]) const {
        if (p) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = on(i) ? p[at(i)] : 0.f;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = other;
        }
    }
};

// Sums of K values over the TPR threads of a row, to all of them.  Up to 32 threads: by
// shuffles in their part of the warp.  More: the block is one row, and the warps' sums
// go through shared memory; `slot` alternates between two buffers, so that one barrier
// a call is enough.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int tpr, float (*buf)[32][K], int slot) {
    const int width = tpr < 32 ? tpr : 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < width)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (tpr <= 32) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = tpr >> 5;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) buf[slot][warp][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lane < warps ? buf[slot][lane][k] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}

__device__ __forceinline__ float inv_rms(float sq, int D, float eps) { return 1.f / sqrtf(sq / (float)D + eps); }

// ------------------------------------------------------------------ gated norm
struct Gated {
    const void *x, *gate, *dout;
    const float* weight;
    void *out, *dx, *dgate;
    float* part;       // backward: [blocks, D] partial sums of dweight
    long rows;
    int D, tpr;
    float eps;
};

template <typename T, bool VECTOR>
__global__ void __launch_bounds__(1024)
gated_fwd_kernel(const __grid_constant__ Gated p) {
    __shared__ float buf[2][32][1];
    const int per = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr;
    const Cols<VECTOR> cols{(int)threadIdx.x % p.tpr, p.tpr, p.D};
    float w[8];
    cols.param(p.weight, 1.f, w);
    int slot = 0;
    for (long r0 = (long)blockIdx.x * per; r0 < p.rows; r0 += (long)gridDim.x * per, slot ^= 1) {
        const bool live = r0 + sub < p.rows;
        const long at = (live ? r0 + sub : p.rows - 1) * p.D;
        float x[8], g[8], sq[1] = {0.f};
        cols.load(static_cast<const T*>(p.x) + at, x);
        cols.load(static_cast<const T*>(p.gate) + at, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) sq[0] = fmaf(x[i], x[i], sq[0]);
        row_sum<1>(sq, p.tpr, buf, slot);
        const float r = inv_rms(sq[0], p.D, p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i] * silu(g[i]);
        if (live) cols.store(static_cast<T*>(p.out) + at, x);
    }
}

// Column sums of K per-thread rows over the row groups of a block, to part[k][block][D].
template <int K, bool VECTOR>
__device__ __forceinline__ void column_sums(const Cols<VECTOR>& cols, float (&acc)[K][8], int per, int sub, float* part,
                                            float* smem) {
    // smem: blockDim.x * 8 floats
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (per > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) smem[i * blockDim.x + threadIdx.x] = acc[k][i];
            __syncthreads();
            if (sub == 0)
                for (int s = 1; s < per; ++s)
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[k][i] += smem[i * blockDim.x + s * cols.tpr + cols.tid];
        }
        if (sub == 0) cols.store(part + ((long)k * gridDim.x + blockIdx.x) * cols.D, acc[k]);
    }
}

// Backward.  With n = x r, s = silu(gate), q = dout w s:
//   dx = r (q - n mean(q n)),  dgate = dout n w silu'(gate),  dweight = sum over rows dout n s.
// Both row sums, of x^2 and q x, are taken at once.
template <typename T, bool VECTOR>
__global__ void __launch_bounds__(1024)
gated_bwd_kernel(const __grid_constant__ Gated p) {
    __shared__ float buf[2][32][2];
    extern __shared__ float smem[];
    const int per = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr;
    const Cols<VECTOR> cols{(int)threadIdx.x % p.tpr, p.tpr, p.D};
    float w[8], dw[1][8];
    cols.param(p.weight, 1.f, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[0][i] = 0.f;
    int slot = 0;
    for (long r0 = (long)blockIdx.x * per; r0 < p.rows; r0 += (long)gridDim.x * per, slot ^= 1) {
        const bool live = r0 + sub < p.rows;
        const long at = (live ? r0 + sub : p.rows - 1) * p.D;
        float x[8], g[8], d[8], s[8], sum[2] = {0.f, 0.f};
        cols.load(static_cast<const T*>(p.x) + at, x);
        cols.load(static_cast<const T*>(p.gate) + at, g);
        cols.load(static_cast<const T*>(p.dout) + at, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[i] = sigmoid(g[i]);
            sum[0] = fmaf(x[i], x[i], sum[0]);
            sum[1] = fmaf(d[i] * w[i] * g[i] * s[i], x[i], sum[1]);
        }
        row_sum<2>(sum, p.tpr, buf, slot);
        const float r = inv_rms(sum[0], p.D, p.eps);
        const float mean = sum[1] * r / (float)p.D;   // mean(q n)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float n = x[i] * r, act = g[i] * s[i], dn = d[i] * n;
            x[i] = r * (d[i] * w[i] * act - n * mean);
            g[i] = dn * w[i] * (s[i] * (1.f + g[i] * (1.f - s[i])));
            if (live) dw[0][i] = fmaf(dn, act, dw[0][i]);
        }
        if (live) {
            cols.store(static_cast<T*>(p.dx) + at, x);
            cols.store(static_cast<T*>(p.dgate) + at, g);
        }
    }
    column_sums<1, VECTOR>(cols, dw, per, sub, p.part, smem);
}

// ------------------------------------------------------------------ residual norm
struct Residual {
    const void *x, *residual, *h_in, *dy, *dh;
    const float *weight, *scale, *post;
    void *out, *h, *dx, *dres;
    float* part;       // backward: [3, blocks, D] partial sums of dweight, dscale, dpost
    long rows;
    int D, tpr;
    float eps;
};

// T: block output, its norm and their cotangents; TR: the residual stream.
template <typename T, typename TR, bool VECTOR, bool POST>
__global__ void __launch_bounds__(1024)
residual_fwd_kernel(const __grid_constant__ Residual p) {
    __shared__ float buf[2][32][1];
    const int per = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr;
    const Cols<VECTOR> cols{(int)threadIdx.x % p.tpr, p.tpr, p.D};
    int slot = 0;
    for (long r0 = (long)blockIdx.x * per; r0 < p.rows; r0 += (long)gridDim.x * per) {
        const bool live = r0 + sub < p.rows;
        const long at = (live ? r0 + sub : p.rows - 1) * p.D;
        float x[8], h[8], a[8], sq[1] = {0.f};
        cols.load(static_cast<const T*>(p.x) + at, x);
        cols.load(static_cast<const TR*>(p.residual) + at, h);
        if (POST) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sq[0] = fmaf(x[i], x[i], sq[0]);
            row_sum<1>(sq, p.tpr, buf, slot);
            slot ^= 1;
            const float r = inv_rms(sq[0], p.D, p.eps);
            cols.param(p.post, 1.f, a);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * a[i];
            sq[0] = 0.f;
        }
        cols.param(p.scale, 1.f, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // the norm reads the stream as it is stored, which is what the backward sees
            h[i] = to_f(from_f<TR>(fmaf(x[i], a[i], h[i])));
            sq[0] = fmaf(h[i], h[i], sq[0]);
        }
        if (live) cols.store(static_cast<TR*>(p.h) + at, h);
        row_sum<1>(sq, p.tpr, buf, slot);
        slot ^= 1;
        const float r = inv_rms(sq[0], p.D, p.eps);
        cols.param(p.weight, 1.f, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = h[i] * r * a[i];
        if (live) cols.store(static_cast<T*>(p.out) + at, h);
    }
}

// Backward, from h as the forward stored it.  With m = h r(h):
//   tot = dh + r(h) (dy w - m mean(dy w m)),  dresidual = tot,  dweight = sum dy m,
//   dscale = sum tot u,  du = scale tot,
//   dx = du, or with n = x r(x), u = n w_post:  r(x) (du w_post - n mean(du w_post n)),
//   dpost = sum du n.
template <typename T, typename TR, bool VECTOR, bool POST>
__global__ void __launch_bounds__(1024)
residual_bwd_kernel(const __grid_constant__ Residual p) {
    __shared__ float buf3[2][32][3];
    __shared__ float buf1[2][32][1];
    extern __shared__ float smem[];
    const int per = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr;
    const Cols<VECTOR> cols{(int)threadIdx.x % p.tpr, p.tpr, p.D};
    float w[8], sc[8], po[8], acc[3][8];
    cols.param(p.weight, 1.f, w);
    cols.param(p.scale, 1.f, sc);
    cols.param(p.post, 1.f, po);
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[k][i] = 0.f;
    int slot = 0;
    for (long r0 = (long)blockIdx.x * per; r0 < p.rows; r0 += (long)gridDim.x * per, slot ^= 1) {
        const bool live = r0 + sub < p.rows;
        const long at = (live ? r0 + sub : p.rows - 1) * p.D;
        float x[8], h[8], d[8], g[8], sum[3] = {0.f, 0.f, 0.f};
        cols.load(static_cast<const T*>(p.x) + at, x);
        cols.load(static_cast<const TR*>(p.h_in) + at, h);
        cols.load(static_cast<const T*>(p.dy) + at, d);
        if (p.dh) {
            cols.load(static_cast<const TR*>(p.dh) + at, g);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum[0] = fmaf(h[i], h[i], sum[0]);
            sum[1] = fmaf(d[i] * w[i], h[i], sum[1]);
            if (POST) sum[2] = fmaf(x[i], x[i], sum[2]);
        }
        row_sum<3>(sum, p.tpr, buf3, slot);
        const float r = inv_rms(sum[0], p.D, p.eps);
        const float mean = sum[1] * r / (float)p.D;
        const float rx = POST ? inv_rms(sum[2], p.D, p.eps) : 1.f;
        float q[1] = {0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float m = h[i] * r, n = x[i] * rx;
            g[i] += r * (d[i] * w[i] - m * mean);        // tot
            const float du = g[i] * sc[i];
            if (live) {
                acc[0][i] = fmaf(d[i], m, acc[0][i]);
                acc[1][i] = fmaf(g[i], n * po[i], acc[1][i]);
                if (POST) acc[2][i] = fmaf(du, n, acc[2][i]);
            }
            x[i] = n;
            d[i] = du * po[i];
            if (POST) q[0] = fmaf(d[i], n, q[0]);
        }
        if (live) cols.store(static_cast<TR*>(p.dres) + at, g);
        if (POST) {
            row_sum<1>(q, p.tpr, buf1, slot);
            const float mq = q[0] / (float)p.D;
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = rx * (d[i] - x[i] * mq);
        }
        if (live) cols.store(static_cast<T*>(p.dx) + at, d);
    }
    column_sums<3, VECTOR>(cols, acc, per, sub, p.part, smem);
}

// ------------------------------------------------------------------ launch shapes
// Threads that share a row of D values, 8 each, as a power of two.
inline int row_threads(int D) {
    int t = 8;
    while (t * 8 < D) t *= 2;
    return t;
}
inline int block_threads(int tpr) { return tpr <= 32 ? 256 : tpr; }
// Blocks of the backward: each walks several rows and leaves one row of partial sums.
inline long bwd_blocks(long rows, int D) {
    const int tpr = row_threads(D), threads = block_threads(tpr);
    const long want = (long)kSMs * (threads >= 1024 ? 1 : 1024 / threads);
    const long need = ceil_div(rows, threads / tpr);
    return need < want ? need : want;
}

}  // namespace norm
}  // namespace comba
