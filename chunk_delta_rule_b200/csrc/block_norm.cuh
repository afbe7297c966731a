// RMS norms at the two ends of a mixer block, fused with what surrounds them:
//
//   gated norm     out = x r(x) w silu(gate),              r(v) = 1 / sqrt(mean v^2 + eps)
//   residual norm  h = residual + scale u,  out = h r(h) w,  u = x, or x r(x) w_post
//
// with x r(x) over the last dimension (a head's values, or the model width).  Each row is
// read and written once and its statistics are two sums, so the kernels are bound by HBM
// bandwidth.  A row lies in the registers of the 8 .. 1024 threads that share it, 8 values
// each: 8 consecutive ones where the rows allow 16-byte accesses, else every TPR-th one,
// so that any width up to 8192 runs.  Parameter gradients are summed in fp32 over a thread's
// rows (111 of 32K rows of 2048), then over the blocks in fp64.
//
// Measured, of a copy's 6.55 TB/s: gated norm of 512K bf16 rows of 128, forward 74 us (5.5 TB/s),
// backward 125 us (5.4); residual norm of 32K rows of 2048, bf16 onto an fp32 stream with
// post norm, forward 136 us (5.9), backward 219 us (5.5).  Above a width of 4096 a block has 1024
// threads of 64 registers, and the backwards spill: 64M values of width 5120 and 8192, the same,
// 753 and 547 us (1.6 and 2.2 TB/s), gated 326 and 234 (2.1 and 2.9); fp32 rows onto fp32 at 2048:
// forward 246 us (4.4, spills too), backward 262 (6.1).
#pragma once

#include <type_traits>

#include "block_common.cuh"

namespace comba {
namespace norm {

using namespace blk;

constexpr int kMaxWidth = 8192;
// Blocks of 256 threads of the backwards that an SM's registers hold: 80 registers a thread,
// and 128 where three column sums and up to four rows are kept (gated with 2, 3, 4 blocks: 152,
// 126, 165 us in bf16, fp32 rows of 2048 with 3: 264 us, 5.1 TB/s, spilling 72 bytes a thread;
// residual with 2, 3: 219, 441 us, the latter for its spills).
constexpr int kGatedBlocks = 3, kResidualBlocks = 2;

// 8 values of a row as they are stored.
template <typename T, bool VECTOR>
struct Raw {
    static constexpr int PARTS = VECTOR ? (int)(8 * sizeof(T) / 16) : 8;
    typename std::conditional<VECTOR, uint4, T>::type v[PARTS];
};

// A thread's 8 columns of its row: consecutive (VECTOR), or tid, tid + TPR, ...
template <bool VECTOR>
struct Cols {
    int tid, tpr, D;
    __device__ __forceinline__ bool on(int i) const { return VECTOR ? tid * 8 < D : tid + i * tpr < D; }
    __device__ __forceinline__ int at(int i) const { return VECTOR ? tid * 8 + i : tid + i * tpr; }
    // Loads carry no condition, so that they stay in flight until widen() needs them: columns
    // past the row's end read its first one.
    template <typename T>
    __device__ __forceinline__ Raw<T, VECTOR> fetch(const void* base, long row) const {
        const T* p = static_cast<const T*>(base) + row * D;
        Raw<T, VECTOR> r;
        if constexpr (VECTOR) {
            p += on(0) ? tid * 8 : 0;
#pragma unroll
            for (int i = 0; i < r.PARTS; ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r.v[i] = p[on(i) ? at(i) : 0];
        }
        return r;
    }
    template <typename T>
    __device__ __forceinline__ void widen(const Raw<T, VECTOR>& r, float (&v)[8]) const {
        if constexpr (VECTOR) {   // all on or all off: row_sum leaves off threads out
            load_v<8>(reinterpret_cast<const T*>(r.v), v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = on(i) ? to_f(r.v[i]) : 0.f;
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
            widen<float>(fetch<float>(p, 0), v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = other;
        }
    }
};

// Sums of K values over the TPR threads of a row (those with columns on), to all of them.  Up to 32 threads: by
// shuffles in their part of the warp.  More: the block is one row, and the warps' sums
// go through shared memory; `slot` alternates between two buffers, so that one barrier
// a call is enough.
template <int K, bool VECTOR>
__device__ __forceinline__ void row_sum(const Cols<VECTOR>& cols, float (&v)[K], float (*buf)[32][K], int slot) {
    const int tpr = cols.tpr, width = tpr < 32 ? tpr : 32;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = cols.on(0) ? v[k] : 0.f;
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
    for (int k = 0; k < K; ++k) v[k] = buf[slot][lane & (warps - 1)][k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < warps)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}

// 1 / sqrt(mean + eps) of a sum of squares, from the hardware's approximation (2 ulp).
__device__ __forceinline__ float inv_rms(float sq, float inv_d, float eps) { return rsqrtf(fmaf(sq, inv_d, eps)); }

// ------------------------------------------------------------------ gated norm
struct Gated {
    const void *x, *gate, *dout;
    const float* weight;
    void *out, *dx, *dgate;
    float* part;       // backward: [blocks, D] partial sums of dweight
    long rows;
    int D, tpr;
    float eps, inv_d;
};

// Blocks walk their rows with the next one's loads in flight.  MAXT: the largest block; up
// to 512 threads have the registers to keep the parameters over the rows.
template <typename T, bool VECTOR, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 512 ? 2 : 1)
gated_fwd_kernel(const __grid_constant__ Gated p) {
    __shared__ float buf[2][32][1];
    const int per = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr;
    const Cols<VECTOR> cols{(int)threadIdx.x % p.tpr, p.tpr, p.D};
    float w[8];
    cols.param(p.weight, 1.f, w);
    int slot = 0;
    const long step = (long)gridDim.x * per;
    long row = min((long)blockIdx.x * per + sub, p.rows - 1);
    Raw<T, VECTOR> xr = cols.template fetch<T>(p.x, row), gr = cols.template fetch<T>(p.gate, row);
    for (long r0 = (long)blockIdx.x * per; r0 < p.rows; r0 += step, slot ^= 1) {
        const long at = row * p.D;
        const bool live = r0 + sub < p.rows;
        float x[8], g[8], sq[1] = {0.f};
        cols.template widen<T>(xr, x);
        cols.template widen<T>(gr, g);
        row = min(r0 + step + sub, p.rows - 1);
        if (r0 + step < p.rows) {
            xr = cols.template fetch<T>(p.x, row);
            gr = cols.template fetch<T>(p.gate, row);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sq[0] = fmaf(x[i], x[i], sq[0]);
        row_sum<1>(cols, sq, buf, slot);
        const float r = inv_rms(sq[0], p.inv_d, p.eps);
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
template <typename T, bool VECTOR, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? kGatedBlocks : 1)
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
    const long step = (long)gridDim.x * per;
    long row = min((long)blockIdx.x * per + sub, p.rows - 1);
    Raw<T, VECTOR> xr = cols.template fetch<T>(p.x, row), gr = cols.template fetch<T>(p.gate, row),
                   dr = cols.template fetch<T>(p.dout, row);
    for (long r0 = (long)blockIdx.x * per; r0 < p.rows; r0 += step, slot ^= 1) {
        const long at = row * p.D;
        const bool live = r0 + sub < p.rows;
        float x[8], g[8], d[8], s[8], sum[2] = {0.f, 0.f};
        cols.template widen<T>(xr, x);
        cols.template widen<T>(gr, g);
        cols.template widen<T>(dr, d);
        row = min(r0 + step + sub, p.rows - 1);
        if (r0 + step < p.rows) {
            xr = cols.template fetch<T>(p.x, row);
            gr = cols.template fetch<T>(p.gate, row);
            dr = cols.template fetch<T>(p.dout, row);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[i] = sigmoid(g[i]);
            sum[0] = fmaf(x[i], x[i], sum[0]);
            sum[1] = fmaf(d[i] * w[i] * g[i] * s[i], x[i], sum[1]);
        }
        row_sum<2>(cols, sum, buf, slot);
        const float r = inv_rms(sum[0], p.inv_d, p.eps);
        const float mean = sum[1] * r * p.inv_d;   // mean(q n)
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
    float eps, inv_d;
};

// T: block output, its norm and their cotangents; TR: the residual stream.
template <typename T, typename TR, bool VECTOR, bool POST, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 512 ? 2 : 1)
residual_fwd_kernel(const __grid_constant__ Residual p) {
    __shared__ float buf[2][32][1];
    const int per = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr;
    const Cols<VECTOR> cols{(int)threadIdx.x % p.tpr, p.tpr, p.D};
    float w[8], sc[8], po[8];
    cols.param(p.weight, 1.f, w);
    cols.param(p.scale, 1.f, sc);
    if (POST) cols.param(p.post, 1.f, po);
    int slot = 0;
    const long step = (long)gridDim.x * per;
    long row = min((long)blockIdx.x * per + sub, p.rows - 1);
    Raw<T, VECTOR> xr = cols.template fetch<T>(p.x, row);
    Raw<TR, VECTOR> hr = cols.template fetch<TR>(p.residual, row);
    for (long r0 = (long)blockIdx.x * per; r0 < p.rows; r0 += step) {
        const long at = row * p.D;
        const bool live = r0 + sub < p.rows;
        float x[8], h[8], sq[1] = {0.f};
        cols.template widen<T>(xr, x);
        cols.template widen<TR>(hr, h);
        row = min(r0 + step + sub, p.rows - 1);
        if (r0 + step < p.rows) {
            xr = cols.template fetch<T>(p.x, row);
            hr = cols.template fetch<TR>(p.residual, row);
        }
        if (POST) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sq[0] = fmaf(x[i], x[i], sq[0]);
            row_sum<1>(cols, sq, buf, slot);
            slot ^= 1;
            const float r = inv_rms(sq[0], p.inv_d, p.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * po[i];
            sq[0] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // the norm reads the stream as it is stored, which is what the backward sees
            h[i] = to_f(from_f<TR>(fmaf(x[i], sc[i], h[i])));
            sq[0] = fmaf(h[i], h[i], sq[0]);
        }
        if (live) cols.store(static_cast<TR*>(p.h) + at, h);
        row_sum<1>(cols, sq, buf, slot);
        slot ^= 1;
        const float r = inv_rms(sq[0], p.inv_d, p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = h[i] * r * w[i];
        if (live) cols.store(static_cast<T*>(p.out) + at, h);
    }
}

// Backward, from h as the forward stored it.  With m = h r(h):
//   tot = dh + r(h) (dy w - m mean(dy w m)),  dresidual = tot,  dweight = sum dy m,
//   dscale = sum tot u,  du = scale tot,
//   dx = du, or with n = x r(x), u = n w_post:  r(x) (du w_post - n mean(du w_post n)),
//   dpost = sum du n.
template <typename T, typename TR, bool VECTOR, bool POST, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? kResidualBlocks : 1)
residual_bwd_kernel(const __grid_constant__ Residual p) {
    __shared__ float buf3[2][32][3];
    __shared__ float buf1[2][32][1];
    extern __shared__ float smem[];
    const int per = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr;
    const Cols<VECTOR> cols{(int)threadIdx.x % p.tpr, p.tpr, p.D};
    float acc[3][8];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[k][i] = 0.f;
    int slot = 0;
    const long step = (long)gridDim.x * per;
    long row = min((long)blockIdx.x * per + sub, p.rows - 1);
    Raw<T, VECTOR> xr = cols.template fetch<T>(p.x, row), dr = cols.template fetch<T>(p.dy, row);
    Raw<TR, VECTOR> hr = cols.template fetch<TR>(p.h_in, row), gr = cols.template fetch<TR>(p.dh ? p.dh : p.h_in, row);
    for (long r0 = (long)blockIdx.x * per; r0 < p.rows; r0 += step, slot ^= 1) {
        const long at = row * p.D;
        const bool live = r0 + sub < p.rows;
        float x[8], h[8], d[8], g[8], sum[3] = {0.f, 0.f, 0.f};
        cols.template widen<T>(xr, x);
        cols.template widen<TR>(hr, h);
        cols.template widen<T>(dr, d);
        cols.template widen<TR>(gr, g);
        row = min(r0 + step + sub, p.rows - 1);
        if (r0 + step < p.rows) {
            xr = cols.template fetch<T>(p.x, row);
            hr = cols.template fetch<TR>(p.h_in, row);
            dr = cols.template fetch<T>(p.dy, row);
            gr = cols.template fetch<TR>(p.dh ? p.dh : p.h_in, row);
        }
        if (!p.dh)
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = 0.f;
        // the parameters come from L1 each time: registers for them would halve the rows in flight
        float w[8];
        cols.param(p.weight, 1.f, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum[0] = fmaf(h[i], h[i], sum[0]);
            sum[1] = fmaf(d[i] * w[i], h[i], sum[1]);
            if (POST) sum[2] = fmaf(x[i], x[i], sum[2]);
        }
        row_sum<3>(cols, sum, buf3, slot);
        const float r = inv_rms(sum[0], p.inv_d, p.eps);
        const float mean = sum[1] * r * p.inv_d;
        const float rx = POST ? inv_rms(sum[2], p.inv_d, p.eps) : 1.f;
        float q[1] = {0.f}, sc[8], po[8];
        cols.param(p.scale, 1.f, sc);
        cols.param(POST ? p.post : nullptr, 1.f, po);
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
            row_sum<1>(cols, q, buf1, slot);
            const float mq = q[0] * p.inv_d;
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
// Blocks of the forward: a few for each SM, which walk the rows.
inline long fwd_blocks(long rows, int tpr) {
    const int threads = block_threads(tpr);
    const long want = (long)kSMs * (threads >= 1024 ? 2 : 2048 / threads), need = ceil_div(rows, threads / tpr);
    return need < want ? need : want;
}
// Blocks of the backward: each walks several rows and leaves one row of partial sums.
inline long bwd_blocks(long rows, int D, int per_sm) {
    const int tpr = row_threads(D), threads = block_threads(tpr);
    const long want = (long)kSMs * (threads <= 256 ? per_sm * 256 / threads : 1);
    const long need = ceil_div(rows, threads / tpr);
    return need < want ? need : want;
}

}  // namespace norm
}  // namespace comba
