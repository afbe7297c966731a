// Selective state space scan: per channel c a diagonal state of N entries, read and
// written through token-dependent B_t and C_t shared by the channels of a group,
//
//   delta = softplus(dt + dt_bias),  a = exp(delta A),  A = -exp(A_log)
//   h_t = a h_{t-1} + delta x_t B_t,   y_t = sum_n h_t C_t + D x_t,   out_t = y_t silu(z_t)
//
// (the discretisation of comba_chunk_fwd_gated, per channel and state entry instead of per
// head).  A thread holds 4 neighbouring entries of one channel's state in registers and
// N / 4 neighbouring lanes hold a channel.
#pragma once

#include "block_common.cuh"

namespace comba {
namespace scan {

using namespace blk;

constexpr int kThreads = 128;
constexpr int kSub = 8;          // tokens between two stored states of the backward
constexpr float kLog2e = 1.44269504088896340736f;

struct Params {
    const void *x, *dt, *Bm, *Cm, *z, *dout;
    const float *A_log, *D, *dt_bias, *h0, *dh_final;
    void *out, *dx, *ddt, *dz;
    float *h_final, *dh0;
    float* ckpt;                 // [slots, C, N]: the state before every kSub-th token of a sequence
    float* part_bc;              // [channel blocks, tokens, 2, N]
    double* part_a;              // [sequences, C, N]
    double* part_d;              // [sequences, 2, C]: dD and ddt_bias
    Seqs seq;
    int C, G, N;
    int* status;
};

// 2^v for v <= 0 by the hardware's approximation (relative error 2^-22).
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Pairs of fp32 values in a 64-bit register: one instruction for two products or sums, so
// that the issue slots do not bound the state's update.
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
__device__ __forceinline__ Pair exp2_pair(Pair v) {
    float a, b;
    unpair(v, a, b);
    return pair(exp2_fast(a), exp2_fast(b));
}
// NP / 2 pairs at p (16-byte aligned for NP >= 4).
template <int NP>
__device__ __forceinline__ void load_pairs(const float* p, Pair (&v)[NP / 2]) {
    if constexpr (NP % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NP / 4; ++i) {
            const ulonglong2 u = reinterpret_cast<const ulonglong2*>(p)[i];
            v[2 * i] = u.x;
            v[2 * i + 1] = u.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) v[i] = reinterpret_cast<const Pair*>(p)[i];
    }
}

template <int NP>
__device__ __forceinline__ void store_pairs(float* p, const Pair (&v)[NP / 2]) {
    if constexpr (NP % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NP / 4; ++i) reinterpret_cast<ulonglong2*>(p)[i] = make_ulonglong2(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) reinterpret_cast<Pair*>(p)[i] = v[i];
    }
}

// Slot of the stored state of sub-chunk k of sequence n that starts at token s: a sequence
// of l tokens has ceil(l / kSub) of them, and s / kSub + n leaves room for them before the
// next sequence's.
__host__ __device__ inline long ckpt_slot(long s, int n, long k) { return s / kSub + n + k; }
inline long ckpt_slots(const Seqs& q) { return q.tokens() / kSub + q.N + 1; }

// Where a thread stands: its channel (of group g) and its first state entry.
template <int LPC>
struct Place {
    int c, g, n0;
    bool on;
    __device__ __forceinline__ Place(const Params& p) {
        constexpr int CB = kThreads / LPC;
        const int cpg = p.C / p.G, bpg = (cpg + CB - 1) / CB;
        g = blockIdx.x / bpg;
        const int i = (blockIdx.x % bpg) * CB + threadIdx.x / LPC;
        on = i < cpg;
        c = g * cpg + (on ? i : 0);
        n0 = (threadIdx.x % LPC) * 4;
    }
};

template <int LPC>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = 1; o < LPC; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of M values over the M lanes (M a power of two) that differ in lane bits [S, S * M):
// the lane whose those bits are r ends with the sum of v[r] in v[0].  M - 1 shuffles, each
// halving the values a lane still holds, instead of M log2 M.
template <int M, int S>
__device__ __forceinline__ void transpose_sum(float (&v)[M], int lane) {
#pragma unroll
    for (int w = M / 2; w > 0; w /= 2) {
        const bool up = lane & (w * S);
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float keep = up ? v[i + w] : v[i], send = up ? v[i] : v[i + w];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, w * S);
        }
    }
}

// Tokens of a tile: what a block stages in shared memory at a time.
__host__ __device__ constexpr int tile_tokens(int lpc) { return lpc == 1 ? 8 : lpc <= 16 ? 16 : 32; }

// One block per (channel block, sequence), tokens in order, a tile at a time.  NP state
// entries a thread, LPC lanes a channel.
//
// A tile passes through three phases.  (1) Each of its (token, channel) pairs has one
// thread, which forms delta and delta x for all the channel's lanes; B and C become fp32 in
// shared memory.  (2) The lanes walk the tile's tokens, with only the state's own chain
// between them, and sum y over a channel's lanes for LPC tokens at a time.  (3) The
// pair's thread adds D x, applies the gate and stores.  The next tile's loads are in
// flight during (2).
// The exponentials bound it (16 a clock and SM), then the issue slots.
// CKPT: no outputs, but the state before every kSub-th token (the backward's first sweep).
template <typename T, int NP, int LPC, bool CKPT>
__global__ void __launch_bounds__(kThreads)
fwd_kernel(const __grid_constant__ Params p) {
    constexpr int N = NP * LPC, TT = tile_tokens(LPC), CB = kThreads / LPC, EL = TT / LPC;
    constexpr int QUADS = TT * N / 4;                         // of B, and as many of C
    constexpr int QP = (2 * QUADS + kThreads - 1) / kThreads;
    __shared__ float2 du_s[TT][CB];                           // delta, delta x
    __shared__ __align__(16) float bc_s[2][TT][N];
    __shared__ float y_s[TT][CB + 8];
    const int n = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    long s, e;
    if (!p.seq.bounds(n, s, e)) {
        if (blockIdx.x == 0 && tid == 0) atomicCAS(p.status, 0, COMBA_EINVAL);
        return;
    }
    const int cpg = p.C / p.G, bpg = (cpg + CB - 1) / CB;
    const int g = blockIdx.x / bpg, c0 = (blockIdx.x % bpg) * CB;   // first channel within the group
    // as a lane of the scan: channel and first state entry
    const bool on = c0 + tid / LPC < cpg;
    const int c = g * cpg + (on ? c0 + tid / LPC : 0), n0 = (tid % LPC) * NP;
    const long hrow = ((long)n * p.C + c) * N + n0;
    Pair A2[NP / 2], h[NP / 2];
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) {
        const float* a = p.A_log + (long)c * N + n0 + 2 * i;
        A2[i] = pair(-expf(a[0]) * kLog2e, -expf(a[1]) * kLog2e);
        h[i] = p.h0 ? pair(p.h0[hrow + 2 * i], p.h0[hrow + 2 * i + 1]) : pair(0.f, 0.f);
    }
    // as the thread of (token, channel) pairs: channel pc, tokens pt, pt + LPC, ...
    const int pi = tid % CB, pt = tid / CB;
    const bool pon = c0 + pi < cpg;
    const int pc = g * cpg + (pon ? c0 + pi : 0);
    const float bias = p.dt_bias ? p.dt_bias[pc] : 0.f;
    const float D = p.D ? p.D[pc] : 0.f;

    T xr[EL], dr[EL], zr[EL];
    float br[QP][4];
    auto fetch = [&](long t0) {
#pragma unroll
        for (int k = 0; k < EL; ++k) {
            const long t = t0 + pt + k * LPC;
            const bool ok = pon && t < e;
            const long o = t * p.C + pc;
            xr[k] = ok ? static_cast<const T*>(p.x)[o] : from_f<T>(0.f);
            dr[k] = ok ? static_cast<const T*>(p.dt)[o] : from_f<T>(0.f);
            if (!CKPT && p.z) zr[k] = ok ? static_cast<const T*>(p.z)[o] : from_f<T>(0.f);
        }
#pragma unroll
        for (int k = 0; k < QP; ++k) {
            const int q = tid + k * kThreads, which = q / QUADS, r = q % QUADS;
            const long t = t0 + r / (N / 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) br[k][i] = 0.f;
            if (which < (CKPT ? 1 : 2) && t < e)
                load_v<4>(static_cast<const T*>(which ? p.Cm : p.Bm) + (t * p.G + g) * N + r % (N / 4) * 4, br[k]);
        }
    };
    fetch(s);
    for (long t0 = s; t0 < e; t0 += TT) {
        float x[EL], z[EL];
#pragma unroll
        for (int k = 0; k < EL; ++k) {
            const int j = pt + k * LPC;
            x[k] = to_f(xr[k]);
            if (!CKPT && p.z) z[k] = to_f(zr[k]);
            // past the end: delta = 0 leaves the state as it is
            const float delta = t0 + j < e ? softplus(to_f(dr[k]) + bias) : 0.f;
            du_s[j][pi] = make_float2(delta, delta * x[k]);
        }
#pragma unroll
        for (int k = 0; k < QP; ++k) {
            const int q = tid + k * kThreads;
            if (q < 2 * QUADS) store_v<4>(&bc_s[0][0][0] + q * 4, br[k]);
        }
        __syncthreads();
        if (t0 + TT < e) fetch(t0 + TT);
#pragma unroll
        for (int j0 = 0; j0 < TT; j0 += LPC) {
            float y[LPC];
#pragma unroll
            for (int jj = 0; jj < LPC; ++jj) {
                const int j = j0 + jj;
                if (CKPT && j % kSub == 0 && on && t0 + j < e) {
                    store_pairs<NP>(p.ckpt + (ckpt_slot(s, n, (t0 - s + j) / kSub) * p.C + c) * N + n0, h);
                }
                const float2 du = du_s[j][tid / LPC];
                const Pair dl = pair(du.x, du.x), u = pair(du.y, du.y);
                Pair b[NP / 2], cc[NP / 2], acc;
                load_pairs<NP>(&bc_s[0][j][n0], b);
                if (!CKPT) load_pairs<NP>(&bc_s[1][j][n0], cc);
#pragma unroll
                for (int i = 0; i < NP / 2; ++i) {
                    h[i] = fma2(exp2_pair(mul2(dl, A2[i])), h[i], mul2(u, b[i]));
                    if (!CKPT) acc = i == 0 ? mul2(h[i], cc[i]) : fma2(h[i], cc[i], acc);
                }
                if (!CKPT) {
                    float lo, hi;
                    unpair(acc, lo, hi);
                    y[jj] = lo + hi;
                }
            }
            if (!CKPT) {
                transpose_sum<LPC, 1>(y, lane);
                y_s[j0 + tid % LPC][tid / LPC] = y[0];
            }
        }
        __syncthreads();
        if (!CKPT) {
#pragma unroll
            for (int k = 0; k < EL; ++k) {
                const int j = pt + k * LPC;
                if (!pon || t0 + j >= e) continue;
                float y = fmaf(D, x[k], y_s[j][pi]);
                if (p.z) y *= silu(z[k]);
                static_cast<T*>(p.out)[(t0 + j) * p.C + pc] = from_f<T>(y);
            }
        }
    }
    if (!CKPT && p.h_final && on) store_pairs<NP>(p.h_final + hrow, h);
}

// Backward: the tokens of a sequence in reverse, kSub at a time.  From the stored state
// before a sub-chunk, its decays a and decayed states q = a h_{t-1} are formed again and
// kept in registers (h_t = q + delta x B); then, with g the state's gradient,
//   dy = dout silu(z),  dz = dout y silu'(z),  g += C dy,
//   dC = sum_c h dy,  dB = sum_c g delta x,  du = sum_n g B,
//   ddelta = sum_n g q A + du x,  dA_log = A sum g q delta,
//   dx = du delta + D dy,  ddt = ddelta sigmoid(dt + dt_bias),  g <- a g.
// Sums over a channel's entries go over its lanes; dB and dC are summed over the block's
// channels and leave one row per channel block.
template <typename T, int LPC>
__global__ void __launch_bounds__(kThreads)
bwd_kernel(const __grid_constant__ Params p) {
    constexpr int N = LPC * 4, WARPS = kThreads / 32;
    __shared__ float bc[WARPS][kSub][2][N];
    const Place<LPC> at(p);
    const int n = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long s, e;
    if (!p.seq.bounds(n, s, e)) return;   // reported by the first sweep
    const long tokens = p.seq.tokens();
    float A2[4], g[4] = {0.f, 0.f, 0.f, 0.f};
    load_v<4>(p.A_log + (long)at.c * N + at.n0, A2);
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] = -expf(A2[i]) * kLog2e;
    const long hrow = ((long)n * p.C + at.c) * N + at.n0;
    if (p.dh_final && at.on) load_v<4>(p.dh_final + hrow, g);
    const float bias = p.dt_bias ? p.dt_bias[at.c] : 0.f;
    const float D = p.D ? p.D[at.c] : 0.f;
    const T* Bm = static_cast<const T*>(p.Bm) + (long)at.g * N + at.n0;
    const T* Cm = static_cast<const T*>(p.Cm) + (long)at.g * N + at.n0;
    double dA[4] = {0.0, 0.0, 0.0, 0.0}, dD = 0.0, dbias = 0.0;
    for (long k = (e - s + kSub - 1) / kSub - 1; k >= 0; --k) {
        const long t0 = s + k * kSub;
        const int len = (int)min((long)kSub, e - t0);
        float a[kSub][4], q[kSub][4], dl[kSub], xs[kSub], dyv[kSub], zv[kSub], yv[kSub], dov[kSub];
        float h[4];
        load_v<4>(p.ckpt + (ckpt_slot(s, n, k) * p.C + at.c) * N + at.n0, h);
#pragma unroll
        for (int j = 0; j < kSub; ++j) {
            const bool live = at.on && j < len;
            const long o = (t0 + j) * p.C + at.c;
            xs[j] = live ? to_f(static_cast<const T*>(p.x)[o]) : 0.f;
            dl[j] = live ? softplus(to_f(static_cast<const T*>(p.dt)[o]) + bias) : 0.f;
            dov[j] = live ? to_f(static_cast<const T*>(p.dout)[o]) : 0.f;
            zv[j] = live && p.z ? to_f(static_cast<const T*>(p.z)[o]) : 0.f;
            dyv[j] = p.z ? dov[j] * silu(zv[j]) : dov[j];
            const float u = dl[j] * xs[j];
            float b[4] = {0.f, 0.f, 0.f, 0.f}, c[4] = {0.f, 0.f, 0.f, 0.f}, y = 0.f;
            if (j < len) {
                load_v<4>(Bm + (t0 + j) * p.G * N, b);
                load_v<4>(Cm + (t0 + j) * p.G * N, c);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[j][i] = exp2_fast(dl[j] * A2[i]);
                q[j][i] = a[j][i] * h[i];
                h[i] = fmaf(u, b[i], q[j][i]);
                y = fmaf(h[i], c[i], y);
            }
            yv[j] = lanes_sum<LPC>(y);
        }
        float dAk[4] = {0.f, 0.f, 0.f, 0.f}, dDk = 0.f, dbk = 0.f;
#pragma unroll
        for (int j = kSub - 1; j >= 0; --j) {
            const bool live = at.on && j < len;
            const float u = dl[j] * xs[j];
            float b[4] = {0.f, 0.f, 0.f, 0.f}, c[4] = {0.f, 0.f, 0.f, 0.f}, db[4], dc[4], du = 0.f, dd = 0.f;
            if (j < len) {
                load_v<4>(Bm + (t0 + j) * p.G * N, b);
                load_v<4>(Cm + (t0 + j) * p.G * N, c);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float ht = fmaf(u, b[i], q[j][i]);
                g[i] = fmaf(c[i], dyv[j], g[i]);
                dc[i] = ht * dyv[j];
                db[i] = g[i] * u;
                du = fmaf(g[i], b[i], du);
                const float gq = g[i] * q[j][i];
                dd = fmaf(gq, A2[i], dd);
                dAk[i] = fmaf(gq, dl[j], dAk[i]);
                g[i] *= a[j][i];
            }
            du = lanes_sum<LPC>(du);
            dd = lanes_sum<LPC>(dd) * (1.f / kLog2e);
            if (live && at.n0 == 0) {
                const long o = (t0 + j) * p.C + at.c;
                const float ddelta = fmaf(du, xs[j], dd);
                const float dv = ddelta * sigmoid(to_f(static_cast<const T*>(p.dt)[o]) + bias);
                static_cast<T*>(p.dx)[o] = from_f<T>(fmaf(du, dl[j], D * dyv[j]));
                static_cast<T*>(p.ddt)[o] = from_f<T>(dv);
                if (p.dz) static_cast<T*>(p.dz)[o] = from_f<T>(dov[j] * fmaf(D, xs[j], yv[j]) * dsilu(zv[j]));
                dDk = fmaf(dyv[j], xs[j], dDk);
                dbk += dv;
            }
            // over the warp's channels
#pragma unroll
            for (int o = LPC; o < 32; o *= 2)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
                    dc[i] += __shfl_xor_sync(0xffffffffu, dc[i], o);
                }
            if (lane < LPC)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    bc[warp][j][0][at.n0 + i] = db[i];
                    bc[warp][j][1][at.n0 + i] = dc[i];
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) dA[i] += (double)dAk[i];
        dD += (double)dDk;
        dbias += (double)dbk;
        __syncthreads();
        for (int i = threadIdx.x; i < len * 2 * N; i += kThreads) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) v += (&bc[w][0][0][0])[i];
            p.part_bc[((long)blockIdx.x * tokens + t0) * 2 * N + i] = v;
        }
        __syncthreads();
    }
    if (!at.on) return;
    if (p.dh0) store_v<4>(p.dh0 + hrow, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) p.part_a[hrow + i] = dA[i];
    if (at.n0 == 0) {
        p.part_d[((long)n * 2) * p.C + at.c] = dD;
        p.part_d[((long)n * 2 + 1) * p.C + at.c] = dbias;
    }
}

// dB and dC of a (token, group) from the group's channel blocks, in a fixed order.
template <typename T>
__global__ void __launch_bounds__(256)
sum_bc_kernel(const float* __restrict__ part, T* __restrict__ dB, T* __restrict__ dC, const Seqs seq, int G, int N, int bpg) {
    const long tokens = seq.tokens();
    const long id = (long)blockIdx.x * 256 + threadIdx.x;   // over [tokens, G, 2, N]
    const int i = (int)(id % (2 * N));
    const long tg = id / (2 * N);
    const int g = (int)(tg % G);
    const long t = tg / G;
    if (t >= tokens) return;
    if (seq.cu) {   // tokens that no sequence covers have no partial sums and keep what they hold
        long s, e;
        if (!seq.bounds(seq.find(t), s, e) || t < s || t >= e) return;
    }
    float v = 0.f;
    for (int b = 0; b < bpg; ++b) v += part[(((long)g * bpg + b) * tokens + t) * 2 * N + i];
    T* out = i < N ? dB : dC;
    out[(t * G + g) * N + (i < N ? i : i - N)] = from_f<T>(v);
}

// dA_log, dD and ddt_bias from the sequences' sums, in a fixed order.
__global__ void __launch_bounds__(256)
sum_params_kernel(const double* __restrict__ part_a, const double* __restrict__ part_d, const float* __restrict__ A_log,
                  float* __restrict__ dA_log, float* __restrict__ dD, float* __restrict__ dbias, const Seqs seq, int C, int N) {
    const long id = (long)blockIdx.x * 256 + threadIdx.x, CN = (long)C * N;
    if (id >= CN + 2 * C) return;
    const long i = id < CN ? id : id - CN;
    const double* part = id < CN ? part_a : part_d;
    const long cols = id < CN ? CN : 2 * C;
    double v = 0.0;
    for (int n = 0; n < seq.N; ++n) {
        long s, e;
        if (seq.bounds(n, s, e)) v += part[(long)n * cols + i];
    }
    if (id < CN) dA_log[i] = (float)(v * -(double)expf(A_log[i]));
    else if (i < C) { if (dD) dD[i] = (float)v; }
    else if (dbias) dbias[i - C] = (float)v;
}

// One token: the state h [B, C, N] is read and written once.
template <typename T, int LPC>
__global__ void __launch_bounds__(kThreads)
step_kernel(const __grid_constant__ Params p) {
    constexpr int N = LPC * 4;
    const Place<LPC> at(p);
    const int n = blockIdx.y;
    float* hp = p.h_final + ((long)n * p.C + at.c) * N + at.n0;
    float h[4], A[4], b[4], c[4];
    load_v<4>(hp, h);
    load_v<4>(p.A_log + (long)at.c * N + at.n0, A);
    load_v<4>(static_cast<const T*>(p.Bm) + ((long)n * p.G + at.g) * N + at.n0, b);
    load_v<4>(static_cast<const T*>(p.Cm) + ((long)n * p.G + at.g) * N + at.n0, c);
    const long o = (long)n * p.C + at.c;
    const float xv = to_f(static_cast<const T*>(p.x)[o]);
    const float delta = softplus(to_f(static_cast<const T*>(p.dt)[o]) + (p.dt_bias ? p.dt_bias[at.c] : 0.f));
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = fmaf(exp2_fast(delta * (-expf(A[i]) * kLog2e)), h[i], delta * xv * b[i]);
        y = fmaf(h[i], c[i], y);
    }
    y = lanes_sum<LPC>(y);
    if (!at.on) return;
    store_v<4>(hp, h);
    if (at.n0 == 0) {
        if (p.D) y = fmaf(p.D[at.c], xv, y);
        if (p.z) y *= silu(to_f(static_cast<const T*>(p.z)[o]));
        static_cast<T*>(p.out)[o] = from_f<T>(y);
    }
}

}  // namespace scan
}  // namespace comba
