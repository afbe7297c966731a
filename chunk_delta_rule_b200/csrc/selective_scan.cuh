// Selective state space scan: per channel c a diagonal state of N entries, read and
// written through token-dependent B_t and C_t shared by the channels of a group,
//
//   delta = softplus(dt + dt_bias),  a = exp(delta A),  A = -exp(A_log)
//   h_t = a h_{t-1} + delta x_t B_t,   y_t = sum_n h_t C_t + D x_t,   out_t = y_t silu(z_t)
//
// (the discretisation of comba_chunk_fwd_gated, per channel and state entry instead of per
// head).  A thread holds 4 neighbouring entries of one channel's state in registers, and
// neighbouring lanes hold a channel.
#pragma once

#include <float.h>

#include "block_common.cuh"

namespace comba {
namespace scan {

using namespace blk;

constexpr int kBatch = 4;        // tokens whose operands a lane holds at a time
constexpr int kSub = 8;          // tokens between two stored states of the backward

struct Params {
    const void *x, *dt, *Bm, *Cm, *z, *dout;
    const float *A_log, *D, *dt_bias, *h0, *dh_final;
    void *out, *dx, *ddt, *dz;
    float *h_final, *dh0;
    long piece;                  // split form: tokens of a piece of the joint token axis
    int pieces;
    float* ends;                 // [pieces, C, N]: state after a piece (see ends_kernel)
    float* dsum;                 // [pieces, C]: sum of delta over it
    float* back_ends;            // [pieces, C, N]: gradient of the state before a piece (see back_ends_kernel)
    float* ckpt;                 // [slots, C, N]: the state before every kSub-th token of a sequence
    float* part_bc;              // [channel blocks, tokens, 2, N]
    double* part_a;              // [sequences or pieces, C, N]
    double* part_d;              // [sequences or pieces, 2, C]: dD and ddt_bias
    Seqs seq;
    int C, G, N;
    bool vec;                    // groups of channels lie whole and aligned (see load_group)
    int* status;
};

// 2^(delta A2) for a pair of entries.  The hardware's 2^v is low by 1e-8 to 2.5e-8 on average
// for v in [-0.3, 0) (measured; its rounding is 3e-8 rms), which a slowly decaying state would
// add up over hundreds of tokens: the exponent is raised by 2.2e-8, which takes the mean error
// within 1e-8 and leaves 2^0 = 1.
__device__ __forceinline__ Pair decay_pair(Pair delta, Pair A2) {
    float a, b;
    unpair(fma2(delta, A2, pair(2.2e-8f, 2.2e-8f)), a, b);
    return pair(exp2_fast(a), exp2_fast(b));
}
// Two pairs at p, 16-byte aligned.
__device__ __forceinline__ void load_pairs(const float* p, Pair (&v)[2]) {
    const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(p);
    v[0] = u.x;
    v[1] = u.y;
}
__device__ __forceinline__ void store_pairs(float* p, const Pair (&v)[2]) {
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(v[0], v[1]);
}

// Slot of the stored state of sub-chunk k of the n-th run of tokens (a sequence, or its part in
// a piece) that starts at token s: a run of l tokens has ceil(l / kSub) of them, and
// s / kSub + n leaves room for them before the next run's.
__host__ __device__ inline long ckpt_slot(long s, int n, long k) { return s / kSub + n + k; }
inline long ckpt_slots(const Seqs& q, int pieces) { return q.tokens() / kSub + q.N + pieces + 1; }

// How the kernels lay out N state entries: NP a lane, LPC lanes a channel, NT threads a block
// (CB channels), and tiles of TT tokens, which a block stages in shared memory at a time.
// Every thread prepares one group of E consecutive channels of one token of a tile.
// Measured for N = 16, forward of B8 T4096 C2048: NP 2, 4, 8 take 668, 571, 676 us (more lanes
// repeat the operands' reads, fewer leave too few warps); NT 64, 128, 256 take 571, 571, 614 us,
// and 2.80, 1.79, 1.86 ms over 64K tokens of one sequence.  The backward prefers the same.
template <int N_>
struct Layout {
    static constexpr int N = N_, NP = 4, PP = NP / 2, LPC = N / NP, NT = 128, TT = N < 32 ? N : N < 128 ? 16 : 32;
    static constexpr int CB = NT / LPC, E = TT / LPC;
    static constexpr int YL = LPC < 4 ? LPC : 4;   // partial sums of a channel, each of LPC / YL lanes
    static_assert(E * LPC == TT && (E == 1 || E == 2 || E == 4) && CB % E == 0 && TT % 8 == 0, "one group a thread");
};

// E consecutive elements.  VEC: as one access (all such groups are whole and aligned), else
// one by one, those past the first `count` from the first one's place.  Loads carry no
// condition, so that they stay in flight until their values are needed; what lies outside
// the tile is masked there.
template <typename T, int E>
struct alignas(E * sizeof(T)) Group {
    T v[E];
};
template <bool VEC, typename T, int E>
__device__ __forceinline__ Group<T, E> load_group(const void* base, long o, int count) {
    const T* p = static_cast<const T*>(base) + o;
    if constexpr (VEC) {
        return *reinterpret_cast<const Group<T, E>*>(p);
    } else {
        Group<T, E> r;
#pragma unroll
        for (int i = 0; i < E; ++i) r.v[i] = p[i < count ? i : 0];
        return r;
    }
}
template <bool VEC, typename T, int E>
__device__ __forceinline__ void store_group(void* base, long o, const float (&f)[E], int count) {
    T* p = static_cast<T*>(base) + o;
    Group<T, E> r;
#pragma unroll
    for (int i = 0; i < E; ++i) r.v[i] = from_f<T>(f[i]);
    if constexpr (VEC) {
        *reinterpret_cast<Group<T, E>*>(p) = r;
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < count) p[i] = r.v[i];
    }
}

// Four elements of B or C, as they are stored.
template <typename T> struct Raw4;
template <> struct Raw4<float> { using type = float4; };
template <> struct Raw4<bf16> { using type = uint2; };
__device__ __forceinline__ void widen(float4 r, float (&v)[4]) { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
__device__ __forceinline__ void widen(uint2 r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x << 16); v[1] = __uint_as_float(r.x & 0xffff0000u);
    v[2] = __uint_as_float(r.y << 16); v[3] = __uint_as_float(r.y & 0xffff0000u);
}

// A thread's two places in a block: a lane of the scan (channel c, entries n0 .. n0+3), and
// the preparer of the channels gc .. gc+E-1 (of which `count` exist) of token gt of a tile.
template <class K>
struct Place {
    int g, c, n0, li;      // group, channel, entry, channel within the block
    bool on;
    int gt, gi, gc, count; // token of the tile, channel within the block, channel
    __device__ __forceinline__ Place(const Params& p) {
        const int tid = threadIdx.x, cpg = p.C / p.G, bpg = (cpg + K::CB - 1) / K::CB;
        g = blockIdx.x / bpg;
        const int c0 = (blockIdx.x % bpg) * K::CB;
        li = tid / K::LPC;
        n0 = tid % K::LPC * K::NP;
        on = c0 + li < cpg;
        c = g * cpg + (on ? c0 + li : 0);
        gt = tid / (K::CB / K::E);
        gi = tid % (K::CB / K::E) * K::E;
        count = min(max(cpg - c0 - gi, 0), K::E);
        gc = g * cpg + (count > 0 ? c0 + gi : 0);
    }
};

template <class K>
struct FwdSmem {
    float2 du[K::TT][K::CB];                 // delta, delta x
    alignas(16) float bc[2][K::TT][K::N];
    alignas(16) float y[K::TT][K::CB][K::YL];   // a channel's partial sums, of up to 4 sets of its lanes
};

// Where channel `ch` of token t lies in a row of du, and in one of partial sums: permuted
// among its group, so that the preparers (a group a thread) and the lanes (a channel each)
// both touch different banks.
template <class K>
__device__ __forceinline__ int du_slot(int t, int ch) {
    return K::E == 4 ? ch ^ (((ch >> 4) & 1) | ((t & 1) << 1)) : K::E == 2 ? ch ^ ((ch >> 4) & 1) : ch;
}
template <class K>
__device__ __forceinline__ int y_slot(int ch) {
    return K::E == 4 ? ch ^ ((ch >> (K::YL == 2 ? 4 : 3)) & 3) : K::E == 2 ? ch ^ ((ch >> 3) & 1) : ch;
}
// Sums v over the lanes of a channel that share one of its YL partial sums.
template <class K>
__device__ __forceinline__ float set_sum(float v) {
#pragma unroll
    for (int o = K::LPC / K::YL / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <class K>
__device__ __forceinline__ int set_of(int tid) { return tid % K::LPC / (K::LPC / K::YL); }

enum Mode {
    kOutputs,   // out
    kStates,    // no outputs, but the state before every kSub-th token (the backward's first sweep)
    kEnds       // no outputs, only the state after the last token (the split form's first sweep)
};

// Tokens [from, to), the n-th run of tokens (see ckpt_slot), from and to the state h of the
// block's lanes, a tile at a time.
//
// A tile passes through three phases.  (1) Each (token, channel) has one thread, which forms
// delta and delta x for all the channel's lanes, 4 channels at a time; B and C become fp32 in
// shared memory.  (2) The lanes walk the tile's tokens, with only the state's own chain
// between them.  (3) The first phase's thread sums y over the lanes, adds D x, applies the
// gate and stores.  The next tile's loads are in flight during (2).
//
// What bounds it: the exponentials, 16 of the state and 5 of softplus and silu a (token,
// channel) at N = 16, of which an SM does 16 a clock: 303 us for B8 T4096 C2048, against 83 us
// for its bytes.  Measured: 569 us, with that unit 59 % busy, the shared-memory pipe 63 %, the
// issue slots 51 %; a block's own chain of phases leaves them idle, and the registers and the
// 3.5 blocks an SM has do not fill the gaps.
template <typename T, class K, Mode M, bool VEC>
__device__ __forceinline__ void walk(const Params& p, FwdSmem<K>& sm, const Place<K>& at, int n, long from,
                                     long to, const Pair (&A2)[K::PP], Pair (&h)[K::PP], float& dsum) {
    constexpr int N = K::N, TT = K::TT, E = K::E, PP = K::PP;
    constexpr int QUADS = TT * N / 4, QP = (2 * QUADS + K::NT - 1) / K::NT;   // of B and C
    if (from >= to) return;   // fetch() needs a last token to clamp to
    const int tid = threadIdx.x, ys = y_slot<K>(at.li);
    float bias[E], D[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = p.dt_bias && i < at.count ? p.dt_bias[at.gc + i] : 0.f;
        D[i] = M == kOutputs && p.D && i < at.count ? p.D[at.gc + i] : 0.f;
    }
    Group<T, E> xr, dr, zr;
    typename Raw4<T>::type br[QP];
    const bool gated = M == kOutputs && p.z;
    auto fetch = [&](long t0) {
        const long o = min(t0 + at.gt, to - 1) * p.C + at.gc;
        xr = load_group<VEC, T, E>(p.x, o, at.count);
        dr = load_group<VEC, T, E>(p.dt, o, at.count);
        if (M == kOutputs) zr = load_group<VEC, T, E>(gated ? p.z : p.x, o, at.count);
        const long ahead = min(t0 + 2 * TT + at.gt, to - 1) * p.C + at.gc;
        prefetch_l2(static_cast<const T*>(p.x) + ahead);
        prefetch_l2(static_cast<const T*>(p.dt) + ahead);
        if (gated) prefetch_l2(static_cast<const T*>(p.z) + ahead);
#pragma unroll
        for (int k = 0; k < QP; ++k) {
            const int q = tid + k * K::NT, r = q % QUADS;
            const long tb = min(t0 + r / (N / 4), to - 1);
            br[k] = *reinterpret_cast<const typename Raw4<T>::type*>(
                static_cast<const T*>(M == kOutputs && q >= QUADS ? p.Cm : p.Bm) + (tb * p.G + at.g) * N + r % (N / 4) * 4);
        }
    };
    fetch(from);
    for (long t0 = from; t0 < to; t0 += TT) {
        const bool live = t0 + at.gt < to;
        const Group<T, E> x = xr, z = zr;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            // past the end: delta = 0 and delta x = 0 leave the state as it is
            const float delta = softplus(to_f(dr.v[i]) + bias[i]);
            sm.du[at.gt][du_slot<K>(at.gt, at.gi + i)] = live ? make_float2(delta, delta * to_f(x.v[i])) : make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < QP; ++k) {
            const int q = tid + k * K::NT;
            float v[4];
            widen(br[k], v);
            const bool in = t0 + q % QUADS / (N / 4) < to;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = in ? v[i] : 0.f;
            if (q < 2 * QUADS) store_v<4>(&sm.bc[0][0][0] + q * 4, v);
        }
        __syncthreads();
        if (t0 + TT < to) fetch(t0 + TT);
        // kBatch tokens at a time: their operands are read, and their decays and inputs formed,
        // before the previous batch's y is stored (a store would hold back later loads)
        float2 du[kBatch];
        Pair b[kBatch][PP], c[kBatch][PP];
        auto operands = [&](int j0) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                du[j] = sm.du[j0 + j][du_slot<K>(j0 + j, at.li)];
                load_pairs(&sm.bc[0][j0 + j][at.n0], b[j]);
            }
        };
        operands(0);
#pragma unroll
        for (int j0 = 0; j0 < TT; j0 += kBatch) {
            Pair a[kBatch][PP];
            float y[kBatch], dl[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                dl[j] = du[j].x;
                const Pair d2 = pair(du[j].x, du[j].x), u = pair(du[j].y, du[j].y);
#pragma unroll
                for (int i = 0; i < PP; ++i) {
                    a[j][i] = decay_pair(d2, A2[i]);
                    b[j][i] = mul2(u, b[j][i]);
                }
                if (M == kOutputs) load_pairs(&sm.bc[1][j0 + j][at.n0], c[j]);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (M == kStates && (j0 + j) % kSub == 0 && at.on && t0 + j0 + j < to)
                    store_pairs(p.ckpt + (ckpt_slot(from, n, (t0 - from + j0 + j) / kSub) * p.C + at.c) * N + at.n0, h);
                Pair acc;
#pragma unroll
                for (int i = 0; i < PP; ++i) {
                    h[i] = fma2(a[j][i], h[i], b[j][i]);
                    if (M == kOutputs) acc = i ? fma2(h[i], c[j][i], acc) : mul2(h[i], c[j][i]);
                }
                if (M == kEnds) dsum += dl[j];
                if (M == kOutputs) {
                    float lo, hi;
                    unpair(acc, lo, hi);
                    y[j] = set_sum<K>(lo + hi);
                }
            }
            if (j0 + kBatch < TT) operands(j0 + kBatch);
            if (M == kOutputs)
#pragma unroll
                for (int j = 0; j < kBatch; ++j) sm.y[j0 + j][ys][set_of<K>(tid)] = y[j];
        }
        __syncthreads();
        if (M == kOutputs && live && at.count > 0) {
            float y[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float* l = sm.y[at.gt][y_slot<K>(at.gi + i)];
                y[i] = l[0] + l[1];
#pragma unroll
                for (int k = 2; k < K::YL; k += 2) y[i] += l[k] + l[k + 1];
                y[i] = fmaf(D[i], to_f(x.v[i]), y[i]);
                if (gated) y[i] *= silu(to_f(z.v[i]));
            }
            store_group<VEC, T, E>(p.out, (t0 + at.gt) * p.C + at.gc, y, at.count);
        }
    }
}

// A log2(e), and -1e30 where that overflows: every delta from 1.5e-28 on gives a decay of 0 all
// the same, delta = 0 (dt = -inf, tokens past the end) one of 1 instead of 0 * inf, and at those
// tokens the backward's sum of g q A, which their sigmoid of 0 takes away, stays finite.
template <class K>
__device__ __forceinline__ void load_decays(const Params& p, const Place<K>& at, Pair (&A2)[K::PP]) {
    float a[K::NP];
    load_v<K::NP>(p.A_log + (long)at.c * K::N + at.n0, a);
#pragma unroll
    for (int i = 0; i < K::NP; ++i) {
        a[i] = -expf(a[i]) * kLog2e;
        a[i] = a[i] < -FLT_MAX ? -1e30f : a[i];   // NaN stays
    }
#pragma unroll
    for (int i = 0; i < K::PP; ++i) A2[i] = pair(a[2 * i], a[2 * i + 1]);
}

// One block per (channel block, sequence).
template <typename T, class K, Mode M, bool VEC>
__global__ void __launch_bounds__(K::NT)
fwd_kernel(const __grid_constant__ Params p) {
    __shared__ FwdSmem<K> sm;
    const Place<K> at(p);
    const int n = blockIdx.y;
    long s, e;
    if (!p.seq.bounds(n, s, e)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(p.status, 0, COMBA_EINVAL);
        return;
    }
    const long hrow = ((long)n * p.C + at.c) * K::N + at.n0;
    Pair A2[K::PP], h[K::PP] = {};
    float dsum;
    load_decays<K>(p, at, A2);
    if (p.h0) load_pairs(p.h0 + hrow, h);
    walk<T, K, M, VEC>(p, sm, at, n, s, e, A2, h, dsum);
    if (M == kOutputs && p.h_final && at.on) store_pairs(p.h_final + hrow, h);
}

// The split form, for too few (channel block, sequence) pairs to fill the GPU: the joint
// token axis is cut into pieces, which run as blocks of their own.  Over a piece, a channel's
// entry goes from h to exp(A sum delta) h + r.
//
// First sweep: for a piece that ends inside a sequence, r from that sequence's tokens in it
// (from h0 where the sequence starts there, so that r is the state itself) and sum delta.
template <typename T, class K, bool VEC>
__global__ void __launch_bounds__(K::NT)
ends_kernel(const __grid_constant__ Params p) {
    __shared__ FwdSmem<K> sm;
    const Place<K> at(p);
    const long t0 = blockIdx.y * p.piece, t1 = min(t0 + p.piece, p.seq.tokens());
    const int n = p.seq.find(t1 - 1);
    long s, e;
    if (!p.seq.bounds(n, s, e) || s >= t1 || e <= t1) return;
    Pair A2[K::PP], h[K::PP] = {};
    float dsum = 0.f;
    load_decays<K>(p, at, A2);
    if (s >= t0 && p.h0) load_pairs(p.h0 + ((long)n * p.C + at.c) * K::N + at.n0, h);
    walk<T, K, kEnds, VEC>(p, sm, at, n, max(s, t0), t1, A2, h, dsum);
    if (!at.on) return;
    const long row = (long)blockIdx.y * p.C + at.c;
    store_pairs(p.ends + row * K::N + at.n0, h);
    if (at.n0 == 0) p.dsum[row] = dsum;
}

// Second sweep: every piece again, each sequence in it from its start state, which the
// block composes from the pieces before it.  (kStates: the same for the backward's first sweep.)
template <typename T, class K, Mode M, bool VEC>
__global__ void __launch_bounds__(K::NT)
split_kernel(const __grid_constant__ Params p) {
    constexpr int N = K::N;
    __shared__ FwdSmem<K> sm;
    const Place<K> at(p);
    const int j = blockIdx.y;
    for (int n = j; n < p.seq.N; n += p.pieces) {   // sequences without tokens, and bad bounds
        long s, e;
        const bool ok = p.seq.bounds(n, s, e);
        if (!ok && blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(p.status, 0, COMBA_EINVAL);
        if (!ok || s < e || M != kOutputs || !p.h_final || !at.on) continue;
        Pair h[K::PP] = {};
        const long hrow = ((long)n * p.C + at.c) * N + at.n0;
        if (p.h0) load_pairs(p.h0 + hrow, h);
        store_pairs(p.h_final + hrow, h);
    }
    Pair A2[K::PP];
    float dsum;
    load_decays<K>(p, at, A2);
    const long t0 = j * p.piece, t1 = min(t0 + p.piece, p.seq.tokens());
    long t = t0;
    for (int n = p.seq.find(t0); n < p.seq.N && t < t1; ++n) {
        long s, e;
        if (!p.seq.bounds(n, s, e) || e <= t) continue;
        if (s >= t1) break;
        t = max(t, s);
        const long hrow = ((long)n * p.C + at.c) * N + at.n0, stop = min(e, t1);
        Pair h[K::PP] = {};
        if (t == s) {
            if (p.h0) load_pairs(p.h0 + hrow, h);
        } else {
            const int j0 = (int)(s / p.piece);
            load_pairs(p.ends + ((long)j0 * p.C + at.c) * N + at.n0, h);
#pragma unroll 4
            for (int i = j0 + 1; i < j; ++i) {
                const long row = (long)i * p.C + at.c;
                const float ds = p.dsum[row];
                Pair r[K::PP];
                load_pairs(p.ends + row * N + at.n0, r);
#pragma unroll
                for (int k = 0; k < K::PP; ++k) h[k] = fma2(decay_pair(pair(ds, ds), A2[k]), h[k], r[k]);
            }
        }
        walk<T, K, M, VEC>(p, sm, at, n + j, t, stop, A2, h, dsum);
        if (M == kOutputs && stop == e && p.h_final && at.on) store_pairs(p.h_final + hrow, h);
        t = stop;
    }
}

// Backward: the tokens of a sequence in reverse, in the forward's tiles and phases, kSub
// tokens of the lanes' walk at a time.  From the stored state before those, their decays a
// and decayed states q = a h_{t-1} are formed again and kept in registers (h_t = q + delta x
// B); then, with g the state's gradient,
//   dy = dout silu(z),  dz = dout y silu'(z),  g += C dy,
//   dC = sum_c h dy,  dB = sum_c g delta x,  du = sum_n g B,
//   ddelta = sum_n g q A + du x,  dA_log = A sum g q delta,
//   dx = du delta + D dy,  ddt = ddelta sigmoid(dt + dt_bias),  g <- a g.
// y, du and ddelta's first part are summed over a channel's lanes by the preparers.  dB and
// dC are summed over a warp's channels by halving shuffles, over the block's warps through
// shared memory, and leave one row per channel block: 2 N values for 512 / N channels, C N^2 / 64
// bytes a token to write and read again (B8 T2048 C1024, N = 16, 32, 64, 128: 661 us, 1.17, 2.65,
// 6.43 ms).
//
// What bounds it: latency, with the 8 warps that an SM's registers hold at 248 a thread; the
// issue slots are 47 % busy with 115 instructions for a token of 8 channels, 28 of which sum dB
// and dC over the channels.  Measured with the sweep that stores the states: 661 us for B8 T2048
// C1024 N16 (bf16), 1.24 ms for C2048.  Storing a state every kSub = 8 tokens costs 8 bytes a
// (token, channel) each way, and spares a third sweep's exponentials.
constexpr int kFlush = 16;
constexpr int kBwdBlocks = 2;   // that an SM's registers hold: 3 would spill, and took 774 us for 732 (B8 T2048 C1024)

template <class K>
struct BwdSmem {
    static constexpr int WARPS = K::NT / 32;
    float2 du[K::TT][K::CB];                        // delta, delta x
    alignas(16) float dy[K::TT][K::CB];
    alignas(16) float bc[2][K::TT][K::N];
    alignas(16) float part[3][K::TT][K::CB][K::YL]; // partial sums of y, du and sum_n g q A
    alignas(16) float dbc[WARPS][K::TT][2][K::N];
    double dd[K::TT][K::CB][2];                     // sums of dD and ddt_bias, of each preparer
};

// Sums a lane's V values (NP of dB, NP of dC) over the M lanes of a warp that differ in their
// channel.  Each shuffle halves the values that a lane still holds; it ends with kKept of
// them, from at() on.
template <class K>
struct ChannelSum {
    static constexpr int M = 32 / K::LPC, V = 2 * K::NP;
    static constexpr int kKept = M >= V ? 1 : V / M;
    static __device__ __forceinline__ int at(int lane) { return M >= V ? lane / K::LPC / (M >= V ? M / V : 1) : lane / K::LPC * kKept; }
    static __device__ __forceinline__ void run(float (&v)[V], int lane) {
        int nv = V;
#pragma unroll
        for (int o = M / 2; o > 0; o /= 2) {
            if (nv > 1) {
                nv /= 2;
                const bool up = lane & (o * K::LPC);
#pragma unroll
                for (int i = 0; i < V / 2; ++i)
                    if (i < nv) {
                        const float keep = up ? v[i + nv] : v[i], send = up ? v[i] : v[i + nv];
                        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o * K::LPC);
                    }
            } else {
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], o * K::LPC);
            }
        }
    }
};

// The backward's split form: a sequence's gradient of the state goes from g behind a piece to
// exp(A sum delta) g + r before it.  For a piece that starts inside a sequence, r from that
// sequence's tokens in it (from dh_final where the sequence ends there, so that r is the
// gradient itself); sum delta is the forward's (ends_kernel).
template <typename T, class K, bool VEC>
__global__ void __launch_bounds__(K::NT)
back_ends_kernel(const __grid_constant__ Params p) {
    constexpr int N = K::N, TT = K::TT, E = K::E, PP = K::PP;
    constexpr int QUADS = TT * N / 4, QP = (QUADS + K::NT - 1) / K::NT;   // of C
    __shared__ FwdSmem<K> sm;   // du: delta and dy, bc[1]: C
    const Place<K> at(p);
    const long begin = blockIdx.y * p.piece;
    const int n = p.seq.find(begin), tid = threadIdx.x;
    long s, e;
    if (!p.seq.bounds(n, s, e) || s >= begin || e <= begin) return;
    const long to = min(e, begin + p.piece);
    Pair A2[PP], g[PP] = {};
    load_decays<K>(p, at, A2);
    if (to == e && p.dh_final) load_pairs(p.dh_final + ((long)n * p.C + at.c) * N + at.n0, g);
    float bias[E];
#pragma unroll
    for (int i = 0; i < E; ++i) bias[i] = p.dt_bias && i < at.count ? p.dt_bias[at.gc + i] : 0.f;
    Group<T, E> dr, zr, orr;
    typename Raw4<T>::type cr[QP];
    auto fetch = [&](long t0) {
        const long o = min(t0 + at.gt, to - 1) * p.C + at.gc;
        dr = load_group<VEC, T, E>(p.dt, o, at.count);
        zr = load_group<VEC, T, E>(p.z ? p.z : p.dout, o, at.count);
        orr = load_group<VEC, T, E>(p.dout, o, at.count);
#pragma unroll
        for (int k = 0; k < QP; ++k) {
            const int q = min(tid + k * K::NT, QUADS - 1);
            const long tc = min(t0 + q / (N / 4), to - 1);
            cr[k] = *reinterpret_cast<const typename Raw4<T>::type*>(static_cast<const T*>(p.Cm) + (tc * p.G + at.g) * N +
                                                                     q % (N / 4) * 4);
        }
    };
    long t0 = begin + (to - begin - 1) / TT * TT;
    fetch(t0);
    for (; t0 >= begin; t0 -= TT) {
        const bool live = t0 + at.gt < to;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            // past the end: delta = 0 and dy = 0 leave g as it is
            const float o = to_f(orr.v[i]), dy = p.z ? o * silu(to_f(zr.v[i])) : o;
            sm.du[at.gt][du_slot<K>(at.gt, at.gi + i)] =
                live ? make_float2(softplus(to_f(dr.v[i]) + bias[i]), dy) : make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < QP; ++k) {
            const int q = tid + k * K::NT;
            float v[4];
            widen(cr[k], v);
            const bool in = t0 + q / (N / 4) < to;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = in ? v[i] : 0.f;
            if (q < QUADS) store_v<4>(&sm.bc[1][0][0] + q * 4, v);
        }
        __syncthreads();
        if (t0 > begin) fetch(t0 - TT);
#pragma unroll
        for (int j0 = TT - kBatch; j0 >= 0; j0 -= kBatch) {
            Pair a[kBatch][PP], c[kBatch][PP];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const float2 dd = sm.du[j0 + j][du_slot<K>(j0 + j, at.li)];
                load_pairs(&sm.bc[1][j0 + j][at.n0], c[j]);
#pragma unroll
                for (int i = 0; i < PP; ++i) {
                    a[j][i] = decay_pair(pair(dd.x, dd.x), A2[i]);
                    c[j][i] = mul2(pair(dd.y, dd.y), c[j][i]);
                }
            }
#pragma unroll
            for (int j = kBatch - 1; j >= 0; --j)
#pragma unroll
                for (int i = 0; i < PP; ++i) g[i] = fma2(a[j][i], g[i], mul2(a[j][i], c[j][i]));
        }
        __syncthreads();
    }
    if (at.on) store_pairs(p.back_ends + ((long)blockIdx.y * p.C + at.c) * N + at.n0, g);
}

template <typename T, class K, bool VEC, bool SPLIT>
__global__ void __launch_bounds__(K::NT, kBwdBlocks)
bwd_kernel(const __grid_constant__ Params p) {
    constexpr int N = K::N, TT = K::TT, E = K::E, PP = K::PP, NP = K::NP, SUBS = TT / kSub;
    constexpr int QUADS = TT * N / 4, QP = (2 * QUADS + K::NT - 1) / K::NT;
    extern __shared__ __align__(16) char smem_raw[];
    BwdSmem<K>& sm = *reinterpret_cast<BwdSmem<K>*>(smem_raw);
    const Place<K> at(p);
    const int row = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long tokens = p.seq.tokens();
    Pair A2[PP];
    load_decays<K>(p, at, A2);
    float bias[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = p.dt_bias && i < at.count ? p.dt_bias[at.gc + i] : 0.f;
        sm.dd[at.gt][at.gi + i][0] = sm.dd[at.gt][at.gi + i][1] = 0.0;
    }
    // long sums: in fp32 over kSub tokens (dA) or kFlush tiles (dD, ddt_bias), then in fp64
    double dA[NP] = {};
    float dD[E], dbias[E];
#pragma unroll
    for (int i = 0; i < E; ++i) dD[i] = dbias[i] = 0.f;
    auto flush = [&]() {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            sm.dd[at.gt][at.gi + i][0] += (double)dD[i];
            sm.dd[at.gt][at.gi + i][1] += (double)dbias[i];
            dD[i] = dbias[i] = 0.f;
        }
    };
    int since = 0;
    if (SPLIT && p.dh0)   // sequences without tokens
        for (int n = row; n < p.seq.N; n += p.pieces) {
            long s, e;
            if (!p.seq.bounds(n, s, e) || s < e || !at.on) continue;
            const long hrow = ((long)n * p.C + at.c) * N + at.n0;
            Pair g[PP] = {};
            if (p.dh_final) load_pairs(p.dh_final + hrow, g);
            store_pairs(p.dh0 + hrow, g);
        }

    // one sequence, or the piece's parts [s, e) of sequences, the last one first
    const long begin = SPLIT ? row * p.piece : 0, end = SPLIT ? min(begin + p.piece, tokens) : tokens;
    for (int n = SPLIT ? p.seq.find(end - 1) : row; n >= 0; --n) {
        long first, last;   // of the whole sequence
        const bool sound = p.seq.bounds(n, first, last);   // if not: reported by the first sweep
        if (SPLIT && sound && last <= begin) break;
        const long s = SPLIT ? max(first, begin) : first, e = SPLIT ? min(last, end) : last;
        if (!sound || (SPLIT && s >= e)) {
            if (SPLIT) continue;
            return;
        }
        const long hrow = ((long)n * p.C + at.c) * N + at.n0;
        Pair g[PP] = {};
        if (e == last) {
            if (p.dh_final && at.on) load_pairs(p.dh_final + hrow, g);
        } else {   // composed from the pieces behind this one
            const int ends_in = (int)((last - 1) / p.piece);
            load_pairs(p.back_ends + ((long)ends_in * p.C + at.c) * N + at.n0, g);
#pragma unroll 4
            for (int i = ends_in - 1; i > row; --i) {
                const long q = (long)i * p.C + at.c;
                const float ds = p.dsum[q];
                Pair r[PP];
                load_pairs(p.back_ends + q * N + at.n0, r);
#pragma unroll
                for (int k = 0; k < PP; ++k) g[k] = fma2(decay_pair(pair(ds, ds), A2[k]), g[k], r[k]);
            }
        }
        Group<T, E> xr, dr, zr, orr;
        typename Raw4<T>::type br[QP];
        auto fetch = [&](long t0) {
            const long o = min(t0 + at.gt, e - 1) * p.C + at.gc;
            xr = load_group<VEC, T, E>(p.x, o, at.count);
            dr = load_group<VEC, T, E>(p.dt, o, at.count);
            zr = load_group<VEC, T, E>(p.z ? p.z : p.x, o, at.count);
            orr = load_group<VEC, T, E>(p.dout, o, at.count);
            const long ahead = max(min(t0 + at.gt, e - 1) - 2 * TT, s) * p.C + at.gc;
            prefetch_l2(static_cast<const T*>(p.x) + ahead);
            prefetch_l2(static_cast<const T*>(p.dt) + ahead);
            prefetch_l2(static_cast<const T*>(p.dout) + ahead);
            if (p.z) prefetch_l2(static_cast<const T*>(p.z) + ahead);
#pragma unroll
            for (int k = 0; k < QP; ++k) {
                const int q = tid + k * K::NT, r = q % QUADS;
                const long tb = min(t0 + r / (N / 4), e - 1);
                br[k] = *reinterpret_cast<const typename Raw4<T>::type*>(
                    static_cast<const T*>(q >= QUADS ? p.Cm : p.Bm) + (tb * p.G + at.g) * N + r % (N / 4) * 4);
            }
        };
        // the stored state before the sub-chunk in hand, read one sub-chunk ahead
        Pair next[PP];
        const float* stored = nullptr;
        if (s < e) {
            fetch(s + (e - s - 1) / TT * TT);
            stored = p.ckpt + (ckpt_slot(s, SPLIT ? n + row : n, (e - s - 1) / kSub) * p.C + at.c) * N + at.n0;
            load_pairs(stored, next);
        }
        for (long t0 = s + (e - s - 1) / TT * TT; t0 >= s && s < e; t0 -= TT) {
            const bool live = t0 + at.gt < e && at.count > 0;
            const Group<T, E> x = xr, dt = dr, z = zr, dout = orr;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                // past the end, and for channels that do not exist: nothing reaches g or a sum
                const bool in = live && i < at.count;
                const float delta = in ? softplus(to_f(dt.v[i]) + bias[i]) : 0.f;
                const float o = in ? to_f(dout.v[i]) : 0.f;
                sm.du[at.gt][du_slot<K>(at.gt, at.gi + i)] = make_float2(delta, in ? delta * to_f(x.v[i]) : 0.f);
                sm.dy[at.gt][at.gi + i] = p.z && in ? o * silu(to_f(z.v[i])) : o;
            }
#pragma unroll
            for (int k = 0; k < QP; ++k) {
                const int q = tid + k * K::NT;
                float v[4];
                widen(br[k], v);
                const bool in = t0 + q % QUADS / (N / 4) < e;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = in ? v[i] : 0.f;
                if (q < 2 * QUADS) store_v<4>(&sm.bc[0][0][0] + q * 4, v);
            }
            __syncthreads();
            if (t0 > s) fetch(t0 - TT);
#pragma unroll 1
            for (int k = SUBS - 1; k >= 0; --k) {
                if (t0 + k * kSub >= e) continue;
                Pair a[kSub][PP], q[kSub][PP], dAk[PP] = {}, h[PP];
#pragma unroll
                for (int i = 0; i < PP; ++i) h[i] = next[i];
                if (t0 + k * kSub > s) {
                    stored -= (long)p.C * N;
                    load_pairs(stored, next);
                    prefetch_l2(t0 + k * kSub > s + 2 * kSub ? stored - 2l * p.C * N : stored);
                }
#pragma unroll
                for (int j = 0; j < kSub; ++j) {
                    const float2 du = sm.du[k * kSub + j][du_slot<K>(j, at.li)];
                    Pair b[PP];
                    load_pairs(&sm.bc[0][k * kSub + j][at.n0], b);
#pragma unroll
                    for (int i = 0; i < PP; ++i) {
                        a[j][i] = decay_pair(pair(du.x, du.x), A2[i]);
                        q[j][i] = mul2(a[j][i], h[i]);
                        h[i] = fma2(pair(du.y, du.y), b[i], q[j][i]);
                    }
                }
#pragma unroll
                for (int j0 = kSub - kBatch; j0 >= 0; j0 -= kBatch) {
                    float2 du[kBatch];
                    float dy[kBatch], sums[3][kBatch], dbc[kBatch][ChannelSum<K>::kKept];
                    Pair b[kBatch][PP], c[kBatch][PP];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const int t = k * kSub + j0 + j;
                        du[j] = sm.du[t][du_slot<K>(t, at.li)];
                        dy[j] = sm.dy[t][at.li];
                        load_pairs(&sm.bc[0][t][at.n0], b[j]);
                        load_pairs(&sm.bc[1][t][at.n0], c[j]);
                    }
#pragma unroll
                    for (int j = kBatch - 1; j >= 0; --j) {
                        const Pair dl = pair(du[j].x, du[j].x), u = pair(du[j].y, du[j].y), dd = pair(dy[j], dy[j]);
                        Pair y, gb, gqa;
                        float v[2 * NP];
#pragma unroll
                        for (int i = 0; i < PP; ++i) {
                            const Pair qq = q[j0 + j][i], ht = fma2(u, b[j][i], qq);
                            g[i] = fma2(c[j][i], dd, g[i]);
                            const Pair gq = mul2(g[i], qq);
                            y = i ? fma2(ht, c[j][i], y) : mul2(ht, c[j][i]);
                            gb = i ? fma2(g[i], b[j][i], gb) : mul2(g[i], b[j][i]);
                            gqa = i ? fma2(gq, A2[i], gqa) : mul2(gq, A2[i]);
                            dAk[i] = fma2(gq, dl, dAk[i]);
                            unpair(mul2(g[i], u), v[2 * i], v[2 * i + 1]);
                            unpair(mul2(ht, dd), v[NP + 2 * i], v[NP + 2 * i + 1]);
                            g[i] = mul2(a[j0 + j][i], g[i]);
                        }
                        float lo, hi;
                        unpair(y, lo, hi);
                        sums[0][j] = lo + hi;
                        unpair(gb, lo, hi);
                        sums[1][j] = lo + hi;
                        unpair(gqa, lo, hi);
                        sums[2][j] = lo + hi;
#pragma unroll
                        for (int m = 0; m < 3; ++m) sums[m][j] = set_sum<K>(sums[m][j]);
                        ChannelSum<K>::run(v, lane);
#pragma unroll
                        for (int i = 0; i < ChannelSum<K>::kKept; ++i) dbc[j][i] = v[i];
                    }
                    const int ys = y_slot<K>(at.li), vi = ChannelSum<K>::at(lane);
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const int t = k * kSub + j0 + j;
#pragma unroll
                        for (int m = 0; m < 3; ++m) sm.part[m][t][ys][set_of<K>(tid)] = sums[m][j];
#pragma unroll
                        for (int i = 0; i < ChannelSum<K>::kKept; ++i)
                            sm.dbc[warp][t][(vi + i) / NP][at.n0 + (vi + i) % NP] = dbc[j][i];
                    }
                }
#pragma unroll
                for (int i = 0; i < PP; ++i) {
                    float lo, hi;
                    unpair(dAk[i], lo, hi);
                    dA[2 * i] += (double)lo;
                    dA[2 * i + 1] += (double)hi;
                }
            }
            __syncthreads();
            if (live) {
                const long o = (t0 + at.gt) * p.C + at.gc;
                float dx[E], ddt[E], dz[E];
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    float sum[3];
#pragma unroll
                    for (int m = 0; m < 3; ++m) {
                        const float* l = sm.part[m][at.gt][y_slot<K>(at.gi + i)];
                        sum[m] = l[0] + l[1];
                        if (K::YL == 4) sum[m] += l[2] + l[3];
                    }
                    const float xv = to_f(x.v[i]), dy = sm.dy[at.gt][at.gi + i];
                    const float delta = sm.du[at.gt][du_slot<K>(at.gt, at.gi + i)].x;
                    const float D = p.D && i < at.count ? p.D[at.gc + i] : 0.f;
                    dx[i] = fmaf(sum[1], delta, D * dy);
                    ddt[i] = fmaf(sum[1], xv, sum[2] * (1.f / kLog2e)) * sigmoid(to_f(dt.v[i]) + bias[i]);
                    dz[i] = p.z ? to_f(dout.v[i]) * fmaf(D, xv, sum[0]) * dsilu(to_f(z.v[i])) : 0.f;
                    if (i < at.count) {
                        dD[i] = fmaf(dy, xv, dD[i]);
                        dbias[i] += ddt[i];
                    }
                }
                store_group<VEC, T, E>(p.dx, o, dx, at.count);
                store_group<VEC, T, E>(p.ddt, o, ddt, at.count);
                if (p.z) store_group<VEC, T, E>(p.dz, o, dz, at.count);
            }
            if (++since == kFlush) {
                flush();
                since = 0;
            }
            for (int i = tid; i < TT * 2 * N / 4; i += K::NT) {
                if (t0 + i / (2 * N / 4) >= e) continue;
                float4 v = reinterpret_cast<const float4*>(&sm.dbc[0][0][0][0])[i];
#pragma unroll
                for (int w = 1; w < BwdSmem<K>::WARPS; ++w) {
                    const float4 o = reinterpret_cast<const float4*>(&sm.dbc[w][0][0][0])[i];
                    v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
                }
                reinterpret_cast<float4*>(p.part_bc + ((long)blockIdx.x * tokens + t0) * 2 * N)[i] = v;
            }
        }
        if (s == first && p.dh0 && at.on) store_pairs(p.dh0 + hrow, g);
        if (!SPLIT) break;
    }
    flush();
    __syncthreads();
    if (!at.on) return;
#pragma unroll
    for (int i = 0; i < NP; ++i) p.part_a[((long)row * p.C + at.c) * N + at.n0 + i] = dA[i];
    if (at.n0 == 0) {
        double sum[2] = {0.0, 0.0};
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int m = 0; m < 2; ++m) sum[m] += sm.dd[t][at.li][m];
        p.part_d[((long)row * 2) * p.C + at.c] = sum[0];
        p.part_d[((long)row * 2 + 1) * p.C + at.c] = sum[1];
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

// dA_log, dD and ddt_bias from the sums of the pieces, or of the sequences (pieces <= 1), in a
// fixed order.
__global__ void __launch_bounds__(256)
sum_params_kernel(const double* __restrict__ part_a, const double* __restrict__ part_d, const float* __restrict__ A_log,
                  float* __restrict__ dA_log, float* __restrict__ dD, float* __restrict__ dbias, const Seqs seq, int pieces, int C, int N) {
    const long id = (long)blockIdx.x * 256 + threadIdx.x, CN = (long)C * N;
    if (id >= CN + 2 * C) return;
    const long i = id < CN ? id : id - CN;
    const double* part = id < CN ? part_a : part_d;
    const long cols = id < CN ? CN : 2 * C;
    double v = 0.0;
    for (int n = 0; n < (pieces > 1 ? pieces : seq.N); ++n) {
        long s, e;
        if (pieces > 1 || seq.bounds(n, s, e)) v += part[(long)n * cols + i];
    }
    if (id < CN) dA_log[i] = (float)(v * -exp((double)A_log[i]));   // in double: v is 0 where fp32's A overflows
    else if (i < C) { if (dD) dD[i] = (float)v; }
    else if (dbias) dbias[i - C] = (float)v;
}

// One token: the state h [B, C, N] is read and written once, which bounds it: 31 us for B256
// C4096 N16, 143 MB at 4.6 TB/s.  A block takes kStepSeqs sequences of its channels, all their
// loads in flight together (2, 4, 8 of them: 33, 31, 35 us; without the streaming hints 35).
constexpr int kStepSeqs = 4;
template <typename T, class K>
__global__ void __launch_bounds__(K::NT)
step_kernel(const __grid_constant__ Params p) {
    constexpr int N = K::N;
    const Place<K> at(p);
    const int first = blockIdx.y * kStepSeqs, count = min(p.seq.N - first, kStepSeqs);
    float h[kStepSeqs][4], b[kStepSeqs][4], c[kStepSeqs][4], x[kStepSeqs], dt[kStepSeqs], z[kStepSeqs];
#pragma unroll
    for (int k = 0; k < kStepSeqs; ++k) {
        const long n = first + min(k, count - 1), o = n * p.C + at.c, g = (n * p.G + at.g) * N + at.n0;
        const float4 hv = __ldcs(reinterpret_cast<const float4*>(p.h_final + o * N + at.n0));   // not read again
        h[k][0] = hv.x; h[k][1] = hv.y; h[k][2] = hv.z; h[k][3] = hv.w;
        load_v<4>(static_cast<const T*>(p.Bm) + g, b[k]);
        load_v<4>(static_cast<const T*>(p.Cm) + g, c[k]);
        x[k] = to_f(static_cast<const T*>(p.x)[o]);
        dt[k] = to_f(static_cast<const T*>(p.dt)[o]);
        z[k] = to_f(static_cast<const T*>(p.z ? p.z : p.x)[o]);
    }
    Pair A2[K::PP];
    load_decays<K>(p, at, A2);
    const float bias = p.dt_bias ? p.dt_bias[at.c] : 0.f, D = p.D ? p.D[at.c] : 0.f;
#pragma unroll
    for (int k = 0; k < kStepSeqs; ++k) {
        if (k >= count) break;
        const long o = (long)(first + k) * p.C + at.c;
        const float delta = softplus(dt[k] + bias), u = delta * x[k];
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float lo, hi;
            const Pair a = decay_pair(pair(delta, delta), A2[i]);
            unpair(fma2(a, pair(h[k][2 * i], h[k][2 * i + 1]), mul2(pair(u, u), pair(b[k][2 * i], b[k][2 * i + 1]))), lo, hi);
            h[k][2 * i] = lo;
            h[k][2 * i + 1] = hi;
            y = fmaf(lo, c[k][2 * i], fmaf(hi, c[k][2 * i + 1], y));
        }
        if (at.on) __stcs(reinterpret_cast<float4*>(p.h_final + o * N + at.n0), make_float4(h[k][0], h[k][1], h[k][2], h[k][3]));
#pragma unroll
        for (int w = 1; w < K::LPC; w *= 2) y += __shfl_xor_sync(0xffffffffu, y, w);
        if (at.on && at.n0 == 0) {
            y = fmaf(D, x[k], y);
            static_cast<T*>(p.out)[o] = from_f<T>(p.z ? y * silu(z[k]) : y);
        }
    }
}

}  // namespace scan
}  // namespace comba
