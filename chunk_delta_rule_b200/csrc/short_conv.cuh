// Short causal convolution over tokens, one filter per channel (the convolution in front
// of a recurrent mixer's projections):
//
//   pre_t = bias + sum_{j < W} w_j x_{t-W+1+j},   out_t = silu(pre_t) or pre_t
//
// with the W-1 inputs before a sequence's first token taken from its carried state.  Every
// token is read and written once, so the kernels are bound by HBM bandwidth: a thread
// keeps the filter and the last W-1 inputs of 4 neighbouring channels in registers and
// walks a tile of tokens (8 channels would take twice the registers, and halve the threads).
// Measured on B8 T4096 C6144 W4 bf16: forward 133 us, 6.05 TB/s of a copy's 6.55; backward
// 249 us, 4.85 TB/s, where latency bounds it: neither the issue slots (63 % busy) nor HBM are
// full with the 16 warps an SM that the 72 values a thread keeps for its 4 channels' filter,
// sums and open rows allow.
#pragma once

#include <limits.h>

#include <type_traits>

#include "block_common.cuh"

namespace comba {
namespace conv {

using namespace blk;

constexpr int kThreads = 128;
constexpr int kMaxChannels = 1 << 23;   // a tile of up to 128 tokens then fits 32-bit offsets
constexpr int kChannels = 4;      // that a thread handles on the vector path

struct Params {
    const float *weight, *bias;     // [C, W], [C] or null
    const void *x, *init;           // [tokens, C], [N, W-1, C] or null
    void *out, *fin;                // [tokens, C], [N, W-1, C] or null
    const void *dout, *dfin;        // backward: cotangents
    void *dx, *dinit;
    float* part;                    // [tiles, W+1, C] partial sums of dweight and dbias
    Seqs seq;
    int C;
    int L;                          // tokens in a tile
    int* status;
};

// The filters and biases of channels c .. c+V-1 (V == 4: their V W weights are 16-byte aligned).
template <int W, int V>
__device__ __forceinline__ void load_filter(const float* __restrict__ weight, const float* __restrict__ bias, int c,
                                            float (&w)[W][V], float (&b)[V]) {
    float f[V * W];
    load_v<V * W>(weight + (long)c * W, f);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = f[i * W + j];
    if (bias) {
        load_v<V>(bias + c, b);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) b[i] = 0.f;
    }
}

// Input of sequence [s, ..) at token t, which may lie up to W-1 before s: there it is the
// carried state of sequence n (zero without one).
template <typename T, int W, int V>
__device__ __forceinline__ void load_x(const Params& p, int n, long s, long t, int c, float (&x)[V]) {
    if (t >= s) {
        load_v<V>(static_cast<const T*>(p.x) + t * p.C + c, x);
    } else if (p.init) {
        load_v<V>(static_cast<const T*>(p.init) + ((long)n * (W - 1) + (t - s + W - 1)) * p.C + c, x);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = 0.f;
    }
}

// A thread's V channels of the next tokens, on their way into a ring of its own in shared
// memory: rows in flight do not cost registers, which alone held too few to cover HBM's
// latency (forward of B8 T4096 C6144 bf16: 209 us with 4 rows a thread in registers).
// Rows go in and out kAhead at a time; K arrays are read side by side.
constexpr int kAhead = 4;
template <typename T, int V, int K>
struct Ring {
    static constexpr int GROUPS = V * sizeof(T) > 8 ? 2 : 4, ROWS = GROUPS * kAhead;
    struct alignas(V * sizeof(T)) Row {
        T v[V];
    };
    using Storage = Row[ROWS][K][kThreads];
    Storage& mem;
    __device__ __forceinline__ void put(int slot, int k, const T* p) {
        Row* r = &mem[slot][k][threadIdx.x];
        if constexpr (sizeof(Row) >= 4) {
            const unsigned at = (unsigned)__cvta_generic_to_shared(r);
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(p), "n"((int)sizeof(Row)) : "memory");
        } else {
            *r = *reinterpret_cast<const Row*>(p);
        }
    }
    __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    template <int LEFT>
    __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }
    __device__ __forceinline__ void get(int slot, int k, float (&x)[V]) const { load_v<V>(mem[slot][k][threadIdx.x].v, x); }
};

// acc[i] += a[i] * b[i], two at a time.
template <int V>
__device__ __forceinline__ void fma_v(const float (&a)[V], const float (&b)[V], float (&acc)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2)
            unpair(fma2(pair(a[i], a[i + 1]), pair(b[i], b[i + 1]), pair(acc[i], acc[i + 1])), acc[i], acc[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(a[i], b[i], acc[i]);
    }
}

// One thread per (tile of tokens, V channels), then one per (sequence, state row, V
// channels) for the final states and the check of the bounds.
template <typename T, int W, int V, bool SILU>
__global__ void __launch_bounds__(kThreads)
fwd_kernel(const __grid_constant__ Params p, long tiles, long total) {
    const long id = (long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= total) return;
    const int cv = p.C / V;
    const long row = id / cv;
    const int c = (int)(id - row * cv) * V;
    if (row >= tiles) {
        const long q = row - tiles;
        const int n = (int)(q / (W - 1)), m = (int)(q % (W - 1));
        long s, e;
        if (!p.seq.bounds(n, s, e)) {
            atomicCAS(p.status, 0, COMBA_EINVAL);
            return;
        }
        if (p.fin) {
            float x[V];
            load_x<T, W, V>(p, n, s, e - (W - 1) + m, c, x);
            store_v<V>(static_cast<T*>(p.fin) + ((long)n * (W - 1) + m) * p.C + c, x);
        }
        return;
    }
    using R = Ring<T, V, 1>;
    __shared__ typename R::Storage mem;
    R ring{mem};
    const long t0 = row * p.L, t1 = min(t0 + (long)p.L, p.seq.tokens());
    float w[W][V], b[V];
    load_filter<W, V>(p.weight, p.bias, c, w, b);
    long t = t0;
    for (int n = p.seq.find(t0); n < p.seq.N && t < t1; ++n) {
        long s, e;
        if (!p.seq.bounds(n, s, e) || e <= t) continue;
        if (s >= t1) break;
        t = max(t, s);
        const long stop = min(e, t1);
        float h[W][V];   // inputs t-W+1 .. t
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_x<T, W, V>(p, n, s, t - (W - 1) + j, c, h[j]);
        const T* xp = static_cast<const T*>(p.x) + t * p.C + c;
        T* op = static_cast<T*>(p.out) + t * p.C + c;
        // the ring runs GROUPS - 1 groups ahead (past the end: the last token's, not used);
        // offsets within a tile fit 32 bits
        const int last = (int)(stop - 1 - t);
        const unsigned C = p.C;
        auto fetch = [&](int at) {
            if (at <= last)
#pragma unroll
                for (int k = 0; k < kAhead; ++k) ring.put((at + k) % R::ROWS, 0, xp + min(at + k, last) * C);
            ring.commit();
        };
#pragma unroll
        for (int k = 0; k < R::GROUPS - 1; ++k) fetch(k * kAhead);
        auto token = [&](int at) {
            ring.get(at % R::ROWS, 0, h[W - 1]);
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = b[i];
#pragma unroll
            for (int j = 0; j < W; ++j) fma_v<V>(w[j], h[j], y);
            if (SILU)
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] = silu(y[i]);
            store_v<V>(op + at * C, y);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) h[j][i] = h[j + 1][i];
        };
        // whole groups without a condition between their tokens: h then moves on by renaming
        int k0 = 0;
        for (; k0 + kAhead <= last + 1; k0 += kAhead) {
            fetch(k0 + R::ROWS - kAhead);
            ring.template wait<R::GROUPS - 1>();
#pragma unroll
            for (int k = 0; k < kAhead; ++k) token(k0 + k);
        }
        if (k0 <= last) {
            ring.template wait<0>();
#pragma unroll
            for (int k = 0; k < kAhead - 1; ++k)
                if (k0 + k <= last) token(k0 + k);
        }
        ring.template wait<0>();
        t = stop;
    }
}

// d pre of one token from its cotangent d; its input is h[W-1], the W-1 before it h[0 .. W-2].
template <int W, int V, bool SILU>
__device__ __forceinline__ void dpre_of(const float (&w)[W][V], const float (&b)[V], const float (&h)[W][V], float (&d)[V]) {
    if (SILU) {
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = b[i];
#pragma unroll
        for (int j = 0; j < W; ++j) fma_v<V>(w[j], h[j], y);
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] *= dsilu(y[i]);
    }
}

// Cotangent of the initial state's row m, the input W-1-m before the first token, and the
// check of the bounds: one thread per (sequence, row, V channels).
template <typename T, int W, int V, bool SILU>
__global__ void __launch_bounds__(kThreads)
bwd_state_kernel(const __grid_constant__ Params p, long total) {
    const long id = (long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= total) return;
    const int cv = p.C / V, c = (int)(id % cv) * V;
    const int n = (int)(id / cv / (W - 1)), m = (int)(id / cv % (W - 1));
    long s, e;
    if (!p.seq.bounds(n, s, e)) {
        atomicCAS(p.status, 0, COMBA_EINVAL);
        return;
    }
    if (!p.dinit) return;
    float w[W][V], b[V], g[V];
    load_filter<W, V>(p.weight, p.bias, c, w, b);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = 0.f;
    const long at = m - (e - s);   // its row of the final state, of a sequence shorter than that
    if (p.dfin && at >= 0) load_v<V>(static_cast<const T*>(p.dfin) + ((long)n * (W - 1) + at) * p.C + c, g);
#pragma unroll 1
    for (int k = 0; k <= m && s + k < e; ++k) {   // token s + k reads it through tap m - k
        float h[W][V], d[V];
#pragma unroll
        for (int j = 0; j < W; ++j) load_x<T, W, V>(p, n, s, s + k - (W - 1) + j, c, h[j]);
        load_v<V>(static_cast<const T*>(p.dout) + (s + k) * p.C + c, d);
        dpre_of<W, V, SILU>(w, b, h, d);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = fmaf(p.weight[(long)(c + i) * W + m - k], d[i], g[i]);
    }
    store_v<V>(static_cast<T*>(p.dinit) + ((long)n * (W - 1) + m) * p.C + c, g);
}

// Backward of one tile.  With dpre_t = dout_t silu'(pre_t) (pre recomputed),
//   dx_t = sum_j w_j dpre_{t+W-1-j} (+ the final state's cotangent),
//   dw_j = sum_t dpre_t x_{t-W+1+j},   dbias = sum_t dpre_t.
// A thread walks its tokens and W-1 more of the same sequence, whose dpre it forms again
// for the tile's last dx; the sums take the tile's own tokens only and go to `part`.
template <typename T, int W, int V, bool SILU>
__global__ void __launch_bounds__(kThreads, 4)
bwd_kernel(const __grid_constant__ Params p, long total) {
    const long id = (long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= total) return;
    const int cv = p.C / V;
    const long row = id / cv;
    const int c = (int)(id - row * cv) * V;
    const T* xb = static_cast<const T*>(p.x) + c;
    const T* ob = static_cast<const T*>(p.dout) + c;
    using R = Ring<T, V, 2>;
    __shared__ typename R::Storage mem;
    R ring{mem};
    float w[W][V], b[V];
    load_filter<W, V>(p.weight, p.bias, c, w, b);
    const long t0 = row * p.L, t1 = min(t0 + (long)p.L, p.seq.tokens());
    float dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
    }
    long t = t0;
    for (int n = p.seq.find(t0); n < p.seq.N && t < t1; ++n) {
        long s, e;
        if (!p.seq.bounds(n, s, e) || e <= t) continue;
        if (s >= t1) break;
        t = max(t, s);
        const long from = t, stop = min(e, t1);
        float h[W][V];   // inputs t-W+1 .. t
        float g[W][V];   // dx of tokens t-W+1 .. t, complete in g[0] once token t is in
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            load_x<T, W, V>(p, n, s, t - (W - 1) + j, c, h[j]);
#pragma unroll
            for (int i = 0; i < V; ++i) g[j][i] = 0.f;
        }
        // tokens are counted from `from` on; offsets within a tile fit 32 bits
        const int count = (int)(stop - from), rest = (int)min(e - from, (long)INT_MAX);
        const unsigned C = p.C;
        const T *xp = xb + from * p.C, *dp = ob + from * p.C;
        T* gp = static_cast<T*>(p.dx) + from * p.C + c;
        // adds a token's d to the open dx and closes that of the token W - 1 before it; END: the
        // token lies behind the tile, and the closed one may reach into the final state
        auto close = [&](int at, const float (&d)[V], auto END) {
#pragma unroll
            for (int i = 0; i < V; ++i) g[W - 1][i] = w[W - 1][i] * d[i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) fma_v<V>(w[j], d, g[j]);
            if (at >= W - 1) {
                if (decltype(END)::value && p.dfin && at >= rest) {
                    float f[V];
                    load_v<V>(static_cast<const T*>(p.dfin) + ((long)n * (W - 1) + (at - rest)) * p.C + c, f);
#pragma unroll
                    for (int i = 0; i < V; ++i) g[0][i] += f[i];
                }
                store_v<V>(gp + (at - (W - 1)) * C, g[0]);
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    h[j][i] = h[j + 1][i];
                    g[j][i] = g[j + 1][i];
                }
        };
        auto fetch = [&](int at) {   // past the tile: its last token's, not used
            if (at < count)
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const unsigned o = min(at + k, count - 1) * C;
                    ring.put((at + k) % R::ROWS, 0, xp + o);
                    ring.put((at + k) % R::ROWS, 1, dp + o);
                }
            ring.commit();
        };
#pragma unroll
        for (int k = 0; k < R::GROUPS - 1; ++k) fetch(k * kAhead);
        auto token = [&](int at) {
            float d[V];
            ring.get(at % R::ROWS, 0, h[W - 1]);
            ring.get(at % R::ROWS, 1, d);
            dpre_of<W, V, SILU>(w, b, h, d);
#pragma unroll
            for (int i = 0; i < V; ++i) db[i] += d[i];
#pragma unroll
            for (int j = 0; j < W; ++j) fma_v<V>(d, h[j], dw[j]);
            close(at, d, std::false_type());
        };
        // whole groups without a condition between their tokens: h and g then move on by renaming
        int k0 = 0;
        for (; k0 + kAhead <= count; k0 += kAhead) {
            fetch(k0 + R::ROWS - kAhead);
            ring.template wait<R::GROUPS - 1>();
#pragma unroll
            for (int k = 0; k < kAhead; ++k) token(k0 + k);
        }
        if (k0 < count) {
            ring.template wait<0>();
#pragma unroll
            for (int k = 0; k < kAhead - 1; ++k)
                if (k0 + k < count) token(k0 + k);
        }
        ring.template wait<0>();
        // the W-1 tokens behind the tile; past the sequence's end there is nothing to add
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            float d[V];
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] = h[W - 1][i] = 0.f;
            if (count + k < rest) {
                load_v<V>(xp + (count + k) * C, h[W - 1]);
                load_v<V>(dp + (count + k) * C, d);
                dpre_of<W, V, SILU>(w, b, h, d);
            }
            close(count + k, d, std::true_type());
        }
        t = stop;
    }
    float* o = p.part + row * (W + 1) * (long)p.C + c;
#pragma unroll
    for (int j = 0; j < W; ++j) store_v<V>(o + (long)j * p.C, dw[j]);
    store_v<V>(o + (long)W * p.C, db);
}

// dweight [C, W] and dbias [C] from the tiles' partial sums, in double and a fixed order.
template <int W>
__global__ void __launch_bounds__(256)
sum_kernel(const float* __restrict__ part, float* __restrict__ dweight, float* __restrict__ dbias, long tiles, int C) {
    __shared__ double s[8][33];
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, j = blockIdx.y;
    double acc = 0.0;
    if (c < C) {
#pragma unroll 8
        for (long i = r; i < tiles; i += 8) acc += (double)part[(i * (W + 1) + j) * C + c];
    }
    s[r][lane] = acc;
    __syncthreads();
    if (r != 0 || c >= C) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) acc += s[i][lane];
    if (j < W) dweight[(long)c * W + j] = (float)acc;
    else if (dbias) dbias[c] = (float)acc;
}

// One token: out = silu(bias + sum_j w_j [state, x]_j), and the state moves on by x.  A thread
// takes `per` sequences of its channels, kStepSeqs of them in flight, for one load of the
// filter; with per = 1 (B256 C4096 and fewer) it reads its one sequence's rows kStepSeqs times.
constexpr int kStepSeqs = 4;
template <typename T, int W, int V, bool SILU>
__global__ void __launch_bounds__(kThreads)
step_kernel(const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
            T* state, T* __restrict__ out, int B, int C, int per) {
    const long id = (long)blockIdx.x * kThreads + threadIdx.x;
    const int cv = C / V;
    const long n0 = id / cv * per;
    if (n0 >= B) return;
    const int c = (int)(id % cv) * V;
    const long end = min(n0 + per, (long)B);
    float w[W][V], b[V];
    load_filter<W, V>(weight, bias, c, w, b);
#pragma unroll 1
    for (long n = n0; n < end; n += kStepSeqs) {   // may pass 2^31 behind the last sequence
        float h[kStepSeqs][W][V];
#pragma unroll
        for (int k = 0; k < kStepSeqs; ++k) {
            const long m = min(n + k, end - 1);   // the last one again where there are fewer
#pragma unroll
            for (int j = 0; j < W - 1; ++j) load_v<V>(state + (m * (W - 1) + j) * C + c, h[k][j]);
            load_v<V>(x + m * C + c, h[k][W - 1]);
        }
#pragma unroll
        for (int k = 0; k < kStepSeqs; ++k) {
            if (n + k >= end) break;
            const long m = n + k;
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = b[i];
#pragma unroll
            for (int j = 0; j < W; ++j) fma_v<V>(w[j], h[k][j], y);
            if (SILU)
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] = silu(y[i]);
            store_v<V>(out + m * C + c, y);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) store_v<V>(state + (m * (W - 1) + j) * C + c, h[k][j + 1]);
        }
    }
}
// Sequences a thread takes: kStepSeqs once that still leaves an SM 512 threads.
inline int step_sequences(long B, int cv) { return B * cv >= (long)kSMs * 512 * kStepSeqs ? kStepSeqs : 1; }

// Tokens in a tile: long tiles read fewer tokens twice (W-1 a tile) and, in the backward,
// write fewer partial sums; short ones give enough threads when the tokens are few.  On B8
// T4096 C6144 tiles of up to 32, 64, 128 tokens took 137, 133, 135 us forward, and of up to 64,
// 128, 256 tokens 265, 249, 251 us backward.
inline int tile_tokens(long tokens, int cv, int most) {
    int L = most;
    while (L > 4 && ceil_div(tokens, L) * cv < (long)kSMs * 1024) L /= 2;
    return L;
}

}  // namespace conv
}  // namespace comba
