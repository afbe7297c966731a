// C ABI of the operators around and beside the recurrence (declared in comba.h): short
// causal convolution, selective scan, gated norm and residual norm.
//
// As in comba.cu, every argument is checked before anything is enqueued, work goes on the
// caller's stream, and no device memory is owned or allocated.
#include <algorithm>

#include "block_norm.cuh"
#include "selective_scan.cuh"
#include "short_conv.cuh"

namespace {

using namespace comba::blk;
namespace conv = comba::conv;
namespace scan = comba::scan;
namespace norm = comba::norm;

constexpr size_t kMaxElements = (size_t)1 << 40;
constexpr long kMaxGrid = 0x7fffffff;

size_t elt_size(int dtype) { return dtype == COMBA_BF16 ? 2 : 4; }
bool dtype_ok(int dtype) { return dtype == COMBA_BF16 || dtype == COMBA_F32; }

// Tokens in all of N uniform sequences of T, or of T packed tokens.
size_t token_count(const int* cu, int N, int T) { return cu ? (size_t)T : (size_t)N * T; }

// a * b * c, or more than kMaxElements where it exceeds that.
size_t volume(size_t a, size_t b, size_t c = 1) {
    if (a && b > kMaxElements / a) return kMaxElements + 1;
    const size_t ab = a * b;
    if (ab && c > kMaxElements / ab) return kMaxElements + 1;
    return ab * c;
}

// Rows of C elements that start aligned for accesses of `per` elements and hold whole ones.
bool vector_rows(int C, int per, size_t align, std::initializer_list<const void*> ptrs) {
    if (C % per) return false;
    for (const void* p : ptrs)
        if (!aligned(p, align)) return false;
    return true;
}

// ------------------------------------------------------------------ short convolution
template <typename T, int W, int V>
int conv_fwd(conv::Params& p, bool silu, cudaStream_t s) {
    const int cv = p.C / V;
    p.L = conv::tile_tokens(p.seq.tokens(), cv, 64);
    const long tiles = ceil_div(p.seq.tokens(), p.L);
    const long states = (p.fin || p.seq.cu) ? (long)p.seq.N * (W - 1) : 0;
    const long total = (tiles + states) * cv, blocks = ceil_div(total, conv::kThreads);
    if (blocks == 0) return COMBA_OK;
    if (blocks > kMaxGrid) return COMBA_EUNSUPPORTED;
    if (silu) conv::fwd_kernel<T, W, V, true><<<(unsigned)blocks, conv::kThreads, 0, s>>>(p, tiles, total);
    else conv::fwd_kernel<T, W, V, false><<<(unsigned)blocks, conv::kThreads, 0, s>>>(p, tiles, total);
    return launched();
}

// Tiles of the backward, and so the rows of partial sums: the same for either path's
// vector width, so that the workspace does not depend on pointers.
int conv_bwd_tile(size_t tokens, int C) { return conv::tile_tokens((long)tokens, (C + conv::kChannels - 1) / conv::kChannels, 128); }

template <typename T, int W, int V>
int conv_bwd(conv::Params& p, float* dweight, float* dbias, bool silu, cudaStream_t s) {
    const int cv = p.C / V;
    p.L = conv_bwd_tile((size_t)p.seq.tokens(), p.C);
    const long tiles = ceil_div(p.seq.tokens(), p.L);
    const long total = tiles * cv, blocks = ceil_div(total, conv::kThreads);
    const long states = (p.dinit || p.seq.cu) ? (long)p.seq.N * (W - 1) * cv : 0, sblocks = ceil_div(states, conv::kThreads);
    if (blocks > kMaxGrid || sblocks > kMaxGrid) return COMBA_EUNSUPPORTED;
    if (blocks) {
        if (silu) conv::bwd_kernel<T, W, V, true><<<(unsigned)blocks, conv::kThreads, 0, s>>>(p, total);
        else conv::bwd_kernel<T, W, V, false><<<(unsigned)blocks, conv::kThreads, 0, s>>>(p, total);
    }
    if (sblocks) {
        if (silu) conv::bwd_state_kernel<T, W, V, true><<<(unsigned)sblocks, conv::kThreads, 0, s>>>(p, states);
        else conv::bwd_state_kernel<T, W, V, false><<<(unsigned)sblocks, conv::kThreads, 0, s>>>(p, states);
    }
    const dim3 grid((unsigned)ceil_div(p.C, 32), W + 1);
    conv::sum_kernel<W><<<grid, 256, 0, s>>>(p.part, dweight, dbias, tiles, p.C);
    return launched();
}

template <typename T, int W, int V>
int conv_step(const T* x, const float* weight, const float* bias, T* state, T* out, int B, int C, bool silu,
              cudaStream_t s) {
    const int cv = C / V, per = conv::step_sequences(B, cv);
    const long blocks = ceil_div(ceil_div(B, per) * cv, conv::kThreads);
    if (blocks > kMaxGrid) return COMBA_EUNSUPPORTED;
    if (silu) conv::step_kernel<T, W, V, true><<<(unsigned)blocks, conv::kThreads, 0, s>>>(x, weight, bias, state, out, B, C, per);
    else conv::step_kernel<T, W, V, false><<<(unsigned)blocks, conv::kThreads, 0, s>>>(x, weight, bias, state, out, B, C, per);
    return launched();
}

// f(element type, taps, vector width) for the runtime values.
#define COMBA_CONV_DISPATCH(f, dtype, W, vec, ...)                                                      \
    ((dtype) == COMBA_BF16                                                                              \
         ? ((vec) ? ((W) == 4 ? f<bf16, 4, 4>(__VA_ARGS__) : (W) == 3 ? f<bf16, 3, 4>(__VA_ARGS__)      \
                                                                      : f<bf16, 2, 4>(__VA_ARGS__))     \
                  : ((W) == 4 ? f<bf16, 4, 1>(__VA_ARGS__) : (W) == 3 ? f<bf16, 3, 1>(__VA_ARGS__)      \
                                                                      : f<bf16, 2, 1>(__VA_ARGS__)))    \
         : ((vec) ? ((W) == 4 ? f<float, 4, 4>(__VA_ARGS__) : (W) == 3 ? f<float, 3, 4>(__VA_ARGS__)    \
                                                                       : f<float, 2, 4>(__VA_ARGS__))   \
                  : ((W) == 4 ? f<float, 4, 1>(__VA_ARGS__) : (W) == 3 ? f<float, 3, 1>(__VA_ARGS__)    \
                                                                       : f<float, 2, 1>(__VA_ARGS__))))

}  // namespace

extern "C" int comba_short_conv_fwd(const void* x, const float* weight, const float* bias, const void* initial_state,
                                    void* out, void* final_state, const int* cu_seqlens, int N, int T, int C, int W,
                                    int silu, int dtype, comba_stream_t stream) {
    if (N < 0 || T < 0 || C < 0 || W < 2 || W > 4 || !dtype_ok(dtype)) return COMBA_EINVAL;
    if (N == 0 || C == 0) return COMBA_OK;
    if (C > conv::kMaxChannels) return COMBA_EUNSUPPORTED;
    const size_t e = elt_size(dtype), tokens = token_count(cu_seqlens, N, T);
    if (volume(tokens, C) > kMaxElements || volume(N, W - 1, C) > kMaxElements) return COMBA_EINVAL;
    const size_t nx = tokens * C * e, ns = (size_t)N * (W - 1) * C * e;
    const Arg ins[] = {{x, nx, e, false}, {weight, (size_t)C * W * 4, 4, false}, {bias, (size_t)C * 4, 4, true},
                       {initial_state, ns, e, true}, {cu_seqlens, ((size_t)N + 1) * 4, 4, true}};
    const Arg outs[] = {{out, nx, e, false}, {final_state, ns, e, true}};
    if (!args_ok(ins, outs)) return COMBA_EINVAL;
    conv::Params p{};
    p.x = x; p.weight = weight; p.bias = bias; p.init = initial_state; p.out = out; p.fin = final_state;
    p.seq = Seqs{cu_seqlens, N, T};
    p.C = C;
    p.status = comba::status_word();
    if (!p.status) return COMBA_ECUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = vector_rows(C, conv::kChannels, conv::kChannels * e, {x, initial_state, out, final_state}) && aligned(weight, 16) && aligned(bias, 16);
    return COMBA_CONV_DISPATCH(conv_fwd, dtype, W, vec, p, silu != 0, s);
}

extern "C" size_t comba_short_conv_bwd_workspace_size(int N, int T, int C, int W, int packed) {
    if (N <= 0 || T < 0 || C <= 0 || W < 2 || W > 4) return 0;
    const size_t tokens = packed ? (size_t)T : (size_t)N * T;
    return (size_t)ceil_div((long)tokens, conv_bwd_tile(tokens, C)) * (W + 1) * C * sizeof(float);
}

extern "C" int comba_short_conv_bwd(const void* x, const float* weight, const float* bias, const void* initial_state,
                                    const void* dout, const void* dfinal_state, void* dx, float* dweight, float* dbias,
                                    void* dinitial_state, const int* cu_seqlens, int N, int T, int C, int W, int silu,
                                    int dtype, void* workspace, size_t workspace_bytes, comba_stream_t stream) {
    if (N < 0 || T < 0 || C < 0 || W < 2 || W > 4 || !dtype_ok(dtype)) return COMBA_EINVAL;
    if (C == 0) return COMBA_OK;
    if (N == 0) T = 0;   // no sequence covers a token
    if (C > conv::kMaxChannels) return COMBA_EUNSUPPORTED;
    const size_t e = elt_size(dtype), tokens = token_count(cu_seqlens, N, T);
    if (volume(tokens, C) > kMaxElements || volume(N, W - 1, C) > kMaxElements) return COMBA_EINVAL;
    const size_t nx = tokens * C * e, ns = (size_t)N * (W - 1) * C * e;
    const size_t need = comba_short_conv_bwd_workspace_size(N, T, C, W, cu_seqlens != nullptr);
    if (workspace_bytes < need) return COMBA_EINVAL;
    const Arg ins[] = {{x, nx, e, false}, {weight, (size_t)C * W * 4, 4, false}, {bias, (size_t)C * 4, 4, true},
                       {initial_state, ns, e, true}, {cu_seqlens, ((size_t)N + 1) * 4, 4, true},
                       {dout, nx, e, false}, {dfinal_state, ns, e, true}};
    const Arg outs[] = {{dx, nx, e, false}, {dweight, (size_t)C * W * 4, 4, false}, {dbias, (size_t)C * 4, 4, true},
                        {dinitial_state, ns, e, true}, {workspace, need, 16, false}};
    if (!args_ok(ins, outs)) return COMBA_EINVAL;
    conv::Params p{};
    p.x = x; p.weight = weight; p.bias = bias; p.init = initial_state;
    p.dout = dout; p.dfin = dfinal_state; p.dx = dx; p.dinit = dinitial_state;
    p.part = static_cast<float*>(workspace);
    p.seq = Seqs{cu_seqlens, N, T};
    p.C = C;
    p.status = comba::status_word();
    if (!p.status) return COMBA_ECUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = vector_rows(C, conv::kChannels, conv::kChannels * e, {x, initial_state, dout, dfinal_state, dx, dinitial_state}) && aligned(weight, 16) && aligned(bias, 16);
    return COMBA_CONV_DISPATCH(conv_bwd, dtype, W, vec, p, dweight, dbias, silu != 0, s);
}

extern "C" int comba_short_conv_step(const void* x, const float* weight, const float* bias, void* state, void* out,
                                     int B, int C, int W, int silu, int dtype, comba_stream_t stream) {
    if (B < 0 || C < 0 || W < 2 || W > 4 || !dtype_ok(dtype)) return COMBA_EINVAL;
    if (B == 0 || C == 0) return COMBA_OK;
    if (C > conv::kMaxChannels) return COMBA_EUNSUPPORTED;
    const size_t e = elt_size(dtype);
    if (volume(B, W, C) > kMaxElements) return COMBA_EINVAL;
    const size_t nx = (size_t)B * C * e;
    const Arg ins[] = {{x, nx, e, false}, {weight, (size_t)C * W * 4, 4, false}, {bias, (size_t)C * 4, 4, true}};
    const Arg outs[] = {{state, nx * (W - 1), e, false}, {out, nx, e, false}};
    if (!args_ok(ins, outs)) return COMBA_EINVAL;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = vector_rows(C, conv::kChannels, conv::kChannels * e, {x, state, out}) && aligned(weight, 16) && aligned(bias, 16);
    const bool act = silu != 0;
    if (dtype == COMBA_BF16) {
        const auto* xt = static_cast<const bf16*>(x);
        auto *st = static_cast<bf16*>(state), *ot = static_cast<bf16*>(out);
        if (vec) return W == 4 ? conv_step<bf16, 4, 4>(xt, weight, bias, st, ot, B, C, act, s)
                      : W == 3 ? conv_step<bf16, 3, 4>(xt, weight, bias, st, ot, B, C, act, s)
                               : conv_step<bf16, 2, 4>(xt, weight, bias, st, ot, B, C, act, s);
        return W == 4 ? conv_step<bf16, 4, 1>(xt, weight, bias, st, ot, B, C, act, s)
             : W == 3 ? conv_step<bf16, 3, 1>(xt, weight, bias, st, ot, B, C, act, s)
                      : conv_step<bf16, 2, 1>(xt, weight, bias, st, ot, B, C, act, s);
    }
    const auto* xt = static_cast<const float*>(x);
    auto *st = static_cast<float*>(state), *ot = static_cast<float*>(out);
    if (vec) return W == 4 ? conv_step<float, 4, 4>(xt, weight, bias, st, ot, B, C, act, s)
                  : W == 3 ? conv_step<float, 3, 4>(xt, weight, bias, st, ot, B, C, act, s)
                           : conv_step<float, 2, 4>(xt, weight, bias, st, ot, B, C, act, s);
    return W == 4 ? conv_step<float, 4, 1>(xt, weight, bias, st, ot, B, C, act, s)
         : W == 3 ? conv_step<float, 3, 1>(xt, weight, bias, st, ot, B, C, act, s)
                  : conv_step<float, 2, 1>(xt, weight, bias, st, ot, B, C, act, s);
}

// ------------------------------------------------------------------ selective scan
namespace {

bool states_ok(int N) { return N == 8 || N == 16 || N == 32 || N == 64 || N == 128; }

// Whether groups of up to 4 consecutive channels lie whole and aligned in every token tensor.
bool scan_vector(int C, int G, int dtype, std::initializer_list<const void*> ptrs) {
    if (C / G % 4) return false;
    for (const void* p : ptrs)
        if (!aligned(p, 4 * elt_size(dtype))) return false;
    return true;
}

// Channel blocks of one group.
int group_blocks(int C, int G, int N) { return (int)ceil_div(C / G, 4 * scan::Layout<16>::NT / N); }

// Pieces of the split form, 1 for the direct one, from the clocks that 16 tokens of a channel
// block cost: the direct form takes as long as its longest sequence, or as all of them on all
// SMs; the split form as one piece, with an SM's other blocks beside it.  Measured at C2048 N16,
// direct and split, forward: T4096 of 1 sequence 322 and 135 us, of 2 322 and 250, of 3 369 and
// 363, of 4 369 and 473; T512 47 and 35; T16384 C64 1257 and 45; T300 C256 29 and 35; T2048 C2048
// N32 162 and 131.  Backward: T4096 of 1 1032 and 561, of 2 1036 and 1079, of 3 1291 and 1568;
// T4096 C1024 of 2 1033 and 516, of 4 1063 and 968, of 6 1299 and 1428; T512 of 1 146 and 98, of
// 2 147 and 164; T4096 C256 1022 and 102; T2048 of 1, C1024 N64 561 and 470, C768 N32 496 and
// 195, C512 N128 514 and 604, C2048 N8 770 and 221.
//
// The lengths of a packed batch are not known here.  Its longest sequence is taken to be 4 times
// the mean, between the two ways to be wrong (direct and split, forward / backward): 8 equal
// sequences of 1024, C1024, run in pieces, 98 and 135 / 348 and 490 us; one of 8192 and 32 of
// 128, C2048, run direct, 658 and 344 / 2137 and 1598 us.
struct SplitCosts {
    double lone, shared, more;   // clocks: alone on an SM, in a full one, the split form's sweeps
    int blocks;                  // that an SM holds
};
constexpr SplitCosts kFwdCosts{2950, 1290, 700, 4};
constexpr SplitCosts bwd_costs(int N) { return N == 64 ? SplitCosts{8300, 4700, 2300, 2} : SplitCosts{7600, 4700, 3550, 2}; }
int scan_pieces(const Seqs& q, int C, int G, int N, const SplitCosts& k) {
    if (q.tokens() <= 0) return 1;
    const double sm_blocks = (double)G * group_blocks(C, G, N) / kSMs;
    const double tiles = q.tokens() / 16.0, mean = tiles / q.N;
    const double longest = q.cu ? (4 * mean < tiles ? 4 * mean : tiles) : mean;
    const long most = std::min<long>(128, q.tokens() / 128);
    const long pieces = std::min(most, (long)(k.blocks / sm_blocks));   // in one wave of blocks
    if (pieces < 2) return 1;
    const double direct = std::max(longest * k.lone, tiles * sm_blocks * k.shared);
    const double split = tiles / pieces * k.blocks * (k.shared + k.more);
    return split < direct ? (int)pieces : 1;
}

// Pieces of whole tiles; they may come out fewer than wanted.
void cut(const Seqs& q, int want, long& piece, int& pieces) {
    if (want < 2) return;
    piece = ceil_div(ceil_div(q.tokens(), want), 32) * 32;
    pieces = (int)ceil_div(q.tokens(), piece);
}

// The forward's cut and workspace (byte offsets).
struct SplitWs {
    long piece = 0;
    int pieces = 1;
    size_t ends = 0, dsum = 0, h0 = 0, total = 0;
};
SplitWs split_ws(const Seqs& q, int C, int G, int N) {
    SplitWs w;
    cut(q, scan_pieces(q, C, G, N, kFwdCosts), w.piece, w.pieces);
    if (w.pieces < 2) return w;
    size_t o = 0;
    auto take = [&](size_t n) { const size_t at = o; o += (n + 255) & ~(size_t)255; return at; };
    w.ends = take((size_t)w.pieces * C * N * 4);
    w.dsum = take((size_t)w.pieces * C * 4);
    w.h0 = take((size_t)q.N * C * N * 4);
    w.total = o;
    return w;
}

// The backward's.
struct ScanWs {
    long piece = 0;
    int pieces = 1;
    size_t ckpt, bc, a, d, ends, back_ends, dsum, total;
};

ScanWs scan_ws(const Seqs& q, int C, int G, int N) {
    ScanWs w{};
    size_t o = 0;
    auto take = [&](size_t n) { const size_t at = o; o += (n + 255) & ~(size_t)255; return at; };
    cut(q, scan_pieces(q, C, G, N, bwd_costs(N)), w.piece, w.pieces);
    const size_t rows = w.pieces > 1 ? w.pieces : q.N;
    w.ckpt = take((size_t)scan::ckpt_slots(q, w.pieces) * C * N * 4);
    w.bc = take((size_t)G * group_blocks(C, G, N) * q.tokens() * 2 * N * 4);
    w.a = take(rows * C * N * 8);
    w.d = take(rows * 2 * C * 8);
    if (w.pieces > 1) {
        w.ends = take((size_t)w.pieces * C * N * 4);
        w.back_ends = take((size_t)w.pieces * C * N * 4);
        w.dsum = take((size_t)w.pieces * C * 4);
    }
    w.total = o;
    return w;
}

template <typename T, class K>
int scan_fwd(const scan::Params& p, cudaStream_t s) {
    const unsigned bx = (unsigned)(p.G * group_blocks(p.C, p.G, p.N));
    if (p.pieces > 1) {
        const dim3 grid(bx, (unsigned)p.pieces);
        if (p.vec) {
            scan::ends_kernel<T, K, true><<<grid, K::NT, 0, s>>>(p);
            scan::split_kernel<T, K, scan::kOutputs, true><<<grid, K::NT, 0, s>>>(p);
        } else {
            scan::ends_kernel<T, K, false><<<grid, K::NT, 0, s>>>(p);
            scan::split_kernel<T, K, scan::kOutputs, false><<<grid, K::NT, 0, s>>>(p);
        }
        return launched();
    }
    const dim3 grid(bx, (unsigned)p.seq.N);
    if (p.vec) scan::fwd_kernel<T, K, scan::kOutputs, true><<<grid, K::NT, 0, s>>>(p);
    else scan::fwd_kernel<T, K, scan::kOutputs, false><<<grid, K::NT, 0, s>>>(p);
    return launched();
}

template <typename T, class K, bool VEC>
int scan_bwd_vec(const scan::Params& p, cudaStream_t s) {
    const dim3 grid((unsigned)(p.G * group_blocks(p.C, p.G, p.N)), (unsigned)(p.pieces > 1 ? p.pieces : p.seq.N));
    constexpr int smem = (int)sizeof(scan::BwdSmem<K>);
    const auto kernel = p.pieces > 1 ? scan::bwd_kernel<T, K, VEC, true> : scan::bwd_kernel<T, K, VEC, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return COMBA_ECUDA;
    if (p.pieces > 1) {
        scan::ends_kernel<T, K, VEC><<<grid, K::NT, 0, s>>>(p);
        scan::split_kernel<T, K, scan::kStates, VEC><<<grid, K::NT, 0, s>>>(p);
        scan::back_ends_kernel<T, K, VEC><<<grid, K::NT, 0, s>>>(p);
    } else {
        scan::fwd_kernel<T, K, scan::kStates, VEC><<<grid, K::NT, 0, s>>>(p);
    }
    kernel<<<grid, K::NT, smem, s>>>(p);
    return launched();
}

template <typename T, class K>
int scan_bwd(const scan::Params& p, cudaStream_t s) {
    return p.vec ? scan_bwd_vec<T, K, true>(p, s) : scan_bwd_vec<T, K, false>(p, s);
}

template <typename T, class K>
int scan_step(const scan::Params& p, cudaStream_t s) {
    const dim3 grid((unsigned)(p.G * group_blocks(p.C, p.G, p.N)), (unsigned)ceil_div(p.seq.N, scan::kStepSeqs));
    scan::step_kernel<T, K><<<grid, K::NT, 0, s>>>(p);
    return launched();
}

template <typename T>
int scan_sums(const scan::Params& p, void* dB, void* dC, float* dA_log, float* dD, float* dbias, cudaStream_t s) {
    const long ids = p.seq.tokens() * p.G * 2 * p.N;
    if (ids)
        scan::sum_bc_kernel<T><<<(unsigned)ceil_div(ids, 256), 256, 0, s>>>(p.part_bc, static_cast<T*>(dB), static_cast<T*>(dC),
                                                                            p.seq, p.G, p.N, group_blocks(p.C, p.G, p.N));
    const long np = (long)p.C * p.N + 2 * p.C;
    scan::sum_params_kernel<<<(unsigned)ceil_div(np, 256), 256, 0, s>>>(p.part_a, p.part_d, p.A_log, dA_log, dD, dbias, p.seq,
                                                                        p.pieces, p.C, p.N);
    return launched();
}

// f<element type, layout> for the runtime values.
#define COMBA_SCAN_N(f, T, N, ...)                                                                                \
    ((N) == 8 ? f<T, scan::Layout<8>>(__VA_ARGS__) : (N) == 16 ? f<T, scan::Layout<16>>(__VA_ARGS__)              \
     : (N) == 32 ? f<T, scan::Layout<32>>(__VA_ARGS__) : (N) == 64 ? f<T, scan::Layout<64>>(__VA_ARGS__)          \
                                                                   : f<T, scan::Layout<128>>(__VA_ARGS__))
#define COMBA_SCAN_DISPATCH(f, dtype, N, ...) \
    ((dtype) == COMBA_BF16 ? COMBA_SCAN_N(f, bf16, N, __VA_ARGS__) : COMBA_SCAN_N(f, float, N, __VA_ARGS__))

// Sizes of a scan: COMBA_OK, or why it is refused.  Without a sequence the groups have to be
// right all the same: the backward goes on there, to zero the parameters' gradients.
int scan_sizes(int nseq, int T, int C, int G, int N, int dtype, size_t tokens) {
    if (nseq < 0 || T < 0 || C < 0 || !states_ok(N) || !dtype_ok(dtype)) return COMBA_EINVAL;
    if (C == 0) return COMBA_OK;
    if (G < 1 || C % G) return COMBA_EINVAL;
    if (nseq == 0) return COMBA_OK;
    if (volume(tokens, C) > kMaxElements || volume(tokens, G, N) > kMaxElements || volume(nseq, C, N) > kMaxElements)
        return COMBA_EINVAL;
    if (nseq > 65535) return COMBA_EUNSUPPORTED;
    return COMBA_OK;
}

}  // namespace

extern "C" size_t comba_selective_scan_fwd_workspace_size(int nseq, int T, int C, int G, int N, int packed) {
    if (nseq <= 0 || T < 0 || C <= 0 || G < 1 || C % G || !states_ok(N)) return 0;
    const int any = 0;
    return split_ws(Seqs{packed ? &any : nullptr, nseq, T}, C, G, N).total;
}

extern "C" int comba_selective_scan_fwd(const void* x, const void* dt, const float* A_log, const void* Bm, const void* Cm,
                                        const float* D, const float* dt_bias, const void* z, const float* h0, void* out,
                                        float* h_final, const int* cu_seqlens, int nseq, int T, int C, int G, int N,
                                        int dtype, void* workspace, size_t workspace_bytes, comba_stream_t stream) {
    const size_t tokens = nseq > 0 && T > 0 ? token_count(cu_seqlens, nseq, T) : 0;
    if (int st = scan_sizes(nseq, T, C, G, N, dtype, tokens)) return st;
    if (nseq == 0 || C == 0) return COMBA_OK;
    const size_t e = elt_size(dtype), nx = tokens * C * e, nb = tokens * G * N * e, ns = (size_t)nseq * C * N * 4;
    const Arg ins[] = {{x, nx, e, false}, {dt, nx, e, false}, {A_log, (size_t)C * N * 4, 16, false}, {Bm, nb, 16, false},
                       {Cm, nb, 16, false}, {D, (size_t)C * 4, 4, true}, {dt_bias, (size_t)C * 4, 4, true},
                       {z, nx, e, true}, {h0 == h_final ? nullptr : h0, ns, 16, true},
                       {cu_seqlens, ((size_t)nseq + 1) * 4, 4, true}};
    const Seqs seq{cu_seqlens, nseq, T};
    const SplitWs ws = split_ws(seq, C, G, N);
    if (workspace_bytes < ws.total) return COMBA_EINVAL;
    const Arg outs[] = {{out, nx, e, false}, {h_final, ns, 16, true}, {workspace, ws.total, 16, false}};
    if (!args_ok(ins, outs)) return COMBA_EINVAL;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    scan::Params p{};
    p.x = x; p.dt = dt; p.A_log = A_log; p.Bm = Bm; p.Cm = Cm; p.D = D; p.dt_bias = dt_bias; p.z = z; p.h0 = h0;
    p.out = out; p.h_final = h_final;
    p.seq = seq;
    p.C = C; p.G = G; p.N = N;
    p.vec = scan_vector(C, G, dtype, {x, dt, z, out});
    p.status = comba::status_word();
    if (!p.status) return COMBA_ECUDA;
    p.piece = ws.piece;
    p.pieces = ws.pieces;
    if (ws.pieces > 1) {
        char* w = static_cast<char*>(workspace);
        p.ends = reinterpret_cast<float*>(w + ws.ends);
        p.dsum = reinterpret_cast<float*>(w + ws.dsum);
        if (h0 && h0 == h_final) {   // one block's final state must not replace another's start
            if (cudaMemcpyAsync(w + ws.h0, h0, ns, cudaMemcpyDeviceToDevice, s) != cudaSuccess) return COMBA_ECUDA;
            p.h0 = reinterpret_cast<const float*>(w + ws.h0);
        }
    }
    return COMBA_SCAN_DISPATCH(scan_fwd, dtype, N, p, s);
}

extern "C" size_t comba_selective_scan_bwd_workspace_size(int nseq, int T, int C, int G, int N, int packed) {
    if (nseq <= 0 || T < 0 || C <= 0 || G < 1 || C % G || !states_ok(N)) return 0;
    const int any = 0;
    return scan_ws(Seqs{packed ? &any : nullptr, nseq, T}, C, G, N).total;
}

extern "C" int comba_selective_scan_bwd(const void* x, const void* dt, const float* A_log, const void* Bm, const void* Cm,
                                        const float* D, const float* dt_bias, const void* z, const float* h0,
                                        const void* dout, const float* dh_final, void* dx, void* ddt, float* dA_log,
                                        void* dBm, void* dCm, float* dD, float* ddt_bias, void* dz, float* dh0,
                                        const int* cu_seqlens, int nseq, int T, int C, int G, int N, int dtype,
                                        void* workspace, size_t workspace_bytes, comba_stream_t stream) {
    const size_t tokens = nseq > 0 && T > 0 ? token_count(cu_seqlens, nseq, T) : 0;
    if (int st = scan_sizes(nseq, T, C, G, N, dtype, tokens)) return st;
    if (C == 0) return COMBA_OK;
    if (nseq == 0) T = 0;   // no sequence covers a token
    if (!z != !dz) return COMBA_EINVAL;
    const size_t e = elt_size(dtype), nx = tokens * C * e, nb = tokens * G * N * e, ns = (size_t)nseq * C * N * 4;
    const size_t na = (size_t)C * N * 4, nc = (size_t)C * 4;
    const size_t need = comba_selective_scan_bwd_workspace_size(nseq, T, C, G, N, cu_seqlens != nullptr);
    if (workspace_bytes < need) return COMBA_EINVAL;
    const Arg ins[] = {{x, nx, e, false}, {dt, nx, e, false}, {A_log, na, 16, false}, {Bm, nb, 16, false},
                       {Cm, nb, 16, false}, {D, nc, 4, true}, {dt_bias, nc, 4, true}, {z, nx, e, true}, {h0, ns, 16, true},
                       {dout, nx, e, false}, {dh_final, ns, 16, true}, {cu_seqlens, ((size_t)nseq + 1) * 4, 4, true}};
    const Arg outs[] = {{dx, nx, e, false}, {ddt, nx, e, false}, {dA_log, na, 4, false}, {dBm, nb, e, false},
                        {dCm, nb, e, false}, {dD, nc, 4, true}, {ddt_bias, nc, 4, true}, {dz, nx, e, true},
                        {dh0, ns, 16, true}, {workspace, need, 16, false}};
    if (!args_ok(ins, outs)) return COMBA_EINVAL;
    scan::Params p{};
    p.x = x; p.dt = dt; p.A_log = A_log; p.Bm = Bm; p.Cm = Cm; p.D = D; p.dt_bias = dt_bias; p.z = z; p.h0 = h0;
    p.dout = dout; p.dh_final = dh_final; p.dx = dx; p.ddt = ddt; p.dz = dz; p.dh0 = dh0;
    p.seq = Seqs{cu_seqlens, nseq, T};
    p.C = C; p.G = G; p.N = N;
    p.vec = scan_vector(C, G, dtype, {x, dt, z, dout, dx, ddt, dz});
    char* w = static_cast<char*>(workspace);
    const ScanWs ws = scan_ws(p.seq, C, G, N);
    p.ckpt = reinterpret_cast<float*>(w + ws.ckpt);
    p.part_bc = reinterpret_cast<float*>(w + ws.bc);
    p.part_a = reinterpret_cast<double*>(w + ws.a);
    p.part_d = reinterpret_cast<double*>(w + ws.d);
    p.piece = ws.piece;
    p.pieces = ws.pieces;
    if (ws.pieces > 1) {
        p.ends = reinterpret_cast<float*>(w + ws.ends);
        p.back_ends = reinterpret_cast<float*>(w + ws.back_ends);
        p.dsum = reinterpret_cast<float*>(w + ws.dsum);
    }
    p.status = comba::status_word();
    if (!p.status) return COMBA_ECUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (nseq > 0)
        if (int st = COMBA_SCAN_DISPATCH(scan_bwd, dtype, N, p, s)) return st;
    return dtype == COMBA_BF16 ? scan_sums<bf16>(p, dBm, dCm, dA_log, dD, ddt_bias, s)
                               : scan_sums<float>(p, dBm, dCm, dA_log, dD, ddt_bias, s);
}

extern "C" int comba_selective_scan_step(const void* x, const void* dt, const float* A_log, const void* Bm, const void* Cm,
                                         const float* D, const float* dt_bias, const void* z, float* h, void* out, int B,
                                         int C, int G, int N, int dtype, comba_stream_t stream) {
    if (int st = scan_sizes(B, 1, C, G, N, dtype, B > 0 ? (size_t)B : 0)) return st;
    if (B == 0 || C == 0) return COMBA_OK;
    const size_t e = elt_size(dtype), nx = (size_t)B * C * e, nb = (size_t)B * G * N * e, ns = (size_t)B * C * N * 4;
    const Arg ins[] = {{x, nx, e, false}, {dt, nx, e, false}, {A_log, (size_t)C * N * 4, 16, false}, {Bm, nb, 16, false},
                       {Cm, nb, 16, false}, {D, (size_t)C * 4, 4, true}, {dt_bias, (size_t)C * 4, 4, true}, {z, nx, e, true}};
    const Arg outs[] = {{h, ns, 16, false}, {out, nx, e, false}};
    if (!args_ok(ins, outs)) return COMBA_EINVAL;
    scan::Params p{};
    p.x = x; p.dt = dt; p.A_log = A_log; p.Bm = Bm; p.Cm = Cm; p.D = D; p.dt_bias = dt_bias; p.z = z;
    p.out = out; p.h_final = h;
    p.seq = Seqs{nullptr, B, 1};
    p.C = C; p.G = G; p.N = N;
    return COMBA_SCAN_DISPATCH(scan_step, dtype, N, p, reinterpret_cast<cudaStream_t>(stream));
}

// ------------------------------------------------------------------ norms
namespace {

int norm_sizes(long long rows, int D, int dtype, float eps) {
    if (rows < 0 || D < 0 || !dtype_ok(dtype) || !(eps >= 0.f)) return COMBA_EINVAL;
    if (volume((size_t)rows, D) > kMaxElements) return COMBA_EINVAL;
    if (D > norm::kMaxWidth) return COMBA_EUNSUPPORTED;
    return COMBA_OK;
}

template <typename T, bool VECTOR>
int gated_fwd(const norm::Gated& p, cudaStream_t s) {
    const int threads = norm::block_threads(p.tpr);
    const unsigned blocks = (unsigned)norm::fwd_blocks(p.rows, p.tpr);
    if (threads <= 512) norm::gated_fwd_kernel<T, VECTOR, 512><<<blocks, threads, 0, s>>>(p);
    else norm::gated_fwd_kernel<T, VECTOR, 1024><<<blocks, threads, 0, s>>>(p);
    return launched();
}

template <typename T, bool VECTOR>
int gated_bwd(const norm::Gated& p, unsigned blocks, cudaStream_t s) {
    const int threads = norm::block_threads(p.tpr);
    const size_t smem = threads > p.tpr ? (size_t)threads * 8 * sizeof(float) : 0;
    if (threads <= 256) norm::gated_bwd_kernel<T, VECTOR, 256><<<blocks, threads, smem, s>>>(p);
    else if (threads <= 512) norm::gated_bwd_kernel<T, VECTOR, 512><<<blocks, threads, smem, s>>>(p);
    else norm::gated_bwd_kernel<T, VECTOR, 1024><<<blocks, threads, smem, s>>>(p);
    return launched();
}

template <typename T, typename TR, bool VECTOR, bool POST>
int residual_fwd_post(const norm::Residual& p, cudaStream_t s) {
    const int threads = norm::block_threads(p.tpr);
    const unsigned blocks = (unsigned)norm::fwd_blocks(p.rows, p.tpr);
    if (threads <= 512) norm::residual_fwd_kernel<T, TR, VECTOR, POST, 512><<<blocks, threads, 0, s>>>(p);
    else norm::residual_fwd_kernel<T, TR, VECTOR, POST, 1024><<<blocks, threads, 0, s>>>(p);
    return launched();
}

template <typename T, typename TR, bool VECTOR>
int residual_fwd(const norm::Residual& p, cudaStream_t s) {
    return p.post ? residual_fwd_post<T, TR, VECTOR, true>(p, s) : residual_fwd_post<T, TR, VECTOR, false>(p, s);
}

template <typename T, typename TR, bool VECTOR, bool POST>
int residual_bwd_post(const norm::Residual& p, unsigned blocks, cudaStream_t s) {
    const int threads = norm::block_threads(p.tpr);
    const size_t smem = threads > p.tpr ? (size_t)threads * 8 * sizeof(float) : 0;
    if (threads <= 256) norm::residual_bwd_kernel<T, TR, VECTOR, POST, 256><<<blocks, threads, smem, s>>>(p);
    else if (threads <= 512) norm::residual_bwd_kernel<T, TR, VECTOR, POST, 512><<<blocks, threads, smem, s>>>(p);
    else norm::residual_bwd_kernel<T, TR, VECTOR, POST, 1024><<<blocks, threads, smem, s>>>(p);
    return launched();
}

template <typename T, typename TR, bool VECTOR>
int residual_bwd(const norm::Residual& p, unsigned blocks, cudaStream_t s) {
    return p.post ? residual_bwd_post<T, TR, VECTOR, true>(p, blocks, s)
                  : residual_bwd_post<T, TR, VECTOR, false>(p, blocks, s);
}

#define COMBA_RESIDUAL_DISPATCH(f, dtype, rdtype, vec, ...)                                                    \
    ((dtype) == COMBA_BF16                                                                                     \
         ? ((rdtype) == COMBA_BF16 ? ((vec) ? f<bf16, bf16, true>(__VA_ARGS__) : f<bf16, bf16, false>(__VA_ARGS__)) \
                                   : ((vec) ? f<bf16, float, true>(__VA_ARGS__) : f<bf16, float, false>(__VA_ARGS__))) \
         : ((vec) ? f<float, float, true>(__VA_ARGS__) : f<float, float, false>(__VA_ARGS__)))

}  // namespace

extern "C" int comba_gated_norm_fwd(const void* x, const void* gate, const float* weight, void* out, long long rows, int D,
                                    float eps, int dtype, comba_stream_t stream) {
    if (int st = norm_sizes(rows, D, dtype, eps)) return st;
    if (rows == 0 || D == 0) return COMBA_OK;
    const size_t e = elt_size(dtype), nx = (size_t)rows * D * e;
    const Arg ins[] = {{x, nx, e, false}, {gate, nx, e, false}, {weight, (size_t)D * 4, 4, false}};
    const Arg outs[] = {{out, nx, e, false}};
    if (!args_ok(ins, outs)) return COMBA_EINVAL;
    norm::Gated p{};
    p.x = x; p.gate = gate; p.weight = weight; p.out = out;
    p.rows = rows; p.D = D; p.eps = eps; p.inv_d = 1.f / (float)D;
    p.tpr = norm::row_threads(D);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = vector_rows(D, kVec, 16, {x, gate, weight, out});
    if (dtype == COMBA_BF16) return vec ? gated_fwd<bf16, true>(p, s) : gated_fwd<bf16, false>(p, s);
    return vec ? gated_fwd<float, true>(p, s) : gated_fwd<float, false>(p, s);
}

extern "C" size_t comba_gated_norm_bwd_workspace_size(long long rows, int D) {
    if (rows <= 0 || D <= 0 || D > norm::kMaxWidth) return 0;
    return (size_t)norm::bwd_blocks(rows, D, norm::kGatedBlocks) * D * sizeof(float);
}

extern "C" int comba_gated_norm_bwd(const void* x, const void* gate, const float* weight, const void* dout, void* dx,
                                    void* dgate, float* dweight, long long rows, int D, float eps, int dtype,
                                    void* workspace, size_t workspace_bytes, comba_stream_t stream) {
    if (int st = norm_sizes(rows, D, dtype, eps)) return st;
    if (D == 0) return COMBA_OK;
    const size_t e = elt_size(dtype), nx = (size_t)rows * D * e, nw = (size_t)D * 4;
    const size_t need = comba_gated_norm_bwd_workspace_size(rows, D);
    if (workspace_bytes < need) return COMBA_EINVAL;
    const Arg ins[] = {{x, nx, e, false}, {gate, nx, e, false}, {weight, nw, 4, false}, {dout, nx, e, false}};
    const Arg outs[] = {{dx, nx, e, false}, {dgate, nx, e, false}, {dweight, nw, 4, false}, {workspace, need, 16, false}};
    if (!args_ok(ins, outs)) return COMBA_EINVAL;
    norm::Gated p{};
    p.x = x; p.gate = gate; p.weight = weight; p.dout = dout; p.dx = dx; p.dgate = dgate;
    p.part = static_cast<float*>(workspace);
    p.rows = rows; p.D = D; p.eps = eps; p.inv_d = 1.f / (float)D;
    p.tpr = norm::row_threads(D);
    const long blocks = rows > 0 ? norm::bwd_blocks(rows, D, norm::kGatedBlocks) : 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = vector_rows(D, kVec, 16, {x, gate, weight, dout, dx, dgate});
    if (blocks) {
        const int st = dtype == COMBA_BF16 ? (vec ? gated_bwd<bf16, true>(p, (unsigned)blocks, s) : gated_bwd<bf16, false>(p, (unsigned)blocks, s))
                                           : (vec ? gated_bwd<float, true>(p, (unsigned)blocks, s) : gated_bwd<float, false>(p, (unsigned)blocks, s));
        if (st) return st;
    }
    sum_rows_kernel<<<(unsigned)ceil_div(D, 32), 256, 0, s>>>(SumRows{p.part, {dweight}, blocks, D});
    return launched();
}

extern "C" int comba_residual_norm_fwd(const void* x, const void* residual, const float* weight, const float* scale,
                                       const float* post_weight, void* out, void* h, long long rows, int D, float eps,
                                       int dtype, int residual_dtype, comba_stream_t stream) {
    if (int st = norm_sizes(rows, D, dtype, eps)) return st;
    if (residual_dtype != COMBA_F32 && residual_dtype != dtype) return COMBA_EINVAL;
    if (rows == 0 || D == 0) return COMBA_OK;
    const size_t e = elt_size(dtype), er = elt_size(residual_dtype), n = (size_t)rows * D, nw = (size_t)D * 4;
    const Arg ins[] = {{x, n * e, e, false}, {residual == h ? nullptr : residual, residual == h ? 0 : n * er, er, false},
                       {weight, nw, 4, false}, {scale, nw, 4, true}, {post_weight, nw, 4, true}};
    const Arg outs[] = {{out, n * e, e, false}, {h, n * er, er, false}};
    if (!args_ok(ins, outs)) return COMBA_EINVAL;
    norm::Residual p{};
    p.x = x; p.residual = residual; p.weight = weight; p.scale = scale; p.post = post_weight; p.out = out; p.h = h;
    p.rows = rows; p.D = D; p.eps = eps; p.inv_d = 1.f / (float)D;
    p.tpr = norm::row_threads(D);
    const bool vec = vector_rows(D, kVec, 16, {x, residual, weight, scale, post_weight, out, h});
    return COMBA_RESIDUAL_DISPATCH(residual_fwd, dtype, residual_dtype, vec, p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t comba_residual_norm_bwd_workspace_size(long long rows, int D) {
    if (rows <= 0 || D <= 0 || D > norm::kMaxWidth) return 0;
    return 3 * (size_t)norm::bwd_blocks(rows, D, norm::kResidualBlocks) * D * sizeof(float);
}

extern "C" int comba_residual_norm_bwd(const void* x, const void* h, const float* weight, const float* scale,
                                       const float* post_weight, const void* dy, const void* dh, void* dx, void* dresidual,
                                       float* dweight, float* dscale, float* dpost_weight, long long rows, int D, float eps,
                                       int dtype, int residual_dtype, void* workspace, size_t workspace_bytes,
                                       comba_stream_t stream) {
    if (int st = norm_sizes(rows, D, dtype, eps)) return st;
    if (residual_dtype != COMBA_F32 && residual_dtype != dtype) return COMBA_EINVAL;
    if ((dscale && !scale) || (dpost_weight && !post_weight)) return COMBA_EINVAL;
    if (D == 0) return COMBA_OK;
    const size_t e = elt_size(dtype), er = elt_size(residual_dtype), n = (size_t)rows * D, nw = (size_t)D * 4;
    const size_t need = comba_residual_norm_bwd_workspace_size(rows, D);
    if (workspace_bytes < need) return COMBA_EINVAL;
    const Arg ins[] = {{x, n * e, e, false}, {h, n * er, er, false}, {weight, nw, 4, false}, {scale, nw, 4, true},
                       {post_weight, nw, 4, true}, {dy, n * e, e, false}, {dh, n * er, er, true}};
    const Arg outs[] = {{dx, n * e, e, false}, {dresidual, n * er, er, false}, {dweight, nw, 4, false}, {dscale, nw, 4, true},
                        {dpost_weight, nw, 4, true}, {workspace, need, 16, false}};
    if (!args_ok(ins, outs)) return COMBA_EINVAL;
    norm::Residual p{};
    p.x = x; p.h_in = h; p.weight = weight; p.scale = scale; p.post = post_weight; p.dy = dy; p.dh = dh;
    p.dx = dx; p.dres = dresidual;
    p.part = static_cast<float*>(workspace);
    p.rows = rows; p.D = D; p.eps = eps; p.inv_d = 1.f / (float)D;
    p.tpr = norm::row_threads(D);
    const long blocks = rows > 0 ? norm::bwd_blocks(rows, D, norm::kResidualBlocks) : 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = vector_rows(D, kVec, 16, {x, h, weight, scale, post_weight, dy, dh, dx, dresidual});
    if (blocks)
        if (int st = COMBA_RESIDUAL_DISPATCH(residual_bwd, dtype, residual_dtype, vec, p, (unsigned)blocks, s)) return st;
    sum_rows_kernel<<<dim3((unsigned)ceil_div(D, 32), 3), 256, 0, s>>>(
        SumRows{p.part, {dweight, dscale, dpost_weight}, blocks, D});
    return launched();
}
