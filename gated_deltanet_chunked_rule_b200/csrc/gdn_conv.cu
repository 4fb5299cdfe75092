// gdn_conv.cu -- short causal convolution, depthwise over the channels, with an
// optional silu: the step in front of a recurrence's q, k, v (or x, B, C).
//
// Per sequence (W taps, the W-1 inputs before its first token in a state row each):
//
//   pre_t = bias + sum_j weight_j x_{t-W+1+j},     y_t = pre_t  or  pre_t sigmoid(pre_t)
//   dpre_t = dy_t (dy/dpre),   dx_t = sum_j weight_j dpre_{t+W-1-j},
//   dweight_j = sum_t dpre_t x_{t-W+1+j},          dbias = sum_t dpre_t
//
// A warp owns 32 x 16 bytes of channels (8 in the backward) and a run of tokens; the last W-1
// inputs stay in registers, so that every row is read once per run (plus W-1 rows of overlap).
// Rows come in batches of eight (four in the backward, with dy's) that are loaded together and
// worked off, two channels per instruction, without a branch while they lie in one sequence; a
// batch that meets a border goes row by row. The backward recomputes pre, and holds dpre of the
// last W-1 tokens. The weight's gradient sums in fp32: over a run in registers, over a block's
// runs in shared memory, over blocks by a second kernel in a fixed order. The runs are as long as
// lets every block be resident at once.
//
// The bytes: forward reads x and writes y, backward reads x and dy and writes dx. What bounds it are
// the rows in flight: they stand in registers, 128 a thread and so 16 warps on an SM, which issue in
// 36 (forward) and 46 % of the cycles and mostly wait for their rows in the others; the work is 17
// and 30 instructions per element. 8192 tokens of 8192 channels forward 60 us (42 by the copy rate), of
// 4352 channels backward 68 us (33). One channel per instruction and runs of 32 tokens: backward 89 us.
// Tried and slower: the next batch loaded ahead into registers (81 us), two channels per thread and
// twice the warps (88 us). Widths or strides off 16 bytes take one channel per thread: 8191 channels
// forward 148 us, 4351 backward 190.
#include <algorithm>

#include "gdn_host.cuh"
#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;   // runs per block
constexpr int kResident = 4;  // blocks of an SM
constexpr int kMinRun = 8;  // tokens
constexpr int kAhead = 8;   // rows loaded together
constexpr int kAheadB = 4;  // (each of x and dy) in the backward

struct ConvP {
    SeqMap m;
    int C, run, runs;  // tokens of a run
    bool silu;
    long long xs;
};

// VEC consecutive channels of a row as loaded: two or four words of one or two elements (or one
// element).
template <typename T, int VEC>
struct Pack {
    static constexpr int kWords = VEC == 1 ? 1 : VEC * (int)sizeof(T) / 4, kPer = VEC / kWords;
    static constexpr int kPairs = VEC == 1 ? 1 : VEC / 2;  // of channels, worked on together (one channel: beside a zero)
    uint32_t w[kWords];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < kWords; ++k) w[k] = 0;
    }
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VEC == 1) {
            w[0] = __float_as_uint(to_f32(*p));
        } else if constexpr (kWords == 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        } else {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (VEC == 1) *p = from_f32<T>(__uint_as_float(w[0]));
        else if constexpr (kWords == 2) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ float get(int k, int e) const {
        if constexpr (kPer == 1) return __uint_as_float(w[k]);
        return __uint_as_float(e ? w[k] & 0xffff0000u : w[k] << 16);
    }
    __device__ __forceinline__ F2 pair(int m) const {
        if constexpr (VEC == 1) return f2(w[0], 0u);
        else if constexpr (kPer == 1) return f2(w[2 * m], w[2 * m + 1]);
        else return f2(w[m] << 16, w[m] & 0xffff0000u);
    }
    __device__ __forceinline__ void put(int m, F2 v) {
        const float2 a = gdn::get(v);
        if constexpr (VEC == 1) {
            w[0] = __float_as_uint(a.x);
        } else if constexpr (kPer == 1) {
            w[2 * m] = __float_as_uint(a.x), w[2 * m + 1] = __float_as_uint(a.y);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
            w[m] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
};

// The taps and bias of VEC channels, contiguous in memory.
template <typename T, int VEC, int W>
struct Taps {
    using P = Pack<T, VEC>;
    P w[W], b;
    __device__ __forceinline__ void load(const T *weight, const T *bias, int c) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j].load(weight + (size_t)c * W + j * VEC);
        b.zero();
        if (bias) b.load(bias + c);
    }
    // tap j of element e of word k: element (k * kPer + e) * W + j of the piece sequence
    __device__ __forceinline__ float tap(int k, int e, int j) const {
        const int i = (k * P::kPer + e) * W + j;
        return w[i / VEC].get(i % VEC / P::kPer, i % P::kPer);
    }
    __device__ __forceinline__ F2 pair(int m, int j) const {
        if constexpr (VEC == 1) return f2(tap(0, 0, j), 0.f);
        else return f2(tap(2 * m / P::kPer, 0, j), tap((2 * m + 1) / P::kPer, 1 % P::kPer, j));
    }
};

// Input row i of sequence n counted from its first state row: the state's rows, then x.
template <typename T, int VEC, int W>
__device__ __forceinline__ void seen_row(const ConvP &p, const T *x, const T *state, int n, int s, int i, int c, Pack<T, VEC> &v) {
    if (i >= W - 1) v.load(x + (size_t)(s + i - (W - 1)) * p.xs + c);
    else if (state) v.load(state + ((size_t)n * (W - 1) + i) * p.C + c);
    else v.zero();
}

// U outputs in place of U inputs; hist: the W-1 inputs before them, then the last W-1 of them.
template <typename T, int VEC, int W, int U>
__device__ __forceinline__ void forward_rows(const Taps<T, VEC, W> &t, bool silu, Pack<T, VEC> (&r)[U], Pack<T, VEC> (&hist)[W - 1]) {
    using P = Pack<T, VEC>;
    P next[W - 1];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) next[i] = U + i >= W - 1 ? r[U + i - (W - 1) < 0 ? 0 : U + i - (W - 1)] : hist[U + i < W - 1 ? U + i : 0];
#pragma unroll
    for (int m = 0; m < P::kPairs; ++m) {
        F2 x[W - 1 + U], w[W];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) x[i] = hist[i].pair(m);
#pragma unroll
        for (int u = 0; u < U; ++u) x[W - 1 + u] = r[u].pair(m);
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = t.pair(m, j);
        const F2 b = t.b.pair(m);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            F2 a = b;
#pragma unroll
            for (int j = 0; j < W; ++j) a = fma2(w[j], x[u + j], a);
            r[u].put(m, silu ? mul2(a, sigmoid<sizeof(T) == 2>(a)) : a);
        }
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) hist[i] = next[i];
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(32 * kWarps, kResident)
conv_fwd_kernel(ConvP p, const T *__restrict__ x, const T *__restrict__ weight, const T *__restrict__ bias,
                const T *__restrict__ state, T *__restrict__ y, T *__restrict__ final_state, unsigned *status) {
    using P = Pack<T, VEC>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_cu(p.m, status, threadIdx.x, blockDim.x);
    const int c = (blockIdx.y * 32 + lane) * VEC;
    if (c >= p.C) return;
    const int run = blockIdx.x * kWarps + warp;
    if (run >= p.runs) {  // the runs behind the tokens': one sequence's final state each
        const int n = run - p.runs;
        if (n >= p.m.N || !final_state) return;
        const int s = p.m.begin(n), len = p.m.end(n) - s;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            P v;
            seen_row<T, VEC, W>(p, x, state, n, s, len + k, c, v);
            v.store(final_state + ((size_t)n * (W - 1) + k) * p.C + c);
        }
        return;
    }
    const int t0 = run * p.run, t1 = min((long long)t0 + p.run, (long long)p.m.total);
    int n = p.m.owner(t0), s = p.m.begin(n), e = p.m.end(n);
    P hist[W - 1];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) seen_row<T, VEC, W>(p, x, state, n, s, max(t0 - s, 0) + i, c, hist[i]);
    Taps<T, VEC, W> taps;
    taps.load(weight, bias, c);
    for (int tb = t0; tb < t1; tb += kAhead) {
        if (tb + kAhead <= min(e, t1)) {  // rows of one sequence
            P r[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) r[u].load(x + (size_t)(tb + u) * p.xs + c);
            forward_rows<T, VEC, W, kAhead>(taps, p.silu, r, hist);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) r[u].store(y + (size_t)(tb + u) * p.C + c);
            continue;
        }
        for (int t = tb; t < min(tb + kAhead, t1); ++t) {
            if (t >= e && n + 1 < p.m.N) {  // the next sequence with tokens begins here
                do ++n, e = p.m.end(n); while (t >= e && n + 1 < p.m.N);
                s = p.m.begin(n);
#pragma unroll
                for (int i = 0; i < W - 1; ++i) seen_row<T, VEC, W>(p, x, state, n, s, i, c, hist[i]);
            }
            P r[1];
            r[0].load(x + (size_t)t * p.xs + c);
            forward_rows<T, VEC, W, 1>(taps, p.silu, r, hist);
            r[0].store(y + (size_t)t * p.C + c);
        }
    }
}

// U tokens: dpre from x and dy, the weight's gradient (ACC), and the finished dx of the
// tokens W-1 earlier, in x's place (plus `add`: the final state's gradient). hist, dh: x and
// dpre of the W-1 tokens before.
template <typename T, int VEC, int W, int U, bool ACC>
__device__ __forceinline__ void backward_rows(const Taps<T, VEC, W> &t, bool silu, Pack<T, VEC> (&r)[U], const Pack<T, VEC> (&dy)[U],
                                              const Pack<T, VEC> &add, Pack<T, VEC> (&hist)[W - 1],
                                              F2 (&dh)[W - 1][Pack<T, VEC>::kPairs], F2 (&dw)[W][Pack<T, VEC>::kPairs],
                                              F2 (&db)[Pack<T, VEC>::kPairs]) {
    using P = Pack<T, VEC>;
    P next[W - 1];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) next[i] = U + i >= W - 1 ? r[U + i - (W - 1) < 0 ? 0 : U + i - (W - 1)] : hist[U + i < W - 1 ? U + i : 0];
    const F2 one = f2(1.f, 1.f), minus = f2(-1.f, -1.f);
#pragma unroll
    for (int m = 0; m < P::kPairs; ++m) {
        F2 x[W - 1 + U], d[W - 1 + U], w[W];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) x[i] = hist[i].pair(m), d[i] = dh[i][m];
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = t.pair(m, j);
        const F2 b = t.b.pair(m);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[W - 1 + u] = r[u].pair(m);
            F2 g = dy[u].pair(m);
            if (silu) {
                F2 a = b;
#pragma unroll
                for (int j = 0; j < W; ++j) a = fma2(w[j], x[u + j], a);
                const F2 s = sigmoid<sizeof(T) == 2>(a);
                g = mul2(g, fma2(mul2(a, s), fma2(s, minus, one), s));
            }
            d[W - 1 + u] = g;
            if (ACC) {
                db[m] = add2(db[m], g);
#pragma unroll
                for (int j = 0; j < W; ++j) dw[j][m] = fma2(g, x[u + j], dw[j][m]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            F2 a = U == 1 ? add.pair(m) : f2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < W; ++j) a = fma2(w[j], d[u + W - 1 - j], a);
            r[u].put(m, a);
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) dh[i][m] = d[U + i];
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) hist[i] = next[i];
}

template <typename T, int VEC, int W, int UB>
__global__ void __launch_bounds__(32 * kWarps, kResident)
conv_bwd_kernel(ConvP p, const T *__restrict__ x, const T *__restrict__ weight, const T *__restrict__ bias,
                const T *__restrict__ state, const T *__restrict__ dy, const T *__restrict__ dfinal, T *__restrict__ dx,
                float *__restrict__ part, unsigned *status) {
    let_next_start();
    using P = Pack<T, VEC>;
    constexpr int U = UB;
    __shared__ float red[kWarps][(W + 1) * VEC][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_cu(p.m, status, threadIdx.x, blockDim.x);
    const int c = (blockIdx.y * 32 + lane) * VEC;
    const int run = blockIdx.x * kWarps + warp;
    const int t0 = run < p.runs ? run * p.run : 0, t1 = run < p.runs ? min((long long)t0 + p.run, (long long)p.m.total) : 0;
    F2 dw[W][P::kPairs], db[P::kPairs], dh[W - 1][P::kPairs];
#pragma unroll
    for (int m = 0; m < P::kPairs; ++m) {
        db[m] = f2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][m] = f2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) dh[i][m] = f2(0.f, 0.f);
    }
    if (c < p.C && t0 < t1) {
        int n = p.m.owner(t0), s = p.m.begin(n), e = p.m.end(n);
        P hist[W - 1];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) seen_row<T, VEC, W>(p, x, state, n, s, max(t0 - s, 0) + i, c, hist[i]);
        Taps<T, VEC, W> taps;
        taps.load(weight, bias, c);
        // token t's part of the final state's gradient
        auto final_part = [&](int t) {
            P f;
            f.zero();
            const long long k = kept_row(n, e, t, W - 1);
            if (dfinal && t >= max(t0, s) && t < t1 && k >= 0) f.load(dfinal + (size_t)k * p.C + c);
            return f;
        };
        auto emit = [&](int t, const P &v) {  // token t is finished, if it is of this sequence and run
            if (t >= max(t0, s) && t < t1) v.store(dx + (size_t)t * p.C + c);
        };
        // the last W-1 tokens before t: nothing later reaches them
        auto flush = [&](int t) {
            P none[1], zero[1];
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                none[0].zero(), zero[0].zero();
                F2 keep[W][P::kPairs], kb[P::kPairs];
                backward_rows<T, VEC, W, 1, false>(taps, false, none, zero, final_part(t - (W - 1) + i), hist, dh, keep, kb);
                emit(t - (W - 1) + i, none[0]);
            }
        };
        const int tend = min(t1 + W - 1, p.m.total);
        bool done = false;
        int t = t0;
        while (t < tend && !done) {
            if (t + U <= e && (t + U <= t1 || t >= t1)) {  // behind the run (t >= t1) for the last dx only
                P r[U], d[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    r[u].load(x + (size_t)(t + u) * p.xs + c);
                    d[u].load(dy + (size_t)(t + u) * p.C + c);
                }
                if (t < t1) {
                    backward_rows<T, VEC, W, U, true>(taps, p.silu, r, d, r[0], hist, dh, dw, db);
                } else {
                    F2 keep[W][P::kPairs], kb[P::kPairs];
                    backward_rows<T, VEC, W, U, false>(taps, p.silu, r, d, r[0], hist, dh, keep, kb);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {  // W-1 <= U: these all lie before e - (W-1)
                    const int te = t - (W - 1) + u;
                    if (te >= t0 && te >= s && te < t1) r[u].store(dx + (size_t)te * p.C + c);
                }
                t += U;
                continue;
            }
            if (t >= e && n + 1 < p.m.N) {  // a sequence ends
                flush(t);
                if (t >= t1) {
                    done = true;
                    break;
                }
                do ++n, e = p.m.end(n); while (t >= e && n + 1 < p.m.N);
                s = p.m.begin(n);
#pragma unroll
                for (int i = 0; i < W - 1; ++i) seen_row<T, VEC, W>(p, x, state, n, s, i, c, hist[i]);
            }
            P r[1], d[1];
            r[0].load(x + (size_t)t * p.xs + c);
            d[0].load(dy + (size_t)t * p.C + c);
            if (t < t1) {
                backward_rows<T, VEC, W, 1, true>(taps, p.silu, r, d, final_part(t - (W - 1)), hist, dh, dw, db);
            } else {
                F2 keep[W][P::kPairs], kb[P::kPairs];
                backward_rows<T, VEC, W, 1, false>(taps, p.silu, r, d, final_part(t - (W - 1)), hist, dh, keep, kb);
            }
            emit(t - (W - 1), r[0]);
            ++t;
        }
        if (!done) flush(t);
    }
#pragma unroll
    for (int m = 0; m < P::kPairs; ++m) {
#pragma unroll
        for (int j = 0; j <= W; ++j) {
            const float2 v = get(j < W ? dw[j < W ? j : 0][m] : db[m]);
            red[warp][j * VEC + 2 * m][lane] = v.x;
            if (VEC > 1) red[warp][j * VEC + 2 * m + 1][lane] = v.y;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * VEC * 32; i += blockDim.x) {
        const int cl = i % (VEC * 32), j = i / (VEC * 32);  // channel within the block, tap
        const int ch = blockIdx.y * 32 * VEC + cl;
        if (ch >= p.C) continue;
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) v += red[k][j * VEC + cl % VEC][cl / VEC];
        part[((size_t)blockIdx.x * (W + 1) + j) * p.C + ch] = v;
    }
}

// Sums the blocks' parts of dweight [C, W] and dbias [C] in a fixed order: 8 threads per
// value, each over every eighth block.
template <typename T>
__global__ void __launch_bounds__(256) conv_dw_kernel(const float *__restrict__ part, int blocks, int C, int W, T *dweight, T *dbias) {
    wait_for_previous();
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, j = blockIdx.y;
    float v = 0.f;
    if (c < C)
        for (int k = row; k < blocks; k += 8) v += part[((size_t)k * (W + 1) + j) * C + c];
    red[row][lane] = v;
    __syncthreads();
    if (row || c >= C) return;
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += red[k][lane];
    if (j < W) dweight[(size_t)c * W + j] = from_f32<T>(v);
    else if (dbias) dbias[c] = from_f32<T>(v);
}

// Gradient of the state rows: row i meets tap j in token i - j.
template <typename T, int W>
__global__ void __launch_bounds__(128)
conv_dstate_kernel(ConvP p, const T *__restrict__ x, const T *__restrict__ weight, const T *__restrict__ bias,
                   const T *__restrict__ state, const T *__restrict__ dy, const T *__restrict__ dfinal, T *__restrict__ dstate) {
    const int c = blockIdx.y * 128 + threadIdx.x, n = blockIdx.x;
    if (c >= p.C) return;
    const int s = p.m.begin(n), len = p.m.end(n) - s;
    float d[W - 1];
    Taps<T, 1, W> taps;
    taps.load(weight, bias, c);
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        d[t] = 0.f;
        if (t >= len) continue;
        d[t] = to_f32(dy[(size_t)(s + t) * p.C + c]);
        if (!p.silu) continue;
        float a = taps.b.get(0, 0);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            Pack<T, 1> v;
            seen_row<T, 1, W>(p, x, state, n, s, t + j, c, v);
            a = fmaf(taps.tap(0, 0, j), v.get(0, 0), a);
        }
        const float g = sigmoid<sizeof(T) == 2>(a);
        d[t] *= fmaf(a, g - g * g, g);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j <= i; ++j) v = fmaf(taps.tap(0, 0, j), d[i - j], v);
        if (dfinal && i >= len) v += to_f32(dfinal[((size_t)n * (W - 1) + i - len) * p.C + c]);
        dstate[((size_t)n * (W - 1) + i) * p.C + c] = from_f32<T>(v);
    }
}

// A few tokens per sequence, the state updated in place.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(128)
conv_update_kernel(ConvP p, const T *__restrict__ x, const T *__restrict__ weight, const T *__restrict__ bias, T *__restrict__ state,
                   T *__restrict__ y) {
    const int c = (blockIdx.y * 128 + threadIdx.x) * VEC, n = blockIdx.x;
    if (c >= p.C) return;
    using P = Pack<T, VEC>;
    P hist[W - 1];
    T *st = state + (size_t)n * (W - 1) * p.C + c;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) hist[i].load(st + (size_t)i * p.C);
    Taps<T, VEC, W> taps;
    taps.load(weight, bias, c);
    for (int t = 0; t < p.m.T; ++t) {
        const size_t tok = (size_t)n * p.m.T + t;
        P r[1];
        r[0].load(x + tok * p.xs + c);
        forward_rows<T, VEC, W, 1>(taps, p.silu, r, hist);
        r[0].store(y + tok * p.C + c);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) hist[i].store(st + (size_t)i * p.C);
}

// Of a call without tokens: the offsets' check alone.
__global__ void __launch_bounds__(128) conv_offsets_kernel(SeqMap m, unsigned *status) { check_cu(m, status, threadIdx.x, 128); }

// Blocks along the tokens (without the final states'): as many as run beside each other, with
// runs of one length, or one wave more would stand half empty.
int token_blocks(int total, unsigned column_blocks) {
    return std::max(1, std::min((total + kMinRun * kWarps - 1) / (kMinRun * kWarps), (int)(kResident * sm_count() / column_blocks)));
}

enum Pass { kFwd, kBwd, kUpdate };

template <typename T, int VEC, int W, Pass PASS>
cudaError_t run_pass(const ConvArgs &a) {
    ConvP p{a.seq, a.C, 0, 0, a.silu, a.x_stride};
    const T *x = (const T *)a.x, *w = (const T *)a.weight, *b = (const T *)a.bias, *st = (const T *)a.state;
    const unsigned cb = (unsigned)((a.C + 32 * VEC - 1) / (32 * VEC));
    const int share = token_blocks(a.seq.total, cb) * kWarps;
    p.run = std::max(kMinRun, ((a.seq.total + share - 1) / share + 7) / 8 * 8);
    p.runs = (a.seq.total + p.run - 1) / p.run;
    if (a.seq.total == 0 && a.seq.cu) conv_offsets_kernel<<<1, 128, 0, a.stream>>>(a.seq, a.status);
    if constexpr (PASS == kFwd) {
        const long long runs = (long long)p.runs + (a.final_state ? a.seq.N : 0);
        if (runs == 0) return cudaGetLastError();
        conv_fwd_kernel<T, VEC, W><<<dim3((unsigned)((runs + kWarps - 1) / kWarps), cb), 32 * kWarps, 0, a.stream>>>(
            p, x, w, b, st, (T *)a.y, (T *)a.final_state, a.status);
    } else if constexpr (PASS == kBwd) {
        const T *dy = (const T *)a.dy, *df = (const T *)a.dfinal;
        const int blocks = (p.runs + kWarps - 1) / kWarps;
        if (blocks) {
            TimedLaunch tl("conv_bwd", a.stream);
            conv_bwd_kernel<T, VEC, W, kAheadB><<<dim3(blocks, cb), 32 * kWarps, 0, a.stream>>>(p, x, w, b, st, dy, df, (T *)a.dx, a.part,
                                                                                      a.status);
        }
        TimedLaunch tl("conv_bwd_sums", a.stream);
        const cudaError_t e = launch(blocks > 0, conv_dw_kernel<T>, dim3((a.C + 31) / 32, W + 1), dim3(256), 0, a.stream, a.part, blocks, a.C, W,
                                     (T *)a.dweight, (T *)a.dbias);
        if (e != cudaSuccess) return e;
        if (a.dstate)
            conv_dstate_kernel<T, W><<<dim3(a.seq.N, (a.C + 127) / 128), 128, 0, a.stream>>>(p, x, w, b, st, dy, df, (T *)a.dstate);
    } else {
        conv_update_kernel<T, VEC, W><<<dim3(a.seq.N, (a.C + 128 * VEC - 1) / (128 * VEC)), 128, 0, a.stream>>>(
            p, x, w, b, (T *)a.state, (T *)a.y);
    }
    return cudaGetLastError();
}

// 16-byte accesses where every row of every tensor starts on a 16-byte boundary.
bool vectorized(const ConvArgs &a) {
    const int el = a.dtype == GDN_DTYPE_BF16 ? 8 : 4;
    return a.C % el == 0 && a.x_stride % el == 0;
}

template <typename T, int VEC, Pass PASS>
cudaError_t by_taps(const ConvArgs &a) {
    switch (a.W) {
        case 2: return run_pass<T, VEC, 2, PASS>(a);
        case 3: return run_pass<T, VEC, 3, PASS>(a);
        case 4: return run_pass<T, VEC, 4, PASS>(a);
    }
    return cudaErrorInvalidValue;
}

template <Pass PASS>
cudaError_t dispatch(const ConvArgs &a) {
    const bool v = vectorized(a);
    // the backward holds ten registers per channel: four channels per thread let twice as many warps run
    constexpr int kBf16 = PASS == kBwd ? 4 : 8;
    if (a.dtype == GDN_DTYPE_BF16) return v ? by_taps<__nv_bfloat16, kBf16, PASS>(a) : by_taps<__nv_bfloat16, 1, PASS>(a);
    return v ? by_taps<float, 4, PASS>(a) : by_taps<float, 1, PASS>(a);
}

}  // namespace

size_t conv_part_bytes(int total, int C, int W) {
    const size_t blocks = total ? token_blocks(total, (C + 255) / 256) : 0;  // of the widest column blocks: the most
    return blocks * (W + 1) * C * sizeof(float);
}

cudaError_t launch_conv_fwd(const ConvArgs &a) { return dispatch<kFwd>(a); }
cudaError_t launch_conv_bwd(const ConvArgs &a) { return dispatch<kBwd>(a); }
cudaError_t launch_conv_update(const ConvArgs &a) { return dispatch<kUpdate>(a); }

}  // namespace gdn
