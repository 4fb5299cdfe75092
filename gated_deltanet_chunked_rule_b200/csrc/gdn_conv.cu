// gdn_conv.cu -- short causal convolution, depthwise over the channels, with an
// optional silu: the step in front of a recurrence's q, k, v (or x, B, C).
//
// Per sequence (W taps, the W-1 inputs before its first token in a state row each):
//
//   pre_t = bias + sum_j weight_j x_{t-W+1+j},     y_t = pre_t  or  pre_t sigmoid(pre_t)
//   dpre_t = dy_t (dy/dpre),   dx_t = sum_j weight_j dpre_{t+W-1-j},
//   dweight_j = sum_t dpre_t x_{t-W+1+j},          dbias = sum_t dpre_t
//
// Memory-bound: forward reads x and writes y, backward reads x and dy and writes dx. A
// warp owns 32 x 16 bytes of channels and a run of tokens; the last W-1 inputs stay in
// registers, so that every row is read once per run (plus W-1 rows of overlap), eight
// rows in flight. The backward recomputes pre, and holds the unfinished dx of the last
// W-1 tokens in registers the same way. The weight's gradient sums in fp32: over a run in
// registers, over a block's runs in shared memory, over blocks by a second kernel in a
// fixed order.
#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;   // runs per block
constexpr int kRunF = 32;   // tokens of a forward run
constexpr int kRunB = 64;   // tokens of a backward run
constexpr int kAhead = 8;   // rows loaded together

struct ConvP {
    SeqMap m;
    int C, runs;
    bool silu;
    long long xs;
};

// Input row i of sequence n counted from its first state row: the state's rows, then x.
template <typename T, int VEC, int W>
__device__ __forceinline__ void seen_row(const ConvP &p, const T *x, const T *state, int n, int s, int i, int c, float (&v)[VEC]) {
    if (i >= W - 1) {
        load_vec<T, VEC>(x + (size_t)(s + i - (W - 1)) * p.xs + c, v);
    } else if (state) {
        load_vec<T, VEC>(state + ((size_t)n * (W - 1) + i) * p.C + c, v);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = 0.f;
    }
}

template <typename T, int VEC, int W>
__device__ __forceinline__ void load_weight(const T *weight, const T *bias, int c, float (&w)[W][VEC], float (&b)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = to_f32(weight[(size_t)(c + e) * W + j]);
        b[e] = bias ? to_f32(bias[c + e]) : 0.f;
    }
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(32 * kWarps)
conv_fwd_kernel(ConvP p, const T *__restrict__ x, const T *__restrict__ weight, const T *__restrict__ bias,
                const T *__restrict__ state, T *__restrict__ y, T *__restrict__ final_state, unsigned *status) {
    constexpr bool kFast = sizeof(T) == 2;
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
            float v[VEC];
            seen_row<T, VEC, W>(p, x, state, n, s, len + k, c, v);
            store_vec<T, VEC>(final_state + ((size_t)n * (W - 1) + k) * p.C + c, v);
        }
        return;
    }
    const int t0 = run * kRunF, t1 = min(t0 + kRunF, p.m.total);
    float w[W][VEC], b[VEC];
    load_weight<T, VEC, W>(weight, bias, c, w, b);
    int n = p.m.owner(t0), s = p.m.begin(n), e = p.m.end(n);
    float win[W][VEC];  // win[i]: input t - (W-1) + i
#pragma unroll
    for (int i = 0; i < W - 1; ++i) seen_row<T, VEC, W>(p, x, state, n, s, max(t0 - s, 0) + i, c, win[i]);
    for (int tb = t0; tb < t1; tb += kAhead) {
        float in[kAhead][VEC];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (tb + u < t1) load_vec<T, VEC>(x + (size_t)(tb + u) * p.xs + c, in[u]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int t = tb + u;
            if (t >= t1) break;
            if (t >= e && n + 1 < p.m.N) {  // the next sequence with tokens begins here
                do ++n, e = p.m.end(n); while (t >= e && n + 1 < p.m.N);
                s = p.m.begin(n);
#pragma unroll
                for (int i = 0; i < W - 1; ++i) seen_row<T, VEC, W>(p, x, state, n, s, i, c, win[i]);
            }
            float out[VEC];
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                win[W - 1][q] = in[u][q];
                float a = b[q];
#pragma unroll
                for (int j = 0; j < W; ++j) a = fmaf(w[j][q], win[j][q], a);
                out[q] = p.silu ? a * sigmoid<kFast>(a) : a;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j][q] = win[j + 1][q];
            }
            store_vec<T, VEC>(y + (size_t)t * p.C + c, out);
        }
    }
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(32 * kWarps)
conv_bwd_kernel(ConvP p, const T *__restrict__ x, const T *__restrict__ weight, const T *__restrict__ bias,
                const T *__restrict__ state, const T *__restrict__ dy, const T *__restrict__ dfinal, T *__restrict__ dx,
                float *__restrict__ part, unsigned *status) {
    constexpr bool kFast = sizeof(T) == 2;
    __shared__ float red[kWarps][(W + 1) * VEC][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_cu(p.m, status, threadIdx.x, blockDim.x);
    const int c = (blockIdx.y * 32 + lane) * VEC;
    const int run = blockIdx.x * kWarps + warp;
    const int t0 = run * kRunB, t1 = min(t0 + kRunB, p.m.total);
    float dw[W][VEC], db[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        db[q] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][q] = 0.f;
    }
    if (c < p.C && t0 < t1) {
        float w[W][VEC], b[VEC];
        load_weight<T, VEC, W>(weight, bias, c, w, b);
        int n = p.m.owner(t0), s = p.m.begin(n), e = p.m.end(n);
        float win[W][VEC], acc[W][VEC];  // acc[i]: dx of token t - (W-1) + i, unfinished
#pragma unroll
        for (int i = 0; i < W - 1; ++i) seen_row<T, VEC, W>(p, x, state, n, s, max(t0 - s, 0) + i, c, win[i]);
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int q = 0; q < VEC; ++q) acc[i][q] = 0.f;
        auto emit = [&](int t, float (&v)[VEC]) {  // token t is finished, if it is of this sequence and run
            if (t < t0 || t >= t1 || t < s) return;
            if (dfinal && t >= e - (W - 1)) {
                float f[VEC];
                load_vec<T, VEC>(dfinal + ((size_t)n * (W - 1) + (W - 1 - (e - t))) * p.C + c, f);
#pragma unroll
                for (int q = 0; q < VEC; ++q) v[q] += f[q];
            }
            store_vec<T, VEC>(dx + (size_t)t * p.C + c, v);
        };
        const int tend = min(t1 + W - 1, p.m.total);
        int t = t0;
        for (int tb = t0; tb < tend; tb += kAhead / 2) {
            float in[kAhead / 2][VEC], dv[kAhead / 2][VEC];
#pragma unroll
            for (int u = 0; u < kAhead / 2; ++u)
                if (tb + u < tend) {
                    load_vec<T, VEC>(x + (size_t)(tb + u) * p.xs + c, in[u]);
                    load_vec<T, VEC>(dy + (size_t)(tb + u) * p.C + c, dv[u]);
                }
            bool done = false;
#pragma unroll
            for (int u = 0; u < kAhead / 2; ++u) {
                if (tb + u >= tend || done) continue;
                t = tb + u;
                if (t >= e && n + 1 < p.m.N) {  // a sequence ends: its last tokens are finished
#pragma unroll
                    for (int i = 0; i < W - 1; ++i) {
                        emit(t - (W - 1) + i, acc[i]);
#pragma unroll
                        for (int q = 0; q < VEC; ++q) acc[i][q] = 0.f;
                    }
                    if (t >= t1) {
                        done = true;
                        continue;
                    }
                    do ++n, e = p.m.end(n); while (t >= e && n + 1 < p.m.N);
                    s = p.m.begin(n);
#pragma unroll
                    for (int i = 0; i < W - 1; ++i) seen_row<T, VEC, W>(p, x, state, n, s, i, c, win[i]);
                }
                float first[VEC];
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    win[W - 1][q] = in[u][q];
                    float a = b[q], d = dv[u][q];
                    if (p.silu) {
#pragma unroll
                        for (int j = 0; j < W; ++j) a = fmaf(w[j][q], win[j][q], a);
                        const float g = sigmoid<kFast>(a);
                        d *= g * (1.f + a * (1.f - g));
                    }
                    acc[W - 1][q] = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        acc[j][q] = fmaf(w[j][q], d, acc[j][q]);  // token t - (W-1) + j meets tap j in t
                        if (t < t1) dw[j][q] = fmaf(d, win[j][q], dw[j][q]);
                    }
                    if (t < t1) db[q] += d;
                    first[q] = acc[0][q];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        win[j][q] = win[j + 1][q];
                        acc[j][q] = acc[j + 1][q];
                    }
                }
                emit(t - (W - 1), first);  // acc[i] is now token t + 1 - (W-1) + i's
            }
            if (done) {
                t = -1;
                break;
            }
        }
        if (t >= 0) {  // the tokens whose later taps lie behind the last token
#pragma unroll
            for (int i = 0; i < W - 1; ++i) emit(t + 1 - (W - 1) + i, acc[i]);
        }
    }
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
#pragma unroll
        for (int j = 0; j < W; ++j) red[warp][j * VEC + q][lane] = dw[j][q];
        red[warp][W * VEC + q][lane] = db[q];
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
    float w[W][1], b[1], d[W - 1];
    load_weight<T, 1, W>(weight, bias, c, w, b);
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        d[t] = 0.f;
        if (t >= len) continue;
        d[t] = to_f32(dy[(size_t)(s + t) * p.C + c]);
        if (!p.silu) continue;
        float a = b[0];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float v[1];
            seen_row<T, 1, W>(p, x, state, n, s, t + j, c, v);
            a = fmaf(w[j][0], v[0], a);
        }
        const float g = sigmoid<sizeof(T) == 2>(a);
        d[t] *= g * (1.f + a * (1.f - g));
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j <= i; ++j) v = fmaf(w[j][0], d[i - j], v);
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
    float win[W][VEC];
    T *st = state + (size_t)n * (W - 1) * p.C + c;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) load_vec<T, VEC>(st + (size_t)i * p.C, win[i]);
    float w[W][VEC], b[VEC];
    load_weight<T, VEC, W>(weight, bias, c, w, b);
    for (int t = 0; t < p.m.T; ++t) {
        const size_t tok = (size_t)n * p.m.T + t;
        load_vec<T, VEC>(x + tok * p.xs + c, win[W - 1]);
        float out[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
            float a = b[q];
#pragma unroll
            for (int j = 0; j < W; ++j) a = fmaf(w[j][q], win[j][q], a);
            out[q] = p.silu ? a * sigmoid<sizeof(T) == 2>(a) : a;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) win[j][q] = win[j + 1][q];
        }
        store_vec<T, VEC>(y + tok * p.C + c, out);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) store_vec<T, VEC>(st + (size_t)i * p.C, win[i]);
}

enum Pass { kFwd, kBwd, kUpdate };

template <typename T, int VEC, int W>
cudaError_t run_pass(const ConvArgs &a, Pass pass) {
    ConvP p{a.seq, a.C, 0, a.silu, a.x_stride};
    const T *x = (const T *)a.x, *w = (const T *)a.weight, *b = (const T *)a.bias, *st = (const T *)a.state;
    const unsigned cb = (unsigned)((a.C + 32 * VEC - 1) / (32 * VEC));
    if (pass == kFwd) {
        p.runs = (a.seq.total + kRunF - 1) / kRunF;
        const long long runs = (long long)p.runs + (a.final_state ? a.seq.N : 0);
        if (runs == 0) return cudaSuccess;
        conv_fwd_kernel<T, VEC, W><<<dim3((unsigned)((runs + kWarps - 1) / kWarps), cb), 32 * kWarps, 0, a.stream>>>(
            p, x, w, b, st, (T *)a.y, (T *)a.final_state, a.status);
    } else if (pass == kBwd) {
        const T *dy = (const T *)a.dy, *df = (const T *)a.dfinal;
        const int blocks = (a.seq.total + kRunB * kWarps - 1) / (kRunB * kWarps);
        if (blocks)
            conv_bwd_kernel<T, VEC, W><<<dim3(blocks, cb), 32 * kWarps, 0, a.stream>>>(p, x, w, b, st, dy, df, (T *)a.dx, a.part,
                                                                                      a.status);
        conv_dw_kernel<T><<<dim3((a.C + 31) / 32, W + 1), 256, 0, a.stream>>>(a.part, blocks, a.C, W, (T *)a.dweight, (T *)a.dbias);
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

template <typename T, int VEC>
cudaError_t by_taps(const ConvArgs &a, Pass pass) {
    switch (a.W) {
        case 2: return run_pass<T, VEC, 2>(a, pass);
        case 3: return run_pass<T, VEC, 3>(a, pass);
        case 4: return run_pass<T, VEC, 4>(a, pass);
    }
    return cudaErrorInvalidValue;
}

cudaError_t dispatch(const ConvArgs &a, Pass pass) {
    const bool v = vectorized(a);
    if (a.dtype == GDN_DTYPE_BF16)
        return v ? by_taps<__nv_bfloat16, 8>(a, pass) : by_taps<__nv_bfloat16, 1>(a, pass);
    return v ? by_taps<float, 4>(a, pass) : by_taps<float, 1>(a, pass);
}

}  // namespace

size_t conv_part_bytes(int total, int C, int W) {
    const size_t blocks = ((size_t)total + kRunB * kWarps - 1) / (kRunB * kWarps);
    return blocks * (W + 1) * C * sizeof(float);
}

cudaError_t launch_conv_fwd(const ConvArgs &a) { return dispatch(a, kFwd); }
cudaError_t launch_conv_bwd(const ConvArgs &a) { return dispatch(a, kBwd); }
cudaError_t launch_conv_update(const ConvArgs &a) { return dispatch(a, kUpdate); }

}  // namespace gdn
