// gdn_scan_simt.cu -- selective state space scan on the CUDA cores, token by
// token in fp32: the decode step, and every prompt that the tensor-core kernels do not
// take (fp32 inputs, and all under GDN_IMPL=simt).
//
// Per sequence, head (group = head / (H / G)) and token, with the state h [K, P]:
//
//   delta = softplus(dt + dt_bias) (or dt + dt_bias),   a = exp(delta A)
//   h <- a h + (delta B) x^T,    y = C^T h + D x
//
// The gradients run the same recurrence forward once more and the adjoint one back (i_t:
// what comes in from later tokens):
//
//   dC_t = h_t dy_t,   i_t = a_{t+1} g_{t+1},   g_t = C_t dy_t^T + i_t,   u_t = B_t^T g_t
//   dx_t = delta u_t + D dy_t,   dB_t = g_t (delta x_t),   w_t = u_t.x_t
//   d(delta A)_t = a_t <h_{t-1}, g_t>,   ddelta_t = A d(delta A)_t + w_t
//
// <h_{t-1}, g_t> is what crosses token t; within its tile of 16 tokens s < t <= r, with h the state on
// entry to the tile, i what comes in at its end and L, E, F, W the decays from s to r, from the tile's start
// through r, from s to the tile's end and over the tile:
//
//   d(delta A)_t = sum L_rs (C_r.B_s)(dy_r.x_s) delta_s + sum E_r r_r + sum F_s delta_s v_s + W <h, i>
//   with r_r = C_r^T h dy_r and v_s = B_s^T i x_s
//
// Every term is there once and none is taken off again. (The recurrence d(delta A)_t = r'_t - delta_t v'_t +
// d(delta A)_{t+1}, run to the tile's end, sums what does not cross t too and then subtracts it; its roundings
// are shared by the tile's tokens, and dA was off by 2e-6 of its norm where this is off by 3e-7.)
//
// One CTA per (sequence or segment of one, head, 32 columns of P): warp w holds state rows
// 32w .. 32w+31, lane l column l, in registers across its tokens. Where sequences, heads and
// slices are too few to fill the device a sequence is cut into segments: a first pass takes each
// from a zero state (the states alone), a small kernel composes their starts, a second pass
// does the work (1000 tokens, 4 heads of 64 x 64, fp32, forward: 198 us whole, 26 us in segments).
// Tokens come in tiles of 16, the next tile's loads in flight while one is worked on. The decode
// step is memory-bound by its state, in and out once (256 sequences, 64 heads of 128 x 64: 177 us
// for 1.08 GB, 94 % of the copy rate); the prompts are bound by the FMAs and shared-memory reads of
// the 32-row columns, short ones by the tokens' chain.
#include "gdn_host.cuh"
#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr int kCols = 32, kTile = 16, kKeep = kTile;

// Segments of a sequence (a multiple of the tile; longer than any sequence where there is no split).
struct Segments {
    int tokens;
    float *state;  // [slots, H, K, P]: each segment's end, then its start
    float *decay;  // [slots, H]: log decay of a segment
};

struct ScanP {
    SeqMap m;
    Segments seg;
    int G, H, P;
    bool softplus;
    long long xs, bs, cs, dts;
    const float *A, *D, *dt_bias;
};

// log1p(exp(v)), or v itself above 20 (where they agree to fp32 precision).
__device__ __forceinline__ float delta_of(float raw, bool softplus) {
    return softplus ? (raw > 20.f ? raw : log1pf(expf(raw))) : raw;
}

// Sum over the warp's lanes of v[i], delivered to lane i.
__device__ __forceinline__ float lane_sums(float (&v)[32], int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0];
}

// Product of 32 values in shared memory (16-byte aligned) with a column's 32 in registers, two at a time.
__device__ __forceinline__ float row_dot(const float *row, const float (&col)[32]) {
    F2 v[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
        const float4 r = *reinterpret_cast<const float4 *>(row + k);
        v[0] = fma2(f2(r.x, r.y), f2(col[k], col[k + 1]), v[0]);
        v[1] = fma2(f2(r.z, r.w), f2(col[k + 2], col[k + 3]), v[1]);
    }
    const float2 a = get(add2(v[0], v[1]));
    return a.x + a.y;
}

// A tile of tokens in registers on its way to shared memory.
template <typename Tin, typename Tdt, int K>
struct Tile {
    static constexpr int kX = kTile * kCols / K;
    float b[kTile], c[kTile], x[kX], dy[kX], dt;

    // tokens t0 + i (step dir) for i < n; Bm, Cm at this group, x at this head and slice
    template <bool GRAD, bool ENDS = false, bool REV = false>
    __device__ __forceinline__ void load(const ScanP &p, const Tin *x_, const Tdt *dt_, const Tin *B, const Tin *C, const Tin *dy_,
                                         int h, int g, int c0, int t0, int dir, int n, int tid) {
#pragma unroll
        for (int i = 0; i < kTile; ++i) {
            const size_t t = (size_t)(t0 + dir * i);
            if (!(ENDS && REV)) b[i] = i < n ? to_f32(B[t * p.bs + (size_t)g * K + tid]) : 0.f;
            if (!(ENDS && !REV)) c[i] = i < n ? to_f32(C[t * p.cs + (size_t)g * K + tid]) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kX; ++j) {
            const int i = j * (K / kCols) + tid / kCols, col = c0 + tid % kCols;
            const size_t t = (size_t)(t0 + dir * i);
            if (!(ENDS && REV)) x[j] = i < n ? to_f32(x_[t * p.xs + (size_t)h * p.P + col]) : 0.f;
            if (GRAD) dy[j] = i < n ? to_f32(dy_[(t * p.H + h) * p.P + col]) : 0.f;
        }
        dt = 0.f;
        if (tid < n) dt = to_f32(dt_[(size_t)(t0 + dir * tid) * p.dts + h]);
    }
};

template <int K>
struct alignas(16) TileSmem {
    float b[kTile][K], c[kTile][K], x[kTile][kCols], dy[kTile][kCols], a[kTile], d[kTile];
    float red[kTile][K / 32][kCols], red2[kTile][K / 32][kCols];
};

// Per token, head and slice of P: r, v, w as above (r and v by the tile's h and i) and x.dy.
enum Dot { kR, kV, kWt, kXd, kDots };
struct Dots {
    float *at;  // [kDots][total, H, P/32]
    size_t n;
    __device__ __forceinline__ float *operator()(Dot d, size_t i) const { return at + d * n + i; }
};

// Sum over a row's columns of a per-warp partial; every lane of the calling warp gets it.
template <int K>
__device__ __forceinline__ float dot_row(const float (&red)[K / 32][kCols], float other, int lane) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < K / 32; ++k) v += red[k][lane];
    v *= other;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename Tin, typename Tdt, int K, bool GRAD, bool ENDS = false, bool REV = false>
__device__ __forceinline__ void put_tile(TileSmem<K> &s, const Tile<Tin, Tdt, K> &r, const ScanP &p, float A, float bias, int n, int tid) {
#pragma unroll
    for (int i = 0; i < kTile; ++i) {
        if (!(ENDS && REV)) s.b[i][tid] = r.b[i];
        if (!(ENDS && !REV)) s.c[i][tid] = r.c[i];
    }
#pragma unroll
    for (int j = 0; j < Tile<Tin, Tdt, K>::kX; ++j) {
        const int i = j * (K / kCols) + tid / kCols;
        if (!(ENDS && REV)) s.x[i][tid % kCols] = r.x[j];
        if (GRAD) s.dy[i][tid % kCols] = r.dy[j];
    }
    if (tid < n) {
        const float d = delta_of(r.dt + bias, p.softplus);
        s.d[tid] = d;
        s.a[tid] = expf(d * A);
    }
}

// What a CTA walks: segment `local` of sequence n.
struct Walk {
    int n, local, t0, len, s_begin, s_len;
    size_t at;      // this thread's first state element in the user's states
    size_t seg_at;  // and in the segments'
    __device__ __forceinline__ bool find(const ScanP &p, int slot, int h, int K, int row, int col) {
        const bool used = p.m.slot(slot, p.seg.tokens, &n, &local);
        s_begin = p.m.begin(n), s_len = p.m.end(n) - s_begin;
        t0 = s_begin + local * p.seg.tokens;
        len = used ? min(p.seg.tokens, s_begin + s_len - t0) : 0;
        at = (((size_t)n * p.H + h) * K + row) * p.P + col;
        seg_at = (((size_t)slot * p.H + h) * K + row) * p.P + col;
        return used || (local == 0 && s_len == 0);  // an empty sequence keeps its state
    }
    __device__ __forceinline__ bool first() const { return local == 0; }
    __device__ __forceinline__ bool last() const { return t0 + len == s_begin + s_len; }
};

// Forward. GRAD: the gradient's forward half instead: dC parts [total, H, P/32, K], r and x.dy,
// kept states [slots of 16, H, K, P] at each tile's end. ENDS: only the state at the segment's
// end from zero, and its log decay.
template <typename Tin, typename Tdt, int K, bool GRAD, bool ENDS>
__global__ void __launch_bounds__(K)
scan_forward_kernel(ScanP p, const Tin *__restrict__ x, const Tdt *__restrict__ dt, const Tin *__restrict__ B, const Tin *__restrict__ C,
                    const Tin *__restrict__ dy, const float *h0, Tin *__restrict__ y, float *final_state, float *__restrict__ dc_part,
                    float *__restrict__ keep, Dots dots, unsigned *status) {
    __shared__ TileSmem<K> s;
    const int h = blockIdx.y, c0 = blockIdx.z * kCols, g = h / (p.H / p.G);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0 && h == 0 && blockIdx.z == 0) check_cu(p.m, status, tid, K);
    Walk wk;
    if (!wk.find(p, blockIdx.x, h, K, 32 * w, c0 + lane) || (ENDS && (wk.last() || wk.len == 0))) return;
    const int n = wk.n, t0 = wk.t0, len = wk.len;
    const float *src = ENDS ? nullptr : wk.first() ? (h0 ? h0 + wk.at : nullptr) : p.seg.state + wk.seg_at;
    float hr[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) hr[i] = src ? src[(size_t)i * p.P] : 0.f;
    const float A = p.A[h], D = p.D ? p.D[h] : 0.f, bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    const int tile0 = p.m.slot0(n, kKeep) + (t0 - wk.s_begin) / kKeep;
    float total = 0.f;
    Tile<Tin, Tdt, K> r;
    if (len) r.template load<GRAD, ENDS>(p, x, dt, B, C, dy, h, g, c0, t0, 1, min(kTile, len), tid);
    for (int q = 0; q < len; q += kTile) {
        const int cnt = min(kTile, len - q);
        put_tile<Tin, Tdt, K, GRAD, ENDS>(s, r, p, A, bias, cnt, tid);
        __syncthreads();
        if (q + kTile < len) r.template load<GRAD, ENDS>(p, x, dt, B, C, dy, h, g, c0, t0 + q + kTile, 1, min(kTile, len - q - kTile), tid);
        if (GRAD)  // C h, with the state on entry
            for (int i = 0; i < cnt; ++i) s.red[i][w][lane] = row_dot(&s.c[i][32 * w], hr);
        for (int i = 0; i < cnt; ++i) {
            const float a = s.a[i], dx = s.d[i] * s.x[i][lane];
            float yv = 0.f;
            if constexpr (ENDS) {
                total = fmaf(s.d[i], A, total);
#pragma unroll
                for (int k = 0; k < 32; ++k) hr[k] = fmaf(s.b[i][32 * w + k], dx, a * hr[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    hr[k] = fmaf(s.b[i][32 * w + k], dx, a * hr[k]);
                    if (!GRAD) yv = fmaf(s.c[i][32 * w + k], hr[k], yv);
                }
                if (!GRAD) s.red[i][w][lane] = yv;
                if (GRAD) {
                    float v[32];
                    const float d = s.dy[i][lane];
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = hr[k] * d;
                    const float sum = lane_sums(v, lane);
                    dc_part[(((size_t)(t0 + q + i) * p.H + h) * gridDim.z + blockIdx.z) * K + 32 * w + lane] = sum;
                }
            }
        }
        __syncthreads();
        if (GRAD) {
            for (int i = w; i < cnt; i += K / 32) {
                const float d = s.dy[i][lane];
                const float rv = dot_row<K>(s.red[i], d, lane);
                float xd = s.x[i][lane] * d;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) xd += __shfl_xor_sync(0xffffffffu, xd, o);
                const size_t e = ((size_t)(t0 + q + i) * p.H + h) * gridDim.z + blockIdx.z;
                if (lane == 0) *dots(kR, e) = rv, *dots(kXd, e) = xd;
            }
            float *dst = keep + ((size_t)(tile0 + q / kKeep) * p.H + h) * K * p.P + c0 + lane;
#pragma unroll
            for (int k = 0; k < 32; ++k) dst[(size_t)(32 * w + k) * p.P] = hr[k];
        } else if (!ENDS) {
            for (int e = tid; e < cnt * kCols; e += K) {
                const int i = e / kCols, col = e % kCols;
                float v = 0.f;
#pragma unroll
                for (int k = 0; k < K / 32; ++k) v += s.red[i][k][col];
                y[((size_t)(t0 + q + i) * p.H + h) * p.P + c0 + col] = from_f32<Tin>(fmaf(D, s.x[i][col], v));
            }
        }
        __syncthreads();
    }
    float *out = ENDS ? p.seg.state + wk.seg_at : wk.last() && final_state ? final_state + wk.at : nullptr;
    if (out)
#pragma unroll
        for (int i = 0; i < 32; ++i) out[(size_t)i * p.P] = hr[i];
    if (ENDS && blockIdx.z == 0 && tid == 0) p.seg.decay[(size_t)blockIdx.x * p.H + h] = total;
}

// Start states of the segments (REV: gradients at their ends), in place of what a pass from zero
// left: start' = e^{decay} start + end. A thread per state element walks a sequence's segments.
template <bool REV>
__global__ void __launch_bounds__(256) scan_segments_kernel(ScanP p, int elements, const float *__restrict__ from) {
    const int n = blockIdx.x, h = blockIdx.y, e = blockIdx.z * 256 + threadIdx.x;
    const int len = p.m.end(n) - p.m.begin(n), segs = (len + p.seg.tokens - 1) / p.seg.tokens;
    if (segs < 2) return;
    const size_t slot0 = p.m.slot0(n, p.seg.tokens);
    auto slot = [&](int i) { return slot0 + (REV ? segs - 1 - i : i); };
    auto at = [&](int i) { return p.seg.state + (slot(i) * p.H + h) * elements + e; };
    float cur = from ? from[((size_t)n * p.H + h) * elements + e] : 0.f, next = *at(0);
    constexpr int kBatch = 8;  // ends loaded together, each before its place is taken
    for (int i = 0; i + 1 < segs; i += kBatch) {
        float end[kBatch + 1], decay[kBatch];
        end[0] = next;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            end[k + 1] = i + k + 2 < segs ? *at(i + k + 1) : 0.f;
            decay[k] = i + k + 1 < segs ? p.seg.decay[slot(i + k) * p.H + h] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (i + k + 1 >= segs) break;
            cur = fmaf(expf(decay[k]), cur, end[k]);
            *at(i + k + 1) = cur;
        }
        next = end[kBatch];
    }
}

// The decode step: a few tokens per sequence. The state's loads are issued before anything else and
// nothing is staged ahead, so that few registers and seven CTAs per SM keep the memory busy:
// 256 sequences x 64 heads of 128 x 64 (1.08 GB, nearly all of it state in and out) at 94 % of the copy
// rate; through the prompt kernel's 16-token tiles it was half of that.
template <typename Tin, typename Tdt, int K>
__global__ void __launch_bounds__(K)
scan_step_kernel(ScanP p, const Tin *__restrict__ x, const Tdt *__restrict__ dt, const Tin *__restrict__ B, const Tin *__restrict__ C,
                 const float *h0, Tin *__restrict__ y, float *final_state, unsigned *status) {
    __shared__ float bs[K], cs[K], red[K / 32][kCols];
    const int n = blockIdx.x, h = blockIdx.y, c0 = blockIdx.z * kCols, g = h / (p.H / p.G);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    if (p.m.cu && n == 0 && h == 0 && blockIdx.z == 0) check_cu(p.m, status, tid, K);
    const int t0 = p.m.begin(n), len = p.m.end(n) - t0;
    const size_t at = ((size_t)n * p.H + h) * K * p.P + c0 + lane;
    float hr[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) hr[i] = h0 ? h0[at + (size_t)(32 * w + i) * p.P] : 0.f;
    const float A = p.A[h], D = p.D ? p.D[h] : 0.f, bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    for (int i = 0; i < len; ++i) {
        const size_t t = (size_t)(t0 + i);
        bs[tid] = to_f32(B[t * p.bs + (size_t)g * K + tid]);
        cs[tid] = to_f32(C[t * p.cs + (size_t)g * K + tid]);
        const float xv = to_f32(x[t * p.xs + (size_t)h * p.P + c0 + lane]);
        const float d = delta_of(to_f32(dt[t * p.dts + h]) + bias, p.softplus), a = expf(d * A), dx = d * xv;
        __syncthreads();
        float yv = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            hr[k] = fmaf(bs[32 * w + k], dx, a * hr[k]);
            yv = fmaf(cs[32 * w + k], hr[k], yv);
        }
        red[w][lane] = yv;
        __syncthreads();
        if (w == 0) {
            yv = 0.f;
#pragma unroll
            for (int k = 0; k < K / 32; ++k) yv += red[k][lane];
            y[(t * p.H + h) * p.P + c0 + lane] = from_f32<Tin>(fmaf(D, xv, yv));
        }
    }
    if (final_state)
#pragma unroll
        for (int i = 0; i < 32; ++i) final_state[at + (size_t)(32 * w + i) * p.P] = hr[i];
}

// The gradient's reverse half: dx, dB parts (without delta), v and w, <h, i> of every tile (h on entry, i at its
// end) [slots, H, P/32], dh0.
// ENDS: only the gradient at the segment's start from zero, and its log decay.
template <typename Tin, typename Tdt, int K, bool ENDS>
__global__ void __launch_bounds__(K)
scan_reverse_kernel(ScanP p, const Tin *__restrict__ x, const Tdt *__restrict__ dt, const Tin *__restrict__ B, const Tin *__restrict__ C,
                    const Tin *__restrict__ dy, const float *__restrict__ h0, const float *__restrict__ dht, const float *__restrict__ keep,
                    Tin *__restrict__ dx, float *__restrict__ db_part, float *__restrict__ chunk_q, float *__restrict__ dh0, Dots dots) {
    __shared__ TileSmem<K> s;
    __shared__ float qs[K / 32];
    const int h = blockIdx.y, c0 = blockIdx.z * kCols, g = h / (p.H / p.G);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    Walk wk;
    if (!wk.find(p, blockIdx.x, h, K, 32 * w, c0 + lane) || (ENDS && (wk.first() || wk.len == 0))) return;
    const int n = wk.n, t0 = wk.t0, len = wk.len;
    const float *from = ENDS ? nullptr : wk.last() ? (dht ? dht + wk.at : nullptr) : p.seg.state + wk.seg_at;
    float gr[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) gr[i] = from ? from[(size_t)i * p.P] : 0.f;
    const int tile0 = p.m.slot0(n, kKeep) + (t0 - wk.s_begin) / kKeep;
    float total = 0.f;
    const float A = p.A[h], D = p.D ? p.D[h] : 0.f, bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    // tiles in reverse: token i of a tile is t0 + q - i; the ragged tile comes first, so that the
    // tiles are the forward half's
    const int first = len ? (len - 1) % kTile + 1 : 0;
    Tile<Tin, Tdt, K> r;
    if (len) r.template load<true, ENDS, true>(p, x, dt, B, C, dy, h, g, c0, t0 + len - 1, -1, first, tid);
    int cnt = first;
    for (int q = len - 1; q >= 0; q -= cnt, cnt = kTile) {
        put_tile<Tin, Tdt, K, true, ENDS, true>(s, r, p, A, bias, cnt, tid);
        if (!ENDS) {
            const size_t slot = (size_t)tile0 + q / kKeep;
            // the state that the tile before ended in
            const float *src = t0 - wk.s_begin + q >= kKeep ? keep + ((slot - 1) * p.H + h) * K * p.P + (size_t)32 * w * p.P + c0 + lane
                               : h0                         ? h0 + wk.at
                                                            : nullptr;
            float v = 0.f;
            if (src) {
#pragma unroll
                for (int k = 0; k < 32; ++k) v = fmaf(src[(size_t)k * p.P], gr[k], v);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) qs[w] = v;
            __syncthreads();
            if (tid == 0) {
                v = 0.f;
#pragma unroll
                for (int k = 0; k < K / 32; ++k) v += qs[k];
                chunk_q[(slot * p.H + h) * gridDim.z + blockIdx.z] = v;
            }
        }
        __syncthreads();
        if (q - cnt >= 0) r.template load<true, ENDS, true>(p, x, dt, B, C, dy, h, g, c0, t0 + q - cnt, -1, kTile, tid);
        if (!ENDS)  // B i, with what comes in at the end
            for (int i = 0; i < cnt; ++i) s.red2[i][w][lane] = row_dot(&s.b[i][32 * w], gr);
        for (int i = 0; i < cnt; ++i) {
            const float d = s.dy[i][lane], a = s.a[i];
            if constexpr (ENDS) {
                total = fmaf(s.d[i], A, total);
#pragma unroll
                for (int k = 0; k < 32; ++k) gr[k] = a * fmaf(s.c[i][32 * w + k], d, gr[k]);
            } else {
                const float xv = s.x[i][lane];
                float u = 0.f, v[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    gr[k] = fmaf(s.c[i][32 * w + k], d, gr[k]);
                    u = fmaf(s.b[i][32 * w + k], gr[k], u);
                    v[k] = gr[k] * xv;
                    gr[k] *= a;
                }
                s.red[i][w][lane] = u;
                const float sum = lane_sums(v, lane);
                db_part[(((size_t)(t0 + q - i) * p.H + h) * gridDim.z + blockIdx.z) * K + 32 * w + lane] = sum;
            }
        }
        __syncthreads();
        for (int e = tid; !ENDS && e < cnt * kCols; e += K) {
            const int i = e / kCols, col = e % kCols;
            float u = 0.f;
#pragma unroll
            for (int k = 0; k < K / 32; ++k) u += s.red[i][k][col];
            dx[((size_t)(t0 + q - i) * p.H + h) * p.P + c0 + col] = from_f32<Tin>(fmaf(s.d[i], u, D * s.dy[i][col]));
        }
        for (int i = w; !ENDS && i < cnt; i += K / 32) {
            const float xv = s.x[i][lane], wv = dot_row<K>(s.red[i], xv, lane), vv = dot_row<K>(s.red2[i], xv, lane);
            const size_t e = ((size_t)(t0 + q - i) * p.H + h) * gridDim.z + blockIdx.z;
            if (lane == 0) *dots(kWt, e) = wv, *dots(kV, e) = vv;
        }
        __syncthreads();
    }
    float *out = ENDS ? p.seg.state + wk.seg_at : wk.first() && dh0 ? dh0 + wk.at : nullptr;
    if (out)
#pragma unroll
        for (int i = 0; i < 32; ++i) out[(size_t)i * p.P] = gr[i];
    if (ENDS && blockIdx.z == 0 && tid == 0) p.seg.decay[(size_t)blockIdx.x * p.H + h] = total;
}

// Per token: dC, dB summed over a group's heads.
template <typename Tin, typename Tdt, int K>
__global__ void __launch_bounds__(K)
scan_gather_kernel(ScanP p, const Tdt *__restrict__ dt, const float *__restrict__ dc_part, const float *__restrict__ db_part,
                   Tin *__restrict__ dB, Tin *__restrict__ dC) {
    const int tid = threadIdx.x, S = p.P / kCols, r = p.H / p.G;
    const size_t t = blockIdx.x;
    for (int g = 0; g < p.G; ++g) {
        float sb = 0.f, sc = 0.f;
        for (int h = g * r; h < (g + 1) * r; ++h) {
            float pb = 0.f;
            for (int k = 0; k < S; ++k) {
                pb += db_part[((t * p.H + h) * S + k) * K + tid];
                sc += dc_part[((t * p.H + h) * S + k) * K + tid];
            }
            sb = fmaf(delta_of(to_f32(dt[t * p.dts + h]) + (p.dt_bias ? p.dt_bias[h] : 0.f), p.softplus), pb, sb);
        }
        dB[(t * p.G + g) * K + tid] = from_f32<Tin>(sb);
        dC[(t * p.G + g) * K + tid] = from_f32<Tin>(sc);
    }
}

// Four elements of a row, by one access.
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}

// Per tile of 16 tokens and head: the gradients of the log decay and dt, and this tile's parts [slots, 3, H]
// of dA, ddt_bias and dD. A thread per pair of tokens for the products, then a lane per token.
template <typename Tin, typename Tdt, int K>
__global__ void __launch_bounds__(128)
scan_gates_kernel(ScanP p, const Tin *__restrict__ x, const Tdt *__restrict__ dt, const Tin *__restrict__ B, const Tin *__restrict__ C,
                  const Tin *__restrict__ dy, Dots dots, const float *__restrict__ chunk_q, Tdt *__restrict__ ddt, float *__restrict__ part) {
    constexpr int T = kKeep, kPad = 4, kMaxP = 128;  // rows of 16 bytes more: a quarter warp's rows meet all banks
    static_assert(T == 16 && T * (T - 1) / 2 <= 128, "a thread per pair, half a warp per tile");
    __shared__ __align__(16) float bs[T][K + kPad], cs[T][K + kPad], xs[T][kMaxP + kPad], ys[T][kMaxP + kPad];
    __shared__ float ds[T], gs[T], pairs[T][T + 1];
    const int tid = threadIdx.x, slot = blockIdx.x, h = blockIdx.y, S = p.P / kCols;
    float *out = part + (size_t)slot * 3 * p.H + h;
    int n, local;
    if (!p.m.slot(slot, T, &n, &local)) {  // an unused slot adds nothing
        if (tid < 3) out[tid * p.H] = 0.f;
        return;
    }
    const int t0 = p.m.begin(n) + local * T, cnt = min(T, p.m.end(n) - t0), g = h / (p.H / p.G);
    // a thread per token and eighth of its row, four elements at a time (the inputs' rows are 16-byte aligned)
    const int i = tid >> 3, c4 = (tid & 7) * 4;
    const bool in = i < cnt;
    const size_t ti = (size_t)(t0 + i);
#pragma unroll
    for (int k = c4; k < K; k += 32) {
        *reinterpret_cast<float4 *>(&bs[i][k]) = in ? load4(B + ti * p.bs + (size_t)g * K + k) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(&cs[i][k]) = in ? load4(C + ti * p.cs + (size_t)g * K + k) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = c4; k < kMaxP; k += 32) {
        if (k >= p.P) break;
        *reinterpret_cast<float4 *>(&xs[i][k]) = in ? load4(x + ti * p.xs + (size_t)h * p.P + k) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(&ys[i][k]) = in ? load4(dy + (ti * p.H + h) * p.P + k) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float A = p.A[h];
    const int t = t0 + tid;
    const size_t at = (size_t)t * p.H + h;
    float raw = 0.f, d = 0.f, rv = 0.f, vv = 0.f, wv = 0.f, q = 0.f, dD = 0.f;
    if (tid < T) {
        for (int k = 0; k < S; ++k) q += chunk_q[((size_t)slot * p.H + h) * S + k];
        if (tid < cnt) {
            raw = to_f32(dt[(size_t)t * p.dts + h]) + (p.dt_bias ? p.dt_bias[h] : 0.f), d = delta_of(raw, p.softplus);
            for (int k = 0; k < S; ++k) {
                rv += *dots(kR, at * S + k), vv += *dots(kV, at * S + k), wv += *dots(kWt, at * S + k);
                dD += *dots(kXd, at * S + k);
            }
        }
        ds[tid] = d, gs[tid] = tid < cnt ? d * A : 0.f;
    }
    __syncthreads();
    int r = 1, s = tid;  // pair (r, s), s < r
    while (s >= r) s -= r++;
    if (r < cnt) {
        auto dot = [&](const float *a, const float *b, int len) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            for (int k = 0; k < len; k += 4) {
                const float4 a4 = *reinterpret_cast<const float4 *>(a + k), b4 = *reinterpret_cast<const float4 *>(b + k);
                v[0] = fmaf(a4.x, b4.x, v[0]), v[1] = fmaf(a4.y, b4.y, v[1]), v[2] = fmaf(a4.z, b4.z, v[2]), v[3] = fmaf(a4.w, b4.w, v[3]);
            }
            return (v[0] + v[1]) + (v[2] + v[3]);
        };
        float between = 0.f;
        for (int j = s + 1; j <= r; ++j) between += gs[j];
        pairs[r][s] = expf(between) * dot(cs[r], bs[s], K) * dot(ys[r], xs[s], p.P) * ds[s];
    }
    __syncthreads();
    if (tid >= T) return;
    constexpr unsigned kLanes = (1u << T) - 1;
    // row tid: the sum of the columns before each; then a column's rows from its own on
    float v[T], before = 0.f;
#pragma unroll
    for (int j = 0; j < T - 1; ++j) v[j] = j < tid && tid < cnt ? pairs[tid][j] : 0.f;
#pragma unroll
    for (int j = 0; j < T; ++j) {
        pairs[tid][j] = before;
        if (j < T - 1) before += v[j];
    }
    __syncwarp(kLanes);
    float carry = 0.f;
#pragma unroll
    for (int j = 0; j < T; ++j) v[j] = j >= tid && j < cnt ? pairs[j][tid] : 0.f;
#pragma unroll
    for (int j = 0; j < T; ++j) carry += v[j];
    // log decays through the token and after it, then the sums from the token on and before it
    float upto = gs[tid], from = gs[tid];
#pragma unroll
    for (int o = 1; o < T; o <<= 1) {
        const float a = __shfl_up_sync(kLanes, upto, o, T), b = __shfl_down_sync(kLanes, from, o, T);
        if (tid >= o) upto += a;
        if (tid + o < T) from += b;
    }
    const float whole = __shfl_sync(kLanes, from, 0, T), next = __shfl_down_sync(kLanes, from, 1, T);
    float on = expf(upto) * rv, past = tid < T - 1 ? expf(next) * d * vv : d * vv;
#pragma unroll
    for (int o = 1; o < T; o <<= 1) {
        const float a = __shfl_down_sync(kLanes, on, o, T), b = __shfl_up_sync(kLanes, past, o, T);
        if (tid + o < T) on += a;
        if (tid >= o) past += b;
    }
    past = __shfl_up_sync(kLanes, past, 1, T);
    carry += on + (tid ? past : 0.f) + expf(whole) * q;
    float dA = 0.f, dbias = 0.f;
    if (tid < cnt) {
        dA = d * carry;
        dbias = fmaf(A, carry, wv);
        if (p.softplus) dbias /= 1.f + expf(-raw);
        ddt[at] = from_f32<Tdt>(dbias);
    }
#pragma unroll
    for (int o = T / 2; o > 0; o >>= 1) {
        dA += __shfl_xor_sync(kLanes, dA, o, T);
        dbias += __shfl_xor_sync(kLanes, dbias, o, T);
        dD += __shfl_xor_sync(kLanes, dD, o, T);
    }
    if (tid == 0) out[0] = dA, out[p.H] = dbias, out[2 * p.H] = dD;
}

// dA, ddt_bias, dD [H] from the slots' parts, in a fixed order.
__global__ void __launch_bounds__(256) scan_sum_kernel(const float *__restrict__ part, int slots, int H, float *dA, float *ddt_bias, float *dD) {
    __shared__ float red[256];
    const int h = blockIdx.x, j = blockIdx.y;
    float v = 0.f;
    for (int k = threadIdx.x; k < slots; k += 256) v += part[((size_t)k * 3 + j) * H + h];
    red[threadIdx.x] = v;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
        if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
        __syncthreads();
    }
    float *out = j == 0 ? dA : j == 1 ? ddt_bias : dD;
    if (threadIdx.x == 0 && out) out[h] = red[0];
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Tokens of a segment; 0: whole sequences. Four CTAs of these kernels run on an SM; where there are
// fewer than two per SM a sequence is cut into about as many segments as would fill them, of at
// least two tiles (a packed batch, of unknown lengths, by its total). 1000 tokens of 4 heads, K = P =
// 64: forward and backward 30 + 90 us with two tiles, 34 + 108 with three, 40 + 125 with four (the
// backward as it was then; 100 with the gates' gradients by pairs).
int segment_tokens(const ScanArgs &a) {
    const long long ctas = (long long)(a.seq.cu ? 1 : a.seq.N) * a.H * (a.P / kCols);
    const int tokens = a.seq.cu ? a.seq.total : a.seq.T;
    if (ctas >= 2 * sm_count() || tokens < 8 * kTile) return 0;
    const long long want = (4ll * sm_count() + ctas - 1) / ctas, per = (tokens + want - 1) / want;
    return (int)((per < 2 * kTile ? 2 * kTile : per) + kTile - 1) / kTile * kTile;
}

size_t segments_bytes(const ScanArgs &a) {
    const int q = segment_tokens(a);
    if (!q) return 0;
    const size_t slots = a.seq.slots(q);
    return up256(slots * a.H * a.K * a.P * 4) + up256(slots * a.H * 4);
}

Segments segments(const ScanArgs &a, char *ws) {
    Segments s;
    s.tokens = segment_tokens(a);
    s.state = (float *)ws;
    s.decay = s.tokens ? (float *)(ws + up256((size_t)a.seq.slots(s.tokens) * a.H * a.K * a.P * 4)) : nullptr;
    if (!s.tokens) s.tokens = ((a.seq.cu ? a.seq.total : a.seq.T) / kTile + 1) * kTile;  // longer than any sequence
    return s;
}

struct SimtWs {
    size_t seg, keep, dc, db, q, rw, part, total;
};

SimtWs simt_ws(const ScanArgs &a) {
    const size_t tok = a.seq.total, S = a.P / kCols, slots = a.seq.slots(kKeep);
    SimtWs w;
    w.seg = 0;
    w.keep = w.seg + segments_bytes(a);
    w.dc = w.keep + up256(slots * a.H * a.K * a.P * 4);
    w.db = w.dc + up256(tok * a.H * S * a.K * 4);
    w.q = w.db + up256(tok * a.H * S * a.K * 4);
    w.rw = w.q + up256(slots * a.H * S * 4);
    w.part = w.rw + up256(kDots * tok * a.H * S * 4);
    w.total = w.part + up256(slots * 3 * a.H * 4);
    return w;
}

ScanP params(const ScanArgs &a, const Segments &seg) {
    return ScanP{a.seq, seg, a.G, a.H, a.P, a.softplus, a.xs, a.bs, a.cs, a.dts, a.A, a.D, a.dt_bias};
}

// CTAs along the sequences: one per segment slot (T = 0: one per sequence, for its state).
int walks(const ScanArgs &a, const Segments &seg) { return a.seq.total ? a.seq.slots(seg.tokens) : a.seq.N; }

// Start states of the segments (REV: gradients at their ends); nothing for whole sequences.
template <typename Tin, typename Tdt, int K, bool REV>
void compose(const ScanArgs &a, const ScanP &p) {
    if (!segment_tokens(a)) return;
    const Tin *x = (const Tin *)a.x, *B = (const Tin *)a.B, *C = (const Tin *)a.C, *dy = (const Tin *)a.dy;
    const dim3 grid(walks(a, p.seg), a.H, a.P / kCols);
    if (REV)
        scan_reverse_kernel<Tin, Tdt, K, true><<<grid, K, 0, a.stream>>>(p, x, (const Tdt *)a.dt, B, C, dy, nullptr, nullptr, nullptr, nullptr,
                                                                        nullptr, nullptr, nullptr, Dots{});
    else
        scan_forward_kernel<Tin, Tdt, K, false, true><<<grid, K, 0, a.stream>>>(p, x, (const Tdt *)a.dt, B, C, nullptr, nullptr, nullptr,
                                                                               nullptr, nullptr, nullptr, Dots{}, a.status);
    scan_segments_kernel<REV><<<dim3(a.seq.N, a.H, K * a.P / 256), 256, 0, a.stream>>>(p, K * a.P, REV ? a.dht : a.h0);
}

template <typename Tin, typename Tdt, int K>
cudaError_t forward(const ScanArgs &a) {
    const ScanP p = params(a, segments(a, (char *)a.ws));
    compose<Tin, Tdt, K, false>(a, p);
    const dim3 grid(walks(a, p.seg), a.H, a.P / kCols);
    scan_forward_kernel<Tin, Tdt, K, false, false><<<grid, K, 0, a.stream>>>(p, (const Tin *)a.x, (const Tdt *)a.dt, (const Tin *)a.B,
                                                                            (const Tin *)a.C, nullptr, a.h0, (Tin *)a.y, a.final_state,
                                                                            nullptr, nullptr, Dots{}, a.status);
    return cudaGetLastError();
}

template <typename Tin, typename Tdt, int K>
cudaError_t step(const ScanArgs &a) {
    const dim3 grid(a.seq.N, a.H, a.P / kCols);
    scan_step_kernel<Tin, Tdt, K><<<grid, K, 0, a.stream>>>(params(a, Segments{}), (const Tin *)a.x, (const Tdt *)a.dt, (const Tin *)a.B,
                                                           (const Tin *)a.C, a.h0, (Tin *)a.y, a.final_state, a.status);
    return cudaGetLastError();
}

template <typename Tin, typename Tdt, int K>
cudaError_t backward(const ScanArgs &a) {
    const SimtWs w = simt_ws(a);
    char *ws = (char *)a.ws;
    const ScanP p = params(a, segments(a, ws + w.seg));
    float *keep = (float *)(ws + w.keep), *dc = (float *)(ws + w.dc), *db = (float *)(ws + w.db), *q = (float *)(ws + w.q);
    float *part = (float *)(ws + w.part);
    const Dots dots{(float *)(ws + w.rw), (size_t)a.seq.total * a.H * (a.P / kCols)};
    const Tin *x = (const Tin *)a.x, *B = (const Tin *)a.B, *C = (const Tin *)a.C, *dy = (const Tin *)a.dy;
    const Tdt *dt = (const Tdt *)a.dt;
    const dim3 grid(walks(a, p.seg), a.H, a.P / kCols);
    const int slots = a.seq.slots(kKeep);
    compose<Tin, Tdt, K, false>(a, p);
    scan_forward_kernel<Tin, Tdt, K, true, false><<<grid, K, 0, a.stream>>>(p, x, dt, B, C, dy, a.h0, nullptr, nullptr, dc, keep, dots, a.status);
    compose<Tin, Tdt, K, true>(a, p);
    scan_reverse_kernel<Tin, Tdt, K, false><<<grid, K, 0, a.stream>>>(p, x, dt, B, C, dy, a.h0, a.dht, keep, (Tin *)a.dx, db, q, a.dh0,
                                                                      dots);
    if (a.seq.total)
        scan_gather_kernel<Tin, Tdt, K><<<a.seq.total, K, 0, a.stream>>>(p, dt, dc, db, (Tin *)a.dB, (Tin *)a.dC);
    if (slots)
        scan_gates_kernel<Tin, Tdt, K><<<dim3(slots, a.H), 128, 0, a.stream>>>(p, x, dt, B, C, dy, dots, q, (Tdt *)a.ddt, part);
    return launch_scan_sum(part, slots, a);
}

enum Pass { kForward, kStep, kBackward };

template <typename Tin, typename Tdt, int K>
cudaError_t run_pass(const ScanArgs &a, Pass pass) {
    return pass == kForward ? forward<Tin, Tdt, K>(a) : pass == kStep ? step<Tin, Tdt, K>(a) : backward<Tin, Tdt, K>(a);
}

template <typename Tin, typename Tdt>
cudaError_t by_k(const ScanArgs &a, Pass pass) {
    return a.K == 128 ? run_pass<Tin, Tdt, 128>(a, pass) : run_pass<Tin, Tdt, 64>(a, pass);
}

cudaError_t dispatch(const ScanArgs &a, Pass pass) {
    if (a.seq.N == 0) return cudaSuccess;
    if (a.dtype == GDN_DTYPE_F32) return by_k<float, float>(a, pass);
    return a.dt_dtype == GDN_DTYPE_F32 ? by_k<__nv_bfloat16, float>(a, pass) : by_k<__nv_bfloat16, __nv_bfloat16>(a, pass);
}

}  // namespace

cudaError_t launch_scan_sum(const float *part, int slots, const ScanArgs &a) {
    scan_sum_kernel<<<dim3(a.H, 3), 256, 0, a.stream>>>(part, slots, a.H, a.dA, a.ddt_bias, a.dD);
    return cudaGetLastError();
}

cudaError_t launch_scan_step(const ScanArgs &a) { return dispatch(a, kStep); }
cudaError_t launch_scan_simt_fwd(const ScanArgs &a) { return dispatch(a, kForward); }
size_t scan_simt_fwd_bytes(const ScanArgs &a) { return segments_bytes(a); }
size_t scan_simt_bwd_bytes(const ScanArgs &a) { return simt_ws(a).total; }
cudaError_t launch_scan_simt_bwd(const ScanArgs &a) { return dispatch(a, kBackward); }

}  // namespace gdn
