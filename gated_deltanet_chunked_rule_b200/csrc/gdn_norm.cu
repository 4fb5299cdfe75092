// gdn_norm.cu -- layer norm over the last axis, centred or not (RMS), with an
// optional silu gate before or after it: the step behind a recurrence's output.
//
//   u = x silu(z) (gate first) or x,   n = (u - mean) rstd,   lin = n weight + bias
//   y = lin silu(z) (gate last) or lin
//   dlin = dy silu(z) or dy,  dn = dlin weight,  du = rstd (dn - n mean(dn n) - [mean(dn)])
//   dweight = sum_rows dlin n,  dbias = sum_rows dlin
//
// A group of 8, 16, 32 or 256 threads owns a row and keeps it in registers between its passes
// (mean, then the centred sum of squares, then the result), so every tensor moves once, and the
// next row's loads are in flight meanwhile. Groups walk the rows with a stride, as many blocks as
// fit at once (one wave), the weights and the weight gradient's sums staying in registers; the
// sums (fp32) are joined over a block's groups in shared memory and over the blocks by a second
// kernel, in a fixed order. Arithmetic on two elements per instruction. Rows that are too long for
// the registers, or whose width does not allow 16-byte accesses, take kernels that read a row
// once per pass.
//
// Bound by the bytes and, with few warps on an SM, by their latency: 262144 gated rows of 128
// forward 36 us (201 MB, 84 % of the copy rate), backward 69 us (335 MB, 76 %; 79 us with two
// blocks on an SM instead of three; two rows ahead instead of one gain nothing). 4096 centred rows
// of 4096, L2-resident: forward 13 us, backward 31 us with the second kernel, bound by the
// barriers of a row's sums. The blocks per SM were set on rows without a gate or with it behind. With the
// gate first the backward keeps two more values per element and spills up to 340 bytes a thread in
// bf16: 262144 rows of 128 72 us as with the gate behind, 65536 rows of 512 87 us against 74, 8192
// rows of 4096 81 us against 72. The kernels that read a row once per pass take a block per row
// whatever its width: 262144 rows of 129 forward 680 us, backward 820; 4096 of 4095, 53 and 94.
#include <algorithm>

#include "gdn_layer.cuh"
#include "gdn_host.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <typename T, int VEC>
struct alignas(16) Raw {
    uint4 v;
    __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ F2 pair(int m) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (sizeof(T) == 4) return f2(w[2 * m], w[2 * m + 1]);
        return f2(w[m] << 16, w[m] & 0xffff0000u);
    }
};

// Sum over the TPR threads of a row group; every thread gets it. buf: 2 x 8 floats per
// value, alternated by the caller's phase so that one barrier per sum is enough.
template <int TPR, int NS>
__device__ __forceinline__ void row_sum(float (&v)[NS], float (*buf)[NS][kThreads / 32], int &phase) {
    constexpr int kW = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = kW / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < NS; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < NS; ++i) buf[phase][i][warp] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kThreads / 32; ++k) s += buf[phase][i][k];
            v[i] = s;
        }
        phase ^= 1;
    }
}

struct NormP {
    long long R;
    int D;
    float eps, inv_d;
};

__device__ __forceinline__ float load_w(const void *w, int wf32, int i) {
    return wf32 ? ((const float *)w)[i] : __bfloat162float(((const __nv_bfloat16 *)w)[i]);
}

// VEC weights from element i on, which lie in one row of them (zeros behind it).
template <int VEC>
__device__ __forceinline__ void load_weights(const void *w, int wf32, int i, bool in, F2 (&v)[VEC / 2]) {
#pragma unroll
    for (int m = 0; m < VEC / 2; ++m) v[m] = f2(0.f, 0.f);
    if (!in || !w) return;
    if (wf32) {
#pragma unroll
        for (int m = 0; m < VEC / 4; ++m) {
            const float4 a = reinterpret_cast<const float4 *>((const float *)w + i)[m];
            v[2 * m] = f2(a.x, a.y), v[2 * m + 1] = f2(a.z, a.w);
        }
    } else {
#pragma unroll
        for (int m = 0; m < VEC / 2; ++m) {
            const uint32_t a = reinterpret_cast<const uint32_t *>((const __nv_bfloat16 *)w + i)[m];
            v[m] = f2(a << 16, a & 0xffff0000u);
        }
    }
}

// GATE: 0 none, 1 before the normalisation, 2 after it
template <typename T, int TPR, int NV, int GATE, bool CENTER>
__global__ void __launch_bounds__(kThreads)
norm_fwd_kernel(NormP p, const T *__restrict__ x, const void *__restrict__ weight, const void *__restrict__ bias, int wf32,
                const T *__restrict__ gate, T *__restrict__ y, float *__restrict__ stats) {
    constexpr int VEC = 16 / sizeof(T), kGroups = kThreads / TPR;
    constexpr bool kFast = sizeof(T) == 2;
    __shared__ float buf[2][1][kThreads / 32];
    const int g = threadIdx.x / TPR, l = threadIdx.x % TPR, nv = p.D / VEC;
    constexpr int PAIRS = VEC / 2;
    F2 w[NV][PAIRS], b[NV][PAIRS];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = i * TPR + l;
        load_weights<VEC>(weight, wf32, v * VEC, v < nv, w[i]);
        load_weights<VEC>(bias, wf32, v * VEC, v < nv, b[i]);
    }
    int phase = 0;
    Raw<T, VEC> q[NV], z[NV];
    auto fetch = [&](long long r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * TPR + l;
            q[i].v = z[i].v = make_uint4(0, 0, 0, 0);
            if (r >= p.R || v >= nv) continue;
            q[i].load(x + r * p.D + v * VEC);
            if (GATE) z[i].load(gate + r * p.D + v * VEC);
        }
    };
    const long long stride = (long long)gridDim.x * kGroups;
    fetch((long long)blockIdx.x * kGroups + g);
    // whole blocks walk together, so that the barriers and shuffles stay uniform
    for (long long r0 = (long long)blockIdx.x * kGroups; r0 < p.R; r0 += stride) {
        const long long r = r0 + g;
        const bool live = r < p.R;
        F2 u[NV][PAIRS], sum = f2(0.f, 0.f), sq = f2(0.f, 0.f);
        Raw<T, VEC> zc[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            zc[i] = z[i];
#pragma unroll
            for (int m = 0; m < PAIRS; ++m) {
                u[i][m] = q[i].pair(m);
                if (GATE == 1) {
                    const F2 zz = z[i].pair(m);
                    u[i][m] = mul2(u[i][m], mul2(zz, sigmoid<kFast>(zz)));
                }
                if (CENTER) sum = add2(sum, u[i][m]);
            }
        }
        fetch(r + stride);
        float s[1], mean = 0.f;
        if (CENTER) {
            s[0] = get(sum).x + get(sum).y;
            row_sum<TPR, 1>(s, buf, phase);
            mean = s[0] * p.inv_d;
        }
        const F2 minus = f2(-mean, -mean);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (i * TPR + l >= nv) continue;
#pragma unroll
            for (int m = 0; m < PAIRS; ++m) {
                if (CENTER) u[i][m] = add2(u[i][m], minus);
                sq = fma2(u[i][m], u[i][m], sq);
            }
        }
        s[0] = get(sq).x + get(sq).y;
        row_sum<TPR, 1>(s, buf, phase);
        const float rstd = rsqrtf(fmaf(s[0], p.inv_d, p.eps));
        if (!live) continue;
        if (l == 0 && stats) {
            stats[2 * r] = mean;
            stats[2 * r + 1] = rstd;
        }
        const F2 rs = f2(rstd, rstd);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * TPR + l;
            if (v >= nv) continue;
            F2 o[PAIRS];
#pragma unroll
            for (int m = 0; m < PAIRS; ++m) {
                o[m] = fma2(mul2(u[i][m], rs), w[i][m], b[i][m]);
                if (GATE == 2) {
                    const F2 zz = zc[i].pair(m);
                    o[m] = mul2(o[m], mul2(zz, sigmoid<kFast>(zz)));
                }
            }
            store_pairs<T, PAIRS>(y + r * p.D + v * VEC, o);
        }
    }
}

template <typename T, int TPR, int NV, int GATE, bool CENTER>
__global__ void __launch_bounds__(kThreads, NV == 1 ? 3 : NV == 2 ? 2 : 1)
norm_bwd_kernel(NormP p, const T *__restrict__ x, const void *__restrict__ weight, const void *__restrict__ bias, int wf32,
                const T *__restrict__ gate, const T *__restrict__ dy, const float *__restrict__ stats, T *__restrict__ dx,
                T *__restrict__ dgate, float *__restrict__ part) {
    let_next_start();
    constexpr int VEC = 16 / sizeof(T), kGroups = kThreads / TPR;
    constexpr bool kFast = sizeof(T) == 2;
    __shared__ float buf[2][CENTER ? 2 : 1][kThreads / 32];
    __shared__ float sum[kGroups > 1 ? 2 * TPR * NV * VEC : 1];
    const int g = threadIdx.x / TPR, l = threadIdx.x % TPR, nv = p.D / VEC;
    constexpr int PAIRS = VEC / 2;
    const F2 zero = f2(0.f, 0.f), one = f2(1.f, 1.f), minus = f2(-1.f, -1.f);
    F2 w[NV][PAIRS], b[GATE == 2 ? NV : 1][PAIRS], dw[NV][PAIRS], db[NV][PAIRS];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = i * TPR + l;
        load_weights<VEC>(weight, wf32, v * VEC, v < nv, w[i]);
        if (GATE == 2) load_weights<VEC>(bias, wf32, v * VEC, v < nv, b[GATE == 2 ? i : 0]);
#pragma unroll
        for (int m = 0; m < PAIRS; ++m) dw[i][m] = db[i][m] = zero;
    }
    int phase = 0;
    Raw<T, VEC> q[NV], z[NV], d[NV];
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](long long r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * TPR + l;
            q[i].v = z[i].v = d[i].v = make_uint4(0, 0, 0, 0);
            if (r >= p.R || v >= nv) continue;
            q[i].load(x + r * p.D + v * VEC);
            d[i].load(dy + r * p.D + v * VEC);
            if (GATE) z[i].load(gate + r * p.D + v * VEC);
        }
        mean = r < p.R ? stats[2 * r] : 0.f;
        rstd = r < p.R ? stats[2 * r + 1] : 0.f;
    };
    const long long stride = (long long)gridDim.x * kGroups;
    // short rows keep what the second pass needs, and the next row is fetched meanwhile; long ones
    // keep the row as it was loaded and compute it again
    constexpr bool kKeep = NV <= 2;
    if (kKeep) fetch((long long)blockIdx.x * kGroups + g);
    for (long long r0 = (long long)blockIdx.x * kGroups; r0 < p.R; r0 += stride) {
        const long long r = r0 + g;
        const bool live = r < p.R;
        if (!kKeep) fetch(r);
        const F2 mu = f2(-mean, -mean), rs = f2(rstd, rstd);
        F2 s0 = zero, s1 = zero;
        // n; dn; gate first: silu(z), x silu'(z)
        F2 kn[kKeep ? NV : 1][PAIRS], kd[kKeep ? NV : 1][PAIRS], ka[kKeep && GATE == 1 ? NV : 1][PAIRS], kb[kKeep && GATE == 1 ? NV : 1][PAIRS];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * TPR + l;
            if (v >= nv) continue;
            F2 og[PAIRS];
#pragma unroll
            for (int m = 0; m < PAIRS; ++m) {
                const F2 xe = q[i].pair(m), de = d[i].pair(m);
                F2 u = xe, dl = de, dsilu = zero;
                if (GATE) {
                    const F2 zz = z[i].pair(m), sg = sigmoid<kFast>(zz), si = mul2(zz, sg);
                    dsilu = fma2(si, fma2(sg, minus, one), sg);
                    if (GATE == 1) u = mul2(u, si);
                    else dl = mul2(dl, si);
                    if (kKeep && GATE == 1) ka[i][m] = si, kb[i][m] = mul2(xe, dsilu);
                }
                const F2 n = mul2(CENTER ? add2(u, mu) : u, rs), dn = mul2(dl, w[i][m]);
                dw[i][m] = fma2(dl, n, dw[i][m]);
                db[i][m] = add2(db[i][m], dl);
                s0 = fma2(dn, n, s0);
                if (CENTER) s1 = add2(s1, dn);
                if (kKeep) kn[i][m] = n, kd[i][m] = dn;
                if (GATE == 2) og[m] = mul2(mul2(dsilu, de), fma2(n, w[i][m], b[GATE == 2 ? i : 0][m]));
            }
            if (GATE == 2 && live) store_pairs<T, PAIRS>(dgate + r * p.D + v * VEC, og);
        }
        if (kKeep) fetch(r + stride);
        float s[CENTER ? 2 : 1];
        s[0] = get(s0).x + get(s0).y;
        if (CENTER) s[CENTER ? 1 : 0] = get(s1).x + get(s1).y;
        row_sum<TPR, CENTER ? 2 : 1>(s, buf, phase);
        if (!live) continue;
        const float a0 = -s[0] * p.inv_d, a1 = CENTER ? -s[CENTER ? 1 : 0] * p.inv_d : 0.f;
        const F2 m0 = f2(a0, a0), m1 = f2(a1, a1);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * TPR + l;
            if (v >= nv) continue;
            F2 o[PAIRS], og[PAIRS];
#pragma unroll
            for (int m = 0; m < PAIRS; ++m) {
                F2 n, dn, a = one, bb = zero;
                if (kKeep) {
                    n = kn[i][m], dn = kd[i][m];
                    if (GATE == 1) a = ka[i][m], bb = kb[i][m];
                } else {
                    F2 u = q[i].pair(m), dl = d[i].pair(m);
                    if (GATE) {
                        const F2 zz = z[i].pair(m), sg = sigmoid<kFast>(zz), si = mul2(zz, sg);
                        if (GATE == 1) bb = mul2(u, fma2(si, fma2(sg, minus, one), sg)), a = si, u = mul2(u, si);
                        else dl = mul2(dl, si);
                    }
                    n = mul2(CENTER ? add2(u, mu) : u, rs), dn = mul2(dl, w[i][m]);
                }
                F2 du = fma2(n, m0, dn);
                if (CENTER) du = add2(du, m1);
                du = mul2(du, rs);
                o[m] = GATE == 1 ? mul2(du, a) : du;
                if (GATE == 1) og[m] = mul2(du, bb);
            }
            store_pairs<T, PAIRS>(dx + r * p.D + v * VEC, o);
            if (GATE == 1) store_pairs<T, PAIRS>(dgate + r * p.D + v * VEC, og);
        }
    }
    // the block's sums of dweight, dbias
    float *out = part + (size_t)blockIdx.x * 2 * p.D;
    if constexpr (kGroups == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * TPR + l;
            if (v >= nv) continue;
#pragma unroll
            for (int m = 0; m < PAIRS; m += 2) {
                const float2 a = get(dw[i][m]), b = get(dw[i][m + 1]), c = get(db[i][m]), d = get(db[i][m + 1]);
                *reinterpret_cast<float4 *>(out + v * VEC + 2 * m) = make_float4(a.x, a.y, b.x, b.y);
                *reinterpret_cast<float4 *>(out + p.D + v * VEC + 2 * m) = make_float4(c.x, c.y, d.x, d.y);
            }
        }
    } else {
        for (int k = 0; k < kGroups; ++k) {
            __syncthreads();
            if (g != k) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int at = (i * VEC + e) * TPR + l;
                    const float2 a = get(dw[i][e / 2]), b = get(db[i][e / 2]);
                    sum[at] = (k ? sum[at] : 0.f) + (e & 1 ? a.y : a.x);
                    sum[TPR * NV * VEC + at] = (k ? sum[TPR * NV * VEC + at] : 0.f) + (e & 1 ? b.y : b.x);
                }
        }
        __syncthreads();
        for (int j = threadIdx.x; j < p.D; j += kThreads) {
            const int v = j / VEC, at = ((v / TPR) * VEC + j % VEC) * TPR + v % TPR;
            out[j] = sum[at];
            out[p.D + j] = sum[TPR * NV * VEC + at];
        }
    }
}

// dweight, dbias [D] from the blocks' parts, in a fixed order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *__restrict__ part, int blocks, int D, int wf32, void *dweight, void *dbias) {
    wait_for_previous();
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < D)
        for (int k = row; k < blocks; k += 32) v += part[((size_t)k * 2 + blockIdx.y) * D + c];
    red[row][lane] = v;
    __syncthreads();
    if (row || c >= D) return;
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += red[k][lane];
    void *o = blockIdx.y ? dbias : dweight;
    if (!o) return;
    if (wf32) ((float *)o)[c] = v;
    else ((__nv_bfloat16 *)o)[c] = __float2bfloat16_rn(v);
}

// --------------------------------------------- any width, any alignment
template <typename T>
struct RowAny {
    const T *x, *z;
    int gate;
    __device__ __forceinline__ float u(long long at) const {
        const float v = to_f32(x[at]);
        if (gate != 1) return v;
        const float zz = to_f32(z[at]);
        return v * zz * sigmoid<sizeof(T) == 2>(zz);
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_fwd_any_kernel(NormP p, const T *__restrict__ x, const void *__restrict__ weight, const void *__restrict__ bias, int wf32,
                    const T *__restrict__ gate, int GATE, int center, T *__restrict__ y, float *__restrict__ stats) {
    __shared__ float buf[2][1][kThreads / 32];
    int phase = 0;
    const RowAny<T> row{x, gate, GATE};
    for (long long r = blockIdx.x; r < p.R; r += gridDim.x) {
        float s[1] = {0.f}, mean = 0.f;
        if (center) {
            for (int j = threadIdx.x; j < p.D; j += kThreads) s[0] += row.u(r * p.D + j);
            row_sum<kThreads, 1>(s, buf, phase);
            mean = s[0] * p.inv_d;
        }
        s[0] = 0.f;
        for (int j = threadIdx.x; j < p.D; j += kThreads) {
            const float u = row.u(r * p.D + j) - mean;
            s[0] = fmaf(u, u, s[0]);
        }
        row_sum<kThreads, 1>(s, buf, phase);
        const float rstd = rsqrtf(fmaf(s[0], p.inv_d, p.eps));
        if (threadIdx.x == 0 && stats) {
            stats[2 * r] = mean;
            stats[2 * r + 1] = rstd;
        }
        for (int j = threadIdx.x; j < p.D; j += kThreads) {
            float o = fmaf((row.u(r * p.D + j) - mean) * rstd, load_w(weight, wf32, j), bias ? load_w(bias, wf32, j) : 0.f);
            if (GATE == 2) {
                const float zz = to_f32(gate[r * p.D + j]);
                o *= zz * sigmoid<sizeof(T) == 2>(zz);
            }
            y[r * p.D + j] = from_f32<T>(o);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_bwd_any_kernel(NormP p, const T *__restrict__ x, const void *__restrict__ weight, const void *__restrict__ bias, int wf32,
                    const T *__restrict__ gate, int GATE, int center, const T *__restrict__ dy, const float *__restrict__ stats,
                    T *__restrict__ dx, T *__restrict__ dgate) {
    __shared__ float buf[2][2][kThreads / 32];
    int phase = 0;
    const RowAny<T> row{x, gate, GATE};
    for (long long r = blockIdx.x; r < p.R; r += gridDim.x) {
        const float mean = stats[2 * r], rstd = stats[2 * r + 1];
        float s[2] = {0.f, 0.f};
        for (int j = threadIdx.x; j < p.D; j += kThreads) {
            const long long at = r * p.D + j;
            float dl = to_f32(dy[at]);
            if (GATE == 2) {
                const float zz = to_f32(gate[at]);
                dl *= zz * sigmoid<sizeof(T) == 2>(zz);
            }
            const float n = (row.u(at) - mean) * rstd, dn = dl * load_w(weight, wf32, j);
            s[0] = fmaf(dn, n, s[0]);
            s[1] += dn;
        }
        row_sum<kThreads, 2>(s, buf, phase);
        const float m0 = s[0] * p.inv_d, m1 = center ? s[1] * p.inv_d : 0.f;
        for (int j = threadIdx.x; j < p.D; j += kThreads) {
            const long long at = r * p.D + j;
            const float w = load_w(weight, wf32, j), de = to_f32(dy[at]);
            float dl = de, zz = 0.f, sg = 0.f;
            if (GATE) {
                zz = to_f32(gate[at]);
                sg = sigmoid<sizeof(T) == 2>(zz);
                if (GATE == 2) dl *= zz * sg;
            }
            const float n = (row.u(at) - mean) * rstd, du = rstd * (dl * w - n * m0 - m1);
            const float xe = to_f32(x[at]);  // read before dx is written
            dx[at] = from_f32<T>(GATE == 1 ? du * zz * sg : du);
            if (GATE) {
                const float dsilu = sg * (1.f + zz * (1.f - sg));
                dgate[at] = from_f32<T>(dsilu * (GATE == 1 ? du * xe : de * fmaf(n, w, bias ? load_w(bias, wf32, j) : 0.f)));
            }
        }
    }
}

// dweight, dbias parts: 32 columns by 8 rows of threads, each block a stride of the rows.
template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_dw_any_kernel(NormP p, const T *__restrict__ x, const T *__restrict__ gate, int GATE, const T *__restrict__ dy,
                   const float *__restrict__ stats, float *__restrict__ part) {
    let_next_start();
    __shared__ float red[2][8][33];
    const int lane = threadIdx.x & 31, wr = threadIdx.x >> 5;
    const int c = blockIdx.y * 32 + lane;
    const RowAny<T> row{x, gate, GATE};
    float dw = 0.f, db = 0.f;
    if (c < p.D)
        for (long long r = (long long)blockIdx.x * 8 + wr; r < p.R; r += (long long)gridDim.x * 8) {
            const long long at = r * p.D + c;
            float dl = to_f32(dy[at]);
            if (GATE == 2) {
                const float zz = to_f32(gate[at]);
                dl *= zz * sigmoid<sizeof(T) == 2>(zz);
            }
            dw = fmaf(dl, (row.u(at) - stats[2 * r]) * stats[2 * r + 1], dw);
            db += dl;
        }
    red[0][wr][lane] = dw;
    red[1][wr][lane] = db;
    __syncthreads();
    if (wr || c >= p.D) return;
    dw = db = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) dw += red[0][k][lane], db += red[1][k][lane];
    part[(size_t)blockIdx.x * 2 * p.D + c] = dw;
    part[(size_t)blockIdx.x * 2 * p.D + p.D + c] = db;
}

// ------------------------------------------------------------------ dispatch
NormP params(const NormArgs &a) { return NormP{a.R, a.D, a.eps, 1.f / a.D}; }
int gate_of(const NormArgs &a) { return !a.gate ? 0 : a.gate_first ? 1 : 2; }

// 16-byte accesses, and at most 8 of them per thread of a whole block.
bool in_registers(const NormArgs &a) {
    const int el = a.dtype == GDN_DTYPE_BF16 ? 8 : 4;
    return a.D % el == 0 && a.D / el <= kThreads * (el == 8 ? 4 : 8);
}

// Blocks that walk the rows: as many as run at once, at most one per row group (and at most eight
// per SM, four of a block per row: a backward's partial sums are one row per block).
int most_per_sm(int tpr) { return tpr > 32 ? 4 : 8; }

int walk_blocks(long long groups, int per_sm) {
    const long long most = (long long)sm_count() * per_sm;
    return (int)(groups < most ? groups : most);
}

template <typename Kernel>
int resident(Kernel kernel, int most) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, 0) != cudaSuccess || n < 1) n = 1;
    return n < most ? n : most;
}

cudaError_t sum_parts(const NormArgs &a, int blocks) {
    return launch(blocks > 0, norm_dw_kernel, dim3((a.D + 31) / 32, a.dbias ? 2 : 1), dim3(1024), 0, a.stream, a.part, blocks, a.D,
                  (int)(a.wdtype == GDN_DTYPE_F32), a.dweight, a.dbias);
}

template <typename T, int TPR, int NV, int GATE, bool CENTER>
cudaError_t run(const NormArgs &a, bool bwd) {
    const NormP p = params(a);
    const long long groups = (a.R + kThreads / TPR - 1) / (kThreads / TPR);
    const int wf32 = a.wdtype == GDN_DTYPE_F32;
    if (!bwd) {
        auto kernel = norm_fwd_kernel<T, TPR, NV, GATE, CENTER>;
        static const int per_sm = resident(kernel, most_per_sm(TPR));  // the kernel's own, the same on every such device
        kernel<<<walk_blocks(groups, per_sm), kThreads, 0, a.stream>>>(
            p, (const T *)a.x, a.weight, a.bias, wf32, (const T *)a.gate, (T *)a.y, a.stats);
    } else {
        auto kernel = norm_bwd_kernel<T, TPR, NV, GATE, CENTER>;
        static const int per_sm = resident(kernel, most_per_sm(TPR));
        const int blocks = walk_blocks(groups, per_sm);
        kernel<<<blocks, kThreads, 0, a.stream>>>(
            p, (const T *)a.x, a.weight, a.bias, wf32, (const T *)a.gate, (const T *)a.dy, a.stats, (T *)a.dx, (T *)a.dgate, a.part);
        return sum_parts(a, blocks);
    }
    return cudaGetLastError();
}

template <typename T, int TPR, int NV>
cudaError_t by_form(const NormArgs &a, bool bwd) {
    switch (gate_of(a) * 2 + (a.center ? 1 : 0)) {
        case 0: return run<T, TPR, NV, 0, false>(a, bwd);
        case 1: return run<T, TPR, NV, 0, true>(a, bwd);
        case 2: return run<T, TPR, NV, 1, false>(a, bwd);
        case 3: return run<T, TPR, NV, 1, true>(a, bwd);
        case 4: return run<T, TPR, NV, 2, false>(a, bwd);
        default: return run<T, TPR, NV, 2, true>(a, bwd);
    }
}

// The fewest threads that hold a row with at most four accesses each (within a warp), or a
// block with as many as it takes: a warp's sums need no barrier.
template <typename T>
cudaError_t by_width(const NormArgs &a, bool bwd) {
    const int nv = a.D / (16 / (int)sizeof(T));
    if (nv <= 8) return by_form<T, 8, 1>(a, bwd);
    if (nv <= 16) return by_form<T, 16, 1>(a, bwd);
    if (nv <= 32) return by_form<T, 32, 1>(a, bwd);
    if (nv <= 64) return by_form<T, 32, 2>(a, bwd);
    if (nv <= 128) return by_form<T, 32, 4>(a, bwd);
    if (nv <= 256) return by_form<T, 256, 1>(a, bwd);
    if (nv <= 512) return by_form<T, 256, 2>(a, bwd);
    if (nv <= 1024) return by_form<T, 256, 4>(a, bwd);
    if constexpr (sizeof(T) == 4) return by_form<T, 256, 8>(a, bwd);
    return cudaErrorInvalidValue;
}

int any_dw_blocks(const NormArgs &a) {
    const long long groups = (a.R + 63) / 64;  // at least 64 rows per block
    return (int)std::min<long long>(groups, sm_count());
}

template <typename T>
cudaError_t run_any(const NormArgs &a, bool bwd) {
    const NormP p = params(a);
    const int wf32 = a.wdtype == GDN_DTYPE_F32, gate = gate_of(a);
    const int grid = walk_blocks(a.R, 8);
    if (!bwd) {
        norm_fwd_any_kernel<T><<<grid, kThreads, 0, a.stream>>>(p, (const T *)a.x, a.weight, a.bias, wf32, (const T *)a.gate, gate,
                                                               a.center, (T *)a.y, a.stats);
        return cudaGetLastError();
    }
    norm_bwd_any_kernel<T><<<grid, kThreads, 0, a.stream>>>(p, (const T *)a.x, a.weight, a.bias, wf32, (const T *)a.gate, gate,
                                                           a.center, (const T *)a.dy, a.stats, (T *)a.dx, (T *)a.dgate);
    const int blocks = any_dw_blocks(a);
    norm_dw_any_kernel<T><<<dim3(blocks, (a.D + 31) / 32), kThreads, 0, a.stream>>>(p, (const T *)a.x, (const T *)a.gate, gate,
                                                                                  (const T *)a.dy, a.stats, a.part);
    return sum_parts(a, blocks);
}

cudaError_t dispatch(const NormArgs &a, bool bwd) {
    if (a.dtype == GDN_DTYPE_BF16) return in_registers(a) ? by_width<__nv_bfloat16>(a, bwd) : run_any<__nv_bfloat16>(a, bwd);
    return in_registers(a) ? by_width<float>(a, bwd) : run_any<float>(a, bwd);
}

}  // namespace

size_t norm_part_bytes(const NormArgs &a) {
    const int wide = a.D / (a.dtype == GDN_DTYPE_BF16 ? 8 : 4) > 128;  // a block per row (by_width)
    const int blocks = in_registers(a) ? walk_blocks(a.R, most_per_sm(wide ? kThreads : 32)) : any_dw_blocks(a);
    return (size_t)blocks * 2 * a.D * sizeof(float);
}

cudaError_t launch_norm_fwd(const NormArgs &a) { return a.R ? dispatch(a, false) : cudaSuccess; }

cudaError_t launch_norm_bwd(const NormArgs &a) {
    if (a.R) return dispatch(a, true);
    return sum_parts(a, 0);  // no rows: the sums are zero
}

}  // namespace gdn
