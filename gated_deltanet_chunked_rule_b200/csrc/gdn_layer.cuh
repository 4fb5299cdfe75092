// gdn_layer.cuh -- declarations shared by the operators around the gated delta
// rule: the short causal convolution, the selective state space scan and the
// gated layer norm.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

// The kernel after this one may come up once every block of this one has started ...
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }
// ... and waits here, in every block, until this one has ended and its writes are there (launched
// the usual way it has waited already).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Sequences on the flattened token axis: B rows of T tokens, or N packed ones whose
// offsets stand in cu (device, [N + 1]). A kernel clamps what it reads from cu to
// [0, total], so an inconsistent copy never leads out of the tensors; one block of
// each call's first kernel that walks the sequences checks it and records GDN_ERR_DEVICE_ARG.
struct SeqMap {
    const int *cu;  // nullptr: no packing
    int N, T, total;

    __host__ __device__ __forceinline__ int begin(int n) const {
        if (!cu) return n * T;
        return min(max(cu[n], 0), total);
    }
    __host__ __device__ __forceinline__ int end(int n) const {
        if (!cu) return (n + 1) * T;
        return max(begin(n), min(max(cu[n + 1], 0), total));
    }
    // Sequence that token t belongs to: the last n with begin(n) <= t.
    __device__ __forceinline__ int owner(int t) const {
        if (!cu) return t / T;
        int lo = 0, hi = N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cu[mid] <= t) lo = mid; else hi = mid - 1;
        }
        return lo;
    }
    // Slots of q tokens each, every sequence's slots one after another: sequence n's
    // begin at begin(n) / q + n. Since ceil(len / q) <= floor(end / q) - floor(begin / q) + 1
    // the ranges do not overlap, and total / q + N slots hold them all; the last slot of a
    // range may be unused. No table has to be built and the host needs no copy of cu.
    __device__ __forceinline__ int slot0(int n, int q) const {
        if (!cu) return n * ((T + q - 1) / q);
        return begin(n) / q + n;
    }
    // Sequence and slot within it of slot i; false if i is unused.
    __device__ __forceinline__ bool slot(int i, int q, int *n, int *local) const {
        if (!cu) {
            const int per = (T + q - 1) / q;
            *n = per ? i / per : i;
            *local = per ? i - *n * per : 0;
            return per && *n < N;
        }
        int lo = 0, hi = N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (slot0(mid, q) <= i) lo = mid; else hi = mid - 1;
        }
        *n = lo;
        *local = i - slot0(lo, q);
        return *local >= 0 && *local < (end(lo) - begin(lo) + q - 1) / q;
    }
    int slots(int q) const { return cu ? total / q + N : N * ((T + q - 1) / q); }  // upper bound (host)
};

// By one block: checks the packed offsets.
__device__ __forceinline__ void check_cu(const SeqMap &m, unsigned *status, int tid, int threads) {
    if (!m.cu) return;
    bool bad = false;
    for (int n = tid; n < m.N; n += threads) bad |= m.cu[n] < 0 || m.cu[n + 1] < m.cu[n] || m.cu[n + 1] > m.total;
    if (tid == 0) bad |= m.cu[0] != 0 || m.cu[m.N] != m.total;
    if (bad) set_status(status, GDN_ERR_DEVICE_ARG);
}

// Two fp32 operations per instruction (sm_100a), on register pairs.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(uint32_t a, uint32_t b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 get(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// kFast: single-instruction exponentials (relative error below 2^-18 for |x| < 16), enough
// where the results are rounded to bf16; the library's expf otherwise.
template <bool kFast>
__device__ __forceinline__ float sigmoid(float x) {
    return kFast ? __fdividef(1.f, 1.f + __expf(-x)) : 1.f / (1.f + expf(-x));
}

template <bool kFast>
__device__ __forceinline__ F2 sigmoid(F2 x) {
    if constexpr (!kFast) {
        const float2 v = get(x);
        return f2(sigmoid<false>(v.x), sigmoid<false>(v.y));
    }
    const float log2e = 1.4426950408889634f;
    const float2 t = get(mul2(x, f2(-log2e, -log2e)));
    float a, b;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(t.y));
    const float2 d = get(add2(f2(a, b), f2(1.f, 1.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(d.y));
    return f2(a, b);
}

// VEC consecutive fp32 values as elements, by one 16-byte access.
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[VEC]) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <typename T, int PAIRS>
__device__ __forceinline__ void store_pairs(T *p, const F2 (&v)[PAIRS]) {
    float f[2 * PAIRS];
#pragma unroll
    for (int m = 0; m < PAIRS; ++m) {
        const float2 a = get(v[m]);
        f[2 * m] = a.x, f[2 * m + 1] = a.y;
    }
    store_vec<T, 2 * PAIRS>(p, f);
}

// --------------------------------------------------------------- convolution
struct ConvArgs {
    SeqMap seq;
    int C, W, dtype;
    bool silu;
    long long x_stride;  // elements between tokens of x
    const void *x, *weight, *bias, *state;  // weight [C, W]; bias [C], state [N, W-1, C] nullable
    void *y, *final_state;                  // final nullable
    // backward
    const void *dy, *dfinal;                // dfinal nullable
    void *dx, *dweight, *dbias, *dstate;    // dbias, dstate nullable
    float *part;                            // [token blocks, W + 1, C]
    unsigned *status;
    cudaStream_t stream;
};
size_t conv_part_bytes(int total, int C, int W);
cudaError_t launch_conv_fwd(const ConvArgs &a);
cudaError_t launch_conv_bwd(const ConvArgs &a);
cudaError_t launch_conv_update(const ConvArgs &a);  // state in place, seq without packing

// Row of the states [N, w1, C] that holds token t of sequence n, which ends at e: one of the last w1
// before e, or -1. (Where the offsets end early, the last sequence is walked on behind its e.)
__host__ __device__ __forceinline__ long long kept_row(int n, int e, int t, int w1) {
    return t < e && t >= e - w1 ? (long long)n * w1 + w1 - (e - t) : -1;
}

// ----------------------------------------------------------------- layer norm
struct NormArgs {
    long long R;
    int D, dtype, wdtype;
    float eps;
    bool center, gate_first;
    const void *x, *weight, *bias, *gate;  // bias, gate nullable
    void *y;
    float *stats;                          // [R, 2]: mean, 1 / standard deviation
    const void *dy;
    void *dx, *dgate, *dweight, *dbias;
    float *part;                           // [blocks, 2, D]
    cudaStream_t stream;
};
size_t norm_part_bytes(const NormArgs &a);
cudaError_t launch_norm_fwd(const NormArgs &a);
cudaError_t launch_norm_bwd(const NormArgs &a);

// ----------------------------------------------------------------------- scan
struct ScanArgs {
    SeqMap seq;
    int G, H, K, P, dtype, dt_dtype;
    bool softplus;
    bool tensor_cores, products;  // the call's path, and how its state passes join segments: decided once per call
    long long xs, bs, cs, dts;  // elements between tokens of x, B, C, dt
    const void *x, *dt, *B, *C;
    const float *A, *D, *dt_bias, *h0;  // D, dt_bias, h0 nullable
    void *y;
    float *final_state;                 // nullable
    // backward
    const void *dy;
    const float *dht;
    void *dx, *ddt, *dB, *dC;
    float *dA, *dD, *ddt_bias, *dh0;
    void *saved, *ws;
    unsigned *status;
    cudaStream_t stream;
};
cudaError_t launch_scan_step(const ScanArgs &a);
cudaError_t launch_scan_simt_fwd(const ScanArgs &a);
size_t scan_simt_fwd_bytes(const ScanArgs &a);
size_t scan_simt_bwd_bytes(const ScanArgs &a);
cudaError_t launch_scan_simt_bwd(const ScanArgs &a);
// dA, ddt_bias, dD from parts [slots, 3, H].
cudaError_t launch_scan_sum(const float *part, int slots, const ScanArgs &a);

}  // namespace gdn
