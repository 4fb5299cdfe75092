// gdn_scan_tc.cuh -- shared pieces of the tensor-core selective scan (bf16; state
// columns in slices of 64, token chunks of 128).
//
// One chunk (rows r, s; gam = in-chunk running sum of delta A; h entry state, g' = dh' the
// gradient of the exit state):
//
//   S = C B^T,  L_rs = e^{gam_r - gam_s} (s <= r)
//   y  = (L o S o delta_s) X + e^{gam_r} C h + D x
//   h' = e^{gam_C} h + B^T diag(delta e^{gam_C - gam}) X
//   g  = e^{gam_C} g' + C^T diag(e^{gam}) dY
//
// A "unit" is a head's slice of 64 state columns; unit u of group g is slice u % S of head
// g (H/G) + u / S, S = P/64. Per chunk slot and unit the state kernel keeps the entry state
// (forward) or exit gradient (reverse) as three bf16 tiles hi + lo + lo2 in a blocked layout: 8-column
// blocks of 16-byte rows, element (k, p) at (p/8) * K*16 + k*16 + (p%8)*2, which a lane-per-row
// store writes contiguously and tcgen05 reads without swizzle along either axis.
#pragma once

#include "gdn_host.cuh"
#include "gdn_layer.cuh"
#include "gdn_warp.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace scan_tc {

constexpr int kC = 128;   // tokens of a chunk
constexpr int kPT = 64;   // state columns of a unit

// The gates of every (chunk slot, head), from one small kernel: step sizes, and the log
// decay's sums (times log2 e) within blocks of 32 tokens, forwards up to and with the token
// and backwards after it, each summed from the end that matters so that it keeps its relative
// precision far into a chunk; tot: the four blocks' totals. A token past the sequence has
// delta 0 and decay 1.
struct Gates {
    float *v;    // [slots, H, 3, 128]: delta, forward, backward
    float *tot;  // [slots, H, 4]
    __device__ __forceinline__ const float *at(size_t slot, int H, int h) const { return v + (slot * H + h) * (3 * kC); }
    __device__ __forceinline__ float4 totals(size_t slot, int H, int h) const {
        return *reinterpret_cast<const float4 *>(tot + (slot * H + h) * 4);
    }
};

struct Params {
    SeqMap m;
    int G, H, K, P, S, U;  // U: units of a group
    int hg, sh;            // heads of a group; S = 1 << sh
    bool softplus;
    int dt_f32;
    long long dts;
    const void *dt;
    const float *A, *D, *dt_bias;
    Gates gates;
    unsigned *status;
    __device__ __forceinline__ int head(int g, int u) const { return g * hg + (u >> sh); }
    __device__ __forceinline__ int col0(int u) const { return (u & (S - 1)) * kPT; }  // a unit's first column
    __device__ __forceinline__ float raw_dt(int t, int h) const {
        const size_t at = (size_t)t * dts + h;
        const float v = dt_f32 ? ((const float *)dt)[at] : __bfloat162float(((const __nv_bfloat16 *)dt)[at]);
        return v + (dt_bias ? dt_bias[h] : 0.f);
    }
};

inline size_t gates_bytes(const ScanArgs &a) { return align_up((size_t)a.seq.slots(kC) * a.H * (3 * kC + 4) * 4); }

inline Gates gates_at(char *at, const ScanArgs &a) {
    Gates g;
    g.v = (float *)at;
    g.tot = g.v + (size_t)a.seq.slots(kC) * a.H * 3 * kC;
    return g;
}

inline Params params(const ScanArgs &a, const Gates &gates) {
    Params p;
    p.m = a.seq;
    p.G = a.G, p.H = a.H, p.K = a.K, p.P = a.P, p.S = a.P / kPT, p.U = a.H / a.G * p.S, p.hg = a.H / a.G, p.sh = p.S == 2;
    p.softplus = a.softplus, p.dt_f32 = a.dt_dtype == GDN_DTYPE_F32, p.dts = a.dts, p.dt = a.dt;
    p.A = a.A, p.D = a.D, p.dt_bias = a.dt_bias, p.gates = gates, p.status = a.status;
    return p;
}

// 2^x (relative error 2^-22)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

using warp::pack_bf16;
__device__ __forceinline__ uint32_t pack_bf16(F2 a) {
    const float2 v = get(a);
    return warp::pack_bf16(v.x, v.y);
}

// Sums of a chunk's block totals before and after block w, and all of them.
__device__ __forceinline__ void around(const float4 &t, int w, float *before, float *after, float *all) {
    const float a[4] = {t.x, t.y, t.z, t.w};
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        lo += k < w ? a[k] : 0.f;
        hi += k > w ? a[k] : 0.f;
    }
    *before = lo, *after = hi, *all = (a[0] + a[1]) + (a[2] + a[3]);
}

// Per-chunk tiles of every (chunk slot, unit): bf16 parts that together hold an fp32 element's 24 bits.
struct Tiles {
    __nv_bfloat16 *hi, *lo, *lo2;  // lo and lo2 both null: hi alone
};
inline size_t tile_bytes(const ScanArgs &a) {  // of one part
    return (size_t)a.seq.slots(kC) * a.H * (a.P / kPT) * a.K * kPT * 2;
}

// Maps of a [T, heads, width] token tensor whose tokens are `stride` elements apart: boxes of
// 64 columns x one head x 128 tokens, 128-byte swizzle.
inline bool token_map(CUtensorMap *m, const void *base, int width, int heads, long long stride, int total) {
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)(total > 0 ? total : 1)};
    const cuuint64_t str[2] = {(cuuint64_t)width * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, kC};
    return warp::make_bf16_map(m, base, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Operand descriptors as two words: the low one (address, leading offset) varies, k-step
// offsets are added to it; the high one (stride, version, layout) is a constant of the kind,
// so that an issuing thread holds one register per operand. Token tiles ([128 rows][64
// columns] bf16, 128-byte swizzle, 16384 bytes; the next 64 columns 16384 bytes on):
// contraction along the columns, or along the rows.
constexpr uint32_t kTokenHi = (1024u >> 4) | (1u << 14) | ((uint32_t)sm100::kSw128 << 29);
__device__ __forceinline__ uint32_t cols(uint32_t base) { return ((base >> 4) & 0x3fffu) | ((16u >> 4) << 16); }
__device__ __forceinline__ uint32_t rows(uint32_t base) { return ((base >> 4) & 0x3fffu) | ((16384u >> 4) << 16); }
constexpr uint32_t cstep(int k) { return (uint32_t)((k >> 2) * 16384 + (k & 3) * 32) >> 4; }
constexpr uint32_t rstep(int k) { return (uint32_t)(k * 2048) >> 4; }
// Blocked state tiles ([K rows][64 columns], no swizzle): contraction along the rows, or the
// columns.
template <int K>
constexpr uint32_t kStateRowsHi = (uint32_t)K | (1u << 14);  // stride K * 16
constexpr uint32_t kStateColsHi = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t state_rows(uint32_t base) { return ((base >> 4) & 0x3fffu) | ((128u >> 4) << 16); }
template <int K>
__device__ __forceinline__ uint32_t state_cols(uint32_t base) { return ((base >> 4) & 0x3fffu) | ((uint32_t)K << 16); }
constexpr uint32_t srstep(int k) { return (uint32_t)(k * 256) >> 4; }
template <int K>
constexpr uint32_t scstep(int k) {
    return (uint32_t)(k * 2 * K * 16) >> 4;
}

// D[tmem] (+)= A B of one k-step.
template <uint32_t A_HI, uint32_t B_HI>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "n"(A_HI), "n"(B_HI)
        : "memory");
}

// Byte offset of 16-byte piece j of row r of a token tile.
__device__ __forceinline__ uint32_t piece(int r, int j) { return r * 128 + ((j ^ (r & 7)) << 4); }

// Waits (bounded) for an asynchronous copy's phase, whatever else has failed.
__device__ __forceinline__ bool drain(uint64_t *bar, uint32_t parity) {
    const uint64_t t0 = warp::globaltimer();
    while (!sm100::mbar_try_wait(sm100::smem_u32(bar), parity))
        if (warp::globaltimer() - t0 > warp::kWaitNs) return false;
    return true;
}

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// What is left of two values beside their bf16 part.
__device__ __forceinline__ uint32_t split(float &x0, float &x1) {
    const uint32_t part = pack_bf16(x0, x1);
    x0 -= bf_lo(part), x1 -= bf_hi(part);
    return part;
}

// Eight consecutive columns of a state row as tile parts, at element `at`.
__device__ __forceinline__ void store_parts(const Tiles &t, size_t at, const float *v) {
    uint32_t hi[4], lo[4], lo2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float x0 = v[2 * j], x1 = v[2 * j + 1];
        hi[j] = split(x0, x1);
        if (t.lo) lo[j] = split(x0, x1), lo2[j] = pack_bf16(x0, x1);
    }
    *reinterpret_cast<uint4 *>(t.hi + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if (t.lo) {
        *reinterpret_cast<uint4 *>(t.lo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4 *>(t.lo2 + at) = make_uint4(lo2[0], lo2[1], lo2[2], lo2[3]);
    }
}

// Launchers of the kernels (see the .cu files).
// State pass over the chunks: REVERSE walks them backwards with C and dY in place of B and x.
struct StateArgs {
    const ScanArgs *a;
    Gates gates;
    bool reverse;
    bool after_gates;    // the launch before is launch_gates'
    int chunks_per_seg;  // 0: whole sequences
    bool products;       // the segments write their chunks' products (ScanArgs::products)
    float *seg;          // those: [chunk slots, units, 64 K]; otherwise [segment slots, units, K, 64]
    float *seg_gam;      // [segment slots, H]
    __nv_bfloat16 *starts;  // nullable: one pass within the segments only (forward, nothing kept); their
    float *before;          // starts as tiles, and the log decay from there to each chunk [slots, H]
    const float *first;  // h0 or dht, nullable
    float *last;         // final state or dh0, nullable
    Tiles tiles;         // hi nullable: no tiles kept
};
cudaError_t launch_gates(const ScanArgs &a, const Gates &g);
cudaError_t launch_states(const StateArgs &s);
// Segments that a problem's state passes are cut into, and their scratch.
int chunks_per_segment(const ScanArgs &a);
bool products_fit(const ScanArgs &a);
size_t segment_bytes(const ScanArgs &a);

// starts, before: as StateArgs', where the tiles are within segments of seg_tokens only.
size_t local_bytes(const ScanArgs &a);
struct Locals {
    int seg_tokens;  // 0: the tiles are whole
    const __nv_bfloat16 *starts;
    const float *before;
};
cudaError_t launch_out(const ScanArgs &a, const Gates &g, const __nv_bfloat16 *tiles_hi, const Locals &locals);

// Gradients from every chunk's entry state h and exit gradient g; scratch of grad_bytes.
size_t grad_bytes(const ScanArgs &a);
cudaError_t launch_grad(const ScanArgs &a, const Gates &gates, const Tiles &h, const Tiles &g, char *ws);

}  // namespace scan_tc
}  // namespace gdn
