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
// (forward) or exit gradient (reverse) as two bf16 tiles hi + lo in a blocked layout: 8-column
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

struct Params {
    SeqMap m;
    int G, H, K, P, S, U;  // U: units of a group
    bool softplus;
    int dt_f32;
    long long dts;
    const void *dt;
    const float *A, *D, *dt_bias;
    unsigned *status;
    __device__ __forceinline__ int head(int g, int u) const { return g * (H / G) + u / S; }
    __device__ __forceinline__ float raw_dt(int t, int h) const {
        const size_t at = (size_t)t * dts + h;
        const float v = dt_f32 ? ((const float *)dt)[at] : __bfloat162float(((const __nv_bfloat16 *)dt)[at]);
        return v + (dt_bias ? dt_bias[h] : 0.f);
    }
    // log1p(exp(v)), or v itself above 20 (where they agree to fp32 precision)
    __device__ __forceinline__ float delta(float raw) const {
        return softplus ? (raw > 20.f ? raw : log1pf(expf(raw))) : raw;
    }
};

inline Params params(const ScanArgs &a) {
    Params p;
    p.m = a.seq;
    p.G = a.G, p.H = a.H, p.K = a.K, p.P = a.P, p.S = a.P / kPT, p.U = a.H / a.G * p.S;
    p.softplus = a.softplus, p.dt_f32 = a.dt_dtype == GDN_DTYPE_F32, p.dts = a.dts, p.dt = a.dt;
    p.A = a.A, p.D = a.D, p.dt_bias = a.dt_bias, p.status = a.status;
    return p;
}

// Per-chunk tiles: hi, then lo, of every (chunk slot, unit).
struct Tiles {
    __nv_bfloat16 *hi, *lo;  // lo nullable
};
inline size_t tile_bytes(const ScanArgs &a) {  // of hi (or lo)
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

// Operand descriptors. Token tiles ([128 rows][64 columns] bf16, 128-byte swizzle, 16384 bytes;
// the next 64 columns 16384 bytes on): contraction along the columns, or along the rows.
__device__ __forceinline__ uint64_t by_cols(uint32_t base, int ks) {
    return sm100::smem_desc(base + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024, sm100::kSw128);
}
__device__ __forceinline__ uint64_t by_rows(uint32_t base, int ks) {
    return sm100::smem_desc(base + ks * 2048, 16384, 1024, sm100::kSw128);
}
// Blocked state tiles ([K rows][64 columns]): contraction along the rows, or the columns.
template <int K>
__device__ __forceinline__ uint64_t state_by_rows(uint32_t base, int ks) {
    return sm100::smem_desc(base + ks * 256, 128, K * 16, sm100::kSwNone);
}
template <int K>
__device__ __forceinline__ uint64_t state_by_cols(uint32_t base, int ks) {
    return sm100::smem_desc(base + ks * (2 * K * 16), K * 16, 128, sm100::kSwNone);
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

// Launchers of the kernels (see the .cu files).
// State pass over the chunks: REVERSE walks them backwards with C and dY in place of B and x.
struct StateArgs {
    const ScanArgs *a;
    bool reverse;
    int chunks_per_seg;  // 0: whole sequences
    float *seg;          // [segment slots, units, 64, K] scratch (segments only)
    float *seg_gam;      // [segment slots, H]
    const float *first;  // h0 or dht, nullable
    float *last;         // final state or dh0, nullable
    Tiles tiles;         // hi nullable: no tiles kept
};
cudaError_t launch_states(const StateArgs &s);
// Segments that a problem's state passes are cut into, and their scratch.
int chunks_per_segment(const ScanArgs &a);
size_t segment_bytes(const ScanArgs &a);

cudaError_t launch_out(const ScanArgs &a, const __nv_bfloat16 *tiles_hi);

// Gradients from every chunk's entry state h and exit gradient g; scratch of grad_bytes.
size_t grad_bytes(const ScanArgs &a);
cudaError_t launch_grad(const ScanArgs &a, const Tiles &h, const Tiles &g, char *ws);

}  // namespace scan_tc
}  // namespace gdn
