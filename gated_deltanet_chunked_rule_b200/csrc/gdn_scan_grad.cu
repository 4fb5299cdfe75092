// gdn_scan_grad.cu -- per-chunk gradients of the tensor-core selective scan. Chunks do not
// depend on each other: the entry states h and the exit-state gradients g' of all chunks are
// there (three bf16 parts each from the state passes).
//
// Per chunk and head (rows r, s; L_rs = e^{gam_r - gam_s} for s <= r; delta = the step sizes):
//
//   S = C B^T,   Q = dY X^T,   W = L o S o Q
//   dx_s = delta_s [ (L o S)^T dY + e^{gam_C - gam_s} B g' ]_s + D dY_s
//   dC   = sum over heads  (L o Q o delta_s) B   + (e^{gam} dY) h^T
//   dB   = sum over heads  (L o Q o delta_s)^T C + (delta e^{gam_C - gam} X) g'^T
//   w_s  = sum_r W_rs + e^{gam_C - gam_s} x_s.(B g')_s                    (d/d delta_s, direct)
//   dgam: the gradient of token t's log decay is what crosses t, every pair once:
//         sum_{r >= t > s} W_rs delta_s + sum_{r >= t} e^{gam_r} dY_r.(C h)_r
//         + sum_{s < t} delta_s e^{gam_C - gam_s} x_s.(B g')_s + e^{gam_C} <h, g'>
//   ddelta_t = A dgam_t + w_t
//
// Everything that ends in an fp32 result (dA, ddt, its bias) is formed in fp32 from exact
// products and states in three bf16 parts, 24 bits; sums of the crossing pairs run forward or
// backward and nothing is taken off again (inside a 32 x 32 diagonal block: a prefix over the columns, summed
// over the rows from each column on). Two parts, and row minus column sums inside the blocks, left dA and the
// bias off by 1e-6 to 4e-6 of their norm; 2e-7 to 1e-6 now, for 17 us of this kernel's and 10 of the state
// kernels' (2 x 4096 tokens, 16 heads of 128). bf16 results take one rounded operand per
// term: L o S and the scaled rows; the summed L o Q o delta is cut in two bf16 parts, its products being taken only
// once (0.6 us; with one, dB and dC came out at 2.3e-3 and up to 2.6e-3 of their norm, half as much again as
// their own rounding).
//
// A CTA (one per SM) takes one chunk and a run of units (a head's 64 columns; linear in them)
// of one group. The products with B and C of the masked Q are taken once, after the masked
// Qs are summed over the units in registers; dC and dB stay in tensor memory meanwhile (S |
// one 128-column work region | dC | dB = 512 columns). The work region holds C h, then Q, then
// (L o S)^T dY and B g'; e^{gam} dY h^T and X g'^T run while the mask is applied. The states' third parts
// have no shared memory of their own: h's stands in P's place until the mask, g's in the scaled dY's once that
// is multiplied, so that <h, g'> is summed in two places. Warps 0-7: a
// thread per row and column half; warp 8 issues the products on the work region, warp 9 those of
// dC and dB, warp 10 loads (TMA, bulk copies) and stores: a tile's next load is issued as soon as
// its last reader is done; dY has two tiles, and dx leaves through its dY's. The row warps need the
// registers of the copying and issuing ones: beside 220 KB of shared memory the L1 holds no spills,
// and with 60 spilled words the mask alone took 12000 cycles. What the gates' gradients are made of
// (row and column sums) goes to memory, and a small kernel scans it: in the row warps the scans and
// the barriers they need cost 2500 cycles per head.
//
// Bound by the chain of one unit's stages, about 11500 cycles: the mask takes 3400 (row block 3,
// whose two warps share a scheduler, has four column blocks to row block 0's one), the products
// after it 1800, reading dx 1000. 2 x 4096 tokens, 16 heads of 128, K = 128: 135 us, and 13 us the
// gates' gradients; its tiles and rows alone are 320 MB, 50 us. With states in two parts 117 us (and then 150
// with one fp32 operation per instruction, 135 with the scans in the row warps and one dY tile). Tried and
// not better: Q in two halves with B g' under the mask (the products' operand reads then slow the row
// warps), 16 row warps (spills), <h, g'> in the idle warp 11 (8 us more).
#include <algorithm>

#include "gdn_scan_tc.cuh"

namespace gdn {
namespace scan_tc {
namespace {

using namespace sm100;
using namespace gdn::warp;

constexpr int kRowThreads = 256;
constexpr int kThreads = kRowThreads + 128;
constexpr int kRowRegs = 208, kAuxRegs = 88;  // 384 threads are launched with 168 each
static_assert(kRowThreads * kRowRegs + 128 * kAuxRegs <= kThreads * 168, "register split");
// B | C | P (before it h's third part; at the end the summed masked Q's high part) | x, then scaled x | dY, then dx | h hi,
// lo (at the end the summed masked Q's low part) | g' hi, lo | scaled dY, then g's third part | dY, then dx, of every second unit
constexpr int kB = 0, kCt = 32768, kPm = 65536, kX = 98304, kY = 114688, kH = 131072, kG = 163840, kSy = 196608, kY1 = 212992;
constexpr int kMl = kH, kH2 = kPm, kG2 = kSy;
static_assert(kG - kMl >= kC * kC * 2 && kMl % 1024 == 0, "the low part takes h's place");
constexpr int kVec = 229376;
struct Vec {
    float v[3][kC];     // [w - 1]: e^{(start of row block w) - gam_s} for s left of block w
    float gl[kC];       // log2 decay from the row block's start
    float delta[kC];
};
constexpr int kBarsAt = kVec + (sizeof(Vec) + 15) / 16 * 16;
constexpr int kSmem = kBarsAt + 192;
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kColS = 0, kColR = 128, kColC = 256, kColB = 384;

// What the gates' gradients are made of, of one unit (a head's 64 columns), per token; h: column
// half, w: row block. The entries of blocks right of the diagonal are not written.
struct Sums {
    float rowi[2][kC];     // [h]: e^{gam_r} dY_r.(C h)_r
    float bt[2][kC];       // [h]: e^{gam_C - gam_s} x_s.(B g')_s
    float dD[2][kC];       // [h]: dY_r.x_r
    float rsum[4][2][kC];  // [block][h]: row sums of W delta, strictly below the diagonal
    float csum[4][kC];     // [w]: column sums of W, strictly below the diagonal
    float wdiag[kC];       // W_tt
    float cross[kC];       // sum_{r >= t, s < t} W_rs delta_s inside t's diagonal block, s in t's half of its columns
    float hg[32];          // [warp]: <h, g'>
};

struct GradP {
    Params p;
    int run, runs;
    Tiles h, g;
    __nv_bfloat16 *dx, *dB, *dC;
    Sums *sums;      // [slots, H, slices of a head]
    float *part_bc;  // [2][runs][total, G, K] where runs > 1
};

// Sum over the warp's lanes of a[i], b[i], delivered to lane i (a), 16 + i (b).
__device__ __forceinline__ float lane_sums(float (&a)[16], const float (&b)[16], int lane) {
    const bool upper = lane & 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float send = upper ? a[i] : b[i], keep = upper ? b[i] : a[i];
        a[i] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? a[i] : a[i + o], keep = up ? a[i + o] : a[i];
            a[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return a[0];
}

// Product of two blocked state tiles: this thread's elements of the row threads'.
template <int K>
__device__ __forceinline__ float dot_elements(uint32_t a, uint32_t b, int tid) {
    F2 v = f2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < K * kPT / 8 / kRowThreads; ++j) {
        const uint32_t at = (j * kRowThreads + tid) * 16;
        const uint4 x = ld_shared_v4(a + at), y = ld_shared_v4(b + at);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) v = fma2(f2(bf_lo(xw[k]), bf_hi(xw[k])), f2(bf_lo(yw[k]), bf_hi(yw[k])), v);
    }
    const float2 s = get(v);
    return s.x + s.y;
}

// Sum over the warp's lanes of a[i], delivered to lanes 2 i and 2 i + 1.
__device__ __forceinline__ float lane_sums(float (&a)[16], int lane) {
#pragma unroll
    for (int o = 16; o > 1; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o / 2; ++i) {
            const float send = up ? a[i] : a[i + o / 2], keep = up ? a[i + o / 2] : a[i];
            a[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return a[0] + __shfl_xor_sync(0xffffffffu, a[0], 1);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int K>
__global__ void __launch_bounds__(kThreads, 1)
scan_grad_kernel(const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_c,
                 const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_dy,
                 const __grid_constant__ CUtensorMap tm_dx, const GradP q) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    const Params &p = q.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (sb & 1023) {  // the swizzled tiles' alignment
        set_status(p.status, GDN_ERR_CUDA);
        return;
    }
    const int g = blockIdx.y / q.runs, run = blockIdx.y % q.runs, u_first = run * q.run;
    const int units = min(q.run, p.U - u_first);
    int n, local;
    if (!p.m.slot(blockIdx.x, kC, &n, &local)) return;
    const int t0 = p.m.begin(n) + local * kC, len = min(kC, p.m.end(n) - t0);
    const bool full_chunk = len == kC;
    constexpr int kTile = K * kPT * 2;

    Vec &vec = *reinterpret_cast<Vec *>(smem + kVec);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kBarsAt);
    uint64_t *cb_full = bars, *h_full = bars + 1, *g_full = bars + 2, *x_full = bars + 3, *y_full = bars + 4;  // loads; dY: two
    uint64_t *ch_full = bars + 6, *q_full = bars + 7, *cd_full = bars + 8, *dx_full = bars + 9, *end_full = bars + 10;  // products
    uint64_t *cb_ready = bars + 11, *r_free = bars + 12, *s_ready = bars + 13, *p_ready = bars + 14, *hg_read = bars + 15,
             *dx_done = bars + 16, *m_ready = bars + 18;  // the row threads; dx_done: two
    uint64_t *h2_full = bars + 19, *g2_full = bars + 20;  // loads of the states' third parts
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 21);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    if (tid == 0) {
        for (int i = 0; i < 11; ++i) mbar_init(bars + i, 1);
        for (int i = 11; i < 19; ++i) mbar_init(bars + i, kRowThreads);
        mbar_init(h2_full, 1), mbar_init(g2_full, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 8) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto fail = [&]() {
        *abort_flag = 1;
        set_status(p.status, GDN_ERR_TIMEOUT);
    };
    constexpr uint32_t idQ = idesc_bf16(128, 128, false, false), idH = idesc_bf16(128, 64, false, true),
                       idO = idesc_bf16(128, K, false, false), idX = idesc_bf16(128, 64, true, true),
                       idC = idesc_bf16(128, K, false, true), idB = idesc_bf16(128, K, true, true);

    if (warp >= 8) {
        reg_dec<kAuxRegs>();
        if (warp == 8) {  // products on the work region
            if (lane == 0) {
                uint32_t b = cols(sb + kB), c = cols(sb + kCt), y = cols(sb + kY), x = cols(sb + kX), yr = rows(sb + kY),
                         pm = rows(sb + kPm), h0 = state_rows(sb + kH), h1 = state_rows(sb + kH + kTile),
                               g0 = state_rows(sb + kG), g1 = state_rows(sb + kG + kTile);
                uint32_t h2 = state_rows(sb + kH2), g2 = state_rows(sb + kG2);
                bool ok = wait_bar(cb_full, 0, abort_flag) && wait_bar(cb_ready, 0, abort_flag);
                tc_fence_after();
                if (ok) {
#pragma unroll
                    for (int k = 0; k < K / 16; ++k) mma<kTokenHi, kTokenHi>(tmem + kColS, c + cstep(k), b + cstep(k), idQ, k > 0);
                }
                for (int i = 0; i < units && ok; ++i) {
                    // or the sums below are all formed ahead, in more registers than there are
                    asm volatile("" : "+r"(b), "+r"(c), "+r"(y), "+r"(x), "+r"(yr), "+r"(pm), "+r"(h0), "+r"(h1), "+r"(g0), "+r"(g1), "+r"(h2), "+r"(g2));
                    const uint32_t y2 = (i & 1) * ((kY1 - kY) >> 4);
                    // C h
                    if (i > 0) ok = wait_bar(&dx_done[(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag);  // the work region is read
                    ok = ok && wait_bar(h_full, i & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < K / 16; ++k) {
                        mma<kTokenHi, kStateRowsHi<K>>(tmem + kColR, c + cstep(k), h0 + srstep(k), idH, k > 0);
                        mma<kTokenHi, kStateRowsHi<K>>(tmem + kColR, c + cstep(k), h1 + srstep(k), idH, true);
                    }
                    ok = wait_bar(h2_full, i & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < K / 16; ++k) mma<kTokenHi, kStateRowsHi<K>>(tmem + kColR, c + cstep(k), h2 + srstep(k), idH, true);
                    mma_commit(ch_full);
                    // Q = dY X^T
                    ok = wait_bar(x_full, i & 1, abort_flag) && wait_bar(&y_full[i & 1], (i >> 1) & 1, abort_flag) && wait_bar(r_free, i & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma<kTokenHi, kTokenHi>(tmem + kColR, y + y2 + cstep(k), x + cstep(k), idQ, k > 0);
                    mma_commit(q_full);
                    // (L o S)^T dY and B g'
                    ok = wait_bar(g_full, i & 1, abort_flag) && wait_bar(p_ready, i & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k) mma<kTokenHi, kTokenHi>(tmem + kColR, pm + rstep(k), yr + y2 + rstep(k), idX, k > 0);
#pragma unroll
                    for (int k = 0; k < K / 16; ++k) {
                        mma<kTokenHi, kStateRowsHi<K>>(tmem + kColR + 64, b + cstep(k), g0 + srstep(k), idH, k > 0);
                        mma<kTokenHi, kStateRowsHi<K>>(tmem + kColR + 64, b + cstep(k), g1 + srstep(k), idH, true);
                    }
                    ok = wait_bar(g2_full, i & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < K / 16; ++k) mma<kTokenHi, kStateRowsHi<K>>(tmem + kColR + 64, b + cstep(k), g2 + srstep(k), idH, true);
                    mma_commit(dx_full);
                }
                if (!ok) fail();
            }
        } else if (warp == 9) {  // dC and dB
            if (lane == 0) {
                const uint32_t sy = cols(sb + kSy), x = cols(sb + kX), h0 = state_cols<K>(sb + kH), h1 = state_cols<K>(sb + kH + kTile),
                               g0 = state_cols<K>(sb + kG), g1 = state_cols<K>(sb + kG + kTile);
                bool ok = true;
                for (int i = 0; i < units && ok; ++i) {
                    // dC += (e^gam dY) h^T, dB += (delta e^{gam_C - gam} X) g'^T
                    ok = wait_bar(h_full, i & 1, abort_flag) && wait_bar(g_full, i & 1, abort_flag) && wait_bar(s_ready, i & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        mma<kTokenHi, kStateColsHi>(tmem + kColC, sy + cstep(k), h0 + scstep<K>(k), idO, i + k > 0);
                        mma<kTokenHi, kStateColsHi>(tmem + kColB, x + cstep(k), g0 + scstep<K>(k), idO, i + k > 0);
                        mma<kTokenHi, kStateColsHi>(tmem + kColC, sy + cstep(k), h1 + scstep<K>(k), idO, true);
                        mma<kTokenHi, kStateColsHi>(tmem + kColB, x + cstep(k), g1 + scstep<K>(k), idO, true);
                    }
                    mma_commit(cd_full);
                }
                ok = ok && wait_bar(m_ready, 0, abort_flag);
                if (ok) {
                    tc_fence_after();
                    const uint32_t b = rows(sb + kB), c = rows(sb + kCt);
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const uint32_t mc = cols(sb + (part ? kMl : kPm)), mr = rows(sb + (part ? kMl : kPm));
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            mma<kTokenHi, kTokenHi>(tmem + kColC, mc + cstep(k), b + rstep(k), idC, true);
                            mma<kTokenHi, kTokenHi>(tmem + kColB, mr + rstep(k), c + rstep(k), idB, true);
                        }
                    }
                    mma_commit(end_full);
                }
                if (!ok) fail();
            }
        } else if (warp == 10) {  // copies
            if (lane == 0) {
                auto tile_at = [&](int i) { return (((size_t)blockIdx.x * p.G + g) * p.U + u_first + i) * (K * kPT); };
                auto load_pair = [&](int at, uint64_t *bar, const Tiles &t, int i) {
                    mbar_arrive_expect_tx(bar, 2 * kTile);
                    bulk_load(smem + at, t.hi + tile_at(i), kTile, bar);
                    bulk_load(smem + at + kTile, t.lo + tile_at(i), kTile, bar);
                };
                auto load_third = [&](int at, uint64_t *bar, const Tiles &t, int i) {
                    mbar_arrive_expect_tx(bar, kTile);
                    bulk_load(smem + at, t.lo2 + tile_at(i), kTile, bar);
                };
                auto load_rows = [&](int at, uint64_t *bar, const CUtensorMap *map, int i) {
                    const int u = u_first + i;
                    mbar_arrive_expect_tx(bar, 16384);
                    tma_load_3d(smem + at, map, bar, p.col0(u), p.head(g, u), t0);
                };
                mbar_arrive_expect_tx(cb_full, 2 * (K / 64) * 16384);
                for (int j = 0; j < K / 64; ++j) {
                    tma_load_3d(smem + kCt + j * 16384, &tm_c, cb_full, 64 * j, g, t0);
                    tma_load_3d(smem + kB + j * 16384, &tm_b, cb_full, 64 * j, g, t0);
                }
                int hs = 1, gs = 1, xs = 1, ys = 1, h2s = 1, g2s = 0;  // loads issued
                load_pair(kH, h_full, q.h, 0);
                load_third(kH2, h2_full, q.h, 0);
                load_rows(kX, x_full, &tm_x, 0);
                load_rows(kY, &y_full[0], &tm_dy, 0);
                if (units > 1) load_rows(kY1, &y_full[1], &tm_dy, 1), ++ys;
                load_pair(kG, g_full, q.g, 0);
                bool ok = true;
                for (int i = 0; i < units && ok; ++i) {
                    const bool more = i + 1 < units;
                    ok = wait_bar(cd_full, i & 1, abort_flag);
                    if (ok) load_third(kG2, g2_full, q.g, i), ++g2s;  // the scaled dY is read
                    if (ok && more) load_rows(kX, x_full, &tm_x, i + 1), ++xs;
                    ok = ok && wait_bar(hg_read, i & 1, abort_flag);
                    if (ok && more) load_pair(kH, h_full, q.h, i + 1), ++hs;
                    ok = ok && wait_bar(dx_full, i & 1, abort_flag);
                    if (ok && more) load_third(kH2, h2_full, q.h, i + 1), ++h2s;  // P is read
                    if (ok && more) load_pair(kG, g_full, q.g, i + 1), ++gs;
                    ok = ok && wait_bar(&dx_done[i & 1], (i >> 1) & 1, abort_flag);
                    if (!ok) break;
                    const int y = i & 1 ? kY1 : kY;
                    if (full_chunk) {  // dx stands in dY's tile
                        const int u = u_first + i;
                        tma_store_3d(&tm_dx, sb + y, p.col0(u), p.head(g, u), t0);
                        bulk_commit();
                        bulk_wait_read<0>();
                    }
                    if (i + 2 < units) load_rows(y, &y_full[i & 1], &tm_dy, i + 2), ++ys;
                }
                if (!ok) fail();
                // no copy outlives the CTA
                bool done = drain(cb_full, 0);
                done = drain(h_full, (hs - 1) & 1) && done;
                done = drain(g_full, (gs - 1) & 1) && done;
                done = drain(h2_full, (h2s - 1) & 1) && done;
                if (g2s) done = drain(g2_full, (g2s - 1) & 1) && done;
                done = drain(x_full, (xs - 1) & 1) && done;
                done = drain(&y_full[0], ((ys + 1) / 2 - 1) & 1) && done;
                if (ys > 1) done = drain(&y_full[1], (ys / 2 - 1) & 1) && done;
                if (!done) fail();
                bulk_wait_all();
            }
        }
    } else {
        reg_inc<kRowRegs>();
        const int wr = warp & 3, half = warp >> 2, row = wr * 32 + lane;  // row block, column half
        const bool live = row < len;
        const uint32_t lanes = (uint32_t)(wr * 32) << 16;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) { ok = __all_sync(0xffffffffu, ok && wait_bar(bar, parity, abort_flag)); };
        // rows of the next sequence: no product may meet them
        wait(cb_full, 0);
        if (ok && !live) {
#pragma unroll
            for (int j = 0; j < K / 8; ++j)
                st_shared_v4(sb + (half ? kCt : kB) + (j >> 3) * 16384 + piece(row, j & 7), 0u, 0u, 0u, 0u);
        }
        fence_proxy_async();
        mbar_arrive(cb_ready);

        // masked Q summed over the units: columns 16 half .. of every block of 32 (so that a row block's
        // two warps share its diagonal block)
        F2 msum[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) msum[k][j] = f2(0.f, 0.f);
        float u_r = 0.f, e_r = 0.f, tail = 0.f, delta = 0.f, D = 0.f;
        float n_delta, n_f, n_r, n_D;  // the next head's gates, on their way
        float4 n_tot;
        auto fetch = [&](int i) {
            const int h = p.head(g, u_first + min(i, units - 1));
            const float *gt = p.gates.at(blockIdx.x, p.H, h) + row;
            n_delta = gt[0], n_f = gt[kC], n_r = gt[2 * kC];
            n_tot = p.gates.totals(blockIdx.x, p.H, h);
            n_D = p.D ? p.D[h] : 0.f;
        };
        fetch(0);
        for (int i = 0; i < units; ++i) {
            const int u = u_first + i, h = p.head(g, u);
            Sums &sums = q.sums[((size_t)blockIdx.x * p.H + h) * p.S + (i & (p.S - 1))];
            if ((i & (p.S - 1)) == 0) {  // another head: its gates (the last one's vectors are read: dx_full)
                delta = n_delta, D = n_D;
                float before, after, all;
                around(n_tot, wr, &before, &after, &all);
                u_r = ex2(n_f), e_r = ex2(before + n_f), tail = ex2(after + n_r);
                if (half == 0) {
                    vec.gl[row] = n_f;
                    vec.delta[row] = delta;
                    const float t[4] = {n_tot.x, n_tot.y, n_tot.z, n_tot.w};
                    float to = n_r;
#pragma unroll
                    for (int w = 1; w < 4; ++w)
                        if (w > wr) {
                            vec.v[w - 1][row] = ex2(to);
                            to += t[w];
                        }
                }
            }
            // ---- rows of x and dY; e^gam dY for dC, dY.(C h)
            wait(x_full, i & 1);
            wait(&y_full[i & 1], (i >> 1) & 1);
            if (i > 0) wait(hg_read, (i - 1) & 1);  // every row thread has read g's third part: the scaled dY takes its place
            const uint32_t yb = sb + (i & 1 ? kY1 : kY);
            uint4 xr[4];  // x, this half's 32 columns
            float ri = 0.f, hg = 0.f;
            if (ok) {
                uint4 yr[4];
                F2 dd2 = f2(0.f, 0.f);
                const F2 ee = f2(e_r, e_r);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t at = piece(row, half * 4 + j);
                    xr[j] = live ? ld_shared_v4(sb + kX + at) : make_uint4(0u, 0u, 0u, 0u);
                    yr[j] = live ? ld_shared_v4(yb + at) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t at = piece(row, half * 4 + j);
                    const uint32_t w[4] = {yr[j].x, yr[j].y, yr[j].z, yr[j].w}, v[4] = {xr[j].x, xr[j].y, xr[j].z, xr[j].w};
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const F2 yy = f2(bf_lo(w[k]), bf_hi(w[k]));
                        dd2 = fma2(yy, f2(bf_lo(v[k]), bf_hi(v[k])), dd2);
                        o[k] = pack_bf16(mul2(ee, yy));
                    }
                    st_shared_v4(sb + kSy + at, o[0], o[1], o[2], o[3]);
                    if (!live) {
                        st_shared_v4(sb + kX + at, 0u, 0u, 0u, 0u);
                        st_shared_v4(yb + at, 0u, 0u, 0u, 0u);
                    }
                }
                sums.dD[half][row] = get(dd2).x + get(dd2).y;
                // <h, g'> (this thread's 32 elements): h's third part, while P is not in its place yet
                wait(h2_full, i & 1);
                wait(g_full, i & 1);
                if (ok) hg = dot_elements<K>(sb + kH2, sb + kG, tid);
                wait(ch_full, i & 1);
                tc_fence_after();
                float v[32];
                if (ok) {
                    tmem_ld32(tmem + lanes + kColR + 32 * half, v);
                    F2 ri2 = f2(0.f, 0.f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t w[4] = {yr[j].x, yr[j].y, yr[j].z, yr[j].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ri2 = fma2(f2(bf_lo(w[k]), bf_hi(w[k])), f2(v[8 * j + 2 * k], v[8 * j + 2 * k + 1]), ri2);
                    }
                    ri = live ? e_r * (get(ri2).x + get(ri2).y) : 0.f;
                }
            }
            fence_proxy_async();
            tc_fence_before();
            mbar_arrive(r_free);
            sums.rowi[half][row] = ri;
            if ((i & (p.S - 1)) == 0) named_sync<kRowThreads>(1);  // the gate vectors are written
            // ---- Q is there and x read by it: scaled x in its place
            wait(q_full, i & 1);
            tc_fence_after();
            if (ok) {
                const float sc = delta * tail;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t v[4] = {xr[j].x, xr[j].y, xr[j].z, xr[j].w};
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[k] = pack_bf16(sc * bf_lo(v[k]), sc * bf_hi(v[k]));
                    st_shared_v4(sb + kX + piece(row, half * 4 + j), o[0], o[1], o[2], o[3]);
                }
            }
            fence_proxy_async();
            mbar_arrive(s_ready);
            // ---- the mask, two column blocks at a time
#pragma unroll
            for (int kp = 0; kp < 2; ++kp) {
                float w[2][16];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int k = 2 * kp + b;
                    const uint32_t pt = sb + kPm + kp * 16384;
                    const uint32_t at[2] = {pt + piece(row, 4 * b + 2 * half), pt + piece(row, 4 * b + 2 * half + 1)};
                    if (k > wr || !ok) {  // right of the diagonal
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[b][j] = 0.f;
                        st_shared_v4(at[0], 0u, 0u, 0u, 0u);
                        st_shared_v4(at[1], 0u, 0u, 0u, 0u);
                        continue;
                    }
                    uint32_t sr[16], vr[16];
                    tmem_ld16_nowait(tmem + lanes + kColS + 32 * k + 16 * half, sr);
                    tmem_ld16_nowait(tmem + lanes + kColR + 32 * k + 16 * half, vr);
                    tmem_landed(sr);
                    tmem_landed(vr);
                    const float4 *dl = reinterpret_cast<const float4 *>(vec.delta + 32 * k + 16 * half);
                    F2 rs2 = f2(0.f, 0.f);
                    uint32_t o[8];
                    if (k < wr) {
                        const float4 *ve = reinterpret_cast<const float4 *>(vec.v[wr - 1] + 32 * k + 16 * half);
                        const F2 uu = f2(u_r, u_r);
#pragma unroll
                        for (int j4 = 0; j4 < 4; ++j4) {
                            const float4 d4 = dl[j4], v4 = ve[j4];
                            const F2 d[2] = {f2(d4.x, d4.y), f2(d4.z, d4.w)}, e[2] = {f2(v4.x, v4.y), f2(v4.z, v4.w)};
#pragma unroll
                            for (int jj = 0; jj < 2; ++jj) {
                                const int j = 2 * j4 + jj;
                                const F2 qv = f2(vr[2 * j], vr[2 * j + 1]), L = mul2(uu, e[jj]);
                                msum[k][j] = fma2(mul2(L, d[jj]), qv, msum[k][j]);
                                const F2 s = mul2(L, f2(sr[2 * j], sr[2 * j + 1])), ww = mul2(s, qv);
                                o[j] = pack_bf16(s);
                                rs2 = fma2(ww, d[jj], rs2);
                                const float2 w2 = get(ww);
                                w[b][2 * j] = w2.x, w[b][2 * j + 1] = w2.y;
                            }
                        }
                    } else {
                        const float4 *gl = reinterpret_cast<const float4 *>(vec.gl + 32 * k + 16 * half);
                        const float me = vec.gl[row];
                        float diag = 0.f;
#pragma unroll
                        for (int j4 = 0; j4 < 4; ++j4) {
                            const float4 d4 = dl[j4], v4 = gl[j4];
                            const F2 d[2] = {f2(d4.x, d4.y), f2(d4.z, d4.w)};
                            const float e[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                            for (int jj = 0; jj < 2; ++jj) {
                                const int j = 2 * j4 + jj, c = 16 * half + 2 * j - lane;
                                // masked by bits, not by a branch: all ones where column <= row, where < row
                                const uint32_t on0 = (uint32_t)((c - 1) >> 31), below0 = (uint32_t)(c >> 31), on1 = below0, below1 = (uint32_t)((c + 1) >> 31);
                                const F2 qv = f2(vr[2 * j], vr[2 * j + 1]);
                                const F2 L = f2(__float_as_uint(ex2(me - e[2 * jj])) & on0, __float_as_uint(ex2(me - e[2 * jj + 1])) & on1);
                                msum[k][j] = fma2(mul2(L, d[jj]), qv, msum[k][j]);
                                const F2 s = mul2(L, f2(sr[2 * j], sr[2 * j + 1]));
                                const float2 w2 = get(mul2(s, qv));
                                o[j] = pack_bf16(s);
                                diag += __uint_as_float(__float_as_uint(w2.x) & (on0 ^ below0)) + __uint_as_float(__float_as_uint(w2.y) & (on1 ^ below1));
                                w[b][2 * j] = __uint_as_float(__float_as_uint(w2.x) & below0);
                                w[b][2 * j + 1] = __uint_as_float(__float_as_uint(w2.y) & below1);
                                rs2 = fma2(f2(w[b][2 * j], w[b][2 * j + 1]), d[jj], rs2);
                            }
                        }
                        if (half == lane >> 4) sums.wdiag[row] = diag;
                    }
                    st_shared_v4(at[0], o[0], o[1], o[2], o[3]);
                    st_shared_v4(at[1], o[4], o[5], o[6], o[7]);
                    const float2 rs = get(rs2);
                    sums.rsum[k][half][row] = rs.x + rs.y;
                }
                if (ok && kp == wr >> 1) {  // the diagonal block: this row's part of what crosses each column, over the rows from it on
                    const float4 *dl = reinterpret_cast<const float4 *>(vec.delta + 32 * wr + 16 * half);
                    float cross[16], before = 0.f;
#pragma unroll
                    for (int j4 = 0; j4 < 4; ++j4) {
                        const float4 d4 = dl[j4];
                        const float d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = 4 * j4 + e;
                            cross[j] = 16 * half + j <= lane ? before : 0.f;
                            before = fmaf(wr & 1 ? w[1][j] : w[0][j], d[e], before);
                        }
                    }
                    const float x = lane_sums(cross, lane);
                    if (!(lane & 1)) sums.cross[32 * wr + 16 * half + (lane >> 1)] = x;
                }
                if (2 * kp <= wr) {
                    const float cs = lane_sums(w[0], w[1], lane);
                    sums.csum[wr][64 * kp + 32 * (lane >> 4) + 16 * half + (lane & 15)] = cs;
                }
            }
            fence_proxy_async();
            tc_fence_before();
            mbar_arrive(p_ready);
            fetch(i + 1);
            // ---- <h, g'>: g's third part (behind the scaled dY), then the first two of both
            wait(g2_full, i & 1);
            if (ok) {
                hg += dot_elements<K>(sb + kH, sb + kG2, tid);
#pragma unroll
                for (int j = 0; j < K * kPT / 8 / kRowThreads; ++j) {
                    const uint32_t at = (j * kRowThreads + tid) * 16;
                    const uint4 a = ld_shared_v4(sb + kH + at), b = ld_shared_v4(sb + kH + kTile + at);
                    const uint4 c = ld_shared_v4(sb + kG + at), d = ld_shared_v4(sb + kG + kTile + at);
                    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w}, cw[4] = {c.x, c.y, c.z, c.w},
                                   dw[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        hg = fmaf(bf_lo(aw[k]) + bf_lo(bw[k]), bf_lo(cw[k]) + bf_lo(dw[k]), hg);
                        hg = fmaf(bf_hi(aw[k]) + bf_hi(bw[k]), bf_hi(cw[k]) + bf_hi(dw[k]), hg);
                    }
                }
            }
            mbar_arrive(hg_read);
            hg = warp_sum(hg);
            if (lane == 0) sums.hg[warp] = hg;
            // ---- dx, in dY's place
            wait(cd_full, i & 1);
            wait(dx_full, i & 1);
            tc_fence_after();
            if (ok) {
                uint32_t ar[32], br[32];
                tmem_ld32_nowait(tmem + lanes + kColR + 32 * half, ar);
                tmem_ld32_nowait(tmem + lanes + kColR + 64 + 32 * half, br);
                uint4 yr[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) yr[j] = ld_shared_v4(yb + piece(row, half * 4 + j));
                tmem_landed(ar);
                tmem_landed(br);
                F2 s2 = f2(0.f, 0.f);
                const F2 tt = f2(tail, tail), de = f2(delta, delta), dd = f2(D, D);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t y[4] = {yr[j].x, yr[j].y, yr[j].z, yr[j].w}, v[4] = {xr[j].x, xr[j].y, xr[j].z, xr[j].w};
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = 8 * j + 2 * k;
                        const F2 bb = f2(br[c], br[c + 1]);
                        s2 = fma2(f2(bf_lo(v[k]), bf_hi(v[k])), bb, s2);
                        o[k] = pack_bf16(fma2(de, fma2(tt, bb, f2(ar[c], ar[c + 1])), mul2(dd, f2(bf_lo(y[k]), bf_hi(y[k])))));
                    }
                    if (full_chunk)
                        st_shared_v4(yb + piece(row, half * 4 + j), o[0], o[1], o[2], o[3]);
                    else if (live)
                        *reinterpret_cast<uint4 *>(q.dx + ((size_t)(t0 + row) * p.H + h) * p.P + p.col0(u) + half * 32 + 8 * j) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                }
                const float2 s = get(s2);
                sums.bt[half][row] = live ? tail * (s.x + s.y) : 0.f;
            }
            fence_proxy_async();
            tc_fence_before();
            mbar_arrive(&dx_done[i & 1]);
        }
        // ---- the summed masked Q in two parts, in P's place (its last product has completed: dx_full) and in
        // h's (its products have: cd_full, and so have its reads: hg_read)
        wait(hg_read, (units - 1) & 1);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t at = (k >> 1) * 16384 + piece(row, 4 * (k & 1) + 2 * half + j);
                uint32_t hi[4] = {}, lo[4] = {};
                if (k <= wr) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 m = get(msum[k][4 * j + e]);
                        hi[e] = pack_bf16(m.x, m.y);
                        lo[e] = pack_bf16(m.x - bf_lo(hi[e]), m.y - bf_hi(hi[e]));
                    }
                    st_shared_v4(sb + kPm + at, hi[0], hi[1], hi[2], hi[3]);  // (right of the diagonal zeros stand)
                }
                st_shared_v4(sb + kMl + at, lo[0], lo[1], lo[2], lo[3]);
            }
        fence_proxy_async();
        tc_fence_before();
        mbar_arrive(m_ready);
        wait(end_full, 0);
        tc_fence_after();
        if (ok) {
            const int c0 = half * (K / 2);
            const size_t at = ((size_t)(t0 + row) * p.G + g) * K + c0;
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                __nv_bfloat16 *out = which ? q.dB : q.dC;
                float *part = q.part_bc + ((size_t)which * q.runs + run) * p.m.total * p.G * K;
#pragma unroll
                for (int c = 0; c < K / 2; c += 32) {
                    float v[32];
                    tmem_ld32(tmem + lanes + (which ? kColB : kColC) + c0 + c, v);
                    if (!live) continue;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (q.runs == 1) {
                            *reinterpret_cast<uint4 *>(out + at + c + 8 * j) =
                                make_uint4(pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                                           pack_bf16(v[8 * j + 4], v[8 * j + 5]), pack_bf16(v[8 * j + 6], v[8 * j + 7]));
                        } else {
                            *reinterpret_cast<float4 *>(part + at + c + 8 * j) = make_float4(v[8 * j], v[8 * j + 1], v[8 * j + 2], v[8 * j + 3]);
                            *reinterpret_cast<float4 *>(part + at + c + 8 * j + 4) =
                                make_float4(v[8 * j + 4], v[8 * j + 5], v[8 * j + 6], v[8 * j + 7]);
                        }
                    }
                }
            }
        } else {
            fail();
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The gates' gradients of one chunk and head, a thread per token: dgam from the sums of crossing
// pairs, ddt, and the chunk's parts [slots, 3, H] of dA, ddt_bias and dD.
__global__ void __launch_bounds__(kC) scan_gate_grad_kernel(const Params p, const Sums *__restrict__ sums, void *ddt_out, float *__restrict__ part) {
    const int row = threadIdx.x, wr = row >> 5, lane = row & 31, h = blockIdx.y;
    __shared__ float tot[4][4];  // per row block: sums of rowi, delta bt, row sums left: of block 0, of block 1
    __shared__ float red[3][4];
    float *out = part + (size_t)blockIdx.x * 3 * p.H + h;
    int n, local;
    if (!p.m.slot(blockIdx.x, kC, &n, &local)) {  // an unused slot adds nothing
        if (row < 3) out[row * p.H] = 0.f;
        return;
    }
    const int t0 = p.m.begin(n) + local * kC;
    const bool live = t0 + row < p.m.end(n);
    const float delta = p.gates.at(blockIdx.x, p.H, h)[row];
    float before, after, all;
    around(p.gates.totals(blockIdx.x, p.H, h), wr, &before, &after, &all);
    // strictly lower W: sums of this token's row left of its block (rs), of its column below it (coff) and inside
    // it (cd), of its row's first half inside it (left)
    float rs[4] = {}, coff = 0.f, cd = 0.f, rw = 0.f, bt = 0.f, wd = 0.f, dD = 0.f, hg = 0.f, cross = 0.f, left = 0.f;
    for (int k = 0; k < p.S; ++k) {
        const Sums &s = sums[((size_t)blockIdx.x * p.H + h) * p.S + k];
        rw += s.rowi[0][row] + s.rowi[1][row];
        bt += s.bt[0][row] + s.bt[1][row];
        dD += s.dD[0][row] + s.dD[1][row];
        wd += s.wdiag[row];
        cross += s.cross[row], left += s.rsum[wr][0][row];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < wr) rs[w] += s.rsum[w][0][row] + s.rsum[w][1][row];
            if (w == wr) cd += s.csum[w][row];
            if (w > wr) coff += s.csum[w][row];
        }
        if (lane < 8) hg += s.hg[lane];
    }
    float roff = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        if (w < wr) roff += rs[w];
    hg = warp_sum(hg);
    float suf = rw + roff, pre = delta * (bt + coff);  // rows from t on, columns up to it
    const float pre_own = pre;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float a = __shfl_down_sync(0xffffffffu, suf, o), b = __shfl_up_sync(0xffffffffu, pre, o);
        const float c = __shfl_down_sync(0xffffffffu, left, o);
        if (lane + o < 32) suf += a, left += c;
        if (lane >= o) pre += b;
    }
    // inside the block: `cross`, and for its second half of columns the rows' first halves
    suf += lane >= 16 ? cross + left : cross;
    const float t_ri = warp_sum(rw), t_bt = warp_sum(delta * bt), r0 = warp_sum(wr > 0 ? rs[0] : 0.f), r1 = warp_sum(wr > 1 ? rs[1] : 0.f);
    if (lane == 0) tot[wr][0] = t_ri, tot[wr][1] = t_bt, tot[wr][2] = r0, tot[wr][3] = r1;
    __syncthreads();
    float dgam = suf + (pre - pre_own);
    for (int k = 0; k < 4; ++k) {
        if (k > wr) dgam += tot[k][0];
        if (k < wr) dgam += tot[k][1];
    }
    // pairs of blocks around this one: rows below, columns left
    if (wr == 1) dgam += tot[2][2] + tot[3][2];
    if (wr == 2) dgam += tot[3][2] + tot[3][3];
    dgam += ex2(all) * hg;
    float ddt = 0.f;
    if (live) {
        ddt = fmaf(p.A[h], dgam, cd + coff + wd + bt);
        if (p.softplus) ddt /= 1.f + expf(-p.raw_dt(t0 + row, h));
        const size_t at = (size_t)(t0 + row) * p.H + h;
        if (p.dt_f32) ((float *)ddt_out)[at] = ddt;
        else ((__nv_bfloat16 *)ddt_out)[at] = __float2bfloat16_rn(ddt);
    }
    const float a = warp_sum(live ? delta * dgam : 0.f), b = warp_sum(ddt), d = warp_sum(dD);
    if (lane == 0) red[0][wr] = a, red[1][wr] = b, red[2][wr] = d;
    __syncthreads();
    if (row < 3) out[row * p.H] = (red[row][0] + red[row][1]) + (red[row][2] + red[row][3]);
}

// dC, dB from the runs' fp32 parts, in a fixed order; 4 elements per thread.
__global__ void __launch_bounds__(256) scan_join_kernel(const float *__restrict__ part, int runs, long long n, __nv_bfloat16 *dC, __nv_bfloat16 *dB) {
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const float *src = part + (long long)blockIdx.y * runs * n + i;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < runs; ++k) {
        const float4 a = *reinterpret_cast<const float4 *>(src + k * n);
        v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
    }
    *reinterpret_cast<uint2 *>((blockIdx.y ? dB : dC) + i) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

// Units per CTA (whole heads): a CTA costs about three units' time besides them; the fewest
// waves times that length.
int units_per_cta(const ScanArgs &a) {
    const int S = a.P / kPT, U = a.H / a.G * S, slots = a.seq.slots(kC), sms = sm_count();
    double best = 1e30;
    int pick = U;
    for (int r = S; r <= U; r += S) {
        const long long ctas = (long long)slots * a.G * ((U + r - 1) / r);
        const double cost = (double)((ctas + sms - 1) / sms) * (r + 3);
        if (cost < best) best = cost, pick = r;
    }
    return pick;
}

int runs_of(const ScanArgs &a) {
    const int U = a.H / a.G * (a.P / kPT), r = units_per_cta(a);
    return (U + r - 1) / r;
}

size_t sums_bytes(const ScanArgs &a) { return align_up((size_t)a.seq.slots(kC) * a.H * (a.P / kPT) * sizeof(Sums)); }

template <int K>
cudaError_t run(const ScanArgs &a, const Gates &gates, const Tiles &h, const Tiles &gr, char *ws) {
    GradP q{};
    q.p = params(a, gates);
    q.run = units_per_cta(a), q.runs = runs_of(a);
    q.h = h, q.g = gr;
    q.dx = (__nv_bfloat16 *)a.dx, q.dB = (__nv_bfloat16 *)a.dB, q.dC = (__nv_bfloat16 *)a.dC;
    const int slots = a.seq.total ? a.seq.slots(kC) : 0;
    float *part = (float *)ws;
    q.sums = (Sums *)(ws + align_up((size_t)slots * 3 * a.H * 4));
    q.part_bc = (float *)((char *)q.sums + sums_bytes(a));
    if (slots) {
        CUtensorMap mb, mc, mx, my, mdx;
        const long long dense = (long long)a.H * a.P;
        if (!token_map(&mb, a.B, K, a.G, a.bs, a.seq.total) || !token_map(&mc, a.C, K, a.G, a.cs, a.seq.total) ||
            !token_map(&mx, a.x, a.P, a.H, a.xs, a.seq.total) || !token_map(&my, a.dy, a.P, a.H, dense, a.seq.total) ||
            !token_map(&mdx, a.dx, a.P, a.H, dense, a.seq.total))
            return cudaErrorInvalidValue;
        auto kernel = scan_grad_kernel<K>;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        {
            TimedLaunch t("scan_grad", a.stream);
            kernel<<<dim3(slots, a.G * q.runs), kThreads, kSmem, a.stream>>>(mb, mc, mx, my, mdx, q);
        }
        {
            TimedLaunch t("scan_gate_grad", a.stream);
            scan_gate_grad_kernel<<<dim3(slots, a.H), kC, 0, a.stream>>>(q.p, q.sums, a.ddt, part);
        }
        if (q.runs > 1) {
            TimedLaunch t("scan_join", a.stream);
            const long long n = (long long)a.seq.total * a.G * K;
            scan_join_kernel<<<dim3((unsigned)((n / 4 + 255) / 256), 2), 256, 0, a.stream>>>(q.part_bc, q.runs, n, q.dC, q.dB);
        }
    }
    TimedLaunch t("scan_sum", a.stream);
    return launch_scan_sum(part, slots, a);
}

}  // namespace

size_t grad_bytes(const ScanArgs &a) {
    if (!a.seq.total) return 256;
    const int runs = runs_of(a);
    return align_up((size_t)a.seq.slots(kC) * 3 * a.H * 4) + sums_bytes(a) + (runs > 1 ? align_up(2ull * runs * a.seq.total * a.G * a.K * 4) : 0);
}

cudaError_t launch_grad(const ScanArgs &a, const Gates &gates, const Tiles &h, const Tiles &g, char *ws) {
    return a.K == 128 ? run<128>(a, gates, h, g, ws) : run<64>(a, gates, h, g, ws);
}

}  // namespace scan_tc
}  // namespace gdn
