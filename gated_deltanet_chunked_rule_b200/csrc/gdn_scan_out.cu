// gdn_scan_out.cu -- outputs of the tensor-core selective scan, chunk by chunk:
//
//   y_r = sum_s P_rs x_s + e^{gam_r} (C h)_r + D x_r,   P_rs = e^{gam_r - gam_s} delta_s (C B^T)_rs, s <= r
//
// from the chunk's entry state h (bf16, kept by the state pass). No chunk depends on another.
// A CTA (one per SM) takes one chunk and a run of heads of one group: S = C B^T is formed once
// for all of them (tcgen05, 128 x 128 in tensor memory). Two pipelines of eight warps take every
// other head: its rows of S are read back, scaled and stored as a bf16 P tile, P X and C h are
// two products of 64 columns per unit, joined by the epilogue in x's place and written by one
// TMA store. A thread has one row and every other 32 columns of it. Each pipeline has a warp that
// issues its products and one that loads (x two units ahead) and stores, so that neither a
// copy's nor a product's latency stands in the other's way. With one unit at a time in each
// of two CTAs per SM (four row warps) a unit took 5 us, nearly all of it waiting.
//
// The mask's exponentials: for a column left of the row's block of 32 tokens
// e^{gam_r - gam_s} delta_s factors at the block's start, into one factor per row and one per
// column and row block: two multiplications per element. Only the 32 x 32 diagonal blocks take
// one exponential each. P and h are the two roundings to bf16 (2^-8 of a term each, on different
// terms) ahead of the output's own.
#include <algorithm>

#include "gdn_scan_tc.cuh"

namespace gdn {
namespace scan_tc {
namespace {

using namespace sm100;
using namespace gdn::warp;

constexpr int kRowThreads = 512;
constexpr int kThreads = kRowThreads + 128;
// Registers: 640 threads are launched with 96 each; see the state kernel.
constexpr int kRowRegs = 104, kAuxRegs = 64;
static_assert(kRowThreads * kRowRegs + 128 * kAuxRegs <= kThreads * 96, "register split");
constexpr int kCt = 0, kP = 32768, kX = 98304, kHt = 163840;  // C | P of each pipeline (B first, in the first's) | x [2][2] | h [2]
struct Vec {
    float col[4][kC];  // [w][s]: e^{(start of row block w) - gam_s} delta_s left of block w, delta_s in it
    float gl[kC];      // log2 decay from the block's start
};
constexpr int kVec = 196608;
constexpr int kBarsAt = kVec + 2 * sizeof(Vec);
constexpr int kSmem = kBarsAt + 256 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kColS = 0, kColY = 128;  // S | per pipeline: P X, C h

struct OutP {
    Params p;
    int run;  // heads of a CTA
    const __nv_bfloat16 *tiles;
    __nv_bfloat16 *y;
};

struct PipeBars {
    uint64_t x_full[2], h_full, p_ready, y_full, y_done;
};

template <int K>
__global__ void __launch_bounds__(kThreads, 1)
scan_out_kernel(const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_c,
                const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y, const OutP q) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    const uint32_t sb = smem_u32(smem);
    const Params &p = q.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hg = p.H / p.G, runs = (hg + q.run - 1) / q.run, g = blockIdx.y / runs, h_first = (blockIdx.y % runs) * q.run;
    const int heads = min(q.run, hg - h_first);
    int n, local;
    if (!p.m.slot(blockIdx.x, kC, &n, &local)) return;
    const int t0 = p.m.begin(n) + local * kC, len = min(kC, p.m.end(n) - t0);
    const bool full_chunk = len == kC;

    uint64_t *cb_full = reinterpret_cast<uint64_t *>(smem + kBarsAt), *s_full = cb_full + 1;
    PipeBars *bars = reinterpret_cast<PipeBars *>(cb_full + 2);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    if (tid == 0) {
        mbar_init(cb_full, 1), mbar_init(s_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[i].x_full[0], 1), mbar_init(&bars[i].x_full[1], 1), mbar_init(&bars[i].h_full, 1);
            mbar_init(&bars[i].p_ready, 256), mbar_init(&bars[i].y_full, 1), mbar_init(&bars[i].y_done, 256);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 16) {
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
    // pipeline: warps 0-7, 16 (products), 18 (copies), and the same plus one
    const int pipe = tid < kRowThreads ? warp >> 3 : warp & 1;
    PipeBars &bar = bars[pipe];
    const int units = (heads - pipe + 1) / 2 * p.S;
    auto unit_at = [&](int i) { return (h_first + pipe + 2 * (i / p.S)) * p.S + i % p.S; };  // of the group
    const uint32_t pt = sb + kP + pipe * 32768, xt = sb + kX + pipe * 32768, ht = sb + kHt + pipe * 16384;
    const uint32_t col_px = kColY + pipe * 128, col_ch = col_px + 64;

    if (warp >= 16) {
    reg_dec<kAuxRegs>();
    if (warp >= 18) {  // copies
        if (lane == 0) {
            auto load_x = [&](int i) {
                const int u = unit_at(i);
                mbar_arrive_expect_tx(&bar.x_full[i & 1], 16384);
                tma_load_3d(smem + kX + pipe * 32768 + (i & 1) * 16384, &tm_x, &bar.x_full[i & 1], (u % p.S) * kPT, p.head(g, u), t0);
            };
            auto load_h = [&](int i) {
                mbar_arrive_expect_tx(&bar.h_full, K * kPT * 2);
                bulk_load(smem + kHt + pipe * 16384, q.tiles + (((size_t)blockIdx.x * p.G + g) * p.U + unit_at(i)) * (K * kPT),
                          K * kPT * 2, &bar.h_full);
            };
            if (pipe == 0) {
                mbar_arrive_expect_tx(cb_full, 2 * (K / 64) * 16384);
                for (int j = 0; j < K / 64; ++j) {
                    tma_load_3d(smem + kCt + j * 16384, &tm_c, cb_full, 64 * j, g, t0);
                    tma_load_3d(smem + kP + j * 16384, &tm_b, cb_full, 64 * j, g, t0);
                }
            }
            int xs = 0, hs = 0;  // loads issued
            if (units > 0) load_h(hs++), load_x(xs++);
            if (units > 1) load_x(xs++);
            bool ok = true;
            for (int i = 0; i < units && ok; ++i) {
                ok = wait_bar(&bar.y_full, i & 1, abort_flag);
                if (ok && i + 1 < units) load_h(hs++);  // the products have read h
                ok = ok && wait_bar(&bar.y_done, i & 1, abort_flag);  // y stands in x's tile (or is written)
                if (!ok) break;
                if (full_chunk) {
                    const int u = unit_at(i);
                    tma_store_3d(&tm_y, xt + (i & 1) * 16384, (u % p.S) * kPT, p.head(g, u), t0);
                    bulk_commit();
                    bulk_wait_read<0>();
                }
                if (i + 2 < units) load_x(xs++);
            }
            if (!ok) fail();
            // no copy outlives the CTA
            bool done = pipe || drain(cb_full, 0);
            for (int k = max(0, xs - 2); k < xs; ++k) done = drain(&bar.x_full[k & 1], (k >> 1) & 1) && done;
            if (hs) done = drain(&bar.h_full, (hs - 1) & 1) && done;
            if (!done) fail();
            bulk_wait_all();
        }
    } else {  // products
        if (lane == 0) {
            bool ok = wait_bar(cb_full, 0, abort_flag);
            tc_fence_after();
            const uint32_t c = cols(sb + kCt);
            if (ok && pipe == 0) {
                constexpr uint32_t id = idesc_bf16(128, 128, false, false);
                const uint32_t b = cols(sb + kP);
#pragma unroll
                for (int k = 0; k < K / 16; ++k) mma<kTokenHi, kTokenHi>(tmem + kColS, c + cstep(k), b + cstep(k), id, k > 0);
                mma_commit(s_full);
            }
            constexpr uint32_t id = idesc_bf16(128, 64, false, true);
            const uint32_t h = state_rows(ht), pm = cols(pt), x0 = rows(xt), x1 = rows(xt + 16384);
            for (int i = 0; i < units && ok; ++i) {
                if (i > 0) ok = wait_bar(&bar.y_done, (i - 1) & 1, abort_flag);  // the accumulators are read
                ok = ok && wait_bar(&bar.h_full, i & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < K / 16; ++k) mma<kTokenHi, kStateRowsHi<K>>(tmem + col_ch, c + cstep(k), h + srstep(k), id, k > 0);
                ok = wait_bar(&bar.x_full[i & 1], (i >> 1) & 1, abort_flag) && wait_bar(&bar.p_ready, i & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint32_t x = i & 1 ? x1 : x0;
#pragma unroll
                for (int k = 0; k < 8; ++k) mma<kTokenHi, kTokenHi>(tmem + col_px, pm + cstep(k), x + rstep(k), id, k > 0);
                mma_commit(&bar.y_full);
            }
            if (!ok) fail();
        }
    }
    } else {
        reg_inc<kRowRegs>();
        const int wr = warp & 3, half = (warp >> 2) & 1, row = wr * 32 + lane;  // row block, column half
        const bool live = row < len;
        const uint32_t lanes = (uint32_t)(wr * 32) << 16;
        Vec &vec = reinterpret_cast<Vec *>(smem + kVec)[pipe];
        float u_r = 0.f, e_r = 0.f, D = 0.f, g_delta, g_f, g_r;
        float4 g_tot;
        bool ok = true;
        auto fetch = [&](int h) {
            const float *gt = p.gates.at(blockIdx.x, p.H, h) + row;
            g_delta = gt[0], g_f = gt[kC], g_r = gt[2 * kC];
            g_tot = p.gates.totals(blockIdx.x, p.H, h);
        };
        if (units > 0) fetch(p.head(g, unit_at(0)));
        for (int i = 0; i < units; ++i) {
            const int u = unit_at(i), h = p.head(g, u);
            if (i % p.S == 0) {  // another head: its gates and its P
                float before, after, all;
                around(g_tot, wr, &before, &after, &all);
                u_r = ex2(g_f);
                e_r = ex2(before + g_f);
                if (half == 0) {
                    vec.gl[row] = g_f;
                    vec.col[wr][row] = g_delta;
                    const float t[4] = {g_tot.x, g_tot.y, g_tot.z, g_tot.w};
                    float to = g_r;
#pragma unroll
                    for (int w = 1; w < 4; ++w)
                        if (w > wr) {
                            vec.col[w][row] = ex2(to) * g_delta;
                            to += t[w];
                        }
                }
                D = p.D ? p.D[h] : 0.f;
                const float me = g_f;
                if (i + p.S < units) fetch(p.head(g, unit_at(i + p.S)));
                if (i == 0) ok = __all_sync(0xffffffffu, wait_bar(s_full, 0, abort_flag));
                if (pipe) named_sync<256>(2);
                else named_sync<256>(1);
                tc_fence_after();
#pragma unroll
                for (int bb = 0; bb < 2; ++bb) {
                    const int blk = half + 2 * bb;
                    const uint32_t at = pt + bb * 16384;
                    if (blk > wr) {  // right of the diagonal: zeros, once
                        if (i == 0)
#pragma unroll
                            for (int j = 0; j < 4; ++j) st_shared_v4(at + piece(row, half * 4 + j), 0u, 0u, 0u, 0u);
                        continue;
                    }
                    if (!ok) continue;
                    float v[32];
                    tmem_ld32(tmem + lanes + kColS + 32 * blk, v);
                    const float4 *vs = reinterpret_cast<const float4 *>(vec.col[wr] + 32 * blk);
                    if (blk < wr) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float4 c = vs[k];
                            v[4 * k] *= u_r * c.x, v[4 * k + 1] *= u_r * c.y, v[4 * k + 2] *= u_r * c.z, v[4 * k + 3] *= u_r * c.w;
                        }
                    } else {
                        const float4 *gs = reinterpret_cast<const float4 *>(vec.gl + 32 * blk);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float4 c = vs[k], l = gs[k];
                            v[4 * k] = 4 * k <= lane ? ex2(me - l.x) * c.x * v[4 * k] : 0.f;
                            v[4 * k + 1] = 4 * k + 1 <= lane ? ex2(me - l.y) * c.y * v[4 * k + 1] : 0.f;
                            v[4 * k + 2] = 4 * k + 2 <= lane ? ex2(me - l.z) * c.z * v[4 * k + 2] : 0.f;
                            v[4 * k + 3] = 4 * k + 3 <= lane ? ex2(me - l.w) * c.w * v[4 * k + 3] : 0.f;
                        }
                    }
                    if (!full_chunk) {  // rows and columns of the next sequence
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = live && 32 * blk + k < len ? v[k] : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        st_shared_v4(at + piece(row, half * 4 + j), pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                                     pack_bf16(v[8 * j + 4], v[8 * j + 5]), pack_bf16(v[8 * j + 6], v[8 * j + 7]));
                }
            }
            const uint32_t xb = xt + (i & 1) * 16384;
            ok = __all_sync(0xffffffffu, ok && wait_bar(&bar.x_full[i & 1], (i >> 1) & 1, abort_flag));
            if (ok && !live) {  // x rows of the next sequence: no product may meet them
#pragma unroll
                for (int j = 0; j < 4; ++j) st_shared_v4(xb + piece(row, half * 4 + j), 0u, 0u, 0u, 0u);
            }
            fence_proxy_async();
            tc_fence_before();
            mbar_arrive(&bar.p_ready);
            ok = __all_sync(0xffffffffu, ok && wait_bar(&bar.y_full, i & 1, abort_flag));
            tc_fence_after();
            if (ok) {
                uint32_t a[32], b[32];
                tmem_ld32_nowait(tmem + lanes + col_px + 32 * half, a);
                tmem_ld32_nowait(tmem + lanes + col_ch + 32 * half, b);
                uint4 xv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) xv[j] = ld_shared_v4(xb + piece(row, half * 4 + j));
                tmem_landed(a);
                tmem_landed(b);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = 8 * j + 2 * k;
                        o[k] = pack_bf16(fmaf(D, bf_lo(w[k]), fmaf(e_r, __uint_as_float(b[c]), __uint_as_float(a[c]))),
                                         fmaf(D, bf_hi(w[k]), fmaf(e_r, __uint_as_float(b[c + 1]), __uint_as_float(a[c + 1]))));
                    }
                    if (full_chunk)
                        st_shared_v4(xb + piece(row, half * 4 + j), o[0], o[1], o[2], o[3]);
                    else if (live)
                        *reinterpret_cast<uint4 *>(q.y + ((size_t)(t0 + row) * p.H + h) * p.P + (u % p.S) * kPT + half * 32 + 8 * j) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            fence_proxy_async();
            tc_fence_before();
            mbar_arrive(&bar.y_done);
        }
        if (!ok) fail();
    }
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int K>
cudaError_t run(const ScanArgs &a, const Gates &gates, const __nv_bfloat16 *tiles) {
    if (a.seq.total == 0) return cudaSuccess;
    CUtensorMap mb, mc, mx, my;
    if (!token_map(&mb, a.B, a.K, a.G, a.bs, a.seq.total) || !token_map(&mc, a.C, a.K, a.G, a.cs, a.seq.total) ||
        !token_map(&mx, a.x, a.P, a.H, a.xs, a.seq.total) || !token_map(&my, a.y, a.P, a.H, (long long)a.H * a.P, a.seq.total))
        return cudaErrorInvalidValue;
    OutP q{params(a, gates), 1, tiles, (__nv_bfloat16 *)a.y};
    const int slots = a.seq.slots(kC), hg = a.H / a.G, sms = sm_count();
    // Heads per CTA: a CTA costs about two units' time before its first (its tiles, S), and its two
    // pipelines share the heads; the fewest waves times that length.
    double best = 1e30;
    for (int r = 1; r <= hg && r <= 64; ++r) {
        const long long ctas = (long long)slots * a.G * ((hg + r - 1) / r);
        const double cost = (double)((ctas + sms - 1) / sms) * ((r + 1) / 2 * q.p.S + 2);
        if (cost < best) best = cost, q.run = r;
    }
    auto kernel = scan_out_kernel<K>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    TimedLaunch t("scan_out", a.stream);
    kernel<<<dim3(slots, a.G * ((hg + q.run - 1) / q.run)), kThreads, kSmem, a.stream>>>(mb, mc, mx, my, q);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_out(const ScanArgs &a, const Gates &g, const __nv_bfloat16 *tiles_hi) {
    return a.K == 128 ? run<128>(a, g, tiles_hi) : run<64>(a, g, tiles_hi);
}

}  // namespace scan_tc
}  // namespace gdn
