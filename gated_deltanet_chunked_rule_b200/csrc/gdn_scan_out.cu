// gdn_scan_out.cu -- outputs of the tensor-core selective scan, chunk by chunk:
//
//   y_r = sum_s P_rs x_s + e^{gam_r} (C h)_r + D x_r,   P_rs = e^{gam_r - gam_s} delta_s (C B^T)_rs, s <= r
//
// from the chunk's entry state h (bf16, kept by the state pass), or with LOCAL from the state within
// its segment, h_l, the segment's start h_s and the decay f between: C h = C h_l + f C h_s (each
// tile rounded once, on terms of its own). No chunk depends on another.
// A CTA (one per SM) takes one chunk and a run of heads of one group: S = C B^T is formed once
// for all of them (tcgen05, 128 x 128 in tensor memory). Per head its rows are read back,
// scaled and stored as a bf16 P tile; P X and C h are two products of 64 columns per unit,
// joined by the epilogue in x's place and written by one TMA store. Sixteen warps work on one
// unit (a thread per row and column quarter) and mask the next head's P before they take up
// this unit's products, so that the tensor core's latency is behind the mask: P, the
// accumulators and h have two buffers, x three. Warp 16 issues the products, warp 17 loads and
// stores, warps 18 and 19 prepare the heads' row and column factors a head ahead. Two units side
// by side in eight warps each, without that overlap, took 4.7 us; a unit takes 1.65 us now.
// 8192 tokens, 64 heads: 57 us, 128 CTAs; 32768 packed tokens, 32 heads in 4 groups: 151 us. Bound by
// the row warps: their schedulers issue in 62 % of the cycles and wait for tensor memory and shared
// memory in the rest (a unit's products and tiles need 0.8 us of the shared memory's bandwidth). With the
// row warps forming their own row factors 64 us; packed pairs of fp32 in the mask, whose operands
// have to be moved together first, 71 us.
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
// C | P [2] (B first, in the first's) | x [3] | h [2] | h_s [2]
constexpr int kCt = 0, kP = 32768, kX = 98304, kHt = 147456, kHs = 180224;
struct Vec {
    float col[4][kC];  // [w][s]: e^{(start of row block w) - gam_s} delta_s left of block w, delta_s in it
    float gl[kC];      // log2 decay from the block's start
    float row[4][kC];  // e^{gam_r}, then (LOCAL) also times f; e^{from the row block's start}; D
};
constexpr int kVec = 212992;
constexpr int kBarsAt = kVec + 2 * sizeof(Vec);
constexpr int kSmem = kBarsAt + 256 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kColS = 0, kColY = 128, kYCols = 192;  // S | [2]: P X, C h, C h_s

struct OutP {
    Params p;
    int run;  // heads of a CTA
    const __nv_bfloat16 *tiles;
    __nv_bfloat16 *y;
    Locals locals;
};

template <int K, bool LOCAL>
__global__ void __launch_bounds__(kThreads, 1)
scan_out_kernel(const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_c,
                const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y, const OutP q) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    const uint32_t sb = smem_u32(smem);
    const Params &p = q.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hg = p.H / p.G, runs = (hg + q.run - 1) / q.run, g = blockIdx.y / runs, h_first = (blockIdx.y % runs) * q.run;
    const int units = min(q.run, hg - h_first) * p.S, u_first = h_first * p.S;
    int n, local;
    if (!p.m.slot(blockIdx.x, kC, &n, &local)) {
        wait_for_previous();
        return;
    }
    const int t0 = p.m.begin(n) + local * kC, len = min(kC, p.m.end(n) - t0);
    const bool full_chunk = len == kC;
    const size_t seg_slot = LOCAL ? p.m.slot0(n, q.locals.seg_tokens) + (size_t)local * kC / q.locals.seg_tokens : 0;

    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kBarsAt);
    uint64_t *cb_full = bars, *s_full = bars + 1, *x_full = bars + 2, *h_full = bars + 5, *y_full = bars + 7, *p_ready = bars + 9,
             *y_done = bars + 11, *v_full = bars + 14, *v_free = bars + 16;
    // (as many of each as phases that can complete before a waiter has seen the first of them)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 18);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    if (tid == 0) {
        for (int i = 0; i < 9; ++i) mbar_init(bars + i, 1);
        for (int i = 9; i < 14; ++i) mbar_init(bars + i, kRowThreads);
        mbar_init(&v_full[0], 64), mbar_init(&v_full[1], 64);
        mbar_init(&v_free[0], kRowThreads), mbar_init(&v_free[1], kRowThreads);
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
    wait_for_previous();
    const uint32_t tmem = *tmem_slot;
    auto fail = [&]() {
        *abort_flag = 1;
        set_status(p.status, GDN_ERR_TIMEOUT);
    };

    if (warp >= 16) {
        reg_dec<kAuxRegs>();
        if (warp == 16) {  // products
            if (lane == 0) {
                bool ok = wait_bar(cb_full, 0, abort_flag);
                tc_fence_after();
                const uint32_t c = cols(sb + kCt);
                if (ok) {
                    constexpr uint32_t id = idesc_bf16(128, 128, false, false);
                    const uint32_t b = cols(sb + kP);
#pragma unroll
                    for (int k = 0; k < K / 16; ++k) mma<kTokenHi, kTokenHi>(tmem + kColS, c + cstep(k), b + cstep(k), id, k > 0);
                    mma_commit(s_full);
                }
                constexpr uint32_t id = idesc_bf16(128, 64, false, true);
                for (int i = 0; i < units && ok; ++i) {
                    const uint32_t d = tmem + kColY + (i & 1) * kYCols, h = state_rows(sb + kHt + (i & 1) * 16384);
                    if (i > 1) ok = wait_bar(&y_done[(i - 2) % 3], ((i - 2) / 3) & 1, abort_flag);  // its accumulators are read
                    ok = ok && wait_bar(&h_full[i & 1], (i >> 1) & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < K / 16; ++k) mma<kTokenHi, kStateRowsHi<K>>(d + 64, c + cstep(k), h + srstep(k), id, k > 0);
                    if (LOCAL) {
                        const uint32_t hs = state_rows(sb + kHs + (i & 1) * 16384);
#pragma unroll
                        for (int k = 0; k < K / 16; ++k) mma<kTokenHi, kStateRowsHi<K>>(d + 128, c + cstep(k), hs + srstep(k), id, k > 0);
                    }
                    ok = wait_bar(&x_full[i % 3], (i / 3) & 1, abort_flag) && wait_bar(&p_ready[i & 1], (i >> 1) & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t pm = cols(sb + kP + ((i >> p.sh) & 1) * 32768), x = rows(sb + kX + i % 3 * 16384);
#pragma unroll
                    for (int k = 0; k < 8; ++k) mma<kTokenHi, kTokenHi>(d, pm + cstep(k), x + rstep(k), id, k > 0);
                    mma_commit(&y_full[i & 1]);
                }
                if (!ok) fail();
            }
        } else if (warp == 17) {  // copies
            if (lane == 0) {
                auto load_x = [&](int i) {
                    const int u = u_first + i;
                    mbar_arrive_expect_tx(&x_full[i % 3], 16384);
                    tma_load_3d(smem + kX + i % 3 * 16384, &tm_x, &x_full[i % 3], p.col0(u), p.head(g, u), t0);
                };
                auto load_h = [&](int i) {
                    mbar_arrive_expect_tx(&h_full[i & 1], (LOCAL ? 2 : 1) * K * kPT * 2);
                    if (LOCAL)
                        bulk_load(smem + kHs + (i & 1) * 16384, q.locals.starts + ((seg_slot * p.G + g) * p.U + u_first + i) * (K * kPT), K * kPT * 2,
                                  &h_full[i & 1]);
                    bulk_load(smem + kHt + (i & 1) * 16384, q.tiles + (((size_t)blockIdx.x * p.G + g) * p.U + u_first + i) * (K * kPT),
                              K * kPT * 2, &h_full[i & 1]);
                };
                mbar_arrive_expect_tx(cb_full, 2 * (K / 64) * 16384);
                for (int j = 0; j < K / 64; ++j) {
                    tma_load_3d(smem + kCt + j * 16384, &tm_c, cb_full, 64 * j, g, t0);
                    tma_load_3d(smem + kP + j * 16384, &tm_b, cb_full, 64 * j, g, t0);
                }
                int xs = 0, hs = 0;  // loads issued
                while (xs < min(units, 3)) load_x(xs++);
                while (hs < min(units, 2)) load_h(hs++);
                bool ok = true;
                for (int i = 0; i < units && ok; ++i) {
                    ok = wait_bar(&y_full[i & 1], (i >> 1) & 1, abort_flag);
                    if (ok && hs < units) load_h(hs++);  // the products have read h
                    ok = ok && wait_bar(&y_done[i % 3], (i / 3) & 1, abort_flag);  // y stands in x's tile (or is written)
                    if (!ok) break;
                    if (full_chunk) {
                        const int u = u_first + i;
                        tma_store_3d(&tm_y, sb + kX + i % 3 * 16384, p.col0(u), p.head(g, u), t0);
                        bulk_commit();
                        bulk_wait_read<0>();
                    }
                    if (xs < units) load_x(xs++);
                }
                if (!ok) fail();
                // no copy outlives the CTA
                bool done = drain(cb_full, 0);
                for (int k = max(0, xs - 3); k < xs; ++k) done = drain(&x_full[k % 3], (k / 3) & 1) && done;
                for (int k = max(0, hs - 2); k < hs; ++k) done = drain(&h_full[k & 1], (k >> 1) & 1) && done;
                if (!done) fail();
                bulk_wait_all();
            }
        } else {  // warps 18, 19: the heads' column factors, a head ahead of the mask
            const int w2 = warp - 18;
            bool ok = true;
            for (int i = 0; i < units; i += p.S) {
                const int hb = (i >> p.sh) & 1, h = p.head(g, u_first + i);
                const float *gt = p.gates.at(blockIdx.x, p.H, h);
                const float4 tot = p.gates.totals(blockIdx.x, p.H, h);
                const float t[4] = {tot.x, tot.y, tot.z, tot.w};
                const float D = p.D ? p.D[h] : 0.f, f = LOCAL ? q.locals.before[(size_t)blockIdx.x * p.H + h] : 0.f;
                float gd[2], gf[2], gr[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int row = (w2 * 2 + k) * 32 + lane;
                    gd[k] = gt[row], gf[k] = gt[kC + row], gr[k] = gt[2 * kC + row];
                }
                // the factors of two heads before are read
                const int j = i >> p.sh;
                if (j >= 2) ok = __all_sync(0xffffffffu, ok && wait_bar(&v_free[hb], ((j - 2) >> 1) & 1, abort_flag));
                Vec &vec = reinterpret_cast<Vec *>(smem + kVec)[hb];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int wr = w2 * 2 + k, row = wr * 32 + lane;
                    vec.gl[row] = gf[k];
                    vec.col[wr][row] = gd[k];
                    float before, after, all;
                    around(tot, wr, &before, &after, &all);
                    vec.row[0][row] = ex2(before + gf[k]);
                    if (LOCAL) vec.row[1][row] = ex2(f + before + gf[k]);
                    vec.row[2][row] = ex2(gf[k]);
                    vec.row[3][row] = D;
                    float to = gr[k];
#pragma unroll
                    for (int w = 1; w < 4; ++w)
                        if (w > wr) {
                            vec.col[w][row] = ex2(to) * gd[k];
                            to += t[w];
                        }
                }
                mbar_arrive(&v_full[hb]);
            }
            if (!ok) fail();
        }
    } else {
        reg_inc<kRowRegs>();
        const int wr = warp & 3, qd = warp >> 2, row = wr * 32 + lane;  // row block, column quarter
        const bool live = row < len;
        const uint32_t lanes = (uint32_t)(wr * 32) << 16;
        bool ok = true;
        float e_next = 0.f, d_next = 0.f, s_next = 0.f;  // e^{gam_r}, D and e^{gam_r} f of the head masked last
        // unit i's P (where it begins a head), and leave for its product
        auto mask = [&](int i) {
            if ((i & (p.S - 1)) == 0) {
                const int hb = (i >> p.sh) & 1;
                Vec &vec = reinterpret_cast<Vec *>(smem + kVec)[hb];
                ok = __all_sync(0xffffffffu, ok && wait_bar(&v_full[hb], (i >> p.sh >> 1) & 1, abort_flag));
                e_next = vec.row[0][row], d_next = vec.row[3][row];
                if (LOCAL) s_next = vec.row[1][row];
                const float me = vec.gl[row], u_r = vec.row[2][row];
                const uint32_t at = sb + kP + hb * 32768;
                // this warp's columns: 8 qd .. of every block of 32, so that a row block's warps share its
                // diagonal block
                uint32_t v[4][8];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k <= wr && ok) tmem_ld8_nowait(tmem + lanes + kColS + 32 * k + 8 * qd, v[k]);
                tmem_landed(v);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t to = at + (k >> 1) * 16384 + piece(row, (k & 1) * 4 + qd);
                    if (k > wr) {  // right of the diagonal: zeros, once per buffer
                        if (i < 2 * p.S) st_shared_v4(to, 0u, 0u, 0u, 0u);
                        continue;
                    }
                    const float4 *vs = reinterpret_cast<const float4 *>(vec.col[wr] + 32 * k + 8 * qd);
                    const float4 ca = vs[0], cb = vs[1];
                    const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
                    float o[8];
                    if (k < wr) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] = u_r * c[j] * __uint_as_float(v[k][j]);
                    } else {
                        const float4 *gs = reinterpret_cast<const float4 *>(vec.gl + 32 * k + 8 * qd);
                        const float4 la = gs[0], lb = gs[1];
                        const float l[8] = {la.x, la.y, la.z, la.w, lb.x, lb.y, lb.z, lb.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t on = (uint32_t)((8 * qd + j - 1 - lane) >> 31);  // all ones where column <= row
                            o[j] = __uint_as_float(__float_as_uint(ex2(me - l[j]) * c[j] * __uint_as_float(v[k][j])) & on);
                        }
                    }
                    if (!full_chunk) {  // rows and columns of the next sequence
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] = live && 32 * k + 8 * qd + j < len ? o[j] : 0.f;
                    }
                    st_shared_v4(to, pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
                }
                mbar_arrive(&v_free[hb]);
            }
            if (!full_chunk) {  // x rows of the next sequence: no product may meet them
                ok = __all_sync(0xffffffffu, ok && wait_bar(&x_full[i % 3], (i / 3) & 1, abort_flag));
                if (ok && !live) {
                    const uint32_t xb = sb + kX + i % 3 * 16384;
                    st_shared_v4(xb + piece(row, 2 * qd), 0u, 0u, 0u, 0u);
                    st_shared_v4(xb + piece(row, 2 * qd + 1), 0u, 0u, 0u, 0u);
                }
            }
            fence_proxy_async();
            tc_fence_before();
            mbar_arrive(&p_ready[i & 1]);
        };
        ok = __all_sync(0xffffffffu, wait_bar(s_full, 0, abort_flag));
        tc_fence_after();
        mask(0);
        for (int i = 0; i < units; ++i) {
            const int u = u_first + i, h = p.head(g, u);
            const float e_r = e_next, D = d_next, s_r = s_next;
            if (i + 1 < units) mask(i + 1);
            const uint32_t xb = sb + kX + i % 3 * 16384;
            ok = __all_sync(0xffffffffu, ok && wait_bar(&y_full[i & 1], (i >> 1) & 1, abort_flag) &&
                                             wait_bar(&x_full[i % 3], (i / 3) & 1, abort_flag));
            tc_fence_after();
            if (ok) {
                const uint32_t d = tmem + lanes + kColY + (i & 1) * kYCols + 16 * qd;
                uint32_t a[16], b[16], hs[LOCAL ? 16 : 1];
                tmem_ld16_nowait(d, a);
                tmem_ld16_nowait(d + 64, b);
                if constexpr (LOCAL) tmem_ld16_nowait(d + 128, hs);
                uint4 xv[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) xv[j] = ld_shared_v4(xb + piece(row, 2 * qd + j));
                tmem_landed(a);
                tmem_landed(b);
                if constexpr (LOCAL) {
                    tmem_landed(hs);
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        a[c] = __float_as_uint(fmaf(s_r, __uint_as_float(hs[c]), __uint_as_float(a[c])));
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t w[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = 8 * j + 2 * k;
                        o[k] = pack_bf16(fmaf(D, bf_lo(w[k]), fmaf(e_r, __uint_as_float(b[c]), __uint_as_float(a[c]))),
                                         fmaf(D, bf_hi(w[k]), fmaf(e_r, __uint_as_float(b[c + 1]), __uint_as_float(a[c + 1]))));
                    }
                    if (full_chunk)
                        st_shared_v4(xb + piece(row, 2 * qd + j), o[0], o[1], o[2], o[3]);
                    else if (live)
                        *reinterpret_cast<uint4 *>(q.y + ((size_t)(t0 + row) * p.H + h) * p.P + p.col0(u) + qd * 16 + 8 * j) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            fence_proxy_async();
            tc_fence_before();
            mbar_arrive(&y_done[i % 3]);
        }
        if (!ok) fail();
    }
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int K, bool LOCAL>
cudaError_t run(const ScanArgs &a, const Gates &gates, const __nv_bfloat16 *tiles, const Locals &locals) {
    if (a.seq.total == 0) return cudaSuccess;
    CUtensorMap mb, mc, mx, my;
    if (!token_map(&mb, a.B, a.K, a.G, a.bs, a.seq.total) || !token_map(&mc, a.C, a.K, a.G, a.cs, a.seq.total) ||
        !token_map(&mx, a.x, a.P, a.H, a.xs, a.seq.total) || !token_map(&my, a.y, a.P, a.H, (long long)a.H * a.P, a.seq.total))
        return cudaErrorInvalidValue;
    OutP q{params(a, gates), 1, tiles, (__nv_bfloat16 *)a.y, locals};
    const int slots = a.seq.slots(kC), hg = a.H / a.G, sms = sm_count();
    // Heads per CTA: a CTA costs about four units' time before its first (its tiles, S); the fewest
    // waves times that length.
    double best = 1e30;
    for (int r = 1; r <= hg && r <= 64; ++r) {
        const long long ctas = (long long)slots * a.G * ((hg + r - 1) / r);
        const double cost = (double)((ctas + sms - 1) / sms) * (r * q.p.S + 4);
        if (cost < best) best = cost, q.run = r;
    }
    auto kernel = scan_out_kernel<K, LOCAL>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    TimedLaunch t("scan_out", a.stream);
    // early behind the state kernels (122 against 128 us for the prompt of 8192 tokens and 64 heads, 303 against
    // 312 for 32768 packed ones), not behind the chunks' recurrence, whose blocks it would crowd (281 against 278 us
    // for the training step of 2 x 4096 tokens)
    const dim3 grid(slots, a.G * ((hg + q.run - 1) / q.run));
    return launch(!a.products, kernel, grid, dim3(kThreads), kSmem, a.stream, mb, mc, mx, my, q);
}

}  // namespace

cudaError_t launch_out(const ScanArgs &a, const Gates &g, const __nv_bfloat16 *tiles_hi, const Locals &locals) {
    if (locals.seg_tokens) return a.K == 128 ? run<128, true>(a, g, tiles_hi, locals) : run<64, true>(a, g, tiles_hi, locals);
    return a.K == 128 ? run<128, false>(a, g, tiles_hi, locals) : run<64, false>(a, g, tiles_hi, locals);
}

}  // namespace scan_tc
}  // namespace gdn
