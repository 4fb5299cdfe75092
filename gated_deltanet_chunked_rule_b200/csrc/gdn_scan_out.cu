// gdn_scan_out.cu -- outputs of the tensor-core selective scan, chunk by chunk:
//
//   y_r = sum_s P_rs x_s + e^{gam_r} (C h)_r + D x_r,   P_rs = e^{gam_r - gam_s} delta_s (C B^T)_rs, s <= r
//
// from the chunk's entry state h (bf16, kept by the state pass). No chunk depends on another.
// A CTA takes one chunk and a run of units of one group: S = C B^T is formed once for all of
// them (tcgen05, 128 x 128 in tensor memory); per head its rows are read back, scaled and
// stored as the bf16 P tile over B's, which is no longer needed; per unit P X and C h are two
// products of 64 columns, joined by the epilogue and written through the x tile by one TMA
// store. Warps 0-3: a thread per row r. Warp 4: loads, products, stores. 97 KB of shared
// memory and 256 tensor-memory columns, so that two CTAs share an SM and hide each other's
// latencies.
//
// The mask's exponentials: warp w holds rows 32w ..; with gam relative to the row block's
// start (in fp64 until then: far into a chunk the running sum is large and differences of it
// are not), columns left of the block factor into e^{gam_r} e^{-gam_s} delta_s, both factors
// at most 1, from one vector per warp: two multiplications per element and no exponential. Only the
// 32 x 32 diagonal block takes one each. P and h are the two roundings to bf16 (2^-8 of a
// term each, on different terms) ahead of the output's own.
#include <algorithm>

#include "gdn_scan_tc.cuh"

namespace gdn {
namespace scan_tc {
namespace {

using namespace sm100;
using namespace gdn::warp;

constexpr int kThreads = 160;
constexpr int kCt = 0, kP = 32768, kX = 65536, kHt = 81920;  // C | B, then P | x, then y | h
constexpr int kVec = 98304;                                  // float v[4][128], gl[128], double wsum[2][4]
constexpr int kBarsAt = kVec + 2048 + 512 + 64;
constexpr int kSmem = kBarsAt + 128 + 1024;
static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
constexpr uint32_t kColS = 0, kColPX = 128, kColCh = 192;

struct OutP {
    Params p;
    int run;  // units of a CTA
    const __nv_bfloat16 *tiles;
    __nv_bfloat16 *y;
};

template <int K>
__global__ void __launch_bounds__(kThreads, 2)
scan_out_kernel(const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_c,
                const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y, const OutP q) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    const uint32_t sb = smem_u32(smem);
    const Params &p = q.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int runs = (p.U + q.run - 1) / q.run, g = blockIdx.y / runs, u_first = (blockIdx.y % runs) * q.run;
    const int units = min(q.run, p.U - u_first);
    int n, local;
    if (!p.m.slot(blockIdx.x, kC, &n, &local)) return;
    const int t0 = p.m.begin(n) + local * kC, len = min(kC, p.m.end(n) - t0);
    const bool full_chunk = len == kC;

    float(*vec)[kC] = reinterpret_cast<float(*)[kC]>(smem + kVec);
    float *gl = reinterpret_cast<float *>(smem + kVec + 2048);
    double *wsum = reinterpret_cast<double *>(smem + kVec + 2560);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kBarsAt);
    uint64_t *cb_full = bars, *s_full = bars + 1, *x_full = bars + 2, *h_full = bars + 3, *p_ready = bars + 4, *y_full = bars + 5,
             *y_done = bars + 6;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 7);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    if (tid == 0) {
        mbar_init(cb_full, 1), mbar_init(s_full, 1), mbar_init(x_full, 1), mbar_init(h_full, 1);
        mbar_init(p_ready, 128), mbar_init(y_full, 1), mbar_init(y_done, 128);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 4) {
        tmem_alloc(tmem_slot, 256);
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

    if (warp == 4) {
        if (lane == 0) {
            int xs = 0, hs = 0;  // loads issued
            auto load_x = [&](int i) {
                const int u = u_first + i;
                mbar_arrive_expect_tx(x_full, 16384);
                tma_load_3d(smem + kX, &tm_x, x_full, (u % p.S) * kPT, p.head(g, u), t0);
                ++xs;
            };
            auto load_h = [&](int i) {
                mbar_arrive_expect_tx(h_full, K * kPT * 2);
                bulk_load(smem + kHt, q.tiles + ((size_t)blockIdx.x * p.G * p.U + g * p.U + u_first + i) * K * kPT, K * kPT * 2, h_full);
                ++hs;
            };
            mbar_arrive_expect_tx(cb_full, 2 * (K / 64) * 16384);
            for (int j = 0; j < K / 64; ++j) {
                tma_load_3d(smem + kCt + j * 16384, &tm_c, cb_full, 64 * j, g, t0);
                tma_load_3d(smem + kP + j * 16384, &tm_b, cb_full, 64 * j, g, t0);
            }
            load_h(0);
            load_x(0);
            bool ok = wait_bar(cb_full, 0, abort_flag);
            tc_fence_after();
            if (ok) {
                const uint32_t id = idesc_bf16(128, 128, false, false);
#pragma unroll
                for (int k = 0; k < K / 16; ++k) mma_bf16(tmem + kColS, by_cols(sb + kCt, k), by_cols(sb + kP, k), id, k > 0);
                mma_commit(s_full);
            }
            const uint32_t id = idesc_bf16(128, 64, false, true);
            for (int i = 0; i < units && ok; ++i) {
                ok = wait_bar(h_full, i & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < K / 16; ++k)
                    mma_bf16(tmem + kColCh, by_cols(sb + kCt, k), state_by_rows<K>(sb + kHt, k), id, k > 0);
                ok = wait_bar(x_full, i & 1, abort_flag) && wait_bar(p_ready, i & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_bf16(tmem + kColPX, by_cols(sb + kP, k), by_rows(sb + kX, k), id, k > 0);
                mma_commit(y_full);
                ok = wait_bar(y_full, i & 1, abort_flag);
                if (ok && i + 1 < units) load_h(i + 1);  // the products have read h
                ok = ok && wait_bar(y_done, i & 1, abort_flag);  // y stands in x's tile (or is written)
                if (!ok) break;
                tc_fence_after();
                if (full_chunk) {
                    const int u = u_first + i;
                    tma_store_3d(&tm_y, sb + kX, (u % p.S) * kPT, p.head(g, u), t0);
                    bulk_commit();
                    bulk_wait_read<0>();
                }
                if (i + 1 < units) load_x(i + 1);
            }
            if (!ok) fail();
            // no copy outlives the CTA
            bool done = drain(cb_full, 0);
            done = drain(x_full, (xs - 1) & 1) && done;
            done = drain(h_full, (hs - 1) & 1) && done;
            if (!done) fail();
            bulk_wait_all();
        }
    } else {
        const int row = tid;
        const bool live = row < len;
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        int done_head = -1;
        float u_r = 0.f, e_r = 0.f, D = 0.f;
        bool ok = true;
        auto fetch = [&](int u) { return live ? p.raw_dt(t0 + row, p.head(g, u)) : 0.f; };
        float raw = fetch(u_first);
        for (int i = 0; i < units; ++i) {
            const int u = u_first + i, h = p.head(g, u);
            if (h != done_head) {  // another head: its gates and its P
                const float delta = live ? p.delta(raw) : 0.f;
                double x = (double)delta * p.A[h];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                double *ws = wsum + (i & 1) * 4;
                if (lane == 31) ws[warp] = x;
                named_sync<128>(1);
                double base = 0.0;  // at the start of this warp's rows
                for (int k = 0; k < warp; ++k) base += ws[k];
                const float rel = (float)x;  // gam relative to it
                gl[row] = rel;
                u_r = expf(rel);
                e_r = expf((float)(base + x));
                // this token as a column of the later row blocks: e^{(their start) - gam_s} delta_s
                vec[warp][row] = delta;
                double to = ws[warp] - x;
                for (int w = warp + 1; w < 4; ++w) {
                    vec[w][row] = expf((float)to) * delta;
                    to += ws[w];
                }
                D = p.D ? p.D[h] : 0.f;
                named_sync<128>(1);
                ok = __all_sync(0xffffffffu, ok && (i > 0 || wait_bar(s_full, 0, abort_flag)));
                tc_fence_after();
                for (int blk = 0; blk < 4 && ok; ++blk) {
                    if (blk > warp) {  // right of the diagonal: zeros, once
                        if (done_head < 0)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                st_shared_v4(sb + kP + (blk >> 1) * 16384 + piece(row, (blk & 1) * 4 + j), 0u, 0u, 0u, 0u);
                        continue;
                    }
                    float v[32];
                    tmem_ld32(tmem + lanes + kColS + 32 * blk, v);
                    const float *vs = vec[warp] + 32 * blk, *gs = gl + 32 * blk;
                    if (blk < warp) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = u_r * vs[k] * v[k];
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = k <= lane ? __expf(rel - gs[k]) * vs[k] * v[k] : 0.f;
                    }
                    if (!full_chunk) {  // rows and columns of the next sequence
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = live && 32 * blk + k < len ? v[k] : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        st_shared_v4(sb + kP + (blk >> 1) * 16384 + piece(row, (blk & 1) * 4 + j), pack_bf16(v[8 * j], v[8 * j + 1]),
                                     pack_bf16(v[8 * j + 2], v[8 * j + 3]), pack_bf16(v[8 * j + 4], v[8 * j + 5]),
                                     pack_bf16(v[8 * j + 6], v[8 * j + 7]));
                }
                done_head = h;
            }
            if (i + 1 < units && p.head(g, u + 1) != h) raw = fetch(u + 1);
            if (!full_chunk) {  // x rows of the next sequence: no product may meet them
                ok = __all_sync(0xffffffffu, ok && wait_bar(x_full, i & 1, abort_flag));
                if (ok && !live)
#pragma unroll
                    for (int j = 0; j < 8; ++j) st_shared_v4(sb + kX + piece(row, j), 0u, 0u, 0u, 0u);
            }
            fence_proxy_async();
            tc_fence_before();
            mbar_arrive(p_ready);
            ok = __all_sync(0xffffffffu, ok && wait_bar(y_full, i & 1, abort_flag));
            tc_fence_after();
            for (int half = 0; half < 2 && ok; ++half) {
                float a[32], b[32];
                tmem_ld32(tmem + lanes + kColPX + 32 * half, a);
                tmem_ld32(tmem + lanes + kColCh + 32 * half, b);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t at = sb + kX + piece(row, half * 4 + j);
                    const uint4 xv = ld_shared_v4(at);
                    const uint32_t w[4] = {xv.x, xv.y, xv.z, xv.w};
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = 8 * j + 2 * k;
                        o[k] = pack_bf16(fmaf(D, bf_lo(w[k]), fmaf(e_r, b[c], a[c])), fmaf(D, bf_hi(w[k]), fmaf(e_r, b[c + 1], a[c + 1])));
                    }
                    if (full_chunk)
                        st_shared_v4(at, o[0], o[1], o[2], o[3]);
                    else if (live)
                        *reinterpret_cast<uint4 *>(q.y + ((size_t)(t0 + row) * p.H + h) * p.P + (u % p.S) * kPT + half * 32 + 8 * j) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            fence_proxy_async();
            tc_fence_before();
            mbar_arrive(y_done);
        }
        if (!ok) fail();
    }
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

template <int K>
cudaError_t run(const ScanArgs &a, const __nv_bfloat16 *tiles) {
    if (a.seq.total == 0) return cudaSuccess;
    CUtensorMap mb, mc, mx, my;
    if (!token_map(&mb, a.B, a.K, a.G, a.bs, a.seq.total) || !token_map(&mc, a.C, a.K, a.G, a.cs, a.seq.total) ||
        !token_map(&mx, a.x, a.P, a.H, a.xs, a.seq.total) || !token_map(&my, a.y, a.P, a.H, (long long)a.H * a.P, a.seq.total))
        return cudaErrorInvalidValue;
    OutP q{params(a), 1, tiles, (__nv_bfloat16 *)a.y};
    const int slots = a.seq.slots(kC), U = q.p.U;
    // Units per CTA: a CTA costs about three units' time before its first (its tiles, S) and two run
    // on an SM; the fewest waves times that length.
    double best = 1e30;
    for (int r = 1; r <= U && r <= 32; ++r) {
        const long long ctas = (long long)slots * a.G * ((U + r - 1) / r);
        const double cost = (double)((ctas + 2 * sm_count() - 1) / (2 * sm_count())) * (r + 3);
        if (cost < best) best = cost, q.run = r;
    }
    auto kernel = scan_out_kernel<K>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    TimedLaunch t("scan_out", a.stream);
    kernel<<<dim3(slots, a.G * ((U + q.run - 1) / q.run)), kThreads, kSmem, a.stream>>>(mb, mc, mx, my, q);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_out(const ScanArgs &a, const __nv_bfloat16 *tiles_hi) {
    return a.K == 128 ? run<128>(a, tiles_hi) : run<64>(a, tiles_hi);
}

}  // namespace scan_tc
}  // namespace gdn
