// gdn_scan_state.cu -- state passes of the tensor-core selective scan: the state at the
// start of every chunk (or, backwards, its gradient at the end), and the last one.
//
//   h' = e^{gam_C} h + B^T Xs,   Xs = diag(delta e^{gam_C - gam}) X        (forward)
//   g  = e^{gam_C} g' + C^T Xs,  Xs = diag(e^{gam}) dY                     (reverse)
//
// The product does not depend on the state, so only one multiply-add per element is
// sequential. A CTA walks the chunks of one segment of a sequence with two units (128
// accumulator columns) of a group: warps 0-7 hold unit 0's state in fp32 registers (a thread
// per row of K and 32 columns), warps 8-15 unit 1's, warp 16 loads the tiles by TMA (two
// stages), warp 17 issues the products. Bound by the sixteen warps' conversions (about 430
// instructions per chunk each), the 24 products of 64 cycles and the 400 KB that both move
// through shared memory (1.6 us of a chunk's 2.7); with eight warps of 64 columns each the
// latencies showed and a chunk took 3.6 us instead. 8192 tokens, 64 heads: 47 us in one pass.
//
// The fp32 state keeps fp32 precision although the tensor core takes bf16: B is bf16 as it
// is, and Xs is cut into three bf16 terms that hold its 24 bits exactly (8 + 8 + 8, by
// truncation); two terms left 2.5e-6 in the final state. (Splitting x times the scale's bf16 terms
// exactly by packed bf16 multiply-adds takes half the instructions, and half as long again.) The
// second and third term are
// multiplied first, so that their buffer is free for the next chunk while the first one's
// product still runs, and the accumulator has two buffers.
//
// A sequence is cut into segments where units and sequences alone would not fill the SMs. Then,
// where every chunk's product fits the L2 cache in fp32, the segments only write those products and
// a second kernel runs the recurrence over the chunks element by element; it reads what it needs
// from L2. Beyond that size the products would go through memory twice, and instead a first pass
// takes every segment from a zero state, one small kernel composes the segments' starts (their
// operator is one scalar decay), and a second pass walks them again. 2 x 4096 tokens, 16 heads of
// 128 (67 MB of products): 26 + 22 us against 25 + 10 + 29 (with two parts kept of each state; three
// now: 26 + 27). A forward that keeps nothing needs no second
// pass: the tiles of the first one, the segments' starts and one factor per chunk are enough for
// the outputs (8192 tokens, 64 heads: 40 us less of 162).
#include <algorithm>

#include "gdn_scan_tc.cuh"

namespace gdn {
namespace scan_tc {
namespace {

using namespace sm100;
using namespace gdn::warp;

// Gates of every chunk slot: a warp per head.
__global__ void __launch_bounds__(256) scan_gates_tc_kernel(Params p) {
    let_next_start();
    const int lane = threadIdx.x & 31, h = blockIdx.y * 8 + (threadIdx.x >> 5);
    if (blockIdx.x == 0 && blockIdx.y == 0) check_cu(p.m, p.status, threadIdx.x, blockDim.x);
    int n, local;
    if (h >= p.H || !p.m.slot(blockIdx.x, kC, &n, &local)) return;
    const int t0 = p.m.begin(n) + local * kC, len = min(kC, p.m.end(n) - t0);
    const float A2 = p.A[h] * 1.44269504f;
    float raw[4], tot[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) raw[b] = b * 32 + lane < len ? p.raw_dt(t0 + b * 32 + lane, h) : 0.f;
    float *v = p.gates.v + ((size_t)blockIdx.x * p.H + h) * (3 * kC) + lane;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        // log1p(exp(v)), or v itself above 20 (where they agree to fp32 precision)
        float d = p.softplus ? (raw[b] > 20.f ? raw[b] : log1pf(expf(raw[b]))) : raw[b];
        const bool live = b * 32 + lane < len;
        if (!live) d = 0.f;
        // 2^-256 and below are 0 with or without the up to 2^116 that other tokens may grow by, but a larger
        // sum would round the tokens behind it in its block by 2^-24 of itself (a NaN stays one)
        float g = live ? d * A2 : 0.f;
        g = g < -256.f ? -256.f : g;
        float f = g, r = g;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, f, o), y = __shfl_down_sync(0xffffffffu, r, o);
            if (lane >= o) f += x;
            if (lane + o < 32) r += y;
        }
        const float after = __shfl_down_sync(0xffffffffu, r, 1);
        tot[b] = __shfl_sync(0xffffffffu, f, 31);
        v[b * 32] = d;
        v[kC + b * 32] = f;
        v[2 * kC + b * 32] = lane < 31 ? after : 0.f;
    }
    if (lane == 0)
        *reinterpret_cast<float4 *>(p.gates.tot + ((size_t)blockIdx.x * p.H + h) * 4) = make_float4(tot[0], tot[1], tot[2], tot[3]);
}

constexpr int kRowThreads = 512;
constexpr int kThreads = kRowThreads + 128;
// Registers: 640 threads are launched with 96 each; the row warps spilled there, and a spill costs
// an L2 access beside 200 KB of shared memory.
constexpr int kRowRegs = 104, kAuxRegs = 64;
static_assert(kRowThreads * kRowRegs + 128 * kAuxRegs <= kThreads * 96, "register split");
constexpr int kHalf = kPT / 2;          // columns of a thread
constexpr int kStage = 65536;           // one stage: B (or C) tile 32 KB, x (or dY) tiles 2 x 16 KB
constexpr int kMid = 2 * kStage;        // second and third terms: 2 x (2 x 16 KB)
constexpr int kSmall = kMid + 65536;    // barriers
constexpr int kSmem = kSmall + 256 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");

// The states; segment ends from zero; every chunk's product; states within each segment (the first
// one's from the start state), its end and the log decay before each chunk.
enum Pass { kWalk, kEnds, kProducts, kLocal };

struct StateP {
    Params p;
    int seg_tokens;   // tokens of a segment
    Pass pass;
    const float *first;
    float *last, *seg, *seg_gam, *before;
    Tiles tiles;
};

// A chunk's product in fp32: [column / 4][row][4], so that a lane-per-row store is contiguous.
__device__ __forceinline__ size_t product_at(size_t slot, size_t units, size_t unit, int K, int quad, int row) {
    return (slot * units + unit) * (size_t)(K * kPT) + ((size_t)quad * K + row) * 4;
}

template <int K, bool REVERSE>
__global__ void __launch_bounds__(kThreads, 1)
scan_state_kernel(const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_x, const StateP q) {
    let_next_start();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    const uint32_t sb = smem_u32(smem);
    const Params &p = q.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pairs = (p.U + 1) / 2, g = blockIdx.y / pairs, u0 = (blockIdx.y % pairs) * 2;

    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kSmall);
    uint64_t *full = bars, *empty = bars + 2, *dfull = bars + 4, *xs_ready = bars + 6, *ml_free = bars + 7;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    // the backward's first kernel where the forward's gates are kept; warps 18 and 19 have no other work
    if (REVERSE && blockIdx.x == 0 && blockIdx.y == 0 && warp >= 18) check_cu(p.m, p.status, tid - 18 * 32, 64);
    int n, local;
    const bool used = p.m.slot(blockIdx.x, q.seg_tokens, &n, &local);
    const int s_begin = p.m.begin(n), s_len = p.m.end(n) - s_begin;
    // (row warps) this thread's unit of the pair, row and first column
    const int unit_of = warp >> 3, wr = warp & 3, c0 = ((warp >> 2) & 1) * kHalf, row = wr * 32 + lane;
    const int u = u0 + unit_of;
    const bool mine = tid < kRowThreads && u < p.U, real = mine && row < K;
    const int h = mine ? p.head(g, u) : 0;
    const size_t user = (((size_t)n * p.H + h) * K + row) * p.P + (mine ? p.col0(u) : 0) + c0;  // in the user's states
    if (!used) {  // an empty sequence keeps its state
        wait_for_previous();
        if (local == 0 && s_len == 0 && (q.pass == kWalk || q.pass == kLocal) && q.last && real)
            for (int i = 0; i < kHalf; ++i) q.last[user + i] = q.first ? q.first[user + i] : 0.f;
        return;
    }
    const int seg_begin = s_begin + local * q.seg_tokens, seg_len = min(q.seg_tokens, s_begin + s_len - seg_begin);
    const bool at_first = REVERSE ? seg_begin + seg_len == s_begin + s_len : local == 0;
    const bool at_last = REVERSE ? local == 0 : seg_begin + seg_len == s_begin + s_len;
    if (q.pass == kEnds && at_last) {  // nothing follows it
        wait_for_previous();
        return;
    }
    const int chunks = (seg_len + kC - 1) / kC;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1), mbar_init(&dfull[i], 1);
        mbar_init(xs_ready, kRowThreads);
        mbar_init(ml_free, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 16) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_for_previous();
    const uint32_t tmem = *tmem_slot;
    auto chunk_at = [&](int i) { return REVERSE ? chunks - 1 - i : i; };
    auto fail = [&]() {
        *abort_flag = 1;
        set_status(p.status, GDN_ERR_TIMEOUT);
    };

    if (warp >= 16) {  // (the register split stands inside the roles: what follows a join keeps the smaller share)
        reg_dec<kAuxRegs>();
        if (warp == 16) {
            if (lane == 0) {
                const int nx = u0 + 1 < p.U ? 2 : 1;
                bool ok = true;
                int i = 0;
                for (; i < chunks && ok; ++i) {
                    const int st = i & 1, t0 = seg_begin + chunk_at(i) * kC;
                    if (i >= 2) ok = wait_bar(&empty[st], ((i >> 1) - 1) & 1, abort_flag);
                    if (!ok) break;
                    uint8_t *dst = smem + st * kStage;
                    mbar_arrive_expect_tx(&full[st], (K / 64 + nx) * 16384);
                    for (int j = 0; j < K / 64; ++j) tma_load_3d(dst + j * 16384, &tm_b, &full[st], 64 * j, g, t0);
                    for (int j = 0; j < nx; ++j)
                        tma_load_3d(dst + 32768 + j * 16384, &tm_x, &full[st], p.col0(u0 + j), p.head(g, u0 + j), t0);
                }
                if (!ok) fail();
                // no copy outlives the CTA: the last two stages issued are waited for
                for (int k = max(0, i - 2); k < i; ++k)
                    if (!drain(&full[k & 1], (k >> 1) & 1)) fail();
            }
        } else if (warp == 17) {
            if (lane == 0) {
                const uint32_t id = idesc_bf16(128, 128, true, true);
                bool ok = true;
                for (int i = 0; i < chunks && ok; ++i) {
                    ok = wait_bar(xs_ready, i & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t st = sb + (i & 1) * kStage, d = tmem + (i & 1) * 128;
                    const uint32_t a = rows(st), hi = rows(st + 32768), md = rows(sb + kMid), lo = rows(sb + kMid + 32768);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        mma<kTokenHi, kTokenHi>(d, a + rstep(k), md + rstep(k), id, k > 0);
                        mma<kTokenHi, kTokenHi>(d, a + rstep(k), lo + rstep(k), id, true);
                    }
                    mma_commit(ml_free);
#pragma unroll
                    for (int k = 0; k < 8; ++k) mma<kTokenHi, kTokenHi>(d, a + rstep(k), hi + rstep(k), id, true);
                    mma_commit(&dfull[i & 1]);
                    mma_commit(&empty[i & 1]);
                }
                if (!ok) fail();
            }
        }
    } else {
        reg_inc<kRowRegs>();
        float st[kHalf];  // this thread's part of the state
        const size_t units = (size_t)p.G * p.U, unit = (size_t)g * p.U + u;
        float *const seg = q.seg + (((size_t)blockIdx.x * units + unit) * K + row) * kPT + c0;
        const bool own = q.pass == kWalk || q.pass == kLocal;
        const float *src = !own ? nullptr : at_first ? (q.first ? q.first + user : nullptr) : q.pass == kWalk ? seg : nullptr;
        if (real && src) {
#pragma unroll
            for (int i = 0; i < kHalf; i += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(src + i);
                st[i] = v.x, st[i + 1] = v.y, st[i + 2] = v.z, st[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kHalf; ++i) st[i] = 0.f;
        }
        const size_t slot0 = (size_t)p.m.slot0(n, kC) + (seg_begin - s_begin) / kC;
        const bool keeps = q.tiles.hi && real && own;
        const bool notes = real && row == 0 && c0 == 0 && (u & (p.S - 1)) == 0;  // (one thread per head)
        auto keep = [&](int i) {  // the state on entry to chunk i of the walk
            if (!keeps) return;
            const size_t at = ((slot0 + chunk_at(i)) * units + unit) * (K * kPT) + (size_t)(c0 / 8) * K * 8 + row * 8;
#pragma unroll
            for (int b = 0; b < kHalf / 8; ++b) store_parts(q.tiles, at + (size_t)b * K * 8, st + 8 * b);
        };
        keep(0);
        // this token's gates of chunk i: what Xs is scaled by, and the chunk's whole decay (log2)
        float g_delta = 0.f, g_sum = 0.f;
        float4 g_tot = make_float4(0.f, 0.f, 0.f, 0.f);
        auto fetch = [&](int i) {
            if (!mine || i >= chunks) return;
            const size_t slot = slot0 + chunk_at(i);
            const float *gt = p.gates.at(slot, p.H, h) + row;
            if (!REVERSE) g_delta = gt[0];
            g_sum = REVERSE ? gt[kC] : gt[2 * kC];
            g_tot = p.gates.totals(slot, p.H, h);
        };
        fetch(0);
        float gam_sum = 0.f, decay_prev = 0.f;
        bool ok = true;
        for (int i = 0; i <= chunks; ++i) {
            float decay = 0.f;
            if (i < chunks) {
                const int len = min(kC, seg_len - chunk_at(i) * kC);
                const bool live = mine && row < len;
                float before, after, all;
                around(g_tot, wr, &before, &after, &all);
                const float scale = REVERSE ? ex2(before + g_sum) : g_delta * ex2(after + g_sum);
                decay = ex2(all);
                if (q.pass == kLocal && notes) q.before[(slot0 + chunk_at(i)) * p.H + h] = gam_sum;
                gam_sum += all;
                fetch(i + 1);
                // a wait that expired: no more work and no more waits, but every barrier of the
                // loop is still met, so that it ends
                ok = ok && wait_bar(&full[i & 1], (i >> 1) & 1, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                const uint32_t stage = sb + (i & 1) * kStage;
                const uint32_t xt = stage + 32768 + unit_of * 16384, mid = sb + kMid + unit_of * 16384;
                uint4 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = ok && live ? ld_shared_v4(xt + piece(row, c0 / 8 + j)) : make_uint4(0u, 0u, 0u, 0u);
                if (i > 0) ok = __all_sync(0xffffffffu, ok && wait_bar(ml_free, (i - 1) & 1, abort_flag));
                if (ok) {
                    if (row >= len && unit_of == 0) {  // rows of the next sequence: no product may meet them
#pragma unroll
                        for (int j = 0; j < K / 16; ++j) {
                            const int k = (c0 ? K / 16 : 0) + j;
                            st_shared_v4(stage + (k >> 3) * 16384 + piece(row, k & 7), 0u, 0u, 0u, 0u);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                        uint32_t hi[4], md[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            // a dead row's value is +0, its scale finite: all terms 0
                            const float a0 = bf_lo(w[k]) * scale, a1 = bf_hi(w[k]) * scale;
                            hi[k] = __byte_perm(__float_as_uint(a0), __float_as_uint(a1), 0x7632);
                            const float b0 = a0 - bf_hi(__float_as_uint(a0)), b1 = a1 - bf_hi(__float_as_uint(a1));
                            md[k] = __byte_perm(__float_as_uint(b0), __float_as_uint(b1), 0x7632);
                            const float d0 = b0 - bf_hi(__float_as_uint(b0)), d1 = b1 - bf_hi(__float_as_uint(b1));
                            lo[k] = __byte_perm(__float_as_uint(d0), __float_as_uint(d1), 0x7632);
                        }
                        const uint32_t at = piece(row, c0 / 8 + j);
                        st_shared_v4(xt + at, hi[0], hi[1], hi[2], hi[3]);
                        st_shared_v4(mid + at, md[0], md[1], md[2], md[3]);
                        st_shared_v4(mid + 32768 + at, lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                fence_proxy_async();
                tc_fence_before();
                mbar_arrive(xs_ready);
            }
            if (i > 0) {
                ok = __all_sync(0xffffffffu, ok && wait_bar(&dfull[(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag));
                tc_fence_after();
                if (ok) {
                    float v[kHalf];
                    tmem_ld32(tmem + ((uint32_t)(wr * 32) << 16) + ((i - 1) & 1) * 128 + unit_of * kPT + c0, v);
                    if (q.pass == kProducts) {
                        if (real) {
                            float *out = q.seg + product_at(slot0 + chunk_at(i - 1), units, unit, K, c0 / 4, row);
#pragma unroll
                            for (int k = 0; k < kHalf; k += 4)
                                *reinterpret_cast<float4 *>(out + (size_t)k * K) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < kHalf; ++k) st[k] = fmaf(decay_prev, st[k], v[k]);
                        if (i < chunks) keep(i);
                    }
                }
            }
            decay_prev = decay;
        }
        if (!ok) fail();
        if (real && ok && q.pass != kProducts) {
            float *out = q.pass == kEnds || q.pass == kLocal ? seg : at_last && q.last ? q.last + user : nullptr;
            if (out)
#pragma unroll
                for (int i = 0; i < kHalf; i += 4)
                    *reinterpret_cast<float4 *>(out + i) = make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]);
            if ((q.pass == kEnds || q.pass == kLocal) && notes) q.seg_gam[(size_t)blockIdx.x * p.H + h] = gam_sum;
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// Start states of the segments, in place of their ends: start' = 2^gam start + end. A
// thread per four state elements walks a sequence's segments.
template <int K, bool REVERSE>
__global__ void __launch_bounds__(256)
scan_compose_kernel(Params p, int seg_tokens, const float *__restrict__ first, float *__restrict__ seg, const float *__restrict__ seg_gam) {
    const int n = blockIdx.x, unit = blockIdx.y, e = (blockIdx.z * 256 + threadIdx.x) * 4;  // e = row * 64 + column
    const int len = p.m.end(n) - p.m.begin(n), segs = (len + seg_tokens - 1) / seg_tokens;
    if (segs < 2) return;
    const int h = p.head(unit / p.U, unit % p.U), col = p.col0(unit % p.U) + e % kPT;
    const size_t slot0 = p.m.slot0(n, seg_tokens), units = (size_t)p.G * p.U;
    float4 cur = make_float4(0.f, 0.f, 0.f, 0.f);
    if (first) cur = *reinterpret_cast<const float4 *>(first + (((size_t)n * p.H + h) * K + e / kPT) * p.P + col);
    auto slot = [&](int i) { return slot0 + (REVERSE ? segs - 1 - i : i); };
    auto at = [&](int i) { return reinterpret_cast<float4 *>(seg + (slot(i) * units + unit) * (K * kPT) + e); };
    float4 end = *at(0);
    float gam = seg_gam[slot(0) * p.H + h];
    for (int i = 0; i + 1 < segs; ++i) {
        const float4 v = end;
        const float d = ex2(gam);
        if (i + 2 < segs) end = *at(i + 1), gam = seg_gam[slot(i + 1) * p.H + h];
        cur = make_float4(fmaf(d, cur.x, v.x), fmaf(d, cur.y, v.y), fmaf(d, cur.z, v.z), fmaf(d, cur.w, v.w));
        *at(i + 1) = cur;  // the first segment starts from `first` itself
    }
}

// After a pass within the segments: each segment's start as a bf16 tile (zero for a sequence's
// first, whose chunks have it in them), and the last state. A thread per row and eight columns.
template <int K>
__global__ void __launch_bounds__(256)
scan_starts_kernel(Params p, int seg_tokens, const float *__restrict__ seg, const float *__restrict__ seg_gam,
                   __nv_bfloat16 *__restrict__ starts, float *__restrict__ last) {
    let_next_start();
    const int n = blockIdx.x, unit = blockIdx.y, e = blockIdx.z * 256 + threadIdx.x, row = e % K, c8 = e / K;
    const int len = p.m.end(n) - p.m.begin(n), segs = (len + seg_tokens - 1) / seg_tokens;
    if (segs == 0) return;
    const int h = p.head(unit / p.U, unit % p.U);
    const size_t slot0 = p.m.slot0(n, seg_tokens), units = (size_t)p.G * p.U;
    float st[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) st[k] = 0.f;
    auto end_at = [&](int i) { return seg + (((slot0 + i) * units + unit) * K + row) * kPT + c8 * 8; };
    float4 a = *reinterpret_cast<const float4 *>(end_at(0)), b = *reinterpret_cast<const float4 *>(end_at(0) + 4);
    float gam = seg_gam[slot0 * p.H + h];
    for (int i = 0; i < segs; ++i) {
        uint32_t hi[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) hi[k] = pack_bf16(st[2 * k], st[2 * k + 1]);
        *reinterpret_cast<uint4 *>(starts + ((slot0 + i) * units + unit) * (K * kPT) + ((size_t)c8 * K + row) * 8) =
            make_uint4(hi[0], hi[1], hi[2], hi[3]);
        const float d = ex2(gam), v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (i + 1 < segs) {
            a = *reinterpret_cast<const float4 *>(end_at(i + 1)), b = *reinterpret_cast<const float4 *>(end_at(i + 1) + 4);
            gam = seg_gam[(slot0 + i + 1) * p.H + h];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) st[k] = i ? fmaf(d, st[k], v[k]) : v[k];
    }
    if (last) {
        float *out = last + (((size_t)n * p.H + h) * K + row) * p.P + p.col0(unit % p.U) + c8 * 8;
        *reinterpret_cast<float4 *>(out) = make_float4(st[0], st[1], st[2], st[3]);
        *reinterpret_cast<float4 *>(out + 4) = make_float4(st[4], st[5], st[6], st[7]);
    }
}

// The recurrence over a sequence's chunks from their products: tiles of every chunk's entry state
// and the last state. A thread per row and eight columns, four chunks' loads ahead.
template <int K, bool REVERSE>
__global__ void __launch_bounds__(256)
scan_chunks_kernel(Params p, const float *__restrict__ products, const float *__restrict__ first, float *__restrict__ last, Tiles tiles) {
    constexpr int kAhead = 4;
    const int n = blockIdx.x, unit = blockIdx.y, e = blockIdx.z * 256 + threadIdx.x, row = e % K, c8 = e / K;
    const int len = p.m.end(n) - p.m.begin(n), chunks = (len + kC - 1) / kC;
    const int h = p.head(unit / p.U, unit % p.U);
    const size_t slot0 = p.m.slot0(n, kC), units = (size_t)p.G * p.U;
    const size_t user = (((size_t)n * p.H + h) * K + row) * p.P + p.col0(unit % p.U) + c8 * 8;
    auto slot = [&](int i) { return slot0 + (REVERSE ? chunks - 1 - i : i); };
    float st[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) st[k] = first ? first[user + k] : 0.f;
    float4 a[kAhead], b[kAhead], t[kAhead];
    auto fetch = [&](int i, int at) {
        if (i >= chunks) return;
        const float *src = products + product_at(slot(i), units, unit, K, 2 * c8, row);
        a[at] = *reinterpret_cast<const float4 *>(src);
        b[at] = *reinterpret_cast<const float4 *>(src + 4 * K);
        t[at] = p.gates.totals(slot(i), p.H, h);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i, i);
    for (int i0 = 0; i0 < chunks; i0 += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j;
            if (i >= chunks) break;
            store_parts(tiles, (slot(i) * units + unit) * (K * kPT) + ((size_t)c8 * K + row) * 8, st);
            const float d = ex2((t[j].x + t[j].y) + (t[j].z + t[j].w));
            const float v[8] = {a[j].x, a[j].y, a[j].z, a[j].w, b[j].x, b[j].y, b[j].z, b[j].w};
#pragma unroll
            for (int k = 0; k < 8; ++k) st[k] = fmaf(d, st[k], v[k]);
            fetch(i + kAhead, j);
        }
    }
    if (last) {
        *reinterpret_cast<float4 *>(last + user) = make_float4(st[0], st[1], st[2], st[3]);
        *reinterpret_cast<float4 *>(last + user + 4) = make_float4(st[4], st[5], st[6], st[7]);
    }
}

template <int K, bool REVERSE>
cudaError_t run(const StateArgs &s) {
    const ScanArgs &a = *s.a;
    CUtensorMap mb, mx;
    const void *b = s.reverse ? a.C : a.B, *x = s.reverse ? a.dy : a.x;
    if (a.seq.total > 0 && (!token_map(&mb, b, a.K, a.G, s.reverse ? a.cs : a.bs, a.seq.total) ||
                            !token_map(&mx, x, a.P, a.H, s.reverse ? (long long)a.H * a.P : a.xs, a.seq.total)))
        return cudaErrorInvalidValue;
    StateP q{};
    q.p = params(a, s.gates);
    q.first = s.first, q.last = s.last, q.seg = s.seg, q.seg_gam = s.seg_gam, q.tiles = s.tiles;
    const bool split = s.chunks_per_seg > 0;
    // without a split a segment is longer than any sequence
    q.seg_tokens = split ? s.chunks_per_seg * kC : std::max(kC, (a.seq.cu ? a.seq.total : a.seq.T) / kC * kC + kC);
    const int slots = a.seq.total == 0 ? a.seq.N : a.seq.slots(q.seg_tokens);
    const int pairs = (q.p.U + 1) / 2;
    auto kernel = scan_state_kernel<K, REVERSE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid(slots, a.G * pairs);
    bool early = s.after_gates && !s.products;
    auto pass = [&](const char *name, Pass which) {
        TimedLaunch t(name, a.stream);
        q.pass = which;
        const cudaError_t rc = launch(early, kernel, grid, dim3(kThreads), kSmem, a.stream, mb, mx, q);
        early = false;
        return rc;
    };
    if (s.products) {
        if ((e = pass(REVERSE ? "scan_products_bwd" : "scan_products", kProducts)) != cudaSuccess) return e;
        TimedLaunch t(REVERSE ? "scan_chunks_bwd" : "scan_chunks", a.stream);
        scan_chunks_kernel<K, REVERSE><<<dim3(a.seq.N, a.G * q.p.U, K * kPT / 2048), 256, 0, a.stream>>>(q.p, s.seg, s.first, s.last, s.tiles);
        return cudaGetLastError();
    }
    if (s.starts) {
        q.before = s.before;
        if ((e = pass("scan_state_local", kLocal)) != cudaSuccess) return e;
        TimedLaunch t("scan_starts", a.stream);
        scan_starts_kernel<K><<<dim3(a.seq.N, a.G * q.p.U, K * kPT / 2048), 256, 0, a.stream>>>(q.p, q.seg_tokens, s.seg, s.seg_gam, s.starts,
                                                                                            s.last);
        return cudaGetLastError();
    }
    if (split) {
        if ((e = pass(REVERSE ? "scan_seg_bwd" : "scan_seg", kEnds)) != cudaSuccess) return e;
        TimedLaunch t("scan_compose", a.stream);
        scan_compose_kernel<K, REVERSE><<<dim3(a.seq.N, a.G * q.p.U, K * kPT / 1024), 256, 0, a.stream>>>(q.p, q.seg_tokens, s.first, s.seg,
                                                                                                     s.seg_gam);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return pass(REVERSE ? "scan_state_bwd" : "scan_state", kWalk);
}

}  // namespace

cudaError_t launch_gates(const ScanArgs &a, const Gates &g) {
    // the kernels behind this one read the offsets unchecked
    const int slots = std::max(1, a.seq.total ? a.seq.slots(kC) : 0);
    TimedLaunch t("scan_gates", a.stream);
    scan_gates_tc_kernel<<<dim3(slots, (a.H + 7) / 8), 256, 0, a.stream>>>(params(a, g));
    return cudaGetLastError();
}

// One CTA per SM at a time: where sequences x unit pairs fill less than the SMs, a sequence is
// cut into as many segments as fit beside each other, of at least 2 chunks (a packed batch, of
// unknown lengths, always by its total). 0: whole sequences.
int chunks_per_segment(const ScanArgs &a) {
    const int S = a.P / kPT, U = a.H / a.G * S, pairs = a.G * ((U + 1) / 2);
    const int rows = a.seq.cu ? 1 : a.seq.N;
    const long long chunks = a.seq.cu ? (a.seq.total + kC - 1) / kC : (a.seq.T + kC - 1) / kC;
    const int fit = sm_count() / std::max(1, pairs * rows);
    if (fit < 2 || chunks < 4) return 0;
    // a packed batch's sequences end inside segments: twice as many even the SMs' shares out (measured on one
    // batch, 16 sequences of 64 .. 8192 tokens, 16 pairs: 124 + 21 us of state and start kernels with 15 or 16
    // chunks, 143 + 20 with 29)
    const int segments = a.seq.cu ? 2 * fit : fit;
    return (int)std::max<long long>(2, (chunks + segments - 1) / segments);
}

// Of sm_100's 126 MB of L2; the tiles that are written meanwhile pass through it too.
constexpr size_t kProductBytes = (size_t)100 << 20;

bool products_fit(const ScanArgs &a) { return chunks_per_segment(a) > 0 && 2 * tile_bytes(a) <= kProductBytes; }

size_t segment_bytes(const ScanArgs &a) {
    const int c = chunks_per_segment(a);
    if (!c) return 0;
    if (a.products) return align_up(2 * tile_bytes(a));
    const size_t slots = a.seq.slots(c * kC);
    return align_up(slots * a.H * (a.P / kPT) * kPT * a.K * 4) + align_up(slots * a.H * 4);
}

size_t local_bytes(const ScanArgs &a) {
    const int c = chunks_per_segment(a);
    if (!c || a.products) return 0;
    return align_up((size_t)a.seq.slots(c * kC) * a.H * a.P * a.K * 2) + align_up((size_t)a.seq.slots(kC) * a.H * 4);
}

cudaError_t launch_states(const StateArgs &s) {
    if (s.a->K == 128) return s.reverse ? run<128, true>(s) : run<128, false>(s);
    return s.reverse ? run<64, true>(s) : run<64, false>(s);
}

}  // namespace scan_tc
}  // namespace gdn
