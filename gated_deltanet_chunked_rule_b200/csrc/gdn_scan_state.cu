// gdn_scan_state.cu -- state passes of the tensor-core selective scan: the state at the
// start of every chunk (or, backwards, its gradient at the end), and the last one.
//
//   h' = e^{gam_C} h + B^T Xs,   Xs = diag(delta e^{gam_C - gam}) X        (forward)
//   g  = e^{gam_C} g' + C^T Xs,  Xs = diag(e^{gam}) dY                     (reverse)
//
// The product does not depend on the state, so only one multiply-add per element is
// sequential. A CTA walks the chunks of one segment of a sequence with two units (128
// accumulator columns) of a group: warps 0-3 hold unit 0's state rows in fp32 registers (a
// thread per row of K, 64 columns), warps 4-7 unit 1's, warp 8 loads the tiles by TMA (two
// stages), warp 9 issues the products.
//
// The fp32 state keeps fp32 precision although the tensor core takes bf16: B is bf16 as it
// is, and Xs is cut into three bf16 terms that hold its 24 bits exactly (8 + 8 + 8, by
// truncation); two terms left 2.5e-6 in the final state. The second and third term are
// multiplied first, so that their buffer is free for the next chunk while the first one's
// product still runs, and the accumulator has two buffers.
//
// A sequence is cut into segments where units and sequences alone would not fill the SMs: a
// first pass takes every segment from a zero state, one small kernel composes the segments'
// starts (their operator is one scalar decay), a second pass walks them again.
#include <algorithm>

#include "gdn_scan_tc.cuh"

namespace gdn {
namespace scan_tc {
namespace {

using namespace sm100;
using namespace gdn::warp;

constexpr int kThreads = 320;
constexpr int kStage = 65536;           // one stage: B (or C) tile 32 KB, x (or dY) tiles 2 x 16 KB
constexpr int kMid = 2 * kStage;        // second and third terms: 2 x (2 x 16 KB)
constexpr int kSmall = kMid + 65536;    // scan scratch, barriers
constexpr int kSmem = kSmall + 512 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");

struct StateP {
    Params p;
    int seg_tokens;   // tokens of a segment
    bool ends_only;   // the first pass: segment ends from zero
    const float *first;
    float *last, *seg, *seg_gam;
    Tiles tiles;
};

template <int K, bool REVERSE>
__global__ void __launch_bounds__(kThreads, 1)
scan_state_kernel(const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_x, const StateP q) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    const uint32_t sb = smem_u32(smem);
    const Params &p = q.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pairs = (p.U + 1) / 2, g = blockIdx.y / pairs, u0 = (blockIdx.y % pairs) * 2;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_cu(p.m, p.status, tid, kThreads);

    float *wsum = reinterpret_cast<float *>(smem + kSmall);  // [2 units][2 parities][4 warps]
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kSmall + 128);
    uint64_t *full = bars, *empty = bars + 2, *dfull = bars + 4, *xs_ready = bars + 6, *ml_free = bars + 7;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    int n, local;
    const bool used = p.m.slot(blockIdx.x, q.seg_tokens, &n, &local);
    const int s_begin = p.m.begin(n), s_len = p.m.end(n) - s_begin;
    const int unit_of = warp >> 2;  // (warps 0-7) this thread's unit of the pair
    const int u = u0 + unit_of;
    const bool mine = warp < 8 && u < p.U;
    const int h = mine ? p.head(g, u) : 0, col0 = mine ? (u % p.S) * kPT : 0;
    const int row = (warp & 3) * 32 + lane;
    const size_t user = (((size_t)n * p.H + h) * K + row) * p.P + col0;  // this row in the user's states
    if (!used) {  // an empty sequence keeps its state
        if (local == 0 && s_len == 0 && !q.ends_only && q.last && mine && row < K)
            for (int i = 0; i < kPT; ++i) q.last[user + i] = q.first ? q.first[user + i] : 0.f;
        return;
    }
    const int seg_begin = s_begin + local * q.seg_tokens, seg_len = min(q.seg_tokens, s_begin + s_len - seg_begin);
    const bool at_first = REVERSE ? seg_begin + seg_len == s_begin + s_len : local == 0;
    const bool at_last = REVERSE ? local == 0 : seg_begin + seg_len == s_begin + s_len;
    if (q.ends_only && at_last) return;  // nothing follows it
    const int chunks = (seg_len + kC - 1) / kC;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1), mbar_init(&dfull[i], 1);
        mbar_init(xs_ready, 256);
        mbar_init(ml_free, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 8) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto chunk_at = [&](int i) { return REVERSE ? chunks - 1 - i : i; };
    auto fail = [&]() {
        *abort_flag = 1;
        set_status(p.status, GDN_ERR_TIMEOUT);
    };

    if (warp == 8) {
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
                    tma_load_3d(dst + 32768 + j * 16384, &tm_x, &full[st], ((u0 + j) % p.S) * kPT, p.head(g, u0 + j), t0);
            }
            if (!ok) fail();
            // no copy outlives the CTA: the last two stages issued are waited for
            for (int k = max(0, i - 2); k < i; ++k)
                if (!drain(&full[k & 1], (k >> 1) & 1)) fail();
        }
    } else if (warp == 9) {
        if (lane == 0) {
            const uint32_t id = idesc_bf16(128, 128, true, true);
            bool ok = true;
            for (int i = 0; i < chunks && ok; ++i) {
                ok = wait_bar(xs_ready, i & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint32_t a = sb + (i & 1) * kStage, d = tmem + (i & 1) * 128;
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    mma_bf16(d, by_rows(a, k & 7), by_rows(sb + kMid + (k >> 3) * 32768, k & 7), id, k > 0);
                mma_commit(ml_free);
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_bf16(d, by_rows(a, k), by_rows(a + 32768, k), id, true);
                mma_commit(&dfull[i & 1]);
                mma_commit(&empty[i & 1]);
            }
            if (!ok) fail();
        }
    } else {
        float st[kPT];  // the state's row
        const size_t units = (size_t)p.G * p.U, seg_at = ((size_t)blockIdx.x * units + g * p.U + u) * kPT * K + row;
        const bool real = mine && row < K;
        if (real && !q.ends_only && (at_first ? q.first != nullptr : true)) {
#pragma unroll
            for (int i = 0; i < kPT; ++i) st[i] = at_first ? q.first[user + i] : q.seg[seg_at + (size_t)i * K];
        } else {
#pragma unroll
            for (int i = 0; i < kPT; ++i) st[i] = 0.f;
        }
        const float A = mine ? p.A[h] : 0.f;
        const int chunk_slot0 = p.m.slot0(n, kC) + (seg_begin - s_begin) / kC;
        auto keep = [&](int i) {  // the state on entry to chunk i of the walk
            if (!q.tiles.hi || !real || q.ends_only) return;
            const size_t at = (((size_t)(chunk_slot0 + chunk_at(i)) * units + g * p.U + u) * kPT) * K + (size_t)row * 8;
#pragma unroll
            for (int b = 0; b < kPT / 8; ++b) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x0 = st[8 * b + 2 * j], x1 = st[8 * b + 2 * j + 1];
                    hi[j] = pack_bf16(x0, x1);
                    lo[j] = pack_bf16(x0 - bf_lo(hi[j]), x1 - bf_hi(hi[j]));
                }
                *reinterpret_cast<uint4 *>(q.tiles.hi + at + (size_t)b * K * 8) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                if (q.tiles.lo)
                    *reinterpret_cast<uint4 *>(q.tiles.lo + at + (size_t)b * K * 8) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        };
        keep(0);
        auto fetch = [&](int i) {  // dt (+ bias) of this thread's token of chunk i
            const int t = chunk_at(i) * kC + row;
            return mine && i < chunks && t < seg_len ? p.raw_dt(seg_begin + t, h) : 0.f;
        };
        float raw = fetch(0), gam_sum = 0.f, decay_prev = 0.f;
        bool ok = true;
        for (int i = 0; i <= chunks; ++i) {
            float decay = 0.f;
            if (i < chunks) {
                const int len = min(kC, seg_len - chunk_at(i) * kC);
                const bool live = row < len;
                const float delta = live ? p.delta(raw) : 0.f;
                raw = fetch(i + 1);
                // running sums of the log decay: to the right of the token (forward), up to and
                // including it (reverse); summed from the end that matters, for their precision
                const float lg = mine ? delta * A : 0.f;
                float x = lg;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float y = REVERSE ? __shfl_up_sync(0xffffffffu, x, o) : __shfl_down_sync(0xffffffffu, x, o);
                    if (REVERSE ? lane >= o : lane + o < 32) x += y;
                }
                float *ws = wsum + (unit_of * 2 + (i & 1)) * 4;
                if (lane == (REVERSE ? 31 : 0)) ws[warp & 3] = x;
                if (unit_of) named_sync<128>(2);
                else named_sync<128>(1);
                float total = 0.f, off = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    total += ws[k];
                    if (REVERSE ? k < (warp & 3) : k > (warp & 3)) off += ws[k];
                }
                const float e = REVERSE ? x + off : (x - lg) + off;
                const float scale = live ? (REVERSE ? expf(e) : delta * expf(e)) : 0.f;
                decay = expf(total);
                gam_sum += total;
                // a wait that expired: no more work and no more waits, but every barrier of the
                // loop is still met, so that it ends
                ok = ok && wait_bar(&full[i & 1], (i >> 1) & 1, abort_flag);
                if (i > 0) ok = ok && wait_bar(ml_free, (i - 1) & 1, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                const uint32_t stage = sb + (i & 1) * kStage;
                if (ok && !live && unit_of == 0) {  // rows of the next sequence: no product may meet them
#pragma unroll
                    for (int j = 0; j < K / 8; ++j) st_shared_v4(stage + (j >> 3) * 16384 + piece(row, j & 7), 0u, 0u, 0u, 0u);
                }
                const uint32_t xt = stage + 32768 + unit_of * 16384, mid = sb + kMid + unit_of * 16384;
#pragma unroll
                for (int j = 0; ok && j < 8; ++j) {
                    uint32_t hi[4] = {}, md[4] = {}, lo[4] = {};
                    if (live && mine) {
                        const uint4 v = ld_shared_v4(xt + piece(row, j));
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float a0 = bf_lo(w[k]) * scale, a1 = bf_hi(w[k]) * scale;
                            hi[k] = __byte_perm(__float_as_uint(a0), __float_as_uint(a1), 0x7632);
                            const float b0 = a0 - bf_hi(__float_as_uint(a0)), b1 = a1 - bf_hi(__float_as_uint(a1));
                            md[k] = __byte_perm(__float_as_uint(b0), __float_as_uint(b1), 0x7632);
                            const float c0 = b0 - bf_hi(__float_as_uint(b0)), c1 = b1 - bf_hi(__float_as_uint(b1));
                            lo[k] = __byte_perm(__float_as_uint(c0), __float_as_uint(c1), 0x7632);
                        }
                    }
                    st_shared_v4(xt + piece(row, j), hi[0], hi[1], hi[2], hi[3]);
                    st_shared_v4(mid + piece(row, j), md[0], md[1], md[2], md[3]);
                    st_shared_v4(mid + 32768 + piece(row, j), lo[0], lo[1], lo[2], lo[3]);
                }
                fence_proxy_async();
                tc_fence_before();
                mbar_arrive(xs_ready);
            }
            if (i > 0) {
                ok = __all_sync(0xffffffffu, ok && wait_bar(&dfull[(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag));
                tc_fence_after();
                const uint32_t d = tmem + ((uint32_t)((warp & 3) * 32) << 16) + ((i - 1) & 1) * 128 + unit_of * kPT;
#pragma unroll
                for (int half = 0; ok && half < 2; ++half) {
                    float v[32];
                    tmem_ld32(d + 32 * half, v);
#pragma unroll
                    for (int k = 0; k < 32; ++k) st[32 * half + k] = fmaf(decay_prev, st[32 * half + k], v[k]);
                }
                if (ok && i < chunks) keep(i);
            }
            decay_prev = decay;
        }
        if (!ok) fail();
        if (real && ok) {
            if (q.ends_only) {
#pragma unroll
                for (int i = 0; i < kPT; ++i) q.seg[seg_at + (size_t)i * K] = st[i];
                if (row == 0 && col0 == 0) q.seg_gam[(size_t)blockIdx.x * p.H + h] = gam_sum;
            } else if (at_last && q.last) {
#pragma unroll
                for (int i = 0; i < kPT / 4; ++i)
                    *reinterpret_cast<float4 *>(q.last + user + 4 * i) =
                        make_float4(st[4 * i], st[4 * i + 1], st[4 * i + 2], st[4 * i + 3]);
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// Start states of the segments, in place of their ends: start' = e^{gam} start + end. A
// thread per state element walks a sequence's segments.
template <int K, bool REVERSE>
__global__ void __launch_bounds__(256)
scan_compose_kernel(Params p, int seg_tokens, const float *__restrict__ first, float *__restrict__ seg, const float *__restrict__ seg_gam) {
    const int n = blockIdx.x, unit = blockIdx.y, e = blockIdx.z * 256 + threadIdx.x;  // e = column * K + row
    const int len = p.m.end(n) - p.m.begin(n), segs = (len + seg_tokens - 1) / seg_tokens;
    if (segs < 2) return;
    const int h = p.head(unit / p.U, unit % p.U), col = (unit % p.U % p.S) * kPT + e / K;
    const size_t slot0 = p.m.slot0(n, seg_tokens), units = (size_t)p.G * p.U;
    float cur = first ? first[(((size_t)n * p.H + h) * K + e % K) * p.P + col] : 0.f;
    for (int i = 0; i < segs; ++i) {
        const size_t s = slot0 + (REVERSE ? segs - 1 - i : i);
        float *at = seg + (s * units + unit) * kPT * K + e;
        const float end = i + 1 < segs ? *at : 0.f;
        *at = cur;
        if (i + 1 < segs) cur = fmaf(expf(seg_gam[s * p.H + h]), cur, end);
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
    q.p = params(a);
    q.first = s.first, q.last = s.last, q.seg = s.seg, q.seg_gam = s.seg_gam, q.tiles = s.tiles;
    const bool split = s.chunks_per_seg > 0;
    // without a split a segment is longer than any sequence
    q.seg_tokens = split ? s.chunks_per_seg * kC : std::max(kC, (a.seq.cu ? a.seq.total : a.seq.T) / kC * kC + kC);
    if (a.seq.total == 0 && !a.seq.cu) q.seg_tokens = kC;
    const int slots = a.seq.total == 0 ? a.seq.N : a.seq.slots(q.seg_tokens);
    const int pairs = (q.p.U + 1) / 2;
    auto kernel = scan_state_kernel<K, REVERSE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid(slots, a.G * pairs);
    if (split) {
        q.ends_only = true;
        {
            TimedLaunch t(REVERSE ? "scan_seg_bwd" : "scan_seg", a.stream);
            kernel<<<grid, kThreads, kSmem, a.stream>>>(mb, mx, q);
        }
        q.ends_only = false;
        TimedLaunch t("scan_compose", a.stream);
        scan_compose_kernel<K, REVERSE><<<dim3(a.seq.N, a.G * q.p.U, K * kPT / 256), 256, 0, a.stream>>>(q.p, q.seg_tokens, s.first, s.seg,
                                                                                                     s.seg_gam);
    }
    TimedLaunch t(REVERSE ? "scan_state_bwd" : "scan_state", a.stream);
    kernel<<<grid, kThreads, kSmem, a.stream>>>(mb, mx, q);
    return cudaGetLastError();
}

}  // namespace

// One CTA per SM at a time: where sequences x unit pairs fill less than the SMs, a sequence is
// cut into as many segments as fit beside each other, of at least 4 chunks (a packed batch, of
// unknown lengths, always by its total). 0: whole sequences.
int chunks_per_segment(const ScanArgs &a) {
    const int S = a.P / kPT, U = a.H / a.G * S, pairs = a.G * ((U + 1) / 2);
    const int rows = a.seq.cu ? 1 : a.seq.N;
    const long long chunks = a.seq.cu ? (a.seq.total + kC - 1) / kC : (a.seq.T + kC - 1) / kC;
    const int fit = sm_count() / std::max(1, pairs * rows);
    if (fit < 2 || chunks < 8) return 0;
    return (int)std::max<long long>(4, (chunks + fit - 1) / fit);
}

size_t segment_bytes(const ScanArgs &a) {
    const int c = chunks_per_segment(a);
    if (!c) return 0;
    const size_t slots = a.seq.slots(c * kC);
    return align_up(slots * a.H * (a.P / kPT) * kPT * a.K * 4) + align_up(slots * a.H * 4);
}

cudaError_t launch_states(const StateArgs &s) {
    if (s.a->K == 128) return s.reverse ? run<128, true>(s) : run<128, false>(s);
    return s.reverse ? run<64, true>(s) : run<64, false>(s);
}

}  // namespace scan_tc
}  // namespace gdn
