// gdn_layer_api.cu -- C entry points of the operators around the gated delta rule:
// the short causal convolution, the selective state space scan and the gated layer norm
// (see include/gdn.h). Validates on the host, then launches on the caller's stream.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include <initializer_list>

#include "gdn_host.cuh"
#include "gdn_layer.cuh"
#include "gdn_scan_tc.cuh"

using namespace gdn;

namespace {

bool known_dtype(int d) { return d == GDN_DTYPE_F32 || d == GDN_DTYPE_BF16; }

size_t elem(int dtype) { return dtype == GDN_DTYPE_F32 ? 4 : 2; }

bool all_aligned16(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (p && !aligned16(p)) return false;
    return true;
}

// Whether an output is one of the call's inputs: other blocks may still read them.
bool over_input(std::initializer_list<const void *> outs, std::initializer_list<const void *> ins) {
    for (const void *o : outs)
        for (const void *i : ins)
            if (o && o == i) return true;
    return false;
}

// The sequences of a problem; GDN_OK or why they are refused.
int make_seq(int B, int T, int num_seqs, const int32_t *cu, SeqMap *m) {
    if (B < 1 || T < 0 || num_seqs < 0) return GDN_ERR_INVALID_ARG;
    const long long total = (long long)B * T;
    if (total > (1ll << 30) || num_seqs > (1 << 30)) return GDN_ERR_INVALID_ARG;  // tokens and slots are counted in int
    if (num_seqs > 0 && (B != 1 || !cu)) return GDN_ERR_INVALID_ARG;
    m->cu = num_seqs > 0 ? cu : nullptr;
    m->N = num_seqs > 0 ? num_seqs : B;
    m->T = T;
    m->total = (int)total;
    return GDN_OK;
}

int conv_args(const gdn_conv_problem *p, ConvArgs *a) {
    if (!p) return GDN_ERR_INVALID_ARG;
    memset(a, 0, sizeof(*a));
    if (!known_dtype(p->dtype)) return GDN_ERR_UNSUPPORTED;
    if (p->C < 1 || p->W < 1) return GDN_ERR_INVALID_ARG;
    if (p->W < 2 || p->W > 4 || p->C > (1 << 20)) return GDN_ERR_UNSUPPORTED;
    const int rc = make_seq(p->B, p->T, p->num_seqs, p->cu_seqlens, &a->seq);
    if (rc != GDN_OK) return rc;
    if (p->x_stride < p->C) return GDN_ERR_INVALID_ARG;
    a->C = p->C, a->W = p->W, a->dtype = p->dtype, a->silu = p->silu != 0, a->x_stride = p->x_stride;
    return GDN_OK;
}

bool env_is(const char *name, const char *value) {
    const char *e = getenv(name);
    return e && strcmp(e, value) == 0;
}

int scan_args(const gdn_scan_problem *p, ScanArgs *a) {
    if (!p) return GDN_ERR_INVALID_ARG;
    memset(a, 0, sizeof(*a));
    if (!known_dtype(p->dtype) || !known_dtype(p->dt_dtype)) return GDN_ERR_UNSUPPORTED;
    if (p->dt_dtype != GDN_DTYPE_F32 && p->dt_dtype != p->dtype) return GDN_ERR_UNSUPPORTED;
    if (p->Hq < 1 || p->Hv < 1 || p->K < 1 || p->V < 1) return GDN_ERR_INVALID_ARG;
    if (p->Hv % p->Hq) return GDN_ERR_INVALID_ARG;
    if ((p->K != 64 && p->K != 128) || (p->V != 64 && p->V != 128) || p->Hv > 1024) return GDN_ERR_UNSUPPORTED;
    const int rc = make_seq(p->B, p->T, p->num_seqs, p->cu_seqlens, &a->seq);
    if (rc != GDN_OK) return rc;
    const int el = 16 / (int)elem(p->dtype);
    if (p->x_stride < (long long)p->Hv * p->V || p->b_stride < (long long)p->Hq * p->K ||
        p->c_stride < (long long)p->Hq * p->K || p->dt_stride < p->Hv || p->x_stride % el || p->b_stride % el || p->c_stride % el)
        return GDN_ERR_INVALID_ARG;
    a->G = p->Hq, a->H = p->Hv, a->K = p->K, a->P = p->V;
    a->dtype = p->dtype, a->dt_dtype = p->dt_dtype, a->softplus = p->dt_softplus != 0;
    a->xs = p->x_stride, a->bs = p->b_stride, a->cs = p->c_stride, a->dts = p->dt_stride;
    // bf16 prompts take the tensor-core kernels; fp32 ones, and all under GDN_IMPL=simt, the CUDA cores. The
    // two switches (see gdn.h) are read here and nowhere else, so that a call and its kernels agree.
    a->tensor_cores = a->dtype == GDN_DTYPE_BF16 && !env_is("GDN_IMPL", "simt");
    a->products = a->tensor_cores && !env_is("GDN_SCAN_SPLIT", "segments") && scan_tc::products_fit(*a);
    return GDN_OK;
}

int norm_args(const gdn_norm_problem *p, NormArgs *a) {
    if (!p) return GDN_ERR_INVALID_ARG;
    memset(a, 0, sizeof(*a));
    if (!known_dtype(p->dtype) || !known_dtype(p->weight_dtype)) return GDN_ERR_UNSUPPORTED;
    if (p->weight_dtype != GDN_DTYPE_F32 && p->weight_dtype != p->dtype) return GDN_ERR_UNSUPPORTED;
    if (p->rows < 0 || p->D < 1 || !(p->eps >= 0.f) || isinf(p->eps)) return GDN_ERR_INVALID_ARG;
    if (p->D > (1 << 20)) return GDN_ERR_UNSUPPORTED;
    a->R = p->rows, a->D = p->D, a->dtype = p->dtype, a->wdtype = p->weight_dtype, a->eps = p->eps;
    a->center = p->center != 0, a->gate_first = p->gate_first != 0;
    return GDN_OK;
}

// What the forward keeps: the gates, and every chunk's entry state in three parts.
size_t scan_saved_bytes(const ScanArgs &a) { return scan_tc::gates_bytes(a) + 3 * align_up(scan_tc::tile_bytes(a)); }

// Forward workspace: segment scratch | for a call that keeps nothing: gates | entry states (hi) |
// segments' starts.
struct ScanFwdLayout {
    size_t seg, gates, tiles, local, total;
};
ScanFwdLayout scan_fwd_layout(const ScanArgs &a) {
    ScanFwdLayout L;
    L.seg = 0;
    L.gates = L.seg + scan_tc::segment_bytes(a);
    L.tiles = L.gates + scan_tc::gates_bytes(a);
    L.local = L.tiles + align_up(scan_tc::tile_bytes(a));
    L.total = L.local + scan_tc::local_bytes(a);
    return L;
}

scan_tc::StateArgs state_pass(const ScanArgs &a, const scan_tc::Gates &gates, bool reverse, char *seg) {
    scan_tc::StateArgs s{};
    s.a = &a;
    s.gates = gates;
    s.reverse = reverse;
    s.after_gates = !reverse;
    s.chunks_per_seg = scan_tc::chunks_per_segment(a);
    if (s.chunks_per_seg) {
        const size_t slots = a.seq.slots(s.chunks_per_seg * scan_tc::kC);
        s.seg = (float *)seg;
        s.products = a.products;
        s.seg_gam = (float *)(seg + align_up(slots * a.H * a.P * a.K * sizeof(float)));
    }
    s.first = reverse ? a.dht : a.h0;
    s.last = reverse ? a.dh0 : a.final_state;
    return s;
}

scan_tc::Tiles tile_parts(char *at, const ScanArgs &a) {
    const size_t part = align_up(scan_tc::tile_bytes(a));
    return scan_tc::Tiles{(__nv_bfloat16 *)at, (__nv_bfloat16 *)(at + part), (__nv_bfloat16 *)(at + 2 * part)};
}

cudaError_t scan_fwd_tc(const ScanArgs &a) {
    const ScanFwdLayout L = scan_fwd_layout(a);
    char *ws = (char *)a.ws, *saved = (char *)a.saved;
    const scan_tc::Gates gates = scan_tc::gates_at(saved ? saved : ws + L.gates, a);
    cudaError_t e = scan_tc::launch_gates(a, gates);
    if (e != cudaSuccess) return e;
    scan_tc::StateArgs s = state_pass(a, gates, false, ws + L.seg);
    s.tiles = saved ? tile_parts(saved + scan_tc::gates_bytes(a), a) : scan_tc::Tiles{(__nv_bfloat16 *)(ws + L.tiles), nullptr, nullptr};
    scan_tc::Locals locals{};
    if (!saved && scan_tc::local_bytes(a)) {
        locals.seg_tokens = s.chunks_per_seg * scan_tc::kC;
        s.starts = (__nv_bfloat16 *)(ws + L.local);
        s.before = (float *)(ws + L.local + align_up((size_t)a.seq.slots(locals.seg_tokens) * a.H * a.P * a.K * 2));
        locals.starts = s.starts, locals.before = s.before;
    }
    if ((e = scan_tc::launch_states(s)) != cudaSuccess) return e;
    return scan_tc::launch_out(a, gates, s.tiles.hi, locals);
}

// Backward workspace: segment scratch | exit-state gradients (three parts) | the gradient kernel's
// parts | gates and entry states, as the forward keeps them: last, since only a call without
// `saved` needs them.
struct ScanBwdLayout {
    size_t seg, g, grad, saved, total;
};
ScanBwdLayout scan_bwd_layout(const ScanArgs &a) {
    ScanBwdLayout L;
    L.seg = 0;
    L.g = L.seg + scan_tc::segment_bytes(a);
    L.grad = L.g + 3 * align_up(scan_tc::tile_bytes(a));
    L.saved = L.grad + scan_tc::grad_bytes(a);
    L.total = L.saved + scan_saved_bytes(a);
    return L;
}

cudaError_t scan_bwd_tc(const ScanArgs &a) {
    const ScanBwdLayout L = scan_bwd_layout(a);
    char *ws = (char *)a.ws, *saved = a.saved ? (char *)a.saved : ws + L.saved;
    const scan_tc::Gates gates = scan_tc::gates_at(saved, a);
    const scan_tc::Tiles g = tile_parts(ws + L.g, a), h = tile_parts(saved + scan_tc::gates_bytes(a), a);
    cudaError_t e;
    if (!a.saved) {
        if ((e = scan_tc::launch_gates(a, gates)) != cudaSuccess) return e;
        scan_tc::StateArgs s = state_pass(a, gates, false, ws + L.seg);
        s.last = nullptr;
        s.tiles = h;
        if ((e = scan_tc::launch_states(s)) != cudaSuccess) return e;
    }
    scan_tc::StateArgs s = state_pass(a, gates, true, ws + L.seg);
    s.tiles = g;
    if ((e = scan_tc::launch_states(s)) != cudaSuccess) return e;
    return scan_tc::launch_grad(a, gates, h, g, ws + L.grad);
}

size_t scan_fwd_bytes(const ScanArgs &a) { return a.tensor_cores ? scan_fwd_layout(a).total : scan_simt_fwd_bytes(a); }
size_t scan_bwd_bytes(const ScanArgs &a) { return a.tensor_cores ? scan_bwd_layout(a).total : align_up(scan_simt_bwd_bytes(a)); }

int finish(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

bool good_ws(const void *ws, size_t have, size_t need) {
    return have >= need && (ws || !need) && !((uintptr_t)ws & 255u);
}

}  // namespace

extern "C" {

// ----------------------------------------------------------------- convolution
size_t gdn_conv_bwd_workspace_size(const gdn_conv_problem *p) {
    ConvArgs a;
    return conv_args(p, &a) == GDN_OK ? align_up(conv_part_bytes(a.seq.total, a.C, a.W)) : 0;
}

int gdn_conv_fwd(const gdn_conv_problem *p, const void *x, const void *weight, const void *bias, const void *initial_state,
                 void *y, void *final_state, void *stream) {
    ConvArgs a;
    const int rc = conv_args(p, &a);
    if (rc != GDN_OK) return rc;
    if (!weight || (a.seq.total && (!x || !y))) return GDN_ERR_INVALID_ARG;
    if (!all_aligned16({x, weight, bias, initial_state, y, final_state})) return GDN_ERR_INVALID_ARG;
    if (over_input({y, final_state}, {x, weight, bias, initial_state})) return GDN_ERR_INVALID_ARG;
    a.x = x, a.weight = weight, a.bias = bias, a.state = initial_state, a.y = y, a.final_state = final_state;
    a.stream = (cudaStream_t)stream;
    if (!(a.status = status_ptr())) return GDN_ERR_CUDA;
    TimedLaunch t("conv_fwd", a.stream);
    return finish(launch_conv_fwd(a));
}

int gdn_conv_bwd(const gdn_conv_problem *p, const void *x, const void *weight, const void *bias, const void *initial_state,
                 const void *dy, const void *dfinal, void *dx, void *dweight, void *dbias, void *dinitial_state, void *workspace,
                 size_t workspace_bytes, void *stream) {
    ConvArgs a;
    const int rc = conv_args(p, &a);
    if (rc != GDN_OK) return rc;
    if (!weight || !dweight || (a.seq.total && (!x || !dy || !dx))) return GDN_ERR_INVALID_ARG;
    if (!all_aligned16({x, weight, bias, initial_state, dy, dfinal, dx, dweight, dbias, dinitial_state})) return GDN_ERR_INVALID_ARG;
    if (!good_ws(workspace, workspace_bytes, conv_part_bytes(a.seq.total, a.C, a.W))) return GDN_ERR_WORKSPACE;
    if (over_input({dx, dweight, dbias, dinitial_state}, {x, weight, bias, initial_state, dy, dfinal})) return GDN_ERR_INVALID_ARG;
    a.x = x, a.weight = weight, a.bias = bias, a.state = initial_state, a.dy = dy, a.dfinal = dfinal;
    a.dx = dx, a.dweight = dweight, a.dbias = dbias, a.dstate = dinitial_state, a.part = (float *)workspace;
    a.stream = (cudaStream_t)stream;
    if (!(a.status = status_ptr())) return GDN_ERR_CUDA;
    return finish(launch_conv_bwd(a));
}

int gdn_conv_update(const gdn_conv_problem *p, const void *x, const void *weight, const void *bias, void *state, void *y,
                    void *stream) {
    ConvArgs a;
    const int rc = conv_args(p, &a);
    if (rc != GDN_OK) return rc;
    if (p->num_seqs || !weight || !state || (a.seq.total && (!x || !y))) return GDN_ERR_INVALID_ARG;
    if (!all_aligned16({x, weight, bias, state, y})) return GDN_ERR_INVALID_ARG;
    if (over_input({y}, {x, weight, bias, state}) || over_input({state}, {x, weight, bias})) return GDN_ERR_INVALID_ARG;
    a.x = x, a.weight = weight, a.bias = bias, a.state = state, a.y = y;
    a.stream = (cudaStream_t)stream;
    TimedLaunch t("conv_update", a.stream);
    return finish(launch_conv_update(a));
}

// ------------------------------------------------------------------------ scan
size_t gdn_scan_saved_size(const gdn_scan_problem *p) {
    ScanArgs a;
    return scan_args(p, &a) == GDN_OK && a.tensor_cores ? scan_saved_bytes(a) : 0;
}

size_t gdn_scan_fwd_workspace_size(const gdn_scan_problem *p) {
    ScanArgs a;
    return scan_args(p, &a) == GDN_OK ? scan_fwd_bytes(a) : 0;
}

size_t gdn_scan_bwd_workspace_size(const gdn_scan_problem *p) {
    ScanArgs a;
    return scan_args(p, &a) == GDN_OK ? scan_bwd_bytes(a) : 0;
}

static int scan_inputs(const gdn_scan_problem *p, ScanArgs *a, const void *x, const void *dt, const float *A, const void *B,
                       const void *C, const float *D, const float *dt_bias, const float *h0, void *stream) {
    const int rc = scan_args(p, a);
    if (rc != GDN_OK) return rc;
    if (!A || (a->seq.total && (!x || !dt || !B || !C))) return GDN_ERR_INVALID_ARG;
    if (!all_aligned16({x, A, B, C, D, dt_bias, h0}) || ((uintptr_t)dt & (elem(a->dt_dtype) - 1))) return GDN_ERR_INVALID_ARG;
    a->x = x, a->dt = dt, a->A = A, a->B = B, a->C = C, a->D = D, a->dt_bias = dt_bias, a->h0 = h0;
    a->stream = (cudaStream_t)stream;
    return GDN_OK;
}

int gdn_scan_fwd(const gdn_scan_problem *p, const void *x, const void *dt, const float *A, const void *B, const void *C,
                 const float *D, const float *dt_bias, const float *h0, void *y, float *final_state, void *saved, void *workspace,
                 size_t workspace_bytes, void *stream) {
    ScanArgs a;
    const int rc = scan_inputs(p, &a, x, dt, A, B, C, D, dt_bias, h0, stream);
    if (rc != GDN_OK) return rc;
    if (a.seq.total && !y) return GDN_ERR_INVALID_ARG;
    if (!all_aligned16({y, final_state}) || ((uintptr_t)saved & 255u)) return GDN_ERR_INVALID_ARG;
    if (!good_ws(workspace, workspace_bytes, scan_fwd_bytes(a))) return GDN_ERR_WORKSPACE;
    if (over_input({y, final_state}, {x, dt, A, B, C, D, dt_bias, h0})) return GDN_ERR_INVALID_ARG;
    a.y = y, a.final_state = final_state, a.saved = saved, a.ws = workspace;
    if (!(a.status = status_ptr())) return GDN_ERR_CUDA;
    if (a.tensor_cores) return finish(scan_fwd_tc(a));
    TimedLaunch t("scan_fwd", a.stream);
    return finish(launch_scan_simt_fwd(a));
}

int gdn_scan_step(const gdn_scan_problem *p, const void *x, const void *dt, const float *A, const void *B, const void *C,
                  const float *D, const float *dt_bias, const float *h0, void *y, float *final_state, void *stream) {
    ScanArgs a;
    const int rc = scan_inputs(p, &a, x, dt, A, B, C, D, dt_bias, h0, stream);
    if (rc != GDN_OK) return rc;
    if (a.seq.total && !y) return GDN_ERR_INVALID_ARG;
    if (!all_aligned16({y, final_state})) return GDN_ERR_INVALID_ARG;
    if (over_input({y}, {x, dt, A, B, C, D, dt_bias, h0, final_state}) || over_input({final_state}, {x, dt, A, B, C, D, dt_bias}))
        return GDN_ERR_INVALID_ARG;  // (h0 may be updated in place)
    a.y = y, a.final_state = final_state;
    if (!(a.status = status_ptr())) return GDN_ERR_CUDA;
    TimedLaunch t("scan_step", a.stream);
    return finish(launch_scan_step(a));
}

int gdn_scan_bwd(const gdn_scan_problem *p, const void *x, const void *dt, const float *A, const void *B, const void *C,
                 const float *D, const float *dt_bias, const float *h0, const void *saved, const void *dy, const float *dht, void *dx,
                 void *ddt, float *dA, void *dB, void *dC, float *dD, float *ddt_bias, float *dh0, void *workspace,
                 size_t workspace_bytes, void *stream) {
    ScanArgs a;
    const int rc = scan_inputs(p, &a, x, dt, A, B, C, D, dt_bias, h0, stream);
    if (rc != GDN_OK) return rc;
    if (!dA || (a.seq.total && (!dy || !dx || !ddt || !dB || !dC))) return GDN_ERR_INVALID_ARG;
    if (!all_aligned16({dy, dht, dx, ddt, dA, dB, dC, dD, ddt_bias, dh0}) || ((uintptr_t)saved & 255u)) return GDN_ERR_INVALID_ARG;
    const size_t kept = a.tensor_cores && saved ? scan_saved_bytes(a) : 0;
    if (!good_ws(workspace, workspace_bytes, scan_bwd_bytes(a) - kept)) return GDN_ERR_WORKSPACE;
    if (over_input({dx, ddt, dA, dB, dC, dD, ddt_bias, dh0}, {x, dt, A, B, C, D, dt_bias, h0, saved, dy, dht})) return GDN_ERR_INVALID_ARG;
    a.saved = const_cast<void *>(saved), a.dy = dy, a.dht = dht, a.dx = dx, a.ddt = ddt, a.dA = dA, a.dB = dB, a.dC = dC, a.dD = dD;
    a.ddt_bias = ddt_bias, a.dh0 = dh0, a.ws = workspace;
    if (!(a.status = status_ptr())) return GDN_ERR_CUDA;
    if (a.tensor_cores) return finish(scan_bwd_tc(a));
    TimedLaunch t("scan_bwd", a.stream);
    return finish(launch_scan_simt_bwd(a));
}

// ------------------------------------------------------------------------ norm
size_t gdn_norm_bwd_workspace_size(const gdn_norm_problem *p) {
    NormArgs a;
    return norm_args(p, &a) == GDN_OK ? align_up(norm_part_bytes(a)) : 0;
}

int gdn_norm_fwd(const gdn_norm_problem *p, const void *x, const void *weight, const void *bias, const void *gate, void *y,
                 float *stats, void *stream) {
    NormArgs a;
    const int rc = norm_args(p, &a);
    if (rc != GDN_OK) return rc;
    if (!weight || (a.R && (!x || !y))) return GDN_ERR_INVALID_ARG;
    if (!all_aligned16({x, weight, bias, gate, y, stats})) return GDN_ERR_INVALID_ARG;
    if (over_input({y, stats}, {x, weight, bias, gate})) return GDN_ERR_INVALID_ARG;
    a.x = x, a.weight = weight, a.bias = bias, a.gate = gate, a.y = y, a.stats = stats, a.stream = (cudaStream_t)stream;
    TimedLaunch t("norm_fwd", a.stream);
    return finish(launch_norm_fwd(a));
}

int gdn_norm_bwd(const gdn_norm_problem *p, const void *x, const void *weight, const void *bias, const void *gate, const void *dy,
                 const float *stats, void *dx, void *dweight, void *dbias, void *dgate, void *workspace, size_t workspace_bytes,
                 void *stream) {
    NormArgs a;
    const int rc = norm_args(p, &a);
    if (rc != GDN_OK) return rc;
    if (!weight || !dweight || (a.R && (!x || !dy || !stats || !dx || (gate && !dgate)))) return GDN_ERR_INVALID_ARG;
    if (!all_aligned16({x, weight, bias, gate, dy, stats, dx, dweight, dbias, dgate})) return GDN_ERR_INVALID_ARG;
    if (!good_ws(workspace, workspace_bytes, norm_part_bytes(a))) return GDN_ERR_WORKSPACE;
    if (over_input({dx, dweight, dbias, dgate}, {x, weight, bias, gate, dy, stats})) return GDN_ERR_INVALID_ARG;
    a.x = x, a.weight = weight, a.bias = bias, a.gate = gate, a.dy = dy, a.stats = const_cast<float *>(stats);
    a.dx = dx, a.dweight = dweight, a.dbias = dbias, a.dgate = dgate, a.part = (float *)workspace, a.stream = (cudaStream_t)stream;
    TimedLaunch t("norm_bwd", a.stream);
    return finish(launch_norm_bwd(a));
}

}  // extern "C"
