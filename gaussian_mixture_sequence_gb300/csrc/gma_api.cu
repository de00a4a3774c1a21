// C ABI of libgma: host-side validation, workspace layout and launch order.
// The operations are those of the GMA explainer "Gaussian Mixture Attention:
// Linear-Time Sequence Mixing via Probabilistic Latent Routing" (technical
// summary, "핵심 메커니즘" and "변형 및 학습"); see include/gma.h.
#include "gma_operators.cuh"

#include <math.h>

#include <atomic>
#include <mutex>

using namespace gma;

namespace {

struct WsPlan {
    size_t zq = 0;        // the routing of Q's zero-lo-plane flags (bounded routing, split layout)
    size_t prm = 0, cst = 0, gq = 0, gk = 0, partial = 0, total = 0, mem = 0, wimg = 0, wimg3 = 0, pimg = 0,
           cimg = 0, pimg2 = 0, dctl = 0, dlist = 0, dlist2 = 0, bytes = 0;
    long long dcap = 0;   // dense-list entries per head
    bool pruned = false;  // the bounded routing (K = 128, d = 64)
    bool gtc = false;     // the tensor-core routing for 17 <= K <= 256 (not 128), d = 64
};

bool valid_width(int w) { return w == 16 || w == 32 || w == 64 || w == 128; }

gma_status make_dims_raw(const gma_shape *s, Dims *dm);
#define GMA_TRY_DIMS(expr)                                                                                 \
    do {                                                                                                   \
        const gma_status _d = (expr);                                                                      \
        if (_d != GMA_OK) return _d;                                                                       \
    } while (0)

// Dims of one operation: only the causal form uses the tensor-core chunking.
gma_status make_dims(const gma_shape *s, Dims *dm, gma_op op = GMA_OP_CAUSAL)
{
    const gma_status st = make_dims_raw(s, dm);
    if (st == GMA_OK && op != GMA_OP_CAUSAL && op != GMA_OP_BIDIR && dm->C == 128) {
        dm->C = 64;
        dm->blk = kBlockRows;
        dm->KG = dm->KP;
    }
    return st;
}

// Dims of the gradient pass: the CUDA-core chunking (C = 64, blocks of kBlockRows rows) and
// fp32 responsibilities whatever the shape's chunk and product type.
gma_status make_dims_bwd(const gma_shape *s, Dims *dm)
{
    if (!s) return GMA_ERR_INVALID_ARG;
    gma_shape t = *s;
    t.chunk = 64;
    t.gemm_dtype = GMA_F32;
    GMA_TRY_DIMS(make_dims_raw(&t, dm));
    return GMA_OK;
}

gma_status make_dims_raw(const gma_shape *s, Dims *dm)
{
    if (!s) return GMA_ERR_INVALID_ARG;
    if (s->B < 1 || s->H < 1 || s->N < 0 || s->K < 1 || s->d_route < 1 || s->d_v < 1 || s->chunk < 0)
        return GMA_ERR_INVALID_ARG;
    if (!(s->eps >= 0.f) || !isfinite(s->eps)) return GMA_ERR_INVALID_ARG;
    if ((unsigned)s->x_dtype > 1u || (unsigned)s->v_dtype > 1u || (unsigned)s->gemm_dtype > 1u)
        return GMA_ERR_INVALID_ARG;
    if (!valid_width(s->d_route) || !valid_width(s->d_v) || s->K > 512) return GMA_ERR_UNSUPPORTED;
    const bool tc = tc_path_eligible(s->K, s->d_v, s->gemm_dtype == GMA_BF16);
    const int C = s->chunk == 0 ? (tc ? 128 : 64) : s->chunk;
    if (C != 16 && C != 32 && C != 64 && !(C == 128 && tc)) return GMA_ERR_UNSUPPORTED;
    const long long BH = (long long)s->B * s->H;
    if (BH > 65535) return GMA_ERR_UNSUPPORTED;
    const long long w = s->K > s->d_v ? (s->K > s->d_route ? s->K : s->d_route)
                                      : (s->d_v > s->d_route ? s->d_v : s->d_route);
    if (BH * (long long)s->N * w >= (1LL << 40)) return GMA_ERR_UNSUPPORTED;
    dm->B = s->B; dm->H = s->H; dm->N = s->N; dm->D = s->d_route; dm->DV = s->d_v; dm->K = s->K;
    dm->KP = (int)round_up(s->K, 8);
    dm->KG = C == 128 ? tc_kpad(s->K) : dm->KP;
    dm->C = C;
    dm->blk = C == 128 ? 128 : kBlockRows;
    dm->eps = s->eps;
    dm->x_bf16 = s->x_dtype == GMA_BF16;
    dm->v_bf16 = s->v_dtype == GMA_BF16;
    dm->g_bf16 = s->gemm_dtype == GMA_BF16;
    return GMA_OK;
}

// The bounded routing's per-head images and its two tile lists (dcap entries per head each), and
// (zq_words > 0) the routing of Q's flags of tiles whose lo plane it leaves unwritten.
template <class Take>
void plan_pruned(WsPlan &p, int H, long long dcap, Take &&take, long long zq_words = 0)
{
    p.pruned = true;
    if (zq_words > 0) p.zq = take((size_t)zq_words * 4);
    p.wimg = take((size_t)H * kPrunedWBytes);
    p.wimg3 = take((size_t)H * kPrunedW3Bytes);
    p.pimg = take((size_t)H * kPrunedPBytes);
    p.cimg = take((size_t)H * kPrunedCBytes);
    p.pimg2 = take((size_t)H * kPrunedP2Bytes);
    p.dcap = dcap;
    p.dctl = take((size_t)H * 2 * 4);
    p.dlist = take((size_t)H * dcap * 8);
    p.dlist2 = take((size_t)H * dcap * 8);
}

int gamma_layout(const Dims &dm);

WsPlan plan(const Dims &dm, gma_op op)
{
    WsPlan p;
    size_t off = 0;
    auto take = [&](size_t n) {
        const size_t o = off;
        off = (size_t)round_up((long long)(off + n), 256);
        return o;
    };
    p.prm = take((size_t)dm.H * dm.K * (dm.D / 2) * 16);
    p.cst = take((size_t)dm.H * dm.K * 4);
    if (op != GMA_OP_DECODE && resp_pruned_applies(dm))   // both routings of a head; the flags where
        plan_pruned(p, dm.H, 2 * routing_tiles(dm.B, dm.N), take,   // the chunk kernels read split planes
                    (op == GMA_OP_BIDIR || op == GMA_OP_CAUSAL) && gamma_layout(dm) == GL_SPLIT
                        ? dm.BH() * ((dm.N + 127) / 128) : 0);
    if (op != GMA_OP_DECODE && resp_gtc_applies(dm)) {
        p.gtc = true;
        p.wimg3 = take(gtc_image_bytes(dm));
    }
    if (op == GMA_OP_USAGE) {   // Gamma in fp32, then the per-block partial sums and counts
        p.gq = take((size_t)dm.BH() * dm.N * dm.K * 4);
        p.partial = take((size_t)dm.BH() * usage_blocks(dm) * dm.K * 4);
        p.total = take((size_t)dm.BH() * usage_blocks(dm) * dm.K * 4);
    }
    if (op == GMA_OP_BIDIR || op == GMA_OP_CAUSAL) {
        const size_t gb = dm.g_bf16 ? 2 : 4;
        p.gq = take((size_t)dm.BH() * dm.N * dm.KG * gb);
        p.gk = take((size_t)dm.BH() * dm.N * dm.KG * gb);
        p.partial = take((size_t)dm.BH() * dm.nblk() * dm.state_size() * 4);
        const bool tc = tc_path_applies(dm);
        if (op == GMA_OP_BIDIR)   // the total memory: fp32, or in operand form on the tensor-core path
            p.total = take((size_t)dm.BH() * (tc ? tc_mem_words(dm) : dm.state_size()) * 4);
        if (op == GMA_OP_CAUSAL && tc)   // the carried memory of every chunk in operand form
            p.mem = take((size_t)dm.BH() * dm.nblk() * tc_mem_words(dm) * 4);
    }
    p.bytes = off;
    return p;
}

// Workspace form of the responsibilities: the fp32 tensor-core path takes split bf16 planes.
int gamma_layout(const Dims &dm) { return dm.g_bf16 ? GL_BF16 : (tc_path_applies(dm) ? GL_SPLIT : GL_F32); }

bool aligned(const void *p) { return ((uintptr_t)p & 15u) == 0; }

gma_status check_ptr(const void *p, bool required = true)
{
    if (!p) return required ? GMA_ERR_INVALID_ARG : GMA_OK;
    return aligned(p) ? GMA_OK : GMA_ERR_ALIGNMENT;
}

gma_status check_params(const gma_params &p)
{
    gma_status s;
    if ((s = check_ptr(p.mu)) != GMA_OK) return s;
    if ((s = check_ptr(p.var_raw)) != GMA_OK) return s;
    return check_ptr(p.logit_pi);
}

gma_status check_ws(void *ws, size_t ws_bytes, const WsPlan &wp)
{
    if (!ws || ws_bytes < wp.bytes) return GMA_ERR_WORKSPACE;
    return aligned(ws) ? GMA_OK : GMA_ERR_ALIGNMENT;
}

#define GMA_TRY(expr)                                                                                      \
    do {                                                                                                   \
        gma_status _s = (expr);                                                                            \
        if (_s != GMA_OK) return _s;                                                                       \
    } while (0)
// The CUDA error behind the last GMA_ERR_CUDA returned on this thread.
thread_local cudaError_t g_last_cuda = cudaSuccess;
#define GMA_CUDA(expr)                                                                                     \
    do {                                                                                                   \
        const cudaError_t _e = (expr);                                                                     \
        if (_e != cudaSuccess) {                                                                           \
            g_last_cuda = _e;                                                                              \
            return GMA_ERR_CUDA;                                                                           \
        }                                                                                                  \
    } while (0)

// A bounded device wait that expired since the last report on the current device:
// GMA_ERR_TIMEOUT once (the flag is cleared), else GMA_OK.  Never allocates and
// never synchronises: a timeout becomes visible once the kernel that hit it has
// written the flag.
gma_status take_timeout()
{
    volatile unsigned int *f = timeout_flag_host();
    if (f && *f) {
        *f = 0u;
        return GMA_ERR_TIMEOUT;
    }
    return GMA_OK;
}

template <typename T>
T *at(void *ws, size_t off) { return reinterpret_cast<T *>(static_cast<char *>(ws) + off); }

// Device copies of the inputs and the output for gma_forward_causal_host.
struct HostStaging {
    size_t q = 0, k = 0, v = 0, out = 0, bytes = 0;
};
HostStaging host_staging(const Dims &dm)
{
    HostStaging h;
    const size_t rows = (size_t)dm.BH() * dm.N;
    auto take = [&](size_t n) {
        const size_t o = h.bytes;
        h.bytes = (size_t)round_up((long long)(h.bytes + n), 256);
        return o;
    };
    h.q = take(rows * dm.D * (dm.x_bf16 ? 2 : 4));
    h.k = take(rows * dm.D * (dm.x_bf16 ? 2 : 4));
    h.v = take(rows * dm.DV * (dm.v_bf16 ? 2 : 4));
    h.out = take(rows * dm.DV * 4);
    return h;
}

// Workspace of the gradient pass.
struct BwdPlan {
    WsPlan w;   // parameters, routing images, gq / gk (fp32), forward memory (partial, total)
    size_t dgq = 0, dgk = 0, u = 0, mem = 0, rtot = 0, pmu = 0, pvar = 0, plp = 0, bytes = 0;
};
BwdPlan plan_bwd_full(const Dims &dm)
{
    BwdPlan b;
    size_t off = 0;
    auto take = [&](size_t n) {
        const size_t o = off;
        off = (size_t)round_up((long long)(off + n), 256);
        return o;
    };
    WsPlan &p = b.w;
    p.prm = take((size_t)dm.H * dm.K * (dm.D / 2) * 16);
    p.cst = take((size_t)dm.H * dm.K * 4);
    if (resp_pruned_applies(dm)) plan_pruned(p, dm.H, 2 * routing_tiles(dm.B, dm.N), take);
    if (resp_gtc_applies(dm)) {
        p.gtc = true;
        p.wimg3 = take(gtc_image_bytes(dm));
    }
    const size_t rows = (size_t)dm.BH() * dm.N, nb = (size_t)dm.BH() * dm.nblk();
    p.gq = take(rows * dm.KP * 4);
    p.gk = take(rows * dm.KP * 4);
    p.partial = take(nb * dm.state_size() * 4);
    p.total = take((size_t)dm.BH() * dm.state_size() * 4);
    b.dgq = take(rows * dm.KP * 4);
    b.dgk = take(rows * dm.KP * 4);
    b.u = take(rows * bwd_u_pitch(dm) * 4);
    b.mem = take(nb * dm.K * bwd_u_pitch(dm) * 4);
    b.rtot = take((size_t)dm.BH() * dm.K * bwd_u_pitch(dm) * 4);
    b.pmu = take(2 * nb * dm.K * dm.D * 4);
    b.pvar = take(2 * nb * dm.K * dm.D * 4);
    b.plp = take(2 * nb * dm.K * 4);
    b.bytes = p.bytes = off;
    return b;
}
WsPlan plan_bwd(const Dims &dm) { return plan_bwd_full(dm).w; }

PrunedImages images(void *ws, const WsPlan &wp)
{
    return PrunedImages{at<unsigned char>(ws, wp.wimg), at<unsigned char>(ws, wp.wimg3), at<float4>(ws, wp.pimg),
                        at<float>(ws, wp.cimg), at<float4>(ws, wp.pimg2), at<unsigned int>(ws, wp.dctl),
                        at<int2>(ws, wp.dlist), at<int2>(ws, wp.dlist2), wp.dcap,
                        wp.zq ? at<unsigned int>(ws, wp.zq) : nullptr};
}

// The routing images a call passes to launch_resp (null for the generic CUDA-core routing).
const PrunedImages *routing_images(const WsPlan &wp, const PrunedImages &img)
{
    return wp.pruned || wp.gtc ? &img : nullptr;
}

// The per-head parameters and the images of the routing kernel the shape takes.
cudaError_t prep_routing(const Dims &dm, const gma_params &params, float4 *prm, float *cst, const WsPlan &wp,
                         const PrunedImages &img, cudaStream_t st)
{
    if (wp.pruned) return launch_prep_all(dm, params, prm, cst, img, st);
    cudaError_t e = launch_prep(dm, params, prm, cst, st);
    if (e == cudaSuccess && wp.gtc) e = launch_prep_gtc(dm, prm, cst, img.w3, st);
    return e;
}

} // namespace

extern "C" {

size_t gma_workspace_size(const gma_shape *shape, gma_op op)
{
    Dims dm;
    if (op == GMA_OP_CAUSAL_HOST) {
        if (make_dims(shape, &dm, GMA_OP_CAUSAL) != GMA_OK) return 0;
        return host_staging(dm).bytes + plan(dm, GMA_OP_CAUSAL).bytes;
    }
    if (op == GMA_OP_BACKWARD) return make_dims_bwd(shape, &dm) == GMA_OK ? plan_bwd(dm).bytes : 0;
    if (((unsigned)op > 3u && op != GMA_OP_USAGE) || make_dims(shape, &dm, op) != GMA_OK) return 0;
    return plan(dm, op).bytes;
}

const char *gma_last_cuda_error(void) { return cudaGetErrorName(g_last_cuda); }

const char *gma_status_string(gma_status status)
{
    switch (status) {
    case GMA_OK: return "ok";
    case GMA_ERR_INVALID_ARG: return "invalid argument";
    case GMA_ERR_UNSUPPORTED: return "unsupported size";
    case GMA_ERR_ALIGNMENT: return "pointer not 16-byte aligned";
    case GMA_ERR_WORKSPACE: return "workspace missing or too small";
    case GMA_ERR_CUDA: return "CUDA error";
    case GMA_ERR_TIMEOUT: return "a bounded device wait expired";
    default: return "unknown status";
    }
}

gma_status gma_responsibilities(const gma_shape *shape, gma_params params, const void *x, float *gamma,
                                void *ws, size_t ws_bytes, gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    Dims dm;
    GMA_TRY(make_dims(shape, &dm, GMA_OP_RESPONSIBILITIES));
    GMA_TRY(check_params(params));
    GMA_TRY(check_ptr(x, dm.N > 0));
    GMA_TRY(check_ptr(gamma, dm.N > 0));
    const WsPlan wp = plan(dm, GMA_OP_RESPONSIBILITIES);
    GMA_TRY(check_ws(ws, ws_bytes, wp));
    if (dm.N == 0) return GMA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float4 *prm = at<float4>(ws, wp.prm);
    float *cst = at<float>(ws, wp.cst);
    const PrunedImages img = images(ws, wp);
    GMA_CUDA(prep_routing(dm, params, prm, cst, wp, img, st));
    GMA_CUDA(launch_resp(dm, prm, cst, routing_images(wp, img), x, gamma, dm.K, GL_F32, st, 0));
    if (wp.pruned) GMA_CUDA(launch_resp_dense(dm, x, gamma, dm, nullptr, nullptr, img, GL_F32, st));
    return GMA_OK;
}

gma_status gma_responsibility_stats(const gma_shape *shape, gma_params params, const void *x, float *usage,
                                    long long *counts, float *entropy, int *assign, void *ws, size_t ws_bytes,
                                    gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    Dims dm;
    GMA_TRY(make_dims(shape, &dm, GMA_OP_USAGE));
    GMA_TRY(check_params(params));
    GMA_TRY(check_ptr(x, dm.N > 0));
    GMA_TRY(check_ptr(usage));
    GMA_TRY(check_ptr(counts));
    GMA_TRY(check_ptr(entropy));
    GMA_TRY(check_ptr(assign, false));
    const WsPlan wp = plan(dm, GMA_OP_USAGE);
    GMA_TRY(check_ws(ws, ws_bytes, wp));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float *gamma = at<float>(ws, wp.gq);
    if (dm.N > 0) {
        float4 *prm = at<float4>(ws, wp.prm);
        float *cst = at<float>(ws, wp.cst);
        const PrunedImages img = images(ws, wp);
        GMA_CUDA(prep_routing(dm, params, prm, cst, wp, img, st));
        GMA_CUDA(launch_resp(dm, prm, cst, routing_images(wp, img), x, gamma, dm.K, GL_F32, st, 0));
        if (wp.pruned) GMA_CUDA(launch_resp_dense(dm, x, gamma, dm, nullptr, nullptr, img, GL_F32, st));
    }
    GMA_CUDA(launch_usage(dm, gamma, dm.K, at<float>(ws, wp.partial), at<int>(ws, wp.total), assign, usage, counts,
                          entropy, st));
    return GMA_OK;
}


} // extern "C"

namespace {

// Records the profiling event of the next launch (no-op without a profile).
struct Marks {
    gma_profile *prof;
    int n = 0;
    cudaStream_t st;
    cudaError_t mark(const char *name)
    {
        if (!prof) return cudaSuccess;
        if (n >= GMA_PROFILE_MAX_STAGES) return cudaErrorInvalidValue;
        prof->stage_name[n] = name;
        return cudaEventRecord(static_cast<cudaEvent_t>(prof->events[n++]), st);
    }
    cudaError_t finish()
    {
        if (!prof) return cudaSuccess;
        prof->n_stages = n;
        return cudaEventRecord(static_cast<cudaEvent_t>(prof->events[n]), st);
    }
};

gma_status check_prof(gma_profile *prof)
{
    if (!prof) return GMA_OK;
    for (int i = 0; i <= GMA_PROFILE_MAX_STAGES; ++i)
        if (!prof->events[i]) return GMA_ERR_INVALID_ARG;
    prof->n_stages = 0;
    return GMA_OK;
}

gma_status run_bidir(const gma_shape *shape, gma_params params, const void *qx, const void *kx, const void *v,
                     float *out, void *ws, size_t ws_bytes, gma_stream_t stream, gma_profile *prof)
{
    Dims dm;
    GMA_TRY(make_dims(shape, &dm, GMA_OP_BIDIR));
    GMA_TRY(check_params(params));
    GMA_TRY(check_ptr(qx, dm.N > 0));
    GMA_TRY(check_ptr(kx, dm.N > 0));
    GMA_TRY(check_ptr(v, dm.N > 0));
    GMA_TRY(check_ptr(out, dm.N > 0));
    const WsPlan wp = plan(dm, GMA_OP_BIDIR);
    GMA_TRY(check_ws(ws, ws_bytes, wp));
    GMA_TRY(check_prof(prof));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Marks mk{prof, 0, st};
    if (dm.N == 0) {
        GMA_CUDA(mk.finish());
        return GMA_OK;
    }
    float4 *prm = at<float4>(ws, wp.prm);
    float *cst = at<float>(ws, wp.cst);
    void *gq = at<char>(ws, wp.gq), *gk = at<char>(ws, wp.gk);
    float *partial = at<float>(ws, wp.partial), *total = at<float>(ws, wp.total);
    const PrunedImages img = images(ws, wp);
    const PrunedImages *imgp = routing_images(wp, img);
    GMA_CUDA(mk.mark(wp.pruned ? "prep" : "prep_params"));
    GMA_CUDA(prep_routing(dm, params, prm, cst, wp, img, st));
    GMA_CUDA(mk.mark("resp_q"));
    GMA_CUDA(launch_resp(dm, prm, cst, imgp, qx, gq, dm.KG, gamma_layout(dm), st, 0));
    GMA_CUDA(mk.mark("resp_k"));
    GMA_CUDA(launch_resp(dm, prm, cst, imgp, kx, gk, dm.KG, gamma_layout(dm), st, 1));
    if (wp.pruned) {
        GMA_CUDA(mk.mark("resp_dense"));
        GMA_CUDA(launch_resp_dense(dm, qx, gq, dm, kx, gk, img, gamma_layout(dm), st));
    }
    if (tc_path_applies(dm)) {
        GMA_CUDA(mk.mark("chunk_state_tc"));
        GMA_CUDA(launch_chunk_state_tc(dm, gk, v, partial, st));
        GMA_CUDA(mk.mark("state_reduce"));
        unsigned char *tot = at<unsigned char>(ws, wp.total);
        GMA_CUDA(launch_scan_split(dm, partial, nullptr, nullptr, tot, nullptr, st));
        GMA_CUDA(mk.mark("bidir_read_tc"));
        GMA_CUDA(launch_chunk_out_tc(dm, false, gq, gk, v, tot, out, st, img.zq));
    } else {
        GMA_CUDA(mk.mark("block_state"));
        GMA_CUDA(launch_block_state(dm, gk, v, partial, st));
        GMA_CUDA(mk.mark("state_reduce"));
        GMA_CUDA(launch_scan(dm, partial, nullptr, total, false, st));
        GMA_CUDA(mk.mark("bidir_read"));
        GMA_CUDA(launch_chunk_out(dm, false, gq, gk, v, total, out, st));
    }
    GMA_CUDA(mk.finish());
    return GMA_OK;
}

// Workspace of the cross form: queries of dm_q, keys and values of dm_kv (same B, H, d, K).
WsPlan plan_cross(const Dims &dq, const Dims &dk)
{
    WsPlan p;
    size_t off = 0;
    auto take = [&](size_t n) {
        const size_t o = off;
        off = (size_t)round_up((long long)(off + n), 256);
        return o;
    };
    p.prm = take((size_t)dq.H * dq.K * (dq.D / 2) * 16);
    p.cst = take((size_t)dq.H * dq.K * 4);
    if (resp_pruned_applies(dq))
        plan_pruned(p, dq.H, routing_tiles(dq.B, dq.N) + routing_tiles(dk.B, dk.N), take,
                    gamma_layout(dq) == GL_SPLIT ? dq.BH() * ((dq.N + 127) / 128) : 0);
    if (resp_gtc_applies(dq)) {
        p.gtc = true;
        p.wimg3 = take(gtc_image_bytes(dq));
    }
    const size_t gb = dq.g_bf16 ? 2 : 4;
    p.gq = take((size_t)dq.BH() * dq.N * dq.KG * gb);
    p.gk = take((size_t)dk.BH() * dk.N * dk.KG * gb);
    p.partial = take((size_t)dk.BH() * dk.nblk() * dk.state_size() * 4);
    p.total = take((size_t)dk.BH() * (tc_path_applies(dq) ? tc_mem_words(dq) : dk.state_size()) * 4);
    p.bytes = off;
    return p;
}

gma_status cross_dims(const gma_shape *shape, int n_kv, Dims *dq, Dims *dk)
{
    GMA_TRY(make_dims(shape, dq, GMA_OP_BIDIR));
    if (n_kv < 0) return GMA_ERR_INVALID_ARG;
    gma_shape sk = *shape;
    sk.N = n_kv;
    return make_dims(&sk, dk, GMA_OP_BIDIR);
}

// Queries of dq read the memory written by all keys of dk: the bidirectional write over
// dk's rows, then the bidirectional read over dq's rows.
gma_status run_cross(const gma_shape *shape, int n_kv, gma_params params, const void *qx, const void *kx,
                     const void *v, float *out, void *ws, size_t ws_bytes, gma_stream_t stream)
{
    Dims dq, dk;
    GMA_TRY(cross_dims(shape, n_kv, &dq, &dk));
    GMA_TRY(check_params(params));
    GMA_TRY(check_ptr(qx, dq.N > 0));
    GMA_TRY(check_ptr(out, dq.N > 0));
    GMA_TRY(check_ptr(kx, dk.N > 0 && dq.N > 0));
    GMA_TRY(check_ptr(v, dk.N > 0 && dq.N > 0));
    const WsPlan wp = plan_cross(dq, dk);
    GMA_TRY(check_ws(ws, ws_bytes, wp));
    if (dq.N == 0) return GMA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float4 *prm = at<float4>(ws, wp.prm);
    float *cst = at<float>(ws, wp.cst);
    void *gq = at<char>(ws, wp.gq), *gk = at<char>(ws, wp.gk);
    float *partial = at<float>(ws, wp.partial), *total = at<float>(ws, wp.total);
    const PrunedImages img = images(ws, wp);
    const PrunedImages *imgp = routing_images(wp, img);
    GMA_CUDA(prep_routing(dq, params, prm, cst, wp, img, st));
    GMA_CUDA(launch_resp(dq, prm, cst, imgp, qx, gq, dq.KG, gamma_layout(dq), st, 0));
    if (dk.N > 0) GMA_CUDA(launch_resp(dk, prm, cst, imgp, kx, gk, dk.KG, gamma_layout(dk), st, 1));
    if (wp.pruned)
        GMA_CUDA(launch_resp_dense(dq, qx, gq, dk, dk.N > 0 ? kx : nullptr, gk, img, gamma_layout(dq), st));
    const bool tc = tc_path_applies(dq);
    if (dk.N == 0) {   // no keys: an empty memory (zeros in either layout)
        GMA_CUDA(cudaMemsetAsync(total, 0, (size_t)dk.BH() * (tc ? tc_mem_words(dk) : dk.state_size()) * 4, st));
    } else {
        if (tc) {
            GMA_CUDA(launch_chunk_state_tc(dk, gk, v, partial, st));
            GMA_CUDA(launch_scan_split(dk, partial, nullptr, nullptr, reinterpret_cast<unsigned char *>(total),
                                       nullptr, st));
        } else {
            GMA_CUDA(launch_block_state(dk, gk, v, partial, st));
            GMA_CUDA(launch_scan(dk, partial, nullptr, total, false, st));
        }
    }
    if (tc)
        GMA_CUDA(launch_chunk_out_tc(dq, false, gq, gq, nullptr, reinterpret_cast<unsigned char *>(total), out, st,
                                     img.zq));
    else
        GMA_CUDA(launch_chunk_out(dq, false, gq, gq, nullptr, total, out, st));
    return GMA_OK;
}

gma_status run_decode(const gma_shape *shape, gma_params params, const void *qx, const void *kx, const void *v,
                      float *state, float *out, void *ws, size_t ws_bytes, gma_stream_t stream, gma_profile *prof)
{
    Dims dm;
    GMA_TRY(make_dims(shape, &dm, GMA_OP_DECODE));
    GMA_TRY(check_params(params));
    GMA_TRY(check_ptr(qx));
    GMA_TRY(check_ptr(kx));
    GMA_TRY(check_ptr(v));
    GMA_TRY(check_ptr(state));
    GMA_TRY(check_ptr(out));
    const WsPlan wp = plan(dm, GMA_OP_DECODE);
    GMA_TRY(check_ws(ws, ws_bytes, wp));
    GMA_TRY(check_prof(prof));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Marks mk{prof, 0, st};
    float4 *prm = at<float4>(ws, wp.prm);
    float *cst = at<float>(ws, wp.cst);
    // one stage: the decode kernel is a programmatic dependent of the parameter preparation and
    // overlaps it (an event recorded between the two would serialise them)
    GMA_CUDA(mk.mark("decode"));
    GMA_CUDA(launch_prep(dm, params, prm, cst, st));
    GMA_CUDA(launch_decode(dm, prm, cst, qx, kx, v, state, out, st));
    GMA_CUDA(mk.finish());
    return GMA_OK;
}

gma_status run_causal(const gma_shape *shape, gma_params params, const void *qx, const void *kx,
                      const void *v, const float *state_in, float *state_out, float *out, void *ws,
                      size_t ws_bytes, gma_stream_t stream, gma_profile *prof)
{
    Dims dm;
    GMA_TRY(make_dims(shape, &dm));
    GMA_TRY(check_params(params));
    GMA_TRY(check_ptr(qx, dm.N > 0));
    GMA_TRY(check_ptr(kx, dm.N > 0));
    GMA_TRY(check_ptr(v, dm.N > 0));
    GMA_TRY(check_ptr(out, dm.N > 0));
    GMA_TRY(check_ptr(state_in, false));
    GMA_TRY(check_ptr(state_out, false));
    const WsPlan wp = plan(dm, GMA_OP_CAUSAL);
    GMA_TRY(check_ws(ws, ws_bytes, wp));
    GMA_TRY(check_prof(prof));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Marks mk{prof, 0, st};
    if (dm.N == 0) {
        if (state_out && state_out != state_in) {
            const size_t bytes = (size_t)dm.BH() * dm.state_size() * 4;
            if (state_in)
                GMA_CUDA(cudaMemcpyAsync(state_out, state_in, bytes, cudaMemcpyDeviceToDevice, st));
            else
                GMA_CUDA(cudaMemsetAsync(state_out, 0, bytes, st));
        }
        GMA_CUDA(mk.finish());
        return GMA_OK;
    }
    float4 *prm = at<float4>(ws, wp.prm);
    float *cst = at<float>(ws, wp.cst);
    void *gq = at<char>(ws, wp.gq), *gk = at<char>(ws, wp.gk);
    float *partial = at<float>(ws, wp.partial);
    const PrunedImages img = images(ws, wp);
    const PrunedImages *imgp = routing_images(wp, img);
    GMA_CUDA(mk.mark(wp.pruned ? "prep" : "prep_params"));
    GMA_CUDA(prep_routing(dm, params, prm, cst, wp, img, st));
    GMA_CUDA(mk.mark("resp_q"));
    GMA_CUDA(launch_resp(dm, prm, cst, imgp, qx, gq, dm.KG, gamma_layout(dm), st, 0));
    GMA_CUDA(mk.mark("resp_k"));
    GMA_CUDA(launch_resp(dm, prm, cst, imgp, kx, gk, dm.KG, gamma_layout(dm), st, 1));
    if (wp.pruned) {
        GMA_CUDA(mk.mark("resp_dense"));
        GMA_CUDA(launch_resp_dense(dm, qx, gq, dm, kx, gk, img, gamma_layout(dm), st));
    }
    if (tc_path_applies(dm)) {
        GMA_CUDA(mk.mark("chunk_state_tc"));
        GMA_CUDA(launch_chunk_state_tc(dm, gk, v, partial, st));
        GMA_CUDA(mk.mark("state_scan"));
        unsigned char *mem = at<unsigned char>(ws, wp.mem);
        GMA_CUDA(launch_scan_split(dm, partial, state_in, mem, nullptr, state_out, st));
        GMA_CUDA(mk.mark("chunk_out_tc"));
        GMA_CUDA(launch_chunk_out_tc(dm, true, gq, gk, v, mem, out, st, img.zq));
    } else {
        GMA_CUDA(mk.mark("block_state"));
        GMA_CUDA(launch_block_state(dm, gk, v, partial, st));
        GMA_CUDA(mk.mark("state_scan"));
        GMA_CUDA(launch_scan(dm, partial, state_in, state_out, true, st));
        GMA_CUDA(mk.mark("chunk_out"));
        GMA_CUDA(launch_chunk_out(dm, true, gq, gk, v, partial, out, st));
    }
    GMA_CUDA(mk.finish());
    return GMA_OK;
}

} // namespace

extern "C" {

gma_status gma_forward_causal(const gma_shape *shape, gma_params params, const void *qx, const void *kx,
                              const void *v, const float *state_in, float *state_out, float *out, void *ws,
                              size_t ws_bytes, gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    return run_causal(shape, params, qx, kx, v, state_in, state_out, out, ws, ws_bytes, stream, nullptr);
}

gma_status gma_forward_bidir(const gma_shape *shape, gma_params params, const void *qx, const void *kx,
                             const void *v, float *out, void *ws, size_t ws_bytes, gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    return run_bidir(shape, params, qx, kx, v, out, ws, ws_bytes, stream, nullptr);
}

gma_status gma_forward_bidir_profiled(const gma_shape *shape, gma_params params, const void *qx,
                                      const void *kx, const void *v, float *out, void *ws, size_t ws_bytes,
                                      gma_stream_t stream, gma_profile *prof)
{
    GMA_TRY(take_timeout());
    if (!prof) return GMA_ERR_INVALID_ARG;
    return run_bidir(shape, params, qx, kx, v, out, ws, ws_bytes, stream, prof);
}

gma_status gma_decode_step(const gma_shape *shape, gma_params params, const void *qx, const void *kx,
                           const void *v, float *state, float *out, void *ws, size_t ws_bytes,
                           gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    return run_decode(shape, params, qx, kx, v, state, out, ws, ws_bytes, stream, nullptr);
}

gma_status gma_decode_step_profiled(const gma_shape *shape, gma_params params, const void *qx, const void *kx,
                                    const void *v, float *state, float *out, void *ws, size_t ws_bytes,
                                    gma_stream_t stream, gma_profile *prof)
{
    GMA_TRY(take_timeout());
    if (!prof) return GMA_ERR_INVALID_ARG;
    return run_decode(shape, params, qx, kx, v, state, out, ws, ws_bytes, stream, prof);
}

gma_status gma_forward_causal_profiled(const gma_shape *shape, gma_params params, const void *qx,
                                       const void *kx, const void *v, const float *state_in,
                                       float *state_out, float *out, void *ws, size_t ws_bytes,
                                       gma_stream_t stream, gma_profile *prof)
{
    GMA_TRY(take_timeout());
    if (!prof) return GMA_ERR_INVALID_ARG;
    return run_causal(shape, params, qx, kx, v, state_in, state_out, out, ws, ws_bytes, stream, prof);
}


} // extern "C"

// ---- causal forward on host buffers ----------------------------------------
namespace {

constexpr int kMaxCopyDevices = 64;
std::once_flag g_copy_once[kMaxCopyDevices];
cudaStream_t g_copy_in[kMaxCopyDevices], g_copy_out[kMaxCopyDevices];
cudaError_t g_copy_err[kMaxCopyDevices];

// The two copy streams of the current device (created once, never destroyed).
gma_status copy_streams(cudaStream_t *in, cudaStream_t *out)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return GMA_ERR_CUDA;
    if (dev < 0 || dev >= kMaxCopyDevices) return GMA_ERR_UNSUPPORTED;
    std::call_once(g_copy_once[dev], [dev] {
        g_copy_err[dev] = cudaStreamCreateWithFlags(&g_copy_in[dev], cudaStreamNonBlocking);
        if (g_copy_err[dev] == cudaSuccess)
            g_copy_err[dev] = cudaStreamCreateWithFlags(&g_copy_out[dev], cudaStreamNonBlocking);
    });
    if (g_copy_err[dev] != cudaSuccess) return GMA_ERR_CUDA;
    *in = g_copy_in[dev];
    *out = g_copy_out[dev];
    return GMA_OK;
}

// Records an event on `from` and makes `to` wait for it.
cudaError_t join(cudaStream_t to, cudaStream_t from)
{
    cudaEvent_t e;
    cudaError_t err = cudaEventCreateWithFlags(&e, cudaEventDisableTiming);
    if (err != cudaSuccess) return err;
    err = cudaEventRecord(e, from);
    if (err == cudaSuccess) err = cudaStreamWaitEvent(to, e, 0);
    cudaEventDestroy(e);   // released once the recorded work completes
    return err;
}

} // namespace

extern "C" gma_status gma_forward_causal_host(const gma_shape *shape, gma_params params, const void *qx,
                                              const void *kx, const void *v, const float *state_in,
                                              float *state_out, float *out, void *ws, size_t ws_bytes,
                                              gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    Dims dm;
    GMA_TRY(make_dims(shape, &dm));
    GMA_TRY(check_params(params));
    if (dm.N > 0 && (!qx || !kx || !v || !out)) return GMA_ERR_INVALID_ARG;
    GMA_TRY(check_ptr(state_in, false));
    GMA_TRY(check_ptr(state_out, false));
    const HostStaging hs = host_staging(dm);
    const WsPlan wp = plan(dm, GMA_OP_CAUSAL);
    if (!ws || ws_bytes < hs.bytes + wp.bytes) return GMA_ERR_WORKSPACE;
    if (!aligned(ws)) return GMA_ERR_ALIGNMENT;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    char *w = static_cast<char *>(ws);
    char *cws = w + hs.bytes;
    const size_t cws_bytes = ws_bytes - hs.bytes;
    if (dm.N == 0)
        return run_causal(shape, params, nullptr, nullptr, nullptr, state_in, state_out, nullptr, cws, cws_bytes,
                          stream, nullptr);
    cudaStream_t cin, cout_;
    GMA_TRY(copy_streams(&cin, &cout_));
    // groups of slices: one batch entry and a range of heads, about eight groups in all
    const int split = dm.B >= 8 ? 1 : (8 + dm.B - 1) / dm.B;
    const int hg = (dm.H + split - 1) / split;
    const size_t xe = dm.x_bf16 ? 2 : 4, ve = dm.v_bf16 ? 2 : 4;
    const size_t xrow = (size_t)dm.N * dm.D * xe, vrow = (size_t)dm.N * dm.DV * ve, orow = (size_t)dm.N * dm.DV * 4;
    const long long SZ = dm.state_size();
    // the staging buffers may still be read by earlier work on `stream`
    GMA_CUDA(join(cin, st));
    for (int b = 0; b < dm.B; ++b)
        for (int h0 = 0; h0 < dm.H; h0 += hg) {
            const int hn = dm.H - h0 < hg ? dm.H - h0 : hg;
            const size_t s0 = (size_t)b * dm.H + h0;   // first slice of the group
            GMA_CUDA(cudaMemcpyAsync(w + hs.q + s0 * xrow, static_cast<const char *>(qx) + s0 * xrow, hn * xrow,
                                     cudaMemcpyHostToDevice, cin));
            GMA_CUDA(cudaMemcpyAsync(w + hs.k + s0 * xrow, static_cast<const char *>(kx) + s0 * xrow, hn * xrow,
                                     cudaMemcpyHostToDevice, cin));
            GMA_CUDA(cudaMemcpyAsync(w + hs.v + s0 * vrow, static_cast<const char *>(v) + s0 * vrow, hn * vrow,
                                     cudaMemcpyHostToDevice, cin));
            GMA_CUDA(join(st, cin));
            gma_shape sg = *shape;
            sg.B = 1;
            sg.H = hn;
            const gma_params pg{params.mu + (size_t)h0 * dm.K * dm.D, params.var_raw + (size_t)h0 * dm.K * dm.D,
                                params.logit_pi + (size_t)h0 * dm.K};
            GMA_TRY(run_causal(&sg, pg, w + hs.q + s0 * xrow, w + hs.k + s0 * xrow, w + hs.v + s0 * vrow,
                               state_in ? state_in + s0 * SZ : nullptr, state_out ? state_out + s0 * SZ : nullptr,
                               reinterpret_cast<float *>(w + hs.out + s0 * orow), cws, cws_bytes, stream, nullptr));
            GMA_CUDA(join(cout_, st));
            GMA_CUDA(cudaMemcpyAsync(reinterpret_cast<char *>(out) + s0 * orow, w + hs.out + s0 * orow, hn * orow,
                                     cudaMemcpyDeviceToHost, cout_));
        }
    GMA_CUDA(join(st, cout_));   // `stream` completes after the last output copy
    return GMA_OK;
}

// ---- decode step whose scratch is a file-scope device array ----------------
namespace {

__device__ __align__(256) unsigned char g_noalloc_scratch[GMA_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::atomic<void *> g_noalloc_addr[kMaxDevices];

// Device address of the array on the current device.  In host code the
// array's name only stands in for it, so the address is looked up with that
// device current, and kept once a lookup has succeeded (a failed lookup, for
// example one made during a stream capture, is retried by the next call).
gma_status noalloc_scratch(void **addr)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return GMA_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return GMA_ERR_UNSUPPORTED;
    void *p = g_noalloc_addr[dev].load(std::memory_order_acquire);
    if (!p) {
        const cudaError_t e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
        if (e != cudaSuccess || !p) {
            g_last_cuda = e != cudaSuccess ? e : cudaErrorInvalidSymbol;
            return GMA_ERR_CUDA;
        }
        g_noalloc_addr[dev].store(p, std::memory_order_release);
    }
    *addr = p;
    return GMA_OK;
}

} // namespace

extern "C" gma_status gma_decode_step_noalloc(const gma_shape *shape, gma_params params, const void *qx,
                                              const void *kx, const void *v, float *state, float *out,
                                              gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    Dims dm;
    GMA_TRY(make_dims(shape, &dm, GMA_OP_DECODE));
    GMA_TRY(check_params(params));
    GMA_TRY(check_ptr(qx));
    GMA_TRY(check_ptr(kx));
    GMA_TRY(check_ptr(v));
    GMA_TRY(check_ptr(state));
    GMA_TRY(check_ptr(out));
    const WsPlan wp = plan(dm, GMA_OP_DECODE);
    if (wp.bytes > GMA_NOALLOC_SCRATCH_BYTES) return GMA_ERR_WORKSPACE;
    void *ws = nullptr;
    GMA_TRY(noalloc_scratch(&ws));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float4 *prm = at<float4>(ws, wp.prm);
    float *cst = at<float>(ws, wp.cst);
    GMA_CUDA(launch_prep(dm, params, prm, cst, st));
    GMA_CUDA(launch_decode(dm, prm, cst, qx, kx, v, state, out, st));
    return GMA_OK;
}

extern "C" gma_status gma_sync_status(gma_stream_t stream)
{
    const cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        g_last_cuda = e;
        return GMA_ERR_CUDA;
    }
    return take_timeout();
}

extern "C" gma_status gma_test_wait_timeout(long long limit_cycles, gma_stream_t stream)
{
    if (limit_cycles < 1 || limit_cycles > 4000000000LL) return GMA_ERR_INVALID_ARG;
    GMA_CUDA(launch_expire_wait(limit_cycles, reinterpret_cast<cudaStream_t>(stream)));
    return GMA_OK;
}

extern "C" size_t gma_cross_workspace_size(const gma_shape *shape, int n_kv)
{
    Dims dq, dk;
    if (cross_dims(shape, n_kv, &dq, &dk) != GMA_OK) return 0;
    return plan_cross(dq, dk).bytes;
}

extern "C" gma_status gma_forward_cross(const gma_shape *shape, int n_kv, gma_params params, const void *qx,
                                        const void *kx, const void *v, float *out, void *ws, size_t ws_bytes,
                                        gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    return run_cross(shape, n_kv, params, qx, kx, v, out, ws, ws_bytes, stream);
}

extern "C" gma_status gma_backward(const gma_shape *shape, int causal, gma_params params, const void *qx,
                                   const void *kx, const void *v, const float *dout, float *dqx, float *dkx,
                                   float *dv, float *dmu, float *dvar_raw, float *dlogit_pi, void *ws,
                                   size_t ws_bytes, gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    Dims dm;
    GMA_TRY(make_dims_bwd(shape, &dm));
    if (causal != 0 && causal != 1) return GMA_ERR_INVALID_ARG;
    GMA_TRY(check_params(params));
    const bool any = dm.N > 0;
    GMA_TRY(check_ptr(qx, any));
    GMA_TRY(check_ptr(kx, any));
    GMA_TRY(check_ptr(v, any));
    GMA_TRY(check_ptr(dout, any));
    GMA_TRY(check_ptr(dqx, any));
    GMA_TRY(check_ptr(dkx, any));
    GMA_TRY(check_ptr(dv, any));
    GMA_TRY(check_ptr(dmu));
    GMA_TRY(check_ptr(dvar_raw));
    GMA_TRY(check_ptr(dlogit_pi));
    const BwdPlan bp = plan_bwd_full(dm);
    const WsPlan &wp = bp.w;
    GMA_TRY(check_ws(ws, ws_bytes, wp));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!any) {
        GMA_CUDA(cudaMemsetAsync(dmu, 0, (size_t)dm.H * dm.K * dm.D * 4, st));
        GMA_CUDA(cudaMemsetAsync(dvar_raw, 0, (size_t)dm.H * dm.K * dm.D * 4, st));
        GMA_CUDA(cudaMemsetAsync(dlogit_pi, 0, (size_t)dm.H * dm.K * 4, st));
        return GMA_OK;
    }
    float4 *prm = at<float4>(ws, wp.prm);
    float *cst = at<float>(ws, wp.cst);
    float *gq = at<float>(ws, wp.gq), *gk = at<float>(ws, wp.gk);
    float *partial = at<float>(ws, wp.partial), *total = at<float>(ws, wp.total);
    const PrunedImages img = images(ws, wp);
    const PrunedImages *imgp = routing_images(wp, img);
    // the forward's responsibilities (fp32) and memory
    GMA_CUDA(prep_routing(dm, params, prm, cst, wp, img, st));
    GMA_CUDA(launch_resp(dm, prm, cst, imgp, qx, gq, dm.KP, GL_F32, st, 0));
    GMA_CUDA(launch_resp(dm, prm, cst, imgp, kx, gk, dm.KP, GL_F32, st, 1));
    if (wp.pruned) GMA_CUDA(launch_resp_dense(dm, qx, gq, dm, kx, gk, img, GL_F32, st));
    GMA_CUDA(launch_block_state(dm, gk, v, partial, st));
    GMA_CUDA(launch_scan(dm, partial, nullptr, causal ? nullptr : total, causal != 0, st));
    // query side, key / value side, then the routings and the parameters
    float *dgq = at<float>(ws, bp.dgq), *dgk = at<float>(ws, bp.dgk), *u = at<float>(ws, bp.u);
    GMA_CUDA(launch_bwd_q(dm, causal != 0, gq, gk, v, dout, causal ? partial : total, u, dgq, st));
    GMA_CUDA(launch_bwd_kv(dm, causal != 0, gq, gk, v, u, at<float>(ws, bp.mem), at<float>(ws, bp.rtot), dgk, dv, st));
    const size_t pass = (size_t)dm.BH() * dm.nblk() * dm.K;
    float *pmu = at<float>(ws, bp.pmu), *pvar = at<float>(ws, bp.pvar), *plp = at<float>(ws, bp.plp);
    GMA_CUDA(launch_bwd_route(dm, qx, prm, gq, dgq, dqx, pmu, pvar, plp, st));
    GMA_CUDA(launch_bwd_route(dm, kx, prm, gk, dgk, dkx, pmu + pass * dm.D, pvar + pass * dm.D, plp + pass, st));
    GMA_CUDA(launch_bwd_final(dm, params, pmu, pvar, plp, dmu, dvar_raw, dlogit_pi, st));
    return GMA_OK;
}

// ---- the gated recurrence ----
namespace {

// Rows of a sequence: positions are 32-bit, some 10^4 rows (a round of a cluster) past the last one included.
constexpr int kMaxRows = 1 << 30;

gma_status scan_dims(const gma_scan_shape *s, ScanDims *sd)
{
    if (!s) return GMA_ERR_INVALID_ARG;
    if (s->B < 1 || s->H < 1 || s->N < 0 || s->D < 1) return GMA_ERR_INVALID_ARG;
    if ((unsigned)s->form > 1u || (unsigned)s->dtype > 1u) return GMA_ERR_INVALID_ARG;
    const long long S = (long long)s->B * s->H;
    if (S > 65535 || s->D > 65536 || s->N > kMaxRows) return GMA_ERR_UNSUPPORTED;
    if (S * (long long)(s->N > 0 ? s->N : 1) >= (1LL << 40) / s->D) return GMA_ERR_UNSUPPORTED;
    *sd = ScanDims{(int)S, s->H, s->N, s->D, s->form == GMA_SCAN_MEAN, s->dtype == GMA_BF16};
    return GMA_OK;
}

// A buffer of a call: its bytes are read or (out) written.
struct Span {
    const void *p;
    size_t n;
    bool out;
};

// No written buffer may overlap another buffer of the call; `same` lists the one pair that may be
// the same buffer.
gma_status check_overlap(const Span *s, int n, const void *same_a = nullptr, const void *same_b = nullptr)
{
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j) {
            if (!s[i].p || !s[j].p || !(s[i].out || s[j].out)) continue;
            if (s[i].p == same_a && s[j].p == same_b && same_a == same_b && s[i].n == s[j].n) continue;
            const uintptr_t a = (uintptr_t)s[i].p, b = (uintptr_t)s[j].p;
            if (a < b + s[j].n && b < a + s[i].n) return GMA_ERR_INVALID_ARG;
        }
    return GMA_OK;
}

} // namespace

extern "C" gma_status gma_gated_scan(const gma_scan_shape *shape, const void *x, const void *gate, const int *lengths,
                                     const float *state_in, float *state_out, void *out, gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    ScanDims sd;
    GMA_TRY(scan_dims(shape, &sd));
    const bool any = sd.N > 0;
    GMA_TRY(check_ptr(x, any));
    GMA_TRY(check_ptr(gate, any));
    GMA_TRY(check_ptr(out, any));
    GMA_TRY(check_ptr(lengths, false));
    GMA_TRY(check_ptr(state_in, false));
    GMA_TRY(check_ptr(state_out, false));
    const size_t seq = (size_t)sd.S * sd.N * sd.D * (sd.bf16 ? 2 : 4), stb = (size_t)sd.S * sd.D * 4;
    const Span sp[] = {{state_in, stb, false}, {state_out, stb, true}, {x, seq, false}, {gate, seq, false},
                       {out, seq, true}, {lengths, (size_t)shape->B * 4, false}};
    GMA_TRY(check_overlap(sp, 6, state_in, state_out));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!any) {
        if (state_out && state_in && state_out != state_in)
            GMA_CUDA(cudaMemcpyAsync(state_out, state_in, stb, cudaMemcpyDeviceToDevice, st));
        else if (state_out && !state_in)
            GMA_CUDA(cudaMemsetAsync(state_out, 0, stb, st));
        return GMA_OK;
    }
    GMA_CUDA(launch_scan_fwd(sd, x, gate, lengths, state_in, state_out, out, st));
    return GMA_OK;
}

extern "C" gma_status gma_gated_scan_backward(const gma_scan_shape *shape, const void *x, const void *gate,
                                              const void *out, const void *dout, const int *lengths,
                                              const float *state_in, const float *dstate_out, void *dx, void *dgate,
                                              float *dstate_in, gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    ScanDims sd;
    GMA_TRY(scan_dims(shape, &sd));
    const bool any = sd.N > 0;
    GMA_TRY(check_ptr(x, any && sd.mean));
    GMA_TRY(check_ptr(gate, any));
    GMA_TRY(check_ptr(out, any));
    GMA_TRY(check_ptr(dout, any));
    GMA_TRY(check_ptr(dx, any));
    GMA_TRY(check_ptr(dgate, any));
    GMA_TRY(check_ptr(lengths, false));
    GMA_TRY(check_ptr(state_in, false));
    GMA_TRY(check_ptr(dstate_out, false));
    GMA_TRY(check_ptr(dstate_in, false));
    const size_t seq = (size_t)sd.S * sd.N * sd.D * (sd.bf16 ? 2 : 4), stb = (size_t)sd.S * sd.D * 4;
    const Span sp[] = {{dstate_out, stb, false}, {dstate_in, stb, true}, {state_in, stb, false}, {x, seq, false},
                       {gate, seq, false}, {out, seq, false}, {dout, seq, false}, {dx, seq, true}, {dgate, seq, true},
                       {lengths, (size_t)shape->B * 4, false}};
    GMA_TRY(check_overlap(sp, 10, dstate_out, dstate_in));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!any) {
        if (dstate_in && dstate_out && dstate_in != dstate_out)
            GMA_CUDA(cudaMemcpyAsync(dstate_in, dstate_out, stb, cudaMemcpyDeviceToDevice, st));
        else if (dstate_in && !dstate_out)
            GMA_CUDA(cudaMemsetAsync(dstate_in, 0, stb, st));
        return GMA_OK;
    }
    GMA_CUDA(launch_scan_bwd(sd, x, gate, out, dout, lengths, state_in, dstate_out, dx, dgate, dstate_in, st));
    return GMA_OK;
}

extern "C" gma_status gma_gated_step(const gma_scan_shape *shape, const void *x, const void *gate, float *state,
                                     void *out, gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    if (!shape) return GMA_ERR_INVALID_ARG;
    gma_scan_shape one = *shape;
    one.N = 1;
    ScanDims sd;
    GMA_TRY(scan_dims(&one, &sd));
    GMA_TRY(check_ptr(x));
    GMA_TRY(check_ptr(gate));
    GMA_TRY(check_ptr(state));
    GMA_TRY(check_ptr(out));
    const size_t row = (size_t)sd.S * sd.D * (sd.bf16 ? 2 : 4);
    const Span sp[] = {{x, row, false}, {gate, row, false}, {state, (size_t)sd.S * sd.D * 4, true}, {out, row, true}};
    GMA_TRY(check_overlap(sp, 4));
    GMA_CUDA(launch_scan_step(sd, x, gate, state, out, reinterpret_cast<cudaStream_t>(stream)));
    return GMA_OK;
}

// ---- beam search over recurrent states ----
namespace {

gma_status beam_dims(const gma_beam_shape *s, BeamDims *bd)
{
    if (!s) return GMA_ERR_INVALID_ARG;
    if (s->B < 1 || s->W < 1 || s->V < 1 || s->ld < 0 || (s->ld > 0 && s->ld < s->V)) return GMA_ERR_INVALID_ARG;
    if (s->eos < -1 || s->eos >= s->V || s->pad < 0 || s->pad >= s->V) return GMA_ERR_INVALID_ARG;
    if ((unsigned)s->dtype > 1u) return GMA_ERR_INVALID_ARG;
    if (s->W > kMaxBeams || (long long)s->B * s->W > 65535 || s->V > (1 << 30)) return GMA_ERR_UNSUPPORTED;
    *bd = BeamDims{s->B, s->W, s->V, s->ld ? s->ld : s->V, s->eos, s->pad, s->dtype == GMA_BF16};
    return GMA_OK;
}

} // namespace

extern "C" size_t gma_beam_workspace_size(const gma_beam_shape *shape)
{
    BeamDims bd;
    return beam_dims(shape, &bd) == GMA_OK ? beam_ws_bytes(bd) : 0;
}

extern "C" gma_status gma_beam_select(const gma_beam_shape *shape, const void *logits, const float *score_in,
                                      const unsigned char *finished_in, float *score_out, int *parent, int *token,
                                      unsigned char *finished_out, void *ws, size_t ws_bytes, gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    BeamDims bd;
    GMA_TRY(beam_dims(shape, &bd));
    GMA_TRY(check_ptr(logits));
    GMA_TRY(check_ptr(score_in));
    GMA_TRY(check_ptr(finished_in, false));
    GMA_TRY(check_ptr(score_out));
    GMA_TRY(check_ptr(parent));
    GMA_TRY(check_ptr(token));
    GMA_TRY(check_ptr(finished_out, false));
    const size_t rows = (size_t)bd.B * bd.W, need = beam_ws_bytes(bd);
    if (need > 0 && (!ws || ws_bytes < need)) return GMA_ERR_WORKSPACE;
    if (need == 0) ws = nullptr;   // (not looked at)
    GMA_TRY(check_ptr(ws, false));
    const size_t lb = ((rows - 1) * bd.ld + bd.V) * (bd.bf16 ? 2 : 4);
    // scores and flags may be updated in place (a request's CTA reads both before it writes);
    // each pair is checked against everything but itself
    const Span a[] = {{score_in, rows * 4, false}, {score_out, rows * 4, true}, {logits, lb, false}, {ws, need, true},
                      {parent, rows * 4, true}, {token, rows * 4, true}};
    GMA_TRY(check_overlap(a, 6, score_in, score_out));
    const Span f[] = {{finished_in, rows, false}, {finished_out, rows, true}, {logits, lb, false}, {ws, need, true},
                      {parent, rows * 4, true}, {token, rows * 4, true}, {score_out, rows * 4, true}};
    GMA_TRY(check_overlap(f, 7, finished_in, finished_out));
    const Span g[] = {{finished_out, rows, true}, {score_in, rows * 4, false}};
    GMA_TRY(check_overlap(g, 2));
    GMA_CUDA(launch_beam_select(bd, logits, score_in, finished_in, score_out, parent, token, finished_out, ws,
                                reinterpret_cast<cudaStream_t>(stream)));
    return GMA_OK;
}

extern "C" gma_status gma_beam_reorder(int B, int W, size_t row_bytes, const int *parent, void *state,
                                       gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    if (B < 1 || W < 1) return GMA_ERR_INVALID_ARG;
    if (W > kMaxBeams || B > 65535 || row_bytes % 4 != 0) return GMA_ERR_UNSUPPORTED;
    if (row_bytes >= (size_t)(1LL << 40) / ((size_t)B * W)) return GMA_ERR_UNSUPPORTED;
    GMA_TRY(check_ptr(parent));
    GMA_TRY(check_ptr(state, row_bytes > 0));
    const Span s[] = {{parent, (size_t)B * W * 4, false}, {state, (size_t)B * W * row_bytes, true}};
    GMA_TRY(check_overlap(s, 2));
    if (row_bytes == 0 || W == 1) return GMA_OK;
    GMA_CUDA(launch_beam_reorder(B, W, row_bytes, parent, state, reinterpret_cast<cudaStream_t>(stream)));
    return GMA_OK;
}

// ---- the balance loss ----
namespace {

// The walk over a head's rows adds two positions of a sequence in 32 bits.
gma_status balance_dims(const gma_shape *shape, Dims *dm)
{
    GMA_TRY(make_dims(shape, dm, GMA_OP_RESPONSIBILITIES));
    return dm->N > kMaxRows ? GMA_ERR_UNSUPPORTED : GMA_OK;
}

// The routing's scratch, then the loss's; the gradients' takes the place of both.  The routing is one that
// evaluates every component: the bounded routing of K = 128 writes 0 for posteriors below e^-30, and a
// head whose rows are all but one-hot has no others beside the best.
struct BalPlan {
    size_t prm, cst, img;
    bool gtc;
    size_t prec, cst2, second, psum, pcnt, inv, terms, n_terms, hist, part, bytes;
};

BalPlan plan_balance(const Dims &dm)
{
    BalPlan p;
    size_t off = 0;
    auto take = [&](size_t n) {
        const size_t o = off;
        off = (size_t)round_up((long long)(off + n), 256);
        return o;
    };
    const size_t hk = (size_t)dm.H * dm.K, nb = (size_t)dm.H * balance_blocks(dm);
    p.prm = take(hk * (dm.D / 2) * 16);
    p.cst = take(hk * 4);
    p.gtc = resp_gtc_fits(dm) && resp_gtc_output_ok(dm, dm.K, GL_F32);
    p.img = take(p.gtc ? gtc_image_bytes(dm) : 0);
    p.prec = take(hk * dm.D * 8);
    p.cst2 = take(hk * 8);
    p.second = take((size_t)dm.H * 4);
    p.psum = take(nb * dm.K * 4);
    p.pcnt = take(nb * dm.K * 4);
    const size_t fwd = off;
    off = 0;   // the gradients need nothing of the routing's scratch
    p.inv = take(hk * dm.D * 8);
    p.terms = take((size_t)dm.BH() * dm.N * dm.K * 8);
    p.n_terms = take((size_t)dm.BH() * dm.N * 4);
    p.hist = take(hk * 4);
    p.part = take((size_t)balance_parts(dm) * hk * (2 * dm.D + 1) * 4);
    p.bytes = fwd > off ? fwd : off;
    return p;
}

size_t row_bytes(const Dims &dm) { return (size_t)dm.BH() * dm.N * dm.D * (dm.x_bf16 ? 2 : 4); }

} // namespace

extern "C" size_t gma_balance_workspace_size(const gma_shape *shape)
{
    Dims dm;
    return balance_dims(shape, &dm) == GMA_OK ? plan_balance(dm).bytes : 0;
}

extern "C" gma_status gma_balance_loss(const gma_shape *shape, gma_params params, const void *x, const int *lengths,
                                       float *gamma, float *loss, long long *counts, float *prob, void *ws,
                                       size_t ws_bytes, gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    Dims dm;
    GMA_TRY(balance_dims(shape, &dm));
    GMA_TRY(check_params(params));
    GMA_TRY(check_ptr(x, dm.N > 0));
    GMA_TRY(check_ptr(gamma, dm.N > 0));
    GMA_TRY(check_ptr(lengths, false));
    GMA_TRY(check_ptr(loss));
    GMA_TRY(check_ptr(counts));
    GMA_TRY(check_ptr(prob));
    const BalPlan bp = plan_balance(dm);
    if (!ws || ws_bytes < bp.bytes) return GMA_ERR_WORKSPACE;
    GMA_TRY(check_ptr(ws));
    const size_t hk = (size_t)dm.H * dm.K, pb = hk * dm.D * 4;
    const Span sp[] = {{x, row_bytes(dm), false}, {params.mu, pb, false}, {params.var_raw, pb, false},
                       {params.logit_pi, hk * 4, false}, {lengths, (size_t)dm.B * 4, false},
                       {gamma, (size_t)dm.BH() * dm.N * dm.K * 4, true}, {loss, (size_t)dm.H * 4, true},
                       {counts, hk * 8, true}, {prob, hk * 4, true}, {ws, bp.bytes, true}};
    GMA_TRY(check_overlap(sp, 10));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float2 *prec = at<float2>(ws, bp.prec), *cst2 = at<float2>(ws, bp.cst2);
    float *second = at<float>(ws, bp.second);
    if (dm.N > 0) {
        float4 *prm = at<float4>(ws, bp.prm);
        float *cst = at<float>(ws, bp.cst);
        unsigned char *img = at<unsigned char>(ws, bp.img);
        GMA_CUDA(launch_balance_prep(dm, params, prec, cst2, second, st));
        GMA_CUDA(launch_prep(dm, params, prm, cst, st));
        if (bp.gtc) {
            GMA_CUDA(launch_prep_gtc(dm, prm, cst, img, st));
            GMA_CUDA(launch_resp_gtc(dm, img, prm, cst, x, gamma, dm.K, GL_F32, st));
        } else {
            GMA_CUDA(launch_resp(dm, prm, cst, nullptr, x, gamma, dm.K, GL_F32, st));
        }
    }
    GMA_CUDA(launch_balance_loss(dm, params, x, lengths, prec, cst2, second, gamma, at<float>(ws, bp.psum),
                                 at<int>(ws, bp.pcnt), loss, counts, prob, st));
    return GMA_OK;
}

extern "C" gma_status gma_balance_backward(const gma_shape *shape, gma_params params, const void *x,
                                           const int *lengths, const float *gamma, const long long *counts,
                                           const float *dloss, float *dx, float *dmu, float *dvar_raw,
                                           float *dlogit_pi, int accumulate, void *ws, size_t ws_bytes,
                                           gma_stream_t stream)
{
    GMA_TRY(take_timeout());
    Dims dm;
    GMA_TRY(balance_dims(shape, &dm));
    if (accumulate != 0 && accumulate != 1) return GMA_ERR_INVALID_ARG;
    GMA_TRY(check_params(params));
    const bool any = dm.N > 0;
    GMA_TRY(check_ptr(x, any));
    GMA_TRY(check_ptr(gamma, any));
    GMA_TRY(check_ptr(dx, any));
    GMA_TRY(check_ptr(lengths, false));
    GMA_TRY(check_ptr(counts));
    GMA_TRY(check_ptr(dloss));
    GMA_TRY(check_ptr(dmu));
    GMA_TRY(check_ptr(dvar_raw));
    GMA_TRY(check_ptr(dlogit_pi));
    const BalPlan bp = plan_balance(dm);
    if (!ws || ws_bytes < bp.bytes) return GMA_ERR_WORKSPACE;
    GMA_TRY(check_ptr(ws));
    const size_t hk = (size_t)dm.H * dm.K, pb = hk * dm.D * 4;
    const Span sp[] = {{x, row_bytes(dm), false}, {params.mu, pb, false}, {params.var_raw, pb, false},
                       {params.logit_pi, hk * 4, false}, {lengths, (size_t)dm.B * 4, false},
                       {gamma, (size_t)dm.BH() * dm.N * dm.K * 4, false}, {counts, hk * 8, false},
                       {dloss, (size_t)dm.H * 4, false}, {dx, (size_t)dm.BH() * dm.N * dm.D * 4, true},
                       {dmu, pb, true}, {dvar_raw, pb, true}, {dlogit_pi, hk * 4, true}, {ws, bp.bytes, true}};
    GMA_TRY(check_overlap(sp, 13));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!any) {
        if (!accumulate) {
            GMA_CUDA(cudaMemsetAsync(dmu, 0, pb, st));
            GMA_CUDA(cudaMemsetAsync(dvar_raw, 0, pb, st));
            GMA_CUDA(cudaMemsetAsync(dlogit_pi, 0, hk * 4, st));
        }
        return GMA_OK;
    }
    GMA_CUDA(launch_balance_grad(dm, params, x, lengths, gamma, counts, dloss, at<float>(ws, bp.inv),
                                 at<float2>(ws, bp.terms), at<int>(ws, bp.n_terms), at<int>(ws, bp.hist),
                                 at<float>(ws, bp.part), dx, dmu, dvar_raw, dlogit_pi, accumulate != 0, st));
    return GMA_OK;
}
