// Balance loss over the mixture components, with its gradients.
//
// loss_h = K sum_k f_hk P_hk with f the share of rows whose most likely component is k and P the
// mean responsibility; the gradient flows through P.  The forward takes the responsibilities from
// the routing kernels and refines them: the routing evaluates log-joints of several hundred in
// fp32 (an error of about 1e-5, enough for the mixer), while the hard counts need the order of near
// ties and the gradients need differences of log-joints: a row's gradient goes with its posteriors
// beside the best, however small those are.  So every component whose posterior is above kKeep of the
// head's scale (the largest second-best posterior among some of its rows) is evaluated again, a few per
// row, as unevaluated sums of two fp32 values (about 2^-45 of the sum; the FP64 pipe of this GPU is far
// too slow for it).
#include "gma_operators.cuh"
#include "gma_pair.cuh"

#include <float.h>

#include <type_traits>

namespace gma {
namespace {

constexpr float kKeep = 1.220703125e-4f;   // 2^-13: below it the routing's error (1e-3 at most, of the
                                           // posterior itself) is below 2^-23 of the head's scale
constexpr int kSample = 512;               // rows of a head that set its scale
constexpr int kWarps = kThreads / 32;

// Sums of two fp32 values for two features side by side, on the packed fp32 pipe.
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.f, -1.f), a); }

// (hi, lo) + ((x - mu)^2 / sigma^2) for two features, 1/sigma^2 = ah + al.  With d = x - mu and its
// rounding error dl: w = d ah and its error, then w d and its error, and the first-order terms of dl
// and al; every error is exact (a fused multiply-add of the negated product).
__device__ __forceinline__ void add_square(float2 &hi, float2 &lo, float2 x, float2 mu, float2 ah, float2 al)
{
    const float2 d = sub2(x, mu), t = sub2(d, x);
    const float2 dl = sub2(sub2(x, sub2(d, t)), __fadd2_rn(mu, t));
    const float2 n = sub2(mu, x);   // -d
    const float2 w = __fmul2_rn(d, ah), ew = __ffma2_rn(n, ah, w);
    const float2 wl = sub2(__ffma2_rn(dl, __fadd2_rn(ah, ah), __fmul2_rn(d, al)), ew);
    const float2 h = __fmul2_rn(w, d), eh = __ffma2_rn(w, n, h);
    const float2 hl = sub2(__fmul2_rn(wl, d), eh);
    const float2 s = __fadd2_rn(hi, h), u = sub2(s, hi);
    const float2 es = __fadd2_rn(sub2(hi, sub2(s, u)), sub2(h, u));
    lo = __fadd2_rn(lo, __fadd2_rn(es, hl));
    hi = s;
}

__device__ __forceinline__ int row_len(const int *lengths, int b, int N)
{
    return lengths ? min(max(lengths[b], 0), N) : N;
}

// A posterior that is read once: not kept in L1, which holds the head's parameters.
__device__ __forceinline__ float stream(const float *p)
{
    float v;
    asm("ld.global.L1::no_allocate.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// FL consecutive features from element i (a multiple of FL).
template <int FL>
__device__ __forceinline__ void load_feats(float (&v)[FL], const void *x, long long i, bool bf16)
{
    if constexpr (FL == 4) {
        const float4 a = load4(x, i, bf16);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    } else if constexpr (FL == 2) {
        if (bf16) {
            const uint32_t u = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(x) + i);
            v[0] = __uint_as_float(u << 16), v[1] = __uint_as_float(u & 0xffff0000u);
        } else {
            const float2 a = *reinterpret_cast<const float2 *>(static_cast<const float *>(x) + i);
            v[0] = a.x, v[1] = a.y;
        }
    } else {
        v[0] = load_elem(x, i, bf16);
    }
}

// CTA -> (head, part of the head's rows), heads x parts CTAs.  The CTAs that share an SM are a whole
// wave of SMs apart; they get the same head where the heads divide the SMs, so that one copy of the
// head's parameters serves them all from L1.
struct HeadPart {
    int h, part;
    __device__ __forceinline__ HeadPart(int H, int parts)
    {
        const int per = parts < max(1, 152 / H) ? parts : max(1, 152 / H);   // a head's CTAs in a wave
        const int full = parts / per * per, bid = blockIdx.x;
        if (bid < H * full) {
            const int in = bid % (H * per);
            h = in / per;
            part = in % per + bid / (H * per) * per;
        } else {   // the parts left over
            const int in = bid - H * full;
            h = in % H;
            part = full + in / H;
        }
    }
};

// The rows of a head in steps of `step`: row t of sequence b, without a division per row (N > 0).
struct Walk {
    int b, t, db, dt, N;
    __device__ __forceinline__ Walk(long long first, long long step, int N_) : N(N_)
    {
        b = (int)(first / N), t = (int)(first - (long long)b * N);
        db = (int)(step / N), dt = (int)(step - (long long)db * N);
    }
    __device__ __forceinline__ void next()
    {
        b += db, t += dt;
        if (t >= N) t -= N, ++b;
    }
};

// Number of rows that take part: sum of the lengths (all threads of a CTA).
template <int THREADS>
__device__ __forceinline__ long long total_rows(const int *lengths, int B, int N)
{
    if (!lengths) return (long long)B * N;
    __shared__ long long part[THREADS / 32];
    long long s = 0;
    for (int b = threadIdx.x; b < B; b += THREADS) s += row_len(lengths, b, N);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) s += part[w];
    __syncthreads();
    return s;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// 1/sigma^2 and the constant logit_pi - 1/2 sum_d log sigma^2 of every component, sigma^2 =
// softplus(var_raw) = max(r, 0) + log(1 + exp(-|r|)), as two fp32 values each (log sum exp of the
// logits is common to a head's components and cancels).  A warp per component.  (In 64-bit arithmetic
// the same took 17 us for 1024 components of 64 features: the FP64 pipe is 64 times narrower.)
__global__ void __launch_bounds__(kThreads) k_bal_prep(int H, int K, int D, const float *__restrict__ var_raw,
                                                       const float *__restrict__ logit_pi, float2 *__restrict__ prec,
                                                       float2 *__restrict__ cst2, unsigned *__restrict__ second)
{
    if (blockIdx.x == 0)
        for (int h = threadIdx.x; h < H; h += kThreads) second[h] = 0;
    const int c = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (c >= H * K) return;
    float2 logs = make_float2(0.f, 0.f);
    for (int f = lane; f < D; f += 32) {
        const float r = var_raw[(long long)c * D + f];
        const float2 e = exp2v(-fabsf(r));
        // log(1 + e) = 2 atanh(e / (2 + e))
        const float2 v = add2(make_float2(fmaxf(r, 0.f), 0.f), atanh2(div2(e, add2(make_float2(2.f, 0.f), e))));
        prec[(long long)c * D + f] = div2(make_float2(1.f, 0.f), v);
        logs = add2(logs, log2v(v));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        logs = add2(logs, make_float2(__shfl_xor_sync(0xffffffffu, logs.x, o),
                                      __shfl_xor_sync(0xffffffffu, logs.y, o)));
    if (lane == 0) cst2[c] = add2(make_float2(logit_pi[c], 0.f), make_float2(-0.5f * logs.x, -0.5f * logs.y));
}

// second[h], zero before: the largest second-best posterior among kSample rows of head h, evenly spread
// (the bits of a float that is not negative: integers in the same order, so the maximum is the same in
// whatever order the CTAs come).  Rows behind a sequence have no say; where none is left every component
// is kept.  A warp per row, kWarps rows a CTA (a CTA per head with 1024 threads took 20 us).
__global__ void __launch_bounds__(kThreads)
    k_bal_scale(int B, int N, int K, int n, const int *__restrict__ lengths, const float *__restrict__ gamma,
                unsigned *__restrict__ second)
{
    __shared__ float red[kWarps];
    const int h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * kWarps + warp;
    float one = 0.f, two = 0.f;   // the lane's two largest
    if (i < n) {
        const long long r = (long long)B * N * i / n;
        const int b = (int)(r / N), t = (int)(r - (long long)b * N);
        if (t < row_len(lengths, b, N)) {
            const float *g = gamma + (((long long)b * gridDim.y + h) * N + t) * K;
            for (int k = lane; k < K; k += 32) {
                const float v = g[k];
                two = fmaxf(two, fminf(one, v));
                one = fmaxf(one, v);
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float a = __shfl_xor_sync(0xffffffffu, one, o), c = __shfl_xor_sync(0xffffffffu, two, o);
        two = fmaxf(fmaxf(two, c), fminf(one, a));
        one = fmaxf(one, a);
    }
    if (lane == 0) red[warp] = two;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kWarps; ++w) two = fmaxf(two, red[w]);
        atomicMax(second + h, __float_as_uint(two));
    }
}

// Log-joint of component c (of all heads) and the row whose features 8 e .. lie in xv: groups of GL
// lanes, each lane FP = D / GL consecutive features; every lane of the group gets the sum.
template <int D, int GL>
__device__ __forceinline__ float2 log_joint(long long c, const float (&xv)[D / GL], int l, const float *__restrict__ mu,
                                            const float2 *__restrict__ prec, float2 cst)
{
    constexpr int FP = D / GL;
    const float *m = mu + c * D + l * FP;
    const float2 *p = prec + c * D + l * FP;
    float2 hi = make_float2(0.f, 0.f), lo = hi;
#pragma unroll
    for (int f = 0; f < FP; f += 2) {
        const float2 u = *reinterpret_cast<const float2 *>(m + f);
        const float4 a = *reinterpret_cast<const float4 *>(p + f);
        add_square(hi, lo, make_float2(xv[f], xv[f + 1]), u, make_float2(a.x, a.z), make_float2(a.y, a.w));
    }
    float2 s = two_sum(hi.x, hi.y);
    s.y = __fadd_rn(s.y, __fadd_rn(lo.x, lo.y));
    s = quick_sum(s.x, s.y);
#pragma unroll
    for (int o = GL / 2; o; o >>= 1)
        s = add2(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
    return add2(cst, make_float2(-0.5f * s.x, -0.5f * s.y));
}

// Rows of one head, every `parts`-th group of kWarps rows of its B N, a warp per row: the row's
// components with posteriors above the head's bound again from their log-joints, the row's argmax, and
// the CTA's partial sums and counts.
// Lane l holds components l, l + 32, ...; the kept ones are listed in shared memory in order and
// taken four at a time, eight lanes each (a warp's sum over all lanes would cost as much as the
// terms themselves).  Bound by instructions (800 a row, most of them log-joints of about eight kept
// components): 148 us for 131072 rows of N(0, 1) at K = 128, D = 64.
template <int J, int D>
__global__ void __launch_bounds__(kThreads)
    k_bal_refine(int B, int H, int N, int K, int parts, const void *__restrict__ x, bool x_bf16,
                 const float *__restrict__ mu,
                 const float2 *__restrict__ prec, const float2 *__restrict__ cst2, const float *__restrict__ second,
                 const int *__restrict__ lengths, float *gamma, float *__restrict__ psum, int *__restrict__ pcnt)
{
    constexpr int GL = 8, FP = D / GL, E = 32 / GL;
    __shared__ int cnt[512];
    __shared__ float2 joint[kWarps][32 * J];       // log-joints of the row's kept components, by position
    __shared__ unsigned short list[kWarps][32 * J];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grp = lane / GL, l = lane % GL;
    const unsigned below = (1u << lane) - 1u;
    const HeadPart hp(H, parts);
    const int h = hp.h, part = hp.part;
    const float keep = kKeep * second[h];
    for (int k = tid; k < K; k += kThreads) cnt[k] = 0;
    __syncthreads();
    float acc[J];
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j] = 0.f;
    float next[J];   // the posteriors of the warp's next row
    long long row = 0, nrow = 0;
    bool live = false, nlive = false;
    Walk at((long long)part * kWarps + warp, (long long)parts * kWarps, N);
    auto load = [&]() {
        if (at.b >= B) return;
        nrow = ((long long)at.b * H + h) * N + at.t;
        nlive = at.t < row_len(lengths, at.b, N);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int k = lane + 32 * j;
            next[j] = nlive && k < K ? stream(gamma + nrow * K + k) : 0.f;
        }
    };
    load();
    while (at.b < B) {
        at.next();
        row = nrow, live = nlive;
        float *g = gamma + row * K;
        if (!live) {   // behind the sequence
            for (int k = lane; k < K; k += 32) g[k] = 0.f;
            load();
            continue;
        }
        float v[J];
        int pos[J];
        int nk = 0, arg = -1;
        float rest = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) v[j] = next[j];
        load();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const unsigned m = __ballot_sync(0xffffffffu, v[j] > keep);
            if (m && nk == 0) arg = 32 * j + __ffs(m) - 1;
            pos[j] = nk + __popc(m & below);
            if (v[j] > keep) list[warp][pos[j]] = (unsigned short)(32 * j + lane);
            nk += __popc(m);
            rest += v[j] > keep ? 0.f : v[j];
        }
        if (nk > 1) {   // (uniform)
            const long long xo = row * D + l * FP;
            float xv[FP];
            if constexpr (FP % 4 == 0) {
#pragma unroll
                for (int f = 0; f < FP; f += 4) {
                    const float4 a = load4(x, xo + f, x_bf16);
                    xv[f] = a.x, xv[f + 1] = a.y, xv[f + 2] = a.z, xv[f + 3] = a.w;
                }
            } else {   // d_route = 16
#pragma unroll
                for (int f = 0; f < FP; ++f) xv[f] = load_elem(x, xo + f, x_bf16);
            }
            rest = warp_sum(rest);
            __syncwarp();
            float2 best = make_float2(-INFINITY, 0.f);
            for (int e = 0; e < nk; e += E) {
                const int slot = min(e + grp, nk - 1);
                const int k = list[warp][slot];
                const long long c = (long long)h * K + k;
                const float2 s = log_joint<D, GL>(c, xv, l, mu, prec, cst2[c]);
                if (l == 0) joint[warp][slot] = s;   // (a repeated last one stores the same value)
                if (s.x > best.x || (s.x == best.x && s.y > best.y)) best = s, arg = k;
            }
            // the best of the four groups; equal ones: the lowest component
#pragma unroll
            for (int o = GL; o < 32; o <<= 1) {
                const float2 s = make_float2(__shfl_xor_sync(0xffffffffu, best.x, o),
                                             __shfl_xor_sync(0xffffffffu, best.y, o));
                const int k = __shfl_xor_sync(0xffffffffu, arg, o);
                if (s.x > best.x || (s.x == best.x && (s.y > best.y || (s.y == best.y && k < arg)))) best = s, arg = k;
            }
            __syncwarp();
            if (fabsf(best.x) < FLT_MAX) {   // else (overflow) the routing's values stay
                // a lane per kept component (not J turns of the lanes that hold them)
                float t = 0.f;
                for (int q = lane; q < nk; q += 32) {
                    const float2 d = add2(joint[warp][q], make_float2(-best.x, -best.y));   // at most 0
                    float e = expf(d.x);
                    e = fmaf(e, d.y, e);
                    joint[warp][q].x = e;
                    t += e;
                }
                t = (1.f - rest) / warp_sum(t);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (v[j] > keep) {
                        v[j] = joint[warp][pos[j]].x * t;
                        g[lane + 32 * j] = v[j];
                    }
            }
            __syncwarp();   // list and joint are used again
        }
#pragma unroll
        for (int j = 0; j < J; ++j) acc[j] += v[j];
        if (lane == 0 && arg >= 0) atomicAdd(&cnt[arg], 1);   // integers: the order does not matter
    }
#pragma unroll
    for (int j = 0; j < J; ++j) joint[warp][lane + 32 * j].x = acc[j];   // (the warp's own places)
    __syncthreads();
    const long long o = ((long long)h * parts + part) * K;
    for (int k = tid; k < K; k += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += joint[w][k].x;
        psum[o + k] = s;
        pcnt[o + k] = cnt[k];
    }
}

// A cluster of CTAs per head, 64 components each: the parts' sums, sixteen threads to a component with
// every sixteenth part (their sums meet in order), then the loss in the cluster's first CTA.  Bound by its
// chain of loads and sums (8 us at H = 8, K = 128).
constexpr int kFinal = 1024, kFinalComps = 64;
__global__ void __launch_bounds__(kFinal)
    k_bal_final(int B, int N, int K, int parts, const int *__restrict__ lengths, const float *__restrict__ psum,
                const int *__restrict__ pcnt, float *__restrict__ loss, long long *__restrict__ counts,
                float *__restrict__ prob)
{
    constexpr int GROUPS = kFinal / kFinalComps;
    __shared__ float2 redp[kFinal];
    __shared__ long long redc[kFinal];
    __shared__ double red[kFinalComps];
    __shared__ double inv_s, total;   // total: sum of f_k P_k over the CTA's components
    const int h = blockIdx.y, tid = threadIdx.x, kl = tid % kFinalComps, grp = tid / kFinalComps;
    const int k = blockIdx.x * kFinalComps + kl;
    const long long T = total_rows<kFinal>(lengths, B, N);
    if (tid == 0) inv_s = T > 0 ? 1.0 / (double)T : 0.0;
    float2 ps = make_float2(0.f, 0.f);   // (the FP64 pipe would take longer than the loads)
    long long c = 0;
    if (k < K) {
#pragma unroll 8
        for (int i = grp; i < parts; i += GROUPS) {
            const long long o = ((long long)h * parts + i) * K + k;
            ps = add2(ps, make_float2(psum[o], 0.f));
            c += pcnt[o];
        }
    }
    redp[tid] = ps;
    redc[tid] = c;
    __syncthreads();
    if (tid < kFinalComps) {
        double part = 0.0;
        if (k < K) {
            for (int q = 1; q < GROUPS; ++q)
                ps = add2(ps, redp[q * kFinalComps + tid]), c += redc[q * kFinalComps + tid];
            const double p = ((double)ps.x + (double)ps.y) * inv_s;
            counts[(long long)h * K + k] = c;
            prob[(long long)h * K + k] = (float)p;
            part = (double)c * inv_s * p;
        }
        red[tid] = part;
    }
    __syncthreads();
    if (tid < 32) {
        double part = red[tid] + red[tid + 32];
#pragma unroll
        for (int o = 16; o; o >>= 1) part += __shfl_down_sync(0xffffffffu, part, o);
        if (tid == 0) total = part;
    }
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    if (blockIdx.x == 0 && tid == 0) {
        double sum = 0.0;
        for (unsigned r = 0; r < gridDim.x; ++r) {   // in order
            uint32_t ra;
            unsigned long long v;
            asm("mapa.shared::cluster.u32 %0, %1, %2;"
                : "=r"(ra)
                : "r"((uint32_t)__cvta_generic_to_shared(&total)), "r"(r));
            asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(ra) : "memory");
            sum += __longlong_as_double((long long)v);
        }
        loss[h] = (float)((double)K * sum);
    }
    // the other CTAs' shared memory stays until the first has read it
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Gradients.

__device__ __forceinline__ float softplus(float r) { return fmaxf(r, 0.f) + log1pf(expf(-fabsf(r))); }

// Place of 1/sigma^2 of element i of [H][K][D] in `inv`, that of mu two further: pairs of features, so
// that a lane reads what it needs of two at once.
template <typename I> __device__ __forceinline__ I inv_at(I i) { return i / 2 * 4 + i % 2; }

// 1/sigma^2 and mu of every component and feature; 0 in `hist`.
__global__ void __launch_bounds__(kThreads) k_bal_inv(long long n, int D, const float *__restrict__ mu,
                                                      const float *__restrict__ var_raw, float *__restrict__ inv,
                                                      int *__restrict__ hist)
{
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i < n / D) hist[i] = 0;
    if (i >= n) return;
    inv[inv_at(i)] = 1.f / softplus(var_raw[i]);
    inv[inv_at(i) + 2] = mu[i];
}
// What may be left out of a row's terms: 2^-24 of its largest delta each with up to 128 components, less
// with more, so that all of them together stay below 128 times that (2^-24 throughout: dx off by 1.8e-6
// of its norm at d = 16 and K = 500, where hundreds of components have a share).
constexpr float kDrop = 5.9604644775390625e-8f;

// The counts of head h for k < 32 J (0 past K), in shared memory; returns dloss K / T^2, so that g_k is
// their product.  (Differences of counts are exact below 2^24; those of rounded g_k would not be.)
template <int THREADS, int J>
__device__ __forceinline__ float stage_g(float *gk, int h, int K, long long T, const long long *counts,
                                         const float *dloss)
{
    for (int k = threadIdx.x; k < 32 * J; k += THREADS) gk[k] = k < K ? (float)counts[(long long)h * K + k] : 0.f;
    const float t = (float)T;
    return T > 0 ? dloss[h] * (float)K / t / t : 0.f;
}

constexpr int kXThreads = 1024, kXWarps = kXThreads / 32;
constexpr int dx_list(int J) { return 32 * J + 4; }
// Shared memory of k_bal_dx: the lists, g, and (where it fits beside them) the head's table.
constexpr size_t dx_smem(int J, int D, bool table)
{
    return (size_t)kXWarps * dx_list(J) * 8 + 2 * 32 * J * 4 + (table ? (size_t)32 * J * D * 8 : 0);
}
constexpr bool dx_table(int J, int D) { return dx_smem(J, D, true) <= (224u << 10); }

// Rows of one head, a warp per row, one CTA per SM: the row's terms and dx.  delta_k = gamma_k ((g_k -
// g_m) - s), m the row's largest posterior and s = sum_j gamma_j (g_j - g_m), so that rows near one-hot
// keep their small differences; terms that do not count (kDrop) are left out, and the others
// (a tenth of the components on rows drawn from N(0, 1)) are listed in shared memory, so that the reads
// of four terms' parameters are in flight together, and in `terms` for the parameter sums: row i's in
// entries [i K, i K + n[i]).  Lane l holds features FL l ...
// Bound by the reads of (1/sigma^2, mu), 8 D bytes per term (the shared memory at 92 % of its rate: 74 us
// for 131072 rows at K = 128, D = 64):
// the head's table lies in shared memory (from L2 it took 205 us at K = 256, D = 64 and 13 terms a row).
template <int J, int D>
__global__ void __launch_bounds__(kXThreads)
    k_bal_dx(int B, int H, int N, int K, int parts, const void *__restrict__ x, bool x_bf16,
             const float *__restrict__ inv, const int *__restrict__ lengths, const float *__restrict__ gamma,
             const long long *__restrict__ counts, const float *__restrict__ dloss, float *dx,
             float2 *__restrict__ terms_out, int *__restrict__ n_out, int *__restrict__ hist, bool accumulate)
{
    constexpr int FL = D <= 32 ? 1 : D / 32;
    constexpr bool TABLE = dx_table(J, D);
    extern __shared__ __align__(16) float2 dyn[];
    float2 *lists = dyn;                                                     // [kXWarps][dx_list]: delta, component
    float *table = reinterpret_cast<float *>(lists + kXWarps * dx_list(J));  // [K][2 D]
    float *gk = table + (TABLE ? 64 * J * D : 0);                            // [32 J]
    int *cnt = reinterpret_cast<int *>(gk + 32 * J);                         // [32 J]: terms of a component
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y;
    const bool mine = D >= 32 || lane < D;
    const unsigned below = (1u << lane) - 1u;
    float2 *list = lists + warp * dx_list(J);
    const long long T = total_rows<kXThreads>(lengths, B, N);
    const float *invh = inv + (long long)h * K * 2 * D;
    if (TABLE) {
        for (int i = tid; i < K * D / 2; i += kXThreads)
            reinterpret_cast<float4 *>(table)[i] = reinterpret_cast<const float4 *>(invh)[i];
        invh = table;
    }
    invh += inv_at(FL * lane);
    const float scale = stage_g<kXThreads, J>(gk, h, K, T, counts, dloss), drop = kDrop * fminf(1.f, 128.f / (float)K);
    for (int k = tid; k < 32 * J; k += kXThreads) cnt[k] = 0;
    __syncthreads();
    float g[J];   // of the lane's components
#pragma unroll
    for (int j = 0; j < J; ++j) g[j] = gk[lane + 32 * j];
    float next[J], nx[FL];
    long long nrow = 0;
    bool nlive = false;
    Walk at((long long)blockIdx.x * kXWarps + warp, (long long)parts * kXWarps, N);
    auto load = [&]() {
        if (at.b >= B) return;
        nrow = ((long long)at.b * H + h) * N + at.t;
        nlive = at.t < row_len(lengths, at.b, N);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int k = lane + 32 * j;
            next[j] = nlive && k < K ? stream(gamma + nrow * K + k) : 0.f;
        }
        if (nlive && mine)
            load_feats<FL>(nx, x, nrow * D + FL * lane, x_bf16);
        else
#pragma unroll
            for (int e = 0; e < FL; ++e) nx[e] = 0.f;
    };
    load();
    while (at.b < B) {
        at.next();
        float d[J], xv[FL], top = 0.f, gl = 0.f;
        const long long row = nrow;
        const bool live = nlive;   // (uniform)
#pragma unroll
        for (int j = 0; j < J; ++j) {
            d[j] = next[j];
            if (d[j] > top) top = d[j], gl = g[j];
        }
#pragma unroll
        for (int e = 0; e < FL; ++e) xv[e] = nx[e];
        load();
        if (!live) {   // behind a sequence
            if (lane == 0) n_out[row] = 0;
            if (!accumulate && mine)
#pragma unroll
                for (int e = 0; e < FL; ++e) dx[row * D + FL * lane + e] = 0.f;
            continue;
        }
        const unsigned best = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
        const float gm =
            __shfl_sync(0xffffffffu, gl, __ffs(__ballot_sync(0xffffffffu, __float_as_uint(top) == best)) - 1);
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) s = fmaf(d[j], g[j] - gm, s);
        s = warp_sum(s);
        float big = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            d[j] = d[j] * ((g[j] - gm) - s) * scale;
            big = fmaxf(big, fabsf(d[j]));
        }
        const float cut = drop * __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
        int terms = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            // a NaN stays; lanes past K have no term (theirs is 0, but NaN beside a NaN or an infinite factor)
            const bool in = lane + 32 * j < K && !(fabsf(d[j]) <= cut);
            const unsigned m = __ballot_sync(0xffffffffu, in);
            if (in) {
                list[terms + __popc(m & below)] = make_float2(d[j], __int_as_float(lane + 32 * j));
                atomicAdd(cnt + lane + 32 * j, 1);
            }
            terms += __popc(m);
        }
        __syncwarp();
        for (int q = lane; q < terms; q += 32) terms_out[row * K + q] = list[q];
        if (lane == 0) n_out[row] = terms;
        if (lane < 4 && terms > 0) list[terms + lane] = make_float2(0.f, list[0].y);   // to whole fours
        __syncwarp();
        // sum delta (mu - x) / sigma^2, two features at a time (FL = 1: the second of a pair is idle)
        constexpr int FV = (FL + 1) / 2;
        float2 sum[FV], xp[FV];
#pragma unroll
        for (int e = 0; e < FV; ++e) {
            sum[e] = make_float2(0.f, 0.f);
            xp[e] = make_float2(xv[2 * e], FL == 1 ? 0.f : xv[(2 * e + 1) % FL]);
        }
        if (mine)
            for (int q = 0; q < terms; q += 4) {
                float2 w[4];
                float4 a[4][FV];
#pragma unroll
                for (int u = 0; u < 4; u += 2) {
                    const float4 two = *reinterpret_cast<const float4 *>(list + q + u);
                    w[u] = make_float2(two.x, two.y), w[u + 1] = make_float2(two.z, two.w);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float *src = invh + __float_as_int(w[u].y) * 2 * D;
                    if constexpr (FL == 1) {
                        a[u][0] = make_float4(src[0], 0.f, src[2], 0.f);
                    } else {
#pragma unroll
                        for (int e = 0; e < FV; ++e) a[u][e] = reinterpret_cast<const float4 *>(src)[e];
                    }
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int e = 0; e < FV; ++e) {
                        const float2 y = sub2(make_float2(a[u][e].z, a[u][e].w), xp[e]);
                        const float2 v = __fmul2_rn(make_float2(w[u].x, w[u].x), make_float2(a[u][e].x, a[u][e].y));
                        sum[e] = __ffma2_rn(v, y, sum[e]);
                    }
            }
        __syncwarp();
        if (mine)
#pragma unroll
            for (int e = 0; e < FL; ++e) {
                float *o = dx + row * D + FL * lane + e;
                const float v = e % 2 ? sum[e / 2].y : sum[e / 2].x;
                *o = accumulate ? *o + v : v;
            }
    }
    __syncthreads();   // integers: the order does not matter
    for (int k = tid; k < K; k += kXThreads)
        if (cnt[k]) atomicAdd(hist + (long long)h * K + k, cnt[k]);
}

constexpr int kGThreads = 1024, kGWarps = kGThreads / 32;
// Rows of a batch of KT components: 64, or 32 where two buffers of 64 outgrow shared memory.
constexpr int sum_rows(int KT) { return KT <= 128 ? 64 : 32; }
constexpr size_t sums_smem(int KT, int D)
{
    return (size_t)(KT * D + KT + 2 * sum_rows(KT) * (KT + D) + 2 * (sum_rows(KT) / 32) * KT) * 4;
}

// Parameter sums: components [k0, k0 + kGWarps C) of one head over every `parts`-th batch of the
// head's B N rows.  A batch's terms (from the lists of k_bal_dx) go to a tile in shared memory, each with
// a bit of its component's mask of rows; the next batch's lists and rows are on their way meanwhile.
// Then a warp takes its C components in turn, walks the rows of each one's mask in order and adds s1 =
// sum delta (x - mu) and s2 = sum delta (x - mu)^2 in registers, s0 = sum delta in shared memory: no two
// warps share a sum, so nothing depends on timing.  One barrier a batch.  The components are dealt to the
// warps there and back in the order of their terms: a batch ends with its slowest warp.  Bound by the
// instructions of the terms (105 us for 131072 rows at K = 128, D = 64).  Lane l holds features FL l ...
template <int C, int D>
__global__ void __launch_bounds__(kGThreads)
    k_bal_sums(int B, int H, int N, int K, int parts, const void *__restrict__ x, bool x_bf16,
               const float *__restrict__ mu, const int *__restrict__ lengths, const int *__restrict__ hist,
               const float2 *__restrict__ terms, const int *__restrict__ n_terms, float *__restrict__ part)
{
    constexpr int FL = D <= 32 ? 1 : D / 32, FV = (FL + 1) / 2;   // features of a lane, in pairs
    constexpr int KT = kGWarps * C, NB = sum_rows(KT), NH = NB / 32, RW = NB / kGWarps;   // RW: a warp's rows
    extern __shared__ __align__(16) float sm[];
    float *ms = sm;                                                     // [KT][D]
    float *s0 = ms + KT * D;                                            // [KT]
    float *xs = s0 + KT;                                                // [2][NB][D]
    float *ds = xs + 2 * NB * D;                                        // [2][NB][KT]
    unsigned *mask = reinterpret_cast<unsigned *>(ds + 2 * NB * KT);    // [2][NH][KT]
    __shared__ unsigned short order[KT];                                // the tile's components by falling terms
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y, p = blockIdx.x, k0 = blockIdx.z * KT;
    const bool mine = D >= 32 || lane < D;
    for (int i = tid; i < KT * D; i += kGThreads)
        ms[i] = k0 * D + i < K * D ? mu[((long long)h * K + k0) * D + i] : 0.f;
    for (int i = tid; i < 2 * NH * KT; i += kGThreads) mask[i] = 0u;
    for (int k = tid; k < KT; k += kGThreads) {
        s0[k] = 0.f;
        const int *ch = hist + (long long)h * K + k0;
        const int own = k0 + k < K ? ch[k] : -1;
        int r = 0;
#pragma unroll 8
        for (int j = 0; j < KT; ++j) {
            const int c = k0 + j < K ? ch[j] : -1;
            r += c > own || (c == own && j < k);
        }
        order[r] = (unsigned short)k;
    }
    float2 s1[C][FV], s2[C][FV];   // (FL = 1: the second of a pair is idle)
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < FV; ++e) s1[c][e] = s2[c][e] = make_float2(0.f, 0.f);
    auto pair = [&](const float *src, int e) {
        if constexpr (FL == 1)
            return make_float2(mine ? src[0] : 0.f, 0.f);
        else
            return *reinterpret_cast<const float2 *>(src + 2 * e);
    };
    const long long rows = (long long)B * N, batches = (rows + NB - 1) / NB;
    Walk at((long long)p * NB + warp * RW, (long long)parts * NB, N);   // this warp's first row
    float xv[RW][FL];
    float2 tv[RW];     // lane l: the row's term l (more than 32 are read when they are needed)
    int nt[RW];
    long long row[RW];
    auto issue = [&]() {
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            int b = at.b, t = at.t + i;
            while (t >= N) t -= N, ++b;
            const bool in = b < B && t < row_len(lengths, b, N);   // (uniform)
            row[i] = ((long long)b * H + h) * N + t;
            nt[i] = in ? n_terms[row[i]] : 0;
#pragma unroll
            for (int e = 0; e < FL; ++e) xv[i][e] = 0.f;
            if (in && mine) load_feats<FL>(xv[i], x, row[i] * D + FL * lane, x_bf16);
            // before the count is known: the entries are there, whatever they hold
            tv[i] = in && lane < K ? terms[row[i] * K + lane] : make_float2(0.f, 0.f);
        }
        at.next();
    };
    issue();
    __syncthreads();   // ms, mask, s0, order
    int buf = 0;
    for (long long bt = p; bt < batches; bt += parts, buf ^= 1) {
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int q = warp * RW + i, d0 = (buf * NB + q) * KT - k0, m0 = (buf * NH + q / 32) * KT - k0;
            const unsigned bit = 1u << (q & 31);
            for (int e = lane; e < nt[i]; e += 32) {
                const float2 v = e < 32 ? tv[i] : terms[row[i] * K + e];
                const int k = __float_as_int(v.y);
                if (k >= k0 && k < k0 + KT) {
                    ds[d0 + k] = v.x;
                    atomicOr(mask + (m0 + k), bit);
                }
            }
            if (mine)
#pragma unroll
                for (int e = 0; e < FL; ++e) xs[(buf * NB + q) * D + FL * lane + e] = xv[i][e];
        }
        __syncthreads();   // this batch is there, and the one before has been summed
        if (bt + parts < batches) issue();
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int kl = order[c * kGWarps + (c % 2 ? kGWarps - 1 - warp : warp)];
#pragma unroll
            for (int half = 0; half < NH; ++half) {
                const int mi = (buf * NH + half) * KT + kl, q0 = buf * NB + 32 * half;
                unsigned m = mask[mi];
                if (m == 0) continue;   // (uniform)
                const float *xh = xs + q0 * D + FL * lane;
                float2 u[FV];
#pragma unroll
                for (int e = 0; e < FV; ++e) u[e] = pair(ms + kl * D + FL * lane, e);
                __syncwarp();
                if (lane == 0) mask[mi] = 0u;
                float z = 0.f;
                while (m) {
                    // two rows at a time; the second may be none (a delta of 0)
                    const int q = __ffs(m) - 1;
                    m &= m - 1;
                    const int q2 = m ? __ffs(m) - 1 : q;
                    const float dq = ds[(q0 + q) * KT + kl], dq2 = m ? ds[(q0 + q2) * KT + kl] : 0.f;
                    m &= m - 1;
                    z += dq;
                    z += dq2;
#pragma unroll
                    for (int e = 0; e < FV; ++e) {
                        const float2 y = sub2(pair(xh + q * D, e), u[e]), y2 = sub2(pair(xh + q2 * D, e), u[e]);
                        const float2 w = __fmul2_rn(make_float2(dq, dq), y), w2 = __fmul2_rn(make_float2(dq2, dq2), y2);
                        s1[c][e] = __fadd2_rn(__fadd2_rn(s1[c][e], w), w2);
                        s2[c][e] = __ffma2_rn(w2, y2, __ffma2_rn(w, y, s2[c][e]));
                    }
                }
                if (lane == 0) s0[kl] += z;   // (this warp's alone)
            }
        }
    }
    // part[h][p][k]: s1, s2 (D each); behind all of those, s0[h][p][k]
    __syncwarp();
    const long long slot = (long long)h * parts + p;
    float *o = part + slot * K * 2 * D, *o0 = part + (long long)H * parts * K * 2 * D + slot * K;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int kl = order[c * kGWarps + (c % 2 ? kGWarps - 1 - warp : warp)], k = k0 + kl;
        if (k >= K) continue;
        float *ok = o + (long long)k * 2 * D;
        if (mine)
#pragma unroll
            for (int e = 0; e < FL; ++e) {
                ok[FL * lane + e] = e % 2 ? s1[c][e / 2].y : s1[c][e / 2].x;
                ok[D + FL * lane + e] = e % 2 ? s2[c][e / 2].y : s2[c][e / 2].x;
            }
        if (lane == 0) o0[k] = s0[kl];
    }
}

// The ranges' sums in order and the reparameterisation: kPGroups threads to a (component, four features),
// each every kPGroups-th range, so that few loads follow one another (7 us at H = 8, K = 128, D = 64 from
// cold caches, 15 with one thread); the last block of a head takes the mixture logits.
constexpr int kPGroups = 4, kPItems = kThreads / kPGroups;
__global__ void __launch_bounds__(kThreads)
    k_bal_params(int H, int K, int D, int parts, const float *__restrict__ part, const float *__restrict__ inv,
                 const float *__restrict__ var_raw, const float *__restrict__ logit_pi, float *dmu, float *dvar,
                 float *dlogit, bool accumulate)
{
    __shared__ float red[kThreads];
    __shared__ float sums[kPGroups][9][kPItems];
    const int h = blockIdx.y, tid = threadIdx.x, D4 = D / 4;
    const float4 *ph = reinterpret_cast<const float4 *>(part) + (long long)h * parts * K * 2 * D4;
    const float *p0 = part + (long long)H * parts * K * 2 * D + (long long)h * parts * K;
    if (blockIdx.x != gridDim.x - 1) {
        const int at = tid % kPItems, grp = tid / kPItems;
        const long long i = (long long)blockIdx.x * kPItems + at;
        const bool on = i < (long long)K * D4;
        const int k = (int)(i / D4), f = (int)(i - (long long)k * D4);
        float a[9] = {};   // s1 and s2 of the features, s0
        if (on) {
#pragma unroll 4
            for (int p = grp; p < parts; p += kPGroups) {
                const float4 *o = ph + ((long long)p * K + k) * 2 * D4 + f;
                const float4 u = o[0], v = o[D4];
                a[0] += u.x, a[1] += u.y, a[2] += u.z, a[3] += u.w;
                a[4] += v.x, a[5] += v.y, a[6] += v.z, a[7] += v.w;
                a[8] += p0[p * K + k];
            }
        }
#pragma unroll
        for (int q = 0; q < 9; ++q) sums[grp][q][at] = a[q];
        __syncthreads();
        if (!on) return;
        // feature `grp` of the four
        float s1 = 0.f, s2 = 0.f, s0 = 0.f;
#pragma unroll
        for (int g = 0; g < kPGroups; ++g) s1 += sums[g][grp][at], s2 += sums[g][4 + grp][at], s0 += sums[g][8][at];
        const long long e = (long long)h * K * D + 4 * i + grp;
        const float w = inv[inv_at(e)];
        const float m = __fmul_rn(w, s1), v = 0.5f * w * fmaf(w, s2, -s0) / (1.f + expf(-var_raw[e]));
        dmu[e] = accumulate ? dmu[e] + m : m;
        dvar[e] = accumulate ? dvar[e] + v : v;
        return;
    }
    auto reduce = [&](float v, bool max_) {
        red[tid] = v;
        __syncthreads();
        for (int s = kThreads / 2; s > 0; s >>= 1) {
            if (tid < s) red[tid] = max_ ? fmaxf(red[tid], red[tid + s]) : red[tid] + red[tid + s];
            __syncthreads();
        }
        const float r = red[0];
        __syncthreads();
        return r;
    };
    float g[2] = {0.f, 0.f}, l[2] = {-FLT_MAX, -FLT_MAX};
    for (int j = 0; j < 2; ++j) {
        const int k = tid + j * kThreads;
        if (k >= K) continue;
#pragma unroll 8
        for (int p = 0; p < parts; ++p) g[j] += p0[p * K + k];
        l[j] = logit_pi[(long long)h * K + k];
    }
    const float top = reduce(fmaxf(l[0], l[1]), true);
    float ex[2] = {0.f, 0.f};
    for (int j = 0; j < 2; ++j)
        if (tid + j * kThreads < K) ex[j] = expf(l[j] - top);
    const float se = reduce(ex[0] + ex[1], false), sg = reduce(g[0] + g[1], false);
    for (int j = 0; j < 2; ++j) {
        const int k = tid + j * kThreads;
        if (k >= K) continue;
        const float v = g[j] - ex[j] / se * sg;
        float *o = dlogit + (long long)h * K + k;
        *o = accumulate ? *o + v : v;
    }
}

// Components of a warp of the gradient sums: all of K's where their sums (2 D / 32 registers each
// and lane) fit 32 registers.
constexpr int grad_comps(int J, int D)
{
    const int fit = D <= 64 ? 8 : 512 / D;
    return J < fit ? J : fit;
}

// f(J, D) with J = the components of a lane (4, 8 or 16) and D = d_route as constants.
template <typename F>
auto by_size(int K, int D, F &&f)
{
    auto with = [&](auto j) {
        switch (D) {
        case 16: return f(j, std::integral_constant<int, 16>());
        case 32: return f(j, std::integral_constant<int, 32>());
        case 64: return f(j, std::integral_constant<int, 64>());
        default: return f(j, std::integral_constant<int, 128>());
        }
    };
    if (K <= 128) return with(std::integral_constant<int, 4>());
    if (K <= 256) return with(std::integral_constant<int, 8>());
    return with(std::integral_constant<int, 16>());
}

} // namespace

// Parts of a head's rows in the refinement (eight CTAs per SM, so that heads with more to refine spread)
// and in the gradient sums (one).
int balance_blocks(const Dims &dm)
{
    const long long groups = ((long long)dm.B * dm.N + kWarps - 1) / kWarps;
    long long parts = (8LL * 152 + dm.H - 1) / dm.H;
    if (parts > groups) parts = groups;
    return parts < 1 ? 1 : (int)parts;
}

int balance_parts(const Dims &dm)
{
    const int J = dm.K <= 128 ? 4 : dm.K <= 256 ? 8 : 16, kt = kGWarps * grad_comps(J, dm.D);
    const int tiles = (dm.K + kt - 1) / kt;
    const long long batches = ((long long)dm.B * dm.N + sum_rows(kt) - 1) / sum_rows(kt);
    long long parts = 152LL / ((long long)dm.H * tiles);   // one CTA per SM
    if (parts > batches) parts = batches;
    return parts < 1 ? 1 : (int)parts;
}

cudaError_t launch_balance_prep(const Dims &dm, const gma_params &p, float2 *prec, float2 *cst2, float *second,
                                cudaStream_t st)
{
    const int hk = dm.H * dm.K;
    k_bal_prep<<<(hk + kWarps - 1) / kWarps, kThreads, 0, st>>>(dm.H, dm.K, dm.D, p.var_raw, p.logit_pi, prec, cst2,
                                                                reinterpret_cast<unsigned *>(second));
    return cudaGetLastError();
}

cudaError_t launch_balance_loss(const Dims &dm, const gma_params &p, const void *x, const int *lengths,
                                const float2 *prec, const float2 *cst2, float *second, float *gamma, float *psum,
                                int *pcnt, float *loss, long long *counts, float *prob, cudaStream_t st)
{
    const int parts = dm.N > 0 ? balance_blocks(dm) : 0;
    if (parts > 0) {   // (the walk over the rows divides by N)
        const long long rows = (long long)dm.B * dm.N;
        const int n = rows < kSample ? (int)rows : kSample;
        k_bal_scale<<<dim3((n + kWarps - 1) / kWarps, dm.H), kThreads, 0, st>>>(
            dm.B, dm.N, dm.K, n, lengths, gamma, reinterpret_cast<unsigned *>(second));
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        e = by_size(dm.K, dm.D, [&](auto j, auto d) {
            k_bal_refine<decltype(j)::value, decltype(d)::value><<<(unsigned)(parts * dm.H), kThreads, 0, st>>>(
                dm.B, dm.H, dm.N, dm.K, parts, x, dm.x_bf16, p.mu, prec, cst2, second, lengths, gamma, psum,
                pcnt);
            return cudaGetLastError();
        });
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    const unsigned nb = (unsigned)((dm.K + kFinalComps - 1) / kFinalComps);   // at most 8: the portable cluster size
    cfg.gridDim = dim3(nb, dm.H);
    cfg.blockDim = dim3(kFinal);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = nb;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_bal_final, dm.B, dm.N, dm.K, parts, lengths, (const float *)psum,
                              (const int *)pcnt, loss, counts, prob);
}

cudaError_t launch_balance_grad(const Dims &dm, const gma_params &p, const void *x, const int *lengths,
                                const float *gamma, const long long *counts, const float *dloss, float *inv,
                                float2 *terms, int *n_terms, int *hist, float *part, float *dx, float *dmu, float *dvar,
                                float *dlogit, bool accumulate, cudaStream_t st)
{
    const long long n = (long long)dm.H * dm.K * dm.D;
    k_bal_inv<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(n, dm.D, p.mu, p.var_raw, inv, hist);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int parts = balance_parts(dm);
    e = by_size(dm.K, dm.D, [&](auto j, auto d) {
        constexpr int J = decltype(j)::value, D = decltype(d)::value, C = grad_comps(J, D), KT = kGWarps * C;
        constexpr size_t dsmem = dx_smem(J, D, dx_table(J, D));
        static std::atomic<unsigned long long> dx_set{0};
        cudaError_t a = allow_smem(k_bal_dx<J, D>, dsmem, dx_set);
        if (a != cudaSuccess) return a;
        const int xparts = (int)(152LL / dm.H > 1 ? 152LL / dm.H : 1);   // one CTA per SM
        k_bal_dx<J, D><<<dim3(xparts, dm.H), kXThreads, dsmem, st>>>(
            dm.B, dm.H, dm.N, dm.K, xparts, x, dm.x_bf16, inv, lengths, gamma, counts, dloss, dx, terms, n_terms,
            hist, accumulate);
        a = cudaGetLastError();
        if (a != cudaSuccess) return a;
        constexpr size_t smem = sums_smem(KT, D);
        static_assert(smem <= 227u << 10, "the batch fits shared memory");
        static std::atomic<unsigned long long> smem_set{0};
        a = allow_smem(k_bal_sums<C, D>, smem, smem_set);
        if (a != cudaSuccess) return a;
        k_bal_sums<C, D><<<dim3(parts, dm.H, (dm.K + KT - 1) / KT), kGThreads, smem, st>>>(
            dm.B, dm.H, dm.N, dm.K, parts, x, dm.x_bf16, p.mu, lengths, hist, terms, n_terms, part);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    static_assert(kPGroups == 4, "a thread finishes one of four features");
    const long long kd = (long long)dm.K * dm.D / 4;
    k_bal_params<<<dim3((unsigned)((kd + kPItems - 1) / kPItems) + 1u, dm.H), kThreads, 0, st>>>(
        dm.H, dm.K, dm.D, parts, part, inv, p.var_raw, p.logit_pi, dmu, dvar, dlogit, accumulate);
    return cudaGetLastError();
}

} // namespace gma
