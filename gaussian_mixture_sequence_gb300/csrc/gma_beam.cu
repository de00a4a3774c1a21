// Beam search over recurrent states: the selection of the W best continuations of every request,
// and the in-place reordering of the per-sequence states that follows it.
//
// A candidate's score is score_in + (logit - lse), lse = log sum_u exp(logit_u) of its beam.  Within
// a beam candidates rank by their logit alone, so a row of logits is read once: the same pass keeps
// a running maximum and sum per thread (for lse) and the W largest logits of the row's part.  The parts
// of each row and then the W rows of a request are joined by the first CTA of a cluster that holds all
// parts of a request, where they are few, or by a second, small kernel.
#include "gma_operators.cuh"
#include "gma_pair.cuh"

#include <cooperative_groups.h>
#include <float.h>

namespace cg = cooperative_groups;

namespace gma {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kVecs = 4;                     // 16-byte vectors of a thread and step
constexpr int kMaxParts = 32;                // parts of a row, at most
constexpr int kKeys = 64;                    // keys of a row's parts, at most, for two or more parts
constexpr int kCap = 1024;                   // candidates held before they are ranked
constexpr int kWarps = kThreads / 32;
constexpr int kLonger = 4;                   // steps of a part of a cluster, where the plan has fewer
constexpr int kCluster = 16;                 // parts of a request that a cluster takes, at most

using u64 = unsigned long long;

__device__ __forceinline__ float ex2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Orders fp32 values as unsigned integers; 0 for -infinity (no candidate).
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 counts as +0
    return x == -INFINITY ? 0u : (u & 0x80000000u ? ~u : u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// Larger keys first: the larger logit, then the lower token.
__device__ __forceinline__ u64 key_of(float x, int token) { return ((u64)ordered(x) << 32) | (uint32_t)~token; }

__device__ __forceinline__ u64 warp_max(u64 v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const u64 w = __shfl_xor_sync(0xffffffffu, v, o);
        v = w > v ? w : v;
    }
    return v;
}

struct BeamWs {
    u64 *keys;      // [rows][parts][W]: falling
    float *top;     // [rows][parts]: largest logit of the part
    float2 *sums;   // [rows][parts]: sum of exp(logit - top), two fp32 values
    // from part i on, W keys a part
    __device__ BeamWs from(long long i, int W) const { return {keys + i * W, top + i, sums + i}; }
};

struct BeamIo {   // of the selection, all requests
    const float *score_in;
    const unsigned char *finished_in;
    float *score_out;
    int *parent, *token;
    unsigned char *finished_out;
};

struct BeamPlan {
    bool cluster;       // a request's parts make a cluster: no workspace
    int parts, steps;   // parts of a row, steps of a part
    size_t keys, top, sums, bytes;
};

// A 32-bit word of logits: one fp32 or two bf16.
__device__ __forceinline__ void logits_of(uint32_t w, float (&x)[1]) { x[0] = __uint_as_float(w); }
__device__ __forceinline__ void logits_of(uint32_t w, float (&x)[2])
{
    x[0] = __uint_as_float(w << 16);
    x[1] = __uint_as_float(w & 0xffff0000u);
}
// The largest of 4 kVecs words' logits, NaN apart (-infinity where nothing else is left).
__device__ __forceinline__ float largest(const uint32_t (&w)[4 * kVecs], float (&)[1])
{
    float t = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4 * kVecs; ++i) t = fmaxf(t, __uint_as_float(w[i]));
    return t;
}
__device__ __forceinline__ float largest(const uint32_t (&w)[4 * kVecs], float (&)[2])
{
    __nv_bfloat162 m = __floats2bfloat162_rn(-INFINITY, -INFINITY);
#pragma unroll
    for (int i = 0; i < 4 * kVecs; ++i) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
    return fmaxf(__low2float(m), __high2float(m));
}

// Ranks the n candidates of `buf` and leaves the W largest, falling, in `best`.
__device__ __forceinline__ void rank_into(const u64 *buf, int n, int W, u64 *best)
{
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const u64 k = buf[i];
        int r = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) r += buf[j] > k;
        if (r < W) best[r] = k;
    }
}

// One part of one row, part `q`: `steps` steps of kStep logits.  Its results go to `out` (of this part).
//
// Bound by HBM (each logit once) with about ten instructions per logit beside it (the conversion, a
// maximum, a difference, an exponential and a sum, and what passes the threshold) and the barriers of its
// groups: 512 rows of 131072 bf16 in 34 us, 4.0 TB/s.  A thread's kE-logit maximum is compared
// with the threshold.  The threshold is the W-th largest logit of the steps before, so that after the
// first step few logits pass; they are pushed into shared memory, without a barrier, and ranked at the
// end of a group of steps.  The first step is a group of its own, with a threshold from its own
// threads' maxima; each later group is as long as all before it (about W pushes), within what the
// buffer holds four times over.  A group that overflows it all the same (rising rows, many equal
// logits) is read again and its best are taken one by one.
//
// ALIGNED: every row starts on a 16-byte boundary.  Which tokens a thread takes does not depend on
// how a row is aligned, so that equal rows get equal sums to the last bit (beams tie when they share
// their history): other rows are read as the two aligned vectors around each token vector.
template <typename T, bool ALIGNED, typename DONE>
__device__ __forceinline__ void beam_part(int W, int V, int ld, int steps, const T *logits, long long row, int q,
                                          const BeamWs &out, DONE done)
{
    constexpr int PW = 4 / (int)sizeof(T), VEC = 4 * PW;          // logits of a word, of a vector
    constexpr int kE = kVecs * VEC, kStep = kThreads * kE;         // of a thread and step, of a CTA and step
    __shared__ u64 buf[kCap];
    __shared__ u64 best[kMaxBeams];
    __shared__ u64 wred[kWarps];
    __shared__ float wthr[kWarps];
    __shared__ float2 wsum[kWarps];
    __shared__ int count[3];   // candidates of a group; the group after next reuses a counter
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long start = row * ld;
    const int off = ALIGNED ? 0 : (int)(start & (VEC - 1));
    const T *base = logits + start;
    const long long first = (long long)q * steps * kStep;
    const int mine = (int)min((long long)steps, (V - first + kStep - 1) / kStep);   // the part's steps in the row
    if (tid < W) best[tid] = 0;
    if (tid < 3) count[tid] = 0;
    __syncthreads();

    // logit e of this thread and step
    auto token = [&](int step, int e) {
        return (int)(first + (long long)step * kStep) + ((e / VEC) * kThreads + tid) * VEC + e % VEC;
    };
    struct Raw {
        uint32_t w[4 * kVecs];
    };
    // vector q of a thread, its first aligned half at `a`
    auto vector = [&](Raw &r, int q, const uint4 *a) {
        const uint4 lo = __ldcs(a);
        r.w[4 * q] = lo.x, r.w[4 * q + 1] = lo.y, r.w[4 * q + 2] = lo.z, r.w[4 * q + 3] = lo.w;
        if (!ALIGNED && off != 0) {
            const uint4 hi = a[1];
            const uint32_t c[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            const int bits = off * (int)sizeof(T) * 8, sh = bits & 31;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (bits >> 5 == k)   // uniform: the shift in whole words
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        r.w[4 * q + e] = __funnelshift_r(c[e + k], e + k + 1 < 8 ? c[e + k + 1] : 0u, sh);
        }
    };
    auto fetch = [&](int step) {
        Raw r;
        const int u0 = (int)(first + (long long)step * kStep), u1 = u0 + tid * VEC;
        if ((long long)u0 + kStep + 2 * VEC <= V) {   // (uniform) no vector reaches behind the row
#pragma unroll
            for (int q = 0; q < kVecs; ++q)
                vector(r, q, reinterpret_cast<const uint4 *>(base + (u1 - off)) + q * kThreads);
        } else {   // the row's end: -infinity behind it, its last vectors one logit at a time
#pragma unroll
            for (int q = 0; q < kVecs; ++q) {
                const int u = u1 + q * kThreads * VEC;
#pragma unroll
                for (int e = 0; e < 4; ++e) r.w[4 * q + e] = PW == 1 ? 0xff800000u : 0xff80ff80u;
                if (u + 2 * VEC <= V) {
                    vector(r, q, reinterpret_cast<const uint4 *>(base + (u - off)));
                    continue;
                }
                for (int e = 0; e < 4; ++e) {
                    const int v = u + e * PW;
                    if (v >= V) break;
                    uint32_t w;
                    if (PW == 1) {
                        w = reinterpret_cast<const uint32_t *>(base)[v];
                    } else {
                        const uint16_t *h = reinterpret_cast<const uint16_t *>(base);
                        w = h[v] | (v + 1 < V ? (uint32_t)h[v + 1] : 0xff80u) << 16;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i == e) r.w[4 * q + i] = w;
                }
            }
        }
        return r;
    };

    float m = -INFINITY, s = 0.f;   // this thread's running maximum and sum of exp(x - m)
    float thr = -FLT_MAX;           // candidates are at least this (-infinity: masked)
    const int group = max(1, kCap / 4 / W);
    Raw next = fetch(0);
    for (int g0 = 0, gi = 0; g0 < mine; ++gi) {
        const int g1 = min(mine, g0 == 0 ? 1 : g0 + min(g0, group));
        for (int step = g0; step < g1; ++step) {
            const Raw cur = next;
            if (step + 1 < mine) next = fetch(step + 1);
            float x[PW];
            const float t = largest(cur.w, x);
            const float nm = fmaxf(m, t);
            if (nm == INFINITY) {   // the infinite logits share the probability
                if (m != INFINITY) s = 0.f;
#pragma unroll
                for (int i = 0; i < 4 * kVecs; ++i) {
                    logits_of(cur.w[i], x);
#pragma unroll
                    for (int e = 0; e < PW; ++e) s += x[e] == INFINITY ? 1.f : 0.f;
                }
            } else if (nm > -INFINITY) {
                // x - nm first: folding nm into a multiply-add would round at the size of the logits
                const float2 sh = make_float2(-nm, -nm), l2 = make_float2(kLog2e, kLog2e);
                float2 p = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 4 * kVecs; i += 2 / PW) {
                    float2 v;
                    if (PW == 1) {
                        const int i1 = i + 1 < 4 * kVecs ? i + 1 : i;
                        v = make_float2(__uint_as_float(cur.w[i]), __uint_as_float(cur.w[i1]));
                    } else {
                        v = make_float2(__uint_as_float(cur.w[i] << 16), __uint_as_float(cur.w[i] & 0xffff0000u));
                    }
                    const float2 d = __fmul2_rn(__fadd2_rn(v, sh), l2);
                    p = __fadd2_rn(p, make_float2(ex2_approx(d.x), ex2_approx(d.y)));
                }
                float ps = p.x + p.y;
                if (ps != ps) {   // a NaN among the logits: masked tokens
                    ps = 0.f;
#pragma unroll
                    for (int i = 0; i < 4 * kVecs; ++i) {
                        logits_of(cur.w[i], x);
#pragma unroll
                        for (int e = 0; e < PW; ++e)
                            if (x[e] == x[e]) ps += ex2_approx((x[e] - nm) * kLog2e);
                    }
                }
                s = (m == nm ? s : s * ex2_approx((m - nm) * kLog2e)) + ps;
            }
            m = nm;
            if (step == 0) {
                // a first threshold: each warp's W-th largest thread maximum has W logits at or above it
                uint32_t cur_k = ordered(t), low = 0;
                for (int i = 0; i < W; ++i) {
                    low = __reduce_max_sync(0xffffffffu, cur_k);
                    if (cur_k == low) cur_k = 0;
                    if (low == 0) break;
                }
                if (lane == 0) wthr[warp] = low ? unordered(low) : -FLT_MAX;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kWarps; ++i) thr = fmaxf(thr, wthr[i]);
            }
            if (t >= thr) {
                unsigned over = 0;
#pragma unroll
                for (int i = 0; i < 4 * kVecs; ++i) {
                    logits_of(cur.w[i], x);
#pragma unroll
                    for (int e = 0; e < PW; ++e) over |= x[e] >= thr ? 1u << (i * PW + e) : 0u;
                }
                for (; over; over &= over - 1) {   // few: read again rather than picked out of registers
                    const int tok = token(step, __ffs(over) - 1);
                    const int at = atomicAdd(&count[gi % 3], 1);
                    if (at < kCap - kMaxBeams) buf[at] = key_of(load_elem(base, tok, PW == 2), tok);
                }
            }
        }
        // the counter of the next group: every thread read it two groups ago, before the last barrier
        if (tid == 0) count[(gi + 1) % 3] = 0;
        __syncthreads();
        const int n = count[gi % 3];
        if (n > 0 && n <= kCap - kMaxBeams) {   // (uniform)
            if (tid < W) buf[n + tid] = best[tid];
            __syncthreads();
            // empty places of `best` hold 0 and rank last; equal zeros share a rank
            rank_into(buf, n + W, W, best);
        } else if (n > 0) {
            for (int step = g0; step < g1; ++step) {
                u64 last = ~0ull;
                __syncthreads();
                if (tid < W) buf[tid] = best[tid];
                __syncthreads();
                for (int i = 0; i < W; ++i) {
                    u64 k = tid < W && buf[tid] < last ? buf[tid] : 0;
#pragma unroll 1
                    for (int e = 0; e < kE; ++e) {   // (from the caches: no registers held for this path)
                        const int tok = token(step, e);
                        const float v = tok < V ? load_elem(base, tok, PW == 2) : -INFINITY;
                        if (v >= thr) {
                            const u64 c = key_of(v, tok);
                            if (c < last && c > k) k = c;
                        }
                    }
                    k = warp_max(k);
                    if (lane == 0) wred[warp] = k;
                    __syncthreads();
                    k = 0;
#pragma unroll
                    for (int j = 0; j < kWarps; ++j) k = wred[j] > k ? wred[j] : k;
                    if (tid == 0) best[i] = k;
                    last = k;
                    __syncthreads();
                    if (k == 0) break;   // (uniform) the places left were 0 before: fewer than W in all
                }
            }
        }
        __syncthreads();
        const uint32_t worst = (uint32_t)(best[W - 1] >> 32);
        thr = worst ? unordered(worst) : thr;
        g0 = g1;
    }
    done();
    // the part's maximum, and the sums relative to it
    float mm = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    if (lane == 0) wthr[warp] = mm;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) mm = fmaxf(mm, wthr[i]);
    float2 v = make_float2(0.f, 0.f);
    if (mm == INFINITY)
        v.x = m == INFINITY ? s : 0.f;
    else if (m > -INFINITY)
        v.x = s * ex2_approx((m - mm) * kLog2e);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    if (lane == 0) wsum[warp] = v;
    __syncthreads();
    if (tid == 0) {
        v = wsum[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) v = add2(v, wsum[i]);
        *out.sums = v;
        *out.top = mm;
    }
    if (tid < W) out.keys[tid] = best[tid];
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 4)
    k_beam_part(int W, int V, int ld, int steps, const T *logits, BeamWs ws)
{
    const long long row = blockIdx.y;
    beam_part<T, ALIGNED>(W, V, ld, steps, logits, row, blockIdx.x, ws.from(row * gridDim.x + blockIdx.x, W), [] {
        // the join may be launched now; it waits for this grid's results before it reads them
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    });
}

// Orders 64-bit values as unsigned integers (-0 as +0; never a NaN here).
__device__ __forceinline__ u64 ordered64(double x)
{
    const u64 u = (u64)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | (1ull << 63);
}

// One request, by one CTA: the W rows' parts to W candidates each, then the W best of all rows.  Both
// joins rank every candidate against every other, in parallel: W rounds of a warp-wide maximum would
// be as many times a chain of ten shuffles.  Bound by its chain of loads, barriers and sums (6.8 us for
// 64 requests of 8 beams, 8.0 with FP64 exponentials and logarithms); the FP64
// pipe takes 16 cycles for an instruction of any warp, however few lanes it has, so comparisons are of
// integers, and exponentials and logarithms of sums of two fp32 values.  MW: beams, MP: parts of a row,
// KEYS: keys of a row.
template <int MW, int MP, int KEYS>
__device__ __forceinline__ void beam_join(int W, int parts, int eos, int pad, long long b, const BeamWs &ws,
                                          const BeamIo &io)
{
    __shared__ u64 pool[MW * KEYS];     // the rows' keys; then all candidates' scores
    __shared__ u64 list[MW][MW];        // a row's W best, falling
    __shared__ float2 sums[MW][MP];
    __shared__ float ptop[MW][MP];
    __shared__ double add[MW];          // score_in - log sum exp(logit - top); a finished beam: its score
    __shared__ float tops[MW];
    __shared__ unsigned char fin[MW], live[MW];
    static_assert(KEYS >= MW, "every candidate's score fits the pool");
    constexpr int EACH = (MW * MP + kThreads - 1) / kThreads;   // parts of a thread
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int np = W * parts, n = parts * W, total = W * n;   // parts of the request, keys of a row, of all
    for (int i = tid; i < total; i += kThreads) pool[i] = ws.keys[i];
    for (int i = tid; i < W * W; i += kThreads) list[i / W][i % W] = 0;
    float2 part[EACH];
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        const int i = tid + j * kThreads;
        if (i < np) {
            part[j] = ws.sums[i];
            ptop[i / parts][i % parts] = ws.top[i];
        }
    }
    float sc = 0.f;
    if (tid < W) {
        sc = io.score_in[b * W + tid];
        fin[tid] = io.finished_in && io.finished_in[b * W + tid];
        live[tid] = sc > -INFINITY;   // false for NaN too
    }
    __syncthreads();
    if (tid < W) {
        float m = -INFINITY;
        for (int q = 0; q < parts; ++q) m = fmaxf(m, ptop[tid][q]);
        tops[tid] = m;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        const int i = tid + j * kThreads;
        if (i < np) {
            const float m = tops[i / parts], top = ptop[i / parts][i % parts];
            float2 s = make_float2(0.f, 0.f);
            if (top > -INFINITY && (m < INFINITY || top == INFINITY)) {
                s = part[j];
                if (top < m) {   // below exp(-80) a part leaves no trace in a sum of at least 1
                    const float2 d = two_sum(top, -m);
                    const float2 e = d.x > -80.f ? exp2v(d.x) : make_float2(0.f, 0.f);
                    const float p = s.x * e.x;
                    s = quick_sum(p, fmaf(s.x, e.x, -p) + fmaf(s.x, e.y, s.y * e.x) + (p > 0.f ? p * d.y : 0.f));
                }
            }
            sums[i / parts][i % parts] = s;
        }
    }
    // the rows' best; a finished beam has the padding token alone, and in a row with infinite logits
    // only those are candidates
    for (int i = tid; i < total; i += kThreads) {
        const int w = i / n;
        const u64 *row = pool + w * n, k = pool[i];
        const u64 least = tops[w] == INFINITY ? (u64)ordered(INFINITY) << 32 : 1;
        if (fin[w] || !live[w] || k < least) continue;
        int r = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) r += row[j] > k;
        if (r < W) list[w][r] = k;
    }
    __syncthreads();
    if (tid < W) {
        float2 s = make_float2(0.f, 0.f);
        for (int q = 0; q < parts; ++q) s = add2(s, sums[tid][q]);
        const bool plain = fin[tid] || tops[tid] == -INFINITY;
        const float2 l = log2v(s);
        add[tid] = plain ? (double)sc : ((double)sc - (double)l.x) - (double)l.y;
        if (fin[tid] && live[tid]) list[tid][0] = ~(u64)0;
    }
    __syncthreads();
    // every candidate's score, then its place: better scores and equal ones of lower beams (or, in its
    // own beam, earlier in the list) come first
    u64 *score = pool;
    const int nc = W * W;
    auto value = [&](int i) {
        const int w = i / W;
        const u64 k = list[w][i - w * W];
        if (fin[w]) return add[w];
        const float x = unordered((uint32_t)(k >> 32));
        return x == INFINITY ? add[w] : add[w] + ((double)x - (double)tops[w]);   // the difference is exact
    };
    for (int i = tid; i < nc; i += kThreads) score[i] = list[i / W][i % W] ? ordered64(value(i)) : 0;
    __syncthreads();
    int found = 0;
    for (int i = tid; i < nc; i += kThreads) {
        const u64 k = score[i];
        if (k == 0) continue;
        int r = 0;
#pragma unroll 4
        for (int j = 0; j < nc; ++j) r += score[j] > k || (score[j] == k && j < i);
        if (r >= W) continue;
        const int w = i / W;
        const long long o = b * W + r;
        const int tok = fin[w] ? pad : (int)~(uint32_t)list[w][i - w * W];
        io.score_out[o] = (float)value(i);
        io.parent[o] = w;
        io.token[o] = tok;
        if (io.finished_out) io.finished_out[o] = fin[w] || tok == eos;
    }
    // the slots past the last candidate
    for (int i = lane; i < nc; i += 32) found += score[i] != 0;
    if (warp != 0) return;
#pragma unroll
    for (int o = 16; o; o >>= 1) found += __shfl_xor_sync(0xffffffffu, found, o);
    for (int i = found + lane; i < W; i += 32) {
        const long long o = b * W + i;
        io.score_out[o] = -INFINITY;
        io.parent[o] = i;
        io.token[o] = pad;
        if (io.finished_out) io.finished_out[o] = 1;
    }
}

__global__ void __launch_bounds__(kThreads)
    k_beam_join(int W, int parts, int eos, int pad, BeamWs ws, BeamIo io)
{
    const long long b = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the parts' kernel has finished
    beam_join<kMaxBeams, kMaxParts, kKeys>(W, parts, eos, pad, b, ws.from(b * W * parts, W), io);
}

// All parts of a request in one cluster, W x parts CTAs: the parts' results go to the first CTA's shared
// memory, which joins them.  One launch and no workspace, for calls that the host cannot issue as fast as
// the GPU runs them: four beams over 32,000 tokens take 9 us of the host instead of 20, and 8.0 us of the
// GPU instead of 7.4; 16 requests of 8 beams over 50,000 tokens 16.7 of the GPU instead of 14.8.  Larger
// calls keep the two kernels, whose CTAs need not wait for one another (32 requests of 5 beams: 17.0 us of
// the GPU against 20.6; 64 of 16: 49 against 68).
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 4)
    k_beam_cluster(int W, int V, int ld, int steps, int parts, int eos, int pad, const T *logits, BeamIo io)
{
    __shared__ u64 keys[kCluster * kCluster];
    __shared__ float2 sums[kCluster];
    __shared__ float top[kCluster];
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = blockIdx.x;
    const long long b = blockIdx.y;
    const BeamWs first{cluster.map_shared_rank(keys, 0), cluster.map_shared_rank(top, 0),
                       cluster.map_shared_rank(sums, 0)};
    cluster.barrier_arrive();
    // every CTA of the cluster has started before the first one's memory is written
    beam_part<T, ALIGNED>(W, V, ld, steps, logits, b * W + rank / parts, rank % parts, first.from(rank, W),
                          [&] { cluster.barrier_wait(); });
    cluster.sync();
    if (rank == 0) beam_join<kCluster, kCluster, kCluster>(W, parts, eos, pad, b, BeamWs{keys, top, sums}, io);
}

BeamPlan beam_plan(const BeamDims &bd)
{
    BeamPlan p;
    const long long step = (long long)kThreads * kVecs * (bd.bf16 ? 8 : 4);
    const long long rows = (long long)bd.B * bd.W, steps = (bd.V + step - 1) / step;
    long long parts = 4LL * 152 / rows;   // one turn of four CTAs per SM: a part costs about as much as three steps
    if (parts < 1) parts = 1;
    // joining n keys takes n^2 comparisons a row: one request of 8 beams over 131,072 fp32 logits took 38 us
    // in 32 parts of a step and takes 13 in 8 parts of 4
    if (parts > kKeys / bd.W) parts = kKeys / bd.W;
    if (parts > kMaxParts) parts = kMaxParts;
    if (parts > steps) parts = steps;
    p.steps = (int)((steps + parts - 1) / parts);
    // one cluster per request, where its parts are few and short enough
    const long long most = kCluster / bd.W < parts ? kCluster / bd.W : parts;
    const long long longer = most > 0 ? (steps + most - 1) / most : 0;
    p.cluster = most > 0 && longer <= kLonger && rows * most <= 2 * 152;
    if (p.cluster) p.steps = (int)longer;
    p.parts = (int)((steps + p.steps - 1) / p.steps);
    if (p.cluster) {
        p.keys = p.top = p.sums = p.bytes = 0;
        return p;
    }
    p.keys = 0;
    p.top = (size_t)round_up(rows * p.parts * bd.W * 8, 256);
    p.sums = p.top + (size_t)round_up(rows * p.parts * 4, 256);
    p.bytes = p.sums + (size_t)round_up(rows * p.parts * 8, 256);
    return p;
}

// Every beam of one request at one place of its state: all values that move are read before the
// first is written, and a place belongs to one thread, so the exchange needs no second buffer.  Bound by
// HBM (a beam that moves is read once and written once).  The stores leave L2 first, as nothing here reads
// them again: 32 requests of 8 states of 520 KB with uniform parents took 35.2 us with plain stores and take
// 31.3 (6.4 TB/s).
template <typename Wd, int WM>
__global__ void __launch_bounds__(kThreads) k_beam_reorder(int W, long long words, const int *parent, Wd *state)
{
    __shared__ int from[kMaxBeams];
    const int tid = threadIdx.x;
    const long long b = blockIdx.y;
    if (tid < W) {
        const int p = parent[b * W + tid];
        from[tid] = p >= 0 && p < W ? p : tid;
    }
    __syncthreads();
    Wd *s = state + b * W * words;
    const long long i = (long long)blockIdx.x * kThreads + tid;
    if (i >= words) return;
    Wd v[WM];
#pragma unroll
    for (int w = 0; w < WM; ++w)
        if (w < W && from[w] != w) v[w] = s[from[w] * words + i];
#pragma unroll
    for (int w = 0; w < WM; ++w)
        if (w < W && from[w] != w) __stcs(&s[w * words + i], v[w]);
}

template <typename Wd>
cudaError_t launch_reorder(int B, int W, long long words, const int *parent, void *state, cudaStream_t st)
{
    const dim3 grid((unsigned)((words + kThreads - 1) / kThreads), (unsigned)B);
    Wd *s = static_cast<Wd *>(state);
    if (W <= 8)
        k_beam_reorder<Wd, 8><<<grid, kThreads, 0, st>>>(W, words, parent, s);
    else if (W <= 16)
        k_beam_reorder<Wd, 16><<<grid, kThreads, 0, st>>>(W, words, parent, s);
    else
        k_beam_reorder<Wd, 32><<<grid, kThreads, 0, st>>>(W, words, parent, s);
    return cudaGetLastError();
}

} // namespace

size_t beam_ws_bytes(const BeamDims &bd) { return beam_plan(bd).bytes; }

cudaError_t launch_beam_select(const BeamDims &bd, const void *logits, const float *score_in,
                               const unsigned char *finished_in, float *score_out, int *parent, int *token,
                               unsigned char *finished_out, void *ws, cudaStream_t st)
{
    const BeamPlan p = beam_plan(bd);
    const BeamIo io{score_in, finished_in, score_out, parent, token, finished_out};
    const bool aligned = bd.ld % (bd.bf16 ? 8 : 4) == 0;
    const __nv_bfloat16 *lh = static_cast<const __nv_bfloat16 *>(logits);
    const float *lf = static_cast<const float *>(logits);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (p.cluster) {
        cfg.gridDim = dim3((unsigned)(bd.W * p.parts), (unsigned)bd.B);
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)(bd.W * p.parts);
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        auto go = [&](auto kern, const auto *l) {
            if (bd.W * p.parts > 8) {   // above the portable size
                const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
                if (e != cudaSuccess) return e;
            }
            return cudaLaunchKernelEx(&cfg, kern, bd.W, bd.V, bd.ld, p.steps, p.parts, bd.eos, bd.pad, l, io);
        };
        if (bd.bf16)
            return aligned ? go(k_beam_cluster<__nv_bfloat16, true>, lh) : go(k_beam_cluster<__nv_bfloat16, false>, lh);
        return aligned ? go(k_beam_cluster<float, true>, lf) : go(k_beam_cluster<float, false>, lf);
    }
    char *w = static_cast<char *>(ws);
    const BeamWs bw{reinterpret_cast<u64 *>(w + p.keys), reinterpret_cast<float *>(w + p.top),
                    reinterpret_cast<float2 *>(w + p.sums)};
    const dim3 grid((unsigned)p.parts, (unsigned)(bd.B * bd.W));
    auto part = [&](auto kern, const auto *l) { kern<<<grid, kThreads, 0, st>>>(bd.W, bd.V, bd.ld, p.steps, l, bw); };
    if (bd.bf16)
        aligned ? part(k_beam_part<__nv_bfloat16, true>, lh) : part(k_beam_part<__nv_bfloat16, false>, lh);
    else
        aligned ? part(k_beam_part<float, true>, lf) : part(k_beam_part<float, false>, lf);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)bd.B);
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, k_beam_join, bd.W, p.parts, bd.eos, bd.pad, bw, io);
}

cudaError_t launch_beam_reorder(int B, int W, size_t row_bytes, const int *parent, void *state, cudaStream_t st)
{
    if (row_bytes % 16 == 0) return launch_reorder<uint4>(B, W, (long long)(row_bytes / 16), parent, state, st);
    return launch_reorder<uint32_t>(B, W, (long long)(row_bytes / 4), parent, state, st);
}

} // namespace gma
