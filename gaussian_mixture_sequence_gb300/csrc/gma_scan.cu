// Gated linear recurrence: h_t = a_t h_{t-1} + u_t per channel, a = sigmoid(gate),
// u = x or (1 - a) x, with its gradients and its one-token step.
//
// The data-dependent decay gates are those the linear-attention page ("선형 어텐션
// 원리 정리") lists beside the ungated memory; the arithmetic is fp32 throughout and
// each result is rounded once when it is stored.
//
// The recurrence composes: over rows i..j, h_j = A h_{i-1} + U with A the product of the
// a_t and U the recurrence started at 0, and (A2, U2) after (A1, U1) is (A2 A1, A2 U1 + U2).
// The gradient runs the same composition backwards in time: c_t = a_t (dout_t + c_{t+1})
// is what lambda_t = dout_t + c_{t+1} hands to the row before.
#include "gma_operators.cuh"
#include "gma_tc.cuh"

#include <type_traits>

namespace gma {
namespace {

__device__ __forceinline__ float ex2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b)   // NaN where either is
{
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a = sigmoid(g) and r = 1 - a = sigmoid(-g).  With e = exp(-g): a = 1 / (1 + e), r = e a,
// which keeps the relative accuracy of both ends (1 - a would lose r for large gates) but for
// the rounding of g log2 e, about |g| units of 2^-24 on the smaller of the two.  The exponent
// is held below 125 powers of two, where 1 / (1 + e) is still a normal number; a NaN gate stays
// NaN.
__device__ __forceinline__ void gate_of(float g, float &a, float &r)
{
    const float e = ex2_approx(min_nan(g * -1.4426950408889634f, 125.f));
    a = rcp_approx(1.f + e);
    r = e * a;
}

// One or two channels of a thread: two go through the packed fp32 instructions.
__device__ __forceinline__ float vset(float, float c) { return c; }
__device__ __forceinline__ float2 vset(float2, float c) { return make_float2(c, c); }
__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float2 vmul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float vadd(float a, float b) { return a + b; }
__device__ __forceinline__ float2 vadd(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 vfma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ void vgate(float g, float &a, float &r) { gate_of(g, a, r); }
__device__ __forceinline__ void vgate(float2 g, float2 &a, float2 &r)
{
    const float2 t = __fmul2_rn(g, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    const float2 e = make_float2(ex2_approx(min_nan(t.x, 125.f)), ex2_approx(min_nan(t.y, 125.f)));
    const float2 s = __fadd2_rn(e, make_float2(1.f, 1.f));
    a = make_float2(rcp_approx(s.x), rcp_approx(s.y));
    r = __fmul2_rn(e, a);
}
__device__ __forceinline__ void unpack(uint32_t w, float &v) { v = __uint_as_float(w); }
__device__ __forceinline__ void unpack(uint32_t w, float2 &v)
{
    v = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t pack(float2 v)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ int slice_len(const int *lengths, int b, int N)
{
    return lengths ? min(max(lengths[b], 0), N) : N;
}

// V consecutive channels of one row as stored, and their values.
template <typename T, int V> struct Word;
template <> struct Word<float, 1> {
    using raw = uint32_t;
    static __device__ __forceinline__ void get(raw w, float (&v)[1]) { v[0] = __uint_as_float(w); }
    static __device__ __forceinline__ raw put(const float (&v)[1]) { return __float_as_uint(v[0]); }
};
template <> struct Word<__nv_bfloat16, 2> {
    using raw = uint32_t;
    static __device__ __forceinline__ void get(raw w, float (&v)[2])
    {
        v[0] = __uint_as_float(w << 16);
        v[1] = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ raw put(const float (&v)[2])
    {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[0], v[1]);
        return *reinterpret_cast<const raw *>(&p);
    }
};
template <> struct Word<__nv_bfloat16, 1> {
    using raw = uint16_t;
    static __device__ __forceinline__ void get(raw w, float (&v)[1]) { v[0] = bf16_bits_to_f32(w); }
    static __device__ __forceinline__ raw put(const float (&v)[1])
    {
        const __nv_bfloat16 p = __float2bfloat16_rn(v[0]);
        return *reinterpret_cast<const raw *>(&p);
    }
};

// Copies one word to the thread's own place in shared memory without waiting for it; a 2-byte
// word is below what an asynchronous copy can move and goes through a register.
__device__ __forceinline__ void fetch(uint32_t *dst, const uint32_t *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void fetch(uint16_t *dst, const uint16_t *src) { *dst = *src; }
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING> __device__ __forceinline__ void fetch_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Stores v at this CTA's address p in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster(float2 *p, uint32_t rank, float2 v)
{
    uint32_t ra;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(ra), "f"(v.x), "f"(v.y) : "memory");
}

struct ScanArgs {
    int H, N, D, LW, G;   // LW words of a row per CTA, G runs of R rows per tile
    const void *x, *gate, *out_in, *dout;
    const int *lengths;
    const float *first;   // state_in (forward) or dstate_out (backward)
    const float *state_in;
    void *out, *dx, *dgate;
    float *last;          // state_out or dstate_in
};

constexpr int kScanCluster = 16;   // CTAs of a cluster along time, at most

// One slice's columns [LW V words] per cluster of C CTAs.  A tile is G R consecutive rows: thread
// (run, word) owns R rows of V channels.  The CTAs of the cluster take consecutive tiles; a round is
// C tiles.  Every thread fetches its own words STAGES - 1 rounds ahead into its own places of shared
// memory (no barrier guards them), composes its R rows to (A, U), and the runs' and then the CTAs'
// (A, U) meet in shared memory, where every thread reads the ones before its own: one CTA barrier
// and one cluster barrier a round, on double-buffered slots.  Then a second sweep over the rows in
// registers applies the carried value.  Every input byte is read once, and the result does not
// depend on timing: all compositions run in a fixed order.
//
// For rows that TMA cannot take.  Bound by the instructions of single words and by the cluster barrier of a
// round: 96 x 5650 x 78 fp32 (half of the rows behind their sequences) 83 us, 41 of HBM.
template <typename T, int V, int R, bool MEAN, bool BWD, int STAGES>
__global__ void __launch_bounds__(kThreads) k_scan_tile(const ScanArgs p)
{
    using W = Word<T, V>;
    using raw = typename W::raw;
    constexpr int NIN = BWD ? (MEAN ? 4 : 3) : 2;
    extern __shared__ __align__(16) unsigned char smem[];
    float2 *agg = reinterpret_cast<float2 *>(smem);                // [2][V][kThreads]: (A, U) of the runs
    float2 *tot = agg + 2 * V * kThreads;                          // [2][kScanCluster][V][32]: of the CTAs
    raw *stage = reinterpret_cast<raw *>(tot + 2 * kScanCluster * V * 32);   // [STAGES][NIN][R][kThreads]
    const int tid = threadIdx.x, run = tid / p.LW, w = tid - run * p.LW;
    const int C = (int)(gridDim.x / ((p.D + p.LW * V - 1) / (p.LW * V)));
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const int col = ((int)(blockIdx.x / C) * p.LW + w) * V, s = blockIdx.y;
    const bool on = run < p.G && col < p.D;
    const int n = slice_len(p.lengths, s / p.H, p.N);
    const int tile = p.G * R, round = tile * C, rounds = (n + round - 1) / round;
    const long long base = (long long)s * p.N * p.D + col;   // element of row 0
    const long long cell = (long long)s * p.D + col;
    const int k0 = rank * tile + run * R;                     // this thread's first position of round 0
    if (C > 1) cluster_sync();                                // every CTA's shared memory is there

    float carry[V], h0[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        carry[v] = on && p.first ? p.first[cell + v] : 0.f;
        h0[v] = BWD && on && p.state_in ? p.state_in[cell + v] : 0.f;
    }

    auto place = [&](int st, int in, int i) { return stage + ((st * NIN + in) * R + i) * kThreads + tid; };
    // position k of the walk is row k, or n - 1 - k backwards in time
    auto issue = [&](int r) {
        const int st = r % STAGES;
        if (on && r < rounds) {
            const int k = r * round + k0;
            long long e = base + (long long)(BWD ? n - 1 - k : k) * p.D;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (k + i < n) {
                    fetch(place(st, 0, i), reinterpret_cast<const raw *>(static_cast<const T *>(p.gate) + e));
                    if (BWD) {
                        fetch(place(st, 1, i), reinterpret_cast<const raw *>(static_cast<const T *>(p.dout) + e));
                        if (k + i < n - 1)   // row 0 has the first state before it
                            fetch(place(st, 2, i),
                                  reinterpret_cast<const raw *>(static_cast<const T *>(p.out_in) + e - p.D));
                        if (MEAN)
                            fetch(place(st, NIN - 1, i),
                                  reinterpret_cast<const raw *>(static_cast<const T *>(p.x) + e));
                    } else {
                        fetch(place(st, 1, i), reinterpret_cast<const raw *>(static_cast<const T *>(p.x) + e));
                    }
                }
                e += BWD ? -(long long)p.D : (long long)p.D;
            }
        }
        fetch_commit();
    };
#pragma unroll
    for (int r = 0; r < STAGES - 1; ++r) issue(r);

    for (int r = 0; r < rounds; ++r) {
        const int st = r % STAGES, par = r & 1;
        const int k = r * round + k0;
        issue(r + STAGES - 1);   // into the places of round r - 1, which this thread has finished with
        fetch_wait<STAGES - 1>();
        float a[R][V], b[R][V];   // forward: a and u; backward: a and 1 - a
        float A[V], U[V];
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 1.f, U[v] = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const bool live = on && k + i < n;
            float g[V], y[V];
            W::get(live ? *place(st, 0, i) : raw(0), g);
            W::get(live ? *place(st, 1, i) : raw(0), y);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float av, rv;
                gate_of(g[v], av, rv);
                const float u = BWD ? av * y[v] : (MEAN ? rv * y[v] : y[v]);
                a[i][v] = live ? av : 1.f;   // a row behind the sequence changes nothing
                b[i][v] = BWD ? rv : u;
                U[v] = fmaf(a[i][v], U[v], live ? u : 0.f);
                A[v] *= a[i][v];
                if (!BWD && !live) b[i][v] = 0.f;
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) agg[(par * V + v) * kThreads + tid] = make_float2(A[v], U[v]);
        __syncthreads();
        // the runs before this one, then the whole CTA
        float pa[V], pu[V], ta[V], tu[V];
#pragma unroll
        for (int v = 0; v < V; ++v) pa[v] = ta[v] = 1.f, pu[v] = tu[v] = 0.f;
        for (int j = 0; j < p.G; ++j) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (j == run) pa[v] = ta[v], pu[v] = tu[v];
                const float2 m = agg[(par * V + v) * kThreads + j * p.LW + w];
                tu[v] = fmaf(m.x, tu[v], m.y);
                ta[v] *= m.x;
            }
        }
        float in[V];
        if (C > 1) {
            if (run == 0)
                for (int q = 0; q < C; ++q)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        st_cluster(tot + ((par * kScanCluster + rank) * V + v) * 32 + w, (uint32_t)q,
                                   make_float2(ta[v], tu[v]));
            cluster_sync();
            for (int q = 0; q < C; ++q) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (q == rank) in[v] = carry[v];
                    const float2 m = tot[((par * kScanCluster + q) * V + v) * 32 + w];
                    carry[v] = fmaf(m.x, carry[v], m.y);
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                in[v] = carry[v];
                carry[v] = fmaf(ta[v], carry[v], tu[v]);
            }
        }
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(pa[v], in[v], pu[v]);
        if (on) {
            long long e = base + (long long)(BWD ? n - 1 - k : k) * p.D;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (k + i < n) {
                    if (!BWD) {
#pragma unroll
                        for (int v = 0; v < V; ++v) h[v] = fmaf(a[i][v], h[v], b[i][v]);
                        *reinterpret_cast<raw *>(static_cast<T *>(p.out) + e) = W::put(h);
                    } else {
                        float y[V], hp[V], xv[V], ox[V], og[V];
                        W::get(*place(st, 1, i), y);
                        if (k + i < n - 1) {
                            W::get(*place(st, 2, i), hp);
                        } else {
#pragma unroll
                            for (int v = 0; v < V; ++v) hp[v] = h0[v];
                        }
                        if (MEAN) W::get(*place(st, NIN - 1, i), xv);
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            const float lam = y[v] + h[v];
                            h[v] = a[i][v] * lam;
                            ox[v] = MEAN ? lam * b[i][v] : lam;
                            og[v] = (MEAN ? hp[v] - xv[v] : hp[v]) * (h[v] * b[i][v]);
                        }
                        *reinterpret_cast<raw *>(static_cast<T *>(p.dx) + e) = W::put(ox);
                        *reinterpret_cast<raw *>(static_cast<T *>(p.dgate) + e) = W::put(og);
                    }
                }
                e += BWD ? -(long long)p.D : (long long)p.D;
            }
        }
    }
    if (BWD && on) {   // rows behind the sequence: no gradient
        for (int t = n + rank * p.G + run; t < p.N; t += C * p.G) {
            const float zero[V] = {};
            const long long e = base + (long long)t * p.D;
            *reinterpret_cast<raw *>(static_cast<T *>(p.dx) + e) = W::put(zero);
            *reinterpret_cast<raw *>(static_cast<T *>(p.dgate) + e) = W::put(zero);
        }
    }
    if (p.last && on && run == 0 && rank == 0)
#pragma unroll
        for (int v = 0; v < V; ++v) p.last[cell + v] = carry[v];
}

// The same for rows of a multiple of 16 bytes: tiles come by TMA, a word of 4 bytes (one fp32 or two
// bf16 channels) per thread and row, and the CTAs of a cluster hand their tile's (A, U) to one another
// by asynchronous stores that complete on the receivers' barriers, so that no fence and no barrier of
// the whole cluster stands in a round.
//
// Bound by HBM: 3 words per element pair forward, 5 or 6 backward.  What takes the time before that
// is instructions, hence the tiles by TMA (no per-word addresses or predicates), the packed
// arithmetic, and R rows per thread between two exchanges.  16 x 65536 x 128 bf16 forward: 147 us, 5.5 TB/s
// (81 % of what a copy reaches); 32 x 4096 x 64 fp32 forward and backward: 54 us, 5.6 TB/s.
template <typename T> using Chan = typename std::conditional<std::is_same<T, float>::value, float, float2>::type;

// Slots of the exchange: (A, U) of one or two channels, 8 or 16 bytes.
__device__ __forceinline__ float2 slot_of(float a, float u) { return make_float2(a, u); }
__device__ __forceinline__ float4 slot_of(float2 a, float2 u) { return make_float4(a.x, a.y, u.x, u.y); }
__device__ __forceinline__ void slot_get(float2 s, float &a, float &u) { a = s.x, u = s.y; }
__device__ __forceinline__ void slot_get(float4 s, float2 &a, float2 &u)
{
    a = make_float2(s.x, s.y), u = make_float2(s.z, s.w);
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank)
{
    uint32_t ra;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(addr), "r"(rank));
    return ra;
}
// Stores v in the shared memory of CTA `rank` at this CTA's address `dst`, counted on its barrier `bar`.
__device__ __forceinline__ void st_async(uint32_t dst, uint32_t bar, uint32_t rank, float2 v)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(
                     map_rank(dst, rank)),
                 "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(map_rank(bar, rank))
                 : "memory");
}
__device__ __forceinline__ void st_async(uint32_t dst, uint32_t bar, uint32_t rank, float4 v)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                     map_rank(dst, rank)),
                 "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)),
                 "r"(__float_as_uint(v.w)), "r"(map_rank(bar, rank))
                 : "memory");
}

__device__ __forceinline__ void unpack_state(const float *p, float &v) { v = *p; }
__device__ __forceinline__ void unpack_state(const float *p, float2 &v) { v = *reinterpret_cast<const float2 *>(p); }
__device__ __forceinline__ void pack_state(float *p, float v) { *p = v; }
__device__ __forceinline__ void pack_state(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }

struct ScanMaps {
    CUtensorMap m[4];   // gate, x (forward) or dout, out, x (backward): [slices][N][D], boxes of LW words
};

// FULL: LW = 32, known to the compiler (rows of 128 bytes: shared-memory offsets are constants).
template <typename T, int R, bool MEAN, bool BWD, int STAGES, bool FULL>
__global__ void __launch_bounds__(kThreads, 2)
    k_scan_tma(const __grid_constant__ ScanMaps maps, const ScanArgs p, int box_rows, unsigned int *flag)
{
    using namespace tc;
    using F = Chan<T>;
    using Slot = typename std::conditional<std::is_same<T, float>::value, float2, float4>::type;
    constexpr int V = sizeof(F) / 4, NIN = BWD ? (MEAN ? 4 : 3) : 2;
    extern __shared__ __align__(128) unsigned char smem[];
    const int LW = FULL ? 32 : p.LW, G = FULL ? kThreads / 32 : p.G;
    const int tid = threadIdx.x, run = tid / LW, w = tid - run * LW;
    const int tile = G * R;
    const uint32_t in_bytes = (uint32_t)round_up((long long)tile * LW * 4, 128);
    unsigned char *stage = smem;                                            // [STAGES][NIN][tile][LW words]
    Slot *agg = reinterpret_cast<Slot *>(stage + (size_t)STAGES * NIN * in_bytes);   // [2][kThreads]
    const int C = (int)(gridDim.x / ((p.D + LW * V - 1) / (LW * V)));
    Slot *tot = agg + 2 * kThreads;                                                  // [2][C][LW]
    unsigned long long *bars = reinterpret_cast<unsigned long long *>(tot + 2 * C * LW);
    const uint32_t full = smem_addr(bars), xbar = full + 8 * STAGES;   // [STAGES] loads, [2] exchanges
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const int col0 = (int)(blockIdx.x / C) * LW * V, col = col0 + w * V, s = blockIdx.y;
    const bool on = run < G && col < p.D;
    const int n = slice_len(p.lengths, s / p.H, p.N);
    const int round = tile * C, rounds = (n + round - 1) / round;
    const long long base = (long long)s * p.N * p.D + col;   // element of row 0
    const long long cell = (long long)s * p.D + col;
    if (tid == 0) {
        for (int i = 0; i < STAGES + 2; ++i) mbar_init(full + 8 * i, 1);
        mbar_init_fence();
    }
    __syncthreads();
    if (C > 1) cluster_sync();   // every CTA's barriers are there (and starting together is worth 2 %)
    bool bad = false;      // a bounded wait expired: nothing more is waited for or issued
    unsigned armed = 0, phase = 0;   // thread 0: stages with loads not yet waited for, and their parities

    // tile q of the walk starts at position q tile; position k is row k, or n - 1 - k backwards
    auto issue = [&](int r) {
        const int k = (r * C + rank) * tile;
        if (tid != 0 || bad || r >= rounds || k >= n) return;
        const int st = r % STAGES, row = BWD ? n - k - tile : k;
        const uint32_t bar = full + 8 * st;
        armed |= 1u << st;
        phase = (phase & ~(1u << st)) | ((unsigned)(r / STAGES) & 1u) << st;
        mbar_expect_tx(bar, (uint32_t)(NIN * tile * LW * 4));
#pragma unroll
        for (int in = 0; in < NIN; ++in)
            for (int b = 0; b < tile; b += box_rows)
                tma_load_3d(smem_addr(stage) + (st * NIN + in) * in_bytes + b * LW * 4, &maps.m[in], col0,
                            row + b - (BWD && in == 2 ? 1 : 0), s, bar);
    };
    for (int r = 0; r < STAGES; ++r) issue(r);

    F carry = vset(F(), 0.f), h0 = carry;
    if (on && p.first) unpack_state(p.first + cell, carry);
    if (BWD && on && p.state_in) unpack_state(p.state_in + cell, h0);
    if (C > 1 && p.last && p.last == p.first) cluster_sync();   // in place: all have read before one writes

    for (int r = 0; r < rounds; ++r) {
        const int st = r % STAGES, par = r & 1;
        const int kt = (r * C + rank) * tile, k = kt + run * R;
        const uint32_t *in0 = reinterpret_cast<const uint32_t *>(stage + (size_t)st * NIN * in_bytes);
        // this thread's first row of the tile in shared memory, and the step to its next
        const int at = (BWD ? tile - 1 - run * R : run * R) * LW + w, step = BWD ? -LW : LW;
        const uint32_t in_words = in_bytes / 4;
        F a[R], b[R], A = vset(F(), 1.f), U = vset(F(), 0.f);   // b: u (forward) or 1 - a (backward)
        auto sweep = [&](auto whole) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const bool live = decltype(whole)::value || (on && k + i < n);
                F g, y, av, rv, u;
                unpack(live ? in0[at + i * step] : 0u, g);
                unpack(live ? in0[in_words + at + i * step] : 0u, y);
                vgate(g, av, rv);
                u = BWD ? vmul(av, y) : (MEAN ? vmul(rv, y) : y);
                a[i] = live ? av : vset(F(), 1.f);   // a row behind the sequence changes nothing
                u = live ? u : vset(F(), 0.f);
                b[i] = BWD ? rv : u;
                U = vfma(a[i], U, u);
                A = vmul(A, a[i]);
            }
        };
        const bool whole = kt + tile <= n && run < G;   // (all but idle threads agree)
        if (kt < n) {
            if (!bad && !mbar_wait(full + 8 * st, (uint32_t)(r / STAGES) & 1u)) bad = true;
            if (tid == 0 && !bad) armed &= ~(1u << st);
        }
        if (whole)
            sweep(std::true_type());
        else
            sweep(std::false_type());
        agg[par * kThreads + tid] = slot_of(A, U);
        __syncthreads();
        // the stage that every thread has finished with: this round's, or the last one's where the
        // second sweep reads shared memory again
        if (!BWD)
            issue(r + STAGES);
        else if (r > 0)
            issue(r - 1 + STAGES);
        // the runs before this one; the whole tile where it is needed
        F ta = vset(F(), 1.f), tu = vset(F(), 0.f);
        auto join = [&](int j) {
            F ma, mu;
            slot_get(agg[par * kThreads + j * LW + w], ma, mu);
            tu = vfma(ma, tu, mu);
            ta = vmul(ta, ma);
        };
        F pa, pu;
        if (FULL) {   // a warp is a run
#pragma unroll 4
            for (int j = 0; j < run; ++j) join(j);
            pa = ta, pu = tu;
            if (C == 1 || run == 0)
#pragma unroll 4
                for (int j = run; j < G; ++j) join(j);
        } else {
            pa = ta, pu = tu;
            for (int j = 0; j < G; ++j) {
                if (j == run) pa = ta, pu = tu;
                join(j);
            }
        }
        F in = carry;
        if (C > 1) {
            const uint32_t bar = xbar + 8 * par;
            if (tid == 0) mbar_expect_tx(bar, (uint32_t)(C * LW * sizeof(Slot)));
            if (run == 0) {
                const uint32_t dst = smem_addr(tot + (par * C + rank) * LW + w);
                for (int q = 0; q < C; ++q) st_async(dst, bar, (uint32_t)q, slot_of(ta, tu));
            }
            if (!bad && !mbar_wait(bar, (uint32_t)(r >> 1) & 1u)) bad = true;
            auto after = [&](int q) {
                F ma, mu;
                slot_get(tot[(par * C + q) * LW + w], ma, mu);
                carry = vfma(ma, carry, mu);
            };
#pragma unroll 4
            for (int q = 0; q < rank; ++q) after(q);
            in = carry;
#pragma unroll 4
            for (int q = rank; q < C; ++q) after(q);
        } else {
            carry = vfma(ta, carry, tu);
        }
        F h = vfma(pa, in, pu);
        if (bad) h = vset(F(), __uint_as_float(0x7fffffffu));
        auto finish = [&](auto whole) {
            // the tile's base is the CTA's; a thread's offset within the tile fits 32 bits
            const long long e0 = ((long long)s * p.N + (BWD ? n - kt - tile : kt)) * p.D + col0;
            char *o = static_cast<char *>(BWD ? p.dx : p.out) + e0 * (long long)sizeof(T);
            char *og = static_cast<char *>(p.dgate) + e0 * (long long)sizeof(T);
            const uint32_t de = (uint32_t)p.D * (uint32_t)sizeof(T);
            uint32_t off = (uint32_t)(BWD ? tile - 1 - run * R : run * R) * de + (uint32_t)w * 4u;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (decltype(whole)::value || (on && k + i < n)) {
                    if (!BWD) {
                        h = vfma(a[i], h, b[i]);
                        *reinterpret_cast<uint32_t *>(o + off) = pack(h);
                    } else {
                        F y, hp, xv;
                        unpack(in0[in_words + at + i * step], y);
                        unpack(in0[2 * in_words + at + i * step], hp);
                        if (k + i == n - 1) hp = h0;   // before row 0: the first state
                        const F lam = vadd(y, h);
                        h = vmul(a[i], lam);
                        if (MEAN) {
                            unpack(in0[(NIN - 1) * in_words + at + i * step], xv);
                            hp = vfma(xv, vset(F(), -1.f), hp);
                        }
                        *reinterpret_cast<uint32_t *>(o + off) = pack(MEAN ? vmul(lam, b[i]) : lam);
                        *reinterpret_cast<uint32_t *>(og + off) = pack(vmul(hp, vmul(h, b[i])));
                    }
                }
                off += BWD ? 0u - de : de;
            }
        };
        if (whole && col < p.D)
            finish(std::true_type());
        else
            finish(std::false_type());
    }
    if (BWD && on) {   // rows behind the sequence: no gradient
        for (int t = n + rank * G + run; t < p.N; t += C * G) {
            const long long e = base + (long long)t * p.D;
            *reinterpret_cast<uint32_t *>(static_cast<T *>(p.dx) + e) = 0u;
            *reinterpret_cast<uint32_t *>(static_cast<T *>(p.dgate) + e) = 0u;
        }
    }
    if (p.last && on && run == 0 && rank == 0) pack_state(p.last + cell, carry);
    if (bad) {   // the loads still in flight, again for a bounded time
        if (tid == 0)
            for (int st = 0; st < STAGES; ++st)
                if (armed >> st & 1) mbar_wait(full + 8 * st, phase >> st & 1u);
        report_timeout(flag);
    }
    if (C > 1) cluster_sync();   // nobody's shared memory goes while another may still write to it
}

// One token of every sequence, a thread per channel: bound by the launch (256 x 16 x 64 fp32: 5.2 MB in
// 1.7 us).
__global__ void __launch_bounds__(kThreads)
    k_scan_step(long long n, bool mean, bool bf16, const void *x, const void *gate, float *state, void *out)
{
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    float a, r;
    gate_of(load_elem(gate, i, bf16), a, r);
    const float v = load_elem(x, i, bf16);
    const float h = fmaf(a, state[i], mean ? r * v : v);
    state[i] = h;
    store_elem(out, i, h, bf16);
}

// A launch of `cols` column blocks x C CTAs of a cluster along time x S slices.
template <typename Kern, typename... Args>
cudaError_t launch_clusters(Kern kern, int cols, int C, int S, size_t smem, std::atomic<unsigned long long> &wide_set,
                            cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(cols * C), (unsigned)S);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    if (C > 1) {
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if (C > 8) {   // beyond the portable size: allowed once per kernel and device
            int dev = 0;
            cudaError_t e = cudaGetDevice(&dev);
            if (e != cudaSuccess) return e;
            const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
            if (!(bit && (wide_set.load(std::memory_order_relaxed) & bit))) {
                e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
                if (e != cudaSuccess) return e;
                if (bit) wide_set.fetch_or(bit, std::memory_order_relaxed);
            }
        }
    }
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// CTAs along time, with a tile each: as many as find a place on the GPU at `per_sm`
// CTAs per SM beside the other columns (more would wait for a second turn), and past the portable
// cluster size of 8 only where each gets an SM of its own (the exchange's slots outgrow the room for
// two, and clusters of 16 pack badly) or `wide`, three and more fit one (4 x 58972 x 99 fp32 forward: 172
// us in clusters of 8, 130 in 16; backward, two to an SM, 310 and 355).  A padded batch takes twice as
// many: its short sequences end early and make room, and the long ones, which set the time, run in fewer
// rounds (8 x 8 x 4001 x 72 bf16, lengths uniform: 37.6 us with as many, 32.7 with twice, 39.0 with four
// times as many).  Between 8 and 16 clusters leave places of a GPC empty (16 x 65536 x 128 bf16: 149 us in
// clusters of 8, 213 in 9); below, a size serves that the GPU has room for all at once, as it says (16 x
// 8192 x 155 fp32 backward: 153 us in clusters of 3, 205 in 2).
template <typename FIT>
int time_ctas(long long columns, int per_sm, bool wide, long long tiles, bool ragged, FIT fit)
{
    const int turns = ragged ? 2 : 1;
    const long long sms = sm_count(), places = sms * per_sm * turns;
    const long long most = places / columns < tiles ? places / columns : tiles;
    if (most >= kScanCluster && columns * kScanCluster <= (wide ? places : sms)) return kScanCluster;
    int C = most < 1 ? 1 : most > 8 ? 8 : (int)most;
    while ((C & (C - 1)) && (long long)fit(C) * turns < columns) --C;
    return C;
}

// Clusters of C CTAs that the GPU runs at once, asked once and kept in `known`.
template <typename Kern> int clusters_at_once(Kern kern, int C, size_t smem, std::atomic<int> &known)
{
    int n = known.load(std::memory_order_relaxed);
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;   // (not known: a power of two)
    }
    known.store(n, std::memory_order_relaxed);
    return n;
}

template <typename T, int V, int R, bool MEAN, bool BWD, int STAGES>
cudaError_t launch_tile(const ScanDims &sd, ScanArgs a, cudaStream_t st)
{
    auto kern = k_scan_tile<T, V, R, MEAN, BWD, STAGES>;
    constexpr int NIN = BWD ? (MEAN ? 4 : 3) : 2;
    constexpr size_t smem = (size_t)2 * V * kThreads * 8 + (size_t)2 * kScanCluster * V * 32 * 8 +
                            (size_t)STAGES * NIN * R * kThreads * sizeof(typename Word<T, V>::raw);
    static std::atomic<unsigned long long> smem_set{0}, wide_set{0};
    cudaError_t e = allow_smem(kern, smem, smem_set);
    if (e != cudaSuccess) return e;
    // words of a row over the column blocks evenly, eight at least (so at most 32 runs a tile)
    const int words = (sd.D + V - 1) / V, blocks = (words + 31) / 32;
    a.LW = (words + blocks - 1) / blocks;
    if (a.LW < 8) a.LW = 8;
    a.G = kThreads / a.LW;
    const int cols = (sd.D + a.LW * V - 1) / (a.LW * V);
    const int per_sm = (int)(232448 / (smem + 1024) < 4 ? 232448 / (smem + 1024) : 4);
    const long long tiles = ((long long)sd.N + a.G * R - 1) / (a.G * R);
    const int C = time_ctas((long long)cols * sd.S, per_sm, per_sm >= 3, tiles, a.lengths != nullptr, [&](int c) {
        static std::atomic<int> known[9];
        return clusters_at_once(kern, c, smem, known[c]);
    });
    return launch_clusters(kern, cols, C, sd.S, smem, wide_set, st, (const ScanArgs)a);
}

// Rows of whole 16-byte units and at least eight words (the TMA box of a tile's row).
bool scan_tma_applies(const ScanDims &sd)
{
    const int bytes = sd.D * (sd.bf16 ? 2 : 4);
    return bytes % 16 == 0 && bytes >= 32;
}

// TMA boxes of a tile: at most 256 rows each, whole, and each on a 128-byte boundary (a row is a multiple
// of 16 bytes); 0 where there is no such division.
int tile_boxes(int tile)
{
    for (int n = (tile + 255) / 256; n <= 4; ++n)
        if (tile % n == 0 && (n == 1 || tile / n % 8 == 0)) return n;
    return 0;
}
constexpr size_t kScanSmem = 160 << 10;   // two CTAs per SM take up to 113 KB each, clusters of 16 more

template <typename T, int R, bool MEAN, bool BWD, int STAGES, bool FULL>
cudaError_t launch_tma_lw(const ScanDims &sd, const ScanArgs &a, cudaStream_t st)
{
    auto kern = k_scan_tma<T, R, MEAN, BWD, STAGES, FULL>;
    constexpr int V = std::is_same<T, float>::value ? 1 : 2, NIN = BWD ? (MEAN ? 4 : 3) : 2;
    const int words = sd.D / V;
    const int cols = (words + a.LW - 1) / a.LW, tile = a.G * R;
    const size_t in_bytes = (size_t)round_up((long long)tile * a.LW * 4, 128);
    const long long tiles = ((long long)sd.N + tile - 1) / tile;
    static std::atomic<unsigned long long> smem_set{0}, wide_set{0};
    const cudaError_t e = allow_smem(kern, kScanSmem, smem_set);
    if (e != cudaSuccess) return e;
    auto bytes = [&](int c) {
        return STAGES * NIN * in_bytes + (2 * kThreads + 2 * c * a.LW) * 8 * V + 8 * (STAGES + 2);
    };
    const int C = time_ctas((long long)cols * sd.S, 2, false, tiles, a.lengths != nullptr, [&](int c) {
        static std::atomic<int> known[17][9];   // (LW is a multiple of 4, 64 at most)
        return clusters_at_once(kern, c, bytes(c), known[a.LW / 4][c]);
    });
    const size_t smem = bytes(C);
    const int boxes = tile_boxes(tile), box_rows = boxes ? tile / boxes : 0;
    if (smem > kScanSmem || boxes == 0) return cudaErrorInvalidValue;
    ScanMaps maps = {};
    const void *src[4] = {a.gate, BWD ? a.dout : a.x, a.out_in, a.x};
    for (int i = 0; i < NIN; ++i)
        if (!make_tma_rows(&maps.m[i], src[i], sd.bf16, (unsigned long long)sd.D, (unsigned long long)sd.N,
                           (unsigned long long)sd.S, (unsigned)(a.LW * V), (unsigned)box_rows))
            return cudaErrorInvalidValue;
    unsigned int *flag = timeout_flag_dev();
    if (!flag) return cudaErrorMemoryAllocation;
    return launch_clusters(kern, cols, C, sd.S, smem, wide_set, st, (const ScanMaps)maps, (const ScanArgs)a, box_rows,
                           flag);
}

// R, the rows of a thread between two exchanges, is as large as registers and shared memory allow for
// two CTAs per SM: the exchange is what a round costs besides its bytes (scan of 65536 x 128 bf16: 228
// us at 8 rows, 176 at 12, 161 at 16, 150 at 20; three CTAs per SM at 10 rows: 204).  RF: rows of whole
// 128-byte blocks; R otherwise (2 x 65536 x 248 bf16 forward: 149 us at 16 rows, 134 at 20; backward of
// 4 x 30000 x 24 fp32: 50 at 8, 41 at 12).
template <typename T, int RF, int R, bool MEAN, bool BWD, int STAGES>
cudaError_t launch_tma(const ScanDims &sd, ScanArgs a, cudaStream_t st)
{
    constexpr int V = std::is_same<T, float>::value ? 1 : 2;
    // words of a row over the column blocks: 128-byte blocks where they come out even, else blocks of
    // up to 64 words (of two channels 56: beyond, one CTA per SM has room) evenly, in whole 16-byte units
    constexpr int most = V == 1 ? 64 : 56;
    const int words = sd.D / V, blocks = words % 32 == 0 ? words / 32 : (words + most - 1) / most;
    a.LW = (int)round_up((words + blocks - 1) / blocks, 4);
    a.G = kThreads / a.LW;
    while (a.LW != 32 && tile_boxes(a.G * R) == 0) --a.G;   // (20 of 21 runs)
    return a.LW == 32 ? launch_tma_lw<T, RF, MEAN, BWD, STAGES, true>(sd, a, st)
                      : launch_tma_lw<T, R, MEAN, BWD, STAGES, false>(sd, a, st);
}

// Rows of words go R rows a thread too, in two stages: 12 forward and 8 backward keep enough CTAs on an SM
// (4 x 58972 x 99 fp32 backward: 416 us with three stages of 8, 386 with two of 12, 312 with two of 8).
template <bool BWD>
cudaError_t launch_any(const ScanDims &sd, const ScanArgs &a, cudaStream_t st)
{
    using b16 = __nv_bfloat16;
    constexpr int RT = BWD ? 8 : 12, R = BWD ? 12 : 20, R4 = BWD ? 12 : 24, R2 = BWD ? 12 : 20;
    if (scan_tma_applies(sd)) {
        if (!sd.bf16)
            return sd.mean ? launch_tma<float, R4, R, true, BWD, 2>(sd, a, st)
                           : launch_tma<float, R4, R, false, BWD, 2>(sd, a, st);
        return sd.mean ? launch_tma<b16, R2, R, true, BWD, 2>(sd, a, st)
                       : launch_tma<b16, R2, R, false, BWD, 2>(sd, a, st);
    }
    if (!sd.bf16)
        return sd.mean ? launch_tile<float, 1, RT, true, BWD, 2>(sd, a, st)
                       : launch_tile<float, 1, RT, false, BWD, 2>(sd, a, st);
    if (sd.D % 2 == 0)
        return sd.mean ? launch_tile<b16, 2, RT, true, BWD, 2>(sd, a, st)
                       : launch_tile<b16, 2, RT, false, BWD, 2>(sd, a, st);
    return sd.mean ? launch_tile<b16, 1, RT, true, BWD, 2>(sd, a, st)
                   : launch_tile<b16, 1, RT, false, BWD, 2>(sd, a, st);
}

} // namespace

cudaError_t launch_scan_fwd(const ScanDims &sd, const void *x, const void *gate, const int *lengths,
                            const float *state_in, float *state_out, void *out, cudaStream_t st)
{
    ScanArgs a = {};
    a.H = sd.H, a.N = sd.N, a.D = sd.D;
    a.x = x, a.gate = gate, a.lengths = lengths, a.first = state_in, a.out = out, a.last = state_out;
    return launch_any<false>(sd, a, st);
}

cudaError_t launch_scan_bwd(const ScanDims &sd, const void *x, const void *gate, const void *out, const void *dout,
                            const int *lengths, const float *state_in, const float *dstate_out, void *dx, void *dgate,
                            float *dstate_in, cudaStream_t st)
{
    ScanArgs a = {};
    a.H = sd.H, a.N = sd.N, a.D = sd.D;
    a.x = x, a.gate = gate, a.out_in = out, a.dout = dout, a.lengths = lengths, a.first = dstate_out;
    a.state_in = state_in, a.dx = dx, a.dgate = dgate, a.last = dstate_in;
    return launch_any<true>(sd, a, st);
}

cudaError_t launch_scan_step(const ScanDims &sd, const void *x, const void *gate, float *state, void *out,
                             cudaStream_t st)
{
    const long long n = (long long)sd.S * sd.D;
    k_scan_step<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(n, sd.mean, sd.bf16, x, gate, state,
                                                                              out);
    return cudaGetLastError();
}

} // namespace gma
