// Token probabilities and the verification of drafted tokens.
//
// Source: frankenocr.pages.dev, "One forward pass", step 7 (the lm_head's logits choose the next token).  The pages
// decode greedily; this is the sampling form for a tree of drafted tokens, which keeps the target's distribution.
//
// focr_token_probs:  p = exp((l - max l) / temperature) / sum, per row of logits.
//
// focr_spec_verify:  the nodes are tried in index order (a parent stands before its children).  cur is the last
// accepted node (the root at first), p and q the target's and the draft's distribution behind it.  Siblings are
// independent draws from q; after k rejections the target's normalised residual is proportional to
//     W(t) = max(p(t) - c q(t), 0),      c = M_0 + ... + M_{k-1},  M_0 = 1,  M_k = sum_t W(t),
// because max(max(p - a q, 0) - b q, 0) = max(p - (a + b) q, 0): one scalar carries the whole chain of residuals.
// A child x is accepted iff u q(x) M < W(x).  Without draft probabilities q is one at x: accept iff u M < W(x), and a
// rejection takes p(x) out of W and M.  The next token is the smallest t with sum_{t' <= t} W(t') > u_N sum W.
// The answers are whole numbers next to borders, so all of it is in fp64 (products and differences of two fp32
// values are exact or nearly so); sums run in a fixed order.
//
// Both are bound by memory (one row of V floats read and written; one row of p and q read per rejection), and by
// latency for few rows.  A row belongs to a cluster of up to eight CTAs, whose sums meet in distributed shared memory.
//
// token_probs: as many clusters as stay resident take rows in turn.  A row is read once, by asynchronous copies that
// are in flight while the row before is worked on, and stays in registers (KEPT groups of four values a thread; what a
// row has beyond that is read again).  The CTAs send each other maximum and sum by st.async on a barrier in shared
// memory; a cluster barrier would wait for the stores of the row's probabilities as well.  A wait that runs out (it
// needs a CTA of the cluster to stop) gives NaN.  289 rows of 129280: 67 us, 4.4 TB/s (a cluster per
// row, without copies ahead: 87 us; taking rows in turn with a cluster barrier: 104 us); one row of 129280: 6.3 us.
// Clusters of eight CTAs of which two share an SM stay on 132 of 148 SMs.  Each row has one
// serial exchange through the cluster between its loads and its stores; that is what is left.
//
// spec_verify: p and q of all drafted tokens are looked up at once before the walk, so an accepted node costs no memory
// latency; a rejection is one pass over the rows, spread over the cluster's warps.  The tiles' sums stay in shared
// memory and lead to the next token's tile without a second pass over the rows.  One tree of 4 nodes: 9.0 us; 32 trees
// of 16 nodes, V = 129280: 24 us (with the warps' tiles summed a second time, the answer agreed on by two more cluster
// barriers and sums fetched instead of stored: 12.3 and 25.4 us).  What is left is the chain of passes: up to one per rejected
// sibling, each over the whole row pair with a cluster-wide sum.
#include <math.h>

#include "abi_util.h"
#include "cluster.cuh"
#include "common.cuh"
#include "launch_state.h"

namespace focr {
namespace {

constexpr int TREE_MAX = FOCR_TREE_NODES_MAX;
constexpr int VT = 512, VWARPS = VT / 32;   // threads of the verification
constexpr int CLUSTER_MAX = 8;

// ------------------------------------------------------------------ probabilities

constexpr int PT = 512, PWARPS = PT / 32;

// values of a row per CTA of its cluster
__host__ __device__ inline int row_share(int V, int C) { return ((V + C - 1) / C + 3) & ~3; }

struct ProbsParams {
    const float* logits;
    float* probs;
    int T, V, C;             // C: CTAs of a row
    float scale, scale_lo;   // log2(e) / temperature, as a sum of two floats
};

// exp((x - base) / temperature).  The exponent's rounding is that of the difference and of one product (the scale
// carries two floats).  -inf is held at a finite value, whose exponential is 0, so that the sum below stays finite.
__device__ __forceinline__ float expo(float x, float base, const ProbsParams& p) {
    const float t = max_nan(x - base, -1e30f);
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(fmaf(t, p.scale, t * p.scale_lo)));
    return y;
}

// How a thread's group of four values lies: FAR, PT values apart (logits and probabilities aligned differently); NEAR, 16
// aligned bytes, all inside the row's part x[0 .. n - 1] or all outside; SKEW, the same with groups that begin `skew` (0 .. 3)
// values ahead of the part, so the ones at its ends are taken value by value.  289 x 129281: SKEW 68 us, FAR 106; 289 x
// 129280: NEAR 67.0, SKEW 69.7.
enum { FAR, NEAR, SKEW };
template <int VEC>
__device__ __forceinline__ int first_of(int g, int tid, int skew) { return VEC == FAR ? 4 * g * PT + tid : 4 * (g * PT + tid) - skew; }
template <int VEC>
__device__ __forceinline__ bool whole(int i, int n) { return VEC == NEAR ? i < n : VEC == SKEW && i >= 0 && i + 3 < n; }
template <int VEC>
__device__ __forceinline__ float4 get4(const float* x, int g, int tid, int n, int skew, float none) {
    const int i = first_of<VEC>(g, tid, skew);
    if (whole<VEC>(i, n)) return *reinterpret_cast<const float4*>(x + i);
    if (VEC == NEAR) return make_float4(none, none, none, none);
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int at = i + j * (VEC == FAR ? PT : 1);
        v[j] = at >= 0 && at < n ? x[at] : none;
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}
template <int VEC>
__device__ __forceinline__ void put4(float* y, int g, int tid, int n, int skew, float4 v) {
    const int i = first_of<VEC>(g, tid, skew);
    if (whole<VEC>(i, n)) {
        *reinterpret_cast<float4*>(y + i) = v;
        return;
    }
    if (VEC == NEAR) return;
    const float o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int at = i + j * (VEC == FAR ? PT : 1);
        if (at >= 0 && at < n) y[at] = o[j];
    }
}
__device__ __forceinline__ float max4(float m, float4 v) { return fmaxf(fmaxf(m, fmaxf(v.x, v.y)), fmaxf(v.z, v.w)); }

// Starts the copy of group g into its place in shared memory (values outside the part become -inf).  A thread reads back
// only what it copied itself, so waiting for its own copies is enough.
template <int VEC>
__device__ __forceinline__ void fetch4(float4* held, const float* x, int g, int tid, int n, int skew) {
    float4* at = held + g * PT + tid;
    const uint32_t dst = smem_u32(at);
    const int i = first_of<VEC>(g, tid, skew);
    if (whole<VEC>(i, n)) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(x + i) : "memory");
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = i + j * (VEC == FAR ? PT : 1);
        if (VEC != NEAR && k >= 0 && k < n)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + 4 * j), "l"(x + k) : "memory");
        else
            reinterpret_cast<float*>(at)[j] = -INFINITY;
    }
}

struct Part {   // maximum of some logits and the sum of their exponentials relative to it
    float m;
    double s;
};
// A part without a finite logit has maximum -inf and sum 0 (NaN, should it hold one), taken relative to 0.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }
// Joins the parts of `width` neighbouring lanes, in every one of them.  A part that sums to 0 adds nothing: its base of 0 may
// lie so far above the others' maximum that the factor is infinite.
__device__ __forceinline__ Part join_lanes(Part a, int width, const ProbsParams& p) {
    float M = a.m;
    for (int o = width / 2; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    double s = a.s == 0. ? 0. : a.s * (double)expo(base_of(a.m), base_of(M), p);
    for (int o = width / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return {M, s};
}

// A cluster takes rows in turn: a row's part goes from shared memory to registers, the next row's copies start, and are
// in flight while this row is worked on, its sums come together and its probabilities are written.
// KEPT: groups of four values a thread keeps; the rest of a long row is read again.
template <int VEC, int KEPT>
__global__ void __launch_bounds__(PT, 2) token_probs_kernel(const __grid_constant__ ProbsParams p) {
    extern __shared__ __align__(16) float4 held[];   // [KEPT][PT]
    __shared__ float wm[PWARPS];
    __shared__ double ws[PWARPS], parts[2][2 * CLUSTER_MAX];   // parts: every CTA's maximum and sum of a row
    __shared__ uint64_t bar[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = p.C > 1 ? (int)cluster_rank() : 0, rows = gridDim.x / p.C;
    const int share = row_share(p.V, p.C), first = min(p.V, rank * share), n = min(share, p.V - first);
    int row = blockIdx.x / p.C, turn = 0, phase = 0;
    pdl_wait();
    auto part = [&](int r) { return p.logits + (size_t)r * p.V + first; };
    auto skew_of = [](const float* x) { return VEC == SKEW ? (int)((uintptr_t)x / 4 % 4) : 0; };
    auto fetch = [&](int r) {
#pragma unroll
        for (int g = 0; g < KEPT; ++g) fetch4<VEC>(held, part(r), g, tid, n, skew_of(part(r)));
    };
    fetch(row);
    if (p.C > 1) {
        if (tid == 0) {
            mbar_init(&bar[0], 1);
            mbar_init(&bar[1], 1);
            fence_barrier_init();
        }
        cluster_sync();
    }
    for (; row < p.T; row += rows, phase ^= turn, turn ^= 1) {
        const float* x = part(row);
        const int skew = skew_of(x), groups = (n + skew + 4 * PT - 1) / (4 * PT);
        float* y = p.probs + (size_t)row * p.V + first;
        asm volatile("cp.async.wait_all;" ::: "memory");
        float4 v[KEPT];
#pragma unroll
        for (int g = 0; g < KEPT; ++g) v[g] = held[g * PT + tid];   // what this thread copied itself
        if (row + rows < p.T) fetch(row + rows);
        // relative to the warp's maximum: sums within the warp need no factors
        Part a{-INFINITY, 0.};
#pragma unroll
        for (int g = 0; g < KEPT; ++g) a.m = max4(a.m, v[g]);
        for (int g = KEPT; g < groups; ++g) a.m = max4(a.m, get4<VEC>(x, g, tid, n, skew, -INFINITY));
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) a.m = fmaxf(a.m, __shfl_xor_sync(0xffffffffu, a.m, o));
        const float base = base_of(a.m);
        const bool masked = a.m == -INFINITY;   // none of the warp's values is finite: all of its exponentials are 0
#pragma unroll
        for (int g = 0; g < KEPT; ++g) {
            v[g] = make_float4(expo(v[g].x, base, p), expo(v[g].y, base, p), expo(v[g].z, base, p), expo(v[g].w, base, p));
            a.s += (double)((v[g].x + v[g].y) + (v[g].z + v[g].w));
        }
        for (int g = KEPT; g < groups; ++g) {
            const float4 t = get4<VEC>(x, g, tid, n, skew, -INFINITY);
            a.s += (double)((expo(t.x, base, p) + expo(t.y, base, p)) + (expo(t.z, base, p) + expo(t.w, base, p)));
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
        // Warps, then CTAs.  The first warp stores the CTA's pair into every CTA of the cluster, completing on their
        // barriers: unlike a cluster barrier this does not wait for the stores of the row before.  A CTA sends a row's
        // pair after it has all pairs of the row before, so two places are enough.
        if (lane == 0) wm[warp] = a.m, ws[warp] = a.s;
        __syncthreads();
        if (warp == 0) {
            a = join_lanes({wm[lane & (PWARPS - 1)], ws[lane & (PWARPS - 1)]}, PWARPS, p);
            if (p.C == 1) {   // st.async belongs to clusters
                if (lane == 0) parts[turn][0] = (double)a.m, parts[turn][1] = a.s;
            } else {
                if (lane == 0) mbar_arrive_expect_tx(&bar[turn], 16 * p.C);
                if (lane < p.C) {
                    const uint32_t at = mapa_shared(&parts[turn][2 * rank], lane), on = mapa_shared(&bar[turn], lane);
                    st_async_f64(at, (double)a.m, on);
                    st_async_f64(at + 8, a.s, on);
                }
            }
        }
        bool arrived = true;
        if (p.C == 1)
            __syncthreads();
        else
            arrived = mbar_wait_bounded(&bar[turn], phase, 2000000000ull);
        const int from = 2 * (lane & (p.C - 1));
        a = join_lanes({(float)parts[turn][from], parts[turn][from + 1]}, p.C, p);
        // a row of -inf alone has no distribution (and a wait that ran out gives no numbers)
        const float f = a.m == -INFINITY || !arrived ? __int_as_float(0x7fc00000) : expo(masked ? a.m : base, a.m, p) / (float)a.s;
#pragma unroll
        for (int g = 0; g < KEPT; ++g) put4<VEC>(y, g, tid, n, skew, make_float4(v[g].x * f, v[g].y * f, v[g].z * f, v[g].w * f));
        for (int g = KEPT; g < groups; ++g) {
            const float4 t = get4<VEC>(x, g, tid, n, skew, -INFINITY);
            put4<VEC>(y, g, tid, n, skew, make_float4(expo(t.x, base, p) * f, expo(t.y, base, p) * f, expo(t.z, base, p) * f, expo(t.w, base, p) * f));
        }
    }
}

template <int VEC, int KEPT>
cudaError_t launch_probs(ProbsParams& p, cudaStream_t st) {
    const void* fn = (const void*)token_probs_kernel<VEC, KEPT>;
    const size_t smem = (size_t)KEPT * PT * 16;
    const cudaError_t e = once_per_device(fn, [&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    // as many clusters as stay resident: they take rows in turn
    int rows = p.T;
    if (p.T * p.C > 128) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)p.C);
        cfg.blockDim = dim3(PT);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)p.C, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int most = 0;
        if (cudaOccupancyMaxActiveClusters(&most, fn, &cfg) == cudaSuccess && most > 0 && rows > most) rows = most;
    }
    void* args[] = {&p};
    return launch_kernel(fn, dim3((unsigned)(rows * p.C)), dim3(PT), smem, p.C, args, st);
}

template <int VEC>
cudaError_t launch_groups(ProbsParams& p, int groups, cudaStream_t st) {
    return groups <= 1 ? launch_probs<VEC, 1>(p, st) : groups <= 4 ? launch_probs<VEC, 4>(p, st) : launch_probs<VEC, 8>(p, st);
}

// ------------------------------------------------------------------ verification

struct VerifyParams {
    const float *target, *draft, *u;
    const int32_t *tokens, *parent, *n_nodes;
    int32_t *n_accept, *path, *next;
    int N, V, C, vec;
};

constexpr int TILE = 128;   // tokens a warp takes at a time
constexpr int BATCH = 4;    // tiles in flight
constexpr int TILES_MAX = (FOCR_V_MAX / TILE + CLUSTER_MAX - 1) / CLUSTER_MAX + VWARPS;   // of a CTA

struct VerifyShared {
    double p[TREE_MAX], q[TREE_MAX], u[TREE_MAX + 1];   // of each node's token behind its parent
    int par[TREE_MAX], tok[TREE_MAX], gone[TREE_MAX];
    double tile_sum[TILES_MAX], warp_sum[VWARPS], cta_sum[2][CLUSTER_MAX];
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// What is left of the target at token t (see the head of the file).
struct Residual {
    const float *p, *q;   // q: nullptr while nothing is taken off
    double c;
    const int* gone;      // rejected tokens of drafts without probabilities
    int n_gone;
    __device__ bool is_gone(int t) const {
        for (int i = 0; i < n_gone; ++i)
            if (gone[i] == t) return true;
        return false;
    }
    __device__ static double left(float p, float q, double c) {
        const double v = fma(-c, (double)q, (double)p);
        return v > 0. ? v : 0.;
    }
    __device__ double at(int t) const {
        if (q) return left(__ldg(p + t), __ldg(q + t), c);
        return is_gone(t) ? 0. : (double)__ldg(p + t);
    }
};

// The lane's share of one tile's sum of W.  vec: four neighbours of an aligned row, else four tokens 32 apart.
__device__ __forceinline__ void tile_load(const float* x, int tile, int lane, int V, bool vec, float (&o)[4]) {
    if (vec) {
        const int t = tile * TILE + 4 * lane;
        const float4 v = t < V ? __ldg(reinterpret_cast<const float4*>(x + t)) : make_float4(0.f, 0.f, 0.f, 0.f);
        o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = tile * TILE + 32 * j + lane;
            o[j] = t < V ? __ldg(x + t) : 0.f;
        }
    }
}
// Sums of W over tiles t0 .. t0 + BATCH - 1 below t1 (this lane's shares).
__device__ __forceinline__ void batch_sums(const Residual& w, int t0, int t1, int lane, int V, bool vec, bool any_gone,
                                           double (&s)[BATCH]) {
    float p[BATCH][4], q[BATCH][4];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
        const int tile = t0 + i < t1 ? t0 + i : V;   // behind the row: zeros
        tile_load(w.p, tile, lane, V, vec, p[i]);
        if (w.q) tile_load(w.q, tile, lane, V, vec, q[i]);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
        double d = 0.;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (w.q)
                d += Residual::left(p[i][j], q[i][j], w.c);
            else if (!any_gone || !w.is_gone((t0 + i) * TILE + (vec ? 4 * lane + j : 32 * j + lane)))
                d += (double)p[i][j];
        }
        s[i] = d;
    }
}

// Sum of W in every thread of the cluster; the tiles', warps' and CTAs' parts stay in shared memory.
__device__ double row_sum(const Residual& w, const VerifyParams& p, VerifyShared& sh, int t0, int t1, int mine0, int& turn) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool any_gone = false;
    if (!w.q)
        for (int i = 0; i < w.n_gone; ++i) any_gone |= w.gone[i] / TILE >= t0 && w.gone[i] / TILE < t1;
    double s = 0.;
    for (int t = t0; t < t1; t += BATCH) {
        double part[BATCH];
        batch_sums(w, t, t1, lane, p.V, p.vec, any_gone, part);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) part[i] = warp_sum(part[i]);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            s += part[i];
            if (lane == 0 && t + i < t1) sh.tile_sum[mine0 + t - t0 + i] = part[i];
        }
    }
    __syncthreads();   // the sums of the pass before have been read
    if (lane == 0) sh.warp_sum[warp] = s;
    __syncthreads();
    double total = 0.;
#pragma unroll
    for (int i = 0; i < VWARPS; ++i) total += sh.warp_sum[i];
    if (p.C == 1) return total;
    // into every CTA of the cluster; two places in turn: a CTA may store its next sum while another still reads this one
    turn ^= 1;
    if (threadIdx.x < p.C) st_cluster(&sh.cta_sum[turn][cluster_rank()], threadIdx.x, total);
    cluster_sync();
    total = 0.;
    for (int r = 0; r < p.C; ++r) total += sh.cta_sum[turn][r];
    return total;
}

__global__ void __launch_bounds__(VT, 2) spec_verify_kernel(const __grid_constant__ VerifyParams p) {
    __shared__ VerifyShared sh;
    const int rank = p.C > 1 ? (int)cluster_rank() : 0, b = blockIdx.x / p.C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, N = p.N, V = p.V;
    const float *P = p.target + (size_t)b * (N + 1) * V, *Q = p.draft ? p.draft + (size_t)b * N * V : nullptr;
    pdl_wait();
    if (p.C > 1) cluster_arrive();
    // every node's parent, token and uniform at once, then p and q of its token behind its parent
    const int L = p.n_nodes ? __ldg(p.n_nodes + b) : N;
    bool wrong = L < 0 || L > N;
    if (tid < N) {
        const int par = p.parent ? __ldg(p.parent + (size_t)b * N + tid) : tid - 1;
        const int x = __ldg(p.tokens + (size_t)b * N + tid);
        const float u = __ldg(p.u + (size_t)b * (N + 1) + tid);
        if (tid < L) {
            if (par < -1 || par >= tid || x < 0 || x >= V) {
                wrong = true;
            } else {
                const size_t at = (size_t)(par + 1) * V + x;
                const float pv = __ldg(P + at), qv = Q ? __ldg(Q + at) : 1.f;
                sh.par[tid] = par, sh.tok[tid] = x;
                sh.p[tid] = (double)pv, sh.q[tid] = (double)qv, sh.u[tid] = (double)u;
            }
        }
    }
    if (tid == TREE_MAX) sh.u[TREE_MAX] = (double)__ldg(p.u + (size_t)b * (N + 1) + N);
    int32_t* path = p.path + (size_t)b * N;
    const bool any_wrong = __syncthreads_or(wrong);   // the whole cluster sees the same
    if (p.C > 1) cluster_wait();                      // every CTA of the cluster runs: its shared memory may be written
    if (any_wrong) {
        if (rank == 0) {
            if (tid < N) path[tid] = -1;
            if (tid == 0) p.n_accept[b] = p.next[b] = -1;
        }
        return;
    }
    // this warp's tiles, and the place of its first one's sum
    const int tiles = (V + TILE - 1) / TILE, per = (tiles + p.C * VWARPS - 1) / (p.C * VWARPS);
    const int t0 = min(tiles, (rank * VWARPS + warp) * per), t1 = min(tiles, t0 + per), mine0 = warp * per;
    int cur = -1, taken = 0, turn = 0;
    double M = 1.;
    bool summed = false;   // M is the sum of W, and its parts are in shared memory
    Residual w{P, nullptr, 0., sh.gone, 0};
    for (int i = 0; i < L; ++i) {
        if (sh.par[i] != cur) continue;
        const int x = sh.tok[i];
        double left = fma(-w.c, sh.q[i], sh.p[i]);
        if (!Q) left = w.is_gone(x) ? 0. : sh.p[i];
        left = left > 0. ? left : 0.;
        if (sh.u[i] * sh.q[i] * M < left) {
            cur = i;
            if (rank == 0 && tid == 0) path[taken] = i;
            ++taken;
            M = 1.;
            w = Residual{P + (size_t)(cur + 1) * V, nullptr, 0., sh.gone, 0};
            summed = false;
        } else if (Q) {
            w.c += M;
            w.q = Q + (size_t)(cur + 1) * V;
            M = row_sum(w, p, sh, t0, t1, mine0, turn);
            summed = true;
        } else if (left > 0.) {
            __syncthreads();
            if (tid == 0) sh.gone[w.n_gone] = x;
            ++w.n_gone;
            M -= left;
            __syncthreads();
        }
    }
    if (rank == 0) {
        if (tid == 0) p.n_accept[b] = taken;
        if (tid >= taken && tid < N) path[tid] = -1;
    }
    double total = summed ? M : row_sum(w, p, sh, t0, t1, mine0, turn);
    if (!(total > 0.)) {   // nothing is left (a draft that equals the target, rejected by rounding): the target itself
        w.q = nullptr;
        w.n_gone = 0;
        total = row_sum(w, p, sh, t0, t1, mine0, turn);
    }
    // The warp whose tiles hold the border looks for it.  Every warp forms the borders between warps from the same sums
    // in the same order, so exactly one warp finds itself: the last one, should rounding put the border behind all sums;
    // the first one, should there be no border (rows that hold no mass, or none that is finite).
    const double want = sh.u[TREE_MAX] * total;
    const bool none = !(total > 0. && want == want);
    double before = 0., after;
    {
        double base = 0., sum = 0.;
        for (int r = 0; r < rank; ++r) base += sh.cta_sum[turn][r];
        for (int i = 0; i < warp; ++i) sum += sh.warp_sum[i];
        before = base + sum, after = base + (sum + sh.warp_sum[warp]);
    }
    const bool first = rank == 0 && warp == 0, last = rank == p.C - 1 && warp == VWARPS - 1;
    if (none ? first : (first || before <= want) && (last || want < after)) {
        int found = -1;
        for (int c = t0; c < t1 && found < 0; c += 32) {   // 32 tiles' sums at a time, in order
            double s = c + lane < t1 ? sh.tile_sum[mine0 + c - t0 + lane] : 0.;
            const bool some = s > 0.;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += up;
            }
            unsigned hit = __ballot_sync(0xffffffffu, some && before + s > want);
            while (hit && found < 0) {   // the first such tile; the next one should rounding leave it without a token
                const int k = __ffs(hit) - 1, tile = c + k;
                hit &= hit - 1;
                double sum = before + (k > 0 ? __shfl_sync(0xffffffffu, s, k > 0 ? k - 1 : 0) : 0.);
                double v[TILE / 32];
#pragma unroll
                for (int j = 0; j < TILE / 32; ++j) {
                    const int tok = tile * TILE + 32 * j + lane;
                    v[j] = tok < V ? w.at(tok) : 0.;
                }
#pragma unroll
                for (int j = 0; j < TILE / 32; ++j) {   // token by token, in order
                    double a = v[j];
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const double up = __shfl_up_sync(0xffffffffu, a, o);
                        if (lane >= o) a += up;
                    }
                    const unsigned at = __ballot_sync(0xffffffffu, v[j] > 0. && sum + a > want);
                    if (at && found < 0) found = tile * TILE + 32 * j + __ffs(at) - 1;
                    sum += __shfl_sync(0xffffffffu, a, 31);
                }
            }
            before += __shfl_sync(0xffffffffu, s, 31);
        }
        // rounding left the border behind the last sum: the last token up to here with any mass (anywhere, if none has)
        for (int t = min(V, t1 * TILE) - 1; t >= 0 && found < 0; t -= 32) {
            const unsigned hit = __ballot_sync(0xffffffffu, t >= lane && w.at(max(0, t - lane)) > 0.);
            if (hit) found = t - __ffs(hit) + 1;
        }
        if (lane == 0) p.next[b] = found < 0 ? V - 1 : found;
    }
}

// CTAs of a row of V values: at most `most` values each, and smaller parts while the device is not full
int row_cluster(int rows, int V, int most, int least) {
    const int sms = device_sms() > 0 ? device_sms() : 148;
    int C = 1;
    while (C < CLUSTER_MAX && (V > C * most || (rows * C < sms && V > C * least))) C *= 2;
    return C;
}

}  // namespace
}  // namespace focr

extern "C" {

focr_status focr_token_probs(const float* logits, int32_t T, int32_t V, float temperature, float* probs, void* stream) {
    using namespace focr;
    report_error(FOCR_OK, "");
    if (!logits || !probs) return report_error(FOCR_ERR_INVALID_ARG, "NULL argument");
    if (T < 1 || T > FOCR_T_MAX) return reportf(FOCR_ERR_INVALID_ARG, "T=%d outside [1, %d]", T, FOCR_T_MAX);
    if (V < 1 || V > FOCR_V_MAX) return reportf(FOCR_ERR_INVALID_ARG, "V=%d outside [1, %d]", V, FOCR_V_MAX);
    if (!(temperature >= 1e-6f && temperature <= 1e6f))
        return reportf(FOCR_ERR_INVALID_ARG, "temperature=%g outside [1e-6, 1e6]", (double)temperature);
    if (misaligned(logits, 4) || misaligned(probs, 4)) return report_error(FOCR_ERR_INVALID_ARG, "misaligned logits or probs");
    const size_t bytes = 4ull * T * V;
    if (probs != logits && ranges_overlap(logits, bytes, probs, bytes))
        return report_error(FOCR_ERR_INVALID_ARG, "probs overlaps logits without being it");
    ProbsParams p;
    p.logits = logits, p.probs = probs, p.T = T, p.V = V;
    p.C = row_cluster(T, V, 4 * PT * 8, 4 * PT);
    const double scale = 1.4426950408889634 / (double)temperature;
    p.scale = (float)scale, p.scale_lo = (float)(scale - (double)p.scale);
    const bool even = ((uintptr_t)logits - (uintptr_t)probs) % 16 == 0, aligned = even && V % 4 == 0 && !misaligned(logits, 16);
    // as few kept groups as hold a row's part: 289 x 2000 with 1 / 8 of them 3.0 / 5.6 us, 289 x 8000 with 4 / 8 5.0 / 6.3
    const int groups = (row_share(V, p.C) + (even && !aligned ? 3 : 0) + 4 * PT - 1) / (4 * PT);
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = aligned ? launch_groups<NEAR>(p, groups, st) : even ? launch_groups<SKEW>(p, groups, st) : launch_groups<FAR>(p, groups, st);
    return report_launch(e, "token_probs_kernel");
}

focr_status focr_spec_verify(const float* target, const float* draft, int32_t V, const int32_t* tokens,
                             const int32_t* parent, const int32_t* n_nodes, const float* u, int32_t B, int32_t N,
                             int32_t* n_accept, int32_t* path, int32_t* next_token, void* stream) {
    using namespace focr;
    report_error(FOCR_OK, "");
    if (!target || !tokens || !u || !n_accept || !path || !next_token)
        return report_error(FOCR_ERR_INVALID_ARG, "NULL argument");
    if (B < 1 || B > FOCR_RSWA_B_MAX) return reportf(FOCR_ERR_INVALID_ARG, "B=%d outside [1, %d]", B, FOCR_RSWA_B_MAX);
    if (N < 1 || N > TREE_MAX) return reportf(FOCR_ERR_INVALID_ARG, "N=%d outside [1, %d]", N, TREE_MAX);
    if (V < 1 || V > FOCR_V_MAX) return reportf(FOCR_ERR_INVALID_ARG, "V=%d outside [1, %d]", V, FOCR_V_MAX);
    const void* all[] = {target, draft, tokens, parent, n_nodes, u, n_accept, path, next_token};
    for (const void* x : all)
        if (misaligned(x, 4)) return report_error(FOCR_ERR_INVALID_ARG, "misaligned argument");
    // the CTAs of a tree read while one of them already answers
    const size_t rows = 4ull * B * N, row = 4ull * V;
    const Span out[] = {{n_accept, 4ull * B}, {path, rows}, {next_token, 4ull * B}};
    const Span in[] = {{target, row * B * (N + 1)}, {draft, row * B * N}, {tokens, rows}, {parent, rows}, {n_nodes, 4ull * B},
                       {u, 4ull * B * (N + 1)}};
    if (outputs_overlap(out, 3, in, 6)) return report_error(FOCR_ERR_INVALID_ARG, "an output overlaps another argument");
    VerifyParams p{target, draft, u, tokens, parent, n_nodes, n_accept, path, next_token, N, V,
                   row_cluster(B, V, VWARPS * TILE * BATCH, VWARPS * TILE),
                   V % 4 == 0 && !misaligned(target, 16) && !misaligned(draft, 16)};
    void* args[] = {&p};
    return report_launch(launch_kernel((const void*)spec_verify_kernel, dim3((unsigned)B * p.C), dim3(VT), 0, p.C, args,
                                       (cudaStream_t)stream),
                         "spec_verify_kernel");
}

}  // extern "C"
