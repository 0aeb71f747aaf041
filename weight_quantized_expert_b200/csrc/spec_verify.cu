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
#include <math.h>

#include "abi_util.h"
#include "common.cuh"

namespace focr {
namespace {

constexpr int TREE_MAX = FOCR_TREE_NODES_MAX;
constexpr int VT = 1024, VWARPS = VT / 32;

struct ProbsParams {
    const float* logits;
    float* probs;
    int V;
    float temp;
};

__global__ void __launch_bounds__(VT) token_probs_kernel(ProbsParams p) {
    __shared__ float sm[VWARPS];
    __shared__ double sum[VWARPS];
    const int tid = threadIdx.x;
    const float* x = p.logits + (size_t)blockIdx.x * p.V;
    float* y = p.probs + (size_t)blockIdx.x * p.V;
    pdl_wait();
    float m = -INFINITY;
    for (int t = tid; t < p.V; t += VT) m = fmaxf(m, x[t]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) sm[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < VWARPS; ++w) m = fmaxf(m, sm[w]);
    double d = 0.;   // a row has up to a million terms
    for (int t = tid; t < p.V; t += VT) d += (double)expf((x[t] - m) / p.temp);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if ((tid & 31) == 0) sum[tid >> 5] = d;
    __syncthreads();
    d = 0.;
#pragma unroll
    for (int w = 0; w < VWARPS; ++w) d += sum[w];
    const float s = (float)d;
    for (int t = tid; t < p.V; t += VT) y[t] = expf((x[t] - m) / p.temp) / s;
}

struct VerifyParams {
    const float *target, *draft, *u;
    const int32_t *tokens, *parent, *n_nodes;
    int32_t *n_accept, *path, *next;
    int N, V;
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// What is left of the target at token t (see the head of the file).
struct Residual {
    const float *p, *q;
    double c;
    const int* gone;   // rejected tokens of drafts without probabilities
    int n_gone;
    __device__ double at(int t) const {
        const double v = (double)__ldg(p + t);
        if (q) return fmax(v - c * (double)__ldg(q + t), 0.);
        for (int i = 0; i < n_gone; ++i)
            if (gone[i] == t) return 0.;
        return v;
    }
};

// Sums of W over the warps' contiguous segments into `seg`, and the total, in every thread.
__device__ double segment_sums(const Residual& w, int V, double* seg) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = (V + VWARPS - 1) / VWARPS, t0 = warp * len, t1 = min(V, t0 + len);
    double s = 0.;
    for (int t = t0 + lane; t < t1; t += 32) s += w.at(t);
    s = warp_sum(s);
    __syncthreads();
    if (lane == 0) seg[warp] = s;
    __syncthreads();
    double total = 0.;
    for (int i = 0; i < VWARPS; ++i) total += seg[i];
    return total;
}

__global__ void __launch_bounds__(VT) spec_verify_kernel(VerifyParams p) {
    __shared__ double seg[VWARPS];
    __shared__ int gone[TREE_MAX];
    __shared__ int sm_bad, sm_next, sm_last;
    const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, N = p.N, V = p.V;
    pdl_wait();
    const int L = p.n_nodes ? __ldg(p.n_nodes + b) : N;
    if (tid == 0) {
        sm_bad = L < 0 || L > N;
        sm_next = V;
        sm_last = -1;
    }
    __syncthreads();
    if (tid < min(L, N)) {
        const int par = p.parent ? __ldg(p.parent + (size_t)b * N + tid) : tid - 1;
        const int x = __ldg(p.tokens + (size_t)b * N + tid);
        if (par < -1 || par >= tid || x < 0 || x >= V) sm_bad = 1;
    }
    __syncthreads();
    int32_t* path = p.path + (size_t)b * N;
    if (sm_bad) {
        if (tid < N) path[tid] = -1;
        if (tid == 0) p.n_accept[b] = p.next[b] = -1;
        return;
    }
    const float *P = p.target + (size_t)b * (N + 1) * V, *Q = p.draft ? p.draft + (size_t)b * N * V : nullptr;
    int cur = -1, taken = 0;
    double M = 1.;
    Residual w{P, Q, 0., gone, 0};
    for (int i = 0; i < L; ++i) {
        const int par = p.parent ? __ldg(p.parent + (size_t)b * N + i) : i - 1;
        if (par != cur) continue;
        const int x = __ldg(p.tokens + (size_t)b * N + i);
        const double left = w.at(x), q = Q ? (double)__ldg(w.q + x) : 1.;
        if ((double)__ldg(p.u + (size_t)b * (N + 1) + i) * q * M < left) {
            cur = i;
            if (tid == 0) path[taken] = i;
            ++taken;
            M = 1.;
            w.p = P + (size_t)(cur + 1) * V;
            w.q = Q && cur + 1 < N ? Q + (size_t)(cur + 1) * V : nullptr;
            w.c = 0.;
            w.n_gone = 0;
        } else if (Q) {
            w.c += M;
            M = segment_sums(w, V, seg);
        } else {
            __syncthreads();
            if (tid == 0) gone[w.n_gone] = x;
            ++w.n_gone;
            M -= left;
            __syncthreads();
        }
    }
    double total = segment_sums(w, V, seg);
    if (!(total > 0.)) {   // nothing is left (a draft that equals the target, rejected by rounding): the target itself
        w.q = nullptr;
        w.n_gone = 0;
        total = segment_sums(w, V, seg);
    }
    const double want = (double)__ldg(p.u + (size_t)b * (N + 1) + N) * total;
    double before = 0.;
    for (int i = 0; i < warp; ++i) before += seg[i];
    const int len = (V + VWARPS - 1) / VWARPS, t0 = warp * len, t1 = min(V, t0 + len);
    // the warp whose segment holds the border scans it; the last token with any mass stands in when rounding
    // leaves the border behind the last sum
    for (int tb = t0; tb < t1; tb += 32) {
        const int t = tb + lane;
        const double v = t < t1 ? w.at(t) : 0.;
        double s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double up = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += up;
        }
        if (v > 0.) {
            if (before + s > want) atomicMin(&sm_next, t);
            atomicMax(&sm_last, t);
        }
        before += __shfl_sync(0xffffffffu, s, 31);
    }
    __syncthreads();
    if (tid == 0) {
        const int last = sm_last < 0 ? V - 1 : sm_last;
        p.next[b] = min(sm_next, last);
        p.n_accept[b] = taken;
        for (int i = taken; i < N; ++i) path[i] = -1;
    }
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
    if (!(temperature > 0.f) || !isfinite(temperature))
        return reportf(FOCR_ERR_INVALID_ARG, "temperature=%g must be positive", (double)temperature);
    if (misaligned(logits, 4) || misaligned(probs, 4)) return report_error(FOCR_ERR_INVALID_ARG, "misaligned logits or probs");
    const size_t bytes = 4ull * T * V;
    if (probs != logits && ranges_overlap(logits, bytes, probs, bytes))
        return report_error(FOCR_ERR_INVALID_ARG, "probs overlaps logits without being it");
    ProbsParams p{logits, probs, V, temperature};
    void* args[] = {&p};
    return report_launch(launch_kernel((const void*)token_probs_kernel, dim3(T), dim3(VT), 0, 1, args, (cudaStream_t)stream),
                         "token_probs_kernel");
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
    VerifyParams p{target, draft, u, tokens, parent, n_nodes, n_accept, path, next_token, N, V};
    void* args[] = {&p};
    return report_launch(launch_kernel((const void*)spec_verify_kernel, dim3(B), dim3(VT), 0, 1, args, (cudaStream_t)stream),
                         "spec_verify_kernel");
}

}  // extern "C"
