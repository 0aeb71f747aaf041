// R-SWA attention for a tree of drafted tokens over a quantised cache; one node is the single-token form.
//
// Source: franken_ocr README, "Design Philosophy" and "Architecture" (R-SWA: each generated token attends to every
// reference token plus the previous 128 generated tokens, a ring buffer); frankenocr.pages.dev, "One forward pass",
// step 6 (ten heads of dimension 128).  Readings as in rswa.cu; the window counts the node itself.
//
//   n = n_gen[b] tokens are committed (positions 0 .. n-1); node i of depth d (0 for a child of the last committed
//   token) stands at position n + d.  It sees the reference rows r < ref_len[b], the ring's tokens p with
//   max(0, n - 128, n + d - 127) <= p < n, its ancestors and itself (k_new / v_new, fp32):
//       out = sum_j softmax_j(q . k_j / sqrt(128)) v_j,   k_j = ks_j * kc_j,  v_j = vs_j * vc_j (codes and scales).
//   Query head x reads kv head x / (heads_q / heads_kv).  In terms of a slot's age a = (n - 1 - slot) mod 128 the
//   window is a < min(n, 127 - d), which needs no sum that could overflow.
#include <math.h>

#include "abi_util.h"
#include "common.cuh"
#include "kv_cache.h"

namespace focr {
namespace {

constexpr int RD = FOCR_RSWA_DIM, RW = FOCR_RSWA_RING;
constexpr int TREE_MAX = FOCR_TREE_NODES_MAX;
constexpr float SCALE = 0.08838834764831845f;   // 1 / sqrt(128)

struct TreeParams {
    const float *q, *k_new, *v_new;
    KvView ref, ring;
    const int32_t *ref_len, *n_gen, *parent, *n_nodes;
    float* out;
    int N, hq, hk, G;
};

// 16 codes of a row, from dim 16 * sub, as floats
__device__ __forceinline__ void load16(const uint8_t* codes, size_t row, int type, int sub, float (&x)[16]) {
    if (type == FOCR_W_INT8) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(codes + row * RD) + sub);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = (float)(int8_t)(u[j / 4] >> 8 * (j % 4));
    } else {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(codes + row * (RD / 2)) + sub);
        const uint32_t u[2] = {w.x, w.y};
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = (float)((int)(u[j / 8] << (28 - 4 * (j % 8))) >> 28);
    }
}

constexpr int PT = 128, GROUPS = PT / 8;

__global__ void __launch_bounds__(PT) rswa_tree_kernel(const __grid_constant__ TreeParams p) {
    __shared__ float sm_m[GROUPS], sm_l[GROUPS];
    __shared__ __align__(16) float sm_acc[GROUPS][RD];
    __shared__ int sm_par[TREE_MAX];
    __shared__ int sm_bad;
    const int b = blockIdx.x / p.hk, h = blockIdx.x % p.hk, node = blockIdx.y / p.G, x = h * p.G + blockIdx.y % p.G;
    const int tid = threadIdx.x, g = tid >> 3, sub = tid & 7;
    pdl_wait();
    const int R = __ldg(p.ref_len + b), n = __ldg(p.n_gen + b), L = p.n_nodes ? __ldg(p.n_nodes + b) : p.N;
    if (tid == 0) sm_bad = R < 0 || R > p.ref.cap || n < 0 || L < 0 || L > p.N;
    __syncthreads();
    if (tid < min(L, p.N)) {
        const int par = p.parent ? __ldg(p.parent + (size_t)b * p.N + tid) : tid - 1;
        sm_par[tid] = par;
        if (par < -1 || par >= tid) sm_bad = 1;
    }
    __syncthreads();
    float* out = p.out + (((size_t)b * p.N + node) * p.hq + x) * RD;
    if (sm_bad) {
        if (node < (L < 0 || L > p.N ? p.N : L)) out[tid] = __int_as_float(0x7fc00000);   // NaN
        return;
    }
    if (node >= L) return;
    unsigned long long line = 0;   // the node and its ancestors
    int depth = -1;
    for (int j = node; j >= 0; j = sm_par[j]) {
        line |= 1ull << j;
        ++depth;
    }
    float qv[16];
    {
        const float4* q4 = reinterpret_cast<const float4*>(p.q + (((size_t)b * p.N + node) * p.hq + x) * RD + 16 * sub);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 t = __ldg(q4 + i);
            qv[4 * i] = t.x, qv[4 * i + 1] = t.y, qv[4 * i + 2] = t.z, qv[4 * i + 3] = t.w;
        }
    }
    const int ages = min(n, RW - 1 - depth);
    const size_t row0 = ((size_t)b * p.hk + h) * p.ref.cap, ring0 = ((size_t)b * p.hk + h) * RW;
    float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    const int nk = R + RW + L;
    for (int jb = 0; jb < nk; jb += GROUPS) {
        const int j = jb + g;
        float kk[16], vv[16], ks = 0.f, vs = 0.f;
        bool live = j < nk;
        if (live && j < R) {
            load16(p.ref.k, row0 + j, p.ref.type, sub, kk);
            load16(p.ref.v, row0 + j, p.ref.type, sub, vv);
            ks = __ldg(p.ref.ks + row0 + j), vs = __ldg(p.ref.vs + row0 + j);
        } else if (live && j < R + RW) {
            const int slot = j - R;
            live = (unsigned)(n - 1 - slot) % RW < (unsigned)ages && n > 0;
            if (live) {
                load16(p.ring.k, ring0 + slot, p.ring.type, sub, kk);
                load16(p.ring.v, ring0 + slot, p.ring.type, sub, vv);
                ks = __ldg(p.ring.ks + ring0 + slot), vs = __ldg(p.ring.vs + ring0 + slot);
            }
        } else if (live) {
            const int a = j - R - RW;
            live = line >> a & 1;
            if (live) {
                const size_t r = (((size_t)b * p.N + a) * p.hk + h) * RD + 16 * sub;
#pragma unroll
                for (int i = 0; i < 16; ++i) kk[i] = __ldg(p.k_new + r + i), vv[i] = __ldg(p.v_new + r + i);
                ks = vs = 1.f;
            }
        }
        float dot = 0.f;
        if (live) {
#pragma unroll
            for (int i = 0; i < 16; ++i) dot = fmaf(qv[i], kk[i], dot);
        }
        dot += __shfl_xor_sync(0xffffffffu, dot, 1);
        dot += __shfl_xor_sync(0xffffffffu, dot, 2);
        dot += __shfl_xor_sync(0xffffffffu, dot, 4);
        if (!live) continue;
        const float sc = dot * ks * SCALE, mn = fmaxf(m, sc);
        const float corr = expf(m - mn), w = expf(sc - mn);
        l = l * corr + w;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = acc[i] * corr + w * vs * vv[i];
        m = mn;
    }
    if (sub == 0) sm_m[g] = m, sm_l[g] = l;
#pragma unroll
    for (int i = 0; i < 16; ++i) sm_acc[g][16 * sub + i] = acc[i];
    __syncthreads();
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) M = fmaxf(M, sm_m[k]);
    float Ls = 0.f, A = 0.f;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
        const float e = expf(sm_m[k] - M);   // 0 for an empty group; the node itself is in one of them
        Ls += sm_l[k] * e;
        A += sm_acc[k][tid] * e;
    }
    out[tid] = A / Ls;
}

}  // namespace
}  // namespace focr

extern "C" focr_status focr_rswa_tree(const float* q, const float* k_new, const float* v_new, int32_t B, int32_t N,
                                      int32_t heads_q, const focr_kv_cache* ref, const int32_t* ref_len,
                                      const focr_kv_cache* ring, const int32_t* n_gen, const int32_t* parent,
                                      const int32_t* n_nodes, float* out, void* stream) {
    using namespace focr;
    report_error(FOCR_OK, "");
    TreeParams p;
    focr_status s = check_kv_cache(ref, "ref", &p.ref);
    if (s == FOCR_OK) s = check_kv_cache(ring, "ring", &p.ring);
    if (s != FOCR_OK) return s;
    if (!q || !k_new || !v_new || !ref_len || !n_gen || !out) return report_error(FOCR_ERR_INVALID_ARG, "NULL argument");
    if (ref->type != ring->type) return report_error(FOCR_ERR_UNSUPPORTED, "ref and ring must have one type");
    if (ring->cap != RW) return reportf(FOCR_ERR_UNSUPPORTED, "the ring has %d slots, not %d", ring->cap, RW);
    if (ref->B != B || ring->B != B || ref->heads != ring->heads)
        return reportf(FOCR_ERR_INVALID_ARG, "caches of %d and %d sequences, %d and %d heads for B=%d", ref->B, ring->B,
                       ref->heads, ring->heads, B);
    if (heads_q < ref->heads || heads_q > FOCR_HEADS_MAX || heads_q % ref->heads)
        return reportf(FOCR_ERR_UNSUPPORTED, "%d query heads over %d kv heads", heads_q, ref->heads);
    const int G = heads_q / ref->heads;
    if (N < 1 || (int64_t)N * G > TREE_MAX)
        return reportf(FOCR_ERR_INVALID_ARG, "%d nodes x %d query heads per kv head outside [1, %d]", N, G, TREE_MAX);
    const void* f[] = {q, k_new, v_new, out};
    for (const void* ptr : f)
        if (misaligned(ptr, 16)) return report_error(FOCR_ERR_INVALID_ARG, "float buffers must be 16-byte aligned");
    if (misaligned(ref_len, 4) || misaligned(n_gen, 4) || misaligned(parent, 4) || misaligned(n_nodes, 4))
        return report_error(FOCR_ERR_INVALID_ARG, "misaligned lengths or tree");
    const size_t qb = 4ull * B * N * heads_q * RD, kb = 4ull * B * N * ref->heads * RD;
    if (ranges_overlap(out, qb, q, qb) || ranges_overlap(out, qb, k_new, kb) || ranges_overlap(out, qb, v_new, kb))
        return report_error(FOCR_ERR_INVALID_ARG, "out overlaps an input");
    p.q = q, p.k_new = k_new, p.v_new = v_new, p.ref_len = ref_len, p.n_gen = n_gen, p.parent = parent, p.n_nodes = n_nodes;
    p.out = out, p.N = N, p.hq = heads_q, p.hk = ref->heads, p.G = G;
    void* args[] = {&p};
    return report_launch(launch_kernel((const void*)rswa_tree_kernel, dim3(B * p.hk, N * G), dim3(PT), 0, 1, args,
                                       (cudaStream_t)stream),
                         "rswa_tree_kernel");
}
