// Norms of queries and keys per head and the position rotation, in one pass over the rows.
//
// Source: frankenocr.pages.dev, "One forward pass", step 6 (ten heads of dimension 128); the pages fix no rotation
// formula, so this is the common one.  For a row x of 128 values (one head of one token at position pos):
//   y = x / sqrt(mean(x^2) + eps) * gamma        (with FOCR_QK_NORM, else y = x)
//   pair i < rot / 2 joins dims (i, i + rot/2), or (2i, 2i+1) with FOCR_ROPE_INTERLEAVED;
//   angle = pos * theta^(-2i / rot);  (a, b) -> (a cos - b sin, b cos + a sin);  dims >= rot pass through.
// The angle is formed in revolutions in fp64 and reduced to [-1/2, 1/2] before it is rounded to fp32, so far
// positions lose nothing: the reduced angle is off by at most 2^-25 revolutions plus pos x 2^-53 x a few.
//
// Bound by memory: every row is read and written once, 1 KB a row.
#include <math.h>

#include "abi_util.h"
#include "common.cuh"

namespace focr {
namespace {

constexpr int RD = FOCR_RSWA_DIM;
constexpr int RT = 256;            // threads: eight warps, one row each at a time
constexpr int RWARPS = RT / 32;

struct RopeParams {
    const float *q, *k;
    float *q_out, *k_out;
    const float *gamma_q, *gamma_k;
    const int32_t* pos;
    int64_t ldq, ldk, ldqo, ldko;
    int T, hq, hk, rot, flags;
    float eps;
    double rev[RD / 2];   // revolutions per position of each pair: theta^(-2i / rot) / (2 pi)
};

__global__ void __launch_bounds__(RT) qk_rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 cs[RD / 2];
    __shared__ __align__(16) float row[RWARPS][RD];
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = p.rot / 2;
    const bool inter = p.flags & FOCR_ROPE_INTERLEAVED, norm = p.flags & FOCR_QK_NORM;
    pdl_wait();
    if (threadIdx.x < half) {
        const double r = (double)__ldg(p.pos + t) * p.rev[threadIdx.x];
        float s, c;
        sincospif(2.f * (float)(r - rint(r)), &s, &c);
        cs[threadIdx.x] = make_float2(c, s);
    }
    __syncthreads();
    for (int h = warp; h < p.hq + p.hk; h += RWARPS) {
        const bool isq = h < p.hq;
        const int hh = isq ? h : h - p.hq;
        const float* src = (isq ? p.q + (size_t)t * p.ldq : p.k + (size_t)t * p.ldk) + (size_t)hh * RD;
        float* dst = (isq ? p.q_out + (size_t)t * p.ldqo : p.k_out + (size_t)t * p.ldko) + (size_t)hh * RD;
        float4 v = reinterpret_cast<const float4*>(src)[lane];
        if (norm) {
            float ss = v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float inv = 1.f / sqrtf(ss * (1.f / RD) + p.eps);
            const float* gamma = isq ? p.gamma_q : p.gamma_k;
            float4 g = make_float4(1.f, 1.f, 1.f, 1.f);
            if (gamma) g = __ldg(reinterpret_cast<const float4*>(gamma) + lane);
            v = make_float4(v.x * inv * g.x, v.y * inv * g.y, v.z * inv * g.z, v.w * inv * g.w);
        }
        __syncwarp();
        reinterpret_cast<float4*>(row[warp])[lane] = v;
        __syncwarp();
        float o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = 4 * lane + j;
            const float x = row[warp][d];
            if (d >= p.rot) {
                o[j] = x;
            } else if (inter) {
                const float2 a = cs[d >> 1];
                o[j] = d & 1 ? x * a.x + row[warp][d - 1] * a.y : x * a.x - row[warp][d + 1] * a.y;
            } else {
                const float2 a = cs[d < half ? d : d - half];
                o[j] = d < half ? x * a.x - row[warp][d + half] * a.y : x * a.x + row[warp][d - half] * a.y;
            }
        }
        reinterpret_cast<float4*>(dst)[lane] = make_float4(o[0], o[1], o[2], o[3]);
    }
}

// Whether rows of `wa` floats at `a` (stride lda) and of `wb` floats at `b` (stride ldb) share an element.
bool rows_overlap(const float* a, int64_t lda, int64_t wa, const float* b, int64_t ldb, int64_t wb, int T) {
    if (!ranges_overlap(a, 4 * (size_t)((T - 1) * lda + wa), b, 4 * (size_t)((T - 1) * ldb + wb))) return false;
    if (lda != ldb || ((uintptr_t)a - (uintptr_t)b) % 4) return true;
    int64_t d = ((int64_t)((uintptr_t)b - (uintptr_t)a) / 4) % lda;
    if (d < 0) d += lda;
    return !(wa <= d && d + wb <= lda);
}

}  // namespace
}  // namespace focr

extern "C" focr_status focr_qk_norm_rope(const float* q, int64_t ldq, int32_t heads_q, const float* k, int64_t ldk,
                                         int32_t heads_k, const int32_t* pos, int32_t T, const float* gamma_q,
                                         const float* gamma_k, float eps, double theta, int32_t rot_dim, int32_t flags,
                                         float* q_out, int64_t ldqo, float* k_out, int64_t ldko, void* stream) {
    using namespace focr;
    report_error(FOCR_OK, "");
    if (!q || !q_out || !pos || (heads_k > 0 && (!k || !k_out))) return report_error(FOCR_ERR_INVALID_ARG, "NULL argument");
    if (T < 1 || T > FOCR_T_MAX) return reportf(FOCR_ERR_INVALID_ARG, "T=%d outside [1, %d]", T, FOCR_T_MAX);
    if (heads_q < 1 || heads_q > FOCR_HEADS_MAX || heads_k < 0 || heads_k > FOCR_HEADS_MAX)
        return reportf(FOCR_ERR_INVALID_ARG, "heads %d / %d outside [1, %d] / [0, %d]", heads_q, heads_k, FOCR_HEADS_MAX,
                       FOCR_HEADS_MAX);
    if (rot_dim < 2 || rot_dim > RD || rot_dim % 2)
        return reportf(FOCR_ERR_UNSUPPORTED, "rot_dim=%d is not an even number in [2, %d]", rot_dim, RD);
    if (flags & ~(FOCR_QK_NORM | FOCR_ROPE_INTERLEAVED)) return reportf(FOCR_ERR_INVALID_ARG, "unknown flags 0x%x", (unsigned)flags);
    if (!(theta > 0.) || !isfinite(theta)) return reportf(FOCR_ERR_INVALID_ARG, "theta=%g must be positive", theta);
    if (!(eps >= 0.f)) return reportf(FOCR_ERR_INVALID_ARG, "eps=%g must not be negative", (double)eps);
    const int64_t wq = (int64_t)heads_q * RD, wk = (int64_t)heads_k * RD;
    if (heads_k == 0) {
        k = k_out = nullptr;
        ldk = ldko = 0;
    }
    const int64_t ld[] = {ldq, ldqo, ldk, ldko}, w[] = {wq, wq, wk, wk};
    const void* ptr[] = {q, q_out, k, k_out, gamma_q, gamma_k};
    for (int i = 0; i < 4; ++i)
        if (ld[i] < w[i] || ld[i] % 4 || ld[i] > (int64_t)1 << 32)
            return reportf(FOCR_ERR_INVALID_ARG, "row stride %lld is below the %lld floats of a row or not a multiple of 4",
                           (long long)ld[i], (long long)w[i]);
    for (const void* x : ptr)
        if (misaligned(x, 16)) return report_error(FOCR_ERR_INVALID_ARG, "float buffers must be 16-byte aligned");
    if (misaligned(pos, 4)) return report_error(FOCR_ERR_INVALID_ARG, "misaligned positions");
    // in place is fine (a warp reads a row before it writes it); any other shared element is a race
    bool bad = !(q_out == q && ldqo == ldq) && rows_overlap(q_out, ldqo, wq, q, ldq, wq, T);
    if (heads_k > 0)
        bad = bad || (!(k_out == k && ldko == ldk) && rows_overlap(k_out, ldko, wk, k, ldk, wk, T)) ||
              rows_overlap(q_out, ldqo, wq, k, ldk, wk, T) || rows_overlap(k_out, ldko, wk, q, ldq, wq, T) ||
              rows_overlap(q_out, ldqo, wq, k_out, ldko, wk, T);
    if (bad) return report_error(FOCR_ERR_INVALID_ARG, "outputs overlap other rows");
    RopeParams p;
    p.q = q, p.k = k, p.q_out = q_out, p.k_out = k_out, p.gamma_q = gamma_q, p.gamma_k = gamma_k, p.pos = pos;
    p.ldq = ldq, p.ldk = ldk, p.ldqo = ldqo, p.ldko = ldko;
    p.T = T, p.hq = heads_q, p.hk = heads_k, p.rot = rot_dim, p.flags = flags, p.eps = eps;
    // powers by repeated products (one pow a call): off by at most i x 2^-53, on angles that shrink with i
    const double ratio = pow(theta, -2. / rot_dim);
    double rev = 0.15915494309189535;   // 1 / (2 pi)
    for (int i = 0; i < RD / 2; ++i, rev *= ratio) p.rev[i] = i < rot_dim / 2 ? rev : 0.;
    void* args[] = {&p};
    return report_launch(launch_kernel((const void*)qk_rope_kernel, dim3(T), dim3(RT), 0, 1, args, (cudaStream_t)stream),
                         "qk_rope_kernel");
}
