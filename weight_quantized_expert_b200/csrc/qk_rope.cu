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
// Bound by memory: every row is read and written once, 1 KB a row.  8192 tokens x 20 heads with norms (168 MB): 29.3 us from a
// graph, 5.7 TB/s, and 32.2 us called on inputs that change (31.6 from a graph with 40 registers instead of 32, a few of them
// spilled); one token: 1.7 us.  A block a token, its rows' loads ahead of the angles, half a warp a row (a warp a row with the
// angles first: 50 us; blocks that stay and take tokens in turn: 66 us, each waiting for the angles of its next token).
#include <math.h>

#include "abi_util.h"
#include "common.cuh"

namespace focr {
namespace {

constexpr int RD = FOCR_RSWA_DIM;
constexpr int RWARPS = 16;         // most warps of a block

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

// A block has one token; half a warp has a row (two rows a warp share its instructions), loaded before the angles are
// formed.  Lane l of a half has dims 4 l .. 4 l + 3 and 64 + 4 l .. 64 + 4 l + 3.
// HOW: 0 pairs (2i, 2i + 1); 1 pairs (i, i + 64): both in a lane.  2 pairs (i, i + rot / 2), rot < 128, through shared memory,
// dim by dim (8192 tokens x 20 heads with norms: 1 29.2 us, 2 with rot 64 / 126 34.2 / 39.7; in chunks of four dims 31.4 with
// rot 64, but 39.4 instead of 36.6 with rot 96).
template <int HOW, bool NORM>
__global__ void __launch_bounds__(32 * RWARPS, 4) qk_rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float2 cs[RD / 2];
    __shared__ __align__(16) float row[HOW == 2 ? 2 * RWARPS : 1][RD];
    const int t = blockIdx.x, l = threadIdx.x & 15, h0 = threadIdx.x >> 4, step = blockDim.x >> 4;
    const int half = p.rot / 2, heads = p.hq + p.hk;
    const float* q = p.q + (size_t)t * p.ldq + 4 * l;
    const float* k = p.k + (size_t)t * p.ldk + 4 * l;
    pdl_wait();
    auto load = [&](int h, float4& a, float4& b) {
        const float4* src = reinterpret_cast<const float4*>(h < p.hq ? q + h * RD : k + (h - p.hq) * RD);
        a = src[0], b = src[16];
    };
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (h0 < heads) load(h0, a, b);
    float4 g0, g1;
    auto weights = [&](int h) {
        const float4* g = reinterpret_cast<const float4*>(h < p.hq ? p.gamma_q : p.gamma_k);
        g0 = g ? __ldg(g + l) : make_float4(1.f, 1.f, 1.f, 1.f);
        g1 = g ? __ldg(g + l + 16) : make_float4(1.f, 1.f, 1.f, 1.f);
    };
    if (NORM) weights(h0);
    if (threadIdx.x < RD / 2) {   // behind the last pair: no turn
        const double r = (double)__ldg(p.pos + t) * p.rev[threadIdx.x];
        float s, c;
        sincospif(2.f * (float)(r - rint(r)), &s, &c);
        cs[threadIdx.x] = make_float2(c, s);
    }
    __syncthreads();
    // cosines and sines of the lane's pairs
    float4 t0, t1;
    if (HOW == 0) t0 = *reinterpret_cast<const float4*>(&cs[2 * l]), t1 = *reinterpret_cast<const float4*>(&cs[32 + 2 * l]);
    if (HOW == 1) t0 = *reinterpret_cast<const float4*>(&cs[4 * l]), t1 = *reinterpret_cast<const float4*>(&cs[4 * l + 2]);
    for (int h = h0; h - (h0 & 1) < heads; h += step) {   // both halves of a warp stay together
        const bool live = h < heads, isq = h < p.hq;
        if (h != h0 && live) {
            load(h, a, b);
            if (NORM) weights(h);
        }
        if (NORM) {
            float ss = (a.x * a.x + a.y * a.y) + (a.z * a.z + a.w * a.w) + ((b.x * b.x + b.y * b.y) + (b.z * b.z + b.w * b.w));
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float inv = rsqrtf(ss * (1.f / RD) + p.eps);
            a = make_float4(a.x * inv * g0.x, a.y * inv * g0.y, a.z * inv * g0.z, a.w * inv * g0.w);
            b = make_float4(b.x * inv * g1.x, b.y * inv * g1.y, b.z * inv * g1.z, b.w * inv * g1.w);
        }
        float4 x = a, y = b;
        if (HOW == 0) {
            x = make_float4(a.x * t0.x - a.y * t0.y, a.y * t0.x + a.x * t0.y, a.z * t0.z - a.w * t0.w, a.w * t0.z + a.z * t0.w);
            y = make_float4(b.x * t1.x - b.y * t1.y, b.y * t1.x + b.x * t1.y, b.z * t1.z - b.w * t1.w, b.w * t1.z + b.z * t1.w);
            if (p.rot < RD) {   // the others pass as they are, infinities too
                if (2 * l >= half) x.x = a.x, x.y = a.y;
                if (2 * l + 1 >= half) x.z = a.z, x.w = a.w;
                if (32 + 2 * l >= half) y.x = b.x, y.y = b.y;
                if (33 + 2 * l >= half) y.z = b.z, y.w = b.w;
            }
        } else if (HOW == 1) {
            x = make_float4(a.x * t0.x - b.x * t0.y, a.y * t0.z - b.y * t0.w, a.z * t1.x - b.z * t1.y, a.w * t1.z - b.w * t1.w);
            y = make_float4(b.x * t0.x + a.x * t0.y, b.y * t0.z + a.y * t0.w, b.z * t1.x + a.z * t1.y, b.w * t1.z + a.w * t1.w);
        } else {
            float* r = row[threadIdx.x >> 4];
            __syncwarp();
            reinterpret_cast<float4*>(r)[l] = a, reinterpret_cast<float4*>(r)[l + 16] = b;
            __syncwarp();
            // a lane has every sixteenth dim
            float* dst = isq ? p.q_out + (size_t)t * p.ldqo + h * RD : p.k_out + (size_t)t * p.ldko + (h - p.hq) * RD;
#pragma unroll
            for (int d = l; d < RD; d += 16) {
                float v = r[d];
                if (d < p.rot) {
                    const float2 c = cs[d < half ? d : d - half];
                    v = d < half ? v * c.x - r[d + half] * c.y : v * c.x + r[d - half] * c.y;
                }
                if (live) dst[d] = v;
            }
            continue;
        }
        if (live) {
            float4* dst = reinterpret_cast<float4*>((isq ? p.q_out + (size_t)t * p.ldqo + h * RD
                                                         : p.k_out + (size_t)t * p.ldko + (h - p.hq) * RD) + 4 * l);
            dst[0] = x, dst[16] = y;
        }
    }
}

template <bool NORM>
const void* rope_kernel(const RopeParams& p) {
    if (p.flags & FOCR_ROPE_INTERLEAVED) return (const void*)qk_rope_kernel<0, NORM>;
    return p.rot == RD ? (const void*)qk_rope_kernel<1, NORM> : (const void*)qk_rope_kernel<2, NORM>;
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
    const Span out[] = {{q_out, 4 * (size_t)((T - 1) * ldqo + wq)}}, out_k[] = {{k_out, 4 * (size_t)((T - 1) * ldko + wk)}};
    const Span in[] = {{pos, 4ull * T}, {gamma_q, 4ull * RD}, {gamma_k, 4ull * RD}};
    if (bad || outputs_overlap(out, 1, in, 3) || outputs_overlap(out_k, 1, in, 3))
        return report_error(FOCR_ERR_INVALID_ARG, "outputs overlap other rows, the positions or the weights");
    RopeParams p;
    p.q = q, p.k = k, p.q_out = q_out, p.k_out = k_out, p.gamma_q = gamma_q, p.gamma_k = gamma_k, p.pos = pos;
    p.ldq = ldq, p.ldk = ldk, p.ldqo = ldqo, p.ldko = ldko;
    p.T = T, p.hq = heads_q, p.hk = heads_k, p.rot = rot_dim, p.flags = flags, p.eps = eps;
    // powers by repeated products (one pow a call): off by at most i x 2^-53, on angles that shrink with i
    const double ratio = pow(theta, -2. / rot_dim);
    double rev = 0.15915494309189535;   // 1 / (2 pi)
    for (int i = 0; i < RD / 2; ++i, rev *= ratio) p.rev[i] = i < rot_dim / 2 ? rev : 0.;
    const int warps = (heads_q + heads_k + 1) / 2;   // two rows each; at least the 64 threads that form the angles
    const int threads = 32 * (warps < 2 ? 2 : warps < RWARPS ? warps : RWARPS);
    void* args[] = {&p};
    return report_launch(launch_kernel(flags & FOCR_QK_NORM ? rope_kernel<true>(p) : rope_kernel<false>(p), dim3(T), dim3(threads), 0,
                                       1, args, (cudaStream_t)stream),
                         "qk_rope_kernel");
}
