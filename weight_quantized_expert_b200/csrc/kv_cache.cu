// Quantised key/value rows: written into a cache as they come, and read back.
//
// Source: franken_ocr README, "Architecture" (R-SWA: a frozen reference block and a 128-slot ring of generated
// tokens); frankenocr.pages.dev, "Four bits, one shared scale" (an int4 code is a two's-complement nibble sharing one
// fp32 scale with its group).  The group is a whole row, the 128 values of one head of one token:
//   s = fp32(max|x|) / Q as one fp32 division (Q = 127 int8, 7 int4); q = round-half-even(fp32(x / s)) clamped to
//   [-127, 127] or [-8, 7]; a row with s = 0 has q = 0;  the value read back is fp32(s * q).
// Both kernels are bound by memory: 512 B of fp32 against 132 B (int8) or 68 B (int4) a row, each moved once.
#include "abi_util.h"
#include "common.cuh"
#include "kv_cache.h"

namespace focr {
namespace {

constexpr int RD = FOCR_RSWA_DIM;
constexpr int CT = 256, CWARPS = CT / 32;

struct WriteParams {
    KvView c;
    const float *k, *v;
    const int32_t *row0, *count, *index, *start;
    int64_t ldk, ldv, n_rows;
    int n_max, wrap;
};

// One row of 128 by a warp (four values a lane).
__device__ __forceinline__ void quantise_row(float4 x, int type, void* codes, float* scale, int lane) {
    float a = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const float s = a / (type == FOCR_W_INT8 ? 127.f : 7.f);
    const float in[4] = {x.x, x.y, x.z, x.w};
    int q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = s > 0.f ? __float2int_rn(in[j] / s) : 0;
        q[j] = type == FOCR_W_INT8 ? max(-127, min(127, r)) : max(-8, min(7, r));
    }
    if (type == FOCR_W_INT8)
        reinterpret_cast<uint32_t*>(codes)[lane] =
            (q[0] & 255) | (q[1] & 255) << 8 | (q[2] & 255) << 16 | (uint32_t)(q[3] & 255) << 24;
    else
        reinterpret_cast<uint16_t*>(codes)[lane] =
            (uint16_t)((q[0] & 15) | (q[1] & 15) << 4 | (q[2] & 15) << 8 | (q[3] & 15) << 12);
    if (lane == 0) *scale = s;
}

// A warp writes one token of one head: its K row and its V row.
__global__ void __launch_bounds__(CT) kv_write_kernel(const __grid_constant__ WriteParams p) {
    const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
    const int i = blockIdx.x * CWARPS + (threadIdx.x >> 5);
    pdl_wait();
    const int n = __ldg(p.count + b), s0 = __ldg(p.start + b);
    if (n < 0 || n > p.n_max || i >= n || s0 < 0) return;
    if (!p.wrap && (int64_t)s0 + n > p.c.cap) return;
    if (p.wrap && i < n - p.c.cap) return;   // a later token of the call takes its slot
    const int64_t src = (p.row0 ? (int64_t)__ldg(p.row0 + b) : (int64_t)b * p.n_max) +
                        (p.index ? __ldg(p.index + (size_t)b * p.n_max + i) : i);
    if (src < 0 || src >= p.n_rows) return;
    const int slot = (int)(((int64_t)s0 + i) % p.c.cap);
    const float4 xk = __ldg(reinterpret_cast<const float4*>(p.k + src * p.ldk + (size_t)h * RD) + lane);
    const float4 xv = __ldg(reinterpret_cast<const float4*>(p.v + src * p.ldv + (size_t)h * RD) + lane);
    const size_t r = ((size_t)b * p.c.heads + h) * p.c.cap + slot;
    const size_t rb = p.c.type == FOCR_W_INT8 ? RD : RD / 2;
    quantise_row(xk, p.c.type, p.c.k + r * rb, p.c.ks + r, lane);
    quantise_row(xv, p.c.type, p.c.v + r * rb, p.c.vs + r, lane);
}

struct ReadParams {
    KvView c;
    const int32_t* len;
    float *k_out, *v_out;
};

__global__ void __launch_bounds__(CT) kv_read_kernel(const __grid_constant__ ReadParams p) {
    const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
    const int i = blockIdx.x * CWARPS + (threadIdx.x >> 5);
    pdl_wait();
    const int n = __ldg(p.len + b);
    if (n < 0 || n > p.c.cap || i >= n) return;
    const size_t r = ((size_t)b * p.c.heads + h) * p.c.cap + i;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const uint8_t* codes = kv ? p.c.v : p.c.k;
        const float s = (kv ? p.c.vs : p.c.ks)[r];
        float o[4];
        if (p.c.type == FOCR_W_INT8) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(codes + r * RD)[lane];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = (float)(int8_t)(w >> 8 * j) * s;
        } else {
            const uint32_t w = reinterpret_cast<const uint16_t*>(codes + r * (RD / 2))[lane];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = (float)((int)(w << (28 - 4 * j)) >> 28) * s;
        }
        reinterpret_cast<float4*>((kv ? p.v_out : p.k_out) + r * RD)[lane] = make_float4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace

focr_status check_kv_cache(const focr_kv_cache* c, const char* what, KvView* v) {
    if (!c || !c->k || !c->k_scale || !c->v || !c->v_scale) return reportf(FOCR_ERR_INVALID_ARG, "%s: NULL argument", what);
    if (c->type != FOCR_W_INT8 && c->type != FOCR_W_INT4)
        return reportf(FOCR_ERR_UNSUPPORTED, "%s: type %d is not int8 or int4", what, c->type);
    if (c->B < 1 || c->B > FOCR_RSWA_B_MAX || c->heads < 1 || c->heads > FOCR_HEADS_MAX || c->cap < 1 ||
        c->cap > FOCR_RSWA_RCAP_MAX)
        return reportf(FOCR_ERR_INVALID_ARG, "%s: %d sequences, %d heads, %d rows outside [1, %d], [1, %d], [1, %d]", what,
                       c->B, c->heads, c->cap, FOCR_RSWA_B_MAX, FOCR_HEADS_MAX, FOCR_RSWA_RCAP_MAX);
    if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scale, 4) || misaligned(c->v_scale, 4))
        return reportf(FOCR_ERR_INVALID_ARG, "%s: codes must be 16-byte and scales 4-byte aligned", what);
    v->k = reinterpret_cast<uint8_t*>(c->k);
    v->v = reinterpret_cast<uint8_t*>(c->v);
    v->ks = c->k_scale;
    v->vs = c->v_scale;
    v->type = c->type, v->heads = c->heads, v->cap = c->cap;
    return FOCR_OK;
}

}  // namespace focr

extern "C" {

focr_status focr_kv_write(const focr_kv_cache* c, const float* k, int64_t ldk, const float* v, int64_t ldv,
                          int64_t n_rows, const int32_t* row0, const int32_t* count, const int32_t* index,
                          int32_t n_max, const int32_t* start, int32_t flags, void* stream) {
    using namespace focr;
    report_error(FOCR_OK, "");
    WriteParams p;
    const focr_status s = check_kv_cache(c, "cache", &p.c);
    if (s != FOCR_OK) return s;
    if (!k || !v || !count || !start) return report_error(FOCR_ERR_INVALID_ARG, "NULL argument");
    if (flags & ~FOCR_KV_WRAP) return reportf(FOCR_ERR_INVALID_ARG, "unknown flags 0x%x", (unsigned)flags);
    if (n_max < 1 || n_max > FOCR_KV_N_MAX) return reportf(FOCR_ERR_INVALID_ARG, "n_max=%d outside [1, %d]", n_max, FOCR_KV_N_MAX);
    if (n_rows < 1) return reportf(FOCR_ERR_INVALID_ARG, "n_rows=%lld below 1", (long long)n_rows);
    const int64_t w = (int64_t)c->heads * RD;
    if (ldk < w || ldk % 4 || ldv < w || ldv % 4)
        return reportf(FOCR_ERR_INVALID_ARG, "row stride %lld / %lld is below the %lld floats of a row or not a multiple of 4",
                       (long long)ldk, (long long)ldv, (long long)w);
    if (misaligned(k, 16) || misaligned(v, 16)) return report_error(FOCR_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
    if (misaligned(count, 4) || misaligned(start, 4) || misaligned(row0, 4) || misaligned(index, 4))
        return report_error(FOCR_ERR_INVALID_ARG, "misaligned row tables");
    p.k = k, p.v = v, p.row0 = row0, p.count = count, p.index = index, p.start = start;
    p.ldk = ldk, p.ldv = ldv, p.n_rows = n_rows, p.n_max = n_max, p.wrap = flags & FOCR_KV_WRAP;
    void* args[] = {&p};
    const dim3 grid((n_max + CWARPS - 1) / CWARPS, c->heads, c->B);
    return report_launch(launch_kernel((const void*)kv_write_kernel, grid, dim3(CT), 0, 1, args, (cudaStream_t)stream),
                         "kv_write_kernel");
}

focr_status focr_kv_read(const focr_kv_cache* c, const int32_t* len, float* k_out, float* v_out, void* stream) {
    using namespace focr;
    report_error(FOCR_OK, "");
    ReadParams p;
    const focr_status s = check_kv_cache(c, "cache", &p.c);
    if (s != FOCR_OK) return s;
    if (!len || !k_out || !v_out) return report_error(FOCR_ERR_INVALID_ARG, "NULL argument");
    if (misaligned(k_out, 16) || misaligned(v_out, 16) || misaligned(len, 4))
        return report_error(FOCR_ERR_INVALID_ARG, "misaligned outputs or lengths");
    const size_t bytes = 4ull * c->B * c->heads * c->cap * RD;
    if (ranges_overlap(k_out, bytes, v_out, bytes)) return report_error(FOCR_ERR_INVALID_ARG, "k_out and v_out overlap");
    p.len = len, p.k_out = k_out, p.v_out = v_out;
    void* args[] = {&p};
    const dim3 grid((c->cap + CWARPS - 1) / CWARPS, c->heads, c->B);
    return report_launch(launch_kernel((const void*)kv_read_kernel, grid, dim3(CT), 0, 1, args, (cudaStream_t)stream),
                         "kv_read_kernel");
}

}  // extern "C"
