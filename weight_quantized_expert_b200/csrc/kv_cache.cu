// Quantised key/value rows: written into a cache as they come, and read back.
//
// Source: franken_ocr README, "Architecture" (R-SWA: a frozen reference block and a 128-slot ring of generated
// tokens); frankenocr.pages.dev, "Four bits, one shared scale" (an int4 code is a two's-complement nibble sharing one
// fp32 scale with its group).  The group is a whole row, the 128 values of one head of one token:
//   s = fp32(max|x|) / Q as one fp32 division (Q = 127 int8, 7 int4); q = round-half-even(fp32(x / s)) clamped to
//   [-127, 127] or [-8, 7]; a row with s = 0 has q = 0;  the value read back is fp32(s * q).
// Both kernels are bound by memory: 512 B of fp32 against 132 B (int8) or 68 B (int4) a row, each moved once.  Half a warp
// has a token of a head, its K and its V row, with all loads issued before the first is used, and a division only where a
// value lies next to a border of the rounding.  8 sequences x 10 heads x ragged 4096 rows, int8, written and read back (659
// MB): 106 us from a graph, 6.2 TB/s, and 111 us called on inputs that change (from a graph: a warp a row, all divided 159 us;
// values rounded, clamped and packed one by one 112 us, bound by the write's instructions); 8 x 9 tokens into an int4 ring 2.3
// us, the ring read back 3.0.
#include "abi_util.h"
#include "common.cuh"
#include "kv_cache.h"

namespace focr {
namespace {

constexpr int RD = FOCR_RSWA_DIM;
constexpr int CT = 256, CROWS = CT / 16;   // half a warp has a token of a head: its K row and its V row

struct WriteParams {
    KvView c;
    const float *k, *v;
    const int32_t *row0, *count, *index, *start;
    int64_t ldk, ldv, n_rows;
    int n_max, wrap;
};

// round-half-even(fp32(x / s)) by the division itself.
template <bool INT4>
__device__ __noinline__ uint32_t codes_by_division(float4 x, float s) {
    const float in[4] = {x.x, x.y, x.z, x.w};
    uint32_t w = 0u;
    for (int j = 0; j < 4; ++j) {
        const int q = __float2int_rn(in[j] / s);
        w |= ((uint32_t)(INT4 ? max(-8, min(7, q)) : max(-127, min(127, q))) & 255u) << 8 * j;
    }
    return w;
}
// Codes of four values, one a byte.  x / s is formed with the reciprocal, rounded by adding 1.5 * 2^23 (the code is then the
// sum's low byte), and its distance from the rounded value returned through `far`.  The reciprocal and the division each
// round by 2^-24 of at most 127, so the code is the division's unless the distance is within 2^-15 of a half.
__device__ __forceinline__ uint32_t codes4(float4 x, float inv, float& far) {
    constexpr float MAGIC = 12582912.f;
    const float in[4] = {x.x, x.y, x.z, x.w};
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float t = fmaf(in[j], inv, MAGIC);
        u[j] = __float_as_uint(t);
        far = fmaxf(far, fabsf(fmaf(in[j], inv, MAGIC - t)));
    }
    return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
}
// A row of 128 by half a warp: lane l has values 4 l .. 4 l + 3 (a) and 64 + 4 l .. 64 + 4 l + 3 (b).
template <bool INT4>
__device__ __forceinline__ void quantise_row(float4 a, float4 b, bool live, uint8_t* codes, float* scale, int l) {
    // a NaN in the row becomes the scale, so that it is not taken for a number later (an infinity does the same by itself)
    float m = max_nan(max_nan(max_nan(fabsf(a.x), fabsf(a.y)), max_nan(fabsf(a.z), fabsf(a.w))),
                      max_nan(max_nan(fabsf(b.x), fabsf(b.y)), max_nan(fabsf(b.z), fabsf(b.w))));
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = m / (INT4 ? 7.f : 127.f), inv = 1.f / s;
    uint32_t w[2] = {0u, 0u};
    if (s > 0.f) {
        float far = 0.f;
        w[0] = codes4(a, inv, far), w[1] = codes4(b, inv, far);
        // scales near the subnormal numbers (reciprocals that overflow, rounded scales) and infinite ones go the same way
        if (!(far < 0.5f - 3.1e-5f) || !(s > 1e-35f) || !(s < 1e35f)) w[0] = codes_by_division<INT4>(a, s), w[1] = codes_by_division<INT4>(b, s);
        if (INT4) {   // bytes to nibbles
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                w[i] &= 0x0F0F0F0Fu;
                w[i] = __byte_perm(w[i] | w[i] >> 4, 0u, 0x4420);
            }
        }
    }
    if (!live) return;
    if (INT4) {
        reinterpret_cast<uint16_t*>(codes)[l] = (uint16_t)w[0];
        reinterpret_cast<uint16_t*>(codes)[l + 16] = (uint16_t)w[1];
    } else {
        reinterpret_cast<uint32_t*>(codes)[l] = w[0];
        reinterpret_cast<uint32_t*>(codes)[l + 16] = w[1];
    }
    if (l == 0) *scale = s;
}

template <bool INT4>
__global__ void __launch_bounds__(CT) kv_write_kernel(const __grid_constant__ WriteParams p) {
    const int b = blockIdx.z, h = blockIdx.y, l = threadIdx.x & 15;
    const int i = blockIdx.x * CROWS + (threadIdx.x >> 4);
    pdl_wait();
    const int n = __ldg(p.count + b), s0 = __ldg(p.start + b);
    bool live = n >= 0 && n <= p.n_max && i < n && s0 >= 0;
    if (p.wrap)
        live = live && i >= n - p.c.cap;   // a later token of the call takes the slot of an earlier one
    else
        live = live && s0 <= p.c.cap - n;
    int64_t src = 0;
    if (live) {
        src = (p.row0 ? (int64_t)__ldg(p.row0 + b) : (int64_t)b * p.n_max) + (p.index ? __ldg(p.index + (size_t)b * p.n_max + i) : i);
        live = src >= 0 && src < p.n_rows;
    }
    if (!__any_sync(0xffffffffu, live)) return;   // both halves stay for the shuffles
    if (!live) src = 0;
    const float4* k = reinterpret_cast<const float4*>(p.k + src * p.ldk + (size_t)h * RD) + l;
    const float4* v = reinterpret_cast<const float4*>(p.v + src * p.ldv + (size_t)h * RD) + l;
    float4 ka = __ldg(k), kb = __ldg(k + 16), va = __ldg(v), vb = __ldg(v + 16);
    const int slot = p.wrap ? (int)(((uint32_t)s0 + (uint32_t)i) % (uint32_t)p.c.cap) : s0 + i;
    const size_t r = ((size_t)b * p.c.heads + h) * p.c.cap + slot;
    constexpr size_t RB = INT4 ? RD / 2 : RD;
    quantise_row<INT4>(ka, kb, live, p.c.k + r * RB, p.c.ks + r, l);
    quantise_row<INT4>(va, vb, live, p.c.v + r * RB, p.c.vs + r, l);
}

struct ReadParams {
    KvView c;
    const int32_t* len;
    float *k_out, *v_out;
};

// four codes as values
template <bool INT4>
__device__ __forceinline__ float4 values4(uint32_t w, float s) {
    if (INT4)
        return make_float4((float)((int)(w << 28) >> 28) * s, (float)((int)(w << 24) >> 28) * s, (float)((int)(w << 20) >> 28) * s,
                           (float)((int)(w << 16) >> 28) * s);
    return make_float4((float)(int8_t)w * s, (float)(int8_t)(w >> 8) * s, (float)(int8_t)(w >> 16) * s, (float)(int8_t)(w >> 24) * s);
}

template <bool INT4>
__global__ void __launch_bounds__(CT) kv_read_kernel(const __grid_constant__ ReadParams p) {
    const int b = blockIdx.z, h = blockIdx.y, l = threadIdx.x & 15;
    const int i = blockIdx.x * CROWS + (threadIdx.x >> 4);
    pdl_wait();
    const int n = __ldg(p.len + b);
    if (n < 0 || n > p.c.cap || i >= n) return;
    const size_t r = ((size_t)b * p.c.heads + h) * p.c.cap + i;
    uint32_t w[2][2];
    float s[2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const uint8_t* codes = (kv ? p.c.v : p.c.k) + r * (INT4 ? RD / 2 : RD);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            w[kv][j] = INT4 ? reinterpret_cast<const uint16_t*>(codes)[l + 16 * j] : reinterpret_cast<const uint32_t*>(codes)[l + 16 * j];
        s[kv] = (kv ? p.c.vs : p.c.ks)[r];
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            reinterpret_cast<float4*>((kv ? p.v_out : p.k_out) + r * RD)[l + 16 * j] = values4<INT4>(w[kv][j], s[kv]);
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
    Span out[4];
    cache_spans(c, out);
    const size_t tab = 4ull * c->B;
    const Span in[] = {{k, 4 * (size_t)((n_rows - 1) * ldk + w)}, {v, 4 * (size_t)((n_rows - 1) * ldv + w)}, {row0, tab},
                       {count, tab}, {index, tab * n_max}, {start, tab}};
    if (outputs_overlap(out, 4, in, 6)) return report_error(FOCR_ERR_INVALID_ARG, "the cache's buffers overlap one another or an input");
    p.k = k, p.v = v, p.row0 = row0, p.count = count, p.index = index, p.start = start;
    p.ldk = ldk, p.ldv = ldv, p.n_rows = n_rows, p.n_max = n_max, p.wrap = flags & FOCR_KV_WRAP;
    void* args[] = {&p};
    const dim3 grid((n_max + CROWS - 1) / CROWS, c->heads, c->B);
    const void* fn = c->type == FOCR_W_INT4 ? (const void*)kv_write_kernel<true> : (const void*)kv_write_kernel<false>;
    return report_launch(launch_kernel(fn, grid, dim3(CT), 0, 1, args, (cudaStream_t)stream),
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
    const Span out[] = {{k_out, bytes}, {v_out, bytes}};
    Span in[5] = {{}, {}, {}, {}, {len, 4ull * c->B}}, own[4];
    cache_spans(c, own);
    for (int i = 0; i < 4; ++i) in[i] = own[i];
    if (outputs_overlap(out, 2, in, 5)) return report_error(FOCR_ERR_INVALID_ARG, "the outputs overlap one another or an input");
    p.len = len, p.k_out = k_out, p.v_out = v_out;
    void* args[] = {&p};
    const dim3 grid((c->cap + CROWS - 1) / CROWS, c->heads, c->B);
    const void* fn = c->type == FOCR_W_INT4 ? (const void*)kv_read_kernel<true> : (const void*)kv_read_kernel<false>;
    return report_launch(launch_kernel(fn, grid, dim3(CT), 0, 1, args, (cudaStream_t)stream),
                         "kv_read_kernel");
}

}  // extern "C"
