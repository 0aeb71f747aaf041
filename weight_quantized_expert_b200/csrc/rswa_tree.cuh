// What the two kernels of the tree attention share (rswa_tree.cu, rswa_ranges.cu).
#pragma once

#include "common.cuh"
#include "kv_cache.h"

namespace focr {

constexpr int TREE_DIM = FOCR_RSWA_DIM, TREE_RING = FOCR_RSWA_RING;
constexpr int TREE_MAX = FOCR_TREE_NODES_MAX;
constexpr int COLS = 16;                        // columns of a unit: the rows of one MMA tile
constexpr int BLK = 64;                         // keys of a block
// A column's partial output in shared memory: its 128 dims with a gap behind each 16, PAD floats, so that neither a warp's
// stores (columns gr, dims 32 c + t) nor its loads (neighbouring dims) meet in a bank.
constexpr int PAD = TREE_DIM + 33;
__device__ __forceinline__ int part_at(int col, int dim) { return col * PAD + dim + 4 * (dim >> 4); }
constexpr float LOG2E = 1.4426950408889634f;
constexpr float SCORE_SCALE = 0.08838834764831845f;   // 1 / sqrt(128)
constexpr float Q_TOP = 8323072.f;              // 127 * 2^16: the largest fixed-point query value
constexpr float P_TOP = 8388604.f;              // 2^23 - 4: the largest fixed-point weight, before up to three roundings
constexpr float P_MAGIC = 8388608.f;            // 2^23: a fixed-point weight added to it is rounded and lies in the low 23 bits
constexpr float MAGIC = 12582912.f;             // 1.5 * 2^23
constexpr int MAGIC_BITS = 0x4B400000;
constexpr float NONE = -1e30f;                  // running maximum of a column that has seen no key
constexpr float TINY = 1e-30f;                  // magnitudes below this share its step

template <bool INT4>
struct Stage {   // where a block of keys lies in shared memory: one block of keys; later its partial output
    static constexpr int ROW = INT4 ? TREE_DIM / 2 : TREE_DIM;
    static constexpr int V = BLK * ROW, KS = 2 * BLK * ROW, VS = KS + 4 * BLK, LOADS = VS + 4 * BLK;
    static constexpr int BYTES = LOADS > COLS * PAD * 4 ? LOADS : COLS * PAD * 4;
};

struct TreeParams {
    const float *q, *k_new, *v_new;
    KvView ref, ring;
    const int32_t *ref_len, *n_gen, *parent, *n_nodes;
    float* out;
    int B, N, hq, hk, G, S, groups;   // groups of 16 columns per kv head; clusters: S CTAs each
    float* part;                      // ranges: two partial results per CTA
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// A value scale that is no number becomes the key scale's, so that it reaches those who see the key and nobody else
// (0 times NaN would reach all).  By the lane that copied key r's scales.
__device__ __forceinline__ void check_scale(uint8_t* ks, uint8_t* vs, int r) {
    float* v = reinterpret_cast<float*>(vs) + r;
    if (!(fabsf(*v) < INFINITY)) *v = 0.f, reinterpret_cast<float*>(ks)[r] = __int_as_float(0x7fc00000);
}

// 65536 d2 + 256 d1 + d0 of three integer accumulators that started at MAGIC_BITS (so they read as MAGIC + sum), as two
// parts: lower() + upper().  The products with the constants are exact (multiples of 256 and 65536 below 2^24 of them),
// the sums round once each.
__device__ __forceinline__ float lower(int d1, int d0) {
    return fmaf(__int_as_float(d1), 256.f, -257.f * MAGIC) + __int_as_float(d0);
}
__device__ __forceinline__ float upper(int d2) { return fmaf(__int_as_float(d2), 65536.f, -65536.f * MAGIC); }

// d = a (16 x 32) * b (32 x 8) + c.  A_S8: a is signed like b (the query's top digit); else a holds unsigned digits.
template <bool A_S8>
__device__ __forceinline__ void mma(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, int c0, int c1, int c2, int c3) {
    if (A_S8)
        asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c0), "r"(c1), "r"(c2), "r"(c3));
    else
        asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c0), "r"(c1), "r"(c2), "r"(c3));
}
// the same, with the accumulator started (FIRST) at the pattern that reads as MAGIC + sum
template <bool A_S8, bool FIRST>
__device__ __forceinline__ void mma(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (FIRST)
        mma<A_S8>(d, a, b0, b1, MAGIC_BITS, MAGIC_BITS, MAGIC_BITS, MAGIC_BITS);
    else
        mma<A_S8>(d, a, b0, b1, d[0], d[1], d[2], d[3]);
}
// bytes of four words, transposed: o[i] = byte i of a, b, c, d
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&o)[4]) {
    const uint32_t t0 = __byte_perm(a, b, 0x5140), t1 = __byte_perm(c, d, 0x5140);
    const uint32_t t2 = __byte_perm(a, b, 0x7362), t3 = __byte_perm(c, d, 0x7362);
    o[0] = __byte_perm(t0, t1, 0x5410), o[1] = __byte_perm(t0, t1, 0x7632);
    o[2] = __byte_perm(t2, t3, 0x5410), o[3] = __byte_perm(t2, t3, 0x7632);
}

// Shared-memory offset of 16-byte chunk j of row r; the swizzles spread the chunks that eight lanes read together
// (K: rows 2i and 2i + 1; V: rows 0, 2, 4, 6) over all banks.
template <bool INT4>
__device__ __forceinline__ int k_off(int r, int j) {
    return INT4 ? r * 64 + j * 16 : r * 128 + ((j ^ ((r & 1) << 2)) << 4);
}
template <bool INT4>
__device__ __forceinline__ int v_off(int r, int j) {
    const int x = ((r >> 1) & 3) << 1;
    return INT4 ? (r >> 1) * 128 + ((((r & 1) << 2 | j) ^ x) << 4) : r * 128 + ((j ^ x) << 4);
}

// Before the blocks all columns of a unit are worked on at once, by TPC neighbouring threads each: thread j of a column has
// the 16-byte chunks j, j + TPC, ... of its rows.  (A column a warp, several in turn: 5 us a unit instead of 2.)
template <int TPC>
struct RowPart {
    static constexpr int N = TREE_DIM / 4 / TPC;
    float4 x[N];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void load(const float* row, int j) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = __ldg(reinterpret_cast<const float4*>(row) + j + TPC * i);
    }
};

// Writes a query row as digits of column `col` into the A fragments qf[k-step * 3 + digit][lane], and returns the row's
// largest magnitude.
template <bool INT4, int TPC>
__device__ __forceinline__ float query_digits(const RowPart<TPC>& q, int col, int j, uint4 (*qf)[32]) {
    float a = TINY;
#pragma unroll
    for (int i = 0; i < q.N; ++i)
        a = fmaxf(a, fmaxf(fmaxf(fabsf(q.x[i].x), fabsf(q.x[i].y)), fmaxf(fabsf(q.x[i].z), fabsf(q.x[i].w))));
#pragma unroll
    for (int o = TPC / 2; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const float inv = Q_TOP / a;
    const int tl = (col & 7) * 4, hi = col >> 3;
#pragma unroll
    for (int i = 0; i < q.N; ++i) {
        const float4 x = q.x[i];
        const int ch = j + TPC * i;
        const int f[4] = {__float2int_rn(x.x * inv), __float2int_rn(x.y * inv), __float2int_rn(x.z * inv), __float2int_rn(x.w * inv)};
#pragma unroll
        for (int d = 0; d < 3; ++d) {
            const uint32_t v0 = (f[0] >> 8 * d) & 255, v1 = (f[1] >> 8 * d) & 255, v2 = (f[2] >> 8 * d) & 255, v3 = (f[3] >> 8 * d) & 255;
            if (INT4) {   // dims 32 c + 8 s + 2 i in the first word of a k-step, + 1 in the second
                const int s = (ch >> 1) & 3, cc = ch >> 3;
                uint16_t* w = reinterpret_cast<uint16_t*>(&qf[s * 3 + d][tl + cc]);
                w[2 * hi + (ch & 1)] = (uint16_t)(v0 | v2 << 8);
                w[2 * (2 + hi) + (ch & 1)] = (uint16_t)(v1 | v3 << 8);
            } else {      // dims 64 (s / 2) + 16 c + 8 (s % 2) + i, + 4 in the second
                const int s = 2 * (ch >> 4) + ((ch >> 1) & 1), cc = (ch >> 2) & 3;
                reinterpret_cast<uint32_t*>(&qf[s * 3 + d][tl + cc])[2 * (ch & 1) + hi] = v0 | v1 << 8 | v2 << 16 | v3 << 24;
            }
        }
    }
    return a;
}

// Attention of one query over its line's drafted keys (`line`: bits of its nodes), fp32, four keys at a time.  load()
// starts the first four rows' loads; attend() is called by whole warps.
template <int TPC>
struct DraftPart {
    RowPart<TPC> k[4], v[4], o;
    float m, l;
    __device__ __forceinline__ void load(const TreeParams& p, int b, int h, int j, unsigned long long line) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (line) {
                const size_t r = (((size_t)b * p.N + __ffsll(line) - 1) * p.hk + h) * TREE_DIM;
                k[n].load(p.k_new + r, j), v[n].load(p.v_new + r, j);
            } else {
                k[n].zero(), v[n].zero();
            }
            line &= line - 1;
        }
    }
    __device__ __forceinline__ void attend(const TreeParams& p, int b, int h, int j, const RowPart<TPC>& q, unsigned long long line) {
        constexpr float k2 = SCORE_SCALE * LOG2E;
        m = NONE, l = 0.f;
        o.zero();
        while (__any_sync(0xffffffffu, line != 0)) {
            float sc[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                sc[n] = 0.f;
#pragma unroll
                for (int i = 0; i < q.N; ++i)
                    sc[n] += (q.x[i].x * k2) * k[n].x[i].x + (q.x[i].y * k2) * k[n].x[i].y + (q.x[i].z * k2) * k[n].x[i].z +
                             (q.x[i].w * k2) * k[n].x[i].w;
            }
#pragma unroll
            for (int e = TPC / 2; e >= 1; e >>= 1)
#pragma unroll
                for (int n = 0; n < 4; ++n) sc[n] += __shfl_xor_sync(0xffffffffu, sc[n], e);
            float mn = m;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (!line) sc[n] = -INFINITY;
                line &= line - 1;
                mn = fmaxf(mn, sc[n]);
            }
            float f = ex2(m - mn);
            l *= f;
#pragma unroll
            for (int i = 0; i < q.N; ++i) o.x[i].x *= f, o.x[i].y *= f, o.x[i].z *= f, o.x[i].w *= f;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                f = ex2(sc[n] - mn);
                l += f;
#pragma unroll
                for (int i = 0; i < q.N; ++i) {
                    o.x[i].x = fmaf(f, v[n].x[i].x, o.x[i].x), o.x[i].y = fmaf(f, v[n].x[i].y, o.x[i].y);
                    o.x[i].z = fmaf(f, v[n].x[i].z, o.x[i].z), o.x[i].w = fmaf(f, v[n].x[i].w, o.x[i].w);
                }
            }
            m = mn;
            if (__any_sync(0xffffffffu, line != 0)) load(p, b, h, j, line);
        }
    }
};

// The many-units kernel (rswa_ranges.cu): its partial results' bytes, its launch.
size_t ranges_part_bytes();
cudaError_t launch_ranges(TreeParams& p, bool int4, cudaStream_t st);

}  // namespace focr
