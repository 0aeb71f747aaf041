// What the two kernels of the tree attention share (rswa_tree.cu, rswa_wide.cu).
#pragma once

#include "common.cuh"
#include "kv_cache.h"

namespace focr {

constexpr int TREE_DIM = FOCR_RSWA_DIM, TREE_RING = FOCR_RSWA_RING;
constexpr int TREE_MAX = FOCR_TREE_NODES_MAX;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float SCORE_SCALE = 0.08838834764831845f;   // 1 / sqrt(128)
constexpr float Q_TOP = 8323072.f;              // 127 * 2^16: the largest fixed-point query value
constexpr float P_TOP = 16711680.f;             // 255 * 2^16: the largest fixed-point weight
constexpr float MAGIC = 12582912.f;             // 1.5 * 2^23
constexpr int MAGIC_BITS = 0x4B400000;
constexpr float NONE = -1e30f;                  // running maximum of a column that has seen no key
constexpr float TINY = 1e-30f;                  // magnitudes below this share its step

struct TreeParams {
    const float *q, *k_new, *v_new;
    KvView ref, ring;
    const int32_t *ref_len, *n_gen, *parent, *n_nodes;
    float* out;
    int B, N, hq, hk, G, S, groups;   // clusters: S CTAs each, groups of 16 columns per kv head
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

// 65536 d2 + 256 d1 + d0 of three integer accumulators that started at MAGIC_BITS (so they read as MAGIC + sum), as two
// parts: lower() + upper().  The products with the constants are exact (multiples of 256 and 65536 below 2^24 of them),
// the sums round once each.
__device__ __forceinline__ float lower(int d1, int d0) {
    return fmaf(__int_as_float(d1), 256.f, -257.f * MAGIC) + __int_as_float(d0);
}
__device__ __forceinline__ float upper(int d2) { return fmaf(__int_as_float(d2), 65536.f, -65536.f * MAGIC); }

// Four drafted rows of a line (`rest`: bits of its nodes, the four lowest are taken), four dims a lane.
__device__ __forceinline__ void draft_load(const TreeParams& p, int b, int h, int lane, unsigned long long& rest, float4 (&k4)[4],
                                           float4 (&v4)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        k4[j] = v4[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (rest) {
            const size_t r = (((size_t)b * p.N + __ffsll(rest) - 1) * p.hk + h) * (TREE_DIM / 4) + lane;
            k4[j] = __ldg(reinterpret_cast<const float4*>(p.k_new) + r);
            v4[j] = __ldg(reinterpret_cast<const float4*>(p.v_new) + r);
        }
        rest &= rest - 1;
    }
}
// Attention of one query over its line's drafted keys, fp32, by a warp; k4, v4 hold the line's first four rows.
struct DraftPart {
    float m, l;
    float4 o;
};
__device__ __forceinline__ DraftPart draft_attend(const TreeParams& p, int b, int h, int lane, float4 q, unsigned long long line,
                                                  float4 (&k4)[4], float4 (&v4)[4]) {
    DraftPart a{NONE, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    const float k2 = SCORE_SCALE * LOG2E;
    q = make_float4(q.x * k2, q.y * k2, q.z * k2, q.w * k2);
    for (bool more = line != 0; more;) {
        float sc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[j] = q.x * k4[j].x + q.y * k4[j].y + q.z * k4[j].z + q.w * k4[j].w;
#pragma unroll
        for (int e = 16; e >= 1; e >>= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) sc[j] += __shfl_xor_sync(0xffffffffu, sc[j], e);
        float mn = a.m;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!line) sc[j] = -INFINITY;
            line &= line - 1;
            mn = fmaxf(mn, sc[j]);
        }
        const float al = ex2(a.m - mn);
        a.l *= al, a.o.x *= al, a.o.y *= al, a.o.z *= al, a.o.w *= al;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float w = ex2(sc[j] - mn);
            a.l += w;
            a.o.x = fmaf(w, v4[j].x, a.o.x), a.o.y = fmaf(w, v4[j].y, a.o.y);
            a.o.z = fmaf(w, v4[j].z, a.o.z), a.o.w = fmaf(w, v4[j].w, a.o.w);
        }
        a.m = mn;
        more = line != 0;
        if (more) {
            unsigned long long rest = line;
            draft_load(p, b, h, lane, rest, k4, v4);
        }
    }
    return a;
}

// The many-units kernel (rswa_wide.cu): its CTAs, its partial results' bytes, its launch.
int wide_ctas();
size_t wide_part_bytes();
cudaError_t launch_wide(TreeParams& p, bool int4, cudaStream_t st);

}  // namespace focr
