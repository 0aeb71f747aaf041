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
//
// Both products run on the integer tensor cores (mma.sync m16n8k32, exact s32 sums) with the cache's codes as they
// lie in memory: nothing is dequantised.  A "column" is one query head of one node.
//   scores    A query row is written as three 8-bit digits of a fixed-point number, q = (max|q| / 8323072) * (65536 d2
//             + 256 d1 + d0), d2 signed, so it is off by half a step of 2^-23 max|q|.  Three products of the digits
//             with the key codes give the exact integer dot; the key's scale, the query's step and log2(e) / sqrt(128)
//             follow in fp32.
//   softmax   online over blocks of 64 keys, base 2.
//   values    out needs sum_j e_j vs_j vc_j.  A block's products of weight and value scale, e_j vs_j, are formed in fp32 and
//             written as three unsigned digits relative to the column's largest one of the block (step 2^-23 of it), so
//             keys that the column does not see, and large values of little weight, cost the others nothing; the three
//             integer sums over the 64 keys are exact, join in fp32 and are added to the fp32 accumulator with the
//             block's factor.  (One bound for all columns, largest weight x largest value scale: 1 to 3% faster, and
//             wrong by any factor where the two belong to different keys.)
//   No sum can wrap or leave a float's exact integers: |sum| <= 128 * 128 * 255 < 2^22, so accumulators start at the
//   bit pattern of 1.5 * 2^23 and are read back as floats by one subtraction.
// Against 64 bits the result is off by 3e-7 of its norm for normal rows (fp32 matrix products and softmax: 2e-7 to 3e-6,
// growing with the number of keys, which this does not).  Where the values cancel, the error is relative to the largest
// product in a block, not to what is left of the sum.
//
// Work split: a unit is one kv head of one sequence with up to 16 columns; its keys are blocks of 64 (reference rows,
// then the ring).  This kernel gives a unit to a cluster of S CTAs, which take its blocks in turn by pairs of warps, each
// pair with its own copies in flight (cp.async into its part of shared memory: the next block's K loads while P V runs,
// its V while Q K runs).  In a pair each warp has the scores of half the keys and the values of half the dims, so 128
// registers hold its accumulators and a block's latency is halved (a warp a block: 19.3 us instead of 16.9 for 8 sequences
// x 10 heads x 16 nodes over 289 rows).  Parts are joined through distributed shared memory, each CTA storing into the
// one that answers for a column (loading them instead: 13.6 instead of 13.0 us).  Drafted keys and values stay fp32 and
// are few: all columns walk their lines at once on the CUDA cores, before the blocks.  Long or many units go to
// rswa_ranges.cu.
// 264 B (int8) or 136 B (int4) a key and head have to be read; for the calls that come here latency is the bound: 1
// sequence x 10 heads x 1 node over 289 rows 7.3 us, 8 x 10 x 16 nodes 13.0 us.  The chain is lengths -> lines -> drafted
// rows (2 us), a block's copies and products (2 us), the join of warps and CTAs (2 us).
#include <math.h>

#include "abi_util.h"
#include "cluster.cuh"
#include "common.cuh"
#include "kv_cache.h"
#include "launch_state.h"
#include "rswa_tree.cuh"

namespace focr {
namespace {

constexpr int RD = TREE_DIM, RW = TREE_RING;
constexpr int WARPS = 8, PAIRS = WARPS / 2, PT = 32 * WARPS;   // two warps work on a block

struct Shared {
    uint4 qf[4 * 3][32];               // query digits as A fragments: [k-step * 3 + digit][lane]
    float part[COLS][RD];              // the drafted keys' part
    float got[COLS][RD];               // from rank r of the cluster, the i-th column this CTA answers for: [r * (COLS / S) + i]
    float got_m[COLS], got_l[COLS];
    float part_m[COLS], part_l[COLS];
    uint4 px[PAIRS][2][3][32];         // a pair's weight digits as A fragments: [32 keys][digit][lane]
    float2 mx[PAIRS][2][COLS];         // each warp's largest score of a block, and its largest product of weight and value scale
    float pair_m[PAIRS][COLS], warp_l[WARPS][COLS], pair_f[PAIRS + 1][COLS];   // f: a part's factor (the last: drafted keys)
    float step[COLS];                  // a score in units of log2 is (integer dot) * key scale * step
    int row[COLS];                     // a column's row of the output, -1 without a live node
    int ages[COLS];                    // ring slots younger than this are seen (0 for a column without a node)
    unsigned long long line[TREE_MAX];
    int par[TREE_MAX];
};

// Starts the copies of a warp's 32 rows of a block's codes; a whole block's addresses are one base and constants.
template <bool INT4>
__device__ __forceinline__ void load_codes(uint32_t dst, const uint8_t* src, int rows, bool is_v, int half, int lane) {
    constexpr int CH = INT4 ? 4 : 8, STEP = 32 / CH;   // STEP rows a round: a multiple of 4, so the swizzle repeats
    const int j = lane % CH, r0 = 32 * half + lane / CH;
    if (rows == BLK) {
        const uint8_t* from = src + half * (32 * CH * 16) + lane * 16;
#pragma unroll
        for (int i = 0; i < 32 / STEP; ++i) {
            const int r = r0 + STEP * i;
            cp16(dst + (is_v ? v_off<INT4>(r, j) : k_off<INT4>(r, j)), from + STEP * i * (CH * 16));
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < 32 / STEP; ++i) {
            const int r = r0 + STEP * i;
            cp16(dst + (is_v ? v_off<INT4>(r, j) : k_off<INT4>(r, j)), src + (size_t)min(r, rows - 1) * (CH * 16) + j * 16);
        }
    }
}
__device__ __forceinline__ void load_scales(uint32_t dst, const float* src, int rows, int half, int lane) {
    const int r = 32 * half + lane;
    cp4(dst + 4 * r, src + min(r, rows - 1));
}

// W16: more than eight columns, so both row halves of the MMA tiles are used (8 x 10 x 8 nodes over 289 rows without it 10.7
// us, with it 11.4; over 32768 rows, in ranges, 98 and 111).
template <bool INT4, bool W16>
__global__ void __launch_bounds__(PT, 2) rswa_tree_kernel(const __grid_constant__ TreeParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    using St = Stage<INT4>;
    constexpr int TPC = PT / COLS;   // threads that prepare a column
    Shared& sh = *reinterpret_cast<Shared*>(smem + PAIRS * St::BYTES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, c = lane & 3;
    const int rank = p.S > 1 ? (int)cluster_rank() : 0;
    const int pair = warp >> 1, half = warp & 1;
    uint8_t* stage = smem + pair * St::BYTES;
    const uint32_t st = smem_u32(stage);
    pdl_wait();
    const int per = p.hk * p.groups, b = (int)(blockIdx.x / p.S) / per, unit = (int)(blockIdx.x / p.S) % per;
    const int h = unit / p.groups, col0 = unit % p.groups * COLS, cols = min(COLS, p.N * p.G - col0);
    // ---- everything that depends on nothing, at once: lengths, parents, queries
    const int R = __ldg(p.ref_len + b), n = __ldg(p.n_gen + b), L = p.n_nodes ? __ldg(p.n_nodes + b) : p.N;
    const int par = tid < p.N && p.parent ? __ldg(p.parent + (size_t)b * p.N + tid) : tid - 1;
    const int col = tid / TPC, j = tid % TPC, node = (col0 + col) / p.G;
    RowPart<TPC> q;
    q.zero();
    if (col < cols) q.load(p.q + (((size_t)b * p.N + node) * p.hq + h * p.G + (col0 + col) % p.G) * RD, j);
    const bool lengths = R >= 0 && R <= p.ref.cap && n >= 0 && L >= 0 && L <= p.N;
    if (tid < p.N) sh.par[tid] = par;
    const bool bad = __syncthreads_or(!lengths || (tid < L && (par < -1 || par >= tid)));
    // ---- this CTA's blocks of the unit; its first ones are on their way while the query is prepared
    const int nref = bad ? 0 : (R + BLK - 1) / BLK, nring = bad ? 0 : (min(n, RW) + BLK - 1) / BLK, nblk = nref + nring;
    if (bad) {
        const int live = L < 0 || L > p.N ? p.N : L;
        for (int c = rank; c < cols; c += p.S) {
            const int x = (col0 + c) / p.G;
            if (x < live && tid < RD)
                p.out[(((size_t)b * p.N + x) * p.hq + h * p.G + (col0 + c) % p.G) * RD + tid] = __int_as_float(0x7fc00000);
        }
        return;
    }
    if (col0 / p.G >= L) return;   // no live node in this group, in any CTA of the cluster
    if (p.S > 1) cluster_arrive();
    const size_t ref0 = ((size_t)b * p.hk + h) * p.ref.cap, ring0 = ((size_t)b * p.hk + h) * RW;
    // Rows of block i that hold a key (later ones are read from the last such row and masked), and its copies' start.
    auto rows_of = [&](int i) { return min(BLK, i >= nref ? min(n, RW) - (i - nref) * BLK : R - i * BLK); };
    auto fetch_k = [&](int i) {
        const KvView& v = i >= nref ? p.ring : p.ref;
        const size_t row = (i >= nref ? ring0 - nref * BLK : ref0) + (size_t)i * BLK;
        const int rows = rows_of(i);
        load_codes<INT4>(st, v.k + row * St::ROW, rows, false, half, lane);
        load_scales(st + St::KS, v.ks + row, rows, half, lane);
        load_scales(st + St::VS, v.vs + row, rows, half, lane);
    };
    auto fetch_v = [&](int i) {
        const KvView& v = i >= nref ? p.ring : p.ref;
        const size_t row = (i >= nref ? ring0 - nref * BLK : ref0) + (size_t)i * BLK;
        load_codes<INT4>(st + St::V, v.v + row * St::ROW, rows_of(i), true, half, lane);
    };
    int blk = rank * PAIRS + pair;
    const int stride = p.S * PAIRS;
    if (blk < nblk) fetch_k(blk);
    cp_commit();
    if (blk < nblk) fetch_v(blk);
    cp_commit();

    // ---- lines of the tree
    if (tid < L) {
        unsigned long long line = 0;
        for (int j = tid; j >= 0; j = sh.par[j]) line |= 1ull << j;
        sh.line[tid] = line;
    }
    __syncthreads();
    // ---- query digits, per-column constants, and the drafted keys' part (a CTA of the cluster takes every S-th column's)
    {
        const bool live = col < cols && node < L;
        if (!live) q.zero();
        const unsigned long long line = live && col % p.S == rank ? sh.line[node] : 0ull;
        DraftPart<TPC> d;
        d.load(p, b, h, j, line);
        const float a = query_digits<INT4>(q, col, j, sh.qf);
        if (j == 0) {
            sh.row[col] = live ? node * p.hq + h * p.G + (col0 + col) % p.G : -1;
            sh.ages[col] = live ? min(n, RW - __popcll(sh.line[node])) : 0;
            sh.step[col] = a / Q_TOP * (SCORE_SCALE * LOG2E * (INT4 ? 1.f / 16.f : 1.f));
        }
        d.attend(p, b, h, j, q, line);
#pragma unroll
        for (int i = 0; i < q.N; ++i) reinterpret_cast<float4*>(sh.part[col])[j + TPC * i] = d.o.x[i];
        if (j == 0) sh.part_m[col] = d.m, sh.part_l[col] = d.l;
    }
    __syncthreads();

    // ---- the blocks.  A warp of a pair has the scores of 32 of the 64 keys, and of the values the dims 16 g + t with t in
    // its half of the 16 tiles.  Lane (gr, c) has columns gr and gr + 8 and, of each 8 keys, keys 2 c and 2 c + 1.
    constexpr int HALVES = W16 ? 2 : 1, VALS = 2 * HALVES;
    float O[8][VALS];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int j = 0; j < VALS; ++j) O[t][j] = 0.f;
    float run_m[HALVES], run_l[HALVES], step[HALVES];
    int ages[HALVES];
#pragma unroll
    for (int e = 0; e < HALVES; ++e) {
        run_m[e] = NONE, run_l[e] = 0.f;
        step[e] = sh.step[gr + 8 * e], ages[e] = sh.ages[gr + 8 * e];
    }
    for (; blk < nblk; blk += stride) {
        cp_wait<1>();
        check_scale(stage + St::KS, stage + St::VS, 32 * half + lane);
        __syncwarp();
        // scores of the warp's own keys, without the column's step: T[j][..] for keys 8 j + 2 c, + 1 of its 32
        float T[4][VALS], vs[4][2];
        const int rows = rows_of(blk), ring_slot = blk >= nref ? (blk - nref) * BLK : -1;
        const bool unmasked = rows == BLK && ring_slot < 0;
#pragma unroll
        for (int jp = 0; jp < 2; ++jp) {
            __syncwarp();   // keeps the second part's loads from being drawn ahead of the first part's use of registers
            int acc[2][3][4];
            uint32_t kb[2][8];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 32 * half + 16 * jp + 8 * j + gr;
                if (INT4) {
                    const uint4 w = lds128(stage + k_off<true>(r, c));
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) kb[j][2 * i] = (u[i] << 4) & 0xF0F0F0F0u, kb[j][2 * i + 1] = u[i] & 0xF0F0F0F0u;
                } else {
                    const uint4 w0 = lds128(stage + k_off<false>(r, c)), w1 = lds128(stage + k_off<false>(r, c + 4));
                    kb[j][0] = w0.x, kb[j][1] = w0.y, kb[j][2] = w0.z, kb[j][3] = w0.w;
                    kb[j][4] = w1.x, kb[j][5] = w1.y, kb[j][6] = w1.z, kb[j][7] = w1.w;
                }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int d = 0; d < 3; ++d) {
                    const uint4 q4 = lds128(&sh.qf[s * 3 + d][lane]);
                    const uint32_t a[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t b0 = kb[j][2 * s], b1 = kb[j][2 * s + 1];
                        if (d == 2)
                            s == 0 ? mma<true, true>(acc[j][d], a, b0, b1) : mma<true, false>(acc[j][d], a, b0, b1);
                        else
                            s == 0 ? mma<false, true>(acc[j][d], a, b0, b1) : mma<false, false>(acc[j][d], a, b0, b1);
                    }
                }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int jj = 2 * jp + j, key = 32 * half + 8 * jj + 2 * c;
                const float2 ks = *reinterpret_cast<const float2*>(stage + St::KS + 4 * key);
                const float2 v2 = *reinterpret_cast<const float2*>(stage + St::VS + 4 * key);
                vs[jj][0] = v2.x, vs[jj][1] = v2.y;
#pragma unroll
                for (int i = 0; i < VALS; ++i)
                    T[jj][i] = (upper(acc[j][2][i]) + lower(acc[j][1][i], acc[j][0][i])) * (i & 1 ? ks.y : ks.x);
                if (!unmasked) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bool in = key + i < rows;
#pragma unroll
                        for (int e = 0; e < HALVES; ++e) {
                            const bool seen = in && (ring_slot < 0 || ((n - 1 - ring_slot - key - i) & (RW - 1)) < ages[e]);
                            if (!seen) T[jj][2 * e + i] = -INFINITY;
                        }
                    }
                }
            }
        }
        __syncwarp();
        // the next block's K and scales take this block's place
        const int next = blk + stride;
        if (next < nblk) fetch_k(next);
        cp_commit();
        // softmax of the block: each warp's weights relative to its own largest score, then both warps' products of weight and
        // value scale as digits, relative to a column's largest one of the block
        float own[HALVES], sum[HALVES], top[HALVES];
#pragma unroll
        for (int e = 0; e < HALVES; ++e) {
            float tm = fmaxf(T[0][2 * e], T[0][2 * e + 1]);
#pragma unroll
            for (int j = 1; j < 4; ++j) tm = fmaxf(tm, fmaxf(T[j][2 * e], T[j][2 * e + 1]));
            tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 1));
            tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 2));
            const bool any = tm != -INFINITY;
            const float mb = any ? tm * step[e] : 0.f;
            own[e] = any ? mb : -INFINITY, sum[e] = 0.f, top[e] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float w = ex2(fmaf(T[j][2 * e + i], step[e], -mb));
                    sum[e] += w;
                    T[j][2 * e + i] = w * vs[j][i];   // 0 for a key that the column does not see
                    top[e] = fmaxf(top[e], T[j][2 * e + i]);
                }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
                sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], o);
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], o));
            }
            if (c == 0) sh.mx[pair][half][gr + 8 * e] = make_float2(own[e], top[e]);
        }
        named_bar_sync(1 + pair, 64);
        float alpha[HALVES], gain[HALVES];
        uint32_t pd[3][4];   // digits of the warp's keys as an A fragment
#pragma unroll
        for (int e = 0; e < HALVES; ++e) {
            const float2 other = sh.mx[pair][half ^ 1][gr + 8 * e];
            const float both = fmaxf(own[e], other.x);
            const bool any = both != -INFINITY;
            const float mb = any ? both : 0.f;
            const float r = ex2(own[e] - mb);   // 0 for a warp whose keys the column does not see
            const float most = fmaxf(fmaxf(top[e] * r, other.y * ex2(other.x - mb)), TINY);
            const float f = r * (P_TOP / most);
            uint32_t u[4][2];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) u[j][i] = __float_as_uint(fmaf(T[j][2 * e + i], f, P_MAGIC));
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint32_t t0 = __byte_perm(u[2 * g][0], u[2 * g][1], 0x5140), t1 = __byte_perm(u[2 * g + 1][0], u[2 * g + 1][1], 0x5140);
                const uint32_t t2 = __byte_perm(u[2 * g][0], u[2 * g][1], 0x0062), t3 = __byte_perm(u[2 * g + 1][0], u[2 * g + 1][1], 0x0062);
                // fragment words: (row gr, keys g = 0), (row gr + 8, g = 0), (gr, g = 1), (gr + 8, g = 1)
                pd[0][2 * g + e] = __byte_perm(t0, t1, 0x5410);
                pd[1][2 * g + e] = __byte_perm(t0, t1, 0x7632);
                pd[2][2 * g + e] = __byte_perm(t2, t3, 0x5410);
            }
            const float mn = any ? fmaxf(run_m[e], mb) : run_m[e];
            alpha[e] = ex2(run_m[e] - mn);
            const float beta = any ? ex2(mb - mn) : 0.f;
            run_l[e] = run_l[e] * alpha[e] + beta * (r * sum[e]);
            gain[e] = beta * most * ((INT4 ? 1.f / 16.f : 1.f) / P_TOP);
            run_m[e] = mn;
        }
#pragma unroll
        for (int d = 0; d < 3; ++d) {
            if (!W16) pd[d][1] = pd[d][3] = 0u;
            sh.px[pair][half][d][lane] = make_uint4(pd[d][0], pd[d][1], pd[d][2], pd[d][3]);
        }
        cp_wait<1>();
        named_bar_sync(1 + pair, 64);   // both warps' digits and values are there
        uint32_t pa[2][3][4];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int d = 0; d < 3; ++d) {
                const uint4 w = lds128(&sh.px[pair][kk][d][lane]);
                pa[kk][d][0] = w.x, pa[kk][d][1] = w.y, pa[kk][d][2] = w.z, pa[kk][d][3] = w.w;
            }
        // values: dim 16 gr + 8 half + t of tile t, from the bytes of the lane's sixteen keys
        uint32_t vb[2][8][2];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int r0 = 32 * kk + 16 * g + 2 * c;
                uint32_t o[4];
                if (INT4) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = *reinterpret_cast<const uint32_t*>(stage + St::V + v_off<true>(r0 + (i & 1) + 8 * (i >> 1), gr >> 1) + (gr & 1) * 8 + 4 * half);
                    transpose4(w[0], w[1], w[2], w[3], o);
#pragma unroll
                    for (int i = 0; i < 4; ++i) vb[kk][2 * i][g] = (o[i] << 4) & 0xF0F0F0F0u, vb[kk][2 * i + 1][g] = o[i] & 0xF0F0F0F0u;
                } else {
                    uint2 w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = *reinterpret_cast<const uint2*>(stage + St::V + v_off<false>(r0 + (i & 1) + 8 * (i >> 1), gr) + 8 * half);
                    transpose4(w[0].x, w[1].x, w[2].x, w[3].x, o);
#pragma unroll
                    for (int i = 0; i < 4; ++i) vb[kk][i][g] = o[i];
                    transpose4(w[0].y, w[1].y, w[2].y, w[3].y, o);
#pragma unroll
                    for (int i = 0; i < 4; ++i) vb[kk][4 + i][g] = o[i];
                }
            }
        named_bar_sync(1 + pair, 64);   // both have read the values: the next block's take their place
        if (next < nblk) fetch_v(next);
        cp_commit();
        bool moved = false;   // a new maximum rescales what there is; mostly there is none
#pragma unroll
        for (int e = 0; e < HALVES; ++e) moved |= alpha[e] != 1.f;
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int i = 0; i < VALS; ++i) O[t][i] *= alpha[i >> 1];
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            int acc[3][4];
#pragma unroll
            for (int d = 0; d < 3; ++d) mma<false, true>(acc[d], pa[0][d], vb[0][t][0], vb[0][t][1]);
#pragma unroll
            for (int d = 0; d < 3; ++d) mma<false, false>(acc[d], pa[1][d], vb[1][t][0], vb[1][t][1]);
#pragma unroll
            for (int i = 0; i < VALS; ++i)
                O[t][i] = fmaf(upper(acc[2][i]), gain[i >> 1], fmaf(lower(acc[1][i], acc[0][i]), gain[i >> 1], O[t][i]));
        }
    }
    // ---- join the pairs
    cp_wait<0>();
    named_bar_sync(1 + pair, 64);
    {
        float* po = reinterpret_cast<float*>(stage);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < HALVES; ++e)
                po[part_at(gr + 8 * e, 32 * c + 8 * half + t)] = O[t][2 * e], po[part_at(gr + 8 * e, 32 * c + 16 + 8 * half + t)] = O[t][2 * e + 1];
        if (c == 0) {
#pragma unroll
            for (int e = 0; e < HALVES; ++e) {
                if (half == 0) sh.pair_m[pair][gr + 8 * e] = run_m[e];
                sh.warp_l[warp][gr + 8 * e] = run_l[e];
            }
        }
    }
    __syncthreads();
    const int slog = 31 - __clz(p.S);
    if (p.S > 1) cluster_wait();   // every CTA of the cluster runs: its shared memory may be written
    if (tid < cols) {   // a column's maximum, the parts' factors, its sum
        const int col = tid;
        const float pm = sh.part_m[col];
        float M = pm;
#pragma unroll
        for (int w = 0; w < PAIRS; ++w) M = fmaxf(M, sh.pair_m[w][col]);
        float f = ex2(pm - M), l = f * sh.part_l[col];
        sh.pair_f[PAIRS][col] = f;
#pragma unroll
        for (int w = 0; w < PAIRS; ++w) {
            f = ex2(sh.pair_m[w][col] - M);
            sh.pair_f[w][col] = f;
            l = fmaf(f, sh.warp_l[2 * w][col] + sh.warp_l[2 * w + 1][col], l);
        }
        sh.part_m[col] = M, sh.part_l[col] = l;
        if (p.S > 1) {
            const int at = rank * (COLS >> slog) + (col >> slog);
            st_cluster(&sh.got_m[at], col & (p.S - 1), M);
            st_cluster(&sh.got_l[at], col & (p.S - 1), l);
        }
    }
    __syncthreads();
    float* out = p.out + (size_t)b * p.N * p.hq * RD + tid % RD;
#pragma unroll 4
    for (int col = tid / RD; col < cols; col += PT / RD) {
        const int d = tid % RD;
        float o = sh.pair_f[PAIRS][col] * sh.part[col][d];
#pragma unroll
        for (int w = 0; w < PAIRS; ++w)
            o = fmaf(sh.pair_f[w][col], reinterpret_cast<const float*>(smem + w * St::BYTES)[part_at(col, d)], o);
        if (p.S > 1) {
            st_cluster(&sh.got[rank * (COLS >> slog) + (col >> slog)][d], col & (p.S - 1), o);
        } else {
            if (sh.row[col] >= 0) out[sh.row[col] * RD] = o / sh.part_l[col];
        }
    }
    if (p.S > 1) {
        // ---- join the CTAs of the cluster: a column's parts have been stored in the CTA that answers for it
        cluster_sync();
        for (int col = rank + tid / RD * p.S; col < cols; col += PT / RD * p.S) {
            const int at = col >> slog, step = COLS >> slog;
            float M = NONE, l = 0.f, o = 0.f;
            for (int r = 0; r < p.S; ++r) M = fmaxf(M, sh.got_m[r * step + at]);
            for (int r = 0; r < p.S; ++r) {
                const float f = ex2(sh.got_m[r * step + at] - M);
                l = fmaf(f, sh.got_l[r * step + at], l);
                o = fmaf(f, sh.got[r * step + at][tid % RD], o);
            }
            if (sh.row[col] >= 0) out[sh.row[col] * RD] = o / l;
        }
    }
}

// How a call is split, from its sizes alone: a cluster for each unit, of as many CTAs as give every pair of warps a block
// and the device no more than two CTAs per SM; or ranges (rswa_ranges.cu), which use the whole device whatever the units
// are, but cost a second kernel and longer beginnings.  Clusters are taken up to 6 blocks a pair while they leave at most
// one CTA to an SM, else up to 4.  Measured, clusters against ranges (us, int8): 1 sequence x 10 heads x 1 node over 3900
// / 8000 / 12000 rows (2, 4, 6 blocks a pair) 9.5 / 14.0 / 18.3 against 12.7 / 14.8 / 16.5; 1 x 10 x 16 nodes over 8000 /
// 12000 rows 17.5 / 22.6 against 20.7 / 22.0; 3 x 10 x 4 over 3000 / 8000 rows (3, 8) 13.5 / 20.9 against 14.8 / 20.0;
// 8 x 10 x 16 over 896 / 1792 rows (2, 4 blocks; 160 CTAs) 16.7 / 22.6 against 20.0 / 23.8; 32 x 10 x 14 over 896 rows
// (4; 320 CTAs) 34.9 against 34.1.
struct TreePlan {
    int groups, S;
    bool ranges;
};
TreePlan tree_plan(int B, int N, int heads_q, int heads, int cap) {
    const int sms = device_sms() > 0 ? device_sms() : 148;
    TreePlan pl;
    pl.groups = (N * (heads_q / heads) + COLS - 1) / COLS;
    const int64_t units = (int64_t)B * heads * pl.groups;
    const int blocks = (cap + BLK - 1) / BLK + RW / BLK;
    pl.S = 1;
    while (pl.S < 8 && pl.S * PAIRS < blocks) pl.S *= 2;
    while (pl.S > 1 && units * pl.S > 2 * sms) pl.S /= 2;
    pl.ranges = blocks > (units * pl.S > sms ? 4 : 6) * pl.S * PAIRS;
    return pl;
}

template <bool INT4, bool W16>
cudaError_t launch_tree(TreeParams& p, const TreePlan& pl, cudaStream_t st) {
    const void* fn = (const void*)rswa_tree_kernel<INT4, W16>;
    const size_t smem = PAIRS * Stage<INT4>::BYTES + sizeof(Shared);
    const cudaError_t e = once_per_device(fn, [&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    p.groups = pl.groups, p.S = pl.S;
    void* args[] = {&p};
    return launch_kernel(fn, dim3((unsigned)p.B * p.hk * p.groups * p.S), dim3(PT), smem, p.S, args, st);
}

}  // namespace
}  // namespace focr

extern "C" size_t focr_rswa_tree_workspace_bytes(int32_t B, int32_t N, int32_t heads_q, int32_t heads, int32_t ref_cap) {
    using namespace focr;
    if (B < 1 || N < 1 || heads < 1 || heads_q < heads || heads_q > FOCR_HEADS_MAX || B > FOCR_RSWA_B_MAX ||
        ref_cap > FOCR_RSWA_RCAP_MAX || N > TREE_MAX)
        return 0;
    return tree_plan(B, N, heads_q, heads, ref_cap).ranges ? ranges_part_bytes() : 0;
}

extern "C" focr_status focr_rswa_tree(const float* q, const float* k_new, const float* v_new, int32_t B, int32_t N,
                                      int32_t heads_q, const focr_kv_cache* ref, const int32_t* ref_len,
                                      const focr_kv_cache* ring, const int32_t* n_gen, const int32_t* parent,
                                      const int32_t* n_nodes, float* out, void* workspace, size_t ws_bytes, void* stream) {
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
    p.q = q, p.k_new = k_new, p.v_new = v_new, p.ref_len = ref_len, p.n_gen = n_gen, p.parent = parent, p.n_nodes = n_nodes;
    const TreePlan pl = tree_plan(B, N, heads_q, ref->heads, ref->cap);
    const size_t need = focr_rswa_tree_workspace_bytes(B, N, heads_q, ref->heads, ref->cap);
    if (need && (!workspace || misaligned(workspace, 256) || ws_bytes < need))
        return reportf(FOCR_ERR_INVALID_ARG, "workspace of %zu bytes (256-byte aligned) is needed, got %zu", need, ws_bytes);
    const size_t qb = 4ull * B * N * heads_q * RD, kb = 4ull * B * N * ref->heads * RD, tab = 4ull * B;
    const Span outs[] = {{out, qb}, {need ? workspace : nullptr, need}};
    Span a[4], b[4];
    cache_spans(ref, a);
    cache_spans(ring, b);
    const Span in[] = {{q, qb}, {k_new, kb}, {v_new, kb}, {ref_len, tab}, {n_gen, tab}, {parent, tab * N}, {n_nodes, tab},
                       a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    if (outputs_overlap(outs, 2, in, 15)) return report_error(FOCR_ERR_INVALID_ARG, "out or workspace overlaps another argument");
    p.out = out, p.B = B, p.N = N, p.hq = heads_q, p.hk = ref->heads, p.G = G;
    p.part = reinterpret_cast<float*>(workspace);
    const bool wide = N * G > 8, int4 = ref->type == FOCR_W_INT4;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = pl.ranges ? (p.groups = pl.groups, launch_ranges(p, int4, st))
                            : int4  ? (wide ? launch_tree<true, true>(p, pl, st) : launch_tree<true, false>(p, pl, st))
                                  : (wide ? launch_tree<false, true>(p, pl, st) : launch_tree<false, false>(p, pl, st));
    return report_launch(e, "rswa_tree_kernel");
}
