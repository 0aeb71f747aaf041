// The tree attention of rswa_tree.cu for many or long units: equal ranges of blocks per CTA.
//
// The mathematics and the fragments are those of rswa_tree.cu.  All units stand in one row, a unit as long as its 64-key
// blocks and BEGIN more for what it costs to begin one, and the row is cut into equal ranges, one per resident CTA (the
// lengths are read on the device, so ragged batches stay balanced).  Units that a cut divides leave partial results in the
// workspace, and a second kernel joins them.  Here a block is one warp's: with no barrier in the loop and 255 registers it
// needs a quarter fewer instructions than two warps a block, which pays once the device is full (217 us against 258 us for
// 8 sequences x 10 heads x 32 nodes over 32768 rows, int8); with few blocks a warp the other form's lower latency wins.
//
// Measured: 8 x 10 x 32 nodes over ragged 32768 rows, int8 (549 MB, 85 us at the copy rate): 210 us from a graph, 239 us called
// on inputs that change; 32 x 10 x 14 columns over ragged 4096 rows, int4 (146 MB, 23 us): 75 us.  A block of 16 columns x 64
// keys takes 192 matrix instructions and some 1590 others (digits taken apart and put together, exponentials, transposed
// values).  No unit is full: over 8192 rows 1.64 of 4 issue slots are used, the tensor pipe 37%, DRAM 34% of the time.  A warp
// does its products and its softmax one after the other, and the two warps of a scheduler overlap too little; registers
// leave no room for a third.  More than 16 columns are several units, each of which copies and takes apart all rows (192 MB
// read for 140 in that profile).  Beginning and ending a unit costs 5 us (13 us with a column a warp at a time and ranges
// that did not count it).  The tensor-memory form of the same products (kind::i8) came to 224 and 125 us when this one
// took 217 and 90: its exponentials wait on tensor-memory loads instead.
#include <math.h>

#include "abi_util.h"
#include "common.cuh"
#include "kv_cache.h"
#include "launch_state.h"
#include "rswa_tree.cuh"

namespace focr {
namespace {

constexpr int RD = TREE_DIM, RW = TREE_RING;
constexpr int WARPS = 4, PT = 32 * WARPS, TPC = PT / COLS;   // TPC: threads that prepare a column
constexpr int JCOLS = 4;                        // columns of a CTA of the joining kernel

// A partial result: 16 columns' maxima, sums and unnormalised outputs.
constexpr int PART_L = COLS, PART_O = 2 * COLS, PART_FLOATS = 2 * COLS + COLS * RD;

// CTAs of the device: two per SM.
int resident() { return 2 * (device_sms() > 0 ? device_sms() : 148); }

struct Shared {
    uint4 qf[4 * 3][32];               // query digits as A fragments: [k-step * 3 + digit][lane]
    float part[COLS][RD];              // the drafted keys' part
    float part_m[COLS], part_l[COLS];
    float warp_m[WARPS][COLS], warp_l[WARPS][COLS], warp_f[WARPS + 1][COLS];   // f: a part's factor (the last: drafted keys)
    float step[COLS];                  // a score in units of log2 is (integer dot) * key scale * step
    int row[COLS];                     // a column's row of the output, -1 without a live node
    int ages[COLS];                    // ring slots younger than this are seen (0 for a column without a node)
    unsigned long long line[TREE_MAX];
    int par[TREE_MAX];
    int scan[WARPS + 4];
};

// A unit's length in the row: what it costs to begin it, in blocks, and its blocks (one at least: the drafted keys need a
// CTA too).  BEGIN = 3 / 6 / 9 made 76.3 / 73.2 / 74.3 us of the int4 call above when it was chosen.
constexpr int BEGIN = 6;
__device__ __forceinline__ int unit_length(const TreeParams& p, int b) {
    const int R = __ldg(p.ref_len + b), n = __ldg(p.n_gen + b);
    if (R < 0 || R > p.ref.cap || n < 0) return BEGIN + 1;
    return BEGIN + max(1, (R + BLK - 1) / BLK + (min(n, RW) + BLK - 1) / BLK);
}
struct Place {   // in the row of all units
    int b, unit, at;   // sequence, unit of the sequence, place in the unit
};
// Sums over all threads of the CTA; the threads' inclusive prefix in `mine`.
template <int NW>
__device__ __forceinline__ int cta_scan(int& mine, int* scan) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, mine, o);
        if (lane >= o) mine += up;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = mine;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < warp) mine += scan[w];
        total += scan[w];
    }
    return total;
}
// The row's length.
__device__ int row_length(const TreeParams& p, int* scan) {
    int mine = 0;
    for (int b = threadIdx.x; b < p.B; b += PT) mine += unit_length(p, b);
    return cta_scan<WARPS>(mine, scan) * p.hk * p.groups;
}
// What is at place `at` of the row.
__device__ Place find_place(const TreeParams& p, int at, int* scan) {
    const int per = p.hk * p.groups;
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += PT) {
        const int b = b0 + threadIdx.x, own = b < p.B ? unit_length(p, b) : 0;
        int sum = own;
        const int total = cta_scan<WARPS>(sum, scan);
        if ((int64_t)(before + total) * per > at) {
            const int64_t first = (int64_t)(before + sum - own) * per;
            if (at >= first && at < first + (int64_t)own * per) scan[WARPS] = b, scan[WARPS + 1] = (int)(at - first), scan[WARPS + 2] = own;
            __syncthreads();
            const Place x{scan[WARPS], scan[WARPS + 1] / scan[WARPS + 2], scan[WARPS + 1] % scan[WARPS + 2]};
            __syncthreads();
            return x;
        }
        before += total;
    }
    return Place{p.B, 0, 0};
}

struct Block {   // where a block's rows are
    const uint8_t *k, *v;
    const float *ks, *vs;
    int rows;        // rows that hold a key; later ones are read from the last such row and masked
    int ring_slot;   // first ring slot, or -1 for reference rows
};

// Starts the copies of a block's codes; a whole block's addresses are one base and constants.
template <bool INT4>
__device__ __forceinline__ void load_codes(uint32_t dst, const uint8_t* src, int rows, bool is_v, int lane) {
    constexpr int CH = INT4 ? 4 : 8, STEP = 32 / CH;   // STEP rows a round: a multiple of 4, so the swizzle repeats
    const int j = lane % CH, r0 = lane / CH;
    if (rows == BLK) {
        const uint8_t* from = src + lane * 16;
#pragma unroll
        for (int i = 0; i < BLK / STEP; ++i) {
            const int r = r0 + STEP * i;
            cp16(dst + (is_v ? v_off<INT4>(r, j) : k_off<INT4>(r, j)), from + STEP * i * (CH * 16));
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < BLK / STEP; ++i) {
            const int r = r0 + STEP * i;
            cp16(dst + (is_v ? v_off<INT4>(r, j) : k_off<INT4>(r, j)), src + (size_t)min(r, rows - 1) * (CH * 16) + j * 16);
        }
    }
}
__device__ __forceinline__ void load_scales(uint32_t dst, const float* src, int rows, int lane) {
    cp4(dst + 4 * lane, src + min(lane, rows - 1));
    cp4(dst + 4 * (lane + 32), src + min(lane + 32, rows - 1));
}

// W16: more than eight columns, so both row halves of the MMA tiles are used.
template <bool INT4, bool W16>
__global__ void __launch_bounds__(PT, 2) rswa_ranges_kernel(const __grid_constant__ TreeParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    using St = Stage<INT4>;
    Shared& sh = *reinterpret_cast<Shared*>(smem + WARPS * St::BYTES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, c = lane & 3;
    uint8_t* stage = smem + warp * St::BYTES;
    const uint32_t st = smem_u32(stage);
    pdl_wait();
    pdl_launch_dependents();
    const int all = row_length(p, sh.scan), per = (all + gridDim.x - 1) / gridDim.x;
    const int from = (int)min((int64_t)blockIdx.x * per, (int64_t)all);
    int left = min(per, all - from);   // of this CTA's range
    if (left == 0) return;
    Place at = find_place(p, from, sh.scan);
    int R = 0, n = 0, L = 0, whole = 0, seq = -1;   // of sequence seq
    bool bad = false;
    while (left > 0) {
    const int b = at.b, h = at.unit / p.groups, col0 = at.unit % p.groups * COLS, cols = min(COLS, p.N * p.G - col0);
    // ---- the query, and what belongs to the sequence if it is another one: lengths and lines of the tree
    const int col = tid / TPC, j = tid % TPC, node = (col0 + col) / p.G;
    RowPart<TPC> q;
    q.zero();
    if (col < cols) q.load(p.q + (((size_t)b * p.N + node) * p.hq + h * p.G + (col0 + col) % p.G) * RD, j);
    if (b != seq) {
        seq = b;
        const int par = tid < p.N && p.parent ? __ldg(p.parent + (size_t)b * p.N + tid) : tid - 1;
        R = __ldg(p.ref_len + b), n = __ldg(p.n_gen + b), L = p.n_nodes ? __ldg(p.n_nodes + b) : p.N;
        whole = unit_length(p, b);
        const bool lengths = R >= 0 && R <= p.ref.cap && n >= 0 && L >= 0 && L <= p.N;
        if (tid < p.N) sh.par[tid] = par;
        bad = __syncthreads_or(!lengths || (tid < L && (par < -1 || par >= tid)));
        if (tid < L && !bad) {
            unsigned long long line = 0;
            for (int i = tid; i >= 0; i = sh.par[i]) line |= 1ull << i;
            sh.line[tid] = line;
        }
        __syncthreads();
    }
    // ---- this CTA's blocks of the unit; its first ones are on their way while the query is prepared
    const int nref = bad ? 0 : (R + BLK - 1) / BLK, nring = bad ? 0 : (min(n, RW) + BLK - 1) / BLK, nblk = nref + nring;
    const int take = min(left, whole - at.at);
    const int first = max(0, at.at - BEGIN), last = max(0, at.at + take - BEGIN);
    if (last > first) {
    const bool head = first == 0, complete = head && last == whole - BEGIN;
    const bool dead = bad || col0 / p.G >= L;   // nothing to compute
    if (bad && head) {
        const int live = L < 0 || L > p.N ? p.N : L;
        for (int c = 0; c < cols; ++c) {
            const int x = (col0 + c) / p.G;
            if (x < live && tid < RD)
                p.out[(((size_t)b * p.N + x) * p.hq + h * p.G + (col0 + c) % p.G) * RD + tid] = __int_as_float(0x7fc00000);
        }
    }
    if (!dead) {
    const int end = min(last, nblk);
    const size_t ref0 = ((size_t)b * p.hk + h) * p.ref.cap, ring0 = ((size_t)b * p.hk + h) * RW;
    auto block_at = [&](int i) {
        Block x;
        const bool ring = i >= nref;
        const KvView& v = ring ? p.ring : p.ref;
        const int from = (ring ? i - nref : i) * BLK;
        const size_t row = (ring ? ring0 : ref0) + from;
        x.k = v.k + row * St::ROW, x.v = v.v + row * St::ROW, x.ks = v.ks + row, x.vs = v.vs + row;
        x.rows = min(BLK, (ring ? min(n, RW) : R) - from);
        x.ring_slot = ring ? from : -1;
        return x;
    };
    int blk = first + warp;
    Block cur{};
    if (blk < end) {
        cur = block_at(blk);
        load_codes<INT4>(st, cur.k, cur.rows, false, lane);
        load_scales(st + St::KS, cur.ks, cur.rows, lane);
        load_scales(st + St::VS, cur.vs, cur.rows, lane);
    }
    cp_commit();
    if (blk < end) load_codes<INT4>(st + St::V, cur.v, cur.rows, true, lane);
    cp_commit();

    // ---- query digits, per-column constants, and the drafted keys' part (the CTA that has the unit's first block has them)
    {
        const bool live = col < cols && node < L;
        if (!live) q.zero();
        const unsigned long long line = live && head ? sh.line[node] : 0ull;
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

    // ---- the blocks.  Lane (gr, c) has columns gr and gr + 8 and, of each 8 keys, keys 2 c and 2 c + 1.
    float O[16][W16 ? 4 : 2];
#pragma unroll
    for (int t = 0; t < 16; ++t)
#pragma unroll
        for (int j = 0; j < (W16 ? 4 : 2); ++j) O[t][j] = 0.f;
    constexpr int HALVES = W16 ? 2 : 1;
    float run_m[HALVES], run_l[HALVES], step[HALVES];
    int ages[HALVES];
#pragma unroll
    for (int e = 0; e < HALVES; ++e) {
        run_m[e] = NONE, run_l[e] = 0.f;
        step[e] = sh.step[gr + 8 * e], ages[e] = sh.ages[gr + 8 * e];
    }
    for (; blk < end; blk += WARPS) {
        cp_wait<1>();
        check_scale(stage + St::KS, stage + St::VS, lane);
        check_scale(stage + St::KS, stage + St::VS, lane + 32);
        __syncwarp();
        // scores, without the column's step: T[j][..] for keys 8 j + 2 c, + 1
        float T[8][W16 ? 4 : 2], vs[8][2];
        const bool unmasked = cur.rows == BLK && cur.ring_slot < 0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            __syncwarp();   // keeps the second half's loads from being drawn ahead of the first half's use of registers
            int acc[4][3][4];
            uint32_t kb[4][8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 32 * half + 8 * j + gr;
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
                    for (int j = 0; j < 4; ++j) {
                        if (s == 0) {
                            if (d == 2)
                                mma<true, true>(acc[j][d], a, kb[j][2 * s], kb[j][2 * s + 1]);
                            else
                                mma<false, true>(acc[j][d], a, kb[j][2 * s], kb[j][2 * s + 1]);
                        } else {
                            if (d == 2)
                                mma<true, false>(acc[j][d], a, kb[j][2 * s], kb[j][2 * s + 1]);
                            else
                                mma<false, false>(acc[j][d], a, kb[j][2 * s], kb[j][2 * s + 1]);
                        }
                    }
                }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = 32 * half + 8 * j + 2 * c, jj = 4 * half + j;
                float2 ks = *reinterpret_cast<const float2*>(stage + St::KS + 4 * key);
                float2 v2 = *reinterpret_cast<const float2*>(stage + St::VS + 4 * key);
                vs[jj][0] = v2.x, vs[jj][1] = v2.y;
#pragma unroll
                for (int i = 0; i < (W16 ? 4 : 2); ++i)
                    T[jj][i] = (upper(acc[j][2][i]) + lower(acc[j][1][i], acc[j][0][i])) * (i & 1 ? ks.y : ks.x);
                if (!unmasked) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bool in = key + i < cur.rows;
#pragma unroll
                        for (int e = 0; e < HALVES; ++e) {
                            const bool seen = in && (cur.ring_slot < 0 || ((n - 1 - cur.ring_slot - key - i) & (RW - 1)) < ages[e]);
                            if (!seen) T[jj][2 * e + i] = -INFINITY;
                        }
                    }
                }
            }
        }
        __syncwarp();
        // the next block's K and scales take this block's place
        const int next = blk + WARPS;
        Block nxt{};
        if (next < end) {
            nxt = block_at(next);
            load_codes<INT4>(st, nxt.k, nxt.rows, false, lane);
            load_scales(st + St::KS, nxt.ks, nxt.rows, lane);
            load_scales(st + St::VS, nxt.vs, nxt.rows, lane);
        }
        cp_commit();
        // softmax of the block; the products of weight and value scale as digits, relative to a column's largest one
        float alpha[HALVES], gain[HALVES];
        uint32_t pd[2][3][4];   // digits as A fragments: [32 keys][digit]
#pragma unroll
        for (int e = 0; e < HALVES; ++e) {
            float tm = T[0][2 * e];
#pragma unroll
            for (int j = 0; j < 8; ++j) tm = fmaxf(tm, fmaxf(T[j][2 * e], T[j][2 * e + 1]));
            tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 1));
            tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 2));
            const bool any = tm != -INFINITY;
            const float mb = any ? tm * step[e] : 0.f;
            float sum = 0.f, top = TINY;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float w = ex2(fmaf(T[j][2 * e + i], step[e], -mb));
                    sum += w;
                    T[j][2 * e + i] = w * vs[j][i];   // 0 for a key that the column does not see
                    top = fmaxf(top, T[j][2 * e + i]);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float inv = P_TOP / top;
            uint32_t u[8][2];
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) u[j][i] = __float_as_uint(fmaf(T[j][2 * e + i], inv, P_MAGIC));
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int j = 4 * kk + 2 * g;
                    const uint32_t t0 = __byte_perm(u[j][0], u[j][1], 0x5140), t1 = __byte_perm(u[j + 1][0], u[j + 1][1], 0x5140);
                    const uint32_t t2 = __byte_perm(u[j][0], u[j][1], 0x0062), t3 = __byte_perm(u[j + 1][0], u[j + 1][1], 0x0062);
                    // fragment words: (row gr, keys g = 0), (row gr + 8, g = 0), (gr, g = 1), (gr + 8, g = 1)
                    pd[kk][0][2 * g + e] = __byte_perm(t0, t1, 0x5410);
                    pd[kk][1][2 * g + e] = __byte_perm(t0, t1, 0x7632);
                    pd[kk][2][2 * g + e] = __byte_perm(t2, t3, 0x5410);
                }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const float mn = any ? fmaxf(run_m[e], mb) : run_m[e];
            alpha[e] = ex2(run_m[e] - mn);
            const float beta = any ? ex2(mb - mn) : 0.f;
            run_l[e] = run_l[e] * alpha[e] + beta * sum;
            gain[e] = beta * top * ((INT4 ? 1.f / 16.f : 1.f) / P_TOP);
            run_m[e] = mn;
        }
        if (!W16) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int d = 0; d < 3; ++d) pd[kk][d][1] = pd[kk][d][3] = 0u;
        }
        cp_wait<1>();
        __syncwarp();
        // values: dim 16 gr + t of tile t, from the bytes of the lane's sixteen keys; eight tiles at a time
        auto load_values = [&](int dh, uint32_t (&vb)[2][8][2]) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int r0 = 32 * kk + 16 * g + 2 * c;
                    uint32_t o[4];
                    if (INT4) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = r0 + (i & 1) + 8 * (i >> 1);
                            w[i] = *reinterpret_cast<const uint32_t*>(stage + St::V + v_off<true>(r, gr >> 1) + (gr & 1) * 8 + 4 * dh);
                        }
                        transpose4(w[0], w[1], w[2], w[3], o);
#pragma unroll
                        for (int i = 0; i < 4; ++i) vb[kk][2 * i][g] = (o[i] << 4) & 0xF0F0F0F0u, vb[kk][2 * i + 1][g] = o[i] & 0xF0F0F0F0u;
                    } else {
                        uint2 w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = *reinterpret_cast<const uint2*>(stage + St::V + v_off<false>(r0 + (i & 1) + 8 * (i >> 1), gr) + 8 * dh);
                        transpose4(w[0].x, w[1].x, w[2].x, w[3].x, o);
#pragma unroll
                        for (int i = 0; i < 4; ++i) vb[kk][i][g] = o[i];
                        transpose4(w[0].y, w[1].y, w[2].y, w[3].y, o);
#pragma unroll
                        for (int i = 0; i < 4; ++i) vb[kk][4 + i][g] = o[i];
                    }
                }
        };
        bool moved = false;   // a new maximum rescales what there is; mostly there is none
#pragma unroll
        for (int e = 0; e < HALVES; ++e) moved |= alpha[e] != 1.f;
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int t = 0; t < 16; ++t)
#pragma unroll
                for (int i = 0; i < (W16 ? 4 : 2); ++i) O[t][i] *= alpha[i >> 1];
        }
#pragma unroll
        for (int dh = 0; dh < 2; ++dh) {
            uint32_t vb[2][8][2];
            load_values(dh, vb);
            __syncwarp();
            if (dh == 1) {   // the values have been read: the next block's take their place
                if (next < end) load_codes<INT4>(st + St::V, nxt.v, nxt.rows, true, lane);
                cp_commit();
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                int acc[3][4];
#pragma unroll
                for (int d = 0; d < 3; ++d) mma<false, true>(acc[d], pd[0][d], vb[0][t][0], vb[0][t][1]);
#pragma unroll
                for (int d = 0; d < 3; ++d) mma<false, false>(acc[d], pd[1][d], vb[1][t][0], vb[1][t][1]);
#pragma unroll
                for (int i = 0; i < (W16 ? 4 : 2); ++i)
                    O[8 * dh + t][i] = fmaf(upper(acc[2][i]), gain[i >> 1], fmaf(lower(acc[1][i], acc[0][i]), gain[i >> 1], O[8 * dh + t][i]));
            }
        }
        cur = nxt;
    }
    // ---- join the warps
    cp_wait<0>();
    __syncwarp();
    {
        float* po = reinterpret_cast<float*>(stage);
#pragma unroll
        for (int t = 0; t < 16; ++t)
#pragma unroll
            for (int e = 0; e < HALVES; ++e)
                po[part_at(gr + 8 * e, 32 * c + t)] = O[t][2 * e], po[part_at(gr + 8 * e, 32 * c + 16 + t)] = O[t][2 * e + 1];
        if (c == 0) {
#pragma unroll
            for (int e = 0; e < HALVES; ++e) sh.warp_m[warp][gr + 8 * e] = run_m[e], sh.warp_l[warp][gr + 8 * e] = run_l[e];
        }
    }
    __syncthreads();
    float* mine = p.part + ((size_t)blockIdx.x * 2 + head) * PART_FLOATS;   // for a unit that is not complete here
    if (tid < cols) {   // a column's maximum, the parts' factors, its sum
        const int col = tid;
        const float pm = sh.part_m[col];
        float M = pm;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sh.warp_m[w][col]);
        float f = ex2(pm - M), l = f * sh.part_l[col];
        sh.warp_f[WARPS][col] = f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            f = ex2(sh.warp_m[w][col] - M);
            sh.warp_f[w][col] = f;
            l = fmaf(f, sh.warp_l[w][col], l);
        }
        sh.part_m[col] = M, sh.part_l[col] = l;
        if (!complete) mine[col] = M, mine[PART_L + col] = l;
    }
    __syncthreads();
    static_assert(PT == RD, "a thread has one dim of every column");
    float* out = p.out + (size_t)b * p.N * p.hq * RD + tid;
#pragma unroll 4
    for (int col = 0; col < cols; ++col) {
        const int d = tid;
        float o = sh.warp_f[WARPS][col] * sh.part[col][d];
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            o = fmaf(sh.warp_f[w][col], reinterpret_cast<const float*>(smem + w * St::BYTES)[part_at(col, d)], o);
        if (complete) {
            if (sh.row[col] >= 0) out[sh.row[col] * RD] = o / sh.part_l[col];
        } else {
            mine[PART_O + col * RD + d] = o;
        }
    }
    }
    }
    // ---- the range's next unit
    left -= take;
    at.at = 0;
    if (++at.unit == p.hk * p.groups) at.unit = 0, ++at.b;
    __syncthreads();
    }
}

// Joins the partial results of the units that the ranges' cuts divide, JCOLS columns a CTA; its JG groups of 128 threads
// take the parts in turn (a unit of a small call may have hundreds: 1 x 10 heads x 1 node over 26000 rows, 296 parts in all,
// with 1 / 4 groups 34 / 22 us; 320 units of two or three parts 73 / 82 us).  Everything but the partial results themselves was there before the
// kernel in front of this one began, so it is read ahead of the wait.
template <int JG>
__global__ void __launch_bounds__(JG * RD) rswa_ranges_join_kernel(const __grid_constant__ TreeParams p, int ctas) {
    constexpr int JT = JG * RD;
    __shared__ int scan[JT / 32 + 4];
    __shared__ float gm[JG][JCOLS], gl[JG][JCOLS], go[JG][JCOLS][RD];
    const int tid = threadIdx.x, per_b = p.hk * p.groups, b = blockIdx.x / per_b, unit = blockIdx.x % per_b;
    int all = 0, before = 0;
    for (int i = tid; i < p.B; i += JT) {
        const int own = unit_length(p, i);
        all += own;
        if (i < b) before += own;
    }
    const int R = __ldg(p.ref_len + b), n = __ldg(p.n_gen + b), L = p.n_nodes ? __ldg(p.n_nodes + b) : p.N;
    const int par = tid < p.N && p.parent ? __ldg(p.parent + (size_t)b * p.N + tid) : tid - 1;
    // the unit's blocks in the row, and the CTAs that had them
    const int own = unit_length(p, b);
    all = cta_scan<JT / 32>(all, scan) * per_b;
    before = cta_scan<JT / 32>(before, scan);
    const int per = (all + ctas - 1) / ctas;
    const int64_t from = (int64_t)before * per_b + (int64_t)unit * own;
    const int c0 = (int)((from + BEGIN) / per), c1 = (int)((from + own - 1) / per);
    const bool bad = __syncthreads_or(R < 0 || R > p.ref.cap || n < 0 || L < 0 || L > p.N || (tid < L && (par < -1 || par >= tid)));
    pdl_wait();
    if (bad || c0 == c1) return;
    const int h = unit / p.groups, col0 = unit % p.groups * COLS, first = blockIdx.y * JCOLS;
    const int group = tid / RD, d = tid % RD;
    float M[JCOLS], l[JCOLS], o[JCOLS];
#pragma unroll
    for (int j = 0; j < JCOLS; ++j) M[j] = NONE, l[j] = o[j] = 0.f;
    auto add = [&](int j, float m, float lp, float op) {
        const float mn = fmaxf(M[j], m), f = ex2(M[j] - mn), g = ex2(m - mn);
        M[j] = mn, l[j] = fmaf(g, lp, f * l[j]), o[j] = fmaf(g, op, f * o[j]);
    };
#pragma unroll 2
    for (int c = c0 + group; c <= c1; c += JG) {
        const float* part = p.part + ((size_t)c * 2 + (c == c0)) * PART_FLOATS;
        float m[JCOLS], lp[JCOLS], op[JCOLS];   // (columns behind the unit's last hold anything, and go nowhere)
#pragma unroll
        for (int j = 0; j < JCOLS; ++j)
            m[j] = __ldcg(part + first + j), lp[j] = __ldcg(part + PART_L + first + j), op[j] = __ldcg(part + PART_O + (first + j) * RD + d);
#pragma unroll
        for (int j = 0; j < JCOLS; ++j) add(j, m[j], lp[j], op[j]);
    }
    if (JG > 1) {
#pragma unroll
        for (int j = 0; j < JCOLS; ++j) {
            go[group][j][d] = o[j];
            if (d == 0) gm[group][j] = M[j], gl[group][j] = l[j];
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g = 1; g < JG; ++g)
#pragma unroll
            for (int j = 0; j < JCOLS; ++j) add(j, gm[g][j], gl[g][j], go[g][j][d]);
    }
#pragma unroll
    for (int j = 0; j < JCOLS; ++j) {
        const int col = col0 + first + j, node = col / p.G;
        if (first + j < COLS && col < p.N * p.G && node < L)
            p.out[(((size_t)b * p.N + node) * p.hq + h * p.G + col % p.G) * RD + d] = o[j] / l[j];
    }
}

template <bool INT4, bool W16>
cudaError_t launch_as(TreeParams& p, cudaStream_t st) {
    const void* fn = (const void*)rswa_ranges_kernel<INT4, W16>;
    const size_t smem = WARPS * Stage<INT4>::BYTES + sizeof(Shared);
    cudaError_t e = once_per_device(fn, [&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    int ctas = resident();
    void* args[] = {&p};
    e = launch_kernel(fn, dim3((unsigned)ctas), dim3(PT), smem, 1, args, st);
    if (e != cudaSuccess) return e;
    void* more[] = {&p, &ctas};
    const int cols = p.N * p.G < COLS ? p.N * p.G : COLS;
    const unsigned units = (unsigned)p.B * p.hk * p.groups;
    const bool few = units < (unsigned)ctas / 4;
    return launch_kernel(few ? (const void*)rswa_ranges_join_kernel<4> : (const void*)rswa_ranges_join_kernel<1>,
                         dim3(units, (cols + JCOLS - 1) / JCOLS), dim3(few ? 4 * RD : RD), 0, 1, more, st);
}

}  // namespace

size_t ranges_part_bytes() { return ((size_t)resident() * 2 * PART_FLOATS * sizeof(float) + 255) & ~(size_t)255; }
cudaError_t launch_ranges(TreeParams& p, bool int4, cudaStream_t st) {
    const bool wide = p.N * p.G > 8;
    return int4 ? (wide ? launch_as<true, true>(p, st) : launch_as<true, false>(p, st))
                : (wide ? launch_as<false, true>(p, st) : launch_as<false, false>(p, st));
}

}  // namespace focr
