// The tree attention of rswa_tree.cu for many units or long reference blocks, on the tcgen05 integer tensor cores.
//
// The mathematics is that of rswa_tree.cu: codes as they lie in memory, a query row as three signed 8-bit digits, a
// key's weight as three unsigned ones, exact s32 sums.  Here the sums live in tensor memory and no code passes through
// a register: per tile of 128 keys
//   S [128 keys x 3 CP]  = K [128 x 128] Q^T          four tcgen05.mma kind::i8, both operands K-major
//   O [128 dims x 3 CP] += V^T [128 x 128 keys] P      four more; V lies [key][dim] and P is written [key][column], so
//                                                      both operands are read along their other axis (transposed)
// with CP columns (query heads of nodes, padded to 16) in three digits.  Layout of every operand: core matrices of 8
// rows x 16 bytes, 128 bytes each, chunk j of row r at (r / 8) * (row group) + j * 128 + (r % 8) * 16.
//
// The softmax has no maximum per tile: a column's reference m is a bound that its scores (base 2) may not exceed; a
// tile with a larger score (or value scale) first moves the bound to MARGIN above it and brings O and the sum along.
// The weight 2^(s - m) vs / vref is then at most 1 and is written with 24 bits, so a weight is off by 2^-25 of the
// bound, at most 2^-23.8 of the largest weight.  O stays in s32 while the bounds stand (at most 65536 keys a unit: |sum| <=
// 33024 * 255 * 128 < 2^31) and is added to fp32 registers when they move and at the unit's end.
//
// Roles of a CTA (one per SM): warps 0-7 softmax (thread = key row of S, dim row of O; warps 0-3 have the first half of
// the columns, 4-7 the second), warps 8-11 load (cp.async; int4 is unpacked to bytes 16 q on the way), warp 12 issues
// the MMAs.  All tiles of all units form one row, cut into equal ranges, one per CTA (the lengths are read on the
// device, so ragged batches stay balanced); units that a cut divides leave partial results in the workspace, and a
// second kernel joins them.  Every wait is bounded; one that runs out turns the CTA's results into NaN.
#include <math.h>

#include "abi_util.h"
#include "common.cuh"
#include "launch_state.h"
#include "rswa_tree.cuh"
#include "umma.cuh"

namespace focr {
namespace {

constexpr int RD = TREE_DIM, RW = TREE_RING, TILE = 128;
constexpr int SOFT = 8, LOADERS = 4, WARPS = SOFT + LOADERS + 1, PT = 32 * WARPS;
constexpr int ST = 32 * SOFT, LT = 32 * LOADERS;
constexpr int JT = 128;                       // threads of the joining kernel
constexpr int CMAX = TREE_MAX;                // columns of a unit
constexpr float MARGIN = 1.f;                 // bounds are set this far (log2) above the largest score seen
constexpr float V_MARGIN = 1.125f;            // and the value scales' bound this factor above the largest one
constexpr uint64_t LIMIT_NS = 2000000000ull;  // bound of every wait
// A partial result: the columns' bounds, sums and unnormalised outputs.
constexpr int PART_L = CMAX, PART_O = 2 * CMAX, PART_FLOATS = 2 * CMAX + CMAX * RD;

// kind::i8: D s32, A s8, B s8 or u8 (b_signed); ta, tb: operand read along its other axis.
__host__ __device__ constexpr uint32_t idesc_i8(int N, bool b_signed, bool ta, bool tb) {
    return (2u << 4) | (1u << 7) | ((b_signed ? 1u : 0u) << 10) | ((ta ? 1u : 0u) << 15) | ((tb ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    const uint32_t acc = accumulate ? 1u : 0u, zero = 0u;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, {%5, %5, %5, %5}, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(zero)
        : "memory");
}
// eight columns of the thread's tensor-memory lane; complete after wait_ld()
__device__ __forceinline__ void ld8(uint32_t taddr, int (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st8(uint32_t taddr, int v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%1,%1,%1,%1,%1,%1,%1};" ::"r"(taddr), "r"(v) : "memory");
}
// a barrier of the softmax threads that also tells whether any of them said so
__device__ __forceinline__ bool any_of_softmax(bool mine) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred p, 1, 256, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)mine)
        : "memory");
    __syncwarp();
    return r != 0;
}
__device__ __forceinline__ void softmax_sync() {
    __syncwarp();
    named_bar_sync(1, ST);
}

template <bool INT4, int CP>
struct Sizes {
    static constexpr int N = 3 * CP;                                  // columns in digits
    static constexpr int STAGES = INT4 ? 2 : CP <= 32 ? 4 : 3;        // tiles of bytes
    static constexpr int PACKED = INT4 ? 4 : 1;                       // tiles of nibbles on their way
    static constexpr int SBUF = 3 * N <= 512 ? 2 : 1;                 // score buffers in tensor memory
    static constexpr int KV = TILE * RD;                              // bytes of K (or V) of a tile
    static constexpr int STAGE = 2 * KV;
    static constexpr int PACK = 2 * KV / 2 + 8 * TILE;                // nibbles of K and V, and scales
    static constexpr int Q_OFF = STAGES * STAGE + (INT4 ? PACKED * PACK : 0), P_OFF = Q_OFF + N * RD, S_OFF = P_OFF + N * TILE;
};

template <int CP>
struct Shared {
    float part[CP][RD];                  // the drafted keys' part
    float part_m[CP], part_l[CP];
    float scales[4][2][TILE];            // of the stages' tiles: ks, vs
    float2 col[CP];                      // a column's step (score in log2 = dot * key scale * step) and bound
    float alpha[CP];                     // what a moved bound does to the column's sums
    float red[SOFT][CP / 2 + 1];
    int ages[CP];                        // ring slots younger than this are seen
    unsigned long long line[TREE_MAX];
    int par[TREE_MAX];
    uint64_t full[4], empty[4], s_full[2], s_free[2], p_full, p_free, q_full;
    int scan[WARPS + 4];
    float vref;                          // bound of the value scales
    int fresh;                           // the next P V starts O anew
    int gave_up;
    uint32_t tmem;
};

// Tiles of a sequence's unit (one at least: the drafted keys need a CTA too).
__device__ __forceinline__ int sequence_tiles(const TreeParams& p, int b) {
    const int R = __ldg(p.ref_len + b), n = __ldg(p.n_gen + b);
    if (R < 0 || R > p.ref.cap || n < 0) return 1;
    return max(1, (R + TILE - 1) / TILE + (n > 0));
}
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
struct Place {   // a tile in the row of all units' tiles
    int b, h, tile;
};
__device__ int all_tiles(const TreeParams& p, int* scan) {
    int mine = 0;
    for (int b = threadIdx.x; b < p.B; b += PT) mine += sequence_tiles(p, b);
    return cta_scan<WARPS>(mine, scan) * p.hk;
}
__device__ Place find_tile(const TreeParams& p, int at, int* scan) {
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += PT) {
        const int b = b0 + threadIdx.x, own = b < p.B ? sequence_tiles(p, b) : 0;
        int sum = own;
        const int total = cta_scan<WARPS>(sum, scan);
        if ((int64_t)(before + total) * p.hk > at) {
            const int64_t first = (int64_t)(before + sum - own) * p.hk;
            if (at >= first && at < first + (int64_t)own * p.hk) scan[WARPS] = b, scan[WARPS + 1] = (int)(at - first), scan[WARPS + 2] = own;
            __syncthreads();
            const Place x{scan[WARPS], scan[WARPS + 1] / scan[WARPS + 2], scan[WARPS + 1] % scan[WARPS + 2]};
            __syncthreads();
            return x;
        }
        before += total;
    }
    return Place{p.B, 0, 0};
}

// The part of a unit that a CTA has.  Every warp reads it for itself.
struct Segment {
    int b, h, R, n, L;
    int first, count;      // its tiles of keys
    int taken;             // tiles of the range that it uses up
    bool bad, head, complete;
};
__device__ Segment segment_at(const TreeParams& p, const Place& at, int left) {
    Segment s;
    const int lane = threadIdx.x & 31;
    s.b = at.b, s.h = at.h;
    s.R = __ldg(p.ref_len + s.b), s.n = __ldg(p.n_gen + s.b), s.L = p.n_nodes ? __ldg(p.n_nodes + s.b) : p.N;
    s.bad = s.R < 0 || s.R > p.ref.cap || s.n < 0 || s.L < 0 || s.L > p.N;
    if (p.parent) {
        bool wrong = false;
        for (int i = lane; i < min(s.L, p.N); i += 32) {
            const int par = __ldg(p.parent + (size_t)s.b * p.N + i);
            wrong |= par < -1 || par >= i;
        }
        s.bad |= __any_sync(0xffffffffu, wrong);
    }
    const int all = sequence_tiles(p, s.b);
    s.first = at.tile, s.taken = min(left, all - at.tile);
    const int keys = s.bad || s.L == 0 ? 0 : (s.R + TILE - 1) / TILE + (s.n > 0);
    s.count = max(0, min(s.first + s.taken, keys) - s.first);
    s.head = s.first == 0, s.complete = s.head && s.taken == all;
    return s;
}
__device__ __forceinline__ void advance(const TreeParams& p, Place& at, int& left, const Segment& s) {
    left -= s.taken;
    at.tile = 0;
    if (++at.h == p.hk) at.h = 0, ++at.b;
}
// Row of the cache where tile t of a segment's unit starts, its rows that hold a key, and whether it is the ring.
struct TileAt {
    size_t row;
    int rows;
    bool ring;
};
__device__ __forceinline__ TileAt tile_at(const TreeParams& p, const Segment& s, int t) {
    const int nref = (s.R + TILE - 1) / TILE;
    const size_t unit = (size_t)s.b * p.hk + s.h;
    if (t >= nref) return {unit * RW, min(s.n, RW), true};
    return {unit * p.ref.cap + (size_t)t * TILE, min(TILE, s.R - t * TILE), false};
}

template <bool INT4, int CP>
__global__ void __launch_bounds__(PT, 1) rswa_wide_kernel(const __grid_constant__ TreeParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using Z = Sizes<INT4, CP>;
    constexpr int N = Z::N, STAGES = Z::STAGES, HALF = CP / 2;   // HALF: columns of a softmax thread
    Shared<CP>& sh = *reinterpret_cast<Shared<CP>*>(smem + Z::S_OFF);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cols = p.N * p.G;

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(&sh.full[i], LT), mbar_init(&sh.empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&sh.s_full[i], 1), mbar_init(&sh.s_free[i], SOFT);
        mbar_init(&sh.p_full, SOFT);
        mbar_init(&sh.p_free, 1);
        mbar_init(&sh.q_full, SOFT);
        fence_barrier_init();
        sh.gave_up = 0;
        sh.fresh = 1;
    }
    if (warp == SOFT + LOADERS) umma::tmem_alloc(smem_u32(&sh.tmem), 512);
    pdl_wait();
    const int all = all_tiles(p, sh.scan), per = (all + gridDim.x - 1) / gridDim.x;   // (its barriers cover the set-up above)
    const int from = (int)min((int64_t)blockIdx.x * per, (int64_t)all), mine = min(per, all - from);
    Place at{p.B, 0, 0};
    if (mine > 0) at = find_tile(p, from, sh.scan);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = sh.tmem, tmem_o = tmem + Z::SBUF * N;
    int left = mine;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_wait_bounded(bar, parity, LIMIT_NS)) return true;
        sh.gave_up = 1;
        return false;
    };

    if (warp < SOFT) {
        // ------------------------------------------------------------ softmax
        const int wg = warp >> 2, row = (warp & 3) * 32 + lane, c0 = wg * HALF;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int dim = INT4 ? 32 * (row / 32) + 2 * (row % 16) + ((row / 16) & 1) : row;   // of the thread's lane of O
        uint8_t* sq = smem + Z::Q_OFF;
        uint8_t* sp = smem + Z::P_OFF;
        auto preset = [&](int buf) {   // S accumulates onto the pattern that reads as MAGIC + sum
#pragma unroll
            for (int d = 0; d < 3; ++d)
#pragma unroll
                for (int c = 0; c < HALF; c += 8) st8(lanes + buf * N + d * CP + c0 + c, MAGIC_BITS);
            umma::wait_st();
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.s_free[buf]);
        };
        for (int i = 0; i < Z::SBUF; ++i) preset(i);
        int it = 0;   // tiles so far
        bool ok = true;
        while (left > 0 && ok) {
            const Segment s = segment_at(p, at, left);
            const bool dead = s.bad || s.L == 0;
            if (s.bad && s.head) {
                const int live = s.L < 0 || s.L > p.N ? p.N : s.L;
                for (int i = tid; i < live * p.G * RD; i += ST)
                    p.out[(((size_t)s.b * p.N + i / RD / p.G) * p.hq + s.h * p.G + i / RD % p.G) * RD + i % RD] = __int_as_float(0x7fc00000);
            }
            if (!dead) {
                // ---- lines of the tree, query digits, drafted keys
                if (tid < s.L) sh.par[tid] = p.parent ? __ldg(p.parent + (size_t)s.b * p.N + tid) : tid - 1;
                softmax_sync();
                if (tid < s.L) {
                    unsigned long long line = 0;
                    for (int j = tid; j >= 0; j = sh.par[j]) line |= 1ull << j;
                    sh.line[tid] = line;
                }
                if (tid == 0) sh.vref = TINY;
                softmax_sync();
                for (int cb = warp; cb < CP; cb += 2 * SOFT) {   // two columns at a time
                    float4 q[2], k4[2][4], v4[2][4];
                    unsigned long long line[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int c = cb + i * SOFT, node = c / p.G;
                        const bool live = c < cols && node < s.L;
                        q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (live) q[i] = __ldg(reinterpret_cast<const float4*>(p.q + (((size_t)s.b * p.N + node) * p.hq + s.h * p.G + c % p.G) * RD) + lane);
                        line[i] = live && s.head ? sh.line[node] : 0ull;
                        unsigned long long rest = line[i];
                        draft_load(p, s.b, s.h, lane, rest, k4[i], v4[i]);
                        if (lane == 0) sh.ages[c] = live ? min(s.n, RW - __popcll(sh.line[node])) : 0;
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int c = cb + i * SOFT;
                        const float4 x = q[i];
                        float a = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
                        for (int o = 16; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                        a = fmaxf(a, TINY);
                        const float inv = Q_TOP / a;
                        int f[4] = {__float2int_rn(x.x * inv), __float2int_rn(x.y * inv), __float2int_rn(x.z * inv), __float2int_rn(x.w * inv)};
#pragma unroll
                        for (int d = 0; d < 3; ++d) {   // signed digits, the lowest first
                            uint32_t v[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int digit = (int)(int8_t)f[j];
                                v[j] = (uint32_t)digit & 255u;
                                f[j] = (f[j] - digit) >> 8;
                            }
                            const int n = d * CP + c;
                            uint8_t* at8 = sq + (n >> 3) * 1024 + (n & 7) * 16;
                            if (INT4) {   // even dims of 32 in one chunk, odd ones in the next
                                uint8_t* w = at8 + (lane >> 3) * 256 + 2 * (lane & 7);
                                *reinterpret_cast<uint16_t*>(w) = (uint16_t)(v[0] | v[2] << 8);
                                *reinterpret_cast<uint16_t*>(w + 128) = (uint16_t)(v[1] | v[3] << 8);
                            } else {
                                *reinterpret_cast<uint32_t*>(at8 + (lane >> 2) * 128 + 4 * (lane & 3)) = v[0] | v[1] << 8 | v[2] << 16 | v[3] << 24;
                            }
                        }
                        if (lane == 0) sh.col[c] = make_float2(a / Q_TOP * (SCORE_SCALE * LOG2E * (INT4 ? 1.f / 16.f : 1.f)), NONE);
                        const DraftPart dp = draft_attend(p, s.b, s.h, lane, x, line[i], k4[i], v4[i]);
                        reinterpret_cast<float4*>(sh.part[c])[lane] = dp.o;
                        if (lane == 0) sh.part_m[c] = dp.m, sh.part_l[c] = dp.l;
                    }
                }
                umma::fence_smem_to_async();
                softmax_sync();
                if (lane == 0 && s.count > 0) mbar_arrive(&sh.q_full);

                float acc[HALF], sum[HALF];
#pragma unroll
                for (int c = 0; c < HALF; ++c) acc[c] = sum[c] = 0.f;
                bool filled = false;   // O holds something
                // adds O to the fp32 accumulators (every P V so far has completed)
                auto drain = [&](float vref) {
                    const float gain = vref * ((INT4 ? 1.f / 16.f : 1.f) / P_TOP);
                    umma::fence_after_sync();
#pragma unroll
                    for (int c = 0; c < HALF; c += 8) {
                        int o2[8], o1[8], o0[8];
                        const uint32_t t = tmem_o + ((uint32_t)((warp & 3) * 32) << 16) + c0 + c;
                        ld8(t, o0);
                        ld8(t + CP, o1);
                        ld8(t + 2 * CP, o2);
                        wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            acc[c + j] = fmaf(fmaf((float)o2[j], 65536.f, fmaf((float)o1[j], 256.f, (float)o0[j])), gain, acc[c + j]);
                    }
                };
                for (int t = s.first; t < s.first + s.count; ++t, ++it) {   // left by all threads at once
                    const int stage = it % STAGES, buf = it % Z::SBUF;
                    const TileAt ta = tile_at(p, s, t);
                    ok = ok && wait(&sh.full[stage], it / STAGES & 1) && wait(&sh.s_full[buf], it / Z::SBUF & 1);
                    if (any_of_softmax(!ok)) {
                        ok = false;
                        break;
                    }
                    umma::fence_after_sync();
                    const bool in = row < ta.rows;
                    const float ks = in ? sh.scales[stage][0][row] : 0.f, vs = in ? sh.scales[stage][1][row] : 0.f;
                    float x[HALF];   // scores without the column's step
#pragma unroll
                    for (int c = 0; c < HALF; c += 8) {
                        int d2[8], d1[8], d0[8];
                        const uint32_t tc = lanes + buf * N + c0 + c;
                        ld8(tc, d0);
                        ld8(tc + CP, d1);
                        ld8(tc + 2 * CP, d2);
                        wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[c + j] = (upper(d2[j]) + lower(d1[j], d0[j])) * ks;
                    }
                    preset(buf);
                    if (ta.ring) {
                        const int age = (s.n - 1 - row) & (RW - 1);
#pragma unroll
                        for (int c = 0; c < HALF; ++c)
                            if (!in || age >= sh.ages[c0 + c]) x[c] = -INFINITY;
                    } else if (!in) {
#pragma unroll
                        for (int c = 0; c < HALF; ++c) x[c] = -INFINITY;
                    }
                    float vref = sh.vref;
                    bool over = vs > vref;
#pragma unroll
                    for (int c = 0; c < HALF; ++c) {
                        const float2 k = sh.col[c0 + c];
                        over |= fmaf(x[c], k.x, -k.y) > 0.f;
                    }
                    if (any_of_softmax(over)) {
                        // ---- bounds move: columns' and scales' largest values of the tile
#pragma unroll
                        for (int c = 0; c < HALF; ++c) {
                            float m = x[c];
#pragma unroll
                            for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                            if (lane == 0) sh.red[warp][c] = m;
                        }
                        float vm = vs;
#pragma unroll
                        for (int o = 16; o >= 1; o >>= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
                        if (lane == 0) sh.red[warp][HALF] = vm;
                        if (filled) {
                            ok = wait(&sh.p_free, (it - 1) & 1) && ok;
                            __syncwarp();
                            drain(vref);
                        }
                        softmax_sync();
                        if (tid < CP) {
                            const int w = tid / HALF * 4, c = tid % HALF;
                            const float m = fmaxf(fmaxf(sh.red[w][c], sh.red[w + 1][c]), fmaxf(sh.red[w + 2][c], sh.red[w + 3][c]));
                            const float2 k = sh.col[tid];
                            const float now = m == -INFINITY ? NONE : m * k.x, to = now > k.y ? now + MARGIN : k.y;
                            sh.alpha[tid] = ex2(k.y - to);
                            sh.col[tid] = make_float2(k.x, to);
                        }
                        if (tid == 0) {
                            const float v = fmaxf(fmaxf(sh.red[0][HALF], sh.red[1][HALF]), fmaxf(sh.red[2][HALF], sh.red[3][HALF]));
                            if (v > sh.vref) sh.vref = V_MARGIN * v;
                            sh.fresh = 1;
                        }
                        softmax_sync();
                        vref = sh.vref;
#pragma unroll
                        for (int c = 0; c < HALF; ++c) {
                            const float al = sh.alpha[c0 + c];
                            acc[c] *= al, sum[c] *= al;
                        }
                        filled = false;
                    }
                    // ---- weights: 24 bits, as three digits, [key][column] for the second product
                    const float vn = vs * (P_TOP / vref);
                    uint32_t w[3][HALF / 4];
#pragma unroll
                    for (int c = 0; c < HALF; c += 4) {
                        uint32_t u[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 k = sh.col[c0 + c + j];
                            const float e = ex2(fmaf(x[c + j], k.x, -k.y));
                            sum[c + j] += e;
                            u[j] = __float2uint_rn(e * vn);
                        }
                        const uint32_t t0 = __byte_perm(u[0], u[1], 0x5140), t1 = __byte_perm(u[2], u[3], 0x5140);
                        const uint32_t t2 = __byte_perm(u[0], u[1], 0x0062), t3 = __byte_perm(u[2], u[3], 0x0062);
                        w[0][c / 4] = __byte_perm(t0, t1, 0x5410);
                        w[1][c / 4] = __byte_perm(t0, t1, 0x7632);
                        w[2][c / 4] = __byte_perm(t2, t3, 0x5410);
                    }
                    if (it > 0) ok = wait(&sh.p_free, (it - 1) & 1) && ok;   // the weights of the tile before have been used
                    {
                        uint8_t* at8 = sp + (row >> 3) * (N / 16 * 128) + (row & 7) * 16;
#pragma unroll
                        for (int d = 0; d < 3; ++d) {
                            const int n = d * CP + c0;   // a multiple of 8; 16 columns a chunk
#pragma unroll
                            for (int c = 0; c < HALF; c += 8)
                                *reinterpret_cast<uint2*>(at8 + ((n + c) >> 4) * 128 + ((n + c) & 15)) = make_uint2(w[d][c / 4], w[d][c / 4 + 1]);
                        }
                    }
                    umma::fence_smem_to_async();
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.p_full);
                    filled = true;
                }
                if (filled && ok) {
                    ok = wait(&sh.p_free, (it - 1) & 1);
                    __syncwarp();
                    drain(sh.vref);
                }
                if (any_of_softmax(!ok)) {
                    ok = false;
                    break;
                }
                // ---- the unit's sums, and the drafted keys
#pragma unroll
                for (int c = 0; c < HALF; ++c) {
                    float l = sum[c];
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                    if (lane == 0) sh.red[warp][c] = l;
                }
                softmax_sync();
                float* part = p.part + ((size_t)blockIdx.x * 2 + s.head) * PART_FLOATS;
#pragma unroll
                for (int c = 0; c < HALF; ++c) {
                    const int cc = c0 + c, node = cc / p.G;
                    if (cc >= cols || node >= s.L) continue;
                    const float l = (sh.red[4 * wg][c] + sh.red[4 * wg + 1][c]) + (sh.red[4 * wg + 2][c] + sh.red[4 * wg + 3][c]);
                    const float m = sh.col[cc].y, pm = sh.part_m[cc], M = fmaxf(m, pm), f = ex2(m - M), g = ex2(pm - M);
                    const float lt = fmaf(f, l, g * sh.part_l[cc]), o = fmaf(f, acc[c], g * sh.part[cc][dim]);
                    if (s.complete) {
                        p.out[(((size_t)s.b * p.N + node) * p.hq + s.h * p.G + cc % p.G) * RD + dim] = o / lt;
                    } else {
                        part[PART_O + cc * RD + dim] = o;
                        if (row == 0) part[cc] = M, part[PART_L + cc] = lt;
                    }
                }
                if (tid == 0) sh.fresh = 1;
                softmax_sync();
            }
            advance(p, at, left, s);
        }
    } else if (warp < SOFT + LOADERS) {
        // ------------------------------------------------------------ loads
        const int t = tid - ST;   // thread of the loaders: row t of a tile's scales
        int it = 0;
        bool ok = true;
        if (!INT4) {
            int signalled = 0;   // tiles whose arrival has been signalled
            auto signal = [&](int upto) {
                umma::fence_smem_to_async();
                for (; signalled < upto; ++signalled) mbar_arrive(&sh.full[signalled % STAGES]);
            };
            while (left > 0 && ok) {
                const Segment s = segment_at(p, at, left);
                for (int tile = s.first; tile < s.first + s.count && ok; ++tile, ++it) {
                    const int stage = it % STAGES;
                    const TileAt ta = tile_at(p, s, tile);
                    if (it >= STAGES) {
                        // nothing that has arrived may wait for a place that only its use sets free
                        if (!mbar_try_wait(&sh.empty[stage], (it / STAGES - 1) & 1)) {
                            cp_wait<0>();
                            signal(it);
                            ok = wait(&sh.empty[stage], (it / STAGES - 1) & 1);
                        }
                    }
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    const KvView& v = ta.ring ? p.ring : p.ref;
                    const uint32_t to = smem_u32(smem) + stage * Z::STAGE;
                    // eight lanes copy one chunk of eight rows: a core matrix
                    const int r0 = t >> 5 << 3 | (t & 7), j0 = (t >> 3) & 3;
#pragma unroll
                    for (int i = 0; i < TILE / 32; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int r = r0 + 32 * i, ch = j0 + 4 * j;
                            const size_t src = (ta.row + min(r, ta.rows - 1)) * RD + ch * 16;
                            const uint32_t dst = to + (r >> 3) * 1024 + ch * 128 + (r & 7) * 16;
                            cp16(dst, v.k + src);
                            cp16(dst + Z::KV, v.v + src);
                        }
                    const size_t sr = ta.row + min(t, ta.rows - 1);
                    cp4(smem_u32(&sh.scales[stage][0][t]), v.ks + sr);
                    cp4(smem_u32(&sh.scales[stage][1][t]), v.vs + sr);
                    cp_commit();
                    if (it - signalled >= STAGES - 1) {
                        cp_wait<STAGES - 2>();
                        signal(it - (STAGES - 2) + 1);
                    }
                }
                advance(p, at, left, s);
            }
            cp_wait<0>();
            signal(it);
        } else {
            // nibbles come ahead into places of their own; a thread unpacks what it copied itself
            Place ahead = at;
            int ahead_left = left, issued = 0, ahead_tile = 0;
            Segment as{};
            bool have = false;
            auto issue = [&] {   // the next tile's copies, if there is one
                while (!have && ahead_left > 0) {
                    as = segment_at(p, ahead, ahead_left);
                    advance(p, ahead, ahead_left, as);
                    ahead_tile = as.first;
                    have = as.count > 0;
                }
                if (have) {
                    const TileAt ta = tile_at(p, as, ahead_tile);
                    const KvView& v = ta.ring ? p.ring : p.ref;
                    uint8_t* to = smem + STAGES * Z::STAGE + issued % Z::PACKED * Z::PACK;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {   // chunk (t % 4) of rows t / 4 + 32 i
                        const int r = t / 4 + 32 * i, j = t & 3;
                        const size_t src = (ta.row + min(r, ta.rows - 1)) * (RD / 2) + j * 16;
                        cp16(smem_u32(to + r * 64 + j * 16), v.k + src);
                        cp16(smem_u32(to + Z::KV / 2 + r * 64 + j * 16), v.v + src);
                    }
                    const size_t sr = ta.row + min(t, ta.rows - 1);
                    cp4(smem_u32(to + Z::KV + 4 * t), v.ks + sr);
                    cp4(smem_u32(to + Z::KV + 4 * TILE + 4 * t), v.vs + sr);
                    ++issued;
                    if (++ahead_tile == as.first + as.count) have = false;
                }
                cp_commit();
            };
            for (int i = 0; i < Z::PACKED - 1; ++i) issue();
            while (left > 0 && ok) {
                const Segment s = segment_at(p, at, left);
                for (int tile = s.first; tile < s.first + s.count && ok; ++tile, ++it) {
                    const int stage = it % STAGES;
                    issue();
                    cp_wait<3>();   // PACKED - 1 younger tiles may be on their way
                    if (it >= STAGES) ok = wait(&sh.empty[stage], (it / STAGES - 1) & 1);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    const uint8_t* fr = smem + STAGES * Z::STAGE + it % Z::PACKED * Z::PACK;
                    uint8_t* to = smem + stage * Z::STAGE;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = t / 4 + 32 * (i & 3), j = t & 3, kv = i >> 2;
                        const uint4 n = lds128(fr + kv * (Z::KV / 2) + r * 64 + j * 16);
                        uint8_t* dst = to + kv * Z::KV + (r >> 3) * 1024 + 2 * j * 128 + (r & 7) * 16;
                        *reinterpret_cast<uint4*>(dst) = make_uint4((n.x << 4) & 0xF0F0F0F0u, (n.y << 4) & 0xF0F0F0F0u, (n.z << 4) & 0xF0F0F0F0u, (n.w << 4) & 0xF0F0F0F0u);
                        *reinterpret_cast<uint4*>(dst + 128) = make_uint4(n.x & 0xF0F0F0F0u, n.y & 0xF0F0F0F0u, n.z & 0xF0F0F0F0u, n.w & 0xF0F0F0F0u);
                    }
                    sh.scales[stage][0][t] = *reinterpret_cast<const float*>(fr + Z::KV + 4 * t);
                    sh.scales[stage][1][t] = *reinterpret_cast<const float*>(fr + Z::KV + 4 * TILE + 4 * t);
                    umma::fence_smem_to_async();
                    mbar_arrive(&sh.full[stage]);
                }
                advance(p, at, left, s);
            }
            cp_wait<0>();
        }
    } else {
        // ------------------------------------------------------------ products
        constexpr uint32_t IS = idesc_i8(N, true, false, false), IO = idesc_i8(N, false, true, true);
        const uint32_t sq = smem_u32(smem) + Z::Q_OFF, sp = smem_u32(smem) + Z::P_OFF;
        int it = 0, seg = 0;
        bool ok = true;
        auto values = [&](int i) {   // O += V^T P of tile i
            const int stage = i % STAGES;
            ok = wait(&sh.p_full, i & 1) && ok;
            umma::fence_after_sync();
            if (lane == 0 && ok) {
                const bool fresh = *(volatile int*)&sh.fresh != 0;
                const uint32_t v = smem_u32(smem) + stage * Z::STAGE + Z::KV;
#pragma unroll
                for (int k = 0; k < 4; ++k)   // 32 keys each: four groups of eight rows
                    mma_i8(tmem_o, umma::sdesc_kmajor(v + 4096 * k, 1024, 128), umma::sdesc_kmajor(sp + 4 * (N / 16 * 128) * k, N / 16 * 128, 128), IO,
                           !(fresh && k == 0));
                sh.fresh = 0;
                umma::commit(smem_u32(&sh.p_free));
                umma::commit(smem_u32(&sh.empty[stage]));
            }
            __syncwarp();
        };
        while (left > 0 && ok) {
            const Segment s = segment_at(p, at, left);
            if (s.count > 0) {
                ok = wait(&sh.q_full, seg & 1);
                ++seg;
                for (int t = 0; t < s.count && ok; ++t, ++it) {
                    const int stage = it % STAGES, buf = it % Z::SBUF;
                    // with one score buffer the tile before has to be through first
                    if (Z::SBUF == 1 && t > 0) values(it - 1);
                    ok = ok && wait(&sh.full[stage], it / STAGES & 1) && wait(&sh.s_free[buf], it / Z::SBUF & 1);
                    umma::fence_after_sync();
                    if (lane == 0 && ok) {
                        const uint32_t k0 = smem_u32(smem) + stage * Z::STAGE;
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 dims each: two chunks
                            mma_i8(tmem + buf * N, umma::sdesc_kmajor(k0 + 256 * k, 128, 1024), umma::sdesc_kmajor(sq + 256 * k, 128, 1024), IS, true);
                        umma::commit(smem_u32(&sh.s_full[buf]));
                    }
                    __syncwarp();
                    if (Z::SBUF == 2 && t > 0) values(it - 1);
                }
                if (ok) values(it - 1);
            }
            advance(p, at, left, s);
        }
    }
    // ---- everybody is through
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    if (sh.gave_up) {   // no numbers from a CTA whose wait ran out
        left = mine;
        at = mine > 0 ? find_tile(p, from, sh.scan) : at;
        while (left > 0) {
            const Segment s = segment_at(p, at, left);
            float* part = p.part + ((size_t)blockIdx.x * 2 + s.head) * PART_FLOATS;
            for (int i = tid; i < cols * RD; i += PT) {
                const int c = i / RD, node = c / p.G;
                const float nan = __int_as_float(0x7fc00000);
                if (!s.complete) {
                    part[PART_O + i] = nan;
                    if (i % RD == 0) part[c] = 0.f, part[PART_L + c] = nan;
                } else if (s.bad || node < s.L) {
                    p.out[(((size_t)s.b * p.N + node) * p.hq + s.h * p.G + c % p.G) * RD + i % RD] = nan;
                }
            }
            advance(p, at, left, s);
        }
    }
    if (warp == SOFT + LOADERS) umma::tmem_free(tmem, 512);
}

// Joins the partial results of the units that the ranges' cuts divide.
__global__ void __launch_bounds__(JT) rswa_wide_join_kernel(const __grid_constant__ TreeParams p, int ctas) {
    __shared__ int scan[JT / 32 + 4];
    const int tid = threadIdx.x, b = blockIdx.x / p.hk, h = blockIdx.x % p.hk;
    pdl_wait();
    // the unit's tiles in the row of all tiles, and the CTAs that had them
    int all = 0, before = 0;
    for (int i = tid; i < p.B; i += JT) {
        const int own = sequence_tiles(p, i);
        all += own;
        if (i < b) before += own;
    }
    all = cta_scan<JT / 32>(all, scan) * p.hk;
    before = cta_scan<JT / 32>(before, scan);
    const int own = sequence_tiles(p, b), per = (all + ctas - 1) / ctas;
    const int64_t from = (int64_t)before * p.hk + (int64_t)h * own;
    const int c0 = (int)(from / per), c1 = (int)((from + own - 1) / per);
    if (c0 == c1) return;
    const Segment s = segment_at(p, Place{b, h, 0}, own);
    if (s.bad) return;
    for (int c = blockIdx.y; c < p.N * p.G; c += gridDim.y) {
        const int node = c / p.G;
        if (node >= s.L) return;
        float M = NONE, l = 0.f, o = 0.f;
        for (int i = c0; i <= c1; ++i) M = fmaxf(M, __ldcg(p.part + ((size_t)i * 2 + (i == c0)) * PART_FLOATS + c));
        for (int i = c0; i <= c1; ++i) {
            const float* part = p.part + ((size_t)i * 2 + (i == c0)) * PART_FLOATS;
            const float f = ex2(__ldcg(part + c) - M);
            l = fmaf(f, __ldcg(part + PART_L + c), l);
            o = fmaf(f, __ldcg(part + PART_O + c * RD + tid), o);
        }
        p.out[(((size_t)b * p.N + node) * p.hq + h * p.G + c % p.G) * RD + tid] = o / l;
    }
}

template <bool INT4, int CP>
cudaError_t launch_wide_as(TreeParams& p, cudaStream_t st) {
    const void* fn = (const void*)rswa_wide_kernel<INT4, CP>;
    const size_t smem = Sizes<INT4, CP>::S_OFF + sizeof(Shared<CP>);
    static_assert(Sizes<INT4, CP>::S_OFF + sizeof(Shared<CP>) <= 232448, "shared memory of an SM");
    cudaError_t e = once_per_device(fn, [&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    int ctas = wide_ctas();
    void* args[] = {&p};
    e = launch_kernel(fn, dim3((unsigned)ctas), dim3(PT), smem, 1, args, st);
    if (e != cudaSuccess) return e;
    void* more[] = {&p, &ctas};
    const int cols = p.N * p.G;
    return launch_kernel((const void*)rswa_wide_join_kernel, dim3((unsigned)p.B * p.hk, cols < 8 ? cols : 8), dim3(JT), 0, 1, more, st);
}
template <bool INT4>
cudaError_t launch_wide_for(TreeParams& p, cudaStream_t st) {
    const int cols = p.N * p.G;
    return cols <= 16   ? launch_wide_as<INT4, 16>(p, st)
           : cols <= 32 ? launch_wide_as<INT4, 32>(p, st)
           : cols <= 48 ? launch_wide_as<INT4, 48>(p, st)
                        : launch_wide_as<INT4, 64>(p, st);
}

}  // namespace

int wide_ctas() { return device_sms() > 0 ? device_sms() : 148; }
size_t wide_part_bytes() { return ((size_t)wide_ctas() * 2 * PART_FLOATS * sizeof(float) + 255) & ~(size_t)255; }
cudaError_t launch_wide(TreeParams& p, bool int4, cudaStream_t st) {
    return int4 ? launch_wide_for<true>(p, st) : launch_wide_for<false>(p, st);
}

}  // namespace focr
