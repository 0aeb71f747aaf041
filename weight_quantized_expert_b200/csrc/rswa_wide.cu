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
// tile with a larger score (or value scale) first moves the bound above it and brings O and the sum along.  The weight
// 2^(s - m) vs / vref is then at most 1 and is written with 24 bits.  The first bound of a column leaves two bits, as the
// largest of many scores lies about that far above the largest of a tile's; later ones leave one.  O stays in s32 while
// the bounds stand (at most 33024 keys a unit: |sum| <= 33024 * 255 * 128 < 2^31) and is added to fp32 when they move
// and at the unit's end.
//
// Roles of a CTA (one per SM): warps 0-7 and 8-15 are two softmax workers (thread = key row of S, dim row of O, and one
// half of the columns), which take the tiles in turn, each with its own S, O, bounds and sums, so one's latencies run
// under the other's work; warps 16-18 load (cp.async; int4 is unpacked to bytes 16 q on the way); warp 19 issues the MMAs.
// Twenty warps leave a thread 96 registers, enough for its columns; with one more it would be 80.  A unit is one kv head of one
// sequence with up to 32 columns.  All tiles of all units form one row, cut into equal ranges, one per CTA (the lengths
// are read on the device, so ragged batches stay balanced); units that a cut divides leave partial results in the
// workspace, and a second kernel joins them.  Every wait is bounded; one that runs out turns the CTA's results into NaN.
#include <math.h>

#include "abi_util.h"
#include "common.cuh"
#include "launch_state.h"
#include "rswa_tree.cuh"
#include "umma.cuh"

namespace focr {
namespace {

constexpr int RD = TREE_DIM, RW = TREE_RING, TILE = 128;
constexpr int SOFT = 16, LOADERS = 3, WARPS = SOFT + LOADERS + 1, PT = 32 * WARPS;
constexpr int ST = 32 * SOFT, LT = 32 * LOADERS;
constexpr int JT = 128;                       // threads of the joining kernel
constexpr int CMAX = 32;                      // columns of a unit
constexpr float MARGIN_FIRST = 2.f, MARGIN = 1.f;   // log2 that a bound leaves above the largest score seen
constexpr float V_MARGIN = 1.125f;            // and the value scales' bound above the largest one
constexpr uint64_t LIMIT_NS = 2000000000ull;  // bound of every wait
// A partial result: the columns' references, sums and unnormalised outputs.
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
// the thread's copies so far arrive on the barrier once they have landed
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
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
__device__ __forceinline__ void st8(uint32_t taddr, const float (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
// a barrier of a worker's threads that also tells whether any of them said so
__device__ __forceinline__ bool any_of_worker(int worker, bool mine) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %2, 0;\n\t"
        "barrier.cta.red.or.pred p, %1, 256, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(2 + worker), "r"((uint32_t)mine)
        : "memory");
    __syncwarp();
    return r != 0;
}
__device__ __forceinline__ void worker_sync(int worker) {
    __syncwarp();
    named_bar_sync(2 + worker, ST / 2);
}
__device__ __forceinline__ void softmax_sync() {   // both workers
    __syncwarp();
    named_bar_sync(1, ST);
}
// the largest of the warp's values (integers that order as the floats do)
__device__ __forceinline__ float warp_max(float x) {
    int i = __float_as_int(x);
    i ^= (i >> 31) & 0x7fffffff;
    i = __reduce_max_sync(0xffffffffu, i);
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

template <bool INT4, int CP>
struct Sizes {
    static constexpr int N = 3 * CP;                                  // columns in digits
    static constexpr int STAGES = INT4 ? 3 : CP == 16 ? 6 : 5;        // tiles of bytes
    static constexpr int PACKED = CP == 16 ? 5 : 3;                   // int4: tiles of nibbles on their way
    static constexpr int KV = TILE * RD;                              // bytes of K (or V) of a tile
    static constexpr int STAGE = 2 * KV;
    static constexpr int PACK = 2 * KV / 2 + 8 * TILE;                // nibbles of K and V, and scales
    static constexpr int Q_OFF = STAGES * STAGE + (INT4 ? PACKED * PACK : 0), P_OFF = Q_OFF + N * RD, S_OFF = P_OFF + 2 * N * TILE;
    // tensor memory: each worker's S, O and fp32 sums
    static constexpr int T_O = 2 * N, T_ACC = 4 * N;
    static_assert(4 * N + 2 * CP <= 512, "tensor memory");
    static_assert(CP * RD * 4 <= 2 * N * TILE, "a worker's results fit where the weights were");
};

constexpr int STAGES_MAX = 6;

template <int CP>
struct Shared {
    float part[CP][RD];                  // the drafted keys' part
    float part_m[CP], part_l[CP];
    float scales[STAGES_MAX][2][TILE];            // of the stages' tiles: ks, vs
    float2 col[2][CP];                   // a column's step (score in log2 = dot * key scale * step) and each worker's bound
    float2 moved[2][CP];                 // bounds that moved: by how much, and the factor for the column's sums
    float red[2][8][CP / 2 + 1];           // by worker and warp
    float4 factor[CP];                   // of the workers' and the drafted keys' parts, and of the result
    float total_m[CP], total_l[CP];
    int ages[CP];                        // ring slots younger than this are seen
    unsigned long long line[TREE_MAX];
    int par[TREE_MAX];
    uint64_t full[STAGES_MAX], empty[STAGES_MAX], s_full[2], s_free[2], p_full[2], p_free[2], q_full;
    int scan[WARPS + 4];
    float vref[2];                       // bounds of the value scales
    int fresh[2];                        // the next P V starts O anew
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
    int b, unit, tile;   // unit of the sequence: kv head * groups + column group
};
__device__ int all_tiles(const TreeParams& p, int* scan) {
    int mine = 0;
    for (int b = threadIdx.x; b < p.B; b += PT) mine += sequence_tiles(p, b);
    return cta_scan<WARPS>(mine, scan) * p.hk * p.groups;
}
__device__ Place find_tile(const TreeParams& p, int at, int* scan) {
    const int per = p.hk * p.groups;
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += PT) {
        const int b = b0 + threadIdx.x, own = b < p.B ? sequence_tiles(p, b) : 0;
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

// The part of a unit that a CTA has.  Every warp reads it for itself.
struct Segment {
    int b, h, R, n, L;
    int col0, cols;        // its columns
    int first, count;      // its tiles of keys
    int taken;             // tiles of the range that it uses up
    bool bad, dead, head, complete;   // dead: nothing to compute
};
__device__ Segment segment_at(const TreeParams& p, const Place& at, int left) {
    Segment s;
    const int lane = threadIdx.x & 31;
    s.b = at.b, s.h = at.unit / p.groups, s.col0 = at.unit % p.groups * CMAX, s.cols = min(CMAX, p.N * p.G - s.col0);
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
    s.dead = s.bad || s.col0 / p.G >= s.L;
    const int keys = s.dead ? 0 : (s.R + TILE - 1) / TILE + (s.n > 0);
    s.count = max(0, min(s.first + s.taken, keys) - s.first);
    s.head = s.first == 0, s.complete = s.head && s.taken == all;
    return s;
}
__device__ __forceinline__ void advance(const TreeParams& p, Place& at, int& left, const Segment& s) {
    left -= s.taken;
    at.tile = 0;
    if (++at.unit == p.hk * p.groups) at.unit = 0, ++at.b;
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

// A worker's O (if `filled`; every P V so far has completed) joins its fp32 sums (if `summed`), times the columns' factors.
// Rare, and kept out of line: inlined it would take registers from the tiles' loop.
template <bool INT4, int CP>
__device__ __noinline__ void drain(uint32_t t_o, uint32_t t_acc, float vref, bool filled, bool summed, const float2* moved) {   // half the columns
    const float gain = vref * ((INT4 ? 1.f / 16.f : 1.f) / P_TOP);
#pragma unroll 1
    for (int c = 0; c < CP / 2; c += 8) {
        int o2[8], o1[8], o0[8], old[8];
        float a[8];
        ld8(t_o + c, o0);
        ld8(t_o + CP + c, o1);
        ld8(t_o + 2 * CP + c, o2);
        ld8(t_acc + c, old);
        wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[j] = summed ? __int_as_float(old[j]) : 0.f;
            if (filled) a[j] = fmaf(fmaf((float)o2[j], 65536.f, fmaf((float)o1[j], 256.f, (float)o0[j])), gain, a[j]);
            if (moved) a[j] *= moved[c + j].y;
        }
        st8(t_acc + c, a);
    }
    umma::wait_st();
}

// Query digits, columns' constants and the drafted keys' part of a unit; by the softmax warps.
template <bool INT4, int CP>
__device__ __noinline__ void prepare_columns(const TreeParams& p, const Segment& s, Shared<CP>& sh, uint8_t* sq) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i0 = 0; i0 < CP / SOFT; ++i0) {
        float4 q[1], k4[1][4], v4[1][4];
        unsigned long long line[1];
#pragma unroll
        for (int i = 0; i < 1; ++i) {
            const int c = warp + (i0 + i) * SOFT, node = (s.col0 + c) / p.G;
            const bool live = c < s.cols && node < s.L;
            q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (live)
                q[i] = __ldg(reinterpret_cast<const float4*>(p.q + (((size_t)s.b * p.N + node) * p.hq + s.h * p.G + (s.col0 + c) % p.G) * RD) + lane);
            line[i] = live && s.head ? sh.line[node] : 0ull;
            unsigned long long rest = line[i];
            draft_load(p, s.b, s.h, lane, rest, k4[i], v4[i]);
            if (lane == 0) sh.ages[c] = live ? min(s.n, RW - __popcll(sh.line[node])) : 0;
        }
#pragma unroll
        for (int i = 0; i < 1; ++i) {
            const int c = warp + (i0 + i) * SOFT;
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
            if (lane == 0)
                sh.col[0][c] = sh.col[1][c] = make_float2(a / Q_TOP * (SCORE_SCALE * LOG2E * (INT4 ? 1.f / 16.f : 1.f)), 0.f);
            const DraftPart dp = draft_attend(p, s.b, s.h, lane, x, line[i], k4[i], v4[i]);
            reinterpret_cast<float4*>(sh.part[c])[lane] = dp.o;
            if (lane == 0) sh.part_m[c] = dp.m, sh.part_l[c] = dp.l;
        }
    }
}

// A unit's result from both workers' sums and the drafted keys' part; by the softmax warps.
template <int CP>
__device__ __noinline__ void finish(const TreeParams& p, const Segment& s, Shared<CP>& sh, float* other, uint32_t t_acc, int dim) {
    const int tid = threadIdx.x, me = tid / (ST / 2), row = tid % TILE, c0 = tid / TILE % 2 * (CP / 2);
    if (tid < CP) {
        const int c = tid;
        const float m0 = s.count > 0 ? sh.col[0][c].y : NONE, m1 = s.count > 1 ? sh.col[1][c].y : NONE, pm = sh.part_m[c];
        const float M = fmaxf(fmaxf(m0, m1), pm), f0 = ex2(m0 - M), f1 = ex2(m1 - M), g = ex2(pm - M);
        const int hf = c / (CP / 2) * 4, cr = c % (CP / 2);
        const float (*r0)[CP / 2 + 1] = sh.red[0] + hf, (*r1)[CP / 2 + 1] = sh.red[1] + hf;
        const float l0 = (r0[0][cr] + r0[1][cr]) + (r0[2][cr] + r0[3][cr]), l1 = (r1[0][cr] + r1[1][cr]) + (r1[2][cr] + r1[3][cr]);
        const float l = fmaf(f0, l0, fmaf(f1, l1, g * sh.part_l[c])), r = s.complete ? 1.f / l : 1.f;
        sh.factor[c] = make_float4(f0 * r, f1 * r, g * r, 0.f);
        sh.total_m[c] = M, sh.total_l[c] = l;
    }
    if (me == 1) {   // worker 1's results go where the weights were
#pragma unroll 1
        for (int c = c0; c < c0 + CP / 2; c += 8) {
            int a[8];
            ld8(t_acc + c - c0, a);
            wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) other[(c + j) * RD + row] = s.count > 1 ? __int_as_float(a[j]) : 0.f;
        }
    }
    softmax_sync();
    if (me == 0) {
        float* part = p.part + ((size_t)blockIdx.x * 2 + s.head) * PART_FLOATS;
#pragma unroll 1
        for (int c = c0; c < c0 + CP / 2; c += 8) {
            int a[8];
            ld8(t_acc + c - c0, a);
            wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int cc = c + j, x = s.col0 + cc, node = x / p.G;
                if (cc >= s.cols || node >= s.L) continue;
                const float4 f = sh.factor[cc];
                const float o = fmaf(f.x, s.count > 0 ? __int_as_float(a[j]) : 0.f, fmaf(f.y, other[cc * RD + row], f.z * sh.part[cc][dim]));
                if (s.complete) {
                    p.out[(((size_t)s.b * p.N + node) * p.hq + s.h * p.G + x % p.G) * RD + dim] = o;
                } else {
                    part[PART_O + cc * RD + dim] = o;
                    if (row == 0) part[cc] = sh.total_m[cc], part[PART_L + cc] = sh.total_l[cc];
                }
            }
        }
    }
}

template <bool INT4, int CP>
__global__ void __launch_bounds__(PT, 1) rswa_wide_kernel(const __grid_constant__ TreeParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using Z = Sizes<INT4, CP>;
    constexpr int N = Z::N, STAGES = Z::STAGES;
    Shared<CP>& sh = *reinterpret_cast<Shared<CP>*>(smem + Z::S_OFF);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < STAGES_MAX; ++i) mbar_init(&sh.full[i], LT), mbar_init(&sh.empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1), mbar_init(&sh.s_free[i], SOFT / 2);
            mbar_init(&sh.p_full[i], SOFT / 2), mbar_init(&sh.p_free[i], 1);
            sh.fresh[i] = 1;
        }
        mbar_init(&sh.q_full, SOFT);
        fence_barrier_init();
        sh.gave_up = 0;
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
    const uint32_t tmem = sh.tmem;
    int left = mine;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_wait_bounded(bar, parity, LIMIT_NS)) return true;
        sh.gave_up = 1;
        return false;
    };

    if (warp < SOFT) {
        // ------------------------------------------------------------ softmax
        constexpr int HALF = CP / 2;   // columns of a thread
        const int me = warp >> 3, row = (warp & 3) * 32 + lane, c0 = (warp >> 2 & 1) * HALF;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16), t_s = lanes + me * N + c0, t_o = lanes + Z::T_O + me * N + c0,
                       t_acc = lanes + Z::T_ACC + me * CP + c0;
        const int dim = INT4 ? 32 * (row / 32) + 2 * (row % 16) + ((row / 16) & 1) : row;   // of the thread's lane of O
        uint8_t* sp = smem + Z::P_OFF + me * N * TILE;
        auto preset = [&] {   // S accumulates onto the pattern that reads as MAGIC + sum
#pragma unroll
            for (int d = 0; d < 3; ++d)
#pragma unroll
                for (int c = 0; c < HALF; c += 8) st8(t_s + d * CP + c, MAGIC_BITS);
            umma::wait_st();
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.s_free[me]);
        };
        preset();
        int it = 0, k = 0;   // tiles of the CTA before this segment; this worker's tiles so far
        bool ok = true;
        while (left > 0 && ok) {   // left by all threads at once
            const Segment s = segment_at(p, at, left);
            if (s.bad && s.head) {
                const int live = min(s.cols, (s.L < 0 || s.L > p.N ? p.N : s.L) * p.G - s.col0);
                for (int i = tid; i < live * RD; i += ST) {
                    const int c = s.col0 + i / RD;
                    p.out[(((size_t)s.b * p.N + c / p.G) * p.hq + s.h * p.G + c % p.G) * RD + i % RD] = __int_as_float(0x7fc00000);
                }
            }
            if (!s.dead) {
                // ---- lines of the tree, query digits, drafted keys
                if (tid < s.L) sh.par[tid] = p.parent ? __ldg(p.parent + (size_t)s.b * p.N + tid) : tid - 1;
                softmax_sync();
                if (tid < s.L) {
                    unsigned long long line = 0;
                    for (int j = tid; j >= 0; j = sh.par[j]) line |= 1ull << j;
                    sh.line[tid] = line;
                }
                if (tid < 2) sh.vref[tid] = TINY;
                softmax_sync();
                prepare_columns<INT4, CP>(p, s, sh, smem + Z::Q_OFF);
                umma::fence_smem_to_async();
                softmax_sync();
                if (lane == 0 && s.count > 0) mbar_arrive(&sh.q_full);

                float sum[HALF];
#pragma unroll
                for (int c = 0; c < HALF; ++c) sum[c] = 0.f;
                bool filled = false, summed = false;   // O holds something; so do the fp32 sums
                for (int i = me; i < s.count; i += 2, ++k) {   // left by all threads of the worker at once
                    const int stage = (it + i) % STAGES;
                    const TileAt ta = tile_at(p, s, s.first + i);
                    ok = ok && wait(&sh.full[stage], (it + i) / STAGES & 1) && wait(&sh.s_full[me], k & 1);
                    __syncwarp();
                    umma::fence_after_sync();
                    const bool in = row < ta.rows;
                    const float ks = in ? sh.scales[stage][0][row] : 0.f, vs = in ? sh.scales[stage][1][row] : 0.f;
                    float x[HALF], top = -INFINITY;   // scores relative to the bounds, base 2
#pragma unroll
                    for (int c = 0; c < HALF; c += 8) {
                        int d2[8], d1[8], d0[8];
                        ld8(t_s + c, d0);
                        ld8(t_s + CP + c, d1);
                        ld8(t_s + 2 * CP + c, d2);
                        wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 b = sh.col[me][c0 + c + j];
                            x[c + j] = fmaf((upper(d2[j]) + lower(d1[j], d0[j])) * ks, b.x, -b.y);
                        }
                    }
                    preset();
                    if (ta.ring) {
                        const int age = (s.n - 1 - row) & (RW - 1);
#pragma unroll
                        for (int c = 0; c < HALF; ++c)
                            if (!in || age >= sh.ages[c0 + c]) x[c] = -INFINITY;
                    } else if (!in) {
#pragma unroll
                        for (int c = 0; c < HALF; ++c) x[c] = -INFINITY;
                    }
#pragma unroll
                    for (int c = 0; c < HALF; ++c) top = fmaxf(top, x[c]);
                    const bool first = !filled && !summed;   // the worker's first tile of the unit sets the bounds
                    if (any_of_worker(me, first || top > 0.f || vs > sh.vref[me] || !ok)) {
                        // ---- bounds move: columns' and scales' largest values of the tile
                        const float vref = sh.vref[me];
#pragma unroll
                        for (int c = 0; c < HALF; ++c) {
                            const float m = warp_max(x[c]);
                            if (lane == 0) sh.red[me][warp & 7][c] = m;
                        }
                        const float vm = warp_max(vs);
                        if (lane == 0) sh.red[me][warp & 7][HALF] = vm;
                        if (filled) ok = wait(&sh.p_free[me], (k - 1) & 1) && ok;
                        __syncwarp();
                        umma::fence_after_sync();
                        if (any_of_worker(me, !ok)) {
                            ok = false;
                            break;
                        }
                        if (row < HALF) {
                            const float (*r)[HALF + 1] = sh.red[me] + (warp & 4);
                            const float over = fmaxf(fmaxf(r[0][row], r[1][row]), fmaxf(r[2][row], r[3][row]));   // above the bound
                            const float2 b = sh.col[me][c0 + row];
                            float by = over > 0.f ? over + MARGIN : 0.f;
                            if (first) by = over == -INFINITY ? 0.f : over + MARGIN_FIRST;   // (a column without a node sees nothing)
                            sh.moved[me][c0 + row] = make_float2(by, ex2(-by));
                            sh.col[me][c0 + row] = make_float2(b.x, b.y + by);
                        }
                        if (row == 0 && c0 == 0) {
                            const float v = fmaxf(fmaxf(sh.red[me][0][HALF], sh.red[me][1][HALF]), fmaxf(sh.red[me][2][HALF], sh.red[me][3][HALF]));
                            if (v > vref) sh.vref[me] = V_MARGIN * v;
                            sh.fresh[me] = 1;
                        }
                        worker_sync(me);
#pragma unroll
                        for (int c = 0; c < HALF; ++c) {
                            const float2 by = sh.moved[me][c0 + c];
                            x[c] -= by.x;
                            sum[c] *= by.y;
                        }
                        if (filled || summed) drain<INT4, CP>(t_o, t_acc, vref, filled, summed, sh.moved[me] + c0);
                        summed |= filled;
                        filled = false;
                    }
                    // ---- weights: 24 bits, as three digits, [key][column] for the second product
                    const float vn = vs * (P_TOP / sh.vref[me]);
                    if (k > 0) ok = wait(&sh.p_free[me], (k - 1) & 1) && ok;   // the weights of the tile before have been used
                    uint8_t* at8 = sp + (row >> 3) * (N / 16 * 128) + (row & 7) * 16;
#pragma unroll
                    for (int c = 0; c < HALF; c += 8) {
                        uint32_t w[3][2];
#pragma unroll
                        for (int e = 0; e < 8; e += 4) {
                            uint32_t u[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float y = ex2(x[c + e + j]);
                                sum[c + e + j] += y;
                                u[j] = __float2uint_rn(y * vn);
                            }
                            const uint32_t t0 = __byte_perm(u[0], u[1], 0x5140), t1 = __byte_perm(u[2], u[3], 0x5140);
                            const uint32_t t2 = __byte_perm(u[0], u[1], 0x0062), t3 = __byte_perm(u[2], u[3], 0x0062);
                            w[0][e / 4] = __byte_perm(t0, t1, 0x5410);
                            w[1][e / 4] = __byte_perm(t0, t1, 0x7632);
                            w[2][e / 4] = __byte_perm(t2, t3, 0x5410);
                        }
#pragma unroll
                        for (int d = 0; d < 3; ++d) {
                            const int n = d * CP + c0 + c;   // a multiple of 8; 16 columns a chunk
                            *reinterpret_cast<uint2*>(at8 + (n >> 4) * 128 + (n & 15)) = make_uint2(w[d][0], w[d][1]);
                        }
                    }
                    umma::fence_smem_to_async();
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.p_full[me]);
                    filled = true;
                }
                // ---- the unit's sums, and the drafted keys
                if (filled) {
                    ok = ok && wait(&sh.p_free[me], (k - 1) & 1);
                    __syncwarp();
                    umma::fence_after_sync();
                    drain<INT4, CP>(t_o, t_acc, sh.vref[me], true, summed, nullptr);
                }
#pragma unroll
                for (int c = 0; c < HALF; ++c) {
                    float l = sum[c];
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                    if (lane == 0) sh.red[me][warp & 7][c] = l;
                }
                if (!ok) sh.gave_up = 1;
                softmax_sync();
                ok = *(volatile int*)&sh.gave_up == 0;
                finish<CP>(p, s, sh, reinterpret_cast<float*>(smem + Z::P_OFF), t_acc, dim);
                if (tid < 2) sh.fresh[tid] = 1;
                softmax_sync();
            }
            it += s.count;
            advance(p, at, left, s);
        }
    } else if (warp < SOFT + LOADERS) {
        // ------------------------------------------------------------ loads
        const int t = tid - ST;
        int it = 0;
        bool ok = true;
        if (!INT4) {
            while (left > 0 && ok) {
                const Segment s = segment_at(p, at, left);
                for (int tile = s.first; tile < s.first + s.count && ok; ++tile, ++it) {
                    const int stage = it % STAGES;
                    const TileAt ta = tile_at(p, s, tile);
                    if (it >= STAGES) ok = wait(&sh.empty[stage], (it / STAGES - 1) & 1);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    const KvView& v = ta.ring ? p.ring : p.ref;
                    const uint32_t to = smem_u32(smem) + stage * Z::STAGE;
                    // an instruction copies four chunks of eight rows, eight lanes a core matrix
                    const int r0 = lane & 7, j0 = lane >> 3;
#pragma unroll
                    for (int e = 0; e < (2 * TILE / 8 + LOADERS - 1) / LOADERS; ++e) {
                        const int i = warp - SOFT + e * LOADERS;
                        if (i >= 2 * TILE / 8) break;
                        const int r = (i >> 1 << 3) + r0, ch = (i & 1) * 4 + j0;
                        const size_t src = (ta.row + min(r, ta.rows - 1)) * RD + ch * 16;
                        const uint32_t dst = to + (r >> 3) * 1024 + ch * 128 + r0 * 16;
                        cp16(dst, v.k + src);
                        cp16(dst + Z::KV, v.v + src);
                    }
                    for (int i = t; i < TILE; i += LT) {
                        const size_t sr = ta.row + min(i, ta.rows - 1);
                        cp4(smem_u32(&sh.scales[stage][0][i]), v.ks + sr);
                        cp4(smem_u32(&sh.scales[stage][1][i]), v.vs + sr);
                    }
                    cp_arrive(&sh.full[stage]);   // once they have landed; the reader passes them on to the tensor core
                }
                advance(p, at, left, s);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
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
                    const int r0 = lane & 7, j = lane >> 3;
#pragma unroll
                    for (int e = 0; e < (TILE / 8 + LOADERS - 1) / LOADERS; ++e) {   // four chunks of eight rows
                        const int i = warp - SOFT + e * LOADERS;
                        if (i >= TILE / 8) break;
                        const size_t src = (ta.row + min(8 * i + r0, ta.rows - 1)) * (RD / 2) + j * 16;
                        cp16(smem_u32(to + (i * 32 + lane) * 16), v.k + src);
                        cp16(smem_u32(to + Z::KV / 2 + (i * 32 + lane) * 16), v.v + src);
                    }
                    for (int i = t; i < TILE; i += LT) {
                        const size_t sr = ta.row + min(i, ta.rows - 1);
                        cp4(smem_u32(to + Z::KV + 4 * i), v.ks + sr);
                        cp4(smem_u32(to + Z::KV + 4 * TILE + 4 * i), v.vs + sr);
                    }
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
                    cp_wait<Z::PACKED - 1>();   // that many younger tiles may be on their way
                    if (it >= STAGES) ok = wait(&sh.empty[stage], (it / STAGES - 1) & 1);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    const uint8_t* fr = smem + STAGES * Z::STAGE + it % Z::PACKED * Z::PACK;
                    uint8_t* to = smem + stage * Z::STAGE;
                    const int r0 = lane & 7, j = lane >> 3;
                    constexpr int EACH = (TILE / 8 + LOADERS - 1) / LOADERS;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        uint4 n[EACH];
#pragma unroll
                        for (int e = 0; e < EACH; ++e) {
                            const int i = min(warp - SOFT + e * LOADERS, TILE / 8 - 1);   // (the last one twice by some warps)
                            n[e] = lds128(fr + kv * (Z::KV / 2) + (i * 32 + lane) * 16);
                        }
#pragma unroll
                        for (int e = 0; e < EACH; ++e) {
                            const int i = warp - SOFT + e * LOADERS;
                            if (i >= TILE / 8) break;
                            uint8_t* dst = to + kv * Z::KV + i * 1024 + 2 * j * 128 + r0 * 16;
                            *reinterpret_cast<uint4*>(dst) = make_uint4((n[e].x << 4) & 0xF0F0F0F0u, (n[e].y << 4) & 0xF0F0F0F0u, (n[e].z << 4) & 0xF0F0F0F0u, (n[e].w << 4) & 0xF0F0F0F0u);
                            *reinterpret_cast<uint4*>(dst + 128) = make_uint4(n[e].x & 0xF0F0F0F0u, n[e].y & 0xF0F0F0F0u, n[e].z & 0xF0F0F0F0u, n[e].w & 0xF0F0F0F0u);
                        }
                    }
                    for (int i = t; i < TILE; i += LT) {
                        sh.scales[stage][0][i] = *reinterpret_cast<const float*>(fr + Z::KV + 4 * i);
                        sh.scales[stage][1][i] = *reinterpret_cast<const float*>(fr + Z::KV + 4 * TILE + 4 * i);
                    }
                    umma::fence_smem_to_async();
                    mbar_arrive(&sh.full[stage]);
                }
                advance(p, at, left, s);
            }
            cp_wait<0>();
        }
    } else {
        // ------------------------------------------------------------ products
        // One thread, with as few instructions a tile as can be: it shares its scheduler with five other warps, and a
        // tile is worth 1500 cycles of memory.
        constexpr uint32_t IS = idesc_i8(N, true, false, false), IO = idesc_i8(N, false, true, true);
        constexpr uint32_t P_GROUP = N / 16 * 128;   // bytes of eight keys' weights
        const uint64_t k_desc = umma::sdesc_kmajor(smem_u32(smem), 128, 1024), v_desc = umma::sdesc_kmajor(smem_u32(smem) + Z::KV, 1024, 128);
        const uint64_t q_desc = umma::sdesc_kmajor(smem_u32(smem) + Z::Q_OFF, 128, 1024);
        const uint64_t p_desc = umma::sdesc_kmajor(smem_u32(smem) + Z::P_OFF, P_GROUP, 128);
        const uint32_t empty0 = smem_u32(&sh.empty[0]);
        int stage_s = 0, phase_s = 0, stage_p = 0, scores = 0, done = 0, seg = 0;   // scores, done: bit w is worker w's phase
        bool ok = true;
        while (left > 0 && ok) {
            const Segment s = segment_at(p, at, left);
            if (lane == 0 && s.count > 0) {
                ok = wait(&sh.q_full, seg & 1);
                ++seg;
                for (int i = 0; i < s.count + 2 && ok; ++i) {
                    const int w = i & 1;
                    if (i > 1) {   // O += V^T P of tile i - 2, which frees its worker's weights and its place
                        ok = wait(&sh.p_full[w], done >> w & 1);
                        if (!ok) break;
                        done ^= 1 << w;
                        umma::fence_after_sync();
                        const bool fresh = *(volatile int*)&sh.fresh[w] != 0;
                        const uint64_t v = v_desc + (uint32_t)(stage_p * (Z::STAGE >> 4)), pw = p_desc + (uint32_t)(w * (N * TILE >> 4));
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 keys each: four groups of eight rows
                            mma_i8(tmem + Z::T_O + w * N, v + (4096 >> 4) * k, pw + (4 * P_GROUP >> 4) * k, IO, k > 0 || !fresh);
                        *(volatile int*)&sh.fresh[w] = 0;
                        umma::commit(smem_u32(&sh.p_free[w]));
                        umma::commit(empty0 + 8 * stage_p);
                        if (++stage_p == STAGES) stage_p = 0;
                    }
                    if (i < s.count) {   // S of tile i
                        ok = wait(&sh.full[stage_s], phase_s) && wait(&sh.s_free[w], scores >> w & 1);
                        if (!ok) break;
                        scores ^= 1 << w;
                        if (!INT4) umma::fence_smem_to_async();   // (the loaders of int4 have done it)
                        umma::fence_after_sync();
                        const uint64_t kd = k_desc + (uint32_t)(stage_s * (Z::STAGE >> 4));
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 dims each: two chunks
                            mma_i8(tmem + w * N, kd + (256 >> 4) * k, q_desc + (256 >> 4) * k, IS, true);
                        umma::commit(smem_u32(&sh.s_full[w]));
                        if (++stage_s == STAGES) stage_s = 0, phase_s ^= 1;
                    }
                }
            }
            ok = __all_sync(0xffffffffu, ok);
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
            for (int i = tid; i < s.cols * RD; i += PT) {
                const int c = i / RD, x = s.col0 + c, node = x / p.G;
                const float nan = __int_as_float(0x7fc00000);
                if (!s.complete) {
                    part[PART_O + i] = nan;
                    if (i % RD == 0) part[c] = 0.f, part[PART_L + c] = nan;
                } else if (s.bad || node < s.L) {
                    p.out[(((size_t)s.b * p.N + node) * p.hq + s.h * p.G + x % p.G) * RD + i % RD] = nan;
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
    const int tid = threadIdx.x, per_b = p.hk * p.groups, b = blockIdx.x / per_b, unit = blockIdx.x % per_b;
    pdl_wait();
    // the unit's tiles in the row of all tiles, and the CTAs that had them
    int all = 0, before = 0;
    for (int i = tid; i < p.B; i += JT) {
        const int own = sequence_tiles(p, i);
        all += own;
        if (i < b) before += own;
    }
    all = cta_scan<JT / 32>(all, scan) * per_b;
    before = cta_scan<JT / 32>(before, scan);
    const int own = sequence_tiles(p, b), per = (all + ctas - 1) / ctas;
    const int64_t from = (int64_t)before * per_b + (int64_t)unit * own;
    const int c0 = (int)(from / per), c1 = (int)((from + own - 1) / per);
    if (c0 == c1) return;
    const Segment s = segment_at(p, Place{b, unit, 0}, own);
    if (s.bad) return;
    for (int c = blockIdx.y; c < s.cols; c += gridDim.y) {
        const int x = s.col0 + c, node = x / p.G;
        if (node >= s.L) return;
        float M = NONE, l = 0.f, o = 0.f;
        for (int i = c0; i <= c1; ++i) M = fmaxf(M, __ldcg(p.part + ((size_t)i * 2 + (i == c0)) * PART_FLOATS + c));
        for (int i = c0; i <= c1; ++i) {
            const float* part = p.part + ((size_t)i * 2 + (i == c0)) * PART_FLOATS;
            const float f = ex2(__ldcg(part + c) - M);
            l = fmaf(f, __ldcg(part + PART_L + c), l);
            o = fmaf(f, __ldcg(part + PART_O + c * RD + tid), o);
        }
        p.out[(((size_t)b * p.N + node) * p.hq + s.h * p.G + x % p.G) * RD + tid] = o / l;
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
    const int cols = p.N * p.G < CMAX ? p.N * p.G : CMAX;
    return launch_kernel((const void*)rswa_wide_join_kernel, dim3((unsigned)p.B * p.hk * p.groups, cols < 8 ? cols : 8), dim3(JT), 0, 1,
                         more, st);
}
template <bool INT4>
cudaError_t launch_wide_for(TreeParams& p, cudaStream_t st) {
    p.groups = (p.N * p.G + CMAX - 1) / CMAX;
    return p.N * p.G <= 16 ? launch_wide_as<INT4, 16>(p, st) : launch_wide_as<INT4, 32>(p, st);
}

}  // namespace

int wide_ctas() { return device_sms() > 0 ? device_sms() : 148; }
size_t wide_part_bytes() { return ((size_t)wide_ctas() * 2 * PART_FLOATS * sizeof(float) + 255) & ~(size_t)255; }
cudaError_t launch_wide(TreeParams& p, bool int4, cudaStream_t st) {
    return int4 ? launch_wide_for<true>(p, st) : launch_wide_for<false>(p, st);
}

}  // namespace focr
