// ck_int4_matvec and ck_int4_quantize: products of a few state rows with 4-bit
// weights, and the rounding that makes such weights.
#include "int4.h"

namespace ck {
namespace {

// The product of a few rows, on tensor cores.  With w = s (q - z) a group's sum is
// s * sum (q - z) x, and q - z, a whole number of at most 15 in magnitude, is exact
// in a 16-bit float; so x meets the weights as they are, sums are held in 32 bits
// and the scale is applied once a group.  A 32-bit x is cut into three bf16 parts
// of eight bits, 24 together over the whole range of the type; the parts are
// columns of their own.  (Two fp16 parts under a scale of the row, and the zero
// points taken off the sums, cost a third fewer instructions and two thirds of the
// columns, but an outlier that meets q = z then drowns the rest of its row.)
//
// What bounds it is the stream of weights: 0.5 byte each, while a column costs
// 2 operations a weight.  So the weights flow through a ring of tensor copies that
// each warp keeps for itself, and no warp waits for another until the end.
//
// Measured: 1 x 211,577 bf16 by 4,096 rows, groups of 128, 94 us (4.9 TB/s), 1 x 5,000
// fp32 by 64,000 rows 40 us (4.3 TB/s), 4 x 20,000 fp16 by 16,384 rows in groups of 32
// with zero points 69 us (2.8 TB/s: with schedulers that issue 44% of their cycles from
// three warps each it waits for a group's way through ldmatrix, unpacking, two products
// and a scale), 1 x 5,000 fp32 by 256 rows 8.8 us (a start, x to shared memory, two units
// a warp, the sums of twelve warps).
//
// A unit is 32 weight rows by 256 columns (4 KB).  K is cut into slabs whose x
// fits in shared memory; the units, in the order (slab, 32-row tile, chunk),
// are dealt to CTAs, and a CTA's to its warps, in equal runs.  A run's first and
// last tile may be shared with its neighbours: those sums meet in shared memory
// and, where a tile crosses CTAs or slabs, in the slots of `partial`, which
// k_join adds up in a fixed order.
constexpr int kHalf = 128;  // columns: scales are taken up for half a unit

// Warps of a CTA, one CTA on an SM, and units of a warp's ring.  Sixteen keep more on its
// way and pay for it at the start and at the end, so they are taken where a warp's run is
// long: 1 x 200,000 fp16 by 4,096 in groups of 128 (55 units a warp of twelve) takes 94 us
// by twelve and 86 by sixteen, 4 x 20,000 by 32,768 (44) 79 and 74, 1 x 5,000 fp32 by 8,192
// (3) 11.9 and 13.6.  Between 10 and 40 units sixteen are up to 10% faster with 16-bit x
// and even with 32-bit x, whose three parts leave them no registers: there the two lie
// within 2% of each other up to 55 units.  4 x 200,000 fp16 loses by sixteen, 100 and 104.
constexpr int kFewWarps = 12, kManyWarps = 16, kLongRun = 40;
__host__ __device__ constexpr int ring_units(int warps) { return warps == kFewWarps ? 3 : 2; }

// Tables of scales and zero points: a second one, filled in the middle of a unit while
// the first is in use, where groups are short (a table a unit) or runs long, and x
// leaves room.  1 x 200,000 x 4,096 in groups of 32 takes 221 us with one and 170 with
// two, 1 x 211,577 x 4,096 in groups of 128 96 and 94; but 1 x 5,000 x 256 8.2 and 9.4.
__host__ __device__ constexpr int tables(int column_tiles, int group, int warps) {
    return column_tiles == 1 && (group == 32 || warps == kManyWarps) ? 2 : 1;
}

struct MatvecPlan {
    int rows;          // rows of x in this launch
    int64_t tiles;     // 32-row tiles of V
    int64_t chunks;    // chunks of K
    int64_t slabs;     // parts of K
    int64_t ctas;
    int warps;         // of a CTA
    int aligned;       // one slab, and CTAs take whole tiles: nothing crosses them
    Deal chunk;        // chunks to slabs
    // Where there are no more slabs than CTAs, a CTA keeps to one slab, whose units
    // are dealt to its CTAs in equal runs; else CTAs take whole slabs.
    Deal cta;          // CTAs to slabs
    Deal slab;         // slabs to CTAs
    Deal tile;         // aligned: tiles to CTAs
    long long timeout; // cycles that a wait for a copy may last
    int extra;         // test hook: arrivals that never come
    int x_pitch;       // bytes between columns of x in shared memory
    int x_cols;        // tensor-core columns that x takes
    size_t smem;

    __host__ __device__ bool shared_slabs() const { return slabs <= ctas; }
    // slot of CTA b's part of a tile in a slab: no two parts share one, as from
    // a part to the next the tile or the CTA moves on and neither goes back
    __host__ __device__ int64_t slot(int64_t s, int64_t t, int64_t b) const {
        return s * tiles + t + (shared_slabs() ? b : 0);
    }
};

// Weights and x in bf16 (for 32-bit and bf16 x) or fp16.
template <bool HALF, bool FIRST>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    const float z = 0.f;  // FIRST: a new sum
    const float c0 = FIRST ? z : c[0], c1 = FIRST ? z : c[1], c2 = FIRST ? z : c[2], c3 = FIRST ? z : c[3];
    if constexpr (HALF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// The tensor-core column of part `part` of row m: the parts of two rows of 32-bit
// x lie in one tile of eight columns such that a lane's two sums are those of the
// two rows, and its neighbours' those of the other parts.
template <typename T> __device__ __forceinline__ int column(int m, int part) {
    return sizeof(T) == 4 ? 8 * (m >> 1) + 2 * part + (m & 1) : m;
}

// x of a slab into shared memory, one line a column, eight columns of K at a
// time in the order 0 4 1 5 2 6 3 7, in which nibbles come out of a word two at a
// time.
template <typename T>
__device__ __forceinline__ void stage_x(const MatvecArgs &a, const MatvecPlan &p, int k0, int blocks, char *xs) {
    constexpr int kParts = sizeof(T) == 4 ? 3 : 1, kBatch = sizeof(T) == 4 ? 2 : 4;
    int m = 0, j = threadIdx.x;
    auto settle = [&] {
        while (j >= blocks && m < p.rows) j -= blocks, ++m;
    };
    settle();
    while (m < p.rows) {
        T v[kBatch][8];
        int at_m[kBatch], at_j[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {  // all loads of a batch are on their way before the first is used
            at_m[i] = m;
            at_j[i] = j;
            if (m < p.rows) load8<T>(a, m, k0 + 8 * j, v[i]);
            j += blockDim.x;
            settle();
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (at_m[i] >= p.rows) break;
            uint16_t part[8][3];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (sizeof(T) == 4)
                    split3(v[i][e], part[e]);
                else
                    memcpy(&part[e][0], &v[i][e], 2);
            }
#pragma unroll
            for (int s = 0; s < kParts; ++s) {
                uint4 w;
                w.x = part[0][s] | (uint32_t)part[4][s] << 16;
                w.y = part[1][s] | (uint32_t)part[5][s] << 16;
                w.z = part[2][s] | (uint32_t)part[6][s] << 16;
                w.w = part[3][s] | (uint32_t)part[7][s] << 16;
                *(uint4 *)(xs + column<T>(at_m[i], s) * p.x_pitch + 16 * at_j[i]) = w;
            }
        }
    }
}

template <bool HALF, int GROUP, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1)
    k_matvec(const __grid_constant__ MatvecArgs a, const __grid_constant__ MatvecPlan p,
             const __grid_constant__ CUtensorMap weights) {
    extern __shared__ __align__(1024) char smem[];
    constexpr int kStages = ring_units(WARPS);
    __shared__ __align__(8) uint64_t bars[WARPS * kStages];
    __shared__ int dead;
    constexpr int kGroups = kHalf / GROUP;  // of half a unit
    // per warp: its ring, in which its last part of a sum is left when it is done; its
    // first part; scales and zero points of eight groups
    const int part_floats = kTileRows * p.rows;
    float *heads = (float *)(smem + WARPS * kStages * kUnitBytes);
    constexpr int kTables = tables(NT, GROUP, WARPS);
    float *all_scales = heads + WARPS * part_floats;  // [warps][tables][rows][8]
    uint8_t *all_zeros = (uint8_t *)(all_scales + WARPS * kTables * kTileRows * 8);
    int *part_tile = (int *)(all_zeros + WARPS * kTables * kTileRows * 8);  // [warps][first, last]
    char *xs = (char *)(part_tile + WARPS * 2);
    const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, (int)(threadIdx.x >> 5), 0);  // known to be the warp's
    const int row = lane >> 2, quad = lane & 3;
    const uint32_t my_ring = smem_at(smem) + warp * kStages * kUnitBytes, my_bars = smem_at(bars) + warp * kStages * 8;
    const Waiter wait{&dead, p.timeout};
    if (threadIdx.x == 0) dead = 0;
    if (lane == 0)
        for (int i = 0; i < kStages; ++i) barrier_init(my_bars + 8 * i, 1 + p.extra);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // A place in the ring, and how often the ring has gone round: the copy that is waited
    // for next and the one that is asked for next.
    int get = 0, get_round = 0, put = 0, under_way = 0;
    bool ok = true;
    const uint32_t my_line = lane * 128, my_swap = (lane & 7) << 4;
    float *my_scales = all_scales + warp * kTables * kTileRows * 8;
    uint8_t *my_zeros = all_zeros + warp * kTables * kTileRows * 8;
    auto part_at = [&](int w, int k) {
        return k ? (float *)(smem + w * kStages * kUnitBytes) : heads + w * part_floats;
    };
    // A lane's columns of x.  Those past the last read it again: their sums are not used.
    int x_at[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        int col = 8 * j + row;
        if (!HALF && a.dtype == CK_F32 && (col & 7) >= 6) col = 8 * j;
        while (!HALF && a.dtype == CK_F32 && 2 * (col >> 3) + (col & 1) >= p.rows) --col;
        x_at[j] = min(col, p.x_cols - 1) * p.x_pitch + quad * 16;
    }
    const int groups = (int)((a.K + GROUP - 1) / GROUP);
    asm volatile("griddepcontrol.launch_dependents;");
    const bool one = p.shared_slabs();
    const int64_t s0 = one ? p.cta.owner(blockIdx.x) : p.slab.first(blockIdx.x);
    const int64_t s1 = one ? s0 + 1 : p.slab.first(blockIdx.x + 1);
    for (int64_t s = s0; s < s1; ++s) {
        const int first = (int)p.chunk.first(s), sc = (int)p.chunk.first(s + 1) - first;  // the slab's chunks
        int64_t u0 = 0, u1 = sc * p.tiles;  // units of the slab
        if (p.aligned) {
            u0 = p.tile.first(blockIdx.x) * sc, u1 = p.tile.first(blockIdx.x + 1) * sc;
        } else if (one) {
            const int64_t b0 = p.cta.first(s);
            const Deal unit = Deal::of(u1, p.cta.first(s + 1) - b0);
            u0 = unit.first(blockIdx.x - b0), u1 = unit.first(blockIdx.x - b0 + 1);
        }
        const int tile0 = (int)quotient(u0, sc), skip = (int)(u0 - (int64_t)tile0 * sc);
        const int span = (int)(u1 - u0);
        const int w0 = (int)((int64_t)span * warp / WARPS), w1 = (int)((int64_t)span * (warp + 1) / WARPS);
        int n = w1 - w0, left = n;
        int t = tile0 + (skip + w0) / sc, c = (skip + w0) % sc;
        __syncthreads();  // the last slab's x and parts of sums are done with
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        int put_t = t, put_c = c;
        auto copy_next = [&] {
            if (left == 0 || !ok) return;
            ++under_way;
            copy_box(weights, (first + put_c) * (kChunk / 2), put_t * kTileRows, my_ring + put * kUnitBytes,
                     my_bars + 8 * put, kUnitBytes);
            put = put + 1 == kStages ? 0 : put + 1;
            if (++put_c == sc) put_c = 0, ++put_t;
            --left;
        };
        for (int i = 0; i < kStages; ++i) copy_next();
        ScaleReader<8> next{};
        constexpr int kUnits = 8 * GROUP / kChunk, kAhead = 4;  // units of eight groups
        // the eight groups after those that `next` holds, and a line of some further on
        auto load_next = [&] {
            int t1 = next.tile, e1 = next.eight + 1;
            if (e1 * kUnits >= first + sc) ++t1, e1 = first / kUnits;
            next.load(a, t1, e1, groups);  // past the last tile: nothing
            int t2 = t1, e2 = e1 + kAhead;
            if (e2 * kUnits >= first + sc) ++t2, e2 += first / kUnits - (first + sc + kUnits - 1) / kUnits;
            ScaleReader<8>::ahead(a, t2, e2, groups, e2 == first / kUnits);
        };
        int table = 0;  // of the eight groups at hand
        if (n > 0) next.load(a, t, (first + c) / kUnits, groups);
        if (lane < 2) part_tile[2 * warp + lane] = -1;
        if constexpr (HALF)
            stage_x<__half>(a, p, first * kChunk, sc * (kChunk / 8), xs);
        else if (a.dtype == CK_F32)
            stage_x<float>(a, p, first * kChunk, sc * (kChunk / 8), xs);
        else
            stage_x<__nv_bfloat16>(a, p, first * kChunk, sc * (kChunk / 8), xs);
        __syncthreads();
        if (n > 0) {
            next.leave(a, my_scales, my_zeros);
            load_next();
            __syncwarp();
        }
        float acc[NT][2][4] = {};  // [.][rows 0-15, 16-31][.]
        bool from_start = c == 0;  // this tile's part began with the slab
        for (; n > 0; --n) {
            ok = __all_sync(~0u, ok && wait(my_bars + 8 * get, get_round & 1));
            const bool whole = c + 1 == sc;
            const int in_eight = (first + c) & (kUnits - 1);
            const bool turn = whole || in_eight == kUnits - 1;  // the next unit has other eight groups
            const float *scales = my_scales + table * kTileRows * 8;
            const uint8_t *zero_points = my_zeros + table * kTileRows * 8;
            const uint32_t lines = my_ring + get * kUnitBytes + my_line;
            if (ok) {
                --under_way;
                if (++get == kStages) get = 0, ++get_round;
            }
            const char *xc = xs + c * (2 * kChunk);
#pragma unroll
            for (int half = 0; half < kChunk / kHalf; ++half) {
                if (kTables == 2 && half == 1 && turn && n > 1) {
                    // in the middle of a unit, whose products go on meanwhile
                    table ^= 1;
                    next.leave(a, my_scales + table * kTileRows * 8, my_zeros + table * kTileRows * 8);
                    load_next();
                }
                float scale[4][kGroups];  // of rows row + 8 h
                uint32_t zeros[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int at = (row + 8 * h) * 8 + (2 * in_eight + half) * kGroups;
                    if constexpr (kGroups == 4) {
                        *(float4 *)scale[h] = *(const float4 *)(scales + at);
                        zeros[h] = *(const uint32_t *)(zero_points + at);
                    } else if constexpr (kGroups == 2) {
                        *(float2 *)scale[h] = *(const float2 *)(scales + at);
                        zeros[h] = *(const uint16_t *)(zero_points + at);
                    } else {
                        scale[h][0] = scales[at];
                        zeros[h] = zero_points[at];
                    }
                }
                float part[NT][2][4];
                uint32_t zero[4];
#pragma unroll
                for (int blk = 0; blk < kHalf / 32; ++blk) {  // 32 columns: a piece of each line
                    constexpr int kBlocks = GROUP / 32;
                    const int g = blk / kBlocks, piece = 4 * half + blk;
                    uint32_t w[4];  // rows row + 8 h
                    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                 : "r"(lines + (my_swap ^ (piece << 4))));
                    uint32_t v[4][4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        if (blk % kBlocks == 0) zero[h] = Nibble<HALF>::minus(zeros[h], g);
                        Nibble<HALF>::pairs(w[h], zero[h], v[h]);
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const uint4 b = *(const uint4 *)(xc + x_at[j] + piece * 64);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t(&lo)[4] = v[2 * i], (&hi)[4] = v[2 * i + 1];
                            if (blk % kBlocks == 0)
                                mma<HALF, true>(part[j][i], lo[0], hi[0], lo[1], hi[1], b.x, b.y);
                            else
                                mma<HALF, false>(part[j][i], lo[0], hi[0], lo[1], hi[1], b.x, b.y);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t(&lo)[4] = v[2 * i], (&hi)[4] = v[2 * i + 1];
                            mma<HALF, false>(part[j][i], lo[2], hi[2], lo[3], hi[3], b.z, b.w);
                        }
                    }
                    if (blk % kBlocks == kBlocks - 1) {
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    acc[j][i][e] = fmaf(scale[2 * i + (e >> 1)][g], part[j][i][e], acc[j][i][e]);
                    }
                }
            }
            __syncwarp();  // the unit is read
            copy_next();
            if (kTables == 1 && turn && n > 1) {
                next.leave(a, my_scales, my_zeros);
                load_next();
                __syncwarp();
            }
            if (whole || n == 1) {  // this tile's part ends here
                if (!HALF && a.dtype == CK_F32) {
                    // the three parts of x lie in lanes quad 0, 1 and 2: smallest first
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float p1 = __shfl_down_sync(~0u, acc[j][i][e], 1),
                                            p2 = __shfl_down_sync(~0u, acc[j][i][e], 2);
                                acc[j][i][e] = (p2 + p1) + acc[j][i][e];
                            }
                }
                const bool done = whole && from_start;  // all of the slab's K: no other warp has a part
                const int last = from_start ? 1 : 0;    // a part that runs on from another warp's is a first one
                float *mine = part_at(warp, last);
                if (!done && lane == 0) part_tile[2 * warp + last] = t;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = 16 * i + row + 8 * (e >> 1);
                            const int m = !HALF && a.dtype == CK_F32 ? (quad ? p.rows : 2 * j + (e & 1))
                                                                     : 8 * j + 2 * quad + (e & 1);
                            const float sum = acc[j][i][e] * (ok ? Nibble<HALF>::kBack : __int_as_float(0x7fc00000));
                            acc[j][i][e] = 0.f;
                            if (m >= p.rows) continue;
                            const int64_t v = (int64_t)t * kTileRows + r;
                            if (!done)
                                mine[m * kTileRows + r] = sum;
                            else if (p.slabs > 1)
                                a.partial[(p.slot(s, t, blockIdx.x) * p.rows + m) * kTileRows + r] = sum;
                            else if (v < a.V)
                                store_y(a, m, v, sum);
                        }
                from_start = true;
            }
            c = whole ? 0 : c + 1;
            t += whole;
        }
        __syncthreads();
        // Where a wait gave up a late copy may have come over a part in its ring: then what is
        // added up here is NaN whatever the parts hold.
        const bool lost = *(volatile int *)&dead != 0;
        // parts of one tile follow one another: the warp that holds the first adds them up
        const int theirs = lane < 2 * WARPS ? part_tile[lane] : -1;
        for (int k = 0; k < 2; ++k) {
            const int at = 2 * warp + k, tile = __shfl_sync(~0u, theirs, at);
            const uint32_t same = __ballot_sync(~0u, theirs == tile);
            if (tile < 0 || __ffs(same) - 1 != at) continue;
            const int64_t tu = (int64_t)tile * sc;
            const bool alone = p.slabs == 1 && tu >= u0 && tu + sc <= u1;
            for (int m = 0; m < p.rows; ++m) {
                float sum = lost ? __int_as_float(0x7fc00000) : 0.f;
                for (uint32_t rest = same; rest; rest &= rest - 1) {
                    const int e = __ffs(rest) - 1;
                    sum += part_at(e >> 1, e & 1)[m * kTileRows + lane];
                }
                const int64_t v = (int64_t)tile * kTileRows + lane;
                if (!alone)
                    a.partial[(p.slot(s, tile, blockIdx.x) * p.rows + m) * kTileRows + lane] = sum;
                else if (v < a.V)
                    store_y(a, m, v, sum);
            }
        }
    }
    if (!ok) {  // a wait gave up: no copy is left on its way into this CTA's memory
        volatile int none = 0;
        const Waiter last_wait{&none, p.timeout};
        for (; under_way > 0; --under_way) {
            last_wait(my_bars + 8 * get, get_round & 1);
            if (++get == kStages) get = 0, ++get_round;
        }
    }
}

// Sums that cross CTAs or slabs, in the order of K: a warp for a tile and a row of
// x, a lane for a row of V.  Its lanes first find the CTAs of a slab each.  Every
// thread waits for the product before it ends: what follows in the stream waits for
// this kernel alone.
__global__ void __launch_bounds__(128) k_join(MatvecArgs a, MatvecPlan p) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    if (item >= p.tiles * p.rows) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int64_t m = quotient(item, p.tiles), tile = item - m * p.tiles, v = tile * kTileRows + lane;
    float sum = 0.f;
    bool crossed = p.slabs > 1;
    for (int64_t s0 = 0; s0 < p.slabs; s0 += 32) {
        int64_t at = 0;
        int parts = 1;
        const int64_t s = s0 + lane;
        if (s < p.slabs) {
            int64_t b0 = 0;
            if (p.shared_slabs()) {
                const int64_t sc = p.chunk.first(s + 1) - p.chunk.first(s), c0 = p.cta.first(s);
                const Deal unit = Deal::of(sc * p.tiles, p.cta.first(s + 1) - c0);
                const int64_t i0 = unit.owner(tile * sc), i1 = unit.owner(tile * sc + sc - 1);
                b0 = c0 + i0;
                parts = (int)(i1 - i0) + 1;
            }
            at = (p.slot(s, tile, b0) * p.rows + m) * kTileRows;
        }
        crossed |= __any_sync(~0u, parts > 1);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (!crossed) return;
        const int n = p.slabs - s0 < 32 ? (int)(p.slabs - s0) : 32;
        for (int i = 0; i < n; i += 4) {
            // the first two parts of four slabs at once: waits for memory add up
            float got[4][2];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t from = __shfl_sync(~0u, at, (i + k) & 31);
                const int np = __shfl_sync(~0u, parts, (i + k) & 31);
                got[k][0] = i + k < n ? a.partial[from + lane] : 0.f;
                got[k][1] = i + k < n && np > 1 ? a.partial[from + p.rows * kTileRows + lane] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                sum += got[k][0];
                sum += got[k][1];
                const int64_t from = __shfl_sync(~0u, at, (i + k) & 31);
                const int np = __shfl_sync(~0u, parts, (i + k) & 31);
                if (i + k < n)
                    for (int q = 2; q < np; ++q) sum += a.partial[from + (int64_t)q * p.rows * kTileRows + lane];
            }
        }
    }
    if (v < a.V) store_y(a, m, v, sum);
}

// Rows of x in one launch: what two tensor-core tiles of eight columns hold.  One row more
// goes to k_wide, at any size: 5 x 5,000 fp32 by 256, 2,000 and 32,000 rows take 8.8, 10.2
// and 34 us there and 19, 21 and 59 in two passes of this kernel, 5 x 200,000 by 256 30
// and 64; 17 rows of bf16 9.2, 10.5, 34 and 31, and 23, 25, 69 and 100.
int rows_at_once(int64_t dtype) { return dtype == CK_F32 ? 4 : 16; }

// Rows of the next pass of `left`: k_wide's most, or what is left of them.
int64_t rows_of_pass(int64_t dtype, int64_t left) {
    return left < wide_rows(dtype) ? left : wide_rows(dtype);
}

MatvecPlan matvec_plan(int64_t dtype, int64_t rows, int64_t K, int64_t V, int64_t group, int sms) {
    MatvecPlan p{};
    p.rows = (int)rows;
    p.tiles = (V + kTileRows - 1) / kTileRows;
    p.chunks = (K + kChunk - 1) / kChunk;
    // the columns in use lie below x_cols; the two spare ones of a tile take no memory
    p.x_cols = dtype == CK_F32 ? (int)(8 * ((rows - 1) / 2) + 6) : (int)rows;
    const int64_t units = p.tiles * p.chunks, by_tile = p.tiles < sms ? p.tiles : sms;
    p.warps = p.x_cols <= 8 && units >= (int64_t)kLongRun * kFewWarps * sms ? kManyWarps : kFewWarps;
    const int scale_tables = tables(p.x_cols > 8 ? 2 : 1, (int)group, p.warps);
    const size_t fixed =
        (size_t)p.warps * (ring_units(p.warps) * kUnitBytes + kTileRows * (4 * rows + 40 * scale_tables) + 8);
    const int64_t most = ((int64_t)(kSmemMost - fixed) / p.x_cols - 64) / (2 * kChunk);
    p.slabs = (p.chunks + most - 1) / most;
    // Whole tiles to each CTA, and no second kernel, or equal runs with one: a
    // unit takes an SM about 0.1 us, the second kernel about 2 us.
    const double unit = 0.1;
    const double whole = (double)((p.tiles + by_tile - 1) / by_tile) * p.chunks * unit;
    const double equal = (double)units / sms * unit + 2.0;
    p.aligned = p.slabs == 1 && whole <= equal;
    const int64_t even = units / p.warps;  // a unit for each warp at least
    p.ctas = p.aligned ? by_tile : even < 1 ? 1 : even < sms ? even : sms;
    // as many CTAs to every slab, or slabs to every CTA, by taking more of them
    if (p.slabs > 1) {
        const int64_t want = p.slabs <= p.ctas ? p.ctas / (p.ctas / p.slabs) : (p.slabs + p.ctas - 1) / p.ctas * p.ctas;
        p.slabs = want < p.chunks ? want : p.chunks;
    }
    p.chunk = Deal::of(p.chunks, p.slabs);
    p.cta = Deal::of(p.ctas, p.slabs);
    p.slab = Deal::of(p.slabs, p.ctas);
    p.tile = Deal::of(p.tiles, p.ctas);
    const int64_t slab = (p.chunks + p.slabs - 1) / p.slabs;
    // 64 bytes past a multiple of 128: two columns side by side fill all banks
    p.x_pitch = (int)slab * 2 * kChunk + 64;
    p.timeout = 2 * options().timeout_ns;  // at 2 GHz
    p.extra = options().barrier_extra;
    p.smem = fixed + (size_t)p.x_cols * p.x_pitch;
    return p;
}

size_t partial_bytes(const MatvecPlan &p) {
    return p.aligned ? 0 : (size_t)(p.slabs * p.tiles + p.ctas) * kTileRows * p.rows * sizeof(float);
}

template <bool HALF, int GROUP, int NT, int WARPS>
cudaError_t launch_matvec(const MatvecArgs &a, const MatvecPlan &p, cudaStream_t stream) {
    CUtensorMap weights;
    cudaError_t mapped = weight_map(a, kTileRows, &weights);
    if (mapped != cudaSuccess) return mapped;
    static std::atomic<uint64_t> told{0};
    cudaError_t e = allow_smem((const void *)k_matvec<HALF, GROUP, NT, WARPS>, (int)kSmemMost, told);
    if (e != cudaSuccess) return e;
    for (int again = 0; again < 2; ++again) {
        k_matvec<HALF, GROUP, NT, WARPS><<<(unsigned)p.ctas, WARPS * 32, p.smem, stream>>>(a, p, weights);
        e = cudaGetLastError();
        if (e != cudaErrorInvalidValue || again) break;
        told = 0;  // the device's context was reset since
        e = allow_smem((const void *)k_matvec<HALF, GROUP, NT, WARPS>, (int)kSmemMost, told);
        if (e != cudaSuccess) return e;
    }
    if (e != cudaSuccess || p.aligned) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.tiles * p.rows + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_join, a, p);
}

template <bool HALF, int GROUP>
cudaError_t launch_columns(const MatvecArgs &a, const MatvecPlan &p, cudaStream_t stream) {
    return p.x_cols > 8            ? launch_matvec<HALF, GROUP, 2, kFewWarps>(a, p, stream)
           : p.warps == kFewWarps ? launch_matvec<HALF, GROUP, 1, kFewWarps>(a, p, stream)
                                  : launch_matvec<HALF, GROUP, 1, kManyWarps>(a, p, stream);
}

template <int GROUP> cudaError_t launch_group(const MatvecArgs &a, const MatvecPlan &p, cudaStream_t stream) {
    return a.dtype == CK_F16 ? launch_columns<true, GROUP>(a, p, stream)
                             : launch_columns<false, GROUP>(a, p, stream);
}

struct QuantArgs {
    const void *w;
    int64_t V, K, w_stride;
    int group, symmetric;
    uint8_t *q;
    int64_t q_pitch;
    void *scales;
    int scale_dtype;
    int64_t s_stride;
    uint8_t *zeros;
    int64_t z_stride;
};

// One warp per group: its range, the scale as it will be stored, then the
// nibbles rounded against that stored scale.  Run once for a readout: 32,000 x 5,000
// take 472 us in fp32 and 479 in bf16 by groups of 128 (1.5 TB/s and 0.8 of what is read
// and written), 1,513 in bf16 by groups of 32, which leave half of the lanes idle in the
// second loop; loads of single elements, each weight twice, bound it.
template <typename T> __global__ void __launch_bounds__(256) k_quantize(QuantArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t G = (a.K + a.group - 1) / a.group, items = a.V * G;
    const T *w = (const T *)a.w;
    for (int64_t it = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; it < items;
         it += (int64_t)gridDim.x * (blockDim.x / 32)) {
        const int64_t v = it / G, g = it % G, k0 = g * a.group;
        const int n = a.K - k0 < a.group ? (int)(a.K - k0) : a.group;
        float lo = 0.f, hi = 0.f;
        bool bad = false;
        for (int j = lane; j < n; j += 32) {
            const float t = to_float(w[v * a.w_stride + k0 + j]);
            bad |= !(fabsf(t) <= 3.402823466e38f);
            lo = fminf(lo, t);
            hi = fmaxf(hi, t);
        }
        for (int o = 16; o; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
        }
        bad = __any_sync(~0u, bad);
        float s = a.symmetric ? fmaxf(lo / -8.f, hi / 7.f) : hi / 15.f - lo / 15.f;
        if (bad) s = __int_as_float(0x7fc00000);
        if (a.scale_dtype == CK_BF16) s = __bfloat162float(__float2bfloat16_rn(s));
        if (a.scale_dtype == CK_F16) s = __half2float(__float2half_rn(s));
        const float z = a.symmetric ? 8.f
                                    : s > 0.f ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f;
        if (lane == 0) {
            if (a.scale_dtype == CK_F32) ((float *)a.scales)[v * a.s_stride + g] = s;
            if (a.scale_dtype == CK_BF16)
                ((__nv_bfloat16 *)a.scales)[v * a.s_stride + g] = __float2bfloat16_rn(s);
            if (a.scale_dtype == CK_F16) ((__half *)a.scales)[v * a.s_stride + g] = __float2half_rn(s);
            if (!a.symmetric) a.zeros[v * a.z_stride + g] = (uint8_t)z;
        }
        for (int j = 2 * lane; j < n; j += 64) {
            uint32_t b = 0;
            for (int h = 0; h < 2; ++h) {
                float t = z;
                if (j + h < n && s > 0.f)
                    t = fminf(fmaxf(rintf(to_float(w[v * a.w_stride + k0 + j + h]) / s) + z, 0.f), 15.f);
                b |= (uint32_t)t << (4 * h);
            }
            a.q[v * a.q_pitch + (k0 + j) / 2] = (uint8_t)b;
        }
    }
}

bool known_group(int64_t g) { return g == 32 || g == 64 || g == 128; }

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" ck_status ck_int4_matvec(const void *x, int64_t dtype, int64_t M, int64_t K,
                                    int64_t x_stride, const uint8_t *qweight, int64_t V,
                                    int64_t q_pitch, const void *scales, int64_t scale_dtype,
                                    int64_t s_stride, const uint8_t *zeros, int64_t z_stride,
                                    const float *bias, int64_t group, void *y, int64_t y_stride,
                                    void *workspace, size_t workspace_bytes, void *stream) {
    if (!known_dtype(dtype) || !known_dtype(scale_dtype))
        return fail(CK_ERR_INVALID_ARG, "int4_matvec: unknown dtype");
    if (!known_group(group))
        return fail(CK_ERR_INVALID_ARG, "int4_matvec: group must be 32, 64 or 128, not %lld", (long long)group);
    if (M < 0 || K < 1 || V < 0) return fail(CK_ERR_INVALID_ARG, "int4_matvec: M, V >= 0 and K >= 1");
    if (K >= ((int64_t)1 << 30) || V >= ((int64_t)1 << 30) || M >= ((int64_t)1 << 30))
        return fail(CK_ERR_UNSUPPORTED, "int4_matvec: a size of 2^30 or more");
    if (M == 0 || V == 0) return CK_OK;
    if (!x || !qweight || !scales || !y) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(x, dtype_size(dtype)) || !aligned(y, dtype_size(dtype)) ||
        !aligned(scales, dtype_size(scale_dtype)) || !aligned(bias, 4))
        return fail(CK_ERR_INVALID_ARG, "int4_matvec: a pointer is not aligned to its elements");
    if (q_pitch % 16 != 0 || ((uintptr_t)qweight & 15u) != 0 || q_pitch < (K + 1) / 2)
        return fail(CK_ERR_INVALID_ARG,
                    "int4_matvec: weight rows must start at multiples of 16 bytes and hold (K + 1) / 2 bytes");
    if (s_stride < (K + group - 1) / group || (zeros && z_stride < (K + group - 1) / group) ||
        x_stride < 0 || y_stride < V)
        return fail(CK_ERR_INVALID_ARG, "int4_matvec: a row stride is shorter than its row");
    size_t need = 0;
    const ck_status st = ck_int4_workspace_size(dtype, M, K, V, group, &need);
    if (st != CK_OK) return st;
    if (need > 0 && !workspace) return fail(CK_ERR_INVALID_ARG, "int4_matvec: workspace is NULL");
    if (workspace_bytes < need || ((uintptr_t)workspace & 15u) != 0)
        return fail(CK_ERR_WORKSPACE, "int4_matvec: workspace of %zu bytes (%zu needed, 16-byte aligned)",
                    workspace_bytes, need);
    const int sms = device_sms();
    cudaError_t e = cudaSuccess;
    for (int64_t m = 0; m < M && e == cudaSuccess;) {
        const int64_t rows = rows_of_pass(dtype, M - m);
        const size_t el = dtype_size(dtype);
        MatvecArgs a{(const char *)x + m * x_stride * el, dtype, rows, K, x_stride, qweight, V, q_pitch,
                     scales, (int)scale_dtype, s_stride, zeros, z_stride, bias,
                     (char *)y + m * y_stride * el, y_stride, (float *)workspace};
        cudaStream_t st = (cudaStream_t)stream;
        m += rows;
        if (rows > rows_at_once(dtype)) {
            e = launch_wide(a, group, workspace, sms, st);
            continue;
        }
        const MatvecPlan p = matvec_plan(dtype, rows, K, V, group, sms);
        e = group == 32 ? launch_group<32>(a, p, st) : group == 64 ? launch_group<64>(a, p, st)
                                                                  : launch_group<128>(a, p, st);
    }
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_matvec launch");
}

extern "C" ck_status ck_int4_workspace_size(int64_t dtype, int64_t M, int64_t K, int64_t V,
                                            int64_t group, size_t *bytes) {
    if (!known_dtype(dtype) || M < 0 || K < 1 || V < 0 || K >= ((int64_t)1 << 30) || V >= ((int64_t)1 << 30) ||
        !known_group(group) || !bytes)
        return fail(CK_ERR_INVALID_ARG, "int4_workspace_size: bad dtype, size, group or NULL bytes");
    *bytes = 0;
    if (M == 0 || V == 0) return CK_OK;
    const int sms = device_sms();
    // passes of the most rows, then smaller ones
    for (int64_t m = 0; m < M;) {
        const int64_t rows = rows_of_pass(dtype, M - m);
        const size_t b = rows > rows_at_once(dtype) ? wide_workspace(dtype, rows, K, V, sms)
                                                    : partial_bytes(matvec_plan(dtype, rows, K, V, group, sms));
        if (b > *bytes) *bytes = b;
        m += rows == wide_rows(dtype) ? (M - m) / rows * rows : rows;
    }
    return CK_OK;
}

extern "C" ck_status ck_int4_quantize(const void *w, int64_t dtype, int64_t V, int64_t K,
                                      int64_t w_stride, int64_t group, int64_t symmetric,
                                      uint8_t *qweight, int64_t q_pitch, void *scales,
                                      int64_t scale_dtype, int64_t s_stride, uint8_t *zeros,
                                      int64_t z_stride, void *stream) {
    if (!known_dtype(dtype) || !known_dtype(scale_dtype))
        return fail(CK_ERR_INVALID_ARG, "int4_quantize: unknown dtype");
    if (!known_group(group))
        return fail(CK_ERR_INVALID_ARG, "int4_quantize: group must be 32, 64 or 128, not %lld", (long long)group);
    if (V < 0 || K < 1) return fail(CK_ERR_INVALID_ARG, "int4_quantize: V >= 0 and K >= 1");
    if (K >= ((int64_t)1 << 30) || V >= ((int64_t)1 << 30))
        return fail(CK_ERR_UNSUPPORTED, "int4_quantize: a size of 2^30 or more");
    if (V == 0) return CK_OK;
    if (!w || !qweight || !scales || (!symmetric && !zeros))
        return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(w, dtype_size(dtype)) || !aligned(scales, dtype_size(scale_dtype)))
        return fail(CK_ERR_INVALID_ARG, "int4_quantize: a pointer is not aligned to its elements");
    const int64_t G = (K + group - 1) / group;
    if (q_pitch < (K + 1) / 2 || s_stride < G || (!symmetric && z_stride < G) || w_stride < 0)
        return fail(CK_ERR_INVALID_ARG, "int4_quantize: a row stride is shorter than its row");
    QuantArgs a{w, V, K, w_stride, (int)group, symmetric != 0, qweight, q_pitch, scales,
                (int)scale_dtype, s_stride, zeros, z_stride};
    const int64_t want = (V * G + 7) / 8, most = 16 * (int64_t)device_sms();
    const int grid = (int)(want < most ? want : most);
    with_dtype(dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        k_quantize<T><<<grid, 256, 0, (cudaStream_t)stream>>>(a);
    });
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_quantize launch");
}
