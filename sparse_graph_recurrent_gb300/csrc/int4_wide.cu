// The product with 4-bit weights for more columns of x than k_matvec takes at a
// time: 32-bit states in batches of tens are three columns each.
//
// The mathematics is k_matvec's: exact weights q - z in 16-bit floats, x in bf16 parts,
// 32-bit sums, the scale once a group.  But with n columns a weight costs n multiply-
// adds, which the warps' own matrix instructions do at a quarter of the tensor cores'
// rate (96 columns: 51 us of them for 32,000 x 5,000 weights that memory delivers in
// 13), so here the products are tcgen05.mma's: 128 rows of weights by n columns, 16
// of K at a time, A in tensor memory, where the warps that unpack it put it by row, B
// from shared memory, sums in tensor memory.  A CTA takes 256 rows, two such products
// that share B, and a run of K:
//
//   warps 0-7    a weight row a lane: the sums of a group, once finished, are
//                fetched, scaled and added up in registers
//   warps 8-15   a weight row a lane: 64 columns of K at a time are unpacked into one
//                of two buffers of tensor memory
//   warps 16, 19 wait for A and B and issue the products, of 128 rows each: one warp's
//                waits, operands and commits for all of them took longer than they do
//   warp 17      keeps weights coming: tensor copies of 256 rows by 128 bytes
//   warp 18      keeps x coming: tiles of 64 of K that k_images has laid out as the
//                products read them, so that each is one bulk copy
//
// Tensor memory: sums of two groups for each half (4 x n columns), A twice for each
// (4 x 32).  Registers move from warps 8-19 to warps 0-7, whose sums take 96.  Every
// wait is bounded: one that gives up makes all others give up, and the CTA's outputs
// NaN.
//
// Measured: 32 x 5,000 fp32 states by 32,000 x 5,000 weights, groups of 128, take 38 us
// (2.3 TB/s of weights and scales; 96 columns at 800 TFLOP/s), in groups of 32 with zero
// points 74; 8 states take 34, 32 of bf16 35 and 96 of bf16 40, each further 96 about as
// long again (512 of bf16 235 us, of fp32 583). k_matvec in eight passes takes 288.  What bounds it is the
// way of a step from warp to warp (unpacked, stored, multiplied, its buffer free again):
// without products, weights or x coming in it is a tenth faster.  A chunk takes 1.5 us.
#include "int4.h"

namespace ck {
namespace {

constexpr int kWideRows = 256;
constexpr int kWorkers = 8, kWideThreads = (2 * kWorkers + 4) * 32;  // warps of a kind; three kinds, whole warpgroups
constexpr int kRing = 3;          // units of weights in shared memory
constexpr int kImages = 4;        // tiles of x in shared memory
constexpr int kStep = 64;         // columns of K of a tile of x, and of a buffer of A
constexpr int kMostColumns = 96;  // of tensor memory's 512, 4 x 96 and 4 x 32
constexpr int kPitch = 9;         // of scales in shared memory: a bank a row

struct WidePlan {
    int rows, parts, cols, n;  // rows of x, parts of each, columns, columns padded to 32, 64 or 96
    int64_t blocks;            // of 256 rows of V
    int64_t chunks, steps;     // of 256 and of 64 columns of K
    int64_t splits;            // runs of K
    Deal chunk;                // chunks to runs
    size_t images;             // bytes of x's tiles
    size_t smem;
    long long timeout;         // cycles that a wait may last
    int extra;                 // test hook: arrivals that never come
};

__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The barrier is arrived at when all products issued so far are done.  This and the
// products are issued by one thread of a warp that runs as one: in a branch of a
// single thread their operands would go from its registers to the warp's one by one,
// 100 cycles a product.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// x as tiles of n columns by 64 of K: 128 bytes a column, whose eight 16-byte pieces
// are exchanged by the column (the 128-byte swizzle that the products read), eight
// columns of K to a piece in the order 0 4 1 5 2 6 3 7 in which nibbles come out of a
// word.
template <typename T> __global__ void __launch_bounds__(256) k_images(MatvecArgs a, WidePlan p, char *images) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, pieces = p.steps * 8;
    const int64_t m = quotient(i, pieces), j = i - m * pieces;
    if (m >= p.rows + (p.n - p.cols)) return;
    char *tile = images + (j >> 3) * (p.n * 128);
    auto place = [&](int col) { return (uint4 *)(tile + col * 128 + (((int)(j & 7) ^ (col & 7)) << 4)); };
    if (m >= p.rows) {  // a spare column
        *place(p.cols + (int)(m - p.rows)) = make_uint4(0, 0, 0, 0);
        return;
    }
    T v[8];
    load8<T>(a, m, 8 * j, v);
    constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
    uint16_t part[8][3];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (sizeof(T) == 4)
            split3(v[e], part[e]);
        else
            memcpy(&part[e][0], &v[e], 2);
    }
#pragma unroll
    for (int s = 0; s < kParts; ++s) {
        uint4 w;
        w.x = part[0][s] | (uint32_t)part[4][s] << 16;
        w.y = part[1][s] | (uint32_t)part[5][s] << 16;
        w.z = part[2][s] | (uint32_t)part[6][s] << 16;
        w.w = part[3][s] | (uint32_t)part[7][s] << 16;
        *place(kParts * (int)m + s) = w;
    }
}

template <bool HALF, int GROUP, int N>
__global__ void __launch_bounds__(kWideThreads, 1)
    k_wide(const __grid_constant__ MatvecArgs a, const __grid_constant__ WidePlan p,
           const __grid_constant__ CUtensorMap weights, const char *images, float *partial) {
    extern __shared__ __align__(1024) char smem[];
    __shared__ __align__(8) uint64_t bars[2 * kImages + 2 * kRing + 15];
    __shared__ uint32_t tmem_base;
    __shared__ int dead;
    char *ring = smem + kImages * N * 128;
    float *all_scales = (float *)(ring + kWorkers * kRing * kUnitBytes);
    uint8_t *all_zeros = (uint8_t *)(all_scales + 2 * kWorkers * kTileRows * kPitch);
    constexpr int kUnits = 8 * GROUP / kChunk;  // units of eight groups
    const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, (int)(threadIdx.x >> 5), 0);  // known to be the warp's
    const uint32_t bar0 = smem_at(bars);
    auto b_full = [&](int i) { return bar0 + 8 * i; };
    auto b_empty = [&](int i) { return bar0 + 8 * (kImages + i); };
    auto a_full = [&](int i) { return bar0 + 8 * (2 * kImages + i); };
    auto a_empty = [&](int i) { return bar0 + 8 * (2 * kImages + 2 + i); };
    auto d_full = [&](int half, int i) { return bar0 + 8 * (2 * kImages + 4 + 2 * half + i); };
    auto d_empty = [&](int half, int i) { return bar0 + 8 * (2 * kImages + 8 + 2 * half + i); };
    auto t_full = [&](int i) { return bar0 + 8 * (2 * kImages + 12 + i); };
    const uint32_t idle = bar0 + 8 * (2 * kImages + 14);
    auto w_full = [&](int i) { return bar0 + 8 * (2 * kImages + 15 + i); };
    auto w_empty = [&](int i) { return bar0 + 8 * (2 * kImages + 15 + kRing + i); };
    const Waiter wait{&dead, p.timeout};

    const int64_t split = quotient(blockIdx.x, p.blocks), block = blockIdx.x - split * p.blocks;
    const int c0 = (int)p.chunk.first(split), c1 = (int)p.chunk.first(split + 1);
    const int step0 = c0 * (kChunk / kStep), steps = min(c1 * (kChunk / kStep), (int)p.steps) - step0;
    const bool second = block * kWideRows + 128 < a.V;  // rows in the second half

    if (threadIdx.x == 0) {
        dead = 0;
        for (int i = 0; i < kImages; ++i) {
            barrier_init(b_full(i), 1);
            barrier_init(b_empty(i), 2);
        }
        for (int i = 0; i < 2; ++i) {
            barrier_init(a_full(i), kWorkers + p.extra);
            barrier_init(a_empty(i), 2);
            for (int half = 0; half < 2; ++half) {
                barrier_init(d_full(half, i), 1);
                barrier_init(d_empty(half, i), kWorkers / 2);
            }
            barrier_init(t_full(i), kWorkers);
        }
        barrier_init(idle, 2);
        for (int i = 0; i < kRing; ++i) {
            barrier_init(w_full(i), 1);
            barrier_init(w_empty(i), kWorkers);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2 * kWorkers) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_at(&tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = __shfl_sync(~0u, *(volatile uint32_t *)&tmem_base, 0);
    auto d_at = [&](int half, int buf) { return tmem + (2 * half + buf) * N; };
    auto a_at = [&](int half, int buf) { return tmem + 4 * kMostColumns + (2 * half + buf) * (kStep / 2); };

    if (warp >= 2 * kWorkers) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 24;");
        constexpr uint32_t kTile = N * 128, kWeights = kWorkers * kUnitBytes;
        bool ok = true;
        volatile int none = 0;
        const Waiter last_wait{&none, p.timeout};
        if (warp == 2 * kWorkers || warp == 2 * kWorkers + 3) {
            asm volatile("griddepcontrol.launch_dependents;");
            const int half = warp == 2 * kWorkers ? 0 : 1;
            const bool there = half == 0 || second;
            // D in 32-bit floats; A and B in fp16 (0) or bf16 (1), both along K; N / 8; 128 / 16 rows
            constexpr uint32_t kType = HALF ? 0u : 1u;
            constexpr uint32_t kInstr = 1u << 4 | kType << 7 | kType << 10 | (uint32_t)(N / 8) << 17 | 8u << 24;
            // of a tile in shared memory: 128-byte swizzle, 1,024 bytes from eight columns to the next
            const uint64_t desc0 =
                (uint64_t)2 << 61 | (uint64_t)1 << 46 | (uint64_t)64 << 32 | (uint64_t)1 << 16 | smem_at(smem) >> 4;
            // A turn is four steps: all that depends on a step is then known beforehand, but
            // for the parities of some barriers.
            static_assert(kImages == 4, "tiles of x: one for each step of a turn");
            constexpr int kPerGroup = GROUP / 16, kGroups = 16 / kPerGroup;  // products of a group, groups of a turn
            for (int i0 = 0, turn = 0; i0 < steps && ok; i0 += 4, ++turn) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (i0 + q >= steps || !ok) break;
                    const bool last = i0 + q == steps - 1;
                    ok = __all_sync(~0u, wait(b_full(q), (uint32_t)turn & 1) && wait(a_full(q & 1), (uint32_t)(q >> 1)));
                    if (!ok) break;
                    fence_after();
#pragma unroll
                    for (int k = 0; k < kStep / 16; ++k) {
                        constexpr int kSteps = kStep / 16;
                        const int at = (q * kSteps + k) % kPerGroup, group = (q * kSteps + k) / kPerGroup;
                        const int buf = group & 1;
                        if (at == 0 && (turn > 0 || group >= 2) && ok) {
                            // the sums of two groups ago
                            const int before = turn * (kGroups / 2) + (group >> 1) - 1;
                            ok = __all_sync(~0u, wait(d_empty(half, buf), (uint32_t)before & 1));
                            fence_after();
                        }
                        if (!ok) break;
                        if (there)
                            asm volatile(
                                "{\n.reg .pred e, p;\nelect.sync _|e, 0xffffffff;\nsetp.ne.b32 p, %4, 0;\n"
                                "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_at(half, buf)),
                                "r"(a_at(half, q & 1) + k * 8), "l"(desc0 + q * (kTile >> 4) + 2 * k), "r"(kInstr),
                                "r"((uint32_t)(at != 0))
                                : "memory");
                        if (at == kPerGroup - 1 || (last && k == kSteps - 1)) commit(d_full(half, buf));
                    }
                    if (!ok) break;
                    commit(a_empty(q & 1));
                    commit(b_empty(q));
                }
            }
            commit(idle);  // no product is left under way
            last_wait(idle, 0);
        } else if (warp == 2 * kWorkers + 1) {
            const int units = c1 - c0;
            int i = 0;
            for (; i < units; ++i) {
                const int slot = i % kRing;
                if (i >= kRing) ok = __all_sync(~0u, wait(w_empty(slot), (uint32_t)(i / kRing - 1) & 1));
                if (!ok) break;
                copy_box(weights, (c0 + i) * (kChunk / 2), (int)block * kWideRows, smem_at(ring) + slot * kWeights,
                         w_full(slot), kWeights);
            }
            // the last copies have landed before the CTA ends, also where nobody takes them up any more
            for (int k = i > kRing ? i - kRing : 0; k < i; ++k) last_wait(w_full(k % kRing), (uint32_t)(k / kRing) & 1);
        } else if (warp == 2 * kWorkers + 2) {
            asm volatile("griddepcontrol.wait;" ::: "memory");  // k_images is done
            asm volatile("fence.proxy.async.global;" ::: "memory");
            int i = 0;
            for (; i < steps; ++i) {
                const int slot = i % kImages;
                if (i >= kImages) ok = __all_sync(~0u, wait(b_empty(slot), (uint32_t)(i / kImages - 1) & 1));
                if (!ok) break;
                asm volatile(
                    "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
                    "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%3], %2;\n"
                    "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n}" ::"r"(
                        smem_at(smem) + slot * kTile),
                    "l"(images + (int64_t)(step0 + i) * kTile), "r"(kTile), "r"(b_full(slot))
                    : "memory");
            }
            for (int k = i > kImages ? i - kImages : 0; k < i; ++k)
                last_wait(b_full(k % kImages), (uint32_t)(k / kImages) & 1);
        }
    } else if (warp >= kWorkers) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        const int w = warp - kWorkers, half = w >> 2;
        const int t = (int)block * (kWideRows / kTileRows) + w, groups = (int)((a.K + GROUP - 1) / GROUP);
        const uint32_t quarter = (uint32_t)(w & 3) << 21;  // lanes 32 (w % 4) on of tensor memory
        const uint32_t my_lines = smem_at(ring) + w * kUnitBytes + lane * 128, my_swap = (lane & 7) << 4;
        uint8_t *my_zeros = all_zeros + w * kTileRows * 8;
        ScaleReader<kPitch> next;
        next.load(a, t, c0 / kUnits, groups);
        bool ok = true;
        for (int c = c0; c < c1 && ok; ++c) {
            const int slot = (c - c0) % kRing;
            const int in_eight = c & (kUnits - 1);
            if (c == c0 || in_eight == 0) {
                // Scales lie in two tables in turn.  The one that is written held groups
                // whose sums have been fetched: A's last buffer was free, so the products
                // of three steps ago were done, and they waited for sums of groups before.
                const int table = (c / kUnits) & 1;
                next.leave(a, all_scales + (table * kWorkers + w) * kTileRows * kPitch, my_zeros);
                next.load(a, t, c / kUnits + 1, groups);
                ScaleReader<kPitch>::ahead(a, t, c / kUnits + 5, groups, false);
                __syncwarp();
                if (lane == 0) barrier_arrive(t_full(table));
            }
            ok = __all_sync(~0u, wait(w_full(slot), (uint32_t)((c - c0) / kRing) & 1));
            if (!ok) break;
            const uint32_t line = my_lines + slot * (kWorkers * kUnitBytes);
            uint4 words[2];  // of a step, asked for before the one before is stored
            auto fetch = [&](int q) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(words[e].x), "=r"(words[e].y), "=r"(words[e].z), "=r"(words[e].w)
                                 : "r"(line + (my_swap ^ ((2 * q + e) << 4))));
            };
            fetch(0);
#pragma unroll
            for (int q = 0; q < kChunk / kStep; ++q) {
                const int i = (c - c0) * (kChunk / kStep) + q;
                if (i >= steps) break;
                const int buf = i & 1;
                uint32_t v[32];
#pragma unroll
                for (int e = 0; e < 2; ++e) {  // pieces of 32 columns
                    const int piece = 2 * q + e;
                    const uint32_t zero = Nibble<HALF>::minus(
                        my_zeros[lane * 8 + in_eight * (kChunk / GROUP) + piece * 32 / GROUP], 0);
                    const uint4 n = words[e];
                    Nibble<HALF>::pairs(n.x, zero, *(uint32_t(*)[4])(v + 16 * e));
                    Nibble<HALF>::pairs(n.y, zero, *(uint32_t(*)[4])(v + 16 * e + 4));
                    Nibble<HALF>::pairs(n.z, zero, *(uint32_t(*)[4])(v + 16 * e + 8));
                    Nibble<HALF>::pairs(n.w, zero, *(uint32_t(*)[4])(v + 16 * e + 12));
                }
                if (q + 1 < kChunk / kStep) fetch(q + 1);
                if (q == kChunk / kStep - 1 || i == steps - 1) {  // the unit is read
                    __syncwarp();
                    if (lane == 0) barrier_arrive(w_empty(slot));
                }
                if (i >= 2) {
                    ok = __all_sync(~0u, wait(a_empty(buf), (uint32_t)((i >> 1) - 1) & 1));
                    if (!ok) break;
                    fence_after();
                }
                asm volatile(
                    "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                    "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                    "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a_at(half, buf) + quarter),
                    "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                    "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
                    "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
                    "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
                    : "memory");
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                fence_before();
                __syncwarp();
                if (lane == 0) barrier_arrive(a_full(buf));
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
        const int half = warp >> 2;
        const uint32_t quarter = (uint32_t)(warp & 3) << 21;
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.f;
        bool ok = true;
        // groups of this run, from its first on: runs begin with a chunk, so with a group
        const int first = c0 * (kChunk / GROUP), count = (steps * kStep + GROUP - 1) / GROUP;
        for (int f = 0; f < count && ok; ++f) {
            const int buf = f & 1, g = first + f, table = (g >> 3) & 1;
            if (f == 0 || (g & 7) == 0) ok = wait(t_full(table), (uint32_t)(((g >> 3) - (first >> 3)) >> 1) & 1);
            const float scale = all_scales[((table * kWorkers + warp) * kTileRows + lane) * kPitch + (g & 7)];
            ok = __all_sync(~0u, ok && wait(d_full(half, buf), (uint32_t)(f >> 1) & 1));
            if (!ok) break;
            fence_after();
            if (half == 0 || second) {
#pragma unroll
                for (int b = 0; b < N / 16; ++b) {
                    uint32_t v[16];
                    asm volatile(
                        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
                          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
                          "=r"(v[14]), "=r"(v[15])
                        : "r"(d_at(half, buf) + quarter + 16 * b));
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[16 * b + i] = fmaf(scale, __uint_as_float(v[i]), acc[16 * b + i]);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) barrier_arrive(d_empty(half, buf));
        }
        const int64_t v = block * kWideRows + 32 * warp + lane;
        const float back = ok ? Nibble<HALF>::kBack : __int_as_float(0x7fc00000);
        if (v < a.V) {
            auto put_y = [&](int m, float sum) {
                if (p.splits > 1)
                    partial[(split * p.rows + m) * a.V + v] = sum;
                else
                    store_y(a, m, v, sum);
            };
            if (p.parts == 3) {
#pragma unroll
                for (int m = 0; m < N / 3; ++m)
                    if (m < p.rows) put_y(m, ((acc[3 * m + 2] + acc[3 * m + 1]) + acc[3 * m]) * back);
            } else {
#pragma unroll
                for (int m = 0; m < N; ++m)
                    if (m < p.rows) put_y(m, acc[m] * back);
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 2 * kWorkers) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// Sums over the runs of K, in their order.
__global__ void __launch_bounds__(256) k_wide_join(MatvecArgs a, WidePlan p, const float *partial) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, n = p.rows * a.V;
    if (i >= n) return;
    float sum = 0.f;
    for (int64_t s = 0; s < p.splits; ++s) sum += partial[s * n + i];
    const int64_t m = quotient(i, a.V);
    store_y(a, m, i - m * a.V, sum);
}

WidePlan wide_plan(int64_t dtype, int64_t rows, int64_t K, int64_t V, int sms) {
    WidePlan p{};
    p.rows = (int)rows;
    p.parts = dtype == CK_F32 ? 3 : 1;
    p.cols = p.rows * p.parts;
    p.n = (p.cols + 31) / 32 * 32;
    p.blocks = (V + kWideRows - 1) / kWideRows;
    p.chunks = (K + kChunk - 1) / kChunk;
    p.steps = (K + kStep - 1) / kStep;
    // Runs of K so that the CTAs fill the device evenly: a chunk takes a CTA about 1 us,
    // its start and end 5 us, the sums of several runs 2 us and their memory traffic.
    double best = 1e30;
    for (int64_t s = 1; s <= p.chunks && s <= 64; ++s) {
        const double waves = (double)((p.blocks * s + sms - 1) / sms), run = (double)((p.chunks + s - 1) / s);
        const double cost = waves * (run + 5.0) + (s > 1 ? 2.0 + 2e-6 * (double)(s * rows * V) : 0.0);
        if (cost < best) best = cost, p.splits = s;
    }
    p.chunk = Deal::of(p.chunks, p.splits);
    p.images = (size_t)p.steps * p.n * 128;
    p.smem = (size_t)kImages * p.n * 128 + kWorkers * (kRing * kUnitBytes + kTileRows * (2 * 4 * kPitch + 8));
    return p;
}

template <bool HALF, int GROUP, int N>
cudaError_t run(const MatvecArgs &a, const WidePlan &p, char *images, float *partial, cudaStream_t stream) {
    static std::atomic<uint64_t> told{0};
    cudaError_t e = allow_smem((const void *)k_wide<HALF, GROUP, N>, (int)p.smem, told);  // N says how much
    CUtensorMap weights;
    if (e == cudaSuccess) e = weight_map(a, kWideRows, &weights);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.blocks * p.splits));
    cfg.blockDim = dim3(kWideThreads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_wide<HALF, GROUP, N>, a, p, weights, (const char *)images, partial);
    if (e == cudaErrorInvalidValue) {  // the device's context was reset since
        cudaGetLastError();
        told = 0;
        e = allow_smem((const void *)k_wide<HALF, GROUP, N>, (int)p.smem, told);
        if (e == cudaSuccess)
            e = cudaLaunchKernelEx(&cfg, k_wide<HALF, GROUP, N>, a, p, weights, (const char *)images, partial);
    }
    if (e != cudaSuccess || p.splits == 1) return e;
    cfg.gridDim = dim3((unsigned)((p.rows * a.V + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, k_wide_join, a, p, (const float *)partial);
}

template <bool HALF, int GROUP>
cudaError_t run_columns(const MatvecArgs &a, const WidePlan &p, char *images, float *partial, cudaStream_t stream) {
    return p.n == 32   ? run<HALF, GROUP, 32>(a, p, images, partial, stream)
           : p.n == 64 ? run<HALF, GROUP, 64>(a, p, images, partial, stream)
                       : run<HALF, GROUP, 96>(a, p, images, partial, stream);
}

}  // namespace

int64_t wide_rows(int64_t dtype) { return dtype == CK_F32 ? kMostColumns / 3 : kMostColumns; }

size_t wide_workspace(int64_t dtype, int64_t rows, int64_t K, int64_t V, int sms) {
    const WidePlan p = wide_plan(dtype, rows, K, V, sms);
    return p.images + (p.splits > 1 ? (size_t)p.splits * p.rows * V * sizeof(float) : 0);
}

cudaError_t launch_wide(const MatvecArgs &a, int64_t group, void *workspace, int sms, cudaStream_t stream) {
    WidePlan p = wide_plan(a.dtype, a.M, a.K, a.V, sms);
    p.timeout = 2 * options().timeout_ns;  // at 2 GHz
    p.extra = options().barrier_extra;
    char *images = (char *)workspace;
    float *partial = (float *)(images + p.images);
    const int64_t items = (p.rows + (p.n - p.cols)) * p.steps * 8;
    with_dtype(a.dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        k_images<T><<<(unsigned)((items + 255) / 256), 256, 0, stream>>>(a, p, images);
    });
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (a.dtype == CK_F16)
        return group == 32   ? run_columns<true, 32>(a, p, images, partial, stream)
               : group == 64 ? run_columns<true, 64>(a, p, images, partial, stream)
                             : run_columns<true, 128>(a, p, images, partial, stream);
    return group == 32   ? run_columns<false, 32>(a, p, images, partial, stream)
           : group == 64 ? run_columns<false, 64>(a, p, images, partial, stream)
                         : run_columns<false, 128>(a, p, images, partial, stream);
}

}  // namespace ck
