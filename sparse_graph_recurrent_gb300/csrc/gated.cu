// ck_gated_forward, ck_gated_backward: a linear recurrence over T steps with a gate for
// every step, sequence and node.
//
//   leak form    l = sigmoid(f), h_t = (1 - l) h_{t-1} + l x_t
//   decay form   h_t = f h_{t-1} + x_t
//
// A step is the map h -> a h + u, and a run of steps is one too: (A2, U2) after (A1, U1)
// is (A2 A1, A2 U1 + U2).  So the steps are cut: a thread takes kSteps steps of V
// neighbouring nodes into registers and composes them, the warps of a CTA that hold
// consecutive stretches of the same nodes exchange their maps through shared memory, and
// each then runs its own steps once more from the state that it now knows.  x and the gate
// are read once.  Where there are too few nodes to fill the device the steps are cut into
// chunks for several CTAs, by two kernels: the first composes each chunk, the second
// begins with the maps of the chunks before its own (it reads x and the gate again, mostly
// from L2).
//
// The gradient runs the other way: with g_t = d_out_t + r_{t+1}, r_t = a_t g_t is a map of
// r_{t+1}, and
//   leak   dx = g l, df = g (x - h_{t-1}) l (1 - l)      decay   dx = g, df = g h_{t-1}
// The states are built again in 32 bits from those that the forward keeps at every
// kSteps-th step (its outputs may be rounded to 16 bits; this also reads less).
//
// What bounds both is memory.
#include "ck_types.h"

namespace ck {
namespace {

constexpr int kSteps = 16;      // steps of a thread
constexpr int kGatedWarps = 8;  // warps of a CTA, at most

struct GatedArgs {
    const void *x, *gate, *dout;  // [T][B][N], nodes dense
    int64_t T, B, N;
    int64_t xt, xb, gt, gb, dt, db;
    const float *state0, *dstate;  // [B][N], may be null
    const int64_t *lengths;        // [B], may be null
    void *out;                     // [T][B][N] dense
    float *state;                  // [B][N]
    float *kept;                   // [ceil(T / kSteps)][B][N]
    void *dx, *dgate;              // [T][B][N] dense, may be null
    float *dstate0;                // may be null
    float2 *maps;                  // [chunks][B][N]
    int chunk_tiles;               // tiles of a chunk
    int64_t tiles;
    int wt, wc;                    // warps along the steps, along the nodes
};

// V elements that lie together, as they are loaded and stored.
template <typename T, int V> struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_pack(const T *p) {
    Pack<T, V> r;
    if constexpr (sizeof(r) == 8) {
        const uint2 w = __ldg((const uint2 *)p);
        memcpy(&r, &w, 8);
    } else if constexpr (sizeof(r) == 4) {
        const uint32_t w = __ldg((const uint32_t *)p);
        memcpy(&r, &w, 4);
    } else {
        const uint16_t w = __ldg((const uint16_t *)p);
        memcpy(&r, &w, 2);
    }
    return r;
}
template <typename T, int V> __device__ __forceinline__ void store_pack(T *p, const Pack<T, V> &r) {
    if constexpr (sizeof(r) == 8) {
        uint2 w;
        memcpy(&w, &r, 8);
        __stcs((uint2 *)p, w);
    } else if constexpr (sizeof(r) == 4) {
        uint32_t w;
        memcpy(&w, &r, 4);
        __stcs((uint32_t *)p, w);
    } else {
        uint16_t w;
        memcpy(&w, &r, 2);
        __stcs((uint16_t *)p, w);
    }
}

// sigmoid(f) and 1 - sigmoid(f), each to a few units of the last place whatever f: from
// exp(-|f|), which does not overflow, and the reciprocal of a number in [1, 2].
__device__ __forceinline__ void sigmoids(float f, float &l, float &a) {
    const float e = expf(-fabsf(f)), r = __fdividef(1.f, 1.f + e), q = e * r;
    l = f >= 0.f ? r : q;
    a = f >= 0.f ? q : r;
    if (f != f) l = a = f;
}

// A thread's nodes: where they lie and how many steps each has.
template <int V> struct Nodes {
    int64_t c, b, n;
    int len[V], most;  // steps of each, of the longest
    __device__ __forceinline__ bool find(const GatedArgs &a) {
        const int lane = threadIdx.x & 31, wc = (threadIdx.x >> 5) / a.wt;
        c = (((int64_t)blockIdx.x * a.wc + wc) * 32 + lane) * V;
        const int64_t C = a.B * a.N;
        const bool valid = c < C;
        const int64_t at = valid ? c : 0;
        if (C < ((int64_t)1 << 31)) {
            b = (uint32_t)at / (uint32_t)a.N;
        } else {
            b = at / a.N;
        }
        n = at - b * a.N;
        most = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            len[v] = (int)a.T;
            if (a.lengths && valid) {
                const int64_t i = n + v >= a.N ? b + (n + v) / a.N : b, l = __ldg(a.lengths + i);
                len[v] = l < 0 ? 0 : l < a.T ? (int)l : (int)a.T;
            }
            if (!valid) len[v] = 0;
            most = len[v] > most ? len[v] : most;
        }
        return valid;
    }
};

// A product of factors of which none is 0 is not 0 either, or an infinite state would
// become NaN where its steps leave it infinite: the least number above 0 stands for it.
__device__ __forceinline__ float not_lost(float product, bool nonzero) {
    return product == 0.f && nonzero ? copysignf(__int_as_float(1), product) : product;
}

__device__ __forceinline__ float2 compose(float2 later, float2 earlier) {
    return make_float2(not_lost(later.x * earlier.x, later.x != 0.f && earlier.x != 0.f),
                       fmaf(later.x, earlier.y, later.y));
}

// The maps of the warps' stretches, [parity][warp][V][lane].
template <int V> struct Exchange {
    float2 m[2][kGatedWarps][V][32];
};

// The map of chunks [first, last) for this thread's nodes, the warps along the steps
// taking a part each.  REVERSE: a later chunk's map is applied first.
template <int V, bool REVERSE>
__device__ __forceinline__ void chunk_maps(const GatedArgs &a, const Nodes<V> &at, bool valid, int first, int last,
                                           Exchange<V> &ex, float (&carry)[V]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wt = warp % a.wt;
    const int n = last - first, lo = first + n * wt / a.wt, hi = first + n * (wt + 1) / a.wt;
    const int64_t C = a.B * a.N;
    float2 m[V];
#pragma unroll
    for (int v = 0; v < V; ++v) m[v] = make_float2(1.f, 0.f);
    if (valid) {
#pragma unroll 4
        for (int i = 0; i < hi - lo; ++i) {
            const float2 *p = a.maps + (int64_t)(REVERSE ? hi - 1 - i : lo + i) * C + at.c;
#pragma unroll
            for (int v = 0; v < V; ++v) m[v] = compose(__ldcg(p + v), m[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) ex.m[0][warp][v][lane] = m[v];
    __syncthreads();
    const int base = warp - wt;
    for (int j = 0; j < a.wt; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float2 p = ex.m[0][base + (REVERSE ? a.wt - 1 - j : j)][v][lane];
            carry[v] = fmaf(p.x, carry[v], p.y);
        }
    __syncthreads();
}

// MAPS: composes the chunk and writes its map.  Otherwise runs it.
template <typename T, int V, bool LEAK, bool MAPS>
__global__ void __launch_bounds__(32 * kGatedWarps, 2) k_gated_forward(const __grid_constant__ GatedArgs a) {
    __shared__ Exchange<V> ex;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wt = warp % a.wt;
    Nodes<V> at;
    const bool valid = at.find(a);
    const int64_t C = a.B * a.N;
    const T *x = (const T *)a.x + at.b * a.xb + at.n, *gate = (const T *)a.gate + at.b * a.gb + at.n;
    const int64_t k0 = (int64_t)blockIdx.y * a.chunk_tiles;
    const int64_t k1 = k0 + a.chunk_tiles < a.tiles ? k0 + a.chunk_tiles : a.tiles;
    float h[V];      // the state before the tile
    float2 all[V];   // MAPS: the map of the tiles so far
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = !MAPS && a.state0 && valid ? __ldg(a.state0 + at.c + v) : 0.f;
        all[v] = make_float2(1.f, 0.f);
    }
    if (!MAPS && blockIdx.y > 0) chunk_maps<V, false>(a, at, valid, 0, blockIdx.y, ex, h);
    for (int64_t k = k0; k < k1; ++k) {
        const int t0 = (int)(k * a.wt + wt) * kSteps;
        Pack<T, V> px[kSteps], pg[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            if (t0 + s < at.most) {
                px[s] = load_pack<T, V>(x + (t0 + s) * a.xt);
                pg[s] = load_pack<T, V>(gate + (t0 + s) * a.gt);
            }
        float keep[kSteps][V], put[kSteps][V];
        float2 m[V];
        float least[V];  // of the factors' magnitudes
#pragma unroll
        for (int v = 0; v < V; ++v) m[v] = make_float2(least[v] = 1.f, 0.f);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float ka = 1.f, u = 0.f;
                if (t0 + s < at.len[v]) {
                    if constexpr (LEAK) {
                        float l;
                        sigmoids(to_float(pg[s].v[v]), l, ka);
                        u = l * to_float(px[s].v[v]);
                    } else {
                        ka = to_float(pg[s].v[v]);
                        u = to_float(px[s].v[v]);
                    }
                }
                keep[s][v] = ka;
                put[s][v] = u;
                m[v] = make_float2(ka * m[v].x, fmaf(ka, m[v].y, u));
                least[v] = fminf(least[v], fabsf(ka));
            }
#pragma unroll
        for (int v = 0; v < V; ++v) m[v].x = not_lost(m[v].x, least[v] > 0.f);
        float mine[V];
        const int p = (int)(k & 1);
#pragma unroll
        for (int v = 0; v < V; ++v) ex.m[p][warp][v][lane] = m[v];
        __syncthreads();
        const int base = warp - wt;
        for (int j = 0; j < a.wt; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 q = ex.m[p][base + j][v][lane];
                if constexpr (MAPS) {
                    all[v] = compose(q, all[v]);
                } else {
                    if (j == wt) mine[v] = h[v];
                    h[v] = fmaf(q.x, h[v], q.y);
                }
            }
        if constexpr (!MAPS) {
            if (!valid || t0 >= a.T) continue;
            if (a.kept) {
#pragma unroll
                for (int v = 0; v < V; ++v) a.kept[(int64_t)(t0 / kSteps) * C + at.c + v] = mine[v];
            }
            T *out = (T *)a.out + (int64_t)t0 * C + at.c;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                if (t0 + s >= a.T) break;
                Pack<T, V> o;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    mine[v] = fmaf(keep[s][v], mine[v], put[s][v]);
                    o.v[v] = from_float<T>(t0 + s < at.len[v] ? mine[v] : 0.f);
                }
                store_pack<T, V>(out + s * C, o);
            }
        }
    }
    if (!valid || wt != 0) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if constexpr (MAPS) {
            a.maps[(int64_t)blockIdx.y * C + at.c + v] = all[v];
        } else {
            if (blockIdx.y + 1 == gridDim.y) a.state[at.c + v] = h[v];
        }
    }
}

// The same with time reversed, and the gradients.
template <typename T, int V, bool LEAK, bool MAPS>
__global__ void __launch_bounds__(32 * kGatedWarps, 2) k_gated_backward(const __grid_constant__ GatedArgs a) {
    __shared__ Exchange<V> ex;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wt = warp % a.wt;
    Nodes<V> at;
    const bool valid = at.find(a);
    const int64_t C = a.B * a.N;
    const T *x = (const T *)a.x + at.b * a.xb + at.n, *gate = (const T *)a.gate + at.b * a.gb + at.n;
    const T *dout = (const T *)a.dout + at.b * a.db + at.n;
    const int64_t k0 = (int64_t)blockIdx.y * a.chunk_tiles;
    const int64_t k1 = k0 + a.chunk_tiles < a.tiles ? k0 + a.chunk_tiles : a.tiles;
    float r[V];
    float2 all[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        r[v] = !MAPS && a.dstate && valid ? __ldg(a.dstate + at.c + v) : 0.f;
        all[v] = make_float2(1.f, 0.f);
    }
    if (!MAPS && blockIdx.y + 1 < gridDim.y)
        chunk_maps<V, true>(a, at, valid, blockIdx.y + 1, gridDim.y, ex, r);
    for (int64_t k = k1 - 1; k >= k0; --k) {
        const int t0 = (int)(k * a.wt + wt) * kSteps;
        Pack<T, V> px[kSteps], pg[kSteps], pd[kSteps];
        float before[kSteps][V];  // decay: the state before the step; leak: x less that
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            if (t0 + s < at.most) {
                pg[s] = load_pack<T, V>(gate + (t0 + s) * a.gt);
                pd[s] = a.dout ? load_pack<T, V>(dout + (t0 + s) * a.dt) : Pack<T, V>{};
                if (!MAPS) px[s] = load_pack<T, V>(x + (t0 + s) * a.xt);
            }
        if constexpr (!MAPS) {
            float h[V];
            if (t0 < at.most) {
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = __ldg(a.kept + (int64_t)(t0 / kSteps) * C + at.c + v);
            }
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (t0 + s < at.len[v]) {
                        const float xs = to_float(px[s].v[v]), f = to_float(pg[s].v[v]);
                        if constexpr (LEAK) {
                            float l, ka;
                            sigmoids(f, l, ka);
                            before[s][v] = xs - h[v];
                            h[v] = fmaf(ka, h[v], l * xs);
                        } else {
                            before[s][v] = h[v];
                            h[v] = fmaf(f, h[v], xs);
                        }
                    }
        }
        float2 m[V];
        float least[V];
#pragma unroll
        for (int v = 0; v < V; ++v) m[v] = make_float2(least[v] = 1.f, 0.f);
#pragma unroll
        for (int s = kSteps - 1; s >= 0; --s)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (t0 + s < at.len[v]) {
                    float l, ka = to_float(pg[s].v[v]);
                    if constexpr (LEAK) sigmoids(ka, l, ka);
                    m[v] = make_float2(ka * m[v].x, ka * (m[v].y + to_float(pd[s].v[v])));
                    least[v] = fminf(least[v], fabsf(ka));
                }
#pragma unroll
        for (int v = 0; v < V; ++v) m[v].x = not_lost(m[v].x, least[v] > 0.f);
        float mine[V];
        const int p = (int)(k & 1);
#pragma unroll
        for (int v = 0; v < V; ++v) ex.m[p][warp][v][lane] = m[v];
        __syncthreads();
        const int base = warp - wt;
        for (int j = a.wt - 1; j >= 0; --j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 q = ex.m[p][base + j][v][lane];
                if constexpr (MAPS) {
                    all[v] = compose(q, all[v]);
                } else {
                    if (j == wt) mine[v] = r[v];
                    r[v] = fmaf(q.x, r[v], q.y);
                }
            }
        if constexpr (!MAPS) {
            if (!valid || t0 >= a.T) continue;
            T *dx = (T *)a.dx + (int64_t)t0 * C + at.c, *dgate = (T *)a.dgate + (int64_t)t0 * C + at.c;
#pragma unroll
            for (int s = kSteps - 1; s >= 0; --s) {
                if (t0 + s >= a.T) continue;
                Pack<T, V> ox, og;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float vx = 0.f, vg = 0.f;
                    if (t0 + s < at.len[v]) {
                        const float g = mine[v] + to_float(pd[s].v[v]);
                        float l, ka = to_float(pg[s].v[v]);
                        if constexpr (LEAK) {
                            sigmoids(ka, l, ka);
                            vx = g * l;
                            vg = vx * ka * before[s][v];
                        } else {
                            vx = g;
                            vg = g * before[s][v];
                        }
                        mine[v] = ka * g;
                    }
                    ox.v[v] = from_float<T>(vx);
                    og.v[v] = from_float<T>(vg);
                }
                if (a.dx) store_pack<T, V>(dx + s * C, ox);
                if (a.dgate) store_pack<T, V>(dgate + s * C, og);
            }
        }
    }
    if (!valid || wt != 0) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if constexpr (MAPS) {
            a.maps[(int64_t)blockIdx.y * C + at.c + v] = all[v];
        } else {
            if (blockIdx.y == 0 && a.dstate0) a.dstate0[at.c + v] = r[v];
        }
    }
}

// How a call is cut.
struct GatedPlan {
    int wt, wc;
    int64_t blocks, tiles;
    int chunk_tiles, chunks;
};

GatedPlan gated_plan(int64_t T, int64_t C, int V, int sms) {
    GatedPlan p{};
    p.wt = 1;
    while (p.wt < kGatedWarps && (int64_t)p.wt * kSteps < T) p.wt *= 2;
    p.wc = kGatedWarps / p.wt;
    while (p.wc > 1 && C < (int64_t)p.wc * 32 * V * sms) p.wc /= 2;
    p.tiles = (T + (int64_t)p.wt * kSteps - 1) / ((int64_t)p.wt * kSteps);
    p.blocks = (C + (int64_t)p.wc * 32 * V - 1) / ((int64_t)p.wc * 32 * V);
    // chunks: so many that every SM has two CTAs, of at least two tiles
    int64_t chunks = p.blocks >= sms ? 1 : (2 * (int64_t)sms + p.blocks - 1) / p.blocks;
    if (chunks > p.tiles / 2) chunks = p.tiles / 2;
    if (chunks < 1) chunks = 1;
    p.chunk_tiles = (int)((p.tiles + chunks - 1) / chunks);
    p.chunks = (int)((p.tiles + p.chunk_tiles - 1) / p.chunk_tiles);
    return p;
}

// Elements that a thread may take at a time: two where every row of steps and sequences
// begins at a multiple of two of them and no pair crosses into a row that does not follow.
bool in_pairs(const void *p, int64_t st, int64_t sb, int64_t B, int64_t N, int64_t T, size_t size) {
    const bool joined = B == 1 || sb == N;
    return aligned(p, 2 * size) && (T == 1 || st % 2 == 0) && (joined ? B * N % 2 == 0 : N % 2 == 0 && sb % 2 == 0);
}

ck_status check_gated(const ck_gated_call *c, bool backward) {
    if (!c) return fail(CK_ERR_INVALID_ARG, "gated recurrence: no arguments");
    if (!known_dtype(c->dtype)) return fail(CK_ERR_INVALID_ARG, "gated recurrence: unknown dtype %lld", (long long)c->dtype);
    if (c->form != CK_GATED_LEAK && c->form != CK_GATED_DECAY)
        return fail(CK_ERR_INVALID_ARG, "gated recurrence: unknown form %lld", (long long)c->form);
    if (c->T < 0 || c->B < 0 || c->N < 0) return fail(CK_ERR_INVALID_ARG, "gated recurrence: negative size");
    constexpr int64_t kMost = (int64_t)1 << 40;
    if (c->T > ((int64_t)1 << 30) || (c->B && c->N > kMost / c->B) ||
        (c->T && c->B && c->N && c->B * c->N > kMost / c->T))
        return fail(CK_ERR_UNSUPPORTED, "gated recurrence: more than 2^40 elements or 2^30 steps");
    if (c->B == 0 || c->N == 0) return CK_OK;
    const size_t e = dtype_size(c->dtype);
    const bool some = c->T > 0;
    if ((some && (!c->x || !c->gate || (!backward && !c->out))) || (!backward && !c->state) || (backward && some && !c->kept))
        return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    for (const void *p : {c->x, c->gate, (const void *)c->out, c->d_out, (const void *)c->dx, (const void *)c->dgate})
        if (!aligned(p, e)) return fail(CK_ERR_INVALID_ARG, "gated recurrence: a pointer is not aligned to its elements");
    for (const void *p : {(const void *)c->state0, (const void *)c->state, (const void *)c->kept, (const void *)c->d_state,
                          (const void *)c->d_state0})
        if (!aligned(p, 4)) return fail(CK_ERR_INVALID_ARG, "gated recurrence: a pointer is not aligned to its elements");
    if (!aligned(c->lengths, 8) || !aligned(c->workspace, 8))
        return fail(CK_ERR_INVALID_ARG, "gated recurrence: a pointer is not aligned to its elements");
    return CK_OK;
}

template <typename T, int V, bool LEAK>
cudaError_t launch_gated(GatedArgs a, const GatedPlan &p, bool backward, cudaStream_t s) {
    a.wt = p.wt;
    a.wc = p.wc;
    a.tiles = p.tiles;
    a.chunk_tiles = p.chunk_tiles;
    const dim3 grid((unsigned)p.blocks, (unsigned)p.chunks), block(32 * p.wt * p.wc);
    if (!backward) {
        if (p.chunks > 1) k_gated_forward<T, V, LEAK, true><<<grid, block, 0, s>>>(a);
        k_gated_forward<T, V, LEAK, false><<<grid, block, 0, s>>>(a);
    } else {
        if (p.chunks > 1) k_gated_backward<T, V, LEAK, true><<<grid, block, 0, s>>>(a);
        k_gated_backward<T, V, LEAK, false><<<grid, block, 0, s>>>(a);
    }
    return cudaGetLastError();
}

ck_status run_gated(const ck_gated_call *c, bool backward, cudaStream_t s) {
    const ck_status st = check_gated(c, backward);
    if (st != CK_OK) return st;
    const int64_t C = c->B * c->N;
    if (C == 0) return CK_OK;
    if (c->T == 0) {  // no step: the state as it was, and its gradient
        float *to = backward ? c->d_state0 : c->state;
        const float *from = backward ? c->d_state : c->state0;
        if (!to) return CK_OK;
        const cudaError_t e = from ? cudaMemcpyAsync(to, from, (size_t)C * 4, cudaMemcpyDeviceToDevice, s)
                                   : cudaMemsetAsync(to, 0, (size_t)C * 4, s);
        return e == cudaSuccess ? CK_OK : cuda_fail(e, "gated recurrence: the state's copy");
    }
    GatedArgs a{};
    a.x = c->x, a.gate = c->gate, a.dout = backward ? c->d_out : nullptr;
    a.T = c->T, a.B = c->B, a.N = c->N;
    a.xt = c->x_step, a.xb = c->x_row, a.gt = c->gate_step, a.gb = c->gate_row, a.dt = c->d_out_step, a.db = c->d_out_row;
    a.state0 = c->state0, a.dstate = c->d_state, a.lengths = c->lengths;
    a.out = c->out, a.state = c->state, a.kept = c->kept;
    a.dx = c->dx, a.dgate = c->dgate, a.dstate0 = c->d_state0;
    const size_t e = dtype_size(c->dtype);
    const bool pairs = in_pairs(a.x, a.xt, a.xb, c->B, c->N, c->T, e) && in_pairs(a.gate, a.gt, a.gb, c->B, c->N, c->T, e) &&
                       (!a.dout || in_pairs(a.dout, a.dt, a.db, c->B, c->N, c->T, e)) && aligned(a.out, 2 * e) &&
                       aligned(a.dx, 2 * e) && aligned(a.dgate, 2 * e) && C % 2 == 0;
    const GatedPlan p = gated_plan(c->T, C, pairs ? 2 : 1, device_sms());
    if (p.blocks > 0x7fffffff || p.chunks > 65535) return fail(CK_ERR_UNSUPPORTED, "gated recurrence: too many nodes");
    if (p.chunks > 1) {
        const size_t need = (size_t)p.chunks * C * sizeof(float2);
        if (!c->workspace || (size_t)c->workspace_bytes < need)
            return fail(CK_ERR_WORKSPACE, "gated recurrence: a workspace of %zu bytes is needed", need);
        a.maps = (float2 *)c->workspace;
    }
    const cudaError_t err = with_dtype(c->dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        if (c->form == CK_GATED_LEAK)
            return pairs ? launch_gated<T, 2, true>(a, p, backward, s) : launch_gated<T, 1, true>(a, p, backward, s);
        return pairs ? launch_gated<T, 2, false>(a, p, backward, s) : launch_gated<T, 1, false>(a, p, backward, s);
    });
    return err == cudaSuccess ? CK_OK : cuda_fail(err, "k_gated launch");
}

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" ck_status ck_gated_sizes(int64_t T, int64_t B, int64_t N, size_t *kept_bytes, size_t *workspace_bytes) {
    if (T < 0 || B < 0 || N < 0) return fail(CK_ERR_INVALID_ARG, "gated recurrence: negative size");
    if (!kept_bytes || !workspace_bytes) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    *kept_bytes = *workspace_bytes = 0;
    constexpr int64_t kMost = (int64_t)1 << 40;
    if (T > ((int64_t)1 << 30) || (B && N > kMost / B) || (T && B && N && B * N > kMost / T))
        return fail(CK_ERR_UNSUPPORTED, "gated recurrence: more than 2^40 elements or 2^30 steps");
    const int64_t C = B * N;
    if (C == 0 || T == 0) return CK_OK;
    *kept_bytes = (size_t)((T + kSteps - 1) / kSteps) * C * 4;
    // of the widths that the alignment may leave, the one with more chunks
    for (int V = 1; V <= 2; ++V) {
        const GatedPlan p = gated_plan(T, C, V, device_sms());
        const size_t need = p.chunks > 1 ? (size_t)p.chunks * C * sizeof(float2) : 0;
        if (need > *workspace_bytes) *workspace_bytes = need;
    }
    return CK_OK;
}

extern "C" ck_status ck_gated_forward(const ck_gated_call *call, void *stream) {
    return run_gated(call, false, (cudaStream_t)stream);
}

extern "C" ck_status ck_gated_backward(const ck_gated_call *call, void *stream) {
    return run_gated(call, true, (cudaStream_t)stream);
}
