// ck_gated_forward, ck_gated_backward: a linear recurrence over T steps with a gate for
// every step, sequence and node.
//
//   leak form    l = sigmoid(f), h_t = (1 - l) h_{t-1} + l x_t
//   decay form   h_t = f h_{t-1} + x_t
//
// A thread takes V neighbouring nodes and walks along the steps, kSteps at a time.  Its warp
// has the next steps copied into shared memory meanwhile, one to three such blocks ahead:
// registers could not hold as much as has to be under way (with loads into registers, one
// block ahead, 64 x 32 x 5,000 fp32 took 27 us and its gradient 45; with copies 23 and 41, and
// 20 and 34 with two nodes' numbers in one operation and kernels that start early).
// Where the nodes alone fill the device that is all: x and the gate are read once, nothing
// is exchanged.
//
// Where they do not, the steps are cut into parts, one for each warp.  A step is the map
// h -> a h + u, and so is a run of steps: (A2, U2) after (A1, U1) is (A2 A1, A2 U1 + U2).
// Each warp first composes its part; the warps of a CTA exchange their maps through shared
// memory; each then runs its part from the state that it now knows, reading it again,
// mostly from L2.  With more parts than a CTA has warps the CTAs of a cluster leave their maps
// in memory and begin with those before their own; with more than a cluster's these are two
// kernels (1,024 x 8 x 1,024 bf16, forward: 20.4 us with a cluster, 21.2 with two kernels).  The
// composing goes through a part in the order opposite to the run that follows, so that what
// was read last, and is in L2 still, is read first again (4,000 x 2 x 1,200 fp32, gradient: 42 us,
// 44 in the same order).
//
// The gradient runs the other way: with g_t = d_out_t + r_{t+1}, r_t = a_t g_t is a map of
// r_{t+1}, and
//   leak   dx = g l, df = g (x - h_{t-1}) l (1 - l)      decay   dx = g, df = g h_{t-1}
// The states are built again in 32 bits from those that the forward keeps at every
// kSteps-th step (its outputs may be rounded to 16 bits; this also reads less).
//
// What bounds it: memory for 32 bits (64 x 32 x 5,000, forward and gradients: 6.2 and
// 6.0 TB/s of what each reads and writes), instructions for 16 (96 x 20 x 5,000 fp16: 5.2 and
// 6.1 TB/s; a step of the gradient is some 30 for each node, 9 of them its sigmoid).
#include "ck_types.h"

namespace ck {
namespace {

constexpr int kSteps = 8;       // steps that a thread takes at a time
constexpr int kGatedWarps = 8;  // warps of a CTA, at most
// How rows lie: at multiples of what a lane copies; at multiples of a pack; anywhere.
constexpr int kInPlace = 0, kWholePacks = 1, kAnywhere = 2;
constexpr int kCluster = 8;  // CTAs that a cluster may have on any device
constexpr int kMostSmem = 128 * 1024;

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
    float2 *maps, *inner;          // [chunks][B][N]; [parts][B][N]: of the CTA's parts before
    int parts;                     // chunks * wt
    int each, more;                // blocks of kSteps steps of a part; parts with one more
    int wt, wc;                    // warps along the steps (1 << wt_shift), along the nodes
    int wt_shift, lane_shift;      // lanes that copy a row, as a power of 2
    int exchange;                  // bytes of shared memory before the rings
    int cluster;                   // the chunks are the CTAs of a cluster
    int early;                     // the next kernel's CTAs may come at once, not when these go
    int copy;                      // bytes that a lane copies at a time
    int apart;                     // rows of outputs that packs cannot be stored to
};

__device__ __forceinline__ void gated_pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void gated_pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// V elements that lie together, as they are loaded and stored.
template <typename T, int V> struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

// Stores a pack: at once, or its first `count` one by one where it may lie anywhere.
template <int SHIFT, typename T, int V> __device__ __forceinline__ void store_pack(const GatedArgs &a, T *p, const Pack<T, V> &r, int count) {
    if (SHIFT == kAnywhere && a.apart) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < count) p[v] = r.v[v];
    } else if constexpr (sizeof(r) == 8) {
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

// A copy of N bytes into shared memory that is waited for later.  Two bytes are too few for
// one: they are loaded and stored.
template <int N> __device__ __forceinline__ void copy_async(uint32_t to, const void *from) {
    if constexpr (N == 2) {
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(*(const uint16_t *)from) : "memory");
    } else if constexpr (N == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(N) : "memory");
    }
}
template <typename P> __device__ __forceinline__ P load_shared(uint32_t from) {
    P r;
    if constexpr (sizeof(P) == 8) {
        uint2 w;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "r"(from));
        memcpy(&r, &w, 8);
    } else if constexpr (sizeof(P) == 4) {
        uint32_t w;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(from));
        memcpy(&r, &w, 4);
    } else {
        uint16_t w;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(from));
        memcpy(&r, &w, 2);
    }
    return r;
}
template <int N> __device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A thread's nodes, and how many steps each has.
template <int V> struct Nodes {
    int64_t c, warp_c;         // of [B][N], the first; the warp's first
    int count;                 // of V, those that there are
    int len[V], most, least;   // steps of each, of the longest, of the shortest
    int warp_most;             // of the warp's longest
    __device__ __forceinline__ bool has(int v) const { return v < count; }
    __device__ __forceinline__ explicit Nodes(const GatedArgs &a) {
        const int lane = threadIdx.x & 31, wc = (threadIdx.x >> 5) >> a.wt_shift;
        warp_c = ((int64_t)blockIdx.x * a.wc + wc) * 32 * V;
        c = warp_c + lane * V;
        const int64_t C = a.B * a.N;
        count = c >= C ? 0 : C - c < V ? (int)(C - c) : V;
        most = 0;
        least = (int)a.T;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            len[v] = v < count ? (int)a.T : 0;
            if (a.lengths && v < count) {
                const int64_t l = a.lengths[(uint32_t)(c + v) / (uint32_t)a.N];
                len[v] = l < 0 ? 0 : l < a.T ? (int)l : (int)a.T;
            }
            most = len[v] > most ? len[v] : most;
            if (v < count) least = len[v] < least ? len[v] : least;
        }
        warp_most = __reduce_max_sync(0xffffffffu, most);
    }
};

// Where a warp's blocks wait on their way from memory: for each of STAGES blocks kSteps rows
// of 32 packs of each of NT tensors, and the states kept before it (KEPT).  The lanes copy
// together, `copy` bytes each at a time, whatever a lane's own pack: with 16 bytes the copies
// pass L1 by, which beside this much shared memory is too small to hold what is under way.
//
// SHIFT: rows that do not begin at multiples of 16 bytes.  The 16-byte pieces that hold a row are copied as they
// lie, one more than it fills, and a row is read from where it begins inside the first.  Of
// a piece that the row ends in, what lies behind the row is not read; what lies before its
// begin shares an aligned 16 bytes with it.
template <typename T, int V, int NT, bool KEPT, int STAGES, int SHIFT> struct Ring {
    using P = Pack<T, V>;
    static constexpr int kRow = 32 * (int)sizeof(P), kPitch = kRow + (SHIFT ? 16 : 0);
    static constexpr int kTensor = kSteps * kPitch, kStage = NT * kTensor + (KEPT ? 128 * V : 0);
    static constexpr int kBytes = STAGES * kStage;
    uint32_t base, put, get;  // stages to be filled and to be read next, times kStage
    int lane, row, copy;  // of the copies: this lane's row of those that go at once
    // SHIFT: the low bits of the addresses of step 0 and of a step (the tensors' agree), and
    // of the block that is read
    uint32_t shift0, shift_step, shift;
    int left, last_left;      // bytes that a row has from this lane's first on, and behind its last whole piece
    const T *p[NT];
    bool absent;  // the second tensor: zeros
    int64_t step[NT];
    const float *kept;    // this thread's
    int64_t kept_step;
    int kept_count;
    // The place that this lane copies from: sequence b, node n.
    int64_t b, n;
    __device__ __forceinline__ void begin(uint32_t smem, const GatedArgs &a, int64_t c) {
        lane = threadIdx.x & 31;
        base = smem + (threadIdx.x >> 5) * kBytes;
        put = get = 0;
        copy = a.copy;
        row = lane >> a.lane_shift;
        const int first = (lane - (row << a.lane_shift)) * copy / (int)sizeof(T);
        const int64_t room = (a.B * a.N - c - first) * (int64_t)sizeof(T);
        left = room < -16 ? -16 : room > kRow ? kRow : (int)room;
        const int64_t behind = (a.B * a.N - c) * (int64_t)sizeof(T) - kRow;
        last_left = behind < -16 ? -16 : behind > 0 ? 0 : (int)behind;
        if (SHIFT) {
            b = 0, n = c + first;  // (sequences join)
        } else {
            c = room > 0 ? c + first : 0;
            b = (uint32_t)c / (uint32_t)a.N;
            n = c - b * a.N;
        }
    }
    __device__ __forceinline__ void tensor(int i, const void *from, int64_t to_step, int64_t to_row) {
        p[i] = (const T *)from + b * to_row + n + row * to_step;
        step[i] = to_step;
        if (i == 1) absent = !from;
        if (i == 0) {
            shift_step = (uint32_t)to_step * (uint32_t)sizeof(T);
            shift0 = (uint32_t)(uintptr_t)((const T *)from + n);
        }
    }
    // Zeros, which nothing is copied over, in the place of a tensor that is not there.
    __device__ __forceinline__ void clear(int i) {
        for (int g = 0; g < kBytes; g += kStage)
            for (int j = lane * 4; j < kTensor; j += 128)
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + g + i * kTensor + j), "r"(0) : "memory");
    }
    template <int W> __device__ __forceinline__ void ask_rows(int steps) {
        if constexpr (W >= (int)sizeof(P)) {
            constexpr int R = W / (int)sizeof(P);
            if (left <= 0) return;
            const uint32_t to = base + put + lane * W;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                if (i == 1 && absent) continue;
                const T *q = p[i];
                if (W >= 8 && steps >= kSteps) {
#pragma unroll
                    for (int s = 0; s < kSteps; s += R, q += R * step[i]) copy_async<W>(to + i * kTensor + s * kRow, q);
                } else {
                    const int most = steps < kSteps ? steps : kSteps;
#pragma unroll 1
                    for (int s = 0; s + row < most; s += R, q += R * step[i]) copy_async<W>(to + i * kTensor + s * kRow, q);
                }
            }
        }
    }
    // The n bytes (at most 16) of the piece that holds q.
    __device__ __forceinline__ void piece(uint32_t to, const T *q, int n) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"((uintptr_t)q & ~(uintptr_t)15), "r"(n) : "memory");
    }
    __device__ __forceinline__ void ask_shifted(int k, int steps) {
        constexpr int R = 16 / (int)sizeof(P), kPieces = kRow / 16;
        const uint32_t to = base + put + row * kPitch + (lane % kPieces) * 16, last = base + put + lane * kPitch + kRow;
        const uint32_t block = shift0 + (uint32_t)(k * kSteps) * shift_step;
#pragma unroll
        for (int s = 0; s < kSteps; s += R) {
            const int n = left + (int)((block + (s + row) * shift_step) & 15);
            if (n <= 0 || s + row >= steps) continue;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i != 1 || !absent) piece(to + i * kTensor + s * kPitch, p[i] + s * step[i], n < 16 ? n : 16);
        }
        // the last piece of row `lane`
        const int n = last_left + (int)((block + lane * shift_step) & 15);
        if (lane < kSteps && lane < steps && n > 0) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i != 1 || !absent) piece(last + i * kTensor, p[i] + (lane - row) * step[i] + (kPieces - lane % kPieces) * (16 / (int)sizeof(T)), n);
        }
    }
    // Asks for the first `steps` steps of block k, and leaves a mark to wait for.
    __device__ __forceinline__ void ask(int k, int steps) {
        if (SHIFT)
            ask_shifted(k, steps);
        else if (copy == 16)
            ask_rows<16>(steps);
        else if (copy == 8)
            ask_rows<8>(steps);
        else if (copy == 4)
            ask_rows<4>(steps);
        else
            ask_rows<2>(steps);
        if constexpr (KEPT) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v < kept_count) copy_async<4>(base + put + kept_place(v), kept + v);
        }
    }
    // Takes the places that are copied from on by n blocks.
    __device__ __forceinline__ void go(int n) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
            p[i] += (int64_t)n * kSteps * step[i];
        if (KEPT) kept += n * kept_step;
    }
    __device__ __forceinline__ void asked(int way) {
        asm volatile("cp.async.commit_group;" ::: "memory");
        go(way);
        put = put == (STAGES - 1) * kStage ? 0 : put + kStage;
    }
    __device__ __forceinline__ uint32_t kept_place(int v) const { return NT * kTensor + v * 128 + lane * 4; }
    // Of the block that is read: where step s of tensor i lies, what it is, the state before.
    __device__ __forceinline__ uint32_t place(int i, int s) const {
        const uint32_t at = base + get + lane * (int)sizeof(P) + i * kTensor + s * kPitch;
        return SHIFT ? at + ((shift + s * shift_step) & 15u) : at;
    }
    __device__ __forceinline__ P step_of(int i, int s) const {
        if constexpr (SHIFT != kAnywhere) {
            return load_shared<P>(place(i, s));
        } else {
            P r;
#pragma unroll
            for (int v = 0; v < V; ++v) r.v[v] = load_shared<T>(place(i, s) + v * (int)sizeof(T));
            return r;
        }
    }
    __device__ __forceinline__ float kept_of(int v) const { return load_shared<float>(base + get + kept_place(v)); }

    // `count` blocks from `first` on in the order of `way` (1 or -1): take(k) for each, when
    // it has come.  most: the steps of the warp's longest sequence.
    template <typename F> __device__ __forceinline__ void each(int first, int count, int way, int most, F take) {
        go(first);
        for (int i = 0; i < count + STAGES - 1; ++i) {  // block i is asked for, then the one STAGES - 1 before it taken
            const int next = first + way * i, k = next - way * (STAGES - 1);
            __syncwarp();  // the stage that is asked for has been read by all lanes
            if (i < count) ask(next, most - next * kSteps);
            asked(way);
            if (i < STAGES - 1) continue;
            wait_copies<STAGES - 1>();
            __syncwarp();
            shift = shift0 + (uint32_t)(k * kSteps) * shift_step;
            take(k);
            get = get == (STAGES - 1) * kStage ? 0 : get + kStage;
        }
        wait_copies<0>();
        __syncwarp();
        put = get = 0;
        go(-(first + way * (count + STAGES - 1)));
    }
};

// Products and sums of a thread's numbers: of two at once, each rounded as by itself.
__device__ __forceinline__ unsigned long long both(float a, float b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
template <int V> __device__ __forceinline__ void multiply(float (&r)[V], const float (&a)[V], const float (&b)[V]) {
    if constexpr (V == 2) {
        unsigned long long w;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(w) : "l"(both(a[0], a[1])), "l"(both(b[0], b[1])));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(r[0]), "=f"(r[1]) : "l"(w));
    } else {
        r[0] = a[0] * b[0];
    }
}
template <int V> __device__ __forceinline__ void add(float (&r)[V], const float (&a)[V], const float (&b)[V]) {
    if constexpr (V == 2) {
        unsigned long long w;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(w) : "l"(both(a[0], a[1])), "l"(both(b[0], b[1])));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(r[0]), "=f"(r[1]) : "l"(w));
    } else {
        r[0] = a[0] + b[0];
    }
}
// r = a b + c
template <int V>
__device__ __forceinline__ void multiply_add(float (&r)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
    if constexpr (V == 2) {
        unsigned long long w;
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(w) : "l"(both(a[0], a[1])), "l"(both(b[0], b[1])), "l"(both(c[0], c[1])));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(r[0]), "=f"(r[1]) : "l"(w));
    } else {
        r[0] = fmaf(a[0], b[0], c[0]);
    }
}
template <int V> struct All {
    float v[V];
    __device__ __forceinline__ explicit All(float x) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = x;
    }
};

// l = sigmoid(f) and a = 1 - l, each to a few units of its last place: with e = exp(-f),
// l = 1 / (1 + e) and a = e l.  2^t for t = -f log2(e) is the device's approximation (2^-22.5
// relative); what the rounding of t lost, -f - t ln 2, is put in again by e (1 + that).  f is
// kept between the borders of e's range, NaN as it is; below -30 a is 1 to the last place.
template <int V> __device__ __forceinline__ void sigmoids(const float (&f)[V], float (&l)[V], float (&a)[V]) {
    float c[V], t[V], lost[V], e[V], d[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(c[v]) : "f"(-f[v]), "f"(-100.f));
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(c[v]) : "f"(c[v]), "f"(87.f));
    }
    multiply(t, c, All<V>(1.4426950408889634f).v);
    multiply_add(lost, t, All<V>(-0.6931471805599453f).v, c);
#pragma unroll
    for (int v = 0; v < V; ++v) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[v]) : "f"(t[v]));
    multiply_add(e, e, lost, e);
    add(d, e, All<V>(1.f).v);
#pragma unroll
    for (int v = 0; v < V; ++v) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(l[v]) : "f"(d[v]));
    multiply(a, e, l);
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = c[v] > 30.f ? 1.f : a[v];
}

// A product of factors of which none is 0 is not 0 either, or an infinite state would
// become NaN where its steps leave it infinite: the least number above 0 stands for it.
__device__ __forceinline__ float not_lost(float product, bool nonzero) {
    return product == 0.f && nonzero ? copysignf(__int_as_float(1), product) : product;
}

// One run of steps after another: the map of both.
__device__ __forceinline__ float2 compose(float2 later, float2 earlier) {
    return make_float2(not_lost(later.x * earlier.x, later.x != 0.f && earlier.x != 0.f),
                       fmaf(later.x, earlier.y, later.y));
}

constexpr float kLeast = 1.17549435e-38f, kMost = 3.402823466e38f;  // normal numbers
// What a decay's factor below the normal numbers leaves of a number, `from`, may be off by 2^-126 of
// it: nothing beside a sum, `to`, of 2^-100 of it, nor where it was 2^23 at most.  Above kFaded it
// says too little.
constexpr float kFaded = 6.6174449e-24f;  // 2^-77
__device__ __forceinline__ float faded(float from, float to) { return fmaf(fabsf(from), 7.8886091e-31f, -fabsf(to)); }

// What maps that were composed one after another have gone through.  A decay's product that has
// come below the normal numbers and up again may have been anything in between: the factor of all
// is NaN then, and where too much has faded.  (Looked at once, beside the chain of products: in
// each of them it was 2 to 8% of 65,536 x 256 bf16 and 40,000 x 6 fp32.)
template <int V, bool LEAK> struct Composed {
    float least[V], most_faded[V];  // of the factors' magnitudes; of what came in
    __device__ __forceinline__ Composed() {
#pragma unroll
        for (int v = 0; v < V; ++v) least[v] = 1.f, most_faded[v] = 0.f;
    }
    // by: the factor of the one that is new
    __device__ __forceinline__ float2 operator()(int v, float2 later, float2 earlier, float by) {
        const float2 all = compose(later, earlier);
        if constexpr (!LEAK) {
            least[v] = fminf(least[v], fminf(fabsf(all.x), fabsf(by)));
            most_faded[v] = fmaxf(most_faded[v], faded(earlier.y, all.y));
        }
        return all;
    }
    __device__ __forceinline__ void settle(float2 (&all)[V]) const {
        if constexpr (!LEAK) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if ((least[v] < kLeast) & ((fabsf(all[v].x) >= kLeast) | (most_faded[v] > kFaded))) all[v].x = __int_as_float(0x7fffffff);
        }
    }
};

// The maps of the warps' parts.
template <int V> struct Exchange {
    float2 m[kGatedWarps][V][32];
};

// The blocks [lo, hi) of a part.
__device__ __forceinline__ int first_block(const GatedArgs &a, int part) { return part * a.each + (part < a.more ? part : a.more); }
struct Part {
    int lo, hi, i;
    __device__ __forceinline__ Part(const GatedArgs &a, int wt) {
        i = (blockIdx.y << a.wt_shift) + wt;
        lo = first_block(a, i);
        hi = lo + a.each + (i < a.more);
    }
};

// What maps that a state is carried through say of it.  Decays beyond 1 take a map out of 32 bits
// where the states may stay inside (they are 0, or begin low): what comes out of it is not finite,
// and stays so.  And too much of a state may have faded.
template <int V, bool LEAK> struct Trust {
    float least[V], most_faded[V];
    __device__ __forceinline__ Trust() {
#pragma unroll
        for (int v = 0; v < V; ++v) least[v] = 1.f, most_faded[v] = 0.f;
    }
    __device__ __forceinline__ void through(int v, float2 map, float &carry) {
        const float from = carry;
        carry = fmaf(map.x, carry, map.y);
        least[v] = fminf(least[v], fabsf(map.x));
        most_faded[v] = fmaxf(most_faded[v], faded(from, carry));
    }
    __device__ __forceinline__ bool holds(int v, float carry) const {
        return LEAK || ((fabsf(carry) <= kMost) & ((least[v] >= kLeast) | (most_faded[v] <= kFaded)));
    }
};

// Node c's state after the steps of blocks [lo, hi), or in REVERSE its gradient before them, step
// by step in the decay form.
template <typename T, bool REVERSE>
__device__ __forceinline__ float walk(const GatedArgs &a, int64_t c, int len, int lo, int hi, float carry) {
    const int64_t b = (uint32_t)c / (uint32_t)a.N, n = c - b * a.N;
    const T *gate = (const T *)a.gate + b * a.gb + n;
    const int t0 = lo * kSteps, t1 = hi * kSteps < len ? hi * kSteps : len;
    if constexpr (REVERSE) {
        const T *d = (const T *)a.dout + b * a.db + n;
#pragma unroll 8
        for (int t = t1 - 1; t >= t0; --t)
            carry = to_float(gate[t * a.gt]) * (carry + (a.dout ? to_float(d[t * a.dt]) : 0.f));
    } else {
        const T *x = (const T *)a.x + b * a.xb + n;
#pragma unroll 8
        for (int t = t0; t < t1; ++t) carry = fmaf(to_float(gate[t * a.gt]), carry, to_float(x[t * a.xt]));
    }
    return carry;
}

// What is carried into blocks [lo, hi), where the maps do not hold: by those of the chunks that do,
// and step by step.  (65,536 x 256 fp32, forward: 44 us where they hold; 0.2 ms with a NaN halfway; 9 ms
// with decays of 2 throughout, whose states only stay inside 32 bits where they are 0.)
template <typename T, bool REVERSE>
__device__ __noinline__ float carried_by_steps(const GatedArgs &a, int64_t c, int len, int lo, int hi) {
    const float *from = REVERSE ? a.dstate : a.state0;
    float carry = from ? from[c] : 0.f;
    const int own = blockIdx.y, chunks = gridDim.y;
#pragma unroll 1
    for (int i = 0; i < (REVERSE ? chunks - 1 - own : own) + 1; ++i) {
        const int chunk = REVERSE ? chunks - 1 - i : i;
        int first = first_block(a, chunk << a.wt_shift), last = first_block(a, (chunk + 1) << a.wt_shift);
        if (chunk == own) {
            (REVERSE ? first : last) = REVERSE ? hi : lo;
        } else {
            const float2 m = load_l2(a.maps + chunk * (a.B * a.N) + c);
            const float to = fmaf(m.x, carry, m.y);
            if (fabsf(m.x) <= kMost && fabsf(m.y) <= kMost && (fabsf(m.x) >= kLeast || !(faded(carry, to) > kFaded))) {
                carry = to;
                continue;
            }
        }
        if (carry != carry) break;  // and stays so
        carry = walk<T, REVERSE>(a, c, len, first, last, carry);
    }
    return carry;
}

// carry through the maps of chunks [first, last), the warps along the steps taking some
// each.  REVERSE: a later chunk's map is applied first.
template <int V, bool LEAK, bool REVERSE>
__device__ __forceinline__ void through_chunks(const GatedArgs &a, const Nodes<V> &at, int first, int last,
                                               Exchange<V> &ex, Trust<V, LEAK> &trust, float (&carry)[V]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wt = warp & (a.wt - 1);
    const int n = last - first, lo = first + (n * wt >> a.wt_shift), hi = first + (n * (wt + 1) >> a.wt_shift);
    const int64_t C = a.B * a.N;
    float2 m[V];
#pragma unroll
    for (int v = 0; v < V; ++v) m[v] = make_float2(1.f, 0.f);
    Composed<V, LEAK> composed;
    const auto load = [&](int i, int v) { return load_l2(a.maps + (int64_t)(REVERSE ? hi - 1 - i : lo + i) * C + at.c + v); };
    if constexpr (LEAK) {
#pragma unroll 4
        for (int i = 0; i < hi - lo; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (at.has(v)) m[v] = compose(load(i, v), m[v]);
    } else {
        // four under way at once (what is looked at besides would keep a loop's from being asked for ahead)
        for (int i = 0; i < hi - lo; i += 4) {
            float2 q[4][V];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int v = 0; v < V; ++v) q[u][v] = i + u < hi - lo && at.has(v) ? load(i + u, v) : make_float2(1.f, 0.f);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int v = 0; v < V; ++v) m[v] = composed(v, q[u][v], m[v], q[u][v].x);
        }
        composed.settle(m);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) ex.m[warp][v][lane] = m[v];
    __syncthreads();
    const int base = warp - wt;
    for (int j = 0; j < a.wt; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float2 p = ex.m[base + (REVERSE ? a.wt - 1 - j : j)][v][lane];
            trust.through(v, p, carry[v]);
        }
}

// What is carried into this warp's part.  MAPS: composes the part with part_map(m) and
// leaves the maps; otherwise carry goes through all that comes before.
template <int V, bool LEAK, bool MAPS, bool REVERSE, typename F>
__device__ __forceinline__ void exchange(const GatedArgs &a, const Nodes<V> &at, Exchange<V> &ex, Trust<V, LEAK> &trust,
                                         float (&carry)[V], F part_map) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wt = warp & (a.wt - 1), base = warp - wt;
    const int64_t C = a.B * a.N;
    const int64_t part = (int64_t)blockIdx.y * a.wt + wt;
    if (!MAPS && gridDim.y > 1 && !a.cluster) {
        if (REVERSE ? blockIdx.y + 1 < gridDim.y : blockIdx.y > 0)
            through_chunks<V, LEAK, REVERSE>(a, at, REVERSE ? blockIdx.y + 1 : 0, REVERSE ? gridDim.y : blockIdx.y, ex, trust, carry);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!at.has(v)) continue;
            trust.through(v, load_l2(a.inner + part * C + at.c + v), carry[v]);
        }
        return;
    }
    const bool maps = MAPS || gridDim.y > 1;
    if (!maps && a.wt == 1) return;
    float2 m[V];
#pragma unroll
    for (int v = 0; v < V; ++v) m[v] = make_float2(1.f, 0.f);
    if (maps || (REVERSE ? wt > 0 : wt + 1 < a.wt)) part_map(m);  // (nothing follows the last)
#pragma unroll
    for (int v = 0; v < V; ++v) ex.m[warp][v][lane] = m[v];
    __syncthreads();
    const int before = REVERSE ? a.wt - 1 - wt : wt;
    if (maps) {
        Composed<V, LEAK> composed;
        float2 p[V];  // of the CTA's parts before
#pragma unroll
        for (int v = 0; v < V; ++v) p[v] = make_float2(1.f, 0.f);
        for (int j = 0; j < before; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 q = ex.m[base + (REVERSE ? a.wt - 1 - j : j)][v][lane];
                p[v] = composed(v, q, p[v], q.x);
            }
        composed.settle(p);
#pragma unroll
        for (int v = 0; v < V; ++v) m[v] = composed(v, m[v], p[v], m[v].x);
        composed.settle(m);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!at.has(v)) continue;
            if (MAPS) a.inner[part * C + at.c + v] = p[v];
            if (before == a.wt - 1) a.maps[(int64_t)blockIdx.y * C + at.c + v] = m[v];
        }
        if constexpr (!MAPS) {
            // all of the cluster's maps are there after this
            asm volatile("barrier.cluster.arrive.release;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
            if (REVERSE ? blockIdx.y + 1 < gridDim.y : blockIdx.y > 0)
                through_chunks<V, LEAK, REVERSE>(a, at, REVERSE ? blockIdx.y + 1 : 0, REVERSE ? gridDim.y : blockIdx.y, ex, trust, carry);
#pragma unroll
            for (int v = 0; v < V; ++v) trust.through(v, p[v], carry[v]);
        }
    } else {
        for (int j = 0; j < before; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 q = ex.m[base + (REVERSE ? a.wt - 1 - j : j)][v][lane];
                trust.through(v, q, carry[v]);
            }
    }
}

// What a step keeps of the states and puts in.
template <bool LEAK, int V>
__device__ __forceinline__ void gates(const float (&f)[V], const float (&x)[V], float (&keep)[V], float (&put)[V]) {
    if constexpr (LEAK) {
        float l[V];
        sigmoids(f, l, keep);
        multiply(put, l, x);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) keep[v] = f[v], put[v] = x[v];
    }
}

template <typename T, int V> __device__ __forceinline__ void floats(const Pack<T, V> &p, float (&r)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = to_float(p.v[v]);
}

// Stages of a ring: more of smaller ones, so that 16 warps of an SM have 64 KB or more under
// way, and as many as 16 warps have room for.
template <typename T, int V> constexpr int kForwardStages = sizeof(T) * V >= 8 ? 3 : 4;
template <typename T, int V> constexpr int kBackwardStages = sizeof(T) * V >= 8 ? 2 : 4;
template <typename T, int V, int SHIFT> using ForwardRing = Ring<T, V, 2, false, kForwardStages<T, V>, SHIFT>;
template <typename T, int V, int SHIFT, bool MAPS>
using BackwardRing = Ring<T, V, MAPS ? 2 : 3, !MAPS, kBackwardStages<T, V>, SHIFT>;

// The map of one block of gates and inputs.  WHOLE: all nodes have all its steps.
template <typename T, int V, bool LEAK, bool WHOLE, typename R>
__device__ __forceinline__ void forward_map(const R &in, const Nodes<V> &at, int t0, Composed<V, LEAK> &blocks, float2 (&all)[V]) {
    float by[V], plus[V], least[V];  // the map; the least of the factors' magnitudes
#pragma unroll
    for (int v = 0; v < V; ++v) by[v] = least[v] = 1.f, plus[v] = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        float f[V], x[V], keep[V], put[V];
        floats(in.step_of(0, s), f);
        floats(in.step_of(1, s), x);
        gates<LEAK>(f, x, keep, put);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!WHOLE && t0 + s >= at.len[v]) keep[v] = 1.f, put[v] = 0.f;
            least[v] = fminf(least[v], fabsf(keep[v]));
        }
        multiply(by, keep, by);
        multiply_add(plus, keep, plus, put);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) all[v] = blocks(v, all[v], make_float2(not_lost(by[v], least[v] > 0.f), plus[v]), by[v]);
}

// One block's steps from the state h on.
template <typename T, int V, bool LEAK, int SHIFT, bool WHOLE, typename R>
__device__ __forceinline__ void forward_run(const GatedArgs &a, const R &in, const Nodes<V> &at, int t0, int64_t C, T *&out, float (&h)[V]) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s, out += C) {
        float f[V], x[V], keep[V], put[V], r[V];
        floats(in.step_of(0, s), f);
        floats(in.step_of(1, s), x);
        gates<LEAK>(f, x, keep, put);
        multiply_add(r, keep, h, put);
        Pack<T, V> o;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool live = WHOLE || t0 + s < at.len[v];
            h[v] = live ? r[v] : h[v];
            o.v[v] = from_float<T>(live ? r[v] : 0.f);
        }
        if (WHOLE || t0 + s < a.T) store_pack<SHIFT>(a, out, o, at.count);
    }
}

// A block behind all sequences, `row` being its first (WAY 1) or last (-1) step's; goes on to the
// next block's.
template <typename T, int V, int SHIFT, int WAY>
__device__ __forceinline__ void store_zeros(const GatedArgs &a, T *&row, const Nodes<V> &at, int t0, int64_t C, bool wanted) {
    Pack<T, V> zero;
#pragma unroll
    for (int v = 0; v < V; ++v) zero.v[v] = from_float<T>(0.f);
    for (int s = WAY > 0 ? 0 : kSteps - 1; s >= 0 && s < kSteps; s += WAY, row += WAY * C)
        if (wanted && t0 + s < a.T) store_pack<SHIFT>(a, row, zero, at.count);
}

// MAPS: composes the parts and writes their maps.  Otherwise runs them.
template <typename T, int V, bool LEAK, int SHIFT, bool MAPS>
__global__ void __maxnreg__(96) k_gated_forward(const __grid_constant__ GatedArgs a) {
    extern __shared__ __align__(16) char shared[];
    gated_pdl_wait();
    if (a.early) gated_pdl_launch();
    const uint32_t smem = (uint32_t)__cvta_generic_to_shared(shared) + a.exchange;
    Exchange<V> &ex = *(Exchange<V> *)shared;  // where there is one
    const int wt = (threadIdx.x >> 5) & (a.wt - 1);
    const Nodes<V> at(a);
    const int64_t C = a.B * a.N;
    ForwardRing<T, V, SHIFT> in;
    in.begin(smem, a, at.warp_c);
    in.tensor(0, a.gate, a.gt, a.gb);
    in.tensor(1, a.x, a.xt, a.xb);
    const Part part(a, wt);
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = !MAPS && a.state0 && at.has(v) ? a.state0[at.c + v] : 0.f;
    Trust<V, LEAK> trust;
    exchange<V, LEAK, MAPS, false>(a, at, ex, trust, h, [&](float2 (&m)[V]) {
        Composed<V, LEAK> blocks;
        in.each(part.hi - 1, part.hi - part.lo, -1, at.warp_most, [&](int k) {
            const int t0 = k * kSteps;
            if (t0 + kSteps <= at.least)
                forward_map<T, V, LEAK, true>(in, at, t0, blocks, m);
            else if (t0 < at.most)
                forward_map<T, V, LEAK, false>(in, at, t0, blocks, m);
        });
        blocks.settle(m);
    });
    if constexpr (!MAPS) {
        if constexpr (!LEAK) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (at.has(v) && !trust.holds(v, h[v])) h[v] = carried_by_steps<T, false>(a, at.c + v, at.len[v], part.lo, part.hi);
        }
        T *out = (T *)a.out + (int64_t)part.lo * kSteps * C + at.c;
        float *kept = a.kept + (int64_t)part.lo * C + at.c;
        in.each(part.lo, part.hi - part.lo, 1, at.warp_most, [&](int k) {
            const int t0 = k * kSteps;
            if (!at.count) return;
            if (a.kept) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (at.has(v)) kept[v] = h[v];
                kept += C;
            }
            if (t0 + kSteps <= at.least)
                forward_run<T, V, LEAK, SHIFT, true>(a, in, at, t0, C, out, h);
            else if (t0 < at.most)
                forward_run<T, V, LEAK, SHIFT, false>(a, in, at, t0, C, out, h);
            else
                store_zeros<T, V, SHIFT, 1>(a, out, at, t0, C, true);
        });
        if (part.i + 1 == a.parts) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (at.has(v)) a.state[at.c + v] = h[v];
        }
    }
}

template <typename T, int V, bool LEAK, bool WHOLE, typename R>
__device__ __forceinline__ void backward_map(const R &in, const Nodes<V> &at, int t0, Composed<V, LEAK> &blocks, float2 (&all)[V]) {
    float by[V], plus[V], least[V];
#pragma unroll
    for (int v = 0; v < V; ++v) by[v] = least[v] = 1.f, plus[v] = 0.f;
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s) {
        float keep[V], d[V], l[V], sum[V];
        floats(in.step_of(0, s), keep);
        floats(in.step_of(1, s), d);
        if constexpr (LEAK) sigmoids(keep, l, keep);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!WHOLE && t0 + s >= at.len[v]) keep[v] = 1.f, d[v] = 0.f;
            least[v] = fminf(least[v], fabsf(keep[v]));
        }
        multiply(by, keep, by);
        add(sum, plus, d);
        multiply(plus, keep, sum);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) all[v] = blocks(v, all[v], make_float2(not_lost(by[v], least[v] > 0.f), plus[v]), by[v]);
}

// One block's gradients, r being that of the state after it.
template <typename T, int V, bool LEAK, int SHIFT, bool WHOLE, typename R>
__device__ __forceinline__ void backward_run(const GatedArgs &a, const R &in, const Nodes<V> &at, int t0, int64_t C, T *&dx, T *&dgate, float (&r)[V]) {
    // of each step: what it keeps, and what the gradients are multiplied with
    float keep[kSteps][V], leak[kSteps][V], by[kSteps][V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = in.kept_of(v);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        float f[V], x[V];
        floats(in.step_of(0, s), f);
        floats(in.step_of(2, s), x);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (!WHOLE && t0 + s >= at.len[v]) f[v] = x[v] = 0.f;
        if constexpr (LEAK) {
            float put[V], apart[V];
            sigmoids(f, leak[s], keep[s]);
            multiply_add(apart, h, All<V>(-1.f).v, x);
            multiply(by[s], keep[s], apart);
            multiply(put, leak[s], x);
            multiply_add(h, keep[s], h, put);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) keep[s][v] = f[v], by[s][v] = h[v];
            multiply_add(h, f, h, x);
        }
    }
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s, dx -= C, dgate -= C) {
        float d[V], g[V], vx[V], vg[V], before[V];
        floats(in.step_of(1, s), d);
        add(g, r, d);
        if constexpr (LEAK) {
            multiply(vx, g, leak[s]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) vx[v] = g[v];
        }
        multiply(vg, vx, by[s]);
        multiply(before, keep[s], g);
        Pack<T, V> ox, og;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool live = WHOLE || t0 + s < at.len[v];
            ox.v[v] = from_float<T>(live ? vx[v] : 0.f);
            og.v[v] = from_float<T>(live ? vg[v] : 0.f);
            r[v] = live ? before[v] : r[v];
        }
        if (WHOLE || t0 + s < a.T) {
            if (a.dx) store_pack<SHIFT>(a, dx, ox, at.count);
            if (a.dgate) store_pack<SHIFT>(a, dgate, og, at.count);
        }
    }
}

// The same with time reversed, and the gradients.
template <typename T, int V, bool LEAK, int SHIFT, bool MAPS>
__global__ void __maxnreg__(sizeof(T) == 4 ? 112 : 128) k_gated_backward(const __grid_constant__ GatedArgs a) {
    extern __shared__ __align__(16) char shared[];
    gated_pdl_wait();
    if (a.early) gated_pdl_launch();
    const uint32_t smem = (uint32_t)__cvta_generic_to_shared(shared) + a.exchange;
    Exchange<V> &ex = *(Exchange<V> *)shared;  // where there is one
    const int wt = (threadIdx.x >> 5) & (a.wt - 1);
    const Nodes<V> at(a);
    const int64_t C = a.B * a.N;
    const Part part(a, wt);
    const auto begin = [&](auto &in) {
        in.begin(smem, a, at.warp_c);
        in.tensor(0, a.gate, a.gt, a.gb);
        in.tensor(1, a.dout, a.dt, a.db);
        if (!a.dout) in.clear(1);
    };
    float r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = !MAPS && a.dstate && at.has(v) ? a.dstate[at.c + v] : 0.f;
    Trust<V, LEAK> trust;
    exchange<V, LEAK, MAPS, true>(a, at, ex, trust, r, [&](float2 (&m)[V]) {
        BackwardRing<T, V, SHIFT, true> in;
        begin(in);
        Composed<V, LEAK> blocks;
        in.each(part.lo, part.hi - part.lo, 1, at.warp_most, [&](int k) {
            const int t0 = k * kSteps;
            if (t0 + kSteps <= at.least)
                backward_map<T, V, LEAK, true>(in, at, t0, blocks, m);
            else if (t0 < at.most)
                backward_map<T, V, LEAK, false>(in, at, t0, blocks, m);
        });
        blocks.settle(m);
    });
    if constexpr (!MAPS) {
        if constexpr (!LEAK) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (at.has(v) && !trust.holds(v, r[v])) r[v] = carried_by_steps<T, true>(a, at.c + v, at.len[v], part.lo, part.hi);
        }
        BackwardRing<T, V, SHIFT, false> in;
        begin(in);
        in.tensor(2, a.x, a.xt, a.xb);
        in.kept = a.kept + at.c, in.kept_count = at.count;
        in.kept_step = C;
        T *dx = (T *)a.dx + ((int64_t)part.hi * kSteps - 1) * C + at.c, *dgate = (T *)a.dgate + ((int64_t)part.hi * kSteps - 1) * C + at.c;
        in.each(part.hi - 1, part.hi - part.lo, -1, at.warp_most, [&](int k) {
            const int t0 = k * kSteps;
            if (!at.count) return;
            if (t0 + kSteps <= at.least) {
                backward_run<T, V, LEAK, SHIFT, true>(a, in, at, t0, C, dx, dgate, r);
            } else if (t0 < at.most) {
                backward_run<T, V, LEAK, SHIFT, false>(a, in, at, t0, C, dx, dgate, r);
            } else {
                store_zeros<T, V, SHIFT, -1>(a, dx, at, t0, C, a.dx);
                store_zeros<T, V, SHIFT, -1>(a, dgate, at, t0, C, a.dgate);
            }
        });
        if (part.i == 0 && a.dstate0) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (at.has(v)) a.dstate0[at.c + v] = r[v];
        }
    }
}

// How a call is cut.
struct GatedPlan {
    int wt, wc, chunks;
    int64_t blocks, grid;  // of kSteps steps; CTAs along the nodes
};

GatedPlan gated_plan(int64_t T, int64_t C, int V, int sms) {
    GatedPlan p{};
    p.blocks = (T + kSteps - 1) / kSteps;
    const int64_t warps = (C + 32 * V - 1) / (32 * V);
    // parts: as many as give every SM kFill warps, which is what fits (65,536 x 256 bf16, both
    // directions: 60 us with 16, 66 with 12, 74 with 24 and 77 with 32), of at least three blocks each
    // (64 x 8 x 5,000 fp32, both directions: 21 us, as with four, and 23 with two)
    constexpr int64_t kFill = 16;
    int64_t parts = warps >= 8 * sms ? 1 : (kFill * sms + warps - 1) / warps;
    if (parts > p.blocks / 3) parts = p.blocks / 3;
    // ...or of fewer, where there are so few warps that the steps' own latency is what counts
    // (64 x 39 x 21 fp32, both directions: 10.6 us, 20.2 with three)
    const int64_t few = 8 * (int64_t)sms / warps < p.blocks ? 8 * (int64_t)sms / warps : p.blocks;
    if (p.blocks >= 6 && parts < few) parts = few;
    if (parts < 1) parts = 1;
    p.wt = 1;
    while (p.wt < kGatedWarps && 2 * p.wt <= parts) p.wt *= 2;
    p.chunks = parts >= 2 * kGatedWarps ? (int)(parts / kGatedWarps) : 1;
    // Clusters do not fill the device to the last CTA: with fewer that are all there at once
    // 2,000 x 5 x 600 fp16, forward, takes 17.9 us instead of 23.7.  (Pairs always fit.)
    if (p.chunks > 2 && p.chunks <= kCluster) {
        const int64_t fewer = 14 * (int64_t)sms / warps / kGatedWarps;
        if (fewer < p.chunks) p.chunks = fewer < 2 ? 2 : (int)fewer;
    }
    p.wc = p.wt == 1 ? 1 : kGatedWarps / p.wt;  // (small CTAs fill an SM, and all SMs alike, to the last warp)
    while (p.wc > 1 && warps < (int64_t)p.wc * sms) p.wc /= 2;
    p.grid = (warps + p.wc - 1) / p.wc;
    return p;
}

size_t maps_bytes(const GatedPlan &p, int64_t C) { return (size_t)p.chunks * (1 + p.wt) * C * sizeof(float2); }

// Whether a thread may take V elements at a time: every row of steps and sequences begins
// at a multiple of them, and none crosses into a row that does not follow.
bool in_packs(const void *p, int V, int64_t st, int64_t sb, int64_t B, int64_t N, int64_t T, size_t size) {
    const bool joined = B == 1 || sb == N;
    return aligned(p, V * size) && (T == 1 || st % V == 0) && (joined ? B * N % V == 0 : N % V == 0 && sb % V == 0);
}

ck_status check_gated_sizes(int64_t T, int64_t B, int64_t N) {
    if (T < 0 || B < 0 || N < 0) return fail(CK_ERR_INVALID_ARG, "gated recurrence: negative size");
    // (a step's nodes are counted, and their bytes, in 32 bits)
    constexpr int64_t kNodes = (int64_t)1 << 28, kSteps30 = (int64_t)1 << 30;
    if (T > kSteps30 || (B && N > kNodes / B)) return fail(CK_ERR_UNSUPPORTED, "gated recurrence: more than 2^28 nodes or 2^30 steps");
    return CK_OK;
}

ck_status check_gated(const ck_gated_call *c, bool backward) {
    if (!c) return fail(CK_ERR_INVALID_ARG, "gated recurrence: no arguments");
    if (!known_dtype(c->dtype)) return fail(CK_ERR_INVALID_ARG, "gated recurrence: unknown dtype %lld", (long long)c->dtype);
    if (c->form != CK_GATED_LEAK && c->form != CK_GATED_DECAY)
        return fail(CK_ERR_INVALID_ARG, "gated recurrence: unknown form %lld", (long long)c->form);
    const ck_status st = check_gated_sizes(c->T, c->B, c->N);
    if (st != CK_OK) return st;
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

template <auto KERNEL>
cudaError_t launch_one(dim3 grid, dim3 block, int smem, const GatedArgs &a, cudaStream_t s) {
    static std::atomic<uint64_t> done;
    const cudaError_t e = smem > 32 * 1024 ? allow_smem((const void *)KERNEL, kMostSmem, done) : cudaSuccess;
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    // Its CTAs may take their places while the kernel before ends; each waits for that first.
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = attr[1].val.clusterDim.z = 1;
    attr[1].val.clusterDim.y = grid.y;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, KERNEL, a);
}

template <typename T, int V, bool LEAK, int SHIFT>
cudaError_t launch_gated(GatedArgs a, const GatedPlan &p, bool backward, cudaStream_t s) {
    a.wt = p.wt;
    a.wc = p.wc;
    a.parts = p.wt * p.chunks;
    a.each = (int)(p.blocks / a.parts);
    a.more = (int)(p.blocks % a.parts);
    while (1 << a.wt_shift < p.wt) ++a.wt_shift;
    while (a.copy << a.lane_shift < 32 * V * (int)sizeof(T)) ++a.lane_shift;
    const dim3 grid((unsigned)p.grid, (unsigned)p.chunks), block(32 * p.wt * p.wc);
    a.exchange = p.wt > 1 ? (int)sizeof(Exchange<V>) : 0;
    a.cluster = p.chunks > 1 && p.chunks <= kCluster;
    // The next kernel, if it is one of these, has its CTAs come while there is room for all of them
    // beside this one's, or where they fill the device many times.  Else those that came early would
    // lie unevenly (96 x 20 x 4,999 fp16, both directions: 45 us then, 35 so).
    const int64_t all = p.grid * p.chunks * p.wt * p.wc;
    a.early = all <= 8 * (int64_t)device_sms() || (a.parts == 1 && all >= 16 * (int64_t)device_sms());
    const int warps = p.wt * p.wc, two = p.chunks > 1 && !a.cluster;
    cudaError_t e = cudaSuccess;
    if (!backward) {
        constexpr int kBytes = ForwardRing<T, V, SHIFT>::kBytes;
        if (two) e = launch_one<k_gated_forward<T, V, LEAK, SHIFT, true>>(grid, block, a.exchange + warps * kBytes, a, s);
        if (e == cudaSuccess) e = launch_one<k_gated_forward<T, V, LEAK, SHIFT, false>>(grid, block, a.exchange + warps * kBytes, a, s);
    } else {
        constexpr int kBytes = BackwardRing<T, V, SHIFT, false>::kBytes, kMapBytes = BackwardRing<T, V, SHIFT, true>::kBytes;
        if (two) e = launch_one<k_gated_backward<T, V, LEAK, SHIFT, true>>(grid, block, a.exchange + warps * kMapBytes, a, s);
        if (e == cudaSuccess) e = launch_one<k_gated_backward<T, V, LEAK, SHIFT, false>>(grid, block, a.exchange + warps * kBytes, a, s);
    }
    return e;
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
    // One step has no other to be apart from.  (A block's absent steps are read too, from where
    // the stride says: a stride that is no multiple of a pack would put them off its alignment.)
    if (c->T == 1) a.xt = a.gt = a.dt = 0;
    a.state0 = c->state0, a.dstate = c->d_state, a.lengths = c->lengths;
    a.out = c->out, a.state = c->state, a.kept = c->kept;
    a.dx = c->dx, a.dgate = c->dgate, a.dstate0 = c->d_state0;
    const size_t e = dtype_size(c->dtype);
    // What a lane copies at once (at most 16 bytes), and the elements of a thread (at most 2)
    const auto takes = [&](int n) {
        return in_packs(a.x, n, a.xt, a.xb, c->B, c->N, c->T, e) && in_packs(a.gate, n, a.gt, a.gb, c->B, c->N, c->T, e) &&
               (!a.dout || in_packs(a.dout, n, a.dt, a.db, c->B, c->N, c->T, e));
    };
    a.copy = 16;
    while (a.copy > (int)e && !takes(a.copy / (int)e)) a.copy /= 2;
    const bool pairs = C % 2 == 0 && aligned(a.out, 2 * e) && aligned(a.dx, 2 * e) && aligned(a.dgate, 2 * e);
    // Rows that 16 bytes cannot be copied of, but that hold all sequences one after another and
    // begin alike in all tensors, are taken as they lie: copies of less go by way of what is left
    // of L1 (96 x 20 x 4,999 fp16, gradient: 27 us, 31 with copies of 8 bytes; 300 x 2 x 3,001 bf16,
    // both directions, 25 and 31).  Rows of an odd width that begin unlike are copied by elements: 4
    // bytes at a time in 32 bits (64 x 32 x 4,999, both directions: 83 us, 55 where they begin
    // alike), but loaded and stored in 16, with nothing under way ahead (96 x 20 x 4,999 fp16, both
    // directions: 346 us, 35 where they begin alike).
    const auto like_x = [&](const void *p, int64_t st, int64_t sb) {
        return ((uintptr_t)p - (uintptr_t)a.x) % 16 == 0 && (c->T == 1 || (st - a.xt) * (int64_t)e % 16 == 0) && (c->B == 1 || sb == c->N);
    };
    const bool shifted = (a.copy < 16 || !pairs) && like_x(a.x, a.xt, a.xb) && like_x(a.gate, a.gt, a.gb) &&
                         (!a.dout || like_x(a.dout, a.dt, a.db));
    const bool whole = pairs && a.copy >= 2 * (int)e;  // packs
    if (shifted) a.copy = 16;
    a.apart = !pairs;
    const int V = shifted || whole ? 2 : 1;
    const GatedPlan p = gated_plan(c->T, C, V, device_sms());
    if (p.grid > 0x7fffffff || p.chunks > 65535) return fail(CK_ERR_UNSUPPORTED, "gated recurrence: too many nodes");
    if (p.chunks > 1) {
        const size_t need = maps_bytes(p, C);
        if (!c->workspace || (size_t)c->workspace_bytes < need)
            return fail(CK_ERR_WORKSPACE, "gated recurrence: a workspace of %zu bytes is needed", need);
        a.maps = (float2 *)c->workspace;
        a.inner = a.maps + (int64_t)p.chunks * C;
    }
    const cudaError_t err = with_dtype(c->dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        const auto go = [&](auto width, auto rows) {
            constexpr int W = decltype(width)::value;
            constexpr int S = decltype(rows)::value;
            return c->form == CK_GATED_LEAK ? launch_gated<T, W, true, S>(a, p, backward, s)
                                            : launch_gated<T, W, false, S>(a, p, backward, s);
        };
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        if (shifted && whole) return go(Two(), std::integral_constant<int, kWholePacks>());
        if (shifted) return go(Two(), std::integral_constant<int, kAnywhere>());
        return V == 2 ? go(Two(), std::integral_constant<int, kInPlace>()) : go(One(), std::integral_constant<int, kInPlace>());
    });
    return err == cudaSuccess ? CK_OK : cuda_fail(err, "k_gated launch");
}

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" ck_status ck_gated_sizes(int64_t T, int64_t B, int64_t N, size_t *kept_bytes, size_t *workspace_bytes) {
    const ck_status st = check_gated_sizes(T, B, N);
    if (st != CK_OK) return st;
    if (!kept_bytes || !workspace_bytes) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    *kept_bytes = *workspace_bytes = 0;
    const int64_t C = B * N;
    if (C == 0 || T == 0) return CK_OK;
    *kept_bytes = (size_t)((T + kSteps - 1) / kSteps) * C * 4;
    // of the widths that the alignment may leave, the one with most chunks
    for (int V = 1; V <= 2; ++V) {
        const GatedPlan p = gated_plan(T, C, V, device_sms());
        const size_t need = p.chunks > 1 ? maps_bytes(p, C) : 0;
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
