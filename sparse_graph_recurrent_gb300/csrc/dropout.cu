// ck_dropout: dropout whose mask comes from a counter-based generator and is
// never stored.  The backward is the same call on the gradient: the element's
// index gives its word again.
#include <cmath>

#include "ck_philox.h"
#include "ck_types.h"

namespace ck {
namespace {

struct DropArgs {
    const void *x;
    void *y;
    int64_t rep, n1, n2, n3;              // the mask's elements [n1][n2][n3], used `rep` times
    int64_t xr, x1, x2, x3;               // element strides of x: repeat, then the mask's axes
    int64_t yr, y1, y2, y3;
    uint32_t threshold;                   // keep an element whose word is >= threshold
    int drop_all;
    float scale;
    uint64_t seed, step;
    const int64_t *step_dev;
};

// A select and not a product: a dropped element is 0 whatever it held.
template <typename T>
__global__ void __launch_bounds__(256) k_dropout(DropArgs a) {
    const PhiloxKey key = philox_key(a.seed, a.step, a.step_dev);
    const T *x = (const T *)a.x;
    T *y = (T *)a.y;
    const int64_t n = a.n1 * a.n2 * a.n3, blocks = (n + 3) / 4;
    for (int64_t q = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; q < blocks;
         q += (int64_t)gridDim.x * blockDim.x) {
        const uint4 r = philox((uint64_t)q, key);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = 4 * q + j;
            if (m >= n) break;
            const int64_t i3 = m % a.n3, t = m / a.n3, i2 = t % a.n2, i1 = t / a.n2;
            const bool keep = !a.drop_all && w[j] >= a.threshold;
            for (int64_t k = 0; k < a.rep; ++k) {
                const float v = to_float(x[k * a.xr + i1 * a.x1 + i2 * a.x2 + i3 * a.x3]);
                y[k * a.yr + i1 * a.y1 + i2 * a.y2 + i3 * a.y3] =
                    from_float<T>(keep ? v * a.scale : 0.f);
            }
        }
    }
}

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" ck_status ck_dropout(const void *x, void *y, int64_t dtype, int64_t n0, int64_t n1,
                                int64_t n2, int64_t x0, int64_t x1, int64_t x2, int64_t y0,
                                int64_t y1, int64_t y2, int64_t locked, double p, uint64_t seed,
                                uint64_t step, const int64_t *step_dev, void *stream) {
    if (!known_dtype(dtype)) return fail(CK_ERR_INVALID_ARG, "dropout: unknown dtype %lld", (long long)dtype);
    if (!(p >= 0.0 && p <= 1.0)) return fail(CK_ERR_INVALID_ARG, "dropout: p must be in [0, 1]");
    if (n0 < 0 || n1 < 0 || n2 < 0) return fail(CK_ERR_INVALID_ARG, "dropout: negative size");
    if (n0 == 0 || n1 == 0 || n2 == 0) return CK_OK;
    if (n0 > INT64_MAX / n1 || n0 * n1 > INT64_MAX / 16 / n2)
        return fail(CK_ERR_UNSUPPORTED, "dropout: more than 2^59 elements");
    if (!x || !y) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    DropArgs a{};
    a.x = x;
    a.y = y;
    a.rep = locked ? n0 : 1;
    a.n1 = locked ? 1 : n0;
    a.n2 = n1;
    a.n3 = n2;
    a.xr = a.x1 = x0;
    a.yr = a.y1 = y0;
    a.x2 = x1, a.x3 = x2, a.y2 = y1, a.y3 = y2;
    const double t = std::nearbyint(p * 4294967296.0);
    a.drop_all = t >= 4294967296.0;
    a.threshold = a.drop_all ? 0u : (uint32_t)t;
    a.scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
    a.seed = seed;
    a.step = step;
    a.step_dev = step_dev;
    const int64_t want = (a.n1 * a.n2 * a.n3 / 4 + 255) / 256, most = 8 * (int64_t)device_sms();
    const int grid = (int)(want < 1 ? 1 : want < most ? want : most);
    with_dtype(dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        k_dropout<T><<<grid, 256, 0, (cudaStream_t)stream>>>(a);
    });
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_dropout launch");
}
