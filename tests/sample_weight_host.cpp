// sample_weight_host.cpp -- the sampling's integer weights on the host: the device functions that they use,
// each rounded once as there, and one call over arrays.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#define __device__
#define __constant__ static const
#define __forceinline__ inline

struct float2 {
    float x, y;
};

namespace vc {

using std::isinf;
using std::max;

inline float2 make_float2(float x, float y) { return {x, y}; }
inline float2 add2(float2 a, float2 b) { return {a.x + b.x, a.y + b.y}; }
inline float2 mul2(float2 a, float2 b) { return {a.x * b.x, a.y * b.y}; }
inline float2 fma2(float2 a, float2 b, float2 c) { return {std::fmaf(a.x, b.x, c.x), std::fmaf(a.y, b.y, c.y)}; }
inline float __frcp_rn(float x) { return 1.0f / x; }
inline float __fmul_rn(float x, float y) { return x * y; }
inline float __fmaf_rn(float x, float y, float z) { return std::fmaf(x, y, z); }
inline int __float2int_rn(float x) { return std::isnan(x) ? 0 : (int)std::lrint(std::min(std::max((double)x, -0x1p31), 0x1p31 - 1)); }
inline int __mulhi(int a, int b) { return (int)((int64_t)a * b >> 32); }
inline int __float_as_int(float x) {
    int i;
    std::memcpy(&i, &x, 4);
    return i;
}

}  // namespace vc

#include "sample_weight.cuh"

extern "C" void sample_weights(float top, float temperature, const float* x, long long n, unsigned long long* weight) {
    vc::FixedWeights w;
    w.powers = vc::kPowers;
    w.set(top, temperature);
    for (long long i = 0; i < n; i++) {
        vc::u64 other;
        w.fixed2(x[i], top, weight[i], other);
    }
}
