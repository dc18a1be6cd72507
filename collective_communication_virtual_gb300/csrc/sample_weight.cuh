// sample_weight.cuh -- a value's weight in the sampling, as an integer: 2^44 exp((x - top) / temperature).
//
// The difference and its product with log2(e) / temperature are taken with their rounding errors, the
// exponent is cut into k / 32 and g, |g| <= 1/64, and 2^(k/32) comes from a table, 2^g from its series.  A
// weight is off by at most 4.4 x 2^-31 < 2^-28.8 of itself, and one unit of 2^-44 that is cut off: in 2^-31, 0.7
// for g's rounding, 1 for the series' last step, 1 for its product with g, 0.1 where that becomes an integer,
// 0.5 for the table, 1 where the product with the table is cut.  (A test takes these steps on the host, over all of
// fp32's exponents and temperatures, against exp in 64 bits; it defines the few device functions itself, so
// this file includes none.)
#pragma once

namespace vc {

typedef unsigned long long u64;
constexpr int kFix = 44;             // weights in units of 2^-44

// 2^31 2^(k / 32), rounded
__constant__ uint32_t kPowers[32] = {
    2147483648u, 2194507417u, 2242560872u, 2291666561u, 2341847524u, 2393127307u, 2445529972u, 2499080105u,
    2553802834u, 2609723834u, 2666869345u, 2725266179u, 2784941738u, 2845924021u, 2908241642u, 2971923842u,
    3037000500u, 3103502151u, 3171459999u, 3240905930u, 3311872529u, 3384393094u, 3458501653u, 3534232978u,
    3611622603u, 3690706840u, 3771522796u, 3854108391u, 3938502376u, 4024744348u, 4112874773u, 4202935003u};

struct FixedWeights {                // x == top gives 1, also where both are infinite
    float top, ch, cl;               // ch + cl = log2(e) / temperature
    const uint32_t* powers;          // kPowers
    __device__ __forceinline__ void set(float largest, float temperature) {
        top = largest;
        // log2(e) / temperature and what its rounding lost, kept off zero and infinity
        const float l2e = 1.44269504088896341f, l2eLow = 1.9259629911266175e-8f;
        const float r = __frcp_rn(temperature), c = __fmul_rn(l2e, r);
        ch = fminf(fmaxf(c, 1.17549435e-38f), 3.40282347e38f);
        cl = (__fmaf_rn(-c, temperature, l2e) + l2eLow) * r;
        if (ch != c || !(fabsf(cl) <= 1e-6f * c)) cl = 0.0f;
    }
    // 2^44 e of two values, as integers: the difference and its product with ch + cl with their rounding
    // errors, 2^(k/32) from a table and 2^g, |g| <= 1/64, from its series; without branches, two at a
    // time, as every exact sum goes through here.
    __device__ __forceinline__ void fixed2(float x, float y, u64& vx, u64& vy) const {
        if (isinf(top)) {            // there is nothing beside infinities
            vx = x == top ? 1ull << kFix : 0;
            vy = y == top ? 1ull << kFix : 0;
            return;
        }
        const auto both = [](float c) { return make_float2(c, c); };
        const float2 f = make_float2(x, y), minus = both(-1.0f);
        // f - top = d + low
        const float2 d = add2(f, both(-top)), b = fma2(f, minus, d), t = fma2(b, minus, d);
        const float2 low = add2(fma2(t, minus, f), fma2(b, minus, both(-top)));
        const float2 np = mul2(d, both(-ch));          // -p, p = log2 e to 24 bits
        float2 pl = fma2(d, both(ch), np);
        pl = fma2(d, both(cl), pl);
        pl = fma2(low, both(ch), pl);
        const float magic = 12582912.0f;               // 1.5 2^23: the sum's low bits are the integer
        const float2 at = make_float2(fminf(np.x, kFix + 2.0f), fminf(np.y, kFix + 2.0f));     // beyond this nothing is left
        const float2 r = fma2(at, both(-32.0f), both(magic));
        const float2 k = add2(r, both(-magic));
        const float2 g = fma2(fma2(k, both(0.03125f), np), minus, pl);
        float2 q = fma2(g, both(0.009618129107628477f), both(0.055504108664821576f));
        q = fma2(g, q, both(0.2402265069591007f));
        q = fma2(g, q, both(0.6931471805599453f));
        q = mul2(mul2(g, q), both(8589934592.0f));     // 2^33
        vx = assemble(r.x, q.x);
        vy = assemble(r.y, q.y);
    }
    __device__ __forceinline__ u64 assemble(float r, float q) const {
        const int k = __float_as_int(r) - __float_as_int(12582912.0f);
        const uint32_t t = powers[k & 31], m = t + (uint32_t)__mulhi((int)(t >> 1), __float2int_rn(q));
        return ((u64)m << (kFix - 31)) >> max(0, -(k >> 5));
    }
};

}  // namespace vc
