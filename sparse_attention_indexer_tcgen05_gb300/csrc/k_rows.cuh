// k_rows.cuh -- eight neighbouring values of a row: loads off the 16-byte boundaries, and the bf16 planes that the products take.
#pragma once

#include "k_linear.cuh"

namespace csa {
namespace linear {

// x = h + m + l with bf16 parts: 8 bits of the significand each.  NaN stays in h; a finite x that would round to an infinity
// is cut off instead.  An infinity goes to l, which meets the other factor's h alone, and h is 1 of its sign: the product is
// then an infinity of the right sign for every other factor that is not 0, infinite ones too (whose l meets this h).  In h it
// would meet the other's m and l, which may be 0 or of the other sign.
__device__ __forceinline__ void split3(float x, bf16 &h, bf16 &m, bf16 &l)
{
    h = __float2bfloat16_rn(x);
    if (fabsf(x) > 3.38e38f && fabsf(x) < INFINITY) h = __ushort_as_bfloat16((unsigned short)(__float_as_uint(x) >> 16));
    const float r = x - __bfloat162float(h);
    const bool fine = fabsf(r) <= 3.0e38f;  // false for NaN and infinities
    m = __float2bfloat16_rn(fine ? r : 0.f);
    l = __float2bfloat16_rn(fine ? r - __bfloat162float(m) : 0.f);
    if (fabsf(x) == INFINITY) {
        l = h;
        h = __float2bfloat16_rn(copysignf(1.f, x));
    }
}

// x = h + m to 2^-16.  h is cut off and m never 0 unless x is, so that both have x's sign: an infinite factor then gives an
// infinity of that sign, not NaN.
__device__ __forceinline__ void split2(float x, bf16 &h, bf16 &m)
{
    h = __ushort_as_bfloat16((unsigned short)(__float_as_uint(x) >> 16));
    const float top = __bfloat162float(h), r = x - top;
    m = __float2bfloat16_rn(r != 0.f && fabsf(x) < INFINITY ? r : top * 5.9604644775390625e-8f);
}

// What holds a staged operand of values V
template <typename V> struct Planes;
template <> struct Planes<bf16> { static constexpr int N = 1; };
template <> struct Planes<float> { static constexpr int N = 3; };

// 8 neighbouring values from p on, of which `valid` (1 to 8) exist; the others 0.  ALIGNED: p lies on 16 bytes and all
// exist.  Otherwise p lies anywhere: the aligned vectors that hold the existing values are loaded, up to the argument's
// `end`, and shifted when the values are taken.
template <typename T, bool ALIGNED> struct Raw8 {
    static constexpr int V = sizeof(T) == 2 ? 1 : 2;   // vectors of 8 values
    uint32_t w[4 * V + (ALIGNED ? 0 : 4)], sh;
    __device__ __forceinline__ void load(const T *p, int valid, const T *end)
    {
        sh = ALIGNED ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
        const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) - sh);
#pragma unroll
        for (int k = 0; k < V + (ALIGNED ? 0 : 1); k++) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (ALIGNED) v = __ldcs(q + k);
            else if ((int)sh + valid * (int)sizeof(T) > 16 * k) v = load16(q + k, end);
            w[4 * k] = v.x; w[4 * k + 1] = v.y; w[4 * k + 2] = v.z; w[4 * k + 3] = v.w;
        }
    }
    __device__ __forceinline__ void floats(int valid, float (&x)[8]) const
    {
        uint32_t u[4 * V + 4];
#pragma unroll
        for (int k = 0; k < 4 * V + 4; k++) u[k] = k < 4 * V + (ALIGNED ? 0 : 4) ? w[k] : 0u;
        if (!ALIGNED) {
            if (sh & 8) {
#pragma unroll
                for (int k = 0; k < 4 * V + 2; k++) u[k] = u[k + 2];
            }
            if (sh & 4) {
#pragma unroll
                for (int k = 0; k < 4 * V + 1; k++) u[k] = u[k + 1];
            }
            if (sizeof(T) == 2 && (sh & 2)) {
#pragma unroll
                for (int k = 0; k < 4; k++) u[k] = __funnelshift_r(u[k], u[k + 1], 16);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const uint32_t b = sizeof(T) == 4 ? u[k] : k % 2 == 0 ? u[k / 2] << 16 : u[k / 2] & 0xffff0000u;
            x[k] = ALIGNED || k < valid ? __uint_as_float(b) : 0.f;
        }
    }
};
template <typename T, bool ALIGNED> __device__ __forceinline__ void load8(const T *p, int valid, const T *end, float (&x)[8])
{
    Raw8<T, ALIGNED> r;
    r.load(p, valid, end);
    r.floats(valid, x);
}

// 8 neighbouring values to the planes
template <int P> __device__ __forceinline__ void put_planes8(bf16 *out, long long plane, long long at, const float (&x)[8])
{
    __nv_bfloat162 w[P][4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        if constexpr (P == 1) {
            w[0][k] = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        } else if constexpr (P == 2) {
            split2(x[2 * k], w[0][k].x, w[1][k].x);
            split2(x[2 * k + 1], w[0][k].y, w[1][k].y);
        } else {
            split3(x[2 * k], w[0][k].x, w[1][k].x, w[2][k].x);
            split3(x[2 * k + 1], w[0][k].y, w[1][k].y, w[2][k].y);
        }
    }
#pragma unroll
    for (int q = 0; q < P; q++) *reinterpret_cast<uint4 *>(out + q * plane + at) = *reinterpret_cast<const uint4 *>(w[q]);
}

}  // namespace linear
}  // namespace csa
