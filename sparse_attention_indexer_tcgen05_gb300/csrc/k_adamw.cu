// k_adamw.cu -- one AdamW step over many tensors in one launch per group of equal types.
//
//   g = s grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p - lr wd p - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// in fp32.  The states are fp32, or 8 bits: e4m3 codes of m and of sqrt(v) with one fp32 scale per 256 elements,
// the block's largest magnitude / 448.  The root is what is stored because the update divides by it: e4m3 then spans
// a factor of 448 / 2^-9 = 2.3e5 of it (the square would leave a factor of 480 in the root).  A code of v > 0 is at
// least the smallest one, 2^-9: a root that rounded to 0 while m did not would leave eps alone in the divisor.
//
// Codes are rounded to nearest or stochastically.  A step changes the root by a factor of sqrt(b2) at most downwards (2.5%
// at 0.95, 0.05% at 0.999) and half an e4m3 step is 3 to 6% of a value, so nearest codes go back to where they were: a root
// whose gradients shrink tenfold stays up to twelve times too large (b2 = 0.99).  Stochastic codes take the upper neighbour
// with the probability that makes the expected m, and the expected v (the square of the held root), what the formula gives:
// the recurrences are linear in both, so the held moments follow them without a bias, whatever the betas; a root then
// scatters by about a code.  The random number is a hash of seed, tensor, element and step: the same bits every time.
//
// Bound by memory: every state, weight and gradient is read and written once.  A warp owns one block of 256 elements,
// 8 consecutive ones per lane, so each tensor is read and written in 8- or 16-byte accesses, the block's two maxima
// are warp reductions and no shared memory is needed.  The tensors' pointers travel in the kernel's parameters (no
// copy, no device table that must outlive the call, any stream capture keeps them); a CTA finds its tensor by a
// binary search over the first chunk of each.  Measured: 412 million bf16 weights with fp32 masters and 8-bit states
// to nearest 1090 us (6.1 TB/s, 89% of a copy's rate; two thirds of the issue slots are taken), stochastic 1235 us (83% of
// the issue slots); 96 small fp32 tensors 6.2 us.
#include "csa_internal.cuh"
#include "tc_ptx.cuh"

#include <cuda_fp8.h>
#include <math.h>
#include <type_traits>

namespace csa {
namespace adamw {

using ptx::add2;
using ptx::fma2;
using ptx::mul2;

constexpr int THREADS = 128;
constexpr int VEC = 8, PAIRS = VEC / 2;        // elements per lane: one warp covers a block of 256
constexpr int CHUNK = THREADS * VEC;           // elements per CTA
constexpr float E4M3_MAX = 448.f;
constexpr float E4M3_TINY = 0.001953125f;      // 2^-9

enum State { F32, NEAREST, STOCHASTIC };  // how a launch's tensors hold their moments

struct Entry {
    void *param;
    const void *grad;
    float *master;
    void *m, *v;
    float *m_scale, *v_scale;
    long long numel;
    unsigned first;  // the tensor's first chunk
    unsigned id;     // its place in the caller's list
};

struct Hyper {
    float lr, lr_wd, b1, nb1, b2, nb2, eps;  // nb = 1 - b, rounded once from the doubles
    float c1, rs2;                           // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    float wd, log_b1, log_b2;                // for lr and step on the device
    const float *lr_dev, *grad_scale, *found_inf;
    const int64_t *step_dev;
    uint32_t seed;
    long long step;
};

template <int CAP> struct Table {
    Entry e[CAP];
    int n;
};

// 8 values from p (element i, n - i of them valid)
template <typename T> __device__ __forceinline__ void load8(const T *p, long long i, long long n, float2 (&x)[PAIRS])
{
    if (i + VEC <= n) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = __ldcs(reinterpret_cast<const float4 *>(p + i));
            const float4 b = __ldcs(reinterpret_cast<const float4 *>(p + i) + 1);
            x[0] = make_float2(a.x, a.y);
            x[1] = make_float2(a.z, a.w);
            x[2] = make_float2(b.x, b.y);
            x[3] = make_float2(b.z, b.w);
        } else {
            const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p + i));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int k = 0; k < PAIRS; k++) x[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
        }
    } else {
#pragma unroll
        for (int k = 0; k < PAIRS; k++)
            x[k] = make_float2(i + 2 * k < n ? ldf<T>(p, i + 2 * k) : 0.f, i + 2 * k + 1 < n ? ldf<T>(p, i + 2 * k + 1) : 0.f);
    }
}

template <typename T> __device__ __forceinline__ void store8(T *p, long long i, long long n, const float2 (&x)[PAIRS])
{
    if (i + VEC <= n) {
        if constexpr (sizeof(T) == 4) {
            __stcs(reinterpret_cast<float4 *>(p + i), make_float4(x[0].x, x[0].y, x[1].x, x[1].y));
            __stcs(reinterpret_cast<float4 *>(p + i) + 1, make_float4(x[2].x, x[2].y, x[3].x, x[3].y));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[k].x, x[k].y);
                w[k] = *reinterpret_cast<const uint32_t *>(&b);
            }
            __stcs(reinterpret_cast<uint4 *>(p + i), make_uint4(w[0], w[1], w[2], w[3]));
        }
    } else {
#pragma unroll
        for (int k = 0; k < PAIRS; k++) {
            if (i + 2 * k < n) p[i + 2 * k] = from_f<T>(x[k].x);
            if (i + 2 * k + 1 < n) p[i + 2 * k + 1] = from_f<T>(x[k].y);
        }
    }
}

__device__ __forceinline__ uint2 load_codes(const void *p, long long i, long long n)
{
    const unsigned char *c = static_cast<const unsigned char *>(p);
    if (i + VEC <= n) return __ldcs(reinterpret_cast<const uint2 *>(c + i));
    uint2 r = make_uint2(0u, 0u);
#pragma unroll
    for (int k = 0; k < VEC; k++)
        if (i + k < n) (k < 4 ? r.x : r.y) |= (uint32_t)c[i + k] << (8 * (k & 3));
    return r;
}

__device__ __forceinline__ void store_codes(void *p, long long i, long long n, uint2 r)
{
    unsigned char *c = static_cast<unsigned char *>(p);
    if (i + VEC <= n) {
        __stcs(reinterpret_cast<uint2 *>(c + i), r);
        return;
    }
#pragma unroll
    for (int k = 0; k < VEC; k++)
        if (i + k < n) c[i + k] = (unsigned char)((k < 4 ? r.x : r.y) >> (8 * (k & 3)));
}

__device__ __forceinline__ void decode8(uint2 r, float scale, float2 (&x)[PAIRS])
{
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const __nv_fp8x2_storage_t c = (__nv_fp8x2_storage_t)(((k < 2 ? r.x : r.y) >> (16 * (k & 1))) & 0xffffu);
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        x[k] = mul2(f, make_float2(scale, scale));
    }
}

__device__ __forceinline__ uint2 encode8(const float2 (&x)[PAIRS])
{
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; k++)
        w[k] = (uint32_t)__nv_cvt_float2_to_fp8x2(x[k], __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The roots of 8 values >= 0 to within a rare last bit: the hardware's reciprocal root (2^-22), then one Newton step
// with the residual v - r^2 taken exactly by a fused multiply-add (Markstein, IBM J. Res. Dev. 34, 1990).  Values
// outside the normal range take the library's root.  (The library's for all of them: 170 us of 1220 us for the 412
// million elements below.)
__device__ __forceinline__ void roots(const float2 (&v)[PAIRS], float2 (&r)[PAIRS])
{
    float lo = v[0].x, hi = v[0].x;
#pragma unroll
    for (int k = 0; k < PAIRS; k++) {
        lo = fminf(lo, fminf(v[k].x, v[k].y));
        hi = fmaxf(hi, fmaxf(v[k].x, v[k].y));
    }
    if (lo >= 1.17549435e-38f && hi <= 3.40282347e38f) {
#pragma unroll
        for (int k = 0; k < PAIRS; k++) {
            float2 y;
            asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(v[k].x));
            asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(v[k].y));
            const float2 r0 = mul2(v[k], y);
            const float2 e = fma2(make_float2(-r0.x, -r0.y), r0, v[k]);
            r[k] = fma2(e, mul2(y, make_float2(0.5f, 0.5f)), r0);
        }
    } else {
#pragma unroll
        for (int k = 0; k < PAIRS; k++) r[k] = make_float2(__fsqrt_rn(v[k].x), __fsqrt_rn(v[k].y));
    }
}

// x / d with y = 1 / d rounded: the product corrected by its exact residual (the same source), so that a code does not
// depend on y's last bit.
__device__ __forceinline__ float2 quotient(float2 x, float d, float y)
{
    const float2 yy = make_float2(y, y), q = mul2(x, yy);
    return fma2(fma2(q, make_float2(-d, -d), x), yy, q);
}

// A bijection of 32-bit words: shifts and odd multipliers, twice, the fractions of the roots of 2 and 3 (5, 7 and the golden
// ratio's below).  One input bit turned turns every output bit with a probability within 0.008 of a half.
__host__ __device__ __forceinline__ uint32_t mixed(uint32_t x)
{
    x = (x ^ (x >> 16)) * 0x6a09e667u;
    x = (x ^ (x >> 14)) * 0xbb67ae85u;
    return x ^ (x >> 16);
}
// Where the random words of one tensor's step start.
__device__ __forceinline__ uint32_t step_key(uint32_t seed, unsigned id, long long step)
{
    return mixed(mixed(seed + (uint32_t)step) + id * 0x9e3779b9u + (uint32_t)(step >> 32));
}

// e4m3 neighbours of a >= 0: codes keep 3 mantissa bits, and below 2^-6 are 2^-9 apart, as fp32 numbers with 3 mantissa
// bits are from 2^-6 on; so those are taken 2^-6 higher.
constexpr float E4M3_NORMAL = 0.015625f;
constexpr uint32_t E4M3_REST = 0xfffffu;       // mantissa bits that a code drops

// Two values with the code above each in magnitude taken with the probability of its place between its neighbours.  A word
// of the random ones serves an element: 12 bits for m, 23 for the root, whose steps are the shorter ones (1 - b2 of a code).
// ALL: every value is finite and E4M3_NORMAL at least.  (412 million weights: 1234 us; 1516 by the general path alone; codes
// to nearest 1090.)
template <bool ALL> __device__ __forceinline__ float2 stochastic(float2 x, uint32_t w0, uint32_t w1)
{
    const uint32_t r0 = (w0 & 0xfffu) << 8 | 0x80u, r1 = (w1 & 0xfffu) << 8 | 0x80u;
    if constexpr (ALL)
        return make_float2(__uint_as_float((__float_as_uint(x.x) + r0) & ~E4M3_REST), __uint_as_float((__float_as_uint(x.y) + r1) & ~E4M3_REST));
    const auto one = [](float v, uint32_t r) {
        const float a = fabsf(v), off = a < E4M3_NORMAL ? E4M3_NORMAL : 0.f;
        const float c = __uint_as_float((__float_as_uint(a + off) + r) & ~E4M3_REST) - off;
        return a <= 3.40282347e38f ? copysignf(c, v) : v;  // NaN stays
    };
    return make_float2(one(x.x, r0), one(x.y, r1));
}
// The same of two roots whose squares are to keep their expected values: hi with (x^2 - lo^2) / (hi^2 - lo^2).
template <bool ALL> __device__ __forceinline__ float2 stochastic_root(float2 x, uint32_t w0, uint32_t w1)
{
    const float2 off = make_float2(!ALL && x.x < E4M3_NORMAL ? E4M3_NORMAL : 0.f, !ALL && x.y < E4M3_NORMAL ? E4M3_NORMAL : 0.f);
    const float2 y = ALL ? x : add2(x, off);
    const uint32_t b0 = __float_as_uint(y.x) & ~E4M3_REST, b1 = __float_as_uint(y.y) & ~E4M3_REST;
    float2 lo = make_float2(__uint_as_float(b0), __uint_as_float(b1));
    float2 hi = make_float2(__uint_as_float(b0 + E4M3_REST + 1u), __uint_as_float(b1 + E4M3_REST + 1u));
    if constexpr (!ALL) {
        lo = make_float2(lo.x - off.x, lo.y - off.y);
        hi = make_float2(hi.x - off.x, hi.y - off.y);
    }
    // u in [1, 2): hi where (u - 1) (hi^2 - lo^2) < x^2 - lo^2
    const float2 u = make_float2(__uint_as_float(0x3f800000u | w0 >> 9), __uint_as_float(0x3f800000u | w1 >> 9));
    const float2 minus = make_float2(-lo.x, -lo.y), q = mul2(add2(hi, minus), add2(hi, lo));
    const float2 d = fma2(make_float2(-u.x, -u.y), q, fma2(add2(x, minus), add2(x, lo), q));
    const float2 c = make_float2(d.x > 0.f ? hi.x : lo.x, d.y > 0.f ? hi.y : lo.y);
    if constexpr (ALL) return c;
    return make_float2(x.x <= 3.40282347e38f ? c.x : x.x, x.y <= 3.40282347e38f ? c.y : x.y);
}
// The largest of `top` and those of a, b >= 0 that are finite: with 2^23 added, their bits are positive numbers alone.
__device__ __forceinline__ float largest_finite(float top, float a, float b)
{
    const auto place = [](float x) { return (int)(__float_as_uint(x) + 0x00800000u); };
    return __int_as_float(max(place(top), max(place(a), place(b))) - 0x00800000);
}
// At least the smallest code; NaN stays
__device__ __forceinline__ float raised(float x)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(E4M3_TINY));
    return r;
}
// min(a, |b|); NaN if one is
__device__ __forceinline__ float least(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

template <typename PT, typename GT, State STATE, int CAP>
__global__ void __launch_bounds__(THREADS, 12) adamw_kernel(const __grid_constant__ Table<CAP> tab, const Hyper h)
{
    constexpr bool E4M3 = STATE != F32;
    if (h.found_inf != nullptr && *h.found_inf != 0.f) return;
    int lo = 0, hi = tab.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.e[mid].first <= blockIdx.x) lo = mid; else hi = mid - 1;
    }
    const Entry &e = tab.e[lo];
    const long long n = e.numel;
    const long long i = (long long)(blockIdx.x - e.first) * CHUNK + threadIdx.x * VEC;
    const float gs = h.grad_scale != nullptr ? *h.grad_scale : 1.f;
    float c1 = h.c1, rs2 = h.rs2, lr_wd = h.lr_wd;
    if (h.lr_dev != nullptr || h.step_dev != nullptr) {
        // 1 - b^t without cancellation for small t: -expm1(t log b)
        const float lr = h.lr_dev != nullptr ? *h.lr_dev : h.lr;
        if (h.step_dev != nullptr) {
            const float t = fmaxf((float)*h.step_dev, 1.f);
            c1 = lr / -expm1f(t * h.log_b1);
            rs2 = rsqrtf(-expm1f(t * h.log_b2));
        } else {
            c1 = lr * h.c1;  // the host left 1 / (1 - b1^t) there
        }
        lr_wd = lr * h.wd;
    }
    PT *param = static_cast<PT *>(e.param);
    const GT *grad = static_cast<const GT *>(e.grad);

    if ((i & ~(long long)(CSA_ADAMW_BLOCK - 1)) >= n) return;  // the whole warp lies behind the end
    float2 p[PAIRS], g[PAIRS], m[PAIRS], v[PAIRS];
    const long long blk = i / CSA_ADAMW_BLOCK;  // the same for the whole warp
    load8<GT>(grad, i, n, g);
    if constexpr (E4M3) {
        const uint2 cm = load_codes(e.m, i, n), cv = load_codes(e.v, i, n);
        const float sm = e.m_scale[blk], sv = e.v_scale[blk];
        if (e.master != nullptr) load8<float>(e.master, i, n, p); else load8<PT>(param, i, n, p);
        decode8(cm, sm, m);
        decode8(cv, sv, v);
#pragma unroll
        for (int k = 0; k < PAIRS; k++) v[k] = mul2(v[k], v[k]);
    } else {
        load8<float>(static_cast<const float *>(e.m), i, n, m);
        load8<float>(static_cast<const float *>(e.v), i, n, v);
        if (e.master != nullptr) load8<float>(e.master, i, n, p); else load8<PT>(param, i, n, p);
    }
    // The moments as the formula has them, each operation rounded: an 8-bit code then depends on the tensors alone.
    // (Not in pairs: a paired product and a paired sum were joined into one rounding.)
    const auto both = [](float x) { return make_float2(x, x); };
    const auto blend = [](float b, float old, float nb, float x) { return __fadd_rn(__fmul_rn(b, old), __fmul_rn(nb, x)); };
#pragma unroll
    for (int k = 0; k < PAIRS; k++) {
        const float2 gk = mul2(g[k], both(gs));
        m[k] = make_float2(blend(h.b1, m[k].x, h.nb1, gk.x), blend(h.b1, m[k].y, h.nb1, gk.y));
        // (1 - b2) g g from the left
        v[k].x = __fadd_rn(__fmul_rn(h.b2, v[k].x), __fmul_rn(__fmul_rn(h.nb2, gk.x), gk.x));
        v[k].y = __fadd_rn(__fmul_rn(h.b2, v[k].y), __fmul_rn(__fmul_rn(h.nb2, gk.y), gk.y));
    }
    float2 r[PAIRS];
    roots(v, r);
    float top_m = 0.f, top_r = 0.f;
#pragma unroll
    for (int k = 0; k < PAIRS; k++) {
        const float2 d = fma2(r[k], both(rs2), both(h.eps));
        const float2 step = make_float2(__fdividef(m[k].x, d.x), __fdividef(m[k].y, d.y));
        p[k] = fma2(both(-c1), step, fma2(both(-lr_wd), p[k], p[k]));
        if constexpr (STATE == STOCHASTIC) {
            top_m = largest_finite(top_m, fabsf(m[k].x), fabsf(m[k].y));
            top_r = largest_finite(top_r, r[k].x, r[k].y);
        } else {
            top_m = fmaxf(top_m, fmaxf(fabsf(m[k].x), fabsf(m[k].y)));
            top_r = fmaxf(top_r, fmaxf(r[k].x, r[k].y));
        }
    }
    if (e.master != nullptr) store8<float>(e.master, i, n, p);
    store8<PT>(param, i, n, p);
    if constexpr (E4M3) {
        top_m = warp_max(top_m);
        top_r = warp_max(top_r);
        // An infinity has no code (it becomes NaN) and is no scale for its block.  (Asked for each value to nearest: 1103 us
        // instead of 1090; this branch in the stochastic kernel, which lacks the registers: 1351 instead of 1234.)
        if (STATE == NEAREST && __builtin_expect(!(fmaxf(top_m, top_r) <= 3.40282347e38f), 0)) {
            top_m = top_r = 0.f;
#pragma unroll
            for (int k = 0; k < PAIRS; k++) {
                top_m = largest_finite(top_m, fabsf(m[k].x), fabsf(m[k].y));
                top_r = largest_finite(top_r, r[k].x, r[k].y);
            }
            top_m = warp_max(top_m);
            top_r = warp_max(top_r);
        }
        const float sm = top_m * (1.f / E4M3_MAX), sr = top_r * (1.f / E4M3_MAX);
        // a block of magnitudes below 448e-36 keeps the codes of zeros (its reciprocal would leave the normal range)
        const float ym = sm >= 1e-36f ? 1.f / sm : 0.f, yr = sr >= 1e-36f ? 1.f / sr : 0.f;
#pragma unroll
        for (int k = 0; k < PAIRS; k++) {
            m[k] = quotient(m[k], sm, ym);
            v[k] = quotient(r[k], sr, yr);
        }
        if constexpr (STATE == STOCHASTIC) {
            const uint32_t key = step_key(h.seed, e.id, h.step_dev != nullptr ? max(*h.step_dev, (int64_t)1) : h.step);
            float low = E4M3_MAX;
#pragma unroll
            for (int k = 0; k < PAIRS; k++) low = least(least(low, m[k].x), least(least(low, m[k].y), least(v[k].x, v[k].y)));
            const auto draw = [&](auto all) {
#pragma unroll
                for (int k = 0; k < PAIRS; k++) {
                    // elements 2^31 apart share their word; a pair's second word is the first one mixed on
                    const uint32_t w0 = mixed(key + 2u * (uint32_t)(i + 2 * k));
                    uint32_t w1 = w0 * 0x3c6ef373u;
                    w1 ^= w1 >> 15;
                    m[k] = stochastic<decltype(all)::value>(m[k], w0, w1);
                    v[k] = stochastic_root<decltype(all)::value>(v[k], w0, w1);
                }
            };
            if (low >= E4M3_NORMAL) draw(std::true_type());
            else draw(std::false_type());
        }
#pragma unroll
        for (int k = 0; k < PAIRS; k++) {
            v[k].x = r[k].x > 0.f ? raised(v[k].x) : v[k].x;
            v[k].y = r[k].y > 0.f ? raised(v[k].y) : v[k].y;
        }
        store_codes(e.m, i, n, encode8(m));
        store_codes(e.v, i, n, encode8(v));
        if ((threadIdx.x & 31) == 0) {
            e.m_scale[blk] = sm;
            e.v_scale[blk] = sr;
        }
    } else {
        store8<float>(static_cast<float *>(e.m), i, n, m);
        store8<float>(static_cast<float *>(e.v), i, n, v);
    }
}

// The tensors of one launch: parameters of a kernel hold up to 32764 bytes; fewer tensors take a shorter
// table, whose upload is part of every launch.
constexpr int CAP_SMALL = 48, CAP_MIDDLE = 128, CAP_LARGE = 440;

template <int CAP> void fill(Table<CAP> &tab, const csa_adamw_tensor *all, const csa_adamw_tensor *const *t, int n)
{
    unsigned first = 0;
    for (int k = 0; k < n; k++) {
        Entry &e = tab.e[k];
        e.param = t[k]->param;
        e.grad = t[k]->grad;
        e.master = t[k]->master;
        e.m = t[k]->m;
        e.v = t[k]->v;
        e.m_scale = t[k]->m_scale;
        e.v_scale = t[k]->v_scale;
        e.numel = t[k]->numel;
        e.first = first;
        e.id = (unsigned)(t[k] - all);
        first += (unsigned)((t[k]->numel + CHUNK - 1) / CHUNK);
    }
    tab.n = n;
}

template <typename PT, typename GT, State Q>
cudaError_t launch_group(const csa_adamw_tensor *all, const csa_adamw_tensor *const *t, int n, unsigned chunks, const Hyper &h, cudaStream_t st)
{
    if (n <= CAP_SMALL) {
        Table<CAP_SMALL> tab;
        fill(tab, all, t, n);
        adamw_kernel<PT, GT, Q, CAP_SMALL><<<chunks, THREADS, 0, st>>>(tab, h);
    } else if (n <= CAP_MIDDLE) {
        Table<CAP_MIDDLE> tab;
        fill(tab, all, t, n);
        adamw_kernel<PT, GT, Q, CAP_MIDDLE><<<chunks, THREADS, 0, st>>>(tab, h);
    } else {
        Table<CAP_LARGE> tab;
        fill(tab, all, t, n);
        adamw_kernel<PT, GT, Q, CAP_LARGE><<<chunks, THREADS, 0, st>>>(tab, h);
    }
    note_launches(1);
    return cudaGetLastError();
}

// kind: 4 (param is bf16) + 2 (grad is bf16) + (8-bit states)
cudaError_t launch_kind(int kind, bool stochastic, const csa_adamw_tensor *all, const csa_adamw_tensor *const *t, int n,
                        unsigned chunks, const Hyper &h, cudaStream_t st)
{
    using bf = __nv_bfloat16;
    const auto run = [&](auto param, auto grad) {
        using P = decltype(param);
        using G = decltype(grad);
        if ((kind & 1) == 0) return launch_group<P, G, F32>(all, t, n, chunks, h, st);
        if (stochastic) return launch_group<P, G, STOCHASTIC>(all, t, n, chunks, h, st);
        return launch_group<P, G, NEAREST>(all, t, n, chunks, h, st);
    };
    switch (kind >> 1) {
    case 0: return run(float(), float());
    case 1: return run(float(), bf());
    case 2: return run(bf(), float());
    default: return run(bf(), bf());
    }
}

}  // namespace adamw

cudaError_t launch_adamw(const csa_adamw_params &p, const csa_adamw_tensor *t, int count, cudaStream_t st)
{
    using namespace adamw;
    Hyper h;
    const double bc1 = 1.0 - pow(p.beta1, (double)p.step), bc2 = 1.0 - pow(p.beta2, (double)p.step);
    h.lr = (float)p.lr;
    h.wd = (float)p.weight_decay;
    h.lr_wd = (float)(p.lr * p.weight_decay);
    h.b1 = (float)p.beta1;
    h.nb1 = (float)(1.0 - p.beta1);
    h.b2 = (float)p.beta2;
    h.nb2 = (float)(1.0 - p.beta2);
    h.eps = (float)p.eps;
    h.c1 = (float)((p.lr_dev != nullptr ? 1.0 : p.lr) / bc1);
    h.rs2 = (float)(1.0 / sqrt(bc2));
    h.log_b1 = (float)log(p.beta1);
    h.log_b2 = (float)log(p.beta2);
    h.lr_dev = p.lr_dev;
    h.step_dev = p.step_dev;
    h.seed = mixed(mixed((uint32_t)p.seed + 0xa54ff53au) + (uint32_t)(p.seed >> 32));
    h.step = p.step;
    h.grad_scale = p.grad_scale;
    h.found_inf = p.found_inf;
    for (int kind = 0; kind < 8; kind++) {
        const csa_adamw_tensor *group[CAP_LARGE];
        int n = 0;
        unsigned long long chunks = 0;
        for (int k = 0; k <= count; k++) {
            if (k < count) {
                const int kk = (t[k].param_dtype == CSA_BF16 ? 4 : 0) + (t[k].grad_dtype == CSA_BF16 ? 2 : 0) +
                               (t[k].state_dtype == CSA_STATE_E4M3 ? 1 : 0);
                if (kk != kind || t[k].numel == 0) continue;
            }
            const unsigned long long c = k < count ? (unsigned long long)(t[k].numel + CHUNK - 1) / CHUNK : 0;
            if (n > 0 && (k == count || n == CAP_LARGE || chunks + c > 0x7fffffffull)) {
                const cudaError_t e = launch_kind(kind, p.stochastic != 0, t, group, n, (unsigned)chunks, h, st);
                if (e != cudaSuccess) return e;
                n = 0;
                chunks = 0;
            }
            if (k < count) {
                group[n++] = t + k;
                chunks += c;
            }
        }
    }
    return cudaSuccess;
}

}  // namespace csa
