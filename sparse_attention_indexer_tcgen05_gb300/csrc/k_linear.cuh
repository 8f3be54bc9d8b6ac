// k_linear.cuh -- what the projections' kernels share: the activations, the epilogue's arguments and the product.
#pragma once

#include "csa_internal.cuh"
#include "tc_ptx.cuh"

namespace csa {
namespace linear {

// s(u) = 1 / (1 + 2^t), t = -u log2(e), with the hardware's base-2 exponential and reciprocal (2 units in the last
// place each)
__device__ __forceinline__ float sigmoid2(float t)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu = 1.5957691216057308f, kCubic = 0.044715f;  // 2 sqrt(2 / pi)
__device__ __forceinline__ float sigmoid(float u) { return sigmoid2(-kLog2e * u); }
// s(kGelu (z + kCubic z^3))
__device__ __forceinline__ float gelu_sigmoid(float z)
{
    return sigmoid2(z * fmaf(-kLog2e * kGelu * kCubic, z * z, -kLog2e * kGelu));
}

template <int ACT> __device__ __forceinline__ float act_fwd(float z)
{
    if constexpr (ACT == CSA_ACT_RELU) return z < 0.f ? 0.f : z;  // keeps NaN
    if constexpr (ACT == CSA_ACT_SILU) return z * sigmoid(z);
    if constexpr (ACT == CSA_ACT_GELU_TANH) return z * gelu_sigmoid(z);
    return z;
}
__device__ __forceinline__ float act_fwd(float z, int act)
{
    if (act == CSA_ACT_RELU) return act_fwd<CSA_ACT_RELU>(z);
    if (act == CSA_ACT_SILU) return act_fwd<CSA_ACT_SILU>(z);
    if (act == CSA_ACT_GELU_TANH) return act_fwd<CSA_ACT_GELU_TANH>(z);
    return z;
}

// The same of two values, GELU in paired arithmetic (8192 x 8192 x 512 with GELU 71 us -> 68; SiLU gains nothing).
template <int ACT> __device__ __forceinline__ float2 act_fwd2(float2 z)
{
    using ptx::fma2;
    using ptx::mul2;
    const auto both = [](float x) { return make_float2(x, x); };
    if constexpr (ACT == CSA_ACT_GELU_TANH) {
        const float2 t = mul2(z, fma2(mul2(z, z), both(-kLog2e * kGelu * kCubic), both(-kLog2e * kGelu)));
        return mul2(z, make_float2(sigmoid2(t.x), sigmoid2(t.y)));
    }
    return make_float2(act_fwd<ACT>(z.x), act_fwd<ACT>(z.y));
}

// act'(z) of two values (SILU or GELU_TANH), in paired arithmetic: the gradient's pass over dy and z is short of issue slots.
//   SILU: s (1 + z (1 - s)), s = s(z);  GELU: s + z s (1 - s) kGelu (1 + 3 kCubic z^2), s = gelu_sigmoid(z)
__device__ __forceinline__ float2 act_grad2(float2 z, int act)
{
    using ptx::fma2;
    using ptx::mul2;
    const auto both = [](float x) { return make_float2(x, x); };
    if (act == CSA_ACT_SILU) {
        const float2 t = mul2(z, both(-kLog2e)), s = make_float2(sigmoid2(t.x), sigmoid2(t.y));
        return mul2(s, fma2(z, fma2(s, both(-1.f), both(1.f)), both(1.f)));
    }
    const float2 zz = mul2(z, z), t = mul2(z, fma2(zz, both(-kLog2e * kGelu * kCubic), both(-kLog2e * kGelu)));
    const float2 s = make_float2(sigmoid2(t.x), sigmoid2(t.y));
    const float2 q = mul2(s, fma2(s, both(-1.f), both(1.f)));  // 0 far out, where z^2 may overflow
    const float2 g = fma2(mul2(z, q), fma2(zz, both(3.f * kCubic * kGelu), both(kGelu)), s);
    return make_float2(q.x > 0.f ? g.x : s.x, q.y > 0.f ? g.y : s.y);
}

// Where a product's sums go.  y = act(alpha sum + bias[n]) + res; with `partial` the bare sums of split s go to
// partial[s][M][partial_stride(N)] instead.
struct Epilogue {
    float alpha;
    int act;
    const float *bias;
    const void *res;
    long long ldr;
    void *out;           // [M][N]
    void *preact;        // [M][N] bf16 or fp32 as `preact_f32` says, or null
    int out_f32, preact_f32;
    float *partial;      // rows partial_stride(N) apart
};

// Rows of partial sums start on 32-byte sectors whatever N is.
__host__ __device__ inline long long partial_stride(long long N) { return (N + 7) & ~7LL; }

// Kernels of one call follow one another closely: each lets the next one's CTAs start as soon as its own are all running
// (they set up barriers and TMEM meanwhile) and waits for the whole of its predecessors before it touches memory.
__device__ __forceinline__ void chain_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    if (e == cudaSuccess) note_launches(1);
    return e;
}

// The aligned 16 bytes at q of an argument that ends at `end`: nothing from there on is read (its place holds 0).
__device__ __forceinline__ uint4 load16(const uint4 *q, const void *end)
{
    if (q + 1 <= end) return __ldcs(q);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(q) + k;
        w[k] = p + 1 <= end ? *p : reinterpret_cast<const unsigned short *>(p) + 1 <= end ? *reinterpret_cast<const unsigned short *>(p) : 0u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One operand of a product over k: element (i, k) of plane q at base + q * plane + (k_major ? i ld + k : k ld + i).
// fp32 values are held as three bf16 planes, x = h + m + l.
struct Operand {
    const __nv_bfloat16 *base;
    long long ld, plane;   // elements; multiples of 8
    bool k_major;
};

// Tile and cut of the k axis of a product (see k_linear_tc.cu).
enum Shape { LONE_64, PAIR_128, PAIR_256 };
struct Plan {
    Shape shape;
    int splits;   // pieces of the k axis: above 1, the caller provides splits * M * partial_stride(N) floats and joins them
    bool exact;   // sums kept in registers (see k_linear_tc.cu)
};
// out_f32: the result itself is fp32 (and not only its pieces)
Plan plan_product(long long M, long long N, long long K, int planes, int passes, bool out_f32, int sms);

// D[m][n] = sum_k A(m, k) B(n, k), M x N x K, with `planes` = 1 or 3.  One plane, two passes: A is the sum of two planes, and
// each stage of the k axis takes the second one and B, then the first one and B.
struct Product {
    Operand a, b;
    long long M, N, K;
    int planes, passes;
    Plan plan;
    Epilogue e;
};
cudaError_t launch_product_tc(const Product &p, int sms, cudaStream_t st);

// The forward of a few rows (k_linear_small.cu); operands where they are, no workspace.
constexpr int kSmallRows = 8, kFewRows = 16;
bool small_linear(const csa_linear_params &p);
cudaError_t launch_linear_small(const csa_linear_params &p, const void *x, const void *w, const Epilogue &e, int sms,
                                cudaStream_t st);

}  // namespace linear
}  // namespace csa
