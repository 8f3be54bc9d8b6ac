// k_linear_small.cu -- projections of a few rows (decoding): y = act(alpha x W^T + bias) + residual for M <= 8.
//
// Every weight is used M times only, so the pass over W is the whole cost: 2 N K bytes.  A tensor-core tile would
// spend its set-up and its epilogue on 128 rows; here a warp takes four rows of W (four output columns) and runs
// along k with 16-byte loads, a lane every 32nd of them, and holds the M x 4 sums in registers, in fp32, as pairs of
// even and odd k.  x is a few KB and comes from L1.  Where N gives too few warps for the GPU, the warps of a CTA share
// the four rows and cut the k axis among them (the join is a fixed order: the same bits every time).
#include "k_linear.cuh"
#include "tc_ptx.cuh"

namespace csa {
namespace linear {

using bf16 = __nv_bfloat16;
constexpr int WARPS = 8, ROWS = 4;   // warps of a CTA, rows of W a warp takes

// E values along k as pairs: a 16-byte vector, or one value and a zero
template <typename V, int E> struct Vec;
template <> struct Vec<bf16, 8> {
    uint4 w;
    __device__ void load(const bf16 *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ void stream(const bf16 *p) { w = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ float2 pair(int i) const
    {
        const uint32_t x = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
    static constexpr int PAIRS = 4;
};
template <> struct Vec<float, 4> {
    float4 w;
    __device__ void load(const float *p) { w = *reinterpret_cast<const float4 *>(p); }
    __device__ void stream(const float *p) { w = __ldcs(reinterpret_cast<const float4 *>(p)); }
    __device__ float2 pair(int i) const { return i == 0 ? make_float2(w.x, w.y) : make_float2(w.z, w.w); }
    static constexpr int PAIRS = 2;
};
template <typename V> struct Vec<V, 1> {
    float w;
    __device__ void load(const V *p) { w = lds<V>(p, 0); }
    __device__ void stream(const V *p) { w = lds<V>(p, 0); }
    __device__ float2 pair(int) const { return make_float2(w, 0.f); }
    static constexpr int PAIRS = 1;
};

// MT rows of x (those behind M repeat the last), KS warps of a CTA on the same rows of W.
template <typename V, int E, int MT>
__global__ void __launch_bounds__(32 * WARPS)
small_kernel(const V *x, long long ldx, const V *w, int M, int N, int K, int ks, const Epilogue e)
{
    __shared__ float part[WARPS][MT * ROWS];
    constexpr int U = MT >= 4 ? 1 : 2;   // vectors along k in flight together
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = (blockIdx.x * (WARPS / ks) + warp / ks) * ROWS, piece = warp % ks;
    chain_start();
    chain_wait();
    const V *wr[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; r++) wr[r] = w + (long long)min(n0 + r, N - 1) * K;
    float2 acc[MT][ROWS] = {};
    if (n0 < N) {
        const int step = 32 * E * ks;
        for (int k0 = (piece * 32 + lane) * E; k0 < K; k0 += step * U) {
            Vec<V, E> b[U][ROWS], a[U][MT];
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int r = 0; r < ROWS; r++)
                    if (k0 + u * step < K) b[u][r].stream(wr[r] + k0 + u * step);
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int m = 0; m < MT; m++)
                    if (k0 + u * step < K) a[u][m].load(x + min(m, M - 1) * ldx + k0 + u * step);
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (k0 + u * step >= K) break;
#pragma unroll
                for (int i = 0; i < Vec<V, E>::PAIRS; i++)
#pragma unroll
                    for (int r = 0; r < ROWS; r++) {
                        const float2 q = b[u][r].pair(i);
#pragma unroll
                        for (int m = 0; m < MT; m++) acc[m][r] = ptx::fma2(a[u][m].pair(i), q, acc[m][r]);
                    }
            }
        }
    }
    float s[MT * ROWS];
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int r = 0; r < ROWS; r++) s[m * ROWS + r] = warp_sum(acc[m][r].x + acc[m][r].y);
    // lane i of a row's first warp finishes sum i
    float t = 0.f;
    if (ks > 1) {
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < MT * ROWS; i++) part[warp][i] = s[i];
        __syncthreads();
        if (piece != 0 || lane >= MT * ROWS) return;
        for (int p = 0; p < ks; p++) t += part[warp + p][lane];
    } else {
        if (lane >= MT * ROWS) return;
#pragma unroll
        for (int i = 0; i < MT * ROWS; i++)
            if (lane == i) t = s[i];
    }
    const int m = lane / ROWS, n = n0 + lane % ROWS;
    if (m >= M || n >= N) return;
    float z = fmaf(e.alpha, t, e.bias != nullptr ? __ldg(e.bias + n) : 0.f);
    const long long at = (long long)m * N + n;
    if (e.preact != nullptr) {
        if (e.preact_f32) ((float *)e.preact)[at] = z;
        else ((bf16 *)e.preact)[at] = __float2bfloat16_rn(z);
    }
    z = act_fwd(z, e.act);
    if (e.out_f32) {
        if (e.res != nullptr) z += ((const float *)e.res)[m * e.ldr + n];
        ((float *)e.out)[at] = z;
    } else {
        if (e.res != nullptr) z += __bfloat162float(((const bf16 *)e.res)[m * e.ldr + n]);
        ((bf16 *)e.out)[at] = __float2bfloat16_rn(z);
    }
}

template <typename V, int E>
static cudaError_t launch_rows(const V *x, long long ldx, const V *w, int M, int N, int K, const Epilogue &e, int sms,
                               cudaStream_t st)
{
    const long long groups = (N + ROWS - 1) / ROWS;
    int ks = 1;
    while (ks < WARPS && groups * ks < 16LL * sms && K > 32 * E * ks) ks *= 2;
    const unsigned grid = (unsigned)((groups * ks + WARPS - 1) / WARPS);
    auto *kernel = M == 1 ? small_kernel<V, E, 1> : M == 2 ? small_kernel<V, E, 2> : M <= 4 ? small_kernel<V, E, 4> : small_kernel<V, E, 8>;
    return launch_chained(kernel, dim3(grid), 32 * WARPS, 0, 1, st, x, ldx, w, M, N, K, ks, e);
}

cudaError_t launch_linear_small(const csa_linear_params &p, const void *x, const void *w, const Epilogue &e, int sms,
                                cudaStream_t st)
{
    const int M = (int)p.rows, N = p.out_features, K = p.in_features;
    // 16-byte vectors where every row starts on one and holds whole ones
    if (p.dtype == CSA_F32) {
        if (((K | p.x_stride) & 3) == 0) return launch_rows<float, 4>((const float *)x, p.x_stride, (const float *)w, M, N, K, e, sms, st);
        return launch_rows<float, 1>((const float *)x, p.x_stride, (const float *)w, M, N, K, e, sms, st);
    }
    if (((K | p.x_stride) & 7) == 0) return launch_rows<bf16, 8>((const bf16 *)x, p.x_stride, (const bf16 *)w, M, N, K, e, sms, st);
    return launch_rows<bf16, 1>((const bf16 *)x, p.x_stride, (const bf16 *)w, M, N, K, e, sms, st);
}

}  // namespace linear
}  // namespace csa
