// k_linear.cu -- projections: y = act(alpha x W^T + bias) + residual and its gradients.
#include "csa_internal.cuh"

namespace csa {
namespace linear {

__device__ __forceinline__ float act_fwd(float z, int act)
{
    if (act == CSA_ACT_RELU) return z > 0.f ? z : (z == z ? 0.f : z);
    if (act == CSA_ACT_SILU) return z / (1.f + __expf(-z));
    if (act == CSA_ACT_GELU_TANH) return z / (1.f + __expf(-1.5957691216057308f * (z + 0.044715f * z * z * z)));
    return z;
}

// act'(z)
__device__ __forceinline__ float act_grad(float z, int act)
{
    if (act == CSA_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if (act == CSA_ACT_SILU) {
        const float s = 1.f / (1.f + __expf(-z));
        return s * (1.f + z * (1.f - s));
    }
    if (act == CSA_ACT_GELU_TANH) {
        const float c = 1.5957691216057308f, k = 0.044715f;
        const float s = 1.f / (1.f + __expf(-c * (z + k * z * z * z)));
        return s + z * s * (1.f - s) * c * (1.f + 3.f * k * z * z);
    }
    return 1.f;
}

constexpr int T = 64, KT = 16;

// D[m][n] = sum_k A[m sam + k sak] B[n sbn + k sbk]
template <typename V, typename O>
__global__ void __launch_bounds__(256)
gemm_simple(const V *A, long long sam, long long sak, const V *B, long long sbn, long long sbk, long long M, int N,
            long long K, float alpha, const float *bias, int act, const O *res, long long ldr, O *out, V *preact)
{
    __shared__ float sa[KT][T + 1], sb[KT][T + 1];
    const long long m0 = (long long)blockIdx.x * T, n0 = (long long)blockIdx.y * T;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (long long k0 = 0; k0 < K; k0 += KT) {
        for (int i = threadIdx.x; i < T * KT; i += 256) {
            const int m = i / KT, k = i % KT;
            sa[k][m] = m0 + m < M && k0 + k < K ? ldf<V>(A, (m0 + m) * sam + (k0 + k) * sak) : 0.f;
            sb[k][m] = n0 + m < N && k0 + k < K ? ldf<V>(B, (n0 + m) * sbn + (k0 + k) * sbk) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < KT; k++)
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) acc[i][j] += sa[k][ty + 16 * i] * sb[k][tx + 16 * j];
        __syncthreads();
    }
    for (int i = 0; i < 4; i++)
        for (int j = 0; j < 4; j++) {
            const long long m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= M || n >= N) continue;
            float z = alpha * acc[i][j] + (bias != nullptr ? bias[n] : 0.f);
            if (preact != nullptr) preact[m * N + n] = from_f<V>(z);
            z = act_fwd(z, act);
            if (res != nullptr) z += ldf<O>(res, m * ldr + n);
            out[m * N + n] = from_f<O>(z);
        }
}

// dz = dy act'(z); db
template <typename V, typename O>
__global__ void dz_simple(const O *dy, long long ldy, const V *z, int act, V *dz, float *db, long long M, int N)
{
    const int n = blockIdx.x * blockDim.x + threadIdx.x;
    if (n >= N) return;
    float sum = 0.f;
    for (long long m = 0; m < M; m++) {
        float d = ldf<O>(dy, m * ldy + n);
        if (act != CSA_ACT_NONE) d *= act_grad(ldf<V>(z, m * N + n), act);
        dz[m * N + n] = from_f<V>(d);
        sum += d;
    }
    if (db != nullptr) db[n] = sum;
}

template <typename V, typename O>
cudaError_t fwd(const csa_linear_params &p, const void *x, const void *w, const float *bias, const void *res, void *y,
                void *preact, cudaStream_t st)
{
    const dim3 grid((unsigned)((p.rows + T - 1) / T), (p.out_features + T - 1) / T);
    gemm_simple<V, O><<<grid, 256, 0, st>>>((const V *)x, p.x_stride, 1, (const V *)w, p.in_features, 1, p.rows,
                                            p.out_features, p.in_features, p.alpha, bias, p.activation, (const O *)res,
                                            p.residual_stride, (O *)y, (V *)preact);
    note_launches(1);
    return cudaGetLastError();
}

template <typename V, typename O>
cudaError_t bwd(const csa_linear_params &p, const void *dy, const void *x, const void *w, const void *z, void *dx,
                void *dw, float *db, void *ws, cudaStream_t st)
{
    V *dz = (V *)ws;
    const int N = p.out_features, K = p.in_features;
    dz_simple<V, O><<<(N + 127) / 128, 128, 0, st>>>((const O *)dy, p.dy_stride, (const V *)z, p.activation, dz, db, p.rows, N);
    note_launches(1);
    if (dx != nullptr && p.rows > 0) {
        const dim3 grid((unsigned)((p.rows + T - 1) / T), (K + T - 1) / T);
        gemm_simple<V, V><<<grid, 256, 0, st>>>(dz, N, 1, (const V *)w, 1, K, p.rows, K, N, p.alpha, nullptr, 0,
                                                (const V *)nullptr, 0, (V *)dx, (V *)nullptr);
        note_launches(1);
    }
    if (dw != nullptr) {
        const dim3 grid((N + T - 1) / T, (K + T - 1) / T);
        gemm_simple<V, V><<<grid, 256, 0, st>>>(dz, 1, N, (const V *)x, 1, p.x_stride, N, K, p.rows, p.alpha, nullptr, 0,
                                                (const V *)nullptr, 0, (V *)dw, (V *)nullptr);
        note_launches(1);
    }
    return cudaGetLastError();
}

}  // namespace linear

size_t linear_fwd_workspace(const csa_linear_params &) { return 0; }
size_t linear_bwd_workspace(const csa_linear_params &p)
{
    return (size_t)p.rows * p.out_features * (p.dtype == CSA_BF16 ? 2 : 4);
}

cudaError_t launch_linear_fwd(const csa_linear_params &p, const void *x, const void *weight, const float *bias,
                              const void *residual, void *y, void *preact, void *, cudaStream_t st)
{
    using bf = __nv_bfloat16;
    note_path("generic");
    if (p.dtype == CSA_F32) return linear::fwd<float, float>(p, x, weight, bias, residual, y, preact, st);
    if (p.out_dtype == CSA_F32) return linear::fwd<bf, float>(p, x, weight, bias, residual, y, preact, st);
    return linear::fwd<bf, bf>(p, x, weight, bias, residual, y, preact, st);
}

cudaError_t launch_linear_bwd(const csa_linear_params &p, const void *dy, const void *x, const void *weight,
                              const void *preact, void *dx, void *dw, float *db, void *ws, cudaStream_t st)
{
    using bf = __nv_bfloat16;
    note_path("generic");
    if (p.dtype == CSA_F32) return linear::bwd<float, float>(p, dy, x, weight, preact, dx, dw, db, ws, st);
    if (p.out_dtype == CSA_F32) return linear::bwd<bf, float>(p, dy, x, weight, preact, dx, dw, db, ws, st);
    return linear::bwd<bf, bf>(p, dy, x, weight, preact, dx, dw, db, ws, st);
}

}  // namespace csa
