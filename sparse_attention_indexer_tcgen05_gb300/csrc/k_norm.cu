// k_norm.cu -- layer norm of rows and its gradients.
//
//   mean = sum_j x_j / n,  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / n + eps),  h_j = (x_j - mean) rstd,  y_j = h_j w_j + b_j
//   a_j = dy_j w_j,  dx_j = rstd (a_j - mean(a) - h_j mean(a h)),  dw_j = sum over rows of dy_j h_j,  db_j = sum of dy_j
//
// Bound by memory: x read and y written once (backward: x and dy read, dx written).  A row's values stay in the registers of
// LANES threads, so that the variance is a second pass over registers and not a difference of two large sums.  The backward's
// threads keep their columns over all the rows that their block takes, and so the gradients of their weights; the blocks'
// sums are joined in a fixed order by a second kernel: the same bits every time.
#include "k_linear.cuh"

#include <type_traits>

namespace csa {
namespace norm {

using bf16 = __nv_bfloat16;
using linear::chain_start;
using linear::chain_wait;
using linear::launch_chained;

__device__ __forceinline__ float from_value(float x) { return x; }
__device__ __forceinline__ float from_value(bf16 x) { return __bfloat162float(x); }

// The two parameters, of either type
__device__ __forceinline__ float param(const void *p, int f32, long long i)
{
    return f32 ? __ldg(static_cast<const float *>(p) + i) : __bfloat162float(static_cast<const bf16 *>(p)[i]);
}

// Values of a row that a thread holds: CH pieces of 8.  VEC: 8 neighbouring ones each, as vectors (rows on 16-byte
// boundaries, whole pieces); else every LANES-th one, so that a warp's accesses are neighbours whatever the alignment.
template <int LANES, int CH, bool VEC> __device__ __forceinline__ int column(int t, int c, int k)
{
    return VEC ? (c * LANES + t) * 8 + k : (c * 8 + k) * LANES + t;
}

template <typename T> __device__ __forceinline__ void load_vec(const T *p, float (&x)[8])
{
    if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 8; k++) x[k] = __uint_as_float(k % 2 == 0 ? u[k / 2] << 16 : u[k / 2] & 0xffff0000u);
    }
}
template <typename T> __device__ __forceinline__ void store_vec(T *p, const float (&x)[8])
{
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
            u[k] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// Columns that do not exist hold 0.
template <typename T, int LANES, int CH, bool VEC> __device__ __forceinline__ void load_row(const T *row, int n, int t, float (&x)[CH][8])
{
#pragma unroll
    for (int c = 0; c < CH; c++) {
        if constexpr (VEC) {
            if (column<LANES, CH, true>(t, c, 0) < n) {
                load_vec(row + column<LANES, CH, true>(t, c, 0), x[c]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; k++) x[c][k] = 0.f;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const int j = column<LANES, CH, false>(t, c, k);
                x[c][k] = j < n ? from_value(row[j]) : 0.f;
            }
        }
    }
}
template <typename T, int LANES, int CH, bool VEC> __device__ __forceinline__ void store_row(T *row, int n, int t, const float (&y)[CH][8])
{
#pragma unroll
    for (int c = 0; c < CH; c++) {
        if constexpr (VEC) {
            if (column<LANES, CH, true>(t, c, 0) < n) store_vec(row + column<LANES, CH, true>(t, c, 0), y[c]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const int j = column<LANES, CH, false>(t, c, k);
                if (j < n) row[j] = from_f<T>(y[c][k]);
            }
        }
    }
}
template <int LANES, int CH, bool VEC>
__device__ __forceinline__ void load_param(const void *p, int f32, int n, int t, float missing, float (&w)[CH][8])
{
#pragma unroll
    for (int c = 0; c < CH; c++)
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const int j = column<LANES, CH, VEC>(t, c, k);
            w[c][k] = p != nullptr && j < n ? param(p, f32, j) : missing;
        }
}

// Sums over the LANES threads of a row, of V values at once.  Rows of more than a warp have the block to themselves.
template <int LANES, int V> __device__ __forceinline__ void row_sums(float (&s)[V], float *part)
{
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
        for (int o = (LANES < 32 ? LANES : 32) / 2; o > 0; o >>= 1) s[v] += __shfl_xor_sync(0xffffffffu, s[v], o);
    if constexpr (LANES > 32) {
        constexpr int W = LANES / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        __syncthreads();  // the last sums have been read
        if (lane == 0) {
#pragma unroll
            for (int v = 0; v < V; v++) part[v * W + warp] = s[v];
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; v++) {
            s[v] = lane < W ? part[v * W + lane] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s[v] += __shfl_xor_sync(0xffffffffu, s[v], o);
        }
    }
}

struct Fwd {
    const void *x, *weight, *bias;
    void *y;
    float *stats;               // [2][rows] or null
    long long rows, stride;
    int n, param_f32;
    float eps;
};

constexpr int threads_of(int lanes) { return lanes <= 32 ? 256 : lanes; }

template <typename T, int LANES, int CH, bool VEC> __global__ void __launch_bounds__(threads_of(LANES)) norm_fwd_kernel(const Fwd a)
{
    constexpr int R = threads_of(LANES) / LANES;
    __shared__ float part[2 * (LANES / 32 + 1)];
    chain_start();
    chain_wait();
    const int t = threadIdx.x % LANES;
    const long long r = (long long)blockIdx.x * R + threadIdx.x / LANES;
    const bool live = r < a.rows;   // the warp's shuffles need all of its lanes
    const int n = live ? a.n : 0;
    float x[CH][8];
    load_row<T, LANES, CH, VEC>(static_cast<const T *>(a.x) + r * a.stride, n, t, x);
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; c++)
#pragma unroll
        for (int k = 0; k < 8; k++) s[0] += x[c][k];
    row_sums<LANES>(s, part);
    const float mean = s[0] / (float)a.n;
    s[0] = 0.f;
#pragma unroll
    for (int c = 0; c < CH; c++)
#pragma unroll
        for (int k = 0; k < 8; k++) {
            x[c][k] = column<LANES, CH, VEC>(t, c, k) < n ? x[c][k] - mean : 0.f;
            s[0] = fmaf(x[c][k], x[c][k], s[0]);
        }
    row_sums<LANES>(s, part);
    const float rstd = 1.f / sqrtf(s[0] / (float)a.n + a.eps);
    float w[CH][8], b[CH][8];
    load_param<LANES, CH, VEC>(a.weight, a.param_f32, n, t, 1.f, w);
    load_param<LANES, CH, VEC>(a.bias, a.param_f32, n, t, 0.f, b);
#pragma unroll
    for (int c = 0; c < CH; c++)
#pragma unroll
        for (int k = 0; k < 8; k++) x[c][k] = fmaf(x[c][k] * rstd, w[c][k], b[c][k]);
    store_row<T, LANES, CH, VEC>(static_cast<T *>(a.y) + r * a.n, n, t, x);
    if (a.stats != nullptr && live && t == 0) {
        a.stats[r] = mean;
        a.stats[a.rows + r] = rstd;
    }
}

struct Bwd {
    const void *dy, *x, *weight;
    const float *stats;
    void *dx;
    float *parts;               // [blocks][2][n]: the blocks' sums of dw and db; null: neither is asked for
    long long rows, x_stride, dy_stride;
    int n, param_f32;
};

template <typename T, int LANES, int CH, bool VEC> __global__ void __launch_bounds__(threads_of(LANES)) norm_bwd_kernel(const Bwd a)
{
    constexpr int R = threads_of(LANES) / LANES;
    __shared__ float part[2 * (LANES / 32 + 1)];
    __shared__ float across[R > 1 ? R : 1][R > 1 ? 2 : 1][R > 1 ? LANES * CH * 8 : 1];
    chain_start();
    chain_wait();
    const int t = threadIdx.x % LANES, group = threadIdx.x / LANES;
    float w[CH][8], dw[CH][8] = {}, db[CH][8] = {};
    load_param<LANES, CH, VEC>(a.weight, a.param_f32, a.n, t, 1.f, w);
    const float inv_n = 1.f / (float)a.n;
    for (long long r0 = (long long)blockIdx.x * R; r0 < a.rows; r0 += (long long)gridDim.x * R) {
        const long long r = r0 + group;
        const bool live = r < a.rows;
        const int n = live ? a.n : 0;
        float x[CH][8], d[CH][8];
        load_row<T, LANES, CH, VEC>(static_cast<const T *>(a.x) + r * a.x_stride, n, t, x);
        load_row<T, LANES, CH, VEC>(static_cast<const T *>(a.dy) + r * a.dy_stride, n, t, d);
        const float mean = live ? __ldg(a.stats + r) : 0.f, rstd = live ? __ldg(a.stats + a.rows + r) : 0.f;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CH; c++)
#pragma unroll
            for (int k = 0; k < 8; k++) {
                x[c][k] = column<LANES, CH, VEC>(t, c, k) < n ? (x[c][k] - mean) * rstd : 0.f;
                dw[c][k] = fmaf(d[c][k], x[c][k], dw[c][k]);
                db[c][k] += d[c][k];
                d[c][k] *= w[c][k];
                s[0] += d[c][k];
                s[1] = fmaf(d[c][k], x[c][k], s[1]);
            }
        if (a.dx != nullptr) {
            row_sums<LANES>(s, part);
            const float ma = s[0] * inv_n, mh = s[1] * inv_n;
#pragma unroll
            for (int c = 0; c < CH; c++)
#pragma unroll
                for (int k = 0; k < 8; k++) x[c][k] = rstd * (d[c][k] - ma - x[c][k] * mh);
            store_row<T, LANES, CH, VEC>(static_cast<T *>(a.dx) + r * a.n, n, t, x);
        }
    }
    if (a.parts == nullptr) return;
    float *out = a.parts + (long long)blockIdx.x * 2 * a.n;
    if constexpr (R > 1) {
#pragma unroll
        for (int c = 0; c < CH; c++)
#pragma unroll
            for (int k = 0; k < 8; k++) {
                across[group][0][column<LANES, CH, VEC>(t, c, k)] = dw[c][k];
                across[group][1][column<LANES, CH, VEC>(t, c, k)] = db[c][k];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * a.n; i += blockDim.x) {
            const int which = i >= a.n, j = i - which * a.n;
            float v = 0.f;
#pragma unroll
            for (int g = 0; g < R; g++) v += across[g][which][j];
            out[i] = v;
        }
    } else {
#pragma unroll
        for (int c = 0; c < CH; c++)
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const int j = column<LANES, CH, VEC>(t, c, k);
                if (j < a.n) {
                    out[j] = dw[c][k];
                    out[a.n + j] = db[c][k];
                }
            }
    }
}

// The blocks' sums joined: 32 columns a block, 32 threads a column.
__global__ void __launch_bounds__(1024) norm_join_kernel(const float *parts, int blocks, int n, void *dw, void *db, int param_f32)
{
    __shared__ float part[32][33];
    chain_start();
    chain_wait();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long long i = (long long)blockIdx.x * 32 + tx;
    float s = 0.f;
    if (i < 2LL * n) {
#pragma unroll 4
        for (int b = ty; b < blocks; b += 32) s += parts[(long long)b * 2 * n + i];
    }
    part[ty][tx] = s;
    __syncthreads();
    if (ty > 0 || i >= 2LL * n) return;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; k++) v += part[k][tx];
    void *out = i < n ? dw : db;
    const long long j = i < n ? i : i - n;
    if (out == nullptr) return;
    if (param_f32) static_cast<float *>(out)[j] = v;
    else static_cast<bf16 *>(out)[j] = __float2bfloat16_rn(v);
}

// ------------------------------------------------------------------ rows longer than the registers hold

// A block a row, read again for each of its sums (from L2 mostly).
template <typename T> __global__ void __launch_bounds__(1024) norm_fwd_long_kernel(const Fwd a)
{
    __shared__ float part[2 * 33];
    chain_start();
    chain_wait();
    const long long r = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + r * a.stride;
    float s[1] = {0.f};
    for (int j = threadIdx.x; j < a.n; j += 1024) s[0] += from_value(x[j]);
    row_sums<1024>(s, part);
    const float mean = s[0] / (float)a.n;
    s[0] = 0.f;
    for (int j = threadIdx.x; j < a.n; j += 1024) {
        const float d = from_value(x[j]) - mean;
        s[0] = fmaf(d, d, s[0]);
    }
    row_sums<1024>(s, part);
    const float rstd = 1.f / sqrtf(s[0] / (float)a.n + a.eps);
    T *y = static_cast<T *>(a.y) + r * a.n;
    for (int j = threadIdx.x; j < a.n; j += 1024) {
        const float w = a.weight != nullptr ? param(a.weight, a.param_f32, j) : 1.f, b = a.bias != nullptr ? param(a.bias, a.param_f32, j) : 0.f;
        y[j] = from_f<T>(fmaf((from_value(x[j]) - mean) * rstd, w, b));
    }
    if (a.stats != nullptr && threadIdx.x == 0) {
        a.stats[r] = mean;
        a.stats[a.rows + r] = rstd;
    }
}
template <typename T> __global__ void __launch_bounds__(1024) norm_dx_long_kernel(const Bwd a)
{
    __shared__ float part[2 * 33];
    chain_start();
    chain_wait();
    const long long r = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + r * a.x_stride, *dy = static_cast<const T *>(a.dy) + r * a.dy_stride;
    const float mean = a.stats[r], rstd = a.stats[a.rows + r];
    float s[2] = {0.f, 0.f};
    const auto at = [&](int j, float &h, float &d) {
        h = (from_value(x[j]) - mean) * rstd;
        d = from_value(dy[j]) * (a.weight != nullptr ? param(a.weight, a.param_f32, j) : 1.f);
    };
    for (int j = threadIdx.x; j < a.n; j += 1024) {
        float h, d;
        at(j, h, d);
        s[0] += d;
        s[1] = fmaf(d, h, s[1]);
    }
    row_sums<1024>(s, part);
    const float ma = s[0] / (float)a.n, mh = s[1] / (float)a.n;
    T *dx = static_cast<T *>(a.dx) + r * a.n;
    for (int j = threadIdx.x; j < a.n; j += 1024) {
        float h, d;
        at(j, h, d);
        dx[j] = from_f<T>(rstd * (d - ma - h * mh));
    }
}
// 256 columns of every gridDim.y-th row
template <typename T> __global__ void __launch_bounds__(256) norm_params_long_kernel(const Bwd a)
{
    chain_start();
    chain_wait();
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= a.n) return;
    float dw = 0.f, db = 0.f;
#pragma unroll 4
    for (long long r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float d = from_value(static_cast<const T *>(a.dy)[r * a.dy_stride + j]);
        dw = fmaf(d, (from_value(static_cast<const T *>(a.x)[r * a.x_stride + j]) - a.stats[r]) * a.stats[a.rows + r], dw);
        db += d;
    }
    float *out = a.parts + (long long)blockIdx.y * 2 * a.n;
    out[j] = dw;
    out[a.n + j] = db;
}

// ------------------------------------------------------------------ host side

constexpr int kLongest = 16384;  // columns that a block's registers hold

// Blocks of the backward, the same on every device: four for each of the GPU's SMs, or a part of the rows each.
int bwd_blocks(const csa_layernorm_params &p)
{
    const long long most = 4LL * linear::kSms;
    if (p.cols > kLongest) return (int)(p.rows < 64 ? (p.rows > 0 ? p.rows : 1) : 64);
    const long long each = p.cols <= 128 ? 16 : p.cols <= 512 ? 8 : 1;
    const long long want = (p.rows + each - 1) / each;
    return (int)(want < 1 ? 1 : want < most ? want : most);
}

// Calls f with the number of a row's threads and of their pieces.
template <typename F> cudaError_t by_cols(int n, const F &f)
{
    using std::integral_constant;
#define CSA_SHAPE(l, c) f(integral_constant<int, l>(), integral_constant<int, c>())
    if (n <= 128) return CSA_SHAPE(16, 1);
    if (n <= 256) return CSA_SHAPE(32, 1);
    if (n <= 512) return CSA_SHAPE(32, 2);
    if (n <= 1024) return CSA_SHAPE(128, 1);
    if (n <= 2048) return CSA_SHAPE(128, 2);
    if (n <= 4096) return CSA_SHAPE(256, 2);
    if (n <= 8192) return CSA_SHAPE(512, 2);
    return CSA_SHAPE(512, 4);
#undef CSA_SHAPE
}

template <typename T> cudaError_t fwd(const Fwd &a, bool vec, cudaStream_t st)
{
    if (a.n > kLongest) return launch_chained(norm_fwd_long_kernel<T>, dim3((unsigned)a.rows), 1024, 0, 1, st, a);
    return by_cols(a.n, [&](auto lanes, auto pieces) {
        constexpr int L = decltype(lanes)::value, C = decltype(pieces)::value, R = threads_of(L) / L;
        const dim3 grid((unsigned)((a.rows + R - 1) / R));
        return launch_chained(vec ? norm_fwd_kernel<T, L, C, true> : norm_fwd_kernel<T, L, C, false>, grid, threads_of(L), 0, 1, st, a);
    });
}
template <typename T> cudaError_t bwd(const Bwd &a, bool vec, int blocks, cudaStream_t st)
{
    if (a.n > kLongest) {
        // dx last: it may lie where dy or x do
        cudaError_t e = cudaSuccess;
        if (a.parts != nullptr)
            e = launch_chained(norm_params_long_kernel<T>, dim3((unsigned)((a.n + 255) / 256), (unsigned)blocks), 256, 0, 1, st, a);
        if (e != cudaSuccess || a.dx == nullptr) return e;
        return launch_chained(norm_dx_long_kernel<T>, dim3((unsigned)a.rows), 1024, 0, 1, st, a);
    }
    return by_cols(a.n, [&](auto lanes, auto pieces) {
        constexpr int L = decltype(lanes)::value, C = decltype(pieces)::value;
        return launch_chained(vec ? norm_bwd_kernel<T, L, C, true> : norm_bwd_kernel<T, L, C, false>, dim3((unsigned)blocks), threads_of(L), 0, 1, st, a);
    });
}

}  // namespace norm

size_t layernorm_bwd_workspace(const csa_layernorm_params &p)
{
    return p.rows == 0 ? 0 : linear::up256((size_t)norm::bwd_blocks(p) * 2 * p.cols * 4);
}

cudaError_t launch_layernorm_fwd(const csa_layernorm_params &p, const void *x, const void *weight, const void *bias, void *y, float *stats,
                                 cudaStream_t st)
{
    note_path("generic");
    const norm::Fwd a = {x, weight, bias, y, stats, p.rows, p.x_stride, p.cols, p.param_dtype == CSA_F32, p.eps};
    const int each = p.dtype == CSA_F32 ? 4 : 8;
    const bool vec = p.cols % 8 == 0 && p.x_stride % each == 0;
    return p.dtype == CSA_F32 ? norm::fwd<float>(a, vec, st) : norm::fwd<__nv_bfloat16>(a, vec, st);
}

cudaError_t launch_layernorm_bwd(const csa_layernorm_params &p, const void *dy, const void *x, const void *weight, const float *stats, void *dx,
                                 void *dweight, void *dbias, void *ws, cudaStream_t st)
{
    note_path("generic");
    const size_t size = p.param_dtype == CSA_F32 ? 4 : 2;
    if (p.rows == 0) {  // sums of nothing
        cudaError_t e = dweight != nullptr ? cudaMemsetAsync(dweight, 0, size * p.cols, st) : cudaSuccess;
        if (e == cudaSuccess && dbias != nullptr) e = cudaMemsetAsync(dbias, 0, size * p.cols, st);
        return e;
    }
    const bool params = dweight != nullptr || dbias != nullptr;
    if (dx == nullptr && !params) return cudaSuccess;
    const norm::Bwd a = {dy, x, weight, stats, dx, params ? static_cast<float *>(ws) : nullptr, p.rows, p.x_stride, p.dy_stride, p.cols,
                         p.param_dtype == CSA_F32};
    const int each = p.dtype == CSA_F32 ? 4 : 8, blocks = norm::bwd_blocks(p);
    const bool vec = p.cols % 8 == 0 && p.x_stride % each == 0 && p.dy_stride % each == 0;
    const cudaError_t e = p.dtype == CSA_F32 ? norm::bwd<float>(a, vec, blocks, st) : norm::bwd<__nv_bfloat16>(a, vec, blocks, st);
    if (e != cudaSuccess || !params) return e;
    return linear::launch_chained(norm::norm_join_kernel, dim3((unsigned)((2LL * p.cols + 31) / 32)), 1024, 0, 1, st, a.parts, blocks, p.cols, dweight,
                                  dbias, a.param_f32);
}

}  // namespace csa
