// k_linear_small.cu -- projections of a few rows (decoding): y = act(alpha x W^T + bias) + residual.
//
// Every weight is used once a row of x, so the pass over W is the whole cost: 2 N K bytes.  A tcgen05 tile would spend
// its set-up, its single CTA per SM and an epilogue over 128 rows on it.
//
// bf16, up to 16 rows (few_kernel): W's rows are the m16 side of warp-level MMAs (m16n8k16) and x's rows the n8 side, so
// fragments come straight from global memory: a lane loads 16 bytes of a row, and the k a fragment names may be any
// order that both operands share, so that four lanes read 64 contiguous bytes.  The 8 to 32 warps of a CTA take the same
// 16 rows of W and cut the k axis among them (their sums are joined in a fixed order: the same bits every time); sums
// move to fp32 registers of their own every 32 MMAs, which cut off rather than round.  The tensor cores are far from
// busy; what counts is the bytes in flight and the few instructions.  Bound by the start-up and W's way from DRAM: 8192
// outputs of 2048 values (33.6 MB) take 7.6 us for one row and 9.2 us for 16 with W in DRAM, 5.0 us for one with W in L2
// (with fp32 multiply-adds, 8 rows took 24 us; on a tcgen05 tile, 16).
//
// Other types and strides, up to 8 rows (small_kernel): a warp takes two rows of W and runs along k with 16-byte loads, a
// lane every 32nd of them, and holds the sums in registers, in fp32, as pairs of even and odd k.  x is a few KB and
// comes from L1.  Where N gives too few warps for the GPU, the warps of a CTA share the rows and cut the k axis.  fp32,
// 4096 outputs of 2048 values (33.6 MB): 7.0 us for one row, 10.6 us for 8.  bf16 rows off the 16-byte boundaries are loaded value by
// value: 8192 outputs of 2047 values 26 us for one row, 50 for 8.
#include "k_linear.cuh"
#include "tc_ptx.cuh"

namespace csa {
namespace linear {

using bf16 = __nv_bfloat16;
constexpr int WARPS = 4, ROWS = 2;   // small_kernel: warps of a CTA, rows of W a warp takes

// E values along k as pairs: a 16-byte vector, or one value and a zero
template <typename V, int E> struct Vec;
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

// The epilogue of one sum.
__device__ __forceinline__ void finish(const Epilogue &e, float t, int m, int n, int N)
{
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
    // every lane's sums added over the warp: halves are exchanged until a lane holds one value (value i: the lanes from
    // 32 i / (MT ROWS) on), then the rest of the lanes are added
    constexpr int V0 = MT * ROWS;
    float s[V0];
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int r = 0; r < ROWS; r++) s[m * ROWS + r] = acc[m][r].x + acc[m][r].y;
    int off = 16;
#pragma unroll
    for (int n = V0; n > 1; n /= 2, off /= 2)
#pragma unroll
        for (int i = 0; i < n / 2; i++) {
            const bool up = (lane & off) != 0;
            const float give = up ? s[i] : s[i + n / 2], keep = up ? s[i + n / 2] : s[i];
            s[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
        }
    for (; off > 0; off /= 2) s[0] += __shfl_xor_sync(0xffffffffu, s[0], off);
    const int value = lane * V0 / 32;
    float t = s[0];
    if (ks > 1) {
        if (lane * V0 % 32 == 0) part[warp][value] = t;
        __syncthreads();
        if (piece != 0) return;
        t = 0.f;
        for (int p = 0; p < ks; p++) t += part[warp + p][value];
    }
    if (lane * V0 % 32 != 0) return;
    const int m = value / ROWS, n = n0 + value % ROWS;
    if (m < M && n < N) finish(e, t, m, n, N);
}

// ------------------------------------------------------------------ bf16, up to 16 rows

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// MT tiles of 8 rows of x, WARPS_K warps of a CTA on the same rows of W, DEPTH pieces of 32 k of a warp in flight.  Lane
// (g, t) = (lane / 4, lane % 4) holds row g (and g + 8) of W's fragments, column g of x's and, of the sums, rows g and
// g + 8 of W at columns 2 t and 2 t + 1 of x.
template <int MT, int WARPS_K, int DEPTH>
__global__ void __launch_bounds__(32 * WARPS_K)
few_kernel(const bf16 *x, long long ldx, const bf16 *w, int M, int N, int K, const Epilogue e)
{
    __shared__ float part[WARPS_K][MT * 4][33];
    chain_start();
    chain_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * 16;
    const bf16 *w0 = w + (long long)min(n0 + g, N - 1) * K + t * 8, *w1 = w + (long long)min(n0 + g + 8, N - 1) * K + t * 8;
    const bf16 *xr[MT];
#pragma unroll
    for (int i = 0; i < MT; i++) xr[i] = x + min(8 * i + g, M - 1) * ldx + t * 8;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    float sum[MT][4] = {}, c[MT][4] = {};
    constexpr int STEP = WARPS_K * DEPTH * 32;
    int count = 0;
    for (int k0 = warp * DEPTH * 32; k0 < K; k0 += STEP) {
        uint4 a[DEPTH][2];
#pragma unroll
        for (int d = 0; d < DEPTH; d++) {
            const int k = k0 + 32 * d;
            a[d][0] = a[d][1] = none;
            if (k + t * 8 < K) {
                a[d][0] = __ldcs(reinterpret_cast<const uint4 *>(w0 + k));
                a[d][1] = __ldcs(reinterpret_cast<const uint4 *>(w1 + k));
            }
        }
#pragma unroll
        for (int d = 0; d < DEPTH; d++) {
            const int k = k0 + 32 * d;
            if (k >= K) break;
#pragma unroll
            for (int i = 0; i < MT; i++) {
                const uint4 b = k + t * 8 < K ? *reinterpret_cast<const uint4 *>(xr[i] + k) : none;
                mma16816(c[i], a[d][0].x, a[d][1].x, a[d][0].y, a[d][1].y, b.x, b.y);
                mma16816(c[i], a[d][0].z, a[d][1].z, a[d][0].w, a[d][1].w, b.z, b.w);
            }
        }
        if (++count * DEPTH == 16) {  // 32 MMAs
            count = 0;
#pragma unroll
            for (int i = 0; i < MT; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    sum[i][j] += c[i][j];
                    c[i][j] = 0.f;
                }
        }
    }
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) part[warp][4 * i + j][lane] = sum[i][j] + c[i][j];
    __syncthreads();
    // 16 neighbouring columns of y of a row of x: 16 threads
    for (int q = threadIdx.x; q < 16 * 8 * MT; q += 32 * WARPS_K) {
        const int n = q & 15, m = q >> 4;                 // output (m, n0 + n)
        const int i = m >> 3, j = (m & 1) + ((n >> 3) << 1), from = ((n & 7) << 2) + ((m & 7) >> 1);
        if (m >= M || n0 + n >= N) continue;
        float s = 0.f;
#pragma unroll
        for (int p = 0; p < WARPS_K; p++) s += part[p][4 * i + j][from];
        finish(e, s, m, n0 + n, N);
    }
}

// 16 warps an SM at least, by more of them on the same rows of W where N is small.
template <int MT, int DEPTH>
static cudaError_t launch_few(const bf16 *x, long long ldx, const bf16 *w, int M, int N, int K, const Epilogue &e, int sms, cudaStream_t st)
{
    const long long tiles = (N + 15LL) / 16;
    const int warps = tiles * 8 >= 16LL * sms ? 8 : tiles * 16 >= 16LL * sms ? 16 : 32;
    auto *kernel = warps == 8 ? few_kernel<MT, 8, DEPTH> : warps == 16 ? few_kernel<MT, 16, DEPTH> : few_kernel<MT, 32, DEPTH>;
    return launch_chained(kernel, dim3((unsigned)tiles), 32 * warps, 0, 1, st, x, ldx, w, M, N, K, e);
}

// ------------------------------------------------------------------ the rest

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

bool small_linear(const csa_linear_params &p)
{
    if (p.dtype == CSA_BF16 && ((p.in_features | p.x_stride) & 7) == 0) return p.rows <= kFewRows;
    return p.rows <= kSmallRows;
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
    if (((K | p.x_stride) & 7) == 0) {
        if (M <= 8) return launch_few<1, 4>((const bf16 *)x, p.x_stride, (const bf16 *)w, M, N, K, e, sms, st);
        return launch_few<2, 2>((const bf16 *)x, p.x_stride, (const bf16 *)w, M, N, K, e, sms, st);
    }
    return launch_rows<bf16, 1>((const bf16 *)x, p.x_stride, (const bf16 *)w, M, N, K, e, sms, st);
}

}  // namespace linear
}  // namespace csa
