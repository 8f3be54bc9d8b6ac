// k_linear.cu -- projections: y = act(alpha x W^T + bias) + residual and its gradients.  This file holds what lies
// around the products: operands made fit for TMA (rows on 16-byte boundaries, fp32 values as three bf16 planes),
// dz = dy act'(z) with the bias gradient, and the join of a split k axis with the epilogue.
#include "k_linear.cuh"
#include "k_rows.cuh"

namespace csa {
namespace linear {

// What holds dz, of values V and gradients O.  fp32 gradients of bf16 values keep 16 bits of it, for twice the MMAs; bf16 ones
// come with 8 bits, and dz has no more.
template <typename V, typename O> struct DzPlanes { static constexpr int N = sizeof(V) == 4 ? 3 : sizeof(O) == 4 ? 2 : 1; };

// Block `b` of up to two operands; a thread makes 8 neighbouring values of a row.
template <typename V> __device__ __forceinline__ void stage_block(const Stage &s0, const Stage &s1, unsigned b)
{
    const Stage &s = b < s0.blocks ? s0 : s1;
    const long long t = (long long)(b - (b < s0.blocks ? 0u : s0.blocks)) * 256 + threadIdx.x;
    const int chunks = (s.cols + 7) / 8;
    const long long r = t <= 0xffffffffLL ? (long long)((uint32_t)t / (uint32_t)chunks) : t / chunks;
    if (r >= s.rows) return;
    const int c = (int)(t - r * chunks) * 8;
    const V *x = static_cast<const V *>(s.x) + r * s.stride + c, *end = static_cast<const V *>(s.x) + (s.rows - 1) * s.stride + s.cols;
    float v[8];
    if (s.aligned && c + 8 <= s.cols) load8<V, true>(x, 8, end, v);
    else load8<V, false>(x, min(8, s.cols - c), end, v);
    put_planes8<Planes<V>::N>(s.out, s.plane, r * s.ld + c, v);
}

template <typename V> __global__ void __launch_bounds__(256) stage_kernel(const Stage s0, const Stage s1)
{
    chain_start();
    chain_wait();
    stage_block<V>(s0, s1, blockIdx.x);
}

// dz = dy act'(z) for `per` rows of a block and 8 TX columns, and their column sums for db.  Bound by memory: dy and
// z are read once, dz is written once, 8 neighbouring columns a thread (VEC: aligned ones), the next row's on their way
// while a row is worked on: bf16 silu of 8192 x 8192 values 62 us (403 MB), db alone 35.  (Two rows loaded and then
// worked on: 79 and 52.)  Blocks behind the `across` x `down` ones stage operands of the products.
// SMOOTH: SiLU or GELU; else ReLU or none.  (One kernel for all of them: db of 8192 x 8192 values with GELU 59 us, two kernels 49 to 57.)
template <typename V, typename O, int TX, bool VEC, bool SMOOTH>
__global__ void __launch_bounds__(256, 4)
dz_kernel(const O *dy, long long ldy, const V *z, int act, bf16 *dz, long long ld, long long plane, float *sums,
          long long M, int N, int per, unsigned across, unsigned down, const Stage s0, const Stage s1)
{
    constexpr int TY = 256 / TX;
    chain_start();
    chain_wait();
    if (blockIdx.x >= across * down) {
        stage_block<V>(s0, s1, blockIdx.x - across * down);
        return;
    }
    const unsigned block_n = blockIdx.x % across, block_m = blockIdx.x / across;
    __shared__ float part[TY][8 * TX + 1];
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    const int n0 = block_n * 8 * TX, n = n0 + 8 * tx, valid = min(8, N - n);
    const long long r0 = (long long)block_m * per, r1 = min(M, r0 + per);
    float s[8] = {};
    if (n < N) {
        Raw8<O, VEC> d0, d1;
        Raw8<V, VEC> z0, z1;
        const auto ask = [&](long long r) {
            if (r >= r1) return;
            d1.load(dy + r * ldy + n, valid, dy + (M - 1) * ldy + N);
            if (SMOOTH || act != CSA_ACT_NONE) z1.load(z + r * N + n, valid, z + M * N);
        };
        ask(r0 + ty);
        for (long long r = r0 + ty; r < r1; r += TY) {
            d0 = d1;
            z0 = z1;
            ask(r + TY);
            float d[8], q[8];
            d0.floats(valid, d);
            if (SMOOTH || act != CSA_ACT_NONE) z0.floats(valid, q);
            if constexpr (SMOOTH) {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float2 g = act_grad2(make_float2(q[j], q[j + 1]), act);
                    d[j] = __fmul_rn(d[j], g.x);  // rounded before it is added, whichever outputs are asked for
                    d[j + 1] = __fmul_rn(d[j + 1], g.y);
                }
            } else if (act == CSA_ACT_RELU) {  // nothing passes where z <= 0, an infinite dy neither
#pragma unroll
                for (int j = 0; j < 8; j++) d[j] = q[j] > 0.f ? d[j] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; j++) s[j] += d[j];
            if (dz != nullptr) put_planes8<DzPlanes<V, O>::N>(dz, plane, r * ld + n, d);  // up to 7 values of padding
        }
    }
    if (sums == nullptr) return;
#pragma unroll
    for (int j = 0; j < 8; j++) part[ty][8 * tx + j] = s[j];
    __syncthreads();
    for (int c = threadIdx.x; c < 8 * TX; c += 256) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < TY; k++) t += part[k][c];
        if (n0 + c < N) sums[(long long)block_m * N + n0 + c] = t;
    }
}

__global__ void __launch_bounds__(1024) db_kernel(const float *sums, int blocks, int N, float *db)
{
    __shared__ float part[32][33];
    chain_start();
    chain_wait();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, n = blockIdx.x * 32 + tx;
    float s = 0.f;
    if (n < N) {
#pragma unroll 8
        for (int b = ty; b < blocks; b += 32) s += sums[(long long)b * N + n];
    }
    part[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && n < N) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 32; k++) t += part[k][tx];
        db[n] = t;
    }
}

// The pieces of a split k axis joined, 4 columns a thread, and the epilogue.  Few outputs take GROUPS warps for each 32 of
// these threads, every one of them a part of the pieces.  VEC: rows of y, preact and the residual hold whole vectors of 4.
template <bool VEC, int GROUPS>
__global__ void __launch_bounds__(256) join_kernel(const float *partial, int splits, long long M, long long N, const Epilogue e)
{
    constexpr int Q = 256 / GROUPS;
    __shared__ float4 part[GROUPS == 1 ? 1 : GROUPS][GROUPS == 1 ? 1 : Q];
    chain_start();
    chain_wait();
    const int q = threadIdx.x % Q, group = threadIdx.x / Q;
    const long long ldp = partial_stride(N), t = (long long)blockIdx.x * Q + q;
    const long long m = t / (ldp / 4), n = (t - m * (ldp / 4)) * 4;
    const bool live = m < M && n < N;
    float v[4] = {};
    if (live) {
#pragma unroll 4
        for (int s = group; s < splits; s += GROUPS) {
            const float4 x = __ldcs(reinterpret_cast<const float4 *>(partial + (s * M + m) * ldp + n));
            v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        }
    }
    if constexpr (GROUPS > 1) {
        part[group][q] = make_float4(v[0], v[1], v[2], v[3]);
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g = 1; g < GROUPS; g++) {
            const float4 x = part[g][q];
            v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        }
    }
    if (!live) return;
    const long long i = m * N + n;
    const float alpha = e.factor();
    float z[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        z[k] = alpha * v[k] + (e.bias != nullptr && n + k < N ? __ldg(e.bias + n + k) : 0.f);
        v[k] = act_fwd(z[k], e.act);
        if (e.res != nullptr && n + k < N)
            v[k] += e.out_f32 ? ((const float *)e.res)[m * e.ldr + n + k] : __bfloat162float(((const bf16 *)e.res)[m * e.ldr + n + k]);
    }
    const auto put = [&](void *out, bool f32, const float (&x)[4]) {
        if constexpr (VEC) {
            if (f32) {
                *reinterpret_cast<float4 *>((float *)out + i) = make_float4(x[0], x[1], x[2], x[3]);
            } else {
                const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
                *reinterpret_cast<uint2 *>((bf16 *)out + i) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; k++) {
                if (n + k >= N) break;
                if (f32) ((float *)out)[i + k] = x[k];
                else ((bf16 *)out)[i + k] = __float2bfloat16_rn(x[k]);
            }
        }
    };
    if (e.preact != nullptr) put(e.preact, e.preact_f32, z);
    put(e.out, e.out_f32, v);
}

// ------------------------------------------------------------------ host side

inline int planes_of(const csa_linear_params &p) { return p.dtype == CSA_F32 ? 3 : 1; }
inline int dz_passes(const csa_linear_params &p) { return p.dtype == CSA_BF16 && p.out_dtype == CSA_F32 ? 2 : 1; }

struct Fwd {
    bool stage_x, stage_w;
    linear::Plan plan;
    size_t off_x, off_w, off_part, total;
};
Fwd plan_fwd(const csa_linear_params &p)
{
    Fwd f = {};
    if (small_linear(p)) return f;
    const long long M = p.rows, K = p.in_features, N = p.out_features;
    f.stage_x = staged(p.dtype, p.x_stride);
    f.stage_w = staged(p.dtype, K);
    size_t at = 0;
    f.off_x = at;
    if (f.stage_x) at += staged_bytes(p.dtype, M, K);
    f.off_w = at;
    if (f.stage_w) at += staged_bytes(p.dtype, N, K);
    f.plan = plan_product(M, N, K, planes_of(p), 1, p.out_dtype == CSA_F32, kSms);
    f.off_part = at;
    if (f.plan.splits > 1) at += up256((size_t)f.plan.splits * M * partial_stride(N) * 4);
    f.total = at;
    return f;
}

// Every part that some choice of outputs needs: the workspace does not depend on which are asked for.
struct Bwd {
    bool stage_x, stage_w, stage_dz;
    linear::Plan dx, dw;
    int per, blocks;
    size_t off_x, off_w, off_dz, off_sums, off_part, total;
};
Bwd plan_bwd(const csa_linear_params &p)
{
    Bwd b = {};
    const long long M = p.rows, K = p.in_features, N = p.out_features;
    if (M == 0) return b;
    b.stage_x = staged(p.dtype, p.x_stride);
    b.stage_w = staged(p.dtype, K);
    b.stage_dz = p.activation != CSA_ACT_NONE || p.dtype != p.out_dtype || staged(p.dtype, p.dy_stride);
    // rows of a block of dz_kernel: enough blocks to fill the GPU twice, a row of each thread at least
    const long long cols = N <= 64 ? 1 : (N + 255) / 256, least = N <= 64 ? 32 : 8;
    const long long want = 8 * kSms;
    long long per = (M * cols + want - 1) / want;
    if (per < least) per = least;
    b.per = (int)(per < M ? per : M);
    b.blocks = (int)((M + b.per - 1) / b.per);
    size_t at = 0;
    b.off_x = at;
    if (b.stage_x) at += staged_bytes(p.dtype, M, K);
    b.off_w = at;
    if (b.stage_w) at += staged_bytes(p.dtype, N, K);
    b.off_dz = at;
    if (b.stage_dz) at += staged_bytes(p.dtype, M, N) * dz_passes(p);
    b.off_sums = at;
    at += up256((size_t)b.blocks * N * 4);
    b.off_part = at;
    b.dx = plan_product(M, K, N, planes_of(p), dz_passes(p), p.dtype == CSA_F32, kSms);
    b.dw = plan_product(N, K, M, planes_of(p), dz_passes(p), p.dtype == CSA_F32, kSms);
    const size_t dx = b.dx.splits > 1 ? (size_t)b.dx.splits * M * partial_stride(K) * 4 : 0;
    const size_t dw = b.dw.splits > 1 ? (size_t)b.dw.splits * N * partial_stride(K) * 4 : 0;
    at += up256(dx > dw ? dx : dw);  // one product after the other
    b.total = at;
    return b;
}

Operand operand(int dtype, const void *x, long long stride, long long rows, int cols, bool stage, void *to, bool k_major,
                Stage *job)
{
    Operand o = {};
    o.k_major = k_major;
    if (!stage) {
        o.base = static_cast<const bf16 *>(x);
        o.ld = stride;
        o.plane = 0;
        return o;
    }
    o.base = static_cast<bf16 *>(to);
    o.ld = up8(cols);
    o.plane = rows * o.ld;
    job->x = x;
    job->out = static_cast<bf16 *>(to);
    job->stride = stride;
    job->rows = rows;
    job->ld = o.ld;
    job->plane = o.plane;
    job->cols = cols;
    job->aligned = stride % (dtype == CSA_F32 ? 4 : 8) == 0;
    job->blocks = (unsigned)((rows * ((cols + 7) / 8) + 255) / 256);
    return o;
}

cudaError_t run_stages(int dtype, const Stage (&job)[2], cudaStream_t st)
{
    const unsigned blocks = job[0].blocks + job[1].blocks;
    if (blocks == 0) return cudaSuccess;
    return launch_chained(dtype == CSA_F32 ? stage_kernel<float> : stage_kernel<bf16>, dim3(blocks), 256, 0, 1, st, job[0], job[1]);
}

cudaError_t product(const Product &p, cudaStream_t st)
{
    // The persistent kernel deals its units to the SMs that are there: CTAs beyond them would start when the first have
    // finished their whole share.
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = (p.counted != nullptr ? launch_product_counted : launch_product_tc)(p, sms > 2 ? sms : 2, st);
    if (e != cudaSuccess || p.plan.splits == 1) return e;
    // Too few whole sums to fill the GPU: cut them (the backward of 15401 x 48 x 24, dW from 61 pieces: 28.9 -> 17.0 us).
    const long long threads = p.M * (partial_stride(p.N) / 4);
    const bool vec = p.N % 4 == 0, cut = threads <= 256LL * kSms && p.plan.splits >= 4;
    auto *kernel = cut ? (vec ? join_kernel<true, 8> : join_kernel<false, 8>) : vec ? join_kernel<true, 1> : join_kernel<false, 1>;
    const unsigned each = cut ? 32 : 256;
    return launch_chained(kernel, dim3((unsigned)((threads + each - 1) / each)), 256, 0, 1, st, p.e.partial, p.plan.splits, p.M, p.N, p.e);
}

template <typename V, typename O, int TX, bool VEC, bool SMOOTH>
cudaError_t run_dz_rows(const csa_linear_params &p, const Bwd &b, const void *dy, const void *z, bf16 *dz, float *sums,
                        const Stage (&job)[2], cudaStream_t st)
{
    const int N = p.out_features;
    const long long ld = up8(N), plane = p.rows * ld;
    const unsigned across = (N + 8 * TX - 1) / (8 * TX), down = b.blocks;
    return launch_chained(dz_kernel<V, O, TX, VEC, SMOOTH>, dim3(across * down + job[0].blocks + job[1].blocks), 256, 0, 1, st, (const O *)dy,
                          p.dy_stride, (const V *)z, p.activation, dz, ld, plane, sums, p.rows, N, b.per, across, down, job[0], job[1]);
}

template <typename V, typename O, bool SMOOTH>
cudaError_t run_dz_act(const csa_linear_params &p, const Bwd &b, const void *dy, const void *z, bf16 *dz, float *sums,
                       const Stage (&job)[2], cudaStream_t st)
{
    const bool vec = (p.out_features & 7) == 0 && (p.dy_stride & 7) == 0;
    auto *run = p.out_features <= 64 ? (vec ? run_dz_rows<V, O, 8, true, SMOOTH> : run_dz_rows<V, O, 8, false, SMOOTH>)
                                     : (vec ? run_dz_rows<V, O, 32, true, SMOOTH> : run_dz_rows<V, O, 32, false, SMOOTH>);
    return run(p, b, dy, z, dz, sums, job, st);
}

template <typename V, typename O>
cudaError_t run_dz(const csa_linear_params &p, const Bwd &b, const void *dy, const void *z, bf16 *dz, float *sums, const Stage (&job)[2],
                   cudaStream_t st)
{
    const bool smooth = p.activation == CSA_ACT_SILU || p.activation == CSA_ACT_GELU_TANH;
    return (smooth ? run_dz_act<V, O, true> : run_dz_act<V, O, false>)(p, b, dy, z, dz, sums, job, st);
}

}  // namespace linear

using namespace linear;

size_t linear_fwd_workspace(const csa_linear_params &p) { return plan_fwd(p).total; }
size_t linear_bwd_workspace(const csa_linear_params &p) { return plan_bwd(p).total; }

#define LIN_TRY(x)                            \
    do {                                      \
        const cudaError_t e_ = (x);           \
        if (e_ != cudaSuccess) return e_;     \
    } while (0)

cudaError_t launch_linear_fwd(const csa_linear_params &p, const void *x, const void *weight, const float *bias,
                              const void *residual, void *y, void *preact, void *ws, cudaStream_t st)
{
    Product q = {};
    q.e.alpha = p.alpha;
    q.e.act = p.activation;
    q.e.bias = bias;
    q.e.res = residual;
    q.e.ldr = p.residual_stride;
    q.e.out = y;
    q.e.preact = preact;
    q.e.out_f32 = p.out_dtype == CSA_F32;
    q.e.preact_f32 = p.dtype == CSA_F32;
    if (small_linear(p)) {
        note_path("generic");
        return launch_linear_small(p, x, weight, q.e, kSms, st);
    }
    note_path("tcgen05");
    const Fwd f = plan_fwd(p);
    char *w = static_cast<char *>(ws);
    Stage job[2] = {};
    q.a = operand(p.dtype, x, p.x_stride, p.rows, p.in_features, f.stage_x, w + f.off_x, true, &job[0]);
    q.b = operand(p.dtype, weight, p.in_features, p.out_features, p.in_features, f.stage_w, w + f.off_w, true, &job[1]);
    LIN_TRY(run_stages(p.dtype, job, st));
    q.M = p.rows;
    q.N = p.out_features;
    q.K = p.in_features;
    q.planes = planes_of(p);
    q.passes = 1;
    q.plan = f.plan;
    q.e.partial = reinterpret_cast<float *>(w + f.off_part);
    return product(q, st);
}

cudaError_t launch_linear_bwd(const csa_linear_params &p, const void *dy, const void *x, const void *weight,
                              const void *preact, void *dx, void *dw, float *db, void *ws, cudaStream_t st)
{
    note_path("tcgen05");
    const long long M = p.rows, K = p.in_features, N = p.out_features;
    if (M == 0) {  // sums of nothing
        if (dw != nullptr) LIN_TRY(cudaMemsetAsync(dw, 0, (size_t)N * K * (p.dtype == CSA_F32 ? 4 : 2), st));
        if (db != nullptr) LIN_TRY(cudaMemsetAsync(db, 0, (size_t)N * 4, st));
        return cudaSuccess;
    }
    const Bwd b = plan_bwd(p);
    char *w = static_cast<char *>(ws);
    bf16 *dz = b.stage_dz && (dx != nullptr || dw != nullptr) ? reinterpret_cast<bf16 *>(w + b.off_dz) : nullptr;
    float *sums = db != nullptr ? reinterpret_cast<float *>(w + b.off_sums) : nullptr;
    Stage job[2] = {};
    Operand ow = {}, ox = {};
    if (dx != nullptr) ow = operand(p.dtype, weight, K, N, (int)K, b.stage_w, w + b.off_w, false, &job[0]);
    if (dw != nullptr) ox = operand(p.dtype, x, p.x_stride, M, (int)K, b.stage_x, w + b.off_x, false, &job[1]);
    // A few staged blocks join dz's launch (1013 x 1023 x 777 in fp32: 47.1 -> 43.8 us); many have their own, with
    // twice the warps an SM (62578 x 684 x 585 in bf16: 204 us, joined 213).
    const bool any_dz = dz != nullptr || sums != nullptr;
    if (!any_dz || job[0].blocks + job[1].blocks > 16u * kSms) {
        LIN_TRY(run_stages(p.dtype, job, st));
        job[0].blocks = job[1].blocks = 0;
    }
    if (any_dz) {
        auto *run = p.dtype == CSA_F32 ? run_dz<float, float> : p.out_dtype == CSA_F32 ? run_dz<bf16, float> : run_dz<bf16, bf16>;
        LIN_TRY(run(p, b, dy, preact, dz, sums, job, st));
    }
    if (db != nullptr) {
        LIN_TRY(launch_chained(db_kernel, dim3((p.out_features + 31) / 32), 1024, 0, 1, st, sums, b.blocks, p.out_features, db));
    }
    Operand d = {};
    d.base = dz != nullptr ? dz : static_cast<const bf16 *>(dy);
    d.ld = dz != nullptr ? up8(N) : p.dy_stride;
    d.plane = dz != nullptr ? M * up8(N) : 0;
    Product q = {};
    q.planes = planes_of(p);
    q.passes = dz_passes(p);
    q.e.alpha = p.alpha;
    q.e.out_f32 = p.dtype == CSA_F32;
    q.e.partial = reinterpret_cast<float *>(w + b.off_part);
    if (dx != nullptr) {
        q.a = d;
        q.a.k_major = true;
        q.b = ow;
        q.M = M;
        q.N = K;
        q.K = N;
        q.plan = b.dx;
        q.e.out = dx;
        LIN_TRY(product(q, st));
    }
    if (dw != nullptr) {
        q.a = d;
        q.a.k_major = false;
        q.b = ox;
        q.M = N;
        q.N = K;
        q.K = M;
        q.plan = b.dw;
        q.e.out = dw;
        LIN_TRY(product(q, st));
    }
    return cudaSuccess;
}

}  // namespace csa
