// k_vocab_tc.cu -- scores of a vocabulary's columns on tcgen05, reduced where they are made.
//
//   z = alpha x W^T;  for each row and group of 64 columns: the largest z, the sum of exp(z - largest), and for a backward
//   pass exp(z - largest) itself; the z that a row's targets name.
//
// The pipeline is the projections' (k_linear_pipe.cuh): 2 M N K operations on tiles of 256 x 256 by pairs of CTAs, bound by the MMAs.
// The scores themselves never go to memory: a lane holds 64 columns of a row in its registers, which is a group.  Sums
// leave TMEM every 512 k (fp32 values: every 64) and are added up in these registers, rounded: the tensor core cuts a sum off
// at its last place with every 16 k, which would bring 2 to 5e-6 into scores of 2048 to 8192 k, and a loss is a difference of
// scores.  The exponentials of a group are at most 1, so that fp16 holds them to 2^-12 where they count (bf16 to 2^-9; the
// gradient is rounded to bf16 once more).
//
// A row's targets are few columns among many: their list is sorted, each lane finds its group's part of it before the
// sums are there, and looks for the columns only where a lane of its warp has one.
#include "k_linear_pipe.cuh"
#include "k_vocab.cuh"

#include <cuda_fp16.h>

namespace csa {

static __device__ int g_vocab_error = 0;

cudaError_t vocab_tc_read_clear_error(int *flag)
{
    *flag = 0;
    cudaError_t e = cudaMemcpyFromSymbol(flag, g_vocab_error, sizeof(int));
    if (e == cudaSuccess && *flag != 0) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_vocab_error, &zero, sizeof(int));
    }
    return e;
}

namespace vocab {

using namespace linear;

constexpr int CHUNK_SUMS = 8;   // stages (512 k) that an accumulator of one plane sums

// 16 consecutive fp32 columns of this thread's TMEM lane (warp-collective), waited.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int CG, int BN, int P, int EW>
__global__ void __launch_bounds__(64 + 32 * EW, 1)
vocab_scores_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_e, const Args a, const Scores s)
{
    using Z = Cfg<CG, BN, P, EW>;
    constexpr int CHUNK = P == 3 ? 1 : CHUNK_SUMS;
    static_assert(BN / (EW / 4) == GROUP, "a warp has 32 rows of a group");
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_align1024(smem_raw);
    const Pipeline<CG, BN, P, EW, CHUNK> p(smem, &g_vocab_error, 700);
    const int warp = p.warp, lane = p.lane;
    chain_start();
    const uint32_t tmem = p.begin();
    chain_wait();

    if (warp == 0) {
        p.template produce<true, true, false>(map_x, map_w, map_w, a);
    } else if (warp == 1) {
        p.template issue<true, true>(tmem, a);
    } else {
        const int quad = warp & 3, side = (warp - 2) >> 2;
        const Buffer b = {smem + Z::TURN + (warp - 2) * 4096, lane};
        const float c2 = s.alpha * kLog2e;
        int tc = 0;
        for (int u = p.u0; u < a.units; u += p.ustep) {
            const Unit x = unit_of<BN>(a, u);
            const long long m0 = ((long long)x.m * CG + p.rank) * BM + quad * 32, m = m0 + lane, n0 = x.n0 + side * GROUP;
            // the row's first target from n0 on
            int at = 0, next = NONE;
            if (m < a.M && n0 < a.N) {
                for (int end = s.slots; at < end;) {
                    const int mid = (at + end) >> 1;
                    if (__ldg(s.ids + mid * s.ld + m) < n0) at = mid + 1;
                    else end = mid;
                }
                if (at < s.slots) next = __ldg(s.ids + at * s.ld + m);
            }
            float v[GROUP] = {};
            for (int it = 0; it < a.ksteps; it += CHUNK, tc++) {
                p.wait_sums(tc);
                const uint32_t t = tmem + (uint32_t)((tc & 1) * BN + side * GROUP) + ((uint32_t)(quad * 32) << 16);
#pragma unroll
                for (int g = 0; g < GROUP; g += 16) {
                    float w[16];
                    tmem_ld16(t + g, w);
                    if (g + 16 == GROUP) p.release_sums(tc);
#pragma unroll
                    for (int k = 0; k < 16; k++) v[g + k] += w[k];
                }
            }
            if (m0 >= a.M || n0 >= a.N) continue;
            if (__any_sync(0xffffffffu, next < n0 + GROUP)) {
#pragma unroll
                for (int k = 0; k < GROUP; k++) {
                    while (next == n0 + k) {   // a column may be named more than once
                        s.z[at * s.ld + m] = s.alpha * v[k];
                        next = ++at < s.slots ? __ldg(s.ids + at * s.ld + m) : NONE;
                    }
                }
            }
            if (n0 + GROUP > a.N) {   // columns that do not exist
                const int valid = (int)(a.N - n0);
                const float none = c2 < 0.f ? INFINITY : -INFINITY;
#pragma unroll
                for (int k = 0; k < GROUP; k++)
                    if (k >= valid) v[k] = none;
            }
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < GROUP; k++) top = fmaxf(top, v[k] * c2);
            const float ref = top == -INFINITY ? 0.f : top;
            float2 sum = make_float2(0.f, 0.f), more = sum;
#pragma unroll
            for (int k = 0; k < GROUP; k += 4) {
                const float2 y = fma2(make_float2(v[k], v[k + 1]), make_float2(c2, c2), make_float2(-ref, -ref));
                const float2 z = fma2(make_float2(v[k + 2], v[k + 3]), make_float2(c2, c2), make_float2(-ref, -ref));
                v[k] = ex2(y.x);
                v[k + 1] = ex2(y.y);
                v[k + 2] = ex2(z.x);
                v[k + 3] = ex2(z.y);
                sum = add2(sum, make_float2(v[k], v[k + 1]));
                more = add2(more, make_float2(v[k + 2], v[k + 3]));
            }
            if (m < a.M) s.parts[n0 / GROUP * a.M + m] = make_float2(top, (sum.x + more.x) + (sum.y + more.y));
            if (s.e == nullptr) continue;
            if constexpr (P == 1) {
                if (lane == 0) bulk_wait_read();   // the last group has left the buffer
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const __half2 q = __floats2half2_rn(v[8 * k + 2 * j], v[8 * k + 2 * j + 1]);
                        h[j] = *reinterpret_cast<const uint32_t *>(&q);
                    }
                    *reinterpret_cast<uint4 *>(b.p + lane * 128 + ((k ^ (lane & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&map_e, b.p, (int)n0, (int)m0, 0);
                    bulk_commit();
                }
            } else {
#pragma unroll
                for (int g = 0; g < GROUP; g += C) {
                    float w[C];
#pragma unroll
                    for (int k = 0; k < C; k++) w[k] = v[g + k];
                    if (n0 + g < a.N) tma_tile<float>(&map_e, w, m0, n0 + g, 0, false, true, b);
                }
            }
        }
        if (lane == 0) bulk_wait();
    }
    p.end(tmem);
}

// ------------------------------------------------------------------ host side

template <int CG, int BN, int P, int EW>
static cudaError_t launch(const Maps &m, const Args &a, const Scores &s, int sms, cudaStream_t st)
{
    using Z = Cfg<CG, BN, P, EW>;
    auto *kernel = vocab_scores_kernel<CG, BN, P, EW>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::SMEM);
    if (e != cudaSuccess) return e;
    const int slots = sms / CG;
    return launch_chained(kernel, dim3((unsigned)((a.units < slots ? a.units : slots) * CG)), Z::THREADS, Z::SMEM, CG, st, m.a, m.b, m.out, a, s);
}

// The tile by estimated time: the projections' model of a stage, a round no shorter than its epilogue.
static Shape plan_scores(long long M, long long N, long long K, int planes, int sms)
{
    const double steps = (double)((K + BK - 1) / BK);
    Shape best = PAIR_128;
    double least = 1e300;
    for (int i = LONE_64; i <= (planes == 3 ? PAIR_128 : PAIR_256); i++) {
        int mt, nt;
        tile_counts((Shape)i, M, N, mt, nt);
        const double slots = i == LONE_64 ? sms : sms / 2, rounds = ceil((double)mt * nt / slots);
        constexpr double STEP[2][3] = {{0.20, 0.20, 0.28}, {0.72, 0.90, 0.0}}, FIXED[3] = {3.8, 5.2, 6.3}, EPILOGUE[3] = {0.9, 1.7, 2.5};
        const double us = rounds * fmax(steps * STEP[planes == 3][i], EPILOGUE[i]) + FIXED[i];
        if (us < least) {
            least = us;
            best = (Shape)i;
        }
    }
    return best;
}

cudaError_t launch_scores(const Operand &x, const Operand &w, long long M, long long N, long long K, int planes, const Scores &s, int sms,
                          cudaStream_t st)
{
    const Shape shape = plan_scores(M, N, K, planes, sms);
    Args a = {};
    a.M = M;
    a.N = N;
    a.ksteps = a.per_split = (int)((K + BK - 1) / BK);
    a.splits = 1;
    tile_counts(shape, M, N, a.mt, a.nt);
    const long long units = (long long)a.mt * a.nt;
    if (units > 0x3fffffffLL || (long long)BAND * a.nt > 0x3fffffffLL) return cudaErrorInvalidConfiguration;
    a.units = a.whole = (int)units;
    a.rows_a = M >= BM ? BM : (int)((M + 7) & ~7LL);
    Maps m = {};
    bool ok = encode(&m.a, x, M, K, planes, a.rows_a, false) && encode(&m.b, w, N, K, planes, shape == PAIR_256 ? 128 : 64, false);
    if (s.e != nullptr) ok = ok && encode_out(&m.out, planes == 3, s.e, N, s.lde, M, 1);
    if (!ok) return cudaErrorInvalidValue;
    if (planes == 3) return shape == LONE_64 ? launch<1, 64, 3, 4>(m, a, s, sms, st) : launch<2, 128, 3, 8>(m, a, s, sms, st);
    if (shape == LONE_64) return launch<1, 64, 1, 4>(m, a, s, sms, st);
    if (shape == PAIR_128) return launch<2, 128, 1, 8>(m, a, s, sms, st);
    return launch<2, 256, 1, 16>(m, a, s, sms, st);
}

}  // namespace vocab
}  // namespace csa
