// k_vocab_tc.cu -- scores of a vocabulary's columns on tcgen05, reduced where they are made.
//
//   z = alpha x W^T;  for each row and group of 64 columns: the largest z, the sum of exp(z - largest), and for a backward
//   pass exp(z - largest) itself; the z that a row's targets name.
//
// The pipeline is the projections' (k_linear_pipe.cuh): 2 M N K operations on tiles of 256 x 256 by pairs of CTAs, bound by the MMAs.
// The scores themselves never go to memory: a lane holds 64 columns of a row in its registers, which is a group.  Sums
// leave TMEM every 512 k (fp32 values: every 64) and are added up in these registers, rounded: the tensor core cuts a sum off
// at its last place with every 16 k, which would bring 2 to 5e-6 into scores of 2048 to 8192 k, and a loss is a difference of
// scores.  The exponentials of a group are at most 1, so that fp16 holds them to 2^-11 where they count (bf16 to 2^-8; the
// gradient is rounded to bf16 once more).
//
// A row's targets are few columns among many: their list is sorted, and marks say which part of it a group has.  Where a
// lane of a warp has a target, every lane selects one of its 64 registers.
//
// Measured (bf16, 4096 rows, 32768 columns; the bare product with its 268 MB of output takes 93, 152 and 283 us): 512 k 78 us,
// 1024 k 145, 2048 k 274 (tensor pipe 81 to 85 %), 20 to 35 more with 64 candidates a row.  Keeping the exponentials costs
// 24 us: they pass through shared memory, whose bandwidth the MMAs and their loads use up.  (Stored by the lanes themselves: 30.)
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

// v[col] of 64 registers, 0 <= col < 64 (anything else: some of them): every lane its own, in 63 selections
__device__ __forceinline__ float pick(const float (&v)[GROUP], int col)
{
    float r[4];
#pragma unroll
    for (int c = 0; c < 4; c++) {
        float t[8];
#pragma unroll
        for (int k = 0; k < 8; k++) t[k] = col & 1 ? v[16 * c + 2 * k + 1] : v[16 * c + 2 * k];
#pragma unroll
        for (int k = 0; k < 4; k++) t[k] = col & 2 ? t[2 * k + 1] : t[2 * k];
        t[0] = col & 4 ? t[1] : t[0];
        t[1] = col & 4 ? t[3] : t[2];
        r[c] = col & 8 ? t[1] : t[0];
    }
    r[0] = col & 16 ? r[1] : r[0];
    r[1] = col & 16 ? r[3] : r[2];
    return col & 32 ? r[1] : r[0];
}

// DYNAMIC: the device counts the rows.
template <int CG, int BN, int P, int EW, bool DYNAMIC>
__global__ void __launch_bounds__(64 + 32 * EW, 1)
vocab_scores_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_e, const Args args, const Scores s)
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
    __shared__ Args here[1];
    if constexpr (DYNAMIC) {
        if (threadIdx.x == 0) here[0] = counted(args, CG * BM);
        __syncthreads();
    }
    const Args &a = DYNAMIC ? static_cast<const Args &>(here[0]) : args;

    if (warp == 0) {
        p.template produce<true, true, false>(map_x, map_w, map_w, a);
    } else if (warp == 1) {
        p.template issue<true, true>(tmem, a);
    } else {
        const int quad = warp & 3, side = (warp - 2) >> 2;
        const Buffer b = {smem + Z::TURN + (warp - 2) * 4096, lane};
        const float c2 = fabsf(s.alpha) * kLog2e;   // > 0
        // Rows, columns and slots are below 2^31, and so are a tile's ends.
        const int M = (int)a.M, N = (int)a.N;
        const auto place = [&](int u, int &m, int &n0) {   // behind the last unit: none
            m = M;
            n0 = N;
            if (u >= a.units) return;
            const Unit x = unit_of<BN>(a, u);
            m = (x.m * CG + (int)p.rank) * BM + quad * 32 + lane;
            n0 = (int)x.n0 + side * GROUP;
        };
        // A unit's targets of this lane: where they begin and how many they are is asked for a unit ahead, the first while the
        // last unit's scores are reduced.  (Found when their unit came, 64 of 32768 columns cost a product of 4096 x 1024 50 us
        // of 227.)  Both in one register: kernels of 96 of them have few to spare.
        const auto ask_marks = [&](int m, int n0) {
            if (m >= M || n0 >= N) return 0;
            if (s.marks == nullptr) return 1 << 16;
            return __ldg(s.marks + m * (long long)s.groups + n0 / GROUP);
        };
        const auto ask_target = [&](int m, int marks) { return marks >> 16 == 0 ? NONE : __ldg(s.ids + (marks & 0xffff) * s.ld + m); };
        int m, n0;
        place(p.u0, m, n0);
        int marks = ask_marks(m, n0), next = ask_target(m, marks);
        int tc = 0;
        for (int u = p.u0; u < a.units; u += p.ustep) {
            int m_then, n0_then;
            place(u + p.ustep, m_then, n0_then);
            const int marks_then = ask_marks(m_then, n0_then);
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
            // this unit's targets, whose scores are wanted; then the next unit's first is asked for
            int left = marks >> 16, col = next - n0;
            if (s.marks == nullptr && (unsigned)col >= GROUP) left = 0;
            long long at = (marks & 0xffff) * s.ld + m;
            marks = marks_then;
            next = ask_target(m_then, marks);
            const int row = m, m0 = m - lane, col0 = n0;
            m = m_then;
            n0 = n0_then;
            if (m0 >= M || col0 >= N) continue;
            while (__any_sync(0xffffffffu, left > 0)) {
                const float x = pick(v, col);
                if (left > 0) {
                    s.z[at] = s.alpha * x;
                    at += s.ld;
                    if (--left > 0) col = __ldg(s.ids + at) - col0;
                }
            }
            if (s.alpha < 0.f) {
#pragma unroll
                for (int k = 0; k < GROUP; k++) v[k] = -v[k];
            }
            if (N - col0 < GROUP) {   // columns that do not exist
                const int valid = N - col0;
#pragma unroll
                for (int k = 0; k < GROUP; k++)
                    if (k >= valid) v[k] = -INFINITY;
            }
            float top = v[0];
#pragma unroll
            for (int k = 1; k + 1 < GROUP; k += 2) top = fmaxf(top, fmaxf(v[k], v[k + 1]));
            top = fmaxf(top, v[GROUP - 1]);
            top = top == top ? top * c2 : -INFINITY;   // of NaN alone: their sum is NaN
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
            if (row < M) s.parts[col0 / GROUP * args.M + row] = make_float2(top, (sum.x + more.x) + (sum.y + more.y));
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
                    tma_store_3d(&map_e, b.p, col0, m0, 0);
                    bulk_commit();
                }
            } else {
#pragma unroll
                for (int g = 0; g < GROUP; g += C) {
                    float w[C];
#pragma unroll
                    for (int k = 0; k < C; k++) w[k] = v[g + k];
                    if (col0 + g < N) tma_tile<float>(&map_e, w, m0, col0 + g, 0, false, true, b);
                }
            }
        }
        if (lane == 0) bulk_wait();
    }
    p.end(tmem);
}

// ------------------------------------------------------------------ host side

template <int CG, int BN, int P, int EW, bool DYNAMIC>
static cudaError_t launch_one(const Maps &m, const Args &a, const Scores &s, int sms, cudaStream_t st)
{
    using Z = Cfg<CG, BN, P, EW>;
    auto *kernel = vocab_scores_kernel<CG, BN, P, EW, DYNAMIC>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::SMEM);
    if (e != cudaSuccess) return e;
    const int slots = sms / CG;
    return launch_chained(kernel, dim3((unsigned)((a.units < slots ? a.units : slots) * CG)), Z::THREADS, Z::SMEM, CG, st, m.a, m.b, m.out, a, s);
}

template <int CG, int BN, int P, int EW> static cudaError_t launch(const Maps &m, const Args &a, const Scores &s, int sms, cudaStream_t st)
{
    return a.counted != nullptr ? launch_one<CG, BN, P, EW, true>(m, a, s, sms, st) : launch_one<CG, BN, P, EW, false>(m, a, s, sms, st);
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
    a.counted = s.counted;
    a.first = s.first;
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
