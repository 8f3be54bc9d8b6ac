// k_linear_tc.cu -- the projections' products on the 5th-generation tensor cores (tcgen05 + TMEM + TMA).
//
// D[m][n] = sum_k A(m, k) B(n, k) with bf16 operands and fp32 sums, for y = x W^T (both operands contiguous along
// k), dx = dz W (B contiguous along n) and dW = dz^T x (both contiguous along m, n): the shared-memory descriptors
// take either order, so no operand is transposed in memory.  fp32 values come as three bf16 planes and take six
// passes over k, (l h) (h l) (m m) (m h) (h m) (h h), the smallest terms first; what is left out is below 2^-23 of
// the terms.
//
// Mapping.  A unit is one output tile and one piece of the k axis.  A CTA pair (two SMs) computes 256 x BN: each CTA
// loads its 128 rows of A and its BN / 2 rows of B, so an operand byte brought to an SM feeds twice the MMAs of a
// lone CTA's 128 x BN tile.  Small M takes lone CTAs with 128 x 64 tiles (more of them, for the memory's sake).
// Roles: warp 0 the TMA producer, warp 1 the MMA issue (the pair's even CTA), warps 2..9 the epilogue, a row
// a lane, whose 32 x 32 tiles go out through shared memory by TMA.  TMEM holds two accumulators, so that a
// tile's epilogue runs under the next tile's MMAs.  Persistent: one CTA per SM, units
// dealt round-robin in an order that keeps the running tiles' operands in L2.
//
// Every mbarrier wait is bounded (see tc_ptx.cuh); site codes 600 + n.
#include "csa_tc.cuh"
#include "k_linear.cuh"
#include "tc_ptx.cuh"

#include <cuda.h>
#include <string.h>

namespace csa {

static __device__ int g_lin_error = 0;

cudaError_t linear_tc_read_clear_error(int *flag)
{
    *flag = 0;
    cudaError_t e = cudaMemcpyFromSymbol(flag, g_lin_error, sizeof(int));
    if (e == cudaSuccess && *flag != 0) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_lin_error, &zero, sizeof(int));
    }
    return e;
}

namespace linear {

using namespace ptx;

constexpr int BM = 128;        // rows of one CTA's accumulator
constexpr int BK = 64;         // k per stage: one 128-byte swizzle row
constexpr int THREADS = 320;
constexpr int EPI_WARPS = 8;

template <int CG, int BN> struct Cfg {
    static constexpr int ROWS_B = BN / CG;                      // B rows this CTA loads
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = ROWS_B * BK * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = STAGE == 32768 ? 6 : 8;       // 192 KB
    static constexpr int TURN = STAGES * STAGE;                 // a warp's 32 x 32 fp32 tile each, for the epilogue
    static constexpr int MISC = TURN + EPI_WARPS * 4096;
    static constexpr int SMEM = MISC + 512 + 1024;              // + alignment
    static constexpr int TMEM = 2 * BN < 512 ? (2 * BN < 128 ? 128 : 2 * BN) : 512;
};

struct Args {
    long long M, N;
    int ksteps;                 // stages of one plane pair over the whole k axis
    int passes;                 // plane pairs: 1 or 6
    int splits, per_split;      // k pieces, stages (over passes * ksteps) of each
    int mt, nt;                 // tiles
    long long whole, units;     // units that are whole tiles (times splits); the rest are halves of the last tiles
    int tma_out;                // the outputs' rows lie on 16-byte boundaries: the epilogue stores by TMA
    Epilogue e;
};

struct Unit {
    int m, s, it0, it1;
    int bn;                     // columns: BN, or BN / 2 for half a tile
    long long n0;               // first column
};

// Tiles in bands of 8 along m, m fastest: the tiles that run together share a few rows of A tiles and a few of B.
// When the last round of whole tiles would leave half of the SMs idle or more, its tiles are cut in two along n.
constexpr int BAND = 8;
template <int BN> __device__ __forceinline__ Unit unit_of(const Args &a, long long u)
{
    Unit x;
    const long long tiles = (long long)a.mt * a.nt;
    long long t;
    int half = 0;
    x.bn = BN;
    x.s = 0;
    if (u < a.whole) {
        if (a.splits > 1) {
            x.s = (int)(u / tiles);
            t = u - x.s * tiles;
        } else {
            t = u;
        }
    } else {
        t = a.whole + ((u - a.whole) >> 1);
        half = (int)((u - a.whole) & 1);
        x.bn = BN / 2;
    }
    const long long per_band = (long long)BAND * a.nt;
    const int band = (int)(t / per_band);
    const int r = (int)(t - band * per_band);
    const int h = min(BAND, a.mt - band * BAND);
    x.m = band * BAND + r % h;
    x.n0 = (long long)(r / h) * BN + half * (BN / 2);
    x.it0 = x.s * a.per_split;
    x.it1 = min(a.passes * a.ksteps, x.it0 + a.per_split);
    return x;
}

// The plane pair of pass q, smallest terms first.
__device__ __forceinline__ void planes_of(int passes, int q, int &pa, int &pb)
{
    if (passes == 1) {
        pa = pb = 0;
        return;
    }
    pa = (0x001102 >> (4 * q)) & 3;   // l h m m h h
    pb = (0x010120 >> (4 * q)) & 3;   // h l m h m h
}

// ------------------------------------------------------------------ epilogue: 32 rows x 32 columns of a warp

// A lane's 32 neighbouring columns of one row of the residual, asked for before the sums are there.
struct Residual {
    uint4 r[8];
    template <typename O> __device__ __forceinline__ void load(const Args &a, long long m, long long n0)
    {
        constexpr int E = 16 / sizeof(O);   // values of a vector
        const O *p = (const O *)a.e.res + m * a.e.ldr + n0;
        if (a.e.ldr % E == 0 && n0 + 32 <= a.N) {
#pragma unroll
            for (int k = 0; k < 32 / E; k++) r[k] = __ldcs(reinterpret_cast<const uint4 *>(p) + k);
        } else {
            O v[32];
#pragma unroll
            for (int k = 0; k < 32; k++) v[k] = n0 + k < a.N ? p[k] : from_f<O>(0.f);
#pragma unroll
            for (int k = 0; k < 32 / E; k++) r[k] = *reinterpret_cast<const uint4 *>(v + E * k);
        }
    }
    template <typename O> __device__ __forceinline__ void add_to(float (&v)[32]) const
    {
#pragma unroll
        for (int k = 0; k < (int)(2 * sizeof(O)); k++) {
            const uint32_t w[4] = {r[k].x, r[k].y, r[k].z, r[k].w};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if constexpr (sizeof(O) == 2) {
                    v[8 * k + 2 * j] += __uint_as_float(w[j] << 16);
                    v[8 * k + 2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
                } else {
                    v[4 * k + j] += __uint_as_float(w[j]);
                }
            }
        }
    }
};

template <int ACT> __device__ __forceinline__ void activate(float (&v)[32])
{
#pragma unroll
    for (int k = 0; k < 32; k++) v[k] = act_fwd<ACT>(v[k]);
}

// Where a warp puts a tile: 4 KB of shared memory, a whole fp32 tile or two bf16 ones in turn, from where TMA stores it.
struct Store {
    unsigned char *buf;
    int lane, turn;
    bool two;          // both halves of buf are in use: only bf16 tiles

    template <typename O> __device__ __forceinline__ void tile(const Args &a, const CUtensorMap *map, const float (&v)[32], long long m0,
                                                               long long n0, int z, O *out, long long ld)
    {
        if (a.tma_out) {
            if (lane == 0) {  // the half's last store has been read
                if (two) bulk_wait_read<1>();
                else bulk_wait_read<0>();
            }
            __syncwarp();
            unsigned char *b = buf + (two ? (turn & 1) * 2048 : 0);
            turn++;
            if constexpr (sizeof(O) == 2) {
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * k + 2 * j], v[8 * k + 2 * j + 1]);
                        w[j] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    *reinterpret_cast<uint4 *>(b + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; k++)
                    *reinterpret_cast<float4 *>(b + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                        make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                if (m0 < a.M && n0 < a.N) tma_store_3d(map, b, (int)n0, (int)m0, z);
                bulk_commit();
            }
        } else {
            // rows at any place: turned in shared memory so that a warp writes 32 neighbouring values at a time
            float *t = reinterpret_cast<float *>(buf);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 32; k++) t[lane * 32 + ((k + lane) & 31)] = v[k];
            __syncwarp();
            if (n0 + lane < a.N) {
#pragma unroll 8
                for (int r = 0; r < 32; r++)
                    if (m0 + r < a.M) out[(m0 + r) * ld + n0 + lane] = from_f<O>(t[r * 32 + ((lane + r) & 31)]);
            }
        }
    }
};

// From sums to the output: z = alpha sum + bias, kept if asked for; act(z) + res.
template <typename O>
__device__ __forceinline__ void finish(const Args &a, const CUtensorMap *map_out, const CUtensorMap *map_pre, Store &st, float (&v)[32],
                                       const Residual &res, long long m0, long long n0)
{
    const Epilogue &e = a.e;
    if (e.bias != nullptr) {
        if (n0 + 32 <= a.N) {
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const float4 b = __ldg(reinterpret_cast<const float4 *>(e.bias + n0) + k);
                v[4 * k] = fmaf(e.alpha, v[4 * k], b.x);
                v[4 * k + 1] = fmaf(e.alpha, v[4 * k + 1], b.y);
                v[4 * k + 2] = fmaf(e.alpha, v[4 * k + 2], b.z);
                v[4 * k + 3] = fmaf(e.alpha, v[4 * k + 3], b.w);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 32; k++) v[k] = fmaf(e.alpha, v[k], n0 + k < a.N ? __ldg(e.bias + n0 + k) : 0.f);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 32; k++) v[k] *= e.alpha;
    }
    if (e.preact != nullptr) {
        if (e.preact_f32) st.tile<float>(a, map_pre, v, m0, n0, 0, (float *)e.preact, a.N);
        else st.tile<__nv_bfloat16>(a, map_pre, v, m0, n0, 0, (__nv_bfloat16 *)e.preact, a.N);
    }
    if (e.act == CSA_ACT_RELU) activate<CSA_ACT_RELU>(v);
    else if (e.act == CSA_ACT_SILU) activate<CSA_ACT_SILU>(v);
    else if (e.act == CSA_ACT_GELU_TANH) activate<CSA_ACT_GELU_TANH>(v);
    if (e.res != nullptr) res.add_to<O>(v);
    st.tile<O>(a, map_out, v, m0, n0, 0, (O *)e.out, a.N);
}

template <int CG, int BN, bool A_K, bool B_K>
__global__ void __launch_bounds__(THREADS, 1)
linear_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_pre, const Args a)
{
    using C = Cfg<CG, BN>;
    constexpr int S = C::STAGES;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_align1024(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::MISC);
    uint64_t *full = bars, *empty = bars + S, *t_full = bars + 2 * S, *t_empty = bars + 2 * S + 2, *done = bars + 2 * S + 4;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::MISC + 256);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::MISC + 264);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
    const long long u0 = blockIdx.x / CG, ustep = gridDim.x / CG;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; i++) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(t_full + i, 1);
            mbar_init(t_empty + i, EPI_WARPS * CG);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        init_fence();
    }
    if (warp == 1) {
        if constexpr (CG == 2) tmem_alloc_pair(tmem_slot, C::TMEM);
        else tmem_alloc(tmem_slot, C::TMEM);
    }
    fence_before();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---------------------------------------------------------- TMA producer
        if (lane == 0) {
            int st = 0;
            uint32_t ph = 0;
            bool wrapped = false;
            int used = 0;
            for (long long u = u0; u < a.units; u += ustep) {
                const Unit x = unit_of<BN>(a, u);
                const int am = (x.m * CG + (int)rank) * BM;
                const int rows_b = x.bn / CG, bn = (int)x.n0 + (int)rank * rows_b;
                const uint32_t bytes = CG * (C::A_BYTES + rows_b * BK * 2);
                int q = x.it0 / a.ksteps, k = x.it0 - q * a.ksteps;
                for (int it = x.it0; it < x.it1; it++) {
                    int pa, pb;
                    planes_of(a.passes, q, pa, pb);
                    wait_bar(empty + st, ph ^ 1, abort_flag, &g_lin_error, 601);
                    unsigned char *sa = smem + st * C::STAGE, *sb = sa + C::A_BYTES;
                    if constexpr (CG == 2) {
                        if (rank == 0) mbar_expect_tx(full + st, bytes);
                        const uint32_t bar = map_rank(full + st, 0);
                        if constexpr (A_K) tma_load_3d_pair(sa, &map_a, bar, k * BK, am, pa);
                        else
                            for (int i = 0; i < BM / 64; i++) tma_load_3d_pair(sa + i * 8192, &map_a, bar, am + 64 * i, k * BK, pa);
                        for (int i = 0; i < rows_b; i += 64) {
                            if constexpr (B_K) tma_load_3d_pair(sb + i * 128, &map_b, bar, k * BK, bn + i, pb);
                            else tma_load_3d_pair(sb + i * 128, &map_b, bar, bn + i, k * BK, pb);
                        }
                    } else {
                        mbar_expect_tx(full + st, bytes);
                        if constexpr (A_K) tma_load_3d(sa, &map_a, full + st, k * BK, am, pa);
                        else
                            for (int i = 0; i < BM / 64; i++) tma_load_3d(sa + i * 8192, &map_a, full + st, am + 64 * i, k * BK, pa);
                        for (int i = 0; i < rows_b; i += 64) {
                            if constexpr (B_K) tma_load_3d(sb + i * 128, &map_b, full + st, k * BK, bn + i, pb);
                            else tma_load_3d(sb + i * 128, &map_b, full + st, bn + i, k * BK, pb);
                        }
                    }
                    if (++k == a.ksteps) {
                        k = 0;
                        q++;
                    }
                    used = max(used, st + 1);
                    if (++st == S) {
                        st = 0;
                        ph ^= 1;
                        wrapped = true;
                    }
                }
            }
            // the copies must have landed before the CTAs of the pair exit (the leader's barriers count both CTAs')
            if (rank == 0)
                for (int i = 0; i < (wrapped ? S : used); i++) drain_bar(full + i, i < st ? ph : ph ^ 1, &g_lin_error);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issue (whole warp, the pair's even CTA)
        if (rank == 0) {
            int st = 0, tc = 0;
            uint32_t ph = 0;
            for (long long u = u0; u < a.units; u += ustep) {
                const Unit x = unit_of<BN>(a, u);
                const uint32_t idesc = x.bn == BN ? idesc_bf16(BM * CG, BN, !A_K, !B_K) : idesc_bf16(BM * CG, BN / 2, !A_K, !B_K);
                const int tb = tc & 1;
                wait_bar(t_empty + tb, ((tc >> 1) & 1) ^ 1, abort_flag, &g_lin_error, 602);
                fence_after();
                const uint32_t d = tmem + (uint32_t)(tb * BN);
                for (int it = x.it0; it < x.it1; it++) {
                    wait_bar(full + st, ph, abort_flag, &g_lin_error, 603);
                    fence_after();
                    const unsigned char *sa = smem + st * C::STAGE, *sb = sa + C::A_BYTES;
                    // along k (16 values): 32 bytes of a k-major row, 16 rows of 128 bytes of an m/n-major tile
                    const uint64_t da = A_K ? desc_kmajor(sa) : desc_sw128(sa, 8192, 1024);
                    const uint64_t db = B_K ? desc_kmajor(sb) : desc_sw128(sb, 8192, 1024);
                    if constexpr (CG == 2)
                        mma4_ss_pair_w(d, da, A_K ? 2 : 128, db, B_K ? 2 : 128, idesc, it != x.it0, su32(empty + st));
                    else
                        mma4_ss_w(d, da, A_K ? 2 : 128, db, B_K ? 2 : 128, idesc, it != x.it0, su32(empty + st));
                    if (++st == S) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                if constexpr (CG == 2) mma_commit_pair_w(t_full + tb);
                else mma_commit_w(t_full + tb);
                tc++;
            }
            if constexpr (CG == 2) mma_commit_pair_w(done);
            else mma_commit_w(done);
            drain_bar(done, 0, &g_lin_error);
        }
    } else {
        // ---------------------------------------------------------- epilogue (warps 2..9)
        const int quad = warp & 3;               // TMEM lanes this warp may access
        const int half = (warp - 2) >> 2;        // half of the columns
        Store out;
        out.buf = smem + C::TURN + (warp - 2) * 4096;
        out.lane = lane;
        out.turn = 0;
        out.two = a.splits == 1 && !a.e.out_f32;
        int tc = 0;
        for (long long u = u0; u < a.units; u += ustep, tc++) {
            const Unit x = unit_of<BN>(a, u);
            const int tb = tc & 1, cols = x.bn / 2;
            const long long m0 = ((long long)x.m * CG + rank) * BM + quad * 32;
            const uint32_t t = tmem + (uint32_t)(tb * BN + half * cols) + ((uint32_t)(quad * 32) << 16);
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) {
                const long long n0 = x.n0 + half * cols + c;
                Residual res;
                if (a.e.res != nullptr && a.splits == 1 && m0 + lane < a.M && n0 < a.N) {
                    if (a.e.out_f32) res.load<float>(a, m0 + lane, n0);
                    else res.load<__nv_bfloat16>(a, m0 + lane, n0);
                }
                if (c == 0) {
                    wait_bar(t_full + tb, (tc >> 1) & 1, abort_flag, &g_lin_error, 604);
                    fence_after();
                }
                float v[32];
                tmem_ld32(t + c, v);
                if (c + 32 == cols) {  // the accumulator is in registers: the next tile's MMAs may have it
                    fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CG == 2) mbar_arrive_cluster(map_rank(t_empty + tb, 0));
                        else mbar_arrive(t_empty + tb);
                    }
                }
                if (m0 >= a.M || n0 >= a.N) continue;
                if (a.splits > 1) out.tile<float>(a, &map_out, v, m0, n0, x.s, nullptr, 0);
                else if (a.e.out_f32) finish<float>(a, &map_out, &map_pre, out, v, res, m0, n0);
                else finish<__nv_bfloat16>(a, &map_out, &map_pre, out, v, res, m0, n0);
            }
        }
        if (lane == 0) bulk_wait<0>();
    }
    __syncwarp();
    fence_before();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    fence_after();
    if (warp == 1) {
        if constexpr (CG == 2) tmem_dealloc_pair(tmem, C::TMEM);
        else tmem_dealloc(tmem, C::TMEM);
    }
}

// ------------------------------------------------------------------ host side

enum Shape { LONE_64, PAIR_128, PAIR_256 };

// Which tile a product takes.  Lone CTAs of 128 x 64 when m fits one of them; pairs otherwise, 256 wide where that
// leaves a tile for more than half of them (a 256-wide tile moves 64 bytes of operands per SM and cycle of MMAs, a
// 128-wide one 96).
static Shape shape_of(long long M, long long N, int sms)
{
    if (M <= 128) return LONE_64;
    return N > 128 && (M + 255) / 256 * ((N + 255) / 256) * 2 > sms / 2 ? PAIR_256 : PAIR_128;
}

static void tile_counts(Shape s, long long M, long long N, int &mt, int &nt)
{
    const int bm = s == LONE_64 ? 128 : 256, bn = s == LONE_64 ? 64 : s == PAIR_128 ? 128 : 256;
    mt = (int)((M + bm - 1) / bm);
    nt = (int)((N + bn - 1) / bn);
}

int product_splits(long long M, long long N, long long K, int planes, int sms)
{
    int mt, nt;
    const Shape s = shape_of(M, N, sms);
    tile_counts(s, M, N, mt, nt);
    const long long tiles = (long long)mt * nt, slots = s == LONE_64 ? sms : sms / 2;
    const long long steps = (K + BK - 1) / BK * (planes == 3 ? 6 : 1);
    if (tiles * 2 > slots || steps < 8) return 1;
    const long long want = slots / tiles, most = steps / 4;
    const long long per = (steps + (want < most ? want : most) - 1) / (want < most ? want : most);
    return (int)((steps + per - 1) / per);  // no piece is empty
}

template <int CG, int BN, bool A_K, bool B_K>
static cudaError_t launch(const CUtensorMap (&map)[4], const Args &a, int sms, cudaStream_t st)
{
    using C = Cfg<CG, BN>;
    auto *kernel = linear_tc_kernel<CG, BN, A_K, B_K>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const long long slots = sms / CG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.units < slots ? a.units : slots) * CG));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = CG;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = CG == 2 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kernel, map[0], map[1], map[2], map[3], a);
    if (e == cudaSuccess) note_launches(1);
    return e;
}

template <int CG, int BN>
static cudaError_t launch_majors(const Product &p, const CUtensorMap (&map)[4], const Args &a, int sms, cudaStream_t st)
{
    if (p.a.k_major) return p.b.k_major ? launch<CG, BN, true, true>(map, a, sms, st) : launch<CG, BN, true, false>(map, a, sms, st);
    return launch<CG, BN, false, false>(map, a, sms, st);
}

// The outputs' tiles: `n` values a row, rows `ld` apart, `z` matrices of M rows.
static bool encode_out(CUtensorMap *m, bool f32, const void *base, long long n, long long ld, long long M, int z)
{
    const long long size = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)n, (cuuint64_t)M, (cuuint64_t)z};
    const cuuint64_t strides[2] = {(cuuint64_t)(ld * size), (cuuint64_t)(M * ld * size)};
    const cuuint32_t box[3] = {32, 32, 1};
    return tc_encode_store(m, f32, base, 3, dims, strides, box);
}

// A map over {contiguous, strided, plane} of an operand of `n` rows (m or n) and K; boxes of 64 contiguous values.
static bool encode(CUtensorMap *m, const Operand &o, long long n, long long K, int planes, int rows)
{
    const long long inner = o.k_major ? K : n, outer = o.k_major ? n : K;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)planes};
    // one plane: its stride is never used, but has to be a legal one (below 2^40 bytes)
    const long long far = 1LL << 38, whole = outer > far / o.ld ? far : outer * o.ld;
    const cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2, (cuuint64_t)(planes > 1 ? o.plane : whole) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)(o.k_major ? rows : 64), 1};
    return tc_encode_bf16(m, o.base, 3, dims, strides, box);
}

cudaError_t launch_product_tc(const Product &p, int sms, cudaStream_t st)
{
    const Shape s = shape_of(p.M, p.N, sms);
    Args a = {};
    a.M = p.M;
    a.N = p.N;
    a.ksteps = (int)((p.K + BK - 1) / BK);
    a.passes = p.planes == 3 ? 6 : 1;
    const int steps = a.ksteps * a.passes;
    a.per_split = (steps + p.splits - 1) / p.splits;
    a.splits = p.splits;
    tile_counts(s, p.M, p.N, a.mt, a.nt);
    a.units = a.whole = (long long)a.mt * a.nt * p.splits;
    const long long slots = sms / 2, rest = a.units % slots;
    if (s == PAIR_256 && p.splits == 1 && a.units > slots && rest > 0 && 2 * rest <= slots) {
        a.whole -= rest;
        a.units += rest;
    }
    a.e = p.e;
    CUtensorMap map[4];
    memset(map, 0, sizeof map);
    if (!encode(&map[0], p.a, p.M, p.K, p.planes, BM) || !encode(&map[1], p.b, p.N, p.K, p.planes, 64)) return cudaErrorInvalidValue;
    if (p.splits > 1) {
        a.tma_out = 1;
        if (!encode_out(&map[2], true, p.e.partial, p.N, partial_stride(p.N), p.M, p.splits)) return cudaErrorInvalidValue;
    } else {
        a.tma_out = p.N % (p.e.out_f32 ? 4 : 8) == 0 && (p.e.preact == nullptr || p.N % (p.e.preact_f32 ? 4 : 8) == 0);
        if (a.tma_out) {
            if (!encode_out(&map[2], p.e.out_f32, p.e.out, p.N, p.N, p.M, 1)) return cudaErrorInvalidValue;
            if (p.e.preact != nullptr && !encode_out(&map[3], p.e.preact_f32, p.e.preact, p.N, p.N, p.M, 1)) return cudaErrorInvalidValue;
        }
    }
    if (s == LONE_64) return launch_majors<1, 64>(p, map, a, sms, st);
    if (s == PAIR_128) return launch_majors<2, 128>(p, map, a, sms, st);
    return launch_majors<2, 256>(p, map, a, sms, st);
}

}  // namespace linear
}  // namespace csa
