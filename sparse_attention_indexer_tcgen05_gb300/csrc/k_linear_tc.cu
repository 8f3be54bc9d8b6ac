// k_linear_tc.cu -- the projections' products on the 5th-generation tensor cores (tcgen05 + TMEM + TMA).
//
// D[m][n] = sum_k A(m, k) B(n, k) with bf16 operands and fp32 sums, for y = x W^T (both operands contiguous along
// k), dx = dz W (B contiguous along n) and dW = dz^T x (both contiguous along m, n): the shared-memory descriptors
// take either order, so no operand is transposed in memory.  fp32 values come as three bf16 planes, x = h + m + l, and each
// 64 k of them take six products, l h, h l, m m, m h, h m, h h, the smallest terms first; what is left out is below
// 2^-23 of the terms.
//
// The tensor core cuts a sum off where it aligns it with a product (it does not round), so a TMEM accumulator loses about
// 2^-24 / 3 of itself with every 16 k, always towards zero, and, once it is large beside the products, which are cut off too,
// four times that: 7e-7 at k = 512, 3e-4 at k = 65536 (positive terms).  That is little beside a bf16 result up to LONGEST k
// (a thirteenth of the largest rounding); longer axes are cut into pieces, joined in fp32 (dW of 2^20 rows came out 6e-3 too
// small in one).  For fp32 results (EXACT below) the accumulator starts anew every 64 k (three planes: the
// small terms then meet a small sum; 9e-8 to 1.5e-7 off, k = 64 to 65536) or every 512 k (4e-7 to 7e-7), and the epilogue's warps add up the
// pieces in registers, rounded.
//
// Mapping.  A unit is one output tile and one piece of the k axis.  A CTA pair (two SMs) computes 256 x BN: each CTA
// loads its 128 rows of A and its BN / 2 rows of B, so an operand byte brought to an SM feeds twice the MMAs of a lone
// CTA's 128 x BN tile.  Few tiles, or few rows, take lone CTAs with 128 x 64 tiles.  Roles: warp 0 the TMA producer,
// warp 1 the MMA issue (the pair's even CTA), warps 2..9 (2..17) the epilogue, a row of the tile a lane.  TMEM holds two
// accumulators, so that a tile's epilogue runs under the next tile's MMAs.  Persistent: one CTA per SM, units dealt
// round-robin in an order that keeps the running tiles' operands in L2.
//
// Measured (bf16, from and to bf16): 8192 x 8192 x 2048 142 us (1.94 PFLOP/s; the library's product takes 140), its two
// gradients 151 to 170 and 163 to 175 us (153 and 163), 8192^3 590 to 634 us (577 to 592), 2048^3 17 to 20 us (22).  Bound by the MMAs (87%
// of the cycles), and at the chip's power limit by its clock; up to 256 k by the epilogue.
//
// Every mbarrier wait is bounded (see tc_ptx.cuh); site codes 600 + n.
#include "csa_tc.cuh"
#include "k_linear.cuh"
#include "tc_ptx.cuh"

#include <cuda.h>
#include <math.h>

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
constexpr long long LONGEST = 65536;  // k that a bf16 result sums in one accumulator
constexpr int CHUNK_1 = 8;     // stages (512 k) that an fp32 result of one plane does
constexpr int MANY_STEPS = 4;  // stages of a unit up to which 256-wide tiles have 16 epilogue warps

// P planes, EW epilogue warps
template <int CG, int BN, int P, int EW> struct Cfg {
    static constexpr int THREADS = 64 + 32 * EW;
    static constexpr int ROWS_B = BN / CG;                      // B rows this CTA loads
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = ROWS_B * BK * 2;
    static constexpr int STAGE = P * (A_BYTES + B_BYTES);
    static constexpr int STAGES = (229376 - EW * 4096) / STAGE; // of 192 KB (EW 8): 6 or 8; 2 of three planes
    static constexpr int TURN = STAGES * STAGE;                 // the epilogue's buffers, 32 rows of 128 bytes a warp
    static constexpr int MISC = TURN + EW * 4096;
    static constexpr int SMEM = MISC + 512 + 1024;              // + alignment
    static constexpr int TMEM = 2 * BN < 512 ? (2 * BN < 128 ? 128 : 2 * BN) : 512;
};

struct Args {
    long long M, N, ldo;        // the output's row stride
    int ksteps;                 // stages over the whole k axis, all passes
    int splits, per_split;      // k pieces, stages of each
    int mt, nt;                 // tiles
    int whole, units;           // units that are whole tiles (times splits); the rest are halves of the last tiles
    int rows_a;                 // rows of A a CTA loads: BM, fewer where M is below BM
    int blocks_a, blocks_b;     // an m/n-contiguous operand's map has 64-wide blocks as an axis of their own
    int tma_out;                // the output goes by TMA
    int many;                   // 16 epilogue warps
    int res32;                  // the residual's rows start on 32-byte sectors
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
template <int BN> __device__ __forceinline__ Unit unit_of(const Args &a, int u)
{
    Unit x;
    const int tiles = a.mt * a.nt;
    int t, half = 0;
    x.bn = BN;
    x.s = 0;
    if (u < a.whole) {
        if (a.splits > 1) {
            x.s = u / tiles;
            t = u - x.s * tiles;
        } else {
            t = u;
        }
    } else {
        t = a.whole + ((u - a.whole) >> 1);
        half = (u - a.whole) & 1;
        x.bn = BN / 2;
    }
    const int per_band = BAND * a.nt;
    const int band = t / per_band;
    const int r = t - band * per_band;
    const int h = min(BAND, a.mt - band * BAND);
    x.m = band * BAND + r % h;
    x.n0 = (long long)(r / h) * BN + half * (BN / 2);
    x.it0 = x.s * a.per_split;
    x.it1 = min(a.ksteps, x.it0 + a.per_split);
    return x;
}

// Shared memory a warp stores from: 32 rows of 128 bytes.
struct Buffer {
    unsigned char *p;
    int lane;
};

// 256-bit accesses, whole sectors
__device__ __forceinline__ void st32(void *p, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ void ld32(const void *p, uint32_t *w)
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}

constexpr int C = 32;   // columns of an epilogue step

// 32 columns of one row of the residual.  Whole sectors are asked for a step before they are used (`early`); other rows
// (and a warp's columns that end behind N) are read where they are added, as the aligned vectors that hold the columns that exist, shifted.  (Value
// by value, bias, GELU and residual of 8200 x 4104 x 264 took 125 us instead of 70.)
template <typename O> struct Residual {
    static constexpr int W = C * sizeof(O) / 4;
    uint32_t r[W];
    static __device__ __forceinline__ const O *at(const Args &a, long long m, long long n0) { return (const O *)a.e.res + m * a.e.ldr + n0; }
    static __device__ __forceinline__ void add(const uint32_t *r, float (&v)[C])
    {
#pragma unroll
        for (int k = 0; k < C; k++) {
            if constexpr (sizeof(O) == 4) v[k] += __uint_as_float(r[k]);
            else v[k] += __uint_as_float(k % 2 == 0 ? r[k / 2] << 16 : r[k / 2] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void load(const Args &a, long long m, long long n0)
    {
        if (m >= a.M) return;
        const O *p = at(a, m, n0);
#pragma unroll
        for (int k = 0; k < W / 8; k++) ld32(p + 32 / sizeof(O) * k, r + 8 * k);
    }
    __device__ __forceinline__ void add_to(const Args &a, long long m, long long n0, bool early, float (&v)[C]) const
    {
        if (early) {
            add(r, v);
        } else if (m < a.M) {
            const O *p = at(a, m, n0);
            const int sh = (int)(reinterpret_cast<uintptr_t>(p) & 15), end = sh + (int)min((long long)C, a.N - n0) * (int)sizeof(O);
            const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) - sh);
            uint32_t u[W + 4];
#pragma unroll
            for (int k = 0; k <= W / 4; k++) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (end > 16 * k) x = load16(q + k, at(a, a.M - 1, a.N));
                u[4 * k] = x.x; u[4 * k + 1] = x.y; u[4 * k + 2] = x.z; u[4 * k + 3] = x.w;
            }
            if (sh & 8) {
#pragma unroll
                for (int k = 0; k < W + 2; k++) u[k] = u[k + 2];
            }
            if (sh & 4) {
#pragma unroll
                for (int k = 0; k < W + 1; k++) u[k] = u[k + 1];
            }
            if (sizeof(O) == 2 && (sh & 2)) {
#pragma unroll
                for (int k = 0; k < W; k++) u[k] = __funnelshift_r(u[k], u[k + 1], 16);
            }
            add(u, v);
        }
    }
};

template <int ACT> __device__ __forceinline__ void activate(float (&v)[C])
{
#pragma unroll
    for (int k = 0; k < C; k += 2) {
        const float2 y = act_fwd2<ACT>(make_float2(v[k], v[k + 1]));
        v[k] = y.x;
        v[k + 1] = y.y;
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The second half of a turn: V neighbouring columns a lane, 32 / V lanes a row.  Rows start on V values.
template <typename O, int V>
__device__ __forceinline__ void turned_rows(O *out, long long ld, long long M, long long N, long long m0, long long n0, int lane, const float *turn)
{
    constexpr int LANES = 32 / V;
    const int c = lane % LANES * V;
    if (n0 + c >= N) return;
    const int rows = (int)min(32LL, M - m0);
    O *p = out + m0 * ld + n0 + c;
#pragma unroll 4
    for (int r = lane / LANES; r < rows; r += V) {
        float x[V];
#pragma unroll
        for (int k = 0; k < V; k++) x[k] = turn[r * 32 + ((c + k + r) & 31)];
        O *q = p + r * ld;
        if (V > 1 && n0 + c + V <= N) {
            if constexpr (sizeof(O) == 4 && V == 2) *reinterpret_cast<float2 *>(q) = make_float2(x[0], x[1]);
            else if constexpr (V == 2) *reinterpret_cast<uint32_t *>(q) = pack2(x[0], x[1]);
        } else {
#pragma unroll
            for (int k = 0; k < V; k++)
                if (n0 + c + k < N) q[k] = from_f<O>(x[k]);
        }
    }
}

// A warp's 32 rows x 32 columns, a row a lane, to memory by the lanes' own stores; rows from M and columns from N on
// are left out.  Rows on 32-byte boundaries: each lane its own sectors; on 16-byte ones: half sectors (kept z of 8200 x
// 4104 x 264: 90 us with everything instead of 123; 103 in a loop at the power limit).  Else: turned in shared memory so that a warp
// writes 32 neighbouring values at a time.
template <typename O>
__device__ __forceinline__ void store_tile(O *out, long long ld, long long M, long long N, const float (&v)[C], long long m0, long long n0,
                                           const Buffer &b)
{
    const int lane = b.lane;
    constexpr int E = 32 / sizeof(O);
    if (ld % E == 0 && (reinterpret_cast<uintptr_t>(out) & 31) == 0) {
        if (m0 + lane >= M) return;
        O *p = out + (m0 + lane) * ld + n0;
#pragma unroll
        for (int k = 0; k < C / E; k++) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; j++) w[j] = sizeof(O) == 2 ? pack2(v[E * k + 2 * j % E], v[E * k + (2 * j + 1) % E]) : __float_as_uint(v[E * k + j]);
            if (n0 + E * k < N) st32(p + E * k, w);
        }
    } else if (ld % (E / 2) == 0) {
        if (m0 + lane >= M) return;
        O *p = out + (m0 + lane) * ld + n0;
#pragma unroll
        for (int k = 0; k < 2 * C / E; k++) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; j++) w[j] = sizeof(O) == 2 ? pack2(v[E / 2 * k + 2 * j % E], v[E / 2 * k + (2 * j + 1) % E]) : __float_as_uint(v[E / 2 * k + j]);
            if (n0 + E / 2 * k < N) *reinterpret_cast<uint4 *>(p + E / 2 * k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        float *turn = reinterpret_cast<float *>(b.p);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < C; k++) turn[lane * 32 + ((k + lane) & 31)] = v[k];
        __syncwarp();
        const int odd = (int)(ld | (reinterpret_cast<uintptr_t>(out) / sizeof(O)));
        if ((odd & 1) == 0) turned_rows<O, 2>(out, ld, M, N, m0, n0, lane, turn);
        else turned_rows<O, 1>(out, ld, M, N, m0, n0, lane, turn);
    }
}

// The same by TMA, from rows of 128 bytes in shared memory (32 fp32 columns, or 64 bf16 ones: two steps), so that a
// request to L2 carries four sectors.  (The lanes' own sectors slowed the loads of the next tile: a product
// of 8192 x 8192 x 8192 took 640 us instead of 572.)  `second`: the right 64 bytes of bf16
// rows; `go`: the rows are complete.
template <typename O>
__device__ __forceinline__ void tma_tile(const CUtensorMap *map, const float (&v)[C], long long m0, long long n0, int s, bool second, bool go,
                                         const Buffer &b)
{
    const int lane = b.lane;
    if (!second) {
        if (lane == 0) bulk_wait_read();  // the last tile has left the buffer
        __syncwarp();
    }
    const int first = sizeof(O) == 2 && second ? 4 : 0;
#pragma unroll
    for (int k = 0; k < (int)(2 * sizeof(O)); k++) {
        uint4 w;
        if constexpr (sizeof(O) == 2)
            w = make_uint4(pack2(v[8 * k], v[8 * k + 1]), pack2(v[8 * k + 2], v[8 * k + 3]), pack2(v[8 * k + 4], v[8 * k + 5]),
                           pack2(v[8 * k + 6], v[8 * k + 7]));
        else
            w = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3]));
        *reinterpret_cast<uint4 *>(b.p + lane * 128 + (((first + k) ^ (lane & 7)) << 4)) = w;
    }
    if (!go) return;
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
        tma_store_3d(map, b.p, (int)n0 - (sizeof(O) == 2 && second ? C : 0), (int)m0, s);
        bulk_commit();
    }
}

// A step's bias, asked for with the residual.  (Loaded where it is added, behind a question for each four columns, it
// cost 50 us of a product of 8192 x 8192 x 512 that takes 51 without.)
struct Bias {
    float own;   // of column n0 + lane; the others come from their lanes (a register instead of 32)
    __device__ __forceinline__ void load(const Args &a, long long n0, int lane) { own = n0 + lane < a.N ? __ldg(a.e.bias + n0 + lane) : 0.f; }
    __device__ __forceinline__ void add_to(float alpha, float (&v)[C]) const
    {
#pragma unroll
        for (int k = 0; k < C; k++) v[k] = fmaf(alpha, v[k], __shfl_sync(0xffffffffu, own, k));
    }
};

// z kept if asked for, then act(z) in place.
__device__ __forceinline__ void to_activation(const Args &a, float (&v)[C], long long m0, long long n0, const Buffer &b)
{
    const Epilogue &e = a.e;
    if (e.preact != nullptr) {
        if (e.preact_f32) store_tile<float>((float *)e.preact, a.N, a.M, a.N, v, m0, n0, b);
        else store_tile<__nv_bfloat16>((__nv_bfloat16 *)e.preact, a.N, a.M, a.N, v, m0, n0, b);
    }
    if (e.act == CSA_ACT_RELU) activate<CSA_ACT_RELU>(v);
    else if (e.act == CSA_ACT_SILU) activate<CSA_ACT_SILU>(v);
    else if (e.act == CSA_ACT_GELU_TANH) activate<CSA_ACT_GELU_TANH>(v);
}

// EXACT: the sums are kept in the epilogue's registers, pieces of CHUNK stages of the k axis in TMEM.  TWO: two passes, whose
// stages take turns (B's second one comes from L2).  (As an argument instead, it cost a product of 37 rows 0.7 us of 11.6.)
template <int CG, int BN, int P, int EW, bool EXACT, bool A_K, bool B_K, bool TWO>
__global__ void __launch_bounds__(64 + 32 * EW, 1)
linear_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ CUtensorMap map_half, const __grid_constant__ CUtensorMap map_out, const Args a)
{
    using Z = Cfg<CG, BN, P, EW>;
    constexpr int S = Z::STAGES;
    constexpr int CHUNK = !EXACT ? 0x40000000 : P == 3 ? 1 : CHUNK_1;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_align1024(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Z::MISC);
    uint64_t *full = bars, *empty = bars + S, *t_full = bars + 2 * S, *t_empty = bars + 2 * S + 2, *done = bars + 2 * S + 4;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Z::MISC + 256);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Z::MISC + 264);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
    const int u0 = blockIdx.x / CG, ustep = gridDim.x / CG;
    chain_start();

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; i++) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(t_full + i, 1);
            mbar_init(t_empty + i, EW * CG);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        init_fence();
    }
    if (warp == 1) {
        if constexpr (CG == 2) tmem_alloc_pair(tmem_slot, Z::TMEM);
        else tmem_alloc(tmem_slot, Z::TMEM);
    }
    fence_before();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    chain_wait();

    if (warp == 0) {
        // ---------------------------------------------------------- TMA producer
        // Few and large copies: with B in two boxes of 64 rows instead of one of 128 the same product took 164 us
        // instead of 150 (8192 x 8192 x 2048).
        if (lane == 0) {
            int st = 0;
            uint32_t ph = 0;
            bool wrapped = false;
            int used = 0;
            const uint32_t bar0 = CG == 2 ? map_rank(full, 0) : su32(full);  // the barriers are the even CTA's
            auto load3 = [&](void *to, const CUtensorMap *map, int i, int x, int y, int z) {
                if constexpr (CG == 2) tma_load_3d_pair(to, map, bar0 + 8 * i, x, y, z);
                else tma_load_3d(to, map, full + i, x, y, z);
            };
            auto load4 = [&](void *to, const CUtensorMap *map, int i, int x, int y, int z, int w) {
                if constexpr (CG == 2) tma_load_4d_pair(to, map, bar0 + 8 * i, x, y, z, w);
                else tma_load_4d(to, map, full + i, x, y, z, w);
            };
            for (int u = u0; u < a.units; u += ustep) {
                const Unit x = unit_of<BN>(a, u);
                const bool half = x.bn != BN;
                const int am = (x.m * CG + (int)rank) * BM;
                const int rows_b = x.bn / CG, bn = (int)x.n0 + (int)rank * rows_b;
                // rows of A that do not exist are not asked for (TMA would send their zeros over the crossbar: 100 MB
                // instead of 45 for 37 rows against 8192 x 2048 weights); what lies in their place in shared memory
                // reaches sums of such rows only
                const bool with_a = am < a.M;
                const int ctas_a = CG == 2 && (x.m * 2 + 1LL) * BM < a.M ? 2 : 1;
                const uint32_t bytes = P * (ctas_a * a.rows_a + CG * rows_b) * BK * 2;
                const CUtensorMap *mb = half ? &map_half : &map_b;
                for (int it = x.it0; it < x.it1; it++) {
                    const int k = (TWO ? it >> 1 : it) * BK, plane_a = TWO ? ~it & 1 : 0;
                    wait_bar(empty + st, ph ^ 1, abort_flag, &g_lin_error, 601);
                    if (rank == 0) mbar_expect_tx(full + st, bytes);
#pragma unroll
                    for (int q = 0; q < P; q++) {
                        unsigned char *sa = smem + st * Z::STAGE + q * Z::A_BYTES, *sb = smem + st * Z::STAGE + P * Z::A_BYTES + q * Z::B_BYTES;
                        const int qa = P == 1 ? plane_a : q;
                        if (!with_a) {
                        } else if constexpr (A_K) {
                            load3(sa, &map_a, st, k, am, qa);
                        } else if (a.blocks_a) {
                            load4(sa, &map_a, st, 0, k, am >> 6, qa);
                        } else {
                            for (int i = 0; i < a.rows_a; i += 64) load3(sa + i * 128, &map_a, st, am + i, k, qa);
                        }
                        if constexpr (B_K) {
                            load3(sb, mb, st, k, bn, q);
                        } else if (a.blocks_b) {
                            load4(sb, mb, st, 0, k, bn >> 6, q);
                        } else {
                            for (int i = 0; i < rows_b; i += 64) load3(sb + i * 128, mb, st, bn + i, k, q);
                        }
                    }
                    used = max(used, st + 1);
                    if (++st == S) {
                        st = 0;
                        ph ^= 1;
                        wrapped = true;
                    }
                }
            }
            // the copies must have landed before the CTAs of the pair exit (the leader's barriers count both CTAs'), and so
            // must the arrivals that the leader's commits send to this CTA's barriers: its shared memory is another's then
            for (int i = 0; i < (wrapped ? S : used); i++) {
                if (rank == 0) drain_bar(full + i, i < st ? ph : ph ^ 1, &g_lin_error);
                drain_bar(empty + i, i < st ? ph : ph ^ 1, &g_lin_error);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issue (whole warp, the pair's even CTA)
        if (rank == 0) {
            int st = 0, tc = 0;
            uint32_t ph = 0;
            for (int u = u0; u < a.units; u += ustep) {
                const Unit x = unit_of<BN>(a, u);
                const uint32_t idesc = x.bn == BN ? idesc_bf16(BM * CG, BN, !A_K, !B_K) : idesc_bf16(BM * CG, BN / 2, !A_K, !B_K);
                for (int it0 = x.it0; it0 < x.it1; it0 += min(CHUNK, x.it1 - it0)) {
                    const int it1 = min(CHUNK, x.it1 - it0) + it0, tb = tc & 1;
                    wait_bar(t_empty + tb, ((tc >> 1) & 1) ^ 1, abort_flag, &g_lin_error, 602);
                    fence_after();
                    const uint32_t d = tmem + (uint32_t)(tb * BN);
                    for (int it = it0; it < it1; it++) {
                        wait_bar(full + st, ph, abort_flag, &g_lin_error, 603);
                        fence_after();
                        const unsigned char *sa = smem + st * Z::STAGE, *sb = sa + P * Z::A_BYTES;
                        constexpr int PRODUCTS = P == 1 ? 1 : 6;
#pragma unroll
                        for (int i = 0; i < PRODUCTS; i++) {
                            constexpr int PA[6] = {2, 0, 1, 1, 0, 0}, PB[6] = {0, 2, 1, 0, 1, 0};
                            const unsigned char *pa = sa + (P == 1 ? 0 : PA[i]) * Z::A_BYTES, *pb = sb + (P == 1 ? 0 : PB[i]) * Z::B_BYTES;
                            // along k (16 values): 32 bytes of a k-major row, 16 rows of 128 bytes of an m/n-major tile
                            const uint64_t da = A_K ? desc_kmajor(pa) : desc_sw128(pa, 8192, 1024);
                            const uint64_t db = B_K ? desc_kmajor(pb) : desc_sw128(pb, 8192, 1024);
                            const uint32_t acc = i > 0 || it != it0, bar = i == PRODUCTS - 1 ? su32(empty + st) : 0u;
                            if constexpr (CG == 2) mma4_ss_pair_w(d, da, A_K ? 2 : 128, db, B_K ? 2 : 128, idesc, acc, bar);
                            else mma4_ss_w(d, da, A_K ? 2 : 128, db, B_K ? 2 : 128, idesc, acc, bar);
                        }
                        if (++st == S) {
                            st = 0;
                            ph ^= 1;
                        }
                    }
                    if constexpr (CG == 2) mma_commit_pair_w(t_full + tb);
                    else mma_commit_w(t_full + tb);
                    tc++;
                }
            }
            if constexpr (CG == 2) mma_commit_pair_w(done);
            else mma_commit_w(done);
        }
        drain_bar(done, 0, &g_lin_error);  // in either CTA: the commit arrives in both
    } else {
        // ---------------------------------------------------------- epilogue (8 or 16 warps)
        const int quad = warp & 3;               // TMEM lanes this warp may access
        const int side = (warp - 2) >> 2;        // part of the columns
        const Buffer b = {smem + Z::TURN + (warp - 2) * 4096, lane};
        // asked once: each of these questions cost a step a miss in the constant and instruction caches
        const bool tma = a.tma_out != 0, with_res = a.e.res != nullptr, with_bias = a.e.bias != nullptr, with_act = a.e.act != CSA_ACT_NONE || a.e.preact != nullptr;
        const float alpha = a.e.alpha;
        auto run = [&](auto type) {
            using O = decltype(type);
            int tc = 0;
            for (int u = u0; u < a.units; u += ustep) {
                const Unit x = unit_of<BN>(a, u);
                const int cols = x.bn / (EW / 4);
                const long long m0 = ((long long)x.m * CG + rank) * BM + quad * 32, nb = x.n0 + side * cols;
                const auto release = [&](int tb) {  // the accumulator is in registers: the next MMAs may have it
                    fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CG == 2) mbar_arrive_cluster(map_rank(t_empty + tb, 0));
                        else mbar_arrive(t_empty + tb);
                    }
                };
                const auto wait = [&] {
                    wait_bar(t_full + (tc & 1), (tc >> 1) & 1, abort_flag, &g_lin_error, 604);
                    fence_after();
                    return tmem + (uint32_t)((tc & 1) * BN + side * cols) + ((uint32_t)(quad * 32) << 16);
                };
                const bool early = with_res && a.res32 && nb + cols <= a.N;
                Residual<O> res;
                Bias bias;
                const auto ask = [&](long long n0) {
                    if (with_bias) bias.load(a, n0, lane);
                    if (early) res.load(a, m0 + lane, n0);
                };
                // 32 columns from sums to memory
                const auto step = [&](int c, float (&v)[C]) {
                    const long long n0 = nb + c;
                    if (m0 >= a.M || n0 >= a.N) return;
                    if (with_bias) {
                        bias.add_to(alpha, v);
                    } else if (alpha != 1.f) {
#pragma unroll
                        for (int k = 0; k < C; k++) v[k] *= alpha;
                    }
                    if (with_act) to_activation(a, v, m0, n0, b);
                    if (with_res) res.add_to(a, m0 + lane, n0, early, v);
                    if (c + C < cols) ask(n0 + C);
                    if (tma) {
                        const bool second = sizeof(O) == 2 && (c & C) != 0;
                        tma_tile<O>(&map_out, v, m0, n0, x.s, second, sizeof(O) == 4 || second || n0 + C >= a.N, b);
                    } else {
                        store_tile<O>((O *)a.e.out + (long long)x.s * a.M * a.ldo, a.ldo, a.M, a.N, v, m0, n0, b);
                    }
                };
                if constexpr (EXACT) {
                    constexpr int G = BN / 2 / C;
                    float sum[G][C] = {};
                    for (int it = x.it0; it < x.it1; it += CHUNK, tc++) {
                        const uint32_t t = wait();
#pragma unroll
                        for (int g = 0; g < G; g++) {
                            float v[C];
                            tmem_ld32(t + g * C, v);
                            if (g == G - 1) release(tc & 1);
#pragma unroll
                            for (int k = 0; k < C; k++) sum[g][k] += v[k];
                        }
                    }
                    ask(nb);
#pragma unroll
                    for (int g = 0; g < G; g++) step(g * C, sum[g]);
                } else {
                    ask(nb);
                    const uint32_t t = wait();
#pragma unroll 1
                    for (int c = 0; c < cols; c += C) {
                        float v[C];
                        tmem_ld32(t + c, v);
                        if (c + C == cols) release(tc & 1);
                        step(c, v);
                    }
                    tc++;
                }
            }
        };
        if constexpr (EXACT) {
            run(float());
        } else {
            if (a.e.out_f32) run(float());
            else run(__nv_bfloat16());
        }
        if (lane == 0) bulk_wait();
    }
    __syncwarp();
    fence_before();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    fence_after();
    if (warp == 1) {
        if constexpr (CG == 2) tmem_dealloc_pair(tmem, Z::TMEM);
        else tmem_dealloc(tmem, Z::TMEM);
    }
}

// ------------------------------------------------------------------ host side

static void tile_counts(Shape s, long long M, long long N, int &mt, int &nt)
{
    const int bm = s == LONE_64 ? 128 : 256, bn = s == LONE_64 ? 64 : s == PAIR_128 ? 128 : 256;
    mt = (int)((M + bm - 1) / bm);
    nt = (int)((N + bn - 1) / bn);
}

// Tile and cut of the k axis by estimated time, of which this is the model (fitted to the timings of 20 products, from
// 37 x 2048 x 8192 to 2048^3 and 64 x 512 x 16384, with every tile and several cuts: its choice takes at most 15% more
// than the best of them, mostly 2%; us):
//   a stage of a unit: 128 x 64 and 256 x 128 tiles 0.20 (the loads), 256 x 256 0.28 (the MMAs' own 512 cycles); of three
//   planes, six products, 0.72 and 0.90;
//   a round is no shorter than its epilogue: 0.9, 1.7 and 2.9 (1.8 with 16 warps);
//   launch, first loads and last epilogue: 3.8, 5.2 and 6.3;
//   a cut k axis: another launch, 2.5, and the pieces' way to memory and back at 4 TB/s.
// A bf16 result's axis is cut into pieces of LONGEST at most, whatever that takes.
// Units run in rounds of one per SM or pair.
Plan plan_product(long long M, long long N, long long K, int planes, int passes, bool out_f32, int sms)
{
    const long long steps = (K + BK - 1) / BK * passes;
    // the registers hold half a row of 128 columns, not of 256
    Plan best = {PAIR_128, 1, planes == 3 || (out_f32 && steps > CHUNK_1)};
    const long long least_cut = best.exact ? 1 : (steps * BK + LONGEST - 1) / LONGEST;
    double least = 1e300;
    for (int s = LONE_64; s <= (best.exact ? PAIR_128 : PAIR_256); s++) {
        const Shape shape = (Shape)s;
        int mt, nt;
        tile_counts(shape, M, N, mt, nt);
        const double tiles = (double)mt * nt;
        const long long slots = shape == LONE_64 ? sms : sms / 2;
        constexpr double STEP[2][3] = {{0.20, 0.20, 0.28}, {0.72, 0.90, 0.0}}, FIXED[3] = {3.8, 5.2, 6.3}, EPILOGUE[3] = {0.9, 1.7, 2.9};
        const double step = STEP[planes == 3][s];
        for (long long cut = least_cut; cut <= steps && (cut == least_cut || (cut <= 64 && tiles * cut <= slots)); cut++) {
            const long long per = (steps + cut - 1) / cut, pieces = (steps + per - 1) / per;
            double rounds = floor(tiles * pieces / slots), rest = tiles * pieces - rounds * slots;
            if (rest > 0) rounds += shape == PAIR_256 && pieces == 1 && per > MANY_STEPS && rounds > 0 && 2 * rest <= slots ? 0.5 : 1.0;
            const double epilogue = shape == PAIR_256 && per <= MANY_STEPS ? 1.8 : EPILOGUE[s];
            double us = rounds * fmax(per * step, epilogue) + FIXED[s];
            if (pieces > 1) us += 2.5 + (double)M * N * 8 * pieces / 4e6;
            if (us < least) {
                least = us;
                best.shape = shape;
                best.splits = (int)pieces;
            }
        }
    }
    return best;
}

struct Maps {
    CUtensorMap a, b, half, out;
};

template <int CG, int BN, int P, int EW, bool EXACT, bool A_K, bool B_K, bool TWO = false>
static cudaError_t launch(const Maps &m, const Args &a, int sms, cudaStream_t st)
{
    using Z = Cfg<CG, BN, P, EW>;
    auto *kernel = linear_tc_kernel<CG, BN, P, EW, EXACT, A_K, B_K, TWO>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::SMEM);
    if (e != cudaSuccess) return e;
    const int slots = sms / CG;
    return launch_chained(kernel, dim3((unsigned)((a.units < slots ? a.units : slots) * CG)), Z::THREADS, Z::SMEM, CG, st, m.a, m.b, m.half, m.out, a);
}

template <int CG, int BN, int P, int EW, bool EXACT>
static cudaError_t launch_majors(const Product &p, const Maps &m, const Args &a, int sms, cudaStream_t st)
{
    if (p.a.k_major && p.b.k_major) return launch<CG, BN, P, EW, EXACT, true, true>(m, a, sms, st);
    if constexpr (P == 1 && !EXACT) {
        if (p.passes == 2 && p.a.k_major) return launch<CG, BN, P, EW, EXACT, true, false, true>(m, a, sms, st);
        if (p.passes == 2) return launch<CG, BN, P, EW, EXACT, false, false, true>(m, a, sms, st);
    }
    if constexpr (P == 3 || !EXACT) {  // gradients have their operands' type
        if (p.a.k_major) return launch<CG, BN, P, EW, EXACT, true, false>(m, a, sms, st);
        return launch<CG, BN, P, EW, EXACT, false, false>(m, a, sms, st);
    }
    return cudaErrorInvalidValue;
}
template <int CG, int BN>
static cudaError_t launch_planes(const Product &p, const Maps &m, const Args &a, int sms, cudaStream_t st)
{
    if constexpr (BN < 256) {
        if (p.planes == 3) return launch_majors<CG, BN, 3, 8, true>(p, m, a, sms, st);
        if (p.plan.exact) return launch_majors<CG, BN, 1, 8, true>(p, m, a, sms, st);
    }
    if constexpr (BN == 256) {
        if (a.many) return launch_majors<CG, BN, 1, 16, false>(p, m, a, sms, st);
    }
    return launch_majors<CG, BN, 1, 8, false>(p, m, a, sms, st);
}

// Boxes of `rows` m or n indices and 64 values of k of an operand with `n` of them.  {contiguous, strided, plane}; an
// m/n-contiguous operand of whole 64-wide blocks has these as an axis of their own (one copy then brings several).
static bool encode(CUtensorMap *m, const Operand &o, long long n, long long K, int planes, int rows, bool blocks)
{
    const long long inner = o.k_major ? K : n, outer = o.k_major ? n : K;
    // one plane: its stride is never used, but has to be a legal one (below 2^40 bytes)
    const long long far = 1LL << 38, whole = outer > far / o.ld ? far : outer * o.ld;
    const cuuint64_t ld = (cuuint64_t)o.ld * 2, plane = (cuuint64_t)(planes > 1 ? o.plane : whole) * 2;
    if (blocks) {
        const cuuint64_t dims[4] = {64, (cuuint64_t)K, (cuuint64_t)(n / 64), (cuuint64_t)planes}, strides[3] = {ld, 128, plane};
        const cuuint32_t box[4] = {64, 64, (cuuint32_t)(rows / 64), 1};
        return tc_encode_bf16(m, o.base, 4, dims, strides, box);
    }
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)planes}, strides[2] = {ld, plane};
    const cuuint32_t box[3] = {64, (cuuint32_t)(o.k_major ? rows : 64), 1};
    return tc_encode_bf16(m, o.base, 3, dims, strides, box);
}

// An output of M rows of n values, `ld` apart, z of them.
static bool encode_out(CUtensorMap *m, bool f32, const void *base, long long n, long long ld, long long M, int z)
{
    const long long size = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)n, (cuuint64_t)M, (cuuint64_t)z};
    const cuuint64_t strides[2] = {(cuuint64_t)(ld * size), (cuuint64_t)(M * ld * size)};
    return tc_encode_store(m, f32, base, dims, strides);
}

cudaError_t launch_product_tc(const Product &p, int sms, cudaStream_t st)
{
    const Shape s = p.plan.shape;
    const int splits = p.plan.splits;
    Args a = {};
    a.M = p.M;
    a.N = p.N;
    a.ksteps = (int)((p.K + BK - 1) / BK * p.passes);
    a.per_split = (a.ksteps + splits - 1) / splits;
    a.splits = splits;
    tile_counts(s, p.M, p.N, a.mt, a.nt);
    const long long units = (long long)a.mt * a.nt * splits, slots = sms / 2, rest = units % slots;
    if (units > 0x3fffffffLL || (long long)BAND * a.nt > 0x3fffffffLL) return cudaErrorInvalidConfiguration;
    a.units = a.whole = (int)units;
    // Up to 256 k a tile's epilogue is longer than its MMAs: 16 warps instead of 8, for a stage less and no half tiles
    // (8192 x 8192 x 128 33.7 -> 27.5 us, with bias, GELU and residual 97 -> 86; x 512 would go from 44.5 to 51).
    a.many = s == PAIR_256 && a.per_split <= MANY_STEPS;
    if (s == PAIR_256 && !a.many && splits == 1 && units > slots && rest > 0 && 2 * rest <= slots) {
        a.whole -= (int)rest;
        a.units += (int)rest;
    }
    a.e = p.e;
    a.ldo = p.N;
    if (splits > 1) {  // bare fp32 sums, piece by piece
        a.e = Epilogue();
        a.e.alpha = 1.f;
        a.e.out = p.e.partial;
        a.e.out_f32 = 1;
        a.ldo = partial_stride(p.N);
    }
    a.res32 = (reinterpret_cast<uintptr_t>(a.e.res) & 31) == 0 && a.e.ldr % (a.e.out_f32 ? 8 : 16) == 0;
    // a warp of the 128 x 64 tile has half a row of bf16 columns; a kept z off 16-byte rows needs the buffer for itself
    a.tma_out = s != LONE_64 && a.ldo % (a.e.out_f32 ? 4 : 8) == 0 &&
                (a.e.preact == nullptr || p.N % (a.e.preact_f32 ? 4 : 8) == 0);
    a.blocks_a = !p.a.k_major && p.M % 64 == 0;
    a.blocks_b = !p.b.k_major && p.N % 64 == 0;
    a.rows_a = p.M >= BM ? BM : p.a.k_major ? (int)((p.M + 7) & ~7LL) : p.M > 64 ? 128 : 64;
    Maps m = {};
    const int rows_b = s == PAIR_256 ? 128 : 64;
    bool ok = encode(&m.a, p.a, p.M, p.K, p.planes * p.passes, a.rows_a, a.blocks_a) && encode(&m.b, p.b, p.N, p.K, p.planes, rows_b, a.blocks_b);
    if (a.units > a.whole) ok = ok && encode(&m.half, p.b, p.N, p.K, p.planes, rows_b / 2, a.blocks_b);
    if (a.tma_out) ok = ok && encode_out(&m.out, a.e.out_f32, a.e.out, p.N, a.ldo, p.M, splits);
    if (!ok) return cudaErrorInvalidValue;
    if (s == LONE_64) return launch_planes<1, 64>(p, m, a, sms, st);
    if (s == PAIR_128) return launch_planes<2, 128>(p, m, a, sms, st);
    return launch_planes<2, 256>(p, m, a, sms, st);
}

}  // namespace linear
}  // namespace csa
