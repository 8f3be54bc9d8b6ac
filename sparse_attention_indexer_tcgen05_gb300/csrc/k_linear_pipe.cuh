// k_linear_pipe.cuh -- what the kernels that run products on tcgen05 share: tiles and their order, the TMA producer, the MMA
// issue and the barriers between them and the epilogue's warps (k_linear_tc.cu tells how they were chosen).
//
// A unit is one output tile and one piece of the k axis.  A CTA pair (two SMs) computes 256 x BN: each CTA loads its 128 rows
// of A and its BN / 2 rows of B, so an operand byte brought to an SM feeds twice the MMAs of a lone CTA's 128 x BN tile.
// Roles: warp 0 the TMA producer, warp 1 the MMA issue (the pair's even CTA), the others the epilogue, a row of the tile a
// lane.  TMEM holds two accumulators, so that a tile's epilogue runs under the next tile's MMAs.
#pragma once

#include "csa_tc.cuh"
#include "k_linear.cuh"
#include "tc_ptx.cuh"

#include <cuda.h>

namespace csa {
namespace linear {

using namespace ptx;

constexpr int BM = 128;        // rows of one CTA's accumulator
constexpr int BK = 64;         // k per stage: one 128-byte swizzle row

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
    // A number of rows (of M, or of k) that is known on the device alone: `counted` rows before `first` are another product's.  With
    // `along_k` the k axis ends there, with whole stages (what lies behind the last row is zeros); never empty for the first.
    const int *counted;
    long long first;
    int along_k;
};

// The arguments with the device's count in them; `bm` rows of a tile.
__device__ __forceinline__ Args counted(const Args &given, int bm)
{
    Args a = given;
    long long n = *a.counted - a.first;
    if (a.along_k) {
        const long long most = (long long)a.ksteps * BK;
        n = n < 0 ? 0 : n > most ? most : n;
        if (n == 0 && a.first > 0) a.units = a.whole = 0;   // nothing to add
        a.ksteps = a.per_split = n > 0 ? (int)((n + BK - 1) / BK) : 1;
    } else {
        a.M = n < 0 ? 0 : n > a.M ? a.M : n;
        a.mt = (int)((a.M + bm - 1) / bm);
        a.units = a.whole = a.mt * a.nt * a.splits;
    }
    return a;
}

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

constexpr int C = 32;   // columns of an epilogue step


__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A warp's 32 rows x 32 columns, a row a lane, to memory by TMA, from rows of 128 bytes in shared memory (32 fp32 columns, or
// 64 bf16 ones: two steps), so that a
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

// One CTA's part in the products of a grid.  Every thread makes one, calls begin(), does what its warp does, and end().  CHUNK:
// stages of the k axis that an accumulator sums before it is handed to the epilogue.
template <int CG, int BN, int P, int EW, int CHUNK> struct Pipeline {
    using Z = Cfg<CG, BN, P, EW>;
    static constexpr int S = Z::STAGES;
    unsigned char *smem;
    uint64_t *full, *empty, *t_full, *t_empty, *done;
    uint32_t *tmem_slot;
    volatile int *abort_flag;
    int *err, site;              // the kernel's error word and the first of its wait sites
    int warp, lane, u0, ustep;
    uint32_t rank;

    __device__ __forceinline__ Pipeline(unsigned char *base, int *error, int first_site) : smem(base), err(error), site(first_site)
    {
        uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Z::MISC);
        full = bars;
        empty = bars + S;
        t_full = bars + 2 * S;
        t_empty = bars + 2 * S + 2;
        done = bars + 2 * S + 4;
        tmem_slot = reinterpret_cast<uint32_t *>(smem + Z::MISC + 256);
        abort_flag = reinterpret_cast<volatile int *>(smem + Z::MISC + 264);
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        rank = CG == 2 ? cluster_rank() : 0u;
        u0 = blockIdx.x / CG;
        ustep = gridDim.x / CG;
    }

    // Barriers and TMEM; returns the accumulators' address.
    __device__ __forceinline__ uint32_t begin() const
    {
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
        return *tmem_slot;
    }

    __device__ __forceinline__ void end(uint32_t tmem) const
    {
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

    // The epilogue's side of accumulator number `tc`: its sums are there; they are in registers, and the next MMAs may have it.
    __device__ __forceinline__ void wait_sums(int tc) const
    {
        wait_bar(t_full + (tc & 1), (tc >> 1) & 1, abort_flag, err, site + 4);
        fence_after();
    }
    __device__ __forceinline__ void release_sums(int tc) const
    {
        fence_before();
        __syncwarp();
        if (lane == 0) {
            if constexpr (CG == 2) mbar_arrive_cluster(map_rank(t_empty + (tc & 1), 0));
            else mbar_arrive(t_empty + (tc & 1));
        }
    }

    // The TMA producer (warp 0).  Few and large copies: with B in two boxes of 64 rows instead of one of 128 the same product
    // took 164 us instead of 150 (8192 x 8192 x 2048).
    template <bool A_K, bool B_K, bool TWO>
    __device__ __forceinline__ void produce(const CUtensorMap &map_a, const CUtensorMap &map_b, const CUtensorMap &map_half, const Args &a) const
    {
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
                    wait_bar(empty + st, ph ^ 1, abort_flag, err, site + 1);
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
                if (rank == 0) drain_bar(full + i, i < st ? ph : ph ^ 1, err);
                drain_bar(empty + i, i < st ? ph : ph ^ 1, err);
            }
        }
    }

    // The MMA issue (the whole of warp 1, the pair's even CTA).
    template <bool A_K, bool B_K> __device__ __forceinline__ void issue(uint32_t tmem, const Args &a) const
    {
        if (rank == 0) {
            int st = 0, tc = 0;
            uint32_t ph = 0;
            for (int u = u0; u < a.units; u += ustep) {
                const Unit x = unit_of<BN>(a, u);
                const uint32_t idesc = x.bn == BN ? idesc_bf16(BM * CG, BN, !A_K, !B_K) : idesc_bf16(BM * CG, BN / 2, !A_K, !B_K);
                for (int it0 = x.it0; it0 < x.it1; it0 += min(CHUNK, x.it1 - it0)) {
                    const int it1 = min(CHUNK, x.it1 - it0) + it0, tb = tc & 1;
                    wait_bar(t_empty + tb, ((tc >> 1) & 1) ^ 1, abort_flag, err, site + 2);
                    fence_after();
                    const uint32_t d = tmem + (uint32_t)(tb * BN);
                    for (int it = it0; it < it1; it++) {
                        wait_bar(full + st, ph, abort_flag, err, site + 3);
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
        drain_bar(done, 0, err);  // in either CTA: the commit arrives in both
    }
};

// ------------------------------------------------------------------ host side

struct Maps {
    CUtensorMap a, b, half, out;
};

inline void tile_counts(Shape s, long long M, long long N, int &mt, int &nt)
{
    const int bm = s == LONE_64 ? 128 : 256, bn = s == LONE_64 ? 64 : s == PAIR_128 ? 128 : 256;
    mt = (int)((M + bm - 1) / bm);
    nt = (int)((N + bn - 1) / bn);
}

// Boxes of `rows` m or n indices and 64 values of k of an operand with `n` of them.  {contiguous, strided, plane}; an
// m/n-contiguous operand of whole 64-wide blocks has these as an axis of their own (one copy then brings several).
inline bool encode(CUtensorMap *m, const Operand &o, long long n, long long K, int planes, int rows, bool blocks)
{
    if (o.held > n) n = o.held;
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
inline bool encode_out(CUtensorMap *m, bool f32, const void *base, long long n, long long ld, long long M, int z)
{
    const long long size = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)n, (cuuint64_t)M, (cuuint64_t)z};
    const cuuint64_t strides[2] = {(cuuint64_t)(ld * size), (cuuint64_t)(M * ld * size)};
    return tc_encode_store(m, f32, base, dims, strides);
}

}  // namespace linear
}  // namespace csa
