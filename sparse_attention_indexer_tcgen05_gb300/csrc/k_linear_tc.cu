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
#include "k_linear_tc.cuh"

#include <cuda.h>
#include <math.h>

namespace csa {

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

// ------------------------------------------------------------------ host side

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

cudaError_t launch_product_tc(const Product &p, int sms, cudaStream_t st)
{
    Args a = {};
    Maps m = {};
    const cudaError_t e = describe(p, sms, a, m);
    if (e != cudaSuccess) return e;
    const Shape s = p.plan.shape;
    if (s == LONE_64) return launch_planes<1, 64>(p, m, a, sms, st);
    if (s == PAIR_128) return launch_planes<2, 128>(p, m, a, sms, st);
    return launch_planes<2, 256>(p, m, a, sms, st);
}

}  // namespace linear
}  // namespace csa
