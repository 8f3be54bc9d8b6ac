// k_linear_tc.cuh -- the kernel of the projections' products and its launch (k_linear_tc.cu tells how it works and was chosen).  A
// file that includes this has an error word of its own.
#pragma once

#include "k_linear_pipe.cuh"

namespace csa {

static __device__ int g_lin_error = 0;

namespace linear {

constexpr long long LONGEST = 65536;  // k that a bf16 result sums in one accumulator
constexpr int CHUNK_1 = 8;     // stages (512 k) that an fp32 result of one plane does
constexpr int MANY_STEPS = 4;  // stages of a unit up to which 256-wide tiles have 16 epilogue warps

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
// stages take turns (B's second one comes from L2).  DYNAMIC: rows or k are counted on the device.  (As an argument instead, it cost a product of 37 rows 0.7 us of 11.6.)
template <int CG, int BN, int P, int EW, bool EXACT, bool A_K, bool B_K, bool TWO, bool DYNAMIC>
__global__ void __launch_bounds__(64 + 32 * EW, 1)
linear_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ CUtensorMap map_half, const __grid_constant__ CUtensorMap map_out, const Args args)
{
    using Z = Cfg<CG, BN, P, EW>;
    constexpr int CHUNK = !EXACT ? 0x40000000 : P == 3 ? 1 : CHUNK_1;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_align1024(smem_raw);
    using Pipe = Pipeline<CG, BN, P, EW, CHUNK>;
    const Pipe p(smem, &g_lin_error, 600);
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
        p.template produce<A_K, B_K, TWO>(map_a, map_b, map_half, a);
    } else if (warp == 1) {
        p.template issue<A_K, B_K>(tmem, a);
    } else {
        // ---------------------------------------------------------- epilogue (8 or 16 warps)
        const int quad = warp & 3;               // TMEM lanes this warp may access
        const int side = (warp - 2) >> 2;        // part of the columns
        const uint32_t rank = p.rank;
        const Buffer b = {smem + Z::TURN + (warp - 2) * 4096, lane};
        // asked once: each of these questions cost a step a miss in the constant and instruction caches
        const bool tma = a.tma_out != 0, with_res = a.e.res != nullptr, with_bias = a.e.bias != nullptr, with_act = a.e.act != CSA_ACT_NONE || a.e.preact != nullptr;
        const float alpha = a.e.alpha;
        auto run = [&](auto type) {
            using O = decltype(type);
            int tc = 0;
            for (int u = p.u0; u < a.units; u += p.ustep) {
                const Unit x = unit_of<BN>(a, u);
                const int cols = x.bn / (EW / 4);
                const long long m0 = ((long long)x.m * CG + rank) * BM + quad * 32, nb = x.n0 + side * cols;
                const auto wait = [&] {
                    p.wait_sums(tc);
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
                    if (a.e.scale != nullptr) {
                        const float f = __ldg(a.e.scale);
#pragma unroll
                        for (int k = 0; k < C; k++) v[k] *= f;
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
                            if (g == G - 1) p.release_sums(tc);
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
                        if (c + C == cols) p.release_sums(tc);
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
    p.end(tmem);
}

// ------------------------------------------------------------------ host side

template <int CG, int BN, int P, int EW, bool EXACT, bool A_K, bool B_K, bool TWO = false, bool DYNAMIC = false>
static cudaError_t launch(const Maps &m, const Args &a, int sms, cudaStream_t st)
{
    using Z = Cfg<CG, BN, P, EW>;
    auto *kernel = linear_tc_kernel<CG, BN, P, EW, EXACT, A_K, B_K, TWO, DYNAMIC>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::SMEM);
    if (e != cudaSuccess) return e;
    const int slots = sms / CG;
    return launch_chained(kernel, dim3((unsigned)((a.units < slots ? a.units : slots) * CG)), Z::THREADS, Z::SMEM, CG, st, m.a, m.b, m.half, m.out, a);
}

// A product's arguments and tensor maps.
inline cudaError_t describe(const Product &p, int sms, Args &a, Maps &m)
{
    const Shape s = p.plan.shape;
    const int splits = p.plan.splits;
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
    a.blocks_a = !p.a.k_major && (p.a.held > p.M ? p.a.held : p.M) % 64 == 0;
    a.blocks_b = !p.b.k_major && p.N % 64 == 0;
    a.rows_a = p.M >= BM ? BM : p.a.k_major ? (int)((p.M + 7) & ~7LL) : p.M > 64 ? 128 : 64;
    const int rows_b = s == PAIR_256 ? 128 : 64;
    bool ok = encode(&m.a, p.a, p.M, p.K, p.planes * p.passes, a.rows_a, a.blocks_a) && encode(&m.b, p.b, p.N, p.K, p.planes, rows_b, a.blocks_b);
    if (a.units > a.whole) ok = ok && encode(&m.half, p.b, p.N, p.K, p.planes, rows_b / 2, a.blocks_b);
    if (a.tma_out) ok = ok && encode_out(&m.out, a.e.out_f32, a.e.out, p.N, a.ldo, p.M, splits);
    return ok ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace linear
}  // namespace csa
