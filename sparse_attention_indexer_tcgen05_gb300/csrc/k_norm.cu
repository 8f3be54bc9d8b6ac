// k_norm.cu -- layer norm of rows and its gradients.
//
//   mean = sum_j x_j / n,  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / n + eps),  h_j = (x_j - mean) rstd,  y_j = h_j w_j + b_j
//   a_j = dy_j w_j,  dx_j = rstd (a_j - mean(a) - h_j mean(a h)),  dw_j = sum over rows of dy_j h_j,  db_j = sum of dy_j
//
// Bound by memory: x read and y written once (backward: x and dy read, dx written).  The variance is a second pass over the row
// where it lies (registers or shared memory), not a difference of two large sums.  The backward's threads keep their columns over all the
// rows that their block takes, and so the gradients of their weights; the blocks' sums are joined in a fixed order by a
// second kernel: the same bits every time.
//
// Rows of up to 512 values lie in the registers of a part of a warp.  Longer ones pass through a ring of rows in a block's
// shared memory, filled by asynchronous copies, in steps: while a row's sum is taken, the row before it is a step further,
// so that no step waits for a sum across the block and a row costs one barrier.
//
// Measured (GB/s of the bytes above; a plain copy moves 6795): bf16 65536 x 4096 forward 5500, backward 5900 (272 us), 65536 x 1024 backward
// 4850; fp32 4096 x 4096 5700 and 5300; 5003 x
// 1537 fp32 backward 27 us, 16384 x 128 bf16 forward 3.2 and backward 7.6 us, 1 x 4096 forward 2.2 us on the device.
#include "k_linear.cuh"

#include <type_traits>

namespace csa {
namespace norm {

using bf16 = __nv_bfloat16;
using linear::chain_start;
using linear::chain_wait;
using linear::launch_chained;
using ptx::add2;
using ptx::fma2;
using ptx::mul2;

__device__ __forceinline__ float from_value(float x) { return x; }
__device__ __forceinline__ float from_value(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A piece of a row: the neighbouring values of 16 bytes, as they lie in memory and as pairs
template <typename T> constexpr int PER = 16 / (int)sizeof(T);
template <typename T> struct Piece;
template <> struct Piece<bf16> {
    uint4 r;
    __device__ __forceinline__ void load(const void *p) { r = *static_cast<const uint4 *>(p); }
    __device__ __forceinline__ void pairs(float2 (&x)[4]) const
    {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; k++) x[k] = make_float2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u));
    }
};
template <> struct Piece<float> {
    uint4 r;
    __device__ __forceinline__ void load(const void *p) { r = *static_cast<const uint4 *>(p); }
    __device__ __forceinline__ void pairs(float2 (&x)[2]) const
    {
        x[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
        x[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
    }
};
__device__ __forceinline__ void store_pairs(bf16 *p, const float2 (&x)[4])
{
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[k].x, x[k].y);
        u[k] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store_pairs(float *p, const float2 (&x)[2])
{
    *reinterpret_cast<float4 *>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
}
// H pairs of a parameter, of either type
template <int H> __device__ __forceinline__ void load_pairs(const float *p, float2 (&x)[H])
{
#pragma unroll
    for (int k = 0; k < H; k += 2) {
        const float4 v = *reinterpret_cast<const float4 *>(p + 2 * k);
        x[k] = make_float2(v.x, v.y);
        x[k + 1] = make_float2(v.z, v.w);
    }
}
template <int H> __device__ __forceinline__ void load_pairs(const bf16 *p, float2 (&x)[H])
{
#pragma unroll
    for (int k = 0; k < H; k += 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p + 2 * k);
        x[k] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
        x[k + 1] = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
    }
}

// The columns of a thread: pieces, as they lie in the aligned vectors of memory.  SHIFT: rows of a block
// (or of a part of a warp) start `shift` values behind a 16-byte boundary, all of them the same, because the rows that it takes
// are a multiple of 8 apart; the vectors at a row's ends hold columns that are not its own.  So rows of any length
// move in whole vectors (value by value, 5003 x 1537 in fp32 took 62 us backward).
template <typename T, int LANES, bool SHIFT> struct Columns {
    static constexpr int H = PER<T> / 2;
    int n, shift, t;
    __device__ __forceinline__ int first(int c) const { return (c * LANES + t) * PER<T> - (SHIFT ? shift : 0); }
    __device__ __forceinline__ bool has(int c) const { return first(c) < n; }
    __device__ __forceinline__ bool full(int c) const { return !SHIFT || (first(c) >= 0 && first(c) + PER<T> <= n); }
    // 0 where columns are not the row's
    __device__ __forceinline__ void clip(float2 (&x)[H], int c) const
    {
        if (full(c)) return;
        const int j = first(c);
#pragma unroll
        for (int k = 0; k < H; k++) {
            if ((unsigned)(j + 2 * k) >= (unsigned)n) x[k].x = 0.f;
            if ((unsigned)(j + 2 * k + 1) >= (unsigned)n) x[k].y = 0.f;
        }
    }
    __device__ __forceinline__ void store(T *row, int c, const float2 (&x)[H]) const
    {
        const int j = first(c);
        if (full(c)) {
            store_pairs(row + j, x);
            return;
        }
#pragma unroll
        for (int k = 0; k < H; k++) {
            if ((unsigned)(j + 2 * k) < (unsigned)n) row[j + 2 * k] = from_f<T>(x[k].x);
            if ((unsigned)(j + 2 * k + 1) < (unsigned)n) row[j + 2 * k + 1] = from_f<T>(x[k].y);
        }
    }
    // a parameter, of either type (as scalars they took longer than the rows: 65536 x 4096 forward 603 us)
    __device__ __forceinline__ void param(const void *p, int f32, int c, float missing, float2 (&w)[H]) const
    {
#pragma unroll
        for (int k = 0; k < H; k++) w[k] = both(missing);
        if (p == nullptr || !has(c)) return;
        const int j = first(c);
        if constexpr (SHIFT) {
            const auto at = [&](int i) {
                if ((unsigned)i >= (unsigned)n) return 0.f;
                return f32 ? __ldg(static_cast<const float *>(p) + i) : __bfloat162float(static_cast<const bf16 *>(p)[i]);
            };
#pragma unroll
            for (int k = 0; k < H; k++) w[k] = make_float2(at(j + 2 * k), at(j + 2 * k + 1));
        } else if (f32) {
            load_pairs(static_cast<const float *>(p) + j, w);
        } else {
            load_pairs(static_cast<const bf16 *>(p) + j, w);
        }
    }
};
// Values between a row's start and the 16-byte boundary before it
template <typename T> __device__ __forceinline__ int shift_of(long long r, long long stride) { return (int)(r * stride & (16 / sizeof(T) - 1)); }

// The piece at p that may lie across an argument's `end`: nothing from there on is read.
template <typename T> __device__ __forceinline__ void load_piece(Piece<T> &e, const T *p, const T *end)
{
    if (p + PER<T> <= end) e.load(p);
    else e.r = linear::load16(reinterpret_cast<const uint4 *>(p), end);
}

template <int H> __device__ __forceinline__ float sum_of(const float2 (&x)[H])
{
    float2 s = add2(x[0], x[1]);
    if constexpr (H == 4) s = add2(s, add2(x[2], x[3]));
    return s.x + s.y;
}
template <int H> __device__ __forceinline__ float dot_of(const float2 (&x)[H], const float2 (&y)[H])
{
    float2 s = mul2(x[0], y[0]);
#pragma unroll
    for (int k = 1; k < H; k++) s = fma2(x[k], y[k], s);
    return s.x + s.y;
}
template <int LANES> __device__ __forceinline__ float lane_sum(float s)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

struct Fwd {
    const void *x, *weight, *bias;
    void *y;
    float *stats;               // [2][rows] or null
    long long rows, stride;
    int n, param_f32;
    float eps;
};
struct Bwd {
    const void *dy, *x, *weight;
    const float *stats;
    void *dx;
    float *parts;               // [blocks][2][n]: the blocks' sums of dw and db; null: neither is asked for
    long long rows, x_stride, dy_stride;
    int n, param_f32;
};

// ------------------------------------------------------------------ rows of up to 512 values

// Rows off the 16-byte boundaries clip the vectors at their ends and store them value by value; with two pieces the forward takes 222
// registers (fp32 248), one block an SM.  2^20 rows in bf16, forward and backward: 256 values 203 and 285 us, 249 326 and 377, 255 (two
// pieces, half of them empty) 836 and 777.
constexpr int U = 2;   // rows of a thread on their way at a time

template <typename T, int LANES, int EIGHTS, bool SHIFT> __global__ void __launch_bounds__(256, sizeof(T) == 2 && EIGHTS == 1 ? 4 : 1) norm_fwd_short_kernel(const Fwd a)
{
    constexpr int C = EIGHTS * 8 / PER<T>, H = PER<T> / 2;
    constexpr int R = 256 / LANES;   // a multiple of 8, as is the grid times it: the shift is the group's own
    chain_start();
    chain_wait();
    const int group = threadIdx.x / LANES;
    const Columns<T, LANES, SHIFT> cols = {a.n, shift_of<T>(group, a.stride), (int)threadIdx.x % LANES};
    const T *end = static_cast<const T *>(a.x) + (a.rows - 1) * a.stride + a.n;
    const float inv_n = 1.f / (float)a.n;
    float2 w[C][H], b[C][H];
    bool loaded = false;
    for (long long r0 = (long long)blockIdx.x * R * U; r0 < a.rows; r0 += (long long)gridDim.x * R * U) {
        Piece<T> raw[U][C];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const long long r = r0 + u * R + group;
            const T *row = static_cast<const T *>(a.x) + r * a.stride;
#pragma unroll
            for (int c = 0; c < C; c++) {
                raw[u][c] = Piece<T>();
                if (r < a.rows && cols.has(c)) load_piece(raw[u][c], row + cols.first(c), end);
            }
        }
        if (!loaded) {
#pragma unroll
            for (int c = 0; c < C; c++) {
                cols.param(a.weight, a.param_f32, c, 1.f, w[c]);
                cols.param(a.bias, a.param_f32, c, 0.f, b[c]);
            }
            loaded = true;
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const long long r = r0 + u * R + group;
            float2 x[C][H];
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < C; c++) {
                raw[u][c].pairs(x[c]);
                cols.clip(x[c], c);
                s += sum_of(x[c]);
            }
            const float mean = lane_sum<LANES>(s) * inv_n;
            s = 0.f;
#pragma unroll
            for (int c = 0; c < C; c++) {
#pragma unroll
                for (int k = 0; k < H; k++) x[c][k] = add2(x[c][k], both(-mean));
                cols.clip(x[c], c);
                if (cols.has(c)) s += dot_of(x[c], x[c]);
            }
            const float rstd = 1.f / sqrtf(lane_sum<LANES>(s) * inv_n + a.eps);
            if (r >= a.rows) continue;
#pragma unroll
            for (int c = 0; c < C; c++) {
#pragma unroll
                for (int k = 0; k < H; k++) x[c][k] = fma2(mul2(x[c][k], both(rstd)), w[c][k], b[c][k]);
                if (cols.has(c)) cols.store(static_cast<T *>(a.y) + r * a.n, c, x[c]);
            }
            if (a.stats != nullptr && cols.t == 0) {
                a.stats[r] = mean;
                a.stats[a.rows + r] = rstd;
            }
        }
    }
}

template <typename T, int LANES, int EIGHTS, bool SHIFT> __global__ void __launch_bounds__(256, EIGHTS == 1 ? 3 : 2) norm_bwd_short_kernel(const Bwd a)
{
    constexpr int C = EIGHTS * 8 / PER<T>, H = PER<T> / 2, R = 256 / LANES;
    __shared__ float across[R][2][LANES * EIGHTS * 8];
    chain_start();
    chain_wait();
    const int group = threadIdx.x / LANES;
    const Columns<T, LANES, SHIFT> cols = {a.n, shift_of<T>(group, a.x_stride), (int)threadIdx.x % LANES};
    const T *end_x = static_cast<const T *>(a.x) + (a.rows - 1) * a.x_stride + a.n, *end_d = static_cast<const T *>(a.dy) + (a.rows - 1) * a.dy_stride + a.n;
    const float inv_n = 1.f / (float)a.n;
    float2 w[C][H], dw[C][H], db[C][H];
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int k = 0; k < H; k++) dw[c][k] = db[c][k] = both(0.f);
    bool loaded = false;
    for (long long r0 = (long long)blockIdx.x * R * U; r0 < a.rows; r0 += (long long)gridDim.x * R * U) {
        Piece<T> rx[U][C], rd[U][C];
        float mean[U], rstd[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const long long r = r0 + u * R + group;
            const bool live = r < a.rows;
#pragma unroll
            for (int c = 0; c < C; c++) {
                rx[u][c] = rd[u][c] = Piece<T>();
                if (live && cols.has(c)) {
                    load_piece(rx[u][c], static_cast<const T *>(a.x) + r * a.x_stride + cols.first(c), end_x);
                    load_piece(rd[u][c], static_cast<const T *>(a.dy) + r * a.dy_stride + cols.first(c), end_d);
                }
            }
            mean[u] = live ? __ldg(a.stats + r) : 0.f;
            rstd[u] = live ? __ldg(a.stats + a.rows + r) : 0.f;
        }
        if (!loaded) {
#pragma unroll
            for (int c = 0; c < C; c++) cols.param(a.weight, a.param_f32, c, 1.f, w[c]);
            loaded = true;
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const long long r = r0 + u * R + group;
            float2 h[C][H], d[C][H];
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int c = 0; c < C; c++) {
                rx[u][c].pairs(h[c]);
                rd[u][c].pairs(d[c]);
                cols.clip(h[c], c);   // what lies beside the row need not be finite
                cols.clip(d[c], c);   // d is 0 where there is no row or column
#pragma unroll
                for (int k = 0; k < H; k++) {
                    h[c][k] = mul2(add2(h[c][k], both(-mean[u])), both(rstd[u]));
                    dw[c][k] = fma2(d[c][k], h[c][k], dw[c][k]);
                    db[c][k] = add2(db[c][k], d[c][k]);
                    d[c][k] = mul2(d[c][k], w[c][k]);
                }
                s0 += sum_of(d[c]);
                s1 += dot_of(d[c], h[c]);
            }
            if (a.dx == nullptr) continue;
            const float ma = lane_sum<LANES>(s0) * inv_n, mh = lane_sum<LANES>(s1) * inv_n;
            if (r >= a.rows) continue;
#pragma unroll
            for (int c = 0; c < C; c++) {
#pragma unroll
                for (int k = 0; k < H; k++) h[c][k] = mul2(both(rstd[u]), fma2(h[c][k], both(-mh), add2(d[c][k], both(-ma))));
                if (cols.has(c)) cols.store(static_cast<T *>(a.dx) + r * a.n, c, h[c]);
            }
        }
    }
    if (a.parts == nullptr) return;
    // by column: the groups' shifts differ
    if constexpr (SHIFT) {
        for (int i = threadIdx.x; i < R * 2 * LANES * EIGHTS * 8; i += 256) (&across[0][0][0])[i] = 0.f;
        __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < C; c++) {
#pragma unroll
        for (int k = 0; k < PER<T>; k++) {
            const int j = cols.first(c) + k;
            if ((unsigned)j < (unsigned)a.n) {
                across[group][0][j] = k % 2 == 0 ? dw[c][k / 2].x : dw[c][k / 2].y;
                across[group][1][j] = k % 2 == 0 ? db[c][k / 2].x : db[c][k / 2].y;
            }
        }
    }
    __syncthreads();
    float *out = a.parts + (long long)blockIdx.x * 2 * a.n;
    for (int i = threadIdx.x; i < 2 * a.n; i += 256) {
        const int which = i >= a.n, j = i - which * a.n;
        float v = 0.f;
#pragma unroll 16
        for (int g = 0; g < R; g++) v += across[g][which][j];
        out[i] = v;
    }
}

// ------------------------------------------------------------------ longer rows: several warps a row

// The first `bytes` of 16, zeros behind them, as one asynchronous copy
__device__ __forceinline__ void cp_async16_part(void *dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::su32(dst)), "l"(src), "r"(bytes) : "memory");
}

constexpr int HELD = 16;   // values of a thread

// Rows of an argument on their way through shared memory, a thread's own pieces by its own copies: no thread reads what
// another one copied.  Copies are of 16 bytes, up to the argument's last value; a warp's are neighbours.  (Pieces of 8 values in fp32
// too, two copies each with 16 bytes left out between threads: 4096 x 4096 forward 38 us, 23 so, backward 56 and 38.)
template <typename T, int LANES, bool SHIFT> struct Ring {
    static constexpr int C = HELD / PER<T>, H = PER<T> / 2;
    const T *at, *end;      // the thread's place in the next row that is asked for; the argument's end
    long long step;         // from row to row
    __device__ __forceinline__ Ring(const void *x, long long stride, long long rows, long long first, long long apart, const Columns<T, LANES, SHIFT> &cols)
        : at(static_cast<const T *>(x) + first * stride + cols.first(0)), end(static_cast<const T *>(x) + (rows - 1) * stride + cols.n),
          step(apart * stride)
    {
    }
    __device__ __forceinline__ void ask(const Columns<T, LANES, SHIFT> &cols, unsigned char *to)
    {
#pragma unroll
        for (int c = 0; c < C; c++) {
            if (cols.has(c)) {
                const T *p = at + c * LANES * PER<T>;
                unsigned char *q = to + (c * LANES + cols.t) * 16;
                if (!SHIFT || p + PER<T> <= end) {
                    ptx::cp_async16(q, p);
                } else {
                    const int left = (int)(end - p) * (int)sizeof(T);
                    cp_async16_part(q, p, left < 0 ? 0 : left);
                }
            }
        }
        at += step;
    }
    static __device__ __forceinline__ void take(const Columns<T, LANES, SHIFT> &cols, const unsigned char *from, int c, float2 (&x)[H])
    {
        Piece<T> e;
        e.load(from + (c * LANES + cols.t) * 16);
        e.pairs(x);
    }
    // What lies beside a row in its first and last vectors becomes 0, once, where it has arrived: it may be anything.
    static __device__ __forceinline__ void clean(const Columns<T, LANES, SHIFT> &cols, unsigned char *from)
    {
        if constexpr (SHIFT) {
#pragma unroll
            for (int c = 0; c < C; c++) {
                if (!cols.has(c) || cols.full(c)) continue;
                T *q = reinterpret_cast<T *>(from + (c * LANES + cols.t) * 16);
                const int j = cols.first(c);
#pragma unroll
                for (int k = 0; k < PER<T>; k++)
                    if ((unsigned)(j + k) >= (unsigned)cols.n) q[k] = from_f<T>(0.f);
            }
        }
    }
};

__device__ __forceinline__ void wait_copies(int pending)   // all but that many of the latest groups
{
    switch (pending) {
    case 0: ptx::cp_async_wait<0>(); break;
    case 1: ptx::cp_async_wait<1>(); break;
    case 2: ptx::cp_async_wait<2>(); break;
    default: ptx::cp_async_wait<3>(); break;
    }
}
constexpr int MOST_PENDING = 3;

// Sums of two values over a warp: lanes 0 to 15 get a's, the others b's.
__device__ __forceinline__ float warp_sum2(float a, float b)
{
    const bool low = (threadIdx.x & 16) == 0;
    float s = (low ? a : b) + __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
// Two sums over the W warps' parts, for every thread; parts up to the next power of two hold 0.
template <int W> __device__ __forceinline__ void group_sum2(const float (&part)[2][32], float &a, float &b)
{
    const int lane = threadIdx.x & 31;
    float s = part[lane >> 4][lane & 15];
    if constexpr (W > 16) s += part[lane >> 4][16 + (lane & 15)];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        if (o < W) s += __shfl_xor_sync(0xffffffffu, s, o);
    a = __shfl_sync(0xffffffffu, s, 0);
    b = __shfl_sync(0xffffffffu, s, 16);
}

// One block an SM, of several groups of LANES threads, each of which takes rows of its own (with a block for each, 1824 blocks
// left 15 MB of sums for 16384 rows of 1000).  What a group needs of this:
template <int LANES> struct Group {
    int index, t, warp, lane;
    long long first, apart;     // its first row, from there to its next one
    int count;                  // its rows
    __device__ __forceinline__ Group(long long rows)
    {
        index = threadIdx.x / LANES;
        t = threadIdx.x - index * LANES;
        warp = t >> 5;
        lane = t & 31;
        first = (long long)index * gridDim.x + blockIdx.x;
        apart = (long long)(blockDim.x / LANES) * gridDim.x;
        count = first < rows ? (int)((rows - first + apart - 1) / apart) : 0;
    }
    __device__ __forceinline__ void sync() const { ptx::named_bar(1 + index, LANES); }
};
// Threads of a block: backward 512 of 128 registers (768 of 80 spilled: 65536 x 4096 636 us instead of 281), forward 768
__host__ __device__ constexpr int most_threads(int lanes, bool backward) { return lanes > 512 ? 1024 : backward ? 512 : 768; }
constexpr int GROUPS = 12;

// Step i: the sum of row i, the squared differences of row i - 1, the result of row i - 2.
template <typename T, int LANES, bool SHIFT> __global__ void __launch_bounds__(most_threads(LANES, false), 1) norm_fwd_ring_kernel(const Fwd a, int stages)
{
    extern __shared__ __align__(16) unsigned char ring[];   // [groups][stages][room]
    __shared__ float parts[GROUPS][2][2][32];
    chain_start();
    chain_wait();
    const Group<LANES> g(a.rows);
    const Columns<T, LANES, SHIFT> cols = {a.n, shift_of<T>(g.first, a.stride), g.t};
    using Rows = Ring<T, LANES, SHIFT>;
    Rows rows(a.x, a.stride, a.rows, g.first, g.apart, cols);
    constexpr int C = Rows::C, H = Rows::H, room = LANES * HELD * (int)sizeof(T);
    const int count = g.count;
    unsigned char *const ring_start = ring + g.index * stages * room, *const ring_end = ring_start + stages * room;
    const auto next = [&](unsigned char *p) { return p + room == ring_end ? ring_start : p + room; };
    unsigned char *fresh = ring_start;
    int asked = 0;
    const auto ask = [&] {
        if (asked < count) rows.ask(cols, fresh);
        ptx::cp_async_commit();
        fresh = next(fresh);
        asked++;
    };
    for (int i = 0; i < stages - 3; i++) ask();
    float2 w[C][H], b[C][H];
#pragma unroll
    for (int c = 0; c < C; c++) {
        cols.param(a.weight, a.param_f32, c, 1.f, w[c]);
        cols.param(a.bias, a.param_f32, c, 0.f, b[c]);
    }
    for (int i = threadIdx.x; i < GROUPS * 128; i += blockDim.x) (&parts[0][0][0][0])[i] = 0.f;
    __syncthreads();
    float(*const part)[2][32] = parts[g.index];
    const float inv_n = 1.f / (float)a.n;
    unsigned char *p0 = ring_start, *p1 = ring_start, *p2 = ring_start;
    float mean1 = 0.f, mean2 = 0.f;
    T *y = static_cast<T *>(a.y) + g.first * a.n;
    float *stats = a.stats != nullptr ? a.stats + g.first : nullptr;
    int p = 0;
    for (int i = 0; i < count + 2 && count > 0; i++) {
        float sum = 0.f, squares = 0.f, var;
        if (i > 0) {
            mean2 = mean1;
            group_sum2<LANES / 32>(part[p ^ 1], mean1, var);   // of row i - 1, of row i - 2
            mean1 *= inv_n;
        }
        if (i < count) {
            wait_copies(stages - 4);
            ask();   // where row i - 3 was
            Rows::clean(cols, p0);
#pragma unroll
            for (int c = 0; c < C; c++) {
                if (!cols.has(c)) continue;
                float2 x[H];
                Rows::take(cols, p0, c, x);
                sum += sum_of(x);
            }
        }
        if (i >= 1 && i <= count) {
#pragma unroll
            for (int c = 0; c < C; c++) {
                if (!cols.has(c)) continue;
                float2 x[H];
                Rows::take(cols, p1, c, x);
#pragma unroll
                for (int k = 0; k < H; k++) x[k] = add2(x[k], both(-mean1));
                cols.clip(x, c);
                squares += dot_of(x, x);
            }
        }
        if (i >= 2) {
            const float rstd = 1.f / sqrtf(var * inv_n + a.eps);
#pragma unroll
            for (int c = 0; c < C; c++) {
                if (!cols.has(c)) continue;
                float2 x[H];
                Rows::take(cols, p2, c, x);
#pragma unroll
                for (int k = 0; k < H; k++) x[k] = fma2(mul2(add2(x[k], both(-mean2)), both(rstd)), w[c][k], b[c][k]);
                cols.store(y, c, x);
            }
            y += g.apart * a.n;
            if (stats != nullptr) {
                if (g.t == 0) {
                    stats[0] = mean2;
                    stats[a.rows] = rstd;
                }
                stats += g.apart;
            }
        }
        const float s = warp_sum2(sum, squares);
        if ((g.lane & 15) == 0) part[p][g.lane >> 4][g.warp] = s;
        p ^= 1;
        p2 = p1;
        p1 = p0;
        p0 = next(p0);
        g.sync();
    }
    ptx::cp_async_wait<0>();
}

// Step i: the sums of row i, dx of row i - 1.  (With dx right behind its own sums, two blocks of 512 threads waited for one another's
// barriers: 65536 rows of 4096 took 460 us.)
template <typename T, int LANES, bool SHIFT> __global__ void __launch_bounds__(most_threads(LANES, true), 1) norm_bwd_ring_kernel(const Bwd a, int stages)
{
    extern __shared__ __align__(16) unsigned char ring[];   // [groups][stages][x, dy][room]; at the end [groups][dw, db][n]
    __shared__ float parts[GROUPS][2][2][32];
    chain_start();
    chain_wait();
    const Group<LANES> g(a.rows);
    // a group without rows adds zeros to every column: of a single row the threads hold no more columns than its own
    const Columns<T, LANES, SHIFT> cols = {a.n, shift_of<T>(g.count > 0 ? g.first : 0, a.x_stride), g.t};
    using Rows = Ring<T, LANES, SHIFT>;
    Rows xs(a.x, a.x_stride, a.rows, g.first, g.apart, cols), ds(a.dy, a.dy_stride, a.rows, g.first, g.apart, cols);
    constexpr int C = Rows::C, H = Rows::H, room = LANES * HELD * (int)sizeof(T);
    const int count = g.count;
    unsigned char *const ring_start = ring + g.index * stages * 2 * room, *const ring_end = ring_start + stages * 2 * room;
    const auto next = [&](unsigned char *p) { return p + 2 * room == ring_end ? ring_start : p + 2 * room; };
    unsigned char *fresh = ring_start;
    int asked = 0;
    const auto ask = [&] {
        if (asked < count) {
            xs.ask(cols, fresh);
            ds.ask(cols, fresh + room);
        }
        ptx::cp_async_commit();
        fresh = next(fresh);
        asked++;
    };
    for (int i = 0; i < stages - 2; i++) ask();
    float2 w[C][H], dw[C][H], db[C][H];
#pragma unroll
    for (int c = 0; c < C; c++) {
        cols.param(a.weight, a.param_f32, c, 1.f, w[c]);
#pragma unroll
        for (int k = 0; k < H; k++) dw[c][k] = db[c][k] = both(0.f);
    }
    for (int i = threadIdx.x; i < GROUPS * 128; i += blockDim.x) (&parts[0][0][0][0])[i] = 0.f;
    __syncthreads();
    float(*const part)[2][32] = parts[g.index];
    const float inv_n = 1.f / (float)a.n;
    unsigned char *p0 = ring_start, *p1 = ring_start;
    const float *stats = a.stats + g.first;
    float mean = count > 0 ? __ldg(stats) : 0.f, rstd = count > 0 ? __ldg(stats + a.rows) : 0.f, mean1 = 0.f, rstd1 = 0.f;
    T *out = a.dx != nullptr ? static_cast<T *>(a.dx) + g.first * a.n : nullptr;
    int p = 0;
    // h and dy of a piece
    const auto take = [&](const unsigned char *from, int c, float m, float q, float2 (&h)[H], float2 (&d)[H]) {
        Rows::take(cols, from, c, h);
        Rows::take(cols, from + room, c, d);
#pragma unroll
        for (int k = 0; k < H; k++) h[k] = mul2(add2(h[k], both(-m)), both(q));
    };
    for (int i = 0; i <= count && count > 0; i++) {
        float sa = 0.f, sh = 0.f;
        const float m = mean, q = rstd;
        if (i < count) {
            wait_copies(stages - 3);
            ask();   // where row i - 2 was
            Rows::clean(cols, p0);
            Rows::clean(cols, p0 + room);
            stats += g.apart;
            if (i + 1 < count) {
                mean = __ldg(stats);
                rstd = __ldg(stats + a.rows);
            }
#pragma unroll
            for (int c = 0; c < C; c++) {
                if (!cols.has(c)) continue;
                float2 h[H], d[H];
                take(p0, c, m, q, h, d);
#pragma unroll
                for (int k = 0; k < H; k++) {
                    dw[c][k] = fma2(d[k], h[k], dw[c][k]);
                    db[c][k] = add2(db[c][k], d[k]);
                    d[k] = mul2(d[k], w[c][k]);
                }
                sa += sum_of(d);
                sh += dot_of(d, h);
            }
        }
        if (out != nullptr) {
            if (i > 0) {
                float ma, mh;
                group_sum2<LANES / 32>(part[p ^ 1], ma, mh);
                ma *= inv_n;
                mh *= inv_n;
#pragma unroll
                for (int c = 0; c < C; c++) {
                    if (!cols.has(c)) continue;
                    float2 h[H], d[H];
                    take(p1, c, mean1, rstd1, h, d);
#pragma unroll
                    for (int k = 0; k < H; k++) h[k] = mul2(both(rstd1), fma2(h[k], both(-mh), fma2(d[k], w[c][k], both(-ma))));
                    cols.store(out, c, h);
                }
                out += g.apart * a.n;
            }
            const float s = warp_sum2(sa, sh);
            if ((g.lane & 15) == 0) part[p][g.lane >> 4][g.warp] = s;
            p ^= 1;
            g.sync();
        }
        mean1 = m;
        rstd1 = q;
        p1 = p0;
        p0 = next(p0);
    }
    ptx::cp_async_wait<0>();
    if (a.parts == nullptr) return;
    // by column: the groups' shifts differ
    const int groups = blockDim.x / LANES;
    float *sums = a.parts + (long long)blockIdx.x * 2 * a.n, *mine = groups == 1 ? sums : reinterpret_cast<float *>(ring) + g.index * 2 * a.n;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; c++) {
        if (!cols.has(c)) continue;
#pragma unroll
        for (int k = 0; k < PER<T>; k++) {
            const int j = cols.first(c) + k;
            if (SHIFT && (unsigned)j >= (unsigned)a.n) continue;
            mine[j] = k % 2 == 0 ? dw[c][k / 2].x : dw[c][k / 2].y;
            mine[a.n + j] = k % 2 == 0 ? db[c][k / 2].x : db[c][k / 2].y;
        }
    }
    if (groups == 1) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.n; i += blockDim.x) {
        float v = 0.f;
        for (int k = 0; k < groups; k++) v += reinterpret_cast<const float *>(ring)[k * 2 * a.n + i];
        sums[i] = v;
    }
}

// Few rows, a block each: the row in registers, nothing to overlap.
template <typename T, int LANES, bool SHIFT> __global__ void __launch_bounds__(LANES) norm_fwd_few_kernel(const Fwd a)
{
    __shared__ float part[2][32];
    chain_start();
    chain_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long r = blockIdx.x;
    const Columns<T, LANES, SHIFT> cols = {a.n, shift_of<T>(r, a.stride), (int)threadIdx.x};
    const T *row = static_cast<const T *>(a.x) + r * a.stride, *end = static_cast<const T *>(a.x) + (a.rows - 1) * a.stride + a.n;
    constexpr int C = HELD / PER<T>, H = PER<T> / 2;
    Piece<T> raw[C];
    float2 x[C][H], w[H], b[H];
#pragma unroll
    for (int c = 0; c < C; c++) {
        raw[c] = Piece<T>();
        if (cols.has(c)) load_piece(raw[c], row + cols.first(c), end);
    }
    const auto total = [&](float s, float *part) {
        s = warp_sum(s);
        if (lane == 0) part[warp] = s;
        __syncthreads();
        return warp_sum(lane < LANES / 32 ? part[lane] : 0.f);
    };
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; c++) {
        raw[c].pairs(x[c]);
        cols.clip(x[c], c);
        s += sum_of(x[c]);
    }
    const float mean = total(s, part[0]) / (float)a.n;
    s = 0.f;
#pragma unroll
    for (int c = 0; c < C; c++) {
#pragma unroll
        for (int k = 0; k < H; k++) x[c][k] = add2(x[c][k], both(-mean));
        cols.clip(x[c], c);
        if (cols.has(c)) s += dot_of(x[c], x[c]);
    }
    const float rstd = 1.f / sqrtf(total(s, part[1]) / (float)a.n + a.eps);
#pragma unroll
    for (int c = 0; c < C; c++) {
        if (!cols.has(c)) continue;
        cols.param(a.weight, a.param_f32, c, 1.f, w);
        cols.param(a.bias, a.param_f32, c, 0.f, b);
#pragma unroll
        for (int k = 0; k < H; k++) x[c][k] = fma2(mul2(x[c][k], both(rstd)), w[k], b[k]);
        cols.store(static_cast<T *>(a.y) + r * a.n, c, x[c]);
    }
    if (a.stats != nullptr && threadIdx.x == 0) {
        a.stats[r] = mean;
        a.stats[a.rows + r] = rstd;
    }
}

// The blocks' sums joined: 8 columns a block (a sector), EACH threads a column.
template <int EACH> __global__ void __launch_bounds__(8 * EACH) norm_join_kernel(const float *parts, int blocks, int n, void *dw, void *db, int param_f32)
{
    __shared__ float part[EACH][9];
    chain_start();
    chain_wait();
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long i = (long long)blockIdx.x * 8 + tx;
    float s = 0.f;
    if (i < 2LL * n) {
#pragma unroll 5
        for (int b = ty; b < blocks; b += EACH) s += parts[(long long)b * 2 * n + i];
    }
    part[ty][tx] = s;
    __syncthreads();
    if (warp >= 8) return;
    float v = part[lane][warp];
    if constexpr (EACH == 128) v = (v + part[lane + 32][warp]) + (part[lane + 64][warp] + part[lane + 96][warp]);
    v = warp_sum(v);
    const long long at = (long long)blockIdx.x * 8 + warp;
    void *out = at < n ? dw : db;
    if (lane > 0 || at >= 2LL * n || out == nullptr) return;
    const long long j = at < n ? at : at - n;
    if (param_f32) static_cast<float *>(out)[j] = v;
    else static_cast<bf16 *>(out)[j] = __float2bfloat16_rn(v);
}

// ------------------------------------------------------------------ any rows, value by value: longer than a block's shared memory holds a few of,
// or with strides that put the rows of x, dy and the result differently between 16-byte boundaries

template <int V> __device__ __forceinline__ void block_sums(float (&s)[V], float *part)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();  // the last sums have been read
#pragma unroll
    for (int v = 0; v < V; v++) {
        s[v] = warp_sum(s[v]);
        if (lane == 0) part[v * 32 + warp] = s[v];
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; v++) s[v] = warp_sum(lane < (int)blockDim.x / 32 ? part[v * 32 + lane] : 0.f);
}
__device__ __forceinline__ float param(const void *p, int f32, long long i)
{
    return f32 ? __ldg(static_cast<const float *>(p) + i) : __bfloat162float(static_cast<const bf16 *>(p)[i]);
}

// A block a row, read again for each of its sums (from L2 mostly).
template <typename T> __global__ void __launch_bounds__(1024) norm_fwd_long_kernel(const Fwd a)
{
    __shared__ float part[2 * 32];
    chain_start();
    chain_wait();
    const long long r = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + r * a.stride;
    float s[1] = {0.f};
    for (int j = threadIdx.x; j < a.n; j += blockDim.x) s[0] += from_value(x[j]);
    block_sums(s, part);
    const float mean = s[0] / (float)a.n;
    s[0] = 0.f;
    for (int j = threadIdx.x; j < a.n; j += blockDim.x) {
        const float d = from_value(x[j]) - mean;
        s[0] = fmaf(d, d, s[0]);
    }
    block_sums(s, part);
    const float rstd = 1.f / sqrtf(s[0] / (float)a.n + a.eps);
    T *y = static_cast<T *>(a.y) + r * a.n;
    for (int j = threadIdx.x; j < a.n; j += blockDim.x) {
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
    __shared__ float part[2 * 32];
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
    for (int j = threadIdx.x; j < a.n; j += blockDim.x) {
        float h, d;
        at(j, h, d);
        s[0] += d;
        s[1] = fmaf(d, h, s[1]);
    }
    block_sums(s, part);
    const float ma = s[0] / (float)a.n, mh = s[1] / (float)a.n;
    T *dx = static_cast<T *>(a.dx) + r * a.n;
    for (int j = threadIdx.x; j < a.n; j += blockDim.x) {
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
    out[(long long)a.n + j] = db;
}

// ------------------------------------------------------------------ host side

// How rows of n values are taken: threads of a row, its groups in a block, the stages of a group's ring; blocks, the same on every
// device.
struct How {
    int lanes, pieces, groups, stages, smem, blocks;   // lanes 0: value by value
    bool shift, few;
};
How how(const csa_layernorm_params &p, bool backward)
{
    How h = {};
    const int n = p.cols, size = p.dtype == CSA_F32 ? 4 : 2, vector = 16 / size;
    const auto blocks = [&](long long each, long long most) {
        const long long want = (p.rows + each - 1) / each;
        h.blocks = (int)(want < 1 ? 1 : want < most ? want : most);
    };
    // rows of all arguments lie alike between boundaries
    const bool alike = (p.x_stride - n) % vector == 0 && (!backward || (p.dy_stride - n) % vector == 0);
    h.shift = n % vector != 0;
    const long long held = (long long)n + (h.shift && p.rows > 1 ? vector - 1 : 0);
    if (!alike || held > (size == 4 ? 8192 : 16384)) {
        blocks(1, 64);
        return h;
    }
    if (held <= 512) {
        h.pieces = held > 256 ? 2 : 1;
        h.lanes = held <= 32 ? 4 : held <= 64 ? 8 : held <= 128 ? 16 : 32;
        blocks(256 / h.lanes * U, backward ? 3LL * linear::kSms : 4LL * linear::kSms);
        return h;
    }
    const int live = backward ? 2 : 3;
    h.lanes = held <= 1024 ? 64 : held <= 2048 ? 128 : held <= 3 * 1024 ? 192 : held <= 4096 ? 256 : held <= 6 * 1024 ? 384 : held <= 8192 ? 512 : 1024;
    h.groups = most_threads(h.lanes, backward) / h.lanes;
    const int room = h.lanes * HELD * size * (backward ? 2 : 1);
    constexpr int shared = 225000 - GROUPS * 512;
    while (shared / h.groups / room < live + 1) h.groups--;   // a row on its way at least; the longest rows' ring holds 3 or 6
    h.stages = shared / h.groups / room;
    if (h.stages > live + 1 + MOST_PENDING) h.stages = live + 1 + MOST_PENDING;
    h.smem = h.groups * h.stages * room;
    blocks(1, linear::kSms);   // a multiple of 8, or a row of a group each
    // few rows: a block each, no ring to fill (37 x 4096: 2.3 us)
    h.few = !backward && p.rows <= 4 * linear::kSms;
    return h;
}

template <int L, int C> struct Shape {
    static constexpr int LANES = L, PIECES = C;
};
template <typename F> cudaError_t short_shape(const How &h, const F &f)
{
    if (h.lanes == 4) return f(Shape<4, 1>());
    if (h.lanes == 8) return f(Shape<8, 1>());
    if (h.lanes == 16) return f(Shape<16, 1>());
    return h.pieces == 1 ? f(Shape<32, 1>()) : f(Shape<32, 2>());
}
template <typename T, typename F> cudaError_t ring_shape(const How &h, const F &f)
{
    if (h.lanes == 64) return f(Shape<64, 2>());
    if (h.lanes == 128) return f(Shape<128, 2>());
    if (h.lanes == 192) return f(Shape<192, 2>());
    if (h.lanes == 256) return f(Shape<256, 2>());
    if (h.lanes == 384) return f(Shape<384, 2>());
    if constexpr (sizeof(T) == 2) {
        if (h.lanes == 1024) return f(Shape<1024, 2>());
    }
    return f(Shape<512, 2>());
}
inline int long_threads(int n) { return n <= 2048 ? 128 : 1024; }

template <typename T> cudaError_t fwd(const Fwd &a, const How &h, cudaStream_t st)
{
    if (h.lanes == 0) return launch_chained(norm_fwd_long_kernel<T>, dim3((unsigned)a.rows), long_threads(a.n), 0, 1, st, a);
    if (h.lanes <= 32) {
        return short_shape(h, [&](auto shape) {
            using S = decltype(shape);
            auto *kernel = h.shift ? norm_fwd_short_kernel<T, S::LANES, S::PIECES, true> : norm_fwd_short_kernel<T, S::LANES, S::PIECES, false>;
            return launch_chained(kernel, dim3((unsigned)h.blocks), 256, 0, 1, st, a);
        });
    }
    return ring_shape<T>(h, [&](auto shape) {
        constexpr int L = decltype(shape)::LANES;
        if (h.few) return launch_chained(h.shift ? norm_fwd_few_kernel<T, L, true> : norm_fwd_few_kernel<T, L, false>, dim3((unsigned)a.rows), L, 0, 1, st, a);
        auto *kernel = h.shift ? norm_fwd_ring_kernel<T, L, true> : norm_fwd_ring_kernel<T, L, false>;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, h.smem);
        if (e != cudaSuccess) return e;
        return launch_chained(kernel, dim3((unsigned)h.blocks), L * h.groups, h.smem, 1, st, a, h.stages);
    });
}
template <typename T> cudaError_t bwd(const Bwd &a, const How &h, cudaStream_t st)
{
    if (h.lanes == 0) {
        // dx last: it may lie where dy or x do
        cudaError_t e = cudaSuccess;
        if (a.parts != nullptr)
            e = launch_chained(norm_params_long_kernel<T>, dim3((unsigned)((a.n + 255) / 256), (unsigned)h.blocks), 256, 0, 1, st, a);
        if (e != cudaSuccess || a.dx == nullptr) return e;
        return launch_chained(norm_dx_long_kernel<T>, dim3((unsigned)a.rows), long_threads(a.n), 0, 1, st, a);
    }
    if (h.lanes <= 32) {
        return short_shape(h, [&](auto shape) {
            using S = decltype(shape);
            auto *kernel = h.shift ? norm_bwd_short_kernel<T, S::LANES, S::PIECES, true> : norm_bwd_short_kernel<T, S::LANES, S::PIECES, false>;
            return launch_chained(kernel, dim3((unsigned)h.blocks), 256, 0, 1, st, a);
        });
    }
    return ring_shape<T>(h, [&](auto shape) {
        constexpr int L = decltype(shape)::LANES;
        auto *kernel = h.shift ? norm_bwd_ring_kernel<T, L, true> : norm_bwd_ring_kernel<T, L, false>;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, h.smem);
        if (e != cudaSuccess) return e;
        return launch_chained(kernel, dim3((unsigned)h.blocks), L * h.groups, h.smem, 1, st, a, h.stages);
    });
}

}  // namespace norm

size_t layernorm_bwd_workspace(const csa_layernorm_params &p)
{
    return p.rows == 0 ? 0 : linear::up256((size_t)norm::how(p, true).blocks * 2 * p.cols * 4);
}

cudaError_t launch_layernorm_fwd(const csa_layernorm_params &p, const void *x, const void *weight, const void *bias, void *y, float *stats,
                                 cudaStream_t st)
{
    note_path("generic");
    const norm::Fwd a = {x, weight, bias, y, stats, p.rows, p.x_stride, p.cols, p.param_dtype == CSA_F32, p.eps};
    const norm::How h = norm::how(p, false);
    return p.dtype == CSA_F32 ? norm::fwd<float>(a, h, st) : norm::fwd<__nv_bfloat16>(a, h, st);
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
    const norm::How h = norm::how(p, true);
    const cudaError_t e = p.dtype == CSA_F32 ? norm::bwd<float>(a, h, st) : norm::bwd<__nv_bfloat16>(a, h, st);
    if (e != cudaSuccess || !params) return e;
    // many columns come from a block an SM, few from more
    const bool wide = p.cols > 512;
    return linear::launch_chained(wide ? norm::norm_join_kernel<32> : norm::norm_join_kernel<128>, dim3((unsigned)((2LL * p.cols + 7) / 8)), wide ? 256 : 1024, 0, 1, st, a.parts, h.blocks, p.cols, dweight,
                                  dbias, a.param_f32);
}

}  // namespace csa
