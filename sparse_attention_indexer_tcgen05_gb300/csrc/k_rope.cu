// k_rope.cu -- rotary positions with several axes on [rows, heads, head_dim] values; the inverse rotation is the
// gradient.
//
// Pair i of a head turns by the angle positions[axis(i)][row] * f_i.  Only the angle modulo a turn matters, and it
// is taken exactly: f_i is kept as F_i = round(2^64 f_i / 2 pi), a 64-bit fraction of a turn, and the product
// positions * F_i in 64-bit integers drops whole turns by itself, for every position the type holds and for negative
// ones.  Its top 32 bits, as a signed number of half turns in [-1, 1), go to sincospif.  (fp32 angles would be off
// by position * 2^-24: 0.06 rad at position 10^6.  fp64 angles per pair cost the GB300's few fp64 lanes; this takes
// three fp64 operations per pair to make F_i.)  F_i itself is off by at most 2^-53 of f_i / 2 pi, as fp64 holds it.
//
// Bound by memory: every value is read once and written once.  A warp takes a unit, a row (a slice of its heads where
// rows are few, several rows where they are short), computes its cosines and sines once into shared memory, while its
// first values are on their way, and shares them among the heads; warps do not wait for one another.  An item of work
// is two vectors of V elements: the two halves of V pairs (or, interleaved, V whole pairs), or two vectors of values
// that are copied.  V is the widest vector (32 bytes at most) that offset, dimensions and strides allow.  Measured (bf16):
// 16384 rows of 64 heads of 128 values, half of which rotate, 83 us (6.5 TB/s, 95% of a copy's rate); 5 rows 3.5 us.
#include "csa_internal.cuh"

namespace csa {
namespace rope {

constexpr int WARPS = 4, THREADS = 32 * WARPS;
constexpr int UNROLL = 2;                       // items of a lane whose loads are in flight together
constexpr int TABLE = 512;                      // cosine and sine pairs of a unit

struct Args {
    const void *x, *positions;
    const double *inv_freq;
    void *out;
    long long rows, xr, xh, yr, yh;             // strides in elements
    long long xv, yv;                           // elements from a unit's vector row (row and head) to the next one
    int heads, offset, pairs, inverse, pos64;
    int end0, end1, end2;                       // the pair after the last one of axes 0, 1, 2
    int rot_items, head_items;                  // items of a head that rotate, all of them
    int copy_lo;                                // vectors before the rotated part
    int copy_half;                              // copy item c moves vectors c and c + copy_half
    int copy_vecs;
    int step_row, step_item;                    // 32 items further: so many vector rows and items of a head
    unsigned long long magic_pairs, magic_head, magic_heads;  // see quotient()
    int rows_unit, heads_unit, slices;          // rows and heads of a unit; units that share the heads of their rows
    long long units;
    int copy;                                   // the values outside the rotation move (not in place)
};

// V elements in registers
template <typename T, int V> struct Vec {
    static constexpr int BYTES = sizeof(T) * V, W = BYTES < 4 ? 1 : BYTES / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (BYTES == 32)
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                         : "l"(p)
                         : "memory");
        else if constexpr (BYTES == 16) {
            const uint4 a = *reinterpret_cast<const uint4 *>(p);
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        } else if constexpr (BYTES == 8) {
            const uint2 a = *reinterpret_cast<const uint2 *>(p);
            w[0] = a.x; w[1] = a.y;
        } else if constexpr (BYTES == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            w[0] = *reinterpret_cast<const unsigned short *>(p);
        }
    }
    __device__ __forceinline__ void store(T *p) const
    {
        if constexpr (BYTES == 32)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                         "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
        else if constexpr (BYTES == 16) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (BYTES == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else if constexpr (BYTES == 4) *reinterpret_cast<uint32_t *>(p) = w[0];
        else *reinterpret_cast<unsigned short *>(p) = (unsigned short)w[0];
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i % 2 == 0 ? w[i / 2] << 16 : w[i / 2] & 0xffff0000u);
    }
    // elements i and i + 1
    __device__ __forceinline__ void set2(int i, float a, float b)
    {
        if constexpr (sizeof(T) == 4) {
            w[i] = __float_as_uint(a);
            w[i + 1] = __float_as_uint(b);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            w[i / 2] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    __device__ __forceinline__ void set1(float a) { w[0] = sizeof(T) == 4 ? __float_as_uint(a) : (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(a)); }
};

// i / d for i < 2^20 and d < 2^20, with magic = 2^40 / d + 1
__device__ __forceinline__ int quotient(int i, unsigned long long magic) { return (int)((unsigned long long)i * magic >> 40); }

// The fraction of a turn that a frequency is, in 2^-64.
__device__ __forceinline__ unsigned long long turn_of(double freq)
{
    double turns = freq * 0.15915494309189533577;  // 1 / 2 pi
    turns -= floor(turns);
    return __double2ull_rn(turns * 18446744073709551616.0);
}

// (a, b) turned by (cos, sin): (a cos - b sin, a sin + b cos)
__device__ __forceinline__ float2 turned(float a, float b, float2 z) { return make_float2(a * z.x - b * z.y, a * z.y + b * z.x); }

template <typename T, int V, bool PAIRED>
__global__ void __launch_bounds__(THREADS, 5) rope_kernel(const Args a)
{
    __shared__ __align__(16) float2 tables[WARPS][TABLE];  // (cos, sin) of [row of the unit][pair]
    const int lane = threadIdx.x & 31;
    float2 *cs = tables[threadIdx.x >> 5];
    const long long unit = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (unit >= a.units) return;
    const long long row0 = unit / a.slices * a.rows_unit;
    const int head0 = (int)(unit % a.slices) * a.heads_unit;
    const int nrow = (int)min((long long)a.rows_unit, a.rows - row0);
    const int total = nrow * min(a.heads_unit, a.heads - head0) * a.head_items;
    const T *x = static_cast<const T *>(a.x) + row0 * a.xr + head0 * a.xh;
    T *out = static_cast<T *>(a.out) + row0 * a.yr + head0 * a.yh;

    // the first angle's inputs are asked for before the values: they are needed first
    const int angles = nrow * a.pairs;
    long long pos = 0;
    double freq = 0.0;
    auto fetch = [&](int t) {
        const int r = quotient(t, a.magic_pairs), i = t - r * a.pairs;
        const int axis = (i >= a.end0) + (i >= a.end1) + (i >= a.end2);
        const long long at = axis * a.rows + row0 + r;
        pos = a.pos64 ? static_cast<const long long *>(a.positions)[at] : (long long)static_cast<const int *>(a.positions)[at];
        freq = a.inv_freq[i];
    };
    if (lane < angles) fetch(lane);

    // item `lane`, then every 32nd: item c of vector row vr
    int vr = quotient(lane, a.magic_head), c = lane - vr * a.head_items;
    for (int base = lane; base - lane < total; base += 32 * UNROLL) {
        Vec<T, V> u[UNROLL], v[UNROLL];
        T *to[UNROLL];               // the item's first vector in out
        int second[UNROLL];          // elements from the first vector to the second (0: there is none); -1: no item
        int pair[UNROLL];            // index into cs of the item's first pair; -1: a copy
#pragma unroll
        for (int k = 0; k < UNROLL; k++) {
            second[k] = -1;
            if (base + 32 * k < total) {
                int el;
                if (c < a.rot_items) {
                    if constexpr (PAIRED) {  // adjacent pairs: 2 V values in a row
                        el = a.offset + 2 * V * c;
                        second[k] = V == 1 || 2 * V * c + V < 2 * a.pairs ? V : 0;
                    } else {
                        el = a.offset + V * c;
                        second[k] = a.pairs;
                    }
                    pair[k] = (a.rows_unit > 1 ? quotient(vr, a.magic_heads) * a.pairs : 0) + V * c;
                } else {
                    const int q = c - a.rot_items, q2 = q + a.copy_half;
                    el = V * q + (q < a.copy_lo ? 0 : 2 * a.pairs);
                    second[k] = q2 < a.copy_vecs ? V * q2 + (q2 < a.copy_lo ? 0 : 2 * a.pairs) - el : 0;
                    pair[k] = -1;
                }
                const T *from = x + vr * a.xv + el;
                to[k] = out + vr * a.yv + el;
                u[k].load(from);
                if (second[k] != 0) v[k].load(from + second[k]);
            }
            vr += a.step_row;
            c += a.step_item;
            if (c >= a.head_items) {
                c -= a.head_items;
                vr++;
            }
        }
        if (base == lane) {
            for (int t = lane; t < angles; t += 32) {
                if (t >= 32) fetch(t);
                const int half = (int)(((unsigned long long)pos * turn_of(freq)) >> 32);  // 2^-31 half turns, whole turns dropped
                float s, co;
                sincospif((float)half * 4.656612873077393e-10f, &s, &co);
                cs[t] = make_float2(co, a.inverse ? -s : s);
            }
            __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < UNROLL; k++) {
            if (second[k] < 0) continue;
            if (pair[k] >= 0) {
                const float2 *t = cs + pair[k];
                if constexpr (V == 1) {
                    const float2 z = turned(u[k].get(0), v[k].get(0), t[0]);
                    u[k].set1(z.x);
                    v[k].set1(z.y);
                } else if constexpr (PAIRED) {
#pragma unroll
                    for (int j = 0; j < V / 2; j++) {
                        const float2 z = turned(u[k].get(2 * j), u[k].get(2 * j + 1), t[j]);
                        u[k].set2(2 * j, z.x, z.y);
                    }
                    if (second[k] != 0) {
#pragma unroll
                        for (int j = 0; j < V / 2; j++) {
                            const float2 z = turned(v[k].get(2 * j), v[k].get(2 * j + 1), t[V / 2 + j]);
                            v[k].set2(2 * j, z.x, z.y);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const float2 z = turned(u[k].get(j), v[k].get(j), t[j]), y = turned(u[k].get(j + 1), v[k].get(j + 1), t[j + 1]);
                        u[k].set2(j, z.x, y.x);
                        v[k].set2(j, z.y, y.y);
                    }
                }
            }
            u[k].store(to[k]);
            if (second[k] != 0) v[k].store(to[k] + second[k]);
        }
    }
}

template <typename T, int V> cudaError_t launch(const csa_rope_params &p, Args &a, int sms, cudaStream_t st)
{
    const bool paired = p.interleaved != 0;
    a.rot_items = paired ? (a.pairs + V - 1) / V : a.pairs / V;
    a.copy_lo = p.rot_offset / V;
    a.copy_vecs = a.copy ? (p.head_dim - p.rot_dim) / V : 0;
    a.copy_half = (a.copy_vecs + 1) / 2;
    a.head_items = a.rot_items + a.copy_half;
    if (a.head_items == 0) return cudaSuccess;  // in place and nothing rotates
    // A warp's unit: a row, or a slice of its heads (each slice computes the row's angles again), or several short rows
    // whose vector rows lie evenly.  About 8 items a lane make the angles' share small; few rows would leave SMs idle so,
    // and the slices shrink down to one item a lane until every SM has 16 warps.
    constexpr long long MOST = 256, LEAST = 32;
    const long long row_items = (long long)a.heads * a.head_items;
    long long per = MOST;
    while (per > LEAST && (row_items * a.rows + per - 1) / per < 16LL * sms) per /= 2;
    const bool even = a.heads == 1 || (a.xr == a.heads * a.xh && a.yr == a.heads * a.yh);
    a.rows_unit = 1;
    if (row_items < per && even) {
        a.rows_unit = (int)(per / row_items);
        if (a.pairs > 0) a.rows_unit = min(a.rows_unit, max(1, TABLE / a.pairs));
    }
    const long long slices = (row_items + per - 1) / per;
    a.heads_unit = (int)((a.heads + slices - 1) / slices);
    a.slices = (a.heads + a.heads_unit - 1) / a.heads_unit;
    a.units = (a.rows + a.rows_unit - 1) / a.rows_unit * a.slices;
    a.xv = a.heads == 1 ? a.xr : a.xh;
    a.yv = a.heads == 1 ? a.yr : a.yh;
    a.step_row = 32 / a.head_items;
    a.step_item = 32 % a.head_items;
    const auto magic = [](long long d) { return (1ull << 40) / (unsigned long long)(d > 0 ? d : 1) + 1; };
    a.magic_pairs = magic(a.pairs);
    a.magic_head = magic(a.head_items);
    a.magic_heads = magic(a.heads_unit);
    const long long ctas = (a.units + WARPS - 1) / WARPS;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (paired) rope_kernel<T, V, true><<<(unsigned)ctas, THREADS, 0, st>>>(a);
    else rope_kernel<T, V, false><<<(unsigned)ctas, THREADS, 0, st>>>(a);
    note_launches(1);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_v(const csa_rope_params &p, Args &a, long long widest, int sms, cudaStream_t st)
{
    constexpr int FULL = 32 / sizeof(T);
    if (widest >= FULL) return launch<T, FULL>(p, a, sms, st);
    if (widest >= FULL / 2) return launch<T, FULL / 2>(p, a, sms, st);
    if (widest >= 2) return launch<T, 2>(p, a, sms, st);
    return launch<T, 1>(p, a, sms, st);
}

}  // namespace rope

cudaError_t launch_rope(const csa_rope_params &p, const void *x, const void *positions, const double *inv_freq,
                        void *out, cudaStream_t st)
{
    rope::Args a = {};
    a.x = x;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.out = out;
    a.rows = p.rows;
    a.xh = p.x_head_stride;
    a.xr = p.x_row_stride;
    a.yh = p.out_head_stride;
    a.yr = p.out_row_stride;
    a.heads = p.heads;
    a.offset = p.rot_offset;
    a.pairs = p.rot_dim / 2;
    a.inverse = p.inverse;
    a.pos64 = p.positions_64;
    a.copy = x != out;
    int end = 0, ends[3];
    for (int i = 0; i < 3; i++) {
        if (i < p.axes) end += p.sections[i];
        ends[i] = i + 1 < p.axes ? end : 0x7fffffff;  // the last axis takes every pair that is left
    }
    a.end0 = ends[0];
    a.end1 = ends[1];
    a.end2 = ends[2];
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // the widest vector: the largest power of two that divides every offset, extent and stride in question
    const long long sizes[] = {p.rot_offset, p.interleaved ? p.rot_dim : p.rot_dim / 2, p.head_dim,
                               p.x_row_stride, p.x_head_stride, p.out_row_stride, p.out_head_stride,
                               (long long)((uintptr_t)x / (p.dtype == CSA_BF16 ? 2 : 4)), (long long)((uintptr_t)out / (p.dtype == CSA_BF16 ? 2 : 4))};
    long long widest = 16;
    for (long long s : sizes)
        while (s % widest != 0) widest /= 2;
    return p.dtype == CSA_BF16 ? rope::launch_v<__nv_bfloat16>(p, a, widest, sms, st)
                               : rope::launch_v<float>(p, a, widest, sms, st);
}

}  // namespace csa
