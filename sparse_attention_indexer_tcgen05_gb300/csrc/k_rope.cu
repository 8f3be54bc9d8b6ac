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
// Bound by memory: every value is read once and written once.  A CTA takes a few rows (or, when there are fewer rows
// than SMs could use, a slice of one row's heads), computes the rows' cosines and sines once into shared memory and
// shares them among the heads.  Each thread issues its loads before it waits for them.  One item of work is two
// vectors of V elements: the two halves of V pairs (or, interleaved, two vectors of V / 2 whole pairs each), or two
// vectors of values that are copied.  V is the widest vector (16 bytes at most) that offset, dimensions and strides
// allow.
#include "csa_internal.cuh"

namespace csa {
namespace rope {

constexpr int THREADS = 256;
constexpr int UNROLL = 2;                       // items of a thread whose loads are in flight together
constexpr int TABLE = 2048;                     // cosine and sine pairs in shared memory

struct Args {
    const void *x, *positions;
    const double *inv_freq;
    void *out;
    long long rows, xr, xh, yr, yh;             // strides in elements
    int heads, offset, pairs, inverse, pos64;
    int end0, end1, end2;                       // the pair after the last one of axes 0, 1, 2
    int rot_items, head_items;                  // items of a head that rotate, all of them
    int copy_lo;                                // vectors before the rotated part
    int copy_half;                              // copy item c moves vectors c and c + copy_half
    int copy_vecs;
    int copy_skip;                              // elements from a copied vector's number to its place behind the pairs
    unsigned long long magic_pairs, magic_row, magic_head;  // see quotient()
    int rows_cta, heads_cta;                    // rows and heads of one CTA
    int slices;                                 // CTAs that share the heads of their rows
    int copy;                                   // the values outside the rotation move (not in place)
};

template <int BYTES> struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };

template <typename T, int V> union Vec {
    typename Word<sizeof(T) * V>::type w;
    T e[V];
    __device__ Vec() {}
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// i / d for i < 2^20 and d < 2^20, with magic = 2^40 / d + 1
__device__ __forceinline__ int quotient(int i, unsigned long long magic) { return (int)((unsigned long long)i * magic >> 40); }

template <typename T, int V, bool PAIRED>
__global__ void __launch_bounds__(THREADS, 4) rope_kernel(const Args a)
{
    __shared__ float2 cs[TABLE];  // (cos, sin) of [row of the CTA][pair]
    const long long row0 = (long long)(blockIdx.x / a.slices) * a.rows_cta;
    const int head0 = (int)(blockIdx.x % a.slices) * a.heads_cta;
    const int nrow = (int)min((long long)a.rows_cta, a.rows - row0);
    const int nhead = min(a.heads_cta, a.heads - head0);
    const int row_items = a.heads_cta * a.head_items;  // the last slice of a row leaves some out
    const int total = nrow * row_items;
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
    if ((int)threadIdx.x < angles) fetch(threadIdx.x);

    for (int base = 0; base < total; base += THREADS * UNROLL) {
        Vec<T, V> u[UNROLL], v[UNROLL];
        T *to[UNROLL];               // the item's first vector in out; null: nothing to do
        int second[UNROLL];          // elements from the first vector to the second (0: there is none)
        int pair[UNROLL];            // index into cs of the item's first pair; -1: a copy
#pragma unroll
        for (int k = 0; k < UNROLL; k++) {
            const int it = base + k * THREADS + threadIdx.x;
            to[k] = nullptr;
            const int r = quotient(it, a.magic_row), rest = it - r * row_items;
            const int hd = quotient(rest, a.magic_head), c = rest - hd * a.head_items;
            if (it >= total || hd >= nhead) continue;
            int el;
            if (c < a.rot_items) {
                if constexpr (PAIRED && V == 1) {
                    el = a.offset + 2 * c;
                    second[k] = 1;
                } else if constexpr (PAIRED) {  // adjacent pairs: 2 V values in a row
                    el = a.offset + 2 * V * c;
                    second[k] = 2 * V * c + V < 2 * a.pairs ? V : 0;
                } else {
                    el = a.offset + V * c;
                    second[k] = a.pairs;
                }
                pair[k] = r * a.pairs + V * c;
            } else {
                const int q = c - a.rot_items, q2 = q + a.copy_half;
                el = V * q + (q < a.copy_lo ? 0 : a.copy_skip);
                second[k] = q2 < a.copy_vecs ? V * q2 + (q2 < a.copy_lo ? 0 : a.copy_skip) - el : 0;
                pair[k] = -1;
            }
            const T *from = x + (r * a.xr + hd * a.xh + el);
            to[k] = out + (r * a.yr + hd * a.yh + el);
            u[k].w = *reinterpret_cast<const decltype(u[k].w) *>(from);
            if (second[k] != 0) v[k].w = *reinterpret_cast<const decltype(v[k].w) *>(from + second[k]);
        }
        if (base == 0) {
            for (int t = threadIdx.x; t < angles; t += THREADS) {
                if (t >= THREADS) fetch(t);
                double turns = freq * 0.15915494309189533577;  // 1 / 2 pi
                turns -= floor(turns);
                const unsigned long long f = __double2ull_rn(turns * 18446744073709551616.0);
                const int half = (int)(((unsigned long long)pos * f) >> 32);  // 2^-31 half turns, whole turns dropped
                float s, c;
                sincospif((float)half * 4.656612873077393e-10f, &s, &c);
                cs[t] = make_float2(c, a.inverse ? -s : s);
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < UNROLL; k++) {
            if (to[k] == nullptr) continue;
            if (pair[k] >= 0) {
                const float2 *t = cs + pair[k];
                if constexpr (PAIRED && V > 1) {
#pragma unroll
                    for (int j = 0; j < V / 2; j++) {
                        const float p = to_f(u[k].e[2 * j]), q = to_f(u[k].e[2 * j + 1]);
                        const float2 z = t[j];
                        u[k].e[2 * j] = from_f<T>(p * z.x - q * z.y);
                        u[k].e[2 * j + 1] = from_f<T>(p * z.y + q * z.x);
                    }
                    if (second[k] != 0) {
#pragma unroll
                        for (int j = 0; j < V / 2; j++) {
                            const float p = to_f(v[k].e[2 * j]), q = to_f(v[k].e[2 * j + 1]);
                            const float2 z = t[V / 2 + j];
                            v[k].e[2 * j] = from_f<T>(p * z.x - q * z.y);
                            v[k].e[2 * j + 1] = from_f<T>(p * z.y + q * z.x);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < V; j++) {
                        const float p = to_f(u[k].e[j]), q = to_f(v[k].e[j]);
                        const float2 z = t[j];
                        u[k].e[j] = from_f<T>(p * z.x - q * z.y);
                        v[k].e[j] = from_f<T>(p * z.y + q * z.x);
                    }
                }
            }
            *reinterpret_cast<decltype(u[k].w) *>(to[k]) = u[k].w;
            if (second[k] != 0) *reinterpret_cast<decltype(v[k].w) *>(to[k] + second[k]) = v[k].w;
        }
    }
}

template <typename T, int V> cudaError_t launch(const csa_rope_params &p, Args &a, int sms, cudaStream_t st)
{
    const bool paired = p.interleaved != 0;
    const int span = paired ? 2 * a.pairs : a.pairs;  // V elements of it make one vector
    a.rot_items = paired ? (span + 2 * V - 1) / (2 * V) : span / V;
    a.copy_lo = p.rot_offset / V;
    a.copy_vecs = a.copy ? (p.head_dim - p.rot_dim) / V : 0;
    a.copy_half = (a.copy_vecs + 1) / 2;
    a.copy_skip = p.rot_dim;
    a.head_items = a.rot_items + a.copy_half;
    if (a.head_items == 0) return cudaSuccess;  // in place and nothing rotates
    // A CTA's share: UNROLL items a thread when there are enough of them for every SM, by whole rows while their
    // angles fit the table, else by slices of the heads (each slice computes the row's angles again).
    const long long want = (long long)THREADS * UNROLL;
    const long long row_items = (long long)a.heads * a.head_items;
    if (row_items >= want || a.rows * row_items <= want * sms) {
        // one row, cut into slices of heads: at most `want` items each, fewer while the SMs are not filled
        long long per = want;
        while (per > THREADS && (row_items + per - 1) / per * a.rows < 2LL * sms) per /= 2;
        a.rows_cta = 1;
        a.heads_cta = (int)max(1LL, min((long long)a.heads, per / a.head_items));
    } else {
        a.heads_cta = a.heads;
        long long r = max(1LL, want / row_items);
        if (a.pairs > 0) r = min(r, (long long)(TABLE / a.pairs));
        a.rows_cta = (int)r;
    }
    a.slices = (a.heads + a.heads_cta - 1) / a.heads_cta;
    const auto magic = [](long long d) { return (1ull << 40) / (unsigned long long)(d > 0 ? d : 1) + 1; };
    a.magic_pairs = magic(a.pairs);
    a.magic_row = magic((long long)a.heads_cta * a.head_items);
    a.magic_head = magic(a.head_items);
    const long long ctas = (a.rows + a.rows_cta - 1) / a.rows_cta * a.slices;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (paired) {
        rope_kernel<T, V, true><<<(unsigned)ctas, THREADS, 0, st>>>(a);
    } else {
        rope_kernel<T, V, false><<<(unsigned)ctas, THREADS, 0, st>>>(a);
    }
    note_launches(1);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_v(const csa_rope_params &p, Args &a, int widest, int sms, cudaStream_t st)
{
    constexpr int FULL = 16 / sizeof(T);
    if (widest >= FULL) return launch<T, FULL>(p, a, sms, st);
    if (widest >= FULL / 2) return launch<T, FULL / 2>(p, a, sms, st);
    if constexpr (FULL == 8) {
        if (widest >= 2) return launch<T, 2>(p, a, sms, st);
    }
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
                               p.x_row_stride, p.x_head_stride, p.out_row_stride, p.out_head_stride};
    int widest = 8;
    for (long long s : sizes)
        while (s % widest != 0) widest /= 2;
    return p.dtype == CSA_BF16 ? rope::launch_v<__nv_bfloat16>(p, a, widest, sms, st)
                               : rope::launch_v<float>(p, a, widest, sms, st);
}

}  // namespace csa
