// k_vocab.cu -- the vocabulary's losses: cross entropy with labels and distillation from a teacher's top logits, from hidden
// states and the vocabulary's weight, with their gradients.
//
//   z = alpha x W^T,  lse_r = log sum_v exp z_rv,  p = exp(z - lse)
//   label of row r:  L_r = lse_r - z_label
//   teacher of row r, candidates v_s with logits l_s:  t_s = exp(l_s - N_r), N_r given or log sum_s exp l_s;
//       L_r = sum_s t_s (log t_s - z_{v_s} + lse_r)
//   loss = sum of both, each with its weight and over the rows that have it
//   dz_rv = c_r p_rv - sum over the row's targets at v of tau,  dx = alpha dz W,  dW = alpha dz^T x
//
// with tau the label's or candidate's weight in the loss and c_r their sum.  A weight that all rows share (one over their number)
// is a factor of the products and not of dz: rounded to bf16 with dz it would be off by up to 2^-8 for all of a gradient
// alike.  The losses need a row's lse and the few scores that its targets name; the gradient needs p.  Rows go piece by
// piece: the scores of a piece are made once and reduced where they are made (k_vocab_tc.cu), and what the backward keeps of
// them is 16 bits a value, exp(z - largest of its group), which the pass below turns into dz in place.  So a piece takes
// three products, where pieces of the vocabulary would need its scores a second time, once the lse is known: four.  dW sums
// over pieces in fp32.
//
// Bound by the three products (2 M K V operations each) at the tensor cores' power limit.  8192 rows of 2048 over 131072 columns, a
// fifth of them without a target and so left out: scores 2.00 ms, this file's kernels 0.60 (dz: 4 bytes a score at 6.4 TB/s), dx
// and dW 1.96 and 1.94; 6.6 ms as one call, 7.0 to 7.5 in a loop of calls, where the clock falls.
#include "k_rows.cuh"
#include "k_vocab.cuh"

#include <cuda_fp16.h>
#include <math.h>

namespace csa {
namespace vocab {

using namespace linear;

constexpr int ROWS = 8;          // rows of a block of prepare_kernel and rows_kernel, a warp each
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Targets as they are given, and what they become: a row's columns in ascending order, with their weights.
struct Targets {
    const void *labels, *ids;    // [M], [M][slots]; int32 or int64
    const float *logits, *lse;   // [M][slots], [M] or null
    int labels_64, ids_64, slots, width;   // width: slots and the label's
    long long rows, vocab;
    int *sorted;                 // [width][rows]
    float *weight;               // [width][rows]: t of a candidate, -1 for the label; NaN and -inf where the id is not a column
    int *marks;                  // [rows][groups]: how many targets lie before each group of columns, and from bit 16 on in it
    int groups;
    int2 *counts;                // [blocks]: rows with a label, rows with a candidate
    int *done;                   // set to 0: blocks of rows_kernel that have finished
    // Rows that have a target, packed (below); null: every row stays where it is
    uint32_t *activity;          // bits of rows with a target
    int *active;                 // rows with a target
    int *index, *place;          // [rows]: the row that a packed row was; where a row is packed, -1 without a target
    float *losses;               // [2][rows], set to 0 for rows without a target
    const void *x;
    long long x_stride;
    bf16 *packed;                // [rows + TAIL][ld], planes apart
    long long ld, plane;
    int features;
};

__device__ __forceinline__ long long candidate_of(const Targets &a, long long at)
{
    return a.ids_64 ? static_cast<const long long *>(a.ids)[at] : static_cast<const int *>(a.ids)[at];
}

__device__ __forceinline__ long long label_of(const Targets &a, long long r)
{
    if (a.labels == nullptr) return -1;
    return a.labels_64 ? static_cast<const long long *>(a.labels)[r] : static_cast<const int *>(a.labels)[r];
}
// Counts of a block's threads or warps, joined.
__device__ __forceinline__ void count(const Targets &a, bool label, bool taught)
{
    __shared__ int2 have[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int2 n = make_int2(__popc(__ballot_sync(0xffffffffu, label)), __popc(__ballot_sync(0xffffffffu, taught)));
    if (lane == 0) have[warp] = n;
    __syncthreads();
    if (threadIdx.x > 0) return;
    int2 sum = make_int2(0, 0);
    for (int w = 0; w < (int)blockDim.x / 32; w++) {
        sum.x += have[w].x;
        sum.y += have[w].y;
    }
    a.counts[blockIdx.x] = sum;
    if (blockIdx.x == 0) *a.done = 0;
}

// Labels alone: a thread a row.
__global__ void __launch_bounds__(256) vocab_labels_kernel(const Targets a)
{
    chain_start();
    chain_wait();
    const long long r = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long v = r < a.rows ? label_of(a, r) : -1;
    if (r < a.rows) {
        a.sorted[r] = v >= 0 && v < a.vocab ? (int)v : NONE;
        a.weight[r] = v < 0 ? 0.f : v < a.vocab ? -1.f : -INFINITY;
    }
    count(a, v >= 0, false);
}

// Rows without a label or candidate (prompts, padding) take no part in the three products: of a large vocabulary the others are packed,
// in their order, and the products' rows are what the device counts.  8192 rows of 2048 over 131072 columns, a fifth of them
// without a label: 8.3 ms -> 7.0.
//
// First a bit for each row, and the counts of 32 rows, a warp a row.  Every block that packs rows then counts the bits before its
// own: 8192 rows have 256 words of them.  (Summed by one block in a kernel between the two: 4 us more.)
__global__ void __launch_bounds__(1024) vocab_count_kernel(const Targets a)
{
    chain_start();
    chain_wait();
    __shared__ int have[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long r = (long long)blockIdx.x * 32 + warp;
    int labelled = 0, any = 0;
    if (r < a.rows) {
        labelled = label_of(a, r) >= 0;
#pragma unroll 4
        for (int s = lane; s < a.slots; s += 32) any |= candidate_of(a, r * a.slots + s) >= 0;
    }
    any = __any_sync(0xffffffffu, any);
    if (lane == 0) have[warp] = labelled | any << 1;
    __syncthreads();
    if (warp > 0) return;
    const uint32_t l = __ballot_sync(0xffffffffu, have[lane] & 1), t = __ballot_sync(0xffffffffu, have[lane] & 2);
    if (lane > 0) return;
    a.counts[blockIdx.x] = make_int2(__popc(l), __popc(t));
    a.activity[blockIdx.x] = l | t;
}

using Key = unsigned long long;
__device__ __forceinline__ void exchange(Key &x, Key &y, bool up)
{
    const bool swap = (x > y) == up;
    const Key t = swap ? y : x;
    y = swap ? x : y;
    x = t;
}
// Ascending over a warp's lanes, R neighbouring ones each
template <int R> __device__ __forceinline__ void sort_warp(Key (&x)[R])
{
    const int lane = threadIdx.x & 31;
    const auto within = [&](bool up) {   // halves of R: one merge
#pragma unroll
        for (int j = R / 2; j > 0; j /= 2) {
#pragma unroll
            for (int r = 0; r < R; r++)
                if ((r & j) == 0) exchange(x[r], x[r | j], up);
        }
    };
#pragma unroll
    for (int k = 2; k < R; k *= 2) {
#pragma unroll
        for (int j = k / 2; j > 0; j /= 2) {
#pragma unroll
            for (int r = 0; r < R; r++)
                if ((r & j) == 0) exchange(x[r], x[r | j], (r & k) == 0);
        }
    }
    within((lane & 1) == 0);
#pragma unroll 1
    for (int k = 2; k <= 32; k *= 2) {
        const bool up = (lane & k) == 0;
#pragma unroll 1
        for (int d = k / 2; d > 0; d /= 2) {
            const bool least = ((lane & d) == 0) == up;
#pragma unroll
            for (int r = 0; r < R; r++) {
                const Key y = __shfl_xor_sync(0xffffffffu, x[r], d);
                if ((x[r] > y) == least) x[r] = y;
            }
        }
        within(up);
    }
}

// More candidates than this are sorted, by a bitonic network of their keys (column, then slot) in a warp's registers: comparing each
// with each takes S^2 / 32 steps, the network S log^2 S / 128 longer ones.  4096 rows of 1024: 594 us -> 177 (the network in shared
// memory 265), 2400 of 300: 75 -> 34, 3001 of 129: 40 -> 29; but of 100, four keys a lane: 22.6 -> 24.
constexpr int MANY = 128;
__host__ __device__ constexpr int keys_of(int slots)
{
    int n = 2 * MANY;   // 8 keys a lane
    while (n < slots) n *= 2;
    return n;
}
// Shared memory of a row: columns, their order, and logits
__host__ __device__ constexpr int prepare_bytes(int slots, int width)
{
    const int room = (width + 3) & ~3;
    return slots > MANY ? 8 * keys_of(slots) + 4 * room : 12 * room;
}

constexpr int TAIL = 64;
// A warp a row.  Each target's place is the number of targets before it (smaller column, or the same and earlier).  V: the
// values' type, where rows are packed; the last TAIL warps then put zeros behind the last packed row, as the k axis of dW takes whole
// stages of 64.  R: keys of a lane where candidates are sorted; 0: they are few.
template <typename V, bool PACK, int R> __global__ void __launch_bounds__(32 * ROWS) vocab_prepare_kernel(const Targets a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    chain_start();
    chain_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, room = (a.width + 3) & ~3;
    const long long r = (long long)blockIdx.x * ROWS + warp;
    constexpr bool many = R > 0;
    constexpr int keyed = 32 * R;
    unsigned char *const mine = raw + warp * prepare_bytes(a.slots, a.width);
    int *ids = reinterpret_cast<int *>(mine), *sorted = ids + room;
    Key *keys = reinterpret_cast<Key *>(mine);
    float *logits = reinterpret_cast<float *>(mine + (many ? 8 * keyed : 8 * room));
    bool taught = false;
    long long label = -1, row = r;   // where the row's targets go
    if constexpr (PACK) {
        // rows before this block's
        __shared__ int sums[ROWS];
        const long long base = min((long long)blockIdx.x * ROWS, (a.rows + 31) / 32 * 32);
        int before = 0;
#pragma unroll 4
        for (int i = threadIdx.x; i < (int)(base / 32); i += 32 * ROWS) before += __popc(a.activity[i]);
        before = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0) sums[warp] = before;
        __syncthreads();
        before = 0;
#pragma unroll
        for (int w = 0; w < ROWS; w++) before += sums[w];
        const long long behind = r - (a.rows + 31) / 32 * 32;
        if (behind >= 0) {
            if (behind == 0 && lane == 0) {
                *a.active = before;
                *a.done = 0;
            }
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            for (int q = 0; q < Planes<V>::N; q++) {
                uint4 *to = reinterpret_cast<uint4 *>(a.packed + q * a.plane + (before + behind) * a.ld);
                for (long long i = lane; i < a.ld / 8; i += 32) to[i] = zero;
            }
            return;
        }
        if (r >= a.rows) return;
        const uint32_t bits = a.activity[r / 32];
        if ((bits >> (r & 31) & 1) == 0) {
            if (lane == 0) {
                a.place[r] = -1;
                a.losses[r] = a.losses[a.rows + r] = 0.f;
            }
            return;
        }
        row = before + __popc(bits & ((1u << (r & 31)) - 1));
        if (lane == 0) {
            a.place[r] = (int)row;
            a.index[row] = (int)r;
        }
        const V *x = static_cast<const V *>(a.x) + r * a.x_stride, *end = static_cast<const V *>(a.x) + (a.rows - 1) * a.x_stride + a.features;
        const bool aligned = a.x_stride % (16 / (int)sizeof(V)) == 0;
        int c = 8 * lane;
        for (; aligned && c + 3 * 256 + 8 <= a.features; c += 4 * 256) {   // four loads under one latency
            Raw8<V, true> raw[4];
#pragma unroll
            for (int k = 0; k < 4; k++) raw[k].load(x + c + k * 256, 8, end);
#pragma unroll
            for (int k = 0; k < 4; k++) {
                float v[8];
                raw[k].floats(8, v);
                put_planes8<Planes<V>::N>(a.packed, a.plane, row * a.ld + c + k * 256, v);
            }
        }
        for (; c < a.features; c += 256) {
            float v[8];
            if (aligned && c + 8 <= a.features) load8<V, true>(x + c, 8, end, v);
            else load8<V, false>(x + c, min(8, a.features - c), end, v);
            put_planes8<Planes<V>::N>(a.packed, a.plane, row * a.ld + c, v);
        }
    }
    if (r < a.rows) {
        label = label_of(a, r);
        const long long at = r * a.slots;
        float top = -INFINITY;
        int any = 0;
#pragma unroll 4
        for (int s = lane; s < room; s += 32) {
            long long v = s == a.slots ? label : -1;
            float l = 0.f;
            if (s < a.slots) {
                v = a.ids_64 ? static_cast<const long long *>(a.ids)[at + s] : static_cast<const int *>(a.ids)[at + s];
                l = __ldg(a.logits + at + s);
                any |= v >= 0;
                if (v < 0) l = -INFINITY;
                if (v >= a.vocab) l = NAN;
                else top = fmaxf(top, l);
            }
            const int id = v >= 0 && v < a.vocab ? (int)v : s < a.width ? NONE - s : NONE;   // behind every column, no two of the row alike
            if (!many) {
                ids[s] = id;
                sorted[s] = -1;
            } else if (s < a.slots) {
                keys[s] = (Key)id << 32 | s;
            }
            logits[s] = l;
        }
        for (int s = a.slots + lane; s < keyed; s += 32) keys[s] = ~0ull;
        taught = __any_sync(0xffffffffu, any);
        float log_sum;
        if (a.lse != nullptr) {
            log_sum = __ldg(a.lse + r);
        } else {
            top = warp_max(top);
            float sum = 0.f;
            for (int s = lane; s < a.slots; s += 32)
                if (logits[s] > -INFINITY) sum += expf(logits[s] - top);
            sum = warp_sum(sum);
            log_sum = top + logf(sum);
        }
        __syncwarp();
        const auto share = [&](int s) {
            if (s < a.slots) return logits[s] == -INFINITY ? 0.f : expf(logits[s] - log_sum);   // also where no logit is finite
            return label < 0 ? 0.f : label < a.vocab ? -1.f : -INFINITY;
        };
        const int own = label >= 0 && label < a.vocab ? (int)label : NONE;
        if constexpr (many) {
            Key x[R];
#pragma unroll
            for (int k = 0; k < R; k++) x[k] = keys[32 * k + lane];
            sort_warp(x);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < R; k++) keys[lane * R + k] = x[k];
            __syncwarp();
            // the label behind the candidates that name its column
            for (int k = lane; k < a.slots; k += 32) {
                const Key x = keys[k];
                const int id = (int)(x >> 32);
                const long long at = (k + (a.slots < a.width && id > own)) * a.rows + row;
                a.sorted[at] = id;
                a.weight[at] = share((int)(x & 0xffff));
            }
            if (a.slots < a.width) {
                int low = 0, high = a.slots;   // candidates up to its column
                while (low < high) {
                    const int mid = (low + high) / 2;
                    if ((int)(keys[mid] >> 32) <= own) low = mid + 1;
                    else high = mid;
                }
                if (lane == 0) {
                    a.sorted[low * a.rows + row] = own;
                    a.weight[low * a.rows + row] = share(a.slots);
                }
            }
        }
        // Places by smaller columns alone, four targets a lane at a time (one read of the others serves them all; with the question for
        // equal ones asked each time, 100 targets of 3001 rows took 30 us).  A place that nobody took tells that a column was
        // named twice: then the earlier one comes first.
        bool twice = false;
        const auto put = [&](auto before) {
            for (int s0 = lane; s0 < a.width; s0 += 128) {
                int id[4], place[4] = {};
#pragma unroll
                for (int q = 0; q < 4; q++) id[q] = s0 + 32 * q < a.width ? ids[s0 + 32 * q] : 0;
#pragma unroll 2
                for (int j = 0; j < room; j += 4) {
                    const int4 x = *reinterpret_cast<const int4 *>(ids + j);
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        place[q] += before(x.x, j, id[q], s0 + 32 * q) + before(x.y, j + 1, id[q], s0 + 32 * q) +
                                    before(x.z, j + 2, id[q], s0 + 32 * q) + before(x.w, j + 3, id[q], s0 + 32 * q);
                }
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const int s = s0 + 32 * q;
                    if (s >= a.width) break;
                    sorted[place[q]] = id[q];
                    a.sorted[place[q] * a.rows + row] = id[q];
                    a.weight[place[q] * a.rows + row] = share(s);
                }
            }
            __syncwarp();
        };
        if constexpr (!many) {
            put([](int x, int, int id, int) { return (int)(x < id); });
            for (int s = lane; s < a.width; s += 32) twice |= sorted[s] < 0;
            if (__any_sync(0xffffffffu, twice)) put([](int x, int j, int id, int s) { return (int)(x < id || (x == id && j < s)); });
        }
        // how many targets lie before group g: steps of halves, five searches at a time under one another's latency (as a walk
        // along the targets, 786 groups of 3001 rows took 20 us)
        int half = 1;
        const int entries = many ? a.slots : a.width;   // the label is beside the keys
        while (2 * half <= entries) half *= 2;
        const auto beyond = [&](int g) { return many && a.slots < a.width && (unsigned)own < (unsigned)g * GROUP ? 1 : 0; };
        for (int g0 = 0; g0 < a.groups && a.marks != nullptr; g0 += 128) {
            int at[5] = {};
            for (int step = half; step > 0; step /= 2) {
#pragma unroll
                for (int q = 0; q < 5; q++) {
                    const int k = at[q] + step;
                    if (k <= entries && (unsigned)(many ? (int)(keys[k - 1] >> 32) : sorted[k - 1]) < (unsigned)(g0 + 32 * q + lane) * GROUP) at[q] = k;
                }
            }
#pragma unroll
            for (int q = 0; q < 5; q++) at[q] += beyond(g0 + 32 * q + lane);
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int g = g0 + 32 * q + lane;
                const int first_then = __shfl_sync(0xffffffffu, at[q + 1], 0), beside = __shfl_down_sync(0xffffffffu, at[q], 1);
                if (g < a.groups) a.marks[row * a.groups + g] = at[q] | ((lane < 31 ? beside : first_then) - at[q]) << 16;
            }
        }
    }
    if constexpr (!PACK) count(a, lane == 0 && label >= 0, lane == 0 && taught);
}

// The blocks' counts joined into the first, where they are many: every block of vocab_rows_kernel reads them all, and their number grows with
// the rows as that of the counts does.  Forward of rows of 8 over 64 columns with a candidate each, 8 rows a count: 2^21 rows 36.4 ms ->
// 3.1, 2^17 273 us -> 209; 16384 (2048 counts) 39.6 -> 37.4, 8192 25.2 -> 27.2.
constexpr int MANY_COUNTS = 2048;
__global__ void __launch_bounds__(1024) vocab_sum_counts_kernel(int2 *counts, int blocks)
{
    __shared__ int2 part[32];
    chain_start();
    chain_wait();
    int2 n = make_int2(0, 0);
#pragma unroll 8
    for (int b = threadIdx.x; b < blocks; b += 1024) {
        const int2 c = counts[b];
        n.x += c.x;
        n.y += c.y;
    }
    n.x = __reduce_add_sync(0xffffffffu, n.x);
    n.y = __reduce_add_sync(0xffffffffu, n.y);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = n;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    n = part[threadIdx.x];
    n.x = __reduce_add_sync(0xffffffffu, n.x);
    n.y = __reduce_add_sync(0xffffffffu, n.y);
    if (threadIdx.x == 0) counts[0] = n;
}

// What a row with a label, or with candidates, weighs in the loss; 0 where no row has one, so that what the others weigh is still a
// factor of the products.  (With a label's weight beside a teacher alone, 1/n was in dz: at n = 3891 the whole gradient was 0.0019 off.)
struct Weights {
    const int2 *counts;
    int blocks, mean;
    float label, teacher;
};
// By a block of T threads: x the label's, y the teacher's.
template <int T> __device__ __forceinline__ float2 weigh(const Weights &w, int2 *part)
{
    int2 n = make_int2(0, 0);
#pragma unroll 4
    for (int b = threadIdx.x; b < w.blocks; b += T) {
        const int2 c = w.counts[b];
        n.x += c.x;
        n.y += c.y;
    }
    n.x = __reduce_add_sync(0xffffffffu, n.x);
    n.y = __reduce_add_sync(0xffffffffu, n.y);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = n;
    __syncthreads();
    n = make_int2(0, 0);
#pragma unroll
    for (int i = 0; i < T / 32; i++) {
        n.x += part[i].x;
        n.y += part[i].y;
    }
    return make_float2(n.x == 0 ? 0.f : w.mean ? w.label / (float)n.x : w.label, n.y == 0 ? 0.f : w.mean ? w.teacher / (float)n.y : w.teacher);
}

// The rows of a piece: their lse, losses and the weights of their gradients.
struct Rows {
    const float2 *parts;         // [groups][count]
    int groups, width;
    long long first, count, all; // the piece's first row, its rows, the call's rows
    float *weight;               // [width][all] from the piece's first row on; becomes tau for a backward pass
    const float *z;              // the same places
    float2 *info;                // [count]: lse in base-2 units, c; null: no backward
    float *losses;               // [2][all]
    Weights w;
    float *factor;               // the weight that tau and c leave to the products
    int *done;
    int blocks;                  // of all pieces
    const int *active, *index;   // packed rows: how many there are, and which they were; null: every row is its own
    float *loss;
};

// A block of T threads joins the groups of its ROWS rows, then a warp takes a row's targets.  The block that finishes last
// adds up the rows' losses, in the same order whichever block it is and however the rows were cut.
template <int T> __global__ void __launch_bounds__(T) vocab_rows_kernel(const Rows a)
{
    constexpr int E = T / ROWS;   // threads that share a row's groups
    __shared__ float2 part[E][ROWS + 1];
    __shared__ int2 counted[T / 32];
    __shared__ float2 lost[T / 32];
    __shared__ int last;
    chain_start();
    chain_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = threadIdx.x % ROWS, each = threadIdx.x / ROWS;
    const float2 w = weigh<T>(a.w, counted);
    // The larger weight is the products' factor: the other's ratio to it may vanish, but not overflow (1 to 1e-39), and what its rounding to
    // bf16 with dz brings to all of its targets alike is a part of the smaller half of the gradient.
    const float most = fmaxf(w.x, w.y), factor = most > 0.f ? most : 1.f;
    const float2 share = make_float2(w.x / factor, w.y / factor);
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.info != nullptr) *a.factor = factor;
    const long long r0 = (long long)blockIdx.x * ROWS, count = a.active != nullptr ? min(a.count, *a.active - a.first) : a.count;
    float top = -INFINITY, sum = 0.f;
    const auto join = [&](float2 q) {   // a group without a finite score has the sum 0, or NaN
        if (q.x > top) {
            sum = sum * ex2(top - q.x) + q.y;
            top = q.x;
        } else {
            sum += q.x == -INFINITY ? q.y : q.y * ex2(q.x - top);
        }
    };
    if (r0 + row < count) {
        const float2 *p = a.parts + r0 + row;
        int g = each;
        for (; g + 7 * E < a.groups; g += 8 * E) {
            float2 q[8];
#pragma unroll
            for (int k = 0; k < 8; k++) q[k] = __ldcs(p + (g + k * (long long)E) * a.count);
#pragma unroll
            for (int k = 0; k < 8; k++) join(q[k]);
        }
        if (g < a.groups) {
            float2 q[8];
#pragma unroll
            for (int k = 0; k < 8; k++) q[k] = g + k * E < a.groups ? __ldcs(p + (g + k * (long long)E) * a.count) : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int k = 0; k < 8; k++) join(q[k]);
        }
    }
    part[each][row] = make_float2(top, sum);
    __syncthreads();
    const long long r = r0 + warp;
    float label = 0.f, teacher = 0.f;
    if (warp < ROWS && r < count) {
        top = -INFINITY;
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < E; k += 32) join(part[k + lane][warp]);
        const float all = warp_max(top);
        sum = warp_sum(top == -INFINITY ? sum : sum * ex2(top - all));
        top = all;
        const float lse2 = top + log2f(sum), lse = lse2 * kLn2;
        float c = 0.f;
        for (int s0 = lane; s0 < a.width; s0 += 128) {
            float t[4], z[4];
#pragma unroll
            for (int q = 0; q < 4; q++) {   // asked for together; a score that no target names is not used
                const long long at = (s0 + 32 * q) * a.all + r;
                t[q] = s0 + 32 * q < a.width ? a.weight[at] : 0.f;
                z[q] = s0 + 32 * q < a.width ? a.z[at] : 0.f;
            }
#pragma unroll
            for (int q = 0; q < 4; q++) {
                float tau = 0.f;
                if (t[q] == -1.f) {
                    label = lse - z[q];
                    tau = share.x;
                } else if (t[q] != 0.f) {
                    // a candidate that is no column: NaN; a label: -inf
                    if (t[q] == -INFINITY) label = NAN;
                    else teacher = t[q] == t[q] ? fmaf(t[q], logf(t[q]) + (lse - z[q]), teacher) : NAN;
                    tau = t[q] == -INFINITY ? NAN : share.y * t[q];
                }
                c += tau;
                if (a.info != nullptr && s0 + 32 * q < a.width) a.weight[(s0 + 32 * q) * a.all + r] = tau;
            }
        }
        label = warp_sum(label);
        teacher = warp_sum(teacher);
        c = warp_sum(c);
        if (lane == 0) {
            const long long was = a.index != nullptr ? a.index[a.first + r] : a.first + r;
            a.losses[was] = label;
            a.losses[a.all + was] = teacher;
            if (a.info != nullptr) a.info[r] = make_float2(lse2, c);
            __threadfence();
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.done, 1) == a.blocks - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    // compensated, so that millions of rows lose nothing
    float2 s = make_float2(0.f, 0.f), low = s;
    const auto add = [](float &sum, float &low, float x) {
        const float y = x - low, t = sum + y;
        low = fabsf(t) < INFINITY ? (t - sum) - y : 0.f;
        sum = t;
    };
#pragma unroll 8
    for (long long i = threadIdx.x; i < a.all; i += T) {
        add(s.x, low.x, __ldcg(a.losses + i));
        add(s.y, low.y, __ldcg(a.losses + a.all + i));
    }
    s.x = warp_sum(s.x);
    s.y = warp_sum(s.y);
    if (lane == 0) lost[warp] = s;
    __syncthreads();
    if (threadIdx.x > 0) return;
    s = lost[0];
#pragma unroll
    for (int i = 1; i < T / 32; i++) {
        s.x += lost[i].x;
        s.y += lost[i].y;
    }
    *a.loss = w.x * s.x + w.y * s.y;
}

// ------------------------------------------------------------------ few rows, forward

// A block a row whose scores lie in memory (a few rows' scores are small): its lse, and its targets' scores where they are.
// Nothing has to be sorted or counted before: one token's loss is two launches.
struct Few {
    Targets t;
    const float *z;              // [rows][vocab]
    float label, teacher;        // weights of the losses
    int mean;
    float *losses, *loss;        // loss: of one row; null: there are more
};

constexpr int FEW = 1024;        // threads of a row
template <typename F> __device__ __forceinline__ float block_join(float x, float *part, const F &join)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = join(x, __shfl_xor_sync(0xffffffffu, x, o));
    __syncthreads();
    if (lane == 0) part[warp] = x;
    __syncthreads();
    x = part[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = join(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

__global__ void __launch_bounds__(FEW) vocab_few_kernel(const Few a)
{
    __shared__ float part[32];
    chain_start();
    chain_wait();
    const Targets &t = a.t;
    const auto add = [](float x, float y) { return x + y; };
    const auto most = [](float x, float y) { return fmaxf(x, y); };
    const long long r = blockIdx.x;
    const float *z = a.z + r * t.vocab;
    float top = -INFINITY, sum = 0.f;
    const auto take = [&](float x) {   // NaN ends up in the sum
        if (x > top) {
            sum *= ex2((top - x) * kLog2e);
            top = x;
        }
        sum += x == -INFINITY ? 0.f : ex2((x - top) * kLog2e);
    };
    long long v = threadIdx.x;
    for (; v + 7 * FEW < t.vocab; v += 8 * FEW) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; k++) x[k] = __ldcg(z + v + k * FEW);
#pragma unroll
        for (int k = 0; k < 8; k++) take(x[k]);
    }
    for (; v < t.vocab; v += FEW) take(__ldcg(z + v));
    const float all = block_join(top, part, most);
    const float lse = all + logf(block_join(top == -INFINITY ? sum : sum * ex2((top - all) * kLog2e), part, add));

    const long long l = label_of(t, r);
    const float label = l < 0 ? 0.f : l < t.vocab ? lse - __ldcg(z + l) : NAN;
    // the candidates
    float teacher = 0.f;
    if (t.slots > 0) {
        const int s = threadIdx.x;   // at most 1024
        const long long at = r * t.slots + s, id = s < t.slots ? candidate_of(t, at) : -1;
        const float logit = id >= 0 ? __ldg(t.logits + at) : -INFINITY;
        float norm;
        if (t.lse != nullptr) {
            norm = __ldg(t.lse + r);
        } else {
            const float high = block_join(id < t.vocab ? logit : -INFINITY, part, most);
            norm = high + logf(block_join(logit > -INFINITY && id < t.vocab ? expf(logit - high) : 0.f, part, add));
        }
        const float share = logit == -INFINITY ? 0.f : expf(logit - norm);
        if (id >= t.vocab) teacher = NAN;
        else if (share != 0.f) teacher = share * (logf(share) + (lse - __ldcg(z + id)));
        teacher = block_join(teacher, part, add);
    }
    if (threadIdx.x > 0) return;
    a.losses[r] = label;
    a.losses[t.rows + r] = teacher;
    if (a.loss != nullptr) *a.loss = a.label * label + a.teacher * teacher;   // one row: a mean is the row's own
}

// The loss of a few rows: what they have is counted here.
__global__ void __launch_bounds__(32 * ROWS) vocab_few_loss_kernel(const Few a, float *loss)
{
    chain_start();
    chain_wait();
    const Targets &t = a.t;
    __shared__ int labelled, taught;
    if (threadIdx.x == 0) labelled = taught = 0;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = warp; r < (int)t.rows; r += ROWS) {   // a warp a row
        int any = 0;
        for (int s = lane; s < t.slots; s += 32) any |= candidate_of(t, (long long)r * t.slots + s) >= 0;
        any = __any_sync(0xffffffffu, any);
        if (lane == 0) {
            atomicAdd(&labelled, label_of(t, r) >= 0);
            atomicAdd(&taught, any);
        }
    }
    __syncthreads();
    if (threadIdx.x > 0) return;
    float x = 0.f, y = 0.f;
    for (int r = 0; r < (int)t.rows; r++) {
        x += a.losses[r];
        y += a.losses[t.rows + r];
    }
    *loss = a.label / (float)(a.mean ? max(labelled, 1) : 1) * x + a.teacher / (float)(a.mean ? max(taught, 1) : 1) * y;
}

struct Dz {
    const void *e;               // [count][ld] fp16 or fp32
    bf16 *dz;                    // [count][ld], planes apart for fp32 values
    long long ld, plane, vocab;
    const float2 *parts, *info;
    long long count, all;
    const int *sorted;
    const float *tau, *z;
    int width;
    int cols;                    // columns of a block, a multiple of 2048
    const int *active;           // packed rows: how many there are of all pieces; null: `count`
    long long first;
};

// dz = c exp(z - lse) - tau of one row's columns, 8 a thread at a time; then the columns that targets name, from their own
// scores.  Bound by memory: 2 bytes read and written a value (fp32: 4 and 6).
template <typename V> __global__ void __launch_bounds__(256) vocab_dz_kernel(const Dz a)
{
    constexpr int P = Planes<V>::N;
    chain_start();
    chain_wait();
    const long long r = blockIdx.x, c0 = (long long)blockIdx.y * a.cols, c1 = min(a.vocab, c0 + a.cols);
    float2 info = make_float2(0.f, 0.f);
    if (a.active != nullptr) {
        // zeros behind the last row, as many as dW's last stage along k takes
        const long long n = min(a.count, max(0LL, *a.active - a.first));
        if (r >= n && r >= (max(n, a.first == 0 ? 1LL : 0LL) + 63) / 64 * 64) return;
        if (r < n) info = a.info[r];
    } else {
        info = a.info[r];
    }
    for (long long v = c0 + 8 * threadIdx.x; v < c1; v += 8 * 256) {
        const long long at = r * a.ld + v;
        float x[8];
        if (info.y == 0.f) {   // nothing passes, whatever the scores are
#pragma unroll
            for (int k = 0; k < 8; k++) x[k] = 0.f;
        } else {
            const float f = info.y * ex2(__ldg(&a.parts[v / GROUP * a.count + r].x) - info.x);
            if constexpr (P == 1) {
                const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __half *>(a.e) + at);
                const uint32_t h[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h[k]));
                    x[2 * k] = f * y.x;
                    x[2 * k + 1] = f * y.y;
                }
            } else {
                const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(a.e) + at);
                const float4 y = q[0], z = q[1];
                x[0] = f * y.x; x[1] = f * y.y; x[2] = f * y.z; x[3] = f * y.w;
                x[4] = f * z.x; x[5] = f * z.y; x[6] = f * z.z; x[7] = f * z.w;
            }
        }
        put_planes8<P>(a.dz, a.plane, at, x);   // up to 7 values of padding
    }
    if (info.y == 0.f) return;
    __syncthreads();
    for (int s = threadIdx.x; s < a.width; s += 256) {
        const int id = a.sorted[s * a.all + r];
        if (id < c0 || id >= c1) continue;
        if (s > 0 && a.sorted[(s - 1) * a.all + r] == id) continue;   // the first of its column takes them all
        float tau = a.tau[s * a.all + r];
        for (int j = s + 1; j < a.width && a.sorted[j * a.all + r] == id; j++) tau += a.tau[j * a.all + r];
        const float d = fmaf(info.y, ex2(fmaf(a.z[s * a.all + r], kLog2e, -info.x)), -tau);
        bf16 *out = a.dz + r * a.ld + id;
        if constexpr (P == 1) {
            *out = __float2bfloat16_rn(d);
        } else {
            split3(d, out[0], out[a.plane], out[2 * a.plane]);
        }
    }
}

// dx of packed rows back in their places, zeros for the others.  W: a vector of a row's bytes, or 2 of them.
template <typename W> __global__ void __launch_bounds__(256) vocab_unpack_kernel(const W *packed, const int *place, long long rows, int words, W *dx)
{
    chain_start();
    chain_wait();
    const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= rows) return;
    const int from = place[r];
    for (int i = threadIdx.x & 31; i < words; i += 32) dx[r * words + i] = from >= 0 ? packed[(long long)from * words + i] : W();
}

// The sums of dW over pieces, rounded.
__global__ void __launch_bounds__(256) vocab_round_kernel(const float *sum, long long n, bf16 *out)
{
    chain_start();
    chain_wait();
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= n) return;
    if (i + 8 <= n) {
        const float4 a = __ldcs(reinterpret_cast<const float4 *>(sum + i)), b = __ldcs(reinterpret_cast<const float4 *>(sum + i + 4));
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        put_planes8<1>(out, 0, i, x);
    } else {
        for (long long j = i; j < n; j++) out[j] = __float2bfloat16_rn(sum[j]);
    }
}

// ------------------------------------------------------------------ host side

inline int planes_of(const csa_vocab_loss_params &p) { return p.dtype == CSA_F32 ? 3 : 1; }

// Bytes of the scores that a backward pass keeps at once, unless the caller names the rows of a piece: small beside the GPU's
// memory, and large enough that dW's sums are read and written again but once in 16384 rows of a vocabulary of 131072.
constexpr long long kKept = 4LL << 30;

// A gradient's product with its k axis cut for more than one round of tiles too, where that fills the last one: dx of 3001 x 1024
// over 50257 columns has 48 tiles for 76 pairs, in three pieces 144 (220 us -> 170).  Times as in plan_product.  Of rows that the
// device counts, a third of the weight goes to a count of three quarters of them (fp32 dx of 517 x 768 over 50257 columns, 414 rows
// with a label: 224 us in 4 pieces, which fill the pairs with 517 rows, 162 in 12).
Plan cut_further(Plan p, long long M, long long N, long long K, bool counted)
{
    if (p.shape == LONE_64) return p;
    const int bn = p.shape == PAIR_256 ? 256 : 128;
    const double slots = kSms / 2, step = p.shape == PAIR_256 ? 0.28 : p.exact ? 0.90 : 0.20;
    const long long steps = (K + 63) / 64;
    const auto of_rows = [&](long long m, long long cut) {
        const double tiles = (double)((m + 255) / 256) * ((N + bn - 1) / bn);
        const long long per = (steps + cut - 1) / cut;
        return ceil(tiles * cut / slots) * per * step + (cut > 1 ? 2.5 + (double)M * N * 8 * cut / 4e6 : 0.0);
    };
    const auto time = [&](long long cut) { return counted ? (2 * of_rows(M, cut) + of_rows(M - M / 4, cut)) / 3 : of_rows(M, cut); };
    long long best = p.splits;
    for (long long cut = p.splits; cut <= 16 && cut * 16 <= steps; cut++)
        if (time(cut) < 0.97 * time(best)) best = cut;
    const long long per = (steps + best - 1) / best;
    p.splits = (int)((steps + per - 1) / per);
    return p;
}

// Few rows' scores by the projections' kernels for few rows, which run at the speed of the pass over the weight (a token over
// 32000 x 2048: 28 us, 19.3 of which W's bytes take; on tiles 37).
inline csa_linear_params product_of(const csa_vocab_loss_params &p)
{
    csa_linear_params q = {};
    q.dtype = p.dtype;
    q.out_dtype = CSA_F32;
    q.in_features = p.features;
    q.out_features = p.vocab;
    q.alpha = p.alpha;
    q.rows = p.rows;
    q.x_stride = p.x_stride;
    return q;
}
inline bool few_rows(const csa_vocab_loss_params &p) { return small_linear(product_of(p)); }

// A row of scores ends with a whole block of 64, as one copy of the product that makes dW takes them (50257 columns of 3001 rows
// by 1024: 200 us in copies of 64 columns, 170 in one).
inline long long ld_of(long long vocab) { return (vocab + 63) & ~63LL; }

// Rows without a target are left out of the products where that costs little beside them: packing x and unpacking dx move 8 M K
// bytes, 350 / V of the products' time (2 % at 16384 columns), and the products' kernels for counted rows have the largest tiles.
// Counting costs 6 us a call (1000 rows of 2048 over 65536 columns, all with candidates: 192 us -> 198), and its bits, which every
// block reads, 0.1 ms of 2^18 rows.
inline bool packs(const csa_vocab_loss_params &p)
{
    return p.rows > 256 && p.rows <= 1 << 18 && p.vocab >= 16384 && p.features >= 512;
}

struct Layout {
    bool packed;
    bool stage_x, stage_w;
    long long piece;     // rows of a piece
    int pieces, width, groups;
    linear::Plan dx, dw;
    long long e_rows;   // of the scores that are kept
    size_t off_x, off_w, off_sorted, off_weight, off_marks, off_z, off_counts, off_activity, off_index, off_place, off_losses, off_info, off_parts, off_e,
        off_dz, off_dx, off_sum, off_part, total;
};
Layout plan(const csa_vocab_loss_params &p, bool backward)
{
    Layout b = {};
    const long long M = p.rows, K = p.features, V = p.vocab, ld = ld_of(V);
    if (M == 0) return b;
    size_t at = 0;
    const auto take = [&](size_t &off, size_t bytes) {
        off = at;
        at += up256(bytes);
    };
    if (!backward && few_rows(p)) {
        take(b.off_z, (size_t)M * V * 4);
        take(b.off_losses, (size_t)M * 8);
        b.total = at;
        return b;
    }
    b.width = p.slots + 1;
    b.groups = (int)((V + GROUP - 1) / GROUP);
    // a piece's bytes a row: the scores, or the groups' sums alone
    const long long row = backward ? ld * (p.dtype == CSA_F32 ? 10 : 2) : (long long)b.groups * 8;
    long long most = p.piece_rows > 0 ? p.piece_rows : kKept / row / 256 * 256;
    if (most < 256 && p.piece_rows <= 0) most = 256;
    b.packed = packs(p);
    if (b.packed && most > 65536) most = 65536;   // dW's k axis in one piece
    b.piece = M < most ? M : most;
    b.pieces = (int)((M + b.piece - 1) / b.piece);
    if (p.piece_rows <= 0 && b.pieces > 1) {  // of one size, whole tiles
        b.piece = ((M + b.pieces - 1) / b.pieces + 255) / 256 * 256;
        b.pieces = (int)((M + b.piece - 1) / b.piece);
    }
    b.stage_x = staged(p.dtype, p.x_stride);
    b.stage_w = staged(p.dtype, K);
    b.e_rows = b.packed ? (b.piece + 63) / 64 * 64 : b.piece;
    take(b.off_x, b.packed ? staged_bytes(p.dtype, M + TAIL, K) : b.stage_x ? staged_bytes(p.dtype, M, K) : 0);
    take(b.off_w, b.stage_w ? staged_bytes(p.dtype, V, K) : 0);
    take(b.off_sorted, (size_t)M * b.width * 4);
    take(b.off_weight, (size_t)M * b.width * 4);
    take(b.off_marks, p.slots > 0 ? (size_t)M * b.groups * 4 : 0);
    take(b.off_z, (size_t)M * b.width * 4);
    take(b.off_counts, (size_t)((M + ROWS - 1) / ROWS) * 8 + 16);   // behind the count of finished blocks, the factor and the count of packed rows
    if (b.packed) {
        take(b.off_activity, (size_t)((M + 31) / 32) * 4);
        take(b.off_index, (size_t)M * 4);
        take(b.off_place, (size_t)M * 4);
    }
    take(b.off_losses, (size_t)M * 8);
    take(b.off_info, (size_t)b.piece * 8);
    take(b.off_parts, (size_t)b.piece * b.groups * 8);
    if (backward) {
        take(b.off_e, (size_t)b.e_rows * ld * (p.dtype == CSA_F32 ? 4 : 2));
        b.off_dz = b.off_e;
        if (p.dtype == CSA_F32) take(b.off_dz, (size_t)b.e_rows * ld * 6);
        if (b.packed) take(b.off_dx, (size_t)M * K * (p.dtype == CSA_F32 ? 4 : 2));
        take(b.off_sum, b.pieces > 1 && p.dtype == CSA_BF16 ? (size_t)V * K * 4 : 0);
        b.dx = cut_further(plan_product(b.piece, K, V, planes_of(p), 1, p.dtype == CSA_F32, kSms), b.piece, K, V, false);
        b.dw = cut_further(plan_product(V, K, b.piece, planes_of(p), 1, p.dtype == CSA_F32, kSms), V, K, b.piece, false);
        if (b.packed) {
            const Shape shape = p.dtype == CSA_F32 ? PAIR_128 : PAIR_256;
            b.dx = cut_further({shape, p.dtype == CSA_F32 ? 1 : (int)((V + 65535) / 65536), p.dtype == CSA_F32}, b.piece, K, V, true);
            b.dw = {shape, 1, p.dtype == CSA_F32};
        }
        const size_t dx = b.dx.splits > 1 ? (size_t)b.dx.splits * b.piece * partial_stride(K) * 4 : 0;
        const size_t dw = b.dw.splits > 1 ? (size_t)b.dw.splits * V * partial_stride(K) * 4 : 0;
        take(b.off_part, dx > dw ? dx : dw);
    }
    b.total = at;
    return b;
}

cudaError_t sms_here(int *sms)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (*sms < 2) *sms = 2;
    return e;
}

}  // namespace vocab

using namespace vocab;

#define VOC_TRY(x)                        \
    do {                                  \
        const cudaError_t e_ = (x);       \
        if (e_ != cudaSuccess) return e_; \
    } while (0)

size_t vocab_loss_workspace(const csa_vocab_loss_params &p, bool backward) { return plan(p, backward).total; }

cudaError_t launch_vocab_loss(const csa_vocab_loss_params &p, const void *x, const void *weight, const csa_vocab_targets &t, float *loss,
                              float *row_loss, void *dx, void *dw, bool backward, void *ws, cudaStream_t st)
{
    const long long M = p.rows, K = p.features, V = p.vocab, ld = ld_of(V);
    const int planes = planes_of(p);
    const size_t size = p.dtype == CSA_F32 ? 4 : 2;
    if (M == 0) {
        if (dw != nullptr) VOC_TRY(cudaMemsetAsync(dw, 0, (size_t)V * K * size, st));
        return cudaMemsetAsync(loss, 0, 4, st);
    }
    const Layout b = plan(p, backward);
    char *w = static_cast<char *>(ws);
    Targets g = {};
    g.labels = t.labels;
    g.ids = t.teacher_ids;
    g.logits = t.teacher_logits;
    g.lse = t.teacher_lse;
    g.labels_64 = p.labels_64;
    g.ids_64 = p.ids_64;
    g.slots = p.slots;
    g.rows = M;
    g.vocab = V;
    float *losses = row_loss != nullptr ? row_loss : reinterpret_cast<float *>(w + b.off_losses);
    if (!backward && few_rows(p)) {
        note_path("generic");
        Epilogue e = {};
        e.alpha = p.alpha;
        e.out = w + b.off_z;
        e.out_f32 = 1;
        VOC_TRY(launch_linear_small(product_of(p), x, weight, e, kSms, st));
        const Few f = {g, reinterpret_cast<const float *>(w + b.off_z), p.label_weight, p.teacher_weight, p.reduction == 0, losses, M == 1 ? loss : nullptr};
        VOC_TRY(launch_chained(vocab_few_kernel, dim3((unsigned)M), FEW, 0, 1, st, f));
        return M == 1 ? cudaSuccess : launch_chained(vocab_few_loss_kernel, dim3(1), 32 * ROWS, 0, 1, st, f, loss);
    }
    note_path("tcgen05");
    int sms = 0;
    VOC_TRY(sms_here(&sms));
    Stage job[2] = {};
    Operand ox = {};
    if (b.packed) {   // by the kernel that prepares the targets
        ox.base = reinterpret_cast<bf16 *>(w + b.off_x);
        ox.ld = up8(K);
        ox.plane = (M + TAIL) * ox.ld;
        ox.k_major = true;
    } else {
        ox = operand(p.dtype, x, p.x_stride, M, (int)K, b.stage_x, w + b.off_x, true, &job[0]);
    }
    Operand ow = operand(p.dtype, weight, K, V, (int)K, b.stage_w, w + b.off_w, true, &job[1]);
    VOC_TRY(run_stages(p.dtype, job, st));

    g.width = p.slots + (t.labels != nullptr);
    g.sorted = reinterpret_cast<int *>(w + b.off_sorted);
    g.weight = reinterpret_cast<float *>(w + b.off_weight);
    g.marks = reinterpret_cast<int *>(w + b.off_marks);
    g.groups = b.groups;
    g.done = reinterpret_cast<int *>(w + b.off_counts);
    float *factor = reinterpret_cast<float *>(g.done + 1);
    g.counts = reinterpret_cast<int2 *>(w + b.off_counts) + 1;
    g.losses = losses;
    const bool single = p.slots == 0;
    if (single) g.marks = nullptr;
    unsigned blocks = (unsigned)((M + ROWS - 1) / ROWS);
    const size_t smem = (size_t)prepare_bytes(p.slots, g.width) * ROWS;
#define VOC_PREPARE(V, PACK) of_keys(vocab_prepare_kernel<V, PACK, 0>, vocab_prepare_kernel<V, PACK, 8>, vocab_prepare_kernel<V, PACK, 16>, vocab_prepare_kernel<V, PACK, 32>)
    const auto of_keys = [&](auto few, auto r8, auto r16, auto r32) { return p.slots <= MANY ? few : p.slots <= 256 ? r8 : p.slots <= 512 ? r16 : r32; };
    const auto prepare = [&](void (*kernel)(Targets)) {
        const cudaError_t e = smem > 48 << 10 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) : cudaSuccess;
        return e != cudaSuccess ? e : launch_chained(kernel, dim3(blocks), 32 * ROWS, smem, 1, st, g);
    };
    if (b.packed) {
        g.active = g.done + 2;
        g.counts++;   // behind it
        g.activity = reinterpret_cast<uint32_t *>(w + b.off_activity);
        g.index = reinterpret_cast<int *>(w + b.off_index);
        g.place = reinterpret_cast<int *>(w + b.off_place);
        g.x = x;
        g.x_stride = p.x_stride;
        g.packed = const_cast<bf16 *>(ox.base);
        g.ld = ox.ld;
        g.plane = ox.plane;
        g.features = (int)K;
        const unsigned words = (unsigned)((M + 31) / 32);
        VOC_TRY(launch_chained(vocab_count_kernel, dim3(words), 1024, 0, 1, st, g));
        blocks = (words * 32 + TAIL) / ROWS;
        VOC_TRY(prepare(p.dtype == CSA_F32 ? VOC_PREPARE(float, true) : VOC_PREPARE(bf16, true)));
        blocks = words;   // of the counts
    } else if (single) {
        blocks = (unsigned)((M + 255) / 256);
        VOC_TRY(launch_chained(vocab_labels_kernel, dim3(blocks), 256, 0, 1, st, g));
    } else {
        VOC_TRY(prepare(VOC_PREPARE(bf16, false)));
    }

    if (blocks > MANY_COUNTS) {
        VOC_TRY(launch_chained(vocab_sum_counts_kernel, dim3(1), 1024, 0, 1, st, const_cast<int2 *>(g.counts), (int)blocks));
        blocks = 1;
    }
    const bool grads = dx != nullptr || dw != nullptr;
    const Weights weights = {g.counts, (int)blocks, p.reduction == 0, p.label_weight, p.teacher_weight};
    float *z = reinterpret_cast<float *>(w + b.off_z);
    float2 *parts = reinterpret_cast<float2 *>(w + b.off_parts), *info = grads ? reinterpret_cast<float2 *>(w + b.off_info) : nullptr;
    int all_blocks = 0;
    for (long long first = 0; first < M; first += b.piece) all_blocks += (int)(((M - first < b.piece ? M - first : b.piece) + ROWS - 1) / ROWS);
    for (long long first = 0; first < M; first += b.piece) {
        const long long count = M - first < b.piece ? M - first : b.piece;
        Operand px = ox;
        px.base += first * ox.ld;
        Scores s = {};
        s.ids = g.sorted + first;
        s.marks = single ? nullptr : g.marks + first * g.groups;
        s.groups = g.groups;
        s.z = z + first;
        s.slots = g.width;
        s.ld = M;
        s.parts = parts;
        s.alpha = p.alpha;
        s.e = grads ? w + b.off_e : nullptr;
        s.lde = ld;
        s.counted = g.active;
        s.first = first;
        VOC_TRY(launch_scores(px, ow, count, V, K, planes, s, sms, st));
        const int row_blocks = (int)((count + ROWS - 1) / ROWS);
        const Rows rows = {parts, b.groups, g.width, first, count, M, g.weight + first, z + first, info, losses, weights,
                           factor, g.done, all_blocks, g.active, g.index, loss};
        // Blocks of one or two rounds: more threads share a row (270 rows of 147322 columns with 180 candidates: 479 us -> 428 of the
        // whole call, 2400 of 65536: 379 -> 367; but 4096 of 65536: 345 -> 365), unless they have few groups (2400 of 16000: 35 -> 39).
        const bool wide = M <= 2LL * kSms * ROWS && b.groups >= 512;
        VOC_TRY(launch_chained(wide ? vocab_rows_kernel<1024> : vocab_rows_kernel<32 * ROWS>, dim3((unsigned)row_blocks), wide ? 1024 : 32 * ROWS, 0, 1, st, rows));
        if (!grads) continue;
        Dz d = {};
        d.e = w + b.off_e;
        d.dz = reinterpret_cast<bf16 *>(w + b.off_dz);
        d.ld = ld;
        d.plane = b.e_rows * ld;
        d.active = g.active;
        d.first = first;
        d.vocab = V;
        d.parts = parts;
        d.info = info;
        d.count = count;
        d.all = M;
        d.sorted = g.sorted + first;
        d.tau = rows.weight;
        d.z = rows.z;
        d.width = g.width;
        // few rows: several blocks each
        const long long chunks = (V + 2047) / 2048, per_row = (4LL * kSms + count - 1) / count;
        d.cols = (int)((chunks + per_row - 1) / per_row) * 2048;
        const long long whole = (count + 63) / 64 * 64;   // stages of dW's k axis
        const dim3 grid((unsigned)(b.packed ? whole : count), (unsigned)((V + d.cols - 1) / d.cols));
        VOC_TRY(launch_chained(p.dtype == CSA_F32 ? vocab_dz_kernel<float> : vocab_dz_kernel<bf16>, grid, 256, 0, 1, st, d));
        Product q = {};
        q.planes = planes;
        q.passes = 1;
        q.e.partial = reinterpret_cast<float *>(w + b.off_part);
        q.e.scale = factor;
        q.counted = g.active;
        q.first = first;
        Operand od = {};
        od.base = d.dz;
        od.ld = ld;
        od.plane = d.plane;
        if (dx != nullptr) {
            q.a = od;
            q.a.k_major = true;
            q.b = ow;
            q.b.k_major = false;
            q.M = count;
            q.N = K;
            q.K = V;
            q.plan = b.dx;
            q.e.alpha = p.alpha;
            q.e.out_f32 = p.dtype == CSA_F32;
            q.along_k = false;
            q.e.out = (b.packed ? w + b.off_dx : static_cast<char *>(dx)) + (size_t)first * K * size;
            VOC_TRY(product(q, st));
        }
        if (dw != nullptr) {
            q.a = od;
            q.a.k_major = false;
            q.a.held = ld;
            q.b = px;
            q.b.k_major = false;
            q.M = V;
            q.N = K;
            q.K = b.packed ? whole : count;
            q.along_k = true;
            q.plan = b.dw;
            // the last piece's k axis may be shorter: no part of it is empty
            const long long steps = (count + 63) / 64, each = (steps + b.dw.splits - 1) / b.dw.splits;
            q.plan.splits = (int)((steps + each - 1) / each);
            q.e.alpha = p.alpha;
            q.e.out_f32 = p.dtype == CSA_F32 || b.pieces > 1;
            q.e.out = p.dtype == CSA_BF16 && b.pieces > 1 ? w + b.off_sum : dw;
            if (first > 0) {   // dW so far
                q.e.res = q.e.out;
                q.e.ldr = K;
            }
            VOC_TRY(product(q, st));
        }
    }
    if (b.packed && dx != nullptr) {
        const char *from = w + b.off_dx;
        const long long bytes = K * (long long)size;
        const dim3 grid((unsigned)((M + 7) / 8));
        if (bytes % 16 == 0) VOC_TRY(launch_chained(vocab_unpack_kernel<uint4>, grid, 256, 0, 1, st, (const uint4 *)from, g.place, M, (int)(bytes / 16), (uint4 *)dx));
        else VOC_TRY(launch_chained(vocab_unpack_kernel<unsigned short>, grid, 256, 0, 1, st, (const unsigned short *)from, g.place, M, (int)(bytes / 2), (unsigned short *)dx));
    }
    if (dw != nullptr && b.pieces > 1 && p.dtype == CSA_BF16) {
        const long long n = V * K;
        VOC_TRY(launch_chained(vocab_round_kernel, dim3((unsigned)((n + 2047) / 2048)), 256, 0, 1, st, reinterpret_cast<float *>(w + b.off_sum), n, (bf16 *)dw));
    }
    return cudaSuccess;
}

}  // namespace csa
