// k_vocab.cuh -- what the kernels of the vocabulary's losses share.
#pragma once

#include "k_linear.cuh"

namespace csa {
namespace vocab {

// Columns of the vocabulary whose scores lie in one thread's registers: they share a reference in their exponentials.
constexpr int GROUP = 64;
constexpr int NONE = 0x7fffffff;   // a slot without a column

// Where the scores of a piece of rows go.
struct Scores {
    const int *ids;        // [slots][ld]: the columns that each row's targets name, ascending, NONE behind them
    const int *marks;      // [M][groups]: how many of them lie before each group, and from bit 16 on in it; null: one slot a row
    float *z;              // [slots][ld]: the scores there
    int slots, groups;
    long long ld;
    float2 *parts;         // [groups][M given]: a group's largest score in base-2 units, and the sum of 2^(score - largest)
    float alpha;
    void *e;               // [M][lde] 2^(score - largest): fp16 of bf16 values, fp32 of fp32 ones; null: not kept
    long long lde;
    const int *counted;    // the device's count of rows, of which those before `first` are other pieces'; null: M rows
    long long first;
};

// z = alpha x W^T of M rows and N columns, of operands contiguous along k.
cudaError_t launch_scores(const linear::Operand &x, const linear::Operand &w, long long M, long long N, long long K, int planes, const Scores &s,
                          int sms, cudaStream_t st);

}  // namespace vocab
}  // namespace csa
