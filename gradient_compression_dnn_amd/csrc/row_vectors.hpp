// Which vectors of a row of logits the threads of the loss hold, and the choice
// of its variant.  Plain arithmetic, the same on the host and in the kernel.
#pragma once

#include <cstdint>

namespace gc {

// Threads of a row, vectors that each holds in registers, and whether the row may go on behind those.
struct LossShape {
    int threads, held;
    bool more;
};

// The variant for rows of `vocab` elements, N of them a vector.  even: every row starts on 16 bytes; else a row may
// begin up to N - 1 elements inside its first vector.  As few threads as hold the row: several rows a unit overlap
// better than one (us, 4096 rows of 65536 bf16: 227 with 512 threads, 352 with 1024).
constexpr LossShape loss_shape(uint32_t vocab, uint32_t N, bool even) {
    if (vocab < N) return {256, 0, true};
    const uint32_t vecs = (vocab + (even ? 0 : N - 1) + N - 1) / N;
    if (vecs <= 256 * 4) return {256, 4, false};
    if (vecs <= 256 * 8) return {256, 8, false};
    if (vecs <= 256 * 16) return {256, 16, false};
    if (vecs <= 512 * 16) return {512, 16, false};
    return {512, 16, true};
}

// The vectors held: number i of thread t, C a thread.  Vectors are cut at 16 bytes of memory, so that the row begins
// `skew` elements inside the first.
// kMore is chosen for what the row's skew may be, not for what it is: a row of less skew may end inside the last
// vector of the last thread (65530 to 65535 columns of 16 bits).  It ends in no vector before that one, and none
// begins past its end: vocab + N - 1 > C kStep, so that C kStep - N < vocab.
template <int N, int NT, int C, bool kMore>
struct RowVectors {
    static constexpr uint32_t kStep = NT * N;
    // the column that a vector begins with
    static constexpr int32_t own(int i, uint32_t t, uint32_t skew) { return static_cast<int32_t>(i * kStep + t * N - skew); }
    // whether another one may stand for it
    static constexpr bool moves(int i) { return i == 0 || i == C - 1 || !kMore; }
    // the column of the one that is read and written: the vector that the row begins or ends with stands for the one
    // that crosses its start or end, and for those past it
    static constexpr int32_t column(int i, uint32_t t, uint32_t skew, uint32_t vocab) {
        const int32_t c = own(i, t, skew), in = i == 0 && c < 0 ? 0 : c, last = static_cast<int32_t>(vocab - N);
        return moves(i) && in > last ? last : in;
    }
};

}  // namespace gc
