// What the layer products' host code and their kernels share.
#pragma once

#include "gc_internal.hpp"

namespace gc {

enum Kind { kForward, kInput, kWeight };

// D[m][n] = sum_k A[m][k] B[n][k], and what becomes of it.
struct Product {
    const void *A, *B;
    uint64_t lda, ldb;
    uint32_t M, N, K;
    const void *bias;       // forward: [N], or null
    const void *add;        // forward: r; input: a
    const void *z;          // input: the argument of the activation
    void *zout;             // forward
    void *out, *out2;       // forward: y; input: dx, dzx; weight: the segment of g
    uint64_t ldadd, ldz, ldout, ldout2;
    float *gbias;           // weight: the bias' segment of g, or null
    int act;
    int accumulate;         // weight
};

// Tiles of a workgroup, kWR x kWC waves.
struct Big {
    static constexpr int kTM = 256, kTN = 256, kWR = 2, kWC = 4, kWavesPerSimd = 2;
};
struct Mid {
    static constexpr int kTM = 128, kTN = 128, kWR = 2, kWC = 2, kWavesPerSimd = 2;
};
struct Thin {
    static constexpr int kTM = 32, kTN = 128, kWR = 1, kWC = 4, kWavesPerSimd = 4;
};
enum TileShape { kBig, kMid, kThin, kFew };  // kFew: 16 rows of W, no tile

// How the operands get into LDS.
//   kDirect  16-byte pieces go straight there; a stage with the last k inside goes through registers
//   kHeld    through registers: rows of any alignment
//   kAny     through registers element by element: rows or sums shorter than a piece, offsets past 32 bits
enum Mode { kDirect, kHeld, kAny };

// How a product is spread over workgroups: tiles, and parts of the common index
// (stages of 128 bytes of it) whose sums linear_join_kernel adds.
struct Cut {
    TileShape shape;
    uint32_t tiles_m, tiles_n, parts, stages, per;  // per: stages of a part; kFew: parts are waves
    Mode mode;
    float *partial;                                 // parts > 1: sums in register order, a tile after the other
    float *colsums;                                 // and [parts][tiles_m * kTM] of the bias
};

template <class T>
gc_status linear_launch(const char *fn, Kind kind, const Product &p, const Cut &c, hipStream_t stream);
extern template gc_status linear_launch<struct F32>(const char *, Kind, const Product &, const Cut &, hipStream_t);
extern template gc_status linear_launch<struct BF16>(const char *, Kind, const Product &, const Cut &, hipStream_t);
extern template gc_status linear_launch<struct F16>(const char *, Kind, const Product &, const Cut &, hipStream_t);

}  // namespace gc
