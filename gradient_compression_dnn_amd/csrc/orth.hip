// Orthogonalised updates of weight matrices (gc_orthogonalize, gc_muon_step):
//
//   X_0 = D / (||D||_F + eps), m x n with m <= n (D or its transpose)
//   A = X X^T,  B = b A + c A^2,  X <- a X + B X       `steps` times
//
// Every product runs on the matrix cores in three fp16 products: an fp32
// value x 2^e is held as hi + lo, hi = fp16(x 2^e), lo = fp16(x 2^e - hi), 22
// bits, and P Q^T = hi hi^T + hi lo^T + lo hi^T with fp32 sums (lo lo^T is
// below the last bit kept).  A third of the fp16 rate, where library products
// in fp32 reach an eighth (154 of 1,247 TFLOP/s at 8192^3).  With five or six of
// the default steps the result is 0.2 to 1.4 times as far from 64 bits as fp32
// products are (up to 0.45 from 600 rows on); with one or two, or with gentle
// coefficients, where fp32 loses only 0.5e-7 to 1e-7, the 22 bits show: 1.3e-7
// to 4.7e-7, up to 5 times as far.
// fp16 has no range to spare, so each array has its own power of two: singular
// values of X_0 are at most 1, the polynomial bounds those of every later X, A
// and B, and no entry exceeds its matrix's largest singular value
// (orth_scales).
//
// All products have the form P Q^T with the common index running along the
// rows of both: X X^T and A A^T (A is symmetric) as they stand, B X = B T^T
// with T = X^T, which is kept beside X.  A and B are symmetric: only tiles on
// and below the diagonal are computed, the others are their mirror images.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <functional>
#include <new>
#include <queue>
#include <string>
#include <vector>

#include "gc_internal.hpp"

namespace gc {

namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct __attribute__((packed, aligned(4))) F32x4 {
    float v[4];
};

// ------------------------------------------------------------------ layout
// A split matrix [rows][ld] (ld a multiple of 32): each row is ld / 32 groups
// of 128 bytes, 32 hi then 32 lo of 32 consecutive columns, so that a group
// of both planes is one cache line.
constexpr uint32_t kPad = 128;  // rows and columns of the split matrices are padded to this with zeros

__host__ __device__ constexpr uint32_t pad_up(uint32_t x) { return (x + kPad - 1) / kPad * kPad; }
// halves from the start of a split row to column k's hi (its lo is 32 on)
__device__ __forceinline__ uint32_t split_at(uint32_t k) { return (k >> 5) * 64 + (k & 31); }

__device__ __forceinline__ void split(float v, _Float16 &hi, _Float16 &lo) {
    hi = static_cast<_Float16>(v);
    lo = static_cast<_Float16>(v - static_cast<float>(hi));
}

// One matrix as the kernels see it.  X is m x n, T = X^T, A and B m x m.
struct MatDev {
    uint64_t off;      // first element in the flat buffer
    uint64_t len;      // R * C
    uint64_t x;        // halves from the workspace arrays' start to this matrix's X (and T)
    uint64_t a;        // and to its A (and B)
    uint32_t R, C;     // as in the flat buffer, row-major
    uint32_t m, n;     // min, max of R and C
    uint32_t mp, np;   // padded
    uint32_t flip;     // R > C: X = D^T
    uint32_t chunk0;   // first norm chunk
    uint32_t nchunk;
    uint32_t reserved;
};

// A workgroup's work: a matrix and a tile (norm: a chunk); products: its
// stages [k0, k1) of 32 columns of the common index, and where a part of a
// split tile goes; joins: k1 parts from `slot` on; slabs: [k0, k1) of a matrix,
// whose j parts begin at slot i, and the slot of their own.
struct Item {
    uint32_t mat, i, j, k0, k1, slot;
};
constexpr uint32_t kNoSlot = 0xFFFFFFFFu;

constexpr int kSplitTile = 64;  // orth_split's tile

// The work lists: D's chunks and tiles, and per kind of product its items and
// the joins of its split tiles; of matrices of few rows, the slabs and the
// matrices with their parts.
enum List { kChunks, kTiles, kGram, kGramJoin, kSquare, kSquareJoin, kApply, kApplyJoin, kSlabs, kSmalls, kLists };

// Products are planned for the workgroups that 256 compute units hold; unit u
// has items [first[u], first[u + 1]) of its list.
struct OrthDev {
    const MatDev *mat;
    const Item *list[kLists];
    const uint32_t *first[kLists];
};

}  // namespace
}  // namespace gc

struct gc_matrix_plan {
    uint64_t n_total = 0;
    uint64_t xhalves = 0, ahalves = 0;  // halves of one X (or T) array and of one A (or B) array
    uint64_t partial = 0;               // floats of split tiles' parts held at once
    bool large[gc::kLists] = {};        // products: tiles of 256 x 256
    bool pairs = false;                 // two steps at a time
    bool narrow = false;                // every matrix has at most kNarrow rows
    bool fused = false;                 // and the slabs' workgroups make B themselves
    std::vector<gc::MatDev> mat;
    std::vector<gc::Item> list[gc::kLists];
    std::vector<uint32_t> first[gc::kLists];  // products only
    std::mutex mu;
    std::vector<std::pair<int, void *>> dev_blob;
};

namespace gc {

namespace {

// ----------------------------------------------------------- tables, scales
struct Blob {
    size_t mat, list[kLists], first[kLists], total;
};

Blob blob_layout(const gc_matrix_plan *p) {
    Blob L{};
    size_t o = 0;
    auto take = [&](size_t bytes) {
        o = (o + 255) & ~size_t(255);
        const size_t at = o;
        o += bytes;
        return at;
    };
    L.mat = take(sizeof(MatDev) * p->mat.size());
    for (int l = 0; l < kLists; ++l) {
        L.list[l] = take(sizeof(Item) * p->list[l].size());
        L.first[l] = take(sizeof(uint32_t) * p->first[l].size());
    }
    L.total = o < 256 ? 256 : o;
    return L;
}

// The plan's tables on the current device, uploaded on first use.
gc_status orth_device(const gc_matrix_plan *cplan, OrthDev *out) {
    gc_matrix_plan *p = const_cast<gc_matrix_plan *>(cplan);
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_error(e, "hipGetDevice");
    const Blob L = blob_layout(p);
    void *blob = nullptr;
    {
        std::lock_guard<std::mutex> lock(p->mu);
        for (auto &pr : p->dev_blob)
            if (pr.first == dev) blob = pr.second;
        if (!blob) {
            std::vector<uint8_t> host;
            try {
                host.resize(L.total);
                p->dev_blob.reserve(p->dev_blob.size() + 1);
            } catch (const std::bad_alloc &) {
                return set_error(GC_EINVAL, "matrix plan tables: out of host memory");
            }
            e = hipMalloc(&blob, L.total);
            if (e != hipSuccess) return hip_error(e, "hipMalloc(matrix plan tables)");
            std::memcpy(host.data() + L.mat, p->mat.data(), sizeof(MatDev) * p->mat.size());
            for (int l = 0; l < kLists; ++l) {
                if (!p->list[l].empty()) std::memcpy(host.data() + L.list[l], p->list[l].data(), sizeof(Item) * p->list[l].size());
                if (!p->first[l].empty())
                    std::memcpy(host.data() + L.first[l], p->first[l].data(), sizeof(uint32_t) * p->first[l].size());
            }
            e = hipMemcpy(blob, host.data(), L.total, hipMemcpyHostToDevice);
            if (e != hipSuccess) {
                (void)hipFree(blob);
                return hip_error(e, "hipMemcpy(matrix plan tables)");
            }
            p->dev_blob.emplace_back(dev, blob);
        }
    }
    auto *b = static_cast<uint8_t *>(blob);
    out->mat = reinterpret_cast<const MatDev *>(b + L.mat);
    for (int l = 0; l < kLists; ++l) {
        out->list[l] = reinterpret_cast<const Item *>(b + L.list[l]);
        out->first[l] = reinterpret_cast<const uint32_t *>(b + L.first[l]);
    }
    return GC_OK;
}

// Exponents of one step's split arrays: X 2^ex, A 2^ea, B 2^eb, where B now is
// a I + b A + c A^2.
struct Scales {
    int ex, ea, eb;
    int es, eq;  // of a pair of steps from this one on: S = B A, and Q
    bool pair;   // whether a pair may begin here
};

// The largest exponent that keeps |v| <= bound below 60000 in fp16.
int exponent_for(double bound) { return static_cast<int>(std::floor(std::log2(60000.0 / bound))); }

// The largest |q(y)| and |x q(x^2)| for y = x^2, x in [0, top], with q(y) = a +
// b y + c y^2: at an end of the range, or where the derivative vanishes.
void largest(double a, double b, double c, double top, double *of_q, double *of_p) {
    const double t2 = top * top;
    auto q = [&](double y) { return std::fabs(a + (b + c * y) * y); };
    auto inside = [&](double y) { return y > 0.0 && y < t2; };  // false for NaN
    *of_q = std::max(q(0.0), q(t2));
    *of_p = top * q(t2);
    const double vertex = -b / (2.0 * c);
    if (inside(vertex)) *of_q = std::max(*of_q, q(vertex));
    const double square = 9.0 * b * b - 20.0 * a * c;  // of a + 3 b y + 5 c y^2 = 0
    if (!(square >= 0.0)) return;
    const double w = -0.5 * (3.0 * b + std::copysign(std::sqrt(square), b));
    for (double y : {w / (5.0 * c), a / w})
        if (inside(y)) *of_p = std::max(*of_p, std::sqrt(y) * q(y));
}

// Bounds of the singular values of X, A and B at every step: the largest value
// of the polynomial on [0, top], and kRounding of the sizes of its terms for
// the step's own roundings (an operand is off by up to 2^-23, A by 2^-21, c A^2
// by 2^-19 of itself).  No more than that: where a schedule is steep at the
// top of its range, what is added at one step comes back 10 to 20 times as
// large at the next.  s[k] is step k's, s[steps] the result's.
// The bounds are worst cases; what a matrix really holds may be smaller by
// as much as the bounds are loose, and where that reaches fp16's subnormals
// the lo parts lose bits (a schedule whose bound rose to 24 and then 3e6 gave
// 5.2e-6 where fp32 gives 2.7e-7).  So false, a refusal, if X's bound passes 8
// before the last step, B's 2^14, the result's 1e12, or one vanishes.
bool orth_scales(const gc_orth_options &o, Scales *s) {
    constexpr double kRounding = 1.0 / (1 << 19);
    double top = 1.0 + kRounding, before = 0.0;
    s[0].ex = exponent_for(top);
    for (int k = 0; k < o.steps; ++k) {
        const double a = o.coef[k][0], b = o.coef[k][1], c = o.coef[k][2];
        const double t2 = top * top;
        double px, pb;
        largest(a, b, c, top, &pb, &px);
        const double next = px + kRounding * (std::fabs(a) + (std::fabs(b) + std::fabs(c) * t2) * t2) * top;
        // before an exponent is formed, which needs bounds that are finite
        if (!(next <= (k + 1 == o.steps ? 1e12 : 8.0)) || !(pb <= 16384.0) || !(next > 1e-12)) return false;
        s[k].ea = exponent_for(t2 * (1.0 + 1.0 / 64));
        s[k].eb = exponent_for(std::max(pb, 1e-12) * (1.0 + 1.0 / 64));
        // S = B A has values s |p(s)|, Q = B' B at most the product of the two bounds
        s[k].es = exponent_for(top * px * (1.0 + 1.0 / 64));
        s[k].pair = false;
        if (k > 0) {
            s[k - 1].eq = exponent_for(before * pb * (1.0 + 1.0 / 32));
            s[k - 1].pair = before * pb <= 16384.0;
        }
        before = pb;
        top = next;
        s[k + 1].ex = exponent_for(top);
    }
    return true;
}

// --------------------------------------------------------------- tile shapes
// kTile x kTile per workgroup by kWR x kWC waves, two stages of 32 columns of
// both planes in LDS; kUnits workgroups at once on 256 compute units.  The
// large tile reads half as much per product, the small one fits small matrices
// and writes out while its neighbour multiplies; the plan's model picks one for
// each kind of product.  Measured, large against small: B A of four matrices of
// 1500 rows 65 us and 76, B X of 4096 x 4096 318 and 353, of ResNet-50's 54
// matrices 112 and 123; their X X^T 75 and 66, their A A^T 55 and 40, X X^T of 28
// matrices of 800 to 2400 rows 655 and 628.  (A small tile with four stages and
// a unit to itself: 1.43 ms for ResNet-50's update where two stages took 1.33.)
struct Large {
    static constexpr uint32_t kUnits = 256;
    static constexpr int kTile = 256, kWR = 2, kWC = 4;
};
struct Small {
    static constexpr uint32_t kUnits = 512;
    static constexpr int kTile = 128, kWR = 2, kWC = 2;
};

// --------------------------------------------------------------- workspace
struct OrthWs {
    _Float16 *X[2], *T[2], *A, *B, *S;
    double *sums, *inv;
    float *partial;
    size_t bytes;
};

OrthWs orth_ws(void *ws, const gc_matrix_plan *p) {
    WsCursor c(ws);
    OrthWs w{};
    for (int k = 0; k < 2; ++k) {
        w.X[k] = c.take<_Float16>(p->narrow ? 0 : p->xhalves);
        w.T[k] = c.take<_Float16>(p->xhalves);
    }
    w.A = c.take<_Float16>(p->ahalves);
    w.B = c.take<_Float16>(p->ahalves);
    w.S = c.take<_Float16>(p->pairs ? p->ahalves : 0);
    w.sums = c.take<double>(p->list[kChunks].size());
    w.inv = c.take<double>(p->mat.size());
    w.partial = c.take<float>(p->partial);
    w.bytes = c.used + 256;  // room to round the base up to 256 bytes
    return w;
}

// ----------------------------------------------------------- momentum, norm
// What is orthogonalised.  U null: D itself.  Otherwise the momentum step on
// (U, G): U <- fl(fl(m U) + G), D = U or fl(fl(m U) + G).
struct Source {
    const float *G;
    float *U;
    float momentum;
    int nesterov;
};

__device__ __forceinline__ float direction(const Source &s, float u, float g) {
    return s.nesterov ? s.momentum * u + g : u;
}

// One chunk of kChunk elements of a matrix: the momentum update and the
// chunk's sum of D^2 in double.  Memory bounds it: 36 M elements with momentum
// take 69 us, 6.3 TB/s.
__global__ __launch_bounds__(kBlock) void orth_norm_kernel(const Item *__restrict__ items, const MatDev *__restrict__ mats,
                                                           Source s, double *__restrict__ sums) {
    const Item it = items[blockIdx.x];
    const MatDev M = mats[it.mat];
    const uint64_t first = static_cast<uint64_t>(it.i) * kChunk;
    const uint32_t cnt = static_cast<uint32_t>(umin64(M.len - first, kChunk));
    const BufRsrc rg = chunk_buf(s.G + M.off + first, cnt);
    double sum = 0.0;
    float g[kRows][4], u[kRows][4];
#pragma unroll
    for (int r = 0; r < kRows; ++r) load4(rg, row_elem(r), g[r]);
    if (s.U) {
        const BufRsrc ru = chunk_buf(s.U + M.off + first, cnt);
#pragma unroll
        for (int r = 0; r < kRows; ++r) load4(ru, row_elem(r), u[r]);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                u[r][k] = s.momentum * u[r][k] + g[r][k];
                g[r][k] = direction(s, u[r][k], g[r][k]);
            }
            store4(ru, row_elem(r), u[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const double d = row_elem(r) + k < cnt ? static_cast<double>(g[r][k]) : 0.0;
            sum += d * d;
        }
    sum = block_tree_sum(sum);
    if (threadIdx.x == 0) sums[M.chunk0 + it.i] = sum;
}

// 1 / (||D|| + eps) from the sum of squares; 0 for D = 0, NaN where D is not finite.
__device__ __forceinline__ double norm_scale(double sum, float eps) {
    return sum == 0.0 ? 0.0 : sum - sum == 0.0 ? 1.0 / (sqrt(sum) + static_cast<double>(eps)) : __builtin_nan("");
}

// Per matrix.
__global__ __launch_bounds__(kBlock) void orth_scale_kernel(const MatDev *__restrict__ mats,
                                                            const double *__restrict__ sums, float eps,
                                                            double *__restrict__ inv) {
    const MatDev M = mats[blockIdx.x];
    double sum = 0.0;
    for (uint32_t c = threadIdx.x; c < M.nchunk; c += kBlock) sum += sums[M.chunk0 + c];
    sum = block_tree_sum(sum);
    if (threadIdx.x == 0) inv[blockIdx.x] = norm_scale(sum, eps);
}

// ---------------------------------------------------------------- products
// One product of the chain: P Q^T for every tile of an item list.
//   kSym    P, Q symmetric or equal: the result is symmetric, tiles on and
//           below the diagonal are computed and mirrored
//   kNext   the next X and T = X^T
//   kOut    the result itself, in fp32, or applied to the weights
enum Kind { kSym, kNext, kOut };

struct GemmArgs {
    const Item *items;
    const uint32_t *first;
    const MatDev *mats;
    const _Float16 *P, *Q;  // operands; P null: of X's shape, else m x m
    uint32_t px, qx;        // whether an operand is an X (or T) array
    // Start behind the tile's own rows (1) or columns (2) of the common index and end with them: where P
    // or Q has a I on its diagonal, the sums, and their roundings with them, stay small until its terms
    // come (error at 2048 x 2048: 1.5e-6, in plain order 2.7e-6, of fp32 products 3.0e-6).
    uint32_t turn;
    const _Float16 *D;      // kSym: symmetric addend, or null
    float acc, add, diag;   // result = acc * (P Q^T) + add * D + diag * I
    _Float16 *S;            // kSym: result
    _Float16 *Xn, *Tn;      // kNext: results
    float *O, *W;           // kOut: the result, or the weights it is applied to
    float decay, lr;        // W <- decay W - lr s O
    int shape;              // GC_MUON_SCALE_*
    float *partial;         // tiles of split items, fp32
};

// s of a matrix for GC_MUON_SCALE_*.
__device__ __forceinline__ double shape_scale(int shape, uint32_t R, uint32_t C) {
    if (shape == GC_MUON_SCALE_SHAPE) return R > C ? sqrt(static_cast<double>(R) / static_cast<double>(C)) : 1.0;
    if (shape == GC_MUON_SCALE_RMS) return 0.2 * sqrt(static_cast<double>(R > C ? R : C));
    return 1.0;
}

template <class T>
struct Shape : T {
    static constexpr int kWaves = T::kWR * T::kWC, kThreads = kWaves * int(kWave);
    static constexpr int kWaveRows = T::kTile / T::kWR, kWaveCols = T::kTile / T::kWC;
    static constexpr int kRA = kWaveRows / 16, kRB = kWaveCols / 16;  // matrix-core tiles of a wave
    static constexpr int kStageBytes = 2 * T::kTile * 128;            // rows of P, then of Q
    static constexpr int kLoads = kStageBytes / kThreads / 16;        // 1 KB loads per wave and stage
    static constexpr int kLds = 2 * kStageBytes;
    static_assert(kWaves * 64 * 64 * 4 <= kLds, "a block of results per wave");
    static_assert(kWaveCols == 64 && kWaveRows % 64 == 0, "the epilogue's blocks");
};

// Whether the wave at (pr, qr) of a tile lies above the diagonal of a symmetric
// result's diagonal tile; the waves below it write its mirror image.
template <class C>
__device__ __forceinline__ bool above(uint32_t pr, uint32_t qr) {
    return qr >= pr + C::kWaveRows;
}
// Whether the block at (r, c) of tile `it` has to write its mirror image.
template <class C>
__device__ __forceinline__ bool mirrors(const Item &it, uint32_t r, uint32_t c) {
    return it.i != it.j || above<C>(c / C::kWaveRows * C::kWaveRows, r);
}

typedef __attribute__((address_space(1))) const char GlobalChar;
typedef __attribute__((address_space(3))) char LdsChar;

// The kLoads loads of a stage: rows [8 q, 8 q + 8) of P and Q straight into
// LDS.  Lane l fills 16 bytes of row l / 8; inside a row part c stands at
// c ^ ((row >> 1) & 7), so that the 16 rows a matrix-core operand reads at once
// lie in different banks (counted: no conflicts).
template <class C>
__device__ __forceinline__ void load_stage(const char *from, uint64_t row8, int32_t odd, char *__restrict__ to) {
#pragma unroll
    for (int q = 0; q < C::kLoads; ++q)
        __builtin_amdgcn_global_load_lds((GlobalChar *)(from + q * row8 + (q & 1 ? odd : 0)), (LdsChar *)(to + q * 1024), 16, 0, 0);
}

template <class C>
__device__ __forceinline__ void multiply_stage(const char *__restrict__ lds, uint32_t pr, uint32_t qr,
                                               f32x4 (&acc)[C::kRA][C::kRB]) {
    // rows 16 a + (lane & 15): a row's parts are permuted alike in every group of 16
    const uint32_t row = lane_id() & 15, part = lane_id() >> 4;
    const uint32_t hi = row * 128 + ((part ^ ((row >> 1) & 7)) << 4), lo = hi ^ 64;
    const char *p = lds + pr * 128, *q = lds + (C::kTile + qr) * 128;
    auto at = [](const char *x) { return *reinterpret_cast<const h8 *>(x); };
    h8 qh[C::kRB], ql[C::kRB];
#pragma unroll
    for (int b = 0; b < C::kRB; ++b) {
        ql[b] = at(q + b * 2048 + lo);
        qh[b] = at(q + b * 2048 + hi);
    }
    // one row of tiles ahead, and no further: hoisted, the loads do not fit the registers
    h8 ph = at(p + hi), pl = at(p + lo);
#pragma unroll
    for (int a = 0; a < C::kRA; ++a) {
        h8 nh = ph, nl = pl;
        if (a + 1 < C::kRA) {
            nh = at(p + (a + 1) * 2048 + hi);
            nl = at(p + (a + 1) * 2048 + lo);
        }
#pragma unroll
        for (int b = 0; b < C::kRB; ++b) acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, ql[b], acc[a][b], 0, 0, 0);
#pragma unroll
        for (int b = 0; b < C::kRB; ++b) acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(pl, qh[b], acc[a][b], 0, 0, 0);
#pragma unroll
        for (int b = 0; b < C::kRB; ++b) acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, qh[b], acc[a][b], 0, 0, 0);
        ph = nh;
        pl = nl;
        __builtin_amdgcn_sched_barrier(0);
    }
}

// One stage: the loads of a later one go out, then this one is multiplied.
// The two are different stages of LDS, which the restrict parameters tell the
// compiler: without them it waits for the loads before it reads.
template <class C, bool kActive>
__device__ __forceinline__ void do_stage(const char *__restrict__ cur, char *__restrict__ next, const char *from,
                                         uint64_t row8, int32_t odd, bool load, uint32_t pr, uint32_t qr,
                                         f32x4 (&acc)[C::kRA][C::kRB]) {
    if (load) load_stage<C>(from, row8, odd, next);
    if (kActive) multiply_stage<C>(cur, pr, qr, acc);
}

// The stages of an item: r = 0 .. n - 1 are columns 32 k on, k = first + r
// around the common index of `all` stages.
struct Stages {
    uint32_t n, first, all;
    __device__ __forceinline__ uint64_t at(uint32_t r) const {
        const uint32_t k = first + r;
        return static_cast<uint64_t>(k < all ? k : k - all) * 128;
    }
};

// All stages of an item.  A wave whose rows or columns lie outside the matrix loads its
// share and multiplies nothing (a loop of its own: with the branch inside, the
// sums were copied at every stage).
template <class C, bool kActive>
__device__ __forceinline__ void run_stages(char *lds, char *to, const char *from, uint64_t row8, int32_t odd, bool load,
                                           const Stages &st, uint32_t pr, uint32_t qr, f32x4 (&acc)[C::kRA][C::kRB]) {
    const uint32_t nk = st.n;
    if (load) load_stage<C>(from + st.at(0), row8, odd, to);
    for (uint32_t k = 0; k < nk; ++k) {
        // stage k has landed, and every wave is done with the stage that is loaded next
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const uint32_t cur = (k & 1) * C::kStageBytes, next = C::kStageBytes - cur;
        do_stage<C, kActive>(lds + cur, to + next, from + st.at(k + 1), row8, odd, load && k + 1 < nk, pr, qr, acc);
    }
}

// acc += P Q^T over an item's stages: rows_p rows of P and rows_q of Q (multiples
// of 64) exist, this wave has rows pr and columns qr on.
template <class C>
__device__ __forceinline__ void all_stages(char *lds, const _Float16 *P, uint32_t ldp, uint32_t rows_p, const _Float16 *Q,
                                           uint32_t ldq, uint32_t rows_q, const Stages &st, bool active, uint32_t pr,
                                           uint32_t qr, f32x4 (&acc)[C::kRA][C::kRB]) {
    // this wave's loads: kLoads groups of 8 rows, all of P or all of Q
    const uint32_t lane = lane_id(), row = __builtin_amdgcn_readfirstlane(wave_id()) * C::kLoads * 8;  // of the stage
    const bool of_p = row < uint32_t(C::kTile);
    const uint32_t r = of_p ? row : row - C::kTile, ld = of_p ? ldp : ldq;
    const bool load = r < (of_p ? rows_p : rows_q);
    // part of this lane's LDS place in its row, for even groups; odd ones differ by the bit of 4 parts
    const uint32_t part = (lane & 7) ^ (lane >> 4);
    const char *from = reinterpret_cast<const char *>((of_p ? P : Q) + static_cast<uint64_t>(r + (lane >> 3)) * ld * 2) + part * 16;
    const int32_t odd = part & 4 ? -64 : 64;
    const uint64_t row8 = static_cast<uint64_t>(ld) * 32;
    char *to = lds + row * 128;
    if (active) run_stages<C, true>(lds, to, from, row8, odd, load, st, pr, qr, acc);
    else run_stages<C, false>(lds, to, from, row8, odd, load, st, pr, qr, acc);
}

// x[0..n) to O, or applied to W, at flat element `at`.
__device__ __forceinline__ void put_out(const GemmArgs &g, uint64_t at, uint32_t n, float step, const float (&x)[4]) {
    if (n == 4) {
        F32x4 v;
        if (g.W) v = *reinterpret_cast<const F32x4 *>(g.W + at);
#pragma unroll
        for (int u = 0; u < 4; ++u) v.v[u] = g.W ? g.decay * v.v[u] - step * x[u] : x[u];
        *reinterpret_cast<F32x4 *>((g.W ? g.W : g.O) + at) = v;
        return;
    }
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u)
        if (u < n) {
            if (g.W) g.W[at + u] = g.decay * g.W[at + u] - step * x[u];
            else g.O[at + u] = x[u];
        }
}

// A word of split value x.
__device__ __forceinline__ uint32_t split_word(float x) {
    _Float16 h, l;
    split(x, h, l);
    return __builtin_bit_cast(uint16_t, h) | (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, l)) << 16);
}

// A block of 64 x 64 results in LDS, [column][row], a word each: fp32 (kOut),
// or hi and lo in its halves.  The 16 parts of 4 rows of a column are permuted
// so that a matrix-core tile's lanes (a column's 4 rows), lanes along a column
// and lanes along a row all meet different banks.
constexpr uint32_t kBlockWords = 64 * 64;
__device__ __forceinline__ uint32_t block_at(uint32_t col, uint32_t part) {
    return col * 64 + ((part ^ (col >> 2) ^ ((col & 3) << 2)) << 2);
}

// A lane's four sums of the block's matrix-core tile (a, b): rows 16 a + 4 q,
// q = lane / 16, of column 16 b + lane % 16.
__device__ __forceinline__ void put_tile(uint32_t *block, uint32_t a, uint32_t b, f32x4 v) {
    *reinterpret_cast<f32x4 *>(block + block_at(16 * b + (lane_id() & 15), 4 * a + (lane_id() >> 4))) = v;
}

// The sums of the block at (i0, j0) scaled, addend and diagonal added, and
// split.  (A short loop over LDS: done in registers for each matrix-core tile
// it was 12 KB of code, which small products waited for.)
template <Kind kKind, int kTeam>
__device__ __forceinline__ void split_block(const GemmArgs &g, const MatDev &M, uint32_t *block, uint32_t i0, uint32_t j0) {
    const uint32_t k = lane_id() & 15, r = lane_id() >> 4, i = i0 + 4 * k;
#pragma unroll 4
    for (uint32_t t = kTeam > 1 ? wave_id() : 0; t < 16; t += kTeam) {
        const uint32_t j = j0 + 4 * t + r;
        uint32_t *at = block + block_at(4 * t + r, k);
        const f32x4 v = *reinterpret_cast<const f32x4 *>(at);
        float x[4] = {v[0] * g.acc, v[1] * g.acc, v[2] * g.acc, v[3] * g.acc};
        if (kKind == kSym) {
            if (g.D) {
                const _Float16 *p = g.D + M.a + static_cast<uint64_t>(j) * M.mp * 2 + split_at(i);
                const h4 dh = *reinterpret_cast<const h4 *>(p), dl = *reinterpret_cast<const h4 *>(p + 32);
#pragma unroll
                for (int u = 0; u < 4; ++u) x[u] = x[u] + g.add * (static_cast<float>(dh[u]) + static_cast<float>(dl[u]));
            }
            const uint32_t on = j - i;  // the diagonal's place among the four, if < 4
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u)
                if (on == u && j < M.m) x[u] = x[u] + g.diag;
        }
        uint32_t y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            _Float16 h, l;
            split(x[u], h, l);
            y[u] = __builtin_bit_cast(uint16_t, h) | (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, l)) << 16);
        }
        *reinterpret_cast<uint4 *>(at) = make_uint4(y[0], y[1], y[2], y[3]);
    }
}

// Eight split values' hi and lo.
__device__ __forceinline__ void unsplit(const uint32_t (&v)[8], h8 &hi, h8 &lo) {
    uint4 h, l;
    h.x = __builtin_amdgcn_perm(v[1], v[0], 0x05040100u);
    h.y = __builtin_amdgcn_perm(v[3], v[2], 0x05040100u);
    h.z = __builtin_amdgcn_perm(v[5], v[4], 0x05040100u);
    h.w = __builtin_amdgcn_perm(v[7], v[6], 0x05040100u);
    l.x = __builtin_amdgcn_perm(v[1], v[0], 0x07060302u);
    l.y = __builtin_amdgcn_perm(v[3], v[2], 0x07060302u);
    l.z = __builtin_amdgcn_perm(v[5], v[4], 0x07060302u);
    l.w = __builtin_amdgcn_perm(v[7], v[6], 0x07060302u);
    hi = __builtin_bit_cast(h8, h);
    lo = __builtin_bit_cast(h8, l);
}

// Consecutive in a split row, to p (hi) and p + 32 (lo).
__device__ __forceinline__ void put_split(_Float16 *p, const uint32_t (&v)[8]) {
    h8 hi, lo;
    unsplit(v, hi, lo);
    *reinterpret_cast<h8 *>(p) = hi;
    *reinterpret_cast<h8 *>(p + 32) = lo;
}

// A block of split values along its columns: row j of the split matrix at `to`
// with `cols` columns i, from (j0, i0) on.  8 lanes by 8 values of a split row.
template <int kTeam>
__device__ __forceinline__ void write_columns(_Float16 *to, uint32_t ld, const uint32_t *block, uint32_t i0, uint32_t j0,
                                              uint32_t cols = 64) {
    const uint32_t k = lane_id() & 7, r = lane_id() >> 3;
    if (8 * k >= cols) return;
    to += static_cast<uint64_t>(j0 + r) * ld * 2 + split_at(i0 + 8 * k);
#pragma unroll 2
    for (uint32_t t = kTeam > 1 ? wave_id() : 0; t < 8; t += kTeam) {
        const uint32_t jj = 8 * t + r;
        const uint4 a = *reinterpret_cast<const uint4 *>(block + block_at(jj, 2 * k));
        const uint4 b = *reinterpret_cast<const uint4 *>(block + block_at(jj, 2 * k + 1));
        put_split(to + static_cast<uint64_t>(8 * t) * ld * 2, {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
    }
}

// The same along its rows: row i, columns j.
template <int kTeam>
__device__ __forceinline__ void write_rows(_Float16 *to, uint32_t ld, const uint32_t *block, uint32_t i0, uint32_t j0) {
    const uint32_t k = lane_id() & 7, r = lane_id() >> 3;
    to += static_cast<uint64_t>(i0 + r) * ld * 2 + split_at(j0 + 8 * k);
#pragma unroll 2
    for (uint32_t t = kTeam > 1 ? wave_id() : 0; t < 8; t += kTeam) {
        const uint32_t ii = 8 * t + r;
        uint32_t v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = block[block_at(8 * k + u, ii >> 2) + (ii & 3)];
        put_split(to + static_cast<uint64_t>(8 * t) * ld * 2, v);
    }
}

// A 64 x 64 tile of X_0, split, into X and T; the padding becomes zeros.
// Memory bounds it: 36 M elements with Nesterov's D formed again from U and G
// take 128 us, 4.5 TB/s (135 with 8-byte stores, and 58 against 44 for 16 M
// elements without momentum); D kept by orth_norm would be 4 more bytes
// written for 4 fewer read.
__global__ __launch_bounds__(kBlock) void orth_split_kernel(const Item *__restrict__ items, const MatDev *__restrict__ mats,
                                                            Source s, const double *__restrict__ inv, float pow2,
                                                            _Float16 *__restrict__ X, _Float16 *__restrict__ T) {
    const Item it = items[blockIdx.x];
    const MatDev M = mats[it.mat];
    __shared__ __attribute__((aligned(16))) uint32_t block[kBlockWords];
    const double scale = inv[it.mat] * static_cast<double>(pow2);
    const uint32_t i0 = it.i * kSplitTile, j0 = it.j * kSplitTile;
    // D is read along its rows: lanes run over j, or over i where X = D^T; a
    // thread has 16 of D's rows r0 + 4 (k % 4) + 16 (k / 4), 4 next to each other
    const uint32_t l = lane_id(), r0 = wave_id() * 4;
    const uint32_t rows = M.flip ? M.n - min(M.n, j0) : M.m - min(M.m, i0), cols = M.flip ? M.m - min(M.m, i0) : M.n - min(M.n, j0);
    const uint64_t at = M.off + (M.flip ? static_cast<uint64_t>(j0) * M.C + i0 : static_cast<uint64_t>(i0) * M.C + j0) + l;
    float d[16];
#pragma unroll
    for (uint32_t k = 0; k < 16; ++k) {
        const uint32_t r = 16 * (k / 4) + r0 + k % 4;
        d[k] = 0.0f;
        if (r < rows && l < cols) {
            const uint64_t e = at + static_cast<uint64_t>(r) * M.C;
            const float g = s.G[e];
            d[k] = s.U ? direction(s, s.U[e], g) : g;
        }
    }
#pragma unroll
    for (uint32_t k = 0; k < 16; k += 4) {
        const uint32_t r = 4 * k + r0;
        uint32_t v[4];
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u) v[u] = split_word(static_cast<float>(static_cast<double>(d[k + u]) * scale));
        if (M.flip) {
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u) block[block_at(r + u, l >> 2) + (l & 3)] = v[u];
        } else {
            *reinterpret_cast<uint4 *>(block + block_at(l, r >> 2)) = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
    __syncthreads();
    write_columns<kWaves>(T + M.x, M.mp, block, i0, j0);
    write_rows<kWaves>(X + M.x, M.np, block, i0, j0);
}

// Writes a block of sums out, by one wave or a team of kTeam: along its columns
// (T, or the symmetric result) and along its rows (X, or the mirror image).
template <Kind kKind, int kTeam>
__device__ __forceinline__ void write_block(const GemmArgs &g, const MatDev &M, uint32_t *block, uint32_t i0, uint32_t j0,
                                            bool mirror) {
    const uint32_t w = kTeam > 1 ? wave_id() : 0, lane = lane_id();
    if (kKind == kOut) {
        const double sc = g.W ? shape_scale(g.shape, M.R, M.C) : 1.0;
        const float step = static_cast<float>(static_cast<double>(g.lr) * sc);
        const uint32_t k = lane & 15, r = lane >> 4;
        // 16 lanes by 4 elements of a row of the flat buffer
#pragma unroll 4
        for (uint32_t t = w; t < 16; t += kTeam) {
            float x[4];
            if (M.flip) {
                const uint32_t jj = 4 * t + r, i = i0 + 4 * k, j = j0 + jj;
                const uint4 v = *reinterpret_cast<const uint4 *>(block + block_at(jj, k));
                x[0] = dev_u2f(v.x) * g.acc;
                x[1] = dev_u2f(v.y) * g.acc;
                x[2] = dev_u2f(v.z) * g.acc;
                x[3] = dev_u2f(v.w) * g.acc;
                put_out(g, M.off + static_cast<uint64_t>(j) * M.C + i, j < M.n && i < M.m ? min(M.m - i, 4u) : 0, step, x);
            } else {
                const uint32_t i = i0 + 4 * t + r, j = j0 + 4 * k;
#pragma unroll
                for (int u = 0; u < 4; ++u) x[u] = dev_u2f(block[block_at(4 * k + u, t) + r]) * g.acc;
                put_out(g, M.off + static_cast<uint64_t>(i) * M.C + j, i < M.m && j < M.n ? min(M.n - j, 4u) : 0, step, x);
            }
        }
        return;
    }
    split_block<kKind, kTeam>(g, M, block, i0, j0);
    if (kTeam > 1) __syncthreads();
    write_columns<kTeam>(kKind == kSym ? g.S + M.a : g.Tn + M.x, M.mp, block, i0, j0);
    if (kKind == kSym && !mirror) return;
    write_rows<kTeam>(kKind == kSym ? g.S + M.a : g.Xn + M.x, kKind == kSym ? M.mp : M.np, block, i0, j0);
}

__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A unit's items, one after the other: stages [it.k0, it.k1) of tile (it.i,
// it.j).  A whole tile is written out; a part of a split one leaves its sums in
// it.slot, in register order, and orth_join_kernel adds the parts.
// The matrix cores bound it, and the card's power them: 1.2 to 1.35 PFLOP/s of
// fp16 at 4096 x 4096, two thirds of the cycles with a matrix instruction in
// flight at 1.9 GHz of 2.4; a library's fp16 product of 8192 x 8192 runs at
// 1.25.  (A main loop with the operands of the next stage read ahead of its
// barrier left no gaps and ran no faster: 325 us against 310 for B X there.)
template <Kind kKind, class C>
__global__ __launch_bounds__(C::kThreads) void orth_gemm_kernel(GemmArgs g) {
    __shared__ __attribute__((aligned(128))) char lds[C::kLds];
    const uint32_t w = __builtin_amdgcn_readfirstlane(wave_id()), lane = lane_id();
    const uint32_t begin = g.first[blockIdx.x], end = g.first[blockIdx.x + 1];
    if (begin == end) return;
    Item next = g.items[begin];
    MatDev next_mat = g.mats[next.mat];
    for (uint32_t at = begin; at < end; ++at) {
        const Item it = next;
        const MatDev M = next_mat;
        lds_barrier();  // every wave is done with the LDS of the item before
        if (at + 1 < end) {  // read while this one is multiplied
            next = g.items[at + 1];
            next_mat = g.mats[next.mat];
        }
        const uint32_t i0 = it.i * C::kTile, j0 = it.j * C::kTile;
        // rows of this tile that exist (multiples of 128)
        const uint32_t rows_p = min(uint32_t(C::kTile), M.mp - i0), rows_q = min(uint32_t(C::kTile), (kKind == kSym ? M.mp : M.np) - j0);
        // the waves of a SIMD differ in row half and column half, so that a tile
        // with half its rows or columns costs half
        const uint32_t wr = w / C::kWC, wc = (w + wr * (C::kWC / 2)) % C::kWC;
        const uint32_t pr = wr * C::kWaveRows, qr = wc * C::kWaveCols;
        const bool active = pr < rows_p && qr < rows_q && !(kKind == kSym && it.i == it.j && above<C>(pr, qr));
        f32x4 acc[C::kRA][C::kRB];
#pragma unroll
        for (int a = 0; a < C::kRA; ++a)
#pragma unroll
            for (int b = 0; b < C::kRB; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        {
            const uint32_t ldp = g.px ? M.np : M.mp, ldq = g.qx && kKind == kSym ? M.np : M.mp;
            const uint32_t all = ((g.px && kKind == kSym ? M.n : M.m) + 31) / 32;
            const Stages st{it.k1 - it.k0, (it.k0 + (g.turn ? ((g.turn == 1 ? i0 : j0) + C::kTile) / 32 : 0)) % all, all};
            all_stages<C>(lds, g.P + (g.px ? M.x : M.a) + static_cast<uint64_t>(i0) * ldp * 2, ldp, rows_p,
                          g.Q + (g.qx ? M.x : M.a) + static_cast<uint64_t>(j0) * ldq * 2, ldq, rows_q, st, active, pr, qr, acc);
        }
        if (it.slot != kNoSlot) {
            if (!active) continue;
            f32x4 *p = reinterpret_cast<f32x4 *>(g.partial + static_cast<uint64_t>(it.slot) * C::kTile * C::kTile) + w * (C::kRA * C::kRB * kWave) + lane;
#pragma unroll
            for (int a = 0; a < C::kRA; ++a)
#pragma unroll
                for (int b = 0; b < C::kRB; ++b) p[(a * C::kRB + b) * kWave] = acc[a][b];
            continue;
        }
        lds_barrier();
        if (!active) continue;
        uint32_t *block = reinterpret_cast<uint32_t *>(lds) + w * kBlockWords;
#pragma unroll
        for (int h = 0; h < C::kRA / 4; ++h) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < C::kRB; ++b)
                    put_tile(block, a, b, acc[4 * h + a][b]);
            write_block<kKind, 1>(g, M, block, i0 + pr + 64 * h, j0 + qr, mirrors<C>(it, pr + 64 * h, qr));
        }
    }
}

// The parts of a split tile, added in order: a 64 x 64 block per workgroup of
// 4 waves.  29 to 35 us at 4096 x 4096, where the 136 tiles of a symmetric product
// would leave 120 of 256 units idle without the cut.
template <Kind kKind, class C>
__global__ __launch_bounds__(kBlock) void orth_join_kernel(GemmArgs g) {
    __shared__ __attribute__((aligned(16))) uint32_t block[kBlockWords];
    constexpr uint32_t kBlocks = C::kWaves * (C::kRA / 4);
    const Item it = g.items[blockIdx.x / kBlocks];
    const MatDev M = g.mats[it.mat];
    const uint32_t part = blockIdx.x % kBlocks, w = part / (C::kRA / 4), h = part % (C::kRA / 4);
    const uint32_t wr = w / C::kWC, wc = (w + wr * (C::kWC / 2)) % C::kWC;
    const uint32_t pr = wr * C::kWaveRows, qr = wc * C::kWaveCols;
    const uint32_t i0 = it.i * C::kTile + pr + 64 * h, j0 = it.j * C::kTile + qr;
    if (i0 >= M.mp || j0 >= (kKind == kSym ? M.mp : M.np)) return;
    if (kKind == kSym && it.i == it.j && above<C>(pr, qr)) return;
    // tiles 4 a + b of the block: a is this wave's
    const uint32_t a = wave_id();
    const f32x4 *p = reinterpret_cast<const f32x4 *>(g.partial + static_cast<uint64_t>(it.slot) * C::kTile * C::kTile) +
                     w * (C::kRA * C::kRB * kWave) + (4 * h + a) * C::kRB * kWave + lane_id();
    constexpr uint64_t kStep = static_cast<uint64_t>(C::kTile) * C::kTile / 4;
    f32x4 v[C::kRB];
#pragma unroll
    for (int b = 0; b < C::kRB; ++b) v[b] = p[b * kWave];
#pragma unroll 2
    for (uint32_t s = 1; s < it.k1; ++s)
#pragma unroll
        for (int b = 0; b < C::kRB; ++b) v[b] = v[b] + p[s * kStep + b * kWave];
#pragma unroll
    for (int b = 0; b < C::kRB; ++b) put_tile(block, a, b, v[b]);
    __syncthreads();
    write_block<kKind, kWaves>(g, M, block, i0, j0, mirrors<C>(it, pr + 64 * h, qr));
}

// ----------------------------------------------------- matrices of few rows
// Where every matrix has at most kNarrow rows, one tile of A and B, a
// workgroup that has X' for 128 columns has all it needs for their share of
// the next A as well.  Two launches a step then:
//   slab   X' = B X for its slabs of 128 columns, T' written (X itself is not
//          needed), and the sum of X' X'^T over them, left as a part
//   small  per matrix: the parts added in order, A, and B = a I + b A + c A^2
// after a first slab launch that makes X_0 from D.  Latency bounds both, of
// operands loaded, multiplied and written out once, and of the instructions
// fetched for it: what a matrix has no rows for is skipped tile by tile (95 us
// at 29 x 1600 and 5 steps, then 84).  Where every matrix has at most 64 rows
// and the slabs are at most kFusedSlabs, each slab's workgroup makes its B
// itself and a step is one launch: 72 us for 29 x 1600 against 84, 83 against 88
// for 16 of them (208 slabs), 203 against 205 for 8 of 64 x 4096 (256 slabs); 141
// against 108 for 507 slabs, and 326 against 315 for 8 of 128 x 4096.
constexpr uint32_t kNarrow = 128;
enum Slab { kFirst, kMiddle, kLast };

// 128 x 128 split values as four blocks, block wave 2 (i / 64) + (j / 64 ^ i / 64).
__device__ __forceinline__ const uint32_t *block_of(const uint32_t *words, uint32_t ib, uint32_t jb) {
    return words + (2 * ib + (jb ^ ib)) * kBlockWords;
}

__device__ __forceinline__ float joined(uint32_t word) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(word))) +
           static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(word >> 16)));
}

// put_tile of the split values.
__device__ __forceinline__ void put_split_tile(uint32_t *block, uint32_t a, uint32_t b, f32x4 v) {
    *reinterpret_cast<uint4 *>(block + block_at(16 * b + (lane_id() & 15), 4 * a + (lane_id() >> 4))) =
        make_uint4(split_word(v[0]), split_word(v[1]), split_word(v[2]), split_word(v[3]));
}

// Rows j .. j + 7 of a block's column.
__device__ __forceinline__ void column_of(const uint32_t *block, uint32_t col, uint32_t j, h8 &hi, h8 &lo) {
    const uint4 x = *reinterpret_cast<const uint4 *>(block + block_at(col, j >> 2));
    const uint4 y = *reinterpret_cast<const uint4 *>(block + block_at(col, (j >> 2) + 1));
    unsplit({x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}, hi, lo);
}

// g += Y Y^T for the wave's 64 x 64, Y's first 32 n columns in `words`. Y has m
// rows: 16-row tiles behind them are neither read nor multiplied, their operands
// stay zero and so do their sums.
template <bool kSymmetric>
__device__ __forceinline__ void add_square(const uint32_t *words, uint32_t wr, uint32_t wc, uint32_t n, uint32_t m,
                                           f32x4 (&g)[4][4]) {
    const uint32_t ra = m - 64 * wr, rb = m - 64 * wc;
    for (uint32_t s = 0; s < n; ++s) {
        auto operand = [&](uint32_t ib, uint32_t t, h8 &hi, h8 &lo) {  // rows 16 t + lane % 16 of row block ib
            const uint32_t r = 16 * t + (lane_id() & 15), j = 32 * (s & 1) + 8 * (lane_id() >> 4);
            if (kSymmetric) {  // column r's rows, which stand together
                column_of(block_of(words, s >> 1, ib), r, j, hi, lo);
                return;
            }
            const uint32_t *b = block_of(words, ib, s >> 1);
            uint32_t v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = b[block_at(j + u, r >> 2) + (r & 3)];
            unsplit(v, hi, lo);
        };
        h8 qh[4] = {}, ql[4] = {};
#pragma unroll
        for (int b = 0; b < 4; ++b)
            if (16u * b < rb) operand(wc, b, qh[b], ql[b]);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            if (16u * a >= ra) break;
            h8 ph, pl;
            operand(wr, a, ph, pl);
#pragma unroll
            for (int b = 0; b < 4; ++b) g[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, ql[b], g[a][b], 0, 0, 0);
#pragma unroll
            for (int b = 0; b < 4; ++b) g[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(pl, qh[b], g[a][b], 0, 0, 0);
#pragma unroll
            for (int b = 0; b < 4; ++b) g[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, qh[b], g[a][b], 0, 0, 0);
        }
    }
}

struct FirstArgs {
    Source s;
    const double *sums;
    float eps, pow2;
};

// X_0's columns j0 .. j0 + 127 into `words`, zeros outside the matrix.
__device__ __forceinline__ void first_slab(const MatDev &M, const FirstArgs &f, double scale, uint32_t j0, uint32_t *words) {
    for (uint32_t e = threadIdx.x; e < kBlockWords; e += kBlock)
        reinterpret_cast<uint4 *>(words)[e] = make_uint4(0, 0, 0, 0);
    lds_barrier();
    const uint32_t cols = min(M.n - j0, kNarrow);
    auto value = [&](uint64_t at) {
        const float g = f.s.G[at];
        const float d = f.s.U ? direction(f.s, f.s.U[at], g) : g;
        return split_word(static_cast<float>(static_cast<double>(d) * scale));
    };
    auto place = [&](uint32_t i, uint32_t j) {
        return const_cast<uint32_t *>(block_of(words, i >> 6, j >> 6)) + block_at(j & 63, (i & 63) >> 2) + (i & 3);
    };
    if (M.flip) {  // D is n x m: the slab is contiguous
        const uint64_t at = M.off + static_cast<uint64_t>(j0) * M.m;
#pragma unroll 8
        for (uint32_t e = threadIdx.x; e < cols * M.m; e += kBlock) *place(e % M.m, e / M.m) = value(at + e);
    } else {
        const uint32_t j = threadIdx.x & (kNarrow - 1);
        if (j < cols)
#pragma unroll 8
            for (uint32_t i = threadIdx.x / kNarrow; i < M.m; i += kBlock / kNarrow)
                *place(i, j) = value(M.off + static_cast<uint64_t>(i) * M.n + j0 + j);
    }
    lds_barrier();
}

// B^T = diag I + add A + square A^2 of one matrix, split, as kBlocks blocks in
// `words`, where A = acc * (the `parts` parts from `slot` on, in order).  All
// waves of the workgroup; ends with every block written but not yet visible to
// all.
struct SmallArgs {
    const float *partial;
    float acc, add, square, diag;
};

// Every wave adds its 16 rows of each of the kBlocks blocks, those that exist;
// one block's (kBlocks == 1) only as far as there are m rows.
template <int kBlocks>
__device__ __forceinline__ void sum_parts(const SmallArgs &g, uint32_t slot, uint32_t parts, uint32_t m, uint32_t *words) {
    constexpr uint32_t kStep = kNarrow * kNarrow / 4;
    const uint32_t w = __builtin_amdgcn_readfirstlane(wave_id());
    const f32x4 *p = reinterpret_cast<const f32x4 *>(g.partial + static_cast<uint64_t>(slot) * kNarrow * kNarrow) +
                     w * (4 * kWave) + lane_id();
    f32x4 v[kBlocks][4];
    const auto add = [&](int b0, int b1) {
#pragma unroll
        for (int q = 0; q < kBlocks; ++q)
#pragma unroll
            for (int b = b0; b < b1; ++b) v[q][b] = p[q * (16 * kWave) + b * kWave];
#pragma unroll(kBlocks == 1 ? 4 : 2)
        for (uint32_t s = 1; s < parts; ++s)
#pragma unroll
            for (int q = 0; q < kBlocks; ++q)
#pragma unroll
                for (int b = b0; b < b1; ++b) v[q][b] = v[q][b] + p[s * kStep + q * (16 * kWave) + b * kWave];
    };
#pragma unroll
    for (int q = 0; q < kBlocks; ++q)
#pragma unroll
        for (int b = 0; b < 4; ++b) v[q][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (kBlocks > 1) {
        add(0, 4);
    } else if (16 * w < m) {
        if (m > 32) add(0, 4);
        else add(0, 2);
    }
#pragma unroll
    for (int q = 0; q < kBlocks; ++q)
#pragma unroll
        for (int b = 0; b < 4; ++b) put_split_tile(words + q * kBlockWords, w, b, v[q][b] * g.acc);
}

template <int kBlocks>
__device__ __forceinline__ void small_poly(const SmallArgs &g, const MatDev &M, uint32_t slot, uint32_t parts, uint32_t *words) {
    const uint32_t w = __builtin_amdgcn_readfirstlane(wave_id());
    const uint32_t wr = w / 2, wc = (w ^ wr) & 1;
    const bool active = 64 * wr < M.m && 64 * wc < M.m;
    sum_parts<kBlocks>(g, slot, parts, M.m, words);
    lds_barrier();
    f32x4 A2[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) A2[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (active) add_square<true>(words, wr, wc, (M.m + 31) / 32, M.m, A2);
    lds_barrier();  // every wave has read A
    if (!active) return;
    uint32_t *block = words + w * kBlockWords;
    const uint32_t c = lane_id() & 15, r = 4 * (lane_id() >> 4);
    const bool diagonal = wr == wc;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            if (64 * wr + 16 * a >= M.m || 64 * wc + 16 * b >= M.m) continue;  // zeros, as A's
            const uint4 v = *reinterpret_cast<const uint4 *>(block + block_at(16 * b + c, 4 * a + (lane_id() >> 4)));
            f32x4 x{joined(v.x), joined(v.y), joined(v.z), joined(v.w)};
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u) {
                x[u] = A2[a][b][u] * g.square + g.add * x[u];
                if (a == b && diagonal && r + u == c && 64 * wr + 16 * a + c < M.m) x[u] = x[u] + g.diag;
            }
            put_split_tile(block, a, b, x);
        }
}

// All columns of the slab's 128 rows of T into LDS, stage by stage as load_stage
// has them.
__device__ __forceinline__ void load_slab(const _Float16 *T, uint32_t stages, char *__restrict__ lds) {
    const uint32_t lane = lane_id(), row = __builtin_amdgcn_readfirstlane(wave_id()) * 32;
    const uint32_t part = (lane & 7) ^ (lane >> 4);
    const int32_t odd = part & 4 ? -64 : 64;
    const char *from = reinterpret_cast<const char *>(T + static_cast<uint64_t>(row + (lane >> 3)) * (2 * kNarrow)) + part * 16;
    for (uint32_t s = 0; s < stages; ++s)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            __builtin_amdgcn_global_load_lds((GlobalChar *)(from + s * 128 + q * (32 * kNarrow) + (q & 1 ? odd : 0)),
                                             (LdsChar *)(lds + s * (128 * kNarrow) + row * 128 + q * 1024), 16, 0, 0);
}

// acc += B X for the wave's 64 x 64, of m rows: B^T's blocks in `words`, the
// slab of T as load_slab left it.
__device__ __forceinline__ void slab_product(const uint32_t *__restrict__ words, const char *__restrict__ lds, uint32_t m,
                                             uint32_t pr, uint32_t qr, f32x4 (&acc)[4][4]) {
    const uint32_t stages = (m + 31) / 32;
    const uint32_t row = lane_id() & 15, part = lane_id() >> 4;
    const uint32_t hi = row * 128 + ((part ^ ((row >> 1) & 7)) << 4), lo = hi ^ 64;
    for (uint32_t s = 0; s < stages; ++s) {
        const char *q = lds + s * (128 * kNarrow) + qr * 128;
        const uint32_t *block = block_of(words, s >> 1, pr >> 6);
        h8 qh[4], ql[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            qh[b] = *reinterpret_cast<const h8 *>(q + b * 2048 + hi);
            ql[b] = *reinterpret_cast<const h8 *>(q + b * 2048 + lo);
        }
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            if (pr + 16 * a >= m) break;
            h8 ph, pl;
            column_of(block, 16 * a + row, 32 * (s & 1) + 8 * part, ph, pl);
#pragma unroll
            for (int b = 0; b < 4; ++b) acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, ql[b], acc[a][b], 0, 0, 0);
#pragma unroll
            for (int b = 0; b < 4; ++b) acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(pl, qh[b], acc[a][b], 0, 0, 0);
#pragma unroll
            for (int b = 0; b < 4; ++b) acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, qh[b], acc[a][b], 0, 0, 0);
        }
    }
}

// Slabs [it.k0, it.k1) of a matrix.  kFused: B comes from the it.j parts from
// it.i on instead of g.P.
template <Slab kSlabKind, bool kFused>
__global__ __launch_bounds__(kBlock, kFused ? 1 : 2) void orth_slab_kernel(GemmArgs g, FirstArgs f, SmallArgs small) {
    using C = Shape<Small>;
    __shared__ __attribute__((aligned(128))) char lds[C::kLds + (kFused ? 4 * kBlockWords : 0)];
    uint32_t *words = reinterpret_cast<uint32_t *>(lds);
    const Item it = g.items[blockIdx.x];
    const MatDev M = g.mats[it.mat];
    const uint32_t w = __builtin_amdgcn_readfirstlane(wave_id());
    const uint32_t wr = w / 2, wc = (w ^ wr) & 1, pr = 64 * wr, qr = 64 * wc;
    uint32_t *block = words + w * kBlockWords;
    const bool active = pr < M.m, squares = active && qr < M.m;
    double scale = 0.0;
    if (kSlabKind == kFirst) {
        double sum = 0.0;
        for (uint32_t c = threadIdx.x; c < M.nchunk; c += kBlock) sum += f.sums[M.chunk0 + c];
        scale = norm_scale(block_tree_sum(sum), f.eps) * static_cast<double>(f.pow2);
    }
    const uint32_t read = (M.m + 31) & ~31u;  // columns of T that a product reads
    uint32_t *bwords = words + 4 * kBlockWords;
    if (kFused) {
        load_slab(g.Q + M.x + static_cast<uint64_t>(it.k0) * kNarrow * M.mp * 2, (M.m + 31) / 32, lds);
        small_poly<1>(small, M, it.i, it.j, bwords);
    }
    f32x4 sums[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) sums[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t s = it.k0; s < it.k1; ++s) {
        const uint32_t j0 = s * kNarrow;
        lds_barrier();  // the slab before is done with LDS
        if (kSlabKind == kFirst) {
            first_slab(M, f, scale, j0, words);
        } else {
            f32x4 acc[4][4];
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            const uint32_t all = (M.m + 31) / 32;
            const _Float16 *T = g.Q + M.x + static_cast<uint64_t>(j0) * M.mp * 2;
            if (kFused) {
                if (s > it.k0) load_slab(T, all, lds);
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the slab has landed
                lds_barrier();
                if (active) slab_product(bwords, lds, M.m, pr, qr, acc);
            } else all_stages<C>(lds, g.P + M.a, M.mp, kNarrow, T, M.mp, kNarrow, Stages{all, 0, all}, active, pr, qr, acc);
            lds_barrier();
            if (active) {
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    if (pr + 16 * a >= read) break;
#pragma unroll
                    for (int b = 0; b < 4; ++b) put_tile(block, a, b, acc[a][b]);
                }
                if (kSlabKind == kLast) write_block<kOut, 1>(g, M, block, pr, j0 + qr, false);
                else split_block<kNext, 1>(g, M, block, pr, j0 + qr);
            }
            if (kSlabKind == kLast) continue;
            lds_barrier();
        }
        if (active) write_columns<1>(g.Tn + M.x, M.mp, block, pr, j0 + qr, read - pr);
        if (squares) add_square<false>(words, wr, wc, 4, M.m, sums);
    }
    if (kSlabKind == kLast || !squares) return;
    f32x4 *p = reinterpret_cast<f32x4 *>(g.partial + static_cast<uint64_t>(it.slot) * kNarrow * kNarrow) + w * (16 * kWave) + lane_id();
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) p[(a * 4 + b) * kWave] = sums[a][b];
}

// Per matrix: B into g.S.
__global__ __launch_bounds__(kBlock) void orth_small_kernel(GemmArgs g, SmallArgs a) {
    __shared__ __attribute__((aligned(128))) uint32_t words[4 * kBlockWords];
    const Item it = g.items[blockIdx.x];
    const MatDev M = g.mats[it.mat];
    const uint32_t w = __builtin_amdgcn_readfirstlane(wave_id());
    const uint32_t wr = w / 2, wc = (w ^ wr) & 1;
    if (M.m <= 64) small_poly<1>(a, M, it.slot, it.k1, words);
    else small_poly<4>(a, M, it.slot, it.k1, words);
    if (64 * wr < M.m && 64 * wc < M.m) write_columns<1>(g.S + M.a, M.mp, words + w * kBlockWords, 64 * wr, 64 * wc);
}

// --------------------------------------------------------------- host side
void *align256(void *p) {
    return reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(p) + 255) & ~uintptr_t(255));
}

gc_status check_orth(const char *fn, const gc_matrix_plan *p, const gc_orth_options *o, const void *ws, size_t ws_bytes,
                     Scales *s) {
    auto fail = [&](gc_status st, const char *what) { return set_error(st, std::string(fn) + ": " + what); };
    if (!p) return fail(GC_EINVAL, "matrix plan is null");
    if (!o) return fail(GC_EINVAL, "opt is null");
    if (o->steps < 1 || o->steps > GC_MAX_ORTH_STEPS) return fail(GC_EINVAL, "steps must be in [1, GC_MAX_ORTH_STEPS]");
    if (!(o->eps >= 0.0f) || !(o->eps - o->eps == 0.0f)) return fail(GC_EINVAL, "eps must be finite and >= 0");
    if (o->reserved[0] || o->reserved[1]) return fail(GC_EINVAL, "reserved fields must be 0");
    if (!orth_scales(*o, s))
        return fail(GC_EINVAL, "coef must be finite and keep the singular values of X at most 8");
    if (!ws) return fail(GC_EINVAL, "ws must be non-null");
    if (ws_bytes < orth_ws(nullptr, p).bytes)
        return fail(GC_ECAPACITY, "workspace smaller than gc_matrix_plan_workspace_bytes");
    return GC_OK;
}

template <Kind kKind, class C>
void product_of(const char *name, const gc_matrix_plan *p, const OrthDev &d, List l, GemmArgs g, hipStream_t stream) {
    g.items = d.list[l];
    g.first = d.first[l];
    GC_LAUNCH(name, stream,
              orth_gemm_kernel<kKind, C><<<static_cast<unsigned>(p->first[l].size() - 1), C::kThreads, 0, stream>>>(g));
    const List joins = static_cast<List>(l + 1);
    if (p->list[joins].empty()) return;
    g.items = d.list[joins];
    const unsigned blocks = static_cast<unsigned>(p->list[joins].size()) * C::kWaves * (C::kRA / 4);
    GC_LAUNCH("orth_join", stream, orth_join_kernel<kKind, C><<<blocks, kBlock, 0, stream>>>(g));
}

template <Kind kKind>
void product(const char *name, const gc_matrix_plan *p, const OrthDev &d, List l, const GemmArgs &g, hipStream_t stream) {
    if (p->large[l]) product_of<kKind, Shape<Large>>(name, p, d, l, g, stream);
    else product_of<kKind, Shape<Small>>(name, p, d, l, g, stream);
}

// The steps of a plan of matrices of few rows, behind the norm.
gc_status narrow_steps(const char *fn, const gc_matrix_plan *p, const OrthDev &d, const OrthWs &w, const gc_orth_options &o,
                       const Scales *sc, Source src, float *O, float *W, float decay, float lr, int shape,
                       hipStream_t stream) {
    auto pow2 = [](double c, int e) { return static_cast<float>(std::ldexp(c, e)); };
    const unsigned slabs = static_cast<unsigned>(p->list[kSlabs].size()), smalls = static_cast<unsigned>(p->list[kSmalls].size());
    GemmArgs g{};
    g.mats = d.mat;
    g.partial = w.partial;
    g.P = w.B;
    g.S = w.B;
    g.O = O;
    g.W = W;
    g.decay = decay;
    g.lr = lr;
    g.shape = shape;
    FirstArgs f{src, w.sums, o.eps, pow2(1.0, sc[0].ex)};
    // a fused step reads the parts of the step before while it writes its own
    float *const parts[2] = {w.partial, w.partial + (p->fused ? p->partial / 2 : 0)};
    int cur = 0;
    g.items = d.list[kSlabs];
    g.Tn = w.T[0];
    GC_LAUNCH("orth_slab", stream, orth_slab_kernel<kFirst, false><<<slabs, kBlock, 0, stream>>>(g, f, SmallArgs{}));
    for (int k = 0; k < o.steps; ++k) {
        const Scales &s = sc[k];
        const SmallArgs b{parts[cur], pow2(1.0, s.ea - 2 * s.ex), pow2(o.coef[k][1], s.eb - s.ea),
                          pow2(o.coef[k][2], s.eb - 2 * s.ea), pow2(o.coef[k][0], s.eb)};
        if (!p->fused) {
            g.items = d.list[kSmalls];
            GC_LAUNCH("orth_small", stream, orth_small_kernel<<<smalls, kBlock, 0, stream>>>(g, b));
        }
        const bool last = k + 1 == o.steps;
        g.items = d.list[kSlabs];
        g.acc = pow2(1.0, (last ? 0 : sc[k + 1].ex) - s.eb - s.ex);
        g.Q = w.T[cur];
        cur ^= 1;
        g.Tn = w.T[cur];
        g.partial = parts[cur];
        const auto kernel = p->fused ? (last ? orth_slab_kernel<kLast, true> : orth_slab_kernel<kMiddle, true>)
                                     : (last ? orth_slab_kernel<kLast, false> : orth_slab_kernel<kMiddle, false>);
        GC_LAUNCH("orth_slab", stream, kernel<<<slabs, kBlock, 0, stream>>>(g, f, b));
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_error(e, fn);
    return GC_OK;
}

gc_status orthogonalize(const char *fn, const gc_matrix_plan *p, const gc_orth_options &o, const Scales *sc, Source src,
                        float *O, float *W, float decay, float lr, int shape, void *ws, hipStream_t stream) {
    OrthDev d;
    gc_status st = orth_device(p, &d);
    if (st != GC_OK) return st;
    const OrthWs w = orth_ws(align256(ws), p);
    auto size = [&](List l) { return static_cast<unsigned>(p->list[l].size()); };
    auto pow2 = [](double c, int e) { return static_cast<float>(std::ldexp(c, e)); };
    GC_LAUNCH("orth_norm", stream,
              orth_norm_kernel<<<size(kChunks), kBlock, 0, stream>>>(d.list[kChunks], d.mat, src, w.sums));
    if (p->narrow) return narrow_steps(fn, p, d, w, o, sc, src, O, W, decay, lr, shape, stream);
    GC_LAUNCH("orth_scale", stream,
              orth_scale_kernel<<<static_cast<unsigned>(p->mat.size()), kBlock, 0, stream>>>(d.mat, w.sums, o.eps, w.inv));
    GC_LAUNCH("orth_split", stream,
              orth_split_kernel<<<size(kTiles), kBlock, 0, stream>>>(d.list[kTiles], d.mat, src, w.inv, pow2(1.0, sc[0].ex),
                                                                   w.X[0], w.T[0]));
    int cur = 0;
    // to <- acc P Q^T + add D + diag I, all m x m
    auto square = [&](const char *name, const _Float16 *P, const _Float16 *Q, _Float16 *to, float acc, const _Float16 *D,
                      float add, float diag, uint32_t turn) {
        GemmArgs g{};
        g.mats = d.mat;
        g.partial = w.partial;
        g.P = P;
        g.Q = Q;
        g.D = D;
        g.S = to;
        g.acc = acc;
        g.add = add;
        g.diag = diag;
        g.turn = turn;
        product<kSym>(name, p, d, kSquare, g, stream);
    };
    // B = a I + b A + c A^2 of step k, into `to`
    auto poly = [&](int k, const _Float16 *A, _Float16 *to) {
        const Scales &s = sc[k];
        square("orth_poly", A, A, to, pow2(o.coef[k][2], s.eb - 2 * s.ea), A, pow2(o.coef[k][1], s.eb - s.ea),
               pow2(o.coef[k][0], s.eb), 0);
    };
    for (int k = 0; k < o.steps;) {
        // an odd step goes first
        const bool pair = p->pairs && (o.steps - k) % 2 == 0 && sc[k].pair;
        const Scales &s = sc[k];
        GemmArgs g{};
        g.mats = d.mat;
        g.partial = w.partial;
        g.P = g.Q = w.X[cur];
        g.px = g.qx = 1;
        g.acc = pow2(1.0, s.ea - 2 * s.ex);
        g.S = w.A;
        product<kSym>("orth_gram", p, d, kGram, g, stream);
        poly(k, w.A, w.B);
        g.P = w.B;
        int ep = s.eb;
        if (pair) {
            // the next A is B A B, the two steps' factor Q = B' B
            const Scales &t = sc[k + 1];
            square("orth_pair", w.B, w.A, w.S, pow2(1.0, s.es - s.eb - s.ea), nullptr, 0.0f, 0.0f, 1);
            square("orth_pair", w.S, w.B, w.A, pow2(1.0, t.ea - s.es - s.eb), nullptr, 0.0f, 0.0f, 2);
            poly(k + 1, w.A, w.S);
            square("orth_pair", w.S, w.B, w.A, pow2(1.0, s.eq - t.eb - s.eb), nullptr, 0.0f, 0.0f, 1);
            g.P = w.A;
            ep = s.eq;
        }
        k += pair ? 2 : 1;
        const bool last = k == o.steps;
        g.px = 0;
        g.turn = 1;
        g.Q = w.T[cur];
        g.acc = pow2(1.0, (last ? 0 : sc[k].ex) - ep - s.ex);
        cur ^= 1;
        if (last) {
            g.O = O;
            g.W = W;
            g.decay = decay;
            g.lr = lr;
            g.shape = shape;
            product<kOut>("orth_apply", p, d, kApply, g, stream);
        } else {
            g.Xn = w.X[cur];
            g.Tn = w.T[cur];
            product<kNext>("orth_apply", p, d, kApply, g, stream);
        }
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_error(e, fn);
    return GC_OK;
}

// ------------------------------------------------------------- work lists
// A tile of a product before it is planned.
struct Tile {
    uint32_t mat, i, j, stages;
    float weight;  // share of a whole tile's rows and columns that exists
};

// us of a stage of a whole tile, of an item (first loads, writing out), of a
// part's sums written and read again, on the memory's account, and of a join.
// Fitted to the 24 products of four plans (ResNet-50's matrices, four of 1500 x
// 6000, 28 of 800 to 2400 rows, one of 4096 x 4096) in both tiles, whose times
// they give to 7 %.  Plans of a few matrices below about 1,000 rows were not
// among them: there the cost of an item is most of the prediction.
struct Costs {
    uint32_t units;
    double stage, item, part, join;
};

// What the units do, in XCD-major order: the first eighth is on XCD 0, ...
struct Schedule {
    std::vector<std::vector<Item>> items;
    std::vector<Item> joins;
    uint32_t slots = 0;
    double time = 0.0;
};

// Tiles by falling length to the unit with the least to do, as long as that
// stays within `limit`; the others are cut to fill what the units have left
// (pieces of at least 4 stages).  False if the work does not fit.
bool fill_units(const std::vector<Tile> &tiles, const Costs &c, double limit, Schedule *s) {
    auto stage = [&](const Tile &t) { return c.stage * std::max(0.4, static_cast<double>(t.weight)); };
    typedef std::pair<double, uint32_t> Load;
    std::priority_queue<Load, std::vector<Load>, std::greater<Load>> least;
    s->items.resize(c.units);
    for (uint32_t u = 0; u < c.units; ++u) least.push({0.0, u});
    std::vector<const Tile *> cut;
    for (const Tile &t : tiles) {
        const Load l = least.top();
        const double end = l.first + c.item + stage(t) * t.stages;
        if (end > limit * (1.0 + 1e-9)) {
            cut.push_back(&t);
            continue;
        }
        least.pop();
        least.push({end, l.second});
        s->items[l.second].push_back({t.mat, t.i, t.j, 0, t.stages, kNoSlot});
        s->time = std::max(s->time, end);
    }
    for (const Tile *t : cut) {
        uint32_t k = 0;
        const uint32_t slot = s->slots;
        while (k < t->stages) {
            const Load l = least.top();
            const double room = limit - l.first - c.item;
            const uint32_t left = t->stages - k;
            uint32_t n = room <= 0.0 ? 0 : static_cast<uint32_t>(std::min<double>(left, room / stage(*t)));
            if (n < left && left - n < 4) n = left > 4 ? left - 4 : 0;  // no short rest
            if (n < left && n < 4) return false;
            if (n == 0 || (k == 0 && n == left)) return false;
            least.pop();
            const double end = l.first + c.item + stage(*t) * n;
            least.push({end, l.second});
            s->time = std::max(s->time, end);
            s->items[l.second].push_back({t->mat, t->i, t->j, k, k + n, s->slots++});
            k += n;
        }
        // a cut tile does not fit the unit with the least to do, so it has parts
        s->joins.push_back({t->mat, t->i, t->j, 0, s->slots - slot, slot});
    }
    return true;
}

// The fastest schedule in the model: limits from an even share of the work up.
Schedule schedule(std::vector<Tile> tiles, const Costs &c) {
    auto length = [&](const Tile &t) { return std::max(0.4f, t.weight) * static_cast<float>(t.stages); };
    std::stable_sort(tiles.begin(), tiles.end(), [&](const Tile &a, const Tile &b) { return length(a) > length(b); });
    double share = 0.0, longest = 0.0;
    for (const Tile &t : tiles) {
        share += (c.item + c.stage * length(t)) / c.units;
        longest = std::max(longest, c.item + c.stage * length(t));
    }
    Schedule best;
    best.time = -1.0;
    const double top = 2.0 * share + longest;  // no tile is cut there
    for (double limit = share;; limit = std::min(top, limit * 1.05 + 0.5)) {
        Schedule s;
        if (fill_units(tiles, c, limit, &s)) {
            s.time += s.slots * c.part + (s.joins.empty() ? 0.0 : c.join);
            if (best.time < 0.0 || s.time < best.time) best = std::move(s);
        }
        if (limit >= top) return best;
    }
}

// The tiles of a product, neighbours in a block of 4 rows next to each other.
std::vector<Tile> tiles_of(const std::vector<MatDev> &mats, uint32_t tile, List l) {
    std::vector<Tile> out;
    for (uint32_t id = 0; id < mats.size(); ++id) {
        const MatDev &M = mats[id];
        const uint32_t rows = M.mp, cols = l == kApply ? M.np : M.mp;
        const uint32_t nr = (rows + tile - 1) / tile, nc = (cols + tile - 1) / tile;
        const uint32_t stages = static_cast<uint32_t>(ceil_div(l == kGram ? M.n : M.m, 32));
        auto share = [&](uint32_t all, uint32_t at) { return static_cast<float>(std::min(tile, all - at * tile)) / tile; };
        for (uint32_t ib = 0; ib < nr; ib += 4)
            for (uint32_t j = 0; j < nc; ++j)
                for (uint32_t i = ib; i < std::min(ib + 4, nr); ++i)
                    if (l == kApply || j <= i) out.push_back({id, i, j, stages, share(rows, i) * share(cols, j)});
    }
    return out;
}

// Two steps at a time: with A' = B A B and Q = B' B, both m x m, the second
// step needs no product with X of its own; 4 more products of m x m instead of
// one X X^T and one B X, and one poly as before.  Only where every matrix has
// kPairRows rows: below, the sums are short and the roundings of Q's entries
// (up to a^2 = 12, which cancel in Q X) stand out against them: at 256 x 1024
// 1.1 times the error of fp32 products after 5 steps and 2.1 times after 3 (0.8
// and 1.0 one at a time), at 512 x 4608 0.4 and 1.2 (0.4 and 0.8), at 1500 x 6000
// 0.5 and 0.9 (0.4 and 0.7).
constexpr uint32_t kPairRows = 512;

// Matrices of few rows: slabs per workgroup so that they fill the units once
// and no matrix has more than kMaxParts parts, which one workgroup adds.
constexpr uint64_t kMaxParts = 16;
// Up to here, and with 64 rows at most, a slab's workgroup makes its B itself
// (times at the slab kernel's section).
constexpr uint64_t kFusedSlabs = 256;

void plan_narrow(gc_matrix_plan *p, uint32_t most) {
    p->narrow = true;
    uint64_t slabs = 0;
    uint32_t slots = 0;
    for (const MatDev &M : p->mat) slabs += M.np / kNarrow;
    for (uint32_t id = 0; id < p->mat.size(); ++id) {
        const uint32_t n = p->mat[id].np / kNarrow;
        const uint32_t per = static_cast<uint32_t>(std::max(ceil_div(n, kMaxParts), ceil_div(slabs, Small::kUnits)));
        const uint32_t parts = static_cast<uint32_t>(ceil_div(n, per));
        const uint32_t slot = slots;
        p->list[kSmalls].push_back({id, 0, 0, 0, parts, slot});
        for (uint32_t q = 0; q < parts; ++q)
            p->list[kSlabs].push_back({id, slot, parts, q * per, std::min((q + 1) * per, n), slots++});
    }
    p->fused = most <= 64 && slabs <= kFusedSlabs;
    p->partial = static_cast<uint64_t>(slots) * kNarrow * kNarrow * (p->fused ? 2 : 1);
}

// The tables of every matrix.
void fill_plan(gc_matrix_plan *p, const gc_plan *plan, const uint32_t *rows) {
    p->n_total = plan->n_total;
    uint64_t x = 0, a = 0;
    uint32_t chunk0 = 0;
    for (int s = 0; s < plan->nseg; ++s) {
        if (!rows[s]) continue;
        MatDev M{};
        M.off = plan->seg[s].off;
        M.len = plan->seg[s].len;
        M.R = rows[s];
        M.C = static_cast<uint32_t>(M.len / M.R);
        M.flip = M.R > M.C ? 1 : 0;
        M.m = M.flip ? M.C : M.R;
        M.n = M.flip ? M.R : M.C;
        M.mp = pad_up(M.m);
        M.np = pad_up(M.n);
        M.x = x;
        M.a = a;
        M.chunk0 = chunk0;
        M.nchunk = static_cast<uint32_t>(ceil_div(M.len, kChunk));
        x += 2 * static_cast<uint64_t>(M.mp) * M.np;
        a += 2 * static_cast<uint64_t>(M.mp) * M.mp;
        chunk0 += M.nchunk;
        const uint32_t id = static_cast<uint32_t>(p->mat.size());
        for (uint32_t c = 0; c < M.nchunk; ++c) p->list[kChunks].push_back({id, c, 0, 0, 0, 0});
        for (uint32_t i = 0; i < M.mp / kSplitTile; ++i)
            for (uint32_t j = 0; j < M.np / kSplitTile; ++j) p->list[kTiles].push_back({id, i, j, 0, 0, 0});
        p->mat.push_back(M);
    }
    p->xhalves = x;
    p->ahalves = a;
    uint32_t least = 0xFFFFFFFFu, most = 0;
    for (const MatDev &M : p->mat) {
        least = std::min(least, M.m);
        most = std::max(most, M.m);
    }
    if (most <= kNarrow) {
        plan_narrow(p, most);
        return;
    }
    // per product the tile shape and schedule that the model finds fastest
    const Costs costs[2] = {{Small::kUnits, 1.18, 17.5, 0.02, 5.5}, {Large::kUnits, 2.33, 14.0, 0.04, 8.0}};
    constexpr List kProducts[3] = {kGram, kSquare, kApply};
    Schedule best[3];
    for (int q = 0; q < 3; ++q) {
        const List l = kProducts[q];
        best[q] = schedule(tiles_of(p->mat, Small::kTile, l), costs[0]);
        Schedule s = schedule(tiles_of(p->mat, Large::kTile, l), costs[1]);
        if (s.time < best[q].time) {
            p->large[l] = true;
            best[q] = std::move(s);
        }
        const uint64_t tile = p->large[l] ? Large::kTile : Small::kTile;
        p->partial = std::max(p->partial, best[q].slots * tile * tile);
    }
    p->pairs = least >= kPairRows && best[0].time + best[2].time > 3.0 * best[1].time;
    for (int q = 0; q < 3; ++q) {
        // workgroup b runs on XCD b % 8; units next to each other, with tiles next to
        // each other, share an XCD and its L2
        std::vector<Item> &items = p->list[kProducts[q]];
        std::vector<uint32_t> &first = p->first[kProducts[q]];
        const uint32_t units = static_cast<uint32_t>(best[q].items.size());
        for (uint32_t b = 0; b < units; ++b) {
            const std::vector<Item> &of = best[q].items[b % 8 * (units / 8) + b / 8];
            first.push_back(static_cast<uint32_t>(items.size()));
            items.insert(items.end(), of.begin(), of.end());
        }
        first.push_back(static_cast<uint32_t>(items.size()));
        p->list[kProducts[q] + 1] = std::move(best[q].joins);
    }
}

// Whether two buffers of n floats share an element.
bool overlap(const float *a, const float *b, uint64_t n) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + 4 * n && y < x + 4 * n;
}

}  // namespace
}  // namespace gc

using namespace gc;

extern "C" gc_status gc_matrix_plan_create(const gc_plan *plan, const uint32_t *rows, gc_matrix_plan **out) {
    clear_error();
    if (!out) return set_error(GC_EINVAL, "gc_matrix_plan_create: out is null");
    if (!plan) return set_error(GC_EINVAL, "gc_matrix_plan_create: plan is null");
    if (!rows) return set_error(GC_EINVAL, "gc_matrix_plan_create: rows is null");
    uint64_t nmat = 0;
    for (int s = 0; s < plan->nseg; ++s) {
        if (!rows[s]) continue;
        const std::string at = "gc_matrix_plan_create: segment " + std::to_string(s) + ": ";
        const uint32_t len = plan->seg[s].len;
        if (len % rows[s]) return set_error(GC_EINVAL, at + "rows must divide the segment's length");
        const uint32_t cols = len / rows[s];
        if (rows[s] > GC_MAX_MATRIX_DIM || cols > GC_MAX_MATRIX_DIM)
            return set_error(GC_ENOTSUP, at + "a matrix has more than GC_MAX_MATRIX_DIM rows or columns");
        ++nmat;
    }
    if (!nmat) return set_error(GC_EINVAL, "gc_matrix_plan_create: no segment is a matrix");
    gc_matrix_plan *p = new (std::nothrow) gc_matrix_plan;
    if (!p) return set_error(GC_EINVAL, "gc_matrix_plan_create: out of host memory");
    try {
        fill_plan(p, plan, rows);
    } catch (const std::bad_alloc &) {
        delete p;
        return set_error(GC_EINVAL, "gc_matrix_plan_create: out of host memory");
    }
    // grids of up to 256 threads (joins: 16 workgroups a tile) stay below 2^32
    for (int l = 0; l < kLists; ++l)
        if (p->list[l].size() >= (size_t(1) << 20) * (l == kGramJoin || l == kSquareJoin || l == kApplyJoin ? 1 : 16)) {
            delete p;
            return set_error(GC_ERANGE, "gc_matrix_plan_create: too many tiles");
        }
    *out = p;
    return GC_OK;
}

extern "C" void gc_matrix_plan_destroy(gc_matrix_plan *p) {
    if (!p) return;
    int cur = 0;
    const bool have = hipGetDevice(&cur) == hipSuccess;
    for (auto &pr : p->dev_blob)
        if (hipSetDevice(pr.first) == hipSuccess) (void)hipFree(pr.second);
    if (have) (void)hipSetDevice(cur);
    delete p;
}

extern "C" gc_status gc_matrix_plan_upload(const gc_matrix_plan *p) {
    clear_error();
    if (!p) return set_error(GC_EINVAL, "gc_matrix_plan_upload: matrix plan is null");
    OrthDev d;
    return orth_device(p, &d);
}

extern "C" size_t gc_matrix_plan_workspace_bytes(const gc_matrix_plan *p) {
    return p ? orth_ws(nullptr, p).bytes : 0;
}

extern "C" gc_status gc_orthogonalize(const gc_matrix_plan *p, const float *D, float *O, const gc_orth_options *opt,
                                      void *ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    Scales sc[GC_MAX_ORTH_STEPS + 1];
    gc_status st = check_orth("gc_orthogonalize", p, opt, ws, ws_bytes, sc);
    if (st != GC_OK) return st;
    if (!D || !O) return set_error(GC_EINVAL, "gc_orthogonalize: buffers must be non-null");
    if (D != O && overlap(D, O, p->n_total))
        return set_error(GC_EINVAL, "gc_orthogonalize: O may be D or must not overlap it");
    Source src{};
    src.G = D;
    return orthogonalize("gc_orthogonalize", p, *opt, sc, src, O, nullptr, 0.0f, 0.0f, 0, ws, stream);
}

extern "C" gc_status gc_muon_step(const gc_matrix_plan *p, const float *G, float *U, float *W, const gc_muon_options *opt,
                                  void *ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    Scales sc[GC_MAX_ORTH_STEPS + 1];
    gc_status st = check_orth("gc_muon_step", p, opt ? &opt->orth : nullptr, ws, ws_bytes, sc);
    if (st != GC_OK) return st;
    if (!(opt->momentum >= 0.0f && opt->momentum < 1.0f))
        return set_error(GC_EINVAL, "gc_muon_step: momentum must be in [0, 1)");
    if (!(opt->lr - opt->lr == 0.0f)) return set_error(GC_EINVAL, "gc_muon_step: lr must be finite");
    if (!(opt->weight_decay >= 0.0f) || !(opt->weight_decay - opt->weight_decay == 0.0f))
        return set_error(GC_EINVAL, "gc_muon_step: weight_decay must be finite and >= 0");
    if (opt->momentum_kind != GC_MOMENTUM_VANILLA && opt->momentum_kind != GC_MOMENTUM_NESTEROV)
        return set_error(GC_EINVAL, "gc_muon_step: unknown momentum_kind");
    if (opt->scale != GC_MUON_SCALE_NONE && opt->scale != GC_MUON_SCALE_SHAPE && opt->scale != GC_MUON_SCALE_RMS)
        return set_error(GC_EINVAL, "gc_muon_step: unknown scale");
    if (opt->reserved) return set_error(GC_EINVAL, "gc_muon_step: reserved must be 0");
    if (!G || !U || !W) return set_error(GC_EINVAL, "gc_muon_step: buffers must be non-null");
    if (overlap(G, U, p->n_total) || overlap(G, W, p->n_total) || overlap(U, W, p->n_total))
        return set_error(GC_EINVAL, "gc_muon_step: G, U and W must not overlap");
    Source src{};
    src.G = G;
    src.U = U;
    src.momentum = opt->momentum;
    src.nesterov = opt->momentum_kind == GC_MOMENTUM_NESTEROV ? 1 : 0;
    const float decay = static_cast<float>(1.0 - static_cast<double>(opt->lr) * static_cast<double>(opt->weight_decay));
    return orthogonalize("gc_muon_step", p, opt->orth, sc, src, nullptr, W, decay, opt->lr, opt->scale, ws, stream);
}
