// Orthogonalised updates of weight matrices (gc_orthogonalize, gc_muon_step):
//
//   X_0 = D / (||D||_F + eps), m x n with m <= n (D or its transpose)
//   A = X X^T,  B = b A + c A^2,  X <- a X + B X       `steps` times
//
// Every product runs on the matrix cores in three fp16 products: an fp32
// value x 2^e is held as hi + lo, hi = fp16(x 2^e), lo = fp16(x 2^e - hi), 22
// bits, and P Q^T = hi hi^T + hi lo^T + lo hi^T with fp32 sums (lo lo^T is
// below the last bit kept).  Measured against 64 bits the result is as near as
// fp32 products are, at a third of the fp16 rate instead of a sixteenth.
// fp16 has no range to spare, so each array has its own power of two: singular
// values of X_0 are at most 1, the polynomial bounds those of every later X, A
// and B, and no entry exceeds its matrix's largest singular value
// (orth_scales).
//
// All products have the form P Q^T with the common index running along the
// rows of both: X X^T and A A^T (A is symmetric) as they stand, B X = B T^T
// with T = X^T, which is kept beside X.  A and B are symmetric: only tiles on
// and below the diagonal are computed, the others are their mirror images.
#include <cmath>
#include <cstring>
#include <new>
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

// A workgroup's work: a matrix and a tile (norm: a chunk).
struct Item {
    uint32_t mat, i, j, reserved;
};

constexpr int kTM = 128, kTN = 128;  // output tile of a product
constexpr int kTK = 32;              // columns of the common index per stage
constexpr int kSplitTile = 64;       // orth_split's tile

struct OrthDev {
    const MatDev *mat;
    const Item *chunks, *tri, *rect, *tiles;
    uint32_t nmat, nchunks, ntri, nrect, ntiles;
};

}  // namespace
}  // namespace gc

struct gc_matrix_plan {
    uint64_t n_total = 0;
    uint64_t xhalves = 0, ahalves = 0;  // halves of one X (or T) array and of one A (or B) array
    std::vector<gc::MatDev> mat;
    std::vector<gc::Item> chunks, tri, rect, tiles;
    std::mutex mu;
    std::vector<std::pair<int, void *>> dev_blob;
};

namespace gc {

namespace {

// ----------------------------------------------------------- tables, scales
struct Blob {
    size_t mat, chunks, tri, rect, tiles, total;
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
    L.chunks = take(sizeof(Item) * p->chunks.size());
    L.tri = take(sizeof(Item) * p->tri.size());
    L.rect = take(sizeof(Item) * p->rect.size());
    L.tiles = take(sizeof(Item) * p->tiles.size());
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
            std::memcpy(host.data() + L.chunks, p->chunks.data(), sizeof(Item) * p->chunks.size());
            std::memcpy(host.data() + L.tri, p->tri.data(), sizeof(Item) * p->tri.size());
            std::memcpy(host.data() + L.rect, p->rect.data(), sizeof(Item) * p->rect.size());
            std::memcpy(host.data() + L.tiles, p->tiles.data(), sizeof(Item) * p->tiles.size());
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
    out->chunks = reinterpret_cast<const Item *>(b + L.chunks);
    out->tri = reinterpret_cast<const Item *>(b + L.tri);
    out->rect = reinterpret_cast<const Item *>(b + L.rect);
    out->tiles = reinterpret_cast<const Item *>(b + L.tiles);
    out->nmat = static_cast<uint32_t>(p->mat.size());
    out->nchunks = static_cast<uint32_t>(p->chunks.size());
    out->ntri = static_cast<uint32_t>(p->tri.size());
    out->nrect = static_cast<uint32_t>(p->rect.size());
    out->ntiles = static_cast<uint32_t>(p->tiles.size());
    return GC_OK;
}

// Exponents of one step's split arrays: X 2^ex, A 2^ea, B 2^eb.
struct Scales {
    int ex, ea, eb;
};

// The largest exponent that keeps |v| <= bound below 60000 in fp16.
int exponent_for(double bound) { return static_cast<int>(std::floor(std::log2(60000.0 / bound))); }

// Bounds of the singular values of X, A and B at every step, from the
// polynomial on [0, top]: sampled at 4096 points, with what it can rise
// between two of them (a derivative's bound times half a spacing) and 1/64
// for rounding.  s[k] is step k's, s[steps] the result's.
// The bounds are worst cases; what a matrix really holds may be smaller by
// as much as the bounds are loose, and where that reaches fp16's subnormals
// the lo parts lose bits (a schedule whose bound rose to 24 and then 3e6 gave
// 5.2e-6 where fp32 gives 2.7e-7).  So false, a refusal, if X's bound passes 8
// before the last step, B's 2^14, the result's 1e12, or one vanishes.
bool orth_scales(const gc_orth_options &o, Scales *s) {
    double top = 1.0 + 1.0 / 64;
    for (int k = 0; k <= o.steps; ++k) {
        s[k].ex = exponent_for(top);
        if (k == o.steps) break;
        const double a = o.coef[k][0], b = o.coef[k][1], c = o.coef[k][2];
        constexpr int kPoints = 4096;
        double px = 0.0, pb = 0.0;
        for (int i = 0; i <= kPoints; ++i) {
            const double x = top * i / kPoints, q = (b + c * x * x) * x * x;
            pb = std::max(pb, std::fabs(q));
            px = std::max(px, std::fabs((a + q) * x));
        }
        const double t2 = top * top, half = 0.5 * top / kPoints;
        pb += half * (2 * std::fabs(b) * top + 4 * std::fabs(c) * t2 * top);
        px += half * (std::fabs(a) + 3 * std::fabs(b) * t2 + 5 * std::fabs(c) * t2 * t2);
        s[k].ea = exponent_for(t2 * (1.0 + 1.0 / 64));
        s[k].eb = exponent_for(std::max(pb, 1e-12) * (1.0 + 1.0 / 64));
        top = px * (1.0 + 1.0 / 64);
        if (!(top <= (k + 1 == o.steps ? 1e12 : 8.0)) || !(pb <= 16384.0) || !(top > 1e-12)) return false;
    }
    return true;
}

// --------------------------------------------------------------- workspace
struct OrthWs {
    _Float16 *X[2], *T[2], *A, *B;
    double *partial, *inv;
    size_t bytes;
};

OrthWs orth_ws(void *ws, const gc_matrix_plan *p) {
    WsCursor c(ws);
    OrthWs w{};
    for (int k = 0; k < 2; ++k) {
        w.X[k] = c.take<_Float16>(p->xhalves);
        w.T[k] = c.take<_Float16>(p->xhalves);
    }
    w.A = c.take<_Float16>(p->ahalves);
    w.B = c.take<_Float16>(p->ahalves);
    w.partial = c.take<double>(p->chunks.size());
    w.inv = c.take<double>(p->mat.size());
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
// chunk's sum of D^2 in double.
__global__ __launch_bounds__(kBlock) void orth_norm_kernel(const Item *__restrict__ items, const MatDev *__restrict__ mats,
                                                           Source s, double *__restrict__ partial) {
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
    if (threadIdx.x == 0) partial[M.chunk0 + it.i] = sum;
}

// Per matrix: 1 / (||D|| + eps); 0 for D = 0, NaN where D is not finite.
__global__ __launch_bounds__(kBlock) void orth_scale_kernel(const MatDev *__restrict__ mats,
                                                            const double *__restrict__ partial, float eps,
                                                            double *__restrict__ inv) {
    const MatDev M = mats[blockIdx.x];
    double sum = 0.0;
    for (uint32_t c = threadIdx.x; c < M.nchunk; c += kBlock) sum += partial[M.chunk0 + c];
    sum = block_tree_sum(sum);
    if (threadIdx.x == 0)
        inv[blockIdx.x] = sum == 0.0 ? 0.0 : sum - sum == 0.0 ? 1.0 / (sqrt(sum) + static_cast<double>(eps)) : __builtin_nan("");
}

// A 64 x 64 tile of X_0, split, into X and T; the padding becomes zeros.
__global__ __launch_bounds__(kBlock) void orth_split_kernel(const Item *__restrict__ items, const MatDev *__restrict__ mats,
                                                            Source s, const double *__restrict__ inv, float pow2,
                                                            _Float16 *__restrict__ X, _Float16 *__restrict__ T) {
    const Item it = items[blockIdx.x];
    const MatDev M = mats[it.mat];
    __shared__ float tile[kSplitTile][kSplitTile + 1];  // [i][j] of X
    const double scale = inv[it.mat] * static_cast<double>(pow2);
    const uint32_t i0 = it.i * kSplitTile, j0 = it.j * kSplitTile;
    // D is read along its rows: lanes run over j, or over i where X = D^T
    const uint32_t l = threadIdx.x & 63, r0 = threadIdx.x >> 6;
    for (uint32_t r = r0; r < kSplitTile; r += kWaves) {
        const uint32_t i = M.flip ? i0 + l : i0 + r, j = M.flip ? j0 + r : j0 + l;
        float v = 0.0f;
        if (i < M.m && j < M.n) {
            const uint64_t at = M.off + (M.flip ? static_cast<uint64_t>(j) * M.C + i : static_cast<uint64_t>(i) * M.C + j);
            const float g = s.G[at];
            const float d = s.U ? direction(s, s.U[at], g) : g;
            v = static_cast<float>(static_cast<double>(d) * scale);
        }
        tile[M.flip ? l : r][M.flip ? r : l] = v;
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < kSplitTile * kSplitTile / 4; e += kBlock) {
        const uint32_t r = e / (kSplitTile / 4), c = e % (kSplitTile / 4) * 4;
        h4 hi, lo;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            _Float16 a, b;
            split(tile[r][c + u], a, b);
            hi[u] = a;
            lo[u] = b;
        }
        _Float16 *p = X + M.x + static_cast<uint64_t>(i0 + r) * M.np * 2 + split_at(j0 + c);
        *reinterpret_cast<h4 *>(p) = hi;
        *reinterpret_cast<h4 *>(p + 32) = lo;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            _Float16 a, b;
            split(tile[c + u][r], a, b);
            hi[u] = a;
            lo[u] = b;
        }
        p = T + M.x + static_cast<uint64_t>(j0 + r) * M.mp * 2 + split_at(i0 + c);
        *reinterpret_cast<h4 *>(p) = hi;
        *reinterpret_cast<h4 *>(p + 32) = lo;
    }
}

// ---------------------------------------------------------------- products
enum Phase { kGram, kPoly, kApply, kLast };

struct GemmArgs {
    const Item *items;
    const MatDev *mats;
    const _Float16 *X, *T;  // this step's
    _Float16 *A, *B;
    _Float16 *Xn, *Tn;      // the next step's
    float acc, add;         // result = acc * (P Q^T) + add * (the addend as stored)
    // kLast: the result, or the weights it is applied to
    float *O, *W;
    float decay, lr;        // W <- decay W - lr s O
    int shape;              // GC_MUON_SCALE_*
};

// s of a matrix for GC_MUON_SCALE_*.
__device__ __forceinline__ double shape_scale(int shape, uint32_t R, uint32_t C) {
    if (shape == GC_MUON_SCALE_SHAPE) return R > C ? sqrt(static_cast<double>(R) / static_cast<double>(C)) : 1.0;
    if (shape == GC_MUON_SCALE_RMS) return 0.2 * sqrt(static_cast<double>(R > C ? R : C));
    return 1.0;
}

// One 128 x 128 tile of P Q^T by 4 waves of 64 x 64 (4 x 4 matrix-core tiles
// of 16 x 16).  A stage holds 32 columns of both planes of 128 rows of P and
// Q, 32 KB; two stages alternate, the next one's global loads are in flight
// while this one is multiplied.  Inside a 128-byte row the 16-byte parts are
// permuted by (row >> 1) & 7, so that the 16 rows a matrix-core operand
// reads at once lie in different banks.
template <Phase kPhase>
__global__ __launch_bounds__(kBlock) void orth_gemm_kernel(GemmArgs g) {
    const Item it = g.items[blockIdx.x];
    const MatDev M = g.mats[it.mat];
    const _Float16 *P, *Q;
    uint32_t ld;  // padded length of the common index
    if (kPhase == kGram) {
        P = g.X + M.x;
        Q = P;
        ld = M.np;
    } else if (kPhase == kPoly) {
        P = g.A + M.a;
        Q = P;
        ld = M.mp;
    } else {
        P = g.B + M.a;
        Q = g.T + M.x;
        ld = M.mp;
    }
    const uint32_t i0 = it.i * kTM, j0 = it.j * kTN;
    const uint32_t kreal = kPhase == kGram ? M.n : M.m;
    const uint32_t nk = (kreal + kTK - 1) / kTK;
    __shared__ _Float16 lp[2][kTM * 64], lq[2][kTN * 64];
    const uint32_t t = threadIdx.x, lane = lane_id(), w = wave_id();
    // staging: 8 parts of 16 bytes a row, thread t takes part t & 7 of rows t / 8 + 32 s
    const uint32_t part = t & 7, row = t >> 3;
    const _Float16 *ps = P + static_cast<uint64_t>(i0 + row) * ld * 2 + part * 8;
    const _Float16 *qs = Q + static_cast<uint64_t>(j0 + row) * ld * 2 + part * 8;
    const uint64_t rstep = static_cast<uint64_t>(32) * ld * 2;
    h8 rp[4], rq[4];
    auto fetch = [&](uint32_t k) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            rp[s] = *reinterpret_cast<const h8 *>(ps + s * rstep + k * 64);
            rq[s] = *reinterpret_cast<const h8 *>(qs + s * rstep + k * 64);
        }
    };
    auto stash = [&](int buf) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t r = row + 32 * s, at = r * 64 + (part ^ ((r >> 1) & 7)) * 8;
            *reinterpret_cast<h8 *>(&lp[buf][at]) = rp[s];
            *reinterpret_cast<h8 *>(&lq[buf][at]) = rq[s];
        }
    };
    const uint32_t wi = (w >> 1) * 64, wj = (w & 1) * 64;  // the wave's corner in the tile
    const uint32_t fr = lane & 15, fc = lane >> 4;         // operand row and 16-byte part
    f32x4 acc[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    fetch(0);
    stash(0);
    __syncthreads();
    for (uint32_t k = 0; k < nk; ++k) {
        const int buf = k & 1;
        if (k + 1 < nk) fetch(k + 1);
        h8 ph[4], pl[4], qh[4], ql[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const uint32_t ri = wi + 16 * a + fr, rj = wj + 16 * a + fr;
            const uint32_t si = (ri >> 1) & 7, sj = (rj >> 1) & 7;
            ph[a] = *reinterpret_cast<const h8 *>(&lp[buf][ri * 64 + (fc ^ si) * 8]);
            pl[a] = *reinterpret_cast<const h8 *>(&lp[buf][ri * 64 + ((fc + 4) ^ si) * 8]);
            qh[a] = *reinterpret_cast<const h8 *>(&lq[buf][rj * 64 + (fc ^ sj) * 8]);
            ql[a] = *reinterpret_cast<const h8 *>(&lq[buf][rj * 64 + ((fc + 4) ^ sj) * 8]);
        }
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph[a], ql[b], acc[a][b], 0, 0, 0);
                acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(pl[a], qh[b], acc[a][b], 0, 0, 0);
                acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph[a], qh[b], acc[a][b], 0, 0, 0);
            }
        if (k + 1 < nk) stash(buf ^ 1);
        __syncthreads();
    }
    // lane: column j = fr, rows 4 fc .. 4 fc + 3 of each 16 x 16 tile
    const bool mirror = (kPhase == kGram || kPhase == kPoly) && it.i != it.j;
    const double sc = kPhase == kLast && g.W ? shape_scale(g.shape, M.R, M.C) : 1.0;
    const float step = static_cast<float>(static_cast<double>(g.lr) * sc);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t i = i0 + wi + 16 * a + 4 * fc, j = j0 + wj + 16 * b + fr;
            float v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = acc[a][b][u] * g.acc;
            if (kPhase != kGram) {
                // the addend, read along the other index: A is symmetric, T = X^T
                const _Float16 *p = kPhase == kPoly ? g.A + M.a + static_cast<uint64_t>(j) * M.mp * 2
                                                    : g.T + M.x + static_cast<uint64_t>(j) * M.mp * 2;
                const h4 hi = *reinterpret_cast<const h4 *>(p + split_at(i));
                const h4 lo = *reinterpret_cast<const h4 *>(p + split_at(i) + 32);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    v[u] = v[u] + g.add * (static_cast<float>(hi[u]) + static_cast<float>(lo[u]));
            }
            if (kPhase == kLast) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (i + u < M.m && j < M.n) {
                        const uint64_t at = M.off + (M.flip ? static_cast<uint64_t>(j) * M.C + i + u
                                                            : static_cast<uint64_t>(i + u) * M.C + j);
                        if (g.W) g.W[at] = g.decay * g.W[at] - step * v[u];
                        else g.O[at] = v[u];
                    }
                }
                continue;
            }
            h4 hi, lo;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                _Float16 x, y;
                split(v[u], x, y);
                hi[u] = x;
                lo[u] = y;
            }
            // [j][i .. i + 3], and [i + u][j] where that is another place
            _Float16 *pt = kPhase == kGram   ? g.A + M.a + static_cast<uint64_t>(j) * M.mp * 2
                           : kPhase == kPoly ? g.B + M.a + static_cast<uint64_t>(j) * M.mp * 2
                                             : g.Tn + M.x + static_cast<uint64_t>(j) * M.mp * 2;
            *reinterpret_cast<h4 *>(pt + split_at(i)) = hi;
            *reinterpret_cast<h4 *>(pt + split_at(i) + 32) = lo;
            if (kPhase == kApply || mirror) {
                _Float16 *px = kPhase == kGram   ? g.A + M.a
                               : kPhase == kPoly ? g.B + M.a
                                                 : g.Xn + M.x;
                const uint32_t ldx = kPhase == kApply ? M.np : M.mp;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    _Float16 *q = px + static_cast<uint64_t>(i + u) * ldx * 2 + split_at(j);
                    q[0] = hi[u];
                    q[32] = lo[u];
                }
            }
        }
}

// --------------------------------------------------------------- host side
void *align256(void *p) {
    return reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(p) + 255) & ~uintptr_t(255));
}

gc_status check_orth(const char *fn, const gc_matrix_plan *p, const gc_orth_options *o, const void *ws, size_t ws_bytes,
                     Scales *s) {
    const std::string at = std::string(fn) + ": ";
    if (!p) return set_error(GC_EINVAL, at + "matrix plan is null");
    if (!o) return set_error(GC_EINVAL, at + "opt is null");
    if (o->steps < 1 || o->steps > GC_MAX_ORTH_STEPS) return set_error(GC_EINVAL, at + "steps must be in [1, GC_MAX_ORTH_STEPS]");
    if (!(o->eps >= 0.0f) || !(o->eps - o->eps == 0.0f)) return set_error(GC_EINVAL, at + "eps must be finite and >= 0");
    if (o->reserved[0] || o->reserved[1]) return set_error(GC_EINVAL, at + "reserved fields must be 0");
    if (!orth_scales(*o, s))
        return set_error(GC_EINVAL, at + "coef must be finite and keep the singular values of X at most 8");
    if (!ws) return set_error(GC_EINVAL, at + "ws must be non-null");
    if (ws_bytes < orth_ws(nullptr, p).bytes)
        return set_error(GC_ECAPACITY, at + "workspace smaller than gc_matrix_plan_workspace_bytes");
    return GC_OK;
}

gc_status orthogonalize(const char *fn, const gc_matrix_plan *p, const gc_orth_options &o, const Scales *sc, Source src,
                        float *O, float *W, float decay, float lr, int shape, void *ws, hipStream_t stream) {
    OrthDev d;
    gc_status st = orth_device(p, &d);
    if (st != GC_OK) return st;
    const OrthWs w = orth_ws(align256(ws), p);
    GC_LAUNCH("orth_norm", stream, orth_norm_kernel<<<d.nchunks, kBlock, 0, stream>>>(d.chunks, d.mat, src, w.partial));
    GC_LAUNCH("orth_scale", stream, orth_scale_kernel<<<d.nmat, kBlock, 0, stream>>>(d.mat, w.partial, o.eps, w.inv));
    GC_LAUNCH("orth_split", stream,
              orth_split_kernel<<<d.ntiles, kBlock, 0, stream>>>(d.tiles, d.mat, src, w.inv,
                                                               static_cast<float>(std::ldexp(1.0, sc[0].ex)), w.X[0], w.T[0]));
    auto pow2 = [](int e) { return static_cast<float>(std::ldexp(1.0, e)); };
    int cur = 0;
    for (int k = 0; k < o.steps; ++k) {
        const Scales &s = sc[k];
        GemmArgs g{};
        g.mats = d.mat;
        g.X = w.X[cur];
        g.T = w.T[cur];
        g.A = w.A;
        g.B = w.B;
        g.Xn = w.X[cur ^ 1];
        g.Tn = w.T[cur ^ 1];
        g.items = d.tri;
        g.acc = pow2(s.ea - 2 * s.ex);
        GC_LAUNCH("orth_gram", stream, orth_gemm_kernel<kGram><<<d.ntri, kBlock, 0, stream>>>(g));
        g.acc = static_cast<float>(std::ldexp(static_cast<double>(o.coef[k][2]), s.eb - 2 * s.ea));
        g.add = static_cast<float>(std::ldexp(static_cast<double>(o.coef[k][1]), s.eb - s.ea));
        GC_LAUNCH("orth_poly", stream, orth_gemm_kernel<kPoly><<<d.ntri, kBlock, 0, stream>>>(g));
        g.items = d.rect;
        const bool last = k + 1 == o.steps;
        const int en = last ? 0 : sc[k + 1].ex;
        g.acc = pow2(en - s.eb - s.ex);
        g.add = static_cast<float>(std::ldexp(static_cast<double>(o.coef[k][0]), en - s.ex));
        if (last) {
            g.O = O;
            g.W = W;
            g.decay = decay;
            g.lr = lr;
            g.shape = shape;
            GC_LAUNCH("orth_apply", stream, orth_gemm_kernel<kLast><<<d.nrect, kBlock, 0, stream>>>(g));
        } else {
            GC_LAUNCH("orth_apply", stream, orth_gemm_kernel<kApply><<<d.nrect, kBlock, 0, stream>>>(g));
        }
        cur ^= 1;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_error(e, fn);
    return GC_OK;
}

// The tables of every matrix.
void fill_plan(gc_matrix_plan *p, const gc_plan *plan, const uint32_t *rows) {
    p->n_total = plan->n_total;    uint64_t x = 0, a = 0;
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
        for (uint32_t c = 0; c < M.nchunk; ++c) p->chunks.push_back({id, c, 0, 0});
        for (uint32_t i = 0; i < M.mp / kTM; ++i)
            for (uint32_t j = 0; j <= i; ++j) p->tri.push_back({id, i, j, 0});
        for (uint32_t j = 0; j < M.np / kTN; ++j)
            for (uint32_t i = 0; i < M.mp / kTM; ++i) p->rect.push_back({id, i, j, 0});
        for (uint32_t i = 0; i < M.mp / kSplitTile; ++i)
            for (uint32_t j = 0; j < M.np / kSplitTile; ++j) p->tiles.push_back({id, i, j, 0});
        p->mat.push_back(M);
    }
    p->xhalves = x;
    p->ahalves = a;
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
