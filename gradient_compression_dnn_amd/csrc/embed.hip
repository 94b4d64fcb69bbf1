// The embedding of a model's flat buffer: the scaled lookup of a batch of
// tokens (gc_embed_lookup) and its gradient by sorted tokens, dense or added
// (gc_embed_grad) or as a sparse message (gc_embed_message).
//
//   y_i  = round(fl32(scale * w[t_i]))
//   g[r] = fl32(scale * sum of dy_i over the positions i with t_i = r)
//
// The sum of a row takes its positions in ascending order, so positions are
// sorted by (row, position) first.  The sort is stable and its result does not
// hang on the order of any atomics, hence every sum has one order and the
// result one bit pattern:
//   rank   each tile of tokens is ranked by counting: the rank of i is the
//          number of keys below key_i, or equal and before i.  4.2 M
//          comparisons a tile of 2048, and nothing waits for another pass.
//   merge  16 sorted runs at a time: an element's rank in the merged run is
//          its own plus its place in each other run.
//   sum    16 sorted positions by 256 (fp32) or 512 columns per wave.  A row
//          whose run lies inside the block is finished there; a run that
//          crosses blocks leaves one partial sum per block.
//   join   the partial sums of each crossing run.
#include <algorithm>
#include <string>

#include "gc_internal.hpp"

namespace gc {

namespace {

// N elements with the alignment of one: the hardware's unaligned mode takes
// 8 or 16 bytes as one access, so odd offsets and strides need no variant.
template <class S, int N>
struct __attribute__((packed, aligned(sizeof(S)))) Pack {
    S v[N];
};

// Storage types.
struct F32 {
    using Store = float;
    static __device__ __forceinline__ float to_f32(float x) { return x; }
    static __device__ __forceinline__ float from_f32(float x) { return x; }
};
struct BF16 {
    using Store = uint16_t;
    static __device__ __forceinline__ float to_f32(uint16_t x) { return dev_u2f(uint32_t(x) << 16); }
    static __device__ __forceinline__ uint16_t from_f32(float x) {
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
    }
};
struct F16 {
    using Store = uint16_t;
    static __device__ __forceinline__ float to_f32(uint16_t x) {
        return static_cast<float>(__builtin_bit_cast(_Float16, x));
    }
    static __device__ __forceinline__ uint16_t from_f32(float x) {
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
    }
};

// N columns of a row from column c on; those at or past cols are 0 / dropped.
// A vector access needs all of them, so a row's last lane goes by elements.
template <class T, int N>
__device__ __forceinline__ void load_cols(const typename T::Store *row, uint32_t c, uint32_t cols, float (&v)[N]) {
    constexpr int kVec = N * int(sizeof(typename T::Store)) <= 16 ? N : 16 / int(sizeof(typename T::Store));
    if (c + N <= cols) {
#pragma unroll
        for (int k = 0; k < N; k += kVec) {
            const auto t = *reinterpret_cast<const Pack<typename T::Store, kVec> *>(row + c + k);
#pragma unroll
            for (int u = 0; u < kVec; ++u) v[k + u] = T::to_f32(t.v[u]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < N; ++u) v[u] = c + u < cols ? T::to_f32(row[c + u]) : 0.0f;
    }
}
template <class T, int N>
__device__ __forceinline__ void store_cols(typename T::Store *row, uint32_t c, uint32_t cols, const float (&v)[N]) {
    constexpr int kVec = N * int(sizeof(typename T::Store)) <= 16 ? N : 16 / int(sizeof(typename T::Store));
    if (c + N <= cols) {
#pragma unroll
        for (int k = 0; k < N; k += kVec) {
            Pack<typename T::Store, kVec> t;
#pragma unroll
            for (int u = 0; u < kVec; ++u) t.v[u] = T::from_f32(v[k + u]);
            *reinterpret_cast<Pack<typename T::Store, kVec> *>(row + c + k) = t;
        }
    } else {
#pragma unroll
        for (int u = 0; u < N; ++u)
            if (c + u < cols) row[c + u] = T::from_f32(v[u]);
    }
}

// Zeros to elements [e0, e0 + 4) of a chunk.  Stored in the cache: with a batch
// of 200 tokens 27 us at 205 MB, a plain fill's time, where non-temporal stores
// took 37; 106 at 600 MB where they took 110.
__device__ __forceinline__ void clear4(BufRsrc r, uint32_t e0) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{0, 0, 0, 0}, r, static_cast<int>(e0 * 4u), 0, 0);
}

// A token's row, or `rows` for one outside [0, rows): padding.
template <class Tok>
__device__ __forceinline__ uint32_t token_key(const Tok *tokens, uint64_t i, uint32_t rows) {
    const int64_t t = static_cast<int64_t>(tokens[i]);
    return t >= 0 && t < static_cast<int64_t>(rows) ? static_cast<uint32_t>(t) : rows;
}

// ------------------------------------------------------------------ lookup
// A flat grid over the groups of kLookupCols columns of all tokens: kLookupVecs per
// thread, a workgroup's stride apart, all loads issued before the first
// store.  Memory bounds it: 32,768 tokens by 4,096 columns to bf16 take 92 us,
// 4.9 TB/s over the distinct rows read and y written, a large copy's rate.  At 700 tokens
// by 1,500 columns 4 us, a launch's own time.
constexpr int kLookupVecs = 4;
template <class T>
constexpr int kLookupCols = 16 / int(sizeof(typename T::Store));  // 16 bytes of y

template <class T, class Tok>
__global__ __launch_bounds__(kBlock) void embed_lookup_kernel(const float *__restrict__ w, const Tok *__restrict__ tokens,
                                                              uint64_t ntok, uint32_t rows, uint32_t cols,
                                                              uint32_t vecs, float scale,
                                                              typename T::Store *__restrict__ y, uint64_t ystride) {
    constexpr int N = kLookupCols<T>;
    const uint64_t first = static_cast<uint64_t>(blockIdx.x) * (kBlock * kLookupVecs);
    const uint64_t tok0 = first / vecs;
    const uint32_t rem0 = static_cast<uint32_t>(first - tok0 * vecs);
    float v[kLookupVecs][N], s[kLookupVecs];  // padding: +0 times +0, whatever the scale's sign
    uint64_t at[kLookupVecs];
    uint32_t col[kLookupVecs];
#pragma unroll
    for (int j = 0; j < kLookupVecs; ++j) {
        const uint32_t r = rem0 + threadIdx.x + j * kBlock;  // vecs < 2^30: no wrap
        const uint32_t dt = r / vecs;
        at[j] = tok0 + dt;
        col[j] = (r - dt * vecs) * N;
#pragma unroll
        for (int u = 0; u < N; ++u) v[j][u] = 0.0f;
        s[j] = 0.0f;
        if (at[j] < ntok) {
            const uint32_t key = token_key(tokens, at[j], rows);
            s[j] = key < rows ? scale : 0.0f;
            if (key < rows) load_cols<F32, N>(w + static_cast<uint64_t>(key) * cols, col[j], cols, v[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < kLookupVecs; ++j) {
        if (at[j] < ntok) {
#pragma unroll
            for (int u = 0; u < N; ++u) v[j][u] = s[j] * v[j][u];
            store_cols<T, N>(y + at[j] * ystride, col[j], cols, v[j]);
        }
    }
}

// -------------------------------------------------------------------- sort
// Tokens ranked together: a batch of up to kOneTile at once, which needs no
// merge; longer ones in tiles of kTile.  (Whole calls at 100 columns: 23.2 us
// in one tile against 24.0 merged at 6,000 tokens, 26.2 against 24.6 at 8,192.)
constexpr uint32_t kTile = 2048, kOneTile = 6144;
static_assert(kTile % kWave == 0 && kOneTile % kWave == 0, "64 tokens of a workgroup lie in one tile");
constexpr int kRankThreads = 1024; // 16 waves: 64 tokens, each wave a 16th of the tile's keys
constexpr uint32_t kRankWaves = kRankThreads / kWave;
constexpr uint32_t kWays = 16;     // runs merged at a time

// Crossing runs, listed by the sum for the join: blocks whose last run goes
// on, those of more than kJoinWaves partial sums apart.
struct Lists {
    uint32_t *count;  // [2]: short, long
    uint2 *few, *many;  // block, row
};

// Workgroup x ranks tokens [64 x, 64 x + 64) inside their tile; workgroups
// from `nrank` on clear the dense gradient meanwhile (nfill > 0), 16 x 1024
// elements each.  A row that has tokens is written again by the sum, one
// launch later.  kSet is the tokens ranked together.  LDS reads bound it, one
// of 16 bytes for 4 comparisons of a wave's 64 tokens: 8 us at 32,000 tokens
// in tiles of kTile; with the clearing of 15 M elements 11 us.  (Half of the
// clearing beside the sum instead, with the rows that have a token left out:
// 19.6 us against 18.7 at 700 tokens into 10,000 x 1,500, 29 against 24 at 3,000.)
template <class Tok, uint32_t kSet>
__global__ __launch_bounds__(kRankThreads) void embed_rank_kernel(const Tok *__restrict__ tokens, uint32_t n,
                                                                  uint32_t rows, uint32_t *__restrict__ key_out,
                                                                  uint32_t *__restrict__ pos_out, uint32_t *list_count,
                                                                  uint32_t nrank, float *__restrict__ fill,
                                                                  uint64_t nfill) {
    if (blockIdx.x >= nrank) {
        const uint64_t base = static_cast<uint64_t>(blockIdx.x - nrank) * (kRankThreads * 16);
        const BufRsrc r = chunk_buf(fill + base, static_cast<uint32_t>(umin64(nfill - base, kRankThreads * 16)));
#pragma unroll
        for (int j = 0; j < 4; ++j) clear4(r, (j * kRankThreads + threadIdx.x) * 4);
        return;
    }
    if (blockIdx.x == 0 && threadIdx.x < 2) list_count[threadIdx.x] = 0;
    __shared__ uint32_t keys[kSet];
    __shared__ uint32_t part[kRankWaves][kWave];
    const uint32_t i0 = blockIdx.x * kWave;
    const uint32_t t0 = i0 / kSet * kSet;
    const uint32_t cnt = min(n - t0, kSet);
    const uint32_t cnt4 = (cnt + 3u) & ~3u;
    for (uint32_t j = threadIdx.x; j < cnt4; j += kRankThreads)
        keys[j] = j < cnt ? token_key(tokens, t0 + j, rows) : 0xFFFFFFFFu;  // above every key
    __syncthreads();
    const uint32_t l0 = i0 - t0, li = l0 + lane_id();  // this lane's token inside the tile
    const bool have = li < cnt;
    const uint32_t key = have ? keys[li] : 0u;
    const uint32_t w = wave_id();
    // wave w counts over its 16th of the tile's keys, in groups of 4: <= key
    // in front of the 64 tokens, < key behind them, by position among them
    const uint32_t groups = cnt4 / 4, per = (groups + kRankWaves - 1) / kRankWaves;
    const uint32_t g0 = min(w * per, groups), g1 = min(g0 + per, groups);
    const uint32_t a = min(max(l0 / 4, g0), g1), b = min(max(l0 / 4 + kWave / 4, g0), g1);
    uint32_t below = 0;
    auto count = [&](uint32_t from, uint32_t to, uint32_t limit) {
#pragma unroll 4
        for (uint32_t g = from; g < to; ++g) {
            const uint4 k = *reinterpret_cast<const uint4 *>(&keys[4 * g]);
            below += k.x < limit;
            below += k.y < limit;
            below += k.z < limit;
            below += k.w < limit;
        }
    };
    count(g0, a, key + 1);
    for (uint32_t g = a; g < b; ++g) {
        const uint4 k = *reinterpret_cast<const uint4 *>(&keys[4 * g]);
        const uint32_t j = 4 * g;
        below += k.x < key + (j < li);
        below += k.y < key + (j + 1 < li);
        below += k.z < key + (j + 2 < li);
        below += k.w < key + (j + 3 < li);
    }
    count(b, g1, key);
    part[w][lane_id()] = below;
    __syncthreads();
    if (w == 0 && have) {
        uint32_t rank = 0;
#pragma unroll
        for (uint32_t v = 0; v < kRankWaves; ++v) rank += part[v][lane_id()];
        key_out[t0 + rank] = key;
        pos_out[t0 + rank] = t0 + li;
    }
}

// Workgroup x: 256 consecutive elements of one run, which are sorted, with
// first key kmin and last kmax.  In each of the other runs of its group, four
// bounds (keys below kmin, up to kmin, below kmax, up to kmax) place the
// elements equal to either, however many there are; the others are placed
// between the two inner bounds, whose keys fit LDS unless a run is much denser
// there.  What bounds this is latency: wave b takes run b, 64 probes cut its
// range to a 64th, and each element's 16 searches are spread over 4 threads.
// (The code is kept short for the same reason: with the 16 runs unrolled it
// took 20 to 24 us at 16,000 to 32,000 tokens, most of them instruction
// fetches; as it stands 9 to 11.)
constexpr int kMergeThreads = 1024;
constexpr uint32_t kMergeElems = 256;
constexpr uint32_t kMergeKeys = 512;  // keys of one other run held in LDS
constexpr uint32_t kMergeParts = kMergeThreads / kMergeElems;
static_assert(kTile % kMergeElems == 0, "a workgroup's elements lie in one run");
static_assert(kMergeThreads / kWave == int(kWays), "one wave per run");

__global__ __launch_bounds__(kMergeThreads) void embed_merge_kernel(const uint32_t *__restrict__ key_in,
                                                                    const uint32_t *__restrict__ pos_in, uint32_t n,
                                                                    uint32_t run, uint32_t *__restrict__ key_out,
                                                                    uint32_t *__restrict__ pos_out) {
    __shared__ uint32_t bound[kWays][4];
    __shared__ uint32_t between[kWays][kMergeKeys];
    __shared__ uint32_t places[kMergeParts][kMergeElems];
    const uint32_t e0 = blockIdx.x * kMergeElems;
    const uint32_t mine = e0 / run, g0 = mine / kWays * kWays;
    const uint32_t cnt = min(n - e0, kMergeElems);
    const uint32_t e = threadIdx.x % kMergeElems, q = threadIdx.x / kMergeElems;
    const uint32_t i = e0 + min(e, cnt - 1);
    const uint32_t key = key_in[i], pos = pos_in[i];
    const uint32_t kmin = key_in[e0], kmax = key_in[e0 + cnt - 1];
    auto run_start = [&](uint32_t b) { return static_cast<uint32_t>(umin64(static_cast<uint64_t>(g0 + b) * run, n)); };
    {
        const uint32_t b = __builtin_amdgcn_readfirstlane(wave_id());
        const uint32_t start = run_start(b), size = g0 + b == mine ? 0 : run_start(b + 1) - start;
        uint32_t lo[4], len[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            lo[t] = start;
            len[t] = size;
        }
        for (uint32_t longest = size; longest;) {
            uint32_t k[4];
            // probe l: the last key of the l-th 64th, of the range's last piece past its end
#pragma unroll
            for (int t = 0; t < 4; ++t)
                k[t] = len[t] ? key_in[lo[t] + min((lane_id() + 1) * ((len[t] + kWave - 1) / kWave), len[t]) - 1] : 0u;
            longest = 0;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint32_t limit = (t < 2 ? kmin : kmax) + (t & 1);
                const uint32_t step = (len[t] + kWave - 1) / kWave, hi = lo[t] + len[t];
                const uint32_t pieces = static_cast<uint32_t>(__popcll(__ballot(k[t] < limit)));
                if (len[t]) {
                    lo[t] = static_cast<uint32_t>(umin64(lo[t] + static_cast<uint64_t>(pieces) * step, hi));
                    len[t] = step == 1 ? 0 : min(step, hi - lo[t]);
                }
                longest = max(longest, len[t]);
            }
        }
        const uint32_t inner = kmin < kmax ? lo[2] - lo[1] : 0;
        for (uint32_t j = lane_id(); j < min(inner, kMergeKeys); j += kWave) between[b][j] = key_in[lo[1] + j];
        const uint32_t l = lane_id();
        if (l < 4) bound[b][l] = (l == 0 ? lo[0] : l == 1 ? lo[1] : l == 2 ? lo[2] : lo[3]) - start;
    }
    __syncthreads();
    uint32_t rank = 0;
    for (uint32_t b = q * (kWays / kMergeParts); b < (q + 1) * (kWays / kMergeParts); ++b) {
        if (g0 + b == mine) continue;
        const uint32_t before = g0 + b < mine ? 1 : 0;  // equal keys of earlier runs come first
        const uint32_t first = bound[b][1], inner = kmin < kmax ? bound[b][2] - first : 0;
        uint32_t lo = 0;
        if (inner <= kMergeKeys) {
            for (uint32_t half = kMergeKeys; half; half >>= 1)
                if (lo + half <= inner && between[b][lo + half - 1] < key + before) lo += half;
        } else {
            uint32_t hi = inner;
            while (lo < hi) {
                const uint32_t mid = (lo + hi) / 2;
                if (key_in[run_start(b) + first + mid] < key + before) lo = mid + 1;
                else hi = mid;
            }
        }
        rank += key == kmin ? bound[b][before] : key == kmax ? bound[b][2 + before] : first + lo;
    }
    places[q][e] = rank;
    __syncthreads();
    if (threadIdx.x >= cnt) return;
    rank = i - mine * run;
#pragma unroll
    for (uint32_t p = 0; p < kMergeParts; ++p) rank += places[p][e];
    const uint64_t to = static_cast<uint64_t>(g0) * run + rank;
    key_out[to] = key;
    pos_out[to] = pos;
}

// ------------------------------------------------------- distinct rows
// A head is a sorted position whose row differs from the one before it.
// heads_before[b] is the number of heads in front of block b of kSpan sorted
// positions, which places the block's rows in a message.
constexpr uint32_t kSpan = 16;
constexpr uint32_t kHeadTile = 4096;
constexpr int kHeadThreads = 1024;

__device__ __forceinline__ bool is_head(const uint32_t *key, uint32_t q, uint32_t rows) {
    const uint32_t k = key[q];
    return k < rows && (q == 0 || key[q - 1] != k);
}

// Long batches only: the heads of each tile.
constexpr uint32_t kCountTiles = 16;  // up to this many tiles every workgroup counts those before it itself

__global__ __launch_bounds__(kHeadThreads) void embed_heads_kernel(const uint32_t *__restrict__ key, uint32_t n,
                                                                   uint32_t rows, uint32_t *__restrict__ tile_heads) {
    uint32_t c = 0;
#pragma unroll
    for (uint32_t j = 0; j < kHeadTile / kHeadThreads; ++j) {
        const uint64_t q = static_cast<uint64_t>(blockIdx.x) * kHeadTile + j * kHeadThreads + threadIdx.x;
        c += q < n && is_head(key, static_cast<uint32_t>(q), rows) ? 1u : 0u;
    }
    uint32_t total;
    (void)block_exclusive_scan<uint32_t, kHeadThreads>(c, &total);
    if (threadIdx.x == 0) tile_heads[blockIdx.x] = total;
}

// Workgroup x places tile x (tile_heads null: it counts the heads in front
// of its tile first, which spares a launch); the last one writes the message's
// offsets.  Latency bounds it: 16,383 tokens take 5 to 6 us.
__global__ __launch_bounds__(kHeadThreads) void embed_rows_kernel(const uint32_t *__restrict__ key, uint32_t n,
                                                                  uint32_t rows, uint32_t cols,
                                                                  const uint32_t *__restrict__ tile_heads,
                                                                  uint32_t *__restrict__ heads_before,
                                                                  uint32_t *__restrict__ seg_off, int nseg, int seg) {
    uint32_t before = 0, total;
    if (tile_heads) {
        for (uint32_t t = threadIdx.x; t < blockIdx.x; t += kHeadThreads) before += tile_heads[t];
    } else {
#pragma unroll 4
        for (uint32_t q = 4 * threadIdx.x; q < blockIdx.x * kHeadTile; q += 4 * kHeadThreads) {
            const uint4 k = *reinterpret_cast<const uint4 *>(key + q);  // workspace arrays are 256-byte aligned
            const uint32_t p = q ? key[q - 1] : ~k.x;
            before += (k.x < rows && k.x != p) + (k.y < rows && k.y != k.x) + (k.z < rows && k.z != k.y) +
                      (k.w < rows && k.w != k.z);
        }
    }
    (void)block_exclusive_scan<uint32_t, kHeadThreads>(before, &total);
    before = total;
    // thread t owns 4 consecutive positions of the tile; 4 threads a block
    const uint64_t q0 = static_cast<uint64_t>(blockIdx.x) * kHeadTile + 4u * threadIdx.x;
    uint32_t c = 0;
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u)
        c += q0 + u < n && is_head(key, static_cast<uint32_t>(q0 + u), rows) ? 1u : 0u;
    const uint32_t ex = block_exclusive_scan<uint32_t, kHeadThreads>(c, &total);
    if (q0 < n && q0 % kSpan == 0) heads_before[q0 / kSpan] = before + ex;
    if (blockIdx.x == gridDim.x - 1)
        for (int s = threadIdx.x; s <= nseg; s += kHeadThreads) seg_off[s] = s <= seg ? 0u : (before + total) * cols;
}

// --------------------------------------------------------------------- sum
// Where a row's sum goes.
struct SumOut {
    float *g;          // dense or added: the embedding's rows; null for a message
    uint32_t *idx;     // message entries
    float *val;
    const uint32_t *heads_before;
    uint32_t idx0;     // flat index of the embedding's first element
    int add;
};

// What a row's sum is added to, loaded before the row's own loads are waited
// for (added gradients only).
template <int N>
__device__ __forceinline__ void old_row(const SumOut &o, uint32_t row, uint32_t c, uint32_t cols, float (&old)[N]) {
    if (o.g && o.add && c < cols) load_cols<F32, N>(o.g + static_cast<uint64_t>(row) * cols, c, cols, old);
}

template <int N>
__device__ __forceinline__ void put_row(const SumOut &o, uint32_t row, uint32_t rank, uint32_t c, uint32_t cols,
                                        float scale, const float (&acc)[N], const float (&old)[N]) {
    if (c >= cols) return;
    float v[N];
#pragma unroll
    for (int u = 0; u < N; ++u) v[u] = scale * acc[u];
    if (o.g) {
        float *p = o.g + static_cast<uint64_t>(row) * cols;
        if (o.add) {
#pragma unroll
            for (int u = 0; u < N; ++u) v[u] = old[u] + v[u];
        }
        store_cols<F32, N>(p, c, cols, v);
    } else {
        const uint64_t at = static_cast<uint64_t>(rank) * cols;
        store_cols<F32, N>(o.val + at, c, cols, v);
        const uint32_t i0 = o.idx0 + row * cols + c;
        if (c + N <= cols) {
#pragma unroll
            for (uint32_t k = 0; k < N; k += 4)
                *reinterpret_cast<Pack<uint32_t, 4> *>(o.idx + at + c + k) = Pack<uint32_t, 4>{{i0 + k, i0 + k + 1, i0 + k + 2, i0 + k + 3}};
        } else {
#pragma unroll
            for (uint32_t u = 0; u < N; ++u)
                if (c + u < cols) o.idx[at + c + u] = i0 + u;
        }
    }
}

// Workgroup (block b of kSpan sorted positions, slab of 256 columns).  A
// piece is a run's part of the block: wave w takes the block's pieces w,
// w + waves, ... and adds each one's rows in order.  part[2 b] holds the sum of
// a run that comes from the block before, part[2 b + 1] of one that begins
// here and goes on; the latter is listed for the join.
// Memory bounds it: 32,000 rows of 1,500 fp16 columns added to g take 37 us, of
// 32 that the bytes of dy and g need at a large copy's rate.
// The body is one short loop: unrolled over the 16 positions it ran 3 times
// longer at 20 tokens and 4 times at 32,000, for its instruction fetches.
// Each lane has 4 columns in every type: the sums leave in fp32, 16 bytes a
// lane next to each other; with 8 columns of a 16-bit dy the two stores of a
// lane took 27 us where fp32's took 22, on twice the bytes read.
constexpr uint32_t kJoinWaves = 16;
constexpr int kLaneCols = 4;
constexpr uint32_t kSlab = kWave * kLaneCols;

// acc += rows dy[pos[l]] for lanes l in [from, to) of the wave's lpos.  Two
// rows ahead: one took 43 us at 32,000 tokens by 1,500 fp16 columns where two
// take 37, eight 40 (most pieces are a row or two).
template <class T>
__device__ __forceinline__ void add_rows(const typename T::Store *__restrict__ dy, uint64_t stride, uint32_t lpos,
                                         uint32_t from, uint32_t to, uint32_t c, uint32_t cols,
                                         float (&acc)[kLaneCols]) {
    constexpr int N = kLaneCols, kAhead = 2;
    for (uint32_t j = from; j < to; j += kAhead) {
        float v[kAhead][N];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const uint32_t p = __builtin_amdgcn_readlane(lpos, min(j + a, to - 1));
            if (c < cols && j + a < to) load_cols<T, N>(dy + p * stride, c, cols, v[a]);
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            if (j + a < to)
#pragma unroll
                for (int u = 0; u < N; ++u) acc[u] = acc[u] + v[a][u];
    }
}

template <class T>
__global__ __launch_bounds__(1024) void embed_sum_kernel(const typename T::Store *__restrict__ dy, uint64_t stride,
                                                         const uint32_t *__restrict__ key,
                                                         const uint32_t *__restrict__ pos, uint32_t n, uint32_t rows,
                                                         uint32_t cols, uint32_t slabs, float scale, SumOut out,
                                                         float *__restrict__ part, uint32_t ldpart, Lists lists) {
    constexpr int N = kLaneCols;
    const uint32_t waves = blockDim.x / kWave, w = __builtin_amdgcn_readfirstlane(wave_id());
    const uint32_t b = blockIdx.x / slabs, slab = blockIdx.x - b * slabs;
    const uint32_t c = (slab * kWave + lane_id()) * N;
    const uint32_t q0 = b * kSpan, cnt = min(n - q0, kSpan);
    const uint32_t l = min(static_cast<uint32_t>(lane_id()), cnt - 1);
    const uint32_t lkey = key[q0 + l], lpos = pos[q0 + l];
    const uint32_t prev = q0 > 0 ? key[q0 - 1] : 0xFFFFFFFFu;
    const uint32_t next = q0 + cnt < n ? key[q0 + cnt] : 0xFFFFFFFFu;
    const uint32_t rank0 = out.g ? 0u : out.heads_before[b];
    // lanes at which a piece begins; padding is none
    const uint32_t lbefore = __shfl_up(lkey, 1, kWave);
    uint32_t starts = static_cast<uint32_t>(__ballot(lane_id() < int(cnt) && lkey < rows && (lane_id() == 0 || lbefore != lkey)));
    const bool from_before = prev == static_cast<uint32_t>(__builtin_amdgcn_readlane(lkey, 0));
    const uint32_t live = static_cast<uint32_t>(__popcll(__ballot(lane_id() < int(cnt) && lkey < rows)));  // padding sorts last
    for (uint32_t p = 0; starts; ++p) {
        const uint32_t from = static_cast<uint32_t>(__builtin_ctz(starts));
        starts &= starts - 1;
        if (p % waves != w) continue;
        const uint32_t to = starts ? static_cast<uint32_t>(__builtin_ctz(starts)) : live;
        const uint32_t k = __builtin_amdgcn_readlane(lkey, from);
        float acc[N], old[N];
        old_row(out, k, c, cols, old);
#pragma unroll
        for (int u = 0; u < N; ++u) acc[u] = 0.0f;
        add_rows<T>(dy, stride, lpos, from, to, c, cols, acc);
        const bool goes_on = to == cnt && next == k, comes = from_before && p == 0;
        if (comes || goes_on) {
            if (c < cols) store_cols<F32, N>(part + (2ull * b + (comes ? 0 : 1)) * ldpart, c, cols, acc);
            if (!comes && slab == 0 && lane_id() == 0) {
                // more than kJoinWaves partials: the run still holds position kJoinWaves blocks on
                const uint64_t far = q0 + static_cast<uint64_t>(kJoinWaves) * kSpan;
                const bool many = far < n && key[far] == k;
                (many ? lists.many : lists.few)[atomicAdd(&lists.count[many ? 1 : 0], 1u)] = make_uint2(b, k);
            }
        } else {
            put_row(out, k, rank0 + p - (from_before ? 1 : 0), c, cols, scale, acc, old);
        }
    }
}

// A batch of at most kSmall tokens in one launch.  Every workgroup of 16
// waves ranks the batch for itself in LDS; workgroup (group g of 16 runs, slab)
// sums a run per wave, block by block of 16 sorted positions as the other
// path's partial sums (at most 16 blocks, so they are added in order); the
// workgroups behind them clear the rows that have no token (dense).  Latency
// bounds it: 20 tokens by 1,500 columns take 5 us, where the other path's four
// launches took 13.
constexpr uint32_t kSmall = 256;
constexpr int kSmallThreads = 1024;
constexpr uint32_t kSmallWaves = kSmallThreads / kWave;
constexpr uint32_t kFill = kSmallThreads * 16;  // elements cleared per workgroup
static_assert(kFill / 32 < kSmallThreads, "a thread per word of held rows");
static_assert(kSmall <= kSpan * kJoinWaves, "a run of a small batch has at most kJoinWaves partial sums");

template <class T, class Tok>
__global__ __launch_bounds__(kSmallThreads) void embed_small_kernel(const typename T::Store *__restrict__ dy,
                                                                    uint64_t stride, const Tok *__restrict__ tokens,
                                                                    uint32_t n, uint32_t rows, uint32_t cols,
                                                                    uint32_t slabs, uint32_t nsum, float scale,
                                                                    SumOut out, uint64_t fill,
                                                                    uint32_t *__restrict__ seg_off, int nseg, int seg) {
    constexpr int N = kLaneCols;
    constexpr uint32_t kParts = kSmallThreads / kSmall;
    __shared__ uint32_t raw[kSmall], key[kSmall + 1], pos[kSmall], part[kParts][kSmall], run_at[kSmall + 1], nruns, live;
    const uint32_t t = threadIdx.x, e = t % kSmall, q = t / kSmall;
    if (blockIdx.x >= nsum) {
        // 16 elements per thread of rows without a token; `held` marks those
        // with one among the rows of this workgroup's elements
        const uint64_t base = static_cast<uint64_t>(blockIdx.x - nsum) * kFill;
        const uint32_t cnt = static_cast<uint32_t>(umin64(fill - base, kFill));
        const BufRsrc r = chunk_buf(out.g + base, cnt);
        const uint32_t r0 = static_cast<uint32_t>(base / cols), rem = static_cast<uint32_t>(base - static_cast<uint64_t>(r0) * cols);
        const uint32_t span = (rem + cnt - 1) / cols + 1;  // rows, at most kFill + 1
        __shared__ uint32_t held[kFill / 32 + 1];
        __shared__ uint32_t any;
        if (t <= kFill / 32) held[t] = 0;
        if (t == 0) any = 0;
        __syncthreads();
        if (t < n) {
            const uint32_t k = token_key(tokens, t, rows);
            if (k < rows && k - r0 < span) {
                atomicOr(&held[(k - r0) / 32], 1u << ((k - r0) % 32));
                any = 1;
            }
        }
        __syncthreads();
        if (!any) {
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) clear4(r, (j * kSmallThreads + t) * 4);
            return;
        }
        for (uint32_t x = t; x < cnt; x += kSmallThreads) {
            const uint32_t row = (rem + x) / cols;
            if (!(held[row / 32] >> (row % 32) & 1)) out.g[base + x] = 0.0f;
        }
        return;
    }
    if (t < kSmall) raw[t] = t < n ? token_key(tokens, t, rows) : 0xFFFFFFFFu;
    if (t == 0) key[n] = 0xFFFFFFFFu;
    __syncthreads();
    {
        // rank of token e: thread q of its 4 compares it with a quarter of the batch
        const uint32_t mine = raw[e], n4 = (n + 3) / 4, per = (n4 + kParts - 1) / kParts;
        uint32_t below = 0;
        for (uint32_t g = q * per; g < min((q + 1) * per, n4); ++g) {
            const uint4 k = *reinterpret_cast<const uint4 *>(&raw[4 * g]);
            const uint32_t j = 4 * g;
            below += k.x < mine + (j < e);
            below += k.y < mine + (j + 1 < e);
            below += k.z < mine + (j + 2 < e);
            below += k.w < mine + (j + 3 < e);
        }
        part[q][e] = below;
    }
    __syncthreads();
    if (t < n) {
        uint32_t rank = 0;
#pragma unroll
        for (uint32_t p = 0; p < kParts; ++p) rank += part[p][t];
        key[rank] = raw[t];
        pos[rank] = t;
    }
    __syncthreads();
    // the runs' first positions, and the end of the last
    {
        const bool in = t < n && key[t] < rows, head = in && (t == 0 || key[t - 1] != key[t]);
        uint32_t total;
        const uint32_t at = block_exclusive_scan<uint32_t, kSmallThreads>(head ? 1u : 0u, &total);
        if (head) run_at[at] = t;
        if (t < n && (in && (t + 1 == n || key[t + 1] >= rows))) live = t + 1;
        if (t == 0) {
            nruns = total;
            if (total == 0) live = 0;
        }
    }
    __syncthreads();
    const uint32_t runs = nruns;
    if (seg_off && blockIdx.x == 0)
        for (int s = t; s <= nseg; s += kSmallThreads) seg_off[s] = s <= seg ? 0u : runs * cols;
    const uint32_t g = blockIdx.x / slabs, slab = blockIdx.x - g * slabs;
    const uint32_t c = (slab * kWave + lane_id()) * N;
    const uint32_t r = g * kSmallWaves + __builtin_amdgcn_readfirstlane(wave_id());
    if (r >= runs) return;
    const uint32_t from = run_at[r], to = r + 1 < runs ? run_at[r + 1] : live;
    float sum[N], old[N];
    old_row(out, key[from], c, cols, old);
    for (uint32_t b = from / kSpan; b * kSpan < to; ++b) {
        const uint32_t q0 = b * kSpan, lo = max(from, q0) - q0, hi = min(to, q0 + kSpan) - q0;
        const uint32_t lpos = pos[min(q0 + (lane_id() & (kSpan - 1)), n - 1)];
        float acc[N];
#pragma unroll
        for (int u = 0; u < N; ++u) acc[u] = 0.0f;
        add_rows<T>(dy, stride, lpos, __builtin_amdgcn_readfirstlane(lo), __builtin_amdgcn_readfirstlane(hi), c, cols, acc);
#pragma unroll
        for (int u = 0; u < N; ++u) sum[u] = b == from / kSpan ? acc[u] : sum[u] + acc[u];
    }
    put_row(out, key[from], r, c, cols, scale, sum, old);
}

// The partial sums of the listed runs: part[2 b + 1], then part[2 (b + i)].
// Runs of at most kJoinWaves partials take a wave each and are added in
// order; for longer ones wave w of a workgroup adds partials w, w + 16, ...,
// and then the 16 sums are added in wave order.  Latency bounds it, of the
// longest run's partials: 11 us at 32,000 tokens by 1,500 columns, 4 at 700.
constexpr int kJoinThreads = kJoinWaves * kWave;

__device__ __forceinline__ uint32_t run_blocks(const uint32_t *__restrict__ key, uint32_t n, uint32_t b, uint32_t k) {
    const uint32_t nblocks = (n + kSpan - 1) / kSpan;
    uint32_t end = b + 1;
    for (;;) {
        const uint32_t bl = end + lane_id();
        const uint64_t m = __ballot(bl < nblocks && key[min(bl, nblocks - 1) * kSpan] == k);
        if (m != ~0ull) return end + static_cast<uint32_t>(__builtin_ctzll(~m)) - b;
        end += kWave;
    }
}

// The rank among the distinct rows of block b's last run, which begins there.
__device__ __forceinline__ uint32_t last_rank(const SumOut &out, const uint32_t *__restrict__ key, uint32_t rows,
                                              uint32_t b) {
    if (out.g) return 0;
    const uint32_t q = b * kSpan + min(static_cast<uint32_t>(lane_id()), kSpan - 1);
    const uint64_t heads = __ballot(lane_id() < int(kSpan) && is_head(key, q, rows));
    return out.heads_before[b] + static_cast<uint32_t>(__popcll(heads)) - 1;
}

// acc += partials first, first + step, ... of the run that begins in block b.
__device__ __forceinline__ void add_partials(const float *__restrict__ part, uint32_t ldpart, uint32_t b, uint32_t first,
                                             uint32_t step, uint32_t count, uint32_t c, uint32_t cols, float (&acc)[4]) {
    if (c >= cols) return;
#pragma unroll 4
    for (uint32_t i = first; i < count; i += step) {
        // the rows of part are padded to 4 columns, so their last lane reads whole vectors too
        const float4 v = *reinterpret_cast<const float4 *>(part + (2ull * (b + i) + (i == 0 ? 1 : 0)) * ldpart + c);
        acc[0] = acc[0] + v.x;
        acc[1] = acc[1] + v.y;
        acc[2] = acc[2] + v.z;
        acc[3] = acc[3] + v.w;
    }
}

__global__ __launch_bounds__(kJoinThreads) void embed_join_kernel(const uint32_t *__restrict__ key, uint32_t n,
                                                                  uint32_t rows, uint32_t cols, uint32_t slabs,
                                                                  float scale, SumOut out,
                                                                  const float *__restrict__ part, uint32_t ldpart,
                                                                  Lists lists) {
    __shared__ float4 sums[kJoinWaves][kWave];
    const uint32_t w = __builtin_amdgcn_readfirstlane(wave_id());
    const uint64_t nfew = static_cast<uint64_t>(lists.count[0]) * slabs, nmany = static_cast<uint64_t>(lists.count[1]) * slabs;
    for (uint64_t it = blockIdx.x; it < nmany; it += gridDim.x) {
        const uint32_t at = static_cast<uint32_t>(it / slabs);
        const uint32_t b = lists.many[at].x, k = lists.many[at].y;
        const uint32_t c = static_cast<uint32_t>(it - static_cast<uint64_t>(at) * slabs) * kSlab + 4u * lane_id();
        const uint32_t count = run_blocks(key, n, b, k);
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, old[4];
        old_row(out, k, c, cols, old);
        add_partials(part, ldpart, b, w, kJoinWaves, count, c, cols, acc);
        __syncthreads();  // the sums of the item before have been read
        sums[w][lane_id()] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        __syncthreads();
        if (w == 0) {
#pragma unroll 5
            for (uint32_t i = 1; i < kJoinWaves; ++i) {
                const float4 s = sums[i][lane_id()];
                acc[0] = acc[0] + s.x;
                acc[1] = acc[1] + s.y;
                acc[2] = acc[2] + s.z;
                acc[3] = acc[3] + s.w;
            }
            put_row(out, k, last_rank(out, key, rows, b), c, cols, scale, acc, old);
        }
    }
    // spread over the workgroups, from the last: the first ones had the long runs
    for (uint64_t it = static_cast<uint64_t>(w) * gridDim.x + (gridDim.x - 1 - blockIdx.x); it < nfew; it += static_cast<uint64_t>(gridDim.x) * kJoinWaves) {
        const uint32_t at = static_cast<uint32_t>(it / slabs);
        const uint32_t b = lists.few[at].x, k = lists.few[at].y;
        const uint32_t c = static_cast<uint32_t>(it - static_cast<uint64_t>(at) * slabs) * kSlab + 4u * lane_id();
        const uint32_t count = run_blocks(key, n, b, k);
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, old[4];
        old_row(out, k, c, cols, old);
        add_partials(part, ldpart, b, 0, 1, count, c, cols, acc);
        put_row(out, k, last_rank(out, key, rows, b), c, cols, scale, acc, old);
    }
}

// --------------------------------------------------------------- host side
constexpr uint64_t kMaxTokens = uint64_t(1) << 28;
constexpr uint64_t kMaxElems = uint64_t(1) << 35;
// Workgroups of a launch: a grid has fewer than 2^32 threads.
constexpr uint64_t max_grid(uint64_t threads) { return 0xFFFFFFFFull / threads; }

struct EmbedWs {
    uint32_t *key[2], *pos[2], *heads_before, *tile_heads;
    Lists lists;
    float *part;
    uint32_t ldpart;
    size_t bytes;
};

EmbedWs embed_ws(void *ws, uint64_t n, uint32_t cols) {
    WsCursor c(ws);
    EmbedWs w{};
    for (int k = 0; k < 2; ++k) {
        w.key[k] = c.take<uint32_t>(n);
        w.pos[k] = c.take<uint32_t>(n);
    }
    const uint64_t blocks = ceil_div(n, kSpan);
    w.heads_before = c.take<uint32_t>(blocks);
    w.tile_heads = c.take<uint32_t>(ceil_div(n, kHeadTile));
    w.lists.count = c.take<uint32_t>(2);
    w.lists.few = c.take<uint2>(blocks);
    w.lists.many = c.take<uint2>(blocks / kJoinWaves + 1);
    w.ldpart = (cols + 3u) & ~3u;
    w.part = c.take<float>(2 * blocks * w.ldpart);
    w.bytes = c.used + 256;  // room to round the base up to 256 bytes
    return w;
}

void *align256(void *p) {
    return reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(p) + 255) & ~uintptr_t(255));
}

// The embedding's shape inside the plan: GC_OK and its columns.
gc_status check_table(const char *fn, const gc_plan *plan, int seg, uint32_t rows, uint32_t *cols) {
    auto fail = [&](gc_status st, const char *what) { return set_error(st, std::string(fn) + ": " + what); };
    if (!plan) return fail(GC_EINVAL, "plan is null");
    if (seg < 0 || seg >= plan->nseg) return fail(GC_EINVAL, "seg is not a segment of the plan");
    const uint32_t len = plan->seg[seg].len;
    if (rows < 1 || len % rows) return fail(GC_EINVAL, "rows must divide the segment's length");
    *cols = len / rows;
    return GC_OK;
}

bool aligned4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

size_t type_bytes(int type) { return type == GC_F32 ? 4 : 2; }

gc_status check_batch(const char *fn, const void *tokens, int token_type, uint64_t n, const void *x, int type,
                      uint64_t stride, uint32_t cols, float scale) {
    auto fail = [&](gc_status st, const char *what) { return set_error(st, std::string(fn) + ": " + what); };
    if (token_type != GC_TOKENS_I32 && token_type != GC_TOKENS_I64)
        return fail(GC_EINVAL, "token_type must be GC_TOKENS_I32 or GC_TOKENS_I64");
    if (type != GC_F32 && type != GC_BF16 && type != GC_F16)
        return fail(GC_EINVAL, "type must be GC_F32, GC_BF16 or GC_F16");
    if (!(scale - scale == 0.0f)) return fail(GC_EINVAL, "scale must be finite");
    if (n >= kMaxTokens) return fail(GC_ERANGE, "n_tokens must be < 2^28");
    if (n * cols > kMaxElems) return fail(GC_ERANGE, "n_tokens * cols must be <= 2^35");
    if (n == 0) return GC_OK;
    if (!tokens || !x) return fail(GC_EINVAL, "buffers must be non-null");
    if (stride < cols) return fail(GC_EINVAL, "the row stride must be at least the columns");
    if (n > 1 && stride > (uint64_t(1) << 48) / n) return fail(GC_ERANGE, "n_tokens * stride must be <= 2^48");
    if (reinterpret_cast<uintptr_t>(tokens) % (token_type == GC_TOKENS_I32 ? 4 : 8) ||
        reinterpret_cast<uintptr_t>(x) % type_bytes(type))
        return fail(GC_EINVAL, "buffers must be aligned to their elements");
    return GC_OK;
}

// Calls f with the storage type's and the token type's tags.
template <class F>
void with_type(int type, F f) {
    if (type == GC_F32) f(F32{});
    else if (type == GC_BF16) f(BF16{});
    else f(F16{});
}
template <class F>
void with_tokens(int token_type, F f) {
    if (token_type == GC_TOKENS_I32) f(int32_t{});
    else f(int64_t{});
}

// Sorts and sums: everything behind the argument checks.  fill: floats to
// clear at `g` (dense), 0 otherwise.
gc_status embed_backward(const char *fn, const gc_plan *plan, int seg, uint32_t rows, uint32_t cols, const void *dy,
                         int type, uint64_t stride, const void *tokens, int token_type, uint64_t n64, float scale,
                         SumOut out, uint64_t fill, uint32_t *seg_off, void *ws, hipStream_t stream) {
    const uint32_t n = static_cast<uint32_t>(n64);
    EmbedWs w = embed_ws(align256(ws), n64, cols);
    const uint64_t nfill = ceil_div(fill, kRankThreads * 16), nrank = ceil_div(n, kWave);
    const uint32_t blocks = static_cast<uint32_t>(ceil_div(n, kSpan));
    const uint32_t slabs = static_cast<uint32_t>(ceil_div(cols, kSlab));
    const uint64_t sums = static_cast<uint64_t>(blocks) * slabs;
    const uint64_t nsum64 = ceil_div(n, kSmallWaves) * slabs;  // of a short batch
    if (n <= kSmall ? nsum64 + nfill > max_grid(kSmallThreads)
                    : nrank + nfill > max_grid(kRankThreads) || sums > max_grid(kBlock))
        return set_error(GC_ERANGE, std::string(fn) + ": more workgroups than a launch has");
    if (n <= kSmall) {
        const uint32_t nsum = static_cast<uint32_t>(nsum64);
        with_type(type, [&](auto t) {
            with_tokens(token_type, [&](auto tok) {
                using T = decltype(t);
                using Tok = decltype(tok);
                GC_LAUNCH("embed_small", stream,
                          embed_small_kernel<T, Tok><<<static_cast<unsigned>(nsum + nfill), kSmallThreads, 0, stream>>>(
                              static_cast<const typename T::Store *>(dy), stride, static_cast<const Tok *>(tokens), n,
                              rows, cols, slabs, nsum, scale, out, fill, seg_off, plan->nseg, seg));
            });
        });
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return hip_error(e, fn);
        return GC_OK;
    }
    with_tokens(token_type, [&](auto tok) {
        using Tok = decltype(tok);
        const auto kernel = n <= kOneTile ? embed_rank_kernel<Tok, kOneTile> : embed_rank_kernel<Tok, kTile>;
        GC_LAUNCH("embed_rank", stream,
                  kernel<<<static_cast<unsigned>(nrank + nfill), kRankThreads, 0, stream>>>(
                      static_cast<const Tok *>(tokens), n, rows, w.key[0], w.pos[0], w.lists.count,
                      static_cast<uint32_t>(nrank), out.g, fill));
    });
    int cur = 0;
    for (uint64_t run = n <= kOneTile ? kOneTile : kTile; run < n; run *= kWays) {
        GC_LAUNCH("embed_merge", stream,
                  embed_merge_kernel<<<grid_1d(n, kMergeElems), kMergeThreads, 0, stream>>>(
                      w.key[cur], w.pos[cur], n, static_cast<uint32_t>(run), w.key[cur ^ 1], w.pos[cur ^ 1]));
        cur ^= 1;
    }
    if (!out.g) {
        const unsigned tiles = grid_1d(n, kHeadTile);
        uint32_t *tile_heads = tiles > kCountTiles ? w.tile_heads : nullptr;
        if (tile_heads)
            GC_LAUNCH("embed_heads", stream,
                      embed_heads_kernel<<<tiles, kHeadThreads, 0, stream>>>(w.key[cur], n, rows, tile_heads));
        GC_LAUNCH("embed_rows", stream,
                  embed_rows_kernel<<<tiles, kHeadThreads, 0, stream>>>(w.key[cur], n, rows, cols, tile_heads,
                                                                      w.heads_before, seg_off, plan->nseg, seg));
        out.heads_before = w.heads_before;
    }
    // one piece per wave while the chip holds them all at once, else 4 waves a block
    const int threads = sums <= 512 ? 1024 : 256;
    with_type(type, [&](auto t) {
        using T = decltype(t);
        GC_LAUNCH("embed_sum", stream,
                  embed_sum_kernel<T><<<static_cast<unsigned>(sums), threads, 0, stream>>>(
                      static_cast<const typename T::Store *>(dy), stride, w.key[cur], w.pos[cur], n, rows, cols, slabs,
                      scale, out, w.part, w.ldpart, w.lists));
    });
    {
        const unsigned grid = static_cast<unsigned>(umin64(ceil_div(static_cast<uint64_t>(blocks - 1) * slabs, 2), 512));
        GC_LAUNCH("embed_join", stream,
                  embed_join_kernel<<<grid, kJoinThreads, 0, stream>>>(w.key[cur], n, rows, cols, slabs, scale, out,
                                                                     w.part, w.ldpart, w.lists));
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_error(e, fn);
    return GC_OK;
}

// An empty batch: nothing to sum, but the dense gradient is still cleared and
// the message still empty.
__global__ __launch_bounds__(kBlock) void embed_empty_kernel(float *g, uint64_t n, uint32_t *seg_off, int nseg) {
    const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kBlock + threadIdx.x;
    if (i < n) g[i] = 0.0f;
    if (seg_off && i <= static_cast<uint64_t>(nseg)) seg_off[i] = 0u;
}

}  // namespace
}  // namespace gc

using namespace gc;

extern "C" gc_status gc_embed_lookup(const gc_plan *plan, int seg, uint32_t rows, const float *w, const void *tokens,
                                     int token_type, uint64_t n_tokens, float scale, void *y, int y_type,
                                     uint64_t y_stride, hipStream_t stream) {
    clear_error();
    uint32_t cols = 0;
    gc_status st = check_table("gc_embed_lookup", plan, seg, rows, &cols);
    if (st != GC_OK) return st;
    st = check_batch("gc_embed_lookup", tokens, token_type, n_tokens, y, y_type, y_stride, cols, scale);
    if (st != GC_OK) return st;
    if (n_tokens == 0) return GC_OK;
    if (!w) return set_error(GC_EINVAL, "gc_embed_lookup: buffers must be non-null");
    if (!aligned4(w)) return set_error(GC_EINVAL, "gc_embed_lookup: buffers must be aligned to their elements");
    const uint32_t vecs = static_cast<uint32_t>(ceil_div(cols, y_type == GC_F32 ? kLookupCols<F32> : kLookupCols<BF16>));
    const uint64_t grid = ceil_div(n_tokens * vecs, kBlock * kLookupVecs);
    if (grid > max_grid(kBlock)) return set_error(GC_ERANGE, "gc_embed_lookup: more workgroups than a launch has");
    with_type(y_type, [&](auto t) {
        with_tokens(token_type, [&](auto tok) {
            using T = decltype(t);
            using Tok = decltype(tok);
            GC_LAUNCH("embed_lookup", stream,
                      embed_lookup_kernel<T, Tok><<<static_cast<unsigned>(grid), kBlock, 0, stream>>>(
                          w + plan->seg[seg].off, static_cast<const Tok *>(tokens), n_tokens, rows, cols, vecs, scale,
                          static_cast<typename T::Store *>(y), y_stride));
        });
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_error(e, "gc_embed_lookup launch");
    return GC_OK;
}

extern "C" size_t gc_embed_workspace_bytes(const gc_plan *plan, int seg, uint32_t rows, uint64_t n_tokens) {
    clear_error();
    uint32_t cols = 0;
    if (check_table("gc_embed_workspace_bytes", plan, seg, rows, &cols) != GC_OK) return 0;
    if (n_tokens >= kMaxTokens) return 0;
    return embed_ws(nullptr, n_tokens, cols).bytes;
}

extern "C" uint64_t gc_embed_message_cap(const gc_plan *plan, int seg, uint32_t rows, uint64_t n_tokens) {
    clear_error();
    uint32_t cols = 0;
    if (check_table("gc_embed_message_cap", plan, seg, rows, &cols) != GC_OK) return 0;
    return umin64(n_tokens, rows) * cols;
}

extern "C" gc_status gc_embed_grad(const gc_plan *plan, int seg, uint32_t rows, const void *dy, int dy_type,
                                   uint64_t dy_stride, const void *tokens, int token_type, uint64_t n_tokens,
                                   float scale, float *g, int accumulate, void *ws, size_t ws_bytes,
                                   hipStream_t stream) {
    clear_error();
    uint32_t cols = 0;
    gc_status st = check_table("gc_embed_grad", plan, seg, rows, &cols);
    if (st != GC_OK) return st;
    st = check_batch("gc_embed_grad", tokens, token_type, n_tokens, dy, dy_type, dy_stride, cols, scale);
    if (st != GC_OK) return st;
    if (!g) return set_error(GC_EINVAL, "gc_embed_grad: g must be non-null");
    if (!aligned4(g)) return set_error(GC_EINVAL, "gc_embed_grad: buffers must be aligned to their elements");
    if (n_tokens && !ws) return set_error(GC_EINVAL, "gc_embed_grad: ws must be non-null");
    if (n_tokens && ws_bytes < embed_ws(nullptr, n_tokens, cols).bytes)
        return set_error(GC_ECAPACITY, "gc_embed_grad: workspace smaller than gc_embed_workspace_bytes");
    const uint64_t fill = accumulate ? 0 : plan->seg[seg].len;
    float *rows_at = g + plan->seg[seg].off;
    if (n_tokens == 0) {
        if (fill)
            GC_LAUNCH("embed_empty", stream, embed_empty_kernel<<<grid_1d(fill, kBlock), kBlock, 0, stream>>>(
                                                 rows_at, fill, nullptr, 0));
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return hip_error(e, "gc_embed_grad launch");
        return GC_OK;
    }
    SumOut out{};
    out.g = rows_at;
    out.add = accumulate ? 1 : 0;
    return embed_backward("gc_embed_grad", plan, seg, rows, cols, dy, dy_type, dy_stride, tokens, token_type, n_tokens,
                          scale, out, fill, nullptr, ws, stream);
}

extern "C" gc_status gc_embed_message(const gc_plan *plan, int seg, uint32_t rows, const void *dy, int dy_type,
                                      uint64_t dy_stride, const void *tokens, int token_type, uint64_t n_tokens,
                                      float scale, gc_sparse *msg, void *ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    uint32_t cols = 0;
    gc_status st = check_table("gc_embed_message", plan, seg, rows, &cols);
    if (st != GC_OK) return st;
    st = check_batch("gc_embed_message", tokens, token_type, n_tokens, dy, dy_type, dy_stride, cols, scale);
    if (st != GC_OK) return st;
    if (!msg || !msg->seg_off || (n_tokens && (!msg->idx || !msg->val)))
        return set_error(GC_EINVAL, "gc_embed_message: out and its idx, val, seg_off must be non-null");
    if (!aligned4(msg->idx) || !aligned4(msg->val) || !aligned4(msg->seg_off))
        return set_error(GC_EINVAL, "gc_embed_message: buffers must be aligned to their elements");
    if (n_tokens && !ws) return set_error(GC_EINVAL, "gc_embed_message: ws must be non-null");
    if (msg->cap < umin64(n_tokens, rows) * cols)
        return set_error(GC_ECAPACITY, "gc_embed_message: out->cap smaller than gc_embed_message_cap");
    if (n_tokens && ws_bytes < embed_ws(nullptr, n_tokens, cols).bytes)
        return set_error(GC_ECAPACITY, "gc_embed_message: workspace smaller than gc_embed_workspace_bytes");
    if (n_tokens == 0) {
        GC_LAUNCH("embed_empty", stream, embed_empty_kernel<<<grid_1d(plan->nseg + 1, kBlock), kBlock, 0, stream>>>(
                                             nullptr, 0, msg->seg_off, plan->nseg));
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return hip_error(e, "gc_embed_message launch");
        return GC_OK;
    }
    SumOut out{};
    out.idx = msg->idx;
    out.val = msg->val;
    out.idx0 = static_cast<uint32_t>(plan->seg[seg].off);
    return embed_backward("gc_embed_message", plan, seg, rows, cols, dy, dy_type, dy_stride, tokens, token_type,
                          n_tokens, scale, out, 0, msg->seg_off, ws, stream);
}
