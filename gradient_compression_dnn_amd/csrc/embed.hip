// The embedding of a model's flat buffer: the scaled lookup of a batch of
// tokens (gc_embed_lookup) and its gradient by sorted tokens, dense or added
// (gc_embed_grad) or as a sparse message (gc_embed_message).
//
//   y_i  = round(fl32(scale * w[t_i]))
//   g[r] = fl32(scale * sum of dy_i over the positions i with t_i = r)
//
// The sum of a row takes its positions in ascending order, so positions are
// sorted by (row, position) first.  The sort is stable and makes no use of
// atomics, hence every sum has one order and the result one bit pattern:
//   rank   each tile of 4096 tokens is ranked by counting: the rank of i is
//          the number of keys below key_i, or equal and before i.  16.8 M
//          comparisons a tile, no pass over the tile has to wait for another.
//   merge  8 sorted runs at a time: an element's rank in the merged run is
//          its own plus, for each other run, a binary search.
//   sum    32 sorted positions by 256 columns per wave.  A row whose run lies
//          inside the block is finished there; a run that crosses blocks
//          leaves one partial sum per block.
//   join   the partial sums of each crossing run.
#include <algorithm>
#include <string>

#include "gc_internal.hpp"

namespace gc {

namespace {

// Accesses of 4 elements with the alignment of one: the hardware's unaligned
// mode takes them as one access, so odd offsets and strides need no variant.
struct __attribute__((packed, aligned(4))) F32x4 {
    float v[4];
};
struct __attribute__((packed, aligned(4))) U32x4 {
    uint32_t v[4];
};
struct __attribute__((packed, aligned(2))) U16x4 {
    uint16_t v[4];
};

struct F32 {
    using Store = float;
    using Vec = F32x4;
    static __device__ __forceinline__ float to_f32(float x) { return x; }
    static __device__ __forceinline__ float from_f32(float x) { return x; }
};
struct BF16 {
    using Store = uint16_t;
    using Vec = U16x4;
    static __device__ __forceinline__ float to_f32(uint16_t x) { return dev_u2f(uint32_t(x) << 16); }
    static __device__ __forceinline__ uint16_t from_f32(float x) {
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
    }
};
struct F16 {
    using Store = uint16_t;
    using Vec = U16x4;
    static __device__ __forceinline__ float to_f32(uint16_t x) {
        return static_cast<float>(__builtin_bit_cast(_Float16, x));
    }
    static __device__ __forceinline__ uint16_t from_f32(float x) {
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
    }
};

// 4 columns of a row from column c on; those at or past cols are 0 / dropped.
template <class T>
__device__ __forceinline__ void load_cols(const typename T::Store *row, uint32_t c, uint32_t cols, float (&v)[4]) {
    if (c + 4 <= cols) {
        const auto t = *reinterpret_cast<const typename T::Vec *>(row + c);
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = T::to_f32(t.v[u]);
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = c + u < cols ? T::to_f32(row[c + u]) : 0.0f;
    }
}
template <class T>
__device__ __forceinline__ void store_cols(typename T::Store *row, uint32_t c, uint32_t cols, const float (&v)[4]) {
    if (c + 4 <= cols) {
        typename T::Vec t;
#pragma unroll
        for (int u = 0; u < 4; ++u) t.v[u] = T::from_f32(v[u]);
        *reinterpret_cast<typename T::Vec *>(row + c) = t;
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (c + u < cols) row[c + u] = T::from_f32(v[u]);
    }
}

// A token's row, or `rows` for one outside [0, rows): padding.
template <class Tok>
__device__ __forceinline__ uint32_t token_key(const Tok *tokens, uint64_t i, uint32_t rows) {
    const int64_t t = static_cast<int64_t>(tokens[i]);
    return t >= 0 && t < static_cast<int64_t>(rows) ? static_cast<uint32_t>(t) : rows;
}

// ------------------------------------------------------------------ lookup
// A flat grid over the groups of 4 columns of all tokens: kLookupVecs per
// thread, a workgroup's stride apart, all loads issued before the first
// store.
constexpr int kLookupVecs = 4;

template <class T, class Tok>
__global__ __launch_bounds__(kBlock) void embed_lookup_kernel(const float *__restrict__ w, const Tok *__restrict__ tokens,
                                                              uint64_t ntok, uint32_t rows, uint32_t cols,
                                                              uint32_t vecs, float scale,
                                                              typename T::Store *__restrict__ y, uint64_t ystride) {
    const uint64_t first = static_cast<uint64_t>(blockIdx.x) * (kBlock * kLookupVecs);
    const uint64_t tok0 = first / vecs;
    const uint32_t rem0 = static_cast<uint32_t>(first - tok0 * vecs);
    float v[kLookupVecs][4];
    uint64_t at[kLookupVecs];
    uint32_t col[kLookupVecs];
#pragma unroll
    for (int j = 0; j < kLookupVecs; ++j) {
        const uint32_t r = rem0 + threadIdx.x + j * kBlock;  // vecs < 2^30: no wrap
        const uint32_t dt = r / vecs;
        at[j] = tok0 + dt;
        col[j] = (r - dt * vecs) * 4;
#pragma unroll
        for (int u = 0; u < 4; ++u) v[j][u] = 0.0f;
        if (at[j] < ntok) {
            const uint32_t key = token_key(tokens, at[j], rows);
            if (key < rows) load_cols<F32>(w + static_cast<uint64_t>(key) * cols, col[j], cols, v[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < kLookupVecs; ++j) {
        if (at[j] < ntok) {
#pragma unroll
            for (int u = 0; u < 4; ++u) v[j][u] = scale * v[j][u];
            store_cols<T>(y + at[j] * ystride, col[j], cols, v[j]);
        }
    }
}

// -------------------------------------------------------------------- sort
constexpr uint32_t kTile = 4096;   // tokens ranked together
constexpr int kRankThreads = 1024; // 16 waves: 64 tokens, each wave a 16th of the tile's keys
constexpr uint32_t kRankWaves = kRankThreads / kWave;
constexpr uint32_t kWays = 8;      // runs merged at a time

// Workgroup x ranks tokens [64 x, 64 x + 64) inside their tile; workgroups
// from `nrank` on clear the dense gradient meanwhile (nfill > 0), 4 x 1024
// threads' stores each.  A row that has tokens is written again by the sum,
// one launch later.
template <class Tok>
__global__ __launch_bounds__(kRankThreads) void embed_rank_kernel(const Tok *__restrict__ tokens, uint32_t n,
                                                                  uint32_t rows, uint32_t *__restrict__ key_out,
                                                                  uint32_t *__restrict__ pos_out, uint32_t nrank,
                                                                  float *__restrict__ fill, uint64_t nfill) {
    if (blockIdx.x >= nrank) {
        const uint64_t base = static_cast<uint64_t>(blockIdx.x - nrank) * (kRankThreads * 16);
        const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint64_t e = base + (static_cast<uint64_t>(j) * kRankThreads + threadIdx.x) * 4;
            if (e < nfill) store_cols<F32>(fill + e, 0, static_cast<uint32_t>(umin64(nfill - e, 4)), zero);
        }
        return;
    }
    __shared__ uint32_t keys[kTile];
    __shared__ uint32_t part[kRankWaves][kWave];
    const uint32_t i0 = blockIdx.x * kWave;
    const uint32_t t0 = i0 / kTile * kTile;
    const uint32_t cnt = min(n - t0, kTile);
    const uint32_t cnt4 = (cnt + 3u) & ~3u;
    for (uint32_t j = threadIdx.x; j < cnt4; j += kRankThreads)
        keys[j] = j < cnt ? token_key(tokens, t0 + j, rows) : 0xFFFFFFFFu;  // above every key
    __syncthreads();
    const uint32_t li = i0 - t0 + lane_id();  // this lane's token inside the tile
    const bool have = li < cnt;
    const uint32_t key = have ? keys[li] : 0u;
    const uint32_t w = wave_id();
    // wave w counts over its 16th of the tile's keys, in groups of 4
    const uint32_t groups = cnt4 / 4, per = (groups + kRankWaves - 1) / kRankWaves;
    const uint32_t g0 = min(w * per, groups), g1 = min(g0 + per, groups);
    uint32_t below = 0;
    for (uint32_t g = g0; g < g1; ++g) {
        const uint4 k = *reinterpret_cast<const uint4 *>(&keys[4 * g]);
        const uint32_t j = 4 * g;
        below += k.x < key || (k.x == key && j < li);
        below += k.y < key || (k.y == key && j + 1 < li);
        below += k.z < key || (k.z == key && j + 2 < li);
        below += k.w < key || (k.w == key && j + 3 < li);
    }
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

// One element per thread of sorted runs of `run` elements: its rank in the
// run merged from kWays of them.  Runs before its own count keys <= key,
// runs after it keys < key; the kWays searches advance together.
__global__ __launch_bounds__(kBlock) void embed_merge_kernel(const uint32_t *__restrict__ key_in,
                                                             const uint32_t *__restrict__ pos_in, uint32_t n,
                                                             uint64_t run, int steps, uint32_t *__restrict__ key_out,
                                                             uint32_t *__restrict__ pos_out) {
    const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kBlock + threadIdx.x;
    if (i >= n) return;
    const uint64_t mine = i / run, g0 = mine / kWays * kWays;
    const uint32_t key = key_in[i];
    // search b: the count of run g0 + b's elements that come before this one
    uint64_t lo[kWays], hi[kWays];
#pragma unroll
    for (uint32_t b = 0; b < kWays; ++b) {
        lo[b] = umin64((g0 + b) * run, n);
        hi[b] = umin64((g0 + b + 1) * run, n);
        if (g0 + b == mine) lo[b] = hi[b] = i;
    }
    for (int s = 0; s < steps; ++s) {
#pragma unroll
        for (uint32_t b = 0; b < kWays; ++b) {
            const uint64_t mid = (lo[b] + hi[b]) / 2;
            const uint32_t k = key_in[umin64(mid, n - 1)];
            const bool before = k < key || (k == key && g0 + b < mine);
            if (lo[b] < hi[b]) {
                if (before) lo[b] = mid + 1;
                else hi[b] = mid;
            }
        }
    }
    uint64_t rank = 0;
#pragma unroll
    for (uint32_t b = 0; b < kWays; ++b) rank += lo[b] - umin64((g0 + b) * run, n);
    key_out[g0 * run + rank] = key;
    pos_out[g0 * run + rank] = pos_in[i];
}

// ------------------------------------------------------- distinct rows
// A head is a sorted position whose row differs from the one before it.
// heads_before[b] is the number of heads in front of block b of kSpan sorted
// positions, which places the block's rows in a message.
constexpr uint32_t kSpan = 32;
constexpr uint32_t kHeadTile = 4096;
constexpr int kHeadThreads = 1024;

__device__ __forceinline__ bool is_head(const uint32_t *key, uint32_t q, uint32_t rows) {
    const uint32_t k = key[q];
    return k < rows && (q == 0 || key[q - 1] != k);
}

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

// Workgroup x places tile x; the last one writes the message's offsets.
__global__ __launch_bounds__(kHeadThreads) void embed_rows_kernel(const uint32_t *__restrict__ key, uint32_t n,
                                                                  uint32_t rows, uint32_t cols,
                                                                  const uint32_t *__restrict__ tile_heads,
                                                                  uint32_t *__restrict__ heads_before,
                                                                  uint32_t *__restrict__ seg_off, int nseg, int seg) {
    uint32_t before = 0, total;
    for (uint32_t t = threadIdx.x; t < blockIdx.x; t += kHeadThreads) before += tile_heads[t];
    (void)block_exclusive_scan<uint32_t, kHeadThreads>(before, &total);
    before = total;
    // thread t owns 4 consecutive positions of the tile; 8 threads a block
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

__device__ __forceinline__ void put_row(const SumOut &o, uint32_t row, uint32_t rank, uint32_t c, uint32_t cols,
                                        float scale, const float (&acc)[4]) {
    if (c >= cols) return;
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = scale * acc[u];
    if (o.g) {
        float *p = o.g + static_cast<uint64_t>(row) * cols;
        if (o.add) {
            float old[4];
            load_cols<F32>(p, c, cols, old);
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = old[u] + v[u];
        }
        store_cols<F32>(p, c, cols, v);
    } else {
        const uint64_t at = static_cast<uint64_t>(rank) * cols;
        store_cols<F32>(o.val + at, c, cols, v);
        const uint32_t i0 = o.idx0 + row * cols + c;
        if (c + 4 <= cols) {
            *reinterpret_cast<U32x4 *>(o.idx + at + c) = U32x4{{i0, i0 + 1, i0 + 2, i0 + 3}};
        } else {
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u)
                if (c + u < cols) o.idx[at + c + u] = i0 + u;
        }
    }
}

// Wave (block b of kSpan sorted positions, slab of 256 columns).  The
// block's keys and positions are held one per lane; the rows are loaded 8 at
// a time and added in order.  part[2 b] holds the sum of a run that comes
// from the block before, part[2 b + 1] of one that begins here and goes on.
constexpr uint32_t kSlab = 256;
constexpr uint32_t kAhead = 8;

template <class T>
__global__ __launch_bounds__(kBlock) void embed_sum_kernel(const typename T::Store *__restrict__ dy, uint64_t stride,
                                                           const uint32_t *__restrict__ key,
                                                           const uint32_t *__restrict__ pos, uint32_t n, uint32_t rows,
                                                           uint32_t cols, uint32_t slabs, uint64_t nwaves, float scale,
                                                           SumOut out, float *__restrict__ part, uint32_t ldpart) {
    const uint64_t wv = static_cast<uint64_t>(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(wave_id());
    if (wv >= nwaves) return;
    const uint32_t b = static_cast<uint32_t>(wv / slabs);
    const uint32_t c = static_cast<uint32_t>(wv - static_cast<uint64_t>(b) * slabs) * kSlab + 4u * lane_id();
    const uint32_t q0 = b * kSpan;
    const uint32_t cnt = min(n - q0, kSpan);
    const uint32_t l = min(static_cast<uint32_t>(lane_id()), cnt - 1);
    const uint32_t lkey = key[q0 + l], lpos = pos[q0 + l];
    const uint32_t prev = q0 > 0 ? key[q0 - 1] : 0xFFFFFFFFu;
    const uint32_t next = q0 + cnt < n ? key[q0 + cnt] : 0xFFFFFFFFu;
    uint32_t rank = out.g ? 0u : out.heads_before[b];  // rank of the next head
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    bool from_before = prev == static_cast<uint32_t>(__builtin_amdgcn_readlane(lkey, 0));
    for (uint32_t j0 = 0; j0 < cnt; j0 += kAhead) {
        float v[kAhead][4];
#pragma unroll
        for (uint32_t j = 0; j < kAhead; ++j) {
            const uint32_t jj = min(j0 + j, cnt - 1);
            const uint32_t k = __builtin_amdgcn_readlane(lkey, jj), p = __builtin_amdgcn_readlane(lpos, jj);
#pragma unroll
            for (int u = 0; u < 4; ++u) v[j][u] = 0.0f;
            if (k < rows && c < cols) load_cols<T>(dy + p * stride, c, cols, v[j]);
        }
#pragma unroll
        for (uint32_t j = 0; j < kAhead; ++j) {
            if (j0 + j < cnt) {
                const uint32_t jj = j0 + j;
                const uint32_t k = __builtin_amdgcn_readlane(lkey, jj);
                const bool last = jj + 1 == cnt;
                const uint32_t after = last ? next : static_cast<uint32_t>(__builtin_amdgcn_readlane(lkey, min(jj + 1, cnt - 1)));
#pragma unroll
                for (int u = 0; u < 4; ++u) acc[u] = acc[u] + v[j][u];
                if (k < rows && (last || after != k)) {
                    const bool goes_on = last && after == k;
                    if (from_before || goes_on) {
                        float *p = part + (2ull * b + (from_before ? 0 : 1)) * ldpart;
                        if (c < cols) store_cols<F32>(p, c, cols, acc);
                    } else {
                        put_row(out, k, rank, c, cols, scale, acc);
                    }
                    if (!from_before) ++rank;
                }
                if (after != k) {
                    from_before = false;
#pragma unroll
                    for (int u = 0; u < 4; ++u) acc[u] = 0.0f;
                }
            }
        }
    }
}

// Workgroup (block b, slab): if a run begins in block b and crosses into the
// next, adds its partial sums: wave w takes partials w, w + 16, ... in order,
// then the 16 sums are added in wave order.
constexpr int kJoinThreads = 1024;
constexpr uint32_t kJoinWaves = kJoinThreads / kWave;

__global__ __launch_bounds__(kJoinThreads) void embed_join_kernel(const uint32_t *__restrict__ key, uint32_t n,
                                                                  uint32_t rows, uint32_t cols, uint32_t slabs,
                                                                  float scale, SumOut out,
                                                                  const float *__restrict__ part, uint32_t ldpart) {
    const uint32_t b = blockIdx.x / slabs;
    const uint32_t c = (blockIdx.x - b * slabs) * kSlab + 4u * lane_id();
    const uint32_t q0 = b * kSpan;  // the grid covers blocks that have a next one
    const uint32_t k = key[q0 + kSpan - 1];
    if (k >= rows || key[q0 + kSpan] != k || (q0 > 0 && key[q0 - 1] == k)) return;
    // blocks whose first position still holds this row
    const uint32_t nblocks = (n + kSpan - 1) / kSpan;
    uint32_t end = b + 1;
    for (;;) {
        const uint32_t bl = end + lane_id();
        const uint64_t m = __ballot(bl < nblocks && key[min(bl, nblocks - 1) * kSpan] == k);
        if (m == ~0ull) {
            end += kWave;
        } else {
            end += __builtin_ctzll(~m);
            break;
        }
    }
    const uint32_t count = end - b;  // partials: part[2 b + 1], then part[2 (b + i)]
    const uint32_t w = wave_id();
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < cols) {
        for (uint32_t i = w; i < count; i += kJoinWaves) {
            float v[4];
            load_cols<F32>(part + (2ull * (b + i) + (i == 0 ? 1 : 0)) * ldpart, c, cols, v);
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[u] = acc[u] + v[u];
        }
    }
    __shared__ float4 sums[kJoinWaves][kWave];
    sums[w][lane_id()] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (w != 0) return;
    uint32_t rank = 0;
    if (!out.g) {
        // heads of block b in front of the crossing run (its last head)
        const uint32_t q = q0 + min(static_cast<uint32_t>(lane_id()), kSpan - 1);
        const uint64_t heads = __ballot(lane_id() < int(kSpan) && is_head(key, q, rows));
        rank = out.heads_before[b] + static_cast<uint32_t>(__popcll(heads)) - 1;
    }
    const uint32_t used = min(count, kJoinWaves);
    for (uint32_t i = 1; i < used; ++i) {
        const float4 s = sums[i][lane_id()];
        acc[0] = acc[0] + s.x;
        acc[1] = acc[1] + s.y;
        acc[2] = acc[2] + s.z;
        acc[3] = acc[3] + s.w;
    }
    put_row(out, k, rank, c, cols, scale, acc);
}

// --------------------------------------------------------------- host side
constexpr uint64_t kMaxTokens = uint64_t(1) << 31;  // positions and blocks are u32
constexpr uint64_t kMaxGrid = 0x7FFFFFFF;

struct EmbedWs {
    uint32_t *key[2], *pos[2], *heads_before, *tile_heads;
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
    const std::string at = std::string(fn) + ": ";
    if (!plan) return set_error(GC_EINVAL, at + "plan is null");
    if (seg < 0 || seg >= plan->nseg) return set_error(GC_EINVAL, at + "seg is not a segment of the plan");
    const uint32_t len = plan->seg[seg].len;
    if (rows < 1 || len % rows) return set_error(GC_EINVAL, at + "rows must divide the segment's length");
    *cols = len / rows;
    return GC_OK;
}

size_t type_bytes(int type) { return type == GC_F32 ? 4 : 2; }

gc_status check_batch(const char *fn, const void *tokens, int token_type, uint64_t n, const void *x, int type,
                      uint64_t stride, uint32_t cols, float scale) {
    const std::string at = std::string(fn) + ": ";
    if (token_type != GC_TOKENS_I32 && token_type != GC_TOKENS_I64)
        return set_error(GC_EINVAL, at + "token_type must be GC_TOKENS_I32 or GC_TOKENS_I64");
    if (type != GC_F32 && type != GC_BF16 && type != GC_F16)
        return set_error(GC_EINVAL, at + "type must be GC_F32, GC_BF16 or GC_F16");
    if (!(scale - scale == 0.0f)) return set_error(GC_EINVAL, at + "scale must be finite");
    if (n >= kMaxTokens) return set_error(GC_ERANGE, at + "n_tokens must be < 2^31");
    if (n == 0) return GC_OK;
    if (!tokens || !x) return set_error(GC_EINVAL, at + "buffers must be non-null");
    if (stride < cols) return set_error(GC_EINVAL, at + "the row stride must be at least the columns");
    if (n > 1 && stride > (uint64_t(1) << 48) / n) return set_error(GC_ERANGE, at + "n_tokens * stride must be <= 2^48");
    if (reinterpret_cast<uintptr_t>(tokens) % (token_type == GC_TOKENS_I32 ? 4 : 8) ||
        reinterpret_cast<uintptr_t>(x) % type_bytes(type))
        return set_error(GC_EINVAL, at + "buffers must be aligned to their elements");
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
    const uint32_t slabs = (cols + kSlab - 1) / kSlab, blocks = static_cast<uint32_t>(ceil_div(n, kSpan));
    const uint64_t waves = static_cast<uint64_t>(blocks) * slabs;
    if (nrank + nfill > kMaxGrid || waves > kMaxGrid)
        return set_error(GC_ERANGE, std::string(fn) + ": n_tokens * cols is above the supported range");
    with_tokens(token_type, [&](auto tok) {
        GC_LAUNCH("embed_rank", stream,
                  embed_rank_kernel<<<static_cast<unsigned>(nrank + nfill), kRankThreads, 0, stream>>>(
                      static_cast<const decltype(tok) *>(tokens), n, rows, w.key[0], w.pos[0],
                      static_cast<uint32_t>(nrank), out.g, fill));
    });
    int cur = 0;
    for (uint64_t run = kTile; run < n; run *= kWays) {
        int steps = 1;  // a search over `run` elements ends after floor(log2 run) + 1 halvings
        while ((run >> steps) != 0) ++steps;
        GC_LAUNCH("embed_merge", stream,
                  embed_merge_kernel<<<grid_1d(n, kBlock), kBlock, 0, stream>>>(w.key[cur], w.pos[cur], n, run, steps,
                                                                              w.key[cur ^ 1], w.pos[cur ^ 1]));
        cur ^= 1;
    }
    if (!out.g) {
        const unsigned tiles = grid_1d(n, kHeadTile);
        if (tiles > 1)
            GC_LAUNCH("embed_heads", stream,
                      embed_heads_kernel<<<tiles, kHeadThreads, 0, stream>>>(w.key[cur], n, rows, w.tile_heads));
        GC_LAUNCH("embed_rows", stream,
                  embed_rows_kernel<<<tiles, kHeadThreads, 0, stream>>>(w.key[cur], n, rows, cols, w.tile_heads,
                                                                      w.heads_before, seg_off, plan->nseg, seg));
        out.heads_before = w.heads_before;
    }
    with_type(type, [&](auto t) {
        using T = decltype(t);
        GC_LAUNCH("embed_sum", stream,
                  embed_sum_kernel<T><<<grid_1d(waves, kWaves), kBlock, 0, stream>>>(
                      static_cast<const typename T::Store *>(dy), stride, w.key[cur], w.pos[cur], n, rows, cols, slabs,
                      waves, scale, out, w.part, w.ldpart));
    });
    if (blocks > 1)
        GC_LAUNCH("embed_join", stream,
                  embed_join_kernel<<<(blocks - 1) * slabs, kJoinThreads, 0, stream>>>(
                      w.key[cur], n, rows, cols, slabs, scale, out, w.part, w.ldpart));
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
    const uint32_t vecs = static_cast<uint32_t>(ceil_div(cols, 4));
    const uint64_t grid = ceil_div(n_tokens * vecs, kBlock * kLookupVecs);
    if (grid > kMaxGrid) return set_error(GC_ERANGE, "gc_embed_lookup: n_tokens * cols is above the supported range");
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
