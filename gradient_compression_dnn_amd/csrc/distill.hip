// Distillation from a teacher's top logits: the exact top k of every row
// (gc_top_logits), and the loss of a student's rows with its gradient
// (gc_distill_loss).  One workgroup a row.
#include <algorithm>
#include <string>
#include <type_traits>

#include "gc_internal.hpp"
#include "row_vectors.hpp"

namespace gc {

namespace {

constexpr double kLog2eExact = 1.44269504088896340736;
constexpr float kLog2e = static_cast<float>(kLog2eExact);
constexpr uint32_t kNone = 0xFFFFFFFFu;

// 16 bytes of a row are one vector of it.
template <class T>
constexpr int kVec = 16 / int(sizeof(typename T::Store));

// How many elements a row's first one is past 16 bytes.  Vectors are cut there, so that they are aligned wherever
// the row starts: column v N - skew on is vector v (4096 rows of 131071 bf16, which start anywhere: 600 us for
// the loss with its gradient by unaligned vectors, 505 by these).
template <class T>
__device__ __forceinline__ uint32_t skew_of(const typename T::Store *row) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) / sizeof(typename T::Store)) % kVec<T>;
}

// N elements of a row from c on; those before it, and at or past `cols`, are -Inf.
template <class T, int N>
__device__ __forceinline__ void load_logits(const typename T::Store *row, int64_t c, uint32_t cols, float (&v)[N]) {
    if (c >= 0 && c + N <= cols) {
        const auto t = *reinterpret_cast<const Pack<typename T::Store, N> *>(row + c);
#pragma unroll
        for (int u = 0; u < N; ++u) v[u] = T::to_f32(t.v[u]);
    } else {
#pragma unroll
        for (int u = 0; u < N; ++u) v[u] = c + u >= 0 && c + u < cols ? T::to_f32(row[c + u]) : -INFINITY;
    }
}

__device__ __forceinline__ float across(float x, int d) { return __shfl_xor(x, d, kWave); }
__device__ __forceinline__ double across(double x, int d) { return __shfl_xor(x, d, kWave); }

// op over the values of the workgroup's threads, in every thread: a tree over
// a wave's lanes, then over the waves.
template <int NT, class V, class Op>
__device__ __forceinline__ V block_reduce(V x, V *lds, Op op) {
    constexpr int kCount = NT / kWave;
    static_assert((kCount & (kCount - 1)) == 0 && kCount <= kWave, "a lane per wave");
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) x = op(x, across(x, d));
    __syncthreads();
    if (lane_id() == 0) lds[wave_id()] = x;
    __syncthreads();
    x = lds[lane_id() & (kCount - 1)];
#pragma unroll
    for (int d = 1; d < kCount; d <<= 1) x = op(x, across(x, d));
    return x;
}

// The maximum leaves NaNs out.
template <int NT>
__device__ __forceinline__ float block_max(float x, float *lds) {
    return block_reduce<NT>(x, lds, [](float a, float b) { return fmaxf(a, b); });
}
template <int NT, class V>
__device__ __forceinline__ V block_sum(V x, V *lds) {
    return block_reduce<NT>(x, lds, [](V a, V b) { return a + b; });
}

// exp2 of the hardware (within a step; results below 2^-126 are 0).
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// log x, within 2^-24: a row's scalars are logarithms of up to some 20 whose differences count, so they are combined in
// double (in fp32 a KL near 0 was off by 1e-6 T^2).
__device__ __forceinline__ double log_of(float x) {
    float m = __builtin_amdgcn_frexp_mantf(x);
    int e = __builtin_amdgcn_frexp_expf(x);
    if (m < 0.70710678f) {
        m = m + m;
        --e;
    }
    return e * 0.693147180559945309 + logf(m);
}

// A sum of exp((x_j - r) / T), r an element near the largest: differences first, so that neither
// a large common part of the logits nor a row of the type's lowest value costs anything.  c is
// log2(e) / T throughout.
struct Sum {
    float r, s;
};
constexpr Sum kNoTerms{-INFINITY, 0.0f};
__device__ __forceinline__ float term(float x, float r, float c) { return exp2_of((x - r) * c); }
__device__ __forceinline__ Sum join(Sum a, Sum b, float c) {
    const float r = fmaxf(a.r, b.r);
    // an empty side has r = -Inf; its s is 0, or NaN where a NaN was its only term
    const float fa = a.r == r ? 1.0f : term(a.r, r, c), fb = b.r == r ? 1.0f : term(b.r, r, c);
    return Sum{r, a.s * fa + b.s * fb};
}
__device__ __forceinline__ Sum across(Sum x, int d) { return Sum{__shfl_xor(x.r, d, kWave), __shfl_xor(x.s, d, kWave)}; }
template <int NT>
__device__ __forceinline__ Sum block_join(Sum x, float c, Sum *lds) {
    return block_reduce<NT>(x, lds, [c](Sum a, Sum b) { return join(a, b, c); });
}

// An element to subtract: 0 where there is none.
__device__ __forceinline__ float base(Sum a) { return a.r == -INFINITY ? 0.0f : a.r; }

// Adds a vector's terms.  `top` is its largest value (NaNs left out).  The
// reference moves only where a term could pass 2^kRoom.
constexpr float kRoom = 32.0f;
template <int N>
__device__ __forceinline__ void add_terms(Sum &a, float c, const float (&v)[N], float top) {
    const bool move = !((top - a.r) * c <= kRoom) && top > -INFINITY;
    if (__builtin_expect(__ballot(move) != 0, 0)) {  // a branch of the wave: as selects its arithmetic ran every time
        a.s = !move || a.r == -INFINITY ? a.s : a.s * term(a.r, top, c);
        a.r = move ? top : a.r;
    }
    const float r = base(a);
#pragma unroll
    for (int u = 0; u < N; ++u) a.s = a.s + term(v[u], r, c);
    asm volatile("" : "+v"(a.s));  // now: the terms of all vectors, kept for later, do not fit the registers
}

template <int N>
__device__ __forceinline__ float largest(const float (&v)[N]) {
    float m = v[0];
#pragma unroll
    for (int u = 1; u < N; ++u) m = fmaxf(m, v[u]);
    return m;
}

// ------------------------------------------------------------------- top k
// Logits in the order of their values as unsigned keys; -0 as +0, and 0 for
// what is no candidate (NaN, -Inf).
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = dev_f2u(x + 0.0f);
    const uint32_t key = b & 0x80000000u ? ~b : b | 0x80000000u;
    return x > -INFINITY ? key : 0u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
    return dev_u2f(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

struct Range {
    float high, low;
};
__device__ __forceinline__ Range across(Range x, int d) { return Range{__shfl_xor(x.high, d, kWave), __shfl_xor(x.low, d, kWave)}; }

// The order of entries as one number: the key above, and below it 2^20 - 1 - column.
constexpr int kColBits = 20;
static_assert(GC_MAX_VOCAB <= 1u << kColBits, "columns fit");
__device__ __forceinline__ uint64_t entry_of(uint32_t key, uint32_t col) {
    return (static_cast<uint64_t>(key) << kColBits) | ((1u << kColBits) - 1 - col);
}

// The digits of an entry, from the highest: 11, 11, 10 bits of the key, 10, 10 of the column.
struct Digit {
    int shift, bits;
};
__device__ __forceinline__ Digit digit_of(int pass) {
    return pass == 0 ? Digit{41, 11} : pass == 1 ? Digit{30, 11} : pass == 2 ? Digit{20, 10} : pass == 3 ? Digit{10, 10} : Digit{0, 10};
}

// The `want` largest of the entries that each(f) calls f for (by all threads alike): every entry with
// (entry & known) > prefix is taken, and every one with (entry & known) == prefix.
template <int NT, class Each>
__device__ __forceinline__ void select_entries(uint32_t want, Each each, uint32_t *hist, uint64_t *known_out, uint64_t *prefix_out) {
    uint64_t known = 0, prefix = 0;
    uint32_t need = want;
    for (int pass = 0; pass < 5; ++pass) {
        const Digit d = digit_of(pass);
        const uint64_t mask = ((1ull << d.bits) - 1) << d.shift;
        for (uint32_t i = threadIdx.x; i < 2048; i += NT) hist[i] = 0;
        __syncthreads();
        each([&](uint64_t e) {
            if ((e & known) == prefix) atomicAdd(&hist[(e & mask) >> d.shift], 1u);
        });
        __syncthreads();
        uint32_t above;
        const uint32_t b = block_find_bucket<2048, NT>(need, [&](int i) { return hist[i]; }, &above);
        need -= above;
        prefix |= static_cast<uint64_t>(b) << d.shift;
        known |= mask;
        const bool all = hist[b] == need;  // the whole bucket is taken
        __syncthreads();
        if (all) break;
    }
    *known_out = known;
    *prefix_out = prefix;
}

constexpr uint32_t kRanked = 256;  // entries that are ranked without a selection

// The top k of a row.  A bound under the k-th largest comes from a sample: the maxima of vectors spread over the
// row; k of those are above it.  One pass then notes the vectors with an element above the bound, with the sums
// beside it (their elements at once, with an atomic each: 350 us at 4096 x 131072 bf16, k = 64, where this takes
// 240); the elements' top k are found digit by digit and ranked by counting.  The sample is chosen so that half of
// the list is expected to fill at most.  Where it overflows, with large ones side by side, the vectors that were
// noted are read again, digit by digit (the first 2000 of 131071 columns 9 larger: 221 us, and 803 by the row), and
// where those are too many (ties, a sample that misses the large ones), the row (all equal: 7.3 ms).  The bound is
// one of 2047 equal steps from the sample's largest to its lowest: a finite mask that fills a vector of the sample
// leaves all other logits in the first of them, and the row is read digit by digit (the last 3% of 131071 columns
// -1e4: 1.26 ms, the type's lowest value: 1.36, half of them 1.65; as -Inf, which the sample leaves out, 240 us).
// Memory bounds the pass, with several rows a unit: 240 us are 4.5 TB/s, where a copy reaches 5.1.  A few rows, and
// long lists, take 1,024 threads each (4096 x 131071, k = 1024: 586 us, and 1,010 with 256 threads; one row of
// 131071, k = 64: 22 us, the latency of its 4 rounds of loads and 5 digits).  Two of those share a unit, for which
// the bounds hold the scalar registers as well (without: 452 us where k = 128 takes 316).
template <class T, int NT, uint32_t kList, uint32_t kMost>
__global__ __launch_bounds__(NT, NT == 1024 ? 8 : 1) void top_kernel(const typename T::Store *__restrict__ logits,
                                                                     uint64_t stride, uint32_t vocab, uint32_t k, uint32_t groups,
                                                                     double inverse, int32_t *__restrict__ idx,
                                                                     float *__restrict__ val, float *__restrict__ lse) {
    constexpr int N = kVec<T>, kAhead = 4;
    __shared__ uint32_t hist[kList > 2048 ? kList : 2048];
    __shared__ uint64_t list[kList], best[kMost];
    __shared__ Range red[NT / kWave];
    __shared__ Sum sums[NT / kWave];
    __shared__ uint32_t listed, spotted, taken;
    float *tops = reinterpret_cast<float *>(list);  // the sample's maxima, before there is a list
    uint32_t *spots = hist;                         // vectors with an element above the bound, while no digits are counted
    const uint64_t r = blockIdx.x;
    const typename T::Store *row = logits + r * stride;
    const uint32_t t = threadIdx.x, skew = skew_of<T>(row), vecs = (vocab + skew + N - 1) / N;
    // vectors that lie inside the row, read without a check each: with one, no load went out before the last was there
    const uint32_t first = skew ? 1 : 0, whole = (vocab + skew) / N > first ? (vocab + skew) / N - first : 0;
    auto inside = [&](uint32_t at, float(&v)[N]) {
        const auto x = *reinterpret_cast<const Pack<typename T::Store, N> *>(row + (at * N - skew));
#pragma unroll
        for (int u = 0; u < N; ++u) v[u] = T::to_f32(x.v[u]);
    };
    // the vectors that the row begins and ends in, a thread each
    const uint32_t cut_at = t == 0 ? 0 : first + whole;
    const bool cut = t < 2 && (t == 0 ? first == 1 : first + whole < vecs);
    float cut_v[N];
    if (cut) load_logits<T>(row, static_cast<int64_t>(cut_at) * N - skew, vocab, cut_v);
    // the sample: runs of 64 vectors, spread evenly (single vectors take as many lines of memory as the row has)
    const uint32_t ng = groups < whole ? groups / kWave * kWave : whole;  // at most 2 kList, what tops holds
    float high = -INFINITY, low = INFINITY;
    for (uint32_t g0 = t; g0 < ng; g0 += NT * kAhead) {
        float v[kAhead][N];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const uint32_t g = min(g0 + i * NT, ng - 1), run = g / kWave;
            inside(first + (ng < whole ? static_cast<uint32_t>(static_cast<uint64_t>(run * kWave) * whole / ng) + g % kWave : g), v[i]);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (g0 + i * NT < ng) {
                const float top = largest(v[i]);
                tops[g0 + i * NT] = top;
                high = fmaxf(high, top);
                if (top > -INFINITY) low = fminf(low, top);
            }
    }
    if (t == 0) listed = spotted = taken = 0;
    for (uint32_t i = t; i < 2048; i += NT) hist[i] = 0;
    const Range range = block_reduce<NT>(Range{high, low}, red, [](Range a, Range b) { return Range{fmaxf(a.high, b.high), fminf(a.low, b.low)}; });
    high = range.high;
    low = range.low;
    // bins of the distance from the largest; its order is the values' reversed
    const float per = 2047.0f / (high - low);
    const bool usable = high < INFINITY && per > 0.0f && per < INFINITY;
    float limit = INFINITY;  // listed is what has (high - x) per < limit
    if (usable) {
        uint32_t mine = 0;
        for (uint32_t g = t; g < ng; g += NT)
            if (tops[g] > -INFINITY) {
                atomicAdd(&hist[2047 - static_cast<uint32_t>((high - tops[g]) * per)], 1u);
                ++mine;
            }
        uint32_t count;
        (void)block_exclusive_scan<uint32_t, NT>(mine, &count);
        if (count >= k) {
            uint32_t above;
            limit = static_cast<float>(2048 - block_find_bucket<2048, NT>(k, [&](int b) { return hist[b]; }, &above));
        }
    }
    // without a bound every logit passes: the distance of a very low one could overflow, and is not below an infinite limit
    const bool bounded = limit < INFINITY;
    const float from = bounded ? high : 0.0f, by = bounded ? per : 0.0f;
    // not below the limit: (0 - x) 0 is NaN for +Inf, which passes
    auto passes = [&](float x) { return x > -INFINITY && !((from - x) * by >= limit); };
    __syncthreads();
    const float c2 = static_cast<float>(inverse * kLog2eExact);
    Sum sum = kNoTerms;
    auto look = [&](uint32_t at, const float(&v)[N]) {
        const float m = largest(v);
        if (passes(m)) {
            const uint32_t p = atomicAdd(&spotted, 1u);
            if (p < kList) spots[p] = at;
        }
        if (lse) add_terms(sum, c2, v, m);
    };
    for (uint32_t at = first + t, end = first + whole; at < end; at += NT * kAhead) {
        float v[kAhead][N];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) inside(min(at + i * NT, end - 1), v[i]);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (at + i * NT < end) look(at + i * NT, v[i]);
    }
    if (cut) look(cut_at, cut_v);
    if (lse) {
        sum = block_join<NT>(sum, c2, sums);
        if (t == 0) lse[r] = static_cast<float>(base(sum) * inverse + log_of(sum.s));
    }
    __syncthreads();
    const bool all_spots = spotted <= kList;
    if (all_spots)
        for (uint32_t i = t; i < spotted; i += NT) {
            float v[N];
            load_logits<T>(row, static_cast<int64_t>(spots[i]) * N - skew, vocab, v);
#pragma unroll
            for (int u = 0; u < N; ++u)
                if (passes(v[u])) {
                    const uint32_t p = atomicAdd(&listed, 1u);
                    if (p < kList) list[p] = entry_of(order_key(v[u]), spots[i] * N + u - skew);
                }
        }
    __syncthreads();
    // a list of fewer than k holds every candidate: a bound has k above it
    const uint32_t n = all_spots ? listed : spotted, want = min(k, n);
    const bool ranked = n <= kRanked;
    if (!ranked) {
        uint64_t known, prefix;
        auto take = [&](uint64_t e) {
            if ((e & known) >= prefix) best[atomicAdd(&taken, 1u)] = e;  // in any order: ranked below
        };
        if (n <= kList) {
            auto each = [&](auto f) {
                for (uint32_t i = t; i < n; i += NT) f(list[i]);
            };
            select_entries<NT>(want, each, hist, &known, &prefix);
            each(take);
        } else {
            // the vectors that were noted, if all of them were, or the row
            uint32_t *noted = reinterpret_cast<uint32_t *>(list);
            const uint32_t vectors = all_spots ? spotted : vecs;
            if (all_spots)
                for (uint32_t i = t; i < vectors; i += NT) noted[i] = spots[i];
            __syncthreads();  // the digits are counted where the spots are
            auto each = [&](auto f) {
                for (uint32_t i = t; i < vectors; i += NT) {
                    const uint32_t at = all_spots ? noted[i] : i;
                    float v[N];
                    load_logits<T>(row, static_cast<int64_t>(at) * N - skew, vocab, v);
#pragma unroll
                    for (int u = 0; u < N; ++u) {
                        const uint32_t key = order_key(v[u]);
                        if (key) f(entry_of(key, at * N + u - skew));
                    }
                }
            };
            select_entries<NT>(want, each, hist, &known, &prefix);
            each(take);
        }
        __syncthreads();
    }
    const uint64_t *of = ranked ? list : best;
    const uint32_t count = ranked ? n : want;
    for (uint32_t i = t; i < count; i += NT) {
        const uint64_t e = of[i];
        uint32_t rank = 0;
#pragma unroll 8
        for (uint32_t j = 0; j < count; ++j) rank += of[j] > e;
        if (rank < want) {
            idx[r * k + rank] = static_cast<int32_t>((1u << kColBits) - 1 - (e & ((1u << kColBits) - 1)));
            val[r * k + rank] = key_value(static_cast<uint32_t>(e >> kColBits));
        }
    }
    for (uint32_t i = want + t; i < k; i += NT) {
        idx[r * k + i] = -1;
        val[r * k + i] = -INFINITY;
    }
}

// -------------------------------------------------------------------- loss
struct Distill {
    const void *logits, *idx, *t, *labels;
    const float *t_lse, *weights;
    float *loss;
    void *dlogits;
    uint64_t stride, idx_stride, t_stride, dstride;
    uint32_t vocab, k;
    int id_type, t_type, rest, bits;
    double inverse;                       // 1 / T
    float kd, kd_slope, ce, grad;         // kd T^2 and kd T
};

__device__ __forceinline__ int64_t id_at(const void *ids, int type, uint64_t at) {
    return type == GC_TOKENS_I32 ? static_cast<const int32_t *>(ids)[at] : static_cast<const int64_t *>(ids)[at];
}
__device__ __forceinline__ float teacher_value(const Distill &d, uint64_t at) {
    if (d.t_type == GC_F32) return static_cast<const float *>(d.t)[at];
    const uint16_t x = static_cast<const uint16_t *>(d.t)[at];
    return d.t_type == GC_BF16 ? BF16::to_f32(x) : F16::to_f32(x);
}

// A row of logits: C vectors a thread, held in registers from the sums to the gradient, so that they
// are read once.  kMore: the row goes on behind them, and that part is read by each sweep.
template <class T, int NT, int C, bool kMore>
struct Row {
    static constexpr int N = kVec<T>;
    using Vectors = RowVectors<N, NT, C, kMore>;
    static constexpr uint32_t kStep = Vectors::kStep;
    using Store = typename T::Store;
    const Store *row;
    uint32_t vocab, skew;
    u32x4 raw[C ? C : 1];

    __device__ __forceinline__ u32x4 vector_at(uint32_t c) const {
        return __builtin_bit_cast(u32x4, *reinterpret_cast<const Pack<Store, N> *>(row + c));
    }
    __device__ __forceinline__ void load() {
#pragma unroll
        for (int i = 0; i < C; ++i) raw[i] = vector_at(Vectors::column(i, threadIdx.x, skew, vocab));
    }
    // f(column, values, count): columns that another call has already are -Inf for kOnce; count of them exist.
    template <bool kOnce, class F>
    __device__ __forceinline__ void each(F f) {
        float v[N];
        auto values = [&](u32x4 w) {
            const auto x = __builtin_bit_cast(Pack<Store, N>, w);
#pragma unroll
            for (int u = 0; u < N; ++u) v[u] = T::to_f32(x.v[u]);
        };
#pragma unroll
        for (int i = 0; i < C; ++i) {
            // a vector at a time, neither its values in fp32 nor its place kept for another sweep: else they do
            // not fit the registers
            uint32_t t = threadIdx.x;
            asm volatile("" : "+v"(raw[i]), "+v"(t));
            const int32_t c = Vectors::column(i, t, skew, vocab), own = Vectors::own(i, t, skew);
            values(raw[i]);
            if (kOnce && Vectors::moves(i) && __ballot(c != own))
#pragma unroll
                for (int32_t u = 0; u < N; ++u) v[u] = c + u < own || c + u >= own + N ? -INFINITY : v[u];
            if (kMore || kOnce || own < static_cast<int32_t>(vocab)) f(c, v, uint32_t(N));
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kMore) {
            constexpr int kAhead = 4;
            int64_t c = static_cast<int64_t>(C * kStep + threadIdx.x * N) - skew;
            if (c >= 0)
                for (; c + (kAhead - 1) * kStep + N <= vocab; c += kAhead * kStep) {
                    u32x4 w[kAhead];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) w[i] = vector_at(c + i * kStep);
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        values(w[i]);
                        f(c + i * kStep, v, uint32_t(N));
                    }
                }
            for (; c < vocab; c += kStep) {
                if (c < 0 || c + N > vocab) {  // the elements that the row has, one by one
                    for (int u = 0; u < N; ++u) {
                        if (c + u < 0 || c + u >= vocab) continue;
                        v[0] = T::to_f32(row[c + u]);
#pragma unroll
                        for (int x = 1; x < N; ++x) v[x] = -INFINITY;
                        f(static_cast<int32_t>(c + u), v, 1u);
                    }
                } else {
                    values(vector_at(c));
                    f(static_cast<int32_t>(c), v, uint32_t(N));
                }
            }
        }
    }
};

// A workgroup a row; several rows share a unit, so that one's sums and exponentials run while others are on their
// way (a loop over rows that fetches the next row meanwhile was slower).  The sums run over the row with the maximum
// beside them, once, and the gradient is formed from the registers that hold it: memory bounds it, one read and one
// write of the logits.  us, 4096 rows of bf16, k = 64: 131072 columns 465 (a copy's rate: 421), 131071 505 (rows
// start anywhere), 65536 213, 32000 118; the loss alone at 131071 235 (211).  Labels at another temperature take a
// second exponential an element: 610.  700 rows of 10000 fp32, k = 32: 22, most of it a launch, a row's latency and
// the sums over 16 vectors a thread, of which the row fills 10.
// LDS: columns, q, q summed over a column's entries, and student logits of the entries, and (GC_DISTILL_REST, or up
// to kBitsVocab columns) a bit per column that an entry names.
// kTwo: the labels' softmax has another temperature than the teacher's.
template <class T, int NT, int C, bool kMore, bool kTwo>
__global__ __launch_bounds__(NT) void distill_kernel(Distill d) {
    constexpr int N = kVec<T>;
    using Store = typename T::Store;
    extern __shared__ __attribute__((aligned(16))) uint32_t dyn[];
    __shared__ float red[NT / kWave];
    __shared__ double redd[NT / kWave];
    __shared__ Sum reds[NT / kWave];
    const uint32_t t = threadIdx.x, V = d.vocab, K = d.k, K4 = (K + 3) & ~3u;
    uint32_t *col = dyn;
    float *q = reinterpret_cast<float *>(dyn + K4), *qs = q + K4, *zk = qs + K4;
    uint32_t *named = dyn + 4 * K4;
    const uint64_t r = blockIdx.x;
    const Store *row = static_cast<const Store *>(d.logits) + r * d.stride;
    Store *out = d.dlogits ? static_cast<Store *>(d.dlogits) + r * d.dstride : nullptr;
    // entry e: its column, or kNone, and the teacher's logit
    auto entry = [&](uint32_t e, uint32_t &c, float &v) {
        c = kNone;
        v = -INFINITY;
        if (e >= K || d.kd_slope == 0.0f) return;
        const int64_t id = id_at(d.idx, d.id_type, r * d.idx_stride + e);
        v = teacher_value(d, r * d.t_stride + e);
        if (id >= 0 && id < static_cast<int64_t>(V) && v != -INFINITY) c = static_cast<uint32_t>(id);
    };
    auto student = [&](uint32_t c) { return c != kNone ? T::to_f32(row[c]) : 0.0f; };

    // This thread's entry and the label come first, then the row, then the logits of the former: memory answers in order.
    uint32_t my_col, label = kNone;
    float my_t;
    entry(t, my_col, my_t);
    if (d.labels && d.ce != 0.0f) {
        const int64_t l = id_at(d.labels, d.id_type, r);
        if (l >= 0 && l < static_cast<int64_t>(V)) label = static_cast<uint32_t>(l);
    }
    Row<T, NT, C, kMore> z{row, V, skew_of<T>(row)};
    z.load();
    const float my_z = student(my_col), zl = student(label);
    const float weight = d.weights ? d.weights[r] : 1.0f;
    // the teacher's distribution
    float tmax = my_col != kNone ? my_t : -INFINITY;
    bool there = my_col != kNone;
    if (t < K4) {
        col[t] = my_col;
        q[t] = my_t;
    }
    for (uint32_t e = t + NT; e < K4; e += NT) {
        uint32_t c;
        float v;
        entry(e, c, v);
        col[e] = c;
        q[e] = v;
        zk[e] = student(c);
        there = there || c != kNone;
        tmax = c != kNone ? fmaxf(tmax, v) : tmax;
    }
    const bool entries = __syncthreads_or(there);
    bool own_label = label != kNone;  // no entry names it
    if (own_label && entries) {
        bool named_here = my_col == label;
        for (uint32_t e = t + NT; e < K; e += NT) named_here = named_here || col[e] == label;
        own_label = !__syncthreads_or(named_here);
    }
    if (weight == 0.0f || !(entries || label != kNone)) {  // the row counts for nothing
        if (t == 0) d.loss[r] = 0.0f;
        if (out)
            for (uint32_t c = t * N; c < V; c += NT * N) {
                if (c + N <= V) *reinterpret_cast<Pack<Store, N> *>(out + c) = Pack<Store, N>{};
                else
                    for (uint32_t u = c; u < V; ++u) out[u] = Store(0);
            }
        return;
    }
    const bool rest = d.rest && entries;
    double qsum = 0.0;
    if (entries) {
        if (d.bits)
            for (uint32_t i = t; i < (V + 31) / 32 + 1; i += NT) named[i] = 0;
        if (!d.rest) tmax = block_max<NT>(tmax, red);
        else __syncthreads();
        tmax = tmax == -INFINITY ? 0.0f : tmax;
        const float tlse = d.rest ? d.t_lse[r] : 0.0f;
        bool again = !d.bits;  // a column may be named again
        for (uint32_t e = t; e < K; e += NT) {
            const uint32_t c = col[e];
            q[e] = c != kNone ? expf(static_cast<float>(d.rest ? q[e] * d.inverse - tlse : (static_cast<double>(q[e]) - tmax) * d.inverse)) : 0.0f;
            qsum += q[e];
            if (d.bits && c != kNone) again = again || (atomicOr(&named[c / 32], 1u << (c % 32)) >> (c % 32) & 1);
        }
        qsum = block_sum<NT>(qsum, redd);
        const float inv = d.rest ? 1.0f : static_cast<float>(1.0 / qsum);
        qsum = d.rest ? qsum : 1.0;
        for (uint32_t e = t; e < K; e += NT) q[e] = q[e] * inv;
        again = __syncthreads_or(again);
        // A column's first entry holds the sum of all of them, the others a negative number.  Every entry against
        // every other is left to rows that name a column again (4096 x 131071, 1,024 entries: 878 us, 634 without).
        // An entry meets itself without a branch: with one, each lane of a wave took it at another time.
        for (uint32_t e = t; e < K; e += NT) {
            const uint32_t c = col[e];
            float sum = q[e];
            uint32_t before = 0;  // entries of this column in front of e
            if (c != kNone && again)
#pragma unroll 4
                for (uint32_t j = 0; j < K4; j += 4) {
                    const uint4 o = *reinterpret_cast<const uint4 *>(col + j);
                    const uint32_t self = e - j;  // below 4 in this piece
                    const bool x = o.x == c && self != 0, y = o.y == c && self != 1, z = o.z == c && self != 2, w = o.w == c && self != 3;
                    if (x || y || z || w) {
                        sum = sum + (x ? q[j] : 0.0f);
                        sum = sum + (y ? q[j + 1] : 0.0f);
                        sum = sum + (z ? q[j + 2] : 0.0f);
                        sum = sum + (w ? q[j + 3] : 0.0f);
                        before += (x && j < e) + (y && j + 1 < e) + (z && j + 2 < e) + (w && j + 3 < e);
                    }
                }
            qs[e] = c != kNone && before == 0 ? sum : -1.0f;
        }
        __syncthreads();
    }
    auto each_own = [&](auto f) {  // f(entry, its student's logit)
        if (t < K) f(t, my_z);
        for (uint32_t e = t + NT; e < K; e += NT) f(e, zk[e]);
    };
    // the row, or the rest of it: sums of exp at 1 / T and, for another softmax of the labels, at 1
    const float c2 = static_cast<float>(d.inverse * kLog2eExact), c1 = kTwo ? kLog2e : c2;
    Sum s2 = kNoTerms, s1 = kNoTerms;
    z.template each<true>([&](uint32_t c, float(&v)[N], uint32_t) {
        if (rest) {
            const uint32_t w = c / 32;
            const uint32_t bits = __builtin_amdgcn_alignbit(named[w + 1], named[w], c % 32);
            if (bits & ((1u << N) - 1))
#pragma unroll
                for (int u = 0; u < N; ++u) v[u] = bits >> u & 1 ? -INFINITY : v[u];
        }
        const float top = largest(v);
        add_terms(s2, c2, v, top);
        if (kTwo) add_terms(s1, c1, v, top);
    });
    const Sum rest2 = block_join<NT>(s2, c2, reds);
    Sum all2 = rest2, all1 = kTwo ? block_join<NT>(s1, c1, reds) : rest2;
    if (rest) {  // the entries that were left out, each column once
        s2 = s1 = kNoTerms;
        each_own([&](uint32_t e, float x) {
            if (qs[e] >= 0.0f || qs[e] != qs[e]) {
                const float v[1] = {x};
                add_terms(s2, c2, v, x);
                if (kTwo) add_terms(s1, c1, v, x);
            }
        });
        all2 = join(rest2, block_join<NT>(s2, c2, reds), c2);
        all1 = kTwo ? join(all1, block_join<NT>(s1, c1, reds), c1) : all2;
    }
    // where nothing is left, as for entries that name all columns but masked ones, rr is r2 and rest2.s 0
    const float r2 = base(all2), r1 = base(all1), rr = rest2.r == -INFINITY ? r2 : rest2.r;
    const double held_mass = rest && rest2.s != 0.0f ? fmax(1.0 - qsum, 0.0) : 0.0;
    const float held = static_cast<float>(held_mass);
    if (out) {
        // the gradient: kd T (mass p_j - held p_j / p_r - q_j) + ce (softmax_j - [j = label])
        const float mass = entries ? static_cast<float>(qsum) + held : 0.0f, f = weight * d.grad;
        const float kt = entries ? f * d.kd_slope : 0.0f, kc = label != kNone ? f * d.ce : 0.0f;
        const float back = term(rr, r2, c2);  // p_j = back term(z_j, rr) / all2.s
        float g2 = kt * (mass * back / all2.s - (held > 0.0f ? held / rest2.s : 0.0f));
        const float g1 = kc / all1.s;
        if (!kTwo) g2 = g2 + g1 * back;
        __syncthreads();  // the entries' logits, whose places may be out's, have been read
        z.template each<false>([&](uint32_t c, float(&v)[N], uint32_t cnt) {
            Pack<Store, N> g;
#pragma unroll
            for (int u = 0; u < N; ++u) {
                float x = g2 * term(v[u], rr, c2);
                if (kTwo) x = x + g1 * term(v[u], r1, c1);
                g.v[u] = T::from_f32(x);
            }
            if (cnt == N) *reinterpret_cast<Pack<Store, N> *>(out + c) = g;
            else
#pragma unroll
                for (uint32_t u = 0; u < N; ++u)
                    if (u < cnt) out[c + u] = g.v[u];
        });
        __syncthreads();
        // columns that an entry or the label names
        auto set = [&](uint32_t c, float x, float sum, bool of_rest) {
            const float p = term(x, r2, c2) / all2.s;
            float g = kt * (mass * p - sum) + kc * (term(x, r1, c1) / all1.s - (c == label ? 1.0f : 0.0f));
            if (of_rest && held > 0.0f) g = g - kt * held * (term(x, rr, c2) / rest2.s);
            out[c] = T::from_f32(g);
        };
        if (entries)
            each_own([&](uint32_t e, float x) {
                if (col[e] != kNone && !(qs[e] < 0.0f)) set(col[e], x, qs[e], false);
            });
        if (own_label && t == NT - 1) set(label, zl, 0.0f, true);
    }
    // the loss, while the gradient is on its way; NaN for a row without a distribution, also where no entry has a term
    double loss = all2.s > 0.0f ? 0.0 : NAN;
    if (entries) {
        const double log2s = log_of(all2.s);
        double kl = 0.0;  // sum of q (log q - z / T), with the row's log sum behind it
        each_own([&](uint32_t e, float x) {
            if (q[e] != 0.0f) kl += q[e] * (log_of(q[e]) - (static_cast<double>(x) - r2) * d.inverse);
        });
        kl = block_sum<NT>(kl, redd) + qsum * log2s;
        if (held > 0.0f) kl += held_mass * (log_of(held) - ((static_cast<double>(rr) - r2) * d.inverse + log_of(rest2.s) - log2s));
        loss = loss + d.kd * kl;
    }
    if (label != kNone) loss = loss + d.ce * (log_of(all1.s) - (static_cast<double>(zl) - r1));
    if (t == 0) d.loss[r] = static_cast<float>(weight * loss);
}

// --------------------------------------------------------------- host side
constexpr uint64_t kMaxRows = uint64_t(1) << 22;
constexpr uint64_t kFewRows = 256;  // rows that have a unit each
constexpr uint32_t kBitsVocab = 1u << 18;  // 32 KiB of bits: as many rows a unit as without
constexpr uint32_t kSmallList = 1024, kBigList = 4096, kSmallK = 128;

size_t type_bytes(int type) { return type == GC_F32 ? 4 : 2; }
bool known_type(int type) { return type == GC_F32 || type == GC_BF16 || type == GC_F16; }
gc_status fail(const char *fn, gc_status st, const char *what) { return set_error(st, std::string(fn) + ": " + what); }
bool misaligned(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

gc_status check_strided(const char *fn, const void *p, uint64_t stride, uint64_t n, uint64_t cols, size_t bytes) {
    if (!p) return fail(fn, GC_EINVAL, "buffers must be non-null");
    if (stride < cols) return fail(fn, GC_EINVAL, "a row stride must be at least the row's length");
    if (n > 1 && stride > (uint64_t(1) << 48) / n) return fail(fn, GC_ERANGE, "n_rows * a stride must be <= 2^48");
    if (misaligned(p, bytes)) return fail(fn, GC_EINVAL, "buffers must be aligned to their elements");
    return GC_OK;
}

gc_status check_sizes(const char *fn, int type, uint64_t n, uint32_t vocab, uint32_t k, float temperature) {
    if (!known_type(type)) return fail(fn, GC_EINVAL, "type must be GC_F32, GC_BF16 or GC_F16");
    if (vocab < 1) return fail(fn, GC_EINVAL, "vocab must be at least 1");
    if (vocab > GC_MAX_VOCAB) return fail(fn, GC_ENOTSUP, "vocab must be <= GC_MAX_VOCAB");
    if (k > GC_MAX_TOP_LOGITS) return fail(fn, GC_ENOTSUP, "k must be <= GC_MAX_TOP_LOGITS");
    const float inverse = static_cast<float>(1.0 / temperature * kLog2eExact);  // as the kernels form it
    if (!(temperature > 0.0f) || !(temperature - temperature == 0.0f) || !(inverse - inverse == 0.0f))
        return fail(fn, GC_EINVAL, "temperature must be positive, and finite with its inverse");
    if (n >= kMaxRows) return fail(fn, GC_ERANGE, "n_rows must be < 2^22");
    return GC_OK;
}

}  // namespace
}  // namespace gc

using namespace gc;

#define GC_TRY(expr)                       \
    do {                                   \
        const gc_status st_ = (expr);      \
        if (st_ != GC_OK) return st_;      \
    } while (0)

extern "C" gc_status gc_top_logits(const void *logits, int type, uint64_t stride, uint64_t n_rows, uint32_t vocab,
                                   uint32_t k, float temperature, int32_t *idx, float *val, float *lse,
                                   hipStream_t stream) {
    static const char fn[] = "gc_top_logits";
    clear_error();
    GC_TRY(check_sizes(fn, type, n_rows, vocab, k, temperature));
    if (k < 1) return fail(fn, GC_EINVAL, "k must be at least 1");
    if (n_rows == 0) return GC_OK;
    GC_TRY(check_strided(fn, logits, stride, n_rows, vocab, type_bytes(type)));
    GC_TRY(check_strided(fn, idx, k, n_rows, k, 4));
    GC_TRY(check_strided(fn, val, k, n_rows, k, 4));
    if (misaligned(lse, 4)) return fail(fn, GC_EINVAL, "buffers must be aligned to their elements");
    auto go = [&](auto t) {
        using T = decltype(t);
        constexpr uint64_t N = kVec<T>;
        const bool few = n_rows <= kFewRows, small = k <= kSmallK && uint64_t(vocab) * k <= N * kSmallList * kSmallList;
        auto with = [&](auto kernel, int threads, uint64_t room) {
            // v k / (groups N) of a row are expected above the bound: half of the list, and for a small k, whose
            // bound scatters more, k / (2 k + 16) of it (a row in 100 overflowed half of it at k = 8, which took twice
            // the time: 4096 x 131071 bf16 444 us, and 211 like this); or fewer, as a load a thread costs no time
            const uint64_t sample = ceil_div((2 * uint64_t(k) + 16) * vocab, N * room);
            const uint64_t groups = ceil_div(std::max<uint64_t>({sample, 2 * uint64_t(k), few ? uint64_t(threads) : 0}), kWave) * kWave;
            GC_LAUNCH("top_logits", stream,
                      kernel<<<static_cast<unsigned>(n_rows), threads, 0, stream>>>(
                          static_cast<const typename T::Store *>(logits), stride, vocab, k, static_cast<uint32_t>(umin64(groups, 2 * room)),
                          1.0 / temperature, idx, val, lse));
        };
        if (!small) with(top_kernel<T, 1024, kBigList, GC_MAX_TOP_LOGITS>, 1024, kBigList);
        else if (few) with(top_kernel<T, 1024, kSmallList, kSmallK>, 1024, kSmallList);
        else with(top_kernel<T, 256, kSmallList, kSmallK>, 256, kSmallList);
    };
    if (type == GC_F32) go(F32{});
    else if (type == GC_BF16) go(BF16{});
    else go(F16{});
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? GC_OK : hip_error(e, fn);
}

extern "C" gc_status gc_distill_loss(const void *logits, int type, uint64_t stride, uint64_t n_rows, uint32_t vocab,
                                     const void *idx, int idx_type, uint64_t idx_stride, const void *t, int t_type,
                                     uint64_t t_stride, uint32_t k, const float *t_lse, const void *labels,
                                     const float *weights, const gc_distill_options *opt, float *loss, void *dlogits,
                                     uint64_t dstride, hipStream_t stream) {
    static const char fn[] = "gc_distill_loss";
    clear_error();
    if (!opt) return fail(fn, GC_EINVAL, "opt must be non-null");
    GC_TRY(check_sizes(fn, type, n_rows, vocab, k, opt->temperature));
    if (idx_type != GC_TOKENS_I32 && idx_type != GC_TOKENS_I64)
        return fail(fn, GC_EINVAL, "idx_type must be GC_TOKENS_I32 or GC_TOKENS_I64");
    if (!known_type(t_type)) return fail(fn, GC_EINVAL, "t_type must be GC_F32, GC_BF16 or GC_F16");
    if (opt->mode != GC_DISTILL_TOP && opt->mode != GC_DISTILL_REST) return fail(fn, GC_EINVAL, "unknown mode");
    if (opt->reserved[0] || opt->reserved[1] || opt->reserved[2]) return fail(fn, GC_EINVAL, "reserved must be 0");
    const float T = opt->temperature, kd = opt->kd_weight * T * T;
    for (float x : {opt->kd_weight, opt->ce_weight, opt->grad_scale, kd})
        if (!(x - x == 0.0f)) return fail(fn, GC_EINVAL, "weights, grad_scale and kd_weight T^2 must be finite");
    if (n_rows == 0) return GC_OK;
    const size_t id_bytes = idx_type == GC_TOKENS_I32 ? 4 : 8;
    GC_TRY(check_strided(fn, logits, stride, n_rows, vocab, type_bytes(type)));
    GC_TRY(check_strided(fn, loss, 1, n_rows, 1, 4));
    if (k) {
        GC_TRY(check_strided(fn, idx, idx_stride, n_rows, k, id_bytes));
        GC_TRY(check_strided(fn, t, t_stride, n_rows, k, type_bytes(t_type)));
        if (opt->mode == GC_DISTILL_REST && !t_lse) return fail(fn, GC_EINVAL, "GC_DISTILL_REST needs t_lse");
    }
    if (misaligned(t_lse, 4) || misaligned(weights, 4) || misaligned(labels, id_bytes))
        return fail(fn, GC_EINVAL, "buffers must be aligned to their elements");
    if (dlogits) {
        GC_TRY(check_strided(fn, dlogits, dstride, n_rows, vocab, type_bytes(type)));
        if (dlogits == logits && dstride != stride)
            return fail(fn, GC_EINVAL, "dlogits in place of logits must have their stride");
    }
    Distill d{logits, idx, t, labels, t_lse, weights, loss, dlogits, stride, idx_stride, t_stride, dstride, vocab, k, idx_type, t_type,
              opt->mode == GC_DISTILL_REST, 0, 1.0 / T, kd, opt->kd_weight * T, opt->ce_weight, opt->grad_scale};
    if (!k) d.kd = d.kd_slope = 0.0f;
    d.bits = k && (d.rest || vocab <= kBitsVocab);
    const size_t lds = 16 * ((size_t(k) + 3) & ~size_t(3)) + (d.bits ? 4 * ((size_t(vocab) + 31) / 32 + 1) : 0);
    const bool two = labels && opt->ce_weight != 0.0f && T != 1.0f;
    hipError_t e = hipSuccess;
    auto go = [&](auto kernel, int threads) {
        if (lds > 48 * 1024)
            e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess) return;
        GC_LAUNCH("distill", stream, kernel<<<static_cast<unsigned>(n_rows), threads, lds, stream>>>(d));
    };
    auto with = [&](auto type_tag, auto is_two) {
        using Tp = decltype(type_tag);
        constexpr bool kTwo = decltype(is_two)::value;
        // rows that start on 16 bytes, or anywhere
        const bool even = !misaligned(logits, 16) && stride * type_bytes(type) % 16 == 0;
        const LossShape s = loss_shape(vocab, kVec<Tp>, even);
        if (s.held == 0) go(distill_kernel<Tp, 256, 0, true, kTwo>, 256);
        else if (s.held == 4) go(distill_kernel<Tp, 256, 4, false, kTwo>, 256);
        else if (s.held == 8) go(distill_kernel<Tp, 256, 8, false, kTwo>, 256);
        else if (s.threads == 256) go(distill_kernel<Tp, 256, 16, false, kTwo>, 256);
        else if (!s.more) go(distill_kernel<Tp, 512, 16, false, kTwo>, 512);
        else go(distill_kernel<Tp, 512, 16, true, kTwo>, 512);
    };
    auto of = [&](auto type_tag) {
        if (two) with(type_tag, std::true_type{});
        else with(type_tag, std::false_type{});
    };
    if (type == GC_F32) of(F32{});
    else if (type == GC_BF16) of(BF16{});
    else of(F16{});
    if (e == hipSuccess) e = hipGetLastError();
    return e == hipSuccess ? GC_OK : hip_error(e, fn);
}
