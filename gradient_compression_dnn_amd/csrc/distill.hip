// Distillation from a teacher's top logits: the exact top k of every row
// (gc_top_logits), and the loss of a student's rows with its gradient
// (gc_distill_loss).  One workgroup a row.
#include <string>

#include "gc_internal.hpp"

namespace gc {

namespace {

constexpr int kThreads = 1024;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr uint32_t kNone = 0xFFFFFFFFu;

// N elements of a row from c on; those at or past `cols` are -Inf.
template <class T, int N>
__device__ __forceinline__ void load_logits(const typename T::Store *row, uint32_t c, uint32_t cols, float (&v)[N]) {
    if (c + N <= cols) {
        const auto t = *reinterpret_cast<const Pack<typename T::Store, N> *>(row + c);
#pragma unroll
        for (int u = 0; u < N; ++u) v[u] = T::to_f32(t.v[u]);
    } else {
#pragma unroll
        for (uint32_t u = 0; u < N; ++u) v[u] = c + u < cols ? T::to_f32(row[c + u]) : -INFINITY;
    }
}

template <class T>
constexpr int kVec = 16 / int(sizeof(typename T::Store));  // 16 bytes

// The workgroup's maximum (NaNs left out) and sums, in every thread.
__device__ __forceinline__ float block_max(float x, float *lds) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) x = fmaxf(x, __shfl_xor(x, d, kWave));
    __syncthreads();
    if (lane_id() == 0) lds[wave_id()] = x;
    __syncthreads();
    x = lds[0];
    for (uint32_t w = 1; w < blockDim.x / kWave; ++w) x = fmaxf(x, lds[w]);
    return x;
}
template <class V>
__device__ __forceinline__ V block_sum(V x, V *lds) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) x = x + __shfl_xor(x, d, kWave);
    __syncthreads();
    if (lane_id() == 0) lds[wave_id()] = x;
    __syncthreads();
    x = lds[0];
    for (uint32_t w = 1; w < blockDim.x / kWave; ++w) x = x + lds[w];
    return x;
}

// A maximum to subtract: 0 where every value was -Inf.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.0f : m; }

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

// Three passes of 11, 11 and 10 bits find the key of the k-th candidate; all
// above it are taken, and of those equal to it the first by index.
template <class T>
__global__ __launch_bounds__(kThreads) void top_kernel(const typename T::Store *__restrict__ logits, uint64_t stride,
                                                       uint32_t vocab, uint32_t k, float scale, int32_t *__restrict__ idx,
                                                       float *__restrict__ val, float *__restrict__ lse) {
    constexpr int N = kVec<T>;
    __shared__ uint32_t hist[2048];
    __shared__ uint32_t keys[GC_MAX_TOP_LOGITS], cols[GC_MAX_TOP_LOGITS];
    __shared__ float red[kThreads / kWave];
    __shared__ uint32_t taken;
    const uint64_t r = blockIdx.x;
    const typename T::Store *row = logits + r * stride;
    const uint32_t t = threadIdx.x;
    // statistics, and the number of candidates
    float m = -INFINITY;
    uint32_t cand = 0;
    for (uint32_t c = t * N; c < vocab; c += kThreads * N) {
        float v[N];
        load_logits<T>(row, c, vocab, v);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            m = fmaxf(m, v[u]);
            cand += v[u] > -INFINITY;
        }
    }
    m = finite_max(block_max(m, red));
    if (lse) {
        float s = 0.0f;
        for (uint32_t c = t * N; c < vocab; c += kThreads * N) {
            float v[N];
            load_logits<T>(row, c, vocab, v);
#pragma unroll
            for (int u = 0; u < N; ++u) s = s + (v[u] == m ? 1.0f : expf((v[u] - m) * scale));
        }
        s = block_sum(s, red);
        if (t == 0) lse[r] = m * scale + logf(s);
    }
    uint32_t total;
    (void)block_exclusive_scan<uint32_t, kThreads>(cand, &total);
    const uint32_t want = min(k, total);
    uint32_t prefix = 0, known = 0, need = want;  // keys with these top bits hold the `need`-th of the rest
    if (want) {
        for (int pass = 0; pass < 3; ++pass) {
            const int bits = pass < 2 ? 11 : 10, low = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            for (uint32_t i = t; i < 2048; i += kThreads) hist[i] = 0;
            __syncthreads();
            for (uint32_t c = t * N; c < vocab; c += kThreads * N) {
                float v[N];
                load_logits<T>(row, c, vocab, v);
#pragma unroll
                for (int u = 0; u < N; ++u) {
                    const uint32_t key = order_key(v[u]);
                    if (key && (key & known) == prefix) atomicAdd(&hist[(key >> low) & ((1u << bits) - 1)], 1u);
                }
            }
            __syncthreads();
            uint32_t above;
            const uint32_t d = block_find_bucket<2048, kThreads>(need, [&](int b) { return hist[b]; }, &above);
            need -= above;
            prefix |= d << low;
            known |= ((1u << bits) - 1) << low;
        }
        if (t == 0) taken = 0;
        __syncthreads();
        const uint32_t over = want - need;  // keys above the threshold
        uint32_t equal = 0;                 // equal ones in front of this part of the row
        for (uint32_t c0 = 0; c0 < vocab; c0 += kThreads * N) {
            float v[N];
            load_logits<T>(row, c0 + t * N, vocab, v);
            uint32_t mine = 0;
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const uint32_t key = order_key(v[u]);
                if (key > prefix) {
                    const uint32_t at = atomicAdd(&taken, 1u);  // any order: ranked below
                    keys[at] = key;
                    cols[at] = c0 + t * N + u;
                }
                mine += key == prefix;
            }
            uint32_t here;
            uint32_t at = equal + block_exclusive_scan<uint32_t, kThreads>(mine, &here);
            if (mine)
#pragma unroll
                for (int u = 0; u < N; ++u)
                    if (order_key(v[u]) == prefix) {
                        if (at < need) {
                            keys[over + at] = prefix;
                            cols[over + at] = c0 + t * N + u;
                        }
                        ++at;
                    }
            equal += here;
        }
        __syncthreads();
    }
    if (t < k) {
        if (t < want) {
            const uint32_t key = keys[t], col = cols[t];
            uint32_t rank = 0;
            for (uint32_t j = 0; j < want; ++j) rank += keys[j] > key || (keys[j] == key && cols[j] < col);
            idx[r * k + rank] = static_cast<int32_t>(col);
            val[r * k + rank] = key_value(key);
        } else {
            idx[r * k + t] = -1;
            val[r * k + t] = -INFINITY;
        }
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
    int t_type, rest;
    float inv_t, kd, kd_slope, ce, grad;  // 1 / T; kd T^2 and kd T
};

// The largest value so far and the sums of exp relative to it, at 1 / T and at 1.
struct Stats {
    float m, st, s1;
};
__device__ __forceinline__ Stats join(const Stats &a, const Stats &b, float ct) {
    Stats o;
    o.m = fmaxf(a.m, b.m);
    const float m = finite_max(o.m);
    // an empty side has m = -Inf and sums of 0
    const float fa = (finite_max(a.m) - m) * kLog2e, fb = (finite_max(b.m) - m) * kLog2e;
    const bool ea = a.m == -INFINITY, eb = b.m == -INFINITY;
    o.st = (ea ? a.st : a.st * exp2f(fa * ct)) + (eb ? b.st : b.st * exp2f(fb * ct));
    o.s1 = (ea ? a.s1 : a.s1 * exp2f(fa)) + (eb ? b.s1 : b.s1 * exp2f(fb));
    return o;
}

__device__ __forceinline__ float teacher_value(const Distill &d, uint64_t at) {
    if (d.t_type == GC_F32) return static_cast<const float *>(d.t)[at];
    const uint16_t x = static_cast<const uint16_t *>(d.t)[at];
    return d.t_type == GC_BF16 ? BF16::to_f32(x) : F16::to_f32(x);
}

// LDS: columns, q and student logits of the entries, then a bit per column
// (GC_DISTILL_REST) of those that an entry names.
template <class T, class Ids>
__global__ __launch_bounds__(kThreads) void distill_kernel(Distill d) {
    constexpr int N = kVec<T>;
    using Store = typename T::Store;
    extern __shared__ __attribute__((aligned(16))) uint32_t dyn[];
    __shared__ float red[kThreads / kWave];
    __shared__ double redd[kThreads / kWave];
    __shared__ Stats reds[kThreads / kWave];
    uint32_t *col = dyn;
    float *q = reinterpret_cast<float *>(dyn + d.k), *zk = q + d.k;
    uint32_t *named = dyn + 3 * d.k;
    const uint64_t r = blockIdx.x;
    const uint32_t t = threadIdx.x, V = d.vocab, K = d.k;
    const Store *row = static_cast<const Store *>(d.logits) + r * d.stride;
    Store *out = d.dlogits ? static_cast<Store *>(d.dlogits) + r * d.dstride : nullptr;

    const float weight = d.weights ? d.weights[r] : 1.0f;
    uint32_t label = kNone;
    if (d.labels && d.ce != 0.0f) {
        const int64_t l = static_cast<const Ids *>(d.labels)[r];
        if (l >= 0 && l < static_cast<int64_t>(V)) label = static_cast<uint32_t>(l);
    }
    // the teacher's entries
    float tmax = -INFINITY;
    uint32_t count = 0;
    if (d.kd != 0.0f)
        for (uint32_t e = t; e < K; e += kThreads) {
            const int64_t c = static_cast<const Ids *>(d.idx)[r * d.idx_stride + e];
            const float v = teacher_value(d, r * d.t_stride + e);
            const bool there = c >= 0 && c < static_cast<int64_t>(V) && v != -INFINITY;
            col[e] = there ? static_cast<uint32_t>(c) : kNone;
            q[e] = v;
            zk[e] = there ? T::to_f32(row[c]) : 0.0f;
            tmax = there ? fmaxf(tmax, v) : tmax;
            count += there;
        }
    uint32_t entries;
    (void)block_exclusive_scan<uint32_t, kThreads>(count, &entries);
    if (weight == 0.0f || (entries == 0 && label == kNone)) {
        if (t == 0) d.loss[r] = 0.0f;
        if (out)
            for (uint32_t c = t; c < V; c += kThreads) out[c] = Store(0);
        return;
    }
    const bool rest = d.rest && entries;
    if (rest) {
        for (uint32_t i = t; i < (V + 31) / 32; i += kThreads) named[i] = 0;
        __syncthreads();
        for (uint32_t e = t; e < K; e += kThreads)
            if (col[e] != kNone) atomicOr(&named[col[e] / 32], 1u << (col[e] % 32));
    }
    tmax = finite_max(block_max(tmax, red));
    const float tlse = d.rest ? (d.t_lse ? d.t_lse[r] : 0.0f) : tmax * d.inv_t;
    double qsum = 0.0;
    if (entries)
        for (uint32_t e = t; e < K; e += kThreads) {
            q[e] = col[e] == kNone ? 0.0f : expf((d.rest ? q[e] * d.inv_t - tlse : (q[e] - tmax) * d.inv_t));
            qsum += q[e];
        }
    qsum = block_sum(qsum, redd);
    if (entries && !d.rest) {
        const float inv = static_cast<float>(1.0 / qsum);
        for (uint32_t e = t; e < K; e += kThreads) q[e] = q[e] * inv;
        qsum = 1.0;
    }
    __syncthreads();

    // the row, or the rest of it
    const float ct = d.inv_t, c1 = kLog2e, c2 = d.inv_t * kLog2e;
    Stats s{-INFINITY, 0.0f, 0.0f};
    for (uint32_t c = t * N; c < V; c += kThreads * N) {
        float v[N];
        load_logits<T>(row, c, V, v);
        if (rest) {
            const uint32_t bits = named[c / 32] >> (c % 32);
#pragma unroll
            for (int u = 0; u < N; ++u) v[u] = bits >> u & 1 ? -INFINITY : v[u];
        }
        Stats p{v[0], 0.0f, 0.0f};
#pragma unroll
        for (int u = 1; u < N; ++u) p.m = fmaxf(p.m, v[u]);
        const float m = finite_max(p.m);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            p.st = p.st + exp2f((v[u] - m) * c2);
            p.s1 = p.s1 + exp2f((v[u] - m) * c1);
        }
        s = join(s, p, ct);
    }
#pragma unroll
    for (int x = 1; x < kWave; x <<= 1)
        s = join(s, Stats{__shfl_xor(s.m, x, kWave), __shfl_xor(s.st, x, kWave), __shfl_xor(s.s1, x, kWave)}, ct);
    if (lane_id() == 0) reds[wave_id()] = s;
    __syncthreads();
    s = reds[0];
    for (int w = 1; w < kThreads / kWave; ++w) s = join(s, reds[w], ct);
    const Stats of_rest = s;
    // the entries that were left out, each column once
    Stats all = s;
    if (rest) {
        Stats mine{-INFINITY, 0.0f, 0.0f};
        for (uint32_t e = t; e < K; e += kThreads) {
            bool first = col[e] != kNone;
            for (uint32_t j = 0; first && j < e; ++j) first = col[j] != col[e];
            if (first) {
                const float z = zk[e], m = finite_max(z);
                mine = join(mine, Stats{z, exp2f((z - m) * c2), exp2f((z - m) * c1)}, ct);
            }
        }
#pragma unroll
        for (int x = 1; x < kWave; x <<= 1)
            mine = join(mine, Stats{__shfl_xor(mine.m, x, kWave), __shfl_xor(mine.st, x, kWave), __shfl_xor(mine.s1, x, kWave)}, ct);
        __syncthreads();
        if (lane_id() == 0) reds[wave_id()] = mine;
        __syncthreads();
        for (int w = 0; w < kThreads / kWave; ++w) all = join(all, reds[w], ct);
    }
    const float m = finite_max(all.m), mr = finite_max(of_rest.m);
    const float logst = logf(all.st), logs1 = logf(all.s1);
    const float held = rest && of_rest.st != 0.0f ? fmaxf(static_cast<float>(1.0 - qsum), 0.0f) : 0.0f;
    const float mass = entries ? static_cast<float>(qsum) + held : 0.0f;
    // the loss
    double kl = 0.0;
    if (entries)
        for (uint32_t e = t; e < K; e += kThreads)
            if (q[e] != 0.0f) kl += q[e] * (logf(q[e]) - ((zk[e] - m) * ct - logst));
    kl = block_sum(kl, redd);
    if (held > 0.0f) kl += held * (logf(held) - ((mr - m) * ct + logf(of_rest.st) - logst));
    const float zl = label != kNone ? T::to_f32(row[label]) : 0.0f;
    if (t == 0) {
        float loss = entries ? d.kd * static_cast<float>(kl) : 0.0f;
        if (label != kNone) loss = loss + d.ce * (logs1 - (zl - m));
        d.loss[r] = weight * loss;
    }
    if (!out) return;
    // the gradient: kd T (mass p_j - held p_j / p_r - q_j) + ce (softmax_j - [j = label])
    const float f = weight * d.grad;
    const float kt = entries ? f * d.kd_slope : 0.0f, kc = label != kNone ? f * d.ce : 0.0f;
    const float pt = mass * exp2f((mr - m) * c2);  // mass p_j = pt exp((z - mr) / T) / st
    const float at = kt * (pt / all.st - (held > 0.0f ? held / of_rest.st : 0.0f));
    const float a1 = kc * (exp2f((mr - m) * c1) / all.s1);
    __syncthreads();  // row[label], which may lie in out, has been read
    for (uint32_t c = t * N; c < V; c += kThreads * N) {
        float v[N];
        load_logits<T>(row, c, V, v);
#pragma unroll
        for (uint32_t u = 0; u < N; ++u) {
            float g = 0.0f;
            if (v[u] != -INFINITY) g = at * exp2f((v[u] - mr) * c2) + a1 * exp2f((v[u] - mr) * c1);
            if (c + u < V) out[c + u] = T::from_f32(g);
        }
    }
    __syncthreads();
    // columns that an entry or the label names
    for (uint32_t e = t; e < K + 1; e += kThreads) {
        const uint32_t c = e < K ? (entries ? col[e] : kNone) : label;
        if (c == kNone) continue;
        bool first = true;
        float qs = 0.0f;
        if (entries)
            for (uint32_t j = 0; j < K; ++j)
                if (col[j] == c) {
                    first = first && j >= e;
                    qs = qs + q[j];
                }
        if (!first) continue;
        const float z = e < K ? zk[e] : zl;
        float g = kt * (mass * (exp2f((z - m) * c2) / all.st) - qs) + kc * (exp2f((z - m) * c1) / all.s1 - (c == label ? 1.0f : 0.0f));
        if (e == K && held > 0.0f) g = g - kt * held * (exp2f((z - mr) * c2) / of_rest.st);  // a label of the rest
        out[c] = T::from_f32(g);
    }
}

// --------------------------------------------------------------- host side
constexpr uint64_t kMaxRows = uint64_t(1) << 22;

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
    const float inverse = 1.0f / temperature;
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
        GC_LAUNCH("top_logits", stream,
                  top_kernel<T><<<static_cast<unsigned>(n_rows), kThreads, 0, stream>>>(
                      static_cast<const typename T::Store *>(logits), stride, vocab, k, 1.0f / temperature, idx, val, lse));
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
    Distill d{logits, idx,       t,        labels,  t_lse, weights, loss, dlogits, stride, idx_stride, t_stride, dstride, vocab, k, t_type,
              opt->mode == GC_DISTILL_REST, 1.0f / T, kd, opt->kd_weight * T, opt->ce_weight, opt->grad_scale};
    if (!k) d.kd = 0.0f;
    const size_t lds = 12 * size_t(k) + (d.rest ? 4 * ((size_t(vocab) + 31) / 32) : 0);
    hipError_t e = hipSuccess;
    auto go = [&](auto type_tag, auto id_tag) {
        const auto kernel = distill_kernel<decltype(type_tag), decltype(id_tag)>;
        if (lds > 48 * 1024)
            e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess) return;
        GC_LAUNCH("distill", stream, kernel<<<static_cast<unsigned>(n_rows), kThreads, lds, stream>>>(d));
    };
    auto ids = [&](auto type_tag) {
        if (idx_type == GC_TOKENS_I32) go(type_tag, int32_t{});
        else go(type_tag, int64_t{});
    };
    if (type == GC_F32) ids(F32{});
    else if (type == GC_BF16) ids(BF16{});
    else ids(F16{});
    if (e == hipSuccess) e = hipGetLastError();
    return e == hipSuccess ? GC_OK : hip_error(e, fn);
}
