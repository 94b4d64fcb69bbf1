// The product of a layer's weight matrix with a batch and its gradients
// (gc_linear_forward, gc_linear_grad_input, gc_linear_grad_weight), and the
// slope of an activation (gc_act_grad).
//
//   forward  z = x W^T + b, y = act(z) + r
//   input    g = dz W + a,  dx = g, dzx = g act'(z)
//   weight   G[W] (+)= dz^T x, G[b] (+)= column sums of dz
//
// All three are D[m][n] = sum_k A[m][k] B[n][k] with D row-major; what differs
// is which of an operand's two indices is contiguous in memory:
//            m        n      k       A           B
//   forward  tokens   rows   cols    x, k        W, k
//   input    tokens   cols   rows    dz, k       W, n
//   weight   rows     cols   tokens  dz, m       x, n
#include <algorithm>
#include <string>

#include "gc_internal.hpp"

namespace gc {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------- activations
__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }
// 2 sqrt(2 / pi) (z + 0.044715 z^3), whose sigmoid is gelu_tanh's factor
constexpr float kTanh2 = 1.5957691216057308f, kCubic = 0.044715f;
constexpr float kSqrtHalf = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;

__device__ __forceinline__ float act_value(int act, float z) {
    switch (act) {
        case GC_ACT_RELU: return z < 0.0f ? 0.0f : z;
        case GC_ACT_GELU: return z * (0.5f * erfcf(-z * kSqrtHalf));
        case GC_ACT_GELU_TANH: return z * sigmoid(kTanh2 * (z + kCubic * z * z * z));
        case GC_ACT_SILU: return z * sigmoid(z);
        default: return z;
    }
}
// Beyond +-kFar every slope here is 0 or 1 in fp32, and z^2 could overflow.
constexpr float kFar = 128.0f;
__device__ __forceinline__ float act_slope(int act, float z) {
    if (act == GC_ACT_NONE) return 1.0f;
    if (act == GC_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if (fabsf(z) > kFar) return z > 0.0f ? 1.0f : 0.0f;
    switch (act) {
        case GC_ACT_GELU: return 0.5f * erfcf(-z * kSqrtHalf) + z * (kInvSqrt2Pi * expf(-0.5f * z * z));
        case GC_ACT_GELU_TANH: {
            const float s = sigmoid(kTanh2 * (z + kCubic * z * z * z));
            return s + z * (s * (1.0f - s)) * (kTanh2 * (1.0f + 3.0f * kCubic * z * z));
        }
        default: {
            const float s = sigmoid(z);
            return s * (1.0f + z * (1.0f - s));
        }
    }
}

// Up to 4 elements of a row.
template <class T>
__device__ __forceinline__ void get4(const void *base, uint64_t at, uint32_t n, float (&v)[4]) {
    const auto *p = static_cast<const typename T::Store *>(base) + at;
    if (n >= 4) {
        const auto t = *reinterpret_cast<const Pack<typename T::Store, 4> *>(p);
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = T::to_f32(t.v[u]);
        return;
    }
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u) v[u] = u < n ? T::to_f32(p[u]) : 0.0f;
}
template <class T>
__device__ __forceinline__ void put4(void *base, uint64_t at, uint32_t n, const float (&v)[4]) {
    auto *p = static_cast<typename T::Store *>(base) + at;
    if (n >= 4) {
        Pack<typename T::Store, 4> t;
#pragma unroll
        for (int u = 0; u < 4; ++u) t.v[u] = T::from_f32(v[u]);
        *reinterpret_cast<Pack<typename T::Store, 4> *>(p) = t;
        return;
    }
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u)
        if (u < n) p[u] = T::from_f32(v[u]);
}

// --------------------------------------------------------------- products
enum Kind { kForward, kInput, kWeight };

struct Product {
    const void *A, *B;
    uint64_t lda, ldb;
    uint32_t M, N, K;
    const void *bias;           // forward: [N], or null; weight: null or not, whether column sums go to gbias
    const void *add;            // forward: r; input: a
    const void *z;              // input: the argument of the activation
    void *zout;                 // forward
    void *out, *out2;           // forward: y; input: dx, dzx; weight: the segment of g
    uint64_t ldadd, ldz, ldout, ldout2;
    float *gbias;               // weight: the bias' segment of g
    int act;
    int accumulate;             // weight
};

// A stage of an operand: kTile rows by 128 bytes of k (64 elements of 16 bits,
// 32 of fp32), kTile * 8 parts of 16 bytes in LDS.
//   k contiguous: [row][128 bytes], part c of a row at c ^ ((row >> 1) & 7), so
//     that the 16 rows a matrix operand reads at once lie in different banks
//   k slow: [k][kTile elements]; 16 elements stay together, at u ^ spread(k)
template <class T, bool kSlow, int kTile>
struct Operand {
    using Store = typename T::Store;
    static constexpr int kElems = 16 / int(sizeof(Store)), kStage = 128 / int(sizeof(Store));
    static constexpr int kUnits = kTile / 16, kRowBytes = kTile * int(sizeof(Store)), kUnitBytes = 16 * int(sizeof(Store));
    static constexpr uint32_t kParts = kTile * 8, kRowParts = kRowBytes / 16;

    static __device__ __forceinline__ uint32_t spread(uint32_t k) {
        return (sizeof(Store) == 2 ? ((k & 3) | ((k >> 1) & 4)) : ((k >> 2) & 3)) & (kUnits - 1);
    }
    // where a part stands, and which row (k contiguous) or k (slow) and which piece of it that is
    static __device__ __forceinline__ uint32_t place(uint32_t part, uint32_t &line, uint32_t &piece) {
        if (!kSlow) {
            line = part >> 3;
            piece = part & 7;
            return line * 128 + ((piece ^ ((line >> 1) & 7)) << 4);
        }
        line = part / kRowParts;
        piece = part % kRowParts;
        constexpr uint32_t kUnitParts = kUnitBytes / 16;
        return line * kRowBytes + ((piece / kUnitParts) ^ spread(line)) * kUnitBytes + (piece % kUnitParts) * 16;
    }
    // a part from memory; what lies past the last k is 0, past the last row anything
    static __device__ __forceinline__ u32x4 fetch(const void *base, uint64_t ld, uint32_t row0, uint32_t rows,
                                                  uint32_t k0, uint32_t K, uint32_t line, uint32_t piece) {
        const uint32_t r = kSlow ? row0 + piece * kElems : min(row0 + line, rows - 1);
        const uint32_t k = kSlow ? k0 + line : k0 + piece * kElems;
        const Store *p = static_cast<const Store *>(base) + (kSlow ? k * ld + r : r * ld + k);
        const uint32_t at = kSlow ? r : k, end = kSlow ? rows : K;
        if (kSlow && k >= K) return u32x4{0, 0, 0, 0};
        if (at + kElems <= end) return __builtin_bit_cast(u32x4, *reinterpret_cast<const Pack<Store, kElems> *>(p));
        Pack<Store, kElems> t;
#pragma unroll
        for (uint32_t u = 0; u < kElems; ++u) t.v[u] = at + u < end ? p[u] : Store(0);
        return __builtin_bit_cast(u32x4, t);
    }
    // rows row0 .. row0 + 15, 16 bytes of k a lane: row lane % 16, k from ((lane / 16) + 4 half) * kElems
    static __device__ __forceinline__ u32x4 read(const char *lds, uint32_t row0, int half) {
        const uint32_t lane = lane_id(), part = (lane >> 4) + 4 * half;
        if (!kSlow) {
            const uint32_t row = row0 + (lane & 15);
            return *reinterpret_cast<const u32x4 *>(lds + row * 128 + ((part ^ ((row >> 1) & 7)) << 4));
        }
        const uint32_t k = part * kElems;
        if constexpr (sizeof(Store) == 2) {
            // a transposing read: of 16 lanes, lane l fetches 4 rows of k + l / 4 and gets 4 k of row l
            typedef __attribute__((address_space(3))) s16x4 LdsS4;
            u32x4 v;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t line = k + 4 * h + ((lane & 15) >> 2);
                const char *p = lds + line * kRowBytes + ((row0 >> 4) ^ spread(line)) * kUnitBytes + (lane & 3) * 8;
                const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS4 *)(p));
                const uint2 w = __builtin_bit_cast(uint2, t);
                v[2 * h] = w.x;
                v[2 * h + 1] = w.y;
            }
            return v;
        } else {
            u32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = *reinterpret_cast<const uint32_t *>(lds + (k + e) * kRowBytes + ((row0 >> 4) ^ spread(k + e)) * kUnitBytes + (lane & 15) * 4);
            return v;
        }
    }
};

// d[i][j] += sum over 16 bytes of k of a[i] b[j]
template <class T>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 d) {
    if constexpr (sizeof(typename T::Store) == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) d = __builtin_amdgcn_mfma_f32_16x16x4f32(dev_u2f(a[e]), dev_u2f(b[e]), d, 0, 0, 0);
        return d;
    } else if constexpr (std::is_same<T, BF16>::value) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), d, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), d, 0, 0, 0);
    }
}

template <class T>
__device__ __forceinline__ u32x4 ones() {
    const uint32_t w = sizeof(typename T::Store) == 4 ? 0x3F800000u : std::is_same<T, BF16>::value ? 0x3F803F80u : 0x3C003C00u;
    return u32x4{w, w, w, w};
}

// What becomes of 4 sums of row m, columns n on.
template <class T, Kind kKind>
__device__ __forceinline__ void finish(const Product &p, uint32_t m, uint32_t n, f32x4 sum) {
    const uint32_t cnt = min(p.N - n, 4u);
    float v[4], t[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = sum[u];
    if constexpr (kKind == kWeight) {
        const uint64_t at = m * p.ldout + n;
        if (p.accumulate) {
            get4<F32>(p.out, at, cnt, t);
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = t[u] + v[u];
        }
        put4<F32>(p.out, at, cnt, v);
    } else if constexpr (kKind == kForward) {
        if (p.bias) {
            get4<T>(p.bias, n, cnt, t);
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = v[u] + t[u];
        }
        if (p.zout) put4<T>(p.zout, m * p.ldz + n, cnt, v);
        if (p.act != GC_ACT_NONE)
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = act_value(p.act, v[u]);
        if (p.add) {
            get4<T>(p.add, m * p.ldadd + n, cnt, t);
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = v[u] + t[u];
        }
        put4<T>(p.out, m * p.ldout + n, cnt, v);
    } else {
        if (p.add) {
            get4<T>(p.add, m * p.ldadd + n, cnt, t);
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = v[u] + t[u];
        }
        if (p.out) put4<T>(p.out, m * p.ldout + n, cnt, v);
        if (p.out2) {
            if (p.act != GC_ACT_NONE) {
                get4<T>(p.z, m * p.ldz + n, cnt, t);
#pragma unroll
                for (int u = 0; u < 4; ++u) v[u] = v[u] * act_slope(p.act, t[u]);
            }
            put4<T>(p.out2, m * p.ldout2 + n, cnt, v);
        }
    }
}

// A workgroup of kWR x kWC waves per tile of kTileM x kTileN, stages of 128
// bytes of k through registers into one of two LDS buffers.
template <class T, Kind kKind, int kTileM, int kTileN, int kWR, int kWC>
__global__ __launch_bounds__(kWR *kWC *kWave) void linear_kernel(Product p, uint32_t tiles_m) {
    constexpr int kThreads = kWR * kWC * kWave;
    using OpA = Operand<T, kKind == kWeight, kTileM>;
    using OpB = Operand<T, kKind != kForward, kTileN>;
    constexpr int kLoadsA = OpA::kParts / kThreads, kLoadsB = OpB::kParts / kThreads;
    constexpr int kRA = kTileM / kWR / 16, kRB = kTileN / kWC / 16;
    constexpr int kBytesA = kTileM * 128, kBytes = kBytesA + kTileN * 128;
    __shared__ __attribute__((aligned(128))) char lds[2 * kBytes];
    const uint32_t m0 = blockIdx.x % tiles_m * kTileM, n0 = blockIdx.x / tiles_m * kTileN;
    const uint32_t w = __builtin_amdgcn_readfirstlane(wave_id()), lane = lane_id();
    const uint32_t wm = w / kWC * (kTileM / kWR), wn = w % kWC * (kTileN / kWC);
    u32x4 ra[kLoadsA], rb[kLoadsB];
    auto fetch = [&](uint32_t k0) {
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i) {
            uint32_t line, piece;
            (void)OpA::place(i * kThreads + threadIdx.x, line, piece);
            ra[i] = OpA::fetch(p.A, p.lda, m0, p.M, k0, p.K, line, piece);
        }
#pragma unroll
        for (int i = 0; i < kLoadsB; ++i) {
            uint32_t line, piece;
            (void)OpB::place(i * kThreads + threadIdx.x, line, piece);
            rb[i] = OpB::fetch(p.B, p.ldb, n0, p.N, k0, p.K, line, piece);
        }
    };
    auto stash = [&](char *to) {
        uint32_t line, piece;
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i)
            *reinterpret_cast<u32x4 *>(to + OpA::place(i * kThreads + threadIdx.x, line, piece)) = ra[i];
#pragma unroll
        for (int i = 0; i < kLoadsB; ++i)
            *reinterpret_cast<u32x4 *>(to + kBytesA + OpB::place(i * kThreads + threadIdx.x, line, piece)) = rb[i];
    };
    f32x4 acc[kRA][kRB], colsum[kRA];
#pragma unroll
    for (int a = 0; a < kRA; ++a) {
        colsum[a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int b = 0; b < kRB; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // the sums of A over k, for the bias: a product with ones in the first column of tiles
    const bool sums = kKind == kWeight && p.gbias && n0 == 0 && wn == 0;
    const uint32_t stages = static_cast<uint32_t>(ceil_div(p.K, OpA::kStage));
    if (stages) {
        fetch(0);
        stash(lds);
    }
    for (uint32_t s = 0; s < stages; ++s) {
        __syncthreads();
        const char *cur = lds + (s & 1) * kBytes;
        if (s + 1 < stages) fetch((s + 1) * OpA::kStage);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 fb[kRB];
#pragma unroll
            for (int b = 0; b < kRB; ++b) fb[b] = OpB::read(cur + kBytesA, wn + 16 * b, h);
#pragma unroll
            for (int a = 0; a < kRA; ++a) {
                const u32x4 fa = OpA::read(cur, wm + 16 * a, h);
#pragma unroll
                for (int b = 0; b < kRB; ++b) acc[a][b] = mma<T>(fb[b], fa, acc[a][b]);
                if (sums) colsum[a] = mma<T>(ones<T>(), fa, colsum[a]);
            }
        }
        if (s + 1 < stages) stash(lds + ((s + 1) & 1) * kBytes);
    }
    // a lane holds 4 columns of row lane % 16 of each block of 16 x 16
#pragma unroll
    for (int a = 0; a < kRA; ++a) {
        const uint32_t m = m0 + wm + 16 * a + (lane & 15);
        if (m >= p.M) continue;
        if (sums && lane < 16) p.gbias[m] = p.accumulate ? p.gbias[m] + colsum[a][0] : colsum[a][0];
#pragma unroll
        for (int b = 0; b < kRB; ++b) {
            const uint32_t n = n0 + wn + 16 * b + 4 * (lane >> 4);
            if (n < p.N) finish<T, kKind>(p, m, n, acc[a][b]);
        }
    }
}

// dz = dy act'(z): 4 elements a thread.
template <class T>
__global__ __launch_bounds__(kBlock) void act_grad_kernel(const void *dy, uint64_t ldy, const void *z, uint64_t ldz, int act,
                                                          uint64_t n, uint64_t cols, void *dz, uint64_t ldd) {
    const uint64_t vecs = ceil_div(cols, 4);
    const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kBlock + threadIdx.x;
    const uint64_t row = i / vecs, c = (i - row * vecs) * 4;
    if (row >= n) return;
    const uint32_t cnt = static_cast<uint32_t>(umin64(cols - c, 4));
    float g[4], t[4];
    get4<T>(dy, row * ldy + c, cnt, g);
    get4<T>(z, row * ldz + c, cnt, t);
#pragma unroll
    for (int u = 0; u < 4; ++u) g[u] = g[u] * act_slope(act, t[u]);
    put4<T>(dz, row * ldd + c, cnt, g);
}

// --------------------------------------------------------------- host side
constexpr uint64_t kMaxTokens = uint64_t(1) << 28;
constexpr uint64_t kMaxElems = uint64_t(1) << 35;
constexpr uint64_t max_grid(uint64_t threads) { return 0xFFFFFFFFull / threads; }

size_t type_bytes(int type) { return type == GC_F32 ? 4 : 2; }
bool known_type(int type) { return type == GC_F32 || type == GC_BF16 || type == GC_F16; }
bool known_act(int act) { return act >= GC_ACT_NONE && act <= GC_ACT_SILU; }

gc_status fail(const char *fn, gc_status st, const char *what) { return set_error(st, std::string(fn) + ": " + what); }

// The layer's shape inside the plan: GC_OK and its columns.
gc_status check_layer(const char *fn, const gc_plan *plan, const gc_linear *l, uint64_t n, uint32_t *cols) {
    if (!plan || !l) return fail(fn, GC_EINVAL, "plan and layer must be non-null");
    if (l->reserved[0] || l->reserved[1]) return fail(fn, GC_EINVAL, "reserved must be 0");
    if (!known_type(l->type)) return fail(fn, GC_EINVAL, "type must be GC_F32, GC_BF16 or GC_F16");
    if (l->seg < 0 || l->seg >= plan->nseg) return fail(fn, GC_EINVAL, "seg is not a segment of the plan");
    const uint32_t len = plan->seg[l->seg].len;
    if (l->rows < 1 || len % l->rows) return fail(fn, GC_EINVAL, "rows must divide the segment's length");
    if (l->bias_seg < -1 || l->bias_seg >= plan->nseg || l->bias_seg == l->seg)
        return fail(fn, GC_EINVAL, "bias_seg must be another segment of the plan, or -1");
    if (l->bias_seg >= 0 && plan->seg[l->bias_seg].len != l->rows)
        return fail(fn, GC_EINVAL, "the bias' segment must have `rows` elements");
    *cols = len / l->rows;
    if (n >= kMaxTokens) return fail(fn, GC_ERANGE, "n_tokens must be < 2^28");
    if (n * std::max(l->rows, *cols) > kMaxElems) return fail(fn, GC_ERANGE, "n_tokens * max(rows, cols) must be <= 2^35");
    return GC_OK;
}

// An array of n rows of `cols` elements (required or not).
gc_status check_rows(const char *fn, const void *p, uint64_t stride, uint64_t n, uint64_t cols, int type, bool required) {
    if (!p) return required ? fail(fn, GC_EINVAL, "buffers must be non-null") : GC_OK;
    if (stride < cols) return fail(fn, GC_EINVAL, "a row stride must be at least the row's length");
    if (n > 1 && stride > (uint64_t(1) << 48) / n) return fail(fn, GC_ERANGE, "n_tokens * a stride must be <= 2^48");
    if (reinterpret_cast<uintptr_t>(p) % type_bytes(type)) return fail(fn, GC_EINVAL, "buffers must be aligned to their elements");
    return GC_OK;
}

constexpr int kTM = 128, kTN = 128, kWR = 2, kWC = 2;

template <Kind kKind>
gc_status launch(const char *fn, int type, const Product &p, hipStream_t stream) {
    const uint64_t tiles_m = ceil_div(p.M, kTM), tiles = tiles_m * ceil_div(p.N, kTN);
    if (tiles > max_grid(kWR * kWC * kWave)) return fail(fn, GC_ERANGE, "more workgroups than a launch has");
    auto go = [&](auto t) {
        using T = decltype(t);
        GC_LAUNCH("linear_product", stream,
                  linear_kernel<T, kKind, kTM, kTN, kWR, kWC><<<static_cast<unsigned>(tiles), kWR * kWC * kWave, 0, stream>>>(
                      p, static_cast<uint32_t>(tiles_m)));
    };
    if (type == GC_F32) go(F32{});
    else if (type == GC_BF16) go(BF16{});
    else go(F16{});
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? GC_OK : hip_error(e, fn);
}

size_t workspace_bytes(const gc_linear *, uint32_t, uint64_t) { return 256; }

const void *at_element(const void *base, uint64_t elem, int type) { return static_cast<const char *>(base) + elem * type_bytes(type); }

gc_status check_ws(const char *fn, const gc_linear *l, uint32_t cols, uint64_t n, const void *ws, size_t ws_bytes) {
    if (!ws) return fail(fn, GC_EINVAL, "ws must be non-null");
    if (ws_bytes < workspace_bytes(l, cols, n)) return fail(fn, GC_ECAPACITY, "workspace smaller than gc_linear_workspace_bytes");
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

extern "C" size_t gc_linear_workspace_bytes(const gc_plan *plan, const gc_linear *layer, uint64_t n_tokens) {
    clear_error();
    uint32_t cols = 0;
    if (check_layer("gc_linear_workspace_bytes", plan, layer, n_tokens, &cols) != GC_OK) return 0;
    return workspace_bytes(layer, cols, n_tokens);
}

extern "C" gc_status gc_linear_forward(const gc_plan *plan, const gc_linear *layer, const void *w, const void *x,
                                       uint64_t x_stride, uint64_t n_tokens, int act, const void *r, uint64_t r_stride,
                                       void *z, uint64_t z_stride, void *y, uint64_t y_stride, void *ws,
                                       size_t ws_bytes, hipStream_t stream) {
    static const char fn[] = "gc_linear_forward";
    clear_error();
    uint32_t cols = 0;
    GC_TRY(check_layer(fn, plan, layer, n_tokens, &cols));
    if (!known_act(act)) return fail(fn, GC_EINVAL, "unknown act");
    if (n_tokens == 0) return GC_OK;
    const int type = layer->type;
    const uint32_t rows = layer->rows;
    GC_TRY(check_rows(fn, w, cols, 1, cols, type, true));
    GC_TRY(check_rows(fn, x, x_stride, n_tokens, cols, type, true));
    GC_TRY(check_rows(fn, r, r_stride, n_tokens, rows, type, false));
    GC_TRY(check_rows(fn, z, z_stride, n_tokens, rows, type, false));
    GC_TRY(check_rows(fn, y, y_stride, n_tokens, rows, type, true));
    if (y == x || y == w || z == y || (z && (z == x || z == w || z == r)) || (r == y && r_stride != y_stride))
        return fail(fn, GC_EINVAL, "an output is another buffer of the call");
    GC_TRY(check_ws(fn, layer, cols, n_tokens, ws, ws_bytes));
    Product p{};
    p.A = x;
    p.lda = x_stride;
    p.B = at_element(w, plan->seg[layer->seg].off, type);
    p.ldb = cols;
    p.M = static_cast<uint32_t>(n_tokens);
    p.N = rows;
    p.K = cols;
    p.bias = layer->bias_seg >= 0 ? at_element(w, plan->seg[layer->bias_seg].off, type) : nullptr;
    p.add = r;
    p.ldadd = r_stride;
    p.zout = z;
    p.ldz = z_stride;
    p.out = y;
    p.ldout = y_stride;
    p.act = act;
    return launch<kForward>(fn, type, p, stream);
}

extern "C" gc_status gc_act_grad(const void *dy, uint64_t dy_stride, const void *z, uint64_t z_stride, int act, int type,
                                 uint64_t n_rows, uint64_t cols, void *dz, uint64_t dz_stride, hipStream_t stream) {
    static const char fn[] = "gc_act_grad";
    clear_error();
    if (!known_type(type)) return fail(fn, GC_EINVAL, "type must be GC_F32, GC_BF16 or GC_F16");
    if (!known_act(act)) return fail(fn, GC_EINVAL, "unknown act");
    if (n_rows >= kMaxTokens) return fail(fn, GC_ERANGE, "n_rows must be < 2^28");
    if (n_rows && cols > kMaxElems / n_rows) return fail(fn, GC_ERANGE, "n_rows * cols must be <= 2^35");
    if (n_rows == 0 || cols == 0) return GC_OK;
    GC_TRY(check_rows(fn, dy, dy_stride, n_rows, cols, type, true));
    GC_TRY(check_rows(fn, z, z_stride, n_rows, cols, type, true));
    GC_TRY(check_rows(fn, dz, dz_stride, n_rows, cols, type, true));
    if ((dz == dy && dz_stride != dy_stride) || (dz == z && dz_stride != z_stride))
        return fail(fn, GC_EINVAL, "dz in place of another array must have its stride");
    const uint64_t grid = ceil_div(n_rows * ceil_div(cols, 4), kBlock);
    if (grid > max_grid(kBlock)) return fail(fn, GC_ERANGE, "more workgroups than a launch has");
    auto go = [&](auto t) {
        GC_LAUNCH("act_grad", stream,
                  act_grad_kernel<decltype(t)><<<static_cast<unsigned>(grid), kBlock, 0, stream>>>(
                      dy, dy_stride, z, z_stride, act, n_rows, cols, dz, dz_stride));
    };
    if (type == GC_F32) go(F32{});
    else if (type == GC_BF16) go(BF16{});
    else go(F16{});
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? GC_OK : hip_error(e, fn);
}

extern "C" gc_status gc_linear_grad_input(const gc_plan *plan, const gc_linear *layer, const void *w, const void *dz,
                                          uint64_t dz_stride, uint64_t n_tokens, const void *a, uint64_t a_stride, int act,
                                          const void *z, uint64_t z_stride, void *dx, uint64_t dx_stride, void *dzx,
                                          uint64_t dzx_stride, void *ws, size_t ws_bytes, hipStream_t stream) {
    static const char fn[] = "gc_linear_grad_input";
    clear_error();
    uint32_t cols = 0;
    GC_TRY(check_layer(fn, plan, layer, n_tokens, &cols));
    if (!known_act(act)) return fail(fn, GC_EINVAL, "unknown act");
    if (n_tokens == 0) return GC_OK;
    const int type = layer->type;
    const uint32_t rows = layer->rows;
    if (!dx && !dzx) return fail(fn, GC_EINVAL, "dx or dzx must be non-null");
    GC_TRY(check_rows(fn, w, cols, 1, cols, type, true));
    GC_TRY(check_rows(fn, dz, dz_stride, n_tokens, rows, type, true));
    GC_TRY(check_rows(fn, a, a_stride, n_tokens, cols, type, false));
    GC_TRY(check_rows(fn, z, z_stride, n_tokens, cols, type, dzx && act != GC_ACT_NONE));
    GC_TRY(check_rows(fn, dx, dx_stride, n_tokens, cols, type, false));
    GC_TRY(check_rows(fn, dzx, dzx_stride, n_tokens, cols, type, false));
    for (const void *out : {static_cast<const void *>(dx), static_cast<const void *>(dzx)})
        if (out && (out == w || out == dz || out == z)) return fail(fn, GC_EINVAL, "an output is another buffer of the call");
    if (dx == dzx || (a && ((a == dx && a_stride != dx_stride) || (a == dzx && a_stride != dzx_stride))))
        return fail(fn, GC_EINVAL, "an output is another buffer of the call");
    GC_TRY(check_ws(fn, layer, cols, n_tokens, ws, ws_bytes));
    Product p{};
    p.A = dz;
    p.lda = dz_stride;
    p.B = at_element(w, plan->seg[layer->seg].off, type);
    p.ldb = cols;
    p.M = static_cast<uint32_t>(n_tokens);
    p.N = cols;
    p.K = rows;
    p.add = a;
    p.ldadd = a_stride;
    p.z = z;
    p.ldz = z_stride;
    p.out = dx;
    p.ldout = dx_stride;
    p.out2 = dzx;
    p.ldout2 = dzx_stride;
    p.act = act;
    return launch<kInput>(fn, type, p, stream);
}

extern "C" gc_status gc_linear_grad_weight(const gc_plan *plan, const gc_linear *layer, const void *dz, uint64_t dz_stride,
                                           const void *x, uint64_t x_stride, uint64_t n_tokens, float *g, int accumulate,
                                           void *ws, size_t ws_bytes, hipStream_t stream) {
    static const char fn[] = "gc_linear_grad_weight";
    clear_error();
    uint32_t cols = 0;
    GC_TRY(check_layer(fn, plan, layer, n_tokens, &cols));
    const int type = layer->type;
    const uint32_t rows = layer->rows;
    GC_TRY(check_rows(fn, g, cols, 1, cols, GC_F32, true));
    if (n_tokens) {
        GC_TRY(check_rows(fn, dz, dz_stride, n_tokens, rows, type, true));
        GC_TRY(check_rows(fn, x, x_stride, n_tokens, cols, type, true));
        if (g == dz || g == x) return fail(fn, GC_EINVAL, "an output is another buffer of the call");
    } else if (accumulate) {
        return GC_OK;
    }
    GC_TRY(check_ws(fn, layer, cols, n_tokens, ws, ws_bytes));
    Product p{};
    p.A = dz;
    p.lda = dz_stride;
    p.B = x;
    p.ldb = x_stride;
    p.M = rows;
    p.N = cols;
    p.K = static_cast<uint32_t>(n_tokens);
    p.out = g + plan->seg[layer->seg].off;
    p.ldout = cols;
    p.gbias = layer->bias_seg >= 0 ? g + plan->seg[layer->bias_seg].off : nullptr;
    p.accumulate = accumulate ? 1 : 0;
    return launch<kWeight>(fn, type, p, stream);
}
