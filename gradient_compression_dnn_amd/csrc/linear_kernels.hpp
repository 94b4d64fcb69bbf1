// The kernels of the layer products, as templates over the storage type; each
// type has a translation unit of its own (linear_f32.hip, linear_bf16.hip,
// linear_f16.hip).
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
#pragma once

#include <type_traits>

#include "activations.hpp"
#include "linear.hpp"

namespace gc {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// --------------------------------------------------------------- products
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

// A stage of an fp32 operand as three bf16 planes (32 k): x = hi + mid + lo exactly, 8 bits each (hi cut, so that
// nothing overflows, mid rounded, so that lo has either sign; bits below 2^-133 are dropped).  Six of the nine
// products of two such sums are formed, all but those with 2^-21 of the whole at most, of either sign, where a
// rounding of the product would cost 2^-24.  6 bf16 matrix instructions take 96 cycles where fp32's own take 256.
// An Inf counts as a NaN.
//   k contiguous: [row][64 bytes], 16-byte part c at c ^ ((row >> 2) & 3);  k slow: as an operand of 16 bits
template <bool kSlow, int kTile>
struct Planes {
    static constexpr uint32_t kBytes = kTile * 64;  // a plane
    using Half = Operand<BF16, true, kTile>;
    // 4 elements' planes
    static __device__ __forceinline__ void split(u32x4 x, uint2 (&planes)[3]) {
        uint32_t h[4], m[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t b = x[e];
            h[e] = b & 0xFFFF0000u;
            const float r = dev_u2f(b) - dev_u2f(h[e]);  // NaN for an Inf: its sums are NaN, as Inf times a plane of 0 is
            m[e] = (dev_f2u(r) + 0x8000u) & 0xFFFF0000u;
            l[e] = dev_f2u(r - dev_u2f(m[e]));
        }
        auto pair = [](uint32_t high, uint32_t low) { return __builtin_amdgcn_perm(high, low, 0x07060302u); };
        planes[0] = make_uint2(pair(h[1], h[0]), pair(h[3], h[2]));
        planes[1] = make_uint2(pair(m[1], m[0]), pair(m[3], m[2]));
        planes[2] = make_uint2(pair(l[1], l[0]), pair(l[3], l[2]));
    }
    // into LDS: piece `piece` of line `line` (a row, or a k) of the fp32 operand
    static __device__ __forceinline__ void put(char *to, uint32_t line, uint32_t piece, const uint2 (&planes)[3]) {
        const uint32_t at = kSlow ? line * (kTile * 2) + ((piece >> 2) ^ Half::spread(line)) * 32 + (piece & 3) * 8
                                  : line * 64 + (((piece >> 1) ^ ((line >> 2) & 3)) << 4) + (piece & 1) * 8;
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<uint2 *>(to + q * kBytes + at) = planes[q];
    }
    // rows row0 .. row0 + 15 of a plane, 8 k a lane
    static __device__ __forceinline__ u32x4 read(const char *lds, uint32_t row0, int plane) {
        if (kSlow) return Half::read(lds + plane * kBytes, row0, 0);
        const uint32_t row = row0 + (lane_id() & 15), part = lane_id() >> 4;
        return *reinterpret_cast<const u32x4 *>(lds + plane * kBytes + row * 64 + ((part ^ ((row >> 2) & 3)) << 4));
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

// d + the sum of 16 bytes of elements
template <class T>
__device__ __forceinline__ float add_all(u32x4 a, float d) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t w = a[e];  // a value of its own: a bit cast of a vector's element took the first one
        if constexpr (sizeof(typename T::Store) == 4) d = d + dev_u2f(w);
        else if constexpr (std::is_same<T, BF16>::value)
            d = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, 0x3F803F80u), d, false);
        else d = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, w), __builtin_bit_cast(f16x2, 0x3C003C00u), d, false);
    }
    return d;
}

// What N sums of row m, columns n on (cnt of them exist), are combined with.
// Loaded before the first store: an output may stand where an input stood, so
// the compiler moves no load across a store by itself.
template <class T, Kind kKind, int N>
struct Beside {
    Cols<T, N> bias, add, z;
    Cols<F32, kKind == kWeight ? N : 0> g;
    __device__ __forceinline__ void load(const Product &p, uint32_t m, uint32_t n, uint32_t cnt) {
        if constexpr (kKind == kWeight) {
            if (p.accumulate) g.load(p.out, m * p.ldout + n, cnt);
        } else {
            if (kKind == kForward && p.bias) bias.load(p.bias, n, cnt);
            if (p.add) add.load(p.add, m * p.ldadd + n, cnt);
            if (kKind == kInput && p.z) z.load(p.z, m * p.ldz + n, cnt);
        }
    }
};

template <class T, Kind kKind, int N>
__device__ __forceinline__ void finish(const Product &p, const Beside<T, kKind, N> &o, uint32_t m, uint32_t n, uint32_t cnt, float (&v)[N]) {
    constexpr bool kFast = sizeof(typename T::Store) == 2;
    auto add = [&](const auto &x) {
#pragma unroll
        for (int u = 0; u < N; ++u) v[u] = x.at(u) + v[u];
    };
    if constexpr (kKind == kWeight) {
        if (p.accumulate) add(o.g);
        put_cols<F32>(p.out, m * p.ldout + n, cnt, v);
    } else if constexpr (kKind == kForward) {
        if (p.bias) add(o.bias);
        if (p.zout) put_cols<T>(p.zout, m * p.ldz + n, cnt, v);
        act_values<kFast>(p.act, v);
        if (p.add) add(o.add);
        put_cols<T>(p.out, m * p.ldout + n, cnt, v);
    } else {
        if (p.add) add(o.add);
        if (p.out) put_cols<T>(p.out, m * p.ldout + n, cnt, v);
        if (p.out2) {
            if (p.z) {
                float t[N];
#pragma unroll
                for (int u = 0; u < N; ++u) t[u] = o.z.at(u);
                act_slopes<kFast>(p.act, t);
#pragma unroll
                for (int u = 0; u < N; ++u) v[u] = v[u] * t[u];
            }
            put_cols<T>(p.out2, m * p.ldout2 + n, cnt, v);
        }
    }
}

template <class T, class S>
struct Shape : S {
    static constexpr int kWaves = S::kWR * S::kWC, kThreads = kWaves * int(kWave);
    static constexpr int kRA = S::kTM / S::kWR / 16, kRB = S::kTN / S::kWC / 16;  // blocks of 16 x 16 of a wave
    // kWide: fp32 by planes, one buffer of them; else two buffers of stages
    static constexpr bool kWide = sizeof(typename T::Store) == 4 && std::is_same<S, Mid>::value;
    static constexpr int kLine = kWide ? 192 : 128, kBytesA = S::kTM * kLine, kBytes = kBytesA + S::kTN * kLine;  // a stage
    static constexpr int kLds = kWide ? kBytes : 2 * kBytes;
    static constexpr int kLoadsA = S::kTM * 8 / kThreads, kLoadsB = S::kTN * 8 / kThreads;  // 16 bytes a thread each
    static_assert(S::kTM * 8 % kThreads == 0 && S::kTN * 8 % kThreads == 0, "every thread loads alike");
};

typedef __attribute__((address_space(1))) const char GlobalChar;
typedef __attribute__((address_space(3))) char LdsChar;

// x shifted down by `bits` (a multiple of an element's), zeros behind.
__device__ __forceinline__ u32x4 shift_down(u32x4 x, uint32_t bits) {
    return __builtin_bit_cast(u32x4, __builtin_bit_cast(unsigned __int128, x) >> bits);
}

// One operand's way into LDS: part i * kThreads + thread of a stage.
template <class T, Mode kMode, bool kWide, bool kSlow, int kTile, int kLoads, int kThreads>
struct Feed {
    using Op = Operand<T, kSlow, kTile>;
    using Store = typename T::Store;
    static constexpr uint32_t kSize = sizeof(Store), kElems = Op::kElems, kLineParts = kSlow ? Op::kRowParts : 8;
    static_assert(kThreads % kLineParts == 0, "a thread's parts are the same piece of different lines");
    const char *base;
    uint64_t step, ld;  // bytes to the next stage, and to the next row
    uint32_t row0, rows, K;
    // kRegular: a thread's parts are permuted alike, so they stand at equal distances in LDS and, where k is slow, in memory
    static constexpr uint32_t kLines = kThreads / kLineParts;
    static constexpr bool kRegular = kLines % 16 == 0;
    static constexpr int kPlaces = kSlow && kRegular ? 1 : kLoads;
    uint32_t at[kPlaces];   // from the stage's first byte
    u32x4 held[kLoads];
    uint2 planes[kWide ? kLoads : 1][3];

    // the line (row, or k) and the piece of it at a thread's part, as it is read from memory
    static __device__ __forceinline__ uint32_t line_of(int i) { return (i * kThreads + threadIdx.x) / kLineParts; }
    static __device__ __forceinline__ uint32_t piece_of() { return threadIdx.x % kLineParts; }

    __device__ __forceinline__ void init(const void *p, uint64_t stride, uint32_t first, uint32_t count, uint32_t k) {
        row0 = first;
        rows = count;
        K = k;
        ld = stride * kSize;
        base = static_cast<const char *>(p) + (kSlow ? 0 : row0 * ld);
        step = kSlow ? Op::kStage * ld : 128;
        const uint32_t ld32 = static_cast<uint32_t>(ld);
#pragma unroll
        for (int i = 0; i < kPlaces; ++i) {
            const uint32_t part = i * kThreads + threadIdx.x;
            uint32_t line = line_of(i), piece = piece_of();
            if (kMode == kDirect)  // the piece that stands at `part`: permuting a line's pieces twice leaves them as they were
                piece = (Op::place(part, line, piece) >> 4) - line * kLineParts;
            // rows past the last one repeat it, pieces past its end its last one: what they give is not kept
            if (kSlow) at[i] = line * ld32 + min(row0 + piece * kElems, rows - kElems) * kSize;
            else at[i] = min(line, rows - 1 - row0) * ld32 + piece * 16;
        }
    }
    __device__ __forceinline__ const char *part_of(const char *from, int i) const {
        return kPlaces == 1 ? from + i * (kLines * ld) + at[0] : from + at[kPlaces == 1 ? 0 : i];
    }
    // A whole stage, straight into LDS.
    __device__ __forceinline__ void direct(uint32_t s, char *__restrict__ to) const {
        const char *from = base + s * step;
        const uint32_t w = __builtin_amdgcn_readfirstlane(wave_id());
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            __builtin_amdgcn_global_load_lds((GlobalChar *)(part_of(from, i)), (LdsChar *)(to + (i * kThreads + w * kWave) * 16), 16, 0, 0);
    }
    // A stage into registers, and from there into LDS.
    __device__ __forceinline__ void fetch(uint32_t s) {
        if constexpr (kMode == kAny) {
            fetch_any(s);
        } else {
            const char *from = base + s * step;
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                held[i] = __builtin_bit_cast(u32x4, *reinterpret_cast<const Pack<Store, int(kElems)> *>(part_of(from, i)));
        }
    }
    __device__ __forceinline__ void put(char *to, int i, u32x4 x) const {
        if constexpr (kWide) {
            uint2 p[3];
            Planes<kSlow, kTile>::split(x, p);
            Planes<kSlow, kTile>::put(to, line_of(i), piece_of(), p);
            return;
        }
        uint32_t line, piece;
        const uint32_t where = kRegular ? Op::place(threadIdx.x, line, piece) + i * kThreads * 16 : Op::place(i * kThreads + threadIdx.x, line, piece);
        *reinterpret_cast<u32x4 *>(to + where) = x;
    }
    __device__ __forceinline__ void stash(char *to) const {
        if (kMode == kHeld && kSlow && row0 + kTile > rows) {  // the piece that ends with the row moves into place
            const uint32_t bits = over(row0, rows) * kSize * 8;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) put(to, i, shift_down(held[i], bits));
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) put(to, i, held[i]);
        }
    }
    // The same in steps, for kWide: pieces into their place, part i of the registers into planes, all planes into LDS.
    __device__ __forceinline__ void settle() {
        if (kMode == kHeld && kSlow && row0 + kTile > rows) {
            const uint32_t bits = over(row0, rows) * kSize * 8;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) held[i] = shift_down(held[i], bits);
        }
    }
    __device__ __forceinline__ void split(int i) { Planes<kSlow, kTile>::split(held[i], planes[i]); }
    __device__ __forceinline__ void put_planes(char *to) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) Planes<kSlow, kTile>::put(to, line_of(i), piece_of(), planes[i]);
    }
    // How many elements of this thread's piece lie past the end, less than all.
    __device__ __forceinline__ uint32_t over(uint32_t start, uint32_t end) const {
        const uint32_t first = start + piece_of() * kElems;
        return first < end && first + kElems > end ? first + kElems - end : 0;
    }
    // The stage with the last k inside, zeros past it.
    __device__ __forceinline__ void ragged(uint32_t s, char *to) {
        if constexpr (kMode == kAny) {
            fetch_any(s);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) put(to, i, held[i]);
        } else {
            const uint32_t k0 = s * Op::kStage;
            u32x4 x[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                // the piece that ends with the row, or the last k
                const uint32_t line = line_of(i);
                const uint32_t r = kSlow ? min(row0 + piece_of() * kElems, rows - kElems) : min(line, rows - 1 - row0);
                const uint32_t k = kSlow ? min(k0 + line, K - 1) : min(k0 + piece_of() * kElems, K - kElems);
                const char *p = kSlow ? base + k * ld + r * kSize : base + r * ld + uint64_t(k) * kSize;
                x[i] = __builtin_bit_cast(u32x4, *reinterpret_cast<const Pack<Store, int(kElems)> *>(p));
            }
            const uint32_t bits = (kSlow ? over(row0, rows) : over(k0, K)) * kSize * 8;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const bool none = kSlow ? k0 + line_of(i) >= K : k0 + piece_of() * kElems >= K;
                u32x4 v = shift_down(x[i], bits);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = none ? 0u : v[e];
                put(to, i, v);
            }
        }
    }

  private:
    __device__ __forceinline__ void fetch_any(uint32_t s) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t line = line_of(i), r = kSlow ? row0 + piece_of() * kElems : min(row0 + line, rows - 1);
            const uint32_t k = s * Op::kStage + (kSlow ? line : piece_of() * kElems), first = kSlow ? r : k, end = kSlow ? rows : K;
            const Store *p = reinterpret_cast<const Store *>((kSlow ? base : base - row0 * ld) + (kSlow ? k : r) * ld) + first;
            Pack<Store, int(kElems)> t;
#pragma unroll
            for (uint32_t u = 0; u < kElems; ++u) t.v[u] = first + u < end && k < K ? p[u] : Store(0);
            held[i] = __builtin_bit_cast(u32x4, t);
        }
    }
};

// Every wave of the workgroup is here and its LDS accesses are done; loads may be on their way.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <class T, Kind kKind, class S, Mode kMode>
struct Run {
    using C = Shape<T, S>;
    static constexpr bool kSlowA = kKind == kWeight, kSlowB = kKind != kForward;
    using OpA = Operand<T, kSlowA, C::kTM>;
    using OpB = Operand<T, kSlowB, C::kTN>;
    using FeedA = Feed<T, kMode, C::kWide, kSlowA, C::kTM, C::kLoadsA, C::kThreads>;
    using FeedB = Feed<T, kMode, C::kWide, kSlowB, C::kTN, C::kLoadsB, C::kThreads>;
    using Acc = f32x4[C::kRA][C::kRB];
    using Sums = float[C::kRA];  // a lane's part of the sums of A's rows over k

    // acc += a stage's product; blocks of A one ahead, and no further: hoisted, they do not fit the registers.
    // Where registers hold the next stage meanwhile, half of this one's k at a time.
    template <bool kSums, class Beneath>
    static __device__ __forceinline__ void multiply(const char *__restrict__ lds, uint32_t wm, uint32_t wn, Acc &acc, Sums &sums, Beneath beneath) {
        const char *la = lds, *lb = lds + C::kBytesA;
        if constexpr (C::kWide) {
            using PlanesA = Planes<kSlowA, C::kTM>;
            using PlanesB = Planes<kSlowB, C::kTN>;
            constexpr int kPairs[6][2] = {{1, 1}, {2, 0}, {0, 2}, {1, 0}, {0, 1}, {0, 0}};  // planes of B and A, the small products first
            u32x4 fb[3][C::kRB], fa[3], na[3];
#pragma unroll
            for (int q = 0; q < 3; ++q) {
#pragma unroll
                for (int b = 0; b < C::kRB; ++b) fb[q][b] = PlanesB::read(lb, wn + 16 * b, q);
                fa[q] = PlanesA::read(la, wm, q);
            }
#pragma unroll
            for (int a = 0; a < C::kRA; ++a) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int q = 0; q < 3; ++q) na[q] = a + 1 < C::kRA ? PlanesA::read(la, wm + 16 * (a + 1), q) : fa[q];
                beneath(a);
#pragma unroll
                for (int q = 0; q < 6; ++q)
#pragma unroll
                    for (int b = 0; b < C::kRB; ++b) acc[a][b] = mma<BF16>(fb[kPairs[q][0]][b], fa[kPairs[q][1]], acc[a][b]);
                if (kSums)
#pragma unroll
                    for (int q = 2; q >= 0; --q) sums[a] = add_all<BF16>(fa[q], sums[a]);
#pragma unroll
                for (int q = 0; q < 3; ++q) fa[q] = na[q];
                // a few vector instructions under each matrix instruction
#pragma unroll
                for (int q = 0; q < 6 * C::kRB; ++q) {
                    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            return;
        } else {
            constexpr int kTogether = kMode == kDirect ? 2 : 1;
#pragma unroll
            for (int h0 = 0; h0 < 2; h0 += kTogether) {
                u32x4 fb[kTogether][C::kRB], fa[kTogether], na[kTogether];
#pragma unroll
                for (int h = 0; h < kTogether; ++h) {
#pragma unroll
                    for (int b = 0; b < C::kRB; ++b) fb[h][b] = OpB::read(lb, wn + 16 * b, h0 + h);
                    fa[h] = OpA::read(la, wm, h0 + h);
                }
#pragma unroll
                for (int a = 0; a < C::kRA; ++a) {
#pragma unroll
                    for (int h = 0; h < kTogether; ++h) na[h] = a + 1 < C::kRA ? OpA::read(la, wm + 16 * (a + 1), h0 + h) : fa[h];
#pragma unroll
                    for (int h = 0; h < kTogether; ++h) {
#pragma unroll
                        for (int b = 0; b < C::kRB; ++b) acc[a][b] = mma<T>(fb[h][b], fa[h], acc[a][b]);
                        if (kSums) sums[a] = add_all<T>(fa[h], sums[a]);
                    }
#pragma unroll
                    for (int h = 0; h < kTogether; ++h) fa[h] = na[h];
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    }

    // The stage to come goes out, then this one is multiplied; the two are different buffers of LDS, which the
    // restrict parameters tell the compiler: without them it waits for the loads before it reads.
    template <bool kActive, bool kSums>
    static __device__ __forceinline__ void step_direct(const char *__restrict__ cur, char *__restrict__ next, const FeedA &fa, const FeedB &fb,
                                                       uint32_t s, bool load, uint32_t wm, uint32_t wn, Acc &acc, Sums &sums) {
        if (load) {
            fa.direct(s, next);
            fb.direct(s, next + C::kBytesA);
        }
        if (kActive) multiply<kSums>(cur, wm, wn, acc, sums, [](int) {});
    }

    // Stages s0 .. s1 - 1 of the tile.  kActive: the wave has rows and columns of the result.
    template <bool kActive, bool kSums>
    static __device__ __forceinline__ void stages(char *lds, FeedA &fa, FeedB &fb, uint32_t s0, uint32_t s1, uint32_t wm, uint32_t wn, Acc &acc,
                                                  Sums &sums) {
        const uint32_t whole = fa.K / OpA::kStage;  // stages without the last k inside
        // the one with it comes first, so that the loop has whole stages only
        const uint32_t ragged = s1 > whole ? 1 : 0, n = s1 - s0;
        if (ragged) {
            fa.ragged(whole, lds);
            fb.ragged(whole, lds + C::kBytesA);
        } else if (kMode == kDirect) {
            fa.direct(s0, lds);
            fb.direct(s0, lds + C::kBytesA);
        } else {
            fa.fetch(s0);
            fb.fetch(s0);
            fa.stash(lds);
            fb.stash(lds + C::kBytesA);
        }
        if constexpr (C::kWide) {
            // One buffer.  While stage i is multiplied, the next is split in registers, and the one behind it is
            // fetched into the registers that leaves.
            static_assert(C::kLoadsA == C::kRA && C::kLoadsB == C::kRA, "a part of each operand per row of blocks");
            const uint32_t last = s1 > whole ? whole - 1 : s1 - 1;  // the last whole stage; fetched again where there is no next
            auto fetch = [&](uint32_t i) {
                const uint32_t s = min(s0 + i - ragged, last);
                fa.fetch(s);
                fb.fetch(s);
            };
            if (n > 1) fetch(1);
            for (uint32_t i = 0; i < n; ++i) {
                const bool more = i + 1 < n;
                lds_barrier();
                fa.settle();
                fb.settle();
                auto beneath = [&](int a) {
                    fa.split(a);
                    fb.split(a);
                };
                if (kActive) multiply<kSums>(lds, wm, wn, acc, sums, beneath);
                else
#pragma unroll
                    for (int a = 0; a < C::kRA; ++a) beneath(a);
                if (more) fetch(i + 2);
                lds_barrier();
                if (more) {
                    fa.put_planes(lds);
                    fb.put_planes(lds + C::kBytesA);
                }
            }
            return;
        }
        for (uint32_t i = 0; i < n; ++i) {
            // this stage has landed, and every wave is done with the buffer that is filled next
            if (kMode == kDirect) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            const uint32_t cur = (i & 1) * C::kBytes, next = C::kBytes - cur, s = s0 + i + 1 - ragged;
            const bool more = i + 1 < n;
            if (kMode == kDirect) {
                step_direct<kActive, kSums>(lds + cur, lds + next, fa, fb, s, more, wm, wn, acc, sums);
            } else {
                if (more) {
                    fa.fetch(s);
                    fb.fetch(s);
                }
                if (kActive) multiply<kSums>(lds + cur, wm, wn, acc, sums, [](int) {});
                if (more) {
                    fa.stash(lds + next);
                    fb.stash(lds + next + C::kBytesA);
                }
            }
        }
    }

    // The sums of kRows rows of the wave (blocks a0 on) by way of LDS, so that a lane gets 8 columns of a row and
    // the code of an epilogue stands there once.  Pieces of 4 columns are permuted against bank conflicts.
    static constexpr int kCols = C::kRB * 16, kRows = C::kRA < 4 ? C::kRA * 16 : C::kWide ? 32 : 64, kWaveBytes = kRows * kCols * 4;
    static_assert(C::kWaves * kWaveBytes <= C::kLds, "a block of results per wave");
    static __device__ __forceinline__ uint32_t block_at(uint32_t row, uint32_t piece) {
        return row * (kCols * 4) + ((piece ^ (row & (kCols / 4 - 1))) << 4);
    }
    static __device__ __forceinline__ void write_out(const Product &p, char *block, uint32_t m0, uint32_t n0, const Acc &acc) {
        const uint32_t lane = lane_id();
#pragma unroll
        for (int a0 = 0; a0 < C::kRA; a0 += kRows / 16) {
#pragma unroll
            for (int a = 0; a < kRows / 16; ++a)
#pragma unroll
                for (int b = 0; b < C::kRB; ++b)
                    *reinterpret_cast<f32x4 *>(block + block_at(16 * a + (lane & 15), 4 * b + (lane >> 4))) = acc[a0 + a][b];
            constexpr uint32_t kLanes = kCols / 8, kStep = kWave / kLanes, kAhead = 4;  // lanes a row, rows at a time, times loaded ahead
            static_assert(kRows % (kStep * kAhead) == 0 || kRows / kStep < kAhead, "whole batches");
            constexpr uint32_t kBatch = kRows / kStep < kAhead ? kRows / kStep : kAhead;
            const uint32_t c = lane % kLanes, n = n0 + 8 * c, cnt = n < p.N ? min(p.N - n, 8u) : 0;
#pragma unroll 1
            for (uint32_t r0 = lane / kLanes; r0 < kRows; r0 += kStep * kBatch) {
                Beside<T, kKind, 8> beside[kBatch];
#pragma unroll
                for (uint32_t i = 0; i < kBatch; ++i) {
                    const uint32_t m = m0 + 16 * a0 + r0 + i * kStep;
                    if (m < p.M && cnt) beside[i].load(p, m, n, cnt);
                }
#pragma unroll
                for (uint32_t i = 0; i < kBatch; ++i) {
                    const uint32_t r = r0 + i * kStep, m = m0 + 16 * a0 + r;
                    const f32x4 lo = *reinterpret_cast<const f32x4 *>(block + block_at(r, 2 * c));
                    const f32x4 hi = *reinterpret_cast<const f32x4 *>(block + block_at(r, 2 * c + 1));
                    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                    if (m < p.M && cnt) finish<T, kKind, 8>(p, beside[i], m, n, cnt, v);
                }
            }
        }
    }
    // The same straight from the registers, for fp32 results of whole blocks: a lane holds 16 bytes of row
    // lane % 16 of each.
    static __device__ __forceinline__ void write_blocks(const Product &p, uint32_t m0, uint32_t n0, const Acc &acc) {
        constexpr int kAhead = C::kRA < 4 ? C::kRA : 4;  // rows of blocks whose old values are on their way at once
        const uint32_t m = m0 + (lane_id() & 15), n = n0 + 4 * (lane_id() >> 4);
#pragma unroll
        for (int a0 = 0; a0 < C::kRA; a0 += kAhead) {
            Beside<T, kKind, 4> beside[kAhead][C::kRB];
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
#pragma unroll
                for (int b = 0; b < C::kRB; ++b) beside[a][b].load(p, m + 16 * (a0 + a), n + 16 * b, 4);
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
#pragma unroll
                for (int b = 0; b < C::kRB; ++b) {
                    float v[4] = {acc[a0 + a][b][0], acc[a0 + a][b][1], acc[a0 + a][b][2], acc[a0 + a][b][3]};
                    finish<T, kKind, 4>(p, beside[a][b], m + 16 * (a0 + a), n + 16 * b, 4, v);
                }
        }
    }
};

// Workgroups go to the 8 XCDs in turn; each XCD gets consecutive ones of this order.
__device__ __forceinline__ uint32_t xcd_order(uint32_t id, uint32_t count) {
    const uint32_t x = id & 7, q = count >> 3, r = count & 7;
    return x * q + min(x, r) + (id >> 3);
}

// Tile t: columns of up to 8 tiles along m, so that the tiles at work at one time share rows of both operands.
constexpr uint32_t kGroupTiles = 8;
__device__ __forceinline__ void tile_of(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, uint32_t &tm, uint32_t &tn) {
    const uint32_t g = t / (kGroupTiles * tiles_n), rest = t - g * (kGroupTiles * tiles_n);
    const uint32_t high = min(kGroupTiles, tiles_m - g * kGroupTiles);
    tn = rest / high;
    tm = g * kGroupTiles + rest - tn * high;
}

// A tile a workgroup, or a part of its sum.  Both operands come through LDS in stages of 128 bytes of k, the next
// one on its way while this one is multiplied; a wave keeps its block of the result in registers, and the epilogue
// is applied to the fp32 sums before the one rounding.
//   Matrix instructions bound long batches, at the clock that the card holds under them (1.8 GHz, 53% of the cycles
//   busy, a third of the waves' time at the stages' barriers).  bf16, us: 8192 x 4096 x 16384 by 256 x 256 (8 waves,
//   one workgroup a unit) 870 to 945, 1.16 to 1.26 PFLOP/s, where the library's product takes 711 to 905 by its
//   operands' order; 2048 x 4096 x 4096 by 128 x 128 (4 waves, two a unit) 63, the library 57.  Four waves of 128 x
//   128 each took 920 to 1,050, stages of 64 bytes in four buffers 910 to 990.  What an epilogue reads and writes is
//   not hidden behind other tiles' products: GELU and z add 25, a residual, z, dx and dzx 215.
//   Operands whose rows are not aligned to 16 bytes go through registers (us, and with aligned ones: 1023 x 4099 x
//   1501 fp16 31 and 26, 700 x 10000 x 1500 bf16 41 and 37; two stages on their way at once made no difference).
//   fp32 by planes: 2048 x 4096 x 4096 330 us, 208 TFLOP/s, 1.25 PFLOP/s of the bf16 products that are formed; by
//   fp32's own instructions 154 TFLOP/s at most.
template <class T, Kind kKind, class S, Mode kMode>
__global__ __launch_bounds__((Shape<T, S>::kThreads), S::kWavesPerSimd) void linear_kernel(Product p, Cut c) {
    using R = Run<T, kKind, S, kMode>;
    using C = Shape<T, S>;
    __shared__ __attribute__((aligned(128))) char lds[C::kLds];
    const uint32_t id = xcd_order(blockIdx.x, gridDim.x), tiles = c.tiles_m * c.tiles_n;
    const uint32_t part = id / tiles, tile = id - part * tiles;
    uint32_t tm, tn;
    tile_of(tile, c.tiles_m, c.tiles_n, tm, tn);
    const uint32_t m0 = tm * C::kTM, n0 = tn * C::kTN;
    const uint32_t w = __builtin_amdgcn_readfirstlane(wave_id()), lane = lane_id();
    const uint32_t wm = w / C::kWC * (C::kRA * 16), wn = w % C::kWC * (C::kRB * 16);
    typename R::Acc acc;
    typename R::Sums sums;
#pragma unroll
    for (int a = 0; a < C::kRA; ++a) {
        sums[a] = 0.0f;
#pragma unroll
        for (int b = 0; b < C::kRB; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const uint32_t s0 = part * c.per, s1 = min(s0 + c.per, c.stages);
    // the sums of A over k, for the bias: in the first column of tiles
    const bool bias = kKind == kWeight && p.gbias && tn == 0 && wn == 0;
    const bool active = m0 + wm < p.M && n0 + wn < p.N;
    if (s0 < s1) {
        typename R::FeedA fa;
        typename R::FeedB fb;
        fa.init(p.A, p.lda, m0, p.M, p.K);
        fb.init(p.B, p.ldb, n0, p.N, p.K);
        if (!active) R::template stages<false, false>(lds, fa, fb, s0, s1, wm, wn, acc, sums);
        else if (kKind == kWeight && bias) R::template stages<true, kKind == kWeight>(lds, fa, fb, s0, s1, wm, wn, acc, sums);
        else R::template stages<true, false>(lds, fa, fb, s0, s1, wm, wn, acc, sums);
    }
    if (bias && active)
#pragma unroll
        for (int a = 0; a < C::kRA; ++a) {  // the four lanes of a row
            sums[a] = sums[a] + __shfl_xor(sums[a], 16, kWave);
            sums[a] = sums[a] + __shfl_xor(sums[a], 32, kWave);
        }
    if (c.parts > 1) {
        if (!active) return;
        f32x4 *to = reinterpret_cast<f32x4 *>(c.partial + static_cast<uint64_t>(id) * (C::kTM * C::kTN)) + w * (C::kRA * C::kRB * kWave) + lane;
#pragma unroll
        for (int a = 0; a < C::kRA; ++a) {
            if (bias && lane < 16) c.colsums[static_cast<uint64_t>(part) * c.tiles_m * C::kTM + m0 + wm + 16 * a + lane] = sums[a];
#pragma unroll
            for (int b = 0; b < C::kRB; ++b) to[(a * C::kRB + b) * kWave] = acc[a][b];
        }
        return;
    }
    if (bias && active && lane < 16)
#pragma unroll
        for (int a = 0; a < C::kRA; ++a) {
            const uint32_t m = m0 + wm + 16 * a + lane;
            if (m < p.M) p.gbias[m] = p.accumulate ? p.gbias[m] + sums[a] : sums[a];
        }
    __syncthreads();  // the last stage has been read
    if (!active) return;
    if constexpr (kKind == kWeight)
        if (m0 + wm + C::kRA * 16 <= p.M && n0 + wn + C::kRB * 16 <= p.N) {
            R::write_blocks(p, m0 + wm, n0 + wn, acc);
            return;
        }
    R::write_out(p, lds + w * R::kWaveBytes, m0 + wm, n0 + wn, acc);
}

// The parts' sums added in order: a workgroup per 4 blocks of 16 x 16 of a tile.  Memory, or the caches, bound it:
// 480 parts of 64 KiB, 9 us.
template <class T, Kind kKind, class S>
__global__ __launch_bounds__(kBlock) void linear_join_kernel(Product p, Cut c) {
    using C = Shape<T, S>;
    constexpr uint32_t kBlocks = C::kWaves * C::kRA * C::kRB, kPer = kBlocks / kWaves;
    const uint32_t tiles = c.tiles_m * c.tiles_n, tile = blockIdx.x / kPer;
    const uint32_t block = (blockIdx.x - tile * kPer) * kWaves + __builtin_amdgcn_readfirstlane(wave_id()), lane = lane_id();
    const uint32_t w = block / (C::kRA * C::kRB), a = block / C::kRB % C::kRA, b = block % C::kRB;
    uint32_t tm, tn;
    tile_of(tile, c.tiles_m, c.tiles_n, tm, tn);
    const uint32_t m = tm * C::kTM + w / C::kWC * (C::kRA * 16) + 16 * a + (lane & 15);
    const uint32_t wn = w % C::kWC * (C::kRB * 16), n = tn * C::kTN + wn + 16 * b + 4 * (lane >> 4);
    if (m >= p.M) return;
    if (kKind == kWeight && p.gbias && tn == 0 && wn == 0 && b == 0 && lane < 16) {
        float v = 0.0f;
        for (uint32_t part = 0; part < c.parts; ++part) v = v + c.colsums[static_cast<uint64_t>(part) * c.tiles_m * C::kTM + m];
        p.gbias[m] = p.accumulate ? p.gbias[m] + v : v;
    }
    if (n >= p.N) return;
    const f32x4 *from = reinterpret_cast<const f32x4 *>(c.partial + static_cast<uint64_t>(tile) * (C::kTM * C::kTN)) + block * kWave + lane;
    Beside<T, kKind, 4> beside;
    beside.load(p, m, n, min(p.N - n, 4u));
    f32x4 v = from[0];
#pragma unroll 4
    for (uint32_t part = 1; part < c.parts; ++part) {
        const f32x4 t = from[part * static_cast<uint64_t>(tiles) * (C::kTM * C::kTN / 4)];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = v[u] + t[u];
    }
    float x[4] = {v[0], v[1], v[2], v[3]};
    finish<T, kKind, 4>(p, beside, m, n, min(p.N - n, 4u), x);
}

// Up to 16 tokens: a workgroup has 16 rows of W, its waves take chunks of 256 bytes of k in turn, straight from
// memory into matrix operands, the next chunk on its way meanwhile, and their sums are added in order.  W is
// read once, at memory's rate (us, 1 x 4096 x 16384: bf16 26.5, 5.1 TB/s, fp32 56, 4.8 TB/s; x 4096 x 4096 bf16, 2 to
// 16 tokens 8.6 to 11.1, where W alone takes 6.6), and nothing is launched behind it.
template <class T>
__global__ __launch_bounds__(16 * kWave) void linear_few_kernel(Product p) {
    using Store = typename T::Store;
    constexpr uint32_t kElems = 16 / sizeof(Store), kStep = 4 * kElems, kSteps = 4, kChunk = kSteps * kStep;  // elements of k
    extern __shared__ __attribute__((aligned(16))) f32x4 sums[];  // [waves][64]
    const uint32_t lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id()), waves = blockDim.x / kWave;
    const uint32_t n0 = blockIdx.x * 16, at = (lane >> 4) * kElems;
    const Store *wrow = static_cast<const Store *>(p.B) + min(n0 + (lane & 15), p.N - 1) * p.ldb;
    const Store *xrow = static_cast<const Store *>(p.A) + min(lane & 15, p.M - 1) * p.lda;
    auto whole = [](const Store *q) { return __builtin_bit_cast(u32x4, *reinterpret_cast<const Pack<Store, int(kElems)> *>(q)); };
    // the piece at k of the step with the last k: the row's last piece, moved into place
    auto part = [&](const Store *q, uint32_t k) {
        if (p.K < kElems) {
            Pack<Store, int(kElems)> t;
#pragma unroll
            for (uint32_t u = 0; u < kElems; ++u) t.v[u] = k + u < p.K ? q[k + u] : Store(0);
            return __builtin_bit_cast(u32x4, t);
        }
        const u32x4 x = whole(q + min(k, p.K - kElems));
        const uint32_t over = k + kElems > p.K ? k + kElems - p.K : 0;
        u32x4 v = shift_down(x, over < kElems ? over * uint32_t(sizeof(Store)) * 8 : 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = over < kElems ? v[e] : 0u;
        return v;
    };
    const uint32_t chunks = p.K / kChunk;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 fw[kSteps], fx[kSteps], nw[kSteps], nx[kSteps];
    auto fetch = [&](uint32_t c, u32x4(&a)[kSteps], u32x4(&b)[kSteps]) {
        const uint32_t k = c * kChunk + at;
#pragma unroll
        for (uint32_t s = 0; s < kSteps; ++s) a[s] = whole(wrow + k + s * kStep);
#pragma unroll
        for (uint32_t s = 0; s < kSteps; ++s) b[s] = whole(xrow + k + s * kStep);
    };
    if (w < chunks) fetch(w, fw, fx);
    for (uint32_t c = w; c < chunks; c += waves) {
        fetch(c + waves < chunks ? c + waves : c, nw, nx);
#pragma unroll
        for (uint32_t s = 0; s < kSteps; ++s) acc = mma<T>(fw[s], fx[s], acc);
#pragma unroll
        for (uint32_t s = 0; s < kSteps; ++s) {
            fw[s] = nw[s];
            fx[s] = nx[s];
        }
    }
    for (uint32_t k = chunks * kChunk, s = chunks; k < p.K; k += kStep, ++s)  // the rest, a step a wave
        if (s % waves == w) acc = mma<T>(part(wrow, k + at), part(xrow, k + at), acc);
    sums[w * kWave + lane] = acc;
    __syncthreads();
    // a lane's 4 sums: columns n0 + 4 (lane / 16) on of token lane % 16
    const uint32_t m = lane & 15, n = n0 + 4 * (lane >> 4);
    if (w || m >= p.M || n >= p.N) return;
    const uint32_t cnt = min(p.N - n, 4u);
    Beside<T, kForward, 4> beside;
    beside.load(p, m, n, cnt);
    for (uint32_t x = 1; x < waves; ++x) {
        const f32x4 t = sums[x * kWave + lane];
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[u] = acc[u] + t[u];
    }
    float y[4] = {acc[0], acc[1], acc[2], acc[3]};
    finish<T, kForward, 4>(p, beside, m, n, cnt, y);
}

template <class T, Kind kKind, class S>
gc_status launch_shape(const char *fn, const Product &p, const Cut &c, hipStream_t stream) {
    using C = Shape<T, S>;
    const unsigned grid = c.tiles_m * c.tiles_n * c.parts;
    auto kernel = linear_kernel<T, kKind, S, kHeld>;
    if constexpr (!C::kWide)
        if (c.mode == kDirect) kernel = linear_kernel<T, kKind, S, kDirect>;
    if constexpr (std::is_same<S, Mid>::value)
        if (c.mode == kAny) kernel = linear_kernel<T, kKind, S, kAny>;
    GC_LAUNCH("linear_product", stream, kernel<<<grid, C::kThreads, 0, stream>>>(p, c));
    if constexpr (!std::is_same<S, Big>::value) {  // whole tiles only
        if (c.parts > 1) {
            const unsigned joins = c.tiles_m * c.tiles_n * (C::kWaves * C::kRA * C::kRB / kWaves);
            GC_LAUNCH("linear_join", stream, linear_join_kernel<T, kKind, S><<<joins, kBlock, 0, stream>>>(p, c));
        }
    }
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? GC_OK : hip_error(e, fn);
}

template <class T>
gc_status linear_launch(const char *fn, Kind kind, const Product &p, const Cut &c, hipStream_t stream) {
    auto of = [&](auto shape) {
        using S = decltype(shape);
        if (kind == kForward) return launch_shape<T, kForward, S>(fn, p, c, stream);
        if (kind == kInput) return launch_shape<T, kInput, S>(fn, p, c, stream);
        return launch_shape<T, kWeight, S>(fn, p, c, stream);
    };
    if (c.shape == kFew) {
        GC_LAUNCH("linear_few", stream,
                  linear_few_kernel<T><<<c.tiles_n, c.parts * kWave, c.parts * kWave * sizeof(f32x4), stream>>>(p));
        const hipError_t e = hipGetLastError();
        return e == hipSuccess ? GC_OK : hip_error(e, fn);
    }
    if constexpr (sizeof(typename T::Store) == 2)
        if (c.shape == kBig) return of(Big{});
    if (c.shape == kMid || kind == kWeight) return of(Mid{});
    if (kind == kForward) return launch_shape<T, kForward, Thin>(fn, p, c, stream);
    return launch_shape<T, kInput, Thin>(fn, p, c, stream);
}

}  // namespace gc
