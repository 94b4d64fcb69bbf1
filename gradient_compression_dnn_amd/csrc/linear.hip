// The product of a layer's weight matrix with a batch and its gradients
// (gc_linear_forward, gc_linear_grad_input, gc_linear_grad_weight), and the
// slope of an activation (gc_act_grad): the calls, their checks, and how a
// product is spread over the chip.  The kernels are in linear_kernels.hpp.
#include <algorithm>
#include <string>

#include "activations.hpp"
#include "linear.hpp"

namespace gc {

namespace {

// dz = dy act'(z): 8 elements a thread.  Memory bounds it: 8192 x 16384 bf16 147 us, 5.5 TB/s.
constexpr int kActCols = 8;
template <class T>
__global__ __launch_bounds__(kBlock) void act_grad_kernel(const void *dy, uint64_t ldy, const void *z, uint64_t ldz, int act,
                                                          uint64_t n, uint64_t cols, void *dz, uint64_t ldd) {
    const uint64_t vecs = ceil_div(cols, kActCols);
    const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kBlock + threadIdx.x;
    const uint64_t row = i / vecs, c = (i - row * vecs) * kActCols;
    if (row >= n) return;
    const uint32_t cnt = static_cast<uint32_t>(umin64(cols - c, kActCols));
    Cols<T, kActCols> g, at;
    g.load(dy, row * ldy + c, cnt);
    at.load(z, row * ldz + c, cnt);
    float t[kActCols];
#pragma unroll
    for (uint32_t u = 0; u < kActCols; ++u) t[u] = at.at(u);
    act_slopes<sizeof(typename T::Store) == 2>(act, t);
#pragma unroll
    for (uint32_t u = 0; u < kActCols; ++u) t[u] = g.at(u) * t[u];
    put_cols<T>(dz, row * ldd + c, cnt, t);
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

// ------------------------------------------------------------- the cut
// A product is cut into tiles, and where those do not fill the chip, into parts of the common index as well; the
// choice is the least of a model of the time.  Its costs are fitted to sweeps over shapes and parts of 59 products
// from 1 to 8,192 tokens, where it is within 13% of the fastest (us, bf16: 512 x 4096 x 4096, 128 tiles in 4 parts 30,
// in 2 32, in 8 39; 2048 x 4096 x 4096, 128 x 128 63 and 256 x 256 92; 8192 x 4096 x 16384, 1,152 and 944; the weight
// gradient of 4100 x 4100 with 1024 tokens, 1,089 tiles and 289: 59 and 74).
struct ShapeModel {
    TileShape shape;
    uint32_t tm, tn, slots;   // workgroups that run at once
    double stage16, stage32;  // us a stage of 128 bytes of k, with every slot busy; 0: not for the type
    double half16, half32;    // what is left of that with half of the slots busy at most
    uint32_t parts;           // at most
};
constexpr ShapeModel kShapes[] = {
    {kBig, Big::kTM, Big::kTN, 256, 2.0, 0.0, 1.0, 1.0, 1},  // in parts it was never the fastest
    {kMid, Mid::kTM, Mid::kTN, 512, 1.3, 1.7, 0.75, 1.0, 32},
    {kThin, Thin::kTM, Thin::kTN, 1024, 1.3, 3.0, 0.65, 0.65, 32},
};
constexpr double kTileUs = 3.0, kJoinUs = 2.0, kPartialBytesPerUs = 4e6;
constexpr uint32_t kThinTokens = 64;
constexpr uint64_t kFewRows = 1024, kFewOutputs = 1 << 16;

uint32_t stages_of(int type, uint32_t K) { return static_cast<uint32_t>(ceil_div(K, 128 / type_bytes(type))); }

// Whether a kind of product takes a shape.
bool takes(const ShapeModel &s, Kind kind, int type, uint32_t M, bool any) {
    if (any) return s.shape == kMid;
    if (s.shape == kThin) return kind != kWeight && M <= kThinTokens;
    return s.shape == kMid || type != GC_F32;
}

Cut plan_cut(Kind kind, int type, uint32_t M, uint32_t N, uint32_t K, bool any) {
    Cut best{};
    // Few tokens: every 16 rows of W read all of x, so a longer batch over many rows goes by tiles (us, few and
    // tiles: 1 x 16384 rows x 4096 columns 26 and 29, 16 x 4096 x 4096 10.0 and 11.7, 16 x 16384 x 4096 35 and 29).
    // Few rows of W as well leave most of the chip idle: 15 x 81 x 5398 18 and 7.6.
    if (kind == kForward && M <= 16 && (M <= 4 || (N >= kFewRows && static_cast<uint64_t>(M) * N <= kFewOutputs))) {
        const uint64_t chunks = ceil_div(static_cast<uint64_t>(K) * type_bytes(type), 256);
        best.shape = kFew;
        best.tiles_m = 1;
        best.tiles_n = static_cast<uint32_t>(ceil_div(N, 16));
        best.parts = 1;  // waves: 16 (26 us; 8 take 29, 4 take 30), or as many as have a chunk
        while (best.parts < 16 && best.parts < chunks) best.parts *= 2;
        return best;
    }
    double least = 0.0;
    const uint32_t stages = stages_of(type, K);
    for (const ShapeModel &s : kShapes) {
        if (!takes(s, kind, type, M, any)) continue;
        const uint64_t tm = ceil_div(M, s.tm), tn = ceil_div(N, s.tn), tiles = tm * tn;
        for (uint32_t parts = 1; parts <= std::min(s.parts, std::max(stages, 1u)); ++parts) {
            if (parts > 1 && tiles * parts > s.slots) break;
            const uint32_t per = static_cast<uint32_t>(ceil_div(stages, parts));
            if (parts > 1 && static_cast<uint64_t>(per) * (parts - 1) >= stages) continue;  // a part without stages
            const uint64_t rounds = ceil_div(tiles * parts, s.slots), last = tiles * parts - (rounds - 1) * s.slots;
            const double stage = type == GC_F32 ? s.stage32 : s.stage16, half = 2 * last > s.slots ? 1.0 : type == GC_F32 ? s.half32 : s.half16;
            double us = per * stage * (static_cast<double>(rounds - 1) + half) + kTileUs * static_cast<double>(rounds);
            if (parts > 1) us += kJoinUs + 2.0 * static_cast<double>(tiles * parts) * s.tm * s.tn * 4 / kPartialBytesPerUs;
            if (best.per == 0 || us < least) {
                least = us;
                best.shape = s.shape;
                best.tiles_m = static_cast<uint32_t>(tm);
                best.tiles_n = static_cast<uint32_t>(tn);
                best.parts = parts;
                best.stages = stages;
                best.per = std::max(per, 1u);
            }
        }
    }
    return best;
}

const ShapeModel &model_of(const Cut &c) { return kShapes[c.shape == kBig ? 0 : c.shape == kMid ? 1 : 2]; }

// Lays the parts' sums out in the workspace.
void cut_ws(Cut &c, void *ws) {
    if (c.parts == 1 || c.shape == kFew) return;
    const ShapeModel &s = model_of(c);
    WsCursor at(ws);
    c.partial = at.take<float>(static_cast<size_t>(c.tiles_m) * c.tiles_n * c.parts * s.tm * s.tn);
    c.colsums = at.take<float>(static_cast<size_t>(c.parts) * c.tiles_m * s.tm);
}

// Bytes that hold the parts of every batch of up to n tokens (a smaller one may be cut into more).
size_t workspace_bytes(const gc_linear *l, uint32_t cols, uint64_t n) {
    size_t most = 0;
    const uint32_t n32 = static_cast<uint32_t>(n);
    auto product = [&](Kind kind, uint32_t M, uint32_t N, uint32_t K) {
        const uint32_t stages = stages_of(l->type, K);
        for (const ShapeModel &s : kShapes) {
            const uint32_t parts = std::min(s.parts, stages);
            if (parts < 2 || !takes(s, kind, l->type, kind == kWeight ? M : 1, false)) continue;
            const uint64_t tiles = ceil_div(std::min(M, s.shape == kThin ? kThinTokens : M), s.tm) * ceil_div(N, s.tn);
            const uint64_t units = umin64(tiles * parts, s.slots);  // no more are ever cut
            WsCursor at(nullptr);
            (void)at.take<float>(units * s.tm * s.tn);
            (void)at.take<float>(units * s.tm);
            most = std::max(most, at.used);
        }
    };
    if (n) {
        product(kForward, n32, l->rows, cols);
        product(kInput, n32, cols, l->rows);
        product(kWeight, l->rows, cols, n32);
    }
    return most + 256;  // room to round the base up to 256 bytes
}

void *align256(void *p) {
    return reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(p) + 255) & ~uintptr_t(255));
}

// How an operand gets into LDS: straight where its 16-byte pieces start on 16
// bytes and, where k is slow, none crosses the end of a row; through registers
// where a row (k slow) or a sum has a piece at least and a stage's offsets fit 31 bits.
Mode mode_of(const void *p, uint64_t ld, bool slow, uint32_t extent, uint32_t K, int type) {
    const uint64_t size = type_bytes(type), piece = 16 / size;
    if ((slow ? extent : K) < piece || ld * size >= (uint64_t(1) << 31) / 256) return kAny;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0 && (!slow || extent * size % 16 == 0) ? kDirect : kHeld;
}

gc_status launch(const char *fn, Kind kind, int type, const Product &p, void *ws, hipStream_t stream) {
    const Mode mode = std::max(mode_of(p.A, p.lda, kind == kWeight, p.M, p.K, type), mode_of(p.B, p.ldb, kind != kForward, p.N, p.K, type));
    Cut c = plan_cut(kind, type, p.M, p.N, p.K, mode == kAny);
    c.mode = mode;
    const uint64_t groups = c.shape == kFew ? c.tiles_n : ceil_div(p.M, model_of(c).tm) * ceil_div(p.N, model_of(c).tn);
    if (groups > max_grid(1024)) return fail(fn, GC_ERANGE, "more workgroups than a launch has");
    cut_ws(c, align256(ws));
    if (type == GC_F32) return linear_launch<F32>(fn, kind, p, c, stream);
    if (type == GC_BF16) return linear_launch<BF16>(fn, kind, p, c, stream);
    return linear_launch<F16>(fn, kind, p, c, stream);
}

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
    return launch(fn, kForward, type, p, ws, stream);
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
    const uint64_t grid = ceil_div(n_rows * ceil_div(cols, kActCols), kBlock);
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
    p.z = dzx && act != GC_ACT_NONE ? z : nullptr;
    p.ldz = z_stride;
    p.out = dx;
    p.ldout = dx_stride;
    p.out2 = dzx;
    p.ldout2 = dzx_stride;
    p.act = act;
    return launch(fn, kInput, type, p, ws, stream);
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
    return launch(fn, kWeight, type, p, ws, stream);
}
