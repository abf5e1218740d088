// Host side of the linear layers in 8 bits: argument checks, the choice of tiles and
// splits, and the launches behind muonstep_linear8.h.
#include <algorithm>
#include <cstring>

#include "../../include/muonstep_linear8.h"
#include "head.h"
#include "host.h"
#include "linear8.h"

namespace muon {
namespace {

static_assert(MUON_BLOCK8 == kBlock8 && MUON_SCALE8_LOW == kScale8Low, "format");
static_assert(MUON_T_BF16 == kTypeBf16 && MUON_T_FP16 == kTypeFp16 && MUON_T_FP32 == kTypeFp32, "types");
static_assert(MUON_ACT_RELU2 == kActRelu2 && MUON_ACT_SILU == kActSilu && MUON_ACT_GELU == kActGelu, "functions");

constexpr int kCus = 256;
constexpr int64_t kFar = (int64_t)1 << 22;     // strides up to here: 256 rows apart fits 32 bits of bytes

int64_t ceil_div(int64_t x, int64_t m) { return (x + m - 1) / m; }
int64_t round_up(int64_t x, int64_t m) { return ceil_div(x, m) * m; }
int64_t size_of(int dtype) { return dtype == MUON_T_FP32 ? 4 : 2; }
Blocks8 blocks(const blocks8_t& b) {
    return {static_cast<uint8_t*>(b.codes), static_cast<uint8_t*>(b.scale), b.stride, b.scale_stride};
}
// Rows of 16-byte chunks.
bool whole_rows(const void* p, int64_t stride, int64_t size) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * size % 16 == 0;
}
// Whether the row-wise passes write a 16 or 32-bit result through the L2 (Through in linear8.h).  Not where an
// instruction's pieces leave no whole lines: float32, of which it holds 16 of every 32 bytes (relu2's backward of
// 8192 x 4096 105 us, by ordinary stores 59, with an encoding of the result behind it 128 and 81), and not large
// results whose rows lie off the 128-byte grid (bfloat16 / float16, us through the L2 and by ordinary stores):
//     25152 x 1000    29.8, 29.7 / 22.6, 24.0       50304 x 1000    64.4, 60.4 / 49.8, 46.9
//     134208 x 1000    170,  153 /  129,  114
// On the grid the two are within a per cent, and small results up to 1 us quicker through the L2.  Past the last cache
// too is no better where a reader follows: 16384 x 4096 decoded to bfloat16 and encoded 69 us (63), the backward pass of
// 16384 x 4096 with both products behind it 247 to 254 us either way.
constexpr int64_t kRaggedBytes = (int64_t)64 << 20;
bool through(const void* p, int64_t rows, int64_t dim, int64_t stride, int dtype) {
    if (dtype == MUON_T_FP32 || !whole_rows(p, stride, 2)) return false;
    const bool lines = reinterpret_cast<uintptr_t>(p) % 128 == 0 && stride * 2 % 128 == 0;
    return lines || rows * dim * 2 < kRaggedBytes;
}

// Checks of one call: each returns its first failure's code, and the next ones return it too.
struct Checks {
    const char* entry;
    int rc = MUON_OK;
    Span read[8], written[8];        // no entry has more
    int reads = 0, writes = 0;

    explicit Checks(const char* name) : entry(name) {}
    void sizes(int64_t rows, int64_t cols, int64_t dim) {
        if (rc) return;
        if (rows < 0 || cols < 1 || dim < 1)
            rc = fail(MUON_ERR_INVALID_ARG, "%s: rows = %lld, cols = %lld, dim = %lld: rows >= 0, cols and dim >= 1", entry,
                      (long long)rows, (long long)cols, (long long)dim);
        else if (rows > MUON_LINEAR8_MAX_ROWS || cols > MUON_LINEAR8_MAX_DIM || dim > MUON_LINEAR8_MAX_DIM)
            rc = fail(MUON_ERR_UNSUPPORTED, "%s: rows = %lld, cols = %lld, dim = %lld beyond the limits", entry, (long long)rows,
                      (long long)cols, (long long)dim);
    }
    void one_of(const char* what, int64_t value, int64_t last) {
        if (!rc && (value < 0 || value > last)) rc = fail(MUON_ERR_INVALID_ARG, "%s: %s = %lld", entry, what, (long long)value);
    }
    void strides(const char* what, int64_t stride, int64_t dim) {
        if (rc) return;
        if (stride < dim) rc = fail(MUON_ERR_INVALID_ARG, "%s: stride of %s smaller than its rows' %lld", entry, what, (long long)dim);
        else if (stride > kFar) rc = fail(MUON_ERR_UNSUPPORTED, "%s: stride of %s beyond 2^22", entry, what);
    }
    void buffer(const char* what, const void* p, int64_t bytes, int64_t align, bool writable) {
        if (rc || bytes <= 0) return;
        if (!p) {
            rc = fail(MUON_ERR_INVALID_ARG, "%s: %s must be non-NULL", entry, what);
            return;
        }
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (lo % align) {
            rc = fail(MUON_ERR_INVALID_ARG, "%s: %s is not %lld-byte aligned", entry, what, (long long)align);
            return;
        }
        (writable ? written[writes++] : read[reads++]) = {lo, lo + (uintptr_t)bytes, 0};
    }
    void matrix(const char* what, const void* p, int64_t rows, int64_t dim, int64_t stride, int64_t size, bool writable) {
        strides(what, stride, dim);
        buffer(what, p, rows > 0 ? ((rows - 1) * stride + dim) * size : 0, size, writable);
    }
    // tall: rows that share a scale
    void coded(const char* what, const blocks8_t& b, int64_t rows, int64_t dim, int64_t tall, bool writable) {
        if (rc) return;
        const int64_t wide = round_up(dim, 16), across = ceil_div(dim, MUON_BLOCK8), down = ceil_div(rows, tall);
        if (b.stride < wide || b.stride % 16 || b.scale_stride < across || b.scale_stride % 4) {
            rc = fail(MUON_ERR_INVALID_ARG, "%s: strides of %s: codes' a multiple of 16 >= %lld, scales' a multiple of 4 >= %lld",
                      entry, what, (long long)wide, (long long)across);
            return;
        }
        if (b.stride > kFar || b.scale_stride > kFar) {
            rc = fail(MUON_ERR_UNSUPPORTED, "%s: stride of %s beyond 2^22", entry, what);
            return;
        }
        buffer(what, b.codes, rows > 0 ? (rows - 1) * b.stride + wide : 0, 16, writable);
        // read in words of 4 scales
        buffer(what, b.scale, down > 0 ? (down - 1) * b.scale_stride + (writable ? across : round_up(across, 4)) : 0, 4, writable);
    }
    // what is written overlaps nothing else
    int done() {
        if (rc) return rc;
        for (int i = 0; i < writes; ++i) {
            auto meets = [&](const Span& x) { return written[i].lo < x.hi && x.lo < written[i].hi; };
            for (int j = 0; j < reads; ++j)
                if (meets(read[j])) return fail(MUON_ERR_UNSUPPORTED, "%s: an output overlaps an input", entry);
            for (int j = 0; j < i; ++j)
                if (meets(written[j])) return fail(MUON_ERR_UNSUPPORTED, "%s: two outputs overlap", entry);
        }
        return MUON_OK;
    }
};

#define LINEAR8_TRY(name, call)                                                                                 \
    do {                                                                                                        \
        const hipError_t err_ = timed_launch(name, s, [&] { return call; });                                    \
        if (err_ != hipSuccess) return fail(MUON_ERR_HIP, "%s launch failed: %s", name, hipGetErrorString(err_)); \
    } while (0)

Rows8 rows8(int64_t rows, int64_t dim) {
    Rows8 r;
    memset(&r, 0, sizeof(r));
    r.rows = rows;
    r.dim = (int)dim;
    return r;
}

// ---------------------------------------------------------------- the product
// Launches' names in messages and in the profiling hook, by Matmul8Variant.
const char* const kMatmulNames[] = {"matmul8_rows", "matmul8_32", "matmul8_64", "matmul8_128", "matmul8_256", "matmul8_exact_64",
                                    "matmul8_exact_128"};
struct MatmulPlan {
    int variant, tile_v, tile_t, splits, stages;     // stages of a split
    int64_t bytes;
};
// Up to 16 rows one kernel; beyond, what a linear estimate of the time says is least: a start, for
// each round of 256 workgroups the stages of K and the tile's ends, and for a split K the partial sums.  The constants are
// fitted to these times (us, before results passed the L2, which takes 0 to 2 us off each; rows x cols x dim, tiles of
// 32 / 64 / 128 / 256, K split where the estimate splits):
//     17 x 512 x 512         4.1 /  4.5 /  4.9 /  8.4        2048 x 2048 x 512    29 /  9.6 /  6.6 / 10.3
//     17 x 512 x 8192       14.9 /  7.9 / 11.1 / 67          2048 x 4096 x 1024   89 / 22   / 12.9 / 15.6
//     64 x 8192 x 8192      35.6 / 20   / 21.9 / 70          4096 x 2048 x 2048  150 / 35   / 21   / 25
//     128 x 1024 x 1024      4.5 /  5.5 /  7.6 / 13          16384 x 2048 x 512  213 / 59   / 27.4 / 23.6
//     256 x 4096 x 4096     36   / 11.1 / 19.6 / 38.6        4096^3              562 / 121  / 70.5 / 56.5
//     2048 x 512 x 512       8.8 /  4.7 /  5.8 /  9.6        8192^3                -        / 520  / 432
// With exact products tiles of 64, two of which a compute unit takes in the time of one, and 128; float32 results, 64 / 128:
//     1 x 8192 x 8192       22.8 / 25.4 (2 and 4 parts)      2048 x 4096 x 1024   27.8 / 26.8
//     17 x 512 x 8192        8.4 / 14.6 (16 and 8)           4096 x 2048 x 2048   46.9 / 43.3
//     256 x 4096 x 4096     21.7 / 26.9 (1 and 4)            16384 x 512 x 2048   46.5 / 41.0
//     1021 x 2000 x 1000    11.0 / 14.6                      4096^3              164   / 142
//     2048 x 2048 x 512     11.7 / 13.3                      8192^3                -   / 1020
MatmulPlan plan_matmul(const matmul8_t& p) {
    const int all = (int)ceil_div(p.dim, kBlock8);
    MatmulPlan best = {kMatmulRows, 16, 16, 1, all, 256};
    if (p.rows <= 16 && !p.exact) return best;
    double least = 1e300;
    auto consider = [&](int variant, int tile, double start, double stage, double ends, int most_splits, int round = kCus) {
        const int64_t tiles = ceil_div(p.rows, tile) * ceil_div(p.cols, tile);
        for (int splits = 1; splits <= most_splits; splits *= 2) {
            const int stages = splits == 1 ? all : (int)round_up(ceil_div(all, splits), 4);
            const int parts = (int)ceil_div(all, stages);
            if (splits > 1 && (parts < 2 || tiles * parts > kCus)) break;
            const double partial = (double)parts * p.rows * p.cols * 8;      // bytes, written and read
            const double us = start + ceil_div(tiles * parts, round) * (stages * stage + ends) + (parts > 1 ? 2.5 + parts * 0.06 + partial * 2e-7 : 0.0);
            if (us < least) {
                least = us;
                best = {variant, tile, tile, parts, stages, 256};
            }
        }
    };
    if (p.exact) {
        consider(kMatmulExactSmall, 64, 3.0, 0.55, 2.0, 64, 2 * kCus);
        consider(kMatmulExactMid, 128, 3.5, 1.08, 3.5, 8);
    } else {
        consider(kMatmulSplit, 32, 2.5, 0.20, 0.6, 1);
        consider(kMatmulSmall, 64, 2.6, 0.24, 0.9, 64);
        consider(kMatmulMid, 128, 3.5, 0.56, 0.75, 8);
        if (all >= kRingStages) consider(kMatmulTile, 256, 3.5, 1.55, 4.4, 1);      // of fewer, 128 is the estimate's choice anyway
    }
    if (best.splits > 1) best.bytes = round_up(4 * (int64_t)best.splits * p.rows * round_up(p.cols, 8), 256);
    return best;
}

int check_matmul_sizes(const matmul8_t* p) {
    if (!p) return fail(MUON_ERR_INVALID_ARG, "matmul8: problem is NULL");
    Checks c("matmul8");
    c.sizes(p->rows, p->cols, p->dim);
    c.one_of("exact", p->exact, 1);
    c.one_of("dtype", p->dtype, p->exact ? MUON_T_FP32 : MUON_T_FP16);
    if (!c.rc && ceil_div(p->rows, 128) * ceil_div(p->cols, 128) > (1 << 22))
        c.rc = fail(MUON_ERR_UNSUPPORTED, "matmul8: rows x cols beyond 2^36");
    return c.rc;
}

// ---------------------------------------------------------------- the weight's gradient
constexpr int kMinStages = 4;     // of a split
struct GradPlan {
    bool pack, deep;
    int edge, splits, stages;     // stages of a split
    int64_t cols8, dim8;
    int64_t grad, partial, bytes; // offsets, -1: not there
};
// As plan_matmul, for tiles of 128 and 256 and any of the splits below.  Fitted to (us; rows x cols x dim: tile / splits):
//     16384 x 2048 x 512    128/4 50, 128/8 54, 256/12 51        8192 x 8192 x 4096    128/1 574, 256/1 437
//     65536 x 128 x 128     128/32 28, 128/64 23                 16384 x 4096 x 1024   256/4 128
//     16384 x 512 x 512     128/12 21                            512 x 512 x 512       128/1 9.8 (256 rows 7.5: a split saves nothing)
// A part costs its sums' way through memory and 0.06 us of the join's latency.
GradPlan plan_grad(const act8_grad_weight_t& p) {
    GradPlan q;
    q.pack = p.cols % 8 || !whole_rows(p.grad, p.grad_stride, 2);
    q.cols8 = round_up(p.cols, 8);
    q.dim8 = round_up(p.dim, 8);
    const int64_t all = std::max<int64_t>(1, ceil_div(p.rows, kHeadK));
    static const int tried[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128};
    double least = 1e300;
    auto consider = [&](int edge, double stage, double ends) {
        const int64_t tiles = ceil_div(p.cols, edge) * ceil_div(p.dim, edge);
        for (int splits : tried) {
            if (splits > 1 && all / splits < kMinStages) break;
            const int64_t stages = ceil_div(all, splits), parts = ceil_div(all, stages);
            const double mb = (double)parts * p.cols * p.dim * 4e-6;         // a part's sums, written and read again
            const double us = 4.5 + ceil_div(tiles * parts, kCus) * (stages * stage + ends) + (parts > 1 ? 2.0 + parts * 0.06 + mb * 0.3 : 0.0);
            if (us >= least) continue;
            least = us;
            q.edge = edge;
            q.splits = (int)parts;
            q.stages = (int)stages;
        }
    };
    consider(128, 0.48, 2.5);
    consider(256, 1.5, 5.0);
    // Tiles of 128, one workgroup per compute unit and many stages: the deep form (16384 x 2048 x 512, 64 stages, the data past the
    // last cache / in it: 50.5 / 47.8 us against 59.4 / 46.9).  Few stages do not earn its longer start and code (22: 25.1
    // against 23.5; 1 to 8: 1 us more), and two workgroups hide each other's loads (512 of 32 stages: 60.6 against 54.0).
    q.deep = q.edge == 128 && ceil_div(p.cols, 128) * ceil_div(p.dim, 128) * q.splits <= kCus && q.stages >= 40;
    int64_t off = 0;
    auto take = [&](bool there, int64_t bytes) {
        const int64_t at = there ? off : -1;
        if (there) off = round_up(off + bytes, 256);
        return at;
    };
    q.grad = take(q.pack, 2 * p.rows * q.cols8);
    q.partial = take(q.splits > 1, 4 * (int64_t)q.splits * p.cols * q.dim8);
    q.bytes = std::max<int64_t>(off, 256);
    return q;
}

int check_grad_sizes(const act8_grad_weight_t* p) {
    if (!p) return fail(MUON_ERR_INVALID_ARG, "act8_grad_weight: problem is NULL");
    Checks c("act8_grad_weight");
    c.sizes(p->rows, p->cols, p->dim);
    if (!c.rc && ceil_div(p->cols, 128) * ceil_div(p->dim, 128) > (1 << 20))
        c.rc = fail(MUON_ERR_UNSUPPORTED, "act8_grad_weight: cols x dim beyond 2^34");
    return c.rc;
}

int check_workspace(const char* entry, const void* workspace, size_t given, int64_t needed) {
    if (!workspace || given < (size_t)needed)
        return fail(MUON_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %lld needed", entry, workspace ? given : (size_t)0,
                    (long long)needed);
    return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int act8_encode(const act8_encode_t* problem, void* stream) {
    if (!problem) return fail(MUON_ERR_INVALID_ARG, "act8_encode: problem is NULL");
    const act8_encode_t& p = *problem;
    Checks c("act8_encode");
    c.sizes(p.rows, 1, p.dim);
    c.one_of("dtype", p.dtype, MUON_T_FP32);
    c.one_of("activation", p.activation, MUON_ACT_GELU);
    if (!c.rc && (p.out.codes != nullptr) != (p.activation != MUON_ACT_NONE) && p.rows > 0)
        c.rc = fail(MUON_ERR_INVALID_ARG, "act8_encode: out is for act(x), and wanted with an activation function");
    if (!c.rc && !p.codes.codes && !p.out.codes && p.rows > 0)
        c.rc = fail(MUON_ERR_INVALID_ARG, "act8_encode: codes and out are both NULL");
    if (!c.rc) c.matrix("x", p.x, p.rows, p.dim, p.x_stride, size_of(p.dtype), false);
    if (p.codes.codes) c.coded("codes", p.codes, p.rows, p.dim, 1, true);
    if (p.out.codes) c.coded("out", p.out, p.rows, p.dim, 1, true);
    if (const int rc = c.done()) return rc;
    if (p.rows == 0) return MUON_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Encode8 a = {rows8(p.rows, p.dim), p.x, p.x_stride, blocks(p.codes), blocks(p.out)};
    LINEAR8_TRY("act8_encode", launch_encode8(a, p.dtype, p.activation, s));
    return MUON_OK;
}

int act8_decode(const blocks8_t* x, int32_t tall, int64_t rows, int64_t dim, void* out, int64_t out_stride, int32_t dtype,
                void* stream) {
    if (!x) return fail(MUON_ERR_INVALID_ARG, "act8_decode: x is NULL");
    Checks c("act8_decode");
    c.sizes(rows, 1, dim);
    c.one_of("dtype", dtype, MUON_T_FP32);
    c.one_of("tall", tall, 1);
    c.coded("x", *x, rows, dim, tall ? MUON_BLOCK8 : 1, false);
    if (!c.rc) c.matrix("out", out, rows, dim, out_stride, size_of(dtype), true);
    if (const int rc = c.done()) return rc;
    if (rows == 0) return MUON_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Decode8 a = {rows8(rows, dim), blocks(*x), tall ? kBlock8 : 1, out, out_stride,
                       through(out, rows, dim, out_stride, dtype)};
    LINEAR8_TRY("act8_decode", launch_decode8(a, dtype, s));
    return MUON_OK;
}

int act8_backward(const act8_backward_t* problem, void* stream) {
    if (!problem) return fail(MUON_ERR_INVALID_ARG, "act8_backward: problem is NULL");
    const act8_backward_t& p = *problem;
    const int64_t size = size_of(p.dtype);
    Checks c("act8_backward");
    c.sizes(p.rows, 1, p.dim);
    c.one_of("dtype", p.dtype, MUON_T_FP32);
    c.one_of("activation", p.activation, MUON_ACT_GELU);
    if (!c.rc && p.activation == MUON_ACT_NONE) c.rc = fail(MUON_ERR_INVALID_ARG, "act8_backward: activation is MUON_ACT_NONE");
    if (!c.rc && !p.out && !p.out8.codes && p.rows > 0)
        c.rc = fail(MUON_ERR_INVALID_ARG, "act8_backward: out and out8 are both NULL");
    c.coded("u", p.u, p.rows, p.dim, 1, false);
    // in place: a lane reads its values of grad before it writes them
    const bool in_place = p.out && p.out == p.grad && p.out_stride == p.grad_stride;
    if (!c.rc) c.matrix("grad", p.grad, p.rows, p.dim, p.grad_stride, size, in_place);
    if (!c.rc && p.out && !in_place) c.matrix("out", p.out, p.rows, p.dim, p.out_stride, size, true);
    if (p.out8.codes) c.coded("out8", p.out8, p.rows, p.dim, 1, true);
    if (const int rc = c.done()) return rc;
    if (p.rows == 0) return MUON_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Backward8 a = {rows8(p.rows, p.dim), blocks(p.u), blocks(p.out8), p.grad, p.out, p.grad_stride, p.out_stride,
                         through(p.out, p.rows, p.dim, p.out_stride, p.dtype)};
    LINEAR8_TRY("act8_backward", launch_backward8(a, p.dtype, p.activation, s));
    return MUON_OK;
}

int weight8_encode(const weight8_encode_t* problem, void* stream) {
    if (!problem) return fail(MUON_ERR_INVALID_ARG, "weight8_encode: problem is NULL");
    const weight8_encode_t& p = *problem;
    Checks c("weight8_encode");
    c.sizes(0, p.rows, p.dim);
    c.one_of("dtype", p.dtype, MUON_T_FP32);
    if (!c.rc && ceil_div(p.rows, kBlock8) * ceil_div(p.dim, kBlock8) > (1 << 22))
        c.rc = fail(MUON_ERR_UNSUPPORTED, "weight8_encode: rows x dim beyond 2^36");
    if (!c.rc) c.matrix("weight", p.weight, p.rows, p.dim, p.weight_stride, size_of(p.dtype), false);
    c.coded("codes", p.codes, p.rows, p.dim, MUON_BLOCK8, true);
    if (p.transposed.codes) c.coded("transposed", p.transposed, p.dim, p.rows, MUON_BLOCK8, true);
    if (const int rc = c.done()) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Weight8 a = {p.weight, p.weight_stride, (int)p.rows, (int)p.dim, blocks(p.codes), blocks(p.transposed)};
    LINEAR8_TRY("weight8_encode", launch_weight8(a, p.dtype, s));
    return MUON_OK;
}

size_t matmul8_workspace_size(const matmul8_t* problem) {
    if (check_matmul_sizes(problem)) return 0;
    return (size_t)plan_matmul(*problem).bytes;
}

int matmul8(const matmul8_t* problem, void* workspace, size_t workspace_bytes, void* stream) {
    if (const int rc = check_matmul_sizes(problem)) return rc;
    const matmul8_t& p = *problem;
    const MatmulPlan q = plan_matmul(p);
    if (const int rc = check_workspace("matmul8", workspace, workspace_bytes, q.bytes)) return rc;
    Checks c("matmul8");
    c.coded("a", p.a, p.rows, p.dim, 1, false);
    c.coded("b", p.b, p.cols, p.dim, MUON_BLOCK8, false);
    if (!c.rc) c.matrix("y", p.y, p.rows, p.cols, p.y_stride, size_of(p.dtype), true);
    c.buffer("workspace", workspace, q.bytes, 256, true);
    if (const int rc = c.done()) return rc;
    if (p.rows == 0) return MUON_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Matmul8 a = {blocks(p.a), blocks(p.b), p.y, p.y_stride, (int)p.rows, (int)p.cols, (int)p.dim,
                       whole_rows(p.y, p.y_stride, size_of(p.dtype)), (int)ceil_div(p.cols, q.tile_v), (int)ceil_div(p.rows, q.tile_t),
                       q.splits, q.stages, q.splits > 1 ? static_cast<float*>(workspace) : nullptr, round_up(p.cols, 8)};
    LINEAR8_TRY(kMatmulNames[q.variant], launch_matmul8(a, p.dtype, q.variant, s));
    if (q.splits > 1) LINEAR8_TRY("matmul8_join", launch_matmul8_join(a, p.dtype, s));
    return MUON_OK;
}

size_t act8_grad_weight_workspace_size(const act8_grad_weight_t* problem) {
    if (check_grad_sizes(problem)) return 0;
    return (size_t)plan_grad(*problem).bytes;
}

int act8_grad_weight(const act8_grad_weight_t* problem, void* workspace, size_t workspace_bytes, void* stream) {
    if (const int rc = check_grad_sizes(problem)) return rc;
    const act8_grad_weight_t& p = *problem;
    const GradPlan q = plan_grad(p);
    if (const int rc = check_workspace("act8_grad_weight", workspace, workspace_bytes, q.bytes)) return rc;
    Checks c("act8_grad_weight");
    c.coded("x", p.x, p.rows, p.dim, 1, false);
    if (!c.rc) c.matrix("grad", p.grad, p.rows, p.cols, p.grad_stride, 2, false);
    if (!c.rc) c.matrix("out", p.out, p.cols, p.dim, p.out_stride, 4, true);
    c.buffer("workspace", workspace, q.bytes, 256, true);
    if (const int rc = c.done()) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Join8 j = {nullptr, q.dim8, q.splits, (int)p.cols, (int)p.dim, p.out, p.out_stride, p.accumulate != 0};
    if (p.rows == 0) {
        j.splits = 0;
        if (!p.accumulate) LINEAR8_TRY("act8_grad_join", launch_join8(j, s));
        return MUON_OK;
    }
    const void* grad = p.grad;
    int64_t grad_stride = p.grad_stride;
    if (q.pack) {
        const HeadPack a = {p.grad, p.grad_stride, ws + q.grad, q.cols8, (int)p.rows, (int)p.rows, (int)p.cols, nullptr, 0};
        LINEAR8_TRY("act8_grad_pack", launch_head_pack(a, s));
        grad = ws + q.grad;
        grad_stride = q.cols8;
    }
    Grad8 a;
    memset(&a, 0, sizeof(a));
    a.x = blocks(p.x);
    a.grad = grad;
    a.grad_stride = grad_stride;
    a.rows = (int)p.rows;
    a.cols = (int)p.cols;
    a.dim = (int)p.dim;
    a.cols8 = (int)q.cols8;
    a.splits = q.splits;
    a.stages_per_split = q.stages;
    a.tiles_c = (int)ceil_div(p.cols, q.edge);
    a.tiles_d = (int)ceil_div(p.dim, q.edge);
    a.out = p.out;
    a.out_stride = p.out_stride;
    a.out_vec = whole_rows(p.out, p.out_stride, 4) && p.dim % 4 == 0;
    a.accumulate = p.accumulate != 0;
    a.partial = q.partial >= 0 ? reinterpret_cast<float*>(ws + q.partial) : nullptr;
    a.partial_pitch = q.dim8;
    LINEAR8_TRY(q.edge == 256 ? "act8_grad_256" : q.deep ? "act8_grad_128_deep" : "act8_grad_128", launch_grad8(a, q.edge, q.deep, s));
    if (a.partial) {
        j.partial = a.partial;
        LINEAR8_TRY("act8_grad_join", launch_join8(j, s));
    }
    return MUON_OK;
}

}  // extern "C"
