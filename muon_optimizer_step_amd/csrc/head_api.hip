// Host side of the language-model head's loss: argument checks, the layout of
// the workspace, the pieces of the tokens and the launch sequence behind
// head_loss in muonstep_train.h.
//
// One call enqueues, on the caller's stream:
//   head_pack   only for inputs that are not 16-byte aligned
//   for each piece of the tokens: head_logits (and the scale of the weights, one
//   workgroup); without gradients head_rows; with them head_prob (the same for
//   each token, a copy of hidden for the gradient of weight, and the
//   probabilities) and head_grads (and the loss, one workgroup), with head_join
//   where K was split or the pieces' sums had to be kept in fp32
//   head_loss   only where the loss is wanted without gradients
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <vector>

#include "../../include/muonstep_train.h"
#include "head.h"
#include "host.h"

namespace muon {
namespace {

constexpr int kCus = 256;                 // compute units of an MI355X
constexpr int kMinStagesPerSplit = 4;     // K stages a workgroup takes at least when K is split

// Piece of probabilities from which head_logits writes past the caches: 256 MB
// of last-level cache hold less of it than head_prob could use (16384 x 8192,
// 268 MB: head_logits 201 -> 187 us, head_prob 102 -> 100; 8192 x 131072, 2.1 GB:
// 3712 -> 3765, but head_prob, past them too, 949 -> 887; 1531 x 12345, 38 MB, the
// other way round: head_logits 57 -> 54, head_prob 20 -> 25).
constexpr int64_t kPastBytes = (int64_t)192 << 20;

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Offsets into the workspace (-1: not there) and sizes, from the problem alone.
struct HeadPlan {
    bool train, pack_h, pack_w, copy_h;
    int variant, tile_v, tile_t;  // of the logits
    int64_t dim8;                 // dim rounded up to whole chunks
    int64_t piece, pieces;        // tokens per piece
    int64_t rows, cols;           // padded size of a piece's probabilities
    int nsub, sub;
    int grad_edge, splits_h, splits_w, stages_h, stages_w;   // tiles and K splits of the two gradients
    bool partial_h, partial_w;
    int64_t scalars, row_weight, ref, sum, e, hidden, weight, part_h, part_w, bytes;
};

// Tile edge and splits of K for the two gradients (hidden: rows x dim, K the
// vocabulary; weight: vocab x dim, K the rows), those that take least by this
// estimate in stages of a 256 x 256 tile (1.6 us).  A tile costs a prologue and
// an epilogue (5 us, 3 stages); a split's partial sums are written and read
// again (13 us a tile with head_join's share).  One 256 x 256 tile or two 128 x
// 128 tiles run on a compute unit at a time; the latter take 0.62 of a stage
// each, both together.  Measured, gradients and join in us, 256 / 128 wide:
//   2048 x 4096 x 512  44 / 38     1531 x 12345 x 600  67 / 69
//   500 x 1000 x 256   25 / 18     8192 x 8192 x 512   133 / 145
//   1000 x 20000 x 200 46 / 39     300 x 50000 x 768   86 / 81
//   16384 x 8192 x 512 244 / 344   8192 x 131072 x 2048  6780 / 9520
struct GradSplit {
    int edge = kHeadTile, splits_h = 1, splits_w = 1;
};
GradSplit split_k(int64_t rows, int64_t vocab, int64_t dim, bool grad_hidden, bool grad_weight) {
    static const int tried[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32};
    auto ceil_div = [](int64_t x, int64_t m) { return (x + m - 1) / m; };
    const int a = (int)ceil_div(vocab, kHeadK), b = (int)ceil_div(rows, kHeadK);
    double best = 1e300;
    GradSplit r;
    for (int edge : {256, 128}) {
        const int64_t tiles_d = ceil_div(dim, edge);
        const int64_t n = grad_hidden ? ceil_div(rows, edge) * tiles_d : 0, m = grad_weight ? ceil_div(vocab, edge) * tiles_d : 0;
        const double stage = edge == 256 ? 1.0 : 0.62, part = edge == 256 ? 8.0 : 3.0, ends = edge == 256 ? 3.0 : 2.0;
        const int slots = edge == 256 ? kCus : 2 * kCus;
        for (int i : tried) {
            if (i > 1 && (n == 0 || a / i < kMinStagesPerSplit)) break;
            for (int j : tried) {
                if (j > 1 && (m == 0 || b / j < kMinStagesPerSplit)) break;
                const double la = n ? ceil_div(a, i) * stage + ends + (i > 1 ? part : 0.0) : 0.0;
                const double lb = m ? ceil_div(b, j) * stage + ends + (j > 1 ? part : 0.0) : 0.0;
                const int64_t items = n * i + m * j;
                const double longest = std::max(la, lb), even = (n * i * la + m * j * lb) / slots;
                // the last items to start are gradient tiles of weight; their round is on average half full
                const double cost = items <= slots ? longest : std::max(longest, even + 0.5 * (m ? lb : la));
                if (cost < best) {
                    best = cost;
                    r.edge = edge;
                    r.splits_h = i;
                    r.splits_w = j;
                }
            }
        }
    }
    return r;
}

// Kernel for the logits of a piece.  Measured (us, bf16, no gradients):
//   tokens x vocab x dim      stream  128 x 32  128 x 64  128 x 128  256 x 256
//   1 x 8192 x 512               7.8       9.2       9.4       10.6       18.4
//   1 x 32768 x 1024            17.0      14.1      15.3       18.1       28.0
//   64 x 131072 x 2048             -       123       111        129        140
//   256 x 32768 x 1024             -         -      29.2       22.8       28.4
//   1531 x 12345 x 600             -         -         -       40.7       42.9
//   2048 x 8192 x 512              -         -         -       25.0       21.9
//   1024 x 50000 x 1024            -         -         -        119        114
//   4096 x 8192 x 512              -         -         -       44.2       39.2
// The last two differ in their rate (a 256 x 256 tile moves half the operand
// bytes per product) and in the waste of their last round, counted here in
// rounds of 256 tiles; two 128 x 128 tiles per compute unit overlap, less so
// where a cap makes the vector work of the tile's end longer (1021 x 50021 x
// 1000 capped: 161 against 143).
int logits_variant(int64_t tokens, int64_t vocab, bool cap) {
    if (tokens <= kHeadStream) return vocab < 16384 ? kLogitsStream : kLogitsMid32;
    if (tokens <= 64) return kLogitsMid64;
    auto tiles = [&](int64_t edge) { return ((tokens + edge - 1) / edge) * ((vocab + edge - 1) / edge); };
    const double big = (double)((tiles(256) + kCus - 1) / kCus);
    const double mid = (cap ? 0.70 : 0.64) * std::max(1.0, (double)tiles(128) / (2 * kCus) + 0.3);
    return mid < big ? kLogitsMid128 : kLogitsTile;
}

HeadPlan make_head_plan(const head_loss_t& p) {
    HeadPlan q;
    q.train = p.loss || p.grad_hidden || p.grad_weight;
    q.dim8 = round_up(p.dim, 8);
    auto odd = [&](const void* ptr, int64_t stride) {
        return p.dim % 8 || stride % 8 || reinterpret_cast<uintptr_t>(ptr) % 16;
    };
    q.pack_h = odd(p.hidden, p.hidden_stride);
    q.copy_h = !q.pack_h && p.grad_weight;
    q.pack_w = odd(p.weight, p.weight_stride);
    const bool grads = p.grad_hidden || p.grad_weight;
    q.cols = round_up(p.vocab, kHeadPad);
    auto piece = [&](int64_t most) {
        const int64_t all = std::max<int64_t>(p.tokens, 1);
        return all * q.cols > most ? std::min(all, std::max<int64_t>(kHeadTile, most / q.cols / kHeadTile * kHeadTile)) : all;
    };
    // gradients: what the workspace holds of the probabilities; scoring: 2^32
    // logits a launch, whose partial sums take 256 MB
    const int64_t grads_piece = piece(MUON_HEAD_PIECE_BYTES / 2);
    q.piece = grads ? grads_piece : piece((int64_t)1 << 32);
    q.pieces = (p.tokens + q.piece - 1) / q.piece;
    q.rows = round_up(q.piece, kHeadPad);
    // the kernel for the pieces of a call with gradients, whatever is asked for: a
    // token's sums are then grouped alike, and its loss has the same bits
    q.variant = logits_variant(grads_piece, p.vocab, p.softcap > 0.f);
    q.tile_v = q.variant == kLogitsTile ? kHeadTile : q.variant == kLogitsStream ? kHeadStreamSub : kHeadMidVocab;
    q.tile_t = q.variant == kLogitsTile ? kHeadTile : q.variant == kLogitsMid128 ? 128 : q.variant == kLogitsMid32 ? 32 : 64;
    q.sub = logits_sub(q.variant);
    q.nsub = (int)(q.variant == kLogitsStream ? q.cols / q.sub : round_up(p.vocab, q.tile_v) / q.sub);
    const int all_h = (int)(q.cols / kHeadK), all_w = (int)(q.rows / kHeadK);
    const GradSplit g = split_k(q.piece, p.vocab, p.dim, p.grad_hidden, p.grad_weight);
    q.grad_edge = g.edge;
    q.splits_h = g.splits_h;
    q.splits_w = g.splits_w;
    q.stages_h = (all_h + q.splits_h - 1) / q.splits_h;
    q.stages_w = (all_w + q.splits_w - 1) / q.splits_w;
    q.partial_h = p.grad_hidden && q.splits_h > 1;
    q.partial_w = p.grad_weight && (q.splits_w > 1 || q.pieces > 1);
    int64_t off = 0;
    auto take = [&](bool there, int64_t bytes) {
        const int64_t at = there ? off : -1;
        if (there) off = round_up(off + bytes, 256);
        return at;
    };
    q.scalars = take(true, 16);
    q.row_weight = take(q.train, 4 * (p.tokens + kHeadPad));
    q.ref = take(true, 4 * (int64_t)q.nsub * q.rows);
    q.sum = take(true, 4 * (int64_t)q.nsub * q.rows);
    q.e = take(grads, 2 * q.rows * q.cols);
    q.hidden = take(q.pack_h || q.copy_h, 2 * (q.pack_h ? round_up(p.tokens, kHeadPad) : q.rows) * q.dim8);
    q.weight = take(q.pack_w, 2 * p.vocab * q.dim8);
    q.part_h = take(q.partial_h, 4 * (int64_t)q.splits_h * q.piece * q.dim8);
    q.part_w = take(q.partial_w, 4 * (int64_t)q.splits_w * p.vocab * q.dim8);
    q.bytes = std::max<int64_t>(off, 256);
    return q;
}

int validate_sizes(const head_loss_t* p) {
    if (!p) return fail(MUON_ERR_INVALID_ARG, "problem is NULL");
    if (p->tokens < 0 || p->vocab < 1 || p->dim < 1)
        return fail(MUON_ERR_INVALID_ARG, "tokens = %lld, vocab = %lld, dim = %lld: tokens >= 0, vocab and dim >= 1",
                    (long long)p->tokens, (long long)p->vocab, (long long)p->dim);
    if (p->tokens > MUON_HEAD_MAX_TOKENS || p->vocab > MUON_HEAD_MAX_VOCAB || p->dim > MUON_HEAD_MAX_DIM)
        return fail(MUON_ERR_UNSUPPORTED, "tokens = %lld, vocab = %lld, dim = %lld beyond the limits", (long long)p->tokens,
                    (long long)p->vocab, (long long)p->dim);
    if (p->dtype != MUON_HEAD_BF16 && p->dtype != MUON_HEAD_FP16)
        return fail(MUON_ERR_INVALID_ARG, "dtype = %d is not MUON_HEAD_BF16 or MUON_HEAD_FP16", p->dtype);
    if (!std::isfinite(p->softcap) || p->softcap < 0.f) return fail(MUON_ERR_INVALID_ARG, "softcap must be finite and >= 0");
    if (p->hidden_stride < p->dim || p->weight_stride < p->dim || (p->grad_hidden && p->grad_hidden_stride < p->dim) ||
        (p->grad_weight && p->grad_weight_stride < p->dim))
        return fail(MUON_ERR_INVALID_ARG, "a row stride is smaller than dim = %lld", (long long)p->dim);
    const int64_t far = (int64_t)1 << 22;   // 256 rows apart fits 32 bits of bytes
    if (p->hidden_stride > far || p->weight_stride > far || (p->grad_hidden && p->grad_hidden_stride > far) ||
        (p->grad_weight && p->grad_weight_stride > far))
        return fail(MUON_ERR_UNSUPPORTED, "a row stride is beyond 2^22");
    return MUON_OK;
}

int validate_buffers(const head_loss_t& p, const void* workspace, size_t bytes) {
    const int64_t n = p.tokens;
    if (!p.weight || (n > 0 && (!p.hidden || !p.targets || !p.nll)))
        return fail(MUON_ERR_INVALID_ARG, "hidden, weight, targets and nll must be non-NULL");
    auto rows = [](int64_t r, int64_t stride, int64_t dim) { return r > 0 ? 2 * ((r - 1) * stride + dim) : 0; };
    // inputs may share memory with each other; what is written may not
    const struct { const void* p; int64_t bytes; int align; bool written; } buf[10] = {
        {p.hidden, rows(n, p.hidden_stride, p.dim), 2, false},
        {p.weight, rows(p.vocab, p.weight_stride, p.dim), 2, false},
        {p.targets, 8 * n, 8, false},
        {p.token_weights, 4 * n, 4, false},
        {p.loss, 4, 4, true},
        {p.nll, 4 * n, 4, true},
        {p.lse, 4 * n, 4, true},
        {p.grad_hidden, rows(n, p.grad_hidden_stride, p.dim), 2, true},
        {p.grad_weight, rows(p.vocab, p.grad_weight_stride, p.dim), 2, true},
        {workspace, (int64_t)bytes, 256, true}};
    for (int i = 0; i < 10; ++i) {
        if (!buf[i].p || buf[i].bytes == 0) continue;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(buf[i].p);
        if (lo % buf[i].align) return fail(MUON_ERR_INVALID_ARG, "buffer %d is not %d-byte aligned", i, buf[i].align);
        for (int j = 0; j < i; ++j) {
            if (!buf[j].p || buf[j].bytes == 0 || !(buf[i].written || buf[j].written)) continue;
            const uintptr_t lj = reinterpret_cast<uintptr_t>(buf[j].p);
            if (lo < lj + buf[j].bytes && lj < lo + buf[i].bytes)
                return fail(MUON_ERR_UNSUPPORTED, "head_loss: buffers %d and %d overlap", j, i);
        }
    }
    return MUON_OK;
}

#define HEAD_TRY(name, call)                                                                                    \
    do {                                                                                                        \
        const hipError_t err_ = timed_launch(name, s, [&] { return call; });                                    \
        if (err_ != hipSuccess) return fail(MUON_ERR_HIP, "%s launch failed: %s", name, hipGetErrorString(err_)); \
    } while (0)

int enqueue_head(const head_loss_t& p, const HeadPlan& q, uint8_t* ws, hipStream_t s) {
    float* scalars = reinterpret_cast<float*>(ws + q.scalars);
    float* row_weight = q.train ? reinterpret_cast<float*>(ws + q.row_weight) : nullptr;
    const int dim = (int)p.dim, vocab = (int)p.vocab;
    const uint8_t* h = static_cast<const uint8_t*>(p.hidden);
    const void* w = p.weight;
    int64_t h_pitch = p.hidden_stride, w_pitch = p.weight_stride;
    if (q.pack_h && p.tokens) {
        const HeadPack a = {p.hidden, p.hidden_stride, ws + q.hidden, q.dim8, (int)round_up(p.tokens, kHeadPad), (int)p.tokens,
                            dim, p.targets, p.ignore_index};
        HEAD_TRY("head_pack", launch_head_pack(a, s));
        h = ws + q.hidden;
        h_pitch = q.dim8;
    }
    if (q.pack_w) {
        const HeadPack a = {p.weight, p.weight_stride, ws + q.weight, q.dim8, vocab, vocab, dim, nullptr, 0};
        HEAD_TRY("head_pack", launch_head_pack(a, s));
        w = ws + q.weight;
        w_pitch = q.dim8;
    }
    float* ref = reinterpret_cast<float*>(ws + q.ref);
    float* sum = reinterpret_cast<float*>(ws + q.sum);
    // finite: zero times it has to stay zero
    const float inv_cap = p.softcap > 0.f ? std::min(1.0f / p.softcap, FLT_MAX) : 0.f;
    auto vec = [&](const void* ptr, int64_t stride) {
        return dim % 8 == 0 && stride % 8 == 0 && reinterpret_cast<uintptr_t>(ptr) % 16 == 0;
    };
    const int tiles_d = (dim + q.grad_edge - 1) / q.grad_edge;
    for (int64_t at = 0; at < p.tokens; at += q.piece) {
        const int tokens = (int)std::min(q.piece, p.tokens - at), rows = (int)round_up(tokens, kHeadPad);
        const uint8_t* hp = h + at * h_pitch * 2;
        HeadLogits a;
        memset(&a, 0, sizeof(a));
        a.h = hp;
        a.w = w;
        a.targets = p.targets + at;
        a.h_pitch = h_pitch;
        a.w_pitch = w_pitch;
        a.e = q.e >= 0 ? ws + q.e : nullptr;
        a.e_pitch = q.cols;
        a.e_rows = rows;
        a.e_past = 2 * (int64_t)rows * q.cols > kPastBytes;
        // a token's partials side by side where head_rows has a workgroup for each token, a partial's tokens otherwise
        const bool by_token = q.e < 0 && rows <= kHeadRowGroups;
        a.stats = {ref, sum, rows, by_token ? 1 : rows, by_token ? q.nsub : 1};
        a.tokens = tokens;
        a.vocab = vocab;
        a.dim = (int)(q.pack_h && q.pack_w ? q.dim8 : p.dim);
        a.cap = p.softcap;
        a.inv_cap = inv_cap;
        a.tiles_v = (vocab + q.tile_v - 1) / q.tile_v;
        a.tiles_t = (tokens + q.tile_t - 1) / q.tile_t;
        if (q.train && at == 0) a.scalars = {p.targets, p.token_weights, scalars, p.ignore_index, (int)p.tokens, p.dtype};
        HEAD_TRY("head_logits", launch_head_logits(a, p.dtype, q.variant, s));
        HeadRows r;
        memset(&r, 0, sizeof(r));
        r.stats = a.stats;
        r.nsub = q.nsub;
        r.h = hp;
        r.w = w;
        r.h_pitch = h_pitch;
        r.w_pitch = w_pitch;
        r.targets = p.targets + at;
        r.weights = p.token_weights ? p.token_weights + at : nullptr;
        r.scalars = scalars;
        r.nll = p.nll + at;
        r.lse = p.lse ? p.lse + at : nullptr;
        r.row_weight = q.train ? row_weight + at : nullptr;
        r.copy = q.copy_h ? ws + q.hidden : nullptr;
        r.copy_pitch = q.dim8;
        r.ignore_index = p.ignore_index;
        r.tokens = tokens;
        r.rows = q.train ? rows : tokens;
        r.vocab = vocab;
        r.dim = a.dim;
        r.cap = p.softcap;
        r.inv_cap = inv_cap;
        r.train = q.train;
        r.e = q.e >= 0 ? ws + q.e : nullptr;
        r.e_pitch = q.cols;
        r.sub = q.sub;
        if (q.e < 0) {
            HEAD_TRY("head_rows", launch_head_rows(r, p.dtype, s));
            continue;
        }
        HEAD_TRY("head_prob", launch_head_prob(r, p.dtype, s));
        const bool last = at + q.piece >= p.tokens;
        HeadGrads g;
        memset(&g, 0, sizeof(g));
        if (last && p.loss) g.loss = {p.nll, row_weight, scalars, p.loss, (int)p.tokens};
        auto common = [&](HeadGrad& x, int64_t cols) {
            x.p = ws + q.e;
            x.p_pitch = q.cols;
            x.p_rows = rows;
            x.p_cols = (int)q.cols;
            x.dim = dim;
            x.cols = (int)cols;
            x.tiles_c = (int)((cols + q.grad_edge - 1) / q.grad_edge);
            x.tiles_d = tiles_d;
            x.partial_pitch = q.dim8;
            x.scalars = scalars;
        };
        HeadJoin j;
        memset(&j, 0, sizeof(j));
        j.dim = dim;
        j.scalars = scalars;
        if (p.grad_hidden) {
            HeadGrad& x = g.hidden;
            common(x, tokens);
            x.a = w;
            x.a_pitch = w_pitch;
            x.a_rows = vocab;
            x.k = (int)q.cols;
            x.splits = q.splits_h;
            x.stages_per_split = q.stages_h;
            x.out = static_cast<uint8_t*>(p.grad_hidden) + at * p.grad_hidden_stride * 2;
            x.out_pitch = p.grad_hidden_stride;
            x.out_vec = vec(x.out, x.out_pitch);
            x.partial = q.partial_h ? reinterpret_cast<float*>(ws + q.part_h) : nullptr;
            if (q.partial_h) j.part[0] = {x.partial, q.dim8, q.splits_h, tokens, x.out, x.out_pitch, x.out_vec};
        }
        if (p.grad_weight) {
            HeadGrad& x = g.weight;
            common(x, vocab);
            x.a = q.copy_h ? ws + q.hidden : hp;     // ignored rows are zero in either
            x.a_pitch = q.dim8;
            x.a_rows = rows;
            x.k = rows;
            x.splits = q.splits_w;
            x.stages_per_split = q.stages_w;
            x.out = p.grad_weight;
            x.out_pitch = p.grad_weight_stride;
            x.out_vec = vec(x.out, x.out_pitch);
            x.partial = q.partial_w ? reinterpret_cast<float*>(ws + q.part_w) : nullptr;
            x.accumulate = at > 0;
            if (q.partial_w && last) j.part[1] = {x.partial, q.dim8, q.splits_w, vocab, x.out, x.out_pitch, x.out_vec};
        }
        HEAD_TRY("head_grads", launch_head_grads(g, p.dtype, q.grad_edge != kHeadTile, s));
        if (j.part[0].cols || j.part[1].cols) HEAD_TRY("head_join", launch_head_join(j, p.dtype, s));
    }
    if (p.tokens == 0 && (p.grad_weight || p.loss)) {
        // no tokens: the sums are empty
        HeadJoin j;
        memset(&j, 0, sizeof(j));
        j.dim = dim;
        j.scalars = scalars;
        const HeadPack a = {nullptr, 0, scalars, 8, 1, 0, 8, nullptr, 0};
        HEAD_TRY("head_pack", launch_head_pack(a, s));
        if (p.grad_weight) {
            j.part[1] = {nullptr, q.dim8, 0, vocab, p.grad_weight, p.grad_weight_stride, vec(p.grad_weight, p.grad_weight_stride)};
            HEAD_TRY("head_join", launch_head_join(j, p.dtype, s));
        }
    }
    if (p.loss && (q.e < 0 || p.tokens == 0)) {
        const HeadLoss a = {p.nll, row_weight, scalars, p.loss, (int)p.tokens};
        HEAD_TRY("head_loss", launch_head_loss(a, s));
    }
    return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t head_loss_workspace_size(const head_loss_t* problem) {
    if (validate_sizes(problem) != MUON_OK) return 0;
    return (size_t)make_head_plan(*problem).bytes;
}

int head_loss(const head_loss_t* problem, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = validate_sizes(problem);
    if (rc) return rc;
    const head_loss_t& p = *problem;
    const HeadPlan q = make_head_plan(p);
    if (!workspace || workspace_bytes < (size_t)q.bytes)
        return fail(MUON_ERR_WORKSPACE, "workspace of %zu bytes given, %lld needed", workspace ? workspace_bytes : (size_t)0,
                    (long long)q.bytes);
    if ((rc = validate_buffers(p, workspace, (size_t)q.bytes))) return rc;
    return enqueue_head(p, q, static_cast<uint8_t*>(workspace), static_cast<hipStream_t>(stream));
}

}  // extern "C"
