// Kernel arguments and launchers of the language-model head's loss (head.hip);
// the host side is head_api.hip.
#pragma once

#include "common.h"
#include "tiles.h"

namespace muon {

enum HeadType { kHeadBf16 = 0, kHeadFp16 = 1 };

constexpr int kHeadPad = 64;       // rows and columns of the probability piece are padded to it
constexpr int kHeadMidVocab = 128; // vocabulary entries of a tile of the kernels for few tokens or small problems
constexpr int kHeadStream = 32;    // tokens that the streaming kernel and the narrowest tile take at most
constexpr int kHeadStreamSub = 32; // vocabulary entries of its workgroups
constexpr int kHeadRowGroups = 256; // tokens up to which head_rows takes a workgroup for each

// Kernels for the logits, and the vocabulary entries of their partial maxima
// and sums (what one wave holds).
enum LogitsVariant { kLogitsStream = 0, kLogitsMid32, kLogitsMid64, kLogitsMid128, kLogitsTile };
constexpr int logits_sub(int variant) { return variant == kLogitsTile ? 128 : variant == kLogitsMid128 ? 64 : 32; }

// What the weights in P and the sums over P are scaled by, over all tokens of
// the call; computed by one more workgroup of the first head_logits launch.
struct HeadScalars {
    const int64_t* targets;
    const float* weights;    // nullable
    float* scalars;          // NULL: nothing to do in this launch
    int64_t ignore_index;
    int tokens;
    int type;
};

// The partials of a piece: a reference and a sum for each sub-tile and token.
struct HeadStats {
    float* ref;
    float* sum;
    int rows;                // tokens that there is room for
    int per_sub, per_token;  // elements from one to the next
    __host__ __device__ int64_t at(int sub, int token) const { return (int64_t)sub * per_sub + (int64_t)token * per_token; }
};

// Logits of a piece of the tokens against the whole vocabulary, reduced to a
// reference exponent and a sum per token and `sub` vocabulary entries, and (e
// set) kept as fp16 exp2(logit - reference), times the cap's
// derivative but at the target.
struct HeadLogits {
    const void* h;           // tokens x dim
    const void* w;           // vocab x dim
    const int64_t* targets;  // per token
    int64_t h_pitch, w_pitch;   // elements
    void* e;                 // nullable; e_rows x e_pitch
    int64_t e_pitch;
    int e_rows;              // rows that exist in e
    int e_past;            // e is larger than the last cache: written past the caches
    HeadStats stats;
    int tokens, vocab, dim;
    float cap, inv_cap;      // 0: no cap
    int tiles_v, tiles_t;
    HeadScalars scalars;
};

// Per token: log-sum-exp and loss; with e also the probabilities' gradient in
// its place.
struct HeadRows {
    HeadStats stats;
    int nsub;
    void* e;                 // in: fp16 values of head_logits; out: probability gradient, input type
    int64_t e_pitch;
    int sub;                 // vocabulary entries per partial
    const void* h;
    const void* w;
    int64_t h_pitch, w_pitch;
    const int64_t* targets;
    const float* weights;    // nullable
    const float* scalars;    // [0] what weights are multiplied by in P, [1] what sums over P are multiplied by
    float* nll;
    float* lse;              // nullable
    float* row_weight;       // train: weight of the token in P
    void* copy;              // nullable: rows x copy_pitch, hidden with zeros for tokens that do not count
    int64_t copy_pitch;
    int64_t ignore_index;
    int tokens, rows, vocab, dim;   // rows: tokens padded
    float cap, inv_cap;
    int train;
};

// sum of weight x nll over all tokens of the call; by one more workgroup of the
// last head_grads launch, or on its own.
struct HeadLoss {
    const float* nll;
    const float* row_weight;
    const float* scalars;
    float* loss;             // NULL: nothing to do in this launch
    int tokens;
};

// out[col][d] = sum over k of P(k, col) A[k][d].
struct HeadGrad {
    const void* a;           // k x d
    int64_t a_pitch;
    int a_rows;              // rows of A that exist
    const void* p;
    int64_t p_pitch;
    int p_rows, p_cols;      // the piece's padded size
    int cols, dim, k;        // k: a multiple of kHeadK
    int splits, stages_per_split;
    int tiles_c, tiles_d;
    void* out;               // cols x dim in the input type, where splits == 1 and !partial
    int64_t out_pitch;
    int out_vec;             // rows of out 16-byte aligned
    float* partial;          // nullable: [split][cols][partial_pitch]
    int64_t partial_pitch;
    int accumulate;          // add to what partial holds
    const float* scalars;
};
// Both gradients of a piece; one without an output has tiles_c == 0.
struct HeadGrads {
    HeadGrad hidden, weight;
    HeadLoss loss;
};

// out[col][d] = sum over the splits' partials, for up to two gradients.
struct HeadJoin {
    struct Part {
        const float* partial;
        int64_t partial_pitch;
        int splits, cols;    // cols == 0: nothing to do
        void* out;
        int64_t out_pitch;
        int out_vec;
    } part[2];
    int dim;
    const float* scalars;
};

struct HeadPack {
    const void* src;
    int64_t src_pitch;
    void* dst;
    int64_t dst_pitch;
    int rows, src_rows, dim; // rows beyond src_rows and ignored ones become zero
    const int64_t* targets;  // nullable
    int64_t ignore_index;
};

hipError_t launch_head_logits(const HeadLogits& a, int type, int variant, hipStream_t s);
hipError_t launch_head_rows(const HeadRows& a, int type, hipStream_t s);
hipError_t launch_head_prob(const HeadRows& a, int type, hipStream_t s);
hipError_t launch_head_grads(const HeadGrads& a, int type, bool mid, hipStream_t s);
hipError_t launch_head_join(const HeadJoin& a, int type, hipStream_t s);
hipError_t launch_head_pack(const HeadPack& a, hipStream_t s);
hipError_t launch_head_loss(const HeadLoss& a, hipStream_t s);

}  // namespace muon
