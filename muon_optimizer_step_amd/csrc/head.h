// Kernel arguments and launchers of the language-model head's loss (head.hip);
// the host side is head_api.hip.
#pragma once

#include "common.h"

namespace muon {

enum HeadType { kHeadBf16 = 0, kHeadFp16 = 1 };

constexpr int kHeadK = 64;         // K elements per LDS stage: 128 bytes of a row
constexpr int kHeadPad = 64;       // rows and columns of the probability piece are padded to it
constexpr int kHeadTile = 256;     // output tile edge of the products
constexpr int kHeadSmall = 64;     // tokens up to which the vocabulary is streamed past all of them at once
constexpr int kHeadSub = 128;      // vocabulary entries per partial maximum and sum, tiled kernel
constexpr int kHeadSmallSub = 32;  // the same, streaming kernel

// Logits of a piece of the tokens against the whole vocabulary, reduced to a
// reference exponent and a sum per token and `sub` vocabulary entries, and (e
// set) kept as fp16 exp2(logit - reference).
struct HeadLogits {
    const void* h;           // tokens x dim
    const void* w;           // vocab x dim
    int64_t h_pitch, w_pitch;   // elements
    void* e;                 // nullable; e_rows x e_pitch
    int64_t e_pitch;
    int e_rows;              // rows that exist in e
    float* ref;              // [sub][stat_pitch]
    float* sum;
    int stat_pitch;
    int tokens, vocab, dim;
    float cap, inv_cap;      // 0: no cap
    int tiles_v, tiles_t;
};

// Per token: log-sum-exp, loss, and the factors of the gradient.
struct HeadRows {
    const float* ref;
    float* sum;              // in: partial sums; out (train): factor from e to probability x weight
    int stat_pitch, nsub;
    const void* h;
    const void* w;
    int64_t h_pitch, w_pitch;
    const int64_t* targets;
    const float* weights;    // nullable
    const float* scalars;    // [0] mean weight, [1] probability scale, [2] its inverse
    float* nll;
    float* lse;              // nullable
    float* row_weight;       // train: weight of the token (times the probability scale)
    int* row_target;         // train: its target, -1 for none
    int64_t ignore_index;
    int tokens, rows, vocab, dim;   // rows: tokens padded
    float cap, inv_cap;
    int train;
};

struct HeadProb {
    void* e;                 // in: fp16 exp2 values; out: probability gradient, input type
    int64_t e_pitch;
    int rows, cols;          // padded
    const float* ref;
    const float* factor;     // [sub][stat_pitch]
    int stat_pitch, sub;
    const float* row_weight;
    const int* row_target;
    float inv_cap;           // 0: no cap
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

struct HeadJoin {
    const float* partial;
    int64_t partial_pitch;
    int splits, cols, dim;
    void* out;
    int64_t out_pitch;
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

struct HeadScalars {
    const int64_t* targets;
    const float* weights;
    float* scalars;
    int64_t ignore_index;
    int64_t tokens;
    int type;
};

struct HeadLoss {
    const float* nll;
    const float* row_weight;
    const float* scalars;
    float* loss;
    int64_t tokens;
};

hipError_t launch_head_logits(const HeadLogits& a, int type, bool small, hipStream_t s);
hipError_t launch_head_rows(const HeadRows& a, int type, hipStream_t s);
hipError_t launch_head_prob(const HeadProb& a, int type, hipStream_t s);
hipError_t launch_head_grad(const HeadGrad& a, int type, bool k_is_token, hipStream_t s);
hipError_t launch_head_join(const HeadJoin& a, int type, hipStream_t s);
hipError_t launch_head_pack(const HeadPack& a, hipStream_t s);
hipError_t launch_head_scalars(const HeadScalars& a, hipStream_t s);
hipError_t launch_head_loss(const HeadLoss& a, hipStream_t s);

}  // namespace muon
