// Kernel arguments and launchers of the linear layers in 8 bits (blocks8.hip,
// matmul8.hip, grad8.hip); the host side is linear8_api.hip.
#pragma once

#include "common.h"

namespace muon {

enum Linear8Type { kTypeBf16 = 0, kTypeFp16, kTypeFp32 };
enum Linear8Act { kActNone = 0, kActRelu2, kActSilu, kActGelu };

constexpr int kBlock8 = 128;      // values of a row that share a scale
constexpr int kScale8Low = 10;    // the smallest scale's byte

// Part of a result from `base` (the same for the whole wave) on, written with the device's scope: through the XCD's
// L2.  What a kernel leaves there is written back when it ends, and the next one waits for that.  Meant for whole
// 128-byte lines: 16 lanes of 8 codes, 32 of 4, 8 of 16 bytes.  Rows that begin or end inside a line break two of them,
// which is no loss in codes and little in y and the weight's gradient.  Through the L2 / by ordinary stores, us, in a
// graph, three sets of inputs in turn; in brackets with a reader behind it:
//     y 2048 x 2048 x 512      6.2 / 6.9  (11.0 / 11.6)      codes of 16384 x 4096    32.0 / 35.0 (59.9 / 62.6)
//     y 16384 x 2048 x 512    26.3 / 28.4 (42 / 46 to 49)    codes of 65536 x 200      9.7 / 10.6 (22.5 / 23.6)
//     y 16384 x 1000 x 512    15.0 / 15.4 (28.2 / 26.6)      gradient 1000 x 4000 x 2004   25.7 / 25.7 (40 / 37)
// Offsets in bytes, below 2^31.
struct Through {
    static constexpr int kDevice = 16;      // the instruction's sc1
    __amdgpu_buffer_rsrc_t out;
    __device__ inline explicit Through(void* base) : out(__builtin_amdgcn_make_buffer_rsrc(base, 0, 0x7fffffff, 0x00027000)) {}
    __device__ inline void store(int offset, const u32x4& w) const { __builtin_amdgcn_raw_buffer_store_b128(w, out, offset, 0, kDevice); }
    __device__ inline void store(int offset, const u32x2& w) const { __builtin_amdgcn_raw_buffer_store_b64(w, out, offset, 0, kDevice); }
    __device__ inline void store(int offset, uint32_t w) const { __builtin_amdgcn_raw_buffer_store_b32(w, out, offset, 0, kDevice); }
};

// 16 and 8 bytes at any multiple of 2: the same instructions as at their own alignment.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef floatx4 floatx4_any __attribute__((aligned(4)));

// Between a wave's writes to LDS and what its other lanes read of them, and before it writes there again: LDS keeps a
// wave's order, and this keeps the compiler from taking some lanes past the others.
__device__ inline void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A matrix in 8 bits: codes and scales, strides in bytes.
struct Blocks8 {
    uint8_t* codes;
    uint8_t* scale;
    int64_t stride, scale_stride;
};

// Which rows and blocks of a row-wise pass a workgroup takes: 2^unit_log units of 16
// lanes side by side on a row, 16 >> unit_log rows of them at a time.
struct Rows8 {
    int64_t rows;
    int dim, dim16;          // dim rounded up to 16
    int unit_log, col_groups, row_groups;      // at most 2^30 of both together
};

struct Encode8 {
    Rows8 r;
    const void* x;
    int64_t x_stride;        // elements
    Blocks8 codes, out;      // codes NULL: not wanted
};
struct Backward8 {
    Rows8 r;
    Blocks8 u, out8;
    const void* grad;
    void* out;
    int64_t grad_stride, out_stride;
    int out_through;         // 16-bit results pass the L2
};
struct Decode8 {
    Rows8 r;
    Blocks8 x;
    int tall;                // rows of a block: 1 or kBlock8
    void* out;
    int64_t out_stride;
    int out_through;         // as above
};
struct Weight8 {
    const void* w;
    int64_t w_stride;
    int rows, dim;
    Blocks8 codes, transposed;
};

hipError_t launch_encode8(const Encode8& a, int type, int act, hipStream_t s);
hipError_t launch_backward8(const Backward8& a, int type, int act, hipStream_t s);
hipError_t launch_decode8(const Decode8& a, int type, hipStream_t s);
hipError_t launch_weight8(const Weight8& a, int type, hipStream_t s);

// The joins of parts: a wave a workgroup, kJoinBatch parts' loads under way together.  A gradient of 128 x 128 in 32
// parts 14.6 us (16384 rows; one load at a time and workgroups of 256: 20.8, 8 at a time 13.7), y of 17 x 512
// in 16 parts of K = 8192 7.9 us (10.8, 8 at a time 8.6).
constexpr int kJoinThreads = 64, kJoinBatch = 4;

// y = a b^T.
// Kernels: up to 16 rows; 32 x 32 with K split over the waves; tiles of 64, 128 and 256; tiles of 64 and 128 with exact
// products, whose result may be float32.
enum Matmul8Variant { kMatmulRows = 0, kMatmulSplit, kMatmulSmall, kMatmulMid, kMatmulTile, kMatmulExactSmall, kMatmulExactMid };
constexpr int kRingStages = 3;      // of 128 K, that kMatmulTile has at least
struct Matmul8 {
    Blocks8 a, b;
    void* y;
    int64_t y_stride;
    int rows, cols, dim;
    int y_vec;               // rows of y 16-byte aligned
    int tiles_v, tiles_t;    // tiles along cols and rows
    int splits, stages_per_split;    // parts of K (tiles of 64 and 128; 1 otherwise), a multiple of 4 stages of 128 each
    float* partial;          // nullable: [split][rows][partial_pitch]
    int64_t partial_pitch;
};
hipError_t launch_matmul8_join(const Matmul8& a, int type, hipStream_t s);
hipError_t launch_matmul8(const Matmul8& a, int type, int variant, hipStream_t s);

// out[c][d] = sum over r of grad[r][c] x[r][d].
struct Grad8 {
    Blocks8 x;
    const void* grad;        // bf16, rows of whole 16-byte chunks
    int64_t grad_stride;     // elements
    int rows, cols, dim;
    int cols8;               // cols rounded up to 8
    int splits, stages_per_split;
    int tiles_c, tiles_d;
    float* out;
    int64_t out_stride;
    int out_vec;             // rows of out 16-byte aligned, dim a multiple of 4
    int accumulate;
    float* partial;          // nullable: [split][cols][partial_pitch]
    int64_t partial_pitch;
};
struct Join8 {
    const float* partial;
    int64_t partial_pitch;
    int splits, cols, dim;   // splits == 0: zeros
    float* out;
    int64_t out_stride;
    int accumulate;
};
hipError_t launch_grad8(const Grad8& a, int edge, bool deep, hipStream_t s);     // tiles of 128 or 256; deep: further ahead, 128 only
hipError_t launch_join8(const Join8& a, hipStream_t s);

}  // namespace muon
