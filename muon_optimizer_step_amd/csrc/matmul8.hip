// y = a b^T on gfx950 for matrices in 8 bits: rows of a (activations, a scale for each
// row and 128 of K) times rows of b (weights, a scale for each 128 x 128).
//
// Mathematics.  y_rc = sum over blocks k of 2^(sa_rk + sb_ck) sum over the block of
// code_a code_b.  Both scales are powers of two, which the scaled MFMAs take as
// bytes: a block's products go into the accumulators unscaled by anything else, at
// the full rate of 8-bit operands, and there is no pass over the accumulators for a block.
// Within a stage of 128 K the order of K does not matter as long as both operands
// have the same, and all of a stage shares its scales; so operands are staged and read like
// 16-bit ones of half the length.
//
// Bound: MFMA for large problems, HBM where there are few rows.
#include <algorithm>

#include "linear8.h"
#include "tiles.h"

namespace muon {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

__device__ inline v8i join(const u32x4& a, const u32x4& b) {
    v8i r;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        r[k] = (int)a[k];
        r[4 + k] = (int)b[k];
    }
    return r;
}
__device__ inline floatx16 mfma8(const v8i& a, const v8i& b, const floatx16& c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, (int)sa, 0, (int)sb);
}

// The scales of 16 stages of one row, a byte each, the current stage's the lowest.
constexpr int kScaleStages = 16;
struct RowScales {
    const uint32_t* row;
    uint32_t w[kScaleStages / 4];
    __device__ inline void init(const Blocks8& b, int64_t r) { row = reinterpret_cast<const uint32_t*>(b.scale + r * b.scale_stride); }
    __device__ inline void load(int stage, int stages) {
#pragma unroll
        for (int k = 0; k < kScaleStages / 4; ++k) w[k] = stage + 4 * k < stages ? row[stage / 4 + k] : 0u;
    }
    __device__ inline void advance() {
#pragma unroll
        for (int k = 0; k + 1 < kScaleStages / 4; ++k) w[k] = __builtin_amdgcn_alignbyte(w[k + 1], w[k], 1);
        w[kScaleStages / 4 - 1] >>= 8;
    }
};

// A wave's tile of TV x 32 columns of y (rows of b, all in one block of 128) x TT x 32 rows.
template <int TV, int TT>
struct Scales {
    RowScales b, a[TT];
    __device__ inline void init(const Matmul8& m, int v0, int t0, int lane) {
        b.init(m.b, min(v0, m.cols - 1) / kBlock8);
#pragma unroll
        for (int j = 0; j < TT; ++j) a[j].init(m.a, min(t0 + 32 * j + lane % 32, m.rows - 1));
    }
    __device__ inline void load(int stage, int stages) {
        b.load(stage, stages);
#pragma unroll
        for (int j = 0; j < TT; ++j) a[j].load(stage, stages);
    }
    __device__ inline void advance() {
        b.advance();
#pragma unroll
        for (int j = 0; j < TT; ++j) a[j].advance();
    }
};

// ---------------------------------------------------------------- K loops
// A step is half a stage: 64 K.
template <int I, typename Op> __device__ inline v8i frag8(const Op& op, uint32_t slot, int step) {
    return join(op.template frag<I>(slot, 2 * step), op.template frag<I>(slot, 2 * step + 1));
}
template <typename Op, int N> __device__ inline void read8(const Op& op, v8i (&f)[N], uint32_t slot, int step) {
    f[0] = frag8<0>(op, slot, step);
    if constexpr (N > 1) f[1] = frag8<1>(op, slot, step);
    if constexpr (N > 2) {
        f[2] = frag8<2>(op, slot, step);
        f[3] = frag8<3>(op, slot, step);
    }
    static_assert(N == 1 || N == 2 || N == 4, "fragments of a wave");
}

// acc += A B^T over `stages` stages of 128 K, which ends after `left` pairs of bytes.  Tile
// 256 x 256, 8 waves of 128 x 64, LDS a ring of five operand slots: A of stage k in
// slot 2 k mod 5, B in 2 k + 1 mod 5.  The barrier is in the middle of a stage, when
// every wave has the fragments of its second half in registers: it frees the stage's two
// slots, which B of stage k + 2 and, half a stage later, A of stage k + 3 are loaded to, and
// publishes stage k + 1, whose first fragments are read while the second half is multiplied.
template <int TA, int TB, typename OA, typename OB>
__device__ inline void k_loop8(floatx16 (&acc)[TA][TB], int stages, OA& A, OB& B, int left, uint32_t lds, int wave, Scales<TA, TB>& s) {
    static_assert(TA == 4 && TB == 2 && OA::kLoads == 4 && OB::kLoads == 4, "eight products and eight loads");
    using std::integral_constant;
    v8i fa[TA], fb[2][TB];
    uint32_t s0 = lds, s1 = lds + kOperand, s2 = lds + 2 * kOperand, s3 = lds + 3 * kOperand, s4 = lds + 4 * kOperand;
    const uint32_t mine = wave * 1024;
    s.load(0, stages);
    load_stage(A, s0 + mine, left);
    load_stage(B, s1 + mine, left);
    if (stages > 1) {
        load_stage(A, s2 + mine, left - kHeadK);
        load_stage(B, s3 + mine, left - kHeadK);
        wait_loads<8>();
    } else {
        wait_loads<0>();
    }
    bare_barrier();
    read8(A, fa, s0, 0);
    read8(B, fb[0], s1, 0);
    auto one = [&](auto& op, auto j, uint32_t dst, bool there, int rest) {
        constexpr int J = decltype(j)::value;
        if (!there) return;
        if (rest >= kHeadK) op.template load<J>(dst + mine);
        else op.template load_tail<J>(dst + mine, rest);
    };
    for (int kt = 0; kt < stages; ++kt) {
        const int rest = left - (kt + 2) * kHeadK;
        const bool ahead = kt + 2 < stages;
        // first half; the second half's fragments; A of stage kt + 2
        read8(B, fb[1], s1, 1);
        auto half = [&](int set, uint32_t slot_a, int step, bool next, auto& op, uint32_t dst) {
            auto row = [&](auto i) {
                constexpr int I = decltype(i)::value;
                acc[I][0] = mfma8(fa[I], fb[set][0], acc[I][0], s.b.w[0], s.a[0].w[0]);
                acc[I][1] = mfma8(fa[I], fb[set][1], acc[I][1], s.b.w[0], s.a[1].w[0]);
                __builtin_amdgcn_sched_barrier(0);
                if (next) fa[I] = frag8<I>(A, slot_a, step);
                one(op, i, dst, ahead, rest);
                __builtin_amdgcn_sched_barrier(0);
            };
            row(integral_constant<int, 0>());
            row(integral_constant<int, 1>());
            row(integral_constant<int, 2>());
            row(integral_constant<int, 3>());
        };
        half(0, s0, 1, true, A, s4);
        A.advance();
        wait_lds();
        const bool next = kt + 1 < stages;
        if (next) {
            if (ahead) wait_loads<4>();
            else wait_loads<0>();
            bare_barrier();
            read8(B, fb[0], s3, 0);
        }
        half(1, s2, 0, next, B, s0);
        B.advance();
        s.advance();
        if (next && (kt + 1) % kScaleStages == 0) s.load(kt + 1, stages);
        const uint32_t t0 = s0, t1 = s1;
        s0 = s2; s1 = s3; s2 = s4; s3 = t0; s4 = t1;
    }
}

// The same for smaller tiles: 4 waves, BUFFERS stages of LDS.
template <int BUFFERS, int TA, int TB, typename OA, typename OB>
__device__ inline void k_loop8_mid(floatx16 (&acc)[TA][TB], int stages, OA& A, OB& B, int left, uint32_t lds, int wave,
                                   Scales<TA, TB>& s) {
    constexpr uint32_t kStage = OA::kBytes + OB::kBytes;
    constexpr int kLoads = OA::kLoads + OB::kLoads;
    const uint32_t mine = wave * 1024;
    uint32_t put = lds, get = lds;
    auto load = [&](int kt) {
        load_stage(A, put + mine, left - kt * kHeadK);
        load_stage(B, put + OA::kBytes + mine, left - kt * kHeadK);
        put = put == lds + (BUFFERS - 1) * kStage ? lds : put + kStage;
    };
    for (int kt = 0; kt < BUFFERS - 1 && kt < stages; ++kt) load(kt);
    for (int k0 = 0; k0 < stages; k0 += kScaleStages) {
        s.load(k0, stages);
        const int end = min(stages, k0 + kScaleStages);
        for (int kt = k0; kt < end; ++kt) {
            if (kt + BUFFERS - 2 < stages) wait_loads<(BUFFERS - 2) * kLoads>();
            else wait_loads<0>();
            wait_lds();
            bare_barrier();      // stage kt is in LDS, and every wave is done with stage kt - 1
            if (kt + BUFFERS - 1 < stages) load(kt + BUFFERS - 1);
#pragma unroll
            for (int step = 0; step < 2; ++step) {
                v8i fa[TA], fb[TB];
                read8(A, fa, get, step);
                read8(B, fb, get + OA::kBytes, step);
#pragma unroll
                for (int i = 0; i < TA; ++i)
#pragma unroll
                    for (int j = 0; j < TB; ++j) acc[i][j] = mfma8(fa[i], fb[j], acc[i][j], s.b.w[0], s.a[j].w[0]);
            }
            s.advance();
            get = get == lds + (BUFFERS - 1) * kStage ? lds : get + kStage;
        }
    }
}

// ---------------------------------------------------------------- output
// acc[tv][tt] holds columns v0 + 32 tv + 16 p + 8 (l / 32) + i (register 8 p + i) of row
// t0 + 32 tt + l % 32.  Through LDS (`stage`, this wave's own), so that a store
// instruction writes whole rows of 32 TV values.
template <int TV> constexpr int kStageBytes = 32 * 32 * TV * 2;
template <typename T, int TV, int TT>
__device__ inline void store_tile(const Matmul8& a, floatx16 (&acc)[TV][TT], int v0, int t0, int lane, uint8_t* stage) {
    constexpr int kChunks = 4 * TV;       // 16-byte chunks of a row; chunk c of row r in slot c ^ (r % kChunks)
    const int half = lane / 32;
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
#pragma unroll
        for (int tv = 0; tv < TV; ++tv)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = acc[tv][tt][8 * p + i];
                const int r = lane % 32, c = 4 * tv + 2 * p + half;
                *reinterpret_cast<u32x4*>(stage + (r * kChunks + (c ^ (r % kChunks))) * 16) = pack8<T>(v);
            }
        // the same wave's data: LDS keeps its order
#pragma unroll
        for (int k = 0; k < kChunks / 2; ++k) {
            const int r = k * (kWave / kChunks) + lane / kChunks, c = lane % kChunks;
            const u32x4 w = *reinterpret_cast<const u32x4*>(stage + (r * kChunks + (c ^ (r % kChunks))) * 16);
            const int row = t0 + 32 * tt + r, v = v0 + 8 * c;
            if (row >= a.rows || v >= a.cols) continue;
            T* dst = static_cast<T*>(a.y) + (int64_t)row * a.y_stride + v;
            if (a.y_vec && v + 8 <= a.cols) {
                *reinterpret_cast<u32x4*>(dst) = w;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (v + e < a.cols) dst[e] = __builtin_bit_cast(T, (uint16_t)(w[e / 2] >> (16 * (e % 2))));
            }
        }
    }
}

// Row tiles in groups of 8, column tiles within: the tiles that an XCD works on at a
// time form a block, which shares operands in its L2.
__device__ inline void tile_of(const Matmul8& a, int item, int& tile_v, int& tile_t) {
    const int group = item / (8 * a.tiles_v), in_group = item - group * 8 * a.tiles_v;
    const int width = min(8, a.tiles_t - 8 * group);
    tile_v = in_group / width;
    tile_t = 8 * group + in_group % width;
}

template <typename T>
__global__ __launch_bounds__(512, 2) void matmul8_kernel(const Matmul8 a) {
    constexpr int WV = 2, WT = 4, TV = 4, TT = 2, NW = WV * WT;
    static_assert(kStageBytes<TV> * NW <= (int)kRingBytes && TV * 32 == kBlock8, "tile");
    extern __shared__ __align__(16) uint8_t lds[];
    const int item = xcd_item(a.tiles_v * a.tiles_t);
    if (item < 0) return;
    int tile_v, tile_t;
    tile_of(a, item, tile_v, tile_t);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wv = wave / WT, wt = wave % WT;
    const int v0 = tile_v * kHeadTile + wv * TV * 32, t0 = tile_t * kHeadTile + wt * TT * 32;
    RowOperand<kHeadTile, NW> B, A;
    B.init(a.b.codes, a.b.stride, (int64_t)tile_v * kHeadTile, a.cols, 0, wv * TV * 32 + swap23(lane % 32), wave, lane);
    A.init(a.a.codes, a.a.stride, (int64_t)tile_t * kHeadTile, a.rows, 0, wt * TT * 32 + lane % 32, wave, lane);
    Scales<TV, TT> s;
    s.init(a, v0, t0, lane);
    floatx16 acc[TV][TT];
    clear(acc);
    k_loop8<TV, TT>(acc, (a.dim + kBlock8 - 1) / kBlock8, B, A, (a.dim + 15) / 16 * 8, lds_address(lds), wave, s);
    bare_barrier();      // every wave is done with the operands, whose slots y passes through
    store_tile<T, TV, TT>(a, acc, v0, t0, lane, lds + wave * kStageBytes<TV>);
}

// 128 x 128, 4 waves of 64 x 64, two workgroups per compute unit.
constexpr int kMid = 128;
constexpr size_t kMidBytes = (size_t)2 * 2 * kMid * kBlock8;
template <typename T>
__global__ __launch_bounds__(256, 2) void matmul8_mid_kernel(const Matmul8 a) {
    constexpr int WV = 2, WT = 2, TV = 2, TT = 2, NW = WV * WT;
    static_assert(kStageBytes<TV> * NW <= (int)kMidBytes, "tile");
    extern __shared__ __align__(16) uint8_t lds[];
    const int item = xcd_item(a.tiles_v * a.tiles_t);
    if (item < 0) return;
    int tile_v, tile_t;
    tile_of(a, item, tile_v, tile_t);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wv = wave / WT, wt = wave % WT;
    const int v0 = tile_v * kMid + wv * TV * 32, t0 = tile_t * kMid + wt * TT * 32;
    RowOperand<kMid, NW> B, A;
    B.init(a.b.codes, a.b.stride, (int64_t)tile_v * kMid, a.cols, 0, wv * TV * 32 + swap23(lane % 32), wave, lane);
    A.init(a.a.codes, a.a.stride, (int64_t)tile_t * kMid, a.rows, 0, wt * TT * 32 + lane % 32, wave, lane);
    Scales<TV, TT> s;
    s.init(a, v0, t0, lane);
    floatx16 acc[TV][TT];
    clear(acc);
    k_loop8_mid<2>(acc, (a.dim + kBlock8 - 1) / kBlock8, B, A, (a.dim + 15) / 16 * 8, lds_address(lds), wave, s);
    bare_barrier();
    store_tile<T, TV, TT>(a, acc, v0, t0, lane, lds + wave * kStageBytes<TV>);
}

// Up to 16 rows: a workgroup for every 16 columns of y, operands straight from memory
// (each row of b is used once), the waves take K in turn, 128 at a time, and meet in LDS.
constexpr int kStreamRows = 16, kStreamCols = 16;
template <typename T, int NW>
__global__ __launch_bounds__(NW * kWave) void matmul8_stream_kernel(const Matmul8 a) {
    __shared__ float part[NW][kStreamCols][kStreamRows];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int v0 = blockIdx.x * kStreamCols, t0 = blockIdx.y * kStreamRows;
    const int v = min(v0 + lane % 16, a.cols - 1), t = min(t0 + lane % 16, a.rows - 1);
    const uint8_t* b = a.b.codes + (int64_t)v * a.b.stride;
    const uint8_t* x = a.a.codes + (int64_t)t * a.a.stride;
    const uint8_t* sb = a.b.scale + (int64_t)(v / kBlock8) * a.b.scale_stride;
    const uint8_t* sa = a.a.scale + (int64_t)t * a.a.scale_stride;
    const int stages = (a.dim + kBlock8 - 1) / kBlock8, dim16 = (a.dim + 15) / 16 * 16;
    floatx4 acc = {0.f, 0.f, 0.f, 0.f};
    auto get = [&](const uint8_t* p, int k) -> u32x4 {
        u32x4 w = {0u, 0u, 0u, 0u};
        if (k < dim16) w = *reinterpret_cast<const u32x4*>(p + k);
        return w;
    };
    for (int kt = wave; kt < stages; kt += NW) {
        const int k = kt * kBlock8 + 32 * (lane / 16);
        const v8i fb = join(get(b, k), get(b, k + 16)), fx = join(get(x, k), get(x, k + 16));
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fx, acc, 0, 0, 0, sb[kt], 0, sa[kt]);
    }
    // register e of lane l: column 4 (l / 16) + e, row l % 16
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][4 * (lane / 16) + e][lane % 16] = acc[e];
    __syncthreads();
    for (int i = threadIdx.x; i < kStreamCols * kStreamRows; i += NW * kWave) {
        const int c = i % kStreamCols, r = i / kStreamCols;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) sum += part[w][c][r];
        if (v0 + c < a.cols && t0 + r < a.rows) static_cast<T*>(a.y)[(int64_t)(t0 + r) * a.y_stride + v0 + c] = (T)sum;
    }
}

template <typename K>
hipError_t allow_lds(K kernel, size_t bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T>
hipError_t typed(const Matmul8& a, int variant, hipStream_t s) {
    if (variant == kMatmulStream) {
        const dim3 grid((a.cols + kStreamCols - 1) / kStreamCols, (a.rows + kStreamRows - 1) / kStreamRows);
        matmul8_stream_kernel<T, 4><<<grid, 4 * kWave, 0, s>>>(a);
        return hipGetLastError();
    }
    const int grid = xcd_grid(a.tiles_v * a.tiles_t);
    if (variant == kMatmulMid) {
        const hipError_t allowed = allow_lds(&matmul8_mid_kernel<T>, kMidBytes);
        if (allowed != hipSuccess) return allowed;
        matmul8_mid_kernel<T><<<grid, 256, kMidBytes, s>>>(a);
        return hipGetLastError();
    }
    const hipError_t allowed = allow_lds(&matmul8_kernel<T>, kRingBytes);
    if (allowed != hipSuccess) return allowed;
    matmul8_kernel<T><<<grid, 512, kRingBytes, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_matmul8(const Matmul8& a, int type, int variant, hipStream_t s) {
    return type == kTypeBf16 ? typed<bf16>(a, variant, s) : typed<f16>(a, variant, s);
}

}  // namespace muon
