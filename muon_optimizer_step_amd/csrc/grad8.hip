// The gradient of a linear layer's weight on gfx950 from the 8-bit checkpoint of its
// input: out[c][d] = sum over r of grad[r][c] x[r][d], in float32.
//
// Mathematics.  K runs over the rows, and a row's values have a scale for each 128 of them: a
// scale per K element, which the scaled 8-bit MFMAs have no place for.  So x is decoded to
// bfloat16, exactly (a code has 4 significant bits, the scale is a power of two), on its way
// into LDS: 16 codes of one row and one scale are a lane's load, and become 8
// conversions and two 16-byte writes.  The products are 16-bit ones with the gradient as it is.
//
// Bound: MFMA (16-bit) for large problems; for small matrices the split of K, whose partial
// sums go through memory.
#include <algorithm>

#include "linear8.h"
#include "tiles.h"

namespace muon {
namespace {

// Columns of x for a tile: 64 rows of K x COLS values per stage, decoded, in the layout of
// ColOperand<COLS>.
template <int COLS, int WAVES, int FRAGS>
struct CodeOperand {
    typedef ColOperand<COLS, WAVES, FRAGS> Col;
    static constexpr int kAcross = COLS / 16, kPer = WAVES * kWave / kAcross, kLoads = kHeadK / kPer;
    static_assert(kPer % 4 == 0 && kLoads >= 1, "the swizzle of a lane's rows is the same");
    const uint8_t* code;
    const uint8_t* scale;
    int64_t code_stride, scale_stride;
    int row;
    uint32_t put[2];         // LDS addresses of the lane's two chunks in its first row, less the slot's
    uint32_t at[FRAGS];
    u32x4 w[kLoads];
    uint32_t byte[kLoads];
    __device__ inline void init(const Blocks8& x, int d0, int dim, int64_t k0, int frag0, int thread, int lane) {
        const int chunk = thread % kAcross;
        row = thread / kAcross;
        const int d = min(d0 + 16 * chunk, (dim + 15) / 16 * 16 - 16);
        code_stride = x.stride;
        scale_stride = x.scale_stride;
        code = x.codes + (k0 + row) * code_stride + d;
        scale = x.scale + (k0 + row) * scale_stride + d / kBlock8;
#pragma unroll
        for (int h = 0; h < 2; ++h) put[h] = row * Col::kRow + (((2 * chunk + h) ^ Col::slot_xor(row)) * 16);
        const int k = 8 * (lane / 32) + (lane % 16) / 4;
        int quad = lane % 4;
        quad = ((quad & 1) << 1) | (quad >> 1);
        quad += 4 * ((lane / 16) % 2);
#pragma unroll
        for (int i = 0; i < FRAGS; ++i)
            at[i] = k * Col::kRow + ((((frag0 + 32 * i) / 8 + quad / 2) ^ Col::slot_xor(k)) * 16) + (quad & 1) * 8;
    }
    // the next stage, of which `left` rows exist (zeros behind them)
    __device__ inline void load(int left) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            w[j] = u32x4{0u, 0u, 0u, 0u};
            byte[j] = kScale8Low;
            if (row + j * kPer < left) {
                w[j] = *reinterpret_cast<const u32x4*>(code + j * kPer * code_stride);
                byte[j] = scale[j * kPer * scale_stride];
            }
        }
        code += kHeadK * code_stride;
        scale += kHeadK * scale_stride;
    }
    __device__ inline void store(uint32_t slot) const {
        typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const float f = __builtin_bit_cast(float, byte[j] << 23);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 v;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    v[2 * k] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[j][2 * h + k], f, false));
                    v[2 * k + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[j][2 * h + k], f, true));
                }
                *(lds_u32x4*)(uintptr_t)(slot + put[h] + j * kPer * Col::kRow) = v;
            }
        }
    }
    template <int I> __device__ inline u32x4 frag(uint32_t slot, int kc) const {
        typedef __attribute__((address_space(3))) short4v lds_short4;
        const uint32_t p = at[I] + slot + kc * 16 * Col::kRow;
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(uintptr_t)p));
        const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(uintptr_t)(p + 4 * Col::kRow)));
        return u32x4{a[0], a[1], b[0], b[1]};
    }
};

template <typename Op> __device__ inline void load_zeros(Op& op, uint32_t dst, int left) {
    if (left >= kHeadK) {
        load_stage(op, dst, left);
        return;
    }
    static_assert(Op::kLoads == 4, "loads of a wave");
    op.template load_zeros<0>(dst, left);
    op.template load_zeros<1>(dst, left);
    op.template load_zeros<2>(dst, left);
    op.template load_zeros<3>(dst, left);
    op.advance();
}

// acc += x^T grad over `stages` stages of 64 rows, `left` rows in all.  Two buffers: while a
// stage is multiplied, the next one's gradient is loaded straight to the other buffer,
// its codes, loaded a stage before, are decoded to it, and the codes of the one after are loaded.
template <int TD, int TC, typename OX, typename OG>
__device__ inline void k_loop_coded(floatx16 (&acc)[TD][TC], int stages, OX& X, OG& G, int left, uint32_t lds, int wave) {
    if (stages <= 0) return;
    constexpr uint32_t kX = kHeadK * OX::Col::kRow, kStage = kX + OG::kBytes;
    const uint32_t mine = wave * 1024;
    uint32_t now = lds, other = lds + kStage;
    X.load(left);
    X.store(now);
    load_zeros(G, now + kX + mine, left);
    if (stages > 1) X.load(left - kHeadK);
    for (int kt = 0; kt < stages; ++kt) {
        wait_loads<0>();
        wait_lds();
        bare_barrier();      // stage kt is in LDS, and every wave is done with stage kt - 1
        u32x4 fa[TD], fb[TC];
        auto multiply = [&](int kc) {
            read_step(X, G, fa, fb, now, now + kX, kc);
#pragma unroll
            for (int i = 0; i < TD; ++i)
#pragma unroll
                for (int j = 0; j < TC; ++j) acc[i][j] = mfma<bf16>(fa[i], fb[j], acc[i][j]);
        };
        if (kt + 1 < stages) {
            X.store(other);
            load_zeros(G, other + kX + mine, left - (kt + 1) * kHeadK);
            if (kt + 2 < stages) X.load(left - (kt + 2) * kHeadK);
        }
#pragma unroll
        for (int kc = 0; kc < kHeadK / 16; ++kc) multiply(kc);
        const uint32_t t = now;
        now = other;
        other = t;
    }
}

// A wave's sums to memory: acc[i][j] holds columns d0 + 32 i + 16 p + 8 (l / 32) + e
// (register 8 p + e) of row c0 + 32 j + l % 32.
template <int TD, int TC>
__device__ inline void store_tile(const Grad8& a, floatx16 (&acc)[TD][TC], int split, int d0, int c0, int lane) {
#pragma unroll
    for (int j = 0; j < TC; ++j) {
        const int c = c0 + 32 * j + lane % 32;
        if (c >= a.cols) continue;
#pragma unroll
        for (int i = 0; i < TD; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int d = d0 + 32 * i + 16 * p + 8 * (lane / 32);
                if (d >= a.dim) continue;
                floatx4 v[2];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e / 4][e % 4] = acc[i][j][8 * p + e];
                if (a.partial) {
                    floatx4* dst = reinterpret_cast<floatx4*>(a.partial + ((int64_t)split * a.cols + c) * a.partial_pitch + d);
                    dst[0] = v[0];
                    dst[1] = v[1];
                    continue;
                }
                float* dst = a.out + (int64_t)c * a.out_stride + d;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (a.out_vec) {
                        if (d + 4 * h >= a.dim) continue;
                        floatx4* q = reinterpret_cast<floatx4*>(dst) + h;
                        if (a.accumulate) v[h] += *q;
                        *q = v[h];
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (d + 4 * h + e < a.dim) dst[4 * h + e] = v[h][e] + (a.accumulate ? dst[4 * h + e] : 0.f);
                    }
                }
            }
    }
}

// EDGE x EDGE: 256 with 8 waves of 128 x 64, or 128 with 4 waves of 64 x 64 and two workgroups
// per compute unit.
template <int EDGE> struct GradTile;
template <> struct GradTile<256> { static constexpr int WD = 2, WC = 4, TD = 4, TC = 2; };
template <> struct GradTile<128> { static constexpr int WD = 2, WC = 2, TD = 2, TC = 2; };
template <int EDGE> constexpr int kGradThreads = GradTile<EDGE>::WD * GradTile<EDGE>::WC * kWave;
template <int EDGE> constexpr size_t kGradBytes = (size_t)2 * 2 * EDGE * kHeadK * 2;

template <int EDGE>
__global__ __launch_bounds__(kGradThreads<EDGE>, 2) void grad8_kernel(const Grad8 a) {
    typedef GradTile<EDGE> S;
    constexpr int NW = S::WD * S::WC;
    static_assert(S::WD * S::TD * 32 == EDGE && S::WC * S::TC * 32 == EDGE, "tile");
    extern __shared__ __align__(16) uint8_t lds[];
    const int item = xcd_item(a.tiles_c * a.tiles_d * a.splits);
    if (item < 0) return;
    const int split = item / (a.tiles_c * a.tiles_d), tile = item - split * a.tiles_c * a.tiles_d;
    const int c0 = tile / a.tiles_d * EDGE, d0 = tile % a.tiles_d * EDGE;
    const int s0 = split * a.stages_per_split, s1 = min((a.rows + kHeadK - 1) / kHeadK, s0 + a.stages_per_split);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wd = wave / S::WC, wc = wave % S::WC;
    CodeOperand<EDGE, NW, S::TD> X;
    ColOperand<EDGE, NW, S::TC> G;
    X.init(a.x, d0, a.dim, (int64_t)s0 * kHeadK, wd * S::TD * 32, threadIdx.x, lane);
    G.init(a.grad, a.grad_stride * 2, c0, a.cols8, (int64_t)s0 * kHeadK, wc * S::TC * 32, false, wave, lane);
    floatx16 acc[S::TD][S::TC];
    clear(acc);
    k_loop_coded<S::TD, S::TC>(acc, s1 - s0, X, G, a.rows - s0 * kHeadK, lds_address(lds), wave);
    store_tile<S::TD, S::TC>(a, acc, split, d0 + wd * S::TD * 32, c0 + wc * S::TC * 32, lane);
}

// The splits' sums in order, added to what is there.
__global__ __launch_bounds__(256) void join8_kernel(const Join8 a) {
    const int64_t quads = (a.dim + 3) / 4, items = quads * a.cols;
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < items; n += (int64_t)gridDim.x * 256) {
        const int64_t c = n / quads, d = (n - c * quads) * 4;
        floatx4 v = {0.f, 0.f, 0.f, 0.f};
        const float* src = a.partial + c * a.partial_pitch + d;
        for (int s = 0; s < a.splits; ++s, src += (int64_t)a.cols * a.partial_pitch) v += *reinterpret_cast<const floatx4*>(src);
        float* dst = a.out + c * a.out_stride + d;
        if (a.out_vec) {
            if (a.accumulate) v += *reinterpret_cast<const floatx4*>(dst);
            *reinterpret_cast<floatx4*>(dst) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < a.dim) dst[e] = v[e] + (a.accumulate ? dst[e] : 0.f);
        }
    }
}

template <int EDGE>
hipError_t launch(const Grad8& a, hipStream_t s) {
    const hipError_t allowed = hipFuncSetAttribute(reinterpret_cast<const void*>(&grad8_kernel<EDGE>),
                                                   hipFuncAttributeMaxDynamicSharedMemorySize, (int)kGradBytes<EDGE>);
    if (allowed != hipSuccess) return allowed;
    grad8_kernel<EDGE><<<xcd_grid(a.tiles_c * a.tiles_d * a.splits), kGradThreads<EDGE>, kGradBytes<EDGE>, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grad8(const Grad8& a, bool mid, hipStream_t s) { return mid ? launch<128>(a, s) : launch<256>(a, s); }

hipError_t launch_join8(const Join8& a, hipStream_t s) {
    const int64_t items = (int64_t)a.cols * ((a.dim + 3) / 4);
    join8_kernel<<<(int)std::min<int64_t>(8192, (items + 255) / 256), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace muon
