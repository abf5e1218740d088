// Kernels of the language-model head's loss on gfx950: softmax cross entropy of
// H W^T without the logits in memory as a whole, and its gradients.
//
// Mathematics, with z_ij = h_i . w_j, l = cap tanh(z / cap) where a cap is set:
//   lse_i = log sum_j exp l_ij;  nll_i = lse_i - l_i,t(i)
//   P_ij = g_i (exp(l_ij - lse_i) - [j = t(i)]) (1 - (l_ij / cap)^2)
//   dH = P W;  dW = P^T H
// head_logits multiplies H W^T tile by tile and reduces each token's logits of
// one sub-tile of the vocabulary to a reference exponent c (base 2) and the sum of
// e_ij = 2^(l_ij log2 e - c); for training it also writes e_ij in fp16 (c is
// the sub-tile's maximum less 15, so the largest e is 2^15: 11 significant
// bits down to 2^-29 of the maximum, which leaves the rounding of P to its
// 16-bit type as the only one that counts).  head_rows joins the sub-tiles of a
// token, head_prob turns e into P in place, and head_grad multiplies P with W
// and P^T with H.  The logits thus cost one product, and only a piece of the
// tokens is in memory at a time.
#include <algorithm>

#include "head.h"

namespace muon {
namespace {

typedef _Float16 f16;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef short short4v __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

template <typename T> __device__ inline floatx16 mfma(const u32x4& a, const u32x4& b, const floatx16& c);
template <> __device__ inline floatx16 mfma<bf16>(const u32x4& a, const u32x4& b, const floatx16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <> __device__ inline floatx16 mfma<f16>(const u32x4& a, const u32x4& b, const floatx16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <typename T> __device__ inline uint32_t pack2(float a, float b);
template <> __device__ inline uint32_t pack2<bf16>(float a, float b) { return pack_bf16x2(a, b); }
template <> __device__ inline uint32_t pack2<f16>(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
}
template <typename T> __device__ inline u32x4 pack8(const float* v) {
    u32x4 r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = pack2<T>(v[2 * k], v[2 * k + 1]);
    return r;
}
template <typename T> __device__ inline void unpack8(const u32x4& w, float* v);
template <> __device__ inline void unpack8<bf16>(const u32x4& w, float* v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) { v[2 * k] = bf16_lo_f(w[k]); v[2 * k + 1] = bf16_hi_f(w[k]); }
}
template <> __device__ inline void unpack8<f16>(const u32x4& w, float* v) {
    const f16x8 h = __builtin_bit_cast(f16x8, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = (float)h[k];
}

template <int N> __device__ inline void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
__device__ inline void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ inline void bare_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// cap tanh(z / cap); exact to a few ulp of cap, which is the scale that counts.
__device__ inline float capped(float z, float cap, float inv_cap) {
    const float t = __builtin_amdgcn_exp2f(z * inv_cap * (2.0f * kLog2e));
    return cap - 2.0f * cap / (t + 1.0f);
}

// 16 bytes per lane straight into LDS, at dst + 16 x lane (dst the wave's).
__device__ inline void direct_load(const uint8_t* src, uint8_t* dst) {
    __builtin_amdgcn_global_load_lds(src, (lds_ptr)dst, 16, 0, 0);
}

// ---------------------------------------------------------------- operand staging
// A row operand (K contiguous): ROWS rows x 128 bytes of K per stage, the
// 16-byte chunk c of row r in slot c ^ ((r / 2) % 8), which keeps the 16-byte
// fragment reads of 32 rows free of bank conflicts.  Direct loads: one wave
// instruction fills 8 rows.
template <int ROWS, int WAVES>
struct RowOperand {
    static constexpr int kBytes = ROWS * 128;
    static constexpr int kLoads = ROWS / 8 / WAVES;
    static_assert(ROWS % (8 * WAVES) == 0, "whole instructions per wave");
    const uint8_t* base;
    uint32_t off[kLoads];
    int chunk;      // source chunk of this lane within a stage

    // rows row0 .. row0 + ROWS of a matrix with `rows` rows; rows beyond its end repeat the last one
    __device__ inline void init(const void* m, int64_t pitch_bytes, int64_t row0, int64_t rows, int wave, int lane) {
        base = static_cast<const uint8_t*>(m) + row0 * pitch_bytes;
        const int last = (int)min<int64_t>(rows - 1 - row0, ROWS - 1);
        chunk = 0;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int r = 8 * (j * WAVES + wave) + lane / 8;
            chunk = (lane % 8) ^ ((r >> 1) & 7);
            off[j] = (uint32_t)(min(r, last) * pitch_bytes) + chunk * 16;
            static_assert(WAVES % 2 == 0, "the chunk is the same for every j");
        }
    }
    __device__ inline void load(uint8_t* lds, int64_t kbyte, int wave) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            direct_load(base + kbyte + off[j], lds + (j * WAVES + wave) * 1024);
    }
    // the last stage where K ends inside it: `chunks` of 8, zeros behind them
    __device__ inline void load_tail(uint8_t* lds, int64_t kbyte, int chunks, int wave, int lane) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            u32x4 v = {0u, 0u, 0u, 0u};
            if (chunk < chunks) v = *reinterpret_cast<const u32x4*>(base + kbyte + off[j]);
            *reinterpret_cast<u32x4*>(lds + (j * WAVES + wave) * 1024 + lane * 16) = v;
        }
    }
    // fragment of 32 rows from `row`: lane l holds row perm(l % 32), K 16 kc + 8 (l / 32) .. + 7
    static __device__ inline u32x4 frag(const uint8_t* lds, int row, int kc, int lane) {
        return *reinterpret_cast<const u32x4*>(lds + row * 128 + (((2 * kc + lane / 32) ^ ((row >> 1) & 7)) << 4));
    }
};

// Row of a 32-row A fragment that MFMA row r stands for: bits 2 and 3 swapped.
// The 32x32 accumulator gives a lane rows 8 q + 4 (l / 32) + e; with the swap the
// values 8 p .. 8 p + 7 of its registers are 8 consecutive rows 16 p + 8 (l / 32) + ..,
// one 16-byte store in a 16-bit type.
__device__ inline int swap23(int r) { return (r & 0x13) | ((r & 4) << 1) | ((r & 8) >> 1); }

// A column operand (K strided): 64 rows of K x 256 columns per stage (512 bytes
// a row), read with the transposing LDS read.  The 16-byte chunk c of row k is
// in slot c ^ 2 f(k % 4), f = 0, 2, 5, 7: the 4 rows x 32 bytes that 16 lanes
// read, and the 4 rows x 64 bytes of 32 lanes, lie in different banks.
template <int WAVES>
struct ColOperand {
    static constexpr int kBytes = kHeadK * 512;
    static constexpr int kLoads = kHeadK / 2 / WAVES;
    const uint8_t* base;
    int64_t pitch;
    uint32_t off[kLoads];
    static __device__ inline int slot_xor(int k) { return 2 * ((0x7520 >> (4 * (k & 3))) & 7); }
    // columns col0 .. of a matrix with cols_pad columns (a multiple of 8); chunks beyond repeat the last
    __device__ inline void init(const void* m, int64_t pitch_bytes, int col0, int cols_pad, int wave, int lane) {
        base = static_cast<const uint8_t*>(m) + (int64_t)col0 * 2;
        pitch = pitch_bytes;
        const int last = (cols_pad - col0) / 8 - 1;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int r = 2 * (j * WAVES + wave) + lane / 32;
            off[j] = (uint32_t)(min((lane % 32) ^ slot_xor(r), last) * 16);
        }
    }
    // K rows k0 .. k0 + 63 of `rows` rows; rows beyond repeat the last
    __device__ inline void load(uint8_t* lds, int64_t k0, int64_t rows, int wave, int lane) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int64_t r = min(k0 + 2 * (j * WAVES + wave) + lane / 32, rows - 1);
            direct_load(base + r * pitch + off[j], lds + (j * WAVES + wave) * 1024);
        }
    }
    // fragment of 32 columns from `col`: lane l holds column (perm of) l % 32, K 16 kc + 8 (l / 32) .. + 7.
    // The transposing read gives lane l' of 16 element l' % 4 of the 8 bytes that lane 4 e + l' / 4 points at.
    template <bool SWAP>
    static __device__ inline u32x4 frag(const uint8_t* lds, int col, int kc, int lane) {
        const int k = 16 * kc + 8 * (lane / 32) + (lane % 16) / 4;
        int quad = lane % 4;
        if (SWAP) quad = ((quad & 1) << 1) | (quad >> 1);
        quad += 4 * ((lane / 16) % 2);
        const int at = ((col / 8 + quad / 2) ^ slot_xor(k)) * 16 + (quad & 1) * 8;
        typedef __attribute__((address_space(3))) short4v lds_short4;
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(lds + k * 512 + at)));
        const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(lds + (k + 4) * 512 + at)));
        u32x4 r;
        r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
        return r;
    }
};

// Work item of this workgroup: workgroups go round-robin over the XCDs, and
// each XCD takes a contiguous range of items, whose operands its L2 shares.
__device__ inline int xcd_item(int items) {
    const int per = (items + kXcds - 1) / kXcds;
    const int at = blockIdx.x / kXcds;
    const int i = (blockIdx.x % kXcds) * per + at;
    return at < per && i < items ? i : -1;
}
inline int xcd_grid(int items) { return (items + kXcds - 1) / kXcds * kXcds; }

// ---------------------------------------------------------------- logits
// What one wave does with its logits: acc[tv][tt] holds 32 vocabulary entries
// (v0 + 32 tv + 16 p + 8 (l / 32) + i in register 8 p + i) of token t0 + 32 tt + l % 32.
template <int TV, int TT, bool STORE, bool CAP>
__device__ inline void logits_epilogue(const HeadLogits& a, floatx16 (&acc)[TV][TT], int v0, int t0, int sub, int lane) {
    const int half = lane / 32;
    const bool whole = v0 + 32 * TV <= a.vocab;
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
        const int token = t0 + 32 * tt + lane % 32;
        float top = -INFINITY;
#pragma unroll
        for (int tv = 0; tv < TV; ++tv)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float z = acc[tv][tt][r];
                if (CAP) z = capped(z, a.cap, a.inv_cap);
                if (!whole && v0 + 32 * tv + 16 * (r / 8) + 8 * half + r % 8 >= a.vocab) z = -INFINITY;
                acc[tv][tt][r] = z;
                top = fmaxf(top, z);
            }
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        // entries beyond the vocabulary only: nothing to add, and no reference
        const float ref = top == -INFINITY ? -INFINITY : top * kLog2e - 15.0f;
        const float minus = top == -INFINITY ? 0.f : -ref;
        float sum = 0.f;
#pragma unroll
        for (int tv = 0; tv < TV; ++tv)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float e[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    e[i] = __builtin_amdgcn_exp2f(fmaf(acc[tv][tt][8 * p + i], kLog2e, minus));
                    sum += e[i];
                }
                if constexpr (STORE) {
                    const int v = v0 + 32 * tv + 16 * p + 8 * half;
                    if (token < a.e_rows && v < a.e_pitch)
                        *reinterpret_cast<u32x4*>(static_cast<f16*>(a.e) + token * a.e_pitch + v) = pack8<f16>(e);
                }
            }
        sum += __shfl_xor(sum, 32, kWave);
        if (half == 0 && token < a.stat_pitch) {
            a.ref[(int64_t)sub * a.stat_pitch + token] = ref;
            a.sum[(int64_t)sub * a.stat_pitch + token] = sum;
        }
    }
}

// Tile of 256 vocabulary entries x 256 tokens: 8 waves of 128 x 64, 32x32x16
// MFMAs, two LDS buffers of 64 K each filled by direct loads.
template <typename T, bool STORE, bool CAP>
__global__ __launch_bounds__(512, 2) void head_logits_kernel(const HeadLogits a) {
    constexpr int WV = 2, WT = 4, TV = 4, TT = 2, BV = WV * TV * 32, BT = WT * TT * 32, NW = WV * WT;
    static_assert(TV * 32 == kHeadSub, "one partial per wave");
    extern __shared__ __align__(16) uint8_t lds[];
    const int item = xcd_item(a.tiles_v * a.tiles_t);
    if (item < 0) return;
    // token tiles in groups of 8, vocabulary tiles within: the tiles that an XCD
    // works on at a time form a block, which shares operands in its L2
    const int group = item / (8 * a.tiles_v), in_group = item - group * 8 * a.tiles_v;
    const int width = min(8, a.tiles_t - 8 * group);
    const int tile_v = in_group / width, tile_t = 8 * group + in_group % width;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, wv = wave / WT, wt = wave % WT;

    typedef RowOperand<BV, NW> WOp;
    typedef RowOperand<BT, NW> HOp;
    WOp W;
    HOp H;
    W.init(a.w, a.w_pitch * 2, (int64_t)tile_v * BV, a.vocab, wave, lane);
    H.init(a.h, a.h_pitch * 2, (int64_t)tile_t * BT, a.tokens, wave, lane);
    constexpr int kStage = WOp::kBytes + HOp::kBytes;
    const int stages = (a.dim + kHeadK - 1) / kHeadK, whole = a.dim / kHeadK;
    auto load = [&](int kt, int b) {
        uint8_t* dst = lds + b * kStage;
        if (kt < whole) {
            W.load(dst, (int64_t)kt * 128, wave);
            H.load(dst + WOp::kBytes, (int64_t)kt * 128, wave);
        } else {
            W.load_tail(dst, (int64_t)kt * 128, a.dim % kHeadK / 8, wave, lane);
            H.load_tail(dst + WOp::kBytes, (int64_t)kt * 128, a.dim % kHeadK / 8, wave, lane);
        }
    };
    floatx16 acc[TV][TT];
#pragma unroll
    for (int i = 0; i < TV; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[i][j] = floatx16(0.f);
    const int arow = wv * TV * 32 + swap23(lane % 32), brow = wt * TT * 32 + lane % 32;
    load(0, 0);
    for (int kt = 0; kt < stages; ++kt) {
        wait_loads<0>();
        wait_lds();
        bare_barrier();      // stage kt is in LDS, and every wave is done with stage kt - 1
        if (kt + 1 < stages) load(kt + 1, (kt + 1) & 1);
        const uint8_t* tw = lds + (kt & 1) * kStage;
        const uint8_t* th = tw + WOp::kBytes;
#pragma unroll
        for (int kc = 0; kc < kHeadK / 16; ++kc) {
            u32x4 fa[TV], fb[TT];
#pragma unroll
            for (int i = 0; i < TV; ++i) fa[i] = WOp::frag(tw, arow + 32 * i, kc, lane);
#pragma unroll
            for (int j = 0; j < TT; ++j) fb[j] = HOp::frag(th, brow + 32 * j, kc, lane);
#pragma unroll
            for (int i = 0; i < TV; ++i)
#pragma unroll
                for (int j = 0; j < TT; ++j) acc[i][j] = mfma<T>(fa[i], fb[j], acc[i][j]);
        }
    }
    logits_epilogue<TV, TT, STORE, CAP>(a, acc, tile_v * BV + wv * TV * 32, tile_t * BT + wt * TT * 32, tile_v * WV + wv, lane);
}

// Up to 32 TT tokens: a workgroup streams 32 vocabulary rows past all of them,
// operands straight from memory (each row of W is used once), the waves take
// every fourth 128 bytes of K and meet in LDS.
template <typename T, int TT, bool STORE, bool CAP>
__global__ __launch_bounds__(256) void head_logits_small_kernel(const HeadLogits a) {
    __shared__ __align__(16) float part[4][TT][16][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int v0 = blockIdx.x * 32;
    const T* w = static_cast<const T*>(a.w) + (int64_t)min(v0 + swap23(lane % 32), a.vocab - 1) * a.w_pitch + 8 * (lane / 32);
    const T* h[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t)
        h[t] = static_cast<const T*>(a.h) + (int64_t)min(32 * t + lane % 32, a.tokens - 1) * a.h_pitch + 8 * (lane / 32);
    floatx16 acc[1][TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[0][t] = floatx16(0.f);
    const int left = a.dim - 8 * (lane / 32);     // this lane's K begins at 8 (l / 32)
    auto get = [&](const T* p, int k) -> u32x4 {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (k < left) v = *reinterpret_cast<const u32x4*>(p + k);
        return v;
    };
    for (int k0 = wave * 64; k0 < a.dim; k0 += 256) {
        u32x4 fw[4], fh[4][TT];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            fw[s] = get(w, k0 + 16 * s);
#pragma unroll
            for (int t = 0; t < TT; ++t) fh[s][t] = get(h[t], k0 + 16 * s);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[0][t] = mfma<T>(fw[s], fh[s][t], acc[0][t]);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) part[wave][t][r][lane] = acc[0][t][r];
    __syncthreads();
    if (wave >= TT) return;
    floatx16 one[1][1];
#pragma unroll
    for (int r = 0; r < 16; ++r)
        one[0][0][r] = (part[0][wave][r][lane] + part[1][wave][r][lane]) + (part[2][wave][r][lane] + part[3][wave][r][lane]);
    logits_epilogue<1, 1, STORE, CAP>(a, one, v0, 32 * wave, blockIdx.x, lane);
}

// ---------------------------------------------------------------- rows
// 256 threads on 256 / S tokens, S threads for each: the sub-tiles' partials
// in a fixed order, the target's logit as a dot product of its own.
template <typename T, int S>
__global__ __launch_bounds__(256) void head_rows_kernel(const HeadRows a) {
    constexpr int R = 256 / S;
    __shared__ float red[256];
    const int r = threadIdx.x % R, s = threadIdx.x / R;
    const int row = blockIdx.x * R + r;
    const bool live = row < a.tokens, held = row < a.rows;
    auto all = [&](float x, auto op) {   // over the S threads of a row, in a fixed order
        __syncthreads();
        red[threadIdx.x] = x;
        __syncthreads();
        for (int w = S / 2; w > 0; w >>= 1) {
            if (s < w) red[threadIdx.x] = op(red[threadIdx.x], red[threadIdx.x + w * R]);
            __syncthreads();
        }
        return red[r];
    };
    float top = -INFINITY;
    if (live)
        for (int k = s; k < a.nsub; k += S) top = fmaxf(top, a.ref[(int64_t)k * a.stat_pitch + row]);
    top = all(top, [](float x, float y) { return fmaxf(x, y); });
    float sum = 0.f;
    if (live)
        for (int k = s; k < a.nsub; k += S)
            sum += a.sum[(int64_t)k * a.stat_pitch + row] *
                   __builtin_amdgcn_exp2f(a.ref[(int64_t)k * a.stat_pitch + row] - top);
    sum = all(sum, [](float x, float y) { return x + y; });
    const float lse2 = top + __builtin_amdgcn_logf(sum);

    const int64_t t = live ? a.targets[row] : a.ignore_index;
    const bool counted = live && t != a.ignore_index, valid = t >= 0 && t < a.vocab;
    float dot = 0.f;
    if (counted && valid) {
        const T* h = static_cast<const T*>(a.h) + (int64_t)row * a.h_pitch;
        const T* w = static_cast<const T*>(a.w) + t * a.w_pitch;
        for (int d = 8 * s; d < a.dim; d += 8 * S) {
            float x[8], y[8];
            unpack8<T>(*reinterpret_cast<const u32x4*>(h + d), x);
            unpack8<T>(*reinterpret_cast<const u32x4*>(w + d), y);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot = fmaf(x[i], y[i], dot);
        }
    }
    dot = all(dot, [](float x, float y) { return x + y; });
    if (a.cap > 0.f) dot = capped(dot, a.cap, a.inv_cap);
    float weight = 0.f;
    if (counted) weight = valid ? (a.train ? (a.weights ? a.weights[row] : a.scalars[0]) * a.scalars[1] : 1.f) : __builtin_nanf("");
    if (s == 0 && live) {
        const float lse = lse2 * kLn2;
        float nll = valid ? lse - dot : __builtin_nanf("");
        if (nll < 0.f) nll = 0.f;       // the target's logit is rounded apart from the sum it is part of
        a.nll[row] = counted ? nll : 0.f;
        if (a.lse) a.lse[row] = counted ? lse : 0.f;
    }
    if (!a.train || !held) return;
    if (s == 0) {
        a.row_weight[row] = weight;
        a.row_target[row] = counted && valid ? (int)t : -1;
    }
    for (int k = s; k < a.nsub; k += S) {
        const int64_t i = (int64_t)k * a.stat_pitch + row;
        a.sum[i] = counted ? __builtin_amdgcn_exp2f(a.ref[i] - lse2) * weight : 0.f;
    }
}

// ---------------------------------------------------------------- probabilities
// 8 rows x 2048 columns of the piece per workgroup, 8 columns of a row per thread.
template <typename T, bool CAP>
__global__ __launch_bounds__(256) void head_prob_kernel(const HeadProb a) {
    const int across = (a.cols + 2047) / 2048, row0 = blockIdx.x / across * 8;
    const int col = (blockIdx.x % across * 256 + threadIdx.x) * 8;
    if (col >= a.cols) return;
    const int sub = col / a.sub;
#pragma unroll 2
    for (int k = 0; k < 8; ++k) {
        const int row = row0 + k;
        if (row >= a.rows) return;
        uint8_t* at = static_cast<uint8_t*>(a.e) + ((int64_t)row * a.e_pitch + col) * 2;
        const float weight = a.row_weight[row];
        u32x4 out = {0u, 0u, 0u, 0u};
        if (weight != 0.f) {     // whatever an ignored token's logits are, its gradient is zero
            const float f = a.factor[(int64_t)sub * a.stat_pitch + row];
            const int target = a.row_target[row] - col;
            float e[8], p[8];
            unpack8<f16>(*reinterpret_cast<const u32x4*>(at), e);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = fmaf(e[i], f, i == target ? -weight : 0.f);
                if (CAP && e[i] > 0.f) {
                    const float x = (a.ref[(int64_t)sub * a.stat_pitch + row] + __builtin_amdgcn_logf(e[i])) * (kLn2 * a.inv_cap);
                    p[i] *= fmaf(-x, x, 1.0f);
                }
            }
            out = pack8<T>(p);
        }
        *reinterpret_cast<u32x4*>(at) = out;
    }
}

// ---------------------------------------------------------------- gradients
// Tile of 256 output columns d x 256 rows, K split over workgroups where the
// tiles alone would leave compute units idle.  A = W or H with K strided; P with K
// contiguous (dH, K the vocabulary) or strided (dW, K the tokens).
template <typename T, bool KTOKEN>
__global__ __launch_bounds__(512, 2) void head_grad_kernel(const HeadGrad a) {
    constexpr int WD = 2, WC = 4, TD = 4, TC = 2, NW = WD * WC;
    extern __shared__ __align__(16) uint8_t lds[];
    const int item = xcd_item(a.tiles_c * a.tiles_d * a.splits);
    if (item < 0) return;
    const int split = item / (a.tiles_c * a.tiles_d), tile = item - split * a.tiles_c * a.tiles_d;
    const int tile_c = tile / a.tiles_d, tile_d = tile % a.tiles_d;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, wd = wave / WC, wc = wave % WC;
    const int d0 = tile_d * kHeadTile, c0 = tile_c * kHeadTile;
    const int s0 = split * a.stages_per_split, s1 = min(a.k / kHeadK, s0 + a.stages_per_split);

    typedef ColOperand<NW> COp;
    typedef RowOperand<kHeadTile, NW> ROp;
    COp A, Q;
    ROp P;
    A.init(a.a, a.a_pitch * 2, d0, (a.dim + 7) / 8 * 8, wave, lane);
    if constexpr (KTOKEN) Q.init(a.p, a.p_pitch * 2, c0, a.p_cols, wave, lane);
    else P.init(a.p, a.p_pitch * 2, c0, a.p_rows, wave, lane);
    constexpr int kStage = 2 * COp::kBytes;
    auto load = [&](int kt, int b) {
        uint8_t* dst = lds + b * kStage;
        A.load(dst, (int64_t)kt * kHeadK, a.a_rows, wave, lane);
        if constexpr (KTOKEN) Q.load(dst + COp::kBytes, (int64_t)kt * kHeadK, a.p_rows, wave, lane);
        else P.load(dst + COp::kBytes, (int64_t)kt * 128, wave);
    };
    floatx16 acc[TD][TC];
#pragma unroll
    for (int i = 0; i < TD; ++i)
#pragma unroll
        for (int j = 0; j < TC; ++j) acc[i][j] = floatx16(0.f);
    if (s0 < s1) load(s0, 0);
    for (int kt = s0; kt < s1; ++kt) {
        wait_loads<0>();
        wait_lds();
        bare_barrier();      // stage kt is in LDS, and every wave is done with stage kt - 1
        if (kt + 1 < s1) load(kt + 1, (kt + 1 - s0) & 1);
        const uint8_t* ta = lds + ((kt - s0) & 1) * kStage;
        const uint8_t* tp = ta + COp::kBytes;
#pragma unroll
        for (int kc = 0; kc < kHeadK / 16; ++kc) {
            u32x4 fa[TD], fb[TC];
#pragma unroll
            for (int i = 0; i < TD; ++i) fa[i] = COp::template frag<true>(ta, wd * TD * 32 + 32 * i, kc, lane);
#pragma unroll
            for (int j = 0; j < TC; ++j) {
                const int c = wc * TC * 32 + 32 * j;
                if constexpr (KTOKEN) fb[j] = COp::template frag<false>(tp, c, kc, lane);
                else fb[j] = ROp::frag(tp, c + lane % 32, kc, lane);
            }
#pragma unroll
            for (int i = 0; i < TD; ++i)
#pragma unroll
                for (int j = 0; j < TC; ++j) acc[i][j] = mfma<T>(fa[i], fb[j], acc[i][j]);
        }
    }
    const float unscale = a.scalars[2];
#pragma unroll
    for (int j = 0; j < TC; ++j) {
        const int c = c0 + wc * TC * 32 + 32 * j + lane % 32;
        if (c >= a.cols) continue;
#pragma unroll
        for (int i = 0; i < TD; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int d = d0 + wd * TD * 32 + 32 * i + 16 * p + 8 * (lane / 32);
                if (d >= a.dim) continue;
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = acc[i][j][8 * p + e];
                if (a.partial) {
                    floatx4* dst = reinterpret_cast<floatx4*>(a.partial + ((int64_t)split * a.cols + c) * a.partial_pitch + d);
                    floatx4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
                    if (a.accumulate) { lo += dst[0]; hi += dst[1]; }
                    dst[0] = lo;
                    dst[1] = hi;
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= unscale;
                T* dst = static_cast<T*>(a.out) + (int64_t)c * a.out_pitch + d;
                if (a.out_vec) *reinterpret_cast<u32x4*>(dst) = pack8<T>(v);
                else
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (d + e < a.dim) dst[e] = (T)v[e];
            }
    }
}

// The splits' sums in order, rounded once.
template <typename T>
__global__ __launch_bounds__(256) void head_join_kernel(const HeadJoin a) {
    const int64_t quads = (a.dim + 3) / 4, items = quads * a.cols;
    const float unscale = a.scalars[2];
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        const int64_t c = i / quads, d = (i - c * quads) * 4;
        floatx4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < a.splits; ++s)
            sum += *reinterpret_cast<const floatx4*>(a.partial + (s * (int64_t)a.cols + c) * a.partial_pitch + d);
        T* dst = static_cast<T*>(a.out) + c * a.out_pitch + d;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < a.dim) dst[e] = (T)(sum[e] * unscale);
    }
}

// ---------------------------------------------------------------- small passes
// Copy with rows padded to whole chunks, ignored rows and rows beyond the end zero.
__global__ __launch_bounds__(256) void head_pack_kernel(const HeadPack a) {
    const int64_t per = a.dst_pitch / 8, items = per * a.rows;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, d = (i - r * per) * 8;
        u32x4 v = {0u, 0u, 0u, 0u};
        if (r < a.src_rows && (!a.targets || a.targets[r] != a.ignore_index)) {
            const uint16_t* src = static_cast<const uint16_t*>(a.src) + r * a.src_pitch + d;
            if (((reinterpret_cast<uintptr_t>(src)) & 15) == 0 && d + 8 <= a.dim) {
                v = *reinterpret_cast<const u32x4*>(src);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (d + e < a.dim) v[e / 2] |= (uint32_t)src[e] << (16 * (e % 2));
            }
        }
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.dst) + r * a.dst_pitch + d) = v;
    }
}

// The weight of a token in the mean, and the power of two that fp16
// probabilities are scaled by (the largest weight becomes 2^13 .. 2^14, so a
// probability of 1e-9 is still a normal number; bf16 has fp32's range).
__global__ __launch_bounds__(1024) void head_scalars_kernel(const HeadScalars a) {
    __shared__ int count[16];
    __shared__ float top[16];
    int n = 0;
    float m = 0.f;
    for (int64_t i = threadIdx.x; i < a.tokens; i += 1024) {
        const bool counted = a.targets[i] != a.ignore_index;
        n += counted;
        if (a.weights && counted) m = fmaxf(m, fabsf(a.weights[i]));
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        n += __shfl_xor(n, off, kWave);
        m = fmaxf(m, __shfl_xor(m, off, kWave));
    }
    if (threadIdx.x % kWave == 0) {
        count[threadIdx.x / kWave] = n;
        top[threadIdx.x / kWave] = m;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < 16; ++w) {
        n += count[w];
        m = fmaxf(m, top[w]);
    }
    const float mean = 1.0f / (float)max(n, 1);
    if (!a.weights) m = mean;
    a.scalars[0] = mean;
    float scale = 1.f;
    if (a.type == kHeadFp16 && m > 1e-30f && m < 1e30f) scale = ldexpf(1.0f, 14 - __builtin_amdgcn_frexp_expf(m));
    a.scalars[1] = scale;
    a.scalars[2] = 1.0f / scale;
}

// sum of weight x nll, in a fixed order.
__global__ __launch_bounds__(1024) void head_loss_kernel(const HeadLoss a) {
    __shared__ float red[16];
    float sum = 0.f;
    for (int64_t i = threadIdx.x; i < a.tokens; i += 1024) {
        const float w = a.row_weight[i];
        if (w != 0.f) sum = fmaf(w, a.nll[i], sum);
    }
    sum = wave_sum(sum);
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = sum;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < 16; ++w) sum += red[w];
    *a.loss = sum * a.scalars[2];
}

template <typename K>
hipError_t allow_lds(K kernel, size_t bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, bool STORE, bool CAP>
hipError_t logits_launch(const HeadLogits& a, bool small, hipStream_t s) {
    if (small) {
        const int groups = (int)(a.e_pitch / kHeadSmallSub);   // the padded columns too: they become zeros
        if (a.tokens <= 32) head_logits_small_kernel<T, 1, STORE, CAP><<<groups, 256, 0, s>>>(a);
        else head_logits_small_kernel<T, 2, STORE, CAP><<<groups, 256, 0, s>>>(a);
        return hipGetLastError();
    }
    constexpr size_t bytes = 2 * 2 * kHeadTile * 128;
    const hipError_t allowed = allow_lds(&head_logits_kernel<T, STORE, CAP>, bytes);
    if (allowed != hipSuccess) return allowed;
    head_logits_kernel<T, STORE, CAP><<<xcd_grid(a.tiles_v * a.tiles_t), 512, bytes, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t logits_typed(const HeadLogits& a, bool small, hipStream_t s) {
    if (a.e) return a.cap > 0.f ? logits_launch<T, true, true>(a, small, s) : logits_launch<T, true, false>(a, small, s);
    return a.cap > 0.f ? logits_launch<T, false, true>(a, small, s) : logits_launch<T, false, false>(a, small, s);
}

template <typename T>
hipError_t rows_typed(const HeadRows& a, hipStream_t s) {
    // many tokens: 16 threads each; few: a workgroup each
    if (a.rows > 256) head_rows_kernel<T, 16><<<(a.rows + 15) / 16, 256, 0, s>>>(a);
    else head_rows_kernel<T, 256><<<a.rows, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t prob_typed(const HeadProb& a, hipStream_t s) {
    const int grid = (a.cols + 2047) / 2048 * ((a.rows + 7) / 8);
    if (a.inv_cap > 0.f) head_prob_kernel<T, true><<<grid, 256, 0, s>>>(a);
    else head_prob_kernel<T, false><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, bool KTOKEN>
hipError_t grad_launch(const HeadGrad& a, hipStream_t s) {
    constexpr size_t bytes = 2 * 2 * kHeadK * 512;
    const hipError_t allowed = allow_lds(&head_grad_kernel<T, KTOKEN>, bytes);
    if (allowed != hipSuccess) return allowed;
    head_grad_kernel<T, KTOKEN><<<xcd_grid(a.tiles_c * a.tiles_d * a.splits), 512, bytes, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_head_logits(const HeadLogits& a, int type, bool small, hipStream_t s) {
    return type == kHeadBf16 ? logits_typed<bf16>(a, small, s) : logits_typed<f16>(a, small, s);
}
hipError_t launch_head_rows(const HeadRows& a, int type, hipStream_t s) {
    return type == kHeadBf16 ? rows_typed<bf16>(a, s) : rows_typed<f16>(a, s);
}
hipError_t launch_head_prob(const HeadProb& a, int type, hipStream_t s) {
    return type == kHeadBf16 ? prob_typed<bf16>(a, s) : prob_typed<f16>(a, s);
}
hipError_t launch_head_grad(const HeadGrad& a, int type, bool k_is_token, hipStream_t s) {
    if (type == kHeadBf16) return k_is_token ? grad_launch<bf16, true>(a, s) : grad_launch<bf16, false>(a, s);
    return k_is_token ? grad_launch<f16, true>(a, s) : grad_launch<f16, false>(a, s);
}
hipError_t launch_head_join(const HeadJoin& a, int type, hipStream_t s) {
    const int64_t groups = std::min<int64_t>(4096, ((int64_t)a.cols * ((a.dim + 3) / 4) + 255) / 256);
    if (type == kHeadBf16) head_join_kernel<bf16><<<(int)groups, 256, 0, s>>>(a);
    else head_join_kernel<f16><<<(int)groups, 256, 0, s>>>(a);
    return hipGetLastError();
}
hipError_t launch_head_pack(const HeadPack& a, hipStream_t s) {
    const int64_t groups = std::min<int64_t>(4096, (a.dst_pitch / 8 * a.rows + 255) / 256);
    head_pack_kernel<<<(int)groups, 256, 0, s>>>(a);
    return hipGetLastError();
}
hipError_t launch_head_scalars(const HeadScalars& a, hipStream_t s) {
    head_scalars_kernel<<<1, 1024, 0, s>>>(a);
    return hipGetLastError();
}
hipError_t launch_head_loss(const HeadLoss& a, hipStream_t s) {
    head_loss_kernel<<<1, 1024, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace muon
