// Row-wise passes of the linear layers in 8 bits on gfx950: activations and
// weights to e4m3 codes with a power of two as scale for each block, back, and the
// gradient of an activation function from such codes.
//
// Mathematics.  For a block with largest finite magnitude t = m 2^p (1 <= m < 2) the
// scale is 2^e, e = p - 8, or p - 7 where m > 448 / 256: the smallest power with
// t / 2^e <= 448.  It comes from t's bits; value / 2^e is exact (a power of two), so a
// code has the conversion's rounding only, and is the same in any
// implementation.
//
// Bound: HBM; every value is read once and written once (a copy of 4 GiB: 4.7 TB/s, reads and
// writes together).  Measured, inputs from memory: 16384 x 2048 bf16 to its codes and relu2's 23.1 us,
// 5.8 TB/s; 16384 x 4096 bf16 to codes 31.2 us, 6.5; relu2's backward of 16384 x 4096, in 16 and in
// 8 bits, 68 us, 6.0 TB/s; gelu's and silu's 90 and 78 us, for which the vector unit is the limit;
// 8192 x 8192 float32 weights to codes and transposed codes 74 us, 5.5 TB/s; 16384 x 4096 codes to
// bf16 30 us, 6.6.  Small calls are a launch: 2048 values 2.9 us of kernel time.
#include <algorithm>
#include <type_traits>

#include "linear8.h"
#include "tiles.h"

namespace muon {
namespace {

constexpr int kLanes = 16;        // lanes of a block: 8 values each, a row of the DPP operations
constexpr int kThreads = 256;
constexpr int kUnits = kThreads / kLanes;
static_assert(kLanes * 8 == kBlock8, "lanes of a block");

// The largest bits over the 16 lanes of a block, in all of them.
__device__ inline uint32_t block_max(uint32_t x) {
    auto step = [&](uint32_t y) { x = x > y ? x : y; };
    step((uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x128, 15, 15, true));    // row_ror:8
    step((uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x124, 15, 15, true));
    step((uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x122, 15, 15, true));
    step((uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x121, 15, 15, true));
    return x;
}
// The bits of the largest magnitude of N values; FINITE: of the finite ones.  Without it a NaN or an infinity is
// larger than any value, so that a block where there is one is found and looked at again.
constexpr uint32_t kInfBits = 0x7F800000u;
template <bool FINITE, int N> __device__ inline uint32_t top_bits(const float* v) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v[k]) & 0x7FFFFFFFu, x = FINITE && b >= kInfBits ? 0u : b;
        top = top > x ? top : x;
    }
    return top;
}
// The scale's byte from the bits of the block's largest magnitude.
__device__ inline int scale_byte(uint32_t top) {
    const int s = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u);
    return s > kScale8Low ? s : kScale8Low;
}
__device__ inline float scale_value(int byte) { return __builtin_bit_cast(float, (uint32_t)byte << 23); }
__device__ inline float scale_inverse(int byte) { return __builtin_bit_cast(float, (uint32_t)(254 - byte) << 23); }

__device__ inline uint32_t codes4(const float* v, float inverse) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inverse, v[1] * inverse, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inverse, v[3] * inverse, w, true);
}
// A lane's 8 values of a block to codes; every lane of the block takes part.
__device__ inline u32x2 encode8(const float* v, int& byte) {
    uint32_t top = block_max(top_bits<false, 8>(v));
    if (top >= kInfBits) top = block_max(top_bits<true, 8>(v));      // all lanes of the block, or none
    byte = scale_byte(top);
    const float inverse = scale_inverse(byte);
    return u32x2{codes4(v, inverse), codes4(v + 4, inverse)};
}
__device__ inline void decode8(const u32x2& w, float scale, float* v) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[k], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[k], true);
        v[4 * k] = lo[0] * scale;
        v[4 * k + 1] = lo[1] * scale;
        v[4 * k + 2] = hi[0] * scale;
        v[4 * k + 3] = hi[1] * scale;
    }
}

// 8 values as they lie in memory.
template <typename T> struct Raw { u32x4 w[sizeof(T) / 2]; };
template <typename T> __device__ inline void to_float(const Raw<T>& r, float* v) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = as_float(r.w[k / 4][k % 4]);
    } else {
        unpack8<T>(r.w[0], v);
    }
}
template <typename T> __device__ inline Raw<T> from_float(const float* v) {
    Raw<T> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 8; ++k) r.w[k / 4][k % 4] = __builtin_bit_cast(uint32_t, v[k]);
    } else {
        r.w[0] = pack8<T>(v);
    }
    return r;
}
// `left` values are there (zeros behind them).
template <typename T> __device__ inline Raw<T> load8(const T* p, int left) {
    Raw<T> r;
    if (left >= 8) {
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) r.w[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p) + k);
        return r;
    }
    uint32_t word[4 * (sizeof(T) / 2)] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < left) {
            if constexpr (sizeof(T) == 4) word[k] = __builtin_bit_cast(uint32_t, p[k]);
            else word[k / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[k]) << (16 * (k % 2));
        }
#pragma unroll
    for (int k = 0; k < 4 * ((int)sizeof(T) / 2); ++k) r.w[k / 4][k % 4] = word[k];
    return r;
}
// To p0 + at, `whole` starts at p0; through: the rows are 16-byte aligned, and 16-bit values pass the L2.
template <typename T>
__device__ inline void store8(const Through& whole, T* p0, int64_t at, const Raw<T>& r, int left, bool through) {
    T* p = p0 + at;
    if (left >= 8) {
        if (sizeof(T) == 2 && through) {
            whole.store((int)at * 2, r.w[0]);
            return;
        }
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) reinterpret_cast<u32x4_any*>(p)[k] = r.w[k];
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < left) {
            if constexpr (sizeof(T) == 4) p[k] = as_float(r.w[k / 4][k % 4]);
            else p[k] = __builtin_bit_cast(T, (uint16_t)(r.w[0][k / 2] >> (16 * (k % 2))));
        }
}

// ---------------------------------------------------------------- activation functions
// exp(x) for -2^127 <= x <= 0 to a few ulp, subnormal results included (which the instruction itself flushes):
// in base 2, with what the product with log2 e loses (and which would be infinite below).
constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.69314718055994530942f;
__device__ inline float exp_of(float x) {
#pragma clang fp contract(off)      // t is one rounded value in both places
    const float t = x * kLog2e, rest = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -t));
    const bool low = t < -64.f;
    return __builtin_amdgcn_exp2f(t + (low ? 64.f : 0.f)) * fmaf(rest, kLn2, 1.f) * (low ? 0x1p-64f : 1.f);
}
// silu's s = 1 / (1 + exp(-u)) and 1 - s, from exp(-|u|), |u| <= 2^127: no overflow, and digits where either is small.
struct Sigmoid {
    float s, rest;
};
__device__ inline Sigmoid sigmoid(float u) {
    const float e = exp_of(-fabsf(u)), r = __builtin_amdgcn_rcpf(1.f + e);
    return u < 0.f ? Sigmoid{e * r, r} : Sigmoid{r, e * r};
}
// gelu's F(u) = erfc(-u / sqrt 2) / 2 and exp(-u^2 / 2).  erfc(z) = exp(-z^2) t P(t), t = 1 / (1 + p z) for z >= 0 (the form
// of Abramowitz and Stegun 7.1.26), p and the eight degrees of P fitted to exp(z^2) erfc(z) for z up to
// 13.5 (minimax, 3.6e-8 of it; 1e-7 with coefficients of float32's digits, 3.4e-7 in float32; the fit is in
// tests/test_linear8_gelu_host.py): F keeps its digits where it is small, and shares the
// exponential with the derivative.  Beyond |u| = 20 the exponential is zero.
struct Gelu {
    float f, e;
};
__device__ inline Gelu gelu_parts(float u) {
    const float a = fminf(fabsf(u), 20.f), sq = a * a;
    const float e = exp_of(-0.5f * sq) * fmaf(-0.5f, fmaf(a, a, -sq), 1.f);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.70710678118654752440f * 0.4965279f, a, 1.f));
    float q = -0.058656517f;
    q = fmaf(q, t, 0.28751397f);
    q = fmaf(q, t, -0.50514156f);
    q = fmaf(q, t, 0.30710346f);
    q = fmaf(q, t, -0.040894862f);
    q = fmaf(q, t, 0.20874296f);
    q = fmaf(q, t, 0.24065824f);
    q = fmaf(q, t, 0.28055322f);
    q = fmaf(q, t, 0.28012112f);
    const float tail = 0.5f * e * (q * t);
    return {u < 0.f ? tail : 1.f - tail, e};
}
constexpr float kInvRoot2Pi = 0.39894228040143267794f;
__device__ inline float positive(float u) { return u <= 0.f ? 0.f : u; }     // NaN stays
template <int ACT> __device__ inline float act(float u) {
    if (ACT == kActRelu2) {
        const float t = positive(u);
        return t * t;
    }
    if (ACT == kActSilu) return u * sigmoid(__builtin_amdgcn_fmed3f(u, -200.f, 200.f)).s;      // beyond, s is 0 or 1; a NaN stays one
    if (ACT == kActGelu) return u * gelu_parts(u).f;
    return u;
}
// The derivative, relu2's less its factor of 2; u: |u| <= 2^127 or NaN.
template <int ACT> __device__ inline float act_slope(float u) {
    if (ACT == kActRelu2) return positive(u);
    if (ACT == kActSilu) {
        const Sigmoid g = sigmoid(u);
        return g.s * fmaf(u, g.rest, 1.f);
    }
    const Gelu g = gelu_parts(u);
    return fmaf(u * kInvRoot2Pi, g.e, g.f);
}

// ---------------------------------------------------------------- rows
// A workgroup takes kBatch rows of each of its units at a time: their loads are
// under way together.  Two: 1531 x 1000 in fp16, gelu's backward 4.9 us (one row 4.1, four 6.4), 16384 x 4096 in 8 bits
// 34.8 (37.5, 34.6).
constexpr int kBatch = 2;
struct Unit {
    int d;               // the lane's first column
    int block;
    int64_t row0;        // the workgroup's first row
    int row, step;       // the unit's first row from there on, and from one row of the batch to the next
};
template <typename F>
__device__ inline void for_units(const Rows8& r, F work) {
    const int unit = threadIdx.x / kLanes, across = 1 << r.unit_log;
    const int64_t per = (int64_t)kBatch * (kUnits >> r.unit_log);
    const uint32_t items = (uint32_t)r.row_groups * r.col_groups;
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t rg = item / (uint32_t)r.col_groups;
        Unit u;
        u.block = (int)(item - rg * r.col_groups) * across + (unit & (across - 1));
        u.d = u.block * kBlock8 + 8 * (threadIdx.x % kLanes);
        u.step = kUnits >> r.unit_log;
        u.row0 = rg * per;
        u.row = unit >> r.unit_log;
        work(u);
    }
}
__device__ inline void store_codes(const Rows8& r, const Blocks8& b, const Unit& u, int row, const u32x2& w, int byte) {
    if (u.row0 + row >= r.rows || u.d >= r.dim16) return;
    Through(b.codes + u.row0 * b.stride).store(row * (int)b.stride + u.d, w);
    if (threadIdx.x % kLanes == 0) b.scale[(u.row0 + row) * b.scale_stride + u.block] = (uint8_t)byte;
}

template <typename T, int ACT, bool KEEP>
__global__ __launch_bounds__(kThreads) void encode8_kernel(const Encode8 a) {
    for_units(a.r, [&](const Unit& u) {
        Raw<T> raw[kBatch];
        const int left = a.r.dim - u.d;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t row = u.row0 + u.row + k * u.step;
            raw[k] = load8(static_cast<const T*>(a.x) + row * a.x_stride + u.d, row < a.r.rows ? left : 0);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int row = u.row + k * u.step;
            float v[8];
            int byte;
            to_float<T>(raw[k], v);
            if (KEEP) {
                const u32x2 w = encode8(v, byte);
                store_codes(a.r, a.codes, u, row, w, byte);
            }
            if (ACT != kActNone) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = act<ACT>(v[e]);
                const u32x2 w = encode8(v, byte);
                store_codes(a.r, a.out, u, row, w, byte);
            }
        }
    });
}

// Larger scales count as this one (2^113), so that u is finite.  silu's and gelu's derivatives are 1 or 0 from |u| = 200 on, which
// with such scales is every code but zero and NaN; relu2's gets the rest of the scale and its factor of 2 behind the product
// with the gradient, so that nothing is infinite where the result is not.
constexpr int kFarScale = 240;

template <typename T, int ACT>
__global__ __launch_bounds__(kThreads) void backward8_kernel(const Backward8 a) {
    for_units(a.r, [&](const Unit& u) {
        Raw<T> grad[kBatch];
        u32x2 code[kBatch];
        int byte[kBatch];
        const int left = a.r.dim - u.d;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t row = u.row0 + u.row + k * u.step;
            const bool there = row < a.r.rows && left > 0;
            grad[k] = load8(static_cast<const T*>(a.grad) + row * a.grad_stride + u.d, there ? left : 0);
            code[k] = u32x2{0u, 0u};
            byte[k] = kScale8Low;
            if (there) {
                code[k] = *reinterpret_cast<const u32x2*>(a.u.codes + row * a.u.stride + u.d);
                byte[k] = a.u.scale[row * a.u.scale_stride + u.block];
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int row = u.row + k * u.step;
            float v[8], g[8];
            const int near = min(byte[k], kFarScale);
            const float rest = scale_value(128 + byte[k] - near);
            decode8(code[k], scale_value(near), v);
            to_float<T>(grad[k], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (ACT == kActRelu2) g[e] = g[e] * act_slope<ACT>(v[e]) * rest;
                else g[e] *= act_slope<ACT>(v[e]);
            }
            if (a.out && u.row0 + row < a.r.rows) {
                T* first = static_cast<T*>(a.out) + u.row0 * a.out_stride;
                store8(Through(first), first, row * a.out_stride + u.d, from_float<T>(g), left, a.out_through);
            }
            if (a.out8.codes) {
                int b;
                const u32x2 w = encode8(g, b);
                store_codes(a.r, a.out8, u, row, w, b);
            }
        }
    });
}

template <typename T>
__global__ __launch_bounds__(kThreads) void decode8_kernel(const Decode8 a) {
    for_units(a.r, [&](const Unit& u) {
        const int left = a.r.dim - u.d;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t row = u.row0 + u.row + k * u.step;
            if (row >= a.r.rows || left <= 0) continue;
            const u32x2 w = *reinterpret_cast<const u32x2*>(a.x.codes + row * a.x.stride + u.d);
            float v[8];
            decode8(w, scale_value(a.x.scale[row / a.tall * a.x.scale_stride + u.block]), v);
            T* first = static_cast<T*>(a.out) + u.row0 * a.out_stride;
            store8(Through(first), first, (row - u.row0) * a.out_stride + u.d, from_float<T>(v), left, a.out_through);
        }
    });
}

// ---------------------------------------------------------------- weights
// A workgroup for each 128 x 128 block.  A lane holds 4 x 4 values of each of 4 pieces:
// 4 rows of 4 consecutive columns, so that both layouts are written from registers
// in words: rows straight to memory (32 lanes cover a row's 128 bytes), columns
// through LDS, whose word (column, 4 rows) sits in slot rows ^ column / 4 ^ column % 4 of its
// column: the 32 lanes that write a row group meet 32 different banks, and so do those that read four columns.
// 8192 x 8192 float32 74 us, 62 where consecutive calls have one input (5.5 and 6.5 TB/s); bfloat16 54 and 43 us (56 and 44
// with its results left in the L2, 72 with loads that wait for one another besides); 512 x 512 4.0 us: 16 workgroups, a launch.
template <typename T> using Quad = std::conditional_t<sizeof(T) == 4, u32x4, u32x2>;      // 4 values as they lie in memory
template <typename T> __device__ inline Quad<T> load_quad(const T* p) {
    if constexpr (sizeof(T) == 4) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
    else return __builtin_nontemporal_load(reinterpret_cast<const u32x2_any*>(p));
}
template <typename T>
__global__ __launch_bounds__(kThreads) void weight8_kernel(const Weight8 a) {
    __shared__ uint32_t tops[kThreads / kWave];
    __shared__ uint32_t turned[kBlock8][kBlock8 / 4];
    const int across = (a.dim + kBlock8 - 1) / kBlock8;
    const int br = blockIdx.x / across, bd = blockIdx.x % across;
    const int col = 4 * (threadIdx.x % 32), group = threadIdx.x / 32;     // rows 4 (group + 8 q) + j
    const int d = bd * kBlock8 + col, row0 = br * kBlock8;
    // All loads are issued before the first value is looked at.  Rows behind the last repeat it, and are zeros below.
    Quad<T> raw[4][4];
    auto at = [&](int q, int j) {
        return static_cast<const T*>(a.w) + (int64_t)min(row0 + 4 * (group + 8 * q) + j, a.rows - 1) * a.w_stride + d;
    };
    if (d + 4 <= a.dim) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) raw[q][j] = load_quad<T>(at(q, j));
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) raw[q][j] = Quad<T>{};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < a.dim) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (sizeof(T) == 4) raw[q][j][e] = __builtin_bit_cast(uint32_t, at(q, j)[e]);
                        else raw[q][j][e / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, at(q, j)[e]) << (16 * (e % 2));
                    }
            }
    }
    float v[4][4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool there = row0 + 4 * (group + 8 * q) + j < a.rows;
            float x[8];
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = as_float(raw[q][j][e]);
            } else {
                unpack8<T>(u32x4{raw[q][j][0], raw[q][j][1], 0u, 0u}, x);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[q][j][e] = there ? x[e] : 0.f;
        }
    auto block_top = [&](auto finite) {
        uint32_t top = block_max(top_bits<decltype(finite)::value, 64>(&v[0][0][0]));
#pragma unroll
        for (int off = 16; off < kWave; off <<= 1) {
            const uint32_t y = (uint32_t)__shfl_xor((int)top, off, kWave);
            top = top > y ? top : y;
        }
        if (threadIdx.x % kWave == 0) tops[threadIdx.x / kWave] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / kWave; ++w) top = top > tops[w] ? top : tops[w];
        return top;
    };
    uint32_t top = block_top(std::false_type());
    if (top >= kInfBits) {       // the whole workgroup, or none of it
        __syncthreads();
        top = block_top(std::true_type());
    }
    const int byte = scale_byte(top);
    const float inverse = scale_inverse(byte);
    const int dim16 = (a.dim + 15) / 16 * 16, rows16 = (a.rows + 15) / 16 * 16;
    if (threadIdx.x == 0) {
        a.codes.scale[br * a.codes.scale_stride + bd] = (uint8_t)byte;
        if (a.transposed.codes) a.transposed.scale[bd * a.transposed.scale_stride + br] = (uint8_t)byte;
    }
    const Through rows_out(a.codes.codes + (int64_t)row0 * a.codes.stride);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = row0 + 4 * (group + 8 * q) + j;
            w[j] = codes4(v[q][j], inverse);
            if (row < a.rows && d < dim16) rows_out.store((row - row0) * (int)a.codes.stride + d, w[j]);
        }
        if (a.transposed.codes) {
            // 4 x 4 bytes turned: pairs of rows, then pairs of pairs
            const uint32_t lo01 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), hi01 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
            const uint32_t lo23 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), hi23 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
            const int slot = (group + 8 * q) ^ (col / 4);
            turned[col][slot] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
            turned[col + 1][slot ^ 1] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
            turned[col + 2][slot ^ 2] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
            turned[col + 3][slot ^ 3] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
        }
    }
    if (!a.transposed.codes) return;
    __syncthreads();
    const Through turned_out(a.transposed.codes + (int64_t)bd * kBlock8 * a.transposed.stride);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = threadIdx.x / 8 + 32 * k, chunk = threadIdx.x % 8;
        const int out_row = bd * kBlock8 + c, out_col = row0 + 16 * chunk;
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = turned[c][(4 * chunk + e) ^ (c / 4) ^ (c % 4)];
        if (out_row < a.dim && out_col < rows16)
            turned_out.store(c * (int)a.transposed.stride + out_col, w);
    }
}

// Workgroups of a row-wise pass: enough to fill the chip many times over, the rest
// by the kernel's own loop.
int rows_grid(const Rows8& r) { return (int)std::min<int64_t>((int64_t)r.row_groups * r.col_groups, 1 << 20); }

template <typename T, int ACT, bool KEEP>
hipError_t encode_kept(const Encode8& a, hipStream_t s) {
    encode8_kernel<T, ACT, KEEP><<<rows_grid(a.r), kThreads, 0, s>>>(a);
    return hipGetLastError();
}
template <typename T, int ACT>
hipError_t encode_typed(const Encode8& a, hipStream_t s) {
    if (ACT == kActNone || a.codes.codes) return encode_kept<T, ACT, true>(a, s);
    return encode_kept<T, ACT, ACT == kActNone>(a, s);
}
template <typename T>
hipError_t encode_act(const Encode8& a, int act, hipStream_t s) {
    if (act == kActRelu2) return encode_typed<T, kActRelu2>(a, s);
    if (act == kActSilu) return encode_typed<T, kActSilu>(a, s);
    if (act == kActGelu) return encode_typed<T, kActGelu>(a, s);
    return encode_typed<T, kActNone>(a, s);
}
template <typename T, int ACT>
hipError_t backward_typed(const Backward8& a, hipStream_t s) {
    backward8_kernel<T, ACT><<<rows_grid(a.r), kThreads, 0, s>>>(a);
    return hipGetLastError();
}
template <typename T>
hipError_t backward_act(const Backward8& a, int act, hipStream_t s) {
    if (act == kActRelu2) return backward_typed<T, kActRelu2>(a, s);
    return act == kActSilu ? backward_typed<T, kActSilu>(a, s) : backward_typed<T, kActGelu>(a, s);
}
template <typename T>
hipError_t decode_typed(const Decode8& a, hipStream_t s) {
    decode8_kernel<T><<<rows_grid(a.r), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

Rows8 plan(const Rows8& r) {
    Rows8 q = r;
    const int blocks = (q.dim + kBlock8 - 1) / kBlock8;
    q.dim16 = (q.dim + 15) / 16 * 16;
    q.unit_log = 0;
    while (q.unit_log < 4 && (1 << q.unit_log) < blocks) ++q.unit_log;
    q.col_groups = (blocks + (1 << q.unit_log) - 1) >> q.unit_log;
    const int64_t per = (int64_t)kBatch * (kUnits >> q.unit_log);
    q.row_groups = (int)((q.rows + per - 1) / per);
    return q;
}

}  // namespace

hipError_t launch_encode8(const Encode8& a0, int type, int act, hipStream_t s) {
    Encode8 a = a0;
    a.r = plan(a0.r);
    if (type == kTypeBf16) return encode_act<bf16>(a, act, s);
    return type == kTypeFp16 ? encode_act<f16>(a, act, s) : encode_act<float>(a, act, s);
}
hipError_t launch_backward8(const Backward8& a0, int type, int act, hipStream_t s) {
    Backward8 a = a0;
    a.r = plan(a0.r);
    if (type == kTypeBf16) return backward_act<bf16>(a, act, s);
    return type == kTypeFp16 ? backward_act<f16>(a, act, s) : backward_act<float>(a, act, s);
}
hipError_t launch_decode8(const Decode8& a0, int type, hipStream_t s) {
    Decode8 a = a0;
    a.r = plan(a0.r);
    if (type == kTypeBf16) return decode_typed<bf16>(a, s);
    return type == kTypeFp16 ? decode_typed<f16>(a, s) : decode_typed<float>(a, s);
}
hipError_t launch_weight8(const Weight8& a, int type, hipStream_t s) {
    const int64_t grid = (int64_t)((a.rows + kBlock8 - 1) / kBlock8) * ((a.dim + kBlock8 - 1) / kBlock8);
    if (type == kTypeBf16) weight8_kernel<bf16><<<(int)grid, kThreads, 0, s>>>(a);
    else if (type == kTypeFp16) weight8_kernel<f16><<<(int)grid, kThreads, 0, s>>>(a);
    else weight8_kernel<float><<<(int)grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace muon
