// AdamW with 8-bit states (muonstep_train.h): the kernels, their launchers and
// the C entry points.
//
// Mathematics.  Both moments live as e4m3 codes with a float32 scale per 256
// values.  The first moment is signed; the second is held as its square root
// (rms), which halves its range in octaves: e4m3 covers 2^-9 .. 448, so a
// block holds rms values from its largest down to 1/229376 of it, second
// moments over 35 octaves.  One pass reads the states, updates in fp32, finds
// the block's largest |m| and sqrt(v) and writes the new codes: the states
// are read and written once.
//
// Bound: HBM.  Per value 8 bytes of param, 2 or 4 of grad, 4 of codes and
// 16/256 of scales, 8 more with an EMA, 2 with a bf16 copy.  Measured: 134.2 M values
// of 96 tensors, bf16 gradients and copies, 2.16 GB: 380 us, 5.7 TB/s (a copy of
// 4 GiB: 4.8, reads and writes together); fp32 gradients of one such tensor 365 us, with
// 32-bit states 759, 5.0 TB/s; 4.2 M values: 15.6 us, launch included.  A small
// tensor is bound by latency: 65536 values are 32 workgroups, each wave of which takes
// two blocks one after the other, 5.4 us, about what the host takes to enqueue it.
//
// Layout: one wave per block of 256 values, 4 consecutive values per lane
// (16-byte param and EMA accesses, 4-byte code accesses: 256 contiguous bytes
// per wave), the block's maxima by a wave reduction, no LDS; nothing is read again
// within a step, so loads and stores pass the caches.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "../../include/muonstep_train.h"
#include "common.h"
#include "host.h"

namespace muon {
namespace {

constexpr int kQBlock = MUON_ADAMW8_BLOCK;
constexpr int kA8Threads = 256;
constexpr int kA8Blocks = 2;                                         // blocks of 256 values per wave
constexpr int kA8Elems = kA8Threads / kWave * kA8Blocks * kQBlock;   // values per workgroup
static_assert(kQBlock == 4 * kWave, "one wave covers a block with 4 values per lane");

// One launch holds at most 2^23 workgroups (2^32 threads is the grid's limit),
// and a tensor at most what one launch covers.
constexpr int64_t kA8MaxGroups = (int64_t)1 << 23;
constexpr int64_t kA8MaxElems = kA8MaxGroups * kA8Elems;

enum A8Flags { kA8Vec = 1, kA8GradBf16 = 2 };

struct A8Tensor {
    float* param;
    const void* grad;
    void* m;             // codes, or fp32 where m_scale is NULL
    void* v;
    float* m_scale;
    float* v_scale;
    float* ema;          // nullable
    bf16* copy;          // nullable
    int64_t numel;
    int block_begin;
    uint16_t flags;
    uint16_t place;      // index in the call's list (MUON_MAX_TENSORS fits)
};
struct A8Scalars {
    int n;
    float keep, beta1, omb1, beta2, omb2, step_size, inv_sqrt_bc2, eps, decay, one_minus_decay;
    int dither;
    uint32_t key;        // mixed bits of seed and step
};
// A launch's table is a kernel argument; its size is one of two, so that a
// single tensor's call does not copy a long one.
template <int CHUNK>
struct A8Args {
    A8Scalars s;
    A8Tensor t[CHUNK];
};
constexpr int kA8Short = 8, kA8Chunk = 192;     // tensors per launch

// 32 mixed bits: xor-shifts and odd multipliers (the leading fraction bits of
// sqrt 2 and sqrt 3).
__host__ __device__ inline uint32_t mix32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x ^ (x >> 16);
}

// The largest bits over the wave.  The bits of non-negative floats order like
// the floats, and those of a NaN are above infinity's, so a NaN wins.
__device__ inline uint32_t wave_max_bits(uint32_t x) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const uint32_t y = (uint32_t)__shfl_xor((int)x, off, kWave);
        x = x > y ? x : y;
    }
    return x;
}

__device__ inline uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu; }

// Scale of a block from the bits of its largest magnitude, and the factor
// from values to codes.
__device__ inline void scale_of(uint32_t top_bits, float& scale, float& inverse) {
#pragma clang fp contract(off)
    const float top = __builtin_bit_cast(float, top_bits);
    scale = top_bits < 0x7F800000u ? top * (1.0f / 448.0f) : __builtin_nanf("");
    inverse = top >= 0x1p-100f ? 448.0f * (1.0f / top) : 0.0f;
}

// e4m3 code of the magnitude y = |x| * inverse.  Scaled by 2^-120 its smallest
// normal, 2^-6, becomes the smallest normal of fp32, and the e4m3 code is the
// top bits of the fp32 pattern, subnormals included; `dither` is added to the
// 20 bits that are cut.  Codes end at 448 (126); 127 is NaN.
__device__ inline uint32_t code_of(float magnitude, float inverse, uint32_t dither) {
#pragma clang fp contract(off)
    const float y = magnitude * inverse * 0x1p-120f;
    const uint32_t c = (abs_bits(y) + dither) >> 20;
    return c < 126u ? c : 126u;
}

constexpr uint32_t kHalfDown = 0x7FFFF;   // nearest code, halves to the smaller

// One value: moments, parameter.  Every operation rounds by itself, so that the
// result is the plain formula's in any implementation.
__device__ inline void update_one(const A8Scalars& a, float g, float& m, float& v, float& root, float& p) {
#pragma clang fp contract(off)
    m = m * a.beta1 + g * a.omb1;
    v = v * a.beta2 + (g * g) * a.omb2;
    root = sqrtf(v);
    p = p * a.keep - (m / (root * a.inv_sqrt_bc2 + a.eps)) * a.step_size;
}

__device__ inline float ema_one(const A8Scalars& a, float e, float p) {
#pragma clang fp contract(off)
    return e * a.decay + p * a.one_minus_decay;
}

__device__ inline float code_value(uint32_t word, int k) {
    switch (k) {
        case 0: return __builtin_amdgcn_cvt_f32_fp8((int)word, 0);
        case 1: return __builtin_amdgcn_cvt_f32_fp8((int)word, 1);
        case 2: return __builtin_amdgcn_cvt_f32_fp8((int)word, 2);
        default: return __builtin_amdgcn_cvt_f32_fp8((int)word, 3);
    }
}

template <typename Tab>
__device__ inline int find_entry(const Tab* t, int n, int blk) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t[mid].block_begin <= blk) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// One block of 256 values (or what is left of the tensor) by one wave.
template <bool VEC>
__device__ inline void adamw8_block(const A8Scalars& a, const A8Tensor& T, int64_t base, uint32_t key) {
    const int lane = threadIdx.x % kWave;
    const int64_t i0 = base + 4 * lane;
    const int left = VEC ? 4 : (int)max((int64_t)0, min((int64_t)4, T.numel - i0));   // values of this lane
    const bool q8 = T.m_scale != nullptr, gb = (T.flags & kA8GradBf16) != 0;
    float p[4] = {}, g[4] = {}, m[4] = {}, v[4] = {}, e[4] = {}, root[4] = {};
    uint32_t mw = 0, vw = 0;
    float ms = 0.f, vs = 0.f;
    const float* mf = static_cast<const float*>(T.m);
    const float* vf = static_cast<const float*>(T.v);
    if (q8) {
        ms = T.m_scale[base / kQBlock];
        vs = T.v_scale[base / kQBlock];
    }
    if constexpr (VEC) {
        const floatx4 pv = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(T.param + i0));
        if (q8) {
            mw = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(T.m) + i0));
            vw = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(T.v) + i0));
        } else {
            const floatx4 m4 = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(mf + i0));
            const floatx4 v4 = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(vf + i0));
#pragma unroll
            for (int k = 0; k < 4; ++k) { m[k] = m4[k]; v[k] = v4[k]; }
        }
        if (gb) {
            const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(static_cast<const bf16*>(T.grad) + i0));
            g[0] = bf16_lo_f(w[0]); g[1] = bf16_hi_f(w[0]); g[2] = bf16_lo_f(w[1]); g[3] = bf16_hi_f(w[1]);
        } else {
            const floatx4 gv = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(static_cast<const float*>(T.grad) + i0));
#pragma unroll
            for (int k = 0; k < 4; ++k) g[k] = gv[k];
        }
        if (T.ema) {
            const floatx4 ev = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(T.ema + i0));
#pragma unroll
            for (int k = 0; k < 4; ++k) e[k] = ev[k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = pv[k];
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k >= left) continue;
            p[k] = T.param[i0 + k];
            g[k] = gb ? from_bf16(static_cast<const bf16*>(T.grad)[i0 + k]) : static_cast<const float*>(T.grad)[i0 + k];
            if (q8) {
                mw |= (uint32_t)static_cast<const uint8_t*>(T.m)[i0 + k] << (8 * k);
                vw |= (uint32_t)static_cast<const uint8_t*>(T.v)[i0 + k] << (8 * k);
            } else {
                m[k] = mf[i0 + k];
                v[k] = vf[i0 + k];
            }
            if (T.ema) e[k] = T.ema[i0 + k];
        }
    }
    if (q8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            m[k] = code_value(mw, k) * ms;
            const float r = code_value(vw, k) * vs;
            v[k] = r * r;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k >= left) { m[k] = root[k] = 0.f; continue; }
        update_one(a, g[k], m[k], v[k], root[k], p[k]);
    }
    if (T.ema) {
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = ema_one(a, e[k], p[k]);
    }
    if constexpr (VEC) {
        floatx4 pv, ev;
#pragma unroll
        for (int k = 0; k < 4; ++k) { pv[k] = p[k]; ev[k] = e[k]; }
        __builtin_nontemporal_store(pv, reinterpret_cast<floatx4*>(T.param + i0));
        if (T.ema) __builtin_nontemporal_store(ev, reinterpret_cast<floatx4*>(T.ema + i0));
        if (T.copy) {
            u32x2 w;
            w[0] = pack_bf16x2(p[0], p[1]);
            w[1] = pack_bf16x2(p[2], p[3]);
            __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(T.copy + i0));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k >= left) continue;
            T.param[i0 + k] = p[k];
            if (T.ema) T.ema[i0 + k] = e[k];
            if (T.copy) T.copy[i0 + k] = to_bf16(p[k]);
        }
    }
    if (!q8) {
        float* mo = static_cast<float*>(T.m);
        float* vo = static_cast<float*>(T.v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k >= left) continue;
            mo[i0 + k] = m[k];
            vo[i0 + k] = v[k];
        }
        return;
    }
    uint32_t mt = 0, rt = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        mt = max(mt, abs_bits(m[k]));
        rt = max(rt, abs_bits(root[k]));
    }
    float mi, ri;
    scale_of(wave_max_bits(mt), ms, mi);
    scale_of(wave_max_bits(rt), vs, ri);
    uint32_t mo = 0, vo = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t dm = kHalfDown, dr = kHalfDown;
        if (a.dither) {
            const uint32_t x = mix32(key + (uint32_t)i0 + (uint32_t)k);
            dm = (x >> 16) << 4;
            dr = (x & 0xFFFFu) << 4;
        }
        const uint32_t sign = (__builtin_bit_cast(uint32_t, m[k]) >> 24) & 0x80u;
        const uint32_t cr = code_of(root[k], ri, dr);
        mo |= (code_of(m[k], mi, dm) | sign) << (8 * k);
        vo |= (root[k] > 0.f && cr == 0u ? 1u : cr) << (8 * k);
    }
    if constexpr (VEC) {
        __builtin_nontemporal_store(mo, reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(T.m) + i0));
        __builtin_nontemporal_store(vo, reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(T.v) + i0));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k >= left) continue;
            static_cast<uint8_t*>(T.m)[i0 + k] = (uint8_t)(mo >> (8 * k));
            static_cast<uint8_t*>(T.v)[i0 + k] = (uint8_t)(vo >> (8 * k));
        }
    }
    if (lane == 0) {
        T.m_scale[base / kQBlock] = ms;
        T.v_scale[base / kQBlock] = vs;
    }
}

template <int CHUNK>
__global__ __launch_bounds__(kA8Threads) void adamw8_kernel(const A8Args<CHUNK> args) {
    const A8Scalars& a = args.s;
    const int ti = find_entry(args.t, a.n, blockIdx.x);
    const A8Tensor& T = args.t[ti];
    const uint32_t key = mix32(a.key + T.place);
    const int64_t first = (int64_t)(blockIdx.x - T.block_begin) * kA8Elems;
    const bool vec = (T.flags & kA8Vec) != 0;
    for (int b = 0; b < kA8Blocks; ++b) {
        const int64_t base = first + (int64_t)(b * (kA8Threads / kWave) + threadIdx.x / kWave) * kQBlock;
        if (base >= T.numel) return;
        if (vec && base + kQBlock <= T.numel) adamw8_block<true>(a, T, base, key);
        else adamw8_block<false>(a, T, base, key);
    }
}

constexpr int64_t kStateGroups = 8192;   // workgroups of the two conversions, which stride over the tensor

// fp32 moments -> 8-bit states, one wave per block.
__global__ __launch_bounds__(kA8Threads) void adamw8_encode_kernel(const float* m, const float* v, uint8_t* mc,
                                                                  float* m_scale, uint8_t* rc, float* r_scale,
                                                                  int64_t numel) {
    const int lane = threadIdx.x % kWave;
    for (int64_t block = (int64_t)blockIdx.x * (kA8Threads / kWave) + threadIdx.x / kWave; block * kQBlock < numel;
         block += (int64_t)gridDim.x * (kA8Threads / kWave)) {
        float mv[4], rv[4];
        uint32_t mt = 0, rt = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t i = block * kQBlock + lane + kWave * k;
            mv[k] = i < numel ? m[i] : 0.f;
            rv[k] = i < numel ? sqrtf(v[i]) : 0.f;
            mt = max(mt, abs_bits(mv[k]));
            rt = max(rt, abs_bits(rv[k]));
        }
        float ms, mi, rs, ri;
        scale_of(wave_max_bits(mt), ms, mi);
        scale_of(wave_max_bits(rt), rs, ri);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t i = block * kQBlock + lane + kWave * k;
            if (i >= numel) continue;
            const uint32_t sign = (__builtin_bit_cast(uint32_t, mv[k]) >> 24) & 0x80u;
            const uint32_t cr = code_of(rv[k], ri, kHalfDown);
            mc[i] = (uint8_t)(code_of(mv[k], mi, kHalfDown) | sign);
            rc[i] = (uint8_t)(rv[k] > 0.f && cr == 0u ? 1u : cr);
        }
        if (lane == 0) {
            m_scale[block] = ms;
            r_scale[block] = rs;
        }
    }
}

__global__ __launch_bounds__(kA8Threads) void adamw8_decode_kernel(const uint8_t* mc, const float* m_scale,
                                                                  const uint8_t* rc, const float* r_scale, float* m,
                                                                  float* v, int64_t numel) {
    for (int64_t i = (int64_t)blockIdx.x * kA8Threads + threadIdx.x; i < numel; i += (int64_t)gridDim.x * kA8Threads) {
        const float r = code_value(rc[i], 0) * r_scale[i / kQBlock];
        m[i] = code_value(mc[i], 0) * m_scale[i / kQBlock];
        v[i] = r * r;
    }
}

int validate_moments(const void* mc, const void* ms, const void* rc, const void* rs, const void* m, const void* v,
                     int64_t numel, const char* what) {
    if (numel < 0) return fail(MUON_ERR_INVALID_ARG, "numel = %lld is negative", (long long)numel);
    if (numel > kA8MaxElems)
        return fail(MUON_ERR_UNSUPPORTED, "numel = %lld beyond %lld", (long long)numel, (long long)kA8MaxElems);
    if (numel == 0) return MUON_OK;
    const void* ptr[6] = {mc, rc, ms, rs, m, v};
    std::vector<Span> spans;
    for (int k = 0; k < 6; ++k) {
        if (!ptr[k]) return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
        const uintptr_t lo = reinterpret_cast<uintptr_t>(ptr[k]);
        if (k >= 2 && lo % 4) return fail(MUON_ERR_INVALID_ARG, "%s: pointer %d is not 4-byte aligned", what, k);
        const size_t bytes = k < 2 ? (size_t)numel : k < 4 ? 4 * (size_t)((numel + kQBlock - 1) / kQBlock) : 4 * (size_t)numel;
        spans.push_back({lo, lo + bytes, k});
    }
    return check_overlaps(spans, what);
}

// The kernels over a validated list: table entries of whole tensors, CHUNK per launch.
template <int CHUNK>
int enqueue_adamw8(const adamw8_tensor_t* tensors, int32_t n, const A8Scalars& scalars, hipStream_t s) {
    A8Args<CHUNK> a;
    a.s = scalars;
    for (int i = 0; i < n;) {
        a.s.n = 0;
        int64_t blocks = 0;
        for (; i < n && a.s.n < CHUNK; ++i) {
            const adamw8_tensor_t& x = tensors[i];
            if (x.numel == 0) continue;
            const int64_t nb = (x.numel + kA8Elems - 1) / kA8Elems;
            if (blocks + nb > kA8MaxGroups) break;
            A8Tensor& T = a.t[a.s.n++];
            T.param = x.param;
            T.grad = x.grad;
            T.m = x.exp_avg;
            T.v = x.rms;
            T.m_scale = x.exp_avg_scale;
            T.v_scale = x.rms_scale;
            T.ema = x.ema;
            T.copy = static_cast<bf16*>(x.copy);
            T.numel = x.numel;
            T.block_begin = (int)blocks;
            T.place = (uint16_t)i;
            const uintptr_t wide = reinterpret_cast<uintptr_t>(x.param) | reinterpret_cast<uintptr_t>(x.ema);
            const uintptr_t half = reinterpret_cast<uintptr_t>(x.copy) | (x.grad_bf16 ? reinterpret_cast<uintptr_t>(x.grad) : 0);
            const uintptr_t codes = reinterpret_cast<uintptr_t>(x.exp_avg) | reinterpret_cast<uintptr_t>(x.rms);
            const bool vec = wide % 16 == 0 && (x.grad_bf16 || reinterpret_cast<uintptr_t>(x.grad) % 16 == 0) && half % 8 == 0 &&
                             codes % (x.exp_avg_scale ? 4 : 16) == 0;
            T.flags = (uint16_t)((vec ? kA8Vec : 0) | (x.grad_bf16 ? kA8GradBf16 : 0));
            blocks += nb;
        }
        if (a.s.n == 0) continue;
        hipError_t err = timed_launch("adamw8", s, [&] {
            adamw8_kernel<CHUNK><<<(int)blocks, kA8Threads, 0, s>>>(a);
            return hipGetLastError();
        });
        if (err != hipSuccess) return fail(MUON_ERR_HIP, "adamw8 launch failed: %s", hipGetErrorString(err));
    }
    return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int adamw8_step(const adamw8_tensor_t* tensors, int32_t n, float lr, float beta1, float beta2, float eps,
                float weight_decay, int32_t step, float ema_decay, int32_t dither, uint64_t seed, void* stream) {
    if (!tensors) return fail(MUON_ERR_INVALID_ARG, "tensors is NULL");
    if (n <= 0 || n > MUON_MAX_TENSORS) return fail(MUON_ERR_INVALID_ARG, "n = %d outside [1, %d]", n, MUON_MAX_TENSORS);
    if (!std::isfinite(lr) || !std::isfinite(weight_decay) || !std::isfinite(eps))
        return fail(MUON_ERR_INVALID_ARG, "lr, weight_decay and eps must be finite");
    if (eps < 0.f) return fail(MUON_ERR_INVALID_ARG, "eps must be >= 0");
    if (!(beta1 >= 0.f && beta1 < 1.f) || !(beta2 >= 0.f && beta2 < 1.f))
        return fail(MUON_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
    if (step < 1) return fail(MUON_ERR_INVALID_ARG, "step = %d must be >= 1", step);
    if (!std::isfinite(ema_decay) || ema_decay < 0.f || ema_decay > 1.f)
        return fail(MUON_ERR_INVALID_ARG, "ema_decay must be finite and in [0, 1]");
    if (dither != 0 && dither != 1) return fail(MUON_ERR_INVALID_ARG, "dither = %d is neither 0 nor 1", dither);
    std::vector<Span> spans;
    spans.reserve(8 * (size_t)n);
    for (int i = 0; i < n; ++i) {
        const adamw8_tensor_t& x = tensors[i];
        if (x.numel < 0) return fail(MUON_ERR_INVALID_ARG, "tensor %d: numel = %lld is negative", i, (long long)x.numel);
        if (x.numel > kA8MaxElems)
            return fail(MUON_ERR_UNSUPPORTED, "tensor %d: numel = %lld beyond %lld", i, (long long)x.numel,
                        (long long)kA8MaxElems);
        if (x.grad_bf16 != 0 && x.grad_bf16 != 1)
            return fail(MUON_ERR_INVALID_ARG, "tensor %d: grad_bf16 = %d is neither 0 nor 1", i, x.grad_bf16);
        if ((x.exp_avg_scale == nullptr) != (x.rms_scale == nullptr))
            return fail(MUON_ERR_INVALID_ARG, "tensor %d: exp_avg_scale and rms_scale must both be set (8-bit states) or both NULL", i);
        if (x.numel == 0) continue;
        if (!x.param || !x.grad || !x.exp_avg || !x.rms)
            return fail(MUON_ERR_INVALID_ARG, "tensor %d: param, grad, exp_avg and rms must be non-NULL", i);
        const bool q8 = x.exp_avg_scale != nullptr;
        const size_t m = (size_t)x.numel, nb = (m + kQBlock - 1) / kQBlock, state = q8 ? 1 : 4, grad = x.grad_bf16 ? 2 : 4;
        const struct { const void* p; size_t bytes, align; } buf[8] = {
            {x.param, 4 * m, 4}, {x.grad, grad * m, grad}, {x.exp_avg, state * m, state}, {x.rms, state * m, state},
            {x.exp_avg_scale, 4 * nb, 4}, {x.rms_scale, 4 * nb, 4}, {x.ema, 4 * m, 4}, {x.copy, 2 * m, 2}};
        for (int k = 0; k < 8; ++k) {
            if (!buf[k].p) continue;
            const uintptr_t lo = reinterpret_cast<uintptr_t>(buf[k].p);
            if (lo % buf[k].align)
                return fail(MUON_ERR_INVALID_ARG, "tensor %d: pointer %d is not %d-byte aligned", i, k, (int)buf[k].align);
            spans.push_back({lo, lo + buf[k].bytes, i});
        }
    }
    const int rc = check_overlaps(spans, "adamw8_step");
    if (rc) return rc;
    A8Scalars a;
    const float decayed = lr * weight_decay;
    a.n = 0;
    a.keep = 1.0f - decayed;
    a.beta1 = beta1;
    a.omb1 = 1.0f - beta1;
    a.beta2 = beta2;
    a.omb2 = 1.0f - beta2;
    // bias corrections in double, folded into two fp32 factors
    a.step_size = (float)((double)lr / (1.0 - std::pow((double)beta1, (double)step)));
    a.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow((double)beta2, (double)step)));
    a.eps = eps;
    a.decay = ema_decay;
    a.one_minus_decay = 1.0f - ema_decay;
    a.dither = dither;
    a.key = mix32(((uint32_t)seed ^ mix32((uint32_t)(seed >> 32))) + 0x9E3779B9u * (uint32_t)step);
    hipStream_t s = static_cast<hipStream_t>(stream);
    return n <= kA8Short ? enqueue_adamw8<kA8Short>(tensors, n, a, s) : enqueue_adamw8<kA8Chunk>(tensors, n, a, s);
}

int adamw8_encode(const float* exp_avg, const float* exp_avg_sq, void* exp_avg_codes, float* exp_avg_scale,
                  void* rms_codes, float* rms_scale, int64_t numel, void* stream) {
    int rc = validate_moments(exp_avg_codes, exp_avg_scale, rms_codes, rms_scale, exp_avg, exp_avg_sq, numel, "adamw8_encode");
    if (rc || numel == 0) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t groups = std::min<int64_t>(kStateGroups, (numel + 4 * kQBlock - 1) / (4 * kQBlock));
    hipError_t err = timed_launch("adamw8_encode", s, [&] {
        adamw8_encode_kernel<<<(int)groups, kA8Threads, 0, s>>>(
            exp_avg, exp_avg_sq, static_cast<uint8_t*>(exp_avg_codes), exp_avg_scale, static_cast<uint8_t*>(rms_codes),
            rms_scale, numel);
        return hipGetLastError();
    });
    return err == hipSuccess ? MUON_OK : fail(MUON_ERR_HIP, "adamw8_encode launch failed: %s", hipGetErrorString(err));
}

int adamw8_decode(const void* exp_avg_codes, const float* exp_avg_scale, const void* rms_codes,
                  const float* rms_scale, float* exp_avg, float* exp_avg_sq, int64_t numel, void* stream) {
    int rc = validate_moments(exp_avg_codes, exp_avg_scale, rms_codes, rms_scale, exp_avg, exp_avg_sq, numel, "adamw8_decode");
    if (rc || numel == 0) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t groups = std::min<int64_t>(kStateGroups, (numel + kA8Threads - 1) / kA8Threads);
    hipError_t err = timed_launch("adamw8_decode", s, [&] {
        adamw8_decode_kernel<<<(int)groups, kA8Threads, 0, s>>>(
            static_cast<const uint8_t*>(exp_avg_codes), exp_avg_scale, static_cast<const uint8_t*>(rms_codes), rms_scale,
            exp_avg, exp_avg_sq, numel);
        return hipGetLastError();
    });
    return err == hipSuccess ? MUON_OK : fail(MUON_ERR_HIP, "adamw8_decode launch failed: %s", hipGetErrorString(err));
}

}  // extern "C"
