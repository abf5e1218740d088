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
// The matrix unit adds 8 products at a time, each cut to 2^-13 of the largest of them, and its sums of 8
// enter the float32 accumulators: 2.6e-5 of y in norm, where rounding y to 16 bits costs 1.7e-3
// (bfloat16) or 2e-4 (float16).  A float32 y would show the difference: it is computed from exact products (below), and so
// are 16-bit ones where the caller asks for it.
//
// Bound and measured, 8-bit products: MFMA for large problems (8192^3: 431 to 440 us, 2.5 PFLOP/s; 400 us, 2.75, where consecutive calls
// have one input; a library's 8-bit product with one scale for each matrix reaches 2.64; MFMA busy two
// thirds of the cycles); y's bytes where K is short (16384 x 2048 x 512: 23.4 to 25.6 us, 3.2 TB/s; MFMA 23 %); the weights' bytes where there are
// few rows (1 x 8192 x 8192 13 us, 5.2 TB/s; 64 x 8192 x 8192 20 us); below, a launch (1 x 4096 x 1024 4.2 us, of which
// 3.2 in the kernel).  Rows of codes off the 128-byte grid cost a quarter (3000 x 700 x 5000: 40 us, K = 4992 32),
// so encoded matrices have whole lines where dim > 512.
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
    // stage0: a multiple of 4
    __device__ inline void init(const Blocks8& b, int64_t r, int stage0) {
        row = reinterpret_cast<const uint32_t*>(b.scale + r * b.scale_stride + stage0);
    }
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
    __device__ inline void init(const Matmul8& m, int v0, int t0, int stage0, int lane) {
        b.init(m.b, min(v0, m.cols - 1) / kBlock8, stage0);
#pragma unroll
        for (int j = 0; j < TT; ++j) a[j].init(m.a, min(t0 + 32 * j + lane % 32, m.rows - 1), stage0);
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

// acc += A B^T over `stages` stages (kRingStages or more) of 128 K, which ends after `left` pairs of bytes.  Tile
// 256 x 256, 8 waves of 128 x 64, LDS a ring of five operand slots: A of stage k in
// slot 2 k mod 5, B in 2 k + 1 mod 5.  The barrier is in the middle of a stage, when
// every wave has the fragments of its second half in registers: it frees the stage's two
// slots, which B of stage k + 2 and, half a stage later, A of stage k + 3 are loaded to, and
// publishes stage k + 1, whose first fragments are read while the second half is multiplied.
// A fragment is read into its own registers as soon as its last product is issued, four
// products before the next one that needs it, and one load follows every second product.
// A stage is 1.55 us in the whole chip's use (1.3 at the matrix unit's rate); the same loop with
// branches spilled hundreds of registers (585 us for 8192^3), raised wave priority around the products changed nothing.
//
// Where K ends inside the last stage, the chunks behind it are loaded from the stage's
// beginning, so that nothing is read out of range, and B's fragments of them are zero (what A
// has there is of the same row: a NaN is in the row's sums anyway).  The body of the loop then has no
// branch, across which the compiler would move products away from what they are to overlap.
template <int TA, int TB, typename OA, typename OB>
__device__ inline void k_loop8(floatx16 (&acc)[TA][TB], int stages, OA& A, OB& B, int left, uint32_t lds, int wave, int lane,
                               Scales<TA, TB>& s) {
    static_assert(TA == 4 && TB == 2 && OA::kLoads == 4 && OB::kLoads == 4, "eight products and eight loads");
    using std::integral_constant;
    v8i fa[TA], fb, fc[2];       // of A; of B: the first, and the second for each half
    uint32_t s0 = lds, s1 = lds + kOperand, s2 = lds + 2 * kOperand, s3 = lds + 3 * kOperand, s4 = lds + 4 * kOperand;
    const uint32_t mine = wave * 1024;
    const int part = left % kHeadK;
    const uint32_t behind = part && 8 * A.chunk >= part ? 16 * A.chunk : 0;      // the same chunk of B
    auto load_all = [&](auto& op, uint32_t dst, uint32_t less) {
        op.template load_before<0>(dst, less);
        op.template load_before<1>(dst, less);
        op.template load_before<2>(dst, less);
        op.template load_before<3>(dst, less);
        op.advance();
    };
    // fragment I of B in half `step` of the last stage
    auto frag_last = [&](auto i, uint32_t slot, int step) {
        u32x4 w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            w[k] = B.template frag<decltype(i)::value>(slot, 2 * step + k);
            const bool there = !part || 16 * (2 * step + k) + 8 * (lane / 32) < part;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[k][e] = there ? w[k][e] : 0u;
        }
        return join(w[0], w[1]);
    };
    s.load(0, stages);
    load_all(A, s0 + mine, 0);
    load_all(B, s1 + mine, 0);
    load_all(A, s2 + mine, 0);
    load_all(B, s3 + mine, 0);
    wait_loads<8>();
    bare_barrier();
    read8(A, fa, s0, 0);
    fb = frag8<0>(B, s1, 0);
    fc[0] = frag8<1>(B, s1, 0);
    // a stage that loads another one; the last but one, the last
    enum { kLoads, kBeforeLast, kLast };
    auto stage = [&](auto kind, uint32_t less) {
        constexpr int kKind = decltype(kind)::value;
        // half a stage: its products, four loads of `op`, and the fragments of the half that follows
        auto half = [&](auto second, auto& op, uint32_t dst, uint32_t next_a, uint32_t next_b) {
            constexpr int H = decltype(second)::value;
            constexpr bool kNext = !(kKind == kLast && H == 1), kMasked = kKind == kLast || (kKind == kBeforeLast && H == 1);
            auto next_of_b = [&](auto i) {
                if constexpr (kMasked) return frag_last(i, next_b, 1 - H);
                else return frag8<decltype(i)::value>(B, next_b, 1 - H);
            };
            auto first = [&](auto i) {
                constexpr int I = decltype(i)::value;
                acc[I][0] = mfma8(fa[I], fb, acc[I][0], s.b.w[0], s.a[0].w[0]);
                if (I % 2 == 1) {
                    __builtin_amdgcn_sched_barrier(0);
                    if (kKind == kLoads) op.template load_before<I / 2>(dst + mine, less);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            auto then = [&](auto i) {
                constexpr int I = decltype(i)::value;
                acc[I][1] = mfma8(fa[I], fc[H], acc[I][1], s.b.w[0], s.a[1].w[0]);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (kNext) fa[I] = frag8<I>(A, next_a, 1 - H);
                if (I % 2 == 1 && kKind == kLoads) op.template load_before<2 + I / 2>(dst + mine, less);
                __builtin_amdgcn_sched_barrier(0);
            };
            if constexpr (kNext) fc[1 - H] = next_of_b(integral_constant<int, 1>());
            first(integral_constant<int, 0>());
            first(integral_constant<int, 1>());
            first(integral_constant<int, 2>());
            first(integral_constant<int, 3>());
            if constexpr (kNext) fb = next_of_b(integral_constant<int, 0>());
            then(integral_constant<int, 0>());
            then(integral_constant<int, 1>());
            then(integral_constant<int, 2>());
            then(integral_constant<int, 3>());
        };
        half(integral_constant<int, 0>(), A, s4, s0, s1);
        A.advance();
        if constexpr (kKind != kLast) {
            wait_lds();          // this wave's last fragments of the stage
            wait_loads<kKind == kLoads ? 4 : 0>();
            bare_barrier();
        }
        half(integral_constant<int, 1>(), B, s0, s2, s3);
        B.advance();
        s.advance();
        const uint32_t t0 = s0, t1 = s1;
        s0 = s2; s1 = s3; s2 = s4; s3 = t0; s4 = t1;
    };
    int kt = 0;
    while (kt < stages - 2) {
        const int end = min(stages - 2, kt + kScaleStages);
#pragma unroll 1
        for (; kt < end; ++kt) stage(integral_constant<int, kLoads>(), kt + 3 == stages ? behind : 0);
        if (kt % kScaleStages == 0) s.load(kt, stages);
    }
    stage(integral_constant<int, kBeforeLast>(), 0);
    if (++kt % kScaleStages == 0) s.load(kt, stages);
    stage(integral_constant<int, kLast>(), 0);
}

// Waits until at most `stages` stages of LOADS loads are under way.
template <int LOADS> __device__ inline void wait_stages(int stages) {
    static_assert(6 * LOADS < 64, "the counter's range");
    switch (stages) {
        case 0: wait_loads<0>(); break;
        case 1: wait_loads<LOADS>(); break;
        case 2: wait_loads<2 * LOADS>(); break;
        case 3: wait_loads<3 * LOADS>(); break;
        case 4: wait_loads<4 * LOADS>(); break;
        case 5: wait_loads<5 * LOADS>(); break;
        default: wait_loads<6 * LOADS>();
    }
}

// The products of half a stage, on top of acc.
template <int TA, int TB>
__device__ inline void multiply8(floatx16 (&acc)[TA][TB], const v8i (&fa)[TA], const v8i (&fb)[TB], const Scales<TA, TB>& s) {
#pragma unroll
    for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = mfma8(fa[i], fb[j], acc[i][j], s.b.w[0], s.a[j].w[0]);
}

// The same without the scales, with every digit: a code is a bfloat16 value, the 16-bit instruction's products are
// exact and its sums float32.  A step's 32 codes of a lane go to four products of 16 K; which K a lane's codes are
// does not matter, as both operands have the same.  The scales come to a stage's sums, so that any power of two will do.
// Half of the 8-bit rate at best: 8192^3 1020 us, 1.08 PFLOP/s of the 1.36 that a 16-bit library product reaches;
// 16384 x 2048 x 512 54 us, y's 134 MB 29 of them at a copy's rate; 1021 x 2000 x 1000 11 us.
__device__ inline void widen8(const v8i& codes, u32x4 (&w)[4]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        w[k / 2][2 * (k % 2)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[k], 1.f, false));
        w[k / 2][2 * (k % 2) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[k], 1.f, true));
    }
}
template <int TA, int TB>
__device__ inline void multiply_exact(floatx16 (&sums)[TA][TB], const v8i (&fa)[TA], const v8i (&fb)[TB]) {
    u32x4 wa[TA][4], wb[TB][4];
#pragma unroll
    for (int i = 0; i < TA; ++i) widen8(fa[i], wa[i]);
#pragma unroll
    for (int j = 0; j < TB; ++j) widen8(fb[j], wb[j]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < TA; ++i)
#pragma unroll
            for (int j = 0; j < TB; ++j) sums[i][j] = mfma<bf16>(wa[i][k], wb[j][k], sums[i][j]);
}
// acc += a stage's sums times both scales, whatever powers of two these are.
template <int TA, int TB>
__device__ inline void add_scaled(floatx16 (&acc)[TA][TB], const floatx16 (&sums)[TA][TB], const Scales<TA, TB>& s) {
#pragma unroll
    for (int j = 0; j < TB; ++j) {
        const int power = (int)(s.b.w[0] & 0xFFu) + (int)(s.a[j].w[0] & 0xFFu) - 254;
#pragma unroll
        for (int i = 0; i < TA; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] += ldexpf(sums[i][j][e], power);
    }
}

// The same for tiles of 128 x 128 by 4 waves, two buffers, two workgroups on a compute unit that fill
// each other's waits: 4096 x 2048 x 2048 19 us (64: 35, 256: 25).  EXACT: sums in float32 (above).
template <bool EXACT, int TA, int TB, typename OA, typename OB>
__device__ inline void k_loop8_mid(floatx16 (&acc)[TA][TB], int stages, OA& A, OB& B, int left, uint32_t lds, int wave,
                                   Scales<TA, TB>& s) {
    constexpr uint32_t kStage = OA::kBytes + OB::kBytes;
    const uint32_t mine = wave * 1024;
    uint32_t now = lds, other = lds + kStage;
    load_stage(A, now + mine, left);
    load_stage(B, now + OA::kBytes + mine, left);
    for (int k0 = 0; k0 < stages; k0 += kScaleStages) {
        s.load(k0, stages);
        const int end = min(stages, k0 + kScaleStages);
        for (int kt = k0; kt < end; ++kt) {
            wait_loads<0>();
            wait_lds();
            bare_barrier();      // stage kt is in LDS, and every wave is done with stage kt - 1
            if (kt + 1 < stages) {
                load_stage(A, other + mine, left - (kt + 1) * kHeadK);
                load_stage(B, other + OA::kBytes + mine, left - (kt + 1) * kHeadK);
            }
            v8i fa[TA], fb[TB];
            if constexpr (EXACT) {
                floatx16 sums[TA][TB];
                clear(sums);
#pragma unroll
                for (int step = 0; step < 2; ++step) {
                    read8(A, fa, now, step);
                    read8(B, fb, now + OA::kBytes, step);
                    multiply_exact(sums, fa, fb);
                }
                add_scaled(acc, sums, s);
            } else {
#pragma unroll
                for (int step = 0; step < 2; ++step) {
                    read8(A, fa, now, step);
                    read8(B, fb, now + OA::kBytes, step);
                    multiply8(acc, fa, fb, s);
                }
            }
            s.advance();
            const uint32_t t = now;
            now = other;
            other = t;
        }
    }
}

// The same for still smaller tiles, which are for problems that leave compute units idle: 4
// waves, BUFFERS stages of LDS.  A wave multiplies a stage from
// registers while it reads the next one's fragments into others, so that a stage costs its
// products or one barrier and its issue, whichever is longer, and not the LDS's latency (0.27 us a
// stage; 0.46 when it reads what it then multiplies).  Four buffers, two workgroups a compute unit:
// eight buffers and one are slower, as are 128 x 64 tiles and fewer or more products a wave.
template <int BUFFERS, int TA, int TB, typename OA, typename OB>
__device__ inline void k_loop8_small(floatx16 (&acc)[TA][TB], int stages, OA& A, OB& B, int left, uint32_t lds, int wave, int lane,
                                     Scales<TA, TB>& s) {
    static_assert(BUFFERS % 2 == 0 && kScaleStages % 2 == 0, "stages in pairs");
    constexpr uint32_t kStage = OA::kBytes + OB::kBytes;
    constexpr int kLoads = OA::kLoads + OB::kLoads;
    const int part = left % kHeadK;
    const uint32_t behind = part && 8 * A.chunk >= part ? 16 * A.chunk : 0;      // as in k_loop8
    const uint32_t mine = wave * 1024;
    uint32_t put = lds, get = lds;
    auto after = [&](uint32_t slot) { return slot == lds + (BUFFERS - 1) * kStage ? lds : slot + kStage; };
    auto load_all = [&](auto& op, uint32_t dst, uint32_t less) {
        typedef std::remove_reference_t<decltype(op)> Op;
        op.template load_before<0>(dst, less);
        if constexpr (Op::kLoads > 1) op.template load_before<1>(dst, less);
        if constexpr (Op::kLoads > 2) {
            op.template load_before<2>(dst, less);
            op.template load_before<3>(dst, less);
        }
        op.advance();
    };
    auto load = [&](int kt) {
        const uint32_t less = kt + 1 == stages ? behind : 0;
        load_all(A, put + mine, less);
        load_all(B, put + OA::kBytes + mine, less);
        put = after(put);
    };
    struct Frags {
        v8i a[2][TA], b[2][TB];
    };
    auto read = [&](Frags& f) {
#pragma unroll
        for (int step = 0; step < 2; ++step) {
            read8(A, f.a[step], get, step);
            read8(B, f.b[step], get + OA::kBytes, step);
        }
        get = after(get);
    };
    auto mask = [&](Frags& f) {      // of the last stage
#pragma unroll
        for (int step = 0; step < 2; ++step)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const bool there = !part || 16 * (2 * step + k) + 8 * (lane / 32) < part;
#pragma unroll
                for (int j = 0; j < TB; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) f.b[step][j][4 * k + e] = there ? f.b[step][j][4 * k + e] : 0;
            }
    };
    auto multiply = [&](const Frags& f) {
#pragma unroll
        for (int step = 0; step < 2; ++step)
#pragma unroll
            for (int i = 0; i < TA; ++i)
#pragma unroll
                for (int j = 0; j < TB; ++j) acc[i][j] = mfma8(f.a[step][i], f.b[step][j], acc[i][j], s.b.w[0], s.a[j].w[0]);
        s.advance();
    };
    s.load(0, stages);
    const int first = min(BUFFERS, stages);
    for (int kt = 0; kt < first; ++kt) load(kt);
    wait_stages<kLoads>(first - 1);
    bare_barrier();
    Frags f, g;
    read(f);
    if (stages == 1) mask(f);
    // multiplies one stage, reads the next, loads the one BUFFERS on
    auto stage = [&](Frags& now, Frags& next, int kt) {
        wait_loads<(BUFFERS - 2) * kLoads>();
        wait_lds();
        bare_barrier();      // stage kt + 1 is in LDS, and every wave has read stage kt
        load(kt + BUFFERS);
        read(next);
        multiply(now);
    };
    int kt = 0;
    const int pairs_end = stages - BUFFERS - 1;
    while (kt < pairs_end) {
        const int end = min(pairs_end, (kt / kScaleStages + 1) * kScaleStages);
#pragma unroll 1
        for (; kt < end; kt += 2) {
            stage(f, g, kt);
            stage(g, f, kt + 1);
        }
        if (kt % kScaleStages == 0) s.load(kt, stages);
    }
    for (; kt < stages; ++kt) {
        const bool next = kt + 1 < stages;
        if (next) {
            wait_stages<kLoads>(min(BUFFERS - 2, stages - 2 - kt));
            wait_lds();
            bare_barrier();
            if (kt + BUFFERS < stages) load(kt + BUFFERS);
            read(g);
            if (kt + 2 == stages) mask(g);
        }
        multiply(f);
        if (next && (kt + 1) % kScaleStages == 0) s.load(kt + 1, stages);
        f = g;
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
    const int half = lane / 32, pitch = (int)a.y_stride * 2, mine = lane % kChunks, left = a.cols - v0 - 8 * mine;
    T* first = static_cast<T*>(a.y) + (int64_t)t0 * a.y_stride + v0;
    const Through whole(first);
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
        wave_order();
        auto values = [&](int r) { return *reinterpret_cast<const u32x4*>(stage + (r * kChunks + (mine ^ (r % kChunks))) * 16); };
        const int end = min(32, a.rows - t0 - 32 * tt);
        if (a.y_vec && left >= 8) {
#pragma unroll
            for (int k = 0; k < kChunks / 2; ++k) {
                const int r = k * (kWave / kChunks) + lane / kChunks;
                if (r < end) whole.store((32 * tt + r) * pitch + 16 * mine, values(r));
            }
        } else if (left > 0) {       // rows that are not aligned, or that end in this chunk
#pragma unroll 2
            for (int r = lane / kChunks; r < end; r += kWave / kChunks) {
                const u32x4 w = values(r);
                T* dst = first + (int64_t)(32 * tt + r) * a.y_stride + 8 * mine;
                if (left >= 8) {
                    *reinterpret_cast<u32x4_any*>(dst) = w;
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < left) dst[e] = __builtin_bit_cast(T, (uint16_t)(w[e / 2] >> (16 * (e % 2))));
            }
        }
        wave_order();
    }
}

// The same as float32 values, straight from the registers: sums of a part of K (PARTIAL: rows of whole 8 values), which stay in the
// caches, or y.  Row r of `out` at out + r pitch, `cols` columns.
template <bool PARTIAL, int TV, int TT>
__device__ inline void store_sums(float* out, int64_t pitch, int rows, int cols, floatx16 (&acc)[TV][TT], int v0, int t0, int lane) {
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
        const int row = t0 + 32 * tt + lane % 32;
        if (row >= rows) continue;
#pragma unroll
        for (int tv = 0; tv < TV; ++tv)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int v = v0 + 32 * tv + 16 * p + 8 * (lane / 32);
                if (PARTIAL && v >= cols) continue;
                float* dst = out + row * pitch + v;
                if (PARTIAL || v + 8 <= cols) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        floatx4 x;
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] = acc[tv][tt][8 * p + 4 * h + e];
                        reinterpret_cast<floatx4_any*>(dst)[h] = x;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (v + e < cols) dst[e] = acc[tv][tt][8 * p + e];
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
    s.init(a, v0, t0, 0, lane);
    floatx16 acc[TV][TT];
    clear(acc);
    k_loop8<TV, TT>(acc, (a.dim + kBlock8 - 1) / kBlock8, B, A, (a.dim + 15) / 16 * 8, lds_address(lds), wave, lane, s);
    bare_barrier();      // every wave is done with the operands, whose slots y passes through
    store_tile<T, TV, TT>(a, acc, v0, t0, lane, lds + wave * kStageBytes<TV>);
}

// 32 WV TV columns x 32 WT TT rows by 4 waves, BUFFERS stages, two workgroups per compute
// unit; K in a.splits parts, whose sums matmul8_join adds.
// EXACT: sums in float32 of products that lose nothing, the only form with float32 results.
template <int WV, int WT, int TV, int TT, int BUFFERS> struct SmallTile {
    static constexpr int kCols = 32 * WV * TV, kRows = 32 * WT * TT;
    static constexpr size_t kBytes = (size_t)BUFFERS * (kCols + kRows) * kBlock8;
    static_assert(WV * WT == 4 && kBlock8 % (32 * TV) == 0 && kStageBytes<TV> * 4 <= (int)kBytes, "tile");
};
template <typename T, bool EXACT, int WV, int WT, int TV, int TT, int BUFFERS>
__global__ __launch_bounds__(256, 2) void matmul8_small_kernel(const Matmul8 a) {
    static_assert(EXACT ? BUFFERS == 2 : sizeof(T) == 2, "forms");
    typedef SmallTile<WV, WT, TV, TT, BUFFERS> S;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tiles = a.tiles_v * a.tiles_t, item = xcd_item(tiles * a.splits);
    if (item < 0) return;
    int tile_v, tile_t;
    const int split = item / tiles;
    tile_of(a, item - split * tiles, tile_v, tile_t);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wv = wave / WT, wt = wave % WT;
    const int v0 = tile_v * S::kCols + wv * TV * 32, t0 = tile_t * S::kRows + wt * TT * 32;
    const int all = (a.dim + kBlock8 - 1) / kBlock8, s0 = split * a.stages_per_split, stages = min(all - s0, a.stages_per_split);
    RowOperand<S::kCols, 4> B;
    RowOperand<S::kRows, 4> A;
    B.init(a.b.codes, a.b.stride, (int64_t)tile_v * S::kCols, a.cols, s0 * kHeadK, wv * TV * 32 + swap23(lane % 32), wave, lane);
    A.init(a.a.codes, a.a.stride, (int64_t)tile_t * S::kRows, a.rows, s0 * kHeadK, wt * TT * 32 + lane % 32, wave, lane);
    Scales<TV, TT> s;
    s.init(a, v0, t0, s0, lane);
    floatx16 acc[TV][TT];
    clear(acc);
    const int left = min((a.dim + 15) / 16 * 8 - s0 * kHeadK, stages * kHeadK);
    if constexpr (BUFFERS == 2) k_loop8_mid<EXACT>(acc, stages, B, A, left, lds_address(lds), wave, s);
    else k_loop8_small<BUFFERS>(acc, stages, B, A, left, lds_address(lds), wave, lane, s);
    if (a.partial) {
        store_sums<true>(a.partial + (int64_t)split * a.rows * a.partial_pitch, a.partial_pitch, a.rows, a.cols, acc, v0, t0, lane);
        return;
    }
    if constexpr (sizeof(T) == 4) {
        store_sums<false>(static_cast<float*>(a.y), a.y_stride, a.rows, a.cols, acc, v0, t0, lane);
    } else {
        bare_barrier();
        store_tile<T, TV, TT>(a, acc, v0, t0, lane, lds + wave * kStageBytes<TV>);
    }
}

// The sums of the parts of K in order, rounded once.
template <typename T>
__global__ __launch_bounds__(kJoinThreads) void matmul8_join_kernel(const Matmul8 a) {
    const int64_t octs = (a.cols + 7) / 8, items = octs * a.rows, step = (int64_t)a.rows * a.partial_pitch;
    for (int64_t n = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; n < items; n += (int64_t)gridDim.x * kJoinThreads) {
        const int64_t row = n / octs;
        const int v = (int)(n - row * octs) * 8;
        floatx4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
        const float* src = a.partial + row * a.partial_pitch + v;
        int s = 0;
        for (; s + kJoinBatch <= a.splits; s += kJoinBatch) {
            floatx4 part[kJoinBatch][2];
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k, src += step) {
                part[k][0] = reinterpret_cast<const floatx4*>(src)[0];
                part[k][1] = reinterpret_cast<const floatx4*>(src)[1];
            }
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) {
                lo += part[k][0];
                hi += part[k][1];
            }
        }
        for (; s < a.splits; ++s, src += step) {
            lo += reinterpret_cast<const floatx4*>(src)[0];
            hi += reinterpret_cast<const floatx4*>(src)[1];
        }
        const float sums[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        T* dst = static_cast<T*>(a.y) + row * a.y_stride + v;
        if (v + 8 <= a.cols) {
            if constexpr (sizeof(T) == 4) {
                reinterpret_cast<floatx4_any*>(dst)[0] = lo;
                reinterpret_cast<floatx4_any*>(dst)[1] = hi;
            } else {
                *reinterpret_cast<u32x4_any*>(dst) = pack8<T>(sums);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (v + e < a.cols) dst[e] = (T)sums[e];
        }
    }
}

// Few rows or few tiles: K is split over the waves of a workgroup, which meet in LDS; operands
// straight from memory, the next stage's under way while one is multiplied.
//
// Up to 16 rows: 16 columns of y a workgroup, 16x16x128 products, each row of b used once, four stages of
// a wave under way: 1 x 8192 x 8192 13.0 us, 5.2 TB/s of weights; 16 x 512 x 8192 10.8 (32 workgroups, whose waves
// have 8 stages each).
template <typename T, int NW>
__global__ __launch_bounds__(NW * kWave) void matmul8_rows_kernel(const Matmul8 a) {
    constexpr int kEdge = 16;
    __shared__ float part[NW][kEdge][kEdge + 1];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int v0 = blockIdx.x * kEdge;
    const int v = min(v0 + lane % 16, a.cols - 1), t = min(lane % 16, a.rows - 1);
    const uint8_t* b = a.b.codes + (int64_t)v * a.b.stride + 32 * (lane / 16);
    const uint8_t* x = a.a.codes + (int64_t)t * a.a.stride + 32 * (lane / 16);
    const uint8_t* sb = a.b.scale + (int64_t)(v / kBlock8) * a.b.scale_stride;
    const uint8_t* sa = a.a.scale + (int64_t)t * a.a.scale_stride;
    const int stages = (a.dim + kBlock8 - 1) / kBlock8, end = (a.dim + 15) / 16 * 16 - 32 * (lane / 16);
    floatx4 acc = {0.f, 0.f, 0.f, 0.f};
    struct Stage {
        u32x4 b[2], x[2];
        int sb, sa;
    };
    auto load = [&](Stage& s, int kt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = kt * kBlock8 + 16 * h;
            s.b[h] = s.x[h] = u32x4{0u, 0u, 0u, 0u};
            if (k < end) {
                s.b[h] = *reinterpret_cast<const u32x4*>(b + k);
                s.x[h] = *reinterpret_cast<const u32x4*>(x + k);
            }
        }
        s.sb = sb[kt];
        s.sa = sa[kt];
    };
    auto multiply = [&](const Stage& s) {
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(s.b[0], s.b[1]), join(s.x[0], s.x[1]), acc, 0, 0, 0, s.sb, 0, s.sa);
    };
    constexpr int kAhead = 4;        // stages under way together
    for (int kt = wave; kt < stages; kt += kAhead * NW) {
        Stage s[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (kt + k * NW < stages) load(s[k], kt + k * NW);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (kt + k * NW < stages) multiply(s[k]);
    }
    // register e of lane l: column 4 (l / 16) + e, row l % 16
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][lane % 16][4 * (lane / 16) + e] = acc[e];
    __syncthreads();
    for (int i = threadIdx.x; i < kEdge * kEdge; i += NW * kWave) {
        const int c = i % kEdge, r = i / kEdge;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) sum += part[w][r][c];
        if (v0 + c < a.cols && r < a.rows) static_cast<T*>(a.y)[(int64_t)r * a.y_stride + v0 + c] = (T)sum;
    }
}

// Otherwise 32 columns x 32 rows a workgroup, where that alone fills the chip and K is short: 128 x 1024 x 1024
// 4.5 us (64: 5.5, 128: 7.6).
template <int NW> constexpr size_t kSplitBytes = (size_t)NW * 16 * kWave * 4;
template <typename T, int NW>
__global__ __launch_bounds__(NW * kWave) void matmul8_split_kernel(const Matmul8 a) {
    extern __shared__ __align__(16) uint8_t lds[];
    const int item = xcd_item(a.tiles_v * a.tiles_t);
    if (item < 0) return;
    int tile_v, tile_t;
    tile_of(a, item, tile_v, tile_t);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), half = lane / 32;
    const int v0 = tile_v * 32, t0 = tile_t * 32;
    const int stages = (a.dim + kBlock8 - 1) / kBlock8, end = (a.dim + 15) / 16 * 16 - 16 * half;
    const int64_t v = min(v0 + swap23(lane % 32), a.cols - 1), t = min(t0 + lane % 32, a.rows - 1);
    const uint8_t* const b = a.b.codes + v * a.b.stride + 16 * half;
    const uint8_t* const x = a.a.codes + t * a.a.stride + 16 * half;
    const uint8_t* const sb = a.b.scale + (int64_t)(v0 / kBlock8) * a.b.scale_stride;      // a tile's columns share a block
    const uint8_t* const sa = a.a.scale + t * a.a.scale_stride;
    struct Stage {
        u32x4 b[4], x[4];
        int sb, sa;
    };
    floatx16 acc(0.f);
    auto load = [&](Stage& s, int kt) {
        auto row = [&](u32x4 (&w)[4], const uint8_t* from) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int k = kt * kBlock8 + 32 * c;
                w[c] = u32x4{0u, 0u, 0u, 0u};
                if (k < end) w[c] = *reinterpret_cast<const u32x4*>(from + k);
            }
        };
        row(s.b, b);
        row(s.x, x);
        s.sb = sb[kt];
        s.sa = sa[kt];
    };
    auto multiply = [&](const Stage& s) {
#pragma unroll
        for (int step = 0; step < 2; ++step)
            acc = mfma8(join(s.b[2 * step], s.b[2 * step + 1]), join(s.x[2 * step], s.x[2 * step + 1]), acc, s.sb, s.sa);
    };
    Stage now, next;
    if (wave < stages) load(now, wave);
    for (int kt = wave; kt < stages; kt += 2 * NW) {
        if (kt + NW < stages) load(next, kt + NW);
        multiply(now);
        if (kt + 2 * NW < stages) load(now, kt + 2 * NW);
        if (kt + NW < stages) multiply(next);
    }
    // 8 consecutive columns of a row: unit (p, lane) holds column 16 p + 8 (l / 32) of row l % 32
    constexpr int kUnits = 2 * kWave;
    floatx4* part = reinterpret_cast<floatx4*>(lds);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            floatx4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = acc[8 * p + 4 * h + e];
            part[((wave * 2 + h) * 2 + p) * kWave + lane] = w;
        }
    __syncthreads();
    for (int u = threadIdx.x; u < kUnits; u += NW * kWave) {
        floatx4 lo = part[u], hi = part[kUnits + u];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            lo += part[2 * w * kUnits + u];
            hi += part[(2 * w + 1) * kUnits + u];
        }
        const int l = u % kWave, row = t0 + l % 32, col = v0 + 16 * (u / kWave) + 8 * (l / 32);
        if (row >= a.rows || col >= a.cols) continue;
        T* dst = static_cast<T*>(a.y) + (int64_t)row * a.y_stride + col;
        const float sums[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        if (col + 8 <= a.cols) {
            *reinterpret_cast<u32x4_any*>(dst) = pack8<T>(sums);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col + e < a.cols) dst[e] = (T)sums[e];
        }
    }
}

template <typename K>
hipError_t allow_lds(K kernel, size_t bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int NW>
hipError_t split_launch(const Matmul8& a, hipStream_t s) {
    const hipError_t allowed = allow_lds(&matmul8_split_kernel<T, NW>, kSplitBytes<NW>);
    if (allowed != hipSuccess) return allowed;
    matmul8_split_kernel<T, NW><<<xcd_grid(a.tiles_v * a.tiles_t), NW * kWave, kSplitBytes<NW>, s>>>(a);
    return hipGetLastError();
}

template <typename T, bool EXACT, int WV, int WT, int TV, int TT, int BUFFERS>
hipError_t small_launch(const Matmul8& a, hipStream_t s) {
    constexpr size_t bytes = SmallTile<WV, WT, TV, TT, BUFFERS>::kBytes;
    const hipError_t allowed = allow_lds(&matmul8_small_kernel<T, EXACT, WV, WT, TV, TT, BUFFERS>, bytes);
    if (allowed != hipSuccess) return allowed;
    matmul8_small_kernel<T, EXACT, WV, WT, TV, TT, BUFFERS><<<xcd_grid(a.tiles_v * a.tiles_t * a.splits), 256, bytes, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t typed(const Matmul8& a, int variant, hipStream_t s) {
    const int grid = xcd_grid(a.tiles_v * a.tiles_t);
    if (variant == kMatmulRows) matmul8_rows_kernel<T, 8><<<a.tiles_v, 8 * kWave, 0, s>>>(a);
    else if (variant == kMatmulSplit) return split_launch<T, 8>(a, s);
    else if (variant == kMatmulSmall) return small_launch<T, false, 2, 2, 1, 1, 4>(a, s);
    else if (variant == kMatmulMid) return small_launch<T, false, 2, 2, 2, 2, 2>(a, s);
    else {
        const hipError_t allowed = allow_lds(&matmul8_kernel<T>, kRingBytes);
        if (allowed != hipSuccess) return allowed;
        matmul8_kernel<T><<<grid, 512, kRingBytes, s>>>(a);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t exact_typed(const Matmul8& a, int variant, hipStream_t s) {
    if (variant == kMatmulExactSmall) return small_launch<T, true, 2, 2, 1, 1, 2>(a, s);
    return small_launch<T, true, 2, 2, 2, 2, 2>(a, s);
}

}  // namespace

hipError_t launch_matmul8_join(const Matmul8& a, int type, hipStream_t s) {
    const int64_t items = (int64_t)a.rows * ((a.cols + 7) / 8);
    const int grid = (int)std::min<int64_t>(32768, (items + kJoinThreads - 1) / kJoinThreads);
    if (type == kTypeBf16) matmul8_join_kernel<bf16><<<grid, kJoinThreads, 0, s>>>(a);
    else if (type == kTypeFp16) matmul8_join_kernel<f16><<<grid, kJoinThreads, 0, s>>>(a);
    else matmul8_join_kernel<float><<<grid, kJoinThreads, 0, s>>>(a);
    return hipGetLastError();
}
hipError_t launch_matmul8(const Matmul8& a, int type, int variant, hipStream_t s) {
    if (variant == kMatmulExactSmall || variant == kMatmulExactMid) {
        if (type == kTypeBf16) return exact_typed<bf16>(a, variant, s);
        return type == kTypeFp16 ? exact_typed<f16>(a, variant, s) : exact_typed<float>(a, variant, s);
    }
    return type == kTypeBf16 ? typed<bf16>(a, variant, s) : typed<f16>(a, variant, s);
}

}  // namespace muon
