// Kernels of the language-model head's loss on gfx950: softmax cross entropy of
// H W^T without the logits in memory as a whole, and its gradients.
//
// Mathematics, with z_ij = h_i . w_j, l = cap tanh(z / cap) where a cap is set:
//   lse_i = log sum_j exp l_ij;  nll_i = lse_i - l_i,t(i)
//   P_ij = g_i (exp(l_ij - lse_i) - [j = t(i)]) (1 - (l_ij / cap)^2)
//   dH = P W;  dW = P^T H
// head_logits multiplies H W^T tile by tile and reduces each token's logits of
// one sub-tile of the vocabulary to a reference exponent c (base 2) and the sum of
// e_ij = 2^(l_ij log2 e - c); for training it also writes e_ij, times 1 - (l_ij / cap)^2
// but at the target, in fp16 (c is the sub-tile's maximum less 15, so the largest e is 2^15: 11
// significant bits down to 2^-29 of the maximum, which leaves the rounding of P to its
// 16-bit type as the only one that counts).  head_rows joins the sub-tiles of a
// token, head_prob turns e into P in place, and head_grads multiplies P with W
// and P^T with H.  The logits thus cost one product, and only a piece of the
// tokens is in memory at a time.
//
// Bound: the three products (6 x tokens x vocab x dim operations), on MFMA, and
// for training the piece's way through HBM (6 bytes per token and vocabulary entry, the
// products' reads of P not counted, which the caches serve in part).
#include <algorithm>
#include <type_traits>

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

// Waits as builtins, which the compiler's own count of outstanding LDS reads
// takes into account (an opaque wait would be followed by another).
template <int N> __device__ inline void wait_loads() {
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
__device__ inline void wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14)); }
__device__ inline void bare_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// cap tanh(z / cap) and its derivative 1 - tanh(z / cap)^2, each to a few ulp of itself
// whatever the cap.  Up to half a cap from zero the value is z + z y p(y), y = (z / cap)^2,
// with p fitted to (tanh(x) / x - 1) / x^2 (minimax on 0 .. 1/4, off by 1.5e-8 of
// tanh): the cap enters only through y, and far above z the result is z itself.
// Beyond, cap (1 - t) / (1 + t) and 4 t / (1 + t)^2 with t = exp(-2 |z| / cap), where
// nothing cancels.
struct Capped {
    float value, slope;
};
constexpr float kCapNear = 0.5f;
__device__ inline Capped capped_near(float z, float inv_cap) {
    const float x = z * inv_cap, y = x * x;
    const float p = fmaf(fmaf(fmaf(0.017256994f, y, -0.05305295f), y, 0.13325988f), y, -0.3333315f);
    Capped r;
    r.value = fmaf(z * y, p, z);
    const float tanh = r.value * inv_cap;
    r.slope = fmaf(-tanh, tanh, 1.0f);
    return r;
}
__device__ inline Capped capped(float z, float cap, float inv_cap) {
    const float x = fabsf(z) * inv_cap, t = __builtin_amdgcn_exp2f(x * (-2.0f * kLog2e)), u = __builtin_amdgcn_rcpf(1.0f + t);
    const Capped near = capped_near(z, inv_cap);
    Capped r;
    r.value = x < kCapNear ? near.value : copysignf(cap * ((1.0f - t) * u), z);
    r.slope = x < kCapNear ? near.slope : 4.0f * t * u * u;
    return r;
}

// 16 bytes per lane, from base + off, straight into LDS at address dst + PLUS +
// 16 x lane (base and dst the wave's).  As assembly because the compiler makes
// every transposing LDS read wait for all direct loads that it knows of, those
// of later stages too; there is no result register, and the K loop waits for
// its loads itself.
template <int PLUS>
__device__ inline void direct_load(const uint8_t* base, uint32_t off, uint32_t dst) {
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst), "v"(off), "s"(base), "n"(PLUS)
                 : "memory", "scc");
}
// The same from an address of each lane's own.
template <int PLUS>
__device__ inline void direct_load_from(const uint8_t* src, uint32_t dst) {
    asm volatile("s_add_u32 m0, %0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(dst), "v"(src), "n"(PLUS)
                 : "memory", "scc");
}
__device__ __align__(16) const uint8_t kZeros[16] = {};   // what K beyond its end is loaded from
__device__ inline uint32_t lds_address(const uint8_t* p) { return (uint32_t)(uintptr_t)(lds_ptr)p; }

// ---------------------------------------------------------------- operand staging
// A stage is 64 K of both operands of a tile.  An operand knows the address of
// the next stage to load (`next`, a scalar that moves by one addition a stage)
// and the LDS addresses of its fragments within a stage's slot, so that a load
// costs two scalar instructions and a fragment one read.
//
// A row operand (K contiguous): ROWS rows x 128 bytes of K per stage (a whole
// cache line: 64-byte pieces cost the vector L1 twice the fills), the 16-byte
// chunk c of row r in slot c ^ ((r / 2) % 8), which keeps the 16-byte fragment
// reads of 32 rows free of bank conflicts.  Direct loads: one wave instruction
// fills 8 rows.
constexpr int kOperand = kHeadTile * kHeadK * 2;     // bytes of one operand of a stage of a 256 x 256 tile
template <int ROWS, int WAVES>
struct RowOperand {
    static constexpr int kBytes = ROWS * kHeadK * 2;
    static constexpr int kLoads = ROWS / 8 / WAVES;
    static_assert(ROWS % (8 * WAVES) == 0 && WAVES % 2 == 0, "whole instructions per wave");
    const uint8_t* next;
    uint32_t off[kLoads];
    int chunk;               // source chunk of this lane within a stage
    uint32_t at[kHeadK / 16];   // LDS address of the first fragment's chunk of each 16 K, less the slot's

    // rows row0 .. row0 + ROWS - 1 of a matrix with `rows` rows (rows beyond its
    // end repeat the last one), from K element k0; `row` is this lane's row of the
    // wave's first fragment
    __device__ inline void init(const void* m, int64_t pitch_bytes, int64_t row0, int64_t rows, int64_t k0, int row, int wave, int lane) {
        next = static_cast<const uint8_t*>(m) + row0 * pitch_bytes + k0 * 2;
        const int last = (int)min<int64_t>(rows - 1 - row0, ROWS - 1);
        chunk = 0;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int r = 8 * (j * WAVES + wave) + lane / 8;
            chunk = (lane % 8) ^ ((r >> 1) & 7);      // the same for every j
            off[j] = (uint32_t)(min(r, last) * pitch_bytes) + chunk * 16;
        }
#pragma unroll
        for (int kc = 0; kc < kHeadK / 16; ++kc) at[kc] = row * 128 + (((2 * kc + lane / 32) ^ ((row >> 1) & 7)) << 4);
    }
    // load J of the next stage to the slot at `dst` (with the wave's 1024 bytes in it)
    template <int J> __device__ inline void load(uint32_t dst) const { direct_load<J * WAVES * 1024>(next, off[J], dst); }
    // the same where K ends `left` elements (a multiple of 8) on: zeros behind it
    template <int J> __device__ inline void load_tail(uint32_t dst, int left) const {
        direct_load_from<J * WAVES * 1024>(8 * chunk < left ? next + off[J] : kZeros, dst);
    }
    __device__ inline void advance() { next += kHeadK * 2; }
    // fragment I (32 rows each): lane l holds K 16 kc + 8 (l / 32) .. + 7 of its row
    template <int I> __device__ inline u32x4 frag(uint32_t slot, int kc) const {
        typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
        return *(lds_u32x4*)(uintptr_t)(at[kc] + slot + I * 32 * 128);
    }
};

// Row of a 32-row A fragment that MFMA row r stands for: bits 2 and 3 swapped.
// The 32x32 accumulator gives a lane rows 8 q + 4 (l / 32) + e; with the swap the
// values 8 p .. 8 p + 7 of its registers are 8 consecutive rows 16 p + 8 (l / 32) + ..,
// one 16-byte store in a 16-bit type.
__device__ inline int swap23(int r) { return (r & 0x13) | ((r & 4) << 1) | ((r & 8) >> 1); }

// A column operand (K strided): 64 rows of K x COLS columns per stage, read
// with the transposing LDS read.  The 16-byte chunk c of row k is in slot c ^ 2
// f(k % 4), f = 0, 2, 5, 7: the 4 rows x 32 bytes that 16 lanes read, and the 4
// rows x 64 bytes of 32 lanes, lie in different banks.
template <int COLS, int WAVES, int FRAGS>
struct ColOperand {
    static constexpr int kRow = COLS * 2, kChunks = COLS / 8, kPer = 1024 / kRow;   // bytes and chunks of a row, rows per instruction
    static constexpr int kBytes = kHeadK * kRow;
    static constexpr int kLoads = kHeadK / kPer / WAVES;
    static_assert(kChunks >= 16, "the slot of a chunk is in its row");
    const uint8_t* next;
    int64_t step;            // bytes of 64 rows
    int pitch;
    uint32_t off[kLoads];
    int chunk[kLoads], row[kLoads];
    uint32_t at[FRAGS];      // LDS address of each fragment's first row, less the slot's
    static __device__ inline int slot_xor(int k) { return 2 * ((0x7520 >> (4 * (k & 3))) & 7); }
    // columns col0 .. of a matrix with cols_pad columns (a multiple of 8; chunks
    // beyond repeat the last), from K row k0; `frag0` is the wave's first fragment's
    // column within the tile; `swap`: fragments hold columns swap23(l % 32)
    __device__ inline void init(const void* m, int64_t pitch_bytes, int col0, int cols_pad, int64_t k0, int frag0, bool swap, int wave,
                                int lane) {
        next = static_cast<const uint8_t*>(m) + (int64_t)col0 * 2 + k0 * pitch_bytes;
        step = kHeadK * pitch_bytes;
        pitch = (int)pitch_bytes;
        const int last = (cols_pad - col0) / 8 - 1;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            row[j] = kPer * (j * WAVES + wave) + lane / kChunks;
            chunk[j] = min((lane % kChunks) ^ slot_xor(row[j]), last) * 16;
            off[j] = (uint32_t)(row[j] * pitch_bytes) + chunk[j];
        }
        // The transposing read gives lane l' of 16 element l' % 4 of the 8 bytes that lane 4 e + l' / 4 points at.
        const int k = 8 * (lane / 32) + (lane % 16) / 4;
        int quad = lane % 4;
        if (swap) quad = ((quad & 1) << 1) | (quad >> 1);
        quad += 4 * ((lane / 16) % 2);
#pragma unroll
        for (int i = 0; i < FRAGS; ++i)
            at[i] = k * kRow + ((((frag0 + 32 * i) / 8 + quad / 2) ^ slot_xor(k)) * 16) + (quad & 1) * 8;
    }
    template <int J> __device__ inline void load(uint32_t dst) const { direct_load<J * WAVES * 1024>(next, off[J], dst); }
    // where only `left` rows of K remain: rows beyond repeat the last
    template <int J> __device__ inline void load_tail(uint32_t dst, int left) const {
        direct_load<J * WAVES * 1024>(next, (uint32_t)(min(row[J], left - 1) * (int64_t)pitch) + chunk[J], dst);
    }
    __device__ inline void advance() { next += step; }
    // fragment I (32 columns): lane l holds K 16 kc + 8 (l / 32) .. + 7 of its column
    template <int I> __device__ inline u32x4 frag(uint32_t slot, int kc) const {
        typedef __attribute__((address_space(3))) short4v lds_short4;
        const uint32_t p = at[I] + slot + kc * 16 * kRow;
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(uintptr_t)p));
        const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(uintptr_t)(p + 4 * kRow)));
        u32x4 r;
        r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
        return r;
    }
};

// All fragments of one step of 16 K, and their products.
template <typename OA, typename OB, int TA, int TB>
__device__ inline void read_step(const OA& A, const OB& B, u32x4 (&fa)[TA], u32x4 (&fb)[TB], uint32_t slot_a, uint32_t slot_b, int kc) {
    fa[0] = A.template frag<0>(slot_a, kc);
    if constexpr (TA > 1) fa[1] = A.template frag<1>(slot_a, kc);
    if constexpr (TA > 2) { fa[2] = A.template frag<2>(slot_a, kc); fa[3] = A.template frag<3>(slot_a, kc); }
    fb[0] = B.template frag<0>(slot_b, kc);
    if constexpr (TB > 1) fb[1] = B.template frag<1>(slot_b, kc);
    static_assert((TA == 1 || TA == 2 || TA == 4) && (TB == 1 || TB == 2), "fragments of a wave");
}

// A whole stage's loads of one operand; `left` K from the stage's beginning.
template <typename Op>
__device__ inline void load_stage(Op& op, uint32_t dst, int left) {
    static_assert(Op::kLoads == 1 || Op::kLoads == 2 || Op::kLoads == 4, "loads of a wave");
    if (left >= kHeadK) {
        op.template load<0>(dst);
        if constexpr (Op::kLoads > 1) op.template load<1>(dst);
        if constexpr (Op::kLoads > 2) { op.template load<2>(dst); op.template load<3>(dst); }
    } else {
        op.template load_tail<0>(dst, left);
        if constexpr (Op::kLoads > 1) op.template load_tail<1>(dst, left);
        if constexpr (Op::kLoads > 2) { op.template load_tail<2>(dst, left); op.template load_tail<3>(dst, left); }
    }
    op.advance();
}

// ---------------------------------------------------------------- K loop
// acc += A B over `stages` stages of 64 K; the operands' K ends after left_a and
// left_b elements, within the last stage.  Tile 256 x 256, 8 waves.
//
// LDS is a ring of five operand slots (all 160 KB): A of stage k is in slot
// 2 k mod 5, B in 2 k + 1 mod 5.  The barrier at the end of stage k - 1 sits before
// the MFMAs of its last 16 K, whose fragments are in registers by then.  It
// frees that stage's two slots, which the loads of B of stage k + 1 and A of
// stage k + 2 fill, one load after every four MFMAs so that their issue does
// not hold the MFMAs up; and it publishes stage k, whose first fragments
// are read while the last MFMAs run.  At its end only B of stage k + 1, issued
// in the first half of the window, has to have arrived; A of k + 2 may be under way.
//
// Measured on 16384 x 8192 x 512 (the gradient of hidden): two buffers filled
// in a burst after the barrier 165 us, this 127.  Counters of the three products of
// 8192 x 131072 x 2048: no LDS bank conflicts, MFMA busy in 66 % of the cycles of
// head_logits and 77 % of head_grads, cycles of a clock of about 1.6 GHz by the
// same counters.
constexpr int kSlots = 5;
constexpr size_t kRingBytes = (size_t)kSlots * kOperand;
template <typename T, int TA, int TB, typename OA, typename OB>
__device__ inline void k_loop(floatx16 (&acc)[TA][TB], int stages, OA& A, OB& B, int left_a, int left_b, uint32_t lds, int wave) {
    static_assert(kHeadK == 64 && OA::kLoads == 4 && OB::kLoads == 4, "four steps of 16 K and eight loads per stage");
    if (stages <= 0) return;
    u32x4 fa[2][TA], fb[2][TB];
    // the slots of A and B of stage kt, A and B of kt + 1, and A of kt + 2; B of kt + 2 takes the first
    uint32_t s0 = lds, s1 = lds + kOperand, s2 = lds + 2 * kOperand, s3 = lds + 3 * kOperand, s4 = lds + 4 * kOperand;
    const uint32_t mine = wave * 1024;
    // the MFMAs of one step, with a load after the second and the sixth eighth
    auto multiply = [&](int set, auto first, auto second) {
#pragma unroll
        for (int n = 0; n < TA * TB; ++n) {
            acc[n / TB][n % TB] = mfma<T>(fa[set][n / TB], fb[set][n % TB], acc[n / TB][n % TB]);
            if (n == TA * TB / 4 || n == TA * TB * 3 / 4) {
                __builtin_amdgcn_sched_barrier(0);
                if (n == TA * TB / 4) first(); else second();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    load_stage(A, s0 + mine, left_a);
    load_stage(B, s1 + mine, left_b);
    if (stages > 1) {
        load_stage(A, s2 + mine, left_a - kHeadK);
        wait_loads<4>();
    } else {
        wait_loads<0>();
    }
    bare_barrier();
    read_step(A, B, fa[0], fb[0], s0, s1, 0);
    const int whole = min(stages, min(left_a, left_b) / kHeadK);     // stages that are complete in both
    // one stage; `fast`: the stages that it loads, kt + 1 and kt + 2, are complete
    auto stage = [&](int kt, auto fast) {
        constexpr bool kFast = decltype(fast)::value;
        const int la = left_a - (kt + 2) * kHeadK, lb = left_b - (kt + 1) * kHeadK;
        auto one = [&](auto& op, auto j, uint32_t dst, int ahead, int left) {
            constexpr int J = decltype(j)::value;
            if (kFast || (kt + ahead < stages && left >= kHeadK)) op.template load<J>(dst + mine);
            else if (kt + ahead < stages) op.template load_tail<J>(dst + mine, left);
        };
        using std::integral_constant;
        read_step(A, B, fa[1], fb[1], s0, s1, 1);
        multiply(0, [&] { one(B, integral_constant<int, 2>(), s3, 1, lb); }, [&] { one(B, integral_constant<int, 3>(), s3, 1, lb); });
        B.advance();
        read_step(A, B, fa[0], fb[0], s0, s1, 2);
        multiply(1, [&] { one(A, integral_constant<int, 0>(), s4, 2, la); }, [&] { one(A, integral_constant<int, 1>(), s4, 2, la); });
        read_step(A, B, fa[1], fb[1], s0, s1, 3);
        multiply(0, [&] { one(A, integral_constant<int, 2>(), s4, 2, la); }, [&] { one(A, integral_constant<int, 3>(), s4, 2, la); });
        A.advance();
        wait_lds();              // this wave's last fragments of stage kt
        if (kFast || kt + 1 < stages) {
            if (kFast || kt + 2 < stages) wait_loads<4>();
            else wait_loads<0>();
            bare_barrier();
            read_step(A, B, fa[0], fb[0], s2, s3, 0);
        }
        const int lb2 = lb - kHeadK;
        multiply(1, [&] { one(B, integral_constant<int, 0>(), s0, 2, lb2); }, [&] { one(B, integral_constant<int, 1>(), s0, 2, lb2); });
        const uint32_t t0 = s0, t1 = s1;
        s0 = s2; s1 = s3; s2 = s4; s3 = t0; s4 = t1;
    };
    if (stages > 1) {            // the first half of B of stage 1; its slot is free from the start
        if (left_b >= 2 * kHeadK) {
            B.template load<0>(s3 + mine);
            B.template load<1>(s3 + mine);
        } else {
            B.template load_tail<0>(s3 + mine, left_b - kHeadK);
            B.template load_tail<1>(s3 + mine, left_b - kHeadK);
        }
    }
    int kt = 0;
    for (; kt + 2 < whole; ++kt) stage(kt, std::true_type());
    for (; kt < stages; ++kt) stage(kt, std::false_type());
}

// The same for the smaller tiles: 4 waves, BUFFERS stages of LDS, two
// workgroups on a compute unit that fill each other's waits.
template <typename T, int BUFFERS, int TA, int TB, typename OA, typename OB>
__device__ inline void k_loop_mid(floatx16 (&acc)[TA][TB], int stages, OA& A, OB& B, int left_a, int left_b, uint32_t lds, int wave) {
    constexpr uint32_t kStage = OA::kBytes + OB::kBytes;
    constexpr int kLoads = OA::kLoads + OB::kLoads;
    const uint32_t mine = wave * 1024;
    uint32_t put = lds, get = lds;
    auto load = [&](int kt) {
        load_stage(A, put + mine, left_a - kt * kHeadK);
        load_stage(B, put + OA::kBytes + mine, left_b - kt * kHeadK);
        put = put == lds + (BUFFERS - 1) * kStage ? lds : put + kStage;
    };
    for (int kt = 0; kt < BUFFERS - 1 && kt < stages; ++kt) load(kt);
    for (int kt = 0; kt < stages; ++kt) {
        if (kt + BUFFERS - 2 < stages) wait_loads<(BUFFERS - 2) * kLoads>();    // stage kt of those under way
        else wait_loads<0>();
        wait_lds();
        bare_barrier();      // stage kt is in LDS, and every wave is done with stage kt - 1
        if (kt + BUFFERS - 1 < stages) load(kt + BUFFERS - 1);
#pragma unroll
        for (int kc = 0; kc < kHeadK / 16; ++kc) {
            u32x4 fa[TA], fb[TB];
            read_step(A, B, fa, fb, get, get + OA::kBytes, kc);
#pragma unroll
            for (int i = 0; i < TA; ++i)
#pragma unroll
                for (int j = 0; j < TB; ++j) acc[i][j] = mfma<T>(fa[i], fb[j], acc[i][j]);
        }
        get = get == lds + (BUFFERS - 1) * kStage ? lds : get + kStage;
    }
}

template <int TA, int TB>
__device__ inline void clear(floatx16 (&acc)[TA][TB]) {
#pragma unroll
    for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = floatx16(0.f);
}

// Work item of this workgroup: workgroups go round-robin over the XCDs, and
// each XCD takes a contiguous range of items, whose operands its L2 shares.
__device__ inline int xcd_item(int items) {
    const int per = (items + kXcds - 1) / kXcds;
    const int at = blockIdx.x / kXcds;
    const int i = (blockIdx.x % kXcds) * per + at;
    return at < per && i < items ? i : -1;
}
inline int xcd_grid(int items) { return (items + kXcds - 1) / kXcds * kXcds; }

// What a token's weight is multiplied by in P, and what the sums over P are
// multiplied by.  The mean's weight 1 / count comes in only after the sums, in
// fp32: in P its own rounding to 16 bits would be one error common to all
// tokens.  fp16 probabilities are scaled by a power of two (the largest weight
// becomes 2^13 .. 2^14, so a probability of 1e-9 is still a normal number; bf16
// has fp32's range).
template <int THREADS>
__device__ inline void head_scalars(const HeadScalars& a, void* lds) {
    constexpr int kWaves = THREADS / kWave;
    int* count = static_cast<int*>(lds);
    float* top = static_cast<float*>(lds) + kWaves;
    int n = 0;
    float m = 0.f;
    for (int i = threadIdx.x; i < a.tokens; i += THREADS) {
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
    for (int w = 1; w < kWaves; ++w) {
        n += count[w];
        m = fmaxf(m, top[w]);
    }
    if (!a.weights) m = 1.f;
    float scale = 1.f;
    if (a.type == kHeadFp16 && m > 1e-30f && m < 1e30f) scale = ldexpf(1.0f, 14 - __builtin_amdgcn_frexp_expf(m));
    a.scalars[0] = scale;
    a.scalars[1] = (a.weights ? 1.0f : 1.0f / (float)max(n, 1)) / scale;
}

// ---------------------------------------------------------------- logits
// What one wave does with its logits: acc[tv][tt] holds 32 vocabulary entries
// (v0 + 32 tv + 16 p + 8 (l / 32) + i in register 8 p + i) of token t0 + 32 tt + l % 32.
// e goes to memory through LDS (`stage`, this wave's own), so that a store
// instruction writes whole rows of 32 TV entries instead of 32 bytes to each of
// 32 tokens.
enum { kNoStore = 0, kStore, kStorePast };    // e not kept; kept; kept, written past the caches
template <int TV> constexpr int kEpilogueBytes = 32 * TV * 64;     // 32 tokens x 32 TV entries of 2 bytes
template <int TV, int TT, int STORE, bool CAP>
__device__ inline void logits_epilogue(const HeadLogits& a, floatx16 (&acc)[TV][TT], int v0, int t0, int sub, int lane,
                                       uint8_t* stage) {
    constexpr int kChunks = 4 * TV;       // 16-byte chunks of a token's row; chunk c of row r in slot c ^ (r % kChunks)
    const int half = lane / 32;
    const bool whole = v0 + 32 * TV <= a.vocab;
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
        const int token = t0 + 32 * tt + lane % 32;
        int end = a.vocab - v0 - 8 * half;
        asm volatile("" : "+v"(end));     // compared with anew for each pass: the masks of all registers do not fit in scalars
        auto beyond = [&](int tv, int r) { return !whole && 32 * tv + 16 * (r / 8) + r % 8 >= end; };
        float top = -INFINITY, most = 0.f;
#pragma unroll
        for (int tv = 0; tv < TV; ++tv)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float z = beyond(tv, r) ? -INFINITY : acc[tv][tt][r];
                top = fmaxf(top, z);
                if (CAP) most = fmaxf(most, fabsf(acc[tv][tt][r]));
                else acc[tv][tt][r] = z;
            }
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        // entries beyond the vocabulary only: nothing to add, and no reference (under a cap -infinity is a logit of -cap)
        const bool none = CAP ? v0 >= a.vocab : top == -INFINITY;
        if (CAP) top = capped(top, a.cap, a.inv_cap).value;
        const float ref = none ? -INFINITY : top * kLog2e - 15.0f;
        const float minus = none ? 0.f : -ref;
        float sum = 0.f;
        int target = -1;        // among this lane's entries
        if constexpr (CAP && STORE != kNoStore) {
            const int64_t t = a.targets[min(token, a.tokens - 1)];
            if (t >= v0 + 8 * half && t < a.vocab) target = (int)t - v0 - 8 * half;
        }
        auto exponentials = [&](auto far) {
            if (CAP) asm volatile("" : "+v"(end));
#pragma unroll
            for (int tv = 0; tv < TV; ++tv)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    float e[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        Capped l = {acc[tv][tt][8 * p + i], 1.f};
                        if (CAP) l = decltype(far)::value ? capped(l.value, a.cap, a.inv_cap) : capped_near(l.value, a.inv_cap);
                        e[i] = __builtin_amdgcn_exp2f(fmaf(l.value, kLog2e, minus));
                        if (CAP && beyond(tv, 8 * p + i)) e[i] = l.slope = 0.f;
                        sum += e[i];
                        if (CAP && STORE != kNoStore) e[i] *= 32 * tv + 16 * p + i == target ? 1.f : l.slope;
                    }
                    if constexpr (STORE != kNoStore) {
                        const int c = 4 * tv + 2 * p + half, r = lane % 32;
                        *reinterpret_cast<u32x4*>(stage + (r * kChunks + (c ^ (r % kChunks))) * 16) = pack8<f16>(e);
                    }
                }
        };
        // few logits are far from zero in units of the cap: the exponential form only where the wave has one
        if (CAP && __any(!(most * a.inv_cap < kCapNear))) exponentials(std::true_type());
        else exponentials(std::false_type());
        if constexpr (STORE != kNoStore) {
            // the same wave's data: LDS keeps its order
#pragma unroll
            for (int k = 0; k < kChunks / 2; ++k) {
                const int r = k * (kWave / kChunks) + lane / kChunks, c = lane % kChunks;
                const u32x4 w = *reinterpret_cast<const u32x4*>(stage + (r * kChunks + (c ^ (r % kChunks))) * 16);
                const int64_t row = t0 + 32 * tt + r;
                const int v = v0 + 8 * c;
                u32x4* dst = reinterpret_cast<u32x4*>(static_cast<f16*>(a.e) + row * a.e_pitch + v);
                if (row < a.e_rows && v < a.e_pitch) {
                    if constexpr (STORE == kStorePast) __builtin_nontemporal_store(w, dst);
                    else *dst = w;
                }
            }
        }
        sum += __shfl_xor(sum, 32, kWave);
        if (half == 0 && token < a.stats.rows) {
            a.stats.ref[a.stats.at(sub, token)] = ref;
            a.stats.sum[a.stats.at(sub, token)] = sum;
        }
    }
}

// Token tiles in groups of 8, vocabulary tiles within: the tiles that an XCD
// works on at a time form a block, which shares operands in its L2.
__device__ inline void tile_of(const HeadLogits& a, int item, int& tile_v, int& tile_t) {
    const int group = item / (8 * a.tiles_v), in_group = item - group * 8 * a.tiles_v;
    const int width = min(8, a.tiles_t - 8 * group);
    tile_v = in_group / width;
    tile_t = 8 * group + in_group % width;
}

// Tile of 256 vocabulary entries x 256 tokens: 8 waves of 128 x 64, 32x32x16
// MFMAs, so that an operand byte from LDS serves the most products that 128
// accumulator registers hold.  Bound by MFMA where dim is long (16384 x 32768 x
// 1024: 882 us, 1.25 PFLOP/s; 8192 x 131072 x 2048: 3.38 ms, 1.30, with e stored
// 3.76, 1.17), by the tile's ends where it is short (16384 x 8192 x 512: 149 us,
// 0.92; with e's 268 MB stored 187).  A cap's polynomial at the tile's end, in bf16:
// 1021 x 50021 x 1000 119 -> 135 us, 155 where the logits reach several caps.
template <typename T, int STORE, bool CAP>
__global__ __launch_bounds__(512, 2) void head_logits_kernel(const HeadLogits a) {
    constexpr int WV = 2, WT = 4, TV = 4, TT = 2, BV = WV * TV * 32, BT = WT * TT * 32, NW = WV * WT;
    static_assert(TV * 32 == logits_sub(kLogitsTile), "one partial per wave");
    extern __shared__ __align__(16) uint8_t lds[];
    if (blockIdx.x == gridDim.x - 1) {
        if (a.scalars.scalars) head_scalars<512>(a.scalars, lds);
        return;
    }
    const int item = xcd_item(a.tiles_v * a.tiles_t);
    if (item < 0) return;
    int tile_v, tile_t;
    tile_of(a, item, tile_v, tile_t);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wv = wave / WT, wt = wave % WT;

    RowOperand<kHeadTile, NW> W, H;
    W.init(a.w, a.w_pitch * 2, (int64_t)tile_v * BV, a.vocab, 0, wv * TV * 32 + swap23(lane % 32), wave, lane);
    H.init(a.h, a.h_pitch * 2, (int64_t)tile_t * BT, a.tokens, 0, wt * TT * 32 + lane % 32, wave, lane);
    floatx16 acc[TV][TT];
    clear(acc);
    k_loop<T, TV, TT>(acc, (a.dim + kHeadK - 1) / kHeadK, W, H, a.dim, a.dim, lds_address(lds), wave);
    if (STORE != kNoStore) bare_barrier();      // every wave is done with the operands, whose slots e passes through
    logits_epilogue<TV, TT, STORE, CAP>(a, acc, tile_v * BV + wv * TV * 32, tile_t * BT + wt * TT * 32, tile_v * WV + wv, lane,
                                        lds + wave * kEpilogueBytes<TV>);
}

// Tile of 128 vocabulary entries x 32, 64 or 128 tokens, two workgroups of 4
// waves per compute unit: for few tokens, where W streams past them (two or
// three stages of 64 K in LDS keep its loads in flight), and for problems with too
// few 256 x 256 tiles.  Bound for few tokens by HBM (64 x 131072 x 2048: 108
// to 113 us, 4.8 TB/s), otherwise by the vector work and the waits of its shorter
// tiles (2048 x 4096 x 512: 13 us, 0.67 PFLOP/s; with e stored 17).
template <int TOKENS> struct MidTile;
template <> struct MidTile<32> { static constexpr int WV = 4, WT = 1, TV = 1, TT = 1, kBuffers = 3; };
template <> struct MidTile<64> { static constexpr int WV = 4, WT = 1, TV = 1, TT = 2, kBuffers = 3; };
template <> struct MidTile<128> { static constexpr int WV = 2, WT = 2, TV = 2, TT = 2, kBuffers = 2; };
template <int TOKENS> constexpr size_t mid_bytes() {
    return (size_t)MidTile<TOKENS>::kBuffers * (kHeadMidVocab + TOKENS) * kHeadK * 2;
}

template <typename T, int TOKENS, int STORE, bool CAP>
__global__ __launch_bounds__(256, 2) void head_logits_mid_kernel(const HeadLogits a) {
    typedef MidTile<TOKENS> M;
    constexpr int WV = M::WV, WT = M::WT, TV = M::TV, TT = M::TT, NW = WV * WT;
    static_assert(WV * TV * 32 == kHeadMidVocab && WT * TT * 32 == TOKENS && NW == 4, "tile");
    extern __shared__ __align__(16) uint8_t lds[];
    if (blockIdx.x == gridDim.x - 1) {
        if (a.scalars.scalars) head_scalars<256>(a.scalars, lds);
        return;
    }
    const int item = xcd_item(a.tiles_v * a.tiles_t);
    if (item < 0) return;
    int tile_v, tile_t;
    tile_of(a, item, tile_v, tile_t);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wv = wave / WT, wt = wave % WT;
    RowOperand<kHeadMidVocab, NW> W;
    RowOperand<TOKENS, NW> H;
    W.init(a.w, a.w_pitch * 2, (int64_t)tile_v * kHeadMidVocab, a.vocab, 0, wv * TV * 32 + swap23(lane % 32), wave, lane);
    H.init(a.h, a.h_pitch * 2, (int64_t)tile_t * TOKENS, a.tokens, 0, wt * TT * 32 + lane % 32, wave, lane);
    floatx16 acc[TV][TT];
    clear(acc);
    k_loop_mid<T, M::kBuffers>(acc, (a.dim + kHeadK - 1) / kHeadK, W, H, a.dim, a.dim, lds_address(lds), wave);
    if (STORE != kNoStore) bare_barrier();
    logits_epilogue<TV, TT, STORE, CAP>(a, acc, tile_v * kHeadMidVocab + wv * TV * 32, tile_t * TOKENS + wt * TT * 32,
                                        tile_v * WV + wv, lane, lds + wave * kEpilogueBytes<TV>);
}

// Up to 32 tokens and a small vocabulary, where there is little to read and
// latency counts: a workgroup for every 32 vocabulary rows, operands straight
// from memory (each row of W is used once), the waves take every fourth 128
// bytes of K and meet in LDS.  1 x 8192 x 512: 5.0 us for 8.4 MB, head_rows 2.5;
// a launch alone is over 2.
template <typename T, int STORE, bool CAP>
__global__ __launch_bounds__(256) void head_logits_stream_kernel(const HeadLogits a) {
    __shared__ __align__(16) float part[4][16][kWave];
    __shared__ __align__(16) uint8_t stage[kEpilogueBytes<1>];
    if (blockIdx.x == gridDim.x - 1) {
        if (a.scalars.scalars) head_scalars<256>(a.scalars, part);
        return;
    }
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int v0 = blockIdx.x * 32;
    const T* w = static_cast<const T*>(a.w) + (int64_t)min(v0 + swap23(lane % 32), a.vocab - 1) * a.w_pitch + 8 * (lane / 32);
    const T* h = static_cast<const T*>(a.h) + (int64_t)min(lane % 32, a.tokens - 1) * a.h_pitch + 8 * (lane / 32);
    floatx16 acc = floatx16(0.f);
    const int left = a.dim - 8 * (lane / 32);     // this lane's K begins at 8 (l / 32)
    auto get = [&](const T* p, int k) -> u32x4 {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (k < left) v = *reinterpret_cast<const u32x4*>(p + k);
        return v;
    };
    for (int k0 = wave * 64; k0 < a.dim; k0 += 256) {
        u32x4 fw[4], fh[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            fw[s] = get(w, k0 + 16 * s);
            fh[s] = get(h, k0 + 16 * s);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) acc = mfma<T>(fw[s], fh[s], acc);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) part[wave][r][lane] = acc[r];
    __syncthreads();
    if (wave != 0) return;
    floatx16 one[1][1];
#pragma unroll
    for (int r = 0; r < 16; ++r) one[0][0][r] = (part[0][r][lane] + part[1][r][lane]) + (part[2][r][lane] + part[3][r][lane]);
    logits_epilogue<1, 1, STORE, CAP>(a, one, v0, 0, blockIdx.x, lane, stage);
}

// ---------------------------------------------------------------- rows
// Two partials joined: the larger reference, the sums in units of it.  The same
// bits in either order of the two.
__device__ inline void join_sums(float& top, float& sum, float top2, float sum2) {
    const float m = fmaxf(top, top2);
    const bool first = top >= top2;
    // both -infinity: vocabulary padding only, nothing to add
    const float d = m == -INFINITY ? 0.f : -fabsf(top - top2);
    sum = fmaf(first ? sum2 : sum, __builtin_amdgcn_exp2f(d), first ? sum : sum2);
    top = m;
}

// THREADS threads on R tokens, THREADS / R for each (thread t: token t % R): joins
// the sub-tiles' partials of a token to its base-2 log-sum-exp, and with `first`
// computes the target's logit as a dot product of its own, writes loss and
// log-sum-exp and the copy of hidden.  Under a cap the target's logit is also
// computed where the target is among the vocabulary entries col0 .. end - 1.
// Every thread returns its token's values.
//
// Both sums run over 64 classes (partials, or 8 elements of the dot product,
// modulo 64), the partials' classes in four parts (partials modulo 256) of their
// own.  Parts meet in pairs, then classes in pairs, fours, eights and sixteens, and the four
// sixteens in turn: an order that does not depend on THREADS and R, so that a
// token's loss has the same bits with and without gradients.
struct Row {
    float lse2, weight;      // weight in P; 0 for tokens that do not count, NaN for a target out of range
    float slope;             // the cap's derivative at the target's logit, where that is computed
    int target;              // -1 for none
};
constexpr int kClasses = 64, kParts = 4, kGroup = 16;
template <int THREADS, int R>
struct RowShape {
    static constexpr int S = THREADS / R;                             // threads of a token
    static constexpr int kOwn = S < kClasses ? kClasses / S : 1;      // classes of a thread
    static constexpr int kHeld = kOwn * (kWave / R < S ? kWave / R : S);   // classes of a token within a wave
    static constexpr int kShared = kHeld < kGroup ? kHeld : kGroup;   // of those, how many meet by shuffles
    static constexpr int kSlots = kClasses / kShared;                 // what then meets through LDS
    static constexpr bool kSpread = S == kClasses * kParts;           // each part of a class has a thread
    static_assert(S <= kClasses || kSpread, "threads of a token");
};
template <typename T, int THREADS, int R>
__device__ inline Row head_row(const HeadRows& a, int row, bool first, int col0, int end,
                               float (*red)[RowShape<THREADS, R>::kSlots][R]) {
    typedef RowShape<THREADS, R> Shape;
    constexpr int S = Shape::S, C = Shape::kOwn, kShared = Shape::kShared, kSlots = Shape::kSlots;
    const int r = threadIdx.x % R, s = threadIdx.x / R;
    const bool live = row < a.tokens, held = row < a.rows, works = s < kClasses;   // the dot product's threads
    float tops[C], sums[C], dots[C];
    // a partial, nothing beyond the last one: loads without a branch, so that many are under way
    auto load = [&](int k, float& top, float& sum) {
        const int64_t at = a.stats.at(min(k, a.nsub - 1), row);
        top = a.stats.ref[at];
        sum = a.stats.sum[at];
        if (k >= a.nsub) {
            top = -INFINITY;
            sum = 0.f;
        }
    };
    if constexpr (Shape::kSpread) {
        __shared__ float meet[2][kParts][kClasses];
        static_assert(C == 1 && R == 1, "one token, one class a thread");
        float top = -INFINITY, sum = 0.f;
        if (live)
#pragma unroll 4
            for (int k = s; k < a.nsub; k += kClasses * kParts) {
                float top2, sum2;
                load(k, top2, sum2);
                join_sums(top, sum, top2, sum2);
            }
        meet[0][s / kClasses][s % kClasses] = top;
        meet[1][s / kClasses][s % kClasses] = sum;
        __syncthreads();
        const int c = s % kClasses;
        tops[0] = meet[0][0][c];
        sums[0] = meet[1][0][c];
        join_sums(tops[0], sums[0], meet[0][1][c], meet[1][1][c]);
        float top2 = meet[0][2][c], sum2 = meet[1][2][c];
        join_sums(top2, sum2, meet[0][3][c], meet[1][3][c]);
        join_sums(tops[0], sums[0], top2, sum2);
    } else {
        float top[kParts][C], sum[kParts][C];
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                top[q][c] = -INFINITY;
                sum[q][c] = 0.f;
            }
        if (live)
            for (int k0 = s * C; k0 < a.nsub; k0 += kClasses * kParts) {
                float top2[kParts][C], sum2[kParts][C];
#pragma unroll
                for (int q = 0; q < kParts; ++q)
#pragma unroll
                    for (int c = 0; c < C; ++c) load(k0 + q * kClasses + c, top2[q][c], sum2[q][c]);
#pragma unroll
                for (int q = 0; q < kParts; ++q)
#pragma unroll
                    for (int c = 0; c < C; ++c) join_sums(top[q][c], sum[q][c], top2[q][c], sum2[q][c]);
            }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            join_sums(top[0][c], sum[0][c], top[1][c], sum[1][c]);
            join_sums(top[2][c], sum[2][c], top[3][c], sum[3][c]);
            join_sums(top[0][c], sum[0][c], top[2][c], sum[2][c]);
            tops[c] = top[0][c];
            sums[c] = sum[0][c];
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) dots[c] = 0.f;
    const int64_t t = live ? a.targets[row] : a.ignore_index;
    const bool counted = live && t != a.ignore_index, valid = t >= 0 && t < a.vocab;
    if (counted && valid && works && (first || (a.cap > 0.f && t >= col0 && t < end))) {
        const T* h = static_cast<const T*>(a.h) + (int64_t)row * a.h_pitch;
        const T* w = static_cast<const T*>(a.w) + t * a.w_pitch;
        for (int d0 = 8 * C * s; d0 < a.dim; d0 += 8 * kClasses)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int d = d0 + 8 * c;
                if (d >= a.dim) continue;
                float x[8], y[8];
                unpack8<T>(*reinterpret_cast<const u32x4*>(h + d), x);
                unpack8<T>(*reinterpret_cast<const u32x4*>(w + d), y);
#pragma unroll
                for (int i = 0; i < 8; ++i) dots[c] = fmaf(x[i], y[i], dots[c]);
            }
    }
    if (first && a.copy && held)
        for (int d = 8 * s; d < a.dim; d += 8 * S) {
            u32x4 v = {0u, 0u, 0u, 0u};
            if (counted) v = *reinterpret_cast<const u32x4*>(static_cast<const T*>(a.h) + (int64_t)row * a.h_pitch + d);
            *reinterpret_cast<u32x4*>(static_cast<T*>(a.copy) + (int64_t)row * a.copy_pitch + d) = v;
        }
#pragma unroll
    for (int w = 1; w < C; w <<= 1)
#pragma unroll
        for (int c = 0; c < C; c += 2 * w) {
            join_sums(tops[c], sums[c], tops[c + w], sums[c + w]);
            dots[c] += dots[c + w];
        }
    float top = tops[0], sum = sums[0], dot = dots[0];
#pragma unroll
    for (int w = C; w < kShared; w <<= 1) {
        const int off = w / C * R;
        join_sums(top, sum, __shfl_xor(top, off, kWave), __shfl_xor(sum, off, kWave));
        dot += __shfl_xor(dot, off, kWave);
    }
    if (works && s * C % kShared == 0) {
        const int at = s * C / kShared;
        red[0][at][r] = top;
        red[1][at][r] = sum;
        red[2][at][r] = dot;
    }
    __syncthreads();
    constexpr int kEach = kGroup / kShared;       // slots of a sixteen
    static_assert(kEach == 1 || kEach == 4, "one sixteen per slot, or four slots per sixteen");
#pragma unroll
    for (int g = 0; g < kSlots / kEach; ++g) {
        float gt = red[0][g * kEach][r], gs = red[1][g * kEach][r], gd = red[2][g * kEach][r];
        if constexpr (kEach == 4) {
            join_sums(gt, gs, red[0][4 * g + 1][r], red[1][4 * g + 1][r]);
            gd += red[2][4 * g + 1][r];
            float ht = red[0][4 * g + 2][r], hs = red[1][4 * g + 2][r], hd = red[2][4 * g + 2][r];
            join_sums(ht, hs, red[0][4 * g + 3][r], red[1][4 * g + 3][r]);
            hd += red[2][4 * g + 3][r];
            join_sums(gt, gs, ht, hs);
            gd += hd;
        }
        if (g == 0) {
            top = gt; sum = gs; dot = gd;
        } else {
            join_sums(top, sum, gt, gs);
            dot += gd;
        }
    }
    Row out;
    out.lse2 = top + __builtin_amdgcn_logf(sum);
    out.target = counted && valid ? (int)t : -1;
    const Capped logit = a.cap > 0.f ? capped(dot, a.cap, a.inv_cap) : Capped{dot, 1.f};
    out.slope = logit.slope;
    out.weight = 0.f;
    if (counted) out.weight = valid ? (a.train ? (a.weights ? a.weights[row] : 1.f) * a.scalars[0] : 1.f) : __builtin_nanf("");
    if (first && s == 0) {
        if (live) {
            const float lse = out.lse2 * kLn2;
            float nll = valid ? lse - logit.value : __builtin_nanf("");
            if (nll < 0.f) nll = 0.f;       // the target's logit is rounded apart from the sum it is part of
            a.nll[row] = counted ? nll : 0.f;
            if (a.lse) a.lse[row] = counted ? lse : 0.f;
        }
        if (a.train && held) a.row_weight[row] = out.weight;
    }
    return out;
}

// Bound by latency: 2.5 us for one token's 256 partials, 7 for 64 tokens' 4096 (13
// where a token's partials lie a row apart, 21 with the 64 threads of the classes
// alone), 23 for 16384 tokens' 256.
template <typename T, int THREADS, int R>
__global__ __launch_bounds__(THREADS) void head_rows_kernel(const HeadRows a) {
    __shared__ float red[3][RowShape<THREADS, R>::kSlots][R];
    head_row<T, THREADS, R>(a, blockIdx.x * R + threadIdx.x % R, true, 0, 0, red);
}

// ---------------------------------------------------------------- probabilities
// 8 tokens x `across` columns per workgroup: first the tokens' values (again by
// each workgroup of their columns), then e -> P in place, 8 columns of the 8
// tokens per thread at a time.  HBM-bound: reads and writes 2 bytes an entry
// (8192 x 131072: 887 us, 4.8 TB/s; 16384 x 8192: 100 us, 5.4 TB/s).  An XCD
// takes consecutive workgroups, whose partials share cache lines (5 % at 8192 x
// 131072, 3 % at 16384 x 8192 when it was built).  All 8 tokens' loads at a time where
// e is past the caches (another 4 %), 4 where it is not (8: 1531 x 12345 capped 22 ->
// 26 us then, 20 now).
// Under a cap head_logits has multiplied e by the derivative 1 - (l / cap)^2, taken from
// the product in fp32, but for the target's e: there the softmax and -1 cancel
// before the derivative, taken from the target's logit, multiplies both.
constexpr int kProbRows = 8;
template <typename T, bool CAP, bool PAST>
__global__ __launch_bounds__(256) void head_prob_kernel(const HeadRows a, int blocks, int across) {
    __shared__ float red[3][RowShape<256, kProbRows>::kSlots][kProbRows];
    constexpr int kBatch = PAST ? kProbRows : kProbRows / 2;
    __shared__ Row rows[kProbRows];
    const int item = xcd_item((a.rows + kProbRows - 1) / kProbRows * blocks);
    if (item < 0) return;
    const int row0 = item / blocks * kProbRows, col0 = item % blocks * across;
    const int end = (int)min<int64_t>(col0 + across, a.e_pitch), live = min(kProbRows, a.rows - row0);
    const Row mine = head_row<T, 256, kProbRows>(a, row0 + threadIdx.x % kProbRows, col0 == 0, col0, end, red);
    if (threadIdx.x < kProbRows) rows[threadIdx.x] = mine;
    __syncthreads();
    for (int col = col0 + 8 * threadIdx.x; col < end; col += 8 * 256) {
        uint8_t* at = static_cast<uint8_t*>(a.e) + ((int64_t)row0 * a.e_pitch + col) * 2;
        const float* ref = a.stats.ref + a.stats.at(col / a.sub, row0);
#pragma unroll 1
        for (int k0 = 0; k0 < live; k0 += kBatch) {
            u32x4 w[kBatch];
            float c[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (k0 + k >= live) continue;
                const u32x4* src = reinterpret_cast<const u32x4*>(at + (int64_t)(k0 + k) * a.e_pitch * 2);
                w[k] = PAST ? __builtin_nontemporal_load(src) : *src;
                c[k] = ref[(int64_t)(k0 + k) * a.stats.per_token];
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (k0 + k >= live) continue;
                const Row row = rows[k0 + k];
                u32x4 out = {0u, 0u, 0u, 0u};
                if (row.weight != 0.f) {     // whatever an ignored token's logits are, its gradient is zero
                    const float f = __builtin_amdgcn_exp2f(c[k] - row.lse2) * row.weight;
                    const int target = row.target - col;
                    float e[8], p[8];
                    unpack8<f16>(w[k], e);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        p[i] = fmaf(e[i], f, i == target ? -row.weight : 0.f);
                        if (CAP) p[i] *= i == target ? row.slope : 1.f;
                    }
                    out = pack8<T>(p);
                }
                u32x4* dst = reinterpret_cast<u32x4*>(at + (int64_t)(k0 + k) * a.e_pitch * 2);
                if constexpr (PAST) __builtin_nontemporal_store(out, dst);
                else *dst = out;
            }
        }
    }
}

// sum of weight x nll, in an order that depends on nothing but THREADS.
template <int THREADS>
__device__ inline void head_loss_sum(const HeadLoss& a, float* red) {
    float sum = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < a.tokens; i += THREADS) sum = fmaf(a.row_weight[i], a.nll[i], sum);
    sum = wave_sum(sum);
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = sum;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < THREADS / kWave; ++w) sum += red[w];
    *a.loss = sum * a.scalars[1];
}

// ---------------------------------------------------------------- gradients
// Tile of 256 output columns d x 256 rows, K split over workgroups where the
// tiles alone would leave compute units idle.  A = W or H with K strided; P with K
// contiguous (dH, K the vocabulary) or strided (dW, K the tokens).  Bound by MFMA:
// 8192 x 131072 x 2048, both gradients 6.71 ms, 1.31 PFLOP/s; 16384 x 8192 x 512,
// 233 us, 1.18, where splits and their partial sums cost the difference.
//
// A wave's sums to memory: acc[i][j] holds columns d0 + 32 i + 16 p + 8 (l / 32) + e
// (register 8 p + e) of row c0 + 32 j + l % 32.
template <typename T, int TD, int TC>
__device__ inline void grad_epilogue(const HeadGrad& a, floatx16 (&acc)[TD][TC], int split, int d0, int c0, int lane) {
    const float unscale = a.scalars[1];
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

// Which tile and part of K an item is.
struct GradItem {
    int split, d0, c0, s0, s1;
};
__device__ inline GradItem grad_item(const HeadGrad& a, int item, int edge) {
    GradItem g;
    g.split = item / (a.tiles_c * a.tiles_d);
    const int tile = item - g.split * a.tiles_c * a.tiles_d;
    g.c0 = tile / a.tiles_d * edge;
    g.d0 = tile % a.tiles_d * edge;
    g.s0 = g.split * a.stages_per_split;
    g.s1 = min(a.k / kHeadK, g.s0 + a.stages_per_split);
    return g;
}

// 256 x 256, 8 waves of 128 x 64.
template <typename T, bool KTOKEN>
__device__ inline void head_grad_tile(const HeadGrad& a, int item, uint8_t* lds) {
    constexpr int WD = 2, WC = 4, TD = 4, TC = 2, NW = WD * WC;
    static_assert(WD * TD * 32 == kHeadTile && WC * TC * 32 == kHeadTile, "tile");
    const GradItem g = grad_item(a, item, kHeadTile);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wd = wave / WC, wc = wave % WC;
    ColOperand<kHeadTile, NW, TD> A;
    A.init(a.a, a.a_pitch * 2, g.d0, (a.dim + 7) / 8 * 8, (int64_t)g.s0 * kHeadK, wd * TD * 32, true, wave, lane);
    const int stages = g.s1 - g.s0, left_a = a.a_rows - g.s0 * kHeadK, left_p = a.k - g.s0 * kHeadK;
    floatx16 acc[TD][TC];
    clear(acc);
    if constexpr (KTOKEN) {
        ColOperand<kHeadTile, NW, TC> P;
        P.init(a.p, a.p_pitch * 2, g.c0, a.p_cols, (int64_t)g.s0 * kHeadK, wc * TC * 32, false, wave, lane);
        k_loop<T, TD, TC>(acc, stages, A, P, left_a, left_p, lds_address(lds), wave);
    } else {
        RowOperand<kHeadTile, NW> P;
        P.init(a.p, a.p_pitch * 2, g.c0, a.p_rows, (int64_t)g.s0 * kHeadK, wc * TC * 32 + lane % 32, wave, lane);
        k_loop<T, TD, TC>(acc, stages, A, P, left_a, left_p, lds_address(lds), wave);
    }
    grad_epilogue<T, TD, TC>(a, acc, g.split, g.d0 + wd * TD * 32, g.c0 + wc * TC * 32, lane);
}

// 128 x 128, 4 waves of 64 x 64, two workgroups per compute unit: for problems
// whose few 256 x 256 tiles would need K split many times (each split's sums
// go to memory and back), and output widths that waste much of a larger tile.
constexpr int kMidEdge = 128;
constexpr size_t kMidGradBytes = (size_t)2 * 2 * kMidEdge * kHeadK * 2;
template <typename T, bool KTOKEN>
__device__ inline void head_grad_mid_tile(const HeadGrad& a, int item, uint8_t* lds) {
    constexpr int WD = 2, WC = 2, TD = 2, TC = 2, NW = WD * WC;
    static_assert(WD * TD * 32 == kMidEdge && WC * TC * 32 == kMidEdge, "tile");
    const GradItem g = grad_item(a, item, kMidEdge);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wd = wave / WC, wc = wave % WC;
    ColOperand<kMidEdge, NW, TD> A;
    A.init(a.a, a.a_pitch * 2, g.d0, (a.dim + 7) / 8 * 8, (int64_t)g.s0 * kHeadK, wd * TD * 32, true, wave, lane);
    const int stages = g.s1 - g.s0, left_a = a.a_rows - g.s0 * kHeadK, left_p = a.k - g.s0 * kHeadK;
    floatx16 acc[TD][TC];
    clear(acc);
    if constexpr (KTOKEN) {
        ColOperand<kMidEdge, NW, TC> P;
        P.init(a.p, a.p_pitch * 2, g.c0, a.p_cols, (int64_t)g.s0 * kHeadK, wc * TC * 32, false, wave, lane);
        k_loop_mid<T, 2>(acc, stages, A, P, left_a, left_p, lds_address(lds), wave);
    } else {
        RowOperand<kMidEdge, NW> P;
        P.init(a.p, a.p_pitch * 2, g.c0, a.p_rows, (int64_t)g.s0 * kHeadK, wc * TC * 32 + lane % 32, wave, lane);
        k_loop_mid<T, 2>(acc, stages, A, P, left_a, left_p, lds_address(lds), wave);
    }
    grad_epilogue<T, TD, TC>(a, acc, g.split, g.d0 + wd * TD * 32, g.c0 + wc * TC * 32, lane);
}

// Both gradients of a piece in one launch, so that their tiles fill the
// compute units together.
template <typename T, bool MID>
__global__ __launch_bounds__(MID ? 256 : 512, 2) void head_grads_kernel(const HeadGrads a) {
    extern __shared__ __align__(16) uint8_t lds[];
    // each XCD an equal number of items and its share of both kinds, those with K
    // the vocabulary (the longer ones) first
    const int items_h = a.hidden.tiles_c * a.hidden.tiles_d * a.hidden.splits;
    const int items_w = a.weight.tiles_c * a.weight.tiles_d * a.weight.splits;
    if (blockIdx.x == gridDim.x - 1) {
        if (a.loss.loss) head_loss_sum<MID ? 256 : 512>(a.loss, reinterpret_cast<float*>(lds));
        return;
    }
    const int per = gridDim.x / kXcds, xcd = blockIdx.x % kXcds, at = blockIdx.x / kXcds;
    const int begin = (int)((int64_t)xcd * items_h / kXcds), end = (int)((int64_t)(xcd + 1) * items_h / kXcds);
    if (at < end - begin) {
        if constexpr (MID) head_grad_mid_tile<T, false>(a.hidden, begin + at, lds);
        else head_grad_tile<T, false>(a.hidden, begin + at, lds);
    } else {
        const int i = xcd * per - begin + at - (end - begin);
        if (i >= items_w) return;
        if constexpr (MID) head_grad_mid_tile<T, true>(a.weight, i, lds);
        else head_grad_tile<T, true>(a.weight, i, lds);
    }
}

// The splits' sums in order, rounded once.  HBM-bound where large: 8 us for 42 MB
// (16384 x 8192 x 512); otherwise latency.
template <typename T>
__global__ __launch_bounds__(256) void head_join_kernel(const HeadJoin a) {
    const int64_t octs = (a.dim + 7) / 8, first = octs * a.part[0].cols, items = first + octs * a.part[1].cols;
    const float unscale = a.scalars[1];
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < items; n += (int64_t)gridDim.x * 256) {
        const bool second = n >= first;
        const HeadJoin::Part& p = a.part[second];
        const int64_t i = second ? n - first : n, c = i / octs, d = (i - c * octs) * 8;
        floatx4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
        const float* src = p.partial + c * p.partial_pitch + d;
        for (int s = 0; s < p.splits; ++s, src += (int64_t)p.cols * p.partial_pitch) {
            lo += reinterpret_cast<const floatx4*>(src)[0];
            hi += reinterpret_cast<const floatx4*>(src)[1];
        }
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) { v[e] = lo[e] * unscale; v[4 + e] = hi[e] * unscale; }
        T* dst = static_cast<T*>(p.out) + c * p.out_pitch + d;
        if (p.out_vec) *reinterpret_cast<u32x4*>(dst) = pack8<T>(v);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (d + e < a.dim) dst[e] = (T)v[e];
    }
}

// ---------------------------------------------------------------- small passes
// Copy with rows padded to whole chunks, ignored rows and rows beyond the end
// zero: for inputs whose rows are not 16-byte aligned, which nothing else here reads.
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

__global__ __launch_bounds__(1024) void head_loss_kernel(const HeadLoss a) {
    __shared__ float red[1024 / kWave];
    head_loss_sum<1024>(a, red);
}

template <typename K>
hipError_t allow_lds(K kernel, size_t bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int TOKENS, int STORE, bool CAP>
hipError_t mid_launch(const HeadLogits& a, hipStream_t s) {
    constexpr size_t bytes = mid_bytes<TOKENS>();
    const hipError_t allowed = allow_lds(&head_logits_mid_kernel<T, TOKENS, STORE, CAP>, bytes);
    if (allowed != hipSuccess) return allowed;
    head_logits_mid_kernel<T, TOKENS, STORE, CAP><<<xcd_grid(a.tiles_v * a.tiles_t) + 1, 256, bytes, s>>>(a);
    return hipGetLastError();
}

template <typename T, int STORE, bool CAP>
hipError_t logits_launch(const HeadLogits& a, int variant, hipStream_t s) {
    if (variant == kLogitsStream) {
        const int groups = (int)(a.e_pitch / kHeadStreamSub);   // the padded columns too: they become zeros
        head_logits_stream_kernel<T, STORE, CAP><<<groups + 1, 256, 0, s>>>(a);
        return hipGetLastError();
    }
    if (variant == kLogitsMid32) return mid_launch<T, 32, STORE, CAP>(a, s);
    if (variant == kLogitsMid64) return mid_launch<T, 64, STORE, CAP>(a, s);
    if (variant == kLogitsMid128) return mid_launch<T, 128, STORE, CAP>(a, s);
    const hipError_t allowed = allow_lds(&head_logits_kernel<T, STORE, CAP>, kRingBytes);
    if (allowed != hipSuccess) return allowed;
    head_logits_kernel<T, STORE, CAP><<<xcd_grid(a.tiles_v * a.tiles_t) + 1, 512, kRingBytes, s>>>(a);
    return hipGetLastError();
}

template <typename T, bool CAP>
hipError_t logits_stored(const HeadLogits& a, int variant, hipStream_t s) {
    if (!a.e) return logits_launch<T, kNoStore, CAP>(a, variant, s);
    return a.e_past ? logits_launch<T, kStorePast, CAP>(a, variant, s) : logits_launch<T, kStore, CAP>(a, variant, s);
}

template <typename T>
hipError_t logits_typed(const HeadLogits& a, int variant, hipStream_t s) {
    return a.cap > 0.f ? logits_stored<T, true>(a, variant, s) : logits_stored<T, false>(a, variant, s);
}

template <typename T>
hipError_t rows_typed(const HeadRows& a, hipStream_t s) {
    // many tokens: 16 per workgroup, which makes 64-byte pieces of the partials
    // and, by their number, 16 or 64 threads for each; few: a workgroup each
    if (a.rows <= kHeadRowGroups) head_rows_kernel<T, 256, 1><<<a.rows, 256, 0, s>>>(a);
    else if (a.nsub <= 128) head_rows_kernel<T, 256, 16><<<(a.rows + 15) / 16, 256, 0, s>>>(a);
    else head_rows_kernel<T, 1024, 16><<<(a.rows + 15) / 16, 1024, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t prob_typed(const HeadRows& a, hipStream_t s) {
    // a workgroup takes whole rows where there are rows enough for 8 on each compute unit
    const int row_blocks = (a.rows + kProbRows - 1) / kProbRows;
    const int wanted = std::max(1, 2048 / row_blocks);
    const int across = (int)(((a.e_pitch + wanted - 1) / wanted + 2047) / 2048 * 2048);
    const int blocks = (int)((a.e_pitch + across - 1) / across), grid = xcd_grid(blocks * row_blocks);
    // far more than the last-level cache holds: past it (8192 x 131072, 2.1 GB: 949 -> 887 us; 16384 x 8192, 268 MB:
    // 100 -> 122)
    const bool past = (int64_t)a.rows * a.e_pitch * 2 > (int64_t)1 << 30;
    if (a.cap > 0.f) {
        if (past) head_prob_kernel<T, true, true><<<grid, 256, 0, s>>>(a, blocks, across);
        else head_prob_kernel<T, true, false><<<grid, 256, 0, s>>>(a, blocks, across);
    } else {
        if (past) head_prob_kernel<T, false, true><<<grid, 256, 0, s>>>(a, blocks, across);
        else head_prob_kernel<T, false, false><<<grid, 256, 0, s>>>(a, blocks, across);
    }
    return hipGetLastError();
}

template <typename T, bool MID>
hipError_t grads_launch(const HeadGrads& a, hipStream_t s) {
    constexpr size_t bytes = MID ? kMidGradBytes : kRingBytes;
    const hipError_t allowed = allow_lds(&head_grads_kernel<T, MID>, bytes);
    if (allowed != hipSuccess) return allowed;
    const int grid = xcd_grid(a.hidden.tiles_c * a.hidden.tiles_d * a.hidden.splits +
                              a.weight.tiles_c * a.weight.tiles_d * a.weight.splits);
    head_grads_kernel<T, MID><<<grid + 1, MID ? 256 : 512, bytes, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_head_logits(const HeadLogits& a, int type, int variant, hipStream_t s) {
    return type == kHeadBf16 ? logits_typed<bf16>(a, variant, s) : logits_typed<f16>(a, variant, s);
}
hipError_t launch_head_rows(const HeadRows& a, int type, hipStream_t s) {
    return type == kHeadBf16 ? rows_typed<bf16>(a, s) : rows_typed<f16>(a, s);
}
hipError_t launch_head_prob(const HeadRows& a, int type, hipStream_t s) {
    return type == kHeadBf16 ? prob_typed<bf16>(a, s) : prob_typed<f16>(a, s);
}
hipError_t launch_head_grads(const HeadGrads& a, int type, bool mid, hipStream_t s) {
    if (type == kHeadBf16) return mid ? grads_launch<bf16, true>(a, s) : grads_launch<bf16, false>(a, s);
    return mid ? grads_launch<f16, true>(a, s) : grads_launch<f16, false>(a, s);
}
hipError_t launch_head_join(const HeadJoin& a, int type, hipStream_t s) {
    const int64_t items = ((int64_t)a.part[0].cols + a.part[1].cols) * ((a.dim + 7) / 8);
    const int groups = (int)std::min<int64_t>(4096, (items + 255) / 256);
    if (type == kHeadBf16) head_join_kernel<bf16><<<groups, 256, 0, s>>>(a);
    else head_join_kernel<f16><<<groups, 256, 0, s>>>(a);
    return hipGetLastError();
}
hipError_t launch_head_pack(const HeadPack& a, hipStream_t s) {
    const int64_t groups = std::min<int64_t>(4096, (a.dst_pitch / 8 * a.rows + 255) / 256);
    head_pack_kernel<<<(int)groups, 256, 0, s>>>(a);
    return hipGetLastError();
}
hipError_t launch_head_loss(const HeadLoss& a, hipStream_t s) {
    head_loss_kernel<<<1, 1024, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace muon
