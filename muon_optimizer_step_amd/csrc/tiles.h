// Tiles of matrix products on gfx950: operand staging through LDS with direct
// loads, the K loops over 32x32 MFMAs, and the map from workgroups to XCDs.  Used by
// the head's loss (head.hip) and the linear layers in 8 bits (matmul8.hip, grad8.hip).
#pragma once

#include <type_traits>

#include "common.h"

namespace muon {

constexpr int kHeadK = 64;         // K elements (of 16 bits) per LDS stage
constexpr int kHeadTile = 256;     // output tile edge of the products

namespace {

typedef _Float16 f16;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef short short4v __attribute__((ext_vector_type(4)));

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
    // the same `less` bytes before
    template <int J> __device__ inline void load_before(uint32_t dst, uint32_t less) const {
        direct_load<J * WAVES * 1024>(next, off[J] - less, dst);
    }
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
    // the same with a row's offset from 24 bits (pitch below 2^24)
    template <int J> __device__ inline void load_clamped(uint32_t dst, int last) const {
        direct_load<J * WAVES * 1024>(next, __umul24(min(row[J], last), pitch) + chunk[J], dst);
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

}  // namespace
}  // namespace muon
