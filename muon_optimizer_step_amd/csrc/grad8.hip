// The gradient of a linear layer's weight on gfx950 from the 8-bit checkpoint of its
// input: out[c][d] = sum over r of grad[r][c] x[r][d], in float32.
//
// Mathematics.  K runs over the rows, and a row's values have a scale for each 128 of them: a
// scale per K element, which the scaled 8-bit MFMAs have no place for.  So x is decoded to
// bfloat16, exactly (a code has 4 significant bits, the scale is a power of two), on its way
// into LDS: 16 codes of one row and one scale are a lane's load, and become 8
// conversions and two 16-byte writes.  The products are 16-bit ones with the gradient as it is.
//
// Bound and measured: for large problems LDS (a stage of a 256 x 256 tile takes 2800 of its cycles, 2048 of the matrix
// unit's) with MFMA close behind: 8192 x 8192 x 4096 (rows, cols, dim) 418 to 429 us, 1.28 to 1.31 PFLOP/s; 70 % of the cycles MFMA busy, no bank
// conflicts.  For small matrices and many rows what a compute unit loads (24 KB a stage at 50 GB/s) and what its
// waves issue (one for each SIMD: 150 instructions a stage, 4 cycles each), and the split of K, whose partial sums
// go through memory: 16384 x 2048 x 512 47 to 48 us, of which start, partial sums and join some 15; the data in the last
// cache 44.  Few rows: a launch and some latencies, 64 x 512 x 512 5.6 us, 1024 x 512 x 512 10.3.
#include <algorithm>

#include "linear8.h"
#include "tiles.h"

namespace muon {
namespace {

// Columns of x for a tile: 64 rows of K x COLS values per stage, decoded and turned: LDS
// holds a row of 128 bytes for each column, K contiguous, so that a fragment is one 16-byte read
// (the transposing reads that the gradient takes have half the rate: 64 bytes a clock). The
// 16-byte chunk c of column d is in slot c ^ f(d), f = d / 2 ^ d / 16 modulo 8: the 8 lanes that are
// served at a time lie in different banks, in fragments (8 columns) and in writes
// (every fourth of 32 columns).
//
// A lane takes 4 columns of 8 rows: a word of codes from each row and one scale's byte, which
// the 16 lanes that share the rows pass on.
template <int COLS, int THREADS>
struct CodeOperand {
    static constexpr int kAcross = COLS / 4, kBytes = COLS * kHeadK * 2;
    static_assert(THREADS / kAcross * 8 == kHeadK && kAcross % 16 == 0, "a stage");
    struct Codes {
        uint32_t w[8], byte;
    };
    uint8_t* code;           // of the next stage to load
    uint8_t* scale;
    int64_t code_step, scale_step;
    int code_stride, scale_stride, code_gap, scale_gap;      // gap: from the end of a row's part in the tile to the next one
    int code_at[8], scale_at;
    uint32_t put[2];         // LDS address of the lane's first and third column's chunk, less the slot's
    uint32_t at[4];          // of its chunk of fragment 0, by step ^ fragment
    // frag0: the wave's first column, step0 its first step (of 16 K) of a stage
    __device__ inline void init(const Blocks8& x, int d0, int dim, int64_t k0, int frag0, int step0, int thread, int lane) {
        const int col = 4 * (thread % kAcross), group = thread / kAcross;
        const int d = min(col, (dim + 15) / 16 * 16 - 4 - d0);
        code_stride = (int)x.stride;
        scale_stride = (int)x.scale_stride;
        code_step = kHeadK * x.stride;
        scale_step = kHeadK * x.scale_stride;
        code = x.codes + k0 * x.stride + d0;
        scale = x.scale + k0 * x.scale_stride + d0 / kBlock8;
        code_gap = code_stride - ((dim + 15) / 16 * 16 - d0);
        scale_gap = scale_stride - ((dim + kBlock8 - 1) / kBlock8 - d0 / kBlock8);
#pragma unroll
        for (int j = 0; j < 8; ++j) code_at[j] = (8 * group + j) * code_stride + d;
        scale_at = (8 * group + lane % 8) * scale_stride + d / kBlock8;
        auto f = [](int c) { return ((c >> 1) ^ (c >> 4)) & 7; };
#pragma unroll
        for (int h = 0; h < 2; ++h) put[h] = (col + 2 * h) * 128 + ((group ^ f(col + 2 * h)) << 4);
        const int r = frag0 + swap23(lane % 32);
#pragma unroll
        for (int j = 0; j < 4; ++j) at[j] = r * 128 + (((2 * (j ^ step0) + lane / 32) ^ f(r)) << 4);
    }
    // The next stage, from which on there are `left` rows (none, or some -64 SETS, behind the last stage).  Buffers that end
    // behind the last row: the loads' own bounds check makes rows beyond zeros, and a lane's offsets are the same in
    // every stage.  (Strides are no smaller than a row: any place in a row beyond is behind the buffer's end.)
    template <int FIRST, int END> __device__ inline void load(Codes& c, int left) const {
        constexpr int kRaw = 0x00027000;
        const int rows = min(kHeadK, left);
        const auto codes = __builtin_amdgcn_make_buffer_rsrc(code, 0, max(rows * code_stride - code_gap, 0), kRaw);
#pragma unroll
        for (int j = FIRST; j < END; ++j) c.w[j] = __builtin_amdgcn_raw_buffer_load_b32(codes, code_at[j], 0, 0);
        if (END == 8) {
            const auto scales = __builtin_amdgcn_make_buffer_rsrc(scale, 0, max(rows * scale_stride - scale_gap, 0), kRaw);
            c.byte = __builtin_amdgcn_raw_buffer_load_b8(scales, scale_at, 0, 0);
        }
    }
    __device__ inline void advance() {
        code += code_step;
        scale += scale_step;
    }
    // rows 2 M and 2 M + 1: word M of each column's eight values
    struct Decoded {
        u32x4 col[4];
    };
    template <int M> __device__ inline void decode(const Codes& c, Decoded& out) const {
        const int bits = (int)(c.byte << 23);       // row_newbcast: lane n of each 16
        const float f0 = as_float((uint32_t)__builtin_amdgcn_mov_dpp(bits, 0x150 + 2 * M, 15, 15, true));
        const float f1 = as_float((uint32_t)__builtin_amdgcn_mov_dpp(bits, 0x151 + 2 * M, 15, 15, true));
        auto half = [&](auto h) {
            constexpr bool H = decltype(h)::value;
            const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c.w[2 * M], f0, H));
            const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c.w[2 * M + 1], f1, H));
            out.col[2 * H][M] = __builtin_amdgcn_perm(b, a, 0x05040100u);
            out.col[2 * H + 1][M] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        };
        half(std::false_type());
        half(std::true_type());
    }
    template <int C> __device__ inline void store(const Decoded& v, uint32_t slot) const {
        typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
        *(lds_u32x4*)(uintptr_t)(slot + put[C / 2] + C % 2 * 128) = v.col[C];
    }
    __device__ inline void decode_all(const Codes& c, uint32_t slot) const {
        Decoded v;
        decode<0>(c, v);
        decode<1>(c, v);
        decode<2>(c, v);
        decode<3>(c, v);
        store<0>(v, slot);
        store<1>(v, slot);
        store<2>(v, slot);
        store<3>(v, slot);
    }
    template <int I> __device__ inline u32x4 frag(uint32_t slot, int step) const {
        typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
        return *(lds_u32x4*)(uintptr_t)(at[step ^ I] + slot + I * 32 * 128);
    }
};

// acc += x^T grad over `stages` stages of 64 rows, `left` rows in all; STEPS steps of 16 rows from
// step0 on are this wave's.  LDS holds two stages of x and SLOTS of the gradient.  While stage k
// is multiplied, x of k + 1 is decoded from registers, the gradient of k + SLOTS - 1 is loaded
// straight to LDS and the codes of x of k + 1 + SETS to registers, a piece after every product or two.
// The barrier sits before the products of a stage's last step, whose fragments are in
// registers by then; the next stage's first ones are read behind it.
// Near the end the gradient's last stage is loaded again and no more of x, which nothing reads, so that the body has no
// branch; rows behind the last are zero in the gradient's fragments of the last stage (and in x).
template <int STEPS, int SLOTS, int SETS, int TD, int TC, typename OX, typename OG>
__device__ inline void k_loop_coded(floatx16 (&acc)[TD][TC], int stages, OX& X, OG& G, int left, int step0, uint32_t lds, int wave, int lane) {
    static_assert(OG::kLoads == 4 && TD * TC == 8 && (STEPS == 2 || STEPS == 4), "pieces of a stage");
    static_assert(SETS == 2 || SETS == 4, "codes in registers");
    constexpr int kLoads = 9 + OG::kLoads;      // of a stage: x and the gradient
    static_assert(kLoads * (SLOTS - 2) < 64, "the counter's range");
    using std::integral_constant;
    constexpr uint32_t kX = OX::kBytes, kG = OG::kBytes;
    const uint32_t mine = wave * 1024, g_first = lds + 2 * kX, g_last = g_first + (SLOTS - 1) * kG;
    uint32_t x0 = lds, x1 = lds + kX, now = g_first, put = g_first;      // slots of this stage, of the gradient's next load
    auto after = [&](uint32_t slot) { return slot == g_last ? g_first : slot + kG; };
    u32x4 fa[2][TD], fb[2][TC];
    typename OX::Codes c[SETS];
    int left_x = left, left_g = left;      // rows from the stage that X and G load next
    auto next_x = [&] {
        X.advance();
        left_x -= kHeadK;
    };
    auto load_x = [&](typename OX::Codes& c) {
        X.template load<0, 8>(c, left_x);
        next_x();
    };
    auto load_g = [&](auto j) { G.template load_clamped<decltype(j)::value>(put + mine, min(kHeadK, left_g) - 1); };
    auto next_g = [&] {
        const bool more = left_g > kHeadK;
        G.next += more ? G.step : 0;
        left_g -= more ? kHeadK : 0;
        put = after(put);
    };
    auto whole_g = [&] {
        load_g(integral_constant<int, 0>());
        load_g(integral_constant<int, 1>());
        load_g(integral_constant<int, 2>());
        load_g(integral_constant<int, 3>());
        next_g();
    };
    // Stage 0, and then, in the order in which the stages before the first would have issued
    // them, the gradient of 1 .. SLOTS - 2 and x of 1 .. SETS: the counts of the loop's
    // waits hold from its first stage on.
    typename OX::Codes first;
    load_x(first);
    whole_g();
    static_assert(SETS >= SLOTS - 2, "x is ahead at least as far");
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
        if (i >= SETS - (SLOTS - 2)) whole_g();
        load_x(c[i]);
    }
    X.decode_all(first, x0);
    wait_loads<9 * SETS + OG::kLoads * (SLOTS - 2)>();       // the gradient of stage 0
    wait_lds();
    bare_barrier();
    auto read = [&](int set, uint32_t x, uint32_t g, int step) { read_step(X, G, fa[set], fb[set], x, g, step); };
    auto mask = [&](u32x4 (&f)[TC], int step) {      // of the last stage
        const int rows = (left - 1) % kHeadK + 1 - 16 * (step0 + step) - 8 * (lane / 32);
#pragma unroll
        for (int j = 0; j < TC; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) f[j][e] &= (2 * e < rows ? 0xFFFFu : 0u) | (2 * e + 1 < rows ? 0xFFFF0000u : 0u);
    };
    // the products of a step, with a piece of other work after each
    auto multiply = [&](int set, auto piece) {
        auto one = [&](auto n) {
            constexpr int N = decltype(n)::value;
            acc[N / TC][N % TC] = mfma<bf16>(fa[set][N / TC], fb[set][N % TC], acc[N / TC][N % TC]);
            __builtin_amdgcn_sched_barrier(0);
            piece(n);
            __builtin_amdgcn_sched_barrier(0);
        };
        one(integral_constant<int, 0>());
        one(integral_constant<int, 1>());
        one(integral_constant<int, 2>());
        one(integral_constant<int, 3>());
        one(integral_constant<int, 4>());
        one(integral_constant<int, 5>());
        one(integral_constant<int, 6>());
        one(integral_constant<int, 7>());
    };
    read(0, x0, now, 0);
    // a stage that another follows; c: x of the next stage, then of the one SETS after that
    auto stage = [&](typename OX::Codes& c) {
        typename OX::Decoded v;
        auto piece_g = [&](auto n) {      // 0 .. 3
            load_g(n);
            if (decltype(n)::value == 3) next_g();
        };
        read(1, x0, now, 1);
        if constexpr (STEPS == 2) {
            multiply(0, [&](auto n) {
                constexpr int N = decltype(n)::value;
                if constexpr (N < 4) X.template decode<N>(c, v);
                if constexpr (N == 4 || N == 5) {        // early: the barrier waits for them
                    X.template store<2 * (N - 4)>(v, x1);
                    X.template store<2 * (N - 4) + 1>(v, x1);
                }
                if constexpr (N >= 4) piece_g(integral_constant<int, N - 4>());
            });
        } else {
            multiply(0, [&](auto n) {
                constexpr int N = decltype(n)::value;
                if constexpr (N % 2 == 0) X.template decode<N / 2>(c, v);
            });
            read(0, x0, now, 2);
            multiply(1, [&](auto n) {
                constexpr int N = decltype(n)::value;
                if constexpr (N % 2 == 0) X.template store<N / 2>(v, x1);
            });
            read(1, x0, now, 3);
            multiply(0, [&](auto n) {
                constexpr int N = decltype(n)::value;
                if constexpr (N % 2 == 0) piece_g(integral_constant<int, N / 2>());
            });
        }
        wait_lds();          // this wave's last fragments of the stage, and its share of the next one's x
        wait_loads<kLoads * (SLOTS - 2)>();      // the gradient of the next stage
        bare_barrier();
        const uint32_t t = x0;
        x0 = x1;
        x1 = t;
        now = after(now);
        read(0, x0, now, 0);
        multiply(1, [&](auto n) {
            constexpr int N = decltype(n)::value;
            X.template load<N, N + 1>(c, left_x);
            if (N == 7) next_x();
        });
    };
    int kt = 0;
#pragma unroll 1
    for (; kt + SETS < stages; kt += SETS) {
        stage(c[0]);
        stage(c[1]);
        if constexpr (SETS == 4) {
            stage(c[2]);
            stage(c[3]);
        }
    }
    if (kt + 1 < stages) stage(c[0]);
    if constexpr (SETS == 4) {
        if (kt + 2 < stages) stage(c[1]);
        if (kt + 3 < stages) stage(c[2]);
    }
#pragma unroll
    for (int step = 0; step < STEPS; ++step) {
        if (step + 1 < STEPS) read((step + 1) % 2, x0, now, step + 1);
        mask(fb[step % 2], step);
        multiply(step % 2, [](auto) {});
    }
    wait_loads<0>();         // nothing under way to LDS behind the end
}

// A wave's sums to memory: acc[i][j] holds columns d0 + 32 i + 16 p + 8 (l / 32) + e
// (register 8 p + e) of row c0 + 32 j + l % 32.  Through LDS (`stage`, this wave's own), so that a store
// instruction writes whole rows of 32 TD values and they can pass the L2: parts of 16384 x 512 x 512 20.6 us, from
// the registers 22.1 (and through the L2 24.4).  Loops are rolled up where they can be: small calls wait for
// their instructions.
template <int TD> constexpr int kStageBytes = 32 * 32 * TD * 4;
template <int TD, int TC>
__device__ inline void store_tile(const Grad8& a, floatx16 (&acc)[TD][TC], int split, int d0, int c0, int lane, uint8_t* stage) {
    constexpr int kChunks = 8 * TD;       // 16-byte chunks of a row; chunk c of row r in slot c ^ (r % kChunks)
    const int64_t pitch = a.partial ? a.partial_pitch : a.out_stride;
    float* first = a.partial ? a.partial + ((int64_t)split * a.cols + c0) * pitch + d0 : a.out + c0 * pitch + d0;
    const Through whole(first);
    const int mine = lane % kChunks, d = d0 + 4 * mine;
    const bool add = !a.partial && a.accumulate, vec = a.partial || (a.out_vec && d + 4 <= a.dim);
#pragma unroll
    for (int j = 0; j < TC; ++j) {
#pragma unroll
        for (int i = 0; i < TD; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {       // registers 4 q ..
                floatx4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
                const int r = lane % 32, c = 8 * i + 4 * (q / 2) + 2 * (lane / 32) + q % 2;
                *reinterpret_cast<floatx4*>(stage + (r * kChunks + (c ^ (r % kChunks))) * 16) = v;
            }
        wave_order();
        auto sums = [&](int r) { return *reinterpret_cast<const floatx4*>(stage + (r * kChunks + (mine ^ (r % kChunks))) * 16); };
        const int end = d < a.dim ? min(32, a.cols - c0 - 32 * j) : 0;
        if (vec) {
#pragma unroll 4
            for (int r = lane / kChunks; r < end; r += kWave / kChunks) {
                floatx4 v = sums(r);
                const int row = 32 * j + r;
                if (add) v += *reinterpret_cast<const floatx4*>(first + row * pitch + 4 * mine);
                whole.store((row * (int)pitch + 4 * mine) * 4, __builtin_bit_cast(u32x4, v));
            }
        } else if (d + 4 <= a.dim) {       // rows that are not aligned
#pragma unroll 8
            for (int r = lane / kChunks; r < end; r += kWave / kChunks) {
                floatx4 v = sums(r);
                floatx4_any* dst = reinterpret_cast<floatx4_any*>(first + (32 * j + r) * pitch + 4 * mine);
                if (add) v += *dst;
                *dst = v;
            }
        } else {                           // that end in this chunk
#pragma unroll 4
            for (int r = lane / kChunks; r < end; r += kWave / kChunks) {
                const floatx4 v = sums(r);
                float* dst = first + (32 * j + r) * pitch + 4 * mine;
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (d + e < a.dim) dst[e] = v[e] + (add ? dst[e] : 0.f);
            }
        }
        wave_order();
    }
}

// EDGE x EDGE, waves of 128 x 64: 256 with 8 waves; 128 with 4, two pairs of waves that take half
// of every stage's K each and meet in LDS (64 x 64 a wave would read a third more fragments
// for its products, and a tile of 256 x 128 is no faster: 46.3 us against 46.8).  DEEP: one workgroup of 128 per compute unit, further ahead with its loads;
// otherwise two.
template <int EDGE, bool DEEP> struct GradTile {
    static constexpr int WD = EDGE / 128, WC = EDGE / 64, kParts = EDGE == 256 ? 1 : 2, NW = WD * WC * kParts, kThreads = NW * kWave;
    static constexpr int kSlots = DEEP ? 6 : 3, kSets = DEEP ? 4 : 2;
    static constexpr size_t kBytes = (size_t)(2 + kSlots) * EDGE * kHeadK * 2;
    static_assert((size_t)NW * 16 * 1024 <= kBytes, "the pairs' meeting, the sums' way out");
};

template <int EDGE, bool DEEP>
__global__ __launch_bounds__((GradTile<EDGE, DEEP>::kThreads), DEEP ? 1 : 2) void grad8_kernel(const Grad8 a) {
    typedef GradTile<EDGE, DEEP> S;
    constexpr int TD = 4, TC = 2, NW = S::NW, kSteps = kHeadK / 16 / S::kParts;
    extern __shared__ __align__(16) uint8_t lds[];
    const int item = xcd_item(a.tiles_c * a.tiles_d * a.splits);
    if (item < 0) return;
    const int split = item / (a.tiles_c * a.tiles_d), tile = item - split * a.tiles_c * a.tiles_d;
    const int c0 = tile / a.tiles_d * EDGE, d0 = tile % a.tiles_d * EDGE;
    const int s0 = split * a.stages_per_split, s1 = min((a.rows + kHeadK - 1) / kHeadK, s0 + a.stages_per_split);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int part = wave / (S::WD * S::WC), wd = wave / S::WC % S::WD, wc = wave % S::WC;
    CodeOperand<EDGE, S::kThreads> X;
    ColOperand<EDGE, NW, TC> G;
    X.init(a.x, d0, a.dim, (int64_t)s0 * kHeadK, wd * TD * 32, part * kSteps, threadIdx.x, lane);
    G.init(a.grad, a.grad_stride * 2, c0, a.cols8, (int64_t)s0 * kHeadK, wc * TC * 32, false, wave, lane);
#pragma unroll
    for (int j = 0; j < TC; ++j) G.at[j] += part * kSteps * 16 * G.kRow;
    floatx16 acc[TD][TC];
    clear(acc);
    k_loop_coded<kSteps, S::kSlots, S::kSets, TD, TC>(acc, s1 - s0, X, G, min(a.rows - s0 * kHeadK, (s1 - s0) * kHeadK), part * kSteps, lds_address(lds),
                                 wave, lane);
    wait_lds();
    bare_barrier();      // every wave is done with the operands, whose LDS the sums pass through
    if constexpr (S::kParts == 1) {
        store_tile<TD, TC>(a, acc, split, d0 + wd * TD * 32, c0 + wc * TC * 32, lane, lds + wave * kStageBytes<TD>);
    } else {
        // each pair keeps half of the columns and gives the other half away
        constexpr int kHalf = TD / 2;
        static_assert(kHalf * TC * 16 * kWave * 4 == 16 * 1024, "what a wave gives");
        floatx4* given = reinterpret_cast<floatx4*>(lds);
        floatx16 mine[kHalf][TC];
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
#pragma unroll
            for (int j = 0; j < TC; ++j) {
                mine[i][j] = part ? acc[kHalf + i][j] : acc[i][j];
                const floatx16 give = part ? acc[i][j] : acc[kHalf + i][j];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    floatx4 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = give[4 * q + e];
                    given[((wave * kHalf + i) * TC + j) * 4 * kWave + q * kWave + lane] = v;
                }
            }
        __syncthreads();
        const int other = wave ^ (S::WD * S::WC);
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
#pragma unroll
            for (int j = 0; j < TC; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const floatx4 v = given[((other * kHalf + i) * TC + j) * 4 * kWave + q * kWave + lane];
#pragma unroll
                    for (int e = 0; e < 4; ++e) mine[i][j][4 * q + e] += v[e];
                }
        // what the other wave gave is this wave's alone, and read
        static_assert(kStageBytes<kHalf> <= 16 * 1024, "room for a stage");
        store_tile<kHalf, TC>(a, mine, split, d0 + wd * TD * 32 + part * kHalf * 32, c0 + wc * TC * 32, lane, lds + other * 16 * 1024);
    }
}

// The splits' sums in order, added to what is there.  5.8 us for 4 parts of 2048 x 512.  Parts written past the last cache, or
// read so, cost 2 to 4 us more.
__global__ __launch_bounds__(kJoinThreads) void join8_kernel(const Join8 a) {
    const int64_t quads = (a.dim + 3) / 4, items = quads * a.cols, step = (int64_t)a.cols * a.partial_pitch;
    for (int64_t n = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; n < items; n += (int64_t)gridDim.x * kJoinThreads) {
        const int64_t c = n / quads, d = (n - c * quads) * 4;
        floatx4 v = {0.f, 0.f, 0.f, 0.f};
        const float* src = a.partial + c * a.partial_pitch + d;
        int s = 0;
        for (; s + kJoinBatch <= a.splits; s += kJoinBatch) {
            floatx4 part[kJoinBatch];
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k, src += step) part[k] = *reinterpret_cast<const floatx4*>(src);
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) v += part[k];
        }
        for (; s < a.splits; ++s, src += step) v += *reinterpret_cast<const floatx4*>(src);
        float* dst = a.out + c * a.out_stride + d;
        if (d + 4 <= a.dim) {
            if (a.accumulate) v += *reinterpret_cast<const floatx4_any*>(dst);
            *reinterpret_cast<floatx4_any*>(dst) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < a.dim) dst[e] = v[e] + (a.accumulate ? dst[e] : 0.f);
        }
    }
}

template <int EDGE, bool DEEP>
hipError_t launch(const Grad8& a, hipStream_t s) {
    typedef GradTile<EDGE, DEEP> S;
    const hipError_t allowed = hipFuncSetAttribute(reinterpret_cast<const void*>(&grad8_kernel<EDGE, DEEP>),
                                                   hipFuncAttributeMaxDynamicSharedMemorySize, (int)S::kBytes);
    if (allowed != hipSuccess) return allowed;
    grad8_kernel<EDGE, DEEP><<<xcd_grid(a.tiles_c * a.tiles_d * a.splits), S::kThreads, S::kBytes, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grad8(const Grad8& a, int edge, bool deep, hipStream_t s) {
    if (edge == 256) return launch<256, false>(a, s);
    return deep ? launch<128, true>(a, s) : launch<128, false>(a, s);
}

hipError_t launch_join8(const Join8& a, hipStream_t s) {
    const int64_t items = (int64_t)a.cols * ((a.dim + 3) / 4);
    join8_kernel<<<(int)std::min<int64_t>(32768, (items + kJoinThreads - 1) / kJoinThreads), kJoinThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace muon
