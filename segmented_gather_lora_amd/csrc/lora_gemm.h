// lora_gemm.h -- the tile product shared by the kernels of the projection with
// adapters (lora_linear.hip) and of the vocabulary cross entropy
// (lora_loss.hip).
//
// A workgroup computes one tile  D[m][n] = sum_k M[m][k] * N[n][k]  on the bf16
// MFMA (v_mfma_f32_16x16x32_bf16, fp32 sums).  The M side is always the side
// whose index is contiguous in the output row (output columns, vocabulary
// entries, ranks), so that every lane ends up with groups of 4 consecutive
// output elements of one output row.
//
// K is walked in steps of 64.  Every step's 128-byte rows are copied from
// memory straight into one of two LDS stages by direct-to-LDS loads (16 bytes a
// lane, 1 KB an instruction); nothing passes through registers.  A side is
// either
//   contiguous: rows of K elements (K contiguous in memory).  LDS holds
//               [row][64]; the 16-byte chunk c of row r sits in slot
//               c ^ f(r), so that the MFMA operand reads (ds_read_b128 of one
//               chunk of 16 rows) spread over the banks;
//   strided:    K is the row index in memory and the side's own index is
//               contiguous (W in dy * W, x and dy in the weight gradients).
//               LDS holds [64][rows]; operands come through the transposing
//               read ds_read_b64_tr_b16 (16 lanes read a 4 x 16 block, lane l
//               gets its column l), with 32-byte pieces of K row k moved to
//               slot p ^ f(k) for the same reason.
// Both give lane (l16, g) of a wave the K elements 32 h + 8 g .. + 8 of half h
// for row l16 of each 16-row tile, the layout the MFMA takes.
//
// A step is 2 NT groups of MFMAs, one 16-row tile of the N side each, half 0 of
// the step and then half 1; a wave holds both halves' operands in registers:
//     groups 0 .. F    the reads of half 1 are between the MFMAs; barrier: every
//                      wave has read the step's stage
//     groups F ..      the copies of step s + 2 into that stage, evenly
//     before group L   barrier: step s + 1 has landed (its copies had L + 2 NT - F
//                      groups or more)
//     groups L ..      the reads of half 0 of step s + 1
// The copies of a step keep a CU's vector cache busy for 1200 of the 2048 cycles
// that its MFMAs take (measured: 53 bytes a cycle where every row gives 128 bytes
// or more, 27 where it gives 64, so that K steps of 32 in more stages are no
// faster), hence the even spread; issued at once behind one barrier they made
// the step 2900 cycles long.  The order is pinned: left to itself the compiler
// puts the reads first, and eight waves, just past a barrier, queue at the LDS.
// K tails and adapters' ranks run after the pinned loop in a plain one that
// holds one half at a time and has two steps' copies in flight.
//
// Tiles too small to be bound by the MFMA have more stages and a plain loop:
// what counts there is the bytes in flight.
//
// The direct-to-LDS loads are written in assembly (they have no output
// registers): the builtin makes the compiler wait for every load in flight
// before each LDS read, since it cannot tell the stages apart.  The waits that
// order them are the explicit ones of the loops.
#pragma once

#include "lora_internal.h"

namespace lora {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) unsigned char lds_byte;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
typedef uint32_t u32x2g __attribute__((ext_vector_type(2)));

constexpr int kStepK = 64;

// Zeros that lanes without data read (K tails, rows outside a segment).
static __device__ __attribute__((aligned(256))) uint16_t zero_page[128];

// 64 lanes x 16 bytes from each lane's `src` to LDS byte `dst` + 16 * lane.  The LDS
// address goes through M0, named as the operand's register, so that the compiler
// knows what is written there (s_nop: the wait state between that write and the load).
__device__ __forceinline__ void dma16(const uint16_t *src, uint32_t dst) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(dst), "v"(src) : "memory");
}

// The same from a scalar base and a lane's byte offset.
__device__ __forceinline__ void dma16(const uint16_t *base, uint32_t offset, uint32_t dst) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(dst), "v"(offset), "s"(base) : "memory");
}

// Which rows (or K rows) and chunks of a side's stage a lane copies, and where
// it reads its operands.  ROWS: rows of the tile's side; WAVES: waves that
// share the copy.  QUADS (contiguous sides): rows of a 64-row group are dealt
// to its four MFMA tiles by fours (row 16 q + 4 t + e is row 4 q + e of tile
// t), so that a lane's outputs of the four tiles are 16 consecutive elements.
template <int ROWS, int WAVES, bool STRIDED, bool QUADS>
struct Side {
    static constexpr int kInstr = ROWS / 8 / WAVES;
    static constexpr int kBytes = ROWS * 128;
    static constexpr int kPairs = ROWS / 16;            // 32-byte pieces of a strided K row
    static constexpr int kLanesPerK = ROWS / 8;         // lanes that copy one K row
    static_assert(ROWS % (8 * WAVES) == 0, "every wave copies whole instructions");
    static_assert(!STRIDED || (ROWS >= 16 && ROWS <= 512 && (ROWS & (ROWS - 1)) == 0), "strided rows");

    __device__ __forceinline__ static int f_row(int r) {
        return QUADS ? ((r & 3) | ((r >> 4) & 1) << 2) : (r & 7);
    }
    __device__ __forceinline__ static int f_k(int k) { return ((k & 3) | ((k >> 3) & 3) << 2) & (kPairs - 1); }

    // copy: the row (contiguous) or K row (strided) of instruction j in this lane
    __device__ __forceinline__ static int row(int j) {
        const int i = wave_id() * kInstr + j;
        return STRIDED ? i * (64 / kLanesPerK) + lane_id() / kLanesPerK : i * 8 + (lane_id() >> 3);
    }
    // copy: first element along the contiguous direction (K, or the side's own index)
    __device__ __forceinline__ static int elem(int j) {
        if (STRIDED) return elem_of(row(j));
        return ((lane_id() & 7) ^ f_row(row(j))) * 8;
    }
    // strided: the same for K row k
    __device__ __forceinline__ static int elem_of(int k) {
        const int slot = lane_id() % kLanesPerK;
        return (((slot >> 1) ^ f_k(k)) * 2 + (slot & 1)) * 8;
    }
    // K offset of the lane's 8 elements (contiguous) or its K row (strided)
    __device__ __forceinline__ static int koff(int j) { return STRIDED ? row(j) : elem(j); }
    __device__ __forceinline__ static uint32_t dst(int j) { return (uint32_t)(wave_id() * kInstr + j) * 1024u; }

    // strided: byte of K row k, element v of the side's own index
    __device__ __forceinline__ static int at(int k, int v) {
        return k * (ROWS * 2) + 32 * ((v >> 4) ^ f_k(k)) + 2 * (v & 15);
    }

    // operand of the 16-row tile `t` counted from row `base` (a multiple of 16;
    // of 64 with QUADS), half h of the step in the stage at `st`
    __device__ __forceinline__ static bf16x8 read(const lds_byte *st, int base, int t, int h) {
        const int l16 = lane_id() & 15, g = lane_id() >> 4;
        if (STRIDED) {
            const int i = l16 >> 2, q = l16 & 3;
            const int fk = (i | g << 2) & (kPairs - 1);
            const int k = 32 * h + 8 * g + i;
            const lds_byte *p = st + k * (ROWS * 2) + 32 * ((base / 16 + t) ^ fk) + 8 * q;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * (ROWS * 2)));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        const int r = QUADS ? base + 64 * (t >> 2) + 16 * (l16 >> 2) + 4 * (t & 3) + (l16 & 3) : base + 16 * t + l16;
        return *(const lds_bf16x8 *)(st + r * 128 + 16 * ((4 * h + g) ^ f_row(QUADS ? (l16 & 3) | (l16 >> 2 & 1) << 4 : l16)));
    }
};

// Tile of BM x BN by WM x WN waves.  SPLIT: 0 plain; 1: the M side's stage
// holds 2 * BM rows, the low parts after the high parts, and both are
// multiplied into the same sums; 2: the same on the N side.
template <int BM_, int BN_, int WM_, int WN_, bool MS_, bool NS_, int SPLIT_ = 0, int STAGES_ = 2>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, SPLIT = SPLIT_, kStages = STAGES_;
    static constexpr bool MS = MS_, NS = NS_;
    static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
    static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    static constexpr bool QUADS = !MS && MT % 4 == 0;
    static constexpr int MROWS = BM * (SPLIT == 1 ? 2 : 1), NROWS = BN * (SPLIT == 2 ? 2 : 1);
    using MSide = Side<MROWS, kWaves, MS, QUADS>;
    using NSide = Side<NROWS, kWaves, NS, false>;
    static constexpr int kStage = MSide::kBytes + NSide::kBytes;
    static constexpr int kLds = kStages * kStage;
    typedef floatx4 Acc[MT][NT];

    __device__ __forceinline__ static int wave_m() { return wave_id() % WM; }
    __device__ __forceinline__ static int wave_n() { return wave_id() / WM; }
    // tile row (output column) of element 0 of acc[mt][..] in this lane
    __device__ __forceinline__ static int m_of(int mt) {
        const int g = lane_id() >> 4;
        return wave_m() * (BM / WM) + (QUADS ? 64 * (mt >> 2) + 16 * g + 4 * (mt & 3) : 16 * mt + 4 * g);
    }
    __device__ __forceinline__ static int n_of(int nt) { return wave_n() * (BN / WN) + 16 * nt + (lane_id() & 15); }

    struct Half {
        bf16x8 m[MT * (SPLIT == 1 ? 2 : 1)], n[NT * (SPLIT == 2 ? 2 : 1)];
    };
    static constexpr int kMReads = MT * (SPLIT == 1 ? 2 : 1), kNReads = NT * (SPLIT == 2 ? 2 : 1);
    static constexpr int kReads = kMReads + kNReads, kLoads = MSide::kInstr + NSide::kInstr;
    // operand i of a half: the M side's, then the N side's
    __device__ __forceinline__ static void read_one(Half &r, const lds_byte *st, int h, int i) {
        if (i < kMReads)
            r.m[i] = MSide::read(st, (i < MT ? 0 : BM) + wave_m() * (BM / WM), i % MT, h);
        else
            r.n[i - kMReads] = NSide::read(st + MSide::kBytes, (i - kMReads < NT ? 0 : BN) + wave_n() * (BN / WN),
                                           (i - kMReads) % NT, h);
    }
    __device__ __forceinline__ static void read(Half &r, const lds_byte *st, int h) {
#pragma unroll
        for (int i = 0; i < kReads; ++i) read_one(r, st, h, i);
    }
    __device__ __forceinline__ static void read_m(Half &r, const lds_byte *st, int h) {
#pragma unroll
        for (int i = 0; i < kMReads; ++i) read_one(r, st, h, i);
    }
    __device__ __forceinline__ static void read_n(Half &r, const lds_byte *st, int h) {
#pragma unroll
        for (int i = kMReads; i < kReads; ++i) read_one(r, st, h, i);
    }
    // the products of one 16-row tile of the N side
    __device__ __forceinline__ static void mma_n(const Half &r, Acc &acc, int nt) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            acc[mt][nt] = mfma16x16x32(r.m[mt], r.n[nt], acc[mt][nt]);
            if constexpr (SPLIT == 1) acc[mt][nt] = mfma16x16x32(r.m[MT + mt], r.n[nt], acc[mt][nt]);
            if constexpr (SPLIT == 2) acc[mt][nt] = mfma16x16x32(r.m[mt], r.n[NT + nt], acc[mt][nt]);
        }
    }
    __device__ __forceinline__ static void mma(const Half &r, Acc &acc) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_n(r, acc, nt);
    }
};

// The product into the N rows [lo, hi) of the tile only: no other row's sums
// are touched, whatever the operands hold.
template <class T>
__device__ __forceinline__ void mma_rows(const typename T::Half &r, typename T::Acc &acc, int lo, int hi) {
    static_assert(T::SPLIT == 0, "plain tiles");
#pragma unroll
    for (int nt = 0; nt < T::NT; ++nt) {
        const int r0 = T::wave_n() * (T::BN / T::WN) + 16 * nt;
        if (r0 + 16 <= lo || r0 >= hi) continue;
        const int n = T::n_of(nt);
        const bool mine = n >= lo && n < hi;
#pragma unroll
        for (int mt = 0; mt < T::MT; ++mt) {
            const floatx4 d = mfma16x16x32(r.m[mt], r.n[nt], acc[mt][nt]);
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[mt][nt][x] = mine ? d[x] : acc[mt][nt][x];
        }
    }
}

template <class T>
__device__ __forceinline__ void clear(typename T::Acc &acc) {
#pragma unroll
    for (int mt = 0; mt < T::MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < T::NT; ++nt) acc[mt][nt] = floatx4{0.f, 0.f, 0.f, 0.f};
}

template <int N>
__device__ __forceinline__ void wait_loads_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ void own_reads_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A product of `nsteps` steps: mma_begin, then mma_loop with the same
// arguments; between them a workgroup may do what does not touch `lds`.
// op.issue(stage) copies the next step's operands to the LDS byte address
// `stage` (called once per step, in order; every wave makes at least Op::kLast
// copies after the last of the N side); op.read(half, stage, s, h) and
// op.mma(half, acc, s, h) read a half of step s (half 1 with half 0's operands at
// hand) and multiply it into the sums.
// The first `plain` steps make T::kLoads copies in every wave: op.load(stage, i)
// are these one by one, op.next() moves on to the next step, op.mma_n(half, acc,
// nt) multiplies.  All threads of the workgroup call it; LDS of T::kLds bytes at
// `lds`, which no one else uses until it returns.
__device__ __forceinline__ uint32_t lds_address(unsigned char *lds) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_byte *)lds);
}
template <class T>
constexpr int kAhead = T::kStages == 2 ? 2 : T::kStages - 1;   // steps copied before the first is multiplied

template <class T, class Op>
__device__ __forceinline__ void mma_begin(Op &op, int nsteps, unsigned char *lds) {
    const uint32_t base = lds_address(lds);
    for (int i = 0; i < kAhead<T> && i < nsteps; ++i) op.issue(base + i * T::kStage);
}

// Small tiles: one barrier a step, kStages - 2 steps' copies in flight across it.
template <class T, class Op>
__device__ __forceinline__ void ring_loop(Op &op, int plain, int nsteps, typename T::Acc &acc, const lds_byte *lds,
                                          uint32_t base) {
    constexpr int S = T::kStages;
    int cur = 0, to = (S - 1) * T::kStage, s = 0;
    auto turn = [&] {
        to = cur;
        cur = cur + T::kStage == T::kLds ? 0 : cur + T::kStage;
    };
    // at the barrier step s has landed, for every wave, and step s - 1 is read
    for (; s + S - 1 < plain; ++s) {
        wait_loads_barrier<(S - 2) * T::kLoads>();
        typename T::Half r0, r1;
        T::read(r0, lds + cur, 0);
        T::read(r1, lds + cur, 1);
        __builtin_amdgcn_sched_barrier(0);
        // the copies go between the MFMAs: a wave that issues them first waits for
        // the whole workgroup's before it reads its operands
#pragma unroll
        for (int g = 0; g < 2 * T::NT; ++g) {
            constexpr int G = 2 * T::NT, D = T::kLoads;
            op.mma_n(g < T::NT ? r0 : r1, acc, g % T::NT);
#pragma unroll
            for (int i = g * D / G; i < (g + 1) * D / G; ++i) op.load(base + to, i);
            if (g == G - 1) op.next();
            __builtin_amdgcn_sched_barrier(0);
        }
        turn();
    }
    for (; s < nsteps; ++s) {
        if (s + S - 1 <= plain)
            wait_loads_barrier<(S - 2) * T::kLoads>();
        else if (s + S - 1 <= nsteps)
            wait_loads_barrier<(S - 2) * Op::kLast>();
        else
            wait_loads_barrier<0>();
        if (s + S - 1 < nsteps) op.issue(base + to);
        typename T::Half r0, r1;
        op.read(r0, lds + cur, s, 0);
        op.read(r1, lds + cur, s, 1, r0);
        op.mma(r0, acc, s, 0);
        op.mma(r1, acc, s, 1);
        turn();
    }
}

template <class T, class Op>
__device__ __forceinline__ void mma_loop(Op &op, int plain, int nsteps, typename T::Acc &acc, unsigned char *lds_generic) {
    const lds_byte *lds = (const lds_byte *)lds_generic;
    const uint32_t base = lds_address(lds_generic);
    if (nsteps <= 0) return;
    if constexpr (T::kStages > 2) {
        ring_loop<T>(op, plain, nsteps, acc, lds, base);
        return;
    }
    int s = 0;
    if (plain > 2) {
        // groups of a step: one 16-row tile of the N side, half 0 then half 1
        constexpr int G = 2 * T::NT, R = T::kReads, D = T::kLoads;
        constexpr int F = T::NT > 1 ? T::NT * 3 / 4 : 1, L = T::NT + T::NT / 4;
        constexpr int kInFlight = D * (L - F) / (G - F);   // (every wave makes the same copies of a pinned step)
        typename T::Half r0, r1;
        wait_loads_barrier<Op::kLast>();
        T::read(r0, lds, 0);
        for (; s + 2 < plain; ++s) {
            const uint32_t cur = (uint32_t)(s & 1) * T::kStage, nxt = T::kStage - cur;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (g == F) own_reads_barrier();
                if (g == L) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kInFlight) : "memory");
                if (g < F) {
#pragma unroll
                    for (int i = g * R / F; i < (g + 1) * R / F; ++i) T::read_one(r1, lds + cur, 1, i);
                } else {
#pragma unroll
                    for (int i = (g - F) * D / (G - F); i < (g - F + 1) * D / (G - F); ++i) op.load(base + cur, i);
                }
                if (g >= L) {
#pragma unroll
                    for (int i = (g - L) * R / (G - L); i < (g - L + 1) * R / (G - L); ++i) T::read_one(r0, lds + nxt, 0, i);
                }
                if (g < T::NT)
                    op.mma_n(r0, acc, g);
                else
                    op.mma_n(r1, acc, g - T::NT);
                if (g == G - 1) op.next();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    for (; s < nsteps; ++s) {
        const uint32_t cur = (uint32_t)(s & 1) * T::kStage;
        // step s has landed; of step s + 1 the copies that every wave makes last may be in flight
        if (s + 1 < nsteps)
            wait_loads_barrier<Op::kLast>();
        else
            wait_loads_barrier<0>();
        typename T::Half r;
        op.read(r, lds + cur, s, 0);
        op.mma(r, acc, s, 0);
        op.read(r, lds + cur, s, 1, r);
        own_reads_barrier();
        if (s + 2 < nsteps) op.issue(base + cur);
        op.mma(r, acc, s, 1);
    }
}

// A side's plain K walk: per instruction a pointer that moves on by `step`
// elements a step; lanes past the end of K read zeros.
template <class S>
struct Walk {
    const uint16_t *p[S::kInstr];
    int64_t step;
    int left;      // K elements (rows) left from the next step on
    __device__ __forceinline__ void load(uint32_t at, int j) { dma16(p[j], at + S::dst(j)); }
    __device__ __forceinline__ void next() {
#pragma unroll
        for (int j = 0; j < S::kInstr; ++j) p[j] += step;
        left -= kStepK;
    }
    __device__ __forceinline__ void issue(uint32_t at) {
#pragma unroll
        for (int j = 0; j < S::kInstr; ++j) dma16(S::koff(j) < left ? p[j] : zero_page, at + S::dst(j));
        next();
    }
};

// The same from a scalar base with 32-bit offsets of the lanes: half the
// registers, where 64 K rows are less than 4 GB.
template <class S>
struct OffsetWalk {
    const uint16_t *base;
    uint32_t off[S::kInstr];   // bytes
    int64_t step;
    int left;
    __device__ __forceinline__ void load(uint32_t at, int j) { dma16(base, off[j], at + S::dst(j)); }
    __device__ __forceinline__ void next() {
        base += step;
        left -= kStepK;
    }
    __device__ __forceinline__ void issue(uint32_t at) {
#pragma unroll
        for (int j = 0; j < S::kInstr; ++j)
            dma16(S::koff(j) < left ? base + off[j] / 2 : zero_page, at + S::dst(j));
        next();
    }
};

// K rows gathered by the sorted token indices (weight gradients: K runs over a
// segment's tokens) for a strided side.  An instruction copies few K rows, so
// the indices of a step are loaded a step ahead as scalars: their wait does not
// touch the count of the copies in flight.
typedef const __attribute__((address_space(4))) int32_t *const_ints;
template <class S>
struct GatherWalk {
    static constexpr int kRows = 64 / S::kLanesPerK;   // K rows of an instruction
    const uint16_t *base;
    const int32_t *sorted;
    int64_t ld;
    int tok[S::kInstr][kRows], col[S::kInstr];
    int pos, end, num_tokens;
    __device__ __forceinline__ void fetch() {
        const_ints from = (const_ints)(uintptr_t)sorted;
#pragma unroll
        for (int j = 0; j < S::kInstr; ++j)
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                const int p = pos + (wave_id() * S::kInstr + j) * kRows + q;
                tok[j][q] = from[__builtin_amdgcn_readfirstlane(p < end ? p : end - 1)];
            }
    }
    __device__ __forceinline__ const uint16_t *at_token(int j) const {
        int t = __builtin_amdgcn_readfirstlane(tok[j][0]);
#pragma unroll
        for (int q = 1; q < kRows; ++q) {   // (a plain select of the entries becomes an array in scratch memory)
            const int u = __builtin_amdgcn_readfirstlane(tok[j][q]);
            t = lane_id() / S::kLanesPerK == q ? u : t;
        }
        return (unsigned)t < (unsigned)num_tokens ? base + (int64_t)t * ld + col[j] : zero_page;
    }
    __device__ __forceinline__ void load(uint32_t at, int j) { dma16(at_token(j), at + S::dst(j)); }
    __device__ __forceinline__ void next() {
        pos += kStepK;
        if (pos < end) fetch();
    }
    __device__ __forceinline__ void issue(uint32_t at) {
#pragma unroll
        for (int j = 0; j < S::kInstr; ++j)
            dma16(pos + S::koff(j) < end ? at_token(j) : zero_page, at + S::dst(j));
        next();
    }
};

// The two sides of a product whose steps are all plain but the last.
template <class T, class WM, class WN>
struct PairOp {
    static constexpr int kLast = T::MSide::kInstr;
    WM wm;
    WN wn;
    __device__ __forceinline__ void read(typename T::Half &r, const lds_byte *st, int, int h) { T::read(r, st, h); }
    __device__ __forceinline__ void read(typename T::Half &r, const lds_byte *st, int, int h, const typename T::Half &) {
        T::read(r, st, h);
    }
    __device__ __forceinline__ void mma(const typename T::Half &h, typename T::Acc &acc, int, int) { T::mma(h, acc); }
    __device__ __forceinline__ void mma_n(const typename T::Half &h, typename T::Acc &acc, int nt) { T::mma_n(h, acc, nt); }
    __device__ __forceinline__ void load(uint32_t at, int i) {
        if (i < T::MSide::kInstr)
            wm.load(at, i);
        else
            wn.load(at + T::MSide::kBytes, i - T::MSide::kInstr);
    }
    __device__ __forceinline__ void next() {
        wm.next();
        wn.next();
    }
    __device__ __forceinline__ void issue(uint32_t at) {
        wn.issue(at + T::MSide::kBytes);
        wm.issue(at);
    }
};
template <class T>
using PlainOp = PairOp<T, Walk<typename T::MSide>, Walk<typename T::NSide>>;

// Adds up the partial sums of `splits` workgroups that share a tile, each over
// its own K steps.  Every workgroup stores its sums in its slot and counts
// itself; the one that comes last adds the slots in split order (so the result
// does not depend on the order of arrival) and returns true: it writes the tile.
// Nobody waits.  The counter starts at zero.  `rows` N rows of the tile are in
// use.  The slots are stored and loaded at device scope, since the
// workgroups run on different XCDs.
constexpr int kScopeDevice = 16;   // sc1
typedef int32_t i32x4g __attribute__((ext_vector_type(4)));
template <class T>
__device__ __forceinline__ bool combine_splits(typename T::Acc &acc, float *slots, int32_t *counter, int split,
                                               int splits, int rows, int *s_flag) {
    constexpr int kSlot = T::BM * T::BN;
    const int tid = threadIdx.x;
    auto rsrc = [&](int k) { return __builtin_amdgcn_make_buffer_rsrc(slots + (int64_t)k * kSlot, 0, kSlot * 4, 0x00020000); };
    {
        const __amdgpu_buffer_rsrc_t own = rsrc(split);
#pragma unroll
        for (int mt = 0; mt < T::MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < T::NT; ++nt)
                if (T::n_of(nt) < rows)
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4g, acc[mt][nt]), own, 16 * tid,
                                                           (mt * T::NT + nt) * 16 * T::kThreads, kScopeDevice);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0)
        *s_flag = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == splits - 1;
    __syncthreads();
    if (!*s_flag) return false;
    typename T::Acc own;
#pragma unroll
    for (int mt = 0; mt < T::MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < T::NT; ++nt) {
            own[mt][nt] = acc[mt][nt];
            acc[mt][nt] = floatx4{0.f, 0.f, 0.f, 0.f};
        }
    for (int k = 0; k < splits; ++k) {
        const __amdgpu_buffer_rsrc_t from = rsrc(k);
#pragma unroll
        for (int mt = 0; mt < T::MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < T::NT; ++nt)
                if (T::n_of(nt) < rows)
                    acc[mt][nt] += k == split ? own[mt][nt]
                                              : __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(
                                                                                from, 16 * tid, (mt * T::NT + nt) * 16 * T::kThreads,
                                                                                kScopeDevice));
    }
    return true;
}

// Dynamic LDS above 64 KB has to be allowed once per kernel and device.
inline hipError_t allow_lds(const void *fn, size_t bytes, unsigned long long (&done)[1]) {
    if (bytes <= 65536) return hipSuccess;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (__atomic_load_n(&done[0], __ATOMIC_RELAXED) & bit) return hipSuccess;
    e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == hipSuccess) __atomic_fetch_or(&done[0], bit, __ATOMIC_RELAXED);
    return e;
}
template <auto *Kernel, class... Args>
hipError_t launch_tiles(unsigned grid, int threads, size_t lds, hipStream_t s, const Args &...args) {
    static unsigned long long done[1];
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(Kernel), lds, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(Kernel, dim3(grid), dim3(threads), lds, s, args...);
    return hipGetLastError();
}

// Workgroup -> tile: the tiles are cut into one contiguous run per XCD
// (workgroup b sits on XCD b % 8), and a run walks the N tiles of a panel of
// `group` for every M tile, so that the tiles running together on an XCD share
// both sides' rows through its L2.  Returns false past the end.
struct TileAt {
    int m, n;
};
__device__ __forceinline__ bool tile_at(int block, int mtiles, int ntiles, int group, TileAt &t) {
    const int total = mtiles * ntiles;
    const int chunk = (total + kNumXcd - 1) / kNumXcd;
    const int j = block / kNumXcd;
    const int u = (block % kNumXcd) * chunk + j;
    if (j >= chunk || u >= total) return false;
    const int panel = u / (group * mtiles);
    const int width = min(group, ntiles - panel * group);
    const int in = u - panel * group * mtiles;
    t.m = in / width;
    t.n = panel * group + in % width;
    return true;
}
inline unsigned tile_grid(long tiles) { return (unsigned)((tiles + kNumXcd - 1) / kNumXcd * kNumXcd); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return float_to_bf16_bits(a) | float_to_bf16_bits(b) << 16;
}
__device__ __forceinline__ void unpack_bf16(uint32_t v, float &a, float &b) {
    a = bf16_bits_to_float(v & 0xffffu);
    b = bf16_bits_to_float(v >> 16);
}

}  // namespace lora
