// lora_mx.h -- microscaled 4-bit numbers: sizes and conversions shared by the kernels
// that read or write them.  A row is blocks of 32 numbers: 16 bytes of E2M1 codes (two a
// byte, the first in the low half) and one byte, the exponent of their common power
// of two plus 127.
#pragma once

#include <string.h>

#include "lora_gemm.h"

namespace lora {

constexpr int kMxBlock = 32;
inline int64_t mx_blocks(int64_t cols) { return (cols + kMxBlock - 1) / kMxBlock; }
inline int64_t mx_code_bytes(int64_t cols) { return 16 * mx_blocks(cols); }
inline int64_t mx_scale_bytes(int64_t cols) { return (mx_blocks(cols) + 3) / 4 * 4; }

// The scale byte (the power's exponent plus 127) of a block whose largest magnitude
// has these bits: floor(log2) - 2, 2 being E2M1's largest exponent; 255 (not a
// number) for a block that is not finite.
__device__ __forceinline__ int mx_scale_of(uint32_t top) {
    const int e = (int)(top >> 23);
    return e == 255 ? 255 : e > 2 ? e - 2 : 0;
}
// 8 codes: v over the power (exact, but for what is far below half of the smallest
// code), to the nearest, ties to even, held at 6.
__device__ __forceinline__ uint32_t mx_codes_of(const float v[8], int scale) {
    if (scale == 255) return 0u;
    const float inv = __uint_as_float((uint32_t)(254 - scale) << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * inv, v[1] * inv, 1.f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * inv, v[3] * inv, 1.f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * inv, v[5] * inv, 1.f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * inv, v[7] * inv, 1.f, 3);
    return c;
}

// A block of 32 bf16 numbers in one lane: its codes, and its scale byte.
__device__ __forceinline__ int mx_block_codes(const u32x4 (&x)[4], u32x4 &codes) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(max(top, x[j][e] << 16 & 0x7fff0000u), x[j][e] & 0x7fff0000u);
    const int scale = mx_scale_of(top);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack_bf16(x[j][e], v[2 * e], v[2 * e + 1]);
        codes[j] = mx_codes_of(v, scale);
    }
    return scale;
}
// 8 codes (a dword) times their power as bf16, exact.  The conversion reads the
// exponent alone: 0 gives 2^-127, 255 NaN.
__device__ __forceinline__ u32x4 mx_numbers(uint32_t codes, uint32_t scale) {
    const float s = __uint_as_float(scale << 23);
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3))};
}

// Sixteen lanes take 128 numbers of a row, 8 each, and with them one dword of
// scales; a lane's codes are a dword.
constexpr int kMxThreads = 256, kMxGroup = 16, kMxSpan = 128, kMxPer = 2;

// 8 numbers of a row as float bits, zeros past its end (which is a multiple of 8).
__device__ __forceinline__ void mx_load(const uint16_t *p, bool in, float v[8]) {
    const u32x4 q = in ? *reinterpret_cast<const u32x4 *>(p) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int x = 0; x < 4; ++x) unpack_bf16(q[x], v[2 * x], v[2 * x + 1]);
}
__device__ __forceinline__ void mx_load(const float *p, bool in, float v[8]) {
    const floatx4 z = {0.f, 0.f, 0.f, 0.f};
    const floatx4 a = in ? *reinterpret_cast<const floatx4 *>(p) : z, b = in ? *reinterpret_cast<const floatx4 *>(p + 4) : z;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        v[x] = a[x];
        v[4 + x] = b[x];
    }
}

struct MxArgs {
    char *x, *codes, *scales;            // x: the numbers, read or written
    int64_t ldx, ldcodes, ldscales;      // bytes
    int64_t rows;
    int32_t cols, blocks, spans;         // of a row
};

// The lane's span: row and number within the row.
struct MxAt {
    int64_t row;
    int32_t span;
};
__device__ __forceinline__ MxAt mx_at(int64_t first, int i, int spans) {
    const int64_t row0 = first / spans;                 // (uniform)
    const uint32_t in = (uint32_t)(first - row0 * spans) + (uint32_t)i;
    const uint32_t r = in / (uint32_t)spans;
    return MxAt{row0 + r, (int32_t)(in - r * (uint32_t)spans)};
}

constexpr int kMxSpans = kMxThreads / kMxGroup * kMxPer;   // of a workgroup
constexpr int64_t kMxMostBlocks = 1 << 23;                 // a launch has fewer than 2^32 threads
inline MxArgs mx_args(const void *x, int type, int64_t ldx, int64_t rows, int cols, const void *codes, int64_t ldcodes,
                      const void *scales, int64_t ldscales) {
    MxArgs a;
    memset(&a, 0, sizeof a);
    a.x = static_cast<char *>(const_cast<void *>(x));
    a.codes = static_cast<char *>(const_cast<void *>(codes));
    a.scales = static_cast<char *>(const_cast<void *>(scales));
    a.ldx = ldx * (type == LORA_BF16 ? 2 : 4);
    a.ldcodes = ldcodes;
    a.ldscales = ldscales;
    a.rows = rows;
    a.cols = cols;
    a.blocks = (int32_t)mx_blocks(cols);
    a.spans = (a.blocks + 3) / 4;
    return a;
}
__host__ __device__ inline int64_t mx_grid(const MxArgs &a) { return (a.rows * a.spans + kMxSpans - 1) / kMxSpans; }

// Exact in float32 and bfloat16: a code has two bits and every power a place in both
// (the smallest as a subnormal number).
template <class F>
__device__ __forceinline__ void dequantize(const MxArgs &a, int block) {
    constexpr int kSpans = kMxThreads / kMxGroup;
    const int l = threadIdx.x % kMxGroup, g = threadIdx.x / kMxGroup;
    uint32_t c[kMxPer], s[kMxPer];
    MxAt at[kMxPer];
    bool in[kMxPer];
#pragma unroll
    for (int q = 0; q < kMxPer; ++q) {
        at[q] = mx_at((int64_t)block * (kSpans * kMxPer), q * kSpans + g, a.spans);
        in[q] = at[q].row < a.rows && at[q].span * kMxSpan + 8 * l < a.cols;
        c[q] = s[q] = 0;
        if (in[q]) {
            c[q] = *reinterpret_cast<const uint32_t *>(a.codes + at[q].row * a.ldcodes + at[q].span * 64 + 4 * l);
            s[q] = (uint8_t)a.scales[at[q].row * a.ldscales + at[q].span * 4 + l / 4];
        }
    }
#pragma unroll
    for (int q = 0; q < kMxPer; ++q) {
        if (!in[q]) continue;
        F *o = reinterpret_cast<F *>(a.x + at[q].row * a.ldx) + at[q].span * kMxSpan + 8 * l;
        const u32x4 b = mx_numbers(c[q], s[q]);
        if constexpr (sizeof(F) == 2) {
            *reinterpret_cast<u32x4 *>(o) = b;
        } else {
            float v[8];
#pragma unroll
            for (int x = 0; x < 4; ++x) unpack_bf16(b[x], v[2 * x], v[2 * x + 1]);
            *reinterpret_cast<floatx4 *>(o) = floatx4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<floatx4 *>(o + 4) = floatx4{v[4], v[5], v[6], v[7]};
        }
    }
}

// A tile whose M side is codes and whose N side is bf16, K in steps of 128, for batches
// that neither the MFMA nor memory bounds: what counts is that copies, reads,
// conversions and MFMAs of different steps overlap, since a SIMD has one or two waves.
// A stage holds the N rows' 256 bytes and the M rows' 64.  The M rows' scales come 32
// steps at a time (128 bytes a row, into one of two buffers): a copy of four bytes a
// row every step would look up as many lines as all the rest.  A lane's 16 bytes of codes
// are one block of 32 (its own scale), operands of four MFMAs; the N side is read in the
// same order of K.  The four waves are two halves of the M rows by two halves of every
// block, each wave over all 64 tokens, so that a code is converted once; the halves of K
// are added up at the end.  256 tokens by 6144 columns over 4096 without adapters: 28 us,
// where waves that share M rows and convert them each for itself took 33.  In a form that
// took 31 the copies alone were 18, everything but the copies 27, but the MFMAs 23; six
// stages, one workgroup a CU, 47.
template <class B>
struct MixedTile : B {
    static constexpr int kStepK = 128, kNBytes = B::BN * 256, kMBytes = B::BM * 64;
    static constexpr int kMAt = kNBytes, kStage = kNBytes + kMBytes;
    static constexpr int kScaleSteps = 32, kScaleBytes = B::BM * 4 * kScaleSteps, kScaleCopies = kScaleBytes / 256 / B::kWaves;
    static constexpr int kScaleAt = B::kStages * kStage, kLds = kScaleAt + 2 * kScaleBytes;
    static constexpr int kNInstr = B::BN / 4 / B::kWaves, kLoads = kNInstr + 1, kTokens = B::BN / 16;
    static_assert(B::BM == 64 && B::DEAL == 2 && B::MT == 2 && B::WM == 2 && B::WN == 2 && kTokens == 2 * B::NT, "two by two waves");
    typedef floatx4 Sums[B::MT][kTokens];   // of a wave's half of K, all tokens
    // half of a step's K that a wave multiplies: codes 16 g .. of every block
    __device__ __forceinline__ static int half() { return wave_id() / B::WM; }

    // tile row in place p of the M side: tile by tile, so that a tile's 16 rows are together
    __device__ __forceinline__ static int m_row(int p) {
        const int l16 = p & 15, t = p >> 4;
        return 32 * (t >> 1) + 8 * (l16 >> 2) + 4 * (t & 1) + (l16 & 3);
    }
    // copies: row and 16-byte chunk of this lane (N: of instruction j)
    __device__ __forceinline__ static int n_copy_row(int j) { return (wave_id() * kNInstr + j) * 4 + lane_id() / 16; }
    __device__ __forceinline__ static int n_copy_chunk(int j) { return (lane_id() & 15) ^ (n_copy_row(j) & 15); }
    __device__ __forceinline__ static int m_copy_row() { return m_row(wave_id() * 16 + lane_id() / 4); }
    __device__ __forceinline__ static int m_copy_chunk() { return (lane_id() & 3) ^ (lane_id() >> 3 & 3); }   // (place / 2) & 3
    // scales: place and step (of 32) that a lane copies with instruction i; a place's
    // dwords are turned by its number, so that 16 rows' bytes of a step are in 16 banks
    __device__ __forceinline__ static int scale_copy_place(int i) { return (wave_id() * kScaleCopies + i) * 2 + lane_id() / 32; }
    __device__ __forceinline__ static int scale_copy_step(int i) { return (lane_id() - scale_copy_place(i)) & 31; }

    struct Step {
        u32x2g codes[B::MT];
        uint32_t scale[B::MT];
        bf16x8 n[kTokens][2];
    };
    // Where a lane reads: its first tile's codes and scales (the second tile's are 16 places
    // on), its tokens' chunks of either j, in a stage and in the scales.
    struct Places {
        uint32_t codes, scales, n[2];
        __device__ __forceinline__ void find() {
            const uint32_t l16 = lane_id() & 15, g = lane_id() >> 4, place = 32 * B::wave_m() + l16;
            codes = kMAt + place * 64 + 16 * (g ^ (l16 >> 1 & 3)) + 8 * half();
            scales = kScaleAt + place * 128 + g;
#pragma unroll
            for (int j = 0; j < 2; ++j) n[j] = l16 * 256 + 16 * ((4 * g + 2 * half() + j) ^ l16);
        }
    };
    // of the stage at byte `cur`, step s of K
    __device__ __forceinline__ static void read(Step &r, const Places &p, const lds_byte *lds, uint32_t cur, uint32_t s) {
        const uint32_t turned = ((s + (lane_id() & 15)) & 31) * 4;
        const lds_byte *scale = lds + p.scales + (s / kScaleSteps & 1) * kScaleBytes;
#pragma unroll
        for (int t = 0; t < B::MT; ++t) {
            r.codes[t] = *(const __attribute__((address_space(3))) u32x2g *)(lds + cur + p.codes + t * 1024);
            r.scale[t] = *(scale + t * 2048 + (turned ^ 64u * t));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int t = 0; t < kTokens; ++t) r.n[t][j] = *(const lds_bf16x8 *)(lds + cur + p.n[j] + t * 4096);
    }
    // keep: 0 where the lane's block is past the last (its scale may be anything, its codes are zeros)
    __device__ __forceinline__ static void mma(const Step &r, Sums &sums, uint32_t keep) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int m = 0; m < B::MT; ++m) {
                const bf16x8 w = as_bf16x8(mx_numbers(r.codes[m][j], r.scale[m] & keep));
#pragma unroll
                for (int t = 0; t < kTokens; ++t) sums[m][t] = mfma16x16x32(w, r.n[t][j], sums[m][t]);
            }
    }
    // Both halves of K added up: a wave keeps the tokens of the tile's own layout and hands
    // the others to the wave that has the same rows (a 16 KB of `lds`, which no one reads).
    __device__ __forceinline__ static void join(const Sums &sums, typename B::Acc &acc, unsigned char *lds) {
        floatx4 *at = reinterpret_cast<floatx4 *>(lds) + lane_id();
        const int mine = half(), wave = wave_id(), partner = wave ^ B::WM;
#pragma unroll
        for (int m = 0; m < B::MT; ++m)
#pragma unroll
            for (int t = 0; t < B::NT; ++t)
                at[((wave * B::MT + m) * B::NT + t) * kWave] = mine ? sums[m][t] : sums[m][B::NT + t];
        __syncthreads();
#pragma unroll
        for (int m = 0; m < B::MT; ++m)
#pragma unroll
            for (int t = 0; t < B::NT; ++t)
                acc[m][t] = (mine ? sums[m][B::NT + t] : sums[m][t]) + at[((partner * B::MT + m) * B::NT + t) * kWave];
        __syncthreads();
    }
};

// The two sides' walk: lanes past the end of K read zeros.
template <class T>
struct MixedWalk {
    const uint16_t *nbase, *mbase;      // of the next step: the tokens' and the tile's W rows
    uint32_t n[T::kNInstr], m;          // this lane's places from there, bytes
    const uint8_t *scales;              // row 0 of W
    int64_t ldscales;
    int m0, cols;               // first row of the tile, rows of W
    int k, blocks, step;        // of the rows; next step to copy
    // the scales of 32 steps; past the last dword any of the row's
    __device__ __forceinline__ void copy_scales(uint32_t base, int group) {
#pragma unroll
        for (int i = 0; i < T::kScaleCopies; ++i) {
            const int d = min(group * T::kScaleSteps + T::scale_copy_step(i), (blocks - 1) / 4);
            const int row = min(m0 + T::m_row(T::scale_copy_place(i)), cols - 1);
            dma4(scales + row * ldscales + 4 * (int64_t)d,
                 base + T::kScaleAt + (group & 1) * T::kScaleBytes + (wave_id() * T::kScaleCopies + i) * 256u);
        }
    }
    __device__ __forceinline__ void issue(uint32_t at) {
        const uint32_t to = at + wave_id() * T::kNInstr * 1024u, mto = at + T::kMAt + wave_id() * 1024u;
        if ((step + 1) * T::kStepK <= k) {
#pragma unroll
            for (int j = 0; j < T::kNInstr; ++j) dma16(nbase, n[j], to + j * 1024u);
            dma16(mbase, m, mto);
        } else {
#pragma unroll
            for (int j = 0; j < T::kNInstr; ++j)
                dma16(step * T::kStepK + 8 * T::n_copy_chunk(j) < k ? nbase + n[j] / 2 : zero_page, to + j * 1024u);
            dma16(step * 4 + T::m_copy_chunk() < blocks ? mbase + m / 2 : zero_page, mto);
        }
        nbase += T::kStepK;
        mbase += 32;
        ++step;
    }
};

template <class T>
__device__ __forceinline__ void mixed_begin(MixedWalk<T> &w, int nsteps, unsigned char *lds) {
    const uint32_t base = lds_address(lds);
    w.copy_scales(base, 0);
    for (int i = 0; i < T::kStages && i < nsteps; ++i) w.issue(base + i * T::kStage);
}
// A step's operands are read while the step before is multiplied.  One barrier a step:
// every wave has read the step before, whose stage takes the copies of kStages steps on.
// At the end nothing is in flight and every wave is done with the stages.
template <class T>
__device__ __forceinline__ void mixed_loop(MixedWalk<T> &w, int nsteps, typename T::Acc &acc, unsigned char *lds_generic) {
    constexpr int S = T::kStages;
    const lds_byte *lds = (const lds_byte *)lds_generic;
    const uint32_t base = lds_address(lds_generic);
    int cur = 0, s = 0;       // stage and number of the step to be read next
    typename T::Sums sums;
#pragma unroll
    for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int t = 0; t < T::kTokens; ++t) sums[m][t] = floatx4{0.f, 0.f, 0.f, 0.f};
    typename T::Places places;
    places.find();
    auto read = [&](typename T::Step &r) {
        T::read(r, places, lds, cur, s);
        cur = cur + T::kStage == T::kScaleAt ? 0 : cur + T::kStage;
        ++s;
    };
    // reads step s while step s - 1 is multiplied
    auto turn = [&](typename T::Step &next, const typename T::Step &now) {
        const bool more = s < nsteps;
        const uint32_t keep = (s - 1) * 4 + lane_id() / 16 < w.blocks ? 0xffu : 0u;
        // the step before is in its registers: said in a way that the compiler knows, or it
        // would wait for the reads below before it multiplies
        __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
        if (more) {
            const int before = (cur == 0 ? T::kScaleAt : cur) - T::kStage;
            if (s + S - 1 <= nsteps)
                wait_loads_barrier<(S - 2) * T::kLoads>();
            else
                wait_loads_barrier<0>();
            // the scales of the 32 steps after the next 32 are asked for once the 32 before have
            // left their buffer; ahead of the step's copies, so that the next wait covers them
            if ((s & (T::kScaleSteps - 1)) == 1 && s + T::kScaleSteps - 1 < nsteps) w.copy_scales(base, s / T::kScaleSteps + 1);
            if (s - 1 + S < nsteps) w.issue(base + before);
            read(next);
        }
        T::mma(now, sums, keep);
        return more;
    };
    typename T::Step a, b;
    if (S <= nsteps)      // the first step has landed
        wait_loads_barrier<(S - 1) * T::kLoads>();
    else
        wait_loads_barrier<0>();
    read(a);
    while (turn(b, a) && turn(a, b)) {
    }
    __syncthreads();
    T::join(sums, acc, lds_generic);
}

}  // namespace lora
