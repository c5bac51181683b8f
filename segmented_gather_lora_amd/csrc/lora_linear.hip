// lora_linear.hip -- a projection that every request shares with the adapters
// of many requests added in the same product, and its backward pass:
//
//   y[t]   = W x[t] + b_w  + (slice i's columns)  B_i[m] s_i[t] + bias_i[m]     m = id_t
//   u_i[t] = scale * B_i[m]^T dy_i[t]
//   dx[t]  = W^T dy[t] + sum_i A_i[m]^T u_i[t]
//   dA_i[m] = sum_{t of m} u_i[t] x[t]^T,  dB_i[m] = sum dy_i[t] s_i[t]^T,  dbias_i[m] = sum dy_i[t]
//
// with s_i[t] = scale * A_i[m] x[t] from the shrink kernels.
//
// The two large products run over the batch in the stable order sorted by id,
// which the prepared metadata holds: a tile of tokens then meets few adapters
// (its share of the batch plus one), and each of them is a continuation of the
// tile's K walk: after W's columns come the ranks of every (adapter, slice)
// the tile meets, each multiplied into its own tokens' rows alone.  The
// sums stay in the MFMA accumulators, so y and dx are rounded once and are
// written once; no pass over y adds the adapters afterwards.
//
// s and u are fp32.  They enter the products as two bf16 parts, hi and
// lo = rne(v - hi) (to 2^-16 of the value together), side by side as 2 r
// K elements; a single bf16 part would add an error as large as the result's
// own rounding, and the ranks are a small share of the work.  hi is the largest
// bf16 below v in magnitude, so that lo has v's sign and is not zero: an infinite
// weight times either part is the infinity that it is times v (a nearest hi leaves
// remainders of 0 or of the other sign, and infinity less infinity).
//
// A packed row (one token, one slice) is made of blocks of 32 ranks, [32 hi |
// 32 lo] each, or of a single block [16 hi | 16 lo] for ranks up to 16; ranks
// past the last are zeros.
#include <string.h>

#include <type_traits>

#include "lora_gemm.h"

namespace lora {
namespace {

extern __shared__ __attribute__((aligned(1024))) unsigned char g_lds[];

// ---------------------------------------------------------------- workspace

// Segment of each LoRA id, and the token tiles of the u product.
struct SegEntry {
    int32_t start, count;
};
struct UTile {
    int32_t id, start, rows, pad;   // sorted positions [start, start + rows)
};

// ---------------------------------------------------------------- pack

__host__ __device__ __forceinline__ int packed_half(int rank) { return rank <= 16 ? 16 : 32; }
__host__ __device__ __forceinline__ int packed_row(int rank) {
    const int h = packed_half(rank);
    return (rank + h - 1) / h * 2 * h;
}
// element of the hi part of rank j; its lo part is packed_half elements on
__device__ __forceinline__ int packed_at(int j, int half) { return j / half * 2 * half + j % half; }

struct PackArgs {
    MetaView meta;
    const int32_t *ids;
    const float *buf;
    uint16_t *packed;
    SegEntry *segs;       // NULL: no tables
    UTile *tiles;
    int32_t *num_tiles;
    int32_t *counters;    // of the u product's split K (kCounterWords of them)
    int32_t num_tokens, rank, slices, max_loras, tile_tokens, tiles_cap;
};
constexpr int kCounterWords = 1024;   // at least the units of the u product whose K may be split (kSplitUnits / 2)

constexpr int kPackThreads = 256;

__device__ __forceinline__ void split_hi_lo(float v, uint32_t &h, uint32_t &l) {
    const uint32_t bits = __float_as_uint(v), mag = bits & 0x7fffffffu;
    if (mag >= 0x7f800000u) {   // inf and NaN: both parts
        h = l = float_to_bf16_bits(v);
    } else {
        h = (bits - (mag != 0u)) >> 16;   // one less in magnitude, cut off
        l = float_to_bf16_bits(v - bf16_bits_to_float(h));
    }
}

// buf's rows in sorted order as packed rows, bound by its launch and bytes (13 us
// for 16384 tokens, 3 slices of rank 128);
// workgroup 0 also writes the tables when they are asked for, and sets the u
// product's counters to zero.
__global__ __launch_bounds__(kPackThreads) void pack_kernel(PackArgs a) {
    const bool none = *a.meta.no_lora != 0;
    const int tid = threadIdx.x;
    if (a.segs && blockIdx.x == 0) {
        __shared__ int s_wsum[kPackThreads / kWave];
        for (int k = tid; k < kCounterWords; k += kPackThreads) a.counters[k] = 0;
        for (int m = tid; m < a.max_loras; m += kPackThreads) a.segs[m] = SegEntry{0, 0};
        __syncthreads();
        constexpr int kPer = (LORA_MAX_LORAS + 1 + kPackThreads - 1) / kPackThreads;
        int id[kPer], st[kPer], cnt[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int k = tid * kPer + i;
            id[i] = -1;
            st[i] = cnt[i] = 0;
            if (!none && k < a.meta.nslots) {
                id[i] = a.meta.active_ids[k];
                st[i] = a.meta.start_loc[k];
                cnt[i] = a.meta.counts[k];
            }
            const bool ok = id[i] >= 0 && id[i] < a.max_loras && st[i] >= 0 && cnt[i] > 0 && st[i] + cnt[i] <= a.num_tokens;
            if (!ok) id[i] = -1, cnt[i] = 0;
            if (ok) a.segs[id[i]] = SegEntry{st[i], cnt[i]};
            sum += (cnt[i] + a.tile_tokens - 1) / a.tile_tokens;
        }
        const int incl = wave_inclusive_scan(sum);
        if (lane_id() == kWave - 1) s_wsum[tid / kWave] = incl;
        __syncthreads();
        int at = incl - sum, total = 0;
        for (int w = 0; w < kPackThreads / kWave; ++w) {
            at += w < tid / kWave ? s_wsum[w] : 0;
            total += s_wsum[w];
        }
        if (tid == 0) *a.num_tiles = total < a.tiles_cap ? total : a.tiles_cap;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            for (int o = 0; o < cnt[i]; o += a.tile_tokens, ++at)
                if (at < a.tiles_cap) a.tiles[at] = UTile{id[i], st[i] + o, min(a.tile_tokens, cnt[i] - o), 0};
    }
    if (none) return;
    const int half = packed_half(a.rank), row_len = packed_row(a.rank), per_row = row_len / 8;
    const int64_t work = (int64_t)a.slices * a.num_tokens * per_row;
    for (int64_t w = (int64_t)blockIdx.x * kPackThreads + tid; w < work; w += (int64_t)gridDim.x * kPackThreads) {
        const int q = (int)(w % per_row);             // 4 ranks
        const int64_t row = w / per_row;              // slice * n + position
        const int p = (int)(row % a.num_tokens);
        const int64_t slice = row / a.num_tokens;
        const int t = a.meta.sorted[p];
        if ((unsigned)t >= (unsigned)a.num_tokens || a.ids[t] < 0) continue;
        floatx4 v = {0.f, 0.f, 0.f, 0.f};
        if (4 * q < a.rank) v = *reinterpret_cast<const floatx4 *>(a.buf + (slice * a.num_tokens + t) * a.rank + 4 * q);
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_hi_lo(v[e], h[e], l[e]);
        uint16_t *out = a.packed + row * row_len + packed_at(4 * q, half);
        *reinterpret_cast<u32x2g *>(out) = u32x2g{h[0] | h[1] << 16, h[2] | h[3] << 16};
        *reinterpret_cast<u32x2g *>(out + half) = u32x2g{l[0] | l[1] << 16, l[2] | l[3] << 16};
    }
}

// ---------------------------------------------------------------- y and dx

struct LinearArgs {
    MetaView meta;
    const int32_t *ids;
    const uint16_t *in;                         // x (forward) or dy (backward), one row per token
    int64_t ldin;
    const uint16_t *w;                          // [out][hidden]
    int64_t ldw;
    const uint16_t *w_bias;
    const uint16_t *lw[LORA_MAX_SLICES];        // B_i (forward) or A_i (backward)
    const uint16_t *bias[LORA_MAX_SLICES];
    int32_t width[LORA_MAX_SLICES], col[LORA_MAX_SLICES];
    const uint16_t *packed;                     // s or u: [slices][n][packed_row]
    const float *s;                             // the same in fp32: [slices][n][rank], batch order
    uint16_t *y;                                // y or dx
    int64_t ldy;
    int32_t num_tokens, cols, k, rank, slices, max_loras;
    int32_t mtiles, ntiles, group, has_bias, row_len;   // row_len: packed_row(rank)
};

// The adapters' share of a tile's K walk is made of units, for every slice that
// meets the tile and every adapter (slices outermost: their arguments are read
// once).  For ranks above 16 a unit is one step: a block of 32 ranks of the
// packed rows, whose hi part is the step's first half and whose lo part the
// second; both are multiplied with the same 32 ranks of the adapter's matrix,
// staged once.  Up to 16 ranks a unit is half a step, [16 hi | 16 lo] against
// the ranks twice, so that a step holds two adapters.
//
// What a unit needs of the two tables in LDS is read a unit ahead and made
// scalar where it is used, so that a unit does not wait for it.
struct SliceEntry {
    uint32_t weights[2];   // the adapters' matrices of the slice
    int32_t width, col;
};
struct SegRow {
    int32_t lo, hi, id;    // rows of the tile, LoRA id
};
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <class T, bool BWD>
struct LinearOp : PlainOp<T> {
    static constexpr int kLast = T::MSide::kInstr / 2;
    const LinearArgs &a;
    const SegRow *segs;        // LDS
    const SliceEntry *slices;  // LDS
    int main_left, main_steps, m0, p0, nseg;
    int sl0, sl1, blocks;      // slices that meet the tile; blocks of 32 ranks (0: ranks up to 16)
    int sl, e, kb;             // next unit to copy
    int me, mleft, munits;     // next unit to multiply: its adapter, that adapter's units left, all units left
    SliceEntry slice;          // of the next unit to copy
    SegRow seg;
    int mlo, mhi;              // rows of the next unit to multiply

    __device__ __forceinline__ LinearOp(const LinearArgs &args, const SegRow *g, const SliceEntry *s)
        : a(args), segs(g), slices(s) {}
    __device__ __forceinline__ int per_seg() const { return blocks ? blocks : 1; }
    __device__ __forceinline__ void start(int units) {
        munits = units;
        sl = sl0;
        e = me = kb = 0;
        mleft = per_seg();
        slice = slices[sl];
        seg = segs[0];
        mlo = seg.lo;
        mhi = seg.hi;
    }
    __device__ __forceinline__ void read(typename T::Half &r, const lds_byte *st, int, int h) { T::read(r, st, h); }
    __device__ __forceinline__ void read(typename T::Half &r, const lds_byte *st, int s, int h, const typename T::Half &first) {
        T::read_n(r, st, h);
        // a block's lo part meets the same ranks as its hi part
        const int hm = s < main_steps || blocks == 0 ? h : 0;
        if (&r != &first || hm == h) T::read_m(r, st, hm);
    }
    // an adapter's units touch its own tokens' sums alone: one whose weights
    // are not finite stays without effect on the others in the tile
    // (W's last steps go the same way with all rows: a branch here would cost the
    // registers of a second set of sums)
    __device__ __forceinline__ void mma(const typename T::Half &h, typename T::Acc &acc, int s, int half) {
        const bool all = s < main_steps;
        mma_rows<T>(h, acc, all ? 0 : scalar(mlo), all ? T::BN : munits > 0 ? scalar(mhi) : 0);
        if (!all && (half == 1 || blocks == 0)) {
            --munits;
            if (--mleft == 0) {
                mleft = per_seg();
                if (++me == nseg) me = 0;
                mlo = segs[me].lo;
                mhi = segs[me].hi;
            }
        }
    }
    __device__ __forceinline__ void next() {
        PlainOp<T>::next();
        --main_left;
    }
    // copies of a unit: N rows of its adapter's tokens (other rows keep what the
    // stage holds: their products are not added), then the ranks of its matrix.
    // H: the half of the step that it fills, or -1 for both.  Lane offsets are 32
    // bits from scalar bases; only a tile across a slice's edge and a block with
    // ranks past the last take the checked way.  Those ranks are zeros on both
    // sides: another rank's weight, which may be infinite, times zero would be NaN.
    template <int H>
    __device__ __forceinline__ void unit(uint32_t at) {
        const int r = a.rank, row_len = a.row_len;
        const bool live = sl < sl1;      // past the last unit: no rows, and ranks that are not used
        const int lo = scalar(seg.lo), count = live ? scalar(seg.hi) - lo : 0;
        const int width = scalar(slice.width), col = scalar(slice.col);
        const uint64_t base = (uint32_t)scalar((int)slice.weights[0]) | (uint64_t)(uint32_t)scalar((int)slice.weights[1]) << 32;
        const uint16_t *lw =
            reinterpret_cast<const uint16_t *>(base) + (uint64_t)(uint32_t)(scalar(seg.id) * r) * (uint32_t)width;
        const uint16_t *rows = a.packed + (uint64_t)(uint32_t)((live ? sl : sl0) * a.num_tokens + p0) * (uint32_t)row_len + kb * 64;
#pragma unroll
        for (int j = 0; j < T::NSide::kInstr; ++j) {
            const int row = T::NSide::row(j), ko = T::NSide::elem(j);
            if ((unsigned)(row - lo) < (unsigned)count && (H < 0 || ko / 32 == H))
                dma16(rows, 2u * (uint32_t)(__umul24(row, row_len) + (H < 0 ? ko : ko & 31)),
                      at + T::MSide::kBytes + T::NSide::dst(j));
        }
        const bool full = H < 0 ? kb * 32 + 32 <= r : r == 16;
        if (BWD) {      // A_i: ranks are K rows, this side's index is the hidden column
            // half of the side's instructions hold the half's 32 K rows
            constexpr int kHalf = T::MSide::kInstr / 2, kRows = 64 / T::MSide::kLanesPerK;
            const uint16_t *block = lw + (uint64_t)(uint32_t)(H < 0 ? kb * 32 : 0) * (uint32_t)width;
            const int ranks = r - (H < 0 ? kb * 32 : 0);
#pragma unroll
            for (int j = 0; j < kHalf; ++j) {
                const int i = wave_id() * kHalf + j + (H > 0 ? T::kWaves * kHalf : 0);
                const int k = i * kRows + lane_id() / T::MSide::kLanesPerK;
                const int rank = H < 0 ? k : k & 15;
                const int c = min(m0 + T::MSide::elem_of(k), width - 8);
                const uint32_t offset = 2u * (uint32_t)(rank * width + c);
                if (full)
                    dma16(block, offset, at + i * 1024u);
                else
                    dma16(rank < ranks ? block + offset / 2 : zero_page, at + i * 1024u);
            }
        } else {        // B_i: rows are the slice's columns, ranks contiguous
            const bool inside = full && m0 >= col && m0 + T::BM <= col + width;
            const uint16_t *block = lw + (int64_t)(m0 - col) * r + (H < 0 ? kb * 32 : 0);
#pragma unroll
            for (int j = 0; j < T::MSide::kInstr; ++j) {
                const int row = T::MSide::row(j), ko = T::MSide::elem(j);
                const int rank = H < 0 ? ko : ko & 15;
                if (ko / 32 == (H > 0 ? 1 : 0)) {
                    if (inside) {
                        dma16(block, 2u * (uint32_t)(__umul24(row, r) + rank), at + T::MSide::dst(j));
                    } else {
                        const int c = m0 + row - col, ranks = r - (H < 0 ? kb * 32 : 0);
                        dma16(c >= 0 && c < width && rank < ranks ? block + row * r + rank : zero_page, at + T::MSide::dst(j));
                    }
                }
            }
        }
        if (live && ++kb == per_seg()) {
            kb = 0;
            if (++e == nseg) {
                e = 0;
                if (++sl < sl1) slice = slices[sl];
            }
            seg = segs[e];
        }
    }
    __device__ __forceinline__ void issue(uint32_t at) {
        if (main_left > 0) {
            PlainOp<T>::issue(at);
            --main_left;
        } else if (blocks) {
            unit<-1>(at);
        } else {
            unit<0>(at);
            unit<1>(at);
        }
    }
};

// The adapters' share of a 64 x 64 tile as fp32 dot products, a lane for its
// token and 16 of the tile's columns, in place of a step of the K walk for every 32
// ranks, adapter and slice.  us with the products and with the steps, for so many
// adapters in each tile:
//   y   gains from four on, at every rank (64 tokens by 1024 over 1024): 2: 31, 25;
//       4: 31, 33; 8: 31, 50 (rank 128); 4: 18, 18; 8: 18, 21 (rank 16)
//   dx  waits for a row of A a rank and gains from 7 to 24 on (whole backward pass):
//       12: 39, 40; 20: 39, 44 (rank 16); 12: 61, 59; 20: 62, 75 (rank 64); 16: 198,
//       233 (3 slices of rank 128); 20: 135, 120; 32: 144, 155 (256 tokens by 2048
//       over 4096, rank 64)
template <bool BWD>
constexpr int kDotSegs = BWD ? 20 : 4;
template <class T, bool BWD>
__device__ __forceinline__ void add_dots(const LinearArgs &a, const SliceEntry *slices, int m0, int t, int id,
                                         typename T::Acc &acc) {
    static_assert(T::NT == 1 && T::MT == 4, "one token a lane");
    const int r = a.rank;
    auto matrices = [&](int i) {
        return reinterpret_cast<const uint16_t *>(slices[i].weights[0] | (uint64_t)slices[i].weights[1] << 32);
    };
    if (BWD) {
        for (int i = 0; i < a.slices; ++i) {
            const uint16_t *w = matrices(i) + (int64_t)id * r * a.cols;
            const float *s = a.s + ((int64_t)i * a.num_tokens + t) * r;
#pragma unroll 4
            for (int j = 0; j < r; ++j, w += a.cols) {
                const float sj = s[j];
#pragma unroll
                for (int mt = 0; mt < T::MT; ++mt) {
                    const int c = min(m0 + T::m_of(mt), a.cols - 4);
                    const u32x2g v = *reinterpret_cast<const u32x2g *>(w + c);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float p, q;
                        unpack_bf16(v[x], p, q);
                        acc[mt][0][2 * x] = fmaf(p, sj, acc[mt][0][2 * x]);
                        acc[mt][0][2 * x + 1] = fmaf(q, sj, acc[mt][0][2 * x + 1]);
                    }
                }
            }
        }
    } else {
#pragma unroll
        for (int mt = 0; mt < T::MT; mt += 2) {      // 8 columns, never across a slice's edge
            const int c = m0 + T::m_of(mt);
            for (int i = 0; i < a.slices; ++i) {
                const int in = c - slices[i].col, width = slices[i].width;
                if (in < 0 || in >= width) continue;
                const uint16_t *b = matrices(i) + ((int64_t)id * width + in) * r;
                const float *s = a.s + ((int64_t)i * a.num_tokens + t) * r;
                float sum[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) sum[x] = 0.f;
                for (int j = 0; j < r; j += 8) {
                    const floatx4 s0 = *reinterpret_cast<const floatx4 *>(s + j), s1 = *reinterpret_cast<const floatx4 *>(s + j + 4);
                    u32x4 v[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) v[x] = *reinterpret_cast<const u32x4 *>(b + x * r + j);
#pragma unroll
                    for (int x = 0; x < 8; ++x)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float p, q;
                            unpack_bf16(v[x][k], p, q);
                            sum[x] = fmaf(p, k < 2 ? s0[2 * k] : s1[2 * k - 4], sum[x]);
                            sum[x] = fmaf(q, k < 2 ? s0[2 * k + 1] : s1[2 * k - 3], sum[x]);
                        }
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) acc[mt + x / 4][0][x % 4] += sum[x];
            }
        }
    }
}

// A tile of y or dx.  16384 tokens, 128 adapters of rank 128: y (10240 columns
// over 8192) 2.4 ms, dx (8192 over 10240, three slices) 3.1 ms, of which W's
// product is about 2.0 ms each; the rest are the adapters' steps, each a barrier
// pair and a trip to memory for 32 ranks.  4096 tokens by 28672 over 4096, 16
// adapters of rank 32: y 0.81 ms, dx 0.67 ms (1.19 and 1.43 PFLOP/s of W's product).
template <class T, bool BWD>
__global__ __launch_bounds__(T::kThreads, 2) void linear_kernel(LinearArgs a) {
    __shared__ int s_tok[T::BN], s_id[T::BN], s_count;
    __shared__ SegRow s_seg[T::BN];
    __shared__ SliceEntry s_slice[LORA_MAX_SLICES];
    static_assert(T::BN <= T::kThreads, "a thread a token row");
    constexpr bool kDots = T::BM == 64 && T::BN == 64;
    const int tid = threadIdx.x;
    TileAt at;
    if (!tile_at(blockIdx.x, a.mtiles, a.ntiles, a.group, at)) return;
    const int m0 = at.m * T::BM, p0 = at.n * T::BN;
    const int rows = min(T::BN, a.num_tokens - p0);
    if (tid == 0) s_count = 0;

    // one memory round trip: the flag, the tile's tokens, the first segments
    // (a batch without adapters has no sorted order: batch order)
    const bool none = *a.meta.no_lora != 0;
    auto token = [&](int r) {
        const int p = p0 + min(r, rows - 1), at = a.meta.sorted[p];   // (read whatever the flag says: no second trip)
        const int t = none ? p : at;
        return (unsigned)t < (unsigned)a.num_tokens ? t : 0;
    };
    const int own = token(min(tid, T::BN - 1));
    int id = -1, st = 0, count = 0;
    if (tid < a.meta.nslots) {
        id = a.meta.active_ids[tid];
        st = a.meta.start_loc[tid];
        count = a.meta.counts[tid];
    }
    LinearOp<T, BWD> op(a, s_seg, s_slice);
    op.m0 = m0;
    op.p0 = p0;
    op.blocks = a.rank <= 16 ? 0 : (a.rank + 31) / 32;
#pragma unroll
    for (int j = 0; j < T::NSide::kInstr; ++j)
        op.wn.p[j] = a.in + (int64_t)token(T::NSide::row(j)) * a.ldin + T::NSide::elem(j);
    op.wn.step = kStepK;
    op.wn.left = a.k;
#pragma unroll
    for (int j = 0; j < T::MSide::kInstr; ++j) {
        if (BWD) {
            const int c = m0 + T::MSide::elem(j);
            op.wm.p[j] = a.w + (int64_t)T::MSide::row(j) * a.ldw + (c < a.cols ? c : a.cols - 8);
        } else {
            op.wm.p[j] = a.w + (int64_t)min(m0 + T::MSide::row(j), a.cols - 1) * a.ldw + T::MSide::elem(j);
        }
    }
    op.wm.step = BWD ? (int64_t)kStepK * a.ldw : kStepK;
    op.wm.left = a.k;
    const int main = (a.k + kStepK - 1) / kStepK;
    op.main_left = op.main_steps = main;
    const bool early = main >= kAhead<T>;
    if (early) mma_begin<T>(op, main, g_lds);

    // while they land: the tile's tokens and ids, and the adapters it meets
    // (any order: each token takes part in one of them)
    __syncthreads();
#pragma unroll
    for (int i = 0; i < LORA_MAX_SLICES; ++i)
        if (tid == i) {
            const uint64_t w = reinterpret_cast<uint64_t>(a.lw[i]);
            s_slice[i] = SliceEntry{{(uint32_t)w, (uint32_t)(w >> 32)}, BWD ? a.cols : a.width[i], BWD ? 0 : a.col[i]};
        }
    if (tid < T::BN) {
        s_tok[tid] = own;
        s_id[tid] = none || (!kDots && (BWD || !a.has_bias)) ? -1 : a.ids[own];
    }
    if (!none)
        for (int k = tid; k < a.meta.nslots; k += T::kThreads) {
            if (k != tid) {
                id = a.meta.active_ids[k];
                st = a.meta.start_loc[k];
                count = a.meta.counts[k];
            }
            const int lo = max(st, p0), hi = min(st + count, p0 + rows);
            if (id >= 0 && id < a.max_loras && lo < hi) {
                const int e = atomicAdd(&s_count, 1);
                if (e < T::BN) s_seg[e] = SegRow{lo - p0, hi - p0, id};
            }
        }
    __syncthreads();
    const int nseg = __builtin_amdgcn_readfirstlane(min(s_count, T::BN));
    op.nseg = nseg;
    op.sl0 = 0;
    op.sl1 = a.slices;
    if (!BWD) {   // the slices that meet the tile's columns
        op.sl0 = a.slices;
        op.sl1 = 0;
#pragma unroll
        for (int i = 0; i < LORA_MAX_SLICES; ++i)
            if (i < a.slices && a.col[i] < m0 + T::BM && a.col[i] + a.width[i] > m0) {
                op.sl0 = min(op.sl0, i);
                op.sl1 = i + 1;
            }
    }
    const bool dots = kDots && nseg >= kDotSegs<BWD>;
    const int units = op.sl1 > op.sl0 && !dots ? nseg * (op.sl1 - op.sl0) * op.per_seg() : 0;
    const int steps = main + (op.blocks ? units : (units + 1) / 2);
    if (units > 0) op.start(units);
    if (!early) mma_begin<T>(op, steps, g_lds);
    typename T::Acc acc;
    clear<T>(acc);
    mma_loop<T>(op, a.k / kStepK, steps, acc, g_lds);

    if constexpr (kDots)
        if (dots) {
            const int row = T::n_of(0), m = s_id[row];
            if (row < rows && m >= 0 && m < a.max_loras) add_dots<T, BWD>(a, s_slice, m0, s_tok[row], m, acc);
        }

    // biases: of the projection for every token, of the adapter where there is one
    if constexpr (T::QUADS) {
        // groups of 8 consecutive columns (never across a slice's edge); a group's loads are issued together
#pragma unroll
        for (int mt = 0; mt < T::MT; mt += 2) {
            const int c = m0 + T::m_of(mt);
            if (c >= a.cols) continue;
            float wb[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) wb[x] = 0.f;
            if (a.w_bias) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(a.w_bias + c);
#pragma unroll
                for (int x = 0; x < 4; ++x) unpack_bf16(v[x], wb[2 * x], wb[2 * x + 1]);
            }
            const uint16_t *bp = nullptr;
            int bw = 0;
            if (a.has_bias)
                for (int i = op.sl0; i < op.sl1; ++i) {
                    const int ci = select_slice(a.col, i), wi = select_slice(a.width, i);
                    const uint16_t *bi = select_slice(a.bias, i);
                    if (bi && c >= ci && c < ci + wi) {
                        bp = bi + (c - ci);
                        bw = wi;
                    }
                }
            u32x4 b[T::NT];
            if (a.has_bias)
#pragma unroll
                for (int nt = 0; nt < T::NT; ++nt) {
                    const int m = s_id[T::n_of(nt)];
                    b[nt] = u32x4{0u, 0u, 0u, 0u};
                    if (bp && m >= 0) b[nt] = *reinterpret_cast<const u32x4 *>(bp + (int64_t)m * bw);
                }
#pragma unroll
            for (int nt = 0; nt < T::NT; ++nt) {
                const int r = T::n_of(nt);
                float v[8];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    v[x] = acc[mt][nt][x] + wb[x];
                    v[4 + x] = acc[mt + 1][nt][x] + wb[4 + x];
                }
                if (a.has_bias)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        float p, q;
                        unpack_bf16(b[nt][x], p, q);
                        v[2 * x] += p;
                        v[2 * x + 1] += q;
                    }
                if (r < rows)
                    *reinterpret_cast<u32x4 *>(a.y + (int64_t)s_tok[r] * a.ldy + c) =
                        u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
            }
        }
    } else {
        // backward: no biases; 4 consecutive columns
#pragma unroll
        for (int nt = 0; nt < T::NT; ++nt) {
            const int r = T::n_of(nt);
            if (r >= rows) continue;
            uint16_t *row = a.y + (int64_t)s_tok[r] * a.ldy;
#pragma unroll
            for (int mt = 0; mt < T::MT; ++mt) {
                const int c = m0 + T::m_of(mt);
                const floatx4 v = acc[mt][nt];
                if (c < a.cols) *reinterpret_cast<u32x2g *>(row + c) = u32x2g{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            }
        }
    }
}

// ---------------------------------------------------------------- few tokens

// Up to 32 tokens: a call is one pass over W and the adapters, bound by their
// bytes and by latency, so it is two launches without a sort or a split over
// workgroups.  s: 16 ranks of one token and slice a workgroup, 4 lanes a rank.
// Batches of up to kRowsShrinks such workgroups that read up to kRowsBytes of
// adapters (once a token) take s from the same kernel, packed too: the shrink
// kernels, which read an adapter once for all of its tokens, need three launches
// (zeroing, shrink, pack) for that.  us of lora_linear this way and that, 4 and 32
// adapters: 64 MB (512 tokens, rank 16 over 4096) 29, 36 and 32, 36; 96 MB (256
// tokens, 3 slices) 34, 36 and 42, 37; 2048 workgroups (2048 tokens, rank 16 over
// 264) 20, 23 and 21, 25; 3000 (1000 tokens, 3 slices) 24, 23 and 26, 23.
struct RowsArgs {
    const int32_t *ids, *no_lora;   // a batch without adapters has no ids
    const uint16_t *x;
    int64_t ldx;
    const uint16_t *w;
    int64_t ldw;
    const uint16_t *w_bias;
    const uint16_t *la[LORA_MAX_SLICES], *lb[LORA_MAX_SLICES], *bias[LORA_MAX_SLICES];
    int32_t width[LORA_MAX_SLICES], col[LORA_MAX_SLICES];
    float *buf;
    const int32_t *sorted;       // with packed: tokens in sorted order
    uint16_t *packed;            // NULL: s in buf alone, tokens in batch order
    uint16_t *y;
    int64_t ldy;
    int32_t num_tokens, cols, k, rank, slices, max_loras, row_len;
    float scale;
};
constexpr long kRowsShrinks = 2048, kRowsBytes = 64L << 20;
constexpr int kRowsTokens = 32, kRowsWaves = 16, kRowsCols = 32, kRowsThreads = kRowsWaves * kWave;
constexpr int kRowsRanks = 16, kRowsShrinkWaves = 16;

__device__ __forceinline__ void fma_bf16x8(const u32x4 &a, const u32x4 &b, float &sum) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        float a0, a1, b0, b1;
        unpack_bf16(a[x], a0, a1);
        unpack_bf16(b[x], b0, b1);
        sum = fmaf(a0, b0, sum);
        sum = fmaf(a1, b1, sum);
    }
}

__global__ __launch_bounds__(kRowsShrinkWaves *kWave) void rows_shrink_kernel(RowsArgs a) {
    __shared__ float s_part[kRowsShrinkWaves][kRowsRanks];
    const int per = a.packed ? a.row_len / (2 * kRowsRanks) : (a.rank + kRowsRanks - 1) / kRowsRanks;
    const int p = blockIdx.x / (per * a.slices), i = blockIdx.x / per % a.slices, r0 = blockIdx.x % per * kRowsRanks;
    const int none = *a.no_lora, st = a.packed ? a.sorted[p] : p;
    const int t = (unsigned)st < (unsigned)a.num_tokens ? st : 0, id = a.ids[t];
    if (none || id < 0 || id >= a.max_loras) return;
    const int rank = min(r0 + (lane_id() >> 2), a.rank - 1), first = (wave_id() * 4 + (lane_id() & 3)) * 8;
    const uint16_t *row = select_slice(a.la, i) + ((int64_t)id * a.rank + rank) * a.k, *x = a.x + t * a.ldx;
    constexpr int kStride = kRowsShrinkWaves * 32;
    float sum = 0.f;
#pragma unroll 8
    for (int k = first; k < a.k; k += kStride)
        fma_bf16x8(*reinterpret_cast<const u32x4 *>(row + k), *reinterpret_cast<const u32x4 *>(x + k), sum);
    sum += __shfl_xor(sum, 1);
    sum += __shfl_xor(sum, 2);
    if ((lane_id() & 3) == 0) s_part[wave_id()][lane_id() >> 2] = sum;
    __syncthreads();
    if (threadIdx.x < kRowsRanks) {
        const int j = r0 + (int)threadIdx.x;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kRowsShrinkWaves; ++w) v += s_part[w][threadIdx.x];
        v = j < a.rank ? a.scale * v : 0.f;
        if (j < a.rank) a.buf[((int64_t)i * a.num_tokens + t) * a.rank + j] = v;
        if (a.packed) {
            const int half = packed_half(a.rank);
            uint16_t *out = a.packed + ((int64_t)i * a.num_tokens + p) * a.row_len + packed_at(j, half);
            uint32_t h, l;
            split_hi_lo(v, h, l);
            out[0] = (uint16_t)h;
            out[half] = (uint16_t)l;
        }
    }
}

// y: 32 columns a workgroup; its 16 waves share K, every operand goes from
// memory straight into the registers of the MFMA, and the waves' sums are added
// in wave order through LDS.  A thread adds its column's and token's adapter as
// a float32 dot product, whose loads travel with the first of W's.
// One token by 6144 columns over 4096: 13.8 us, W at 3.6 TB/s (a kernel that reads
// its 50 MB and does nothing else takes 8.6 us).
template <int NT>
__global__ __launch_bounds__(kRowsThreads) void rows_kernel(RowsArgs a) {
    constexpr int kOut = kRowsCols * 16 * NT, kPer = kOut > kRowsThreads ? kOut / kRowsThreads : 1;
    __shared__ float s_sum[kRowsWaves][16 * NT][kRowsCols];   // column c of token t in slot c ^ t: 64 banks
    const int tid = threadIdx.x, l16 = lane_id() & 15, g = lane_id() >> 4, c0 = blockIdx.x * kRowsCols;
    const uint16_t *wp[2], *xp[NT];
#pragma unroll
    for (int m = 0; m < 2; ++m) wp[m] = a.w + (int64_t)min(c0 + 16 * m + l16, a.cols - 1) * a.ldw;
#pragma unroll
    for (int t = 0; t < NT; ++t) xp[t] = a.x + (int64_t)min(16 * t + l16, a.num_tokens - 1) * a.ldx;
    floatx4 acc[2][NT];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = floatx4{0.f, 0.f, 0.f, 0.f};

    // the wave's K: chunks of 32 elements wave, wave + 16, ..., four at a time
    constexpr int kChunk = 4, kStride = kRowsWaves * 32;
    u32x4 wv[kChunk][2], xv[kChunk][NT];
    auto load = [&](int k0) {
#pragma unroll
        for (int q = 0; q < kChunk; ++q) {
            const int k = k0 + q * kStride + 8 * g;
            const bool in = k < a.k;
#pragma unroll
            for (int m = 0; m < 2; ++m) wv[q][m] = in ? *reinterpret_cast<const u32x4 *>(wp[m] + k) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int t = 0; t < NT; ++t) xv[q][t] = in ? *reinterpret_cast<const u32x4 *>(xp[t] + k) : u32x4{0u, 0u, 0u, 0u};
        }
    };
    int k0 = wave_id() * 32;
    load(k0);

    float add[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int o = tid + q * kRowsThreads, c = c0 + o % kRowsCols, t = o / kRowsCols;
        add[q] = 0.f;
        if (t >= a.num_tokens || c >= a.cols) continue;
        const int none = *a.no_lora, id = a.ids[t];
        if (a.w_bias) add[q] = bf16_bits_to_float(a.w_bias[c]);
        if (none || id < 0 || id >= a.max_loras) continue;
        for (int i = 0; i < a.slices; ++i) {
            const int in = c - select_slice(a.col, i), width = select_slice(a.width, i);
            if (in < 0 || in >= width) continue;
            const uint16_t *b = select_slice(a.lb, i) + ((int64_t)id * width + in) * a.rank;
            const float *s = a.buf + ((int64_t)i * a.num_tokens + t) * a.rank;
            float dot = 0.f;
            for (int j = 0; j < a.rank; j += 8) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(b + j);
                const floatx4 s0 = *reinterpret_cast<const floatx4 *>(s + j), s1 = *reinterpret_cast<const floatx4 *>(s + j + 4);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float b0, b1;
                    unpack_bf16(v[x], b0, b1);
                    dot = fmaf(b0, x < 2 ? s0[2 * x] : s1[2 * x - 4], dot);
                    dot = fmaf(b1, x < 2 ? s0[2 * x + 1] : s1[2 * x - 3], dot);
                }
            }
            const uint16_t *bias = select_slice(a.bias, i);
            if (bias) dot += bf16_bits_to_float(bias[(int64_t)id * width + in]);
            add[q] += dot;
        }
    }

    for (;;) {
#pragma unroll
        for (int q = 0; q < kChunk; ++q)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[m][t] = mfma16x16x32(as_bf16x8(wv[q][m]), as_bf16x8(xv[q][t]), acc[m][t]);
        k0 += kChunk * kStride;
        if (k0 >= a.k) break;
        load(k0);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) s_sum[wave_id()][16 * t + l16][(16 * m + 4 * g + x) ^ (16 * t + l16)] = acc[m][t][x];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int o = tid + q * kRowsThreads, c = o % kRowsCols, t = o / kRowsCols;
        if (o >= kOut || t >= a.num_tokens || c0 + c >= a.cols) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kRowsWaves; ++w) v += s_sum[w][t][c ^ t];
        a.y[t * a.ldy + c0 + c] = (uint16_t)float_to_bf16_bits(v + add[q]);
    }
}

// ---------------------------------------------------------------- u

struct UArgs {
    const UTile *tiles;
    const int32_t *num_tiles;
    const int32_t *sorted;
    const uint16_t *dy;
    int64_t lddy;
    const uint16_t *b[LORA_MAX_SLICES];
    int32_t width[LORA_MAX_SLICES], col[LORA_MAX_SLICES];
    float *dbuf;
    uint16_t *packed;
    float *slots;
    int32_t *counters;
    int32_t num_tokens, rank, slices, splits;
    float scale;
};

// u_i[t] = scale * B_i[m]^T dy_i[t] for one tile of a segment's tokens and one
// slice: K is the slice's width, all ranks are in the tile.  Bound by dy's and
// B's bytes: 16384 tokens, 10240 columns, rank 128: 184 us for 670 MB.  Few tiles
// split K (joined by the last to arrive) to fill the CUs.
template <class T>
__global__ __launch_bounds__(T::kThreads) void u_kernel(UArgs a) {
    __shared__ int s_tok[T::BN], s_flag;
    const int split = blockIdx.x % a.splits, unit = blockIdx.x / a.splits;
    const int tile = unit / a.slices, i = unit % a.slices;
    if (tile >= *a.num_tiles) return;
    const UTile ut = a.tiles[tile];
    for (int r = threadIdx.x; r < T::BN; r += T::kThreads) {
        const int t = a.sorted[ut.start + min(r, ut.rows - 1)];
        s_tok[r] = (unsigned)t < (unsigned)a.num_tokens ? t : 0;
    }
    __syncthreads();
    const int width = select_slice(a.width, i), col = select_slice(a.col, i);
    const uint16_t *b = select_slice(a.b, i) + (int64_t)ut.id * width * a.rank;
    const int all = (width + kStepK - 1) / kStepK, per = (all + a.splits - 1) / a.splits;
    const int s0 = min(all, split * per), s1 = min(all, s0 + per);
    PlainOp<T> op;
#pragma unroll
    for (int j = 0; j < T::NSide::kInstr; ++j)
        op.wn.p[j] = a.dy + (int64_t)s_tok[T::NSide::row(j)] * a.lddy + col + s0 * kStepK + T::NSide::elem(j);
    op.wn.step = kStepK;
    op.wn.left = width - s0 * kStepK;
#pragma unroll
    for (int j = 0; j < T::MSide::kInstr; ++j) {
        const int c = min(T::MSide::elem(j), a.rank - 8);
        op.wm.p[j] = b + (int64_t)(s0 * kStepK + T::MSide::row(j)) * a.rank + c;
    }
    op.wm.step = (int64_t)kStepK * a.rank;
    op.wm.left = width - s0 * kStepK;
    typename T::Acc acc;
    clear<T>(acc);
    mma_begin<T>(op, s1 - s0, g_lds);
    mma_loop<T>(op, min(s1, width / kStepK) - s0, s1 - s0, acc, g_lds);
    if (a.splits > 1 && !combine_splits<T>(acc, a.slots + (int64_t)unit * a.splits * (T::BM * T::BN), a.counters + unit,
                                           split, a.splits, ut.rows, &s_flag))
        return;
    const int half = packed_half(a.rank), row_ranks = packed_row(a.rank) / 2;
#pragma unroll
    for (int nt = 0; nt < T::NT; ++nt) {
        const int r = T::n_of(nt);
        if (r >= ut.rows) continue;
        float *out = a.dbuf + ((int64_t)i * a.num_tokens + s_tok[r]) * a.rank;
        uint16_t *pk = a.packed + ((int64_t)i * a.num_tokens + ut.start + r) * packed_row(a.rank);
#pragma unroll
        for (int mt = 0; mt < T::MT; ++mt) {
            const int j = T::m_of(mt);
            if (j >= row_ranks) continue;
            const floatx4 v = j < a.rank ? acc[mt][nt] * a.scale : floatx4{0.f, 0.f, 0.f, 0.f};
            if (j < a.rank) *reinterpret_cast<floatx4 *>(out + j) = v;
            uint32_t h[4], l[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) split_hi_lo(v[x], h[x], l[x]);
            uint16_t *at = pk + packed_at(j, half);
            *reinterpret_cast<u32x2g *>(at) = u32x2g{h[0] | h[1] << 16, h[2] | h[3] << 16};
            *reinterpret_cast<u32x2g *>(at + half) = u32x2g{l[0] | l[1] << 16, l[2] | l[3] << 16};
        }
    }
}

// ---------------------------------------------------------------- dA, dB, dbias

struct GradArgs {
    const SegEntry *segs;
    const int32_t *sorted;
    const uint16_t *act;                      // x (dA) or dy (dB), gathered token rows
    int64_t ldact;
    const uint16_t *packed;                   // u (dA) or s (dB): [slices][n][packed_row]
    uint16_t *out[LORA_MAX_SLICES];           // dA_i [id][r][hidden] or dB_i [id][width][r]
    uint16_t *dbias[LORA_MAX_SLICES];
    int32_t width[LORA_MAX_SLICES], col[LORA_MAX_SLICES];   // of act (dA: hidden, 0)
    int32_t runs_before[LORA_MAX_SLICES + 1], run_tiles;
    int32_t num_tokens, rank, slices;
};

// dA_i[m] (DA: M side = x columns, N side = u's hi and lo parts) or dB_i[m]
// (M side = s's hi and lo parts, N side = dy columns) over one segment's
// tokens, one tile of the activation's columns.  An id without tokens gets
// zeros: every adapter's gradient is written.  128 adapters of 100 tokens, rank
// 128: dA (3 slices over 8192, 805 MB written) 423 us, dB (335 MB) 217 us.
template <class T, bool DA>
struct GradOp {
    using ASide = typename std::conditional<DA, typename T::MSide, typename T::NSide>::type;   // activations
    using PSide = typename std::conditional<DA, typename T::NSide, typename T::MSide>::type;   // packed ranks
    static constexpr int kLast = T::MSide::kInstr;
    GatherWalk<ASide> wa;
    Walk<PSide> wp;
    floatx4 colsum[DA ? 1 : T::NT];
    bool sums;
    __device__ __forceinline__ void issue(uint32_t at) {
        if (DA) {
            wp.issue(at + T::MSide::kBytes);
            wa.issue(at);
        } else {
            wa.issue(at + T::MSide::kBytes);
            wp.issue(at);
        }
    }
    __device__ __forceinline__ void load(uint32_t at, int i) {
        constexpr int nm = T::MSide::kInstr;
        const uint32_t to = i < nm ? at : at + T::MSide::kBytes;
        const int j = i < nm ? i : i - nm;
        if ((i < nm) == DA)
            wa.load(to, j);
        else
            wp.load(to, j);
    }
    __device__ __forceinline__ void next() {
        wa.next();
        wp.next();
    }
    __device__ __forceinline__ void read(typename T::Half &r, const lds_byte *st, int, int h) { T::read(r, st, h); }
    __device__ __forceinline__ void read(typename T::Half &r, const lds_byte *st, int, int h, const typename T::Half &) {
        T::read(r, st, h);
    }
    // dB: the column sums of dy as one more MFMA row of ones
    __device__ __forceinline__ void mma_n(const typename T::Half &h, typename T::Acc &acc, int nt) {
        T::mma_n(h, acc, nt);
        if constexpr (!DA) {
            const bf16x8 ones = as_bf16x8(u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
            if (sums) colsum[nt] = mfma16x16x32(ones, h.n[nt], colsum[nt]);
        }
    }
    __device__ __forceinline__ void mma(const typename T::Half &h, typename T::Acc &acc, int, int) {
#pragma unroll
        for (int nt = 0; nt < T::NT; ++nt) mma_n(h, acc, nt);
    }
};

// The tile's results (and dbias) to memory.
template <class T, bool DA>
__device__ __forceinline__ void grad_store(const typename T::Acc &acc, const floatx4 *colsum, uint16_t *out, uint16_t *dbias,
                                           int m, int c0, int width, int r) {
#pragma unroll
    for (int nt = 0; nt < T::NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < T::MT; ++mt) {
            const floatx4 v = acc[mt][nt];
            const int j = DA ? T::n_of(nt) : T::m_of(mt), c = c0 + (DA ? T::m_of(mt) : T::n_of(nt));
            if (j >= r || c >= width) continue;
            uint16_t *at = out + (DA ? ((int64_t)m * r + j) * width + c : ((int64_t)m * width + c) * r + j);
            *reinterpret_cast<u32x2g *>(at) = u32x2g{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        }
    if constexpr (!DA) {
        if (dbias && T::wave_m() == 0 && lane_id() < 16)
#pragma unroll
            for (int nt = 0; nt < T::NT; ++nt) {
                const int c = c0 + T::n_of(nt);
                if (c < width) dbias[(int64_t)m * width + c] = (uint16_t)float_to_bf16_bits(colsum[nt][0]);
            }
    }
}

// An adapter of at most 128 tokens: its packed rows (two K steps at most) stay
// in LDS for the whole run, and only the activations' columns change from tile
// to tile; they are asked for as soon as the tile before is read.
template <class T, bool DA>
__device__ __forceinline__ void short_run(const GradArgs &a, const SegEntry &sg, int m, int i, int begin, int end, int width,
                                          int col, uint16_t *out, uint16_t *dbias) {
    using Op = GradOp<T, DA>;
    using ASide = typename Op::ASide;
    using PSide = typename Op::PSide;
    constexpr int BA = DA ? T::BM : T::BN, BR = DA ? T::BN : T::BM;
    const int r = a.rank, half = packed_half(r), row_len = packed_row(r), steps = (sg.count + kStepK - 1) / kStepK;
    const lds_byte *lds = (const lds_byte *)g_lds;
    const uint32_t base = lds_address(g_lds);
    // LDS: the packed rows of both steps, then the activations of both (of one step: of two tiles)
    constexpr uint32_t kActs = 2 * PSide::kBytes;
    const uint16_t *row[2][ASide::kInstr];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int j = 0; j < ASide::kInstr; ++j) {
            const int k = b * kStepK + ASide::row(j);
            const int t = a.sorted[sg.start + min(k, sg.count - 1)];
            row[b][j] = k < sg.count && (unsigned)t < (unsigned)a.num_tokens ? a.act + (int64_t)t * a.ldact + col : nullptr;
        }
    auto copy = [&](int c0, int b, uint32_t to) {
#pragma unroll
        for (int j = 0; j < ASide::kInstr; ++j) {
            const uint16_t *p = b ? row[1][j] : row[0][j];
            dma16(p ? p + min(c0 + ASide::elem(j), width - 8) : zero_page, to + ASide::dst(j));
        }
    };
    for (int b = 0; b < steps; ++b)
#pragma unroll
        for (int j = 0; j < PSide::kInstr; ++j) {
            const int c = PSide::elem(j), k = b * kStepK + PSide::row(j);
            const int from = c < BR ? packed_at(min(c, r - 8), half) : packed_at(min(c - BR, r - 8), half) + half;
            dma16(k < sg.count ? a.packed + ((int64_t)i * a.num_tokens + sg.start + k) * row_len + from : zero_page,
                  base + b * PSide::kBytes + PSide::dst(j));
        }
    const int ahead = steps == 1 ? 2 : 1;    // tiles in LDS
    for (int t = 0; t < ahead; ++t)
        for (int b = 0; b < steps; ++b)
            if (begin + t * BA < end) copy(begin + t * BA, b, base + kActs + (t + b) * ASide::kBytes);
    int slot = 0;
    for (int c0 = begin; c0 < end; c0 += BA) {
        typename T::Acc acc;
        clear<T>(acc);
        Op op;
        op.sums = !DA && dbias && T::wave_m() == 0;
#pragma unroll
        for (int nt = 0; nt < (DA ? 1 : T::NT); ++nt) op.colsum[nt] = floatx4{0.f, 0.f, 0.f, 0.f};
        wait_loads_barrier<0>();
        for (int b = 0; b < steps; ++b) {
            const lds_byte *packed = lds + b * PSide::kBytes, *acts = lds + kActs + (slot + b) * ASide::kBytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                typename T::Half x;
                T::read_m(x, DA ? acts : packed, h);
                T::read_n(x, (DA ? packed : acts) - T::MSide::kBytes, h);
                op.mma(x, acc, b, h);
            }
        }
        own_reads_barrier();
        if (c0 + ahead * BA < end)
            for (int b = 0; b < steps; ++b) copy(c0 + ahead * BA, b, base + kActs + (slot + b) * ASide::kBytes);
        slot ^= steps == 1;
        grad_store<T, DA>(acc, op.colsum, out, dbias, m, c0, width, r);
    }
}

template <class T, bool DA>
__global__ __launch_bounds__(T::kThreads, 2) void grad_kernel(GradArgs a) {
    using Op = GradOp<T, DA>;
    using ASide = typename Op::ASide;
    using PSide = typename Op::PSide;
    static_assert(T::kStages == 2, "mma_loop ends with every wave's reads done");
    constexpr int BA = DA ? T::BM : T::BN, BR = DA ? T::BN : T::BM;   // activation columns, ranks
    const int per_id = a.runs_before[a.slices];
    const int m = blockIdx.x / per_id, run = blockIdx.x % per_id;
    int i = 0;
    while (i + 1 < a.slices && run >= a.runs_before[i + 1]) ++i;
    const int width = select_slice(a.width, i), col = select_slice(a.col, i), r = a.rank;
    const int begin = (run - select_slice(a.runs_before, i)) * a.run_tiles * BA, end = min(width, begin + a.run_tiles * BA);
    const SegEntry sg = a.segs[m];
    const int steps = (sg.count + kStepK - 1) / kStepK;
    uint16_t *out = select_slice(a.out, i), *dbias = DA ? nullptr : select_slice(a.dbias, i);
    if (sg.count > 0 && steps <= 2) {
        short_run<T, DA>(a, sg, m, i, begin, end, width, col, out, dbias);
        return;
    }
    const int half = packed_half(r), row_len = packed_row(r);
    for (int c0 = begin; c0 < end; c0 += BA) {
        Op op;
        typename T::Acc acc;
        clear<T>(acc);
        op.sums = !DA && dbias && T::wave_m() == 0;
#pragma unroll
        for (int nt = 0; nt < (DA ? 1 : T::NT); ++nt) op.colsum[nt] = floatx4{0.f, 0.f, 0.f, 0.f};
        if (sg.count > 0) {
            op.wa.base = a.act + col;
            op.wa.sorted = a.sorted;
            op.wa.ld = a.ldact;
            op.wa.pos = sg.start;
            op.wa.end = sg.start + sg.count;
            op.wa.num_tokens = a.num_tokens;
#pragma unroll
            for (int j = 0; j < ASide::kInstr; ++j) op.wa.col[j] = min(c0 + ASide::elem(j), width - 8);
            op.wa.fetch();
#pragma unroll
            for (int j = 0; j < PSide::kInstr; ++j) {
                const int c = PSide::elem(j);
                const int from = c < BR ? packed_at(min(c, r - 8), half) : packed_at(min(c - BR, r - 8), half) + half;
                op.wp.p[j] = a.packed + ((int64_t)i * a.num_tokens + sg.start + PSide::row(j)) * row_len + from;
            }
            op.wp.step = (int64_t)kStepK * row_len;
            op.wp.left = sg.count;
            mma_begin<T>(op, steps, g_lds);
            mma_loop<T>(op, sg.count / kStepK, steps, acc, g_lds);
        }
        grad_store<T, DA>(acc, op.colsum, out, dbias, m, c0, width, r);
    }
}

// ---------------------------------------------------------------- plans

constexpr size_t kRound = 256;
size_t up(size_t v) { return (v + kRound - 1) / kRound * kRound; }
long ceil_div(long a, long b) { return (a + b - 1) / b; }

enum LinearTile { kBig, kMid, kSmall };
struct LinearPlan {
    LinearTile tile;
    int mtiles, ntiles;
};

// The tile of y or dx (n x cols): the largest of 256 x 256, 128 x 128 and 64 x 64
// of which there are enough for the GPU's 256 CUs (one of the first a CU at a time,
// two of the others).  The limits lie where batches of few adapters and of many,
// which the host cannot tell apart, part.  us of lora_linear over 4096, larger tile
// and smaller, one adapter of rank 16 first:
//   256 x 256, 128 x 128
//     128 tiles (2048 by 4096): 106, 89;  32 adapters of rank 16: 112, 91
//     160 (2048 by 5120): 112, 120;  128 adapters of rank 64, 3 slices: 366, 263
//     192 (2048 by 6144): 116, 123;  200 (1100 by 10240), 32 of rank 64: 157, 156
//   128 x 128, 64 x 64
//     160 tiles (256 by 10240): 52, 56;  32 adapters of rank 16: 72, 61
//     192 (129 by 12288): 51, 55;  32 adapters: 87, 57
//     224 (256 by 14336): 54, 67;  8 adapters of rank 64: 77, 96
//     240 (520 by 6144): 59, 73;  32 adapters of rank 16: 68, 76
// 64 columns x 128 tokens is slower than one of its neighbours at every size (192
// of the last two lists: 65, and 118 with 32 adapters).  K is not split: joining
// fp32 partial tiles across XCDs took 22 of the 70 us of a product of 256 tokens by
// 6144 columns over 4096.
LinearPlan plan_linear(long n, long cols) {
    auto tiles = [&](long bm, long bn) { return ceil_div(cols, bm) * ceil_div(n, bn); };
    LinearPlan p;
    long bm = 64, bn = 64;
    p.tile = kSmall;
    if (n > 128 && tiles(256, 256) >= 192) {
        p.tile = kBig;
        bm = bn = 256;
    } else if (tiles(128, 128) >= 224) {
        p.tile = kMid;
        bm = bn = 128;
    }
    p.mtiles = (int)ceil_div(cols, bm);
    p.ntiles = (int)ceil_div(n, bn);
    return p;
}

struct UPlan {
    int bm, tile_tokens, tiles_cap, splits;
    size_t slot_bytes;
};
constexpr long kSplitUnits = 768, kMaxSplits = 8;   // workgroups that a split K is to give
static_assert(kSplitUnits / 2 <= kCounterWords, "a counter for each unit whose K is split");
UPlan plan_u(long n, int max_loras, int slices, int rank, long widest) {
    UPlan p;
    p.bm = rank <= 32 ? 32 : rank <= 64 ? 64 : 128;
    p.tile_tokens = 64;
    const long segs = n < max_loras ? n : max_loras;
    p.tiles_cap = (int)(ceil_div(n, p.tile_tokens) + segs);
    const long units = (long)p.tiles_cap * slices;
    const long steps = ceil_div(widest, kStepK);
    const long most = steps / 8 < kMaxSplits ? steps / 8 : kMaxSplits;
    long splits = kSplitUnits / (units > 0 ? units : 1);
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
    p.splits = (int)splits;
    // room for every smaller batch too, which may split more: `units` grows with n,
    // and units * splits is at most kSplitUnits where K is split at all
    const long slots = units * most < kSplitUnits ? units * most : kSplitUnits;
    p.slot_bytes = most > 1 ? sizeof(float) * (size_t)slots * p.bm * p.tile_tokens : 0;
    return p;
}

struct Layout {
    size_t counters, segs, num_tiles, tiles, s, u, slots, total;
};
Layout layout(long n, int max_loras, int slices, int rank, const UPlan &u, bool backward) {
    Layout l;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up(bytes);
        return o;
    };
    l.counters = take(sizeof(int32_t) * kCounterWords);
    l.segs = take(backward ? sizeof(SegEntry) * (size_t)max_loras : 0);
    l.num_tiles = take(backward ? sizeof(int32_t) : 0);
    l.tiles = take(backward ? sizeof(UTile) * (size_t)u.tiles_cap : 0);
    const size_t rows = sizeof(uint16_t) * (size_t)slices * (size_t)n * (size_t)packed_row(rank);
    l.s = take(rows);
    l.u = take(backward ? rows : 0);
    l.slots = take(backward ? u.slot_bytes : 0);
    l.total = at;
    return l;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_sizes(int num_tokens, int max_loras, int hidden, const int *slice_widths, int num_slices, int rank) {
    if (num_tokens < 0 || num_tokens > LORA_MAX_TOKENS) return LORA_ERR_NUM_TOKENS;
    if (max_loras < 1 || max_loras > LORA_MAX_LORAS) return LORA_ERR_MAX_LORAS;
    if (num_slices < 1 || num_slices > LORA_MAX_SLICES) return LORA_ERR_SLICES;
    if (!slice_widths) return LORA_ERR_NULL;
    if (hidden < 8 || hidden % 8 || hidden > LORA_MAX_HIDDEN) return LORA_ERR_SHAPE;
    if (rank < 8 || rank > LORA_MAX_RANK || rank % 8) return LORA_ERR_SHAPE;
    for (int i = 0; i < num_slices; ++i)
        if (slice_widths[i] <= 0 || slice_widths[i] % 8) return LORA_ERR_SHAPE;
    return LORA_OK;
}

// Everything the forward and the backward pass check alike.
int check_call(int64_t ldx, int num_tokens, int hidden, const void *w, int64_t ldw, int out, const void *const *lora_a,
               const void *const *lora_b, const int *slice_widths, int num_slices, int rank, int64_t ldy,
               int offset_start, const lora_meta_t *meta, const void *workspace) {
    int st = check_meta(meta);
    if (st) return st;
    if (meta->num_tokens < 0 || num_tokens != meta->num_tokens) return LORA_ERR_NUM_TOKENS;
    if ((st = check_sizes(num_tokens, meta->max_loras, hidden, slice_widths, num_slices, rank))) return st;
    if (!w || !lora_a || !lora_b || !workspace) return LORA_ERR_NULL;
    if (ldx < hidden || ldx % 8 || ldw < hidden || ldw % 8 || out < 8 || out % 8 || ldy < out || ldy % 8)
        return LORA_ERR_SHAPE;
    if (offset_start < 0 || offset_start % 8) return LORA_ERR_SHAPE;
    int64_t end = offset_start;
    for (int i = 0; i < num_slices; ++i) {
        end += slice_widths[i];
        if (!lora_a[i] || !lora_b[i]) return LORA_ERR_NULL;
        if (!aligned16(lora_a[i]) || !aligned16(lora_b[i])) return LORA_ERR_ALIGN;
    }
    if (end > out) return LORA_ERR_SHAPE;
    if (!aligned16(w)) return LORA_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(workspace) & (kRound - 1)) != 0) return LORA_ERR_BUFFER;
    return LORA_OK;
}

int widest(const int *w, int n) {
    int s = 0;
    for (int i = 0; i < n; ++i) s = w[i] > s ? w[i] : s;
    return s;
}

hipError_t launch_pack(const lora_meta_t *meta, const MetaView &view, const float *buf, uint16_t *packed, int slices,
                       int rank, char *ws, const Layout *l, const UPlan *u, hipStream_t s) {
    PackArgs a;
    memset(&a, 0, sizeof a);
    a.meta = view;
    a.ids = meta->token_lora_mapping;
    a.buf = buf;
    a.packed = packed;
    if (l) {
        a.segs = reinterpret_cast<SegEntry *>(ws + l->segs);
        a.tiles = reinterpret_cast<UTile *>(ws + l->tiles);
        a.num_tiles = reinterpret_cast<int32_t *>(ws + l->num_tiles);
        a.counters = reinterpret_cast<int32_t *>(ws + l->counters);
        a.tiles_cap = u->tiles_cap;
        a.tile_tokens = u->tile_tokens;
    }
    a.num_tokens = meta->num_tokens;
    a.rank = rank;
    a.slices = slices;
    a.max_loras = meta->max_loras;
    const long work = (long)slices * meta->num_tokens * (packed_row(rank) / 8);
    long grid = ceil_div(work, kPackThreads);
    if (grid > 2048) grid = 2048;
    if (grid < 1) grid = 1;
    hipLaunchKernelGGL(pack_kernel, dim3((unsigned)grid), dim3(kPackThreads), 0, s, a);
    return hipGetLastError();
}

template <bool BWD>
hipError_t launch_linear(LinearArgs &a, hipStream_t s) {
    const LinearPlan p = plan_linear(a.num_tokens, a.cols);
    a.mtiles = p.mtiles;
    a.ntiles = p.ntiles;
    a.group = 8;
    a.row_len = packed_row(a.rank);
    const unsigned grid = tile_grid((long)p.mtiles * p.ntiles);
    auto launch = [&](auto tile) {
        using T = decltype(tile);
        return launch_tiles<linear_kernel<T, BWD>>(grid, T::kThreads, T::kLds, s, a);
    };
    switch (p.tile) {
        case kBig: return launch(Tile<256, 256, 4, 2, BWD, false>{});
        case kMid: return launch(Tile<128, 128, 2, 2, BWD, false>{});
        default: return launch(Tile<64, 64, 1, 4, BWD, false, 0, 4>{});
    }
}

template <int BR>
hipError_t launch_u(const UArgs &a, const UPlan &p, hipStream_t s) {
    using T = Tile<BR, 64, (BR == 32 ? 1 : 2), (BR == 32 ? 4 : 2), true, false>;
    return launch_tiles<u_kernel<T>>((unsigned)((long)p.tiles_cap * a.slices * p.splits), T::kThreads, T::kLds, s, a);
}

template <int BR, bool DA>
hipError_t launch_grad(GradArgs &a, int max_loras, hipStream_t s) {
    // 128 columns of the activations; 64 where more would leave room for one workgroup a CU
    constexpr int BA = BR == 128 ? 64 : 128;
    using T = typename std::conditional<DA, Tile<BA, BR, (BR == 16 ? 4 : 2), (BR == 16 ? 1 : 2), true, true, 2>,
                                        Tile<BR, BA, (BR == 16 ? 1 : 2), (BR == 16 ? 4 : 2), true, true, 1>>::type;
    long tiles = 0;
    for (int i = 0; i < a.slices; ++i) tiles += ceil_div(a.width[i], BA);
    // runs of up to 16 tiles while eight workgroups a CU remain
    const long run = tiles * max_loras / 2048;
    a.run_tiles = (int)(run < 1 ? 1 : run > 16 ? 16 : run);
    a.runs_before[0] = 0;
    for (int i = 0; i < a.slices; ++i)
        a.runs_before[i + 1] = a.runs_before[i] + (int)ceil_div(a.width[i], (long)BA * a.run_tiles);
    const long grid = (long)max_loras * a.runs_before[a.slices];
    return launch_tiles<grad_kernel<T, DA>>((unsigned)grid, T::kThreads, T::kLds, s, a);
}
template <bool DA>
hipError_t launch_grads(GradArgs &a, int max_loras, hipStream_t s) {
    if (a.rank <= 16) return launch_grad<16, DA>(a, max_loras, s);
    if (a.rank <= 32) return launch_grad<32, DA>(a, max_loras, s);
    if (a.rank <= 64) return launch_grad<64, DA>(a, max_loras, s);
    return launch_grad<128, DA>(a, max_loras, s);
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t lora_linear_workspace_bytes(int num_tokens, int max_loras, int hidden, const int *slice_widths, int num_slices,
                                   int rank, int backward) {
    if (check_sizes(num_tokens, max_loras, hidden, slice_widths, num_slices, rank)) return 0;
    const long n = num_tokens;
    const UPlan u = plan_u(n, max_loras, num_slices, rank, widest(slice_widths, num_slices));
    return layout(n, max_loras, num_slices, rank, u, backward != 0).total;
}

int lora_linear(const void *x, int64_t ldx, int num_tokens, int hidden, const void *w, int64_t ldw, int out_features,
                const void *w_bias, const void *const *lora_a, const void *const *lora_b, const void *const *bias,
                const int *slice_widths, int num_slices, int rank, float *buf, void *y, int64_t ldy, int offset_start,
                const lora_meta_t *meta, float scale, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    int st = check_call(ldx, num_tokens, hidden, w, ldw, out_features, lora_a, lora_b, slice_widths, num_slices, rank,
                        ldy, offset_start, meta, workspace);
    if (st) return st;
    if (w_bias && !aligned16(w_bias)) return LORA_ERR_ALIGN;
    for (int i = 0; bias && i < num_slices; ++i)
        if (bias[i] && !aligned16(bias[i])) return LORA_ERR_ALIGN;
    if (num_tokens > 0 && (!x || !buf || !y)) return LORA_ERR_NULL;
    if (num_tokens > 0 && (!aligned16(x) || !aligned16(buf) || !aligned16(y))) return LORA_ERR_ALIGN;
    const UPlan u = plan_u(num_tokens, meta->max_loras, num_slices, rank, widest(slice_widths, num_slices));
    const Layout l = layout(num_tokens, meta->max_loras, num_slices, rank, u, false);
    if (l.total > workspace_bytes) return LORA_ERR_BUFFER;
    if (num_tokens == 0) return LORA_OK;
    char *ws = static_cast<char *>(workspace);
    const MetaView view = view_of(meta);
    uint16_t *packed = reinterpret_cast<uint16_t *>(ws + l.s);
    const bool few = num_tokens <= kRowsTokens;
    const long shrinks = (long)num_tokens * num_slices * (few ? ceil_div(rank, kRowsRanks) : packed_row(rank) / (2 * kRowsRanks));
    if (few || (shrinks <= kRowsShrinks && (long)num_tokens * num_slices * rank * hidden * 2 <= kRowsBytes)) {
        RowsArgs r;
        memset(&r, 0, sizeof r);
        r.ids = meta->token_lora_mapping;
        r.no_lora = view.no_lora;
        r.x = static_cast<const uint16_t *>(x);
        r.ldx = ldx;
        r.w = static_cast<const uint16_t *>(w);
        r.ldw = ldw;
        r.w_bias = static_cast<const uint16_t *>(w_bias);
        for (int i = 0, off = offset_start; i < num_slices; off += slice_widths[i++]) {
            r.la[i] = static_cast<const uint16_t *>(lora_a[i]);
            r.lb[i] = static_cast<const uint16_t *>(lora_b[i]);
            r.bias[i] = bias ? static_cast<const uint16_t *>(bias[i]) : nullptr;
            r.width[i] = slice_widths[i];
            r.col[i] = off;
        }
        r.buf = buf;
        r.sorted = view.sorted;
        r.packed = few ? nullptr : packed;
        r.row_len = packed_row(rank);
        r.y = static_cast<uint16_t *>(y);
        r.ldy = ldy;
        r.num_tokens = num_tokens;
        r.cols = out_features;
        r.k = hidden;
        r.rank = rank;
        r.slices = num_slices;
        r.max_loras = meta->max_loras;
        r.scale = scale;
        hipLaunchKernelGGL(rows_shrink_kernel, dim3((unsigned)shrinks), dim3(kRowsShrinkWaves * kWave), 0, stream, r);
        if (hipGetLastError() != hipSuccess) return LORA_ERR_LAUNCH;
        if (few) {
            const dim3 grid((unsigned)ceil_div(out_features, kRowsCols)), block(kRowsThreads);
            if (num_tokens <= 16)
                hipLaunchKernelGGL(rows_kernel<1>, grid, block, 0, stream, r);
            else
                hipLaunchKernelGGL(rows_kernel<2>, grid, block, 0, stream, r);
            return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_LAUNCH;
        }
    } else {
        if ((st = shrink_fresh(x, ldx, num_tokens, hidden, lora_a, num_slices, rank, buf, meta, scale, stream))) return st;
        if (launch_pack(meta, view, buf, packed, num_slices, rank, ws, nullptr, nullptr, stream) != hipSuccess)
            return LORA_ERR_LAUNCH;
    }
    LinearArgs a;
    memset(&a, 0, sizeof a);
    a.meta = view;
    a.ids = meta->token_lora_mapping;
    a.in = static_cast<const uint16_t *>(x);
    a.ldin = ldx;
    a.w = static_cast<const uint16_t *>(w);
    a.ldw = ldw;
    a.w_bias = static_cast<const uint16_t *>(w_bias);
    int off = offset_start;
    for (int i = 0; i < num_slices; ++i) {
        a.lw[i] = static_cast<const uint16_t *>(lora_b[i]);
        a.bias[i] = bias ? static_cast<const uint16_t *>(bias[i]) : nullptr;
        a.has_bias |= a.bias[i] != nullptr;
        a.width[i] = slice_widths[i];
        a.col[i] = off;
        off += slice_widths[i];
    }
    a.packed = packed;
    a.s = buf;
    a.y = static_cast<uint16_t *>(y);
    a.ldy = ldy;
    a.num_tokens = num_tokens;
    a.cols = out_features;
    a.k = hidden;
    a.rank = rank;
    a.slices = num_slices;
    a.max_loras = meta->max_loras;
    return launch_linear<false>(a, stream) == hipSuccess ? LORA_OK : LORA_ERR_LAUNCH;
}

int lora_linear_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx, int num_tokens, int hidden,
                         const void *w, int64_t ldw, int out_features, const void *const *lora_a,
                         const void *const *lora_b, const int *slice_widths, int num_slices, int rank,
                         const float *buf, float *dbuf, void *dx, int64_t lddx, void *const *da, void *const *db,
                         void *const *dbias, int offset_start, const lora_meta_t *meta, float scale, void *workspace,
                         size_t workspace_bytes, hipStream_t stream) {
    int st = check_call(ldx, num_tokens, hidden, w, ldw, out_features, lora_a, lora_b, slice_widths, num_slices, rank,
                        lddy, offset_start, meta, workspace);
    if (st) return st;
    if (!da || !db) return LORA_ERR_NULL;
    for (int i = 0; i < num_slices; ++i) {
        if (!da[i] || !db[i]) return LORA_ERR_NULL;
        if (!aligned16(da[i]) || !aligned16(db[i])) return LORA_ERR_ALIGN;
        if (dbias && dbias[i] && !aligned16(dbias[i])) return LORA_ERR_ALIGN;
    }
    if (dx && (lddx < hidden || lddx % 8)) return LORA_ERR_SHAPE;
    if (num_tokens > 0 && (!dy || !x || !buf || !dbuf)) return LORA_ERR_NULL;
    if (num_tokens > 0 && (!aligned16(dy) || !aligned16(x) || !aligned16(buf) || !aligned16(dbuf) || !aligned16(dx)))
        return LORA_ERR_ALIGN;
    const UPlan u = plan_u(num_tokens, meta->max_loras, num_slices, rank, widest(slice_widths, num_slices));
    const Layout l = layout(num_tokens, meta->max_loras, num_slices, rank, u, true);
    if (l.total > workspace_bytes) return LORA_ERR_BUFFER;
    char *ws = static_cast<char *>(workspace);
    const MetaView view = view_of(meta);
    uint16_t *s = reinterpret_cast<uint16_t *>(ws + l.s), *up = reinterpret_cast<uint16_t *>(ws + l.u);
    float *slots = reinterpret_cast<float *>(ws + l.slots);
    int32_t *counters = reinterpret_cast<int32_t *>(ws + l.counters);
    const SegEntry *segs = reinterpret_cast<const SegEntry *>(ws + l.segs);
    // (an empty batch still writes the adapters' gradients: zeros)
    if (launch_pack(meta, view, buf, s, num_slices, rank, ws, &l, &u, stream) != hipSuccess) return LORA_ERR_LAUNCH;
    int cols[LORA_MAX_SLICES], off = offset_start;
    for (int i = 0; i < num_slices; ++i) {
        cols[i] = off;
        off += slice_widths[i];
    }
    if (num_tokens > 0) {
        UArgs ua;
        memset(&ua, 0, sizeof ua);
        ua.tiles = reinterpret_cast<const UTile *>(ws + l.tiles);
        ua.num_tiles = reinterpret_cast<const int32_t *>(ws + l.num_tiles);
        ua.sorted = view.sorted;
        ua.dy = static_cast<const uint16_t *>(dy);
        ua.lddy = lddy;
        for (int i = 0; i < num_slices; ++i) {
            ua.b[i] = static_cast<const uint16_t *>(lora_b[i]);
            ua.width[i] = slice_widths[i];
            ua.col[i] = cols[i];
        }
        ua.dbuf = dbuf;
        ua.packed = up;
        ua.slots = slots;
        ua.counters = counters;
        ua.num_tokens = num_tokens;
        ua.rank = rank;
        ua.slices = num_slices;
        ua.splits = u.splits;
        ua.scale = scale;
        const hipError_t e = u.bm == 32 ? launch_u<32>(ua, u, stream) : u.bm == 64 ? launch_u<64>(ua, u, stream) : launch_u<128>(ua, u, stream);
        if (e != hipSuccess) return LORA_ERR_LAUNCH;
    }
    if (dx && num_tokens > 0) {
        LinearArgs a;
        memset(&a, 0, sizeof a);
        a.meta = view;
        a.ids = meta->token_lora_mapping;
        a.in = static_cast<const uint16_t *>(dy);
        a.ldin = lddy;
        a.w = static_cast<const uint16_t *>(w);
        a.ldw = ldw;
        for (int i = 0; i < num_slices; ++i) a.lw[i] = static_cast<const uint16_t *>(lora_a[i]);
        a.packed = up;
        a.s = dbuf;
        a.y = static_cast<uint16_t *>(dx);
        a.ldy = lddx;
        a.num_tokens = num_tokens;
        a.cols = hidden;
        a.k = out_features;
        a.rank = rank;
        a.slices = num_slices;
        a.max_loras = meta->max_loras;
        if (launch_linear<true>(a, stream) != hipSuccess) return LORA_ERR_LAUNCH;
    }
    GradArgs g;
    memset(&g, 0, sizeof g);
    g.segs = segs;
    g.sorted = view.sorted;
    g.num_tokens = num_tokens;
    g.rank = rank;
    g.slices = num_slices;
    g.act = static_cast<const uint16_t *>(x);
    g.ldact = ldx;
    g.packed = up;
    for (int i = 0; i < num_slices; ++i) {
        g.out[i] = static_cast<uint16_t *>(da[i]);
        g.width[i] = hidden;
    }
    if (launch_grads<true>(g, meta->max_loras, stream) != hipSuccess) return LORA_ERR_LAUNCH;
    g.act = static_cast<const uint16_t *>(dy);
    g.ldact = lddy;
    g.packed = s;
    for (int i = 0; i < num_slices; ++i) {
        g.out[i] = static_cast<uint16_t *>(db[i]);
        g.dbias[i] = dbias ? static_cast<uint16_t *>(dbias[i]) : nullptr;
        g.width[i] = slice_widths[i];
        g.col[i] = cols[i];
    }
    return launch_grads<false>(g, meta->max_loras, stream) == hipSuccess ? LORA_OK : LORA_ERR_LAUNCH;
}

}  // extern "C"
