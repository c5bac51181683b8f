// lora_loss.hip -- softmax cross entropy of hidden states x against a
// vocabulary matrix w, in pieces of the vocabulary, without the logits in
// memory, and its gradients:
//
//   z[t] = w x[t],  lse[t] = log sum_v exp z[t][v],  loss[t] = lse[t] - z[t][target[t]]
//   g[t][v] = dloss[t] (exp(z[t][v] - lse[t]) - [v = target[t]])
//   dx[t] = w^T g[t],  dw = sum_t g[t] x[t]^T;  ignored tokens: loss 0, g 0
//
// Forward: every workgroup computes a tile of logits (vocabulary rows on the M
// side, tokens on the N side, so that a token's logits lie in one lane and its
// three neighbours 16 apart), reduces it to one (maximum, sum of exponentials)
// pair per token in fp32 and forgets it; a second launch joins the pairs of a
// token over the vocabulary tiles.  The target's logit is picked out by the
// tile that holds it.
//
// Backward: the logits are computed again, a piece of the vocabulary at a time;
// the epilogue turns them into g (bf16, the piece's buffer), from which two
// products make the piece's part of dx (fp32 planes, added up in piece order)
// and the piece's rows of dw.  Only the tokens that count take part: a first
// launch lists them in order.  g is rounded to bf16 because the matrix
// products take bf16; its fp32 value is formed from fp32 logits before that.
// The target's is always among a token's largest entries, and its rounding
// alone can add as much error to dx and dw as their own rounding: what it
// loses is kept in fp32 and comes back, to dx as one more row of w at the end,
// to dw as one more K step of the tokens whose target a tile holds.  The other
// entries' rounding stays: rms errors of dx and dw are those of their own rounding
// (0.00166) for flat softmaxes and sure targets, 0.0018 to 0.0020 where one to
// sixteen wrong entries are 9 to 12 above the rest.
#include <string.h>

#include <type_traits>

#include "lora_gemm.h"

namespace lora {
namespace {

extern __shared__ __attribute__((aligned(1024))) unsigned char g_lds[];

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kMaxFloat = 0x1.fffffep127f;

// exp(d): the hardware's 2^x of d log2(e).
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

struct Stat {
    float max, sum;   // sum of exp(z - max)
};
// What exponents are taken against: the maximum, or the finite number next to an
// infinite one, so that its own terms do not become infinity - infinity (all
// entries -inf: a sum of 0; an entry of +inf: a sum of +inf).
__device__ __forceinline__ float exp_base(float max) { return fminf(fmaxf(max, -kMaxFloat), kMaxFloat); }
__device__ __forceinline__ Stat join(const Stat &a, const Stat &b) {
    const float m = fmaxf(a.max, b.max);
    const float base = exp_base(m);
    return Stat{m, a.sum * exp_of(a.max - base) + b.sum * exp_of(b.max - base)};
}

struct LogitArgs {
    const uint16_t *x;          // gradient: the listed tokens' rows
    int64_t ldx;
    const uint16_t *w;          // the piece's first row
    int64_t ldw;
    const int32_t *targets;
    // statistics
    Stat *stats;                // [vocabulary tile][all_tokens]
    float *target_logit;        // [num_tokens]
    int32_t all_tokens;         // num_tokens, or more where a launch takes a part of them
    int32_t *status;
    // gradient
    const int32_t *list, *count;   // tokens that count
    const float *lse, *dloss;
    uint16_t *g;                // [listed token][ldg]
    int64_t ldg;
    float *lost;                // [listed token]: the target's g less its rounded value
    int32_t num_tokens, hidden, first, rows;   // piece: vocabulary [first, first + rows)
    int32_t mtiles, ntiles, group;
};

// 4096 tokens by 128256 entries over 4096: statistics 3.11 ms (1.38 PFLOP/s; the
// library's product without them 3.07), g 0.83 ms a piece of 32256; 256 tokens 0.24
// ms; 16 tokens 166 us (W at 6.3 TB/s).
template <class T, bool GRAD>
__global__ __launch_bounds__(T::kThreads) void logit_kernel(LogitArgs a) {
    __shared__ Stat s_stat[GRAD ? 1 : T::WM][GRAD ? 1 : T::BN];
    const int tid = threadIdx.x;
    const int n = GRAD ? *a.count : a.num_tokens;
    const int ntiles = GRAD ? (n + T::BN - 1) / T::BN : a.ntiles;
    if (!GRAD && blockIdx.x == 0 && tid == 0) *a.status = 0;
    TileAt at;
    if (!tile_at(blockIdx.x, a.mtiles, ntiles, a.group, at)) return;
    const int m0 = at.m * T::BM, p0 = at.n * T::BN, rows = min(T::BN, n - p0);
    PlainOp<T> op;
#pragma unroll
    for (int j = 0; j < T::NSide::kInstr; ++j)
        op.wn.p[j] = a.x + (int64_t)(p0 + min(T::NSide::row(j), rows - 1)) * a.ldx + T::NSide::elem(j);
#pragma unroll
    for (int j = 0; j < T::MSide::kInstr; ++j)
        op.wm.p[j] = a.w + (int64_t)min(m0 + T::MSide::row(j), a.rows - 1) * a.ldw + T::MSide::elem(j);
    op.wn.step = op.wm.step = kStepK;
    op.wn.left = op.wm.left = a.hidden;
    typename T::Acc acc;
    clear<T>(acc);
    mma_begin<T>(op, (a.hidden + kStepK - 1) / kStepK, g_lds);
    mma_loop<T>(op, a.hidden / kStepK, (a.hidden + kStepK - 1) / kStepK, acc, g_lds);

    if constexpr (!GRAD) {
        // vocabulary entries past the last (the last tile alone)
        if (m0 + T::BM > a.rows)
#pragma unroll
            for (int mt = 0; mt < T::MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m0 + T::m_of(mt) + e >= a.rows)
#pragma unroll
                        for (int nt = 0; nt < T::NT; ++nt) acc[mt][nt][e] = kNegInf;
        int target[T::NT];
#pragma unroll
        for (int nt = 0; nt < T::NT; ++nt) {
            const int r = T::n_of(nt);
            target[nt] = (r < rows ? a.targets[p0 + r] : -1) - m0;
        }
#pragma unroll
        for (int nt = 0; nt < T::NT; ++nt) {
            const int r = T::n_of(nt);
            // few tiles hold a token's target
            if ((unsigned)target[nt] < (unsigned)min(T::BM, a.rows - m0))
#pragma unroll
                for (int mt = 0; mt < T::MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (T::m_of(mt) + e == target[nt]) a.target_logit[p0 + r] = acc[mt][nt][e];
            float top = kNegInf;
#pragma unroll
            for (int mt = 0; mt < T::MT; ++mt)
                top = fmaxf(fmaxf(top, fmaxf(acc[mt][nt][0], acc[mt][nt][1])), fmaxf(acc[mt][nt][2], acc[mt][nt][3]));
            // the maximum of this token's four lanes first: one scale for all of their terms
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float base = exp_base(top);
            float sum = 0.f;
#pragma unroll
            for (int mt = 0; mt < T::MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum += exp_of(acc[mt][nt][e] - base);
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (lane_id() < 16) s_stat[T::wave_m()][r] = Stat{top, sum};
        }
        __syncthreads();
        for (int r = tid; r < rows; r += T::kThreads) {
            Stat s = s_stat[0][r];
#pragma unroll
            for (int w = 1; w < T::WM; ++w) s = join(s, s_stat[w][r]);
            a.stats[(int64_t)at.m * a.all_tokens + p0 + r] = s;
        }
    } else {
        // all the tokens' values in two round trips
        int target[T::NT];
        float lse[T::NT], dl[T::NT];
#pragma unroll
        for (int nt = 0; nt < T::NT; ++nt) target[nt] = a.list[p0 + min(T::n_of(nt), rows - 1)];
#pragma unroll
        for (int nt = 0; nt < T::NT; ++nt) {
            const int t = target[nt];
            lse[nt] = a.lse[t];
            dl[nt] = a.dloss[t];
            target[nt] = a.targets[t] - a.first;
        }
#pragma unroll
        for (int nt = 0; nt < T::NT; ++nt) {
            const int r = T::n_of(nt);
            if (r >= rows) continue;
            uint16_t *row = a.g + (int64_t)(p0 + r) * a.ldg;
            static_assert(T::DEAL > 1, "8 consecutive entries a lane");
#pragma unroll
            for (int mt = 0; mt < T::MT; mt += 2) {
                const int v = m0 + T::m_of(mt);
                if (v >= a.ldg) continue;
                float g[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float p = exp_of(acc[mt + x / 4][nt][x % 4] - lse[nt]);
                    g[x] = v + x < a.rows ? (p - (v + x == target[nt] ? 1.f : 0.f)) * dl[nt] : 0.f;
                }
                if ((unsigned)(target[nt] - v) < 8u)   // one lane of one piece
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (v + x == target[nt]) a.lost[p0 + r] = g[x] - bf16_bits_to_float(float_to_bf16_bits(g[x]));
                *reinterpret_cast<u32x4 *>(row + v) =
                    u32x4{pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]), pack_bf16(g[4], g[5]), pack_bf16(g[6], g[7])};
            }
        }
    }
}

// ---------------------------------------------------------------- joining the pieces' statistics

struct JoinArgs {
    const Stat *stats;
    const float *target_logit;
    const int32_t *targets;
    float *loss, *lse;
    int32_t *status;
    int32_t num_tokens, mtiles, vocab;
};

// 16 tokens a workgroup, 64 threads each, eight pairs at a time: 5 to 7 us for 16
// to 4096 tokens of 128256 entries, mostly latency.
constexpr int kJoinParts = 64, kJoinTokens = 16, kJoinChunk = 8;
__global__ __launch_bounds__(kJoinParts *kJoinTokens) void join_kernel(JoinArgs a) {
    __shared__ Stat s_part[kJoinParts][kJoinTokens];
    const int tok = threadIdx.x % kJoinTokens, part = threadIdx.x / kJoinTokens, t = blockIdx.x * kJoinTokens + tok;
    Stat s{kNegInf, 0.f};
    if (t < a.num_tokens)
        for (int k = part; k < a.mtiles; k += kJoinParts * kJoinChunk) {
            Stat v[kJoinChunk];
#pragma unroll
            for (int i = 0; i < kJoinChunk; ++i) {
                const int q = k + i * kJoinParts;
                v[i] = q < a.mtiles ? a.stats[(int64_t)q * a.num_tokens + t] : Stat{kNegInf, 0.f};
            }
#pragma unroll
            for (int w = kJoinChunk / 2; w; w /= 2)
#pragma unroll
                for (int i = 0; i < w; ++i) v[i] = join(v[i], v[i + w]);
            s = join(s, v[0]);
        }
    s_part[part][tok] = s;
#pragma unroll
    for (int w = kJoinParts / 2; w; w /= 2) {
        __syncthreads();
        if (part < w) s_part[part][tok] = s = join(s, s_part[part + w][tok]);
    }
    if (part == 0 && t < a.num_tokens) {
        // the loss from its two terms: lse, rounded at the logits' size, would lose the
        // digits of a loss that is small against them
        const float log_sum = logf(s.sum);
        const int target = a.targets[t];
        a.lse[t] = s.max + log_sum;
        a.loss[t] = target >= 0 && target < a.vocab ? (s.max - a.target_logit[t]) + log_sum : 0.f;
        if (target < -1 || target >= a.vocab)
            __hip_atomic_store(a.status, (int)LORA_ERR_ID_RANGE, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// ---------------------------------------------------------------- the tokens that count

struct ListArgs {
    const int32_t *targets;
    int32_t *list, *place, *count;   // listed tokens; each token's place in the list or -1
    int32_t *list_targets;           // targets of the listed tokens
    int32_t num_tokens, vocab;
};
constexpr int kListThreads = 1024;

// One workgroup (5 us for 4096 tokens): the list is short against the products it
// shortens.
__global__ __launch_bounds__(kListThreads) void list_kernel(ListArgs a) {
    __shared__ int s_wsum[kListThreads / kWave];
    int base = 0;
    for (int t0 = 0; t0 < a.num_tokens; t0 += kListThreads) {
        const int t = t0 + threadIdx.x;
        const int target = t < a.num_tokens ? a.targets[t] : -1;
        const bool counts = target >= 0 && target < a.vocab;
        const uint64_t mask = ballot(counts);
        if (lane_id() == 0) s_wsum[wave_id()] = __popcll(mask);
        __syncthreads();
        int before = base, all = 0;
        for (int w = 0; w < kListThreads / kWave; ++w) {
            before += w < wave_id() ? s_wsum[w] : 0;
            all += s_wsum[w];
        }
        const int p = before + __popcll(mask & lanemask_lt());
        if (counts) {
            a.list[p] = t;
            a.list_targets[p] = target;
        }
        if (t < a.num_tokens) a.place[t] = counts ? p : -1;
        base += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) *a.count = base;
}

// The listed tokens' rows of x one after the other: read through the list
// instead, as K rows of dw, they cost dw 15 % (4096 tokens by 4096 by 32000).
struct RowsOfArgs {
    const uint16_t *x;
    int64_t ldx;
    const int32_t *list, *count;
    uint16_t *out;
    int32_t hidden;
};
__global__ __launch_bounds__(256) void rows_of_kernel(RowsOfArgs a) {
    const int per = a.hidden / 8;
    const int64_t work = (int64_t)*a.count * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < work; i += (int64_t)gridDim.x * 256) {
        const int p = (int)(i / per), c = (int)(i % per) * 8;
        *reinterpret_cast<u32x4 *>(a.out + i * 8) = *reinterpret_cast<const u32x4 *>(a.x + (int64_t)a.list[p] * a.ldx + c);
    }
}

// ---------------------------------------------------------------- dx and dw of a piece

struct DxArgs {
    const uint16_t *w;          // the piece's first row
    int64_t ldw;
    const uint16_t *g;
    int64_t ldg;
    float *planes;              // [split][n][hidden]
    const int32_t *count;
    int32_t num_tokens, hidden, rows, add;
    int32_t mtiles, group, splits, split_steps;
};

// planes[split][p] (+)= sum over the split's vocabulary rows of g[p][v] w[v].  0.76
// ms a piece of 32256 entries for 3686 tokens over 4096 (1.28 PFLOP/s; the library's
// product of such strides 1.32).
template <class T>
__global__ __launch_bounds__(T::kThreads) void dx_kernel(DxArgs a) {
    const int n = *a.count, ntiles = (n + T::BN - 1) / T::BN;
    const int split = blockIdx.x % a.splits;
    TileAt at;
    if (!tile_at(blockIdx.x / a.splits, a.mtiles, ntiles, a.group, at)) return;
    const int m0 = at.m * T::BM, p0 = at.n * T::BN, rows = min(T::BN, n - p0);
    const int all = (a.rows + kStepK - 1) / kStepK, s0 = min(all, split * a.split_steps), s1 = min(all, s0 + a.split_steps);
    PlainOp<T> op;
#pragma unroll
    for (int j = 0; j < T::NSide::kInstr; ++j)
        op.wn.p[j] = a.g + (int64_t)(p0 + min(T::NSide::row(j), rows - 1)) * a.ldg + s0 * kStepK + T::NSide::elem(j);
    op.wn.step = kStepK;
#pragma unroll
    for (int j = 0; j < T::MSide::kInstr; ++j)
        op.wm.p[j] = a.w + (int64_t)(s0 * kStepK + T::MSide::row(j)) * a.ldw + min(m0 + T::MSide::elem(j), a.hidden - 8);
    op.wm.step = (int64_t)kStepK * a.ldw;
    op.wn.left = op.wm.left = a.rows - s0 * kStepK;
    typename T::Acc acc;
    clear<T>(acc);
    mma_begin<T>(op, s1 - s0, g_lds);
    mma_loop<T>(op, min(s1, a.rows / kStepK) - s0, s1 - s0, acc, g_lds);
#pragma unroll
    for (int nt = 0; nt < T::NT; ++nt) {
        const int r = T::n_of(nt);
        if (r >= rows) continue;
        float *row = a.planes + ((int64_t)split * a.num_tokens + p0 + r) * a.hidden;
#pragma unroll
        for (int mt = 0; mt < T::MT; ++mt) {
            const int c = m0 + T::m_of(mt);
            if (c >= a.hidden) continue;
            floatx4 *at4 = reinterpret_cast<floatx4 *>(row + c);
            *at4 = a.add ? *at4 + acc[mt][nt] : acc[mt][nt];
        }
    }
}

struct FinishArgs {
    const float *planes;
    const int32_t *place;
    const float *lost;
    const int32_t *targets;
    const uint16_t *w;
    int64_t ldw;
    uint16_t *dx;
    int64_t lddx;
    int32_t num_tokens, hidden, splits;
};
__global__ __launch_bounds__(256) void finish_kernel(FinishArgs a) {
    const int per = a.hidden / 8;
    const int64_t work = (int64_t)a.num_tokens * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < work; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / per;
        const int c = (int)(i % per) * 8, p = a.place[t];
        floatx4 v0 = {0.f, 0.f, 0.f, 0.f}, v1 = v0;
        if (p >= 0) {
            const float lost = a.lost[p];
            const u32x4 w = *reinterpret_cast<const u32x4 *>(a.w + (int64_t)a.targets[t] * a.ldw + c);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float lo, hi;
                unpack_bf16(w[x], lo, hi);
                (x < 2 ? v0 : v1)[2 * (x & 1)] = lost * lo;
                (x < 2 ? v0 : v1)[2 * (x & 1) + 1] = lost * hi;
            }
            for (int s = 0; s < a.splits; ++s) {
                const floatx4 *q = reinterpret_cast<const floatx4 *>(a.planes + ((int64_t)s * a.num_tokens + p) * a.hidden + c);
                v0 += q[0];
                v1 += q[1];
            }
        }
        *reinterpret_cast<u32x4 *>(a.dx + t * a.lddx + c) =
            u32x4{pack_bf16(v0[0], v0[1]), pack_bf16(v0[2], v0[3]), pack_bf16(v1[0], v1[1]), pack_bf16(v1[2], v1[3])};
    }
}

struct DwArgs {
    const uint16_t *x;          // the listed tokens' rows
    int64_t ldx;
    const uint16_t *g;
    int64_t ldg;
    uint16_t *dw;               // the piece's first row
    int64_t lddw;
    const int32_t *count, *targets;   // targets: of the listed tokens
    const float *lost;
    int32_t hidden, first, rows;
    int32_t mtiles, ntiles, group;
};

// dw's tile += sum over the listed tokens p whose target it holds of lost[p]
// x[p]: K steps of 64 such tokens in list order, the N side built in LDS (one
// entry a K row).  About one step a tile.
template <class T>
__device__ __forceinline__ void add_lost(const DwArgs &a, int n, int m0, int v0, typename T::Acc &acc) {
    constexpr int kChunk = 4;
    __shared__ int s_match[kChunk * T::kThreads], s_wave[kChunk][T::kWaves];   // place << 8 | row of the tile
    static_assert(T::BN <= 256 && LORA_MAX_TOKENS <= 1 << 22, "a match in 31 bits");
    const lds_byte *lds = (const lds_byte *)g_lds;
    const uint32_t base = lds_address(g_lds);
    const int tid = threadIdx.x, width = min(T::BN, a.rows - v0);
    own_reads_barrier();   // the stages are free
    for (int from = 0; from < n; from += kChunk * T::kThreads) {
        int row[kChunk], at[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            const int p = from + i * T::kThreads + tid;
            row[i] = p < n ? a.targets[p] - a.first - v0 : -1;
        }
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            const uint64_t mask = ballot((unsigned)row[i] < (unsigned)width);
            at[i] = __popcll(mask & lanemask_lt());
            if (lane_id() == 0) s_wave[i][wave_id()] = __popcll(mask);
        }
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
#pragma unroll
            for (int w = 0; w < T::kWaves; ++w) {
                at[i] += w == wave_id() ? total : 0;
                total += s_wave[i][w];
            }
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            if ((unsigned)row[i] < (unsigned)width) s_match[at[i]] = (from + i * T::kThreads + tid) << 8 | row[i];
        __syncthreads();
        total = __builtin_amdgcn_readfirstlane(total);
        for (int k0 = 0; k0 < total; k0 += kStepK) {
            const int count = min(kStepK, total - k0);
#pragma unroll
            for (int j = 0; j < T::MSide::kInstr; ++j) {
                const int k = T::MSide::row(j), p = s_match[k0 + min(k, count - 1)] >> 8;
                dma16(k < count ? a.x + (int64_t)p * a.ldx + min(m0 + T::MSide::elem(j), a.hidden - 8) : zero_page,
                      base + T::MSide::dst(j));
            }
            for (int o = 16 * tid; o < T::NSide::kBytes; o += 16 * T::kThreads)
                *reinterpret_cast<u32x4 *>(g_lds + T::MSide::kBytes + o) = u32x4{0u, 0u, 0u, 0u};
            __syncthreads();
            if (tid < count) {
                const int match = s_match[k0 + tid];
                *reinterpret_cast<uint16_t *>(g_lds + T::MSide::kBytes + T::NSide::at(tid, match & 255)) =
                    (uint16_t)float_to_bf16_bits(a.lost[match >> 8]);
            }
            wait_loads_barrier<0>();
            typename T::Half r;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                T::read(r, lds, h);
                T::mma(r, acc);
            }
            own_reads_barrier();
        }
        __syncthreads();
    }
}
// dw[v] = sum over the listed tokens of g[p][v] x[p]: both sides have K
// (the tokens) as their row index.  0.85 ms a piece of 32256 entries for 3686
// tokens over 4096 (1.15 PFLOP/s: transposing LDS reads for both sides; the
// library's product of such strides 1.11).
template <class T>
__global__ __launch_bounds__(T::kThreads) void dw_kernel(DwArgs a) {
    TileAt at;
    if (!tile_at(blockIdx.x, a.mtiles, a.ntiles, a.group, at)) return;
    const int n = *a.count, m0 = at.m * T::BM, v0 = at.n * T::BN;
    typename T::Acc acc;
    clear<T>(acc);
    if (n > 0) {
        PairOp<T, OffsetWalk<typename T::MSide>, OffsetWalk<typename T::NSide>> op;
#pragma unroll
        for (int j = 0; j < T::MSide::kInstr; ++j)
            op.wm.off[j] = 2u * ((uint32_t)T::MSide::row(j) * (uint32_t)a.ldx + min(m0 + T::MSide::elem(j), a.hidden - 8));
        op.wm.base = a.x;
        op.wm.step = (int64_t)kStepK * a.ldx;
#pragma unroll
        for (int j = 0; j < T::NSide::kInstr; ++j)
            op.wn.off[j] = 2u * ((uint32_t)T::NSide::row(j) * (uint32_t)a.ldg + min(v0 + T::NSide::elem(j), (int)a.ldg - 8));
        op.wn.base = a.g;
        op.wn.step = (int64_t)kStepK * a.ldg;
        op.wm.left = op.wn.left = n;
        mma_begin<T>(op, (n + kStepK - 1) / kStepK, g_lds);
        mma_loop<T>(op, n / kStepK, (n + kStepK - 1) / kStepK, acc, g_lds);
        add_lost<T>(a, n, m0, v0, acc);
    }
#pragma unroll
    for (int nt = 0; nt < T::NT; ++nt) {
        const int v = v0 + T::n_of(nt);
        if (v >= a.rows) continue;
        uint16_t *row = a.dw + (int64_t)v * a.lddw;
#pragma unroll
        for (int mt = 0; mt < T::MT; ++mt) {
            const int c = m0 + T::m_of(mt);
            const floatx4 q = acc[mt][nt];
            if (c < a.hidden) *reinterpret_cast<u32x2g *>(row + c) = u32x2g{pack_bf16(q[0], q[1]), pack_bf16(q[2], q[3])};
        }
    }
}

// ---------------------------------------------------------------- plans

constexpr size_t kRound = 256;
size_t up(size_t v) { return (v + kRound - 1) / kRound * kRound; }
long ceil_div(long a, long b) { return (a + b - 1) / b; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

enum LossTile { kBig, kMid, kSmall, kRow };
// The tile of a product of m by n outputs: 256 x 256 where 128 x 128, two of which
// run on a CU, would take a second round; 128 x 128 from 384 tiles on; 64 x 64 below;
// 128 x 32 for few tokens.  us over 4096, larger tile and smaller:
//   256 x 256, 128 x 128 (tiles of the latter)
//     384 (129 tokens by 24576) 85, 76;  512 (2048 by 4096) 87, 82
//     640 (2048 by 5120) 91, 119;  640 (256 by 40960) 108, 132;  g and dw, 2048 by
//     5120 over 2048: 120, 147
//   128 x 128, 64 x 64
//     300 (301 by 12800) 69, 56;  384 (301 by 16384) 73, 71;  384 (256 by 24576) 77, 87
//     420 (301 by 17920) 74, 77;  g and dw, 120 (301 by 5003 over 264): 30, 23
LossTile pick_tile(long m, long n) {
    if (n <= 32) return kRow;
    const long tiles = ceil_div(m, 128) * ceil_div(n, 128);
    if (n > 128 && tiles > 512) return kBig;
    return tiles >= 384 ? kMid : kSmall;
}
int tile_m(LossTile t) { return t == kBig ? 256 : t == kSmall ? 64 : 128; }
int tile_n(LossTile t) { return t == kBig ? 256 : t == kMid ? 128 : t == kSmall ? 64 : 32; }

// Tiles of a launch, whose threads are fewer than 2^32: past that the forward pass
// takes the tokens in parts.  (g has at most kPieceElems elements or kPieceMin rows.)
constexpr long kLaunchTiles = (1L << 32) / 512 - kNumXcd;
static_assert(kLaunchTiles > LORA_MAX_VOCAB / 64, "a part has a tile of tokens at least");

struct LossPlan {
    LossTile logits, grad, dx, dw;
    long mtiles;         // vocabulary tiles of the statistics
    long piece;          // vocabulary rows of a piece (a multiple of 256)
    int splits, split_steps;
};
// g's buffer: 2^27 elements (256 MB, the size of the last-level cache), at
// least 4096 vocabulary rows.
constexpr long kPieceElems = 1L << 27, kPieceMin = 4096;
constexpr long kMaxSplits = 16, kSplitSteps = 16;   // dx: parts of a split K, steps of each at least

LossPlan plan_loss(long n, long hidden, long vocab) {
    LossPlan p;
    p.logits = pick_tile(vocab, n);
    p.mtiles = ceil_div(vocab, tile_m(p.logits));
    const long whole = ceil_div(vocab, 256) * 256;
    long piece = kPieceElems / (n > 0 ? n : 1) / 256 * 256;
    if (piece < kPieceMin) piece = kPieceMin;
    if (piece > whole) piece = whole;
    piece = ceil_div(ceil_div(whole, ceil_div(whole, piece)), 256) * 256;   // pieces of equal size
    p.piece = piece;
    p.grad = pick_tile(piece, n);
    const long steps = piece / kStepK;
    // dx: K (the piece) is split until the CUs are full; the tile is the largest that
    // does so (us of g and dx, 256 x 256, 128 x 128 and 64 x 64: 2048 tokens by 4096 over
    // 32000 849, 1013, 1553; 100 by 8192 over 32000 285, 263, 316; 301 by 264 over 5003
    // 45, 35, 29; 600 by 264 over 20000 70, 57, 68)
    auto splits_of = [&](LossTile t) {
        const long tiles = ceil_div(hidden, tile_m(t)) * ceil_div(n > 0 ? n : 1, tile_n(t));
        long s = (t == kBig ? 256 : 512) / tiles;
        if (s > steps / kSplitSteps) s = steps / kSplitSteps;
        if (s > kMaxSplits) s = kMaxSplits;
        return s < 1 ? 1 : s;
    };
    p.dx = kRow;
    if (n > 32) p.dx = kSmall;
    if (n > 128 && ceil_div(hidden, 256) * ceil_div(n, 256) * splits_of(kBig) >= 192) p.dx = kBig;
    else if (n > 32 && ceil_div(hidden, 128) * ceil_div(n, 128) * splits_of(kMid) >= 384) p.dx = kMid;
    const long s = splits_of(p.dx);
    p.split_steps = (int)ceil_div(steps, s);
    p.splits = (int)ceil_div(steps, p.split_steps);
    p.dw = pick_tile(hidden, piece);
    return p;
}

struct LossLayout {
    size_t status, target_logit, stats, list, list_targets, place, count, lost, x, g, planes, total;
};
size_t least(size_t a, size_t b) { return a < b ? a : b; }
size_t largest(size_t a, size_t b) { return a > b ? a : b; }
// The areas whose sizes follow the plan have room for every smaller batch too,
// whose plan may need more of them (more vocabulary tiles, larger pieces, a split
// K): each is a bound on the plans of up to n tokens that grows with n.
//   stats   128 x 32 and 128 x 128 tiles serve up to 128 tokens, 256 x 256 tiles the
//           largest batches; other 128 x 128 tiles are at most 512, 64 x 64 ones fewer
//           than 384 of 128 x 128 (tokens times vocabulary tiles: at most 128 * 512, and
//           below 2 * 128 * 384)
//   g       a piece is at most the vocabulary, and at most kPieceElems elements or
//           kPieceMin rows
//   planes  a split K fills at most 256 workgroups of 256 x 256 or 512 smaller ones, and
//           has at most kMaxSplits parts of at least kSplitSteps steps
LossLayout loss_layout(const LossPlan &p, long n, long hidden, long vocab, bool train) {
    LossLayout l;
    const size_t tokens = (size_t)n, whole = (size_t)ceil_div(vocab, 256) * 256;
    size_t stats = tokens * (size_t)ceil_div(vocab, 256);
    stats = largest(stats, least(tokens, 128) * (size_t)ceil_div(vocab, 128));
    stats = largest(stats, least(tokens * (size_t)ceil_div(vocab, 64), 2 * 128 * 384));
    const size_t g = least(tokens * whole, largest((size_t)kPieceElems, tokens * (size_t)kPieceMin));
    const size_t parts = least(kMaxSplits, whole / kStepK / kSplitSteps);
    const size_t planes = largest(tokens, least(tokens * parts, ceil_div((size_t)256 * 256 * 256, hidden)));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up(bytes);
        return o;
    };
    l.status = take(sizeof(int32_t));
    // the forward pass's areas and the backward pass's are not in use together
    const size_t begin = at;
    l.target_logit = take(sizeof(float) * (size_t)n);
    l.stats = take(sizeof(Stat) * largest(stats, (size_t)p.mtiles * tokens));
    const size_t forward = at;
    at = begin;
    l.list = take(train ? sizeof(int32_t) * (size_t)n : 0);
    l.list_targets = take(train ? sizeof(int32_t) * (size_t)n : 0);
    l.place = take(train ? sizeof(int32_t) * (size_t)n : 0);
    l.count = take(train ? sizeof(int32_t) : 0);
    l.lost = take(train ? sizeof(float) * (size_t)n : 0);
    l.x = take(train ? sizeof(uint16_t) * (size_t)n * (size_t)hidden : 0);
    l.g = take(train ? sizeof(uint16_t) * largest(g, tokens * (size_t)p.piece) : 0);
    l.planes = take(train ? sizeof(float) * largest(planes, tokens * (size_t)p.splits) * (size_t)hidden : 0);
    l.total = at > forward ? at : forward;
    return l;
}

int check_sizes(int num_tokens, int hidden, int vocab) {
    if (num_tokens < 0 || num_tokens > LORA_MAX_TOKENS) return LORA_ERR_NUM_TOKENS;
    if (hidden < 8 || hidden % 8 || hidden > LORA_MAX_HIDDEN || vocab < 1 || vocab > LORA_MAX_VOCAB) return LORA_ERR_SHAPE;
    return LORA_OK;
}
int check_loss(const void *x, int64_t ldx, int num_tokens, int hidden, const void *w, int64_t ldw, int vocab,
               const int32_t *targets, const void *workspace, size_t workspace_bytes, bool train) {
    const int st = check_sizes(num_tokens, hidden, vocab);
    if (st) return st;
    if (ldx < hidden || ldx % 8 || ldw < hidden || ldw % 8) return LORA_ERR_SHAPE;
    if (!w || !workspace || (num_tokens > 0 && (!x || !targets))) return LORA_ERR_NULL;
    if (!aligned16(w) || (num_tokens > 0 && !aligned16(x))) return LORA_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(workspace) & (kRound - 1)) != 0) return LORA_ERR_BUFFER;
    const LossPlan p = plan_loss(num_tokens, hidden, vocab);
    if (loss_layout(p, num_tokens, hidden, vocab, train).total > workspace_bytes) return LORA_ERR_BUFFER;
    return LORA_OK;
}

// Runs F with the tile type of `t` (M side strided: MS, N side: NS).  The 128 x 32
// tile is for few tokens on the N side; dw has vocabulary entries there, 256 or more.
template <bool MS, bool NS, class F>
hipError_t with_tile(LossTile t, F f) {
    switch (t) {
        case kBig: return f(Tile<256, 256, 4, 2, MS, NS>{});
        case kMid: return f(Tile<128, 128, 2, 2, MS, NS>{});
        case kSmall: return f(Tile<64, 64, 1, 4, MS, NS, 0, 4>{});
        case kRow:
            if constexpr (!NS) return f(Tile<128, 32, 2, 2, MS, NS, 0, 4>{});
    }
    return hipErrorInvalidValue;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t lora_cross_entropy_workspace_bytes(int num_tokens, int hidden, int vocab, int backward) {
    if (check_sizes(num_tokens, hidden, vocab)) return 0;
    return loss_layout(plan_loss(num_tokens, hidden, vocab), num_tokens, hidden, vocab, backward != 0).total;
}

int lora_cross_entropy(const void *x, int64_t ldx, int num_tokens, int hidden, const void *w, int64_t ldw, int vocab,
                       const int32_t *targets, float *loss, float *lse, void *workspace, size_t workspace_bytes,
                       hipStream_t stream) {
    const int st = check_loss(x, ldx, num_tokens, hidden, w, ldw, vocab, targets, workspace, workspace_bytes, false);
    if (st) return st;
    if (num_tokens > 0 && (!loss || !lse)) return LORA_ERR_NULL;
    if (num_tokens == 0) return LORA_OK;
    const LossPlan p = plan_loss(num_tokens, hidden, vocab);
    const LossLayout l = loss_layout(p, num_tokens, hidden, vocab, false);
    char *ws = static_cast<char *>(workspace);
    LogitArgs a;
    memset(&a, 0, sizeof a);
    a.ldx = ldx;
    a.w = static_cast<const uint16_t *>(w);
    a.ldw = ldw;
    a.status = reinterpret_cast<int32_t *>(ws + l.status);
    a.hidden = hidden;
    a.rows = vocab;
    a.mtiles = (int)p.mtiles;
    a.group = 8;
    a.all_tokens = num_tokens;
    Stat *stats = reinterpret_cast<Stat *>(ws + l.stats);
    float *target_logit = reinterpret_cast<float *>(ws + l.target_logit);
    const long part = kLaunchTiles / p.mtiles * tile_n(p.logits);
    for (long t0 = 0; t0 < num_tokens; t0 += part) {
        a.x = static_cast<const uint16_t *>(x) + t0 * ldx;
        a.targets = targets + t0;
        a.stats = stats + t0;
        a.target_logit = target_logit + t0;
        a.num_tokens = (int)(num_tokens - t0 < part ? num_tokens - t0 : part);
        a.ntiles = (int)ceil_div(a.num_tokens, tile_n(p.logits));
        const unsigned grid = tile_grid((long)a.mtiles * a.ntiles);
        const hipError_t e = with_tile<false, false>(p.logits, [&](auto tile) {
            using T = decltype(tile);
            return launch_tiles<logit_kernel<T, false>>(grid, T::kThreads, T::kLds, stream, a);
        });
        if (e != hipSuccess) return LORA_ERR_LAUNCH;
    }
    JoinArgs j;
    j.stats = stats;
    j.target_logit = target_logit;
    j.targets = targets;
    j.loss = loss;
    j.lse = lse;
    j.status = a.status;
    j.num_tokens = num_tokens;
    j.mtiles = a.mtiles;
    j.vocab = vocab;
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)ceil_div(num_tokens, kJoinTokens)), dim3(kJoinParts * kJoinTokens), 0, stream, j);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_LAUNCH;
}

int lora_cross_entropy_backward(const void *x, int64_t ldx, int num_tokens, int hidden, const void *w, int64_t ldw,
                                int vocab, const int32_t *targets, const float *lse, const float *dloss, void *dx,
                                int64_t lddx, void *dw, int64_t lddw, void *workspace, size_t workspace_bytes,
                                hipStream_t stream) {
    const int st = check_loss(x, ldx, num_tokens, hidden, w, ldw, vocab, targets, workspace, workspace_bytes, true);
    if (st) return st;
    if ((dx && (lddx < hidden || lddx % 8)) || (dw && (lddw < hidden || lddw % 8))) return LORA_ERR_SHAPE;
    if (num_tokens > 0 && (!lse || !dloss)) return LORA_ERR_NULL;
    if (!aligned16(dx) || !aligned16(dw)) return LORA_ERR_ALIGN;
    if (!dx && !dw) return LORA_OK;
    const LossPlan p = plan_loss(num_tokens, hidden, vocab);
    const LossLayout l = loss_layout(p, num_tokens, hidden, vocab, true);
    char *ws = static_cast<char *>(workspace);
    ListArgs la;
    la.targets = targets;
    la.list = reinterpret_cast<int32_t *>(ws + l.list);
    la.list_targets = reinterpret_cast<int32_t *>(ws + l.list_targets);
    la.place = reinterpret_cast<int32_t *>(ws + l.place);
    la.count = reinterpret_cast<int32_t *>(ws + l.count);
    la.num_tokens = num_tokens;
    la.vocab = vocab;
    hipLaunchKernelGGL(list_kernel, dim3(1), dim3(kListThreads), 0, stream, la);
    if (hipGetLastError() != hipSuccess) return LORA_ERR_LAUNCH;
    RowsOfArgs ra;
    ra.x = static_cast<const uint16_t *>(x);
    ra.ldx = ldx;
    ra.list = la.list;
    ra.count = la.count;
    ra.out = reinterpret_cast<uint16_t *>(ws + l.x);
    ra.hidden = hidden;
    if (num_tokens > 0) {
        long grid = ceil_div((long)num_tokens * (hidden / 8), 256);
        if (grid > 2048) grid = 2048;
        hipLaunchKernelGGL(rows_of_kernel, dim3((unsigned)grid), dim3(256), 0, stream, ra);
        if (hipGetLastError() != hipSuccess) return LORA_ERR_LAUNCH;
    }
    uint16_t *g = reinterpret_cast<uint16_t *>(ws + l.g);
    float *planes = reinterpret_cast<float *>(ws + l.planes);
    for (long first = 0; first < vocab; first += p.piece) {
        const int rows = (int)(vocab - first < p.piece ? vocab - first : p.piece);
        const uint16_t *wp = static_cast<const uint16_t *>(w) + first * ldw;
        const long ldg = p.piece;
        if (num_tokens > 0) {
            LogitArgs a;
            memset(&a, 0, sizeof a);
            a.x = ra.out;
            a.ldx = hidden;
            a.w = wp;
            a.ldw = ldw;
            a.targets = targets;
            a.list = la.list;
            a.count = la.count;
            a.lse = lse;
            a.dloss = dloss;
            a.g = g;
            a.ldg = ldg;
            a.lost = reinterpret_cast<float *>(ws + l.lost);
            a.num_tokens = num_tokens;
            a.hidden = hidden;
            a.first = (int)first;
            a.rows = rows;
            a.mtiles = (int)ceil_div(rows, tile_m(p.grad));
            a.ntiles = (int)ceil_div(num_tokens, tile_n(p.grad));
            a.group = 8;
            const unsigned grid = tile_grid((long)a.mtiles * a.ntiles);
            if (with_tile<false, false>(p.grad, [&](auto tile) {
                    using T = decltype(tile);
                    return launch_tiles<logit_kernel<T, true>>(grid, T::kThreads, T::kLds, stream, a);
                }) != hipSuccess)
                return LORA_ERR_LAUNCH;
        }
        if (dx && num_tokens > 0) {
            DxArgs d;
            memset(&d, 0, sizeof d);
            d.w = wp;
            d.ldw = ldw;
            d.g = g;
            d.ldg = ldg;
            d.planes = planes;
            d.count = la.count;
            d.num_tokens = num_tokens;
            d.hidden = hidden;
            d.rows = rows;
            d.add = first > 0;
            d.mtiles = (int)ceil_div(hidden, tile_m(p.dx));
            d.group = 8;
            d.splits = p.splits;
            d.split_steps = p.split_steps;
            const unsigned grid = tile_grid((long)d.mtiles * ceil_div(num_tokens, tile_n(p.dx))) * (unsigned)p.splits;
            if (with_tile<true, false>(p.dx, [&](auto tile) {
                    using T = decltype(tile);
                    return launch_tiles<dx_kernel<T>>(grid, T::kThreads, T::kLds, stream, d);
                }) != hipSuccess)
                return LORA_ERR_LAUNCH;
        }
        if (dw) {
            DwArgs d;
            memset(&d, 0, sizeof d);
            d.x = ra.out;
            d.ldx = hidden;
            d.g = g;
            d.ldg = ldg;
            d.dw = static_cast<uint16_t *>(dw) + first * lddw;
            d.lddw = lddw;
            d.count = la.count;
            d.targets = la.list_targets;
            d.lost = reinterpret_cast<const float *>(ws + l.lost);
            d.hidden = hidden;
            d.first = (int)first;
            d.rows = rows;
            d.mtiles = (int)ceil_div(hidden, tile_m(p.dw));
            d.ntiles = (int)ceil_div(rows, tile_n(p.dw));
            d.group = 8;
            const unsigned grid = tile_grid((long)d.mtiles * d.ntiles);
            if (with_tile<true, true>(p.dw, [&](auto tile) {
                    using T = decltype(tile);
                    return launch_tiles<dw_kernel<T>>(grid, T::kThreads, T::kLds, stream, d);
                }) != hipSuccess)
                return LORA_ERR_LAUNCH;
        }
    }
    if (dx && num_tokens > 0) {
        FinishArgs f;
        f.planes = planes;
        f.place = la.place;
        f.lost = reinterpret_cast<const float *>(ws + l.lost);
        f.targets = targets;
        f.w = static_cast<const uint16_t *>(w);
        f.ldw = ldw;
        f.dx = static_cast<uint16_t *>(dx);
        f.lddx = lddx;
        f.num_tokens = num_tokens;
        f.hidden = hidden;
        f.splits = p.splits;
        long grid = ceil_div((long)num_tokens * (hidden / 8), 256);
        if (grid > 2048) grid = 2048;
        hipLaunchKernelGGL(finish_kernel, dim3((unsigned)grid), dim3(256), 0, stream, f);
        if (hipGetLastError() != hipSuccess) return LORA_ERR_LAUNCH;
    }
    return LORA_OK;
}

}  // extern "C"
