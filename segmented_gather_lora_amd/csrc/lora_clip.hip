// lora_clip.hip -- norms over many gradient tensors, and the gradients scaled
// down to a largest norm:
//
//   norm_g = sqrt( sum over tensors of sum over group g of v^2 )
//   out    = v * min(1, max_norm / (norm_g + 1e-6))
//
// A tensor's elements fall into `groups` equal consecutive parts (one an adapter),
// a part into pieces; a workgroup takes a piece.  The first launch writes a
// piece's sum of squares, the second adds a group's sums in their order (every
// workgroup for itself: the same order, so the same bits) and scales the piece.
// Both are bound by the bytes: read once for the norm, read and written once
// for the scaling.  Where they are more than the last-level cache holds, the scaling
// walks the pieces of a launch backwards, from what the norms' launch read last, and all
// else is read and written past the cache: the gradients of 128 adapters of rank 128
// (1.14 GB of bfloat16) take 167 and 411 us, 6.8 and 5.5 TB/s; without either 227 and 425,
// with the walk alone 209 and 418.  More tensors than a launch describes (246, 164 with
// results of their own) take several launches of either kind in the same order, and the
// cache then holds the end of the last one: 448 tensors of 2 MB 489 us in place and 508
// into results, one of as many bytes 491 and 474.
//
// Squares and sums are double: the square of a float32 may be beyond float32, and
// the rate (a conversion and a multiply-add an element) is far from a bound.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "lora_internal.h"

namespace lora {
namespace {

constexpr int kThreads = 256;
constexpr size_t kArgBytes = 4000;               // of a launch, for its tensors' descriptions
constexpr long kMinPiece = 32 << 10, kMaxPiece = 256 << 10, kPieces = 4096;   // bytes; pieces that are enough
// (bfloat16 of 1088 MB in pieces of 32, 64, 128, 256 and 512 KB: 561, 585, 568, 571, 580 us;
// 32 MB: 22, 22, 23, 28, 44; 8 MB: 10, 13, 16, 23, 37.)
// Partial sums of a group that every workgroup adds up by itself; more are added
// once, by a launch of their own: 1024 sums 9.2 us the one way and 9.6 the other, 2048
// 19.4 and 18.7, 4096 37 and 31.
constexpr int kSelfSums = 2048;
constexpr int64_t kMaxUnits = 1 << 23;   // workgroups of a launch
// Gradients of so many bytes do not stay in the 256 MB of last-level cache from one
// launch to the next; the end that the first launch leaves there.  us into the cache and
// past it, with results of their own: 160 MB 87, 85; 192 MB 107, 100; 256 MB 155, 136;
// in place, where half as much is touched, 192 MB 96, 105; 320 MB 165, 172; 512 MB 292,
// 276 (the limit is that of results).  Kept, 320 MB in place: nothing 182, 64 MB 176, 128 MB
// 173, 160 MB 168, 192 MB 166, 224 MB 163; 1088 MB 602, 595, 578, 581, 577, 580.
constexpr int64_t kStreamBytes = 192 << 20, kKeptBytes = 160 << 20;

// A factor as a float and a power of two: gradients near 2^128 and a small largest norm
// give factors far below float32's (the product with the float is rounded in its normal
// range, and the power then rounds subnormal results alone).
struct Factor {
    float first;
    int power;
    __device__ __forceinline__ float of(float v) const { return __builtin_amdgcn_ldexpf(v * first, power); }
    __device__ __forceinline__ bool one() const { return first == 1.f && power == 0; }
};

struct ClipTensor {
    const void *in;
    uint32_t part;       // elements of one group
    uint32_t first;      // first piece (of a group) of this tensor, counted over the call's tensors; top bit: float32
};
// What every launch has, and its tensors: results of their own (OUT), or in place.
struct ClipCall {
    double *sums;        // [groups][pieces of a group]
    Factor *factors;     // [groups] where a launch of its own makes them, or NULL
    float *norms;
    double max_norm;
    int32_t count, first, pieces, all_pieces;   // tensors; pieces of a group: first of this launch, of it, of the call
    int32_t piece, stream;                      // bytes of a piece; more than the cache holds
};
template <bool OUT>
struct ClipArgs {
    static constexpr int kTensors = (int)((kArgBytes - sizeof(ClipCall)) / (sizeof(ClipTensor) + (OUT ? sizeof(void *) : 0)));
    ClipCall c;
    ClipTensor t[kTensors];
    void *out[OUT ? kTensors : 1];
};

template <class F>
__device__ __forceinline__ void add_vector(const u32x4 &v, double &sum, F) {
    if (sizeof(F) == 2) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const double a = bf16_bits_to_float(v[x] & 0xffffu), b = bf16_bits_to_float(v[x] >> 16);
            sum = fma(a, a, sum);
            sum = fma(b, b, sum);
        }
    } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const double a = __uint_as_float(v[x]);
            sum = fma(a, a, sum);
        }
    }
}
__device__ __forceinline__ float value(uint16_t v) { return bf16_bits_to_float(v); }
__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ void store(uint16_t *p, float v) { *p = (uint16_t)float_to_bf16_bits(v); }
__device__ __forceinline__ void store(float *p, float v) { *p = v; }
__device__ __forceinline__ u32x4 scaled(const u32x4 &v, Factor f, uint16_t) {
    u32x4 r;
#pragma unroll
    for (int x = 0; x < 4; ++x)
        r[x] = float_to_bf16_bits(f.of(bf16_bits_to_float(v[x] & 0xffffu))) | float_to_bf16_bits(f.of(bf16_bits_to_float(v[x] >> 16))) << 16;
    return r;
}
__device__ __forceinline__ u32x4 scaled(const u32x4 &v, Factor f, float) {
    u32x4 r;
#pragma unroll
    for (int x = 0; x < 4; ++x) r[x] = __float_as_uint(f.of(__uint_as_float(v[x])));
    return r;
}

// The sum over the workgroup, in thread 0 (and in a fixed order).
__device__ __forceinline__ double workgroup_sum(double v) {
    __shared__ double s_part[kThreads / kWave];
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if (lane_id() == 0) s_part[wave_id()] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) v += s_part[w];
    __syncthreads();
    return v;
}

struct Piece {
    int tensor, group, index;    // index: of the group's pieces, over the call
    bool wide;                   // float32
    int64_t at, count;           // first element of the tensor, elements
};
template <class A>
__device__ __forceinline__ Piece piece_at(const A &a, int64_t unit) {
    Piece p;
    p.group = (int)(unit / a.c.pieces);
    p.index = a.c.first + (int)(unit - (int64_t)p.group * a.c.pieces);
    int lo = 0, hi = a.c.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if ((int)(a.t[mid].first & 0x7fffffffu) <= p.index)
            lo = mid;
        else
            hi = mid;
    }
    p.tensor = lo;
    const ClipTensor t = a.t[lo];
    p.wide = t.first >> 31 != 0;
    const int64_t each = a.c.piece / (p.wide ? 4 : 2), in = (p.index - (int)(t.first & 0x7fffffffu)) * each;
    p.at = (int64_t)p.group * t.part + in;
    p.count = t.part - in < each ? t.part - in : each;
    return p;
}

// Elements before the first 16-byte boundary.
template <class F>
__device__ __forceinline__ int64_t head_of(const F *p, int64_t count) {
    const int64_t h = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(F);
    return h < count ? h : count;
}

constexpr int kBatch = 8;   // vectors of a thread in flight

// PAST: past the last-level cache.
template <bool PAST>
__device__ __forceinline__ u32x4 load(const u32x4 *p) {
    return PAST ? __builtin_nontemporal_load(p) : *p;
}
template <bool PAST>
__device__ __forceinline__ void put(u32x4 *p, const u32x4 &v) {
    if (PAST)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}

template <bool PAST, class F>
__device__ __forceinline__ double squares(const F *p, int64_t count) {
    const int tid = threadIdx.x;
    double sum = 0.0;
    const int64_t head = head_of(p, count);
    if (tid < head) {
        const double v = value(p[tid]);
        sum = v * v;
    }
    constexpr int kVec = 16 / (int)sizeof(F);
    const u32x4 *q = reinterpret_cast<const u32x4 *>(p + head);
    const int64_t vectors = (count - head) / kVec;
    int64_t i = tid;
    for (; i + (kBatch - 1) * kThreads < vectors; i += kBatch * kThreads) {
        u32x4 v[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) v[b] = load<PAST>(q + i + b * kThreads);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) add_vector(v[b], sum, F());
    }
    for (; i < vectors; i += kThreads) add_vector(q[i], sum, F());
    const int64_t rest = head + vectors * kVec + tid;
    if (rest < count) {
        const double v = value(p[rest]);
        sum = fma(v, v, sum);
    }
    return sum;
}

template <bool PAST, class F>
__device__ __forceinline__ void scale_piece(const F *p, F *o, int64_t count, Factor f) {
    const int tid = threadIdx.x;
    const bool keep = f.one();   // bit for bit: a product with 1 changes NaN
    auto one = [&](int64_t i) {
        if (keep)
            o[i] = p[i];
        else
            store(o + i, f.of(value(p[i])));
    };
    if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) != 0) {
        for (int64_t i = tid; i < count; i += kThreads) one(i);
        return;
    }
    auto many = [&](const u32x4 &v) {
        const u32x4 s = scaled(v, f, F());
        return u32x4{keep ? v[0] : s[0], keep ? v[1] : s[1], keep ? v[2] : s[2], keep ? v[3] : s[3]};
    };
    const int64_t head = head_of(p, count);
    if (tid < head) one(tid);
    constexpr int kVec = 16 / (int)sizeof(F);
    const u32x4 *q = reinterpret_cast<const u32x4 *>(p + head);
    u32x4 *r = reinterpret_cast<u32x4 *>(o + head);
    const int64_t vectors = (count - head) / kVec;
    int64_t i = tid;
    for (; i + (kBatch - 1) * kThreads < vectors; i += kBatch * kThreads) {
        u32x4 v[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) v[b] = load<PAST>(q + i + b * kThreads);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) put<PAST>(r + i + b * kThreads, many(v[b]));
    }
    for (; i < vectors; i += kThreads) r[i] = many(q[i]);
    const int64_t rest = head + vectors * kVec + tid;
    if (rest < count) one(rest);
}

__global__ __launch_bounds__(kThreads) void squares_kernel(ClipArgs<false> a) {
    const Piece p = piece_at(a, blockIdx.x);
    const uint16_t *half = static_cast<const uint16_t *>(a.t[p.tensor].in) + p.at;
    const float *wide = static_cast<const float *>(a.t[p.tensor].in) + p.at;
    const bool past = a.c.stream && (int64_t)(gridDim.x - blockIdx.x) * a.c.piece > kKeptBytes;
    double sum;
    if (past)
        sum = p.wide ? squares<true>(wide, p.count) : squares<true>(half, p.count);
    else
        sum = p.wide ? squares<false>(wide, p.count) : squares<false>(half, p.count);
    sum = workgroup_sum(sum);
    if (threadIdx.x == 0) a.c.sums[(int64_t)p.group * a.c.all_pieces + p.index] = sum;
}

// A group's norm and factor; 1 where its gradients stay as they are (also where the norm is not finite).
__device__ __forceinline__ Factor factor_of(const ClipCall &c, int group, float &norm) {
    const double *sums = c.sums + (int64_t)group * c.all_pieces;
    double v = 0.0;
    for (int i = threadIdx.x; i < c.all_pieces; i += kThreads) v += sums[i];
    const double n = sqrt(workgroup_sum(v));
    norm = (float)n;
    const double f = c.max_norm / (n + 1e-6);
    if (!(n < __builtin_huge_val() && f < 1.0)) return Factor{1.f, 0};
    if (f >= 0x1p-60) return Factor{(float)f, 0};
    int power;
    const float first = (float)frexp(f, &power);
    return Factor{first, power};
}

__global__ __launch_bounds__(kThreads) void factors_kernel(ClipCall c) {
    float norm;
    const Factor f = factor_of(c, blockIdx.x, norm);
    if (threadIdx.x == 0) {
        c.norms[blockIdx.x] = norm;
        if (c.factors) c.factors[blockIdx.x] = f;
    }
}

template <bool OUT>
__global__ __launch_bounds__(kThreads) void scale_kernel(ClipArgs<OUT> a) {
    const Piece p = piece_at(a, (int64_t)gridDim.x - 1 - blockIdx.x);
    Factor f;
    if (a.c.factors) {
        f = a.c.factors[p.group];
    } else {
        float norm;
        f = factor_of(a.c, p.group, norm);
        if (p.index == 0 && threadIdx.x == 0) a.c.norms[p.group] = norm;
    }
    const void *in = a.t[p.tensor].in;
    void *out = OUT ? a.out[p.tensor] : const_cast<void *>(in);
    if (f.one() && in == out) return;
    const uint16_t *half = static_cast<const uint16_t *>(in) + p.at;
    const float *wide = static_cast<const float *>(in) + p.at;
    uint16_t *half_out = static_cast<uint16_t *>(out) + p.at;
    float *wide_out = static_cast<float *>(out) + p.at;
    if (a.c.stream) {
        if (p.wide)
            scale_piece<true>(wide, wide_out, p.count, f);
        else
            scale_piece<true>(half, half_out, p.count, f);
    } else {
        if (p.wide)
            scale_piece<false>(wide, wide_out, p.count, f);
        else
            scale_piece<false>(half, half_out, p.count, f);
    }
}

int size_of(int type) { return type == LORA_BF16 ? 2 : 4; }

int check_tensors(const int64_t *sizes, const int *types, int num_tensors, int groups) {
    if (groups < 1 || groups > LORA_MAX_LORAS) return LORA_ERR_MAX_LORAS;
    if (num_tensors < 0 || num_tensors > LORA_MAX_TENSORS) return LORA_ERR_SLICES;
    if (num_tensors && (!sizes || !types)) return LORA_ERR_NULL;
    for (int i = 0; i < num_tensors; ++i)
        if (sizes[i] < 0 || sizes[i] % groups || sizes[i] / groups > UINT32_MAX || (types[i] != LORA_BF16 && types[i] != LORA_F32))
            return LORA_ERR_SHAPE;
    return LORA_OK;
}

struct ClipPlan {
    int64_t piece, pieces;     // bytes; pieces of a group
    bool stream;
    size_t factors, total;     // workspace
};
ClipPlan plan_clip(const int64_t *sizes, const int *types, int num_tensors, int groups) {
    ClipPlan p;
    double bytes = 0;
    for (int i = 0; i < num_tensors; ++i) bytes += (double)sizes[i] * size_of(types[i]);
    p.piece = kMinPiece;
    while (p.piece < kMaxPiece && (double)p.piece * kPieces < bytes) p.piece *= 2;
    p.stream = bytes > (double)kStreamBytes;
    p.pieces = 0;
    for (int i = 0; i < num_tensors; ++i) {
        const int64_t part = sizes[i] / groups * size_of(types[i]);
        p.pieces += (part + p.piece - 1) / p.piece;
    }
    p.factors = ((size_t)p.pieces * groups * sizeof(double) + 255) / 256 * 256;
    p.total = p.factors + ((size_t)groups * sizeof(Factor) + 255) / 256 * 256;
    return p;
}

// Whether no result shares memory with another (one in two places would be scaled twice, or
// by whoever comes last) or with a gradient but its own in its own place (it would be scaled
// after it was written over).
struct Span {
    uintptr_t at, end;
};
std::vector<Span> spans_of(const void *const *p, const void *const *but, const int64_t *sizes, const int *types, int num_tensors) {
    std::vector<Span> spans;
    spans.reserve((size_t)num_tensors);
    bool ordered = true;   // (buffers made one after the other are: no sort)
    for (int i = 0; i < num_tensors; ++i) {
        if (!sizes[i] || (but && p[i] == but[i])) continue;
        const uintptr_t at = reinterpret_cast<uintptr_t>(p[i]);
        ordered = ordered && (spans.empty() || at >= spans.back().at);
        spans.push_back(Span{at, at + (uintptr_t)sizes[i] * (uintptr_t)size_of(types[i])});
    }
    if (!ordered) std::sort(spans.begin(), spans.end(), [](const Span &a, const Span &b) { return a.at < b.at; });
    return spans;
}
bool apart(const void *const *grads, void *const *out, const int64_t *sizes, const int *types, int num_tensors) {
    const std::vector<Span> written = spans_of(out, nullptr, sizes, types, num_tensors), read = spans_of(grads, out, sizes, types, num_tensors);
    uintptr_t written_to = 0, read_to = 0;
    auto in = read.begin();
    for (const Span &o : written) {
        for (; in != read.end() && in->at <= o.at; ++in) {
            if (in->at < written_to) return false;
            read_to = std::max(read_to, in->end);
        }
        if (o.at < written_to || o.at < read_to) return false;
        written_to = o.end;
    }
    return in == read.end() || in->at >= written_to;
}

// The tensors in launches of as many as their arguments hold.
struct ClipList {
    const void *const *grads;
    void *const *out;
    const int64_t *sizes;
    const int *types;
    int num_tensors, groups;
    int64_t piece;
};
template <bool OUT, class K>
int each_launch(const ClipList &l, const ClipCall &c, K kernel, hipStream_t stream) {
    ClipArgs<OUT> a;
    a.c = c;
    int64_t at = 0;
    for (int i = 0; i < l.num_tensors;) {
        a.c.count = 0;
        a.c.first = (int32_t)at;
        for (; i < l.num_tensors && a.c.count < ClipArgs<OUT>::kTensors; ++i) {
            const int64_t part = l.sizes[i] / l.groups;
            if (part == 0) continue;
            a.t[a.c.count] = ClipTensor{l.grads[i], (uint32_t)part, (uint32_t)at | (l.types[i] == LORA_F32 ? 0x80000000u : 0u)};
            if (OUT) a.out[a.c.count] = l.out[i];
            ++a.c.count;
            at += (part * size_of(l.types[i]) + l.piece - 1) / l.piece;
        }
        a.c.pieces = (int32_t)(at - a.c.first);
        if (a.c.count == 0) break;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(a.c.pieces * (int64_t)l.groups)), dim3(kThreads), 0, stream, a);
        if (hipGetLastError() != hipSuccess) return LORA_ERR_LAUNCH;
    }
    return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t lora_clip_gradients_workspace_bytes(const int64_t *sizes, const int *types, int num_tensors, int groups) {
    if (check_tensors(sizes, types, num_tensors, groups)) return 0;
    const ClipPlan p = plan_clip(sizes, types, num_tensors, groups);
    return p.pieces * groups > kMaxUnits ? 0 : p.total;
}

int lora_clip_gradients(const void *const *grads, void *const *out, const int64_t *sizes, const int *types,
                        int num_tensors, int groups, double max_norm, float *norms, void *workspace,
                        size_t workspace_bytes, hipStream_t stream) {
    int st = check_tensors(sizes, types, num_tensors, groups);
    if (st) return st;
    if (!(max_norm > 0.0)) return LORA_ERR_SHAPE;
    if (!norms || !workspace || (num_tensors && (!grads || !out))) return LORA_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(norms) & 3u) != 0) return LORA_ERR_ALIGN;
    const ClipPlan p = plan_clip(sizes, types, num_tensors, groups);
    if (p.pieces * groups > kMaxUnits) return LORA_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || p.total > workspace_bytes) return LORA_ERR_BUFFER;
    bool same = true;
    for (int i = 0; i < num_tensors; ++i) {
        if (!sizes[i]) continue;
        if (!grads[i] || !out[i]) return LORA_ERR_NULL;
        if (((reinterpret_cast<uintptr_t>(grads[i]) | reinterpret_cast<uintptr_t>(out[i])) & (size_of(types[i]) - 1)) != 0)
            return LORA_ERR_ALIGN;
        same = same && grads[i] == out[i];
    }
    try {
        if (!apart(grads, out, sizes, types, num_tensors)) return LORA_ERR_BUFFER;
    } catch (...) {   // (no memory for the spans)
        return LORA_ERR_SCRATCH;
    }

    ClipCall c;
    memset(&c, 0, sizeof c);
    c.sums = static_cast<double *>(workspace);
    c.norms = norms;
    c.max_norm = max_norm;
    c.all_pieces = (int32_t)p.pieces;
    c.piece = (int32_t)p.piece;
    c.stream = p.stream;
    const bool only_norms = same && isinf(max_norm), own_launch = only_norms || p.pieces > kSelfSums || p.pieces == 0;
    const ClipList list = {grads, out, sizes, types, num_tensors, groups, p.piece};
    if ((st = each_launch<false>(list, c, squares_kernel, stream))) return st;
    if (own_launch) {
        if (!only_norms) c.factors = reinterpret_cast<Factor *>(static_cast<char *>(workspace) + p.factors);
        hipLaunchKernelGGL(factors_kernel, dim3((unsigned)groups), dim3(kThreads), 0, stream, c);
        if (hipGetLastError() != hipSuccess) return LORA_ERR_LAUNCH;
        if (only_norms) return LORA_OK;
    }
    return same ? each_launch<false>(list, c, scale_kernel<false>, stream) : each_launch<true>(list, c, scale_kernel<true>, stream);
}

}  // extern "C"
