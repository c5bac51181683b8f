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
// for the scaling, which walks the pieces backwards, so that what the first
// launch read last is still in the last-level cache.
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

constexpr int kThreads = 256, kTensors = 120;   // tensors a launch takes: its arguments stay below 4 KB
constexpr long kMinPiece = 32 << 10, kMaxPiece = 256 << 10, kPieces = 4096;   // bytes; pieces that are enough
// Partial sums of a group that every workgroup adds up by itself; more are added
// once, by a launch of their own.
constexpr int kSelfSums = 2048;
constexpr int64_t kMaxUnits = 1 << 23;   // workgroups of a launch

// A factor as two floats, v * first * second: one below 2^-60 by itself could be
// subnormal and have lost its digits.
struct Factor {
    float first, second;
    __device__ __forceinline__ float of(float v) const { return v * first * second; }
    __device__ __forceinline__ bool one() const { return first == 1.f && second == 1.f; }
};

struct ClipTensor {
    const void *in;
    void *out;
    int64_t part;        // elements of one group
    int32_t first;       // first piece (of a group) of this tensor, counted over the call's tensors
    int32_t type;
};
struct ClipArgs {
    ClipTensor t[kTensors];
    double *sums;        // [groups][pieces of a group]
    Factor *factors;     // [groups] where a launch of its own makes them, or NULL
    float *norms;
    double max_norm;
    int32_t count, groups, first, pieces, all_pieces;   // tensors; pieces of a group: first of this launch, of it, of the call
    int32_t piece;       // bytes
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
    int64_t at;                  // first element of the tensor
    int64_t count;
};
__device__ __forceinline__ Piece piece_at(const ClipArgs &a, int64_t unit) {
    Piece p;
    p.group = (int)(unit / a.pieces);
    p.index = a.first + (int)(unit - (int64_t)p.group * a.pieces);
    int lo = 0, hi = a.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.t[mid].first <= p.index)
            lo = mid;
        else
            hi = mid;
    }
    p.tensor = lo;
    const int64_t each = a.piece / (a.t[lo].type == LORA_BF16 ? 2 : 4), part = a.t[lo].part;
    const int64_t in = (p.index - a.t[lo].first) * each;
    p.at = p.group * part + in;
    p.count = part - in < each ? part - in : each;
    return p;
}

// Elements before the first 16-byte boundary.
template <class F>
__device__ __forceinline__ int64_t head_of(const F *p, int64_t count) {
    const int64_t h = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(F);
    return h < count ? h : count;
}

constexpr int kBatch = 8;   // vectors of a thread in flight

template <class F>
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
        for (int b = 0; b < kBatch; ++b) v[b] = q[i + b * kThreads];
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

template <class F>
__device__ __forceinline__ void scale_piece(const F *p, F *o, int64_t count, Factor f) {
    const int tid = threadIdx.x;
    if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) != 0) {
        for (int64_t i = tid; i < count; i += kThreads) store(o + i, f.of(value(p[i])));
        return;
    }
    const int64_t head = head_of(p, count);
    if (tid < head) store(o + tid, f.of(value(p[tid])));
    constexpr int kVec = 16 / (int)sizeof(F);
    const u32x4 *q = reinterpret_cast<const u32x4 *>(p + head);
    u32x4 *r = reinterpret_cast<u32x4 *>(o + head);
    const int64_t vectors = (count - head) / kVec;
    int64_t i = tid;
    for (; i + (kBatch - 1) * kThreads < vectors; i += kBatch * kThreads) {
        u32x4 v[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) v[b] = q[i + b * kThreads];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) r[i + b * kThreads] = scaled(v[b], f, F());
    }
    for (; i < vectors; i += kThreads) r[i] = scaled(q[i], f, F());
    const int64_t rest = head + vectors * kVec + tid;
    if (rest < count) store(o + rest, f.of(value(p[rest])));
}

__global__ __launch_bounds__(kThreads) void squares_kernel(ClipArgs a) {
    const Piece p = piece_at(a, blockIdx.x);
    const ClipTensor &t = a.t[p.tensor];
    double sum = t.type == LORA_BF16 ? squares(static_cast<const uint16_t *>(t.in) + p.at, p.count)
                                     : squares(static_cast<const float *>(t.in) + p.at, p.count);
    sum = workgroup_sum(sum);
    if (threadIdx.x == 0) a.sums[(int64_t)p.group * a.all_pieces + p.index] = sum;
}

// A group's norm and factor; 1 where its gradients stay as they are (also where the norm is not finite).
__device__ __forceinline__ Factor factor_of(const ClipArgs &a, int group, float &norm) {
    const double *sums = a.sums + (int64_t)group * a.all_pieces;
    double v = 0.0;
    for (int i = threadIdx.x; i < a.all_pieces; i += kThreads) v += sums[i];
    const double n = sqrt(workgroup_sum(v));
    norm = (float)n;
    const double f = a.max_norm / (n + 1e-6);
    if (!(n < __builtin_huge_val() && f < 1.0)) return Factor{1.f, 1.f};
    return f < 0x1p-60 ? Factor{(float)(f * 0x1p60), 0x1p-60f} : Factor{(float)f, 1.f};
}

__global__ __launch_bounds__(kThreads) void factors_kernel(ClipArgs a) {
    float norm;
    const Factor f = factor_of(a, blockIdx.x, norm);
    if (threadIdx.x == 0) {
        a.norms[blockIdx.x] = norm;
        if (a.factors) a.factors[blockIdx.x] = f;
    }
}

__global__ __launch_bounds__(kThreads) void scale_kernel(ClipArgs a) {
    const Piece p = piece_at(a, (int64_t)gridDim.x - 1 - blockIdx.x);
    const ClipTensor &t = a.t[p.tensor];
    Factor f;
    if (a.factors) {
        f = a.factors[p.group];
    } else {
        float norm;
        f = factor_of(a, p.group, norm);
        if (p.index == 0 && threadIdx.x == 0) a.norms[p.group] = norm;
    }
    if (f.one() && t.in == t.out) return;
    if (t.type == LORA_BF16)
        scale_piece(static_cast<const uint16_t *>(t.in) + p.at, static_cast<uint16_t *>(t.out) + p.at, p.count, f);
    else
        scale_piece(static_cast<const float *>(t.in) + p.at, static_cast<float *>(t.out) + p.at, p.count, f);
}

int size_of(int type) { return type == LORA_BF16 ? 2 : 4; }

int check_tensors(const int64_t *sizes, const int *types, int num_tensors, int groups) {
    if (groups < 1 || groups > LORA_MAX_LORAS) return LORA_ERR_MAX_LORAS;
    if (num_tensors < 0 || num_tensors > LORA_MAX_TENSORS) return LORA_ERR_SLICES;
    if (num_tensors && (!sizes || !types)) return LORA_ERR_NULL;
    for (int i = 0; i < num_tensors; ++i)
        if (sizes[i] < 0 || sizes[i] % groups || sizes[i] > ((int64_t)1 << 40) || (types[i] != LORA_BF16 && types[i] != LORA_F32))
            return LORA_ERR_SHAPE;
    return LORA_OK;
}

struct ClipPlan {
    int64_t piece, pieces;     // bytes; pieces of a group
    size_t factors, total;     // workspace
};
ClipPlan plan_clip(const int64_t *sizes, const int *types, int num_tensors, int groups) {
    ClipPlan p;
    double bytes = 0;
    for (int i = 0; i < num_tensors; ++i) bytes += (double)sizes[i] * size_of(types[i]);
    p.piece = kMinPiece;
    while (p.piece < kMaxPiece && (double)p.piece * kPieces < bytes) p.piece *= 2;
    p.pieces = 0;
    for (int i = 0; i < num_tensors; ++i) {
        const int64_t part = sizes[i] / groups * size_of(types[i]);
        p.pieces += (part + p.piece - 1) / p.piece;
    }
    p.factors = ((size_t)p.pieces * groups * sizeof(double) + 255) / 256 * 256;
    p.total = p.factors + ((size_t)groups * sizeof(Factor) + 255) / 256 * 256;
    return p;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t lora_clip_gradients_workspace_bytes(const int64_t *sizes, const int *types, int num_tensors, int groups) {
    if (check_tensors(sizes, types, num_tensors, groups)) return 0;
    return plan_clip(sizes, types, num_tensors, groups).total;
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
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || p.total > workspace_bytes) return LORA_ERR_BUFFER;
    if (p.pieces * groups > kMaxUnits) return LORA_ERR_SHAPE;
    bool same = true;
    for (int i = 0; i < num_tensors; ++i) {
        if (!sizes[i]) continue;
        if (!grads[i] || !out[i]) return LORA_ERR_NULL;
        if (((reinterpret_cast<uintptr_t>(grads[i]) | reinterpret_cast<uintptr_t>(out[i])) & (size_of(types[i]) - 1)) != 0)
            return LORA_ERR_ALIGN;
        same = same && grads[i] == out[i];
    }
    // two results in one place would be scaled twice, or by whoever comes last
    try {
        std::vector<std::pair<uintptr_t, uintptr_t>> spans;
        spans.reserve((size_t)num_tensors);
        for (int i = 0; i < num_tensors; ++i)
            if (sizes[i]) {
                const uintptr_t at = reinterpret_cast<uintptr_t>(out[i]);
                spans.emplace_back(at, at + (uintptr_t)sizes[i] * (uintptr_t)size_of(types[i]));
            }
        std::sort(spans.begin(), spans.end());
        for (size_t i = 1; i < spans.size(); ++i)
            if (spans[i].first < spans[i - 1].second) return LORA_ERR_BUFFER;
    } catch (...) {
        return LORA_ERR_SCRATCH;
    }

    ClipArgs a;
    memset(&a, 0, sizeof a);
    a.sums = static_cast<double *>(workspace);
    a.norms = norms;
    a.max_norm = max_norm;
    a.groups = groups;
    a.all_pieces = (int32_t)p.pieces;
    a.piece = (int32_t)p.piece;
    const bool only_norms = same && isinf(max_norm), own_launch = only_norms || p.pieces > kSelfSums || p.pieces == 0;
    Factor *factors = reinterpret_cast<Factor *>(static_cast<char *>(workspace) + p.factors);
    // the tensors in launches of kTensors each
    auto each_launch = [&](auto kernel, Factor *given) -> int {
        int64_t at = 0;
        a.factors = given;
        for (int i = 0; i < num_tensors;) {
            a.count = 0;
            a.first = (int32_t)at;
            for (; i < num_tensors && a.count < kTensors; ++i) {
                const int64_t part = sizes[i] / groups;
                if (part == 0) continue;
                a.t[a.count++] = ClipTensor{grads[i], out[i], part, (int32_t)at, types[i]};
                at += (part * size_of(types[i]) + p.piece - 1) / p.piece;
            }
            a.pieces = (int32_t)(at - a.first);
            if (a.count == 0) break;
            hipLaunchKernelGGL(kernel, dim3((unsigned)(a.pieces * (int64_t)groups)), dim3(kThreads), 0, stream, a);
            if (hipGetLastError() != hipSuccess) return LORA_ERR_LAUNCH;
        }
        return LORA_OK;
    };
    if ((st = each_launch(squares_kernel, nullptr))) return st;
    if (own_launch) {
        a.factors = only_norms ? nullptr : factors;
        hipLaunchKernelGGL(factors_kernel, dim3((unsigned)groups), dim3(kThreads), 0, stream, a);
        if (hipGetLastError() != hipSuccess) return LORA_ERR_LAUNCH;
        if (only_norms) return LORA_OK;
    }
    return each_launch(scale_kernel, own_launch ? factors : nullptr);
}

}  // extern "C"
