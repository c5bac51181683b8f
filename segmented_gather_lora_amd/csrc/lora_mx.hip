// lora_mx.hip -- microscaled 4-bit numbers (E2M1 codes with a power of two for
// every 32 of a row): from and to bfloat16 and float32, and the entry points of the
// shared projection with adapters whose matrix is held so.
#include "lora_linear.h"

using namespace lora;

namespace lora {
namespace {

// Bound by the bytes.  28672 rows of 4096: from bf16 53 to 65 us (57 at the least beside
// other calls, 5.2 TB/s), back 50 (5.9); from float32 96 (5.5), back 122 (4.4).
template <class F>
__global__ __launch_bounds__(kMxThreads) void quantize_kernel(MxArgs a) {
    constexpr int kSpans = kMxThreads / kMxGroup;
    const int l = threadIdx.x % kMxGroup, g = threadIdx.x / kMxGroup;
    float v[kMxPer][8];
    MxAt at[kMxPer];
#pragma unroll
    for (int q = 0; q < kMxPer; ++q) {
        at[q] = mx_at((int64_t)blockIdx.x * (kSpans * kMxPer), q * kSpans + g, a.spans);
        const int k = at[q].span * kMxSpan + 8 * l;
        mx_load(reinterpret_cast<const F *>(a.x + at[q].row * a.ldx) + k, at[q].row < a.rows && k < a.cols, v[q]);
    }
#pragma unroll
    for (int q = 0; q < kMxPer; ++q) {
        uint32_t top = 0;
#pragma unroll
        for (int x = 0; x < 8; ++x) top = max(top, __float_as_uint(v[q][x]) & 0x7fffffffu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        const int scale = mx_scale_of(top), block = at[q].span * 4 + l / 4;
        const uint32_t codes = mx_codes_of(v[q], scale);
        // four blocks' bytes to one lane
        uint32_t s = block < a.blocks ? (uint32_t)scale << 8 * (l / 4) : 0u;
        s |= (uint32_t)__shfl_xor((int)s, 4);
        s |= (uint32_t)__shfl_xor((int)s, 8);
        if (at[q].row >= a.rows) continue;
        if (block < a.blocks)
            *reinterpret_cast<uint32_t *>(a.codes + at[q].row * a.ldcodes + at[q].span * 64 + 4 * l) = codes;
        if (l == 0) *reinterpret_cast<uint32_t *>(a.scales + at[q].row * a.ldscales + at[q].span * 4) = s;
    }
}

template <class F>
__global__ __launch_bounds__(kMxThreads) void dequantize_kernel(MxArgs a) {
    dequantize<F>(a, blockIdx.x);
}

int check_codes(const void *codes, int64_t ldcodes, const void *scales, int64_t ldscales, int64_t rows, int64_t cols) {
    if (rows < 0 || rows > INT32_MAX || cols < 8 || cols % 8 || cols > LORA_MAX_HIDDEN) return LORA_ERR_SHAPE;
    if (ldcodes < mx_code_bytes(cols) || ldcodes % 16 || ldscales < mx_scale_bytes(cols) || ldscales % 4) return LORA_ERR_SHAPE;
    if (rows > 0 && (!codes || !scales)) return LORA_ERR_NULL;
    if (!aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & 3u) != 0) return LORA_ERR_ALIGN;
    return LORA_OK;
}

// The numbers' own checks: bfloat16 or float32 rows.
int check_numbers(const void *x, int type, int64_t ldx, int64_t rows, int64_t cols) {
    if (type != LORA_BF16 && type != LORA_F32) return LORA_ERR_SHAPE;
    if (ldx < cols || ldx % (type == LORA_BF16 ? 8 : 4)) return LORA_ERR_SHAPE;
    if (rows > 0 && !x) return LORA_ERR_NULL;
    return aligned16(x) ? LORA_OK : LORA_ERR_ALIGN;
}

// Rows to (TO) or from codes.
template <bool TO>
hipError_t launch_mx(const void *x, int type, int64_t ldx, int64_t rows, int cols, const void *codes, int64_t ldcodes,
                     const void *scales, int64_t ldscales, hipStream_t s) {
    const MxArgs all = mx_args(x, type, ldx, rows, cols, codes, ldcodes, scales, ldscales);
    const int64_t most = kMxMostBlocks * kMxSpans / all.spans;
    for (int64_t r = 0; r < rows; r += most) {
        MxArgs a = all;
        a.rows = rows - r < most ? rows - r : most;
        a.x += r * a.ldx;
        a.codes += r * ldcodes;
        a.scales += r * ldscales;
        const dim3 grid((unsigned)mx_grid(a)), block(kMxThreads);
        if (TO && type == LORA_BF16)
            hipLaunchKernelGGL(quantize_kernel<uint16_t>, grid, block, 0, s, a);
        else if (TO)
            hipLaunchKernelGGL(quantize_kernel<float>, grid, block, 0, s, a);
        else if (type == LORA_BF16)
            hipLaunchKernelGGL(dequantize_kernel<uint16_t>, grid, block, 0, s, a);
        else
            hipLaunchKernelGGL(dequantize_kernel<float>, grid, block, 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// ---------------------------------------------------------------- plans

// Rows of the matrix' codes are this far apart at most: a tile's 128 rows are within 32 bits.
constexpr int64_t kMaxPitch = 1 << 25;

// The workspace: that of the bf16 projection, then its matrix as numbers, or what
// prep_kernel writes (no call has both; the forward pass of few tokens has neither).
struct MxLayout {
    size_t w, codes, scales, mscales, total;
    int steps;
};
MxLayout mx_layout(size_t linear, long n, int hidden, int out, bool backward) {
    MxLayout l;
    l.steps = (int)((mx_blocks(hidden) + 7) / 8);
    const size_t groups = (size_t)(n + 255) / 256 * 4, wide = (size_t)(out + 255) / 256 * 4;   // whole tiles
    l.w = linear;
    l.codes = linear;
    l.scales = l.codes + up((size_t)n * mx_code_bytes(hidden));
    l.mscales = l.scales + up(groups * l.steps * 512);
    const size_t numbers = l.w + up(2 * (size_t)out * hidden), codes = l.mscales + up(wide * l.steps * 512);
    l.total = !backward && n <= kRowsTokens ? linear : numbers > codes ? numbers : codes;
    return l;
}

}  // namespace
}  // namespace lora

extern "C" {

int lora_mx_quantize(const void *x, int type, int64_t ldx, int64_t rows, int cols, void *codes, int64_t ldcodes,
                     void *scales, int64_t ldscales, hipStream_t stream) {
    int st = check_codes(codes, ldcodes, scales, ldscales, rows, cols);
    if (st || (st = check_numbers(x, type, ldx, rows, cols))) return st;
    return launch_mx<true>(x, type, ldx, rows, cols, codes, ldcodes, scales, ldscales, stream) == hipSuccess ? LORA_OK
                                                                                                             : LORA_ERR_LAUNCH;
}

int lora_mx_dequantize(const void *codes, int64_t ldcodes, const void *scales, int64_t ldscales, int64_t rows, int cols,
                       void *out, int type, int64_t ldout, hipStream_t stream) {
    int st = check_codes(codes, ldcodes, scales, ldscales, rows, cols);
    if (st || (st = check_numbers(out, type, ldout, rows, cols))) return st;
    return launch_mx<false>(out, type, ldout, rows, cols, codes, ldcodes, scales, ldscales, stream) == hipSuccess
               ? LORA_OK
               : LORA_ERR_LAUNCH;
}

size_t lora_linear_mx_workspace_bytes(int num_tokens, int max_loras, int hidden, int out_features, const int *slice_widths,
                                      int num_slices, int rank, int backward) {
    if (check_sizes(num_tokens, max_loras, hidden, slice_widths, num_slices, rank)) return 0;
    if (out_features < 8 || out_features % 8) return 0;
    const UPlan u = plan_u(num_tokens, max_loras, num_slices, rank, widest(slice_widths, num_slices));
    return mx_layout(layout(num_tokens, max_loras, num_slices, rank, u, backward != 0).total, num_tokens, hidden, out_features, backward != 0).total;
}

int lora_linear_mx(const void *x, int64_t ldx, int num_tokens, int hidden, const void *codes, int64_t ldcodes,
                   const void *scales, int64_t ldscales, int out_features, const void *w_bias, const void *const *lora_a,
                   const void *const *lora_b, const void *const *bias, const int *slice_widths, int num_slices, int rank,
                   float *buf, void *y, int64_t ldy, int offset_start, const lora_meta_t *meta, float scale,
                   int quantize_x, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    int st = check_call(ldx, num_tokens, hidden, codes, hidden, out_features, lora_a, lora_b, slice_widths, num_slices,
                        rank, ldy, offset_start, meta, workspace);
    if (st) return st;
    if ((st = check_codes(codes, ldcodes, scales, ldscales, out_features, hidden))) return st;
    if (ldcodes > kMaxPitch) return LORA_ERR_SHAPE;
    if ((st = check_forward(x, num_tokens, w_bias, bias, num_slices, buf, y))) return st;
    const UPlan u = plan_u(num_tokens, meta->max_loras, num_slices, rank, widest(slice_widths, num_slices));
    const Layout l = layout(num_tokens, meta->max_loras, num_slices, rank, u, false);
    const MxLayout m = mx_layout(l.total, num_tokens, hidden, out_features, false);
    if (m.total > workspace_bytes) return LORA_ERR_BUFFER;
    if (num_tokens == 0) return LORA_OK;
    char *ws = static_cast<char *>(workspace);
    LinearCall c = linear_call(x, ldx, ws + m.w, hidden, w_bias, lora_a, lora_b, bias, slice_widths, num_tokens, hidden, out_features,
                               num_slices, rank, offset_start, meta, scale, workspace, stream);
    if (quantize_x && num_tokens > kRowsTokens) {
        PrepArgs p;
        memset(&p, 0, sizeof p);
        const MetaView view = view_of(meta);
        p.x = static_cast<const uint16_t *>(x);
        p.ldx = ldx;
        p.sorted = view.sorted;
        p.no_lora = view.no_lora;
        p.scales = static_cast<const uint8_t *>(scales);
        p.ldscales = ldscales;
        p.codes = reinterpret_cast<uint8_t *>(ws + m.codes);
        p.nscales = reinterpret_cast<uint8_t *>(ws + m.scales);
        p.mscales = reinterpret_cast<uint8_t *>(ws + m.mscales);
        p.num_tokens = num_tokens;
        p.hidden = hidden;
        p.out = out_features;
        p.blocks = (int)mx_blocks(hidden);
        p.steps = m.steps;
        p.x_groups = (int)ceil_div(num_tokens, 64);
        c.in = p.codes;
        c.ldin = 8 * (int64_t)p.blocks;
        c.w = codes;
        c.ldw = ldcodes / 2;
        c.k = 8 * p.blocks;
        c.mscales = p.mscales;
        c.nscales = p.nscales;
        c.prep = &p;
        return linear_forward<kCodes>(c, l, buf, y, ldy);
    }
    // Where the bf16 projection takes 64 x 64 tiles, W's codes go into the product as they
    // are; larger tiles are bound by the MFMA or by x, and turn W into numbers first.  us of
    // the product from codes, and of both launches, over 4096 by 6144 columns, 32 adapters:
    // 33 tokens 26, 45; 256: 31, 50; 512: 55, 66; (640: 63, 68; 1024: 90, 80).  The limit is
    // that of the bf16 product's tiles; few tokens by more columns stay faster from the codes
    // beyond it: whole calls of 256 tokens by 14336 columns 69, 93
    // (that product's places in x are 32 bits)
    const bool near = (int64_t)num_tokens * ldx * 2 < ((int64_t)1 << 32);
    if (num_tokens <= kRowsTokens || (!quantize_x && near && plan_linear(num_tokens, out_features).tile == kSmall)) {
        c.w = codes;
        c.ldw = ldcodes / 2;
        c.mscales = static_cast<const uint8_t *>(scales);
        c.ldscales = ldscales;
        return quantize_x ? linear_forward<kCodes>(c, l, buf, y, ldy) : linear_forward<kMixed>(c, l, buf, y, ldy);
    }
    const MxArgs turn = mx_args(ws + m.w, LORA_BF16, hidden, out_features, hidden, codes, ldcodes, scales, ldscales);
    c.turn = &turn;
    return linear_forward<kTurned>(c, l, buf, y, ldy);
}

int lora_linear_mx_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx, int num_tokens, int hidden,
                            const void *codes, int64_t ldcodes, const void *scales, int64_t ldscales, int out_features,
                            const void *const *lora_a, const void *const *lora_b, const int *slice_widths, int num_slices,
                            int rank, const float *buf, float *dbuf, void *dx, int64_t lddx, void *const *da,
                            void *const *db, void *const *dbias, int offset_start, const lora_meta_t *meta, float scale,
                            void *workspace, size_t workspace_bytes, hipStream_t stream) {
    int st = check_call(ldx, num_tokens, hidden, codes, hidden, out_features, lora_a, lora_b, slice_widths, num_slices,
                        rank, lddy, offset_start, meta, workspace);
    if (st) return st;
    if ((st = check_codes(codes, ldcodes, scales, ldscales, out_features, hidden))) return st;
    if (ldcodes > kMaxPitch) return LORA_ERR_SHAPE;
    const Gradients g = {dy, lddy, buf, dbuf, dx, lddx, da, db, dbias};
    if ((st = check_gradients(g, x, num_tokens, hidden, num_slices))) return st;
    const UPlan u = plan_u(num_tokens, meta->max_loras, num_slices, rank, widest(slice_widths, num_slices));
    const Layout l = layout(num_tokens, meta->max_loras, num_slices, rank, u, true);
    const MxLayout m = mx_layout(l.total, num_tokens, hidden, out_features, true);
    if (m.total > workspace_bytes) return LORA_ERR_BUFFER;
    char *ws = static_cast<char *>(workspace);
    const MxArgs turn = mx_args(ws + m.w, LORA_BF16, hidden, out_features, hidden, codes, ldcodes, scales, ldscales);
    LinearCall c = linear_call(x, ldx, ws + m.w, hidden, nullptr, lora_a, lora_b, nullptr, slice_widths, num_tokens, hidden,
                               out_features, num_slices, rank, offset_start, meta, scale, workspace, stream);
    c.turn = &turn;
    return linear_backward<kTurned>(c, l, u, g);
}

}  // extern "C"
