// lora_linear.hip -- the entry points of the shared projection with adapters,
// its matrix in bfloat16.
#include "lora_linear.h"

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
    if ((st = check_forward(x, num_tokens, w_bias, bias, num_slices, buf, y))) return st;
    const UPlan u = plan_u(num_tokens, meta->max_loras, num_slices, rank, widest(slice_widths, num_slices));
    const Layout l = layout(num_tokens, meta->max_loras, num_slices, rank, u, false);
    if (l.total > workspace_bytes) return LORA_ERR_BUFFER;
    if (num_tokens == 0) return LORA_OK;
    const LinearCall c = linear_call(x, ldx, w, ldw, w_bias, lora_a, lora_b, bias, slice_widths, num_tokens, hidden, out_features,
                                     num_slices, rank, offset_start, meta, scale, workspace, stream);
    return linear_forward<kWide>(c, l, buf, y, ldy);
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
    const Gradients g = {dy, lddy, buf, dbuf, dx, lddx, da, db, dbias};
    if ((st = check_gradients(g, x, num_tokens, hidden, num_slices))) return st;
    const UPlan u = plan_u(num_tokens, meta->max_loras, num_slices, rank, widest(slice_widths, num_slices));
    const Layout l = layout(num_tokens, meta->max_loras, num_slices, rank, u, true);
    if (l.total > workspace_bytes) return LORA_ERR_BUFFER;
    const LinearCall c = linear_call(x, ldx, w, ldw, nullptr, lora_a, lora_b, nullptr, slice_widths, num_tokens, hidden, out_features,
                                     num_slices, rank, offset_start, meta, scale, workspace, stream);
    return linear_backward<kWide>(c, l, u, g);
}

}  // extern "C"
