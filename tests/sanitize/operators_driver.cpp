// Calls the entry points of include/lora_mi355x.h that abi_driver.cpp does not (the
// projection with adapters, its matrix in bfloat16 or in 4 bits, the vocabulary cross
// entropy, the conversions, clipping) with arguments that the host-side checks reject,
// and their workspace queries, in a build whose host code has AddressSanitizer and
// UndefinedBehaviorSanitizer.  No call reaches a kernel launch, so no GPU is needed.
// Prints "ok" on success.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <vector>

#include "lora_mi355x.h"

static int failures = 0;
#define EXPECT(expr, want)                                                          \
    do {                                                                            \
        const int got_ = (expr);                                                    \
        if (got_ != (want)) {                                                       \
            fprintf(stderr, "%s:%d: %s = %d, want %d\n", __FILE__, __LINE__, #expr, \
                    got_, (int)(want));                                            \
            ++failures;                                                             \
        }                                                                           \
    } while (0)

// Addresses that no one reads.
static void *at(size_t v) { return reinterpret_cast<void *>(v); }

static int queries() {
    int seen = 0;
    const int widths[LORA_MAX_SLICES] = {4096, 8, 1024, 72, 16, 8, 264, 8};
    for (int slices = 1; slices <= LORA_MAX_SLICES; slices += 3)
        for (int rank = 8; rank <= LORA_MAX_RANK; rank += 24)
            for (int loras = 1; loras <= LORA_MAX_LORAS; loras = loras * 3 + 1)
                for (int hidden = 8; hidden <= LORA_MAX_HIDDEN; hidden *= 8)
                    for (int backward = 0; backward < 2; ++backward) {
                        size_t linear = 0, mx = 0;
                        for (int n = 0; n <= LORA_MAX_TOKENS; n = n * 4 + 1) {
                            const size_t a = lora_linear_workspace_bytes(n, loras, hidden, widths, slices, rank, backward);
                            const size_t b = lora_linear_mx_workspace_bytes(n, loras, hidden, 8192, widths, slices, rank, backward);
                            if (a < linear || b < mx || b < a || !a) ++failures;
                            linear = a;
                            mx = b;
                            ++seen;
                        }
                    }
    for (int vocab = 1; vocab <= LORA_MAX_VOCAB; vocab = vocab * 5 + 3)
        for (int n = 0; n <= LORA_MAX_TOKENS; n = n * 4 + 1) {
            if (lora_cross_entropy_workspace_bytes(n, 4096, vocab, 1) < lora_cross_entropy_workspace_bytes(n, 4096, vocab, 0)) ++failures;
            ++seen;
        }
    EXPECT((int)(lora_linear_mx_workspace_bytes(1, 1, 8, 12, widths, 1, 8, 0) == 0), 1);
    EXPECT((int)(lora_linear_mx_workspace_bytes(LORA_MAX_TOKENS + 1, 1, 8, 8, widths, 1, 8, 0) == 0), 1);
    EXPECT((int)(lora_linear_workspace_bytes(1, 1, 8, nullptr, 1, 8, 0) == 0), 1);
    EXPECT((int)(lora_linear_workspace_bytes(1, 1, 8, widths, 9, 8, 0) == 0), 1);
    EXPECT((int)(lora_cross_entropy_workspace_bytes(1, 12, 8, 0) == 0), 1);
    return seen;
}

static void conversions() {
    EXPECT(lora_mx_quantize(at(16), LORA_BF16, 72, 5, 72, at(32), 32, at(4), 4, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_mx_quantize(at(8), LORA_F32, 72, 5, 72, at(32), 48, at(4), 4, nullptr), LORA_ERR_ALIGN);
    EXPECT(lora_mx_quantize(at(16), 7, 72, 5, 72, at(32), 48, at(4), 4, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_mx_quantize(nullptr, LORA_F32, 72, 5, 72, at(32), 48, at(4), 4, nullptr), LORA_ERR_NULL);
    EXPECT(lora_mx_quantize(nullptr, LORA_F32, 72, 0, 72, nullptr, 48, nullptr, 4, nullptr), LORA_OK);
    EXPECT(lora_mx_dequantize(at(32), 48, at(2), 4, 5, 72, at(16), LORA_F32, 72, nullptr), LORA_ERR_ALIGN);
    EXPECT(lora_mx_dequantize(at(32), 48, at(4), 4, 5, LORA_MAX_HIDDEN + 8, at(16), LORA_F32, LORA_MAX_HIDDEN + 8, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_mx_dequantize(at(32), 48, at(4), 4, 0, 72, at(16), LORA_BF16, 72, nullptr), LORA_OK);
}

static void products() {
    void *raw = nullptr;
    const size_t nb = lora_meta_bytes(7, 300);
    if (posix_memalign(&raw, 256, nb) != 0) exit(2);
    lora_meta_t m;
    EXPECT(lora_meta_bind(raw, nb, 7, 300, &m), LORA_OK);
    m.num_tokens = 64;
    const int widths[2] = {64, 32};
    const void *a[2] = {at(256), at(512)}, *bad[2] = {at(256), at(520)}, *none[2] = {at(256), nullptr};
    void *da[2] = {at(1024), at(2048)}, *less[2] = {at(1024), nullptr};
    float *buf = static_cast<float *>(at(4096));
    const size_t big = (size_t)1 << 40;
#define FORWARD(N, LDX, H, LDW, OUT, A, OFF, WS, BYTES) \
    lora_linear(at(64), LDX, N, H, at(128), LDW, OUT, nullptr, A, a, nullptr, widths, 2, 16, buf, at(8192), OUT, OFF, &m, 1.f, at(WS), BYTES, nullptr)
    EXPECT(FORWARD(63, 72, 72, 72, 104, a, 8, 0x10000, big), LORA_ERR_NUM_TOKENS);
    EXPECT(FORWARD(64, 64, 72, 72, 104, a, 8, 0x10000, big), LORA_ERR_SHAPE);
    EXPECT(FORWARD(64, 72, 72, 64, 104, a, 8, 0x10000, big), LORA_ERR_SHAPE);
    EXPECT(FORWARD(64, 72, 72, 72, 96, a, 8, 0x10000, big), LORA_ERR_SHAPE);
    EXPECT(FORWARD(64, 72, 72, 72, 104, bad, 8, 0x10000, big), LORA_ERR_ALIGN);
    EXPECT(FORWARD(64, 72, 72, 72, 104, none, 8, 0x10000, big), LORA_ERR_NULL);
    EXPECT(FORWARD(64, 72, 72, 72, 104, a, 8, 0x10010, big), LORA_ERR_BUFFER);
    EXPECT(FORWARD(64, 72, 72, 72, 104, a, 8, 0x10000, 0), LORA_ERR_BUFFER);
#define BACKWARD(H, DA, BUF, BYTES) \
    lora_linear_backward(at(64), 104, at(64), 72, 64, H, at(128), 72, 104, a, a, widths, 2, 16, BUF, buf, nullptr, 0, DA, da, nullptr, 8, &m, 1.f, at(0x10000), BYTES, nullptr)
    EXPECT(BACKWARD(76, da, buf, big), LORA_ERR_SHAPE);
    EXPECT(BACKWARD(72, less, buf, big), LORA_ERR_NULL);
    EXPECT(BACKWARD(72, nullptr, buf, big), LORA_ERR_NULL);
    EXPECT(BACKWARD(72, da, nullptr, big), LORA_ERR_NULL);
    EXPECT(BACKWARD(72, da, buf, 4096), LORA_ERR_BUFFER);
#define MX(LDC, LDS, CODES, SCALES, BYTES) \
    lora_linear_mx(at(64), 72, 64, 72, at(CODES), LDC, at(SCALES), LDS, 104, nullptr, a, a, nullptr, widths, 2, 16, buf, at(8192), 104, 8, &m, 1.f, 1, at(0x10000), BYTES, nullptr)
    EXPECT(MX(48, 4, 128, 4, 256), LORA_ERR_BUFFER);
    EXPECT(MX(32, 4, 128, 4, big), LORA_ERR_SHAPE);
    EXPECT(MX((1 << 25) + 16, 4, 128, 4, big), LORA_ERR_SHAPE);
    EXPECT(MX(48, 2, 128, 4, big), LORA_ERR_SHAPE);
    EXPECT(MX(48, 4, 136, 4, big), LORA_ERR_ALIGN);
    EXPECT(MX(48, 4, 128, 2, big), LORA_ERR_ALIGN);
    EXPECT(MX(48, 4, 0, 4, big), LORA_ERR_NULL);
    EXPECT(MX(48, 4, 128, 0, big), LORA_ERR_NULL);
#define MX_BACKWARD(LDC, DB, BYTES) \
    lora_linear_mx_backward(at(64), 104, at(64), 72, 64, 72, at(128), LDC, at(4), 4, 104, a, a, widths, 2, 16, buf, buf, at(64), 72, da, DB, nullptr, 8, &m, 1.f, at(0x10000), BYTES, nullptr)
    EXPECT(MX_BACKWARD(40, da, big), LORA_ERR_SHAPE);
    EXPECT(MX_BACKWARD(48, less, big), LORA_ERR_NULL);
    EXPECT(MX_BACKWARD(48, da, 1024), LORA_ERR_BUFFER);
    m.num_tokens = 0;
    EXPECT(FORWARD(0, 72, 72, 72, 104, a, 8, 0x10000, big), LORA_OK);
    free(raw);

    const int32_t *targets = static_cast<int32_t *>(at(64));
    EXPECT(lora_cross_entropy(at(64), 72, 5, 76, at(64), 72, 9, targets, buf, buf, at(0x10000), big, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_cross_entropy(at(64), 72, 5, 72, at(64), 72, 9, targets, buf, buf, at(0x10000), 0, nullptr), LORA_ERR_BUFFER);
    EXPECT(lora_cross_entropy(nullptr, 72, 5, 72, at(64), 72, 9, targets, buf, buf, at(0x10000), big, nullptr), LORA_ERR_NULL);
    EXPECT(lora_cross_entropy_backward(at(64), 72, 5, 72, at(64), 72, 9, targets, buf, buf, at(64), 64, nullptr, 0, at(0x10000), big, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_cross_entropy_backward(at(64), 72, 5, 72, at(64), 72, 9, targets, buf, nullptr, at(64), 72, nullptr, 0, at(0x10000), big, nullptr), LORA_ERR_NULL);
}

// Whether two results, or a result and another place's gradient, share memory, spelled out.
struct Tensor {
    size_t in, out, bytes;
};
static bool overlap(size_t a, size_t b, size_t n, size_t m) { return n && m && a < b + m && b < a + n; }
static bool refused(const std::vector<Tensor> &t) {
    for (size_t i = 0; i < t.size(); ++i)
        for (size_t j = 0; j < t.size(); ++j) {
            if (i != j && overlap(t[i].out, t[j].out, t[i].bytes, t[j].bytes)) return true;
            if (t[j].in != t[j].out && overlap(t[i].out, t[j].in, t[i].bytes, t[j].bytes)) return true;
        }
    return false;
}

static int clipping() {
    float *norms = static_cast<float *>(at(0x100));
    int64_t sizes[2] = {64, 32};
    int types[2] = {LORA_BF16, LORA_F32};
    const void *g[2] = {at(0x10000), at(0x20000)};
    void *o[2] = {at(0x30000), at(0x40000)};
    const size_t big = (size_t)1 << 40;
    EXPECT(lora_clip_gradients(g, o, sizes, types, 2, 3, 1.0, norms, at(0x200), big, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_clip_gradients(g, o, sizes, types, 2, 0, 1.0, norms, at(0x200), big, nullptr), LORA_ERR_MAX_LORAS);
    EXPECT(lora_clip_gradients(g, o, sizes, types, LORA_MAX_TENSORS + 1, 4, 1.0, norms, at(0x200), big, nullptr), LORA_ERR_SLICES);
    EXPECT(lora_clip_gradients(g, o, sizes, types, 2, 4, NAN, norms, at(0x200), big, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_clip_gradients(g, nullptr, sizes, types, 2, 4, 1.0, norms, at(0x200), big, nullptr), LORA_ERR_NULL);
    EXPECT(lora_clip_gradients(g, o, sizes, types, 2, 4, 1.0, norms, at(0x200), 8, nullptr), LORA_ERR_BUFFER);
    sizes[0] = (int64_t)1 << 62;   // a part of more than 2^32 elements
    EXPECT((int)(lora_clip_gradients_workspace_bytes(sizes, types, 2, 4) == 0), 1);
    EXPECT(lora_clip_gradients(g, o, sizes, types, 2, 4, 1.0, norms, at(0x200), big, nullptr), LORA_ERR_SHAPE);
    for (int k = 0; k < 64; ++k) {
        sizes[0] = k < 40 ? (int64_t)1 << k : 0;
        sizes[1] = 7;
        lora_clip_gradients_workspace_bytes(sizes, types, 2, 1);
    }
    // spans in no order, some empty, some in place: those that overlap are refused (the
    // others would be launched, and are not tried)
    uint32_t state = 12345;
    auto next = [&](uint32_t n) {
        state = state * 1664525u + 1013904223u;
        return (state >> 8) % n;
    };
    int seen = 0;
    for (int round = 0; round < 20000; ++round) {
        std::vector<Tensor> t;
        const int n = 1 + next(8);
        for (int i = 0; i < n; ++i) {
            Tensor x;
            x.bytes = 4 * next(12);
            x.in = 0x10000 + 4 * next(200);
            x.out = next(3) ? 0x10000 + 4 * next(200) : x.in;
            t.push_back(x);
        }
        if (!refused(t)) continue;
        std::vector<int64_t> s;
        std::vector<int> kinds;
        std::vector<const void *> in;
        std::vector<void *> out;
        for (const Tensor &x : t) {
            const bool wide = next(2);
            s.push_back((int64_t)(x.bytes / (wide ? 4 : 2)));
            kinds.push_back(wide ? LORA_F32 : LORA_BF16);
            in.push_back(at(x.in));
            out.push_back(at(x.out));
        }
        EXPECT(lora_clip_gradients(in.data(), out.data(), s.data(), kinds.data(), n, 1, 1.0, norms, at(0x200), big, nullptr), LORA_ERR_BUFFER);
        ++seen;
    }
    return seen;
}

int main() {
    const int sizes = queries();
    conversions();
    products();
    const int spans = clipping();
    if (failures) {
        fprintf(stderr, "%d check(s) failed\n", failures);
        return 1;
    }
    printf("ok %d %d\n", sizes, spans);
    return 0;
}
