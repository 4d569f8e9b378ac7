// Memory- and UB-sanitizer driver for the host side of the calls around the attention (include/kv8mla.h: kv8_rope_freqs, kv8_rope,
// kv8_norm_rope_rows, kv8_quant_blocks, kv8_matmul8).  As abi_driver.cpp: built by tests/test_layer_sanitizers.py, run with every GPU
// hidden, so that no kernel can start; invalid arguments give KV8_EINVAL, well-formed calls KV8_ECUDA.  Device pointers are
// aligned host addresses that the library never dereferences on the host.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>

#include "kv8mla.h"

static int g_fail = 0;
#define EXPECT(call, want)                                                                               \
    do {                                                                                                 \
        const int rc_ = (call);                                                                          \
        if (rc_ != (want)) {                                                                             \
            fprintf(stderr, "line %d: %s returned %d, expected %d\n", __LINE__, #call, rc_, (int)(want)); \
            g_fail = 1;                                                                                  \
        }                                                                                                \
    } while (0)

int main() {
    unsigned char *arena = static_cast<unsigned char *>(aligned_alloc(256, (size_t)1 << 20));
    void *x = arena, *y = arena + 65536, *z = arena + 131072, *mis = arena + 1;
    auto *f = reinterpret_cast<float *>(arena + 196608);
    auto *i32 = reinterpret_cast<int32_t *>(arena + 262144);
    auto *i64 = reinterpret_cast<int64_t *>(arena + 327680);
    auto *u8 = arena + 393216, *w8 = arena + 458752;
    int err_word = 0;
    const int64_t big = (int64_t)1 << 40, most = INT64_MAX, least = INT64_MIN;

    // ---- the frequency table: the largest and smallest it takes, in a buffer of exactly its size
    for (int dim = 2; dim <= KV8_MAX_ROPE; dim += dim < 16 ? 2 : 30) {
        float *table = static_cast<float *>(malloc(sizeof(float) * (dim / 2))), *scale = static_cast<float *>(malloc(sizeof(float)));
        const double theta[] = {1.0000001, 10000.0, 1e30}, factor[] = {1.0, 40.0, 1e6}, context[] = {1.0, 4096.0, 1e15};
        for (double t : theta)
            for (double k : factor)
                for (double c : context) {
                    EXPECT(kv8_rope_freqs(dim, t, k, c, 32.0, 1.0, table, scale), KV8_OK);
                    EXPECT(kv8_rope_freqs(dim, t, k, c, 1e6, 1e-300, table, scale), KV8_OK);
                    for (int i = 0; i < dim / 2; ++i)
                        if (!(table[i] >= 0.f && table[i] <= 1.f)) g_fail = 1;
                }
        EXPECT(kv8_rope_freqs(dim, NAN, 1.0, 4096.0, 32.0, 1.0, table, scale), KV8_EINVAL);
        EXPECT(kv8_rope_freqs(dim, 1e4, INFINITY, 4096.0, 32.0, 1.0, table, scale), KV8_EINVAL);
        EXPECT(kv8_rope_freqs(dim + 1, 1e4, 1.0, 4096.0, 32.0, 1.0, table, scale), KV8_EINVAL);
        EXPECT(kv8_rope_freqs(dim, 1e4, 1.0, 4096.0, 32.0, 1.0, table, nullptr), KV8_EINVAL);
        free(table);
        free(scale);
    }

#define ROPE(n, h, w, at, d, xr, xh, rr, rh, rest, er, eh) \
    kv8_rope(x, KV8_BF16, n, h, w, at, d, xr, xh, i32, f, 1.f, KV8_ROPE_HALF, y, rr, rh, rest, er, eh, KV8_F32, nullptr)
    // ---- strides of every size, sizes at their limits: no overflow on the way to the answer
    for (int64_t s : {big + 1, most, least, (int64_t)-1}) {
        EXPECT(ROPE(4, 8, 192, 128, 64, s, 192, 512, 64, z, 1024, 128), KV8_EINVAL);
        EXPECT(ROPE(4, 8, 192, 128, 64, 1536, s, 512, 64, z, 1024, 128), KV8_EINVAL);
        EXPECT(ROPE(4, 8, 192, 128, 64, 1536, 192, s, 64, z, 1024, 128), KV8_EINVAL);
        EXPECT(ROPE(4, 8, 192, 128, 64, 1536, 192, 512, s, z, 1024, 128), KV8_EINVAL);
        EXPECT(ROPE(4, 8, 192, 128, 64, 1536, 192, 512, 64, z, s, 128), KV8_EINVAL);
        EXPECT(ROPE(4, 8, 192, 128, 64, 1536, 192, 512, 64, z, 1024, s), KV8_EINVAL);
        EXPECT(kv8_norm_rope_rows(x, KV8_F32, 4, s, f, 0.f, i32, f, 1.f, 0, i64, u8, f, 10, &err_word, nullptr), KV8_EINVAL);
        EXPECT(kv8_quant_blocks(x, KV8_F32, 4, 256, s, f, 0.f, u8, f, 4, nullptr), KV8_EINVAL);
        EXPECT(kv8_quant_blocks(x, KV8_F32, 4, 256, 256, f, 0.f, u8, f, s, nullptr), KV8_EINVAL);
        EXPECT(kv8_matmul8(u8, s, f, 4, 4, 128, 256, w8, f, y, KV8_F32, 128, &err_word, nullptr), KV8_EINVAL);
        EXPECT(kv8_matmul8(u8, 256, f, s, 4, 128, 256, w8, f, y, KV8_F32, 128, &err_word, nullptr), KV8_EINVAL);
        EXPECT(kv8_matmul8(u8, 256, f, 4, 4, 128, 256, w8, f, y, KV8_F32, s, &err_word, nullptr), KV8_EINVAL);
    }
    EXPECT(kv8_rope(x, KV8_BF16, 4, 8, 192, INT32_MAX, 64, 1536, 192, i32, f, 1.f, 0, y, 512, 64, z, 1024, 128, KV8_F32, nullptr), KV8_EINVAL);
    EXPECT(kv8_rope(x, KV8_BF16, 4, 8, INT32_MIN, 0, 64, 1536, 192, i32, f, 1.f, 0, y, 512, 64, z, 1024, 128, KV8_F32, nullptr), KV8_EINVAL);
    EXPECT(kv8_rope(mis, KV8_BF16, 4, 8, 192, 128, 64, 1536, 192, i32, f, 1.f, 0, y, 512, 64, z, 1024, 128, KV8_F32, nullptr), KV8_EINVAL);
    EXPECT(kv8_norm_rope_rows(x, KV8_F32, most, 576, f, 0.f, i32, f, INFINITY, 0, i64, u8, f, 10, &err_word, nullptr), KV8_EINVAL);
    EXPECT(kv8_quant_blocks(x, 7, 4, 256, 256, f, 0.f, u8, f, 4, nullptr), KV8_EINVAL);
    EXPECT(kv8_matmul8(u8, 256, f, 4, INT32_MAX, 128, 256, w8, f, y, KV8_F32, 128, &err_word, nullptr), KV8_EINVAL);
    EXPECT(kv8_matmul8(u8, 256, f, 4, 4, INT32_MAX, 256, w8, f, y, KV8_F32, most, &err_word, nullptr), KV8_EINVAL);

    // ---- nothing to do
    EXPECT(ROPE(0, 8, 192, 128, 64, 0, 0, 0, 0, nullptr, 0, 0), KV8_OK);
    EXPECT(kv8_norm_rope_rows(nullptr, KV8_F32, 0, 0, nullptr, 0.f, nullptr, nullptr, 1.f, 0, nullptr, nullptr, nullptr, 0, nullptr, nullptr), KV8_OK);
    EXPECT(kv8_quant_blocks(nullptr, KV8_F32, 0, 256, 0, nullptr, 0.f, nullptr, nullptr, 0, nullptr), KV8_OK);
    EXPECT(kv8_matmul8(nullptr, 0, nullptr, 0, 0, 128, 256, nullptr, nullptr, nullptr, KV8_F32, 0, nullptr, nullptr), KV8_OK);

    // ---- well-formed calls, the largest ones too (the plans and grids of every form): the launch is refused
    for (int64_t n : {(int64_t)1, (int64_t)37, (int64_t)KV8_MAX_ROWS})
        for (int heads : {1, 7, KV8_MAX_HEADS})
            for (int dim : {2, 64, 96, KV8_MAX_ROPE})
                for (int width : {dim, dim + 1, dim + 128, KV8_MAX_WIDTH}) {
                    const int64_t row = (int64_t)heads * KV8_MAX_WIDTH;
                    for (int type = 0; type < 2; ++type)
                        for (int layout = 0; layout < 2; ++layout)
                            EXPECT(kv8_rope(x, type, n, heads, width, 0, dim, row, width, i32, f, 1.f, layout, y, (int64_t)heads * dim, dim, z, row, KV8_MAX_WIDTH,
                                            1 - type, nullptr), KV8_ECUDA);
                }
    for (int type = 0; type < 2; ++type) {
        for (int64_t n : {(int64_t)1, (int64_t)KV8_MAX_ROWS}) {
            for (int layout = 0; layout < 2; ++layout)
                EXPECT(kv8_norm_rope_rows(x, type, n, 576, f, 1e-6f, i32, f, 1.f, layout, i64, u8, f, 10, &err_word, nullptr), KV8_ECUDA);
            for (int width : {16, 512, 1024, 2048, 4096, 8192, KV8_MAX_NORM_WIDTH, KV8_MAX_WIDTH}) {
                if (width <= KV8_MAX_NORM_WIDTH) EXPECT(kv8_quant_blocks(x, type, n, width, width, f, 1e-6f, u8, f, n, nullptr), KV8_ECUDA);
                EXPECT(kv8_quant_blocks(x, type, n, width, width, nullptr, 0.f, u8, f, n, nullptr), KV8_ECUDA);
            }
        }
        for (int M : {1, 16, 17, 64, 65, 300, 1000, 8192, KV8_MAX_ROWS})
            for (int N : {1, 576, 24576, KV8_MAX_ROWS})
                for (int K : {16, 512, 4112, KV8_MAX_WIDTH})
                    EXPECT(kv8_matmul8(u8, K, f, M, M, N, K, w8, f, y, type, N, &err_word, nullptr), KV8_ECUDA);
    }

    free(arena);
    if (g_fail) return 1;
    printf("layer driver ok\n");
    return 0;
}
