// Drives the 4-bit key/value cache's entry points with arguments that host
// validation must reject, and its size functions over the range of sizes,
// from one thread and then from four.  Nothing reaches a device.
#include "awq.h"

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <thread>
#include <vector>

#define CHECK(x)                                                        \
    do {                                                                \
        if (!(x)) {                                                     \
            std::printf("FAILED %s:%d: %s\n", __FILE__, __LINE__, #x);  \
            std::exit(1);                                               \
        }                                                               \
    } while (0)

static void *const P = reinterpret_cast<void *>(0x10000);
static const int32_t *const I = reinterpret_cast<const int32_t *>(0x10000);

static void refuse(const awq_kv_cache *c, const awq_kv_batch *b, awq_status want) {
    CHECK(awq_kv_append(c, b, P, P, AWQ_BF16, 512, 512, nullptr) == want);
    CHECK(std::strlen(awq_last_error()) > 0);
    CHECK(awq_kv_read(c, b, P, P, AWQ_F16, 512, 512, nullptr) == want);
    CHECK(awq_kv_attention(c, b, P, AWQ_BF16, 8, 1024, 1, 1.0f, 1, 0, P, 1024, nullptr, P, size_t(1) << 40, nullptr) == want);
    CHECK(std::strlen(awq_last_error()) > 0);
}

static void all() {
    awq_kv_cache good{};
    good.pages = P, good.n_pages = 8, good.page_stride = 4 * 16 * 136, good.heads = 4, good.dim = 128, good.group = 128,
    good.page = 16;
    awq_kv_batch batch{};
    batch.rows = 6, batch.batch = 3, batch.max_pages = 64, batch.kv_len = I, batch.block_table = I;
    refuse(nullptr, &batch, AWQ_ERR_ARG);
    refuse(&good, nullptr, AWQ_ERR_ARG);
    for (int v : {-1, 0, 1, 15, 17, 96, 257, 1 << 30, INT32_MIN}) {
        awq_kv_cache c = good;
        c.page = v;
        refuse(&c, &batch, AWQ_ERR_ARG);
        c = good, c.group = v;
        refuse(&c, &batch, AWQ_ERR_ARG);
        c = good, c.dim = v;
        refuse(&c, &batch, AWQ_ERR_SHAPE);
    }
    const int64_t huge[] = {INT64_MAX, INT64_MIN, -1, int64_t(1) << 62, int64_t(1) << 45};
    for (int64_t v : huge) {
        awq_kv_cache c = good;
        c.heads = v;
        refuse(&c, &batch, AWQ_ERR_SHAPE);
        if (v < 0 || v > INT32_MAX) {
            c = good, c.n_pages = v;
            refuse(&c, &batch, AWQ_ERR_SHAPE);
        }
        awq_kv_batch b = batch;
        b.batch = v;
        refuse(&good, &b, AWQ_ERR_SHAPE);
        b = batch, b.max_pages = v;
        refuse(&good, &b, AWQ_ERR_SHAPE);
        b = batch, b.rows = v, b.row_start = I;
        refuse(&good, &b, AWQ_ERR_SHAPE);
        CHECK(awq_kv_page_size(16, v, 128, 128) == 0);
        CHECK(awq_kv_append(&good, &batch, P, P, AWQ_BF16, v, 512, nullptr) == AWQ_ERR_SHAPE);
        CHECK(awq_kv_attention_workspace_size(&good, &batch, v, 0) == 0);
    }
    for (float s : {0.0f, -1.0f, INFINITY, -INFINITY, NAN})
        CHECK(awq_kv_attention(&good, &batch, P, AWQ_F16, 8, 1024, 0, s, 1, 0, P, 1024, nullptr, P, size_t(1) << 40,
                               nullptr) == AWQ_ERR_ARG);
    CHECK(awq_kv_attention(&good, &batch, P, AWQ_F16, 8, 1024, 0, 1.0f, 1, 0, P, 1024, nullptr, P, 1, nullptr) ==
          AWQ_ERR_WORKSPACE);
    for (int t : {-1, 3, 100})
        CHECK(awq_kv_append(&good, &batch, P, P, static_cast<awq_dtype>(t), 512, 512, nullptr) == AWQ_ERR_DTYPE);
    // sizes over the range, the largest batches that are accepted included
    for (int dim : {64, 128, 256})
        for (int group : {32, 64, 128})
            for (int page = 16; page <= 256; page *= 2)
                for (int64_t heads : {1, 8, 65535})
                    for (int64_t n : {int64_t(1), int64_t(1000), int64_t(1) << 20, int64_t(1) << 30})
                        for (int64_t mp : {int64_t(1), int64_t(77), int64_t(1) << 22})
                            for (int ragged = 0; ragged < 2; ++ragged) {
                                awq_kv_cache c = good;
                                c.dim = dim, c.group = group, c.page = page, c.heads = heads;
                                awq_kv_batch b = batch;
                                b.batch = n, b.rows = 2 * n, b.max_pages = mp, b.row_start = ragged ? I : nullptr;
                                (void)awq_kv_attention_workspace_size(&c, &b, heads, 0);
                                (void)awq_kv_attention_workspace_size(&c, &b, heads, INT64_MAX);
                                (void)awq_kv_page_size(page, heads, dim, group);
                            }
}

int main() {
    all();
    std::vector<std::thread> t;
    for (int i = 0; i < 4; ++i) t.emplace_back(all);
    for (auto &x : t) x.join();
    std::printf("sanitized key/value cache checks passed\n");
    return 0;
}
