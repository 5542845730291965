// product_check.cpp -- CPU checks of the products' host side (ob_product.h): refusals, layouts, the 16-byte rule and the
// tile counts.  Prints "ok <checks>".
#include <cstdio>
#include <cstdlib>

#include "ob_product.h"

static int checks = 0;
#define CHECK(x)                                              \
    do {                                                      \
        ++checks;                                             \
        if (!(x)) {                                           \
            std::printf("line %d: %s\n", __LINE__, #x);       \
            std::exit(1);                                     \
        }                                                     \
    } while (0)

static ob_product good()
{
    ob_product p{};
    p.batch = 3;
    p.m = 40;
    p.n = 56;
    p.k = 24;
    p.a = reinterpret_cast<void*>(0x10000);
    p.a_row = 24;
    p.a_col = 1;
    p.a_batch = 40 * 24;
    p.b = reinterpret_cast<void*>(0x20000);
    p.b_row = 56;
    p.b_col = 1;
    p.b_batch = 24 * 56;
    p.c = reinterpret_cast<void*>(0x30000);
    p.c_row = 56;
    p.c_batch = 40 * 56;
    p.d = reinterpret_cast<void*>(0x40000);
    p.d_row = 56;
    p.d_batch = 40 * 56;
    p.in_type = OB_BF16;
    p.out_type = OB_F32;
    p.alpha = 1.0f;
    p.beta = 1.0f;
    return p;
}

template <class F>
static ob_status with(F&& change)
{
    ob_product p = good();
    change(p);
    return ob::check_product(&p);
}

int main()
{
    using P = ob_product;
    const float nan = std::nanf("");
    CHECK(with([](P&) {}) == OB_OK);
    CHECK(ob::check_product(nullptr) == OB_ERR_ARG);
    // extents, types, factors
    CHECK(with([](P& p) { p.m = -1; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.k = INT64_C(1) << 31; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.batch = INT64_C(1) << 40; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.in_type = OB_F32; }) == OB_ERR_DTYPE);
    CHECK(with([](P& p) { p.out_type = 5; }) == OB_ERR_DTYPE);
    CHECK(with([&](P& p) { p.alpha = nan; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.beta = INFINITY; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.symmetric = 2; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.symmetric = 1; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.reserved = 1; }) == OB_ERR_ARG);
    // nothing to do needs no pointers
    CHECK(with([](P& p) { p.m = 0; p.a = p.b = p.c = nullptr; p.d = nullptr; }) == OB_OK);
    CHECK(with([](P& p) { p.batch = 0; p.d = nullptr; }) == OB_OK);
    CHECK(with([](P& p) { p.k = 0; p.a = p.b = nullptr; }) == OB_OK);
    CHECK(with([](P& p) { p.k = 0; p.a = p.b = nullptr; p.d = nullptr; }) == OB_ERR_ARG);
    // pointers
    CHECK(with([](P& p) { p.a = nullptr; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.b = nullptr; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.c = nullptr; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.c = nullptr; p.beta = 0.0f; }) == OB_OK);
    CHECK(with([](P& p) { p.d = nullptr; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.a = reinterpret_cast<void*>(0x10001); }) == OB_ERR_ALIGN);
    CHECK(with([](P& p) { p.b = reinterpret_cast<void*>(0x10002); }) == OB_OK);
    CHECK(with([](P& p) { p.c = reinterpret_cast<void*>(0x30002); }) == OB_ERR_ALIGN);
    CHECK(with([](P& p) { p.d = reinterpret_cast<void*>(0x40002); }) == OB_ERR_ALIGN);
    CHECK(with([](P& p) { p.d = reinterpret_cast<void*>(0x40002); p.out_type = OB_F16; }) == OB_OK);
    // strides
    CHECK(with([](P& p) { p.a_col = 2; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.a_row = 1; p.a_col = 40; }) == OB_OK);
    CHECK(with([](P& p) { p.b_row = 1; p.b_col = 24; }) == OB_OK);
    CHECK(with([](P& p) { p.b_row = 2; p.b_col = 24; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.a_row = -24; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.a_row = 0; p.a_batch = 0; }) == OB_OK);
    CHECK(with([](P& p) { p.a_row = INT64_MAX; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.b_batch = INT64_MAX / 2; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.c_row = INT64_MAX; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.d_row = 55; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.d_batch = 40 * 56 - 1; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.d_row = 60; p.d_batch = 39 * 60 + 56; }) == OB_OK);
    CHECK(with([](P& p) { p.d_row = INT64_MAX; }) == OB_ERR_ARG);
    CHECK(with([](P& p) { p.n = 40; p.b_row = 40; p.symmetric = 1; }) == OB_OK);
    // layouts: by K where K's stride is one, whatever an extent of one pretends
    CHECK(ob::product_operand(24, 1, 40, 24).k_major && ob::product_operand(24, 1, 40, 24).ld == 24);
    CHECK(!ob::product_operand(1, 40, 40, 24).k_major && ob::product_operand(1, 40, 40, 24).ld == 40);
    CHECK(ob::product_operand(1, 1, 1, 24).k_major);     // one row
    CHECK(!ob::product_operand(1, 1, 40, 1).k_major);    // one k
    CHECK(ob::product_operand(0, 1, 40, 24).k_major && ob::product_operand(0, 1, 40, 24).ld == 0);
    CHECK(ob::product_operand(1, 1, 40, 24).k_major && ob::product_operand(1, 1, 40, 24).ld == 1);   // overlapping rows
    // 16-byte chunks
    void* p16 = reinterpret_cast<void*>(0x1000);
    void* p2 = reinterpret_cast<void*>(0x1002);
    CHECK(ob::product_chunks({true, 64}, p16, 1, 0, 33, 64));
    CHECK(!ob::product_chunks({true, 64}, p2, 1, 0, 33, 64));
    CHECK(!ob::product_chunks({true, 65}, p16, 1, 0, 33, 64));
    CHECK(ob::product_chunks({true, 65}, p16, 1, 0, 1, 64));      // one row has no next one
    CHECK(!ob::product_chunks({true, 64}, p16, 1, 0, 33, 60));
    CHECK(!ob::product_chunks({false, 40}, p16, 1, 0, 33, 64));   // 33 rows lie behind each other
    CHECK(ob::product_chunks({false, 40}, p16, 1, 0, 40, 63));
    CHECK(!ob::product_chunks({false, 40}, p16, 2, 40 * 63 + 4, 40, 63));
    CHECK(ob::product_chunks({false, 40}, p16, 2, 40 * 63 + 8, 40, 63));
    CHECK(!ob::product_chunks({true, INT64_C(1) << 21}, p16, 1, 0, 33, 64));
    // tiles
    CHECK(ob::product_tiles(256, 256, 256, false) == 1 && ob::product_tiles(257, 256, 256, false) == 2);
    CHECK(ob::product_tiles(1024, 1024, 256, true) == 10 && ob::product_tiles(1, 1, 64, true) == 1);
    std::printf("ok %d\n", checks);
    return 0;
}
