// ops_sanitize.cpp -- the argument checks of the scan, norm and beam calls under
// AddressSanitizer and UndefinedBehaviorSanitizer (built and run by
// tests/test_ops_sanitizers.py): sizes at the ends of their types must neither
// overflow nor be let through. Pointers are never dereferenced.
#include <stdio.h>

#include "../gated_deltanet_token_amd/csrc/gdn_ops_validate.hpp"

using namespace gdn::val;

static const char *at(int i) { return reinterpret_cast<const char *>(((uintptr_t)i + 1) << 40); }
static const float *F(int i) { return reinterpret_cast<const float *>(at(i)); }
static const int32_t *I(int i) { return reinterpret_cast<const int32_t *>(at(i)); }
static const uint8_t *U(int i) { return reinterpret_cast<const uint8_t *>(at(i)); }

static int fails = 0;
static void want(bool ok, const char *what) {
    if (!ok) {
        printf("FAILED: %s\n", what);
        ++fails;
    }
}

int main() {
    const int64_t big[] = {0, 1, 127, 128, 1 << 20, (int64_t)1 << 31, (int64_t)1 << 40,
                           INT64_MAX / 2, INT64_MAX};
    const int32_t wide[] = {1, 7, 64, 6144, 1 << 22, INT32_MAX};
    for (int64_t tokens : big)
        for (int64_t n : {(int64_t)1, (int64_t)1000, (int64_t)INT32_MAX})
            for (int32_t D : wide) {
                ScanArgs s{at(0), at(1), at(2), F(3), nullptr, 0, tokens, n, tokens, D, GDN_BF16, 0,
                           F(4), 2, tokens / 128, nullptr, 0};
                const gdn_status_t f = check_scan(s, at(5), F(6));
                const gdn_status_t b = check_scan_backward(s, at(5), F(6), at(7), at(8), at(9), F(10));
                if (tokens >= (int64_t)1 << 40) want(f != GDN_OK && b != GDN_OK, "huge scan refused");
                check_scan_decode(at(0), at(1), at(2), F(3), INT32_MAX, I(4), I(5), at(6), INT32_MAX,
                                  INT32_MAX, D, GDN_F32, 0);
            }
    for (int64_t rows : big)
        for (int32_t D : {1, 128, 16384, 16385, INT32_MAX}) {
            check_norm(at(0), at(1), at(2), at(3), at(4), at(5), F(6), 128, rows, D, GDN_F32, 1e-6f);
            check_norm_backward(at(0), at(1), at(2), at(3), at(4), F(5), rows, D, GDN_F32, 1e-6f,
                                at(6), SIZE_MAX, 1);
        }
    for (int32_t B : {1, 1000, INT32_MAX})
        for (int32_t W : {1, 32, 33, INT32_MAX})
            for (int64_t V : big) {
                const gdn_status_t st =
                    check_beam(at(0), F(1), U(2), I(3), F(4), I(5), I(6), U(7), I(8), B, W, V, 0,
                               GDN_F32, at(9), (size_t)1 << 39, 64);
                if (V >= (int64_t)1 << 31) want(st != GDN_OK, "huge vocabulary refused");
            }
    for (int64_t rows : big)
        for (int64_t rb : {(int64_t)0, (int64_t)16, (int64_t)24, (int64_t)1 << 40, INT64_MAX - 15})
            check_gather(at(0), 8, I(1), at(2), rows, rb);
    want(check_norm(at(0), at(1), at(2), at(3), at(4), at(5), F(6), 128, 100, 5120, GDN_BF16,
                    1e-6f) == GDN_OK, "a plain norm passes");
    want(check_beam(at(0), F(1), U(2), I(3), F(4), I(5), I(6), U(7), I(8), 4, 8, 1000, 2, GDN_BF16,
                    at(9), 4096, 4096) == GDN_OK, "a plain selection passes");
    want(check_gather(at(0), 8, I(1), at(2), 4, 4096) == GDN_OK, "a plain gather passes");
    if (!fails) printf("sanitized checks ok\n");
    return fails != 0;
}
