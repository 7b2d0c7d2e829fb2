// Reads products (M N K, then offset from a whole line and row distance of a and of w, in bytes), a
// line each, and prints the launches that each of them becomes: first row, rows, form and whether
// fragments are moved into place.
#include <cstdio>

#include "i8_plan.h"

int main() {
    static const char* const names[] = {"16x16", "32x32", "32x64", "128x64", "128x128 deep", "128x128", "192x256", "256x256"};
    long long M, N, K, a_off, a_stride, w_off, w_stride;
    while (std::scanf("%lld %lld %lld %lld %lld %lld %lld", &M, &N, &K, &a_off, &a_stride, &w_off, &w_stride) == 7) {
        const gdr::Operands g{(1ull << 40) + (unsigned long long)a_off, (1ull << 41) + (unsigned long long)w_off,
                              (int)M, (int)N, (int)K, a_stride, w_stride};
        gdr::launches(g, 0, [](int first, int rows, gdr::Form form, bool moved) {
            std::printf("%d,%d,%s,%s;", first, rows, names[(int)form], moved ? "moved" : "in place");
            return true;
        });
        std::printf("\n");
    }
    return 0;
}
