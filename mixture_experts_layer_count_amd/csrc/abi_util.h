// What the sources of the public entry points share: workspace layout and
// status handling.
#pragma once

#include "common.h"

namespace moe {

constexpr size_t kAlign = 256;
constexpr int kMaxDim = 1 << 20;  // largest H or F (keeps every size product in range)

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// Bump allocator over a caller-provided workspace. With base == NULL it only
// measures.
struct Carver {
    char *base;
    size_t used = 0;
    explicit Carver(void *b) : base(static_cast<char *>(b)) {}
    void *take(size_t bytes) {
        void *p = base ? base + used : nullptr;
        used += align_up(bytes);
        return p;
    }
};

inline moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// tiles of bm rows that `rows` rows in `groups` groups need at most
inline long long max_tiles_for(long long rows, int groups, int bm) { return (rows + bm - 1) / bm + groups; }

}  // namespace moe

#define MOE_TRY(expr)                                  \
    do {                                               \
        hipError_t e_ = (expr);                        \
        if (e_ != hipSuccess) return MOE_ERR_HIP;      \
    } while (0)
