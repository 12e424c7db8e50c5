// MXFP4: E2M1 codes (magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6) with one E8M0 scale
// per 32 values.
//
// Scale: 2^e with e = floor(log2 max|x|) - 2 (2 is E2M1's largest exponent),
// at least -127, byte e + 127; a group of zeros has e = 0. Code: E2M1(x 2^-e),
// round to nearest, ties to even, magnitudes past 6 to 6: the one rounding, as
// the scale is a power of two. A group that holds a NaN or an infinity has the
// NaN scale (byte 255), since the codes have neither: what is computed from it
// is then NaN.
#pragma once

#include "common.h"

namespace moe {
namespace mx4 {

constexpr int kGroup = 32;

// |x| bits: ordered as the magnitudes are, infinity and NaN above them all
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// scale byte of a group whose largest |x| has these bits
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const int b = max((int)(amax >> 23) - 2, 0);
    return amax >= 0x7f800000u ? 255u : amax == 0 ? 127u : (uint32_t)b;
}
// fp32 bits whose exponent field is the scale's: what the conversions below
// read (field 0 is 2^-127 to them, 255 is kept from them)
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// the codes of 8 values, value i in bits 4 i .. 4 i + 3 (0 under the NaN scale)
__device__ __forceinline__ uint32_t codes8(const float *v, uint32_t byte) {
    const float s = scale_of(byte == 255u ? 127u : byte);
    uint32_t w = 0;
    w = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
    w = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
    w = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
    w = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
    return byte == 255u ? 0u : w;
}

__device__ __forceinline__ bf16x2 pair_of(uint32_t w) { return __builtin_bit_cast(bf16x2, w); }
// the same of 8 bf16 values as they lie in memory, and the bits of their largest
// magnitude (as fp32's: infinity and NaN above the others here too)
__device__ __forceinline__ uint32_t codes8(const u32x4 &x, uint32_t byte) {
    const float s = scale_of(byte == 255u ? 127u : byte);
    uint32_t w = 0;
    w = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(x[0]), s, 0);
    w = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(x[1]), s, 1);
    w = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(x[2]), s, 2);
    w = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(x[3]), s, 3);
    return byte == 255u ? 0u : w;
}
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 mags(uint32_t pair) { return __builtin_bit_cast(u16x2, pair & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t max_bits(const u16x2 &m) { return (uint32_t)max(m[0], m[1]) << 16; }
__device__ __forceinline__ uint32_t max_bits(const u32x4 &x) {
    return max_bits(__builtin_elementwise_max(__builtin_elementwise_max(mags(x[0]), mags(x[1])),
                                              __builtin_elementwise_max(mags(x[2]), mags(x[3]))));
}

// The layout that the 4-bit product reads rows in: for each 128 columns (a
// panel, the last one filled up with zeros) 64 bytes of codes a row, row after
// row, and one word of 4 scale bytes a row. A tile's K step is then one
// contiguous piece of each.
__host__ __device__ inline int panels(int C) { return (C + 127) / 128; }

}  // namespace mx4

// Rows quantised to that layout: GEMM row r < rows is X[row_src[r] / gk]
// (X[r] if row_src is NULL), rows [rows, rows + extra) are X[0 .. extra).
// n_rows: rows in use among the first `rows` (device, NULL: all); the others
// are left as they are. A [panels(C)][ld][64], As [panels(C)][ld]. X bf16 [*][C].
// row_of: row_of[a] = the row that holds assignment a < rows, as a hint (an entry
// that does not name a row of a is passed over, and rows that no entry names are
// found all the same); a token is then read once for its gk rows. NULL: not known;
// then room for it may be given in `scratch` (int32 [rows]), and where it pays it is
// made there, in a launch before.
// With `tiles`, the tile list of the products too.
struct Mx4Panels {
    const void *X;
    const int32_t *row_src;
    int gk, C;
    int rows, extra;
    const int32_t *n_rows;
    uint8_t *A;
    uint32_t *As;
    long long ld;
    const int32_t *row_of;
    int32_t *scratch;
    int a_rows;  // rows of X (the bounds-checked build's checks only; 0: not known)
};
struct TilesJob;
hipError_t launch_mx4_panels(const Mx4Panels &p, const TilesJob *tiles, hipStream_t s);
bool mx4_panels_fit(long long rows, int C);  // in one launch, rows and extra together

// The grouped product of MXFP4 weights and MXFP4 rows (tiled_a4.hip): A holds the rows'
// panels and As their scale words, as_ld = cqs_ld their rows a panel (at least M + 256:
// whole tiles are read); output bf16, or h as panels of Cq and Cqs words (gate/up).
// Tiles of bm = tiled_a4_bm(rows, groups) rows.
hipError_t launch_tiled_a4(const GemmProblem &p, bool swiglu, int bm, hipStream_t s);
int tiled_a4_bm(long long rows, int groups);
bool tiled_a4_fits(long long max_tiles, int N, bool swiglu);  // in one launch
unsigned bounds_take_a4();  // bounds-checked build
unsigned bounds_take_mx4();

}  // namespace moe
