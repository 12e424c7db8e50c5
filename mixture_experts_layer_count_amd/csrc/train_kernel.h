// Device helpers of the training GEMMs, beside the tiled GEMM's.
#pragma once

#include "tiled_gemm_kernel.h"
#include "train.h"

namespace moe {
namespace tiled {
namespace {

// a buffer descriptor's last word: raw 32-bit elements, no swizzle
constexpr int kBufferWord3 = 0x00020000;
// copy16 from byte offset off of [base, base + bytes): zeros where the 16 bytes
// pass the end (the hardware's range check)
__device__ __forceinline__ void copy16_buffer(const void *base, uint32_t bytes, uint32_t off, uint8_t *l) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, kBufferWord3);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (AS3 void *)l, 16, off, 0, 0, 0);
}

template <int OFF>
__device__ __forceinline__ u32x2 ds_tr16_at(uint32_t addr) {
    static_assert(OFF >= 0 && OFF < 65536, "ds offset field");
    u32x2 r;
    asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(r) : "v"(addr), "i"(OFF));
    return r;
}

// Two 16-column blocks' packed bf16 results of a lane (columns 4 gq .. + 3 of
// each, gq = lane / 16) -> 8 adjacent columns, 16 (gq % 2) + 8 (gq / 2) .. of
// the pair: the odd 16-lane rows of the first block change places with the
// even ones of the second. A 16-byte store of it covers 64 contiguous bytes of
// 16 rows.
__device__ __forceinline__ u32x4 pair_columns(const f32x4 &x0, const f32x4 &x1) {
    const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16x2(x0[0], x0[1]), pack_bf16x2(x1[0], x1[1]), false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16x2(x0[2], x0[3]), pack_bf16x2(x1[2], x1[3]), false, false);
    return u32x4{lo[0], hi[0], lo[1], hi[1]};
}
__device__ __forceinline__ int pair_column(int gq) { return 16 * (gq & 1) + 8 * (gq >> 1); }

// Two 16-byte pieces of row l16 (lane % 16) in every lane -> of row l16 % 8,
// then of row 8 + l16 % 8: the first piece in lanes below 8, the second in the
// others. A row's 8 lanes then store 128 contiguous bytes at a time.
__device__ __forceinline__ void whole_lines(u32x4 &a, u32x4 &b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = a[i];
        a[i] = __builtin_amdgcn_update_dpp(x, b[i], 0x128, 0xf, 0xc, false);     // row_ror:8
        b[i] = __builtin_amdgcn_update_dpp(b[i], x, 0x128, 0xf, 0x3, false);
    }
}

}  // namespace
}  // namespace tiled
}  // namespace moe
