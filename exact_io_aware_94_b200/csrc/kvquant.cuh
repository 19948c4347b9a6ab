// Format of the quantised paged KV cache and its device-side error checks,
// shared by the kernels that write it, read it back and attend over it.
//
// A group of 32 values of a row is stored as its least value lo (bf16, exact), a
// step s (bf16) and unsigned codes c of BITS = 4 or 8 bits; it stands for lo + s c.
//
// The cache of one (page, KV head) is a run of page_size / 16 tiles of 16 tokens:
//   codes   kPlanes planes of [16 tokens][kPlaneBytes]
//   params  [16 tokens][D / 32] words: lo in bits 0-15, s in bits 16-31
// A plane holds kPlaneDims dimensions (kPlaneGroups groups) of each token, at most
// 64 bytes, so that eight rows of 16-byte pieces read side by side touch every
// shared-memory bank once.  Inside a token's kPlaneBytes, the groups' units of U
// consecutive dimensions are interleaved: unit u of group g (dimensions 32 g + U u
// and up) starts U BITS / 8 * (u * kPlaneGroups + g) bytes in, low nibble first.
// U is 8 for K and 4 for V: what one thread of an m16n8k16 A fragment wants of
// every group is then contiguous (see decode_quant.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_internal.h"

namespace fa {

constexpr int kKvqGroup = 32;   // values that share lo and s
constexpr int kKvqTile = 16;    // tokens of a tile; page sizes are multiples of it
constexpr int kKvqUnitK = 8, kKvqUnitV = 4;
constexpr int kKvqMaxHeads = 2048;  // KV heads: a row is 32,768 pieces of 16 at most, a page's bytes / 16 fit uint32

template <int D, int BITS>
struct KvqFormat {
    static constexpr int kCodeBytes = D * BITS / 8;  // of one token
    static constexpr int kParamBytes = D / kKvqGroup * 4;
    static constexpr int kRowBytes = kCodeBytes + kParamBytes;
    static constexpr int kTileBytes = kKvqTile * kRowBytes;
    static constexpr int kPlaneBytes = kCodeBytes < 64 ? kCodeBytes : 64;
    static constexpr int kPlanes = kCodeBytes / kPlaneBytes;
    static constexpr int kPlaneDims = kPlaneBytes * 8 / BITS;
    static constexpr int kPlaneGroups = kPlaneDims / kKvqGroup;
    static constexpr int kGroups = D / kKvqGroup;
    static constexpr int kParamOff = kKvqTile * kCodeBytes;
};

// Bytes of a token's codes and (lo, s) pairs.
__host__ __device__ constexpr int kvq_row_bytes(int d, int bits) { return d * bits / 8 + d / kKvqGroup * 4; }

// Checks that the host entry points share: sizes of a pool and its block table.
inline int kvq_check_pool(int B, int H, int Hkv, int num_pages, int page_size, int max_blocks, int d, int bits) {
    if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
    if (bits != 4 && bits != 8) return FA_ERR_UNSUPPORTED;
    if (B <= 0 || H <= 0 || Hkv <= 0 || H % Hkv != 0 || num_pages <= 0 || max_blocks <= 0) return FA_ERR_INVALID_ARG;
    if (Hkv > kKvqMaxHeads) return FA_ERR_INVALID_ARG;
    if (page_size < kKvqTile || page_size > 65536 || (page_size & (page_size - 1)) != 0) return FA_ERR_INVALID_ARG;
    if (static_cast<long long>(max_blocks) * page_size > 0x7FFFFFFFLL || static_cast<long long>(B) * H > (1LL << 30) ||
        static_cast<long long>(B) * max_blocks > 0x7FFFFFFFLL)
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}
inline int kvq_page_shift(int page_size) {
    int shift = 0;
    while ((1 << shift) < page_size) ++shift;
    return shift;
}
// Launches a kernel whose blocks may be set up while the stream's previous kernel ends; it has to call
// kvq_wait_for_previous before it touches memory.  Calls in a row are 1 to 2.5 us closer so (decode when this came: 96 x
// 4,001 keys at d = 64 30.0 -> 28.0 us, 5 x 65,536 at d = 256 41.0 -> 38.4 us).
template <typename... P, typename... A>
inline cudaError_t kvq_launch(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// Returns once the stream's previous kernel has ended and its writes are visible.
__device__ __forceinline__ void kvq_wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
inline bool kvq_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace fa
