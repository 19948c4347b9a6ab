// Writing and reading the quantised paged KV cache: fa_kvcache_append_quant and
// fa_kvcache_read_quant (declared in include/fa.h, format in kvquant.cuh).
//
// Both are one pass over the rows that they touch.  A block takes 16 tokens of one
// sequence, all KV heads, K and V, as one run of pieces dealt to its threads in order:
// 16 consecutive values of K and of V, half a group.  Two threads do what is done once
// a group, and a piece of bf16 is one 32-byte sector.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "fa_internal.h"
#include "kvquant.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kKvqThreads = 256;
constexpr int kKvqTokens = 16;  // tokens of a block

struct KvqParams {
    const __nv_bfloat16* k;  // append: token t's heads at k + t * stride_k
    const __nv_bfloat16* v;
    long long stride_k, stride_v;
    uint8_t* kpages;         // [num_pages, Hkv, page_size / 16 tiles]
    uint8_t* vpages;
    const int* cu;           // [B + 1] packed rows of each sequence
    const int* block_table;  // [B, max_blocks]
    const int* kv_lens;      // [B]
    void* k_out;             // read: [total, H, D]
    void* v_out;
    int* status;
    int B, H, Hkv, total, max_rows, num_pages, page_shift, max_blocks, chunks;
    bool wide;               // read: k_out and v_out are 32-byte aligned
};

// What a block works on: rows [first, first + n) of the packed rows, which are the
// positions from pos0 on of sequence b.  False if the sequence has nothing for this
// block or its numbers are invalid (then flagged once, by its first block).
__device__ __forceinline__ bool kvq_block(const KvqParams& p, int& b, int& first, int& n, int& pos0) {
    b = blockIdx.x / p.chunks;
    const int chunk = blockIdx.x - b * p.chunks;
    const int r0 = p.cu[b], r1 = p.cu[b + 1], len = p.kv_lens[b];
    const int rows = r1 - r0;
    int bad = 0;
    if (len < 0 || (static_cast<long long>(len) > (static_cast<long long>(p.max_blocks) << p.page_shift)))
        bad = FA_ERR_KV_LEN;
    else if (r0 < 0 || r1 < r0 || r1 > p.total || rows > p.max_rows || rows > len)
        bad = FA_ERR_SEQLEN;
    if (bad) {
        if (chunk == 0 && threadIdx.x == 0) atomicCAS(p.status, 0, bad);
        return false;
    }
    const int i0 = chunk * kKvqTokens;
    first = r0 + i0;
    n = min(kKvqTokens, rows - i0);
    pos0 = len - rows + i0;
    return n > 0;
}

// Byte offset in a pool of each of the block's tokens' tile (KV head 0), or -1 where
// the table's entry is outside the pool (read as page 0 if `clamp`).
template <int D, int BITS>
__device__ __forceinline__ void kvq_tiles(const KvqParams& p, int b, int n, int pos0, bool clamp, long long* s_tile) {
    using F = KvqFormat<D, BITS>;
    if (threadIdx.x < n) {
        const int pos = pos0 + threadIdx.x;
        int pg = p.block_table[static_cast<size_t>(b) * p.max_blocks + (pos >> p.page_shift)];
        const bool ok = static_cast<unsigned>(pg) < static_cast<unsigned>(p.num_pages);
        if (!ok) {
            atomicCAS(p.status, 0, FA_ERR_PAGE);
            pg = 0;
        }
        const int slot = pos & ((1 << p.page_shift) - 1);
        const long long at = (static_cast<long long>(pg) * p.Hkv * F::kRowBytes << p.page_shift) +
                             static_cast<long long>(slot / kKvqTile) * F::kTileBytes;
        s_tile[threadIdx.x] = ok || clamp ? at : -1;
    }
    __syncthreads();
}

// Byte offset in a tile of unit `u` of the group that holds 8-dimension chunk c, for token row 0.
template <int D, int BITS, int U>
__device__ __forceinline__ int kvq_code_off(int c, int u) {
    using F = KvqFormat<D, BITS>;
    const int plane = c / (F::kPlaneDims / 8), g = (c % (F::kPlaneDims / 8)) >> 2;
    return plane * (kKvqTile * F::kPlaneBytes) + (u * F::kPlaneGroups + g) * (U * BITS / 8);
}

// i / n for i < 16 n and n < 65536: the quotient's distance to the next integer, at
// least 1 / (2 n), is far above the product's rounding.
__device__ __forceinline__ int kvq_div(int i, float inv_n) { return __float2int_rz((static_cast<float>(i) + 0.5f) * inv_n); }

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
__device__ __forceinline__ uint32_t as_word(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Quantises the thread's 16 values, half of a group whose other half the neighbouring
// thread has: code[i] holds BITS * i / 4 bits and on.  Every thread of the warp takes
// part in the shuffle.  Each step of the format's definition is one fp32 operation
// rounded to nearest, so none may be contracted into another.  An infinity or NaN
// anywhere in the group makes hi - lo, and with it s, infinite or NaN (the minimum and
// maximum pass NaN on).
template <int BITS>
__device__ __forceinline__ void kvq_quantise(const uint32_t (&w)[8], uint32_t (&code)[BITS / 2], uint32_t& param) {
    __nv_bfloat162 lo2 = as_bf162(w[0]), hi2 = lo2;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo2 = __hmin2_nan(lo2, as_bf162(w[i]));
        hi2 = __hmax2_nan(hi2, as_bf162(w[i]));
    }
    lo2 = __hmin2_nan(lo2, __lowhigh2highlow(lo2));
    hi2 = __hmax2_nan(hi2, __lowhigh2highlow(hi2));
    // lo in the low half, hi in the high half
    const uint32_t other = __shfl_xor_sync(0xffffffffu, __byte_perm(as_word(lo2), as_word(hi2), 0x7610), 1);
    lo2 = __hmin2_nan(lo2, as_bf162(other));  // low half
    hi2 = __hmax2_nan(hi2, as_bf162(other));  // high half
    float lo = __uint_as_float(as_word(lo2) << 16);
    const float hi = __uint_as_float(as_word(hi2) & 0xFFFF0000u);
    constexpr float kMax = static_cast<float>((1 << BITS) - 1);
    // (hi - lo) / kMax rounded to nearest, by Markstein's theorem: with y the nearest to 1 / kMax, the residual of
    // q = d y is exact and one fused step rounds correctly (from d = kMax 2^-126 on, below which s is 0)
    constexpr float y = 1.0f / kMax;
    const float d = __fsub_rn(hi, lo), q = __fmul_rn(d, y);
    float s = __bfloat162float(__float2bfloat16_rn(fmaf(fmaf(-kMax, q, d), y, q)));
    // 1 / s rounded to nearest, by a step of Newton's method: the approximation is within 2^-22, the step squares that, and
    // 1 / s of an 8-bit s is a power of two or at least 2^-34 of itself away from where the rounding turns
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    float inv = fmaf(fmaf(-s, r, 1.0f), r, r);
    uint32_t keep = 0xFFFFFFFFu;
    if (!(s >= FLT_MIN && s <= FLT_MAX)) {  // below, 1 / s would overflow: the group stands for lo
        if (!(s <= FLT_MAX)) lo = __uint_as_float(0x7FC00000u);  // it reads back as NaN
        s = 0.0f, inv = 0.0f, keep = 0u;
    }
    uint32_t c[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float x = __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        float t = __fmul_rn(__fsub_rn(x, lo), inv);
        // s is at least (1 - 2^-8) of the exact step: 15 / (1 - 2^-8) still rounds to 15, 255 / (1 - 2^-8) to 256
        if (BITS == 8) t = fminf(t, kMax);
        // 2^23 + 2^22 has an ulp of 1: the sum's low bits are the nearest integer
        c[i] = __float_as_uint(__fadd_rn(t, 12582912.0f));
    }
    constexpr uint32_t kMagic = 0x4B400000u;  // the bits of 2^23 + 2^22
    if constexpr (BITS == 4) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t x = c[8 * j];
#pragma unroll
            for (int i = 1; i < 8; ++i) x += c[8 * j + i] << (4 * i);
            code[j] = (x - kMagic * 0x11111111u) & keep;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            code[j] = __byte_perm(__byte_perm(c[4 * j], c[4 * j + 1], 0x0040), __byte_perm(c[4 * j + 2], c[4 * j + 3], 0x0040),
                                  0x5410) & keep;
    }
    param = (__float_as_uint(lo) >> 16) | __float_as_uint(s);
}

// Where a thread's pieces lie: D / 16 divides the threads of a block, so a thread always
// has the same dimensions of a head.  Of V, it has units 4 half to 4 half + 3 of its
// group; of two neighbouring groups the even one's thread stores (loads) the first two
// of both, the odd one's the others, so that an access holds both groups' units.
template <int D, int BITS>
struct KvqPiece {
    using F = KvqFormat<D, BITS>;
    static constexpr int kUnitStepK = F::kPlaneGroups * kKvqUnitK * BITS / 8;  // from a unit to the next one of its group
    static constexpr int kUnitStepV = F::kPlaneGroups * kKvqUnitV * BITS / 8;
    int c, k_off, v_off, p_off;
    bool odd;
    __device__ __forceinline__ explicit KvqPiece(int thread) {
        c = thread % (D / 16);
        odd = (c >> 1) & 1;
        k_off = kvq_code_off<D, BITS, kKvqUnitK>(2 * c, 2 * (c & 1));
        v_off = kvq_code_off<D, BITS, kKvqUnitV>((2 * c) & ~4, 4 * (c & 1) + 2 * odd);
        p_off = F::kParamOff + (c >> 1) * 4;
    }
    // The piece's codes of V to the two units that the thread stores, and back.
    __device__ __forceinline__ void to_stored(const uint32_t (&vc)[BITS / 2], uint32_t (&x)[BITS / 2]) const {
        if constexpr (BITS == 4) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? vc[0] : vc[1], 2);
            const uint32_t even_g = odd ? other : vc[0], odd_g = odd ? vc[1] : other;
            x[0] = __byte_perm(even_g, odd_g, 0x5410);
            x[1] = __byte_perm(even_g, odd_g, 0x7632);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? vc[j] : vc[2 + j], 2);
                x[2 * j] = odd ? other : vc[j];
                x[2 * j + 1] = odd ? vc[2 + j] : other;
            }
        }
    }
    __device__ __forceinline__ void from_stored(const uint32_t (&x)[BITS / 2], uint32_t (&vc)[BITS / 2]) const {
        if constexpr (BITS == 4) {
            const uint32_t even_g = __byte_perm(x[0], x[1], 0x5410), odd_g = __byte_perm(x[0], x[1], 0x7632);
            const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? even_g : odd_g, 2);
            vc[0] = odd ? other : even_g;
            vc[1] = odd ? odd_g : other;
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? x[2 * j] : x[2 * j + 1], 2);
                vc[j] = odd ? other : x[2 * j];
                vc[2 + j] = odd ? x[2 * j + 1] : other;
            }
        }
    }
};

template <int D, int BITS>
__global__ void __launch_bounds__(kKvqThreads) fa_kvq_append(const KvqParams p) {
    using F = KvqFormat<D, BITS>;
    __shared__ long long s_tile[kKvqTokens];
    kvq_wait_for_previous();
    if (*p.status == FA_ERR_TIMEOUT) return;
    int b, first, n, pos0;
    if (!kvq_block(p, b, first, n, pos0)) return;
    kvq_tiles<D, BITS>(p, b, n, pos0, false, s_tile);
    const KvqPiece<D, BITS> piece(threadIdx.x);
    constexpr int C = D / 16;  // threads of a head
    const int row = p.Hkv * C, total = n * row;
    const float inv_row = 1.0f / static_cast<float>(row);
    const uint32_t block_bytes = static_cast<uint32_t>(F::kRowBytes) << p.page_shift;
    for (int e0 = 0; e0 < total; e0 += kKvqThreads) {
        const int e = e0 + threadIdx.x;
        const int at = min(e, total - C + piece.c);  // the last head's, for threads past the end
        const int i = kvq_div(at, inv_row), y = at - i * row;
        uint32_t kw[8], vw[8];
        {
            const uint4* kf = reinterpret_cast<const uint4*>(p.k + (first + i) * p.stride_k + y * 16);
            const uint4* vf = reinterpret_cast<const uint4*>(p.v + (first + i) * p.stride_v + y * 16);
            const uint4 k0 = kf[0], k1 = kf[1], v0 = vf[0], v1 = vf[1];
            kw[0] = k0.x, kw[1] = k0.y, kw[2] = k0.z, kw[3] = k0.w, kw[4] = k1.x, kw[5] = k1.y, kw[6] = k1.z, kw[7] = k1.w;
            vw[0] = v0.x, vw[1] = v0.y, vw[2] = v0.z, vw[3] = v0.w, vw[4] = v1.x, vw[5] = v1.y, vw[6] = v1.z, vw[7] = v1.w;
        }
        uint32_t kc[BITS / 2], vc[BITS / 2], kp, vp;
        kvq_quantise<BITS>(kw, kc, kp);
        kvq_quantise<BITS>(vw, vc, vp);
        uint32_t x[BITS / 2];
        piece.to_stored(vc, x);
        const long long tile = s_tile[i];
        if (e >= total || tile < 0) continue;
        const int r = static_cast<unsigned>(pos0 + i) % kKvqTile;
        const size_t off = tile + static_cast<uint64_t>(static_cast<unsigned>(y) / C) * block_bytes;
        uint8_t* kt = p.kpages + off;
        uint8_t* vt = p.vpages + off;
        uint8_t* kd = kt + piece.k_off + r * F::kPlaneBytes;
        uint8_t* vd = vt + piece.v_off + r * F::kPlaneBytes;
        if constexpr (BITS == 4) {
            *reinterpret_cast<uint32_t*>(kd) = kc[0];
            *reinterpret_cast<uint32_t*>(kd + piece.kUnitStepK) = kc[1];
            *reinterpret_cast<uint32_t*>(vd) = x[0];
            *reinterpret_cast<uint32_t*>(vd + piece.kUnitStepV) = x[1];
        } else {
            *reinterpret_cast<uint2*>(kd) = make_uint2(kc[0], kc[1]);
            *reinterpret_cast<uint2*>(kd + piece.kUnitStepK) = make_uint2(kc[2], kc[3]);
            *reinterpret_cast<uint2*>(vd) = make_uint2(x[0], x[1]);
            *reinterpret_cast<uint2*>(vd + piece.kUnitStepV) = make_uint2(x[2], x[3]);
        }
        if ((piece.c & 1) == 0) {
            *reinterpret_cast<uint32_t*>(kt + piece.p_off + r * F::kParamBytes) = kp;
            *reinterpret_cast<uint32_t*>(vt + piece.p_off + r * F::kParamBytes) = vp;
        }
    }
}

// The 16 values lo + s c of a piece, each rounded once to the output type, written to the
// G query heads that share the KV head.
template <int D, int BITS, bool F32>
__device__ __forceinline__ void kvq_emit(const uint32_t (&code)[BITS / 2], uint32_t param, void* out, size_t at, int G,
                                         bool wide) {
    if constexpr (F32) {
        const float lo = __uint_as_float(param << 16), s = __uint_as_float(param & 0xFFFF0000u);
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t c = BITS == 4 ? (code[i / 8] >> (4 * (i % 8))) & 15u : (code[i / 4] >> (8 * (i % 4))) & 255u;
            x[i] = fmaf(s, __uint_as_float(0x4B000000u | c) - 8388608.0f, lo);
        }
        float* o = static_cast<float*>(out) + at;
        for (int g = 0; g < G; ++g, o += D)
#pragma unroll
            for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4*>(o + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
        const __nv_bfloat162 lo = as_bf162(__byte_perm(param, 0, 0x1010)), s = as_bf162(__byte_perm(param, 0, 0x3232));
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            __nv_bfloat162 c;  // codes 2 i and 2 i + 1
            if constexpr (BITS == 4) {
                // 0x4300 | c is 128 + c in bf16
                const uint32_t w = code[i / 4];
                const int b = 8 * (i % 4);
                const uint32_t up = b < 12 ? w << (12 - b) : w >> (b - 12);
                c = __hsub2(as_bf162(((w >> b) & 0xFu) | (up & 0xF0000u) | 0x43004300u), as_bf162(0x43004300u));
            } else {
                // 2^23 + c in fp32; less 2^23, c fits the high half
                const uint32_t w = code[i / 2];
                const float x0 = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + 2 * (i & 1))) - 8388608.0f;
                const float x1 = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + 2 * (i & 1) + 1)) - 8388608.0f;
                c = as_bf162(__byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632));
            }
            y[i] = as_word(__hfma2(s, c, lo));
        }
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + at;
        for (int g = 0; g < G; ++g, o += D) {
            if (wide) {  // 32-byte aligned outputs: whole sectors
                st_global_v8(o, y);
            } else {
                *reinterpret_cast<uint4*>(o) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4*>(o + 8) = make_uint4(y[4], y[5], y[6], y[7]);
            }
        }
    }
}

template <int D, int BITS, bool F32>
__global__ void __launch_bounds__(kKvqThreads) fa_kvq_read(const KvqParams p) {
    using F = KvqFormat<D, BITS>;
    __shared__ long long s_tile[kKvqTokens];
    kvq_wait_for_previous();
    if (*p.status == FA_ERR_TIMEOUT) return;
    int b, first, n, pos0;
    if (!kvq_block(p, b, first, n, pos0)) return;
    kvq_tiles<D, BITS>(p, b, n, pos0, true, s_tile);  // a bad entry is flagged and read as page 0
    const KvqPiece<D, BITS> piece(threadIdx.x);
    constexpr int C = D / 16;
    const int row = p.Hkv * C, total = n * row, G = p.H / p.Hkv;
    const float inv_row = 1.0f / static_cast<float>(row);
    const uint32_t block_bytes = static_cast<uint32_t>(F::kRowBytes) << p.page_shift;
    const bool wide = p.wide;
    constexpr int kAtOnce = 2;  // pieces whose loads are in flight together
    for (int e0 = 0; e0 < total; e0 += kAtOnce * kKvqThreads) {
        uint32_t kc[kAtOnce][BITS / 2], vx[kAtOnce][BITS / 2], kp[kAtOnce], vp[kAtOnce];
        size_t to[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int e = min(e0 + j * kKvqThreads + static_cast<int>(threadIdx.x), total - C + piece.c);  // the last head's past the end
            const int i = kvq_div(e, inv_row), h = static_cast<unsigned>(e - i * row) / C;
            const int r = static_cast<unsigned>(pos0 + i) % kKvqTile;
            const size_t off = s_tile[i] + static_cast<uint64_t>(static_cast<uint32_t>(h)) * block_bytes;
            const uint8_t* kt = p.kpages + off;
            const uint8_t* vt = p.vpages + off;
            const uint8_t* kd = kt + piece.k_off + r * F::kPlaneBytes;
            const uint8_t* vd = vt + piece.v_off + r * F::kPlaneBytes;
            if constexpr (BITS == 4) {
                kc[j][0] = *reinterpret_cast<const uint32_t*>(kd);
                kc[j][1] = *reinterpret_cast<const uint32_t*>(kd + piece.kUnitStepK);
                vx[j][0] = *reinterpret_cast<const uint32_t*>(vd);
                vx[j][1] = *reinterpret_cast<const uint32_t*>(vd + piece.kUnitStepV);
            } else {
                const uint2 k0 = *reinterpret_cast<const uint2*>(kd), k1 = *reinterpret_cast<const uint2*>(kd + piece.kUnitStepK);
                const uint2 v0 = *reinterpret_cast<const uint2*>(vd), v1 = *reinterpret_cast<const uint2*>(vd + piece.kUnitStepV);
                kc[j][0] = k0.x, kc[j][1] = k0.y, kc[j][2] = k1.x, kc[j][3] = k1.y;
                vx[j][0] = v0.x, vx[j][1] = v0.y, vx[j][2] = v1.x, vx[j][3] = v1.y;
            }
            kp[j] = *reinterpret_cast<const uint32_t*>(kt + piece.p_off + r * F::kParamBytes);
            vp[j] = *reinterpret_cast<const uint32_t*>(vt + piece.p_off + r * F::kParamBytes);
            to[j] = (static_cast<size_t>(first + i) * p.H + h * G) * D + piece.c * 16;
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            uint32_t vc[BITS / 2];
            piece.from_stored(vx[j], vc);
            if (e0 + j * kKvqThreads + static_cast<int>(threadIdx.x) >= total) continue;
            kvq_emit<D, BITS, F32>(kc[j], kp[j], p.k_out, to[j], G, wide);
            kvq_emit<D, BITS, F32>(vc, vp[j], p.v_out, to[j], G, wide);
        }
    }
}

// launch(D, BITS) of the kernels for a head dimension and code width.
template <typename F>
cudaError_t by_format(int d, int bits, F&& launch) {
    if (bits == 4) {
        if (d == 64) return launch(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
        if (d == 128) return launch(std::integral_constant<int, 128>(), std::integral_constant<int, 4>());
        return launch(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
    }
    if (d == 64) return launch(std::integral_constant<int, 64>(), std::integral_constant<int, 8>());
    if (d == 128) return launch(std::integral_constant<int, 128>(), std::integral_constant<int, 8>());
    return launch(std::integral_constant<int, 256>(), std::integral_constant<int, 8>());
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" size_t fa_kvcache_quant_page_bytes(int page_size, int d, int bits) {
    if (kvq_check_pool(1, 1, 1, 1, page_size, 1, d, bits) != FA_OK) return 0;
    return static_cast<size_t>(page_size) * kvq_row_bytes(d, bits);
}

extern "C" int fa_kvcache_append_quant(const void* k, const void* v, long long stride_k, long long stride_v, void* kpages,
                                       void* vpages, const int* cu_seqlens_new, const int* block_table,
                                       const int* kv_lens, int B, int Hkv, int total_new, int max_seqlen_new,
                                       int num_pages, int page_size, int max_blocks, int d, int bits, void* stream) {
    if (!k || !v || !kpages || !vpages || !cu_seqlens_new || !block_table || !kv_lens) return FA_ERR_INVALID_ARG;
    int rc = kvq_check_pool(B, Hkv, Hkv, num_pages, page_size, max_blocks, d, bits);
    if (rc != FA_OK) return rc;
    if (total_new < 0 || max_seqlen_new < 0) return FA_ERR_INVALID_ARG;
    if (stride_k < static_cast<long long>(Hkv) * d || stride_v < static_cast<long long>(Hkv) * d || stride_k % 8 != 0 ||
        stride_v % 8 != 0)
        return FA_ERR_INVALID_ARG;
    if (!kvq_aligned(k, 16) || !kvq_aligned(v, 16) || !kvq_aligned(kpages, 16) || !kvq_aligned(vpages, 16) ||
        !kvq_aligned(cu_seqlens_new, 4) || !kvq_aligned(block_table, 4) || !kvq_aligned(kv_lens, 4))
        return FA_ERR_INVALID_ARG;
    const long long chunks = (static_cast<long long>(max_seqlen_new) + kKvqTokens - 1) / kKvqTokens;
    if (B * chunks > 0x7FFFFFFFLL) return FA_ERR_INVALID_ARG;
    if (total_new == 0 || chunks == 0) return FA_OK;
    KvqParams p{};
    if ((rc = prepare_device(&p.status)) != FA_OK) return rc;
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.stride_k = stride_k;
    p.stride_v = stride_v;
    p.kpages = static_cast<uint8_t*>(kpages);
    p.vpages = static_cast<uint8_t*>(vpages);
    p.cu = cu_seqlens_new;
    p.block_table = block_table;
    p.kv_lens = kv_lens;
    p.B = B;
    p.H = p.Hkv = Hkv;
    p.total = total_new;
    p.max_rows = max_seqlen_new;
    p.num_pages = num_pages;
    p.page_shift = kvq_page_shift(page_size);
    p.max_blocks = max_blocks;
    p.chunks = static_cast<int>(chunks);
    const cudaError_t e = by_format(d, bits, [&](auto D, auto BITS) {
        return kvq_launch(fa_kvq_append<D(), BITS()>, static_cast<unsigned>(B * chunks), kKvqThreads, 0,
                          static_cast<cudaStream_t>(stream), p);
    });
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" int fa_kvcache_read_quant(const void* kpages, const void* vpages, const int* cu_seqlens, const int* block_table,
                                     const int* kv_lens, void* k_out, void* v_out, int B, int H, int Hkv, int total,
                                     int max_seqlen, int num_pages, int page_size, int max_blocks, int d, int bits,
                                     int o_dtype, void* stream) {
    if (!kpages || !vpages || !cu_seqlens || !block_table || !kv_lens || !k_out || !v_out) return FA_ERR_INVALID_ARG;
    int rc = kvq_check_pool(B, H, Hkv, num_pages, page_size, max_blocks, d, bits);
    if (rc != FA_OK) return rc;
    if (o_dtype != FA_DT_BF16 && o_dtype != FA_DT_F32) return FA_ERR_UNSUPPORTED;
    if (total < 0 || max_seqlen < 0) return FA_ERR_INVALID_ARG;
    if (!kvq_aligned(kpages, 16) || !kvq_aligned(vpages, 16) || !kvq_aligned(k_out, 16) || !kvq_aligned(v_out, 16) ||
        !kvq_aligned(cu_seqlens, 4) || !kvq_aligned(block_table, 4) || !kvq_aligned(kv_lens, 4))
        return FA_ERR_INVALID_ARG;
    const long long chunks = (static_cast<long long>(max_seqlen) + kKvqTokens - 1) / kKvqTokens;
    if (B * chunks > 0x7FFFFFFFLL) return FA_ERR_INVALID_ARG;
    if (total == 0 || chunks == 0) return FA_OK;
    KvqParams p{};
    if ((rc = prepare_device(&p.status)) != FA_OK) return rc;
    p.kpages = static_cast<uint8_t*>(const_cast<void*>(kpages));
    p.vpages = static_cast<uint8_t*>(const_cast<void*>(vpages));
    p.cu = cu_seqlens;
    p.block_table = block_table;
    p.kv_lens = kv_lens;
    p.k_out = k_out;
    p.v_out = v_out;
    p.wide = kvq_aligned(k_out, 32) && kvq_aligned(v_out, 32);
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.total = total;
    p.max_rows = max_seqlen;
    p.num_pages = num_pages;
    p.page_shift = kvq_page_shift(page_size);
    p.max_blocks = max_blocks;
    p.chunks = static_cast<int>(chunks);
    const cudaError_t e = by_format(d, bits, [&](auto D, auto BITS) {
        const unsigned grid = static_cast<unsigned>(B * chunks);
        const cudaStream_t st = static_cast<cudaStream_t>(stream);
        return o_dtype == FA_DT_F32 ? kvq_launch(fa_kvq_read<D(), BITS(), true>, grid, kKvqThreads, 0, st, p)
                                    : kvq_launch(fa_kvq_read<D(), BITS(), false>, grid, kKvqThreads, 0, st, p);
    });
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
