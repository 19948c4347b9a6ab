// Writing and reading the quantised paged KV cache: fa_kvcache_append_quant and
// fa_kvcache_read_quant (declared in include/fa.h, format in kvquant.cuh).
//
// Both are one pass over the rows that they touch.  A block takes 16 tokens of one
// sequence, all KV heads, K and V.  A warp takes 256 consecutive values of a token's
// row at a time, K and V: a thread has 8 consecutive dimensions (16 bytes of bf16)
// and always the same ones of a head, and the four threads of a 32-value group find
// its least and largest value with two shuffles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "fa_internal.h"
#include "kvquant.cuh"

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

// Page of each of the block's tokens, -1 where the table's entry is outside the pool.
__device__ __forceinline__ void kvq_pages(const KvqParams& p, int b, int n, int pos0, int* s_page) {
    if (threadIdx.x < n) {
        const int pg = p.block_table[static_cast<size_t>(b) * p.max_blocks + ((pos0 + threadIdx.x) >> p.page_shift)];
        const bool ok = static_cast<unsigned>(pg) < static_cast<unsigned>(p.num_pages);
        if (!ok) atomicCAS(p.status, 0, FA_ERR_PAGE);
        s_page[threadIdx.x] = ok ? pg : -1;
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

// The block's items: (token, 256 values of its row), dealt to the warps in turn.
struct KvqItems {
    int token, part, parts;
    __device__ __forceinline__ KvqItems(int warp, int parts_) : token(0), part(warp), parts(parts_) { wrap(); }
    __device__ __forceinline__ void wrap() {
        while (part >= parts) part -= parts, ++token;
    }
    __device__ __forceinline__ void next() {
        part += kKvqThreads / 32;
        wrap();
    }
};

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
__device__ __forceinline__ uint32_t as_word(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Quantises the thread's 8 values.  Every thread of the warp takes part in the shuffles.
// Each step of the format's definition is one fp32 operation rounded to nearest, so
// none may be contracted into another.  An infinity or NaN anywhere in the group makes
// hi - lo, and with it s, infinite or NaN (the minimum and maximum pass NaN on).
template <int BITS>
__device__ __forceinline__ void kvq_quantise(const uint4& raw, uint32_t (&code)[2], uint32_t& param) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    __nv_bfloat162 lo2 = __hmin2_nan(__hmin2_nan(as_bf162(w[0]), as_bf162(w[1])), __hmin2_nan(as_bf162(w[2]), as_bf162(w[3])));
    __nv_bfloat162 hi2 = __hmax2_nan(__hmax2_nan(as_bf162(w[0]), as_bf162(w[1])), __hmax2_nan(as_bf162(w[2]), as_bf162(w[3])));
    // lo in the low half, hi in the high half, each over the thread's 8 values
    lo2 = __hmin2_nan(lo2, __lowhigh2highlow(lo2));
    hi2 = __hmax2_nan(hi2, __lowhigh2highlow(hi2));
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, __byte_perm(as_word(lo2), as_word(hi2), 0x7610), o);
        lo2 = __hmin2_nan(lo2, as_bf162(other));  // low half
        hi2 = __hmax2_nan(hi2, as_bf162(other));  // high half
    }
    float lo = __uint_as_float(as_word(lo2) << 16);
    const float hi = __uint_as_float(as_word(hi2) & 0xFFFF0000u);
    constexpr float kMax = static_cast<float>((1 << BITS) - 1);
    float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), kMax)));
    if (!(s <= FLT_MAX)) {
        s = 0.0f;
        lo = __uint_as_float(0x7FC00000u);  // the group reads back as NaN
    } else if (s < FLT_MIN) {
        s = 0.0f;  // 1 / s would overflow
    }
    const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
    const uint32_t keep = s > 0.0f ? 0xFFFFFFFFu : 0u;
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        float t = __fmul_rn(__fsub_rn(x, lo), inv);
        // s is at least (1 - 2^-8) of the exact step: 15 / (1 - 2^-8) still rounds to 15, 255 / (1 - 2^-8) to 256
        if (BITS == 8) t = fminf(t, kMax);
        // 2^23 + 2^22 has an ulp of 1: the sum's low bits are the nearest integer
        c[i] = __float_as_uint(__fadd_rn(t, 12582912.0f));
    }
    constexpr uint32_t kMagic = 0x4B400000u;  // the bits of 2^23 + 2^22
    if constexpr (BITS == 4) {
        uint32_t x = c[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) x += c[i] << (4 * i);
        code[0] = (x - kMagic * 0x11111111u) & keep;
        code[1] = 0;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            code[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040),
                                  0x5410) & keep;
    }
    param = (__float_as_uint(lo) >> 16) | (__float_as_uint(s) & 0xFFFF0000u);
}

template <int D, int BITS>
__global__ void __launch_bounds__(kKvqThreads) fa_kvq_append(const KvqParams p) {
    using F = KvqFormat<D, BITS>;
    __shared__ int s_page[kKvqTokens];
    if (*p.status == FA_ERR_TIMEOUT) return;
    int b, first, n, pos0;
    if (!kvq_block(p, b, first, n, pos0)) return;
    kvq_pages(p, b, n, pos0, s_page);
    constexpr int C = D / 8;       // threads of a head
    constexpr int HW = 32 / C;     // heads of an item
    const int lane = threadIdx.x & 31;
    const int c = lane % C, u = c & 3, h0 = lane / C;
    const size_t block_bytes = static_cast<size_t>(F::kRowBytes) << p.page_shift;
    const int k_off = kvq_code_off<D, BITS, kKvqUnitK>(c, u);
    // V's units 2 u and 2 u + 1 of this group: of two neighbouring groups the even one writes unit 2 u of both,
    // the odd one unit 2 u + 1
    const bool odd = (c >> 2) & 1;
    const int v_off = kvq_code_off<D, BITS, kKvqUnitV>(c & ~4, 2 * u + odd);
    const int p_off = F::kParamOff + (c >> 2) * 4;
    for (KvqItems it(threadIdx.x >> 5, (p.Hkv + HW - 1) / HW); it.token < n; it.next()) {
        const int i = it.token, h = it.part * HW + h0;
        const bool live = h < p.Hkv;
        const int at = (live ? h : 0) * D + c * 8;
        const uint4 kr = __ldcs(reinterpret_cast<const uint4*>(p.k + (first + i) * p.stride_k + at));
        const uint4 vr = __ldcs(reinterpret_cast<const uint4*>(p.v + (first + i) * p.stride_v + at));
        uint32_t kc[2], vc[2], kp, vp;
        kvq_quantise<BITS>(kr, kc, kp);
        kvq_quantise<BITS>(vr, vc, vp);
        uint32_t vw[2];  // V's word or words to write
        if constexpr (BITS == 4) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, vc[0], 4);
            vw[0] = odd ? __byte_perm(other, vc[0], 0x7632) : __byte_perm(vc[0], other, 0x5410);
        } else {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? vc[0] : vc[1], 4);
            vw[0] = odd ? other : vc[0];
            vw[1] = odd ? vc[1] : other;
        }
        const int pg = s_page[i];
        if (!live || pg < 0) continue;
        const int slot = (pos0 + i) & ((1 << p.page_shift) - 1), r = slot % kKvqTile;
        const size_t off = (static_cast<size_t>(pg) * p.Hkv + h) * block_bytes +
                           static_cast<size_t>(slot / kKvqTile) * F::kTileBytes;
        uint8_t* kt = p.kpages + off;
        uint8_t* vt = p.vpages + off;
        uint8_t* kd = kt + k_off + r * F::kPlaneBytes;
        uint8_t* vd = vt + v_off + r * F::kPlaneBytes;
        if constexpr (BITS == 4) {
            *reinterpret_cast<uint32_t*>(kd) = kc[0];
            *reinterpret_cast<uint32_t*>(vd) = vw[0];
        } else {
            *reinterpret_cast<uint2*>(kd) = make_uint2(kc[0], kc[1]);
            *reinterpret_cast<uint2*>(vd) = make_uint2(vw[0], vw[1]);
        }
        if (u == 0) {
            *reinterpret_cast<uint32_t*>(kt + p_off + r * F::kParamBytes) = kp;
            *reinterpret_cast<uint32_t*>(vt + p_off + r * F::kParamBytes) = vp;
        }
    }
}

// The 8 values lo + s c of a chunk, each rounded once to the output type, written to the
// G query heads that share the KV head.
template <int D, int BITS>
__device__ __forceinline__ void kvq_emit(const uint32_t (&code)[2], uint32_t param, void* out, size_t at, int G, bool f32) {
    if (f32) {
        const float lo = __uint_as_float(param << 16), s = __uint_as_float(param & 0xFFFF0000u);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = BITS == 4 ? (code[0] >> (4 * i)) & 15u : (code[i >> 2] >> (8 * (i & 3))) & 255u;
            x[i] = fmaf(s, static_cast<float>(c), lo);
        }
        float* o = static_cast<float*>(out) + at;
        for (int g = 0; g < G; ++g, o += D) {
            *reinterpret_cast<float4*>(o) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(o + 4) = make_float4(x[4], x[5], x[6], x[7]);
        }
    } else {
        const __nv_bfloat162 lo = as_bf162(__byte_perm(param, 0, 0x1010)), s = as_bf162(__byte_perm(param, 0, 0x3232));
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 c;  // codes 2 i and 2 i + 1
            if constexpr (BITS == 4) {
                // 0x4300 | c is 128 + c in bf16
                const uint32_t up = i < 2 ? code[0] << (12 - 8 * i) : code[0] >> (8 * i - 12);
                const uint32_t two = ((code[0] >> (8 * i)) & 0xFu) | (up & 0xF0000u) | 0x43004300u;
                c = __hsub2(as_bf162(two), as_bf162(0x43004300u));
            } else {
                // 2^23 + c in fp32; less 2^23, c fits the high half
                const uint32_t w = code[i >> 1] >> (16 * (i & 1));
                const float x0 = __uint_as_float(0x4B000000u | (w & 255u)) - 8388608.0f;
                const float x1 = __uint_as_float(0x4B000000u | ((w >> 8) & 255u)) - 8388608.0f;
                c = as_bf162(__byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632));
            }
            y[i] = as_word(__hfma2(s, c, lo));
        }
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + at;
        for (int g = 0; g < G; ++g, o += D) *reinterpret_cast<uint4*>(o) = make_uint4(y[0], y[1], y[2], y[3]);
    }
}

template <int D, int BITS>
__global__ void __launch_bounds__(kKvqThreads) fa_kvq_read(const KvqParams p, int f32) {
    using F = KvqFormat<D, BITS>;
    __shared__ int s_page[kKvqTokens];
    if (*p.status == FA_ERR_TIMEOUT) return;
    int b, first, n, pos0;
    if (!kvq_block(p, b, first, n, pos0)) return;
    kvq_pages(p, b, n, pos0, s_page);
    constexpr int C = D / 8, HW = 32 / C;
    const int lane = threadIdx.x & 31;
    const int c = lane % C, u = c & 3, h0 = lane / C;
    const int G = p.H / p.Hkv;
    const size_t block_bytes = static_cast<size_t>(F::kRowBytes) << p.page_shift;
    const int k_off = kvq_code_off<D, BITS, kKvqUnitK>(c, u);
    const int v_off0 = kvq_code_off<D, BITS, kKvqUnitV>(c, 2 * u), v_off1 = kvq_code_off<D, BITS, kKvqUnitV>(c, 2 * u + 1);
    const int p_off = F::kParamOff + (c >> 2) * 4;
    for (KvqItems it(threadIdx.x >> 5, (p.Hkv + HW - 1) / HW); it.token < n; it.next()) {
        const int i = it.token, h = it.part * HW + h0;
        if (h >= p.Hkv) continue;
        const int pg = max(s_page[i], 0);  // a bad entry is flagged and read as page 0
        const int slot = (pos0 + i) & ((1 << p.page_shift) - 1), r = slot % kKvqTile;
        const size_t off = (static_cast<size_t>(pg) * p.Hkv + h) * block_bytes +
                           static_cast<size_t>(slot / kKvqTile) * F::kTileBytes;
        const uint8_t* kt = p.kpages + off;
        const uint8_t* vt = p.vpages + off;
        const uint8_t* kd = kt + k_off + r * F::kPlaneBytes;
        const uint8_t* v0 = vt + v_off0 + r * F::kPlaneBytes;
        const uint8_t* v1 = vt + v_off1 + r * F::kPlaneBytes;
        uint32_t kc[2] = {0, 0}, vc[2] = {0, 0};
        if constexpr (BITS == 4) {
            kc[0] = *reinterpret_cast<const uint32_t*>(kd);
            vc[0] = *reinterpret_cast<const uint16_t*>(v0) |
                    (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(v1)) << 16);
        } else {
            const uint2 k2 = *reinterpret_cast<const uint2*>(kd);
            kc[0] = k2.x, kc[1] = k2.y;
            vc[0] = *reinterpret_cast<const uint32_t*>(v0);
            vc[1] = *reinterpret_cast<const uint32_t*>(v1);
        }
        const uint32_t kp = *reinterpret_cast<const uint32_t*>(kt + p_off + r * F::kParamBytes);
        const uint32_t vp = *reinterpret_cast<const uint32_t*>(vt + p_off + r * F::kParamBytes);
        const size_t at = (static_cast<size_t>(first + i) * p.H + h * G) * D + c * 8;
        kvq_emit<D, BITS>(kc, kp, p.k_out, at, G, f32 != 0);
        kvq_emit<D, BITS>(vc, vp, p.v_out, at, G, f32 != 0);
    }
}

template <typename F>
cudaError_t by_format(int d, int bits, F&& launch) {
    if (bits == 4) {
        if (d == 64) launch(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
        else if (d == 128) launch(std::integral_constant<int, 128>(), std::integral_constant<int, 4>());
        else launch(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
    } else {
        if (d == 64) launch(std::integral_constant<int, 64>(), std::integral_constant<int, 8>());
        else if (d == 128) launch(std::integral_constant<int, 128>(), std::integral_constant<int, 8>());
        else launch(std::integral_constant<int, 256>(), std::integral_constant<int, 8>());
    }
    return cudaGetLastError();
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
        fa_kvq_append<D(), BITS()><<<static_cast<unsigned>(B * chunks), kKvqThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
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
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.total = total;
    p.max_rows = max_seqlen;
    p.num_pages = num_pages;
    p.page_shift = kvq_page_shift(page_size);
    p.max_blocks = max_blocks;
    p.chunks = static_cast<int>(chunks);
    const int f32 = o_dtype == FA_DT_F32;
    const cudaError_t e = by_format(d, bits, [&](auto D, auto BITS) {
        fa_kvq_read<D(), BITS()><<<static_cast<unsigned>(B * chunks), kKvqThreads, 0, static_cast<cudaStream_t>(stream)>>>(p, f32);
    });
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
