// Single-query decode over the quantised paged cache: fa_decode_paged_quant
// (declared in include/fa.h, cache format in kvquant.cuh).
//
// With K and V held as lo + s c per group of 32 dimensions, a score is
//     q . k_j = sum_g [ s_jg (q_g . c_jg) + lo_jg sum(q_g) ]
// and the output follows the online softmax of fa_decode: running max, running
// sum, unnormalised accumulator, split over the keys and merged by log-sum-exp.
//   fa_decode_quant_split    a CTA per (b, h, split): every kMaxSplits-th tile of 128 keys
//   fa_decode_quant_combine  a CTA per (b, h): merges the splits
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fa_internal.h"
#include "kvquant.cuh"

namespace fa {
namespace {

constexpr int kSplitKeys = 128;  // keys of a tile, threads of a CTA
constexpr int kMaxSplits = 64;

struct DecodeQuantParams {
    const __nv_bfloat16* q;  // [B, H, D]
    const uint8_t* kpages;
    const uint8_t* vpages;
    const int* block_table;
    const int* kv_lens;
    void* o;
    float* lse;
    int* status;
    float* part_o;    // [B * H, splits, D], normalised
    float* part_lse;  // [B * H, splits]
    int B, H, Hkv, num_pages, page_shift, max_blocks, splits, cap;
    float scale;
    int o_dtype;
};

template <int D, int BITS, int U>
__device__ __forceinline__ uint32_t code_at(const uint8_t* tile, int r, int dim) {
    using F = KvqFormat<D, BITS>;
    const int plane = dim / F::kPlaneDims, i = dim % F::kPlaneDims;
    const int g = i / kKvqGroup, u = (i % kKvqGroup) / U, j = i % U;
    const int bit = (u * F::kPlaneGroups + g) * U * BITS + j * BITS;
    const uint32_t byte = tile[plane * kKvqTile * F::kPlaneBytes + r * F::kPlaneBytes + bit / 8];
    return (byte >> (bit % 8)) & ((1u << BITS) - 1u);
}

template <int D, int BITS>
__global__ void __launch_bounds__(kSplitKeys) fa_decode_quant_split(const DecodeQuantParams p) {
    using F = KvqFormat<D, BITS>;
    __shared__ float s_q[D], s_qsum[F::kGroups], s_p[kSplitKeys], s_red[kSplitKeys / 32];
    __shared__ const uint8_t* s_v[kSplitKeys];
    if (*p.status == FA_ERR_TIMEOUT) return;
    const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H, hkv = h / (p.H / p.Hkv);
    const int tid = threadIdx.x;
    int len = p.kv_lens[b];
    if (len < 0 || len > p.cap) {
        if (tid == 0) atomicCAS(p.status, 0, FA_ERR_KV_LEN);
        len = len < 0 ? 0 : p.cap;
    }
    for (int i = tid; i < D; i += kSplitKeys) s_q[i] = __bfloat162float(p.q[static_cast<size_t>(bh) * D + i]);
    __syncthreads();
    if (tid < F::kGroups) {
        float a = 0.0f;
        for (int i = 0; i < kKvqGroup; ++i) a += s_q[tid * kKvqGroup + i];
        s_qsum[tid] = a;
    }
    const size_t block_bytes = static_cast<size_t>(F::kRowBytes) << p.page_shift;
    float m = -INFINITY, l = 0.0f, acc[(D + kSplitKeys - 1) / kSplitKeys] = {};
    for (int k0 = blockIdx.y * kSplitKeys; k0 < len; k0 += gridDim.y * kSplitKeys) {
        __syncthreads();
        const int key = k0 + tid;
        float x = -INFINITY;
        if (key < len) {
            int pg = p.block_table[static_cast<size_t>(b) * p.max_blocks + (key >> p.page_shift)];
            if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.num_pages)) {
                atomicCAS(p.status, 0, FA_ERR_PAGE);
                pg = 0;
            }
            const int slot = key & ((1 << p.page_shift) - 1), r = slot % kKvqTile;
            const size_t off = (static_cast<size_t>(pg) * p.Hkv + hkv) * block_bytes +
                               static_cast<size_t>(slot / kKvqTile) * F::kTileBytes;
            const uint8_t* kt = p.kpages + off;
            s_v[tid] = p.vpages + off;
            x = 0.0f;
            for (int g = 0; g < F::kGroups; ++g) {
                float dot = 0.0f;
                for (int i = 0; i < kKvqGroup; ++i)
                    dot = fmaf(s_q[g * kKvqGroup + i],
                               static_cast<float>(code_at<D, BITS, kKvqUnitK>(kt, r, g * kKvqGroup + i)), dot);
                const uint32_t w = *reinterpret_cast<const uint32_t*>(kt + F::kParamOff + r * F::kParamBytes + g * 4);
                x = fmaf(__uint_as_float(w & 0xFFFF0000u), dot, fmaf(__uint_as_float(w << 16), s_qsum[g], x));
            }
            x *= p.scale;
        }
        float mx = x;
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (tid % 32 == 0) s_red[tid / 32] = mx;
        __syncthreads();
        float m_new = m;
        for (int i = 0; i < kSplitKeys / 32; ++i) m_new = fmaxf(m_new, s_red[i]);
        const float mb = m_new == -INFINITY ? 0.0f : m_new;
        const float alpha = m == -INFINITY ? 0.0f : expf(m - mb);
        s_p[tid] = expf(x - mb);
        __syncthreads();
        l *= alpha;
        m = m_new;
        const int n = min(kSplitKeys, len - k0);
        for (int j = 0; j < n; ++j) l += s_p[j];
#pragma unroll
        for (int e = 0; e < (D + kSplitKeys - 1) / kSplitKeys; ++e) {
            const int dim = e * kSplitKeys + tid;
            if (dim >= D) break;
            float a = acc[e] * alpha;
            for (int j = 0; j < n; ++j) {
                const int r = ((k0 + j) & ((1 << p.page_shift) - 1)) % kKvqTile;
                const uint32_t w = *reinterpret_cast<const uint32_t*>(s_v[j] + F::kParamOff + r * F::kParamBytes +
                                                                      dim / kKvqGroup * 4);
                const float c = static_cast<float>(code_at<D, BITS, kKvqUnitV>(s_v[j], r, dim));
                a = fmaf(s_p[j], fmaf(__uint_as_float(w & 0xFFFF0000u), c, __uint_as_float(w << 16)), a);
            }
            acc[e] = a;
        }
    }
    const size_t part = static_cast<size_t>(bh) * p.splits + blockIdx.y;
#pragma unroll
    for (int e = 0; e < (D + kSplitKeys - 1) / kSplitKeys; ++e)
        if (e * kSplitKeys + tid < D) p.part_o[part * D + e * kSplitKeys + tid] = l > 0.0f || l != l ? acc[e] / l : 0.0f;
    if (tid == 0) p.part_lse[part] = m == -INFINITY && l == 0.0f ? -INFINITY : m + logf(l);
}

template <int D>
__global__ void __launch_bounds__(D) fa_decode_quant_combine(const DecodeQuantParams p) {
    if (*p.status == FA_ERR_TIMEOUT) return;
    const size_t bh = blockIdx.x;
    const float* lse = p.part_lse + bh * p.splits;
    float M = -INFINITY;
    for (int s = 0; s < p.splits; ++s) M = fmaxf(M, lse[s]);
    float L = 0.0f, O = 0.0f;
    for (int s = 0; s < p.splits; ++s) {
        if (lse[s] == -INFINITY) continue;
        const float w = expf(lse[s] - M);
        L += w;
        O = fmaf(w, p.part_o[(bh * p.splits + s) * D + threadIdx.x], O);
    }
    O = L > 0.0f || L != L ? O / L : 0.0f;
    if (p.o_dtype == FA_DT_F32) static_cast<float*>(p.o)[bh * D + threadIdx.x] = O;
    else static_cast<__nv_bfloat16*>(p.o)[bh * D + threadIdx.x] = __float2bfloat16_rn(O);
    if (threadIdx.x == 0) p.lse[bh] = L > 0.0f || L != L ? M + logf(L) : -INFINITY;
}

template <int D, int BITS>
cudaError_t launch(const DecodeQuantParams& p, cudaStream_t stream) {
    fa_decode_quant_split<D, BITS><<<dim3(p.B * p.H, p.splits), kSplitKeys, 0, stream>>>(p);
    fa_decode_quant_combine<D><<<p.B * p.H, D, 0, stream>>>(p);
    return cudaGetLastError();
}

size_t workspace_bytes_of(int B, int H, int d) { return static_cast<size_t>(B) * H * kMaxSplits * (d + 1) * sizeof(float); }

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" size_t fa_decode_paged_quant_workspace_size(int B, int H, int Hkv, int max_blocks, int page_size, int d, int bits) {
    if (kvq_check_pool(B, H, Hkv, 1, page_size, max_blocks, d, bits) != FA_OK) return 0;
    return workspace_bytes_of(B, H, d);
}

extern "C" int fa_decode_paged_quant(const void* q, const void* kpages, const void* vpages, const int* block_table,
                                     const int* kv_lens, void* o, float* lse, int B, int H, int Hkv, int num_pages,
                                     int page_size, int max_blocks, int d, int bits, float scale, int o_dtype,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !kpages || !vpages || !block_table || !kv_lens || !o || !lse) return FA_ERR_INVALID_ARG;
    int rc = kvq_check_pool(B, H, Hkv, num_pages, page_size, max_blocks, d, bits);
    if (rc != FA_OK) return rc;
    if (o_dtype != FA_DT_BF16 && o_dtype != FA_DT_F32) return FA_ERR_UNSUPPORTED;
    if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
    if (!kvq_aligned(q, 16) || !kvq_aligned(kpages, 16) || !kvq_aligned(vpages, 16) || !kvq_aligned(o, 16) ||
        !kvq_aligned(lse, 4) || !kvq_aligned(block_table, 4) || !kvq_aligned(kv_lens, 4))
        return FA_ERR_INVALID_ARG;
    if (!workspace || !kvq_aligned(workspace, 256) || workspace_bytes < workspace_bytes_of(B, H, d)) return FA_ERR_WORKSPACE;
    DecodeQuantParams p{};
    if ((rc = prepare_device(&p.status)) != FA_OK) return rc;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.kpages = static_cast<const uint8_t*>(kpages);
    p.vpages = static_cast<const uint8_t*>(vpages);
    p.block_table = block_table;
    p.kv_lens = kv_lens;
    p.o = o;
    p.lse = lse;
    p.part_o = static_cast<float*>(workspace);
    p.part_lse = p.part_o + static_cast<size_t>(B) * H * kMaxSplits * d;
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.num_pages = num_pages;
    p.page_shift = kvq_page_shift(page_size);
    p.max_blocks = max_blocks;
    p.cap = max_blocks * page_size;
    p.splits = (p.cap - 1) / kSplitKeys + 1 < kMaxSplits ? (p.cap - 1) / kSplitKeys + 1 : kMaxSplits;
    p.scale = scale;
    p.o_dtype = o_dtype;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (bits == 4) e = d == 64 ? launch<64, 4>(p, s) : d == 128 ? launch<128, 4>(p, s) : launch<256, 4>(p, s);
    else e = d == 64 ? launch<64, 8>(p, s) : d == 128 ? launch<128, 8>(p, s) : launch<256, 8>(p, s);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
