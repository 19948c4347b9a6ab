// Single-query decode over the quantised paged cache: fa_decode_paged_quant
// (declared in include/fa.h, cache format in kvquant.cuh).
//
// Mathematics.  With K and V held as lo + s c per group of 32 dimensions,
//     q . k_j = sum_g [ s_jg (q_g . c_jg) + lo_jg sum(q_g) ]
//     o_d     = sum_j p_j lo_jg + sum_j (p_j s_jg) c_jd          (g = d / 32)
// so the codes go into the matrix instructions as they are and a group's lo and s
// are applied to its 16x8 partial sums (scores) or to the probabilities (output).
// The rest is the online softmax of fa_decode, in base 2.
//
// Codes as fp16.  A code c in the low bits of a half is the fp16 subnormal c 2^-24,
// exactly: an AND with 0x000f000f (0x00ff00ff) of a 32-bit word gives two of them,
// no conversion.  With 0x00f000f0 it gives 16 c 2^-24, and the 1/16 goes into the
// other operand (scores) or the result (output).  q is scaled by a power of two per
// head so that its largest value is in [2^14, 2^15): fp16 then holds every bf16 of
// it exactly down to 2^-29 of that, and to 2^-40 in absolute terms.
//
// Weights.  u = 2^6 2^(x - m), below 2^14 because the reference m follows the maximum to
// within 8 bits, is rounded to fp16 (11 bits; bf16 has 8) once for a key and head, and
// u s again.  The offsets are scaled by 2^-E and s, which a group's range has 2^BITS - 1 times, by 2^(BITS - 1 - E): that
// keeps those of every unit below 2, and u s below 2^15.  Each group of dimensions has an E of its own, so that one with large
// values takes nothing from the others.  fp16 ends at 2^-24, so a value is off by at most 2^-25 2^E for its offset and twice
// that for s: beside a token whose values in the group are 2^13 times larger it has bf16's digits left.
// One product of the rounded u with [offset of each group; ones] gives the sums of u times the offset
// and of u: the output is divided by the sum of the same rounded weights, so their errors only weigh values against
// each other.  lse takes the fp32 sum.
//
// Long sums.  The matrix instruction truncates its fp32 accumulator, half a unit in the last place
// a step on average, and sums of p s c and of p lo over many keys are large and of
// opposite sign: over 10,000 keys a warp that bias was 2 % of the output.  So half of the keys of
// every product (t + 8 and t + 12) enter as lo + C s - s (C - c), C = 2^BITS - 1: the complement
// of the code, which the AND takes with no instruction more, a negative s and the offset lo + C s.
// The two halves' terms cancel as they are summed, and the accumulators stay as small as the result.
//
// mma.sync m16n8k16 with the keys (scores) or dimensions (output) as the 16 rows and
// the heads that share the KV head as the 8 columns: NT = 1 or 2 tiles of 8.  Scores
// come out as [key][head] and go through shared memory once, where each thread picks
// up 4 keys of a head: the layout the weights need as the second product's B operand.
// A fragments are one 16-byte (K) or 8-byte (V) shared-memory load a key and plane,
// which is what the cache's order of dimensions inside a token is for.
//
// Work.  A unit is a run of KT keys of one (sequence, KV head, head set).  To begin and end
// a set costs a warp about as much as 64 keys, so a set counts as that many units more,
// ahead of its own (batches with short sequences: 5 % of the time; 48 and 96 keys are within 2 % of it).  The units
// of the whole batch, in that order, are cut into equal runs, one a CTA, and a CTA's run
// into equal runs for its warps.  There is one CTA an SM: its warps advance together.
// (Of three smaller CTAs on an SM the one that came first ran ahead, and the last one was left alone at the end: 64 x
// 32,768 keys, calls in a row at the power limit, 1.72 GHz, took 311 us against 298.)  A warp copies its units into a ring of S
// stages of its own with 16-byte asynchronous copies (a 16-token tile of K or of V is
// one run of bytes) and waits for no other warp: a set that lies in its run whole it
// writes out itself.  A set that is cut at a warp's border leaves a part (normalised output and log-sum-exp) on
// either side; the CTA merges its parts once, at its end, and writes those of a set that
// is cut at its own border for fa_decode_quant_combine.  (Dealing a CTA's units to its warps in turn takes a
// merge of the warps for every set: batches of short sequences then had CTAs that took 1.5
// times as long as the rest.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "fa_internal.h"
#include "kvquant.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kMaxSms = 160;  // CTAs of a launch, one an SM; bounds the workspace
// Warps of a CTA: 16, 12 or 8 leave a thread 128, 168 or 255 registers, of which O alone
// takes nt d / 4.  (Four more with q in shared memory were no faster, the two in turn when a call took more for other
// reasons: 281 -> 289 us for 64 x 32,768 keys at d = 128, 48 -> 51 us for 5 x 65,536 at d = 256.)  At d = 64 in 4 bits, 12 leave the shared memory for units of 64 keys.
__host__ __device__ constexpr int warps_of(int d, int bits, int nt) {
    return nt * d <= 64 && bits == 8 ? 16 : nt * d <= 128 ? 12 : 8;
}
constexpr float kRefBits = 6.0f;    // u is 2^kRefBits at the running maximum
constexpr float kGrowBits = 8.0f;   // ... and the maximum may be passed by this before a rescale
constexpr float kNoMax = -FLT_MAX;  // the maximum of no score: below any, and finite, so that no difference is NaN

struct DecodeQuantParams {
    const __nv_bfloat16* q;  // [B, H, D]
    const uint8_t* kpages;
    const uint8_t* vpages;
    const int* block_table;
    const int* kv_lens;
    void* o;
    float* lse;
    int* status;
    float* part_o;    // [2 * CTAs][8 NT][D], normalised
    float* part_lse;  // [2 * CTAs][8 NT], base 2
    int4* cut;        // [CTAs]: the set that is cut at a CTA's first unit: (first row of o, heads, first CTA of it, CTAs); 0 CTAs if none is
    int* used;        // CTAs that have units
    int B, H, Hkv, num_pages, page_shift, max_blocks, cap, sets;  // sets: head sets of a KV head
    float scale_log2;
    int o_dtype;
};

template <int D, int BITS, int NT>
struct Cfg {
    using F = KvqFormat<D, BITS>;
    static constexpr int NC = warps_of(D, BITS, NT);
    static constexpr int kBudget = 227 * 1024;
    static constexpr int kFixed = NC * 8 * NT * D * 4 + NC * (64 + 8 * 8 * NT) + 256;  // the warps' first parts, what is kept of parts, the plan
    static constexpr int kThreads = 32 * NC;
    // a warp's scores, parameters and stages of a unit of n tiles
    static constexpr int per_warp(int n, int stages) {
        return 8 * NT * (16 * n + 4) * 4 + n * F::kGroups * 64 + stages * 2 * n * F::kTileBytes;
    }
    // tiles of a unit: what is done once a unit is the smaller a part, the more it has
    static constexpr int kBlocks = D == 64 && kFixed + NC * per_warp(4, 2) <= kBudget ? 4 : kFixed + NC * per_warp(2, 2) <= kBudget ? 2 : 1;
    static constexpr int S = kFixed + NC * per_warp(kBlocks, 4) <= kBudget ? 4 : kFixed + NC * per_warp(kBlocks, 3) <= kBudget ? 3 : 2;
    static constexpr int KT = 16 * kBlocks;
    static constexpr int kVisit = (64 + KT - 1) / KT;      // units that a set counts for beside its own
    static constexpr int kHalf = kBlocks * F::kTileBytes;  // K (or V) of a stage
    static constexpr int kStageBytes = 2 * kHalf;
    static constexpr int HP = 8 * NT;  // heads of a set
    static constexpr int kScoreStride = KT + 4;
    static constexpr int kSUp = BITS - 1;  // s is held times 2^kSUp
    // V's s 2^kSUp and offsets of a unit over 2^E in fp16: s [tile][key % 4][group][key / 4], offset [tile][group][key % 4][key / 4]
    static constexpr int kSBytes = kBlocks * F::kGroups * 32;
    static constexpr int kPairs = kBlocks * F::kGroups / 4;  // pairs of keys of a group that a thread converts
    static_assert(kPairs > 0, "a unit has a pair for every thread");
    static constexpr int kParBytes = 2 * kSBytes;
    static constexpr int kZSteps = (F::kGroups + 3) / 4;  // products of lo, 4 groups each
    // shared memory; a warp's last part is kept in its ring
    static constexpr int kScoreBytes = HP * kScoreStride * 4;
    static constexpr int kRingBytes = S * kStageBytes;  // of a warp
    static constexpr int kRingOff = 0;
    static constexpr int kScoreOff = kRingOff + NC * kRingBytes;
    static constexpr int kParOff = kScoreOff + NC * kScoreBytes;
    static constexpr int kFirstOff = kParOff + NC * kParBytes;         // [warp][head][D]
    static constexpr int kMetaOff = kFirstOff + NC * HP * D * 4;       // [warp][first, last part] of Part
    static constexpr int kLseOff = kMetaOff + NC * 2 * 32;             // [warp][first, last part][head], base 2
    static constexpr int kMiscOff = kLseOff + NC * 2 * HP * 4;
    static constexpr int kBytes = kMiscOff + 32 * 4;
    static_assert(NC <= 16, "a lane for each of the parts");
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    static_assert(S >= 2, "a stage is copied while another is read");
    static_assert(HP * D * 4 <= kRingBytes, "a part fits a warp's ring");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with a zero accumulator.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// fp16 pair, lo in bits 0-15
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float lo_of(uint32_t param) { return __uint_as_float(param << 16); }
__device__ __forceinline__ float s_of(uint32_t param) { return __uint_as_float(param & 0xFFFF0000u); }

template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&r)[N], const uint8_t* p) {
    if constexpr (N == 1) {
        r[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r[0] = v.x, r[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[i];
            r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
        }
    }
}

template <int KT>
__device__ __forceinline__ int units_of(int len) {
    return static_cast<int>((static_cast<unsigned>(len) + KT - 1) / KT);
}
// What a set of that length counts for.
template <int KT, int kVisit>
__device__ __forceinline__ int weight_of(int len) {
    return len > 0 ? units_of<KT>(len) + kVisit : 0;
}
__device__ __forceinline__ int clamp_len(int len, int cap) { return min(max(len, 0), cap); }

// floor(a / b) for 0 <= a < 2^42 and 0 < b < 2^31 with a quotient below 2^31 where b < 2^10, below 2^10 otherwise: the
// quotient is at least 1 / b below the next integer, far more than its rounding to 53 bits.
__device__ __forceinline__ int div_floor(long long a, int b) { return static_cast<int>(static_cast<double>(a) / static_cast<double>(b)); }

// A place in the batch's order of units: the set that place v belongs to.  Its own units
// are the last n - kVisit of its places.
template <int KT, int kVisit>
struct Cursor {
    int b, hkv, set, begin, n, len;  // sequence, KV head, head set, first place, places, keys
    __device__ __forceinline__ void seek(const DecodeQuantParams& p, int v) {
        while (v >= begin + n) {
            begin += n;
            if (++set < p.sets) continue;
            set = 0;
            if (++hkv < p.Hkv) continue;
            hkv = 0;
            do {
                ++b;
                len = clamp_len(p.kv_lens[b], p.cap);
            } while (len == 0);
            n = weight_of<KT, kVisit>(len);
        }
    }
};

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {  // all but the last N groups of this thread have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What a warp leaves of a set that is cut at the border of its run.
struct Part {
    int kind;  // 0: none; first part: 1 ends in the run, 2 goes on after it; last part: 1
    int b, hkv, set;
    int pad[4];
};

template <int D, int BITS, int NT>
__global__ void __launch_bounds__((Cfg<D, BITS, NT>::kThreads), 1) fa_decode_quant_split(const __grid_constant__ DecodeQuantParams p) {
    using C = Cfg<D, BITS, NT>;
    using F = KvqFormat<D, BITS>;
    constexpr int KT = C::KT, kVisit = C::kVisit, S = C::S, HP = C::HP, NG = F::kGroups, PG = F::kPlaneGroups, NB = C::kBlocks;
    constexpr int NC = C::NC, kThreads = C::kThreads;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;");  // the combine kernel may be set up while this one runs
    kvq_wait_for_previous();
    Part* parts = reinterpret_cast<Part*>(smem + C::kMetaOff);
    float* part_lse = reinterpret_cast<float*>(smem + C::kLseOff);
    int* misc = reinterpret_cast<int*>(smem + C::kMiscOff);  // [0] exit, [1..4] first set, [8..] scan

    // ---- plan: the number of units and the set of this CTA's first one
    if (tid == 0) misc[0] = *static_cast<volatile const int*>(p.status) == FA_ERR_TIMEOUT;
    const int HH = p.Hkv * p.sets;
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int mine = 0, empty = 0;
    for (int b = b0; b < b1; ++b) {
        const int len = p.kv_lens[b];
        if (blockIdx.x == 0 && (len < 0 || len > p.cap)) atomicCAS(p.status, 0, FA_ERR_KV_LEN);
        mine += weight_of<KT, kVisit>(clamp_len(len, p.cap));
        empty |= len <= 0;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) misc[8 + warp] = incl;
    empty = __syncthreads_or(empty);
    if (misc[0]) {  // the combine kernel may see the status cleared by then
        if (tid == 0) {
            p.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
            if (blockIdx.x == 0) *p.used = 0;
        }
        return;
    }
    int total = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        if (i == warp) incl += total;
        total += misc[8 + i];
    }
    const int U = total * HH;
    // a CTA has a unit for each of its SM's four schedulers before another one is used
    const int n_cta = max(1, min(static_cast<int>(gridDim.x), U / 4));
    const int cta = blockIdx.x;
    if (cta == 0 && tid == 0) *p.used = n_cta;
    if (cta >= n_cta) return;
    // sequences without keys
    for (int b = empty ? cta : p.B; b < p.B; b += n_cta) {
        if (p.kv_lens[b] > 0) continue;
        for (int i = tid; i < p.H * D; i += kThreads) {
            const size_t at = static_cast<size_t>(b) * p.H * D + i;
            if (p.o_dtype == FA_DT_F32) static_cast<float*>(p.o)[at] = 0.0f;
            else static_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(0.0f);
        }
        for (int i = tid; i < p.H; i += kThreads) p.lse[static_cast<size_t>(b) * p.H + i] = -INFINITY;
    }
    if (U == 0) return;
    const int u0 = div_floor(static_cast<long long>(U) * cta, n_cta);
    const int u1 = div_floor(static_cast<long long>(U) * (cta + 1), n_cta);
    {
        // the thread whose sequences hold unit u0
        const int lo = (incl - mine) * HH, hi = incl * HH;
        if (u0 >= lo && u0 < hi) {
            int at = lo;
            for (int b = b0; b < b1; ++b) {
                const int len = clamp_len(p.kv_lens[b], p.cap), n = weight_of<KT, kVisit>(len);
                if (u0 < at + n * HH) {
                    const int hh = (u0 - at) / n;
                    misc[1] = b, misc[2] = hh, misc[3] = at + hh * n, misc[4] = len;
                    break;
                }
                at += n * HH;
            }
        }
    }
    __syncthreads();
    Cursor<KT, kVisit> cur{misc[1], misc[2] / p.sets, misc[2] % p.sets, misc[3], weight_of<KT, kVisit>(misc[4]), misc[4]};
    const int group = p.H / p.Hkv;

    // ---- copies: this warp's units [w0, w1), unit w0 + i in stage i % S
    uint8_t* ring = smem + C::kRingOff + warp * C::kRingBytes;
    const uint32_t ring_lane = smem_u32(ring) + lane * 16;
    const size_t block_bytes = static_cast<size_t>(F::kRowBytes) << p.page_shift;
    const uint32_t page_stride16 = static_cast<uint32_t>(block_bytes * p.Hkv / 16);
    const bool two = NB == 2 && p.page_shift == 4;  // the tiles of a unit lie in different pages
    Cursor<KT, kVisit> ahead = cur;
    const int w0 = u0 + static_cast<int>(static_cast<long long>(u1 - u0) * warp / NC);
    const int w1 = u0 + static_cast<int>(static_cast<long long>(u1 - u0) * (warp + 1) / NC);
    int v_load = w0, s_load = 0;
    int key = 0, left = 0, page0 = 0, page1 = 0;  // of unit v_load (four tiles: page0 of lane i is tile i's)
    int set_end = 0;                               // of ahead
    const int* table = nullptr;
    size_t head_off = 0;
    auto look_up = [&]() {
        if (v_load >= w1) return;
        if (v_load >= set_end) {
            ahead.seek(p, v_load);
            set_end = ahead.begin + ahead.n;
            table = p.block_table + static_cast<size_t>(ahead.b) * p.max_blocks;
            head_off = ahead.hkv * block_bytes + lane * 16;
            v_load = max(v_load, ahead.begin + kVisit);
            if (v_load >= w1) return;
        }
        key = (v_load - ahead.begin - kVisit) * KT;
        left = ahead.len - key;
        if constexpr (NB == 4) {
            if (lane < NB && lane * 16 < left) page0 = table[(key + lane * 16) >> p.page_shift];
        } else {
            const int* entry = table + (key >> p.page_shift);
            page0 = entry[0];
            if (two && left > 16) page1 = entry[1];
        }
    };
    auto page_in = [&](int page) {
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) return page;
        atomicCAS(p.status, 0, FA_ERR_PAGE);
        return 0;
    };
    auto issue = [&]() {
        if (v_load < w1) {
            const uint32_t dst = ring_lane + s_load * C::kStageBytes;
            if constexpr (NB == 4) {
                const int page = lane < NB && lane * 16 < left ? page_in(page0) : 0;
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) {
                    const uint32_t pg = __shfl_sync(0xffffffffu, page, kb);
                    if (kb * 16 >= left) continue;
                    const size_t off = static_cast<uint64_t>(pg) * page_stride16 * 16 + head_off +
                                       static_cast<uint32_t>(((key + kb * 16) & ((1 << p.page_shift) - 1)) / kKvqTile) * F::kTileBytes;
#pragma unroll
                    for (int i = 0; i < F::kTileBytes; i += 512) {
                        if (i + 512 <= F::kTileBytes || i + lane * 16 < F::kTileBytes) {
                            copy16(dst + kb * F::kTileBytes + i, p.kpages + off + i);
                            copy16(dst + C::kHalf + kb * F::kTileBytes + i, p.vpages + off + i);
                        }
                    }
                }
            } else {
                const uint32_t tile = (key & ((1 << p.page_shift) - 1)) / kKvqTile;
                const size_t off = static_cast<uint64_t>(static_cast<uint32_t>(page_in(page0))) * page_stride16 * 16 + head_off +
                                   tile * F::kTileBytes;
                // where the unit's bytes lie: those before kTileBytes from off, the others from off1
                size_t off1 = off;
                if (two && left > 16)
                    off1 = static_cast<uint64_t>(static_cast<uint32_t>(page_in(page1))) * page_stride16 * 16 + head_off - F::kTileBytes;
                const int bytes = left > 16 ? C::kHalf : F::kTileBytes;
#pragma unroll
                for (int i = 0; i < C::kHalf; i += 512) {
                    const size_t at = i + 512 <= F::kTileBytes ? off : i >= F::kTileBytes || i + lane * 16 >= F::kTileBytes ? off1 : off;
                    if ((i + 512 <= F::kTileBytes) || i + lane * 16 < bytes) {
                        copy16(dst + i, p.kpages + at + i);
                        copy16(dst + C::kHalf + i, p.vpages + at + i);
                    }
                }
            }
            ++v_load;
            s_load = s_load + 1 == S ? 0 : s_load + 1;
            look_up();
        }
        copy_commit();
    };
    look_up();
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue();

    if (tid == 0) {
        // for the combine kernel: the set of the CTA's first place, if earlier units of the set are another CTA's
        const int b = misc[1], hkv = misc[2] / p.sets, h_in = (misc[2] - hkv * p.sets) * HP, own = misc[3] + kVisit;
        const int c0 = div_floor((own + 1LL) * n_cta - 1, U);
        const int c1 = div_floor((own + static_cast<long long>(units_of<KT>(misc[4]))) * n_cta - 1, U);
        p.cut[cta] = make_int4(b * p.H + hkv * group + h_in, min(HP, group - h_in), c0, u0 > own ? c1 - c0 + 1 : 0);
    }

    // ---- the sets of this warp's run
    if (lane < 2) parts[2 * warp + lane].kind = 0;
    __syncwarp();
    const int r = lane >> 2, t = lane & 3;
    // V's parameters: thread (pair, group) of 32 / NG pairs at once, pair 8 kb + 2 k4 + x being keys k4 + 8 x and + 4 of tile kb
    const int pair_group = lane % NG;
    auto pair_of = [&](int i) { return i * (32 / NG) + lane / NG; };
    auto pair_key = [&](int i) { return (pair_of(i) / 2) % 4 + 8 * (pair_of(i) % 2); };
    // keys t + 8 and t + 12 enter by their complements (32 / NG and so a thread's pairs are even steps apart)
    const bool complement = (lane / NG) % 2;
    const float to_offset = complement ? static_cast<float>((1 << BITS) - 1) : 0.0f;  // offset = lo + this s
    float* sc = reinterpret_cast<float*>(smem + C::kScoreOff + warp * C::kScoreBytes);  // [head][key]: scores
    uint8_t* par = smem + C::kParOff + warp * C::kParBytes;
    auto first_part = [&](int w) { return reinterpret_cast<float*>(smem + C::kFirstOff) + w * HP * D; };
    int s = 0;
    for (int at = w0; at < w1;) {
        cur.seek(p, at);
        const int end = min(w1, cur.begin + cur.n), own = cur.begin + kVisit;
        if (end <= own) {  // no unit of the set itself is this warp's
            at = end;
            continue;
        }
        at = max(at, own);
        const int h_in = cur.set * HP;
        const int G = min(HP, group - h_in);  // heads of the set
        const size_t head0 = static_cast<size_t>(cur.b) * p.H + cur.hkv * group + h_in;

        float o[NT][D / 16][4];
        float oc[NT][4];  // heads 2 t, 2 t + 1: sums of u times the offset of group r, sums of u
        float m[NT], l[NT];
        int E = -100;                      // of group pair_group
        float down = 0.0f, s_down = 0.0f;  // 2^-E, and 2^(kSUp - E) with the sign of s in this thread's pairs
        // q as the B operand: thread (head r, t) holds dimensions 32 g + 8 t + [0, 8)
        uint32_t qb[NT][NG][4];
        uint32_t qz[NT][C::kZSteps][2];  // sums of q over a group, as the B operand of the lo product
        float A[NT][2];                  // of the score fragment's heads 2 t, 2 t + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt] = kNoMax;
            l[nt] = 0.0f;
            oc[nt][0] = oc[nt][1] = oc[nt][2] = oc[nt][3] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.0f;
            uint4 raw[NG];
            const int h = nt * 8 + r;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                raw[g] = h < G ? *reinterpret_cast<const uint4*>(p.q + (head0 + h) * D + g * kKvqGroup + t * 8)
                               : make_uint4(0, 0, 0, 0);
            }
            uint32_t big = 0;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = (&raw[g].x)[i];
                    big = max(big, max((w << 16) & 0x7FFFFFFFu, w & 0x7FFF0000u));
                }
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
            const int e = max(static_cast<int>(big >> 23) - 127, -100);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);  // 2^(14 - e)
            const float a_own = ldexpf(p.scale_log2, 10 + e);                             // undoes it and the codes' 2^-24
            float own = 0.0f, own4 = 0.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float f[8], sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = (&raw[g].x)[i];
                    f[2 * i] = bf16lo_to_f32(w);
                    f[2 * i + 1] = bf16hi_to_f32(w);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sum += f[i];
                    f[i] *= up;
                }
                uint4 b;
                if constexpr (BITS == 4)
                    b = make_uint4(pack_f16x2(f[0], f[4]), pack_f16x2(f[1] * 0.0625f, f[5] * 0.0625f), pack_f16x2(f[2], f[6]),
                                   pack_f16x2(f[3] * 0.0625f, f[7] * 0.0625f));
                else
                    b = make_uint4(pack_f16x2(f[0], f[2]), pack_f16x2(f[1], f[3]), pack_f16x2(f[4], f[6]), pack_f16x2(f[5], f[7]));
                qb[nt][g][0] = b.x, qb[nt][g][1] = b.y, qb[nt][g][2] = b.z, qb[nt][g][3] = b.w;
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                sum *= p.scale_log2;
                if (g == t) own = sum;
                if (g == t + 4) own4 = sum;
            }
            // thread t's slots of the 16 are group t (or t + 4): the sum in three bf16, which hold all of its 24 bits
#pragma unroll
            for (int zs = 0; zs < C::kZSteps; ++zs) {
                const float x = zs ? own4 : own;
                const float hi = round_bf16(x), mid = round_bf16(x - hi);
                qz[nt][zs][0] = pack_bf16x2(hi, mid);
                qz[nt][zs][1] = pack_bf16x2(x - hi - mid, 0.0f);
            }
            A[nt][0] = __shfl_sync(0xffffffffu, a_own, 8 * t);
            A[nt][1] = __shfl_sync(0xffffffffu, a_own, 8 * t + 4);
        }

        const int last = cur.begin + cur.n - 1;  // the only unit that may be short
        for (int v = at; v < end; ++v) {
            issue();
            copy_wait<S - 1>();
            __syncwarp();
            uint8_t* ks = ring + s * C::kStageBytes;
            uint8_t* vs = ks + C::kHalf;
            const int valid = v == last ? cur.len - (v - own) * KT : KT;
            if (valid < KT) {
                // Slots past the last key may hold anything, tiles not copied too: their V parameters
                // become zero (a zero probability would not cancel a NaN), their scores -inf below.
                for (int i = lane; i < KT * NG; i += 32) {
                    const int key = i / NG;
                    if (key >= valid)
                        *reinterpret_cast<uint32_t*>(vs + (key / 16) * F::kTileBytes + F::kParamOff +
                                                     (key % 16) * F::kParamBytes + (i % NG) * 4) = 0u;
                }
                __syncwarp();
            }
            // ---- scores
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                const uint8_t* kt = ks + kb * F::kTileBytes;
                uint32_t par0[NG], par1[NG];  // keys r and r + 8
                lds_words(par0, kt + F::kParamOff + r * F::kParamBytes);
                lds_words(par1, kt + F::kParamOff + (r + 8) * F::kParamBytes);
                float x1[NT][4], x2[NT][4];
                // x2 = sum over groups of lo sum(q): lo is the A operand, twice in each of thread t's registers
#pragma unroll
                for (int zs = 0; zs < C::kZSteps; ++zs) {
                    const int at_z = F::kParamOff + r * F::kParamBytes + (NG < 4 ? t % NG : zs * 4 + t) * 4;
                    const uint32_t w0 = *reinterpret_cast<const uint32_t*>(kt + at_z);
                    const uint32_t w1 = *reinterpret_cast<const uint32_t*>(kt + at_z + 8 * F::kParamBytes);
                    const uint32_t z0 = __byte_perm(w0, w0, 0x1010), z1 = __byte_perm(w1, w1, 0x1010);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (zs == 0) mma_bf16_zero(x2[nt], z0, z1, z0, z1, qz[nt][0][0], qz[nt][0][1]);
                        else mma_bf16(x2[nt], z0, z1, z0, z1, qz[nt][zs][0], qz[nt][zs][1]);
                    }
                }
#pragma unroll
                for (int pl = 0; pl < F::kPlanes; ++pl) {
                    constexpr int W = F::kPlaneBytes / 16;  // words of a thread and row
                    uint32_t c0[W], c1[W];
                    lds_words(c0, kt + (pl * 16 + r) * F::kPlaneBytes + t * (F::kPlaneBytes / 4));
                    lds_words(c1, kt + (pl * 16 + r + 8) * F::kPlaneBytes + t * (F::kPlaneBytes / 4));
#pragma unroll
                    for (int gp = 0; gp < PG; ++gp) {
                        const int g = pl * PG + gp;
                        float acc[NT][4];
#pragma unroll
                        for (int st = 0; st < 2; ++st) {
                            uint32_t a0, a1, a2, a3;
                            if constexpr (BITS == 4) {
                                const uint32_t w0 = c0[gp] >> (8 * st), w1 = c1[gp] >> (8 * st);
                                a0 = w0 & 0x000F000Fu, a1 = w1 & 0x000F000Fu;
                                a2 = w0 & 0x00F000F0u, a3 = w1 & 0x00F000F0u;
                            } else {
                                const uint32_t w0 = c0[2 * gp + st], w1 = c1[2 * gp + st];
                                a0 = w0 & 0x00FF00FFu, a1 = w1 & 0x00FF00FFu;
                                a2 = (w0 >> 8) & 0x00FF00FFu, a3 = (w1 >> 8) & 0x00FF00FFu;
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if (st == 0) mma_f16_zero(acc[nt], a0, a1, a2, a3, qb[nt][g][0], qb[nt][g][1]);
                                else mma_f16(acc[nt], a0, a1, a2, a3, qb[nt][g][2], qb[nt][g][3]);
                            }
                        }
                        const float s0 = s_of(par0[g]), s1 = s_of(par1[g]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            x1[nt][0] = g == 0 ? s0 * acc[nt][0] : fmaf(s0, acc[nt][0], x1[nt][0]);
                            x1[nt][1] = g == 0 ? s0 * acc[nt][1] : fmaf(s0, acc[nt][1], x1[nt][1]);
                            x1[nt][2] = g == 0 ? s1 * acc[nt][2] : fmaf(s1, acc[nt][2], x1[nt][2]);
                            x1[nt][3] = g == 0 ? s1 * acc[nt][3] : fmaf(s1, acc[nt][3], x1[nt][3]);
                        }
                    }
                }
                // key j of the block is kept in column 4 (j % 4) + j / 4
                const int col = kb * 16 + 4 * (r & 3) + (r >> 2);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float* row = sc + (nt * 8 + 2 * t) * C::kScoreStride + col;
                    row[0] = fmaf(x1[nt][0], A[nt][0], x2[nt][0]);
                    row[C::kScoreStride] = fmaf(x1[nt][1], A[nt][1], x2[nt][1]);
                    row[2] = fmaf(x1[nt][2], A[nt][0], x2[nt][2]);
                    row[C::kScoreStride + 2] = fmaf(x1[nt][3], A[nt][1], x2[nt][3]);
                }
            }
            // V's parameters as the products want them: a thread converts those of a group of two keys, 4 apart, for each i.
            // fp16 bit 14 tells a value of 2 or more, an infinity or NaN: then E has to be looked at below.
            uint32_t over = 0;
            auto convert = [&]() {
#pragma unroll
                for (int i = 0; i < C::kPairs; ++i) {
                    const int kb = pair_of(i) / 8, j = pair_key(i);
                    const uint8_t* from = vs + kb * F::kTileBytes + F::kParamOff + j * F::kParamBytes + pair_group * 4;
                    const uint32_t x = *reinterpret_cast<const uint32_t*>(from);
                    const uint32_t y = *reinterpret_cast<const uint32_t*>(from + 4 * F::kParamBytes);
                    const uint32_t sp = pack_f16x2(s_of(x) * s_down, s_of(y) * s_down);
                    const uint32_t zp = pack_f16x2(fmaf(s_of(x), to_offset, lo_of(x)) * down, fmaf(s_of(y), to_offset, lo_of(y)) * down);
                    over |= sp | zp;
                    *reinterpret_cast<uint32_t*>(par + ((kb * 4 + j % 4) * NG + pair_group) * 8 + j / 8 * 4) = sp;
                    *reinterpret_cast<uint32_t*>(par + C::kSBytes + (kb * NG + pair_group) * 32 + (j % 4) * 8 + j / 8 * 4) = zp;
                }
            };
            convert();
            __syncwarp();
            // ---- softmax: thread (head r, t) takes keys t, t + 4, t + 8, t + 12 of each block
            float u[NT][4 * NB], mx[NT];
            bool grow = (over & 0x40004000u) != 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) {
                    const float4 x = *reinterpret_cast<const float4*>(sc + (nt * 8 + r) * C::kScoreStride + kb * 16 + 4 * t);
                    u[nt][4 * kb] = x.x, u[nt][4 * kb + 1] = x.y, u[nt][4 * kb + 2] = x.z, u[nt][4 * kb + 3] = x.w;
                }
                if (valid < KT) {
#pragma unroll
                    for (int i = 0; i < 4 * NB; ++i)
                        if ((i >> 2) * 16 + (i & 3) * 4 + t >= valid) u[nt][i] = -INFINITY;
                }
                mx[nt] = u[nt][0];
#pragma unroll
                for (int i = 1; i < 4 * NB; ++i) mx[nt] = fmaxf(mx[nt], u[nt][i]);
                mx[nt] = fmaxf(mx[nt], __shfl_xor_sync(0xffffffffu, mx[nt], 1));
                mx[nt] = fmaxf(mx[nt], __shfl_xor_sync(0xffffffffu, mx[nt], 2));
                grow |= mx[nt] + (kRefBits - m[nt]) > kRefBits + kGrowBits;  // u's exponent, rounded as below
            }
            if (__any_sync(0xffffffffu, grow)) {
                uint32_t top = 0;  // greatest magnitude of the group's s 2^kSUp and offsets in the unit, as fp32 bits; NaN left out
#pragma unroll
                for (int i = 0; i < C::kPairs; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t w = *reinterpret_cast<const uint32_t*>(
                            vs + (pair_of(i) / 8) * F::kTileBytes + F::kParamOff + (pair_key(i) + 4 * x) * F::kParamBytes + pair_group * 4);
                        const uint32_t step = __float_as_uint(s_of(w) * static_cast<float>(1 << C::kSUp)) & 0x7FFFFFFFu;
                        const uint32_t off = __float_as_uint(fmaf(s_of(w), to_offset, lo_of(w))) & 0x7FFFFFFFu;
                        top = max(top, max(step < 0x7F800000u ? step : 0u, off < 0x7F800000u ? off : 0u));
                    }
#pragma unroll
                for (int x = NG; x < 32; x *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
                const int e_new = max(E, min(max(static_cast<int>(top >> 23) - 126, -100), 126));
                const float own_fall = ex2_approx(static_cast<float>(E - e_new));
                float fall[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) fall[g] = __shfl_sync(0xffffffffu, own_fall, g);
                const float fall_r = __shfl_sync(0xffffffffu, own_fall, r % NG);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float m_new = fmaxf(m[nt], mx[nt]);
                    const float alpha = ex2_approx(m[nt] - m_new);
                    m[nt] = m_new;
                    l[nt] *= alpha;
                    const float al0 = __shfl_sync(0xffffffffu, alpha, 8 * t), al1 = __shfl_sync(0xffffffffu, alpha, 8 * t + 4);
                    oc[nt][0] *= al0 * fall_r;
                    oc[nt][1] *= al1 * fall_r;
                    oc[nt][2] *= al0;
                    oc[nt][3] *= al1;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        o[nt][j][0] *= al0 * fall[j / 2];
                        o[nt][j][1] *= al1 * fall[j / 2];
                        o[nt][j][2] *= al0 * fall[j / 2];
                        o[nt][j][3] *= al1 * fall[j / 2];
                    }
                }
                E = e_new;
                down = __uint_as_float(static_cast<uint32_t>(127 - E) << 23);  // 2^-E
                s_down = (complement ? -down : down) * static_cast<float>(1 << C::kSUp);
                __syncwarp();  // the scores have been read: not before the parameters are written anew
                convert();
            }
            uint32_t uh[NT][NB][2];  // the weights in fp16: keys (t, t + 4) and (t + 8, t + 12)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float bias = kRefBits - m[nt];
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) {
                    float* x = u[nt] + 4 * kb;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = ex2_approx(x[i] + bias);
                        l[nt] += x[i];
                    }
                    uh[nt][kb][0] = pack_f16x2(x[0], x[1]);
                    uh[nt][kb][1] = pack_f16x2(x[2], x[3]);
                }
            }
            __syncwarp();
            // ---- output
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                const uint8_t* vt = vs + kb * F::kTileBytes;
                uint32_t wb[NT][NG][2];  // u s of keys (t, t + 4) and (t + 8, t + 12)
                {
                    uint32_t sw[2 * NG], zw[2];
                    lds_words(sw, par + (kb * 4 + t) * NG * 8);
                    lds_words(zw, par + C::kSBytes + (kb * NG + r % NG) * 32 + t * 8);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        constexpr uint32_t kOnes = 0x3C003C00u;
                        mma_f16(oc[nt], zw[0], kOnes, zw[1], kOnes, uh[nt][kb][0], uh[nt][kb][1]);
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            wb[nt][g][0] = mul_f16x2(uh[nt][kb][0], sw[2 * g]);
                            wb[nt][g][1] = mul_f16x2(uh[nt][kb][1], sw[2 * g + 1]);
                        }
                    }
                }
#pragma unroll
                for (int pl = 0; pl < F::kPlanes; ++pl) {
                    constexpr int W = F::kPlaneBytes / 32;
                    uint32_t c[4][W];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        lds_words(c[i], vt + (pl * 16 + 4 * i + t) * F::kPlaneBytes + r * (F::kPlaneBytes / 8));
#pragma unroll
                    for (int gp = 0; gp < PG; ++gp) {
                        const int g = pl * PG + gp;
                        // per 32-bit word: 2 groups of 4 nibbles, or 1 group of 4 bytes
                        const int w = BITS == 4 ? gp / 2 : gp;
#pragma unroll
                        for (int st = 0; st < 2; ++st) {
                            uint32_t a0, a1, a2, a3;
                            if constexpr (BITS == 4) {
                                const int sel = gp % 2 ? 0x7632 : 0x5410;
                                // the low row is given both nibbles of its bytes, 16 hi + lo; the high row's sum
                                // is taken off it at the end
                                const uint32_t x = __byte_perm(c[0][w], c[1][w], sel);
                                const uint32_t y = __byte_perm(c[2][w], c[3][w], sel);
                                a0 = st ? __byte_perm(x, 0, 0x4341) : x & 0x00FF00FFu, a1 = a0 & 0x00F000F0u;
                                a2 = (st ? ~(y >> 8) : ~y) & 0x00FF00FFu, a3 = a2 & 0x00F000F0u;
                            } else {
                                const int sel = st ? 0x7632 : 0x5410;
                                const uint32_t x = __byte_perm(c[0][w], c[1][w], sel);
                                const uint32_t y = __byte_perm(c[2][w], c[3][w], sel);
                                a0 = x & 0x00FF00FFu, a1 = (x >> 8) & 0x00FF00FFu;
                                a2 = ~y & 0x00FF00FFu, a3 = ~(y >> 8) & 0x00FF00FFu;
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16(o[nt][2 * g + st], a0, a1, a2, a3, wb[nt][g][0], wb[nt][g][1]);
                        }
                    }
                }
            }
            __syncwarp();  // the stage and the scores may be overwritten
            s = s + 1 == S ? 0 : s + 1;
        }

        // ---- the set's output, or this warp's part of it: thread (r, t) has dimensions 32 g + 4 r + [0, 4) of
        // heads 2 t, 2 t + 1
        const bool before = at > own, after = end < cur.begin + cur.n;
        const bool whole = !before && !after;
        float* part = before ? first_part(warp) : reinterpret_cast<float*>(ring);
        __syncwarp();  // the ring has been read
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], 1);
            l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], 2);
            // no finite score (only NaN and -inf): l says so
            const float lse = m[nt] - kRefBits + log2f(l[nt]);
            const int h = nt * 8 + r;
            if (t == 0 && h < G) {
                if (whole) p.lse[head0 + h] = lse * 0.6931471805599453f;
                else part_lse[(2 * warp + (before ? 0 : 1)) * HP + h] = lse;
            }
            constexpr float kUp = static_cast<float>(1 << (24 - C::kSUp));  // 2^24 of the codes, less that of s
            constexpr float kUp1 = BITS == 4 ? kUp / 16.0f : kUp;
            const float own_e = __uint_as_float(static_cast<uint32_t>(127 + E) << 23);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int hc = nt * 8 + 2 * t + c;
                const float inv = oc[nt][2 + c] == 0.0f ? 0.0f : 1.0f / oc[nt][2 + c];  // 0: every score is -inf
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float z = __shfl_sync(0xffffffffu, oc[nt][c], 4 * g + t), scale_e = __shfl_sync(0xffffffffu, own_e, g);
                    float* o0 = o[nt][2 * g];
                    float* o1 = o[nt][2 * g + 1];
                    if (BITS == 4) o0[c] -= o0[c + 2], o1[c] -= o1[c + 2];
                    float4 x = make_float4(fmaf(o0[c], kUp, z) * inv * scale_e, fmaf(o0[c + 2], kUp1, z) * inv * scale_e,
                                           fmaf(o1[c], kUp, z) * inv * scale_e, fmaf(o1[c + 2], kUp1, z) * inv * scale_e);
                    const int d = g * kKvqGroup + 4 * r;
                    if (hc >= G) continue;
                    if (!whole) {
                        *reinterpret_cast<float4*>(part + hc * D + d) = x;
                    } else if (p.o_dtype == FA_DT_F32) {
                        *reinterpret_cast<float4*>(static_cast<float*>(p.o) + (head0 + hc) * D + d) = x;
                    } else {
                        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + (head0 + hc) * D + d) =
                            make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
                    }
                }
            }
        }
        if (!whole && lane == 0) parts[2 * warp + (before ? 0 : 1)] = Part{before && after ? 2 : 1, cur.b, cur.hkv, cur.set, {}};
        at = end;
    }

    // ---- the CTA's parts: in the order first, last of warp 0, first, last of warp 1, ... those of a set are neighbours.
    // A set begins with a last part, or with the very first one if it begins before the CTA: NC + 1 sets at most.  The
    // warps share them out.
    __syncthreads();
    const int kind = lane < 2 * NC ? parts[lane].kind : 0;
    const uint32_t any = __ballot_sync(0xffffffffu, kind != 0), ends = __ballot_sync(0xffffffffu, kind == 1) & 0x55555555u;
    const uint32_t begins = any & (0xAAAAAAAAu | (any & (0u - any)));
    const int n_sets = __popc(begins), at_once = min(n_sets, NC);
    for (int k = n_sets ? warp % at_once : 1; k < n_sets; k += NC) {
        const int rank = warp / at_once, ranks = (NC - 1 - warp % at_once) / at_once + 1;
        uint32_t from = begins;
        for (int i = 0; i < k; ++i) from &= from - 1;
        const int i0 = __ffs(from) - 1;
        from &= from - 1;
        const uint32_t in = any & (0xFFFFFFFFu << i0) & (from ? (from & (0u - from)) - 1 : 0xFFFFFFFFu);  // its parts
        const int n_in = (31 - __clz(in)) / 2 - i0 / 2 + 1;  // the warps from i0 / 2 on: first parts, but for the first one's
        const bool before = i0 % 2 == 0, after = (in & ends) == 0, whole = !before && !after;
        const Part of = parts[i0];
        const int h_in = of.set * HP, G = min(HP, group - h_in);
        const size_t head0 = static_cast<size_t>(of.b) * p.H + of.hkv * group + h_in;
        const size_t slot = static_cast<size_t>(2 * cta + (before ? 0 : 1)) * HP;
        auto at = [&](int j) { return j ? (i0 & ~1) + 2 * j : i0; };
        for (int e = rank * 32 + lane; e < G * (D / 4); e += ranks * 32) {
            const int h = e / (D / 4), d = e % (D / 4) * 4;
            float M = -INFINITY, L = 0.0f;
            float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const float* lse = part_lse + h;
            const float* first = first_part(i0 / 2) + h * D + d;
            const float* y0 = before ? first : reinterpret_cast<const float*>(smem + C::kRingOff + i0 / 2 * C::kRingBytes) + h * D + d;
#pragma unroll 4
            for (int j = 0; j < n_in; ++j)
                if (in >> at(j) & 1) M = fmaxf(M, lse[at(j) * HP]);
#pragma unroll 4
            for (int j = 0; j < n_in; ++j) {
                const float x = lse[at(j) * HP];
                const float4 y = *reinterpret_cast<const float4*>(j ? first + j * HP * D : y0);
                if (!(in >> at(j) & 1)) continue;  // a warp without units
                const float w = x == M ? 1.0f : ex2_approx(x - M);
                L += w;
                O.x = fmaf(w, y.x, O.x), O.y = fmaf(w, y.y, O.y), O.z = fmaf(w, y.z, O.z), O.w = fmaf(w, y.w, O.w);
            }
            const float inv = 1.0f / L;
            O.x *= inv, O.y *= inv, O.z *= inv, O.w *= inv;
            if (!whole) {
                *reinterpret_cast<float4*>(p.part_o + (slot + h) * D + d) = O;
                if (d == 0) p.part_lse[slot + h] = M + log2f(L);
            } else {
                if (p.o_dtype == FA_DT_F32) *reinterpret_cast<float4*>(static_cast<float*>(p.o) + (head0 + h) * D + d) = O;
                else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + (head0 + h) * D + d) =
                    make_uint2(pack_bf16x2(O.x, O.y), pack_bf16x2(O.z, O.w));
                if (d == 0) p.lse[head0 + h] = (M + log2f(L)) * 0.6931471805599453f;
            }
        }
    }
}

// CTA i - 1 of the grid: the set that is cut at CTA i's first unit.  A set cut over P
// CTAs has P - 1 such blocks, each of which merges a share of its outputs, four at a time.  What bounds it
// is latency, so all that a thread needs is asked for at once.  Of the 3 us from the split kernel's last CTA to its own end
// (96 x 4,001 keys at d = 64, calls in a row) 1.7 pass before its first block runs; by itself and with cold caches, as a
// profiler runs it, it takes 5 to 6.
constexpr int kCombineThreads = 256;
template <int D, int BITS, int NT>
__global__ void __launch_bounds__(kCombineThreads) fa_decode_quant_combine(const __grid_constant__ DecodeQuantParams p) {
    constexpr int HP = 8 * NT, D4 = D / 4;
    __shared__ float s_w[HP][kMaxSms];  // of part c0 + i, normalised
    __shared__ float4 s_o[kCombineThreads];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int i = blockIdx.x + 1;
    // (No launch_dependents here: blocks of the next call's split kernel would be dealt out while this kernel's hold
    // places, unevenly: calls in a row, 28 -> 34 us at 96 x 4,001 keys, 57 -> 71 us at 16 x 8,192.)
    kvq_wait_for_previous();
    const int status = *static_cast<volatile const int*>(p.status);
    const int used = *p.used;
    const int4 cut = p.cut[i];
    if (status == FA_ERR_TIMEOUT || i >= used || cut.w == 0) return;
    const size_t head0 = cut.x;
    const int G = cut.y, c0 = cut.z, P = cut.w;
    // outputs 4 e0 to 4 e1 of the set's G D
    const int share = (G * D4 + P - 2) / (P - 1);
    const int e0 = (i - c0 - 1) * share, e1 = min(G * D4, e0 + share);
    if (e0 >= e1) return;
    // part c is the last one CTA c0 wrote (slot 2 c0 + 1), or the first one of a later CTA
    auto slot = [&](int c) { return static_cast<size_t>(2 * (c0 + c) + (c == 0)) * HP; };
    auto part = [&](int c, int e) { return *reinterpret_cast<const float4*>(p.part_o + slot(c) * D + 4 * e); };
    auto add = [](float4& o, float w, const float4& y) {
        o.x = fmaf(w, y.x, o.x), o.y = fmaf(w, y.y, o.y), o.z = fmaf(w, y.z, o.z), o.w = fmaf(w, y.w, o.w);
    };
    auto store = [&](int e, const float4& x) {
        const size_t at = head0 * D + 4 * e;
        if (p.o_dtype == FA_DT_F32) *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at) = x;
        else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
    };
    constexpr int kFew = 6;
    if (P <= kFew) {  // a thread four outputs
        for (int e = e0 + tid; e < e1; e += kCombineThreads) {
            const int h = e / D4;
            float x[kFew], M = -INFINITY;
            float4 y[kFew];
#pragma unroll
            for (int c = 0; c < kFew; ++c) {
                x[c] = c < P ? p.part_lse[slot(c) + h] : -INFINITY;
                y[c] = c < P ? part(c, e) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int c = 0; c < kFew; ++c) M = fmaxf(M, x[c]);
            float L = 0.0f;
            float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int c = 0; c < kFew; ++c) {
                if (c >= P) break;
                const float w = x[c] == M ? 1.0f : ex2_approx(x[c] - M);
                L += w;
                add(O, w, y[c]);
            }
            store(e, make_float4(O.x / L, O.y / L, O.z / L, O.w / L));
            if (e % D4 == 0) p.lse[head0 + h] = (M + log2f(L)) * 0.6931471805599453f;
        }
        return;
    }
    // W columns of four outputs, kCombineThreads / W threads each; a thread's first kAhead parts are asked for
    // before the weights are known
    constexpr int kAhead = 4;
    int W = kCombineThreads / 2;
    while (W > 4 && W / 2 >= share) W /= 2;
    const int col = tid % W, row = tid / W, rows = kCombineThreads / W;
    float4 ahead[kAhead];
    {
        const int e = min(e0 + col, e1 - 1);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (row + k * rows < P) ahead[k] = part(row + k * rows, e);
    }
    for (int h = e0 / D4 + warp; h <= (e1 - 1) / D4; h += kCombineThreads / 32) {
        float M = -INFINITY;
        for (int c = lane; c < P; c += 32) {
            s_w[h][c] = p.part_lse[slot(c) + h];
            M = fmaxf(M, s_w[h][c]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float L = 0.0f;
        for (int c = lane; c < P; c += 32) {
            const float w = s_w[h][c] == M ? 1.0f : ex2_approx(s_w[h][c] - M);
            s_w[h][c] = w;
            L += w;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        for (int c = lane; c < P; c += 32) s_w[h][c] /= L;
        if (lane == 0 && h * D4 >= e0) p.lse[head0 + h] = (M + log2f(L)) * 0.6931471805599453f;
    }
    __syncthreads();
    for (int eb = e0; eb < e1; eb += W) {
        const int e = min(eb + col, e1 - 1), h = e / D4;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        int c = row;
        if (eb == e0) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k, c += rows)
                if (c < P) add(x, s_w[h][c], ahead[k]);
        }
#pragma unroll 4
        for (; c < P; c += rows) add(x, s_w[h][c], part(c, e));
        s_o[tid] = x;
        __syncthreads();
        for (int k = rows / 2; k > 0; k /= 2) {
            if (row < k) add(s_o[tid], 1.0f, s_o[tid + k * W]);
            __syncthreads();
        }
        if (row == 0 && eb + col < e1) store(e, s_o[col]);
        __syncthreads();
    }
}

// What a batch of full sequences counts for.  The kernels count in int32, a little past the last unit too.
template <int D, int BITS, int NT>
long long units_at_capacity(int B, int Hkv, int sets, int cap) {
    using C = Cfg<D, BITS, NT>;
    return static_cast<long long>(B) * Hkv * sets * ((cap - 1) / C::KT + 1 + C::kVisit);
}
constexpr long long kMaxUnits = 0x7FFFFF00LL;

template <int D, int BITS, int NT>
cudaError_t launch(const DecodeQuantParams& p, int dev, int num_sms, cudaStream_t stream) {
    using C = Cfg<D, BITS, NT>;
    cudaError_t e;
    static std::atomic<uint64_t> ready{0};  // a bit a device whose kernel has its shared memory set
    const uint64_t bit = 1ull << (dev & 63);
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) & bit)) {
        if ((e = cudaFuncSetAttribute(fa_decode_quant_split<D, BITS, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      C::kBytes)) != cudaSuccess)
            return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const long long units = units_at_capacity<D, BITS, NT>(p.B, p.Hkv, p.sets, p.cap);
    const int grid = static_cast<int>(std::max(1LL, std::min<long long>(std::min(kMaxSms, num_sms), units / 4)));
    e = kvq_launch(fa_decode_quant_split<D, BITS, NT>, grid, C::kThreads, C::kBytes, stream, p);
    if (e != cudaSuccess || grid == 1) return e;
    return kvq_launch(fa_decode_quant_combine<D, BITS, NT>, grid - 1, kCombineThreads, 0, stream, p);
}

// 8-head tiles of a set: two (O takes NT D / 4 registers a thread) only where a second
// one has heads, and D leaves room for it.
int tiles_of(int group, int d) { return d <= 128 && group > 8 ? 2 : 1; }
int sets_of(int group, int nt) { return (group - 1) / (8 * nt) + 1; }

// f(D, BITS, NT) of the kernels for a head dimension, code width and number of tiles.
template <typename F>
auto by_kernel(int d, int bits, int nt, F&& f) {
    auto with_bits = [&](auto D, auto NT) {
        return bits == 4 ? f(D, std::integral_constant<int, 4>(), NT) : f(D, std::integral_constant<int, 8>(), NT);
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    if (d == 256) return with_bits(std::integral_constant<int, 256>(), One());
    if (d == 128) return nt == 1 ? with_bits(std::integral_constant<int, 128>(), One()) : with_bits(std::integral_constant<int, 128>(), Two());
    return nt == 1 ? with_bits(std::integral_constant<int, 64>(), One()) : with_bits(std::integral_constant<int, 64>(), Two());
}

// kvq_check_pool, and whether the batch at its capacity can be counted.
int check_sizes(int B, int H, int Hkv, int num_pages, int page_size, int max_blocks, int d, int bits) {
    const int rc = kvq_check_pool(B, H, Hkv, num_pages, page_size, max_blocks, d, bits);
    if (rc != FA_OK) return rc;
    const int nt = tiles_of(H / Hkv, d);
    const long long units = by_kernel(d, bits, nt, [&](auto D, auto BITS, auto NT) {
        return units_at_capacity<D(), BITS(), NT()>(B, Hkv, sets_of(H / Hkv, nt), max_blocks * page_size);
    });
    return units > kMaxUnits ? FA_ERR_INVALID_ARG : FA_OK;
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
struct Workspace {
    size_t lse, cut, used, total;  // offsets of the arrays after part_o
};
Workspace workspace_of(int H, int Hkv, int d) {
    const int nt = tiles_of(H / Hkv, d);
    const size_t ctas = kMaxSms, heads = 8 * nt;
    Workspace w{};
    w.lse = up256(2 * ctas * heads * d * sizeof(float));
    w.cut = w.lse + up256(2 * ctas * heads * sizeof(float));
    w.used = w.cut + up256(ctas * sizeof(int4));
    w.total = w.used + 256;
    return w;
}

}  // namespace

}  // namespace fa

using namespace fa;

extern "C" size_t fa_decode_paged_quant_workspace_size(int B, int H, int Hkv, int max_blocks, int page_size, int d, int bits) {
    if (check_sizes(B, H, Hkv, 1, page_size, max_blocks, d, bits) != FA_OK) return 0;
    return workspace_of(H, Hkv, d).total;
}

extern "C" int fa_decode_paged_quant(const void* q, const void* kpages, const void* vpages, const int* block_table,
                                     const int* kv_lens, void* o, float* lse, int B, int H, int Hkv, int num_pages,
                                     int page_size, int max_blocks, int d, int bits, float scale, int o_dtype,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !kpages || !vpages || !block_table || !kv_lens || !o || !lse) return FA_ERR_INVALID_ARG;
    int rc = check_sizes(B, H, Hkv, num_pages, page_size, max_blocks, d, bits);
    if (rc != FA_OK) return rc;
    if (o_dtype != FA_DT_BF16 && o_dtype != FA_DT_F32) return FA_ERR_UNSUPPORTED;
    if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
    if (!kvq_aligned(q, 16) || !kvq_aligned(kpages, 16) || !kvq_aligned(vpages, 16) || !kvq_aligned(o, 16) ||
        !kvq_aligned(lse, 4) || !kvq_aligned(block_table, 4) || !kvq_aligned(kv_lens, 4))
        return FA_ERR_INVALID_ARG;
    const int nt = tiles_of(H / Hkv, d);
    DecodeQuantParams p{};
    p.sets = sets_of(H / Hkv, nt);
    p.cap = max_blocks * page_size;
    const Workspace at = workspace_of(H, Hkv, d);
    if (!workspace || !kvq_aligned(workspace, 256) || workspace_bytes < at.total) return FA_ERR_WORKSPACE;
    if ((rc = prepare_device(&p.status)) != FA_OK) return rc;
    int dev = 0, num_sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return FA_ERR_CUDA;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.kpages = static_cast<const uint8_t*>(kpages);
    p.vpages = static_cast<const uint8_t*>(vpages);
    p.block_table = block_table;
    p.kv_lens = kv_lens;
    p.o = o;
    p.lse = lse;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_lse = reinterpret_cast<float*>(ws + at.lse);
    p.cut = reinterpret_cast<int4*>(ws + at.cut);
    p.used = reinterpret_cast<int*>(ws + at.used);
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.num_pages = num_pages;
    p.page_shift = kvq_page_shift(page_size);
    p.max_blocks = max_blocks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.o_dtype = o_dtype;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = by_kernel(d, bits, nt, [&](auto D, auto BITS, auto NT) { return launch<D(), BITS(), NT()>(p, dev, num_sms, s); });
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
