// decode_kernel.cuh -- attention of few query rows per K/V head over many keys:
// of the newest tokens of each sequence over a paged cache held in 16 or in 4
// bits (decode.cu), the same beside a prefix that the batch shares, whose part
// comes from the tensor-core forward (decode_shared.cu), and of few rows over an
// encoder's states, dense tensors by strides (decode_cross.cu).
//
// One row of K and V is read per key, for all query rows that share the K/V
// head (G = H/Hkv heads times Nq tokens): the call is bound by the cache's
// bytes, so the kernel is built to keep them streaming.
//
// Products.  Both run transposed on mma.sync m16n8k16 (M = 16 keys or dims, N =
// 8 query rows): S^T = K Q^T and O^T += V^T P^T.  Eight query rows fill N, so a
// group of up to 8 wastes no tensor work and O needs only D/4 registers; NT =
// 1, 2 or 4 tiles of 8 rows share one pass over the keys, and more rows than 32
// take further passes.  (tcgen05 needs M >= 64 rows of S, 8 to 16 times what a
// decode step has, and its operands in shared memory; the rate needed here,
// two m16n8k16 per 16 keys and 16 dims, keeps the tensor pipe 23 % busy.)
//
// Keys.  A unit of work is 8 warps' stages of keys of one target: a sequence, a
// K/V head and a block of query rows.  The units of the whole call are numbered
// in that order, and CTA c of a fixed grid takes an equal share [c U / G, (c+1)
// U / G), whatever the lengths: only device memory knows them, each CTA forms
// the prefix sums itself.  A target counts a few units more than it has, for
// being started and joined; without that, shares of short sequences ran twice
// as long as others (decode of 64 sequences of up to 8192 keys, 32 heads on 8:
// 183 -> 166 us in 16 bits, 114 -> 90 us in 4).  Within a unit a warp takes one
// stage, with a ring of stages of its own in shared memory filled by cp.async
// (zero-filled behind the last key), so that warps never wait for one another
// until their share of a sequence is done; then the CTA joins its eight warps'
// (max, sum, O).  A sequence that lies in one CTA is written out there; of the
// others each CTA writes its part to the workspace, and the CTA whose part
// comes last joins them all, in the order of the keys (so that the result does
// not depend on which one that is).  At most two parts per CTA (its first and
// its last sequence) are ever cut.
//
// Softmax.  A lane keeps the reference max of its query rows; O and the sums
// are rescaled only when a score passes it by more than 8 (log2), by a vote
// that costs one instruction otherwise.  Sums stay in the lanes until the end.
//
// Measured (GB300, D = 128, the 64 sequences above, 1.11 GB of 16-bit rows):
// 165 to 168 us, 6.7 TB/s, the rate of a plain copy.  In 4 bits the same call
// (347 MB) takes 86 us, 4.0 TB/s, and 3 sequences of 120001 keys (461 MB) 96 us,
// 4.8 TB/s.  No unit is full there (integer pipe 58 %, issue slots 63 %): four
// warps a scheduler, each one chain of dependent steps of 23 warp instructions a
// key, wait for fixed latencies and for the math pipe; and the ragged batch
// pays for 512 targets' starts and joins, with no copy in flight meanwhile.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "internal.h"

namespace fattn {
namespace {

// Each translation unit that includes this file instantiates one mode and has
// the error word of its own kernels.
__device__ uint32_t g_decode_error_word;

//   kBehindPrefix: writes its rows as a part, beside those of the prefix.
//   kWithPrefix: every sequence reads the prefix for itself.  Its keys come first,
//   up to a whole unit of virtual keys (those behind its last are masked), then the
//   sequence's own.
enum Mode { kCache, kBehindPrefix, kWithPrefix, kCross };
template <Mode MODE>
using DecodeArgsOf = std::conditional_t<
    MODE == kCross, CrossDecodeArgs,
    std::conditional_t<MODE == kBehindPrefix, SharedDecodeArgs,
                       std::conditional_t<MODE == kWithPrefix, PrefixDecodeArgs, DecodeArgs>>>;

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kPart = 16;                 // keys that lie in one page and take one pass of the products
constexpr int kMaxCtas = 320;             // parts in the workspace: two per CTA
constexpr int kAloneUnits = 2;            // longest target that one warp takes alone
constexpr int kMaxParts = 64;             // CTAs a sequence is cut between: one CTA joins the parts
constexpr float kLow = -3.0e38f;          // the running max of a row that has seen no key
constexpr float kRescaleThreshold = 8.0f; // log2 units: P <= 2^8 while the max is stale
// Weights that enter the products as fp16 numbers are taken 2^kUp times: up to
// 2^15 while the max is stale, and with all their bits down to 2^-21 of the
// largest, not 2^-14: the small weights of a long sequence add up.
template <bool BF16, bool KV4>
constexpr float kUp = BF16 && !KV4 ? 0.f : 7.f;

// ---- instructions ----------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes, of which the first `bytes` come from src and the rest are zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c = a b: no accumulator to set to zero first.
template <bool BF16>
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// The same in fp16, with +-65504 for what is past it (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_finite(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

// ---- a warp's stage in shared memory ----------------------------------------
// 16 bits: K rows, then V rows, 16-byte chunk c of key r at chunk c ^ (r mod 8)
// (ldmatrix reads 8 rows of one chunk without bank conflicts).
// 4 bits: K codes (D/2 a key), K scales (D/8 a key), then V rows of codes and
// scales, 16 bytes wider than the codes: lanes that take keys 2t of 8 bytes (4
// at D = 64) then meet 32 different banks.
template <int D, bool KV4, int NT, int WARPS>
struct Stage {
    // Keys of a warp's stage.  4 bits: two parts of 16, whose loop, votes and
    // addresses are paid once, where registers allow; 16 bits: one, as a stage
    // is 4 times as large.
    static constexpr int kKeys = KV4 && NT == 1 ? 32 : 16;
    static constexpr int kParts = kKeys / kPart;
    static constexpr int kUnit = WARPS * kKeys;  // keys of a unit
    static constexpr int kCode = D / 2, kMeta = D / kKv4Group * 4;
    static constexpr int kVRow = KV4 ? kCode + 16 : 2 * D;
    static constexpr int kKMetaOff = kKeys * kCode;
    static constexpr int kVOff = KV4 ? kKMetaOff + kKeys * kMeta : kKeys * 2 * D;
    static constexpr int kBytes = kVOff + kKeys * kVRow;
};

template <int D, bool KV4, int NT, int WARPS>
struct Config {
    static constexpr int kWarps = WARPS, kThreads = 32 * WARPS;
    static constexpr int kStages = KV4 ? (NT == 1 ? 2 : 4) : (WARPS == 6 ? 2 : 3);
    static constexpr int kCtasPerSm = WARPS == 8 && (NT == 4 || (D == 128 && (NT == 2 || !KV4))) ? 1 : 2;
    static constexpr int kRows = 8 * NT;
    // What starting and joining a target costs, in units of keys.
    static constexpr int kTargetCost = KV4 ? 2 : 32 / WARPS;
    static constexpr int kRing = kWarps * kStages * Stage<D, KV4, NT, WARPS>::kBytes;
    // The warps' O is joined in the same memory.
    static constexpr int kPitch = D + 4;  // of a row of O there
    static constexpr int kJoin = kWarps * kRows * kPitch * 4;
    static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
    static_assert(kSmem * kCtasPerSm <= 224 * 1024, "shared memory budget");
    static_assert(8 * kPitch * 4 <= kStages * Stage<D, KV4, NT, WARPS>::kBytes, "a warp's O, eight rows at a time, in its ring");
};

// A part of a cut sequence: per row the max (log2 units), the sum, then O.
template <int D>
__device__ __forceinline__ float* part_of(void* ws, int slot, int rows) {
    return static_cast<float*>(ws) + 4 * kMaxCtas + static_cast<int64_t>(slot) * rows * (D + 2);
}
// Per CTA, the arrivals of the parts of the cut sequence that starts in it: a
// mark in the upper 48 bits, the count in the lower 16.  A call leaves its words
// marked with count 0, so that in a workspace that was used before an arrival
// is one atomicAdd; a word without the mark is whatever the caller's memory
// held: the first arrival to replace it counts 1, and what others added to it
// meanwhile is not counted (they find no mark either and come again).
constexpr unsigned long long kMark = 0x5bd1e995a7c3ull << 16;
__device__ __forceinline__ unsigned long long* arrivals_of(void* ws) { return static_cast<unsigned long long*>(ws); }
__device__ __forceinline__ int arrive(unsigned long long* word) {  // the arrivals so far, this one among them
    unsigned long long seen = atomicAdd(word, 1ull);
    while ((seen >> 16) != (kMark >> 16)) {
        const unsigned long long now = atomicCAS(word, seen, kMark | 1ull);
        if (now == seen) return 1;
        seen = (now >> 16) == (kMark >> 16) ? atomicAdd(word, 1ull) : now;
    }
    return static_cast<int>(seen & 0xffffull) + 1;
}

// The share of CTA c.
__device__ __forceinline__ int64_t share_begin(int64_t units, int c, int ctas) { return units * c / ctas; }
// The CTA whose share holds a unit.
__device__ __forceinline__ int cta_of(int64_t unit, int64_t units, int ctas) {
    int c = static_cast<int>(unit * ctas / units);
    while (share_begin(units, c + 1, ctas) <= unit) ++c;
    return c;
}

// The prefix's keys, and the virtual keys that they take.
struct Prefix {
    int keys, end;
};
__device__ __forceinline__ Prefix prefix_of(const PrefixDecodeArgs& a, bool report) {
    int len = *a.prefix_len;
    if (len < 0 || len > a.prefix_max) {
        if (report) atomicOr(&g_decode_error_word, 1u << kDevErrInvalidArg);
        len = len < 0 ? 0 : a.prefix_max;
    }
    constexpr int kUnit = 128;  // of the largest units of 16-bit keys
    return {len, (len + kUnit - 1) / kUnit * kUnit};
}

template <typename ARGS>
__device__ __forceinline__ int visible_len(const ARGS& a, int b, bool report) {
    if constexpr (std::is_same_v<ARGS, CrossDecodeArgs>) {
        if (a.seq_lens == nullptr) return a.Nk;
        const int len = a.seq_lens[b];
        if (len < 0 || len > a.Nk) {
            if (report) atomicOr(&g_decode_error_word, 1u << kDevErrInvalidArg);
            return len < 0 ? 0 : a.Nk;
        }
        return len;
    }
    const int64_t most = a.table_width * a.page_size;
    const int len = a.seq_lens[b];
    if (len < 0 || len > most) {
        if (report) atomicOr(&g_decode_error_word, 1u << kDevErrInvalidArg);
        return len < 0 ? 0 : static_cast<int>(most);
    }
    return len;
}
template <int UNIT>
__device__ __forceinline__ int units_of(int len) {
    return max(1, static_cast<int>((static_cast<uint32_t>(len) + UNIT - 1) / UNIT));
}

// Writes 4 dims of one query row (of K/V head kvh) from its unnormalised sum: 4
// bits, of half the values (Warp::accumulate), whose mean may lie a little past
// fp16's range, as the values do.
// Behind a prefix: as the last part of the row, which is joined to the prefix's.
template <int D, bool BF16, bool KV4, typename ARGS>
__device__ __forceinline__ void store_out(const ARGS& a, int b, int kvh, int row, int d, const float (&acc)[4],
                                          float mx, float sum) {
    const int share = a.H / a.Hkv;
    if (row >= share * a.Nq) return;
    const int h = kvh * share + row / a.Nq, i = row % a.Nq;
    if constexpr (std::is_same_v<ARGS, SharedDecodeArgs>) {
        const int hq = row / a.Nq;
        const int u = (b / a.box_b * a.n_h + hq / a.box_h) * a.n_i + i / a.box_i;
        const int trow = ((b % a.box_b) * a.box_h + hq % a.box_h) * a.box_i + i % a.box_i;
        const int64_t at = ((static_cast<int64_t>(kvh) * a.tiles + u) * kTcBM + trow) * a.part_pitch + a.part_pitch - 1;
        const bool empty = sum == 0.f;  // (as below)
        __stcg(reinterpret_cast<float4*>(a.part_o + at * D + d),
               empty ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(acc[0], acc[1], acc[2], acc[3]));
        if (d == 0) __stcg(a.part_ml + at, empty ? make_float2(-INFINITY, 0.f) : make_float2(mx, sum));
        return;
    }
    const bool none = sum == 0.f;  // the row sees no key (its sum of values: 0, or 0 times what is not finite)
    const float inv = (KV4 ? 2.f : 1.f) / sum;
    auto pack = [](float x, float y) { return KV4 && !BF16 ? pack_finite(x, y) : pack16<BF16>(x, y); };
    uint16_t* o = static_cast<uint16_t*>(a.o) + b * a.o_bs + h * a.o_hs + i * a.o_ns + d;
    *reinterpret_cast<uint2*>(o) =
        none ? make_uint2(0u, 0u) : make_uint2(pack(acc[0] * inv, acc[1] * inv), pack(acc[2] * inv, acc[3] * inv));
    if (d == 0 && a.lse != nullptr)
        a.lse[(static_cast<int64_t>(b) * a.H + h) * a.Nq + i] =
            none ? -INFINITY : (mx + kUp<BF16, KV4> + log2f(sum * exp2f(-kUp<BF16, KV4>))) * kLn2;
}

// ---- one warp's keys ----------------------------------------------------------
template <int D, bool BF16, bool KV4, int NT, int WARPS>
struct Warp {
    using S = Stage<D, KV4, NT, WARPS>;
    static constexpr int kQ = D / 16;   // k-steps of S^T, m-tiles of O^T
    uint32_t q[NT][kQ][2];              // B fragments of Q^T
    uint32_t qsum[NT];                  // 4 bits: (high, low) part of the sum of q over group t
    float f[NT][2];                     // log2-score of one unit of S, rows 2t and 2t+1 (> 0)
    float m[NT][2], l[NT][2];           // the max (less kUp) that a row's weights are relative to; their sum
    float o[NT][kQ][4];

    // Query rows of K/V head kvh, row block rb.  Lane (g, t) = (lane/4, lane%4).
    __device__ __forceinline__ void load_q(const DecodeArgs& a, int b, int kvh, int rb) {
        const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
        const int rows = (a.H / a.Hkv) * a.Nq;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = rb * 8 * NT + n * 8 + g;
            const uint16_t* src = nullptr;
            if (r < rows)
                src = static_cast<const uint16_t*>(a.q) + b * a.q_bs +
                      static_cast<int64_t>(kvh * (a.H / a.Hkv) + r / a.Nq) * a.q_hs + (r % a.Nq) * a.q_ns;
            if constexpr (!KV4) {
#pragma unroll
                for (int kk = 0; kk < kQ; ++kk) {
                    q[n][kk][0] = src ? *reinterpret_cast<const uint32_t*>(src + 16 * kk + 2 * t) : 0u;
                    q[n][kk][1] = src ? *reinterpret_cast<const uint32_t*>(src + 16 * kk + 8 + 2 * t) : 0u;
                }
                f[n][0] = f[n][1] = fmaxf(a.scale_log2, kLeastFactor);
                qsum[n] = 0u;
            } else {
                // q as fp16 whatever its type: scaled by a power of two so that
                // the row's largest element lies in [2^9, 2^10), which keeps
                // every element within 2^-20 of it exact, and sums of 32 below
                // fp16's largest.
                float x[D / 32][8];
                float big = 0.f;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
                    if (src) raw = *reinterpret_cast<const uint4*>(src + 32 * i + 8 * t);
                    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        if (BF16) {
                            x[i][2 * p] = __uint_as_float(w[p] << 16);
                            x[i][2 * p + 1] = __uint_as_float(w[p] & 0xffff0000u);
                        } else {
                            const float2 v = __half22float2(as_half2(w[p]));
                            x[i][2 * p] = v.x;
                            x[i][2 * p + 1] = v.y;
                        }
                        big = fmaxf(big, fmaxf(fabsf(x[i][2 * p]), fabsf(x[i][2 * p + 1])));
                    }
                }
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                const int e = max(static_cast<int>((__float_as_uint(big) >> 23) & 255u) - 127, -100);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + 9 - e) << 23);
                float mine = 0.f;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    float sum = 0.f;
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        // pairs 1 and 3 meet codes that sit 4 bits higher
                        const float k = (p & 1) ? up * 0.0625f : up;
                        q[n][2 * i + p / 2][p & 1] = pack16<false>(x[i][2 * p] * k, x[i][2 * p + 1] * k);
                        sum += x[i][2 * p] * up + x[i][2 * p + 1] * up;
                    }
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    if (i == t) mine = sum;
                }
                const float hi = __half2float(__float2half_rn(mine));
                qsum[n] = pack16<false>(hi, mine - hi);
                const float down = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - 9 + e) << 23);
                f[n][0] = fmaxf(__shfl_sync(0xffffffffu, down, 8 * t), kLeastFactor);
                f[n][1] = fmaxf(__shfl_sync(0xffffffffu, down, 8 * t + 4), kLeastFactor);
            }
            m[n][0] = m[n][1] = kLow;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int j = 0; j < kQ; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
        }
    }

    // What rows_of() adds a page's row to: this lane's first 16 bytes (and, 4
    // bits, its key's scales), for K/V head kvh.
    struct Source {
        const uint8_t* k;
        const uint8_t* v;
        const uint8_t* scales;
    };
    template <typename ARGS>
    static __device__ __forceinline__ Source source(const ARGS& a, int kvh) {
        const int lane = threadIdx.x % 32;
        if constexpr (std::is_same_v<ARGS, CrossDecodeArgs>) {
            constexpr int kChunks = D / 8;
            const int64_t row = lane / kChunks;
            return {static_cast<const uint8_t*>(a.k_pages) + 2 * (kvh * a.k_hs + row * a.k_ns) + 16 * (lane % kChunks),
                    static_cast<const uint8_t*>(a.v_pages) + 2 * (kvh * a.v_hs + row * a.v_ns) + 16 * (lane % kChunks),
                    nullptr};
        }
        const int64_t head = static_cast<int64_t>(kvh) * a.page_size;  // rows before this head in a page
        Source f;
        if constexpr (!KV4) {
            f.k = static_cast<const uint8_t*>(a.k_pages) + head * 2 * D + 16 * lane;
            f.v = static_cast<const uint8_t*>(a.v_pages) + head * 2 * D + 16 * lane;
            f.scales = nullptr;
        } else {
            f.k = static_cast<const uint8_t*>(a.k_pages) + head * S::kCode + 16 * lane;
            f.v = static_cast<const uint8_t*>(a.v_pages) + head * S::kCode + 16 * lane;
            f.scales = static_cast<const uint8_t*>(lane < 16 ? a.k_scales : a.v_scales) + (head + lane % 16) * S::kMeta;
        }
        return f;
    }

    // The rows from place `off` of `page` on.
    static __device__ __forceinline__ Source rows_of(const DecodeArgs& a, const Source& f, int page, int off) {
        Source r;
        if constexpr (!KV4) {
            const int64_t at = 2 * (page * a.page_stride + static_cast<int64_t>(off) * D);
            r.k = f.k + at;
            r.v = f.v + at;
            r.scales = nullptr;
        } else {
            const uint64_t row = static_cast<uint64_t>(static_cast<uint32_t>(page)) *
                                     static_cast<uint32_t>(a.Hkv * a.page_size) + static_cast<uint32_t>(off);
            r.k = f.k + row * S::kCode;
            r.v = f.v + row * S::kCode;
            r.scales = f.scales + row * S::kMeta;
        }
        return r;
    }

    // Starts the copies of part `part` of a stage: 16 keys, `skip` rows further
    // (`valid` of them are keys of the sequence; the rest become zero).  FULL:
    // all of them are.
    template <bool FULL>
    static __device__ __forceinline__ void copy(const Source& f, uint32_t stage, int part, int skip, int valid) {
        const int lane = threadIdx.x % 32;
        if constexpr (!KV4) {
            constexpr int kChunks = D / 8, kRowsAtOnce = 32 / kChunks;
            const int c = lane % kChunks;
#pragma unroll
            for (int i = 0; i < kPart / kRowsAtOnce; ++i) {
                const int r = i * kRowsAtOnce + lane / kChunks;
                const uint32_t dst = stage + r * 2 * D + ((c ^ (r & 7)) << 4);
                const int bytes = FULL || r < valid ? 16 : 0;
                cp_async16(dst, f.k + skip * 2 * D + i * 512, bytes);
                cp_async16(dst + S::kVOff, f.v + skip * 2 * D + i * 512, bytes);
            }
        } else {
            constexpr int kChunks = D / 32;  // 16-byte chunks of a row of codes
#pragma unroll
            for (int i = 0; i < kPart * kChunks / 32; ++i) {
                const int r = i * (32 / kChunks) + lane / kChunks, c = lane % kChunks;
                const int bytes = FULL || r < valid ? 16 : 0;
                cp_async16(stage + part * kPart * S::kCode + i * 512 + lane * 16, f.k + skip * S::kCode + i * 512, bytes);
                cp_async16(stage + S::kVOff + (part * kPart + r) * S::kVRow + c * 16, f.v + skip * S::kCode + i * 512,
                           bytes);
            }
            const int r = lane % 16;
            const uint32_t dst = lane < 16 ? stage + S::kKMetaOff + (part * kPart + r) * S::kMeta
                                           : stage + S::kVOff + (part * kPart + r) * S::kVRow + S::kCode;
            cp_async_small<S::kMeta>(dst, f.scales + skip * S::kMeta, FULL || r < valid ? S::kMeta : 0);
        }
    }

    // The same for keys `key` .. key + 15 of batch entry b's own tensors, a row by
    // its stride.
    template <bool FULL>
    static __device__ __forceinline__ void copy_rows(const CrossDecodeArgs& a, const Source& f, uint32_t stage, int b,
                                                     int key, int valid) {
        constexpr int kChunks = D / 8, kRowsAtOnce = 32 / kChunks;
        const int lane = threadIdx.x % 32, c = lane % kChunks;
        const uint8_t* k = f.k + 2 * (b * a.k_bs + key * a.k_ns);
        const uint8_t* v = f.v + 2 * (b * a.v_bs + key * a.v_ns);
        const int64_t k_step = 2 * kRowsAtOnce * a.k_ns, v_step = 2 * kRowsAtOnce * a.v_ns;
#pragma unroll
        for (int i = 0; i < kPart / kRowsAtOnce; ++i) {
            const int r = i * kRowsAtOnce + lane / kChunks;
            const uint32_t dst = stage + r * 2 * D + ((c ^ (r & 7)) << 4);
            const bool on = FULL || r < valid;  // (no key: zeros, and an address inside the tensor)
            cp_async16(dst, on ? k + i * k_step : static_cast<const uint8_t*>(a.k_pages), on ? 16 : 0);
            cp_async16(dst + S::kVOff, on ? v + i * v_step : static_cast<const uint8_t*>(a.v_pages), on ? 16 : 0);
        }
    }

    // S^T of 16 keys of the stage, in units of f: s[n][0..1] key g, s[n][2..3] key
    // g + 8, rows 2t and 2t+1.
    __device__ __forceinline__ void scores(uint32_t stage, int part, float (&s)[NT][4]) const {
        const int lane = threadIdx.x % 32;
        if constexpr (!KV4) {
            const int r = (lane & 7) + (lane & 8);
#pragma unroll
            for (int kk = 0; kk < kQ; ++kk) {
                uint32_t k[4];
                ldmatrix4(k, stage + r * 2 * D + (((2 * kk + lane / 16) ^ (r & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (kk == 0)
                        mma16816_first<BF16>(s[n], k, q[n][kk][0], q[n][kk][1]);
                    else
                        mma16816<BF16>(s[n], k, q[n][kk][0], q[n][kk][1]);
            }
        } else {
            // sum_d q_d (c_d scale + zero) = sum over groups of scale (sum q c) +
            // zero (sum q): the codes enter as fp16 subnormals, c 2^-24 (or 16
            // times that), which the tensor cores multiply exactly, the scales
            // in fp32, and the zeros as one more product, (zero, zero) with
            // (high, low) part of the sum of q, group t in lane t.
            // The sum of products keeps a fixed number of bits below the largest
            // exponent, and a subnormal's is taken as 2^-14 whatever its leading
            // zeros.  With the 11 bits of an fp16 q that cost scores 1e-6 of
            // their size (bf16's 8 bits: 1e-7, fp32's own), so there the codes
            // sit two bits higher, for one more shift a word.
            constexpr int kShift = BF16 ? 0 : 2;
            constexpr uint32_t kLoCode = 0x000f000fu << kShift, kHiCode = 0x00f000f0u << kShift;
            const int g = lane / 4, t = lane % 4;
            uint32_t w[2][D / 32], meta[2][D / 32];
            uint32_t z[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int key = part * kPart + g + 8 * u;
                const uint32_t mt = stage + S::kKMetaOff + key * S::kMeta;
                lds_words(w[u], stage + key * S::kCode + t * (D / 8));
                lds_words(meta[u], mt);
                // (D = 64 has two groups: lanes 2 and 3 repeat them, and meet a
                // sum of q that is zero.)
                z[u] = lds_word(mt + 4 * (t % (D / 32)));
                z[u] = __byte_perm(z[u], 0u, 0x3232);
            }
            float zs[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816_first<false>(zs[n], z, qsum[n], 0u);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint32_t a0[4], a1[4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t lo = w[u][i] << kShift, hi = w[u][i] >> (8 - kShift);
                    a0[u] = lo & kLoCode;
                    a0[u + 2] = lo & kHiCode;
                    a1[u] = hi & kLoCode;
                    a1[u + 2] = hi & kHiCode;
                }
                const float sc0 = __low2float(as_half2(meta[0][i])), sc1 = __low2float(as_half2(meta[1][i]));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float c[4];
                    mma16816_first<false>(c, a0, q[n][2 * i][0], q[n][2 * i][1]);
                    mma16816<false>(c, a1, q[n][2 * i + 1][0], q[n][2 * i + 1][1]);
                    s[n][0] = i == 0 ? c[0] * sc0 : fmaf(c[0], sc0, s[n][0]);
                    s[n][1] = i == 0 ? c[1] * sc0 : fmaf(c[1], sc0, s[n][1]);
                    s[n][2] = i == 0 ? c[2] * sc1 : fmaf(c[2], sc1, s[n][2]);
                    s[n][3] = i == 0 ? c[3] * sc1 : fmaf(c[3], sc1, s[n][3]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[n][x] = fmaf(s[n][x], 16777216.f / (1 << kShift), zs[n][x]);
        }
    }

    template <int N>
    static __device__ __forceinline__ void lds_words(uint32_t (&w)[N], uint32_t addr) {
        if constexpr (N == 4)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(addr)
                         : "memory");
        else
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    }
    static __device__ __forceinline__ uint32_t lds_word(uint32_t addr) {
        uint32_t w;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(addr) : "memory");
        return w;
    }

    // O^T += V^T P^T; p[n][u]: B fragments (keys 2t, 2t+1 and 8 further, row g).
    __device__ __forceinline__ void accumulate(uint32_t stage, int part, const uint32_t (&p)[NT][2]) {
        const int lane = threadIdx.x % 32;
        const uint32_t base = stage + S::kVOff + part * kPart * S::kVRow;
        if constexpr (!KV4) {
            const int r = (lane & 7) + ((lane & 16) >> 1);
#pragma unroll
            for (int j = 0; j < kQ; ++j) {
                uint32_t v[4];
                ldmatrix4_trans(v, base + r * 2 * D + (((2 * j + ((lane >> 3) & 1)) ^ (r & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816<BF16>(o[n][j], v, p[n][0], p[n][1]);
            }
        } else {
            // ldmatrix, transposed, on the codes' 16-bit pieces (4 codes each): lane
            // (g, t) gets piece g of a 16-byte chunk for keys 2t and 2t+1 side by
            // side, 4 pairs of codes.  Each pair is made fp16 by setting exponent
            // bits (512 + c/2, or 32 + c/2 where the code sits 4 bits higher), taking
            // that off again (exact), and one fused (c/2) scale + zero/2: half the
            // value, as 15 scale + zero of a group whose largest element is 65504
            // can lie past fp16's range (its scale is rounded to nearest).  Which
            // dims the lane's rows of O^T are is dim_of().
            const int g = lane / 4, t = lane % 4;
            uint32_t x[2][D / 32];                   // [keys 0-7, 8-15][chunk]
            const uint32_t row = base + ((lane & 7) + (lane & 8)) * S::kVRow + (lane >> 4) * 16;
#pragma unroll
            for (int c = 0; c < D / 32; c += 2) {
                uint32_t y[4];
                ldmatrix4_trans(y, row + c * 16);
                x[0][c] = y[0];
                x[1][c] = y[1];
                x[0][c + 1] = y[2];
                x[1][c + 1] = y[3];
            }
            uint32_t sc[2][2], ze[2][2];             // of the two groups that this lane's dims lie in
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t at = base + (2 * t + 8 * u) * S::kVRow + S::kCode + (D == 128 ? 8 * (g & 1) : 0);
                uint32_t m0[2], m1[2];
                lds_words(m0, at);
                lds_words(m1, at + S::kVRow);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    sc[u][i] = __byte_perm(m0[i], m1[i], 0x5410);
                    ze[u][i] = as_u32(__hmul2(as_half2(__byte_perm(m0[i], m1[i], 0x7632)), as_half2(0x38003800u)));
                }
            }
#pragma unroll
            for (int j = 0; j < kQ; ++j) {
                uint32_t v[4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t piece = (j & 1) ? x[u][j / 2] >> 8 : x[u][j / 2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t magic = h ? 0x50005000u : 0x60006000u;
                        const uint32_t up = (piece & (h ? 0x00f000f0u : 0x000f000fu)) | magic;
                        const __half2 c = __hsub2(as_half2(up), as_half2(magic));
                        v[2 * u + h] = as_u32(__hfma2(c, as_half2(sc[u][j & 1]), as_half2(ze[u][j & 1])));
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816<false>(o[n][j], v, p[n][0], p[n][1]);
            }
        }
    }

    // The dim that row g + 8 h of m-tile j of O^T is.
    static __device__ __forceinline__ int dim_of(int j, int h, int g) {
        if (!KV4) return 16 * j + 8 * h + g;
        const int q = 2 * (j & 1) + h, c = j / 2;  // nibble of the piece, 16-byte chunk
        return D == 128 ? 16 * (4 * (g & 1) + q) + 8 * ((g >> 1) & 1) + 2 * c + (g >> 2)
                        : 16 * q + 8 * (g & 1) + 4 * c + (g >> 1);
    }

    // The stage's keys: `key` is the first one's index, ends[n][x] the number of
    // keys that row 2t + x sees (tested when `masked`); bit p of `skip`: part p
    // holds nothing.
    // (`cap`: keys from there on are hidden from every row.)
    __device__ __forceinline__ void keys(uint32_t stage, int key, bool masked, uint32_t skip, const int (&ends)[NT][2],
                                         int cap = 0x7fffffff) {
        const int lane = threadIdx.x % 32, g = lane / 4;
        constexpr int P = S::kParts;
        float s[P][NT][4];
#pragma unroll
        for (int u = 0; u < P; ++u) scores(stage, u, s[u]);
        if (masked) {
#pragma unroll
            for (int u = 0; u < P; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (key + u * kPart + g + (x & 2) * 4 >= min(ends[n][x & 1], cap) || ((skip >> u) & 1u))
                            s[u][n][x] = -INFINITY;
        }
        float mx[NT][2];
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                mx[n][x] = fmaxf(s[0][n][x], s[0][n][x + 2]);
#pragma unroll
                for (int u = 1; u < P; ++u) mx[n][x] = fmaxf(mx[n][x], fmaxf(s[u][n][x], s[u][n][x + 2]));
                mx[n][x] *= f[n][x];
                grow |= mx[n][x] > m[n][x] + (kRescaleThreshold + kUp<BF16, KV4>);
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float top = mx[n][x];
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    const float mn = fmaxf(m[n][x], top - kUp<BF16, KV4>);
                    const float alpha = ex2(m[n][x] - mn);
                    m[n][x] = mn;
                    l[n][x] *= alpha;
#pragma unroll
                    for (int j = 0; j < kQ; ++j) {
                        o[n][j][x] *= alpha;
                        o[n][j][x + 2] *= alpha;
                    }
                }
        }
#pragma unroll
        for (int u = 0; u < P; ++u) {
            uint32_t p[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float p0 = ex2(fmaf(s[u][n][0], f[n][0], -m[n][0])), p1 = ex2(fmaf(s[u][n][1], f[n][1], -m[n][1]));
                const float p2 = ex2(fmaf(s[u][n][2], f[n][0], -m[n][0])), p3 = ex2(fmaf(s[u][n][3], f[n][1], -m[n][1]));
                l[n][0] += p0 + p2;
                l[n][1] += p1 + p3;
                // P rounded to the operands' type (fp16 beside 4-bit values), key by
                // row to row by key.
                p[n][0] = movmatrix_trans(pack16<BF16 && !KV4>(p0, p1));
                p[n][1] = movmatrix_trans(pack16<BF16 && !KV4>(p2, p3));
            }
            accumulate(stage, u, p);
        }
    }
};

template <int D, bool BF16, bool KV4, int NT, bool ALONE, Mode MODE, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, Config<D, KV4, NT, WARPS>::kCtasPerSm)
    decode_kernel(const __grid_constant__ DecodeArgsOf<MODE> a) {
    static_assert(MODE == kCache || !KV4, "16-bit keys");
    using C = Config<D, KV4, NT, WARPS>;
    using S = Stage<D, KV4, NT, WARPS>;
    constexpr int kWarps = WARPS, kThreads = 32 * WARPS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_scan[kWarps];
    __shared__ int s_most[kWarps];
    __shared__ int64_t s_begin;   // units before the first sequence of this share
    __shared__ int s_first;       // that sequence
    __shared__ int s_last;        // this CTA's part was the last to come
    __shared__ float s_m[kWarps][C::kRows], s_l[kWarps][C::kRows];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int rows = (a.H / a.Hkv) * a.Nq;
    const int row_blocks = (rows + C::kRows - 1) / C::kRows;
    const int per_key = a.Hkv * row_blocks;  // targets of one sequence

    grid_dependency();
    Prefix prefix = {0, 0};
    if constexpr (MODE == kWithPrefix) prefix = prefix_of(a, blockIdx.x == 0 && tid == 0);
    auto visible_len = [&](const auto& args, int seq, bool report) {
        return fattn::visible_len(args, seq, report) + (MODE == kWithPrefix ? prefix.end : 0);
    };
    // All units of the call, and this CTA's share of them.  A target (K/V head
    // and row block of a sequence) counts C::kTargetCost units more than it has, so
    // that shares of many short sequences take no longer than others.
    int64_t units = 0;
    int most = 0, first_cost = 0, upto = 0;
    const bool few = a.B <= 32;  // every warp does it for itself
    if (few) {
        first_cost = lane < a.B ? units_of<S::kUnit>(visible_len(a, lane, blockIdx.x == 0 && warp == 0)) + C::kTargetCost : 0;
        upto = first_cost;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        units = __shfl_sync(0xffffffffu, upto, 31);
        most = __reduce_max_sync(0xffffffffu, first_cost);
    } else {
        int64_t mine = 0;
        for (int b = tid; b < a.B; b += kThreads) {
            const int n = units_of<S::kUnit>(visible_len(a, b, blockIdx.x == 0)) + C::kTargetCost;
            if (b == tid) first_cost = n;
            mine += n;
            most = max(most, n);
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) mine += __shfl_xor_sync(0xffffffffu, mine, d);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) {
            s_scan[warp] = mine;
            s_most[warp] = most;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            units += s_scan[w];
            most = max(most, s_most[w]);
        }
    }
    units *= per_key;
    // CTAs that get a share: no more than units, so that the CTAs a sequence is
    // cut between are neighbours, and so few that the longest sequence is cut
    // into about kMaxParts.
    const int cta = blockIdx.x;
    const int ctas = static_cast<int>(min(min(static_cast<int64_t>(gridDim.x), units),
                                          max(units * kMaxParts / most, static_cast<int64_t>(1))));
    if (cta >= ctas) return;
    const int64_t begin = share_begin(units, cta, ctas), end = share_begin(units, cta + 1, ctas);
    // The sequence of unit `begin`: prefix sums, kThreads sequences at a time.
    int b;
    int64_t seq_at;  // first unit of sequence b
    if (few) {
        const uint32_t past = __ballot_sync(0xffffffffu, lane < a.B && static_cast<int64_t>(upto) * per_key > begin);
        b = __ffs(past) - 1;
        seq_at = static_cast<int64_t>(__shfl_sync(0xffffffffu, upto - first_cost, b)) * per_key;
    } else {
        int64_t before = 0;
        for (int b0 = 0;; b0 += kThreads) {
            __syncthreads();  // s_scan is read by all before it is written again
            const int b = b0 + tid;
            int64_t own = 0;
            if (b < a.B)
                own = static_cast<int64_t>(b0 == 0 ? first_cost
                                                   : units_of<S::kUnit>(visible_len(a, b, false)) + C::kTargetCost) * per_key;
            int64_t x = own;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            if (lane == 31) s_scan[warp] = x;
            __syncthreads();
            int64_t left = before, all = before;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) left += s_scan[w];
                all += s_scan[w];
            }
            x += left;
            if (own > 0 && begin >= x - own && begin < x) {
                s_first = b;
                s_begin = x - own;
            }
            before = all;
            if (before > begin || b0 + kThreads >= a.B) break;
        }
        __syncthreads();
        b = s_first;
        seq_at = s_begin;
    }

    uint32_t ring = smem_addr(smem) + warp * C::kStages * S::kBytes;
    const int page_shift = (a.page_size & (a.page_size - 1)) == 0 ? __ffs(a.page_size) - 1 : -1;
    const bool one_page = a.page_size % S::kKeys == 0;  // a stage never crosses pages
    Warp<D, BF16, KV4, NT, WARPS> w;
    int64_t at = begin;
    int next_b = b;
    while (at < end) {
        const int len = visible_len(a, b, false);
        const int tiles = units_of<S::kUnit>(len);
        const int cost = tiles + C::kTargetCost;
        const int64_t in_seq = at - seq_at;
        const int target = static_cast<int>(in_seq / cost);  // K/V head and row block
        const int place = static_cast<int>(in_seq - static_cast<int64_t>(target) * cost);
        const int taken = static_cast<int>(min(static_cast<int64_t>(cost - place), end - at));
        // The extra units come first; tiles [t0, t1) are this CTA's.
        const int t0 = max(place - C::kTargetCost, 0), t1 = place + taken - C::kTargetCost;
        const int64_t target_at = at - place;  // the target's first unit

        // Short targets that lie whole in this share: up to kWarps of them at
        // once, a warp each, and nothing to join.  Worth it where there are
        // more of them than units in the longest (a warp alone takes kWarps
        // turns a unit, about what starting and joining a target costs).
        int batch = 0, my_b = b, my_target = target, my_len = len;
        if (ALONE && place <= C::kTargetCost && tiles <= kAloneUnits) {
            int w_b = b, w_target = target, w_len = len, longest = 0;
            int64_t w_at = target_at, w_seq = seq_at;
            while (batch < kWarps) {
                const int n = units_of<S::kUnit>(w_len);
                if (n > kAloneUnits || w_at + n + C::kTargetCost > end) break;
                if (batch == warp) {
                    my_b = w_b;
                    my_target = w_target;
                    my_len = w_len;
                }
                longest = max(longest, n);
                ++batch;
                w_at += n + C::kTargetCost;
                if (++w_target == per_key) {
                    w_target = 0;
                    ++w_b;
                    w_seq = w_at;
                    if (w_at >= end) break;
                    w_len = visible_len(a, w_b, false);
                }
                if (w_at >= end) break;
            }
            if (batch > longest && batch > 1) {
                at = w_at;
                seq_at = w_seq;
                next_b = w_b;
            } else {
                batch = 0;
                my_b = b;
                my_target = target;
                my_len = len;
            }
        }
        const bool alone = ALONE && batch > 0;
        if (!alone) {
            at += taken;
            if (at - seq_at == static_cast<int64_t>(cost) * per_key) {
                seq_at = at;
                ++next_b;
            }
            if (t1 <= t0) {
                b = next_b;
                continue;
            }
        }
        const int kvh = my_target / row_blocks, rb = my_target - kvh * row_blocks;
        const int32_t* table = MODE == kCross ? nullptr : a.block_table + my_b * a.table_width;

        int ends[NT][2];
        const int min_end = MODE == kCross ? my_len : my_len - a.Nq + 1;
        const int first_end = MODE == kWithPrefix ? max(min_end, prefix.end) : min_end;  // every row sees the prefix
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = rb * C::kRows + n * 8 + (lane % 4) * 2 + x;
                ends[n][x] = MODE != kCross && r < rows ? min_end + r % a.Nq : my_len;  // rows that are none: anything finite
                if constexpr (MODE == kWithPrefix) ends[n][x] = max(ends[n][x], prefix.end);
            }

        // This warp's keys: kKeys at first + stride i.
        const int stride = alone ? S::kKeys : S::kUnit;
        const int first = alone ? 0 : t0 * S::kUnit + warp * S::kKeys;
        const int last = alone ? (warp < batch ? my_len : 0) : min(len, t1 * S::kUnit);
        const int turns = first < last ? (last - first + stride - 1) / stride : 0;
        const typename Warp<D, BF16, KV4, NT, WARPS>::Source source = w.template source<DecodeArgsOf<MODE>>(a, kvh);
        struct Pages {
            int p[S::kParts];
        };
        auto pages_at = [&](int i) -> Pages {  // the pages of turn i's parts (any where there are none)
            const int key = first + i * stride;
            Pages r;
            if constexpr (MODE == kCross) {
                r.p[0] = 0;
                return r;
            }
            if constexpr (MODE == kWithPrefix) {
                const bool own = key >= prefix.end;
                const int k = own ? key - prefix.end : key;
                r.p[0] = i < turns && key < (own ? last : prefix.keys)
                             ? (own ? table : a.prefix_table)[page_shift >= 0 ? k >> page_shift : k / a.page_size] : 0;
                return r;
            }
#pragma unroll
            for (int u = 0; u < S::kParts; ++u) {
                const int k = key + u * kPart;
                if (u > 0 && one_page)
                    r.p[u] = r.p[0];
                else
                    r.p[u] = i < turns && k < last ? table[page_shift >= 0 ? k >> page_shift : k / a.page_size] : 0;
            }
            return r;
        };
        uint32_t skip = 0u;  // bit s * kParts + u: part u of stage s holds nothing
        auto start = [&](int i, const Pages& pages) {
            if (i < turns) {
                const int stage = i % C::kStages;
                const uint32_t at = ring + stage * S::kBytes;
                const int key = first + i * stride;
                if constexpr (MODE == kCross) {
                    if (last - key >= S::kKeys)
                        w.template copy_rows<true>(a, source, at, my_b, key, kPart);
                    else
                        w.template copy_rows<false>(a, source, at, my_b, key, last - key);
                    cp_async_commit();
                    return;
                }
                if constexpr (MODE == kWithPrefix) {
                    const bool own = key >= prefix.end;
                    const int k = own ? key - prefix.end : key, left = (own ? last : prefix.keys) - key;
                    const int off = page_shift >= 0 ? k & (a.page_size - 1) : k % a.page_size;
                    int page = pages.p[0], valid = left;
                    skip &= ~(1u << stage);
                    if (left > 0 && static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages)) {
                        if (lane == 0) atomicOr(&g_decode_error_word, 1u << kDevErrInvalidArg);
                        if (own) skip |= 1u << stage;  // (a page of the prefix: zeros that are seen)
                        page = valid = 0;
                    }
                    if (valid >= S::kKeys)
                        w.template copy<true>(w.rows_of(a, source, page, off), at, 0, 0, kPart);
                    else
                        w.template copy<false>(w.rows_of(a, source, left > 0 ? page : 0, off), at, 0, 0, valid);
                    cp_async_commit();
                    return;
                }
                const uint32_t bits = ((1u << S::kParts) - 1u) << (stage * S::kParts);
                bool fine = last - key >= S::kKeys;
#pragma unroll
                for (int u = 0; u < S::kParts; ++u)
                    fine = fine && static_cast<uint32_t>(pages.p[u]) < static_cast<uint32_t>(a.num_pages);
                skip &= ~bits;
                if (fine && one_page) {
                    const int off = page_shift >= 0 ? key & (a.page_size - 1) : key % a.page_size;
                    const auto rows = w.rows_of(a, source, pages.p[0], off);
#pragma unroll
                    for (int u = 0; u < S::kParts; ++u) w.template copy<true>(rows, at, u, u * kPart, kPart);
                } else if (fine) {
                    int off = page_shift >= 0 ? key & (a.page_size - 1) : key % a.page_size;
#pragma unroll
                    for (int u = 0; u < S::kParts; ++u) {
                        w.template copy<true>(w.rows_of(a, source, pages.p[u], off), at, u, 0, kPart);
                        off += kPart;
                        if (off == a.page_size) off = 0;
                    }
                } else {
#pragma unroll 1
                    for (int u = 0; u < S::kParts; ++u) {
                        const int k = key + u * kPart;
                        int page = u == 0 ? pages.p[0] : pages.p[S::kParts - 1];
                        if (k >= last) {
                            page = 0;  // no key: zeros, from anywhere inside the pool
                        } else if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages)) {
                            if (lane == 0) atomicOr(&g_decode_error_word, 1u << kDevErrInvalidArg);
                            skip |= 1u << (stage * S::kParts + u);
                            page = 0;
                        }
                        const int valid = ((skip >> (stage * S::kParts + u)) & 1u) ? 0 : last - k;
                        w.template copy<false>(w.rows_of(a, source, page, k % a.page_size), at, u, 0, valid);
                    }
                }
            }
            cp_async_commit();
        };
        Pages pages;
        {
            Pages early[C::kStages];  // all on their way before the first is used
#pragma unroll
            for (int i = 0; i < C::kStages; ++i) early[i] = pages_at(i);
#pragma unroll
            for (int i = 0; i < C::kStages - 1; ++i) start(i, early[i]);
            pages = early[C::kStages - 1];
        }
        w.load_q(a, my_b, kvh, rb);
        for (int i = 0; i < turns; ++i) {
            start(i + C::kStages - 1, pages);
            pages = pages_at(i + C::kStages);  // needed one turn later
            cp_async_wait<C::kStages - 1>();
            __syncwarp();
            const int stage = i % C::kStages;
            const int key = first + i * stride;
            const uint32_t none = (skip >> (stage * S::kParts)) & ((1u << S::kParts) - 1u);
            if constexpr (MODE == kWithPrefix) {
                const int cap = key < prefix.end ? prefix.keys : 0x7fffffff;
                w.keys(ring + stage * S::kBytes, key, key + S::kKeys > min(first_end, cap) || none != 0u, none, ends, cap);
            } else {
                w.keys(ring + stage * S::kBytes, key, key + S::kKeys > first_end || none != 0u, none, ends);
            }
            __syncwarp();  // every lane is done with the stage before it is filled again
        }
        cp_async_wait<0>();

        if (alone) {
            // The warp's own O, eight rows at a time through its ring.
            if (warp < batch) {
                float* mine = reinterpret_cast<float*>(smem + warp * C::kStages * S::kBytes);
                const int g = lane / 4, t = lane % 4;
                __syncwarp();
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float l[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        l[x] = w.l[n][x];
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) l[x] += __shfl_xor_sync(0xffffffffu, l[x], d);
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            mine[(2 * t + x) * C::kPitch + w.dim_of(j, 0, g)] = w.o[n][j][x];
                            mine[(2 * t + x) * C::kPitch + w.dim_of(j, 1, g)] = w.o[n][j][x + 2];
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float sum = __shfl_sync(0xffffffffu, l[r & 1], r / 2);
                        const float mx = __shfl_sync(0xffffffffu, w.m[n][r & 1], r / 2);
                        if (4 * lane < D) {
                            const float4 v = *reinterpret_cast<const float4*>(mine + r * C::kPitch + 4 * lane);
                            const float acc[4] = {v.x, v.y, v.z, v.w};
                            store_out<D, BF16, KV4>(a, my_b, kvh, rb * C::kRows + n * 8 + r, 4 * lane, acc, mx, sum);
                        }
                    }
                    __syncwarp();
                }
            }
            b = next_b;
            continue;
        }

        // Join the eight warps: their O by rows, in the ring's memory.
        __syncthreads();
        float* so = reinterpret_cast<float*>(smem) + warp * C::kRows * C::kPitch;
        {
            const int g = lane / 4, t = lane % 4;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float l = w.l[n][x];
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
                    const int r = n * 8 + 2 * t + x;
                    if (g == 0) {
                        s_m[warp][r] = w.m[n][x];
                        s_l[warp][r] = l;
                    }
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        so[r * C::kPitch + w.dim_of(j, 0, g)] = w.o[n][j][x];
                        so[r * C::kPitch + w.dim_of(j, 1, g)] = w.o[n][j][x + 2];
                    }
                }
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == tiles;
        const int slot = 2 * cta + (target_at <= begin ? 0 : 1);
        float* part = part_of<D>(a.workspace, slot, C::kRows);
        for (int x = tid; x < C::kRows * D / 4; x += kThreads) {
            const int r = x / (D / 4), d = 4 * (x % (D / 4));
            float mx = s_m[0][r];
#pragma unroll
            for (int y = 1; y < kWarps; ++y) mx = fmaxf(mx, s_m[y][r]);
            float sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int y = 0; y < kWarps; ++y) {
                const float wt = ex2(s_m[y][r] - mx);
                sum = fmaf(wt, s_l[y][r], sum);
                const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) +
                                                                  (y * C::kRows + r) * C::kPitch + d);
                acc[0] = fmaf(wt, v.x, acc[0]);
                acc[1] = fmaf(wt, v.y, acc[1]);
                acc[2] = fmaf(wt, v.z, acc[2]);
                acc[3] = fmaf(wt, v.w, acc[3]);
            }
            if (whole) {
                store_out<D, BF16, KV4>(a, b, kvh, rb * C::kRows + r, d, acc, mx, sum);
            } else {
                __stcg(reinterpret_cast<float4*>(part + 2 * C::kRows + r * D + d), make_float4(acc[0], acc[1], acc[2], acc[3]));
                if (d == 0) {
                    __stcg(part + r, mx);
                    __stcg(part + C::kRows + r, sum);
                }
            }
        }
        if (!whole) {
            const int c0 = t0 == 0 ? cta : cta_of(target_at + C::kTargetCost, units, ctas);
            const int parts = cta_of(target_at + cost - 1, units, ctas) - c0 + 1;
            const int slot0 = 2 * c0 + (target_at <= share_begin(units, c0, ctas) ? 0 : 1);
            unsigned long long* word = arrivals_of(a.workspace) + c0;
            __threadfence();  // this thread's part, before the arrival
            __syncthreads();
            if (tid == 0) {
                s_last = arrive(word) == parts;
                if (s_last) atomicExch(word, kMark);
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                for (int x = tid; x < C::kRows * D / 4; x += kThreads) {
                    const int r = x / (D / 4), d = 4 * (x % (D / 4));
                    float mx = kLow, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
                    constexpr int kAtOnce = 8;
                    for (int y0 = 0; y0 < parts; y0 += kAtOnce) {
                        float pm[kAtOnce], pl[kAtOnce];
                        float4 v[kAtOnce];
#pragma unroll
                        for (int y = 0; y < kAtOnce; ++y) {
                            const int z = min(y0 + y, parts - 1);
                            const float* p = part_of<D>(a.workspace, z == 0 ? slot0 : 2 * (c0 + z), C::kRows);
                            pm[y] = __ldcg(p + r);
                            pl[y] = __ldcg(p + C::kRows + r);
                            v[y] = __ldcg(reinterpret_cast<const float4*>(p + 2 * C::kRows + r * D + d));
                        }
#pragma unroll
                        for (int y = 0; y < kAtOnce; ++y) {
                            if (y0 + y >= parts) continue;
                            const float mn = fmaxf(mx, pm[y]);
                            const float wo = ex2(mx - mn), wt = ex2(pm[y] - mn);
                            mx = mn;
                            sum = fmaf(wt, pl[y], sum * wo);
                            acc[0] = fmaf(wt, v[y].x, acc[0] * wo);
                            acc[1] = fmaf(wt, v[y].y, acc[1] * wo);
                            acc[2] = fmaf(wt, v[y].z, acc[2] * wo);
                            acc[3] = fmaf(wt, v[y].w, acc[3] * wo);
                        }
                    }
                    store_out<D, BF16, KV4>(a, b, kvh, rb * C::kRows + r, d, acc, mx, sum);
                }
            }
        }
        __syncthreads();  // the joined memory becomes the ring again
        b = next_b;
    }
}

// Warps of a CTA.  Eight, but six where two such CTAs fit an SM and targets are short
// (the own keys behind a prefix, one tile of rows, D = 128: decode_shared.cu; over an
// encoder's states six took 49.3 us where eight take 48.2).
template <int D, int NT, Mode MODE>
constexpr int kWarpsOf = MODE == kBehindPrefix && D == 128 && NT == 1 ? 6 : 8;

template <int D, bool BF16, bool KV4, int NT, bool ALONE, Mode MODE>
cudaError_t launch_one(const DecodeArgsOf<MODE>& a, int sms, cudaStream_t s) {
    using C = Config<D, KV4, NT, kWarpsOf<D, NT, MODE>>;
    auto* fn = decode_kernel<D, BF16, KV4, NT, ALONE, MODE, C::kWarps>;
    static std::atomic<bool> done[kMaxDevices] = {};
    cudaError_t e = opt_in_smem_once(fn, C::kSmem, done);
    if (e != cudaSuccess) return e;
    const int grid = sms * C::kCtasPerSm < kMaxCtas ? sms * C::kCtasPerSm : kMaxCtas;
    return launch_overlapped(fn, grid, C::kThreads, C::kSmem, s, a);
}

// Tiles of 8 query rows that share one pass over the keys.
int row_tiles(int64_t rows) { return rows <= 8 ? 1 : (rows <= 16 ? 2 : 4); }

// Whether short targets may be taken by one warp each: only where a CTA's share
// holds two targets or more on average.  (200 sequences of up to 300 tokens, 32
// heads on 8, D = 128, 4 bits: 42.6 -> 33.6 us.  The kernel that can loses 2 % on long sequences
// and 4 to 10 % on the smallest calls to the registers that this takes, and
// with 32 query rows 6 to 10 % everywhere, so that form does not exist.)
template <int D, bool BF16, bool KV4, int NT, Mode MODE>
cudaError_t launch_targets(const DecodeArgsOf<MODE>& a, int sms, cudaStream_t s) {
    if constexpr (NT <= 2) {
        const int64_t targets = static_cast<int64_t>(a.B) * a.Hkv;
        if (targets >= 2 * sms * Config<D, KV4, NT, kWarpsOf<D, NT, MODE>>::kCtasPerSm) return launch_one<D, BF16, KV4, NT, true, MODE>(a, sms, s);
    }
    return launch_one<D, BF16, KV4, NT, false, MODE>(a, sms, s);
}

template <int D, bool BF16, bool KV4, Mode MODE>
cudaError_t launch_rows(const DecodeArgsOf<MODE>& a, int sms, cudaStream_t s) {
    switch (row_tiles(static_cast<int64_t>(a.H / a.Hkv) * a.Nq)) {
        case 1: return launch_targets<D, BF16, KV4, 1, MODE>(a, sms, s);
        case 2: return launch_targets<D, BF16, KV4, 2, MODE>(a, sms, s);
        default: return launch_targets<D, BF16, KV4, 4, MODE>(a, sms, s);
    }
}

// 16-bit keys.
template <Mode MODE>
cudaError_t launch16(const DecodeArgsOf<MODE>& a, int D, bool bf16, int sms, cudaStream_t s) {
    if (D == 128)
        return bf16 ? launch_rows<128, true, false, MODE>(a, sms, s) : launch_rows<128, false, false, MODE>(a, sms, s);
    return bf16 ? launch_rows<64, true, false, MODE>(a, sms, s) : launch_rows<64, false, false, MODE>(a, sms, s);
}

cudaError_t read_and_clear(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_decode_error_word, sizeof(v));
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_decode_error_word, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace
}  // namespace fattn
