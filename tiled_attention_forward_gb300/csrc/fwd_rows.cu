// fwd_rows.cu -- the tensor-core forward (fwd_tc_kernel.cuh) on query rows over
// keys of a length of their own, and the kernel that joins the parts of rows whose
// keys were cut.
//
//     O_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp2(scale log2e q_i.k_j - m_i)
//
// over all keys j of a source: an encoder's states of one batch entry, or a prefix
// that the whole batch shares, in pages.  Every row of a K/V head sees the same
// keys, so rows are stacked into tiles of 128 whatever heads, tokens and (for a
// prefix) batch entries they belong to: a box of a 4-D tensor map, which one copy
// brings.  130 tokens of 4 heads are 5 tiles and not 8.
//
// Few tiles leave most SMs idle: their keys are then cut into parts (choose_cut), of
// which each gives the row's maximum m, sum l and sum of values in fp32, and
//     O = sum_p 2^(m_p - m) O_p / sum_p 2^(m_p - m) l_p
// is formed by a kernel of its own, in a fixed order.  Parts are written through
// shared memory as whole lines, and read from L2.
//
// Measured (GB300).  Enough tiles: 2 entries of 32 heads on 8, 8192 tokens over 4096
// keys, D = 128, bf16, 674 us in a burst of 20 calls = 1630 TFLOP/s (0.85 of the measured
// peak; tensor pipe 72 %), 719 to 724 among other calls or for seconds, at the power limit
// (0.80), the dense forward's chain; 64 heads of 4096 tokens and keys 346 to 355 us where
// the dense forward takes 336, the difference being what a task costs: with every role
// decoding tasks for itself 370.  Few: 3 entries of 16 heads on 4, 130 tokens over up
// to 8192 keys, D = 64, 29 us, of which 17 the forward (2 its setup, 3 its first
// loads, 10 tiles of 0.85, 2.5 the parts) and 7 the join.  A prefix of 16000 tokens, 256
// rows a K/V head, D = 128 (66 MB): 22 us, of 120001 tokens and 128 rows (492 MB) 77
// us = 6.4 TB/s, bound by memory.
#include "fwd_tc_kernel.cuh"

namespace fattn {
namespace {

constexpr int kJoinThreads = 256;

// A warp a row of the output: lanes weigh the parts, four at most each, then take
// D/32 elements of every part, kAtOnce parts on their way at once.  In one order
// (own keys, then the prefix's), so that the result does not depend on anything else.
template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) rows_join_kernel(const __grid_constant__ RowsArgs a) {
    constexpr int kPer = D / 32, kAtOnce = 8;
    static_assert(kMaxSplits + 1 <= 5 * 32, "parts of a row in the lanes");
    // (Fewer than 2^32 rows: rows_join_launch.)
    const uint32_t w = (blockIdx.x * kJoinThreads + threadIdx.x) / 32;
    const int lane = threadIdx.x % 32;
    const uint32_t bh = w / static_cast<uint32_t>(a.Nq);
    const int i = static_cast<int>(w - bh * a.Nq);
    const int b = static_cast<int>(bh / static_cast<uint32_t>(a.H)), h = static_cast<int>(bh - b * a.H);
    const int kvh = h / a.share, hq = h % a.share;
    const int source = a.sources > 1 ? b : 0, among = b - source;  // (one source: the entry among its rows)
    const int u = (among / a.box_b * a.n_h + hq / a.box_h) * a.n_i + i / a.box_i;
    const int trow = ((among % a.box_b) * a.box_h + hq % a.box_h) * a.box_i + i % a.box_i;
    const int64_t at = (((static_cast<int64_t>(source) * a.Hkv + kvh) * a.tiles + u) * kTcBM + trow) * a.part_pitch;
    grid_dependency();
    if (b >= a.B) return;
    // What does not depend on the number of parts is on its way with it: the places
    // that may hold one (what lies in those that hold none is not used), the own
    // keys' part as place 0.
    const float* rows = a.part_o + at * D + lane * kPer;
    auto place = [&](int s) { return a.own_part ? (s == 0 ? a.part_pitch - 1 : s - 1) : s; };
    const int most = a.max_parts + a.own_part;
    const int per = __ldcg(a.part_count);
    const int tiles = (visible_keys(a, source, false) + kTcBN - 1) / kTcBN;
    float2 ml[5];
    float early[kAtOnce][kPer];
#pragma unroll
    for (int x = 0; x < 5; ++x)
        if (lane + 32 * x < most) ml[x] = __ldcg(a.part_ml + at + place(lane + 32 * x));
    auto load = [&](float (&v)[kPer], int s) {
        const float* src = rows + place(s) * D;
        if constexpr (kPer == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(src));
            v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(src));
            v[0] = f.x, v[1] = f.y;
        }
    };
#pragma unroll
    for (int y = 0; y < kAtOnce; ++y) load(early[y], min(y, most - 1));
    // (No more than the workspace has room for, whatever a forward that gave up left as `per`.)
    const int all = min(max((tiles + per - 1) / max(per, 1), 1), a.max_parts) + a.own_part;
    float m = -INFINITY;
#pragma unroll
    for (int x = 0; x < 5; ++x) {
        if (lane + 32 * x >= all) ml[x] = make_float2(-INFINITY, 0.f);
        m = fmaxf(m, ml[x].x);
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const bool none = m == -INFINITY;
    float acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int x = 0; x < 5; ++x) {
        if (32 * x >= all) break;
        const float mine = none ? 0.f : ex2_approx(ml[x].x - m);
        sum = fmaf(mine, ml[x].y, sum);
        const int upto = min(32, all - 32 * x);
        for (int s0 = 0; s0 < upto; s0 += kAtOnce) {
            float v[kAtOnce][kPer];
            const bool more = 32 * x + s0 + kAtOnce < all;
            if (more)  // the next ones
#pragma unroll
                for (int y = 0; y < kAtOnce; ++y) load(v[y], min(32 * x + s0 + kAtOnce + y, all - 1));
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) {
                const float wt = __shfl_sync(0xffffffffu, mine, min(s0 + y, 31));
                if (s0 + y < upto)
#pragma unroll
                    for (int e = 0; e < kPer; ++e) acc[e] = fmaf(wt, early[y][e], acc[e]);
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (more) early[y][e] = v[y][e];
            }
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const float inv = none ? 0.f : 1.f / sum;
    uint16_t* o = static_cast<uint16_t*>(a.o) + b * a.o_bs + h * a.o_hs + i * a.o_ns + lane * kPer;
    if constexpr (kPer == 4)
        *reinterpret_cast<uint2*>(o) =
            make_uint2(pack2(acc[0] * inv, acc[1] * inv, BF16), pack2(acc[2] * inv, acc[3] * inv, BF16));
    else
        *reinterpret_cast<uint32_t*>(o) = pack2(acc[0] * inv, acc[1] * inv, BF16);
    if (lane == 0 && a.lse != nullptr) a.lse[w] = none ? -INFINITY : (m + log2f(sum)) * kLn2;
}

template <int D, bool BF16>
cudaError_t launch_one(const RowsArgs& a, int grid, cudaStream_t stream) {
    auto* fn = attn_fwd_tc_kernel<D, BF16, false, kRows>;
    static std::atomic<bool> done[kMaxDevices] = {};
    const cudaError_t e = opt_in_smem_once(fn, kRowsAlloc<D>, done);
    if (e != cudaSuccess) return e;
    return launch_overlapped(fn, grid, kTcThreads, kRowsAlloc<D>, stream, a);
}

}  // namespace

cudaError_t rows_launch(const RowsArgs& a, int D, bool bf16, int grid, cudaStream_t s) {
    if (D == 128) return bf16 ? launch_one<128, true>(a, grid, s) : launch_one<128, false>(a, grid, s);
    return bf16 ? launch_one<64, true>(a, grid, s) : launch_one<64, false>(a, grid, s);
}

cudaError_t rows_join_launch(const RowsArgs& a, int D, bool bf16, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.H * a.Nq;
    if (rows * 32 + kJoinThreads > 0xffffffffll) return cudaErrorInvalidValue;  // (the entry points refuse it)
    const unsigned grid = static_cast<unsigned>((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
    auto* fn = D == 128 ? (bf16 ? rows_join_kernel<128, true> : rows_join_kernel<128, false>)
                        : (bf16 ? rows_join_kernel<64, true> : rows_join_kernel<64, false>);
    return launch_overlapped(fn, grid, kJoinThreads, 0, s, a);
}

cudaError_t rows_read_and_clear_error_word(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_error_word, sizeof(v));
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace fattn
