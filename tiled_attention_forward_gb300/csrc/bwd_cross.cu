// bwd_cross.cu -- the backward (bwd_tc_kernel.cuh) of cross attention: keys of a
// length of their own, rows by strides; the kernel of its row statistics, and the one
// that adds the parts of gradients that were cut.
//
// The query rows of all heads that share a K/V head are stacked into tiles, as in the
// forward, but of whole heads' boxes: a K/V head's dK and dV are sums over them, and
// no box may bring another group's rows.  The key kernel (dK, dV) and the query
// kernel (dQ) need nothing of one another, so the second starts as the first one's
// last CTAs run.  Where there are few blocks their inner tiles are cut into parts; where
// there are many of few inner tiles a CTA takes a run of them (bwd_cross_dq.cuh,
// bwd_cross_dkv.cuh).
//
// Measured (GB300): 4 entries of 16 heads, 4096 queries over up to 2000 keys, D = 128,
// bf16 (344 GFLOP, ragged) 474 us = 726 TFLOP/s: statistics 31, dK/dV 254, dQ 225, the
// last two overlapping.  dK/dV keeps the tensor pipe 53 % busy (three and a half waves of
// CTAs), dQ 44 %.
// Dense-shaped, 64 heads of 4096: 1471 us = 934 TFLOP/s (fattn_bwd 910).  2 entries of
// 8 heads on 2, 257 queries over up to 777 keys, D = 64: 19 us (one kernel after the
// other, uncut: 37).  32 heads on 4, D = 64, 28 queries over up to 5342 keys, 12
// entries: 113 us (a tile per head: 230).  fp16 over more than kLongKeys keys (what
// cross_most_kernel costs, two launches and a third read of the values): one query of 8
// heads over a million keys, D = 64, 1403 -> 1564 us; 300 over 100000, D = 128, 605 -> 649;
// 4 entries of 16 heads, 4096 over 17000 6040 -> 6120; 20 of 8 heads on 2 over 20000, D =
// 64, 39 -> 49.
#include "bwd_cross_dkv.cuh"
#include "bwd_cross_dq.cuh"
#include "bwd_tc_kernel.cuh"

#include <algorithm>

namespace fattn {
namespace {

// The largest |dO_i|^2 and |v_j|^2 of each K/V head of a batch entry, over its query rows
// and seen keys (rows that are not finite, whose gradients are not either, do not count):
// what grad_scale takes for fp16 over long keys.  `chunks` CTAs a K/V head; D/8 lanes a
// row, kMostLoads such rows on their way; a.most is zero before.  Maxima: whatever the
// order, the same.
constexpr int kMostLoads = 4;
template <int D>
__global__ void __launch_bounds__(256) cross_most_kernel(const __grid_constant__ CrossBwdArgs a, int chunks) {
    constexpr int kLanes = D / 8, kStep = 256 / kLanes;
    const int kvh = blockIdx.x / chunks, chunk = blockIdx.x % chunks, b = kvh / a.Hkv, kv_h = kvh - b * a.Hkv;
    const int share = a.H / a.Hkv, piece = threadIdx.x % kLanes;
    int keys = a.Nk;
    if (a.lens != nullptr) keys = min(max(a.lens[b], 0), a.Nk);
    float most[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {  // rows of dO, values
        const int rows = t == 0 ? share * a.N : keys, end = part_begin(rows, chunk + 1, chunks);
        const uint16_t* base = t == 0 ? static_cast<const uint16_t*>(a.dout) + b * a.do_bs + kv_h * share * a.do_hs
                                      : static_cast<const uint16_t*>(a.v) + b * a.v_bs + kv_h * a.v_hs;
        float mx = 0.f;
        // (Every lane of a warp takes as many turns.)
        for (int at = part_begin(rows, chunk, chunks); at < end; at += kMostLoads * kStep) {
            uint4 x[kMostLoads];
#pragma unroll
            for (int k = 0; k < kMostLoads; ++k) {
                const int r = at + k * kStep + static_cast<int>(threadIdx.x) / kLanes;
                x[k] = make_uint4(0u, 0u, 0u, 0u);
                if (r >= end) continue;
                const int hq = t == 0 ? r / a.N : 0;
                const int64_t off = t == 0 ? hq * a.do_hs + (r - hq * a.N) * a.do_ns : r * a.v_ns;
                x[k] = *reinterpret_cast<const uint4*>(base + off + 8 * piece);
            }
#pragma unroll
            for (int k = 0; k < kMostLoads; ++k) {
                const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                    sum = fmaf(u.x, u.x, sum);
                    sum = fmaf(u.y, u.y, sum);
                }
#pragma unroll
                for (int d = kLanes / 2; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (sum < INFINITY) mx = fmaxf(mx, sum);
            }
        }
        most[t] = mx;
    }
    // (Numbers that are not negative compare as their bits.)
    const uint32_t m0 = __reduce_max_sync(0xffffffffu, __float_as_uint(most[0]));
    const uint32_t m1 = __reduce_max_sync(0xffffffffu, __float_as_uint(most[1]));
    if (threadIdx.x % 32 == 0) {
        atomicMax(reinterpret_cast<uint32_t*>(&a.most[kvh].x), m0);
        atomicMax(reinterpret_cast<uint32_t*>(&a.most[kvh].y), m1);
    }
}

// -LSE_i * log2(e) and -Delta_i, Delta_i = dO_i . O_i, into the workspace in the order
// of the tiles' rows, [B*Hkv][tiles][2][128]; rows past Nq or behind a tile's box, and
// rows that saw no key (LSE = -inf), get -inf and 0.  fp16: of 2^kHeldP P, and f Delta
// (grad_scale).  A row is read as 16-byte pieces by D/8 lanes, kStatLoads such rows of O
// and of dO in flight a lane; rows are taken in the order in which they lie in
// memory (`heads_inner`: a token's heads one after the other).
constexpr int kStatLoads = 4;
template <int D>
constexpr int kStatRows = (32 / (D / 8)) * kStatLoads;  // of a warp

template <int D, bool BF16>
__global__ void __launch_bounds__(256) cross_stats_kernel(const __grid_constant__ CrossBwdArgs a, bool heads_inner) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    const int padded = a.n_i * a.box_i, share = a.H / a.Hkv;  // tokens, to whole boxes
    const int64_t rows = static_cast<int64_t>(a.BH) * padded;
    const int lane = threadIdx.x % 32, piece = lane % kLanes;
    // Row `lane / kLanes` of a warp's rows, and from one of a lane's rows to its next:
    // inner and outer index, batch entry.  (Fewer than 2^31 rows of an entry: 32-bit
    // divisions, which were half of all instructions with one a row.)
    const uint32_t per_b = static_cast<uint32_t>(a.H) * padded, inner = heads_inner ? a.H : padded;
    struct At {
        uint32_t b, outer, in;
    };
    auto first_of = [&](int64_t warp) {
        const int64_t row = warp * kStatRows<D> + lane / kLanes;
        At x;
        x.b = (row >> 32) == 0 ? static_cast<uint32_t>(row) / per_b : static_cast<uint32_t>(row / per_b);
        const uint32_t rest = static_cast<uint32_t>(row - static_cast<int64_t>(x.b) * per_b);
        x.outer = rest / inner;
        x.in = rest - x.outer * inner;
        return x;
    };
    const uint32_t outer_end = per_b / inner, entries = static_cast<uint32_t>(a.BH / a.H);
    auto step = [&](At& x) {
        x.in += kRows;
        while (x.in >= inner) {
            x.in -= inner;
            if (++x.outer == outer_end) {
                x.outer = 0;
                ++x.b;
            }
        }
    };
    grid_dependency();
    const int64_t warps = (rows + kStatRows<D> - 1) / kStatRows<D>, stride = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t warp = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / 32; warp < warps; warp += stride) {
        uint4 o[kStatLoads], g[kStatLoads];
        float lse[kStatLoads], f[kStatLoads];
        int64_t dst[kStatLoads];  // of the row's first statistic; < 0: no row
        At x = first_of(warp);
#pragma unroll
        for (int k = 0; k < kStatLoads; ++k) {
            if (k > 0) step(x);
            const uint32_t h = heads_inner ? x.in : x.outer, i = heads_inner ? x.outer : x.in;
            const int64_t bh = static_cast<int64_t>(x.b) * a.H + h;
            o[k] = g[k] = make_uint4(0u, 0u, 0u, 0u);
            lse[k] = -INFINITY;
            f[k] = 1.f;
            dst[k] = -1;
            if (x.b < entries) {
                if (a.box_h == 1 && a.box_i == kBT) {
                    dst[k] = (bh * a.n_i + i / kBT) * (2 * kBT) + i % kBT;
                } else {
                    const uint32_t kvh = h / share, hq = h - kvh * share, uh = hq / a.box_h, ui = i / a.box_i;
                    const int64_t tile = (static_cast<int64_t>(x.b) * a.Hkv + kvh) * a.tiles + uh * a.n_i + ui;
                    const uint32_t r = (hq - uh * a.box_h) * a.box_i + (i - ui * a.box_i);
                    dst[k] = tile * (2 * kBT) + r;
                    if (r == 0)  // the rows behind the box
                        for (int y = a.box_h * a.box_i + piece; y < kBT; y += kLanes) {
                            a.ws[dst[k] + y] = -INFINITY;
                            a.ws[dst[k] + kBT + y] = 0.f;
                        }
                }
            }
            if (x.b < entries && i < static_cast<uint32_t>(a.N)) {
                o[k] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.o) + x.b * a.o_bs + h * a.o_hs +
                                                       i * a.o_ns + 8 * piece);
                g[k] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dout) + x.b * a.do_bs +
                                                       h * a.do_hs + i * a.do_ns + 8 * piece);
                if (piece == 0) lse[k] = a.lse[bh * a.N + i];
                if (!BF16) f[k] = grad_scale<BF16>(a, static_cast<int>(x.b * a.Hkv + h / share)).f;
            }
        }
#pragma unroll
        for (int k = 0; k < kStatLoads; ++k) {
            const uint32_t x[4] = {o[k].x, o[k].y, o[k].z, o[k].w}, y[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                float2 u, v;
                if (BF16) {
                    u = make_float2(__uint_as_float(x[w] << 16), __uint_as_float(x[w] & 0xffff0000u));
                    v = make_float2(__uint_as_float(y[w] << 16), __uint_as_float(y[w] & 0xffff0000u));
                } else {
                    u = __half22float2(*reinterpret_cast<const __half2*>(&x[w]));
                    v = __half22float2(*reinterpret_cast<const __half2*>(&y[w]));
                }
                sum = fmaf(u.x, v.x, sum);
                sum = fmaf(u.y, v.y, sum);
            }
#pragma unroll
            for (int d = kLanes / 2; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (piece == 0 && dst[k] >= 0) {
                const bool none = lse[k] == -INFINITY;
                a.ws[dst[k]] = none ? -INFINITY : fmaf(-lse[k], 1.4426950408889634f, BF16 ? 0.f : kHeldP);
                a.ws[dst[k] + kBT] = none ? 0.f : -sum * f[k];
            }
        }
    }
}

// Adds the parts, in order: a thread 8 elements of a row, of dk and dv (blocks of
// row tiles first) and then of dq.  Rows that no part has are zeros.
constexpr int kAddThreads = 256;
template <int D, bool BF16>
__global__ void __launch_bounds__(kAddThreads) cross_add_kernel(const __grid_constant__ CrossBwdArgs a, int64_t kv_rows) {
    constexpr int kPieces = D / 8;
    grid_dependency();
    int64_t row = (static_cast<int64_t>(blockIdx.x) * kAddThreads + threadIdx.x) / kPieces;
    const int d = 8 * (threadIdx.x % kPieces);
    const bool kv = row < kv_rows;  // rows of dk and dv: [B * Hkv][Nk][2]
    if (!kv) row -= kv_rows;
    const int n = kv ? a.Nk : a.N, heads = kv ? a.Hkv : a.H, accs = kv ? 2 : 1;
    const int acc = static_cast<int>(row % accs);
    row /= accs;
    const int64_t bh = row / n;
    const int i = static_cast<int>(row - bh * n);
    const int64_t b = bh / heads, h = bh - b * heads;
    if (b >= a.BH / a.H || (!kv && a.parts_q == 1)) return;
    int keys = a.Nk;
    if (a.lens != nullptr) keys = min(max(a.lens[b], 0), a.Nk);
    const int parts = kv ? a.parts_k : a.parts_q, tiles = (keys + kBT - 1) / kBT;
    const int64_t padded = (kv ? a.tiles_k : a.tiles) * kBT, step = static_cast<int64_t>(a.BHkv) * padded * accs * D;
    int64_t at = bh * padded + i;
    if (!kv) {
        const int share = a.H / a.Hkv, hq = static_cast<int>(h) % share, uh = hq / a.box_h, ui = i / a.box_i;
        at = (bh / share) * padded + (uh * a.n_i + ui) * kBT + (hq - uh * a.box_h) * a.box_i + (i - ui * a.box_i);
    }
    const float* src = (kv ? a.part_kv : a.part_q) + (at * accs + acc) * D + d;
    float sum[8] = {};
    const int upto = kv && i >= keys ? 0 : parts;
#pragma unroll 4
    for (int p = 0; p < upto; ++p) {
        if (!kv && part_begin(tiles, p, parts) == part_begin(tiles, p + 1, parts)) continue;
        const float4 x = __ldcg(reinterpret_cast<const float4*>(src + p * step));
        const float4 y = __ldcg(reinterpret_cast<const float4*>(src + p * step + 4));
        sum[0] += x.x, sum[1] += x.y, sum[2] += x.z, sum[3] += x.w;
        sum[4] += y.x, sum[5] += y.y, sum[6] += y.z, sum[7] += y.w;
    }
    uint16_t* dst;
    if (!kv)
        dst = static_cast<uint16_t*>(a.dq) + b * a.dq_bs + h * a.dq_hs + i * a.dq_ns;
    else if (acc == 0)
        dst = static_cast<uint16_t*>(a.dv) + b * a.dv_bs + h * a.dv_hs + i * a.dv_ns;
    else
        dst = static_cast<uint16_t*>(a.dk) + b * a.dk_bs + h * a.dk_hs + i * a.dk_ns;
    *reinterpret_cast<uint4*>(dst + d) = make_uint4(pack16(sum[0], sum[1], BF16), pack16(sum[2], sum[3], BF16),
                                                    pack16(sum[4], sum[5], BF16), pack16(sum[6], sum[7], BF16));
}

// launch_overlapped with a second argument.
template <typename X>
cudaError_t launch_two(void (*fn)(CrossBwdArgs, X), unsigned grid, unsigned threads, cudaStream_t s,
                       const CrossBwdArgs& a, X x) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, a, x);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

template <int D, bool BF16>
cudaError_t launch_add(const CrossBwdArgs& a, cudaStream_t s) {
    if (a.parts_k == 1 && a.parts_q == 1) return cudaSuccess;
    const int64_t kv_rows = a.parts_k > 1 ? static_cast<int64_t>(a.BHkv) * a.Nk * 2 : 0;
    const int64_t rows = kv_rows + (a.parts_q > 1 ? static_cast<int64_t>(a.BH) * a.N : 0);
    return launch_two(cross_add_kernel<D, BF16>, static_cast<unsigned>((rows * (D / 8) + kAddThreads - 1) / kAddThreads),
                      kAddThreads, s, a, kv_rows);
}

// The CTAs that share a K/V head's key blocks, of one query tile, that end first: 12 a
// CTA's start and end, 6 a block.
int key_chunks_of(const CrossBwdArgs& a, int sms) {
    int64_t least = INT64_MAX, chunks = a.tiles_k;
    for (int64_t m = 1, last_c = 0; m <= std::min(a.tiles_k, 128); ++m) {
        const int64_t c = (a.tiles_k + m - 1) / m;
        if (c == last_c) continue;
        last_c = c;
        const int64_t each = 6 * m + 12, cost = (c * a.BHkv + sms - 1) / sms * each + each / 4;
        if (cost < least) {
            least = cost;
            chunks = c;
        }
    }
    return static_cast<int>(chunks);
}

// The CTAs that share a K/V head's query tiles: those with which the query kernel, which
// starts as the key kernel's CTAs leave, ends first.  In units of 0.2 us: a key block's
// CTA takes 8 a query tile and 24, a run of query tiles 6 a key tile, 3 a query tile and
// 24; all keys are taken to be seen.  (8 heads of K/V, 4 query heads each, 222 queries
// over 334 keys, D = 64, 7 entries: 2 CTAs a head 37.3 us, 4 43.6; 4 entries of 16 heads,
// 4096 queries over up to 900 keys, D = 64: 8 CTAs a head 178, 2 205.)
int chunks_of(const CrossBwdArgs& a, int sms) {
    const int64_t blocks = static_cast<int64_t>(a.tiles_k) * a.BHkv * a.parts_k;
    const int64_t block = 8 * ((a.tiles + a.parts_k - 1) / a.parts_k) + 24;
    const int64_t early = blocks / sms * block, late = early + block;  // SMs free: at first and at last
    const int64_t n_late = blocks % sms, n_early = sms - n_late;
    int64_t least = INT64_MAX, chunks = 1, last_c = 0;
    for (int64_t m = 1; m <= std::min(a.tiles, 128); ++m) {  // query tiles of a CTA
        const int64_t c = (a.tiles + m - 1) / m, ctas = c * a.BHkv, each = m * (6 * a.tiles_k + 3) + 24;
        if (c == last_c) continue;  // (as many with a shorter run: seen)
        last_c = c;
        // CTAs that have ended by `t`.
        auto ended = [&](int64_t t) {
            return n_early * ((t - early) / each) + (t > late ? n_late * ((t - late) / each) : 0);
        };
        int64_t lo = early, hi = late + (ctas / sms + 1) * each;  // (by then all have)
        while (hi - lo > 1) {
            const int64_t t = lo + (hi - lo) / 2;
            (ended(t) >= ctas ? hi : lo) = t;
        }
        const int64_t cost = hi + each / 8;  // (lengths differ: rather shorter ones)
        if (cost < least) {
            least = cost;
            chunks = c;
        }
    }
    return static_cast<int>(chunks);
}

template <int D, bool BF16, bool ONE>
cudaError_t launch_dq(const CrossBwdArgs& a, int chunks, cudaStream_t s) {
    static std::atomic<bool> opted_in[kMaxDevices] = {};
    auto* kernel = cross_dq_kernel<D, BF16, ONE>;
    const cudaError_t e = opt_in_smem_once(kernel, CrossDqLayout<D, ONE>::kBytes, opted_in);
    if (e != cudaSuccess) return e;
    CrossBwdArgs x = a;
    x.chunks_q = chunks;
    return launch_overlapped(kernel, static_cast<unsigned>(static_cast<int64_t>(x.chunks_q) * a.BHkv), kBwdThreads,
                             CrossDqLayout<D, ONE>::kBytes, s, x);
}

template <int D, bool BF16>
cudaError_t launch_all(const CrossBwdArgs& a, int sms, cudaStream_t s) {
    // (Without queries the key kernel, without keys the query kernel writes zeros.)
    const int64_t warps = (static_cast<int64_t>(a.BH) * a.n_i * a.box_i + kStatRows<D> - 1) / kStatRows<D>;
    cudaError_t e = cudaSuccess;
    if (a.N > 0 && a.Nk > 0) {
        if (!BF16 && a.most != nullptr) {
            // (Neither lets the next one start early.)
            if ((e = cudaMemsetAsync(a.most, 0, static_cast<size_t>(a.BHkv) * sizeof(float2), s)) != cudaSuccess) return e;
            const int chunks = std::min(std::max(4 * sms / a.BHkv, 1), 64);
            cross_most_kernel<D><<<static_cast<unsigned>(chunks) * static_cast<unsigned>(a.BHkv), 256, 0, s>>>(a, chunks);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
        }
        const int64_t blocks = (warps + 7) / 8;
        e = launch_two(cross_stats_kernel<D, BF16>, static_cast<unsigned>(std::min<int64_t>(blocks, 16 * sms)), 256, s, a,
                       a.o_hs < a.o_ns);
        if (e != cudaSuccess) return e;
    }
    static std::atomic<bool> run_done[kMaxDevices] = {};
    static std::atomic<bool> kv_done[kMaxDevices] = {};
    static std::atomic<bool> q_done[kMaxDevices] = {};
    const int key_chunks = a.tiles == 1 ? key_chunks_of(a, sms) : a.tiles_k;
    if (key_chunks < a.tiles_k) {  // one query tile: runs of key blocks
        auto* run = cross_dkv_kernel<D, BF16>;
        if ((e = opt_in_smem_once(run, CrossDkvLayout<D>::kBytes, run_done)) != cudaSuccess) return e;
        CrossBwdArgs x = a;
        x.chunks_k = key_chunks;
        e = launch_overlapped(run, static_cast<unsigned>(static_cast<int64_t>(key_chunks) * a.BHkv), kBwdThreads,
                              CrossDkvLayout<D>::kBytes, s, x);
        if (e != cudaSuccess) return e;
    } else if (a.tiles_k > 0) {
        auto* kkv = attn_bwd_kernel<D, BF16, true, false, true>;
        if ((e = opt_in_smem_once(kkv, BwdLayout<D, true>::kBytes, kv_done)) != cudaSuccess) return e;
        e = launch_overlapped(kkv, static_cast<unsigned>(a.tiles_k * a.BHkv * a.parts_k), kBwdThreads, BwdLayout<D, true>::kBytes, s, a);
        if (e != cudaSuccess) return e;
    }
    if (a.tiles == 0) return cudaSuccess;
    // A run of query tiles a CTA, where that ends earlier; else, and for parts, one each.
    // (One each by the run's kernel: 8 heads on 2, 257 queries over up to 777 keys, D =
    // 128, 2 entries 23.8 us, and not 22.8.)
    const int chunks = a.parts_q == 1 && a.tiles_k > 0 ? chunks_of(a, sms) : a.tiles;
    if (chunks < a.tiles) {
        e = a.tiles_k == 1 ? launch_dq<D, BF16, true>(a, chunks, s) : launch_dq<D, BF16, false>(a, chunks, s);
        return e == cudaSuccess ? launch_add<D, BF16>(a, s) : e;
    }
    auto* kq = attn_bwd_kernel<D, BF16, false, false, true>;
    if ((e = opt_in_smem_once(kq, BwdLayout<D, false>::kBytes, q_done)) != cudaSuccess) return e;
    const unsigned grid_q = static_cast<unsigned>(a.tiles * a.BHkv * a.parts_q);
    // (Behind the key kernel only: it reads and writes without waiting first.)
    if (a.tiles_k > 0) {
        e = launch_overlapped(kq, grid_q, kBwdThreads, BwdLayout<D, false>::kBytes, s, a);
        return e == cudaSuccess ? launch_add<D, BF16>(a, s) : e;
    }
    kq<<<grid_q, kBwdThreads, BwdLayout<D, false>::kBytes, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t bwd_cross_launch(const CrossBwdArgs& a, int D, bool bf16, int sms, cudaStream_t s) {
    if (D == 128) return bf16 ? launch_all<128, true>(a, sms, s) : launch_all<128, false>(a, sms, s);
    return bf16 ? launch_all<64, true>(a, sms, s) : launch_all<64, false>(a, sms, s);
}

cudaError_t bwd_cross_read_and_clear_error_word(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_error_word, sizeof(v));
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace fattn
