// bwd_cross_dkv.cuh -- dK and dV of cross attention whose queries fit one tile: the rows
// of all heads that share a K/V head, at most 128 (latents or single tokens over long
// keys).
//
//   dV_j = sum_i P_ij dO_i,  dK_j = scale sum_i dS_ij q_i,
//   P_ij = exp(s_ij - LSE_i),  dS_ij = P_ij (dO_i . v_j - Delta_i)
//
// A CTA for each key block (attn_bwd_kernel) is then one tile between its start and its
// end.  Here a CTA has a run of one K/V head's key blocks: Q, dO and their statistics
// stay, (K, V) pairs come through a ring, and the next block's scores are made while the
// warps finish this one and write its rows.  TMEM as there at D = 128: S^T [0,128), dP^T
// [128,256) under the 16-bit P^T and dS^T, then dV and dK.
//
// Measured (GB300; all of the gradients, a CTA a key block -> this, D = 64 / 128), 16
// heads: 85 queries over 7488 keys, 8 entries 374 -> 205 / 473 -> 291 us; 64 over 2000,
// 12 entries 172 -> 91 / 225 -> 127; 1 over up to 2729, 8 entries 131 -> 69 / 156 -> 94;
// 100 over 1000, one entry (a block a CTA in either) 16.7 / 20.1.  32 heads on 8, 2 over
// up to 3036, 9 entries 83 -> 49 / 102 -> 66.  Bound by the chain S -> P, dS -> dV, dK ->
// rows of a block.
#pragma once

#include "bwd_tc_kernel.cuh"

namespace fattn {
namespace {

template <int D>
struct CrossDkvLayout {
    static constexpr int kTile = kBT * D * 2;
    static constexpr int kSlots = D == 128 ? 2 : 4;              // of (K, V)
    static constexpr int kKv = 2 * kTile;                        // behind Q and dO
    static constexpr int kRows = kKv + kSlots * 2 * kTile;       // 4 KB of each elementwise warp
    static constexpr int kStats = kRows + 8 * 4096;
    static constexpr int kBar = kStats + 2 * kBT * 4;
    // barriers: q_full, full[], empty[], s_full, acc_full, done; abort flag; TMEM slot
    static constexpr int kBytes = kBar + (4 + 2 * kSlots) * 8 + 16;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kBwdThreads, 1) cross_dkv_kernel(const __grid_constant__ CrossBwdArgs a) {
    using L = CrossDkvLayout<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    grid_dependency();  // the statistics; the query kernel may start beside the last CTAs here
    if ((smem_u32(smem) & 1023u) != 0u) {
        if (threadIdx.x == 0) atomicOr(&g_error_word, 1u << kDevErrInternal);
        return;
    }
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* full = q_full + 1;
    uint64_t* empty = full + L::kSlots;
    uint64_t* s_full = empty + L::kSlots;
    uint64_t* acc_full = s_full + 1;
    uint64_t* done = acc_full + 1;
    uint32_t* abort_flag = reinterpret_cast<uint32_t*>(done + 1);
    uint32_t* tmem_slot = abort_flag + 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int kvh = blockIdx.x / a.chunks_k, chunk = blockIdx.x % a.chunks_k;
    const int b = kvh / a.Hkv, kv_h = kvh - b * a.Hkv;
    int keys = a.Nk;
    if (a.lens != nullptr) {
        const int len = a.lens[b];
        if ((len < 0 || len > a.Nk) && threadIdx.x == 0) atomicOr(&g_error_word, 1u << kDevErrInvalidArg);
        keys = min(max(len, 0), a.Nk);
    }
    const int j0 = part_begin(a.tiles_k, chunk, a.chunks_k), end = part_begin(a.tiles_k, chunk + 1, a.chunks_k);
    const int n = max(0, min(end, (keys + kBT - 1) / kBT) - j0);  // blocks with keys
    BwdTask behind = {};
    behind.bh = kvh;
    for (behind.blk = j0 + n; behind.blk < end; ++behind.blk) bwd_store_zeros<D, true>(a, behind);
    if (n == 0) return;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * L::kSlots + 4; ++i) mbar_init(&q_full[i], 1);  // (all of them)
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = t_dv + D;

    if (warp == kTmaWarp) {
        if (lane == 0) {
            const QueryBox q = query_box(a, kvh, 0);
            mbar_arrive_expect_tx(q_full, 2 * (D / 64) * a.box_h * a.box_i * 128 + 2 * kBT * 4);
            for (int at = 0; at < D / 64; ++at) {
                tma_load_4d(smem + at * kBT * 128, &a.tmap_q, q_full, at * 64, q.i, q.h, b);
                tma_load_4d(smem + L::kTile + at * kBT * 128, &a.tmap_do, q_full, at * 64, q.i, q.h, b);
            }
            bulk_load(smem + L::kStats, a.ws + static_cast<int64_t>(kvh) * (2 * kBT), 2 * kBT * 4, q_full);
            int issued = 0;
            bool ok = true;
            for (int g = 0; g < n; ++g) {
                const int s = g % L::kSlots;
                if (g >= L::kSlots)
                    ok = mbar_wait_bounded(&empty[s], ((g / L::kSlots) - 1) & 1u, abort_flag, &g_error_word, a.timeout_ns);
                if (!ok) break;
                uint8_t* st = smem + L::kKv + s * 2 * L::kTile;
                mbar_arrive_expect_tx(&full[s], 2 * L::kTile);
                for (int at = 0; at < D / 64; ++at) {
                    tma_load_4d(st + at * kBT * 128, &a.tmap_k, &full[s], at * 64, (j0 + g) * kBT, kv_h, b);
                    tma_load_4d(st + L::kTile + at * kBT * 128, &a.tmap_v, &full[s], at * 64, (j0 + g) * kBT, kv_h, b);
                }
                ++issued;
            }
            if (!ok) {
                // Let the copies already started land before the CTA leaves.
                for (int i = max(0, issued - L::kSlots); i < issued; ++i)
                    mbar_wait_bounded(&full[i % L::kSlots], (i / L::kSlots) & 1u, nullptr, &g_error_word, a.timeout_ns);
                mbar_wait_bounded(q_full, 0u, nullptr, &g_error_word, a.timeout_ns);
            }
        }
    } else if (warp == kMmaWarp || warp == kHelperWarp) {
        // The issuing warp and its helper, which does the waits, run one schedule; after
        // an abort they run it dry (no waits, no products), as in attn_bwd_kernel.
        const bool issuer = warp == kMmaWarp;
        constexpr uint32_t kIdescS = idesc_f16_f32(kBT, kBT, BF16 ? 1u : 0u, 0u, 0u);
        constexpr uint32_t kIdescAcc = idesc_f16_f32(kBT, D, BF16 ? 1u : 0u, 0u, 1u);
        const uint64_t kmaj = smem_desc_sw128(0u, 16u, 1024u);
        const uint64_t mnmaj = smem_desc_sw128(0u, kBT * 128u, 1024u);
        const uint32_t q_s = smem_u32(smem), do_s = q_s + L::kTile;
        auto k_s = [&](int g) { return smem_u32(smem + L::kKv + g % L::kSlots * 2 * L::kTile); };
        // dst = rows x cols^T, both K-major over D.
        auto scores = [&](uint32_t dst, uint32_t rows, uint32_t cols) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = ((kk / 4) * (kBT * 128) + (kk % 4) * 32) >> 4;
                mma_ss(dst, kmaj + (rows >> 4) + off, kmaj + (cols >> 4) + off, kIdescS, kk > 0 ? 1u : 0u);
            }
        };
        auto issue_s = [&](int g) { scores(t_s, k_s(g), q_s); };
        auto issue_dp = [&](int g) {  // (the pair's last reader)
            scores(t_dp, k_s(g) + L::kTile, do_s);
            mma_commit(s_full);
            mma_commit(&empty[g % L::kSlots]);
        };
        // dV += P^T dO, dK += dS^T Q over queries [64 h, 64 h + 64): 16-bit operands in
        // the first and second 16 of each 32 columns of dP^T.
        auto issue_acc = [&](int h) {
#pragma unroll
            for (int kk = 4 * h; kk < 4 * (h + 1); ++kk) {
                const uint64_t boff = (kk * 16 * 128) >> 4;
                const uint32_t acol = (kk / 2) * 32 + (kk % 2) * 8;
                mma_ts(t_dv, t_dp + acol, mnmaj + (do_s >> 4) + boff, kIdescAcc, kk > 0 ? 1u : 0u);
                mma_ts(t_dk, t_dp + acol + 16, mnmaj + (q_s >> 4) + boff, kIdescAcc, kk > 0 ? 1u : 0u);
            }
        };
        bool ok = true;
        auto wait_kv = [&](int g) {
            if (!issuer && ok) ok = warp_wait(&full[g % L::kSlots], (g / L::kSlots) & 1u, abort_flag, a.timeout_ns);
        };
        auto sync = [&]() {
            ok = named_barrier_and(kSyncBar, kSyncThreads, ok);
            if (issuer) tc_fence_after();
        };
        auto take = [&](uint32_t bar) {
            if (issuer) {
                named_barrier_sync(bar, kEwThreads);
                tc_fence_after();
            }
        };
        auto issue = [&](auto&& f) {
            if (issuer && ok) {
                if (elect_one_sync()) f();
                __syncwarp();
            }
        };
        if (!issuer) {
            ok = warp_wait(q_full, 0u, abort_flag, a.timeout_ns);
            if (ok) {  // rows behind the box: zeros, which their weights of 0 meet
                bwd_zero_tail<D>(smem, a.box_h * a.box_i);
                bwd_zero_tail<D>(smem + L::kTile, a.box_h * a.box_i);
            }
        }
        wait_kv(0);
        sync();
        issue([&] {
            issue_s(0);
            issue_dp(0);
        });
        for (int g = 0; g < n; ++g) {
            const bool more = g + 1 < n;
            take(kPBar);
            issue([&] { issue_acc(0); });
            take(kLdBar);
            if (more) {  // the next block's scores over those just loaded
                wait_kv(g + 1);
                sync();
                issue([&] { issue_s(g + 1); });
            }
            take(kPBar + 1);
            issue([&] {
                issue_acc(1);
                mma_commit(acc_full);
                if (more) issue_dp(g + 1);  // over the operands just read, in issue order
            });
        }
        if (issuer) {
            if (elect_one_sync()) mma_commit(done);  // fires once every product above has completed
            __syncwarp();
        }
    } else {
        // Warps w and w+4 share TMEM lanes (a thread a key row) and split the columns.
        const int quarter = warp % 4, half = warp / 4;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        uint8_t* stage = smem + L::kRows + warp * 4096;
        const float* nlse2s = reinterpret_cast<const float*>(smem + L::kStats);
        const float* ndeltas = nlse2s + kBT;
        const GradScale held = grad_scale<BF16>(a, kvh);
        // Block g's gradients, through the warp's own memory, whole halves of rows at a
        // time; rows of keys that no query sees are zeros.
        auto store = [&](int g) {
            const int row0 = (j0 + g) * kBT + quarter * 32;
#pragma unroll 1
            for (int acc = 0; acc < 2; ++acc) {
                const float mul = acc == 0 ? kDvMul<BF16> : held.mul;
                __syncwarp();
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t v[32];
                    tmem_ld32((acc == 0 ? t_dv : t_dk) + lane_off + (half * (D / 64) + c) * 32, v);
                    tmem_wait_ld();
                    reg_fence(v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t y[4];
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            y[w] = pack16(__uint_as_float(v[8 * e + 2 * w]) * mul, __uint_as_float(v[8 * e + 2 * w + 1]) * mul, BF16);
                        *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * c + e) ^ (lane & 7)) << 4)) =
                            make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                __syncwarp();
                constexpr int kPieces = D / 16;  // of 16 bytes in half a row
                const int64_t ns = acc == 0 ? a.dv_ns : a.dk_ns;
                uint16_t* base = (acc == 0 ? static_cast<uint16_t*>(a.dv) + b * a.dv_bs + kv_h * a.dv_hs
                                           : static_cast<uint16_t*>(a.dk) + b * a.dk_bs + kv_h * a.dk_hs) +
                                 half * (D / 2) + 8 * (lane % kPieces);
#pragma unroll
                for (int e = 0; e < kPieces; ++e) {
                    const int rr = e * (32 / kPieces) + lane / kPieces, i = row0 + rr;
                    uint4 y = *reinterpret_cast<const uint4*>(stage + rr * 128 + (((lane % kPieces) ^ (rr & 7)) << 4));
                    if (i >= keys) y = make_uint4(0u, 0u, 0u, 0u);
                    if (i < a.Nk) *reinterpret_cast<uint4*>(base + i * ns) = y;
                }
            }
        };
        bool ok = warp_wait(q_full, 0u, abort_flag, a.timeout_ns);  // (the statistics)
        int failed_at = 0;  // first block not handed over when a wait gave up
        for (int g = 0; g < n && ok; ++g) {
            if (g > 0) {  // the last block's rows, before the issuing warp may overwrite them
                ok = warp_wait(acc_full, (g - 1) & 1u, abort_flag, a.timeout_ns);
                tc_fence_after();
                if (ok) store(g - 1);
            }
            if (ok) ok = warp_wait(s_full, g & 1u, abort_flag, a.timeout_ns);
            if (!ok) {
                failed_at = g;
                break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int cq = 64 * h + 32 * half;  // this warp's first query column
                uint32_t sv[32], dpv[32];
                tmem_ld32(t_s + lane_off + cq, sv);
                tmem_ld32(t_dp + lane_off + cq, dpv);
                tmem_wait_ld();
                reg_fence(sv);
                reg_fence(dpv);
                if (h == 1) {
                    tc_fence_before();
                    __syncwarp();
                    named_barrier_arrive(kLdBar, kEwThreads);
                }
                // P^T = exp2(s*scale*log2e - LSE2) and dS^T = P^T (dP^T - Delta).
                uint32_t pk[16], dsk[16];
#pragma unroll
                for (int e4 = 0; e4 < 32; e4 += 4) {
                    const float4 nl = *reinterpret_cast<const float4*>(nlse2s + cq + e4);
                    const float4 nd = *reinterpret_cast<const float4*>(ndeltas + cq + e4);
#pragma unroll
                    for (int h2 = 0; h2 < 2; ++h2) {
                        const int e = e4 + 2 * h2;
                        float x0, x1, d0, d1;
                        fma2(x0, x1, __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]), a.sl2, a.sl2, h2 ? nl.z : nl.x,
                             h2 ? nl.w : nl.y);
                        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                        minus_delta<!BF16>(d0, d1, dpv[e], dpv[e + 1], held.f, h2 ? nd.z : nd.x, h2 ? nd.w : nd.y);
                        mul2(d0, d1, p0, p1, d0, d1);
                        pk[e / 2] = pack16(p0, p1, BF16);
                        dsk[e / 2] = pack16(d0, d1, BF16);
                    }
                }
                tmem_st16(t_dp + lane_off + cq, pk);
                tmem_st16(t_dp + lane_off + cq + 16, dsk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                named_barrier_arrive(kPBar + h, kEwThreads);
            }
        }
        if (!ok)  // meet the issuing warp, which runs its schedule to the end
            for (int g = failed_at; g < n; ++g) {
                __syncwarp();
                named_barrier_arrive(kPBar, kEwThreads);
                named_barrier_arrive(kLdBar, kEwThreads);
                named_barrier_arrive(kPBar + 1, kEwThreads);
            }
        const bool fin = warp_wait(done, 0u, nullptr, a.timeout_ns);
        tc_fence_after();
        if (ok && fin) store(n - 1);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace
}  // namespace fattn
