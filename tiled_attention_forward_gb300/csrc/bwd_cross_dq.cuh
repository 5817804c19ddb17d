// bwd_cross_dq.cuh -- dQ of cross attention, several query tiles a CTA.
//
//   dQ_i = scale sum_j dS_ij k_j,  dS_ij = exp(s_ij - LSE_i) (dO_i . v_j - Delta_i)
//
// A CTA for each query tile (attn_bwd_kernel) is, over few key tiles, mostly its own
// start and end.  Here a CTA has a run of one K/V head's query tiles, and their key
// tiles follow one another without a gap: (Q, dO) pairs come through a ring, the scores
// of the next key tile are made while the warps work on this one (S in two buffers of
// TMEM), and a query tile's dQ is read from TMEM together with the first dS of the
// next, so that no warp waits for a product.  Rows leave through 4 KB of shared memory
// a warp, whole halves of rows at a time.  ONE, keys of one tile (Nk <= 128): K and V
// stay.  Otherwise they stream, in rings of their own.  At D = 128 the memory then holds
// one pair of Q and dO, which the next one's copy follows, and threads write their own
// half rows.
//
// Measured (GB300; all of the gradients, a CTA a query tile -> this).  Keys of one tile:
// 8 heads on 1, 3572 queries over 87 keys, D = 128, 18 entries 303 -> 225 us; 16 heads,
// 7594 over 7, D = 64, 14 entries 669 -> 344.  16 heads, D = 64 / 128: 2000 queries over
// 200 keys, 12 entries 209 -> 154 / 290 -> 289; 4 entries of 4096 over 512 206 -> 162 /
// 289 -> 272, over up to 900 210 -> 178 / 293 -> 283, over up to 2000 346 -> 322 / 484 ->
// 474.  Bound by the chain S -> dS -> dQ of a tile, with one key tile by memory too.
#pragma once

#include "bwd_tc_kernel.cuh"

namespace fattn {
namespace {

template <int D, bool ONE>
struct CrossDqLayout {
    static constexpr int kTile = kBT * D * 2;
    static constexpr int kQs = ONE ? (D == 64 ? 4 : 2) : (D == 64 ? 2 : 1);  // slots of (Q, dO), K and V
    static constexpr int kKs = ONE ? 1 : (D == 64 ? 4 : 3);
    static constexpr int kVs = ONE ? 1 : (D == 64 ? 4 : 2);
    static constexpr bool kStaged = ONE || D == 64;  // rows leave through memory of their own
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + kQs * 2 * kTile;
    static constexpr int kV = kK + kKs * kTile;
    static constexpr int kRows = kV + kVs * kTile;               // 4 KB of each elementwise warp
    static constexpr int kBar = kRows + (kStaged ? 8 * 4096 : 0);
    // barriers: full and empty of Q, K and V slots, s_full[2], acc_full, done; abort flag; TMEM slot
    static constexpr int kBytes = kBar + (4 + 2 * (kQs + kKs + kVs)) * 8 + 16;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int D, bool BF16, bool ONE>
__global__ void __launch_bounds__(kBwdThreads, 1) cross_dq_kernel(const __grid_constant__ CrossBwdArgs a) {
    using L = CrossDqLayout<D, ONE>;
    extern __shared__ __align__(1024) uint8_t smem[];
    // As of attn_bwd_kernel: starts as the key kernel's last CTAs run, of which it reads
    // nothing; its end waits for that one's.
    auto wait_key_kernel = [&]() { asm volatile("griddepcontrol.wait;" ::: "memory"); };
    if ((smem_u32(smem) & 1023u) != 0u) {
        if (threadIdx.x == 0) atomicOr(&g_error_word, 1u << kDevErrInternal);
        wait_key_kernel();
        return;
    }
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* q_empty = q_full + L::kQs;
    uint64_t* k_full = q_empty + L::kQs;
    uint64_t* k_empty = k_full + L::kKs;
    uint64_t* v_full = k_empty + L::kKs;
    uint64_t* v_empty = v_full + L::kVs;
    uint64_t* s_full = v_empty + L::kVs;  // by key tile parity
    uint64_t* acc_full = s_full + 2;
    uint64_t* done = acc_full + 1;
    uint32_t* abort_flag = reinterpret_cast<uint32_t*>(done + 1);
    uint32_t* tmem_slot = abort_flag + 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int kvh = blockIdx.x / a.chunks_q, chunk = blockIdx.x % a.chunks_q;
    const int b = kvh / a.Hkv, kv_h = kvh - b * a.Hkv;
    const int u0 = part_begin(a.tiles, chunk, a.chunks_q), n = part_begin(a.tiles, chunk + 1, a.chunks_q) - u0;
    int keys = a.Nk;
    // (Read through L2, like the statistics: launch_overlapped.  The key kernel reports one out of range.)
    if (a.lens != nullptr) keys = min(max(__ldcg(a.lens + b), 0), a.Nk);
    // Key tiles of a query tile, and of the CTA: tile g is key tile g % nk of query
    // tile u0 + g / nk.
    const int nk = ONE ? 1 : (keys + kBT - 1) / kBT, tiles = n * nk;
    if (keys == 0) {
        BwdTask tk = {};
        tk.bh = kvh;
        for (int it = 0; it < n; ++it) {
            tk.blk = u0 + it;
            bwd_store_zeros<D, false>(a, tk);
        }
        wait_key_kernel();
        return;
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * (L::kQs + L::kKs + L::kVs) + 4; ++i) mbar_init(&q_full[i], 1);  // (all of them)
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
    // TMEM columns: S (then the 16-bit dS) [0,128) and [128,256) by tile parity,
    // dP [256,384), dQ [384,384+D).
    const uint32_t t_s = tmem, t_dp = tmem + 256, t_acc = tmem + 384;

    if (warp == kTmaWarp) {
        if (lane == 0) {
            const uint32_t q_bytes = 2 * (D / 64) * a.box_h * a.box_i * 128;
            bool ok = true;
            int issued_q = 0, issued_k = 0, issued_v = 0;
            // Waits until slot `x` of `slots` is free again.
            auto slot_free = [&](uint64_t* empty, int x, int slots) {
                if (ok && x >= slots)
                    ok = mbar_wait_bounded(&empty[x % slots], ((x / slots) - 1) & 1u, abort_flag, &g_error_word, a.timeout_ns);
                return ok;
            };
            auto load_kv = [&](int g, int j) {
                if (!slot_free(k_empty, g, L::kKs)) return;
                const int sk = g % L::kKs, sv = g % L::kVs;
                mbar_arrive_expect_tx(&k_full[sk], L::kTile);
                for (int at = 0; at < D / 64; ++at)
                    tma_load_4d(smem + L::kK + sk * L::kTile + at * kBT * 128, &a.tmap_k, &k_full[sk], at * 64, j * kBT, kv_h, b);
                ++issued_k;
                if (!slot_free(v_empty, g, L::kVs)) return;
                mbar_arrive_expect_tx(&v_full[sv], L::kTile);
                for (int at = 0; at < D / 64; ++at)
                    tma_load_4d(smem + L::kV + sv * L::kTile + at * kBT * 128, &a.tmap_v, &v_full[sv], at * 64, j * kBT, kv_h, b);
                ++issued_v;
            };
            for (int it = 0; it < n && ok; ++it) {
                if (!ONE || it == 0) load_kv(it * nk, 0);
                if (!slot_free(q_empty, it, L::kQs)) break;
                const QueryBox q = query_box(a, kvh, u0 + it);
                const int s = it % L::kQs;
                uint8_t* st = smem + L::kQ + s * 2 * L::kTile;
                mbar_arrive_expect_tx(&q_full[s], q_bytes);
                for (int at = 0; at < D / 64; ++at) {
                    tma_load_4d(st + at * kBT * 128, &a.tmap_q, &q_full[s], at * 64, q.i, q.h, b);
                    tma_load_4d(st + L::kTile + at * kBT * 128, &a.tmap_do, &q_full[s], at * 64, q.i, q.h, b);
                }
                ++issued_q;
                if (L::kQs == 1 && it + 1 < n) {  // the next tile's rows, on their way to L2
                    const QueryBox x = query_box(a, kvh, u0 + it + 1);
                    for (int at = 0; at < D / 64; ++at) {
                        tma_prefetch_4d(&a.tmap_q, at * 64, x.i, x.h, b);
                        tma_prefetch_4d(&a.tmap_do, at * 64, x.i, x.h, b);
                    }
                }
                for (int j = 1; j < nk && ok; ++j) load_kv(it * nk + j, j);
            }
            if (!ok) {
                // Let the copies already started land before the CTA leaves.
                auto land = [&](uint64_t* full, int issued, int slots) {
                    for (int i = max(0, issued - slots); i < issued; ++i)
                        mbar_wait_bounded(&full[i % slots], (i / slots) & 1u, nullptr, &g_error_word, a.timeout_ns);
                };
                land(q_full, issued_q, L::kQs);
                land(k_full, issued_k, L::kKs);
                land(v_full, issued_v, L::kVs);
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
        auto q_s = [&](int it) { return smem_u32(smem + L::kQ + it % L::kQs * 2 * L::kTile); };
        auto k_s = [&](int g) { return smem_u32(smem + L::kK + (ONE ? 0 : g % L::kKs) * L::kTile); };
        auto v_s = [&](int g) { return smem_u32(smem + L::kV + (ONE ? 0 : g % L::kVs) * L::kTile); };
        // dst = rows x cols^T, both K-major over D.
        auto scores = [&](uint32_t dst, uint32_t rows, uint32_t cols) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = ((kk / 4) * (kBT * 128) + (kk % 4) * 32) >> 4;
                mma_ss(dst, kmaj + (rows >> 4) + off, kmaj + (cols >> 4) + off, kIdescS, kk > 0 ? 1u : 0u);
            }
        };
        bool ok = true;
        // The helper's waits, for the (Q, dO) pair of key tile g where that is a query
        // tile's first, and for its K and V.
        auto wait = [&](uint64_t* full, int x, int slots) {
            if (!issuer && ok) ok = warp_wait(&full[x % slots], (x / slots) & 1u, abort_flag, a.timeout_ns);
        };
        auto wait_qk = [&](int g, int it, int j) {
            if (j == 0) wait(q_full, it, L::kQs);
            if (ONE && g > 0) return;
            wait(k_full, g, L::kKs);
            if (!issuer && ok) bwd_zero_tail<D>(smem + L::kK + g % L::kKs * L::kTile, keys - j * kBT);
        };
        auto wait_v = [&](int g, int j) {
            if (ONE && g > 0) return;
            wait(v_full, g, L::kVs);
            if (!issuer && ok) bwd_zero_tail<D>(smem + L::kV + g % L::kVs * L::kTile, keys - j * kBT);
        };
        auto issue_s = [&](int g, int it) { scores(t_s + 128u * static_cast<uint32_t>(g & 1), q_s(it), k_s(g)); };
        auto issue_dp = [&](int g, int it, int j) {
            scores(t_dp, q_s(it) + L::kTile, v_s(g));
            mma_commit(&s_full[g & 1]);
            if (!ONE) mma_commit(&v_empty[g % L::kVs]);
            if (j + 1 == nk) mma_commit(&q_empty[it % L::kQs]);
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
        wait_qk(0, 0, 0);
        wait_v(0, 0);
        sync();
        issue([&] {
            issue_s(0, 0);
            issue_dp(0, 0, 0);
        });
        for (int g = 0, it = 0, j = 0; g < tiles; ++g) {
            const bool more = g + 1 < tiles, last = j + 1 == nk;  // a query tile's last key tile
            const int next_it = last ? it + 1 : it, next_j = last ? 0 : j + 1;
            // With one slot the next query tile's rows are still on their way: this
            // tile's product first.
            const bool late = L::kQs == 1 && last;
            if (more && !late) {
                wait_qk(g + 1, next_it, next_j);
                sync();
                issue([&] { issue_s(g + 1, next_it); });
            }
            take(kDpBar);
            if (more && !late) {
                if (!ONE) {
                    wait_v(g + 1, next_j);
                    sync();
                }
                issue([&] { issue_dp(g + 1, next_it, next_j); });
            }
            take(kPBar + (g & 1));
            issue([&] {  // dQ += dS K: 16-bit dS in the first 16 of each 32 columns of S
#pragma unroll
                for (int kk = 0; kk < kBT / 16; ++kk)
                    mma_ts(t_acc, t_s + 128u * static_cast<uint32_t>(g & 1) + (kk / 2) * 32 + (kk % 2) * 8,
                           mnmaj + (k_s(g) >> 4) + ((kk * 16 * 128) >> 4), kIdescAcc, j > 0 || kk > 0 ? 1u : 0u);
                if (!ONE) mma_commit(&k_empty[g % L::kKs]);
                if (last) mma_commit(acc_full);
            });
            if (more && late) {
                wait_qk(g + 1, next_it, next_j);
                wait_v(g + 1, next_j);
                sync();
                issue([&] {
                    issue_s(g + 1, next_it);
                    issue_dp(g + 1, next_it, next_j);
                });
            }
            it = next_it;
            j = next_j;
        }
        if (issuer) {
            if (elect_one_sync()) mma_commit(done);  // fires once every product above has completed
            __syncwarp();
        }
    } else {
        // Warps w and w+4 share TMEM lanes (a thread a query row) and split the columns.
        const int quarter = warp % 4, half = warp / 4, r = quarter * 32 + lane, c0 = half * 64;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        uint8_t* stage = smem + L::kRows + warp * 4096;
        const float* stats = a.ws + (static_cast<int64_t>(kvh) * a.tiles + u0) * (2 * kBT) + r;
        const GradScale held = grad_scale<BF16>(a, kvh);
        constexpr int kChunks = D / 64;  // of 32 columns in half a row
        uint32_t acc[kChunks][32];
        auto load_acc = [&]() {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) tmem_ld32(t_acc + lane_off + (half * kChunks + c) * 32, acc[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < kChunks; ++c) reg_fence(acc[c]);
        };
        auto store = [&](int it) {
            const QueryBox box = query_box(a, kvh, u0 + it);
            if (!L::kStaged) {  // a thread its half row
                int h, i;
                if (!query_row(a, box, r, h, i)) return;
                uint16_t* dst = static_cast<uint16_t*>(a.dq) + b * a.dq_bs + h * a.dq_hs + i * a.dq_ns + half * (D / 2);
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t y[4];
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            y[w] = pack16(__uint_as_float(acc[c][8 * e + 2 * w]) * held.mul,
                                          __uint_as_float(acc[c][8 * e + 2 * w + 1]) * held.mul, BF16);
                        *reinterpret_cast<uint4*>(dst + 32 * c + 8 * e) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                return;
            }
            __syncwarp();
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t y[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        y[w] = pack16(__uint_as_float(acc[c][8 * e + 2 * w]) * held.mul,
                                      __uint_as_float(acc[c][8 * e + 2 * w + 1]) * held.mul, BF16);
                    *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * c + e) ^ (lane & 7)) << 4)) =
                        make_uint4(y[0], y[1], y[2], y[3]);
                }
            __syncwarp();
            constexpr int kPieces = D / 16;  // of 16 bytes in half a row
            uint16_t* base = static_cast<uint16_t*>(a.dq) + b * a.dq_bs + half * (D / 2) + 8 * (lane % kPieces);
#pragma unroll
            for (int e = 0; e < kPieces; ++e) {
                const int rr = e * (32 / kPieces) + lane / kPieces;
                const uint4 y = *reinterpret_cast<const uint4*>(stage + rr * 128 + (((lane % kPieces) ^ (rr & 7)) << 4));
                int h, i;
                if (query_row(a, box, quarter * 32 + rr, h, i))
                    *reinterpret_cast<uint4*>(base + h * a.dq_hs + i * a.dq_ns) = y;
            }
        };
        bool ok = true;
        int failed_at = 0;  // first tile not handed over when a wait gave up
        float nlse2 = __ldcg(stats), ndelta = __ldcg(stats + kBT);  // -LSE*log2(e) (past Nq: -inf) and -Delta of this row
        float nlse2_next = 0.f, ndelta_next = 0.f;
        for (int g = 0, it = 0, j = 0; g < tiles && ok; ++g) {
            if (j == 0 && it + 1 < n) {
                nlse2_next = __ldcg(stats + (it + 1) * (2 * kBT));
                ndelta_next = __ldcg(stats + (it + 1) * (2 * kBT) + kBT);
            }
            ok = warp_wait(&s_full[g & 1], (g >> 1) & 1u, abort_flag, a.timeout_ns);
            if (!ok) {
                failed_at = g;
                break;
            }
            tc_fence_after();
            const uint32_t sb = t_s + 128u * static_cast<uint32_t>(g & 1) + lane_off + c0;
            uint32_t dpv[2][32], sv[32];
            tmem_ld32(t_dp + lane_off + c0, dpv[0]);
            tmem_ld32(t_dp + lane_off + c0 + 32, dpv[1]);
            tmem_ld32(sb, sv);
            tmem_wait_ld();
            reg_fence(dpv[0]);
            reg_fence(dpv[1]);
            reg_fence(sv);
            tc_fence_before();
            __syncwarp();
            named_barrier_arrive(kDpBar, kEwThreads);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (c == 1) {
                    tmem_ld32(sb + 32, sv);
                    tmem_wait_ld();
                    reg_fence(sv);
                }
                const int vis = keys - j * kBT - (c0 + c * 32);
                uint32_t dsk[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float x0, x1, d0, d1;
                    fma2(x0, x1, __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]), a.sl2, a.sl2, nlse2, nlse2);
                    float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                    if (vis < 32) {
                        if (e >= vis) p0 = 0.f;
                        if (e + 1 >= vis) p1 = 0.f;
                    }
                    minus_delta<!BF16>(d0, d1, dpv[c][e], dpv[c][e + 1], held.f, ndelta, ndelta);
                    mul2(d0, d1, p0, p1, d0, d1);
                    dsk[e / 2] = pack16(d0, d1, BF16);
                }
                tmem_st16(sb + c * 32, dsk);  // columns of this chunk, already read
            }
            tmem_wait_st();
            const bool last_dq = j == 0 && it > 0;
            if (last_dq) {  // the last query tile's dQ, before the issuing warp may overwrite it
                ok = warp_wait(acc_full, (it - 1) & 1u, abort_flag, a.timeout_ns);
                tc_fence_after();
                load_acc();
            }
            tc_fence_before();
            __syncwarp();
            named_barrier_arrive(kPBar + (g & 1), kEwThreads);
            if (!ok) failed_at = g + 1;  // every barrier of this tile was met
            if (ok && last_dq) store(it - 1);
            if (++j == nk) {
                j = 0;
                ++it;
                nlse2 = nlse2_next;
                ndelta = ndelta_next;
            }
        }
        if (!ok)  // meet the issuing warp, which runs its schedule to the end
            for (int g = failed_at; g < tiles; ++g) {
                __syncwarp();
                named_barrier_arrive(kDpBar, kEwThreads);
                named_barrier_arrive(kPBar + (g & 1), kEwThreads);
            }
        const bool fin = warp_wait(done, 0u, nullptr, a.timeout_ns);
        tc_fence_after();
        if (ok && fin) {
            load_acc();
            store(n - 1);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    wait_key_kernel();
}

}  // namespace
}  // namespace fattn
