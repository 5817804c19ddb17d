// internal.h -- declarations shared by the translation units of libfattn.
// Not part of the public ABI (see include/fattn.h).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fattn {

constexpr int kMaxDevices = 64;
constexpr float kLeastFactor = 1.2e-38f;  // a score factor of 0 becomes this: a masked score stays -inf times it

// Raises one kernel's dynamic shared-memory limit once per device.  Each call
// site passes its own flag array; the flags are atomics, so host threads that
// launch at the same time never race on them (setting the attribute twice is
// harmless).
template <typename K>
inline cudaError_t opt_in_smem_once(K* fn, int bytes, std::atomic<bool> (&done)[kMaxDevices]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kMaxDevices;
    if (known && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (known) done[dev].store(true, std::memory_order_release);
    return cudaSuccess;
}

// Launches a kernel whose start may overlap the end of the kernel before it on
// the stream (programmatic stream serialization): it calls grid_dependency()
// before it touches memory, which waits for that kernel to complete.
//
// Three kernels wait only at their end: the prefix's rows (fwd_rows.cu, own_part) and
// the dQ kernels of cross attention (attn_bwd_kernel and cross_dq_kernel), which run
// beside the kernel before them, K.  They read nothing that K writes and write nothing
// that K touches.  What they read, kernels before K wrote: every CTA of K passes its
// grid_dependency(), behind the end of those, before the first CTA here starts, so
// their writes have reached L2 by then.  But no wait of this grid's own has dropped
// what an SM's L1 may hold: all such reads, plain loads of tables, lengths and
// statistics, go to L2 (__ldcg), as TMA copies do.
template <typename A>
inline cudaError_t launch_overlapped(void (*fn)(A), unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                                     const A& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, a);
    if (e != cudaSuccess) (void)cudaGetLastError();  // reported here, not left for the caller's next check
    return e;
}
#ifdef __CUDACC__
// Every thread of a kernel launched so calls this first.  (The next kernel may
// be set up as soon as every CTA of this one has come here; it waits likewise.)
__device__ __forceinline__ void grid_dependency() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

// ---- tensor-core path (bf16 / fp16), fwd_tc.cu ------------------------------
constexpr int kTcBM = 128;        // Q rows per MMA tile (tcgen05 M)
constexpr int kTcQTiles = 2;      // Q tiles per task (rows per task = 256)
constexpr int kTcBN = 128;        // keys per K/V tile (N of S = Q K^T)
constexpr int kTcThreads = 384;   // 2 softmax warpgroups + 1 control warpgroup (MMA, TMA)

struct TcArgs {
    CUtensorMap tmap_q;  // 3-D {D, N, B*H}, box {64, 128, 1}, 128-byte swizzle
    CUtensorMap tmap_k;
    CUtensorMap tmap_v;
    void* o;             // [B,H,N,D] output, input dtype
    float* lse;          // [B,H,N] or nullptr
    int N;
    int BH;              // B * H query heads (task space)
    int H;               // query heads per batch
    int Hkv;             // key/value heads per batch (H % Hkv == 0)
    int num_qblk;        // ceil(N / 256)
    int num_tasks;       // BH * num_qblk
    int head_group;      // causal task order: query heads per group (K/V of a group stays in L2)
    float scale_log2;    // scale * log2(e)
    uint64_t timeout_ns; // bound of every barrier wait
};

int tc_smem_bytes(int D);
int tc_num_stages(int D);
// Encodes the three tensor maps of `a` for these buffers (host).
cudaError_t tc_encode_maps(TcArgs& a, const void* q, const void* k, const void* v, int64_t BH,
                           int64_t BHkv, int64_t N, int64_t D, bool bf16);
cudaError_t tc_launch(const TcArgs& a, int D, bool bf16, bool causal, int grid,
                      cudaStream_t stream);

// ---- packed sequences on the tensor-core path, fwd_packed.cu -------------------
struct PackedPlan {  // in the caller's workspace
    int blocks;
    int pad[3];
    int4 list[1];    // [blocks]: first token and length of the sequence, Q block within it
};
struct PackedArgs : TcArgs {  // tmaps {D, T, heads}; N, BH, num_qblk and num_tasks are unused
    PackedPlan* plan;    // the workspace
    int plan_stride;     // few blocks: each CTA has a list of its own, so many bytes apart (else 0)
    const int32_t* cu;   // [B + 1]
    int B;
    int64_t T;
    int64_t o_ts;        // token and head stride of o, elements
    int64_t o_hs;
};
constexpr int kSmallPlan = 64;       // Q blocks that a CTA lists for itself
constexpr int kSmallPlanCtas = 160;  // lists of their own in the workspace
constexpr int kSmallPlanBytes = 16 * (1 + kSmallPlan);
cudaError_t packed_launch(const PackedArgs& a, int D, bool bf16, bool causal, int capacity, int grid, cudaStream_t s);
cudaError_t packed_read_and_clear_error_word(uint32_t* out);

// ---- rows over keys of a length of their own, on the tensor-core path -------------
// (fwd_rows.cu: cross attention, and the prefix that a batch shares)
struct RowsArgs : TcArgs {  // N, BH, num_qblk, num_tasks and head_group are unused
    // tmap_q: {D, Nq, H, B}, box {64, box_i, box_h, box_b}, a tile's rows in that
    // order (at most 128).  tmap_k, tmap_v: {D, keys, Hkv, sources}, or {D,
    // page_size, Hkv, pages} with a table; box {64, piece, 1, 1}.
    int64_t o_bs, o_hs, o_ns;  // batch, head and token stride of o, elements
    const int32_t* lens;       // keys of each source, or nullptr: max_keys
    const int32_t* table;      // pages of the one source's keys, or nullptr
    float* part_o;             // fp32 [sources][Hkv][tiles][128][part_pitch][D], or nullptr: O and LSE are written
    float2* part_ml;           // .. [part_pitch]: max (log2 units) and sum of the weights
    int32_t* part_count;       // receives the K/V tiles of a part, which the launch chooses
    int part_pitch;            // parts that the workspace has room for
    int max_parts;             // of those, the ones that the keys may be cut into
    int own_part;              // 1: the last part of the workspace is joined too
    int num_pages;
    int page_size;
    int piece;                 // keys of a copy
    int max_keys;
    int sources;               // batch entries with keys of their own, or 1
    int B;
    int Nq;
    int share;                 // query heads of a K/V head
    int box_i, box_h, box_b;   // tokens, heads, batch entries of a tile
    uint32_t box_bytes;        // of the tile's 64-element columns
    int n_i, n_h;              // tiles along tokens and heads
    int tiles;                 // tiles of a K/V head of a source
    int pairs;                 // ceil(tiles / 2)
};
constexpr int kMaxSplits = 128;
constexpr int kSplitCtas = 152;  // CTAs that workspaces are sized for
// Parts that `targets` tasks may be cut into: two waves of tasks.
inline int max_splits(int64_t targets) {
    const int64_t n = 2 * kSplitCtas / (targets > 0 ? targets : 1);
    return static_cast<int>(n < 1 ? 1 : (n > kMaxSplits ? kMaxSplits : n));
}
cudaError_t rows_launch(const RowsArgs& a, int D, bool bf16, int grid, cudaStream_t s);
cudaError_t rows_join_launch(const RowsArgs& a, int D, bool bf16, cudaStream_t s);
cudaError_t rows_read_and_clear_error_word(uint32_t* out);

// ---- CUDA-core path (fp32), fwd_ffma.cu --------------------------------------
constexpr int kFfmaBr = 128;      // Q rows per CTA
int ffma_bc(int D);               // keys per K/V tile
int ffma_threads(int D);          // threads per CTA
int ffma_smem_bytes(int D);
cudaError_t ffma_launch(const float* q, const float* k, const float* v, float* o, float* lse,
                        int64_t BH, int64_t H, int64_t Hkv, int64_t N, int64_t D,
                        float scale_log2, bool causal, cudaStream_t stream);
// One query row per thread (Br = 128 threads), the page's own design.
int ffma_row_bc(int D);
int ffma_row_smem_bytes(int D);
cudaError_t ffma_row_launch(const float* q, const float* k, const float* v, float* o, float* lse,
                            int64_t BH, int64_t H, int64_t Hkv, int64_t N, int64_t D,
                            float scale_log2, bool causal, cudaStream_t stream);

// ---- unfused comparator (bf16 / fp16), fwd_unfused.cu ----------------------
struct UnfusedArgs {
    CUtensorMap tmap_q;  // as TcArgs: 3-D {D, N, heads}, box {64, 128, 1}, 128-byte swizzle
    CUtensorMap tmap_k;
    CUtensorMap tmap_v;
    CUtensorMap tmap_p;  // 3-D {Np, N, B*H} over the P part of the workspace, same box
    float* s;            // workspace: S fp32 [B*H][N][Np]
    void* p;             // workspace: P 16-bit [B*H][N][Np]
    void* o;             // [B,H,N,D] output, input dtype
    float* lse;          // [B,H,N] or nullptr
    int N;
    int Np;              // row pitch of S and P in elements (N rounded up to 8)
    int BH;
    int H;
    int Hkv;
    float scale;         // natural-log units (S = scale Q K^T)
    uint64_t timeout_ns;
};

int64_t unfused_row_pitch(int64_t N);
size_t unfused_workspace_bytes(int64_t BH, int64_t N);
cudaError_t unfused_encode_p_map(UnfusedArgs& a, int64_t BH, int64_t N, bool bf16);
cudaError_t unfused_launch(const UnfusedArgs& a, int D, bool bf16, bool causal, cudaStream_t s);
cudaError_t unfused_read_and_clear_error_word(uint32_t* out);
// Device address of the fixed workspace of fattn_fwd_unfused_static on the
// current device (looked up once per device).
constexpr size_t kUnfusedStaticBytes = size_t(64) << 20;
cudaError_t unfused_static_scratch(void** ptr);

// ---- backward (bf16 / fp16), bwd_tc.cu --------------------------------------
struct BwdArgs {
    CUtensorMap tmap_q;   // 3-D {D, N, B*H}, box {64, 128, 1}, 128-byte swizzle
    CUtensorMap tmap_k;
    CUtensorMap tmap_v;
    CUtensorMap tmap_do;
    float* ws;            // [B*H][2][Npad]: LSE*log2(e) (+inf past N), Delta (0 past N)
    void* dq;             // [B,H,N,D] outputs, input dtype
    void* dk;
    void* dv;
    int N;
    int Npad;             // N rounded up to 128
    int BH;               // B * H query heads
    int H;                // query heads per batch
    int Hkv;              // key/value heads per batch (H % Hkv == 0)
    int BHkv;             // B * Hkv
    int num_tiles;        // Npad / 128
    float sl2;            // scale * log2(e)
    float scale;
    uint64_t timeout_ns;
};

int64_t bwd_padded_rows(int64_t N);
cudaError_t bwd_launch(const BwdArgs& a, const void* o, const void* dout, const float* lse, int D,
                       bool bf16, bool causal, cudaStream_t s);
cudaError_t bwd_read_and_clear_error_word(uint32_t* out);

// Keys past which an fp16 dS is held by a power of two of the data (grad_scale,
// bwd_tc_kernel.cuh): up to there weights of 1 / Nk are normal numbers of the type.
constexpr int64_t kLongKeys = 1 << 14;
struct CrossBwdArgs : BwdArgs {
    // tmaps {D, Nq or Nk, heads, B}, boxes {64, box_i, box_h, 1} of q and dO, {64, 128,
    // 1, 1} of k and v; N = Nq; Npad and num_tiles are unused; ws [B*Hkv][tiles][2][128]
    int box_i, box_h;          // tokens and heads of a tile of query rows (box_h divides H/Hkv)
    int n_i;                   // tiles along tokens
    int tiles;                 // tiles of a K/V head: n_i * (H/Hkv) / box_h
    int Nk;
    int tiles_k;               // ceil(Nk / 128)
    int chunks_k;              // CTAs that share a K/V head's key blocks, where tiles = 1
    int chunks_q;              // CTAs that share a K/V head's query tiles, where parts_q = 1
    int parts_k, parts_q;      // parts that the inner tiles of a key block / a query tile are cut into
    float* part_kv;            // fp32 [parts_k][B*Hkv][tiles_k * 128][dv, dk][D], where parts_k > 1
    float* part_q;             // fp32 [parts_q][B*Hkv][tiles * 128][D], where parts_q > 1
    const int32_t* lens;       // visible keys of each batch entry, or nullptr: Nk
    int64_t dq_bs, dq_hs, dq_ns, dk_bs, dk_hs, dk_ns, dv_bs, dv_hs, dv_ns;  // element strides
    float2* most;              // fp16 and long keys: [B*Hkv] largest |dO_i|^2 and |v_j|^2 (seen keys); or nullptr
    const void* v;             // .. whose values are read for that
    int64_t v_bs, v_hs, v_ns;
    const void* o;             // the row statistics' inputs, by strides
    const void* dout;
    const float* lse;
    int64_t o_bs, o_hs, o_ns, do_bs, do_hs, do_ns;
};
cudaError_t bwd_cross_launch(const CrossBwdArgs& a, int D, bool bf16, int sms, cudaStream_t s);
cudaError_t bwd_cross_read_and_clear_error_word(uint32_t* out);

// ---- rotation by positions with several axes, rotate.cu ----------------------------
constexpr int kMaxAxes = 8;
struct RotateArgs {
    void* x[2];            // q and k [B][heads][N][D] by strides (k: or nullptr)
    void* y[2];
    int64_t x_bs[2], x_hs[2], x_ns[2], y_bs[2], y_hs[2], y_ns[2];
    int heads[2];
    const int32_t* pos;    // [axes][B][N]
    const float* cos;      // [max_pos][rot/2]
    const float* sin;
    int64_t max_pos;
    int64_t tokens;        // B * N
    int N;
    int rot;
    int interleaved;
    int inverse;
    int axes;
    alignas(8) uint8_t axis[64];  // of each pair
};
cudaError_t rotate_launch(const RotateArgs& a, int D, bool bf16, int sms, cudaStream_t s);
cudaError_t rotate_read_and_clear_error_word(uint32_t* out);

// ---- paged cache: append (cache_append.cu) and attention (decode.cu) --------
constexpr uint32_t kDevErrInvalidArg = 1u;  // error-word bit: an index in device memory is out of range
constexpr int kKv4Group = 32;               // elements of a 4-bit row that share one scale and zero

struct AppendArgs {
    const void* q;        // [T][H][D] by strides, or nullptr
    const void* k;        // [T][Hkv][D] by strides
    const void* v;
    void* q_out;          // or nullptr
    void* k_out;
    void* v_out;
    uint32_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;        // token and head strides, elements
    uint32_t qo_ts, qo_hs, ko_ts, ko_hs, vo_ts, vo_hs;
    void* k_pages;        // 16-bit [pages][Hkv][page_size][D], or codes [pages][Hkv][page_size][D/2] bytes
    void* v_pages;
    void* k_scales;       // 4-bit: fp16 [pages][Hkv][page_size][D/32][2]
    void* v_scales;
    int64_t page_stride;  // 16-bit: elements from one page to the next
    const int64_t* slots; // [T]
    const int32_t* pos;   // [T]
    const float* cos;     // [max_pos][rot/2]
    const float* sin;
    int64_t T;
    int64_t num_slots;    // num_pages * page_size
    int64_t max_pos;
    int page_size;
    int H;                // 0 when q is nullptr
    int Hkv;
    int rot;
    int interleaved;
    int held;             // 4-bit: k_out / v_out receive the values that the cache stands for
    uint32_t kv_blocks;   // blocks of key and value rows, tokens of a block (set by append_launch)
    uint32_t kv_tokens;
    uint32_t q_tokens;
    int apart;            // 4-bit: key rows and value rows have blocks of their own; likewise
    int axes;             // 0: pos is [T]; else [axes][T], and pair i turns by the position on axis[i]
    uint8_t axis[64];
};
cudaError_t append_launch(AppendArgs a, int D, bool bf16, bool kv4, int sms, cudaStream_t s);
cudaError_t append_read_and_clear_error_word(uint32_t* out);

struct DecodeArgs {
    const void* q;        // [B][H][Nq][D] by strides
    void* o;
    float* lse;           // [B][H][Nq] or nullptr
    int64_t q_bs, q_hs, q_ns, o_bs, o_hs, o_ns;  // element strides
    const void* k_pages;  // as AppendArgs
    const void* v_pages;
    const void* k_scales;
    const void* v_scales;
    int64_t page_stride;
    const int32_t* block_table;  // [B][table_width]
    const int32_t* seq_lens;     // [B]
    void* workspace;
    int64_t num_pages;
    int64_t table_width;
    int page_size;
    int B;
    int H;
    int Hkv;
    int Nq;
    float scale_log2;
};
struct SharedDecodeArgs : DecodeArgs {  // the parts, as RowsArgs has them (one source); the last is the own keys'
    float* part_o;
    float2* part_ml;
    int part_pitch;
    int box_i, box_h, box_b, n_i, n_h, tiles;
};
struct PrefixDecodeArgs : DecodeArgs {
    const int32_t* prefix_table;  // [prefix_max / page_size]
    const int32_t* prefix_len;    // [1]
    int prefix_max;
};
cudaError_t decode_prefix_launch(const PrefixDecodeArgs& a, int D, bool bf16, int sms, cudaStream_t s);
struct CrossDecodeArgs : DecodeArgs {  // k_pages and v_pages: [B][Nk][Hkv][D] by strides; seq_lens may be nullptr
    int64_t k_bs, k_hs, k_ns, v_bs, v_hs, v_ns;
    int Nk;
};
cudaError_t decode_shared_launch(const SharedDecodeArgs& a, int D, bool bf16, int sms, cudaStream_t s);
cudaError_t decode_shared_read_and_clear_error_word(uint32_t* out);
cudaError_t decode_cross_launch(const CrossDecodeArgs& a, int D, bool bf16, int sms, cudaStream_t s);
cudaError_t decode_cross_read_and_clear_error_word(uint32_t* out);
cudaError_t decode_launch(const DecodeArgs& a, int D, bool bf16, bool kv4, int sms, cudaStream_t s);
int64_t decode_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t Nq, int64_t D);
cudaError_t decode_read_and_clear_error_word(uint32_t* out);

// Key/value head read by query head bh = b*H + h: b*Hkv + h / (H/Hkv).
__host__ __device__ __forceinline__ int kv_head_of(int bh, int H, int Hkv) {
    return (bh / H) * Hkv + (bh % H) / (H / Hkv);
}

// ---- device error word (fwd_tc.cu) -----------------------------------------
cudaError_t read_and_clear_error_word(uint32_t* out);
cudaError_t launch_wait_selftest(uint64_t timeout_ns, cudaStream_t stream);

}  // namespace fattn
