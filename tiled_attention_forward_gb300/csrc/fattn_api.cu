// fattn_api.cu -- the C ABI of libfattn (declared in include/fattn.h):
// argument validation, launch planning, TMA tensor-map encoding and dispatch
// to the tensor-core (bf16/fp16) or CUDA-core (fp32) kernel.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <utility>
#include <cudaTypedefs.h>

#include "fattn.h"
#include "internal.h"

namespace fattn {
namespace {

constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;  // 2 s per barrier wait
constexpr int64_t kMaxElements = int64_t(1) << 52;      // bound of B*H*N*D accepted by validate()

// The fixed array behind fattn_fwd_unfused_static and the size the header
// promises are one number.
static_assert(static_cast<long long>(kUnfusedStaticBytes) == FATTN_UNFUSED_STATIC_BYTES,
              "static workspace size must match the public header");
constexpr float kLog2e = 1.4426950408889634f;

// The tensor-core forward sets masked scores to -inf and multiplies by the scale
// afterwards, where -inf * 0 would be NaN: a scale of 0, or one that underflows,
// is raised to about the smallest normal number, beside which no score differs from 0.
float score_factor(float scale) { return std::max(scale * kLog2e, kLeastFactor); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0u; }

size_t elem_bytes(int dtype) { return dtype == FATTN_F32 ? 4u : 2u; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Validation shared by every compute entry point; returns FATTN_OK when the
// call may proceed (which includes the empty problem, flagged by *empty).
int validate(const void* q, const void* k, const void* v, const void* o, const float* lse,
             int64_t B, int64_t H, int64_t Hkv, int64_t N, int64_t D, float scale, int dtype,
             bool* empty) {
    *empty = false;
    if (dtype != FATTN_F32 && dtype != FATTN_F16 && dtype != FATTN_BF16) return FATTN_ERR_INVALID_ARG;
    if (B < 0 || H < 0 || N < 0 || D < 0) return FATTN_ERR_INVALID_ARG;
    if (H > 0 && (Hkv <= 0 || H % Hkv != 0)) return FATTN_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || scale < 0.f) return FATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return FATTN_ERR_UNSUPPORTED;
    if (B == 0 || H == 0 || N == 0) {
        *empty = true;
        return FATTN_OK;
    }
    // Index ranges: N and B*H fit int32 (kernel indices, TMA coordinates,
    // grid.y <= 65535 on the FFMA path), and B*H*N*D is bounded by 2^52
    // elements, so that every byte count formed below stays far inside int64
    // (no device holds a problem anywhere near that size).
    if (N > (int64_t(1) << 30) || B > (int64_t(1) << 30) || H > (int64_t(1) << 30))
        return FATTN_ERR_UNSUPPORTED;
    const int64_t BH = B * H;
    if (BH > (int64_t(1) << 30)) return FATTN_ERR_UNSUPPORTED;
    if (BH * N > kMaxElements / D) return FATTN_ERR_UNSUPPORTED;  // BH*N <= 2^60: no overflow
    if (dtype == FATTN_F32 && BH > 65535) return FATTN_ERR_UNSUPPORTED;
    if (!q || !k || !v || !o) return FATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return FATTN_ERR_MISALIGNED;
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return FATTN_ERR_MISALIGNED;
    const size_t bytes = static_cast<size_t>(BH * N * D) * elem_bytes(dtype);
    const size_t kvbytes = static_cast<size_t>(B * Hkv * N * D) * elem_bytes(dtype);
    if (overlaps(o, bytes, q, bytes) || overlaps(o, bytes, k, kvbytes) ||
        overlaps(o, bytes, v, kvbytes))
        return FATTN_ERR_INVALID_ARG;
    if (lse) {
        const size_t lb = static_cast<size_t>(BH * N) * sizeof(float);
        if (overlaps(lse, lb, o, bytes) || overlaps(lse, lb, q, bytes) ||
            overlaps(lse, lb, k, kvbytes) || overlaps(lse, lb, v, kvbytes))
            return FATTN_ERR_INVALID_ARG;
    }
    return FATTN_OK;
}

int current_sm_count(int* sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FATTN_ERR_NO_DEVICE;
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return FATTN_ERR_NO_DEVICE;
    if (major != 10 || minor != 3) return FATTN_ERR_NO_DEVICE;  // built for sm_103a only
    return FATTN_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A set of equal intervals of bytes, `outer` apart: the rows of a strided
// tensor, or the pages of a pool.  `inner` is the extent of one interval.
struct View {
    uintptr_t p = 0;
    uintptr_t total = 0;  // first byte to past the last one; 0: empty
    uintptr_t outer = 0;
    uintptr_t inner = 0;
};

// 16-bit rows of D elements at strides (s0, s1), n0 x n1 of them.
View rows_view(const void* p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t D) {
    View v;
    if (!p || n0 <= 0 || n1 <= 0) return v;
    v.p = reinterpret_cast<uintptr_t>(p);
    const bool first_outer = s0 >= s1;
    const int64_t no = first_outer ? n0 : n1, so = first_outer ? s0 : s1;
    const int64_t ni = first_outer ? n1 : n0, si = first_outer ? s1 : s0;
    v.inner = static_cast<uintptr_t>(2 * ((ni - 1) * si + D));
    v.outer = static_cast<uintptr_t>(2 * so);
    v.total = static_cast<uintptr_t>(2 * (no - 1) * so) + v.inner;
    return v;
}

View dense_view(const void* p, int64_t bytes) {
    View v;
    if (!p || bytes <= 0) return v;
    v.p = reinterpret_cast<uintptr_t>(p);
    v.total = v.inner = v.outer = static_cast<uintptr_t>(bytes);
    return v;
}

// Whether two views share a byte.  Views with one outer stride whose intervals
// fit into it (slices of one tensor) are compared modulo that stride; all
// others by their whole ranges.
bool views_overlap(const View& a, const View& b) {
    if (a.total == 0 || b.total == 0) return false;
    if (!(a.p < b.p + b.total && b.p < a.p + a.total)) return false;
    if (a.outer == b.outer && a.inner <= a.outer && b.inner <= b.outer) {
        const uintptr_t m = a.outer;
        const uintptr_t d = (b.p >= a.p) ? (b.p - a.p) % m : (m - (a.p - b.p) % m) % m;  // b's place in a's period
        return d < a.inner || d + b.inner > m;
    }
    return true;
}

// 16-bit rows of D elements at three strides, in bytes; s ascending, dimensions
// of one element left out (n = 1, s = 0).
struct Rows3 {
    uintptr_t p, row;
    uintptr_t n[3], s[3];
    uintptr_t below(uintptr_t m) const {  // extent of what is stepped by less than m
        uintptr_t x = row;
        for (int i = 0; i < 3; ++i)
            if (s[i] < m) x += (n[i] - 1) * s[i];
        return x;
    }
};

Rows3 rows3(const void* p, const int64_t (&n)[3], const int64_t* s, int64_t D) {
    Rows3 r = {reinterpret_cast<uintptr_t>(p), static_cast<uintptr_t>(2 * D), {}, {}};
    for (int i = 0; i < 3; ++i) {
        r.n[i] = static_cast<uintptr_t>(n[i]);
        r.s[i] = n[i] > 1 ? static_cast<uintptr_t>(2 * s[i]) : 0;
    }
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (r.s[j] > r.s[j + 1]) {
                std::swap(r.s[j], r.s[j + 1]);
                std::swap(r.n[j], r.n[j + 1]);
            }
    return r;
}

// Whether two sets of rows share a byte: their whole ranges do, and so do they
// modulo each stride m of one whose multiples all larger strides of both are
// (slices of one tensor lie apart within such a period).
bool rows3_overlap(const Rows3& a, const Rows3& b) {
    const uintptr_t all = UINTPTR_MAX;
    if (!(a.p < b.p + b.below(all) && b.p < a.p + a.below(all))) return false;
    for (int level = 0; level < 6; ++level) {
        const uintptr_t m = level < 3 ? a.s[level] : b.s[level - 3];
        if (m == 0) continue;
        bool whole = true;
        for (int i = 0; i < 3; ++i)
            whole = whole && (a.s[i] < m || a.s[i] % m == 0) && (b.s[i] < m || b.s[i] % m == 0);
        const uintptr_t na = a.below(m), nb = b.below(m);
        if (!whole || na > m || nb > m) continue;
        const uintptr_t d = b.p >= a.p ? (b.p - a.p) % m : (m - (a.p - b.p) % m) % m;  // b's place in a's period
        if (d >= na && d + nb <= m) return false;
    }
    return true;
}

bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s <= kMaxElements; }

// Sizes of a paged cache and of its rows.
int validate_cache(int64_t num_pages, int64_t page_size, int64_t Hkv, int64_t D, int dtype) {
    if (dtype != FATTN_F32 && dtype != FATTN_F16 && dtype != FATTN_BF16) return FATTN_ERR_INVALID_ARG;
    if (Hkv <= 0 || num_pages < 0 || page_size <= 0 || D < 0) return FATTN_ERR_INVALID_ARG;
    if (dtype == FATTN_F32 || (D != 64 && D != 128)) return FATTN_ERR_UNSUPPORTED;
    if (page_size % 16 != 0 || page_size > 65536) return FATTN_ERR_UNSUPPORTED;
    if (num_pages > 0x7fffffffll || Hkv > (int64_t(1) << 16) || Hkv * page_size > (int64_t(1) << 30) ||
        num_pages * page_size > kMaxElements / (Hkv * D))
        return FATTN_ERR_UNSUPPORTED;
    return FATTN_OK;
}

// K/V tiles one task visits: Q rows [r0, r0+rows) against keys, Bc-key tiles.
int64_t kv_tiles_for(int64_t r0, int64_t rows, int64_t N, int64_t bc, bool causal) {
    if (r0 >= N) return 0;
    const int64_t kv_limit = causal ? std::min(r0 + rows, N) : N;
    return ceil_div(kv_limit, bc);
}

PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn() {
    // Looked up once; a function-local static is initialised exactly once even
    // when several host threads make their first call at the same time.
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult qres;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &qres) == cudaSuccess &&
            qres == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
    }();
    return fn;
}

// Per-device helpers of fattn_fwd_host: a copy-in stream, a copy-out stream
// and the events that chain them to the caller's stream, created on the first
// call on the device and kept for the process lifetime.
constexpr int kHostChunks = 4;

struct HostPipe {
    cudaStream_t in = nullptr;
    cudaStream_t out = nullptr;
    cudaEvent_t fork = nullptr;
    cudaEvent_t join = nullptr;
    cudaEvent_t in_done[kHostChunks] = {};
    cudaEvent_t k_done[kHostChunks] = {};
    bool ready = false;
};

HostPipe g_host_pipes[kMaxDevices];
std::mutex g_host_mu;  // also serialises the enqueue sequence of fattn_fwd_host

cudaError_t host_pipe(HostPipe** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    HostPipe& p = g_host_pipes[dev];
    if (!p.ready) {
        const unsigned ev = cudaEventDisableTiming;
        if ((e = cudaStreamCreateWithFlags(&p.in, cudaStreamNonBlocking)) != cudaSuccess ||
            (e = cudaStreamCreateWithFlags(&p.out, cudaStreamNonBlocking)) != cudaSuccess ||
            (e = cudaEventCreateWithFlags(&p.fork, ev)) != cudaSuccess ||
            (e = cudaEventCreateWithFlags(&p.join, ev)) != cudaSuccess)
            return e;
        for (int c = 0; c < kHostChunks; ++c)
            if ((e = cudaEventCreateWithFlags(&p.in_done[c], ev)) != cudaSuccess ||
                (e = cudaEventCreateWithFlags(&p.k_done[c], ev)) != cudaSuccess)
                return e;
        p.ready = true;
    }
    *out = &p;
    return cudaSuccess;
}

// Causal task order: query heads per group.  A group's K/V (16-bit) is
// sized to stay in L2 while its tasks run (about 48 MB, so that the next
// group's first tasks fit beside the last ones of this group), whole K/V
// heads at a time (H / Hkv query heads share one), and the groups are made
// as equal as the head count allows.
int causal_head_group(int64_t BH, int64_t H, int64_t Hkv, int64_t N, int64_t D) {
    constexpr int64_t kL2Budget = 48ll << 20;
    const int64_t share = H / Hkv;
    const int64_t kv_bytes = 2 * N * D * 2;
    const int64_t kv_heads = std::max<int64_t>(1, kL2Budget / std::max<int64_t>(kv_bytes, 1));
    const int64_t cap = std::min<int64_t>(BH, kv_heads * share);
    const int64_t groups = ceil_div(BH, cap);
    int64_t hg = ceil_div(BH, groups);
    hg = ceil_div(hg, share) * share;  // whole K/V heads
    return static_cast<int>(std::min<int64_t>(hg, BH));
}

// One 16-bit tensor of T x heads rows at strides (ts, hs), as the map of
// tc_encode_maps with tokens in the place of rows.
cudaError_t packed_encode_map(CUtensorMap* map, const void* p, int64_t T, int64_t ts, int64_t heads, int64_t hs,
                              int64_t D, bool bf16) {
    auto encode = get_encode_fn();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(T), static_cast<cuuint64_t>(heads)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ts * 2), static_cast<cuuint64_t>(hs * 2)};
    const cuuint32_t box[3] = {64, 128, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                              const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t tc_encode_maps(TcArgs& a, const void* q, const void* k, const void* v, int64_t BH,
                           int64_t BHkv, int64_t N, int64_t D, bool bf16) {
    auto encode = get_encode_fn();
    if (!encode) return cudaErrorNotSupported;
    const CUtensorMapDataType dt =
        bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    // [heads][N][D] row-major, 16-bit: innermost D, then rows, then heads
    // (B*H heads for Q, B*Hkv for K and V).
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D * 2), static_cast<cuuint64_t>(N * D * 2)};
    const cuuint32_t box[3] = {64, 128, 1};  // one 128-byte swizzle atom wide, 128 rows
    const cuuint32_t estr[3] = {1, 1, 1};
    const void* ptrs[3] = {q, k, v};
    const int64_t heads[3] = {BH, BHkv, BHkv};
    CUtensorMap* maps[3] = {&a.tmap_q, &a.tmap_k, &a.tmap_v};
    for (int i = 0; i < 3; ++i) {
        const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(N),
                                    static_cast<cuuint64_t>(heads[i])};
        CUresult r = encode(maps[i], dt, 3, const_cast<void*>(ptrs[i]), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
    }
    return cudaSuccess;
}

cudaError_t unfused_encode_p_map(UnfusedArgs& a, int64_t BH, int64_t N, bool bf16) {
    auto encode = get_encode_fn();
    if (!encode) return cudaErrorNotSupported;
    const int64_t np = unfused_row_pitch(N);
    const CUtensorMapDataType dt =
        bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    // P: [B*H][N][Np] 16-bit; keys innermost, 64 keys (128 bytes) per box row
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(np), static_cast<cuuint64_t>(N),
                                static_cast<cuuint64_t>(BH)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(np * 2), static_cast<cuuint64_t>(N * np * 2)};
    const cuuint32_t box[3] = {64, 128, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = encode(&a.tmap_p, dt, 3, a.p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace fattn

using namespace fattn;

extern "C" {

int fattn_version(void) { return 10000; }

const char* fattn_status_string(int status) {
    switch (status) {
        case FATTN_OK: return "FATTN_OK";
        case FATTN_ERR_INVALID_ARG: return "FATTN_ERR_INVALID_ARG";
        case FATTN_ERR_UNSUPPORTED: return "FATTN_ERR_UNSUPPORTED";
        case FATTN_ERR_MISALIGNED: return "FATTN_ERR_MISALIGNED";
        case FATTN_ERR_CUDA: return "FATTN_ERR_CUDA";
        case FATTN_ERR_TIMEOUT: return "FATTN_ERR_TIMEOUT";
        case FATTN_ERR_NO_DEVICE: return "FATTN_ERR_NO_DEVICE";
        case FATTN_ERR_INTERNAL: return "FATTN_ERR_INTERNAL";
        default: return "FATTN_ERR_UNKNOWN";
    }
}

int fattn_plan_head_group(int64_t B, int64_t H, int64_t Hkv, int64_t N, int64_t D,
                          int64_t* head_group) {
    if (!head_group) return FATTN_ERR_INVALID_ARG;
    *head_group = 0;
    if (B < 1 || H < 1 || Hkv < 1 || N < 1 || (D != 64 && D != 128) || H % Hkv != 0)
        return FATTN_ERR_INVALID_ARG;
    if (N > (int64_t(1) << 30) || B > (int64_t(1) << 30) || H > (int64_t(1) << 30) ||
        B * H > (int64_t(1) << 30))
        return FATTN_ERR_UNSUPPORTED;
    *head_group = causal_head_group(B * H, H, Hkv, N, D);
    return FATTN_OK;
}

int fattn_plan(int64_t B, int64_t H, int64_t N, int64_t D, int causal, int dtype, int num_sms,
               int64_t out[9]) {
    if (!out) return FATTN_ERR_INVALID_ARG;
    for (int i = 0; i < 9; ++i) out[i] = 0;
    if (dtype != FATTN_F32 && dtype != FATTN_F16 && dtype != FATTN_BF16) return FATTN_ERR_INVALID_ARG;
    if (B < 0 || H < 0 || N < 0 || D < 0) return FATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return FATTN_ERR_UNSUPPORTED;
    if (B == 0 || H == 0 || N == 0) return FATTN_OK;
    if (N > (int64_t(1) << 30) || B > (int64_t(1) << 30) || H > (int64_t(1) << 30) ||
        B * H > (int64_t(1) << 30))
        return FATTN_ERR_UNSUPPORTED;
    const int64_t BH = B * H;
    const bool c = causal != 0;
    if (dtype == FATTN_F32) {
        const int64_t bc = ffma_bc(static_cast<int>(D));
        const int64_t nq = ceil_div(N, kFfmaBr);
        int64_t tiles = 0;
        for (int64_t qb = 0; qb < nq; ++qb) tiles += kv_tiles_for(qb * kFfmaBr, kFfmaBr, N, bc, c);
        out[0] = 1;
        out[1] = nq;
        out[2] = BH;
        out[3] = ffma_threads(static_cast<int>(D));
        out[4] = ffma_smem_bytes(static_cast<int>(D));
        out[5] = nq * BH;
        out[6] = tiles * BH;
        out[7] = kFfmaBr;
        out[8] = bc;
        return FATTN_OK;
    }
    if (num_sms <= 0) {
        int st = current_sm_count(&num_sms);
        if (st != FATTN_OK) return st;
    }
    const int64_t rows = int64_t(kTcBM) * kTcQTiles;
    const int64_t nq = ceil_div(N, rows);
    int64_t tiles = 0;
    for (int64_t qb = 0; qb < nq; ++qb) {
        const int64_t t0 = kv_tiles_for(qb * rows, kTcBM, N, kTcBN, c);
        const int64_t t1 = kv_tiles_for(qb * rows + kTcBM, kTcBM, N, kTcBN, c);
        tiles += std::max(t0, t1);  // the CTA streams each K/V tile once for both Q tiles
    }
    const int64_t tasks = nq * BH;
    out[0] = 2;
    out[1] = std::min<int64_t>(tasks, num_sms);
    out[2] = 1;
    out[3] = kTcThreads;
    out[4] = tc_smem_bytes(static_cast<int>(D));
    out[5] = tasks;
    out[6] = tiles * BH;
    out[7] = rows;
    out[8] = kTcBN;
    return FATTN_OK;
}

int fattn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t H,
              int64_t N, int64_t D, float scale, int causal, int dtype, fattn_stream_t stream_h) {
    return fattn_fwd_gqa(q, k, v, o, lse, B, H, H, N, D, scale, causal, dtype, stream_h);
}

int fattn_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B,
                  int64_t H, int64_t Hkv, int64_t N, int64_t D, float scale, int causal, int dtype,
                  fattn_stream_t stream_h) {
    bool empty = false;
    int st = validate(q, k, v, o, lse, B, H, Hkv, N, D, scale, dtype, &empty);
    if (st != FATTN_OK || empty) return st;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_h);
    const int64_t BH = B * H;

    if (dtype == FATTN_F32) {
        int sms = 0;
        st = current_sm_count(&sms);
        if (st != FATTN_OK) return st;
        cudaError_t e = ffma_launch(static_cast<const float*>(q), static_cast<const float*>(k),
                                    static_cast<const float*>(v), static_cast<float*>(o), lse, BH, H,
                                    Hkv, N, D, scale * kLog2e, causal != 0, stream);
        return e == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
    }

    // Task indices (256-row Q blocks x heads) are ints in the kernel.
    if (ceil_div(N, int64_t(kTcBM) * kTcQTiles) * BH > (int64_t(1) << 30)) return FATTN_ERR_UNSUPPORTED;
    int sms = 0;
    st = current_sm_count(&sms);
    if (st != FATTN_OK) return st;
    TcArgs a;
    std::memset(&a, 0, sizeof(a));
    const bool bf16 = dtype == FATTN_BF16;
    if (tc_encode_maps(a, q, k, v, BH, B * Hkv, N, D, bf16) != cudaSuccess) return FATTN_ERR_CUDA;
    a.o = o;
    a.lse = lse;
    a.N = static_cast<int>(N);
    a.BH = static_cast<int>(BH);
    a.H = static_cast<int>(H);
    a.Hkv = static_cast<int>(Hkv);
    a.num_qblk = static_cast<int>(ceil_div(N, int64_t(kTcBM) * kTcQTiles));
    a.num_tasks = a.num_qblk * a.BH;
    a.head_group = causal_head_group(BH, H, Hkv, N, D);
    a.scale_log2 = score_factor(scale);
    a.timeout_ns = kDefaultTimeoutNs;
    const int grid = static_cast<int>(std::min<int64_t>(a.num_tasks, sms));
    cudaError_t e = tc_launch(a, static_cast<int>(D), bf16, causal != 0, grid, stream);
    return e == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

int fattn_fwd_f32_rowwise(const float* q, const float* k, const float* v, float* o, float* lse,
                          int64_t B, int64_t H, int64_t N, int64_t D, float scale, int causal,
                          fattn_stream_t stream_h) {
    bool empty = false;
    int st = validate(q, k, v, o, lse, B, H, H, N, D, scale, FATTN_F32, &empty);
    if (st != FATTN_OK || empty) return st;
    int sms = 0;
    st = current_sm_count(&sms);
    if (st != FATTN_OK) return st;
    cudaError_t e = ffma_row_launch(q, k, v, o, lse, B * H, H, H, N, D, scale * kLog2e, causal != 0,
                                    reinterpret_cast<cudaStream_t>(stream_h));
    return e == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

int fattn_fwd_host(const void* q_host, const void* k_host, const void* v_host, void* o_host,
                   float* lse_host, void* q_dev, void* k_dev, void* v_dev, void* o_dev, float* lse_dev,
                   int64_t B, int64_t H, int64_t N, int64_t D, float scale, int causal, int dtype,
                   fattn_stream_t stream_h) {
    bool empty = false;
    int st = validate(q_dev, k_dev, v_dev, o_dev, lse_dev, B, H, H, N, D, scale, dtype, &empty);
    if (st != FATTN_OK || empty) return st;
    if (!q_host || !k_host || !v_host || !o_host) return FATTN_ERR_INVALID_ARG;
    int sms = 0;
    st = current_sm_count(&sms);
    if (st != FATTN_OK) return st;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_h);
    std::lock_guard<std::mutex> lock(g_host_mu);
    HostPipe* p = nullptr;
    if (host_pipe(&p) != cudaSuccess) return FATTN_ERR_CUDA;
    // Heads in up to kHostChunks groups: the copies of group c+1 run on the
    // copy-in stream while the kernel of group c runs on `stream`, and O of
    // group c returns on the copy-out stream meanwhile.  The fp32 kernel runs
    // far longer than the copies and loses more to the partial last wave of
    // each group than the overlap gains, so it runs as one group.
    const int64_t BH = B * H;
    const int chunks = dtype == FATTN_F32 ? 1 : static_cast<int>(std::min<int64_t>(kHostChunks, BH));
    const size_t row = static_cast<size_t>(N * D) * elem_bytes(dtype);  // one head of Q, K, V or O
    const bool with_lse = lse_host && lse_dev;
    auto bptr = [](const void* base, size_t off) {
        return static_cast<void*>(static_cast<uint8_t*>(const_cast<void*>(base)) + off);
    };
    if (cudaEventRecord(p->fork, stream) != cudaSuccess || cudaStreamWaitEvent(p->in, p->fork, 0) != cudaSuccess)
        return FATTN_ERR_CUDA;
    for (int c = 0; c < chunks; ++c) {
        const int64_t h0 = BH * c / chunks, h1 = BH * (c + 1) / chunks;
        const size_t off = static_cast<size_t>(h0) * row, len = static_cast<size_t>(h1 - h0) * row;
        if (cudaMemcpyAsync(bptr(q_dev, off), bptr(q_host, off), len, cudaMemcpyHostToDevice, p->in) != cudaSuccess ||
            cudaMemcpyAsync(bptr(k_dev, off), bptr(k_host, off), len, cudaMemcpyHostToDevice, p->in) != cudaSuccess ||
            cudaMemcpyAsync(bptr(v_dev, off), bptr(v_host, off), len, cudaMemcpyHostToDevice, p->in) != cudaSuccess ||
            cudaEventRecord(p->in_done[c], p->in) != cudaSuccess ||
            cudaStreamWaitEvent(stream, p->in_done[c], 0) != cudaSuccess)
            return FATTN_ERR_CUDA;
        float* lse_c = lse_dev ? lse_dev + h0 * N : nullptr;
        st = fattn_fwd(bptr(q_dev, off), bptr(k_dev, off), bptr(v_dev, off), bptr(o_dev, off), lse_c, 1,
                       h1 - h0, N, D, scale, causal, dtype, stream_h);
        if (st != FATTN_OK) return st;
        if (cudaEventRecord(p->k_done[c], stream) != cudaSuccess ||
            cudaStreamWaitEvent(p->out, p->k_done[c], 0) != cudaSuccess ||
            cudaMemcpyAsync(bptr(o_host, off), bptr(o_dev, off), len, cudaMemcpyDeviceToHost, p->out) != cudaSuccess)
            return FATTN_ERR_CUDA;
        if (with_lse &&
            cudaMemcpyAsync(lse_host + h0 * N, lse_dev + h0 * N, static_cast<size_t>((h1 - h0) * N) * sizeof(float),
                            cudaMemcpyDeviceToHost, p->out) != cudaSuccess)
            return FATTN_ERR_CUDA;
    }
    if (cudaEventRecord(p->join, p->out) != cudaSuccess || cudaStreamWaitEvent(stream, p->join, 0) != cudaSuccess)
        return FATTN_ERR_CUDA;
    return FATTN_OK;
}

int64_t fattn_unfused_workspace_bytes(int64_t B, int64_t H, int64_t N) {
    if (B <= 0 || H <= 0 || N <= 0) return 0;
    if (B > (int64_t(1) << 30) || H > (int64_t(1) << 30) || N > (int64_t(1) << 30)) return 0;
    const int64_t BH = B * H;
    const int64_t np = unfused_row_pitch(N);
    // 6 * BH * N * np must stay below 2^62
    if (BH > (int64_t(1) << 30) || static_cast<double>(BH) * N * np * 6.0 > 4.0e18) return 0;
    return static_cast<int64_t>(unfused_workspace_bytes(BH, N));
}

int fattn_fwd_unfused(const void* q, const void* k, const void* v, void* o, float* lse,
                      void* workspace, int64_t workspace_bytes, int64_t B, int64_t H, int64_t N,
                      int64_t D, float scale, int causal, int dtype, fattn_stream_t stream_h) {
    bool empty = false;
    int st = validate(q, k, v, o, lse, B, H, H, N, D, scale, dtype, &empty);
    if (st != FATTN_OK || empty) return st;
    if (dtype == FATTN_F32) return FATTN_ERR_UNSUPPORTED;
    const int64_t BH = B * H;
    if (BH > 65535 || ceil_div(N, 128) > 65535) return FATTN_ERR_UNSUPPORTED;
    const int64_t need = fattn_unfused_workspace_bytes(B, H, N);
    if (need <= 0) return FATTN_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < need) return FATTN_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return FATTN_ERR_MISALIGNED;
    const size_t bytes = static_cast<size_t>(BH * N * D) * 2u;
    const size_t ws = static_cast<size_t>(need);
    if (overlaps(workspace, ws, q, bytes) || overlaps(workspace, ws, k, bytes) ||
        overlaps(workspace, ws, v, bytes) || overlaps(workspace, ws, o, bytes) ||
        (lse && overlaps(workspace, ws, lse, static_cast<size_t>(BH * N) * sizeof(float))))
        return FATTN_ERR_INVALID_ARG;
    int sms = 0;
    st = current_sm_count(&sms);
    if (st != FATTN_OK) return st;
    UnfusedArgs a;
    std::memset(&a, 0, sizeof(a));
    const bool bf16 = dtype == FATTN_BF16;
    TcArgs t;
    std::memset(&t, 0, sizeof(t));
    if (tc_encode_maps(t, q, k, v, BH, BH, N, D, bf16) != cudaSuccess) return FATTN_ERR_CUDA;
    a.tmap_q = t.tmap_q;
    a.tmap_k = t.tmap_k;
    a.tmap_v = t.tmap_v;
    a.s = static_cast<float*>(workspace);
    a.p = static_cast<uint8_t*>(workspace) + static_cast<size_t>(BH * N * unfused_row_pitch(N)) * 4u;
    if (unfused_encode_p_map(a, BH, N, bf16) != cudaSuccess) return FATTN_ERR_CUDA;
    a.o = o;
    a.lse = lse;
    a.N = static_cast<int>(N);
    a.Np = static_cast<int>(unfused_row_pitch(N));
    a.BH = static_cast<int>(BH);
    a.H = static_cast<int>(H);
    a.Hkv = static_cast<int>(H);
    a.scale = scale;
    a.timeout_ns = kDefaultTimeoutNs;
    cudaError_t e = unfused_launch(a, static_cast<int>(D), bf16, causal != 0,
                                   reinterpret_cast<cudaStream_t>(stream_h));
    return e == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

int fattn_fwd_unfused_static(const void* q, const void* k, const void* v, void* o, float* lse,
                             int64_t B, int64_t H, int64_t N, int64_t D, float scale, int causal,
                             int dtype, fattn_stream_t stream_h) {
    bool empty = false;
    int st = validate(q, k, v, o, lse, B, H, H, N, D, scale, dtype, &empty);
    if (st != FATTN_OK || empty) return st;
    if (dtype == FATTN_F32) return FATTN_ERR_UNSUPPORTED;
    const int64_t need = fattn_unfused_workspace_bytes(B, H, N);
    if (need <= 0 || need > static_cast<int64_t>(kUnfusedStaticBytes)) return FATTN_ERR_UNSUPPORTED;
    int sms = 0;
    st = current_sm_count(&sms);
    if (st != FATTN_OK) return st;
    void* scratch = nullptr;
    if (unfused_static_scratch(&scratch) != cudaSuccess) return FATTN_ERR_CUDA;
    return fattn_fwd_unfused(q, k, v, o, lse, scratch, static_cast<int64_t>(kUnfusedStaticBytes), B, H,
                             N, D, scale, causal, dtype, stream_h);
}

int64_t fattn_bwd_workspace_bytes(int64_t B, int64_t H, int64_t N) {
    if (B <= 0 || H <= 0 || N <= 0) return 0;
    if (B > (int64_t(1) << 30) || H > (int64_t(1) << 30) || N > (int64_t(1) << 30) ||
        B * H > (int64_t(1) << 30))
        return 0;
    return B * H * 2 * bwd_padded_rows(N) * static_cast<int64_t>(sizeof(float));
}

int fattn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
              const float* lse, void* dq, void* dk, void* dv, void* workspace,
              int64_t workspace_bytes, int64_t B, int64_t H, int64_t N, int64_t D, float scale,
              int causal, int dtype, fattn_stream_t stream_h) {
    return fattn_bwd_gqa(q, k, v, o, dout, lse, dq, dk, dv, workspace, workspace_bytes, B, H, H, N, D,
                         scale, causal, dtype, stream_h);
}

int fattn_bwd_gqa(const void* q, const void* k, const void* v, const void* o, const void* dout,
                  const float* lse, void* dq, void* dk, void* dv, void* workspace,
                  int64_t workspace_bytes, int64_t B, int64_t H, int64_t Hkv, int64_t N, int64_t D,
                  float scale, int causal, int dtype, fattn_stream_t stream_h) {
    bool empty = false;
    // q, k, v and dq share the forward's rules (dq plays O's part).
    int st = validate(q, k, v, dq, nullptr, B, H, Hkv, N, D, scale, dtype, &empty);
    if (st != FATTN_OK || empty) return st;
    if (dtype == FATTN_F32) return FATTN_ERR_UNSUPPORTED;
    if (!o || !dout || !lse || !dk || !dv || !workspace) return FATTN_ERR_INVALID_ARG;
    if (!aligned16(o) || !aligned16(dout) || !aligned16(dk) || !aligned16(dv) || !aligned16(workspace) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u))
        return FATTN_ERR_MISALIGNED;
    const int64_t BH = B * H, BHkv = B * Hkv;
    const int64_t need = fattn_bwd_workspace_bytes(B, H, N);
    if (need <= 0) return FATTN_ERR_UNSUPPORTED;
    if (bwd_padded_rows(N) / 128 * BH > 0x7fffffffll) return FATTN_ERR_UNSUPPORTED;
    if (workspace_bytes < need) return FATTN_ERR_INVALID_ARG;
    const size_t bytes = static_cast<size_t>(BH * N * D) * 2u;
    const size_t kvbytes = static_cast<size_t>(BHkv * N * D) * 2u;
    const size_t lb = static_cast<size_t>(BH * N) * sizeof(float);
    const void* ins[6] = {q, k, v, o, dout, lse};
    const size_t in_sz[6] = {bytes, kvbytes, kvbytes, bytes, bytes, lb};
    void* outs[4] = {dq, dk, dv, workspace};
    const size_t out_sz[4] = {bytes, kvbytes, kvbytes, static_cast<size_t>(need)};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 6; ++j)
            if (overlaps(outs[i], out_sz[i], ins[j], in_sz[j])) return FATTN_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(outs[i], out_sz[i], outs[j], out_sz[j])) return FATTN_ERR_INVALID_ARG;
    }
    int sms = 0;
    st = current_sm_count(&sms);
    if (st != FATTN_OK) return st;
    const bool bf16 = dtype == FATTN_BF16;
    BwdArgs a;
    std::memset(&a, 0, sizeof(a));
    TcArgs t;
    std::memset(&t, 0, sizeof(t));
    if (tc_encode_maps(t, q, k, v, BH, BHkv, N, D, bf16) != cudaSuccess) return FATTN_ERR_CUDA;
    a.tmap_q = t.tmap_q;
    a.tmap_k = t.tmap_k;
    a.tmap_v = t.tmap_v;
    if (tc_encode_maps(t, dout, dout, dout, BH, BH, N, D, bf16) != cudaSuccess) return FATTN_ERR_CUDA;
    a.tmap_do = t.tmap_q;
    a.ws = static_cast<float*>(workspace);
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.N = static_cast<int>(N);
    a.Npad = static_cast<int>(bwd_padded_rows(N));
    a.BH = static_cast<int>(BH);
    a.H = static_cast<int>(H);
    a.Hkv = static_cast<int>(Hkv);
    a.BHkv = static_cast<int>(BHkv);
    a.num_tiles = a.Npad / 128;
    a.sl2 = scale * kLog2e;
    a.scale = scale;
    a.timeout_ns = kDefaultTimeoutNs;
    cudaError_t e = bwd_launch(a, o, dout, lse, static_cast<int>(D), bf16, causal != 0,
                               reinterpret_cast<cudaStream_t>(stream_h));
    return e == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

int fattn_bwd_host(const void* q_host, const void* k_host, const void* v_host, const void* o_host,
                   const void* dout_host, const float* lse_host, void* dq_host, void* dk_host,
                   void* dv_host, void* q_dev, void* k_dev, void* v_dev, void* o_dev, void* dout_dev,
                   float* lse_dev, void* dq_dev, void* dk_dev, void* dv_dev, void* workspace,
                   int64_t workspace_bytes, int64_t B, int64_t H, int64_t N, int64_t D, float scale,
                   int causal, int dtype, fattn_stream_t stream_h) {
    bool empty = false;
    int st = validate(q_dev, k_dev, v_dev, dq_dev, nullptr, B, H, H, N, D, scale, dtype, &empty);
    if (st != FATTN_OK || empty) return st;
    if (!q_host || !k_host || !v_host || !o_host || !dout_host || !lse_host || !dq_host || !dk_host ||
        !dv_host)
        return FATTN_ERR_INVALID_ARG;
    if (dtype == FATTN_F32) return FATTN_ERR_UNSUPPORTED;
    if (!o_dev || !dout_dev || !lse_dev || !dk_dev || !dv_dev || !workspace) return FATTN_ERR_INVALID_ARG;
    const int64_t need = fattn_bwd_workspace_bytes(B, H, N);
    if (need <= 0) return FATTN_ERR_UNSUPPORTED;
    if (workspace_bytes < need) return FATTN_ERR_INVALID_ARG;
    int sms = 0;
    st = current_sm_count(&sms);
    if (st != FATTN_OK) return st;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_h);
    std::lock_guard<std::mutex> lock(g_host_mu);
    HostPipe* p = nullptr;
    if (host_pipe(&p) != cudaSuccess) return FATTN_ERR_CUDA;
    // As fattn_fwd_host: groups of heads whose copies overlap the previous
    // group's three kernels.  A group's statistics use its own slice of the
    // workspace ([heads][2][Npad] floats).
    const int64_t BH = B * H;
    const int chunks = static_cast<int>(std::min<int64_t>(kHostChunks, BH));
    const size_t row = static_cast<size_t>(N * D) * 2u;  // one head of a 16-bit tensor
    const int64_t ws_head = need / BH;                   // bytes of workspace per head
    auto bptr = [](const void* base, size_t off) {
        return static_cast<void*>(static_cast<uint8_t*>(const_cast<void*>(base)) + off);
    };
    if (cudaEventRecord(p->fork, stream) != cudaSuccess || cudaStreamWaitEvent(p->in, p->fork, 0) != cudaSuccess)
        return FATTN_ERR_CUDA;
    for (int c = 0; c < chunks; ++c) {
        const int64_t h0 = BH * c / chunks, h1 = BH * (c + 1) / chunks;
        const size_t off = static_cast<size_t>(h0) * row, len = static_cast<size_t>(h1 - h0) * row;
        const size_t loff = static_cast<size_t>(h0 * N) * sizeof(float);
        const size_t llen = static_cast<size_t>((h1 - h0) * N) * sizeof(float);
        const void* hin[5] = {q_host, k_host, v_host, o_host, dout_host};
        void* din[5] = {q_dev, k_dev, v_dev, o_dev, dout_dev};
        for (int t = 0; t < 5; ++t)
            if (cudaMemcpyAsync(bptr(din[t], off), bptr(hin[t], off), len, cudaMemcpyHostToDevice, p->in) !=
                cudaSuccess)
                return FATTN_ERR_CUDA;
        if (cudaMemcpyAsync(bptr(lse_dev, loff), bptr(lse_host, loff), llen, cudaMemcpyHostToDevice, p->in) !=
                cudaSuccess ||
            cudaEventRecord(p->in_done[c], p->in) != cudaSuccess ||
            cudaStreamWaitEvent(stream, p->in_done[c], 0) != cudaSuccess)
            return FATTN_ERR_CUDA;
        st = fattn_bwd(bptr(q_dev, off), bptr(k_dev, off), bptr(v_dev, off), bptr(o_dev, off),
                       bptr(dout_dev, off), reinterpret_cast<const float*>(bptr(lse_dev, loff)),
                       bptr(dq_dev, off), bptr(dk_dev, off), bptr(dv_dev, off),
                       bptr(workspace, static_cast<size_t>(h0 * ws_head)), (h1 - h0) * ws_head, 1, h1 - h0,
                       N, D, scale, causal, dtype, stream_h);
        if (st != FATTN_OK) return st;
        if (cudaEventRecord(p->k_done[c], stream) != cudaSuccess ||
            cudaStreamWaitEvent(p->out, p->k_done[c], 0) != cudaSuccess)
            return FATTN_ERR_CUDA;
        void* hout[3] = {dq_host, dk_host, dv_host};
        void* dout3[3] = {dq_dev, dk_dev, dv_dev};
        for (int t = 0; t < 3; ++t)
            if (cudaMemcpyAsync(bptr(hout[t], off), bptr(dout3[t], off), len, cudaMemcpyDeviceToHost, p->out) !=
                cudaSuccess)
                return FATTN_ERR_CUDA;
    }
    if (cudaEventRecord(p->join, p->out) != cudaSuccess || cudaStreamWaitEvent(stream, p->join, 0) != cudaSuccess)
        return FATTN_ERR_CUDA;
    return FATTN_OK;
}

namespace {

// fattn_cache_append and fattn_cache_append_kv4: `a` comes filled but for what
// is derived here.
int run_append(AppendArgs& a, const int64_t* strides, int64_t num_pages, int64_t page_size, int64_t rot,
               int64_t T, int64_t H, int64_t Hkv, int64_t D, int dtype, bool kv4, fattn_stream_t stream_h) {
    int st = validate_cache(num_pages, page_size, Hkv, D, dtype);
    if (st != FATTN_OK) return st;
    if (T < 0 || rot < 0 || rot > D || !strides) return FATTN_ERR_INVALID_ARG;
    if (rot % 16 != 0) return FATTN_ERR_UNSUPPORTED;
    if (T == 0) return FATTN_OK;
    if (T > (int64_t(1) << 30)) return FATTN_ERR_UNSUPPORTED;
    if ((a.q == nullptr) != (a.q_out == nullptr)) return FATTN_ERR_INVALID_ARG;
    if (!a.q) H = 0;
    if (H < 0 || (a.q && H == 0)) return FATTN_ERR_INVALID_ARG;
    if (H > (int64_t(1) << 16)) return FATTN_ERR_UNSUPPORTED;
    if (!a.k || !a.v || !a.k_pages || !a.v_pages || !a.slots || (kv4 && (!a.k_scales || !a.v_scales)))
        return FATTN_ERR_INVALID_ARG;
    if (rot > 0 && (!a.pos || !a.cos || !a.sin || a.max_pos < 0)) return FATTN_ERR_INVALID_ARG;
    const void* rows[6] = {a.q, a.k, a.v, a.q_out, a.k_out, a.v_out};
    const int64_t heads[6] = {H, Hkv, Hkv, H, Hkv, Hkv};
    uint32_t* dst[6][2] = {{&a.q_ts, &a.q_hs},   {&a.k_ts, &a.k_hs},   {&a.v_ts, &a.v_hs},
                          {&a.qo_ts, &a.qo_hs}, {&a.ko_ts, &a.ko_hs}, {&a.vo_ts, &a.vo_hs}};
    View views[6];
    for (int i = 0; i < 6; ++i) {
        if (!rows[i]) continue;
        const int64_t ts = strides[2 * i], hs = strides[2 * i + 1];
        if (!stride_ok(ts) || !stride_ok(hs)) return FATTN_ERR_INVALID_ARG;
        if (ts >= (int64_t(1) << 31) || hs >= (int64_t(1) << 31)) return FATTN_ERR_UNSUPPORTED;
        if (!aligned16(rows[i])) return FATTN_ERR_MISALIGNED;
        if (i >= 3 && ((T > 1 && ts < D) || (heads[i] > 1 && hs < D))) return FATTN_ERR_INVALID_ARG;
        *dst[i][0] = static_cast<uint32_t>(ts);
        *dst[i][1] = static_cast<uint32_t>(hs);
        views[i] = rows_view(rows[i], T, ts, heads[i], hs, D);
    }
    const int64_t page_rows = num_pages * page_size * Hkv;
    if (!aligned16(a.k_pages) || !aligned16(a.v_pages) || (kv4 && (!aligned16(a.k_scales) || !aligned16(a.v_scales))) ||
        (reinterpret_cast<uintptr_t>(a.slots) & 7u) || (rot > 0 && ((reinterpret_cast<uintptr_t>(a.pos) & 3u) ||
        !aligned16(a.cos) || !aligned16(a.sin))))
        return FATTN_ERR_MISALIGNED;
    View cache[4];
    if (kv4) {
        cache[0] = dense_view(a.k_pages, page_rows * (D / 2));
        cache[1] = dense_view(a.v_pages, page_rows * (D / 2));
        cache[2] = dense_view(a.k_scales, page_rows * (D / kKv4Group) * 4);
        cache[3] = dense_view(a.v_scales, page_rows * (D / kKv4Group) * 4);
    } else {
        const int64_t inner = Hkv * page_size * D;
        if (!stride_ok(a.page_stride) || a.page_stride < inner) return FATTN_ERR_INVALID_ARG;
        if (a.page_stride > kMaxElements / std::max<int64_t>(num_pages, 1)) return FATTN_ERR_UNSUPPORTED;
        cache[0] = rows_view(a.k_pages, num_pages, a.page_stride, 1, 0, inner);
        cache[1] = rows_view(a.v_pages, num_pages, a.page_stride, 1, 0, inner);
    }
    // (Positions are int32: no row past 2^31 is read.)
    const int64_t table_bytes = std::min<int64_t>(a.max_pos, int64_t(1) << 31) * (rot / 2) * 4;
    const View tables[4] = {dense_view(a.slots, T * 8), dense_view(rot > 0 ? a.pos : nullptr, T * 4),
                            dense_view(rot > 0 ? a.cos : nullptr, table_bytes),
                            dense_view(rot > 0 ? a.sin : nullptr, table_bytes)};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 6; ++j)
            if (views_overlap(cache[i], views[j])) return FATTN_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (views_overlap(cache[i], cache[j])) return FATTN_ERR_INVALID_ARG;
        for (int j = 0; j < 4; ++j)
            if (views_overlap(cache[i], tables[j])) return FATTN_ERR_INVALID_ARG;
    }
    for (int i = 3; i < 6; ++i) {
        if (!rows[i]) continue;
        // An output's own rows must not run into one another.
        if (T > 1 && heads[i] > 1 && views[i].inner > views[i].outer) return FATTN_ERR_INVALID_ARG;
        for (int j = 0; j < 6; ++j) {
            if (j == i) continue;
            const bool itself = j == i - 3 && rows[j] == rows[i] && *dst[j][0] == *dst[i][0] && *dst[j][1] == *dst[i][1];
            if (!itself && views_overlap(views[i], views[j])) return FATTN_ERR_INVALID_ARG;
        }
        for (int j = 0; j < 4; ++j)
            if (views_overlap(views[i], tables[j])) return FATTN_ERR_INVALID_ARG;
    }
    int sms = 0;
    st = current_sm_count(&sms);
    if (st != FATTN_OK) return st;
    a.T = T;
    a.num_slots = num_pages * page_size;
    a.page_size = static_cast<int>(page_size);
    a.H = static_cast<int>(H);
    a.Hkv = static_cast<int>(Hkv);
    a.rot = static_cast<int>(rot);
    const cudaError_t e = append_launch(a, static_cast<int>(D), dtype == FATTN_BF16, kv4, sms,
                                        reinterpret_cast<cudaStream_t>(stream_h));
    return e == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

// fattn_decode and fattn_decode_kv4.
int run_decode(DecodeArgs& a, const int64_t* strides, int64_t num_pages, int64_t page_size, int64_t table_width,
               int64_t ws_bytes, int64_t B, int64_t H, int64_t Hkv, int64_t Nq, int64_t D, float scale, int dtype,
               bool kv4, fattn_stream_t stream_h) {
    int st = validate_cache(num_pages, page_size, Hkv, D, dtype);
    if (st != FATTN_OK) return st;
    if (B < 0 || H < 0 || Nq < 0 || table_width < 0 || !strides || H % Hkv != 0) return FATTN_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || scale < 0.f) return FATTN_ERR_INVALID_ARG;
    if (B == 0 || H == 0 || Nq == 0) return FATTN_OK;
    const int64_t need = fattn_decode_workspace_bytes(B, H, Hkv, Nq, D);
    // Key indices are ints, and the last unit of keys ends past the last key.
    if (need <= 0 || table_width > (0x7fffffffll - 65536) / page_size) return FATTN_ERR_UNSUPPORTED;
    if (!a.q || !a.o || !a.k_pages || !a.v_pages || (kv4 && (!a.k_scales || !a.v_scales)) || !a.seq_lens ||
        (table_width > 0 && !a.block_table) || !a.workspace || ws_bytes < need)
        return FATTN_ERR_INVALID_ARG;
    for (int i = 0; i < 6; ++i) {
        if (!stride_ok(strides[i])) return FATTN_ERR_INVALID_ARG;
        if (strides[i] > kMaxElements / (i % 3 == 0 ? B : (i % 3 == 1 ? H : Nq))) return FATTN_ERR_UNSUPPORTED;
    }
    if (!aligned16(a.q) || !aligned16(a.o) || !aligned16(a.k_pages) || !aligned16(a.v_pages) ||
        (kv4 && (!aligned16(a.k_scales) || !aligned16(a.v_scales))) || !aligned16(a.workspace) ||
        (reinterpret_cast<uintptr_t>(a.lse) & 3u) || (reinterpret_cast<uintptr_t>(a.block_table) & 3u) ||
        (reinterpret_cast<uintptr_t>(a.seq_lens) & 3u))
        return FATTN_ERR_MISALIGNED;
    // o's rows must not run into one another: its strides nest.
    const int64_t sizes[3] = {B, H, Nq};
    const Rows3 q_rows = rows3(a.q, sizes, strides, D), o_rows = rows3(a.o, sizes, strides + 3, D);
    uintptr_t nested = o_rows.row;
    for (int i = 0; i < 3; ++i) {
        if (o_rows.n[i] <= 1) continue;
        if (o_rows.s[i] < nested) return FATTN_ERR_INVALID_ARG;
        nested += (o_rows.n[i] - 1) * o_rows.s[i];
    }
    if (rows3_overlap(q_rows, o_rows)) return FATTN_ERR_INVALID_ARG;
    const int64_t page_rows = num_pages * page_size * Hkv;
    const int64_t inner = Hkv * page_size * D;
    if (!kv4) {
        if (!stride_ok(a.page_stride) || a.page_stride < inner) return FATTN_ERR_INVALID_ARG;
        if (a.page_stride > kMaxElements / std::max<int64_t>(num_pages, 1)) return FATTN_ERR_UNSUPPORTED;
    }
    const int64_t page_bytes = kv4 ? page_rows * (D / 2)
                                   : (num_pages > 0 ? 2 * ((num_pages - 1) * a.page_stride + inner) : 0);
    const int64_t scale_bytes = kv4 ? page_rows * (D / kKv4Group) * 4 : 0;
    auto range = [](const Rows3& r) { return dense_view(reinterpret_cast<const void*>(r.p), r.below(UINTPTR_MAX)); };
    const View in[7] = {range(q_rows),                       dense_view(a.k_pages, page_bytes),
                        dense_view(a.v_pages, page_bytes),   dense_view(a.k_scales, scale_bytes),
                        dense_view(a.v_scales, scale_bytes), dense_view(a.block_table, B * table_width * 4),
                        dense_view(a.seq_lens, B * 4)};
    const View out[3] = {range(o_rows), dense_view(a.lse, B * H * Nq * 4), dense_view(a.workspace, need)};
    for (int i = 0; i < 3; ++i) {
        for (int j = i == 0 ? 1 : 0; j < 7; ++j)  // (o beside q: above)
            if (views_overlap(out[i], in[j])) return FATTN_ERR_INVALID_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (views_overlap(out[i], out[j])) return FATTN_ERR_INVALID_ARG;
    }
    int sms = 0;
    st = current_sm_count(&sms);
    if (st != FATTN_OK) return st;
    a.q_bs = strides[0];
    a.q_hs = strides[1];
    a.q_ns = strides[2];
    a.o_bs = strides[3];
    a.o_hs = strides[4];
    a.o_ns = strides[5];
    a.num_pages = num_pages;
    a.table_width = table_width;
    a.page_size = static_cast<int>(page_size);
    a.B = static_cast<int>(B);
    a.H = static_cast<int>(H);
    a.Hkv = static_cast<int>(Hkv);
    a.Nq = static_cast<int>(Nq);
    a.scale_log2 = scale * kLog2e;
    const cudaError_t e = decode_launch(a, static_cast<int>(D), dtype == FATTN_BF16, kv4, sms,
                                        reinterpret_cast<cudaStream_t>(stream_h));
    return e == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

}  // namespace

int fattn_cache_append(const void* q, const void* k, const void* v, void* q_out, void* k_out,
                       const int64_t* strides, void* k_pages, void* v_pages, int64_t page_stride,
                       int64_t num_pages, int64_t page_size, const int64_t* slots, const int32_t* pos,
                       const float* cos, const float* sin, int64_t max_pos, int64_t rot, int interleaved,
                       int64_t T, int64_t H, int64_t Hkv, int64_t D, int dtype, fattn_stream_t stream_h) {
    AppendArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_out = k_out;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.page_stride = page_stride;
    a.slots = slots;
    a.pos = pos;
    a.cos = cos;
    a.sin = sin;
    a.max_pos = max_pos;
    a.interleaved = interleaved != 0;
    return run_append(a, strides, num_pages, page_size, rot, T, H, Hkv, D, dtype, false, stream_h);
}

int fattn_cache_append_kv4(const void* q, const void* k, const void* v, void* q_out, void* k_out, void* v_out,
                           const int64_t* strides, void* k_codes, void* k_scales, void* v_codes,
                           void* v_scales, int64_t num_pages, int64_t page_size, const int64_t* slots,
                           const int32_t* pos, const float* cos, const float* sin, int64_t max_pos,
                           int64_t rot, int interleaved, int held, int64_t T, int64_t H, int64_t Hkv,
                           int64_t D, int dtype, fattn_stream_t stream_h) {
    AppendArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_out = k_out;
    a.v_out = v_out;
    a.k_pages = k_codes;
    a.v_pages = v_codes;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.slots = slots;
    a.pos = pos;
    a.cos = cos;
    a.sin = sin;
    a.max_pos = max_pos;
    a.interleaved = interleaved != 0;
    a.held = held != 0;
    return run_append(a, strides, num_pages, page_size, rot, T, H, Hkv, D, dtype, true, stream_h);
}

int64_t fattn_packed_workspace_bytes(int64_t B, int64_t T) {
    if (B <= 0 || T <= 0 || B > (int64_t(1) << 30) || T > (int64_t(1) << 30)) return 0;
    const int64_t blocks = T / (kTcBM * kTcQTiles) + B;
    return blocks <= kSmallPlan ? int64_t(kSmallPlanCtas) * kSmallPlanBytes : 16 * (1 + blocks);
}

int fattn_fwd_packed(const void* q, const void* k, const void* v, void* o, float* lse, const int64_t* strides,
                     const int32_t* cu_seqlens, void* workspace, int64_t workspace_bytes, int64_t B, int64_t T,
                     int64_t H, int64_t Hkv, int64_t D, float scale, int causal, int dtype,
                     fattn_stream_t stream_h) {
    if (dtype != FATTN_F32 && dtype != FATTN_F16 && dtype != FATTN_BF16) return FATTN_ERR_INVALID_ARG;
    if (B < 0 || T < 0 || H < 0 || D < 0 || !strides) return FATTN_ERR_INVALID_ARG;
    if (H > 0 && (Hkv <= 0 || H % Hkv != 0)) return FATTN_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || scale < 0.f) return FATTN_ERR_INVALID_ARG;
    if (dtype == FATTN_F32 || (D != 64 && D != 128)) return FATTN_ERR_UNSUPPORTED;
    if (B == 0 || T == 0 || H == 0) return FATTN_OK;
    const int64_t need = fattn_packed_workspace_bytes(B, T);
    if (need <= 0 || H > (int64_t(1) << 16)) return FATTN_ERR_UNSUPPORTED;
    // Task indices (Q blocks x heads) are ints in the kernel.
    const int64_t capacity = T / (kTcBM * kTcQTiles) + B;
    if (capacity * H > (int64_t(1) << 30)) return FATTN_ERR_UNSUPPORTED;
    if (!q || !k || !v || !o || !cu_seqlens || !workspace || workspace_bytes < need) return FATTN_ERR_INVALID_ARG;
    const void* ptrs[4] = {q, k, v, o};
    const int64_t heads[4] = {H, Hkv, Hkv, H};
    int64_t ts[4], hs[4];
    View views[4];
    for (int i = 0; i < 4; ++i) {
        ts[i] = strides[2 * i];
        hs[i] = strides[2 * i + 1];
        if (!stride_ok(ts[i]) || !stride_ok(hs[i])) return FATTN_ERR_INVALID_ARG;
        if ((T > 1 && ts[i] == 0) || (heads[i] > 1 && hs[i] == 0)) return FATTN_ERR_INVALID_ARG;
        // A tensor map's strides are below 2^40 bytes.
        if (ts[i] >= (int64_t(1) << 39) || hs[i] >= (int64_t(1) << 39) || ts[i] > kMaxElements / T ||
            hs[i] > kMaxElements / heads[i])
            return FATTN_ERR_UNSUPPORTED;
        if (!aligned16(ptrs[i])) return FATTN_ERR_MISALIGNED;
        if (T == 1) ts[i] = D;  // strides that are never stepped by
        if (heads[i] == 1) hs[i] = D;
        views[i] = rows_view(ptrs[i], T, ts[i], heads[i], hs[i], D);
    }
    if (!aligned16(workspace) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
        (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u))
        return FATTN_ERR_MISALIGNED;
    // o's rows must not run into one another.
    if ((T > 1 && ts[3] < D) || (H > 1 && hs[3] < D) || (T > 1 && H > 1 && views[3].inner > views[3].outer))
        return FATTN_ERR_INVALID_ARG;
    const View ins[4] = {views[0], views[1], views[2], dense_view(cu_seqlens, (B + 1) * 4)};
    const View outs[3] = {views[3], dense_view(lse, H * T * 4), dense_view(workspace, need)};
    for (int i = 0; i < 3; ++i) {
        for (const View& x : ins)
            if (views_overlap(outs[i], x)) return FATTN_ERR_INVALID_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (views_overlap(outs[i], outs[j])) return FATTN_ERR_INVALID_ARG;
    }
    int sms = 0;
    int st = current_sm_count(&sms);
    if (st != FATTN_OK) return st;
    PackedArgs a;
    std::memset(static_cast<void*>(&a), 0, sizeof(a));
    CUtensorMap* maps[3] = {&a.tmap_q, &a.tmap_k, &a.tmap_v};
    for (int i = 0; i < 3; ++i)
        if (packed_encode_map(maps[i], ptrs[i], T, ts[i], heads[i], hs[i], D, dtype == FATTN_BF16) != cudaSuccess)
            return FATTN_ERR_CUDA;
    a.o = o;
    a.lse = lse;
    a.H = static_cast<int>(H);
    a.Hkv = static_cast<int>(Hkv);
    a.BH = a.H;
    a.head_group = causal_head_group(H, H, Hkv, T, D);  // as one sequence of all tokens
    a.scale_log2 = score_factor(scale);
    a.timeout_ns = kDefaultTimeoutNs;
    a.plan = static_cast<PackedPlan*>(workspace);
    a.cu = cu_seqlens;
    a.B = static_cast<int>(B);
    a.T = T;
    a.o_ts = ts[3];
    a.o_hs = hs[3];
    const int grid = static_cast<int>(std::min<int64_t>(capacity * H, sms));
    a.plan_stride = capacity <= kSmallPlan && grid <= kSmallPlanCtas ? kSmallPlanBytes : 0;
    const cudaError_t e = packed_launch(a, static_cast<int>(D), dtype == FATTN_BF16, causal != 0,
                                        static_cast<int>(capacity), grid, reinterpret_cast<cudaStream_t>(stream_h));
    return e == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

int64_t fattn_decode_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t Nq, int64_t D) {
    if (B <= 0 || H <= 0 || Hkv <= 0 || Nq <= 0 || H % Hkv != 0 || (D != 64 && D != 128)) return 0;
    const int64_t lim = int64_t(1) << 30;
    if (B > lim || H > lim || Nq > lim || B * H > lim || B * H * Nq > lim) return 0;
    return decode_workspace_bytes(B, H, Hkv, Nq, D);
}

int fattn_decode(const void* q, void* o, float* lse, const int64_t* strides, const void* k_pages,
                 const void* v_pages, int64_t page_stride, int64_t num_pages, int64_t page_size,
                 const int32_t* block_table, int64_t table_width, const int32_t* seq_lens, void* workspace,
                 int64_t workspace_bytes, int64_t B, int64_t H, int64_t Hkv, int64_t Nq, int64_t D, float scale,
                 int dtype, fattn_stream_t stream_h) {
    DecodeArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.o = o;
    a.lse = lse;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.page_stride = page_stride;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.workspace = workspace;
    return run_decode(a, strides, num_pages, page_size, table_width, workspace_bytes, B, H, Hkv, Nq, D, scale,
                      dtype, false, stream_h);
}

int fattn_decode_kv4(const void* q, void* o, float* lse, const int64_t* strides, const void* k_codes,
                     const void* k_scales, const void* v_codes, const void* v_scales, int64_t num_pages,
                     int64_t page_size, const int32_t* block_table, int64_t table_width, const int32_t* seq_lens,
                     void* workspace, int64_t workspace_bytes, int64_t B, int64_t H, int64_t Hkv, int64_t Nq,
                     int64_t D, float scale, int dtype, fattn_stream_t stream_h) {
    DecodeArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.o = o;
    a.lse = lse;
    a.k_pages = k_codes;
    a.v_pages = v_codes;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.workspace = workspace;
    return run_decode(a, strides, num_pages, page_size, table_width, workspace_bytes, B, H, Hkv, Nq, D, scale,
                      dtype, true, stream_h);
}

int fattn_get_device_status(fattn_stream_t stream_h) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_h);
    if (cudaStreamSynchronize(stream) != cudaSuccess) return FATTN_ERR_CUDA;
    uint32_t word = 0, word_unfused = 0, word_bwd = 0, word_append = 0, word_decode = 0, word_packed = 0;
    if (read_and_clear_error_word(&word) != cudaSuccess ||
        unfused_read_and_clear_error_word(&word_unfused) != cudaSuccess ||
        bwd_read_and_clear_error_word(&word_bwd) != cudaSuccess ||
        append_read_and_clear_error_word(&word_append) != cudaSuccess ||
        decode_read_and_clear_error_word(&word_decode) != cudaSuccess ||
        packed_read_and_clear_error_word(&word_packed) != cudaSuccess)
        return FATTN_ERR_CUDA;
    word |= word_unfused | word_bwd | word_append | word_decode | word_packed;
    if (word & (1u << FATTN_ERR_INTERNAL)) return FATTN_ERR_INTERNAL;
    if (word & (1u << FATTN_ERR_TIMEOUT)) return FATTN_ERR_TIMEOUT;
    if (word & (1u << FATTN_ERR_INVALID_ARG)) return FATTN_ERR_INVALID_ARG;
    return FATTN_OK;
}

int fattn_selftest_wait_timeout(uint64_t timeout_ns, fattn_stream_t stream_h) {
    if (timeout_ns == 0 || timeout_ns > 1000000000ull) return FATTN_ERR_INVALID_ARG;
    int sms = 0;
    int st = current_sm_count(&sms);
    if (st != FATTN_OK) return st;
    cudaError_t e = launch_wait_selftest(timeout_ns, reinterpret_cast<cudaStream_t>(stream_h));
    return e == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

}  // extern "C"
