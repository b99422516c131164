// C-ABI entry points of libgqa (declared and documented in include/gqa.h): argument checks,
// workspace sizing, TMA descriptor encoding and kernel launches.  No device memory is
// allocated here.
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "gqa.h"
#include "launch.h"
#include "schedule.cuh"
#include "spans.cuh"

namespace gqa {
namespace {

constexpr unsigned long long kDefaultWaitNs = 2000000000ull;
std::atomic<unsigned long long> g_wait_ns{kDefaultWaitNs};
std::atomic<cudaEvent_t> g_ev_before{nullptr};
std::atomic<cudaEvent_t> g_ev_after{nullptr};

constexpr int kMaxDevices = 64;
int g_sm_count[kMaxDevices] = {};
std::mutex g_mu;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// SM count of the current device, or <= 0 when there is none (or it is not sm_100).
int current_sm_count(int *dev_out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return 0;
    }
    *dev_out = dev;
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_sm_count[dev] == 0) {
        int sms = 0, major = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        g_sm_count[dev] = (major == 10) ? sms : -1;
    }
    return g_sm_count[dev];
}

struct Geometry {
    int r, rb, RB, HB, UB;
    long long units, slots, slot_floats, slot_base;
    size_t bytes;
};

// Units: (sequence, key/value head, block of rb query heads) with Q query tokens each; a unit
// has RB = Q * rb <= kMaxUnitCols columns.  A group of more than 32 query heads is cut into
// blocks of 32 that read the same K/V tiles (the second read of a tile finds it in L2 when the
// blocks' pieces run close together), which keeps every softmax thread's per-column state in
// registers.
constexpr int kMaxUnitCols = 32;
Geometry geometry(int B, int H_q, int H_kv, int d, int G, int Q = 1) {
    Geometry g;
    g.r = H_q / H_kv;
    g.rb = g.r < kMaxUnitCols / Q ? g.r : kMaxUnitCols / Q;
    g.RB = Q * g.rb;
    g.HB = (g.r + g.rb - 1) / g.rb;
    g.UB = H_kv * g.HB;
    g.units = static_cast<long long>(B) * g.UB;
    g.slots = G + g.units - 1;
    // O [RB][d], m [RB], l [RB], rounded up to whole 16-byte vectors (the merge reads o with
    // 16-byte loads)
    g.slot_floats = (static_cast<long long>(g.RB) * (d + 2) + 3) / 4 * 4;
    // the per-unit piece counters (int32, kPieceGroups per unit) at offset 0, then the slots
    // from the next 256-byte boundary
    g.slot_base = (g.units * kPieceGroups * 4 + 255) / 256 * 64;
    g.bytes = static_cast<size_t>((g.slot_base + g.slots * g.slot_floats) * 4 + 255) / 256 * 256;
    return g;
}

int check_shape(int B, int H_q, int H_kv, int d, int L_max, gqa_dtype_t dtype,
                bool allow_e4m3 = false) {
    if (dtype != GQA_DTYPE_F32 && dtype != GQA_DTYPE_BF16 &&
        !(allow_e4m3 && dtype == GQA_DTYPE_E4M3))
        return GQA_ERR_UNSUPPORTED_DTYPE;
    if (B <= 0 || H_q <= 0 || H_kv <= 0 || L_max <= 0) return GQA_ERR_SHAPE;
    if (H_q % H_kv != 0) return GQA_ERR_HEADS_NOT_DIVISIBLE;
    if (d != 64 && d != 128) return GQA_ERR_UNSUPPORTED_DIM;
    // Index arithmetic in the kernels: rows of q and tiles per launch stay well inside int32.
    if (static_cast<long long>(B) * H_q > (1ll << 30) || static_cast<long long>(B) * H_kv > (1ll << 30))
        return GQA_ERR_SHAPE;
    return GQA_OK;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
        else
            cudaGetLastError();
    });
    return fn;
}

bool encode_cache_map(CUtensorMap *m, const void *base, int B, int H_kv, int d, int L_max, int rows) {
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H_kv),
                                static_cast<cuuint64_t>(L_max), static_cast<cuuint64_t>(B)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2,
                                   static_cast<cuuint64_t>(H_kv) * d * 2,
                                   static_cast<cuuint64_t>(L_max) * H_kv * d * 2};
    const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(rows), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims,
                       strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B,
                       // L2 fetches as wide as a cached row of one head: 256 bytes would also bring
                       // the next head's half of a 128-byte row, which another CTA reads later
                       d == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An e4m3 cache as (d, H_kv, rows, sequences or pages) of bytes; boxes of `rows` rows of one
// key/value head, d bytes wide, swizzled as the UMMA operands expect (128-byte swizzle for
// d = 128, 64-byte for d = 64).
bool encode_cache_map8(CUtensorMap *m, const void *base, int outer, int H_kv, int d, int rows_dim,
                       int rows) {
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H_kv),
                                static_cast<cuuint64_t>(rows_dim), static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d),
                                   static_cast<cuuint64_t>(H_kv) * d,
                                   static_cast<cuuint64_t>(rows_dim) * H_kv * d};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(d), 1, static_cast<cuuint32_t>(rows), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims,
                       strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_128B,  // a row is at most 128 bytes
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as (d, H_q, tokens); one unit's tile is the box (64 columns, rb heads, Q tokens), which lands
// in shared memory as rows j * rb + h'.
bool encode_q_map(CUtensorMap *m, const void *q, int tokens, int Q, int H_q, int d, int rb) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H_q),
                                static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                                   static_cast<cuuint64_t>(H_q) * d * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(rb), static_cast<cuuint32_t>(Q)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims,
                       strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" int gqa_kv_append(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                             int32_t *seq_lens, int B, int H_kv, int d, int L_max,
                             gqa_dtype_t dtype, int32_t *status, cudaStream_t stream) {
    if (!k_new || !v_new || !k_cache || !v_cache || !seq_lens) return GQA_ERR_NULL;
    if (dtype != GQA_DTYPE_F32 && dtype != GQA_DTYPE_BF16) return GQA_ERR_UNSUPPORTED_DTYPE;
    if (B <= 0 || H_kv <= 0 || L_max <= 0 || static_cast<long long>(B) * H_kv > (1ll << 30))
        return GQA_ERR_SHAPE;
    if (d != 64 && d != 128) return GQA_ERR_UNSUPPORTED_DIM;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(seq_lens, 4) || (status && !aligned(status, 4)))
        return GQA_ERR_ALIGNMENT;
    int dev = 0;
    if (current_sm_count(&dev) <= 0) return GQA_ERR_NO_DEVICE;
    const int row_bytes = d * (dtype == GQA_DTYPE_BF16 ? 2 : 4);
    return launch_append(k_new, v_new, k_cache, v_cache, seq_lens, B, H_kv, row_bytes, L_max, 1,
                         status, stream);
}

extern "C" int gqa_kv_append_multi(const void *k_new, const void *v_new, void *k_cache,
                                   void *v_cache, int32_t *seq_lens, int B, int Q, int H_kv,
                                   int d, int L_max, gqa_dtype_t dtype, int32_t *status,
                                   cudaStream_t stream) {
    if (!k_new || !v_new || !k_cache || !v_cache || !seq_lens) return GQA_ERR_NULL;
    if (dtype != GQA_DTYPE_F32 && dtype != GQA_DTYPE_BF16) return GQA_ERR_UNSUPPORTED_DTYPE;
    if (B <= 0 || Q <= 0 || Q > kMaxUnitCols || H_kv <= 0 || L_max <= 0 ||
        static_cast<long long>(B) * H_kv > (1ll << 30))
        return GQA_ERR_SHAPE;
    if (d != 64 && d != 128) return GQA_ERR_UNSUPPORTED_DIM;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(seq_lens, 4) || (status && !aligned(status, 4)))
        return GQA_ERR_ALIGNMENT;
    int dev = 0;
    if (current_sm_count(&dev) <= 0) return GQA_ERR_NO_DEVICE;
    const int row_bytes = d * (dtype == GQA_DTYPE_BF16 ? 2 : 4);
    return launch_append(k_new, v_new, k_cache, v_cache, seq_lens, B, H_kv, row_bytes, L_max, Q,
                         status, stream);
}

extern "C" size_t gqa_decode_multi_workspace_size(int B, int Q, int H_q, int H_kv, int d,
                                                  gqa_dtype_t dtype) {
    if (Q < 1 || Q > kMaxUnitCols || check_shape(B, H_q, H_kv, d, 1, dtype) != GQA_OK) return 0;
    int dev = 0;
    const int sms = current_sm_count(&dev);
    if (sms <= 0) return 0;
    return geometry(B, H_q, H_kv, d, sms, Q).bytes;
}

int gqa::device_sm_count(int *dev_out) { return current_sm_count(dev_out); }

size_t gqa::decode_counter_region(int B, int H_q, int H_kv, int d, size_t *offset) {
    if (check_shape(B, H_q, H_kv, d, 1, GQA_DTYPE_BF16) != GQA_OK) return 0;
    int dev = 0;
    const int sms = current_sm_count(&dev);
    if (sms <= 0) return 0;
    const Geometry g = geometry(B, H_q, H_kv, d, sms);
    *offset = 0;
    return static_cast<size_t>(g.slot_base) * 4;
}

extern "C" size_t gqa_decode_workspace_size(int B, int H_q, int H_kv, int d, gqa_dtype_t dtype) {
    if (check_shape(B, H_q, H_kv, d, 1, dtype, true) != GQA_OK) return 0;
    int dev = 0;
    const int sms = current_sm_count(&dev);
    if (sms <= 0) return 0;
    return geometry(B, H_q, H_kv, d, sms).bytes;
}

namespace {

// Paged cache description for decode_impl (block_table == nullptr: contiguous caches).
struct PagedArgs {
    const int32_t *block_table = nullptr;
    int max_pages = 0, page_size = 0, n_pages = 0;
};

// The append fused into the decode (k_new == nullptr: none).
struct AppendArgs {
    const void *k_new = nullptr, *v_new = nullptr;
    void *k_cache = nullptr, *v_cache = nullptr;
    int32_t *lens_out = nullptr;
};

int decode_impl(const void *q, const void *k_cache, const void *v_cache, const int32_t *seq_lens,
                int B, int H_q, int H_kv, int d, int L_max, int window, float scale,
                gqa_dtype_t dtype, float *out, void *workspace, size_t workspace_bytes,
                int32_t *status, cudaStream_t stream, const PagedArgs &pg = PagedArgs(),
                int Q = 1, const float *k_scale = nullptr, const float *v_scale = nullptr,
                bool dry_run = false, const AppendArgs &ap = AppendArgs()) {
    if (!q || !k_cache || !v_cache || !seq_lens || !out) return GQA_ERR_NULL;
    const bool fp8 = k_scale != nullptr;
    const int rc = check_shape(B, H_q, H_kv, d, L_max, dtype, fp8);
    if (rc != GQA_OK) return rc;
    if (fp8 && (dtype != GQA_DTYPE_E4M3 || !v_scale)) return GQA_ERR_NULL;
    if (fp8 && (!aligned(k_scale, 4) || !aligned(v_scale, 4))) return GQA_ERR_ALIGNMENT;
    if (!workspace) return GQA_ERR_WORKSPACE;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(seq_lens, 4) || !aligned(workspace, 256) || (status && !aligned(status, 4)))
        return GQA_ERR_ALIGNMENT;
    if (!std::isfinite(scale)) return GQA_ERR_SHAPE;
    int dev = 0;
    const int sms = current_sm_count(&dev);
    if (sms <= 0) return GQA_ERR_NO_DEVICE;
    if (Q < 1 || Q > kMaxUnitCols) return GQA_ERR_SHAPE;
    const Geometry g = geometry(B, H_q, H_kv, d, sms, Q);
    if (workspace_bytes < g.bytes) return GQA_ERR_WORKSPACE;
    if (g.slot_floats % 4 != 0 || g.slot_base % 4 != 0) return GQA_ERR_SHAPE;  // 16-byte slot vectors

    DecodeParams p;
    p.seq_lens = seq_lens;
    p.out = out;
    p.ws = static_cast<float *>(workspace);
    p.status = status;
    p.B = B;
    p.H_q = H_q;
    p.H_kv = H_kv;
    p.d = d;
    p.L_max = L_max;
    p.r = g.r;
    p.Q = Q;
    p.rb = g.rb;
    p.q_box_bytes = (d / 64) * Q * g.rb * 128;
    p.RB = g.RB;
    p.HB = g.HB;
    p.UB = g.UB;
    p.T = fp8 ? tc8_tile_rows(g.RB) : (dtype == GQA_DTYPE_BF16 ? tc_tile_rows(d, g.RB) : 64);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k_new = ap.k_new;
    p.v_new = ap.v_new;
    p.k_cache = ap.k_cache;
    p.v_cache = ap.v_cache;
    p.lens_out = ap.lens_out;
    p.append = ap.k_new != nullptr ? 1 : 0;
    p.window = window;
    p.block_table = pg.block_table;
    p.max_pages = pg.max_pages;
    p.page_size = pg.page_size;
    p.n_pages = pg.n_pages;
    // One persistent CTA per SM, but never more CTAs than the largest possible tile count
    // (the workspace is sized for one per SM, which bounds this).
    const long long span = (window > 0 && window < L_max) ? window : L_max;
    const long long max_tiles = g.units * ((span + p.T - 1) / p.T);
    p.G = max_tiles < sms ? static_cast<int>(max_tiles) : sms;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    p.wait_ns = g_wait_ns.load();
    p.slot_floats = g.slot_floats;
    p.slot_base = g.slot_base;
    p.cnt = static_cast<int32_t *>(workspace);

    cudaEvent_t ev0 = g_ev_before.load(), ev1 = g_ev_after.load();
    const bool profile = ev0 != nullptr && ev1 != nullptr;
    int res;
    if (fp8) {
        if (encode_fn() == nullptr) return GQA_ERR_CUDA;
        TmaMaps maps;
        const int rows_dim = pg.block_table ? pg.page_size : L_max;
        const int outer_dim = pg.block_table ? pg.n_pages : B;
        const int box = pg.block_table ? (pg.page_size < p.T ? pg.page_size : p.T) : p.T;
        if (!encode_cache_map8(&maps.k, k_cache, outer_dim, H_kv, d, rows_dim, box) ||
            !encode_cache_map8(&maps.k8, k_cache, outer_dim, H_kv, d, rows_dim, 8) ||
            !encode_cache_map8(&maps.v, v_cache, outer_dim, H_kv, d, rows_dim, box) ||
            !encode_cache_map8(&maps.v8, v_cache, outer_dim, H_kv, d, rows_dim, 8))
            return GQA_ERR_SHAPE;
        if (dry_run) return GQA_OK;
        if (profile && cudaEventRecord(ev0, stream) != cudaSuccess) return GQA_ERR_CUDA;
        res = launch_split_tc8(maps, q, p, stream);
    } else if (dtype == GQA_DTYPE_BF16) {
        const int rp = tc_q_box_rows(g.RB);
        if (encode_fn() == nullptr) return GQA_ERR_CUDA;
        TmaMaps maps;
        // The cache as (d, H_kv, rows, sequences) -- or, paged, (d, H_kv, page_size, n_pages).
        const int rows_dim = pg.block_table ? pg.page_size : L_max;
        const int outer_dim = pg.block_table ? pg.n_pages : B;
        const int box = pg.block_table ? (pg.page_size < p.T ? pg.page_size : p.T) : p.T;
        (void)rp;
        if (!encode_q_map(&maps.q, q, B * Q, Q, H_q, d, g.rb) ||
            !encode_cache_map(&maps.k, k_cache, outer_dim, H_kv, d, rows_dim, box) ||
            !encode_cache_map(&maps.k8, k_cache, outer_dim, H_kv, d, rows_dim, 8) ||
            !encode_cache_map(&maps.v, v_cache, outer_dim, H_kv, d, rows_dim, box) ||
            !encode_cache_map(&maps.v8, v_cache, outer_dim, H_kv, d, rows_dim, 8))
            return GQA_ERR_SHAPE;
        if (dry_run) return GQA_OK;
        if (profile && cudaEventRecord(ev0, stream) != cudaSuccess) return GQA_ERR_CUDA;
        res = launch_split_tc(maps, p, stream);
    } else {
        if (dry_run) return GQA_OK;
        if (profile && cudaEventRecord(ev0, stream) != cudaSuccess) return GQA_ERR_CUDA;
        res = launch_split_f32(p, static_cast<const float *>(q), static_cast<const float *>(k_cache),
                               static_cast<const float *>(v_cache), stream);
    }
    if (res != GQA_OK) return res;
    if (profile && cudaEventRecord(ev1, stream) != cudaSuccess) return GQA_ERR_CUDA;
    return GQA_OK;
}

}  // namespace

int gqa::decode_check(const void *q, const void *k_cache, const void *v_cache,
                      const int32_t *seq_lens, int B, int H_q, int H_kv, int d, int L_max,
                      float scale, gqa_dtype_t dtype, float *out, int32_t *status) {
    // A stand-in workspace, never dereferenced: every check but the workspace's runs, and
    // nothing is launched.
    return decode_impl(q, k_cache, v_cache, seq_lens, B, H_q, H_kv, d, L_max, 0, scale, dtype,
                       out, reinterpret_cast<void *>(static_cast<uintptr_t>(256)), SIZE_MAX, status,
                       nullptr, PagedArgs(), 1, nullptr, nullptr, true);
}

extern "C" int gqa_decode(const void *q, const void *k_cache, const void *v_cache,
                          const int32_t *seq_lens, int B, int H_q, int H_kv, int d, int L_max,
                          float scale, gqa_dtype_t dtype, float *out, void *workspace,
                          size_t workspace_bytes, int32_t *status, cudaStream_t stream) {
    return decode_impl(q, k_cache, v_cache, seq_lens, B, H_q, H_kv, d, L_max, 0, scale, dtype,
                       out, workspace, workspace_bytes, status, stream);
}

extern "C" int gqa_kv_append_decode(const void *q, const void *k_new, const void *v_new,
                                    void *k_cache, void *v_cache, const int32_t *seq_lens,
                                    int32_t *seq_lens_out, int B, int H_q, int H_kv, int d,
                                    int L_max, float scale, gqa_dtype_t dtype, float *out,
                                    void *workspace, size_t workspace_bytes, int32_t *status,
                                    cudaStream_t stream) {
    if (!k_new || !v_new || !seq_lens_out) return GQA_ERR_NULL;
    if (dtype != GQA_DTYPE_BF16) return GQA_ERR_UNSUPPORTED_DTYPE;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(seq_lens_out, 4))
        return GQA_ERR_ALIGNMENT;
    if (B > 0 && seq_lens != nullptr) {
        const uintptr_t a0 = reinterpret_cast<uintptr_t>(seq_lens), b0 = reinterpret_cast<uintptr_t>(seq_lens_out);
        const uintptr_t n = static_cast<uintptr_t>(B) * sizeof(int32_t);
        if (a0 < b0 + n && b0 < a0 + n) return GQA_ERR_OVERLAP;
    }
    AppendArgs ap;
    ap.k_new = k_new;
    ap.v_new = v_new;
    ap.k_cache = k_cache;
    ap.v_cache = v_cache;
    ap.lens_out = seq_lens_out;
    return decode_impl(q, k_cache, v_cache, seq_lens, B, H_q, H_kv, d, L_max, 0, scale, dtype, out,
                       workspace, workspace_bytes, status, stream, PagedArgs(), 1, nullptr, nullptr,
                       false, ap);
}

extern "C" int gqa_kv_append_paged(const void *k_new, const void *v_new, void *k_pool,
                                   void *v_pool, const int32_t *block_table, int max_pages,
                                   int32_t *seq_lens, int B, int H_kv, int d, int page_size,
                                   int n_pages, gqa_dtype_t dtype, int32_t *status,
                                   cudaStream_t stream) {
    if (!k_new || !v_new || !k_pool || !v_pool || !block_table || !seq_lens) return GQA_ERR_NULL;
    if (dtype != GQA_DTYPE_F32 && dtype != GQA_DTYPE_BF16) return GQA_ERR_UNSUPPORTED_DTYPE;
    if (B <= 0 || H_kv <= 0 || max_pages <= 0 || n_pages <= 0 || page_size <= 0 ||
        page_size % 8 != 0 || static_cast<long long>(max_pages) * page_size > (1ll << 30) ||
        static_cast<long long>(B) * H_kv > (1ll << 30))
        return GQA_ERR_SHAPE;
    if (d != 64 && d != 128) return GQA_ERR_UNSUPPORTED_DIM;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_pool, 16) ||
        !aligned(v_pool, 16) || !aligned(seq_lens, 4) || !aligned(block_table, 4) ||
        (status && !aligned(status, 4)))
        return GQA_ERR_ALIGNMENT;
    int dev = 0;
    if (current_sm_count(&dev) <= 0) return GQA_ERR_NO_DEVICE;
    const int row_bytes = d * (dtype == GQA_DTYPE_BF16 ? 2 : 4);
    return launch_append_paged(k_new, v_new, k_pool, v_pool, block_table, max_pages, seq_lens, B,
                               H_kv, row_bytes, page_size, n_pages, status, stream);
}

extern "C" int gqa_decode_paged(const void *q, const void *k_pool, const void *v_pool,
                                const int32_t *block_table, int max_pages,
                                const int32_t *seq_lens, int B, int H_q, int H_kv, int d,
                                int page_size, int n_pages, float scale, gqa_dtype_t dtype,
                                float *out, void *workspace, size_t workspace_bytes,
                                int32_t *status, cudaStream_t stream) {
    if (!block_table) return GQA_ERR_NULL;
    if (!aligned(block_table, 4)) return GQA_ERR_ALIGNMENT;
    if (max_pages <= 0 || n_pages <= 0 || page_size <= 0 || page_size % 8 != 0 ||
        static_cast<long long>(max_pages) * page_size > (1ll << 30))
        return GQA_ERR_SHAPE;
    // a tile (128 rows, or 256 for 64-wide heads of groups up to 8) must lie in one page or
    // cover whole pages
    if (dtype == GQA_DTYPE_BF16 && H_kv > 0 && H_q % H_kv == 0) {
        const int tr = tc_tile_rows(d, H_q / H_kv < 32 ? H_q / H_kv : 32);
        if (tr % page_size != 0 && page_size % tr != 0) return GQA_ERR_SHAPE;
    }
    PagedArgs pg;
    pg.block_table = block_table;
    pg.max_pages = max_pages;
    pg.page_size = page_size;
    pg.n_pages = n_pages;
    return decode_impl(q, k_pool, v_pool, seq_lens, B, H_q, H_kv, d, max_pages * page_size, 0,
                       scale, dtype, out, workspace, workspace_bytes, status, stream, pg);
}

extern "C" int gqa_decode_multi(const void *q, const void *k_cache, const void *v_cache,
                                const int32_t *seq_lens, int B, int Q, int H_q, int H_kv, int d,
                                int L_max, float scale, gqa_dtype_t dtype, float *out,
                                void *workspace, size_t workspace_bytes, int32_t *status,
                                cudaStream_t stream) {
    if (Q < 1 || Q > kMaxUnitCols) return GQA_ERR_SHAPE;
    return decode_impl(q, k_cache, v_cache, seq_lens, B, H_q, H_kv, d, L_max, 0, scale, dtype,
                       out, workspace, workspace_bytes, status, stream, PagedArgs(), Q);
}

extern "C" int gqa_decode_window(const void *q, const void *k_cache, const void *v_cache,
                                 const int32_t *seq_lens, int B, int H_q, int H_kv, int d,
                                 int L_max, int window, float scale, gqa_dtype_t dtype,
                                 float *out, void *workspace, size_t workspace_bytes,
                                 int32_t *status, cudaStream_t stream) {
    if (window <= 0) return GQA_ERR_SHAPE;
    return decode_impl(q, k_cache, v_cache, seq_lens, B, H_q, H_kv, d, L_max, window, scale,
                       dtype, out, workspace, workspace_bytes, status, stream);
}

extern "C" int gqa_kv_append_fp8(const void *k_new, const void *v_new, gqa_dtype_t new_dtype,
                                 void *k_cache, void *v_cache, const float *k_scale,
                                 const float *v_scale, int32_t *seq_lens, int B, int H_kv, int d,
                                 int L_max, int32_t *status, cudaStream_t stream) {
    if (!k_new || !v_new || !k_cache || !v_cache || !k_scale || !v_scale || !seq_lens)
        return GQA_ERR_NULL;
    if (new_dtype != GQA_DTYPE_F32 && new_dtype != GQA_DTYPE_BF16) return GQA_ERR_UNSUPPORTED_DTYPE;
    if (B <= 0 || H_kv <= 0 || L_max <= 0 || static_cast<long long>(B) * H_kv > (1ll << 30))
        return GQA_ERR_SHAPE;
    if (d != 64 && d != 128) return GQA_ERR_UNSUPPORTED_DIM;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
        !aligned(seq_lens, 4) || (status && !aligned(status, 4)))
        return GQA_ERR_ALIGNMENT;
    int dev = 0;
    if (current_sm_count(&dev) <= 0) return GQA_ERR_NO_DEVICE;
    return launch_append_fp8(k_new, v_new, new_dtype == GQA_DTYPE_BF16, k_cache, v_cache, k_scale,
                             v_scale, seq_lens, nullptr, 0, 0, 0, B, H_kv, d, L_max, 1, status,
                             stream);
}

extern "C" int gqa_kv_append_paged_fp8(const void *k_new, const void *v_new, gqa_dtype_t new_dtype,
                                       void *k_pool, void *v_pool, const float *k_scale,
                                       const float *v_scale, const int32_t *block_table,
                                       int max_pages, int32_t *seq_lens, int B, int H_kv, int d,
                                       int page_size, int n_pages, int32_t *status,
                                       cudaStream_t stream) {
    if (!k_new || !v_new || !k_pool || !v_pool || !k_scale || !v_scale || !block_table || !seq_lens)
        return GQA_ERR_NULL;
    if (new_dtype != GQA_DTYPE_F32 && new_dtype != GQA_DTYPE_BF16) return GQA_ERR_UNSUPPORTED_DTYPE;
    if (B <= 0 || H_kv <= 0 || max_pages <= 0 || n_pages <= 0 || page_size <= 0 ||
        page_size % 8 != 0 || static_cast<long long>(max_pages) * page_size > (1ll << 30) ||
        static_cast<long long>(B) * H_kv > (1ll << 30))
        return GQA_ERR_SHAPE;
    if (d != 64 && d != 128) return GQA_ERR_UNSUPPORTED_DIM;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_pool, 16) ||
        !aligned(v_pool, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
        !aligned(block_table, 4) || !aligned(seq_lens, 4) || (status && !aligned(status, 4)))
        return GQA_ERR_ALIGNMENT;
    int dev = 0;
    if (current_sm_count(&dev) <= 0) return GQA_ERR_NO_DEVICE;
    return launch_append_fp8(k_new, v_new, new_dtype == GQA_DTYPE_BF16, k_pool, v_pool, k_scale,
                             v_scale, seq_lens, block_table, max_pages, page_size, n_pages, B,
                             H_kv, d, 0, 1, status, stream);
}

extern "C" int gqa_decode_fp8(const void *q, const void *k_cache, const void *v_cache,
                              const float *k_scale, const float *v_scale, const int32_t *seq_lens,
                              int B, int H_q, int H_kv, int d, int L_max, int window, float scale,
                              float *out, void *workspace, size_t workspace_bytes,
                              int32_t *status, cudaStream_t stream) {
    if (!k_scale || !v_scale) return GQA_ERR_NULL;
    if (window < 0) return GQA_ERR_SHAPE;
    return decode_impl(q, k_cache, v_cache, seq_lens, B, H_q, H_kv, d, L_max, window, scale,
                       GQA_DTYPE_E4M3, out, workspace, workspace_bytes, status, stream,
                       PagedArgs(), 1, k_scale, v_scale);
}

extern "C" int gqa_decode_paged_fp8(const void *q, const void *k_pool, const void *v_pool,
                                    const float *k_scale, const float *v_scale,
                                    const int32_t *block_table, int max_pages,
                                    const int32_t *seq_lens, int B, int H_q, int H_kv, int d,
                                    int page_size, int n_pages, float scale, float *out,
                                    void *workspace, size_t workspace_bytes, int32_t *status,
                                    cudaStream_t stream) {
    if (!block_table || !k_scale || !v_scale) return GQA_ERR_NULL;
    if (!aligned(block_table, 4)) return GQA_ERR_ALIGNMENT;
    if (max_pages <= 0 || n_pages <= 0 || page_size <= 0 || page_size % 8 != 0 ||
        static_cast<long long>(max_pages) * page_size > (1ll << 30))
        return GQA_ERR_SHAPE;
    // a tile (256 or 128 rows) must lie in one page or cover whole pages
    if (256 % page_size != 0 && page_size % 256 != 0) return GQA_ERR_SHAPE;
    PagedArgs pg;
    pg.block_table = block_table;
    pg.max_pages = max_pages;
    pg.page_size = page_size;
    pg.n_pages = n_pages;
    return decode_impl(q, k_pool, v_pool, seq_lens, B, H_q, H_kv, d, max_pages * page_size, 0,
                       scale, GQA_DTYPE_E4M3, out, workspace, workspace_bytes, status, stream,
                       pg, 1, k_scale, v_scale);
}

namespace {

constexpr int kFewRows = 16;  // query rows of a unit of span_few.cu

// What the span calls share: sizes that follow from the arguments, and the workspace's sections
// (byte offsets).
struct SpanPlan {
    int r, rb, HB, tb, blk, nblkQ, T, RT, unit_rows;
    long long u1, units, slot_floats;
    size_t uinfo, slots, res, res_ml, bytes;
    // The launch for few query rows a span (span_few.cu): the own rows of sequences with few of
    // them, or all of a cross attention of few tokens per sequence.
    bool few = false;
    bool few_all = false;  // the few-row launch takes every span
    int few_rb, few_workers;
    long long few_u1;
    size_t few_rec, few_uinfo, few_slots;
};

// P shared spans over N tokens, and own spans of B sequences (none: B = 0) of Q tokens.
bool span_plan(SpanPlan &s, int P, int N, int B, int Q, int H_q, int H_kv, int d, gqa_dtype_t dtype, int sms) {
    const bool tc = dtype == GQA_DTYPE_BF16;
    s.T = s.RT = tc ? 128 : 64;
    s.r = H_q / H_kv;
    s.rb = s.r < s.RT ? s.r : s.RT;
    s.HB = (s.r + s.rb - 1) / s.rb;
    s.tb = s.RT / s.rb;
    // two row tiles per unit on the tensor cores: both use a cached tile while it is in shared memory
    s.blk = tc ? 2 * s.tb : s.tb;
    s.unit_rows = tc ? 2 * s.RT : s.RT;
    s.nblkQ = (Q + s.blk - 1) / s.blk;
    const long long heads = static_cast<long long>(H_kv) * s.HB;
    s.u1 = static_cast<long long>(N) / s.blk + P + 1;
    s.units = (s.u1 + static_cast<long long>(B) * s.nblkQ) * heads;
    if (heads > 65535 || s.units > (1ll << 30) || static_cast<long long>(N) * H_q > (1ll << 30)) return false;
    s.slot_floats = static_cast<long long>(s.unit_rows) * (d + 2);
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    s.uinfo = up(static_cast<size_t>(sms) * sizeof(SpanRecord));
    s.slots = s.uinfo + up(B > 0 ? s.units * sizeof(int4) : 0);
    s.res = s.slots + up(2ull * sms * s.slot_floats * 4);
    const size_t rows = B > 0 ? 2ull * N * H_q : 0;
    s.res_ml = s.res + up(rows * d * 4);
    s.bytes = s.res_ml + up(rows * 8);
    // With few query rows per span -- up to 32, on average over the encoder sequences; 17 to 32 of them
    // read the span twice -- a product of 128 of them is mostly padding and its chain of waits what is
    // paid for.  64 encoder sequences of 600 states, 24 rows: 35 us, in span_tc.cu 52; 32 of 500 under 64
    // heads, 32 rows: 111 and 145; 16 of 1200, 32 rows: 26 and 26; 4 of 4000 (d = 128), 32 rows: 33 and 30.
    const long long few_tokens = B > 0 ? Q : (static_cast<long long>(N) + P - 1) / P;
    // float32: units of 16 rows in span_f32.cu for up to 16 rows.  16 sequences of 4000 rows, 4 query
    // rows: 130 us, in units of 64 rows 292; 64 of 600, 12 rows (d = 64): 90 and 123, 16 rows: 110 and
    // 124, 32 rows: 204 and 135.
    s.few = few_tokens * s.r <= (tc ? 2 * kFewRows : kFewRows) && s.r <= kFewRows;
    if (s.few) {
        s.few_rb = s.r;
        s.few_workers = sms * (tc ? span_few_warps(d) : 2);
        const int blk = kFewRows / s.r;
        // The same launch takes the shared rows when the groups have as few query rows on average.  bf16,
        // 32/8 heads, d = 128, prompts of 2000 rows and 300 own ones: 8 prompts of 2 sequences (8 rows) 25 us,
        // by two launches 43; 4 of 8 (32 rows) 29 and 40; 16 prompts of 4 (64/8 heads, 32 rows) 58 and 57, of
        // 12 (48 rows) 93 and 72.  float32, 4 samples of 192 rows (16): 11.8 and 14.8.
        s.few_all = B == 0 || (static_cast<long long>(N) + P - 1) / P * s.r <= (tc ? 2 * kFewRows : kFewRows);
        s.few_u1 = s.few_all ? static_cast<long long>(N) / blk + P + 1 : 0;
        const size_t at = B > 0 ? s.bytes : 0;
        const long long units = (s.few_u1 + static_cast<long long>(B) * ((Q + blk - 1) / blk)) * H_kv;
        if (units > (1ll << 30)) return false;
        s.few_rec = at;
        s.few_uinfo = s.few_rec + up(static_cast<size_t>(s.few_workers) * sizeof(SpanRecord));
        s.few_slots = s.few_uinfo + up(B > 0 ? units * sizeof(int4) : 0);
        s.bytes = s.few_slots + up(2ull * s.few_workers * kFewRows * (d + 2) * 4);
    }
    return true;
}

size_t span_workspace(int P, long long N, int B, int Q, int H_q, int H_kv, int d, gqa_dtype_t dtype) {
    if (P < 1 || N < 1 || N > (1ll << 30) || check_shape(1, H_q, H_kv, d, 1, dtype) != GQA_OK) return 0;
    int dev = 0;
    const int sms = current_sm_count(&dev);
    SpanPlan s;
    return sms > 0 && span_plan(s, P, static_cast<int>(N), B, Q, H_q, H_kv, d, dtype, sms) ? s.bytes : 0;
}

// The arrays and sizes of one span call; own caches are absent for cross attention.
struct SpanArgs {
    const void *q = nullptr, *k_shared = nullptr, *v_shared = nullptr, *k_own = nullptr, *v_own = nullptr;
    const int32_t *gstart = nullptr, *glen = nullptr, *lens = nullptr, *block_table = nullptr;
    int P = 0, N = 0, B = 0, Q = 1, H_q = 0, H_kv = 0, d = 0, g_max = 0, own_max = 0;
    int max_pages = 0, page_size = 0, n_pages = 0;
};

int span_impl(const SpanArgs &a, float scale, gqa_dtype_t dtype, float *out, void *workspace, size_t workspace_bytes,
              int32_t *status, cudaStream_t stream) {
    const int rc = check_shape(1, a.H_q, a.H_kv, a.d, a.g_max, dtype);
    if (rc != GQA_OK) return rc;
    if (a.P <= 0 || a.N <= 0 || (a.B > 0 && a.own_max <= 0)) return GQA_ERR_SHAPE;
    if (!workspace) return GQA_ERR_WORKSPACE;
    for (const void *p : {a.q, a.k_shared, a.v_shared, a.k_own, a.v_own, static_cast<const void *>(out)})
        if (!aligned(p, 16)) return GQA_ERR_ALIGNMENT;
    for (const int32_t *p : {a.gstart, a.glen, a.lens, a.block_table, static_cast<const int32_t *>(status)})
        if (!aligned(p, 4)) return GQA_ERR_ALIGNMENT;
    if (!aligned(workspace, 256)) return GQA_ERR_ALIGNMENT;
    if (!std::isfinite(scale)) return GQA_ERR_SHAPE;
    int dev = 0;
    const int sms = current_sm_count(&dev);
    if (sms <= 0) return GQA_ERR_NO_DEVICE;
    SpanPlan s;
    if (!span_plan(s, a.P, a.N, a.B, a.Q, a.H_q, a.H_kv, a.d, dtype, sms)) return GQA_ERR_SHAPE;
    if (workspace_bytes < s.bytes) return GQA_ERR_WORKSPACE;

    const bool paged = a.block_table != nullptr, tc = dtype == GQA_DTYPE_BF16;
    SpanParams p = {};
    p.gstart = a.gstart;
    p.glen = a.glen;
    p.P = a.P;
    p.g_max = a.g_max;
    p.g_step = paged ? a.page_size : 1;
    p.lens = a.lens;
    p.B = a.B;
    p.own_max = a.own_max;
    p.own_after = paged;
    p.Q = a.Q;
    p.N = a.N;
    p.H_q = a.H_q;
    p.H_kv = a.H_kv;
    p.d = a.d;
    p.r = s.r;
    p.rb = s.rb;
    p.HB = s.HB;
    p.tb = s.tb;
    p.blk = s.blk;
    p.nblkQ = s.nblkQ;
    p.T = s.T;
    p.RT = s.RT;
    p.unit_rows = s.unit_rows;
    p.u1 = static_cast<int>(s.u1);
    p.block_table = a.block_table;
    p.max_pages = a.max_pages;
    p.page_size = a.page_size;
    p.n_pages = a.n_pages;
    p.wait_ns = g_wait_ns.load();
    p.out = out;
    p.status = status;
    // One CTA per SM, but no more than there can be tiles.
    const long long tiles_g = (static_cast<long long>(a.g_max) + s.T - 1) / s.T, tiles_o = (static_cast<long long>(a.own_max) + s.T - 1) / s.T;
    const long long most = s.units * (tiles_g > tiles_o ? tiles_g : tiles_o);
    p.G = most < sms ? static_cast<int>(most) : sms;
    const double scale_log2 = static_cast<double>(scale) * 1.4426950408889634;
    p.scale_log2 = static_cast<float>(scale_log2);
    if (tc) {
        // The bf16 kernel finds a row's maximum before it scales, so the sign goes to q; and it
        // masks by -infinity, which times 0 would be NaN: a scale whose products all round to 0
        // stands in for 0.
        p.negate = scale_log2 < 0;
        p.scale_log2 = static_cast<float>(std::fabs(scale_log2));
        if (p.scale_log2 < 1e-37f) p.scale_log2 = 1e-37f;
    }
    p.s_begin = 0;
    p.s_end = a.P + a.B;
    auto *w = static_cast<unsigned char *>(workspace);
    p.rec = reinterpret_cast<SpanRecord *>(w);
    p.uinfo = reinterpret_cast<int4 *>(w + s.uinfo);
    p.slots = reinterpret_cast<float *>(w + s.slots);
    p.slot_floats = s.slot_floats;
    p.res = reinterpret_cast<float *>(w + s.res);
    p.res_ml = reinterpret_cast<float *>(w + s.res_ml);

    SpanParams fp = p;
    if (s.few) {
        fp.rb = s.few_rb;
        fp.HB = 1;
        fp.tb = fp.blk = kFewRows / s.few_rb;
        fp.nblkQ = (a.Q + fp.blk - 1) / fp.blk;
        fp.T = tc ? 16 : 64;
        fp.RT = fp.unit_rows = kFewRows;
        fp.G = s.few_workers;
        fp.u1 = static_cast<int>(s.few_u1);
        fp.rec = reinterpret_cast<SpanRecord *>(w + s.few_rec);
        fp.uinfo = reinterpret_cast<int4 *>(w + s.few_uinfo);
        fp.slots = reinterpret_cast<float *>(w + s.few_slots);
        fp.slot_floats = kFewRows * (a.d + 2);
        if (!s.few_all) {
            p.s_end = fp.s_begin = a.P;
            fp.behind_shared = 1;
        }
    }
    const bool all_few = s.few && s.few_all;  // the only launch
    if (a.B == 0) {
        // As many workers as 8 to a unit, were all encoder sequences alike: a unit's pieces are joined by all
        // of them.  One token of 64/8 heads (d = 128) over 100000 states, 148 pieces a row: the call takes
        // 78 us, by the first one's warps alone 122; with 2 pieces a row of 8 x 509 tokens 196 and 189.
        SpanParams &last = all_few ? fp : p;
        const long long tokens = (static_cast<long long>(a.N) + a.P - 1) / a.P;
        last.spread = last.G >= 8 * static_cast<long long>(a.P) * a.H_kv * last.HB * ((tokens + last.blk - 1) / last.blk);
    }
    if (!tc) {
        const float *q = static_cast<const float *>(a.q), *ks = static_cast<const float *>(a.k_shared), *vs = static_cast<const float *>(a.v_shared);
        const float *ko = static_cast<const float *>(a.k_own), *vo = static_cast<const float *>(a.v_own);
        int res = all_few ? GQA_OK : launch_span_f32(p, q, ks, vs, ko, vo, stream);
        if (res == GQA_OK && s.few) res = launch_span_f32(fp, q, ks, vs, ko, vo, stream);
        return res != GQA_OK ? res : launch_span_merge(all_few ? fp : p, fp, stream);
    }
    if (encode_fn() == nullptr) return GQA_ERR_CUDA;
    // caches as (d, H_kv, rows, prefixes or sequences) or (d, H_kv, page_size, n_pages)
    const int rows_g = paged ? a.page_size : a.g_max, rows_o = paged ? a.page_size : a.own_max;
    const int outer_g = paged ? a.n_pages : a.P, outer_o = paged ? a.n_pages : a.B;
    const int box = paged && a.page_size < s.T ? a.page_size : s.T;
    SpanFewMaps few;
    if (all_few && (!encode_cache_map(&few.kv[0], a.k_shared, outer_g, a.H_kv, a.d, rows_g, 8) ||
                    !encode_cache_map(&few.kv[1], a.v_shared, outer_g, a.H_kv, a.d, rows_g, 8)))
        return GQA_ERR_SHAPE;
    if (s.few && a.B > 0 && (!encode_cache_map(&few.kv[2], a.k_own, outer_o, a.H_kv, a.d, rows_o, 8) ||
                             !encode_cache_map(&few.kv[3], a.v_own, outer_o, a.H_kv, a.d, rows_o, 8)))
        return GQA_ERR_SHAPE;
    if (all_few) {
        const int res = launch_span_few(fp, few, a.q, stream);
        return res != GQA_OK ? res : launch_span_merge(fp, fp, stream);
    }
    SpanMaps m;
    if (!encode_q_map(&m.q_shared, a.q, a.N, s.tb, a.H_q, a.d, s.rb) ||
        !encode_cache_map(&m.k_shared, a.k_shared, outer_g, a.H_kv, a.d, rows_g, box) ||
        !encode_cache_map(&m.k_shared8, a.k_shared, outer_g, a.H_kv, a.d, rows_g, 8) ||
        !encode_cache_map(&m.v_shared, a.v_shared, outer_g, a.H_kv, a.d, rows_g, box) ||
        !encode_cache_map(&m.v_shared8, a.v_shared, outer_g, a.H_kv, a.d, rows_g, 8))
        return GQA_ERR_SHAPE;
    m.q_own = m.q_shared;
    m.k_own = m.k_shared;
    m.k_own8 = m.k_shared8;
    m.v_own = m.v_shared;
    m.v_own8 = m.v_shared8;
    const bool own_here = a.B > 0 && !s.few;
    if (own_here && !encode_q_map(&m.q_own, a.q, a.N, a.Q < s.tb ? a.Q : s.tb, a.H_q, a.d, s.rb)) return GQA_ERR_SHAPE;
    if (own_here && !paged &&
        (!encode_cache_map(&m.k_own, a.k_own, outer_o, a.H_kv, a.d, rows_o, box) ||
         !encode_cache_map(&m.k_own8, a.k_own, outer_o, a.H_kv, a.d, rows_o, 8) ||
         !encode_cache_map(&m.v_own, a.v_own, outer_o, a.H_kv, a.d, rows_o, box) ||
         !encode_cache_map(&m.v_own8, a.v_own, outer_o, a.H_kv, a.d, rows_o, 8)))
        return GQA_ERR_SHAPE;
    int res = launch_span_tc(m, p, stream);
    if (res == GQA_OK && s.few) res = launch_span_few(fp, few, a.q, stream);
    return res != GQA_OK ? res : launch_span_merge(p, fp, stream);
}

}  // namespace

extern "C" size_t gqa_decode_shared_workspace_size(int B, int Q, int P, int H_q, int H_kv, int d, gqa_dtype_t dtype) {
    if (B < 1 || Q < 1 || Q > kMaxUnitCols) return 0;
    return span_workspace(P, static_cast<long long>(B) * Q, B, Q, H_q, H_kv, d, dtype);
}

extern "C" size_t gqa_cross_attend_workspace_size(int E, int N, int H_q, int H_kv, int d, gqa_dtype_t dtype) {
    return span_workspace(E, N, 0, 1, H_q, H_kv, d, dtype);
}

extern "C" int gqa_decode_shared(const void *q, const void *k_prefix, const void *v_prefix,
                                 const int32_t *prefix_lens, const int32_t *group_start, int P,
                                 int L_prefix, const void *k_cache, const void *v_cache,
                                 const int32_t *seq_lens, int B, int Q, int H_q, int H_kv, int d,
                                 int L_max, float scale, gqa_dtype_t dtype, float *out,
                                 void *workspace, size_t workspace_bytes, int32_t *status,
                                 cudaStream_t stream) {
    if (!q || !k_prefix || !v_prefix || !prefix_lens || !group_start || !k_cache || !v_cache || !seq_lens || !out)
        return GQA_ERR_NULL;
    if (B <= 0 || Q < 1 || Q > kMaxUnitCols || static_cast<long long>(B) * Q > (1ll << 30)) return GQA_ERR_SHAPE;
    SpanArgs a;
    a.q = q;
    a.k_shared = k_prefix;
    a.v_shared = v_prefix;
    a.k_own = k_cache;
    a.v_own = v_cache;
    a.gstart = group_start;
    a.glen = prefix_lens;
    a.lens = seq_lens;
    a.P = P;
    a.N = B * Q;
    a.B = B;
    a.Q = Q;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.d = d;
    a.g_max = L_prefix;
    a.own_max = L_max;
    return span_impl(a, scale, dtype, out, workspace, workspace_bytes, status, stream);
}

extern "C" int gqa_decode_shared_paged(const void *q, const void *k_pool, const void *v_pool,
                                       const int32_t *block_table, int max_pages,
                                       const int32_t *seq_lens, const int32_t *group_start,
                                       const int32_t *shared_rows, int P, int B, int Q, int H_q,
                                       int H_kv, int d, int page_size, int n_pages, float scale,
                                       gqa_dtype_t dtype, float *out, void *workspace,
                                       size_t workspace_bytes, int32_t *status, cudaStream_t stream) {
    if (!q || !k_pool || !v_pool || !block_table || !seq_lens || !group_start || !shared_rows || !out)
        return GQA_ERR_NULL;
    if (B <= 0 || Q < 1 || Q > kMaxUnitCols || static_cast<long long>(B) * Q > (1ll << 30)) return GQA_ERR_SHAPE;
    if (max_pages <= 0 || n_pages <= 0 || page_size <= 0 || page_size % 8 != 0 ||
        static_cast<long long>(max_pages) * page_size > (1ll << 30))
        return GQA_ERR_SHAPE;
    // a tile of 128 rows must lie in one page or cover whole pages
    if (dtype == GQA_DTYPE_BF16 && 128 % page_size != 0 && page_size % 128 != 0) return GQA_ERR_SHAPE;
    SpanArgs a;
    a.q = q;
    a.k_shared = a.k_own = k_pool;
    a.v_shared = a.v_own = v_pool;
    a.gstart = group_start;
    a.glen = shared_rows;
    a.lens = seq_lens;
    a.block_table = block_table;
    a.max_pages = max_pages;
    a.page_size = page_size;
    a.n_pages = n_pages;
    a.P = P;
    a.N = B * Q;
    a.B = B;
    a.Q = Q;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.d = d;
    a.g_max = a.own_max = max_pages * page_size;
    return span_impl(a, scale, dtype, out, workspace, workspace_bytes, status, stream);
}

extern "C" int gqa_cross_attend(const void *q, const void *k_enc, const void *v_enc,
                                const int32_t *enc_lens, const int32_t *q_start, int E, int N,
                                int H_q, int H_kv, int d, int S_max, float scale,
                                gqa_dtype_t dtype, float *out, void *workspace,
                                size_t workspace_bytes, int32_t *status, cudaStream_t stream) {
    if (!q || !k_enc || !v_enc || !enc_lens || !q_start || !out) return GQA_ERR_NULL;
    SpanArgs a;
    a.q = q;
    a.k_shared = k_enc;
    a.v_shared = v_enc;
    a.gstart = q_start;
    a.glen = enc_lens;
    a.P = E;
    a.N = N;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.d = d;
    a.g_max = S_max;
    return span_impl(a, scale, dtype, out, workspace, workspace_bytes, status, stream);
}

extern "C" const char *gqa_status_string(int code) {
    switch (code) {
        case GQA_OK: return "ok";
        case GQA_ERR_NULL: return "a required pointer is NULL";
        case GQA_ERR_SHAPE: return "a size is not positive, too large, or not representable";
        case GQA_ERR_HEADS_NOT_DIVISIBLE: return "H_q is not a multiple of H_kv";
        case GQA_ERR_UNSUPPORTED_DIM: return "head dimension d must be 64 or 128";
        case GQA_ERR_UNSUPPORTED_DTYPE: return "unsupported element type";
        case GQA_ERR_ALIGNMENT: return "a pointer is not aligned as required";
        case GQA_ERR_WORKSPACE: return "workspace is NULL or too small";
        case GQA_ERR_CUDA: return "a CUDA runtime call failed";
        case GQA_ERR_NO_DEVICE: return "no usable sm_100 device is current";
        case GQA_ERR_SCRATCH_LIMIT: return "sizes need more scratch than the library's fixed no-allocation array";
        case GQA_ERR_OVERLAP: return "the input and output length arrays overlap";
        default: return "unknown status code";
    }
}

extern "C" int gqa_set_wait_timeout_ns(unsigned long long ns) {
    g_wait_ns.store(ns == 0 ? kDefaultWaitNs : ns);
    return GQA_OK;
}

extern "C" int gqa_profile_events(cudaEvent_t before_split, cudaEvent_t after_split) {
    g_ev_before.store(before_split);
    g_ev_after.store(after_split);
    return GQA_OK;
}
