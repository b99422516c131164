// Groups of query rows against spans of a float32 cache, on CUDA cores in float32.
//
// The float32 form of span_tc.cu and span_few.cu: the same line of tiles (spans.cuh), 64 cached rows
// per tile and RT = 64 or 16 query rows per unit.  256 threads as 16 x 16: thread (ty, tx) holds
// RT/16 x 4 scores and RT/16 x d/16 sums, and a query row's 16 threads are half a warp, which takes
// its maximum and sum by shuffles.  With 64 rows the two products read 8 (16) values from shared
// memory per 16 (32) fused multiply-adds of a thread and run at 35 TFLOP/s (4 encoder sequences of
// 2048 rows under 256 tokens, 32/8 heads, d = 128: 980 us), half of what the CUDA cores have: one CTA
// fits an SM, two warps a scheduler, and so few hide little of each other's reads.  With 16 rows
// they are bound by those reads and by issue, so warps whose rows are padding leave them out: 16 sequences of 4000 rows
// under 4 rows a head take 130 us (82 at the speed of memory), 302 with every warp at work.
#include <cstdint>

#include "device.cuh"
#include "gqa.h"
#include "launch.h"
#include "spans.cuh"

namespace gqa {

namespace {

template <int D, int ROWS>
struct SpanF32Cfg {
    static constexpr int T = 64, RT = ROWS, THREADS = 256;
    static constexpr int A = RT / 16;  // rows a thread
    static constexpr int CTAS = RT == 64 ? 1 : 2;  // of an SM
    static constexpr int QP = D + 4;  // padded rows: 16 threads read 16 rows without bank conflicts
    static constexpr int PP = T + 4;
    static constexpr int SMEM_BYTES = (RT * QP + T * QP + T * D + RT * PP) * 4;
};

__device__ __forceinline__ void copy_16(float *dst, const float *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_all;" ::: "memory"); }

}  // namespace

template <int D, int ROWS>
__global__ void __launch_bounds__(256, SpanF32Cfg<D, ROWS>::CTAS)
span_f32_kernel(const float *__restrict__ q, const float *__restrict__ ks, const float *__restrict__ vs,
                const float *__restrict__ ko, const float *__restrict__ vo, const __grid_constant__ SpanParams p) {
    using C = SpanF32Cfg<D, ROWS>;
    constexpr int T = C::T, QP = C::QP, PP = C::PP, A = C::A, E = D / 16;  // E output columns a thread
    extern __shared__ float4 span_smem[];
    float *const sq = reinterpret_cast<float *>(span_smem);  // [RT][QP]
    float *const sk = sq + C::RT * QP;                        // [T][QP]
    float *const sv = sk + T * QP;                            // [T][D]
    float *const sp = sv + T * D;                             // [RT][PP]
    __shared__ long long scratch[C::THREADS / 32];
    __shared__ SpanRange range;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;

    if (!p.behind_shared) grid_dependency_wait();  // see span_few.cu
    locate_span_range<C::THREADS>(p, blockIdx.x, scratch, &range);
    grid_launch_dependents();
    const SpanRange cr = range;
    SpanWalker w;
    w.init(p, cr);
    SpanSegment g;
    if (tid == 0) open_notes(p, blockIdx.x);
    while (w.next(p, g)) {
        if (tid == 0) note_unit(p, g, cr, blockIdx.x);
        const bool shared = g.s < p.P;
        const float *const kc = shared ? ks : ko, *const vc = shared ? vs : vo;
        for (int i = tid; i < C::RT * (D / 4); i += 256) {
            const int row = i / (D / 4), c = i - row * (D / 4);
            int token;
            const long long orow = span_row(p, g, 0, row, token);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (orow >= 0) v = __ldg(reinterpret_cast<const float4 *>(q + orow * D) + c);
            *reinterpret_cast<float4 *>(sq + row * QP + 4 * c) = v;
        }
        long long orow[A];
        int seen[A];
        float m[A], l[A], o[A][E];
#pragma unroll
        for (int a = 0; a < A; ++a) {
            int token;
            orow[a] = span_row(p, g, 0, ty * A + a, token);
            seen[a] = orow[a] >= 0 ? seen_rows(p, g, token) : 0;
            m[a] = -INFINITY;
            l[a] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[a][e] = 0.f;
        }
        bool some = false;
#pragma unroll
        for (int a = 0; a < A; ++a) some |= orow[a] >= 0;
        const bool idle = !__any_sync(kFullMask, some);  // a warp of padding only copies
        // Rows of tile jj into shared memory, 16 bytes a copy, zeros behind the span's end.
        const auto copy_tile = [&](float *dst, int pitch, const float *cache, int jj) {
            const int t0 = (g.j0 + jj) * T, rows = min(T, g.rows - t0), c = tid % (D / 4);
#pragma unroll 4
            for (int t = tid / (D / 4); t < T; t += C::THREADS / (D / 4)) {
                const int row = g.row0 + t0 + min(t, rows - 1);
                long long at = row;
                if (p.block_table != nullptr) {
                    const int i_page = row / p.page_size;
                    int pg = __ldg(p.block_table + static_cast<long long>(g.src) * p.max_pages + i_page);
                    if (pg < 0 || pg >= p.n_pages) {
                        if (p.status != nullptr) atomicOr(p.status, GQA_STATUS_PAGE_RANGE);
                        pg = 0;
                    }
                    at = static_cast<long long>(pg) * p.page_size + (row - i_page * p.page_size);
                } else {
                    at += static_cast<long long>(g.src) * (shared ? p.g_max : p.own_max);
                }
                copy_16(dst + t * pitch + 4 * c, cache + ((at * p.H_kv + g.kvh) * D + 4 * c), t < rows);
            }
        };
        // K of the next tile arrives during the second product, V during the first.
        copy_tile(sk, QP, kc, 0);
        for (int jj = 0; jj < g.len; ++jj) {
            const int t0 = (g.j0 + jj) * T, rows = min(T, g.rows - t0);
            wait_copies();
            __syncthreads();  // q and K are there, the V before has been read
            copy_tile(sv, D, vc, jj);
            if (idle) {  // the barriers of the others
                wait_copies();
                __syncthreads();
                if (jj + 1 < g.len) copy_tile(sk, QP, kc, jj + 1);
                continue;
            }
            // scores of rows A ty + a and cached rows tx + 16 b
            float s[A][4] = {};
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                float4 qa[A], kb[4];
#pragma unroll
                for (int a = 0; a < A; ++a) qa[a] = *reinterpret_cast<const float4 *>(sq + (ty * A + a) * QP + c);
#pragma unroll
                for (int b = 0; b < 4; ++b) kb[b] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * b) * QP + c);
#pragma unroll
                for (int a = 0; a < A; ++a)
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        s[a][b] = fmaf(qa[a].x, kb[b].x, s[a][b]);
                        s[a][b] = fmaf(qa[a].y, kb[b].y, s[a][b]);
                        s[a][b] = fmaf(qa[a].z, kb[b].z, s[a][b]);
                        s[a][b] = fmaf(qa[a].w, kb[b].w, s[a][b]);
                    }
            }
#pragma unroll
            for (int a = 0; a < A; ++a) {
                float top = -INFINITY;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    s[a][b] = t0 + tx + 16 * b < seen[a] ? s[a][b] * p.scale_log2 : -INFINITY;
                    top = fmaxf(top, s[a][b]);
                }
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, x));
                const float m_new = fmaxf(m[a], top);
                const float ref = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = ex2_approx(m[a] - ref);  // 0 from m = -infinity
                m[a] = m_new;
                float sum = 0.f;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float e = ex2_approx(s[a][b] - ref);
                    sp[(ty * A + a) * PP + tx + 16 * b] = e;
                    sum += e;
                }
                l[a] = l[a] * alpha + sum;  // this thread's columns; joined at the end
#pragma unroll
                for (int e = 0; e < E; ++e) o[a][e] *= alpha;
            }
            wait_copies();
            __syncthreads();  // P and V are there, K has been read
            if (jj + 1 < g.len) copy_tile(sk, QP, kc, jj + 1);
            const int steps = (rows + 3) & ~3;  // rows past the end are zeros
#pragma unroll 2
            for (int t = 0; t < steps; t += 4) {
                float4 pr[A];
#pragma unroll
                for (int a = 0; a < A; ++a) pr[a] = *reinterpret_cast<const float4 *>(sp + (ty * A + a) * PP + t);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float4 vv[E / 4];
#pragma unroll
                    for (int e = 0; e < E / 4; ++e) vv[e] = *reinterpret_cast<const float4 *>(sv + (t + u) * D + 64 * e + 4 * tx);
#pragma unroll
                    for (int a = 0; a < A; ++a) {
                        const float pa = u == 0 ? pr[a].x : u == 1 ? pr[a].y : u == 2 ? pr[a].z : pr[a].w;
#pragma unroll
                        for (int e = 0; e < E / 4; ++e) {
                            o[a][4 * e] = fmaf(pa, vv[e].x, o[a][4 * e]);
                            o[a][4 * e + 1] = fmaf(pa, vv[e].y, o[a][4 * e + 1]);
                            o[a][4 * e + 2] = fmaf(pa, vv[e].z, o[a][4 * e + 2]);
                            o[a][4 * e + 3] = fmaf(pa, vv[e].w, o[a][4 * e + 3]);
                        }
                    }
                }
            }
        }
        __syncthreads();  // the next unit's q may overwrite sq
#pragma unroll
        for (int a = 0; a < A; ++a) {
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) l[a] += __shfl_xor_sync(kFullMask, l[a], x);
            if (orow[a] < 0) continue;
            float *dst;
            float norm = 1.f;
            if (!g.whole()) {
                float *slot = p.slots + (2ll * blockIdx.x + (g.first ? 0 : 1)) * p.slot_floats;
                dst = slot + (ty * A + a) * D;
                if (tx == 0) *reinterpret_cast<float2 *>(slot + p.unit_rows * D + 2 * (ty * A + a)) = make_float2(m[a], l[a]);
            } else if (p.B > 0) {
                const long long rr = (shared ? 0 : static_cast<long long>(p.N) * p.H_q) + orow[a];
                dst = p.res + rr * D;
                if (tx == 0) *reinterpret_cast<float2 *>(p.res_ml + 2 * rr) = make_float2(m[a], l[a]);
            } else {
                dst = p.out + orow[a] * D;
                norm = 1.f / l[a];
            }
#pragma unroll
            for (int e = 0; e < E / 4; ++e)
                *reinterpret_cast<float4 *>(dst + 64 * e + 4 * tx) =
                    make_float4(o[a][4 * e] * norm, o[a][4 * e + 1] * norm, o[a][4 * e + 2] * norm, o[a][4 * e + 3] * norm);
        }
    }
    if (p.behind_shared) grid_dependency_wait();
}

namespace {

template <int D, int ROWS>
int launch_span_f32_impl(const SpanParams &p, const float *q, const float *ks, const float *vs, const float *ko,
                         const float *vo, cudaStream_t stream) {
    using C = SpanF32Cfg<D, ROWS>;
    auto kern = span_f32_kernel<D, ROWS>;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GQA_ERR_CUDA;
    if (dev < 64 && !attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
            return GQA_ERR_CUDA;
        attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.G);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, q, ks, vs, ko, vo, p) != cudaSuccess) return GQA_ERR_CUDA;
    return GQA_OK;
}

}  // namespace

int launch_span_f32(const SpanParams &p, const float *q, const float *ks, const float *vs, const float *ko,
                    const float *vo, cudaStream_t stream) {
    if (p.RT == 16)
        return p.d == 128 ? launch_span_f32_impl<128, 16>(p, q, ks, vs, ko, vo, stream)
                          : launch_span_f32_impl<64, 16>(p, q, ks, vs, ko, vo, stream);
    return p.d == 128 ? launch_span_f32_impl<128, 64>(p, q, ks, vs, ko, vo, stream)
                      : launch_span_f32_impl<64, 64>(p, q, ks, vs, ko, vo, stream);
}

}  // namespace gqa
