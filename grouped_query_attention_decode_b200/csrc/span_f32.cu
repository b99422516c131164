// Groups of query rows against spans of a float32 cache, on CUDA cores in float32.
//
// The float32 form of span_tc.cu: the same line of tiles (spans.cuh), with 64 query rows per unit
// and 64 cached rows per tile.  256 threads as 16 x 16: thread (ty, tx) holds 4 x 4 scores and
// 4 x d/16 sums, so the two products read 8 (16) values from shared memory per 16 (32) fused
// multiply-adds of each thread.  A query row's 16 threads are half a warp, which takes its maximum
// and sum by shuffles.
#include <cstdint>

#include "device.cuh"
#include "gqa.h"
#include "launch.h"
#include "spans.cuh"

namespace gqa {

namespace {

template <int D>
struct SpanF32Cfg {
    static constexpr int T = 64, RT = 64, THREADS = 256;
    static constexpr int QP = D + 4;  // padded rows: 16 threads read 16 rows without bank conflicts
    static constexpr int PP = T + 4;
    static constexpr int SMEM_BYTES = (RT * QP + T * QP + T * D + RT * PP) * 4;
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(256)
span_f32_kernel(const float *__restrict__ q, const float *__restrict__ ks, const float *__restrict__ vs,
                const float *__restrict__ ko, const float *__restrict__ vo, const __grid_constant__ SpanParams p) {
    using C = SpanF32Cfg<D>;
    constexpr int T = C::T, QP = C::QP, PP = C::PP, E = D / 16;  // E output columns a thread
    extern __shared__ float4 span_smem[];
    float *const sq = reinterpret_cast<float *>(span_smem);  // [RT][QP]
    float *const sk = sq + C::RT * QP;                        // [T][QP]
    float *const sv = sk + T * QP;                            // [T][D]
    float *const sp = sv + T * D;                             // [RT][PP]
    __shared__ long long scratch[C::THREADS / 32];
    __shared__ SpanRange range;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;

    grid_dependency_wait();
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
        long long orow[4];
        int seen[4];
        float m[4], l[4], o[4][E];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            int token;
            orow[a] = span_row(p, g, 0, ty * 4 + a, token);
            seen[a] = orow[a] >= 0 ? seen_rows(p, g, token) : 0;
            m[a] = -INFINITY;
            l[a] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[a][e] = 0.f;
        }
        for (int jj = 0; jj < g.len; ++jj) {
            const int t0 = (g.j0 + jj) * T, rows = min(T, g.rows - t0);
            __syncthreads();  // the tile before has been read
            for (int i = tid; i < T * (D / 4); i += 256) {
                const int t = i / (D / 4), c = i - t * (D / 4);
                float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
                if (t < rows) {
                    long long at = g.row0 + t0 + t;
                    if (p.block_table != nullptr) {
                        int pg = __ldg(p.block_table + static_cast<long long>(g.src) * p.max_pages + at / p.page_size);
                        if (pg < 0 || pg >= p.n_pages) {
                            if (p.status != nullptr) atomicOr(p.status, GQA_STATUS_PAGE_RANGE);
                            pg = 0;
                        }
                        at = static_cast<long long>(pg) * p.page_size + at % p.page_size;
                    } else {
                        at += static_cast<long long>(g.src) * (shared ? p.g_max : p.own_max);
                    }
                    at = (at * p.H_kv + g.kvh) * (D / 4) + c;
                    kv = __ldg(reinterpret_cast<const float4 *>(kc) + at);
                    vv = __ldg(reinterpret_cast<const float4 *>(vc) + at);
                }
                *reinterpret_cast<float4 *>(sk + t * QP + 4 * c) = kv;
                *reinterpret_cast<float4 *>(sv + t * D + 4 * c) = vv;
            }
            __syncthreads();
            // scores of rows ty * 4 + a and cached rows tx + 16 b
            float s[4][4] = {};
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                float4 qa[4], kb[4];
#pragma unroll
                for (int a = 0; a < 4; ++a) qa[a] = *reinterpret_cast<const float4 *>(sq + (ty * 4 + a) * QP + c);
#pragma unroll
                for (int b = 0; b < 4; ++b) kb[b] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * b) * QP + c);
#pragma unroll
                for (int a = 0; a < 4; ++a)
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        s[a][b] = fmaf(qa[a].x, kb[b].x, s[a][b]);
                        s[a][b] = fmaf(qa[a].y, kb[b].y, s[a][b]);
                        s[a][b] = fmaf(qa[a].z, kb[b].z, s[a][b]);
                        s[a][b] = fmaf(qa[a].w, kb[b].w, s[a][b]);
                    }
            }
#pragma unroll
            for (int a = 0; a < 4; ++a) {
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
                    sp[(ty * 4 + a) * PP + tx + 16 * b] = e;
                    sum += e;
                }
                l[a] = l[a] * alpha + sum;  // this thread's columns; joined at the end
#pragma unroll
                for (int e = 0; e < E; ++e) o[a][e] *= alpha;
            }
            __syncwarp();  // a row's P is written and read by the same half warp
            const int steps = (rows + 3) & ~3;  // rows past the end are zeros
#pragma unroll 2
            for (int t = 0; t < steps; t += 4) {
                float4 pr[4];
#pragma unroll
                for (int a = 0; a < 4; ++a) pr[a] = *reinterpret_cast<const float4 *>(sp + (ty * 4 + a) * PP + t);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float4 vv[E / 4];
#pragma unroll
                    for (int e = 0; e < E / 4; ++e) vv[e] = *reinterpret_cast<const float4 *>(sv + (t + u) * D + 64 * e + 4 * tx);
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
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
        for (int a = 0; a < 4; ++a) {
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) l[a] += __shfl_xor_sync(kFullMask, l[a], x);
            if (orow[a] < 0) continue;
            float *dst;
            float norm = 1.f;
            if (!g.whole()) {
                float *slot = p.slots + (2ll * blockIdx.x + (g.first ? 0 : 1)) * p.slot_floats;
                dst = slot + (ty * 4 + a) * D;
                if (tx == 0) *reinterpret_cast<float2 *>(slot + p.unit_rows * D + 2 * (ty * 4 + a)) = make_float2(m[a], l[a]);
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
}

namespace {

template <int D>
int launch_span_f32_impl(const SpanParams &p, const float *q, const float *ks, const float *vs, const float *ko,
                         const float *vo, cudaStream_t stream) {
    using C = SpanF32Cfg<D>;
    auto kern = span_f32_kernel<D>;
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
    return p.d == 128 ? launch_span_f32_impl<128>(p, q, ks, vs, ko, vo, stream)
                      : launch_span_f32_impl<64>(p, q, ks, vs, ko, vo, stream);
}

}  // namespace gqa
