// Joins the pieces that the span kernels left in the workspace (spans.cuh): with pieces c of a
// row's attended rows, each an unnormalised sum o_c, its reference m_c and l_c,
//     M = max_c m_c,  out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c.
// One warp per query row, d / 32 columns a lane.  It is launched with the programmatic
// attribute, so its blocks are resident when the span kernel's last CTA ends.
#include <cstdint>

#include "device.cuh"
#include "gqa.h"
#include "spans.cuh"

namespace gqa {

namespace {

template <int V>
struct Vec;
template <>
struct Vec<2> { using type = float2; };
template <>
struct Vec<4> { using type = float4; };

// A row's running join; V columns a lane.
template <int V>
struct Join {
    float M = -INFINITY, L = 0.f, o[V] = {};

    __device__ void add(float m, float l, typename Vec<V>::type ov) {
        if (m == -INFINITY) return;  // a piece in which the row saw nothing: its sum is not looked at
        const float top = fmaxf(M, m);
        const float a = M == -INFINITY ? 0.f : ex2_approx(M - top), b = ex2_approx(m - top);
        const float *x = reinterpret_cast<const float *>(&ov);
        M = top;
        L = L * a + l * b;
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = o[k] * a + x[k] * b;
    }
    __device__ void store(float *dst) const {
        typename Vec<V>::type r;
        float *x = reinterpret_cast<float *>(&r);
        const float inv = L > 0.f || L != L ? 1.f / L : 0.f;  // no rows at all: zeros
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] = o[k] * inv;
        *reinterpret_cast<typename Vec<V>::type *>(dst) = r;
    }
};

// Adds row `srow` of every piece of a unit cut at CTA boundaries c0 .. c1.  The CTAs between
// hold one piece each, except that with fewer tiles than CTAs some hold none.
template <int V>
__device__ void add_pieces(const SpanParams &p, long long total, int c0, int k0, int c1, int srow, int lane, Join<V> &j) {
    using T = typename Vec<V>::type;
    constexpr int AT_ONCE = 8;  // pieces whose loads are in flight together
    for (int c = c0; c <= c1; c += AT_ONCE) {
        float2 ml[AT_ONCE];
        T o[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const int cc = c + u;
            ml[u] = make_float2(-INFINITY, 0.f);
            if (cc <= c1 && (total >= p.G || cta_range_begin(cc, total, p.G) < cta_range_begin(cc + 1, total, p.G))) {
                const float *slot = p.slots + (2ll * cc + (cc == c0 ? k0 : 0)) * p.slot_floats;
                ml[u] = __ldcg(reinterpret_cast<const float2 *>(slot + p.unit_rows * p.d + 2 * srow));
                o[u] = __ldcg(reinterpret_cast<const T *>(slot + static_cast<long long>(srow) * p.d) + lane);
            }
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u)
            if (c + u <= c1) j.add(ml[u].x, ml[u].y, o[u]);
    }
}

// What note_unit wrote.  A span kernel that gave up a wait may not have: whatever stands there
// then is kept inside the workspace.
__device__ __forceinline__ int4 unit_pieces_of(const SpanParams &p, int unit) {
    int4 u = __ldcg(p.uinfo + unit);
    u.x = min(max(u.x, 0), p.G - 1);
    u.z = min(max(u.z, u.x), p.G - 1);
    u.y &= 1;
    return u;
}

// Row of a slot that (token tl of the unit, head hp of the head block) is.
__device__ __forceinline__ int slot_row(const SpanParams &p, int tl, int hp) {
    const int tile = tl / p.tb;
    return tile * p.RT + (tl - tile * p.tb) * p.rb + hp;
}

// Shared and own rows: one block per (token, key/value head), a warp per query head.  p[0] is the
// launch over the shared spans, p[1] the one over the own ones.
template <int V>
__global__ void __launch_bounds__(256) span_merge_shared_kernel(const __grid_constant__ SpanParams p0, const __grid_constant__ SpanParams p1) {
    grid_dependency_wait();
    const int tok = blockIdx.x, kvh = blockIdx.y;
    const int b = tok / p0.Q, lane = threadIdx.x & 31;
    // the token's spans, found by two warps at once
    __shared__ Span span_s[2];
    __shared__ int valid_s[2];
    __shared__ long long total_s[2];
    if (threadIdx.x == 0) {
        const int g = group_of(p0, b);
        Span sp = {0, 0, 0, 0, 0};
        valid_s[0] = 1;
        if (g >= 0) {
            sp = span_at(p0, g, false);
            if (tok < sp.tok0 || tok >= sp.tok0 + sp.ntok) sp.rows = 0;  // a group whose start is out of range
            valid_s[0] = shared_rows_of(p0, g) >= 0;
        }
        sp.src = g;
        span_s[0] = sp;
        total_s[0] = __ldcg(&p0.rec->total);
    } else if (threadIdx.x == 32) {
        Span sp = {b * p0.Q, p0.Q, 0, 0, p0.P + b};
        valid_s[1] = own_rows_of(p1, b, sp.row0, sp.rows);
        span_s[1] = sp;
        total_s[1] = __ldcg(&p1.rec->total);
    }
    __syncthreads();
    const bool valid = valid_s[0] && valid_s[1];
    for (int h = threadIdx.x >> 5; h < p0.r; h += 8) {
        const long long row = static_cast<long long>(tok) * p0.H_q + kvh * p0.r + h;
        Join<V> j;
        if (valid) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const SpanParams &p = c == 0 ? p0 : p1;
                const Span sp = span_s[c];
                if (sp.rows == 0) continue;
                const int hb = h / p.rb, tl = tok - sp.tok0, block = tl / p.blk;
                const int4 u = unit_pieces_of(p, unit_number(p, sp.src, sp, block, kvh, hb));
                if (u.x == u.z) {
                    const long long rr = (c == 0 ? 0 : static_cast<long long>(p.N) * p.H_q) + row;
                    const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p.res_ml) + rr);
                    j.add(ml.x, ml.y, __ldcg(reinterpret_cast<const typename Vec<V>::type *>(p.res + rr * p.d) + lane));
                } else {
                    add_pieces<V>(p, total_s[c], u.x, u.y, u.z, slot_row(p, tl - block * p.blk, h - hb * p.rb), lane, j);
                }
            }
        }
        j.store(p0.out + row * p0.d + lane * V);
    }
}

// Cross attention: block (c, part) joins a part of the rows of the cut unit that starts in CTA c,
// and of the tokens whose encoder sequence has no states writes zeros.
template <int V>
__global__ void __launch_bounds__(256) span_merge_cross_kernel(const __grid_constant__ SpanParams p) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = blockIdx.y * 8 + (threadIdx.x >> 5), warps = gridDim.y * 8;
    const SpanRecord u = p.rec[blockIdx.x];
    if (u.valid) {
        const int heads = min(p.rb, p.r - u.hb * p.rb);
        for (int i = warp; i < u.ntok * heads; i += warps) {
            const int tl = i / heads, hp = i - tl * heads;
            Join<V> j;
            add_pieces<V>(p, u.total, blockIdx.x, u.k0, u.c1, slot_row(p, tl, hp), lane, j);
            j.store(p.out + (static_cast<long long>(u.tok0 + tl) * p.H_q + u.kvh * p.r + u.hb * p.rb + hp) * p.d + lane * V);
        }
    }
    for (int e = blockIdx.x; e < p.P; e += gridDim.x) {
        const Span sp = span_at(p, e, false);
        if (sp.rows > 0) continue;
        const long long n = static_cast<long long>(sp.ntok) * p.H_q * p.d / 4, at = static_cast<long long>(sp.tok0) * p.H_q * p.d / 4;
        for (long long i = blockIdx.y * 256 + threadIdx.x; i < n; i += gridDim.y * 256)
            reinterpret_cast<float4 *>(p.out)[at + i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

template <class... K, class... A>
int launch(void (*kern)(K...), dim3 grid, cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace

int launch_span_merge(const SpanParams &shared, const SpanParams &own, cudaStream_t stream) {
    const SpanParams &p = shared;
    if (own.B > 0) {
        const dim3 grid(p.N, p.H_kv);
        return p.d == 128 ? launch(span_merge_shared_kernel<4>, grid, stream, p, own) : launch(span_merge_shared_kernel<2>, grid, stream, p, own);
    }
    // A cut unit's rows: with few of them a warp or two each, with 256 enough warps that each has one or two.
    const dim3 grid(p.G, p.unit_rows <= 16 ? 1 : p.unit_rows / 16);
    return p.d == 128 ? launch(span_merge_cross_kernel<4>, grid, stream, p) : launch(span_merge_cross_kernel<2>, grid, stream, p);
}

}  // namespace gqa
