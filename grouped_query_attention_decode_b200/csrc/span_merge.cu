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

// Shared and own rows: one block per (token, key/value head, head block), a warp per query head.
template <int V>
__global__ void __launch_bounds__(256) span_merge_shared_kernel(const __grid_constant__ SpanParams p) {
    grid_dependency_wait();
    const int tok = blockIdx.x, kh = blockIdx.y, kvh = kh / p.HB, hb = kh - kvh * p.HB;
    const int b = tok / p.Q;
    const int lane = threadIdx.x & 31;
    // the token's unit in its group's span and in its own, with the pieces of each
    __shared__ int4 info[2];
    __shared__ int tl_s[2], tiles_s[2], valid_s;
    __shared__ long long total_s;
    if (threadIdx.x == 0) {
        int row0, rows, g = group_of(p, b);
        bool valid = own_rows_of(p, b, row0, rows);
        tiles_s[0] = 0;
        if (g >= 0) {
            const Span sp = span_at(p, g, false);
            const int n = shared_rows_of(p, g);
            valid = valid && n >= 0;
            if (tok >= sp.tok0 && tok < sp.tok0 + sp.ntok && n > 0) {
                const int block = (tok - sp.tok0) / p.blk;
                tiles_s[0] = tiles_of(n, p.T);
                tl_s[0] = tok - sp.tok0 - block * p.blk;
                info[0] = unit_pieces_of(p, unit_number(p, g, sp.tok0, block, kvh, hb));
            }
        }
        const int j = tok - b * p.Q, block = j / p.blk;
        tiles_s[1] = tiles_of(rows, p.T);
        tl_s[1] = j - block * p.blk;
        if (rows > 0) info[1] = unit_pieces_of(p, unit_number(p, p.P + b, 0, block, kvh, hb));
        valid_s = valid;
        total_s = __ldcg(&p.rec->total);
    }
    __syncthreads();
    const int heads = min(p.rb, p.r - hb * p.rb);
    for (int hp = threadIdx.x >> 5; hp < heads; hp += 8) {
        const long long row = static_cast<long long>(tok) * p.H_q + kvh * p.r + hb * p.rb + hp;
        Join<V> j;
        if (valid_s) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (tiles_s[c] == 0) continue;
                const int4 u = info[c];
                if (u.x == u.z) {
                    const long long rr = (c == 0 ? 0 : static_cast<long long>(p.N) * p.H_q) + row;
                    const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p.res_ml) + rr);
                    j.add(ml.x, ml.y, __ldcg(reinterpret_cast<const typename Vec<V>::type *>(p.res + rr * p.d) + lane));
                } else {
                    add_pieces<V>(p, total_s, u.x, u.y, u.z, slot_row(p, tl_s[c], hp), lane, j);
                }
            }
        }
        j.store(p.out + row * p.d + lane * V);
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

template <class K>
int launch(K kern, dim3 grid, const SpanParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace

int launch_span_merge(const SpanParams &p, cudaStream_t stream) {
    if (p.B > 0) {
        const dim3 grid(p.N, p.H_kv * p.HB);
        return p.d == 128 ? launch(span_merge_shared_kernel<4>, grid, p, stream) : launch(span_merge_shared_kernel<2>, grid, p, stream);
    }
    const dim3 grid(p.G, 4);
    return p.d == 128 ? launch(span_merge_cross_kernel<4>, grid, p, stream) : launch(span_merge_cross_kernel<2>, grid, p, stream);
}

}  // namespace gqa
