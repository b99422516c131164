// Joins the pieces that the span kernels left in the workspace (spans.cuh): with pieces c of a
// row's attended rows, each an unnormalised sum o_c, its reference m_c and l_c,
//     M = max_c m_c,  out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c.
// Eight lanes per query row.
#include <cstdint>

#include "device.cuh"
#include "gqa.h"
#include "spans.cuh"

namespace gqa {

namespace {

// A row's running join, eight lanes a row: lane `sub` holds the columns 32 k + 4 sub .. + 3.
template <int D>
struct Join {
    static constexpr int NV = D / 32;
    float M = -INFINITY, L = 0.f;
    float4 o[NV] = {};

    __device__ __forceinline__ void add(float2 ml, const float4 (&x)[NV]) {
        const float top = fmaxf(M, ml.x);
        // a piece in which the row saw nothing weighs nothing, and its sum is not looked at
        const float a = M == -INFINITY ? 0.f : ex2_approx(M - top), b = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top);
        M = top;
        L = L * a + ml.y * b;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            o[k].x = o[k].x * a + (b == 0.f ? 0.f : x[k].x * b);
            o[k].y = o[k].y * a + (b == 0.f ? 0.f : x[k].y * b);
            o[k].z = o[k].z * a + (b == 0.f ? 0.f : x[k].z * b);
            o[k].w = o[k].w * a + (b == 0.f ? 0.f : x[k].w * b);
        }
    }
    __device__ __forceinline__ void store(float *dst, int sub) const {
        const float inv = L > 0.f || L != L ? 1.f / L : 0.f;  // no rows at all: zeros
#pragma unroll
        for (int k = 0; k < NV; ++k)
            *reinterpret_cast<float4 *>(dst + 32 * k + 4 * sub) = make_float4(o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv);
    }
};

// Threads of a row: eight for each of `parts` shares of its pieces, 1, 4 (a warp) or 16 (a team of
// four warps).  The sum of the shares, in the first eight threads.
constexpr int kTeam = 128;
template <int D>
struct TeamSums {
    float2 ml[256 / kTeam][3][8];
    float4 o[256 / kTeam][3][8][D / 32];
};
__device__ __forceinline__ void team_sync() {
    if (threadIdx.x < kTeam) asm volatile("bar.sync 1, 128;" ::: "memory");
    else asm volatile("bar.sync 2, 128;" ::: "memory");
}
template <int D>
__device__ __forceinline__ void join_parts(Join<D> &j, int parts, TeamSums<D> &sums) {
    constexpr int NV = D / 32;
    if (parts == 1) return;
#pragma unroll 1
    for (int x = 8; x <= 16; x <<= 1) {
        float4 o[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k)
            o[k] = make_float4(__shfl_xor_sync(kFullMask, j.o[k].x, x), __shfl_xor_sync(kFullMask, j.o[k].y, x),
                               __shfl_xor_sync(kFullMask, j.o[k].z, x), __shfl_xor_sync(kFullMask, j.o[k].w, x));
        j.add(make_float2(__shfl_xor_sync(kFullMask, j.M, x), __shfl_xor_sync(kFullMask, j.L, x)), o);
    }
    if (parts == 4) return;
    const int team = threadIdx.x / kTeam, w = threadIdx.x % kTeam / 32, lane = threadIdx.x & 31;
    if (w > 0 && lane < 8) {
        sums.ml[team][w - 1][lane] = make_float2(j.M, j.L);
#pragma unroll
        for (int k = 0; k < NV; ++k) sums.o[team][w - 1][lane][k] = j.o[k];
    }
    team_sync();
    if (w == 0 && lane < 8) {
#pragma unroll 1
        for (int i = 0; i < 3; ++i) j.add(sums.ml[team][i][lane], sums.o[team][i][lane]);
    }
    team_sync();  // the sums may be overwritten
}

// Adds row `srow` of the pieces c0 + part, c0 + part + parts, ... of a cut unit's c0 .. c1, two
// pieces' reads in flight at a time.  (Short code: it runs once, and every 8 instructions are a
// fetch.)
template <int D>
__device__ __forceinline__ void add_pieces(const SpanParams &p, int c0, int k0, int c1, int srow, int sub, int part, int parts,
                                           Join<D> &j) {
    constexpr int NV = D / 32, AT_ONCE = 2;
    const int ml_at = p.unit_rows * D + 2 * srow, o_at = srow * D + 4 * sub;
#pragma unroll 1
    for (int c = c0 + part; c <= c1; c += AT_ONCE * parts) {
        float2 ml[AT_ONCE];
        float4 x[AT_ONCE][NV];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const int cc = c + u * parts;
            if (cc <= c1) {
                const float *at = p.slots + (2ll * cc + (cc == c0 ? k0 : 0)) * p.slot_floats;
                ml[u] = __ldcg(reinterpret_cast<const float2 *>(at + ml_at));
#pragma unroll
                for (int k = 0; k < NV; ++k) x[u][k] = __ldcg(reinterpret_cast<const float4 *>(at + o_at + 32 * k));
            }
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u)
            if (c + u * parts <= c1) j.add(ml[u], x[u]);
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

// Row `row` (token tok, head h of its group) of span sp of a launch, added to the join.
template <int D>
__device__ __forceinline__ void add_span(const SpanParams &p, int s, const Span &sp, int tok, int kvh, int h, long long row, bool own,
                                         int sub, int part, int parts, Join<D> &j) {
    const int hb = h / p.rb, tl = tok - sp.tok0, block = tl / p.blk;
    const int4 u = unit_pieces_of(p, unit_number(p, s, sp, block, kvh, hb));
    if (u.x == u.z) {
        if (part != 0) return;
        const long long rr = (own ? static_cast<long long>(p.N) * p.H_q : 0) + row;
        float4 x[D / 32];
        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p.res_ml) + rr);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) x[k] = __ldcg(reinterpret_cast<const float4 *>(p.res + rr * D + 32 * k + 4 * sub));
        j.add(ml, x);
    } else {
        add_pieces<D>(p, u.x, u.y, u.z, slot_row(p, tl - block * p.blk, h - hb * p.rb), sub, part, parts, j);
    }
}

// Shared and own rows, 8 * parts threads per (token, query head).  p0 is the launch over the shared
// spans, p1 the one over the own ones.  What bounds it is the chain of reads -- group, lengths,
// pieces of the unit, the pieces -- so nothing is looked up by one thread for others.
template <int D>
__global__ void __launch_bounds__(256, 3) span_merge_shared_kernel(const __grid_constant__ SpanParams p0, const __grid_constant__ SpanParams p1, int parts) {
    __shared__ TeamSums<D> sums;
    grid_dependency_wait();
    const int sub = threadIdx.x & 7, part = (threadIdx.x >> 3) & (parts - 1);
    const long long row = (static_cast<long long>(blockIdx.x) * 32 + (threadIdx.x >> 3)) / parts;
    if (row >= static_cast<long long>(p0.N) * p0.H_q) return;  // all threads of a row
    const int tok = static_cast<int>(row / p0.H_q), head = static_cast<int>(row - static_cast<long long>(tok) * p0.H_q);
    const int kvh = head / p0.r, h = head - kvh * p0.r;
    const int b = tok / p0.Q;
    const int n = __ldg(p1.lens + b);
    const int g = group_of(p0, b);
    Span sg = {0, 0, 0, 0, 0}, so = {b * p0.Q, p0.Q, 0, 0, 0};
    bool valid = true;
    if (g >= 0) {
        sg = span_at(p0, g, false, false);  // a row that is valid has a holder in its group: its sequence
        valid = shared_rows_of(p0, g) >= 0;
        if (p1.own_after) so.row0 = max(sg.rows, 0);
        if (tok < sg.tok0 || tok >= sg.tok0 + sg.ntok) sg.rows = 0;  // a group whose start is out of range
    }
    // as own_rows_of; an empty sequence of a paged cache attends nothing, shared rows neither
    valid = valid && !(p1.own_after && n == 0) && n >= so.row0 && n <= p1.own_max && (p1.Q == 1 || n - so.row0 >= p1.Q);
    so.rows = n - so.row0;
    Join<D> j;
    if (valid && sg.rows > 0) add_span<D>(p0, g, sg, tok, kvh, h, row, false, sub, part, parts, j);
    if (valid && so.rows > 0) add_span<D>(p1, p1.P + b, so, tok, kvh, h, row, true, sub, part, parts, j);
    join_parts(j, parts, sums);
    if (part == 0) j.store(p0.out + row * D, sub);
}

// Cross attention.  `slices` warps (a multiple of a team's four) belong to each worker and join the
// rows of the cut unit that starts in it, four rows at a time.  SPREAD: a cut unit's rows are divided
// over the warps of all the workers that have a piece of it, so the more pieces there are to join, the
// more warps join them.  Tokens whose encoder sequence has no states get zeros.
template <int D, bool SPREAD>
__global__ void __launch_bounds__(256, 3) span_merge_cross_kernel(const __grid_constant__ SpanParams p, int slices) {
    __shared__ TeamSums<D> sums;  // SPREAD
    grid_dependency_wait();
    const int sub = threadIdx.x & 7, warp = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int worker = warp / slices, slice = warp - worker * slices;
    if (worker < p.G) {
        SpanRecord u = p.rec[worker];
        const int cont = SPREAD ? u.cont : -1;
        int c0 = worker;
#pragma unroll 1
        while (true) {  // the unit that starts here and the one that this worker's first piece goes on with
            if (u.valid) {
                const int heads = min(p.rb, p.r - u.hb * p.rb), rows = u.ntok * heads, n = SPREAD ? u.c1 - c0 + 1 : 1;
                const int parts = !SPREAD ? 1 : rows * 4 <= n * slices ? 16 : rows <= n * slices ? 4 : 1;
                // among the unit's groups of eight threads
                const int group = ((worker - c0) * slices + slice) * 4 + (threadIdx.x >> 3 & 3);
                const int part = group & (parts - 1);
#pragma unroll 1
                for (int i = group / parts; i < rows; i += n * slices * 4 / parts) {
                    const int tl = i / heads, hp = i - tl * heads;
                    Join<D> j;
                    add_pieces<D>(p, c0, u.k0, u.c1, slot_row(p, tl, hp), sub, part, parts, j);
                    if constexpr (SPREAD) join_parts(j, parts, sums);
                    if (part == 0)
                        j.store(p.out + (static_cast<long long>(u.tok0 + tl) * p.H_q + u.kvh * p.r + u.hb * p.rb + hp) * D, sub);
                }
            }
            if (cont < 0 || c0 == cont) break;
            c0 = cont;
            u = p.rec[c0];
        }
    }
    for (int e = blockIdx.x; e < p.P; e += gridDim.x) {
        const Span sp = span_at(p, e, false);
        if (sp.rows > 0) continue;
        const long long n = static_cast<long long>(sp.ntok) * p.H_q * D / 4, at = static_cast<long long>(sp.tok0) * p.H_q * D / 4;
        for (long long i = threadIdx.x; i < n; i += 256) reinterpret_cast<float4 *>(p.out)[at + i] = make_float4(0.f, 0.f, 0.f, 0.f);
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
        // With few rows the shared spans are cut into many pieces (19 for 16 sequences over 8
        // key/value heads: 14 us by eight lanes a row, 9 by a warp; 148 for 2 sequences under one
        // prompt of 4096 rows: the call takes 32 us by a warp, 20 by a team) and there are SMs enough;
        // 8192 rows of few pieces take 11 us by eight lanes and 19 by a warp.
        const long long rows = static_cast<long long>(p.N) * p.H_q;
        const int parts = rows <= 512 ? 16 : rows <= 2048 ? 4 : 1;
        const dim3 grid(static_cast<unsigned>((rows * parts + 31) / 32));
        return p.d == 128 ? launch(span_merge_shared_kernel<128>, grid, stream, p, own, parts) : launch(span_merge_shared_kernel<64>, grid, stream, p, own, parts);
    }
    // Warps that take a full unit's rows at once: a multiple of four, as unit_rows is 16 times something.
    const int slices = p.unit_rows / 4;
    const dim3 grid(static_cast<unsigned>((static_cast<long long>(p.G) * slices + 7) / 8));
    if (p.spread)
        return p.d == 128 ? launch(span_merge_cross_kernel<128, true>, grid, stream, p, slices) : launch(span_merge_cross_kernel<64, true>, grid, stream, p, slices);
    return p.d == 128 ? launch(span_merge_cross_kernel<128, false>, grid, stream, p, slices) : launch(span_merge_cross_kernel<64, false>, grid, stream, p, slices);
}

}  // namespace gqa
