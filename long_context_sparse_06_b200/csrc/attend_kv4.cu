// attend_kv4.cu -- shared-KV MQA over a paged cache held in 4 bits (CSA sparse; HCA dense).
//
// "DeepSeek V4 深度解析" §2, CSA step 3 and HCA paragraph (the attention), §4 (the cache in
// blocks).  For query (b,q) and head h, over the compressed rows and the window rows R
// that the query sees:
//   o_h = sum_r softmax_r(scale * q_h . K_r) V_r,   V_r = the d_c content dims of K_r.
// A compressed row is stored as E2M1 codes with an E4M3 scale per 32 content dims and bf16
// RoPE dims (LCS_KV_FP4); entry e of request b lies in block table[b][e / be], row e mod be.
#include <utility>

#include "lcs_common.cuh"
#include "lcs_internal.h"

namespace lcs {

namespace {

// Loads that stay where they are written: a plain __ldg may be moved down to its first use, behind the
// barriers and waits that it should have run under.
__device__ __forceinline__ int64_t ld_now(const int64_t* p) {
    int64_t v;
    asm volatile("ld.global.nc.s64 %0, [%1];" : "=l"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ int32_t ld_now(const int32_t* p) {
    int32_t v;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld_now(const uint2* p) {
    uint2 v;
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 ld_now(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// What query g of request b is told about its rows: loads that depend on nothing, asked for together.
struct Kv4Query {
    int64_t n, pos, win;   // n_entries; q_pos; win_pos0 (causal) or n_win
};
__device__ __forceinline__ Kv4Query kv4_query(const AttendKv4Args& a, int64_t g, int64_t b) {
    Kv4Query x{ld_now(a.n_entries + b), 0, a.Tw};
    if (a.q_pos != nullptr) x.pos = ld_now(a.q_pos + g), x.win = ld_now(a.win_pos0 + b);
    else if (a.n_win != nullptr) x.win = ld_now(a.n_win + b);
    return x;
}

// Entries of the request that exist: n_entries, within what the table can hold.
__device__ __forceinline__ int64_t kv4_entries(const AttendKv4Args& a, const Kv4Query& x, int* status) {
    int64_t n = x.n;
    const int64_t most = a.max_blocks * a.be;
    if (n > most) {
        set_status(status, LCS_ERR_DEVICE, 601);
        n = most;
    }
    return n < 0 ? 0 : n;
}

// Entries that an HCA query attends.
__device__ __forceinline__ int64_t kv4_avail(const AttendKv4Args& a, const Kv4Query& x, int64_t n) {
    if (a.q_pos == nullptr) return n;
    const int64_t p = x.pos < 0 ? 0 : (x.pos < INT64_MAX ? x.pos + 1 : x.pos);   // (no sum past 64 bits)
    // nearly always of 32 bits, where the division is several times cheaper
    const int64_t av = (p >> 31) == 0 ? (int64_t)((uint32_t)p / (uint32_t)a.m) : p / a.m;
    return av < n ? av : n;
}

struct Kv4Window {
    int64_t lo, n;
};
__device__ __forceinline__ Kv4Window kv4_window(const AttendKv4Args& a, const Kv4Query& x) {
    Kv4Window w{0, x.win < 0 ? 0 : (x.win < a.Tw ? x.win : a.Tw)};
    if (a.q_pos == nullptr) return w;
    // the query's own row, counted from the window's first: none if it lies before that, or so far past it that the
    // difference takes the 64th bit
    int64_t hi = x.pos < x.win ? -1 : (int64_t)((uint64_t)x.pos - (uint64_t)x.win);
    int64_t lo = hi < 0 ? 0 : hi - a.W + 1;
    if (lo < 0) lo = 0;
    if (hi > a.Tw - 1) hi = a.Tw - 1;
    w.lo = lo;
    w.n = hi >= lo ? hi - lo + 1 : 0;
    return w;
}

// Row of entry e (0 <= e < kv4_entries) of request b, or null when its block is not one of the
// pool's.
__device__ __forceinline__ const uint8_t* kv4_row(const AttendKv4Args& a, int64_t b, int e) {
    const int bi = e / a.be;
    const int32_t id = __ldg(a.table + b * a.max_blocks + bi);
    if (id < 0 || id >= a.n_blocks) return nullptr;
    return a.pool + ((int64_t)id * a.be + (e - bi * a.be)) * a.row_bytes;
}

// ------------------------------------------------------------ CUDA-core path
// Every shape: H <= 128, d_c % 32 == 0 and <= 512, d_r <= 128, fp32 or bf16 queries.  A CTA serves one
// query and group of 8 heads (and one of the splits of its rows, which form a cluster); its warps work
// alone, each on 16 rows at a time with an online softmax of its own, and join their partials at the
// end.  Shared-memory reads are what it runs out of, so both products reuse what they read:
//   S: a lane holds rows r, r + 8 and two heads; a warp's read of 4 dims is 8 rows and 8 heads, each
//      once (a pitch of D + 4 floats puts the eight on different banks) for 512 multiply-adds;
//   O: a lane holds 4 dims of 8 / G heads, kPass times 128 / G dims apart; a row's dims are read once for
//      all of them, its weights in one or two 16-byte broadcasts.
// (A CTA that stepped through 64 rows together, a warp per head, read each row eight times.)  Measured,
// before and now: 1024 causal fp32 queries of 8 heads, 64 + 16 dims, 192 rows each 58.6 and 32.1 us
// (without S 22, without O 26, without the window's copies 29); one fp32 query of 64 heads, 512 + 64
// dims, over 8320 rows 3251 and 184 us (clusters of 8); 128 such queries of 328 rows 1271 and 546 us.
// Registers: 64 a thread for up to 128 dims (80: 34.4 us); packed fp32 pairs halve the multiply-adds.
constexpr int kSRows = 16, kSHeads = 8;
constexpr int kSMaxCluster = 8;

__device__ __forceinline__ float4 axpy4(float p, float4 v, float4 o) {
    return make_float4(fmaf(p, v.x, o.x), fmaf(p, v.y, o.y), fmaf(p, v.z, o.z), fmaf(p, v.w, o.w));
}
__device__ __forceinline__ float4 scale4(float4 v, float f) { return make_float4(v.x * f, v.y * f, v.z * f, v.w * f); }
// Eight bf16 -> eight floats.
__device__ __forceinline__ void put_bf16x8(float* o, uint4 w) {
    reinterpret_cast<float4*>(o)[0] = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                                                  __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
    reinterpret_cast<float4*>(o)[1] = make_float4(__uint_as_float(w.z << 16), __uint_as_float(w.z & 0xFFFF0000u),
                                                  __uint_as_float(w.w << 16), __uint_as_float(w.w & 0xFFFF0000u));
}

// Floats of shared memory: q, then per warp its rows, weights and (m, l) of the heads.
__host__ __device__ constexpr int simt_warp_floats(int D) { return kSRows * (D + 4) + kSRows * kSHeads + 2 * kSHeads; }

template <int G, int kPass>
__global__ void __launch_bounds__(256, kPass == 1 ? 4 : 1) attend_kv4_kernel(const AttendKv4Args a, int splits, int* status) {
    extern __shared__ float4 sh4[];
    float* sh = reinterpret_cast<float*>(sh4);
    const int D = a.d_c + a.d_r, pitch = D + 4, c4n = a.d_c / 4;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, nw = blockDim.x >> 5;
    const int wf = simt_warp_floats(D);
    float* qs = sh;                              // [8, D + 4]
    float* rows = qs + kSHeads * pitch + warp * wf;   // [16, D + 4]
    float* wt = rows + kSRows * pitch;           // [16, 8] weights
    float* ml = wt + kSRows * kSHeads;           // [2, 8]: rescaling factors; at the end m and l
    __shared__ int nsel_s;
    __shared__ float joint[2][kSHeads];          // this CTA's m and l
    const int64_t g = blockIdx.x, b = g / a.Q;
    const int h0 = blockIdx.y * kSHeads, nh = min(kSHeads, a.H - h0), sp = blockIdx.z;
    const Kv4Query x = kv4_query(a, g, b);

    for (int i = t; i < kSHeads * (D / 8); i += blockDim.x) {
        const int h = i / (D / 8), c = i - h * (D / 8);
        float* o = qs + h * pitch + 8 * c;
        const int64_t at = (g * a.H + h0 + h) * D + 8 * c;
        if (h >= nh) {
            reinterpret_cast<float4*>(o)[0] = reinterpret_cast<float4*>(o)[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else if (a.q_dtype == LCS_F32) {
            const float4* q4 = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
            reinterpret_cast<float4*>(o)[0] = __ldg(q4);
            reinterpret_cast<float4*>(o)[1] = __ldg(q4 + 1);
        } else {
            put_bf16x8(o, __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at)));
        }
    }
    const int64_t n = kv4_entries(a, x, status);
    const int32_t* sel = a.idx != nullptr ? a.idx + g * a.k : nullptr;
    if (t == 0) nsel_s = sel != nullptr ? a.k : (int)kv4_avail(a, x, n);
    __syncthreads();
    if (sel != nullptr) {
        int bad = a.k;
        for (int i = t; i < a.k && bad == a.k; i += blockDim.x) {
            const int32_t v = __ldg(sel + i);
            if (v < 0 || v >= n) bad = i;
        }
        bad = __reduce_min_sync(0xffffffffu, bad);
        if (lane == 0 && bad < a.k) atomicMin(&nsel_s, bad);
    }
    __syncthreads();
    const int nsel = nsel_s;
    if (sel != nullptr && t == 0 && nsel < a.k && sel[nsel] >= 0) set_status(status, LCS_ERR_DEVICE, 603);
    const Kv4Window win = kv4_window(a, x);
    const int R = nsel + (int)win.n;
    const int my = lane & 15, half = lane >> 4;   // this lane's row of a block, and every other piece of it
    // window rows lie one after the other: pieces of 16 bytes of them, lane + 32 i: row and column
    const int esz = a.q_dtype == LCS_F32 ? 4 : 2, pieces = D * esz / 16;
    const int wr0 = lane / pieces, wc0 = lane - wr0 * pieces, wrs = 32 / pieces, wcs = 32 - wrs * pieces;
    const uint8_t* wrows = static_cast<const uint8_t*>(a.win) + (b * a.Tw + win.lo) * D * esz;
    // address of list row r, a compressed one (null if there is none, or its block is not one of the pool's)
    auto row_at = [&](int r) -> const uint8_t* {
        if (r >= nsel) return nullptr;
        const uint8_t* p = kv4_row(a, b, sel != nullptr ? __ldg(sel + r) : r);
        if (p == nullptr) set_status(status, LCS_ERR_DEVICE, 602);
        return p;
    };
    const int stride = nw * splits * kSRows;
    int r0 = (sp * nw + warp) * kSRows;
    const uint8_t* nxt = row_at(r0 + my);

    constexpr int kH8 = kSHeads / G, kSpan = 32 / G;
    const int grp = lane / kSpan, col = lane % kSpan;
    uint64_t acc[kPass][kH8][2];
#pragma unroll
    for (int i = 0; i < kPass; ++i)
#pragma unroll
        for (int h = 0; h < kH8; ++h) acc[i][h][0] = acc[i][h][1] = 0;
    const int qr = lane & 7, qh = 2 * (lane >> 3);   // scores: rows qr, qr + 8 and heads qh, qh + 1
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // (l: of this lane's rows)
    for (; r0 < R; r0 += stride) {
        const uint8_t* src = nxt;
        nxt = row_at(r0 + stride + my);
        const int nr = min(kSRows, R - r0);
        float* o = rows + my * pitch;
        const int nc = max(0, min(nr, nsel - r0));   // compressed ones of the rows
        if (nc < nr) {
            const uint8_t* w = wrows + (int64_t)(r0 + nc - nsel) * D * esz + 16 * lane;
            int r = nc + wr0, c = wc0;
            while (r < nr) {
                if (a.q_dtype == LCS_F32) cp_async_16(rows + r * pitch + 4 * c, w, true);
                else put_bf16x8(rows + r * pitch + 8 * c, __ldg(reinterpret_cast<const uint4*>(w)));
                w += 512;
                r += wrs, c += wcs;
                if (c >= pieces) c -= pieces, ++r;
            }
            cp_async_commit();
        }
        if (my < nc) {
            for (int c = half; c < a.d_c / 32; c += 2) {   // 32 codes and their scale
                const uint4 w = src != nullptr ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
                const float s = src != nullptr ? e4m3_to_f32(__ldg(src + a.d_c / 2 + 2 * a.d_r + c)) : 0.f;
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t y = x[i >> 1] >> (16 * (i & 1));
                    const float2 u = e2m1x2_to_f32(y), v = e2m1x2_to_f32(y >> 8);
                    reinterpret_cast<float4*>(o + 32 * c)[i] = make_float4(u.x * s, u.y * s, v.x * s, v.y * s);
                }
            }
            for (int c = half; c < a.d_r / 8; c += 2)
                put_bf16x8(o + a.d_c + 8 * c,
                           src != nullptr ? __ldg(reinterpret_cast<const uint4*>(src + a.d_c / 2) + c) : make_uint4(0, 0, 0, 0));
        }
        cp_async_wait<0>();
        __syncwarp();
        float s[2][2];   // [row][head]
        {
            const ulonglong2* qa = reinterpret_cast<const ulonglong2*>(qs + qh * pitch);
            const ulonglong2* qb = reinterpret_cast<const ulonglong2*>(qs + (qh + 1) * pitch);
            const ulonglong2* ra = reinterpret_cast<const ulonglong2*>(rows + qr * pitch);
            const ulonglong2* rb = reinterpret_cast<const ulonglong2*>(rows + (qr + 8) * pitch);
            uint64_t s2[2][2] = {{0, 0}, {0, 0}};
#pragma unroll 4
            for (int c = 0; c < D / 4; ++c) {
                const ulonglong2 u = qa[c], v = qb[c], x = ra[c], y = rb[c];
                s2[0][0] = fma2(u.y, x.y, fma2(u.x, x.x, s2[0][0]));
                s2[0][1] = fma2(v.y, x.y, fma2(v.x, x.x, s2[0][1]));
                s2[1][0] = fma2(u.y, y.y, fma2(u.x, y.x, s2[1][0]));
                s2[1][1] = fma2(v.y, y.y, fma2(v.x, y.x, s2[1][1]));
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 v = unpack2(s2[r][h]);   // (rows past nr hold anything: dropped)
                    s[r][h] = qr + 8 * r < nr ? (v.x + v.y) * a.scale : -INFINITY;
                }
        }
        float p[2][2], al[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float mx = fmaxf(s[0][h], s[1][h]);
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            mx = fmaxf(mx, m[h]);
            al[h] = m[h] == -INFINITY ? 0.f : expf(m[h] - mx);
#pragma unroll
            for (int r = 0; r < 2; ++r) p[r][h] = s[r][h] == -INFINITY ? 0.f : expf(s[r][h] - mx);
            l[h] = fmaf(l[h], al[h], p[0][h] + p[1][h]);
            m[h] = mx;
        }
        *reinterpret_cast<float2*>(wt + qr * kSHeads + qh) = make_float2(p[0][0], p[0][1]);
        *reinterpret_cast<float2*>(wt + (qr + 8) * kSHeads + qh) = make_float2(p[1][0], p[1][1]);
        if (qr == 0) *reinterpret_cast<float2*>(ml + qh) = make_float2(al[0], al[1]);
        __syncwarp();
#pragma unroll
        for (int h = 0; h < kH8; ++h) {
            const uint64_t f = pack2(ml[grp * kH8 + h], ml[grp * kH8 + h]);
#pragma unroll
            for (int i = 0; i < kPass; ++i) acc[i][h][0] = mul2(acc[i][h][0], f), acc[i][h][1] = mul2(acc[i][h][1], f);
        }
#pragma unroll 2
        for (int r = 0; r < nr; ++r) {
            float w[kH8];
            if constexpr (kH8 == 2) {
                const float2 x = *reinterpret_cast<const float2*>(wt + r * kSHeads + 2 * grp);
                w[0] = x.x, w[1] = x.y;
            } else {
#pragma unroll
                for (int h = 0; h < kH8; h += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(wt + r * kSHeads + kH8 * grp + h);
                    w[h] = x.x, w[h + 1] = x.y, w[h + 2] = x.z, w[h + 3] = x.w;
                }
            }
#pragma unroll
            for (int i = 0; i < kPass; ++i) {
                const int c = col + kSpan * i;
                if (c >= c4n) break;
                const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(rows + r * pitch + 4 * c);
#pragma unroll
                for (int h = 0; h < kH8; ++h) {
                    const uint64_t p2 = pack2(w[h], w[h]);
                    acc[i][h][0] = fma2(p2, v.x, acc[i][h][0]);
                    acc[i][h][1] = fma2(p2, v.y, acc[i][h][1]);
                }
            }
        }
        __syncwarp();
    }
    // ---- the warps' partials: O [8, d_c] where their rows were, m and l
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], d);
        if (qr == 0) ml[qh + h] = m[h], ml[kSHeads + qh + h] = l[h];
    }
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
        const int c = col + kSpan * i;
        if (c >= c4n) break;
#pragma unroll
        for (int h = 0; h < kH8; ++h)
            *reinterpret_cast<ulonglong2*>(rows + (grp * kH8 + h) * a.d_c + 4 * c) = make_ulonglong2(acc[i][h][0], acc[i][h][1]);
    }
    __syncthreads();
    // ---- joined over the CTA's warps and written, or (of several splits) left in the first warp's place
    float* base = qs + kSHeads * pitch;
    const int in_ml = kSRows * pitch + kSRows * kSHeads;   // of a warp's floats
    auto out_at = [&](int h, int c, float4 o, float M, float L) {
        const float iv = L != 0.f ? 1.f / L : 0.f;   // (L is 0 where no row was seen; a NaN stays one)
        o = scale4(o, iv);
        const int64_t at = (g * a.H + h0 + h) * a.d_c + 4 * c;
        if (a.out_dtype == LCS_F32) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = o;
        else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(cvt_bf16x2(o.x, o.y), cvt_bf16x2(o.z, o.w));
        if (c == 0 && a.lse != nullptr) a.lse[g * a.H + h0 + h] = L != 0.f ? M + logf(L) : -INFINITY;
    };
    for (int j = t; j < nh * c4n; j += blockDim.x) {
        const int h = j / c4n, c = j - h * c4n;
        float M = -INFINITY, L = 0.f;
        for (int w = 0; w < nw; ++w) M = fmaxf(M, base[w * wf + in_ml + h]);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < nw; ++w) {
            const float* x = base + w * wf;
            const float lw = x[in_ml + kSHeads + h], f = lw != 0.f ? expf(x[in_ml + h] - M) : 0.f;
            L = fmaf(lw, f, L);
            o = axpy4(f, *reinterpret_cast<const float4*>(x + h * a.d_c + 4 * c), o);
        }
        if (splits == 1) out_at(h, c, o, M, L);
        else {
            *reinterpret_cast<float4*>(base + h * a.d_c + 4 * c) = o;
            if (c == 0) joint[0][h] = M, joint[1][h] = L;
        }
    }
    if (splits == 1) return;
    // ---- and over the cluster's CTAs, each a share of the outputs
    __syncwarp();
    cluster_sync_all();
    for (int j = sp * blockDim.x + t; j < nh * c4n; j += splits * blockDim.x) {
        const int h = j / c4n, c = j - h * c4n;
        float M = -INFINITY, L = 0.f;
        for (int s = 0; s < splits; ++s) M = fmaxf(M, ld_dsmem_f32(dsmem_addr(&joint[0][h], s)));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < splits; ++s) {
            const float ls = ld_dsmem_f32(dsmem_addr(&joint[1][h], s));
            const float f = ls != 0.f ? expf(ld_dsmem_f32(dsmem_addr(&joint[0][h], s)) - M) : 0.f;
            L = fmaf(ls, f, L);
            o = axpy4(f, ld_dsmem_f4(dsmem_addr(base + h * a.d_c + 4 * c, s)), o);
        }
        out_at(h, c, o, M, L);
    }
    __syncwarp();
    cluster_sync_all();   // no CTA leaves while its partials are read
}

// Warps per CTA and splits (CTAs of a cluster) per query and group of heads: CTAs of four warps while
// there are enough of them; few ones get eight warps, then up to eight splits, while every warp has rows.
struct SimtPlan {
    int warps, splits;
    size_t smem;
};
SimtPlan simt_plan(const AttendKv4Args& a) {
    const int D = a.d_c + a.d_r;
    const int64_t most_w = a.q_pos == nullptr ? a.Tw : (a.W < a.Tw ? a.W : a.Tw);
    const int64_t blocks = ((a.idx != nullptr ? a.k : a.max_blocks * a.be) + most_w + kSRows - 1) / kSRows;
    const int64_t ctas = a.B * a.Q * ((a.H + kSHeads - 1) / kSHeads);
    const size_t fixed = sizeof(float) * kSHeads * (D + 4), per = sizeof(float) * simt_warp_floats(D), most = 227 * 1024 - 1024;
    SimtPlan p{ctas < num_sms() ? 8 : 4, 1, 0};
    while (p.warps > 1 && (p.warps / 2 >= blocks || fixed + p.warps * per > most)) p.warps /= 2;
    while (p.splits < kSMaxCluster && ctas * p.splits * 2 <= num_sms() && blocks > p.warps * p.splits) p.splits *= 2;
    p.smem = fixed + p.warps * per;
    return p;
}

template <int G, int kPass>
cudaError_t launch_simt(const AttendKv4Args& a, int* status, cudaStream_t s) {
    const SimtPlan p = simt_plan(a);
    auto kern = attend_kv4_kernel<G, kPass>;
    cudaError_t e = set_smem_here(reinterpret_cast<const void*>(kern), p.smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * a.Q), (unsigned)((a.H + kSHeads - 1) / kSHeads), (unsigned)p.splits);
    cfg.blockDim = dim3((unsigned)p.warps * 32);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = (unsigned)p.splits;
    cfg.attrs = attr;
    cfg.numAttrs = p.splits > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a, p.splits, status);
}

// ----------------------------------------------------------- tensor-core path
// bf16 queries, d_c = 512, d_r = 64.  One CTA (18 warps) per (query, tile of 64 heads, split of its
// row list); the row list is the selected or available entries, padded to whole chunks of 48, then
// the window rows; chunk i goes to split i mod splits.
//
//   S [64 heads x 48 rows] = Q [64 x 576] . K_chunk^T,  O [64 x 512] += P [64 x 48] . V_chunk
//
// on tcgen05.mma with the heads as M = 64, fp32 accumulators in TMEM.
//
//  * Widening.  code x scale has at most six significant bits and lies in [2^-10, 2688], so it is
//    exact in fp16: one conversion per pair of codes and one fp16 multiply by the scale, half of what
//    bf16 would take.  Both operands of a kind::f16 MMA have one type, so the content dims of Q are
//    fp16 too, scaled per head by a power of two that puts the head's largest element in
//    [2^14, 2^15) (8 bits: exact from 2^-17 on, 2^-31 of it, below that off by 2^-25, 2^-39 of it), and
//    P is fp16 (11 bits; 2^-11 a weight, against 2^-9 of bf16, or 2^-31 of the largest below 2^-20 of
//    it).  RoPE dims stay bf16: four MMAs of the same accumulation.  Window rows' content goes from
//    bf16 to fp16 as well: exact from 2^-17 (8 bits) to 65280, off by 2^-25 below, where 4-bit rows
//    resolve 2^-10; from 2^16 on, where 4-bit rows end at 2688, it is an error.
//  * Shared memory is what an SM runs out of: its bandwidth (an MMA with both operands in it takes
//    4 KB per 32 cycles) and its size (a chunk is the K-major B of Q.K^T and the MN-major B of P.V).
//    So 384 of Q's dims are an A operand in TMEM, in the lanes of the accumulator they meet: S of
//    even and of odd chunks uses the two halves of every 32 lanes (as O's dims 0-255 and
//    256-511 do), and Q is kept in both.  That leaves room for three stages of 48 rows, each
//    released in two halves of the columns as P.V leaves them: widening, Q.K^T, softmax and P.V of
//    different chunks run side by side (two stages of 64 rows took 3400 cycles per 64 rows, where
//    each step was the others' wait).
//  * Warps 4-9 fill the even chunks, warps 10-15 the odd ones: a warp owns 8 rows and holds its next
//    chunk's 400-byte rows in registers (seven loads a lane), which then have two chunks' time to
//    arrive (one group alone waited 1500 cycles for them, chunk after chunk).  Three of four words of
//    codes are widened by conversions, one by byte permutes (half and half: 279 against 287 us for 1000
//    queries).
//  * Warps 16 and 17 issue the MMAs with the whole warp in step and an elected lane's predicate on
//    the instruction: 35 cycles per M = 64, N = 64 MMA alone on the SM (32 is its rate), where
//    issue from a branch of one thread took 55 to 72.
//  * Every warp but the first group of producers, which fills the first chunk meanwhile, brings in Q,
//    converts it and moves its TMEM part (12 warps: three per quarter of TMEM's lanes).  (Q in one bulk
//    copy: a decode step of 16 x 8320 rows 1.0 us faster with its inputs in L2, 1.9 slower from HBM.)
//  * Warps 0-3 run the online softmax (fp32, exp2).  Weights are kept 2^6 above 1, so that fp16
//    reaches down to 2^-31 of the largest; O is rescaled when a head's maximum grows by more than 2^8.
//
// What a CTA takes, in cycles (hca, 1000 causal queries of 64 heads, 24 chunks each; 269 us in all): 860
// until TMEM is there, 3800 until Q and the row counts are, 5000 for Q's conversion beside the first
// chunk's widening, 1100 into TMEM, 1700 to the first S, 2150 a chunk (its MMAs alone: 1680 at M = 64,
// half the rate of M = 128, which O's 512 columns leave no TMEM for), 4900 for the rest.  csa, 1500 causal
// queries over 1024 selected rows: 2400 a chunk, its rows scattered; 457 us.  Decode steps back to
// back: 16 x 8320 rows 37.6 us, 32 x 640 19.4, one x 8320 20.8, 4 x 1152 15.9, one of 160 rows 13.6.
constexpr int kH = 64, kD = 576, kDv = 512, kChunk = 48, kStages = 3;
constexpr int kBlk = kChunk * 128;            // one SW128 column block of a chunk: 48 rows x 128 B
constexpr int kStageBytes = 9 * kBlk;         // 54 KB
constexpr int kQBlk = kH * 128;               // one SW128 column block of Q
constexpr int kTQ = 384;                      // Q's dims 0 .. kTQ-1 in TMEM, the others in shared memory
constexpr int kQBytes = (9 - kTQ / 64) * kQBlk;
constexpr int kSoftWarps = 4, kProdWarps = 6, kProdGroups = 2;
constexpr int kWarpQK = kSoftWarps + kProdGroups * kProdWarps, kWarpPV = kWarpQK + 1, kTcWarps = kWarpPV + 1;
constexpr int kTcThreads = kTcWarps * 32;
constexpr int kQWarps = kTcWarps - kProdWarps;                // warps that bring in Q
constexpr int kRowsPerWarp = kChunk / kProdWarps;             // rows of a chunk per producer warp
constexpr int kPieces = 32 / kRowsPerWarp;                    // lanes that share a row
static_assert(kRowsPerWarp == 8, "a store's eight lanes hold eight rows: eight bank groups");
constexpr int kHalfBlocks = 4;                // column blocks of a stage's first half
constexpr int kPBytes = kH * 128;             // P: 64 heads x 48 rows, fp16, K-major SW128 rows of 128 B
constexpr size_t kTcSmem = 1024 + kQBytes + kStages * kStageBytes + 2 * kPBytes;
constexpr int kMaxSplits = 64, kMaxCluster = 16;
constexpr int kOPitchF32 = kDv * 4 + 16;      // staged O rows (padded)
constexpr int kOPitchBF16 = kDv * 2 + 16;
static_assert(kH * kOPitchF32 <= kStages * kStageBytes, "staged O fits in the stages");
static_assert(kTQ / 64 * kQBlk <= kStageBytes && kH * 128 == kQBlk, "Q's TMEM part passes through the last stage");
// TMEM columns: O, S (even chunks in lanes 0-15 of each 32, odd ones in lanes 16-31), Q (twice, for
// both halves of the lanes).
constexpr uint32_t kTmS = 256, kTmQ = kTmS + kChunk, kHi16 = 16u << 16;
static_assert(kTmQ + kTQ / 2 <= 512, "TMEM columns");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.0f;              // log2 of the tolerated growth before O is rescaled
constexpr float kLift = 6.0f;                 // log2 of the largest weight when the maximum is current

struct TcBars {
    uint64_t kfull[kStages][2], kempty[kStages][2];   // [stage][half]
    uint64_t sfull[2], sempty[2];             // per chunk parity, like the next two
    uint64_t pfull[2];
    uint64_t ofull[2];                        // P.V of the chunk done
    uint64_t odone;                           // every P.V of this CTA done
    uint64_t qfull;                           // Q is where the MMAs read it
    uint32_t tmem_base;
    int first_bad[kTcWarps];
    float qscale[kH];                         // 2^-e of head h: the true q is the stored one times it
    float inv_l[kH];
};

// One lane of the (converged) warp, the same at every call.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// kind::f16 MMA issued by the elected lane, the whole warp in step.  a, b: the low words of the
// operands' descriptors (address and lbo), hi: their common high word (sbo, version, swizzle).
__device__ __forceinline__ void mma_ss_if(uint32_t on, uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                          uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "mov.b64 da, {%1, %6};\n\t"
        "mov.b64 db, {%2, %6};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(on), "r"(hi)
        : "memory");
}
// The same with A in TMEM (fp16 pairs, row i in the lane of the accumulator's row i).
__device__ __forceinline__ void mma_ts_if(uint32_t on, uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t hi,
                                          uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "mov.b64 db, {%2, %6};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b), "r"(idesc), "r"(acc), "r"(on), "r"(hi)
        : "memory");
}
// The elected lane's commit: arrives once on `bar` when its MMAs so far are complete.
__device__ __forceinline__ void commit_if(uint32_t on, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(on)
        : "memory");
}
// The same instruction descriptor with fp16 operands.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t bf16) { return bf16 & ~((1u << 7) | (1u << 10)); }

// A bounded wait that the whole warp leaves with one answer.  The thread sleeps in the hardware's wait
// (up to the hint, 20 us) instead of polling.  The clock and the workspace's status words are looked at
// after every 16 sleeps: another wait that ran out (whether it or an earlier error is the one recorded) ends
// this one, an error in a request's data does not, since only that request's output may suffer from it.
__device__ __forceinline__ bool mbar_sleep(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __noinline__ bool warp_wait_on(uint64_t* bar, uint32_t parity, int* status, int where) {
    uint64_t t0 = 0;
    for (uint32_t polls = 1;; ++polls) {
        if (__all_sync(0xffffffffu, mbar_sleep(bar, parity))) return true;
        if (polls & 15u) continue;
        const uint64_t now = globaltimer();
        if (t0 == 0) t0 = now;
        const bool late = now - t0 > kWaitBudgetNs;
        volatile int* st = status;
        if (late) {
            set_status(status, LCS_ERR_TIMEOUT, where);
            st[2] = LCS_ERR_TIMEOUT;
        }
        if (__any_sync(0xffffffffu, late || st[0] == LCS_ERR_TIMEOUT || st[2] == LCS_ERR_TIMEOUT)) return false;
    }
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status, int where) {
    if (__all_sync(0xffffffffu, mbar_sleep(bar, parity))) return true;
    return warp_wait_on(bar, parity, status, where);
}
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Two floats -> two fp16 packed (low half = a).
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// Two bf16 -> two fp16: exact from 2^-17 (8 bits above fp16's last, 2^-24) to 65280, off by at most 2^-25
// below, saturating above.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(w & 0xFFFF0000u)), "f"(__uint_as_float(w << 16)));
    return r;
}
// Eight E2M1 codes (low nibble first) times the scale (in both halves) -> eight fp16, exact.  Two
// forms, so that neither pipe carries all of it: with the conversion instruction (16 lanes a
// clock per SM, shared with exp2), and with byte permutes: the high byte of a magnitude's fp16 is
// looked up by its three low bits (the low byte is 0), the sign bits are moved to the bytes' tops.
__device__ __forceinline__ uint4 widen8_cvt(uint32_t w, uint32_t s2) {
    uint32_t a, b, c, d;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
        : "r"(w));
    return make_uint4(f16x2_mul(a, s2), f16x2_mul(b, s2), f16x2_mul(c, s2), f16x2_mul(d, s2));
}
__device__ __forceinline__ uint4 widen8_perm(uint32_t w, uint32_t s2) {
    constexpr uint32_t lo = 0x3E3C3800u, hi = 0x46444240u;   // 0, 0.5, 1, 1.5 | 2, 3, 4, 6
    const uint32_t m = w & 0x77777777u, ws = w << 4;
    const uint32_t r0 = __byte_perm(lo, hi, m) | (__byte_perm(ws, w, 0x5140) & 0x80808080u);
    const uint32_t r1 = __byte_perm(lo, hi, m >> 16) | (__byte_perm(ws, w, 0x7362) & 0x80808080u);
    return make_uint4(f16x2_mul(__byte_perm(r0, 0, 0x1404), s2), f16x2_mul(__byte_perm(r0, 0, 0x3424), s2),
                      f16x2_mul(__byte_perm(r1, 0, 0x1404), s2), f16x2_mul(__byte_perm(r1, 0, 0x3424), s2));
}
// 16 lanes x 32 bits, two column ranges 24 apart: threads 0-15 read lanes base..base+15 at columns
// [c, c+n), threads 16-31 the same lanes at columns [c+24, c+24+n).
__device__ __forceinline__ void tmem_ld16x2_8(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], 24;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16x2_16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], 24;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// The E4M3 scale in byte `at` of w, as fp16 in both halves.
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t w, int at) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
        : "=r"(r)
        : "r"(__byte_perm(w, 0, (uint32_t)at * 0x11u)));
    return r;
}

// A lane's part of row lane % kRowsPerWarp of its warp's rows of a chunk: the 16-byte pieces p =
// lane / kRowsPerWarp + kPieces i of the 16 of codes and the 8 of RoPE dims, and the scales of either
// half of the columns.
struct RawRow {
    uint4 codes[16 / kPieces], rope[8 / kPieces];
    uint2 scales[2];
};

// Split partials lie as the attention's lanes held them: per unit and split 256 rows of 32 lanes x 16
// bytes; row 64 quarter + j holds 4 dims of 16 heads in either half of the output (lane l: head 16
// quarter + (l & 15), dims 4 j .. + 3, + 256 for l >= 16).  One warp merges the R rows of task t (of
// 256 / R): quarter t & 3, j = R (t >> 2) .. + R - 1.  A lane forms its head's weights 2^(m_s - M)
// itself, in split order with a running maximum, S splits' loads in flight.
template <int R, int S>
__device__ __forceinline__ void merge_task(const AttendKv4Args& a, int tiles, int splits, int unit, int t,
                                           const float* part_o, const float* part_ml) {
    const int lane = threadIdx.x & 31, quarter = t & 3, j0 = R * (t >> 2);
    const int g = tiles == 2 ? unit >> 1 : unit, in_tile = 16 * quarter + (lane & 15);
    const int head = (tiles == 2 ? (unit & 1) * kH : 0) + in_tile;
    const float4* src = reinterpret_cast<const float4*>(part_o) + ((int64_t)unit * splits * 256 + 64 * quarter + j0) * 32 + lane;
    const float2* ml = reinterpret_cast<const float2*>(part_ml) + (int64_t)unit * splits * kH + in_tile;
    float M = -INFINITY, L = 0.f;
    float4 acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < splits; s0 += S) {
        float4 v[R][S];
        float2 x[S];
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const int s = min(s0 + k, splits - 1);   // (past the last one: read again, weight 0)
            x[k] = __ldcg(ml + (int64_t)s * kH);
#pragma unroll
            for (int r = 0; r < R; ++r) v[r][k] = __ldcg(src + ((int64_t)s * 256 + r) * 32);
        }
        float m = M;
#pragma unroll
        for (int k = 0; k < S; ++k) m = fmaxf(m, x[k].x);
        const float f = L != 0.f ? exp2f(M - m) : 0.f;
        M = m;
        L *= f;
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = make_float4(acc[r].x * f, acc[r].y * f, acc[r].z * f, acc[r].w * f);
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const float e = s0 + k < splits && x[k].y != 0.f ? exp2f(x[k].x - m) : 0.f;   // no rows, no weight
            L += x[k].y * e;
#pragma unroll
            for (int r = 0; r < R; ++r)
                acc[r] = make_float4(acc[r].x + v[r][k].x * e, acc[r].y + v[r][k].y * e, acc[r].z + v[r][k].z * e,
                                     acc[r].w + v[r][k].w * e);
        }
    }
    if (head >= a.H) return;
    const float iv = L != 0.f ? 1.f / L : 0.f;   // (a NaN stays one)
    const int64_t at = ((int64_t)g * a.H + head) * kDv + (lane < 16 ? 0 : 256) + 4 * j0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float4 o = make_float4(acc[r].x * iv, acc[r].y * iv, acc[r].z * iv, acc[r].w * iv);
        if (a.out_dtype == LCS_F32) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + 4 * r) = o;
        else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at + 4 * r) = make_uint2(cvt_bf16x2(o.x, o.y), cvt_bf16x2(o.z, o.w));
    }
    if (a.lse != nullptr && j0 == 0 && lane < 16)
        a.lse[(int64_t)g * a.H + head] = L != 0.f ? (M + log2f(L)) / kLog2e : -INFINITY;
}

// kCsa: a selection (else every entry).  kJoin: the splits of a unit are a cluster and merge in it.  (Four
// kernels and not one: what a CTA runs once comes cold from beyond the SM's instruction cache.)
template <bool kCsa, bool kJoin>
__global__ void __launch_bounds__(kTcThreads, 1)
    attend_kv4_tc_kernel(const AttendKv4Args a, int tiles, int splits, float* __restrict__ part_o,
                         float* __restrict__ part_ml, int* status) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ TcBars bars;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* q_s = smem;
    uint8_t* stage_s = smem + kQBytes;
    uint8_t* p_s = stage_s + kStages * kStageBytes;

    // values that steer whole warps come from lane 0, so that the compiler keeps them (and what the MMA
    // issue derives from them) in uniform registers
    auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    const int warp = uni(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int unit = splits > 1 ? blockIdx.y : blockIdx.x;   // (query, head tile)
    const int sp = splits > 1 ? blockIdx.x : 0;
    const int g = tiles == 2 ? unit >> 1 : unit;
    const int h0 = tiles == 2 ? (unit & 1) * kH : 0;
    const int nh = min(kH, a.H - h0);
    const int b = a.Q == 1 ? g : (int)((unsigned)g / (unsigned)a.Q);
    const bool producer = warp >= kSoftWarps && warp < kWarpQK;
    const int pg = warp >= kSoftWarps + kProdWarps ? 1 : 0;   // a producer's group, and its place there
    const int pw = warp - kSoftWarps - pg * kProdWarps;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i)
            for (int hf = 0; hf < 2; ++hf) {
                mbar_init(&bars.kfull[i][hf], kProdWarps);
                mbar_init(&bars.kempty[i][hf], 1);
            }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.pfull[i], kSoftWarps);
            mbar_init(&bars.sfull[i], 1);
            mbar_init(&bars.sempty[i], kSoftWarps);
            mbar_init(&bars.ofull[i], 1);
        }
        mbar_init(&bars.odone, 1);
        mbar_init(&bars.qfull, kQWarps);
        fence_barrier_init();
    }
    if (warp == kWarpQK) {
        tmem_alloc(&bars.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uni((int)bars.tmem_base);
#if defined(__CUDA_ARCH__)
    asm volatile("griddepcontrol.wait;" ::: "memory");   // everything above reads no memory of the call
#endif
    // column block k of Q: the first ones pass through the last stage into TMEM
    auto q_block = [&](int k) { return k < kTQ / 64 ? stage_s + (kStages - 1) * kStageBytes + k * kQBlk : q_s + (k - kTQ / 64) * kQBlk; };
    // ---- the loads that nothing waits for, before everything else: the selection (CSA), of which the valid
    // prefix counts, and the producers' first two rows (a group takes every other chunk).  How many entries
    // there are, and which of a chunk's rows are attended (the selection's length), is known later: rows
    // past it are dropped when they are widened ...
    const int32_t* sel = kCsa ? a.idx + (int64_t)g * a.k : nullptr;
    const int held = (int)(a.max_blocks * a.be);   // entries that the table can hold
    auto gcof = [&](int c) -> int { return sp + splits * c; };
    const int my_row = pw * kRowsPerWarp + lane % kRowsPerWarp, my_piece = lane / kRowsPerWarp;
    int e0 = -1, e1 = -1, seen[2] = {0, 0};
    if (producer) {
        const int j0 = gcof(pg) * kChunk + my_row, j1 = gcof(pg + kProdGroups) * kChunk + my_row, lim = kCsa ? a.k : held;
        if (j0 < lim) e0 = kCsa ? ld_now(sel + j0) : j0;
        if (j1 < lim) e1 = kCsa ? ld_now(sel + j1) : j1;
    }
    if (kCsa) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if ((int)threadIdx.x + i * kTcThreads < a.k) seen[i] = ld_now(sel + threadIdx.x + i * kTcThreads);
    }
    // ... and Q as it is, in the SW128 layout (by every warp but the first group of producers, which fills the
    // first chunk meanwhile)
    const Kv4Query x = kv4_query(a, g, b);
    const bool q_warp = !producer || pg != 0;
    const int q_id = warp < kSoftWarps ? warp : warp - kProdWarps;   // 0 .. kQWarps - 1
    if (q_warp) {
        const uint8_t* qg = static_cast<const uint8_t*>(a.q) + ((int64_t)g * a.H + h0) * (kD * 2);
        static_assert(kQWarps * 32 == 384 && kH * 72 % 384 == 0, "twelve pieces a thread, 5 rows and 24 pieces apart");
        int h = (q_id * 32 + lane) / 72, c = (q_id * 32 + lane) - h * 72;
#pragma unroll 1
        for (int i = q_id * 32 + lane; i < kH * 72; i += 384) {
            cp_async_16(q_block(c >> 3) + sw128_off(h, c & 7), qg + (h < nh ? i * 16 : 0), h < nh);
            h += 5, c += 24;
            if (c >= 72) c -= 72, ++h;
        }
        cp_async_commit();
    }
    auto row_of = [&](int c, int lim) -> const uint8_t* {   // this lane's row of local chunk c, null if there is none
        const int j = gcof(c) * kChunk + my_row;
        if (j >= (kCsa ? a.k : lim)) return nullptr;
        const int e = kCsa ? __ldg(sel + j) : j;
        return e >= 0 && e < lim ? kv4_row(a, b, e) : nullptr;
    };
    RawRow raw;
    auto load_half = [&](const uint8_t* src, int hf) {
        const uint4* p = reinterpret_cast<const uint4*>(src) + my_piece;
        if (src != nullptr) {
            raw.scales[hf] = ld_now(reinterpret_cast<const uint2*>(src + 384) + hf);
#pragma unroll
            for (int i = hf * (8 / kPieces); i < (hf + 1) * (8 / kPieces); ++i) raw.codes[i] = ld_now(p + kPieces * i);
            if (hf) {
#pragma unroll
                for (int i = 0; i < 8 / kPieces; ++i) raw.rope[i] = ld_now(p + 16 + kPieces * i);
            }
        }
    };
    const bool in0 = e0 >= 0 && e0 < held, in1 = e1 >= 0 && e1 < held;
    const int b0 = in0 ? e0 / a.be : 0, b1 = in1 ? e1 / a.be : 0;
    const int32_t id0 = in0 ? ld_now(a.table + (int64_t)b * a.max_blocks + b0) : -1;
    const int32_t id1 = in1 ? ld_now(a.table + (int64_t)b * a.max_blocks + b1) : -1;
    const Kv4Window wp = kv4_window(a, x);
    const int64_t n = kv4_entries(a, x, status);
    const int most = kCsa ? a.k : (int)kv4_avail(a, x, n);
    int nsel = most;
    if (kCsa) {   // the selection's valid prefix: a minimum per warp, joined
        int first_bad = a.k;
        auto look = [&](int i, int32_t v) {
            if (i < a.k && (v < 0 || v >= n)) first_bad = min(first_bad, i);
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) look((int)threadIdx.x + i * kTcThreads, seen[i]);
        for (int i = threadIdx.x + 2 * kTcThreads; i < a.k; i += kTcThreads) look(i, __ldg(sel + i));
        first_bad = __reduce_min_sync(0xffffffffu, first_bad);
        if (lane == 0) bars.first_bad[warp] = first_bad;
    }
    const uint8_t *cur = nullptr, *nxt = nullptr;
    if (id0 >= 0 && id0 < a.n_blocks) cur = a.pool + ((int64_t)id0 * a.be + (e0 - b0 * a.be)) * a.row_bytes;
    load_half(cur, 0);
    load_half(cur, 1);
    if (id1 >= 0 && id1 < a.n_blocks) nxt = a.pool + ((int64_t)id1 * a.be + (e1 - b1 * a.be)) * a.row_bytes;
    if (kCsa) {
        __syncthreads();
        for (int i = 0; i < kTcWarps; ++i) nsel = min(nsel, bars.first_bad[i]);
        // an index past the entries ended it; -1 is the padding
        if (threadIdx.x == 0 && nsel < a.k && __ldg(sel + nsel) >= 0) set_status(status, LCS_ERR_DEVICE, 603);
    }
    // this split's chunks, and the compressed ones among them, which come first
    const int ncc_all = (nsel + kChunk - 1) / kChunk, nch_all = ncc_all + (int)((wp.n + kChunk - 1) / kChunk);
    const int nch = uni(sp < nch_all ? (nch_all - sp + splits - 1) / splits : 0);
    const int ncc = uni(sp < ncc_all ? (ncc_all - sp + splits - 1) / splits : 0);
    // window chunk c into its stage: bf16 rows by 16-byte cp.async, pieces my_piece + 4 k of this lane's row, zeros
    // past the last row (all 18 copies unrolled: csa prefill 461 us, 457 with two, whose code is shorter)
    const uint32_t wo0 = sw128_off(my_row, my_piece), wo1 = sw128_off(my_row, my_piece + kPieces);
    auto copy_window = [&](int c, int st) {
        uint8_t* dst = stage_s + st * kStageBytes;
        const int r = (gcof(c) - ncc_all) * kChunk + my_row;
        const bool valid = r < (int)wp.n;
        const uint8_t* src = static_cast<const uint8_t*>(a.win) + (((int64_t)b * a.Tw + wp.lo + (valid ? r : 0)) * kD) * 2 + 16 * my_piece;
#pragma unroll 2
        for (int k = 0; k < 72 / kPieces; ++k)
            cp_async_16(dst + (k >> 1) * kBlk + (k & 1 ? wo1 : wo0), src + 16 * kPieces * k, valid);
        cp_async_commit();
    };
    if (producer && pg >= ncc && pg < nch) copy_window(pg, pg);
    if (q_warp) {
        const uint32_t neg = a.scale < 0.f ? 0x80008000u : 0u;
        auto q_sync = []() { asm volatile("bar.sync 1, %0;" ::"n"(kQWarps * 32) : "memory"); };
        cp_async_wait<0>();
        q_sync();
        // ---- Q scaled by 2^e (and by the sign of the scale) in place, a warp per head; content to fp16
#pragma unroll 1
        for (int h = q_id; h < kH; h += kQWarps) {
            const uint32_t at = sw128_off(h, lane & 7);   // chunks lane, lane + 32, lane + 64
            uint4* x0 = reinterpret_cast<uint4*>(q_block(lane >> 3) + at);
            uint4* x1 = reinterpret_cast<uint4*>(q_block(4 + (lane >> 3)) + at);
            uint4* x2 = reinterpret_cast<uint4*>(q_block(8) + at);
            const uint4 v0 = *x0, v1 = *x1, v2 = *x2;     // (four lanes read each of the last 8 chunks)
            uint32_t m2 = bf16x2_maxabs(bf16x2_maxabs(v0.x, v0.y), bf16x2_maxabs(v0.z, v0.w));
            m2 = bf16x2_maxabs(m2, bf16x2_maxabs(bf16x2_maxabs(v1.x, v1.y), bf16x2_maxabs(v1.z, v1.w)));
            m2 = bf16x2_maxabs(m2, bf16x2_maxabs(bf16x2_maxabs(v2.x, v2.y), bf16x2_maxabs(v2.z, v2.w)));
            const uint32_t mag = __reduce_max_sync(0xffffffffu, max(m2 & 0x7FFFu, (m2 >> 16) & 0x7FFFu));   // bf16 bits
            const int ex = (int)(mag >> 7) - 127;               // of the largest element (subnormals: -127)
            int e = mag == 0 || mag >= 0x7F80u ? 0 : 14 - ex;   // zero, infinite or NaN heads stay as they are
            e = e > 126 ? 126 : e;
            const uint32_t up2 = (uint32_t)(127 + e) * 0x00800080u | neg;
            if (lane == 0) bars.qscale[h] = __uint_as_float((uint32_t)(127 - e) << 23);
            auto half8 = [&](uint4 v) {
                auto half2 = [&](uint32_t w) {
                    w = bf16x2_mul(w, up2);
                    return pack_f16x2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
                };
                return make_uint4(half2(v.x), half2(v.y), half2(v.z), half2(v.w));
            };
            *x0 = half8(v0);
            *x1 = half8(v1);
            if (lane < 8)
                *x2 = make_uint4(bf16x2_mul(v2.x, up2), bf16x2_mul(v2.y, up2), bf16x2_mul(v2.z, up2), bf16x2_mul(v2.w, up2));
        }
        fence_proxy_async_smem();
        q_sync();
        // ---- Q's dims 0 .. kTQ-1 into TMEM, both halves of the lanes: three warps per quarter of the lanes, two
        // column blocks each
        const int rank = warp < kSoftWarps ? 0 : (warp < kWarpQK - 2 ? 1 : 2), head = (warp & 3) * 16 + (lane & 15);
        static_assert(kTQ / 64 == 6 && kWarpQK == 16 && kProdWarps == 6, "warps 0-3, 10-13 and 14-17");
#pragma unroll 1
        for (int k = 2 * rank; k < 2 * rank + 2; ++k) {
            uint4 v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = *reinterpret_cast<const uint4*>(q_block(k) + sw128_off(head, c));
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
                const uint32_t o[8] = {v[c].x, v[c].y, v[c].z, v[c].w, v[c + 1].x, v[c + 1].y, v[c + 1].z, v[c + 1].w};
                tmem_st8(tmem_addr(tmem, (warp & 3) * 32, kTmQ + 32 * k + 4 * c), o);
            }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.qfull);
    }
    auto chunk_valid = [&](int c) -> int {   // rows of local chunk c
        const int gc = gcof(c);
        const int v = c < ncc ? nsel - gc * kChunk : (int)wp.n - (gc - ncc_all) * kChunk;
        return v < kChunk ? v : kChunk;
    };
    const bool only = splits == 1;

    if (warp == kWarpQK) {
        // ---------------- Q.K^T issue
        const uint32_t on = elect_lane();
        constexpr uint32_t id_b = idesc_bf16(64, kChunk, false, false), id_h = idesc_f16(id_b);
        const uint64_t q_desc = sw128_desc(smem_u32(q_s), 16, 1024);
        const uint32_t qa = (uint32_t)q_desc, hi = (uint32_t)(q_desc >> 32);
        const uint32_t ka0 = (uint32_t)sw128_desc(smem_u32(stage_s), 16, 1024);
        int st = 0;
        uint32_t ph = 0;
        if (nch > 0 && warp_wait(&bars.qfull, 0, status, 604)) {
            tc_fence_after();
            for (int c = 0; c < nch; ++c) {
                const uint32_t half = c & 1 ? kHi16 : 0u;
                if (c >= 2 && !warp_wait(&bars.sempty[c & 1], (uint32_t)(((c - 2) >> 1) & 1), status, 605)) break;
                const uint32_t ka = ka0 + (uint32_t)((st * kStageBytes) >> 4);
                const uint32_t d = tmem + kTmS + half, qt = tmem + kTmQ + half;
                auto issue = [&](int s0, int s1) {
#pragma unroll
                    for (int s = s0; s < s1; ++s) {
                        const uint32_t kb = ka + (uint32_t)(((s >> 2) * kBlk + (s & 3) * 32) >> 4);
                        if (s < kTQ / 16) mma_ts_if(on, d, qt + 8 * s, kb, hi, id_h, s ? 1u : 0u);
                        else
                            mma_ss_if(on, d, qa + (uint32_t)((((s >> 2) - kTQ / 64) * kQBlk + (s & 3) * 32) >> 4), kb, hi,
                                      s < 32 ? id_h : id_b, 1u);
                    }
                };
                if (!warp_wait(&bars.kfull[st][0], ph, status, 606)) break;
                tc_fence_after();
                issue(0, 4 * kHalfBlocks);
                if (!warp_wait(&bars.kfull[st][1], ph, status, 607)) break;
                tc_fence_after();
                issue(4 * kHalfBlocks, 36);
                commit_if(on, &bars.sfull[c & 1]);
                if (++st == kStages) st = 0, ph ^= 1;
            }
        }
    } else if (warp == kWarpPV) {
        // ---------------- P.V issue (its own warp: it never waits behind the next Q.K^T's rows)
        const uint32_t on = elect_lane();
        constexpr uint32_t id = idesc_f16(idesc_bf16(64, 256, false, true));
        const uint64_t v_desc = sw128_desc(smem_u32(stage_s), kBlk, 1024);
        const uint32_t va0 = (uint32_t)v_desc, hi = (uint32_t)(v_desc >> 32);
        const uint32_t pa0 = (uint32_t)sw128_desc(smem_u32(p_s), 16, 1024);
        int st = 0;
        for (int c = 0; c < nch; ++c) {
            if (!warp_wait(&bars.pfull[c & 1], (uint32_t)((c >> 1) & 1), status, 608)) break;
            tc_fence_after();
            const uint32_t va = va0 + (uint32_t)((st * kStageBytes) >> 4);
            const uint32_t pa = pa0 + (uint32_t)(((c & 1) * kPBytes) >> 4);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int kk = 0; kk < kChunk / 16; ++kk)
                    mma_ss_if(on, tmem + (half ? kHi16 : 0u), pa + (uint32_t)((kk * 32) >> 4),
                              va + (uint32_t)((half * kHalfBlocks * kBlk + kk * 2048) >> 4), hi, id, (c | kk) ? 1u : 0u);
                // dims 0-255 read column blocks 0-3; blocks 4-8 are released after the rest
                commit_if(on, &bars.kempty[st][half]);
            }
            commit_if(on, &bars.ofull[c & 1]);
            if (++st == kStages) st = 0;
        }
        if (nch > 0) commit_if(on, &bars.odone);
    } else if (producer) {
        // ---------------- producers: this group's chunks in order
        int st = pg;
        uint32_t ph = 1;   // of the stage's last release
        for (int c = pg; c < nch; c += kProdGroups) {
            uint8_t* dst = stage_s + st * kStageBytes;
            // Q's TMEM part leaves the last stage before its first rows come in
            if (c == kStages - 1 && !warp_wait(&bars.qfull, 0, status, 613)) break;
            if (c >= ncc) {
                // window chunk: bf16 rows by 16-byte cp.async, zeros past the last row; content to fp16 in place
                if (c >= kStages && (!warp_wait(&bars.kempty[st][0], ph, status, 609) ||
                                     !warp_wait(&bars.kempty[st][1], ph, status, 610)))
                    break;
                if (c != pg) copy_window(c, st);   // the first is on its way
                cp_async_wait<0>();
                uint32_t m2 = 0;
#pragma unroll 4
                for (int k = 0; k < 64 / kPieces; ++k) {   // a lane's own copies
                    uint4* x = reinterpret_cast<uint4*>(dst + (k >> 1) * kBlk + (k & 1 ? wo1 : wo0));
                    const uint4 v = *x;
                    m2 = bf16x2_maxabs(m2, bf16x2_maxabs(bf16x2_maxabs(v.x, v.y), bf16x2_maxabs(v.z, v.w)));
                    *x = make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z), bf16x2_to_f16x2(v.w));
                }
                // a magnitude of 2^16 or more does not fit
                if (max(m2 & 0x7FFFu, (m2 >> 16) & 0x7FFFu) >= 0x4780u) set_status(status, LCS_ERR_DEVICE, 614);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars.kfull[st][0]);
                    mbar_arrive(&bars.kfull[st][1]);
                }
            } else {
                const bool attended = my_row < chunk_valid(c);
                if (attended && cur == nullptr) set_status(status, LCS_ERR_DEVICE, 602);
                const bool live = attended && cur != nullptr;
                bool ok = true;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    if (c >= kStages && !warp_wait(&bars.kempty[st][hf], ph, status, 611 + hf)) {
                        ok = false;
                        break;
                    }
                    // piece p: codes 32 p .. 32 p + 31, 16-byte chunks 4 (p & 1) .. + 3 of column block p / 2
#pragma unroll
                    for (int i = hf * (8 / kPieces); i < (hf + 1) * (8 / kPieces); ++i) {
                        const int p = my_piece + kPieces * i;
                        const uint32_t sw = i & 1 ? raw.scales[hf].y : raw.scales[hf].x;
                        const uint32_t s2 = live ? scale_f16x2(sw, my_piece) : 0u;
                        const uint4 cv = live ? raw.codes[i] : make_uint4(0, 0, 0, 0);
                        uint8_t* blk = dst + (p >> 1) * kBlk;
                        const int ch = 4 * (p & 1);
                        *reinterpret_cast<uint4*>(blk + sw128_off(my_row, ch)) = widen8_cvt(cv.x, s2);
                        *reinterpret_cast<uint4*>(blk + sw128_off(my_row, ch + 1)) = widen8_cvt(cv.y, s2);
                        *reinterpret_cast<uint4*>(blk + sw128_off(my_row, ch + 2)) = widen8_cvt(cv.z, s2);
                        *reinterpret_cast<uint4*>(blk + sw128_off(my_row, ch + 3)) = widen8_perm(cv.w, s2);
                    }
                    if (hf) {
#pragma unroll
                        for (int i = 0; i < 8 / kPieces; ++i)
                            *reinterpret_cast<uint4*>(dst + 8 * kBlk + sw128_off(my_row, my_piece + kPieces * i)) =
                                live ? raw.rope[i] : make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.kfull[st][hf]);
                    // this half's registers are free: the group's next chunk's rows are asked for at once (asked for after
                    // both halves, they came 2000 cycles after the group was ready for them)
                    if (c + kProdGroups < ncc) load_half(nxt, hf);
                }
                if (!ok) break;
                cur = nxt;   // and where the rows of the one after lie
                if (c + 2 * kProdGroups < ncc) nxt = row_of(c + 2 * kProdGroups, (int)(kCsa ? n : most));
            }
            if ((st += kProdGroups) >= kStages) st -= kStages, ph ^= 1;
        }
        cp_async_wait<0>();
    } else {
        // ---------------- softmax: warp w owns heads 16w .. + 15; lane l works on head 16w + (l & 15)
        const int head = warp * 16 + (lane & 15), hi16 = lane >> 4;
        float m_used = -INFINITY, l_sum = 0.f;   // log2 domain; weights are 2^(s - m_used + kLift)
        const float sl2 = fabsf(a.scale) * kLog2e * bars.qscale[head];
        for (int c = 0; c < nch; ++c) {
            const int pb = c & 1;
            if (!warp_wait(&bars.sfull[pb], (uint32_t)((c >> 1) & 1), status, 620)) break;
            tc_fence_after();
            // S columns 0-23 (lanes 0-15) or 24-47 (lanes 16-31) of this lane's head
            uint32_t sv[24];
            const uint32_t ts = tmem_addr(tmem, warp * 32 + 16 * pb, kTmS);
            tmem_ld16x2_16(ts, sv);
            tmem_ld16x2_8(ts + 16, sv + 16);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.sempty[pb]);
            // (scale and 2^-e are not negative: the maximum of the scores is that of s, times them)
            const int valid = chunk_valid(c) - 24 * hi16;
            if (valid < 24) {
#pragma unroll
                for (int j = 0; j < 24; ++j)
                    if (j >= valid) sv[j] = 0xFF800000u;   // -inf: no part of the maximum
            }
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 24; ++j) mx4[j & 3] = fmaxf(mx4[j & 3], __uint_as_float(sv[j]));
            float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)) * sl2;
            float alpha = 1.f;
            bool rescale = false;
            if (mx > m_used + kRescale || m_used == -INFINITY) {
                const float m_new = fmaxf(mx, m_used);
                alpha = (m_used == -INFINITY) ? 0.f : exp2f(m_used - m_new);
                rescale = (c > 0);
                m_used = m_new;
            }
            const float off = m_used == -INFINITY ? 0.f : m_used - kLift;   // every score -inf: weights 0
#pragma unroll
            for (int j = 0; j < 24; ++j) sv[j] = __float_as_uint(ex2(fmaf(__uint_as_float(sv[j]), sl2, -off)));
            if (valid < 24) {   // columns past the chunk's rows weigh nothing (0 times -inf above is no number)
#pragma unroll
                for (int j = 0; j < 24; ++j)
                    if (j >= valid) sv[j] = 0u;
            }
            float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 24; ++j) ps[j & 3] += __uint_as_float(sv[j]);
            // P goes where P.V of chunk c - 2 read it
            if (c >= 2 && !warp_wait(&bars.ofull[pb], (uint32_t)(((c - 2) >> 1) & 1), status, 623)) break;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                uint32_t pk[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    pk[q] = pack_f16x2(__uint_as_float(sv[8 * k + 2 * q]), __uint_as_float(sv[8 * k + 2 * q + 1]));
                *reinterpret_cast<uint4*>(p_s + pb * kPBytes + sw128_off(head, 3 * hi16 + k)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
            if (__any_sync(0xffffffffu, rescale)) {
                // O may be written once the previous chunk's P.V is done
                if (!warp_wait(&bars.ofull[pb ^ 1], (uint32_t)(((c - 1) >> 1) & 1), status, 621)) break;
                tc_fence_after();
                const float f = rescale ? alpha : 1.f;
#pragma unroll 1
                for (int j = 0; j < 256 / 16; ++j) {
                    uint32_t ov[16];
                    const uint32_t ta = tmem_addr(tmem, warp * 32, j * 16);
                    tmem_ld16(ta, ov);
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 16; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * f);
                    tmem_st16(ta, ov);
                }
                tmem_st_wait();
                tc_fence_before();
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.pfull[pb]);
            float psum = (ps[0] + ps[1]) + (ps[2] + ps[3]);
            psum += __shfl_xor_sync(0xffffffffu, psum, 16);
            l_sum = l_sum * alpha + psum;
        }
        if (nch > 0) warp_wait(&bars.odone, 0, status, 622);
        if (lane < 16) {
            const float m = l_sum != 0.f ? m_used - kLift : -INFINITY;   // (0: no row seen; a NaN stays one)
            bars.inv_l[head] = l_sum != 0.f ? 1.f / l_sum : 0.f;
            if (only) {
                if (a.lse != nullptr && head < nh)
                    a.lse[(int64_t)g * a.H + h0 + head] = l_sum != 0.f ? (m + log2f(l_sum)) / kLog2e : -INFINITY;
            } else {
                float* ml = part_ml + ((int64_t)(unit * splits + sp) * kH + head) * 2;
                ml[0] = m;
                ml[1] = l_sum;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // ---- O, 16 warps: lane l of warp w holds the O row of head 16 (w & 3) + (l & 15), dims 64 (w / 4) .. + 63
    // (+ 256 for l >= 16).  The only split: normalised, staged through shared memory.  One of
    // several: the partial as the lanes hold it ([quarter][4 dims][lane], 512 bytes a store).
    if (warp < 16) {
        tc_fence_after();
        const int quarter = warp & 3, head = quarter * 16 + (lane & 15);
        const float fs = only ? bars.inv_l[head] : 1.f;
        const int dim0 = (lane < 16) ? 0 : 256;
        const bool f32 = a.out_dtype == LCS_F32;
        uint8_t* rowp = stage_s + head * (f32 ? kOPitchF32 : kOPitchBF16);
        float4* gpart = reinterpret_cast<float4*>(part_o) + ((int64_t)(unit * splits + sp) * 4 + quarter) * (64 * 32) + lane;
        {
            const int j0 = (warp >> 2) * 4;
            uint32_t ov[4][16];
            if (nch > 0) {
#pragma unroll
                for (int u = 0; u < 4; ++u) tmem_ld16(tmem_addr(tmem, quarter * 32, (j0 + u) * 16), ov[u]);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int q = 0; q < 16; ++q) ov[u][q] = 0;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = j0 + u;
                if (!only || f32) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 v =
                            make_float4(__uint_as_float(ov[u][4 * q]) * fs, __uint_as_float(ov[u][4 * q + 1]) * fs,
                                        __uint_as_float(ov[u][4 * q + 2]) * fs, __uint_as_float(ov[u][4 * q + 3]) * fs);
                        if (only) reinterpret_cast<float4*>(rowp + (dim0 + j * 16) * 4)[q] = v;
                        else __stcg(gpart + (4 * j + q) * 32, v);
                    }
                } else {
                    uint32_t pk[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        pk[q] = cvt_bf16x2(__uint_as_float(ov[u][2 * q]) * fs, __uint_as_float(ov[u][2 * q + 1]) * fs);
                    reinterpret_cast<uint4*>(rowp + (dim0 + j * 16) * 2)[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    reinterpret_cast<uint4*>(rowp + (dim0 + j * 16) * 2)[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (only) {
        // the staged output rows with coalesced 16-byte stores
        const bool f32 = a.out_dtype == LCS_F32;
        const int pitch = f32 ? kOPitchF32 : kOPitchBF16;
        const int rb = f32 ? kDv * 4 : kDv * 2;
        uint8_t* gout = static_cast<uint8_t*>(a.out) + ((int64_t)g * a.H + h0) * rb;
#pragma unroll 2
        for (int off = (int)threadIdx.x * 16; off < nh * rb; off += kTcThreads * 16) {
            const int h = f32 ? off >> 11 : off >> 10, cb = off & (rb - 1);
            *reinterpret_cast<uint4*>(gout + off) = *reinterpret_cast<const uint4*>(stage_s + h * pitch + cb);
        }
    }
    if constexpr (kJoin) {
        // a unit's splits are one cluster: its barrier orders the partials, each CTA merges every splits-th task
        cluster_sync_all();
        const int t0 = sp + splits * warp, dt = splits * kTcWarps;
        if (splits <= 2)
            for (int t = t0; t < 64; t += dt) merge_task<4, 2>(a, tiles, splits, unit, t, part_o, part_ml);
        else if (splits <= 4)
            for (int t = t0; t < 64; t += dt) merge_task<4, 4>(a, tiles, splits, unit, t, part_o, part_ml);
        else
            for (int t = t0; t < 256; t += dt) merge_task<1, 8>(a, tiles, splits, unit, t, part_o, part_ml);
    }
#if defined(__CUDA_ARCH__)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the split merge
#endif
    if (warp == kWarpQK) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Merges the split partials of a launch whose splits are no clusters: a warp per task.
constexpr int kMergeThreads = 256;
template <int S>
__global__ void __launch_bounds__(kMergeThreads)
    kv4_merge_kernel(const AttendKv4Args a, int tiles, int splits, const float* __restrict__ part_o,
                     const float* __restrict__ part_ml) {
    const int w = blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
#if defined(__CUDA_ARCH__)
    asm volatile("griddepcontrol.wait;" ::: "memory");
#endif
    merge_task<1, S>(a, tiles, splits, w >> 8, w & 255, part_o, part_ml);
#if defined(__CUDA_ARCH__)
    // the partials are read: the next kernel of the stream may be set up
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#endif
}

// The waits above on a barrier that warp 1 completes after delay_ns: out = {warp 0 saw it complete, its ns}.
__global__ void selftest_warp_wait_kernel(uint64_t delay_ns, int* status, long long* out) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
    }
    __syncthreads();
    const uint64_t t0 = globaltimer();
    if (threadIdx.x < 32) {
        const bool ok = warp_wait(&bar, 0, status, 903);
        const uint64_t t1 = globaltimer();
        if (threadIdx.x == 0) {
            out[0] = ok;
            out[1] = (long long)(t1 - t0);
        }
    } else {
        for (int i = 0; i < (1 << 20) && globaltimer() - t0 < delay_ns; ++i) __nanosleep(1000);
        __syncwarp();
        if (threadIdx.x == 32) mbar_arrive(&bar);
    }
    __syncthreads();
}

bool use_tc(const AttendKv4Args& a) { return a.q_dtype == LCS_BF16 && a.d_c == kDv && a.d_r == kD - kDv; }

// Splits per (query, head tile): every CTA resident at once (one per SM); the count that minimises the
// longest split's chunks plus the merge, both in chunk times (about 1.1 us).  Measured, us a call by
// splits when the rule was made: 4 chunks of one query 14.1 (1), 16.1 (2); 14 chunks of 32 queries 25.9
// (2), 23.4 (3), 20.4 (4); 25 of 4: 20.6 (8), 17.7 (9), 16.4 (13); 177 of one 26.7 (16), 22.1 (29),
// 20.8 (58); 177 of 16: 40.2 (8, clusters), 39.4 (9, merged by a kernel).
int64_t kv4_units(const AttendKv4Args& a) { return a.B * a.Q * ((a.H + kH - 1) / kH); }
int64_t kv4_entry_chunks(const AttendKv4Args& a) {
    return ((a.idx != nullptr ? a.k : a.max_blocks * a.be) + kChunk - 1) / kChunk;
}
int kv4_splits_of(int64_t units, int64_t chunks) {   // (a call's host time: 32-bit whole numbers, 1/32 of a chunk)
    const int sms = num_sms();
    if (units < 1 || units * 2 > sms || chunks < 2) return 1;
    const unsigned n = (unsigned)(chunks < (1 << 26) ? chunks : 1 << 26);
    const int most = (int)(sms / units < kMaxSplits ? sms / units : kMaxSplits), u = (int)units;
    int best = 1;
    unsigned best_cost = 32u * n;
    for (int s = 2; s <= most && (unsigned)s <= n; ++s) {
        const bool cluster = s <= 8 || (s == kMaxCluster && u * s <= sms / 2);
        const unsigned cost = 32u * ((n + s - 1) / s) + (cluster ? 112u : 144u + s);   // 3.5, or 4.5 + s / 32, chunk times
        if (cost < best_cost) {
            best = s;
            best_cost = cost;
        }
    }
    return best;
}
int kv4_splits(const AttendKv4Args& a) {
    const int64_t most_w = a.q_pos == nullptr ? a.Tw : (a.W < a.Tw ? a.W : a.Tw);
    return kv4_splits_of(kv4_units(a), (most_w + kChunk - 1) / kChunk + kv4_entry_chunks(a));
}
// Split partials: fp32 O [units, splits, 64, 512] and (m, l) [units, splits, 64, 2].
int64_t kv4_partial_bytes(int64_t units, int64_t splits) {
    return splits == 1 ? 0 : align256(units * splits * kH * kDv * 4) + align256(units * splits * kH * 2 * 4);
}

using TcKernel = void (*)(const AttendKv4Args, int, int, float*, float*, int*);
TcKernel tc_kernel(bool csa, bool join) {
    return csa ? (join ? attend_kv4_tc_kernel<true, true> : attend_kv4_tc_kernel<true, false>)
               : (join ? attend_kv4_tc_kernel<false, true> : attend_kv4_tc_kernel<false, false>);
}

// Whether the launch's clusters of `splits` CTAs can all be resident at once (asked once per kernel, device
// and split count; clusters of more than 8 are not portable, but open on this device).
bool kv4_cluster_ok(bool csa, int splits, int64_t units) {
    if (splits < 2 || splits > kMaxCluster) return false;
    constexpr int kDevices = 16;
    static std::mutex mu;
    static int cache[2][kDevices][kMaxCluster + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return false;
    std::lock_guard<std::mutex> lock(mu);
    int& most = cache[csa][dev][splits];
    if (most == 0) {
        const TcKernel kern = tc_kernel(csa, true);
        int n = 0;
        if (set_smem_here(reinterpret_cast<const void*>(kern), kTcSmem) == cudaSuccess &&
            cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)splits);
            cfg.blockDim = dim3(kTcThreads);
            cfg.dynamicSmemBytes = kTcSmem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)splits;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) n = 0;
        }
        cudaGetLastError();
        most = n > 0 ? n : -1;
    }
    return most >= units;
}

cudaError_t launch_tc(const AttendKv4Args& a, void* scratch, int* status, cudaStream_t s) {
    const int tiles = (a.H + kH - 1) / kH;
    const int64_t units = kv4_units(a);
    const int splits = kv4_splits(a);
    const bool clustered = kv4_cluster_ok(a.idx != nullptr, splits, units);
    const TcKernel kern = tc_kernel(a.idx != nullptr, clustered);
    cudaError_t e = set_smem_here(reinterpret_cast<const void*>(kern), kTcSmem);
    if (e != cudaSuccess) return e;
    float* part_o = nullptr;
    float* part_ml = nullptr;
    if (splits > 1) {
        part_o = static_cast<float*>(scratch);
        part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + align256(units * splits * kH * kDv * 4));
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = splits > 1 ? dim3((unsigned)splits, (unsigned)units) : dim3((unsigned)units);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = kTcSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = clustered ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, a, tiles, splits, part_o, part_ml, status);
    if (e != cudaSuccess || splits == 1 || clustered) return e;
    // (44 splits of one query: 16 in flight 21.3 us a call, 8 22.8; 9 splits of 16: 40.7 and 39.4)
    return launch_k(splits > 16 ? kv4_merge_kernel<16> : kv4_merge_kernel<8>, dim3((unsigned)(units * 32)), dim3(kMergeThreads), 0, s, true, a, tiles, splits,
                    part_o, part_ml);
}

}  // namespace

int64_t attend_kv4_scratch_bytes(const AttendKv4Args& a) {
    return use_tc(a) ? kv4_partial_bytes(kv4_units(a), kv4_splits(a)) : 0;
}

// The most that a call of these sizes needs, whatever its W: fewer window rows can mean more splits (the
// longest split's chunks are rounded up).  Short windows: every chunk count.  Long ones: as many splits
// as there can be.
int64_t attend_kv4_scratch_bound(const AttendKv4Args& a) {
    if (!use_tc(a) || a.B * a.Q <= 0) return 0;
    const int64_t units = kv4_units(a), entries = kv4_entry_chunks(a), window = (a.Tw + kChunk - 1) / kChunk;
    int64_t s = 1;
    if (window <= 8) {
        for (int64_t w = window > 0; w <= window; ++w) {
            const int64_t x = kv4_splits_of(units, entries + w);
            s = x > s ? x : s;
        }
    } else if (units * 2 <= num_sms()) {
        s = num_sms() / units < kMaxSplits ? num_sms() / units : kMaxSplits;
        if (s > entries + window) s = entries + window;
    }
    return kv4_partial_bytes(units, s);
}

cudaError_t launch_selftest_warp_wait(uint64_t delay_ns, int* status, long long* out, cudaStream_t stream) {
    selftest_warp_wait_kernel<<<1, 64, 0, stream>>>(delay_ns, status, out);
    return cudaGetLastError();
}

cudaError_t launch_attend_kv4(const AttendKv4Args& a, void* scratch, int* status, cudaStream_t s) {
    const int64_t queries = a.B * a.Q;
    if (queries == 0) return cudaSuccess;
    if (use_tc(a)) return launch_tc(a, scratch, status, s);
    if (a.d_c <= 32) return launch_simt<4, 1>(a, status, s);
    if (a.d_c <= 64) return launch_simt<2, 1>(a, status, s);
    if (a.d_c <= 128) return launch_simt<1, 1>(a, status, s);
    if (a.d_c <= 256) return launch_simt<1, 2>(a, status, s);
    return launch_simt<1, 4>(a, status, s);
}

}  // namespace lcs
