// paged.cu -- the paged compressed cache in 4 bits: block tables and slot maps from the
// requests' lengths, and the cache writer and reader of LCS_KV_FP4 rows.
//
// "DeepSeek V4 深度解析" §4 keeps the compressed cache in blocks that cover lcm(4, 128)
// raw tokens; its FP4 paragraph has 4 bits for the indexer's QK path.  The rows here are KV content in
// that format (E2M1 codes, an E4M3 scale per 32), which the page keeps in FP8: this library's choice.
#include <type_traits>
#include <utility>

#include "lcs_common.cuh"
#include "lcs_internal.h"

namespace lcs {

namespace {

// ------------------------------------------------------------------ page plan
// Request b holds len tokens and appends n.  With P tokens per block it needs the blocks
// [ceil(len/P), ceil((len+n)/P)), and it completes the entries [len/m, (len+n)/m) of m
// tokens each.  Three exclusive scans over the requests (blocks, entries of m, entries of
// m2) place them: blocks come from the free list in request order, entry j sits in slot
// table[b][j/(P/m)] * (P/m) + j mod (P/m).
//
// Every CTA repeats the scan (a few KB of lengths, from L2) and then writes its share of
// the outputs, so that the call is one launch: a decode step's plan is bound by the launch,
// a batch of prompts by the slots it writes.  An entry's block id comes from the free list
// directly when this call assigns it, so no CTA waits for another's table writes.  32 requests of one
// token each: 5.0 us a call back to back; 64 prompts with 1.05 million slots: 11.8 (22.7 with four
// neighbouring slots a thread, each looked up by itself), half of it the scan and the launch.
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 8192;
constexpr int64_t kPlanFar = int64_t(1) << 52;   // tokens

// Quotient of a length: nearly always of 32 bits, where the division is several times cheaper.
__device__ __forceinline__ int64_t plan_div(int64_t a, int b) {
    return (a >> 31) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

struct PlanReq {
    int64_t len, n;
};
__device__ __forceinline__ PlanReq plan_req(const int64_t* len, const int64_t* n_new, int64_t b) {
    PlanReq r;
    r.len = len[b];
    r.n = n_new[b];
    if (r.len < 0) r.n = 0, r.len = 0;
    if (r.n < 0) r.n = 0;
    // a table holds less than 2^31 blocks of at most 2^20 tokens: the check against max_blocks refuses what
    // is clamped here, and len + n does not wrap
    if (r.len > kPlanFar) r.len = kPlanFar;
    if (r.n > kPlanFar) r.n = kPlanFar;
    return r;
}

// The request that output i belongs to: the last b with off[b] <= i (off ascending, off[0] = 0).
__device__ __forceinline__ int plan_find(const int* off, int B, int i) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

struct PlanOut {
    int m;
    int64_t max;
    int64_t* slots;
    int64_t* off;
};

template <int kPlanRun>   // slots per thread and turn
__global__ void __launch_bounds__(kPlanThreads)
    page_plan_kernel(int B, const int64_t* __restrict__ len, const int64_t* __restrict__ n_new, int P,
                     const int32_t* __restrict__ free_blocks, int64_t n_free, int32_t* __restrict__ table,
                     int64_t max_blocks, PlanOut o0, PlanOut o1, int64_t* __restrict__ taken, int* status) {
    extern __shared__ int sh[];
    int* off[3] = {sh, sh + B + 1, sh + 2 * (B + 1)};   // blocks, entries of o0.m, entries of o1.m
    __shared__ int64_t wsum[3][kPlanThreads / 32];
    __shared__ int bad_s;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int m1 = o1.m > 0 ? o1.m : 1;
    if (t == 0) bad_s = 0;
    __syncthreads();
    int64_t carry[3] = {0, 0, 0};
    for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
        const int b = b0 + t;
        int64_t v[3] = {0, 0, 0};
        if (b < B) {
            const PlanReq r = plan_req(len, n_new, b);
            const int64_t nb1 = plan_div(r.len + r.n + P - 1, P);
            v[0] = nb1 - plan_div(r.len + P - 1, P);
            v[1] = plan_div(r.len + r.n, o0.m) - plan_div(r.len, o0.m);
            v[2] = o1.m > 0 ? plan_div(r.len + r.n, m1) - plan_div(r.len, m1) : 0;
            if (r.n > 0 && nb1 > max_blocks) bad_s = 1;
            // (a count from 2^31 on is refused below by itself; cut there, 8192 of them add up without a wrap)
#pragma unroll
            for (int i = 0; i < 3; ++i) v[i] = v[i] < (int64_t(1) << 32) ? v[i] : int64_t(1) << 32;
        }
        int64_t x[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            x[i] = v[i];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x[i], d);
                if (lane >= d) x[i] += y;
            }
            if (lane == 31) wsum[i][warp] = x[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            int64_t before = carry[i], total = 0;
            for (int w = 0; w < kPlanThreads / 32; ++w) {
                if (w < warp) before += wsum[i][w];
                total += wsum[i][w];
            }
            // values past int32 mean a total that the checks below refuse
            if (b < B) off[i][b] = (int)(before + x[i] - v[i]);
            carry[i] += total;
        }
        __syncthreads();
    }
    const bool bad = bad_s != 0 || carry[0] > n_free || carry[1] > o0.max || (o1.m > 0 && carry[2] > o1.max);
    const int64_t total[3] = {bad ? 0 : carry[0], bad ? 0 : carry[1], bad ? 0 : carry[2]};
    if (t < 3) off[t][B] = (int)total[t];
    __syncthreads();

    const int64_t gt = (int64_t)blockIdx.x * kPlanThreads + t, gn = (int64_t)gridDim.x * kPlanThreads;
    if (blockIdx.x == 0) {
        if (t == 0) {
            taken[0] = total[0];
            if (bad) set_status(status, LCS_ERR_DEVICE, 501);
        }
        for (int b = t; b <= B; b += kPlanThreads) {
            o0.off[b] = bad ? 0 : off[1][b];
            if (o1.m > 0) o1.off[b] = bad ? 0 : off[2][b];
        }
    }
    for (int64_t i = gt; i < total[0]; i += gn) {
        const int b = plan_find(off[0], B, (int)i);
        const PlanReq r = plan_req(len, n_new, b);
        table[(int64_t)b * max_blocks + plan_div(r.len + P - 1, P) + (i - off[0][b])] = free_blocks[i];
    }
    // slots: a warp takes 32 kPlanRun in a row, a thread every 32nd of them: one search and one request's
    // lengths for all of them as a rule, their block ids in flight together, whole lines written
    const int lane32 = t & 31;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const PlanOut o = s ? o1 : o0;
        if (o.m == 0) continue;
        const int* of = off[1 + s];
        const int n_out = (int)o.max, n_slot = (int)total[1 + s];
        const uint32_t per = (uint32_t)(P / o.m);
        const int sh = (per & (per - 1)) == 0 ? 31 - __clz((int)per) : -1;
        for (int64_t j0 = ((int64_t)blockIdx.x * kPlanThreads + (t - lane32)) * kPlanRun; j0 < n_out;
             j0 += (int64_t)gridDim.x * kPlanThreads * kPlanRun) {
            const int i0 = (int)j0 + lane32;   // (j0 is a multiple of 32 kPlanRun: i0 + 32 k ends at 2^31 - 1)
            int b = -1, end = 0;             // the request at hand and the end of its slots
            uint32_t first = 0;              // position of slot i0 counted from the first block of b's new entries
            const int32_t *held = nullptr, *got = nullptr;
            int nb = 0;                      // blocks held, from that one on
            const int32_t* src[kPlanRun];
            uint32_t r[kPlanRun];
#pragma unroll
            for (int k = 0; k < kPlanRun; ++k) {
                const int i = i0 + 32 * k;
                src[k] = nullptr;
                r[k] = 0;
                if (i >= n_slot) continue;
                if (i >= end) {
                    if (b < 0) b = plan_find(of, B, i);
                    else
                        while (of[b + 1] <= i) ++b;
                    end = of[b + 1];
                    const PlanReq q = plan_req(len, n_new, b);
                    const int64_t e0 = plan_div(q.len, o.m), b0 = plan_div(e0, (int)per);
                    first = (uint32_t)(e0 - b0 * per) + (uint32_t)(i0 - of[b]);   // (wraps back with + 32 k)
                    held = table + (int64_t)b * max_blocks + b0;
                    nb = (int)(plan_div(q.len + P - 1, P) - b0);
                    got = free_blocks + off[0][b];
                }
                const uint32_t at = first + 32u * k, bi = sh >= 0 ? at >> sh : at / per;
                r[k] = at - bi * per;
                src[k] = (int)bi < nb ? held + bi : got + (bi - nb);
            }
            int32_t id[kPlanRun];
#pragma unroll
            for (int k = 0; k < kPlanRun; ++k) id[k] = src[k] != nullptr ? *src[k] : -1;
#pragma unroll
            for (int k = 0; k < kPlanRun; ++k) {
                const int i = i0 + 32 * k;
                if (i < n_out) o.slots[i] = id[k] < 0 ? -1 : (int64_t)id[k] * per + r[k];
            }
        }
    }
}

// ---------------------------------------------------------- 4-bit rows: write, read
// E2M1 codes of v / sc without a division per element: v (r + rl) in one fused step, r the reciprocal
// rounded down and rl what it lacks, is (v / sc)(1 + 2^-46) before its rounding to fp32.  The codes can
// only differ from the quotient's at the code grid's midpoints, which have three bits: times sc
// (four bits) they are fp32 values, so a v that is not one of them lies at least a step of its 24 bits
// away, more than half a step of the quotient's; a v that is one gives the midpoint itself, which goes to
// the even code.  (rl is not negative and not 0: -0 stays -0, an infinity infinite.)
struct Recip {
    uint64_t r, rl;   // in both halves
};
__device__ __forceinline__ Recip recip_of(float sc) {
    const float r = __frcp_rd(sc), rl = fmaxf(fmaf(-r, sc, 1.f) * r, 1.17549435e-38f);
    return {pack2(r, r), pack2(rl, rl)};
}
__device__ __forceinline__ float2 quotients(uint64_t v, const Recip& q) { return unpack2(fma2(v, q.r, mul2(v, q.rl))); }
// Eight floats -> eight E2M1 codes, low nibble first, saturating.
__device__ __forceinline__ uint32_t cvt_e2m1x8(float2 a, float2 b, float2 c, float2 d) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
    return r;
}

// 16 elements of a lane, fp32 ...
struct LaneF32 {
    float4 v[4];
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __ldg(reinterpret_cast<const float4*>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ float amax() const {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(fmaxf(m, fmaxf(fabsf(v[i].x), fabsf(v[i].y))), fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
        return m;
    }
    static __device__ __forceinline__ float sixth(float amax) { return amax / 6.0f; }
    __device__ __forceinline__ uint2 codes(float sc) const {
        const Recip q = recip_of(sc);
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 a = v[2 * h], b = v[2 * h + 1];
            w[h] = cvt_e2m1x8(quotients(pack2(a.x, a.y), q), quotients(pack2(a.z, a.w), q), quotients(pack2(b.x, b.y), q),
                              quotients(pack2(b.z, b.w), q));
        }
        return make_uint2(w[0], w[1]);
    }
};
// ... and bf16.
struct LaneBf16 {
    uint4 v[2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ float amax() const {
        uint32_t m = 0;   // (a NaN loses)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            m = bf16x2_maxabs(bf16x2_maxabs(bf16x2_maxabs(m, v[i].x), bf16x2_maxabs(v[i].y, v[i].z)), v[i].w);
        return fmaxf(fabsf(__uint_as_float(m << 16)), fabsf(__uint_as_float(m & 0xFFFF0000u)));
    }
    // (for every amax of 8 bits the product has the E4M3 value of the quotient: all of them compared on the host)
    static __device__ __forceinline__ float sixth(float amax) { return amax * (1.0f / 6.0f); }
    __device__ __forceinline__ uint2 codes(float sc) const {
        const Recip q = recip_of(sc);
        auto two = [&](uint32_t w) { return quotients(pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)), q); };
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) w[h] = cvt_e2m1x8(two(v[h].x), two(v[h].y), two(v[h].z), two(v[h].w));
        return make_uint2(w[0], w[1]);
    }
};
__device__ __forceinline__ uint16_t to_bf16_bits(float v) { return f32_to_bf16_bits(v); }
__device__ __forceinline__ uint16_t to_bf16_bits(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }

// One warp takes kRowsFly rows at a time, their loads in flight together and the next slots on their way;
// two lanes share a 32-element block, 16 elements each: the block's amax is one shuffle, a lane's codes
// one 8-byte store.  Bound by HBM: 1152 or 2304 bytes read and 400 written a row.  262144 rows, us (at the
// measured copy rate): bf16 stored 82 (63), loaded 76 (63); fp32 stored 121 (110), loaded 131 (110).  With
// seven thresholds per element in place of the quotient, and slots asked for when they are needed, the
// stores took 127 and 174.  bf16 stored and loaded, by rows in flight x CTAs per SM: 162 (2 x 5), 170
// (2 x 6), 172 (4 x 4).
constexpr int kRowsFly = 2;
template <typename T>
constexpr int rows_ctas() {   // CTAs per SM: what the registers allow
    return sizeof(T) == 4 ? 4 : 5;
}
template <typename T, typename Lane>
__global__ void __launch_bounds__(256, rows_ctas<T>()) kv4_store_kernel(const T* __restrict__ x, const int64_t* __restrict__ slots,
                                                        int64_t n, int d_c, int d_r, int row_bytes,
                                                        uint8_t* __restrict__ pool, int64_t n_slots, int fly, int* status) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5), w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int D = d_c + d_r;
    int64_t next = lane < fly && w * fly + lane < n ? __ldg(slots + w * fly + lane) : -1;
    for (int64_t r0 = w * fly; r0 < n; r0 += warps * fly) {
        int64_t mine = next;
        next = -1;
        if (lane < fly && r0 + lane < n) {
            if (r0 + warps * fly + lane < n) next = __ldg(slots + r0 + warps * fly + lane);   // (on its way meanwhile)
            if (mine >= n_slots) {
                set_status(status, LCS_ERR_DEVICE, 502);
                mine = -1;
            }
        }
        int64_t slot[kRowsFly];
#pragma unroll
        for (int u = 0; u < kRowsFly; ++u) slot[u] = __shfl_sync(0xffffffffu, mine, u);
        for (int p0 = 0; p0 < d_c / 16; p0 += 32) {
            const int p = p0 + lane;
            const bool in = p < d_c / 16;   // the same for both lanes of a block: d_c / 16 is even
            Lane v[kRowsFly];
#pragma unroll
            for (int u = 0; u < kRowsFly; ++u) {
                v[u].zero();
                if (in && slot[u] >= 0) v[u].load(x + (r0 + u) * D + 16 * p);
            }
#pragma unroll
            for (int u = 0; u < kRowsFly; ++u) {
                float amax = v[u].amax();
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                if (!in || slot[u] < 0) continue;
                uint8_t sc_code = f32_to_e4m3(Lane::sixth(amax));
                if ((sc_code & 0x7F) == 0) sc_code = 0x38;   // 1.0
                uint8_t* o = pool + slot[u] * row_bytes;
                *reinterpret_cast<uint2*>(o + 8 * p) = v[u].codes(e4m3_to_f32(sc_code));
                if ((p & 1) == 0) o[d_c / 2 + 2 * d_r + p / 2] = sc_code;
            }
        }
#pragma unroll
        for (int u = 0; u < kRowsFly; ++u) {
            if (slot[u] < 0) continue;
            const T* xr = x + (r0 + u) * D + d_c;
            uint8_t* o = pool + slot[u] * row_bytes;
            for (int j = 2 * lane; j < d_r; j += 64)
                *reinterpret_cast<uint32_t*>(o + d_c / 2 + 2 * j) = (uint32_t)to_bf16_bits(xr[j]) | ((uint32_t)to_bf16_bits(xr[j + 1]) << 16);
            // the bytes past the last scale (row padding) are zeros
            for (int j = d_c / 2 + 2 * d_r + d_c / 32 + lane; j < row_bytes; j += 32) o[j] = 0;
        }
    }
}

// A lane's 32 bytes of a row: 8 fp32 or 16 bf16 values, eight packed codes a word, times the scale.
__device__ __forceinline__ void store_lane(float* o, uint32_t c, float sc) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = e2m1x2_to_f32(c >> (16 * i)), b = e2m1x2_to_f32(c >> (16 * i + 8));
        reinterpret_cast<float4*>(o)[i] = make_float4(a.x * sc, a.y * sc, b.x * sc, b.y * sc);
    }
}
__device__ __forceinline__ void store_lane(__nv_bfloat16* o, uint2 c, float sc) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w = i ? c.y : c.x;
        uint32_t r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 a = e2m1x2_to_f32(w >> (8 * k));
            r[k] = cvt_bf16x2(a.x * sc, a.y * sc);
        }
        reinterpret_cast<uint4*>(o)[i] = make_uint4(r[0], r[1], r[2], r[3]);
    }
}

// The same split of the work: code x scale is exact in bf16 (six significant bits), the RoPE dims are bf16.
template <typename T>
__global__ void __launch_bounds__(256, rows_ctas<T>()) kv4_load_kernel(const uint8_t* __restrict__ pool, int64_t n_slots,
                                                       const int64_t* __restrict__ slots, int64_t n, int d_c, int d_r,
                                                       int row_bytes, T* __restrict__ out, int fly, int* status) {
    using Codes = typename std::conditional<sizeof(T) == 4, uint32_t, uint2>::type;
    constexpr int kDims = 32 / sizeof(T);
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5), w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int D = d_c + d_r;
    int64_t next = lane < fly && w * fly + lane < n ? __ldg(slots + w * fly + lane) : -2;
    for (int64_t r0 = w * fly; r0 < n; r0 += warps * fly) {
        int64_t mine = -2;                       // past the last row
        if (lane < fly && r0 + lane < n) {
            mine = next;
            if (r0 + warps * fly + lane < n) next = __ldg(slots + r0 + warps * fly + lane);
            if (mine >= n_slots) set_status(status, LCS_ERR_DEVICE, 503);
            if (mine < 0 || mine >= n_slots) mine = -1;   // a row of zeros
        }
        int64_t slot[kRowsFly];
#pragma unroll
        for (int u = 0; u < kRowsFly; ++u) slot[u] = __shfl_sync(0xffffffffu, mine, u);
        for (int p = lane; p < d_c / kDims; p += 32) {
            Codes c[kRowsFly];
            uint8_t sb[kRowsFly];
#pragma unroll
            for (int u = 0; u < kRowsFly; ++u) {
                c[u] = Codes{};
                sb[u] = 0;
                if (slot[u] >= 0) {
                    const uint8_t* src = pool + slot[u] * row_bytes;
                    c[u] = __ldg(reinterpret_cast<const Codes*>(src) + p);
                    sb[u] = __ldg(src + d_c / 2 + 2 * d_r + p / (32 / kDims));
                }
            }
#pragma unroll
            for (int u = 0; u < kRowsFly; ++u)
                if (slot[u] > -2) store_lane(out + (r0 + u) * D + kDims * p, c[u], e4m3_to_f32(sb[u]));
        }
        for (int j = 2 * lane; j < d_r; j += 64) {
            uint32_t h[kRowsFly];
#pragma unroll
            for (int u = 0; u < kRowsFly; ++u)
                h[u] = slot[u] >= 0 ? __ldg(reinterpret_cast<const uint32_t*>(pool + slot[u] * row_bytes + d_c / 2 + 2 * j)) : 0u;
#pragma unroll
            for (int u = 0; u < kRowsFly; ++u) {
                if (slot[u] == -2) continue;
                T* o = out + (r0 + u) * D + d_c + j;
                if constexpr (sizeof(T) == 4)
                    *reinterpret_cast<float2*>(o) = make_float2(__uint_as_float(h[u] << 16), __uint_as_float(h[u] & 0xFFFF0000u));
                else *reinterpret_cast<uint32_t*>(o) = h[u];
            }
        }
    }
}

// Rows per warp and turn, and the CTAs: rows are spread over the SMs first (a decode step's few rows get a
// warp each), then taken kRowsFly at a time.
struct RowsPlan {
    int fly;
    unsigned ctas;
};
RowsPlan rows_plan(int64_t n, int per_sm) {
    const int64_t most = (int64_t)num_sms() * per_sm;   // CTAs of 8 warps, all resident
    int fly = 1;
    while (fly < kRowsFly && n > most * 8 * fly) fly *= 2;
    const int64_t ctas = (n + 8 * fly - 1) / (8 * fly);
    return {fly, (unsigned)(ctas < most ? ctas : most)};
}

}  // namespace

int page_plan_max_requests() { return kPlanMaxB; }

cudaError_t launch_page_plan(int64_t B, const int64_t* len, const int64_t* n_new, int block_tokens,
                             const int32_t* free_blocks, int64_t n_free, int32_t* table, int64_t max_blocks, int m,
                             int64_t* slots, int64_t max_slots, int64_t* off, int m2, int64_t* slots2,
                             int64_t max_slots2, int64_t* off2, int64_t* taken, int* status, cudaStream_t s) {
    const size_t smem = 3 * (size_t)(B + 1) * sizeof(int);
    // a decode step's few slots get a thread each; many, four.  At most two CTAs per SM: each repeats the
    // scan of the lengths
    const int64_t outs = max_slots > max_slots2 || m2 == 0 ? max_slots : max_slots2;
    const int run = outs > 4 * (int64_t)num_sms() * kPlanThreads ? 4 : 1;
    int64_t ctas = (outs + run * kPlanThreads - 1) / (run * kPlanThreads);
    if (ctas < 1) ctas = 1;
    if (ctas > 2 * num_sms()) ctas = 2 * num_sms();
    auto kern = run == 4 ? page_plan_kernel<4> : page_plan_kernel<1>;
    cudaError_t e = set_smem_here(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    const PlanOut o0{m, max_slots, slots, off}, o1{m2, max_slots2, slots2, off2};
    return launch_k(kern, dim3((unsigned)ctas), dim3(kPlanThreads), smem, s, false, (int)B, len, n_new, block_tokens,
                    free_blocks, n_free, table, max_blocks, o0, o1, taken, status);
}

cudaError_t launch_kv4_store(const void* x, int x_dtype, int64_t n, int d_c, int d_r, const int64_t* slots, void* pool,
                             int64_t n_slots, int* status, cudaStream_t s) {
    if (n == 0) return cudaSuccess;
    const int rb = kv4_row_bytes(d_c, d_r);
    const RowsPlan rp = rows_plan(n, x_dtype == LCS_F32 ? rows_ctas<float>() : rows_ctas<__nv_bfloat16>());
    if (x_dtype == LCS_F32)
        return launch_k(kv4_store_kernel<float, LaneF32>, dim3(rp.ctas), dim3(256), 0, s, false,
                        static_cast<const float*>(x), slots, n, d_c, d_r, rb, static_cast<uint8_t*>(pool), n_slots,
                        rp.fly, status);
    return launch_k(kv4_store_kernel<__nv_bfloat16, LaneBf16>, dim3(rp.ctas), dim3(256), 0, s, false,
                    static_cast<const __nv_bfloat16*>(x), slots, n, d_c, d_r, rb, static_cast<uint8_t*>(pool), n_slots,
                    rp.fly, status);
}

cudaError_t launch_kv4_load(const void* pool, int64_t n_slots, const int64_t* slots, int64_t n, int d_c, int d_r,
                            void* out, int out_dtype, int* status, cudaStream_t s) {
    if (n == 0) return cudaSuccess;
    const int rb = kv4_row_bytes(d_c, d_r);
    const RowsPlan rp = rows_plan(n, out_dtype == LCS_F32 ? rows_ctas<float>() : rows_ctas<__nv_bfloat16>());
    if (out_dtype == LCS_F32)
        return launch_k(kv4_load_kernel<float>, dim3(rp.ctas), dim3(256), 0, s, false,
                        static_cast<const uint8_t*>(pool), n_slots, slots, n, d_c, d_r, rb, static_cast<float*>(out),
                        rp.fly, status);
    return launch_k(kv4_load_kernel<__nv_bfloat16>, dim3(rp.ctas), dim3(256), 0, s, false,
                    static_cast<const uint8_t*>(pool), n_slots, slots, n, d_c, d_r, rb,
                    static_cast<__nv_bfloat16*>(out), rp.fly, status);
}

}  // namespace lcs
