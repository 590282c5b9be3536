// paged.cu -- the paged compressed cache in 4 bits: block tables and slot maps from the
// requests' lengths, and the cache writer and reader of LCS_KV_FP4 rows.
//
// "DeepSeek V4 深度解析" §4 keeps the compressed cache in blocks that cover lcm(4, 128)
// raw tokens; its FP4 paragraph gives the 4-bit format (E2M1 codes, an E4M3 scale per 32).
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
// directly when this call assigns it, so no CTA waits for another's table writes.
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 8192;

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
    // lengths past 2^40 tokens cannot be held by any table: the check against max_blocks
    // refuses them, and the clamp keeps the sums below from wrapping
    if (r.len > (int64_t(1) << 40)) r.len = int64_t(1) << 40;
    if (r.n > (int64_t(1) << 40)) r.n = int64_t(1) << 40;
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
            const int i0 = (int)j0 + lane32;
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
                if (i >= n_slot || i < 0) continue;   // (i < 0: past 2^31)
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
                if (i >= 0 && i < n_out) o.slots[i] = id[k] < 0 ? -1 : (int64_t)id[k] * per + r[k];
            }
        }
    }
}

// ---------------------------------------------------------- 4-bit rows: write, read
// E2M1 code (magnitude bits) of |v| / sc without the division: |v| against the code grid's midpoints
// times sc (0.25 .. 5 times an E4M3 value: exact, even in bf16).  Ties go to the even code, so the
// midpoints below odd codes count to the code under them: a search of three steps, the first two with
// >=, the last with >.  (A quotient rounded to fp32 meets a midpoint only when the exact one does:
// a midpoint has 3 bits, a value within 2^-24 of it but not on it would need more than 24.)
//
// fp32 rows: 16 elements of a lane, eight codes a word.
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
    __device__ __forceinline__ uint2 codes(float sc) const {
        const float t0 = 0.25f * sc, t1 = 0.75f * sc, t2 = 1.25f * sc, t3 = 1.75f * sc, t4 = 2.5f * sc, t5 = 3.5f * sc, t6 = 5.f * sc;
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = i & 2 ? (i & 1 ? v[i >> 2].w : v[i >> 2].z) : (i & 1 ? v[i >> 2].y : v[i >> 2].x);
            const float a = fabsf(x);
            const bool p1 = a >= t3, p2 = a >= (p1 ? t5 : t1);
            const bool p3 = a > (p1 ? (p2 ? t6 : t4) : (p2 ? t2 : t0));
            const uint32_t c = (p1 ? 4u : 0u) + (p2 ? 2u : 0u) + (p3 ? 1u : 0u) + ((__float_as_uint(x) >> 28) & 8u);
            w[i >> 3] |= c << (4 * (i & 7));
        }
        return make_uint2(w[0], w[1]);
    }
};
// bf16 rows: two elements an instruction.
struct LaneBf16 {
    uint4 v[2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ uint32_t word(int i) const {
        const uint4 x = v[i >> 2];
        return i & 2 ? (i & 1 ? x.w : x.z) : (i & 1 ? x.y : x.x);
    }
    static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
    __device__ __forceinline__ float amax() const {
        __nv_bfloat162 m = two(0u);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __hmax2(m, two(word(i) & 0x7FFF7FFFu));   // (a NaN loses)
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ __forceinline__ uint2 codes(float sc) const {
        uint32_t t[7];
        constexpr float mid[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.f};
#pragma unroll
        for (int k = 0; k < 7; ++k) t[k] = cvt_bf16x2(mid[k] * sc, mid[k] * sc);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t x = word(i);
            const __nv_bfloat162 a = two(x & 0x7FFF7FFFu);
            const uint32_t m1 = __hge2_mask(a, two(t[3]));
            const uint32_t m2 = __hge2_mask(a, two((m1 & t[5]) | (~m1 & t[1])));
            const uint32_t hi = (m2 & t[6]) | (~m2 & t[4]), lo = (m2 & t[2]) | (~m2 & t[0]);
            const uint32_t m3 = __hgt2_mask(a, two((m1 & hi) | (~m1 & lo)));
            uint32_t c = (m1 & 0x00040004u) | (m2 & 0x00020002u);
            c |= (m3 & 0x00010001u) | ((x >> 12) & 0x00080008u);
            w[i >> 2] |= ((c | (c >> 12)) & 0xFFu) << (8 * (i & 3));   // element 2j in the low nibble
        }
        return make_uint2(w[0], w[1]);
    }
};
__device__ __forceinline__ uint16_t to_bf16_bits(float v) { return f32_to_bf16_bits(v); }
__device__ __forceinline__ uint16_t to_bf16_bits(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }

// One warp takes kRowsFly rows at a time, their loads in flight together; two lanes share a 32-element
// block, 16 elements each: the block's amax is one shuffle, a lane's codes one 8-byte store.  Bound by HBM:
// 1152 or 2304 bytes read and 400 written a row.
constexpr int kRowsFly = 2, kRowsCtas = 5;   // CTAs per SM (262144 bf16 rows stored and read: 211 us; 1 x 6: 235, 4 x 4: 219)
template <typename T, typename Lane>
__global__ void __launch_bounds__(256, kRowsCtas) kv4_store_kernel(const T* __restrict__ x, const int64_t* __restrict__ slots,
                                                        int64_t n, int d_c, int d_r, int row_bytes,
                                                        uint8_t* __restrict__ pool, int64_t n_slots, int fly, int* status) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5), w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int D = d_c + d_r;
    for (int64_t r0 = w * fly; r0 < n; r0 += warps * fly) {
        int64_t mine = -1;
        if (lane < fly && r0 + lane < n) {
            mine = __ldg(slots + r0 + lane);
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
                uint8_t sc_code = f32_to_e4m3(amax / 6.0f);
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

// 16 values of a lane: eight packed codes a word, times the scale.
__device__ __forceinline__ void store16(float* o, uint2 c, float sc) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = (i < 2 ? c.x : c.y) >> (16 * (i & 1));
        const float2 a = e2m1x2_to_f32(w), b = e2m1x2_to_f32(w >> 8);
        reinterpret_cast<float4*>(o)[i] = make_float4(a.x * sc, a.y * sc, b.x * sc, b.y * sc);
    }
}
__device__ __forceinline__ void store16(__nv_bfloat16* o, uint2 c, float sc) {
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
__global__ void __launch_bounds__(256, kRowsCtas) kv4_load_kernel(const uint8_t* __restrict__ pool, int64_t n_slots,
                                                       const int64_t* __restrict__ slots, int64_t n, int d_c, int d_r,
                                                       int row_bytes, T* __restrict__ out, int fly, int* status) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5), w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int D = d_c + d_r;
    for (int64_t r0 = w * fly; r0 < n; r0 += warps * fly) {
        int64_t mine = -2;                       // past the last row
        if (lane < fly && r0 + lane < n) {
            mine = __ldg(slots + r0 + lane);
            if (mine >= n_slots) set_status(status, LCS_ERR_DEVICE, 503);
            if (mine < 0 || mine >= n_slots) mine = -1;   // a row of zeros
        }
        int64_t slot[kRowsFly];
#pragma unroll
        for (int u = 0; u < kRowsFly; ++u) slot[u] = __shfl_sync(0xffffffffu, mine, u);
        for (int p = lane; p < d_c / 16; p += 32) {
            uint2 c[kRowsFly];
            uint8_t sb[kRowsFly];
#pragma unroll
            for (int u = 0; u < kRowsFly; ++u) {
                c[u] = make_uint2(0, 0);
                sb[u] = 0;
                if (slot[u] >= 0) {
                    const uint8_t* src = pool + slot[u] * row_bytes;
                    c[u] = __ldg(reinterpret_cast<const uint2*>(src + 8 * p));
                    sb[u] = __ldg(src + d_c / 2 + 2 * d_r + p / 2);
                }
            }
#pragma unroll
            for (int u = 0; u < kRowsFly; ++u)
                if (slot[u] > -2) store16(out + (r0 + u) * D + 16 * p, c[u], e4m3_to_f32(sb[u]));
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
RowsPlan rows_plan(int64_t n) {
    const int64_t most = (int64_t)num_sms() * kRowsCtas;   // CTAs of 8 warps, all resident
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
    const RowsPlan rp = rows_plan(n);
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
    const RowsPlan rp = rows_plan(n);
    if (out_dtype == LCS_F32)
        return launch_k(kv4_load_kernel<float>, dim3(rp.ctas), dim3(256), 0, s, false,
                        static_cast<const uint8_t*>(pool), n_slots, slots, n, d_c, d_r, rb, static_cast<float*>(out),
                        rp.fly, status);
    return launch_k(kv4_load_kernel<__nv_bfloat16>, dim3(rp.ctas), dim3(256), 0, s, false,
                    static_cast<const uint8_t*>(pool), n_slots, slots, n, d_c, d_r, rb,
                    static_cast<__nv_bfloat16*>(out), rp.fly, status);
}

}  // namespace lcs
