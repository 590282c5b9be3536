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
            const int64_t nb1 = (r.len + r.n + P - 1) / P;
            v[0] = nb1 - (r.len + P - 1) / P;
            v[1] = (r.len + r.n) / o0.m - r.len / o0.m;
            v[2] = o1.m > 0 ? (r.len + r.n) / m1 - r.len / m1 : 0;
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
        table[(int64_t)b * max_blocks + (r.len + P - 1) / P + (i - off[0][b])] = free_blocks[i];
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const PlanOut o = s ? o1 : o0;
        if (o.m == 0) continue;
        const int per = P / o.m;
        for (int64_t i = gt; i < o.max; i += gn) {
            int64_t slot = -1;
            if (i < total[1 + s]) {
                const int b = plan_find(off[1 + s], B, (int)i);
                const PlanReq r = plan_req(len, n_new, b);
                const int64_t j = r.len / o.m + (i - off[1 + s][b]);
                const int64_t bi = j / per, nb0 = (r.len + P - 1) / P;
                const int64_t id = bi >= nb0 ? free_blocks[off[0][b] + (bi - nb0)] : table[(int64_t)b * max_blocks + bi];
                slot = id < 0 ? -1 : id * per + (j - bi * per);
            }
            o.slots[i] = slot;
        }
    }
}

// ---------------------------------------------------------- 4-bit rows: write, read
// Loads 16 consecutive elements as fp32.
__device__ __forceinline__ void load16(const float* p, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
        v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
            v[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ uint16_t to_bf16_bits(float v) { return f32_to_bf16_bits(v); }
__device__ __forceinline__ uint16_t to_bf16_bits(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }

// One warp per row; two lanes share a 32-element block, 16 elements each: the block's amax is
// one shuffle, the lane's codes one 8-byte store.
template <typename T>
__global__ void __launch_bounds__(256) kv4_store_kernel(const T* __restrict__ x, const int64_t* __restrict__ slots,
                                                        int64_t n, int d_c, int d_r, int row_bytes,
                                                        uint8_t* __restrict__ pool, int64_t n_slots, int* status) {
    const int lane = threadIdx.x & 31;
    const int64_t stride = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t r = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < n; r += stride) {
        const int64_t slot = __ldg(slots + r);
        if (slot < 0) continue;
        if (slot >= n_slots) {
            if (lane == 0) set_status(status, LCS_ERR_DEVICE, 502);
            continue;
        }
        const T* xr = x + r * (d_c + d_r);
        uint8_t* o = pool + slot * row_bytes;
        for (int p0 = 0; p0 < d_c / 16; p0 += 32) {
            const int p = p0 + lane;
            const bool in = p < d_c / 16;   // the same for both lanes of a block: d_c / 16 is even
            float v[16] = {};
            if (in) load16(xr + 16 * p, v);
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            if (!in) continue;
            uint8_t sc_code = f32_to_e4m3(amax / 6.0f);
            if ((sc_code & 0x7F) == 0) sc_code = 0x38;   // 1.0
            const float sc = e4m3_to_f32(sc_code);
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i >> 3] |= (uint32_t)f32_to_e2m1(v[i] / sc) << (4 * (i & 7));
            *reinterpret_cast<uint2*>(o + 8 * p) = make_uint2(w[0], w[1]);
            if ((p & 1) == 0) o[d_c / 2 + 2 * d_r + p / 2] = sc_code;
        }
        for (int j = lane; j < d_r; j += 32) *reinterpret_cast<uint16_t*>(o + d_c / 2 + 2 * j) = to_bf16_bits(xr[d_c + j]);
        // the bytes past the last scale (row padding) are zeros
        for (int j = d_c / 2 + 2 * d_r + d_c / 32 + lane; j < row_bytes; j += 32) o[j] = 0;
    }
}

// One warp per row: code x scale is exact in bf16 (six significant bits), the RoPE dims are bf16.
template <typename T>
__global__ void __launch_bounds__(256) kv4_load_kernel(const uint8_t* __restrict__ pool, int64_t n_slots,
                                                       const int64_t* __restrict__ slots, int64_t n, int d_c, int d_r,
                                                       int row_bytes, T* __restrict__ out, int* status) {
    const int lane = threadIdx.x & 31;
    const int64_t stride = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t r = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < n; r += stride) {
        int64_t slot = __ldg(slots + r);
        if (slot >= n_slots) {
            if (lane == 0) set_status(status, LCS_ERR_DEVICE, 503);
            slot = -1;
        }
        T* o = out + r * (d_c + d_r);
        const uint8_t* src = pool + (slot < 0 ? 0 : slot) * row_bytes;
        for (int p = lane; p < d_c / 16; p += 32) {
            float v[16];
            if (slot >= 0) {
                const uint2 c = *reinterpret_cast<const uint2*>(src + 8 * p);
                const float sc = e4m3_to_f32(src[d_c / 2 + 2 * d_r + p / 2]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t byte = ((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xFFu;
                    const float2 f = e2m1x2_to_f32(byte);
                    v[2 * i] = f.x * sc, v[2 * i + 1] = f.y * sc;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = 0.f;
            }
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    reinterpret_cast<float4*>(o + 16 * p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    reinterpret_cast<uint4*>(o + 16 * p)[i] =
                        make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                   pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
            }
        }
        for (int j = lane; j < d_r; j += 32) {
            const uint16_t h = slot >= 0 ? *reinterpret_cast<const uint16_t*>(src + d_c / 2 + 2 * j) : (uint16_t)0;
            if constexpr (sizeof(T) == 4) o[d_c + j] = bf16_bits_to_f32(h);
            else o[d_c + j] = __ushort_as_bfloat16(h);
        }
    }
}

unsigned rows_grid(int64_t n) {
    const int64_t ctas = (n + 7) / 8, most = (int64_t)num_sms() * 8;
    return (unsigned)(ctas < most ? ctas : most);
}

}  // namespace

int page_plan_max_requests() { return kPlanMaxB; }

cudaError_t launch_page_plan(int64_t B, const int64_t* len, const int64_t* n_new, int block_tokens,
                             const int32_t* free_blocks, int64_t n_free, int32_t* table, int64_t max_blocks, int m,
                             int64_t* slots, int64_t max_slots, int64_t* off, int m2, int64_t* slots2,
                             int64_t max_slots2, int64_t* off2, int64_t* taken, int* status, cudaStream_t s) {
    const size_t smem = 3 * (size_t)(B + 1) * sizeof(int);
    cudaError_t e = set_smem_here(reinterpret_cast<const void*>(page_plan_kernel), smem);
    if (e != cudaSuccess) return e;
    // a CTA per 4 slots a thread, at most one per SM (each repeats the scan of the lengths)
    const int64_t outs = max_slots + (m2 > 0 ? max_slots2 : 0);
    int64_t ctas = (outs + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
    if (ctas < 1) ctas = 1;
    if (ctas > num_sms()) ctas = num_sms();
    const PlanOut o0{m, max_slots, slots, off}, o1{m2, max_slots2, slots2, off2};
    return launch_k(page_plan_kernel, dim3((unsigned)ctas), dim3(kPlanThreads), smem, s, false, (int)B, len, n_new,
                    block_tokens, free_blocks, n_free, table, max_blocks, o0, o1, taken, status);
}

cudaError_t launch_kv4_store(const void* x, int x_dtype, int64_t n, int d_c, int d_r, const int64_t* slots, void* pool,
                             int64_t n_slots, int* status, cudaStream_t s) {
    if (n == 0) return cudaSuccess;
    const int rb = kv4_row_bytes(d_c, d_r);
    if (x_dtype == LCS_F32)
        return launch_k(kv4_store_kernel<float>, dim3(rows_grid(n)), dim3(256), 0, s, false,
                        static_cast<const float*>(x), slots, n, d_c, d_r, rb, static_cast<uint8_t*>(pool), n_slots,
                        status);
    return launch_k(kv4_store_kernel<__nv_bfloat16>, dim3(rows_grid(n)), dim3(256), 0, s, false,
                    static_cast<const __nv_bfloat16*>(x), slots, n, d_c, d_r, rb, static_cast<uint8_t*>(pool), n_slots,
                    status);
}

cudaError_t launch_kv4_load(const void* pool, int64_t n_slots, const int64_t* slots, int64_t n, int d_c, int d_r,
                            void* out, int out_dtype, int* status, cudaStream_t s) {
    if (n == 0) return cudaSuccess;
    const int rb = kv4_row_bytes(d_c, d_r);
    if (out_dtype == LCS_F32)
        return launch_k(kv4_load_kernel<float>, dim3(rows_grid(n)), dim3(256), 0, s, false,
                        static_cast<const uint8_t*>(pool), n_slots, slots, n, d_c, d_r, rb, static_cast<float*>(out),
                        status);
    return launch_k(kv4_load_kernel<__nv_bfloat16>, dim3(rows_grid(n)), dim3(256), 0, s, false,
                    static_cast<const uint8_t*>(pool), n_slots, slots, n, d_c, d_r, rb,
                    static_cast<__nv_bfloat16*>(out), status);
}

}  // namespace lcs
