// attend_kv4.cu -- shared-KV MQA over a paged cache held in 4 bits (CSA sparse; HCA dense).
//
// "DeepSeek V4 深度解析" §2, CSA step 3 and HCA paragraph (the attention), §4 (the cache in
// blocks; FP4).  For query (b,q) and head h, over the compressed rows and the window rows R
// that the query sees:
//   o_h = sum_r softmax_r(scale * q_h . K_r) V_r,   V_r = the d_c content dims of K_r.
// A compressed row is stored as E2M1 codes with an E4M3 scale per 32 content dims and bf16
// RoPE dims (LCS_KV_FP4); entry e of request b lies in block table[b][e / be], row e mod be.
#include <utility>

#include "lcs_common.cuh"
#include "lcs_internal.h"

namespace lcs {

namespace {

// Entries of request b that exist: n_entries[b], within what the table can hold.
__device__ __forceinline__ int64_t kv4_entries(const AttendKv4Args& a, int64_t b, int* status) {
    int64_t n = a.n_entries[b];
    const int64_t most = a.max_blocks * a.be;
    if (n > most) {
        set_status(status, LCS_ERR_DEVICE, 601);
        n = most;
    }
    return n < 0 ? 0 : n;
}

// Entries that HCA query g attends.
__device__ __forceinline__ int64_t kv4_avail(const AttendKv4Args& a, int64_t g, int64_t n) {
    if (a.q_pos == nullptr) return n;
    const int64_t p = a.q_pos[g];
    const int64_t av = p < 0 ? 0 : (p + 1) / a.m;
    return av < n ? av : n;
}

struct Kv4Window {
    int64_t lo, n;
};
__device__ __forceinline__ Kv4Window kv4_window(const AttendKv4Args& a, int64_t g, int64_t b) {
    Kv4Window w{0, a.Tw};
    if (a.q_pos == nullptr) {
        if (a.n_win != nullptr) {
            const int64_t n = a.n_win[b];
            w.n = n < 0 ? 0 : (n < a.Tw ? n : a.Tw);
        }
        return w;
    }
    const int64_t t = a.q_pos[g], p0 = a.win_pos0[b];
    int64_t lo = t - a.W + 1 - p0, hi = t - p0;
    if (lo < 0) lo = 0;
    if (hi > a.Tw - 1) hi = a.Tw - 1;
    w.lo = lo;
    w.n = hi >= lo ? hi - lo + 1 : 0;
    return w;
}

// Row of entry e (0 <= e < kv4_entries) of request b, or null when its block is not one of the
// pool's (recorded in the status word).
__device__ __forceinline__ const uint8_t* kv4_row(const AttendKv4Args& a, int64_t b, int e, int* status) {
    const int bi = e / a.be;
    const int32_t id = __ldg(a.table + b * a.max_blocks + bi);
    if (id < 0 || id >= a.n_blocks) {
        set_status(status, LCS_ERR_DEVICE, 602);
        return nullptr;
    }
    return a.pool + ((int64_t)id * a.be + (e - bi * a.be)) * a.row_bytes;
}

// ------------------------------------------------------------ CUDA-core path
// Every shape: H <= 128, d_c % 32 == 0 and <= 512, d_r <= 128, fp32 or bf16 queries.  One CTA per
// query and group of 8 heads: 32 rows at a time widened to fp32 in shared memory, the scores
// by one thread per (head, row), an online softmax by one warp per head, the outputs in
// registers.  Bound by shared-memory reads (two per multiply-add); it serves the small shapes.
constexpr int kSThreads = 256, kSRows = 32, kSHeads = 8;
constexpr int kSMaxDc = 512;
constexpr int kSAcc = kSHeads * kSMaxDc / kSThreads;

__device__ __forceinline__ float ld_elem(const void* p, int64_t i, int dtype) {
    return dtype == LCS_F32 ? static_cast<const float*>(p)[i]
                            : bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

__global__ void __launch_bounds__(kSThreads) attend_kv4_kernel(const AttendKv4Args a, int* status) {
    extern __shared__ float sh[];
    const int D = a.d_c + a.d_r, pitch = D + 1;
    float* qs = sh;                          // [heads, D]
    float* rows = qs + kSHeads * D;          // [32, D + 1]
    float* sc = rows + kSRows * pitch;       // [heads, 33]
    float* al = sc + kSHeads * (kSRows + 1); // [heads] rescale of this chunk
    float* lh = al + kSHeads;                // [heads] sums
    __shared__ int nsel_s;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t g = blockIdx.x, b = g / a.Q;
    const int h0 = blockIdx.y * kSHeads, nh = min(kSHeads, a.H - h0);

    for (int i = t; i < nh * D; i += kSThreads) qs[i] = ld_elem(a.q, (g * a.H + h0) * D + i, a.q_dtype);
    const int64_t n = kv4_entries(a, b, status);
    const int32_t* sel = a.idx != nullptr ? a.idx + g * a.k : nullptr;
    if (t == 0) nsel_s = sel != nullptr ? a.k : (int)kv4_avail(a, g, n);
    __syncthreads();
    if (sel != nullptr)
        for (int i = t; i < a.k; i += kSThreads) {
            const int32_t v = sel[i];
            if (v >= 0 && v < n) continue;
            if (v >= n) set_status(status, LCS_ERR_DEVICE, 603);
            atomicMin(&nsel_s, i);
        }
    __syncthreads();
    const int64_t nsel = nsel_s;
    const Kv4Window win = kv4_window(a, g, b);
    const int64_t R = nsel + win.n;

    float acc[kSAcc];
#pragma unroll
    for (int i = 0; i < kSAcc; ++i) acc[i] = 0.f;
    float m = -INFINITY, l = 0.f;            // of head `warp`, the same in every lane
    const int blocks = a.d_c / 32;
    for (int64_t r0 = 0; r0 < R; r0 += kSRows) {
        const int nr = (int)(R - r0 < kSRows ? R - r0 : kSRows);
        const int nc = (int)(nsel - r0 < 0 ? 0 : (nsel - r0 < nr ? nsel - r0 : nr));   // compressed rows among them
        for (int i = t; i < nc * blocks; i += kSThreads) {
            const int r = i / blocks, bl = i - r * blocks;
            const uint8_t* src = kv4_row(a, b, sel != nullptr ? sel[r0 + r] : (int)(r0 + r), status);
            float* o = rows + r * pitch + 32 * bl;
            const uint4 c = src != nullptr ? __ldg(reinterpret_cast<const uint4*>(src) + bl) : make_uint4(0, 0, 0, 0);
            const float s = src != nullptr ? e4m3_to_f32(src[a.d_c / 2 + 2 * a.d_r + bl]) : 0.f;
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float2 f = e2m1x2_to_f32(w[k >> 2] >> (8 * (k & 3)));
                o[2 * k] = f.x * s;
                o[2 * k + 1] = f.y * s;
            }
        }
        for (int i = t; i < nc * a.d_r; i += kSThreads) {
            const int r = i / a.d_r, j = i - r * a.d_r;
            const uint8_t* src = kv4_row(a, b, sel != nullptr ? sel[r0 + r] : (int)(r0 + r), status);
            rows[r * pitch + a.d_c + j] =
                src != nullptr ? bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(src + a.d_c / 2 + 2 * j)) : 0.f;
        }
        for (int i = t; i < (nr - nc) * D; i += kSThreads) {
            const int r = i / D, j = i - r * D;
            rows[(nc + r) * pitch + j] = ld_elem(a.win, (b * a.Tw + win.lo + (r0 + nc + r - nsel)) * D + j, a.q_dtype);
        }
        __syncthreads();
        {   // thread = (head, row): a warp's lanes take the 32 rows of one head
            float s = -INFINITY;
            if (warp < nh && lane < nr) {
                const float* qh = qs + warp * D;
                const float* rr = rows + lane * pitch;
                s = 0.f;
                for (int c = 0; c < D; ++c) s = fmaf(qh[c], rr[c], s);
                s *= a.scale;
            }
            const float mx = fmaxf(m, warp_max(s));
            const float alpha = m == -INFINITY ? 0.f : expf(m - mx);
            const float p = s == -INFINITY ? 0.f : expf(s - mx);
            l = l * alpha + warp_sum(p);
            m = mx;
            if (warp < nh) {
                sc[warp * (kSRows + 1) + lane] = p;
                if (lane == 0) al[warp] = alpha;
            }
        }
        __syncthreads();
        // thread = (head, output dim): 16 per thread at most
#pragma unroll
        for (int i = 0; i < kSAcc; ++i) {
            const int j = t + kSThreads * i;
            if (j >= nh * a.d_c) break;
            const int h = j / a.d_c, c = j - h * a.d_c;
            float o = acc[i] * al[h];
            for (int r = 0; r < nr; ++r) o = fmaf(sc[h * (kSRows + 1) + r], rows[r * pitch + c], o);
            acc[i] = o;
        }
        __syncthreads();
    }
    if (warp < nh && lane == 0) {
        lh[warp] = l;
        if (a.lse != nullptr) a.lse[g * a.H + h0 + warp] = l > 0.f ? m + logf(l) : -INFINITY;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSAcc; ++i) {
        const int j = t + kSThreads * i;
        if (j >= nh * a.d_c) break;
        const int h = j / a.d_c;
        const float o = lh[h] > 0.f ? acc[i] / lh[h] : 0.f;
        const int64_t at = (g * a.H + h0) * a.d_c + j;
        if (a.out_dtype == LCS_F32) static_cast<float*>(a.out)[at] = o;
        else static_cast<uint16_t*>(a.out)[at] = f32_to_bf16_bits(o);
    }
}

}  // namespace

int64_t attend_kv4_scratch_bytes(const AttendKv4Args&) { return 0; }

cudaError_t launch_attend_kv4(const AttendKv4Args& a, void*, int* status, cudaStream_t s) {
    const int64_t queries = a.B * a.Q;
    if (queries == 0) return cudaSuccess;
    const int D = a.d_c + a.d_r;
    const size_t smem = sizeof(float) * (kSHeads * D + kSRows * (D + 1) + kSHeads * (kSRows + 1) + 2 * kSHeads);
    cudaError_t e = set_smem_here(reinterpret_cast<const void*>(attend_kv4_kernel), smem);
    if (e != cudaSuccess) return e;
    return launch_k(attend_kv4_kernel, dim3((unsigned)queries, (unsigned)((a.H + kSHeads - 1) / kSHeads)),
                    dim3(kSThreads), smem, s, false, a, status);
}

}  // namespace lcs
