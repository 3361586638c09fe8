// Bookkeeping of the paged key/value cache: block tables and slot maps from request lengths,
// and the copy of new rows to their slots.
//
// Plan. Request b holds cached_b tokens in ceil(cached_b / P) pages and brings new_b more, so it
// needs ceil((cached_b + new_b) / P) - ceil(cached_b / P) pages from the free list. Two prefix
// sums over the requests (new tokens and pages needed, one packed 64-bit scan) say where its
// queries start and which free pages are its own; everything else is a lookup. The work is a few
// hundred kilobytes at most, so a launch is bound by latency, not by bytes: one launch in all.
// Every block repeats the scan, whose result sits in shared memory, and fills its share of the
// slots. kv_len may be cached_len and free_head_out may be free_head (a step replayed from a
// CUDA graph advances them in place): up to kOneBlockTokens slots one block does everything;
// beyond, the blocks form one cluster and meet after their last read of those arrays.
// In a graph: 32 requests with a token each 4.9 us, 256 requests with 65000 tokens 7.6 us.
#include <cstdint>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "relattn_paged.cuh"

namespace relattn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;          // portable cluster size
constexpr int kOneBlockTokens = 8192;
constexpr int kInvalidArg = 1;           // RELATTN_ERR_INVALID_ARG in the status word
// The packed scan: tokens in the low kTokenBits (at most kPlanMaxSeqs * kPlanMaxTokens = 2^37),
// pages above. A request is placed only while the tokens so far fit max_tokens <= 2^23, and each
// new page holds a new token, so up to there the pages stay below 2^24 and nothing wraps.
constexpr int kTokenBits = 40;
static_assert((1ull << kTokenBits) > (uint64_t)kPlanMaxSeqs * kPlanMaxTokens, "token sum");
static_assert(kPlanMaxTokens < (1 << (64 - kTokenBits)), "page sum");

struct PlanParams {
    PagedPlanArgs a;
    int shift;                           // log2(page_size)
};

__device__ __forceinline__ uint64_t scan_warp(uint64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Shared memory: start[B + 1] (first query row of each request), cached[B], page[B]: the index in
// the free list of the request's first new page, or -1 for a request that is not placed.
template <int CL>
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PlanParams p) {
    extern __shared__ int sm[];
    const PagedPlanArgs &a = p.a;
    const int B = a.B, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = a.page_size, sh = p.shift;
    int *start = sm, *cached_s = sm + B + 1, *page_s = cached_s + B;
    __shared__ uint64_t warp_sum[kPlanThreads / 32];
    __shared__ int taken_s;
    const int head = *a.free_head;
    const bool first_block = CL == 1 || blockIdx.x == 0;
    if (tid == 0) taken_s = 0;
    // ---- the scan, kPlanThreads requests at a time
    uint64_t carry = 0;
    bool bad_any = false;
    for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int c = 0, n = 0, need = 0;
        bool bad = false;
        if (b < B) {
            c = a.cached_len[b];
            n = a.new_len[b];
            bad = c < 0 || n < 0 || n > a.max_tokens;
            const long long tot = ((long long)c + n + P - 1) >> sh;
            const int old = (int)(((long long)c + P - 1) >> sh);
            bad = bad || tot > a.max_pages || (long long)c + n > 0x7fffffffLL;
            need = bad ? 0 : (int)tot - old;
        }
        n = n < 0 || n > a.max_tokens ? 0 : n;
        const uint64_t mine = ((uint64_t)need << kTokenBits) | (uint64_t)n;
        uint64_t v = scan_warp(mine, lane);
        __syncthreads();  // the previous round's sums have been read
        if (lane == 31) warp_sum[warp] = v;
        __syncthreads();
        if (warp == 0) {
            const uint64_t s = scan_warp(warp_sum[lane], lane);
            warp_sum[lane] = s;
        }
        __syncthreads();
        if (warp > 0) v += warp_sum[warp - 1];
        v += carry;
        carry += warp_sum[kPlanThreads / 32 - 1];
        if (b < B) {
            const long long incl = (long long)(v >> kTokenBits);
            const long long tokens = (long long)(v & ((1ull << kTokenBits) - 1));
            const bool placed = !bad && tokens <= a.max_tokens && (need == 0 || (head >= 0 && head + incl <= a.num_free));
            start[b + 1] = (int)(tokens < 0x7fffffffLL ? tokens : 0x7fffffffLL);
            cached_s[b] = c;
            page_s[b] = placed ? (need ? head + (int)incl - need : 0) : -1;
            if (placed && need) atomicMax(&taken_s, (int)incl);
            bad_any = bad_any || !placed;
        }
    }
    if (tid == 0) start[0] = 0;
    // every read of arrays that may be written in place is done in all blocks after this
    if (CL > 1)
        cooperative_groups::this_cluster().sync();
    else
        __syncthreads();
    const int total = start[B];
    const int taken = taken_s;
    if (first_block) {
        for (int b = tid; b <= B; b += kPlanThreads) a.q_start[b] = start[b];
        for (int b = tid; b < B; b += kPlanThreads)
            a.kv_len[b] = cached_s[b] + (page_s[b] >= 0 ? start[b + 1] - start[b] : 0);
        if (tid == 0) {
            *a.free_head_out = head + taken;
            bad_any = bad_any || total > a.max_tokens;
        }
        if (bad_any) atomicCAS(a.err, 0, kInvalidArg);
    }
    // ---- new entries of the block table, one warp per request
    const int gwarp = (CL > 1 ? (int)blockIdx.x : 0) * (kPlanThreads / 32) + warp;
    for (int b = gwarp; b < B; b += CL * (kPlanThreads / 32)) {
        if (page_s[b] < 0) continue;
        const int c = cached_s[b], n = start[b + 1] - start[b];
        const int old = (int)(((long long)c + P - 1) >> sh);
        const int need = (int)(((long long)c + n + P - 1) >> sh) - old;
        int *row = a.block_table + (long long)b * a.bt_stride + old;
        for (int i = lane; i < need; i += 32) row[i] = a.free_pages[page_s[b] + i];
    }
    // ---- slots, four tokens at a time: a binary search finds the first one's request
    const int gtid = (CL > 1 ? (int)blockIdx.x : 0) * kPlanThreads + tid;
    for (int t0 = 4 * gtid; t0 < a.max_tokens; t0 += 4 * CL * kPlanThreads) {
        int b = 0;
        if (t0 < total) {  // the last b with start[b] <= t0 (it has tokens: start[b + 1] > t0)
            int hi = B;
            while (hi - b > 1) {
                const int mid = (b + hi) >> 1;
                if (start[mid] <= t0) b = mid; else hi = mid;
            }
        }
        int out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + i;
            out[i] = -1;
            if (t >= total || t >= a.max_tokens) continue;
            while (start[b + 1] <= t) ++b;
            if (page_s[b] < 0) continue;
            const int c = cached_s[b], pos = c + (t - start[b]);
            const int old = (int)(((long long)c + P - 1) >> sh), pg = pos >> sh;
            const int page = pg < old ? a.block_table[(long long)b * a.bt_stride + pg]
                                      : a.free_pages[page_s[b] + pg - old];
            out[i] = page * P + (pos & (P - 1));
        }
        if (t0 + 4 <= a.max_tokens && (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0) {
            *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(out[0], out[1], out[2], out[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t0 + i < a.max_tokens) a.slots[t0 + i] = out[i];
        }
    }
}

// ---- append: row t of K and V to slot slots[t]. A pure copy, bound by HBM (each byte read and
// written once). One thread moves one vector of ROWS tokens' K and V, loads before stores.
// 16384 tokens of 8 heads of 128 (bf16): 22.2 us, 6.0 TB/s; 32 tokens of 16 heads of 64: 2.1 us.
constexpr int kAppendThreads = 256;

template <typename V, int ROWS>
__global__ void __launch_bounds__(kAppendThreads)
    paged_append_kernel(const __grid_constant__ PagedAppendArgs a, int vpt, int vpr, int shift) {
    // vpt: vectors per token, vpr: vectors per row of d elements
    const long long idx = (long long)blockIdx.x * kAppendThreads + threadIdx.x;
    const int tb = (int)(idx / vpt);
    const int i = (int)(idx - (long long)tb * vpt);
    const int t0 = tb * ROWS;
    if (t0 >= a.tokens) return;
    constexpr int E = sizeof(V);
    const int h = i / vpr, c = i - h * vpr;
    const long long eb = a.elem_bytes;
    V kx[ROWS], vx[ROWS];
    int slot[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int t = t0 + r;
        slot[r] = t < a.tokens ? a.slots[t] : -1;
        if (t < a.tokens) {
            kx[r] = *reinterpret_cast<const V *>(static_cast<const char *>(a.k) + (long long)t * a.k_stride * eb +
                                                 (long long)i * E);
            vx[r] = *reinterpret_cast<const V *>(static_cast<const char *>(a.v) + (long long)t * a.v_stride * eb +
                                                 (long long)i * E);
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (slot[r] < 0) continue;
        const int page = slot[r] >> shift, row = slot[r] & (a.page_size - 1);
        if (page >= a.num_pages) {
            if (i == 0) atomicCAS(a.err, 0, kInvalidArg);
            continue;
        }
        const long long off = (long long)page * a.page_stride * eb +
                              ((long long)h * a.page_size + row) * a.d * eb + (long long)c * E;
        *reinterpret_cast<V *>(static_cast<char *>(a.k_pages) + off) = kx[r];
        *reinterpret_cast<V *>(static_cast<char *>(a.v_pages) + off) = vx[r];
    }
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

template <typename V, int ROWS>
cudaError_t append_v(const PagedAppendArgs &a, cudaStream_t s) {
    const long long vpr = (long long)a.d * a.elem_bytes / (long long)sizeof(V), vpt = a.Hkv * vpr;
    if (vpt > 0x7fffffffLL) return cudaErrorNotSupported;
    const long long units = ((long long)a.tokens + ROWS - 1) / ROWS * vpt;
    const long long blocks = (units + kAppendThreads - 1) / kAppendThreads;
    if (blocks > 0x7fffffffLL) return cudaErrorNotSupported;
    paged_append_kernel<V, ROWS><<<(unsigned)blocks, kAppendThreads, 0, s>>>(a, (int)vpt, (int)vpr,
                                                                             log2_of(a.page_size));
    return cudaGetLastError();
}

template <typename V>
cudaError_t append_rows(const PagedAppendArgs &a, cudaStream_t s) {
    // few tokens: one row a thread, so that more threads share the latency; many: two in flight
    return a.tokens < 1024 ? append_v<V, 1>(a, s) : append_v<V, 2>(a, s);
}

}  // namespace

cudaError_t launch_paged_plan(const PagedPlanArgs &a, cudaStream_t s) {
    PlanParams p{a, log2_of(a.page_size)};
    const size_t smem = (size_t)(3 * a.B + 1) * sizeof(int);
    const bool one = a.max_tokens <= kOneBlockTokens;
    const void *kern = one ? reinterpret_cast<const void *>(paged_plan_kernel<1>)
                           : reinterpret_cast<const void *>(paged_plan_kernel<kPlanCluster>);
    if (smem > 48 * 1024) {
        const cudaError_t e = paged::opt_in_smem(kern, paged::device_info());
        if (e != cudaSuccess) return e;
    }
    if (one) {
        paged_plan_kernel<1><<<1, kPlanThreads, smem, s>>>(p);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kPlanCluster);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kPlanCluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_plan_kernel<kPlanCluster>, p);
}

cudaError_t launch_paged_append(const PagedAppendArgs &a, cudaStream_t s) {
    const long long row = (long long)a.d * a.elem_bytes;
    const uint64_t m = (uint64_t)row | (uint64_t)(a.k_stride * a.elem_bytes) |
                       (uint64_t)(a.v_stride * a.elem_bytes) | (uint64_t)(a.page_stride * a.elem_bytes) |
                       reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                       reinterpret_cast<uintptr_t>(a.k_pages) | reinterpret_cast<uintptr_t>(a.v_pages);
    if (m % 16 == 0) return append_rows<uint4>(a, s);
    if (m % 4 == 0) return append_rows<uint32_t>(a, s);
    return append_rows<uint16_t>(a, s);
}

}  // namespace relattn
