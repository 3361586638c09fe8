// Eviction from the paged cache: of every request that has grown past `limit` keys, each key/value
// head keeps `budget`: its first `sinks`, its last `recent`, and of the others those with the most
// accumulated weight, ties to the earlier key. The kept keys close up in place, in their order.
//
// Selection. A unit is one head of one such request, taken by a cluster of 1, 2, 4 or 8 CTAs (as many
// as the longest row of the table can use, 16384 keys each; shorter tables have smaller CTAs). The CTAs hold their keys' weights in
// registers, as integers in the same order, and find the budget's last weight by three histograms
// (11, 11 and 10 bits) that they add up over distributed shared memory: the weights are read once. A
// unit past the cluster's registers reads them again (out of L2) in each pass. What comes out is
// 128 bits for every run of 128 keys, and the kept keys in front of it.
//
// Moving. Key r of the kept ones comes from place j_r >= r. A block is a run of consecutive places to
// fill; CTAs take the blocks by ticket, in order, read their rows into registers, and write them
// when what still stands in those places has been read: it goes to the same or an earlier block, so
// a wait is always for a CTA that is already running and that reads before it waits. Rows that stay
// in place are neither read nor written. HBM bounds it: every moved row is read once, written once.
// A block is as many places (128 at most) as a CTA's registers hold at once.
//
// Measured in a graph, each pass on a cache that no other has cut (what a cut leaves behind its budget are copies of what it
// has kept, so a second cut of the same cache moves other rows, in the end few). 64 requests of 2000 - 2304 keys cut to 2048,
// 4 heads of 128: 123 us, 441 MB read and written (3.6 TB/s), 21 us of them the selection. 131071 keys cut to 32768, 4 heads:
// 66 us (135 MB), of which 30 are the selection (four units, so 32 CTAs: three passes of 5 us and the runs' list); the moving
// takes four rounds of 9 us, each a chain of the list's lookups, the rows' latency and the flags. Tried and dropped, on caches
// that had been cut before: the next block's lookups while this one's rows arrive (101 -> 118 us), blocks of 64 places with
// three or four CTAs an SM (106, 112), clusters of 16 for few units (evict of one long request 75 -> 84 us).
#include <cstdint>
#include <cstring>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "relattn_paged.cuh"

namespace relattn {
namespace {

namespace cg = cooperative_groups;

constexpr int kRun = 128;                    // keys of a run
constexpr int kLeastBlock = 16;              // places of a block at least
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
// runs whose weights a selecting CTA holds: four of each warp
__host__ __device__ constexpr int runs_held(int threads) { return threads / 8; }
constexpr int kMoveThreads = 256;
constexpr int kInFlight = 16;                // vectors of a thread on their way
constexpr int kTimeout = 4;                  // RELATTN_ERR_TIMEOUT in the status word
constexpr int kBitWords = kPlanMaxSeqs / 32;

struct EvictParams {
    PagedEvictArgs a;
    int shift, cap, runs;                    // log2(page_size), keys and runs that a table row can hold
    int block, blocks;                       // places of a block (a power of two), blocks of a table row at most
    int *state;                              // {ticket, requests to cut}
    int2 *list;                              // [B] of those requests: {request, keys}
    uint32_t *mask;                          // [unit][runs][4]: the kept keys of a run
    int *off;                                // [unit][runs + 1]: kept keys in front of it
    int *start;                              // [unit][blocks]: the run that holds a block's first key
    int *done;                               // [unit][blocks]: the block's rows have been read
};

size_t round16(size_t x) { return (x + 15) & ~(size_t)15; }

// the weights' bits in their order: equal weights have equal bits, a NaN counts as the largest
__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 becomes 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int length_of(const EvictParams &p, int b) { return min(max(p.a.kv_len[b], 0), p.cap); }

template <bool VEC, int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads)
    evict_select_kernel(const __grid_constant__ EvictParams p, int C) {
    constexpr int kSelWarps = kSelThreads / 32, kRunsHeld = runs_held(kSelThreads), kMine = kBins / kSelThreads;
    constexpr int kSums = kRunsHeld / 32;    // runs of a lane where a warp adds them all up
    __shared__ uint32_t hist[2][kBins];
    __shared__ uint32_t bits[kBitWords];
    __shared__ int before[kBitWords];        // requests to cut in front of each word
    __shared__ int warp_sum[kSelWarps], count[kRunsHeld];
    __shared__ int pick_bin, pick_rest, unit_b, totals[2], cut;
    const PagedEvictArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    paged::grid_wait();
    paged::grid_release();
    // ---- which requests are cut: a bit each
    for (int b0 = 0; b0 < a.B; b0 += kSelThreads) {
        const int b = b0 + tid;
        const unsigned m = __ballot_sync(0xffffffffu, b < a.B && length_of(p, b) > a.limit);
        if (lane == 0 && b0 + 32 * warp < a.B) bits[(b0 >> 5) + warp] = m;
    }
    __syncthreads();
    const int words = (a.B + 31) / 32;
    if (warp == 0) {
        int at = 0;
        for (int w0 = 0; w0 < words; w0 += 32) {
            const int n = w0 + lane < words ? __popc(bits[w0 + lane]) : 0;
            int v = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (w0 + lane < words) before[w0 + lane] = at + v - n;
            at += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) cut = at;
    }
    __syncthreads();
    const int requests = cut;
    if (blockIdx.x == 0) {
        if (tid == 0) {
            p.state[0] = 0;
            p.state[1] = requests;
        }
        for (int b = tid; b < a.B; b += kSelThreads) {
            const uint32_t w = bits[b >> 5];
            if (w >> (b & 31) & 1) p.list[before[b >> 5] + __popc(w & ((1u << (b & 31)) - 1))] = make_int2(b, length_of(p, b));
        }
    }
    const int units = requests * a.Hkv, groups = (int)gridDim.x / C;
    for (int u = (int)blockIdx.x / C; u < units; u += groups) {
        const int r = u / a.Hkv, h = u - r * a.Hkv;
        __syncthreads();
        for (int at = tid; at < words; at += kSelThreads) {
            const int i = r - before[at];
            if (i >= 0 && i < __popc(bits[at])) {   // the i-th bit of the word
                uint32_t w = bits[at];
                for (int q = 0; q < i; ++q) w &= w - 1;
                unit_b = 32 * at + __ffs(w) - 1;
            }
        }
        if (tid < 2) totals[tid] = 0;
        for (int i = tid; i < 2 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
        __syncthreads();
        const int b = unit_b, n = length_of(p, b);
        const int *bt = a.block_table + (long long)b * a.bt_stride;
        const int runs = (n + kRun - 1) / kRun, per = (runs + C - 1) / C;
        const int c0 = min(rank * per, runs), c1 = min(c0 + per, runs);
        const bool held = per <= kRunsHeld;
        const int lo = a.sinks, hi = n - a.recent;   // the keys that are weighed
        uint32_t key[4][4];
        auto load = [&](int base) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = base + i * kSelWarps + warp, j = c * kRun + 4 * lane;
#pragma unroll
                for (int e = 0; e < 4; ++e) key[i][e] = 0;
                if (c >= c1 || j >= n) continue;
                if (VEC) {
                    const int pg = bt[j >> p.shift];
                    if ((unsigned)pg >= (unsigned)a.num_pages) {
                        atomicCAS(a.err, 0, paged::kInvalidArg);
                        continue;
                    }
                    const float4 x = *reinterpret_cast<const float4 *>(a.mass + (long long)pg * a.mass_stride +
                                                                       (long long)h * a.page_size + (j & (a.page_size - 1)));
                    key[i][0] = ordered(x.x);
                    key[i][1] = ordered(x.y);
                    key[i][2] = ordered(x.z);
                    key[i][3] = ordered(x.w);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (j + e >= n) continue;
                        const int pg = bt[(j + e) >> p.shift];
                        if ((unsigned)pg >= (unsigned)a.num_pages) {
                            atomicCAS(a.err, 0, paged::kInvalidArg);
                            continue;
                        }
                        key[i][e] = ordered(a.mass[(long long)pg * a.mass_stride + (long long)h * a.page_size +
                                                   ((j + e) & (a.page_size - 1))]);
                    }
                }
            }
        };
        // ---- the last weight that is kept (bits T) and how many of that weight are
        uint32_t T = 0;
        int rest = a.budget - a.sinks - a.recent;
        if (held) load(c0);
        if (rest == 0) {
            T = 0xffffffffu;
        } else {
#pragma unroll 1
            for (int pass = 0; pass < 3; ++pass) {
                const int sh = pass == 0 ? 21 : pass == 1 ? 10 : 0, top = pass == 0 ? 0 : pass == 1 ? 21 : 10;
                uint32_t *hs = hist[pass & 1];
                for (int base = c0; base < c1; base += kRunsHeld) {
                    if (!held) load(base);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = base + i * kSelWarps + warp, j = c * kRun + 4 * lane;
                        if (c >= c1) continue;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (j + e >= lo && j + e < hi && (pass == 0 || key[i][e] >> top == T >> top))
                                atomicAdd(&hs[key[i][e] >> sh & (pass == 2 ? 1023u : 2047u)], 1u);
                    }
                }
                cluster.sync();
                for (int i = tid; i < kBins; i += kSelThreads) hist[(pass + 1) & 1][i] = 0;
                // bins from the top, kMine a thread, over the cluster
                const int d0 = kBins - kMine * (tid + 1);   // the thread's lowest
                int n[kMine];
#pragma unroll
                for (int e = 0; e < kMine; ++e) n[e] = 0;
                if (C == 1) {
#pragma unroll
                    for (int e = 0; e < kMine; ++e) n[e] = (int)hs[d0 + e];
                } else {
                    uint2 v[kMaxCluster][kMine / 2];   // (all on their way together)
#pragma unroll
                    for (int q = 0; q < kMaxCluster; ++q)
#pragma unroll
                        for (int e = 0; e < kMine; e += 2)
                            v[q][e / 2] = q < C ? *reinterpret_cast<const uint2 *>(cluster.map_shared_rank(hs, q) + d0 + e)
                                                : make_uint2(0, 0);
#pragma unroll
                    for (int q = 0; q < kMaxCluster; ++q)
#pragma unroll
                        for (int e = 0; e < kMine; e += 2) {
                            n[e] += (int)v[q][e / 2].x;
                            n[e + 1] += (int)v[q][e / 2].y;
                        }
                }
                int mine = 0;
#pragma unroll
                for (int e = 0; e < kMine; ++e) mine += n[e];
                int v = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += x;
                }
                if (lane == 31) warp_sum[warp] = v;
                __syncthreads();
                int s = lane < warp ? warp_sum[lane] : 0;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                int above = s + v - mine;   // keys in higher bins
#pragma unroll
                for (int e = kMine - 1; e >= 0; --e) {
                    if (above < rest && rest <= above + n[e]) {
                        pick_bin = d0 + e;
                        pick_rest = rest - above;
                    }
                    above += n[e];
                }
                __syncthreads();
                T |= (uint32_t)pick_bin << sh;
                rest = pick_rest;
            }
        }
        // ---- kept keys as bits. above: kept whatever happens; even: of the last weight
        auto flags = [&](int i, int c, unsigned &above, unsigned &even) {
            const int j = c * kRun + 4 * lane;
            above = even = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (c >= c1 || j + e >= n) continue;
                if (j + e < lo || j + e >= hi || key[i][e] > T) above |= 1u << e;
                else if (key[i][e] == T) even |= 1u << e;
            }
        };
        auto warp_total = [&](int x) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            return x;
        };
        int at_above = 0, at_even = 0;       // in front of this CTA's runs
        if (C > 1) {
            for (int base = c0; base < c1; base += kRunsHeld) {
                if (!held) load(base);
                int both = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    unsigned x, y;
                    flags(i, base + i * kSelWarps + warp, x, y);
                    both += __popc(x) + (__popc(y) << 16);
                }
                both = warp_total(both);     // at most 512 of either
                if (lane == 0) {
                    atomicAdd(&totals[0], both & 0xffff);
                    atomicAdd(&totals[1], both >> 16);
                }
            }
            cluster.sync();
            for (int q = 0; q < rank; ++q) {
                const int *t = cluster.map_shared_rank(totals, q);
                at_above += t[0];
                at_even += t[1];
            }
        }
        const long long ub = (long long)u * p.runs;
        for (int base = c0; base < c1; base += kRunsHeld) {
            if (!held) load(base);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                unsigned x, y;
                flags(i, base + i * kSelWarps + warp, x, y);
                const int both = warp_total(__popc(x) + (__popc(y) << 16));
                if (lane == 0) count[i * kSelWarps + warp] = both;
            }
            __syncthreads();
            // sums in front of every run: lane l of each warp has runs kSums l .. kSums l + kSums - 1
            int q[kSums], x_all = 0, y_all = 0;
#pragma unroll
            for (int e = 0; e < kSums; ++e) {
                q[e] = count[kSums * lane + e];
                x_all += q[e] & 0xffff;
                y_all += q[e] >> 16;
            }
            int xi = x_all, yi = y_all;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int s = __shfl_up_sync(0xffffffffu, xi, o), t = __shfl_up_sync(0xffffffffu, yi, o);
                if (lane >= o) {
                    xi += s;
                    yi += t;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int w = i * kSelWarps + warp, c = base + w;
                int xs = 0, ys = 0;          // of the runs in front of w
                {
                    int xa = xi - x_all, ya = yi - y_all;
#pragma unroll
                    for (int e = 0; e < kSums; ++e) {
                        if (e == w % kSums) {
                            xs = xa;
                            ys = ya;
                        }
                        xa += q[e] & 0xffff;
                        ya += q[e] >> 16;
                    }
                    xs = __shfl_sync(0xffffffffu, xs, w / kSums) + at_above;
                    ys = __shfl_sync(0xffffffffu, ys, w / kSums) + at_even;
                }
                if (c >= c1) continue;       // the whole warp alike
                unsigned x, y;
                flags(i, c, x, y);
                int rank_even = __popc(y);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int s = __shfl_up_sync(0xffffffffu, rank_even, o);
                    if (lane >= o) rank_even += s;
                }
                rank_even += ys - __popc(y);   // of the last weight, in front of this lane's keys
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (y >> e & 1) x |= rank_even++ < rest ? 1u << e : 0u;
                unsigned word = x << (4 * (lane & 7));
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
                const int kept = warp_total(__popc(x)), off = xs + min(ys, rest);
                if ((lane & 7) == 0) p.mask[(ub + c) * 4 + (lane >> 3)] = word;
                if (lane == 0) {
                    p.off[(long long)u * (p.runs + 1) + c] = off;
                    if (c == runs - 1) p.off[(long long)u * (p.runs + 1) + runs] = off + kept;
                }
                const int each = kRun / p.block, t = (off + p.block - 1) / p.block + lane;
                if (lane < each) p.done[(long long)u * p.blocks + c * each + lane] = 0;
                if (t < p.blocks && t * p.block < off + kept) p.start[(long long)u * p.blocks + t] = c;
            }
            at_above += __shfl_sync(0xffffffffu, xi, 31);
            at_even += __shfl_sync(0xffffffffu, yi, 31);
            __syncthreads();
        }
        if (C > 1) cluster.sync();           // the others have read this CTA's totals and histogram
    }
    if (C > 1) cluster.sync();               // nobody leaves while its shared memory may be read
}

// ------------------------------------------------------------------ lengths and free pages
// One block: kv_len_out, and the pages behind the budget back onto the list, request by request. Entries outside
// the cache are no pages and stay off it.
__device__ void evict_lengths(const EvictParams &p) {
    const PagedEvictArgs &a = p.a;
    __shared__ int warp_sum[kMoveThreads / 32], count_s[kMoveThreads], to_s[kMoveThreads];
    constexpr int kManyPages = 64;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = (int)(((long long)a.budget + a.page_size - 1) >> p.shift);
    const int requests = p.state[1];
    auto pages = [&](int i) { return (int)(((long long)p.list[i].y + a.page_size - 1) >> p.shift) - first; };
    auto row_of = [&](int i) { return a.block_table + (long long)p.list[i].x * a.bt_stride + first; };
    auto exists = [&](int page) { return (unsigned)page < (unsigned)a.num_pages; };
    // a request's length may be overwritten in place: only those in the list change
    if (a.kv_len_out != a.kv_len)
        for (int b = tid; b < a.B; b += kMoveThreads) {
            const int n = a.kv_len[b];
            if (min(max(n, 0), p.cap) <= a.limit) a.kv_len_out[b] = n;
        }
    for (int i = tid; i < requests; i += kMoveThreads) a.kv_len_out[p.list[i].x] = a.budget;
    if (!a.free_pages) return;
    auto block_scan = [&](int v, int &all) {   // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = v;
        __syncthreads();
        all = 0;
        for (int w = 0; w < kMoveThreads / 32; ++w) {
            if (w < warp) v += warp_sum[w];
            all += warp_sum[w];
        }
        return v;
    };
    // f(number, place on the list) of every entry: a warp takes a request's, or the block where they are many (again: their
    // numbers and places are in shared memory from the last time, where all requests fit)
    auto entries = [&](bool again, auto f) {
        int at = 0;
        for (int i0 = 0; i0 < requests; i0 += kMoveThreads) {
            if (!again || requests > kMoveThreads) {
                const int i = i0 + tid, n = i < requests ? pages(i) : 0;
                int sum;
                const int mine = at + block_scan(n, sum) - n;
                at += sum;
                __syncthreads();
                count_s[tid] = n;
                to_s[tid] = mine;
                __syncthreads();
            }
            const int here = min(kMoveThreads, requests - i0);
            for (int q = warp; q < here; q += kMoveThreads / 32) {
                const int nn = count_s[q];
                if (nn > kManyPages) continue;
                const int *row = row_of(i0 + q);
                for (int e = lane; e < nn; e += 32) f(row[e], to_s[q] + e);
            }
            for (int q = 0; q < here; ++q) {
                const int nn = count_s[q];
                if (nn <= kManyPages) continue;
                const int *row = row_of(i0 + q);
#pragma unroll 4
                for (int e = tid; e < nn; e += kMoveThreads) f(row[e], to_s[q] + e);
            }
            __syncthreads();
        }
        return at;
    };
    const int head = *a.free_head;
    int good = 0, all;
    const int total = entries(false, [&](int page, int) { good += exists(page); });
    block_scan(good, all);
    __syncthreads();
    if (all < total && tid == 0) atomicCAS(a.err, 0, paged::kInvalidArg);
    if (head > a.num_free || head < all) {   // not the list that the pages came from
        if (tid == 0) {
            *a.free_head_out = head;
            atomicCAS(a.err, 0, paged::kInvalidArg);
        }
        return;
    }
    if (tid == 0) *a.free_head_out = head - all;
    int *dst = a.free_pages + head - all;
    if (all == total) {
        entries(true, [&](int page, int to) { dst[to] = page; });
        return;
    }
    int at = 0;                                // some are left out: the places are counted
    for (int i = 0; i < requests; ++i) {
        const int n = pages(i), *row = row_of(i);
        for (int e0 = 0; e0 < n; e0 += kMoveThreads) {
            const int page = e0 + tid < n ? row[e0 + tid] : -1;
            int sum;
            const int to = at + block_scan(exists(page), sum) - 1;
            if (exists(page)) dst[to] = page;
            at += sum;
            __syncthreads();
        }
    }
}

// ------------------------------------------------------------------ moving
__device__ __forceinline__ int load_acquire(const int *p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(int *p, int v) {
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// vpr: vectors of a row of d elements. EVEN: a key's vectors (2 vpr) divide the threads, so that a thread's are
// all of one place in their rows (what goes for every row of a power of two; the addresses of a block take
// four times its loads otherwise)
template <typename V, bool EVEN>
__global__ void __launch_bounds__(kMoveThreads, 2) evict_move_kernel(const __grid_constant__ EvictParams p, int vpr) {
    __shared__ long long from_at[kRun], to_at[kRun];   // where the rows are: bytes behind k_pages or v_pages
    __shared__ int from[kRun], to[kRun];     // slots; -1: the row stays where it is
    __shared__ int item_s, ok_s;
    const PagedEvictArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    paged::grid_wait();
    paged::grid_release();
    if (blockIdx.x == 0) evict_lengths(p);
    const int units = p.state[1] * a.Hkv, blocks = (a.budget + p.block - 1) / p.block;
    const long long items = (long long)units * blocks;
    const int row_vecs = 2 * vpr;            // a block's fit the CTA's registers
    const int my_rem = tid % row_vecs, my_row = tid / row_vecs, row_step = kMoveThreads / row_vecs;   // EVEN
    const int P = a.page_size;
    auto base = [&](bool v) { return static_cast<char *>(v ? a.v_pages : a.k_pages); };
    int ahead = 0;                           // the next ticket, taken while this one's block is moved
    if (tid == 0) ahead = atomicAdd(&p.state[0], 1);
    for (;;) {
        if (tid == 0) item_s = ahead;
        if (tid < kRun) from[tid] = -1;
        __syncthreads();
        const int item = item_s;
        if (item < 0 || item >= items) break;
        if (tid == 0) ahead = atomicAdd(&p.state[0], 1);
        const int t = item / units, u = item - t * units, r = u / a.Hkv, h = u - r * a.Hkv;
        const int2 req = p.list[r];
        const int runs = (req.y + kRun - 1) / kRun;
        const int *bt = a.block_table + (long long)req.x * a.bt_stride;
        const int *off = p.off + (long long)u * (p.runs + 1);
        int *done = p.done + (long long)u * p.blocks;
        const int i0 = t * p.block, cnt = min(p.block, a.budget - i0), here = i0 / kRun;
        auto slot_of = [&](int j) -> int {
            const int pg = bt[j >> p.shift];
            if ((unsigned)pg < (unsigned)a.num_pages) return pg * P + (j & (P - 1));
            atomicCAS(a.err, 0, paged::kInvalidArg);
            return -1;
        };
        // the blocks that the kept keys of the places' run go to, as far as they are earlier ones
        const int dep0 = off[here] / p.block, dep1 = min((off[here + 1] - 1) / p.block, t - 1);
        // ---- the block's rows: a warp takes a run, four of its keys a lane
        for (int c = p.start[(long long)u * p.blocks + t] + warp; c < runs; c += kMoveThreads / 32) {
            int at = off[c];
            if (at >= i0 + cnt) break;
            const unsigned word = p.mask[((long long)u * p.runs + c) * 4 + (lane >> 3)], x = word >> (4 * (lane & 7)) & 15u;
            int s = __popc(x);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += v;
            }
            at += s - __popc(x) - i0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (x >> e & 1) {
                    const int j = c * kRun + 4 * lane + e;
                    if (at >= 0 && at < cnt) from[at] = j == i0 + at ? -1 : slot_of(j);
                    ++at;
                }
        }
        if (tid < cnt) to[tid] = slot_of(i0 + tid);
        __syncthreads();
        auto place = [&](int slot) { return (long long)(slot >> p.shift) * a.page_bytes + ((long long)h * P + (slot & (P - 1))) * a.row_bytes; };
        if (tid < cnt) {
            const bool moves = from[tid] >= 0 && to[tid] >= 0;
            from_at[tid] = moves ? place(from[tid]) : -1;
            to_at[tid] = moves ? place(to[tid]) : -1;
        }
        __syncthreads();
        // ---- rows into registers
        V x[kInFlight];
        float w = 0.f;
        // the k-th of this thread's vectors: its row (no less than cnt: none), and where in the row
        auto vector = [&](int k, int &row, char *&at) {
            int rem = my_rem;
            row = my_row + k * row_step;
            if (!EVEN) {
                const int i = tid + k * kMoveThreads;
                row = i / row_vecs;
                rem = i - row * row_vecs;
            }
            const bool kv = rem >= vpr;
            at = base(kv) + (long long)(rem - (kv ? vpr : 0)) * sizeof(V);
        };
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            int row;
            char *at;
            vector(k, row, at);
            if (row < cnt && from_at[row] >= 0) x[k] = *reinterpret_cast<const V *>(at + from_at[row]);
        }
        const int mine = tid < cnt && to[tid] >= 0 ? from[tid] : -1;
        if (mine >= 0) w = a.mass[(long long)(mine >> p.shift) * a.mass_stride + (long long)h * P + (mine & (P - 1))];
        __threadfence();                     // the rows have been read
        __syncthreads();
        if (tid == 0) {
            if (!a.withhold || t > 0) store_release(done + t, 1);
            int ok = 1;
            const long long t0 = clock64();
            for (int q = dep0; q <= dep1 && ok; ++q)
                while (!load_acquire(done + q))
                    if (clock64() - t0 > a.wait_limit) {
                        atomicCAS(a.err, 0, kTimeout);
                        ok = 0;
                        break;
                    }
            ok_s = ok;
        }
        __syncthreads();
        if (ok_s) {
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) {
                int row;
                char *at;
                vector(k, row, at);
                if (row < cnt && to_at[row] >= 0) *reinterpret_cast<V *>(at + to_at[row]) = x[k];
            }
            if (mine >= 0) {
                const int s = to[tid];
                a.mass[(long long)(s >> p.shift) * a.mass_stride + (long long)h * P + (s & (P - 1))] = w;
            }
        }
        __syncthreads();                     // from and to are free
    }
}


}  // namespace

// workspace: {ticket, count, -, -}, list, masks, offsets, starts, flags
unsigned long long paged_evict_workspace_bytes(int B, int Hkv, long long max_keys) {
    const size_t runs = (size_t)((max_keys + kRun - 1) / kRun), units = (size_t)B * Hkv;
    return 16 + round16((size_t)B * 8) + units * runs * (16 + 8 * (kRun / kLeastBlock)) + units * (runs + 1) * 4;
}

cudaError_t launch_paged_evict(const PagedEvictArgs &a, cudaStream_t s) {
    EvictParams p;
    std::memset(&p, 0, sizeof(p));
    p.a = a;
    while ((1 << p.shift) < a.page_size) ++p.shift;
    p.cap = a.max_pages << p.shift;
    p.runs = (p.cap + kRun - 1) / kRun;
    const size_t units = (size_t)a.B * a.Hkv;
    char *w = static_cast<char *>(a.workspace);
    p.state = reinterpret_cast<int *>(w);
    w += 16;
    p.list = reinterpret_cast<int2 *>(w);
    w += round16((size_t)a.B * 8);
    p.mask = reinterpret_cast<uint32_t *>(w);
    w += units * p.runs * 16;
    p.start = reinterpret_cast<int *>(w);
    w += units * p.runs * 4 * (kRun / kLeastBlock);
    p.done = reinterpret_cast<int *>(w);
    w += units * p.runs * 4 * (kRun / kLeastBlock);
    p.off = reinterpret_cast<int *>(w);
    // vectors as wide as every row allows
    const uint64_t m = (uint64_t)a.row_bytes | (uint64_t)a.page_bytes | reinterpret_cast<uintptr_t>(a.k_pages) |
                       reinterpret_cast<uintptr_t>(a.v_pages);
    const int wide = m % 16 == 0 ? 16 : m % 4 == 0 ? 4 : 2, vpr = (int)(a.row_bytes / wide);
    p.block = kRun;
    while (p.block > kLeastBlock && p.block * 2 * vpr > kInFlight * kMoveThreads) p.block /= 2;
    if (p.block * 2 * vpr > kInFlight * kMoveThreads) return cudaErrorNotSupported;
    p.blocks = p.runs * (kRun / p.block);
    const paged::DeviceInfo di = paged::device_info();
    if (di.sms <= 0) return cudaErrorInvalidDevice;
    // the smallest CTAs that hold a row of the table, then clusters of the largest
    const int threads = p.runs <= runs_held(256) ? 256 : p.runs <= runs_held(512) ? 512 : 1024;
    int C = 1;
    while (C < kMaxCluster && (long long)C * runs_held(threads) < p.runs) C *= 2;
    const size_t most = (size_t)(2 * di.sms * (1024 / threads) / C);
    const int groups = (int)(units < most ? units : most);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(groups * C);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const bool vec = a.page_size % 4 == 0 && a.mass_stride % 4 == 0 && reinterpret_cast<uintptr_t>(a.mass) % 16 == 0;
    auto select = threads == 256 ? (vec ? evict_select_kernel<true, 256> : evict_select_kernel<false, 256>)
                  : threads == 512 ? (vec ? evict_select_kernel<true, 512> : evict_select_kernel<false, 512>)
                                   : (vec ? evict_select_kernel<true, 1024> : evict_select_kernel<false, 1024>);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, select, p, C);
    if (e != cudaSuccess) return e;
    auto move = wide == 16 ? evict_move_kernel<uint4, false> : wide == 4 ? evict_move_kernel<uint32_t, false> : evict_move_kernel<uint16_t, false>;
    if (wide == 16 && kMoveThreads % (2 * vpr) == 0) move = evict_move_kernel<uint4, true>;
    return paged::launch_early(move, dim3(2 * di.sms), kMoveThreads, 0, s, p, vpr);
}

}  // namespace relattn
