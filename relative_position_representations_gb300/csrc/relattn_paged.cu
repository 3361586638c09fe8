// Paged attention, the parts that every path shares: parameters, workspace, the merge of split
// items; and the SIMT kernel, which covers every type, head dimension and page size.
#include <cstdint>
#include <cstring>
#include <mutex>

#include "relattn_paged.cuh"

namespace relattn {
namespace paged {

DeviceInfo device_info() {
    static DeviceInfo cache[64];
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DeviceInfo{};
    std::lock_guard<std::mutex> lk(mu);
    if (cache[dev].sms == 0) {
        cudaDeviceGetAttribute(&cache[dev].sms, cudaDevAttrMultiProcessorCount, dev);
        cudaDeviceGetAttribute(&cache[dev].smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    }
    return cache[dev];
}

cudaError_t opt_in_smem(const void *kern, const DeviceInfo &di) {
    // a fixed table: nothing here may throw through the C entry points (past its end a kernel is
    // only set again)
    static struct { int dev; const void *kern; } done[512];
    static int n = 0;
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < n; ++i)
        if (done[i].dev == dev && done[i].kern == kern) return cudaSuccess;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             di.smem_optin - (int)fa.sharedSizeBytes);
    if (e == cudaSuccess && n < 512) {
        done[n].dev = dev;
        done[n++].kern = kern;
    }
    return e;
}

bool wide_rows(const PagedArgs &a) {
    const long long es = a.bf16 ? 2 : 4;
    const uint64_t m = (uint64_t)(a.d * es) | (uint64_t)(a.q_stride * es) | (uint64_t)(a.page_stride * es) |
                       (uint64_t)(a.ths * es) | reinterpret_cast<uintptr_t>(a.q) |
                       reinterpret_cast<uintptr_t>(a.k_pages) | reinterpret_cast<uintptr_t>(a.v_pages) |
                       reinterpret_cast<uintptr_t>(a.aK) | reinterpret_cast<uintptr_t>(a.aV) |
                       reinterpret_cast<uintptr_t>(a.out);
    return m % 16 == 0;
}

void fill_params(const PagedArgs &a, Params *p) {
    std::memset(p, 0, sizeof(*p));
    p->q = a.q;
    p->k = a.k_pages;
    p->v = a.v_pages;
    p->aK = a.aK;
    p->aV = a.aV;
    p->q_stride = a.q_stride;
    p->page_stride = a.page_stride;
    p->bt_stride = a.bt_stride;
    p->ths = a.ths;
    p->bt = a.block_table;
    p->q_start = a.q_start;
    p->kv_len = a.kv_len;
    p->num_pages = a.num_pages;
    while ((1 << p->pshift) < a.page_size) ++p->pshift;
    const long long cap = (long long)a.max_pages << p->pshift;
    p->cap = cap > 0x7fffff00LL ? 0x7fffff00 : (int)cap;
    p->clip_k = a.clip_k;
    p->window = a.window >= p->cap ? 0 : a.window;   // a window over every key a table can hold
    p->sinks = a.sinks;
    p->scale_log2 = a.scale * kLog2e;
    p->B = a.B;
    p->tokens = a.tokens;
    p->H = a.H;
    p->Hkv = a.Hkv;
    p->g = a.H / a.Hkv;
    p->d = a.d;
    p->out = a.out;
    p->lse = a.lse;
    p->desc = static_cast<Desc *>(a.workspace);
    p->part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + desc_bytes());
    p->err = a.err;
    p->withhold = a.withhold;
    p->wait_limit = a.wait_limit > 0 ? a.wait_limit : 2000000000ll;
}

void fill_params(const PagedArgs &a, PartParams *p) {
    fill_params(a, static_cast<Params *>(p));
    p->step = a.flat ? 0 : 1;
    p->f32_out = a.f32_out;
    p->overlap = a.overlap;
    p->first_key = a.first_key;
    p->row_of = a.row_of;
    p->ctas = a.ctas;
    p->owner = a.owner;
    p->left = a.left;
}

// ------------------------------------------------------------------ merge
// CTA (c, y): the item that goes on behind CTA c's range. A row's pieces have maxima m_i, sums l_i
// and unnormalised outputs O_i: M = max m_i, z = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i, taken
// kUnroll pieces at a time under a running maximum, in the order of the keys. A thread holds V
// columns of a row and reads the row's statistics itself, so that all the loads of a row, mostly two
// pieces, are one latency; the records come out of the L2 that they have just gone to. Bound by that
// latency and the threads that an SM holds. 40 MB of records of four prompts (d = 128): 9 us with 8
// columns and 2 pieces a thread, 12.5 with 4 columns and 3 pieces, 23 with a warp per row that first
// joined the statistics. Few rows come from generated tokens, whose keys may lie in many pieces: 4
// columns and 8 pieces there.
constexpr int kMergeThreads = 256;

// lanes: threads of a row, as a power of two
template <typename T, int V, int kUnroll>
__global__ void __launch_bounds__(kMergeThreads, V == 8 ? 4 : 3)
    paged_merge_kernel(const __grid_constant__ Params p, int G, int lanes) {
    __shared__ short piece[kMaxGrid];
    __shared__ int n_s;
    grid_wait();
    grid_release();
    const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const Desc d = p.desc[c];
    if (!d.valid) return;
    const int D = p.d, rows = d.cnt * p.g, per = kMergeThreads >> lanes;   // rows of a CTA at a time
    const int r_first = (int)blockIdx.y * per;
    if (r_first >= rows) return;
    int n = d.n;
    if (n == 0) {   // short ranges: the first warp lists the CTAs that hold a piece, in order
        if (tid < 32) {
            auto tile_at = [&](long long y) -> int { return tiles_before(y, d.c0, d.wt, d.nt); };
            for (int e0 = c; e0 < G; e0 += 32) {
                const int e = e0 + lane;
                int t0 = d.nt, t1 = d.nt;
                if (e < G) {
                    const long long x0 = range_begin(d.total, e, G) - d.x, x1 = range_begin(d.total, e + 1, G) - d.x;
                    t0 = e == c ? 0 : tile_at(x0);
                    t1 = tile_at(x1);
                }
                const unsigned has = __ballot_sync(0xffffffffu, t1 > t0);
                if (t1 > t0) piece[n + __popc(has & ((1u << lane) - 1))] = (short)e;
                n += __popc(has);
                if (__any_sync(0xffffffffu, e >= G || t0 >= d.nt)) break;
            }
            if (lane == 0) n_s = n;
        }
        __syncthreads();
        n = n_s;
    }
    for (int r = r_first + (tid >> lanes); r < rows; r += (int)gridDim.y * per) {
        const int tok = r / p.g, hh = r - tok * p.g;
        T *out = static_cast<T *>(p.out) + ((long long)(d.row0 + tok) * p.H + d.kvh * p.g + hh) * D;
        for (int col = (tid & ((1 << lanes) - 1)) * V; col < D; col += V << lanes) {
            float m = -INFINITY, l = 0.f, acc[V] = {};
            for (int i0 = 0; i0 < n; i0 += kUnroll) {
                float mi[kUnroll], li[kUnroll], x[kUnroll][V];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int i = i0 + u;
                    mi[u] = -INFINITY;
                    li[u] = 0.f;
#pragma unroll
                    for (int e = 0; e < V; ++e) x[u][e] = 0.f;
                    if (i < n) {
                        const int e = d.n ? c + i : piece[i];
                        const float *q = record(p, e, e == c ? 1 : 0);
                        mi[u] = q[r];
                        li[u] = q[p.rec_rows + r];
                        const float *o = q + 2 * p.rec_rows + (long long)r * D + col;
                        if (V == 1) {
                            x[u][0] = o[0];
                        } else {
#pragma unroll
                            for (int e = 0; e + 3 < V; e += 4)
                                *reinterpret_cast<float4 *>(&x[u][e]) = *reinterpret_cast<const float4 *>(o + e);
                        }
                    }
                }
                float mn = m;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) mn = fmaxf(mn, mi[u]);
                const float mu = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m - mu);
                m = mn;
                l *= f;
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] *= f;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const float w = exp2f(mi[u] - mu);
                    l = fmaf(w, li[u], l);
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = fmaf(w, x[u][e], acc[e]);
                }
            }
            const float inv = l > 0.f ? 1.f / l : 0.f;
            if (p.lse && col == 0) p.lse[(long long)(d.row0 + tok) * p.H + d.kvh * p.g + hh] = row_lse(m, l);
            alignas(16) T z[V];
#pragma unroll
            for (int e = 0; e < V; ++e) z[e] = from_f<T>(acc[e] * inv);
            using W = std::conditional_t<V * sizeof(T) >= 16, uint4, std::conditional_t<V * sizeof(T) == 8, uint2, T>>;
#pragma unroll
            for (int e = 0; e < V * (int)sizeof(T) / (int)sizeof(W); ++e)
                reinterpret_cast<W *>(out + col)[e] = reinterpret_cast<const W *>(z)[e];
        }
    }
}

template <typename T>
cudaError_t launch_merge_t(const Params &p, int grid, cudaStream_t s) {
    // eight or four columns a thread where rows are as wide (those of the records are, at 16 bytes)
    const bool four = p.d % 4 == 0 && reinterpret_cast<uintptr_t>(p.out) % (4 * sizeof(T)) == 0;
    const bool eight = p.d % 8 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && p.rec_rows > 16;
    const int want = eight ? p.d / 8 : four ? p.d / 4 : p.d;
    int lanes = 0;
    while (lanes < 5 && (1 << lanes) < want) ++lanes;
    const int per = kMergeThreads >> lanes;
    const dim3 g(grid, (p.likely_rows + per - 1) / per);
    if (eight) return launch_early(paged_merge_kernel<T, 8, 2>, g, kMergeThreads, 0, s, p, grid, lanes);
    return four ? launch_early(paged_merge_kernel<T, 4, 8>, g, kMergeThreads, 0, s, p, grid, lanes)
                : launch_early(paged_merge_kernel<T, 1, 4>, g, kMergeThreads, 0, s, p, grid, lanes);
}

cudaError_t launch_merge(const Params &p, int grid, bool bf16, cudaStream_t s) {
    return bf16 ? launch_merge_t<__nv_bfloat16>(p, grid, s) : launch_merge_t<float>(p, grid, s);
}

cudaError_t launch_merge(const PartParams &p, int grid, bool bf16, cudaStream_t s) {
    if (!p.owner) return launch_merge(static_cast<const Params &>(p), grid, bf16, s);
    *p.left = PagedLeft{p.rec_rows, grid, p.ctas};
    return cudaSuccess;
}

// ------------------------------------------------------------------ SIMT kernel
// 32 query rows at a time (an item has T = max(1, 32 / g) tokens, so more only when g > 32: then
// the rows go in groups of 32 over the same keys), 8 warps of 4 rows. 32 keys at a time are
// staged in shared memory as fp32: lane = key for the scores (four rows share each load of a key),
// lane = N4 columns for P V. The next 32 keys are on their way into registers meanwhile, and the
// page numbers of the ones behind them. The edge tables go the same way: R = Q aK^T takes table
// rows for keys, beta aV takes beta for P. All sums and statistics fp32. Bound by
// shared memory (a lane's 16 products of scores take 5 loads of 16 bytes, its 32 of outputs 8: 1800
// cycles of its wavefronts for a run of 32 keys at d = 64, two CTAs to an SM) and by latency: a run
// takes a CTA on its own 2 us. Three chunks of 61 - 127 tokens over 100 - 700 keys (8 heads of 64, both
// terms, fp32) take 47 us, 6 TFLOP/s: 10 are a step's fixed cost, 5 the two terms, the rest one or two
// tiles (four runs each) of every CTA, cut into pieces, and their merge.
constexpr int kSimtThreads = 256;
constexpr int kSimtRows = 32;
constexpr int kSimtKeys = 32;

template <typename T>
__device__ __forceinline__ float4 load4(const T *row, int c, int d, bool vec) {
    if (vec) {
        if (sizeof(T) == 4) return *reinterpret_cast<const float4 *>(row + c);
        const uint2 w = *reinterpret_cast<const uint2 *>(row + c);
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                           __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    }
    float4 r;
    r.x = to_f(row[c]);
    r.y = c + 1 < d ? to_f(row[c + 1]) : 0.f;
    r.z = c + 2 < d ? to_f(row[c + 2]) : 0.f;
    r.w = c + 3 < d ? to_f(row[c + 3]) : 0.f;
    return r;
}

struct SimtLayout {
    int d4, ld, W, lw;                       // columns rounded to 4, row stride of K and V, table rows, their stride
    int q, k, v, pr, R, Bn, words;           // offsets in floats
    __host__ __device__ SimtLayout(int d, int clip_k) {
        d4 = (d + 3) & ~3;
        ld = d4 + 4;                         // 16-byte loads of 8 rows fall in distinct banks
        W = clip_k + 1;
        lw = (W + kSimtKeys - 1) / kSimtKeys * kSimtKeys + 1;
        int o = 0;
        q = o;  o += kSimtRows * d4;
        k = o;  o += kSimtKeys * ld;
        v = o;  o += kSimtKeys * ld;
        pr = o; o += kSimtRows * kSimtKeys;
        R = o;  o += kSimtRows * lw;
        Bn = o; o += kSimtRows * lw;
        words = o;
    }
};

// N4: 16-byte chunks of a row that a thread's share of 32 rows needs, ceil(d / 4 / 8). One kernel for plain calls and parts:
// the same time (chunk_f32 of the measured cases 47.3 us with and without what parts have).
template <typename T, int N4>
__global__ void __launch_bounds__(kSimtThreads, 2) paged_simt_kernel(const __grid_constant__ PartParams p, int vec) {
    extern __shared__ __align__(16) float smf[];
    __shared__ Range rg_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_wait();
    grid_release();
    if (warp == 0) {
        const Range r = find_range(p);
        if (lane == 0) rg_s = r;
    }
    __syncthreads();
    const Range rg = rg_s;
    const SimtLayout L(p.d, p.clip_k);
    const int d = p.d, d4 = L.d4, n4 = d4 / 4, k = p.clip_k;
    const bool ak = p.aK != nullptr, av = p.aV != nullptr;
    const int P = 1 << p.pshift;
    float *qs = smf + L.q, *Ks = smf + L.k, *Vs = smf + L.v, *ps = smf + L.pr, *Rs = smf + L.R, *Bs = smf + L.Bn;
    // a thread stages chunks my_c, my_c + 8, ... of row my_key
    const int my_key = tid >> 3, my_c = tid & 7;
    const bool wide = vec != 0;
    auto fetch = [&](float4 (&x)[N4], const T *row, bool on) {
#pragma unroll
        for (int i = 0; i < N4; ++i) {
            const int c = my_c + 8 * i;
            x[i] = on && c < n4 ? load4(row, 4 * c, d, wide) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    auto put = [&](float *dst, const float4 (&x)[N4]) {
#pragma unroll
        for (int i = 0; i < N4; ++i) {
            const int c = my_c + 8 * i;
            if (c < n4) *reinterpret_cast<float4 *>(dst + my_key * L.ld + 4 * c) = x[i];
        }
    };
    // products of this lane's staged row with the warp's four query rows
    auto scores = [&](float (&s)[4]) {
#pragma unroll
        for (int u = 0; u < 4; ++u) s[u] = 0.f;
#pragma unroll 2
        for (int c = 0; c < d4; c += 4) {
            const float4 kx = *reinterpret_cast<const float4 *>(Ks + lane * L.ld + c);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 qx = *reinterpret_cast<const float4 *>(qs + (warp * 4 + u) * d4 + c);
                s[u] = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, fmaf(qx.z, kx.z, fmaf(qx.w, kx.w, s[u]))));
            }
        }
    };
    // o += weights of the warp's rows (ps) times the staged rows, N4 columns of this lane
    auto outputs = [&](float (&o)[4][N4]) {
        if (N4 * lane >= d4) return;
#pragma unroll 1
        for (int kk = 0; kk < kSimtKeys; kk += 4) {
            float4 pr[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) pr[u] = *reinterpret_cast<const float4 *>(ps + (warp * 4 + u) * kSimtKeys + kk);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float vx[N4];
                const float *row = Vs + (kk + e) * L.ld + N4 * lane;
                if (N4 == 4) {
                    const float4 t = *reinterpret_cast<const float4 *>(row);
                    vx[0] = t.x; vx[N4 - 3] = t.y; vx[N4 - 2] = t.z; vx[N4 - 1] = t.w;
                } else if (N4 == 2) {
                    const float2 t = *reinterpret_cast<const float2 *>(row);
                    vx[0] = t.x; vx[N4 - 1] = t.y;
                } else {
                    vx[0] = row[0];
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float w = e == 0 ? pr[u].x : e == 1 ? pr[u].y : e == 2 ? pr[u].z : pr[u].w;
#pragma unroll
                    for (int i = 0; i < N4; ++i) o[u][i] = fmaf(w, vx[i], o[u][i]);
                }
            }
        }
    };
    Walk walk(p, rg);
    Segment g{};
    bool any = false;
    while (walk.next(p, g)) {
        any = true;
        if (warp == 0) write_owner(p, g);
        const int rows = g.it.cnt * p.g;
        const T *aK = static_cast<const T *>(p.aK) + (long long)g.kvh * p.ths;
        const T *aV = static_cast<const T *>(p.aV) + (long long)g.kvh * p.ths;
        const int *bt = p.bt + (long long)table_row(p, g.b) * p.bt_stride;
        const int first = p.window > 0 ? max(0, max(g.it.pos_lo, 0) - p.window + 1) : 0;
        const int pos_hi = g.it.pos_hi;
        // the piece's runs of 32 keys that some row sees: run q of tile t0 + q / 4
        const int runs = (g.t1 - g.t0) * (kTile / kSimtKeys);
        auto run_key = [&](int q) { return g.it.tile(g.t0 + (q >> 2)) * kTile + (q & 3) * kSimtKeys; };
        auto next_run = [&](int q) {
            for (; q < runs; ++q) {
                const int j0 = run_key(q);
                if (j0 <= pos_hi && (j0 + kSimtKeys > first || j0 < p.sinks)) break;
            }
            return q;
        };
        // page of this thread's key of run q (-1: not seen, -2: no such page)
        auto page_of = [&](int q) -> int {
            if (q >= runs) return -1;
            const int j = run_key(q) + my_key;
            if (!(j <= pos_hi && (j >= first || j < p.sinks))) return -1;
            const int pg = bt[j >> p.pshift];
            return (unsigned)pg < (unsigned)p.num_pages ? pg : -2;
        };
        auto row_of = [&](const void *base, int q, int pg) -> const T * {
            const long long at = (long long)pg * p.page_stride + ((long long)g.kvh * P + ((run_key(q) + my_key) & (P - 1))) * d;
            return static_cast<const T *>(base) + (pg >= 0 ? at : 0);
        };
        for (int r0 = 0; r0 < rows; r0 += kSimtRows) {
            const int nr = min(kSimtRows, rows - r0);
            // the first run's keys and the second one's pages, under way during the set-up
            int q0 = next_run(0), q1 = next_run(q0 + 1);
            int pg0 = page_of(q0), pg1 = page_of(q1);
            float4 kx[N4], vx[N4];
            if (pg0 == -2 && my_c == 0) report_page(p);
            fetch(kx, row_of(p.k, q0, pg0), pg0 >= 0);
            fetch(vx, row_of(p.v, q0, pg0), pg0 >= 0);
            __syncthreads();   // the previous rows are done with everything
            {
                const int tok = (r0 + my_key) / p.g, hh = (r0 + my_key) - tok * p.g;
                const T *q = static_cast<const T *>(p.q) + (long long)(g.s.q0 + g.it.i0 + tok) * p.q_stride +
                             (long long)(g.kvh * p.g + hh) * d;
                float4 x[N4];
                fetch(x, q, my_key < nr);
#pragma unroll
                for (int i = 0; i < N4; ++i)
                    if (my_c + 8 * i < n4) *reinterpret_cast<float4 *>(qs + my_key * d4 + 4 * (my_c + 8 * i)) = x[i];
            }
            if (av)
                for (int i = tid; i < kSimtRows * L.lw; i += kSimtThreads) Bs[i] = -INFINITY;
            if (ak) {   // R = Q aK^T in the log2 domain
                for (int w0 = 0; w0 < L.W; w0 += kSimtKeys) {
                    float4 x[N4];
                    fetch(x, aK + (long long)min(w0 + my_key, k) * d, w0 + my_key <= k);
                    put(Ks, x);
                    __syncthreads();
                    float s[4];
                    scores(s);
#pragma unroll
                    for (int u = 0; u < 4; ++u) Rs[(warp * 4 + u) * L.lw + w0 + lane] = s[u] * p.scale_log2;
                    __syncthreads();
                }
            }
            int pos[4];
            float m[4], l[4], far[4];
            float o[4][N4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int r = warp * 4 + u;
                pos[u] = r < nr ? g.it.pos_lo + (r0 + r) / p.g * p.step : -1;
                m[u] = -INFINITY;
                l[u] = far[u] = 0.f;
#pragma unroll
                for (int i = 0; i < N4; ++i) o[u][i] = 0.f;
            }
#pragma unroll 1
            while (q0 < runs) {
                const int j = run_key(q0) + lane;
                __syncthreads();   // the previous run's rows have been read
                put(Ks, kx);
                put(Vs, vx);
                q0 = q1;
                pg0 = pg1;
                if (pg0 == -2 && my_c == 0) report_page(p);
                fetch(kx, row_of(p.k, q0, pg0), pg0 >= 0);
                fetch(vx, row_of(p.v, q0, pg0), pg0 >= 0);
                q1 = next_run(q1 + 1);
                pg1 = page_of(q1);
                __syncthreads();
                float s[4], mx[4];
                scores(s);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int r = warp * 4 + u;
                    const int lab = max(j - pos[u], -k) + k;   // table row; > k for later keys
                    const bool seen = j <= pos[u] && (p.window == 0 || j > pos[u] - p.window || j < p.sinks);
                    s[u] = s[u] * p.scale_log2 + (ak && seen ? Rs[r * L.lw + lab] : 0.f);
                    s[u] = seen ? s[u] : -INFINITY;
                    if (av && seen && lab > 0) Bs[r * L.lw + lab] = s[u];
                    mx[u] = s[u];
                }
#pragma unroll
                for (int sh = 16; sh > 0; sh >>= 1)
#pragma unroll
                    for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], sh));
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float mn = fmaxf(m[u], mx[u]), mu = mn == -INFINITY ? 0.f : mn;
                    const float e = exp2f(s[u] - mu);
                    if (mn != m[u]) {   // uniform over the warp
                        const float al = exp2f(m[u] - mu);
                        m[u] = mn;
                        l[u] *= al;
                        far[u] *= al;
#pragma unroll
                        for (int i = 0; i < N4; ++i) o[u][i] *= al;
                    }
                    l[u] += e;          // per lane; summed at the end
                    if (av && j - pos[u] + k <= 0) far[u] += e;
                    ps[(warp * 4 + u) * kSimtKeys + lane] = e;
                }
                __syncwarp();
                outputs(o);
            }
            // ---- the rows' sums, the value term, the result
#pragma unroll
            for (int sh = 16; sh > 0; sh >>= 1)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    l[u] += __shfl_xor_sync(0xffffffffu, l[u], sh);
                    far[u] += __shfl_xor_sync(0xffffffffu, far[u], sh);
                }
            if (av) {
                for (int w0 = 0; w0 < L.W; w0 += kSimtKeys) {
                    float4 x[N4];
                    fetch(x, aV + (long long)min(w0 + my_key, k) * d, w0 + my_key <= k);
                    __syncthreads();
                    put(Vs, x);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int w = w0 + lane;
                        const float mu = m[u] == -INFINITY ? 0.f : m[u];
                        ps[(warp * 4 + u) * kSimtKeys + lane] =
                            w == 0 ? far[u] : w <= k ? exp2f(Bs[(warp * 4 + u) * L.lw + w] - mu) : 0.f;
                    }
                    __syncthreads();
                    outputs(o);
                }
            }
            const bool whole = g.whole();
            float *rec = whole ? nullptr : record(p, blockIdx.x, g.record());
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int r = warp * 4 + u, rr = r0 + r;
                if (r >= nr) continue;
                if (whole) {
                    const float inv = l[u] > 0.f ? 1.f / l[u] : 0.f;
                    const int tok = rr / p.g, hh = rr - tok * p.g;
                    const long long at = (long long)(g.s.q0 + g.it.i0 + tok) * p.H + g.kvh * p.g + hh;
                    T *out = static_cast<T *>(p.out) + at * d;
                    if (p.lse && lane == 0) p.lse[at] = row_lse(m[u], l[u]);
#pragma unroll
                    for (int i = 0; i < N4; ++i)
                        if (N4 * lane + i < d) {
                            if (p.f32_out) static_cast<float *>(p.out)[at * d + N4 * lane + i] = o[u][i] * inv;
                            else out[N4 * lane + i] = from_f<T>(o[u][i] * inv);
                        }
                } else {
                    if (lane == 0) {
                        rec[rr] = m[u];
                        rec[p.rec_rows + rr] = l[u];
                    }
#pragma unroll
                    for (int i = 0; i < N4; ++i)
                        if (N4 * lane + i < d) rec[2 * p.rec_rows + (long long)rr * d + N4 * lane + i] = o[u][i];
                }
            }
        }
    }
    if (tid == 0) write_desc(p, any ? &g : nullptr, rg.total);
}

template <typename T, int N4>
cudaError_t launch_simt_t(const PagedArgs &a, cudaStream_t s) {
    PartParams p;
    fill_params(a, &p);
    p.T = p.g >= kSimtRows ? 1 : kSimtRows / p.g;
    p.T1 = p.T;
    p.c0 = 1;
    p.wt = p.wt2 = 2;
    p.rec_rows = kRecordRows;
    p.long_line = line_is_long(p);
    p.likely_rows = likely_rows(a, p.T, p.g);
    const SimtLayout L(a.d, a.clip_k);
    const int smem = L.words * (int)sizeof(float);
    // 16-byte (fp32) or 8-byte (bf16) loads where every row starts on such a boundary
    const long long es = sizeof(T);
    const uint64_t al = (uint64_t)(a.d * es) | (uint64_t)(a.q_stride * es) | (uint64_t)(a.page_stride * es) |
                        (uint64_t)(a.ths * es) | reinterpret_cast<uintptr_t>(a.q) |
                        reinterpret_cast<uintptr_t>(a.k_pages) | reinterpret_cast<uintptr_t>(a.v_pages) |
                        reinterpret_cast<uintptr_t>(a.aK) | reinterpret_cast<uintptr_t>(a.aV);
    const int vec = al % (4 * es) == 0;
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return cudaErrorInvalidDevice;
    cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(paged_simt_kernel<T, N4>), di);
    if (e != cudaSuccess) return e;
    const int grid = 2 * di.sms < kMaxGrid ? 2 * di.sms : kMaxGrid;
    e = launch_early(paged_simt_kernel<T, N4>, dim3(grid), kSimtThreads, smem, s, p, vec);
    if (e != cudaSuccess) return e;
    return launch_merge(p, grid, sizeof(T) == 2, s);
}

template <typename T>
cudaError_t launch_simt_d(const PagedArgs &a, cudaStream_t s) {
    return a.d <= 32 ? launch_simt_t<T, 1>(a, s) : a.d <= 64 ? launch_simt_t<T, 2>(a, s) : launch_simt_t<T, 4>(a, s);
}

}  // namespace paged

unsigned long long paged_workspace_bytes(int d) {
    return (unsigned long long)paged::desc_bytes() +
           (unsigned long long)paged::kMaxGrid * 2 * paged::kRecordRows * (d + 2) * sizeof(float);
}

cudaError_t launch_paged(const PagedArgs &a, cudaStream_t s) {
    if (paged_decode_covers(a)) {
        const cudaError_t e = launch_paged_decode(a, s);
        if (e != cudaErrorNotSupported) return e;
    }
    if (paged_tc_covers(a)) {
        const cudaError_t e = launch_paged_tc(a, s);
        if (e != cudaErrorNotSupported) return e;
    }
    PagedArgs all = a;   // the whole grid, in its turn
    all.ctas = nullptr;
    all.overlap = 0;
    return launch_paged_simt(all, s);
}

cudaError_t launch_paged_simt(const PagedArgs &a, cudaStream_t s) {
    return a.bf16 ? paged::launch_simt_d<__nv_bfloat16>(a, s) : paged::launch_simt_d<float>(a, s);
}

}  // namespace relattn
