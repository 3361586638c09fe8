// Paged attention, the parts that every path shares: parameters, workspace, the merge of split
// items; and the SIMT kernel, which covers every type, head dimension and page size.
#include <cstdint>
#include <cstring>
#include <mutex>
#include <set>
#include <utility>

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
    static std::set<std::pair<int, const void *>> done;
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    if (done.count({dev, kern})) return cudaSuccess;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             di.smem_optin - (int)fa.sharedSizeBytes);
    if (e == cudaSuccess) done.insert({dev, kern});
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
    p->max_pages = a.max_pages;
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
    p->desc = static_cast<Desc *>(a.workspace);
    p->part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + desc_bytes());
    p->err = a.err;
    p->wait_limit = a.wait_limit > 0 ? a.wait_limit : 2000000000ll;
}

// ------------------------------------------------------------------ merge
// CTA (c, y): the item that goes on behind CTA c's range. A row's pieces have maxima m_i, sums l_i
// and unnormalised outputs O_i: M = max m_i, z = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i. One warp
// takes a row and NV groups of 32 columns: the statistics with one piece per lane, then the
// outputs with kUnroll pieces' loads in flight (a row is a chain of dependent loads, so the work is
// spread over many warps: for the few rows of generated tokens, NV = 1, else whole rows).
constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;

template <typename T, int NV>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const __grid_constant__ Params p, int G) {
    constexpr int kUnroll = 16 / NV;
    __shared__ short piece[kMaxGrid];
    __shared__ int n_s;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Desc d = p.desc[c];
    if (!d.valid) return;
    const int D = p.d, groups = NV == 1 ? (D + 31) / 32 : 1, units = d.cnt * p.g * groups;
    if ((int)blockIdx.y * kMergeWarps >= units) return;
    auto tile_at = [&](long long y) -> int { return tiles_before(y, d.c0, d.wt, d.nt); };
    // the CTAs that hold a piece, in order (the first warp lists them)
    if (warp == 0) {
        int n = 0;
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
    const int n = n_s;
    auto rec = [&](int i) -> const float * {
        return record(p, piece[i], piece[i] == c ? 1 : 0);
    };
    for (int u0 = blockIdx.y * kMergeWarps + warp; u0 < units; u0 += (int)gridDim.y * kMergeWarps) {
        const int r = u0 / groups, col = (u0 - r * groups) * 32 + lane;
        float m = -INFINITY;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, rec(i)[r]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float mu = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        for (int i = lane; i < n; i += 32) l += rec(i)[p.rec_rows + r] * exp2f(rec(i)[r] - mu);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        float acc[NV] = {};
        for (int i0 = 0; i0 < n; i0 += kUnroll) {
            float w[kUnroll], x[kUnroll][NV];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const bool on = i0 + u < n;
                const float *q = rec(on ? i0 + u : i0);
                w[u] = on ? exp2f(q[r] - mu) : 0.f;
                const float *o = q + 2 * p.rec_rows + (long long)r * D;
#pragma unroll
                for (int e = 0; e < NV; ++e) x[u][e] = col + 32 * e < D ? o[col + 32 * e] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                for (int e = 0; e < NV; ++e) acc[e] = fmaf(w[u], x[u][e], acc[e]);
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int tok = r / p.g, hh = r - tok * p.g;
        T *o = static_cast<T *>(p.out) + ((long long)(d.row0 + tok) * p.H + d.kvh * p.g + hh) * D;
#pragma unroll
        for (int e = 0; e < NV; ++e)
            if (col + 32 * e < D) o[col + 32 * e] = from_f<T>(acc[e] * inv);
    }
}

cudaError_t launch_merge(const Params &p, int grid, bool bf16, cudaStream_t s) {
    // a warp per row and 32 columns up to 16 rows, else a warp per two rows
    const bool few = p.rec_rows <= 16;
    const int warps = few ? p.rec_rows * ((p.d + 31) / 32) : p.rec_rows / 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid, (warps + kMergeWarps - 1) / kMergeWarps);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (!bf16) return cudaLaunchKernelEx(&cfg, paged_merge_kernel<float, 4>, p, grid);
    return few ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<__nv_bfloat16, 1>, p, grid)
               : cudaLaunchKernelEx(&cfg, paged_merge_kernel<__nv_bfloat16, 4>, p, grid);
}

// ------------------------------------------------------------------ SIMT kernel
// 32 query rows at a time (an item has T = max(1, 32 / g) tokens, so more only when g > 32: then
// the rows go in groups of 32 over the same keys), 8 warps of 4 rows. 32 keys at a time are
// staged in shared memory as fp32; lane = key for the scores (four rows share each load of a
// key), lane = four columns for P V. All sums and statistics fp32.
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
        lw = W | 1;
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

template <typename T>
__global__ void __launch_bounds__(kSimtThreads) paged_simt_kernel(const __grid_constant__ Params p, int vec) {
    extern __shared__ __align__(16) float smf[];
    __shared__ Range rg_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
    Walk walk(p, rg);
    Segment g{};
    bool any = false;
    while (walk.next(p, g)) {
        any = true;
        const int rows = g.it.cnt * p.g;
        const T *aK = static_cast<const T *>(p.aK) + (long long)g.kvh * p.ths;
        const T *aV = static_cast<const T *>(p.aV) + (long long)g.kvh * p.ths;
        const int *bt = p.bt + (long long)g.b * p.bt_stride;
        for (int r0 = 0; r0 < rows; r0 += kSimtRows) {
            const int nr = min(kSimtRows, rows - r0);
            __syncthreads();   // the previous rows are done with everything
            for (int i = tid; i < kSimtRows * n4; i += kSimtThreads) {
                const int r = i / n4, c = (i - r * n4) * 4;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < nr) {
                    const int tok = (r0 + r) / p.g, hh = (r0 + r) - tok * p.g;
                    x = load4(static_cast<const T *>(p.q) + (long long)(g.s.q0 + g.it.i0 + tok) * p.q_stride +
                                  (long long)(g.kvh * p.g + hh) * d, c, d, vec != 0);
                }
                *reinterpret_cast<float4 *>(qs + r * d4 + c) = x;
            }
            __syncthreads();
            if (ak) {   // R = Q aK^T in the log2 domain, rows 0 .. k
                for (int i = tid; i < nr * L.W; i += kSimtThreads) {
                    const int r = i / L.W, w = i - r * L.W;
                    float acc = 0.f;
                    for (int c = 0; c < d; ++c) acc = fmaf(qs[r * d4 + c], to_f(aK[(long long)w * d + c]), acc);
                    Rs[r * L.lw + w] = acc * p.scale_log2;
                }
            }
            if (av)
                for (int i = tid; i < kSimtRows * L.lw; i += kSimtThreads) Bs[i] = -INFINITY;
            __syncthreads();
            int pos[4];
            bool live[4];
            float m[4], l[4], far[4];
            float4 o[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int r = warp * 4 + u;
                live[u] = r < nr;
                pos[u] = g.it.pos_lo + (live[u] ? (r0 + r) / p.g : 0);
                m[u] = -INFINITY;
                l[u] = far[u] = 0.f;
                o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            const int first = p.window > 0 ? max(0, max(g.it.pos_lo, 0) - p.window + 1) : 0;
            for (int t = g.t0; t < g.t1; ++t) {
                for (int j0 = g.it.tile(t) * kTile; j0 < g.it.tile(t) * kTile + kTile; j0 += kSimtKeys) {
                    if (j0 > g.it.pos_hi || (j0 + kSimtKeys <= first && j0 >= p.sinks)) continue;  // seen by no row
                    __syncthreads();
                    for (int i = tid; i < kSimtKeys * n4; i += kSimtThreads) {
                        const int kk = i / n4, c = (i - kk * n4) * 4, j = j0 + kk;
                        float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
                        if (j <= g.it.pos_hi && (j >= first || j < p.sinks)) {
                            const int pg = bt[j >> p.pshift];
                            if ((unsigned)pg < (unsigned)p.num_pages) {
                                const long long off = (long long)pg * p.page_stride +
                                                      ((long long)g.kvh * P + (j & (P - 1))) * d;
                                kx = load4(static_cast<const T *>(p.k) + off, c, d, vec != 0);
                                vx = load4(static_cast<const T *>(p.v) + off, c, d, vec != 0);
                            } else if (c == 0) {
                                report_page(p);
                            }
                        }
                        *reinterpret_cast<float4 *>(Ks + kk * L.ld + c) = kx;
                        *reinterpret_cast<float4 *>(Vs + kk * L.ld + c) = vx;
                    }
                    __syncthreads();
                    float s[4] = {0.f, 0.f, 0.f, 0.f};
                    for (int c = 0; c < d4; c += 4) {
                        const float4 kx = *reinterpret_cast<const float4 *>(Ks + lane * L.ld + c);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float4 qx = *reinterpret_cast<const float4 *>(qs + (warp * 4 + u) * d4 + c);
                            s[u] = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, fmaf(qx.z, kx.z, fmaf(qx.w, kx.w, s[u]))));
                        }
                    }
                    const int j = j0 + lane;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int r = warp * 4 + u;
                        const int lab = max(j - pos[u], -k) + k;   // table row; > k for later keys
                        const bool seen = live[u] && j <= pos[u] &&
                                          (p.window == 0 || j > pos[u] - p.window || j < p.sinks);
                        float x = s[u] * p.scale_log2;
                        if (ak && seen) x += Rs[r * L.lw + lab];
                        x = seen ? x : -INFINITY;
                        float mx = x;
#pragma unroll
                        for (int sh = 16; sh > 0; sh >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
                        const float mn = fmaxf(m[u], mx);
                        const float mu = mn == -INFINITY ? 0.f : mn;
                        const float al = exp2f(m[u] - mu);
                        const float e = exp2f(x - mu);
                        m[u] = mn;
                        l[u] = l[u] * al + e;      // per lane; summed at the end
                        if (av) {
                            far[u] *= al;
                            if (seen && lab > 0) Bs[r * L.lw + lab] = x;
                            else far[u] += e;
                        }
                        o[u].x *= al;
                        o[u].y *= al;
                        o[u].z *= al;
                        o[u].w *= al;
                        ps[r * kSimtKeys + lane] = e;
                    }
                    __syncwarp();
                    if (4 * lane < d4) {
#pragma unroll 2
                        for (int kk = 0; kk < kSimtKeys; kk += 4) {
                            float4 pr[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                pr[u] = *reinterpret_cast<const float4 *>(ps + (warp * 4 + u) * kSimtKeys + kk);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float4 vx = *reinterpret_cast<const float4 *>(Vs + (kk + e) * L.ld + 4 * lane);
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    const float w = e == 0 ? pr[u].x : e == 1 ? pr[u].y : e == 2 ? pr[u].z : pr[u].w;
                                    o[u].x = fmaf(w, vx.x, o[u].x);
                                    o[u].y = fmaf(w, vx.y, o[u].y);
                                    o[u].z = fmaf(w, vx.z, o[u].z);
                                    o[u].w = fmaf(w, vx.w, o[u].w);
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
            }
            // ---- the rows' sums, the value term, the result
            const bool whole = g.whole();
            float *rec = whole ? nullptr : record(p, blockIdx.x, g.record());
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int r = warp * 4 + u;
                if (!live[u]) continue;   // the whole warp's row
                float ls = l[u], fs = far[u];
#pragma unroll
                for (int sh = 16; sh > 0; sh >>= 1) {
                    ls += __shfl_xor_sync(0xffffffffu, ls, sh);
                    fs += __shfl_xor_sync(0xffffffffu, fs, sh);
                }
                if (av) {
                    const float mu = m[u] == -INFINITY ? 0.f : m[u];
                    for (int w = 0; w < L.W; ++w) {
                        const float pw = w == 0 ? fs : exp2f(Bs[r * L.lw + w] - mu);
                        if (pw == 0.f || 4 * lane >= d4) continue;
                        const float4 x = load4(aV + (long long)w * d, 4 * lane, d, vec != 0);
                        o[u].x = fmaf(pw, x.x, o[u].x);
                        o[u].y = fmaf(pw, x.y, o[u].y);
                        o[u].z = fmaf(pw, x.z, o[u].z);
                        o[u].w = fmaf(pw, x.w, o[u].w);
                    }
                }
                const float os[4] = {o[u].x, o[u].y, o[u].z, o[u].w};
                const int rr = r0 + r;
                if (whole) {
                    const float inv = ls > 0.f ? 1.f / ls : 0.f;
                    const int tok = rr / p.g, hh = rr - tok * p.g;
                    T *out = static_cast<T *>(p.out) +
                             ((long long)(g.s.q0 + g.it.i0 + tok) * p.H + g.kvh * p.g + hh) * d;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (4 * lane + e < d) out[4 * lane + e] = from_f<T>(os[e] * inv);
                } else {
                    if (lane == 0) {
                        rec[rr] = m[u];
                        rec[p.rec_rows + rr] = ls;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (4 * lane + e < d) rec[2 * p.rec_rows + (long long)rr * d + 4 * lane + e] = os[e];
                }
            }
        }
    }
    if (tid == 0) write_desc(p, any ? &g : nullptr, rg.total);
}

template <typename T>
cudaError_t launch_simt_t(const PagedArgs &a, cudaStream_t s) {
    Params p;
    fill_params(a, &p);
    p.T = p.g >= kSimtRows ? 1 : kSimtRows / p.g;
    p.T1 = p.T;
    p.c0 = 1;
    p.wt = p.wt2 = 2;
    p.rec_rows = kRecordRows;
    p.long_line = line_is_long(p);
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
    cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(paged_simt_kernel<T>), di);
    if (e != cudaSuccess) return e;
    const int grid = 2 * di.sms < kMaxGrid ? 2 * di.sms : kMaxGrid;
    paged_simt_kernel<T><<<grid, kSimtThreads, smem, s>>>(p, vec);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_merge(p, grid, sizeof(T) == 2, s);
}

}  // namespace paged

unsigned long long paged_workspace_bytes(int d) {
    return (unsigned long long)paged::desc_bytes() +
           (unsigned long long)paged::kMaxGrid * 2 * paged::kRecordRows * (d + 2) * sizeof(float);
}

cudaError_t launch_paged_simt(const PagedArgs &a, cudaStream_t s) {
    return a.bf16 ? paged::launch_simt_t<__nv_bfloat16>(a, s) : paged::launch_simt_t<float>(a, s);
}

}  // namespace relattn
