// Attention of requests that share prefixes: groups of requests whose first keys lie in the same pages.
//
// In two parts, whose softmaxes are joined: over the shared keys, where the rows of all requests of
// a group go through the same products (so each shared key is read once for a group and meets full tiles of
// rows), and over each request's own keys. With L the shared part's length, chosen on a tile's border and
// so that every row of the group stands at least clip_k behind its last key, all of its keys have
// the first table row in common:
//   e_ij = scale q_i . (k_j + aK_0),  sum_j p_ij (v_j + aV_0) = sum_j p_ij v_j + aV_0 sum_j p_ij,
// so the part needs neither positions nor masks nor tables: it is plain attention, and the two constants
// enter where the parts are joined. Both parts run on the kernels of relattn_paged_fwd, which leave
// fp32 outputs and log-sum-exps: the first with a group for a request and all of its tokens at the
// shared part's end, the second from the shared part's end on. They run side by side: the first is bound by
// its chain of products and softmax, the second by HBM, and neither needs the other, so a kernel in front
// measures their work and gives each as many SMs that both end together; the second's CTAs come up where
// the first's have nothing to do. (One after the other: 64 requests behind 8192 shared keys, 16 / 4 heads of 128, 68 us in
// place of 50; 256 behind 32768, 16 / 2 heads, 115 and 113.)
// What bounds it: the shared part the chain of the kernel for chunks (6000 cycles a tile of 256 rows where the tensor
// cores work 2048), the own keys the pieces (2 us each beside their tiles), both the fixed cost of four launches in a
// row: 15 us in a graph, 23 where the host makes the call.
#include <cstdint>
#include <cstring>

#include "relattn_paged.cuh"

namespace relattn {
namespace paged {
namespace {

constexpr int kSplitThreads = 1024;
constexpr int kSplitWarps = kSplitThreads / 32;
constexpr int kJoinThreads = 256;

// What the parts take, in SM cycles: an item, a tile of keys of an item of at most one query tile (of the
// first part; the only kind of the second), one of two; and what a CTA takes beside its work.
struct Costs {
    float item, tile, tile2, fixed;
};

struct SplitParams {
    Params p;                         // q_start, kv_len, B, tokens, cap, clip_k
    const int *group_start, *prefix_len;
    int groups, most;                 // entries of the lists below
    int *first_key;                   // [tokens]: where the own keys of the token's request begin
    int *q_start, *kv_len, *row_of;   // [most + 1], [most], [most]: the shared parts as requests
    int *ctas;                        // [2]: CTAs of the two parts, which run side by side
    int sms, own_per_sm;              // SMs; CTAs of the second part that an SM holds
    int tile_tokens;                  // tokens of a query tile of the first part
    int own_tokens;                   // tokens of an item of the second part
    Costs shared, own;
};

// Which groups share what. Entry 2 i is the i-th group that shares keys, entry 2 i + 1 the rows up to the
// next one (without keys). A warp per group.
__global__ void __launch_bounds__(kSplitThreads) shared_split_kernel(const __grid_constant__ SplitParams sp) {
    __shared__ int on_s[kSplitWarps], end_s;
    __shared__ float work_s[2][kSplitWarps];
    const Params &p = sp.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_wait();
    grid_release();
    for (int t = tid; t < p.tokens; t += kSplitThreads) sp.first_key[t] = 0;
    if (tid == 0) end_s = 0;
    int done = 0;
    float work = 0.f;
    for (int g0 = 0; g0 < sp.groups; g0 += kSplitWarps) {
        const int g = g0 + warp;
        int keys = 0, q0 = 0, q1 = 0, row = 0;
        if (g < sp.groups) {
            const int b0 = min(max(sp.group_start[g], 0), p.B), b1 = min(max(sp.group_start[g + 1], b0), p.B);
            const int most = sp.prefix_len[g];
            int least = 0x7fffffff, busy = 0, first = p.B;
            for (int b = b0 + lane; b < b1; b += 32) {
                const Seq s = load_seq(p, b);
                if (s.n == 0) continue;
                least = min(least, s.pos0);
                first = min(first, b);
                ++busy;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
                first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
                busy += __shfl_xor_sync(0xffffffffu, busy, o);
            }
            if (busy > 1) {
                keys = max(min(most, least - p.clip_k + 1), 0) / kTile * kTile;
                q0 = min(max(p.q_start[b0], 0), p.tokens);
                q1 = min(max(p.q_start[b1], q0), p.tokens);
                row = first;
            }
        }
        const bool on = keys > 0 && q1 > q0;
        if (lane == 0) on_s[warp] = on;
        __syncthreads();
        const unsigned all = __ballot_sync(0xffffffffu, on_s[lane] != 0);
        const int i = done + __popc(all & ((1u << warp) - 1));
        if (on && 2 * i + 1 < sp.most + 1) {
            const int n = q1 - q0, pairs = n / (2 * sp.tile_tokens), rest = n - pairs * 2 * sp.tile_tokens;
            if (lane == 0)
                work += (float)p.Hkv * (pairs * (sp.shared.item + sp.shared.tile2 * (keys / kTile)) +
                                        (rest ? sp.shared.item + (rest > sp.tile_tokens ? sp.shared.tile2 : sp.shared.tile) * (keys / kTile) : 0.f));
            for (int t = q0 + lane; t < q1; t += 32) sp.first_key[t] = keys;
            if (lane == 0) {
                sp.q_start[2 * i] = q0;
                sp.q_start[2 * i + 1] = q1;
                sp.kv_len[2 * i] = keys;
                sp.row_of[2 * i] = row;
                if (2 * i + 1 < sp.most) {
                    sp.kv_len[2 * i + 1] = 0;
                    sp.row_of[2 * i + 1] = 0;
                }
                atomicMax(&end_s, q1);
            }
        }
        done += __popc(all);
        __syncthreads();
    }
    for (int i = 2 * done + tid; i <= sp.most; i += kSplitThreads) {
        sp.q_start[i] = end_s;
        if (i < sp.most) sp.kv_len[i] = sp.row_of[i] = 0;
    }
    // the own keys' work, and the SMs of either part: as many that both end together
    float own = 0.f;
    for (int b = tid; b < p.B; b += kSplitThreads) {
        const Seq s = load_seq(p, b);
        const int last = s.pos0 + s.n - 1;
        if (s.n == 0 || last < 0) continue;
        const int tiles = max(last / kTile + 1 - sp.first_key[s.q0] / kTile, 0);
        own += (float)p.Hkv * ((s.n + sp.own_tokens - 1) / sp.own_tokens) * (sp.own.item + sp.own.tile * tiles);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        own += __shfl_xor_sync(0xffffffffu, own, o);
        work += __shfl_xor_sync(0xffffffffu, work, o);
    }
    if (lane == 0) {
        work_s[0][warp] = work;
        work_s[1][warp] = own;
    }
    __syncthreads();
    if (warp == 0) {
        work = work_s[0][lane];
        own = work_s[1][lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            work += __shfl_xor_sync(0xffffffffu, work, o);
            own += __shfl_xor_sync(0xffffffffu, own, o);
        }
        float best = INFINITY;
        int at = 1;
        for (int n = 1 + lane; n < sp.sms; n += 32) {
            const float t = fmaxf(work / n + sp.shared.fixed, own / (sp.sms - n) + sp.own.fixed);
            if (t < best) {
                best = t;
                at = n;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float t = __shfl_xor_sync(0xffffffffu, best, o);
            const int n = __shfl_xor_sync(0xffffffffu, at, o);
            if (t < best || (t == best && n < at)) {
                best = t;
                at = n;
            }
        }
        if (work == 0.f) at = 1;
        if (lane == 0) {   // behind everything that this block has written (grid_start)
            __threadfence();
            const int n[2] = {at, max(sp.sms - at, 1) * sp.own_per_sm};
#pragma unroll
            for (int i = 0; i < 2; ++i)
                asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(sp.ctas + i), "r"(n[i]) : "memory");
        }
    }
}

// What a part has left: rows of whole items in o (normalised, with their log-sum-exps in lse), the others in
// the records of the CTAs that hold a piece.
struct Part {
    const float *o, *lse, *rec;
    const int *owner, *ctas;
    const Desc *desc;
    int rec_rows, launched;
};

struct JoinParams {
    const void *q, *aK, *aV;
    long long q_stride, ths;
    int tokens, H, Hkv, g, d;
    float scale_log2;
    const int *first_key, *q_start;
    int B;
    Part part[2];                     // shared keys, own keys
    void *out;
    float *lse;
};

// A warp per row, N columns from lane + 32 i: joins the pieces of either part in the order of their keys, under a
// running maximum: z = sum f_i (acc_i + l_i aV_0) / sum f_i l_i, f_i = 2^(m_i - M), aV_0 and the constant of aK_0 in m_i for
// the shared keys alone. Both parts go through one loop: the code runs once and cold, and its fetching took longer
// than its loads when each part had a copy (17 us a step in place of 9).
template <typename T, int N>
__global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(const __grid_constant__ JoinParams p) {
    constexpr int kBatch = 4;                // pieces on their way together
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
    grid_wait();
    grid_release();
    if (row >= (long long)p.tokens * p.H) return;
    const int t = (int)(row / p.H), h = (int)(row - (long long)t * p.H), kvh = h / p.g;
    // where the row's parts are (everything that depends on nothing is on its way at once)
    const int from = p.q_start[0], end = p.q_start[p.B], shared = p.first_key[t];
    const int c0 = p.part[0].owner[(long long)t * p.Hkv + kvh], c1 = p.part[1].owner[(long long)t * p.Hkv + kvh];
    float r = 0.f, v0[N];
    {
        const long long table = (long long)kvh * p.ths;
        const T *q = static_cast<const T *>(p.q) + (long long)t * p.q_stride + (long long)h * p.d;
        const T *k0 = static_cast<const T *>(p.aK) + table, *av = static_cast<const T *>(p.aV) + table;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = lane + 32 * i;
            v0[i] = p.aV && c < p.d ? to_f(av[c]) : 0.f;
            if (p.aK && c < p.d) r = fmaf(to_f(q[c]), to_f(k0[c]), r);
        }
    }
    if (t < from || t >= end) return;        // no request's
    if (p.aK) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    }
    float m = -INFINITY, l = 0.f, acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
#pragma unroll 1
    for (int x = shared > 0 ? 0 : 1; x < 2; ++x) {
        const Part &a = p.part[x];
        const int c = min(x ? c1 : c0, a.launched - 1);
        const float add = x ? 0.f : r * p.scale_log2;
        Desc d{};
        int rr = 0, left = 1, e = c, G = a.launched;
        if (c >= 0) {
            d = a.desc[c];
            if (a.ctas) G = min(max(*a.ctas, 1), G);
            rr = (t - d.row0) * p.g + (h - kvh * p.g);
            left = d.n;
            // (offsets that do not ascend may leave a token without an owner: what follows stays within the arrays)
            if (!d.valid || rr < 0 || rr >= min(d.cnt * p.g, a.rec_rows)) continue;
        }
        const bool listed = c < 0 || d.n > 0;   // the pieces are counted
        bool more = true;
        while (more) {
            float mi[kBatch], li[kBatch], y[kBatch][N], mn = m;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                mi[u] = -INFINITY;
                li[u] = 0.f;
#pragma unroll
                for (int i = 0; i < N; ++i) y[u][i] = 0.f;
                if (!more) continue;
                if (listed) more = left-- > 0 && e < a.launched;   // in the CTAs c .. c + n - 1
                else {                                             // short ranges: those whose range begins another tile
                    while (e < G) {
                        const int t0 = e == c ? 0 : tiles_before(range_begin(d.total, e, G) - d.x, d.c0, d.wt, d.nt);
                        const int t1 = tiles_before(range_begin(d.total, e + 1, G) - d.x, d.c0, d.wt, d.nt);
                        if (t0 >= d.nt) e = G;
                        else if (t1 > t0) break;
                        else ++e;
                    }
                    more = e < G;
                }
                if (!more) continue;
                const float *o = a.o + row * p.d;
                if (c < 0) {                     // all of it
                    mi[u] = a.lse[row];
                    li[u] = mi[u] == -INFINITY ? 0.f : 1.f;
                    mi[u] *= kLog2e;
                } else {
                    const float *rec = a.rec + ((long long)e * 2 + (e == c ? 1 : 0)) * a.rec_rows * (p.d + 2);
                    mi[u] = rec[rr];
                    li[u] = rec[a.rec_rows + rr];
                    o = rec + 2 * a.rec_rows + (long long)rr * p.d;
                }
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (lane + 32 * i < p.d) y[u][i] = o[lane + 32 * i];
                ++e;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                mi[u] += add;
                mn = fmaxf(mn, mi[u]);
            }
            const float mu = mn == -INFINITY ? 0.f : mn, f = exp2f(m - mu);
            m = mn;
            l *= f;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] *= f;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const float w = exp2f(mi[u] - mu);
                l = fmaf(w, li[u], l);
                const float lv = x ? 0.f : li[u];
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = fmaf(w, fmaf(lv, v0[i], y[u][i]), acc[i]);
            }
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (lane + 32 * i < p.d) static_cast<T *>(p.out)[row * p.d + lane + 32 * i] = from_f<T>(acc[i] * inv);
    if (p.lse && lane == 0) p.lse[row] = row_lse(m == -INFINITY ? 0.f : m, l);
}

template <typename T>
cudaError_t launch_join(const JoinParams &j, cudaStream_t s) {
    const long long rows = (long long)j.tokens * j.H;
    const dim3 grid((unsigned)((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
    if (j.d <= 32) return launch_early(shared_join_kernel<T, 1>, grid, kJoinThreads, 0, s, j);
    if (j.d <= 64) return launch_early(shared_join_kernel<T, 2>, grid, kJoinThreads, 0, s, j);
    return launch_early(shared_join_kernel<T, 4>, grid, kJoinThreads, 0, s, j);
}

// [d > 64] as measured: tiles of the kernel for chunks with one and two query tiles; tiles of the one for generated
// tokens, which HBM bounds
constexpr Costs kChunkCosts[2] = {{6400.f, 2900.f, 3900.f, 6400.f}, {8600.f, 4500.f, 6000.f, 8600.f}};
constexpr Costs kTokenCosts[2] = {{1500.f, 1500.f, 1500.f, 3000.f}, {3000.f, 3000.f, 3000.f, 6000.f}};

size_t round16(size_t x) { return (x + 15) & ~(size_t)15; }

}  // namespace
}  // namespace paged

// workspace: that of either part, their outputs, log-sum-exps and owners, first keys, the shared parts' list, CTAs
unsigned long long paged_shared_workspace_bytes(int tokens, int H, int d) {
    const size_t rows = (size_t)tokens * H;
    return 2 * paged_workspace_bytes(d) + 16 + 2 * paged::round16(rows * d * 4) + 4 * paged::round16(rows * 4) +
           4 * paged::round16(((size_t)tokens + 2) * 4);
}

cudaError_t launch_paged_shared(const PagedSharedArgs &sa, cudaStream_t s) {
    using namespace paged;
    const PagedArgs &a = sa.a;
    // Under a window a token sees little of a prefix; one token shares with nobody. The requests' own rows of
    // the table hold the prefix too.
    if (a.window > 0 || sa.groups == 0 || a.tokens < 2) return launch_paged(a, s);
    // Requests that fill a tile of 128 rows by themselves share their reads in the L2 as it is, and two parts cost more
    // than they save (32 requests behind 8192 keys, 16 / 4 heads of 128: 16 new tokens 75 us here, 103 without; 24 tokens
    // 95 and 105; 32 tokens, 128 rows, 115 and 106). The host knows the average alone: one long chunk among generated tokens
    // turns the sharing off for all of them.
    if ((long long)a.tokens * (a.H / a.Hkv) >= 128LL * a.B) return launch_paged(a, s);
    const size_t rows = (size_t)a.tokens * a.H, ints = round16(((size_t)a.tokens + 2) * 4);
    char *w = static_cast<char *>(a.workspace) + 2 * paged_workspace_bytes(a.d);
    auto take = [&](size_t bytes) {
        char *at = w;
        w += bytes;
        return at;
    };
    float *o_a = reinterpret_cast<float *>(take(round16(rows * a.d * 4)));
    float *o_b = reinterpret_cast<float *>(take(round16(rows * a.d * 4)));
    float *lse_a = reinterpret_cast<float *>(take(round16(rows * 4)));
    float *lse_b = reinterpret_cast<float *>(take(round16(rows * 4)));
    int *owner_a = reinterpret_cast<int *>(take(round16(rows * 4)));
    int *owner_b = reinterpret_cast<int *>(take(round16(rows * 4)));
    SplitParams sp;
    std::memset(&sp, 0, sizeof(sp));
    fill_params(a, &sp.p);
    sp.group_start = sa.group_start;
    sp.prefix_len = sa.prefix_len;
    sp.groups = sa.groups;
    sp.most = 2LL * sa.groups < a.tokens ? 2 * sa.groups : a.tokens;   // (a group that shares has two tokens)
    sp.first_key = reinterpret_cast<int *>(take(ints));
    sp.q_start = reinterpret_cast<int *>(take(ints));
    sp.kv_len = reinterpret_cast<int *>(take(ints));
    sp.row_of = reinterpret_cast<int *>(take(ints));
    sp.ctas = reinterpret_cast<int *>(take(16));
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return cudaErrorInvalidDevice;
    const int g = sp.p.g;
    sp.sms = di.sms;
    sp.tile_tokens = 128 / g;
    sp.shared = kChunkCosts[a.d > 64];
    // (a.max_new is a hint; the split of the SMs follows it, the results do not)
    const bool few = paged_decode_covers(a);
    sp.own_tokens = few ? 16 / g : 2 * sp.tile_tokens;
    sp.own = few ? kTokenCosts[a.d > 64] : kChunkCosts[a.d > 64];
    if (few && a.max_new * g > 8) sp.own = Costs{1.5f * sp.own.item, 1.5f * sp.own.tile, 1.5f * sp.own.tile2, 1.5f * sp.own.fixed};
    sp.own_per_sm = few && a.d <= 64 ? 2 : 1;
    cudaError_t e = launch_early(shared_split_kernel, dim3(1), kSplitThreads, 0, s, sp);
    if (e != cudaSuccess) return e;
    PagedArgs part = a;      // the shared keys
    part.aK = part.aV = nullptr;
    part.ths = 0;
    part.clip_k = 0;
    part.q_start = sp.q_start;
    part.kv_len = sp.kv_len;
    part.row_of = sp.row_of;
    part.B = sp.most;
    part.max_new = a.tokens;
    part.flat = 1;
    part.owner = owner_a;
    part.ctas = sp.ctas;
    JoinParams j;
    std::memset(&j, 0, sizeof(j));
    auto run = [&](PagedArgs &x, Part &r, float *o, float *lse) {
        PagedLeft left{};
        x.left = &left;
        x.f32_out = 1;
        x.out = o;
        x.lse = lse;
        const cudaError_t st = launch_paged(x, s);
        const char *ws = static_cast<const char *>(x.workspace);
        r = Part{o, lse, reinterpret_cast<const float *>(ws + desc_bytes()), x.owner, left.ctas,
                 reinterpret_cast<const Desc *>(ws), left.rec_rows, left.grid};
        return st;
    };
    if ((e = run(part, j.part[0], o_a, lse_a)) != cudaSuccess) return e;
    part = a;                // each request's own
    part.first_key = sp.first_key;
    part.workspace = static_cast<char *>(a.workspace) + paged_workspace_bytes(a.d);
    part.owner = owner_b;
    part.ctas = sp.ctas + 1;
    part.overlap = 1;
    if ((e = run(part, j.part[1], o_b, lse_b)) != cudaSuccess) return e;
    j.q = a.q;
    j.aK = a.aK;
    j.aV = a.aV;
    j.q_stride = a.q_stride;
    j.ths = a.ths;
    j.tokens = a.tokens;
    j.H = a.H;
    j.Hkv = a.Hkv;
    j.g = a.H / a.Hkv;
    j.d = a.d;
    j.scale_log2 = sp.p.scale_log2;
    j.first_key = sp.first_key;
    j.q_start = a.q_start;
    j.B = a.B;
    j.out = a.out;
    j.lse = a.lse;
    return a.bf16 ? launch_join<__nv_bfloat16>(j, s) : launch_join<float>(j, s);
}

}  // namespace relattn
