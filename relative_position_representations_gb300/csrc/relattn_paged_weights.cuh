// What the kernels share that gather the attention weights of cached keys: parameters, and the list
// of units that the tickets count.
//
// mass[page][h'][row] (+)= sum over the new tokens i and the query heads h of group h' that see key j of
// exp(e_ij - lse_ih). In the log2 domain a weight is 2^(s2 q.k_j + R_i - lse2_i), R_i the table term;
// for keys at least clip_k back R_i is q.aK_0, a constant of the row, so the rows' constants nl_i =
// R_i0 - lse2_i are formed once in front (in fp32) and only the last keys need a table row of their own.
#pragma once

#include "relattn_paged.cuh"

namespace relattn {
namespace paged {

struct WeightParams {
    Params p;                    // T: every token of a request makes one item
    const float *lse;            // [tokens][H]
    float *mass;
    long long mass_stride;
    int accumulate;
    int per_tile;                // units: 0: pairs of tiles (below); else units of one tile
    int tile_tokens;             // tokens of a query tile
    // pairs of tiles in a unit: the rows of one query tile stay while four pairs of key tiles pass by
    __host__ __device__ int pairs(int n) const { return n <= tile_tokens ? 4 : 1; }
    unsigned long long *ticket;  // the next unit
    int *count;                  // requests with new tokens ...
    int *busy;                   // ... their numbers ...
    long long *start;            // ... and the unit that each begins with; start[count]: all units
    float *nl;                   // [tokens][H]
};

// the request and the unit within it; one warp calls it, u below start[count]
__device__ __forceinline__ int find_unit(const WeightParams &w, int count, long long u, long long &rest) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = count;       // the last entry with start <= u lies in lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, lane * step < n && w.start[at] <= u);
        const int k = 31 - __clz((int)m);
        lo += k * step;
        n = min(step, n - k * step);
    }
    rest = u - w.start[lo];
    return lo;
}

__device__ __forceinline__ int units_of(const WeightParams &w, int nt, int n) {
    const int step = 2 * w.pairs(n);
    return w.per_tile ? nt * w.per_tile : (nt + step - 1) / step;
}
// What a request's rows have given a key at position j, the first new token's being pos0. Several requests of the
// call may share the page of a key in front of theirs, so its entry is added to in the L2; where they do not, it is one
// addition a call, the same bits in every call.
__device__ __forceinline__ void leave_mass(const WeightParams &w, float *at, float sum, int j, int pos0) {
    if (w.accumulate && j < pos0) atomicAdd(at, sum);
    else *at = sum;
}

// tokens of a request that see some key of j0 .. j0 + len - 1 (window and sinks taken into account)
__device__ __forceinline__ int first_token(int j0, int pos0) { return max(0, j0 - pos0); }
__device__ __forceinline__ int end_token(const Params &p, int j0, int len, int pos0, int n) {
    if (p.window == 0 || j0 < p.sinks) return n;
    return (int)max(0LL, min((long long)n, (long long)j0 + len - 1 + p.window - pos0));
}

// units and row constants; in front of the kernels that take tickets
cudaError_t launch_weights_prep(const WeightParams &w, bool bf16, cudaStream_t s);
bool weights_tc_covers(const PagedWeightsArgs &a);
cudaError_t launch_weights_tc(const PagedWeightsArgs &a, WeightParams w, cudaStream_t s);

}  // namespace paged
}  // namespace relattn
