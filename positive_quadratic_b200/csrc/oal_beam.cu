// oal_beam.cu -- beam search on recurrent state: the selection of the best continuations over
// beams and vocabulary, and the copies of prefix states that follow the chosen parents.
//
// Selection.  A candidate (row r, token t) of a search scores running[r] + x_rt - lse_r with
// lse_r = log sum_t exp(x_rt); the n best of the search's beams x V candidates are returned,
// equal scores in the order of their flat place (row, then token).
//   select_scan_kernel   one pass over the logits: the maximum and the sum of exponentials of
//                        every slice, the maximum of every group of 32 logits (those that a
//                        thread holds in registers at a time) and of every bundle of 32 groups
//                        (a warp's);
//   select_merge_kernel  one block per search: lse of each row; the n best bundles bound the n
//                        best candidates from below (n different candidates reach the n-th), so
//                        only bundles that reach it, a few n of them, have their groups looked
//                        at; of these the n best give a better bound, and only groups that reach
//                        it, about n, are read again and their candidates ranked.  Scores are
//                        compared in 64 bits, so that a row's candidates keep the order of their
//                        logits and those of different rows the order that the log-sums give them.
// A log-sum is joined from fp32 exponentials in 64 bits.  With u = 2^-24: x - max, the factor log2 e
// and their product are off by 2.5 u of a term's exponent d = max - x, ex2 by 4 u, and a thread's sum of
// 32 terms by 10 u.  Terms weigh e^-d, so that the mean of d is below log V <= 21.5; with the
// same for a partial sum that moves to a larger maximum: below 128 u = 2^-17 in all.
// The scan reads every logit once (128 rows of 151,936 in bf16, a fifth of them ended, 31 MB: 11 us,
// 2.8 TB/s); the merge is a chain of dependent loads and barriers, 10 to 12 us whatever the size.  The
// call takes 20.7 us there: the merge's launch is hidden behind the scan.
#pragma once

#include <cmath>
#include <type_traits>

#include "oal_common.cuh"
#include "oal_kernels.cuh"

namespace oal {
namespace beam {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSelect = 32;
constexpr int kMaxBeams = 256;
constexpr int kGroup = 32;                     // logits of a group
constexpr int kTile = kGroup * kThreads;       // logits that a block holds at a time
constexpr int kMergeThreads = 1024;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kList = 2048;                    // candidates that are ranked in shared memory
constexpr int kFew = (kList - kMaxBeams) / kGroup;  // groups whose logits the list is sure to hold

struct Slice {  // of one (row, slice)
    double sum;   // sum of exp(x - max)
    float max;    // -inf: every logit of the slice is; NaN: one is NaN
    int pad;
};

template <typename T> struct VecOf;
template <> struct VecOf<float> { static constexpr int n = 4; };
template <> struct VecOf<__nv_bfloat16> { static constexpr int n = 8; };

__device__ __forceinline__ void unpack(uint4 a, float* x, float)
{
    x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y);
    x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
}
__device__ __forceinline__ void unpack(uint4 a, float* x, __nv_bfloat16)
{
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Where a row's groups lie.  Tiles, threads and partial sums follow the row's tokens, wherever the
// row starts in memory: equal rows go through the same operations and have the same log-sum to the
// last bit, so that their equal scores compare equal.  (Cut by 16-byte addresses, their log-sums
// differed by about 1e-8, which decided the order.)  A warp of a tile has 1024 tokens in a row, as
// vectors of 16 bytes; element j of the group of the tile's thread t is at place_of(t, j).  Group
// tile * 256 + t of a row belongs to bundle (tile * 256 + t) / 32.
template <typename T>
__device__ __forceinline__ int place_of(int t, int j)
{
    constexpr int kN = VecOf<T>::n;
    return ((t / 32 * (kGroup / kN) + j / kN) * 32 + t % 32) * kN + j % kN;
}

// Floats in the order of unsigned integers, and back.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u)
{
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// Block (slice, row): `tiles` tiles from slice * tiles on.  gmax [rows][all tiles][256], bmax
// [rows][all tiles][8].  kSkew: rows need not start on 16 bytes; their vectors are put together from
// the aligned ones that a lane and its neighbour hold.  128 rows of 50,257: a call of 15.6 us in bf16
// and 17.0 in fp32, against 15.4 and 16.6 when rows were cut by address; 128 rows of 151,936 in bf16,
// which start on 16 bytes: 22.5, against 23.0.  (Three blocks per SM: 64 to 80 registers.  Left to
// itself the compiler gives bf16 64 and fp32 87 where rows are skewed: with a fifth of the rows
// ended 20.3 and 17.4 us for these two sizes, against 18.5 and 15.6.)
template <typename T, bool kSkew>
__global__ void __launch_bounds__(kThreads, 3) select_scan_kernel(
    const T* __restrict__ logits, long long ld, int rows, int V, int tiles, int all_tiles,
    const float* __restrict__ running, const uint8_t* __restrict__ ended,
    float* __restrict__ gmax, float* __restrict__ bmax, Slice* __restrict__ part)
{
    constexpr int kN = VecOf<T>::n, kVecs = kGroup / kN;
    const int row = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the merge does not look at such a row's groups
    if ((ended && ended[row]) || !isfinite(running[row])) return;
    const long long first = row * ld;
    const int skew = kSkew ? int(first % kN) : 0;
    const long long end = (rows - 1) * ld + V;  // of the whole array
    // tokens of this row from here on lie in the array's last vector, which `end` cuts short
    const int cut = max(int(min(end - end % kN - first, (long long)V)), 0);
    const int t_first = blockIdx.x * tiles, t_last = min(t_first + tiles, all_tiles);
    float m = -INFINITY;   // this thread's maximum, and its sum of exp(x - m)
    double s = 0.0;
    bool nan = false;
    uint4 raw[kVecs], behind;  // behind: the vector after the warp's (lane 0)
    auto vector = [&](long long at) {
        return at + kN <= end ? __ldcs(reinterpret_cast<const uint4*>(logits + at))
                              : make_uint4(0, 0, 0, 0);
    };
    auto load = [&](int tile) {
        const long long at = first - skew + (long long)tile * kTile + place_of<T>(tid, 0);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) raw[i] = vector(at + i * 32 * kN);
        if (kSkew && lane == 0) behind = vector(at + kVecs * 32 * kN);
    };
    load(t_first);
    for (int tile = t_first; tile < t_last; ++tile) {
        float x[kGroup];
        if (kSkew) {
            // the row's vectors start kW words (and half a word, in bf16) into the aligned ones
            auto unpack_from = [&](auto words) {
                constexpr int kW = decltype(words)::value, kHalf = sizeof(T) == 2;
                const int half = kHalf ? 16 * (skew & 1) : 0;
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    const uint4 a = raw[i], last = i + 1 < kVecs ? raw[(i + 1) % kVecs] : behind;
                    uint32_t w[8] = {a.x, a.y, a.z, a.w, last.x, last.y, last.z, last.w}, v[4];
#pragma unroll
                    for (int e = 0; e < kW + kHalf; ++e)  // lane 31's neighbour: lane 0's next vector
                        w[4 + e] = __shfl_sync(~0u, lane == 0 ? w[4 + e] : w[e], (lane + 1) & 31);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = kHalf ? __funnelshift_r(w[kW + e], w[kW + e + kHalf], half) : w[kW + e];
                    unpack(make_uint4(v[0], v[1], v[2], v[3]), x + i * kN, T());
                }
            };
            switch (skew * int(sizeof(T)) / 4) {
            case 0: unpack_from(std::integral_constant<int, 0>{}); break;
            case 1: unpack_from(std::integral_constant<int, 1>{}); break;
            case 2: unpack_from(std::integral_constant<int, 2>{}); break;
            default: unpack_from(std::integral_constant<int, 3>{});
            }
        } else {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) unpack(raw[i], x + i * kN, T());
        }
        const int t0 = tile * kTile;  // token of the tile's place 0
        if (t0 + kTile > cut) {
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                if (t0 + place_of<T>(tid, j) >= V) x[j] = -INFINITY;
#pragma unroll 1
            for (int t = max(cut, t0); t < min(V, t0 + kTile); ++t) {
                const float one = to_f32(logits[first + t]);
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    if (t0 + place_of<T>(tid, j) == t) x[j] = one;
            }
        }
        if (tile + 1 < t_last) load(tile + 1);
        float g = x[0];
        float chk = 0.f;
#pragma unroll
        for (int j = 1; j < kGroup; ++j) g = fmaxf(g, x[j]);
        const float up = fmaxf(m, g);
        if (up > -INFINITY) {  // (else all -inf, or NaN, which the sum below shows)
            float p[4] = {0.f, 0.f, 0.f, 0.f};
            // x - max first: what the largest terms lose is then next to nothing
#pragma unroll
            for (int j = 0; j < kGroup; ++j) p[j & 3] += exp2_fast((x[j] - up) * kLog2e);
            chk = (p[0] + p[1]) + (p[2] + p[3]);
            s = (up > m && m > -INFINITY ? s * double(exp2_fast((m - up) * kLog2e)) : s) + double(chk);
            m = up;
        } else {
#pragma unroll
            for (int j = 0; j < kGroup; ++j) nan |= x[j] != x[j];
        }
        nan |= chk != chk;
        gmax[((long long)row * all_tiles + tile) * kThreads + tid] = g;
        const uint32_t best = __reduce_max_sync(~0u, ordered(g));
        if (lane == 0)
            bmax[((long long)row * all_tiles + tile) * kWarps + (tid >> 5)] = unordered(best);
    }
    // the slice: sums brought to the common maximum
    __shared__ float wmax[kWarps];
    __shared__ double wsum[kWarps];
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) wmax[tid >> 5] = top;
    nan = __syncthreads_or(nan);
    top = wmax[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, wmax[w]);
    double sum = m > -INFINITY && top < INFINITY ? s * double(exp2_fast((m - top) * kLog2e)) : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) wsum[tid >> 5] = sum;
    __syncthreads();
    if (tid == 0) {
        sum = 0.0;
        for (int w = 0; w < kWarps; ++w) sum += wsum[w];
        // (a +inf logit makes inf - inf in the sums: it is not a NaN of the row's)
        part[(long long)row * gridDim.x + blockIdx.x] = {sum, top == INFINITY ? top : nan ? NAN : top, 0};
    }
}

struct Candidate {
    double score;
    long long place;  // row of the search * V + token
};
__device__ __forceinline__ bool better(const Candidate& a, const Candidate& b)
{
    return a.score > b.score || (a.score == b.score && a.place < b.place);
}

// Block = one search.  A row is live if it has a log-softmax (a finite running score and maximum,
// no NaN).  The candidates of the others: of an ended row the padding token at its running score;
// everything else scores -inf.  The block may start while the scan still writes the maxima and sums:
// these are no read-only data of this kernel (no __restrict__), or a load of them might be taken to
// before the wait.
template <typename T>
__global__ void __launch_bounds__(kMergeThreads, 1) select_merge_kernel(
    const T* __restrict__ logits, long long ld, const float* gmax, const float* bmax, const Slice* part,
    int beams, int V, int n, int slices, int all_tiles,
    const float* __restrict__ running, const uint8_t* __restrict__ ended, int pad_token,
    float* __restrict__ scores, int32_t* __restrict__ parents, int32_t* __restrict__ tokens)
{
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row0 = b * beams;
    // of each row its running score, its largest logit and log sum exp(x - max): apart, since a
    // row of the type's lowest value would swallow the sum
    __shared__ double shift[kMaxBeams];  // running - log sum; NaN: not live
    __shared__ float rowmax[kMaxBeams];
    __shared__ Candidate list[kList];
    __shared__ uint32_t wlow[kMergeWarps];
    __shared__ Candidate wbest[kMergeWarps];
    __shared__ int groups, found;
    __shared__ int picked[kList];
    if (tid == 0) groups = found = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int r = warp; r < beams; r += kMergeWarps) {
        double out = NAN;
        float m = -INFINITY;
        const float run = running[row0 + r];
        if (!(ended && ended[row0 + r]) && isfinite(run)) {
            const Slice* p = part + (long long)(row0 + r) * slices;
            bool nan = false;
            for (int i = lane; i < slices; i += 32) {
                nan |= p[i].max != p[i].max;
                m = fmaxf(m, p[i].max);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            if (!__any_sync(~0u, nan) && isfinite(m)) {
                double s = 0.0;
                for (int i = lane; i < slices; i += 32)
                    if (p[i].sum > 0.0) s += p[i].sum * exp(double(p[i].max) - double(m));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
                out = double(run) - log(s);
            }
        }
        if (lane == 0) {
            shift[r] = out;
            rowmax[r] = m;
        }
    }
    __syncthreads();
    auto score = [&](int r, float x) { return (double(x) - double(rowmax[r])) + shift[r]; };
    const int per = all_tiles * kThreads;  // groups of a row
    const int all_groups = beams * per;    // group i is number i % per of row i / per
    // the group's best score; -inf where nothing is to be had
    auto group_score = [&](int i) -> double {
        const int r = i / per;
        if (shift[r] != shift[r]) return -INFINITY;
        const float x = gmax[(long long)row0 * per + i];
        return x > -INFINITY ? score(r, x) : -INFINITY;
    };
    const int all_bundles = all_groups / 32;
    auto bundle_score = [&](int i) -> double {
        const int r = i / (per / 32);
        if (shift[r] != shift[r]) return -INFINITY;
        const float x = bmax[(long long)row0 * (per / 32) + i];
        return x > -INFINITY ? score(r, x) : -INFINITY;
    };
    // Each warp's best bundle, a warp having every 32nd of them: the rows' scores differ, and a
    // warp with one row's bundles alone would have a poor best.  The bound is the n-th best of the
    // warps' bests, which n <= 32 bundles reach; rounded down to fp32, where a warp's maximum is
    // one instruction.
    double best = -INFINITY;
    for (int i = 32 * lane + warp; i < all_bundles; i += kMergeThreads)
        best = fmax(best, bundle_score(i));
    const uint32_t warp_best = __reduce_max_sync(~0u, ordered(__double2float_rd(best)));
    if (lane == 0) wlow[warp] = warp_best;
    __syncthreads();
    double bound;
    {
        const uint32_t mine = wlow[lane];
        int rank = 0;
#pragma unroll
        for (int w = 0; w < 32; ++w) {
            const uint32_t o = wlow[w];
            rank += o > mine || (o == mine && w < lane);
        }
        const uint32_t who = __ballot_sync(~0u, rank == n - 1);
        bound = unordered(__shfl_sync(~0u, mine, __ffs(who) - 1));
    }
    // The bundles that reach the bound, the groups of theirs that do, and the n-th best of these,
    // which is a better bound.
    for (int i = tid; i < all_bundles; i += kMergeThreads) {
        const double v = bundle_score(i);
        if (v >= bound && v > -INFINITY) {
            const int at = atomicAdd(&found, 1);
            if (at < kList) picked[at] = i;
        }
    }
    __syncthreads();
    for (int k = warp; k < min(found, kList); k += kMergeWarps) {
        const int i = picked[k] * 32 + lane;
        const double v = group_score(i);
        if (v >= bound && v > -INFINITY) {
            const int at = atomicAdd(&groups, 1);
            if (at < kList) list[at] = {v, i};
        }
    }
    __syncthreads();
    int have = groups;
    __shared__ double tighter;
    // whether, of the groups that count, every one is listed
    const bool all = found <= kList && have <= kList;
    if (!all) {
        // Many groups share the bound: the n-th best by taking one after another.
        Candidate last{INFINITY, -1};
        for (int k = 0; k < n; ++k) {
            Candidate c{-INFINITY, 0x7FFFFFFFFFFFFFFFll};
            for (int i = tid; i < all_groups; i += kMergeThreads) {
                const Candidate x{group_score(i), i};
                if (better(last, x) && better(x, c)) c = x;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const Candidate x{__shfl_xor_sync(~0u, c.score, o), __shfl_xor_sync(~0u, c.place, o)};
                if (better(x, c)) c = x;
            }
            if (lane == 0) wbest[warp] = c;
            __syncthreads();
            for (int w = 0; w < kMergeWarps; ++w)
                if (better(wbest[w], c)) c = wbest[w];
            __syncthreads();
            last = c;
        }
        bound = last.score;
    } else if (have > kFew) {
        if (tid == 0) tighter = bound;
        __syncthreads();
        for (int i = tid; i < have; i += kMergeThreads) {
            const Candidate c = list[i];
            int rank = 0;
            for (int j = 0; j < have; ++j) rank += better(list[j], c);
            if (rank == n - 1) tighter = c.score;
        }
        __syncthreads();
        bound = tighter;
    }
    // The groups that reach the bound: few, unless many tie.
    __syncthreads();
    if (tid == 0) groups = found = 0;
    __syncthreads();
    if (all) {
        for (int i = tid; i < have; i += kMergeThreads)
            if (list[i].score >= bound) picked[atomicAdd(&groups, 1)] = int(list[i].place);
    } else {
        for (int i = tid; i < all_groups; i += kMergeThreads) {
            const double v = group_score(i);
            if (v >= bound && v > -INFINITY) {
                const int at = atomicAdd(&groups, 1);
                if (at < kList) picked[at] = i;
            }
        }
    }
    __syncthreads();
    have = groups;
    // A group's logits, one per lane; `keep` says which count.
    auto expand = [&](int r, int g, auto keep) {
        const int t = g / kThreads * kTile + place_of<T>(g % kThreads, lane);
        if (t < V) {
            const float x = to_f32(logits[(row0 + r) * ld + t]);
            const double v = x > -INFINITY ? score(r, x) : -INFINITY;
            if (keep(v) && v > -INFINITY) {
                const int i = atomicAdd(&found, 1);
                if (i < kList) list[i] = {v, (long long)r * V + t};
            }
        }
    };
    const bool tied = have > kFew;
    if (!tied) {
        for (int i = warp; i < have; i += kMergeWarps)
            expand(picked[i] / per, picked[i] % per, [&](double v) { return v >= bound; });
    } else {
        // Candidates above the bound are in the fewer than n groups above it.  Of those at the
        // bound the first n in the order of their places are enough: tile by tile (places of one
        // tile all lie before those of the next) until n are found.
        for (int i = tid; i < all_groups; i += kMergeThreads) {  // (a multiple of 256 groups)
            uint32_t hit = __ballot_sync(~0u, group_score(i) > bound);
            for (; hit; hit &= hit - 1) {
                const int g = i - lane + __ffs(hit) - 1;
                expand(g / per, g % per, [&](double u) { return u > bound; });
            }
        }
        __syncthreads();
        int ties = 0;
        for (int r = 0; r < beams && ties < n && bound > -INFINITY; ++r)
            for (int tile = 0; tile < all_tiles && ties < n; ++tile) {
                const double v = tid < kThreads ? group_score(r * per + tile * kThreads + tid) : -INFINITY;
                if (!__syncthreads_or(v >= bound)) continue;
                // the tile's logits in the order of their places, 1024 at a time
                const long long first = (row0 + r) * ld;
                for (int at = 0; at < kTile && ties < n; at += kMergeThreads) {
                    const int t = tile * kTile + at + tid;
                    const bool hit = t < V &&
                                     score(r, to_f32(logits[first + t])) == bound;
                    const uint32_t in_warp = __ballot_sync(~0u, hit);
                    __shared__ int before[kMergeWarps];
                    if (lane == 0) before[warp] = __popc(in_warp);
                    __syncthreads();
                    int lower = 0, total = 0;
                    for (int w = 0; w < kMergeWarps; ++w) {
                        lower += w < warp ? before[w] : 0;
                        total += before[w];
                    }
                    lower += __popc(in_warp & ((1u << lane) - 1));
                    if (hit && ties + lower < n) {
                        const int i = atomicAdd(&found, 1);
                        if (i < kList) list[i] = {bound, (long long)r * V + t};
                    }
                    ties += total;
                    __syncthreads();
                }
            }
    }
    // the padding tokens of ended rows
    for (int r = tid; r < beams; r += kMergeThreads)
        if (ended && ended[row0 + r] && isfinite(running[row0 + r])) {
            const int i = atomicAdd(&found, 1);
            if (i < kList) list[i] = {double(running[row0 + r]), (long long)r * V + pad_token};
        }
    __syncthreads();
    have = found;
    for (int i = tid; i < have; i += kMergeThreads) {
        const Candidate c = list[i];
        int rank = 0;
        for (int j = 0; j < have; ++j) rank += better(list[j], c);
        if (rank < n) {
            scores[(long long)b * n + rank] = float(c.score);
            parents[(long long)b * n + rank] = row0 + int(c.place / V);
            tokens[(long long)b * n + rank] = int(c.place % V);
        }
    }
    // Fewer than n candidates with a score: the rest at -inf, in the order of their places.  Of
    // the first n + have places at most `have` are taken.
    if (have < n && warp == 0) {
        int rank = have;
        for (int at = 0; rank < n; at += 32) {
            const long long place = at + lane;
            bool taken = false;
            for (int j = 0; j < have; ++j) taken |= list[j].place == place;
            const uint32_t free = __ballot_sync(~0u, !taken && place < (long long)beams * V);
            const int mine = rank + __popc(free & ((1u << lane) - 1));
            if (((free >> lane) & 1) && mine < n) {
                scores[(long long)b * n + mine] = -INFINITY;
                parents[(long long)b * n + mine] = row0 + int(place / V);
                tokens[(long long)b * n + mine] = int(place % V);
            }
            rank += __popc(free);
        }
    }
}

// ------------------------------------------------------------------------------------------
// dst row i = src row parents[i], rows of `units` 16-byte words; block (part of a row, i).  The
// last row of blocks copies the `head` words before the rows, with the batch size of dst.
// Memory-bound: 64 states of 2 heads, 120 MB with the parents that are read, in 22.8 us, 5.3 TB/s.
// ------------------------------------------------------------------------------------------
constexpr int kCopy = 8;  // words in flight per thread

__global__ void __launch_bounds__(kThreads) gather_rows_kernel(const uint4* __restrict__ src,
                                                               int src_rows,
                                                               const int32_t* __restrict__ parents,
                                                               uint4* __restrict__ dst, int rows,
                                                               int units, int head)
{
    const int i = blockIdx.y;
    if (i == rows) {
        for (int e = blockIdx.x * kThreads + threadIdx.x; e < head; e += gridDim.x * kThreads) {
            uint4 w = src[e];
            if (e == 0) w.z = uint32_t(rows);  // StateHeader::B
            dst[e] = w;
        }
        return;
    }
    int from = parents[i];
    if (head) src_rows = state_sequences(src, src_rows);  // a buffer may have room for more
    if (from < 0 || from >= src_rows) {
        if (threadIdx.x == 0) raise_error(OAL_ERR_VALUE);
        from = from < 0 ? 0 : src_rows - 1;
    }
    const uint4* s = src + head + size_t(from) * units;
    uint4* d = dst + head + size_t(i) * units;
    const int at = blockIdx.x * (kCopy * kThreads) + threadIdx.x;
    uint4 w[kCopy];
#pragma unroll
    for (int x = 0; x < kCopy; ++x)
        if (at + x * kThreads < units) w[x] = s[at + x * kThreads];
#pragma unroll
    for (int x = 0; x < kCopy; ++x)
        if (at + x * kThreads < units) __stcs(d + at + x * kThreads, w[x]);
}
static_assert(offsetof(StateHeader, B) == 8, "the batch size is the header's third word");

int gather_rows(const void* src, int src_rows, const int32_t* parents, void* dst, int rows,
                size_t row_bytes, size_t head_bytes, cudaStream_t st)
{
    const int units = int(row_bytes / 16), per = kCopy * kThreads;
    LaunchScope ls("gather_rows", st);
    gather_rows_kernel<<<dim3((units + per - 1) / per, rows + (head_bytes > 0)), kThreads, 0, st>>>(
        static_cast<const uint4*>(src), src_rows, parents, static_cast<uint4*>(dst), rows, units,
        int(head_bytes / 16));
    OAL_LAUNCH_CHECK();
    return OAL_OK;
}

int tiles_of(int V) { return (V + kTile - 1) / kTile; }

// Tiles per block of the scan: one, until the grid has four blocks for every SM (about as many as
// are resident); then more, so that a block loads a tile while it works on the one before.  128 rows
// of 151,936 in bf16: 20.7 us, against 23.1 with three blocks per SM and 22.1 with eight (512 rows of
// 32,000 in fp32: 26.1, and 25.2 with eight).
int tiles_per_block(int rows, int all_tiles)
{
    const long long tiles = (long long)rows * all_tiles, blocks = std::max(4 * sm_count(), 1);
    return int(std::min<long long>(all_tiles, (tiles + blocks - 1) / blocks));
}

struct SelectLayout {
    size_t gmax, bmax, total;  // the slices' sums lie before the maxima
};
SelectLayout select_layout(int rows, int V)
{
    const size_t tiles = size_t(rows) * tiles_of(V);  // at least as many as slices
    SelectLayout l;
    l.gmax = align256(tiles * sizeof(Slice));
    l.bmax = l.gmax + tiles * kThreads * sizeof(float);
    l.total = l.bmax + tiles * kWarps * sizeof(float);
    return l;
}

// (A tile may reach past the last logit, by less than a tile: its places stay below 2^31.)
int check_select(int B, int beams, int V, int n, int dtype)
{
    if (B < 0 || beams < 1 || V < 1 || n < 1) return OAL_ERR_SHAPE;
    if (dtype != OAL_F32 && dtype != OAL_BF16) return OAL_ERR_UNSUPPORTED;
    if (n > kMaxSelect || beams > kMaxBeams) return OAL_ERR_UNSUPPORTED;
    if ((long long)n > (long long)beams * V || (long long)beams * V >= (1LL << 31) - 2 * kTile ||
        (long long)B * beams > kMaxGridPlanes)
        return OAL_ERR_SHAPE;
    return OAL_OK;
}

template <typename T>
cudaError_t launch_select(const void* logits, long long ld, const float* running,
                          const uint8_t* ended, int pad_token, int B, int beams, int V, int n,
                          float* scores, int32_t* parents, int32_t* tokens, void* ws,
                          cudaStream_t st)
{
    const int rows = B * beams, all_tiles = tiles_of(V);
    const int tiles = tiles_per_block(rows, all_tiles), slices = (all_tiles + tiles - 1) / tiles;
    Slice* part = static_cast<Slice*>(ws);
    const SelectLayout l = select_layout(rows, V);
    float* gmax = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + l.gmax);
    float* bmax = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + l.bmax);
    const T* x = static_cast<const T*>(logits);
    {
        LaunchScope ls("select_scan", st);
        const auto scan = ld % VecOf<T>::n ? select_scan_kernel<T, true> : select_scan_kernel<T, false>;
        scan<<<dim3(slices, rows), kThreads, 0, st>>>(x, ld, rows, V, tiles, all_tiles, running, ended,
                                                      gmax, bmax, part);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    LaunchScope ls("select_merge", st);
    return launch_ex(select_merge_kernel<T>, dim3(B), dim3(kMergeThreads), 0, st, true, x, ld,
                     static_cast<const float*>(gmax), static_cast<const float*>(bmax),
                     static_cast<const Slice*>(part), beams, V, n,
                     slices, all_tiles, running, ended, pad_token, scores, parents, tokens);
}

int check_reorder(const void* src, int src_B, const int32_t* parents, const void* dst,
                  const oal_shape* s)
{
    int rc = check_common(s);
    if (rc) return rc;
    oal_shape from = *s;
    from.B = src_B;
    if (src_B < 1) return OAL_ERR_SHAPE;
    if ((rc = check_common(&from)) || (rc = check_planes(s->B + 1ll))) return rc;
    if (s->Hkv * state_unit_bytes() / 16 >= (size_t(1) << 31)) return OAL_ERR_SHAPE;
    if (!src || !dst || (s->B > 0 && !parents)) return OAL_ERR_NULL;
    if (!aligned16(src) || !aligned16(dst) || (reinterpret_cast<uintptr_t>(parents) & 3))
        return OAL_ERR_ALIGN;
    return OAL_OK;
}

}  // namespace beam
}  // namespace oal

extern "C" {

using namespace oal;

int oal_beam_select_workspace_bytes(int B, int beams, int V, int n, int dtype, size_t* bytes)
{
    const int rc = beam::check_select(B, beams, V, n, dtype);
    if (rc) return rc;
    if (!bytes) return OAL_ERR_NULL;
    *bytes = beam::select_layout(B * beams, V).total;
    return OAL_OK;
}

int oal_beam_select(const void* logits, long long row_stride, int dtype, const float* running,
                    const uint8_t* ended, int pad_token, int B, int beams, int V, int n,
                    float* scores, int32_t* parents, int32_t* tokens, void* workspace,
                    size_t workspace_bytes, void* stream)
{
    int rc = beam::check_select(B, beams, V, n, dtype);
    if (rc) return rc;
    if (row_stride < V) return OAL_ERR_SHAPE;
    if (ended && (pad_token < 0 || pad_token >= V)) return OAL_ERR_SHAPE;
    if (B == 0) return OAL_OK;
    if (!logits || !running || !scores || !parents || !tokens) return OAL_ERR_NULL;
    if (!aligned16(logits) || ((reinterpret_cast<uintptr_t>(running) |
                                reinterpret_cast<uintptr_t>(scores) |
                                reinterpret_cast<uintptr_t>(parents) |
                                reinterpret_cast<uintptr_t>(tokens)) & 3))
        return OAL_ERR_ALIGN;
    size_t need = 0;
    if ((rc = oal_beam_select_workspace_bytes(B, beams, V, n, dtype, &need))) return rc;
    if (!workspace || workspace_bytes < need) return OAL_ERR_WORKSPACE;
    if (!aligned16(workspace)) return OAL_ERR_ALIGN;
    // (one search's block may write its results while another's reads its logits again)
    const size_t n_out = size_t(B) * n * 4, rows = size_t(B) * beams;
    const size_t n_in = ((rows - 1) * size_t(row_stride) + V) * (dtype == OAL_BF16 ? 2 : 4);
    if (any_overlap({{scores, n_out}, {parents, n_out}, {tokens, n_out}},
                    {{logits, n_in}, {running, rows * 4}, {ended, rows}}))
        return OAL_ERR_OVERLAP;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const auto go = dtype == OAL_BF16 ? beam::launch_select<__nv_bfloat16>
                                      : beam::launch_select<float>;
    OAL_CUDA_TRY(go(logits, row_stride, running, ended, pad_token, B, beams, V, n, scores, parents,
                    tokens, workspace, st));
    return OAL_OK;
}

int oal_state_reorder(const void* src, int src_B, const int32_t* parents, void* dst,
                      const oal_shape* s, void* stream)
{
    int rc = beam::check_reorder(src, src_B, parents, dst, s);
    if (rc) return rc;
    if (any_overlap({{dst, state_bytes(s->B, s->Hq, s->Hkv)}},
                    {{src, state_bytes(src_B, s->Hq, s->Hkv)}, {parents, size_t(s->B) * 4}}))
        return OAL_ERR_OVERLAP;
    return beam::gather_rows(src, src_B, parents, dst, s->B, size_t(s->Hkv) * state_unit_bytes(),
                             kHeaderBytes + coef_bytes(s->Hq), static_cast<cudaStream_t>(stream));
}

int oal_decay_state_reorder(const float* src, int src_B, const int32_t* parents, float* dst,
                            const oal_shape* s, void* stream)
{
    int rc = beam::check_reorder(src, src_B, parents, dst, s);
    if (rc) return rc;
    const size_t row = size_t(s->Hkv) * kD * kDV * 4;
    if (any_overlap({{dst, s->B * row}}, {{src, src_B * row}, {parents, size_t(s->B) * 4}}))
        return OAL_ERR_OVERLAP;
    if (s->B == 0) return OAL_OK;
    return beam::gather_rows(src, src_B, parents, dst, s->B, row, 0,
                             static_cast<cudaStream_t>(stream));
}

int oal_decode_step_beam(const void* q, const void* k, const void* v, const void* src, int src_B,
                         const int32_t* parents, void* dst, float* out, void* workspace,
                         size_t workspace_bytes, const oal_shape* s, void* stream)
{
    int rc = beam::check_reorder(src, src_B, parents, dst, s);
    if (rc) return rc;
    if ((rc = check_planes((long long)s->B * s->Hkv))) return rc;
    oal_shape one = *s;
    one.T = 1;
    if ((rc = check_io(&one, q, k, v, out))) return rc;
    size_t need = 0;
    oal_decode_workspace_bytes(s, &need);
    if (!workspace || workspace_bytes < need) return OAL_ERR_WORKSPACE;
    if (!aligned16(workspace)) return OAL_ERR_ALIGN;
    const size_t token = size_t(s->B) * kD, nq = token * s->Hq, nk = token * s->Hkv;
    const size_t es = s->dtype == OAL_BF16 ? 2 : 4;
    if (any_overlap({{dst, state_bytes(s->B, s->Hq, s->Hkv)}, {out, nq * sizeof(float)}},
                    {{src, state_bytes(src_B, s->Hq, s->Hkv)}, {q, nq * es}, {k, nk * es},
                     {v, nk * es}, {parents, size_t(s->B) * 4}}))
        return OAL_ERR_OVERLAP;
    if (s->B == 0) return oal_state_reorder(src, src_B, parents, dst, s, stream);  // tables alone
    return launch_decode(q, k, v, dst, out,
                         reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                                  decode_ticket_bytes(s)),
                         s->B, s->Hq, s->Hkv, s->dtype, static_cast<cudaStream_t>(stream), src,
                         src_B, parents);
}

}  // extern "C"
