// oal_beam.cu -- beam search on recurrent state: the selection of the best continuations over
// beams and vocabulary, and the copies of prefix states that follow the chosen parents.
//
// Selection.  A candidate (row r, token t) of a search scores running[r] + x_rt - lse_r with
// lse_r = log sum_t exp(x_rt); the n best of the search's beams x V candidates are returned,
// equal scores in the order of their flat place (row, then token).  Within a row the order of
// scores is the order of logits, so no candidate outside a row's n best logits can be chosen:
//   select_slice_kernel  one pass over the logits: each block holds a slice of a row in
//                        registers, reduces its maximum and sum of exponentials, and lists its
//                        n best logits;
//   select_merge_kernel  one block per search: lse of each row from its slices, the scores of
//                        the listed candidates in 64 bits (candidates of different rows may lie
//                        closer than fp32 resolves), and the n best of them.
#pragma once

#include <cmath>

#include "oal_common.cuh"
#include "oal_kernels.cuh"

namespace oal {
namespace beam {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSelect = 32;
constexpr int kMaxBeams = 256;
constexpr int kList = 1024;  // survivors of the threshold that are ranked in shared memory

struct Slice {  // of one (row, slice)
    double sum;   // sum of exp(x - max)
    float max;    // -inf: every logit of the slice is; NaN: one is NaN
    int pad;
};

// Logits in the order of unsigned integers (-0 as 0, which it equals).
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u)
{
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// A logit and its place as one number: larger is better, the lower place first among equals.
__device__ __forceinline__ unsigned long long key_of(float x, int t)
{
    return (static_cast<unsigned long long>(ordered(x)) << 32) | (0xFFFFFFFFu - uint32_t(t));
}
__device__ __forceinline__ int place_of(unsigned long long key)
{
    return int(0xFFFFFFFFu - uint32_t(key));
}

template <typename T> struct VecOf;
template <> struct VecOf<float> { static constexpr int n = 4; };
template <> struct VecOf<__nv_bfloat16> { static constexpr int n = 8; };

__device__ __forceinline__ void unpack(uint4 a, float (&x)[4])
{
    x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y);
    x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
}
__device__ __forceinline__ void unpack(uint4 a, float (&x)[8])
{
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Block (slice, row).  Thread t holds kVecs vectors of 16 bytes, vector i at place
// (i * 256 + t) of the slice.  A row need not start on 16 bytes: the slice starts at the
// aligned address before it, and places outside the row count as absent.
template <typename T, int kVecs>
__global__ void __launch_bounds__(kThreads) select_slice_kernel(
    const T* __restrict__ logits, long long ld, int rows, int V, int n,
    const float* __restrict__ running, const uint8_t* __restrict__ ended,
    unsigned long long* __restrict__ best, Slice* __restrict__ part)
{
    constexpr int kN = VecOf<T>::n, kE = kVecs * kN;
    const int row = blockIdx.y, slices = gridDim.x, tid = threadIdx.x, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (ended && ended[row]) return;  // the merge does not read it
    if (!isfinite(running[row])) return;
    const long long first = row * ld;                 // the row's first element
    const int skew = int(first % kN);                 // elements before it in its vector
    const long long end = (rows - 1) * ld + V;        // of the whole array
    const long long base = first - skew + (long long)blockIdx.x * (kE * kThreads);
    const int t0 = int(blockIdx.x) * (kE * kThreads) - skew;  // token of the slice's place 0
    __shared__ unsigned long long list[kList];
    __shared__ float wmax[kWarps], wlow[kWarps];
    __shared__ double wsum[kWarps];
    __shared__ unsigned long long wkey[kWarps];
    __shared__ int count;
    if (tid == 0) count = 0;

    float x[kE];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const long long at = base + (long long)(i * kThreads + tid) * kN;
        float v[kN];
        if (at + kN <= end) {
            unpack(__ldcs(reinterpret_cast<const uint4*>(logits + at)), v);
        } else {
#pragma unroll
            for (int e = 0; e < kN; ++e) v[e] = at + e < end ? to_f32(logits[at + e]) : 0.f;
        }
        const int t = t0 + (i * kThreads + tid) * kN;
#pragma unroll
        for (int e = 0; e < kN; ++e)
            x[i * kN + e] = (unsigned(t + e) < unsigned(V)) ? v[e] : -INFINITY;
    }
    auto token = [&](int i) { return t0 + ((i / kN) * kThreads + tid) * kN + i % kN; };

    // the slice's maximum; a NaN stays one (fmaxf drops it, so it is looked for by itself)
    float m = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        m = fmaxf(m, x[i]);
        nan |= x[i] != x[i];
    }
    uint32_t mo = ordered(m);
    const uint32_t wm = __reduce_max_sync(~0u, mo);
    // a bound below which no chosen logit lies: each warp's ceil(n / 8)-th best lane maximum,
    // and the least of those of the block's 8 warps (8 ceil(n / 8) >= n logits reach it)
    uint32_t low = wm;
    for (int r = (n + kWarps - 1) / kWarps; r > 1; --r) {
        const uint32_t who = __ballot_sync(~0u, mo == low);
        if (lane == __ffs(who) - 1) mo = 0;
        low = __reduce_max_sync(~0u, mo);
    }
    if (lane == 0) {
        wmax[tid >> 5] = unordered(wm);
        wlow[tid >> 5] = low ? unordered(low) : -INFINITY;
    }
    nan = __syncthreads_or(nan);
    float top = wmax[0], bound = wlow[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
        top = fmaxf(top, wmax[w]);
        bound = fminf(bound, wlow[w]);
    }
    const bool live = top > -INFINITY && top < INFINITY && !nan;
    if (!live) {  // no finite sum: the row has no log-softmax, or this slice adds nothing to it
        if (tid == 0) part[size_t(row) * slices + blockIdx.x] = {0.0, nan ? NAN : top, 0};
        if (nan || top == INFINITY) return;  // the merge takes no candidate of the row
    } else {
        constexpr float kLog2e = 1.4426950408889634f;
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < kE; i += 8) {  // fp32 sums of 8, then 64 bits
            float p = 0.f;
#pragma unroll
            for (int e = i; e < i + 8; ++e) {
                // x - top first: what the largest terms lose is then next to nothing
                float y;
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((x[e] - top) * kLog2e));
                p += y;
            }
            s += double(p);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        if (lane == 0) wsum[tid >> 5] = s;
    }
    // every logit at or above the bound goes on the list
#pragma unroll
    for (int i = 0; i < kE; ++i)
        if (x[i] >= bound && unsigned(token(i)) < unsigned(V)) {
            const int at = atomicAdd(&count, 1);
            if (at < kList) list[at] = key_of(x[i], token(i));
        }
    __syncthreads();
    if (live && tid == 0) {
        double s = 0.0;
        for (int w = 0; w < kWarps; ++w) s += wsum[w];
        part[size_t(row) * slices + blockIdx.x] = {s, top, 0};
    }
    unsigned long long* out = best + (size_t(row) * slices + blockIdx.x) * n;
    const int found = count;
    if (found <= kList) {
        // the place of a listed logit is the number of better ones (keys are all different)
        for (int i = tid; i < found; i += kThreads) {
            const unsigned long long k = list[i];
            int rank = 0;
            for (int j = 0; j < found; ++j) rank += list[j] > k;
            if (rank < n) out[rank] = k;
        }
        for (int i = found + tid; i < n; i += kThreads) out[i] = 0;  // fewer logits than n
        return;
    }
    // too many equal logits at the bound: one after another, each the best below the last
    unsigned long long last = ~0ull;
    for (int r = 0; r < n; ++r) {
        unsigned long long k = 0;
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            if (unsigned(token(i)) >= unsigned(V)) continue;
            const unsigned long long c = key_of(x[i], token(i));
            if (c < last && c > k) k = c;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long c = __shfl_xor_sync(~0u, k, o);
            k = c > k ? c : k;
        }
        if (lane == 0) wkey[tid >> 5] = k;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) k = wkey[w] > k ? wkey[w] : k;
        __syncthreads();
        if (tid == 0) out[r] = k;
        last = k;
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

// Block = one search.  A row's candidates: its slices' lists; of an ended row the padding token
// at its running score, and (to fill up) others at -inf; of a row without a log-softmax (a NaN
// or +inf logit, no finite logit, a running score that is not finite) tokens at -inf.
__global__ void __launch_bounds__(kThreads) select_merge_kernel(
    const unsigned long long* __restrict__ best, const Slice* __restrict__ part, int beams, int V,
    int n, int slices, const float* __restrict__ running, const uint8_t* __restrict__ ended,
    int pad_token, float* __restrict__ scores, int32_t* __restrict__ parents,
    int32_t* __restrict__ tokens)
{
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row0 = b * beams;
    // of each row its largest logit and log sum exp(x - max), apart: a row of the type's lowest
    // value would swallow the sum.  NaN: no log-softmax; not used of an ended row
    __shared__ double lse[kMaxBeams];
    __shared__ float rowmax[kMaxBeams];
    __shared__ Candidate list[kList];
    __shared__ Candidate wbest[kWarps];
    __shared__ int count;
    if (tid == 0) count = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int r = warp; r < beams; r += kWarps) {
        double out = NAN;
        float m = -INFINITY;
        if (!(ended && ended[row0 + r]) && isfinite(running[row0 + r])) {
            const Slice* p = part + size_t(row0 + r) * slices;
            bool nan = false;
            for (int i = lane; i < slices; i += 32) {
                const float x = p[i].max;
                nan |= x != x;
                m = fmaxf(m, x);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            nan = __any_sync(~0u, nan);
            if (!nan && isfinite(m)) {
                double s = 0.0;
                for (int i = lane; i < slices; i += 32)
                    if (p[i].sum > 0.0) s += p[i].sum * exp(double(p[i].max) - double(m));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
                out = log(s);
            }
        }
        if (lane == 0) {
            lse[r] = out;
            rowmax[r] = m;
        }
    }
    __syncthreads();
    const int per = max(slices * n, n + 1), total = beams * per;
    auto candidate = [&](int i) -> Candidate {
        const int r = i / per, j = i % per;
        const Candidate none{-INFINITY, 0x7FFFFFFFFFFFFFFFll};
        if (ended && ended[row0 + r]) {
            const float run = running[row0 + r];
            if (j == 0 && unsigned(pad_token) < unsigned(V))
                return {isfinite(run) ? double(run) : -INFINITY, (long long)r * V + pad_token};
            const int t = j - 1;
            if (j == 0 || t >= min(n, V) || t == pad_token) return none;
            return {-INFINITY, (long long)r * V + t};
        }
        if (lse[r] != lse[r]) {
            if (j >= min(n, V)) return none;
            return {-INFINITY, (long long)r * V + j};
        }
        if (j >= slices * n) return none;
        const unsigned long long k = best[size_t(row0 + r) * slices * n + j];
        if (k == 0) return none;
        const double x = double(unordered(uint32_t(k >> 32)));
        return {double(running[row0 + r]) + ((x - double(rowmax[r])) - lse[r]),
                (long long)r * V + place_of(k)};
    };
    auto write = [&](int rank, const Candidate& c) {
        scores[size_t(b) * n + rank] = float(c.score);
        parents[size_t(b) * n + rank] = row0 + int(c.place / V);
        tokens[size_t(b) * n + rank] = int(c.place % V);
    };
    // as in the slices: a bound that n candidates reach, the list of those that reach it, ranks
    double m = -INFINITY;
    for (int i = tid; i < total; i += kThreads) m = fmax(m, candidate(i).score);
    double low = m;
    for (int r = (n + kWarps - 1) / kWarps;; --r) {
        low = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) low = fmax(low, __shfl_xor_sync(~0u, low, o));
        if (r == 1) break;
        const uint32_t who = __ballot_sync(~0u, m == low);
        if (lane == __ffs(who) - 1) m = -INFINITY;
    }
    if (lane == 0) wbest[warp].score = low;
    __syncthreads();
    double bound = wbest[0].score;
    for (int w = 1; w < kWarps; ++w) bound = fmin(bound, wbest[w].score);
    for (int i = tid; i < total; i += kThreads) {
        const Candidate c = candidate(i);
        if (c.score >= bound && c.place != 0x7FFFFFFFFFFFFFFFll) {
            const int at = atomicAdd(&count, 1);
            if (at < kList) list[at] = c;
        }
    }
    __syncthreads();
    const int found = count;
    if (found <= kList) {
        for (int i = tid; i < found; i += kThreads) {
            const Candidate c = list[i];
            int rank = 0;
            for (int j = 0; j < found; ++j) rank += better(list[j], c);
            if (rank < n) write(rank, c);
        }
        return;
    }
    Candidate last{INFINITY, -1};
    for (int r = 0; r < n; ++r) {
        Candidate k{-INFINITY, 0x7FFFFFFFFFFFFFFFll};
        for (int i = tid; i < total; i += kThreads) {
            const Candidate c = candidate(i);
            if (better(last, c) && better(c, k)) k = c;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const Candidate c{__shfl_xor_sync(~0u, k.score, o), __shfl_xor_sync(~0u, k.place, o)};
            if (better(c, k)) k = c;
        }
        if (lane == 0) wbest[warp] = k;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w)
            if (better(wbest[w], k)) k = wbest[w];
        __syncthreads();
        if (tid == 0) write(r, k);
        last = k;
    }
}

// ------------------------------------------------------------------------------------------
// dst row i = src row parents[i], rows of `units` 16-byte words (a multiple of kCopy * 256 in
// none of the uses: the last block of a row checks).  Block (part of a row, i).
// ------------------------------------------------------------------------------------------
constexpr int kCopy = 8;  // words in flight per thread

__global__ void __launch_bounds__(kThreads) gather_rows_kernel(const uint4* __restrict__ src,
                                                               int src_rows,
                                                               const int32_t* __restrict__ parents,
                                                               uint4* __restrict__ dst, int units)
{
    const int i = blockIdx.y;
    int from = parents[i];
    if (from < 0 || from >= src_rows) {
        if (threadIdx.x == 0) raise_error(OAL_ERR_VALUE);
        from = from < 0 ? 0 : src_rows - 1;
    }
    const uint4* s = src + size_t(from) * units;
    uint4* d = dst + size_t(i) * units;
    const int at = blockIdx.x * (kCopy * kThreads) + threadIdx.x;
    uint4 w[kCopy];
#pragma unroll
    for (int x = 0; x < kCopy; ++x)
        if (at + x * kThreads < units) w[x] = s[at + x * kThreads];
#pragma unroll
    for (int x = 0; x < kCopy; ++x)
        if (at + x * kThreads < units) __stcs(d + at + x * kThreads, w[x]);
}

// The header (with the batch size of dst) and the coefficient tables of a state.
__global__ void __launch_bounds__(kThreads) copy_head_kernel(const uint4* __restrict__ src,
                                                             uint4* __restrict__ dst, int units,
                                                             int B)
{
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < units; i += gridDim.x * kThreads) {
        uint4 w = src[i];
        if (i == 0) w.z = uint32_t(B);  // StateHeader::B
        dst[i] = w;
    }
}
static_assert(offsetof(StateHeader, B) == 8, "the batch size is the header's third word");

int gather_rows(const void* src, int src_rows, const int32_t* parents, void* dst, int rows,
                size_t row_bytes, cudaStream_t st)
{
    const int units = int(row_bytes / 16);
    const int per = kCopy * kThreads;
    LaunchScope ls("gather_rows", st);
    gather_rows_kernel<<<dim3((units + per - 1) / per, rows), kThreads, 0, st>>>(
        static_cast<const uint4*>(src), src_rows, parents, static_cast<uint4*>(dst), units);
    OAL_LAUNCH_CHECK();
    return OAL_OK;
}

// Slices of a row, given the logits per thread; a misaligned row needs up to a vector more.
int slices_of(int dtype, int V, int each)
{
    const int per = each * kThreads, skew = (dtype == OAL_BF16 ? 8 : 4) - 1;
    return (V + skew + per - 1) / per;
}

// Logits per thread: 32 when that still gives every SM two blocks, else 8 (more, smaller
// slices, so that one search's rows reach more SMs).
int logits_per_thread(int dtype, int rows, int V)
{
    return (long long)rows * slices_of(dtype, V, 32) >= 2 * sm_count() ? 32 : 8;
}

int check_select(int B, int beams, int V, int n, int dtype)
{
    if (B < 0 || beams < 1 || V < 1 || n < 1) return OAL_ERR_SHAPE;
    if (dtype != OAL_F32 && dtype != OAL_BF16) return OAL_ERR_UNSUPPORTED;
    if (n > kMaxSelect || beams > kMaxBeams) return OAL_ERR_UNSUPPORTED;
    if ((long long)n > (long long)beams * V || (long long)beams * V >= (1LL << 31) - 64 ||
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
    constexpr int dtype = sizeof(T) == 2 ? OAL_BF16 : OAL_F32;
    const int rows = B * beams, each = logits_per_thread(dtype, rows, V);
    const int slices = slices_of(dtype, V, each);
    Slice* part = static_cast<Slice*>(ws);
    unsigned long long* best = reinterpret_cast<unsigned long long*>(
        static_cast<unsigned char*>(ws) + align256(size_t(rows) * slices * sizeof(Slice)));
    {
        LaunchScope ls("select_slice", st);
        auto go = [&](auto kern) {
            kern<<<dim3(slices, rows), kThreads, 0, st>>>(static_cast<const T*>(logits), ld, rows,
                                                          V, n, running, ended, best, part);
        };
        if (each == 32) go(select_slice_kernel<T, 32 / VecOf<T>::n>);
        else go(select_slice_kernel<T, 8 / VecOf<T>::n>);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    LaunchScope ls("select_merge", st);
    return launch_ex(select_merge_kernel, dim3(B), dim3(kThreads), 0, st, true,
                     static_cast<const unsigned long long*>(best), static_cast<const Slice*>(part),
                     beams, V, n, slices, running, ended, pad_token, scores, parents, tokens);
}

int check_reorder(const void* src, int src_B, const int32_t* parents, const void* dst,
                  const oal_shape* s)
{
    int rc = check_common(s);
    if (rc) return rc;
    oal_shape from = *s;
    from.B = src_B;
    if (src_B < 1) return OAL_ERR_SHAPE;
    if ((rc = check_common(&from)) || (rc = check_planes(s->B))) return rc;
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
    // the most slices that any launch of these sizes takes
    const size_t parts = size_t(B) * beams * beam::slices_of(dtype, V, 8);
    *bytes = std::max<size_t>(align256(parts * sizeof(beam::Slice)) + parts * n * 8, 256);
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
    if (overlap(src, state_bytes(src_B, s->Hq, s->Hkv), dst,
                      state_bytes(s->B, s->Hq, s->Hkv)))
        return OAL_ERR_OVERLAP;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t head = kHeaderBytes + coef_bytes(s->Hq);
    {
        LaunchScope ls("copy_state_head", st);
        beam::copy_head_kernel<<<int((head / 16 + beam::kThreads - 1) / beam::kThreads),
                                 beam::kThreads, 0, st>>>(
            static_cast<const uint4*>(src), static_cast<uint4*>(dst), int(head / 16), s->B);
        OAL_LAUNCH_CHECK();
    }
    if (s->B == 0) return OAL_OK;
    return beam::gather_rows(static_cast<const unsigned char*>(src) + head, src_B, parents,
                             static_cast<unsigned char*>(dst) + head, s->B,
                             size_t(s->Hkv) * state_unit_bytes(), st);
}

int oal_decay_state_reorder(const float* src, int src_B, const int32_t* parents, float* dst,
                            const oal_shape* s, void* stream)
{
    int rc = beam::check_reorder(src, src_B, parents, dst, s);
    if (rc) return rc;
    const size_t row = size_t(s->Hkv) * kD * kDV * 4;
    if (overlap(src, src_B * row, dst, s->B * row)) return OAL_ERR_OVERLAP;
    if (s->B == 0) return OAL_OK;
    return beam::gather_rows(src, src_B, parents, dst, s->B, row,
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
    if (overlap(src, state_bytes(src_B, s->Hq, s->Hkv), dst,
                      state_bytes(s->B, s->Hq, s->Hkv)))
        return OAL_ERR_OVERLAP;
    return launch_decode(q, k, v, dst, out,
                         reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                                  decode_ticket_bytes(s)),
                         s->B, s->Hq, s->Hkv, s->dtype, static_cast<cudaStream_t>(stream), src,
                         src_B, parents);
}

}  // extern "C"
