// oal_decay.cu -- linear attention with a decay per key/value head: the scan over chunks, the
// single-token step, the fp32 kernels of the other parts, and the entry points.
#pragma once

#include "oal_common.cuh"
#include "oal_decay.cuh"
#include "oal_decay_tc.cuh"
#include "oal_kernels.cuh"

namespace oal {
namespace decay {

constexpr int kC = 64;          // tokens per chunk of the fp32 kernels
constexpr int kThreads = 256;
constexpr int kLd = kD + 4;     // padded row: 16-byte reads of 8 consecutive rows touch all banks

// Starts copying rows [t0, t0 + n) of head plane `src` into a [64][kLd] tile; zeros from row n on.
__device__ __forceinline__ void fetch_tile(float (*dst)[kLd], const float* src, int t0, int n)
{
#pragma unroll
    for (int i = 0; i < kC * kD / 4 / kThreads; ++i) {
        const int e = i * kThreads + threadIdx.x, r = e / (kD / 4), c = 4 * (e % (kD / 4));
        const float* from = src + size_t(t0 + min(r, n - 1)) * kD + c;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(&dst[r][c])),
                     "l"(from), "r"(r < n ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void fetch_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void fetch_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ float2 lo2(float4 v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi2(float4 v) { return make_float2(v.z, v.w); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// ------------------------------------------------------------------------------------------
// E_c of one (chunk, kv, b): a 64 x 64 product over the chunk's tokens, for every y head of the
// kv head.  Thread (ty, tx) owns rows 4 ty .. + 3 and columns 4 tx .. + 3, in pairs of columns
// (packed fp32 FMAs); the next head's tiles arrive while one is worked on.  The heads of a group are
// summed in parts, a block each, where there are few chunks: the gradient of 4096 tokens of 14/2 heads
// (1024 products of 64^3) takes 24 us, 22 TFLOP/s, and took 36 us with a group per block; 61 us on
// single FMAs with tiles loaded in turn.
// ------------------------------------------------------------------------------------------
struct DeltaSmem {
    float Y[2][kC][kLd], Z[2][kC][kLd];
    float w[kC];
};

__global__ void __launch_bounds__(kThreads) delta_simt_kernel(DecayShape S, DecaySum a, DecaySum b2)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    DeltaSmem& sm = *reinterpret_cast<DeltaSmem*>(smem_raw);
    // the first sum, then the parts of the second (the first has one)
    const DecaySum& J = blockIdx.z ? b2 : a;
    const int part = blockIdx.z ? blockIdx.z - 1 : 0;
    const int c = blockIdx.x, bkv = blockIdx.y, b = bkv / S.Hkv, kv = bkv % S.Hkv;
    tc::grid_dep_launch();
    const int n = min(kC, decay_len(S, b) - c * kC);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    if (n <= 0) {  // the scan does not read it
        if (S.chunks == 1)
            for (int i = 0; i < 4; ++i)
                scan_one<float>(J, bkv, (4 * ty + i) * kDV + 4 * tx, 1.f,
                                make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }
    const int grp = J.hy / S.Hkv, per = (grp + J.parts - 1) / J.parts;
    const int h0 = part * per, nh = min(per, grp - h0);
    const size_t plane = (size_t(b) * J.hy + kv * grp + h0) * S.T * kD, next = size_t(S.T) * kD;
    auto fetch = [&](int h) {
        fetch_tile(sm.Y[h & 1], static_cast<const float*>(J.y) + plane + h * next, c * kC, n);
        fetch_tile(sm.Z[h & 1], static_cast<const float*>(J.z) + plane + h * next, c * kC, n);
        fetch_end();
    };
    fetch(0);
    const float g = decay_log(S.log_decay, kv);
    if (threadIdx.x < kC)
        sm.w[threadIdx.x] = J.rev ? S.scale * decay_pow(g, threadIdx.x + 1)
                                  : decay_pow(g, max(0, n - 1 - int(threadIdx.x)));
    float2 acc[4][2] = {};
    for (int h = 0; h < nh; ++h) {
        if (h + 1 < nh) {
            fetch(h + 1);
            fetch_wait<1>();
        } else {
            fetch_wait<0>();
        }
        __syncthreads();
        const float (*Y)[kLd] = sm.Y[h & 1];
        const float (*Z)[kLd] = sm.Z[h & 1];
#pragma unroll 4
        for (int j = 0; j < kC; ++j) {
            const float w = sm.w[j];
            const float4 y = *reinterpret_cast<const float4*>(&Y[j][4 * ty]);
            const float4 z = *reinterpret_cast<const float4*>(&Z[j][4 * tx]);
            const float yv[4] = {y.x * w, y.y * w, y.z * w, y.w * w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i][0] = __ffma2_rn(both(yv[i]), lo2(z), acc[i][0]);
                acc[i][1] = __ffma2_rn(both(yv[i]), hi2(z), acc[i][1]);
            }
        }
        __syncthreads();
    }
    float* out = J.delta + ((size_t(part) * S.B * S.Hkv + bkv) * S.chunks + c) * kDecayState;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = (4 * ty + i) * kDV + 4 * tx;
        const float4 sum = make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
        if (S.chunks > 1) *reinterpret_cast<float4*>(out + e) = sum;
        else scan_one<float>(J, bkv, e, decay_pow(g, n), sum);
    }
}

// ------------------------------------------------------------------------------------------
// The scan over the chunks of every (b, kv): cur <- l^n cur + E_c, cur written before each.
// Block = 32 kVec state entries (kVec per lane) and up to 64 chunks at a time, 8 per warp: a warp
// sums its chunks by themselves, all of them loaded at once, then starts over from what the warps
// before it leave.  One round trip to memory for 64 chunks instead of 64, and bound by it until
// there are many planes: 64 planes of 64 chunks (100 MB) in 27 us, 3.7 TB/s.  kVec = 2 gives
// twice the blocks of kVec = 4, which pays where there are few planes: both directions of 2 planes
// of 32 chunks 8.6 us against 10.0 (one direction 6.7 against 6.9); 16 planes 12.8 against 10.7 and
// 64 planes 31.9 against 27.7 are the other way round.
// ------------------------------------------------------------------------------------------
constexpr int kScanRun = 8;

template <int kVec> struct Entries {
    float v[kVec];
};
template <int kVec>
__device__ __forceinline__ Entries<kVec> load_entries(const float* p)
{
    Entries<kVec> e;
    if constexpr (kVec == 4)
        *reinterpret_cast<float4*>(e.v) = *reinterpret_cast<const float4*>(p);
    else
        *reinterpret_cast<float2*>(e.v) = *reinterpret_cast<const float2*>(p);
    return e;
}
__device__ __forceinline__ void store_entries(float* p, const Entries<2>& e)
{
    *reinterpret_cast<float2*>(p) = make_float2(e.v[0], e.v[1]);
}
__device__ __forceinline__ void store_entries(__nv_bfloat16* p, const Entries<2>& e)
{
    *reinterpret_cast<uint32_t*>(p) = tc::pack_bf16x2(e.v[0], e.v[1]);
}
template <typename Tm>
__device__ __forceinline__ void store_entries(Tm* p, const Entries<4>& e)
{
    store_state(p, make_float4(e.v[0], e.v[1], e.v[2], e.v[3]));
}
template <int kVec>
__device__ __forceinline__ void fma_decay(float l, Entries<kVec>& cur, const Entries<kVec>& d)
{
#pragma unroll
    for (int x = 0; x < kVec; ++x) cur.v[x] = fmaf(l, cur.v[x], d.v[x]);
}

template <typename Tm, int kVec>
__global__ void __launch_bounds__(kThreads) scan_kernel(DecayShape S, DecaySum a, DecaySum b2,
                                                        int chunk)
{
    const DecaySum& J = blockIdx.z ? b2 : a;
    const int bkv = blockIdx.y, b = bkv / S.Hkv, kv = bkv % S.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = (blockIdx.x * 32 + lane) * kVec;
    __shared__ Entries<kVec> tot[8][32];
    __shared__ float pw[8];
    tc::grid_dep_launch();
    const int len = decay_len(S, b);
    const int nc = (len + chunk - 1) / chunk, tail = len - (nc - 1) * chunk;
    const float g = decay_log(S.log_decay, kv);
    const float l_full = decay_pow(g, chunk), l_tail = decay_pow(g, tail);
    const size_t plane = (size_t(bkv) * S.chunks) * kDecayState + e;
    const size_t part = size_t(S.B) * S.Hkv * S.chunks * kDecayState;
    const int run = min(kScanRun, (nc + 7) / 8);  // chunks per warp at a time
    tc::grid_dep_wait();
    Entries<kVec> cur{};
    if (J.first) cur = load_entries<kVec>(J.first + size_t(bkv) * kDecayState + e);
    for (int base = 0; base < nc; base += 8 * run) {
        const int i0 = base + warp * run, cnt = max(0, min(run, nc - i0));
        auto chunk_at = [&](int i) { return J.rev ? nc - 1 - (i0 + i) : i0 + i; };
        auto decay_at = [&](int i) { return chunk_at(i) == nc - 1 ? l_tail : l_full; };
        Entries<kVec> d[kScanRun];
#pragma unroll
        for (int i = 0; i < kScanRun; ++i)
            if (i < cnt) d[i] = load_entries<kVec>(J.delta + plane + size_t(chunk_at(i)) * kDecayState);
        for (int p = 1; p < J.parts; ++p) {
#pragma unroll
            for (int i = 0; i < kScanRun; ++i)
                if (i < cnt) {
                    const Entries<kVec> x = load_entries<kVec>(J.delta + p * part + plane +
                                                               size_t(chunk_at(i)) * kDecayState);
                    fma_decay(1.f, d[i], x);
                }
        }
        Entries<kVec> sum{};
        int tokens = 0;
#pragma unroll
        for (int i = 0; i < kScanRun; ++i)
            if (i < cnt) {
                fma_decay(decay_at(i), sum, d[i]);
                tokens += chunk_at(i) == nc - 1 ? tail : chunk;
            }
        tot[warp][lane] = sum;
        if (lane == 0) pw[warp] = decay_pow(g, tokens);
        __syncthreads();
        Entries<kVec> mine = cur;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w == warp) mine = cur;
            fma_decay(pw[w], cur, tot[w][lane]);
        }
#pragma unroll
        for (int i = 0; i < kScanRun; ++i)
            if (i < cnt) {
                store_entries(static_cast<Tm*>(J.mem) + plane + size_t(chunk_at(i)) * kDecayState, mine);
                fma_decay(decay_at(i), mine, d[i]);
            }
        __syncthreads();
    }
    if (J.last && warp == 0) store_entries(J.last + size_t(bkv) * kDecayState + e, cur);
}

// ------------------------------------------------------------------------------------------
// The mix of one (chunk, x head, b).  Thread (ty, tx) owns rows 4 ty .. + 3; of products of rows
// (x . y) the columns tx + 16 e (conflict-free reads of y rows), of the output the columns
// 4 tx .. + 3.  Packed fp32 FMAs; tiles arrive while others are worked on.  Of the products beyond
// the diagonal each warp forms and uses those of its own rows' block alone.  Bound by the CUDA
// cores, not by memory: 4096 tokens of 14/2 heads take 41 us (34 MB, 5 us of memory; 25 TFLOP/s of the
// products formed), 49 us with the whole square, 75 us on single FMAs with tiles loaded in turn.
// M in Y's place, for three blocks per SM, was slower where there are few items (2 x 1001 tokens of
// 8 heads: a call of 28.8 us against 24.7).
// ------------------------------------------------------------------------------------------
struct MixSmem {
    float X[kC][kLd], Y[kC][kLd], Z[kC][kLd], M[kC][kLd], P[kC][kLd];
    float pw[kC + 1];  // powers of l
};

// s[i][e] = A[4 ty + i] . B[tx + 16 e], e < kE
template <int kE>
__device__ __forceinline__ void row_products(const float (*A)[kLd], const float (*B)[kLd],
                                             float (&s)[4][kE])
{
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    float2 acc[4][kE] = {};
#pragma unroll 4
    for (int k = 0; k < kD; k += 4) {
        float4 a[4], b[kE];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(&A[4 * ty + i][k]);
#pragma unroll
        for (int e = 0; e < kE; ++e) b[e] = *reinterpret_cast<const float4*>(&B[tx + 16 * e][k]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                acc[i][e] = __ffma2_rn(lo2(a[i]), lo2(b[e]), acc[i][e]);
                acc[i][e] = __ffma2_rn(hi2(a[i]), hi2(b[e]), acc[i][e]);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < kE; ++e) s[i][e] = acc[i][e].x + acc[i][e].y;
}

// Columns 16 e0 .. + 16 kE - 1 of P = (X Y^T) o D: all that a warp's rows read of it.
template <int kE>
__device__ __forceinline__ void decayed_scores(MixSmem& sm, int e0, int rev)
{
    const int ty = threadIdx.x >> 4, col0 = 16 * e0 + (threadIdx.x & 15);
    float s[4][kE];
    row_products<kE>(sm.X, sm.Y + 16 * e0, s);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const int row = 4 * ty + i, col = col0 + 16 * e;
            const int d = rev ? col - row : row - col;
            sm.P[row][col] = d >= 0 ? s[i][e] * sm.pw[d] : 0.f;
        }
}

// acc[i] += row 4 ty + i of A times B, columns 4 tx .. + 3, over k0 <= k < k1 (multiples of 4)
__device__ __forceinline__ void add_product(const float (*A)[kLd], const float (*B)[kLd],
                                            float2 (&acc)[4][2], int k0 = 0, int k1 = kC)
{
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 4
    for (int k = k0; k < k1; k += 4) {
        float4 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(&A[4 * ty + i][k]);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const float4 b = *reinterpret_cast<const float4*>(&B[k + kk][4 * tx]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = kk == 0 ? a[i].x : kk == 1 ? a[i].y : kk == 2 ? a[i].z : a[i].w;
                acc[i][0] = __ffma2_rn(both(v), lo2(b), acc[i][0]);
                acc[i][1] = __ffma2_rn(both(v), hi2(b), acc[i][1]);
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads, 2) mix_simt_kernel(DecayShape S, DecayJob j0, DecayJob j1,
                                                               DecayJob j2)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    MixSmem& sm = *reinterpret_cast<MixSmem*>(smem_raw);
    const DecayJob& J = blockIdx.z == 0 ? j0 : blockIdx.z == 1 ? j1 : j2;
    const int c = blockIdx.x, b = blockIdx.y / J.hx, hx = blockIdx.y % J.hx;
    // the jobs share a grid of the largest head count
    const int n = b < S.B ? min(kC, decay_len(S, b) - c * kC) : 0;
    if (n <= 0) {
        tc::grid_dep_wait();  // as every block does: the kernel ends after the ones before it
        return;
    }
    const int kv = hx * S.Hkv / J.hx;
    const int nh = J.hy > J.hx ? J.hy / J.hx : 1;
    const int y0 = J.hy > J.hx ? hx * nh : hx * J.hy / J.hx;
    const size_t next = size_t(S.T) * kD, plane = (size_t(b) * J.hy + y0) * next;
    const float* y = static_cast<const float*>(J.y) + plane;
    const float* z = static_cast<const float*>(J.z) + plane;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    // the inputs were there before the kernels whose results this one waits for
    fetch_tile(sm.X, static_cast<const float*>(J.x) + (size_t(b) * J.hx + hx) * next, c * kC, n);
    fetch_tile(sm.Y, y, c * kC, n);
    fetch_end();
    fetch_tile(sm.Z, z, c * kC, n);
    const float g = decay_log(S.log_decay, kv);
    if (threadIdx.x <= kC) sm.pw[threadIdx.x] = decay_pow(g, threadIdx.x);
    tc::grid_dep_wait();
    fetch_tile(sm.M,
               static_cast<const float*>(J.mem) + ((size_t(b) * S.Hkv + kv) * S.chunks + c) * kDecayState,
               0, kC);
    fetch_end();
    fetch_wait<1>();
    __syncthreads();
    // a warp's eight rows and the keys on their side of the diagonal
    const int r8 = 8 * (threadIdx.x >> 5), k0 = J.rev ? r8 : 0, k1 = J.rev ? kC : r8 + 8;
    float2 near[4][2] = {};
    for (int h = 0; h < nh; ++h) {
        // blocks of 16 keys: the diagonal's and those on its side
        const int at = threadIdx.x >> 6, e0 = J.rev ? at : 0;
        switch (J.rev ? 4 - at : at + 1) {
        case 1: decayed_scores<1>(sm, e0, J.rev); break;
        case 2: decayed_scores<2>(sm, e0, J.rev); break;
        case 3: decayed_scores<3>(sm, e0, J.rev); break;
        default: decayed_scores<4>(sm, e0, J.rev);
        }
        fetch_wait<0>();
        __syncthreads();  // P and Z (and M) are there, Y is free
        if (h + 1 < nh) {
            fetch_tile(sm.Y, y + (h + 1) * next, c * kC, n);
            fetch_end();
        }
        add_product(sm.P, sm.Z, near, k0, k1);
        if (h + 1 < nh) {
            fetch_wait<0>();
            __syncthreads();  // the next Y is there, Z and P are free
            fetch_tile(sm.Z, z + (h + 1) * next, c * kC, n);
            fetch_end();
        }
    }
    float2 far[4][2] = {};
    if (J.mem_t) {
        float s[4][4];
        row_products<4>(sm.X, sm.M, s);
        __syncthreads();  // P is free
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sm.P[4 * ty + i][tx + 16 * e] = s[i][e];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(&sm.P[4 * ty + i][4 * tx]);
            far[i][0] = lo2(v);
            far[i][1] = hi2(v);
        }
    } else {
        add_product(sm.X, sm.M, far);
    }
    float* out = static_cast<float*>(J.out) + ((size_t(b) * J.hx + hx) * S.T + c * kC) * kD;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 4 * ty + i;
        if (row >= n) continue;
        const float bi = J.rev ? sm.pw[n - 1 - row] : S.scale * sm.pw[row + 1];
        *reinterpret_cast<float4*>(out + size_t(row) * kD + 4 * tx) = make_float4(
            fmaf(S.scale, near[i][0].x, bi * far[i][0].x), fmaf(S.scale, near[i][0].y, bi * far[i][0].y),
            fmaf(S.scale, near[i][1].x, bi * far[i][1].x), fmaf(S.scale, near[i][1].y, bi * far[i][1].y));
    }
}

// ------------------------------------------------------------------------------------------
// One token: block = (kv, b).  Thread (r0, c4) holds rows r0 + 16 i of the columns 4 c4 .. + 3.  The
// state passes through registers once, all of it requested before anything is computed:
// memory-bound, 1024 sequences of 16 heads (545 MB) in 84 to 86 us a call, 6.3 to 6.5 TB/s.  64 sequences of 2 heads
// take 6 us, less than the host's call (10 us).
// ------------------------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads) step_kernel(const T* __restrict__ q,
                                                        const T* __restrict__ k,
                                                        const T* __restrict__ v,
                                                        const float* __restrict__ log_decay,
                                                        float scale, const float* src,
                                                        const int32_t* __restrict__ parents,
                                                        int src_B, float* state,
                                                        T* __restrict__ out, int Hq, int Hkv)
{
    const int b = blockIdx.x / Hkv, kv = blockIdx.x % Hkv, grp = Hq / Hkv;
    __shared__ float qs[kMaxGroup][kD], ks[kD];
    __shared__ __align__(16) float red[8][kMaxGroup][kDV];
    const int tid = threadIdx.x, c4 = tid & 15, r0 = tid >> 4, warp = tid >> 5;
    int from = b;
    if (parents) {
        from = parents[b];
        if (from < 0 || from >= src_B) {
            if (tid == 0) raise_error(OAL_ERR_VALUE);
            from = from < 0 ? 0 : src_B - 1;
        }
    }
    const float4* in = reinterpret_cast<const float4*>(src + (size_t(from) * Hkv + kv) * kDecayState);
    float4 s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = in[(r0 + 16 * i) * (kDV / 4) + c4];
    for (int e = tid; e < grp * kD; e += kThreads)
        qs[e / kD][e % kD] = to_f32(q[(size_t(b) * Hq + kv * grp) * kD + e]);
    if (tid < kD) ks[tid] = to_f32(k[(size_t(b) * Hkv + kv) * kD + tid]);
    const T* vp = v + (size_t(b) * Hkv + kv) * kDV + 4 * c4;
    const float4 v4 = make_float4(to_f32(vp[0]), to_f32(vp[1]), to_f32(vp[2]), to_f32(vp[3]));
    const float l = expf(decay_log(log_decay, kv));
    __syncthreads();
    float4* dst = reinterpret_cast<float4*>(state + (size_t(b) * Hkv + kv) * kDecayState);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float kr = ks[r0 + 16 * i];
        s[i] = make_float4(fmaf(l, s[i].x, kr * v4.x), fmaf(l, s[i].y, kr * v4.y),
                           fmaf(l, s[i].z, kr * v4.z), fmaf(l, s[i].w, kr * v4.w));
        dst[(r0 + 16 * i) * (kDV / 4) + c4] = s[i];
    }
    for (int h = 0; h < grp; ++h) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float w = qs[h][r0 + 16 * i];
            o = make_float4(fmaf(w, s[i].x, o.x), fmaf(w, s[i].y, o.y), fmaf(w, s[i].z, o.z),
                            fmaf(w, s[i].w, o.w));
        }
        o.x += __shfl_xor_sync(~0u, o.x, 16);
        o.y += __shfl_xor_sync(~0u, o.y, 16);
        o.z += __shfl_xor_sync(~0u, o.z, 16);
        o.w += __shfl_xor_sync(~0u, o.w, 16);
        if ((tid & 31) < 16) *reinterpret_cast<float4*>(&red[warp][h][4 * c4]) = o;
    }
    __syncthreads();
    for (int e = tid; e < grp * kDV; e += kThreads) {
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) o += red[w][e / kDV][e % kDV];
        out[(size_t(b) * Hq + kv * grp) * kDV + e] = T(scale * o);
    }
}

// ---- host ----------------------------------------------------------------------------------
bool on_tensor_cores(const oal_shape* s) { return s->dtype == OAL_BF16; }

int chunk_of(const oal_shape* s) { return on_tensor_cores(s) ? dtc::kC : kC; }

int chunks_of(const oal_shape* s) { return int((s->T + (long long)chunk_of(s) - 1) / chunk_of(s)); }

template <typename F>
int by_type(int dtype, F f)
{
    return dtype == OAL_BF16 ? f(__nv_bfloat16{}) : f(float{});
}

// Parts in which the heads of a group are summed (the gradient's R): enough CTAs for two per SM
// where the chunks alone are too few, at the price of a 16 KB partial sum each.  The gradient of 4096
// tokens of 14/2 heads: 34.9 us with two per SM, 37.0 with three; in fp32 119 us, 131 without parts.
// (The workspace's size follows from it, so it counts the SMs of the chip the library is built for, not
// those of the device that is current when the size is asked for.)
constexpr int kSms = 148;
int parts_of(const oal_shape* s, int grp)
{
    const long long items = (long long)s->B * s->Hkv * chunks_of(s);
    if (chunks_of(s) <= 1 || s->B == 0) return 1;
    const int parts = int(std::min<long long>(grp, (2 * kSms + items - 1) / items));
    const int per = (grp + parts - 1) / parts;
    return (grp + per - 1) / per;  // none of them empty
}

// Workspace of one sum: the chunks' products, and (bf16) the images of the states before them.
struct SumLayout {
    size_t delta, mem, total;
};
SumLayout sum_layout(const oal_shape* s, int parts)
{
    const size_t states = size_t(s->B) * s->Hkv * chunks_of(s);
    const size_t one = align256(states * kDecayState * 4);
    SumLayout l{0, 0, one * parts};
    if (on_tensor_cores(s)) {
        l.mem = one * parts;
        l.total += align256(states * kDecayState * 2);
    }
    return l;
}

DecaySum make_sum(const void* y, const void* z, int hy, int rev, int parts, unsigned char* ws,
                  const oal_shape* s, const float* first, float* last)
{
    const SumLayout l = sum_layout(s, parts);
    return {y, z, hy, rev, parts, reinterpret_cast<float*>(ws + l.delta), ws + l.mem, first, last};
}

cudaError_t set_attributes_once()
{
    constexpr int kMaxDev = 64;
    static std::atomic<int> done[kMaxDev] = {};
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDev && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const std::pair<const void*, int> smem[] = {
        {reinterpret_cast<const void*>(dtc::delta_kernel), int(dtc::kDeltaSmem)},
        {reinterpret_cast<const void*>(dtc::mix_kernel), int(dtc::kMixSmem)},
        {reinterpret_cast<const void*>(delta_simt_kernel), int(sizeof(DeltaSmem))},
        {reinterpret_cast<const void*>(mix_simt_kernel), int(sizeof(MixSmem))}};
    for (const auto& k : smem) {
        if ((e = cudaFuncSetAttribute(k.first, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      k.second)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(k.first, cudaFuncAttributePreferredSharedMemoryCarveout,
                                      100)) != cudaSuccess)
            return e;
    }
    if (dev >= 0 && dev < kMaxDev) done[dev].store(1, std::memory_order_release);
    return cudaSuccess;
}

// [heads][T][64] bf16 for copies out of 32 rows by 32 columns (what a warp has)
bool make_out_map(CUtensorMap* m, const void* base, int T, int heads)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {64, cuuint64_t(T), cuuint64_t(heads)};
    const cuuint64_t strides[2] = {64 * 2, cuuint64_t(T) * 64 * 2};
    const cuuint32_t box[3] = {32, 32, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [planes][64] bf16 state images of 64 rows each, as 2D {64, planes * 64}
bool make_state_map(CUtensorMap* m, const void* base, size_t planes)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {64, cuuint64_t(planes) * 64};
    const cuuint64_t strides[1] = {128};
    const cuuint32_t box[2] = {64, 64};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The sums of `n` directions (1 or 2) and their scans.  (A sequence of one chunk needs no scan.)
int launch_sums(const DecayShape& S, const DecaySum* a, int n, const oal_shape* s, cudaStream_t st)
{
    const DecaySum& b2 = a[n - 1];
    const int planes = s->B * s->Hkv;
    if (S.chunks > 0) {
        LaunchScope ls("decay_delta", st);
        if (on_tensor_cores(s)) {
            dtc::SumMaps maps;
            int items = 0;
            for (int i = 0; i < n; ++i) {
                const DecaySum& j = a[i];
                if (!make_map_uncached(&maps.y[i], j.y, s->T, s->B * j.hy) ||
                    !make_map_uncached(&maps.z[i], j.z, s->T, s->B * j.hy))
                    return OAL_ERR_CUDA;
                items += j.parts * planes * S.chunks;
            }
            dtc::delta_kernel<<<items, dtc::kThreads, dtc::kDeltaSmem, st>>>(maps, S, a[0], b2);
        } else {
            delta_simt_kernel<<<dim3(S.chunks, planes, n == 1 ? 1 : 1 + b2.parts), kThreads,
                                sizeof(DeltaSmem), st>>>(S, a[0], b2);
        }
        OAL_LAUNCH_CHECK();
    }
    if (S.chunks == 1) return OAL_OK;  // there is nothing to scan
    LaunchScope ls("decay_scan", st);
    const bool wide = n * planes >= 8;
    const auto scan = on_tensor_cores(s) ? (wide ? scan_kernel<__nv_bfloat16, 4> : scan_kernel<__nv_bfloat16, 2>)
                                         : (wide ? scan_kernel<float, 4> : scan_kernel<float, 2>);
    OAL_CUDA_TRY(launch_ex(scan, dim3(kDecayState / (wide ? 128 : 64), planes, n), dim3(kThreads), 0, st,
                           S.chunks > 0, S, a[0], b2, chunk_of(s)));
    return OAL_OK;
}

int launch_mix(const DecayShape& S, const DecayJob* j, const DecaySum* const* sums, int n,
               const oal_shape* s, cudaStream_t st)
{
    if (S.chunks == 0) return OAL_OK;
    LaunchScope ls("decay_mix", st);
    if (!on_tensor_cores(s)) {
        int hx = 0;
        for (int i = 0; i < n; ++i) hx = std::max(hx, j[i].hx);
        OAL_CUDA_TRY(launch_ex(mix_simt_kernel, dim3(S.chunks, s->B * hx, n), dim3(kThreads),
                               sizeof(MixSmem), st, true, S, j[0], j[n > 1 ? 1 : 0],
                               j[n > 2 ? 2 : 0]));
        return OAL_OK;
    }
    dtc::MixJobs jobs;
    jobs.n = n;
    long long items = 0;
    for (int i = 0; i < n; ++i) {
        dtc::MixJob& m = jobs.job[i];
        m.j = j[i];
        m.has_first = sums[i]->first != nullptr;
        items += (long long)s->B * j[i].hx * S.chunks;
        if (!make_map_uncached(&m.x, j[i].x, s->T, s->B * j[i].hx) ||
            !make_map_uncached(&m.y, j[i].y, s->T, s->B * j[i].hy) ||
            !make_map_uncached(&m.z, j[i].z, s->T, s->B * j[i].hy) ||
            !make_out_map(&m.o, j[i].out, s->T, s->B * j[i].hx) ||
            !make_state_map(&m.m, j[i].mem, size_t(s->B) * s->Hkv * S.chunks))
            return OAL_ERR_CUDA;
    }
    OAL_CUDA_TRY(launch_ex(dtc::mix_kernel, dim3(int(std::min<long long>(items, 2 * sm_count()))),
                           dim3(dtc::kMixThreads), dtc::kMixSmem, st, true, jobs, S));
    return OAL_OK;
}

int check(const oal_shape* s)
{
    const int rc = check_common(s);
    if (rc) return rc;
    return check_planes((long long)s->B * s->Hq);
}

// Bytes of T tokens of `heads` heads.
size_t io_bytes(const oal_shape* s, int heads)
{
    return size_t(s->B) * heads * s->T * kD * (s->dtype == OAL_BF16 ? 2 : 4);
}

size_t state_bytes(const oal_shape* s) { return size_t(s->B) * s->Hkv * kDecayState * 4; }

int prefill(const void* q, const void* k, const void* v, const float* log_decay, float scale,
            const int32_t* lens, void* out, float* state, void* ws, size_t ws_bytes,
            const oal_shape* s, void* stream, bool cont)
{
    int rc = check(s);
    if (rc) return rc;
    if (s->B == 0) return OAL_OK;
    if (!log_decay || (cont ? !state : !state && !out)) return OAL_ERR_NULL;
    if ((rc = check_io(s, out ? q : k, k, v, out ? out : v))) return rc;
    if (!aligned16(state) || (reinterpret_cast<uintptr_t>(log_decay) & 3) ||
        (reinterpret_cast<uintptr_t>(lens) & 3))
        return OAL_ERR_ALIGN;
    size_t need = 0;
    if ((rc = oal_decay_prefill_workspace_bytes(s, &need))) return rc;
    if (!ws || ws_bytes < need) return OAL_ERR_WORKSPACE;
    if (!aligned16(ws)) return OAL_ERR_ALIGN;
    if (cont && s->T == 0) return OAL_OK;  // nothing is written
    const size_t nq = io_bytes(s, s->Hq), nk = io_bytes(s, s->Hkv);
    if (any_overlap({{out, nq}, {state, state_bytes(s)}},
                    {{out ? q : nullptr, nq}, {k, nk}, {v, nk}, {log_decay, size_t(s->Hkv) * 4},
                     {lens, size_t(s->B) * 4}}))
        return OAL_ERR_OVERLAP;
    OAL_CUDA_TRY(set_attributes_once());
    const DecayShape S{s->B, s->T, s->Hkv, chunks_of(s), lens, log_decay, scale};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const DecaySum sum = make_sum(k, v, s->Hkv, 0, 1, static_cast<unsigned char*>(ws), s,
                                  cont ? state : nullptr, state);
    if ((rc = launch_sums(S, &sum, 1, s, st)) || !out) return rc;
    const DecayJob job{q, k, v, out, sum.mem, s->Hq, s->Hkv, 0, 0};
    const DecaySum* of[] = {&sum};
    return launch_mix(S, &job, of, 1, s, st);
}

}  // namespace decay
}  // namespace oal

extern "C" {

using namespace oal;

int oal_decay_state_bytes(const oal_shape* s, size_t* bytes)
{
    const int rc = check_common(s);
    if (rc) return rc;
    if (!bytes) return OAL_ERR_NULL;
    *bytes = decay::state_bytes(s);
    return OAL_OK;
}

int oal_decay_prefill_workspace_bytes(const oal_shape* s, size_t* bytes)
{
    const int rc = decay::check(s);
    if (rc) return rc;
    if (!bytes) return OAL_ERR_NULL;
    *bytes = std::max<size_t>(decay::sum_layout(s, 1).total, 256);
    return OAL_OK;
}

int oal_decay_prefill(const void* q, const void* k, const void* v, const float* log_decay,
                      float scale, const int32_t* lens, void* out, float* state, void* workspace,
                      size_t workspace_bytes, const oal_shape* s, void* stream)
{
    return decay::prefill(q, k, v, log_decay, scale, lens, out, state, workspace, workspace_bytes,
                          s, stream, false);
}

int oal_decay_prefill_continue(const void* q, const void* k, const void* v,
                               const float* log_decay, float scale, const int32_t* lens,
                               void* out, float* state, void* workspace, size_t workspace_bytes,
                               const oal_shape* s, void* stream)
{
    return decay::prefill(q, k, v, log_decay, scale, lens, out, state, workspace, workspace_bytes,
                          s, stream, true);
}

int oal_decay_step(const void* q, const void* k, const void* v, const float* log_decay,
                   float scale, const float* src, int src_B, const int32_t* parents, float* state,
                   void* out, const oal_shape* s, void* stream)
{
    if (!s) return OAL_ERR_NULL;
    oal_shape one = *s;
    one.T = 1;
    int rc = check_common(&one);
    if (rc) return rc;
    if (s->B == 0) return OAL_OK;
    if ((src == nullptr) != (parents == nullptr)) return OAL_ERR_NULL;
    if (!log_decay || !state) return OAL_ERR_NULL;
    if ((rc = check_io(&one, q, k, v, out))) return rc;
    if (!aligned16(state) || !aligned16(src) || (reinterpret_cast<uintptr_t>(log_decay) & 3) ||
        (reinterpret_cast<uintptr_t>(parents) & 3))
        return OAL_ERR_ALIGN;
    oal_shape from = one;
    if (src) {
        if (src_B < 1) return OAL_ERR_SHAPE;
        from.B = src_B;
        if ((rc = check_common(&from))) return rc;
    }
    const size_t nq = decay::io_bytes(&one, s->Hq), nk = decay::io_bytes(&one, s->Hkv);
    if (any_overlap({{out, nq}, {state, decay::state_bytes(s)}},
                    {{q, nq}, {k, nk}, {v, nk}, {log_decay, size_t(s->Hkv) * 4},
                     {src, decay::state_bytes(&from)}, {parents, size_t(s->B) * 4}}))
        return OAL_ERR_OVERLAP;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return decay::by_type(s->dtype, [&](auto t) {
        using T = decltype(t);
        LaunchScope ls("decay_step", st);
        decay::step_kernel<T><<<s->B * s->Hkv, decay::kThreads, 0, st>>>(
            static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v),
            log_decay, scale, src ? src : state, parents, src_B, state, static_cast<T*>(out),
            s->Hq, s->Hkv);
        OAL_LAUNCH_CHECK();
        return int(OAL_OK);
    });
}

int oal_decay_backward_workspace_bytes(const oal_shape* s, size_t* bytes)
{
    const int rc = decay::check(s);
    if (rc) return rc;
    if (!bytes) return OAL_ERR_NULL;
    *bytes = std::max<size_t>(decay::sum_layout(s, 1).total +
                                  decay::sum_layout(s, decay::parts_of(s, s->Hq / s->Hkv)).total,
                              256);
    return OAL_OK;
}

int oal_decay_backward(const void* q, const void* k, const void* v, const float* log_decay,
                       float scale, const int32_t* lens, const void* dout, const float* state,
                       const float* dlast, void* dq, void* dk, void* dv, float* dstate,
                       void* workspace, size_t workspace_bytes, const oal_shape* s, void* stream)
{
    int rc = decay::check(s);
    if (rc) return rc;
    if (s->B == 0) return OAL_OK;
    if (!log_decay) return OAL_ERR_NULL;
    if ((rc = check_io(s, q, k, v, dout)) || (rc = check_io(s, dq, dk, dv, dout))) return rc;
    if (!aligned16(state) || !aligned16(dlast) || !aligned16(dstate) ||
        (reinterpret_cast<uintptr_t>(log_decay) & 3) || (reinterpret_cast<uintptr_t>(lens) & 3))
        return OAL_ERR_ALIGN;
    size_t need = 0;
    if ((rc = oal_decay_backward_workspace_bytes(s, &need))) return rc;
    if (!workspace || workspace_bytes < need) return OAL_ERR_WORKSPACE;
    if (!aligned16(workspace)) return OAL_ERR_ALIGN;
    const size_t nq = decay::io_bytes(s, s->Hq), nk = decay::io_bytes(s, s->Hkv);
    const size_t ns = decay::state_bytes(s);
    // (dstate over dlast itself: the block that writes an entry has read it before)
    if (any_overlap({{dq, nq}, {dk, nk}, {dv, nk}, {dstate, ns}},
                    {{q, nq}, {k, nk}, {v, nk}, {dout, nq}, {state, ns},
                     {log_decay, size_t(s->Hkv) * 4}, {lens, size_t(s->B) * 4}}) ||
        any_overlap({{dq, nq}, {dk, nk}, {dv, nk}, {dstate == dlast ? nullptr : dstate, ns}},
                    {{dlast, ns}}))
        return OAL_ERR_OVERLAP;
    OAL_CUDA_TRY(decay::set_attributes_once());
    const DecayShape S{s->B, s->T, s->Hkv, decay::chunks_of(s), lens, log_decay, scale};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned char* w = static_cast<unsigned char*>(workspace);
    const DecaySum sums[2] = {
        decay::make_sum(k, v, s->Hkv, 0, 1, w, s, state, nullptr),
        decay::make_sum(q, dout, s->Hq, 1, decay::parts_of(s, s->Hq / s->Hkv),
                        w + decay::sum_layout(s, 1).total, s, dlast, dstate)};
    if ((rc = decay::launch_sums(S, sums, 2, s, st))) return rc;
    // the long items (every head of a group) first
    const DecayJob jobs[3] = {{v, dout, q, dk, sums[1].mem, s->Hkv, s->Hq, 1, 1},
                              {k, q, dout, dv, sums[1].mem, s->Hkv, s->Hq, 1, 0},
                              {dout, v, k, dq, sums[0].mem, s->Hq, s->Hkv, 0, 1}};
    const DecaySum* const of[3] = {&sums[1], &sums[1], &sums[0]};
    return decay::launch_mix(S, jobs, of, 3, s, st);
}

}  // extern "C"
