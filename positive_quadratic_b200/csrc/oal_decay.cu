// oal_decay.cu -- linear attention with a decay per key/value head: the scan over chunks, the
// single-token step, the fp32 kernels of the other parts, and the entry points.
#pragma once

#include "oal_common.cuh"
#include "oal_decay.cuh"
#include "oal_kernels.cuh"

namespace oal {
namespace decay {

constexpr int kC = 64;          // tokens per chunk of the fp32 kernels
constexpr int kThreads = 256;
constexpr int kLd = kD + 4;     // padded row: 16-byte reads of 8 consecutive rows touch all banks

// Rows [t0, t0 + n) of head plane `src` as fp32 into a [64][kLd] tile, zero from row n on.
template <typename T>
__device__ __forceinline__ void load_tile(float (*dst)[kLd], const T* src, int t0, int n,
                                          const float* row_scale = nullptr)
{
    for (int e = threadIdx.x; e < kC * kD / 4; e += kThreads) {
        const int r = e / (kD / 4), c = 4 * (e % (kD / 4));
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n) {
            const T* p = src + size_t(t0 + r) * kD + c;
            a = make_float4(to_f32(p[0]), to_f32(p[1]), to_f32(p[2]), to_f32(p[3]));
            if (row_scale) {
                const float w = row_scale[r];
                a = make_float4(a.x * w, a.y * w, a.z * w, a.w * w);
            }
        }
        *reinterpret_cast<float4*>(&dst[r][c]) = a;
    }
}

// ------------------------------------------------------------------------------------------
// E_c of one (chunk, kv, b): a 64 x 64 product over the chunk's tokens, for every y head of the
// kv head.  Thread (ty, tx) owns rows 4 ty .. + 3 and columns 4 tx .. + 3.
// ------------------------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads) delta_simt_kernel(DecayShape S, DecaySum a, DecaySum b2)
{
    const DecaySum& J = blockIdx.z ? b2 : a;
    const int c = blockIdx.x, bkv = blockIdx.y, b = bkv / S.Hkv, kv = bkv % S.Hkv;
    const int n = min(kC, decay_len(S, b) - c * kC);
    if (n <= 0) return;  // the scan does not read it
    __shared__ __align__(16) float Y[kC][kLd], Z[kC][kLd];
    __shared__ float w[kC];
    const float g = decay_log(S.log_decay, kv);
    if (threadIdx.x < kC)
        w[threadIdx.x] = J.rev ? S.scale * decay_pow(g, threadIdx.x + 1)
                               : decay_pow(g, max(0, n - 1 - int(threadIdx.x)));
    const int grp = J.hy / S.Hkv, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    float acc[4][4] = {};
    for (int h = 0; h < grp; ++h) {
        const size_t plane = (size_t(b) * J.hy + kv * grp + h) * S.T * kD;
        __syncthreads();
        load_tile(Y, static_cast<const T*>(J.y) + plane, c * kC, n, w);
        load_tile(Z, static_cast<const T*>(J.z) + plane, c * kC, n);
        __syncthreads();
#pragma unroll 4
        for (int j = 0; j < kC; ++j) {
            const float4 y = *reinterpret_cast<const float4*>(&Y[j][4 * ty]);
            const float4 z = *reinterpret_cast<const float4*>(&Z[j][4 * tx]);
            const float yv[4] = {y.x, y.y, y.z, y.w}, zv[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(yv[i], zv[e], acc[i][e]);
        }
    }
    float* out = J.delta + (size_t(bkv) * S.chunks + c) * kDecayState;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(out + (4 * ty + i) * kDV + 4 * tx) =
            make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
}

// ------------------------------------------------------------------------------------------
// The scan over chunks of every (b, kv): thread = one state entry.
// ------------------------------------------------------------------------------------------
template <typename Tm>
__global__ void __launch_bounds__(kThreads) scan_kernel(DecayShape S, DecaySum a, DecaySum b2,
                                                        int chunk)
{
    const DecaySum& J = blockIdx.z ? b2 : a;
    const int bkv = blockIdx.y, b = bkv / S.Hkv, kv = bkv % S.Hkv;
    const int e = blockIdx.x * kThreads + threadIdx.x;
    const int len = decay_len(S, b);
    const int nc = (len + chunk - 1) / chunk;
    const float g = decay_log(S.log_decay, kv);
    const float full = decay_pow(g, chunk), tail = decay_pow(g, len - (nc - 1) * chunk);
    const size_t base = size_t(bkv) * S.chunks * kDecayState + e;
    float cur = J.first ? J.first[size_t(bkv) * kDecayState + e] : 0.f;
    for (int i = 0; i < nc; ++i) {
        const int c = J.rev ? nc - 1 - i : i;
        const size_t at = base + size_t(c) * kDecayState;
        const float d = J.delta[at];
        static_cast<Tm*>(J.mem)[at] = Tm(cur);
        cur = fmaf(c == nc - 1 ? tail : full, cur, d);
    }
    if (J.last) J.last[size_t(bkv) * kDecayState + e] = cur;
}

// ------------------------------------------------------------------------------------------
// The mix of one (chunk, x head, b).  Thread (ty, tx) owns rows 4 ty .. + 3; of the scores the
// columns tx + 16 e (conflict-free reads of y rows), of the output the columns 4 tx .. + 3.
// ------------------------------------------------------------------------------------------
template <typename T>
struct MixSmem {
    float X[kC][kLd], Y[kC][kLd], Z[kC][kLd], P[kC][kLd];
    float pw[kC + 1];  // powers of l
};

template <typename T>
__global__ void __launch_bounds__(kThreads) mix_simt_kernel(DecayShape S, DecayJob j0, DecayJob j1,
                                                            DecayJob j2)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    MixSmem<T>& sm = *reinterpret_cast<MixSmem<T>*>(smem_raw);
    const DecayJob& J = blockIdx.z == 0 ? j0 : blockIdx.z == 1 ? j1 : j2;
    const int c = blockIdx.x, b = blockIdx.y / J.hx, hx = blockIdx.y % J.hx;
    if (b >= S.B) return;  // the jobs share a grid of the largest head count
    const int n = min(kC, decay_len(S, b) - c * kC);
    if (n <= 0) return;
    const int kv = hx * S.Hkv / J.hx;
    const int nh = J.hy > J.hx ? J.hy / J.hx : 1;
    const int y0 = J.hy > J.hx ? hx * nh : hx * J.hy / J.hx;
    const float g = decay_log(S.log_decay, kv);
    for (int e = threadIdx.x; e <= kC; e += kThreads) sm.pw[e] = decay_pow(g, e);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    load_tile(sm.X, static_cast<const T*>(J.x) + (size_t(b) * J.hx + hx) * S.T * kD, c * kC, n);
    // M (or its transpose) where Z goes later
    const float* M = static_cast<const float*>(J.mem) +
                     ((size_t(b) * S.Hkv + kv) * S.chunks + c) * kDecayState;
    for (int e = threadIdx.x; e < kDecayState; e += kThreads) {
        const int r = e / kDV, cc = e % kDV;
        if (J.mem_t) sm.Z[cc][r] = M[e];
        else sm.Z[r][cc] = M[e];
    }
    __syncthreads();
    auto product = [&](const float (*A)[kLd], const float (*Bm)[kLd], float (&acc)[4][4]) {
#pragma unroll 2
        for (int k = 0; k < kC; k += 4) {
            float av[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 t4 = *reinterpret_cast<const float4*>(&A[4 * ty + i][k]);
                av[i][0] = t4.x; av[i][1] = t4.y; av[i][2] = t4.z; av[i][3] = t4.w;
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const float4 b4 = *reinterpret_cast<const float4*>(&Bm[k + kk][4 * tx]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[i][0] = fmaf(av[i][kk], b4.x, acc[i][0]);
                    acc[i][1] = fmaf(av[i][kk], b4.y, acc[i][1]);
                    acc[i][2] = fmaf(av[i][kk], b4.z, acc[i][2]);
                    acc[i][3] = fmaf(av[i][kk], b4.w, acc[i][3]);
                }
            }
        }
    };
    float far[4][4] = {}, near[4][4] = {};
    product(sm.X, sm.Z, far);
    for (int h = 0; h < nh; ++h) {
        const size_t plane = (size_t(b) * J.hy + y0 + h) * S.T * kD;
        __syncthreads();
        load_tile(sm.Y, static_cast<const T*>(J.y) + plane, c * kC, n);
        load_tile(sm.Z, static_cast<const T*>(J.z) + plane, c * kC, n);
        __syncthreads();
        float s[4][4] = {};
#pragma unroll 2
        for (int k = 0; k < kD; k += 4) {
            float4 x4[4], y4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x4[i] = *reinterpret_cast<const float4*>(&sm.X[4 * ty + i][k]);
                y4[i] = *reinterpret_cast<const float4*>(&sm.Y[tx + 16 * i][k]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[i][e] = fmaf(x4[i].x, y4[e].x, s[i][e]);
                    s[i][e] = fmaf(x4[i].y, y4[e].y, s[i][e]);
                    s[i][e] = fmaf(x4[i].z, y4[e].z, s[i][e]);
                    s[i][e] = fmaf(x4[i].w, y4[e].w, s[i][e]);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 4 * ty + i, col = tx + 16 * e;
                const int d = J.rev ? col - row : row - col;
                sm.P[row][col] = d >= 0 ? s[i][e] * sm.pw[d] : 0.f;
            }
        __syncthreads();
        product(sm.P, sm.Z, near);
    }
    T* out = static_cast<T*>(J.out) + ((size_t(b) * J.hx + hx) * S.T + c * kC) * kD;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 4 * ty + i;
        if (row >= n) continue;
        const float bi = J.rev ? sm.pw[n - 1 - row] : S.scale * sm.pw[row + 1];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            out[size_t(row) * kD + 4 * tx + e] = T(fmaf(S.scale, near[i][e], bi * far[i][e]));
    }
}

// ------------------------------------------------------------------------------------------
// One token: block = (kv, b).  Thread (r0, c4) holds rows r0 + 16 i of the columns 4 c4 .. + 3.
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
int chunk_of(const oal_shape*) { return kC; }

size_t sum_bytes(const oal_shape* s)
{
    const size_t nc = (size_t(s->T) + chunk_of(s) - 1) / chunk_of(s);
    return align256(size_t(s->B) * s->Hkv * nc * kDecayState * 4);
}

template <typename F>
int by_type(int dtype, F f)
{
    return dtype == OAL_BF16 ? f(__nv_bfloat16{}) : f(float{});
}

// The sums of `n` directions (1 or 2) and their scans.
int launch_sums(const DecayShape& S, const DecaySum* a, int n, const oal_shape* s, cudaStream_t st)
{
    const DecaySum& b2 = a[n - 1];
    if (S.chunks > 0)
        if (const int rc = by_type(s->dtype, [&](auto t) {
                LaunchScope ls("decay_delta", st);
                delta_simt_kernel<decltype(t)>
                    <<<dim3(S.chunks, s->B * s->Hkv, n), kThreads, 0, st>>>(S, a[0], b2);
                OAL_LAUNCH_CHECK();
                return int(OAL_OK);
            }))
            return rc;
    LaunchScope ls("decay_scan", st);
    scan_kernel<float><<<dim3(kDecayState / kThreads, s->B * s->Hkv, n), kThreads, 0, st>>>(
        S, a[0], b2, chunk_of(s));
    OAL_LAUNCH_CHECK();
    return OAL_OK;
}

int launch_mix(const DecayShape& S, const DecayJob* j, int n, const oal_shape* s, cudaStream_t st)
{
    if (S.chunks == 0) return OAL_OK;
    int hx = 0;
    for (int i = 0; i < n; ++i) hx = std::max(hx, j[i].hx);
    return by_type(s->dtype, [&](auto t) {
        using T = decltype(t);
        OAL_CUDA_TRY(cudaFuncSetAttribute(mix_simt_kernel<T>,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          int(sizeof(MixSmem<T>))));
        LaunchScope ls("decay_mix", st);
        mix_simt_kernel<T><<<dim3(S.chunks, s->B * hx, n), kThreads, sizeof(MixSmem<T>), st>>>(
            S, j[0], j[n > 1 ? 1 : 0], j[n > 2 ? 2 : 0]);
        OAL_LAUNCH_CHECK();
        return int(OAL_OK);
    });
}

int check(const oal_shape* s)
{
    const int rc = check_common(s);
    if (rc) return rc;
    return check_planes((long long)s->B * s->Hq);
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
    if (cont && s->T == 0) return OAL_OK;
    const DecayShape S{s->B, s->T, s->Hkv, (s->T + chunk_of(s) - 1) / chunk_of(s), lens, log_decay,
                       scale};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float* d = static_cast<float*>(ws);
    const DecaySum sum{k, v, s->Hkv, 0, d, d, cont ? state : nullptr, state};
    if ((rc = launch_sums(S, &sum, 1, s, st)) || !out) return rc;
    const DecayJob job{q, k, v, out, d, s->Hq, s->Hkv, 0, 0};
    return launch_mix(S, &job, 1, s, st);
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
    *bytes = std::max<size_t>(decay::sum_bytes(s), 256);
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
    if (src) {
        if (src_B < 1) return OAL_ERR_SHAPE;
        oal_shape from = one;
        from.B = src_B;
        if ((rc = check_common(&from))) return rc;
        if (overlap(src, decay::state_bytes(&from), state, decay::state_bytes(s)))
            return OAL_ERR_OVERLAP;
    }
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
    *bytes = std::max<size_t>(2 * decay::sum_bytes(s), 256);
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
    const int C = decay::chunk_of(s);
    const DecayShape S{s->B, s->T, s->Hkv, (s->T + C - 1) / C, lens, log_decay, scale};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned char* w = static_cast<unsigned char*>(workspace);
    float* fs = reinterpret_cast<float*>(w);
    float* rs = reinterpret_cast<float*>(w + decay::sum_bytes(s));
    const DecaySum sums[2] = {{k, v, s->Hkv, 0, fs, fs, state, nullptr},
                              {q, dout, s->Hq, 1, rs, rs, dlast, dstate}};
    if ((rc = decay::launch_sums(S, sums, 2, s, st))) return rc;
    const DecayJob jobs[3] = {{dout, v, k, dq, fs, s->Hq, s->Hkv, 0, 1},
                              {v, dout, q, dk, rs, s->Hkv, s->Hq, 1, 1},
                              {k, q, dout, dv, rs, s->Hkv, s->Hq, 1, 0}};
    return decay::launch_mix(S, jobs, 3, s, st);
}

}  // extern "C"
