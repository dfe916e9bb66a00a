// oal_decay_tc.cuh -- bf16 linear attention with a decay per key/value head on tensor cores: the
// products of a chunk and the mix (oal_decay.cuh), in chunks of 128 tokens.
//
// Every wait is bounded (1 s); one that runs out sets OAL_ERR_TIMEOUT and every role leaves its
// loop in order (copies drained, MMAs completed, tensor memory freed).
#pragma once

#include "oal_decay.cuh"
#include "oal_tc_util.cuh"

namespace oal {
namespace decay {
namespace dtc {

using namespace oal::tc;  // PTX layer

constexpr int kC = 128;
constexpr int kThreads = 288;   // of the delta kernel: 8 compute warps and a control warp
constexpr int kCtrlWarp = 8;
constexpr uint32_t kTile = kC * 128;      // a 128 x 64 bf16 tile
constexpr uint32_t kMTile = 64 * 128;     // a 64 x 64 bf16 state image

// 32 lanes x 32 consecutive 32-bit columns (see tmem_ld16).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
        "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
}

// Rows [n, 128) of a tile to zero, by the first kBy threads.
template <int kBy>
__device__ __forceinline__ void zero_rows(unsigned char* tile, int n)
{
    for (int e = n * 8 + threadIdx.x; e < kC * 8; e += kBy)
        *reinterpret_cast<uint4*>(tile + e * 16) = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------------------------------
// E_c = sum_h sum_j w_j y_hj z_hj^T.  The weights are fp32, so w_j y_j has more digits than a
// bf16 operand: it is split into three bf16 parts (8 + 8 + 8 digits, all of an fp32 product), and
// the state keeps fp32 accuracy.  Rows of the accumulator: [hi; mid] in one MMA group of M = 128
// and [lo; hi] in a second, of which lo is used, so that E = hi + (mid + lo).
// One CTA per (sum, part of the heads, b, kv, chunk); two fit an SM.
// ------------------------------------------------------------------------------------------
struct SumMaps {
    CUtensorMap y[2], z[2];
};

struct DeltaCtl {
    uint64_t y_full, z_full[2], parts, done;
    uint32_t tmem_base;
    int abort_flag;
};

constexpr uint32_t kDOffY = 0, kDOffZ = kTile, kDOffLo = 3 * kTile, kDOffHi = 4 * kTile;
constexpr uint32_t kDOffCtl = 6 * kTile;
constexpr uint32_t kDeltaSmem = kDOffCtl + 128 + 1024;
constexpr uint32_t kDeltaTmem = 128;
static_assert(sizeof(DeltaCtl) <= 128 && 2 * (kDeltaSmem + 1024) <= 233472, "two CTAs per SM");

__global__ void __launch_bounds__(kThreads, 2)
    delta_kernel(const __grid_constant__ SumMaps maps, DecayShape S, DecaySum a, DecaySum b2)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = smem_raw + (-smem_u32(smem_raw) & 1023u);  // still known to be shared
    DeltaCtl& ctl = *reinterpret_cast<DeltaCtl*>(sm + kDOffCtl);
    volatile int* abort_flag = &ctl.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // items of the first sum, then of the second
    int item = blockIdx.x;
    const int planes = S.B * S.Hkv, first_items = a.parts * planes * S.chunks;
    const int which = item >= first_items;
    const DecaySum& J = which ? b2 : a;
    if (which) item -= first_items;
    const int c = item % S.chunks, bkv = (item / S.chunks) % planes, part = item / S.chunks / planes;
    const int b = bkv / S.Hkv, kv = bkv % S.Hkv;
    const int n = min(kC, decay_len(S, b) - c * kC);
    const int grp = J.hy / S.Hkv, per = (grp + J.parts - 1) / J.parts;
    const int h0 = part * per, nh = min(per, grp - h0);
    // launched before the trigger below: every CTA holds its tensor memory by then, and the
    // dependents, which allocate too, cannot keep it from one
    if (warp == kCtrlWarp) {
        tmem_alloc(&ctl.tmem_base, kDeltaTmem);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        mbar_init(&ctl.y_full, 1);
        mbar_init(&ctl.z_full[0], 1);
        mbar_init(&ctl.z_full[1], 1);
        mbar_init(&ctl.parts, 8);
        mbar_init(&ctl.done, 1);
        ctl.abort_flag = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;
    grid_dep_launch();

    if (n > 0 && nh > 0) {
        if (warp < 8) {
            const int row = threadIdx.x >> 1, half = threadIdx.x & 1;
            const float g = decay_log(S.log_decay, kv);
            const float w = row >= n ? 0.f
                            : J.rev  ? S.scale * decay_pow(g, row + 1)
                                     : decay_pow(g, n - 1 - row);
            const uint32_t lo = smem_u32(sm + kDOffLo);
            bool ok = true;
            for (int i = 0; i < nh; ++i) {
                ok = wait_all(&ctl.y_full, i & 1, abort_flag) &&
                     wait_all(&ctl.z_full[i & 1], (i >> 1) & 1, abort_flag) &&
                     (i == 0 || wait_all(&ctl.done, (i - 1) & 1, abort_flag));
                if (!ok) break;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t off = kmajor_chunk(row, 4 * half + x);
                    uint4 y = *reinterpret_cast<const uint4*>(sm + kDOffY + off);
                    if (row >= n) y = make_uint4(0, 0, 0, 0);  // whatever lies there
                    const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
                    uint32_t p[3][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float u = bf16lo_to_f32(yw[e]) * w, v = bf16hi_to_f32(yw[e]) * w;
#pragma unroll
                        for (int q = 0; q < 3; ++q) {
                            p[q][e] = pack_bf16x2(u, v);
                            u -= bf16lo_to_f32(p[q][e]);
                            v -= bf16hi_to_f32(p[q][e]);
                        }
                    }
                    sts128(lo + kTile + off, p[0][0], p[0][1], p[0][2], p[0][3]);
                    sts128(lo + 2 * kTile + off, p[1][0], p[1][1], p[1][2], p[1][3]);
                    sts128(lo + off, p[2][0], p[2][1], p[2][2], p[2][3]);
                }
                if (n < kC) zero_rows<256>(sm + kDOffZ + (i & 1) * kTile, n);
                fence_proxy_async();
                warp_arrive(&ctl.parts);
            }
            ok = ok && wait_all(&ctl.done, (nh - 1) & 1, abort_flag);
            ok = named_bar_and(1, 256, ok);
            if (ok) {
                tc_fence_after();
                const int qw = warp & 3, kh = warp >> 2, r = (32 * qw + lane) & 63;
                const uint32_t base = tmem + (uint32_t(qw * 32) << 16) + 32 * kh;
                float (*stage)[68] = reinterpret_cast<float(*)[68]>(sm + kDOffLo);
                float d[32];
                tmem_ld32(base, d);
                tmem_ld_wait();
                if (qw >= 2)
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(&stage[r][32 * kh + e]) =
                            make_float4(d[e], d[e + 1], d[e + 2], d[e + 3]);
                float l[32];
                if (qw < 2) {
                    tmem_ld32(base + 64, l);
                    tmem_ld_wait();
                }
                named_bar_sync(1, 256);
                if (qw < 2)
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float4* s = reinterpret_cast<float4*>(&stage[r][32 * kh + e]);
                        const float4 m = *s;
                        *s = make_float4(d[e] + (m.x + l[e]), d[e + 1] + (m.y + l[e + 1]),
                                         d[e + 2] + (m.z + l[e + 2]), d[e + 3] + (m.w + l[e + 3]));
                    }
                named_bar_sync(1, 256);
                float4* out = reinterpret_cast<float4*>(
                    J.delta + ((size_t(part) * planes + bkv) * S.chunks + c) * kDecayState);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = i * 256 + threadIdx.x;
                    out[e] = *reinterpret_cast<const float4*>(&stage[e >> 4][4 * (e & 15)]);
                }
                tc_fence_before();
            }
        } else if (lane == 0) {
            constexpr uint32_t id = idesc_bf16(128, 64, true, true);
            const CUtensorMap* my = &maps.y[which];
            const CUtensorMap* mz = &maps.z[which];
            const int plane = b * J.hy + kv * grp + h0;
            const uint32_t lo = smem_u32(sm + kDOffLo), z = smem_u32(sm + kDOffZ);
            int ny = 0, nz = 0, nmma = 0;
            auto load_y = [&](int i) {
                mbar_expect_tx(&ctl.y_full, kTile);
                tma_load_3d(sm + kDOffY, my, &ctl.y_full, 0, c * kC, plane + i);
                ++ny;
            };
            auto load_z = [&](int i) {
                mbar_expect_tx(&ctl.z_full[i & 1], kTile);
                tma_load_3d(sm + kDOffZ + (i & 1) * kTile, mz, &ctl.z_full[i & 1], 0, c * kC,
                            plane + i);
                ++nz;
            };
            load_y(0);
            load_z(0);
            if (nh > 1) load_z(1);
            for (int i = 0; i < nh; ++i) {
                if (!mbar_wait(&ctl.parts, i & 1, abort_flag)) break;
                if (i + 1 < nh) load_y(i + 1);  // the parts of head i have been formed
                tc_fence_after();
                const uint32_t zi = z + (i & 1) * kTile;
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_bf16(tmem + 64 * g,
                                 sdesc_sw128(lo + (1 - g) * kTile + ks * 2048, kTile, 1024),
                                 sdesc_sw128(zi + ks * 2048, kTile, 1024), id,
                                 (i > 0 || ks > 0) ? 1u : 0u);
                mma_commit(&ctl.done);
                ++nmma;
                if (i + 2 < nh) {
                    if (!mbar_wait(&ctl.done, i & 1, abort_flag)) break;
                    load_z(i + 2);
                }
            }
            // nothing of this CTA is in flight when it ends
            bounded_spin_done(&ctl.y_full, (ny - 1) & 1);
            bounded_spin_done(&ctl.z_full[(nz - 1) & 1], ((nz - 1) >> 1) & 1);
            if (nz > 1) bounded_spin_done(&ctl.z_full[nz & 1], ((nz - 2) >> 1) & 1);
            if (nmma) bounded_spin_done(&ctl.done, (nmma - 1) & 1);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kCtrlWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kDeltaTmem);
    }
}

// ------------------------------------------------------------------------------------------
// The mix of one (job, b, x head, chunk) item:
//   S_h = X Y_h^T (tensor memory), P_h = bf16(S_h o D) written over it, U = sum_h P_h Z_h,
//   F = X M (the bf16 state before the chunk), out = scale U + b F.
// The decay of the far part is applied to F's rows in fp32, so that q and S are rounded once.
// Persistent: two CTAs per SM, each walking items blockIdx.x, blockIdx.x + gridDim.x, ...
// Warps 0-7 compute: warp (qw, kh) holds rows 32 qw .. + 31 (its tensor-memory lanes), keys
// 64 kh .. + 63 of the scores and columns 32 kh .. + 31 of the output.  Warp 8 issues the MMAs;
// the next item's scores are formed while the compute warps write out the present one's result.
// Warp 9 looks ahead: it works out the next items' places and powers of l and loads their tiles
// as soon as buffers are free.
// ------------------------------------------------------------------------------------------
struct MixJob {
    CUtensorMap x, y, z, m;
    DecayJob j;
    int has_first;  // the chunk at the start of the scan has a state, too
    int items;      // of this job
};
struct MixJobs {
    MixJob job[3];
    int n;
};

constexpr int kMixWarps = 8;  // compute warps
constexpr int kMixThreads = (kMixWarps + 2) * 32;
constexpr int kMmaWarp = kMixWarps, kAheadWarp = kMixWarps + 1;
constexpr int kInfos = 4;  // items that the look-ahead warp may have described and not seen done

// What the other warps need to know of an item, and the powers of l: l^i at pw[kPw0 + i], so that
// pairs that start at an odd power are 8-byte aligned and 31 places lie before the first.
constexpr int kPw0 = 33;
struct MixInfo {
    __nv_bfloat16* out;  // the tile's first row
    int n, nh, rev, has_m, mem_t, garbage, none, pad;
    float pw[kPw0 + kC + 3];
};

struct MixCtl {
    uint64_t x_full, m_full, yz_full[2], yz_free[2], s_full, p_full, pv_done, x_free, out_free;
    uint64_t info_full[kInfos], info_free[kInfos];
    uint32_t tmem_base;
    int abort_flag;
};

constexpr uint32_t kMOffX = 0, kMOffYZ = kTile, kMOffM = 5 * kTile;
constexpr uint32_t kMOffInfo = kMOffM + kMTile;
constexpr uint32_t kMOffCtl = kMOffInfo + kInfos * sizeof(MixInfo);
constexpr uint32_t kMixSmem = kMOffCtl + 256 + 1024;
constexpr uint32_t kMixTmem = 256;
constexpr uint32_t kColS = 0, kColU = 128, kColF = 192;
static_assert(sizeof(MixCtl) <= 256 && kMOffCtl % 8 == 0 && 2 * (kMixSmem + 1024) <= 233472,
              "two CTAs per SM");
static_assert(sizeof(MixInfo) % 8 == 0 && offsetof(MixInfo, pw) % 8 == 0 && kPw0 % 2 == 1, "alignment of pw");

struct MixItem {
    int w, b, hx, kv, c, n, nh, y0, has_m;
};

// Item `idx`; n <= 0 if it has no tokens.  Items of a job: (b, kv, chunk, head of the group), so
// that the heads that share keys, values and a state run side by side.
__device__ __forceinline__ MixItem mix_item(const MixJobs& jobs, const DecayShape& S, int idx)
{
    MixItem it;
    it.w = 0;
    while (it.w + 1 < jobs.n && idx >= jobs.job[it.w].items) idx -= jobs.job[it.w++].items;
    const DecayJob& j = jobs.job[it.w].j;
    const int grpx = j.hx / S.Hkv;
    const int gi = idx % grpx, r = idx / grpx;
    it.c = r % S.chunks;
    it.kv = (r / S.chunks) % S.Hkv;
    it.b = r / S.chunks / S.Hkv;
    it.hx = it.kv * grpx + gi;
    it.nh = j.hy > j.hx ? j.hy / j.hx : 1;
    it.y0 = j.hy > j.hx ? it.hx * it.nh : it.kv * (j.hy / S.Hkv) + (j.hy == j.hx ? gi : 0);
    const int len = decay_len(S, it.b);
    it.n = min(kC, len - it.c * kC);
    it.has_m = it.c != (j.rev ? (len - 1) / kC : 0) || jobs.job[it.w].has_first;
    return it;
}

// P = S o D for rows 32 qw + lane and keys 32 jb .. + 31, written over the scores.
template <bool kRev>
__device__ __forceinline__ void decay_scores(uint32_t scores, const float* pw, int qw, int jb,
                                             int lane, int n)
{
    uint32_t p[16];
    if (jb == qw) {  // the diagonal block
        float s[32];
        tmem_ld32(scores, s);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 32; ++x) {
            // on the wrong side of the diagonal the factor is whatever lies there, and the
            // product (which may be NaN, as may what lies behind the end) is not taken
            const float d = kRev ? pw[kPw0 + x - lane] : pw[kPw0 + lane - x];
            const float v = s[x] * d;
            s[x] = (kRev ? x >= lane && 32 * jb + x < n : x <= lane) ? v : 0.f;
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) p[x] = pack_bf16x2(s[2 * x], s[2 * x + 1]);
    } else if (kRev ? jb > qw : jb < qw) {
        // l^|i-j| = l^(from the row to its block's edge) l^(from there to j)
        float s[32];
        tmem_ld32(scores, s);
        const float rf = pw[kPw0 + (kRev ? 31 - lane : lane)];
        const float2 rf2 = make_float2(rf, rf);
        // the pair of columns (x, x + 1): powers at + x and at + x + 1 (kRev), or - x, - x - 1
        const float* at = pw + kPw0 + (kRev ? 32 * (jb - qw) - 31 : 32 * (qw - jb) - 1);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
            float2 d = *reinterpret_cast<const float2*>(kRev ? at + x : at - x);
            if (!kRev) d = make_float2(d.y, d.x);
            const float2 v = __fmul2_rn(make_float2(s[x], s[x + 1]), __fmul2_rn(rf2, d));
            s[x] = v.x;
            s[x + 1] = v.y;
        }
        if (kRev && n < kC)  // keys behind the sequence's end, whatever they gave
#pragma unroll
            for (int x = 0; x < 32; ++x)
                if (32 * jb + x >= n) s[x] = 0.f;
#pragma unroll
        for (int x = 0; x < 16; ++x) p[x] = pack_bf16x2(s[2 * x], s[2 * x + 1]);
    } else {
#pragma unroll
        for (int x = 0; x < 16; ++x) p[x] = 0u;
    }
    tmem_st16(scores, p);
}

// Stores 16 bf16 values (32 bytes; one store where the address allows it).
__device__ __forceinline__ void store16(__nv_bfloat16* out, const uint32_t (&p)[8], bool wide)
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out),
                     "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3]), "r"(p[4]), "r"(p[5]), "r"(p[6]),
                     "r"(p[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(out)[0] = make_uint4(p[0], p[1], p[2], p[3]);
        reinterpret_cast<uint4*>(out)[1] = make_uint4(p[4], p[5], p[6], p[7]);
    }
}

__global__ void __launch_bounds__(kMixThreads, 2)
    mix_kernel(const __grid_constant__ MixJobs jobs, DecayShape S, int items)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = smem_raw + (-smem_u32(smem_raw) & 1023u);  // still known to be shared
    MixCtl& ctl = *reinterpret_cast<MixCtl*>(sm + kMOffCtl);
    MixInfo* infos = reinterpret_cast<MixInfo*>(sm + kMOffInfo);
    volatile int* abort_flag = &ctl.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(&ctl.x_full, 1);
        mbar_init(&ctl.m_full, 1);
        mbar_init(&ctl.s_full, 1);
        mbar_init(&ctl.p_full, kMixWarps);
        mbar_init(&ctl.pv_done, 1);
        mbar_init(&ctl.x_free, 1);
        mbar_init(&ctl.out_free, kMixWarps);
        mbar_init(&ctl.yz_full[0], 1);
        mbar_init(&ctl.yz_full[1], 1);
        mbar_init(&ctl.yz_free[0], 1);
        mbar_init(&ctl.yz_free[1], 1);
        for (int i = 0; i < kInfos; ++i) {
            mbar_init(&ctl.info_full[i], 1);
            mbar_init(&ctl.info_free[i], kMixWarps);
        }
        ctl.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&ctl.tmem_base, kMixTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;

    if (warp < kMixWarps) {
        const int qw = warp & 3, kh = warp >> 2, row = 32 * qw + lane;
        const uint32_t lanes = tmem + (uint32_t(qw * 32) << 16);
        bool ok = true;
        for (int done = 0, step = 0; ok; ++done) {
            ok = wait_all(&ctl.info_full[done % kInfos], (done / kInfos) & 1, abort_flag);
            const MixInfo& I = infos[done % kInfos];
            if (!ok || I.none) break;
            const int n = I.n, nh = I.nh, rev = I.rev, has_m = I.has_m;
            for (int h = 0; h < nh; ++h, ++step) {
                ok = wait_all(&ctl.s_full, step & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int jb = 2 * kh + half;
                    if (rev) decay_scores<true>(lanes + kColS + 32 * jb, I.pw, qw, jb, lane, n);
                    else decay_scores<false>(lanes + kColS + 32 * jb, I.pw, qw, jb, lane, n);
                }
                tmem_st_wait();
                tc_fence_before();
                if (I.garbage) {
                    // rows behind the sequence's end: zero times what lies there has to be zero
                    ok = wait_all(&ctl.yz_full[step & 1], (step >> 1) & 1, abort_flag);
                    if (!ok) break;
                    zero_rows<kMixWarps * 32>(sm + kMOffYZ + (step & 1) * 2 * kTile + kTile, n);
                    fence_proxy_async();
                }
                warp_arrive(&ctl.p_full);
            }
            const float bi = rev ? (row < n ? I.pw[kPw0 + n - 1 - row] : 0.f)
                                 : S.scale * I.pw[kPw0 + row + 1];
            __nv_bfloat16* out = I.out + row * kD + 32 * kh;
            ok = ok && wait_all(&ctl.pv_done, (step - 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            float u[32];
            tmem_ld32(lanes + kColU + 32 * kh, u);
            if (has_m) {
                float f[32];
                tmem_ld32(lanes + kColF + 32 * kh, f);
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 32; ++x) u[x] = fmaf(bi, f[x], S.scale * u[x]);
            } else {
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 32; ++x) u[x] *= S.scale;
            }
            tc_fence_before();
            warp_arrive(&ctl.out_free);
            if (row < n) {
                const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        p[x] = pack_bf16x2(u[16 * half + 2 * x], u[16 * half + 2 * x + 1]);
                    store16(out + 16 * half, p, wide);
                }
            }
            warp_arrive(&ctl.info_free[done % kInfos]);
        }
    } else if (warp == kAheadWarp) {
        int nx = 0, nm = 0, nyz = 0, done = 0;
        bool ok = true, waited = false;
        for (int idx = blockIdx.x;; idx += gridDim.x, ++done) {
            MixItem it;
            it.n = 0;
            for (; idx < items; idx += gridDim.x)
                if ((it = mix_item(jobs, S, idx)).n > 0) break;
            if (done >= kInfos)
                ok = wait_all_sleep(&ctl.info_free[done % kInfos], (done / kInfos - 1) & 1, abort_flag);
            if (!ok) break;
            MixInfo& I = infos[done % kInfos];
            const bool none = idx >= items;
            const MixJob& J = jobs.job[it.n > 0 ? it.w : 0];
            if (!none) {
                const float g = decay_log(S.log_decay, it.kv);
                I.pw[1 + lane] = 0.f;
                #pragma unroll
                for (int i = 0; i < kC; i += 32) I.pw[kPw0 + i + lane] = decay_pow(g, i + lane);
                if (lane == 0) I.pw[kPw0 + kC] = decay_pow(g, kC);
                if (lane == 0) {
                    const int left = S.T - it.c * kC, plane = it.b * J.j.hx + it.hx;
                    I.out = static_cast<__nv_bfloat16*>(J.j.out) +
                            (size_t(plane) * S.T + it.c * kC) * kD;
                    I.n = it.n;
                    I.nh = it.nh;
                    I.rev = J.j.rev;
                    I.has_m = it.has_m;
                    I.mem_t = J.j.mem_t;
                    I.garbage = it.n < kC && it.n < left;
                }
            }
            if (lane == 0) I.none = none;
            warp_arrive(&ctl.info_full[done % kInfos]);
            if (none) break;
            if (lane == 0) {
                // Y and Z of a step go where those of two steps before were, once P Z has read them
                // (a barrier of each stage: this warp may lag behind pv_done by two phases, which
                // a parity cannot tell from none)
                auto load_yz = [&](int h) {
                    if (nyz >= 2)
                        ok = mbar_wait_sleep(&ctl.yz_free[nyz & 1], ((nyz >> 1) - 1) & 1, abort_flag);
                    if (!ok) return;
                    unsigned char* dst = sm + kMOffYZ + (nyz & 1) * 2 * kTile;
                    uint64_t* bar = &ctl.yz_full[nyz & 1];
                    const int plane = it.b * J.j.hy + it.y0 + h;
                    mbar_expect_tx(bar, 2 * kTile);
                    tma_load_3d(dst, &J.y, bar, 0, it.c * kC, plane);
                    tma_load_3d(dst + kTile, &J.z, bar, 0, it.c * kC, plane);
                    ++nyz;
                };
                if (done > 0) ok = mbar_wait_sleep(&ctl.x_free, (done - 1) & 1, abort_flag);
                if (ok) {
                    mbar_expect_tx(&ctl.x_full, kTile);
                    tma_load_3d(sm + kMOffX, &J.x, &ctl.x_full, 0, it.c * kC, it.b * J.j.hx + it.hx);
                    ++nx;
                    load_yz(0);
                }
                // (the inputs were there before the kernels whose results this one waits for)
                if (!waited) grid_dep_wait();
                waited = true;
                if (ok && it.has_m) {
                    mbar_expect_tx(&ctl.m_full, kMTile);
                    tma_load_2d(sm + kMOffM, &J.m, &ctl.m_full, 0,
                                ((it.b * S.Hkv + it.kv) * S.chunks + it.c) * 64);
                    ++nm;
                }
                for (int h = 1; ok && h < it.nh; ++h) load_yz(h);
            }
            ok = __shfl_sync(~0u, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
        }
        if (lane == 0) {
            if (!waited) grid_dep_wait();
            // no copy is in flight when the CTA ends
            if (nx) bounded_spin_done(&ctl.x_full, (nx - 1) & 1);
            if (nm) bounded_spin_done(&ctl.m_full, (nm - 1) & 1);
            if (nyz) bounded_spin_done(&ctl.yz_full[(nyz - 1) & 1], ((nyz - 1) >> 1) & 1);
            if (nyz > 1) bounded_spin_done(&ctl.yz_full[nyz & 1], ((nyz - 2) >> 1) & 1);
        }
    } else if (lane == 0) {
        constexpr uint32_t id_s = idesc_bf16(128, 128, false, false);
        constexpr uint32_t id_mn = idesc_bf16(128, 64, false, true), id_k = idesc_bf16(128, 64, false, false);
        const uint32_t x = smem_u32(sm + kMOffX), m = smem_u32(sm + kMOffM);
        const uint32_t yz = smem_u32(sm + kMOffYZ);
        int nm = 0, npv = 0, nfree = 0, step = 0;
        bool ok = true;
        for (int done = 0; ok; ++done) {
            ok = mbar_wait(&ctl.info_full[done % kInfos], (done / kInfos) & 1, abort_flag);
            const MixInfo& I = infos[done % kInfos];
            if (!ok || I.none) break;
            const int nh = I.nh, has_m = I.has_m, mem_t = I.mem_t;
            ok = mbar_wait(&ctl.x_full, done & 1, abort_flag);
            for (int h = 0; ok && h < nh; ++h, ++step) {
                ok = mbar_wait(&ctl.yz_full[step & 1], (step >> 1) & 1, abort_flag) &&
                     // the scores go over P of the step before
                     (step == 0 || mbar_wait(&ctl.pv_done, (step - 1) & 1, abort_flag));
                if (!ok) break;
                const uint32_t y = yz + (step & 1) * 2 * kTile, z = y + kTile;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16(tmem + kColS, sdesc_sw128(x + ks * 32, 16, 1024),
                             sdesc_sw128(y + ks * 32, 16, 1024), id_s, ks > 0 ? 1u : 0u);
                mma_commit(&ctl.s_full);
                if (h == 0) {
                    // U and F of the item before have been read
                    if (done > 0) ok = mbar_wait(&ctl.out_free, (done - 1) & 1, abort_flag);
                    if (ok && has_m) {
                        ok = mbar_wait(&ctl.m_full, nm & 1, abort_flag);
                        ++nm;
                        if (ok) {
                            tc_fence_after();
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_bf16(tmem + kColF, sdesc_sw128(x + ks * 32, 16, 1024),
                                         mem_t ? sdesc_sw128(m + ks * 32, 16, 1024)
                                               : sdesc_sw128(m + ks * 2048, kTile, 1024),
                                         mem_t ? id_k : id_mn, ks > 0 ? 1u : 0u);
                        }
                    }
                    if (!ok) break;
                }
                if (h == nh - 1) {
                    mma_commit(&ctl.x_free);  // no later MMA of the item reads X or M
                    ++nfree;
                }
                ok = mbar_wait(&ctl.p_full, step & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_bf16_ts(tmem + kColU, tmem + kColS + 32 * (ks >> 1) + 8 * (ks & 1),
                                sdesc_sw128(z + ks * 2048, kTile, 1024), id_mn,
                                (h > 0 || ks > 0) ? 1u : 0u);
                mma_commit(&ctl.pv_done);
                mma_commit(&ctl.yz_free[step & 1]);
                ++npv;
            }
        }
        // every MMA has completed before tensor memory is freed
        if (nfree) bounded_spin_done(&ctl.x_free, (nfree - 1) & 1);
        if (npv) bounded_spin_done(&ctl.yz_free[(npv - 1) & 1], ((npv - 1) >> 1) & 1);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kMixTmem);
    }
}

}  // namespace dtc
}  // namespace decay
}  // namespace oal
