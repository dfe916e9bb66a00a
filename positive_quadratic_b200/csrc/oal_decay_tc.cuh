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
constexpr int kThreads = 288;   // 8 compute warps and one that issues copies and MMAs
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

__device__ __forceinline__ void tma_store_3d(const void* tmap, const void* src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
                 : "memory");
}

// Rows [n, 128) of a tile to zero, by the 256 compute threads.
__device__ __forceinline__ void zero_rows(unsigned char* tile, int n)
{
    for (int e = n * 8 + threadIdx.x; e < kC * 8; e += 256)
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
    unsigned char* sm = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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
                if (n < kC) zero_rows(sm + kDOffZ + (i & 1) * kTile, n);
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
// Persistent: two CTAs per SM, each walking items blockIdx.x, blockIdx.x + gridDim.x, ...  The
// control warp loads the next step's Y and Z while the present one is worked on, and issues the
// next item's scores while the compute warps write out the present one's result.
// Compute warp (qw, kh): rows 32 qw .. + 31 (its tensor-memory lanes) and keys 64 kh .. + 63 of
// the scores, columns 32 kh .. + 31 of the output.
// ------------------------------------------------------------------------------------------
struct MixJob {
    CUtensorMap x, y, z, m, o;
    DecayJob j;
    int has_first;  // the chunk at the start of the scan has a state, too
    int items;      // of this job
};
struct MixJobs {
    MixJob job[3];
    int n;
};

constexpr int kMixThreads = 320;  // the compute warps, the control warp and one that looks ahead
constexpr int kAheadWarp = 9;

// What the compute warps need to know of an item, and the powers of l, prepared by the look-ahead
// warp while they work on the item before (two buffers, by the item's parity).  l^i is at
// pw[1 + i]: pairs that start at an odd power are 8-byte aligned.
struct MixInfo {
    __nv_bfloat16* out;    // the tile's first row
    const CUtensorMap* o;  // for the copy out; NULL: rows behind the sequence's end may not be written
    int n, nh, rev, has_m, t0, plane, garbage, none;
    float pw[132];
};

struct MixCtl {
    uint64_t x_full, m_full, yz_full[2], s_full, p_full, pv_done, x_free, out_free;
    uint64_t info_full[2], info_free[2];
    uint32_t tmem_base;
    int abort_flag;
};

constexpr uint32_t kMOffX = 0, kMOffYZ = kTile, kMOffM = 5 * kTile, kMOffO = kMOffM + kMTile;
constexpr uint32_t kMOffInfo = kMOffO + kTile;
constexpr uint32_t kMOffCtl = kMOffInfo + 2 * sizeof(MixInfo);
constexpr uint32_t kMixSmem = kMOffCtl + 128 + 1024;
constexpr uint32_t kMixTmem = 256;
constexpr uint32_t kColS = 0, kColU = 128, kColF = 192;
static_assert(sizeof(MixCtl) <= 128 && kMOffCtl % 8 == 0 && 2 * (kMixSmem + 1024) <= 233472,
              "two CTAs per SM");
static_assert(sizeof(MixInfo) % 16 == 0 && offsetof(MixInfo, pw) % 8 == 0, "alignment of pw");

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

// P = S o D for 32 rows (lane + 32 qw) and keys 64 kh .. + 63, written over the scores.
template <bool kRev>
__device__ __forceinline__ void decay_scores(uint32_t scores, const float* pw, int qw, int kh,
                                             int lane, int n)
{
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int jb = 2 * kh + half;  // keys 32 jb .. + 31
        uint32_t p[16];
        if (jb == qw) {  // the diagonal block
            float s[32];
            tmem_ld32(scores + 32 * half, s);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                const float d = pw[1 + ((kRev ? x - lane : lane - x) & 31)];
                s[x] = (kRev ? x >= lane && 32 * jb + x < n : x <= lane) ? s[x] * d : 0.f;
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) p[x] = pack_bf16x2(s[2 * x], s[2 * x + 1]);
        } else if (kRev ? jb > qw : jb < qw) {
            // l^|i-j| = l^(from the row to its block's edge) l^(from there to j)
            float s[32];
            tmem_ld32(scores + 32 * half, s);
            const float rf = pw[1 + (kRev ? 31 - lane : lane)];
            const float2 rf2 = make_float2(rf, rf);
            // the pair of columns (x, x + 1): powers at + x and at + x + 1 (kRev), or - x, - x - 1
            const float* at = kRev ? pw + 1 + 32 * (jb - qw) - 31 : pw + 1 + 32 * (qw - jb) - 1;
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
        tmem_st16(scores + 16 * half, p);  // over this warp's own scores, which it has read
    }
    tmem_st_wait();
}

__global__ void __launch_bounds__(kMixThreads, 2)
    mix_kernel(const __grid_constant__ MixJobs jobs, DecayShape S, int items)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    MixCtl& ctl = *reinterpret_cast<MixCtl*>(sm + kMOffCtl);
    MixInfo* infos = reinterpret_cast<MixInfo*>(sm + kMOffInfo);
    volatile int* abort_flag = &ctl.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(&ctl.x_full, 1);
        mbar_init(&ctl.m_full, 1);
        mbar_init(&ctl.s_full, 1);
        mbar_init(&ctl.p_full, 8);
        mbar_init(&ctl.pv_done, 1);
        mbar_init(&ctl.x_free, 1);
        mbar_init(&ctl.out_free, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.yz_full[i], 1);
            mbar_init(&ctl.info_full[i], 1);
            mbar_init(&ctl.info_free[i], 8);
        }
        ctl.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kCtrlWarp) {
        tmem_alloc(&ctl.tmem_base, kMixTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;

    if (warp < 8) {
        const int qw = warp & 3, kh = warp >> 2, row = 32 * qw + lane;
        const uint32_t lanes = tmem + (uint32_t(qw * 32) << 16);
        // the two warps of 32 rows agree once per item whether to go on: a wait that ran out in
        // one must not leave the other at their barrier
        for (int done = 0, step = 0;; ++done) {
            bool ok = wait_all(&ctl.info_full[done & 1], (done >> 1) & 1, abort_flag);
            const MixInfo& I = infos[done & 1];
            ok = ok && !I.none;
            const int n = I.n, nh = I.nh, rev = I.rev, has_m = I.has_m;
            for (int h = 0; ok && h < nh; ++h, ++step) {
                ok = wait_all(&ctl.s_full, step & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                if (rev) decay_scores<true>(lanes + kColS + 64 * kh, I.pw, qw, kh, lane, n);
                else decay_scores<false>(lanes + kColS + 64 * kh, I.pw, qw, kh, lane, n);
                tc_fence_before();
                if (I.garbage) {
                    // rows behind the sequence's end: zero times what lies there has to be zero
                    ok = wait_all(&ctl.yz_full[step & 1], (step >> 1) & 1, abort_flag);
                    if (!ok) break;
                    zero_rows(sm + kMOffYZ + (step & 1) * 2 * kTile + kTile, n);
                    fence_proxy_async();
                }
                warp_arrive(&ctl.p_full);
            }
            ok = ok && wait_all(&ctl.pv_done, (step - 1) & 1, abort_flag);
            if (lane == 0 && kh == 0) bulk_wait_read0();  // the copy before has read these rows
            if (!named_bar_and(1 + qw, 64, ok)) break;
            const float bi = rev ? (row < n ? I.pw[n - row] : 0.f) : S.scale * I.pw[row + 2];
            const uint32_t o = smem_u32(sm + kMOffO);
            const bool copied = I.o != nullptr;
            tc_fence_after();
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                float u[16], f[16];
                tmem_ld16(lanes + kColU + 32 * kh + 16 * part, u);
                if (has_m) tmem_ld16(lanes + kColF + 32 * kh + 16 * part, f);
                tmem_ld_wait();
                uint32_t p[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    float a = S.scale * u[2 * x], b = S.scale * u[2 * x + 1];
                    if (has_m) {
                        a = fmaf(bi, f[2 * x], a);
                        b = fmaf(bi, f[2 * x + 1], b);
                    }
                    p[x] = pack_bf16x2(a, b);
                }
                if (copied) {
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        sts128(o + kmajor_chunk(row, 4 * kh + 2 * part + x), p[4 * x], p[4 * x + 1],
                               p[4 * x + 2], p[4 * x + 3]);
                } else if (row < n) {
                    uint4* g = reinterpret_cast<uint4*>(I.out + row * kD + 32 * kh + 16 * part);
                    g[0] = make_uint4(p[0], p[1], p[2], p[3]);
                    g[1] = make_uint4(p[4], p[5], p[6], p[7]);
                }
            }
            tc_fence_before();
            warp_arrive(&ctl.out_free);
            if (copied) {
                fence_proxy_async();
                named_bar_sync(1 + qw, 64);
                if (lane == 0 && kh == 0 && 32 * qw < n) {
                    tma_store_3d(I.o, sm + kMOffO + qw * 32 * 128, 0, I.t0 + 32 * qw, I.plane);
                    bulk_commit();
                }
            }
            warp_arrive(&ctl.info_free[done & 1]);
        }
        if (lane == 0 && kh == 0) bulk_wait0();
    } else if (warp == kAheadWarp) {
        bool ok = true;
        for (int idx = blockIdx.x, done = 0; ok; idx += gridDim.x) {
            MixItem it;
            it.n = 0;
            for (; idx < items; idx += gridDim.x)
                if ((it = mix_item(jobs, S, idx)).n > 0) break;
            if (done >= 2) ok = wait_all(&ctl.info_free[done & 1], ((done >> 1) - 1) & 1, abort_flag);
            if (!ok) break;
            MixInfo& I = infos[done & 1];
            if (idx < items) {
                const MixJob& J = jobs.job[it.w];
                const float g = decay_log(S.log_decay, it.kv);
                for (int i = lane; i <= kC; i += 32) I.pw[1 + i] = decay_pow(g, i);
                if (lane == 0) {
                    const int left = S.T - it.c * kC, plane = it.b * J.j.hx + it.hx;
                    I.out = static_cast<__nv_bfloat16*>(J.j.out) +
                            (size_t(plane) * S.T + it.c * kC) * kD;
                    I.o = it.n == min(kC, left) ? &J.o : nullptr;
                    I.n = it.n;
                    I.nh = it.nh;
                    I.rev = J.j.rev;
                    I.has_m = it.has_m;
                    I.t0 = it.c * kC;
                    I.plane = plane;
                    I.garbage = it.n < kC && it.n < left;
                }
            }
            if (lane == 0) I.none = idx >= items;
            warp_arrive(&ctl.info_full[done & 1]);
            ++done;
            if (idx >= items) break;
        }
    } else if (lane == 0) {
        constexpr uint32_t id_s = idesc_bf16(128, 128, false, false);
        constexpr uint32_t id_mn = idesc_bf16(128, 64, false, true), id_k = idesc_bf16(128, 64, false, false);
        const uint32_t x = smem_u32(sm + kMOffX), m = smem_u32(sm + kMOffM);
        const uint32_t yz = smem_u32(sm + kMOffYZ);
        int nx = 0, nm = 0, nyz = 0, npv = 0, nfree = 0;
        auto load_x = [&](const MixItem& it) {
            const MixJob& J = jobs.job[it.w];
            mbar_expect_tx(&ctl.x_full, kTile);
            tma_load_3d(sm + kMOffX, &J.x, &ctl.x_full, 0, it.c * kC, it.b * J.j.hx + it.hx);
            ++nx;
        };
        auto load_m = [&](const MixItem& it) {
            if (!it.has_m) return;
            mbar_expect_tx(&ctl.m_full, kMTile);
            tma_load_2d(sm + kMOffM, &jobs.job[it.w].m, &ctl.m_full, 0,
                        ((it.b * S.Hkv + it.kv) * S.chunks + it.c) * 64);
            ++nm;
        };
        auto load_yz = [&](const MixItem& it, int h) {
            unsigned char* dst = sm + kMOffYZ + (nyz & 1) * 2 * kTile;
            uint64_t* bar = &ctl.yz_full[nyz & 1];
            const MixJob& J = jobs.job[it.w];
            const int plane = it.b * J.j.hy + it.y0 + h;
            mbar_expect_tx(bar, 2 * kTile);
            tma_load_3d(dst, &J.y, bar, 0, it.c * kC, plane);
            tma_load_3d(dst + kTile, &J.z, bar, 0, it.c * kC, plane);
            ++nyz;
        };
        auto next = [&](int& idx, MixItem& it) {
            for (; idx < items; idx += gridDim.x)
                if ((it = mix_item(jobs, S, idx)).n > 0) return true;
            return false;
        };
        int idx = blockIdx.x, step = 0, used_m = 0;
        MixItem it, nit;
        bool more = next(idx, it), ok = true;
        // the inputs were there before the kernels whose results this one waits for
        if (more) {
            load_x(it);
            load_yz(it, 0);
        }
        grid_dep_wait();
        if (more) load_m(it);
        for (int done = 0; more && ok; ++done) {
            int nidx = idx;
            bool nmore = false;
            ok = mbar_wait(&ctl.x_full, done & 1, abort_flag);
            for (int h = 0; h < it.nh && ok; ++h, ++step) {
                const bool last = h == it.nh - 1;
                ok = mbar_wait(&ctl.yz_full[step & 1], (step >> 1) & 1, abort_flag);
                if (!ok) break;
                const uint32_t y = yz + (step & 1) * 2 * kTile, z = y + kTile;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16(tmem + kColS, sdesc_sw128(x + ks * 32, 16, 1024),
                             sdesc_sw128(y + ks * 32, 16, 1024), id_s, ks > 0 ? 1u : 0u);
                mma_commit(&ctl.s_full);
                if (h == 0) nmore = next(nidx += gridDim.x, nit);  // while the scores are formed
                // the other stage is free: the products that read it are done
                if (!last) load_yz(it, h + 1);
                else if (nmore) load_yz(nit, 0);
                if (h == 0) {
                    // U and F of the item before have been read
                    if (done > 0) ok = mbar_wait(&ctl.out_free, (done - 1) & 1, abort_flag);
                    if (ok && it.has_m) {
                        ok = mbar_wait(&ctl.m_full, used_m & 1, abort_flag);
                        ++used_m;
                        if (ok) {
                            tc_fence_after();
                            const bool t = jobs.job[it.w].j.mem_t;
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_bf16(tmem + kColF, sdesc_sw128(x + ks * 32, 16, 1024),
                                         t ? sdesc_sw128(m + ks * 32, 16, 1024)
                                           : sdesc_sw128(m + ks * 2048, kTile, 1024),
                                         t ? id_k : id_mn, ks > 0 ? 1u : 0u);
                        }
                    }
                    if (!ok) break;
                }
                if (last) {
                    mma_commit(&ctl.x_free);  // no later MMA of the item reads X or M
                    ++nfree;
                }
                ok = mbar_wait(&ctl.p_full, step & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_bf16_ts(tmem + kColU, tmem + kColS + (ks < 4 ? 8 * ks : 64 + 8 * (ks - 4)),
                                sdesc_sw128(z + ks * 2048, kTile, 1024), id_mn,
                                (h > 0 || ks > 0) ? 1u : 0u);
                mma_commit(&ctl.pv_done);
                ++npv;
                if (last && nmore) {
                    ok = mbar_wait(&ctl.x_free, done & 1, abort_flag);
                    if (!ok) break;
                    load_x(nit);
                    load_m(nit);
                }
                // the next scores go over P, and the next loads over this step's Y and Z
                ok = mbar_wait(&ctl.pv_done, step & 1, abort_flag);
            }
            idx = nidx;
            it = nit;
            more = nmore;
        }
        // nothing of this CTA is in flight when it ends
        if (nx) bounded_spin_done(&ctl.x_full, (nx - 1) & 1);
        if (nm) bounded_spin_done(&ctl.m_full, (nm - 1) & 1);
        if (nyz) bounded_spin_done(&ctl.yz_full[(nyz - 1) & 1], ((nyz - 1) >> 1) & 1);
        if (nyz > 1) bounded_spin_done(&ctl.yz_full[nyz & 1], ((nyz - 2) >> 1) & 1);
        if (nfree) bounded_spin_done(&ctl.x_free, (nfree - 1) & 1);
        if (npv) bounded_spin_done(&ctl.pv_done, (npv - 1) & 1);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kCtrlWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kMixTmem);
    }
}

}  // namespace dtc
}  // namespace decay
}  // namespace oal
