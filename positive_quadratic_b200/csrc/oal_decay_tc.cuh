// oal_decay_tc.cuh -- bf16 linear attention with a decay per key/value head on tensor cores: the
// products of a chunk and the mix (oal_decay.cuh), in chunks of 128 tokens.
//
// Every wait is bounded (1 s); one that runs out sets OAL_ERR_TIMEOUT and every role leaves its
// loop in order (copies drained, MMAs completed, tensor memory freed).
#pragma once

#include "oal_decay.cuh"

namespace oal {
namespace decay {
namespace dtc {

using namespace oal::tc;  // PTX layer

constexpr int kC = 128;
constexpr int kThreads = 288;   // of the delta kernel: 8 compute warps and a control warp
constexpr int kCtrlWarp = 8;
constexpr uint32_t kTile = kC * 128;      // a 128 x 64 bf16 tile
constexpr uint32_t kMTile = 64 * 128;     // a 64 x 64 bf16 state image

// tc::mbar_wait with its time limit taken from the SM's clock: a wait costs two or three
// instructions per poll.  (Reading the global timer takes about a thousand cycles, which every
// wait that does not succeed at once would pay before it looks again.)
constexpr long long kWaitLimitCycles = 2000000000ll;  // 1 s at 1.965 GHz

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag)
{
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (clock64() - t0 > kWaitLimitCycles) {
            *abort_flag = 1;
            raise_error(OAL_ERR_TIMEOUT);
            return false;
        }
    }
}

// The same by a whole warp.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag)
{
    return __all_sync(~0u, wait(bar, parity, abort_flag));
}

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

// MMAs from descriptors whose low words are at hand (the high word is the same for every tile here).
// One thread issues them all, at a few cycles an instruction, and the chain from one item to the next
// goes through it: forming each descriptor from an address again took it longer than the products.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // see tc::sdesc_sw128
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo)
{
    return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}
template <bool kAdd>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "n"(int(kAdd))
        : "memory");
}
template <bool kAdd>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(kDescHi), "r"(idesc), "n"(int(kAdd))
        : "memory");
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
// One CTA per (sum, part of the heads, b, kv, chunk); three fit an SM, since the high part is written
// over y itself.  It does little with each byte (48 KB a chunk), and is bound by the row of latencies
// from the copy over parts, products and tensor memory to the store, which the SM's other CTAs have to
// cover: 4 x 8192 tokens of 16 heads (4096 chunks, 201 MB) take 60 us, 3.3 TB/s; with two CTAs per
// SM it was 76 us.
// ------------------------------------------------------------------------------------------
struct SumMaps {
    CUtensorMap y[2], z[2];
};

struct DeltaCtl {
    uint64_t full, parts, done;
    uint32_t tmem_base;
    int abort_flag;
};

constexpr uint32_t kDOffLo = 0, kDOffY = kTile, kDOffZ = 3 * kTile;  // lo | y, then hi | mid | z
constexpr uint32_t kDOffCtl = 4 * kTile;
constexpr uint32_t kDeltaSmem = kDOffCtl + 128 + 1024;
constexpr uint32_t kDeltaTmem = 128;
static_assert(sizeof(DeltaCtl) <= 128 && 3 * (kDeltaSmem + 1024) <= 233472, "three CTAs per SM");

__global__ void __launch_bounds__(kThreads, 3)
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
        mbar_init(&ctl.full, 1);
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
                ok = wait_warp(&ctl.full, i & 1, abort_flag);
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
                if (n < kC) zero_rows<256>(sm + kDOffZ, n);
                fence_proxy_async();
                warp_arrive(&ctl.parts);
            }
            ok = ok && wait_warp(&ctl.done, (nh - 1) & 1, abort_flag);
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
                    const float4 sum = *reinterpret_cast<const float4*>(&stage[e >> 4][4 * (e & 15)]);
                    if (S.chunks > 1) out[e] = sum;
                    else scan_one<__nv_bfloat16>(J, bkv, 4 * e, decay_pow(decay_log(S.log_decay, kv), n), sum);
                }
                tc_fence_before();
            }
        } else if (lane == 0) {
            constexpr uint32_t id = idesc_bf16(128, 64, true, true);
            const CUtensorMap* my = &maps.y[which];
            const CUtensorMap* mz = &maps.z[which];
            const int plane = b * J.hy + kv * grp + h0;
            const uint32_t lo = smem_u32(sm + kDOffLo), z = smem_u32(sm + kDOffZ);
            int loads = 0, products = 0;
            auto load = [&](int i) {
                mbar_expect_tx(&ctl.full, 2 * kTile);
                tma_load_3d(sm + kDOffY, my, &ctl.full, 0, c * kC, plane + i);
                tma_load_3d(sm + kDOffZ, mz, &ctl.full, 0, c * kC, plane + i);
                ++loads;
            };
            load(0);
            for (int i = 0; i < nh; ++i) {
                if (!wait(&ctl.parts, i & 1, abort_flag)) break;
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const uint32_t a_lo = desc_lo(lo + (1 - g) * kTile, kTile), b_lo = desc_lo(z, kTile);
                    if (i > 0) mma_ss<true>(tmem + 64 * g, a_lo, b_lo, id);
                    else mma_ss<false>(tmem + 64 * g, a_lo, b_lo, id);
#pragma unroll
                    for (int ks = 1; ks < 8; ++ks)
                        mma_ss<true>(tmem + 64 * g, a_lo + 128 * ks, b_lo + 128 * ks, id);
                }
                mma_commit(&ctl.done);
                ++products;
                if (i + 1 < nh) {
                    if (!wait(&ctl.done, i & 1, abort_flag)) break;
                    load(i + 1);
                }
            }
            // nothing of this CTA is in flight when it ends
            bounded_spin_done(&ctl.full, (loads - 1) & 1);
            if (products) bounded_spin_done(&ctl.done, (products - 1) & 1);
        }
    }
    if (n <= 0 && S.chunks == 1 && warp < 8)
        for (int e = threadIdx.x; e < kDecayState / 4; e += 256)
            scan_one<__nv_bfloat16>(J, bkv, 4 * e, 1.f, make_float4(0.f, 0.f, 0.f, 0.f));
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
// Persistent: two CTAs per SM, each with a run of neighbouring items of about equal work.  The
// items of a job are ordered (b, chunk, kv, head of the group): query heads that share keys,
// values and a state follow one another, and Y, Z and M stay where they are for them.
// Warps 0-7 compute: warp (qw, kh) holds rows 32 qw .. + 31 (its tensor-memory lanes), keys
// 64 kh .. + 63 of the scores and columns 32 kh .. + 31 of the output.  Warp 8 issues the MMAs;
// the next item's scores are formed while the compute warps write out the present one's result.
// Warp 9 looks ahead: it works out the next items' places and powers of l and loads their tiles
// as soon as buffers are free.
// What bounds it is the chain of an item, about 4400 cycles from one to the next.  Measured parts:
// Q K^T 650; scores to P 1000 to 1500 (the latencies of tensor-memory loads and stores: a block
// behind the diagonal, a store alone, takes 430); P to the end of its products 900; from there to the
// next item's first MMA 700.  Scores, U and F fill 256 columns, so two such chains run per SM, and
// tensor memory has room for no third.
// 8 x 4096 tokens of 14/2 heads: 45 us, of a call of 57 us whose 134 MB are 21 us of memory.  Tried and
// not faster there (44 to 47 us at the time): 16 compute warps 48; two MMA warps taking turns 47; halves
// of 64 keys, so that products and decays overlap, 57; rows stored straight from registers cost 1200
// cycles an item in the shared-memory pipe.
// ------------------------------------------------------------------------------------------
struct MixJob {
    CUtensorMap x, y, z, m, o;
    DecayJob j;
    int has_first;  // the chunk at the start of the scan has a state, too
};
struct MixJobs {
    MixJob job[3];
    int n;
};

constexpr int kMixWarps = 8;  // compute warps
constexpr int kMixThreads = (kMixWarps + 2) * 32;
constexpr int kMmaWarp = kMixWarps, kAheadWarp = kMixWarps + 1;
constexpr int kInfos = 4;  // items that the look-ahead warp may have described and not seen done

// What the other warps need to know of an item, and a table of powers of l: entry kT0 + j is l^j
// (rev) or l^(127 - j), so that a row's factors l^|i-j| are read in the order of its keys whatever
// the direction; zeros follow where the other side of the diagonal begins.  Two copies, the second
// shifted by one place: rows at even and odd places both read aligned pairs (and, 16 banks apart,
// without conflicts).
constexpr int kT0 = 32, kTab = 208;
static_assert(kTab % 32 == 16, "the copies lie 16 banks apart");
struct MixInfo {
    __nv_bfloat16* out;    // the tile's first row
    const CUtensorMap* o;  // of the output; NULL: rows behind the sequence's end are not to be written
    int n, nh, rev, has_m, mem_t, t0, plane, garbage, none;
    int fresh, last;  // first, last item of a run that shares Y, Z and M
    int pad;
    float tab[2][kTab];
};

struct MixCtl {
    uint64_t x_full[2];            // an item's X has arrived (and its description, before)
    uint64_t x_free[2];            // its output has left the buffer, where it is staged
    uint64_t yz_full[2], m_full;
    uint64_t s_full, p_full;       // of a step
    uint64_t yz_free[2], m_free;   // the products that read them are done
    uint64_t item_done[2];         // every product of the item is done
    uint64_t info_full[kInfos], info_free[kInfos], drained;
    uint32_t tmem_base;
    int abort_flag;
};

constexpr uint32_t kMOffX = 0, kMOffYZ = 2 * kTile, kMOffM = 6 * kTile;
constexpr uint32_t kMOffInfo = kMOffM + kMTile;
constexpr uint32_t kMOffCtl = kMOffInfo + kInfos * sizeof(MixInfo);
constexpr uint32_t kMixSmem = kMOffCtl + 256 + 1024;
constexpr uint32_t kMixTmem = 256;
constexpr uint32_t kColS = 0, kColU = 128, kColF = 192;
static_assert(sizeof(MixCtl) <= 256 && kMOffCtl % 8 == 0 && 2 * (kMixSmem + 1024) <= 233472,
              "two CTAs per SM");
static_assert(sizeof(MixInfo) % 8 == 0 && offsetof(MixInfo, tab) % 8 == 0, "alignment of the table");
static_assert(kMixWarps * 2048 <= kTile, "output staging");

// A CTA's place in the work: item `i` of job w, at (b, chunk c, kv, head gi of the group).  Held by
// the look-ahead warp, whose lanes all carry the same values.
struct MixWalk {
    int w, i, items, b, c, kv, gi, len, n;
    long long left;  // work units of this CTA from the present item on

    __device__ __forceinline__ static int chunks_of(const DecayShape& S, int b)
    {
        return (decay_len(S, b) + kC - 1) / kC;
    }
    // chunks of all sequences
    __device__ __forceinline__ static int live_chunks(const DecayShape& S, int lane)
    {
        if (!S.lens) return S.B * S.chunks;
        int sum = 0;
        for (int b = lane; b < S.B; b += 32) sum += chunks_of(S, b);
        return __reduce_add_sync(~0u, sum);
    }
    // the place of the q-th chunk
    __device__ __forceinline__ void at_chunk(const DecayShape& S, int q, int lane)
    {
        if (!S.lens) {
            b = q / S.chunks;
            c = q % S.chunks;
        } else {
            b = 0;
            while (true) {  // 32 sequences at a time
                const int mine = b + lane < S.B ? chunks_of(S, b + lane) : 0;
                int upto = mine;
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(~0u, upto, o);
                    if (lane >= o) upto += x;
                }
                const uint32_t hit = __ballot_sync(~0u, upto > q);
                if (hit || b + 32 >= S.B) {
                    const int l = hit ? __ffs(hit) - 1 : 31;
                    c = q - __shfl_sync(~0u, upto - mine, l);
                    b += l;
                    break;
                }
                q -= __shfl_sync(~0u, upto, 31);
                b += 32;
            }
        }
        len = decay_len(S, b);
    }
    __device__ __forceinline__ static int heads(const DecayJob& j, int Hkv) { return j.hx / Hkv; }
    __device__ __forceinline__ static int steps(const DecayJob& j)
    {
        return j.hy > j.hx ? j.hy / j.hx : 1;
    }
    __device__ __forceinline__ void place(const MixJobs& jobs, const DecayShape& S, int lane)
    {
        const int grp = heads(jobs.job[w].j, S.Hkv);
        gi = i % grp;
        kv = i / grp % S.Hkv;
        at_chunk(S, i / grp / S.Hkv, lane);
    }
    // This CTA's share: the items that start within [total k / grid, total (k + 1) / grid).
    __device__ __forceinline__ void start(const MixJobs& jobs, const DecayShape& S, int lane)
    {
        const long long rows = (long long)live_chunks(S, lane) * S.Hkv;
        long long total = 0;
        for (int k = 0; k < jobs.n; ++k)
            total += rows * heads(jobs.job[k].j, S.Hkv) * steps(jobs.job[k].j);
        long long lo = total * blockIdx.x / gridDim.x;
        left = total * (blockIdx.x + 1) / gridDim.x - lo;
        for (w = 0;; ++w) {
            const int st = steps(jobs.job[w].j);
            items = int(rows * heads(jobs.job[w].j, S.Hkv));
            const long long first = (lo + st - 1) / st;
            if (first < items || w + 1 == jobs.n) {
                i = int(min(first, (long long)items));
                left -= first * st - lo;
                break;
            }
            // the next job's first item may start later than lo
            const long long over = (long long)items * st - lo;
            left -= max(over, 0ll);
            lo = max(-over, 0ll);
        }
        if (more()) place(jobs, S, lane);
    }
    __device__ __forceinline__ bool more() const { return left > 0 && i < items; }
    // To the next item; whether there is one.
    __device__ __forceinline__ void advance(const MixJobs& jobs, const DecayShape& S, int lane)
    {
        left -= steps(jobs.job[w].j);
        if (++i == items) {
            if (w + 1 == jobs.n) return;
            const int rows = items / heads(jobs.job[w].j, S.Hkv);
            ++w;
            i = 0;
            items = rows * heads(jobs.job[w].j, S.Hkv);
            if (more()) place(jobs, S, lane);
            return;
        }
        if (++gi < heads(jobs.job[w].j, S.Hkv)) return;
        gi = 0;
        if (++kv < S.Hkv) return;
        kv = 0;
        if (++c * kC < len) return;
        c = 0;
        do
            len = ++b < S.B ? decay_len(S, b) : 1;
        while (len == 0);
    }
};

// P = S o D for rows 32 qw + lane and keys 32 jb .. + 31, written over the scores.  Rounded once to bf16,
// as an operand of the next product has to be: formed and decayed in fp32, each term off by at most 2^-8
// of itself, the sums over them in fp32 (see store_state for what it comes to).
__device__ __forceinline__ void decay_scores(uint32_t scores, const MixInfo& I, int qw, int jb,
                                             int lane)
{
    const int rev = I.rev;
    const int ahead = rev ? jb - qw : qw - jb;  // blocks between the rows and the keys
    uint32_t p[16];
    if (ahead < 0) {
#pragma unroll
        for (int x = 0; x < 16; ++x) p[x] = 0u;
    } else {
        float s[32];
        tmem_ld32(scores, s);
        const int at = kT0 - lane + (rev ? 32 * ahead : 127 - 32 * ahead);
        const float* d = I.tab[at & 1] + at + (at & 1);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
            const float2 v = __fmul2_rn(make_float2(s[x], s[x + 1]),
                                        *reinterpret_cast<const float2*>(d + x));
            s[x] = v.x;
            s[x + 1] = v.y;
        }
        if (I.garbage) {
            // keys behind the sequence's end may be anything: their products are chosen to be zero,
            // as multiplied by zero they might be NaN
            const int left = I.n - 32 * jb;
            uint32_t live = left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1;
            if (ahead == 0) live &= rev ? ~0u << lane : ~0u >> (31 - lane);
#pragma unroll
            for (int x = 0; x < 32; ++x) s[x] = (live >> x) & 1 ? s[x] : 0.f;
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) p[x] = pack_bf16x2(s[2 * x], s[2 * x + 1]);
    }
    tmem_st16(scores, p);
}

__device__ __forceinline__ void tma_store_3d(const void* tmap, const void* src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
                 : "memory");
}

__global__ void __launch_bounds__(kMixThreads, 2)
    mix_kernel(const __grid_constant__ MixJobs jobs, DecayShape S)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = smem_raw + (-smem_u32(smem_raw) & 1023u);  // still known to be shared
    MixCtl& ctl = *reinterpret_cast<MixCtl*>(sm + kMOffCtl);
    MixInfo* infos = reinterpret_cast<MixInfo*>(sm + kMOffInfo);
    volatile int* abort_flag = &ctl.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(&ctl.m_full, 1);
        mbar_init(&ctl.m_free, 1);
        mbar_init(&ctl.drained, 1);
        mbar_init(&ctl.s_full, 1);
        mbar_init(&ctl.p_full, kMixWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.x_full[i], 1);
            mbar_init(&ctl.item_done[i], 1);
            mbar_init(&ctl.x_free[i], kMixWarps);
            mbar_init(&ctl.yz_full[i], 1);
            mbar_init(&ctl.yz_free[i], 1);
        }
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
        bool ok = wait_warp(&ctl.info_full[0], 0, abort_flag);
        for (int done = 0, step = 0, tile = -1; ok; ++done) {
            const MixInfo& I = infos[done % kInfos];
            if (I.none) break;
            const int n = I.n, nh = I.nh, rev = I.rev, has_m = I.has_m;
            for (int h = 0; h < nh; ++h, ++step) {
                ok = wait_warp(&ctl.s_full, step & 1, abort_flag);
                if (!ok) break;
                const bool fresh = h > 0 || I.fresh;  // another Y and Z than the step before
                tile += fresh;
                tc_fence_after();
#pragma unroll 1
                for (int jb = 2 * kh; jb < 2 * kh + 2; ++jb)
                    decay_scores(lanes + kColS + 32 * jb, I, qw, jb, lane);
                tmem_st_wait();
                tc_fence_before();
                if (I.garbage && fresh) {
                    // rows behind the sequence's end: zero times what lies there has to be zero
                    ok = wait_warp(&ctl.yz_full[tile & 1], (tile >> 1) & 1, abort_flag);
                    if (!ok) break;
                    zero_rows<kMixWarps * 32>(sm + kMOffYZ + (tile & 1) * 2 * kTile + kTile, n);
                    fence_proxy_async();
                }
                // P is there; and U and F of the item before have been read
                warp_arrive(&ctl.p_full);
            }
            if (!ok) break;
            const float bi = rev ? (row < n ? I.tab[0][kT0 + n - 1 - row] : 0.f)
                                 : S.scale * I.tab[0][kT0 + 126 - row];
            __nv_bfloat16* out = I.out + row * kD + 32 * kh;
            const CUtensorMap* o = I.o;
            const int t0 = I.t0 + 32 * qw, plane = I.plane;
            // the next item's description has been there for long: looked for here, where there is
            // time
            ok = wait_warp(&ctl.info_full[(done + 1) % kInfos], ((done + 1) / kInfos) & 1, abort_flag) &&
                 wait_warp(&ctl.item_done[done & 1], (done >> 1) & 1, abort_flag);
            if (!ok) break;
            warp_arrive(&ctl.info_free[done % kInfos]);
            tc_fence_after();
            float u[32];
            tmem_ld32(lanes + kColU + 32 * kh, u);
            if (has_m) {
                float f[32];
                tmem_ld32(lanes + kColF + 32 * kh, f);
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    const float2 v = __ffma2_rn(make_float2(bi, bi), make_float2(f[x], f[x + 1]),
                                                __fmul2_rn(make_float2(S.scale, S.scale),
                                                           make_float2(u[x], u[x + 1])));
                    u[x] = v.x;
                    u[x + 1] = v.y;
                }
            } else {
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 32; ++x) u[x] *= S.scale;
            }
            tc_fence_before();
            uint32_t p[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) p[x] = pack_bf16x2(u[2 * x], u[2 * x + 1]);
            if (o) {
                // this warp's 32 x 32 tile goes out as one copy, staged (64-byte swizzle) where the
                // item's X was
                unsigned char* tile_out = sm + kMOffX + (done & 1) * kTile + warp * 2048;
                const uint32_t at = smem_u32(tile_out) + lane * 64, sw = (lane >> 1) & 3;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    sts128(at + ((x ^ sw) << 4), p[4 * x], p[4 * x + 1], p[4 * x + 2], p[4 * x + 3]);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    if (32 * qw < n) {
                        tma_store_3d(o, tile_out, 32 * kh, t0, plane);
                        bulk_commit();
                        bulk_wait_read0();
                    }
                    mbar_arrive(&ctl.x_free[done & 1]);
                }
            } else {
                if (row < n)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        reinterpret_cast<uint4*>(out)[x] =
                            make_uint4(p[4 * x], p[4 * x + 1], p[4 * x + 2], p[4 * x + 3]);
                warp_arrive(&ctl.x_free[done & 1]);
            }
        }
        if (lane == 0) bulk_wait0();
    } else if (warp == kAheadWarp) {
        int nx = 0, nm = 0, nyz = 0;
        bool ok = true, waited = false, fresh = true;
        MixWalk at;
        at.start(jobs, S, lane);
        for (int done = 0;; ++done) {
            if (done >= kInfos)
                ok = wait_warp(&ctl.info_free[done % kInfos], (done / kInfos - 1) & 1, abort_flag);
            if (!ok) break;
            MixInfo& I = infos[done % kInfos];
            if (!at.more()) {
                if (lane == 0) {
                    I.none = 1;
                    if (nx >= 2)
                        ok = wait(&ctl.x_free[nx & 1], ((nx >> 1) - 1) & 1, abort_flag);
                    if (ok) mbar_arrive(&ctl.x_full[nx & 1]);
                }
                warp_arrive(&ctl.info_full[done % kInfos]);
                break;
            }
            const MixJob& J = jobs.job[at.w];
            const int grp = MixWalk::heads(J.j, S.Hkv), nh = MixWalk::steps(J.j);
            const int b = at.b, c = at.c, kv = at.kv, hx = kv * grp + at.gi, left = S.T - c * kC;
            const int plane = b * J.j.hx + hx;
            const int y0 = b * J.j.hy + (nh > 1 ? hx * nh : J.j.hy == J.j.hx ? hx : kv);
            const int n = min(kC, at.len - c * kC);
            const bool has_m = c != (J.j.rev ? (at.len - 1) / kC : 0) || J.has_first;
            const bool shares = nh == 1 && J.j.hy < J.j.hx;  // the group's heads share Y, Z and M
            const float g = decay_log(S.log_decay, kv);
            const bool first = fresh;
            const int gi = at.gi;
            at.advance(jobs, S, lane);
            const bool last = !shares || gi + 1 == grp || !at.more();
#pragma unroll 1
            for (int e = lane; e < 6 * 32; e += 32) {
                const int m = J.j.rev ? e - kT0 : 127 - (e - kT0);
                const float l = m >= 0 && m <= kC ? decay_pow(g, m) : 0.f;
                I.tab[0][e] = l;
                I.tab[1][e + 1] = l;
            }
            if (lane == 0) {
                I.out = static_cast<__nv_bfloat16*>(J.j.out) + (size_t(plane) * S.T + c * kC) * kD;
                I.o = n == min(kC, left) ? &J.o : nullptr;
                I.t0 = c * kC;
                I.plane = plane;
                I.n = n;
                I.nh = nh;
                I.rev = J.j.rev;
                I.has_m = has_m;
                I.mem_t = J.j.mem_t;
                I.garbage = n < kC && n < left;
                I.none = 0;
                I.fresh = first;
                I.last = last;
            }
            warp_arrive(&ctl.info_full[done % kInfos]);
            fresh = last;
            if (lane == 0) {
                if (nx >= 2) ok = wait(&ctl.x_free[nx & 1], ((nx >> 1) - 1) & 1, abort_flag);
                if (ok) {
                    uint64_t* bar = &ctl.x_full[nx & 1];
                    mbar_expect_tx(bar, kTile);
                    tma_load_3d(sm + kMOffX + (nx & 1) * kTile, &J.x, bar, 0, c * kC, plane);
                    ++nx;
                }
                auto load_yz = [&](int h) {
                    if (nyz >= 2)
                        ok = wait(&ctl.yz_free[nyz & 1], ((nyz >> 1) - 1) & 1, abort_flag);
                    if (!ok) return;
                    unsigned char* dst = sm + kMOffYZ + (nyz & 1) * 2 * kTile;
                    uint64_t* bar = &ctl.yz_full[nyz & 1];
                    mbar_expect_tx(bar, 2 * kTile);
                    tma_load_3d(dst, &J.y, bar, 0, c * kC, y0 + h);
                    tma_load_3d(dst + kTile, &J.z, bar, 0, c * kC, y0 + h);
                    ++nyz;
                };
                if (ok && first) load_yz(0);
                // (the inputs were there before the kernels whose results this one waits for)
                if (!waited) grid_dep_wait();
                waited = true;
                if (ok && first && has_m) {
                    if (nm >= 1) ok = wait(&ctl.m_free, (nm - 1) & 1, abort_flag);
                    if (ok) {
                        mbar_expect_tx(&ctl.m_full, kMTile);
                        tma_load_2d(sm + kMOffM, &J.m, &ctl.m_full, 0,
                                    ((b * S.Hkv + kv) * S.chunks + c) * 64);
                        ++nm;
                    }
                }
                for (int h = 1; ok && h < nh; ++h) load_yz(h);
            }
            ok = __shfl_sync(~0u, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
        }
        if (lane == 0) {
            if (!waited) grid_dep_wait();
            // no copy is in flight when the CTA ends: the MMA warp has waited for each, unless
            // this warp gave up
            for (int k = 1; !ok && k <= 2; ++k) {
                if (nx >= k) bounded_spin_done(&ctl.x_full[(nx - k) & 1], ((nx - k) >> 1) & 1);
                if (nyz >= k) bounded_spin_done(&ctl.yz_full[(nyz - k) & 1], ((nyz - k) >> 1) & 1);
            }
            if (!ok && nm) bounded_spin_done(&ctl.m_full, (nm - 1) & 1);
        }
    } else if (lane == 0) {
        constexpr uint32_t id_s = idesc_bf16(128, 128, false, false);
        constexpr uint32_t id_mn = idesc_bf16(128, 64, false, true), id_k = idesc_bf16(128, 64, false, false);
        // low words of the descriptors; the other buffer's is kTile / 16 further on
        const uint32_t x0 = desc_lo(smem_u32(sm + kMOffX), 16);
        const uint32_t y0 = desc_lo(smem_u32(sm + kMOffYZ), 16);
        const uint32_t z0 = desc_lo(smem_u32(sm + kMOffYZ + kTile), kTile);
        const uint32_t m0 = desc_lo(smem_u32(sm + kMOffM), kTile);
        int nm = 0, step = 0, tile = -1;
        bool ok = true;
        // Every wait and every commit of this thread costs a few hundred cycles of the chain from
        // one item to the next, so it has few: three waits and two commits for an item of one step
        // that shares its tiles with the item before.
        // What it can look at early (the next item's description and whether its X is there), it
        // looks at while the compute warps work on the scores.
        struct Next {
            int none, nh, has_m, mem_t, first, last;
        };
        auto read = [&](int k) {
            const MixInfo& I = infos[k % kInfos];
            return Next{I.none, I.nh, I.has_m, I.mem_t, I.fresh, I.last};
        };
        ok = wait(&ctl.x_full[0], 0, abort_flag);
        Next it = read(0);
        bool ready = true;  // X of the present item has been seen
        for (int done = 0; ok; ++done) {
            if (!ready) {
                ok = wait(&ctl.x_full[done & 1], (done >> 1) & 1, abort_flag);
                it = read(done);
            }
            if (!ok || it.none) break;
            const Next now = it;
            ready = false;
            const uint32_t x = x0 + (done & 1) * (kTile / 16);
            for (int h = 0; ok && h < now.nh; ++h, ++step) {
                if (h > 0 || now.first) {
                    ++tile;
                    ok = wait(&ctl.yz_full[tile & 1], (tile >> 1) & 1, abort_flag);
                }
                // the scores go over P of the step before
                if (ok && h > 0) ok = wait(&ctl.yz_free[(tile - 1) & 1], ((tile - 1) >> 1) & 1, abort_flag);
                else if (ok && done > 0)
                    ok = wait(&ctl.item_done[(done - 1) & 1], ((done - 1) >> 1) & 1, abort_flag);
                if (!ok) break;
                const uint32_t y = y0 + (tile & 1) * (2 * kTile / 16);
                const uint32_t z = z0 + (tile & 1) * (2 * kTile / 16);
                mma_ss<false>(tmem + kColS, x, y, id_s);
#pragma unroll
                for (int ks = 1; ks < 4; ++ks) mma_ss<true>(tmem + kColS, x + 2 * ks, y + 2 * ks, id_s);
                mma_commit(&ctl.s_full);
                if (h == 0 && now.has_m && now.first) {
                    ok = wait(&ctl.m_full, nm & 1, abort_flag);
                    ++nm;
                    if (!ok) break;
                }
                if (h == now.nh - 1 &&
                    mbar_try_wait(&ctl.x_full[(done + 1) & 1], ((done + 1) >> 1) & 1)) {
                    ready = true;
                    it = read(done + 1);
                }
                ok = wait(&ctl.p_full, step & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                if (h > 0) mma_ts<true>(tmem + kColU, tmem + kColS, z, id_mn);
                else mma_ts<false>(tmem + kColU, tmem + kColS, z, id_mn);
#pragma unroll
                for (int ks = 1; ks < 8; ++ks)
                    mma_ts<true>(tmem + kColU, tmem + kColS + 32 * (ks >> 1) + 8 * (ks & 1),
                                 z + 128 * ks, id_mn);
                if (h == 0 && now.has_m) {
                    const uint32_t id = now.mem_t ? id_k : id_mn, by = now.mem_t ? 2 : 128;
                    mma_ss<false>(tmem + kColF, x, m0, id);
#pragma unroll
                    for (int ks = 1; ks < 4; ++ks) mma_ss<true>(tmem + kColF, x + 2 * ks, m0 + by * ks, id);
                    if (now.last) mma_commit(&ctl.m_free);
                }
                if (h == now.nh - 1) mma_commit(&ctl.item_done[done & 1]);
                if (h < now.nh - 1 || now.last) mma_commit(&ctl.yz_free[tile & 1]);
            }
        }
        // every MMA has completed before tensor memory is freed (a commit covers all before it)
        mma_commit(&ctl.drained);
        bounded_spin_done(&ctl.drained, 0);
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
