// oal_decay.cuh -- shared definitions of linear attention with a decay per key/value head.
//
//     S_t = l S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,   l = exp(log_decay[kv head]) <= 1
//
// In chunks of C tokens (local index i, n tokens in the chunk), with S_c the state before it:
//     o_i     = scale (sum_{j<=i} l^(i-j) (q_i . k_j) v_j + l^(i+1) S_c^T q_i)
//     S_{c+1} = l^n S_c + sum_j l^(n-1-j) k_j v_j^T
// The gradients have the same form.  With R_c the sum over the tokens after chunk c,
//     dq_i = scale (sum_{j<=i} l^(i-j) (do_i . v_j) k_j + l^(i+1) S_c do_i)
//     dk_j = scale sum_{i>=j} l^(i-j) (v_j . do_i) q_i  + l^(n-1-j) R_c v_j
//     dv_j = scale sum_{i>=j} l^(i-j) (k_j . q_i) do_i  + l^(n-1-j) R_c^T k_j
//     R_{c-1} = l^n R_c + scale sum_i l^(i+1) q_i do_i^T,   R_last = dLoss/dS_last,
// dLoss/dS_0 being what the last of these steps leaves, and dk, dv and R summing over the query
// heads of a key/value head.  So three kernels serve every direction: the products y z^T of a
// chunk ("delta"), their scan over chunks, and the mix
//     u_i = a sum_h sum_j D_ij (x_i . y_hj) z_hj + b_i (x_i M  or  x_i M^T)
// with D_ij = l^|i-j| on one side of the diagonal and zero on the other.  A DecayJob names the
// arrays of one such mix; a gradient runs three of them.
#pragma once

#include "oal_common.cuh"
#include "oal_tc_util.cuh"

namespace oal {

constexpr int kDecayState = kD * kDV;  // fp32 values of one (b, kv) state

// One mix: x [B][hx][T][64] against y and z [B][hy][T][64], into out (x's layout).  Each x head
// takes hy / hx of the y heads (the gradients of a shared head), or hx / hy x heads share one.
struct DecayJob {
    const void* x;
    const void* y;
    const void* z;
    void* out;
    const void* mem;  // M of every (b, kv, chunk)
    int hx, hy;
    int rev;          // 0: j <= i and b_i = scale l^(i+1); 1: j >= i and b_i = l^(n-1-i)
    int mem_t;        // x M^T instead of x M
};

// One sum of products: E_c = sum_h sum_j w_j y_hj z_hj^T with w_j = l^(n-1-j) (rev = 0) or
// scale l^(j+1) (rev = 1), and its scan over the chunks: M_c before each chunk (rev = 0: the
// chunks before it, rev = 1: the chunks after it) and the total, starting from `first`.
struct DecaySum {
    const void* y;
    const void* z;
    int hy;
    int rev;
    int parts;           // the heads of a group are summed in so many parts, joined by the scan
    float* delta;        // [parts][B * Hkv][chunks][64][64]
    void* mem;           // [B * Hkv][chunks][64][64], fp32 (may be `delta`) or bf16
    const float* first;  // [B * Hkv][64][64], or NULL for zero
    float* last;         // the total, or NULL
};

struct DecayShape {
    int B, T, Hkv, chunks;
    const int32_t* lens;      // [B], or NULL: every sequence has T tokens
    const float* log_decay;   // [Hkv]
    float scale;
};

// log l of kv head: at most 0.  A positive or NaN entry is an error of the caller's that only the
// device sees.  exp(-1e4) is 0 in fp32, so that a decay of 0 (log -inf) keeps l^0 = 1.
__device__ __forceinline__ float decay_log(const float* log_decay, int kv)
{
    const float g = __ldg(log_decay + kv);
    if (!(g <= 0.f)) {
        raise_error(OAL_ERR_VALUE);
        return 0.f;
    }
    return fmaxf(g, -1e4f);
}

// l^m for m >= 0: exp of the exactly rounded product, corrected by its rounding error (m g has
// more digits than fp32 holds, and exp turns an absolute error into a relative one).
__device__ __forceinline__ float decay_pow(float g, int m)
{
    const float fm = float(m), p = fm * g;
    return expf(p) * (1.f + fmaf(fm, g, -p));
}

// The state before a chunk, as the mix multiplies it.  In bf16 it is rounded once, to the type of the
// q that it meets (states that are carried or returned stay in fp32): with the scores, rounded alike,
// an error of 0.0023 of the outputs' size where 32 bits and the rounding of the result alone make 0.0017.
// Scores and states in two bf16 parts each make 0.0017 too, at twelve more products an item: 8 x 4096
// tokens of 14/2 heads took 60.5 us then, 55.7 so, and the gradient of 4 x 4096 102 us, 87 so.
__device__ __forceinline__ void store_state(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store_state(__nv_bfloat16* p, float4 v)
{
    *reinterpret_cast<uint2*>(p) =
        make_uint2(tc::pack_bf16x2(v.x, v.y), tc::pack_bf16x2(v.z, v.w));
}

// The scan of a sequence of one chunk, done by the kernel that has the chunk's sum: entries e .. e + 3.
template <typename Tm>
__device__ __forceinline__ void scan_one(const DecaySum& J, int bkv, int e, float l, float4 sum)
{
    const size_t at = size_t(bkv) * kDecayState + e;
    float4 cur = make_float4(0.f, 0.f, 0.f, 0.f);
    if (J.first) cur = *reinterpret_cast<const float4*>(J.first + at);
    store_state(static_cast<Tm*>(J.mem) + at, cur);
    if (J.last)
        *reinterpret_cast<float4*>(J.last + at) =
            make_float4(fmaf(l, cur.x, sum.x), fmaf(l, cur.y, sum.y), fmaf(l, cur.z, sum.z),
                        fmaf(l, cur.w, sum.w));
}

// Tokens of sequence b.
__device__ __forceinline__ int decay_len(const DecayShape& s, int b)
{
    if (!s.lens) return s.T;
    const int n = __ldg(s.lens + b);
    if (n < 0 || n > s.T) {
        raise_error(OAL_ERR_VALUE);
        return n < 0 ? 0 : s.T;
    }
    return n;
}

}  // namespace oal
