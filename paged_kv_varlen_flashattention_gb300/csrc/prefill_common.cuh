// What the tensor-core prefill kernels share: their parameters, the work item, the bounded wait
// of a role, and the transpose of an epilogue's quads.
#pragma once

#include "tc_common.cuh"

namespace pa {

struct PrefillParams {
    void* out;
    int64_t o_s0, o_s1;
    float* lse;
    int64_t lse_s0, lse_sb;  // lse of (head h, token t, sequence b) at h lse_s0 + t + b lse_sb
    const int32_t* cu_q;
    const int32_t* cu_k;
    const int32_t* bt;
    int64_t bt_s0;
    int bt_cols;
    int batch, H, Hkv, G, D, P;
    int64_t num_blocks, total_q;
    int paged;
    int box_rows, boxes_per_tile;
    int max_sq, max_sk;
    float scale_log2;
    int wl, wr;
    const float* alibi;  // per-query-head slopes of the linear position bias, or nullptr
    int rows_cap;
    int pairs;     // an upper bound of the number of work units (tile pairs or tiles) per kv head
    int* counter;  // the take counter of (work unit, kv head) items, zeroed before the launch
    unsigned int* err;
    uint64_t wait_ns;  // bound on every wait
    int withhold;      // test hook: issue no loads
};

// Bounded wait that also gives up as soon as another role of the CTA has aborted.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                         unsigned int* err, uint64_t limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > limit_ns) {
            *abort_flag = 1u;
            flag_error(err, PA_ERR_DEVICE_TIMEOUT);
            return false;
        }
    }
}

// 4 x 4 transpose of 32-bit values over the four threads of a quad (t = lane % 4): thread t
// holds a[j] = M[t][j] on entry and a[j] = M[j][t] on exit.  Two butterfly stages: lanes t and
// t ^ 1 swap the odd/even entries of each pair, then lanes t and t ^ 2 swap the pairs.
__device__ __forceinline__ void quad_transpose(uint32_t (&a)[4], int t) {
    const bool b = t & 1, h = t & 2;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint32_t r = __shfl_xor_sync(0xffffffffu, b ? a[2 * c] : a[2 * c + 1], 1);
        if (b) a[2 * c] = r; else a[2 * c + 1] = r;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t r = __shfl_xor_sync(0xffffffffu, h ? a[e] : a[2 + e], 2);
        if (h) a[e] = r; else a[2 + e] = r;
    }
}

// The work of one item.  Warp 0 computes it and publishes it in a slot; every role reads it.
struct PfItem {
    int b, u, hk, q0, sq, sk, k0, i0, kt0, n_tiles, has_b, bad;
};
static_assert(sizeof(PfItem) <= 64, "item slot");

__device__ __forceinline__ void pf_item(const PrefillParams& p, int qpt, PfItem& it) {
    it.q0 = p.cu_q[it.b];
    const int q1 = p.cu_q[it.b + 1];
    it.k0 = p.cu_k[it.b];
    const int k1 = p.cu_k[it.b + 1];
    it.sq = q1 - it.q0;
    it.sk = k1 - it.k0;
    it.bad = it.sq < 0 || it.sk < 0 || it.sq > p.max_sq || it.sk > p.max_sk || it.q0 < 0 || q1 > p.total_q ||
             (!p.paged && (it.k0 < 0 || k1 > p.num_blocks));
    it.n_tiles = 0;
    if (it.bad) return;
    it.i0 = it.u * 2 * qpt;
    it.has_b = it.i0 + qpt < it.sq;
    const int i_last = min(it.sq - 1, it.i0 + (it.has_b ? 2 : 1) * qpt - 1);
    const int64_t cdiag = (int64_t)it.sk - it.sq;
    const int64_t lo = p.wl >= 0 ? max64(0, it.i0 + cdiag - p.wl) : 0;
    const int64_t hi = p.wr >= 0 ? min64((int64_t)it.sk - 1, i_last + cdiag + p.wr) : (int64_t)it.sk - 1;
    it.kt0 = hi >= lo ? (int)(lo & ~int64_t(127)) : 0;
    it.n_tiles = hi >= lo ? (int)((hi - it.kt0) / 128 + 1) : 0;
}

}  // namespace pa
