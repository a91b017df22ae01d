// What the two tensor-core prefill kernels over an 8-bit cache share.
#pragma once

#include <algorithm>

#include "prefill_common.cuh"

namespace pa {

struct PrefillQ8Params : PrefillParams {
    const float* ks;
    const float* vs;
    int64_t ks_s0, ks_s1, vs_s0, vs_s1;
    int single;  // items of one query tile (always so beyond head_dim 128)
};

// An item of one query tile of qpt whole queries, with its key tiles of NT.
template <int NT>
__device__ __forceinline__ void pf_single_item(const PrefillParams& p, int qpt, PfItem& it) {
    it.q0 = p.cu_q[it.b];
    const int q1 = p.cu_q[it.b + 1];
    it.k0 = p.cu_k[it.b];
    const int k1 = p.cu_k[it.b + 1];
    it.sq = q1 - it.q0;
    it.sk = k1 - it.k0;
    it.bad = it.sq < 0 || it.sk < 0 || it.sq > p.max_sq || it.sk > p.max_sk || it.q0 < 0 || q1 > p.total_q;
    it.n_tiles = 0;
    it.has_b = 0;
    if (it.bad) return;
    it.i0 = it.u * qpt;
    const int i_last = min(it.sq - 1, it.i0 + qpt - 1);
    const int64_t cdiag = (int64_t)it.sk - it.sq;
    const int64_t lo = p.wl >= 0 ? max64(0, it.i0 + cdiag - p.wl) : 0;
    const int64_t hi = p.wr >= 0 ? min64((int64_t)it.sk - 1, i_last + cdiag + p.wr) : (int64_t)it.sk - 1;
    it.kt0 = hi >= lo ? (int)(lo & ~int64_t(NT - 1)) : 0;
    it.n_tiles = hi >= lo ? (int)((hi - it.kt0) / NT + 1) : 0;
}

// Upper bound of the query tiles per kv head, of 128 / G whole queries each: every sequence ends in one that
// may be part full.
inline int64_t prefill_q8_tiles(const Args& a) {
    const int64_t qpt = 128 / (a.H / a.Hkv);
    return std::min<int64_t>((a.total_q + qpt - 1) / qpt + a.batch, a.batch * ((a.max_sq + qpt - 1) / qpt));
}

// Whether a call's items have one query tile: head_dim beyond 128 has no room for two, and at most 128 two share
// their key tiles' loads and V's conversion, but where items of one would not fill the SMs either, a
// step of one is shorter (256 queries over 4,256 keys, 32 / 8 heads of 128: 79.9 to 70.3 us; eight times 64 over
// 1,064: 36.0 to 31.7).
inline bool prefill_q8_single(const Args& a, int num_sms) {
    return a.D > 128 || prefill_q8_tiles(a) * a.Hkv <= num_sms;
}

inline int device_sms() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
}

// The parameters of a call, for key tiles of `tile_keys`.
inline PrefillQ8Params prefill_q8_params(const Args& a, int* counter, unsigned int* err, int tile_keys, int num_sms) {
    PrefillQ8Params pp{};
    pp.counter = counter;
    pp.out = a.out;
    pp.o_s0 = a.o_s0;
    pp.o_s1 = a.o_s1;
    pp.lse = a.lse;
    pp.lse_s0 = a.lse_s0;
    pp.lse_sb = a.lse_sb;
    pp.cu_q = a.cu_q;
    pp.cu_k = a.cu_k;
    pp.bt = a.block_table;
    pp.bt_s0 = a.bt_s0;
    pp.bt_cols = a.bt_cols;
    pp.batch = a.batch;
    pp.H = a.H;
    pp.Hkv = a.Hkv;
    pp.G = a.H / a.Hkv;
    pp.D = a.D;
    pp.P = a.page;
    pp.num_blocks = a.num_blocks;
    pp.total_q = a.total_q;
    pp.paged = 1;
    pp.max_sq = a.max_sq;
    pp.max_sk = a.max_sk;
    pp.scale_log2 = a.scale * 1.4426950408889634f;
    pp.alibi = a.alibi;
    pp.wl = a.wl;
    pp.wr = a.wr;
    pp.rows_cap = prefill_rows_threshold();
    pp.err = err;
    pp.wait_ns = a.wait_ns;
    pp.withhold = a.withhold_loads;
    pp.box_rows = a.page % 128 == 0 && tile_keys == 128 ? 128 : a.page % 64 == 0 ? 64 : 32;
    pp.boxes_per_tile = tile_keys / pp.box_rows;
    pp.single = prefill_q8_single(a, num_sms);
    pp.pairs = (int)(pp.single ? prefill_q8_tiles(a) : prefill_items_bound(a) / a.Hkv);
    pp.ks = a.k_scale;
    pp.vs = a.v_scale;
    pp.ks_s0 = a.ks_s0;
    pp.ks_s1 = a.ks_s1;
    pp.vs_s0 = a.vs_s0;
    pp.vs_s1 = a.vs_s1;
    return pp;
}

}  // namespace pa
