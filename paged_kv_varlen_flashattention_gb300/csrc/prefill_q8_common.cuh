// What the two tensor-core prefill kernels over an 8-bit cache share on the host.
#pragma once

#include "prefill_common.cuh"

namespace pa {

struct PrefillQ8Params : PrefillParams {
    const float* ks;
    const float* vs;
    int64_t ks_s0, ks_s1, vs_s0, vs_s1;
};

// The parameters of a call, for key tiles of `tile_keys`.
inline PrefillQ8Params prefill_q8_params(const Args& a, int* counter, unsigned int* err, int tile_keys) {
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
    pp.pairs = (int)(prefill_items_bound(a) / a.Hkv);
    pp.ks = a.k_scale;
    pp.vs = a.v_scale;
    pp.ks_s0 = a.ks_s0;
    pp.ks_s1 = a.ks_s1;
    pp.vs_s0 = a.vs_s0;
    pp.vs_s1 = a.vs_s1;
    return pp;
}

}  // namespace pa
