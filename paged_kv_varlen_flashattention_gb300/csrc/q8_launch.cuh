// Host-side launch of the 8-bit cache's split-KV kernels for one element type of q and out.
// Included by one translation unit per type so the instantiations compile in parallel.
#pragma once

#include <cstdio>

#include "q8_decode.cuh"
#include "splitkv_launch.cuh"

namespace pa {

// Consumer warps, keys per tile and ring stages per padded head dim: two CTAs an SM with 96 KB of
// rings each.
template <int DP>
struct Q8Shape;
template <>
struct Q8Shape<64> {
    static constexpr int NW = 4, NT = 128, STAGES = 6;
};
template <>
struct Q8Shape<128> {
    static constexpr int NW = 4, NT = 128, STAGES = 3;
};

template <typename T, int DP, int MG>
struct Q8Kernel {
    using S = Q8Shape<DP>;
    using C = Q8Cfg<DP, MG, S::NW, S::NT, S::STAGES>;
    static constexpr int NT = S::NT;
    static auto kernel() { return decode_q8_kernel<T, DP, MG, S::NW, S::NT, S::STAGES>; }
};
template <typename T, int MG>
struct Q8Kernel<T, 256, MG> {
    using C = Q8WideCfg<256, MG>;
    static constexpr int NT = C::NT;
    static auto kernel() { return decode_q8_wide_kernel<T, 256, MG>; }
};
template <typename T, int MG>
struct Q8Kernel<T, 512, MG> {
    using C = Q8WideCfg<512, MG>;
    static constexpr int NT = C::NT;
    static auto kernel() { return decode_q8_wide_kernel<T, 512, MG>; }
};

template <typename T, int DP, int MG>
static int q8_occupancy_of() {
    using K = Q8Kernel<T, DP, MG>;
    static const int n = resident_ctas(K::kernel(), K::C::THREADS, K::C::SMEM);  // also sets the shared-memory size
    return n;
}

template <typename T, int DP, int MG>
static int run_q8(const CUtensorMap& tk, const CUtensorMap& tv, const Q8Params& sp, const SplitPlan& plan,
                  cudaStream_t stream, char* msg, size_t msg_len) {
    using K = Q8Kernel<T, DP, MG>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = set_shared_memory(K::kernel(), K::C::SMEM, configured);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "cudaFuncSetAttribute(q8 decode, %d bytes): %s", K::C::SMEM, cudaGetErrorString(e));
        return PA_ERR_CUDA;
    }
    if (sp.order) {
        const int rc = launch_longest_first(sp.cu_k, sp.batch, const_cast<int*>(sp.order), stream, msg, msg_len);
        if (rc != PA_OK) return rc;
    }
    if (sp.work) {
        NvtxRange nvw("pa::work_list_kernel");
        work_list_kernel<K::C::M, K::NT><<<1, kMaxOrderBatch, 0, stream>>>(sp, sp.work);
        if ((e = cudaGetLastError()) != cudaSuccess) {
            snprintf(msg, msg_len, "q8 work list launch: %s", cudaGetErrorString(e));
            return PA_ERR_CUDA;
        }
        count_launches(1);
    }
    const dim3 grid = sp.work ? dim3(plan.slots, 1, 1) : dim3(plan.max_splits, sp.Hkv * plan.row_tiles, sp.batch);
    {
        NvtxRange nv("pa::decode_q8_kernel");
        timer_begin(PA_KC_SPLITKV, stream);
        if (sp.cluster > 1) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(sp.cluster, sp.Hkv, sp.batch);
            cfg.blockDim = dim3(K::C::THREADS);
            cfg.dynamicSmemBytes = K::C::SMEM;
            cfg.stream = stream;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = sp.cluster;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaLaunchKernelEx(&cfg, K::kernel(), tk, tv, sp);
            if (e == cudaSuccess) e = cudaGetLastError();
        } else {
            K::kernel()<<<grid, K::C::THREADS, K::C::SMEM, stream>>>(tk, tv, sp);
            e = cudaGetLastError();
        }
        if (e != cudaSuccess) {
            snprintf(msg, msg_len, "q8 decode launch: %s", cudaGetErrorString(e));
            return PA_ERR_CUDA;
        }
        timer_end(PA_KC_SPLITKV, stream);
        count_launches(1);
    }
    if (plan.max_splits > 1) {
        const dim3 g2(((plan.tile_rows + kCombineRows - 1) / kCombineRows) * ((sp.D + 63) / 64), sp.Hkv * plan.row_tiles,
                      sp.batch);
        timer_begin(PA_KC_COMBINE, stream);
        if ((e = launch_combine<T, K::C::M, K::NT>(g2, sp, stream)) != cudaSuccess) {
            snprintf(msg, msg_len, "q8 combine launch: %s", cudaGetErrorString(e));
            return PA_ERR_CUDA;
        }
        timer_end(PA_KC_COMBINE, stream);
        count_launches(1);
    }
    return PA_OK;
}

template <typename T>
static int q8_occupancy_t(const SplitPlan& plan) {
    switch (plan.dp * 4 + plan.mt) {
        case 64 * 4 + 1: return q8_occupancy_of<T, 64, 1>();
        case 64 * 4 + 2: return q8_occupancy_of<T, 64, 2>();
        case 128 * 4 + 1: return q8_occupancy_of<T, 128, 1>();
        case 128 * 4 + 2: return q8_occupancy_of<T, 128, 2>();
        case 256 * 4 + 1: return q8_occupancy_of<T, 256, 1>();
        case 256 * 4 + 2: return q8_occupancy_of<T, 256, 2>();
        case 512 * 4 + 1: return q8_occupancy_of<T, 512, 1>();
        default: return q8_occupancy_of<T, 512, 2>();
    }
}

template <typename T>
static int launch_q8_t(const Args& a, const SplitPlan& plan, void* workspace, unsigned int* err, char* msg,
                       size_t msg_len) {
    const int NT = plan.nt;
    // box rows: the largest of {NT, 64, 32} that divides the page, so a box never straddles pages
    const int box_rows = a.page % NT == 0 ? NT : a.page % 64 == 0 && NT > 64 ? 64 : 32;
    const uint64_t dims[4] = {(uint64_t)a.D, (uint64_t)a.Hkv, (uint64_t)a.page, (uint64_t)a.num_blocks};
    const uint64_t strides[3] = {(uint64_t)a.kv_s2, (uint64_t)a.kv_s1, (uint64_t)a.kv_s0};
    const uint32_t box[4] = {(uint32_t)std::min(plan.dp, 128), 1u, (uint32_t)box_rows, 1u};
    CUtensorMap tk, tv;
    int rc = encode_tmap_4d(&tk, PA_E4M3, a.k, dims, strides, box, plan.dp == 64 ? 2 : 1, msg, msg_len);
    if (rc != PA_OK) return rc;
    rc = encode_tmap_4d(&tv, PA_E4M3, a.v, dims, strides, box, plan.dp == 64 ? 2 : 1, msg, msg_len);
    if (rc != PA_OK) return rc;
    Q8Params sp{};
    sp.q = a.q;
    sp.q_s0 = a.q_s0;
    sp.q_s1 = a.q_s1;
    sp.out = a.out;
    sp.o_s0 = a.o_s0;
    sp.o_s1 = a.o_s1;
    sp.lse = a.lse;
    sp.lse_s0 = a.lse_s0;
    sp.lse_sb = a.lse_sb;
    sp.cu_q = a.cu_q;
    sp.cu_k = a.cu_k;
    sp.bt = a.block_table;
    sp.bt_s0 = a.bt_s0;
    sp.bt_cols = a.bt_cols;
    sp.batch = a.batch;
    sp.H = a.H;
    sp.Hkv = a.Hkv;
    sp.G = a.H / a.Hkv;
    sp.D = a.D;
    sp.P = a.page;
    sp.num_blocks = a.num_blocks;
    sp.total_q = a.total_q;
    sp.paged = 1;
    sp.box_rows = box_rows;
    sp.boxes_per_tile = NT / box_rows;
    sp.max_sq = a.max_sq;
    sp.max_sk = a.max_sk;
    sp.scale_log2 = a.scale * 1.4426950408889634f;
    sp.alibi = a.alibi;
    sp.wl = a.wl;
    sp.wr = a.wr;
    sp.rows_cap = plan.rows_cap;
    sp.row_tiles = plan.row_tiles;
    sp.split_tiles = plan.split_tiles;
    sp.max_splits = plan.max_splits;
    sp.part_stride = a.total_q * a.H;
    if (plan.order_bytes) sp.order = static_cast<const int*>(workspace);
    if (plan.work_bytes) sp.work = reinterpret_cast<int*>(static_cast<char*>(workspace) + plan.order_bytes);
    sp.rank_in_cta = plan.rank_in_cta;
    if (plan.max_splits > 1) {
        sp.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.order_bytes + plan.work_bytes);
        sp.part_lse = sp.part_o + (size_t)plan.max_splits * sp.part_stride * a.D;
    }
    sp.err = err;
    sp.wait_ns = a.wait_ns;
    sp.withhold = a.withhold_loads;
    sp.cluster = plan.cluster;
    sp.ks = a.k_scale;
    sp.vs = a.v_scale;
    sp.ks_s0 = a.ks_s0;
    sp.ks_s1 = a.ks_s1;
    sp.vs_s0 = a.vs_s0;
    sp.vs_s1 = a.vs_s1;
    switch (plan.dp * 4 + plan.mt) {
        case 64 * 4 + 1: return run_q8<T, 64, 1>(tk, tv, sp, plan, a.stream, msg, msg_len);
        case 64 * 4 + 2: return run_q8<T, 64, 2>(tk, tv, sp, plan, a.stream, msg, msg_len);
        case 128 * 4 + 1: return run_q8<T, 128, 1>(tk, tv, sp, plan, a.stream, msg, msg_len);
        case 128 * 4 + 2: return run_q8<T, 128, 2>(tk, tv, sp, plan, a.stream, msg, msg_len);
        case 256 * 4 + 1: return run_q8<T, 256, 1>(tk, tv, sp, plan, a.stream, msg, msg_len);
        case 256 * 4 + 2: return run_q8<T, 256, 2>(tk, tv, sp, plan, a.stream, msg, msg_len);
        case 512 * 4 + 1: return run_q8<T, 512, 1>(tk, tv, sp, plan, a.stream, msg, msg_len);
        default: return run_q8<T, 512, 2>(tk, tv, sp, plan, a.stream, msg, msg_len);
    }
}

}  // namespace pa
