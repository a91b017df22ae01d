// Tensor-core prefill / chunked prefill over an 8-bit paged cache (sm_103a), head_dim <= 128.
//
// The structure of prefill_kernel (prefill_tc.cu): one persistent CTA per SM takes items of two
// 128-row query tiles (A, B) of one (sequence, kv head) from a device counter, so every K/V
// tile feeds both; S, P and O live in tensor memory.  What the 8-bit cache changes:
//
//  * Q.K^T runs on the 8-bit tensor cores with K as it is in the cache (no conversion, half the
//    shared memory).  q is written as a sum of e4m3 terms, q 2^e = t0 + t1 [+ t2], each the
//    rounding of what the ones before leave, and the terms' products accumulate in the same S.
//    A term takes 4 significant bits and its remainder is at most half its last place, so two
//    terms hold bf16's 8 bits and three hold f16's 11; e, a power of two per row, brings the row's
//    largest magnitude to 224..448, so what a term cannot hold (half of e4m3's smallest step, 2^-10)
//    is at most 2^-17.8 of that largest.  An 8-bit product takes half the time of a 16-bit one, so two terms cost what
//    one bf16 product does.
//  * P.V runs on f16: converter warps read the V tiles as TMA leaves them, turn the codes into
//    f16 (exact) in the layout the matrix unit reads, and zero the rows of keys that no row of
//    the item attends (0 x NaN is NaN).  P is f16 too, in every call.
//  * A page's scales enter the softmax as in q8_decode.cuh: x = c ks s + log2 vs, weights
//    2^(x - m + 7), l = sum of weights / vs, per group of 32 keys (pages are multiples of 32).
//    The reference m is raised only when some x is more than 8 above it, so weights are at most
//    2^15, within f16.
//
// Roles (512 threads, four warpgroups):
//   warp 0       takes items and publishes them; K tiles and their scales
//   warp 2       V tiles
//   warps 1, 3   MMA issuers of tiles A and B
//   warps 4..11  softmax, a row (TMEM lane) a thread: 4..7 tile A, 8..11 tile B
//   warps 12..15 converters: q into its terms at the start of an item, then V tile by tile
//
// Tensor-core bound: 4 D flops per (row, key) at the f16 rate (f16 q: 5 D).
#include <algorithm>
#include <cfloat>
#include <cstdio>
#include <type_traits>

#include "prefill_q8_common.cuh"
#include "q8_common.cuh"
#include "rope_common.cuh"

namespace pa {
namespace {

constexpr int kPqThreads = 512;
// Register split (setmaxnreg) of the launch's 512 x 128: control 96, softmax 152, converters 112:
// 128 x 96 + 256 x 152 + 128 x 112 = 65,536.  (56 / 192 / 72 spilled in the issuers: 7 % slower.)
constexpr int kPqRegsControl = 96, kPqRegsSoftmax = 152, kPqRegsConvert = 112;
constexpr float kPqOffset = 7.f;

// DP: padded head dim, 64 or 128 (rows of the 8-bit tiles are 128 bytes either way, zero filled
// past the head dim); NTERM: e4m3 terms of q.
template <int DP, int NTERM>
struct PqCfg {
    static constexpr int TILE = 128 * 128;  // a q term, a K tile, a V tile as loaded
    static constexpr int KS = NTERM == 2 ? 3 : 2, VR = 2;
    static constexpr int VC_TILE = (DP / 64) * TILE;  // a V tile in f16
    static constexpr int OFF_Q = 0;                   // tile x, term t at (x NTERM + t) TILE
    static constexpr int OFF_K = 2 * NTERM * TILE;
    static constexpr int OFF_VR = OFF_K + KS * TILE;
    static constexpr int OFF_VC = OFF_VR + VR * TILE;
    static constexpr int OFF_BAR = OFF_VC + 2 * VC_TILE;
    // q_raw[2], q_full[2], q_free[2], k_full[KS], k_empty[KS], vr_full[VR], vr_empty[VR], vc_full[2],
    // vc_empty[2], s_full[2], p_full[2], pv_done[2], drain[2], item_ready[2], item_free[2]
    static constexpr int NBAR = 6 + 2 * KS + 2 * VR + 16;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;  // tmem base, abort flag
    static constexpr int OFF_SLOT = OFF_MISC + 16;       // two item slots
    static constexpr int SC_RING = 8;
    static constexpr int OFF_SC = OFF_SLOT + 128;        // [K ring position % 8]: ks[4], log2 vs[4], 1 / vs[4]
    static constexpr int OFF_EXP = OFF_SC + SC_RING * 48;  // [item parity][tile][row]: e of the row, int8
    static constexpr int SMEM = OFF_EXP + 512 + 1024;
    static constexpr uint32_t T_S0 = 0, T_S1 = 128, T_O0 = 256, T_O1 = 256 + DP;
    // The scale ring: the K producer writes position g after stage g % KS was released, once both
    // tiles' S of g - KS were seen; S of a tile follows the P of the one before from all its softmax
    // warps, so each is at g - KS - 1 or later, and what is overwritten (g - 8) has been read.
    static_assert(KS + 1 < SC_RING, "scale ring");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <typename T, int DP, bool ALIBI>
__global__ void __launch_bounds__(kPqThreads, 1)
    prefill_q8_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PrefillQ8Params p) {
    constexpr int NTERM = std::is_same<T, __half>::value ? 3 : 2;
    using C = PqCfg<DP, NTERM>;
    constexpr int KS = C::KS, VR = C::VR;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    uint64_t* q_raw = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [tile]: q as loaded
    uint64_t* q_full = q_raw + 2;   // [tile]: q in its terms
    uint64_t* q_free = q_full + 2;  // [tile]: the item's Q.K^T products have completed
    uint64_t* k_full = q_free + 2;
    uint64_t* k_empty = k_full + KS;
    uint64_t* vr_full = k_empty + KS;
    uint64_t* vr_empty = vr_full + VR;
    uint64_t* vc_full = vr_empty + VR;
    uint64_t* vc_empty = vc_full + 2;
    uint64_t* s_full = vc_empty + 2;       // [tile]
    uint64_t* p_full = s_full + 2;         // [tile]
    uint64_t* pv_done = p_full + 2;        // [tile]
    uint64_t* drain = pv_done + 2;         // [issuer]
    uint64_t* item_ready = drain + 2;      // [slot]
    uint64_t* item_free = item_ready + 2;  // [slot]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    PfItem* slots = reinterpret_cast<PfItem*>(smem + C::OFF_SLOT);
    float* sc_ring = reinterpret_cast<float*>(smem + C::OFF_SC);
    int8_t* row_exp = reinterpret_cast<int8_t*>(smem + C::OFF_EXP);
    if (tid == 64) {
        for (int s = 0; s < KS; ++s) {
            mbar_init(&k_full[s], 2);   // the copies, the scales
            mbar_init(&k_empty[s], 2);  // one arrive per query tile: the softmax, or issuer B without a tile B
        }
        for (int s = 0; s < VR; ++s) {
            mbar_init(&vr_full[s], 1);
            mbar_init(&vr_empty[s], 4);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_raw[x], 1);
            mbar_init(&q_full[x], 4);  // converter warps
            mbar_init(&q_free[x], 1);
            mbar_init(&vc_full[x], 4);
            mbar_init(&vc_empty[x], 2);
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 4);  // softmax warps of the tile
            mbar_init(&pv_done[x], 1);
            mbar_init(&drain[x], 1);
            mbar_init(&item_ready[x], 1);
            mbar_init(&item_free[x], 15);  // the V producer, two issuers, eight softmax warps, four converters
        }
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int qpt = 128 / p.G;    // whole queries per 128-row tile
    const int trows = qpt * p.G;  // rows of a tile that hold queries
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        const bool r = __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, p.err, p.wait_ns));
        tc::fence_after_sync();
        return r;
    };
    auto take_slot = [&](int k, PfItem& it) -> bool {
        if (!wait_all(&item_ready[k & 1], (k >> 1) & 1)) return false;
        it = slots[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_free[k & 1]);
        return true;
    };
    // First key of step j of an item.  Under a bias the nearest keys come first: the score falls with
    // the distance, so the reference stands from the first tiles on; in ascending order it would grow,
    // and the accumulator be rescaled, at almost every tile (256 queries over 4,256 keys, 15 heads of
    // 96: 121 us in ascending order, 109 so; unbiased 81).
    auto tile_key = [&](const PfItem& it, int j) { return it.kt0 + (ALIBI ? it.n_tiles - 1 - j : j) * 128; };
    // The item's key tiles into the K ring (with the scales of each tile's four 32-key groups) or the V
    // ring.  Lane i holds the block id (and scales) of box i of a window of 32 boxes.
    auto produce = [&](const PfItem& it, const CUtensorMap* map, uint8_t* ring, uint64_t* fullb, uint64_t* emptyb,
                       int stages, int g0, bool scales) -> bool {
        const int32_t* bt_row = p.bt + (int64_t)it.b * p.bt_s0;
        const int bpt = p.boxes_per_tile, win_tiles = 32 / bpt;
        int jw = -win_tiles, id = -1;
        float ksc = 0.f, vsc = 0.f;
        for (int j = 0; j < it.n_tiles; ++j) {
            if (j >= jw + win_tiles) {
                jw = j;
                const int jl = j + lane / bpt;
                const int key = jl < it.n_tiles ? tile_key(it, jl) + lane % bpt * p.box_rows : it.sk;
                id = box_block(bt_row, p.bt_cols, p.num_blocks, p.P, key, it.sk, p.err);
                if (scales && id >= 0) {
                    ksc = __ldg(p.ks + (int64_t)id * p.ks_s0 + (int64_t)it.hk * p.ks_s1);
                    vsc = __ldg(p.vs + (int64_t)id * p.vs_s0 + (int64_t)it.hk * p.vs_s1);
                }
            }
            const int g = g0 + j, s = g % stages;
            if (g >= stages && !wait_all(&emptyb[s], ((g / stages) - 1) & 1)) return false;
            int blk[4];
            uint32_t bytes = 0;
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                const int b = __shfl_sync(0xffffffffu, id, ((j - jw) * bpt + jj) & 31);
                blk[jj] = jj < bpt ? b : -1;
                if (blk[jj] >= 0) bytes += (uint32_t)(p.box_rows * 128);
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&fullb[s], bytes);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    if (blk[jj] < 0) continue;
                    const int key = tile_key(it, j) + jj * p.box_rows;
                    tma_load_4d(ring + s * C::TILE + jj * p.box_rows * 128, map, &fullb[s], 0, it.hk,
                                key - (key / p.P) * p.P, blk[jj], 0ull);
                }
            }
            __syncwarp();
            if (scales) {  // after the copies are on their way: the gather's latency runs beside theirs
                const int src = (j - jw) * bpt + ((lane & 3) * 32) / p.box_rows;
                const float a = __shfl_sync(0xffffffffu, ksc, src), v = __shfl_sync(0xffffffffu, vsc, src);
                if (lane < 4) {
                    float* slot = sc_ring + (g % C::SC_RING) * 12 + lane;
                    const float lv = v > 7.8886090522101181e-31f ? fminf(log2f(v), 126.f) : (float)kScaleExpMin;
                    slot[0] = a;
                    slot[4] = lv;
                    slot[8] = exp2f(-lv);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&fullb[s]);
            }
        }
        return true;
    };

    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPqRegsControl));
    if (warp == 0) {
        // ---------------- item taker, K producer ----------------
        // Items as in prefill_kernel: w = pair * Hkv + kv head, each sequence's last pair first.
        const int total = p.pairs * p.Hkv;
        const int per = p.single ? qpt : 2 * qpt;  // queries of an item
        if (!p.withhold) prefetch_tmap(&tm_k);
        int w_next = lane == 0 ? atomicAdd(p.counter, 1) : 0;
        int gk = 0;
        for (int k = 0;; ++k) {
            const int w = __shfl_sync(0xffffffffu, w_next, 0);
            PfItem it{};
            it.b = -1;
            if (w < total) {
                const int pair = w / p.Hkv;
                it.hk = w - pair * p.Hkv;
                int remaining = pair;
                for (int base = 0; base < p.batch && it.b < 0; base += 32) {
                    const int bb = base + lane;
                    int pairs = 0;
                    if (bb < p.batch) {
                        const int sqb = p.cu_q[bb + 1] - p.cu_q[bb];
                        pairs = (int64_t)sqb * p.G > p.rows_cap ? (sqb + per - 1) / per : 0;
                    }
                    int incl = pairs;
#pragma unroll
                    for (int off = 1; off < 32; off <<= 1) {
                        const int v = __shfl_up_sync(0xffffffffu, incl, off);
                        if (lane >= off) incl += v;
                    }
                    const unsigned hit = __ballot_sync(0xffffffffu, remaining < incl);
                    if (hit) {
                        const int src = __ffs(hit) - 1;
                        const int excl = __shfl_sync(0xffffffffu, incl - pairs, src);
                        const int cnt = __shfl_sync(0xffffffffu, pairs, src);
                        it.b = base + src;
                        it.u = cnt - 1 - (remaining - excl);
                    } else {
                        remaining -= __shfl_sync(0xffffffffu, incl, 31);
                    }
                }
                if (it.b >= 0) {
                    if (p.single)
                        pf_single_item<128>(p, qpt, it);
                    else
                        pf_item(p, qpt, it);
                }
            }
            if (it.b >= 0 && lane == 0) w_next = atomicAdd(p.counter, 1);
            if (k >= 2 && !wait_all(&item_free[k & 1], ((k >> 1) - 1) & 1)) break;
            if (lane == 0) {
                slots[k & 1] = it;
                mbar_arrive(&item_ready[k & 1]);
            }
            if (it.b < 0) break;
            if (it.bad) {
                if (lane == 0) flag_error(p.err, PA_ERR_DEVICE_BOUNDS);
                continue;
            }
            if (it.n_tiles == 0) continue;
            if (!p.withhold && !produce(it, &tm_k, smem + C::OFF_K, k_full, k_empty, KS, gk, true)) break;
            gk += it.n_tiles;
        }
    } else if (warp == 2) {
        // ---------------- V producer ----------------
        if (!p.withhold) prefetch_tmap(&tm_v);
        int gv = 0;
        for (int k = 0;; ++k) {
            PfItem it;
            if (!take_slot(k, it) || it.b < 0) break;
            if (it.bad || it.n_tiles == 0) continue;
            if (!p.withhold && !produce(it, &tm_v, smem + C::OFF_VR, vr_full, vr_empty, VR, gv, false)) break;
            gv += it.n_tiles;
        }
    } else {
        // ---------------- MMA issuers: warp 1 for tile A, warp 3 for tile B ----------------
        constexpr uint32_t IDESC_S = tc::idesc_e4m3(128, 128);
        constexpr uint32_t IDESC_O = tc::idesc_f16(128, DP, false, false, true);
        const int x = warp == 1 ? 0 : 1;
        const uint64_t da = tc::smem_desc_sw128(smem_addr(smem + C::OFF_Q + x * NTERM * C::TILE), 16, 1024);
        const uint64_t dk0 = tc::smem_desc_sw128(smem_addr(smem + C::OFF_K), 16, 1024);
        const uint64_t dv0 = tc::smem_desc_sw128(smem_addr(smem + C::OFF_VC), C::TILE, 1024);
        const uint32_t d_s = tmem + (x ? C::T_S1 : C::T_S0);
        const uint32_t d_o = tmem + (x ? C::T_O1 : C::T_O0);
        int lq = 0, gk = 0, gv = 0, sx = 0;
        bool ok = true;
        auto issue_s = [&](int g) {  // S_x = (sum of q terms) K^T of the K tile at ring position g
            const uint64_t db = dk0 + (uint64_t)((g % KS) * (C::TILE >> 4));
#pragma unroll
            for (int t = 0; t < NTERM; ++t)
#pragma unroll
                for (int kk = 0; kk < DP / 32; ++kk)
                    tc::mma_f8_ss_elect(d_s, da + (uint64_t)(t * (C::TILE >> 4) + kk * 2), db + (uint64_t)(kk * 2), IDESC_S,
                                        t + kk > 0 ? 1u : 0u);
            tc::commit_elect(&s_full[x]);
        };
        for (int k = 0; ok; ++k) {
            PfItem it;
            if (!take_slot(k, it) || it.b < 0) break;
            if (it.bad || it.n_tiles == 0) continue;
            const int n = it.n_tiles;
            if (!(ok = wait_all(&q_full[x], lq & 1))) break;
            if (x == 0 || it.has_b) {
                if (!(ok = wait_all(&k_full[gk % KS], (gk / KS) & 1))) break;
                issue_s(gk);
                if (n == 1) tc::commit_elect(&q_free[x]);
                __syncwarp();
                for (int j = 0; ok && j < n; ++j) {
                    const int g_v = gv + j;
                    if (!(ok = wait_all(&vc_full[g_v & 1], (g_v >> 1) & 1))) break;
                    const bool more = j + 1 < n;
                    const int g_k = gk + j + 1;
                    if (more && !(ok = wait_all(&k_full[g_k % KS], (g_k / KS) & 1))) break;
                    if (!(ok = wait_all(&p_full[x], (sx + j) & 1))) break;
                    const uint64_t db = dv0 + (uint64_t)((g_v & 1) * (C::VC_TILE >> 4));
                    const uint32_t first = j > 0 ? 1u : 0u;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        tc::mma_ts_elect(d_o, d_s + kk * 8, db + (uint64_t)(kk * (2048 / 16)), IDESC_O, kk > 0 ? 1u : first);
                    if (j + 1 == n) tc::commit_elect(&pv_done[x]);
                    if (more) {
                        issue_s(g_k);
                        if (j + 2 == n) tc::commit_elect(&q_free[x]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                sx += n;
            } else {
                // An item without tile B: this issuer goes through the same phases and releases its
                // share of q and of every stage.  Were it to skip them, its next wait could meet
                // a barrier whose phase before that one has yet to complete, and pass at once.
                if (lane == 0) mbar_arrive(&q_free[x]);
                for (int j = 0; ok && j < n; ++j) {
                    if (!(ok = wait_all(&k_full[(gk + j) % KS], ((gk + j) / KS) & 1))) break;
                    if (lane == 0) mbar_arrive(&k_empty[(gk + j) % KS]);
                    if (!(ok = wait_all(&vc_full[(gv + j) & 1], ((gv + j) >> 1) & 1))) break;
                    if (lane == 0) mbar_arrive(&vc_empty[(gv + j) & 1]);
                }
                if (!ok) break;
            }
            __syncwarp();
            gk += n;
            gv += n;
            ++lq;
        }
        if (lane == 0) {
            tc::commit(&drain[x]);
            mbar_wait(&drain[x], 0, p.wait_ns);  // not cut short by an abort: MMAs may be in flight
        }
        __syncwarp();
    }
    } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPqRegsConvert));
    {
        // ---------------- converters ----------------
        const int cw = warp - 12;
        if (cw == 0 && !p.withhold) prefetch_tmap(&tm_q);
        int ld = 0, gv = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            PfItem it;
            if (!take_slot(k, it) || it.b < 0) break;
            if (it.bad || it.n_tiles == 0) continue;
            // q: tile x is loaded over the terms of the item before once its last Q.K^T products have
            // completed (a step before the item ends: the load and the conversion run beside its
            // last softmax and its epilogue), the 128-byte chunks of a row into that row of terms 0
            // and 1, and converted in place, DP / 8 lanes a row.
            for (int x = 0; ok && x < 2; ++x) {
                if (ld >= 1 && !(ok = wait_all(&q_free[x], (ld - 1) & 1))) break;
                if (cw == 0 && lane == 0 && !p.withhold) {
                    if (x == 0 || it.has_b) {
                        mbar_arrive_expect_tx(&q_raw[x], (DP / 64) * trows * 128);
                        for (int c = 0; c < DP / 64; ++c)
                            tma_load_4d(smem + C::OFF_Q + (x * NTERM + c) * C::TILE, &tm_q, &q_raw[x], c * 64, it.hk * p.G,
                                        it.q0 + it.i0 + x * qpt, 0, 0ull);
                    } else {
                        mbar_arrive(&q_raw[x]);
                    }
                }
                __syncwarp();
            }
            for (int x = 0; ok && x < 2; ++x) {
                if (!(ok = wait_all(&q_raw[x], ld & 1))) break;
                if (x == 0 || it.has_b) {
                    constexpr int LPR = DP / 8, RPP = 32 / LPR;  // lanes of a row, rows of a pass
                    const int u = lane % LPR;
                    uint8_t* tile = smem + C::OFF_Q + x * (NTERM * C::TILE);
                    constexpr int NB = 2;  // rows of a lane whose chains of shuffles and roundings overlap
#pragma unroll 1
                    for (int i0 = 0; i0 < 32 / RPP; i0 += NB) {
                        uint4 w[NB];
                        float mx[NB];
#pragma unroll
                        for (int i = 0; i < NB; ++i) {
                            const int r = cw * 32 + (i0 + i) * RPP + lane / LPR;
                            w[i] = *reinterpret_cast<const uint4*>(tile + (u >> 3) * C::TILE + swz128(r, u & 7));
                        }
#pragma unroll
                        for (int i = 0; i < NB; ++i) {
                            const float2 f0 = unpack2<T>(w[i].x), f1 = unpack2<T>(w[i].y), f2 = unpack2<T>(w[i].z),
                                         f3 = unpack2<T>(w[i].w);
                            mx[i] = max3f(max3f(fabsf(f0.x), fabsf(f0.y), fabsf(f1.x)),
                                          max3f(fabsf(f1.y), fabsf(f2.x), fabsf(f2.y)), fmaxf(fabsf(f3.x), fabsf(f3.y)));
                        }
#pragma unroll
                        for (int off = LPR / 2; off > 0; off >>= 1)
#pragma unroll
                            for (int i = 0; i < NB; ++i) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], off));
                        __syncwarp();  // every lane of these rows has read its columns
#pragma unroll
                        for (int i = 0; i < NB; ++i) {
                            const int r = cw * 32 + (i0 + i) * RPP + lane / LPR;
                            // the largest power of two with mx 2^e2 <= 448 = 1.75 x 2^8
                            const int bits = __float_as_int(mx[i]);
                            const int e2 = min(126, 8 - ((bits >> 23) - 127) - ((bits & 0x7fffff) > 0x600000 ? 1 : 0));
                            // (a row with an infinite element becomes NaN, and so do its scores)
                            const float up = mx[i] <= FLT_MAX ? __int_as_float((127 + e2) << 23) : NAN;
                            const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                            uint32_t c2[NTERM][4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float2 y = unpack2<T>(ww[e]);
                                y.x *= up;
                                y.y *= up;
#pragma unroll
                                for (int t = 0; t < NTERM; ++t) {
                                    c2[t][e] = e4m3x2(y.x, y.y);
                                    if (t + 1 < NTERM) {
                                        const float2 f = unpack2<__half>(e4m3x2_to_half2(c2[t][e]));
                                        y.x -= f.x;
                                        y.y -= f.y;
                                    }
                                }
                            }
                            uint8_t* dst = tile + swz128(r, u >> 1) + (u & 1) * 8;
#pragma unroll
                            for (int t = 0; t < NTERM; ++t)
                                *reinterpret_cast<uint2*>(dst + t * C::TILE) =
                                    make_uint2(c2[t][0] | (c2[t][1] << 16), c2[t][2] | (c2[t][3] << 16));
                            if (u == 0) row_exp[(ld & 1) * 256 + x * 128 + r] = (int8_t)e2;
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[x]);
            }
            if (!ok) break;
            // V tiles: warp cw converts rows 32 cw .. + 31
            const int64_t cdiag = (int64_t)it.sk - it.sq;
            const int i_last = min(it.sq - 1, it.i0 + (it.has_b ? 2 : 1) * qpt - 1);
            const int key_lo = p.wl >= 0 ? (int)max64(0, it.i0 + cdiag - p.wl) : 0;
            const int key_hi = p.wr >= 0 ? (int)min64((int64_t)it.sk - 1, i_last + cdiag + p.wr) : it.sk - 1;
            for (int j = 0; j < it.n_tiles; ++j) {
                const int g = gv + j, s = g % VR, c = g & 1;
                if (!(ok = wait_all(&vr_full[s], (g / VR) & 1))) break;
                if (g >= 2 && !(ok = wait_all(&vc_empty[c], ((g >> 1) - 1) & 1))) break;
                const uint8_t* src = smem + C::OFF_VR + s * C::TILE;
                uint8_t* dst = smem + C::OFF_VC + c * C::VC_TILE;
                const int kt = tile_key(it, j);
                constexpr int UPR = DP / 16;          // 16-byte units of a row
                constexpr int RPP = 32 / UPR;         // rows a warp converts a pass
                const int uu = lane % UPR;
                uint8_t* d = dst + (uu >> 2) * C::TILE;
                const int u0 = (uu & 3) * 2;
                const bool sw = (uu & 4) != 0;
#pragma unroll 1
                for (int i = 0; i < 32 / RPP; ++i) {
                    const int r = cw * 32 + i * RPP + lane / UPR;
                    uint4 v = *reinterpret_cast<const uint4*>(src + swz128(r, uu));
                    if (kt + r < key_lo || kt + r > key_hi) v = make_uint4(0, 0, 0, 0);
                    uint4 a, b;
                    a.x = e4m3x2_to_half2(v.x);
                    a.y = e4m3x2_hi_to_half2(v.x);
                    a.z = e4m3x2_to_half2(v.y);
                    a.w = e4m3x2_hi_to_half2(v.y);
                    b.x = e4m3x2_to_half2(v.z);
                    b.y = e4m3x2_hi_to_half2(v.z);
                    b.z = e4m3x2_to_half2(v.w);
                    b.w = e4m3x2_hi_to_half2(v.w);
                    *reinterpret_cast<uint4*>(d + swz128(r, u0 + (sw ? 1 : 0))) = sw ? b : a;
                    *reinterpret_cast<uint4*>(d + swz128(r, u0 + (sw ? 0 : 1))) = sw ? a : b;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&vc_full[c]);
                    mbar_arrive(&vr_empty[s]);
                }
            }
            if (!ok) break;
            gv += it.n_tiles;
            ++ld;
        }
    }
    } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPqRegsSoftmax));
    {
        // ---------------- softmax: warps 4..7 for tile A, 8..11 for tile B ----------------
        // Thread t of warp w holds row (TMEM lane) 32 (w % 4) + t with all 128 keys of a tile, so a row
        // needs no exchange, and the two warps of a scheduler, one of each tile, are at different
        // points of their steps: one's exponentials run under the other's loads and waits.  On eight
        // prompts of 1024..8192 tokens: 1,596 us (1,546 with the later steps); with all eight warps on tile A and then on tile B, two
        // rows and 64 keys of each a thread, as in prefill_kernel, 1,793; with sixteen warps, half a row a
        // thread, 1,750.
        const int x = (warp - 4) >> 2;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_addr + (x ? C::T_S1 : C::T_S0);
        const uint32_t o_addr = tmem + lane_addr + (x ? C::T_O1 : C::T_O0);
        T* out = static_cast<T*>(p.out);
        const int qi = row / p.G, gi = row - qi * p.G;  // query of the tile, head of the group
        const bool pad = row >= trows;
        int gk = 0, gv = 0, sx = 0, px = 0, ld = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            PfItem it;
            if (!take_slot(k, it) || it.b < 0) break;
            if (it.bad) continue;
            const int qrow = it.i0 + x * qpt + qi;  // query of the sequence
            const bool live = !pad && qrow < it.sq;
            const int h = it.hk * p.G + gi;
            const int64_t t_row = (int64_t)it.q0 + qrow;
            T* orow = out + t_row * p.o_s0 + (int64_t)h * p.o_s1;
            float* lse = p.lse + (int64_t)h * p.lse_s0 + t_row + (int64_t)it.b * p.lse_sb;
            if (it.n_tiles == 0) {  // no row attends any key: out = 0, lse = -inf
                if (live) {
                    for (int d = 0; d < p.D; d += 8) *reinterpret_cast<int4*>(orow + d) = make_int4(0, 0, 0, 0);
                    *lse = -INFINITY;
                }
                continue;
            }
            const int n = it.n_tiles;
            if (x == 1 && !it.has_b) {
                gk += n;
                gv += n;
                ++ld;
                continue;
            }
            const int64_t diag = qrow + ((int64_t)it.sk - it.sq);
            const int lo = p.wl >= 0 ? (int)max64(0, diag - p.wl) : 0;
            // (rows past the tile's queries keep the mask of the query they would be: one that is empty
            // would send their whole warp through the masked path at every tile: 81 to 138 us)
            const int hi = p.wr >= 0 ? (int)max64(-1, min64((int64_t)it.sk - 1, diag + p.wr)) : it.sk - 1;
            const float ab = ALIBI && live ? p.alibi[h] * kLog2e : 0.f;
            float m = -INFINITY, l = 0.f, sl = 0.f;

            // One key tile: S -> running reference -> (rare) O rescale -> P.
            auto step = [&](int j) -> bool {
                const int kt = tile_key(it, j);
                if (!__all_sync(0xffffffffu, wait_bar(&s_full[x], (sx + j) & 1, abort_flag, p.err, p.wait_ns))) return false;
                tc::fence_after_sync();
                const float* slot = sc_ring + ((gk + j) % C::SC_RING) * 12;
                if (j == 0) sl = p.scale_log2 * __int_as_float((127 - row_exp[(ld & 1) * 256 + x * 128 + row]) << 23);
                const bool masked = kt < lo || kt + 127 > hi;
                // Scores of keys 64 hb .. + 63 (two groups); rolled over the halves, and read from tensor
                // memory once for the maximum and once for the weights, to keep the code small: the
                // four warps of a scheduler run three different roles, and 1.4 of their 9 cycles per
                // instruction went to instruction fetches with straight-line code for 128 keys.
                auto load_half = [&](int hb, float(&v)[2][32]) {
                    tc::ld_32cols(s_addr + 64 * hb, v[0]);
                    tc::ld_32cols(s_addr + 64 * hb + 32, v[1]);
                    tc::wait_ld();
                    if (masked) {
#pragma unroll
                        for (int g = 0; g < 2; ++g)
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const int key = kt + 64 * hb + 32 * g + i;
                                v[g][i] = key >= lo && key <= hi ? v[g][i] : -INFINITY;
                            }
                    }
                };
                // c and log2 vs of group 2 hb + g (c positive: -inf x c stays -inf under a scale of 0)
                auto scales = [&](int hb, int g, float& c, float& lv) {
                    c = fmaxf(sl * slot[2 * hb + g], 1e-37f);
                    lv = slot[4 + 2 * hb + g];
                };
                // the whole x of a biased score: x = c v - ab |diag - key| + add, two keys at a time where
                // no row has live keys on both sides of its own position (the same call: 144 us key by key)
                const bool above = kt >= diag;
                const bool one_sided = ALIBI && __all_sync(0xffffffffu, above || kt + 127 <= diag || hi <= diag);
                auto bias = [&](int hb, int g, float c, float add, float(&v)[32]) {
                    float d0 = (float)((int)diag - kt - 64 * hb - 32 * g);
                    if (one_sided) {
                        const float na = above ? ab : -ab;
                        float d1 = d0 - 1.f;
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            ffma2(v[i], v[i + 1], v[i], v[i + 1], c, c, add, add);
                            ffma2(v[i], v[i + 1], d0, d1, na, na, v[i], v[i + 1]);
                            fadd2_acc(d0, d1, -2.f, -2.f);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = fmaf(-ab, fabsf(d0 - (float)i), fmaf(v[i], c, add));
                    }
                };
                float mx = -INFINITY;
#pragma unroll 1
                for (int hb = 0; hb < 2; ++hb) {
                    float v[2][32];
                    load_half(hb, v);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        float c, lv;
                        scales(hb, g, c, lv);
                        if (ALIBI) bias(hb, g, c, lv, v[g]);
                        float t0 = fmaxf(v[g][0], v[g][1]), t1 = fmaxf(v[g][2], v[g][3]);
#pragma unroll
                        for (int i = 4; i < 32; i += 4) {
                            t0 = max3f(t0, v[g][i], v[g][i + 1]);
                            t1 = max3f(t1, v[g][i + 2], v[g][i + 3]);
                        }
                        t0 = fmaxf(t0, t1);
                        mx = fmaxf(mx, ALIBI ? t0 : fmaf(t0, c, lv));
                    }
                }
                // S is complete, and so is the P.V before it: their stages are free.  (Told here, not as
                // soon as S is seen, and not by the issuers' own commits: the copies and the
                // conversion that follow then fall beside the second pass; 8 % and 15 % faster.)
                if ((warp & 3) == 0 && lane == 0) {
                    mbar_arrive(&k_empty[(gk + j) % KS]);
                    if (j > 0) mbar_arrive(&vc_empty[(gv + j - 1) & 1]);
                }
                const bool grow = mx > m + 8.f;
                if (__any_sync(0xffffffffu, grow)) {
                    const float alpha = grow ? fast_exp2(m - mx) : 1.f;
                    if (grow) m = mx;
                    l *= alpha;
                    // the tile's last P.V precedes S(j) on its issuer: complete now
                    if (j > 0) {
#pragma unroll 1
                        for (int cc = 0; cc < DP / 16; ++cc) {
                            uint32_t o[16];
                            tc::ld_32x32b_x16(o_addr + cc * 16, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tc::st_32x32b_x16(o_addr + cc * 16, o);
                        }
                    }
                }
                const float nm = m == -INFINITY ? 0.f : kPqOffset - m;
#pragma unroll 1
                for (int hb = 0; hb < 2; ++hb) {
                    float v[2][32];
                    load_half(hb, v);
                    uint32_t pk[32];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        float c, lv;
                        scales(hb, g, c, lv);
                        if (ALIBI) bias(hb, g, c, lv, v[g]);
                        const float cg = ALIBI ? 1.f : c, ag = ALIBI ? nm : nm + lv;
                        float s0 = 0.f, s1 = 0.f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x0, x1;
                            ffma2(x0, x1, v[g][2 * i], v[g][2 * i + 1], cg, cg, ag, ag);
                            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                            fadd2_acc(s0, s1, p0, p1);
                            pk[16 * g + i] = pack2<__half>(p0, p1);
                        }
                        l = fmaf(s0 + s1, slot[8 + 2 * hb + g], l);
                    }
                    // P of these keys over columns whose S has been read (the first half's)
                    tc::st_32x32b_x32(s_addr + 32 * hb, pk);
                }
                tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[x]);
                return true;
            };
#pragma unroll 1
            for (int j = 0; ok && j < n; ++j) ok = step(j);
            if (ok) ok = __all_sync(0xffffffffu, wait_bar(&pv_done[x], px & 1, abort_flag, p.err, p.wait_ns));
            if (ok) {
                tc::fence_after_sync();
                if ((warp & 3) == 0 && lane == 0) mbar_arrive(&vc_empty[(gv + n - 1) & 1]);
                const float inv_l = l == 0.f ? 0.f : 1.f / l;
                if (live) *lse = l == 0.f ? -INFINITY : (m - kPqOffset + log2f(l)) * 0.69314718055994531f;
#pragma unroll 1
                for (int cc = 0; cc < DP / 32; ++cc) {  // 64 bytes of the row a pass
                    float o[32];
                    tc::ld_32cols(o_addr + cc * 32, o);
                    tc::wait_ld();
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int d = cc * 32 + v * 8;
                        if (live && d < p.D)
                            *reinterpret_cast<uint4*>(orow + d) =
                                make_uint4(pack2<T>(o[8 * v] * inv_l, o[8 * v + 1] * inv_l),
                                           pack2<T>(o[8 * v + 2] * inv_l, o[8 * v + 3] * inv_l),
                                           pack2<T>(o[8 * v + 4] * inv_l, o[8 * v + 5] * inv_l),
                                           pack2<T>(o[8 * v + 6] * inv_l, o[8 * v + 7] * inv_l));
                    }
                }
                tc::fence_before_sync();  // before this warp's next arrival on p_full[x]
            }
            sx += n;
            ++px;
            gk += n;
            gv += n;
            ++ld;
        }
        tc::fence_before_sync();
    }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <typename T, int DP, bool ALIBI>
int run_prefill_q8(const Args& a, const PrefillQ8Params& pp, char* msg, size_t msg_len) {
    constexpr int SMEM = PqCfg<DP, std::is_same<T, __half>::value ? 3 : 2>::SMEM;
    auto kern = prefill_q8_kernel<T, DP, ALIBI>;
    static std::atomic<uint64_t> configured{0};
    const int sms = device_sms();
    cudaError_t e = set_shared_memory(kern, SMEM, configured);
    if (e != cudaSuccess || sms <= 0) {
        snprintf(msg, msg_len, "configuring the q8 prefill (%d bytes of shared memory): %s", SMEM, cudaGetErrorString(e));
        return PA_ERR_CUDA;
    }
    if ((int64_t)pp.pairs * a.Hkv + sms >= (int64_t)INT32_MAX) {
        snprintf(msg, msg_len, "q8 prefill: %lld work items (tiles x kv heads) exceed the item counter's range",
                 (long long)pp.pairs * a.Hkv);
        return PA_ERR_UNSUPPORTED;
    }
    const uint64_t dims[4] = {(uint64_t)a.D, (uint64_t)a.Hkv, (uint64_t)a.page, (uint64_t)a.num_blocks};
    const uint64_t strides[3] = {(uint64_t)a.kv_s2, (uint64_t)a.kv_s1, (uint64_t)a.kv_s0};
    const uint32_t box[4] = {128u, 1u, (uint32_t)pp.box_rows, 1u};
    const uint64_t qdims[4] = {(uint64_t)a.D, (uint64_t)a.H, (uint64_t)a.total_q, 1};
    const uint64_t qstrides[3] = {(uint64_t)a.q_s1 * 2, (uint64_t)a.q_s0 * 2, (uint64_t)a.q_s0 * 2 * a.total_q};
    const uint32_t qbox[4] = {64u, (uint32_t)pp.G, (uint32_t)(128 / pp.G), 1u};
    CUtensorMap tq, tk, tv;
    int rc = encode_tmap_4d(&tq, a.dtype, a.q, qdims, qstrides, qbox, 1, msg, msg_len);
    if (rc == PA_OK) rc = encode_tmap_4d(&tk, PA_E4M3, a.k, dims, strides, box, 1, msg, msg_len);
    if (rc == PA_OK) rc = encode_tmap_4d(&tv, PA_E4M3, a.v, dims, strides, box, 1, msg, msg_len);
    if (rc != PA_OK) return rc;
    NvtxRange nv("pa::prefill_q8_kernel");
    e = cudaMemsetAsync(pp.counter, 0, sizeof(int), a.stream);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "q8 prefill: zeroing the item counter: %s", cudaGetErrorString(e));
        return PA_ERR_CUDA;
    }
    timer_begin(PA_KC_PREFILL, a.stream);
    kern<<<std::min(sms, pp.pairs * a.Hkv), kPqThreads, SMEM, a.stream>>>(tq, tk, tv, pp);
    if ((e = cudaGetLastError()) != cudaSuccess) {
        snprintf(msg, msg_len, "q8 prefill launch: %s", cudaGetErrorString(e));
        return PA_ERR_CUDA;
    }
    timer_end(PA_KC_PREFILL, a.stream);
    count_launches(1);
    return PA_OK;
}

template <typename T>
int launch_prefill_q8_t(const Args& a, const PrefillQ8Params& pp, char* msg, size_t msg_len) {
    if (a.D <= 64)
        return a.alibi ? run_prefill_q8<T, 64, true>(a, pp, msg, msg_len) : run_prefill_q8<T, 64, false>(a, pp, msg, msg_len);
    return a.alibi ? run_prefill_q8<T, 128, true>(a, pp, msg, msg_len) : run_prefill_q8<T, 128, false>(a, pp, msg, msg_len);
}

}  // namespace

// Long queries of these calls go to the kernel above or, beyond head_dim 128, to prefill_q8_wide.cu's (the
// same conditions as the 16-bit kernels').
bool prefill_q8_supported(const Args& a) { return prefill_supported(a); }

int64_t prefill_q8_items_bound(const Args& a, int num_sms) {
    return prefill_q8_single(a, num_sms) ? prefill_q8_tiles(a) * a.Hkv : prefill_items_bound(a);
}

int launch_prefill_q8(const Args& a, int* counter, unsigned int* err, char* msg, size_t msg_len) {
    if (a.D > 128) return launch_prefill_q8_wide(a, counter, err, msg, msg_len);
    if (!counter) {
        snprintf(msg, msg_len, "the prefill kernels need a device item counter");
        return PA_ERR_ARG;
    }
    const PrefillQ8Params pp = prefill_q8_params(a, counter, err, 128, device_sms());
    return a.dtype == PA_BF16 ? launch_prefill_q8_t<__nv_bfloat16>(a, pp, msg, msg_len)
                              : launch_prefill_q8_t<__half>(a, pp, msg, msg_len);
}

}  // namespace pa
