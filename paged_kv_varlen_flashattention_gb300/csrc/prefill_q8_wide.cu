// Tensor-core prefill / chunked prefill over an 8-bit paged cache (sm_103a), head_dim 129..256.
//
// The mathematics of prefill_q8.cu (q in e4m3 terms against K as it is in the cache, P.V on f16 with V
// converted in the CTA, the page's scales in the softmax) for rows whose accumulator takes half of the
// tensor memory: an item is one 128-row query tile of one (sequence, kv head), key tiles have 64 keys, and S
// has four buffers, so that its products run up to three tiles ahead of the softmax. A thread of the softmax
// holds its row's 64 scores in registers.
//
// Roles (512 threads, four warpgroups):
//   warp 0      takes items and publishes them; K tiles and their scales
//   warp 1      MMA issuer: S(0), S(1), S(2), then S(j + 3), P.V(j)
//   warp 2      V tiles
//   warps 4..7  softmax, a row (TMEM lane) a thread
//   warps 8..15 converters: q into its terms at the start of an item, then V tile by tile
//
// Tensor-core bound: 4 D flops per (row, key) at the f16 rate (f16 q: 5 D).
// Two prompts of 4,096 tokens, 32 / 8 heads: 521 us at head_dim 256 in bf16 (1.05 PFLOP/s, 0.55 of the
// measured bf16 rate), 580 in f16; the same on row tiles of the split-KV kernel takes 2,965 and 2,915, and
// with two buffers of S 512 and 623. The tensor pipe is active 46 % of the time. What bounds it is the
// softmax: one warp a scheduler takes 1.2 us for its 32 rows of 64 keys, most of it waiting (tensor
// memory, dependent instructions), not issuing. A K ring of three or two stages with the V ring at
// three or four is 2 and 3 % slower. Columns past the head dim are computed on zeros (head_dim 192 takes what
// 256 does).
#include <algorithm>
#include <cfloat>
#include <cstdio>
#include <type_traits>

#include "prefill_q8_common.cuh"
#include "q8_common.cuh"
#include "rope_common.cuh"

namespace pa {
namespace {

constexpr int kPwThreads = 512;
constexpr int kPwConverters = 8;
// Register split (setmaxnreg) of the launch's 512 x 128: control 96, softmax 192, converters 112:
// 128 x 96 + 128 x 192 + 256 x 112 = 65,536.
constexpr int kPwRegsControl = 96, kPwRegsSoftmax = 192, kPwRegsConvert = 112;
constexpr float kPwOffset = 7.f;

template <int NTERM>
struct PwCfg {
    static constexpr int DP = 256, NT = 64, NS = 4;  // NS: buffers of S
    static constexpr int QTILE = 128 * 128;  // 128 rows of 64 columns of q as loaded, or of 128 columns of a term
    static constexpr int CHUNK = NT * 128;   // 64 keys of 128 columns of codes, or of 64 columns of V in f16
    static constexpr int KS = NTERM == 2 ? 4 : 2, VR = 2;
    static constexpr int TILE = 2 * CHUNK;     // a K or V tile as loaded
    static constexpr int VC_TILE = 4 * CHUNK;  // a V tile in f16
    static constexpr int OFF_Q = 0;            // term t, column half c at (2 t + c) QTILE
    static constexpr int OFF_K = 2 * NTERM * QTILE;
    static constexpr int OFF_VR = OFF_K + KS * TILE;
    static constexpr int OFF_VC = OFF_VR + VR * TILE;
    static constexpr int OFF_BAR = OFF_VC + 2 * VC_TILE;
    // q_raw, q_full, q_free, k_full[KS], k_empty[KS], vr_full[VR], vr_empty[VR], vc_full[2], vc_empty[2],
    // s_full[4], pv_done[4], p_full[4], drain, item_ready[2], item_free[2]
    static constexpr int NBAR = 3 + 2 * KS + 2 * VR + 4 + 3 * NS + 1 + 4;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;  // tmem base, abort flag
    static constexpr int OFF_SLOT = OFF_MISC + 16;       // two item slots
    static constexpr int SC_RING = 8;
    static constexpr int OFF_SC = OFF_SLOT + 128;          // [tile % 8]: ks[2], log2 vs[2], 1 / vs[2]
    static constexpr int OFF_EXP = OFF_SC + SC_RING * 32;  // [item parity][row]: e of the row, int8
    static constexpr int SMEM = OFF_EXP + 256 + 1024;
    static constexpr uint32_t T_S = 0, T_O = 256;  // the buffers of S, 64 columns each; O
    // The scale ring: the K producer writes position g after S(g - KS) has completed, which follows P.V of
    // g - KS - NS and so that tile's softmax; what is overwritten (g - 8) has been read.
    static_assert(KS + NS <= SC_RING, "scale ring");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <typename T, bool ALIBI>
__global__ void __launch_bounds__(kPwThreads, 1)
    prefill_q8_wide_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const PrefillQ8Params p) {
    constexpr int NTERM = std::is_same<T, __half>::value ? 3 : 2;
    using C = PwCfg<NTERM>;
    constexpr int KS = C::KS, VR = C::VR, DP = C::DP, NT = C::NT, NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    uint64_t* q_raw = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // q as loaded
    uint64_t* q_full = q_raw + 1;   // q in its terms
    uint64_t* q_free = q_full + 1;  // the item's Q.K^T products have completed
    uint64_t* k_full = q_free + 1;
    uint64_t* k_empty = k_full + KS;
    uint64_t* vr_full = k_empty + KS;
    uint64_t* vr_empty = vr_full + VR;
    uint64_t* vc_full = vr_empty + VR;
    uint64_t* vc_empty = vc_full + 2;
    uint64_t* s_full = vc_empty + 2;  // [buffer]
    uint64_t* pv_done = s_full + NS;  // [buffer]
    uint64_t* p_full = pv_done + NS;  // [buffer]: a softmax warp can be NS - 1 tiles ahead of another
    uint64_t* drain = p_full + NS;
    uint64_t* item_ready = drain + 1;      // [slot]
    uint64_t* item_free = item_ready + 2;  // [slot]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    PfItem* slots = reinterpret_cast<PfItem*>(smem + C::OFF_SLOT);
    float* sc_ring = reinterpret_cast<float*>(smem + C::OFF_SC);
    int8_t* row_exp = reinterpret_cast<int8_t*>(smem + C::OFF_EXP);
    if (tid == 64) {
        mbar_init(q_raw, 1);
        mbar_init(q_full, kPwConverters);
        mbar_init(q_free, 1);
        for (int s = 0; s < KS; ++s) {
            mbar_init(&k_full[s], 2);  // the copies, the scales
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < VR; ++s) {
            mbar_init(&vr_full[s], 1);
            mbar_init(&vr_empty[s], kPwConverters);
        }
        for (int x = 0; x < NS; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&pv_done[x], 1);
            mbar_init(&p_full[x], 4);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&vc_full[x], kPwConverters);
            mbar_init(&vc_empty[x], 1);
            mbar_init(&item_ready[x], 1);
            mbar_init(&item_free[x], 6 + kPwConverters);  // the V producer, the issuer, four softmax warps, the converters
        }
        mbar_init(drain, 1);
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
    // First key of step j of an item (under a bias the nearest keys come first: prefill_q8.cu).
    auto tile_key = [&](const PfItem& it, int j) { return it.kt0 + (ALIBI ? it.n_tiles - 1 - j : j) * NT; };
    // The item's key tiles into the K ring (with the scales of each tile's two 32-key groups) or the V
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
            int blk[2];
            uint32_t bytes = 0;
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const int b = __shfl_sync(0xffffffffu, id, ((j - jw) * bpt + jj) & 31);
                blk[jj] = jj < bpt ? b : -1;
                if (blk[jj] >= 0) bytes += (uint32_t)(p.box_rows * DP);
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&fullb[s], bytes);
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    if (blk[jj] < 0) continue;
                    const int key = tile_key(it, j) + jj * p.box_rows;
                    const int slot = key - (key / p.P) * p.P;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tma_load_4d(ring + s * C::TILE + c * C::CHUNK + jj * p.box_rows * 128, map, &fullb[s], c * 128,
                                    it.hk, slot, blk[jj], 0ull);
                }
            }
            __syncwarp();
            if (scales) {  // after the copies are on their way: the gather's latency runs beside theirs
                const int src = (j - jw) * bpt + ((lane & 1) * 32) / p.box_rows;
                const float a = __shfl_sync(0xffffffffu, ksc, src), v = __shfl_sync(0xffffffffu, vsc, src);
                if (lane < 2) {
                    float* slot = sc_ring + (g % C::SC_RING) * 8 + lane;
                    const float lv = v > 7.8886090522101181e-31f ? fminf(log2f(v), 126.f) : (float)kScaleExpMin;
                    slot[0] = a;
                    slot[2] = lv;
                    slot[4] = exp2f(-lv);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&fullb[s]);
            }
        }
        return true;
    };

    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPwRegsControl));
    if (warp == 0) {
        // ---------------- item taker, K producer ----------------
        // w = tile * Hkv + kv head, each sequence's last tile first.
        const int total = p.pairs * p.Hkv;
        if (!p.withhold) prefetch_tmap(&tm_k);
        int w_next = lane == 0 ? atomicAdd(p.counter, 1) : 0;
        int gk = 0;
        for (int k = 0;; ++k) {
            const int w = __shfl_sync(0xffffffffu, w_next, 0);
            PfItem it{};
            it.b = -1;
            if (w < total) {
                const int tile = w / p.Hkv;
                it.hk = w - tile * p.Hkv;
                int remaining = tile;
                for (int base = 0; base < p.batch && it.b < 0; base += 32) {
                    const int bb = base + lane;
                    int tiles = 0;
                    if (bb < p.batch) {
                        const int sqb = p.cu_q[bb + 1] - p.cu_q[bb];
                        tiles = (int64_t)sqb * p.G > p.rows_cap ? (sqb + qpt - 1) / qpt : 0;
                    }
                    int incl = tiles;
#pragma unroll
                    for (int off = 1; off < 32; off <<= 1) {
                        const int v = __shfl_up_sync(0xffffffffu, incl, off);
                        if (lane >= off) incl += v;
                    }
                    const unsigned hit = __ballot_sync(0xffffffffu, remaining < incl);
                    if (hit) {
                        const int src = __ffs(hit) - 1;
                        const int excl = __shfl_sync(0xffffffffu, incl - tiles, src);
                        const int cnt = __shfl_sync(0xffffffffu, tiles, src);
                        it.b = base + src;
                        it.u = cnt - 1 - (remaining - excl);
                    } else {
                        remaining -= __shfl_sync(0xffffffffu, incl, 31);
                    }
                }
                if (it.b >= 0) pf_single_item<NT>(p, qpt, it);
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
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        constexpr uint32_t IDESC_S = tc::idesc_e4m3(128, NT);
        constexpr uint32_t IDESC_O = tc::idesc_f16(128, DP, false, false, true);
        const uint64_t da = tc::smem_desc_sw128(smem_addr(smem + C::OFF_Q), 16, 1024);
        const uint64_t dk0 = tc::smem_desc_sw128(smem_addr(smem + C::OFF_K), 16, 1024);
        const uint64_t dv0 = tc::smem_desc_sw128(smem_addr(smem + C::OFF_VC), C::CHUNK, 1024);
        const uint32_t d_o = tmem + C::T_O;
        int lq = 0, g0 = 0;
        bool ok = true;
        auto issue_s = [&](int g, bool last) -> bool {  // S(g) = (sum of q terms) K^T of tile g
            if (!wait_all(&k_full[g % KS], (g / KS) & 1)) return false;
            const uint64_t db = dk0 + (uint64_t)((g % KS) * (C::TILE >> 4));
#pragma unroll
            for (int t = 0; t < NTERM; ++t)
#pragma unroll
                for (int kk = 0; kk < DP / 32; ++kk)
                    tc::mma_f8_ss_elect(tmem + C::T_S + g % NS * NT,
                                        da + (uint64_t)((t * 2 + kk / 4) * (C::QTILE >> 4) + (kk & 3) * 2),
                                        db + (uint64_t)((kk / 4) * (C::CHUNK >> 4) + (kk & 3) * 2), IDESC_S,
                                        t + kk > 0 ? 1u : 0u);
            tc::commit_elect(&s_full[g % NS]);
            tc::commit_elect(&k_empty[g % KS]);
            if (last) tc::commit_elect(q_free);
            __syncwarp();
            return true;
        };
        for (int k = 0; ok; ++k) {
            PfItem it;
            if (!take_slot(k, it) || it.b < 0) break;
            if (it.bad || it.n_tiles == 0) continue;
            const int n = it.n_tiles;
            if (!(ok = wait_all(q_full, lq & 1))) break;
            // S(g) takes the buffer of P(g - NS), whose P.V has been issued before it
            for (int j = 0; ok && j < min(n, NS - 1); ++j) ok = issue_s(g0 + j, j + 1 == n);
            for (int j = 0; ok && j < n; ++j) {
                const int g = g0 + j;
                if (j + NS - 1 < n && !(ok = issue_s(g + NS - 1, j + NS == n))) break;
                if (!(ok = wait_all(&vc_full[g & 1], (g >> 1) & 1))) break;
                if (!(ok = wait_all(&p_full[g % NS], (g / NS) & 1))) break;
                const uint64_t db = dv0 + (uint64_t)((g & 1) * (C::VC_TILE >> 4));
                const uint32_t first = j > 0 ? 1u : 0u;
#pragma unroll
                for (int kk = 0; kk < NT / 16; ++kk)
                    tc::mma_ts_elect(d_o, tmem + C::T_S + g % NS * NT + kk * 8, db + (uint64_t)(kk * (2048 / 16)), IDESC_O,
                                     kk > 0 ? 1u : first);
                tc::commit_elect(&vc_empty[g & 1]);
                tc::commit_elect(&pv_done[g % NS]);
                __syncwarp();
            }
            g0 += n;
            ++lq;
        }
        if (lane == 0) {
            tc::commit(drain);
            mbar_wait(drain, 0, p.wait_ns);  // not cut short by an abort: MMAs may be in flight
        }
        __syncwarp();
    }
    } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPwRegsConvert));
    {
        // ---------------- converters ----------------
        const int cw = warp - 8;
        if (cw == 0 && !p.withhold) prefetch_tmap(&tm_q);
        int ld = 0, gv = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            PfItem it;
            if (!take_slot(k, it) || it.b < 0) break;
            if (it.bad || it.n_tiles == 0) continue;
            // q is loaded over the terms of the item before once its last Q.K^T products have completed, 64
            // columns a 16 KB tile, and converted in place, a warp a row.
            if (ld >= 1 && !(ok = wait_all(q_free, (ld - 1) & 1))) break;
            if (cw == 0 && lane == 0 && !p.withhold) {
                mbar_arrive_expect_tx(q_raw, (DP / 64) * trows * 128);
                for (int c = 0; c < DP / 64; ++c)
                    tma_load_4d(smem + C::OFF_Q + c * C::QTILE, &tm_q, q_raw, c * 64, it.hk * p.G, it.q0 + it.i0, 0, 0ull);
            }
            __syncwarp();
            if (!(ok = wait_all(q_raw, ld & 1))) break;
            {
                uint8_t* tile = smem + C::OFF_Q;
                constexpr int ROWS = 128 / kPwConverters, NB = 2;
#pragma unroll 1
                for (int i0 = 0; i0 < ROWS; i0 += NB) {
                    uint4 w[NB];
                    float mx[NB];
#pragma unroll
                    for (int i = 0; i < NB; ++i)
                        w[i] = *reinterpret_cast<const uint4*>(tile + (lane >> 3) * C::QTILE +
                                                               swz128(cw * ROWS + i0 + i, lane & 7));
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        const float2 f0 = unpack2<T>(w[i].x), f1 = unpack2<T>(w[i].y), f2 = unpack2<T>(w[i].z),
                                     f3 = unpack2<T>(w[i].w);
                        mx[i] = max3f(max3f(fabsf(f0.x), fabsf(f0.y), fabsf(f1.x)),
                                      max3f(fabsf(f1.y), fabsf(f2.x), fabsf(f2.y)), fmaxf(fabsf(f3.x), fabsf(f3.y)));
                    }
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
                        for (int i = 0; i < NB; ++i) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], off));
                    __syncwarp();  // every lane has read its columns of these rows
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        const int r = cw * ROWS + i0 + i;
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
                            for (int t = 0; t < NTERM; ++t) c2[t][e] = e4m3x2_take(y.x, y.y);
                        }
                        uint8_t* dst = tile + (lane >> 4) * C::QTILE + swz128(r, (lane & 15) >> 1) + (lane & 1) * 8;
#pragma unroll
                        for (int t = 0; t < NTERM; ++t)
                            *reinterpret_cast<uint2*>(dst + 2 * t * C::QTILE) =
                                make_uint2(c2[t][0] | (c2[t][1] << 16), c2[t][2] | (c2[t][3] << 16));
                        if (lane == 0) row_exp[(ld & 1) * 128 + r] = (int8_t)e2;
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            // V tiles: warp cw converts rows 8 cw .. + 7
            const int64_t cdiag = (int64_t)it.sk - it.sq;
            const int i_last = min(it.sq - 1, it.i0 + qpt - 1);
            const int key_lo = p.wl >= 0 ? (int)max64(0, it.i0 + cdiag - p.wl) : 0;
            const int key_hi = p.wr >= 0 ? (int)min64((int64_t)it.sk - 1, i_last + cdiag + p.wr) : it.sk - 1;
            for (int j = 0; j < it.n_tiles; ++j) {
                const int g = gv + j, s = g % VR, c = g & 1;
                if (!(ok = wait_all(&vr_full[s], (g / VR) & 1))) break;
                if (g >= 2 && !(ok = wait_all(&vc_empty[c], ((g >> 1) - 1) & 1))) break;
                const uint8_t* src = smem + C::OFF_VR + s * C::TILE;
                uint8_t* dst = smem + C::OFF_VC + c * C::VC_TILE;
                const int kt = tile_key(it, j);
                const int uu = lane & 15;  // 16-byte unit of a row
                uint8_t* d = dst + (uu >> 2) * C::CHUNK;
                const int u0 = (uu & 3) * 2;
                const bool sw = (uu & 4) != 0;
#pragma unroll 2
                for (int i = 0; i < NT / kPwConverters / 2; ++i) {
                    const int r = cw * (NT / kPwConverters) + i * 2 + (lane >> 4);
                    uint4 v = *reinterpret_cast<const uint4*>(src + (uu >> 3) * C::CHUNK + swz128(r, uu & 7));
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPwRegsSoftmax));
    {
        // ---------------- softmax: thread t of warp 4 + w holds row (TMEM lane) 32 w + t ----------------
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t o_addr = tmem + lane_addr + C::T_O;
        T* out = static_cast<T*>(p.out);
        const int qi = row / p.G, gi = row - qi * p.G;  // query of the tile, head of the group
        const bool pad = row >= trows;
        int g0 = 0, ld = 0;
        bool ok = true;
        // P.V of tile g, the last whose P was given. Its barrier is not a phase on (P.V of g + NS is not issued
        // yet) nor one behind (P.V of g - NS precedes S(g), which has been seen).
        auto wait_pv = [&](int g) {
            return __all_sync(0xffffffffu, wait_bar(&pv_done[g % NS], (g / NS) & 1, abort_flag, p.err, p.wait_ns));
        };
        for (int k = 0; ok; ++k) {
            PfItem it;
            if (!take_slot(k, it) || it.b < 0) break;
            if (it.bad) continue;
            const int qrow = it.i0 + qi;  // query of the sequence
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
            const int64_t diag = qrow + ((int64_t)it.sk - it.sq);
            const int lo = p.wl >= 0 ? (int)max64(0, diag - p.wl) : 0;
            // (rows past the tile's queries keep the mask of the query they would be: prefill_q8.cu)
            const int hi = p.wr >= 0 ? (int)max64(-1, min64((int64_t)it.sk - 1, diag + p.wr)) : it.sk - 1;
            const float ab = ALIBI && live ? p.alibi[h] * kLog2e : 0.f;
            float m = -INFINITY, l = 0.f, sl = 0.f;

            // One key tile: S -> running reference -> (rare) O rescale -> P.
            auto step = [&](int j) -> bool {
                const int g = g0 + j, kt = tile_key(it, j);
                const uint32_t s_addr = tmem + lane_addr + C::T_S + g % NS * NT;
                if (!__all_sync(0xffffffffu, wait_bar(&s_full[g % NS], (g / NS) & 1, abort_flag, p.err, p.wait_ns))) return false;
                tc::fence_after_sync();
                const float* slot = sc_ring + (g % C::SC_RING) * 8;
                if (j == 0) sl = p.scale_log2 * __int_as_float((127 - row_exp[(ld & 1) * 128 + row]) << 23);
                float v[2][32];
                tc::ld_32cols(s_addr, v[0]);
                tc::ld_32cols(s_addr + 32, v[1]);
                tc::wait_ld();
                if (kt < lo || kt + NT - 1 > hi) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int key = kt + 32 * q + i;
                            v[q][i] = key >= lo && key <= hi ? v[q][i] : -INFINITY;
                        }
                }
                const bool above = kt >= diag;
                const bool one_sided = ALIBI && __all_sync(0xffffffffu, above || kt + NT - 1 <= diag || hi <= diag);
                float c[2], lv[2], mx = -INFINITY;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    c[q] = fmaxf(sl * slot[q], 1e-37f);  // positive: -inf x c stays -inf under a scale of 0
                    lv[q] = slot[2 + q];
                    if (ALIBI) {  // v becomes the whole x
                        float d0 = (float)((int)diag - kt - 32 * q);
                        if (one_sided) {
                            const float na = above ? ab : -ab;
                            float d1 = d0 - 1.f;
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                ffma2(v[q][i], v[q][i + 1], v[q][i], v[q][i + 1], c[q], c[q], lv[q], lv[q]);
                                ffma2(v[q][i], v[q][i + 1], d0, d1, na, na, v[q][i], v[q][i + 1]);
                                fadd2_acc(d0, d1, -2.f, -2.f);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[q][i] = fmaf(-ab, fabsf(d0 - (float)i), fmaf(v[q][i], c[q], lv[q]));
                        }
                    }
                    float t0 = fmaxf(v[q][0], v[q][1]), t1 = fmaxf(v[q][2], v[q][3]);
#pragma unroll
                    for (int i = 4; i < 32; i += 4) {
                        t0 = max3f(t0, v[q][i], v[q][i + 1]);
                        t1 = max3f(t1, v[q][i + 2], v[q][i + 3]);
                    }
                    t0 = fmaxf(t0, t1);
                    mx = fmaxf(mx, ALIBI ? t0 : fmaf(t0, c[q], lv[q]));
                }
                const bool grow = mx > m + 8.f;
                if (__any_sync(0xffffffffu, grow)) {
                    const float alpha = grow ? fast_exp2(m - mx) : 1.f;
                    if (grow) m = mx;
                    l *= alpha;
                    if (j > 0) {
                        if (!wait_pv(g - 1)) return false;
                        tc::fence_after_sync();
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
                const float nm = m == -INFINITY ? 0.f : kPwOffset - m;
                uint32_t pk[32];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float cg = ALIBI ? 1.f : c[q], ag = ALIBI ? nm : nm + lv[q];
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x0, x1;
                        ffma2(x0, x1, v[q][2 * i], v[q][2 * i + 1], cg, cg, ag, ag);
                        const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                        fadd2_acc(s0, s1, p0, p1);
                        pk[16 * q + i] = pack2<__half>(p0, p1);
                    }
                    l = fmaf(s0 + s1, slot[4 + q], l);
                }
                tc::st_32x32b_x32(s_addr, pk);  // P over its own S
                tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[g % NS]);
                return true;
            };
#pragma unroll 1
            for (int j = 0; ok && j < n; ++j) ok = step(j);
            if (ok) ok = wait_pv(g0 + n - 1);
            if (ok) {
                tc::fence_after_sync();
                const float inv_l = l == 0.f ? 0.f : 1.f / l;
                if (live) *lse = l == 0.f ? -INFINITY : (m - kPwOffset + log2f(l)) * 0.69314718055994531f;
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
                tc::fence_before_sync();  // before this warp's next arrival on p_full
            }
            g0 += n;
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

template <typename T, bool ALIBI>
int run_prefill_q8_wide(const Args& a, const PrefillQ8Params& pp, char* msg, size_t msg_len) {
    constexpr int SMEM = PwCfg<std::is_same<T, __half>::value ? 3 : 2>::SMEM;
    auto kern = prefill_q8_wide_kernel<T, ALIBI>;
    static std::atomic<uint64_t> configured{0};
    const int sms = device_sms();
    cudaError_t e = set_shared_memory(kern, SMEM, configured);
    if (e != cudaSuccess || sms <= 0) {
        snprintf(msg, msg_len, "configuring the wide q8 prefill (%d bytes of shared memory): %s", SMEM, cudaGetErrorString(e));
        return PA_ERR_CUDA;
    }
    if ((int64_t)pp.pairs * a.Hkv + sms >= (int64_t)INT32_MAX) {
        snprintf(msg, msg_len, "wide q8 prefill: %lld work items (tiles x kv heads) exceed the item counter's range",
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
    NvtxRange nv("pa::prefill_q8_wide_kernel");
    e = cudaMemsetAsync(pp.counter, 0, sizeof(int), a.stream);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "wide q8 prefill: zeroing the item counter: %s", cudaGetErrorString(e));
        return PA_ERR_CUDA;
    }
    timer_begin(PA_KC_PREFILL, a.stream);
    kern<<<std::min(sms, pp.pairs * a.Hkv), kPwThreads, SMEM, a.stream>>>(tq, tk, tv, pp);
    if ((e = cudaGetLastError()) != cudaSuccess) {
        snprintf(msg, msg_len, "wide q8 prefill launch: %s", cudaGetErrorString(e));
        return PA_ERR_CUDA;
    }
    timer_end(PA_KC_PREFILL, a.stream);
    count_launches(1);
    return PA_OK;
}

}  // namespace

int launch_prefill_q8_wide(const Args& a, int* counter, unsigned int* err, char* msg, size_t msg_len) {
    if (!counter) {
        snprintf(msg, msg_len, "the prefill kernels need a device item counter");
        return PA_ERR_ARG;
    }
    const PrefillQ8Params pp = prefill_q8_params(a, counter, err, 64, device_sms());
    if (a.dtype == PA_BF16)
        return a.alibi ? run_prefill_q8_wide<__nv_bfloat16, true>(a, pp, msg, msg_len)
                       : run_prefill_q8_wide<__nv_bfloat16, false>(a, pp, msg, msg_len);
    return a.alibi ? run_prefill_q8_wide<__half, true>(a, pp, msg, msg_len)
                   : run_prefill_q8_wide<__half, false>(a, pp, msg, msg_len);
}

}  // namespace pa
