// Attention over an 8-bit paged cache (pa_varlen_fwd_q8): the split-KV kernels on mma.sync,
// for decode-class rows and, tile by tile, for every call the tensor-core prefill kernel
// does not take.
//
// K and V elements are e4m3 codes with one scale per page and kv head: K = ks Kc, V = vs Vc.
// Neither is ever scaled element by element.  With c = softmax_scale log2(e) and a running
// reference m, the softmax works on
//     x_j = c ks_j (q . Kc_j) [- bias] + log2 vs_j,     w_j = 2^(x_j - m + 10),
//     O = sum_j w_j Vc_j,     l = sum_j w_j / vs_j,     out = O / l,
//     lse = (m - 10 + log2 l) ln 2,
// which is softmax(s) V with the page's value scale moved into the exponent: O and its reference
// live in units of V, so pages of very different magnitude keep their precision, and l takes
// the scale back out, one multiplication per 16 keys.  m is the largest x so far; the offset of
// 10 keeps weights down to 2^-24 of the largest in the normal range of f16 (2^-34 above zero).
//
// The codes become f16 on the way into the matrix instructions, where every e4m3 value is exact
// (two elements an instruction; bf16 has no such conversion), and q and the weights are f16 beside
// them: f16 q as it is; bf16 q times a power of two per row that brings the row's largest
// magnitude to 2^14..2^15, taken back out in fp32 with the score's scale (bf16 has fewer
// significant bits than f16, so only elements below 2^-28 of the row's largest lose any); the
// weights rounded to 11 bits, where the 16-bit kernels of bf16 calls round them to 8.
//
// The column order inside a fragment is free as long as both operands share it, so a lane's
// 4 bytes of a K row (one 32-bit ldmatrix element pair) are used as columns 4t..4t+3 without
// any shuffle, and q is read to match.  V is loaded two columns at a time with ldmatrix.trans,
// one byte permute per register puts the two keys of a column side by side, and even and odd
// columns go to two accumulators, whose lanes hold four consecutive columns.
//
// (That is the body for 9..32 rows; fewer rows take their terms side by side in one e4m3 product, below.)
//
// HBM-bound: 2 bytes per (key, kv head, column). 64 sequences of 512..4,096 keys, 32 / 8 heads of 128 in bf16 take
// 63.4 us, 0.71 of the copy rate (4.8 TB/s); copies of the kernel without any arithmetic took 57: what is
// not hidden is a unit's start, about 6 us of dependent reads until its first keys are there, and its merge.
#pragma once

#include "q8_common.cuh"
#include "rope_common.cuh"
#include "splitkv_kernel.cuh"

namespace pa {

struct Q8Params : SplitParams {
    const float* ks;
    const float* vs;
    int64_t ks_s0, ks_s1, vs_s0, vs_s1;
    int cluster;    // CTAs of a cluster that share a unit's keys (1: none; splits then go through partials)
};

constexpr int kQ8MaxBoxes = 256;         // TMA boxes (32 rows or more) of one split
static_assert(kMaxSplitKeys <= 32 * kQ8MaxBoxes, "the boxes of the longest split");
constexpr float kQ8Offset = 10.f;

__device__ __forceinline__ bool q8_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
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

// log2 of a value scale; scales below 2^-100 (zero among them) are read as 2^-100.
__device__ __forceinline__ float q8_log2_scale(float vs) {
    return vs > 7.8886090522101181e-31f ? fminf(log2f(vs), 126.f) : (float)kScaleExpMin;
}

// ---- a unit's keys over the CTAs of a cluster --------------------------------------------------
// Few units (a small batch) or units much longer than the average leave SMs idle or late.  A cluster of
// 2, 4 or 8 CTAs then takes equal shares of a unit's tiles, leaves each warp's (O, m, l) in its own
// shared memory, and after a cluster barrier every CTA merges a share of the columns of all of them:
// no partials in memory and no second launch.  All CTAs of a cluster see the same unit, so they
// return early together or meet at both barriers; one that gave up says so in its flag, and
// nobody leaves before the others have read its memory.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// The part of a warp without a share in the merge: both barriers.
__device__ __forceinline__ void q8_cluster_passive() {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    cluster_arrive();
    cluster_wait();
}

// The tiles of a CTA: a fixed count per split, or an equal share of the unit's in a cluster.  False:
// no work (the same answer in every CTA of a cluster).
__device__ __forceinline__ bool q8_tiles(const Q8Params& p, const TileView& tv, int split, int& t_begin, int& n_iter,
                                         bool& single) {
    if (p.cluster > 1) {
        t_begin = (int)((int64_t)tv.ntiles * split / p.cluster);
        n_iter = (int)((int64_t)tv.ntiles * (split + 1) / p.cluster) - t_begin;
        single = true;
        return true;
    }
    if (split >= max(tv.nsplit, 1)) return false;
    t_begin = split * p.split_tiles;
    n_iter = max(0, min(tv.ntiles, t_begin + p.split_tiles) - t_begin);
    single = tv.nsplit <= 1;
    return true;
}

// Byte offset of 16-byte unit `u` of row `r` in a tile of rows of DP bytes as TMA leaves it:
// 128-byte column chunks (chunk-major, NT rows each) under the 128-byte swizzle, or 64-byte rows
// under the 64-byte swizzle (unit bits XOR address bits 7..8).
template <int DP, int NT>
__device__ __forceinline__ uint32_t q8_off(int r, int u) {
    if constexpr (DP == 64)
        return (uint32_t)(r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
    else
        return (uint32_t)((u >> 3) * (NT * 128)) + swz128(r, u & 7);
}

// Rows' bounds and bias of a tile into shared memory.  Padding rows attend every key: their q is zero,
// nothing of theirs is written, and so a tile inside the real rows' intervals needs no mask.
struct Q8Rows {
    int* lo;
    int* hi;
    int* dg;
    float* ab;
    float* sc;  // score scale of the row: c / (power of two on its q)
};
__device__ __forceinline__ Q8Rows q8_rows(uint8_t* base, int M) {
    int* p = reinterpret_cast<int*>(base);
    return {p, p + M, p + 2 * M, reinterpret_cast<float*>(p + 3 * M), reinterpret_cast<float*>(p + 4 * M)};
}
__device__ __forceinline__ void q8_row_bounds(const SplitParams& p, const TileView& tv, const Q8Rows& rows, int hk,
                                              int M) {
    const int r = threadIdx.x;
    if (r >= M) return;
    int lo = 0, hi = INT32_MAX, dg = 0;
    float ab = 0.f;
    if (r < tv.rows) {
        const int64_t i = (tv.row0 + r) / p.G;
        const int64_t diag = i + tv.sk - tv.sq;
        lo = p.wl >= 0 ? (int)max64(0, diag - p.wl) : 0;
        hi = p.wr >= 0 ? (int)max64(-1, min64(tv.sk - 1, diag + p.wr)) : tv.sk - 1;
        dg = (int)diag;
        if (p.alibi) ab = p.alibi[hk * p.G + (int)(tv.row0 + r - i * p.G)] * kLog2e;
    }
    rows.lo[r] = lo;
    rows.hi[r] = hi;
    rows.dg[r] = dg;
    rows.ab[r] = ab;
}

// q rows as f16 into shared memory (row pitch `pitch` bytes, zero padded), warp w of NW taking
// rows w, w + NW, ...; each row's power of two and score scale into rows.sc.
template <typename T, int DP, int M, int NW>
__device__ __forceinline__ void q8_stage_q(const SplitParams& p, const TileView& tv, const Q8Rows& rows, uint8_t* qs,
                                           int pitch, int hk, int warp, int lane) {
    constexpr int RPW = M / NW;
    constexpr int UL = (DP / 8 + 31) / 32;  // 16-byte units a lane takes of a row
    const T* q = static_cast<const T*>(p.q);
    uint4 x[RPW][UL];
#pragma unroll
    for (int k = 0; k < RPW; ++k) {
        const int r = warp + k * NW;
        const int rho = tv.row0 + r, i = rho / p.G, g = rho - i * p.G;
#pragma unroll
        for (int c = 0; c < UL; ++c) {
            const int u = lane + 32 * c;
            x[k][c] = make_uint4(0, 0, 0, 0);
            if (r < tv.rows && u * 8 < p.D)
                x[k][c] = __ldg(reinterpret_cast<const uint4*>(q + (int64_t)(tv.q0 + i) * p.q_s0 +
                                                               (int64_t)(hk * p.G + g) * p.q_s1 + u * 8));
        }
    }
#pragma unroll
    for (int k = 0; k < RPW; ++k) {
        const int r = warp + k * NW;
        float sc = p.scale_log2;
        if constexpr (!std::is_same<T, __half>::value) {
            float v[UL][8], mx = 0.f;
#pragma unroll
            for (int c = 0; c < UL; ++c) {
                const uint32_t w[4] = {x[k][c].x, x[k][c].y, x[k][c].z, x[k][c].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack2<T>(w[e]);
                    v[c][2 * e] = f.x;
                    v[c][2 * e + 1] = f.y;
                    mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const int e2 = min(126, 14 - ((__float_as_int(mx) >> 23) - 127));
            const float up = __int_as_float((127 + e2) << 23), down = __int_as_float((127 - e2) << 23);
            sc *= down;
#pragma unroll
            for (int c = 0; c < UL; ++c)
                x[k][c] = make_uint4(pack2<__half>(v[c][0] * up, v[c][1] * up), pack2<__half>(v[c][2] * up, v[c][3] * up),
                                     pack2<__half>(v[c][4] * up, v[c][5] * up), pack2<__half>(v[c][6] * up, v[c][7] * up));
        }
        if (lane == 0) rows.sc[r] = sc;
#pragma unroll
        for (int c = 0; c < UL; ++c) {
            const int u = lane + 32 * c;
            if (u * 8 < DP) *reinterpret_cast<uint4*>(qs + r * pitch + u * 16) = x[k][c];
        }
    }
}

// One producer warp (K or V): the block ids of the split's boxes into `ids`, the tiles into the
// ring.  Whole warp; lane 0 issues.  The K producer reports bad block ids.
template <int DP, int NT, int STAGES>
__device__ __forceinline__ void q8_produce(const Q8Params& p, const CUtensorMap* map, uint8_t* ring, uint64_t* full,
                                           uint64_t* empty, int* ids, bool report, int b, int hk, int sk, int kbeg,
                                           int n_iter, int g0, volatile uint32_t* abort_flag) {
    constexpr int CB = DP < 128 ? DP : 128, CH = DP / CB;
    const int lane = threadIdx.x & 31;
    const int32_t* bt_row = p.bt + (int64_t)b * p.bt_s0;
    const int n_boxes = min(n_iter * p.boxes_per_tile, kQ8MaxBoxes);
    // every table entry is requested before the first is looked at: one memory latency
    int blk[kQ8MaxBoxes / 32];
#pragma unroll
    for (int i = 0; i < kQ8MaxBoxes / 32; ++i) {
        const int bi = lane + 32 * i, key = kbeg + bi * p.box_rows;
        blk[i] = -1;  // past the sequence: not loaded
        if (bi < n_boxes && key < sk) {
            const int page = key / p.P;
            blk[i] = page < p.bt_cols ? __ldg(bt_row + page) : -2;
        }
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kQ8MaxBoxes / 32; ++i) {
        const int bi = lane + 32 * i;
        if (bi >= n_boxes) continue;
        if (kbeg + bi * p.box_rows < sk && (blk[i] < 0 || blk[i] >= p.num_blocks)) {
            bad = true;
            blk[i] = -2;
        }
        ids[bi] = blk[i];
    }
    if (bad && report) flag_error(p.err, PA_ERR_DEVICE_BOUNDS);
    __syncwarp();
    if (lane != 0 || p.withhold) return;
    const uint64_t policy = l2_policy_evict_first();
    for (int it = 0; it < n_iter; ++it) {
        const int gi = g0 + it, stage = gi % STAGES;
        if (gi >= STAGES && !q8_wait(&empty[stage], ((gi / STAGES) - 1) & 1, abort_flag, p.err, p.wait_ns)) return;
        uint8_t* st = ring + stage * (NT * DP);
        uint32_t bytes = 0;
        for (int j = 0; j < p.boxes_per_tile; ++j)
            if (ids[it * p.boxes_per_tile + j] >= 0) bytes += (uint32_t)(p.box_rows * DP);
        mbar_arrive_expect_tx(&full[stage], bytes);
        for (int j = 0; j < p.boxes_per_tile; ++j) {
            const int box = ids[it * p.boxes_per_tile + j];
            if (box < 0) continue;
            const int key = kbeg + it * NT + j * p.box_rows;
            const int slot = key - (key / p.P) * p.P;
#pragma unroll
            for (int c = 0; c < CH; ++c)
                tma_load_4d(st + c * (NT * CB) + j * p.box_rows * CB, map, &full[stage], c * CB, hk, slot, box, policy);
        }
    }
}

// The scales of a consumer warp's blocks of keys (each inside one page), K's as it is and V's as
// log2: lane i holds those of block n & ~31 + i of the warp's sequence of blocks, read straight from
// the table and the scales beside the producers' copies, 32 blocks ahead of their use.  (Gathered by
// the producers into shared memory they arrived 4 to 6 us into a unit, after the first copies
// had been issued; its first keys are there after 3.)
struct Q8Scales {
    float ks, lv, ks_next, lv_next;
    template <typename KeyOf>
    __device__ __forceinline__ void fetch(const Q8Params& p, int b, int hk, int sk, int n, int n_blocks, KeyOf key_of) {
        const int i = n + (int)(threadIdx.x & 31);
        ks_next = 1.f;
        lv_next = 0.f;
        if (i >= n_blocks) return;
        const int key = key_of(i), page = key / p.P;
        if (key >= sk || page >= p.bt_cols) return;
        const int blk = __ldg(p.bt + (int64_t)b * p.bt_s0 + page);
        if (blk < 0 || blk >= p.num_blocks) return;
        ks_next = __ldg(p.ks + (int64_t)blk * p.ks_s0 + (int64_t)hk * p.ks_s1);
        lv_next = __ldg(p.vs + (int64_t)blk * p.vs_s0 + (int64_t)hk * p.vs_s1);
    }
    // the scales of block n (n goes up by one from call to call; whole warp)
    template <typename KeyOf>
    __device__ __forceinline__ void take(const Q8Params& p, int b, int hk, int sk, int n, int n_blocks, KeyOf key_of,
                                         float& k, float& v) {
        if ((n & 31) == 0) {
            ks = ks_next;
            lv = q8_log2_scale(lv_next);
            if (n + 32 < n_blocks) fetch(p, b, hk, sk, n + 32, n_blocks, key_of);
        }
        k = __shfl_sync(0xffffffffu, ks, n & 31);
        v = __shfl_sync(0xffffffffu, lv, n & 31);
    }
};

// Score of a (row, key): masked by select, biased, in units of V (lv = log2 of its scale).
__device__ __forceinline__ float q8_score(float s, float c, float lv, bool in, float ab, int dg, int key) {
    return in ? fmaf(-ab, fabsf((float)(dg - key)), fmaf(s, c, lv)) : -INFINITY;
}
// Keys [lo, hi] that both of every lane's rows attend and that carry no bias: there a score is one
// multiply-add (the masks and the bias cost seven instructions a score, a fifth of the kernel).
__device__ __forceinline__ void q8_plain_keys(bool biased, int& lo, int& hi) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        lo = max(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = min(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    if (biased) hi = -1;
}

// ---------------------------------------------------------------------------------------------
// decode_q8_kernel: head_dim <= 128, NW consumer warps with private key slices of every tile
// (as decode_kernel), one producer warp for K and one for V.
template <int DP_, int MG, int NW, int NT, int STAGES, int ML = MG>
struct Q8Cfg {
    static constexpr int DP = DP_;
    static constexpr int M = 16 * MG;
    static constexpr int KW = NW / MG;   // warps sharing a row group
    static constexpr int KPW = NT / KW;  // keys per warp and tile
    static constexpr int CK = 2;  // 16-key chunks whose scores are in registers together
    static constexpr int TILE = NT * DP;
    static constexpr int QP = DP * 2 + 32;  // q row pitch: the four rows of a load phase in different banks
    static constexpr int OFF_V = STAGES * TILE;
    static constexpr int OFF_Q = 2 * STAGES * TILE;
    static constexpr int OFF_ROW = OFF_Q + 16 * ML * QP;
    static constexpr int OFF_BAR = (OFF_ROW + 5 * 16 * ML * 4 + 15) & ~15;  // k_full, k_empty, v_full, v_empty
    static constexpr int OFF_FLAG = OFF_BAR + 4 * STAGES * 8;
    static constexpr int OFF_IDS = (OFF_FLAG + 4 + 15) & ~15;
    static constexpr int SMEM = OFF_IDS + 2 * kQ8MaxBoxes * 4 + 1024;
    static constexpr int THREADS = NW * 32 + 64;
    static constexpr int MERGE = NW * (DP / 8) * 32 * 16 + NW * 32 * 16;
    static_assert(KPW % (16 * CK) == 0, "keys per warp");
    static_assert((DP / 16) % KW == 0, "columns per warp in the merge");
    static_assert(MERGE <= 2 * STAGES * TILE, "merge scratch");
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

// One (sequence, kv head, row tile, split) on a CTA, whose rings go through n_done tiles.  Returns
// whether there was work (uniform).
template <typename T, int DP, int MG, int NW, int NT, int STAGES, int ML>
__device__ __forceinline__ bool decode_q8_unit(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Q8Params& p,
                                               uint8_t* smem, int b, int hk, int rt, int split, int g0,
                                               int& n_done) {
    using C = Q8Cfg<DP, MG, NW, NT, STAGES, ML>;
    constexpr int M = C::M;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    TileView tv;
    n_done = 0;
    if (!tile_view<M, NT>(p, b, rt, tv, split == 0)) return false;
    bool single;
    int t_begin, n_iter;
    if (!q8_tiles(p, tv, split, t_begin, n_iter, single)) return false;
    n_done = n_iter;
    const int kbeg = tv.kt0 + t_begin * NT;

    const Q8Rows rows = q8_rows(smem + C::OFF_ROW, M);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* k_empty = k_full + STAGES;
    uint64_t* v_full = k_empty + STAGES;
    uint64_t* v_empty = v_full + STAGES;
    volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(smem + C::OFF_FLAG);
    if (warp >= NW) {
        int* ids = reinterpret_cast<int*>(smem + C::OFF_IDS);
        if (warp == NW)
            q8_produce<DP, NT, STAGES>(p, &tm_k, smem, k_full, k_empty, ids, true, b, hk, tv.sk, kbeg, n_iter, g0, abort_flag);
        else
            q8_produce<DP, NT, STAGES>(p, &tm_v, smem + C::OFF_V, v_full, v_empty, ids + kQ8MaxBoxes, false, b, hk, tv.sk,
                                       kbeg, n_iter, g0, abort_flag);
        if (p.cluster > 1) q8_cluster_passive();
        return true;
    }
    q8_row_bounds(p, tv, rows, hk, M);
    const int rg = warp / C::KW, kq = warp % C::KW;
    constexpr int BPT = C::KPW / 32;  // blocks of 32 keys of this warp's slice of a tile
    static_assert(C::KPW % 32 == 0 && C::CK == 2, "a block is two chunks");
    auto block_key = [&](int n) { return kbeg + (n / BPT) * NT + kq * C::KPW + (n % BPT) * 32; };
    Q8Scales scales;
    scales.fetch(p, b, hk, tv.sk, 0, n_iter * BPT, block_key);
    q8_stage_q<T, DP, M, NW>(p, tv, rows, smem + C::OFF_Q, C::QP, hk, warp, lane);
    named_barrier_sync(1, NW * 32);

    const int gq = lane >> 2, tq = lane & 3;
    const int mi = lane >> 3, rr = lane & 7;
    const int r0 = rg * 16 + gq, r1 = r0 + 8;
    const int lo0 = rows.lo[r0], hi0 = rows.hi[r0], lo1 = rows.lo[r1], hi1 = rows.hi[r1];
    const int dg0 = rows.dg[r0], dg1 = rows.dg[r1];
    const float ab0 = rows.ab[r0], ab1 = rows.ab[r1];
    const float c0 = rows.sc[r0], c1 = rows.sc[r1];
    const uint8_t* q0p = smem + C::OFF_Q + r0 * C::QP + tq * 8;
    const uint8_t* q1p = smem + C::OFF_Q + r1 * C::QP + tq * 8;
    // A fragment of k-step ks: columns 16 ks + 4 tq + {0, 1} and + {2, 3} of rows r0 and r1
    auto q_frag = [&](int ks, uint32_t (&a)[4]) {
        const uint2 x = *reinterpret_cast<const uint2*>(q0p + ks * 32), y = *reinterpret_cast<const uint2*>(q1p + ks * 32);
        a[0] = x.x;
        a[1] = y.x;
        a[2] = x.y;
        a[3] = y.y;
    };
    int plain_lo = max(lo0, lo1), plain_hi = min(hi0, hi1);
    q8_plain_keys(p.alibi != nullptr, plain_lo, plain_hi);
    uint32_t qf[DP / 16][4];
#pragma unroll
    for (int ks = 0; ks < DP / 16; ++ks) q_frag(ks, qf[ks]);
    float o[DP / 8][4];  // [2 x unit + column parity]
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    bool ok = true;

    for (int it = 0; ok && it < n_iter; ++it) {
        const int gi = g0 + it, stage = gi % STAGES;
        const uint32_t par = (gi / STAGES) & 1;
        const int kt = kbeg + it * NT;
        const int key0 = kq * C::KPW;
        const uint32_t k_base = smem_addr(smem + stage * C::TILE), v_base = smem_addr(smem + C::OFF_V + stage * C::TILE);
        // V rows of this warp's slice that no row of the tile attends become 0 (0 x NaN is NaN):
        // keys before the first interval, past the last, and slots that were never loaded
        const int z_lo = min(max(tv.lo - kt, key0), key0 + C::KPW), z_hi = min(max(tv.hi + 1 - kt, key0), key0 + C::KPW);
        const bool zeroed = z_lo > key0 || z_hi < key0 + C::KPW;
        ok = __all_sync(0xffffffffu, q8_wait(&k_full[stage], par, abort_flag, p.err, p.wait_ns));
        if (!ok) break;
#pragma unroll
        for (int kb = 0; kb < C::KPW / (16 * C::CK); ++kb) {
            float s[C::CK][2][4];
#pragma unroll
            for (int kc = 0; kc < C::CK; ++kc) {
                const int kk0 = key0 + (kb * C::CK + kc) * 16;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[kc][n][e] = 0.f;
#pragma unroll
                for (int kp = 0; kp < DP / 32; ++kp) {
                    uint32_t b0, b1, b2, b3;  // (keys 0..7, k-step 2 kp), (same, 2 kp + 1), (keys 8..15, ...)
                    ldsm_x4(k_base + q8_off<DP, NT>(kk0 + rr + ((mi >> 1) << 3), 2 * kp + (mi & 1)), b0, b1, b2, b3);
                    uint32_t a0[4], a1[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        a0[e] = qf[2 * kp][e];
                        a1[e] = qf[2 * kp + 1][e];
                    }
                    MmaOp<__half>::run(s[kc][0], a0, e4m3x2_to_half2(b0), e4m3x2_hi_to_half2(b0));
                    MmaOp<__half>::run(s[kc][1], a0, e4m3x2_to_half2(b2), e4m3x2_hi_to_half2(b2));
                    MmaOp<__half>::run(s[kc][0], a1, e4m3x2_to_half2(b1), e4m3x2_hi_to_half2(b1));
                    MmaOp<__half>::run(s[kc][1], a1, e4m3x2_to_half2(b3), e4m3x2_hi_to_half2(b3));
                }
            }
            if (kb + 1 == C::KPW / (16 * C::CK)) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&k_empty[stage]);
            }
            // scores, row maxima, weights
            float mx0 = -INFINITY, mx1 = -INFINITY;
            float kss, lv;
            scales.take(p, b, hk, tv.sk, it * BPT + kb, n_iter * BPT, block_key, kss, lv);
            const float inv = fast_exp2(-lv), k0 = c0 * kss, k1 = c1 * kss;
#pragma unroll
            for (int kc = 0; kc < C::CK; ++kc) {
                const int kk0 = key0 + (kb * C::CK + kc) * 16;
                if (kt + kk0 >= plain_lo && kt + kk0 + 15 <= plain_hi) {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        s[kc][n][0] = fmaf(s[kc][n][0], k0, lv);
                        s[kc][n][1] = fmaf(s[kc][n][1], k0, lv);
                        s[kc][n][2] = fmaf(s[kc][n][2], k1, lv);
                        s[kc][n][3] = fmaf(s[kc][n][3], k1, lv);
                        mx0 = max3f(mx0, s[kc][n][0], s[kc][n][1]);
                        mx1 = max3f(mx1, s[kc][n][2], s[kc][n][3]);
                    }
                    continue;
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = kt + kk0 + n * 8 + tq * 2 + (e & 1);
                        float& x = s[kc][n][e];
                        if (e < 2) {
                            x = q8_score(x, k0, lv, key >= lo0 && key <= hi0, ab0, dg0, key);
                            mx0 = fmaxf(mx0, x);
                        } else {
                            x = q8_score(x, k1, lv, key >= lo1 && key <= hi1, ab1, dg1, key);
                            mx1 = fmaxf(mx1, x);
                        }
                    }
            }
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
            const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
            if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
                const float f0 = n0 == -INFINITY ? 1.f : fast_exp2(m0 - n0);
                const float f1 = n1 == -INFINITY ? 1.f : fast_exp2(m1 - n1);
#pragma unroll
                for (int n = 0; n < DP / 8; ++n) {
                    o[n][0] *= f0;
                    o[n][1] *= f0;
                    o[n][2] *= f1;
                    o[n][3] *= f1;
                }
                l0 *= f0;
                l1 *= f1;
                m0 = n0;
                m1 = n1;
            }
            const float u0 = m0 == -INFINITY ? 0.f : m0 - kQ8Offset, u1 = m1 == -INFINITY ? 0.f : m1 - kQ8Offset;
            uint32_t pa[C::CK][4];
#pragma unroll
            for (int kc = 0; kc < C::CK; ++kc) {
                float w[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    w[n][0] = fast_exp2(s[kc][n][0] - u0);
                    w[n][1] = fast_exp2(s[kc][n][1] - u0);
                    w[n][2] = fast_exp2(s[kc][n][2] - u1);
                    w[n][3] = fast_exp2(s[kc][n][3] - u1);
                }
                l0 = fmaf((w[0][0] + w[0][1]) + (w[1][0] + w[1][1]), inv, l0);
                l1 = fmaf((w[0][2] + w[0][3]) + (w[1][2] + w[1][3]), inv, l1);
                pa[kc][0] = pack2<__half>(w[0][0], w[0][1]);
                pa[kc][1] = pack2<__half>(w[0][2], w[0][3]);
                pa[kc][2] = pack2<__half>(w[1][0], w[1][1]);
                pa[kc][3] = pack2<__half>(w[1][2], w[1][3]);
            }
            if (kb == 0) {
                ok = __all_sync(0xffffffffu, q8_wait(&v_full[stage], par, abort_flag, p.err, p.wait_ns));
                if (!ok) break;
                if (zeroed) {
                    uint8_t* vst = smem + C::OFF_V + stage * C::TILE;
                    for (int idx = lane; idx < C::KPW * (DP / 16); idx += 32) {
                        const int r = key0 + idx / (DP / 16), u = idx % (DP / 16);
                        if (r < z_lo || r >= z_hi)
                            *reinterpret_cast<uint4*>(vst + q8_off<DP, NT>(r, u)) = make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                }
            }
#pragma unroll
            for (int kc = 0; kc < C::CK; ++kc) {
                const int kk0 = key0 + (kb * C::CK + kc) * 16;
#pragma unroll
                for (int np = 0; np < DP / 32; ++np) {
                    uint32_t v[4];  // (keys 0..7, unit 2 np), (keys 8..15, same), (keys 0..7, unit 2 np + 1), ...
                    ldsm_x4_t(v_base + q8_off<DP, NT>(kk0 + rr + ((mi & 1) << 3), 2 * np + (mi >> 1)), v[0], v[1], v[2],
                              v[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = __byte_perm(v[e], 0, 0x3120);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        MmaOp<__half>::run(o[2 * (2 * np + j)], pa[kc], e4m3x2_to_half2(v[2 * j]),
                                           e4m3x2_to_half2(v[2 * j + 1]));
                        MmaOp<__half>::run(o[2 * (2 * np + j) + 1], pa[kc], e4m3x2_hi_to_half2(v[2 * j]),
                                           e4m3x2_hi_to_half2(v[2 * j + 1]));
                    }
                }
            }
        }
        if (!ok) break;
        if (zeroed) fence_proxy_async_smem();  // the stage is rewritten by TMA later
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_empty[stage]);
    }

    // ---- merge the key slices of each row group, each warp a share of the columns ----
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    const bool gave_up = named_barrier_or(1, NW * 32, !ok || *abort_flag != 0u);
    if (gave_up && p.cluster <= 1) return true;  // all leave together
    float4* xo = reinterpret_cast<float4*>(smem);  // [warp][n][lane], in the rings
    float4* xml = xo + NW * (DP / 8) * 32;         // [warp][lane]: m0, m1, l0, l1
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) xo[(warp * (DP / 8) + n) * 32 + lane] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
    xml[warp * 32 + lane] = make_float4(m0, m1, l0, l1);
    T* out = static_cast<T*>(p.out);
    if (p.cluster > 1) {
        if (gave_up && tid == 0) *abort_flag = 1u;
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        uint32_t bad = 0;
        for (int c = 0; c < p.cluster; ++c) bad |= ld_cluster_u32(cluster_addr(const_cast<uint32_t*>(abort_flag), c));
        if (bad == 0) {
            // the row group's maxima and sums over the KW slices of every CTA, then this CTA's and warp's
            // units of its columns
            const int n_part = p.cluster * C::KW;
            auto part = [&](int k) { return (rg * C::KW + k % C::KW); };
            float mm0 = -INFINITY, mm1 = -INFINITY, L0 = 0.f, L1 = 0.f;
#pragma unroll 4
            for (int k = 0; k < n_part; ++k) {
                const float4 ml = ld_cluster_f4(cluster_addr(&xml[part(k) * 32 + lane], k / C::KW));
                mm0 = fmaxf(mm0, ml.x);
                mm1 = fmaxf(mm1, ml.y);
            }
            const float w0 = mm0 == -INFINITY ? 0.f : mm0, w1 = mm1 == -INFINITY ? 0.f : mm1;
#pragma unroll 4
            for (int k = 0; k < n_part; ++k) {
                const float4 ml = ld_cluster_f4(cluster_addr(&xml[part(k) * 32 + lane], k / C::KW));
                L0 = fmaf(ml.z, fast_exp2(ml.x - w0), L0);
                L1 = fmaf(ml.w, fast_exp2(ml.y - w1), L1);
            }
            const float inv0 = L0 == 0.f ? 0.f : 1.f / L0, inv1 = L1 == 0.f ? 0.f : 1.f / L1;
            for (int u = split * C::KW + kq; u < DP / 16; u += n_part) {
                float x[2][4] = {};
#pragma unroll 2
                for (int k = 0; k < n_part; ++k) {
                    const float4 ml = ld_cluster_f4(cluster_addr(&xml[part(k) * 32 + lane], k / C::KW));
                    const float4 ev = ld_cluster_f4(cluster_addr(&xo[(part(k) * (DP / 8) + 2 * u) * 32 + lane], k / C::KW));
                    const float4 od = ld_cluster_f4(cluster_addr(&xo[(part(k) * (DP / 8) + 2 * u + 1) * 32 + lane], k / C::KW));
                    const float e0 = fast_exp2(ml.x - w0) * inv0, e1 = fast_exp2(ml.y - w1) * inv1;
                    x[0][0] = fmaf(e0, ev.x, x[0][0]);
                    x[0][1] = fmaf(e0, od.x, x[0][1]);
                    x[0][2] = fmaf(e0, ev.y, x[0][2]);
                    x[0][3] = fmaf(e0, od.y, x[0][3]);
                    x[1][0] = fmaf(e1, ev.z, x[1][0]);
                    x[1][1] = fmaf(e1, od.z, x[1][1]);
                    x[1][2] = fmaf(e1, ev.w, x[1][2]);
                    x[1][3] = fmaf(e1, od.w, x[1][3]);
                }
                const int d = u * 16 + tq * 4;
#pragma unroll
                for (int hr = 0; hr < 2; ++hr) {
                    const int row = hr ? r1 : r0;
                    if (row >= tv.rows || d >= p.D) continue;
                    const int rho = tv.row0 + row, i = rho / p.G;
                    const int64_t t = tv.q0 + i;
                    const int h = hk * p.G + (rho - i * p.G);
                    *reinterpret_cast<uint2*>(out + t * p.o_s0 + (int64_t)h * p.o_s1 + d) =
                        make_uint2(pack2<T>(x[hr][0], x[hr][1]), pack2<T>(x[hr][2], x[hr][3]));
                }
            }
            if (split == 0 && kq == 0 && tq == 0) {
#pragma unroll
                for (int hr = 0; hr < 2; ++hr) {
                    const int row = hr ? r1 : r0;
                    if (row >= tv.rows) continue;
                    const int rho = tv.row0 + row, i = rho / p.G;
                    const int64_t t = tv.q0 + i;
                    const int h = hk * p.G + (rho - i * p.G);
                    const float L = hr ? L1 : L0, mm = hr ? mm1 : mm0;
                    p.lse[(int64_t)h * p.lse_s0 + t + (int64_t)b * p.lse_sb] =
                        L == 0.f ? -INFINITY : (mm - kQ8Offset + log2f(L)) * 0.69314718055994531f;
                }
            }
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        return true;
    }
    named_barrier_sync(1, NW * 32);
    float f0[C::KW], f1[C::KW];
    float L0 = 0.f, L1 = 0.f, mm0 = -INFINITY, mm1 = -INFINITY;
#pragma unroll
    for (int k = 0; k < C::KW; ++k) {
        const float4 ml = xml[(rg * C::KW + k) * 32 + lane];
        mm0 = fmaxf(mm0, ml.x);
        mm1 = fmaxf(mm1, ml.y);
    }
    const float w0 = mm0 == -INFINITY ? 0.f : mm0, w1 = mm1 == -INFINITY ? 0.f : mm1;
#pragma unroll
    for (int k = 0; k < C::KW; ++k) {
        const float4 ml = xml[(rg * C::KW + k) * 32 + lane];
        f0[k] = fast_exp2(ml.x - w0);
        f1[k] = fast_exp2(ml.y - w1);
        L0 += f0[k] * ml.z;
        L1 += f1[k] * ml.w;
    }
    const float inv0 = L0 == 0.f ? 0.f : 1.f / L0, inv1 = L1 == 0.f ? 0.f : 1.f / L1;
    constexpr int UPW = (DP / 16) / C::KW;  // 16-column units this warp stores
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
        const int row = hr ? r1 : r0;
        if (row >= tv.rows) continue;
        const int rho = tv.row0 + row;
        const int i = rho / p.G, g = rho - i * p.G;
        const int64_t t = tv.q0 + i;
        const int h = hk * p.G + g;
        const float iv = hr ? inv1 : inv0;
#pragma unroll
        for (int uu = 0; uu < UPW; ++uu) {
            const int u = kq * UPW + uu, d = u * 16 + tq * 4;
            if (d >= p.D) continue;
            float x[4] = {0.f, 0.f, 0.f, 0.f};  // columns d .. d + 3: even, odd, even, odd
#pragma unroll
            for (int k = 0; k < C::KW; ++k) {
                const float4 ev = xo[((rg * C::KW + k) * (DP / 8) + 2 * u) * 32 + lane];
                const float4 od = xo[((rg * C::KW + k) * (DP / 8) + 2 * u + 1) * 32 + lane];
                const float f = hr ? f1[k] : f0[k];
                x[0] += f * (hr ? ev.z : ev.x);
                x[1] += f * (hr ? od.z : od.x);
                x[2] += f * (hr ? ev.w : ev.y);
                x[3] += f * (hr ? od.w : od.y);
            }
            if (single)
                *reinterpret_cast<uint2*>(out + t * p.o_s0 + (int64_t)h * p.o_s1 + d) =
                    make_uint2(pack2<T>(x[0] * iv, x[1] * iv), pack2<T>(x[2] * iv, x[3] * iv));
            else
                *reinterpret_cast<float4*>(p.part_o + ((int64_t)split * p.part_stride + t * p.H + h) * p.D + d) =
                    make_float4(x[0] * iv, x[1] * iv, x[2] * iv, x[3] * iv);
        }
        if (kq == 0 && tq == 0) {
            const float L = hr ? L1 : L0, mm = hr ? mm1 : mm0;
            const float lse = L == 0.f ? -INFINITY : (mm - kQ8Offset + log2f(L)) * 0.69314718055994531f;
            if (single)
                p.lse[(int64_t)h * p.lse_s0 + t + (int64_t)b * p.lse_sb] = lse;
            else
                p.part_lse[(int64_t)split * p.part_stride + t * p.H + h] = lse;
        }
    }
    return true;
}

// ---------------------------------------------------------------------------------------------
// The unit above for at most 8 rows (bf16) or 4 (f16), the common decode step: no conversion at all.
//
// A 16-row product has room for several e4m3 terms of each row beside one another, so q and the
// weights are written as sums of terms, t0 + t1 / 16 [+ t2 / 256], each the rounding of what the ones
// before leave (times 16), term t of row r in row t S + r of the product (S = 8 and two terms, or S = 4
// and three): one e4m3 product of K or V as they are in the cache takes all terms of a row, and
// the row's result is the sum over its terms.  Each term takes 4 significant bits and its remainder is
// at most half its last place: two terms hold a value to 2^-9, three to 2^-13, and the first term's
// scale (largest q of a row 224..448, largest weight 256) puts the absolute resolution at 2^-14 and
// 2^-18 of that scale.  Per 32 keys of 128 columns: 32 products and 16 ldmatrix, where the f16
// form takes 64 products, 16 ldmatrix, 128 conversions and their byte shuffles.  (The e4m3 mma.sync
// takes 20 cycles of a sub-partition's tensor pipe, two f16 ones of half its depth 17: it is the
// instructions around them that go.)
//
// Each warp takes 32 keys of a 128-key tile.  K rows are read in the order that leaves a lane with the
// scores of keys 4 t .. 4 t + 3 of each 16, which is how the weights' A fragment wants them.
template <typename T>
struct Q8Terms {
    static constexpr int N = std::is_same<T, __half>::value ? 3 : 2;
    static constexpr int S = N == 2 ? 8 : 4;   // rows a unit can have
    static constexpr int SW = N == 2 ? 4 : 2;  // with the terms in the product's columns
};
constexpr float kQ8TermOffset = 8.f;  // largest weight 2^8

// The terms of a row of q, eight columns a lane, each term `pitch` bytes after the one before; sc takes
// the power of two back out.  Whole warp.
template <typename T>
__device__ __forceinline__ void q8_store_terms(const uint4& x, bool store, uint8_t* dst, int pitch, float& sc) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float v[8], mx = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = unpack2<T>(w[e]);
        v[2 * e] = f.x;
        v[2 * e + 1] = f.y;
        mx = max3f(mx, fabsf(f.x), fabsf(f.y));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    // the largest power of two with mx 2^e2 <= 448 = 1.75 x 2^8; an infinite element makes the row NaN
    const int bits = __float_as_int(mx);
    const int e2 = min(126, 8 - ((bits >> 23) - 127) - ((bits & 0x7fffff) > 0x600000 ? 1 : 0));
    const float up = mx <= 3.4028235e38f ? __int_as_float((127 + e2) << 23) : NAN;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= up;
#pragma unroll
    for (int t = 0; t < Q8Terms<T>::N; ++t) {
        uint32_t c2[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            c2[e] = e4m3x2_take(v[2 * e], v[2 * e + 1]);
            v[2 * e] *= 16.f;
            v[2 * e + 1] *= 16.f;
        }
        if (store)
            *reinterpret_cast<uint2*>(dst + t * pitch) = make_uint2(c2[0] | (c2[1] << 16), c2[2] | (c2[3] << 16));
    }
    sc = __int_as_float((127 - e2) << 23);
}

template <typename T, int DP, int NW, int NT, int STAGES, int ML>
__device__ __forceinline__ bool decode_q8_few_rows(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Q8Params& p,
                                                   uint8_t* smem, int b, int hk, int split, int g0,
                                                   int& n_done) {
    using C = Q8Cfg<DP, 1, NW, NT, STAGES, ML>;
    constexpr int NTERM = Q8Terms<T>::N, S = Q8Terms<T>::S;
    constexpr int QP = DP + 16;  // q row pitch: eight rows of a fragment load in different banks
    static_assert(C::KPW == 32, "keys per warp");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    TileView tv;
    n_done = 0;
    if (!tile_view<16, NT>(p, b, 0, tv, split == 0)) return false;
    bool single;
    int t_begin, n_iter;
    if (!q8_tiles(p, tv, split, t_begin, n_iter, single)) return false;
    n_done = n_iter;
    const int kbeg = tv.kt0 + t_begin * NT;

    const Q8Rows rows = q8_rows(smem + C::OFF_ROW, 16);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* k_empty = k_full + STAGES;
    uint64_t* v_full = k_empty + STAGES;
    uint64_t* v_empty = v_full + STAGES;
    volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(smem + C::OFF_FLAG);
    if (warp >= NW) {
        int* ids = reinterpret_cast<int*>(smem + C::OFF_IDS);
        if (warp == NW)
            q8_produce<DP, NT, STAGES>(p, &tm_k, smem, k_full, k_empty, ids, true, b, hk, tv.sk, kbeg, n_iter, g0, abort_flag);
        else
            q8_produce<DP, NT, STAGES>(p, &tm_v, smem + C::OFF_V, v_full, v_empty, ids + kQ8MaxBoxes, false, b, hk, tv.sk,
                                       kbeg, n_iter, g0, abort_flag);
        if (p.cluster > 1) q8_cluster_passive();
        return true;
    }
    q8_row_bounds(p, tv, rows, hk, 16);
    auto block_key = [&](int n) { return kbeg + n * NT + warp * 32; };  // 32 aligned keys lie in one page
    Q8Scales scales;
    scales.fetch(p, b, hk, tv.sk, 0, n_iter, block_key);
    // q in its terms, warp w rows w, w + NW, ..., DP / 8 lanes a row; rows without a query are zero
    uint8_t* qs = smem + C::OFF_Q;
    {
        const T* q = static_cast<const T*>(p.q);
        uint4 x[S / NW];
#pragma unroll
        for (int k = 0; k < S / NW; ++k) {
            const int r = warp + k * NW, i = r / p.G, g = r - i * p.G;
            x[k] = make_uint4(0, 0, 0, 0);
            if (r < tv.rows && lane * 8 < p.D)
                x[k] = __ldg(reinterpret_cast<const uint4*>(q + (int64_t)(tv.q0 + i) * p.q_s0 +
                                                            (int64_t)(hk * p.G + g) * p.q_s1 + lane * 8));
        }
        if (S == 4 && lane * 8 < DP)  // the fourth slot of terms
            *reinterpret_cast<uint2*>(qs + (12 + warp) * QP + lane * 8) = make_uint2(0, 0);
#pragma unroll
        for (int k = 0; k < S / NW; ++k) {
            const int r = warp + k * NW;
            float sc;
            q8_store_terms<T>(x[k], lane * 8 < DP, qs + r * QP + lane * 8, S * QP, sc);
            if (lane == 0) rows.sc[r] = p.scale_log2 * sc;
        }
    }
    named_barrier_sync(1, NW * 32);

    const int gq = lane >> 2, tq = lane & 3;
    const int mi = lane >> 3, rr = lane & 7;
    const int row = gq % S;  // with S = 4 lanes of gq and gq + 4 work on the same row
    const int lo = rows.lo[row], hi = rows.hi[row], dg = rows.dg[row];
    const float ab = rows.ab[row], cs = rows.sc[row];
    int plain_lo = lo, plain_hi = hi;
    q8_plain_keys(p.alibi != nullptr, plain_lo, plain_hi);
    uint32_t qf[DP / 32][4];
#pragma unroll
    for (int ks = 0; ks < DP / 32; ++ks) {
        const uint8_t* a = qs + gq * QP + ks * 32 + tq * 4;
        qf[ks][0] = *reinterpret_cast<const uint32_t*>(a);
        qf[ks][1] = *reinterpret_cast<const uint32_t*>(a + 8 * QP);
        qf[ks][2] = *reinterpret_cast<const uint32_t*>(a + 16);
        qf[ks][3] = *reinterpret_cast<const uint32_t*>(a + 8 * QP + 16);
    }
    // key of row rr of an 8-key score tile (even or odd) of a 16-key half
    const int key_of = 4 * (rr >> 1) + (rr & 1);
    float o[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    float m = -INFINITY, l = 0.f;
    bool ok = true;

    const int key0 = warp * 32;
    for (int it = 0; ok && it < n_iter; ++it) {
        const int gi = g0 + it, stage = gi % STAGES;
        const uint32_t par = (gi / STAGES) & 1;
        const int kt = kbeg + it * NT + key0;  // the warp's first key
        ok = __all_sync(0xffffffffu, q8_wait(&k_full[stage], par, abort_flag, p.err, p.wait_ns));
        if (!ok) break;
        const uint32_t k_base = smem_addr(smem + stage * C::TILE), v_base = smem_addr(smem + C::OFF_V + stage * C::TILE);
        float kss, lv;
        scales.take(p, b, hk, tv.sk, it, n_iter, block_key, kss, lv);
        kss *= cs;
        float s[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < DP / 32; ++ks)
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 16-key halves: their even and odd score tiles
                uint32_t b0, b1, b2, b3;
                ldsm_x4(k_base + q8_off<DP, NT>(key0 + 16 * h + key_of + (mi & 2), 2 * ks + (mi & 1)), b0, b1, b2, b3);
                mma_e4m3(s[2 * h], qf[ks], b0, b1);
                mma_e4m3(s[2 * h + 1], qf[ks], b2, b3);
            }
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_empty[stage]);
        // this lane's scores of keys kt + 16 h + 4 tq + {0, 1, 2, 3}
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if constexpr (S == 8) {
                    x[2 * j + e] = fmaf(s[j][2 + e], 1.f / 16.f, s[j][e]);
                } else {  // terms 0 and 2 here and term 1 in lane gq ^ 4, or the other way round
                    const float mine = gq < 4 ? fmaf(s[j][2 + e], 1.f / 256.f, s[j][e]) : s[j][e] * (1.f / 16.f);
                    x[2 * j + e] = mine + __shfl_xor_sync(0xffffffffu, mine, 16);
                }
            }
        float mx = -INFINITY;
        if (kt >= plain_lo && kt + 31 <= plain_hi) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], kss, lv);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int key = kt + 16 * (i >> 2) + 4 * tq + (i & 3);
                x[i] = q8_score(x[i], kss, lv, key >= lo && key <= hi, ab, dg, key);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) mx = max3f(mx, x[i], x[i + 1]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (__any_sync(0xffffffffu, mx > m)) {
            const float nm = fmaxf(m, mx);
            const float f = nm == -INFINITY ? 1.f : fast_exp2(m - nm);
            m = nm;
            l *= f;
            // rows gq and gq + 8 of the product hold terms of the same row
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] *= f;
        }
        const float u = m == -INFINITY ? 0.f : m - kQ8TermOffset;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = fast_exp2(x[i] - u);
            sum += x[i];
        }
        l = fmaf(sum, fast_exp2(-lv), l);
        // the weights' terms: A rows gq (columns 4 tq .. + 3 of either half) and gq + 8
        uint32_t pa[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float* w = &x[4 * h];
            uint32_t t[3];
#pragma unroll
            for (int k = 0; k < NTERM; ++k) {
                const uint32_t c0 = e4m3x2_take(w[0], w[1]), c1 = e4m3x2_take(w[2], w[3]);
                t[k] = c0 | (c1 << 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] *= 16.f;
            }
            if constexpr (S == 8) {
                pa[2 * h] = t[0];
                pa[2 * h + 1] = t[1];
            } else {
                pa[2 * h] = gq < 4 ? t[0] : t[1];
                pa[2 * h + 1] = gq < 4 ? t[2] : 0u;
            }
        }
        ok = __all_sync(0xffffffffu, q8_wait(&v_full[stage], par, abort_flag, p.err, p.wait_ns));
        if (!ok) break;
        // V rows of this warp's keys that no row attends become 0 (0 x NaN is NaN): keys before the first
        // interval, past the last, and slots that were never loaded
        const bool zeroed = kt < tv.lo || kt + 31 > tv.hi;
        if (zeroed) {
            if (kt + lane < tv.lo || kt + lane > tv.hi) {
                uint8_t* vst = smem + C::OFF_V + stage * C::TILE;
#pragma unroll
                for (int un = 0; un < DP / 16; ++un)
                    *reinterpret_cast<uint4*>(vst + q8_off<DP, NT>(key0 + lane, un)) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
        }
#pragma unroll
        for (int un = 0; un < DP / 16; ++un) {
            uint32_t v0, v1, v2, v3;
            ldsm_b8_x2_t(v_base + q8_off<DP, NT>(key0 + lane, un), v0, v1, v2, v3);
            mma_e4m3(o[2 * un], pa, v0, v2);
            mma_e4m3(o[2 * un + 1], pa, v1, v3);
        }
        if (zeroed) fence_proxy_async_smem();  // the stage is rewritten by TMA later
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_empty[stage]);
    }

    // ---- sum the terms, then merge the key slices of the warps, each a share of the columns ----
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const bool gave_up = named_barrier_or(1, NW * 32, !ok || *abort_flag != 0u);
    if (gave_up && p.cluster <= 1) return true;  // all leave together
    float2* xo = reinterpret_cast<float2*>(smem);  // [warp][n][lane], in the rings
    float2* xml = xo + NW * (DP / 8) * 32;         // [warp][lane]: m, l
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
        float2 v;
        if constexpr (S == 8) {
            v = make_float2(fmaf(o[n][2], 1.f / 16.f, o[n][0]), fmaf(o[n][3], 1.f / 16.f, o[n][1]));
        } else {
            v = gq < 4 ? make_float2(fmaf(o[n][2], 1.f / 256.f, o[n][0]), fmaf(o[n][3], 1.f / 256.f, o[n][1]))
                       : make_float2(o[n][0] * (1.f / 16.f), o[n][1] * (1.f / 16.f));
            v.x += __shfl_xor_sync(0xffffffffu, v.x, 16);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, 16);
        }
        xo[(warp * (DP / 8) + n) * 32 + lane] = v;
    }
    xml[warp * 32 + lane] = make_float2(m, l);
    const int oi = row / p.G, oh = hk * p.G + (row - oi * p.G);  // the row's query and head
    T* orow = static_cast<T*>(p.out) + ((int64_t)tv.q0 + oi) * p.o_s0 + (int64_t)oh * p.o_s1;
    const bool mine = gq < S && gq < tv.rows;
    if (p.cluster > 1) {
        if (gave_up && tid == 0) *abort_flag = 1u;
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        uint32_t bad = 0;
        for (int c = 0; c < p.cluster; ++c) bad |= ld_cluster_u32(cluster_addr(const_cast<uint32_t*>(abort_flag), c));
        if (bad == 0 && mine) {
            const int n_part = p.cluster * NW;
            float mm = -INFINITY, L = 0.f;
#pragma unroll 8
            for (int k = 0; k < n_part; ++k)
                mm = fmaxf(mm, ld_cluster_f2(cluster_addr(&xml[(k % NW) * 32 + lane], k / NW)).x);
            const float um = mm == -INFINITY ? 0.f : mm;
#pragma unroll 8
            for (int k = 0; k < n_part; ++k) {
                const float2 ml = ld_cluster_f2(cluster_addr(&xml[(k % NW) * 32 + lane], k / NW));
                L = fmaf(ml.y, fast_exp2(ml.x - um), L);
            }
            const float iv = L == 0.f ? 0.f : 1.f / L;
            for (int n = split * NW + warp; n < DP / 8; n += n_part) {
                float x0 = 0.f, x1 = 0.f;
#pragma unroll 8
                for (int k = 0; k < n_part; ++k) {
                    const float2 ml = ld_cluster_f2(cluster_addr(&xml[(k % NW) * 32 + lane], k / NW));
                    const float2 v = ld_cluster_f2(cluster_addr(&xo[((k % NW) * (DP / 8) + n) * 32 + lane], k / NW));
                    const float e = fast_exp2(ml.x - um) * iv;
                    x0 = fmaf(e, v.x, x0);
                    x1 = fmaf(e, v.y, x1);
                }
                const int d = n * 8 + tq * 2;
                if (d < p.D) *reinterpret_cast<uint32_t*>(orow + d) = pack2<T>(x0, x1);
            }
            if (split == 0 && warp == 0 && tq == 0)
                p.lse[(int64_t)oh * p.lse_s0 + tv.q0 + oi + (int64_t)b * p.lse_sb] =
                    L == 0.f ? -INFINITY : (mm - kQ8TermOffset + log2f(L)) * 0.69314718055994531f;
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        return true;
    }
    named_barrier_sync(1, NW * 32);
    float f[NW], L = 0.f, mm = -INFINITY;
#pragma unroll
    for (int k = 0; k < NW; ++k) mm = fmaxf(mm, xml[k * 32 + lane].x);
    const float um = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
        const float2 ml = xml[k * 32 + lane];
        f[k] = fast_exp2(ml.x - um);
        L += f[k] * ml.y;
    }
    if (!mine) return true;
    const float iv = L == 0.f ? 0.f : 1.f / L;
    const int64_t t = tv.q0 + oi;
#pragma unroll
    for (int nn = 0; nn < (DP / 8) / NW; ++nn) {
        const int n = warp * ((DP / 8) / NW) + nn, d = n * 8 + tq * 2;
        if (d >= p.D) continue;
        float x0 = 0.f, x1 = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const float2 v = xo[(k * (DP / 8) + n) * 32 + lane];
            x0 = fmaf(f[k], v.x, x0);
            x1 = fmaf(f[k], v.y, x1);
        }
        if (single)
            *reinterpret_cast<uint32_t*>(orow + d) = pack2<T>(x0 * iv, x1 * iv);
        else
            *reinterpret_cast<float2*>(p.part_o + ((int64_t)split * p.part_stride + t * p.H + oh) * p.D + d) =
                make_float2(x0 * iv, x1 * iv);
    }
    if (warp == 0 && tq == 0) {
        const float lse = L == 0.f ? -INFINITY : (mm - kQ8TermOffset + log2f(L)) * 0.69314718055994531f;
        if (single)
            p.lse[(int64_t)oh * p.lse_s0 + t + (int64_t)b * p.lse_sb] = lse;
        else
            p.part_lse[(int64_t)split * p.part_stride + t * p.H + oh] = lse;
    }
    return true;
}

// The same for at most 4 rows (bf16) or 2 (f16), a group of 4 heads or fewer for one token: all terms of
// all rows fit the 8 columns of a product, so K and V are its 16-row operand and q and the weights the
// other, and 32 keys of 128 columns take 16 products, half the softmax and half the accumulators.
// Term t of row r is column TS r + t (TS = 2, or 4 with three terms): lane 4 g + t holds columns 2 t
// and 2 t + 1, so of bf16 both terms of row t.
//
//   S^T = K q^T: keys are rows; lane 4 g + t has four keys of its row, k(g, j) = 8 j + (g + 2 j) % 8, j = 0..3.
//   O^T = V^T w^T: columns of V are rows; the weights go through 256 bytes of shared memory a warp to
//   get from a lane per key to a lane per column, as term words w(4 g + j) of keys k(g, j), and the rows of V
//   are read in that order.  Both orders leave every eight rows of an ldmatrix in different banks.
template <typename T, int DP, int NW, int NT, int STAGES, int ML>
__device__ __forceinline__ bool decode_q8_swapped(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Q8Params& p,
                                                  uint8_t* smem, int b, int hk, int split, int g0, int& n_done) {
    using C = Q8Cfg<DP, 1, NW, NT, STAGES, ML>;
    constexpr int NTERM = Q8Terms<T>::N, TS = NTERM == 2 ? 2 : 4, S = Q8Terms<T>::SW;
    constexpr int QP = DP + 16;            // q column pitch: eight columns of a fragment load in different banks
    constexpr int WP = 12;                 // words between the columns of a warp's weights, likewise
    constexpr int OFF_W = C::OFF_Q + 8 * QP;
    static_assert(C::KPW == 32 && S <= NW && 8 * QP + NW * 8 * WP * 4 <= 16 * ML * C::QP, "shared memory of q");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    TileView tv;
    n_done = 0;
    if (!tile_view<16, NT>(p, b, 0, tv, split == 0)) return false;
    bool single;
    int t_begin, n_iter;
    if (!q8_tiles(p, tv, split, t_begin, n_iter, single)) return false;
    n_done = n_iter;
    const int kbeg = tv.kt0 + t_begin * NT;

    const Q8Rows rows = q8_rows(smem + C::OFF_ROW, 16);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* k_empty = k_full + STAGES;
    uint64_t* v_full = k_empty + STAGES;
    uint64_t* v_empty = v_full + STAGES;
    volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(smem + C::OFF_FLAG);
    if (warp >= NW) {
        int* ids = reinterpret_cast<int*>(smem + C::OFF_IDS);
        if (warp == NW)
            q8_produce<DP, NT, STAGES>(p, &tm_k, smem, k_full, k_empty, ids, true, b, hk, tv.sk, kbeg, n_iter, g0, abort_flag);
        else
            q8_produce<DP, NT, STAGES>(p, &tm_v, smem + C::OFF_V, v_full, v_empty, ids + kQ8MaxBoxes, false, b, hk, tv.sk,
                                       kbeg, n_iter, g0, abort_flag);
        if (p.cluster > 1) q8_cluster_passive();
        return true;
    }
    q8_row_bounds(p, tv, rows, hk, 16);
    auto block_key = [&](int n) { return kbeg + n * NT + warp * 32; };  // 32 aligned keys lie in one page
    Q8Scales scales;
    scales.fetch(p, b, hk, tv.sk, 0, n_iter, block_key);
    uint8_t* qs = smem + C::OFF_Q;
    if (warp < S) {  // q in its terms, a row a warp; rows without a query are zero
        const int r = warp, i = r / p.G, g = r - i * p.G;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < tv.rows && lane * 8 < p.D)
            x = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (int64_t)(tv.q0 + i) * p.q_s0 +
                                                     (int64_t)(hk * p.G + g) * p.q_s1 + lane * 8));
        float sc;
        q8_store_terms<T>(x, lane * 8 < DP, qs + r * TS * QP + lane * 8, QP, sc);
        if (TS > NTERM && lane * 8 < DP) *reinterpret_cast<uint2*>(qs + (r * TS + NTERM) * QP + lane * 8) = make_uint2(0, 0);
        if (lane == 0) rows.sc[r] = p.scale_log2 * sc;
    }
    named_barrier_sync(1, NW * 32);

    const int gq = lane >> 2, tq = lane & 3;
    const int mi = lane >> 3, rr = lane & 7;
    const int row = TS == 2 ? tq : tq >> 1;
    const bool first = TS == 2 || (tq & 1) == 0;  // holds terms 0 and 1 (and not term 2)
    const int lo = rows.lo[row], hi = rows.hi[row], dg = rows.dg[row];
    const float ab = rows.ab[row], cs = rows.sc[row];
    int plain_lo = lo, plain_hi = hi;
    q8_plain_keys(p.alibi != nullptr, plain_lo, plain_hi);
    uint32_t qf[DP / 32][2];
#pragma unroll
    for (int ks = 0; ks < DP / 32; ++ks) {
        qf[ks][0] = *reinterpret_cast<const uint32_t*>(qs + gq * QP + ks * 32 + tq * 4);
        qf[ks][1] = *reinterpret_cast<const uint32_t*>(qs + gq * QP + ks * 32 + 16 + tq * 4);
    }
    auto key_at = [](int g, int j) { return 8 * j + ((g + 2 * j) & 7); };
    auto sum_terms = [&](float c0, float c1) { return first ? fmaf(c1, 1.f / 16.f, c0) : c0 * (1.f / 256.f); };
    uint32_t* wbuf = reinterpret_cast<uint32_t*>(smem + OFF_W) + warp * 8 * WP;
    float o[DP / 16][4];  // columns 16 u + gq and + 8 of V, this lane's two terms each
#pragma unroll
    for (int u = 0; u < DP / 16; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[u][e] = 0.f;
    float m = -INFINITY, l = 0.f;
    bool ok = true;

    const int key0 = warp * 32, v_row = key0 + key_at(lane >> 2, lane & 3);
    for (int it = 0; ok && it < n_iter; ++it) {
        const int gi = g0 + it, stage = gi % STAGES;
        const uint32_t par = (gi / STAGES) & 1;
        const int kt = kbeg + it * NT + key0;  // the warp's first key
        ok = __all_sync(0xffffffffu, q8_wait(&k_full[stage], par, abort_flag, p.err, p.wait_ns));
        if (!ok) break;
        const uint32_t k_base = smem_addr(smem + stage * C::TILE), v_base = smem_addr(smem + C::OFF_V + stage * C::TILE);
        float kss, lv;
        scales.take(p, b, hk, tv.sk, it, n_iter, block_key, kss, lv);
        kss *= cs;
        float s[2][2][4];  // [chain][16-key tile]
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[c][h][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < DP / 32; ++ks)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a[4];
                ldsm_x4(k_base + q8_off<DP, NT>(key0 + key_at(rr, 2 * h + (mi & 1)), 2 * ks + (mi >> 1)), a[0], a[1], a[2], a[3]);
                mma_e4m3(s[ks & 1][h], a, qf[ks][0], qf[ks][1]);
            }
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_empty[stage]);
        float x[4];  // of keys k(gq, j)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int h = j >> 1, e = 2 * (j & 1);
            x[j] = sum_terms(s[0][h][e] + s[1][h][e], s[0][h][e + 1] + s[1][h][e + 1]);
            if (TS == 4) x[j] += __shfl_xor_sync(0xffffffffu, x[j], 1);
        }
        if (kt >= plain_lo && kt + 31 <= plain_hi) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = fmaf(x[j], kss, lv);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = kt + key_at(gq, j);
                x[j] = q8_score(x[j], kss, lv, key >= lo && key <= hi, ab, dg, key);
            }
        }
        float mx = max3f(x[0], x[1], fmaxf(x[2], x[3]));
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        if (__any_sync(0xffffffffu, mx > m)) {
            const float nm = fmaxf(m, mx);
            const float f = nm == -INFINITY ? 1.f : fast_exp2(m - nm);
            m = nm;
            l *= f;
#pragma unroll
            for (int u = 0; u < DP / 16; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[u][e] *= f;
        }
        const float ref = m == -INFINITY ? 0.f : m - kQ8TermOffset;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = fast_exp2(x[j] - ref);
            sum += x[j];
        }
        l = fmaf(sum, fast_exp2(-lv), l);
        uint32_t t[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < NTERM; ++k) {
            const uint32_t c0 = e4m3x2_take(x[0], x[1]), c1 = e4m3x2_take(x[2], x[3]);
            t[k] = c0 | (c1 << 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] *= 16.f;
        }
        wbuf[2 * tq * WP + gq] = first ? t[0] : t[2];
        wbuf[(2 * tq + 1) * WP + gq] = first ? t[1] : 0u;
        __syncwarp();
        const uint32_t w0 = wbuf[gq * WP + tq], w1 = wbuf[gq * WP + 4 + tq];
        ok = __all_sync(0xffffffffu, q8_wait(&v_full[stage], par, abort_flag, p.err, p.wait_ns));
        if (!ok) break;
        // V rows of this warp's keys that no row attends become 0 (0 x NaN is NaN): keys before the first
        // interval, past the last, and slots that were never loaded
        const bool zeroed = kt < tv.lo || kt + 31 > tv.hi;
        if (zeroed) {
            if (kt + lane < tv.lo || kt + lane > tv.hi) {
                uint8_t* vst = smem + C::OFF_V + stage * C::TILE;
#pragma unroll
                for (int u = 0; u < DP / 16; ++u)
                    *reinterpret_cast<uint4*>(vst + q8_off<DP, NT>(key0 + lane, u)) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
        }
#pragma unroll
        for (int u = 0; u < DP / 16; ++u) {
            uint32_t a[4];
            ldsm_b8_x2_t(v_base + q8_off<DP, NT>(v_row, u), a[0], a[1], a[2], a[3]);
            mma_e4m3(o[u], a, w0, w1);
        }
        if (zeroed) fence_proxy_async_smem();  // the stage is rewritten by TMA later
        __syncwarp();                          // (and the weights by the next step)
        if (lane == 0) mbar_arrive(&v_empty[stage]);
    }

    // ---- sum the terms, then merge the key slices of the warps (and of the cluster's CTAs) ----
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    const bool gave_up = named_barrier_or(1, NW * 32, !ok || *abort_flag != 0u);
    if (gave_up && p.cluster <= 1) return true;  // all leave together
    constexpr int OP = DP + 8;                           // row pitch of a warp's sums
    float* xo = reinterpret_cast<float*>(smem);          // [warp][row][column], in the rings
    float2* xml = reinterpret_cast<float2*>(xo + NW * S * OP);  // [warp][row]: m, l
#pragma unroll
    for (int u = 0; u < DP / 16; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float v = sum_terms(o[u][2 * e], o[u][2 * e + 1]);
            if (TS == 4) v += __shfl_xor_sync(0xffffffffu, v, 1);
            if (first) xo[(warp * S + row) * OP + 16 * u + 8 * e + gq] = v;
        }
    if (gq == 0 && first) xml[warp * S + row] = make_float2(m, l);
    auto emit = [&](int r, int d, float mm, float L, float x0, float x1) {
        const int i = r / p.G, h = hk * p.G + (r - i * p.G);
        const int64_t t = tv.q0 + i;
        if (single)
            *reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + t * p.o_s0 + (int64_t)h * p.o_s1 + d) = pack2<T>(x0, x1);
        else
            *reinterpret_cast<float2*>(p.part_o + ((int64_t)split * p.part_stride + t * p.H + h) * p.D + d) =
                make_float2(x0, x1);
        if (d == 0) {
            const float lse = L == 0.f ? -INFINITY : (mm - kQ8TermOffset + log2f(L)) * 0.69314718055994531f;
            if (single)
                p.lse[(int64_t)h * p.lse_s0 + t + (int64_t)b * p.lse_sb] = lse;
            else
                p.part_lse[(int64_t)split * p.part_stride + t * p.H + h] = lse;
        }
    };
    if (p.cluster > 1) {
        if (gave_up && tid == 0) *abort_flag = 1u;
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        uint32_t bad = 0;
        for (int c = 0; c < p.cluster; ++c) bad |= ld_cluster_u32(cluster_addr(const_cast<uint32_t*>(abort_flag), c));
        const int n_part = p.cluster * NW;
        for (int i = tid * p.cluster + split; bad == 0 && i < S * DP / 2; i += NW * 32 * p.cluster) {
            const int r = i / (DP / 2), d = i % (DP / 2) * 2;
            if (r >= tv.rows || d >= p.D) continue;
            float mm = -INFINITY, L = 0.f, x0 = 0.f, x1 = 0.f;
#pragma unroll 8
            for (int k = 0; k < n_part; ++k) mm = fmaxf(mm, ld_cluster_f2(cluster_addr(&xml[k % NW * S + r], k / NW)).x);
            const float um = mm == -INFINITY ? 0.f : mm;
#pragma unroll 8
            for (int k = 0; k < n_part; ++k) {
                const float2 ml = ld_cluster_f2(cluster_addr(&xml[k % NW * S + r], k / NW));
                const float2 v = ld_cluster_f2(cluster_addr(&xo[(k % NW * S + r) * OP + d], k / NW));
                const float f = fast_exp2(ml.x - um);
                L = fmaf(ml.y, f, L);
                x0 = fmaf(f, v.x, x0);
                x1 = fmaf(f, v.y, x1);
            }
            const float iv = L == 0.f ? 0.f : 1.f / L;
            emit(r, d, mm, L, x0 * iv, x1 * iv);
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        return true;
    }
    named_barrier_sync(1, NW * 32);
    for (int i = tid; i < S * DP / 2; i += NW * 32) {
        const int r = i / (DP / 2), d = i % (DP / 2) * 2;
        if (r >= tv.rows || d >= p.D) continue;
        float mm = -INFINITY, L = 0.f, x0 = 0.f, x1 = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) mm = fmaxf(mm, xml[k * S + r].x);
        const float um = mm == -INFINITY ? 0.f : mm;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const float2 ml = xml[k * S + r], v = *reinterpret_cast<const float2*>(&xo[(k * S + r) * OP + d]);
            const float f = fast_exp2(ml.x - um);
            L = fmaf(ml.y, f, L);
            x0 = fmaf(f, v.x, x0);
            x1 = fmaf(f, v.y, x1);
        }
        const float iv = L == 0.f ? 0.f : 1.f / L;
        emit(r, d, mm, L, x0 * iv, x1 * iv);
    }
    return true;
}

// The sequence of a grid index: longest first (order from a ranking pass, or ranked here).
__device__ __forceinline__ int q8_sequence(const SplitParams& p, int* rank_len, int* rank_pick) {
    const int z = (int)blockIdx.z, tid = threadIdx.x;
    if (p.order) return p.order[z];
    if (!p.rank_in_cta) return z;
    if (tid < p.batch) rank_len[tid] = p.cu_k[tid + 1] - p.cu_k[tid];
    if (tid == 0) *rank_pick = z;
    __syncthreads();
    if (tid < p.batch) {
        const int ls = rank_len[tid];
        int rank = 0;
        for (int t = 0; t < p.batch; ++t) {
            const int lt = rank_len[t];
            rank += (lt > ls) || (lt == ls && t < tid);
        }
        if (rank == z) *rank_pick = tid;
    }
    __syncthreads();
    return *rank_pick;
}

template <typename T, int DP, int MG, int NW, int NT, int STAGES>
__global__ void __launch_bounds__(NW * 32 + 64, 2)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const Q8Params p) {
    using C = Q8Cfg<DP, MG, NW, NT, STAGES>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x;
    allow_dependent_launch();
    if (tid == NW * 32) prefetch_tmap(&tm_k);
    if (tid == NW * 32 + 32) prefetch_tmap(&tm_v);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(smem + C::OFF_FLAG);
    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&bars[s], 1);                // k_full
            mbar_init(&bars[STAGES + s], NW);      // k_empty
            mbar_init(&bars[2 * STAGES + s], 1);   // v_full
            mbar_init(&bars[3 * STAGES + s], NW);  // v_empty
        }
        *abort_flag = 0u;
        fence_mbar_init();
    }
    __syncthreads();
    // A sequence of few rows runs on the body for them, and in a kernel for two row groups one of at
    // most 16 rows on the one-group body.
    auto run_unit = [&](int b, int hk, int rt, int split, int g0, int& n_done) -> bool {
        const int64_t n_rows = b >= 0 && b < p.batch ? (int64_t)(p.cu_q[b + 1] - p.cu_q[b]) * p.G : INT32_MAX;
        if (rt == 0 && n_rows <= Q8Terms<T>::SW)
            return decode_q8_swapped<T, DP, NW, NT, STAGES, MG>(tm_k, tm_v, p, smem, b, hk, split, g0, n_done);
        if (rt == 0 && n_rows <= Q8Terms<T>::S)
            return decode_q8_few_rows<T, DP, NW, NT, STAGES, MG>(tm_k, tm_v, p, smem, b, hk, split, g0, n_done);
        if constexpr (MG == 2) {
            using L1 = Q8Cfg<DP, 1, NW, NT, STAGES, 2>;
            static_assert(L1::OFF_ROW == C::OFF_ROW && L1::OFF_BAR == C::OFF_BAR && L1::OFF_IDS == C::OFF_IDS &&
                              L1::SMEM == C::SMEM,
                          "both bodies share one shared-memory layout");
            if (n_rows <= 16)
                return decode_q8_unit<T, DP, 1, NW, NT, STAGES, 2>(tm_k, tm_v, p, smem, b, hk, rt, split, g0, n_done);
        }
        return decode_q8_unit<T, DP, MG, NW, NT, STAGES, MG>(tm_k, tm_v, p, smem, b, hk, rt, split, g0, n_done);
    };
    if (p.work) {  // persistent: (sequence, split) x kv head items in list order
        __shared__ int s_item;
        const int total = p.work[1] * p.Hkv;
        int g0 = 0;
        for (;;) {
            if (tid == 0) s_item = atomicAdd(p.work, 1);
            __syncthreads();
            const int w = s_item;
            if (w >= total) break;
            const int pair = w / p.Hkv;
            int n_done = 0;
            run_unit(p.work[2 + 2 * pair], w - pair * p.Hkv, 0, p.work[3 + 2 * pair], g0, n_done);
            fence_proxy_async_smem();  // the merge's writes come before the next item's copies
            __syncthreads();
            if (*abort_flag) break;
            g0 += n_done;
        }
        return;
    }
    __shared__ int rank_len[kRankInCta];
    __shared__ int rank_pick;
    const int b = q8_sequence(p, rank_len, &rank_pick);
    if (tid >= NW * 32 && tid < NW * 32 + 32) prefetch_split_pages<NT>(p, b, (int)blockIdx.x, tid - NW * 32);
    int n_done = 0;
    run_unit(b, (int)blockIdx.y % p.Hkv, (int)blockIdx.y / p.Hkv, (int)blockIdx.x, 0, n_done);
}

// ---------------------------------------------------------------------------------------------
// decode_q8_wide_kernel: head_dim 129..512.
//
// One warp cannot hold 16 rows x 512 columns of O, and at 256 columns it spills.  Eight warps take key slices of a 64-key tile
// for Q.K^T (8 keys each of all 16 rows, or 16 keys of one of two row groups), write their
// weights to shared memory, and after one barrier take DP / 8-column slices for P.V, all keys and
// both row groups, so V is converted once.  The warps share one reference m per row: a tile whose
// scores all lie below m + 5 needs no exchange (weights up to 2^15 fit f16); otherwise, a vote
// folded into that barrier, they exchange row maxima, rescale and write the weights again.  The
// weights are double-buffered, so the common tile costs one barrier.
template <int DP_, int MG>
struct Q8WideCfg {
    static constexpr int DP = DP_, NW = 8, NT = 64, M = 16 * MG;
    static constexpr int KST = DP == 256 && MG == 2 ? 5 : 3, VST = DP == 256 && MG == 2 ? 5 : DP == 512 && MG == 1 ? 3 : 2;
    static constexpr int CTAS = DP == 256 && MG == 1 ? 2 : 1;  // an SM
    static constexpr int UW = DP / 16 / NW;         // 16-column units of a warp's slice
    static constexpr int KS = NW / MG;      // key slices
    static constexpr int NB = NT / KS / 8;  // 8-key tiles per warp
    static constexpr int TILE = NT * DP;
    static constexpr int QP = DP * 2 + 32;
    static constexpr int OFF_V = KST * TILE;
    static constexpr int OFF_P = OFF_V + VST * TILE;         // weights, two buffers of M rows x 128 bytes
    static constexpr int OFF_Q = OFF_P + 2 * M * 128;
    static constexpr int OFF_ROW = OFF_Q + M * QP;
    static constexpr int OFF_MAX = OFF_ROW + 5 * M * 4;      // [key slice][row]: maxima, then sums
    static constexpr int OFF_BAR = (OFF_MAX + KS * M * 4 + 15) & ~15;
    static constexpr int OFF_FLAG = OFF_BAR + (2 * KST + 2 * VST) * 8;
    static constexpr int OFF_IDS = (OFF_FLAG + 4 + 15) & ~15;
    static constexpr int SMEM = OFF_IDS + 2 * kQ8MaxBoxes * 4 + 1024;
    static constexpr int THREADS = NW * 32 + 64;
    static_assert(CTAS * (SMEM + 2048) <= 228 * 1024 && SMEM <= 227 * 1024, "shared memory");  // + static and reserved
};

template <typename T, int DP_, int MG>
__global__ void __launch_bounds__(Q8WideCfg<DP_, MG>::THREADS, Q8WideCfg<DP_, MG>::CTAS)
    decode_q8_wide_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const Q8Params p) {
    using C = Q8WideCfg<DP_, MG>;
    constexpr int DP = C::DP, UW = C::UW, NT = C::NT, NW = C::NW, M = C::M, NB = C::NB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    allow_dependent_launch();
    if (tid == NW * 32) prefetch_tmap(&tm_k);
    if (tid == NW * 32 + 32) prefetch_tmap(&tm_v);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* k_empty = k_full + C::KST;
    uint64_t* v_full = k_empty + C::KST;
    uint64_t* v_empty = v_full + C::VST;
    volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(smem + C::OFF_FLAG);
    if (tid == 0) {
        for (int s = 0; s < C::KST; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], NW);
        }
        for (int s = 0; s < C::VST; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], NW);
        }
        *abort_flag = 0u;
        fence_mbar_init();
    }
    __syncthreads();
    __shared__ int rank_len[kRankInCta];
    __shared__ int rank_pick;
    const int b = q8_sequence(p, rank_len, &rank_pick);
    const int hk = (int)blockIdx.y % p.Hkv, rt = (int)blockIdx.y / p.Hkv, split = (int)blockIdx.x;
    TileView tv;
    if (!tile_view<M, NT>(p, b, rt, tv, split == 0)) return;
    if (split >= max(tv.nsplit, 1)) return;
    const bool single = tv.nsplit <= 1;
    const int t_begin = split * p.split_tiles;
    const int n_iter = max(0, min(tv.ntiles, t_begin + p.split_tiles) - t_begin);
    const int kbeg = tv.kt0 + t_begin * NT;
    const Q8Rows rows = q8_rows(smem + C::OFF_ROW, M);
    float* xmax = reinterpret_cast<float*>(smem + C::OFF_MAX);
    if (warp >= NW) {
        int* ids = reinterpret_cast<int*>(smem + C::OFF_IDS);
        if (warp == NW)
            q8_produce<DP, NT, C::KST>(p, &tm_k, smem, k_full, k_empty, ids, true, b, hk, tv.sk, kbeg, n_iter, 0, abort_flag);
        else
            q8_produce<DP, NT, C::VST>(p, &tm_v, smem + C::OFF_V, v_full, v_empty, ids + kQ8MaxBoxes, false, b, hk, tv.sk,
                                       kbeg, n_iter, 0, abort_flag);
        return;
    }
    q8_row_bounds(p, tv, rows, hk, M);
    const int rg = warp / C::KS, slice = warp % C::KS;
    auto block_key = [&](int n) { return kbeg + n * NT + slice * NB * 8; };
    Q8Scales scales;
    scales.fetch(p, b, hk, tv.sk, 0, n_iter, block_key);
    q8_stage_q<T, DP, M, NW>(p, tv, rows, smem + C::OFF_Q, C::QP, hk, warp, lane);
    named_barrier_sync(1, NW * 32);

    const int gq = lane >> 2, tq = lane & 3;
    const int mi = lane >> 3, rr = lane & 7;
    const int r0 = rg * 16 + gq, r1 = r0 + 8;  // this warp's rows in Q.K^T
    const int key0 = slice * NB * 8;
    const int lo0 = rows.lo[r0], hi0 = rows.hi[r0], lo1 = rows.lo[r1], hi1 = rows.hi[r1];
    const int dg0 = rows.dg[r0], dg1 = rows.dg[r1];
    const float ab0 = rows.ab[r0], ab1 = rows.ab[r1];
    const float c0 = rows.sc[r0], c1 = rows.sc[r1];
    const uint8_t* q0p = smem + C::OFF_Q + r0 * C::QP + tq * 8;
    const uint8_t* q1p = smem + C::OFF_Q + r1 * C::QP + tq * 8;
    int plain_lo = max(lo0, lo1), plain_hi = min(hi0, hi1);
    q8_plain_keys(p.alibi != nullptr, plain_lo, plain_hi);
    auto q_frag = [&](int ks, uint32_t (&a)[4]) {
        const uint2 x = *reinterpret_cast<const uint2*>(q0p + ks * 32), y = *reinterpret_cast<const uint2*>(q1p + ks * 32);
        a[0] = x.x;
        a[1] = y.x;
        a[2] = x.y;
        a[3] = y.y;
    };
    float o[MG][2 * UW][4];  // [row group][2 x unit + parity]: columns 16 (UW warp + unit) + 4 tq + ...
    float m[MG][2];     // references of rows 16 g + gq and + 8
#pragma unroll
    for (int g = 0; g < MG; ++g) {
        m[g][0] = m[g][1] = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2 * UW; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[g][n][e] = 0.f;
    }
    auto mine = [&](int q) { return MG == 2 && rg ? m[MG - 1][q] : m[0][q]; };  // of this warp's Q.K^T rows
    float l0 = 0.f, l1 = 0.f;  // sums of this warp's rows over its keys
    bool ok = true;

    for (int it = 0; it < n_iter; ++it) {
        const int kst = it % C::KST, vst = it % C::VST;
        const int kt = kbeg + it * NT;
        if (ok) ok = __all_sync(0xffffffffu, q8_wait(&k_full[kst], (it / C::KST) & 1, abort_flag, p.err, p.wait_ns));
        const uint32_t k_base = smem_addr(smem + kst * C::TILE), v_base = smem_addr(smem + C::OFF_V + vst * C::TILE);
        float s[2][NB][4];  // two chains of products each
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[ch][n][e] = 0.f;
        if (ok) {
            if constexpr (NB == 1) {
#pragma unroll
                for (int kp = 0; kp < DP / 64; ++kp) {
                    uint32_t bq[4];  // k-steps 4 kp .. 4 kp + 3 of the eight keys
                    ldsm_x4(k_base + q8_off<DP, NT>(key0 + rr, 4 * kp + mi), bq[0], bq[1], bq[2], bq[3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t a[4];
                        q_frag(4 * kp + j, a);
                        MmaOp<__half>::run(s[j & 1][0], a, e4m3x2_to_half2(bq[j]), e4m3x2_hi_to_half2(bq[j]));
                    }
                }
            } else {
#pragma unroll
                for (int kp = 0; kp < DP / 32; ++kp) {
                    uint32_t bq[4];
                    ldsm_x4(k_base + q8_off<DP, NT>(key0 + rr + ((mi >> 1) << 3), 2 * kp + (mi & 1)), bq[0], bq[1], bq[2],
                            bq[3]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t a[4];
                        q_frag(2 * kp + j, a);
                        MmaOp<__half>::run(s[j][0], a, e4m3x2_to_half2(bq[j]), e4m3x2_hi_to_half2(bq[j]));
                        MmaOp<__half>::run(s[j][NB - 1], a, e4m3x2_to_half2(bq[2 + j]), e4m3x2_hi_to_half2(bq[2 + j]));
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_empty[kst]);
        float kss, lv;
        scales.take(p, b, hk, tv.sk, it, n_iter, block_key, kss, lv);
        const float inv = fast_exp2(-lv);
        const float k0 = c0 * kss, k1 = c1 * kss;
        const bool plain = MG == 1 && kt + key0 >= plain_lo && kt + key0 + NB * 8 - 1 <= plain_hi;  // (two groups: spills)
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = kt + key0 + n * 8 + tq * 2 + (e & 1);
                float& x = s[0][n][e];
                x += s[1][n][e];
                if (plain)
                    x = fmaf(x, e < 2 ? k0 : k1, lv);
                else if (e < 2)
                    x = q8_score(x, k0, lv, key >= lo0 && key <= hi0, ab0, dg0, key);
                else
                    x = q8_score(x, k1, lv, key >= lo1 && key <= hi1, ab1, dg1, key);
                if (e < 2)
                    mx0 = fmaxf(mx0, x);
                else
                    mx1 = fmaxf(mx1, x);
            }
        uint8_t* ps = smem + C::OFF_P + (it & 1) * (M * 128);
        float sum0, sum1;
        auto weights = [&]() {
            const float ma = mine(0), mb = mine(1);
            const float u0 = ma == -INFINITY ? 0.f : ma - kQ8Offset, u1 = mb == -INFINITY ? 0.f : mb - kQ8Offset;
            sum0 = sum1 = 0.f;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const float w0 = fast_exp2(s[0][n][0] - u0), w1 = fast_exp2(s[0][n][1] - u0);
                const float w2 = fast_exp2(s[0][n][2] - u1), w3 = fast_exp2(s[0][n][3] - u1);
                sum0 += w0 + w1;
                sum1 += w2 + w3;
                const int col = key0 + n * 8;  // a 16-byte unit of eight keys
                *reinterpret_cast<uint32_t*>(ps + swz128(r0, col >> 3) + tq * 4) = pack2<__half>(w0, w1);
                *reinterpret_cast<uint32_t*>(ps + swz128(r1, col >> 3) + tq * 4) = pack2<__half>(w2, w3);
            }
        };
        weights();
        const bool grow = mx0 > mine(0) + 5.f || mx1 > mine(1) + 5.f;
        if (named_barrier_or(1, NW * 32, grow || !ok)) {  // also publishes the weights
            if (named_barrier_or(2, NW * 32, !ok)) {
                ok = false;
                break;
            }
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
            if (tq == 0) {
                xmax[slice * M + r0] = mx0;
                xmax[slice * M + r1] = mx1;
            }
            named_barrier_sync(1, NW * 32);
#pragma unroll
            for (int g = 0; g < MG; ++g) {
                float f[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float nm = m[g][q];
#pragma unroll
                    for (int k = 0; k < C::KS; ++k) nm = fmaxf(nm, xmax[k * M + g * 16 + gq + 8 * q]);
                    f[q] = nm == -INFINITY ? 1.f : fast_exp2(m[g][q] - nm);
                    m[g][q] = nm;
                }
#pragma unroll
                for (int n = 0; n < 2 * UW; ++n) {
                    o[g][n][0] *= f[0];
                    o[g][n][1] *= f[0];
                    o[g][n][2] *= f[1];
                    o[g][n][3] *= f[1];
                }
                if (g == rg) {
                    l0 *= f[0];
                    l1 *= f[1];
                }
            }
            weights();
            named_barrier_sync(1, NW * 32);
        }
        l0 = fmaf(sum0, inv, l0);
        l1 = fmaf(sum1, inv, l1);
        if (ok) ok = __all_sync(0xffffffffu, q8_wait(&v_full[vst], (it / C::VST) & 1, abort_flag, p.err, p.wait_ns));
        // V rows that no row attends -> 0, each warp the columns it reads
        const int z_lo = max(tv.lo - kt, 0), z_hi = min(tv.hi + 1 - kt, NT);
        const bool zeroed = z_lo > 0 || z_hi < NT;
        if (zeroed) {
            uint8_t* vp = smem + C::OFF_V + vst * C::TILE;
            for (int idx = lane; idx < NT * UW; idx += 32) {
                const int r = idx / UW;
                if (r < z_lo || r >= z_hi)
                    *reinterpret_cast<uint4*>(vp + q8_off<DP, NT>(r, warp * UW + idx % UW)) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
        }
        if (ok) {
            const uint32_t p_base = smem_addr(ps);
#pragma unroll
            for (int ks = 0; ks < NT / 16; ++ks) {
                uint32_t a[MG][4];
#pragma unroll
                for (int g = 0; g < MG; ++g)
                    ldsm_x4(p_base + swz128(g * 16 + rr + ((mi & 1) << 3), 2 * ks + (mi >> 1)), a[g][0], a[g][1], a[g][2],
                            a[g][3]);
#pragma unroll
                for (int np = 0; np < UW / 2; ++np) {
                    uint32_t v[4];
                    ldsm_x4_t(v_base + q8_off<DP, NT>(ks * 16 + rr + ((mi & 1) << 3), warp * UW + 2 * np + (mi >> 1)), v[0],
                              v[1], v[2], v[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = __byte_perm(v[e], 0, 0x3120);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t e0 = e4m3x2_to_half2(v[2 * j]), e1 = e4m3x2_to_half2(v[2 * j + 1]);
                        const uint32_t d0 = e4m3x2_hi_to_half2(v[2 * j]), d1 = e4m3x2_hi_to_half2(v[2 * j + 1]);
#pragma unroll
                        for (int g = 0; g < MG; ++g) {
                            MmaOp<__half>::run(o[g][2 * (2 * np + j)], a[g], e0, e1);
                            MmaOp<__half>::run(o[g][2 * (2 * np + j) + 1], a[g], d0, d1);
                        }
                    }
                }
            }
        }
        if (zeroed) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_empty[vst]);
    }
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (named_barrier_or(1, NW * 32, !ok || *abort_flag != 0u)) return;
    if (tq == 0) {
        xmax[slice * M + r0] = l0;
        xmax[slice * M + r1] = l1;
    }
    named_barrier_sync(1, NW * 32);
    T* out = static_cast<T*>(p.out);
#pragma unroll
    for (int g = 0; g < MG; ++g)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int row = g * 16 + gq + 8 * q;
            if (row >= tv.rows) continue;
            float L = 0.f;
#pragma unroll
            for (int k = 0; k < C::KS; ++k) L += xmax[k * M + row];
            const float iv = L == 0.f ? 0.f : 1.f / L;
            const int rho = tv.row0 + row;
            const int i = rho / p.G, gg = rho - i * p.G;
            const int64_t t = tv.q0 + i;
            const int h = hk * p.G + gg;
#pragma unroll
            for (int u = 0; u < UW; ++u) {
                const int d = (warp * UW + u) * 16 + tq * 4;
                if (d >= p.D) continue;
                const float x0 = o[g][2 * u][2 * q] * iv, x1 = o[g][2 * u + 1][2 * q] * iv;
                const float x2 = o[g][2 * u][2 * q + 1] * iv, x3 = o[g][2 * u + 1][2 * q + 1] * iv;
                if (single)
                    *reinterpret_cast<uint2*>(out + t * p.o_s0 + (int64_t)h * p.o_s1 + d) =
                        make_uint2(pack2<T>(x0, x1), pack2<T>(x2, x3));
                else
                    *reinterpret_cast<float4*>(p.part_o + ((int64_t)split * p.part_stride + t * p.H + h) * p.D + d) =
                        make_float4(x0, x1, x2, x3);
            }
            if (warp == 0 && tq == 0) {
                const float lse = L == 0.f ? -INFINITY : (m[g][q] - kQ8Offset + log2f(L)) * 0.69314718055994531f;
                if (single)
                    p.lse[(int64_t)h * p.lse_s0 + t + (int64_t)b * p.lse_sb] = lse;
                else
                    p.part_lse[(int64_t)split * p.part_stride + t * p.H + h] = lse;
            }
        }
}

}  // namespace pa
