// KV append with the position rotation on the way (pa_kv_append_rope): the step's q and k
// are rotated by their tokens' logical positions, k and v go to their pages, q to q_out.
//
// A byte mover: every input element is read once and every output written once (2 bytes each),
// and the rotation adds ~1.5 fp32 operations per element.  One warp takes one token (or, when
// the step has few tokens, a few heads of one), its heads in the order q, k, v.  A lane keeps
// one 16-column unit for every head of the token, so the eight cosines and sines it needs stay
// in registers; a pass of the warp covers 32 / (units per head) heads, and the loads of four
// passes are issued together, ahead of the chain of dependent lookups (sequence, position,
// block) that the stores wait for.
#include <algorithm>
#include <cstdio>

#include "rope_common.cuh"

namespace pa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopePasses = 4;  // passes whose loads are in flight together

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads)
    rope_append_kernel(const RopeArgs a, int passes, int per_item, int items_per_token, int64_t items,
                       unsigned int* err) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    if (item >= items) return;
    const int64_t t = item / items_per_token;
    const int pass0 = (int)(item - t * items_per_token) * per_item, pass1 = min(passes, pass0 + per_item);
    const AppendArgs& k = a.kv;
    const int units = (k.D + 15) / 16;
    const int heads_per_pass = 32 / units;
    const int u = lane % units, sub = lane / units;
    const int heads = a.H + 2 * k.Hkv;
    int o0, o1;
    unit_columns(u, a.rot, INTERLEAVED, o0, o1);
    const bool rotated = u < (a.rot >> 4), has1 = o1 < k.D;

    auto source = [&](int h) -> const T* {
        if (h < a.H) return static_cast<const T*>(a.q) + t * a.q_s0 + (int64_t)h * a.q_s1;
        h -= a.H;
        if (h < k.Hkv) return static_cast<const T*>(k.k_new) + t * k.kn_s0 + (int64_t)h * k.kn_s1;
        h -= k.Hkv;
        return static_cast<const T*>(k.v_new) + t * k.vn_s0 + (int64_t)h * k.vn_s1;
    };
    uint4 x0[kRopePasses], x1[kRopePasses];
    auto load = [&](int pass) {
#pragma unroll
        for (int i = 0; i < kRopePasses; ++i) {
            const int h = (pass + i) * heads_per_pass + sub;
            if (pass + i < pass1 && sub < heads_per_pass && h < heads) {
                const T* src = source(h);
                x0[i] = __ldcs(reinterpret_cast<const uint4*>(src + o0));
                if (has1) x1[i] = __ldcs(reinterpret_cast<const uint4*>(src + o1));
            }
        }
    };
    load(pass0);
    const TokenPlace p = place_token(a, t, lane, err);
    if (!p.live) return;
    float c[8], s[8];
    if (rotated) {
        load_row8(a.cos + p.pos * a.cos_s0, u, c);
        load_row8(a.sin + p.pos * a.sin_s0, u, s);
    }
    const int64_t cache_row = (int64_t)p.blk * k.c_s0 + (int64_t)p.slot * k.c_s1;
    for (int pass = pass0; pass < pass1; pass += kRopePasses) {
        if (pass > pass0) load(pass);
#pragma unroll
        for (int i = 0; i < kRopePasses; ++i) {
            int h = (pass + i) * heads_per_pass + sub;
            if (!(pass + i < pass1 && sub < heads_per_pass && h < heads)) continue;
            T* dst;
            if (h < a.H) {
                dst = static_cast<T*>(a.q_out) + t * a.qo_s0 + (int64_t)h * a.qo_s1;
            } else {
                if (p.blk < 0) continue;
                const bool is_k = h < a.H + k.Hkv;
                dst = static_cast<T*>(is_k ? k.k_cache : k.v_cache) + cache_row +
                      (int64_t)(is_k ? h - a.H : h - a.H - k.Hkv) * k.c_s2;
            }
            if (rotated && h < a.H + k.Hkv) {
                float x[16];
                unpack16<T>(x0[i], x1[i], x);
                rotate16<INTERLEAVED>(x, c, s);
                pack16<T>(x, x0[i], x1[i]);
            }
            *reinterpret_cast<uint4*>(dst + o0) = x0[i];
            if (has1) *reinterpret_cast<uint4*>(dst + o1) = x1[i];
        }
    }
}

}  // namespace

int launch_rope_append(const RopeArgs& a, unsigned int* err, char* msg, size_t msg_len) {
    const AppendArgs& k = a.kv;
    if (k.total_new == 0 || k.batch == 0) return PA_OK;
    const int units = (k.D + 15) / 16, heads_per_pass = 32 / units;
    const int passes = (a.H + 2 * k.Hkv + heads_per_pass - 1) / heads_per_pass;
    // A warp per token once that alone gives the GPU some 16 warps an SM; fewer tokens (a decode
    // step) are cut into items of one batch of passes, so that no warp waits on memory twice.
    const int per_item = k.total_new >= 2432 ? passes : std::min(passes, kRopePasses);
    const int items_per_token = (passes + per_item - 1) / per_item;
    const int64_t items = k.total_new * items_per_token;
    const int64_t grid = (items + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    if (grid > 0x7fffffff) {
        snprintf(msg, msg_len, "rope append: %lld items exceed one launch", (long long)items);
        return PA_ERR_UNSUPPORTED;
    }
    NvtxRange nv("pa::rope_append_kernel");
    timer_begin(PA_KC_APPEND, k.stream);
    const bool bf16 = a.dtype == PA_BF16;
    auto kern = bf16 ? (a.interleaved ? rope_append_kernel<__nv_bfloat16, true> : rope_append_kernel<__nv_bfloat16, false>)
                     : (a.interleaved ? rope_append_kernel<__half, true> : rope_append_kernel<__half, false>);
    kern<<<(unsigned)grid, kRopeThreads, 0, k.stream>>>(a, passes, per_item, items_per_token, items, err);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "rope append launch: %s", cudaGetErrorString(e));
        return PA_ERR_CUDA;
    }
    timer_end(PA_KC_APPEND, k.stream);
    count_launches(1);
    return PA_OK;
}

}  // namespace pa
