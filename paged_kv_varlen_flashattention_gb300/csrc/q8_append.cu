// KV append into an 8-bit cache (pa_kv_append_q8): the step's k (rotated by its tokens'
// positions when tables are given) and v are held as e4m3 codes with one scale for each page
// and kv head, and the step's q is rotated beside them.
//
// One CTA owns one (page, kv head) that receives new tokens, so a page's scale has one writer:
// it takes the absolute maxima of the page's new keys and values over the CTA, picks each scale
//   s = 2^k, the least with max |x| <= 448 s           (a page that starts with a new token)
//   s = max(the page's scale, that)                    (a page with earlier tokens)
// holds the earlier tokens again when the scale grew (by a power of two: only codes that fall
// below the normal range of e4m3 are rounded a second time) and writes the new codes.  A power
// of two costs a floating-point format no precision, and makes the scale, and with it the whole
// page, the same however the tokens were cut into calls (but for that second rounding).
//
// A byte mover: 2 bytes read and 1 written per element of k and v, 2 and 2 of q.  The new tokens are
// read once, into registers as they came (two 16-column units of K and of V a thread; the rotation and
// the conversion to fp32 are done again for the codes, which costs less than the registers would), where
// 128, 256 or 512 threads can hold them: up to 128 tokens of 128 columns; a larger page is read twice,
// the second time from L1/L2.  q takes warps of its own, a token's heads each, and their CTAs stand
// evenly among the pages': a page is a chain of dependent steps, q a stream that fills its waits.
// Eight prompts of 1,024 to 8,192 tokens (32 / 8 heads of 128, 64-token pages): 162 us, 79 % of the
// copy rate; with fp32 units held and the pages' CTAs first 182, with q cut into four passes a warp 166,
// with two 193.
#include <algorithm>
#include <cfloat>
#include <cstdio>

#include "q8_common.cuh"
#include "rope_common.cuh"

namespace pa {
namespace {

constexpr int kQ8Resident = 768;  // threads an SM holds at this kernel's registers (80)
constexpr int kQ8Held = 2;   // units of K and of V a thread keeps in registers
constexpr int kQ8QPasses = 4;  // passes of q heads whose loads are in flight together

// 8 values as e4m3 codes under 1 / scale (exact: a power of two, or the caller's own scale); a
// value that is not finite becomes NaN.
__device__ __forceinline__ uint2 codes8(const float* x, float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        w[i] = e4m3x2(fabsf(a) <= FLT_MAX ? a * inv : NAN, fabsf(b) <= FLT_MAX ? b * inv : NAN);
    }
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ float finite_absmax16(const float (&x)[16]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float v = fabsf(x[i]);
        m = fmaxf(m, v <= FLT_MAX ? v : 0.f);
    }
    return m;
}

// Earlier tokens of a page (slots 0 .. kept - 1 of one head) held again under a larger scale.
template <int NT>
__device__ __forceinline__ void rescale_slots(uint8_t* row0, int64_t slot_stride, int kept, int D, float ratio) {
    const int units = D / 16;
    for (int i = threadIdx.x; i < kept * units; i += NT) {
        uint4* p = reinterpret_cast<uint4*>(row0 + (int64_t)(i / units) * slot_stride + (i % units) * 16);
        uint4 v = *p;
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t l = e4m3x2_to_half2(w[j]), h = e4m3x2_hi_to_half2(w[j]);
            const float2 a = unpack2<__half>(l), b = unpack2<__half>(h);
            w[j] = e4m3x2(a.x * ratio, a.y * ratio) | (e4m3x2(b.x * ratio, b.y * ratio) << 16);
        }
        *p = v;
    }
}

template <typename T, bool INTERLEAVED, int NT>
__global__ void __launch_bounds__(NT, kQ8Resident / NT)
    q8_append_kernel(const RopeArgs a, int64_t page_ctas, int passes, int per_item, int items_per_token, int64_t q_items,
                     unsigned int* err) {
    const AppendArgs& k = a.kv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int units = k.D / 16;
    // page CTAs stand evenly among those of q: their chains of dependent loads run beside its stream
    const int64_t before = (int64_t)blockIdx.x * page_ctas / gridDim.x;
    if ((int64_t)(blockIdx.x + 1) * page_ctas / gridDim.x == before) {
        // ---- q: one (token, few heads) item a warp ----
        const int64_t item = ((int64_t)blockIdx.x - before) * (NT / 32) + warp;
        if (item >= q_items) return;
        const int64_t t = item / items_per_token;
        const int pass0 = (int)(item - t * items_per_token) * per_item, pass1 = min(passes, pass0 + per_item);
        const int heads_per_pass = 32 / units;
        const int u = lane % units, sub = lane / units;
        int o0, o1;
        unit_columns(u, a.rot, INTERLEAVED, o0, o1);
        uint4 x0[kQ8QPasses], x1[kQ8QPasses];
        auto load = [&](int pass) {
#pragma unroll
            for (int i = 0; i < kQ8QPasses; ++i) {
                const int h = (pass + i) * heads_per_pass + sub;
                if (pass + i < pass1 && sub < heads_per_pass && h < a.H) {
                    const T* src = static_cast<const T*>(a.q) + t * a.q_s0 + (int64_t)h * a.q_s1;
                    x0[i] = __ldcs(reinterpret_cast<const uint4*>(src + o0));
                    x1[i] = __ldcs(reinterpret_cast<const uint4*>(src + o1));
                }
            }
        };
        load(pass0);
        // the token's position alone (its page is the page CTAs' concern)
        const int b = warp_search(k.batch, t, lane, [&](int i) { return (int64_t)__ldg(k.cu_new + i); });
        const int64_t n0 = k.cu_new[b], n1 = k.cu_new[b + 1], sk = (int64_t)k.cu_k[b + 1] - k.cu_k[b];
        const int64_t pos = sk - (n1 - t);
        if (t < n0 || t >= n1 || n1 - n0 > sk || pos < 0 || pos >= a.max_pos) {
            if (!(t >= n1 && b + 1 == k.batch) && lane == 0) flag_error(err, PA_ERR_DEVICE_BOUNDS);
            return;
        }
        const bool rotated = u < (a.rot >> 4);
        float c[8], s[8];
        if (rotated) {
            load_row8(a.cos + pos * a.cos_s0, u, c);
            load_row8(a.sin + pos * a.sin_s0, u, s);
        }
        for (int pass = pass0; pass < pass1; pass += kQ8QPasses) {
            if (pass > pass0) load(pass);
#pragma unroll
            for (int i = 0; i < kQ8QPasses; ++i) {
                const int h = (pass + i) * heads_per_pass + sub;
                if (!(pass + i < pass1 && sub < heads_per_pass && h < a.H)) continue;
                if (rotated) {
                    float x[16];
                    unpack16<T>(x0[i], x1[i], x);
                    rotate16<INTERLEAVED>(x, c, s);
                    pack16<T>(x, x0[i], x1[i]);
                }
                T* dst = static_cast<T*>(a.q_out) + t * a.qo_s0 + (int64_t)h * a.qo_s1;
                *reinterpret_cast<uint4*>(dst + o0) = x0[i];
                *reinterpret_cast<uint4*>(dst + o1) = x1[i];
            }
        }
        return;
    }
    // ---- k and v: one (page, kv head) ----
    // Sequence b owns the indices [cu_new[b] / P + 2 b, that of b + 1): at least as many as the
    // pages its n_b new tokens can touch (n_b / P + 2), so no prefix sum over pages is needed.
    const int64_t index = before / k.Hkv;
    const int hk = (int)(before - index * k.Hkv);
    auto first_index = [&](int i) { return (int64_t)__ldg(k.cu_new + i) / k.P + 2 * (int64_t)i; };
    const int b = warp_search(k.batch, index, lane, first_index);
    const int64_t n0 = k.cu_new[b], n1 = k.cu_new[b + 1];
    const int64_t sk = (int64_t)k.cu_k[b + 1] - k.cu_k[b];
    if (n0 == n1) return;
    if (n0 < 0 || n1 < n0 || n1 > k.total_new || n1 - n0 > sk) {
        if (tid == 0) flag_error(err, PA_ERR_DEVICE_BOUNDS);
        return;
    }
    const int64_t pos0 = sk - (n1 - n0);
    const int64_t page = pos0 / k.P + (index - first_index(b));
    if (page > (sk - 1) / k.P) return;
    int blk = -1;
    if (page < k.bt_cols) blk = k.bt[(int64_t)b * k.bt_s0 + page];
    const int s_lo = (int)max64(0, pos0 - page * k.P), s_hi = (int)min64(k.P, sk - page * k.P);
    if (blk < 0 || blk >= k.num_blocks || (a.rot > 0 && page * k.P + s_hi > a.max_pos)) {
        if (tid == 0) flag_error(err, PA_ERR_DEVICE_BOUNDS);
        return;
    }
    const int64_t t0 = n0 + page * k.P - pos0;  // the token at slot 0 of the page, were it new
    float* ks = a.k_scale + (int64_t)blk * a.ks_s0 + (int64_t)hk * a.ks_s1;
    float* vs = a.v_scale + (int64_t)blk * a.vs_s0 + (int64_t)hk * a.vs_s1;
    const float old_k = s_lo > 0 ? *ks : 0.f, old_v = s_lo > 0 ? *vs : 0.f;
    uint8_t* kc = static_cast<uint8_t*>(k.k_cache) + (int64_t)blk * k.c_s0 + (int64_t)hk * k.c_s2;
    uint8_t* vc = static_cast<uint8_t*>(k.v_cache) + (int64_t)blk * k.c_s0 + (int64_t)hk * k.c_s2;

    // unit i of the page's new tokens: 16 columns of K (rotated) and of V
    const int n_units = (s_hi - s_lo) * units;
    auto fetch = [&](int i, uint4 (&w)[4]) {
        const int slot = s_lo + i / units, u = i % units;
        const T* sk_ = static_cast<const T*>(k.k_new) + (t0 + slot) * k.kn_s0 + (int64_t)hk * k.kn_s1;
        const T* sv_ = static_cast<const T*>(k.v_new) + (t0 + slot) * k.vn_s0 + (int64_t)hk * k.vn_s1;
        int o0, o1;
        unit_columns(u, a.rot, INTERLEAVED, o0, o1);
        w[0] = __ldg(reinterpret_cast<const uint4*>(sk_ + o0));
        w[1] = __ldg(reinterpret_cast<const uint4*>(sk_ + o1));
        w[2] = __ldg(reinterpret_cast<const uint4*>(sv_ + 16 * u));
        w[3] = __ldg(reinterpret_cast<const uint4*>(sv_ + 16 * u + 8));
    };
    auto keys_of = [&](int i, const uint4 (&w)[4], float (&x)[16]) {
        const int u = i % units;
        unpack16<T>(w[0], w[1], x);
        if (u < (a.rot >> 4)) {
            float c[8], s[8];
            const int64_t pos = page * k.P + s_lo + i / units;
            load_row8(a.cos + pos * a.cos_s0, u, c);
            load_row8(a.sin + pos * a.sin_s0, u, s);
            rotate16<INTERLEAVED>(x, c, s);
        }
    };
    float mk = 0.f, mv = 0.f;
    auto measure = [&](int i, const uint4 (&w)[4]) {
        float x[16];
        keys_of(i, w, x);
        mk = fmaxf(mk, finite_absmax16(x));
        unpack16<T>(w[2], w[3], x);
        mv = fmaxf(mv, finite_absmax16(x));
    };
    const bool held = n_units <= NT * kQ8Held;
    uint4 w[kQ8Held][4];
    if (held) {
#pragma unroll
        for (int r = 0; r < kQ8Held; ++r)
            if (tid + r * NT < n_units) fetch(tid + r * NT, w[r]);
#pragma unroll
        for (int r = 0; r < kQ8Held; ++r)
            if (tid + r * NT < n_units) measure(tid + r * NT, w[r]);
    } else {
        for (int i = tid; i < n_units; i += NT) {
            fetch(i, w[0]);
            measure(i, w[0]);
        }
    }
    __shared__ float red[2][NT / 32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, off));
        mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, off));
    }
    if (lane == 0) {
        red[0][warp] = mk;
        red[1][warp] = mv;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        mk = fmaxf(mk, red[0][w]);
        mv = fmaxf(mv, red[1][w]);
    }
    const float new_k = fmaxf(old_k, pow2_scale(mk)), new_v = fmaxf(old_v, pow2_scale(mv));
    if (s_lo > 0) {
        if (new_k > old_k) rescale_slots<NT>(kc, k.c_s1, s_lo, k.D, old_k / new_k);
        if (new_v > old_v) rescale_slots<NT>(vc, k.c_s1, s_lo, k.D, old_v / new_v);
    }
    if (tid == 0) {
        *ks = new_k;
        *vs = new_v;
    }
    const float ik = 1.f / new_k, iv = 1.f / new_v;
    auto put = [&](int i, const uint4 (&w)[4]) {
        const int slot = s_lo + i / units, u = i % units;
        int o0, o1;
        unit_columns(u, a.rot, INTERLEAVED, o0, o1);
        float x[16];
        keys_of(i, w, x);
        uint8_t* kr = kc + (int64_t)slot * k.c_s1;
        *reinterpret_cast<uint2*>(kr + o0) = codes8(&x[0], ik);
        *reinterpret_cast<uint2*>(kr + o1) = codes8(&x[8], ik);
        unpack16<T>(w[2], w[3], x);
        const uint2 v0 = codes8(&x[0], iv), v1 = codes8(&x[8], iv);
        *reinterpret_cast<uint4*>(vc + (int64_t)slot * k.c_s1 + 16 * u) = make_uint4(v0.x, v0.y, v1.x, v1.y);
    };
    if (held) {
#pragma unroll
        for (int r = 0; r < kQ8Held; ++r)
            if (tid + r * NT < n_units) put(tid + r * NT, w[r]);
    } else {
        for (int i = tid; i < n_units; i += NT) {
            fetch(i, w[0]);
            put(i, w[0]);
        }
    }
}

using Q8AppendKernel = void (*)(const RopeArgs, int64_t, int, int, int, int64_t, unsigned int*);

template <typename T>
Q8AppendKernel q8_append_kernel_of(bool interleaved, int nt) {
    if (nt == 128) return interleaved ? q8_append_kernel<T, true, 128> : q8_append_kernel<T, false, 128>;
    if (nt == 256) return interleaved ? q8_append_kernel<T, true, 256> : q8_append_kernel<T, false, 256>;
    return interleaved ? q8_append_kernel<T, true, 512> : q8_append_kernel<T, false, 512>;
}

}  // namespace

int launch_q8_append(const RopeArgs& a, unsigned int* err, char* msg, size_t msg_len) {
    const AppendArgs& k = a.kv;
    if (k.total_new == 0 || k.batch == 0) return PA_OK;
    const int64_t page_ctas = (k.total_new / k.P + 2 * (int64_t)k.batch) * k.Hkv;
    const int units = k.D / 16, heads_per_pass = 32 / units;
    const int passes = a.q ? (a.H + heads_per_pass - 1) / heads_per_pass : 0;
    // a warp takes a token's q heads whole once the tokens alone give some 16 warps an SM
    const int per_item = k.total_new >= 2432 ? passes : std::min(passes, kQ8QPasses);
    const int items_per_token = a.q ? (passes + per_item - 1) / per_item : 0;
    const int64_t q_items = k.total_new * items_per_token;
    // as many threads as hold a page's new tokens in registers, where that many can be had
    const int64_t most = std::min<int64_t>(k.P, k.total_new) * units;
    const int nt = most <= 128 * kQ8Held ? 128 : most <= 256 * kQ8Held ? 256 : 512;
    const int64_t grid = page_ctas + (q_items + nt / 32 - 1) / (nt / 32);
    if (grid > 0x7fffffff) {
        snprintf(msg, msg_len, "q8 append: %lld CTAs exceed one launch", (long long)grid);
        return PA_ERR_UNSUPPORTED;
    }
    NvtxRange nv("pa::q8_append_kernel");
    timer_begin(PA_KC_APPEND, k.stream);
    auto kern = a.dtype == PA_BF16 ? q8_append_kernel_of<__nv_bfloat16>(a.interleaved, nt)
                                   : q8_append_kernel_of<__half>(a.interleaved, nt);
    kern<<<(unsigned)grid, nt, 0, k.stream>>>(a, page_ctas, passes, per_item, items_per_token, q_items, err);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "q8 append launch: %s", cudaGetErrorString(e));
        return PA_ERR_CUDA;
    }
    timer_end(PA_KC_APPEND, k.stream);
    count_launches(1);
    return PA_OK;
}

}  // namespace pa
