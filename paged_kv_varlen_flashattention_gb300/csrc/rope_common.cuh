// The rotation of 16 elements of a head by their token's position, shared by the appends
// into 16-bit and 8-bit caches.
//
// With rot rotated columns and the table rows c = cos[pos], s = sin[pos] of rot / 2 entries,
// pair i of a head becomes (a, b) -> (a c_i - b s_i, b c_i + a s_i), where (a, b) are columns
// (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved; columns at or past rot stay.  A head
// is cut into units of 16 columns that hold whole pairs:
//   u < rot / 16, halves       columns [8 u, 8 u + 8) and [rot / 2 + 8 u, rot / 2 + 8 u + 8)
//   u < rot / 16, interleaved  columns [16 u, 16 u + 16)
//   u >= rot / 16              columns [16 u, 16 u + 16), not rotated (8 of them in the last
//                              unit of a head_dim that is no multiple of 16)
// so both rotated forms read entries [8 u, 8 u + 8) of the table rows, and a unit is two
// 16-byte loads.  The products and the difference are rounded one by one in fp32 (no fused
// multiply-add): the values an elementwise implementation in fp32 gets.
#pragma once

#include "device_common.cuh"

namespace pa {

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Column offsets of the two 8-column halves of unit u.
__device__ __forceinline__ void unit_columns(int u, int rot, bool interleaved, int& o0, int& o1) {
    const bool split = u < (rot >> 4) && !interleaved;
    o0 = split ? 8 * u : 16 * u;
    o1 = split ? (rot >> 1) + 8 * u : 16 * u + 8;
}

// Entries [8 u, 8 u + 8) of a table row.
__device__ __forceinline__ void load_row8(const float* row, int u, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(row + 8 * u));
    const float4 b = __ldg(reinterpret_cast<const float4*>(row + 8 * u + 4));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

template <typename T>
__device__ __forceinline__ void unpack16(const uint4& lo, const uint4& hi, float (&x)[16]) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 v = unpack2<T>(w[i]);
        x[2 * i] = v.x;
        x[2 * i + 1] = v.y;
    }
}

template <typename T>
__device__ __forceinline__ void pack16(const float (&x)[16], uint4& lo, uint4& hi) {
    lo = make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
    hi = make_uint4(pack2<T>(x[8], x[9]), pack2<T>(x[10], x[11]), pack2<T>(x[12], x[13]), pack2<T>(x[14], x[15]));
}

template <bool INTERLEAVED>
__device__ __forceinline__ void rotate16(float (&x)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float& a = INTERLEAVED ? x[2 * i] : x[i];
        float& b = INTERLEAVED ? x[2 * i + 1] : x[8 + i];
        const float na = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
        const float nb = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
        a = na;
        b = nb;
    }
}

// The last sequence b < batch with key(b) <= x, by a 32-way search over the warp (one probe
// per lane and round): key is non-decreasing with key(0) <= x.
template <typename Key>
__device__ __forceinline__ int warp_search(int batch, int64_t x, int lane, Key key) {
    int lo = 0, span = batch;
    while (span > 1) {
        const int step = (span + 31) / 32;
        const int idx = lo + lane * step;
        const bool le = idx < lo + span && key(idx) <= x;
        const unsigned ok = __ballot_sync(0xffffffffu, le);
        const int last = ok ? 31 - __clz((int)ok) : 0;
        lo += last * step;
        span = min(step, span - last * step);
    }
    return lo;
}

// Where a new token goes: its sequence's position and physical page.  `live` is false for a
// token behind the last sequence (left alone); bad metadata is flagged by lane 0.
struct TokenPlace {
    bool live;    // the token belongs to a sequence and its position is in range
    int64_t pos;  // logical key of its sequence
    int blk;      // physical block, -1: not written
    int slot;
};

__device__ __forceinline__ TokenPlace place_token(const RopeArgs& a, int64_t t, int lane, unsigned int* err) {
    const AppendArgs& k = a.kv;
    TokenPlace p{false, 0, -1, 0};
    const int b = warp_search(k.batch, t, lane, [&](int i) { return (int64_t)__ldg(k.cu_new + i); });
    const int64_t n0 = k.cu_new[b], n1 = k.cu_new[b + 1];
    const int64_t sk = (int64_t)k.cu_k[b + 1] - k.cu_k[b];
    if (t >= n1 && b + 1 == k.batch) return p;  // behind the last sequence
    const int64_t pos = sk - (n1 - t);
    if (t < n0 || t >= n1 || n1 - n0 > sk || pos < 0 || (a.rot > 0 && pos >= a.max_pos)) {
        if (lane == 0) flag_error(err, PA_ERR_DEVICE_BOUNDS);
        return p;
    }
    p.live = true;
    p.pos = pos;
    const int64_t page = pos / k.P;
    int blk = -1;
    if (page < k.bt_cols) blk = k.bt[(int64_t)b * k.bt_s0 + page];
    if (blk < 0 || blk >= k.num_blocks) {
        if (lane == 0) flag_error(err, PA_ERR_DEVICE_BOUNDS);
        blk = -1;
    }
    p.blk = blk;
    p.slot = (int)(pos - page * k.P);
    return p;
}

}  // namespace pa
