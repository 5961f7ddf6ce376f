// lora.hpp -- device helpers of the low-rank adapters: the rows of a batch by
// request, fp32 values as sums of bf16 ones, and the adapter term that the
// GEMM epilogues add.
//
// A batch of M rows holds S requests: request s owns the rows seg_start[s] ..
// seg_start[s+1]-1 and uses adapter seg_adapter[s] of a pool of n (negative
// or >= n: none).  Rows before seg_start[0] and from seg_start[S] on belong
// to no request.  The boundaries live in device memory and are never trusted:
// every one is clamped to 0 .. M, so ranges that are not ascending give
// unspecified values but no access out of bounds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"
#include "internal.hpp"

namespace dmpq {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int seg_clamp(int v, int M) { return v < 0 ? 0 : v > M ? M : v; }

__device__ __forceinline__ int seg_adapter_of(const LoraBatch &B, int s) {
    const int a = B.seg_adapter[s];
    return a >= 0 && a < B.nA ? a : -1;
}

// A tile of at most TM rows of one request (or of the rows before the first
// and after the last one, adapter -1).
struct SegTile {
    int row0, rows, adapter;
};

// Tile `idx` of the batch cut into tiles of TM rows request by request; false
// if there are fewer.  Called by whole waves with a wave-uniform idx; the
// S + 2 row ranges are counted 64 at a time by a prefix sum over the lanes.
__device__ __forceinline__ bool seg_tile(const LoraBatch &B, int idx, int TM, SegTile &out) {
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int c = 0; c < B.S + 2; c += 64) {
        const int p = c + lane;  // 0: rows before the first request; s + 1: request s; S + 1: the rest
        const int before = p == 0 ? 0 : p - 1 < B.S ? p - 1 : B.S;
        const int v0 = B.seg_start[before], v1 = B.seg_start[p < B.S ? p : B.S];
        const int ad = B.S > 0 ? B.seg_adapter[before < B.S ? before : B.S - 1] : -1;
        const int lo = p == 0 ? 0 : seg_clamp(v0, B.M);
        const int hi = p > B.S + 1 ? 0 : p == B.S + 1 ? B.M : seg_clamp(v1, B.M);
        const int n = hi > lo ? (hi - lo + TM - 1) / TM : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(inc, o, 64);
            if (lane >= o) inc += v;
        }
        const int total = __builtin_amdgcn_readlane(inc, 63);
        if (idx < base + total) {
            const int src = __builtin_ctzll(__ballot(idx < base + inc));
            const int k = idx - base - (__builtin_amdgcn_readlane(inc, src) - __builtin_amdgcn_readlane(n, src));
            const int l = __builtin_amdgcn_readlane(lo, src), h = __builtin_amdgcn_readlane(hi, src);
            out.row0 = l + k * TM;
            out.rows = h - out.row0 < TM ? h - out.row0 : TM;
            const int q = c + src, a = __builtin_amdgcn_readlane(ad, src);
            out.adapter = q >= 1 && q <= B.S && a >= 0 && a < B.nA ? a : -1;
            return true;
        }
        base += total;
    }
    return false;
}

// The request of a row by bisection (the last s with seg_start[s] <= row),
// or -1; its adapter through seg_adapter_of.
__device__ __forceinline__ int row_adapter(const LoraBatch &B, int row) {
    int lo = 0, hi = B.S + 1;  // seg_start[lo - 1] <= row < seg_start[hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (B.seg_start[mid] <= row)
            lo = mid + 1;
        else
            hi = mid;
    }
    const int s = lo - 1;
    return s >= 0 && s < B.S ? seg_adapter_of(B, s) : -1;
}

__device__ __forceinline__ int adapter_rank(const LoraBatch &B, int a) {
    const int r = B.rank[a];
    return r < 0 ? 0 : r > B.R ? B.R : r;
}

// ---- fp32 as a sum of bf16 values -------------------------------------------
// The bf16 MFMA multiplies an fp32 operand as NS bf16 parts, each the nearest
// to what the parts before it leave: 2 parts keep 16 bits and more of it
// (error at most 2^-18 of the value), 3 parts all 24.  bf16 has fp32's
// exponents, so nothing overflows but values within half a bf16 step of
// FLT_MAX; an infinite or NaN value is its own first part, the others 0.
template <int NS>
__device__ __forceinline__ void split8(const float v[8], v4i (&out)[NS]) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; i++) r[i] = v[i];
#pragma unroll
    for (int p = 0; p < NS; p++) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t w = cvt_pk_bf16(r[2 * i], r[2 * i + 1]);
            out[p][i] = (int)w;
            if (p + 1 < NS) {
                const float lo = bf16_lo(w), hi = bf16_hi(w);
                r[2 * i] = __builtin_isfinite(lo) ? r[2 * i] - lo : 0.0f;
                r[2 * i + 1] = __builtin_isfinite(hi) ? r[2 * i + 1] - hi : 0.0f;
            }
        }
    }
}

// The first n of 8 bf16 values, zeros in place of the others.
__device__ __forceinline__ v4i keep8(v4i v, int n) {
#pragma unroll
    for (int d = 0; d < 4; d++) {
        const uint32_t m = (2 * d < n ? 0xFFFFu : 0u) | (2 * d + 1 < n ? 0xFFFF0000u : 0u);
        v[d] &= (int)m;
    }
    return v;
}

__device__ __forceinline__ v16f mfma32(const v4i &a, const v4i &b, const v16f &c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

__device__ __forceinline__ v4f mfma16(const v4i &a, const v4i &b, const v4f &c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// ---- the adapter term of a GEMM's epilogue -----------------------------------
// v += scale * t b^T for 32 rows x 128 columns in the GEMMs' accumulator
// layout: lane l holds row l % 32 (`row`; past M: nothing is added) and, in
// v[j][4g + e], column n0 + 32 j + 8 g + 4 (l / 32) + e.  b's rows are the
// MFMA's first operand, scale * t in NS bf16 parts (split8) the second.  Where
// all rows share an adapter the products accumulate straight onto v.  Rows of
// several adapters take one product per adapter over all 32 rows, added where
// it belongs and never multiplied by zero elsewhere: one adapter's infinity
// must not reach another request's rows.
template <int NS>
__device__ __forceinline__ void lora_t_frag(const float *tr, float sc, v4i (&tf)[NS]) {
    const v4f a0 = *reinterpret_cast<const v4f *>(tr), a1 = *reinterpret_cast<const v4f *>(tr + 4);
    const float v[8] = {sc * a0[0], sc * a0[1], sc * a0[2], sc * a0[3], sc * a1[0], sc * a1[1], sc * a1[2], sc * a1[3]};
    split8<NS>(v, tf);
}

template <int NS>
__device__ __forceinline__ void lora_slice(const LoraEpi &L, int64_t row, int64_t n0, int64_t N, int lane,
                                           v16f (&v)[4]) {
    const LoraBatch &B = L.batch;
    const int lm = lane & 31, lh = lane >> 5;
    const int mine = row < B.M ? row_adapter(B, (int)row) : -1;
    const float *tr = L.t + (row < B.M ? row : B.M - 1) * B.R + 8 * lh;
    const uint16_t *bl[4];  // the lane's row of b, of adapter 0
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int64_t n = n0 + 32 * j + lm;
        bl[j] = L.b + (n < N ? n : N - 1) * B.R + 8 * lh;
    }
    uint64_t todo = __ballot(mine >= 0);
    const uint64_t in_m = __ballot(row < B.M);
    while (todo) {
        const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
        const uint64_t own = __ballot(mine == a);
        todo &= ~own;
        const int rank = adapter_rank(B, a);
        const float sc = B.scale[a];
        const int64_t off = (int64_t)a * N * B.R;
        if (own == in_m) {
            for (int c = 0; c < rank; c += 16) {
                v4i tf[NS];
                lora_t_frag<NS>(tr + c, sc, tf);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    v4i bf = *reinterpret_cast<const v4i *>(bl[j] + off + c);
                    if (c + 16 > rank) bf = keep8(bf, rank - c - 8 * lh);
#pragma unroll
                    for (int p = NS - 1; p >= 0; p--) v[j] = mfma32(bf, tf[p], v[j]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                v16f d;
#pragma unroll
                for (int e = 0; e < 16; e++) d[e] = 0.0f;
                for (int c = 0; c < rank; c += 16) {
                    v4i tf[NS];
                    lora_t_frag<NS>(tr + c, sc, tf);
                    v4i bf = *reinterpret_cast<const v4i *>(bl[j] + off + c);
                    if (c + 16 > rank) bf = keep8(bf, rank - c - 8 * lh);
#pragma unroll
                    for (int p = NS - 1; p >= 0; p--) d = mfma32(bf, tf[p], d);
                }
#pragma unroll
                for (int e = 0; e < 16; e++) v[j][e] = mine == a ? v[j][e] + d[e] : v[j][e];
            }
        }
    }
}

}  // namespace dmpq
