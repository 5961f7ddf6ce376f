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
// The bf16 MFMA multiplies an fp32 operand as 3 bf16 parts, each the leading 8
// bits of what the parts before it leave: together all its 24 bits.  Results
// that are rounded to bf16 take 3 parts too: where the adapter term cancels
// against what it is added to, what 2 parts lose is many bf16 steps of the
// result.  Cut off and not rounded, no part exceeds the value, so the largest
// fp32 numbers do not become infinite.  An infinite or NaN value is its own
// first part (a quiet NaN, as arithmetic gives, has its mark in the upper
// half); the later parts are then some finite values, which change neither.
//
// The other factor's infinities and NaN may meet the first part only: the
// later ones may be 0, and 0 * inf is not what the whole value gives.  Where
// that factor is at hand as fragments, the later parts multiply finite8() of
// it.  Where it lies in LDS it does so as ones8(), and a product that is taken
// only if such a value was seen adds odd8() of it times the value's sign
// (sign8): a branch in every product instead cost the INT8 GEMM 6% at rank 64,
// this way 3%.
// Either way inf * value is infinite with the right sign and inf * 0 NaN; with
// finite8() a value below bf16's range (2^-133) counts as 0 there.
constexpr int kParts = 3;

__device__ __forceinline__ float split_rest(float v) {  // v without its first part
    return v - __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
}
__device__ __forceinline__ float split_finite(float v) {
    return __builtin_amdgcn_fmed3f(v, -3.402823466e38f, 3.402823466e38f);
}

__device__ __forceinline__ void split8(const float v[8], v4i (&out)[kParts]) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; i++) r[i] = v[i];
#pragma unroll
    for (int p = 0; p < kParts; p++) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            out[p][i] = (int)__builtin_amdgcn_perm(__float_as_uint(r[2 * i + 1]), __float_as_uint(r[2 * i]), 0x07060302u);
        if (p + 1 < kParts)
#pragma unroll
            for (int i = 0; i < 8; i++) r[i] = split_rest(p == 0 ? split_finite(r[i]) : r[i]);
    }
}

// Bits 15 and 31 of a word: its two bf16 values are infinite or NaN (all ones
// in the exponent, which adding one carries out of).
__device__ __forceinline__ uint32_t nonfinite2(int w) { return (((uint32_t)w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// The same question for many words at once: magnitudes8() takes the largest
// of each half's bits without the sign, which is 0x7F80 or more after such a
// value (two operations a word).
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void magnitudes8(const v4i &v, u16x2 &top) {
#pragma unroll
    for (int d = 0; d < 4; d++) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, v[d] & 0x7FFF7FFF));
}
__device__ __forceinline__ bool nonfinite_in(u16x2 top) { return top[0] >= 0x7F80 || top[1] >= 0x7F80; }

// All ones in the halves of a word that nonfinite2 found.
__device__ __forceinline__ uint32_t halves(uint32_t found) { return (found >> 15) * 0xFFFFu; }

// 8 bf16 values with 0 in place of infinities and NaN;
__device__ __forceinline__ v4i finite8(v4i v) {
#pragma unroll
    for (int d = 0; d < 4; d++) v[d] &= (int)~halves(nonfinite2(v[d]));
    return v;
}

// with 1 of their sign in their place;
__device__ __forceinline__ v4i ones8(v4i v) {
#pragma unroll
    for (int d = 0; d < 4; d++) {
        const uint32_t h = halves(nonfinite2(v[d]));
        v[d] = (int)(((uint32_t)v[d] & (~h | 0x80008000u)) | (h & 0x3F803F80u));
    }
    return v;
}

// and only infinities and NaN, 0 in place of the others.
__device__ __forceinline__ v4i odd8(v4i v) {
#pragma unroll
    for (int d = 0; d < 4; d++) v[d] &= (int)halves(nonfinite2(v[d]));
    return v;
}

// The signs of 8 fp32 values as bf16 1, -1 and 0 (of a NaN: 1 or -1; the
// products with ones8() are NaN by then).
__device__ __forceinline__ v4i sign8(const float v[8]) {
    v4i o;
#pragma unroll
    for (int d = 0; d < 4; d++) {
        const uint32_t lo = v[2 * d] == 0.0f ? 0u : (__float_as_uint(v[2 * d]) >> 16 & 0x8000u) | 0x3F80u;
        const uint32_t hi = v[2 * d + 1] == 0.0f ? 0u : (__float_as_uint(v[2 * d + 1]) >> 16 & 0x8000u) | 0x3F80u;
        o[d] = (int)(lo | hi << 16);
    }
    return o;
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
// y = projection + scale * (t b^T) by request: the scale multiplies the sum of
// the products, as in the expand kernel, so that the two agree for every scale.
//
// Of one 32-row slice, run by one wave on its own (the fixup of split tiles):
// v = scale * (t b^T) for 32 rows x 128 columns in the GEMMs' accumulator
// layout: lane l holds row l % 32 (`row`; past M: unspecified) and, in
// v[j][4g + e], column n0 + 32 j + 8 g + 4 (l / 32) + e.  Rows without adapter or
// of rank 0 get -0, which adds nothing to any number.  b's rows are the MFMA's
// first operand, t in bf16 parts (split8) the second.  Where all rows share an
// adapter the products accumulate straight onto v.  Rows of several adapters
// take one product per adapter over all 32 rows, kept where it belongs and never
// multiplied by zero elsewhere: one adapter's infinity must not reach another
// request's rows.
__device__ __forceinline__ void lora_t_frag(const float *tr, v4i (&tf)[kParts]) {
    const v4f a0 = *reinterpret_cast<const v4f *>(tr), a1 = *reinterpret_cast<const v4f *>(tr + 4);
    const float v[8] = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
    split8(v, tf);
}

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
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int e = 0; e < 16; e++) v[j][e] = -0.0f;
    uint64_t todo = __ballot(mine >= 0);
    const uint64_t in_m = __ballot(row < B.M);
    while (todo) {
        const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
        const uint64_t own = __ballot(mine == a);
        todo &= ~own;
        const int rank = adapter_rank(B, a);
        if (rank == 0) continue;
        const float sc = B.scale[a];
        const int64_t off = (int64_t)a * N * B.R;
        if (own == in_m) {
            for (int c = 0; c < rank; c += 16) {
                v4i tf[kParts];
                lora_t_frag(tr + c, tf);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    v4i bf = *reinterpret_cast<const v4i *>(bl[j] + off + c);
                    if (c + 16 > rank) bf = keep8(bf, rank - c - 8 * lh);
                    const v4i fin = finite8(bf);
#pragma unroll
                    for (int p = kParts - 1; p >= 0; p--) v[j] = mfma32(p > 0 ? fin : bf, tf[p], v[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int e = 0; e < 16; e++) v[j][e] *= sc;
        } else {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                v16f d;
#pragma unroll
                for (int e = 0; e < 16; e++) d[e] = 0.0f;
                for (int c = 0; c < rank; c += 16) {
                    v4i tf[kParts];
                    lora_t_frag(tr + c, tf);
                    v4i bf = *reinterpret_cast<const v4i *>(bl[j] + off + c);
                    if (c + 16 > rank) bf = keep8(bf, rank - c - 8 * lh);
                    const v4i fin = finite8(bf);
#pragma unroll
                    for (int p = kParts - 1; p >= 0; p--) d = mfma32(p > 0 ? fin : bf, tf[p], d);
                }
#pragma unroll
                for (int e = 0; e < 16; e++) v[j][e] = mine == a ? sc * d[e] : v[j][e];
            }
        }
    }
}

// Of a 256 x 256 tile of 2 x 2 waves, slice by slice: the epilogue writes 32
// rows of every wave's scaled fp32 values to LDS bands, and lora_band_add adds
// the adapters' products to the bands.  (Onto the scaled values in registers
// the products need no LDS traffic, but the code between the main loop and the
// stores then spills: the INT8 GEMM of 17776 x 1920 x 5760, 211 us without the
// term, took 269 without a single adapter and 303 at rank 16; 253 and 284 with
// the bands.)
//
// The workgroup copies b's 256 rows of one request into LDS (entries past the
// rank as zeros); a tile that belongs to one request does so once.  A lane
// loads its row of t straight from memory, a slice ahead of its use and so
// before the stores of the slice between.  The products of a request start
// from zero and are added to its own rows only, never zero times b: one
// adapter's infinity must not reach another request's rows.
constexpr int kLoraBandStride = 128 * 4 + 16;             // an fp32 band row of 128 columns
constexpr int kLoraBandBytes = 32 * kLoraBandStride;      // one wave's slice
constexpr int kLoraBOff = 4 * kLoraBandBytes;
constexpr int kLoraMeta = 4 * 64 * 4;  // the first 64 of seg_start, seg_adapter, rank and scale
// beside it: the INT8 GEMM's scales, the meta words, the amax words
constexpr int kLoraLds = 160 * 1024 - 2048 - kLoraMeta - 256;

// Copies the meta words by LDS DMA, one array a wave, in the kernel's prologue:
// they land during the main loop and are visible after its barriers, so that
// the epilogue starts without a chain of dependent loads.
__device__ __forceinline__ void lora_meta_dma(const LoraBatch &B, uint8_t *meta, int tid) {
    typedef __attribute__((address_space(3))) void lds_void;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const void *src = nullptr;
    if (wave == 0) src = B.seg_start + (lane < B.S ? lane : B.S);
    if (wave == 1 && B.S > 0) src = B.seg_adapter + (lane < B.S ? lane : B.S - 1);
    if (wave == 2 && B.nA > 0) src = B.rank + (lane < B.nA ? lane : B.nA - 1);
    if (wave == 3 && B.nA > 0) src = B.scale + (lane < B.nA ? lane : B.nA - 1);
    if (src) __builtin_amdgcn_global_load_lds(src, (lds_void *)(meta + 256 * wave), 4, 0, 0);
}

// Request s's first row, its adapter, and an adapter's rank and scale: from
// the meta words where they are among the first 64.  All wave-uniform.
struct LoraWords {
    const int *w;
    __device__ __forceinline__ int start(const LoraBatch &B, int s) const {
        return __builtin_amdgcn_readfirstlane(s < 64 ? w[s] : B.seg_start[s]);
    }
    __device__ __forceinline__ int adapter(const LoraBatch &B, int s) const {
        const int a = __builtin_amdgcn_readfirstlane(s < 64 ? w[64 + s] : B.seg_adapter[s]);
        return a >= 0 && a < B.nA ? a : -1;
    }
    __device__ __forceinline__ int rank(const LoraBatch &B, int a) const {
        const int r = __builtin_amdgcn_readfirstlane(a < 64 ? w[128 + a] : B.rank[a]);
        return r < 0 ? 0 : r > B.R ? B.R : r;
    }
    __device__ __forceinline__ float scale(const LoraBatch &B, int a) const {
        return __int_as_float(__builtin_amdgcn_readfirstlane(a < 64 ? w[192 + a] : __float_as_int(B.scale[a])));
    }
};

// the last words of the area: for each wave, whether the b it copied holds an
// infinity or NaN
constexpr int kLoraOddOff = kLoraLds - 16;
static_assert(kLoraBOff + 256 * (2 * kMaxLoraRank + 16) <= kLoraOddOff && kLoraOddOff % 16 == 0, "bands and b fit");

// AHEAD: the 16-rank pieces of t that a lane holds a slice ahead; the others
// are loaded as they are used.  3 (a rank of 48) in the fp32-accumulator GEMMs:
// with 4 the NVFP4 kernels spill up to 25 registers (17776 x 1920 x 5760, rank
// 16: 434 us against 427; x 3072 x 9216, rank 64: 914 and 911; with 2: 423 and
// 919).  The INT8 GEMM's registers hold no more than 1: with 4 it takes 277 us
// without any adapter where it takes 253 with 1.
template <int AHEAD>
struct LoraRows {
    v4f v[AHEAD][2];
};

// What a workgroup keeps over the slices of its tile: the tile's rows, the
// first request that may have some, and the request whose b is in LDS with
// its rows of the tile, rank and scale, and whether that b is all finite.
struct LoraTile {
    LoraWords words;
    int r0, r1, s0, staged;
    int lo, hi, rank, odd;
    float sc;

    // request s's rows of the tile; false if there are none or no adapter
    __device__ __forceinline__ bool rows_of(const LoraBatch &B, int s, int &l, int &h, int &a) const {
        const int start = words.start(B, s), end = words.start(B, s + 1);
        a = words.adapter(B, s);
        l = start > r0 ? start : r0;
        h = end < r1 ? end : r1;
        return l < h && a >= 0;
    }
    // its b into LDS; the barriers around the copy are the caller's, who then
    // calls read_odd
    __device__ __forceinline__ void stage_b(const LoraEpi &L, int s, int l, int h, int a, int64_t n0, int64_t N,
                                            uint8_t *lds) {
        const LoraBatch &B = L.batch;
        const int brow = 2 * B.R + 16, per_row = B.R >> 3;
        const uint16_t *bw = L.b + (int64_t)a * N * B.R;
        staged = s, lo = l, hi = h;
        rank = words.rank(B, a);
        sc = words.scale(B, a);
        u16x2 top = {0, 0};
        auto at = [&](int e, int &n, int &c) {  // piece e: its row and place in it, its values
            n = e / per_row, c = e - n * per_row;
            const int64_t g = n0 + n < N ? n0 + n : N - 1;
            return keep8(*reinterpret_cast<const v4i *>(bw + g * B.R + 8 * c), rank - 8 * c);
        };
        int n, c;
#pragma unroll 4
        for (int e = threadIdx.x; e < 256 * per_row; e += 256) {
            const v4i f = at(e, n, c);
            *reinterpret_cast<v4i *>(lds + kLoraBOff + n * brow + 16 * c) = f;
            magnitudes8(f, top);
        }
        const uint64_t any = __ballot(nonfinite_in(top));
        if ((threadIdx.x & 63) == 0) reinterpret_cast<int *>(lds + kLoraOddOff)[threadIdx.x >> 6] = any != 0;
        if (__builtin_expect(any != 0, 0))
#pragma unroll 1
            for (int e = threadIdx.x; e < 256 * per_row; e += 256) {
                const v4i f = at(e, n, c);
                *reinterpret_cast<v4i *>(lds + kLoraBOff + n * brow + 16 * c) = ones8(f);
            }
    }
    __device__ __forceinline__ void read_odd(const uint8_t *lds) {
        const v4i w = *reinterpret_cast<const v4i *>(lds + kLoraOddOff);
        odd = __builtin_amdgcn_readfirstlane(w[0] | w[1] | w[2] | w[3]);
    }
    // the lane's row of t in slice i of its wave
    __device__ __forceinline__ const float *row(const LoraEpi &L, int i) const {
        const int r = r0 + (threadIdx.x >> 7) * 128 + 32 * i + (threadIdx.x & 31);
        return L.t + (int64_t)(r < L.batch.M ? r : L.batch.M - 1) * L.batch.R + 8 * ((threadIdx.x >> 5) & 1);
    }
    template <int AHEAD>
    __device__ __forceinline__ void load_t(const LoraEpi &L, int i, LoraRows<AHEAD> &t) const {
        const float *p = row(L, i);
#pragma unroll
        for (int c = 0; c < AHEAD; c++)
#pragma unroll
            for (int h = 0; h < 2; h++)
                t.v[c][h] = *reinterpret_cast<const v4f *>(p + (16 * c < L.batch.R ? 16 * c : 0) + 4 * h);
    }
};

// meta: the words of lora_meta_dma.
template <int AHEAD>
__device__ __forceinline__ LoraTile lora_tile_begin(const LoraEpi &L, int64_t m0, int64_t n0, int64_t N, uint8_t *lds,
                                                    const uint8_t *meta, LoraRows<AHEAD> &t) {
    const LoraBatch &B = L.batch;
    const int lane = threadIdx.x & 63;
    LoraTile T;
    T.words.w = reinterpret_cast<const int *>(meta);
    T.r0 = (int)m0;
    T.r1 = m0 + 256 < B.M ? (int)m0 + 256 : B.M;
    T.s0 = 0;
    T.staged = -1;
    T.lo = T.hi = T.rank = T.odd = 0;
    T.sc = 0.0f;
    T.load_t(L, 0, t);
    for (int c = 0; c <= B.S; c += 64) {  // the last request that starts at or before the tile
        const int at = c + lane <= B.S ? c + lane : B.S;
        const uint64_t below = __ballot(c + lane <= B.S && (c == 0 ? T.words.w[lane] : B.seg_start[at]) <= T.r0);
        const int n = __builtin_popcountll(below);
        T.s0 = c + n - 1;
        if (n < 64) break;
    }
    if (T.s0 < 0) T.s0 = 0;
    int l, h, a;
    if (T.s0 < B.S && T.rows_of(B, T.s0, l, h, a)) T.stage_b(L, T.s0, l, h, a, n0, N, lds);
    __syncthreads();
    if (T.staged >= 0) T.read_odd(lds);
    return T;
}

// Slice i of every wave.  Called by all four waves after they wrote their
// bands (lds + wave * kLoraBandBytes); returns with the wave's own band ready.
template <int AHEAD>
__device__ __forceinline__ void lora_band_add(const LoraEpi &L, LoraTile &T, int i, int64_t n0, int64_t N,
                                              uint8_t *lds, const LoraRows<AHEAD> &t) {
    const LoraBatch &B = L.batch;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lm = lane & 31, lh = lane >> 5, wm = wave >> 1, wn = wave & 1;
    const int brow = 2 * B.R + 16;
    uint8_t *band = lds + wave * kLoraBandBytes, *bs = lds + kLoraBOff;
    const int q0 = T.r0 + 32 * i, q1 = q0 + 128;  // the first rows of the two slices of this step
    const int mine0 = wm ? q1 : q0;
    for (int s = T.s0; s < B.S; s++) {
        if (T.staged != s || T.hi < T.r1) {  // (the staged request may be the tile's last)
            int l, h, a;
            const bool some = T.rows_of(B, s, l, h, a);
            if (T.words.start(B, s) >= T.r1) break;
            const bool in0 = l < q0 + 32 && h > q0, in1 = l < q1 + 32 && h > q1;
            if (!some || !(in0 || in1)) continue;  // workgroup-uniform
            if (T.staged != s) {
                __syncthreads();  // every wave is done with the last request's b
                T.stage_b(L, s, l, h, a, n0, N, lds);
                __syncthreads();
                T.read_odd(lds);
            }
        }
        const bool last = T.hi >= T.r1;
        if (T.rank > 0 && T.lo < mine0 + 32 && T.hi > mine0) {  // wave-uniform, no barrier inside
            v16f d[4];
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int e = 0; e < 16; e++) d[j][e] = 0.0f;
            auto piece = [&](int c, const v4f &a0, const v4f &a1) {
                const float v[8] = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
                v4i tf[kParts], bf[4];
                split8(v, tf);
#pragma unroll
                for (int j = 0; j < 4; j++)
                    bf[j] = *reinterpret_cast<const v4i *>(bs + (wn * 128 + 32 * j + lm) * brow + 2 * c + 16 * lh);
#pragma unroll
                for (int p = kParts - 1; p >= 0; p--)
#pragma unroll
                    for (int j = 0; j < 4; j++) d[j] = mfma32(bf[j], tf[p], d[j]);
            };
#pragma unroll
            for (int k = 0; k < AHEAD; k++)
                if (16 * k < T.rank) piece(16 * k, t.v[k][0], t.v[k][1]);
            if (T.rank > 16 * AHEAD) {
                const float *p = T.row(L, i);
                for (int c = 16 * AHEAD; c < T.rank; c += 16)
                    piece(c, *reinterpret_cast<const v4f *>(p + c), *reinterpret_cast<const v4f *>(p + c + 4));
            }
            if (__builtin_expect(T.odd, 0)) {  // b's infinities and NaN, from memory
                // (the empty asm keeps this branch's addresses from being computed, and
                // held in registers, before it)
                int tid = threadIdx.x;
                asm volatile("" : "+v"(tid));
                const int lm = tid & 31, lh = tid >> 5 & 1, wn = tid >> 6 & 1;
                const int r = T.r0 + (tid >> 7) * 128 + 32 * i + lm;
                const float *p = L.t + (int64_t)(r < B.M ? r : B.M - 1) * B.R + 8 * lh;
                const uint16_t *bw = L.b + (int64_t)T.words.adapter(B, s) * N * B.R + 8 * lh;
#pragma unroll 1
                for (int c = 0; c < T.rank; c += 16) {
                    const v4f a0 = *reinterpret_cast<const v4f *>(p + c), a1 = *reinterpret_cast<const v4f *>(p + c + 4);
                    const float v[8] = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
                    const v4i sf = sign8(v);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int64_t n = n0 + wn * 128 + 32 * j + lm;
                        const v4i f = *reinterpret_cast<const v4i *>(bw + (n < N ? n : N - 1) * B.R + c);
                        d[j] = mfma32(odd8(keep8(f, T.rank - c - 8 * lh)), sf, d[j]);
                    }
                }
            }
            const bool own = mine0 + lm >= T.lo && mine0 + lm < T.hi;
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    float4 *p = reinterpret_cast<float4 *>(band + lm * kLoraBandStride + (32 * j + 8 * g + 4 * lh) * 4);
                    float4 o = *p;
                    if (own) {
                        o.x = __builtin_fmaf(T.sc, d[j][4 * g], o.x), o.y = __builtin_fmaf(T.sc, d[j][4 * g + 1], o.y);
                        o.z = __builtin_fmaf(T.sc, d[j][4 * g + 2], o.z), o.w = __builtin_fmaf(T.sc, d[j][4 * g + 3], o.w);
                        *p = o;
                    }
                }
        }
        if (T.staged == s && last) break;
    }
}

}  // namespace dmpq
