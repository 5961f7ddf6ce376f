// gemm_common.hpp -- tile scheduling shared by the quantized GEMMs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device.hpp"
#include "internal.hpp"
#include "linear.hpp"
#include "lora.hpp"

namespace dmpq {

// Map a 1-D workgroup id onto an (m, n) output tile.
// 1. XCD-aware: the dispatcher deals workgroups round-robin to the 8 XCDs
//    (id % 8), each with its own L2.  Renumber so that each XCD receives a
//    contiguous range of logical ids (the ids beyond the last multiple of 8
//    keep their number).
// 2. Grouped order: consecutive logical ids walk down a band of `group_m`
//    tile rows before moving right, so the A rows and W columns one XCD is
//    working on at a time stay few and L2-resident.
struct TileCoord {
    unsigned m, n;
};

__device__ __forceinline__ unsigned xcd_order(unsigned bid, unsigned nwg) {
    const unsigned full = nwg & ~7u;
    return bid < full ? (bid & 7u) * (full >> 3) + (bid >> 3) : bid;
}

__device__ __forceinline__ TileCoord tile_at(unsigned pid, unsigned tiles_m, unsigned tiles_n,
                                             unsigned group_m) {
    const unsigned per_group = group_m * tiles_n;
    const unsigned g = pid / per_group;
    const unsigned first_m = g * group_m;
    const unsigned rows = min(tiles_m - first_m, group_m);
    const unsigned in_group = pid - g * per_group;
    return TileCoord{first_m + in_group % rows, in_group / rows};
}

__device__ __forceinline__ TileCoord tile_of(unsigned bid, unsigned nwg, unsigned tiles_m,
                                             unsigned tiles_n, unsigned group_m) {
    return tile_at(xcd_order(bid, nwg), tiles_m, tiles_n, group_m);
}

// The tile in scalar registers: the forms of the whole linear use it in vector
// arithmetic too, and the compiler may keep it there only.
template <int EPI>
__device__ __forceinline__ TileCoord tile_scalar(TileCoord tc);

// A split workgroup of a SplitPlan launch: workgroup j runs the K stages
// [s * nk / splits, (s + 1) * nk / splits) of tail tile full + j / splits,
// s = j % splits.
struct SplitUnit {
    TileCoord tc;
    int kt0, kt1;
};

__device__ __forceinline__ SplitUnit split_unit(const SplitPlan &sp, unsigned tiles_m, unsigned tiles_n,
                                                unsigned group_m) {
    const unsigned j = blockIdx.x;
    const unsigned s = j % sp.splits;
    SplitUnit u;
    u.tc = tile_at(sp.full + j / sp.splits, tiles_m, tiles_n, group_m);
    u.kt0 = (int)((int64_t)s * sp.nk / sp.splits);
    u.kt1 = (int)((int64_t)(s + 1) * sp.nk / sp.splits);
    return u;
}

// Host: the split plan of a launch of `tiles` tiles with nk K stages each.
// The tail is split into as many parts as fit in one wave of kMaxSplitUnits
// workgroups (at most one stage each; 2, 3, 4 or 8 parts); a tail that
// cannot be split at least in two is not split.
inline SplitPlan plan_split(int64_t tiles, int nk, bool enable) {
    SplitPlan p{(unsigned)tiles, 0u, 1u, nk};
    const int64_t tail = tiles % 256;
    if (!enable || tail == 0) return p;
    int64_t S = (int64_t)kMaxSplitUnits / tail;
    if (S > nk) S = nk;
    S = S >= 8 ? 8 : S >= 4 ? 4 : S;  // 2, 3, 4 or 8: the fixup is compiled per count
    if (S < 2) return p;
    p.full = (unsigned)(tiles - tail);
    p.tail = (unsigned)tail;
    p.splits = (unsigned)S;
    return p;
}

// Raw accumulators of one split workgroup: 256 words per thread, as 64
// 16-byte pieces (register group g of MFMA block (i, j) is piece 4(4i+j)+g);
// for each piece the workgroup writes 4 KB contiguously.
template <class AccV>
__device__ __forceinline__ void store_split_partial(const AccV (&acc)[4][4], uint32_t *part, int tid) {
    typedef decltype(acc[0][0][0] + 0) T;
    uint4 *p4 = reinterpret_cast<uint4 *>(part);
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                // copy the elements out first: a bit cast of a vector-element
                // lvalue reads from the vector's base, i.e. element 0
                const T v0 = acc[i][j][4 * g], v1 = acc[i][j][4 * g + 1];
                const T v2 = acc[i][j][4 * g + 2], v3 = acc[i][j][4 * g + 3];
                p4[((i * 4 + j) * 4 + g) * 256 + tid] =
                    make_uint4(__builtin_bit_cast(uint32_t, v0), __builtin_bit_cast(uint32_t, v1),
                               __builtin_bit_cast(uint32_t, v2), __builtin_bit_cast(uint32_t, v3));
            }
}

}  // namespace dmpq

namespace dmpq {

// ---------------------------------------------------------------------------
// Epilogue staging.  A wave's output tile is 128 x 128; it is written out in
// two bands of 64 rows.  The accumulators (transposed MFMA layout: lane =
// row, 4 consecutive columns per register group) are converted and written
// into a per-wave LDS band, which is then read back row-contiguous so that
// every global store instruction writes whole rows, 16 bytes per lane.
// ---------------------------------------------------------------------------
constexpr int kEpiRows = 64;
template <int ESIZE>
struct EpiBand {
    static constexpr int ROW_BYTES = 128 * ESIZE;      // 128 output columns
    static constexpr int STRIDE = ROW_BYTES + 16;      // padded LDS row
    static constexpr int BYTES = kEpiRows * STRIDE;    // per-wave LDS band
    static constexpr int LANES_PER_ROW = ROW_BYTES / 16;
    static constexpr int ROWS_PER_PASS = 64 / LANES_PER_ROW;
};

// Epilogue options (bit flags).  kEpiGelu: GELU(v) = v Phi(v) of the output
// value as a separate bf16 (or fp32) activation op would see it: the GEMM
// result is rounded to the output type first, GELU runs in fp32 and its
// result is rounded again.  kEpiAmax (bf16 output, N % 16 == 0): the maximum
// of |FWHT16(row block)| over the stored bf16 values of the tile -- the next
// layer's NVFP4 tensor-amax term, with the same fp32 butterfly order as the
// quantizer -- is written to the tile's entry of the maxima.  kEpiLora: the
// adapter term of the row's request is added to the fp32 value before any of
// that, so it costs no pass over y of its own.  kEpiLinear: the whole linear's
// epilogue (linear.hpp), whose operands are known at run time; with kEpiHeads
// it norms and rotates the heads of q and k, with kEpiBand through LDS bands
// (adapters, and shapes that the form from registers does not take).
enum { kEpiGelu = 1, kEpiAmax = 2, kEpiLora = 4, kEpiLinear = 8, kEpiHeads = 16, kEpiBand = 32 };
// the flags of one call
inline int linear_epi(bool amax, const LinearEpi &L, int64_t N) {
    return kEpiLinear | (amax ? kEpiAmax : 0) | (L.lora.t ? kEpiLora : 0) | (L.qk.D ? kEpiHeads : 0) |
           (L.qk.D && !L.lora.t && !heads_from_regs(L, N) ? kEpiBand : 0);
}
constexpr bool heads_in_regs(int epi) { return (epi & kEpiHeads) != 0 && (epi & (kEpiLora | kEpiBand)) == 0; }

template <int EPI>
__device__ __forceinline__ TileCoord tile_scalar(TileCoord tc) {
    if constexpr ((EPI & kEpiLinear) != 0)
        return TileCoord{(unsigned)__builtin_amdgcn_readfirstlane((int)tc.m), (unsigned)__builtin_amdgcn_readfirstlane((int)tc.n)};
    return tc;
}

// The epilogue's operands as a kernel argument.  (A member type, not an
// expression of EPI: that one would enter the kernels' names, where host and
// device spell an unnamed enum differently.)
template <bool LINEAR>
struct EpiOperands {
    typedef LoraEpi type;
};
template <>
struct EpiOperands<true> {
    typedef LinearEpi type;
};
template <int EPI>
struct EpiArgOf {
    typedef typename EpiOperands<(EPI & kEpiLinear) != 0>::type type;
};
template <int EPI>
using EpiArg = typename EpiArgOf<EPI>::type;
__device__ __forceinline__ const LoraEpi &lora_of(const LoraEpi &e) { return e; }
__device__ __forceinline__ const LoraEpi &lora_of(const LinearEpi &e) { return e.lora; }

// The other half of a wave's value (lane l: that of lane l ^ 32), by the swap of
// the halves of two registers.
__device__ __forceinline__ float other_half(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);  // {lower, lower}, {upper, upper}
    return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// max |value| of the rotated 16-block whose elements 0..7 (lo) or 8..15 the
// lane holds as bf16; the other half is its neighbour's.  Stages 1, 2, 4 in the
// lane, stage 8 across the pair, then * 1/4: the quantizer's order.
__device__ __forceinline__ float block16_amax(const uint4 &v, bool lo) {
    float f[8];
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
#pragma unroll
        for (int i = 0; i < 8; i++)
            if ((i & h) == 0) {
                const float a = f[i], b = f[i + h];
                f[i] = a + b;
                f[i + h] = a - b;
            }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        // the partner lane's value: DPP quad_perm [1, 0, 3, 2] swaps
        // lanes 2k and 2k+1 inside the VALU (no LDS round trip)
        const float o = dpp_f32<0xB1>(f[i]);
        const float w = lo ? f[i] + o : o - f[i];
        m = fmaxf(m, __builtin_fabsf(w * 0.25f));
    }
    return m;
}

// Copy one wave's LDS band (ROWS x 128 values of ESIZE bytes) to y at
// (row0, col0), clipping to M x N.  vec: rows of y are 16-byte aligned.
// kEpiGelu: each value passes through GELU on its way out.  kEpiAmax (bf16
// only): the two lanes holding one 16-block finish its Hadamard (stages 1,
// 2, 4 in-lane, stage 8 across the lane pair, then * 1/4) and the lane's max
// |value| over valid blocks is returned.  BAND32: the band holds fp32 (rows of
// kLoraBandStride bytes) whatever the output type.
template <int ESIZE, int EPI = 0, int ROWS = kEpiRows, bool BAND32 = false>
__device__ __forceinline__ float epi_band_to_global(const uint8_t *band, void *y, int64_t M,
                                                    int64_t N, int64_t row0, int64_t col0,
                                                    int lane, bool vec) {
    using B = EpiBand<ESIZE>;
    constexpr int PER = 16 / ESIZE;  // values per lane per pass
    constexpr bool AMAX = (EPI & kEpiAmax) != 0;
    static_assert(!AMAX || ESIZE == 2, "the fused amax reads bf16 outputs");
    const int chunk = lane % B::LANES_PER_ROW;
    const int64_t col = col0 + chunk * PER;
    float amax = 0.0f;
#pragma unroll 4
    for (int p = 0; p < ROWS / B::ROWS_PER_PASS; p++) {
        const int r = p * B::ROWS_PER_PASS + lane / B::LANES_PER_ROW;
        const int64_t row = row0 + r;
        uint4 v;
        if constexpr (BAND32 && ESIZE == 2) {
            const float4 a = *reinterpret_cast<const float4 *>(band + r * kLoraBandStride + chunk * 32);
            const float4 b = *reinterpret_cast<const float4 *>(band + r * kLoraBandStride + chunk * 32 + 16);
            v = make_uint4(cvt_pk_bf16(a.x, a.y), cvt_pk_bf16(a.z, a.w), cvt_pk_bf16(b.x, b.y), cvt_pk_bf16(b.z, b.w));
        } else {
            v = *reinterpret_cast<const uint4 *>(band + r * B::STRIDE + chunk * 16);
        }
        if constexpr ((EPI & kEpiGelu) != 0) {
            if constexpr (ESIZE == 2) {
                v.x = cvt_pk_bf16(gelu_f32(bf16_lo(v.x)), gelu_f32(bf16_hi(v.x)));
                v.y = cvt_pk_bf16(gelu_f32(bf16_lo(v.y)), gelu_f32(bf16_hi(v.y)));
                v.z = cvt_pk_bf16(gelu_f32(bf16_lo(v.z)), gelu_f32(bf16_hi(v.z)));
                v.w = cvt_pk_bf16(gelu_f32(bf16_lo(v.w)), gelu_f32(bf16_hi(v.w)));
            } else {
                v.x = __float_as_uint(gelu_f32(__uint_as_float(v.x)));
                v.y = __float_as_uint(gelu_f32(__uint_as_float(v.y)));
                v.z = __float_as_uint(gelu_f32(__uint_as_float(v.z)));
                v.w = __float_as_uint(gelu_f32(__uint_as_float(v.w)));
            }
        }
        if constexpr (AMAX) {
            const float m = block16_amax(v, (chunk & 1) == 0);
            if (row < M && col < N) amax = fmaxf(amax, m);
        }
        if (row >= M || col >= N) continue;
        uint8_t *dst = static_cast<uint8_t *>(y) + (row * N + col) * ESIZE;
        if (vec && col + PER <= N) {
            // streaming store: every tile of a launch finishes at about the same
            // time, and the burst of outputs drains faster without L2 allocation
            store_nt16(dst, v);
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < PER; e++) {
                if (col + e >= N) break;
                if constexpr (ESIZE == 4)
                    reinterpret_cast<uint32_t *>(dst)[e] = w[e];
                else
                    reinterpret_cast<uint16_t *>(dst)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
            }
        }
    }
    return amax;
}

// The whole linear's epilogue for the 16 bytes of columns from `col` on that a
// lane holds of one row: v are the scaled sums (with the adapter term); bias, pre,
// heads, activation, gate, residual, one rounding, store.  A lane has the same
// columns in every row, so what depends on the column is loaded once (T, Q).
// chunk: the lane's place in the row; residual: the lane's 16 bytes of it, where
// they are loaded already.
// Returns the lane's part of the fused amax (kEpiAmax, where want_amax).  All lanes
// of the wave call it together.
template <int ESIZE, int EPI>
__device__ __forceinline__ float linear_row_out(float (&v)[16 / ESIZE], void *y, int64_t M, int64_t N, int64_t row,
                                                int64_t col, int chunk, bool vec, const LinearEpi &L,
                                                const LinearLane<16 / ESIZE> &T, const QkLane<16 / ESIZE> &Q,
                                                bool want_amax, const uint4 *residual = nullptr) {
    constexpr int PER = 16 / ESIZE;
    const bool in = row < M && col < N;
#pragma unroll
    for (int i = 0; i < PER; i++) v[i] += T.bias[i];
    if (L.pre && in) store_values<ESIZE, PER>(L.pre, row * N + col, N - col, vec, v);
    if constexpr ((EPI & kEpiHeads) != 0)
        Q.apply(L.qk, row < M ? row : M - 1, v);
    else
        act_apply<PER>(v, L.act);
    T.template finish<ESIZE>(L, row, N, col, in, vec, v, residual);
    float m = 0.0f;
    if constexpr ((EPI & kEpiAmax) != 0) {
        static_assert(ESIZE == 2, "the fused amax reads bf16 outputs");
        if (want_amax) {
            m = block16_amax(make_uint4(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]), cvt_pk_bf16(v[4], v[5]),
                                        cvt_pk_bf16(v[6], v[7])), (chunk & 1) == 0);
            if (!in) m = 0.0f;
        }
    }
    if (in) store_values<ESIZE, PER>(y, row * N + col, N - col, vec, v);
    return m;
}

// A pointer that is the same in every lane, in scalar registers.
__device__ __forceinline__ uint8_t *uniform_ptr(uint8_t *p) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u), hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
    return reinterpret_cast<uint8_t *>((uint64_t)hi << 32 | lo);
}

// The rows of a band where they are whole 16-byte pieces: one pass of the loop is
// one store of 64 lanes, with as little around it as the call leaves (its wave is
// alone on its SIMD, and every instruction counts): the activation, and whether
// there is more than it and the bias, are chosen outside.
constexpr int64_t kMaxFastN = int64_t(1) << 26;
template <int ESIZE>
struct BandPlace {
    static constexpr int PER = 16 / ESIZE, LPR = 128 / PER, RPP = 64 / LPR, GROUP = 4;  // passes of a group
    int64_t base, step;  // bytes: of the band's first row and column in y, pre and the residual; of a pass
    uint32_t off;        // the lane's
    int rows;            // there are, from the lane's on; none for lanes whose columns are past the end
    int last;            // the band's last row, or its first where there is none
    __device__ __forceinline__ BandPlace(int64_t M, int64_t N, int64_t row0, int64_t col0, int lane, int most) {
        const int lr = lane / LPR, chunk = lane % LPR;
        base = (row0 * N + col0) * ESIZE, step = RPP * N * ESIZE;
        off = (uint32_t)lr * (uint32_t)N * ESIZE + 16 * chunk;
        const int count = M <= row0 ? 0 : (int)(M - row0 < most ? M - row0 : most);
        rows = col0 + chunk * PER < N ? count - lr : 0;
        last = count > 0 ? count - 1 : 0;
    }
    // the residual of group g
    __device__ __forceinline__ void ahead(const LinearEpi &L, int g, uint4 (&r)[GROUP]) const {
        const uint8_t *p = uniform_ptr(const_cast<uint8_t *>(static_cast<const uint8_t *>(L.residual)) + base + g * GROUP * step);
#pragma unroll
        for (int k = 0; k < GROUP; k++) {
            r[k] = make_uint4(0, 0, 0, 0);
            if ((g * GROUP + k) * RPP < rows) r[k] = load_nt16(p + k * step + off);
        }
    }
};

// With more than bias and activation (MORE) the residual comes in a group of
// passes ahead, the first one (r) before the band was written (INT8 17776 x 1920 x 7680
// with gate and residual: 302 us, 333 with each pass's loads waited for).
template <int ESIZE, int EPI, int ROWS, int ACT, bool MORE>
__device__ __forceinline__ float linear_band_rows(const uint8_t *band, void *y, int64_t N, int64_t row0, int64_t col0, int lane,
                                                  const LinearEpi &L, LinearLane<16 / ESIZE> &T,
                                                  const BandPlace<ESIZE> &B, uint4 (&r)[4]) {
    typedef BandPlace<ESIZE> P;
    constexpr int PER = P::PER, LPR = P::LPR, RPP = P::RPP, GROUP = P::GROUP;
    const int chunk = lane % LPR, lr = lane / LPR;
    const uint8_t *src = band + lr * kLoraBandStride + 4 * PER * chunk;
    uint8_t *py = uniform_ptr(static_cast<uint8_t *>(y) + B.base), *pp = nullptr;
    if (MORE && L.pre) pp = uniform_ptr(static_cast<uint8_t *>(L.pre) + B.base);
    float amax = 0.0f;
    int requests = 0;  // of the band's rows, in its first ROWS lanes
    if (MORE && T.mode == kGateMixed) requests = request_of(L.gate_start, L.S, (int)(row0 + (lane < B.last ? lane : B.last)));
#pragma unroll 1
    for (int g = 0; g < ROWS / RPP / GROUP; g++) {
        uint4 next[GROUP];
        if (MORE && L.residual && (g + 1) * GROUP < ROWS / RPP) B.ahead(L, g + 1, next);
#pragma unroll
        for (int k = 0; k < GROUP; k++) {
            const bool in = (g * GROUP + k) * RPP < B.rows;
            float v[PER];
#pragma unroll
            for (int i = 0; i < PER; i += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(src + k * RPP * kLoraBandStride + 4 * i);
                v[i] = a.x + T.bias[i], v[i + 1] = a.y + T.bias[i + 1];
                v[i + 2] = a.z + T.bias[i + 2], v[i + 3] = a.w + T.bias[i + 3];
            }
            auto store = [&](uint8_t *to) __attribute__((always_inline)) {
                uint4 u;
                if constexpr (ESIZE == 4)
                    u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
                else
                    u = make_uint4(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]), cvt_pk_bf16(v[PER - 4], v[PER - 3]),
                                   cvt_pk_bf16(v[PER - 2], v[PER - 1]));
                if (in) store_nt16(to + k * B.step + B.off, u);
                return u;
            };
            if (MORE && pp) store(pp);
            act_apply<PER>(v, ACT);
            if constexpr (MORE) {
                if (T.mode == kGateMixed) T.turn(L, __shfl(requests, (g * GROUP + k) * RPP + lr, 64), N, col0 + chunk * PER);
                if (T.mode == kGateOne) {
#pragma unroll
                    for (int i = 0; i < PER; i++) v[i] *= T.gate[i];
                } else if (T.mode != kGateNone) {
                    // rows of no request take no term at all, not zero times one
                    const bool some = T.mode == kGateMixed && T.held >= 0 && T.held < L.S;
#pragma unroll
                    for (int i = 0; i < PER; i++) v[i] = some ? v[i] * T.gate[i] : L.residual ? -0.0f : 0.0f;
                }
                if (L.residual) {
                    const uint32_t w[4] = {r[k].x, r[k].y, r[k].z, r[k].w};
#pragma unroll
                    for (int i = 0; i < PER; i++)
                        v[i] += ESIZE == 4 ? __uint_as_float(w[i * ESIZE / 4]) : i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
                }
            }
            const uint4 u = store(py);
            if constexpr ((EPI & kEpiAmax) != 0) {
                const float m = block16_amax(u, (chunk & 1) == 0);
                if (in) amax = fmaxf(amax, m);
            }
        }
        src += GROUP * RPP * kLoraBandStride;
        py += GROUP * B.step;
        if (MORE) {
            if (pp) pp += GROUP * B.step;
#pragma unroll
            for (int k = 0; k < GROUP; k++) r[k] = next[k];
        }
    }
    return amax;
}

template <int ESIZE, int EPI, int ROWS>
__device__ __forceinline__ float linear_band_fast(const uint8_t *band, void *y, int64_t M, int64_t N, int64_t row0,
                                                  int64_t col0, int lane, const LinearEpi &L,
                                                  LinearLane<16 / ESIZE> &T, uint4 (&r)[4]) {
    const bool more = L.pre || L.residual || T.mode != kGateNone;
    const BandPlace<ESIZE> B(M, N, row0, col0, lane, ROWS);
#define DMPQ_ROWS(ACT_)                                                                                            \
    return more ? linear_band_rows<ESIZE, EPI, ROWS, ACT_, true>(band, y, N, row0, col0, lane, L, T, B, r)        \
                : linear_band_rows<ESIZE, EPI, ROWS, ACT_, false>(band, y, N, row0, col0, lane, L, T, B, r)
    if (L.act == kActNone) DMPQ_ROWS(kActNone);
    if (L.act == kActGelu) DMPQ_ROWS(kActGelu);
    if (L.act == kActGeluTanh) DMPQ_ROWS(kActGeluTanh);
    DMPQ_ROWS(kActSilu);
#undef DMPQ_ROWS
}

// The first rows' residual of a band, to be loaded before the band is written.
template <int ESIZE>
__device__ __forceinline__ void linear_residual(const LinearEpi &L, int64_t M, int64_t N, int64_t row0, int64_t col0, int lane,
                                                bool vec, int rows, uint4 (&r)[4]) {
    if (L.residual && vec && N <= kMaxFastN) BandPlace<ESIZE>(M, N, row0, col0, lane, rows).ahead(L, 0, r);
}

// The epilogue of one wave's fp32 LDS band of ROWS rows of 128 columns from row0 on
// (kLoraBandStride bytes apart).  residual: linear_residual's.
template <int ESIZE, int EPI, int ROWS>
__device__ __forceinline__ float linear_band_out(const uint8_t *band, void *y, int64_t M, int64_t N, int64_t row0,
                                                 int64_t col0, int lane, bool vec, const LinearEpi &L,
                                                 LinearLane<16 / ESIZE> &T, const QkLane<16 / ESIZE> &Q,
                                                 uint4 (&residual)[4]) {
    constexpr int PER = 16 / ESIZE, LPR = 128 / PER, RPP = 64 / LPR;
    const int chunk = lane % LPR;
    const int64_t col = col0 + chunk * PER;
    if constexpr ((EPI & kEpiHeads) == 0)
        if (vec && N <= kMaxFastN) return linear_band_fast<ESIZE, EPI, ROWS>(band, y, M, N, row0, col0, lane, L, T, residual);
    float amax = 0.0f;
    int request = 0;
    if (T.mode == kGateMixed) {
        const int64_t r = row0 + (lane & (ROWS - 1));
        request = request_of(L.gate_start, L.S, (int)(r < M ? r : M - 1));
    }
#pragma unroll 2
    for (int p = 0; p < ROWS / RPP; p++) {
        const int r = p * RPP + lane / LPR;
        float v[PER];
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(band + r * kLoraBandStride + (chunk * PER + i) * 4);
            v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
        }
        T.turn(L, __shfl(request, r, 64), N, col);
        amax = fmaxf(amax, linear_row_out<ESIZE, EPI>(v, y, M, N, row0 + r, col, chunk, vec, L, T, Q, true));
    }
    return amax;
}

typedef float v16f __attribute__((ext_vector_type(16)));

// The fused amax of a 256 x 256 tile: every wave's maximum, combined through
// LDS, written by one lane to *slot (the tile's own entry).  Called by all
// four waves.
__device__ __forceinline__ void epi_tile_amax(float m, int wave, int lane, float *slot) {
    __shared__ float red[4];
    m = wave_max(m);
    if (lane == 0) red[wave] = m;
    __syncthreads();
    if (wave == 0 && lane == 0) *slot = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

// Output scaling of fp32 accumulators: y = (acc * gA) * gW.
struct EpiScaleF32 {
    float gA, gW;
    __device__ __forceinline__ void row(int64_t) {}
    __device__ __forceinline__ float operator()(float a, int, int, int) const { return (a * gA) * gW; }
};

// Generic band epilogue: accumulators in the transposed MFMA layout (lane l
// owns row l % 32 of A-subtile i and four consecutive output columns
// 8g + 4*(l/32) + 0..3 of W-subtile j per register group g) -> sc (scaling)
// -> (GELU) -> fp32 or bf16 into the per-wave LDS band, then row-contiguous
// stores (and the fused amax).  The caller guarantees that no other wave
// still reads this wave's band region.
template <int OUT, int EPI, class AccV, class Scale>
__device__ __forceinline__ void band_epilogue(AccV (&acc)[4][4], Scale &sc, uint8_t *lds, int64_t M,
                                              int64_t N, int64_t m0, int64_t n0, int wave, int wm,
                                              int wn, int lane, void *y, float *slot) {
    constexpr int ES = OUT == 1 ? 2 : 4;
    constexpr bool AMAX = (EPI & kEpiAmax) != 0;
    static_assert(!AMAX || OUT == 1, "the fused amax needs bf16 output");
    using Band = EpiBand<ES>;
    const int lm = lane & 31, lh = lane >> 5;
    uint8_t *band = lds + wave * Band::BYTES;
    const bool vec = ((N * ES) & 15) == 0;
    float amax = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
        for (int ii = 0; ii < 2; ii++) {
            const int i = 2 * h + ii;
            sc.row(m0 + wm * 128 + i * 32 + lm);
#pragma unroll
            for (int j = 0; j < 4; j++) {
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    uint8_t *dst = band + (ii * 32 + lm) * Band::STRIDE + (j * 32 + 8 * g + 4 * lh) * ES;
                    float v4[4];
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        v4[e] = sc((float)acc[i][j][4 * g + e], j, g, e);
                    if constexpr (OUT == 0)
                        *reinterpret_cast<float4 *>(dst) = make_float4(v4[0], v4[1], v4[2], v4[3]);
                    else
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(cvt_pk_bf16(v4[0], v4[1]), cvt_pk_bf16(v4[2], v4[3]));
                }
            }
        }
        amax = fmaxf(amax, epi_band_to_global<ES, EPI>(band, y, M, N, m0 + wm * 128 + h * 64,
                                                        n0 + wn * 128, lane, vec));
    }
    if constexpr (AMAX) epi_tile_amax(amax, wave, lane, slot);
}

// Dynamic LDS of a GEMM kernel whose main loop takes `bytes` (the INT8 scales
// lie after them, without the adapter term and with it).
constexpr int kLoraMetaOff = kLoraLds + 2048;
template <int EPI>
constexpr size_t epi_lds(size_t bytes) {
    constexpr size_t bands = (EPI & kEpiLinear) != 0 ? 8 * kLoraBandBytes : 0;  // 4 of 64 rows
    return (EPI & kEpiLora) != 0 ? (size_t)kLoraMetaOff + kLoraMeta : bytes > bands ? bytes : bands;
}

// The epilogue with the adapter term: as band_epilogue, but in slices of 32
// rows through fp32 bands, to which the adapters' products are added before
// GELU, the amax and the rounding.  lds: kLoraLds bytes, and at kLoraMetaOff
// the words that lora_meta_dma copied before the main loop.
template <int OUT, int EPI, int AHEAD, class AccV, class Scale>
__device__ __forceinline__ void lora_epilogue(AccV (&acc)[4][4], Scale &sc, uint8_t *lds, int64_t M, int64_t N,
                                              int64_t m0, int64_t n0, int wave, int wm, int wn, int lane, void *y,
                                              float *slot, const LoraEpi &lora) {
    constexpr int ES = OUT == 1 ? 2 : 4;
    const int lm = lane & 31, lh = lane >> 5;
    uint8_t *band = lds + wave * kLoraBandBytes;
    const bool vec = ((N * ES) & 15) == 0;
    LoraRows<AHEAD> t;
    LoraTile T = lora_tile_begin(lora, m0, n0, N, lds, lds + kLoraMetaOff, t);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        sc.row(m0 + wm * 128 + i * 32 + lm);
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int g = 0; g < 4; g++)
                *reinterpret_cast<float4 *>(band + lm * kLoraBandStride + (j * 32 + 8 * g + 4 * lh) * 4) = make_float4(
                    sc((float)acc[i][j][4 * g], j, g, 0), sc((float)acc[i][j][4 * g + 1], j, g, 1),
                    sc((float)acc[i][j][4 * g + 2], j, g, 2), sc((float)acc[i][j][4 * g + 3], j, g, 3));
        LoraRows<AHEAD> next;
        if (i < 3) T.load_t(lora, i + 1, next);
        lora_band_add<AHEAD>(lora, T, i, n0, N, lds, t);
        if (i < 3) t = next;
        amax = fmaxf(amax, epi_band_to_global<ES, EPI, 32, true>(band, y, M, N, m0 + wm * 128 + i * 32,
                                                                 n0 + wn * 128, lane, vec));
        __builtin_amdgcn_sched_barrier(0);  // one slice at a time: its accumulators are free now
    }
    if constexpr ((EPI & kEpiAmax) != 0) epi_tile_amax(amax, wave, lane, slot);
}

// The epilogue of the whole linear: fp32 bands of 64 rows (32 with adapters, as
// lora_epilogue and with it), bias to store row by row.  A wave's band is its own,
// so nothing waits for other waves unless b of an adapter is staged.
template <int OUT, int EPI, int AHEAD, class AccV, class Scale>
__device__ __forceinline__ void linear_band_epilogue(AccV (&acc)[4][4], Scale &sc, uint8_t *lds, int64_t M, int64_t N,
                                                     int64_t m0, int64_t n0, int wave, int wm, int wn, int lane, void *y,
                                                     float *slot, const LinearEpi &L) {
    constexpr int ES = OUT == 1 ? 2 : 4, PER = 16 / ES;
    constexpr bool LORA = (EPI & kEpiLora) != 0;
    constexpr int SLICES = LORA ? 1 : 2;  // of 32 rows a band
    const int lm = lane & 31, lh = lane >> 5;
    uint8_t *band = lds + wave * SLICES * kLoraBandBytes;
    const bool vec = ((N * ES) & 15) == 0;
    const int64_t row0 = m0 + __builtin_amdgcn_readfirstlane(wm) * 128, col0 = n0 + __builtin_amdgcn_readfirstlane(wn) * 128;
    const int64_t col = col0 + (lane % (128 / PER)) * PER;
    LinearLane<PER> T;
    T.begin(L, row0, 128, M, N, col);
    QkLane<PER> Q;
    if constexpr ((EPI & kEpiHeads) != 0) Q.begin(L.qk, col);
    LoraRows<LORA ? AHEAD : 1> t;
    LoraTile A;
    if constexpr (LORA) A = lora_tile_begin(L.lora, m0, n0, N, lds, lds + kLoraMetaOff, t);
    float amax = 0.0f;
    auto one = [&](auto number) __attribute__((always_inline)) {
        constexpr int h = decltype(number)::value;
        uint4 residual[4];
        linear_residual<ES>(L, M, N, row0 + 32 * SLICES * h, col0, lane, vec, 32 * SLICES, residual);
#pragma unroll
        for (int ii = 0; ii < SLICES; ii++) {
            const int i = SLICES * h + ii;
            sc.row(m0 + wm * 128 + i * 32 + lm);
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int g = 0; g < 4; g++)
                    *reinterpret_cast<float4 *>(band + (32 * ii + lm) * kLoraBandStride + (j * 32 + 8 * g + 4 * lh) * 4) =
                        make_float4(sc((float)acc[i][j][4 * g], j, g, 0), sc((float)acc[i][j][4 * g + 1], j, g, 1),
                                    sc((float)acc[i][j][4 * g + 2], j, g, 2), sc((float)acc[i][j][4 * g + 3], j, g, 3));
        }
        if constexpr (LORA) {
            LoraRows<AHEAD> next;
            if (h < 3) A.load_t(L.lora, h + 1, next);
            lora_band_add<AHEAD>(L.lora, A, h, n0, N, lds, t);
            if (h < 3) t = next;
        }
        amax = fmaxf(amax, linear_band_out<ES, EPI, 32 * SLICES>(band, y, M, N, row0 + 32 * SLICES * h, col0, lane, vec, L, T, Q,
                                                                     residual));
        __builtin_amdgcn_sched_barrier(0);  // one band at a time: its accumulators are free now
    };
    // written out: as a loop that is not unrolled the accumulators would live in memory
    one(std::integral_constant<int, 0>()), one(std::integral_constant<int, 1>());
    if constexpr (LORA) one(std::integral_constant<int, 2>()), one(std::integral_constant<int, 3>());
    if constexpr ((EPI & kEpiAmax) != 0) epi_tile_amax(amax, wave, lane, slot);
}

// ---- the heads of a QKV linear from registers ------------------------------------------
// The accumulators are transposed: lane (row lm, half lh) has columns 8 g + 4 lh ..
// + 3 of register group g.  Swapping the upper half of group 2 q with the lower
// one of group 2 q + 1 gives every lane 8 consecutive columns of its row, 16 p +
// 8 lh with p = 2 j + q.  Two lanes then hold a row's head, so that its sums take
// one exchange, where 8 lanes that read it from a band take three for each sum
// (17776 x 1920 x 5760, NVFP4: 506 us through bands, 398 from registers).  The
// columns' parameters are in LDS, the wave's own.
template <class AccV>
__device__ __forceinline__ void acc_row8(const AccV &a, int q, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float lo = (float)a[8 * q + e], hi = (float)a[8 * q + 4 + e];
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(lo), __float_as_uint(hi), false, false);
        v[e] = __uint_as_float(r[0]);
        v[4 + e] = __uint_as_float(r[1]);
    }
}

// The wave's column parameters in LDS: bias, the heads' w and b, each of 128.
constexpr int kColParams = 3 * 128;
struct ColParams {
    const float *p;  // the lane's, columns 8 lh ..
    __device__ __forceinline__ void get(int which, int at, float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 u = *reinterpret_cast<const float4 *>(p + which * 128 + at + i);
            v[i] = u.x, v[i + 1] = u.y, v[i + 2] = u.z, v[i + 3] = u.w;
        }
    }
};

// The heads of 128 columns (16 p + 8 lh .. of row lm a lane): a head of D columns is
// NP = D / 16 eights of a lane and as many of its partner's in the other half, so
// its sums are in the lane but for one exchange, and both members of a rotated
// pair are the lane's own (2 P = D, or nothing is rotated).  The results of 32 rows go out through
// the wave's bf16 band, whole rows a store: partial lines are slow.
template <int D, bool PRE, class Get, class Cols>
__device__ __forceinline__ void linear_heads_out(Get &&get, Cols &&cols, const ColParams &C, void *y, int64_t M, int64_t N,
                                                 int64_t row0, int64_t col0, int lm, int lh, uint8_t *band, const LinearEpi &L) {
    constexpr int NP = D / 16, HEADS = 128 / D;
    const QkHeads &H = L.qk;
    const float inv = 1.0f / (float)D;
    const int h0 = (int)(col0 / D);
    uint8_t *mine_at = band + lm * EpiBand<2>::STRIDE + 16 * lh;
    // The row's turns of the lane's pairs, two at a time: neighbours, 4 of each eight;
    // halves, 8 of each eight of the first half.  They come a slice ahead.
    float4 z[NP][2];
    auto turns = [&](int i) __attribute__((always_inline)) {
        if (PRE || H.P == 0 || h0 >= H.nq + H.nk) return;
        const int64_t row = row0 + 32 * i + lm < M ? row0 + 32 * i + lm : M - 1;
        const float2 *t = reinterpret_cast<const float2 *>(H.table) + row * H.P;
#pragma unroll
        for (int p = 0; p < NP; p++)
#pragma unroll
            for (int e = 0; e < 2; e++)
                z[p][e] = *reinterpret_cast<const float4 *>(
                    t + (H.layout == 0 ? 8 * p + 4 * lh + 2 * e : 16 * (p >> 1) + 8 * lh + 4 * (p & 1) + 2 * e));
    };
    turns(0);
#pragma unroll
    for (int i = 0; i < 4; i++) {
#pragma unroll
        for (int hh = 0; hh < HEADS; hh++) {
            const bool mine = h0 + hh < H.nq + H.nk;  // wave-uniform
            float x[NP][8];
            auto out = [&](int p) __attribute__((always_inline)) {
                *reinterpret_cast<uint4 *>(mine_at + 32 * (NP * hh + p)) =
                    make_uint4(cvt_pk_bf16(x[p][0], x[p][1]), cvt_pk_bf16(x[p][2], x[p][3]), cvt_pk_bf16(x[p][4], x[p][5]),
                               cvt_pk_bf16(x[p][6], x[p][7]));
            };
#pragma unroll
            for (int p = 0; p < NP; p++) {
                float bias[8];
                cols(16 * (NP * hh + p));
                get(i, NP * hh + p, x[p]);
                C.get(0, D * hh + 16 * p, bias);
#pragma unroll
                for (int e = 0; e < 8; e++) x[p][e] += bias[e];
            }
            if (PRE) {
#pragma unroll
                for (int p = 0; p < NP; p++) out(p);
                continue;
            }
            if (mine && H.norm != 0) {
                if (H.norm == 2) {
                    float s = 0.0f;
#pragma unroll
                    for (int p = 0; p < NP; p++)
#pragma unroll
                        for (int e = 0; e < 8; e++) s += x[p][e];
                    s = (s + other_half(s)) * inv;
#pragma unroll
                    for (int p = 0; p < NP; p++)
#pragma unroll
                        for (int e = 0; e < 8; e++) x[p][e] -= s;
                }
                float s = 0.0f;
#pragma unroll
                for (int p = 0; p < NP; p++)
#pragma unroll
                    for (int e = 0; e < 8; e++) s = __builtin_fmaf(x[p][e], x[p][e], s);
                s += other_half(s);
                const float r = rsqrt_f32(__builtin_fmaf(s, inv, H.eps));
#pragma unroll
                for (int p = 0; p < NP; p++) {
                    float w[8], b[8];
                    C.get(1, D * hh + 16 * p, w);
                    C.get(2, D * hh + 16 * p, b);
#pragma unroll
                    for (int e = 0; e < 8; e++) x[p][e] = __builtin_fmaf(x[p][e] * r, w[e], b[e]);
                }
            }
            if (mine && H.P > 0) {
                if (H.layout == 0) {
#pragma unroll
                    for (int p = 0; p < NP; p++)
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const float4 f = z[p][e >> 1];
                            const float cs = e & 1 ? f.z : f.x, sn = e & 1 ? f.w : f.y;
                            const float a = x[p][2 * e], b = x[p][2 * e + 1];
                            x[p][2 * e] = a * cs - b * sn;
                            x[p][2 * e + 1] = b * cs + a * sn;
                        }
                } else {
#pragma unroll
                    for (int p = 0; p < NP / 2; p++)
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const float4 f = z[2 * p + (e >> 2)][e >> 1 & 1];
                            const float cs = e & 1 ? f.z : f.x, sn = e & 1 ? f.w : f.y;
                            const float a = x[p][e], b = x[p + NP / 2][e];
                            x[p][e] = a * cs - b * sn;
                            x[p + NP / 2][e] = b * cs + a * sn;
                        }
                }
            }
#pragma unroll
            for (int p = 0; p < NP; p++) out(p);
        }
        if (i < 3) turns(i + 1);
        epi_band_to_global<2, 0, 32>(band, PRE ? L.pre : y, M, N, row0 + 32 * i, col0, 32 * lh + lm, true);
        __builtin_amdgcn_sched_barrier(0);  // one row's heads at a time
    }
}

// Output scalings for it: cols(at) before 8 columns, then each value of slice i,
// column e of them.
struct RegScaleF32 {
    float gA, gW;
    __device__ __forceinline__ void cols(int) {}
    __device__ __forceinline__ float operator()(float a, int, int) const { return (a * gA) * gW; }
};

// The epilogue of a QKV tile.  lds: 16 * kColParams bytes and four bf16 bands.
template <class AccV, class Scale>
__device__ __forceinline__ void linear_heads_epilogue(AccV (&acc)[4][4], Scale &sc, uint8_t *lds, int64_t M, int64_t N,
                                                      int64_t m0, int64_t n0, int wave, int wm, int wn, int lane, void *y,
                                                      const LinearEpi &L) {
    const int64_t row0 = m0 + __builtin_amdgcn_readfirstlane(wm) * 128, col0 = n0 + __builtin_amdgcn_readfirstlane(wn) * 128;
    // two columns a lane into the wave's LDS
    LinearLane<2> T;
    T.begin(L, row0, 128, M, N, col0 + 2 * lane);
    QkLane<2> Q;
    Q.begin(L.qk, col0 + 2 * lane);
    float *params = reinterpret_cast<float *>(lds) + wave * kColParams;
    const int lm = lane & 31, lh = lane >> 5;
    const ColParams P{params + 8 * lh};
    *reinterpret_cast<float2 *>(params + 2 * lane) = make_float2(T.bias[0], T.bias[1]);
    *reinterpret_cast<float2 *>(params + 128 + 2 * lane) = make_float2(Q.w[0], Q.w[1]);
    *reinterpret_cast<float2 *>(params + 256 + 2 * lane) = make_float2(Q.b[0], Q.b[1]);
    auto get = [&](int i, int p, float (&v)[8]) __attribute__((always_inline)) {
        acc_row8(acc[i][p >> 1], p & 1, v);
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] = sc(v[e], i, e);
    };
    auto cols = [&](int at) __attribute__((always_inline)) { sc.cols(at); };
    uint8_t *band = lds + 16 * kColParams + wave * 32 * EpiBand<2>::STRIDE;
    // (with pre the accumulators are read twice: both at once would not fit the registers)
    if (L.qk.D == 64) {
        if (L.pre) linear_heads_out<64, true>(get, cols, P, y, M, N, row0, col0, lm, lh, band, L);
        linear_heads_out<64, false>(get, cols, P, y, M, N, row0, col0, lm, lh, band, L);
    } else {
        if (L.pre) linear_heads_out<128, true>(get, cols, P, y, M, N, row0, col0, lm, lh, band, L);
        linear_heads_out<128, false>(get, cols, P, y, M, N, row0, col0, lm, lh, band, L);
    }
}

// fp32 accumulators -> y = (acc * gA) * gW (fp32 or bf16).  slot: the tile's
// entry of the fused-amax maxima (used with kEpiAmax only).
template <int OUT, int EPI = 0>
__device__ __forceinline__ void f32_band_epilogue(v16f (&acc)[4][4], uint8_t *lds, float gA,
                                                  float gW, int64_t M, int64_t N, int64_t m0,
                                                  int64_t n0, int wave, int wm, int wn, int lane,
                                                  void *y, float *slot, const EpiArg<EPI> &ep) {
    if constexpr ((EPI & kEpiLinear) != 0) {
        if constexpr (heads_in_regs(EPI)) {
            RegScaleF32 sc{gA, gW};
            linear_heads_epilogue(acc, sc, lds, M, N, m0, n0, wave, wm, wn, lane, y, ep);
        } else {
            EpiScaleF32 sc{gA, gW};
            linear_band_epilogue<OUT, EPI, 3>(acc, sc, lds, M, N, m0, n0, wave, wm, wn, lane, y, slot, ep);
        }
    } else if constexpr ((EPI & kEpiLora) != 0) {
        EpiScaleF32 sc{gA, gW};
        lora_epilogue<OUT, EPI, 3>(acc, sc, lds, M, N, m0, n0, wave, wm, wn, lane, y, slot, ep);
    } else {
        EpiScaleF32 sc{gA, gW};
        band_epilogue<OUT, EPI>(acc, sc, lds, M, N, m0, n0, wave, wm, wn, lane, y, slot);
    }
}

// The epilogue of one 32-row slice i of a 128 x 128 quadrant of a split
// tile, run by a one-wave workgroup straight from the tile's partials (no
// accumulator array: a register-resident tile plus the loads in flight would
// spill).  A tail of T tiles so gets 16 T waves, enough to keep the partial
// reads in flight on every CU.  For each MFMA block (i, j), the lane's four
// 16-byte pieces of all S splits are loaded together, added in split order
// as T (int32: exact; fp32: fixed order), scaled by sc and written to a
// 32-row band, which then goes out as in band_epilogue.  part: the tile's
// first split; wave: the quadrant (the wave of the whole-tile kernels whose
// lanes' layout the partials follow).  The fused amax goes to *slot by an
// atomic max (the split kernel zeroed it; the maximum does not depend on the
// order).
constexpr int kFixupRows = 32;
// its LDS: a band of outputs, or of fp32 values where the whole linear's
// epilogue reads it
template <int OUT, int EPI>
constexpr size_t fixup_lds() {
    return (size_t)kFixupRows * ((EPI & kEpiLinear) != 0 ? kLoraBandStride : EpiBand<OUT == 1 ? 2 : 4>::STRIDE);
}

template <int OUT, int EPI, class T, int S, class Scale>
__device__ __forceinline__ void split_fixup_epilogue(const uint32_t *part, Scale &sc, uint8_t *lds,
                                                     int64_t M, int64_t N, int64_t m0, int64_t n0,
                                                     int wave, int i, int lane, void *y, float *slot,
                                                     const EpiArg<EPI> &ep) {
    constexpr int ES = OUT == 1 ? 2 : 4;
    constexpr bool LORA = (EPI & kEpiLora) != 0, LINEAR = (EPI & kEpiLinear) != 0;
    using Band = EpiBand<ES>;
    constexpr size_t kPieces = kSplitWords / 4;
    const uint4 *p4 = reinterpret_cast<const uint4 *>(part);
    const int wm = wave >> 1, wn = wave & 1, tid = wave * 64 + lane;
    const int lm = lane & 31, lh = lane >> 5;
    uint8_t *band = lds;
    const bool vec = ((N * ES) & 15) == 0;
    sc.row(m0 + wm * 128 + i * 32 + lm);
    v16f add[4];
    if constexpr (LORA) lora_slice(lora_of(ep), m0 + wm * 128 + i * 32 + lm, n0 + wn * 128, N, lane, add);
#pragma unroll
    for (int j = 0; j < 4; j++) {
        uint4 v[S][4];
#pragma unroll
        for (int s = 0; s < S; s++)
#pragma unroll
            for (int g = 0; g < 4; g++) v[s][g] = p4[s * kPieces + ((i * 4 + j) * 4 + g) * 256 + tid];
#pragma unroll
        for (int g = 0; g < 4; g++) {
            T x[4] = {__builtin_bit_cast(T, v[0][g].x), __builtin_bit_cast(T, v[0][g].y),
                      __builtin_bit_cast(T, v[0][g].z), __builtin_bit_cast(T, v[0][g].w)};
#pragma unroll
            for (int s = 1; s < S; s++) {
                x[0] += __builtin_bit_cast(T, v[s][g].x);
                x[1] += __builtin_bit_cast(T, v[s][g].y);
                x[2] += __builtin_bit_cast(T, v[s][g].z);
                x[3] += __builtin_bit_cast(T, v[s][g].w);
            }
            float v4[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                v4[e] = sc((float)x[e], j, g, e);
                if constexpr (LORA) v4[e] += add[j][4 * g + e];
            }
            constexpr int STRIDE = LINEAR ? kLoraBandStride : Band::STRIDE, BES = LINEAR ? 4 : ES;
            uint8_t *dst = band + lm * STRIDE + (j * 32 + 8 * g + 4 * lh) * BES;
            if constexpr (OUT == 0 || LINEAR)
                *reinterpret_cast<float4 *>(dst) = make_float4(v4[0], v4[1], v4[2], v4[3]);
            else
                *reinterpret_cast<uint2 *>(dst) = make_uint2(cvt_pk_bf16(v4[0], v4[1]), cvt_pk_bf16(v4[2], v4[3]));
        }
        // bound the loads in flight (one block's, two for few splits)
        if (S > 4 || (j & 1)) __builtin_amdgcn_sched_barrier(0);
    }
    float amax;
    if constexpr (LINEAR) {
        constexpr int PER = 16 / ES;
        const int64_t row0 = m0 + wm * 128 + i * 32, col = n0 + wn * 128 + (lane % (128 / PER)) * PER;
        LinearLane<PER> cols;
        cols.begin(ep, row0, kFixupRows, M, N, col);
        QkLane<PER> Q;
        if constexpr ((EPI & kEpiHeads) != 0) Q.begin(ep.qk, col);
        uint4 residual[4];
        linear_residual<ES>(ep, M, N, row0, n0 + wn * 128, lane, vec, kFixupRows, residual);
        amax = linear_band_out<ES, EPI, kFixupRows>(band, y, M, N, row0, n0 + wn * 128, lane, vec, ep, cols, Q, residual);
    } else {
        amax = epi_band_to_global<ES, EPI, kFixupRows>(band, y, M, N, m0 + wm * 128 + i * 32, n0 + wn * 128, lane, vec);
    }
    if constexpr ((EPI & kEpiAmax) != 0) {
        // non-negative floats order as their bit patterns
        amax = wave_max(amax);
        if (lane == 0) atomicMax(reinterpret_cast<unsigned *>(slot), __float_as_uint(amax));
    }
}

// Host: the fixup launch of a form (fp32 accumulators).
template <int OUT, int EPI>
inline hipError_t launch_fixup_of(hipStream_t s, const float *ga, const float *gw, int64_t M, int64_t N, void *y,
                                  unsigned tiles_m, unsigned tiles_n, unsigned group_m, float *partial,
                                  const SplitPlan &sp, const uint32_t *spart, const EpiArg<EPI> &ep) {
    if constexpr ((EPI & kEpiLinear) != 0)
        return launch_f32_fixup_linear(s, ga, gw, M, N, y, tiles_m, tiles_n, group_m, partial, sp, spart, OUT, EPI, ep);
    else
        return launch_f32_fixup(s, ga, gw, M, N, y, tiles_m, tiles_n, group_m, partial, sp, spart, OUT, EPI, &ep);
}

}  // namespace dmpq
