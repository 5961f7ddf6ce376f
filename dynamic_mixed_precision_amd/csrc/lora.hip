// lora.hip -- low-rank adapters of many requests beside a shared projection,
// and their gradients.  Request i adds scale_i (x a_i^T) b_i^T to the rows of
// the frozen projection that are its own; a is [R x K], b is [N x R].
//
//   shrink   t = x a^T               [M x R] fp32
//   expand   y = base + scale t b^T  [M x N] bf16 or fp32
//   backward u = scale dy b, dx = dx_base + u a, da = u^T x, db = scale dy^T t
//
// Every product has one dimension of at most 128, so all of them are bound by
// the passes over their widest tensor: one, but two over dy in the backward
// pass (u needs whole rows of it, db whole columns).  MFMA does the products: x,
// dy, a and b are bf16 and exact in it; t and u are fp32 and enter as 3 bf16
// parts that hold all their bits (split8).  Sums are fp32 in a fixed order: no
// atomics, the same bits on every call.
#include <type_traits>

#include "device.hpp"
#include "gemm_common.hpp"
#include "gemm_dma.hpp"
#include "internal.hpp"
#include "lora.hpp"

namespace dmpq {

namespace {

// t and u as the gradients' products read them: 3 bf16 parts, for each 32 rows
// and 16 ranks the 64 lanes' 16-byte pieces of a 16x16x32 MFMA operand (lane
// c + 16 q: rank c, rows 8 q .. 8 q + 7) one after the other, so that a
// fragment is one contiguous load.  The place of rank j of row m in part p:
__device__ __forceinline__ int64_t packed_at(int m, int p, int j, int R) {
    return ((((int64_t)(m >> 5) * 3 + p) * (R >> 4) + (j >> 4)) * 64 + ((m >> 3) & 3) * 16 + (j & 15)) * 8 + (m & 7);
}

__device__ __forceinline__ v4i ld16(const void *p) { return *reinterpret_cast<const v4i *>(p); }

// ---------------------------------------------------------------------------
// Shrink: t[m, j] = sum_k x[m, k] a[j, k] for `tile` <= 16 RT rows of one
// request and 16 RC of its ranks (part blockIdx.y).  The WAVES waves share K
// in stages of 64: a wave loads whole 128-byte lines (8 lanes a row) of its
// own stages, two stages ahead in registers, passes them through an LDS area
// of its own (no barrier) and reads them back as 16x16x32 MFMA fragments.
// Loading the fragments straight from memory, where neighbouring lanes hold
// different rows, ran at 1.9 TB/s however many loads were in flight.  The
// waves' sums meet in LDS at the end, added in wave order.  UP: the same
// product for u = scale dy b (x is dy, a the transposed b), stored times
// scale, and once more packed for the gradients' products over the rows.
// ---------------------------------------------------------------------------

template <int RT, int RC, int WAVES, bool UP>
__global__ __launch_bounds__(64 * WAVES) void lora_shrink_kernel(const uint16_t *__restrict__ x,
                                                                 const uint16_t *__restrict__ a, LoraBatch B,
                                                                 int64_t K, int tile, unsigned first,
                                                                 float *__restrict__ t,
                                                                 uint16_t *__restrict__ packed) {
    constexpr int TM = 16 * RT, TJ = 16 * RC, ROWS = TM + TJ, LOADS = ROWS / 8;
    constexpr int STRIDE = TJ + 4;  // of the sums
    constexpr int STAGE = ROWS * 128, SUMS = TM * STRIDE * 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[WAVES * (STAGE > SUMS ? STAGE : SUMS)];
    SegTile st;
    if (!seg_tile(B, (int)(first + blockIdx.x), tile, st)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j0 = blockIdx.y * TJ;
    const int rank = st.adapter < 0 ? 0 : adapter_rank(B, st.adapter);
    float *part = reinterpret_cast<float *>(lds);
    if (rank > j0) {  // workgroup-uniform
        const int c = lane & 15, q = lane >> 4;
        const int lr = lane >> 3, lc = lane & 7;  // the lane's row of 8 and its 16-byte piece of a stage
        const uint16_t *src[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; i++) {
            const int r = 8 * i + lr;
            if (r < TM) {
                src[i] = x + (int64_t)(st.row0 + (r < st.rows ? r : st.rows - 1)) * K + 8 * lc;
            } else {
                const int jj = j0 + r - TM;
                src[i] = a + ((int64_t)st.adapter * B.R + (jj < B.R ? jj : B.R - 1)) * K + 8 * lc;
            }
        }
        v4f acc[RT][RC];
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int k = 0; k < RC; k++) acc[i][k] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
        const int stages = (int)((K + 63) / 64);
        uint8_t *own = lds + wave * STAGE;
        // a piece past K (the last stage of a K that is no multiple of 64) is
        // loaded from the stage's first piece and written as zeros
        auto load = [&](v4i(&v)[LOADS], int s) {
            const int64_t o = 64 * (int64_t)s - (64 * (int64_t)s + 8 * lc < K ? 0 : 8 * lc);
#pragma unroll
            for (int i = 0; i < LOADS; i++) v[i] = ld16(src[i] + o);
        };
        auto use = [&](v4i(&v)[LOADS], int s) {
            const bool in = 64 * (int64_t)s + 8 * lc < K;
#pragma unroll
            for (int i = 0; i < LOADS; i++)
                *reinterpret_cast<v4i *>(own + (8 * i + lr) * 128 + swz128(8 * i + lr, lc) * 16) =
                    in ? v[i] : (v4i){0, 0, 0, 0};
        };
        auto mul = [&]() {
#pragma unroll
            for (int u = 0; u < 2; u++) {
                v4i xf[RT], af[RC];
#pragma unroll
                for (int i = 0; i < RT; i++)
                    xf[i] = *reinterpret_cast<const v4i *>(own + (16 * i + c) * 128 + swz128(c, 4 * u + q) * 16);
#pragma unroll
                for (int k = 0; k < RC; k++)
                    af[k] = *reinterpret_cast<const v4i *>(own + (TM + 16 * k + c) * 128 + swz128(c, 4 * u + q) * 16);
#pragma unroll
                for (int i = 0; i < RT; i++)
#pragma unroll
                    for (int k = 0; k < RC; k++) acc[i][k] = mfma16(af[k], xf[i], acc[i][k]);
            }
        };
        v4i va[LOADS], vb[LOADS];
        // every WAVES-th stage: at a time the workgroup reads WAVES neighbouring
        // lines of each row
        if (wave < stages) load(va, wave);
        if (wave + WAVES < stages) load(vb, wave + WAVES);
        for (int s = wave; s < stages; s += 2 * WAVES) {
            use(va, s);
            if (s + 2 * WAVES < stages) load(va, s + 2 * WAVES);
            mul();
            if (s + WAVES < stages) {
                use(vb, s + WAVES);
                if (s + 3 * WAVES < stages) load(vb, s + 3 * WAVES);
                mul();
            }
        }
        __syncthreads();  // the stages' LDS becomes the sums'
        // D: lane column = token, registers = 4 consecutive ranks
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int k = 0; k < RC; k++)
                *reinterpret_cast<v4f *>(part + (wave * TM + 16 * i + c) * STRIDE + 16 * k + 4 * q) = acc[i][k];
    }
    __syncthreads();
    const float sc = UP && st.adapter >= 0 ? B.scale[st.adapter] : 1.0f;
    for (int e = threadIdx.x; e < TM * TJ; e += 64 * WAVES) {
        // UP: lanes along the rows, as the parts are stored
        const int r = UP ? e % TM : e / TJ, j = UP ? e / TM : e % TJ;
        if (r >= st.rows || j0 + j >= B.R) continue;
        float v = 0.0f;
        if (j0 + j < rank) {
            v = part[r * STRIDE + j];
#pragma unroll
            for (int w = 1; w < WAVES; w++) v += part[(w * TM + r) * STRIDE + j];
            v *= sc;
        }
        t[(int64_t)(st.row0 + r) * B.R + j0 + j] = v;
        if constexpr (UP) {
            float rest = v;  // as split8
#pragma unroll
            for (int p = 0; p < kParts; p++) {
                packed[packed_at(st.row0 + r, p, j0 + j, B.R)] = (uint16_t)(__float_as_uint(rest) >> 16);
                rest = split_rest(p == 0 ? split_finite(rest) : rest);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Expand: y = base + scale t b^T for 128 rows of one request, 32 to each wave,
// and 128 columns.  A workgroup does one such block and ends: base and y are
// all the traffic, and a wave that goes on to another block waits for its
// stores before the next loads (one counter holds both), which a copy of the
// same shape showed to cost a quarter to a third (5.0 TB/s against 3.8 with
// four blocks a workgroup, at 17776 x 12288 bf16).  Neighbouring workgroups
// take neighbouring columns (rows first: 4.5 TB/s).  The block's b, one
// contiguous piece of memory, goes through registers into LDS, entries past
// the rank as zeros.  t, in bf16 parts, is the 32x32x16 MFMA's first operand,
// so a lane's 16 accumulators are 16 rows of one column; the second operand of
// MFMA p holds b's rows n0 + 4 i + p for lanes i, so the four MFMAs leave every
// lane four consecutive columns of those rows, and base and y move in 8- or
// 16-byte pieces, 32 lanes a row, straight between memory and registers.
// ---------------------------------------------------------------------------
constexpr int kExpandRows = 128, kExpandCols = 128, kExpandWaves = 4;

// Four values of base or y.  Rows of an odd N start anywhere, so the accesses
// ask for no more than the value's own alignment (the hardware takes them).
template <int ES>
struct Quad {
    typedef uint32_t V __attribute__((ext_vector_type(ES), aligned(ES)));
    V v;
    static __device__ __forceinline__ Quad load(const uint8_t *p) {
        return Quad{__builtin_nontemporal_load(reinterpret_cast<const V *>(p))};
    }
    __device__ __forceinline__ void store(uint8_t *p) const { __builtin_nontemporal_store(v, reinterpret_cast<V *>(p)); }
    // the first n < 4 values
    static __device__ __forceinline__ Quad load_some(const uint8_t *p, int n) {
        Quad q = zero();
        if constexpr (ES == 2) {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
            q.v[0] = h[0] | (n > 1 ? (uint32_t)h[1] << 16 : 0u);
            if (n > 2) q.v[1] = h[2];
        } else {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(p);
            q.v[0] = w[0];
            if (n > 1) q.v[1] = w[1];
            if (n > 2) q.v[2] = w[2];
        }
        return q;
    }
    __device__ __forceinline__ void store_some(uint8_t *p, int n) const {
        if constexpr (ES == 2) {
            uint16_t *h = reinterpret_cast<uint16_t *>(p);
            h[0] = (uint16_t)v[0];
            if (n > 1) h[1] = (uint16_t)(v[0] >> 16);
            if (n > 2) h[2] = (uint16_t)v[1];
        } else {
            uint32_t *w = reinterpret_cast<uint32_t *>(p);
            w[0] = v[0];
            if (n > 1) w[1] = v[1];
            if (n > 2) w[2] = v[2];
        }
    }
    static __device__ __forceinline__ Quad zero() {
        Quad q;
#pragma unroll
        for (int e = 0; e < ES; e++) q.v[e] = 0u;
        return q;
    }
    __device__ __forceinline__ Quad plus(float sc, float d0, float d1, float d2, float d3) const {
        Quad q;
        if constexpr (ES == 2) {
            q.v[0] = cvt_pk_bf16(bf16_lo(v[0]) + sc * d0, bf16_hi(v[0]) + sc * d1);
            q.v[1] = cvt_pk_bf16(bf16_lo(v[1]) + sc * d2, bf16_hi(v[1]) + sc * d3);
        } else {
            q.v[0] = __float_as_uint(__uint_as_float(v[0]) + sc * d0);
            q.v[1] = __float_as_uint(__uint_as_float(v[1]) + sc * d1);
            q.v[2] = __float_as_uint(__uint_as_float(v[2]) + sc * d2);
            q.v[3] = __float_as_uint(__uint_as_float(v[3]) + sc * d3);
        }
        return q;
    }
};

template <int ES, int RC>
__global__ __launch_bounds__(64 * kExpandWaves, 2) void lora_expand_kernel(const float *__restrict__ t,
                                                                           const void *base,
                                                                           const uint16_t *__restrict__ b, LoraBatch B,
                                                                           int64_t N, unsigned cols, unsigned first,
                                                                           void *y) {
    // b's row 4 i + p of the block lies at LDS row 32 p + i; 16 bytes of
    // padding spread the lanes' 16-byte reads over the banks
    constexpr int ROW = 32 * RC + 16;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kExpandCols * ROW];
    constexpr int TROW = 16 * 4 + 16;  // 16 ranks of a row of t and padding
    __shared__ __attribute__((aligned(16))) uint8_t tlds[kExpandWaves][32 * TROW];
    __shared__ int odd_b[kExpandWaves];  // whether the b that a wave copied holds an infinity or NaN
    typedef Quad<ES> Q;
    const unsigned down = blockIdx.x / cols, cb = blockIdx.x - down * cols;
    SegTile st;
    if (!seg_tile(B, (int)(first + down), kExpandRows, st)) return;
    if (st.adapter < 0 && base == y) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 31, lh = lane >> 5;
    const int row0 = st.row0 + 32 * wave, wrows = st.rows - 32 * wave;  // this wave's; <= 0: none
    // row of accumulator r: 8 (r / 4) + r % 4 from a scalar base, + 4 lh and
    // the column in the lane's 32-bit offset (N <= 2^26)
    const int64_t ld = N * ES, coff = (int64_t)cb * kExpandCols * ES;
    const uint8_t *bp = static_cast<const uint8_t *>(base) + row0 * ld + coff;
    uint8_t *yp = static_cast<uint8_t *>(y) + row0 * ld + coff;
    const uint32_t lane_off = (uint32_t)(4 * lh * ld + 4 * li * ES);
    const int rows = wrows - 4 * lh;
    const int left = (int)(N - (int64_t)cb * kExpandCols) - 4 * li;  // the lane's columns
    Q bv[16];
#pragma unroll
    for (int r = 0; r < 16; r++) {
        const int m = 8 * (r >> 2) + (r & 3);
        bv[r] = Q::zero();
        if (base && m < rows && left > 0)
            bv[r] = left >= 4 ? Q::load(bp + m * ld + lane_off) : Q::load_some(bp + m * ld + lane_off, left);
    }
    // an adapter of rank 0 adds nothing, whatever its scale (alpha / rank: infinite)
    const int rank = st.adapter < 0 ? 0 : adapter_rank(B, st.adapter);
    v16f acc[4];
    float sc = 1.0f;
#pragma unroll
    for (int p = 0; p < 4; p++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[p][e] = 0.0f;
    if (rank > 0) {
        const int64_t bn = N * B.R;  // values of one adapter's b
        const uint16_t *bw = b + st.adapter * bn;
        v4i piece[RC];
#pragma unroll
        for (int k = 0; k < RC; k++) {
            const int64_t at = (int64_t)cb * kExpandCols * B.R + 8 * (tid + 256 * k);
            piece[k] = ld16(bw + (at < bn ? at : 0));  // past b: of columns past N
        }
        // t: 4 lanes a row (64 bytes), rows l / 4 and 16 + l / 4
        v4f tv[RC][2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int r = 32 * wave + 16 * h + (lane >> 2);
            const float *tr = t + (int64_t)(st.row0 + (r < st.rows ? r : st.rows - 1)) * B.R + 4 * (lane & 3);
#pragma unroll
            for (int c = 0; c < RC; c++) tv[c][h] = *reinterpret_cast<const v4f *>(tr + (16 * c < B.R ? 16 * c : 0));
        }
        if (B.scale) sc = B.scale[st.adapter];
        const int per_row = B.R / 8;  // 16-byte pieces of a row of b
        u16x2 top = {0, 0};
#pragma unroll
        for (int k = 0; k < RC; k++) {
            const int e = tid + 256 * k, n = e / per_row, c = e - n * per_row;
            piece[k] = keep8(piece[k], rank - 8 * c);
            if (n < kExpandCols) {
                *reinterpret_cast<v4i *>(lds + (32 * (n & 3) + (n >> 2)) * ROW + 16 * c) = piece[k];
                magnitudes8(piece[k], top);
            }
        }
        const uint64_t any = __ballot(nonfinite_in(top));
        if (lane == 0) odd_b[wave] = any != 0;
        if (__builtin_expect(any != 0, 0))
#pragma unroll
            for (int k = 0; k < RC; k++) {
                const int e = tid + 256 * k, n = e / per_row, c = e - n * per_row;
                if (n < kExpandCols)
                    *reinterpret_cast<v4i *>(lds + (32 * (n & 3) + (n >> 2)) * ROW + 16 * c) = ones8(piece[k]);
            }
        __syncthreads();
        if (wrows <= 0) return;
#pragma unroll
        for (int c = 0; c < RC; c++) {
            if (16 * c >= rank) break;  // workgroup-uniform
            // the wave turns its 16 ranks of t into fragments in its own LDS
            // (a wave's LDS operations keep their order)
            uint8_t *tw = tlds[wave];
#pragma unroll
            for (int h = 0; h < 2; h++)
                *reinterpret_cast<v4f *>(tw + (16 * h + (lane >> 2)) * TROW + 16 * (lane & 3)) = tv[c][h];
            const v4f a0 = *reinterpret_cast<const v4f *>(tw + li * TROW + 32 * lh);
            const v4f a1 = *reinterpret_cast<const v4f *>(tw + li * TROW + 32 * lh + 16);
            const float v[8] = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
            v4i tf[kParts], bf[4];
            split8(v, tf);
#pragma unroll
            for (int p = 0; p < 4; p++)
                bf[p] = *reinterpret_cast<const v4i *>(lds + (32 * p + li) * ROW + 32 * c + 16 * lh);
#pragma unroll
            for (int s = kParts - 1; s >= 0; s--)
#pragma unroll
                for (int p = 0; p < 4; p++) acc[p] = mfma32(tf[s], bf[p], acc[p]);
        }
        if (__builtin_expect(__builtin_amdgcn_readfirstlane(odd_b[0] | odd_b[1] | odd_b[2] | odd_b[3]), 0)) {
            // b's infinities and NaN, from memory
            const float *tr = t + (int64_t)(row0 + (li < wrows ? li : wrows - 1)) * B.R + 8 * lh;
            const int64_t n = (int64_t)cb * kExpandCols + 4 * li;
#pragma unroll 1
            for (int c = 0; c < rank; c += 16) {
                const v4f a0 = *reinterpret_cast<const v4f *>(tr + c), a1 = *reinterpret_cast<const v4f *>(tr + c + 4);
                const float v[8] = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
                const v4i sf = sign8(v);
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    const v4i f = ld16(bw + (n + p < N ? n + p : N - 1) * B.R + c + 8 * lh);
                    acc[p] = mfma32(sf, odd8(keep8(f, rank - c - 8 * lh)), acc[p]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 16; r++) {
        const int m = 8 * (r >> 2) + (r & 3);
        if (m >= rows || left <= 0) continue;
        // (base alone is copied, not added to: all bits of a NaN or -0 stay)
        const Q o = rank > 0 ? bv[r].plus(sc, acc[0][r], acc[1][r], acc[2][r], acc[3][r]) : bv[r];
        if (left >= 4)
            o.store(yp + m * ld + lane_off);
        else
            o.store_some(yp + m * ld + lane_off, left);
    }
}

// ---------------------------------------------------------------------------
// Backward, first launch: what the products over the other dimension need.
//   blocks 0 ..            b [N x R] -> bt [R x N], 64 x R tiles through LDS
//   then                   a [R x K] -> at [K x R]
//   then                   t [M x R] packed
// Entries past an adapter's rank become zeros.
// ---------------------------------------------------------------------------
struct PrepPlan {
    int nb, na;  // tiles of one adapter's b and a
};

__global__ __launch_bounds__(256) void lora_prep_kernel(const uint16_t *__restrict__ a, const uint16_t *__restrict__ b,
                                                        const float *__restrict__ t, LoraBatch B, int64_t N, int64_t K,
                                                        PrepPlan pl, unsigned first, uint16_t *__restrict__ at,
                                                        uint16_t *__restrict__ bt, uint16_t *__restrict__ tp) {
    __shared__ __attribute__((aligned(16))) uint16_t tile[64 * (kMaxLoraRank + 2)];
    int blk = (int)(first + blockIdx.x);
    const int tid = threadIdx.x, R = B.R;
    const int pieces = R / 8;
    // 8 values of 8 different rows of the tile, packed as one piece
    auto column = [&](int r, int j) {
        v4i o;
#pragma unroll
        for (int d = 0; d < 4; d++)
            o[d] = tile[(r + 2 * d) * (R + 2) + j] | (uint32_t)tile[(r + 2 * d + 1) * (R + 2) + j] << 16;
        return o;
    };
    if (blk < pl.nb * B.nA) {
        const int i = blk / pl.nb, rank = adapter_rank(B, i);
        const int64_t n0 = (int64_t)(blk % pl.nb) * 64;
        const uint16_t *src = b + (int64_t)i * N * R;
        for (int e = tid; e < 64 * pieces; e += 256) {
            const int r = e / pieces, j = e % pieces * 8;
            v4i v = {0, 0, 0, 0};
            if (n0 + r < N) v = keep8(ld16(src + (n0 + r) * R + j), rank - j);
#pragma unroll
            for (int d = 0; d < 4; d++) *reinterpret_cast<int *>(tile + r * (R + 2) + j + 2 * d) = v[d];
        }
        __syncthreads();
        uint16_t *dst = bt + (int64_t)i * R * N;
        for (int e = tid; e < 8 * R; e += 256) {
            const int r = (e & 7) * 8, j = e >> 3;
            if (n0 + r < N) *reinterpret_cast<v4i *>(dst + (int64_t)j * N + n0 + r) = column(r, j);
        }
        return;
    }
    blk -= pl.nb * B.nA;
    if (blk < pl.na * B.nA) {
        const int i = blk / pl.na, rank = adapter_rank(B, i);
        const int64_t k0 = (int64_t)(blk % pl.na) * 64;
        const uint16_t *src = a + (int64_t)i * R * K;
        for (int e = tid; e < 8 * R; e += 256) {
            const int r = (e & 7) * 8, j = e >> 3;
            v4i v = {0, 0, 0, 0};
            if (k0 + r < K && j < rank) v = ld16(src + (int64_t)j * K + k0 + r);
#pragma unroll
            for (int d = 0; d < 4; d++) {
                tile[(r + 2 * d) * (R + 2) + j] = (uint16_t)v[d];
                tile[(r + 2 * d + 1) * (R + 2) + j] = (uint16_t)((uint32_t)v[d] >> 16);
            }
        }
        __syncthreads();
        uint16_t *dst = at + (int64_t)i * K * R;
        for (int e = tid; e < 64 * pieces; e += 256) {
            const int r = e / pieces, j = e % pieces * 8;
            v4i v;
#pragma unroll
            for (int d = 0; d < 4; d++) v[d] = *reinterpret_cast<const int *>(tile + r * (R + 2) + j + 2 * d);
            if (k0 + r < K) *reinterpret_cast<v4i *>(dst + (k0 + r) * R + j) = v;
        }
        return;
    }
    blk -= pl.na * B.nA;
    // 8 rows of one rank per thread
    const int64_t e = (int64_t)blk * 256 + tid;
    const int j = (int)(e % R);
    const int64_t m0 = e / R * 8;
    if (m0 >= B.M) return;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = m0 + i < B.M ? t[(m0 + i) * R + j] : 0.0f;
    v4i p[kParts];
    split8(v, p);
#pragma unroll
    for (int i = 0; i < 3; i++) *reinterpret_cast<v4i *>(tp + packed_at((int)m0, i, j, R)) = p[i];
}

// ---------------------------------------------------------------------------
// Gradients of the weights: G[c, j] = sum_m src[m, c] p[m, j] over the rows of
// one request (src = dy or x, p = t or u in 3 bf16 parts).  A wave owns 128
// columns; 32 rows are one 16x16x32 MFMA step.  The contraction runs over
// rows, but memory holds columns together: a lane loads 8 columns of 8 rows
// (16 bytes each, 256 contiguous bytes per 16 lanes) and turns the 8 x 8
// values in registers with 32 byte permutes, so that its q-th fragment holds
// 8 rows of column n0 + 8 (l % 16) + q: one MFMA per q, no LDS.  Loads are
// hidden by the other workgroup of the compute unit, so the registers of one
// step have to let two in: with a second step's rows in flight, ranks above 32
// left one, and 17776 x (7680 + 1920) took 125 us at rank 64 and 245 at 128,
// against 90 and 157 (rank 32, two workgroups either way: 72 and 71).  The four
// waves take every fourth step of the chunk's rows and add up in LDS in wave
// order; a workgroup writes one partial per request that its chunk meets, at
// slot chunk + request (unique, both only grow).  Rows of other requests in
// the same step are read as zeros in both operands.  Where a wave's sums come out
// not finite, it takes its rows again with dy's or x's infinities kept from the
// later parts of p (split8): looking for them beforehand would cost every call.
// WIDE (da): G is stored [j][c], else (db) [c][j].
// ---------------------------------------------------------------------------
constexpr int kGradRows = 128;  // rows of a chunk: a multiple of 4 waves x 32

struct GradPlan {
    int chunk;       // rows of a chunk
    int strips_n, strips_k;  // 128-column strips of dy and x
};

template <int RC, bool WIDE>
__device__ __forceinline__ void grad_strip(const uint16_t *__restrict__ src, const uint16_t *__restrict__ pk,
                                           const LoraBatch &B, int64_t C, const GradPlan &pl, int strip, int chunk,
                                           int jb, float *__restrict__ out, float *lds) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int64_t n0 = (int64_t)strip * 128;
    const int64_t col = n0 + 8 * c;
    const bool in_col = col < C;
    const int j0 = jb * 16 * RC;
    // the lane's place in a step: its first row and column (C <= 2^26: below 2^32 bytes)
    const uint32_t at = 2 * ((uint32_t)(8 * q) * (uint32_t)C + 8 * c);
    const int r0 = chunk * pl.chunk, r1 = r0 + pl.chunk < B.M ? r0 + pl.chunk : B.M;
    for (int s = 0; s < B.S; s++) {
        int lo = seg_clamp(B.seg_start[s], B.M), hi = seg_clamp(B.seg_start[s + 1], B.M);
        lo = lo > r0 ? lo : r0;
        hi = hi < r1 ? hi : r1;
        if (lo >= hi || seg_adapter_of(B, s) < 0) continue;  // workgroup-uniform
        v4f acc[8][RC];
        v4i w[8], pf[RC][3];
        auto load = [&](int m0) {
            const int m = m0 + 8 * q;  // the lane's 8 rows
            const bool edge = m0 < lo || m0 + 32 > hi;  // wave-uniform
#pragma unroll
            for (int r = 0; r < 8; r++) {
                const bool ok = in_col && (!edge || (m + r >= lo && m + r < hi));
                const char *row = reinterpret_cast<const char *>(src + (int64_t)(m0 + r) * C + n0);  // wave-uniform
                w[r] = ok ? ld16(row + at) : (v4i){0, 0, 0, 0};
            }
        };
        auto parts = [&](int m0) {
#pragma unroll
            for (int k = 0; k < RC; k++)
#pragma unroll
                for (int p = 0; p < 3; p++)
                    pf[k][p] = ld16(pk + packed_at(m0, p, j0 + 16 * k < B.R ? j0 + 16 * k : 0, B.R) + 8 * lane);
        };
        // apart: infinities of src kept from the later parts of p
        auto mul = [&](int m0, auto apart) {
            const int m = m0 + 8 * q;
            if (m0 < lo || m0 + 32 > hi) {  // wave-uniform
#pragma unroll
                for (int k = 0; k < RC; k++)
#pragma unroll
                    for (int p = 0; p < 3; p++) {
                        v4i f = keep8(pf[k][p], hi - m);   // without the rows from hi on
                        const v4i low = keep8(f, lo - m);  // and those before lo
#pragma unroll
                        for (int d = 0; d < 4; d++) f[d] &= ~low[d];
                        pf[k][p] = f;
                    }
            }
#pragma unroll
            for (int d = 0; d < 4; d++) {
                v4i f0, f1;  // columns 2d and 2d + 1: 8 rows each
                auto turn = [&]() {
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        f0[r] = (int)__builtin_amdgcn_perm((uint32_t)w[2 * r + 1][d], (uint32_t)w[2 * r][d], 0x05040100u);
                        f1[r] = (int)__builtin_amdgcn_perm((uint32_t)w[2 * r + 1][d], (uint32_t)w[2 * r][d], 0x07060302u);
                    }
                };
                auto part = [&](int k, int p) {
                    if constexpr (WIDE) {
                        acc[2 * d][k] = mfma16(f0, pf[k][p], acc[2 * d][k]);
                        acc[2 * d + 1][k] = mfma16(f1, pf[k][p], acc[2 * d + 1][k]);
                    } else {
                        acc[2 * d][k] = mfma16(pf[k][p], f0, acc[2 * d][k]);
                        acc[2 * d + 1][k] = mfma16(pf[k][p], f1, acc[2 * d + 1][k]);
                    }
                };
                turn();
                if constexpr (apart) f0 = finite8(f0), f1 = finite8(f1);
#pragma unroll
                for (int k = 0; k < RC; k++) {
                    part(k, 2), part(k, 1);  // the small parts first
                    if constexpr (!apart) part(k, 0);
                }
                if constexpr (apart) {
                    turn();
#pragma unroll
                    for (int k = 0; k < RC; k++) part(k, 0);
                }
            }
        };
        // the next step's operands go out once this step's products have taken theirs
        const int first = (lo & ~31) + 32 * wave;
        auto clear = [&]() {
#pragma unroll
            for (int i = 0; i < 8; i++)
#pragma unroll
                for (int k = 0; k < RC; k++) acc[i][k] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
        };
        clear();
        if (first < hi) {
            parts(first);
            load(first);
        }
        for (int m0 = first; m0 < hi; m0 += 128) {
            mul(m0, std::false_type());
            if (m0 + 128 < hi) {
                parts(m0 + 128);
                load(m0 + 128);
            }
        }
        float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // NaN after a value that is not finite
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int k = 0; k < RC; k++)
#pragma unroll
                for (int r = 0; r < 4; r++) zero[r] = __builtin_fmaf(acc[i][k][r], 0.0f, zero[r]);
        const bool odd = !((zero[0] + zero[1]) + (zero[2] + zero[3]) == 0.0f);
        if (__builtin_expect(__ballot(odd) != 0, 0)) {
            clear();
            for (int m0 = first; m0 < hi; m0 += 128) {
                parts(m0);
                load(m0);
                mul(m0, std::true_type());
            }
        }
        // waves 1..3 add to wave 0 in order, 8 * RC pieces of 64 x 16 bytes
        v4f *buf = reinterpret_cast<v4f *>(lds);
        for (int wv = 1; wv < 4; wv++) {
            __syncthreads();
            if (wave == wv)
#pragma unroll
                for (int i = 0; i < 8; i++)
#pragma unroll
                    for (int k = 0; k < RC; k++) buf[(i * RC + k) * 64 + lane] = acc[i][k];
            __syncthreads();
            if (wave == 0)
#pragma unroll
                for (int i = 0; i < 8; i++)
#pragma unroll
                    for (int k = 0; k < RC; k++) acc[i][k] += buf[(i * RC + k) * 64 + lane];
        }
        if (wave == 0) {
            float *o = out + (int64_t)(chunk + s) * C * B.R;
            if constexpr (WIDE) {
                // lane = rank c; register r of fragment i is column 8 (4 q + r) + i
#pragma unroll
                for (int k = 0; k < RC; k++) {
                    const int j = j0 + 16 * k + c;
                    if (j >= B.R) continue;
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        const int64_t cc = n0 + 8 * (4 * q + r);
                        if (cc >= C) continue;
                        float *d = o + (int64_t)j * C + cc;
                        *reinterpret_cast<float4 *>(d) = make_float4(acc[0][k][r], acc[1][k][r], acc[2][k][r], acc[3][k][r]);
                        *reinterpret_cast<float4 *>(d + 4) = make_float4(acc[4][k][r], acc[5][k][r], acc[6][k][r], acc[7][k][r]);
                    }
                }
            } else {
                // lane = column 8 c + i of fragment i; registers = 4 consecutive ranks
#pragma unroll
                for (int i = 0; i < 8; i++)
#pragma unroll
                    for (int k = 0; k < RC; k++)
                        if (in_col && j0 + 16 * k < B.R)
                            *reinterpret_cast<v4f *>(o + (col + i) * B.R + j0 + 16 * k + 4 * q) = acc[i][k];
            }
        }
        __syncthreads();
    }
}

template <int RC>
__global__ __launch_bounds__(256, 2) void lora_grad_kernel(const uint16_t *__restrict__ dy,
                                                        const uint16_t *__restrict__ x,
                                                        const uint16_t *__restrict__ tp,
                                                        const uint16_t *__restrict__ up, LoraBatch B, int64_t N,
                                                        int64_t K, GradPlan pl, float *__restrict__ pb,
                                                        float *__restrict__ pa) {
    __shared__ float lds[8 * RC * 64 * 4];
    const int strip = blockIdx.x;
    if (strip < pl.strips_n)
        grad_strip<RC, false>(dy, tp, B, N, pl, strip, blockIdx.y, blockIdx.z, pb, lds);
    else
        grad_strip<RC, true>(x, up, B, K, pl, strip - pl.strips_n, blockIdx.y, blockIdx.z, pa, lds);
}

// The partials of an adapter's requests, added in row order; zeros past its
// rank and for adapters without rows.  4 values per thread.
__global__ __launch_bounds__(256) void lora_grad_sum_kernel(const float *__restrict__ pb,
                                                            const float *__restrict__ pa, LoraBatch B, int64_t N,
                                                            int64_t K, int chunk, unsigned first,
                                                            float *__restrict__ da, float *__restrict__ db) {
    const int i = blockIdx.y, rank = adapter_rank(B, i);
    const int64_t nb = N * B.R, na = K * B.R;
    int64_t e = (((int64_t)first + blockIdx.x) * 256 + threadIdx.x) * 4;
    const bool is_b = e < nb;
    if (!is_b) e -= nb;
    if (!is_b && e >= na) return;
    const float *p = (is_b ? pb : pa) + e;
    const int64_t stride = is_b ? nb : na;
    v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < B.S; s++) {
        if (B.seg_adapter[s] != i) continue;
        const int lo = seg_clamp(B.seg_start[s], B.M), hi = seg_clamp(B.seg_start[s + 1], B.M);
        if (lo >= hi) continue;
        for (int c = lo / chunk; c <= (hi - 1) / chunk; c++)
            v += *reinterpret_cast<const v4f *>(p + (int64_t)(c + s) * stride);
    }
    const float sc = is_b ? B.scale[i] : 1.0f;  // u already carries the scale
    v4f o;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const int j = is_b ? (int)((e + k) % B.R) : (int)(e / K);
        o[k] = j < rank ? v[k] * sc : 0.0f;
    }
    *reinterpret_cast<v4f *>((is_b ? db + (int64_t)i * nb : da + (int64_t)i * na) + e) = o;
}

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Rows of a chunk, a multiple of kGradRows: up to 512 workgroups (the two that
// each compute unit holds), counting the two for ranks above 64.  More write
// more partials that are read again (8000 x 1920 + 1920, rank 128, the whole
// backward pass: 121 us with 512, 147 with twice as many).
int grad_chunk(int64_t M, int64_t N, int64_t K, int64_t R) {
    const int64_t strips = ((N + 127) / 128 + (K + 127) / 128) * ((R + 63) / 64);
    int64_t chunks = 512 / (strips > 0 ? strips : 1);
    if (chunks < 1) chunks = 1;
    return (int)round_up(M > 0 ? (M + chunks - 1) / chunks : 1, kGradRows);
}

struct BackwardLayout {
    int chunk, slots;
    size_t at, bt, tp, up, u, pb, pa, total;
};

BackwardLayout backward_layout(int64_t M, int64_t N, int64_t K, int64_t R, int64_t S, int64_t nA) {
    BackwardLayout L;
    L.chunk = grad_chunk(M, N, K, R);
    L.slots = (int)((M + L.chunk - 1) / L.chunk + S);
    const size_t packed = 2 * 3 * (size_t)R * round_up(M, 32);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) / 256 * 256;
        return at;
    };
    L.at = take(2 * (size_t)nA * R * K);
    L.bt = take(2 * (size_t)nA * R * N);
    L.tp = take(packed);
    L.up = take(packed);
    L.u = take(4 * (size_t)M * R);
    L.pb = take(4 * (size_t)L.slots * N * R);
    L.pa = take(4 * (size_t)L.slots * K * R);
    L.total = o;
    return L;
}

// Tiles of TM rows that seg_tile() can give: whole ones plus one ragged one
// per row range, and never more than there are rows.
unsigned seg_tiles(const LoraBatch &B, int TM) {
    const int64_t n = (int64_t)B.M / TM + B.S + 2;
    return (unsigned)(n < B.M ? n : B.M);
}

// launch(first, n) for `count` units in runs of at most `most` (units of one
// workgroup of 256 threads: what a grid holds).
template <class Launch>
hipError_t in_launches(int64_t count, Launch launch, int64_t most = kMaxGroups) {
    for (int64_t first = 0; first < count; first += most) {
        launch((unsigned)first, (unsigned)(count - first < most ? count - first : most));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// From 8192 rows on, one tile of 48 to 80 rows to each compute unit, or to
// each of a multiple of them (M / 256 rows: with 64 each, 17776 rows made 278
// tiles, and the 22 units with two set the time: 75 us where 16384 rows took
// 49).  Below, by the number of 16 x 16 pieces of t: few, and each is a
// workgroup of 16 waves, so that one token's K is read by 16 waves at once;
// more, and 2 or 8 pieces share a workgroup's reads of x and a (1693 x 1920,
// rank 64, 424 pieces: 6.9 us with 2, 9.3 with 1, 9.9 with 8; 8000 x 1920, rank
// 64, 2000 pieces: 16.8, 31.4, 12.5).
template <bool UP>
hipError_t shrink(hipStream_t st, const uint16_t *x, const uint16_t *a, const LoraBatch &B, int64_t K, float *t,
                  uint16_t *packed) {
    if (B.M == 0) return hipSuccess;
    if (B.M < 8192) {
        const int pieces = (B.M + 15) / 16 * (B.R / 16);
        if (pieces < 256)
            hipLaunchKernelGGL((lora_shrink_kernel<1, 1, 16, UP>), dim3(seg_tiles(B, 16), B.R / 16), dim3(1024), 0, st,
                               x, a, B, K, 16, 0u, t, packed);
        else if (pieces < 1024)
            hipLaunchKernelGGL((lora_shrink_kernel<1, 2, 8, UP>), dim3(seg_tiles(B, 16), (B.R + 31) / 32), dim3(512), 0,
                               st, x, a, B, K, 16, 0u, t, packed);
        else
            hipLaunchKernelGGL((lora_shrink_kernel<2, 4, 8, UP>), dim3(seg_tiles(B, 32), (B.R + 63) / 64), dim3(512), 0,
                               st, x, a, B, K, 32, 0u, t, packed);
        return hipGetLastError();
    }
    const int64_t rounds = ((int64_t)B.M + 256 * 80 - 1) / (256 * 80);
    const int64_t ragged = B.S < 64 ? B.S : 64;  // a request may end in a short tile
    int64_t tile = (B.M + 256 * rounds - ragged - 1) / (256 * rounds - ragged);
    if (tile > 80) tile = 80;
    return in_launches(seg_tiles(B, (int)tile), [&](unsigned first, unsigned n) {
        const dim3 grid(n, (B.R + 63) / 64);
#define DMPQ_SHRINK(RC_)                                                                                         \
    hipLaunchKernelGGL((lora_shrink_kernel<5, RC_, 4, UP>), grid, dim3(256), 0, st, x, a, B, K, (int)tile, first, t, \
                       packed)
        if (B.R <= 16)
            DMPQ_SHRINK(1);
        else if (B.R <= 32)
            DMPQ_SHRINK(2);
        else
            DMPQ_SHRINK(4);
#undef DMPQ_SHRINK
    });
}

template <int ES>
hipError_t expand(hipStream_t st, const float *t, const void *base, const uint16_t *b, const LoraBatch &B, int64_t N,
                  void *y) {
    const unsigned cols = (unsigned)((N + kExpandCols - 1) / kExpandCols);  // <= 2^19
    return in_launches(
        seg_tiles(B, kExpandRows),
        [&](unsigned first, unsigned n) {
#define DMPQ_EXPAND(RC_)                                                                                           \
    hipLaunchKernelGGL((lora_expand_kernel<ES, RC_>), dim3(n * cols), dim3(64 * kExpandWaves), 0, st, t, base, b, B, N, \
                       cols, first, y)
            if (B.R <= 16)
                DMPQ_EXPAND(1);
            else if (B.R <= 32)
                DMPQ_EXPAND(2);
            else if (B.R <= 64)
                DMPQ_EXPAND(4);
            else
                DMPQ_EXPAND(8);
#undef DMPQ_EXPAND
        },
        kMaxGroups / cols);
}

}  // namespace

hipError_t launch_lora_shrink(hipStream_t s, const uint16_t *x, const uint16_t *a, const LoraBatch &B, int64_t K,
                              float *t) {
    return shrink<false>(s, x, a, B, K, t, nullptr);
}

hipError_t launch_lora_expand(hipStream_t s, const float *t, const void *base, const uint16_t *b, const LoraBatch &B,
                              int64_t N, int out_dtype, void *y) {
    if (B.M == 0 || N == 0) return hipSuccess;
    return out_dtype == 1 ? expand<2>(s, t, base, b, B, N, y) : expand<4>(s, t, base, b, B, N, y);
}

size_t lora_backward_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int64_t S, int64_t nA) {
    // backward_layout's sizes without their rounding, in fp64: they can pass 64 bits
    const double slots = (double)M / kGradRows + 1 + (double)S;
    const double bytes = (double)(N + K) * R * (2.0 * nA + 4.0 * slots) + 16.0 * (double)R * (M + 32.0);
    if (bytes > 4e18) return SIZE_MAX;
    return backward_layout(M, N, K, R, S, nA).total;
}

hipError_t launch_lora_backward(hipStream_t s, const uint16_t *dy, const uint16_t *x, const float *t,
                                const uint16_t *a, const uint16_t *b, const LoraBatch &B, int64_t N, int64_t K,
                                const uint16_t *dx_base, uint16_t *dx, float *da, float *db, void *ws) {
    const BackwardLayout L = backward_layout(B.M, N, K, B.R, B.S, B.nA);
    uint8_t *w = static_cast<uint8_t *>(ws);
    uint16_t *at = reinterpret_cast<uint16_t *>(w + L.at), *bt = reinterpret_cast<uint16_t *>(w + L.bt);
    uint16_t *tp = reinterpret_cast<uint16_t *>(w + L.tp), *up = reinterpret_cast<uint16_t *>(w + L.up);
    float *u = reinterpret_cast<float *>(w + L.u);
    float *pb = reinterpret_cast<float *>(w + L.pb), *pa = reinterpret_cast<float *>(w + L.pa);
    if (B.M > 0) {
        PrepPlan pp{(int)((N + 63) / 64), (int)((K + 63) / 64)};
        const int64_t pack = ((int64_t)(B.M + 7) / 8 * B.R + 255) / 256;
        hipError_t e = in_launches((int64_t)(pp.nb + pp.na) * B.nA + pack, [&](unsigned first, unsigned n) {
            hipLaunchKernelGGL(lora_prep_kernel, dim3(n), dim3(256), 0, s, a, b, t, B, N, K, pp, first, at, bt, tp);
        });
        if (e == hipSuccess) e = shrink<true>(s, dy, bt, B, N, u, up);
        if (e != hipSuccess) return e;
        GradPlan gp{L.chunk, (int)((N + 127) / 128), (int)((K + 127) / 128)};
        const unsigned strips = (unsigned)(gp.strips_n + gp.strips_k), chunks = (unsigned)((B.M + L.chunk - 1) / L.chunk);
        // 16 ranks a workgroup while the chunks are short (a wave takes at most two
        // steps of one) and all workgroups fit on the chip at once, four to a
        // compute unit: then a workgroup's latency is the time.  The whole backward
        // pass at 1920 + 1920 with 16 ranks a workgroup and with all of them (at
        // most 64): 903 rows, rank 64: 36 and 43 us; 300 rows, rank 128: 42 and 53;
        // 2000 rows, rank 32, chunks of 128: 34 and 37; 4000, of 256: 40.1 and 41.2;
        // 6000, of 384: 50.8 and 49.5; 10000, of 640: 73 and 69, since dy and x are
        // read once more.
#define DMPQ_GRAD(RC_) \
    hipLaunchKernelGGL(lora_grad_kernel<RC_>, dim3(strips, chunks, (B.R + 16 * RC_ - 1) / (16 * RC_)), dim3(256), 0, s, dy, \
                       x, tp, up, B, N, K, gp, pb, pa)
        if (B.R <= 16 || (L.chunk <= 256 && (int64_t)strips * chunks * (B.R / 16) <= 1024))
            DMPQ_GRAD(1);
        else if (B.R <= 32)
            DMPQ_GRAD(2);
        else
            DMPQ_GRAD(4);
#undef DMPQ_GRAD
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        LoraBatch one = B;  // u already carries the scales, at the ranks' zeros
        one.scale = nullptr;
        if (dx) {
            e = launch_lora_expand(s, u, dx_base, at, one, K, 1, dx);
            if (e != hipSuccess) return e;
        }
    }
    if (B.nA == 0) return hipSuccess;
    const int64_t vals = (N + K) * B.R;
    return in_launches((vals / 4 + 255) / 256, [&](unsigned first, unsigned n) {
        hipLaunchKernelGGL(lora_grad_sum_kernel, dim3(n, (unsigned)B.nA), dim3(256), 0, s, pb, pa, B, N, K, L.chunk, first,
                           da, db);
    });
}

}  // namespace dmpq
