// lora.hip -- low-rank adapters of many requests beside a shared projection,
// and their gradients.  Request i adds scale_i (x a_i^T) b_i^T to the rows of
// the frozen projection that are its own; a is [R x K], b is [N x R].
//
//   shrink   t = x a^T               [M x R] fp32
//   expand   y = base + scale t b^T  [M x N] bf16 or fp32
//   backward u = scale dy b, dx = dx_base + u a, da = u^T x, db = scale dy^T t
//
// Every product has one dimension of at most 128, so all of them are bound by
// the one pass over their widest tensor.  MFMA does the products: x, dy, a and
// b are bf16 and exact in it; t and u are fp32 and enter as 2 bf16 parts where
// the result is rounded to bf16 anyway and as 3 where it stays fp32 (split8).
// Sums are fp32 in a fixed order: no atomics, the same bits on every call.
#include "device.hpp"
#include "gemm_common.hpp"
#include "internal.hpp"
#include "lora.hpp"

namespace dmpq {

namespace {

__device__ __forceinline__ v4i ld16(const void *p) { return *reinterpret_cast<const v4i *>(p); }

// ---------------------------------------------------------------------------
// Shrink: t[m, j] = sum_k x[m, k] a[j, k] for a tile of 16 RT rows of one
// request and 16 RC of its ranks (part blockIdx.y).  The WAVES waves share the
// K steps of 32 (16x16x32 MFMA, fragments straight from global memory: lane l
// holds 8 k of row l % 16, so a row's 64 bytes are one segment) and their sums
// meet in LDS, added in wave order.  UP: the same product for u = scale dy b
// (x is dy, a the transposed b), stored times scale, and once more as 3 bf16
// parts [part][j][m] for the gradients' products over m.
// ---------------------------------------------------------------------------
struct PackedOut {
    uint16_t *p;   // [3][R][ld]
    int64_t ld;
};

template <int RT, int RC, int WAVES, bool UP>
__global__ __launch_bounds__(64 * WAVES) void lora_shrink_kernel(const uint16_t *__restrict__ x,
                                                                 const uint16_t *__restrict__ a, LoraBatch B,
                                                                 int64_t K, float *__restrict__ t, PackedOut pk) {
    constexpr int TM = 16 * RT, TJ = 16 * RC;
    __shared__ float part[WAVES][TM][TJ + 4];
    SegTile st;
    if (!seg_tile(B, blockIdx.x, TM, st)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int j0 = blockIdx.y * TJ;
    const int rank = st.adapter < 0 ? 0 : adapter_rank(B, st.adapter);
    if (rank > j0) {  // workgroup-uniform
        const int c = lane & 15, q = lane >> 4;
        const uint16_t *xr[RT], *ar[RC];
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const int r = 16 * i + c;
            xr[i] = x + (int64_t)(st.row0 + (r < st.rows ? r : st.rows - 1)) * K + 8 * q;
        }
#pragma unroll
        for (int i = 0; i < RC; i++) {
            const int j = j0 + 16 * i + c;
            ar[i] = a + ((int64_t)st.adapter * B.R + (j < B.R ? j : B.R - 1)) * K + 8 * q;
        }
        v4f acc[RT][RC];
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int k = 0; k < RC; k++) acc[i][k] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
        const int64_t full = K / 32;  // whole steps; K % 32 == 16 leaves half a step to the last wave
        const int64_t k1 = full * (wave + 1) / WAVES;
#pragma unroll 4
        for (int64_t s = full * wave / WAVES; s < k1; s++) {
            v4i xf[RT], af[RC];
#pragma unroll
            for (int i = 0; i < RT; i++) xf[i] = ld16(xr[i] + 32 * s);
#pragma unroll
            for (int i = 0; i < RC; i++) af[i] = ld16(ar[i] + 32 * s);
#pragma unroll
            for (int i = 0; i < RT; i++)
#pragma unroll
                for (int k = 0; k < RC; k++) acc[i][k] = mfma16(af[k], xf[i], acc[i][k]);
        }
        if (wave == WAVES - 1 && (K & 16)) {
            v4i xf[RT], af[RC];
            const v4i zero = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < RT; i++) xf[i] = q < 2 ? ld16(xr[i] + 32 * full) : zero;
#pragma unroll
            for (int i = 0; i < RC; i++) af[i] = q < 2 ? ld16(ar[i] + 32 * full) : zero;
#pragma unroll
            for (int i = 0; i < RT; i++)
#pragma unroll
                for (int k = 0; k < RC; k++) acc[i][k] = mfma16(af[k], xf[i], acc[i][k]);
        }
        // D: lane column = token, registers = 4 consecutive ranks
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int k = 0; k < RC; k++)
                *reinterpret_cast<v4f *>(&part[wave][16 * i + c][16 * k + 4 * q]) = acc[i][k];
    }
    __syncthreads();
    const float sc = UP && st.adapter >= 0 ? B.scale[st.adapter] : 1.0f;
    for (int e = threadIdx.x; e < TM * TJ; e += 64 * WAVES) {
        const int r = e / TJ, j = e % TJ;
        if (r >= st.rows || j0 + j >= B.R) continue;
        float v = 0.0f;
        if (j0 + j < rank) {
            v = part[0][r][j];
#pragma unroll
            for (int w = 1; w < WAVES; w++) v += part[w][r][j];
            v *= sc;
        }
        t[(int64_t)(st.row0 + r) * B.R + j0 + j] = v;
        if constexpr (UP) {
            float rest = v;
#pragma unroll
            for (int p = 0; p < 3; p++) {
                const uint32_t h = f32_to_bf16(rest);
                pk.p[((int64_t)p * B.R + j0 + j) * pk.ld + st.row0 + r] = (uint16_t)h;
                const float f = bf16_lo(h);
                rest = __builtin_isfinite(f) ? rest - f : 0.0f;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Expand: y = base + scale t b^T for a tile of 32 rows of one request.  A wave
// keeps its rows' t as MFMA fragments (2 bf16 parts for a bf16 y, 3 for fp32)
// and walks over 128-column blocks: the block's base rows are loaded first
// (row-contiguous, 16 bytes per lane), the 32x32x16 MFMAs with b's rows as
// the first operand leave each lane 4 consecutive columns of one row, the
// wave's LDS band turns them row-contiguous, and base + scale * delta goes out
// in 16-byte pieces.
// ---------------------------------------------------------------------------
template <int ES>
__device__ __forceinline__ void expand_piece(const float *d, float sc, const void *base, void *y, int64_t at, bool vec,
                                             int left) {
    constexpr int PER = 16 / ES;
    const uint8_t *bp = static_cast<const uint8_t *>(base) + at * ES;
    uint8_t *yp = static_cast<uint8_t *>(y) + at * ES;
    if (vec && left >= PER) {
        const uint4 bv = base ? *reinterpret_cast<const uint4 *>(bp) : make_uint4(0u, 0u, 0u, 0u);
        uint4 o;
        if constexpr (ES == 2) {
            o.x = cvt_pk_bf16(bf16_lo(bv.x) + sc * d[0], bf16_hi(bv.x) + sc * d[1]);
            o.y = cvt_pk_bf16(bf16_lo(bv.y) + sc * d[2], bf16_hi(bv.y) + sc * d[3]);
            o.z = cvt_pk_bf16(bf16_lo(bv.z) + sc * d[4], bf16_hi(bv.z) + sc * d[5]);
            o.w = cvt_pk_bf16(bf16_lo(bv.w) + sc * d[6], bf16_hi(bv.w) + sc * d[7]);
        } else {
            o.x = __float_as_uint(__uint_as_float(bv.x) + sc * d[0]);
            o.y = __float_as_uint(__uint_as_float(bv.y) + sc * d[1]);
            o.z = __float_as_uint(__uint_as_float(bv.z) + sc * d[2]);
            o.w = __float_as_uint(__uint_as_float(bv.w) + sc * d[3]);
        }
        *reinterpret_cast<uint4 *>(yp) = o;
        return;
    }
#pragma unroll
    for (int e = 0; e < PER; e++) {
        if (e >= left) break;
        if constexpr (ES == 2) {
            const float b = base ? bf16_lo(reinterpret_cast<const uint16_t *>(bp)[e]) : 0.0f;
            reinterpret_cast<uint16_t *>(yp)[e] = (uint16_t)cvt_pk_bf16(b + sc * d[e], 0.0f);
        } else {
            const float b = base ? reinterpret_cast<const float *>(bp)[e] : 0.0f;
            reinterpret_cast<float *>(yp)[e] = b + sc * d[e];
        }
    }
}

constexpr int kExpandRows = 32, kExpandCols = 128, kExpandWaves = 4;

template <int ES, int RC>
__global__ __launch_bounds__(64 * kExpandWaves) void lora_expand_kernel(const float *__restrict__ t,
                                                                        const void *base, const uint16_t *__restrict__ b,
                                                                        LoraBatch B, int64_t N, int blocks, void *y) {
    constexpr int NS = ES == 2 ? 2 : 3;
    constexpr int PER = 16 / ES, LPR = kExpandCols / PER, RPP = 64 / LPR;  // lanes a row, rows a pass
    constexpr int STRIDE = kExpandCols + 4;
    __shared__ float band[kExpandWaves][kExpandRows * STRIDE];
    SegTile st;
    if (!seg_tile(B, blockIdx.x, kExpandRows, st)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lm = lane & 31, lh = lane >> 5;
    const int rank = st.adapter < 0 ? 0 : adapter_rank(B, st.adapter);
    if (rank == 0 && base == y) return;
    // rows of no adapter: base + 1 * -0, which is base bit for bit
    const float sc = rank == 0 || !B.scale ? 1.0f : B.scale[st.adapter];
    const bool vec = ((N * ES) & 15) == 0;
    v4i tf[RC][NS];
    if (rank > 0) {
        const float *tr = t + (int64_t)(st.row0 + (lm < st.rows ? lm : st.rows - 1)) * B.R + 8 * lh;
#pragma unroll
        for (int c = 0; c < RC; c++) {
            float v[8];
            const bool in = 16 * c < B.R;
            const v4f a0 = in ? *reinterpret_cast<const v4f *>(tr + 16 * c) : (v4f){0.0f, 0.0f, 0.0f, 0.0f};
            const v4f a1 = in ? *reinterpret_cast<const v4f *>(tr + 16 * c + 4) : (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                v[e] = a0[e];
                v[4 + e] = a1[e];
            }
            split8<NS>(v, tf[c]);
        }
    }
    const uint16_t *bw = b + (int64_t)(st.adapter < 0 ? 0 : st.adapter) * N * B.R;
    float *bd = band[wave];
    const int cols_blocks = (int)((N + kExpandCols - 1) / kExpandCols);
    const int first = blockIdx.y * blocks;
    const int last = first + blocks < cols_blocks ? first + blocks : cols_blocks;
    for (int cb = first + wave; cb < last; cb += kExpandWaves) {
        const int64_t n0 = (int64_t)cb * kExpandCols;
        if (rank > 0) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                v16f acc;
#pragma unroll
                for (int e = 0; e < 16; e++) acc[e] = 0.0f;
                const int64_t n = n0 + 32 * j + lm;
                const uint16_t *br = bw + (n < N ? n : N - 1) * B.R + 8 * lh;
#pragma unroll
                for (int c = 0; c < RC; c++) {
                    if (16 * c >= rank) break;  // wave-uniform
                    v4i bf = ld16(br + 16 * c);
                    if (16 * c + 16 > rank) bf = keep8(bf, rank - 16 * c - 8 * lh);
#pragma unroll
                    for (int p = 0; p < NS; p++) acc = mfma32(bf, tf[c][p], acc);
                }
#pragma unroll
                for (int g = 0; g < 4; g++)
                    *reinterpret_cast<float4 *>(bd + lm * STRIDE + 32 * j + 8 * g + 4 * lh) =
                        make_float4(acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]);
            }
        }
        const int64_t col = n0 + (lane % LPR) * PER;
#pragma unroll 4
        for (int p = 0; p < kExpandRows / RPP; p++) {
            const int r = p * RPP + lane / LPR;
            float d[PER];
#pragma unroll
            for (int e = 0; e < PER; e++) d[e] = -0.0f;
            if (rank > 0) {
#pragma unroll
                for (int e = 0; e < PER; e += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(bd + r * STRIDE + (lane % LPR) * PER + e);
                    d[e] = f.x, d[e + 1] = f.y, d[e + 2] = f.z, d[e + 3] = f.w;
                }
            }
            if (r < st.rows && col < N)
                expand_piece<ES>(d, sc, base, y, (int64_t)(st.row0 + r) * N + col, vec,
                                 (int)(N - col < PER ? N - col : PER));
        }
    }
}

// ---------------------------------------------------------------------------
// Backward, first launch: what the products over the other dimension need.
//   blocks 0 ..            b [N x R] -> bt [R x N], 64 x R tiles through LDS
//   then                   a [R x K] -> at [K x R]
//   then                   t [M x R] -> 3 bf16 parts [part][j][m]
// Entries past an adapter's rank become zeros.
// ---------------------------------------------------------------------------
struct PrepPlan {
    int nb, na;      // tiles of one adapter's b and a
    int64_t ld;      // row length of the packed t
};

__global__ __launch_bounds__(256) void lora_prep_kernel(const uint16_t *__restrict__ a, const uint16_t *__restrict__ b,
                                                        const float *__restrict__ t, LoraBatch B, int64_t N, int64_t K,
                                                        PrepPlan pl, uint16_t *__restrict__ at,
                                                        uint16_t *__restrict__ bt, uint16_t *__restrict__ tp) {
    __shared__ uint16_t tile[64 * (kMaxLoraRank + 2)];
    int blk = blockIdx.x;
    const int tid = threadIdx.x, R = B.R;
    if (blk < pl.nb * B.nA) {
        const int i = blk / pl.nb, rank = adapter_rank(B, i);
        const int64_t n0 = (int64_t)(blk % pl.nb) * 64;
        const uint16_t *src = b + (int64_t)i * N * R;
        for (int e = tid; e < 64 * R; e += 256) {
            const int r = e / R, j = e % R;
            tile[r * (R + 2) + j] = n0 + r < N && j < rank ? src[(n0 + r) * R + j] : (uint16_t)0;
        }
        __syncthreads();
        uint16_t *dst = bt + (int64_t)i * R * N;
        for (int e = tid; e < 64 * R; e += 256) {
            const int r = e & 63, j = e >> 6;
            if (n0 + r < N) dst[(int64_t)j * N + n0 + r] = tile[r * (R + 2) + j];
        }
        return;
    }
    blk -= pl.nb * B.nA;
    if (blk < pl.na * B.nA) {
        const int i = blk / pl.na, rank = adapter_rank(B, i);
        const int64_t k0 = (int64_t)(blk % pl.na) * 64;
        const uint16_t *src = a + (int64_t)i * R * K;
        for (int e = tid; e < 64 * R; e += 256) {
            const int r = e & 63, j = e >> 6;
            tile[r * (R + 2) + j] = k0 + r < K && j < rank ? src[(int64_t)j * K + k0 + r] : (uint16_t)0;
        }
        __syncthreads();
        uint16_t *dst = at + (int64_t)i * K * R;
        for (int e = tid; e < 64 * R; e += 256) {
            const int r = e / R, j = e % R;
            if (k0 + r < K) dst[(k0 + r) * R + j] = tile[r * (R + 2) + j];
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
    v4i p[3];
    split8<3>(v, p);
#pragma unroll
    for (int i = 0; i < 3; i++) *reinterpret_cast<v4i *>(tp + ((int64_t)i * R + j) * pl.ld + m0) = p[i];
}

// ---------------------------------------------------------------------------
// Gradients of the weights: G[c, j] = sum_m src[m, c] p[m, j] over the rows of
// one request (src = dy or x, p = t or u in 3 bf16 parts).  A wave owns 128
// columns; 32 rows are one 16x16x32 MFMA step.  The contraction runs over
// rows, but memory holds columns together: a lane loads 8 columns of 8 rows
// (16 bytes each, 256 contiguous bytes per 16 lanes) and turns the 8 x 8
// values in registers with 32 byte permutes, so that its q-th fragment holds
// 8 rows of column n0 + 8 (l % 16) + q: one MFMA per q, no LDS.  The four
// waves take every fourth step of the chunk's rows and add up in LDS in wave
// order; a workgroup writes one partial per request that its chunk meets, at
// slot chunk + request (unique, both only grow).  Rows of other requests in
// the same step are read as zeros in both operands.
// WIDE (da): G is stored [j][c], else (db) [c][j].
// ---------------------------------------------------------------------------
constexpr int kGradRows = 128;  // rows of a chunk: a multiple of 4 waves x 32

struct GradPlan {
    int chunk;       // rows of a chunk
    int strips_n, strips_k;  // 128-column strips of dy and x
    int64_t ld;      // row length of the packed operands
};

template <int RC, bool WIDE>
__device__ __forceinline__ void grad_strip(const uint16_t *__restrict__ src, const uint16_t *__restrict__ pk,
                                           const LoraBatch &B, int64_t C, const GradPlan &pl, int strip, int chunk,
                                           int jb, float *__restrict__ out, float *lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, q = lane >> 4;
    const int64_t n0 = (int64_t)strip * 128;
    const int64_t col = n0 + 8 * c;
    const bool in_col = col < C;
    const int j0 = jb * 16 * RC;
    const int r0 = chunk * pl.chunk, r1 = r0 + pl.chunk < B.M ? r0 + pl.chunk : B.M;
    for (int s = 0; s < B.S; s++) {
        int lo = seg_clamp(B.seg_start[s], B.M), hi = seg_clamp(B.seg_start[s + 1], B.M);
        lo = lo > r0 ? lo : r0;
        hi = hi < r1 ? hi : r1;
        if (lo >= hi || seg_adapter_of(B, s) < 0) continue;  // workgroup-uniform
        v4f acc[8][RC];
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int k = 0; k < RC; k++) acc[i][k] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
        for (int m0 = (lo & ~31) + 32 * wave; m0 < hi; m0 += 128) {
            const int m = m0 + 8 * q;  // the lane's 8 rows
            v4i w[8], pf[RC][3];
            const bool edge = m0 < lo || m0 + 32 > hi;  // wave-uniform
#pragma unroll
            for (int r = 0; r < 8; r++) {
                const bool ok = in_col && (!edge || (m + r >= lo && m + r < hi));
                w[r] = ok ? ld16(src + (int64_t)(m + r) * C + col) : (v4i){0, 0, 0, 0};
            }
#pragma unroll
            for (int k = 0; k < RC; k++)
#pragma unroll
                for (int p = 0; p < 3; p++) {
                    const int j = j0 + 16 * k + c;
                    v4i f = ld16(pk + ((int64_t)p * B.R + (j < B.R ? j : B.R - 1)) * pl.ld + m);
                    if (edge) {
                        f = keep8(f, hi - m);                 // rows from hi on
                        const v4i low = keep8(f, lo - m);     // rows before lo
#pragma unroll
                        for (int d = 0; d < 4; d++) f[d] &= ~low[d];
                    }
                    pf[k][p] = f;
                }
#pragma unroll
            for (int d = 0; d < 4; d++) {
                v4i f0, f1;  // columns 2d and 2d + 1: 8 rows each
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    f0[r] = (int)__builtin_amdgcn_perm((uint32_t)w[2 * r + 1][d], (uint32_t)w[2 * r][d], 0x05040100u);
                    f1[r] = (int)__builtin_amdgcn_perm((uint32_t)w[2 * r + 1][d], (uint32_t)w[2 * r][d], 0x07060302u);
                }
#pragma unroll
                for (int k = 0; k < RC; k++)
#pragma unroll
                    for (int p = 2; p >= 0; p--) {  // the small parts first
                        if constexpr (WIDE) {
                            acc[2 * d][k] = mfma16(f0, pf[k][p], acc[2 * d][k]);
                            acc[2 * d + 1][k] = mfma16(f1, pf[k][p], acc[2 * d + 1][k]);
                        } else {
                            acc[2 * d][k] = mfma16(pf[k][p], f0, acc[2 * d][k]);
                            acc[2 * d + 1][k] = mfma16(pf[k][p], f1, acc[2 * d + 1][k]);
                        }
                    }
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
__global__ __launch_bounds__(256) void lora_grad_kernel(const uint16_t *__restrict__ dy,
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
                                                            int64_t K, int chunk, float *__restrict__ da,
                                                            float *__restrict__ db) {
    const int i = blockIdx.y, rank = adapter_rank(B, i);
    const int64_t nb = N * B.R, na = K * B.R;
    int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
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

// Rows of a chunk: enough chunks that strips x chunks keep the card's 256
// compute units busy, each at least kGradRows.
int grad_chunk(int64_t M, int64_t N, int64_t K) {
    const int64_t strips = (N + 127) / 128 + (K + 127) / 128;
    int64_t chunks = 2048 / (strips > 0 ? strips : 1) + 1;
    const int64_t most = (M + kGradRows - 1) / kGradRows;
    if (chunks > most) chunks = most;
    if (chunks < 1) chunks = 1;
    return (int)round_up(M > 0 ? (M + chunks - 1) / chunks : 1, kGradRows);
}

struct BackwardLayout {
    int chunk, slots;
    int64_t ld;
    size_t at, bt, tp, up, u, pb, pa, total;
};

BackwardLayout backward_layout(int64_t M, int64_t N, int64_t K, int64_t R, int64_t S, int64_t nA) {
    BackwardLayout L;
    L.chunk = grad_chunk(M, N, K);
    L.slots = (int)((M + L.chunk - 1) / L.chunk + S);
    L.ld = round_up(M, 64);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) / 256 * 256;
        return at;
    };
    L.at = take(2 * (size_t)nA * R * K);
    L.bt = take(2 * (size_t)nA * R * N);
    L.tp = take(2 * 3 * (size_t)R * L.ld);
    L.up = take(2 * 3 * (size_t)R * L.ld);
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

// Two forms by the number of 64-row tiles: from 128 on the card is filled by
// tiles of 64 rows (32 from rank 48 on) whose 4 waves share K; below, a
// workgroup of 16 waves takes 16 rows and 16 ranks, so that one token's K is
// read by 16 waves at once and ranks spread over workgroups.
template <bool UP>
hipError_t shrink(hipStream_t st, const uint16_t *x, const uint16_t *a, const LoraBatch &B, int64_t K, float *t,
                  const PackedOut &pk) {
    if (B.M == 0) return hipSuccess;
    if (B.M < 128 * 64) {
        hipLaunchKernelGGL((lora_shrink_kernel<1, 1, 16, UP>), dim3(seg_tiles(B, 16), B.R / 16), dim3(1024), 0, st, x,
                           a, B, K, t, pk);
    } else if (B.R <= 16) {
        hipLaunchKernelGGL((lora_shrink_kernel<4, 1, 4, UP>), dim3(seg_tiles(B, 64)), dim3(256), 0, st, x, a, B, K, t, pk);
    } else if (B.R <= 32) {
        hipLaunchKernelGGL((lora_shrink_kernel<4, 2, 4, UP>), dim3(seg_tiles(B, 64)), dim3(256), 0, st, x, a, B, K, t, pk);
    } else if (B.R <= 64) {
        hipLaunchKernelGGL((lora_shrink_kernel<2, 4, 4, UP>), dim3(seg_tiles(B, 32)), dim3(256), 0, st, x, a, B, K, t, pk);
    } else {
        hipLaunchKernelGGL((lora_shrink_kernel<2, 8, 2, UP>), dim3(seg_tiles(B, 32)), dim3(128), 0, st, x, a, B, K, t, pk);
    }
    return hipGetLastError();
}

template <int ES>
hipError_t expand(hipStream_t st, const float *t, const void *base, const uint16_t *b, const LoraBatch &B, int64_t N,
                  void *y) {
    const int64_t cb = (N + kExpandCols - 1) / kExpandCols;
    const unsigned tiles = seg_tiles(B, kExpandRows);
    // 1 to 8 blocks a wave: as many as leave 4 workgroups to every compute unit
    int64_t per = (int64_t)tiles * cb / (4 * 1024);
    per = per < 1 ? 1 : per > 8 ? 8 : per;
    const int blocks = (int)per * kExpandWaves;
    const dim3 grid(tiles, (unsigned)((cb + blocks - 1) / blocks));
#define DMPQ_EXPAND(RC_) \
    hipLaunchKernelGGL((lora_expand_kernel<ES, RC_>), grid, dim3(64 * kExpandWaves), 0, st, t, base, b, B, N, blocks, y)
    if (B.R <= 16)
        DMPQ_EXPAND(1);
    else if (B.R <= 32)
        DMPQ_EXPAND(2);
    else if (B.R <= 64)
        DMPQ_EXPAND(4);
    else
        DMPQ_EXPAND(8);
#undef DMPQ_EXPAND
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_shrink(hipStream_t s, const uint16_t *x, const uint16_t *a, const LoraBatch &B, int64_t K,
                              float *t) {
    return shrink<false>(s, x, a, B, K, t, PackedOut{nullptr, 0});
}

hipError_t launch_lora_expand(hipStream_t s, const float *t, const void *base, const uint16_t *b, const LoraBatch &B,
                              int64_t N, int out_dtype, void *y) {
    if (B.M == 0 || N == 0) return hipSuccess;
    return out_dtype == 1 ? expand<2>(s, t, base, b, B, N, y) : expand<4>(s, t, base, b, B, N, y);
}

size_t lora_backward_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int64_t S, int64_t nA) {
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
        PrepPlan pp{(int)((N + 63) / 64), (int)((K + 63) / 64), L.ld};
        const int64_t pack = ((int64_t)(B.M + 7) / 8 * B.R + 255) / 256;
        hipLaunchKernelGGL(lora_prep_kernel, dim3((unsigned)((int64_t)(pp.nb + pp.na) * B.nA + pack)), dim3(256), 0, s, a,
                           b, t, B, N, K, pp, at, bt, tp);
        hipError_t e = hipGetLastError();
        if (e == hipSuccess) e = shrink<true>(s, dy, bt, B, N, u, PackedOut{up, L.ld});
        if (e != hipSuccess) return e;
        GradPlan gp{L.chunk, (int)((N + 127) / 128), (int)((K + 127) / 128), L.ld};
        const unsigned strips = (unsigned)(gp.strips_n + gp.strips_k), chunks = (unsigned)((B.M + L.chunk - 1) / L.chunk);
        if (B.R <= 16)
            hipLaunchKernelGGL(lora_grad_kernel<1>, dim3(strips, chunks, 1), dim3(256), 0, s, dy, x, tp, up, B, N, K, gp, pb, pa);
        else if (B.R <= 32)
            hipLaunchKernelGGL(lora_grad_kernel<2>, dim3(strips, chunks, 1), dim3(256), 0, s, dy, x, tp, up, B, N, K, gp, pb, pa);
        else
            hipLaunchKernelGGL(lora_grad_kernel<4>, dim3(strips, chunks, (B.R + 63) / 64), dim3(256), 0, s, dy, x, tp, up, B, N, K,
                               gp, pb, pa);
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
    hipLaunchKernelGGL(lora_grad_sum_kernel, dim3((unsigned)((vals / 4 + 255) / 256), (unsigned)B.nA), dim3(256), 0, s, pb,
                       pa, B, N, K, L.chunk, da, db);
    return hipGetLastError();
}

}  // namespace dmpq
