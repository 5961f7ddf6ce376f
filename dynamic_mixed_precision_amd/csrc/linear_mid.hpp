// linear_mid.hpp -- the whole linear where 256 x 256 tiles are too few to fill
// the chip (prompts, batches of short requests, narrow projections).
//
// BF16 and INT8 (linear_staged_kernel): tiles of 64 x 64, 64 x 128 and 128 x 128.
// Groups of 4 waves bring stages of 128 bytes of every row into LDS by DMA, three or
// four stages ahead, with a barrier a stage; two groups share K between them (one in
// the 128 x 128 tile).  A round of 256 tiles costs a part that does not depend on K
// (the first stages' loads, the epilogue) and one a stage: us, BF16 and INT8 alike,
// 64 x 64 5.5 + 0.2, 64 x 128 6 + 0.33, 128 x 128 10 + 0.52 a stage (256 tiles, K 1920 and
// 3840: BF16 11.5 / 17.2, 15.6 / 25, 25.1 / 41; INT8 8.2 / 11.1, 11.3 / 15.9, 18.5 / 26.3).
// The 128 x 128 tile's four waves are one a SIMD, so nothing hides their waits.
//
// NVFP4 (linear_codes_kernel): 8 waves take a tile of 64 x 64 (or 32 x 128), and each
// computes the whole of it over its own part of K, stages of 128 values of every row,
// straight from memory into fragments of 32 x 32 MFMAs: no LDS and no barrier in the
// loop, two stages in flight a wave (one with 32 x 128).  Every wave dequantizes both
// operands for its part of K.  A lane's 16-byte pieces of a stage are its rows' own,
// and x and w pair the same k.
//
// The groups' or waves' sums meet in LDS and are added in their order, 16 bytes of y
// a lane.  An adapter's term is added row by row from b in memory (lora_row), at a
// cost that grows with its rank: 900 x 1920 x 1920 BF16 13.7 us, with rank 16 / 64 / 128
// 24 / 46 / 75.
#pragma once

#include "device.hpp"
#include "gemm_common.hpp"
#include "gemm_dma.hpp"
#include "internal.hpp"
#include "linear.hpp"
#include "linear_plan.hpp"
#include "lora.hpp"

namespace dmpq {

typedef _Float16 lm_h2 __attribute__((ext_vector_type(2)));
typedef _Float16 lm_h8 __attribute__((ext_vector_type(8)));
namespace lmid {
constexpr int WAVES = 8;
}

// The adapter term of one row and N_ columns from col on, in fp32: the sums of
// short batches are not worth MFMA tiles of their own.
template <int N_>
__device__ __forceinline__ void lora_row(const LoraEpi &L, int64_t row, int64_t col, int64_t N, float (&v)[N_]) {
    const LoraBatch &B = L.batch;
    const int a = row_adapter(B, (int)row);
    const int rank = a < 0 ? 0 : adapter_rank(B, a);
    if (rank == 0) return;
    const float sc = B.scale[a];
    const float *t = L.t + row * B.R;
    const uint16_t *b[N_];
#pragma unroll
    for (int i = 0; i < N_; i++) b[i] = L.b + ((int64_t)a * N + (col + i < N ? col + i : N - 1)) * B.R;
    float s[N_];
#pragma unroll
    for (int i = 0; i < N_; i++) s[i] = 0.0f;
    for (int r = 0; r < rank; r += 8) {
        float tv[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const float4 u = *reinterpret_cast<const float4 *>(t + r + e);
            tv[e] = u.x, tv[e + 1] = u.y, tv[e + 2] = u.z, tv[e + 3] = u.w;
        }
#pragma unroll
        for (int i = 0; i < N_; i++) {
            const uint4 u = *reinterpret_cast<const uint4 *>(b[i] + r);
            const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 8; e++)
                if (r + e < rank) s[i] = __builtin_fmaf(tv[e], e & 1 ? bf16_hi(d[e >> 1]) : bf16_lo(d[e >> 1]), s[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < N_; i++) v[i] = __builtin_fmaf(sc, s[i], v[i]);
}

// The tile's maximum joins that of its 256 x 256 tile: non-negative floats order
// as their bit patterns.
__device__ __forceinline__ void mid_amax_max(float *amax, float top, int64_t m0, int64_t n0, int64_t M) {
    if (!amax) return;
    top = wave_max(top);
    const int64_t tile = (m0 / 256) + (n0 / 256) * ((M + 255) / 256);
    if ((threadIdx.x & 63) == 0) atomicMax(reinterpret_cast<unsigned *>(amax + tile), __float_as_uint(top));
}

// ---- bf16 and int8: operands staged through LDS -------------------------------------

struct MidBF16 {
    static constexpr LinearRoute ROUTE = kLinearBF16;
    typedef v16f acc_t;
    struct Arg {
        const uint16_t *x, *w;
    };
    __host__ __device__ static __forceinline__ int64_t extent(int64_t K) { return 2 * K; }  // bytes of a row
    __device__ static __forceinline__ void mfma(acc_t &c, const v4i &x, const v4i &w) { c = mfma32(w, x, c); }
    template <int N>
    __device__ static __forceinline__ void scale(const Arg &, int64_t, int64_t, int64_t, const float (&sum)[N], float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = sum[i];
    }
};

struct MidI8 {
    static constexpr LinearRoute ROUTE = kLinearInt8;
    typedef v16i acc_t;
    struct Arg {
        const int8_t *x, *w;
        const float *sx, *sw;
    };
    __host__ __device__ static __forceinline__ int64_t extent(int64_t K) { return K; }
    __device__ static __forceinline__ void mfma(acc_t &c, const v4i &x, const v4i &w) {
        c = __builtin_amdgcn_mfma_i32_32x32x32_i8(w, x, c, 0, 0, 0);
    }
    // row m (below M), columns n ..
    template <int N>
    __device__ static __forceinline__ void scale(const Arg &a, int64_t m, int64_t n, int64_t cols, const int (&sum)[N],
                                                 float (&v)[N]) {
        const float r = a.sx[m];
        float c[N];
        load_values<N>(a.sw, false, n, cols - n, c);
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = ((float)sum[i] * r) * c[i];
    }
};

namespace lmid {
// Tiles of 64 MI x 64 NI: groups of 4 waves, each with its own stages, and as many
// stage buffers as fit a CU.
template <int MI, int NI>
constexpr int groups() { return MI * NI == 4 ? 1 : 2; }
template <int MI, int NI>
constexpr int bufs() { return MI * NI == 2 ? 3 : 4; }
template <int MI, int NI>
constexpr int stage() { return 64 * (MI + NI) * 128; }
template <int MI, int NI>
constexpr size_t band() { return (size_t)64 * MI * (64 * NI * 4 + 16); }
template <int MI, int NI>
constexpr size_t staged_lds() {  // the stage buffers, later the groups' sums
    constexpr size_t a = (size_t)groups<MI, NI>() * bufs<MI, NI>() * stage<MI, NI>(), b = groups<MI, NI>() * band<MI, NI>();
    return a > b ? a : b;
}
}  // namespace lmid

// One wave's view of the staged operands: the lane's source offsets (block b =
// wave + 4 q of 1 KB covers rows 8 b .. 8 b + 7 of the tile's x rows, then w rows;
// chunk kc of row r lies at slot kc ^ (r >> 1 & 7), which makes the 32-row fragment
// reads conflict-free) and fragment rows.
template <int MI, int NI, bool TAIL>
struct MidStage {
    static constexpr int P = 2 * (MI + NI);
    const uint8_t *x, *w;
    uint32_t off[P];
    int kc[P];
    int wave, lh, key, fa, fb;
    __device__ __forceinline__ void begin(const uint8_t *x_, const uint8_t *w_, int64_t Kb, int64_t M, int64_t N, int64_t m0,
                                          int64_t n0) {
        const int lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3;
        x = x_ + m0 * Kb, w = w_ + n0 * Kb;
#pragma unroll
        for (int q = 0; q < P; q++) {
            const int r = 8 * (wave + 4 * q) + (lane >> 3), rr = q < 2 * MI ? r : r - 64 * MI;
            const int64_t first = q < 2 * MI ? m0 : n0, end = q < 2 * MI ? M : N;
            const int64_t row = first + rr < end ? first + rr : end - 1;  // past the end: the last one
            kc[q] = (lane & 7) ^ ((r >> 1) & 7);
            off[q] = (uint32_t)((row - first) * Kb) + 16 * kc[q];
        }
        lh = lane >> 5, key = ((lane & 31) >> 1) & 7;
        fa = ((wave >> 1) * 32 * MI + (lane & 31)) * 128;
        fb = (64 * MI + (wave & 1) * 32 * NI + (lane & 31)) * 128;
    }
    // a stage's loads, from byte b of every row on (TAIL: chunks past the row load the
    // stage's first, which is in it)
    __device__ __forceinline__ void issue(uint8_t *dst, int64_t b, int64_t left) const {
        typedef __attribute__((address_space(3))) void lds_void;
#pragma unroll
        for (int q = 0; q < P; q++) {
            const uint8_t *base = (q < 2 * MI ? x : w) + b;
            asm("" : "+s"(base));
            uint32_t o = off[q];
            if (TAIL && 16 * kc[q] >= left) o -= 16 * kc[q];
            __builtin_amdgcn_global_load_lds((const void *)(base + o), (lds_void *)(dst + (wave + 4 * q) * 1024), 16, 0, 0);
        }
    }
    __device__ __forceinline__ void read(const uint8_t *src, int64_t left, v4i (&a)[4][MI], v4i (&b)[4][NI]) const {
#pragma unroll
        for (int s = 0; s < 4; s++) {
            const int slot = ((2 * s + lh) ^ key) * 16;
#pragma unroll
            for (int i = 0; i < MI; i++) a[s][i] = *reinterpret_cast<const v4i *>(src + fa + i * 4096 + slot);
#pragma unroll
            for (int j = 0; j < NI; j++) b[s][j] = *reinterpret_cast<const v4i *>(src + fb + j * 4096 + slot);
            if (TAIL && 32 * s + 16 * lh >= left) {
#pragma unroll
                for (int i = 0; i < MI; i++) a[s][i] = (v4i){0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < NI; j++) b[s][j] = (v4i){0, 0, 0, 0};
            }
        }
    }
};

// What a wave does between two stages: behind the barrier the next stage is in LDS
// and every wave has the current one in registers, so its buffer takes the loads
// of the stage that many ahead, and the next one's fragments are read beside the
// current one's products.  `rd` and `wr` are restrict, so that the compiler does not
// wait for the loads that are in flight to other buffers before it reads.
//
// The accumulators take turns (SETS of them), as an MFMA waits for the one before
// it on the same accumulator.  b0, b1: the byte where the next stage and the one
// to load begin (past the row, its last one again: the count of loads in flight
// stays the same).
template <class Op, int MI, int NI, bool TAIL, int SETS>
__device__ __forceinline__ void mid_step(const MidStage<MI, NI, TAIL> &S, const uint8_t *__restrict__ rd,
                                         uint8_t *__restrict__ wr, int64_t b0, int64_t b1, int64_t Kb,
                                         typename Op::acc_t (&acc)[SETS][MI][NI], const v4i (&a)[4][MI],
                                         const v4i (&b)[4][NI], v4i (&an)[4][MI], v4i (&bn)[4][NI]) {
    constexpr int BUFS = lmid::bufs<MI, NI>(), P = MidStage<MI, NI, TAIL>::P;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(vmcnt_imm((BUFS - 2) * P) & ~(15 << 8));  // the next stage has landed, reads are done
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    S.read(rd, Kb - b0, an, bn);
    S.issue(wr, b1, Kb - b1);
#pragma unroll
    for (int s = 0; s < 4; s++)
#pragma unroll
        for (int i = 0; i < MI; i++)
#pragma unroll
            for (int j = 0; j < NI; j++) Op::mfma(acc[s % SETS][i][j], a[s][i], b[s][j]);
}

// A tile of 64 MI x 64 NI: KG groups of 4 waves; group g takes stages g, g + KG, ...
// amax: the maxima of the 256 x 256 tiles (bf16 output), already zero, or NULL.
template <class Op, int MI, int NI, int OUT, int EPI, bool TAIL>
__global__ __launch_bounds__((256 * lmid::groups<MI, NI>()), (lmid::groups<MI, NI>())) void linear_staged_kernel(
    typename Op::Arg op, int64_t M, int64_t N, int64_t K, void *__restrict__ y, LinearEpi L, unsigned tiles_m,
    unsigned tiles_n, float *__restrict__ amax) {
    using namespace lmid;
    constexpr int BM = 64 * MI, BN = 64 * NI, ES = OUT == 1 ? 2 : 4, PER = 16 / ES, BUFS = bufs<MI, NI>(), STAGE = stage<MI, NI>();
    constexpr int P = MidStage<MI, NI, TAIL>::P, KG = groups<MI, NI>(), SETS = MI * NI == 1 ? 2 : 1;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), group = wave >> 2;
    const int wm = wave >> 1 & 1, wn = wave & 1, lm = lane & 31, lh = lane >> 5;
    const TileCoord tc = tile_of(blockIdx.x, gridDim.x, tiles_m, tiles_n, 8);
    const int64_t m0 = (int64_t)tc.m * BM, n0 = (int64_t)tc.n * BN;
    // turns of all groups; a group's last one may be past the row, and is then left out of its sums
    const int64_t Kb = Op::extent(K), nk = (Kb + 127) / 128, turns = (nk + KG - 1) / KG;
    auto byte = [&](int64_t t) {  // where the group's stage t begins, or its last one
        const int64_t kt = t * KG + group;
        return (kt < nk ? kt : nk - 1) * 128;
    };
    MidStage<MI, NI, TAIL> S;
    S.begin(reinterpret_cast<const uint8_t *>(op.x), reinterpret_cast<const uint8_t *>(op.w), Kb, M, N, m0, n0);
    typename Op::acc_t acc[SETS][MI][NI];
#pragma unroll
    for (int k = 0; k < SETS; k++)
#pragma unroll
        for (int i = 0; i < MI; i++)
#pragma unroll
            for (int j = 0; j < NI; j++)
#pragma unroll
                for (int r = 0; r < 16; r++) acc[k][i][j][r] = 0;
    uint8_t *own = lds + group * BUFS * STAGE;
#pragma unroll
    for (int d = 0; d < BUFS; d++) S.issue(own + d * STAGE, byte(d), Kb - byte(d));
    __builtin_amdgcn_s_waitcnt(vmcnt_imm((BUFS - 1) * P));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    v4i a0[4][MI], b0[4][NI], a1[4][MI], b1[4][NI];
    S.read(own, Kb - byte(0), a0, b0);
    // the last turn by itself: a group past the row's end has nothing in it
    int cur = 0;  // the buffer of turn t
    int64_t t = 0;
    auto next = [](int n) { return n + 1 < BUFS ? n + 1 : 0; };
    for (; t + 2 < turns; t += 2) {
#pragma unroll
        for (int s = 0; s < P; s++) asm("" : "+v"(S.off[s]));  // (keeps the offsets 32 bits wide)
        const int n1 = next(cur), n2 = next(n1);
        mid_step<Op, MI, NI, TAIL, SETS>(S, own + n1 * STAGE, own + cur * STAGE, byte(t + 1), byte(t + BUFS), Kb, acc, a0, b0, a1, b1);
        mid_step<Op, MI, NI, TAIL, SETS>(S, own + n2 * STAGE, own + n1 * STAGE, byte(t + 2), byte(t + 1 + BUFS), Kb, acc, a1, b1, a0, b0);
        cur = n2;
    }
    if (t + 1 < turns)
        mid_step<Op, MI, NI, TAIL, SETS>(S, own + next(cur) * STAGE, own + cur * STAGE, byte(t + 1), byte(t + BUFS), Kb, acc, a0, b0, a1, b1);
    if ((turns - 1) * KG + group < nk) {
        const bool odd = t + 1 < turns;
#pragma unroll
        for (int s = 0; s < 4; s++)
#pragma unroll
            for (int i = 0; i < MI; i++)
#pragma unroll
                for (int j = 0; j < NI; j++) Op::mfma(acc[s % SETS][i][j], odd ? a1[s][i] : a0[s][i], odd ? b1[s][j] : b0[s][j]);
    }
    __builtin_amdgcn_s_waitcnt(0);  // every load has landed, and no wave reads on: the buffers take the tile's sums
    __syncthreads();
    constexpr int LPR = BN / PER, RPP = 64 / LPR, ROWS = BM / (4 * KG);  // lanes of a row, rows of a step, of a wave
    const int chunk = lane % LPR;
    const int64_t col = n0 + chunk * PER;
    const bool vec = ((N * ES) & 15) == 0;
    // The epilogue's operands before the sums go through LDS: the residual of a group
    // of steps is on its way together, a group ahead, and each row's request is
    // looked up once.
    constexpr int STEPS = ROWS / RPP, GROUP = STEPS < 4 ? STEPS : 4;
    uint4 residual[GROUP];
    auto ahead = [&](int q0) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < GROUP; q++) {
            const int64_t row = m0 + wave * ROWS + (q0 + q) * RPP + lane / LPR;
            residual[q] = make_uint4(0, 0, 0, 0);
            if (L.residual && row < M && col < N) residual[q] = fetch_raw<ES>(L.residual, row * N + col, N - col, vec);
        }
    };
    ahead(0);
    LinearLane<PER> T0;
    T0.begin(L, m0, BM, M, N, col);
    int requests = 0;  // of the wave's rows, in its first ROWS lanes
    if (T0.mode == kGateMixed) {
        const int64_t row = m0 + wave * ROWS + lane % ROWS;
        requests = request_of(L.gate_start, L.S, (int)(row < M ? row : M - 1));
    }
    QkLane<PER> Q;
    if constexpr ((EPI & kEpiHeads) != 0) Q.begin(L.qk, col);
    constexpr int STRIDE = BN * 4 + 16, BAND = (int)band<MI, NI>();
    typedef decltype(acc[0][0][0][0] + 0) T;
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int j = 0; j < NI; j++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                T v[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    v[e] = acc[0][i][j][4 * g + e];
                    if (SETS == 2) v[e] += acc[SETS - 1][i][j][4 * g + e];
                }
                *reinterpret_cast<uint4 *>(lds + group * BAND + (wm * 32 * MI + 32 * i + lm) * STRIDE +
                                           4 * (wn * 32 * NI + 32 * j + 8 * g + 4 * lh)) =
                    make_uint4(__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]),
                               __builtin_bit_cast(uint32_t, v[2]), __builtin_bit_cast(uint32_t, v[3]));
            }
    __syncthreads();
    constexpr int FORM = EPI | (OUT == 1 && (EPI & kEpiHeads) == 0 ? kEpiAmax : 0);
    float top = 0.0f;
#pragma unroll 1
    for (int q0 = 0; q0 < STEPS; q0 += GROUP) {
        uint4 now[GROUP];
#pragma unroll
        for (int q = 0; q < GROUP; q++) now[q] = residual[q];
        if (q0 + GROUP < STEPS) ahead(q0 + GROUP);
#pragma unroll
        for (int q = 0; q < GROUP; q++) {
            const int r0 = (q0 + q) * RPP;
            const int r = wave * ROWS + r0 + lane / LPR;
            const int64_t row = m0 + r, mr = row < M ? row : M - 1;
            T sum[PER];
#pragma unroll
            for (int i = 0; i < PER; i += 4) {
#pragma unroll
                for (int k = 0; k < KG; k++) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(lds + k * BAND + r * STRIDE + 4 * (PER * chunk + i));
                    const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const T p = __builtin_bit_cast(T, d[e]);
                        sum[i + e] = k == 0 ? p : sum[i + e] + p;
                    }
                }
            }
            float v[PER];
            Op::template scale<PER>(op, mr, col, N, sum, v);
            if constexpr ((EPI & kEpiLora) != 0) lora_row<PER>(L.lora, mr, col, N, v);
            T0.turn(L, __shfl(requests, r0 + lane / LPR, 64), N, col);
            top = fmaxf(top, linear_row_out<ES, FORM>(v, y, M, N, row, col, chunk, vec, L, T0, Q, amax != nullptr,
                                                      &now[q]));
        }
    }
    mid_amax_max(amax, top, m0, n0, M);
}

// ---- NVFP4: operands straight into fragments ---------------------------------------

// An operand of a tile: a scalar base (the tile's first row, then the stage) and
// each lane's 32-bit offset of its rows, so that a load takes no 64-bit vector
// arithmetic (with it, two stages in flight do not fit the registers).
template <class T>
__device__ __forceinline__ T at_base(const uint8_t *base, uint32_t off) {
    asm("" : "+s"(base));
    return *reinterpret_cast<const T *>(base + off);
}

// NVFP4: a stage is 128 values of a row, 64 code bytes and 8 scales.  The lane
// takes 32 values (16 bytes, two scales) of each half of it; TAIL as above, in
// groups of 16.
struct MidCodes {
    const uint8_t *c, *s;
    uint32_t co, so;  // the row's, with the lane's half
    struct raw {
        uint32_t w[8];  // codes of piece 0, of piece 1
        uint32_t e[2];  // their scales, two bytes each
    };
    template <bool TAIL>
    __device__ __forceinline__ void get(raw &r, int64_t k, int64_t left, int h, bool on) const {
        const uint8_t *cb = c + (on ? k / 2 : 0), *sb = s + (on ? k / 16 : 0);
        if constexpr (!TAIL) {  // rows of codes are 64-byte aligned, of scales 8-byte
#pragma unroll
            for (int q = 0; q < 2; q++) {
                const v4i u = at_base<v4i>(cb, on ? co + 32 * q : 0);
                r.w[4 * q] = u[0], r.w[4 * q + 1] = u[1], r.w[4 * q + 2] = u[2], r.w[4 * q + 3] = u[3];
                r.e[q] = at_base<uint16_t>(sb, on ? so + 4 * q : 0);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 2; q++)
#pragma unroll
                for (int g = 0; g < 2; g++) {
                    const bool in = on && 64 * q + 32 * h + 16 * g < left;
                    const uint2 u = at_base<uint2>(cb, in ? co + 32 * q + 8 * g : on ? co - 16 * h : 0);
                    r.w[4 * q + 2 * g] = u.x, r.w[4 * q + 2 * g + 1] = u.y;
                    const uint32_t e = at_base<uint8_t>(sb, in ? so + 4 * q + g : on ? so - 2 * h : 0);
                    r.e[q] = g ? r.e[q] | e << 8 : e;
                }
        }
    }
    __device__ static __forceinline__ void cut(raw &r, int64_t left, int h) {
#pragma unroll
        for (int q = 0; q < 2; q++)
#pragma unroll
            for (int g = 0; g < 2; g++)
                if (64 * q + 32 * h + 16 * g >= left) {
                    r.w[4 * q + 2 * g] = r.w[4 * q + 2 * g + 1] = 0;
                    r.e[q] &= g ? 0xFFu : 0xFF00u;
                }
    }
    __device__ __forceinline__ void begin(const uint8_t *codes, const uint8_t *scales, int64_t K, int64_t first, int64_t row,
                                          int h) {
        c = codes + first * (K / 2), s = scales + first * (K / 16);
        co = (uint32_t)((row - first) * (K / 2)) + 16 * h, so = (uint32_t)((row - first) * (K / 16)) + 2 * h;
    }
    // the 8 values of code word i: the products of code and scale are exact in fp16
    __device__ static __forceinline__ v4i frag(const raw &r, int i) {
        const lm_h2 t = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r.e[i >> 2], 1.0f, false);
        const lm_h2 sc = i & 2 ? __builtin_shufflevector(t, t, 1, 1) : __builtin_shufflevector(t, t, 0, 0);
        const lm_h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(r.w[i], 1.0f, 0) * sc;
        const lm_h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(r.w[i], 1.0f, 1) * sc;
        const lm_h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(r.w[i], 1.0f, 2) * sc;
        const lm_h2 e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(r.w[i], 1.0f, 3) * sc;
        return (v4i){__builtin_bit_cast(int, a), __builtin_bit_cast(int, b), __builtin_bit_cast(int, d),
                     __builtin_bit_cast(int, e)};
    }
};

struct MidFP4 {
    static constexpr LinearRoute ROUTE = kLinearNVFP4;
    typedef v16f acc_t;
    typedef MidCodes Row;
    struct Arg {
        const uint8_t *x, *sx;
        const float *gx;
        const uint8_t *w, *sw;
        const float *gw;
    };
    static constexpr int STEPS = 8;
    __host__ __device__ static __forceinline__ int64_t extent(int64_t K) { return K; }
    __device__ static __forceinline__ void x_row(Row &r, const Arg &a, int64_t K, int64_t first, int64_t row, int h) {
        r.begin(a.x, a.sx, K, first, row, h);
    }
    __device__ static __forceinline__ void w_row(Row &r, const Arg &a, int64_t K, int64_t first, int64_t row, int h) {
        r.begin(a.w, a.sw, K, first, row, h);
    }
    __device__ static __forceinline__ void mfma(acc_t &c, const v4i &x, const v4i &w) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(lm_h8, w), __builtin_bit_cast(lm_h8, x), c, 0, 0, 0);
    }
    template <int N>
    __device__ static __forceinline__ void scale(const Arg &a, int64_t, int64_t, int64_t, const float (&sum)[N], float (&v)[N]) {
        const float gx = *a.gx, gw = *a.gw;
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = (sum[i] * gx) * gw;
    }
};

namespace lmid {
// the waves' sums
template <int MI, int NI>
constexpr int stride() { return 128 * NI + 16; }
template <int MI, int NI>
constexpr size_t lds_bytes() {
    return (size_t)WAVES * 32 * MI * stride<MI, NI>();
}
}  // namespace lmid

// A tile of 32 MI x 32 NI.  amax: the maxima of the 256 x 256 tiles (bf16 output),
// already zero, or NULL.
template <class Op, int MI, int NI, int OUT, int EPI, bool TAIL>
__global__ __launch_bounds__(64 * lmid::WAVES, 2) void linear_codes_kernel(typename Op::Arg op, int64_t M, int64_t N,
                                                                         int64_t K, void *__restrict__ y, LinearEpi L,
                                                                         unsigned tiles_m, unsigned tiles_n,
                                                                         float *__restrict__ amax) {
    using namespace lmid;
    constexpr int BM = 32 * MI, BN = 32 * NI, ES = OUT == 1 ? 2 : 4, PER = 16 / ES, STRIDE = stride<MI, NI>();
    constexpr int SETS = MI + NI > 4 ? 1 : 2;  // stages in flight
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lm = lane & 31, lh = lane >> 5;
    const TileCoord tc = tile_of(blockIdx.x, gridDim.x, tiles_m, tiles_n, 8);
    const int64_t m0 = (int64_t)tc.m * BM, n0 = (int64_t)tc.n * BN;
    const int64_t E = Op::extent(K), nk = (E + 127) / 128;
    typename Op::Row xr[MI], wr[NI];  // rows past the end read the last one
#pragma unroll
    for (int i = 0; i < MI; i++) Op::x_row(xr[i], op, K, m0, m0 + 32 * i + lm < M ? m0 + 32 * i + lm : M - 1, lh);
#pragma unroll
    for (int j = 0; j < NI; j++) Op::w_row(wr[j], op, K, n0, n0 + 32 * j + lm < N ? n0 + 32 * j + lm : N - 1, lh);
    typename Op::acc_t acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int j = 0; j < NI; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[i][j][r] = 0;
    // the wave's stages are wave, wave + 8, ...: `mine` of them
    const int64_t mine = nk > wave ? (nk - wave + WAVES - 1) / WAVES : 0;
    typedef typename Op::Row::raw raw;
    raw a[SETS][MI], b[SETS][NI];
    auto get = [&](int set, int64_t i) {
        const int64_t k = (wave + WAVES * i) * 128;
        const bool on = i < mine;
#pragma unroll
        for (int r = 0; r < MI; r++) xr[r].template get<TAIL>(a[set][r], k, E - k, lh, on);
#pragma unroll
        for (int r = 0; r < NI; r++) wr[r].template get<TAIL>(b[set][r], k, E - k, lh, on);
    };
    auto use = [&](int set, int64_t i) {
        const int64_t left = E - (wave + WAVES * i) * 128;
        if (TAIL && left < 128) {
#pragma unroll
            for (int r = 0; r < MI; r++) Op::Row::cut(a[set][r], left, lh);
#pragma unroll
            for (int r = 0; r < NI; r++) Op::Row::cut(b[set][r], left, lh);
        }
#pragma unroll
        for (int s = 0; s < Op::STEPS; s++) {
            v4i fa[MI], fb[NI];
#pragma unroll
            for (int r = 0; r < MI; r++) fa[r] = Op::Row::frag(a[set][r], s);
#pragma unroll
            for (int r = 0; r < NI; r++) fb[r] = Op::Row::frag(b[set][r], s);
#pragma unroll
            for (int r = 0; r < MI; r++)
#pragma unroll
                for (int j = 0; j < NI; j++) Op::mfma(acc[r][j], fa[r], fb[j]);
            // NVFP4: one step's values at a time, or their dequantized forms spill
            if (Op::STEPS == 8) __builtin_amdgcn_sched_barrier(0);
        }
    };
    // No branch between a set's loads and their use, or the compiler waits for all
    // loads there: a stage that is not there loads a few bytes that nobody uses.
#pragma unroll
    for (int d = 0; d < SETS; d++) get(d, d);
    int64_t i0 = 0;
    for (; i0 + SETS <= mine; i0 += SETS) {
#pragma unroll
        for (int d = 0; d < SETS; d++) {
            use(d, i0 + d);
            get(d, i0 + d + SETS);
        }
    }
    if (SETS == 2 && i0 < mine) use(0, i0);
    constexpr int LPR = BN / PER, RPP = 64 / LPR;  // lanes of a row, rows of a wave's step
    const int chunk = lane % LPR;
    const int64_t col = n0 + chunk * PER;
    const bool vec = ((N * ES) & 15) == 0;
    uint4 residual[BM / (RPP * WAVES)];  // before the sums go through LDS
#pragma unroll
    for (int q = 0; q < BM / (RPP * WAVES); q++) {
        const int64_t row = m0 + (q * WAVES + wave) * RPP + lane / LPR;
        residual[q] = make_uint4(0, 0, 0, 0);
        if (L.residual && row < M && col < N) residual[q] = fetch_raw<ES>(L.residual, row * N + col, N - col, vec);
    }
    typedef decltype(acc[0][0][0] + 0) T;
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int j = 0; j < NI; j++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const T v0 = acc[i][j][4 * g], v1 = acc[i][j][4 * g + 1], v2 = acc[i][j][4 * g + 2], v3 = acc[i][j][4 * g + 3];
                *reinterpret_cast<uint4 *>(lds + (wave * BM + 32 * i + lm) * STRIDE + 4 * (32 * j + 8 * g + 4 * lh)) =
                    make_uint4(__builtin_bit_cast(uint32_t, v0), __builtin_bit_cast(uint32_t, v1),
                               __builtin_bit_cast(uint32_t, v2), __builtin_bit_cast(uint32_t, v3));
            }
    LinearLane<PER> P;
    P.begin(L, m0, BM, M, N, col);
    QkLane<PER> Q;
    if constexpr ((EPI & kEpiHeads) != 0) Q.begin(L.qk, col);
    __syncthreads();
    constexpr int FORM = EPI | (OUT == 1 && (EPI & kEpiHeads) == 0 ? kEpiAmax : 0);
    float top = 0.0f;
#pragma unroll
    for (int r0 = 0; r0 < BM; r0 += RPP * WAVES) {
        const int r = r0 + wave * RPP + lane / LPR;
        const int64_t row = m0 + r, mr = row < M ? row : M - 1;
        const uint8_t *at = lds + r * STRIDE + 4 * PER * chunk;
        T sum[PER];
#pragma unroll
        for (int w = 0; w < WAVES; w++)
#pragma unroll
            for (int i = 0; i < PER; i += 4) {
                const uint4 u = *reinterpret_cast<const uint4 *>(at + w * BM * STRIDE + 4 * i);
                const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const T t = __builtin_bit_cast(T, d[e]);
                    sum[i + e] = w == 0 ? t : sum[i + e] + t;
                }
            }
        float v[PER];
        Op::template scale<PER>(op, mr, col, N, sum, v);
        if constexpr ((EPI & kEpiLora) != 0) lora_row<PER>(L.lora, mr, col, N, v);
        if (P.mode == kGateMixed) P.turn(L, request_of(L.gate_start, L.S, (int)mr), N, col);
        top = fmaxf(top, linear_row_out<ES, FORM>(v, y, M, N, row, col, chunk, vec, L, P, Q, amax != nullptr,
                                                  &residual[r0 / (RPP * WAVES)]));
    }
    mid_amax_max(amax, top, m0, n0, M);
}

// ---- launches ------------------------------------------------------------------------

template <class Op, int MI, int NI, int OUT, int EPI, bool TAIL>
static hipError_t launch_mid_one(hipStream_t s, const typename Op::Arg &op, int64_t M, int64_t N, int64_t K, void *y,
                                 const LinearEpi &L, float *amax) {
    constexpr bool CODES = Op::ROUTE == kLinearNVFP4;
    constexpr int BM = (CODES ? 32 : 64) * MI, BN = (CODES ? 32 : 64) * NI;
    const int64_t tm = (M + BM - 1) / BM, tn = (N + BN - 1) / BN;
    const dim3 grid((unsigned)(tm * tn));
    if constexpr (CODES) {
        constexpr size_t bytes = lmid::lds_bytes<MI, NI>();
        static const hipError_t attr =
            hipFuncSetAttribute(reinterpret_cast<const void *>(linear_codes_kernel<Op, MI, NI, OUT, EPI, TAIL>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (attr != hipSuccess) return attr;
        hipLaunchKernelGGL((linear_codes_kernel<Op, MI, NI, OUT, EPI, TAIL>), grid, dim3(64 * lmid::WAVES), bytes, s, op, M, N,
                           K, y, L, (unsigned)tm, (unsigned)tn, amax);
    } else {
        constexpr size_t bytes = lmid::staged_lds<MI, NI>();
        static const hipError_t attr =
            hipFuncSetAttribute(reinterpret_cast<const void *>(linear_staged_kernel<Op, MI, NI, OUT, EPI, TAIL>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (attr != hipSuccess) return attr;
        hipLaunchKernelGGL((linear_staged_kernel<Op, MI, NI, OUT, EPI, TAIL>), grid, dim3(256 * lmid::groups<MI, NI>()), bytes, s,
                           op, M, N, K, y, L, (unsigned)tm, (unsigned)tn, amax);
    }
    return hipGetLastError();
}

template <class Op, int OUT, int EPI, bool TAIL>
static hipError_t launch_mid_tail(hipStream_t s, const typename Op::Arg &op, int64_t M, int64_t N, int64_t K, void *y,
                                  const LinearEpi &L, float *amax) {
    const bool wide = (EPI & kEpiHeads) != 0 && L.qk.D == 128;
    const MidTile t = mid_tile(Op::ROUTE, wide, M, N);
    if constexpr (Op::ROUTE == kLinearNVFP4) {
        if constexpr ((EPI & kEpiHeads) != 0)
            if (t.rows == 32) return launch_mid_one<Op, 1, 4, OUT, EPI, TAIL>(s, op, M, N, K, y, L, amax);
        return launch_mid_one<Op, 2, 2, OUT, EPI, TAIL>(s, op, M, N, K, y, L, amax);
    } else {
        if (t.rows == 128) return launch_mid_one<Op, 2, 2, OUT, EPI, TAIL>(s, op, M, N, K, y, L, amax);
        if (t.cols == 128) return launch_mid_one<Op, 1, 2, OUT, EPI, TAIL>(s, op, M, N, K, y, L, amax);
        return launch_mid_one<Op, 1, 1, OUT, EPI, TAIL>(s, op, M, N, K, y, L, amax);
    }
}

template <class Op, int OUT, int EPI>
static hipError_t launch_mid_form(hipStream_t s, const typename Op::Arg &op, int64_t M, int64_t N, int64_t K, void *y,
                                  const LinearEpi &L, float *amax) {
    return Op::extent(K) % 128 != 0 ? launch_mid_tail<Op, OUT, EPI, true>(s, op, M, N, K, y, L, amax)
                                    : launch_mid_tail<Op, OUT, EPI, false>(s, op, M, N, K, y, L, amax);
}

template <class Op>
static hipError_t launch_mid(hipStream_t s, const typename Op::Arg &op, int64_t M, int64_t N, int64_t K, int out_dtype,
                             void *y, const LinearEpi &L, float *amax) {
    const int epi = kEpiLinear | (L.lora.t ? kEpiLora : 0) | (L.qk.D ? kEpiHeads : 0);
#define DMPQ_MID(OUT_, EPI_) return launch_mid_form<Op, OUT_, (EPI_)>(s, op, M, N, K, y, L, amax)
    if (out_dtype == 0) {
        if (epi == kEpiLinear) DMPQ_MID(0, kEpiLinear);
        if (epi == (kEpiLinear | kEpiLora)) DMPQ_MID(0, kEpiLinear | kEpiLora);
    }
    if (out_dtype != 1) return hipErrorInvalidValue;
    switch (epi) {
        case kEpiLinear: DMPQ_MID(1, kEpiLinear);
        case kEpiLinear | kEpiLora: DMPQ_MID(1, kEpiLinear | kEpiLora);
        case kEpiLinear | kEpiHeads: DMPQ_MID(1, kEpiLinear | kEpiHeads);
        case kEpiLinear | kEpiHeads | kEpiLora: DMPQ_MID(1, kEpiLinear | kEpiHeads | kEpiLora);
    }
#undef DMPQ_MID
    return hipErrorInvalidValue;
}

}  // namespace dmpq
