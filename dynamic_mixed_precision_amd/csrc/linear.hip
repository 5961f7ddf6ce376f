// linear.hip -- the whole linear for few rows, and the gradients of its
// epilogue.
//
// Few rows (a request's conditioning vector, a handful of tokens): what costs
// time is reading the weight once, w [N x K] from HBM, so the work is cut by
// columns: a workgroup takes 16 columns (or the columns of one head) and its 8
// waves share K between them in pieces of 64 bytes of every row.  The products
// are 16x16 MFMAs straight from memory (no operand is used twice in a
// workgroup, so LDS would add a trip); the waves' sums meet in LDS in a fixed
// order, and the epilogue is that of linear.hpp on four columns a lane.
#include "device.hpp"
#include "internal.hpp"
#include "linear.hpp"
#include "lora.hpp"

namespace dmpq {

namespace skinny {
constexpr int WAVES = 8;
}  // namespace skinny

typedef int v2i __attribute__((ext_vector_type(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

// An operand of `rows` rows: its place, rows past the end read the last one
// (their results are never stored).
struct SkinnyBF16 {
    typedef v4f acc_t;
    struct Arg {
        const uint16_t *x, *w;
    };
    static constexpr int KSTEP = 32;  // K of one piece
    typedef v4i frag_t;
    __device__ static __forceinline__ frag_t load(const uint16_t *p, int64_t row, int64_t K, int64_t k) {
        return k < K ? *reinterpret_cast<const v4i *>(p + row * K + k) : (v4i){0, 0, 0, 0};
    }
    __device__ static __forceinline__ frag_t load_x(const Arg &a, int64_t row, int64_t K, int64_t k0, int q) {
        return load(a.x, row, K, k0 + 8 * q);
    }
    __device__ static __forceinline__ frag_t load_w(const Arg &a, int64_t row, int64_t K, int64_t k0, int q) {
        return load(a.w, row, K, k0 + 8 * q);
    }
    __device__ static __forceinline__ void mac(acc_t &c, const frag_t &x, const frag_t &w) { c = mfma16(w, x, c); }
    __device__ static __forceinline__ float value(const Arg &, float sum, int64_t, int64_t) { return sum; }
};

struct SkinnyI8 {
    typedef v4i acc_t;
    struct Arg {
        const int8_t *x, *w;
        const float *sx, *sw;
    };
    static constexpr int KSTEP = 64;
    typedef v4i frag_t;
    __device__ static __forceinline__ frag_t load(const int8_t *p, int64_t row, int64_t K, int64_t k) {
        return k < K ? *reinterpret_cast<const v4i *>(p + row * K + k) : (v4i){0, 0, 0, 0};
    }
    __device__ static __forceinline__ frag_t load_x(const Arg &a, int64_t row, int64_t K, int64_t k0, int q) {
        return load(a.x, row, K, k0 + 16 * q);
    }
    __device__ static __forceinline__ frag_t load_w(const Arg &a, int64_t row, int64_t K, int64_t k0, int q) {
        return load(a.w, row, K, k0 + 16 * q);
    }
    __device__ static __forceinline__ void mac(acc_t &c, const frag_t &x, const frag_t &w) {
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, c, 0, 0, 0);
    }
    __device__ static __forceinline__ float value(const Arg &a, int sum, int64_t m, int64_t n) {
        return ((float)sum * a.sx[m]) * a.sw[n];
    }
};

// 32 codes (two scale groups) of a row a lane: a piece is 128 values of K.
// The fp16 products of code and scale are exact, as in the large kernels.
struct SkinnyFP4 {
    typedef v4f acc_t;
    struct Arg {
        const uint8_t *x, *sx;
        const float *gx;
        const uint8_t *w, *sw;
        const float *gw;
    };
    static constexpr int KSTEP = 128;
    struct frag_t {
        uint32_t c[4], s;
    };
    __device__ static __forceinline__ frag_t load(const uint8_t *p, const uint8_t *s, int64_t row, int64_t K, int64_t k) {
        frag_t f = {{0, 0, 0, 0}, 0};
        const uint8_t *c = p + row * (K / 2) + k / 2, *b = s + row * (K / 16) + k / 16;
        if (k < K) {  // rows are 8-byte aligned
            const uint2 u = *reinterpret_cast<const uint2 *>(c);
            f.c[0] = u.x, f.c[1] = u.y, f.s = b[0];
        }
        if (k + 16 < K) {
            const uint2 u = *reinterpret_cast<const uint2 *>(c + 8);
            f.c[2] = u.x, f.c[3] = u.y, f.s |= (uint32_t)b[1] << 8;
        }
        return f;
    }
    __device__ static __forceinline__ frag_t load_x(const Arg &a, int64_t row, int64_t K, int64_t k0, int q) {
        return load(a.x, a.sx, row, K, k0 + 32 * q);
    }
    __device__ static __forceinline__ frag_t load_w(const Arg &a, int64_t row, int64_t K, int64_t k0, int q) {
        return load(a.w, a.sw, row, K, k0 + 32 * q);
    }
    // the 8 values of code word i as fp16
    __device__ static __forceinline__ h8 values(const frag_t &f, int i) {
        const h2 s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(f.s, 1.0f, false);
        const h2 sc = i < 2 ? __builtin_shufflevector(s, s, 0, 0) : __builtin_shufflevector(s, s, 1, 1);
        const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(f.c[i], 1.0f, 0) * sc;
        const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(f.c[i], 1.0f, 1) * sc;
        const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(f.c[i], 1.0f, 2) * sc;
        const h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(f.c[i], 1.0f, 3) * sc;
        return (h8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
    __device__ static __forceinline__ void mac(acc_t &c, const frag_t &x, const frag_t &w) {
#pragma unroll
        for (int i = 0; i < 4; i++) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(values(w, i), values(x, i), c, 0, 0, 0);
    }
    __device__ static __forceinline__ float value(const Arg &a, float sum, int64_t, int64_t) {
        return (sum * *a.gx) * *a.gw;
    }
};

// scale * t b^T of one row and four columns, in fp32.
__device__ __forceinline__ void lora_few(const LoraEpi &L, int64_t row, int64_t col, int64_t N, float (&v)[4]) {
    const LoraBatch &B = L.batch;
    const int a = row_adapter(B, (int)row);
    if (a < 0) return;
    const int rank = adapter_rank(B, a);
    if (rank == 0) return;
    const float sc = B.scale[a];
    const float *t = L.t + row * B.R;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t n = col + i < N ? col + i : N - 1;
        const uint16_t *b = L.b + ((int64_t)a * N + n) * B.R;
        float s = 0.0f;
        for (int r = 0; r < rank; r++) s = __builtin_fmaf(t[r], __uint_as_float((uint32_t)b[r] << 16), s);
        v[i] += sc * s;
    }
}

// 16 NT columns and 16 MT rows a workgroup.
template <class Op, int NT, int MT, int OUT, bool HEADS>
__global__ __launch_bounds__(64 * skinny::WAVES) void skinny_kernel(typename Op::Arg op, int64_t M, int64_t N, int64_t K,
                                                                    void *__restrict__ y, LinearEpi L) {
    using namespace skinny;
    // pieces of K in flight per wave (NVFP4 fragments of 8 blocks, four deep, spill 52 registers)
    constexpr int STEPS = NT * MT >= 8 && Op::KSTEP == 128 ? 2 : 4;
    constexpr int ES = OUT == 1 ? 2 : 4, TR = 16 * MT, TC = 16 * NT, QUADS = TR * TC / 4;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * TC, m0 = (int64_t)blockIdx.y * TR;
    int64_t xr[MT], wr[NT];
#pragma unroll
    for (int i = 0; i < MT; i++) xr[i] = m0 + 16 * i + l16 < M ? m0 + 16 * i + l16 : M - 1;
#pragma unroll
    for (int j = 0; j < NT; j++) wr[j] = n0 + 16 * j + l16 < N ? n0 + 16 * j + l16 : N - 1;
    typename Op::acc_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int j = 0; j < NT; j++) acc[i][j] = typename Op::acc_t{0, 0, 0, 0};
    // pieces wave, wave + WAVES, ...: together the waves read whole lines of w
    for (int64_t k = (int64_t)wave * Op::KSTEP; k < K; k += (int64_t)STEPS * WAVES * Op::KSTEP) {
        typename Op::frag_t x[STEPS][MT], w[STEPS][NT];
#pragma unroll
        for (int s = 0; s < STEPS; s++) {
            const int64_t ks = k + (int64_t)s * WAVES * Op::KSTEP;  // past K: zeros
#pragma unroll
            for (int j = 0; j < NT; j++) w[s][j] = Op::load_w(op, wr[j], K, ks, q);
#pragma unroll
            for (int i = 0; i < MT; i++) x[s][i] = Op::load_x(op, xr[i], K, ks, q);
        }
#pragma unroll
        for (int s = 0; s < STEPS; s++)
#pragma unroll
            for (int i = 0; i < MT; i++)
#pragma unroll
                for (int j = 0; j < NT; j++) Op::mac(acc[i][j], x[s][i], w[s][j]);
    }
    // lane l has row l % 16 and columns 4 (l / 16) + 0..3 of every block
    typedef decltype(acc[0][0][0] + 0) T;
    T *red = reinterpret_cast<T *>(lds);
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int j = 0; j < NT; j++)
            *reinterpret_cast<typename Op::acc_t *>(red + ((wave * TR + 16 * i + l16) * TC + 16 * j + 4 * q)) = acc[i][j];
    __syncthreads();
    const bool vec = ((N * ES) & 15) == 0;
    // whole waves stay together: the heads' sums cross lanes
    for (int e = tid; e < (QUADS + 63) / 64 * 64; e += 64 * WAVES) {
        const int at = e < QUADS ? e : QUADS - 1;
        const int r = at / (TC / 4), c = 4 * (at % (TC / 4));
        const int64_t row = m0 + r, col = n0 + c;
        const int64_t mr = row < M ? row : M - 1;
        const bool in = e < QUADS && row < M && col < N;
        typename Op::acc_t sum = *reinterpret_cast<typename Op::acc_t *>(red + r * TC + c);
#pragma unroll
        for (int w = 1; w < WAVES; w++) sum += *reinterpret_cast<typename Op::acc_t *>(red + (w * TR + r) * TC + c);
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const T part = sum[i];
            v[i] = Op::value(op, part, mr, col + i < N ? col + i : N - 1);
        }
        if (L.lora.t) lora_few(L.lora, mr, col, N, v);
        if (L.bias && in) {
            float b[4];
            load_values<4>(L.bias, L.bias_bf16, col, N - col, b);
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] += b[i];
        }
        if (L.pre && in) store_values<ES, 4>(L.pre, row * N + col, N - col, vec, v);
        if constexpr (HEADS) {
            QkLane<4> Q;
            Q.begin(L.qk, col);
            Q.apply(L.qk, mr, v);
        } else {
            act_apply<4>(v, L.act);
        }
        LinearLane<4> G;
        G.mode = kGateNone, G.held = -2;
        if (L.gate) {
            G.mode = kGateMixed;
            G.turn(L, L.gate_start ? request_of(L.gate_start, L.S, (int)mr) : 0, N, col);
        }
        G.template finish<ES>(L, row, N, col, in, vec, v);
        if (in) store_values<ES, 4>(y, row * N + col, N - col, vec, v);
    }
}

template <class Op, int NT, int MT, int OUT, bool HEADS>
static hipError_t launch_skinny_one(hipStream_t s, const typename Op::Arg &op, int64_t M, int64_t N, int64_t K, void *y,
                                    const LinearEpi &L) {
    const dim3 grid((unsigned)((N + 16 * NT - 1) / (16 * NT)), (unsigned)((M + 16 * MT - 1) / (16 * MT)));
    const size_t lds = (size_t)skinny::WAVES * 16 * NT * 16 * MT * 4;
    hipLaunchKernelGGL((skinny_kernel<Op, NT, MT, OUT, HEADS>), grid, dim3(64 * skinny::WAVES), lds, s, op, M, N, K, y, L);
    return hipGetLastError();
}

template <class Op>
static hipError_t launch_skinny(hipStream_t s, const typename Op::Arg &op, int64_t M, int64_t N, int64_t K, int out_dtype,
                                void *y, const LinearEpi &L) {
    if (L.qk.D) {
        if (out_dtype != 1) return hipErrorInvalidValue;
        switch (L.qk.D) {
            case 32: return launch_skinny_one<Op, 2, 2, 1, true>(s, op, M, N, K, y, L);
            case 64: return launch_skinny_one<Op, 4, 2, 1, true>(s, op, M, N, K, y, L);
            case 128: return launch_skinny_one<Op, 8, 1, 1, true>(s, op, M, N, K, y, L);
        }
        return hipErrorInvalidValue;
    }
#define DMPQ_SKINNY(MT_)                                                                   \
    return out_dtype == 1 ? launch_skinny_one<Op, 1, MT_, 1, false>(s, op, M, N, K, y, L) \
                          : launch_skinny_one<Op, 1, MT_, 0, false>(s, op, M, N, K, y, L)
    if (M <= 16) DMPQ_SKINNY(1);
    if (M <= 32) DMPQ_SKINNY(2);
    DMPQ_SKINNY(4);
#undef DMPQ_SKINNY
}

hipError_t launch_few_bf16(hipStream_t s, const uint16_t *x, const uint16_t *w, int64_t M, int64_t N, int64_t K,
                           int out_dtype, void *y, const LinearEpi &L) {
    return launch_skinny<SkinnyBF16>(s, {x, w}, M, N, K, out_dtype, y, L);
}
hipError_t launch_few_int8(hipStream_t s, const int8_t *qa, const float *sa, const int8_t *qw, const float *sw, int64_t M,
                           int64_t N, int64_t K, int out_dtype, void *y, const LinearEpi &L) {
    return launch_skinny<SkinnyI8>(s, {qa, qw, sa, sw}, M, N, K, out_dtype, y, L);
}
hipError_t launch_few_nvfp4(hipStream_t s, const uint8_t *ca, const uint8_t *sa, const float *ga, const uint8_t *cw,
                            const uint8_t *sw, const float *gw, int64_t M, int64_t N, int64_t K, int out_dtype, void *y,
                            const LinearEpi &L) {
    return launch_skinny<SkinnyFP4>(s, {ca, sa, ga, cw, sw, gw}, M, N, K, out_dtype, y, L);
}

__global__ __launch_bounds__(256) void zero_kernel(float *__restrict__ p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0.0f;
}

hipError_t launch_zero(hipStream_t s, float *p, int64_t n) {
    hipLaunchKernelGGL(zero_kernel, dim3(stride_grid(n, 256, 256)), dim3(256), 0, s, p, n);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Gradients of y = residual + gate[s] * act(pre):
//   du = gate[s] act'(pre) dy            (0 in rows of no request)
//   dgate[s] = sum over the rows of s of dy act(pre)
//   dbias = sum over all rows of du
// dy and pre are read and du written once: bound by HBM.  A wave takes a chunk
// of `rows` consecutive rows of 512 columns, 8 a lane, and sums its columns in
// registers.  Sums are stored per chunk and added in chunk order by a second
// kernel: the same bits on every call.  A chunk that meets several requests
// stores one sum for each, at chunk + request, which no other pair has: along
// the rows one of the two goes up at every step.
// ---------------------------------------------------------------------------
namespace lgrad {
constexpr int COLS = 512;  // columns of a wave
constexpr int DEEP = 4;    // rows on their way together
}

// act(v) and act'(v).  Far out the derivative is its limit and what it is made
// of would be infinity times zero, so the factors that grow are taken at
// +-kActFar at most, where e^-kActFar is 0 in fp32 (NaN stays: it comes with the
// exponential).  The sigmoids share one exponential: with E = e^-z,
// s(z) = 1 / (1 + E) and s(-z) = E s(z); where E is past 1e30 s(z) is nothing next to it.
constexpr float kActFar = 128.0f;
template <int ACT>
__device__ __forceinline__ void act_and_slope(float v, float &a, float &d) {
    if constexpr (ACT == kActNone) {
        a = v, d = 1.0f;
    } else if constexpr (ACT == kActGelu) {
        const float u = v > kActFar ? kActFar : v < -kActFar ? -kActFar : v;
        const float phi2 = gelu_phi2(u);
        a = 0.5f * v * phi2;
        d = 0.5f * phi2 + u * 0.3989422804014327f * __builtin_amdgcn_exp2f(-0.5f * kLog2e * u * u);
    } else {
        const float u = __builtin_amdgcn_fmed3f(v, -kActFar, kActFar);
        const float t = ACT == kActSilu ? -kLog2e * v : gelu_tanh_exponent(v);
        const float E = __builtin_amdgcn_exp2f(t), e = __builtin_amdgcn_rcpf(1.0f + E);
        const float f = __builtin_fminf(E, 1e30f) * e;
        a = v * e;
        d = __builtin_fmaf(u * e * f, ACT == kActSilu ? 1.0f : __builtin_fmaf(kGt * 0.134145f * u, u, kGt), e);
    }
}

// VEC: rows are 16-byte aligned and a lane has 8 columns in a row; otherwise
// its columns are 64 apart, so that every access of a wave is contiguous.
template <int ES, bool VEC>
struct GradValues {  // as they lie, so that many rows fit the registers
    static constexpr int WORDS = ES == 2 && VEC ? 4 : 8;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const void *p, int64_t row, int64_t N, const int64_t (&cols)[8]) {
#pragma unroll
        for (int i = 0; i < WORDS; i++) w[i] = 0;
        if constexpr (VEC) {
            const uint8_t *q = static_cast<const uint8_t *>(p) + (row * N + cols[0]) * ES;
#pragma unroll
            for (int i = 0; i < WORDS; i += 4)
                if (cols[i] < N) {
                    const uint4 u = load_nt16(q + 4 * i);
                    w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
                }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (cols[i] < N)
                    w[i] = ES == 4 ? static_cast<const uint32_t *>(p)[row * N + cols[i]]
                                   : (uint32_t) static_cast<const uint16_t *>(p)[row * N + cols[i]] << 16;
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (WORDS == 8) return __uint_as_float(w[i]);
        return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    }
};

template <int ES, bool VEC>
__device__ __forceinline__ void grad_store(void *p, int64_t row, int64_t N, const int64_t (&cols)[8], const float (&v)[8]) {
    if constexpr (VEC) {
        if (cols[0] >= N) return;
        float a[16 / ES];
#pragma unroll
        for (int i = 0; i < 16 / ES; i++) a[i] = v[i];
        store_values<ES, 16 / ES>(p, row * N + cols[0], 16 / ES, true, a);
        if constexpr (ES == 4) {
            if (cols[0] + 4 >= N) return;
#pragma unroll
            for (int i = 0; i < 4; i++) a[i] = v[4 + i];
            store_values<ES, 4>(p, row * N + cols[0] + 4, 4, true, a);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (cols[i] < N) {
                if constexpr (ES == 4)
                    static_cast<float *>(p)[row * N + cols[i]] = v[i];
                else
                    static_cast<uint16_t *>(p)[row * N + cols[i]] = (uint16_t)f32_to_bf16(v[i]);
            }
    }
}

template <bool VEC>
__device__ __forceinline__ void grad_sums(float *out, int64_t at, int64_t N, const int64_t (&cols)[8], const float (&v)[8]) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 8; i += 4)
            if (cols[i] < N)
                *reinterpret_cast<float4 *>(out + at * N + cols[i]) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (cols[i] < N) out[at * N + cols[i]] = v[i];
    }
}

template <int ES, bool VEC, int ACT>
__global__ __launch_bounds__(256) void linear_grad_kernel(LinearGrad G, int64_t M, int64_t N, int rows, int64_t chunks,
                                                          float *__restrict__ bias_part, float *__restrict__ gate_part) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t chunk = (int64_t)blockIdx.x * 4 + wave;
    if (chunk >= chunks) return;
    const int64_t r0 = chunk * rows, r1 = r0 + rows < M ? r0 + rows : M;
    for (int64_t c0 = (int64_t)blockIdx.y * lgrad::COLS; c0 < N; c0 += (int64_t)gridDim.y * lgrad::COLS) {
        int64_t cols[8];
#pragma unroll
        for (int i = 0; i < 8; i++) cols[i] = VEC ? c0 + 8 * lane + i : c0 + 64 * i + lane;
        float db[8];
#pragma unroll
        for (int i = 0; i < 8; i++) db[i] = 0.0f;
        int s = 0, unused;
        if (G.gate_start) requests_of(G.gate_start, G.S, (int)r0, (int)r0, s, unused);
        for (int64_t row = r0; row < r1;) {
            int64_t end = r1;
            if (G.gate_start) {
                if (row > r0) s = next_request(G.gate_start, G.S, s, (int)row);
                if (s < G.S) {
                    const int64_t e = G.gate_start[s + 1];
                    end = e <= row ? row + 1 : e < r1 ? e : r1;
                }
            }
            const bool some = s >= 0 && s < G.S;
            if (G.gate && !some) {  // rows of no request: zeros, whatever they hold
                const float zero[8] = {};
                if (G.du)
                    for (; row < end; row++) grad_store<ES, VEC>(G.du, row, N, cols, zero);
                row = end;
                continue;
            }
            float g[8], dg[8];
#pragma unroll
            for (int i = 0; i < 8; i++) g[i] = 1.0f, dg[i] = 0.0f;
            if (G.gate) {
                if constexpr (VEC) {
                    load_values<8>(G.gate, G.gate_bf16, s * N + cols[0], N - cols[0], g);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        if (cols[i] < N)
                            g[i] = G.gate_bf16
                                       ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(G.gate)[s * N + cols[i]] << 16)
                                       : static_cast<const float *>(G.gate)[s * N + cols[i]];
                }
            }
            typedef GradValues<ES, VEC> Row;
            auto one = [&](int64_t r, const Row &dy, const Row &pre) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    float a, d;
                    act_and_slope<ACT>(pre.get(i), a, d);
                    dg[i] = __builtin_fmaf(dy.get(i), a, dg[i]);
                    o[i] = g[i] * dy.get(i) * d;
                    db[i] += o[i];
                }
                if (G.du) grad_store<ES, VEC>(G.du, r, N, cols, o);
            };
            constexpr int DEEP = lgrad::DEEP;
            // rows past the request's end are loaded as its last one and left out
            for (; row < end; row += DEEP) {
                Row dy[DEEP], u[DEEP];
#pragma unroll
                for (int k = 0; k < DEEP; k++) dy[k].load(G.dy, row + k < end ? row + k : end - 1, N, cols);
                if (G.pre) {
#pragma unroll
                    for (int k = 0; k < DEEP; k++) u[k].load(G.pre, row + k < end ? row + k : end - 1, N, cols);
                } else {
#pragma unroll
                    for (int k = 0; k < DEEP; k++) u[k] = Row();
                }
#pragma unroll
                for (int k = 0; k < DEEP; k++)
                    if (row + k < end) one(row + k, dy[k], u[k]);
            }
            row = end;
            if (G.dgate) grad_sums<VEC>(gate_part, chunk + s, N, cols, dg);
        }
        if (G.dbias) grad_sums<VEC>(bias_part, chunk, N, cols, db);
    }
}

// The chunks' sums of one request (blockIdx.y < S) or of the bias, 32 columns a
// workgroup: 8 lanes' worth of chunks side by side, then added in order.
__global__ __launch_bounds__(256) void linear_grad_sums_kernel(LinearGrad G, int64_t M, int64_t N, int rows, int64_t chunks,
                                                               const float *__restrict__ bias_part,
                                                               const float *__restrict__ gate_part) {
    __shared__ float part[8][32];
    const int x = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + x;
    const int64_t last = (G.dgate ? G.S : 0) + (G.dbias ? 1 : 0);
    for (int64_t s = blockIdx.y; s < last; s += gridDim.y) {
        const bool bias = s >= (G.dgate ? G.S : 0);
        int64_t c0 = 0, c1 = chunks;  // the chunks that hold rows of it
        if (!bias && G.gate_start) {
            const int lo = seg_clamp(G.gate_start[s], (int)M), hi = seg_clamp(G.gate_start[s + 1], (int)M);
            c0 = lo / rows, c1 = hi > lo ? (hi - 1) / rows + 1 : c0;
        }
        const float *p = bias ? bias_part : gate_part + s * N;
        float sum = 0.0f;
        if (col < N)
#pragma unroll 8
            for (int64_t c = c0 + k; c < c1; c += 8) sum += p[c * N + col];
        __syncthreads();
        part[k][x] = sum;
        __syncthreads();
        if (k == 0 && col < N) {
#pragma unroll
            for (int i = 1; i < 8; i++) sum += part[i][x];
            (bias ? G.dbias : G.dgate + s * N)[col] = sum;
        }
    }
}

// Rows of a chunk: about 4096 waves, and 8 rows at least, as far as M has them (a
// chunk's sums are written and read again as fp32).
static int grad_rows(int64_t M, int64_t N) {
    const int64_t blocks = (N + lgrad::COLS - 1) / lgrad::COLS;
    const int64_t r = (M * blocks + 4095) / 4096;
    return (int)(r < 8 ? 8 : r > M ? (M > 8 ? M : 8) : r);
}

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

size_t linear_grad_bytes(int64_t M, int64_t N, int64_t S) {
    if (M == 0 || N == 0) return 0;
    const unsigned __int128 chunks = (unsigned __int128)((M + grad_rows(M, N) - 1) / grad_rows(M, N));
    const unsigned __int128 bytes = (2 * chunks + S) * N * sizeof(float) + 512;
    return bytes > (unsigned __int128)4000000000000000000ull ? SIZE_MAX : up256((size_t)bytes);
}

hipError_t launch_linear_grad(hipStream_t s, const LinearGrad &G, int64_t M, int64_t N, int dtype, void *ws) {
    if (N == 0) return hipSuccess;
    const int rows = grad_rows(M, N);
    const int64_t chunks = (M + rows - 1) / rows, blocks = (N + lgrad::COLS - 1) / lgrad::COLS;
    float *bias_part = static_cast<float *>(ws);
    float *gate_part = bias_part + up256((size_t)(chunks * N) * 4) / 4;
    const bool vec = (N * (dtype == 0 ? 4 : 2)) % 16 == 0;
    if (M > 0) {
        const dim3 grid((unsigned)((chunks + 3) / 4), (unsigned)(blocks < 65535 ? blocks : 65535));
#define DMPQ_GRAD(ES_, VEC_, ACT_) \
    hipLaunchKernelGGL((linear_grad_kernel<ES_, VEC_, ACT_>), grid, dim3(256), 0, s, G, M, N, rows, chunks, bias_part, gate_part)
#define DMPQ_GRAD_ACT(ES_, VEC_)                          \
    switch (G.act) {                                      \
        case kActNone: DMPQ_GRAD(ES_, VEC_, kActNone); break;         \
        case kActGelu: DMPQ_GRAD(ES_, VEC_, kActGelu); break;         \
        case kActGeluTanh: DMPQ_GRAD(ES_, VEC_, kActGeluTanh); break; \
        default: DMPQ_GRAD(ES_, VEC_, kActSilu);          \
    }
        if (dtype == 0) {
            if (vec) DMPQ_GRAD_ACT(4, true)
            else DMPQ_GRAD_ACT(4, false)
        } else {
            if (vec) DMPQ_GRAD_ACT(2, true)
            else DMPQ_GRAD_ACT(2, false)
        }
#undef DMPQ_GRAD_ACT
#undef DMPQ_GRAD
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t sums = (G.dgate ? G.S : 0) + (G.dbias ? 1 : 0);
    if (sums == 0) return hipSuccess;
    hipLaunchKernelGGL(linear_grad_sums_kernel, dim3((unsigned)((N + 31) / 32), (unsigned)(sums < 65535 ? sums : 65535)),
                       dim3(256), 0, s, G, M, N, rows, chunks, bias_part, gate_part);
    return hipGetLastError();
}

}  // namespace dmpq
