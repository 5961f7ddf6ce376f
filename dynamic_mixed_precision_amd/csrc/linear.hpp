// linear.hpp -- device helpers of the whole linear: what lies between the sums
// of a GEMM and its output.
//   v = x w^T (+ the adapter term) + bias         (pre, if asked for: v rounded)
//   v = the heads of q and k normed and rotated   (a QKV linear)
//   y = residual + gate[request of the row] * act(v), all in fp32, rounded once
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"
#include "internal.hpp"

namespace dmpq {

// ---- activations ---------------------------------------------------------------

// GELU(v) = v Phi(v) = (v / 2) erfc(-v / sqrt 2) in fp32.  erfc comes from
// the Chebyshev fit published in Numerical Recipes (Press et al., section
// 6.2, "erfcc": erfc(z) = t exp(-z^2 + P(t)), t = 1 / (1 + z/2), z >= 0, and
// 2 - erfc(-x) for x < 0), whose fractional error is below 1.2e-7 for every
// argument.  The fp32 evaluation adds a few ulp plus the rounding of the
// exponent, a relative error of about v^2 * 1.2e-7 in erfc's tail.  About 20
// VALU operations, no branches: the library erfcf costs several times that.
// gelu_phi2 is 2 Phi(v).
__device__ __forceinline__ float gelu_phi2(float v) {
    const float x = v * -0.70710678118654752f;
    const float z = __builtin_fabsf(x);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, z, 1.0f));
    float p = 0.17087277f;
    p = __builtin_fmaf(t, p, -0.82215223f);
    p = __builtin_fmaf(t, p, 1.48851587f);
    p = __builtin_fmaf(t, p, -1.13520398f);
    p = __builtin_fmaf(t, p, 0.27886807f);
    p = __builtin_fmaf(t, p, -0.18628806f);
    p = __builtin_fmaf(t, p, 0.09678418f);
    p = __builtin_fmaf(t, p, 0.37409196f);
    p = __builtin_fmaf(t, p, 1.00002368f);
    p = __builtin_fmaf(t, p, -1.26551223f);
    const float e = t * __builtin_amdgcn_exp2f(__builtin_fmaf(-z, z, p) * 1.44269504088896341f);
    return x >= 0.0f ? e : 2.0f - e;
}

__device__ __forceinline__ float gelu_f32(float v) { return 0.5f * v * gelu_phi2(v); }

constexpr float kLog2e = 1.44269504088896341f;

// 1 / (1 + e^-z): 0 and 1 where e^-z leaves fp32's range
__device__ __forceinline__ float sigmoid_f32(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

// GELU with tanh, v / 2 (1 + tanh(u)) = v sigmoid(2u), 2u = kGt (v + 0.044715 v^3)
constexpr float kGt = 1.5957691216057308f;  // 2 sqrt(2 / pi)
// the exponent of e^-2u as a power of 2
__device__ __forceinline__ float gelu_tanh_exponent(float v) {
    return v * __builtin_fmaf(-kLog2e * kGt * 0.044715f, v * v, -kLog2e * kGt);
}

enum { kActNone = 0, kActGelu = 1, kActGeluTanh = 2, kActSilu = 3 };

// v[i] = act(v[i]); act is the same for every lane.
template <int N>
__device__ __forceinline__ void act_apply(float (&v)[N], int act) {
    if (act == kActGelu) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = gelu_f32(v[i]);
    } else if (act == kActGeluTanh) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] *= __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(gelu_tanh_exponent(v[i])));
    } else if (act == kActSilu) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] *= sigmoid_f32(v[i]);
    }
}

// ---- parameters and rows of a request -------------------------------------------

// N values of an fp32 or bf16 vector from index `at` on, zeros from the left-th on.
template <int N>
__device__ __forceinline__ void load_values(const void *p, bool bf16, int64_t at, int64_t left, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = 0.0f;
    if (N >= 4 && left >= N && at % N == 0) {
        if (bf16) {
            const uint16_t *q = static_cast<const uint16_t *>(p) + at;
            uint32_t w[N / 2] = {};
            if constexpr (N == 8) {
                const uint4 u = *reinterpret_cast<const uint4 *>(q);
                w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
            } else if constexpr (N == 4) {
                const uint2 u = *reinterpret_cast<const uint2 *>(q);
                w[0] = u.x, w[1] = u.y;
            }
#pragma unroll
            for (int i = 0; i < N / 2; i++) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i + 3 < N; i += 4) {
                const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at + i);
                v[i] = u.x, v[i + 1] = u.y, v[i + 2] = u.z, v[i + 3] = u.w;
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; i++)
        if (i < left)
            v[i] = bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[at + i] << 16)
                        : static_cast<const float *>(p)[at + i];
}

// The request of a row: how many of the S + 1 boundaries are at or before it,
// less one (-1 and S: none).  Of each lane's own row, by bisection:
__device__ __forceinline__ int request_of(const int32_t *start, int S, int row) {
    int lo = 0, hi = S + 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= row)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo - 1;
}

// of two rows a <= b that are the same in every lane, by one load for up to 63
// requests;
__device__ __forceinline__ void requests_of(const int32_t *start, int S, int a, int b, int &ra, int &rb) {
    if (S < 64) {
        const int lane = threadIdx.x & 63;
        const int v = start[lane <= S ? lane : S];
        ra = __builtin_popcountll(__ballot(lane <= S && v <= a)) - 1;
        rb = __builtin_popcountll(__ballot(lane <= S && v <= b)) - 1;
    } else {
        ra = __builtin_amdgcn_readfirstlane(request_of(start, S, a));
        rb = a == b ? ra : __builtin_amdgcn_readfirstlane(request_of(start, S, b));
    }
}

// and of a later row, the same in every lane, than one of request s, 64
// boundaries a load.
__device__ __forceinline__ int next_request(const int32_t *start, int S, int s, int row) {
    const int lane = threadIdx.x & 63;
    while (s < S) {
        const int at = s + 1 + lane;
        const int n = __builtin_popcountll(__ballot(at <= S && start[at <= S ? at : S] <= row));
        s += n;
        if (n < 64) break;
    }
    return s;
}

// ---- the heads of q and k ---------------------------------------------------------

// 1 / sqrt(x); the instruction takes values below fp32's normal range as 0.
__device__ __forceinline__ float rsqrt_f32(float x) {
    return x < 0x1p-100f ? __builtin_amdgcn_rsqf(x * 0x1p100f) * 0x1p50f : __builtin_amdgcn_rsqf(x);
}

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}

// The sum over aligned groups of 4, 8 or 16 lanes, in every lane of the group:
// quad_perm swaps, then the mirrors of 8 and of 16 lanes (whose halves already
// agree).
__device__ __forceinline__ float group_sum(float v, int lanes) {
    v += dpp_f32<0xB1>(v);
    v += dpp_f32<0x4E>(v);
    if (lanes >= 8) v += dpp_f32<0x141>(v);
    if (lanes >= 16) v += dpp_f32<0x140>(v);
    return v;
}

// What a lane needs of the heads when it holds the N columns from `col` on of
// every row: their place in the head, weights, and whether they are in one.
template <int N>
struct QkLane {
    float w[N], b[N];
    int c;      // first column within the head
    bool mine;  // columns of a head of q or k
    __device__ __forceinline__ void begin(const QkHeads &H, int64_t col) {
        const int h = (int)(col / H.D);
        c = (int)(col - (int64_t)h * H.D);
        mine = h < H.nq + H.nk;
        const bool q = h < H.nq;
#pragma unroll
        for (int i = 0; i < N; i++) w[i] = 1.0f, b[i] = 0.0f;
        const void *pw = q ? H.wq : H.wk, *pb = q ? H.bq : H.bk;
        if (mine && pw) load_values<N>(pw, H.w_bf16, c, N, w);
        if (mine && pb) load_values<N>(pb, H.w_bf16, c, N, b);
    }
    // v of row `row` (below M) normed over the D / N lanes of its head and
    // rotated.  Every lane of the wave calls it; other columns stay.
    __device__ __forceinline__ void apply(const QkHeads &H, int64_t row, float (&v)[N]) const {
        const int lanes = H.D / N;
        float y[N];
#pragma unroll
        for (int i = 0; i < N; i++) y[i] = v[i];
        if (H.norm != 0) {
            const float inv = 1.0f / (float)H.D;
            if (H.norm == 2) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < N; i++) s += y[i];
                s = group_sum(s, lanes);
                if (lanes >= 32) s += __shfl_xor(s, 16, 64);
                s *= inv;
#pragma unroll
                for (int i = 0; i < N; i++) y[i] -= s;
            }
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < N; i++) s = __builtin_fmaf(y[i], y[i], s);
            s = group_sum(s, lanes);
            if (lanes >= 32) s += __shfl_xor(s, 16, 64);
            const float r = rsqrt_f32(__builtin_fmaf(s, inv, H.eps));
#pragma unroll
            for (int i = 0; i < N; i++) y[i] = __builtin_fmaf(y[i] * r, w[i], b[i]);
        }
        if (H.P > 0) {
            const float2 *cs = reinterpret_cast<const float2 *>(H.table) + row * H.P;
            if (H.layout == 0) {
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const int p = (c + i) >> 1;
                    const bool turned = p < H.P;
                    const float2 z = cs[turned ? p : 0];
                    const float lo = y[i], hi = y[i + 1];
                    y[i] = turned ? lo * z.x - hi * z.y : lo;
                    y[i + 1] = turned ? hi * z.x + lo * z.y : hi;
                }
            } else {  // P is a multiple of N: a lane's columns are all in one half
                const bool first = c < H.P, turned = c < 2 * H.P;
                const int from = (threadIdx.x & 63) + (turned ? (first ? H.P / N : -H.P / N) : 0);
                const float2 *z = cs + (turned ? (first ? c : c - H.P) : 0);
#pragma unroll
                for (int i = 0; i < N; i++) {
                    const float o = __shfl(y[i], from, 64);
                    const float2 zi = z[turned ? i : 0];
                    const float t = first ? -(o * zi.y) : o * zi.y;
                    y[i] = turned ? __builtin_fmaf(y[i], zi.x, t) : y[i];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = mine ? y[i] : v[i];
    }
};

// ---- outputs ----------------------------------------------------------------------

// N values of y's type at element `at` of p; `left` columns remain in the row.
// vec: rows are 16-byte aligned.
template <int ESIZE, int N>
__device__ __forceinline__ void store_values(void *p, int64_t at, int64_t left, bool vec, const float (&v)[N]) {
    uint8_t *dst = static_cast<uint8_t *>(p) + at * ESIZE;
    uint32_t w[N * ESIZE / 4];
#pragma unroll
    for (int i = 0; i < N * ESIZE / 4; i++)
        w[i] = ESIZE == 4 ? __float_as_uint(v[i]) : cvt_pk_bf16(v[2 * i], v[2 * i + 1]);
    if (vec && left >= N) {
        if constexpr (N * ESIZE == 16)
            store_nt16(dst, make_uint4(w[0], w[1], w[2], w[3]));
        else
            *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        return;
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
        if (i >= left) break;
        if constexpr (ESIZE == 4)
            reinterpret_cast<uint32_t *>(dst)[i] = w[i];
        else
            reinterpret_cast<uint16_t *>(dst)[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}

// N values of that type, zeros from the left-th on.
template <int ESIZE, int N>
__device__ __forceinline__ void fetch_values(const void *p, int64_t at, int64_t left, bool vec, float (&v)[N]) {
    if (vec && left >= N) {
        const uint8_t *src = static_cast<const uint8_t *>(p) + at * ESIZE;
        uint32_t w[N * ESIZE / 4];
        if constexpr (N * ESIZE == 16) {
            const uint4 u = load_nt16(src);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(src);
            w[0] = u.x, w[1] = u.y;
        }
#pragma unroll
        for (int i = 0; i < N; i++)
            v[i] = ESIZE == 4 ? __uint_as_float(w[i * ESIZE / 4]) : i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
        return;
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
        v[i] = 0.0f;
        if (i < left)
            v[i] = ESIZE == 4 ? static_cast<const float *>(p)[at + i]
                              : __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[at + i] << 16);
    }
}

// The same as they lie, 16 bytes.
template <int ESIZE>
__device__ __forceinline__ uint4 fetch_raw(const void *p, int64_t at, int64_t left, bool vec) {
    constexpr int N = 16 / ESIZE;
    if (vec && left >= N) return load_nt16(static_cast<const uint8_t *>(p) + at * ESIZE);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < N; i++)
        if (i < left) {
            if constexpr (ESIZE == 4)
                w[i] = static_cast<const uint32_t *>(p)[at + i];
            else
                w[i >> 1] |= (uint32_t) static_cast<const uint16_t *>(p)[at + i] << (16 * (i & 1));
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// What a lane that holds the N columns from `col` on keeps over its rows: the
// bias, and the gate where all rows belong to one request.
enum { kGateNone = 0, kGateOne = 1, kGateZero = 2, kGateMixed = 3 };
template <int N>
struct LinearLane {
    float bias[N], gate[N];
    int mode;  // wave-uniform
    int held;  // kGateMixed: the request whose gate the lane has

    // rows row0 .. row0 + rows - 1 (those below M count)
    __device__ __forceinline__ void begin(const LinearEpi &L, int64_t row0, int rows, int64_t M, int64_t N_, int64_t col) {
#pragma unroll
        for (int i = 0; i < N; i++) bias[i] = 0.0f, gate[i] = 1.0f;
        if (L.bias) load_values<N>(L.bias, L.bias_bf16, col, N_ - col, bias);
        mode = kGateNone, held = -2;
        if (L.gate) {
            int a = 0, b = 0;
            if (L.gate_start) {
                const int64_t r1 = row0 + rows < M ? row0 + rows : M;
                if (r1 <= row0) return;
                requests_of(L.gate_start, L.S, (int)row0, (int)r1 - 1, a, b);
            }
            mode = a != b ? kGateMixed : a >= 0 && a < L.S ? kGateOne : kGateZero;
            if (mode == kGateOne) load_values<N>(L.gate, L.gate_bf16, a * N_ + col, N_ - col, gate);
        }
    }
    // On to a row of that request (kGateMixed): its gate is loaded where it is not the
    // one that the lane has.
    __device__ __forceinline__ void turn(const LinearEpi &L, int request, int64_t N_, int64_t col) {
        if (mode != kGateMixed || request == held) return;
        held = request;
        if (request >= 0 && request < L.S) load_values<N>(L.gate, L.gate_bf16, request * N_ + col, N_ - col, gate);
    }
    // gate (of the row's request, turn) and residual of one row: v becomes y.  in: the
    // lane has columns there; ahead: its residual, where it is loaded already.
    template <int ESIZE>
    __device__ __forceinline__ void finish(const LinearEpi &L, int64_t row, int64_t N_, int64_t col, bool in, bool vec,
                                           float (&v)[N], const uint4 *ahead = nullptr) const {
        if (mode == kGateOne) {
#pragma unroll
            for (int i = 0; i < N; i++) v[i] *= gate[i];
        } else if (mode != kGateNone) {
            // rows of no request take no term at all, not zero times one
            const bool some = mode == kGateMixed && held >= 0 && held < L.S;
#pragma unroll
            for (int i = 0; i < N; i++) v[i] = some ? v[i] * gate[i] : L.residual ? -0.0f : 0.0f;
        }
        if (L.residual && in) {
            float r[N];
            if (ahead) {
                const uint32_t w[4] = {ahead->x, ahead->y, ahead->z, ahead->w};
#pragma unroll
                for (int i = 0; i < N; i++)
                    r[i] = ESIZE == 4 ? __uint_as_float(w[i & 3]) : i & 1 ? bf16_hi(w[i >> 1 & 3]) : bf16_lo(w[i >> 1 & 3]);
            } else {
                fetch_values<ESIZE, N>(L.residual, row * N_ + col, N_ - col, vec, r);
            }
#pragma unroll
            for (int i = 0; i < N; i++) v[i] += r[i];
        }
    }
};

}  // namespace dmpq
