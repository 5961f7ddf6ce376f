// adamw.hip -- the AdamW step (Loshchilov and Hutter, "Decoupled Weight Decay
// Regularization") over many tensors in one launch, with 32-bit states or
// with states in 8 bits, and the global norm of all gradients.
//
//   g' = g * clip
//   m  = beta1 m + (1 - beta1) g'
//   v  = beta2 v + (1 - beta2) g'^2
//   p  = p (1 - lr wd) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// all in fp32, every operation rounded by itself; p as fp32 or bf16, with an
// optional bf16 copy.  8-bit states: each 256 consecutive values of a tensor
// share an fp32 scale; m is kept as E4M3(m / s) with s = max |m| / 448, and v
// through its square root, E4M3(sqrt(v) / s) with s = max sqrt(v) / 448: the
// root halves the exponents, so that 17 bits of range below the block's
// largest root hold 35 of v.  A root that is not zero keeps at least the
// smallest code, so that no denominator falls to eps by rounding.
//
// The step moves 28 bytes per fp32 parameter and does some 60 operations on
// them, so memory bounds it.
#include "device.hpp"
#include "internal.hpp"

namespace dmpq {

namespace {

constexpr int kUnits = kAdamwChunk / kAdamwBlock / 4;  // 256-value blocks per wave of a chunk

// 4 values at p + i (fp32 or bf16), of which n are there.
template <int DT>
__device__ __forceinline__ void load4(const void *p, int64_t i, int n, float v[4]) {
    if constexpr (DT == 0) {
        const float *f = static_cast<const float *>(p) + i;
        if (n >= 4) {
            const float4 q = *reinterpret_cast<const float4 *>(f);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = e < n ? f[e] : 0.0f;
        }
    } else {
        const uint16_t *h = static_cast<const uint16_t *>(p) + i;
        if (n >= 4) {
            const uint2 q = *reinterpret_cast<const uint2 *>(h);
            v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = e < n ? bf16_lo(h[e]) : 0.0f;
        }
    }
}

template <int DT>
__device__ __forceinline__ void store4(void *p, int64_t i, int n, const float v[4]) {
    if constexpr (DT == 0) {
        float *f = static_cast<float *>(p) + i;
        if (n >= 4) {
            *reinterpret_cast<float4 *>(f) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (e < n) f[e] = v[e];
        }
    } else {
        uint16_t *h = static_cast<uint16_t *>(p) + i;
        const uint2 q = make_uint2(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]));
        if (n >= 4) {
            *reinterpret_cast<uint2 *>(h) = q;
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (e < n) h[e] = (uint16_t)((e < 2 ? q.x : q.y) >> (16 * (e & 1)));
        }
    }
}

// 4 codes (one word) and back.
__device__ __forceinline__ uint32_t load_codes(const void *p, int64_t i, int n) {
    const uint8_t *c = static_cast<const uint8_t *>(p) + i;
    if (n >= 4) return *reinterpret_cast<const uint32_t *>(c);
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; e++)
        if (e < n) w |= (uint32_t)c[e] << (8 * e);
    return w;
}

__device__ __forceinline__ void store_codes(void *p, int64_t i, int n, uint32_t w) {
    uint8_t *c = static_cast<uint8_t *>(p) + i;
    if (n >= 4) {
        *reinterpret_cast<uint32_t *>(c) = w;
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; e++)
        if (e < n) c[e] = (uint8_t)(w >> (8 * e));
}

__device__ __forceinline__ void decode4(uint32_t w, float s, float v[4]) {
    v[0] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * s;
    v[1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * s;
    v[2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * s;
    v[3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * s;
}

__device__ __forceinline__ uint32_t encode4(const float v[4], float inv) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, w, true);
    return (uint32_t)w;
}

// A block's scale and its reciprocal from its largest magnitude; a block whose
// reciprocal overflows (all zeros, or nothing above 448 / FLT_MAX) is zeros.
__device__ __forceinline__ void block_scale(float top, float &scale, float &inv) {
    inv = 448.0f / top;
    const bool fine = __builtin_isfinite(inv);
    scale = fine ? top / 448.0f : 0.0f;
    inv = fine ? inv : 0.0f;
}

template <int PT, int GT, int BITS>
__global__ __launch_bounds__(256) void adamw_kernel(AdamwTable T, AdamwHyper h, const double *__restrict__ norm) {
    float clip = 1.0f;
    if (norm) {
        const double nv = *norm;
        if (!__builtin_isfinite(nv)) return;  // nothing of this step is taken
        if (h.max_norm > 0.0 && nv > h.max_norm) clip = (float)(h.max_norm / nv);
    }
    const AdamwTensor &t = T.tensors[T.chunk_tensor[blockIdx.x]];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t base = ((int64_t)blockIdx.x - t.first_chunk) * kAdamwChunk;
#pragma unroll
    for (int u = 0; u < kUnits; u++) {
        const int64_t b0 = base + (int64_t)(wave * kUnits + u) * kAdamwBlock;
        if (b0 >= t.n) break;
        const int64_t i = b0 + 4 * lane;
        const int n = (int)(t.n - i < 4 ? t.n - i : 4);  // <= 0: this lane has none
        float p[4], g[4], m[4], v[4], root[4];
        load4<PT>(t.p, i, n, p);
        load4<GT>(t.g, i, n, g);
        if constexpr (BITS == 32) {
            load4<0>(t.m, i, n, m);
            load4<0>(t.v, i, n, v);
        } else {
            decode4(load_codes(t.m, i, n), t.ms[b0 / kAdamwBlock], m);
            decode4(load_codes(t.v, i, n), t.vs[b0 / kAdamwBlock], v);
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = v[e] * v[e];
        }
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float gc = g[e] * clip;
            m[e] = h.beta1 * m[e] + h.omb1 * gc;
            v[e] = h.beta2 * v[e] + h.omb2 * (gc * gc);
            root[e] = __builtin_sqrtf(v[e]);
            const float den = root[e] * h.rbc2 + h.eps;
            p[e] = p[e] * h.decay - h.step * (m[e] / den);
        }
        store4<PT>(t.p, i, n, p);
        if (t.copy) store4<1>(t.copy, i, n, p);
        if constexpr (BITS == 32) {
            store4<0>(t.m, i, n, m);
            store4<0>(t.v, i, n, v);
        } else {
            float tm = 0.0f, tv = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                if (e < n) {
                    tm = fmaxf(tm, __builtin_fabsf(m[e]));
                    tv = fmaxf(tv, root[e]);
                }
            }
            float sm, im, sv, iv;
            block_scale(wave_max(tm), sm, im);
            block_scale(wave_max(tv), sv, iv);
            uint32_t cv = encode4(root, iv);
            if (sv > 0.0f) {
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (root[e] > 0.0f && ((cv >> (8 * e)) & 0xFFu) == 0u) cv |= 1u << (8 * e);
            }
            store_codes(t.m, i, n, encode4(m, im));
            store_codes(t.v, i, n, cv);
            if (lane == 0) {
                t.ms[b0 / kAdamwBlock] = sm;
                t.vs[b0 / kAdamwBlock] = sv;
            }
        }
    }
}

// Sum of squares in fp64 (an fp32 gradient's square overflows fp32 above
// 1.8e19): each workgroup walks over chunks, then one workgroup adds the
// partials in order and takes the root.
template <int GT>
__global__ __launch_bounds__(256) void grad_squares_kernel(AdamwTable T, double *__restrict__ partial) {
    __shared__ double red[4];
    double acc = 0.0;
    for (int64_t c = blockIdx.x; c < T.chunks; c += gridDim.x) {
        const AdamwTensor &t = T.tensors[T.chunk_tensor[c]];
        const int64_t base = (c - t.first_chunk) * kAdamwChunk;
#pragma unroll
        for (int u = 0; u < kAdamwChunk / 1024; u++) {
            const int64_t i = base + 1024 * u + 4 * (int64_t)threadIdx.x;
            const int n = (int)(t.n - i < 4 ? t.n - i : 4);
            float g[4];
            load4<GT>(t.g, i, n, g);
#pragma unroll
            for (int e = 0; e < 4; e++) acc += (double)g[e] * (double)g[e];
        }
    }
    acc = wave_sum(acc);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
    __syncthreads();
    if (threadIdx.x == 0) partial[blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ __launch_bounds__(256) void grad_norm_kernel(const double *__restrict__ partial, int n,
                                                        double *__restrict__ norm) {
    __shared__ double red[4];
    double acc = 0.0;
#pragma unroll
    for (int k = 0; k < kMaxPartials / 256; k++) {
        const int i = threadIdx.x + 256 * k;
        acc += i < n ? partial[i] : 0.0;
    }
    acc = wave_sum(acc);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
    __syncthreads();
    if (threadIdx.x == 0) *norm = sqrt((red[0] + red[1]) + (red[2] + red[3]));
}

template <int PT, int GT>
void step(hipStream_t s, const AdamwTable &t, const AdamwHyper &h, const double *norm) {
    const dim3 grid((unsigned)t.chunks), block(256);
    if (t.state_bits == 8)
        hipLaunchKernelGGL((adamw_kernel<PT, GT, 8>), grid, block, 0, s, t, h, norm);
    else
        hipLaunchKernelGGL((adamw_kernel<PT, GT, 32>), grid, block, 0, s, t, h, norm);
}

}  // namespace

hipError_t launch_grad_norm(hipStream_t s, const AdamwTable &t, double *norm, const Workspace &ws) {
    const unsigned grid = stride_grid(t.chunks, 1, kMaxPartials);
    if (t.g_dtype == 0)
        hipLaunchKernelGGL(grad_squares_kernel<0>, dim3(grid), dim3(256), 0, s, t, ws.partial);
    else
        hipLaunchKernelGGL(grad_squares_kernel<1>, dim3(grid), dim3(256), 0, s, t, ws.partial);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(256), 0, s, ws.partial, (int)grid, norm);
    return hipGetLastError();
}

hipError_t launch_adamw(hipStream_t s, const AdamwTable &t, const AdamwHyper &h, const double *norm) {
    if (t.chunks == 0) return hipSuccess;
    if (t.p_dtype == 0)
        t.g_dtype == 0 ? step<0, 0>(s, t, h, norm) : step<0, 1>(s, t, h, norm);
    else
        t.g_dtype == 0 ? step<1, 0>(s, t, h, norm) : step<1, 1>(s, t, h, norm);
    return hipGetLastError();
}

}  // namespace dmpq
