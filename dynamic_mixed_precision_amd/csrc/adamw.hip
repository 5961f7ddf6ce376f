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

// The table's pointers come out of memory: without their address space the
// compiler takes flat accesses, which also occupy the LDS path.
#define DMPQ_GLOBAL __attribute__((address_space(1)))
template <class T>
__device__ __forceinline__ DMPQ_GLOBAL T *global_ptr(const void *p) {
    return (DMPQ_GLOBAL T *)(uintptr_t)p;
}
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// 4 values at p + i (DT 0: fp32, 1: bf16).  ALL: all four are there, else the
// first n are (n may be 0 or less).
template <int DT, bool ALL>
__device__ __forceinline__ void load4(const void *p, int64_t i, int n, float v[4]) {
    if constexpr (DT == 0) {
        const DMPQ_GLOBAL float *f = global_ptr<const float>(p) + i;
        if constexpr (ALL) {
            const f32x4 q = *reinterpret_cast<const DMPQ_GLOBAL f32x4 *>(f);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = e < n ? f[e] : 0.0f;
        }
    } else {
        const DMPQ_GLOBAL uint16_t *h = global_ptr<const uint16_t>(p) + i;
        if constexpr (ALL) {
            const u32x2 q = *reinterpret_cast<const DMPQ_GLOBAL u32x2 *>(h);
            v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = e < n ? bf16_lo(h[e]) : 0.0f;
        }
    }
}

template <int DT, bool ALL>
__device__ __forceinline__ void store4(void *p, int64_t i, int n, const float v[4]) {
    if constexpr (DT == 0) {
        DMPQ_GLOBAL float *f = global_ptr<float>(p) + i;
        if constexpr (ALL) {
            const f32x4 q = {v[0], v[1], v[2], v[3]};
            __builtin_nontemporal_store(q, reinterpret_cast<DMPQ_GLOBAL f32x4 *>(f));
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (e < n) f[e] = v[e];
        }
    } else {
        DMPQ_GLOBAL uint16_t *h = global_ptr<uint16_t>(p) + i;
        const u32x2 q = {cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
        if constexpr (ALL) {
            __builtin_nontemporal_store(q, reinterpret_cast<DMPQ_GLOBAL u32x2 *>(h));
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (e < n) h[e] = (uint16_t)((e < 2 ? q.x : q.y) >> (16 * (e & 1)));
        }
    }
}

// 4 codes (one word) and back.
template <bool ALL>
__device__ __forceinline__ uint32_t load_codes(const void *p, int64_t i, int n) {
    const DMPQ_GLOBAL uint8_t *c = global_ptr<const uint8_t>(p) + i;
    if constexpr (ALL) return *reinterpret_cast<const DMPQ_GLOBAL uint32_t *>(c);
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; e++)
        if (e < n) w |= (uint32_t)c[e] << (8 * e);
    return w;
}

template <bool ALL>
__device__ __forceinline__ void store_codes(void *p, int64_t i, int n, uint32_t w) {
    DMPQ_GLOBAL uint8_t *c = global_ptr<uint8_t>(p) + i;
    if constexpr (ALL) {
        __builtin_nontemporal_store(w, reinterpret_cast<DMPQ_GLOBAL uint32_t *>(c));
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (e < n) c[e] = (uint8_t)(w >> (8 * e));
    }
}

__device__ __forceinline__ void decode4(uint32_t w, float s, float v[4]) {
    v[0] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * s;
    v[1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * s;
    v[2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * s;
    v[3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * s;
}

__device__ __forceinline__ uint32_t encode4(const float v[4]) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
    return (uint32_t)w;
}

// The maximum of the wave's values, none negative (NaN counts as none), by DPP
// shifts within the rows of 16 lanes and broadcasts between them: lane 63 ends
// up with all.
__device__ __forceinline__ float wave_max_dpp(float v) {
#define DMPQ_DPP_MAX(CTRL, ROWS)                                                                        \
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false)))
    DMPQ_DPP_MAX(0x111, 0xF);  // row_shr 1, 2, 4, 8
    DMPQ_DPP_MAX(0x112, 0xF);
    DMPQ_DPP_MAX(0x114, 0xF);
    DMPQ_DPP_MAX(0x118, 0xF);
    DMPQ_DPP_MAX(0x142, 0xA);  // the last lane of row 0 to row 1, of row 2 to row 3
    DMPQ_DPP_MAX(0x143, 0xC);  // lane 31 to rows 2 and 3
#undef DMPQ_DPP_MAX
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// A block's scale and its reciprocal from its largest magnitude; a block whose
// reciprocal overflows (all zeros, or nothing above 448 / FLT_MAX) is zeros.
__device__ __forceinline__ void block_scale(float top, float &scale, float &inv) {
    inv = 448.0f / top;
    const bool fine = __builtin_isfinite(inv);
    scale = fine ? top / 448.0f : 0.0f;
    inv = fine ? inv : 0.0f;
}

// One block of 256 values, 4 to a lane: i is the lane's first, n what is left
// of the tensor from there.
template <int PT, int GT, int BITS, bool ALL>
__device__ __forceinline__ void adamw_block(const AdamwTensor &t, const AdamwHyper &h, float clip, int64_t i, int n) {
    float p[4], g[4], m[4], v[4], root[4];
    const int64_t blk = i / kAdamwBlock;  // the same for all lanes
    load4<PT, ALL>(t.p, i, n, p);
    load4<GT, ALL>(t.g, i, n, g);
    if constexpr (BITS == 32) {
        load4<0, ALL>(t.m, i, n, m);
        load4<0, ALL>(t.v, i, n, v);
    } else {
        const uint32_t cm = load_codes<ALL>(t.m, i, n), cv = load_codes<ALL>(t.v, i, n);
        decode4(cm, global_ptr<const float>(t.ms)[blk], m);
        decode4(cv, global_ptr<const float>(t.vs)[blk], v);
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
    store4<PT, ALL>(t.p, i, n, p);
    if (t.copy) store4<1, ALL>(t.copy, i, n, p);
    if constexpr (BITS == 32) {
        store4<0, ALL>(t.m, i, n, m);
        store4<0, ALL>(t.v, i, n, v);
    } else {
        float tm = 0.0f, tv = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            if (ALL || e < n) {
                tm = fmaxf(tm, __builtin_fabsf(m[e]));
                tv = fmaxf(tv, root[e]);
            }
        }
        float sm, im, sv, iv;
        block_scale(wave_max_dpp(tm), sm, im);
        block_scale(wave_max_dpp(tv), sv, iv);
        const float least = sv > 0.0f ? 0.001953125f : 0.0f;  // 2^-9, code 1
#pragma unroll
        for (int e = 0; e < 4; e++) {
            m[e] = m[e] * im;
            const float q = root[e] * iv;
            root[e] = root[e] > 0.0f && q < least ? least : q;
        }
        store_codes<ALL>(t.m, i, n, encode4(m));
        store_codes<ALL>(t.v, i, n, encode4(root));
        if ((threadIdx.x & 63) == 0) {
            global_ptr<float>(t.ms)[blk] = sm;
            global_ptr<float>(t.vs)[blk] = sv;
        }
    }
}

// One workgroup to a chunk of 1024 values, a block to each wave: a wave's
// loads all go out at once and nothing waits for its stores.  The chunks go
// from `last` down to the first: the norm read the gradients' end last, so part
// of it is still in the Infinity Cache (82.6 M fp32 parameters with their norm:
// 520 us, 539 from the first on).
template <int PT, int GT, int BITS>
__global__ __launch_bounds__(256) void adamw_kernel(AdamwTable T, AdamwHyper h, const double *__restrict__ norm,
                                                    unsigned last) {
    const unsigned chunk = last - blockIdx.x;
    const AdamwTensor t = T.tensors[T.chunk_tensor[chunk]];
    float clip = 1.0f;
    if (norm) {
        const double nv = *norm;
        if (!__builtin_isfinite(nv)) return;  // nothing of this step is taken
        if (h.max_norm > 0.0 && nv > h.max_norm) clip = (float)(h.max_norm / nv);
    }
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t b0 = ((int64_t)chunk - t.first_chunk) * kAdamwChunk + wave * kAdamwBlock;
    if (b0 >= t.n) return;
    const int64_t i = b0 + 4 * (threadIdx.x & 63);
    if (b0 + kAdamwBlock <= t.n)  // wave-uniform
        adamw_block<PT, GT, BITS, true>(t, h, clip, i, 4);
    else
        adamw_block<PT, GT, BITS, false>(t, h, clip, i, (int)(t.n - i < 4 ? t.n - i : 4));
}

// Sum of squares in fp64 (an fp32 gradient's square overflows fp32 above
// 1.8e19): each workgroup takes 4 neighbouring chunks at a time (all
// workgroups together walk through memory once; a run of its own for each was
// 10% slower), then one workgroup adds the partials in order and takes the
// root.
template <int GT>
__global__ __launch_bounds__(256) void grad_squares_kernel(AdamwTable T, double *__restrict__ partial) {
    __shared__ double red[4];
    static_assert(kAdamwChunk == 1024, "a chunk is 4 values a thread");
    double acc = 0.0;
    constexpr int RUN = 4;  // neighbouring chunks at a time
    for (int64_t c0 = (int64_t)blockIdx.x * RUN; c0 < T.chunks; c0 += (int64_t)gridDim.x * RUN) {
        const int64_t c1 = c0 + RUN < T.chunks ? c0 + RUN : T.chunks;
        const AdamwTensor t = T.tensors[__builtin_amdgcn_readfirstlane(T.chunk_tensor[c0])];
        int64_t i = (c0 - t.first_chunk) * kAdamwChunk + 4 * (int64_t)threadIdx.x;
        if ((c0 + RUN - t.first_chunk) * kAdamwChunk <= t.n) {
            float g[RUN][4];
#pragma unroll
            for (int u = 0; u < RUN; u++) load4<GT, true>(t.g, i + u * kAdamwChunk, 4, g[u]);
#pragma unroll
            for (int u = 0; u < RUN; u++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc += (double)g[u][e] * (double)g[u][e];
            continue;
        }
        for (int64_t c = c0; c < c1; c++) {  // a tensor's end, or several tensors
            const AdamwTensor q = T.tensors[__builtin_amdgcn_readfirstlane(T.chunk_tensor[c])];
            i = (c - q.first_chunk) * kAdamwChunk + 4 * (int64_t)threadIdx.x;
            float g[4];
            load4<GT, false>(q.g, i, (int)(q.n - i < 4 ? q.n - i : 4), g);
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
    for (int64_t end = t.chunks; end > 0; end -= kMaxGroups) {  // once, below 8.6e9 values
        const dim3 grid((unsigned)(end < kMaxGroups ? end : kMaxGroups)), block(256);
        const unsigned last = (unsigned)(end - 1);
        if (t.state_bits == 8)
            hipLaunchKernelGGL((adamw_kernel<PT, GT, 8>), grid, block, 0, s, t, h, norm, last);
        else
            hipLaunchKernelGGL((adamw_kernel<PT, GT, 32>), grid, block, 0, s, t, h, norm, last);
    }
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
