// qk.hip -- the heads of q and k between the QKV linear and attention: the
// table of rotations of positions with several axes, the per-head norm with the
// rotation in one pass, and that pass's gradients.
//
// Norm of a head x of D values (RMS: m = 0):
//   n = (x - m) / sqrt(mean((x - m)^2) + eps),  y = n w + b,  m = mean(x)
// Rotation of pair p by the angle a of its row and axis:
//   (lo, hi) -> (lo cos a - hi sin a, hi cos a + lo sin a)
// All in fp32, one rounding at the end.  Both passes read and write each head
// once and are bound by HBM.  A lane holds 8 values of a head, so that a head
// of 64 is 8 lanes and one wave takes 8 heads of a row in a step; their
// rotations are the same for every head of the row and stay in registers.
#include "device.hpp"
#include "internal.hpp"
#include "linear.hpp"

namespace dmpq {

// ---- rotations -----------------------------------------------------------------

// (cos, sin) of pos[m, axis(p)] * freq[p].  The angle is made in 64 bits, as
// turns, so that its distance to the nearest quarter turn is off by |angle| 2^-51
// at most: less than half a step of fp32 at 1 up to angles of 2^27, and 10^-6 at
// 2^31.  Writes 8 bytes a pair (17776 rows of 32: 4.5 MB in 5.5 us).
__global__ __launch_bounds__(256) void rope_table_kernel(const void *__restrict__ pos, int pos_f32, RopeAxes ax,
                                                         const double *__restrict__ freq, int64_t M, int P,
                                                         float2 *__restrict__ table) {
    const int64_t total = M * P, per = 256;
    for (int64_t base = (int64_t)blockIdx.x * per; base < total; base += (int64_t)gridDim.x * per) {
        const int64_t m0 = base / P;
        const unsigned p0 = (unsigned)(base - m0 * P);
        const unsigned o = p0 + threadIdx.x;
        const int64_t m = m0 + o / (unsigned)P;
        const int p = (int)(o % (unsigned)P);
        if (m >= M) continue;
        int a = 0;
#pragma unroll
        for (int i = 0; i < kMaxRopeAxes - 1; i++) a += i < ax.n - 1 && p >= ax.end[i];
        const double at = pos_f32 ? (double)static_cast<const float *>(pos)[m * ax.n + a]
                                  : (double)static_cast<const int32_t *>(pos)[m * ax.n + a];
        const double turns = at * freq[p] * 0.15915494309189533577;
        const double quarter = __builtin_rint(4.0 * turns);
        const float r = (float)(turns - 0.25 * quarter);
        float s, c;
        sincospif(2.0f * r, &s, &c);
        // which quarter: by a remainder in 64 bits, as it may pass 2^31
        const int q = (int)(quarter - 4.0 * __builtin_floor(0.25 * quarter));
        const float cs = q & 1 ? s : c, sn = q & 1 ? c : s;
        table[m * P + p] = make_float2(q == 1 || q == 2 ? -cs : cs, q >= 2 ? -sn : sn);
    }
}

hipError_t launch_rope_table(hipStream_t s, const void *pos, bool pos_f32, const RopeAxes &ax, const double *freq, int64_t M,
                             float *table) {
    const int P = ax.end[ax.n - 1];
    if (M == 0 || P == 0) return hipSuccess;
    hipLaunchKernelGGL(rope_table_kernel, dim3(stride_grid(M * P, 256, 1u << 18)), dim3(256), 0, s, pos, pos_f32 ? 1 : 0, ax,
                       freq, M, P, reinterpret_cast<float2 *>(table));
    return hipGetLastError();
}

// ---- the heads -----------------------------------------------------------------

// A lane's 8 values of a head: two runs of four, so that both members of its
// four pairs 4 sub .. 4 sub + 3 are the lane's own.  Neighbours (2p, 2p + 1) lie
// in one run of 8; halves (p, p + P) in one of 4 in either half, and what is
// behind 2P in runs of 8 again.
template <int LAYOUT>
struct Lane8 {
    int a, b;   // where the runs begin
    bool live;  // the lane has a part of the head
    __device__ __forceinline__ Lane8(const QkHeads &H, int sub) {
        live = 8 * sub < H.D;
        a = 8 * sub, b = a + 4;
        if (LAYOUT == 1 && 4 * sub < H.P) a = 4 * sub, b = H.P + a;
        if (!live) a = 0, b = 4;
    }
    // the two members of pair i in the lane's 8 values
    __device__ static __forceinline__ int lo(int i) { return LAYOUT == 0 ? 2 * i : i; }
    __device__ static __forceinline__ int hi(int i) { return LAYOUT == 0 ? 2 * i + 1 : i + 4; }
    template <int ES>
    __device__ __forceinline__ void load(const void *p, int64_t at, float (&v)[8]) const {
        if constexpr (ES == 2 && LAYOUT == 0) {
            fetch_values<2, 8>(p, at + a, 8, true, v);
        } else {
            float u[4], w[4];
            fetch_values<ES, 4>(p, at + a, 4, true, u);
            fetch_values<ES, 4>(p, at + b, 4, true, w);
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] = u[i], v[4 + i] = w[i];
        }
    }
    template <int ES>
    __device__ __forceinline__ void store(void *p, int64_t at, const float (&v)[8]) const {
        if constexpr (ES == 2 && LAYOUT == 0) {
            store_values<2, 8>(p, at + a, 8, true, v);
        } else {
            float u[4], w[4];
#pragma unroll
            for (int i = 0; i < 4; i++) u[i] = v[i], w[i] = v[4 + i];
            store_values<ES, 4>(p, at + a, 4, true, u);
            store_values<ES, 4>(p, at + b, 4, true, w);
        }
    }
    __device__ __forceinline__ void weights(const void *p, bool bf16, float other, float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = other;
        if (!p) return;
        float u[4], w[4];
        load_values<4>(p, bf16, a, 4, u);
        load_values<4>(p, bf16, b, 4, w);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = u[i], v[4 + i] = w[i];
    }
};

// The sum over the G lanes of a head (a power of two), in each of them.
template <int G>
__device__ __forceinline__ float head_sum(float v) {
    if (G >= 2) v += dpp_f32<0xB1>(v);
    if (G >= 4) v += dpp_f32<0x4E>(v);
    if (G >= 8) v += dpp_f32<0x141>(v);
    if (G >= 16) v += dpp_f32<0x140>(v);
    if (G >= 32) v += __shfl_xor(v, 16, 64);
    return v;
}

// The rotations of the lane's four pairs in row m.
struct Turns {
    float c[4], s[4];
    bool on[4];
    __device__ __forceinline__ void load(const QkHeads &H, int64_t m, int sub) {
        const float2 *t = reinterpret_cast<const float2 *>(H.table) + m * H.P;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int p = 4 * sub + i;
            on[i] = p < H.P;
            const float2 z = on[i] ? t[p] : make_float2(1.0f, 0.0f);
            c[i] = z.x, s[i] = z.y;
        }
    }
    // values that are not rotated stay as they are (not times 1 plus times 0)
    template <int LAYOUT, bool BACK>
    __device__ __forceinline__ void apply(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float lo = v[Lane8<LAYOUT>::lo(i)], hi = v[Lane8<LAYOUT>::hi(i)], sn = BACK ? -s[i] : s[i];
            v[Lane8<LAYOUT>::lo(i)] = on[i] ? lo * c[i] - hi * sn : lo;
            v[Lane8<LAYOUT>::hi(i)] = on[i] ? hi * c[i] + lo * sn : hi;
        }
    }
};

// n = the normed values; returns the factor 1 / sqrt(...).
template <int G>
__device__ __forceinline__ float norm8(const QkHeads &H, bool live, const float (&x)[8], float (&n)[8]) {
    const float inv = 1.0f / (float)H.D;
#pragma unroll
    for (int i = 0; i < 8; i++) n[i] = x[i];
    if (H.norm == 2) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) s += n[i];
        s = head_sum<G>(live ? s : 0.0f) * inv;
#pragma unroll
        for (int i = 0; i < 8; i++) n[i] -= s;
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) s = __builtin_fmaf(n[i], n[i], s);
    s = head_sum<G>(live ? s : 0.0f);
    const float r = rsqrt_f32(__builtin_fmaf(s, inv, H.eps));
#pragma unroll
    for (int i = 0; i < 8; i++) n[i] *= r;
    return r;
}

// The steps of a row: 64 / G heads of q each, then of k.  A wave takes `per`
// consecutive steps of one row, one after the other: a full chip of waves keeps
// more loads on their way than several steps of fewer waves do (17776 rows of 30 +
// 30 heads of 64, bf16, with the table: 1 / 2 / 4 / 8 steps at once 61 / 62 / 74 / 85 us).
template <int ES, int LAYOUT, int G>
__global__ __launch_bounds__(256) void qk_kernel(QkTensors T, QkHeads H, int64_t M, int sq, int steps, int per,
                                                 int64_t units, int parts) {
    constexpr int HEADS = 64 / G;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
    if (unit >= units) return;
    const int64_t m = unit / parts;
    const int first = (int)(unit - m * parts) * per, last = first + per < steps ? first + per : steps;
    const int sub = lane % G, slot = lane / G;
    const Lane8<LAYOUT> L(H, sub);
    Turns t;
    t.load(H, m, sub);
    for (int side = 0; side < 2; side++) {  // q, then k: one set of weights at a time
        const int s0 = side ? (first > sq ? first : sq) : first, s1 = side ? last : (last < sq ? last : sq);
        if (s0 >= s1) continue;
        const void *x = side ? T.k : T.q;
        void *y = side ? T.k_out : T.q_out;
        const int64_t at = m * (side ? T.ldk : T.ldq), to = m * (side ? T.ldk_out : T.ldq_out);
        const int heads = side ? H.nk : H.nq, base = side ? sq : 0;
        float w[8], b[8];
        L.weights(side ? H.wk : H.wq, H.w_bf16, 1.0f, w);
        L.weights(side ? H.bk : H.bq, H.w_bf16, 0.0f, b);
        for (int st = s0; st < s1; st++) {
            const int head = (st - base) * HEADS + slot;
            const bool on = L.live && head < heads;
            const int64_t h = (int64_t)head * H.D;
            float v[8] = {};
            if (on) L.template load<ES>(x, at + h, v);
            if (H.norm != 0) {
                float n[8];
                norm8<G>(H, L.live, v, n);
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] = __builtin_fmaf(n[i], w[i], b[i]);
            }
            t.apply<LAYOUT, false>(v);
            if (on) L.template store<ES>(y, to + h, v);
        }
    }
}

// The gradients.  With g' = the rotation's transpose of g, h = g' w, r = the norm's factor:
//   dx = r (h - mean(h) - n mean(h n))   (RMS: without mean(h));  dw += g' n;  db += g'
// The weights' sums stay in registers over all a wave's rows, and each
// workgroup stores its own; a second kernel adds them in order.  Four workgroups a
// CU (17776 rows of 30 + 30 heads of 64, bf16, with the second kernel: 2 / 3 / 4 / 5 / 8 a CU
// 108 / 89 / 81 / 97 / 90 us; two steps at once 120, four 130).
constexpr int kQkGroups = 1024;

template <int ES, int LAYOUT, int G>
__global__ __launch_bounds__(256) void qk_grad_kernel(QkTensors T, QkHeads H, int64_t M, int sq, int steps, int per,
                                                      int64_t units, int parts, float *__restrict__ part) {
    constexpr int HEADS = 64 / G;
    __shared__ float red[4][4][kMaxHeadDim];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = lane % G, slot = lane / G;
    const Lane8<LAYOUT> L(H, sub);
    float w[2][8], dw[2][8], db[2][8];
    L.weights(H.wq, H.w_bf16, 1.0f, w[0]);
    L.weights(H.wk, H.w_bf16, 1.0f, w[1]);
#pragma unroll
    for (int i = 0; i < 8; i++) dw[0][i] = dw[1][i] = db[0][i] = db[1][i] = 0.0f;
    const float inv = 1.0f / (float)H.D;
    for (int64_t unit = (int64_t)blockIdx.x * 4 + wave; unit < units; unit += (int64_t)gridDim.x * 4) {
        const int64_t m = unit / parts;
        const int first = (int)(unit - m * parts) * per, last = first + per < steps ? first + per : steps;
        Turns t;
        t.load(H, m, sub);
#pragma unroll
        for (int side = 0; side < 2; side++) {
            const int s0 = side ? (first > sq ? first : sq) : first, s1 = side ? last : (last < sq ? last : sq);
            const void *x = side ? T.k : T.q, *g = side ? T.dk : T.dq;
            void *y = side ? T.k_out : T.q_out;
            const int64_t at = m * (side ? T.ldk : T.ldq), gat = m * (side ? T.lddk : T.lddq),
                          to = m * (side ? T.ldk_out : T.ldq_out);
            const int heads = side ? H.nk : H.nq, base = side ? sq : 0;
            for (int st = s0; st < s1; st++) {
                const int head = (st - base) * HEADS + slot;
                const bool on = L.live && head < heads;
                const int64_t h = (int64_t)head * H.D;
                float v[8] = {}, e[8] = {};
                if (on) {
                    L.template load<ES>(g, gat + h, e);
                    if (H.norm != 0) L.template load<ES>(x, at + h, v);
                }
                t.apply<LAYOUT, true>(e);
                if (H.norm != 0) {
                    float n[8], k[8];
                    const float r = norm8<G>(H, L.live, v, n);
                    float mh = 0.0f, mn = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        if (on) {  // (a head that is not there has n = 0 r, which eps 0 makes NaN)
                            dw[side][i] = __builtin_fmaf(e[i], n[i], dw[side][i]);
                            db[side][i] += e[i];
                        }
                        k[i] = e[i] * w[side][i];
                        mh += k[i];
                        mn = __builtin_fmaf(k[i], n[i], mn);
                    }
                    mn = head_sum<G>(L.live ? mn : 0.0f) * inv;
                    mh = H.norm == 2 ? head_sum<G>(L.live ? mh : 0.0f) * inv : 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; i++) e[i] = r * (k[i] - mh - n[i] * mn);
                }
                if (on) L.template store<ES>(y, to + h, e);
            }
        }
    }
    if (!part) return;
    // over the wave's heads, then the workgroup's waves
#pragma unroll
    for (int side = 0; side < 2; side++)
#pragma unroll
        for (int i = 0; i < 8; i++) {
            float a = dw[side][i], b = db[side][i];
#pragma unroll
            for (int o = G; o < 64; o <<= 1) {
                a += __shfl_xor(a, o, 64);
                b += __shfl_xor(b, o, 64);
            }
            if (slot == 0 && L.live) {
                const int c = i < 4 ? L.a + i : L.b + i - 4;
                red[wave][2 * side][c] = a;
                red[wave][2 * side + 1][c] = b;
            }
        }
    __syncthreads();
    for (int e = threadIdx.x; e < 4 * H.D; e += 256) {
        const int k = e / H.D, c = e - k * H.D;
        part[(int64_t)blockIdx.x * 4 * H.D + e] = ((red[0][k][c] + red[1][k][c]) + red[2][k][c]) + red[3][k][c];
    }
}

// dwq, dbq, dwk, dbk [D] from the workgroups' sums: 8 columns and 32 parts of
// the workgroups a workgroup.
__global__ __launch_bounds__(256) void qk_grad_sums_kernel(const float *__restrict__ part, int groups, int D, float *dwq,
                                                           float *dbq, float *dwk, float *dbk) {
    __shared__ float red[32][8];
    const int x = threadIdx.x & 7, k = threadIdx.x >> 3, e = blockIdx.x * 8 + x;
    float sum = 0.0f;
    if (e < 4 * D)
#pragma unroll 8
        for (int g = k; g < groups; g += 32) sum += part[(int64_t)g * 4 * D + e];
    red[k][x] = sum;
    __syncthreads();
    if (k == 0 && e < 4 * D) {
#pragma unroll
        for (int i = 1; i < 32; i++) sum += red[i][x];
        const int which = e / D, c = e - which * D;
        float *out = which == 0 ? dwq : which == 1 ? dbq : which == 2 ? dwk : dbk;
        if (out) out[c] = sum;
    }
}

// How the rows' steps are dealt to waves: at most `most` steps of a row each (as
// evenly as they go), less where `waves` waves are not there yet.
struct QkPlan {
    int sq, steps, per, parts;
    int64_t units;
};
static QkPlan qk_plan(const QkHeads &H, int64_t M, int heads_per_step, int64_t waves, int most) {
    QkPlan p;
    p.sq = (H.nq + heads_per_step - 1) / heads_per_step;
    p.steps = p.sq + (H.nk + heads_per_step - 1) / heads_per_step;
    int64_t per = (M * p.steps + waves - 1) / waves;
    if (per > most) per = most;
    if (per > p.steps) per = p.steps;
    if (per < 1) per = 1;
    p.parts = (int)((p.steps + per - 1) / per);
    p.per = p.parts ? (p.steps + p.parts - 1) / p.parts : 1;
    p.units = M * p.parts;
    return p;
}

// The forward pass of a plan in launches of at most kMaxGroups workgroups, four units
// each, every one of which begins with the first unit of a row: launch i has the rows
// from `row` on and `units` units are left.  False: there is no such launch.
struct QkLaunch {
    int64_t row, units;
    unsigned groups;
};
static bool qk_launch(const QkPlan &p, int64_t i, QkLaunch &l) {
    const int64_t most = kMaxGroups / p.parts * p.parts, first = i * most, groups = (p.units + 3) / 4;
    if (first >= groups) return false;
    l.row = first * 4 / p.parts, l.units = p.units - first * 4;
    l.groups = (unsigned)(groups - first < most ? groups - first : most);
    return true;
}

// Waves and steps of the forward pass (17776 rows of 4 + 4 steps: 2 / 3 / 4 / 8 steps a
// wave 72 / 65 / 61 / 66 us).
static QkPlan qk_forward_plan(const QkHeads &H, int64_t M, int lanes) { return qk_plan(H, M, 64 / lanes, 32768, 4); }

template <int ES, int LAYOUT, int G>
static hipError_t launch_qk_one(hipStream_t s, const QkTensors &T, const QkHeads &H, int64_t M, bool grad, float *part) {
    if (!grad) {
        const QkPlan p = qk_forward_plan(H, M, G);
        QkLaunch l;
        for (int64_t i = 0; qk_launch(p, i, l); i++) {
            QkTensors t = T;
            QkHeads h = H;
            t.q = static_cast<const uint8_t *>(T.q) + l.row * T.ldq * ES;
            t.k = static_cast<const uint8_t *>(T.k) + l.row * T.ldk * ES;
            t.q_out = static_cast<uint8_t *>(T.q_out) + l.row * T.ldq_out * ES;
            t.k_out = static_cast<uint8_t *>(T.k_out) + l.row * T.ldk_out * ES;
            h.table = H.table + l.row * H.P * 2;
            hipLaunchKernelGGL((qk_kernel<ES, LAYOUT, G>), dim3(l.groups), dim3(256), 0, s, t, h, M, p.sq, p.steps, p.per,
                               l.units, p.parts);
        }
        return hipGetLastError();
    }
    // the gradients' waves go on to other rows, and take whole ones
    const QkPlan p = qk_plan(H, M, 64 / G, 8192, 1 << 30);
    const unsigned groups = stride_grid(p.units, 4, kQkGroups);
    hipLaunchKernelGGL((qk_grad_kernel<ES, LAYOUT, G>), dim3(groups), dim3(256), 0, s, T, H, M, p.sq, p.steps, p.per, p.units,
                       p.parts, part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !part) return e;
    hipLaunchKernelGGL(qk_grad_sums_kernel, dim3((4 * H.D + 7) / 8), dim3(256), 0, s, part, (int)groups, H.D, T.dwq, T.dbq,
                       T.dwk, T.dbk);
    return hipGetLastError();
}

// Launch i of a forward pass, for the tests of the split; not part of the ABI.  out:
// parts of a row, first row, units left, workgroups.
extern "C" int dmpq_test_qk_launch(int64_t M, int n_q, int n_k, int dim, int64_t i, int64_t *out) {
    QkHeads H{};
    H.nq = n_q, H.nk = n_k, H.D = dim;
    int lanes = 1;
    while (8 * lanes < dim) lanes *= 2;
    const QkPlan p = qk_forward_plan(H, M, lanes);
    QkLaunch l;
    if (!qk_launch(p, i, l)) return 0;
    out[0] = p.parts, out[1] = l.row, out[2] = l.units, out[3] = l.groups;
    return 1;
}

template <int ES, int LAYOUT>
static hipError_t launch_qk_width(hipStream_t s, const QkTensors &T, const QkHeads &H, int64_t M, bool grad, float *part) {
    const int n = H.D / 8;
    if (n <= 1) return launch_qk_one<ES, LAYOUT, 1>(s, T, H, M, grad, part);
    if (n <= 2) return launch_qk_one<ES, LAYOUT, 2>(s, T, H, M, grad, part);
    if (n <= 4) return launch_qk_one<ES, LAYOUT, 4>(s, T, H, M, grad, part);
    if (n <= 8) return launch_qk_one<ES, LAYOUT, 8>(s, T, H, M, grad, part);
    if (n <= 16) return launch_qk_one<ES, LAYOUT, 16>(s, T, H, M, grad, part);
    return launch_qk_one<ES, LAYOUT, 32>(s, T, H, M, grad, part);
}

size_t qk_grad_bytes(int D) { return (size_t)kQkGroups * 4 * D * sizeof(float); }

hipError_t launch_qk(hipStream_t s, const QkTensors &T, const QkHeads &H, int64_t M, int dtype, bool grad, void *ws) {
    float *part = grad && (T.dwq || T.dbq || T.dwk || T.dbk) ? static_cast<float *>(ws) : nullptr;
    if ((M == 0 || H.nq + H.nk == 0) && !part) return hipSuccess;
    if (dtype == 0) return H.layout == 0 ? launch_qk_width<4, 0>(s, T, H, M, grad, part) : launch_qk_width<4, 1>(s, T, H, M, grad, part);
    return H.layout == 0 ? launch_qk_width<2, 0>(s, T, H, M, grad, part) : launch_qk_width<2, 1>(s, T, H, M, grad, part);
}

}  // namespace dmpq
