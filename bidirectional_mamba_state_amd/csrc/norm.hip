// The norms around a layer of the hybrid (bdssm_gated_norm, bdssm_residual_norm): kernels and
// their host entry points.
//
// Both are one pass over HBM: a row (or one channel group of a row) is read once into float32
// registers, its mean square (LayerNorm: its mean, then the mean square about it) is summed in
// float32 over the lanes that hold it, and the outputs are written once, each rounded once.
//
//   gated:     v = y silu(z);  out = v rsqrt(mean_group(v^2) + eps) w
//              (or, norm first, out = y rsqrt(mean_group(y^2) + eps) w silu(z))
//   residual:  t = o  (post_w given: norm(o) post_w);   r = x + res_scale gate_b t
//              u = norm(r) pre_w gain_b + shift_b
//
// LPR lanes hold a row, VPT pieces of 8 channels each: 16 lanes to 256 channels, a wavefront
// to 2048 (no barrier: the sums stay in one wavefront), a workgroup of four to 16384. Where there
// are too few rows to fill the GPU anyway, a workgroup takes any row of more than 512 channels:
// the time is then one row's chain of loads and sums. Rows of any length and alignment take the
// same path: a global load of 16 bytes needs no more than its element's alignment on gfx950,
// and the last piece of a row is read by elements.
//
// Bound by HBM with many rows (gated, 65,536 x 2,048 bf16 in 8 groups: 137 us, 5.9 TB/s;
// residual, 65,536 x 1,024 bf16: 94 us, 5.7 TB/s; a large copy reaches 4.9), by one row's chain
// of loads and sums with few (32 x 2,048: 3.0 us; 32 x 2,560 with post norm and modulation: 5.0 us).
#include <limits.h>

#include "bdssm.h"
#include "host_checks.h"
#include "internal.h"
#include "mfma_tiles.h"
#include "wave_ops.h"

namespace bdssm {
namespace {

struct GatedArgs {
    const void *y, *z;
    const float *w;  // NULL = ones
    void *out;
    int64_t z_stride;
    int rows, width, groups;
    float eps;
};

struct ResidualArgs {
    const void *x, *o;  // o NULL: r = x
    const float *post_w, *pre_w;
    const void *gate, *gain, *shift;
    void *x_out, *u;
    int64_t mod_stride;
    int rows, width, rps;
    float eps, res_scale;
    int layer;
};

// Eight channels as loaded (one 16-byte piece of bf16, two of float32; the element's alignment
// is enough), and their float32 values. Kept apart so that a load can be issued early and
// waited for where its values are used.
template <typename T>
struct Piece;

template <>
struct Piece<__bf16> {
    typedef __bf16 v __attribute__((ext_vector_type(8), aligned(2)));
    bf16x8 a;
    __device__ __forceinline__ void load(const __bf16 *p) { a = *reinterpret_cast<const v *>(p); }
    __device__ __forceinline__ void set(int k, __bf16 x) { a[k] = x; }
    __device__ __forceinline__ float get(int k) const { return static_cast<float>(a[k]); }
    static __device__ __forceinline__ void store(__bf16 *p, const float (&f)[8])
    {
        *reinterpret_cast<v *>(p) = to_bf16x8(f);
    }
};

template <>
struct Piece<float> {
    typedef float v __attribute__((ext_vector_type(4), aligned(4)));
    f32x4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = *reinterpret_cast<const v *>(p);
        b = *reinterpret_cast<const v *>(p + 4);
    }
    __device__ __forceinline__ void set(int k, float x) { k < 4 ? a[k & 3] = x : b[k & 3] = x; }
    __device__ __forceinline__ float get(int k) const { return k < 4 ? a[k & 3] : b[k & 3]; }
    static __device__ __forceinline__ void store(float *p, const float (&f)[8])
    {
        *reinterpret_cast<v *>(p) = f32x4{f[0], f[1], f[2], f[3]};
        *reinterpret_cast<v *>(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
    }
};

// channels c .. c+7 of a row of n; channels past the end read as zero, their stores are dropped
template <typename T>
__device__ __forceinline__ void load8(const T *p, int c, int n, Piece<T> &f)
{
    if (c + 8 <= n) {
        f.load(p + c);
    } else {
        f = Piece<T>{};
        if (c < n) {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                if (c + k < n)
                    f.set(k, p[c + k]);
        }
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, int c, int n, const float (&f)[8])
{
    if (c + 8 <= n) {
        Piece<T>::store(p + c, f);
    } else if (c < n) {
#pragma unroll
        for (int k = 0; k < 7; ++k)
            if (c + k < n)
                p[c + k] = static_cast<T>(f[k]);
    }
}

// z / (1 + exp(-z)); exp overflows to infinity below z = -88, where the result is -0
__device__ __forceinline__ float silu(float z) { return z * __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// 1 / sqrt(v); the instruction takes numbers below 2^-126 for zero (a row of zeros with an eps
// that small would be 0 x infinity)
__device__ __forceinline__ float inv_sqrt(float v)
{
    const bool tiny = v < 0x1p-126f;
    return __builtin_amdgcn_rsqf(tiny ? v * 0x1p64f : v) * (tiny ? 0x1p32f : 1.f);
}

// Sum over the LPR lanes of a row, in every one of them. `red`: four floats of LDS of this sum's
// own (LPR = 256 only), so that one barrier is enough.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float *red)
{
    v += wave_dpp_move<0x128, 0xf>(v);  // rotations inside 16 lanes by 8, 4, 2, 1
    v += wave_dpp_move<0x124, 0xf>(v);
    v += wave_dpp_move<0x122, 0xf>(v);
    v += wave_dpp_move<0x121, 0xf>(v);
    if (LPR >= 64) {
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
    }
    if (LPR == 256) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = (red[0] + red[1]) + (red[2] + red[3]);
    }
    return v;
}

// x <- (x - mean) * rsqrt(var + eps) (layer) or x * rsqrt(mean(x^2) + eps), over n channels
template <int LPR, int VPT>
__device__ __forceinline__ void normalize(float (&x)[VPT][8], int lane, int n, float eps, int layer, float *red)
{
    const float inv = 1.f / static_cast<float>(n);
    if (layer) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                s += x[i][k];
        const float mu = row_sum<LPR>(s, red) * inv;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[i][k] = (lane + i * LPR) * 8 + k < n ? x[i][k] - mu : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s = fmaf(x[i][k], x[i][k], s);
    const float r = inv_sqrt(row_sum<LPR>(s, red + 4) * inv + eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[i][k] *= r;
}

// Whether weights and modulation are loaded ahead of the sums: in the shapes that few rows take.
// With many rows other rows' loads fill that time, and the registers cost more (65,536 rows of
// 1,024: 95 us, 118 us with everything ahead).
template <int LPR, int VPT>
constexpr bool kAhead = LPR == 256 && VPT <= 2;

// Workgroup number in a grid folded over y (the threads along x have to fit 32 bits)
__device__ __forceinline__ int64_t block_index()
{
    return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
}

// The lane's VPT pieces of a row of n channels, loaded ahead (AHEAD) or when they are used.
template <typename T, int LPR, int VPT, bool AHEAD>
struct RowLoad {
    const T *p;
    int lane, n;
    Piece<T> f[AHEAD ? VPT : 1];
    __device__ __forceinline__ RowLoad(const T *row, int lane_, int n_) : p(row), lane(lane_), n(n_)
    {
        if (AHEAD && p) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                load8(p, (lane + i * LPR) * 8, n, f[AHEAD ? i : 0]);
        }
    }
    __device__ __forceinline__ void get(int i, float (&x)[8])
    {
        if (!AHEAD)
            load8(p, (lane + i * LPR) * 8, n, f[0]);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = f[AHEAD ? i : 0].get(k);
    }
    __device__ __forceinline__ void values(float (&x)[VPT][8])
    {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            get(i, x[i]);
    }
    __device__ __forceinline__ void multiply(float (&x)[VPT][8])  // x *= the row; nothing where it is NULL
    {
        if (!p)
            return;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float w[8];
            get(i, w);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[i][k] *= w[k];
        }
    }
};

template <typename Ty, typename T, int LPR, int VPT, bool NORM_FIRST>
__global__ __launch_bounds__(256) void k_gated_norm(GatedArgs a)
{
    __shared__ float red[8];
    constexpr int RPW = 256 / LPR;
    const int64_t unit = block_index() * RPW + threadIdx.x / LPR;
    const int lane = threadIdx.x % LPR;
    if (unit >= static_cast<int64_t>(a.rows) * a.groups)
        return;  // never part of a workgroup that has a barrier (LPR = 256: one row each)
    const int64_t row = unit / a.groups;
    const int n = a.width / a.groups, c0 = static_cast<int>(unit % a.groups) * n;
    const Ty *y = static_cast<const Ty *>(a.y) + row * a.width + c0;
    const T *z = static_cast<const T *>(a.z) + row * a.z_stride + c0;
    RowLoad<Ty, LPR, VPT, true> y_row(y, lane, n);
    RowLoad<T, LPR, VPT, true> z_row(z, lane, n);
    RowLoad<float, LPR, VPT, kAhead<LPR, VPT>> weight(a.w ? a.w + c0 : nullptr, lane, n);
    float v[VPT][8], g[VPT][8];
    y_row.values(v);
    z_row.values(g);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            g[i][k] = silu(g[i][k]);
            if (!NORM_FIRST)
                v[i][k] *= g[i][k];
        }
    normalize<LPR, VPT>(v, lane, n, a.eps, 0, red);
    weight.multiply(v);
    T *out = static_cast<T *>(a.out) + row * a.width + c0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (NORM_FIRST) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[i][k] *= g[i][k];
        }
        store8(out, (lane + i * LPR) * 8, n, v[i]);
    }
}

template <typename Tx, typename T, int LPR, int VPT>
__global__ __launch_bounds__(256) void k_residual_norm(ResidualArgs a)
{
    __shared__ float red[16];
    constexpr int RPW = 256 / LPR;
    const int64_t row = block_index() * RPW + threadIdx.x / LPR;
    const int lane = threadIdx.x % LPR, n = a.width;
    if (row >= a.rows)
        return;
    const Tx *x = static_cast<const Tx *>(a.x) + row * n;
    const int64_t mod = static_cast<int64_t>(static_cast<int>(row) / a.rps) * a.mod_stride;
    auto modulation = [&](const void *p) { return p ? static_cast<const T *>(p) + mod : nullptr; };
    constexpr bool AHEAD = kAhead<LPR, VPT>;
    RowLoad<Tx, LPR, VPT, true> x_row(x, lane, n);
    RowLoad<T, LPR, VPT, true> o_row(a.o ? static_cast<const T *>(a.o) + row * n : nullptr, lane, n);
    RowLoad<float, LPR, VPT, AHEAD> post_w(a.post_w, lane, n), pre_w(a.pre_w, lane, n);
    RowLoad<T, LPR, VPT, AHEAD> gate(modulation(a.gate), lane, n), gain(modulation(a.gain), lane, n),
        shift(modulation(a.shift), lane, n);
    float r[VPT][8], t[VPT][8];
    x_row.values(r);
    if (a.o) {
        o_row.values(t);
        if (a.post_w) {
            normalize<LPR, VPT>(t, lane, n, a.eps, a.layer, red);
            post_w.multiply(t);
        }
        gate.multiply(t);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                r[i][k] = fmaf(a.res_scale, t[i][k], r[i][k]);
    }
    if (a.x_out) {
        Tx *xo = static_cast<Tx *>(a.x_out) + row * n;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            store8(xo, (lane + i * LPR) * 8, n, r[i]);
    }
    if (!a.u)
        return;
    normalize<LPR, VPT>(r, lane, n, a.eps, a.layer, red + 8);
    pre_w.multiply(r);
    gain.multiply(r);
    T *u = static_cast<T *>(a.u) + row * n;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (a.shift) {
            float w[8];
            shift.get(i, w);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                r[i][k] += w[k];
        }
        store8(u, (lane + i * LPR) * 8, n, r[i]);
    }
}

// f<LPR, VPT>(): the lanes of a row and the pieces of a lane for `rows` rows of n channels. Few
// rows: less than two workgroups per CU with a row each (32 rows of 2,048: 4.9 us with a
// wavefront per row, 3.9 us with a workgroup).
template <typename F>
hipError_t by_width(int64_t rows, int n, F f)
{
    const int pieces = (n + 7) / 8;
    const bool few = rows <= 2 * device_cus();
    if (few && pieces > 64 && pieces <= 256)
        return f.template operator()<256, 1>();
    if (pieces <= 32)
        return f.template operator()<16, 2>();
    if (pieces <= 64)
        return f.template operator()<64, 1>();
    if (pieces <= 128)
        return f.template operator()<64, 2>();
    if (pieces <= 256)
        return f.template operator()<64, 4>();
    if (pieces <= 512)
        return f.template operator()<256, 2>();
    if (pieces <= 1024)
        return f.template operator()<256, 4>();
    return f.template operator()<256, 8>();
}

template <int LPR>
dim3 grid_of(int64_t units)
{
    constexpr int RPW = 256 / LPR;
    const int64_t blocks = (units + RPW - 1) / RPW, x = blocks < (1 << 20) ? blocks : (1 << 20);
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>((blocks + x - 1) / x));
}

template <typename Ty, typename T>
struct LaunchGated {
    GatedArgs a;
    bool norm_first;
    hipStream_t st;
    template <int LPR, int VPT>
    hipError_t operator()() const
    {
        const dim3 g = grid_of<LPR>(static_cast<int64_t>(a.rows) * a.groups);
        if (norm_first)
            k_gated_norm<Ty, T, LPR, VPT, true><<<g, 256, 0, st>>>(a);
        else
            k_gated_norm<Ty, T, LPR, VPT, false><<<g, 256, 0, st>>>(a);
        return hipGetLastError();
    }
};

template <typename Tx, typename T>
struct LaunchResidual {
    ResidualArgs a;
    hipStream_t st;
    template <int LPR, int VPT>
    hipError_t operator()() const
    {
        k_residual_norm<Tx, T, LPR, VPT><<<grid_of<LPR>(a.rows), 256, 0, st>>>(a);
        return hipGetLastError();
    }
};

constexpr int kMaxNormWidth = 16384;

bdssm_status check_norm(const bdssm_norm_dims *d)
{
    if (!d)
        return BDSSM_ERR_NULL;
    if (d->rows < 0 || d->width < 1 || d->groups < 1 || d->width % d->groups != 0)
        return BDSSM_ERR_SHAPE;
    if ((d->dtype != BDSSM_F32 && d->dtype != BDSSM_BF16) || (d->x_dtype != BDSSM_F32 && d->x_dtype != BDSSM_BF16) ||
        (d->x_dtype == BDSSM_BF16 && d->dtype == BDSSM_F32))
        return BDSSM_ERR_UNSUPPORTED;
    if ((d->kind != BDSSM_NORM_RMS && d->kind != BDSSM_NORM_LAYER) || !(d->eps > 0.f))
        return BDSSM_ERR_UNSUPPORTED;
    if (d->width / d->groups > kMaxNormWidth || d->rows > INT_MAX / d->groups)
        return BDSSM_ERR_UNSUPPORTED;
    return BDSSM_OK;
}

// bytes from the first to past the last element of `rows` rows of `width`, `stride` apart
int64_t span(int64_t rows, int64_t stride, int64_t width, int e)
{
    return rows > 0 ? ((rows - 1) * stride + width) * e : 0;
}

// whether span() of these is a number of 64 bits
bool span_fits(int64_t rows, int64_t stride, int64_t width, int e)
{
    return rows <= 1 || stride <= (INT64_MAX / e - width) / (rows - 1);
}

bool element_aligned(const void *p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (elt(dtype) - 1)) == 0; }

}  // namespace
}  // namespace bdssm

using namespace bdssm;

extern "C" bdssm_status bdssm_gated_norm(const bdssm_norm_dims *dims, const void *y, const void *z, int64_t z_stride,
                                         const float *weight, int32_t norm_first, void *out, void *stream)
{
    bdssm_status rc = check_norm(dims);
    if (rc != BDSSM_OK)
        return rc;
    if (dims->rows > 0 && (!y || !z || !out))  // an empty tensor may have no address
        return BDSSM_ERR_NULL;
    if (z_stride < dims->width)
        return BDSSM_ERR_SHAPE;
    if (dims->kind != BDSSM_NORM_RMS || (norm_first != 0 && norm_first != 1))
        return BDSSM_ERR_UNSUPPORTED;
    if (!element_aligned(y, dims->x_dtype) || !element_aligned(z, dims->dtype) || !element_aligned(out, dims->dtype) ||
        !element_aligned(weight, BDSSM_F32))
        return BDSSM_ERR_ALIGN;
    const int64_t n = dims->rows * dims->width;
    const int e = elt(dims->dtype);
    if (!span_fits(dims->rows, z_stride, dims->width, e))
        return BDSSM_ERR_UNSUPPORTED;
    const Range ro = rng(out, n * e), ry = rng(y, n * elt(dims->x_dtype));
    if (overlap(ro, rng(z, span(dims->rows, z_stride, dims->width, e))) || overlap(ro, rng(weight, dims->width * 4ll)) ||
        (overlap(ro, ry) && !(out == y && dims->dtype == dims->x_dtype)))
        return BDSSM_ERR_ALIAS;
    if (n == 0)
        return BDSSM_OK;
    const GatedArgs a{y, z, weight, out, z_stride, static_cast<int>(dims->rows), dims->width, dims->groups, dims->eps};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int w = dims->width / dims->groups;
    if (dims->dtype == BDSSM_F32)
        return launched(by_width(dims->rows * dims->groups, w, LaunchGated<float, float>{a, norm_first != 0, st}));
    if (dims->x_dtype == BDSSM_F32)
        return launched(by_width(dims->rows * dims->groups, w, LaunchGated<float, __bf16>{a, norm_first != 0, st}));
    return launched(by_width(dims->rows * dims->groups, w, LaunchGated<__bf16, __bf16>{a, norm_first != 0, st}));
}

extern "C" bdssm_status bdssm_residual_norm(const bdssm_norm_dims *dims, const bdssm_residual *r, void *x_out, void *u,
                                            void *stream)
{
    bdssm_status rc = check_norm(dims);
    if (rc != BDSSM_OK)
        return rc;
    if (!r || (dims->rows > 0 && (!r->x || (!x_out && !u))))
        return BDSSM_ERR_NULL;
    const bool mod = r->gate || r->gain || r->shift;
    if (dims->groups != 1 || (mod && (dims->rows_per_stream < 1 || r->mod_stride < dims->width)))
        return BDSSM_ERR_SHAPE;
    for (const void *p : {r->o, r->gate, r->gain, r->shift, static_cast<const void *>(u)})
        if (!element_aligned(p, dims->dtype))
            return BDSSM_ERR_ALIGN;
    for (const void *p : {r->x, static_cast<const void *>(x_out)})
        if (!element_aligned(p, dims->x_dtype))
            return BDSSM_ERR_ALIGN;
    if (!element_aligned(r->post_w, BDSSM_F32) || !element_aligned(r->pre_w, BDSSM_F32))
        return BDSSM_ERR_ALIGN;
    const int64_t n = dims->rows * dims->width;
    const int e = elt(dims->dtype), xe = elt(dims->x_dtype);
    const int64_t streams = mod ? (dims->rows + dims->rows_per_stream - 1) / dims->rows_per_stream : 0;
    if (!span_fits(streams, r->mod_stride, dims->width, e))
        return BDSSM_ERR_UNSUPPORTED;
    const int64_t mb = span(streams, r->mod_stride, dims->width, e);
    const Range rx = rng(r->x, n * xe), rxo = rng(x_out, n * xe), ru = rng(u, n * e);
    for (Range q : {rxo, ru}) {
        if (overlap(q, rng(r->o, n * e)) || overlap(q, rng(r->post_w, dims->width * 4ll)) ||
            overlap(q, rng(r->pre_w, dims->width * 4ll)) || overlap(q, rng(r->gate, mb)) ||
            overlap(q, rng(r->gain, mb)) || overlap(q, rng(r->shift, mb)))
            return BDSSM_ERR_ALIAS;
    }
    if (overlap(rxo, ru) || overlap(ru, rx) || (overlap(rxo, rx) && x_out != r->x))
        return BDSSM_ERR_ALIAS;
    if (n == 0)
        return BDSSM_OK;
    const ResidualArgs a{r->x, r->o, r->post_w, r->pre_w, r->gate, r->gain, r->shift, x_out, u, r->mod_stride,
                         static_cast<int>(dims->rows), dims->width, mod ? dims->rows_per_stream : 1, dims->eps,
                         r->res_scale, dims->kind == BDSSM_NORM_LAYER};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (dims->dtype == BDSSM_F32)
        return launched(by_width(dims->rows, dims->width, LaunchResidual<float, float>{a, st}));
    if (dims->x_dtype == BDSSM_F32)
        return launched(by_width(dims->rows, dims->width, LaunchResidual<float, __bf16>{a, st}));
    return launched(by_width(dims->rows, dims->width, LaunchResidual<__bf16, __bf16>{a, st}));
}
