// RMS norm with the residual's addition and an 8-bit output, and its backward.
//
//   h = x + residual          (rounded to the residual's type)
//   r = 1 / sqrt(mean(h^2) + eps),  n = h r,  y = n weight
//   8-bit output: blocks of 32 elements of y (MOE_Q_OUTPUT) or of n
//   (MOE_Q_NORMALIZED, the checkpoint the backward reads) as e4m3 codes with
//   one e8m0 scale 2^e, e the least with max|v| <= 448 2^e.
//   backward: g = dy weight,  dh = dres + r (g - n mean(g n)),
//             dweight = sum over tokens of dy n
//
// Both directions are bound by HBM traffic: every input is read once into
// registers and every output written once.
#include "train/train.hpp"

namespace moe {

namespace {

constexpr int kNormMaxWaves = 16;

// Waves per row and chunks of 8 elements per lane for a row of H elements:
// two chunks (32 bytes of bf16, two loads in flight per stream) up to 16 waves
// of them, then eight.
struct RowShape {
    int v, waves;
};
RowShape row_shape(int H) {
    if (H <= 2 * 8 * kWave * kNormMaxWaves) return {2, (H + 2 * 8 * kWave - 1) / (2 * 8 * kWave)};
    return {8, (H + 8 * 8 * kWave - 1) / (8 * 8 * kWave)};
}

// A double as the float with the same leading 21 significant bits, the last
// of them set when anything below was cut off.  Rounding that float to the 4
// bits of e4m3 or the 8 of bf16, and comparing it with 448 2^e, gives what
// the double itself would: no second rounding moves a value over a border.
__device__ __forceinline__ float sticky_f32(double d) {
    const uint64_t u = __builtin_bit_cast(uint64_t, d);
    const uint32_t lo = (uint32_t)u, hi = (uint32_t)(u >> 32) | (lo != 0u ? 1u : 0u);
    return (float)__builtin_bit_cast(double, (uint64_t)hi << 32);
}

// Least e with amax <= 448 2^e, clamped to e8m0's [-127, 127]; amax finite.
__device__ __forceinline__ int mx_exponent(float amax) {
    int e = (int)((__float_as_uint(amax) >> 23) & 255u) - 127 - 8;   // amax / 2^e in [256, 512)
    if (amax > ldexpf(448.0f, e)) ++e;
    return e < -127 ? -127 : (e > 127 ? 127 : e);
}

// Block maximum over the four lanes that hold 32 consecutive elements, on the
// magnitudes' bits (a NaN or an infinity is above every finite value).
__device__ __forceinline__ uint32_t quad_max_bits(uint32_t m) {
    const uint32_t a = (uint32_t)dpp_mov<kDppXor1>((int)m);
    m = m > a ? m : a;
    const uint32_t b = (uint32_t)dpp_mov<kDppXor2>((int)m);
    return m > b ? m : b;
}

// Codes of eight values and the scale byte of their 32-element block (every
// lane of the four must call it).  A block with a non-finite value is NaN
// throughout: scale 255, codes 0x7f.
__device__ __forceinline__ uint2 mx_encode(const float *f, uint32_t *scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(f[i]) & 0x7fffffffu;
        m = m > u ? m : u;
    }
    m = quad_max_bits(m);
    if (m >= 0x7f800000u) {
        *scale = 255u;
        return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    }
    const int e = mx_exponent(__uint_as_float(m));
    *scale = (uint32_t)(e + 127);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(ldexpf(f[i], -e), -448.0f), 448.0f);
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], b, true);
    return make_uint2((uint32_t)a, (uint32_t)b);
}

__device__ __forceinline__ float as_stored(float, float v) { return v; }
__device__ __forceinline__ float as_stored(Bf16, float v) { return (float)(__bf16)v; }

// One block per token, the row in registers.  The square sum and the 8-bit
// output's values are in 64 bits: the sum cannot overflow whatever the type
// holds, and a code is the one the exact value rounds to.
template <int V, typename X, typename R>
__global__ __launch_bounds__(1024) void rms_norm(NormArgs a) {
    __shared__ double part[kNormMaxWaves];
    const size_t row = blockIdx.x;
    const int tid = threadIdx.x, nthr = blockDim.x, nch = a.H / 8;
    const size_t base = row * (size_t)a.H;
    Raw8<X> rx[V];
    Raw8<R> rr[V];
    Raw8<float> rw[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = tid + j * nthr;
        if (c < nch) {
            rx[j].load(a.x, base + 8 * c);
            if (a.res) rr[j].load(a.res, base + 8 * c);
            rw[j].load(a.weight, 8 * c);
        } else {
            rx[j].zero();
            rr[j].zero();
            rw[j].zero();
        }
    }
    float h[V][8];
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        rx[j].get(h[j]);
        if (a.res) {
            float r[8];
            rr[j].get(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[j][i] = as_stored(R{}, h[j][i] + r[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[j][i] = as_stored(R{}, h[j][i]);
        }
        const int c = tid + j * nthr;
        if (a.res_out && c < nch) store8(R{}, a.res_out, base + 8 * c, h[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double d = (double)h[j][i];
            s = fma(d, d, s);
        }
    }
    s = wave_sum_f64(s);
    if (nthr > kWave) {
        if ((tid & 63) == 0) part[tid >> 6] = s;
        __syncthreads();
        s = 0.0;
        for (int w = 0; w < nthr / kWave; ++w) s += part[w];
    }
    const double r = 1.0 / sqrt(s / (double)a.H + (double)a.eps);
    if (a.rstd && tid == 0) a.rstd[row] = (float)r;
    const float rf = (float)r;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = tid + j * nthr;
        float w[8], y[8];
        rw[j].get(w);
        if (a.q_kind == MOE_Q_NONE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = h[j][i] * rf * w[i];
        } else {
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const double n = (double)h[j][i] * r;
                const float v = sticky_f32(n * (double)w[i]);
                q[i] = a.q_kind == MOE_Q_OUTPUT ? v : sticky_f32(n);
                y[i] = v;
            }
            uint32_t sc;
            const uint2 codes = mx_encode(q, &sc);   // H % 32 == 0: the four lanes of a block are in or out together
            if (c < nch) {
                *reinterpret_cast<uint2 *>(a.codes + base + 8 * c) = codes;
                if ((c & 3) == 0) a.scales[(base >> 5) + (c >> 2)] = (uint8_t)sc;
            }
        }
        if (a.y && c < nch) store8(Bf16{}, a.y, base + 8 * c, y);
    }
}

template <int V, typename X>
hipError_t norm_v(const NormArgs &a, int waves, hipStream_t st) {
    const dim3 g(a.T), b(kWave * waves);
    if (a.res_dtype == MOE_OUT_F32)
        MOE_LAUNCH("rms_norm", (rms_norm<V, X, float>), g, b, 0, st, a);
    else
        MOE_LAUNCH("rms_norm", (rms_norm<V, X, Bf16>), g, b, 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs &a, hipStream_t st) {
    const RowShape r = row_shape(a.H);
    const bool xf = a.x_dtype == MOE_OUT_F32;
    if (r.v == 2) return xf ? norm_v<2, float>(a, r.waves, st) : norm_v<2, Bf16>(a, r.waves, st);
    return xf ? norm_v<8, float>(a, r.waves, st) : norm_v<8, Bf16>(a, r.waves, st);
}

// ---------------------------------------------------------------------------
// Backward.  Block b takes the tokens b, b + blocks, ...; every thread keeps
// the same columns for all of them, so dweight's sums over tokens stay in
// registers until the end: one partial row per block, added by column_sum.
// ---------------------------------------------------------------------------
namespace {

// Blocks (partial rows of dweight).  A constant, so that the order of the sums
// depends on the sizes alone.
constexpr int kNormBwdBlocks = 512;

int norm_bwd_blocks(int T) { return T < kNormBwdBlocks ? T : kNormBwdBlocks; }

template <typename S>
__device__ __forceinline__ void load_src(Raw8<S> &r, const NormBwdArgs &a, size_t i) {
    if constexpr (__is_same(S, Mx8))
        r.load2(a.codes, a.scales, i);
    else
        r.load(a.h, i);
}

template <int V, typename DY, typename S, typename DR, typename DX>
__global__ __launch_bounds__(1024) void rms_norm_backward(NormBwdArgs a, float *__restrict__ dwpart) {
    __shared__ float part[2][kNormMaxWaves];
    const int tid = threadIdx.x, nthr = blockDim.x, nch = a.H / 8, nw = nthr / kWave;
    float w[V][8], dw[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = tid + j * nthr;
        Raw8<float> rw;
        if (c < nch)
            rw.load(a.weight, 8 * c);
        else
            rw.zero();
        rw.get(w[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
    }
    int par = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, par ^= 1) {
        const size_t base = (size_t)t * a.H;
        if (a.mask && a.mask[t] == 0) {   // the same for the whole block
            const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = tid + j * nthr;
                if (a.dx && c < nch) store8(DX{}, a.dx, base + 8 * c, z);
            }
            par ^= 1;   // no barrier was passed: keep the parity
            continue;
        }
        Raw8<DY> ry[V];
        Raw8<S> rs[V];
        Raw8<DR> rd[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = tid + j * nthr;
            if (c < nch) {
                ry[j].load(a.dy, base + 8 * c);
                load_src<S>(rs[j], a, base + 8 * c);
                if (a.dres) rd[j].load(a.dres, base + 8 * c);
            } else {
                ry[j].zero();
                rs[j].zero();
                rd[j].zero();
            }
        }
        const float r = a.rstd[t];
        float dy[V][8], n[V][8];
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            ry[j].get(dy[j]);
            rs[j].get(n[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (!__is_same(S, Mx8)) n[j][i] *= r;
                dw[j][i] = fmaf(dy[j][i], n[j][i], dw[j][i]);
                dy[j][i] *= w[j][i];
                s = fmaf(dy[j][i], n[j][i], s);
            }
        }
        if (a.dx == nullptr) {
            par ^= 1;
            continue;
        }
        s = wave_sum(s);
        if (nw > 1) {
            // two slots in turn: a slot is written again only after the
            // barrier of the row between, which its readers have reached
            if ((tid & 63) == 0) part[par][tid >> 6] = s;
            __syncthreads();
            s = 0.f;
            for (int q = 0; q < nw; ++q) s += part[par][q];
        }
        const float m = s / (float)a.H;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = tid + j * nthr;
            float d[8], o[8];
            if (a.dres)
                rd[j].get(d);
            else {
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(r, dy[j][i] - n[j][i] * m, d[i]);
            if (c < nch) store8(DX{}, a.dx, base + 8 * c, o);
        }
    }
    if (a.dweight) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = tid + j * nthr;
            if (c < nch) store8(float{}, dwpart, (size_t)blockIdx.x * a.H + 8 * c, dw[j]);
        }
    }
}

// Column sums: block = 64 columns, sixteen waves take the rows w, w + 16, ...,
// eight in flight each.
__global__ __launch_bounds__(1024) void column_sum(const float *__restrict__ part, int R, int C,
                                                   float *__restrict__ out) {
    __shared__ float lds[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane, cc = c < C ? c : C - 1;
    float s = 0.f;
    for (int r = wave; r < R; r += 128) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = part[(size_t)(r + 16 * i < R ? r + 16 * i : r) * C + cc];
#pragma unroll
        for (int i = 0; i < 8; ++i) s += r + 16 * i < R ? v[i] : 0.f;
    }
    lds[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < C) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = (lds[4 * i][lane] + lds[4 * i + 1][lane]) + (lds[4 * i + 2][lane] + lds[4 * i + 3][lane]);
        out[c] = (v[0] + v[1]) + (v[2] + v[3]);
    }
}

template <int V, typename DY, typename S, typename DR>
void bwd_dx(const NormBwdArgs &a, int waves, float *part, hipStream_t st) {
    const dim3 g(norm_bwd_blocks(a.T)), b(kWave * waves);
    if (a.dx_dtype == MOE_OUT_F32)
        MOE_LAUNCH("rms_norm_backward", (rms_norm_backward<V, DY, S, DR, float>), g, b, 0, st, a, part);
    else
        MOE_LAUNCH("rms_norm_backward", (rms_norm_backward<V, DY, S, DR, Bf16>), g, b, 0, st, a, part);
}
template <int V, typename DY, typename S>
void bwd_dr(const NormBwdArgs &a, int waves, float *part, hipStream_t st) {
    if (a.dres_dtype == MOE_OUT_F32)
        bwd_dx<V, DY, S, float>(a, waves, part, st);
    else
        bwd_dx<V, DY, S, Bf16>(a, waves, part, st);
}
template <int V, typename DY>
void bwd_src(const NormBwdArgs &a, int waves, float *part, hipStream_t st) {
    if (a.h == nullptr)
        bwd_dr<V, DY, Mx8>(a, waves, part, st);
    else if (a.h_dtype == MOE_OUT_F32)
        bwd_dr<V, DY, float>(a, waves, part, st);
    else
        bwd_dr<V, DY, Bf16>(a, waves, part, st);
}
template <int V>
void bwd_dy(const NormBwdArgs &a, int waves, float *part, hipStream_t st) {
    if (a.dy_dtype == MOE_OUT_F32)
        bwd_src<V, float>(a, waves, part, st);
    else
        bwd_src<V, Bf16>(a, waves, part, st);
}

}  // namespace

hipError_t launch_column_sum(const char *name, const float *part, int R, int C, float *out, hipStream_t st) {
    MOE_LAUNCH(name, column_sum, dim3((C + 63) / 64), dim3(1024), 0, st, part, R, C, out);
    return hipGetLastError();
}

size_t norm_bwd_ws_bytes(int T, int H) { return WsLayout::up((size_t)norm_bwd_blocks(T) * H * 4); }

hipError_t launch_rms_norm_backward(const NormBwdArgs &a, char *ws, hipStream_t st) {
    const RowShape r = row_shape(a.H);
    float *part = reinterpret_cast<float *>(ws);
    if (a.T > 0) {
        if (r.v == 2)
            bwd_dy<2>(a, r.waves, part, st);
        else
            bwd_dy<8>(a, r.waves, part, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dweight) return launch_column_sum("dweight_sum", part, norm_bwd_blocks(a.T), a.H, a.dweight, st);
    return hipSuccess;
}

}  // namespace moe
