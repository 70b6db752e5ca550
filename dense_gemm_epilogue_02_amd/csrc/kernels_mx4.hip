// kernels_mx4.hip -- MXFP4 operands: quantisation, its inverse, and the
// linear layer's product for a few rows (the product of many rows is
// gemm_plan_run_mx's).
#include "block.hpp"

namespace mg {

namespace {

constexpr int QT = 128;   // quantiser tile: QT rows x QT columns, 256 threads

// ---- quantisation ----------------------------------------------------------
//
// scale = 2^(floor(log2 amax) - 2) of 32 elements, code = RNE(x / scale).
// Memory-bound: x is read once and 17/32 of a byte per element and direction
// is written. Blocks along the columns never leave registers: a lane loads
// eight neighbouring elements, four lanes make a block, and its amax takes two
// lane exchanges. Blocks along the rows go through LDS, where a thread reads
// 32 rows of two columns; four neighbouring lanes take the four row blocks of
// the same columns, so that the transposed codes leave in 64-byte pieces.
template <class T, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const T *x, int64_t rows, int64_t cols,
                                                           int64_t ld, int64_t gx, uint8_t *rc, uint8_t *rs,
                                                           uint8_t *cc, uint8_t *cs) {
    constexpr int LW = QT * (int)sizeof(T) / 4 + 1;   // LDS row in words, padded off the banks
    __shared__ uint32_t tile[COLS ? QT * LW : 1];
    const int64_t ty = blockIdx.x / gx, r0 = ty * QT, c0 = (blockIdx.x - ty * gx) * QT;
    const int64_t kpc = mx4_kp(cols), kpr = mx4_kp(rows);
    const int tid = threadIdx.x, seg = tid & 15, rr = tid >> 4;   // 16 lanes x 8 elements a row
    const int64_t c = c0 + seg * 8;
#pragma unroll
    for (int i = 0; i < QT / 16; ++i) {
        const int64_t r = r0 + rr + i * 16;
        Vec8<T> v;
        v.load(x + (r < rows ? r : 0) * ld + (c < cols ? c : 0), r < rows ? cols - c : 0);
        if constexpr (COLS) {
            uint32_t *t = tile + (rr + i * 16) * LW + seg * (2 * sizeof(T));
#pragma unroll
            for (int w = 0; w < Vec8<T>::W; ++w)
#pragma unroll
                for (int j = 0; j < 4; ++j) t[w * 4 + j] = v.w[w][j];
        }
        if constexpr (ROWS) {
            float f[8];
            v.get(f);
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, abs_bits(f[j]));
            m = max(m, (uint32_t)__shfl_xor((int)m, 1));
            m = max(m, (uint32_t)__shfl_xor((int)m, 2));
            const uint32_t byte = mx4_scale_byte(m);
            const uint32_t codes = mx4_pack8(f, mx4_unscale(byte));
            // the row's four bytes of this tile, gathered by its first lane
            const uint32_t b1 = __shfl_down((int)byte, 4), b2 = __shfl_down((int)byte, 8),
                           b3 = __shfl_down((int)byte, 12);
            if (r < rows) {
                *reinterpret_cast<uint32_t *>(rc + (r * kpc + c) / 2) = codes;
                if (seg == 0)
                    *reinterpret_cast<uint32_t *>(rs + (r * kpc + c) / 32) =
                        byte | b1 << 8 | b2 << 16 | b3 << 24;
            }
        }
    }
    if constexpr (COLS) {
        __syncthreads();
        const int rb = tid & 3, cp = tid >> 2;   // row block, pair of columns
        const int64_t col = c0 + cp * 2;
        float f[2][32];
        uint32_t m[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint32_t *t = tile + (rb * 32 + i) * LW + cp * (sizeof(T) / 2);
            T e[2];
            if constexpr (sizeof(T) == 2) {
                __builtin_memcpy(e, t, 4);
            } else {
                __builtin_memcpy(e, t, 4);
                __builtin_memcpy(e + 1, t + 1, 4);
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                f[p][i] = to_f(e[p]);
                m[p] = max(m[p], abs_bits(f[p][i]));
            }
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t byte = mx4_scale_byte(m[p]);
            const float un = mx4_unscale(byte);
            u32x4 q;
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = mx4_pack8(f[p] + 8 * j, un);
            if (col + p < cols) {
                const int64_t at = (col + p) * kpr + r0 + rb * 32;
                *reinterpret_cast<u32x4 *>(cc + at / 2) = q;
                cs[at / 32] = (uint8_t)byte;
            }
        }
    }
}

template <class T>
hipError_t quantize(const T *x, int64_t rows, int64_t cols, int64_t ld, uint8_t *rc, uint8_t *rs,
                    uint8_t *cc, uint8_t *cs, hipStream_t st) {
    // the grid covers the padding of each dimension that is packed
    const int64_t pr = cc ? mx4_kp(rows) : rows, pc = rc ? mx4_kp(cols) : cols;
    const int64_t gx = (pc + QT - 1) / QT, tiles = (pr + QT - 1) / QT * gx;
    if (tiles > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)tiles);
    if (rc && cc)
        mx4_quantize_kernel<T, true, true><<<grid, 256, 0, st>>>(x, rows, cols, ld, gx, rc, rs, cc, cs);
    else if (rc)
        mx4_quantize_kernel<T, true, false><<<grid, 256, 0, st>>>(x, rows, cols, ld, gx, rc, rs, cc, cs);
    else
        mx4_quantize_kernel<T, false, true><<<grid, 256, 0, st>>>(x, rows, cols, ld, gx, rc, rs, cc, cs);
    return hipGetLastError();
}

// ---- the way back -------------------------------------------------------------

// A lane turns one dword of codes into eight values; the code's value times
// its scale is exact in fp32 and rounded once.
template <class T>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint8_t *codes,
                                                             const uint8_t *scales, int64_t rows,
                                                             int64_t k, T *out, int64_t ld) {
    const int64_t per = (k + 7) / 8, kp = mx4_kp(k), n = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, c = (i - r * per) * 8;
        const uint32_t q = *reinterpret_cast<const uint32_t *>(codes + (r * kp + c) / 2);
        const float s = mx4_scale_value(scales[(r * kp + c) / 32]);
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0),
                    b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1),
                    d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2),
                    e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
        const float f[8] = {a[0] * s, a[1] * s, b[0] * s, b[1] * s,
                            d[0] * s, d[1] * s, e[0] * s, e[1] * s};
        Vec8<T> v;
        v.set(f);
        v.store(out + r * ld + c, k - c);
    }
}

// ---- the product of a few rows ---------------------------------------------------
//
// y[m][n] = act(sum_k Q(x)[m][k] W[n][k] + bias[n]) on v_mfma_scale
// 16x16x128: operand A is 16 rows of W, operand B 16 rows of x, so a lane ends
// with four consecutive n of one m. Bound by the one read of W (17/32 byte an
// element). A lane of the instruction holds 32 consecutive k of one row under
// one scale byte, which is exactly an MX block: x is quantised in the lanes
// that multiply it, without any exchange between lanes. A wave takes 256 k at
// a time (a whole 128-byte line of each row of W; lane group g holds the k at
// 64 g .. 64 g + 63), the workgroup's waves take turns over K, and their
// partial sums are added in wave order in LDS.
template <class T, int MT, int NB, int W>
__global__ __launch_bounds__(W * 64) void mx4_few_kernel(const T *x, int64_t ldx, const uint8_t *wc,
                                                         const uint8_t *ws, const __bf16 *bias,
                                                         __bf16 *y, int64_t M, int64_t N, int64_t K,
                                                         int act) {
    __shared__ float part[W][NB * 16][MT * 16 + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (NB * 16), kp = mx4_kp(K), units = kp / 256;
    f32x4 acc[MT][NB];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mt][nb] = f32x4{0, 0, 0, 0};
    const uint8_t *wp[NB], *sp[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int64_t n = min(n0 + nb * 16 + r, N - 1);   // rows past N repeat the last, unused
        wp[nb] = wc + n * (kp / 2) + g * 32;
        sp[nb] = ws + n * (kp / 32) + g * 2;
    }
    for (int64_t u = wave; u < units; u += W) {
        i32x8 a[NB][2];
        uint32_t sa[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const u32x4 lo = *reinterpret_cast<const u32x4 *>(wp[nb] + u * 128),
                        hi = *reinterpret_cast<const u32x4 *>(wp[nb] + u * 128 + 16);
            sa[nb] = *reinterpret_cast<const uint16_t *>(sp[nb] + u * 8);
            a[nb][0] = i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], 0, 0, 0, 0};
            a[nb][1] = i32x8{(int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3], 0, 0, 0, 0};
        }
        const int64_t k0 = u * 256 + g * 64;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int64_t m = min((int64_t)(mt * 16 + r), M - 1);
            const T *xp = x + m * ldx;
            i32x8 b[2];
            uint32_t sb = 0;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                float f[32];
                uint32_t mx = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t k = k0 + s * 32 + j * 8;
                    Vec8<T> v;
                    v.load(xp + (k < K ? k : 0), K - k);
                    v.get(f + 8 * j);
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) mx = max(mx, abs_bits(f[j]));
                const uint32_t byte = mx4_scale_byte(mx);
                const float un = mx4_unscale(byte);
                b[s] = i32x8{(int)mx4_pack8(f, un), (int)mx4_pack8(f + 8, un),
                             (int)mx4_pack8(f + 16, un), (int)mx4_pack8(f + 24, un), 0, 0, 0, 0};
                sb |= byte << (8 * s);
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                acc[mt][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    a[nb][0], b[0], acc[mt][nb], 4, 4, 0, (int)sa[nb], 0, (int)sb);
                acc[mt][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    a[nb][1], b[1], acc[mt][nb], 4, 4, 1, (int)sa[nb], 1, (int)sb);
            }
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[wave][nb * 16 + g * 4 + i][mt * 16 + r] = acc[mt][nb][i];
    __syncthreads();
    for (int i = threadIdx.x; i < NB * 16 * MT * 16; i += W * 64) {
        const int n = i % (NB * 16), m = i / (NB * 16);
        if (m >= M || n0 + n >= N) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += part[w][n][m];
        if (bias) v += (float)bias[n0 + n];
        y[m * N + n0 + n] = (__bf16)apply_act(v, act);
    }
}

template <class T>
hipError_t few(const T *x, int64_t ldx, const uint8_t *wc, const uint8_t *ws, const __bf16 *bias,
               __bf16 *y, int64_t M, int64_t N, int64_t K, int act, hipStream_t st) {
    constexpr int NB = 2, W = 8;
    const int64_t grid = (N + NB * 16 - 1) / (NB * 16);
    if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    if (M <= 16)
        mx4_few_kernel<T, 1, NB, W>
            <<<(unsigned)grid, W * 64, 0, st>>>(x, ldx, wc, ws, bias, y, M, N, K, act);
    else
        mx4_few_kernel<T, 2, NB, W>
            <<<(unsigned)grid, W * 64, 0, st>>>(x, ldx, wc, ws, bias, y, M, N, K, act);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_quantize(const void *x, int type, int64_t rows, int64_t cols, int64_t ld,
                               uint8_t *rc, uint8_t *rs, uint8_t *cc, uint8_t *cs, hipStream_t st) {
    if (type == GEMM_F32)
        return quantize(static_cast<const float *>(x), rows, cols, ld, rc, rs, cc, cs, st);
    if (type == GEMM_F16)
        return quantize(static_cast<const _Float16 *>(x), rows, cols, ld, rc, rs, cc, cs, st);
    return quantize(static_cast<const __bf16 *>(x), rows, cols, ld, rc, rs, cc, cs, st);
}

hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                 int64_t k, void *out, int type, int64_t ld, hipStream_t st) {
    const int64_t jobs = rows * ((k + 7) / 8), wgs = (jobs + 255) / 256;
    const unsigned grid = (unsigned)(wgs < (1 << 20) ? wgs : (1 << 20));
    if (type == GEMM_F32)
        mx4_dequantize_kernel<<<grid, 256, 0, st>>>(codes, scales, rows, k, static_cast<float *>(out), ld);
    else if (type == GEMM_F16)
        mx4_dequantize_kernel<<<grid, 256, 0, st>>>(codes, scales, rows, k, static_cast<_Float16 *>(out), ld);
    else
        mx4_dequantize_kernel<<<grid, 256, 0, st>>>(codes, scales, rows, k, static_cast<__bf16 *>(out), ld);
    return hipGetLastError();
}

hipError_t launch_mx4_few(const void *x, int type, int64_t ldx, const uint8_t *wc,
                          const uint8_t *ws, const void *bias, void *y, int64_t M, int64_t N,
                          int64_t K, int act, hipStream_t st) {
    const __bf16 *b = static_cast<const __bf16 *>(bias);
    __bf16 *d = static_cast<__bf16 *>(y);
    if (type == GEMM_F32)
        return few(static_cast<const float *>(x), ldx, wc, ws, b, d, M, N, K, act, st);
    if (type == GEMM_F16)
        return few(static_cast<const _Float16 *>(x), ldx, wc, ws, b, d, M, N, K, act, st);
    return few(static_cast<const __bf16 *>(x), ldx, wc, ws, b, d, M, N, K, act, st);
}

}  // namespace mg
