// kernels_mx4.hip -- MXFP4 operands: quantisation, its inverse, and the
// linear layer's product for a few rows (the product of many rows is
// gemm_plan_run_mx's).
#include "block.hpp"

namespace mg {

namespace {

constexpr int QT = 128;   // columns of a quantiser tile, of 256 threads

// ---- quantisation ----------------------------------------------------------
//
// scale = 2^(floor(log2 amax) - 2) of 32 elements, code = RNE(x / scale).
// Memory-bound: x is read once and 17/32 of a byte per element and direction
// is written. A thread asks for all its rows before it uses the first. Blocks
// along the columns never leave registers: a lane holds eight neighbouring
// elements, four lanes make a block. Blocks along the rows go through LDS,
// where a thread reads the 32 rows of a block of one column; the column's other
// block is its neighbour's, so that the transposed codes leave in 32-byte
// pieces. Tiles are small, so that few rows still fill the chip: of 128 rows,
// 777 x 1000 fp16 took 5.6 us in both directions against 3.8, and 4096 x 8192
// bf16 28.2 against 25.9 (now 23.5, 20.6 for the bytes); along the rows alone 21.8
// against 19.9 for 32 rows, along the columns alone 19.4 for 64, 21.2 for 32.
// Two matrices share a launch (the first `na` workgroups are a's): the gradients
// of 777 x 1000 x 2057 took 34.4 us with two launches, 31.3 with one. Where COLS
// is set, a matrix whose rc is null is not packed along its columns.
template <class T, bool ROWS, bool COLS, bool EVEN>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(Mx4Quant a, Mx4Quant b, unsigned na) {
    const bool second = blockIdx.x >= na;
    const unsigned block = second ? blockIdx.x - na : blockIdx.x;
    const T *const x = static_cast<const T *>(second ? b.x : a.x);
    const int64_t rows = second ? b.rows : a.rows, cols = second ? b.cols : a.cols, ld = second ? b.ld : a.ld;
    uint8_t *const rc = second ? b.rc : a.rc, *const rs = second ? b.rs : a.rs;
    uint8_t *const cc = second ? b.cc : a.cc, *const cs = second ? b.cs : a.cs;
    constexpr int QR = COLS ? 64 : 32;                // rows of a tile
    constexpr int LW = QT * (int)sizeof(T) / 4 + 1;   // LDS row in words, padded off the banks
    constexpr int RPT = QR / 16;                      // rows of a thread
    __shared__ uint32_t tile[COLS ? QR * LW : 1];
    const int64_t kpc = mx4_kp(cols), kpr = mx4_kp(rows);
    const unsigned gx = (unsigned)(((ROWS && rc ? kpc : cols) + QT - 1) / QT), ty = block / gx;
    const int64_t r0 = (int64_t)ty * QR, c0 = (int64_t)(block - ty * gx) * QT;
    const int tid = threadIdx.x, seg = tid & 15, rr = tid >> 4;   // 16 lanes x 8 elements a row
    const int64_t c = c0 + seg * 8;
    Vec8<T> v[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int64_t r = min(r0 + rr + i * 16, rows - 1);
        fetch_row<EVEN>(v[i], x + r * ld, c, cols);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int64_t r = r0 + rr + i * 16;
        float f[8];
        row_values<EVEN>(v[i], f, r < rows ? c : cols, cols);
        if constexpr (COLS) {
            Vec8<T> q;
            q.set(f);   // exact: the values came from T
            uint32_t *t = tile + (rr + i * 16) * LW + seg * (2 * sizeof(T));
#pragma unroll
            for (int w = 0; w < Vec8<T>::W; ++w)
#pragma unroll
                for (int j = 0; j < 4; ++j) t[w * 4 + j] = q.w[w][j];
        }
        if (ROWS && (!COLS || rc)) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, abs_bits(f[j]));
            const uint32_t byte = mx4_scale_byte(max_of_four(m));
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
        const int rb = tid & 1, j0 = tid >> 1;   // row block and column of the tile
        const int64_t col = c0 + j0;
        float f[32];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            f[i] = to_f(reinterpret_cast<const T *>(tile + (rb * 32 + i) * LW)[j0]);
            m = max(m, abs_bits(f[i]));
        }
        const uint32_t byte = mx4_scale_byte(m);
        const float un = mx4_unscale(byte);
        u32x4 q;
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = mx4_pack8(f + 8 * j, un);
        if (col < cols) {
            const int64_t at = col * kpr + r0 + rb * 32;
            *reinterpret_cast<u32x4 *>(cc + at / 2) = q;
            cs[at / 32] = (uint8_t)byte;
        }
    }
}

// Tiles of a matrix: they cover the padding of each dimension that is packed.
int64_t quant_tiles(const Mx4Quant &a, bool with_cols) {
    const int64_t pr = a.cc ? mx4_kp(a.rows) : a.rows, pc = a.rc ? mx4_kp(a.cols) : a.cols, qr = with_cols ? 64 : 32;
    return (pc + QT - 1) / QT * ((pr + qr - 1) / qr);
}
template <class T, bool EVEN> hipError_t quantize(const Mx4Quant &a, const Mx4Quant *b, hipStream_t st) {
    const int64_t na = quant_tiles(a, a.cc != nullptr), n = na + (b ? quant_tiles(*b, true) : 0);
    if (n > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    const Mx4Quant &c = b ? *b : a;
    if (a.rc && a.cc)
        mx4_quantize_kernel<T, true, true, EVEN><<<(unsigned)n, 256, 0, st>>>(a, c, (unsigned)na);
    else if (a.rc)
        mx4_quantize_kernel<T, true, false, EVEN><<<(unsigned)n, 256, 0, st>>>(a, c, (unsigned)na);
    else
        mx4_quantize_kernel<T, false, true, EVEN><<<(unsigned)n, 256, 0, st>>>(a, c, (unsigned)na);
    return hipGetLastError();
}
template <class T> hipError_t quantize(const Mx4Quant &a, const Mx4Quant *b, hipStream_t st) {
    return a.cols % 8 == 0 && (!b || b->cols % 8 == 0) ? quantize<T, true>(a, b, st) : quantize<T, false>(a, b, st);
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
// element). A lane of the instruction holds 32 k of one row under one scale
// byte, which is exactly an MX block. The workgroup's waves share K in runs of
// units of 256 k (a line of codes of each row); a wave loads whole lines,
// several units ahead, and turns them through LDS of its own, since lanes that
// load what they multiply would touch a line each. The waves' sums are added in
// wave order.
//
// x comes quantised (XS = 0, XB blocks of 16 rows), or a wave quantises its own
// units of XS pairs of rows, 32 lanes a row and four a block. The latter saves a
// launch but is done by every workgroup.
// NB: blocks of 16 rows of W; SPAN: units of a run that one load of scale bytes
// covers.
constexpr int FEW_W = 8, SPAN = 4;
template <int XS, int XB, int NB> constexpr int few_lds() {
    constexpr int rows = (NB + (XS ? 0 : XB)) * 16;   // rows of codes that come from memory
    constexpr int wave = rows * 128 + rows * SPAN * 8 + (XS ? 16 * (128 + 8) : 0);
    constexpr int sums = NB * 16 * (XB * 16 + 1) * 4;
    return FEW_W * (wave > sums ? wave : sums);
}
struct FewArgs {
    const void *x;   // XS > 0
    int64_t ldx;
    const uint8_t *xc, *xs, *wc, *ws;
    const __bf16 *bias;
    __bf16 *y;
    int64_t M, N, K;
    int act;
};

template <class T, int XS, int XB, int NB, bool EVEN>
__global__ __launch_bounds__(FEW_W * 64) void mx4_few_kernel(FewArgs f) {
    static_assert(XS <= 8 && (XS == 0 || XB == 1), "rows of x");
    constexpr int MT = XB, CB = NB + (XS ? 0 : XB);             // CB: 16-row blocks of codes from memory
    constexpr int STAGE = CB * 8 + XS * 2 * (int)sizeof(T);   // registers of a unit in flight
    // one token leaves few waves' worth of work, so each asks for more ahead
    // (8192 x 8192: 8.0 us against 9.1 with 40 registers; 16 tokens, N = 28672:
    // 33 against 27)
    constexpr int REGS = XS == 1 ? 80 : 40;
    constexpr int DEPTH = REGS / STAGE > 4 ? 4 : REGS / STAGE > 1 ? REGS / STAGE : 1;
    __shared__ __align__(16) char lds[few_lds<XS, XB, NB>()];
    const int64_t M = f.M, N = f.N, K = f.K;
    const T *x = static_cast<const T *>(f.x);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    char *const wl = lds + wave * (few_lds<XS, XB, NB>() / FEW_W), *const sl = wl + CB * 16 * 128,
               *const xl = sl + CB * 16 * SPAN * 8,
               *const xsl = XS ? xl + 16 * 128 : sl + NB * 16 * SPAN * 8;
    const int64_t n0 = (int64_t)blockIdx.x * (NB * 16), kp = mx4_kp(K);
    const int units = (int)(kp / 256), last = (int)min(N - 1 - n0, (int64_t)NB * 16 - 1);
    const int begin = wave * units / FEW_W, end = (wave + 1) * units / FEW_W;
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(f.wc + n0 * (kp / 2)), sr = make_rsrc(f.ws + n0 * (kp / 32)),
                                 xr = make_rsrc(f.xc), xsr = make_rsrc(f.xs);
    uint32_t off[CB * 2];
#pragma unroll
    for (int i = 0; i < CB * 2; ++i) {   // rows past N (M) repeat the last, unused
        const int row = i * 8 + (lane >> 3);
        const int at = i < NB * 2 ? min(row, last) : (int)min((int64_t)(row - NB * 16), M - 1);
        off[i] = (uint32_t)(at * (kp / 2) + (lane & 7) * 16);
    }
    f32x4 acc[MT][NB];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mt][nb] = f32x4{0, 0, 0, 0};
    for (int at = begin; at < end; at += SPAN) {
        const int stop = min(at + SPAN, end);
        u32x4 w[DEPTH][CB * 2];
        Vec8<T> v[DEPTH][XS ? XS : 1];
        const auto load = [&](int d, int u) {
            const bool in = u < stop;
#pragma unroll
            for (int s = 0; s < XS; ++s) {
                const int64_t m = min((int64_t)(s * 2 + (lane >> 5)), M - 1);
                fetch_row<EVEN>(v[d][s], x + m * f.ldx, (int64_t)min(u, stop - 1) * 256 + (lane & 31) * 8, K);
            }
#pragma unroll
            for (int i = 0; i < CB * 2; ++i)
                w[d][i] = __builtin_amdgcn_raw_buffer_load_b128(i < NB * 2 ? wr : xr, in ? off[i] : OOB_OFFSET,
                                                                u * 128, 0);
        };
        // 8 SPAN scale bytes of each row, eight a lane
        constexpr int SL = CB * 16 * SPAN / 64;
        u32x2 scales[SL];
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            const int row = (i * 64 + lane) / SPAN, c = at * 8 + lane % SPAN * 8;
            const int64_t r_ = row < NB * 16 ? min(row, last) : min((int64_t)(row - NB * 16), M - 1);
            const uint32_t o = c < kp / 32 ? (uint32_t)(r_ * (kp / 32) + c) : OOB_OFFSET;
            const bool of_w = i * 64 / SPAN < NB * 16;   // 64 / SPAN rows a load, all of one operand
            scales[i] = __builtin_amdgcn_raw_buffer_load_b64(of_w ? sr : xsr, o, 0, 0);
        }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load(d, at + d);
#pragma unroll
        for (int i = 0; i < SL; ++i) *reinterpret_cast<u32x2 *>(sl + (i * 64 + lane) * 8) = scales[i];
        for (int u = at; u < stop; u += DEPTH)
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                // past the end zeros of W are multiplied: a branch would pull the loads into it
                const int now = min(u + d, stop - 1);
                const int64_t k = (int64_t)now * 256 + (lane & 31) * 8;
#pragma unroll
                for (int s = 0; s < XS; ++s) {
                    float q[8];
                    row_values<EVEN>(v[d][s], q, k, K);
                    uint32_t mx = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) mx = max(mx, abs_bits(q[j]));
                    const uint32_t byte = mx4_scale_byte(max_of_four(mx));
                    const int row = s * 2 + (lane >> 5);
                    *reinterpret_cast<uint32_t *>(xl + lds_off<8>(row, (lane & 31) >> 2) + (lane & 3) * 4) =
                        mx4_pack8(q, mx4_unscale(byte));
                    if ((lane & 3) == 0) xsl[row * 8 + ((lane & 31) >> 2)] = (char)byte;
                }
#pragma unroll
                for (int i = 0; i < CB * 2; ++i)
                    *reinterpret_cast<u32x4 *>(wl + lds_off<8>(i * 8 + (lane >> 3), lane & 7)) = w[d][i];
                const auto operand = [&](const char *p, int row, int half) {
                    const u32x4 q = *reinterpret_cast<const u32x4 *>(p + lds_off<8>(row, half * 4 + g));
                    return i32x8{(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0};
                };
                const auto scale = [&](const char *p) {
                    return (int)((uint32_t)(uint8_t)p[g] | (uint32_t)(uint8_t)p[4 + g] << 8);
                };
                i32x8 a[NB][2];
                int sa[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    a[nb][0] = operand(wl, nb * 16 + r, 0);
                    a[nb][1] = operand(wl, nb * 16 + r, 1);
                    sa[nb] = scale(sl + (nb * 16 + r) * (SPAN * 8) + (now - at) * 8);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    // from memory x's rows follow those of W, under the same swizzle
                    const char *const xb = XS ? xl : wl;
                    const int row = (XS ? 0 : NB * 16) + mt * 16 + r;
                    const i32x8 b0 = operand(xb, row, 0), b1 = operand(xb, row, 1);
                    const int sb = scale(XS ? xsl + r * 8 : xsl + (mt * 16 + r) * (SPAN * 8) + (now - at) * 8);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        acc[mt][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            a[nb][0], b0, acc[mt][nb], 4, 4, 0, sa[nb], 0, sb);
                        acc[mt][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            a[nb][1], b1, acc[mt][nb], 4, 4, 1, sa[nb], 1, sb);
                    }
                }
                load(d, u + d + DEPTH);
            }
    }
    __syncthreads();   // every wave is done with its LDS
    float(*part)[NB * 16][MT * 16 + 1] = reinterpret_cast<float(*)[NB * 16][MT * 16 + 1]>(lds);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[wave][nb * 16 + g * 4 + i][mt * 16 + r] = acc[mt][nb][i];
    __syncthreads();
    for (int i = threadIdx.x; i < NB * 16 * (int)M; i += FEW_W * 64) {
        const int n = i % (NB * 16), m = i / (NB * 16);
        if (n0 + n >= N) continue;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < FEW_W; ++k) s += part[k][n][m];
        if (f.bias) s += (float)f.bias[n0 + n];
        f.y[m * N + n0 + n] = (__bf16)apply_act(s, f.act);
    }
}

template <class T, int XS, int XB, bool EVEN>
hipError_t few(const FewArgs &f, hipStream_t st) {
    // Two blocks of W share a wave's x, where that leaves a workgroup for every CU
    // (four tokens, 8192 x 8192: 9.4 us against 21). With one or two tokens there
    // is little to share, and the form that takes fewer rounds of blocks over
    // the CUs is used (N = 28672, K = 8192: one block 23.8 us, two 26; N = 8192,
    // the same number of rounds: two 8.4 us, one 9.2).
    const int64_t ones = (f.N + 15) / 16, twos = (f.N + 31) / 32;
    const bool two = XS == 1 ? (twos + 255) / 256 * 2 <= (ones + 255) / 256 : f.N >= 256 * 32;
    const int64_t grid = two ? twos : ones;
    if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    if (two) mx4_few_kernel<T, XS, XB, 2, EVEN><<<(unsigned)grid, FEW_W * 64, 0, st>>>(f);
    else mx4_few_kernel<T, XS, XB, 1, EVEN><<<(unsigned)grid, FEW_W * 64, 0, st>>>(f);
    return hipGetLastError();
}
template <class T> hipError_t few(const FewArgs &f, hipStream_t st) {
    const bool even = f.K % 8 == 0;
    if (f.M <= 2) return even ? few<T, 1, 1, true>(f, st) : few<T, 1, 1, false>(f, st);
    return even ? few<T, 4, 1, true>(f, st) : few<T, 4, 1, false>(f, st);
}

}  // namespace

hipError_t launch_mx4_quantize(int type, const Mx4Quant &a, const Mx4Quant *b, hipStream_t st) {
    if (type == GEMM_F32) return quantize<float>(a, b, st);
    if (type == GEMM_F16) return quantize<_Float16>(a, b, st);
    return quantize<__bf16>(a, b, st);
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

hipError_t launch_mx4_few(const void *x, int type, int64_t ldx, const uint8_t *xc, const uint8_t *xs,
                          const uint8_t *wc, const uint8_t *ws, const void *bias, void *y, int64_t M,
                          int64_t N, int64_t K, int act, hipStream_t st) {
    const int64_t kp = mx4_kp(K);
    if (xc && M * (kp / 2) > NUM_RECORDS) {   // the last rows' codes would lie past a buffer's range
        const int64_t half = M / 2;
        const hipError_t e = launch_mx4_few(x, type, ldx, xc, xs, wc, ws, bias, y, half, N, K, act, st);
        if (e != hipSuccess) return e;
        return launch_mx4_few(x, type, ldx, xc + half * (kp / 2), xs + half * (kp / 32), wc, ws, bias,
                              static_cast<__bf16 *>(y) + half * N, M - half, N, K, act, st);
    }
    const FewArgs f = {x, ldx, xc, xs, wc, ws, static_cast<const __bf16 *>(bias), static_cast<__bf16 *>(y),
                       M, N, K, act};
    if (xc && M <= 16) return few<__bf16, 0, 1, true>(f, st);
    if (xc) return M <= 32 ? few<__bf16, 0, 2, true>(f, st) : few<__bf16, 0, 4, true>(f, st);
    if (type == GEMM_F32) return few<float>(f, st);
    if (type == GEMM_F16) return few<_Float16>(f, st);
    return few<__bf16>(f, st);
}

}  // namespace mg
