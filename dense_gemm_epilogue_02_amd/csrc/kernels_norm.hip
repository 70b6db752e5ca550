// kernels_norm.hip -- the norms before and after a block, fused with its gate
// and residual scale, and their gradients.
#include "block.hpp"

namespace mg {

namespace {

// Sum over the lanes of a wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Sum over the WPR waves that share a row. The slots alternate between calls
// (`turn`), so one barrier per sum is enough: a slot is written again only
// after the barrier of the call between.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float (*slot)[WPR], int &turn) {
    v = wave_sum(v);
    if constexpr (WPR > 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) slot[turn][wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) v += slot[turn][w];
        turn ^= 1;
    }
    return v;
}

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + __expf(-v)); }

// ---- forward --------------------------------------------------------------------
//
//   y = b rstd(b) w_post,  out = residual + scale act(gate) y,
//   next = out rstd(out) w_next
// Bound by memory: two reads and two writes of [rows][cols]. WPR waves hold a
// row in registers from its first load to its last store (VPT groups of eight
// elements a thread), so nothing is read twice and the two row sums cost one
// barrier each.
template <class T, int WPR, int VPT>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void norm_forward_kernel(gemm_norm_args a) {
    constexpr int RPB = WPR == 1 ? 4 : 1, NT = WPR * 64;
    __shared__ float slot[2][WPR];
    int turn = 0;
    const int t = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * RPB + (WPR == 1 ? threadIdx.x >> 6 : 0);
    if (row >= a.rows) return;   // whole waves; no barrier where a row is one wave's
    const int64_t H = a.cols;
    const float inv = 1.0f / (float)H;
    float r[VPT][8];
    const T *res = static_cast<const T *>(a.residual) + row * a.ld_residual;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t c = ((int64_t)v * NT + t) * 8;
        Vec8<T> x;
        x.load(res + (c < H ? c : 0), H - c);
        x.get(r[v]);
    }
    if (a.block) {
        const T *blk = static_cast<const T *>(a.block) + row * a.ld_block;
        float b[VPT][8];
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t c = ((int64_t)v * NT + t) * 8;
            Vec8<T> x;
            x.load(blk + (c < H ? c : 0), H - c);
            x.get(b[v]);
#pragma unroll
            for (int j = 0; j < 8; ++j) s += b[v][j] * b[v][j];
        }
        float rb = 1.0f;
        if (a.w_post) {
            rb = rsqrtf(row_sum<WPR>(s, slot, turn) * inv + a.eps);
            if (a.rstd_post && t == 0) a.rstd_post[row] = rb;
        }
        const T *gate = a.gate ? static_cast<const T *>(a.gate) +
                                     row / (a.rows / a.gate_rows) * a.ld_gate
                               : nullptr;
        T *out = static_cast<T *>(a.out) + row * a.ld_out;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t c = ((int64_t)v * NT + t) * 8, at = c < H ? c : 0;
            float f[8];
            Vec8<T> x;
#pragma unroll
            for (int j = 0; j < 8; ++j) b[v][j] *= rb;
            if (a.w_post) {
                x.load(static_cast<const T *>(a.w_post) + at, H - c);
                x.get(f);
#pragma unroll
                for (int j = 0; j < 8; ++j) b[v][j] *= f[j];
            }
            if (a.scale) {
                x.load(static_cast<const T *>(a.scale) + at, H - c);
                x.get(f);
#pragma unroll
                for (int j = 0; j < 8; ++j) b[v][j] *= f[j];
            }
            if (gate) {
                x.load(gate + at, H - c);
                x.get(f);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    b[v][j] *= a.gate_act == GEMM_EPI_SIGMOID ? sigmoid(f[j]) : f[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) r[v][j] += b[v][j];
            x.set(r[v]);   // the next norm reads what is stored, as the backward pass does
            x.get(r[v]);
            if (c < H) x.store(out + c, H - c);
        }
    }
    if (!a.w_next) return;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s += ((int64_t)v * NT + t) * 8 + j < H ? r[v][j] * r[v][j] : 0.0f;
    const float rr = rsqrtf(row_sum<WPR>(s, slot, turn) * inv + a.eps);
    if (a.rstd_next && t == 0) a.rstd_next[row] = rr;
    T *next = static_cast<T *>(a.next) + row * a.ld_next;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t c = ((int64_t)v * NT + t) * 8;
        if (c < H) {
            float f[8];
            Vec8<T> x;
            x.load(static_cast<const T *>(a.w_next) + c, H - c);
            x.get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= r[v][j] * rr;
            x.set(f);
            x.store(next + c, H - c);
        }
    }
}

// ---- backward --------------------------------------------------------------------
//
// With xn = out rstd_next, xb = block rstd_post, act the gate's value:
//   g  = d_next w_next,  d = d_out + rstd_next (g - xn mean(g xn))  (d_residual)
//   y  = xb w_post,  dy = d scale act
//   d_block = rstd_post (dy w_post - xb mean(dy w_post xb))
//   column sums: d_w_next += d_next xn, d_scale += d act y, d_w_post += dy xb,
//                d_gate += d scale y act'
// Bound by memory: four reads and two writes of [rows][cols]. A workgroup walks
// the rows of its part with a fixed set of columns per thread and keeps the
// column sums in registers; the parts' sums are added by norm_columns_kernel in
// part order, so no result depends on the order of execution.
struct ColumnSums {
    float *part;        // [parts][3][cols]: d_w_post, d_scale, d_w_next
    float *gate_part;   // [parts][cols], where a group is cut into chunks
    NormCut cut;
};

template <class T, int WPR, int VPT>
__global__ __launch_bounds__(WPR * 64) void norm_backward_kernel(gemm_norm_backward_args a,
                                                                 ColumnSums cs) {
    constexpr int NT = WPR * 64;
    __shared__ float slot[2][WPR];
    int turn = 0;
    const int t = threadIdx.x;
    const int64_t H = a.cols, part = blockIdx.x;
    const NormCut cut = cs.cut;
    int64_t row, end;
    if (cut.chunks > 1) {
        const int64_t group = part / cut.chunks, chunk = part - group * cut.chunks;
        row = group * cut.rows_per_group + chunk * cut.rows_per_part;
        end = min(row + cut.rows_per_part, (group + 1) * cut.rows_per_group);
    } else {
        row = part * cut.groups_per_part * cut.rows_per_group;
        end = min(row + cut.groups_per_part * cut.rows_per_group, a.rows);
    }
    const float inv = 1.0f / (float)H;
    float s_post[VPT][8] = {}, s_scale[VPT][8] = {}, s_next[VPT][8] = {}, s_gate[VPT][8] = {};
    const bool sig = a.gate_act == GEMM_EPI_SIGMOID;
    for (; row < end; ++row) {
        const float rr = a.w_next ? a.rstd_next[row] : 0.0f;
        const float rb = a.w_post ? a.rstd_post[row] : 1.0f;
        float d[VPT][8], xn[VPT][8], g[VPT][8], xb[VPT][8];
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t c = ((int64_t)v * NT + t) * 8, at = c < H ? c : 0;
            Vec8<T> x;
#pragma unroll
            for (int j = 0; j < 8; ++j) d[v][j] = g[v][j] = xn[v][j] = xb[v][j] = 0.0f;
            if (a.d_out) {
                x.load(static_cast<const T *>(a.d_out) + row * a.ld_d_out + at, H - c);
                x.get(d[v]);
            }
            if (a.block) {
                x.load(static_cast<const T *>(a.block) + row * a.ld_block + at, H - c);
                x.get(xb[v]);
            }
            if (a.d_next) {
                float w[8];
                x.load(static_cast<const T *>(a.out) + row * a.ld_out + at, H - c);
                x.get(xn[v]);
                x.load(static_cast<const T *>(a.d_next) + row * a.ld_d_next + at, H - c);
                x.get(g[v]);
                x.load(static_cast<const T *>(a.w_next) + at, H - c);
                x.get(w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    xn[v][j] *= rr;
                    s_next[v][j] += g[v][j] * xn[v][j];
                    g[v][j] *= w[j];
                    s += g[v][j] * xn[v][j];
                }
            }
        }
        if (a.d_next) {
            const float mean = row_sum<WPR>(s, slot, turn) * inv;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) d[v][j] += rr * (g[v][j] - xn[v][j] * mean);
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t c = ((int64_t)v * NT + t) * 8;
            Vec8<T> x;
            x.set(d[v]);
            if (c < H)
                x.store(static_cast<T *>(a.d_residual) + row * a.ld_d_residual + c, H - c);
        }
        if (!a.block) continue;
        const int64_t group = row / cut.rows_per_group;
        const T *gate = a.gate ? static_cast<const T *>(a.gate) + group * a.ld_gate : nullptr;
        s = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t c = ((int64_t)v * NT + t) * 8, at = c < H ? c : 0;
            float wp[8], sc[8], ga[8];
            Vec8<T> x;
#pragma unroll
            for (int j = 0; j < 8; ++j) wp[j] = sc[j] = ga[j] = 1.0f;
            if (a.w_post) {
                x.load(static_cast<const T *>(a.w_post) + at, H - c);
                x.get(wp);
            }
            if (a.scale) {
                x.load(static_cast<const T *>(a.scale) + at, H - c);
                x.get(sc);
            }
            if (gate) {
                x.load(gate + at, H - c);
                x.get(ga);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float slope = 1.0f;
                if (gate && sig) {
                    ga[j] = sigmoid(ga[j]);
                    slope = ga[j] * (1.0f - ga[j]);
                }
                xb[v][j] *= rb;
                const float y = xb[v][j] * wp[j], dv = d[v][j];
                s_gate[v][j] += dv * sc[j] * y * slope;
                s_scale[v][j] += dv * ga[j] * y;
                const float dy = dv * sc[j] * ga[j];
                s_post[v][j] += dy * xb[v][j];
                g[v][j] = dy * wp[j];   // d block, but for the norm's second term
                s += g[v][j] * xb[v][j];
            }
        }
        if (a.w_post) {
            const float mean = row_sum<WPR>(s, slot, turn) * inv;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) g[v][j] = rb * (g[v][j] - xb[v][j] * mean);
        }
        const bool last_of_group = row + 1 == (group + 1) * cut.rows_per_group;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t c = ((int64_t)v * NT + t) * 8;
            Vec8<T> x;
            x.set(g[v]);
            if (c < H) x.store(static_cast<T *>(a.d_block) + row * a.ld_d_block + c, H - c);
            if (a.d_gate && cut.chunks == 1 && last_of_group) {
                x.set(s_gate[v]);
                if (c < H) x.store(static_cast<T *>(a.d_gate) + group * H + c, H - c);
#pragma unroll
                for (int j = 0; j < 8; ++j) s_gate[v][j] = 0.0f;
            }
        }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t c = ((int64_t)v * NT + t) * 8;
        if (c >= H) continue;
        float *p = cs.part + part * 3 * H + c;
        Vec8<float> x;
        if (a.d_w_post) {
            x.set(s_post[v]);
            x.store(p, H - c);
        }
        if (a.d_scale) {
            x.set(s_scale[v]);
            x.store(p + H, H - c);
        }
        if (a.d_w_next) {
            x.set(s_next[v]);
            x.store(p + 2 * H, H - c);
        }
        if (a.d_gate && cut.chunks > 1) {
            x.set(s_gate[v]);
            x.store(cs.gate_part + part * H + c, H - c);
        }
    }
}

// out[c] = sum over n rows, `stride` apart, of the column partials, in row
// order within each of 16 interleaved strands and then in strand order. One
// workgroup per 64 columns of one output vector.
template <class T>
__global__ __launch_bounds__(1024) void norm_columns_kernel(gemm_norm_backward_args a, ColumnSums cs) {
    __shared__ float sum[16][64];
    const int64_t H = a.cols, blocks = (H + 63) / 64, job = blockIdx.x / blocks;
    const int lane = threadIdx.x & 63, strand = threadIdx.x >> 6;
    const int64_t c = (blockIdx.x - job * blocks) * 64 + lane;
    const float *src;
    int64_t n, stride;
    T *dst;
    if (job < 3) {
        dst = static_cast<T *>(job == 0 ? a.d_w_post : job == 1 ? a.d_scale : a.d_w_next);
        if (!dst) return;
        src = cs.part + job * H;
        n = cs.cut.parts;
        stride = 3 * H;
    } else {
        dst = static_cast<T *>(a.d_gate) + (job - 3) * H;
        src = cs.gate_part + (job - 3) * cs.cut.chunks * H;
        n = cs.cut.chunks;
        stride = H;
    }
    float s = 0.0f;
    if (c < H)
        for (int64_t i = strand; i < n; i += 16) s += src[i * stride + c];
    sum[strand][lane] = s;
    __syncthreads();
    if (strand == 0 && c < H) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += sum[i][lane];
        dst[c] = from_f<T>(s);
    }
}

template <class T>
hipError_t forward(const gemm_norm_args &a, hipStream_t st) {
    const unsigned rows = (unsigned)a.rows, by4 = (unsigned)((a.rows + 3) / 4);
    if (a.cols <= 512) norm_forward_kernel<T, 1, 1><<<by4, 256, 0, st>>>(a);
    else if (a.cols <= 1024) norm_forward_kernel<T, 1, 2><<<by4, 256, 0, st>>>(a);
    else if (a.cols <= 2048) norm_forward_kernel<T, 4, 1><<<rows, 256, 0, st>>>(a);
    else if (a.cols <= 4096) norm_forward_kernel<T, 4, 2><<<rows, 256, 0, st>>>(a);
    else if (a.cols <= 8192) norm_forward_kernel<T, 16, 1><<<rows, 1024, 0, st>>>(a);
    else norm_forward_kernel<T, 16, 2><<<rows, 1024, 0, st>>>(a);
    return hipGetLastError();
}

template <class T>
hipError_t backward(const gemm_norm_backward_args &a, hipStream_t st) {
    ColumnSums cs;
    cs.cut = norm_cut(a.rows, a.cols, a.gate ? a.gate_rows : 1);
    cs.part = static_cast<float *>(a.workspace);
    cs.gate_part = cs.part + cs.cut.parts * 3 * a.cols;
    const unsigned parts = (unsigned)cs.cut.parts;
    if (parts > 0) {
        if (a.cols <= 512) norm_backward_kernel<T, 1, 1><<<parts, 64, 0, st>>>(a, cs);
        else if (a.cols <= 1024) norm_backward_kernel<T, 2, 1><<<parts, 128, 0, st>>>(a, cs);
        else if (a.cols <= 2048) norm_backward_kernel<T, 4, 1><<<parts, 256, 0, st>>>(a, cs);
        else if (a.cols <= 4096) norm_backward_kernel<T, 8, 1><<<parts, 512, 0, st>>>(a, cs);
        else if (a.cols <= 8192) norm_backward_kernel<T, 16, 1><<<parts, 1024, 0, st>>>(a, cs);
        else norm_backward_kernel<T, 16, 2><<<parts, 1024, 0, st>>>(a, cs);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t gates = a.d_gate && cs.cut.chunks != 1 ? a.gate_rows : 0;
    if (!a.d_w_post && !a.d_scale && !a.d_w_next && gates == 0) return hipSuccess;
    const int64_t grid = (3 + gates) * ((a.cols + 63) / 64);
    norm_columns_kernel<T><<<(unsigned)grid, 1024, 0, st>>>(a, cs);
    return hipGetLastError();
}

}  // namespace

NormCut norm_cut(int64_t rows, int64_t cols, int64_t gate_rows) {
    NormCut c;
    c.rows_per_group = rows > 0 ? rows / (gate_rows > 0 ? gate_rows : 1) : 0;
    if (rows == 0) {
        c.parts = 0;
        c.rows_per_part = 0;
        c.chunks = 0;   // every sum is over nothing
        c.groups_per_part = 1;
        return c;
    }
    const int64_t most = cols > 4096 ? 256 : cols > 2048 ? 512 : 1024;
    int64_t R = (rows + most - 1) / most;
    if (c.rows_per_group > R) {
        c.rows_per_part = R;
        c.chunks = (c.rows_per_group + R - 1) / R;
        c.groups_per_part = 1;
        c.parts = gate_rows * c.chunks;
    } else {
        c.chunks = 1;
        c.groups_per_part = R / c.rows_per_group;
        c.rows_per_part = c.groups_per_part * c.rows_per_group;
        c.parts = (gate_rows + c.groups_per_part - 1) / c.groups_per_part;
    }
    return c;
}

hipError_t launch_norm_forward(const gemm_norm_args &a, hipStream_t st) {
    if (a.type == GEMM_F32) return forward<float>(a, st);
    if (a.type == GEMM_F16) return forward<_Float16>(a, st);
    return forward<__bf16>(a, st);
}

hipError_t launch_norm_backward(const gemm_norm_backward_args &a, hipStream_t st) {
    if (a.type == GEMM_F32) return backward<float>(a, st);
    if (a.type == GEMM_F16) return backward<_Float16>(a, st);
    return backward<__bf16>(a, st);
}

}  // namespace mg
