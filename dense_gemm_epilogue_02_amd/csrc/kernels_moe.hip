// kernels_moe.hip -- a mixture-of-experts layer for a few tokens.
//
// Bound by the one read of every chosen expert's weights. Three launches:
// the router (logits and the choice), the gate and up products with their
// activation, and the down product with the weighted sum over a token's
// experts. A slot is one choice of one token (token * k + rank); everything
// that belongs to it is stored under that number, so nothing is permuted.
#include "block.hpp"

namespace mg {

namespace {

constexpr int RT = 4;           // tokens per router workgroup
constexpr int ROUTER_W = 8;     // its waves
constexpr int ST_STRIDE = 32;   // words between the router's counters, one cache line each
constexpr int CHUNKS = (GEMM_MOE_MAX_TOKENS + RT - 1) / RT;

struct Active {
    int expert, first, count, pad;   // its slots are slots[first .. first + count)
};

struct Ws {
    unsigned *chunk_state;    // [ST_STRIDE * chunk] router arrivals, then those of the chunks
    unsigned *column_state;   // [H / 16] arrivals at a column block's expert groups
    double *logits;           // [T][E]
    int *ids;                 // [T][k]
    float *probs;             // [T][k]
    int *slots;               // the routed slots, ordered by expert
    int *n_active;            // then the list of the experts that have any
    Active *active;
    char *h;                  // the activations: [T * k][3][ip] in bf16, or [T * k][ip] in fp32
    uint32_t *peak;           // [T * k] largest of a slot's activations that pass 2^15 (fp32 bits), else 0
    float *y;                 // [column block][T * k][ROWS] products of the down matrices
    int64_t ip;
};

__host__ __device__ inline Ws moe_ws(char *p, const MoeLayout &l) {
    Ws w;
    w.chunk_state = reinterpret_cast<unsigned *>(p);
    w.column_state = reinterpret_cast<unsigned *>(p + l.columns);
    w.logits = reinterpret_cast<double *>(p + l.logits);
    w.ids = reinterpret_cast<int *>(p + l.ids);
    w.probs = reinterpret_cast<float *>(p + l.probs);
    w.slots = reinterpret_cast<int *>(p + l.slots);
    w.n_active = reinterpret_cast<int *>(p + l.active);
    w.active = reinterpret_cast<Active *>(p + l.active + 16);
    w.h = p + l.h;
    w.peak = reinterpret_cast<uint32_t *>(p + l.peak);
    w.y = reinterpret_cast<float *>(p + l.y);
    w.ip = l.ip;
    return w;
}

// True in the workgroup that arrives last of n; the counter is left zero and
// nobody waits. What the others wrote with device-scope stores before their
// arrival (the barrier drains them) is seen by its device-scope loads, so no
// cache is written back or invalidated: a __threadfence() here instead cost
// the router 12 us of 19 for one token, 36 of 43 for 64.
__device__ __forceinline__ bool last_of(unsigned *counter, unsigned n, int *flag) {
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): this wave's stores have arrived
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned old =
            __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *flag = old == n - 1;
        if (old == n - 1)
            __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    return *flag != 0;
}
template <class T> __device__ __forceinline__ void put(T *p, T v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T> __device__ __forceinline__ T got(const T *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ double shfl_xor_d(double v, int o) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __shfl_xor((int)(uint32_t)b, o), hi = __shfl_xor((int)(b >> 32), o);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ int64_t shfl_xor_l(int64_t v, int o) {
    const uint32_t lo = __shfl_xor((int)(uint32_t)v, o), hi = __shfl_xor((int)(v >> 32), o);
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// An integer that orders like the number; NaN below every number, both zeros alike.
__device__ __forceinline__ int64_t order_key(double v) {
    if (v != v) return INT64_MIN;
    const int64_t b = __builtin_bit_cast(int64_t, v + 0.0);
    return b < 0 ? (b ^ INT64_MAX) : b;
}

// ---- router ---------------------------------------------------------------------
//
// l[t][e] = sum_h x[t][h] router[e][h] in 64 bits: products of 16-bit values
// are exact there and the sum's order no longer decides between experts that
// are close. `split` waves share h for one expert and RT tokens; the workgroup
// that completes a chunk of tokens chooses for it, a wave per token, and the
// one that completes the last chunk lists the experts that have tokens.

// A wave's lanes hold the logits of experts i * 64 + lane of one token.
// rank: how many experts come before each (larger, or equal with a lower
// index), by comparing every pair; 4 instructions an expert and held value,
// where finding one maximum after the other waits for 18 lane exchanges each.
template <int PER>
__device__ __forceinline__ void rank_all(const int64_t (&key)[PER], int E, int (&rank)[PER]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < PER; ++i) rank[i] = 0;
#pragma unroll
    for (int b = 0; b < PER; ++b) {
        const int n = min(64, E - b * 64);
        const uint32_t lo = (uint32_t)key[b], hi = (uint32_t)(key[b] >> 32);
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            const int64_t o = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)hi, j) << 32 |
                                        (uint32_t)__builtin_amdgcn_readlane((int)lo, j));
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const bool earlier = b < i || (b == i && j < lane);
                rank[i] += earlier ? o >= key[i] : o > key[i];
            }
        }
    }
}

// The same for many experts, where all pairs are too many: the k largest, one
// maximum after the other; rank stays INT32_MAX for the others.
template <int PER>
__device__ __forceinline__ void rank_largest(const int64_t (&key)[PER], int E, int k, int (&rank)[PER]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < PER; ++i) rank[i] = INT32_MAX;
    for (int j = 0; j < k; ++j) {
        int64_t best = INT64_MIN;
        int at = INT32_MAX;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int x = i * 64 + lane;
            if (x < E && rank[i] == INT32_MAX && (at == INT32_MAX || key[i] > best)) {
                best = key[i];
                at = x;
            }
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const int64_t ob = shfl_xor_l(best, o);
            const int oa = __shfl_xor(at, o);
            if (oa != INT32_MAX && (at == INT32_MAX || ob > best || (ob == best && oa < at))) {
                best = ob;
                at = oa;
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (at == i * 64 + lane) rank[i] = j;
    }
}

template <int PER, bool ONE>
__device__ __forceinline__ void choose(const MoeArgs &a, const Ws &w, int t, int *ids) {
    const int lane = threadIdx.x & 63;
    const bool live = !a.mask || a.mask[t] != 0;
    double l[PER];
    int64_t key[PER];
    int rank[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int x = i * 64 + lane;
        l[i] = x < a.E ? got(w.logits + (int64_t)t * a.E + x) : 0.0;
        key[i] = x < a.E ? order_key(l[i]) : INT64_MIN;
    }
    if constexpr (PER <= 2) rank_all<PER>(key, a.E, rank);
    else rank_largest<PER>(key, a.E, a.k, rank);
    double top = 0.0, sum = 0.0, p[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint64_t first = __ballot(i * 64 + lane < a.E && rank[i] == 0);
        if (first != 0) {
            const uint64_t v = __builtin_bit_cast(uint64_t, l[i]);
            const int from = __builtin_ctzll(first);
            const uint32_t lo = __shfl((int)(uint32_t)v, from), hi = __shfl((int)(v >> 32), from);
            top = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int x = i * 64 + lane;
        p[i] = x < a.E && (!a.renorm || rank[i] < a.k) ? exp(l[i] - top) : 0.0;
        sum += p[i];
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += shfl_xor_d(sum, o);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int x = i * 64 + lane;
        if (x >= a.E || rank[i] >= a.k) continue;
        const int slot = t * a.k + rank[i];
        const int id = live ? x : -1;
        const float v = live ? (float)(p[i] / sum) : 0.0f;
        if constexpr (ONE) {   // each choice is an active expert of one slot
            w.ids[slot] = id;
            w.slots[slot] = slot;
            w.active[slot] = Active{x, slot, 1, 0};
        } else {
            put(w.ids + slot, id);
            ids[rank[i]] = id;
        }
        w.probs[slot] = v;
        w.peak[slot] = 0u;
        if (a.ids) a.ids[slot] = id;
        if (a.probs) a.probs[slot] = v;
    }
}

// The sums over the wave's lanes of R values: value i in the lanes i * 64 / R on.
template <int R> __device__ __forceinline__ double sum_over_lanes(const double (&v)[R]) {
    static_assert(R == 1 || R == 4, "values");
    const int lane = threadIdx.x & 63;
    double s = v[0];
    if constexpr (R == 4) {
        const bool high = lane & 32, odd = lane & 16;
        const double a = (high ? v[2] : v[0]) + shfl_xor_d(high ? v[0] : v[2], 32),
                     b = (high ? v[3] : v[1]) + shfl_xor_d(high ? v[1] : v[3], 32);
        s = (odd ? b : a) + shfl_xor_d(odd ? a : b, 16);
    } else {
        s += shfl_xor_d(s, 32);
        s += shfl_xor_d(s, 16);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += shfl_xor_d(s, o);
    return s;
}

// NT: tokens of a workgroup, 1 or RT.
template <class T, int NT>
__global__ __launch_bounds__(ROUTER_W * 64) void moe_router_kernel(MoeArgs a, MoeLayout lay, int split) {
    constexpr int BATCH = 2;   // loads in flight, times 512 h
    __shared__ int flag;
    __shared__ double sums[ROUTER_W][NT];
    __shared__ int place[GEMM_MOE_MAX_EXPERTS], chosen[NT][GEMM_MOE_MAX_TOP_K];
    const Ws w = moe_ws(a.ws, lay);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, per = ROUTER_W / split;
    const int e0 = blockIdx.x * per, t0 = blockIdx.y * NT, nt = min(NT, a.T - t0);
    const T *rp = static_cast<const T *>(a.router) + (int64_t)min(e0 + wave / split, a.E - 1) * a.H;
    const T *xp[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) xp[i] = static_cast<const T *>(a.x) + (int64_t)min(t0 + i, a.T - 1) * a.ldx;
    double acc[NT] = {};
    for (int64_t h = (wave % split) * 512 + lane * 8; h - lane * 8 < a.H; h += BATCH * split * 512) {
        Vec8<T> r[BATCH], x[BATCH][NT];
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            const int64_t c = h + q * split * 512;
            fetch_row<false>(r[q], rp, c, a.H);
#pragma unroll
            for (int i = 0; i < NT; ++i) fetch_row<false>(x[q][i], xp[i], c, a.H);
        }
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            const int64_t c = h + q * split * 512;
            float f[8], g[8];
            row_values<false>(r[q], f, c, a.H);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                row_values<false>(x[q][i], g, c, a.H);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i] = __builtin_fma((double)f[j], (double)g[j], acc[i]);
            }
        }
    }
    const double sum = sum_over_lanes(acc);
    if (lane % (64 / NT) == 0) sums[wave][lane / (64 / NT)] = sum;
    __syncthreads();
    if ((int)threadIdx.x < per * nt) {
        const int i = threadIdx.x % nt, e = threadIdx.x / nt;
        double v = 0.0;
        for (int q = 0; q < split; ++q) v += sums[e * split + q][i];
        if (e0 + e < a.E) put(w.logits + (int64_t)(t0 + i) * a.E + e0 + e, v);
    }
    if (!last_of(w.chunk_state + blockIdx.y * ST_STRIDE, gridDim.x, &flag)) return;
    if (wave < nt) {
        int *const ids = chosen[wave];
        if (a.E <= 64) choose<1, NT == 1>(a, w, t0 + wave, ids);
        else if (a.E <= 128) choose<2, NT == 1>(a, w, t0 + wave, ids);
        else choose<GEMM_MOE_MAX_EXPERTS / 64, NT == 1>(a, w, t0 + wave, ids);
    }
    if constexpr (NT == 1) {
        if (threadIdx.x == 0) *w.n_active = a.mask && a.mask[0] == 0 ? 0 : a.k;
        return;
    }
    if (gridDim.y > 1) {
        if (!last_of(w.chunk_state + CHUNKS * ST_STRIDE, gridDim.y, &flag)) return;
    } else {
        __syncthreads();
    }

    // The order within an expert is that of the atomics and changes no result:
    // a slot's products do not depend on its place.
    for (int i = threadIdx.x; i < a.E; i += ROUTER_W * 64) place[i] = 0;
    __syncthreads();
    const int n = a.T * a.k;
    int mine[GEMM_MOE_MAX_TOKENS * GEMM_MOE_MAX_TOP_K / (ROUTER_W * 64)];
#pragma unroll
    for (int q = 0; q < (int)(sizeof(mine) / sizeof(mine[0])); ++q) {
        const int i = q * ROUTER_W * 64 + threadIdx.x;
        mine[q] = i >= n ? -1 : gridDim.y > 1 ? got(w.ids + i) : chosen[i / a.k][i % a.k];
        if (mine[q] >= 0) atomicAdd(&place[mine[q]], 1);
    }
    __syncthreads();
    if (wave == 0) {
        int base = 0, actives = 0;
        for (int b = 0; b < a.E; b += 64) {
            const int x = b + lane, c = x < a.E ? place[x] : 0;
            int run = c;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int r = __shfl_up(run, o);
                if (lane >= o) run += r;
            }
            const uint64_t some = __ballot(c > 0);
            const int at = actives + (int)__popcll(some & ((1ull << lane) - 1));
            if (x < a.E) place[x] = base + run - c;
            if (c > 0) w.active[at] = Active{x, base + run - c, c, 0};
            base += __builtin_amdgcn_readlane(run, 63);
            actives += (int)__popcll(some);
        }
        if (lane == 0) *w.n_active = actives;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < (int)(sizeof(mine) / sizeof(mine[0])); ++q)
        if (mine[q] >= 0) w.slots[atomicAdd(&place[mine[q]], 1)] = q * ROUTER_W * 64 + threadIdx.x;
}

// ---- the products ------------------------------------------------------------------
//
// v_mfma 16x16x32 with 16 weight rows as operand A and 16 tokens as operand B:
// a lane (r, g) supplies 8 k of weight row r and of token r, and ends with four
// consecutive rows of one token. In that layout sixteen neighbouring lanes
// touch sixteen rows, and loads straight into it were bound by the L1's line
// lookups (80 % busy, at 3.5 TB/s of MXFP4 weights). So a wave loads whole
// lines, 8 lanes to 128 bytes of a row (4 to 64 of MXFP4), several units ahead
// into registers, and turns a unit through a piece of LDS of its own: a wave's
// LDS instructions run in order, so no barrier is needed. Tokens go the same
// way.
template <class T> __device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c);
template <> __device__ __forceinline__ f32x4 mma16<__bf16>(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <> __device__ __forceinline__ f32x4 mma16<_Float16>(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Byte offset of 16-byte chunk `c` of row `r` in an LDS array of rows of N
// chunks, spread over the banks for reads of one chunk of 16 rows.
template <int N> __device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    if constexpr (N == 16) return (uint32_t)(r * 256 + ((c ^ (r & 15)) << 4));
    else return lds_off<N>(r, c);
}

// Weights and tokens are read with buffer loads: a load past the end of K is
// given an offset out of the buffer's range, so the hardware drops it and
// returns zeros, and no branch stands between the loads (the compiler moves
// loads into the branch that uses them, and waits for them there).
__device__ __forceinline__ u32x4 load_chunk(__amdgpu_buffer_rsrc_t rs, uint32_t off, int soff, bool in) {
    return __builtin_amdgcn_raw_buffer_load_b128(rs, in ? off : OOB_OFFSET, soff, 0);
}
// Eight elements from k = c on of a row's last n, zeros after them.
template <class T> __device__ __forceinline__ u32x4 end_chunk(const T *row, int c, int n) {
    T t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const T v = row[min(c + e, n - 1)];
        t[e] = c + e < n ? v : (T)0.0f;
    }
    return __builtin_bit_cast(u32x4, t);
}

// Sixteen rows of 16-bit weights.
template <class T> struct Rows16 {
    static constexpr int UK = 64, NF = 2;   // k of a unit; its fragments
    static constexpr int WI = 2;            // loads of a unit: 8 rows x 8 chunks each
    static constexpr int XC = 8;            // chunks of a token's unit
    static constexpr int LDS = 16 * 128;    // bytes of a unit
    static constexpr int SCALES = 0;
    static constexpr bool PADDED = false;   // rows end with K
    static constexpr bool WIDE_UP = false;  // 32 rows of each matrix a wave in the up product
    static __device__ __forceinline__ int chunk_of(int j, int g) { return j * 4 + g; }
    using Unit = u32x4[WI];
    const T *base;
    uint32_t off[WI];
    // rows row0 .. row0 + last exist, later ones repeat the last
    __device__ __forceinline__ void at(const void *p, const uint8_t *, int64_t row0, int last, int64_t K) {
        const int lane = threadIdx.x & 63;
        base = static_cast<const T *>(p) + row0 * K;
#pragma unroll
        for (int i = 0; i < WI; ++i)
            off[i] = (uint32_t)(min(i * 8 + (lane >> 3), last) * (int)K * 2 + (lane & 7) * 16);
    }
    // in: the lane's chunk exists
    __device__ __forceinline__ void load(Unit &t, int u, bool in) const {
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(base);
#pragma unroll
        for (int i = 0; i < WI; ++i) t[i] = load_chunk(rs, off[i], u * (UK * 2), in);
    }
    // the unit that K ends in, n of whose k exist
    __device__ __forceinline__ void load_end(Unit &t, int u, int n) const {
        const int c = (threadIdx.x & 7) * 8;
#pragma unroll
        for (int i = 0; i < WI; ++i) t[i] = end_chunk(base + (off[i] >> 1) - c + (int64_t)u * UK, c, n);
    }
    static __device__ __forceinline__ void store(char *lds, const Unit &t) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < WI; ++i)
            *reinterpret_cast<u32x4 *>(lds + chunk_at<8>(i * 8 + (lane >> 3), lane & 7)) = t[i];
    }
    struct Frags {
        u32x4 f[NF];
        __device__ __forceinline__ void read(const char *lds, const char *, int, int r, int g) {
#pragma unroll
            for (int j = 0; j < NF; ++j)
                f[j] = *reinterpret_cast<const u32x4 *>(lds + chunk_at<8>(r, chunk_of(j, g)));
        }
        __device__ __forceinline__ u32x4 get(int j) const { return f[j]; }
    };
    struct Scales {};
    __device__ __forceinline__ void load_scales(Scales &, int) const {}
    static __device__ __forceinline__ void store_scales(char *, const Scales &) {}
};

// Sixteen rows of MXFP4 weights (their padding holds zeros, so no load is cut).
// An element times its block's scale is exact in bf16.
struct Rows4 {
    static constexpr int UK = 128, NF = 4;
    static constexpr int WI = 1;      // 16 rows x 4 chunks
    static constexpr int XC = 16;
    static constexpr int LDS = 16 * 64;
    static constexpr int SCALES = 16 * 64;   // scale bytes of SPAN units of 16 rows
    static constexpr int SPAN = 16;
    static constexpr bool PADDED = true;
    static constexpr bool WIDE_UP = true;   // a token's unit is four times a weight row's bytes
    static __device__ __forceinline__ int chunk_of(int j, int g) { return g * 4 + j; }
    using Unit = u32x4[WI];
    const uint8_t *base, *scales;
    uint32_t off, soff;
    int ks;   // scale bytes of a row
    __device__ __forceinline__ void at(const void *p, const uint8_t *s, int64_t row0, int last, int64_t K) {
        const int lane = threadIdx.x & 63, row = min(lane >> 2, last);
        const int64_t kp = mx4_kp(K);
        base = static_cast<const uint8_t *>(p) + row0 * (kp / 2);
        scales = s + row0 * (kp / 32);
        ks = (int)(kp / 32);
        off = (uint32_t)(row * (int)(kp / 2) + (lane & 3) * 16);
        soff = (uint32_t)(row * ks);
    }
    __device__ __forceinline__ void load(Unit &t, int u, bool in) const {
        t[0] = load_chunk(make_rsrc(base), off, u * 64, in);
    }
    __device__ __forceinline__ void load_end(Unit &t, int u, int) const { load(t, u, true); }
    static __device__ __forceinline__ void store(char *lds, const Unit &t) {
        const int lane = threadIdx.x & 63;
        *reinterpret_cast<u32x4 *>(lds + chunk_at<4>(lane >> 2, lane & 3)) = t[0];
    }
    struct Frags {
        u32x4 c;
        float s;
        // i: the unit's place among those whose scales were loaded
        __device__ __forceinline__ void read(const char *lds, const char *sc, int i, int r, int g) {
            c = *reinterpret_cast<const u32x4 *>(lds + chunk_at<4>(r, g));
            s = mx4_scale_value((uint8_t)sc[r * 64 + i * 4 + g]);
        }
        __device__ __forceinline__ u32x4 get(int j) const {
            typedef __attribute__((ext_vector_type(2))) __bf16 b2;
            const b2 x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], s, 0),
                     y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], s, 1),
                     z = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], s, 2),
                     v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], s, 3);
            return u32x4{__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y),
                         __builtin_bit_cast(uint32_t, z), __builtin_bit_cast(uint32_t, v)};
        }
    };
    // The scale bytes of SPAN units from unit u (an even one: rows of scales
    // are multiples of eight bytes), 16 bytes a lane.
    struct Scales {
        u32x2 lo, hi;
    };
    __device__ __forceinline__ void load_scales(Scales &v, int u) const {
        const int c = u * 4 + (threadIdx.x & 3) * 16;
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(scales);
        v.lo = __builtin_amdgcn_raw_buffer_load_b64(rs, c < ks ? soff + c : OOB_OFFSET, 0, 0);
        v.hi = __builtin_amdgcn_raw_buffer_load_b64(rs, c + 8 < ks ? soff + c + 8 : OOB_OFFSET, 0, 0);
    }
    static __device__ __forceinline__ void store_scales(char *lds, const Scales &v) {
        *reinterpret_cast<u32x4 *>(lds + (threadIdx.x & 63) * 16) = u32x4{v.lo[0], v.lo[1], v.hi[0], v.hi[1]};
    }
};

// LDS of a wave: a unit of NM blocks of 16 weight rows and of XR tokens.
template <class R, int NM, int XR> constexpr int wave_lds() {
    return NM * (R::LDS + R::SCALES) + XR * R::XC * 16;
}

// What the weights are multiplied with, tiles of 16 columns one after the
// other. A source says how many registers a unit takes (LOADS of 16 bytes),
// asks for a unit, puts the rows of a tile into LDS, and names the row that a
// column reads and the sum that the tile is added to. off: byte offset of a
// lane's chunk, lane % XC of its row (OOB_OFFSET where there is no such row).
//
// XR rows of numbers of the type, a sum for each 16 of them (eight are
// multiplied as sixteen).
template <class T, class R, int XR> struct Plain {
    static constexpr int LOADS = XR * R::XC / 64, TILES = XR > 16 ? XR / 16 : 1, LDS_ROWS = XR;
    const T *base;
    uint32_t off[LOADS];
    using Unit = u32x4[LOADS];
    __device__ __forceinline__ void load(Unit &x, __amdgpu_buffer_rsrc_t rs, int u, bool in) const {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) x[i] = load_chunk(rs, off[i], u * (R::UK * 2), in);
    }
    // the unit that K ends in, n of whose k exist
    __device__ __forceinline__ void load_end(Unit &x, int u, int n) const {
        const int c = (threadIdx.x & 63) % R::XC * 8;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            x[i] = off[i] == OOB_OFFSET ? u32x4{0, 0, 0, 0}
                                        : end_chunk(base + (off[i] >> 1) - c + (int64_t)u * R::UK, c, n);
    }
    __device__ __forceinline__ void stage(char *xl, const Unit &x, int tile) const {
        const int lane = threadIdx.x & 63;
        if (tile == 0)
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                *reinterpret_cast<u32x4 *>(
                    xl + chunk_at<R::XC>(i * (64 / R::XC) + lane / R::XC, lane % R::XC)) = x[i];
    }
    static __device__ __forceinline__ int row(int tile, int r) { return XR > 8 ? tile * 16 + r : r & 7; }
    static constexpr int sum(int tile) { return tile; }
};

// The three numbers of S slots' h in bf16, a tile for each, all added to one sum.
template <class R, int S> struct Thirds {
    static constexpr int PER = S * R::XC / 64, LOADS = 3 * PER, TILES = 3, LDS_ROWS = S;
    const __bf16 *base;
    uint32_t off[PER];
    int part;   // bytes from a slot's number to its next
    using Unit = u32x4[LOADS];
    __device__ __forceinline__ void load(Unit &x, __amdgpu_buffer_rsrc_t rs, int u, bool in) const {
#pragma unroll
        for (int t = 0; t < 3; ++t)
#pragma unroll
            for (int i = 0; i < PER; ++i) x[t * PER + i] = load_chunk(rs, off[i], u * (R::UK * 2) + t * part, in);
    }
    // h is padded with zeros to whole chunks
    __device__ __forceinline__ void load_end(Unit &x, int u, int n) const {
        load(x, make_rsrc(base), u, (int)((threadIdx.x & 63) % R::XC * 8) < n);
    }
    __device__ __forceinline__ void stage(char *xl, const Unit &x, int tile) const {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            *reinterpret_cast<u32x4 *>(xl + chunk_at<R::XC>(i * (64 / R::XC) + lane / R::XC, lane % R::XC)) =
                x[tile * PER + i];
    }
    static __device__ __forceinline__ int row(int, int r) { return S > 8 ? r : r & 7; }
    static constexpr int sum(int) { return 0; }
};

// fp16 h: MT tiles of eight slots' fp32 activations, split on their way to LDS
// into an fp16 number and what it leaves, that times 2^11: 22 bits of whatever
// is 2^-14 or more, and 2^-36 of the rest. A slot whose activations pass fp16's
// range is scaled below 2^15 by a power of two. The split costs less than it
// saves in registers (64 experts of 2048 x 1000, 64 tokens: 72 us, 73 with the
// two numbers stored).
constexpr float SPLIT = 2048.0f;
__device__ __forceinline__ float peak_scale(uint32_t peak) {   // peak: 0, or of 2^15 and more
    return peak == 0u ? 1.0f : __builtin_bit_cast(float, (268u - (peak >> 23)) << 23);
}
__device__ __forceinline__ float peak_unscale(uint32_t peak) {
    return peak == 0u ? 1.0f : __builtin_bit_cast(float, ((peak >> 23) - 14u) << 23);
}
template <class R, int MT> struct Halves {
    static_assert(R::XC == 8, "a chunk of each of eight slots a lane");
    static constexpr int LOADS = 2 * MT, TILES = MT, LDS_ROWS = 16;
    const float *base;
    uint32_t off[MT];
    float scale[MT];
    using Unit = u32x4[LOADS];
    __device__ __forceinline__ void load(Unit &x, __amdgpu_buffer_rsrc_t rs, int u, bool in) const {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) x[i] = load_chunk(rs, off[i / 2], u * (R::UK * 4) + i % 2 * 16, in);
    }
    __device__ __forceinline__ void load_end(Unit &x, int u, int n) const {
        load(x, make_rsrc(base), u, (int)((threadIdx.x & 63) % R::XC * 8) < n);
    }
    __device__ __forceinline__ void stage(char *xl, const Unit &x, int tile) const {
        const int lane = threadIdx.x & 63;
        _Float16 hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = __builtin_bit_cast(f32x4, x[tile * 2 + j / 4])[j % 4] * scale[tile];
            hi[j] = (_Float16)y;
            const float rest = y - (float)hi[j];   // NaN where y is infinite
            lo[j] = (_Float16)(rest == rest ? rest * SPLIT : 0.0f);
        }
        *reinterpret_cast<u32x4 *>(xl + chunk_at<8>(lane >> 3, lane & 7)) = __builtin_bit_cast(u32x4, hi);
        *reinterpret_cast<u32x4 *>(xl + chunk_at<8>(8 + (lane >> 3), lane & 7)) = __builtin_bit_cast(u32x4, lo);
    }
    static __device__ __forceinline__ int row(int, int r) { return r; }
    static constexpr int sum(int tile) { return tile; }
};

// acc[sum][m] += 16 rows of each of NM weight blocks times the tiles of x over
// share `share` of `shares` of K. A unit's weights and tokens are asked for
// together, as many units before they are multiplied as STAGE_REGS registers
// hold (loads return in order: tokens asked for later would wait for the next
// units' weights). 72 registers: the down product of 32 MXFP4 experts of 4096 x
// 2048 40.6 us against 38.5, of 64 fp16 experts of 2048 x 1000 70.4 against 71.8,
// one bf16 token's up product 15.2 against 13.9. The units are taken round from
// unit `turn0` on: were every wave to start at the same k, all rows would be read
// at the same offset of their equal length, which the memory's channels do not
// share evenly.
constexpr int STAGE_REGS = 48;
template <class T, class R, class X, int NM>
__device__ __forceinline__ void multiply(const R *w, const X &src, int64_t K, int share, int shares, unsigned turn0,
                                         char *lds, f32x4 (*acc)[NM]) {
    constexpr int STAGE = (NM * R::WI + X::LOADS) * 4;
    constexpr int DEPTH = STAGE_REGS / STAGE > 4 ? 4 : STAGE_REGS / STAGE > 1 ? STAGE_REGS / STAGE : 1;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int k = uniform((int)K), c = lane % R::XC * 8;   // c: the lane's first k of a unit
    share = uniform(share);
    char *const wl = lds, *const xl = lds + NM * R::LDS, *const sl = xl + X::LDS_ROWS * R::XC * 16;
    const auto turn = [&](const typename R::Unit *t, const typename X::Unit &x, int scale_at) {
#pragma unroll
        for (int m = 0; m < NM; ++m) R::store(wl + m * R::LDS, t[m]);
        src.stage(xl, x, 0);
        typename R::Frags f[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) f[m].read(wl + m * R::LDS, sl + m * R::SCALES, scale_at, r, g);
#pragma unroll
        for (int mt = 0; mt < X::TILES; ++mt) {
            if (mt > 0) src.stage(xl, x, mt);
            u32x4 b[R::NF];
#pragma unroll
            for (int j = 0; j < R::NF; ++j)
                b[j] = *reinterpret_cast<const u32x4 *>(xl + chunk_at<R::XC>(X::row(mt, r), R::chunk_of(j, g)));
#pragma unroll
            for (int j = 0; j < R::NF; ++j)
#pragma unroll
                for (int m = 0; m < NM; ++m)
                    acc[X::sum(mt)][m] = mma16<T>(f[m].get(j), b[j], acc[X::sum(mt)][m]);
        }
    };
    // Units of whole chunks: 16-bit ones in turn; MXFP4 ones in runs of pairs (a
    // line of codes), and the scales of a run at once.
    const int units = k % 8 == 0 ? (k + R::UK - 1) / R::UK : k / R::UK, pairs = (units + 1) / 2;
    const int begin = R::SCALES ? share * pairs / shares * 2 : share;
    const int end = R::SCALES ? min((share + 1) * pairs / shares * 2, units) : units;
    const int step = R::SCALES ? 1 : shares;
    const int span = R::SCALES ? 16 : 1 << 30;
    const __amdgpu_buffer_rsrc_t xs = make_rsrc(src.base);
    for (int at = begin; at < end; at += span) {
        const int stop = end - at > span ? at + span : end;
        const int len = (stop - at + step - 1) / step, from = uniform((int)(turn0 * 2 % (unsigned)len));
        typename R::Scales sc[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) w[m].load_scales(sc[m], at);
        typename R::Unit t[DEPTH][NM];
        typename X::Unit x[DEPTH];
        const auto unit = [&](int i) { return at + (i + from < len ? i + from : i + from - len) * step; };
        const auto load_w = [&](int d, int i) {
            const int u = i < len ? unit(i) : at;
#pragma unroll
            for (int m = 0; m < NM; ++m) w[m].load(t[d][m], u, i < len && (R::PADDED || u * R::UK + c < k));
        };
        const auto load_x = [&](int d, int i) {
            const int u = i < len ? unit(i) : at;
            src.load(x[d], xs, u, i < len && u * R::UK + c < k);
        };
        // The first weights wait neither for the list of slots that the tokens'
        // offsets follow from nor for the scales: with the lists' own loads asked
        // for together, one token on 64 bf16 experts 34.2 us against 37.4 in all,
        // 64 tokens on 64 fp16 experts 176.6 against 181.
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load_w(d, d);
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load_x(d, d);
#pragma unroll
        for (int m = 0; m < NM; ++m) R::store_scales(sl + m * R::SCALES, sc[m]);
        for (int i = 0; i < len; i += DEPTH)
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                turn(t[d], x[d], unit(min(i + d, len - 1)) - at);   // past the end zeros are added
                load_w(d, i + d + DEPTH);
                load_x(d, i + d + DEPTH);
            }
    }
    const int n = k - units * R::UK;
    if (n > 0 && (R::SCALES ? shares - 1 : units % shares) == share) {   // K ends inside a chunk
        typename R::Unit t[NM];
        typename X::Unit x;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            typename R::Scales sc;
            w[m].load_scales(sc, units & ~1);
            w[m].load_end(t[m], units, n);
            R::store_scales(sl + m * R::SCALES, sc);
        }
        src.load_end(x, units, n);
        turn(t, x, units & 1);
    }
}

// h = silu(g) u for ROWS rows of the gate and of the up matrix and every token
// of one expert: a workgroup per (active expert, ROWS rows), whose waves take
// units of K in turn. h keeps its bits on its way to the down product. bf16 takes
// it as three numbers of eight bits each that add up to it (cut off, not rounded,
// so that none passes the type's range), for which the down product has columns
// to spare; fp16, whose range h may pass, as fp32 (Halves). Two numbers, 16 bits,
// took the down product of 32 MXFP4 experts of 4096 x 2048 and 16 tokens 36 us
// against 38.5, and changed one rounding of the output in a thousand.
constexpr int UP_W = 4;
template <class T> constexpr bool WIDE_H = false;   // h in fp32
template <> constexpr bool WIDE_H<_Float16> = true;
__device__ __forceinline__ float high_half(float v) {   // its first eight bits
    return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xFFFF0000u);
}
template <class T, class R, int ROWS, int XR>
__device__ __forceinline__ void up_body(const MoeArgs &a, const Ws &w, const Active &x, int m0, int64_t i0,
                                        char *lds) {
    constexpr int RB = ROWS / 16, MT = XR > 16 ? XR / 16 : 1;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    R wt[2 * RB];
    const int64_t row = (int64_t)x.expert * 2 * a.I + i0;
    const int last = (int)(a.I - 1 - i0);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int skip = b * 16 <= last ? b * 16 : 0;   // a block past the end repeats the first
        wt[b].at(a.up, a.up_s, row + skip, min(last - skip, 15), a.H);
        wt[RB + b].at(a.up, a.up_s, row + a.I + skip, min(last - skip, 15), a.H);
    }
    Plain<T, R, XR> src;
    src.base = static_cast<const T *>(a.x);
#pragma unroll
    for (int i = 0; i < src.LOADS; ++i) {
        const int p = m0 + i * (64 / R::XC) + lane / R::XC;
        const int slot = w.slots[x.first + min(p, x.count - 1)];
        src.off[i] = p < x.count ? (uint32_t)(slot / a.k * (int)a.ldx * 2 + lane % R::XC * 16) : OOB_OFFSET;
    }
    f32x4 acc[MT][2 * RB];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int m = 0; m < 2 * RB; ++m) acc[mt][m] = f32x4{0, 0, 0, 0};
    multiply<T>(wt, src, a.H, wave, UP_W, blockIdx.x, lds + wave * wave_lds<R, 2 * RB, XR>(), acc);
    const int tokens = min(x.count - m0, XR);
    float(*part)[2 * ROWS + 1] = reinterpret_cast<float(*)[2 * ROWS + 1]>(lds);
    __syncthreads();   // every wave is done with its LDS
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        if (mt * 16 + r < tokens)
#pragma unroll
            for (int m = 0; m < 2 * RB; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    part[wave * tokens + mt * 16 + r][m * 16 + g * 4 + i] = acc[mt][m][i];
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * ROWS; i += UP_W * 64) {
        const int n = i & (ROWS - 1), p = i / ROWS;
        if (i0 + n >= w.ip) continue;
        const int slot = w.slots[x.first + m0 + p];
        float gate = 0.0f, up = 0.0f;
#pragma unroll
        for (int v = 0; v < UP_W; ++v) {
            gate += part[v * tokens + p][n];
            up += part[v * tokens + p][ROWS + n];
        }
        const float y = i0 + n < a.I ? gate / (1.0f + __expf(-gate)) * up : 0.0f;
        const uint32_t mag = abs_bits(y);
        if constexpr (WIDE_H<T>) {
            reinterpret_cast<float *>(w.h)[(int64_t)slot * w.ip + i0 + n] = y;
            if (mag >= 0x47000000u && mag < 0x7F800000u) atomicMax(w.peak + slot, mag);   // 2^15 and more
        } else {
            // an infinite or NaN h is its first number
            const float rest = mag < 0x7F800000u ? y - high_half(y) : 0.0f, last = rest - high_half(rest);
            uint16_t *q = reinterpret_cast<uint16_t *>(w.h) + (int64_t)slot * 3 * w.ip + i0 + n;
            q[0] = (uint16_t)(mag > 0x7F800000u ? 0x7FC0u : __builtin_bit_cast(uint32_t, y) >> 16);
            q[w.ip] = (uint16_t)(__builtin_bit_cast(uint32_t, rest) >> 16);
            q[2 * w.ip] = (uint16_t)(__builtin_bit_cast(uint32_t, last) >> 16);
        }
    }
}

template <class T, class R, int ROWS>
__global__ __launch_bounds__(UP_W * 64) void moe_up_kernel(MoeArgs a, MoeLayout lay, int blocks) {
    extern __shared__ __align__(16) char up_lds[];   // the waves' units, then [UP_W * tokens][2 * ROWS + 1] sums
    const Ws w = moe_ws(a.ws, lay);
    const int at = blockIdx.x / blocks;
    const Active x = w.active[at];   // asked for together with their number
    if ((at >= *w.n_active) | (x.count == 0)) return;
    const int64_t i0 = (int64_t)(blockIdx.x - at * blocks) * ROWS;
    if (x.count <= 8) {
        up_body<T, R, ROWS, 8>(a, w, x, 0, i0, up_lds);
    } else if (x.count <= 16) {
        up_body<T, R, ROWS, 16>(a, w, x, 0, i0, up_lds);
    } else {
        // more than 32 tokens read the weights again, from the L2
        for (int m0 = 0; m0 < x.count; m0 += 32) {
            if (m0 > 0) __syncthreads();   // the sums are read
            up_body<T, R, ROWS, 32>(a, w, x, m0, i0, up_lds);
        }
    }
}
template <class R, int ROWS> constexpr size_t up_lds_bytes(int tokens) {
    constexpr int NM = 2 * ROWS / 16;
    const size_t unit = tokens <= 8 ? wave_lds<R, NM, 8>() : tokens <= 16 ? wave_lds<R, NM, 16>() : wave_lds<R, NM, 32>();
    const size_t sum = (size_t)(tokens < 32 ? tokens : 32) * (2 * ROWS + 1) * 4;
    return UP_W * (unit > sum ? unit : sum);
}

// out[t] = sum over the token's experts of p down[e] h: a workgroup per ROWS
// columns of out and group of at most DOWN_W active experts, a wave per expert.
// With one group (its waves share an expert's K where it has fewer experts) the
// products meet in LDS and the weighted sum follows there; with several, each
// stores its slots' products and the last to arrive at a column block adds them.
// Either way the sum runs over a token's choices in order, so the bits do not
// depend on the order of execution.
constexpr int DOWN_W = 8;
template <class T, class R, int ROWS, class X, class Sums>
__device__ __forceinline__ void down_rows(const MoeArgs &a, const Ws &w, const Active &x, int64_t n0, const X &src,
                                          int share, int shares, char *lds, const Sums &sums) {
    constexpr int RB = ROWS / 16, NS = X::sum(X::TILES - 1) + 1;
    R wt[RB];
    const int last = (int)min(a.H - 1 - n0, (int64_t)ROWS - 1);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int skip = b * 16 <= last ? b * 16 : 0;   // a block past the end repeats the first
        wt[b].at(a.down, a.down_s, (int64_t)x.expert * a.H + n0 + skip, min(last - skip, 15), a.I);
    }
    f32x4 acc[NS][RB];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int b = 0; b < RB; ++b) acc[s][b] = f32x4{0, 0, 0, 0};
    multiply<T>(wt, src, a.I, share, shares, blockIdx.x + 3 * (threadIdx.x >> 6), lds, acc);
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int b = 0; b < RB; ++b) sums(s, b * 16, acc[s][b]);
}

// Up to five slots of bf16 h as 3 x 5 columns of one tile; up to S from place m0
// on, a tile for each number; or 8 MT of fp16 h. sink(place, slot, column of the
// block, products). Sixteen slots a pass read the weights of 64 tokens on 32 MXFP4
// experts once where eight read them twice: 140 us the layer against 149.
constexpr int PACKED = 5;
template <class T, class R, int ROWS, class Sink>
__device__ __forceinline__ void down_packed(const MoeArgs &a, const Ws &w, const Active &x, int64_t n0, int share,
                                            int shares, char *lds, const Sink &sink) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    Plain<T, R, 16> src;
    src.base = reinterpret_cast<const T *>(w.h);
#pragma unroll
    for (int i = 0; i < src.LOADS; ++i) {
        const int row = i * (64 / R::XC) + lane / R::XC, part = row / PACKED, p = row - part * PACKED;
        const int slot = w.slots[x.first + min(p, x.count - 1)];
        src.off[i] = p < x.count && part < 3 ? (uint32_t)((slot * 3 + part) * (int)w.ip * 2 + lane % R::XC * 16)
                                             : OOB_OFFSET;
    }
    const int slot = w.slots[x.first + min(r % PACKED, x.count - 1)];   // of the products that the lane ends with
    down_rows<T, R, ROWS>(a, w, x, n0, src, share, shares, lds, [&](int, int c, f32x4 v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += __shfl_down(v[i], PACKED) + __shfl_down(v[i], 2 * PACKED);
        if (r < PACKED && r < x.count) sink(r, slot, c + g * 4, v);
    });
}
template <class R, int ROWS, int S, class Sink>
__device__ __forceinline__ void down_thirds(const MoeArgs &a, const Ws &w, const Active &x, int m0, int64_t n0,
                                            int share, int shares, char *lds, const Sink &sink) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    Thirds<R, S> src;
    src.base = reinterpret_cast<const __bf16 *>(w.h);
    src.part = (int)w.ip * 2;
#pragma unroll
    for (int i = 0; i < src.PER; ++i) {
        const int p = m0 + i * (64 / R::XC) + lane / R::XC, slot = w.slots[x.first + min(p, x.count - 1)];
        src.off[i] = p < x.count ? (uint32_t)(slot * 3 * (int)w.ip * 2 + lane % R::XC * 16) : OOB_OFFSET;
    }
    const int p = m0 + r, slot = w.slots[x.first + min(p, x.count - 1)];
    down_rows<__bf16, R, ROWS>(a, w, x, n0, src, share, shares, lds, [&](int, int c, f32x4 v) {
        if (r < S && p < x.count) sink(p, slot, c + g * 4, v);
    });
}
template <class R, int ROWS, int MT, class Sink>
__device__ __forceinline__ void down_halves(const MoeArgs &a, const Ws &w, const Active &x, int m0, int64_t n0,
                                            int share, int shares, char *lds, const Sink &sink) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    Halves<R, MT> src;
    src.base = reinterpret_cast<const float *>(w.h);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int p = m0 + t * 8 + (lane >> 3), slot = w.slots[x.first + min(p, x.count - 1)];
        src.off[t] = p < x.count ? (uint32_t)(slot * (int)w.ip * 4 + (lane & 7) * 32) : OOB_OFFSET;
        src.scale[t] = peak_scale(w.peak[slot]);
    }
    int slot_of[MT];
    float unscale[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        slot_of[t] = w.slots[x.first + min(m0 + t * 8 + (r & 7), x.count - 1)];
        unscale[t] = peak_unscale(w.peak[slot_of[t]]);
    }
    down_rows<_Float16, R, ROWS>(a, w, x, n0, src, share, shares, lds, [&](int t, int c, f32x4 v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (v[i] + __shfl_xor(v[i], 8) * (1.0f / SPLIT)) * unscale[t];
        const int p = m0 + t * 8 + r;
        if (r < 8 && p < x.count) sink(p, slot_of[t], c + g * 4, v);
    });
}

template <class T, class R, int ROWS>
__global__ __launch_bounds__(DOWN_W * 64, 4) void moe_down_kernel(MoeArgs a, MoeLayout lay) {
    extern __shared__ __align__(16) char down_lds[];   // the waves' units; with one group [DOWN_W * T][ROWS] products
    __shared__ int flag;
    __shared__ int16_t where[GEMM_MOE_MAX_TOKENS * DOWN_W];   // a slot's row of the first share, with one group
    constexpr int UNIT = wave_lds<R, ROWS / 16, 16>();
    constexpr int SC1 = 16;   // device scope: read by another workgroup, maybe of another XCD
    const Ws w = moe_ws(a.ws, lay);
    float(*y)[ROWS] = reinterpret_cast<float(*)[ROWS]>(down_lds + DOWN_W * UNIT);
    const int wave = uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63, slots = a.T * a.k;
    const int groups = gridDim.y, group = blockIdx.y, most = min(slots, a.E);
    const int64_t n0 = (int64_t)blockIdx.x * ROWS;
    // asked for together with their number: the entry if all that could be are active
    const int guess = groups > 1 ? min(group + wave * groups, most - 1) : wave % most;
    Active x = w.active[guess];
    const int active = *w.n_active;
    const int mine = active > group ? (active - group + groups - 1) / groups : 0;   // <= DOWN_W
    const int shares = mine == 0 ? 0 : groups > 1 ? 1 : DOWN_W / mine, share = mine > 0 ? wave / mine : 0;
    const __amdgpu_buffer_rsrc_t yg = make_rsrc(w.y + (int64_t)blockIdx.x * slots * ROWS);
    if (share < shares) {
        if (const int at = group + (wave - share * mine) * groups; at != guess) x = w.active[at];
        if (groups == 1 && share == 0 && lane < x.count)
            where[w.slots[x.first + lane]] = (int16_t)(wave * a.T + lane);
        const auto sink = [&](int p, int slot, int c, f32x4 v) {
            if (groups == 1)
                *reinterpret_cast<f32x4 *>(&y[wave * a.T + p][c]) = v;
            else
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), yg,
                                                       (slot * ROWS + c) * 4, 0, SC1);
        };
        char *const unit = down_lds + wave * UNIT;
        // the weights are read again for more slots than a pass takes, from the L2
        if constexpr (WIDE_H<T>) {
            if (x.count <= 8) down_halves<R, ROWS, 1>(a, w, x, 0, n0, share, shares, unit, sink);
            else
                for (int m0 = 0; m0 < x.count; m0 += 16)
                    down_halves<R, ROWS, 2>(a, w, x, m0, n0, share, shares, unit, sink);
        } else {
            if (x.count <= PACKED) down_packed<T, R, ROWS>(a, w, x, n0, share, shares, unit, sink);
            else if (x.count <= 8) down_thirds<R, ROWS, 8>(a, w, x, 0, n0, share, shares, unit, sink);
            else
                for (int m0 = 0; m0 < x.count; m0 += 16)
                    down_thirds<R, ROWS, 16>(a, w, x, m0, n0, share, shares, unit, sink);
        }
    }
    if (groups > 1) {
        if (!last_of(w.column_state + blockIdx.x, groups, &flag)) return;
    } else {
        __syncthreads();
    }
    // four columns of a token a thread; no load waits for another
    for (int i = threadIdx.x; i < a.T * (ROWS / 4); i += DOWN_W * 64) {
        const int n = i % (ROWS / 4) * 4, t = i / (ROWS / 4);
        f32x4 v{0, 0, 0, 0};
#pragma unroll 4
        for (int j = 0; j < a.k; ++j) {
            const int slot = t * a.k + j;
            const bool live = w.ids[slot] >= 0;
            const float p = w.probs[slot];
            f32x4 d{0, 0, 0, 0};
            if (groups > 1) {
                d = __builtin_bit_cast(
                    f32x4, __builtin_amdgcn_raw_buffer_load_b128(yg, (slot * ROWS + n) * 4, 0, SC1));
            } else {
                const int row = live ? where[slot] : 0;
                for (int s = 0; s < shares; ++s)
                    d += *reinterpret_cast<const f32x4 *>(&y[row + s * mine * a.T][n]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += live ? p * d[e] : 0.0f;
        }
        T *o = static_cast<T *>(a.out) + t * a.ldo + n0 + n;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n0 + n + e < a.H) o[e] = from_f<T>(v[e]);
    }
}
template <class R, int ROWS> constexpr size_t down_lds_bytes(int tokens, int groups) {
    return (size_t)DOWN_W * (wave_lds<R, ROWS / 16, 16>() + (groups > 1 ? 0 : tokens * ROWS * 4));
}

// Groups of at most DOWN_W experts that the active ones are cut into for the
// down product.
int down_groups(int E, int k, int T) {
    const int most = T * k < E ? T * k : E;
    return (most + DOWN_W - 1) / DOWN_W;
}

constexpr size_t MOE_LDS = 160 * 1024 - 2048;   // what a workgroup may ask for besides its fixed arrays

template <class T, class R, int ROWS>
hipError_t up(const MoeArgs &a, const MoeLayout &lay, int most, hipStream_t st) {
    static_assert(up_lds_bytes<R, ROWS>(GEMM_MOE_MAX_TOKENS) <= MOE_LDS, "LDS of a workgroup");
    const int64_t blocks = (lay.ip + ROWS - 1) / ROWS;
    if (blocks * most > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    moe_up_kernel<T, R, ROWS><<<(unsigned)(blocks * most), UP_W * 64, up_lds_bytes<R, ROWS>(a.T), st>>>(
        a, lay, (int)blocks);
    return hipGetLastError();
}

template <class T, class R, int ROWS>
hipError_t down(const MoeArgs &a, const MoeLayout &lay, int groups, hipStream_t st) {
    static_assert(down_lds_bytes<R, ROWS>(GEMM_MOE_MAX_TOKENS, 1) <= MOE_LDS, "LDS of a workgroup");
    const dim3 grid((unsigned)((a.H + ROWS - 1) / ROWS), (unsigned)groups);
    moe_down_kernel<T, R, ROWS><<<grid, DOWN_W * 64, down_lds_bytes<R, ROWS>(a.T, groups), st>>>(a, lay);
    return hipGetLastError();
}

template <class T, class R>
hipError_t run(const MoeArgs &a, hipStream_t st) {
    const MoeLayout lay = moe_layout(a.H, a.I, a.E, a.k, a.T, WIDE_H<T>);
    // as many waves an expert as leave one workgroup to a CU: one token on 64
    // experts 9.0 us with eight, 9.7 with two; 16 on 32 10.7 and 11.8; but 64 on
    // 64, where eight make 1024 workgroups, 19.7 and 12.2
    const int nt = a.T == 1 ? 1 : RT, chunks = (a.T + nt - 1) / nt;
    int split = ROUTER_W;
    while (split > 2 && (int64_t)a.E * split / ROUTER_W * chunks > 256) split /= 2;
    const int per = ROUTER_W / split;
    const dim3 rg((a.E + per - 1) / per, chunks);
    if (nt == 1) moe_router_kernel<T, 1><<<rg, ROUTER_W * 64, 0, st>>>(a, lay, split);
    else moe_router_kernel<T, RT><<<rg, ROUTER_W * 64, 0, st>>>(a, lay, split);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int most = a.T * a.k < a.E ? a.T * a.k : a.E, groups = down_groups(a.E, a.k, a.T);
    // 32 weight rows a wave read a token's h half as often as 16 and ask for the
    // lists half as often, if enough workgroups are left: up, 32 MXFP4 experts of
    // 4096 x 2048, 16 tokens, 55 us against 66 (but fp16 weights, which outweigh
    // the tokens, 98 against 93); down, the same experts 39 against 48, 64 fp16
    // experts of 2048 x 1000, 64 tokens, 72 against 81, but one token on two bf16
    // experts of 1024 x 4096, 32 workgroups, 13.8 against 11.0.
    if (lay.ip > 0) {
        e = R::WIDE_UP && lay.ip / 32 * most >= 512 ? up<T, R, R::WIDE_UP ? 32 : 16>(a, lay, most, st)
                                                    : up<T, R, 16>(a, lay, most, st);
        if (e != hipSuccess) return e;
    }
    if (a.H == 0) return hipSuccess;
    return a.H / 32 * groups >= 256 ? down<T, R, 32>(a, lay, groups, st) : down<T, R, 16>(a, lay, groups, st);
}

}  // namespace

int64_t moe_state_bytes(int64_t H) {
    return ((CHUNKS + 1) * ST_STRIDE + (H + 15) / 16) * 4;
}

MoeLayout moe_layout(int64_t H, int64_t I, int E, int k, int T, bool wide_h) {
    MoeLayout l;
    int64_t at = (moe_state_bytes(H) + 15) / 16 * 16;
    const auto take = [&](int64_t bytes) {
        const int64_t p = at;
        at += (bytes + 15) / 16 * 16;
        return p;
    };
    const int64_t n = (int64_t)T * k;
    l.columns = (CHUNKS + 1) * ST_STRIDE * 4;
    l.ip = (I + 7) / 8 * 8;
    l.logits = take((int64_t)T * E * 8);
    l.ids = take(n * 4);
    l.probs = take(n * 4);
    l.slots = take(n * 4);
    l.active = take(16 + (int64_t)(n < E ? n : E) * 16);
    l.h = take(n * l.ip * (wide_h ? 4 : 3 * 2));
    l.peak = take(n * 4);
    l.y = take(down_groups(E, k, T) > 1 ? (H + 31) / 32 * 32 * n * 4 : 0);
    l.total = at;
    return l;
}

hipError_t launch_moe(int type, int weight_type, const MoeArgs &a, hipStream_t st) {
    if (weight_type == GEMM_F4_E2M1) return run<__bf16, Rows4>(a, st);
    if (type == GEMM_F16) return run<_Float16, Rows16<_Float16>>(a, st);
    return run<__bf16, Rows16<__bf16>>(a, st);
}

}  // namespace mg
