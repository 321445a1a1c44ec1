// Attention of many query rows over a paged 8-bit key-value cache, on the 5th-generation
// tensor cores (prompts and prompt pieces; bf16 queries).
//
// A block holds two tiles of 128 query rows (row = new token x query head of the cached
// head) and goes through the cached keys 128 at a time:
//     S = Q K^T            tcgen05, operands in shared memory, S in TMEM
//     P = 2^(c S - m)      one thread a row, S from TMEM, P (f16) over S's place in TMEM
//     O += P V             tcgen05, P from TMEM, O in TMEM
// with the running row maximum m and sum in registers.  While one tile's softmax runs,
// the tensor cores work for the other.  m moves only when a row's maximum grew by more
// than 2^8, so the accumulator is rescaled a few times a row, not once a tile (weights
// then reach 2^8 at most, which f16 and the fp32 sums hold without loss).
//
// Bound by the tensor cores (4 D operations for each visible pair) with the exponentials
// close behind.  The codes would have to be f16 for the products anyway (weights and
// queries as 8-bit floats would cost the result 4 bits), so they are widened once for
// the 256 rows on the way into shared memory: eight warps load 16 bytes a thread, widen
// (exact) and store in the 128-byte-swizzled layout that the products read.  There the
// page scales come in too, as powers of two relative to the largest scale that the block
// sees (2^0 .. 2^-24 in f16, exact while a code times that ratio is at least 2^-24).  So
// scores and outputs carry one factor a row and no scale inside the loop.
//
// When the blocks are fewer than the SMs, a cluster splits the keys of a row chunk and
// joins its shares over distributed shared memory.
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace caat {
namespace {

using namespace tc;

constexpr int TILE = 128;                    // rows of a tile; keys of a step
constexpr int STAGES = 2;
constexpr int WARPS = 17, THREADS = WARPS * 32;
// warps 0-3 and 4-7: softmax of tile 0 and 1; 8-11: keys; 12-15: values; 16: products
constexpr int W_KEYS = 8, W_VALUES = 12, W_MMA = 16;
constexpr uint32_t TMEM_COLS = 512, O_COL = 256;
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr float LAZY = 8.f;

struct TileParams {
    const void *q;
    int64_t q_st, q_sk, q_sg;
    void *o;
    int64_t o_st, o_sh;
    float scale_log2;
    int window, sinks, group, chunks, splits;
    int *err;
    PagedKV kv;
    PagedBatch pb;
};

struct Ctl {
    uint64_t q_full[2], k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES], s_full[2], p_full[2];
    uint32_t tmem;
    int abort, v_nan;
    float ref_k, ref_v;
    float part[2][4];
};

__host__ __device__ constexpr int half_bytes() { return TILE * 128; }       // 128 rows of 64 f16
__host__ __device__ constexpr int tile_bytes(int DP) { return DP / 64 * half_bytes(); }
__host__ __device__ constexpr int pitch(int DP) { return DP + 4; }          // floats of a row's share
__host__ __device__ constexpr int smem_bytes(int DP)
{
    const int run = (2 + 2 * STAGES) * tile_bytes(DP);
    const int join = 2 * TILE * (pitch(DP) + 2) * 4;
    return 1024 + 1024 + (run > join ? run : join);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, __half2 f)
{
    const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&a), f);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// D[tmem] (+)= A[tmem] * B[smem]: A is 128 lanes of f16 pairs
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// kind::f16 with f16 operands, fp32 accumulator
constexpr uint32_t idesc_f16(int M, int N, bool b_mn)
{
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16-byte chunk `ch` (of 8) of row r in a 128-byte-swizzled block of rows
__device__ __forceinline__ uint32_t swizzled(int r, int ch) { return (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4)); }

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ float ld_cluster(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ void give_up(volatile int *abort, int *err)
{
    *abort = 1;
    *(volatile int *)err = CAAT_ERR_TIMEOUT;
}

template <int DP>
__global__ void __launch_bounds__(THREADS, 1) paged_attn_tile_kernel(const __grid_constant__ TileParams p)
{
    extern __shared__ uint8_t raw[];
    uint8_t *base = (uint8_t *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    Ctl *ctl = (Ctl *)base;
    uint8_t *bufs = base + 1024;
    constexpr int TB = tile_bytes(DP), HB = half_bytes();
    const uint32_t q_s = smem_u32(bufs), k_s = q_s + 2 * TB, v_s = k_s + STAGES * TB;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort = &ctl->abort;
    const int P = p.kv.page, D = p.kv.dim;

    const int split = (int)(blockIdx.x % p.splits);
    int64_t unit = blockIdx.x / p.splits;
    // the last rows of a prompt see the most keys: their chunks start first
    const int64_t per_chunk = (int64_t)p.pb.batch * p.kv.kv_heads;
    const int chunk = p.chunks - 1 - (int)(unit / per_chunk);
    unit %= per_chunk;
    const int h = (int)(unit % p.kv.kv_heads), b = (int)(unit / p.kv.kv_heads);
    const Seq sq = load_seq(p.pb, P, b, p.err);
    const int rows_all = sq.n * p.group;
    const int row0 = chunk * 2 * TILE;
    if (row0 >= rows_all) return;            // the whole cluster
    const int rows = min(2 * TILE, rows_all - row0);
    const int tiles = rows > TILE ? 2 : 1;
    const int p_lo = sq.pos0 + row0 / p.group;
    const int p_hi[2] = {sq.pos0 + (row0 + min(rows, TILE) - 1) / p.group, sq.pos0 + (row0 + rows - 1) / p.group};

    // steps of 128 keys: those of the first tokens, then the window's
    const int win_lo = p.window > 0 ? max(0, p_lo - p.window + 1) : 0;
    const int t_lo = win_lo >> 7;
    const int n_sink = min((int)(((int64_t)p.sinks + TILE - 1) >> 7), t_lo);
    int nk[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) nk[t] = p_hi[t] < 0 ? 0 : n_sink + (p_hi[t] >> 7) + 1 - t_lo;
    const int n_all = nk[tiles - 1];
    const int j_lo = (int)((int64_t)n_all * split / p.splits), j_hi = (int)((int64_t)n_all * (split + 1) / p.splits);
    const int steps = j_hi - j_lo;           // tile t takes part in the first `last[t]` of them
    const int last[2] = {max(0, min(nk[0], j_hi) - j_lo), tiles > 1 ? steps : 0};
    auto key0 = [&](int j) { return (j < n_sink ? j : t_lo + j - n_sink) << 7; };

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl->q_full[i]), 4);
            mbar_init(smem_u32(&ctl->s_full[i]), 1);
            mbar_init(smem_u32(&ctl->p_full[i]), 4);
        }
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_u32(&ctl->k_full[i]), 4);
            mbar_init(smem_u32(&ctl->v_full[i]), 4);
            mbar_init(smem_u32(&ctl->k_empty[i]), 1);
            mbar_init(smem_u32(&ctl->v_empty[i]), 1);
        }
        ctl->abort = 0;
        ctl->v_nan = 0;
        fence_mbar_init();
    }
    if (warp == W_MMA) {
        tmem_alloc(smem_u32(&ctl->tmem), TMEM_COLS);
        tmem_relinquish();
    }
    const int32_t *table = p.pb.table + (int64_t)b * p.pb.table_stride;

    // the largest scale of each side that the block's steps see
    if (warp >= W_KEYS && warp < W_MMA && steps > 0) {
        const bool keys = warp < W_VALUES;
        const float *sc = keys ? p.kv.ks : p.kv.vs;
        float m = 0.f;
        const int per = max(1, TILE >> p.kv.log2_page);          // pages of a step
        const int n = steps * per;
        for (int i = tid & 127; i < n; i += 128) {
            const int key = key0(j_lo + i / per) + (i % per) * P;
            if (key > p_hi[1]) continue;
            const int64_t pg = checked_page(__ldg(table + (key >> p.kv.log2_page)), p.kv, p.err);
            if (pg >= 0) m = fmaxf(m, __ldg(sc + pg * p.kv.scale_stride + h));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) ctl->part[keys ? 0 : 1][warp & 3] = m;
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = ctl->tmem;
    float ref[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float m = fmaxf(fmaxf(ctl->part[i][0], ctl->part[i][1]), fmaxf(ctl->part[i][2], ctl->part[i][3]));
        ref[i] = steps > 0 && m > 0.f ? m : 1.f;
    }

    if (warp < W_KEYS) {
        // ---------------- softmax: one thread a row
        const int t = warp >> 2, r = tid & 127;
        const int row = row0 + t * TILE + r;
        const bool live = t * TILE + r < rows;
        const int pos = sq.pos0 + row / p.group;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t s_t = tmem + lanes + (uint32_t)t * TILE, o_t = tmem + lanes + O_COL + (uint32_t)t * TILE;
        float c = 0.f, m_ref = -INFINITY, sum = 0.f;
        bool ok = true;
        if (last[t] > 0) {
            // the row as f16 times a power of two that brings its largest magnitude to [2^14, 2^15)
            const uint16_t *src = reinterpret_cast<const uint16_t *>(p.q) + (sq.t0 + row / p.group) * p.q_st +
                                  h * p.q_sk + (row % p.group) * p.q_sg;
            float m = 0.f;
            for (int d = 0; d < D && live; d += 8) {
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(src + d));
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = fabsf(__uint_as_float(x[e] << 16)), z = fabsf(__uint_as_float(x[e] & 0xffff0000u));
                    m = fmaxf(m, a <= 3.402823466e38f ? a : 0.f);
                    m = fmaxf(m, z <= 3.402823466e38f ? z : 0.f);
                }
            }
            const int e = m > 0.f ? max((int)(__float_as_uint(m) >> 23) - 127, -100) : 0;
            const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
            c = p.scale_log2 / up * ref[0];
            for (int d = 0; d < D; d += 8) {
                uint32_t y[4] = {0u, 0u, 0u, 0u};
                if (live) {
                    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(src + d));
                    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        y[i] = pack_f16(__uint_as_float(x[i] << 16) * up, __uint_as_float(x[i] & 0xffff0000u) * up);
                }
                st_shared16(q_s + t * TB + (d >> 6) * HB + swizzled(r, (d >> 3) & 7), y[0], y[1], y[2], y[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->q_full[t]));
        }
        const int t_lo_pos = sq.pos0 + (row0 + t * TILE) / p.group, t_hi_pos = p_hi[t];
        for (int j = 0; j < last[t]; ++j) {
            ok = mbar_wait(smem_u32(&ctl->s_full[t]), (uint32_t)j & 1u, abort, WAIT_NS);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                give_up(abort, p.err);
                break;
            }
            fence_after_sync();
            const int k0 = key0(j_lo + j);
            // every row of the tile sees every key of the step?
            const bool all = k0 + TILE - 1 <= t_lo_pos &&
                             (p.window == 0 || k0 > t_hi_pos - p.window || k0 + TILE - 1 < p.sinks);
            // visible columns: [0, first) of the first tokens and (from, upto]
            const int upto = pos - k0, from = p.window > 0 ? pos - p.window - k0 : -1;
            const int first = p.window > 0 ? p.sinks - k0 : 0;
            auto sees = [&](int col) { return col <= upto && (col > from || col < first); };
            float mx = -INFINITY;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t v0[32], v1[32];
                tmem_ld32x2(s_t + 64 * q, s_t + 64 * q + 32, v0, v1);
                if (all) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fmaxf(__uint_as_float(v0[i]), __uint_as_float(v1[i])));
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (sees(64 * q + i)) mx = fmaxf(mx, __uint_as_float(v0[i]));
                        if (sees(64 * q + 32 + i)) mx = fmaxf(mx, __uint_as_float(v1[i]));
                    }
                }
            }
            mx *= c;
            const bool grow = mx > m_ref + LAZY;
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? exp2_approx(m_ref - mx) : 1.f;
                if (grow) m_ref = mx;
                sum *= f;
                if (j > 0) {
#pragma unroll 1
                    for (int d = 0; d < D; d += 32) {
                        uint32_t v[32];
                        tmem_ld32(o_t + d, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                        tmem_st32(o_t + d, v);
                    }
                }
            }
            const float sub = m_ref == -INFINITY ? 0.f : m_ref;
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t v[32], w[16];
                tmem_ld32(s_t + 32 * q, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float a = fmaf(__uint_as_float(v[2 * i]), c, -sub), z = fmaf(__uint_as_float(v[2 * i + 1]), c, -sub);
                    if (!all) {
                        if (!sees(32 * q + 2 * i)) a = -INFINITY;
                        if (!sees(32 * q + 2 * i + 1)) z = -INFINITY;
                    }
                    a = exp2_approx(a);
                    z = exp2_approx(z);
                    s0 += a;
                    s1 += z;
                    w[i] = pack_f16(a, z);
                }
                tmem_st16(s_t + 16 * q, w);
            }
            sum += s0 + s1;
            tmem_wait_st();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->p_full[t]));
        }
        // the products' last commit follows the last step
        if (ok && last[t] > 0) {
            ok = mbar_wait(smem_u32(&ctl->s_full[t]), (uint32_t)last[t] & 1u, abort, WAIT_NS);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) give_up(abort, p.err);
            fence_after_sync();
        }
        const bool have = ok && last[t] > 0;
        const bool nan = have && *(volatile int *)&ctl->v_nan != 0;
        if (p.splits == 1) {
            if (ok && t < tiles) {
                const float f = have && sum != 0.f ? ref[1] / sum : 0.f;
                __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(p.o) + (sq.t0 + row / p.group) * p.o_st +
                                     (h * p.group + row % p.group) * p.o_sh;
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                    uint32_t v[32];
                    if (have) {
                        tmem_ld32(o_t + d, v);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0u;
                    }
                    if (nan) {
                        // rare: a value the row sees is NaN; go through its keys' codes
                        for (int j = 0; j < last[t] && live; ++j)
                            for (int i = 0; i < TILE; ++i) {
                                const int key = key0(j_lo + j) + i;
                                if (!(key <= pos && (p.window == 0 || key > pos - p.window || key < p.sinks))) continue;
                                const int64_t pg = checked_page(__ldg(table + (key >> p.kv.log2_page)), p.kv, p.err);
                                if (pg < 0) continue;
                                const uint8_t *code = p.kv.v + pg * p.kv.page_stride + ((int64_t)h * P + (key & (P - 1))) * D;
                                for (int e = 0; e < 32 && d + e < D; ++e)
                                    if ((code[d + e] & 0x7f) == 0x7f) {
#pragma unroll
                                        for (int x = 0; x < 32; ++x)
                                            if (x == e) v[x] = 0x7fffffffu;
                                    }
                            }
                    }
                    if (live) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (d + 8 * i >= D) break;
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(v[8 * i + 2 * e]) * f,
                                                                               __uint_as_float(v[8 * i + 2 * e + 1]) * f);
                                w[e] = *reinterpret_cast<const uint32_t *>(&x);
                            }
                            *reinterpret_cast<uint4 *>(out + d + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            }
        }
    } else if (warp < W_MMA) {
        // ---------------- codes to f16: keys (warps 8-11) and values (12-15)
        const bool keys = warp < W_VALUES;
        constexpr int CH = DP / 16;              // 16-code chunks of a row: lanes of a row
        constexpr int RPL = 32 / CH;             // rows of one load of the warp
        constexpr int LOADS = 32 / RPL;          // loads for the warp's 32 rows
        const int ch = lane % CH, rl = lane / CH;
        const int r_base = (warp & 3) * 32;
        const uint8_t *codes = (keys ? p.kv.k : p.kv.v) + (int64_t)h * P * D;
        const float *sc = keys ? p.kv.ks : p.kv.vs;
        const float r_ref = 1.f / ref[keys ? 0 : 1];
        const uint32_t stage0 = keys ? k_s : v_s;
        uint64_t *full = keys ? ctl->k_full : ctl->v_full, *empty = keys ? ctl->k_empty : ctl->v_empty;
        const bool in = ch * 16 < D;
        // the warp's rows are two groups of 16 keys, each within a page
        auto page_id = [&](int j, int g) {
            const int key = key0(j_lo + j) + r_base + 16 * g;
            return j < steps && key <= p_hi[1] ? __ldg(table + (key >> p.kv.log2_page)) : -1;
        };
        uint4 cur[LOADS];
        float f_cur[2];
        auto load = [&](int j, const int (&id)[2]) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int key = key0(j_lo + j) + r_base + 16 * g;
                int64_t pg = -1;
                if (id[g] >= 0 || (j < steps && key <= p_hi[1])) pg = checked_page(id[g], p.kv, p.err);
                f_cur[g] = pg >= 0 ? __ldg(sc + pg * p.kv.scale_stride + h) * r_ref : 0.f;
                const uint8_t *src = codes + (pg >= 0 ? pg : 0) * p.kv.page_stride + (int64_t)(key & (P - 1)) * D + ch * 16;
#pragma unroll
                for (int i = 0; i < LOADS / 2; ++i) {
                    const int r = i * RPL + rl;
                    cur[g * (LOADS / 2) + i] =
                        pg >= 0 && in ? __ldg(reinterpret_cast<const uint4 *>(src + (int64_t)r * D)) : make_uint4(0, 0, 0, 0);
                }
            }
        };
        int id[2] = {page_id(0, 0), page_id(0, 1)};
        if (steps > 0) load(0, id);
        id[0] = page_id(1, 0);
        id[1] = page_id(1, 1);
        bool ok = true;
        uint32_t bad = 0;
        for (int j = 0; j < steps; ++j) {
            const int st = j % STAGES;
            ok = mbar_wait(smem_u32(&empty[st]), ((uint32_t)(j / STAGES) & 1u) ^ 1u, abort, WAIT_NS);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                give_up(abort, p.err);
                break;
            }
            const uint32_t dst = stage0 + st * TB + (ch >> 2) * HB;
            const int k0 = key0(j_lo + j);
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int g = i / (LOADS / 2);
                const int r = r_base + i * RPL + rl;
                uint32_t w[4] = {cur[i].x, cur[i].y, cur[i].z, cur[i].w};
                if (!keys) {
                    // NaN values are taken out; where some row may see one, the epilogue looks
                    // for it (0x7f + 1 and 0xff + 1 carry into the sign bit of the masked byte)
                    uint32_t nan[4], any = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        nan[e] = ((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                        any |= nan[e];
                    }
                    if (any) {
                        if (k0 + r <= p_hi[1]) bad = 1;
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] &= ~((nan[e] >> 7) * 0xffu);
                    }
                }
                const __half2 f = __float2half2_rn(f_cur[g]);
                uint32_t y[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[2 * e] = mul_f16x2(e4m3x2_f16x2(w[e] & 0xffffu), f);
                    y[2 * e + 1] = mul_f16x2(e4m3x2_f16x2(w[e] >> 16), f);
                }
                // lanes of the two 64-column halves store their two chunks in opposite order,
                // so that eight lanes always meet eight different bank groups
                const int flip = (ch >> 2) & 1, c2 = (ch & 3) * 2;
                if (in) {
                    const uint32_t a0 = dst + swizzled(r, c2 + flip), a1 = dst + swizzled(r, c2 + 1 - flip);
                    st_shared16(a0, flip ? y[4] : y[0], flip ? y[5] : y[1], flip ? y[6] : y[2], flip ? y[7] : y[3]);
                    st_shared16(a1, flip ? y[0] : y[4], flip ? y[1] : y[5], flip ? y[2] : y[6], flip ? y[3] : y[7]);
                }
            }
            if (bad) *(volatile int *)&ctl->v_nan = 1;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&full[st]));
            if (j + 1 < steps) load(j + 1, id);
            id[0] = page_id(j + 2, 0);
            id[1] = page_id(j + 2, 1);
        }
    } else {
        // ---------------- products, issued by one thread
        if (lane == 0) {
            const uint32_t id_s = idesc_f16(TILE, TILE, false), id_o = idesc_f16(TILE, D, true);
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t ph) {
                ok = ok && mbar_wait(smem_u32(bar), ph & 1u, abort, WAIT_NS);
                fence_after_sync();
            };
            auto scores = [&](int t, int j) {
                const uint32_t a = q_s + t * TB, bk = k_s + (j % STAGES) * TB;
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (uint32_t)(k >> 2) * HB + (uint32_t)(k & 3) * 32u;
                    mma_f16(tmem + t * TILE, desc_kmajor_sw128(a + off), desc_kmajor_sw128(bk + off), id_s, k > 0);
                }
                mma_commit(smem_u32(&ctl->s_full[t]));
            };
            auto outputs = [&](int t, int j) {
                const uint32_t bv = v_s + (j % STAGES) * TB;
#pragma unroll
                for (int k = 0; k < TILE / 16; ++k)
                    mma_f16_ta(tmem + O_COL + t * TILE, tmem + t * TILE + 8 * k, desc_sw128(bv + 2048u * k, HB, 1024u), id_o,
                               j > 0 || k > 0);
            };
            for (int t = 0; t < tiles; ++t)
                if (last[t] > 0) wait(&ctl->q_full[t], 0);
            if (steps > 0) {
                wait(&ctl->k_full[0], 0);
                if (ok) {
                    for (int t = 0; t < 2; ++t)
                        if (last[t] > 0) scores(t, 0);
                    mma_commit(smem_u32(&ctl->k_empty[0]));
                }
            }
            for (int j = 0; j < steps && ok; ++j) {
                const uint32_t ph = (uint32_t)(j / STAGES), st = j % STAGES;
                wait(&ctl->v_full[st], ph);
                if (j + 1 < steps) wait(&ctl->k_full[(j + 1) % STAGES], (uint32_t)((j + 1) / STAGES));
                for (int t = 0; t < 2 && ok; ++t) {
                    if (j >= last[t]) continue;
                    wait(&ctl->p_full[t], (uint32_t)j);
                    if (!ok) break;
                    outputs(t, j);
                    if (j + 1 < last[t]) scores(t, j + 1);
                    else mma_commit(smem_u32(&ctl->s_full[t]));
                }
                if (ok) {
                    mma_commit(smem_u32(&ctl->v_empty[st]));
                    if (j + 1 < steps) mma_commit(smem_u32(&ctl->k_empty[(j + 1) % STAGES]));
                }
            }
            if (!ok) give_up(abort, p.err);
        }
        __syncwarp();
    }
    fence_before_sync();
    __syncthreads();
    if (*abort) {
        if (tid == 0) {                          // let the products in flight end before TMEM goes
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 2000000ull) { }
        }
        __syncthreads();
    }
    if (warp == W_MMA) {
        fence_after_sync();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <int DP>
caat_status launch_tile(TileParams &p, cudaStream_t s)
{
    const int64_t rows = (int64_t)p.pb.q_max * p.group;
    const int64_t chunks = (rows + 2 * TILE - 1) / (2 * TILE);
    const int64_t units = (int64_t)p.pb.batch * p.kv.kv_heads * chunks;
    if (chunks > 0x7fffffff) return CAAT_ERR_INVALID_ARG;
    p.chunks = (int)chunks;
    p.splits = 1;
    if (units * p.splits > 0x7fffffff) return CAAT_ERR_INVALID_ARG;
    auto kern = paged_attn_tile_kernel<DP>;
    if (prepare_kernel_smem((const void *)kern, smem_bytes(DP)) != CAAT_OK) return CAAT_ERR_CUDA;
    kern<<<(unsigned)(units * p.splits), THREADS, smem_bytes(DP), s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return CAAT_ERR_CUDA;
    note_launch("paged_attn_tile");
    return CAAT_OK;
}

}  // namespace

caat_status launch_paged_attention_tile(const PagedKV &kv, const PagedBatch &pb, int heads, const void *q, int64_t q_st,
                                        int64_t q_sk, int64_t q_sg, float scale, int window, int sinks, void *o,
                                        int64_t o_st, int64_t o_sh, cudaStream_t s)
{
    TileParams p{q, q_st, q_sk, q_sg, o, o_st, o_sh, scale * 1.4426950408889634f, window, sinks, heads / kv.kv_heads,
                 1, 1, serve_error_word(), kv, pb};
    if (p.err == nullptr) return CAAT_ERR_CUDA;
    return kv.dim <= 64 ? launch_tile<64>(p, s) : launch_tile<128>(p, s);
}

}  // namespace caat
