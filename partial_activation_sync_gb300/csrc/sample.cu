// The next token of each row of logits from a given uniform number: temperature,
// top-k, top-p and min-p.
//
// With z the logits, ordered by value (largest first, equal values by index):
//     w_i = e^((z_i - max z) / T)
//     top-k: the first k;  top-p: of those the shortest prefix whose weights reach
//     top_p of their sum (the token that reaches it stays);  min-p: w_i >= min_p;
//     the token is the smallest index i with  sum of kept w_j, j <= i  >  u * sum of kept.
// T <= 0 takes the largest logit, the lowest index of equals.  NaN counts as -inf.  The
// first of the order is always kept.  The log probability returned is the token's
// under softmax(z), before temperature and filters.
//
// Every filter keeps a prefix of the order, so together they are one threshold: a
// value and how many of its equals stay.  Nothing is sorted: the threshold is found by
// bisection over the 32-bit ordered form of the values, each step one pass over the
// row for a count or a sum of weights.  Weights are summed in fp32 over at most a few
// hundred terms and then in 64 bits, in a fixed order.
#include "paged.cuh"

namespace caat {
namespace {

constexpr int THREADS = 1024, WARPS = THREADS / 32;

struct SampleParams {
    const void *logits;
    int64_t ld, V;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *token;
    float *logprob;
};

// floats in an order that unsigned integers keep; NaN below everything (0)
__device__ __forceinline__ uint32_t ordered(float z)
{
    if (z != z) return 0u;
    const uint32_t b = __float_as_uint(z == 0.f ? 0.f : z);      // -0 equals 0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float unordered(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

constexpr uint32_t KEY_NEG_INF = 0x007fffffu;   // ordered(-inf)

__device__ __forceinline__ float value(const float *p, int64_t i) { return __ldg(p + i); }
__device__ __forceinline__ float value(const __nv_bfloat16 *p, int64_t i)
{
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(p) + i) << 16);
}

struct Shared {
    double d[WARPS];
    unsigned long long l[WARPS];
    double bd;
    unsigned long long bl;
};

__device__ __forceinline__ double block_sum(double x, Shared &sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.d[threadIdx.x >> 5] = x;
    __syncthreads();
    x = sh.d[threadIdx.x & 31];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ unsigned long long block_max(unsigned long long x, Shared &sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.l[threadIdx.x >> 5] = x;
    __syncthreads();
    x = sh.l[threadIdx.x & 31];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

template <typename E>
__global__ void __launch_bounds__(THREADS) sample_kernel(SampleParams p)
{
    __shared__ Shared sh;
    const int64_t row = blockIdx.x;
    const E *z = reinterpret_cast<const E *>(p.logits) + row * p.ld;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int V = (int)p.V;
    // each warp owns one run of the row, so that sums in index order are sums over warps
    const int seg = (V + WARPS - 1) / WARPS;
    const int lo = min(V, warp * seg), hi = min(V, lo + seg);

    // largest value and its lowest index
    unsigned long long best = 0;
    for (int i = lo + lane; i < hi; i += 32)
        best = max(best, (unsigned long long)ordered(value(z, i)) << 32 | (uint32_t)~i);
    best = block_max(best, sh);
    const uint32_t kmax = (uint32_t)(best >> 32);
    if (kmax <= KEY_NEG_INF) {                    // no token can be drawn
        if (threadIdx.x == 0) {
            p.token[row] = -1;
            p.logprob[row] = -INFINITY;
        }
        return;
    }
    const float zmax = unordered(kmax);
    const float T = p.temperature[row];
    // equal values weigh 1 even where both are infinite; -inf, NaN and all below +inf
    // weigh 0.  The gap stays finite, so that an infinite T makes it 0 and not NaN.
    auto weight = [&](float x, float inv) {
        return x == zmax ? 1.f
               : x > -INFINITY && zmax < INFINITY ? expf(fmaxf(x - zmax, -3.402823466e38f) * inv) : 0.f;
    };
    float part = 0.f;
    for (int i = lo + lane; i < hi; i += 32) part += weight(value(z, i), 1.f);
    const double all = block_sum(part, sh);
    int token = (int)~(uint32_t)best;
    if (T > 0.f) {
        const float inv = 1.f / T;
        auto count_ge = [&](uint32_t key) {
            int n = 0;
            for (int i = lo + lane; i < hi; i += 32) n += ordered(value(z, i)) >= key;
            return (int64_t)block_sum(n, sh);
        };
        auto weight_ge = [&](uint32_t key) {
            float s = 0.f;
            for (int i = lo + lane; i < hi; i += 32) {
                const float x = value(z, i);
                if (ordered(x) >= key) s += weight(x, inv);
            }
            return block_sum(s, sh);
        };
        // kept: keys above thr, and the first `ties` of those equal to it
        uint32_t thr = 0;
        int64_t ties = V;
        const int k = p.top_k[row];
        if (k > 0 && k < V) {
            uint32_t a = 0, b = kmax;             // count_ge(a) >= k; the largest such key
            while (a < b) {
                const uint32_t mid = a + (b - a) / 2 + 1;
                if (count_ge(mid) >= k) a = mid;
                else b = mid - 1;
            }
            thr = a;
            ties = thr == 0xffffffffu ? k : k - count_ge(thr + 1);
        }
        const float tp = p.top_p[row], mp = p.min_p[row];
        const float wthr = weight(unordered(thr), inv);
        if (tp < 1.f) {
            auto kept_ge = [&](uint32_t key) {    // weight of the kept with keys >= key
                if (thr == 0) return weight_ge(key);
                return key > thr ? weight_ge(key) : weight_ge(thr + 1) + (double)ties * wthr;
            };
            const double target = (double)tp * kept_ge(0);
            uint32_t a = thr, b = kmax;
            while (a < b) {
                const uint32_t mid = a + (b - a) / 2 + 1;
                if (kept_ge(mid) >= target) a = mid;
                else b = mid - 1;
            }
            const double above = a == 0xffffffffu ? 0.0 : kept_ge(a + 1);
            const double w = weight(unordered(a), inv);
            // equals i = 0, 1, ... stay while above + i w < target
            const double n = w > 0.0 ? ceil((target - above) / w) : (above < target ? 4e18 : 0.0);
            int64_t stay = n < 1.0 ? (a == kmax ? 1 : 0) : n > 4e18 ? (int64_t)4e18 : (int64_t)n;
            if (a != thr || stay < ties) {
                thr = a;
                ties = stay;
            }
        }
        // where the equals that stay end, in index order
        int cut = V;
        if (ties < V) {
            int n = 0;
            for (int i = lo + lane; i < hi; i += 32) n += ordered(value(z, i)) == thr;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
            __syncthreads();
            if (lane == 0) sh.l[warp] = (unsigned long long)n;
            if (threadIdx.x == 0) sh.bl = (unsigned long long)V;
            __syncthreads();
            int64_t before = 0;
            for (int w = 0; w < warp; ++w) before += (int64_t)sh.l[w];
            if (before <= ties && before + n > ties) {       // the first equal that goes is here
                for (int i0 = lo; i0 < hi; i0 += 32) {
                    const bool eq = i0 + lane < hi && ordered(value(z, i0 + lane)) == thr;
                    const uint32_t m = __ballot_sync(0xffffffffu, eq);
                    if (eq && before + __popc(m & ((1u << lane) - 1)) == ties) sh.bl = (unsigned long long)(i0 + lane);
                    before += __popc(m);
                }
            }
            __syncthreads();
            cut = (int)sh.bl;
        }
        auto kept = [&](int i) {                  // weight of token i, 0 when it goes
            const float x = value(z, i);
            const uint32_t key = ordered(x);
            if (key < thr || (key == thr && i >= cut)) return 0.f;
            const float w = weight(x, inv);
            return key == kmax || w >= mp ? w : 0.f;
        };
        float s = 0.f;
        for (int i = lo + lane; i < hi; i += 32) s += kept(i);
        double ws = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
        __syncthreads();
        if (lane == 0) sh.d[warp] = ws;
        if (threadIdx.x == 0) sh.bl = 0;
        __syncthreads();
        double before = 0, total = 0;
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) before += sh.d[w];
            total += sh.d[w];
        }
        const double target = (double)p.u[row] * total;
        // the last warp with anything kept answers when rounding leaves no prefix above the target
        if (ws > 0 && before <= target) {
            int last = -1, found = -1;
            double run = before;
            for (int i0 = lo; i0 < hi && found < 0; i0 += 32) {
                const double w = i0 + lane < hi ? (double)kept(i0 + lane) : 0.0;
                double inc = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                const uint32_t pos = __ballot_sync(0xffffffffu, w > 0.0);
                const uint32_t hit = __ballot_sync(0xffffffffu, w > 0.0 && run + inc > target);
                if (pos) last = i0 + 31 - __clz((int)pos);
                if (hit) found = i0 + __ffs((int)hit) - 1;
                run += __shfl_sync(0xffffffffu, inc, 31);
            }
            // the lowest warp that holds the target wins: it writes its candidate with
            // the highest rank
            if (lane == 0)
                atomicMax(&sh.bl, (unsigned long long)(found >= 0 ? 2 * WARPS - warp : 0) << 32 |
                                      (uint32_t)(found >= 0 ? found : last));
        }
        __syncthreads();
        token = (int)(uint32_t)sh.bl;
    }
    if (threadIdx.x == 0) {
        const float x = value(z, token);
        p.token[row] = token;
        p.logprob[row] = (float)((x == zmax ? 0.0 : (double)x - (double)zmax) - log(all));
    }
}

}  // namespace

caat_status launch_sample_tokens(int64_t B, int64_t V, caat_dtype dt, const void *logits, int64_t ld, const float *u,
                                 const float *temperature, const int32_t *top_k, const float *top_p,
                                 const float *min_p, int32_t *token, float *logprob, cudaStream_t s)
{
    const SampleParams p{logits, ld, V, u, temperature, top_p, min_p, top_k, token, logprob};
    if (dt == CAAT_BF16) sample_kernel<__nv_bfloat16><<<(unsigned)B, THREADS, 0, s>>>(p);
    else sample_kernel<float><<<(unsigned)B, THREADS, 0, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return CAAT_ERR_CUDA;
    note_launch("sample_tokens");
    return CAAT_OK;
}

}  // namespace caat
