// Shared by the kernels that write and read the paged 8-bit key-value cache: what a
// launch gets of the cache and the batch, the bounds checks of the device-side
// indices, and the e4m3 conversions.
#pragma once

#include <climits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "caat_internal.h"

namespace caat {

struct PagedKV {
    uint8_t *k, *v;                  // codes [pages][kv_heads][page][dim]
    float *ks, *vs;                  // scales [pages][kv_heads]
    int64_t page_stride;             // elements from one page to the next
    int64_t scale_stride;            // scales from one page to the next
    int64_t pages;
    int kv_heads, page, log2_page, dim;
};

struct PagedBatch {
    const int32_t *table;            // [batch][width], row stride table_stride
    const int32_t *q_start, *kv_len;
    int64_t table_stride, tokens;
    int batch, width, q_max;
};

// The new tokens of one sequence: tokens [t0, t0 + n) of the packed rows at cache
// positions [pos0, pos0 + n).  pos0 < 0 when the cache holds fewer tokens than the
// call brings; the tokens below position 0 then see nothing and are not stored.
struct Seq {
    int64_t t0;
    int n, pos0, len;
    bool ok;
};

// Reads and checks the lengths of sequence b; a sequence whose numbers do not fit
// the buffers is recorded in *err and reported as not ok.
__device__ __forceinline__ Seq load_seq(const PagedBatch &pb, int page, int b, int *err)
{
    Seq s;
    const int a = __ldg(pb.q_start + b), e = __ldg(pb.q_start + b + 1);
    s.len = __ldg(pb.kv_len + b);
    s.t0 = a;
    s.n = e - a;
    s.pos0 = s.len - s.n;
    s.ok = a >= 0 && e >= a && (int64_t)e <= pb.tokens && s.n <= pb.q_max && s.len >= 0 &&
           (int64_t)s.len <= (int64_t)pb.width * page;
    if (!s.ok) {
        *(volatile int *)err = CAAT_ERR_INVALID_ARG;
        s.n = 0;
    }
    return s;
}

constexpr int MAX_RANKED = 1024;     // sequences that by_length takes

// The sequence with the b-th most cached tokens (equals by number).  Blocks that do not all
// run at once start in order, and a long sequence left for the end keeps the others waiting.
// For all threads of a block; shared: MAX_RANKED + 1 words, 16-byte aligned, free again after.
__device__ __forceinline__ int by_length(const PagedBatch &pb, int b, int *shared)
{
    int *mine = shared + MAX_RANKED;
    for (int i = threadIdx.x; i < MAX_RANKED; i += blockDim.x) shared[i] = i < pb.batch ? __ldg(pb.kv_len + i) : INT_MIN;
    __syncthreads();
    for (int i = threadIdx.x; i < pb.batch; i += blockDim.x) {
        const int n = shared[i];
        int before = 0;
        for (int j = 0; j < pb.batch; j += 4) {
            const int4 o = *reinterpret_cast<const int4 *>(shared + j);
            before += (o.x > n || (o.x == n && j < i)) + (o.y > n || (o.y == n && j + 1 < i)) +
                      (o.z > n || (o.z == n && j + 2 < i)) + (o.w > n || (o.w == n && j + 3 < i));
        }
        if (before == b) *mine = i;
    }
    __syncthreads();
    b = *mine;
    __syncthreads();
    return b;
}

// a page number of the table, or -1 (recorded in *err) when the cache has no such page
__device__ __forceinline__ int64_t checked_page(int id, const PagedKV &kv, int *err)
{
    if (id >= 0 && (int64_t)id < kv.pages) return id;
    *(volatile int *)err = CAAT_ERR_INVALID_ARG;
    return -1;
}

// Four e4m3 codes (low byte first) -> two pairs of f16, exact.  (The conversion
// functions of cuda_fp8.h go through 16-bit halves: 3 to 4 more instructions a pair.)
__device__ __forceinline__ void e4m3x4_f16(uint32_t four, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}

// four floats -> four e4m3 codes, nearest even, magnitudes above 448 to 448, NaN kept
__device__ __forceinline__ uint32_t f32x4_e4m3(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\tmov.b32 %0, {x, y};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// two floats -> two f16 in one register, nearest even
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// many rows, bf16 (paged_attn_tc.cu)
caat_status launch_paged_attention_tile(const PagedKV &kv, const PagedBatch &pb, int heads, const void *q, int64_t q_st,
                                        int64_t q_sk, int64_t q_sg, float scale, int window, int sinks, void *o,
                                        int64_t o_st, int64_t o_sh, cudaStream_t s);

// Launch attributes of these kernels: a cluster of `cluster` blocks (1: none), and a
// programmatic dependent of the previous launch unless CAAT_PDL=0 (the kernel waits for
// that launch before its first access).  Returns how many attributes it set.
unsigned serve_attrs(cudaLaunchAttribute (&attr)[2], int cluster);

int *serve_error_word();             // device address of these kernels' error word, or null
caat_status read_and_clear_serve_error();

}  // namespace caat
