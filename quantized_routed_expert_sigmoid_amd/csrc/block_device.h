/*
 * block_device.h -- device helpers shared by the operators around the layer:
 * typed loads and stores of activations, the cache's page layout, and the
 * bounds of one sequence of a batch.
 */
#ifndef COLI_BLOCK_DEVICE_H
#define COLI_BLOCK_DEVICE_H

#include "block.h"
#include "device_common.h"

namespace coli {

/* bf16 as its bits: the upper half of an fp32. */
struct bf16 {
    uint16_t u;
};

__device__ __forceinline__ float to_f32(float v)
{
    return v;
}

__device__ __forceinline__ float to_f32(bf16 v)
{
    return __uint_as_float((uint32_t)v.u << 16);
}

/* Two fp32 as bf16, each rounded to nearest even, in one word (lo in its
 * lower half). */
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    b2 p = {(__bf16)lo, (__bf16)hi};
    uint32_t u;
    __builtin_memcpy(&u, &p, 4);
    return u;
}

__device__ __forceinline__ void store1(float* p, float v)
{
    *p = v;
}

__device__ __forceinline__ void store1(bf16* p, float v)
{
    p->u = (uint16_t)pack_bf16(v, 0.0f);
}

__device__ __forceinline__ float4 load4(const float* p)
{
    return *reinterpret_cast<const float4*>(p);
}

__device__ __forceinline__ float4 load4(const bf16* p)
{
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}

__device__ __forceinline__ void store4(float* p, float4 v)
{
    *reinterpret_cast<float4*>(p) = v;
}

__device__ __forceinline__ void store4(bf16* p, float4 v)
{
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

/* The same where only the element's own alignment is known (the memory takes
 * vectors at any address). */
__device__ __forceinline__ float4 load4_any(const float* p)
{
    float4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

__device__ __forceinline__ float4 load4_any(const bf16* p)
{
    uint2 u;
    __builtin_memcpy(&u, p, 8);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}

__device__ __forceinline__ void store4_any(float* p, float4 v)
{
    __builtin_memcpy(p, &v, 16);
}

__device__ __forceinline__ void store4_any(bf16* p, float4 v)
{
    const uint2 u = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    __builtin_memcpy(p, &u, 8);
}

/* LDS address of a byte of shared memory. */
__device__ __forceinline__ uint32_t lds_address(const void* p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

/* Sixteen (four) bytes per lane from base + off into LDS at `to` + 16 (4) lane;
 * base and `to` are uniform, so a loop that moves only these spends no vector
 * instructions on addresses.  Written out because the compiler, which cannot
 * tell the buffers apart, would wait for every such load before the next LDS
 * read; whoever uses it waits himself (arrive_all).  M0 holds the LDS address;
 * no other instruction of these kernels takes M0. */
__device__ __forceinline__ void to_lds(const void* base, uint32_t off, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(off), "s"(base)
                 : "memory");
}

__device__ __forceinline__ void word_to_lds(const void* base, uint32_t off, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(to), "v"(off), "s"(base)
                 : "memory");
}

/* The wave of the workgroup, as a uniform value. */
__device__ __forceinline__ int wave_of()
{
    return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

/* Waits until at most LEFT of this wave's loads are outstanding and its LDS
 * accesses are done, then for the workgroup: past it every wave's earlier loads
 * have arrived, and every wave has left the buffer that is written next. */
template <int LEFT>
__device__ __forceinline__ void arrive_all()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

/* Workgroups go to the eight XCDs in turn; each XCD takes a contiguous run of
 * units (the grid is a multiple of eight), so that what it works on at a time
 * shares its L2. */
__device__ __forceinline__ int64_t xcd_unit()
{
    return (int64_t)(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
}

/* Byte of (token t, dim c) inside a page's keys and values of one head. */
__device__ __forceinline__ int key_byte(int t, int c, int D)
{
    return (t >> 5) * (32 * D) + (c >> 4) * 512 + (t & 31) * 16 + (c & 15);
}

__device__ __forceinline__ int value_byte(int t, int c, int D)
{
    return (t >> 5) * (32 * D) + c * 32 + ((t >> 2) & 1) * 16 + ((t & 31) >> 3) * 4 + (t & 3);
}

/* One sequence of a batch: its packed rows [row0, row0 + q_len), its cached
 * tokens [0, kv_len), the token number of row0 (negative if the rows outnumber
 * the tokens).  Every bound that addresses memory is clamped. */
struct SeqBounds {
    int row0, q_len, kv_len, first;
};

__device__ __forceinline__ SeqBounds seq_bounds(const coli_kv_batch& b, int s)
{
    SeqBounds r;
    const int lo = min(max(b.cu_q[s], 0), b.n_tokens), hi = min(max(b.cu_q[s + 1], 0), b.n_tokens);
    const int64_t cap = (int64_t)b.max_pages * COLI_KV_BLOCK;
    r.row0 = lo;
    r.q_len = max(hi - lo, 0);
    r.kv_len = (int)min((int64_t)max(b.kv_len[s], 0), cap);
    r.first = r.kv_len - r.q_len;
    return r;
}

/* The page of block `blk` of sequence s, or -1 for a missing one. */
__device__ __forceinline__ int page_of(const coli_kv_batch& b, int n_pages, int s, int blk)
{
    const int p = b.page_table[(int64_t)s * b.max_pages + blk];
    return (uint32_t)p < (uint32_t)n_pages ? p : -1;
}

} // namespace coli

#endif
