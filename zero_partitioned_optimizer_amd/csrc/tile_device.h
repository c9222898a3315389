// tile_device.h -- device code shared by the products on the matrix cores (linear_kernels.hip,
// orth_kernels.hip): tiles of 16-bit operands in LDS, how they are read, and the waits around
// loads that go there from memory.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zk {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));

// Staged tiles hold eight-element chunks (16 bytes), permuted within a row so that
// the lanes that read together meet different banks.
//   outer rows:   [rows][BR], BR reduction elements, chunk c of row o at c ^ (o & 7): the
//                 8 lanes of a 16-byte read hold 8 rows at one c.
//   reduced rows: [BR][cols], chunk c of row r at c ^ perm(r): a transposing read
//                 takes 4 rows x 32 bytes per 16 lanes, and two such groups 8 rows apart
//                 (of 64 columns, even and odd rows have different banks as it is).
template <int COLS>
__device__ __forceinline__ int perm_reduced(int r) {
    return COLS >= 128 ? (r & 3) << 1 | (r >> 3 & 1) << 3 : (r >> 1 & 1) << 2 | (r >> 3 & 1) << 1;
}

template <typename E>
__device__ __forceinline__ uint32_t lds_address(const E* p) {
    typedef __attribute__((address_space(3))) const E lds;
    return (uint32_t)reinterpret_cast<uintptr_t>((lds*)p);
}

// Until at most N of this wave's loads are under way.
template <int N>
__device__ __forceinline__ void loads_landed() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// All waves have come here and their LDS reads and writes are done.
__device__ __forceinline__ void meet_waves() {
    asm volatile("" : : : "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);         // lgkmcnt(0), where the compiler counts it too
    asm volatile("s_barrier" : : : "memory");
}

// The buffer that starts at `from`, the same in all lanes, and reaches `records` bytes:
// with 0 its range check stops all loads (which still count as loads).
__device__ __forceinline__ v4i descriptor(const char* from, int records) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(from);
    return v4i{__builtin_amdgcn_readfirstlane((int)(uint32_t)b), __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32)),
               records, 0x00020000};
}
constexpr int kAllRecords = 0x7FFFFFFF;     // more than a tile's rows reach

// The matrix instruction's operands, of type V (eight 16-bit elements), from a staged tile of
// BR reduction elements: for block i, lane l holds
// outer index o0 + 16 i + (l & 15) and reduction elements 32 s + 8 (l >> 4) .. + 7.
// o0 is a multiple of the outer indices that the wave's blocks cover, a power of
// two, so one byte offset per lane serves all blocks: a constant is added to it,
// or, where a block's chunks lie under the permutation, exchanged into it.
template <int ROWS, bool T, int BR, typename V>
struct TileFragments {
    uint32_t at;
    __device__ __forceinline__ explicit TileFragments(int o0) {
        const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
        if constexpr (T) {
            const int r = 8 * g + (i >> 2), chunk = (o0 >> 3) + ((i & 3) >> 1);
            at = 2 * (r * ROWS + 8 * (chunk ^ perm_reduced<ROWS>(r)) + 4 * (i & 1));
        } else {
            const int o = o0 + i;
            at = 2 * (o * BR + 8 * (g ^ (o & 7)));
        }
    }
    __device__ __forceinline__ V get(uint32_t tile, int i, int s) const {
        typedef __attribute__((address_space(3))) const V lds_v;
        typedef __attribute__((address_space(3))) v4s lds_v4s;
        if constexpr (T) {
            // rows 32 further on have the same permutation
            const uint32_t p = tile + (at ^ (32u * i)) + 2 * 32 * ROWS * s;
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p);
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 2 * 4 * ROWS));
            return __builtin_bit_cast(V, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return *(lds_v*)(tile + (at ^ (64u * s)) + 2 * 16 * BR * i);
        }
    }
};

}  // namespace zk
