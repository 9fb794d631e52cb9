// paged.cuh -- slots of a paged cache: the page of a token, and whether a slot is one.
#pragma once

#include "common.cuh"

namespace dspark {

// division by the page: a shift where it is a power of two
struct Page {
    unsigned size;
    int shift;  // or -1
    __device__ __forceinline__ unsigned of(unsigned t) const { return shift >= 0 ? t >> shift : t / size; }
};

inline Page page_of_size(int size) { return Page{(unsigned)size, (size & (size - 1)) == 0 ? __builtin_ctz((unsigned)size) : -1}; }

// slots that a cache has, at most 2^31: what a slot is compared with
__device__ __forceinline__ unsigned slots_of(int n_pages, int page) { return (unsigned)min((long long)n_pages * page, 0x80000000ll); }

// -1 for a slot that is to be skipped: a negative one, or one beyond the cache, reported
__device__ __forceinline__ int checked_slot(int slot, unsigned slots, int32_t *err) {
    if (slot >= 0 && (unsigned)slot >= slots) {
        set_err(err, DSPARK_ERR_RANGE);
        return -1;
    }
    return slot < 0 ? -1 : slot;
}

}  // namespace dspark
