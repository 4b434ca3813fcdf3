// kvd_pool.h — the pool handle and the host helpers that the entry points share.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/kvd.h"

struct kvd_pool {
    kvd_pool_desc desc;
    uint8_t* mem;
    int32_t* err;       // device error word
    int device;
    int num_sms;
    size_t layer_bytes;
    // host tier (T1): records in pinned host memory (device address) and two HBM staging slots
    uint8_t* host_kv;      // device address of the host records
    uint8_t* host_mem;     // the same records' host address (the prefetch's DMA source)
    uint8_t* staging;
    int64_t host_blocks;
    size_t host_layer_bytes;
    int host_direct;       // no staging: the decode kernel reads host records over the host link
    // mixed pools: precision code of every physical block (device, caller-owned)
    const uint8_t* block_fmt;
    int64_t block_fmt_count;
};

namespace kvd {

inline bool mul_ok(size_t a, size_t b, size_t* out) {
    if (a != 0 && b > SIZE_MAX / a) return false;
    *out = a * b;
    return true;
}

// A kernel runs on the current device, where the pool's memory has to be.
inline kvd_status check_device(int device) {
    int now = 0;
    if (cudaGetDevice(&now) != cudaSuccess) {
        cudaGetLastError();
        return KVD_ERR_CUDA;
    }
    return now == device ? KVD_OK : KVD_ERR_INVALID;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + b_bytes && y < x + a_bytes;
}

// Whether rows share memory: n rows of a_row and b_row bytes, a_pitch and b_pitch apart (slices of one tensor have one
// pitch, and each its own part of it).
inline bool rows_overlap(const void* a, size_t a_row, size_t a_pitch, const void* b, size_t b_row, size_t b_pitch, size_t n) {
    if (!overlap(a, (n - 1) * a_pitch + a_row, b, (n - 1) * b_pitch + b_row)) return false;
    if (a_pitch != b_pitch) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    const size_t ahead = y >= x ? (y - x) % a_pitch : (a_pitch - (x - y) % a_pitch) % a_pitch;   // of b in a's rows
    return ahead < a_row || a_pitch - ahead < b_row;
}

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline kvd_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KVD_OK : KVD_ERR_CUDA; }

inline bool latent_dtype(int32_t t) { return t == KVD_LATENT_BF16 || t == KVD_LATENT_FP8; }
// The entry points of K and V pools do not take a latent pool.
inline bool is_latent(const kvd_pool* pool) { return pool && latent_dtype(pool->desc.kv_dtype); }

}  // namespace kvd
